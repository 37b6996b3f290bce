// Multi-head decay attention for any head size and type: causal linear attention whose
// (D, D) state of each head decays by e^{-w} per token,
//
//   out_t = scale_intra * sum_{s <= t} e^{-w (t-s)} (q_t . k_s) v_s
//         + scale_inter * e^{-w (t+e0)} q_t X_in,
//   X_out = e^{-w n} X_in + scale_upd * sum_s e^{-w (n-1-s+1-e0)} k_s^T v_s     (n tokens)
//
// One operator serves the forward pass and, with its arguments exchanged, the
// three token gradients: with g = dL/dout, S the states of the forward pass
// and G_t = dL/dS_t,
//   gq = the operator on (g, v, k) with X = S^T,
//   gk = the operator on (v, g, q) in reversed time with X = G^T,
//   gv = the operator on (k, q, g) in reversed time with X = G.
// Reversed time processes token n-1 first; its state is handed over already
// decayed (e0 = 0), so the last X_out is the gradient of the initial state.
//
// A launch runs up to three such problems, the same head's in adjacent CTAs
// (they share their inputs in L2).  Long sequences are cut into segments: a first launch forms
// each segment's own X_out from X_in = 0 (out == nullptr), decay_chain_kernel
// chains them, and the main launch starts every segment from its own X_in.
//
// This file holds the kernel for any head size, the chain and the single-token
// step; decay_attn_tc.cuh, decay_attn_tc64.cuh and decay_attn_tcf.cuh are the
// same operator on the fifth-generation tensor cores.
#pragma once

#include "common.cuh"
#include "passes.cuh"

namespace vrwkv {
namespace decay {

struct Problem {
    const char* q;          // (B, T, H*D) rows of ldq elements, batch stride T*ldq; unused without out
    const char* k;
    const char* v;
    char* out;              // dense (B, T, H*D); nullptr: the state alone
    long long ldq, ldk, ldv;
    const float* x_in;      // states [(b*H + h)*nseg + seg][D][D], or nullptr for zeros
    float* x_out;           // the same layout, or nullptr
    int x_in_t, x_out_t;    // stored transposed: [v channel][k channel]
    int reverse;
    float scale_intra, scale_inter, scale_upd;
    int skip;               // without out: a segment whose own state is not needed, or -1
};

struct Params {
    Problem pr[3];
    const float* w;         // (H)
    const int* lengths;     // (B) or nullptr
    int B, T, H, D;
    int S;                  // a state is (S, S): D, but for spread heads (decay_pack.cuh)
    int seg_tokens, nseg;   // tokens of a segment, segments of a sequence
    int nprob;              // problems of this launch; CTA x: problem x % nprob of segment x / nprob
    int vec;                // rows can be read and written 4 elements at a time
};

// Valid tokens of a sequence, and of segment `seg` of it.
__device__ __forceinline__ int seq_tokens(const int* lengths, int b, int T) {
    if (!lengths) return T;
    const int n = __ldg(lengths + b);
    return n < 0 ? 0 : (n > T ? T : n);
}
__device__ __forceinline__ int seg_count(int n, int seg, int seg_tokens) {
    const int r = n - seg * seg_tokens;
    return r < 0 ? 0 : (r > seg_tokens ? seg_tokens : r);
}

// e^{-w n} as 2^{n c}, c = -w log2 e held as a float pair: the exponent is
// rounded once, so the relative error of the power stays below |w n| 2^-24 plus
// exp2f's own 2 units in the last place (2^-22).  Above 2^24 tokens n is rounded
// too: |w n| 2^-23.
struct DecayBase {
    float hi, lo;
};
__device__ __forceinline__ DecayBase decay_base(float w) {
    constexpr float L = 1.44269502162933349609375f, Llo = 1.92596299112661748e-8f;  // log2 e = L + Llo
    DecayBase c;
    c.hi = -w * L;
    c.lo = fmaf(-w, L, -c.hi) - w * Llo;
    return c;
}
__device__ __forceinline__ float decay_pow(const DecayBase& c, int n) {
    if (n == 0) return 1.0f;
    const float f = (float)n, x = f * c.hi;
    return exp2f(fabsf(x) < 1e30f ? x + (fmaf(f, c.hi, -x) + f * c.lo) : x);  // an infinite w has no low part
}
__device__ __forceinline__ float decay_pow(float w, int n) { return decay_pow(decay_base(w), n); }

template <typename IO>
__device__ __forceinline__ float4 ld4(const char* p) {
    if (sizeof(IO) == 4) return *reinterpret_cast<const float4*>(p);
    const uint2 r = *reinterpret_cast<const uint2*>(p);
    return make_float4(__uint_as_float(r.x << 16), __uint_as_float(r.x & 0xffff0000u),
                       __uint_as_float(r.y << 16), __uint_as_float(r.y & 0xffff0000u));
}
// ---------------------------------------------------------------------------
// The operator for any D <= DP (zero-padded) and either storage type, in
// chunks of 32 tokens: inside a chunk the products q.k weighted by the decays,
// across chunks the state X.  The products run on the warp-level tensor cores
// as tf32 (m16n8k8): a float32 operand is split into a tf32 value and the
// remainder as another, hi hi + hi lo + lo hi (what is left out is 2^-22 of a
// product); a bfloat16 operand is a tf32 value as it stands.  The tensor cores
// truncate when they add, so a chain is two instructions' sums long (16
// products) and joins the float32 sums on the FP32 pipes.
// Why not the FP32 pipes: fed from shared memory with 8 products an operand
// they measured a quarter of their rate (float32 B=8 T=1024 16 heads of 64:
// 223 us), while a fragment of m16n8k8 serves 16 products and more (183 us).
// Bound by those instructions: float32 21 x 256, 12 heads of 128, takes 176 us, a
// little over half of the 489 products a clock and SM that tf32 measures here.  bfloat16
// heads of an odd width also load by element: 3 x 7518, 15 heads of 89: 1.75 ms.
//
// Warps: the token tiles of 16 rows (2), times 2 (DP = 128: 4) parts of the v
// channels.  X^T is kept in registers, 16 v channels a warp (at DP = 32 with
// half of the k channels), and copied to shared memory for q X.  The next
// chunk's tiles are on their way in registers while one is worked on.  Sums over
// tokens take them in the order 2t, 2t + 1 of a group of 8 that the
// accumulator layout has, so P goes from accumulators to operands in place;
// with rows of DP + 4 floats every fragment load is free of bank conflicts.
// ---------------------------------------------------------------------------
template <int DP>
struct Cfg {
    static constexpr int C = 32;                            // tokens of a chunk
    static constexpr int LD = DP + 4;
    static constexpr int kWarps = DP == 128 ? 8 : 4;
    static constexpr int kThreads = 32 * kWarps;
    static constexpr int NT = DP / 8 / (kWarps / 2);        // 8-channel tiles of a warp's output rows
    static constexpr int NL = 3 * C * (DP / 4) / kThreads;  // float4s a thread loads
    static constexpr int UM = DP / 16;                      // 16-channel tiles of X^T's rows
    static constexpr int UT = DP / 8 / (kWarps / UM);       // 8-channel tiles of a warp's part of X^T
    static constexpr int kSmemFloats = 3 * C * LD + DP * LD + C + 4;
    static constexpr int kResident = DP == 128 ? 1 : 3;     // CTAs of an SM, by registers
};

// A float32 operand as tf32 values, of which the tensor core reads the upper 19
// bits: hi, then lo, the remainder.  Before bits are cut off a value is multiplied,
// which adds half a step of them: to hi 0.72 * 2^-11 of it, half a step on average
// over a binade, so that lo leans to neither side (the product of two remainders is
// left out; with 2^-11 it is 5e-8 of a product, always the same way); to lo 2^-11.
// hi is off by at most 2^-10.6, lo by 2^-11 of itself: a product of two operands by
// 2^-20.  Multiplications, since they keep a NaN (the GPU's own has all bits set:
// adding to them wraps it to 0), and towards zero, since a finite value then stays
// finite.  What an infinity leaves is NaN.
// Measured, outputs of 2 x 200, heads of 128, against 64 bits: 2.85e-7 of the norm;
// half steps added to the bits, at the same time, 2.80e-7.  To nearest by the
// exponent's power of two, 2.80e-7: 21 x 256, 12 heads of 128 194 us in place of 176.
template <bool EXACT>
__device__ __forceinline__ void tf32_split(float x, uint32_t& hi, uint32_t& lo) {
    if (EXACT) {
        hi = __float_as_uint(x);
        lo = 0u;
    } else {
        hi = __float_as_uint(__fmul_rz(x, 1.0003515625f)) & 0xffffe000u;
        lo = __float_as_uint((x - __uint_as_float(hi)) * 1.00048828125f);
    }
}
__device__ __forceinline__ void mma_tf32(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// An A operand of two steps (16 summed indices), and a product with a B operand
// of two steps added to c.  AX, BX: the operand is exactly tf32.
struct FragA {
    uint32_t hi[2][4], lo[2][4];
    template <bool AX>
    __device__ __forceinline__ void set(int step, float a0, float a1, float a2, float a3) {
        tf32_split<AX>(a0, hi[step][0], lo[step][0]);
        tf32_split<AX>(a1, hi[step][1], lo[step][1]);
        tf32_split<AX>(a2, hi[step][2], lo[step][2]);
        tf32_split<AX>(a3, hi[step][3], lo[step][3]);
    }
};
// N tiles at a time, instruction by instruction over the tiles: a tile's own
// instructions wait for one another.  load(i, h): the tile's B values, two
// steps of two.
template <bool AX, bool BX, int N, typename Load>
__device__ __forceinline__ void mma_tiles(float (*c)[4], const FragA& a, Load load) {
    float t[N][4];
    uint32_t h[N][4], l[N][4];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        float b[4];
        load(i, b);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            tf32_split<BX>(b[e], h[i][e], l[i][e]);
            t[i][e] = 0.f;
        }
    }
#pragma unroll
    for (int step = 0; step < 2; ++step) {
        if (!AX) {
#pragma unroll
            for (int i = 0; i < N; ++i) mma_tf32(t[i], a.lo[step], h[i][2 * step], h[i][2 * step + 1]);
        }
        if (!BX) {
#pragma unroll
            for (int i = 0; i < N; ++i) mma_tf32(t[i], a.hi[step], l[i][2 * step], l[i][2 * step + 1]);
        }
#pragma unroll
        for (int i = 0; i < N; ++i) mma_tf32(t[i], a.hi[step], h[i][2 * step], h[i][2 * step + 1]);
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) c[i][e] += t[i][e];
}

template <typename IO, int DP>
__global__ void __launch_bounds__(Cfg<DP>::kThreads, Cfg<DP>::kResident)
    decay_attn_kernel(const __grid_constant__ Params p) {
    using F = Cfg<DP>;
    constexpr int C = F::C, LD = F::LD, NT = F::NT, UT = F::UT, UM = F::UM, kThreads = F::kThreads;
    constexpr bool IX = sizeof(IO) == 2;     // inputs are exactly tf32
    constexpr int es = sizeof(IO);
    extern __shared__ __align__(16) float sm[];
    float* sq = sm;                          // [token][LD]
    float* sk = sq + C * LD;
    float* sv = sk + C * LD;
    float* sx = sv + C * LD;                 // X^T [v channel][LD]
    float* pw = sx + DP * LD;                // e^{-w n}, n = 0 .. C
    const Problem& pr = p.pr[blockIdx.x % p.nprob];
    const int hid = blockIdx.x / p.nprob, seg = hid % p.nseg, bh = hid / p.nseg, b = bh / p.H, h = bh % p.H;
    next_pass();
    if (!pr.out && seg == pr.skip) return;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int D = p.D;
    const float w = __ldg(p.w + h);
    const int n_seq = seq_tokens(p.lengths, b, p.T);
    const int t0 = seg * p.seg_tokens;
    const int n = seg_count(n_seq, seg, p.seg_tokens);               // valid tokens of this segment
    const int t_end = min(t0 + p.seg_tokens, p.T) - t0;              // its rows of the tensors
    const int rev = pr.reverse, e0 = rev ? 0 : 1;
    const size_t xo = ((size_t)bh * p.nseg + seg) * (size_t)D * D;
    const bool want_out = pr.out != nullptr;
    const size_t row0 = (size_t)b * p.T + t0;
    const size_t col0 = (size_t)h * D;
    const int nchunk = (n + C - 1) / C;

    if (tid <= C) pw[tid] = decay_pow(w, tid);
    // this warp's rows of a chunk and first v channel of its output; its v and first k channel of X^T
    const int mt = warp % 2, c0 = (warp / 2) * NT * 8;
    const int um = (warp % UM) * 16, u0 = (warp / UM) * UT * 8;
    last_pass();
    float X[UT][4];                          // rows um + g, um + g + 8, columns u0 + 8 i + 2 t, + 1
#pragma unroll
    for (int i = 0; i < UT; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int dv = um + g + (e >> 1) * 8, dk = u0 + 8 * i + 2 * t + (e & 1);
            X[i][e] = pr.x_in && dv < D && dk < D
                          ? __ldcg(pr.x_in + xo + (pr.x_in_t ? (size_t)dv * D + dk : (size_t)dk * D + dv)) : 0.f;
        }

    // a thread's part of a chunk's q, k, v tiles, zero past the chunk's tokens and the head's channels
    constexpr int NL = F::NL, kPer = NL / 3;
    float4 next[NL];
    auto fetch = [&](int ci) {
        const int a = (rev ? nchunk - 1 - ci : ci) * C, m = min(C, n - a);
#pragma unroll
        for (int i = 0; i < NL; ++i) {
            const int which = i / kPer, y = (i % kPer) * kThreads + tid, r = y / (DP / 4), c = 4 * (y % (DP / 4));
            next[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r < m && c < D && (which != 0 || want_out)) {
                const char* base = which == 0 ? pr.q : which == 1 ? pr.k : pr.v;
                const long long ld = which == 0 ? pr.ldq : which == 1 ? pr.ldk : pr.ldv;
                const char* src = base + ((row0 + a + r) * (size_t)ld + col0 + c) * es;
                if (p.vec) {
                    next[i] = ld4<IO>(src);
                } else {
                    next[i].x = Io<IO>::ld1(src);
                    if (c + 1 < D) next[i].y = Io<IO>::ld1(src + es);
                    if (c + 2 < D) next[i].z = Io<IO>::ld1(src + 2 * es);
                    if (c + 3 < D) next[i].w = Io<IO>::ld1(src + 3 * es);
                }
            }
        }
    };
    if (nchunk > 0) fetch(0);

    for (int ci = 0; ci < nchunk; ++ci) {
        const int a = (rev ? nchunk - 1 - ci : ci) * C;              // first token of the chunk, in the segment
        const int m = min(C, n - a);                                 // its tokens
        const bool with_x = ci > 0 || pr.x_in != nullptr, update = ci + 1 < nchunk || pr.x_out != nullptr;
        __syncthreads();                                             // the previous chunk's readers are done
#pragma unroll
        for (int i = 0; i < NL; ++i) {
            const int which = i / kPer, y = (i % kPer) * kThreads + tid;
            *reinterpret_cast<float4*>((which == 0 ? sq : which == 1 ? sk : sv) + y / (DP / 4) * LD + 4 * (y % (DP / 4))) =
                next[i];
        }
        if (want_out && with_x) {
#pragma unroll
            for (int i = 0; i < UT; ++i)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    *reinterpret_cast<float2*>(sx + (um + g + 8 * e) * LD + u0 + 8 * i + 2 * t) = f2(X[i][2 * e], X[i][2 * e + 1]);
        }
        __syncthreads();
        if (ci + 1 < nchunk) fetch(ci + 1);
        if (want_out && 16 * mt < m) {
            // O = q X and A = q k^T share q's fragments.  Of A, the tiles in these rows' past.
            float o[NT][4], A[4][4];
#pragma unroll
            for (int i = 0; i < NT; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) A[i][0] = A[i][1] = A[i][2] = A[i][3] = 0.f;
            const float* qr = sq + (16 * mt + g) * LD + t;
#pragma unroll 2
            for (int k = 0; k < DP; k += 16) {
                FragA fq;
#pragma unroll
                for (int s = 0; s < 2; ++s)
                    fq.set<IX>(s, qr[k + 8 * s], qr[8 * LD + k + 8 * s], qr[k + 8 * s + 4], qr[8 * LD + k + 8 * s + 4]);
                if (with_x)
                    mma_tiles<IX, false, NT>(o, fq, [&](int i, float (&v)[4]) {
                        const float* x = sx + (c0 + 8 * i + g) * LD + k + t;
                        v[0] = x[0], v[1] = x[4], v[2] = x[8], v[3] = x[12];
                    });
                auto keys = [&](int i, float (&v)[4]) {
                    const float* x = sk + (8 * i + g) * LD + k + t;
                    v[0] = x[0], v[1] = x[4], v[2] = x[8], v[3] = x[12];
                };
                // the upper rows reach the near half of the columns only
                if (mt == (rev ? 1 : 0)) {
                    if (rev) mma_tiles<IX, IX, 2>(A + 2, fq, [&](int i, float (&v)[4]) { keys(i + 2, v); });
                    else mma_tiles<IX, IX, 2>(A, fq, keys);
                } else {
                    mma_tiles<IX, IX, 4>(A, fq, keys);
                }
            }
            if (with_x) {
                float f[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int row = 16 * mt + g + 8 * e;
                    f[e] = pw[max(rev ? m - 1 - row : row, 0) + e0] * pr.scale_inter;
                }
#pragma unroll
                for (int i = 0; i < NT; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[i][e] *= f[e >> 1];
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int r = 16 * mt + g + 8 * (e >> 1), c = 8 * i + 2 * t + (e & 1), d = rev ? c - r : r - c;
                    A[i][e] = d < 0 ? 0.f : A[i][e] * pw[d] * pr.scale_intra;
                }
            }
            // O += P v, two tiles of P (16 tokens) at a time
#pragma unroll
            for (int i = 0; i < 4; i += 2) {
                if (rev ? i < 2 * mt : i > 2 * mt) continue;         // all in these rows' future
                FragA fp;
#pragma unroll
                for (int s = 0; s < 2; ++s) fp.set<false>(s, A[i + s][0], A[i + s][2], A[i + s][1], A[i + s][3]);
                mma_tiles<false, IX, NT>(o, fp, [&](int j, float (&v)[4]) {
                    const float* x = sv + (8 * i + 2 * t) * LD + c0 + g + 8 * j;
                    v[0] = x[0], v[1] = x[LD], v[2] = x[8 * LD], v[3] = x[9 * LD];
                });
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int row = 16 * mt + g + 8 * e;
                if (row >= m) continue;
                char* dst = pr.out + ((row0 + a + row) * (size_t)p.H * D + col0) * es;
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    const int c = c0 + 8 * j + 2 * t;
                    if (p.vec) {  // D % 4 == 0: pairs are whole
                        if (c < D) Io<IO>::st_pair(dst + c * es, f2(o[j][2 * e], o[j][2 * e + 1]));
                    } else {
                        if (c < D) Io<IO>::st1(dst + c * es, o[j][2 * e]);
                        if (c + 1 < D) Io<IO>::st1(dst + (c + 1) * es, o[j][2 * e + 1]);
                    }
                }
            }
        }
        if (!update) break;                                          // no one reads the last state
        // X^T <- e^{-w m} X^T + sum_s f_s v_s^T k_s, 16 tokens at a time
        float U[UT][4];
#pragma unroll
        for (int i = 0; i < UT; ++i) U[i][0] = U[i][1] = U[i][2] = U[i][3] = 0.f;
#pragma unroll
        for (int s0 = 0; s0 < C; s0 += 16) {
            if (s0 >= m) break;
            FragA fv;
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const int r = s0 + 8 * s + 2 * t;                    // tokens r and r + 1
                const float f0 = r < m ? pw[rev ? r + 1 : m - 1 - r] * pr.scale_upd : 0.f;
                const float f1 = r + 1 < m ? pw[rev ? r + 2 : m - 2 - r] * pr.scale_upd : 0.f;
                const float* vv = sv + r * LD + um + g;
                fv.set<false>(s, vv[0] * f0, vv[8] * f0, vv[LD] * f1, vv[LD + 8] * f1);
            }
            constexpr int UB = UT < 4 ? UT : 4;
#pragma unroll
            for (int j = 0; j < UT; j += UB)
                mma_tiles<false, IX, UB>(U + j, fv, [&](int i, float (&v)[4]) {
                    const float* x = sk + (s0 + 2 * t) * LD + u0 + g + 8 * (i + j);
                    v[0] = x[0], v[1] = x[LD], v[2] = x[8 * LD], v[3] = x[9 * LD];
                });
        }
        const float fx = pw[m];
#pragma unroll
        for (int i = 0; i < UT; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) X[i][e] = fmaf(fx, X[i][e], U[i][e]);
    }

    if (pr.x_out) {
#pragma unroll
        for (int i = 0; i < UT; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int dv = um + g + (e >> 1) * 8, dk = u0 + 8 * i + 2 * t + (e & 1);
                if (dv < D && dk < D) pr.x_out[xo + (pr.x_out_t ? (size_t)dv * D + dk : (size_t)dk * D + dv)] = X[i][e];
            }
    }
    if (want_out) {  // rows past the sequence's end
        for (int x = tid; x < (t_end - n) * D; x += kThreads)
            Io<IO>::st1(pr.out + ((row0 + n + x / D) * (size_t)p.H * D + col0 + x % D) * es, 0.f);
    }
}

// ---------------------------------------------------------------------------
// Chain the segments' own states: on entry u[seg] is segment seg's X_out from
// X_in = 0; on return it is the segment's X_in, and x_last, if given, the
// state after the last segment (whose own state is read for it alone).  Bound by
// latency (8 heads of 128, 16 segments: 8.4 MB, two round trips of eight reads
// each; one read at a time made the whole call 20 us longer).  The
// segments in order, last to first in reversed time, a thread 4 (or 1) of a
// head's elements; the loads of the next segments do not wait for the chain.
// ---------------------------------------------------------------------------
struct ChainProblem {
    float* u;             // [(b*H + h)*nseg + seg][D*D]
    const float* x0;      // (B, H, D, D) or nullptr
    float* x_last;        // (B, H, D, D) or nullptr
    int reverse;
};
struct ChainParams {
    ChainProblem pr[2];
    const float* w;
    const int* lengths;
    int T, H, dd;         // dd = D * D
    int seg_tokens, nseg;
};

template <typename V>
__device__ __forceinline__ void chain(const ChainParams& p, const ChainProblem& pr, int bh, int i, DecayBase w, int n_seq) {
    constexpr int N = sizeof(V) / 4;
    constexpr int kAhead = 8;
    V x, own[kAhead];
    float* xs = reinterpret_cast<float*>(&x);
#pragma unroll
    for (int e = 0; e < N; ++e) xs[e] = pr.x0 ? __ldg(pr.x0 + (size_t)bh * p.dd + i + e) : 0.f;
    float* u = pr.u + (size_t)bh * p.nseg * p.dd + i;
    const int step = pr.reverse ? -1 : 1;
    int seg = pr.reverse ? p.nseg - 1 : 0;
    const int reads = p.nseg - (pr.x_last ? 0 : 1);
    // eight segments are read before any is written
    for (int s0 = 0; s0 < reads; s0 += kAhead) {
#pragma unroll
        for (int s = 0; s < kAhead; ++s)
            if (s0 + s < reads) own[s] = __ldcg(reinterpret_cast<const V*>(u + (size_t)(seg + s * step) * p.dd));
#pragma unroll
        for (int s = 0; s < kAhead; ++s) {
            if (s0 + s >= reads) break;
            *reinterpret_cast<V*>(u + (size_t)seg * p.dd) = x;
            const float f = decay_pow(w, seg_count(n_seq, seg, p.seg_tokens));
            const float* os = reinterpret_cast<const float*>(&own[s]);
#pragma unroll
            for (int e = 0; e < N; ++e) xs[e] = fmaf(f, xs[e], os[e]);
            seg += step;
        }
    }
    if (reads < p.nseg) {
        *reinterpret_cast<V*>(u + (size_t)seg * p.dd) = x;
    } else {
#pragma unroll
        for (int e = 0; e < N; ++e) pr.x_last[(size_t)bh * p.dd + i + e] = xs[e];
    }
}

__global__ void __launch_bounds__(256) decay_chain_kernel(const ChainParams p) {
    next_pass();
    const ChainProblem& pr = p.pr[blockIdx.z];
    const int bh = blockIdx.x, b = bh / p.H, h = bh % p.H;
    const int x = blockIdx.y * 256 + threadIdx.x;
    const DecayBase w = decay_base(__ldg(p.w + h));
    const int n_seq = seq_tokens(p.lengths, b, p.T);
    last_pass();
    if (p.dd % 4 == 0) {
        if (4 * x < p.dd) chain<float4>(p, pr, bh, 4 * x, w, n_seq);
    } else if (x < p.dd) {
        chain<float>(p, pr, bh, x, w, n_seq);
    }
}

// ---------------------------------------------------------------------------
// One token per sequence on a pool of states (N, H, D, D), updated in place:
//   S = e^{-w} S + k^T v,  out = scale q S.
// Bound by the state's bytes (read and written once).  A CTA takes a slab of
// 32 columns of one head's state: independent of the other slabs, 128-byte
// rows, and enough CTAs at batch 1.  Thread (r, c4): rows r, r + RT, .. and
// the 4 columns c4, NP passes over the rows; the columns' partial sums over the
// rows meet in shared memory.  Measured at 256 sequences of 16 heads of 64:
// 27.1 us for 134 MB (4.95 TB/s; 31.4 us with loads for 128 channels, masked, and
// no streaming hints).  One sequence of 12 heads: 2.4 us in a graph,
// launch-bound.
// ---------------------------------------------------------------------------
struct StepParams {
    const char* q;          // (B, H*D), row strides in elements
    const char* k;
    const char* v;
    char* out;              // dense (B, H*D)
    long long ldq, ldk, ldv;
    const float* w;
    float* state;           // (N, H, D, D)
    const int* slots;       // (B) or nullptr: row b has slot b
    int B, N, H, D;
    float scale;
    int vec;                // D % 4 == 0 and 16-byte-aligned states
    unsigned int* err;
};

constexpr unsigned kErrSlot = 16u;
constexpr int kStepThreads = 128;
constexpr int kStepCols = 32;                       // columns of a CTA
constexpr int kStepRows = kStepThreads / (kStepCols / 4);  // rows of one pass
constexpr int kStepMaxD = 128;

template <typename IO, int NP>
__global__ void __launch_bounds__(kStepThreads) decay_step_kernel(const StepParams p) {
    __shared__ float sq[kStepMaxD], sk[kStepMaxD];
    __shared__ float4 part[kStepRows / 4][kStepCols / 4];  // one row per warp
    const int b = blockIdx.x, h = blockIdx.y, slab = blockIdx.z, tid = threadIdx.x, D = p.D;
    const int c4 = tid % (kStepCols / 4), r0 = tid / (kStepCols / 4);
    // columns j, j + dj, ..: four in a row as a vector, else 8 apart, so that 8
    // lanes read 8 in a row
    const int dj = p.vec ? 1 : kStepCols / 4, j = slab * kStepCols + (p.vec ? 4 * c4 : c4);
    const int slot = p.slots ? __ldg(p.slots + b) : b;
    const bool in_range = slot >= 0 && slot < p.N;
    constexpr int es = sizeof(IO);
    float* S = p.state + ((size_t)(in_range ? slot : 0) * p.H + h) * D * D;

    float4 x[NP];
#pragma unroll
    for (int m = 0; m < NP; ++m) {
        const int i = r0 + kStepRows * m;
        x[m] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (in_range && i < D && j < D) {
            const float* s = S + (size_t)i * D + j;
            if (p.vec) {
                x[m] = __ldcs(reinterpret_cast<const float4*>(s));
            } else {
                x[m].x = s[0];
                if (j + dj < D) x[m].y = s[dj];
                if (j + 2 * dj < D) x[m].z = s[2 * dj];
                if (j + 3 * dj < D) x[m].w = s[3 * dj];
            }
        }
    }
    for (int i = tid; i < D; i += kStepThreads) {
        sq[i] = Io<IO>::ld1(p.q + ((size_t)b * p.ldq + (size_t)h * D + i) * es) * p.scale;
        sk[i] = Io<IO>::ld1(p.k + ((size_t)b * p.ldk + (size_t)h * D + i) * es);
    }
    float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (j + e * dj < D) v[e] = Io<IO>::ld1(p.v + ((size_t)b * p.ldv + (size_t)h * D + j + e * dj) * es);
    const float lam = decay_pow(__ldg(p.w + h), 1);
    // a slot that an earlier row names belongs to that row
    bool taken = false;
    if (p.slots)
        for (int i = tid; i < b; i += kStepThreads) taken |= __ldg(p.slots + i) == slot;
    taken = __syncthreads_or(taken && slot >= 0);
    const bool live = in_range && !taken;
    if (tid == 0 && (taken || slot >= p.N)) atomicOr(p.err, kErrSlot);

    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    if (live) {
#pragma unroll
        for (int m = 0; m < NP; ++m) {
            const int i = r0 + kStepRows * m;
            if (i >= D) break;
            const float kk = sk[i], qq = sq[i];
            x[m].x = fmaf(lam, x[m].x, kk * v[0]);
            x[m].y = fmaf(lam, x[m].y, kk * v[1]);
            x[m].z = fmaf(lam, x[m].z, kk * v[2]);
            x[m].w = fmaf(lam, x[m].w, kk * v[3]);
            o.x = fmaf(qq, x[m].x, o.x);
            o.y = fmaf(qq, x[m].y, o.y);
            o.z = fmaf(qq, x[m].z, o.z);
            o.w = fmaf(qq, x[m].w, o.w);
            if (j < D) {
                float* s = S + (size_t)i * D + j;
                if (p.vec) {
                    __stcs(reinterpret_cast<float4*>(s), x[m]);
                } else {
                    s[0] = x[m].x;
                    if (j + dj < D) s[dj] = x[m].y;
                    if (j + 2 * dj < D) s[2 * dj] = x[m].z;
                    if (j + 3 * dj < D) s[3 * dj] = x[m].w;
                }
            }
        }
    }
    // sum over the rows: the warp's 4 row groups, then the 4 warps
#pragma unroll
    for (int d = 8; d <= 16; d <<= 1) {
        o.x += __shfl_xor_sync(0xffffffffu, o.x, d);
        o.y += __shfl_xor_sync(0xffffffffu, o.y, d);
        o.z += __shfl_xor_sync(0xffffffffu, o.z, d);
        o.w += __shfl_xor_sync(0xffffffffu, o.w, d);
    }
    if ((tid & 31) < kStepCols / 4) part[tid >> 5][c4] = o;
    __syncthreads();
    if (tid < kStepCols) {
        const int jj = slab * kStepCols + (p.vec ? tid : tid / 4 + tid % 4 * (kStepCols / 4));
        float s = 0.f;
#pragma unroll
        for (int q = 0; q < kStepRows / 4; ++q) s += reinterpret_cast<const float*>(&part[q][0])[tid];
        if (jj < D) Io<IO>::st1(p.out + ((size_t)b * p.H * D + (size_t)h * D + jj) * es, s);
    }
}

}  // namespace decay
}  // namespace vrwkv
