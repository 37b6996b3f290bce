// Multi-head decay attention on the FP32 pipes: causal linear attention whose
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
#pragma once

#include "common.cuh"

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
};

struct Params {
    Problem pr[3];
    const float* w;         // (H)
    const int* lengths;     // (B) or nullptr
    int B, T, H, D;
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
// rounded once, so the relative error of the power stays below |w n| 2^-24.
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
template <typename IO>
__device__ __forceinline__ void st4(char* p, float4 v) {
    if (sizeof(IO) == 4) {
        *reinterpret_cast<float4*>(p) = v;
    } else {
        const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
        *reinterpret_cast<uint2*>(p) =
            make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
    }
}

__device__ __forceinline__ void fma4(float4& a, float s, const float4& b) {
    const float2 lo = fma2(f2(s), f2(b.x, b.y), f2(a.x, a.y)), hi = fma2(f2(s), f2(b.z, b.w), f2(a.z, a.w));
    a = make_float4(lo.x, lo.y, hi.x, hi.y);
}
__device__ __forceinline__ float at4(const float4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// The operator for any D <= DP (zero-padded) and either storage type, in
// chunks of 32 tokens: inside a chunk the (32 x 32) products q.k weighted by
// the decays, across chunks the state.  A CTA takes 32 of the v channels (the
// products with them and their columns of the state are independent of the
// others; the products q.k are formed again in each of a head's DP / 32 CTAs,
// at DP = 64 a sixth of the work, for twice the CTAs).  Thread (ty, tx) owns
// output columns 4 tx .. +3 of rows ty and ty + 16, and the state's rows of
// its ty at the same columns, in registers; a copy of the state in shared
// memory feeds the products with q.  The next chunk's tiles are in registers
// while one is worked on.  Bound by FP32 issue and shared-memory loads.
constexpr int kFpThreads = 128;
constexpr int kFpCols = 32;

template <int DP>
struct Cfg {
    static constexpr int C = 32;                            // tokens of a chunk
    static constexpr int LD = DP + 4;                       // padded row: rows 1 apart are 4 banks apart
    static constexpr int LV = kFpCols + 4;
    static constexpr int SR = DP / 16;                      // state rows of a thread
    static constexpr int SG = SR < 4 ? SR : 4;              // of which SG are adjacent
    static constexpr int NL = (2 * C * (DP / 4) + C * (kFpCols / 4)) / kFpThreads;  // float4s a thread loads
    static constexpr int kSmemFloats = 2 * C * LD + C * LV + DP * LV + C * LV + C + 4;
    static constexpr int kResident = DP == 128 ? 3 : DP == 64 ? 5 : 6;  // CTAs of an SM
};

template <typename IO, int DP>
__global__ void __launch_bounds__(kFpThreads, Cfg<DP>::kResident)
    decay_attn_kernel(const __grid_constant__ Params p) {
    using F = Cfg<DP>;
    constexpr int C = F::C, LD = F::LD, LV = F::LV, SR = F::SR, SG = F::SG, NL = F::NL, NS = DP / kFpCols;
    extern __shared__ __align__(16) float sm[];
    float* sq = sm;                         // [C][LD]
    float* sk = sq + C * LD;
    float* sv = sk + C * LD;                // [C][LV]
    float* sx = sv + C * LV;                // X [k channel][LV]
    float* sp = sx + DP * LV;               // weighted q.k [C][LV]
    float* pw = sp + C * LV;                // e^{-w n}, n = 0 .. C
    const int j0 = (blockIdx.x % NS) * kFpCols;                      // first v channel
    const int sid = blockIdx.x / NS;
    const Problem& pr = p.pr[sid % p.nprob];
    const int hid = sid / p.nprob, seg = hid % p.nseg, bh = hid / p.nseg, b = bh / p.H, h = bh % p.H;
    const int tid = threadIdx.x, tx = tid % 8, ty = tid / 8;
    const int D = p.D;
    if (j0 >= D) return;
    const float w = __ldg(p.w + h);
    const int n_seq = seq_tokens(p.lengths, b, p.T);
    const int t0 = seg * p.seg_tokens;
    const int n = seg_count(n_seq, seg, p.seg_tokens);               // valid tokens of this segment
    const int t_end = min(t0 + p.seg_tokens, p.T) - t0;              // its rows of the tensors
    const int rev = pr.reverse, e0 = rev ? 0 : 1;
    constexpr int es = sizeof(IO);
    const size_t dd = (size_t)D * D;
    const size_t xo = ((size_t)bh * p.nseg + seg) * dd;
    const bool want_out = pr.out != nullptr;
    const size_t row0 = (size_t)b * p.T + t0;
    const size_t col0 = (size_t)h * D;
    const int nchunk = (n + C - 1) / C;
    const int j = j0 + 4 * tx;                                       // this thread's columns

    // float4 x of a chunk's tiles: q, k (rows of DP) and v (rows of this CTA's columns), zero past the
    // chunk's tokens and the head's channels
    float4 next[NL];
    auto place = [&](int x, int& which, int& r, int& c) {
        constexpr int PQ = C * (DP / 4);
        which = x < PQ ? 0 : x < 2 * PQ ? 1 : 2;
        const int y = x - which * PQ, per = which == 2 ? kFpCols / 4 : DP / 4;
        r = y / per;
        c = 4 * (y % per);
    };
    auto fetch = [&](int ci) {
        const int a = (rev ? nchunk - 1 - ci : ci) * C, m = min(C, n - a);
#pragma unroll
        for (int i = 0; i < NL; ++i) {
            int which, r, c;
            place(i * kFpThreads + tid, which, r, c);
            const int ch = c + (which == 2 ? j0 : 0);
            next[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r < m && ch < D && (which != 0 || want_out)) {
                const char* base = which == 0 ? pr.q : which == 1 ? pr.k : pr.v;
                const long long ld = which == 0 ? pr.ldq : which == 1 ? pr.ldk : pr.ldv;
                const char* src = base + ((row0 + a + r) * (size_t)ld + col0 + ch) * es;
                if (p.vec) {
                    next[i] = ld4<IO>(src);
                } else {
                    next[i].x = Io<IO>::ld1(src);
                    if (ch + 1 < D) next[i].y = Io<IO>::ld1(src + es);
                    if (ch + 2 < D) next[i].z = Io<IO>::ld1(src + 2 * es);
                    if (ch + 3 < D) next[i].w = Io<IO>::ld1(src + 3 * es);
                }
            }
        }
    };
    if (nchunk > 0) fetch(0);
    if (tid <= C) pw[tid] = decay_pow(w, tid);
    // rows of the state a thread owns: SG adjacent ones per 16 * SG
    auto state_row = [&](int r) { return (r / SG) * (16 * SG) + ty * SG + r % SG; };
    float4 X[SR];
#pragma unroll
    for (int r = 0; r < SR; ++r) {
        const int i = state_row(r);
        float e[4] = {0.f, 0.f, 0.f, 0.f};
        if (pr.x_in && i < D) {
#pragma unroll
            for (int m = 0; m < 4; ++m)
                if (j + m < D) e[m] = __ldg(pr.x_in + xo + (pr.x_in_t ? (size_t)(j + m) * D + i : (size_t)i * D + j + m));
        }
        X[r] = make_float4(e[0], e[1], e[2], e[3]);
    }

    for (int ci = 0; ci < nchunk; ++ci) {
        const int a = (rev ? nchunk - 1 - ci : ci) * C;              // first token of the chunk, in the segment
        const int m = min(C, n - a);                                 // its tokens
        const bool with_x = ci > 0 || pr.x_in != nullptr, update = ci + 1 < nchunk || pr.x_out != nullptr;
        __syncthreads();                                             // the previous chunk's readers are done
#pragma unroll
        for (int i = 0; i < NL; ++i) {
            int which, r, c;
            place(i * kFpThreads + tid, which, r, c);
            *reinterpret_cast<float4*>(which == 2 ? sv + r * LV + c : (which ? sk : sq) + r * LD + c) = next[i];
        }
        if (want_out && with_x) {
#pragma unroll
            for (int r = 0; r < SR; ++r) *reinterpret_cast<float4*>(sx + state_row(r) * LV + 4 * tx) = X[r];
        }
        __syncthreads();
        if (ci + 1 < nchunk) fetch(ci + 1);
        if (want_out) {
            // weighted products: rows ty, ty + 16, columns tx + 8 z; the far quarter has no past
            float acc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll 4
            for (int i = 0; i < DP; i += 4) {
                float4 qa[2], kb[4];
#pragma unroll
                for (int y = 0; y < 2; ++y) qa[y] = *reinterpret_cast<const float4*>(sq + (ty + 16 * y) * LD + i);
#pragma unroll
                for (int z = 0; z < 4; ++z) kb[z] = *reinterpret_cast<const float4*>(sk + (tx + 8 * z) * LD + i);
#pragma unroll
                for (int z = 0; z < 4; ++z) {
                    const int near = z < 2 ? 0 : 1;                  // (0, z) and (1, z), less one of the far quarters
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        if (y != near && (rev ? y > near : y < near)) continue;
                        acc[y][z] = fmaf(qa[y].x, kb[z].x, acc[y][z]);
                        acc[y][z] = fmaf(qa[y].y, kb[z].y, acc[y][z]);
                        acc[y][z] = fmaf(qa[y].z, kb[z].z, acc[y][z]);
                        acc[y][z] = fmaf(qa[y].w, kb[z].w, acc[y][z]);
                    }
                }
            }
#pragma unroll
            for (int y = 0; y < 2; ++y)
#pragma unroll
                for (int z = 0; z < 4; ++z) {
                    const int d = rev ? tx + 8 * z - ty - 16 * y : ty + 16 * y - tx - 8 * z;
                    sp[(ty + 16 * y) * LV + tx + 8 * z] = d < 0 ? 0.f : acc[y][z] * pw[d] * pr.scale_intra;
                }
            __syncthreads();
            float4 o[2];
            o[0] = o[1] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (with_x) {
#pragma unroll 4
                for (int i = 0; i < DP; i += 4) {
                    float4 qa[2];
#pragma unroll
                    for (int r = 0; r < 2; ++r) qa[r] = *reinterpret_cast<const float4*>(sq + (ty + 16 * r) * LD + i);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float4 xv = *reinterpret_cast<const float4*>(sx + (i + e) * LV + 4 * tx);
#pragma unroll
                        for (int r = 0; r < 2; ++r) fma4(o[r], at4(qa[r], e), xv);
                    }
                }
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const int row = ty + 16 * r, d = rev ? m - 1 - row : row;
                    const float f = row < m ? pw[d + e0] * pr.scale_inter : 0.f;
                    o[r] = make_float4(o[r].x * f, o[r].y * f, o[r].z * f, o[r].w * f);
                }
            }
            // in the half a row does not reach its products are zeros
#pragma unroll 2
            for (int s = 0; s < C; s += 4) {
                const bool reach[2] = {!(!rev && s >= 16), !(rev && s < 16)};
                float4 pa[2];
#pragma unroll
                for (int r = 0; r < 2; ++r)
                    if (reach[r]) pa[r] = *reinterpret_cast<const float4*>(sp + (ty + 16 * r) * LV + s);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float4 vv = *reinterpret_cast<const float4*>(sv + (s + e) * LV + 4 * tx);
#pragma unroll
                    for (int r = 0; r < 2; ++r)
                        if (reach[r]) fma4(o[r], at4(pa[r], e), vv);
                }
            }
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int row = ty + 16 * r;
                if (row >= m || j >= D) continue;
                char* dst = pr.out + ((row0 + a + row) * (size_t)p.H * D + col0 + j) * es;
                if (p.vec) {
                    st4<IO>(dst, o[r]);
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (j + e < D) Io<IO>::st1(dst + e * es, at4(o[r], e));
                }
            }
        }
        if (!update) break;                                          // no one reads the last state
        // X <- e^{-w m} X + sum_s f_s k_s^T v_s
        const float fx = pw[m];
#pragma unroll
        for (int r = 0; r < SR; ++r) X[r] = make_float4(X[r].x * fx, X[r].y * fx, X[r].z * fx, X[r].w * fx);
#pragma unroll 4
        for (int s = 0; s < m; ++s) {
            const float f = pw[rev ? s + 1 : m - 1 - s] * pr.scale_upd;
            float4 vv = *reinterpret_cast<const float4*>(sv + s * LV + 4 * tx);
            vv = make_float4(vv.x * f, vv.y * f, vv.z * f, vv.w * f);
            if constexpr (SG == 4) {
#pragma unroll
                for (int g = 0; g < SR / 4; ++g) {
                    const float4 kk = *reinterpret_cast<const float4*>(sk + s * LD + g * 64 + ty * 4);
#pragma unroll
                    for (int e = 0; e < 4; ++e) fma4(X[4 * g + e], at4(kk, e), vv);
                }
            } else {
#pragma unroll
                for (int r = 0; r < SR; ++r) fma4(X[r], sk[s * LD + state_row(r)], vv);
            }
        }
    }

    if (pr.x_out) {
#pragma unroll
        for (int r = 0; r < SR; ++r) {
            const int i = state_row(r);
            if (i >= D) continue;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (j + e < D) pr.x_out[xo + (pr.x_out_t ? (size_t)(j + e) * D + i : (size_t)i * D + j + e)] = at4(X[r], e);
        }
    }
    if (want_out) {  // rows past the sequence's end
        const int cols = min(kFpCols, D - j0);
        for (int x = tid; x < (t_end - n) * cols; x += kFpThreads)
            Io<IO>::st1(pr.out + ((row0 + n + x / cols) * (size_t)p.H * D + col0 + j0 + x % cols) * es, 0.f);
    }
}

// ---------------------------------------------------------------------------
// Chain the segments' own states: on entry u[seg] is segment seg's X_out from
// X_in = 0; on return it is the segment's X_in, and x_last, if given, the
// state after the last segment.  One thread per state element, the segments
// in order (last to first in reversed time); loads of the next segment do not
// wait for the chain.
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

__global__ void __launch_bounds__(256) decay_chain_kernel(const ChainParams p) {
    const ChainProblem& pr = p.pr[blockIdx.z];
    const int bh = blockIdx.x, b = bh / p.H, h = bh % p.H;
    const int i = blockIdx.y * 256 + threadIdx.x;
    if (i >= p.dd) return;
    const float w = __ldg(p.w + h);
    const int n_seq = seq_tokens(p.lengths, b, p.T);
    float x = pr.x0 ? __ldg(pr.x0 + (size_t)bh * p.dd + i) : 0.f;
    float* u = pr.u + (size_t)bh * p.nseg * p.dd + i;
    const int step = pr.reverse ? -1 : 1;
    int seg = pr.reverse ? p.nseg - 1 : 0;
    float next = u[(size_t)seg * p.dd];
    for (int s = 0; s < p.nseg; ++s, seg += step) {
        const float own = next;
        if (s + 1 < p.nseg) next = u[(size_t)(seg + step) * p.dd];
        u[(size_t)seg * p.dd] = x;
        x = fmaf(decay_pow(w, seg_count(n_seq, seg, p.seg_tokens)), x, own);
    }
    if (pr.x_last) pr.x_last[(size_t)bh * p.dd + i] = x;
}

// ---------------------------------------------------------------------------
// One token per sequence on a pool of states (N, H, D, D), updated in place:
//   S = e^{-w} S + k^T v,  out = scale q S.
// Bound by the state's bytes (read and written once).  A CTA takes a slab of
// 32 columns of one head's state: independent of the other slabs, 128-byte
// rows, and enough CTAs at batch 1.  Thread (r, c4): rows r, r + RT, .. and
// the 4 columns c4; the columns' partial sums over the rows meet in shared
// memory.
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

template <typename IO>
__global__ void __launch_bounds__(kStepThreads) decay_step_kernel(const StepParams p) {
    __shared__ float sq[kStepMaxD], sk[kStepMaxD];
    __shared__ float4 part[kStepRows / 4][kStepCols / 4];  // one row per warp
    const int b = blockIdx.x, h = blockIdx.y, slab = blockIdx.z, tid = threadIdx.x, D = p.D;
    const int c4 = tid % (kStepCols / 4), r0 = tid / (kStepCols / 4);
    const int j = slab * kStepCols + 4 * c4;
    const int slot = p.slots ? __ldg(p.slots + b) : b;
    const bool in_range = slot >= 0 && slot < p.N;
    constexpr int es = sizeof(IO);
    constexpr int NP = kStepMaxD / kStepRows;       // passes over the rows
    float* S = p.state + ((size_t)(in_range ? slot : 0) * p.H + h) * D * D;

    float4 x[NP];
#pragma unroll
    for (int m = 0; m < NP; ++m) {
        const int i = r0 + kStepRows * m;
        x[m] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (in_range && i < D && j < D) {
            const float* s = S + (size_t)i * D + j;
            if (p.vec) {
                x[m] = *reinterpret_cast<const float4*>(s);
            } else {
                x[m].x = s[0];
                if (j + 1 < D) x[m].y = s[1];
                if (j + 2 < D) x[m].z = s[2];
                if (j + 3 < D) x[m].w = s[3];
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
        if (j + e < D) v[e] = Io<IO>::ld1(p.v + ((size_t)b * p.ldv + (size_t)h * D + j + e) * es);
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
                    *reinterpret_cast<float4*>(s) = x[m];
                } else {
                    s[0] = x[m].x;
                    if (j + 1 < D) s[1] = x[m].y;
                    if (j + 2 < D) s[2] = x[m].z;
                    if (j + 3 < D) s[3] = x[m].w;
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
        const int jj = slab * kStepCols + tid;
        float s = 0.f;
#pragma unroll
        for (int q = 0; q < kStepRows / 4; ++q) s += reinterpret_cast<const float*>(&part[q][0])[tid];
        if (jj < D) Io<IO>::st1(p.out + ((size_t)b * p.H * D + (size_t)h * D + jj) * es, s);
    }
}

}  // namespace decay
}  // namespace vrwkv
