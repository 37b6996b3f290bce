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
// the decays, across chunks the state.  Thread (ty, tx) owns output columns
// 4 tx + 64 c of rows ty + TY r, and the state's rows 4 ty + 64 r (DP 128, 64)
// at the same columns, in registers; a copy of the state in shared memory
// feeds the products with q.
template <int DP>
struct Cfg {
    static constexpr int kThreads = 256;
    static constexpr int C = 32;                            // tokens of a chunk
    static constexpr int TX = DP / 4 < 16 ? DP / 4 : 16;    // threads along the columns
    static constexpr int TY = kThreads / TX;
    static constexpr int R = C / TY;                        // output rows of a thread
    static constexpr int NC = DP / 4 / TX;                  // its column groups of 4
    static constexpr int LD = DP + 4;                       // padded row: rows 1 apart are 4 banks apart
    static constexpr int SR = DP * DP / (kThreads * 4 * NC);  // state rows of a thread
    static constexpr int SG = SR < 4 ? SR : 4;              // of which SG are adjacent
    static constexpr int kPowers = C + 1;
    static constexpr int kSmemFloats = 3 * C * LD + DP * LD + C * (C + 4) + kPowers;
};

template <typename IO, int DP>
__global__ void __launch_bounds__(256) decay_attn_kernel(const __grid_constant__ Params p) {
    using F = Cfg<DP>;
    constexpr int C = F::C, LD = F::LD, TX = F::TX, TY = F::TY, R = F::R, NC = F::NC, SR = F::SR, SG = F::SG;
    extern __shared__ __align__(16) float sm[];
    float* sq = sm;
    float* sk = sq + C * LD;
    float* sv = sk + C * LD;
    float* sx = sv + C * LD;                // X [k channel][v channel]
    float* sp = sx + DP * LD;               // weighted q.k [C][C + 4]
    float* pw = sp + C * (C + 4);           // e^{-w n}, n = 0 .. C
    const Problem& pr = p.pr[blockIdx.x % p.nprob];
    const int sx_id = blockIdx.x / p.nprob, seg = sx_id % p.nseg, bh = sx_id / p.nseg, b = bh / p.H, h = bh % p.H;
    const int tid = threadIdx.x, tx = tid % TX, ty = tid / TX;
    const int D = p.D;
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

    if (tid <= C) pw[tid] = decay_pow(w, tid);
    // state registers: rows 4-aligned groups, columns 4 tx + 64 c
    float4 X[SR][NC];
#pragma unroll
    for (int r = 0; r < SR; ++r) {
        const int i = (r / SG) * (TY * SG) + ty * SG + r % SG;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int j = 4 * tx + 64 * c;
            float e[4] = {0.f, 0.f, 0.f, 0.f};
            if (pr.x_in && i < D) {
#pragma unroll
                for (int m = 0; m < 4; ++m)
                    if (j + m < D)
                        e[m] = __ldg(pr.x_in + xo + (pr.x_in_t ? (size_t)(j + m) * D + i : (size_t)i * D + j + m));
            }
            X[r][c] = make_float4(e[0], e[1], e[2], e[3]);
        }
    }

    const size_t row0 = (size_t)b * p.T + t0;
    const size_t col0 = (size_t)h * D;
    const int nchunk = (n + C - 1) / C;
    for (int ci = 0; ci < nchunk; ++ci) {
        const int a = (rev ? nchunk - 1 - ci : ci) * C;              // first token of the chunk, in the segment
        const int m = min(C, n - a);                                 // its tokens
        __syncthreads();                                             // the previous chunk's readers are done
        // tiles, zero past the chunk's tokens and the head's channels
        for (int x = tid; x < 3 * C * (DP / 4); x += F::kThreads) {
            const int which = x / (C * (DP / 4)), y = x % (C * (DP / 4)), r = y / (DP / 4), c = 4 * (y % (DP / 4));
            if (which == 0 && !want_out) continue;
            const char* base = which == 0 ? pr.q : which == 1 ? pr.k : pr.v;
            const long long ld = which == 0 ? pr.ldq : which == 1 ? pr.ldk : pr.ldv;
            float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r < m && c < D) {
                const char* src = base + ((row0 + a + r) * (size_t)ld + col0 + c) * es;
                if (p.vec) {
                    f = ld4<IO>(src);
                } else {
                    f.x = Io<IO>::ld1(src);
                    if (c + 1 < D) f.y = Io<IO>::ld1(src + es);
                    if (c + 2 < D) f.z = Io<IO>::ld1(src + 2 * es);
                    if (c + 3 < D) f.w = Io<IO>::ld1(src + 3 * es);
                }
            }
            float* dst = (which == 0 ? sq : which == 1 ? sk : sv) + r * LD + c;
            *reinterpret_cast<float4*>(dst) = f;
        }
        if (want_out) {
#pragma unroll
            for (int r = 0; r < SR; ++r) {
                const int i = (r / SG) * (TY * SG) + ty * SG + r % SG;
#pragma unroll
                for (int c = 0; c < NC; ++c) *reinterpret_cast<float4*>(sx + i * LD + 4 * tx + 64 * c) = X[r][c];
            }
        }
        __syncthreads();
        if (want_out) {
            // weighted products: rows py, py + 16, columns px, px + 16
            const int py = tid / 16, px = tid % 16;
            float acc[2][2] = {{0.f, 0.f}, {0.f, 0.f}};
#pragma unroll 4
            for (int i = 0; i < DP; i += 4) {
                float4 qa[2], kb[2];
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    qa[y] = *reinterpret_cast<const float4*>(sq + (py + 16 * y) * LD + i);
                    kb[y] = *reinterpret_cast<const float4*>(sk + (px + 16 * y) * LD + i);
                }
#pragma unroll
                for (int y = 0; y < 2; ++y)
#pragma unroll
                    for (int z = 0; z < 2; ++z) {
                        acc[y][z] = fmaf(qa[y].x, kb[z].x, acc[y][z]);
                        acc[y][z] = fmaf(qa[y].y, kb[z].y, acc[y][z]);
                        acc[y][z] = fmaf(qa[y].z, kb[z].z, acc[y][z]);
                        acc[y][z] = fmaf(qa[y].w, kb[z].w, acc[y][z]);
                    }
            }
#pragma unroll
            for (int y = 0; y < 2; ++y)
#pragma unroll
                for (int z = 0; z < 2; ++z) {
                    const int d = rev ? px + 16 * z - py - 16 * y : py + 16 * y - px - 16 * z;
                    sp[(py + 16 * y) * (C + 4) + px + 16 * z] = d < 0 ? 0.f : acc[y][z] * pw[d] * pr.scale_intra;
                }
            __syncthreads();
            float4 o[R][NC];
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int c = 0; c < NC; ++c) o[r][c] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
            for (int i = 0; i < DP; i += 4) {
                float4 qa[R];
#pragma unroll
                for (int r = 0; r < R; ++r) qa[r] = *reinterpret_cast<const float4*>(sq + (ty + TY * r) * LD + i);
#pragma unroll
                for (int e = 0; e < 4; ++e)
#pragma unroll
                    for (int c = 0; c < NC; ++c) {
                        const float4 xv = *reinterpret_cast<const float4*>(sx + (i + e) * LD + 4 * tx + 64 * c);
#pragma unroll
                        for (int r = 0; r < R; ++r) fma4(o[r][c], at4(qa[r], e), xv);
                    }
            }
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const int row = ty + TY * r;
                const int d = rev ? m - 1 - row : row;
                const float f = row < m ? pw[d + e0] * pr.scale_inter : 0.f;
#pragma unroll
                for (int c = 0; c < NC; ++c)
                    o[r][c] = make_float4(o[r][c].x * f, o[r][c].y * f, o[r][c].z * f, o[r][c].w * f);
            }
#pragma unroll 2
            for (int s = 0; s < C; s += 4) {
                float4 pa[R];
#pragma unroll
                for (int r = 0; r < R; ++r) pa[r] = *reinterpret_cast<const float4*>(sp + (ty + TY * r) * (C + 4) + s);
#pragma unroll
                for (int e = 0; e < 4; ++e)
#pragma unroll
                    for (int c = 0; c < NC; ++c) {
                        const float4 vv = *reinterpret_cast<const float4*>(sv + (s + e) * LD + 4 * tx + 64 * c);
#pragma unroll
                        for (int r = 0; r < R; ++r) fma4(o[r][c], at4(pa[r], e), vv);
                    }
            }
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const int row = ty + TY * r;
                if (row >= m) continue;
#pragma unroll
                for (int c = 0; c < NC; ++c) {
                    const int j = 4 * tx + 64 * c;
                    if (j >= D) continue;
                    char* dst = pr.out + ((row0 + a + row) * (size_t)p.H * D + col0 + j) * es;
                    if (p.vec) {
                        st4<IO>(dst, o[r][c]);
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (j + e < D) Io<IO>::st1(dst + e * es, at4(o[r][c], e));
                    }
                }
            }
        }
        if (ci + 1 == nchunk && !pr.x_out) break;                    // no one reads the last state
        // X <- e^{-w m} X + sum_s f_s k_s^T v_s
        const float fx = pw[m];
#pragma unroll
        for (int r = 0; r < SR; ++r)
#pragma unroll
            for (int c = 0; c < NC; ++c)
                X[r][c] = make_float4(X[r][c].x * fx, X[r][c].y * fx, X[r][c].z * fx, X[r][c].w * fx);
        for (int s = 0; s < m; ++s) {
            const float f = pw[rev ? s + 1 : m - 1 - s] * pr.scale_upd;
            float4 vv[NC];
#pragma unroll
            for (int c = 0; c < NC; ++c) vv[c] = *reinterpret_cast<const float4*>(sv + s * LD + 4 * tx + 64 * c);
#pragma unroll
            for (int r = 0; r < SR; ++r) {
                const float kf = sk[s * LD + (r / SG) * (TY * SG) + ty * SG + r % SG] * f;
#pragma unroll
                for (int c = 0; c < NC; ++c) fma4(X[r][c], kf, vv[c]);
            }
        }
    }

    if (pr.x_out) {
#pragma unroll
        for (int r = 0; r < SR; ++r) {
            const int i = (r / SG) * (TY * SG) + ty * SG + r % SG;
            if (i >= D) continue;
#pragma unroll
            for (int c = 0; c < NC; ++c)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int j = 4 * tx + 64 * c + e;
                    if (j < D) pr.x_out[xo + (pr.x_out_t ? (size_t)j * D + i : (size_t)i * D + j)] = at4(X[r][c], e);
                }
        }
    }
    if (want_out) {  // rows past the sequence's end
        for (int x = tid; x < (t_end - n) * D; x += F::kThreads)
            Io<IO>::st1(pr.out + ((row0 + n + x / D) * (size_t)p.H * D + col0 + x % D) * es, 0.f);
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
