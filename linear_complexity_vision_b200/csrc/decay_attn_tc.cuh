// Multi-head decay attention on the 5th-generation tensor cores: the operator
// of decay_attn.cuh (the same problems, segments and states) for bfloat16 and
// heads of up to D = 128 (states: also 64) channels, in chunks of 128 tokens.
// Narrower heads, of whole 16-byte vectors, are zero-padded to D by TMA.
//
// Per chunk, with q, k, v tiles brought by TMA (128-byte swizzle) and X^T, the
// state, in float32 registers:
//   A  = q k^T                        (128 x 128)  accumulators in tensor memory
//   O  = q X                          (128 x D)    from X as bfloat16 hi + lo
//   O *= scale e^{-w (t+e0)} by rows
//   P  = decays, masked, times A      back into tensor memory as bfloat16 hi + lo,
//                                     in the columns A had
//   O += P v                          P from tensor memory, v as it lies in its tile
//   U  = v^T K~                       K~ = e^{-w (..)} k as bfloat16 pieces
//   X^T = e^{-w n} X^T + U            in registers
// X ends in bfloat16 outputs and is split in two, off by at most 2^-17 (half a
// step of a remainder below 2^-8).  P and K~ are split so too (PIECES = 2); a
// state that leaves the call (PIECES = 3) is formed from three pieces, which
// hold a float32 value exactly.  (P and K~ as one bfloat16 each: 8 x 4096, 16
// heads of 64 in 70 us in place of 87, outputs 1.41 times as far from the exact
// ones as their own rounding leaves them.)
//
// Decays.  Where |w| <= 1/2 (and the scale is of a size to spare, factored()), e^{-w (t - s)} = e^{-w (t - 63)} e^{-w (63 - s)}
// stays within e^{+-32}: P takes the column's factor alone, the row's factor
// multiplies the finished row of O, and X enters times e^{-64 w}, so that
// O = q X and O += P v add up without a pass between them.  (A sum may then
// grow to e^32 times the output before the last multiplication: outputs below
// 1e24 are safe.)  For faster decays a 32 x 32 block of P off the diagonal takes
// e^{-w (t - s_end)} e^{-w (s_end - s)}, both exponents >= 0, which underflow to
// 0 instead of overflowing, the diagonal block takes a table by t - s, and
// O = q X is scaled by rows in tensor memory.
//
// All working warps share every step; a warp's quarter of tensor memory (its
// number mod 4) decides its rows, its warpgroup the columns.  One more warp
// issues loads and MMAs and works on nothing else, since issuing waits for the
// tensor pipe.  The tiles are loaded for the next chunk as soon as their last
// readers are done: q and k (unless it holds the third piece) after A, O = q X
// and K~, a whole chunk's work ahead; v after O += P v (without outputs there is
// room for two tiles of v and for the third piece: loads are two chunks ahead).
// D = 128: 16 working warps, 224 KB of tiles, 384 of the 512 tensor-memory
// columns, one CTA per SM.  Without outputs (the states at the cuts of long
// sequences) D = 64 runs here too: 8 warps, 98 KB, two CTAs per SM.  Its outputs
// have a kernel of their own (decay_attn_tc64.cuh).
//
// Measured: B = 1, T = 16384, 8 heads of 128, with a final state: 73 us (states
// 30, chain 4, outputs 43; floor 20.7, its bytes).  128 CTAs walk 8 chunks each;
// the tensor pipe is busy a third of that time and DRAM less: what is left is
// the chain A -> P -> O -> next chunk of one CTA, whose steps wait for one another.
// Two chunks at a time, as heads of 64 run them, do not fit: 224 KB of tiles.
//
// Every wait is bounded: a wait that runs out records flag 8 in the device
// error word, makes every warp leave its loop, waits (bounded) for copies and
// MMAs in flight and frees the tensor memory before the CTA exits.
#pragma once

#include "decay_attn.cuh"
#include "tc_util.cuh"

namespace vrwkv {
namespace decay {

constexpr int kTcChunk = 128;
constexpr unsigned kTcErr = 8u;

struct TcParams {
    CUtensorMap map[4];      // (D, H, T, B) tensors: box (64, 1, 128, 1), 128-byte swizzle, zeros past D and T
    CUtensorMap omap[3];     // the problems' outputs, likewise
    Params p;
    int mq[3], mk[3], mv[3]; // maps of the problems' q, k, v
    int wide_out;            // the outputs' rows of a head are 32-byte aligned
    int nitems;              // CTAs, or work items of the persistent kernel
    int step[4];             // its CTAs' stride in items, as (problem, segment, head, sequence)
    unsigned int* err;
    unsigned long long wait_ns;
};

// Whether a problem's decays are taken as a column's factor times a row's, within
// e^{+-32}.  The column's carries the scale: where that is tiny or huge, bits or
// values would be lost between the two.
__device__ __forceinline__ bool factored(float w, const Problem& pr) {
    const float s = fabsf(pr.scale_intra);
    return fabsf(w) <= 0.5f && s >= 1e-12f && s <= 1e12f;
}

template <int D>
__host__ __device__ constexpr int tc_threads() {
    return D == 64 ? 288 : 544;  // the last warp issues
}

// Tiles of a CTA; without outputs neither q nor the state's operands.
template <int D, bool OUT>
struct alignas(1024) TcSmem {
    static constexpr int kSub = D / 64;                 // 64-channel subtiles of a tile
    static constexpr int kTile = kSub * 128 * 128;      // bytes of a token tile
    static constexpr int kState = kSub * D * 128;       // bytes of a state operand
    uint8_t k[kTile], v[OUT ? 1 : 2][kTile], kh[kTile], km[kTile];
    uint8_t q[kTile];                                   // without outputs: K~'s third piece
    uint8_t xh[OUT ? kState : 1024], xl[OUT ? kState : 1024];  // X^T: rows v channel, K-major
    float pw[kTcChunk + 4];                             // e^{-w n}, n = 0 .. 128
    // fast: scale_intra e^{-w (63 - s)} (reversed: s - 63); else [i] scale_intra e^{-w (31 - i)} (reversed: i)
    float col[kTcChunk];
    // fast: e^{-w (t - 63)} (reversed: 63 - t); else scale_intra e^{-w d}, 0 for d < 0, with d = t - s (s - t) at
    // [31 - d] ([31 + d])
    float row[kTcChunk];
    unsigned long long fa, fv[2], a, kt, u, pr, o, xr, of, drain;
    unsigned tmem;
    int abort;
};

template <int D, bool OUT>
constexpr int tc_smem_bytes() {
    return (int)sizeof(TcSmem<D, OUT>) + 1024;
}

__device__ __forceinline__ uint32_t pack_bf16(float2 x) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x.x, x.y);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 unpack_bf16(uint32_t h) {
    return f2(__uint_as_float(h << 16), __uint_as_float(h & 0xffff0000u));
}
// x rounded to bfloat16 (returned), at most to the largest finite value: x becomes
// what the rounding left out, and the last piece, not bounded, keeps an infinity.
__device__ __forceinline__ uint32_t split_bf16(float2& x) {
    uint32_t h;
    asm("cvt.rn.satfinite.bf16x2.f32 %0, %1, %2;" : "=r"(h) : "f"(x.y), "f"(x.x));
    x = fma2(unpack_bf16(h), f2(-1.0f), x);
    return h;
}

// One 32 x 32 block of P, in the columns at taddr that hold the same block of A:
// the thread's row (lane, in a quarter of the chunk's rows), columns 32 j .., d4
// blocks back in (walked) time.  16 columns of A become 8 of hi and 8 of lo.
// pw, col, row: the tables of TcSmem.
__device__ __forceinline__ void p_block(uint32_t taddr, int j, int d4, bool fast, int rev, int lane, int m,
                                        const float* pw, const float* col, const float* row) {
    float all[32];
    tc::tmem_ld32(taddr, all);
    const float2 f = f2(fast ? 1.0f : pw[d4 == 0 ? 0 : rev ? 32 * d4 - lane : 32 * d4 - 31 + lane]);
    const float* dg = row + 31 - lane;
    const float* cl = fast ? col + 32 * j : col;
#pragma unroll
    for (int g = 0; g < 32; g += 16) {
        float v[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = all[g + i];
        if (d4 == 0 && !fast) {
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] *= dg[g + i];
        } else {
#pragma unroll
            for (int i = 0; i < 16; i += 4) {
                const float4 c = *reinterpret_cast<const float4*>(cl + g + i);
                float2 x = mul2(f2(v[i], v[i + 1]), f2(c.x, c.y));
                float2 y = mul2(f2(v[i + 2], v[i + 3]), f2(c.z, c.w));
                if (!fast) {
                    x = mul2(x, f);
                    y = mul2(y, f);
                }
                v[i] = x.x;
                v[i + 1] = x.y;
                v[i + 2] = y.x;
                v[i + 3] = y.y;
            }
            if (d4 == 0) {
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (rev ? g + i < lane : g + i > lane) v[i] = 0.f;
            }
        }
        if (32 * j + g + 16 > m) {  // columns past the chunk's tokens
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (32 * j + g + i >= m) v[i] = 0.f;
        }
        uint32_t out[16];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float2 x = f2(v[2 * i], v[2 * i + 1]);
            out[i] = split_bf16(x);
            out[8 + i] = pack_bf16(x);
        }
        tc::tmem_st16(taddr + g, out);
    }
}

// Row jr of X^T, columns c0 .. c0 + NX, from a (d, d) state, zeros past d (the
// first state 16-byte aligned).  No load waits for a branch.
template <int NX>
__device__ __forceinline__ void load_x(float (&X)[NX], const float* x, bool transposed, int jr, int c0, int d) {
    const int here = jr < d ? d - c0 : 0;
    if (transposed && d % 4 == 0) {
#pragma unroll
        for (int i = 0; i < NX; i += 4) {
            const float4 y = __ldcg(reinterpret_cast<const float4*>(x + (i < here ? jr * d + c0 + i : 0)));
            X[i] = i < here ? y.x : 0.f;
            X[i + 1] = i < here ? y.y : 0.f;
            X[i + 2] = i < here ? y.z : 0.f;
            X[i + 3] = i < here ? y.w : 0.f;
        }
    } else {
#pragma unroll
        for (int i = 0; i < NX; ++i) {
            const float y = __ldcg(x + (i < here ? (transposed ? jr * d + c0 + i : (c0 + i) * d + jr) : 0));
            X[i] = i < here ? y : 0.f;
        }
    }
}
template <int NX>
__device__ __forceinline__ void store_x_out(const float (&X)[NX], float* x, bool transposed, int jr, int c0, int d) {
    const int here = jr < d ? d - c0 : 0;
#pragma unroll
    for (int i = 0; i < NX; ++i)
        if (i < here) x[transposed ? jr * d + c0 + i : (c0 + i) * d + jr] = X[i];
}

__device__ __forceinline__ void st_global_32(char* p, const uint32_t (&r)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(r[0]), "r"(r[1]), "r"(r[2]),
                 "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}

// PAD: heads may be narrower than D.  (With the width a variable in every
// launch, B = 1, T = 16384, 8 heads of 128 took 87 us in place of 80.)
template <int D, bool OUT, int PIECES, bool PAD>
__global__ void __launch_bounds__(tc_threads<D>(), D == 64 ? 2 : 1)
    decay_attn_tc_kernel(const __grid_constant__ TcParams P) {
    static_assert(D == 128 || !OUT, "outputs of D = 64 have a kernel of their own");
    using Sm = TcSmem<D, OUT>;
    constexpr int C = kTcChunk, SUB = Sm::kSub, SUBB = 128 * 128, kThreads = tc_threads<D>();
    constexpr int NWG = kThreads / 128, NW = 4 * NWG, kWork = 32 * NW;
    constexpr uint32_t kColO = 128, kColU = OUT ? 128 + D : 0;
    constexpr uint32_t kCols = OUT ? 512 : D;
    constexpr int NX = D * D / kWork;                   // state values of a thread
    extern __shared__ __align__(1024) char smem_raw[];
    Sm& S = *reinterpret_cast<Sm*>(smem_raw + ((1024u - (tc::smem_u32(smem_raw) & 1023u)) & 1023u));
    const Params& p = P.p;
    const int prob = blockIdx.x % p.nprob;
    const Problem& pr = p.pr[prob];
    const int sid = blockIdx.x / p.nprob, seg = sid % p.nseg, bh = sid / p.nseg, b = bh / p.H, h = bh % p.H;
    next_pass();
    if (!OUT && seg == pr.skip) return;
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31, quad = warp & 3, wg = warp >> 2;
    const float w = __ldg(p.w + h);
    const int n_seq = seq_tokens(p.lengths, b, p.T);
    const int t0 = seg * p.seg_tokens;
    const int n = seg_count(n_seq, seg, p.seg_tokens);
    const int t_end = min(t0 + p.seg_tokens, p.T) - t0;
    const int rev = pr.reverse, e0 = rev ? 0 : 1;
    const int nchunk = (n + C - 1) / C;
    const bool has_in = pr.x_in != nullptr, has_out = pr.x_out != nullptr;
    const int d = PAD ? p.D : D;                        // channels there are; operands are zero past them
    const int sd = PAD ? p.S : D;                       // and of a state
    const size_t xo = ((size_t)bh * p.nseg + seg) * sd * sd;

    if (tid == 0) {
        tc::mbar_init(&S.fa, 1);
        tc::mbar_init(&S.fv[0], 1);
        tc::mbar_init(&S.fv[1], 1);
        tc::mbar_init(&S.a, 1);
        tc::mbar_init(&S.kt, NW);
        tc::mbar_init(&S.u, 1);
        tc::mbar_init(&S.pr, NW);
        tc::mbar_init(&S.o, 1);
        tc::mbar_init(&S.xr, NW);
        tc::mbar_init(&S.of, NW);
        tc::mbar_init(&S.drain, 1);
        S.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) tc::tmem_alloc(&S.tmem, kCols);
    const DecayBase base = decay_base(w);
    const bool fast = factored(w, pr);
    for (int i = tid; i <= C; i += kThreads) S.pw[i] = decay_pow(base, i);
    if (OUT && tid < C) {
        if (fast) {
            S.col[tid] = decay_pow(base, rev ? tid - 63 : 63 - tid) * pr.scale_intra;
            S.row[tid] = decay_pow(base, rev ? 63 - tid : tid - 63);
        } else {
            const int d = rev ? tid - 31 : 31 - tid;
            if (tid < 32) S.col[tid] = decay_pow(base, rev ? tid : 31 - tid) * pr.scale_intra;
            if (tid < 64) S.row[tid] = d < 0 ? 0.f : decay_pow(base, d) * pr.scale_intra;
        }
    }

    volatile int* abort = &S.abort;
    auto wait = [&](unsigned long long& bar, int phase) {
        return tc::mbar_test(&bar, (unsigned)phase & 1u) ||
               tc::wait_slow(&bar, (unsigned)phase & 1u, abort, P.err, kTcErr, P.wait_ns);
    };
    auto wait_warp = [&](unsigned long long& bar, int phase) {
        return __all_sync(0xffffffffu, wait(bar, phase) ? 1 : 0) != 0;
    };
    auto arrive_warp = [&](unsigned long long& bar) {
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&bar);
    };
    // chunk ci of the walk: its first token in the segment
    auto first = [&](int ci) { return (rev ? nchunk - 1 - ci : ci) * C; };
    constexpr int NV = OUT ? 1 : 2;                     // tiles of v
    const uint32_t sq = tc::smem_u32(S.q), sk = tc::smem_u32(S.k);
    auto sv = [&](int ci) { return tc::smem_u32(S.v[ci % NV]); };
    uint8_t* third = OUT ? S.k : S.q;                   // of K~'s pieces
    const uint32_t s3 = tc::smem_u32(third);
    const uint32_t skh = tc::smem_u32(S.kh), skm = tc::smem_u32(S.km), sxh = tc::smem_u32(S.xh), sxl = tc::smem_u32(S.xl);
    auto load = [&](uint32_t dst, int map, int ci, unsigned long long* bar) {
#pragma unroll
        for (int s = 0; s < SUB; ++s)
            tc::tma_load_4d(dst + s * SUBB, &P.map[map], 64 * s, h, t0 + first(ci), b, bar);
    };
    __syncthreads();
    const bool issuer = warp == NW;
    auto load_q = [&](int ci) {  // begins fa's phase; k completes it
        tc::mbar_expect_tx(&S.fa, (OUT ? 2 : 1) * Sm::kTile);
        if (OUT) load(sq, P.mq[prob], ci, &S.fa);
    };
    auto load_k = [&](int ci) { load(sk, P.mk[prob], ci, &S.fa); };
    auto load_v = [&](int ci) {
        tc::mbar_expect_tx(&S.fv[ci % NV], Sm::kTile);
        load(sv(ci), P.mv[prob], ci, &S.fv[ci % NV]);
    };
    if (issuer && nchunk > 0 && tc::elect_one()) {
        load_q(0);
        load_k(0);
        load_v(0);
        if (!OUT && nchunk > 1) load_v(1);
    }

    // X: row jr of X^T (a v channel), columns c0 .. (k channels).  For D = 64
    // U has its rows twice: v's tile is read as both halves of M = 128.
    const int jr = D == 64 ? (quad & 1) * 32 + lane : quad * 32 + lane;
    const int c0 = D == 64 ? ((quad >> 1) * 2 + wg) * NX : wg * NX;
    float X[NX];
    last_pass();
    if (has_in && !issuer) {
        load_x(X, pr.x_in + xo, pr.x_in_t, jr, c0, sd);
    } else {
#pragma unroll
        for (int i = 0; i < NX; ++i) X[i] = 0.f;
    }
    // X^T as operands of a chunk of m tokens: row jr, 16-byte piece c of 64 channels at piece c ^ (jr & 7)
    auto store_x = [&](int m) {
        const float2 f = f2(fast ? decay_pow(base, rev ? m - 64 : 64) * pr.scale_inter : 1.0f);
#pragma unroll
        for (int i = 0; i < NX; i += 8) {
            const int c = c0 + i;
            const uint32_t off = (c / 64) * D * 128 + jr * 128 + ((((c % 64) / 8) ^ (jr & 7)) << 4);
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float2 x = mul2(f2(X[i + 2 * e], X[i + 2 * e + 1]), f);
                hi[e] = split_bf16(x);
                lo[e] = pack_bf16(x);
            }
            *reinterpret_cast<uint4*>(S.xh + off) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            *reinterpret_cast<uint4*>(S.xl + off) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
        tc::fence_async_smem();
        arrive_warp(S.xr);
    };
    if (OUT && has_in && !issuer && nchunk > 0) store_x(min(C, n - first(0)));
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = S.tmem;
    const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16);
    constexpr uint32_t kIdA = tc::idesc_bf16(128, 128, false, false);
    constexpr uint32_t kIdX = tc::idesc_bf16(128, D, false, false);
    constexpr uint32_t kIdP = tc::idesc_bf16(128, D, false, true);
    constexpr uint32_t kIdU = tc::idesc_bf16(128, D, true, true);
    if (issuer) {
        int loads_a = 1, loads_v = OUT ? 1 : 2;  // loads of k and v begun, if there are as many chunks
        bool issued = false;
        for (int ci = 0; ci < nchunk; ++ci) {
            const bool more = ci + 1 < nchunk, update = more || has_out, with_x = OUT && (ci > 0 || has_in);
            if (!wait_warp(S.fa, ci)) break;
            tc::fence_after();
            if (OUT) {                                  // A = q k^T
                issued = true;
                if (tc::elect_one()) {
#pragma unroll
                    for (int s = 0; s < SUB; ++s) {
                        const uint64_t da = tc::sw128_desc(sq + s * SUBB, 16), db = tc::sw128_desc(sk + s * SUBB, 16);
#pragma unroll
                        for (int k = 0; k < 4; ++k) tc::mma_ss(tmem, da + 2 * k, db + 2 * k, kIdA, s + k > 0);
                    }
                    if (!with_x) tc::commit(&S.a);
                }
                __syncwarp();
            }
            if (with_x) {                               // O = q X
                if (!wait_warp(S.xr, ci - (has_in ? 0 : 1)) || (ci > 0 && !wait_warp(S.of, ci - 1))) break;
                tc::fence_after();
                if (tc::elect_one()) {
#pragma unroll
                    for (int half = 0; half < 2; ++half)
#pragma unroll
                        for (int s = 0; s < SUB; ++s) {
                            const uint64_t da = tc::sw128_desc(sq + s * SUBB, 16);
                            const uint64_t db = tc::sw128_desc((half ? sxl : sxh) + s * D * 128, 16);
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                tc::mma_ss(tmem + kColO, da + 2 * k, db + 2 * k, kIdX, half + s + k > 0);
                        }
                    tc::commit(&S.a);
                }
                __syncwarp();
            }
            if (!wait_warp(S.kt, ci) || !wait_warp(S.fv[ci % NV], ci / NV)) break;
            tc::fence_after();
            if (update) {                               // U = v^T K~
                issued = true;
                if (tc::elect_one()) {
                    const uint64_t da = tc::sw128_desc(sv(ci), D == 64 ? 0 : SUBB);
#pragma unroll
                    for (int piece = 0; piece < PIECES; ++piece) {
                        const uint64_t db = tc::sw128_desc(piece == 0 ? skh : piece == 1 ? skm : s3, SUBB);
#pragma unroll
                        for (int k = 0; k < C / 16; ++k)
                            tc::mma_ss(tmem + kColU, da + 128 * k, db + 128 * k, kIdU, piece + k > 0);
                    }
                    tc::commit(&S.u);
                }
                __syncwarp();
            }
            if (more) {                                 // q's tile is read, and k's or nearly
                if (OUT && !wait_warp(S.a, ci)) break;
                if (tc::elect_one()) {
                    load_q(ci + 1);
                    if (PIECES < 3 || !OUT) load_k(ci + 1);
                }
                ++loads_a;
                __syncwarp();
            }
            if (OUT) {                                  // O += P v
                if (!wait_warp(S.pr, ci)) break;
                tc::fence_after();
                if (tc::elect_one()) {
                    const uint64_t db = tc::sw128_desc(sv(ci), SUBB);
                    const uint32_t acc = with_x ? 1u : 0u;
#pragma unroll
                    for (int k = 0; k < C / 16; ++k)
#pragma unroll
                        for (int half = 0; half < 2; ++half)
                            tc::mma_ts(tmem + kColO, tmem + 16 * k + 8 * half, db + 128 * k, kIdP, k + half > 0 ? 1u : acc);
                    tc::commit(&S.o);
                }
                __syncwarp();
            }
            if (!more) break;
            if ((OUT && !wait_warp(S.o, ci)) || !wait_warp(S.u, ci)) break;
            if (ci + NV < nchunk) {
                if (tc::elect_one()) {
                    if (PIECES == 3 && OUT) load_k(ci + 1);
                    load_v(ci + NV);
                }
                ++loads_v;
                __syncwarp();
            }
        }
        if (*abort) {
            // what was begun ends before the CTA's memory is given back
            const unsigned long long s0 = tc::global_ns();
            auto landed = [&]() {
                bool all = tc::mbar_test(&S.fa, (unsigned)(loads_a - 1) & 1u);
                for (int i = max(0, min(loads_v, nchunk) - NV); i < min(loads_v, nchunk); ++i)
                    all = all && tc::mbar_test(&S.fv[i % NV], (unsigned)(i / NV) & 1u);
                return all;
            };
            while (nchunk > 0 && !landed() && tc::global_ns() - s0 <= P.wait_ns) {
            }
            __syncwarp();
            if (issued) {
                if (tc::elect_one()) tc::commit(&S.drain);
                __syncwarp();
                while (!tc::mbar_test(&S.drain, 0) && tc::global_ns() - s0 <= 2 * P.wait_ns) {
                }
            }
        }
        __syncwarp();
    }

    const int wq = rev ? 3 - quad : quad;               // blocks of P off the diagonal in this quarter
    int ci = 0;
    for (; ci < nchunk && !issuer; ++ci) {
        const int a = first(ci), m = min(C, n - a);
        const bool more = ci + 1 < nchunk, update = more || has_out, with_x = OUT && (ci > 0 || has_in);
        if (!wait_warp(S.fa, ci)) break;
        if (m < C) {  // rows of v past the chunk's tokens meet zeros of P and K~: 0 * NaN is NaN
            if (!wait_warp(S.fv[ci % NV], ci / NV)) break;
            for (int x = tid; x < (C - m) * 8 * SUB; x += kWork)
                *reinterpret_cast<uint4*>(S.v[ci % NV] + (x / ((C - m) * 8)) * SUBB + (m + x % ((C - m) * 8) / 8) * 128 +
                                          (x % 8) * 16) = make_uint4(0u, 0u, 0u, 0u);
        }
        if (update) {
            if (OUT && PIECES == 3 && !wait_warp(S.a, ci)) break;  // the third piece takes k's own tile
            constexpr int kUnits = 8 * SUB * 128 / kWork;  // 16-byte pieces of a thread
            uint4 raws[kUnits];
            float fs[kUnits];
#pragma unroll
            for (int i = 0; i < kUnits; ++i) {
                const int x = i * kWork + tid, r = (x % 1024) / 8;
                raws[i] = *reinterpret_cast<const uint4*>(S.k + x * 16);
                fs[i] = S.pw[rev ? r + 1 : max(m - 1 - r, 0)] * pr.scale_upd;
                if (r >= m) raws[i] = make_uint4(0u, 0u, 0u, 0u);
            }
#pragma unroll
            for (int i = 0; i < kUnits; ++i) {
                const uint32_t off = (i * kWork + tid) * 16;
                const float2 f = f2(fs[i]);
                const uint32_t rw[4] = {raws[i].x, raws[i].y, raws[i].z, raws[i].w};
                uint32_t hi[4], mi[4], lo[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float2 y = mul2(unpack_bf16(rw[e]), f);
                    hi[e] = split_bf16(y);
                    if (PIECES == 3) {
                        mi[e] = split_bf16(y);
                        lo[e] = pack_bf16(y);
                    } else {
                        mi[e] = pack_bf16(y);
                    }
                }
                *reinterpret_cast<uint4*>(S.kh + off) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                *reinterpret_cast<uint4*>(S.km + off) = make_uint4(mi[0], mi[1], mi[2], mi[3]);
                if (PIECES == 3) *reinterpret_cast<uint4*>(third + off) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
            }
        }
        tc::fence_async_smem();
        arrive_warp(S.kt);
        if (OUT) {
            if (!wait_warp(S.a, ci)) break;
            tc::fence_after();
            // P: the quarter's rows, the block wg blocks back in (walked) time
            const int j = rev ? (quad + wg) & 3 : (quad - wg) & 3;
            if (wg > wq || 32 * j >= m) tc::tmem_zero<32>(lanes + 32 * j);  // before the sequence's start, or past the chunk's end
            else p_block(lanes + 32 * j, j, wg, fast, rev, lane, m, S.pw, S.col, S.row);
            if (!fast && with_x) {
                const int row = quad * 32 + lane;
                const float2 f = f2(S.pw[max(rev ? m - 1 - row : row, 0) + e0] * pr.scale_inter);
#pragma unroll
                for (int g = 0; g < 32; g += 16) {
                    float v[16];
                    uint32_t out[16];
                    tc::tmem_ld16(lanes + kColO + wg * 32 + g, v);
#pragma unroll
                    for (int i = 0; i < 16; i += 2) {
                        const float2 x = mul2(f2(v[i], v[i + 1]), f);
                        out[i] = __float_as_uint(x.x);
                        out[i + 1] = __float_as_uint(x.y);
                    }
                    tc::tmem_st16(lanes + kColO + wg * 32 + g, out);
                }
            }
            tc::tmem_wait_st();
            tc::fence_before();
            arrive_warp(S.pr);
        }
        if (update) {
            if (!wait_warp(S.u, ci)) break;
            tc::fence_after();
            const float2 fx = f2(S.pw[m]);
            float v[NX];
            if constexpr (NX == 16) tc::tmem_ld16(lanes + kColU + c0, v);
            else tc::tmem_ld32(lanes + kColU + c0, v);
#pragma unroll
            for (int i = 0; i < NX; i += 2) {
                const float2 x = fma2(fx, f2(X[i], X[i + 1]), f2(v[i], v[i + 1]));
                X[i] = x.x;
                X[i + 1] = x.y;
            }
            tc::fence_before();
            if (OUT && more) store_x(min(C, n - first(ci + 1)));
        }
        if (OUT) {
            if (!wait_warp(S.o, ci)) break;
            tc::fence_after();
            const int row = quad * 32 + lane;
            float v[32];
            tc::tmem_ld32(lanes + kColO + wg * 32, v);
            tc::fence_before();
            arrive_warp(S.of);
            if (row < m) {
                const float2 f = f2(fast ? S.row[row] : 1.0f);
                char* dst = pr.out + ((((size_t)b * p.T + t0 + a + row) * p.H + h) * d + wg * 32) * 2;
                const int here = d - wg * 32;           // channels there are
#pragma unroll
                for (int i = 0; i < 32; i += 16) {
                    uint32_t o[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) o[e] = pack_bf16(mul2(f2(v[i + 2 * e], v[i + 2 * e + 1]), f));
                    if (P.wide_out) {
                        if (i < here) st_global_32(dst + 2 * i, o);
                    } else {
                        if (i < here) *reinterpret_cast<uint4*>(dst + 2 * i) = make_uint4(o[0], o[1], o[2], o[3]);
                        if (i + 8 < here) *reinterpret_cast<uint4*>(dst + 2 * i + 16) = make_uint4(o[4], o[5], o[6], o[7]);
                    }
                }
            }
        }
    }
    if (has_out && !issuer && ci == nchunk) store_x_out(X, pr.x_out + xo, pr.x_out_t, jr, c0, sd);
    if (OUT) {  // rows past the sequence's end
        for (int x = tid; x < (t_end - n) * (d / 8); x += kThreads)
            *reinterpret_cast<uint4*>(pr.out + (((size_t)b * p.T + t0 + n + x / (d / 8)) * p.H + h) * d * 2 +
                                      (x % (d / 8)) * 16) = make_uint4(0u, 0u, 0u, 0u);
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    if (warp == 1) tc::tmem_free(tmem, kCols);
}

}  // namespace decay
}  // namespace vrwkv
