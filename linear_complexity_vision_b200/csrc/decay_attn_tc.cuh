// Multi-head decay attention on the 5th-generation tensor cores: the operator
// of decay_attn.cuh (the same problems, segments and states) for bfloat16 and
// heads of D = 64 or 128 channels, in chunks of 128 tokens.
//
// Per chunk, with q, k, v tiles brought by TMA (128-byte swizzle) and X^T, the
// state, in float32 registers of one warpgroup:
//   A  = q k^T                        (128 x 128)  accumulators in tensor memory
//   O  = q X                          (128 x D)    from X as bfloat16 hi + lo
//   O *= scale e^{-w (t+e0)} by rows
//   P  = decays, masked, times A      back into tensor memory as bfloat16 hi + lo,
//                                     in the columns A had
//   O += P v                          P from tensor memory, v as it lies in its tile
//   U  = v^T K~                       K~ = e^{-w (..)} k, three bfloat16 pieces
//   X^T = e^{-w n} X^T + U            in registers
// A float32 value is exactly the sum of three bfloat16 pieces, so the state,
// which is an output and lives on, loses nothing to the tensor cores' operand
// type; P and X, which end in bfloat16 outputs, are split in two, off by half
// a step of the second piece (2^-16).
//
// Decays inside a chunk: a 32 x 32 block of P off the diagonal takes
// e^{-w (t - s)} = e^{-w (t - s_end)} e^{-w (s_end - s)}, both exponents >= 0,
// so fast decays underflow to 0 instead of overflowing; the diagonal block
// takes it from a table by t - s.
//
// Roles (256 threads: a ninth warp would cost each of the others a quarter of
// its registers):
//  * warps 0-3: P, the rows of O and their store.  Thread = token row.  One
//    lane of warp 0 also issues the loads and the MMAs of A and O, all of
//    which wait for warp 0's own work or precede it.
//  * warps 4-7: K~ and X.  Thread = row of X^T; for D = 64 the rows of U come
//    twice (v's tile is read as both halves of M = 128, the second half at
//    distance 0) and a thread takes half of its row.  One lane of warp 4
//    issues the MMAs of U (and, without outputs, the loads).
// D = 64: 96 KB of tiles and 256 tensor-memory columns, two CTAs per SM, which
// hide each other's loads and waits.  D = 128: 224 KB, 384 of 512 columns, one.
// K~'s third piece takes k's own tile once A is done with it.
//
// Every wait is bounded: a wait that runs out records flag 8 in the device
// error word, makes every role leave its loop, waits (bounded) for copies and
// MMAs in flight and frees the tensor memory before the CTA exits.
#pragma once

#include "decay_attn.cuh"
#include "tc_util.cuh"

namespace vrwkv {
namespace decay {

constexpr int kTcChunk = 128;
constexpr int kTcThreads = 256;
constexpr unsigned kTcErr = 8u;

struct TcParams {
    CUtensorMap map[4];      // (C, T, B) tensors: box (64, 128, 1), 128-byte swizzle
    Params p;
    int mq[3], mk[3], mv[3]; // maps of the problems' q, k, v
    unsigned int* err;
    unsigned long long wait_ns;
};

template <int D>
struct alignas(1024) TcSmem {
    static constexpr int kSub = D / 64;                 // 64-channel subtiles of a tile
    static constexpr int kTile = kSub * 128 * 128;      // bytes of a token tile
    static constexpr int kState = kSub * D * 128;       // bytes of a state operand
    uint8_t q[kTile], k[kTile], v[kTile], kh[kTile], km[kTile];
    uint8_t xh[kState], xl[kState];                     // X^T: rows v channel, K-major
    float pw[kTcChunk + 4];                             // e^{-w n}, n = 0 .. 128
    float diag[64];                                     // [31 + d]: e^{-w d}, 0 for d < 0
    float col[32];                                      // forward e^{-w (31-i)}, reversed e^{-w i}
    unsigned long long full, qk, qs, kt, u, pr, o, xr, of, drain[2];
    unsigned tmem;
    int abort;
};

template <int D>
constexpr int tc_smem_bytes() {
    return (int)sizeof(TcSmem<D>) + 1024;
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
// a, b rounded to bfloat16 (returned) and what the rounding left out.
__device__ __forceinline__ uint32_t split_bf16(float& a, float& b) {
    const uint32_t h = pack_bf16(a, b);
    const float2 r = add2(f2(a, b), f2(-__uint_as_float(h << 16), -__uint_as_float(h & 0xffff0000u)));
    a = r.x;
    b = r.y;
    return h;
}

template <int D, bool OUT>
__global__ void __launch_bounds__(kTcThreads, D == 64 ? 2 : 1) decay_attn_tc_kernel(const __grid_constant__ TcParams P) {
    using Sm = TcSmem<D>;
    constexpr int C = kTcChunk, SUB = Sm::kSub, SUBB = 128 * 128;
    constexpr uint32_t kCols = D == 64 ? 256 : 512;
    constexpr uint32_t kColO = 128, kColU = 128 + D;
    constexpr int NX = D == 64 ? 32 : 128;              // state values of a thread
    extern __shared__ __align__(1024) char smem_raw[];
    Sm& S = *reinterpret_cast<Sm*>(smem_raw + ((1024u - (tc::smem_u32(smem_raw) & 1023u)) & 1023u));
    const Params& p = P.p;
    const int prob = blockIdx.x % p.nprob;
    const Problem& pr = p.pr[prob];
    const int sid = blockIdx.x / p.nprob, seg = sid % p.nseg, bh = sid / p.nseg, b = bh / p.H, h = bh % p.H;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const float w = __ldg(p.w + h);
    const int n_seq = seq_tokens(p.lengths, b, p.T);
    const int t0 = seg * p.seg_tokens;
    const int n = seg_count(n_seq, seg, p.seg_tokens);
    const int t_end = min(t0 + p.seg_tokens, p.T) - t0;
    const int rev = pr.reverse, e0 = rev ? 0 : 1;
    const int nchunk = (n + C - 1) / C;
    const bool has_in = pr.x_in != nullptr, has_out = pr.x_out != nullptr;
    const size_t xo = ((size_t)bh * p.nseg + seg) * D * D;

    if (tid == 0) {
        tc::mbar_init(&S.full, 1);
        tc::mbar_init(&S.qk, 1);
        tc::mbar_init(&S.qs, 1);
        tc::mbar_init(&S.kt, 4);
        tc::mbar_init(&S.u, 1);
        tc::mbar_init(&S.pr, 4);
        tc::mbar_init(&S.o, 1);
        tc::mbar_init(&S.xr, 4);
        tc::mbar_init(&S.of, 4);
        tc::mbar_init(&S.drain[0], 1);
        tc::mbar_init(&S.drain[1], 1);
        S.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    for (int i = tid; i <= C; i += kTcThreads) S.pw[i] = decay_pow(w, i);
    if (tid < 64) S.diag[tid] = tid < 31 ? 0.f : decay_pow(w, tid - 31);
    if (tid < 32) S.col[tid] = decay_pow(w, rev ? tid : 31 - tid);
    if (warp == 4) tc::tmem_alloc(&S.tmem, kCols);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = S.tmem;
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
    // chunk ci of the walk: its first token in the segment, and its tokens
    auto first = [&](int ci) { return (rev ? nchunk - 1 - ci : ci) * C; };

    constexpr uint32_t kIdA = tc::idesc_bf16(128, 128, false, false);
    constexpr uint32_t kIdX = tc::idesc_bf16(128, D, false, false);
    constexpr uint32_t kIdP = tc::idesc_bf16(128, D, false, true);
    constexpr uint32_t kIdU = tc::idesc_bf16(128, D, true, true);
    const uint32_t sq = tc::smem_u32(S.q), sk = tc::smem_u32(S.k), sv = tc::smem_u32(S.v);
    int loading = -1;     // (issuing lanes) chunk whose tiles are on their way
    bool issued = false;  // (issuing lanes) MMAs were issued
    auto load = [&](int ci) {
        const int t = t0 + first(ci);
        loading = ci;
        tc::mbar_expect_tx(&S.full, (OUT ? 3 : 2) * Sm::kTile);
#pragma unroll
        for (int s = 0; s < SUB; ++s) {
            const int c = h * D + 64 * s;
            tc::tma_load_3d(sk + s * SUBB, &P.map[P.mk[prob]], c, t, b, &S.full);
            if (OUT) tc::tma_load_3d(sq + s * SUBB, &P.map[P.mq[prob]], c, t, b, &S.full);
            tc::tma_load_3d(sv + s * SUBB, &P.map[P.mv[prob]], c, t, b, &S.full);
        }
    };
    // A and, from the state, O
    auto issue_front = [&](int ci) {
        if (!wait(S.full, ci)) return;
        tc::fence_after();
        issued = true;
#pragma unroll
        for (int s = 0; s < SUB; ++s) {
            const uint64_t a = tc::sw128_desc(sq + s * SUBB, 16), bb = tc::sw128_desc(sk + s * SUBB, 16);
#pragma unroll
            for (int k = 0; k < 4; ++k) tc::mma_ss(tmem, a + 2 * k, bb + 2 * k, kIdA, s + k > 0);
        }
        tc::commit(&S.qk);
        if (ci == 0 && !has_in) return;
        if (!wait(S.xr, ci) || (ci > 0 && !wait(S.of, ci - 1))) return;
        tc::fence_after();
#pragma unroll
        for (int half = 0; half < 2; ++half)
#pragma unroll
            for (int s = 0; s < SUB; ++s) {
                const uint64_t a = tc::sw128_desc(sq + s * SUBB, 16);
                const uint64_t bb = tc::sw128_desc(tc::smem_u32(half ? S.xl : S.xh) + s * D * 128, 16);
#pragma unroll
                for (int k = 0; k < 4; ++k) tc::mma_ss(tmem + kColO, a + 2 * k, bb + 2 * k, kIdX, half + s + k > 0);
            }
        tc::commit(&S.qs);
    };
    // O += P v, once P is there and v's tile is clean
    auto issue_pv = [&](int ci) {
        if (!wait(S.pr, ci) || !wait(S.kt, ci)) return;
        tc::fence_after();
        const bool with_x = ci > 0 || has_in;
        const uint64_t bb = tc::sw128_desc(sv, SUBB);
#pragma unroll
        for (int k = 0; k < C / 16; ++k)
#pragma unroll
            for (int half = 0; half < 2; ++half)
                tc::mma_ts(tmem + kColO, tmem + 32 * (k / 2) + 16 * half + 8 * (k % 2), bb + 128 * k, kIdP,
                           with_x || k + half > 0);
        tc::commit(&S.o);
    };
    auto issue_u = [&](int ci) {
        if (!wait(S.kt, ci)) return;
        tc::fence_after();
        issued = true;
        // rows of v^T beyond D = 64: the tile once more
        const uint64_t a = tc::sw128_desc(sv, D == 64 ? 0 : SUBB);
#pragma unroll
        for (int piece = 0; piece < 3; ++piece) {
            const uint64_t bb =
                tc::sw128_desc(piece == 0 ? tc::smem_u32(S.kh) : piece == 1 ? tc::smem_u32(S.km) : sk, SUBB);
#pragma unroll
            for (int k = 0; k < C / 16; ++k)
                tc::mma_ss(tmem + kColU, a + 128 * k, bb + 128 * k, kIdU, piece + k > 0);
        }
        tc::commit(&S.u);
    };
    // abort: what an issuing lane started ends before the CTA's memory is given back
    auto drain = [&](int which) {
        const unsigned long long s0 = tc::global_ns();
        while (loading >= 0 && !tc::mbar_test(&S.full, (unsigned)loading & 1u) && tc::global_ns() - s0 <= P.wait_ns) {
        }
        if (!issued) return;
        tc::commit(&S.drain[which]);
        while (!tc::mbar_test(&S.drain[which], 0) && tc::global_ns() - s0 <= 2 * P.wait_ns) {
        }
    };

    if (warp < 4) {
        // P, O: thread = token row of the chunk
        if (OUT) {
            const int row = tid;
            if (tid == 0 && nchunk > 0) load(0);
            const uint32_t lanes = tmem + ((uint32_t)(warp * 32) << 16);
            for (int ci = 0; ci < nchunk; ++ci) {
                const int a = first(ci), m = min(C, n - a);
                const bool with_x = ci > 0 || has_in;
                if (tid == 0) issue_front(ci);
                __syncwarp();
                if (!wait_warp(S.qk, ci)) break;
                tc::fence_after();
#pragma unroll 1
                for (int j = 0; j < 4; ++j) {
                    uint32_t out[32];
                    const int dj = rev ? j - warp : warp - j;  // blocks back in (walked) time
                    if (dj < 0 || 32 * j >= m) {
#pragma unroll
                        for (int i = 0; i < 32; ++i) out[i] = 0u;
                    } else {
                        float v[32];
                        tc::tmem_ld32(lanes + 32 * j, v);
                        if (dj == 0) {
                            const float* dg = S.diag + 31 + (rev ? -lane : lane);
#pragma unroll
                            for (int i = 0; i < 32; ++i) {
                                const bool keep = rev ? i >= lane : i <= lane;
                                v[i] = keep ? v[i] * dg[rev ? i : -i] * pr.scale_intra : 0.f;
                            }
                        } else {
                            const float f = S.pw[rev ? 32 * dj - lane : 32 * dj - 31 + lane] * pr.scale_intra;
#pragma unroll
                            for (int i = 0; i < 32; i += 4) {
                                const float4 c = *reinterpret_cast<const float4*>(S.col + i);
                                v[i] *= c.x * f;
                                v[i + 1] *= c.y * f;
                                v[i + 2] *= c.z * f;
                                v[i + 3] *= c.w * f;
                            }
                        }
                        if (32 * j + 32 > m) {  // columns past the chunk's tokens
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if (32 * j + i >= m) v[i] = 0.f;
                        }
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            out[i] = split_bf16(v[2 * i], v[2 * i + 1]);
                            out[16 + i] = pack_bf16(v[2 * i], v[2 * i + 1]);
                        }
                    }
                    tc::tmem_st32(lanes + 32 * j, out);
                }
                if (with_x) {
                    if (!wait_warp(S.qs, ci - (has_in ? 0 : 1))) break;
                    tc::fence_after();
                    const float f = S.pw[max(rev ? m - 1 - row : row, 0) + e0] * pr.scale_inter;
#pragma unroll 1
                    for (int c = 0; c < D; c += 32) {
                        float v[32];
                        uint32_t out[32];
                        tc::tmem_ld32(lanes + kColO + c, v);
#pragma unroll
                        for (int i = 0; i < 32; ++i) out[i] = __float_as_uint(v[i] * f);
                        tc::tmem_st32(lanes + kColO + c, out);
                    }
                }
                tc::tmem_wait_st();
                tc::fence_before();
                arrive_warp(S.pr);
                if (tid == 0) issue_pv(ci);
                __syncwarp();
                if (!wait_warp(S.o, ci)) break;
                tc::fence_after();
                if (tid == 0 && ci + 1 < nchunk && wait(S.u, ci)) load(ci + 1);  // the tiles are free
                __syncwarp();
                char* dst = pr.out + (((size_t)b * p.T + t0 + a + row) * p.H + h) * D * 2;
#pragma unroll 1
                for (int c = 0; c < D; c += 32) {
                    float v[32];
                    tc::tmem_ld32(lanes + kColO + c, v);
                    if (row < m) {
#pragma unroll
                        for (int i = 0; i < 32; i += 8)
                            *reinterpret_cast<uint4*>(dst + (c + i) * 2) =
                                make_uint4(pack_bf16(v[i], v[i + 1]), pack_bf16(v[i + 2], v[i + 3]),
                                           pack_bf16(v[i + 4], v[i + 5]), pack_bf16(v[i + 6], v[i + 7]));
                    }
                }
                tc::fence_before();
                arrive_warp(S.of);
            }
            if (tid == 0 && *abort) drain(0);
            // rows past the sequence's end
            for (int x = tid; x < (t_end - n) * (D / 8); x += 128)
                *reinterpret_cast<uint4*>(pr.out + (((size_t)b * p.T + t0 + n + x / (D / 8)) * p.H + h) * D * 2 +
                                          (x % (D / 8)) * 16) = make_uint4(0u, 0u, 0u, 0u);
        }
    } else {
        // K~ and X: thread = row of X^T (v channel) and, for D = 64, half of its columns (k channels)
        const int tw = tid - 128, jr = D == 64 ? tw & 63 : tw, c0 = D == 64 ? (tw >> 6) * 32 : 0;
        const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        float X[NX];
        if (has_in) {
            const float* x = pr.x_in + xo;
#pragma unroll
            for (int i = 0; i < NX; ++i) X[i] = __ldg(pr.x_in_t ? x + (size_t)jr * D + c0 + i : x + (size_t)(c0 + i) * D + jr);
        } else {
#pragma unroll
            for (int i = 0; i < NX; ++i) X[i] = 0.f;
        }
        // X^T as operands: row jr, 16-byte piece c of 64 channels at piece c ^ (jr & 7)
        auto store_x = [&]() {
#pragma unroll
            for (int i = 0; i < NX; i += 8) {
                const int c = c0 + i;
                const uint32_t off = (c / 64) * D * 128 + jr * 128 + ((((c % 64) / 8) ^ (jr & 7)) << 4);
                float v[8];
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = X[i + e];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    hi[e] = split_bf16(v[2 * e], v[2 * e + 1]);
                    lo[e] = pack_bf16(v[2 * e], v[2 * e + 1]);
                }
                *reinterpret_cast<uint4*>(S.xh + off) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                *reinterpret_cast<uint4*>(S.xl + off) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
            }
            tc::fence_async_smem();
            arrive_warp(S.xr);
        };
        if (OUT) store_x();
        else if (tw == 0 && nchunk > 0) load(0);
        bool okay = true;
        for (int ci = 0; ci < nchunk; ++ci) {
            const int m = min(C, n - first(ci));
            const bool update = ci + 1 < nchunk || has_out;
            okay = wait_warp(S.full, ci);
            if (!okay) break;
            if (m < C) {  // rows of v past the chunk's tokens meet zeros of P and K~: 0 * NaN is NaN
                for (int x = tw; x < (C - m) * 8 * SUB; x += 128)
                    *reinterpret_cast<uint4*>(S.v + (x / ((C - m) * 8)) * SUBB + (m + x % ((C - m) * 8) / 8) * 128 +
                                              (x % 8) * 16) = make_uint4(0u, 0u, 0u, 0u);
            }
            if (update) {
                if (OUT) {  // A is done with k's own tile, which takes the third piece
                    okay = wait_warp(S.qk, ci);
                    if (!okay) break;
                }
#pragma unroll 4
                for (int i = 0; i < 8 * SUB; ++i) {  // 16-byte pieces of a thread
                    const int x = i * 128 + tw, r = (x % 1024) / 8;
                    const uint32_t off = x * 16;
                    const float f = S.pw[rev ? r + 1 : max(m - 1 - r, 0)] * pr.scale_upd;
                    const uint4 raw = *reinterpret_cast<const uint4*>(S.k + off);
                    const uint32_t rw[4] = {raw.x, raw.y, raw.z, raw.w};
                    uint32_t hi[4], mi[4], lo[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float x0 = __uint_as_float(rw[e] << 16) * f, x1 = __uint_as_float(rw[e] & 0xffff0000u) * f;
                        if (r >= m) x0 = x1 = 0.f;
                        hi[e] = split_bf16(x0, x1);
                        mi[e] = split_bf16(x0, x1);
                        lo[e] = pack_bf16(x0, x1);
                    }
                    *reinterpret_cast<uint4*>(S.kh + off) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                    *reinterpret_cast<uint4*>(S.km + off) = make_uint4(mi[0], mi[1], mi[2], mi[3]);
                    *reinterpret_cast<uint4*>(S.k + off) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                }
            }
            tc::fence_async_smem();
            arrive_warp(S.kt);
            if (!update) break;
            if (tw == 0) issue_u(ci);
            __syncwarp();
            okay = wait_warp(S.u, ci);
            if (!okay) break;
            tc::fence_after();
            if (!OUT && tw == 0 && ci + 1 < nchunk) load(ci + 1);
            const float fx = S.pw[m];
#pragma unroll
            for (int c = 0; c < NX; c += 32) {
                float v[32];
                tc::tmem_ld32(lanes + kColU + c0 + c, v);
#pragma unroll
                for (int i = 0; i < 32; ++i) X[c + i] = fmaf(fx, X[c + i], v[i]);
            }
            tc::fence_before();
            if (OUT && ci + 1 < nchunk) {
                // O = q X of this chunk has read the operands
                if (ci > 0 || has_in) okay = wait_warp(S.qs, ci - (has_in ? 0 : 1));
                if (!okay) break;
                store_x();
            }
        }
        if (tw == 0 && *abort) drain(1);
        if (has_out && okay) {
            float* x = pr.x_out + xo;
#pragma unroll
            for (int i = 0; i < NX; ++i) x[pr.x_out_t ? (size_t)jr * D + c0 + i : (size_t)(c0 + i) * D + jr] = X[i];
        }
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    if (warp == 4) tc::tmem_free(tmem, kCols);
}

}  // namespace decay
}  // namespace vrwkv
