// Multi-head decay attention on the 5th-generation tensor cores for float32
// heads of up to 64 channels, whole 16-byte vectors, zero-padded to 64: the
// operator of decay_attn.cuh (the same problems, segments and states) in chunks of 128 tokens, as in decay_attn_tc.cuh.
//
// A float32 value is exactly the sum of three bfloat16 pieces h + m + l, each
// the rounded remainder of the last.  A product is taken as the six products
// of pieces down to 2^-16 of the first,
//   hh + (hm + mh + mm + hl + lh);
// what is left out is below 2^-23 of it.  The tensor cores truncate when they
// add to an accumulator, so hh, four or eight additions long, has an
// accumulator of its own, and the five small ones share another, whose
// truncations are 2^-8 smaller; the two meet on the FP32 pipes.
//
// Per chunk (all in tensor memory unless said):
//   A  = q K'^T     (128 x 128, two accumulators)
//   O  = q X        (128 x 64, two)     X^T in registers, pieces in shared memory
//   P  = mask(A)    as three pieces, in the columns A had
//   O += P v
//   U  = v^T K'     (twice 64 x 64, two)
//   X^T = e^{-w m} X^T + c U            in registers
// Where |w| <= 1/2, K' = scale_intra e^{-w (63 - s)} k (reversed: s - 63): A then
// has every decay but the row's e^{-w (t - 63)}, which multiplies the finished
// row, and the same K' serves U (c = e^{-w (m - 64)} scale_upd / scale_intra).
// Faster decays take K' = k for A, P with the decays of a table by t - s, O = q X
// scaled by rows, and then K' = scale_upd e^{-w (..)} k for U.
//
// 16 working warps (a warp's number mod 4: its quarter of the rows; its
// warpgroup: a block of P's columns, 16 columns of O, 16 of U) and one that
// issues.  The next chunk's rows are brought to L2 as soon as v is there; the
// workers read, split and write them to shared memory in the swizzled layout (any
// row stride that keeps 16-byte alignment), v behind A; the next chunk's q and k
// are split while P v runs, the first one's while barriers, tables and tensor
// memory are set up.
// 168 KB of shared memory, all of tensor memory, one CTA per SM.  Bounded waits
// as in decay_attn_tc.cuh.
//
// Measured: 32 x 196 ragged, 6 heads: 32.9 us (floor 4.7: its bytes); backward 3
// x 1001, 6 heads, eight segments: 49.2 us (3.7); the kernel for any size takes
// 52 and 62 us.  A chunk takes 6.3 us, a CTA of one chunk 10 us.  The working
// warps are busy 5.5 us of a chunk: splitting q, k and v 2.4 with their loads
// from L2, P 1.4, X and the output 0.8; the products, fed from shared memory,
// run beside that.  Loads begun earlier, and v's held in registers, spill (96 a
// thread): 37.9 and 52.3 us.
#pragma once

#include "decay_attn_tc.cuh"

namespace vrwkv {
namespace decay {

constexpr int kTfThreads = 544;

template <bool OUT>
struct alignas(1024) TfSmem {
    static constexpr int kTile = 128 * 128;      // bytes of a token tile's piece
    uint8_t k[3][kTile], v[3][kTile];
    uint8_t q[OUT ? 3 : 1][OUT ? kTile : 1024];
    uint8_t x[OUT ? 3 : 1][OUT ? 8192 : 1024];   // X^T: rows v channel, K-major
    float pw[kTcChunk + 4];                      // e^{-w n}, n = 0 .. 128
    float col[kTcChunk];                         // fast: the factors of K'
    float row[kTcChunk];                         // fast: the rows' factors
    unsigned long long kt, kt2, kv, a, qx, u, pr, o, xr, of, rd[4], drain;
    unsigned tmem;
    int abort;
};
template <bool OUT>
constexpr int tf_smem_bytes() {
    return (int)sizeof(TfSmem<OUT>) + 1024;
}

template <bool OUT>
__global__ void __launch_bounds__(kTfThreads, 1) decay_attn_tcf_kernel(const __grid_constant__ TcParams P) {
    using Sm = TfSmem<OUT>;
    constexpr int C = kTcChunk, D = 64, NW = 16, kWork = 512, kTile = Sm::kTile;
    constexpr uint32_t kColO = 256, kColU = OUT ? 384 : 0, kCols = OUT ? 512 : 128;
    extern __shared__ __align__(1024) char smem_raw[];
    Sm& S = *reinterpret_cast<Sm*>(smem_raw + ((1024u - (tc::smem_u32(smem_raw) & 1023u)) & 1023u));
    const Params& p = P.p;
    const int prob = blockIdx.x % p.nprob;
    const Problem& pr = p.pr[prob];
    const int sid = blockIdx.x / p.nprob, seg = sid % p.nseg, bh = sid / p.nseg, b = bh / p.H, h = bh % p.H;
    next_pass();
    if (!OUT && seg == pr.skip) return;
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31, quad = warp & 3, wg = warp >> 2;
    const bool issuer = warp == NW;
    const float w = __ldg(p.w + h);
    const DecayBase base = decay_base(w);
    const bool fast = factored(w, pr);           // K' carries the scale, which the state's update takes out again
    const int n_seq = seq_tokens(p.lengths, b, p.T);
    const int t0 = seg * p.seg_tokens;
    const int n = seg_count(n_seq, seg, p.seg_tokens);
    const int t_end = min(t0 + p.seg_tokens, p.T) - t0;
    const int rev = pr.reverse, e0 = rev ? 0 : 1;
    const int nchunk = (n + C - 1) / C;
    const bool has_in = pr.x_in != nullptr, has_out = pr.x_out != nullptr;
    const int d = p.D;                           // channels there are; operands are zero past them
    const size_t xo = ((size_t)bh * p.nseg + seg) * p.S * p.S;

    // chunk ci of the walk: its first token in the segment
    auto first = [&](int ci) { return (rev ? nchunk - 1 - ci : ci) * C; };

    // two 16-byte vectors (8 channels) of a tile a thread: rows vr, vr + 64, channels 8 vc ..
    const int vr = tid / 8, vc = tid % 8;
    const uint32_t voff = vr * 128 + ((vc ^ (vr & 7)) << 4);  // the second is 64 rows on: the same swizzle
    const size_t row0 = (size_t)b * p.T + t0;
    auto source = [&](int which, int token) {
        const char* x = which == 0 ? pr.q : which == 1 ? pr.k : pr.v;
        const long long ld = which == 0 ? pr.ldq : which == 1 ? pr.ldk : pr.ldv;
        return reinterpret_cast<const float4*>(x + ((row0 + token) * (size_t)ld + h * d + 8 * vc) * 4);
    };
    auto fetch = [&](int which, int i, int a, int m, float (&x)[8]) {
        float4 lo = make_float4(0.f, 0.f, 0.f, 0.f), hi = lo;
        if (vr + 64 * i < m) {
            const float4* src = source(which, a + vr + 64 * i);
            if (8 * vc < d) lo = __ldg(src);
            if (8 * vc + 4 < d) hi = __ldg(src + 1);
        }
        x[0] = lo.x, x[1] = lo.y, x[2] = lo.z, x[3] = lo.w, x[4] = hi.x, x[5] = hi.y, x[6] = hi.z, x[7] = hi.w;
    };
    auto prefetch = [&](int ci, int from) {             // q, k, v from the from-th on
        const int a = first(ci), m = min(C, n - a);
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (vr + 64 * i < m && 8 * vc < d) {
#pragma unroll
                for (int which = 0; which < 3; ++which)
                    if (which >= from) asm volatile("prefetch.global.L2 [%0];" ::"l"(source(which, a + vr + 64 * i)));
            }
    };
    // 8 values times f as the three pieces' vectors at off
    auto put = [&](uint8_t* p0, uint8_t* p1, uint8_t* p2, uint32_t off, const float* x, float f) {
        uint32_t w0[4], w1[4], w2[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float2 y = mul2(f2(x[2 * e], x[2 * e + 1]), f2(f));
            w0[e] = split_bf16(y);
            w1[e] = split_bf16(y);
            w2[e] = pack_bf16(y);
        }
        *reinterpret_cast<uint4*>(p0 + off) = make_uint4(w0[0], w0[1], w0[2], w0[3]);
        *reinterpret_cast<uint4*>(p1 + off) = make_uint4(w1[0], w1[1], w1[2], w1[3]);
        *reinterpret_cast<uint4*>(p2 + off) = make_uint4(w2[0], w2[1], w2[2], w2[3]);
    };
    // the first chunk's q and k are on their way before all else
    float rq[2][8], rk[2][8];
    if (!issuer && nchunk > 0) {
        const int a = first(0), m = min(C, n - a);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (OUT) fetch(0, i, a, m, rq[i]);
            fetch(1, i, a, m, rk[i]);
        }
        prefetch(0, 2);
    }

    if (tid == 0) {
        tc::mbar_init(&S.kt, NW);
        tc::mbar_init(&S.kt2, NW);
        tc::mbar_init(&S.kv, NW);
        tc::mbar_init(&S.a, 1);
        tc::mbar_init(&S.qx, 1);
        tc::mbar_init(&S.u, 1);
        tc::mbar_init(&S.pr, NW);
        tc::mbar_init(&S.o, 1);
        tc::mbar_init(&S.xr, NW);
        tc::mbar_init(&S.of, NW);
        for (int i = 0; i < 4; ++i) tc::mbar_init(&S.rd[i], 4);
        tc::mbar_init(&S.drain, 1);
        S.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) tc::tmem_alloc(&S.tmem, kCols);
    if (tid <= C) S.pw[tid] = decay_pow(base, tid);
    if (tid < C) {
        S.col[tid] = decay_pow(base, rev ? tid - 63 : 63 - tid) * pr.scale_intra;
        S.row[tid] = decay_pow(base, rev ? 63 - tid : tid - 63);
    }

    volatile int* abort = &S.abort;
    auto wait = [&](unsigned long long& bar, int phase) {  // the whole warp
        const bool ok = tc::mbar_test(&bar, (unsigned)phase & 1u) ||
                        tc::wait_slow(&bar, (unsigned)phase & 1u, abort, P.err, kTcErr, P.wait_ns);
        return __all_sync(0xffffffffu, ok ? 1 : 0) != 0;
    };
    auto arrive = [&](unsigned long long& bar) {
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&bar);
    };

    // X: row jr of X^T (a v channel), columns c0 .. (k channels); U has its rows twice
    constexpr int NX = D * D / kWork;
    const int jr = (quad & 1) * 32 + lane, c0 = ((quad >> 1) * 4 + wg) * NX;
    float X[NX];
    last_pass();
    if (has_in && !issuer) {
        load_x(X, pr.x_in + xo, pr.x_in_t, jr, c0, p.S);
    } else {
#pragma unroll
        for (int i = 0; i < NX; ++i) X[i] = 0.f;
    }

    // factors of a whole chunk; a shorter one has its own
    const float x_full = fast ? decay_pow(base, 64) * pr.scale_inter : 1.0f;
    const float u_scale = fast ? pr.scale_upd / pr.scale_intra : 1.0f;
    const float u_full = fast ? decay_pow(base, 64) * u_scale : 1.0f;
    // X^T as the operand of a chunk of m tokens
    auto store_x = [&](int m) {
        const float f = fast && rev && m < C ? decay_pow(base, m - 64) * pr.scale_inter : x_full;
#pragma unroll
        for (int i = 0; i < NX; i += 8) {
            const uint32_t off = jr * 128 + ((((c0 + i) / 8) ^ (jr & 7)) << 4);
            put(S.x[0], S.x[OUT ? 1 : 0], S.x[OUT ? 2 : 0], off, X + i, f);
        }
    };
    // q's and k's pieces; f: K' 's factor of a row
    auto put_qk = [&](auto f) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t off = voff + i * 64 * 128;
            if (OUT) put(S.q[0], S.q[OUT ? 1 : 0], S.q[OUT ? 2 : 0], off, rq[i], 1.0f);
            put(S.k[0], S.k[1], S.k[2], off, rk[i], f(vr + 64 * i));
        }
        tc::fence_async_smem();
    };
    if (!issuer && nchunk > 0) {
        const int m = min(C, n - first(0));
        if (OUT && has_in) store_x(m);
        put_qk([&](int r) {
            return fast ? decay_pow(base, rev ? r - 63 : 63 - r) * pr.scale_intra
                   : OUT ? 1.0f : decay_pow(base, rev ? r + 1 : max(m - 1 - r, 0)) * pr.scale_upd;
        });
    }
    __syncthreads();  // tables, barriers, tensor memory's address, the first chunk's pieces
    tc::fence_after();
    if (!issuer && nchunk > 0) {
        if (OUT && has_in) arrive(S.xr);
        arrive(S.kt);
    }
    const uint32_t tmem = S.tmem;
    const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16);

    if (issuer) {
        constexpr uint32_t kIdA = tc::idesc_bf16(128, 128, false, false);
        constexpr uint32_t kIdX = tc::idesc_bf16(128, D, false, false);
        constexpr uint32_t kIdP = tc::idesc_bf16(128, D, false, true);
        constexpr uint32_t kIdU = tc::idesc_bf16(128, D, true, true);
        // hh and hm at once, B's pieces h and m side by side as are the two accumulators
        constexpr uint32_t kIdA2 = tc::idesc_bf16(128, 256, false, false);
        constexpr uint32_t kIdX2 = tc::idesc_bf16(128, 2 * D, false, false);
        constexpr uint32_t kIdP2 = tc::idesc_bf16(128, 2 * D, false, true);
        constexpr uint32_t kIdU2 = tc::idesc_bf16(128, 2 * D, true, true);
        // the products of pieces: hh into an accumulator (and hm), the others into the next
        constexpr int kPa[5] = {0, 1, 1, 0, 2}, kPb[5] = {0, 0, 1, 2, 0};
        const uint32_t sq = tc::smem_u32(S.q), sk = tc::smem_u32(S.k), sv = tc::smem_u32(S.v), sx = tc::smem_u32(S.x);
        bool issued = false;
        auto issue_u = [&]() {                          // U = v^T K'
#pragma unroll
            for (int i = 0; i < 5; ++i) {
                const uint64_t da = tc::sw128_desc(sv + kPa[i] * kTile, 0), db = tc::sw128_desc(sk + kPb[i] * kTile, kTile);
#pragma unroll
                for (int k = 0; k < C / 16; ++k)
                    tc::mma_ss(tmem + kColU + (i ? 64 : 0), da + 128 * k, db + 128 * k, i ? kIdU : kIdU2, i > 0 || k > 0);
            }
            tc::commit(&S.u);
        };
        for (int ci = 0; ci < nchunk; ++ci) {
            const bool more = ci + 1 < nchunk, update = more || has_out, with_x = ci > 0 || has_in;
            if (!wait(S.kt, ci)) break;
            if (OUT && ci > 0 && !wait(S.o, ci - 1)) break;  // P, in A's columns, is read
            tc::fence_after();
            issued = true;
            if (tc::elect_one()) {
                if (OUT) {
#pragma unroll
                    for (int i = 0; i < 5; ++i) {       // A = q K'^T
                        const uint64_t da = tc::sw128_desc(sq + kPa[i] * kTile, 16), db = tc::sw128_desc(sk + kPb[i] * kTile, 16);
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            tc::mma_ss(tmem + (i ? 128 : 0), da + 2 * k, db + 2 * k, i ? kIdA : kIdA2, i > 0 || k > 0);
                    }
                    tc::commit(&S.a);
                }
            }
            __syncwarp();
            if (OUT && with_x && (!wait(S.xr, ci - (has_in ? 0 : 1)) || (ci > 0 && !wait(S.of, ci - 1)))) break;
            if (OUT && !with_x && ci > 0 && !wait(S.of, ci - 1)) break;
            if (!wait(S.kv, ci)) break;
            tc::fence_after();
            if (tc::elect_one()) {
                if (OUT) {
                    if (with_x) {
#pragma unroll
                        for (int i = 0; i < 5; ++i) {   // O = q X
                            const uint64_t da = tc::sw128_desc(sq + kPa[i] * kTile, 16), db = tc::sw128_desc(sx + kPb[i] * 8192, 16);
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                tc::mma_ss(tmem + kColO + (i ? 64 : 0), da + 2 * k, db + 2 * k, i ? kIdX : kIdX2, i > 0 || k > 0);
                        }
                        tc::commit(&S.qx);
                    }
                }
                if (update && fast) issue_u();
            }
            __syncwarp();
            if (update && !fast) {
                if (!wait(S.kt2, ci)) break;
                tc::fence_after();
                if (tc::elect_one()) issue_u();
                __syncwarp();
            }
            if (OUT) {
                if (!wait(S.pr, ci)) break;
                tc::fence_after();
                if (tc::elect_one()) {                  // O += P v
                    const uint32_t acc = with_x ? 1u : 0u;
#pragma unroll
                    for (int i = 0; i < 5; ++i) {
                        const uint64_t db = tc::sw128_desc(sv + kPb[i] * kTile, kTile);
#pragma unroll
                        for (int k = 0; k < C / 16; ++k)
                            tc::mma_ts(tmem + kColO + (i ? 64 : 0), tmem + 64 * (k / 2) + 16 * kPa[i] + 8 * (k % 2), db + 128 * k,
                                       i ? kIdP : kIdP2, i > 0 || k > 0 ? 1u : acc);
                    }
                    tc::commit(&S.o);
                }
                __syncwarp();
            }
        }
        if (*abort && issued) {
            // what was begun ends before the CTA's memory is given back
            const unsigned long long s0 = tc::global_ns();
            if (tc::elect_one()) tc::commit(&S.drain);
            __syncwarp();
            while (!tc::mbar_test(&S.drain, 0) && tc::global_ns() - s0 <= P.wait_ns) {
            }
        }
        __syncwarp();
    }

    int ci = 0;
    for (; ci < nchunk && !issuer; ++ci) {
        const int a = first(ci), m = min(C, n - a);
        const bool more = ci + 1 < nchunk, update = more || has_out, with_x = OUT && (ci > 0 || has_in);
        // v's pieces; q's and k's were formed while the chunk before ended
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float rv[8];
            fetch(2, i, a, m, rv);
            put(S.v[0], S.v[1], S.v[2], voff + i * 64 * 128, rv, 1.0f);
        }
        tc::fence_async_smem();
        arrive(S.kv);
        if (more) prefetch(ci + 1, OUT ? 0 : 1);
        if (!OUT && !fast && update) arrive(S.kt2);     // K' was U's at once
        if (OUT) {
            if (!wait(S.a, ci)) break;
            tc::fence_after();
            if (!fast && update) {                      // A is done with k: now U's K'
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int r = vr + 64 * i;
                    float rk[8];
                    fetch(1, i, a, m, rk);
                    put(S.k[0], S.k[1], S.k[2], voff + i * 64 * 128, rk,
                        S.pw[rev ? r + 1 : max(m - 1 - r, 0)] * pr.scale_upd);
                }
                tc::fence_async_smem();
                arrive(S.kt2);
            }
            // P: this warpgroup's block of the quarter's rows, wg blocks back in (walked) time
            const int wq = rev ? 3 - quad : quad, j = rev ? (quad + wg) & 3 : (quad - wg) & 3;
            // block j of P: hi, mid, lo in columns 64 j, + 16, + 32, of A's first accumulator
            // (blocks 0, 1) and second (2, 3): every column is read before any is written
            const int row = quad * 32 + lane;
            const bool live = wg <= wq && 32 * j < m;
            float v[32];
            if (live) {
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    float y[16], s[16];
                    tc::tmem_ld16_pair(lanes + 32 * j + 16 * half, y, lanes + 128 + 32 * j + 16 * half, s);
#pragma unroll
                    for (int i = 0; i < 16; i += 2) {
                        const float2 x = add2(f2(y[i], y[i + 1]), f2(s[i], s[i + 1]));
                        v[16 * half + i] = x.x;
                        v[16 * half + i + 1] = x.y;
                    }
                }
                if (!fast) {
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        const int c = 32 * j + i;
                        v[i] *= S.pw[max(rev ? c - row : row - c, 0)] * pr.scale_intra;
                    }
                }
                if (wg == 0) {                          // the diagonal block: columns in the row's future
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (rev ? i < lane : i > lane) v[i] = 0.f;
                }
                if (32 * j + 32 > m) {                  // columns past the chunk's tokens
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (32 * j + i >= m) v[i] = 0.f;
                }
            }
            tc::fence_before();
            arrive(S.rd[quad]);                         // the quarter's four warps have read
            if (!wait(S.rd[quad], ci)) break;
            tc::fence_after();
            if (live) {
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    uint32_t hi[8], mi[8], lo[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        float2 x = f2(v[16 * half + 2 * i], v[16 * half + 2 * i + 1]);
                        hi[i] = split_bf16(x);
                        mi[i] = split_bf16(x);
                        lo[i] = pack_bf16(x);
                    }
                    tc::tmem_st8(lanes + 64 * j + 8 * half, hi);
                    tc::tmem_st8(lanes + 64 * j + 16 + 8 * half, mi);
                    tc::tmem_st8(lanes + 64 * j + 32 + 8 * half, lo);
                }
            } else {
                tc::tmem_zero<48>(lanes + 64 * j);
            }
            if (!fast && with_x) {
                if (!wait(S.qx, ci - (has_in ? 0 : 1))) break;
                tc::fence_after();
                const float2 f = f2(S.pw[max(rev ? m - 1 - row : row, 0) + e0] * pr.scale_inter);
#pragma unroll
                for (int part = 0; part < 2; ++part) {
                    float y[16];
                    uint32_t out[16];
                    tc::tmem_ld16(lanes + kColO + 64 * part + wg * 16, y);
#pragma unroll
                    for (int i = 0; i < 16; i += 2) {
                        const float2 x = mul2(f2(y[i], y[i + 1]), f);
                        out[i] = __float_as_uint(x.x);
                        out[i + 1] = __float_as_uint(x.y);
                    }
                    tc::tmem_st16(lanes + kColO + 64 * part + wg * 16, out);
                }
            }
            tc::tmem_wait_st();
            tc::fence_before();
            arrive(S.pr);
        }
        if (update) {
            if (!wait(S.u, ci)) break;
            tc::fence_after();
            const float fx = S.pw[m];
            const float c = fast && !rev && m < C ? decay_pow(base, m - 64) * u_scale : u_full;
            float y[8], s[8];
            tc::tmem_ld8_pair(lanes + kColU + c0, y, lanes + kColU + 64 + c0, s);
#pragma unroll
            for (int i = 0; i < NX; ++i) X[i] = fmaf(fx, X[i], c * (y[i] + s[i]));
            tc::fence_before();
            if (OUT && more) {
                store_x(min(C, n - first(ci + 1)));
                tc::fence_async_smem();
                arrive(S.xr);
            }
            if (more) {  // U was the last to read k, and followed O = q X: the next chunk's, while P v runs
                const int a2 = first(ci + 1), m2 = min(C, n - a2);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    if (OUT) fetch(0, i, a2, m2, rq[i]);
                    fetch(1, i, a2, m2, rk[i]);
                }
                put_qk([&](int r) {
                    return fast ? S.col[r] : OUT ? 1.0f : S.pw[rev ? r + 1 : max(m2 - 1 - r, 0)] * pr.scale_upd;
                });
                arrive(S.kt);
            }
        }
        if (OUT) {
            if (!wait(S.o, ci)) break;
            tc::fence_after();
            const int row = quad * 32 + lane;
            const float f = fast ? S.row[row] : 1.0f;
            char* dst = pr.out + ((((size_t)b * p.T + t0 + a + row) * p.H + h) * d + wg * 16) * 4;
            const int here = d - wg * 16;               // channels there are
            float y[16], s[16];
            tc::tmem_ld16_pair(lanes + kColO + wg * 16, y, lanes + kColO + 64 + wg * 16, s);
            tc::fence_before();
            arrive(S.of);
#pragma unroll
            for (int i = 0; i < 16; i += 8) {
                uint32_t o[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) o[e] = __float_as_uint((y[i + e] + s[i + e]) * f);
                if (row >= m) continue;
                if (P.wide_out) {
                    if (i < here) st_global_32(dst + 4 * i, o);
                } else {
                    if (i < here) *reinterpret_cast<uint4*>(dst + 4 * i) = make_uint4(o[0], o[1], o[2], o[3]);
                    if (i + 4 < here) *reinterpret_cast<uint4*>(dst + 4 * i + 16) = make_uint4(o[4], o[5], o[6], o[7]);
                }
            }
        }
    }
    if (has_out && !issuer && ci == nchunk) store_x_out(X, pr.x_out + xo, pr.x_out_t, jr, c0, p.S);
    if (OUT) {  // rows past the sequence's end
        for (int x = tid; x < (t_end - n) * (d / 4); x += kTfThreads)
            *reinterpret_cast<uint4*>(pr.out + ((((size_t)b * p.T + t0 + n + x / (d / 4)) * p.H + h) * d + (x % (d / 4)) * 4) * 4) =
                make_uint4(0u, 0u, 0u, 0u);
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    if (warp == 1) tc::tmem_free(tmem, kCols);
}

}  // namespace decay
}  // namespace vrwkv
