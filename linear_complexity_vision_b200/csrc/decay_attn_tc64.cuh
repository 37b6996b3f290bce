// Multi-head decay attention on the 5th-generation tensor cores for bfloat16
// heads of up to 64 channels (zero-padded to 64): the operator and the steps of
// a chunk are those of decay_attn_tc.cuh.  Here a persistent CTA (one per SM) keeps two chunks at
// work at a time, each on a stream of its own (tiles, tensor memory, 8 worker
// warps, an issuing warp), and walks all its work items, one head's segment
// after the other, without a break: the next item's tiles are loaded and its
// first chunk begins while the last one's is finished.  Only the state X is
// serial: four warps keep it in registers, add each chunk's U in turn and hand
// the operands of O = q X to the stream whose chunk is next.
//
// Measured: forward 8 x 4096, 16 heads: 73 us (floor 41.0: its bytes), one
// chunk 2.15 us of an SM; 128 of 148 SMs work, since one head's chunks are
// serial and a cut would form the states first (two segments: 120 us).
// Backward, three problems of it: 8 x 4096, 16 heads 210 us (floor 71.8), 64 x
// 196, 12 heads 68 us (20.6).  Issue slots are 45 % busy, the tensor pipe 28 to
// 36 %: bound by the latency of a chunk's steps, of which two overlap; a
// third stream has no tensor memory left.  One chunk at a time, in the manner
// of decay_attn_tc.cuh with two CTAs an SM: 8 x 4096 100 us.
//
// Roles (704 threads): warps 0-7 and 8-15 the workers of streams 0 and 1,
// warps 16-19 the state, warps 20-21 the issuers.  512 tensor-memory columns:
// per stream A / P 128, O 64, U 64.  Bounded waits as in decay_attn_tc.cuh; here
// only the state warps need the pass before, so a wait's time begins after it.
//
// A barrier is waited for by its phase's parity, so no phase may complete
// before every waiter has seen the one before.  That holds because each phase
// of a barrier needs an arrival that its waiters make after the last one: fa,
// fv, a, o need kt or pr of the stream's workers, u needs uf of the state
// warps, qs needs their xr.
#pragma once

#include "decay_attn_tc.cuh"

namespace vrwkv {
namespace decay {

constexpr int kT64Threads = 704;

struct alignas(1024) T64Smem {
    struct Tables {                  // of one work item
        float pw[kTcChunk + 4];      // e^{-w n}, n = 0 .. 128
        float col[kTcChunk];         // as TcSmem's
        float row[kTcChunk];
    };
    struct Stream {
        uint8_t q[16384], k[16384], v[16384], kh[16384], km[16384];
        uint8_t out[16384];          // the rows of O on their way out
    } st[2];
    uint8_t x[16384];                // X^T as operands of the next chunk, hi and lo
    Tables tab[2][2];                // [stream][item's turn]
    struct Bars {
        unsigned long long fa, fv, a, kt, u, pr, o, xr, of, uf, tb, qs, so, qk, drain;
    } bar[2];
    unsigned tmem;
    int abort;
};

constexpr int t64_smem_bytes() { return (int)sizeof(T64Smem) + 1024; }

// A work item: one head's segment of one problem.
struct T64Item {
    int prob, seg, h, b;  // its number's digits, the problem fastest
    int t0, n, nchunk, rev, has_in, has_out, fast;
    float w;
    __device__ __forceinline__ void at(const TcParams& P, int item) {
        const Params& p = P.p;
        prob = item % p.nprob;
        item /= p.nprob;
        seg = item % p.nseg;
        item /= p.nseg;
        h = item % p.H;
        b = item / p.H;
        fill(P);
    }
    // gridDim.x items on: digit by digit, without divisions
    __device__ __forceinline__ void step(const TcParams& P) {
        const Params& p = P.p;
        prob += P.step[0];
        seg += P.step[1];
        h += P.step[2];
        b += P.step[3];
        if (prob >= p.nprob) prob -= p.nprob, ++seg;
        if (seg >= p.nseg) seg -= p.nseg, ++h;
        if (h >= p.H) h -= p.H, ++b;
        if (b < p.B) fill(P);
    }
    __device__ __forceinline__ void fill(const TcParams& P) {
        const Params& p = P.p;
        w = __ldg(p.w + h);
        t0 = seg * p.seg_tokens;
        n = seg_count(seq_tokens(p.lengths, b, p.T), seg, p.seg_tokens);
        nchunk = (n + kTcChunk - 1) / kTcChunk;
        const Problem& pr = p.pr[prob];
        rev = pr.reverse;
        fast = factored(w, pr);
        has_in = pr.x_in != nullptr;
        has_out = pr.x_out != nullptr;
    }
    __device__ __forceinline__ long long state_at(const Params& p) const {
        return (((long long)b * p.H + h) * p.nseg + seg) * p.S * p.S;
    }
};

// A stream's walk over its chunks: every second one of the items' chunks in
// a row.
struct T64Cursor {
    int item, ci;
    T64Item it;
    __device__ __forceinline__ void start(const TcParams& P, int nitems, int stream) {
        item = blockIdx.x;
        ci = stream;
        it.at(P, item);
        settle(P, nitems);
    }
    __device__ __forceinline__ void next(const TcParams& P, int nitems) {
        ci += 2;
        settle(P, nitems);
    }
    __device__ __forceinline__ bool valid(int nitems) const { return item < nitems; }
    __device__ __forceinline__ void settle(const TcParams& P, int nitems) {
        while (ci >= it.nchunk) {
            ci -= it.nchunk;
            item += gridDim.x;
            if (item >= nitems) return;
            it.step(P);
        }
    }
    __device__ __forceinline__ int first() const { return (it.rev ? it.nchunk - 1 - ci : ci) * kTcChunk; }
    __device__ __forceinline__ int tokens() const { return min(kTcChunk, it.n - first()); }
    __device__ __forceinline__ bool more() const { return ci + 1 < it.nchunk; }  // the item has a next chunk
    __device__ __forceinline__ bool update() const { return more() || it.has_out; }
    __device__ __forceinline__ bool with_x() const { return ci > 0 || it.has_in; }
};

template <int PIECES>
__global__ void __launch_bounds__(kT64Threads, 1) decay_attn_tc64_kernel(const __grid_constant__ TcParams P) {
    constexpr int C = kTcChunk, D = 64;
    extern __shared__ __align__(1024) char smem_raw[];
    T64Smem& S = *reinterpret_cast<T64Smem*>(smem_raw + ((1024u - (tc::smem_u32(smem_raw) & 1023u)) & 1023u));
    const Params& p = P.p;
    const int nitems = P.nitems;
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;

    if (tid < 2) {
        T64Smem::Bars& B = S.bar[tid];
        tc::mbar_init(&B.fa, 1);
        tc::mbar_init(&B.fv, 1);
        tc::mbar_init(&B.a, 1);
        tc::mbar_init(&B.kt, 8);
        tc::mbar_init(&B.u, 1);
        tc::mbar_init(&B.pr, 8);
        tc::mbar_init(&B.o, 1);
        tc::mbar_init(&B.xr, 4);
        tc::mbar_init(&B.of, 8);
        tc::mbar_init(&B.uf, 4);
        tc::mbar_init(&B.tb, 8);
        tc::mbar_init(&B.qs, 1);
        tc::mbar_init(&B.qk, 1);
        tc::mbar_init(&B.so, 8);
        tc::mbar_init(&B.drain, 1);
        if (tid == 0) S.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 16) tc::tmem_alloc(&S.tmem, 512);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    volatile int* abort = &S.abort;
    auto wait = [&](unsigned long long& bar, int phase) {  // the whole warp
        bool w = tc::mbar_test(&bar, (unsigned)phase & 1u);
        if (!w) {
            last_pass();  // what the pass before still takes is not counted
            w = tc::wait_slow(&bar, (unsigned)phase & 1u, abort, P.err, kTcErr, P.wait_ns);
        }
        return __all_sync(0xffffffffu, w ? 1 : 0) != 0;
    };
    auto arrive = [&](unsigned long long& bar) {
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&bar);
    };

    if (warp < 16) {
        // ---- workers of a stream ----
        const int s = warp >> 3, wt = tid & 255, quad = warp & 3, wg = (warp >> 2) & 1;
        T64Smem::Stream& T = S.st[s];
        T64Smem::Bars& B = S.bar[s];
        const uint32_t lanes = S.tmem + (uint32_t)(s * 256) + ((uint32_t)(quad * 32) << 16);
        constexpr uint32_t kColO = 128;
        int tables_of = -1, turn = 0;                   // item whose tables are built, and how many were
        T64Cursor cu;
        cu.start(P, nitems, s);
        for (int ph = 0; cu.valid(nitems); ++ph) {      // ph: chunks of this stream so far
            const T64Item& it = cu.it;
            const Problem& pr = p.pr[it.prob];
            const bool fast = it.fast;
            const int rev = it.rev, m = cu.tokens();
            const bool update = cu.update();
            if (tables_of != cu.item) {
                // the other buffer: its last readers are past the barrier of the tables in use
                ++turn;
                tables_of = cu.item;
                T64Smem::Tables& N = S.tab[s][turn & 1];
                const DecayBase w = decay_base(it.w);
                if (wt <= C) N.pw[wt] = decay_pow(w, wt);
                if (wt < C) {
                    if (fast) {
                        N.col[wt] = decay_pow(w, rev ? wt - 63 : 63 - wt) * pr.scale_intra;
                    } else if (wt < 32) {
                        N.col[wt] = decay_pow(w, rev ? wt : 31 - wt) * pr.scale_intra;
                    }
                } else {
                    const int i = wt - C;
                    if (fast) {
                        N.row[i] = decay_pow(w, rev ? 63 - i : i - 63);
                    } else if (i < 64) {
                        const int d = rev ? i - 31 : 31 - i;
                        N.row[i] = d < 0 ? 0.f : decay_pow(w, d) * pr.scale_intra;
                    }
                }
                arrive(B.tb);
                if (!wait(B.tb, turn - 1)) break;
            }
            const T64Smem::Tables& N = S.tab[s][turn & 1];
            if (!wait(B.fa, ph)) break;
            if (m < C) {  // rows of v past the chunk's tokens meet zeros of P and K~: 0 * NaN is NaN
                if (!wait(B.fv, ph)) break;
                for (int x = wt; x < (C - m) * 8; x += 256)
                    *reinterpret_cast<uint4*>(T.v + (m + x / 8) * 128 + (x % 8) * 16) = make_uint4(0u, 0u, 0u, 0u);
            }
            if (update) {
                if (PIECES == 3 && !wait(B.qk, ph)) break;  // the third piece takes k's own tile
                uint4 raws[4];
                float fs[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {  // 16-byte pieces of a thread
                    const int x = i * 256 + wt, r = x / 8;
                    raws[i] = *reinterpret_cast<const uint4*>(T.k + x * 16);
                    fs[i] = N.pw[rev ? r + 1 : max(m - 1 - r, 0)] * pr.scale_upd;
                    if (r >= m) raws[i] = make_uint4(0u, 0u, 0u, 0u);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t off = (i * 256 + wt) * 16;
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
                    *reinterpret_cast<uint4*>(T.kh + off) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                    *reinterpret_cast<uint4*>(T.km + off) = make_uint4(mi[0], mi[1], mi[2], mi[3]);
                    if (PIECES == 3) *reinterpret_cast<uint4*>(T.k + off) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                }
            }
            tc::fence_async_smem();
            arrive(B.kt);
            if (!wait(B.a, ph)) break;
            tc::fence_after();
            // P: this warpgroup's blocks of the quarter's rows, d4 blocks back in (walked) time
            const int wq = rev ? 3 - quad : quad;       // blocks off the diagonal in this quarter
#pragma unroll
            for (int jj = 0; jj < 2; ++jj) {
                const int d4 = wg == 0 ? 3 * jj : 1 + jj;
                const int j = rev ? (quad + d4) & 3 : (quad - d4) & 3;
                if (d4 > wq || 32 * j >= m) {           // before the sequence's start, or past the chunk's end
                    tc::tmem_zero<32>(lanes + 32 * j);
                    continue;
                }
                p_block(lanes + 32 * j, j, d4, fast, rev, lane, m, N.pw, N.col, N.row);
            }
            const int row = quad * 32 + lane;
            if (!fast && cu.with_x()) {
                const float2 f = f2(N.pw[rev ? max(m - 1 - row, 0) : row + 1] * pr.scale_inter);
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
            arrive(B.pr);
            if (!wait(B.o, ph)) break;
            tc::fence_after();
            float v[32];
            tc::tmem_ld32(lanes + kColO + wg * 32, v);
            tc::fence_before();
            arrive(B.of);
            // into the tile that TMA stores; rows past the chunk's tokens are zeros
            const float2 f = f2(fast ? N.row[row] : 1.0f);
#pragma unroll
            for (int i = 0; i < 32; i += 8) {
                uint32_t o[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 x = mul2(f2(v[i + 2 * e], v[i + 2 * e + 1]), f);
                    o[e] = row < m ? pack_bf16(x) : 0u;
                }
                *reinterpret_cast<uint4*>(T.out + row * 128 + (((wg * 4 + i / 8) ^ (row & 7)) << 4)) =
                    make_uint4(o[0], o[1], o[2], o[3]);
            }
            tc::fence_async_smem();
            arrive(B.so);
            cu.next(P, nitems);
        }
        // whole blocks of rows past the sequences' ends
        if (p.lengths) {
            T64Item it;
            it.at(P, blockIdx.x);
            for (int item = blockIdx.x; item < nitems; item += gridDim.x, it.step(P)) {
                const int r0 = it.nchunk * C, rows = min(p.seg_tokens, p.T - it.t0) - r0;
                const int vecs = p.D / 8;
                for (int x = tid; x < rows * vecs; x += 512)
                    *reinterpret_cast<uint4*>(p.pr[it.prob].out +
                                              (((size_t)it.b * p.T + it.t0 + r0 + x / vecs) * p.H + it.h) * p.D * 2 +
                                              (x % vecs) * 16) = make_uint4(0u, 0u, 0u, 0u);
            }
        }
    } else if (warp < 20) {
        // ---- the state: thread = half a row of X^T (v channel jr, k channels c0 ..); U has its rows twice ----
        last_pass();
        constexpr int NX = 32;
        const int quad = warp & 3, jr = (quad & 1) * 32 + lane, c0 = (quad >> 1) * NX;
        const uint32_t lanes = S.tmem + ((uint32_t)(quad * 32) << 16) + 192 + c0;
        int g = 0;                                       // chunks so far
        int uphase[2] = {0, 0}, stored[2] = {0, 0}, last = 0;  // operands stored, the stream of the last
        bool okay = true;
        T64Item it;
        it.at(P, blockIdx.x);
        for (int item = blockIdx.x; item < nitems && okay; item += gridDim.x, it.step(P)) {
            const Problem& pr = p.pr[it.prob];
            const DecayBase w = decay_base(it.w);
            const bool fast = it.fast;
            const long long xo = it.state_at(p);
            float X[NX];
            if (it.has_in) {
                load_x(X, pr.x_in + xo, pr.x_in_t, jr, c0, p.S);
            } else {
#pragma unroll
                for (int i = 0; i < NX; ++i) X[i] = 0.f;
            }
            const float full = decay_pow(w, C);
            // X^T as the operand of a chunk of m tokens: row jr, 16-byte piece c at piece c ^ (jr & 7)
            auto store_x = [&](int m, int stream) {
                const float2 f = f2(fast ? decay_pow(w, it.rev ? m - 64 : 64) * pr.scale_inter : 1.0f);
#pragma unroll
                for (int i = 0; i < NX; i += 8) {
                    const uint32_t off = jr * 128 + ((((c0 + i) / 8) ^ (jr & 7)) << 4);
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float2 x = mul2(f2(X[i + 2 * e], X[i + 2 * e + 1]), f);
                        hi[e] = split_bf16(x);
                        lo[e] = pack_bf16(x);
                    }
                    *reinterpret_cast<uint4*>(S.x + off) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                    *reinterpret_cast<uint4*>(S.x + 8192 + off) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                }
                tc::fence_async_smem();
                arrive(S.bar[stream].xr);
            };
            // after the last O = q X has read the buffer (a barrier of its own: a
            // may be a chunk without X ahead)
            auto next_x = [&](int m, int stream) {
                if (stored[0] + stored[1] > 0 && !wait(S.bar[last].qs, stored[last] - 1)) return false;
                store_x(m, stream);
                ++stored[stream];
                last = stream;
                return true;
            };
            // tokens of chunk ci of the walk
            auto tokens = [&](int ci) { return min(C, it.n - (it.rev ? it.nchunk - 1 - ci : ci) * C); };
            if (it.has_in && it.nchunk > 0) okay = next_x(tokens(0), g & 1);
            if (!okay) break;
            for (int ci = 0; ci < it.nchunk; ++ci, ++g) {
                const int s = g & 1, m = tokens(ci);
                const bool more = ci + 1 < it.nchunk;
                if (more || it.has_out) {
                    okay = wait(S.bar[s].u, uphase[s]++);
                    if (!okay) break;
                    tc::fence_after();
                    const float2 fx = f2(m == C ? full : decay_pow(w, m));
                    float v[NX];
                    tc::tmem_ld32(lanes + s * 256, v);
#pragma unroll
                    for (int i = 0; i < NX; i += 2) {
                        const float2 x = fma2(fx, f2(X[i], X[i + 1]), f2(v[i], v[i + 1]));
                        X[i] = x.x;
                        X[i + 1] = x.y;
                    }
                    tc::fence_before();
                    arrive(S.bar[s].uf);
                }
                if (more) okay = next_x(tokens(ci + 1), s ^ 1);
                if (!okay) break;
            }
            if (it.has_out && okay) store_x_out(X, pr.x_out + xo, pr.x_out_t, jr, c0, p.S);
        }
    } else {
        // ---- issuer of a stream ----
        const int s = warp - 20;
        T64Smem::Stream& T = S.st[s];
        T64Smem::Bars& B = S.bar[s];
        const uint32_t tmem = S.tmem + (uint32_t)(s * 256);
        constexpr uint32_t kIdA = tc::idesc_bf16(128, 128, false, false);
        constexpr uint32_t kIdX = tc::idesc_bf16(128, D, false, false);
        constexpr uint32_t kIdP = tc::idesc_bf16(128, D, false, true);
        constexpr uint32_t kIdU = tc::idesc_bf16(128, D, true, true);
        const uint32_t sq = tc::smem_u32(T.q), sk = tc::smem_u32(T.k), sv = tc::smem_u32(T.v);
        const uint32_t skh = tc::smem_u32(T.kh), skm = tc::smem_u32(T.km);
        const uint32_t sxh = tc::smem_u32(S.x), sxl = sxh + 8192, sout = tc::smem_u32(T.out);
        auto load = [&](uint32_t dst, int map, const T64Cursor& c, unsigned long long* bar) {
            tc::tma_load_4d(dst, &P.map[map], 0, c.it.h, c.it.t0 + c.first(), c.it.b, bar);
        };
        auto load_q = [&](const T64Cursor& c) {         // begins fa's phase; k completes it
            tc::mbar_expect_tx(&B.fa, 2 * 16384);
            load(sq, P.mq[c.it.prob], c, &B.fa);
        };
        auto load_k = [&](const T64Cursor& c) { load(sk, P.mk[c.it.prob], c, &B.fa); };
        auto load_v = [&](const T64Cursor& c) {
            tc::mbar_expect_tx(&B.fv, 16384);
            load(sv, P.mv[c.it.prob], c, &B.fv);
        };
        int loads_a = 0, loads_v = 0, xphase = 0, uphase = 0;
        bool issued = false;
        T64Cursor cu, nx;
        cu.start(P, nitems, s);
        if (cu.valid(nitems)) {
            if (tc::elect_one()) {
                load_q(cu);
                load_k(cu);
                load_v(cu);
            }
            __syncwarp();
            loads_a = loads_v = 1;
        }
        // the finished chunk's output tile; the lane that begins stores also waits for them
        int out_map = 0, out_h = 0, out_t = 0, out_b = 0, out_ph = -1;
        auto store_out = [&]() {
            if (out_ph < 0) return true;
            if (!wait(B.so, out_ph)) return false;
            if (tc::elect_one()) tc::tma_store_4d(&P.omap[out_map], sout, 0, out_h, out_t, out_b);
            __syncwarp();
            out_ph = -1;
            return true;
        };
        for (int ph = 0; cu.valid(nitems); ++ph) {
            nx = cu;
            nx.next(P, nitems);
            const bool next = nx.valid(nitems), update = cu.update(), with_x = cu.with_x();
            if (!wait(B.fa, ph)) break;
            tc::fence_after();
            issued = true;
            if (tc::elect_one()) {                      // A = q k^T
                const uint64_t da = tc::sw128_desc(sq, 16), db = tc::sw128_desc(sk, 16);
#pragma unroll
                for (int k = 0; k < 4; ++k) tc::mma_ss(tmem, da + 2 * k, db + 2 * k, kIdA, k > 0);
                if (PIECES == 3) tc::commit(&B.qk);
                if (!with_x) tc::commit(&B.a);
            }
            __syncwarp();
            auto issue_x = [&]() {                      // O = q X
                tc::fence_after();
                if (tc::elect_one()) {
                    const uint64_t da = tc::sw128_desc(sq, 16);
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const uint64_t db = tc::sw128_desc(half ? sxl : sxh, 16);
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            tc::mma_ss(tmem + 128, da + 2 * k, db + 2 * k, kIdX, half + k > 0);
                    }
                    tc::commit(&B.qs);
                    tc::commit(&B.a);
                }
                __syncwarp();
            };
            auto x_ready = [&]() {
                return __all_sync(0xffffffffu, tc::mbar_ready(&B.xr, (unsigned)xphase & 1u) ? 1 : 0) != 0;
            };
            // U does not wait for X: what is ready first goes first
            if (ph > 0 && !wait(B.of, ph - 1)) break;   // O's columns are read
            if (!store_out()) break;
            bool x_due = with_x;
            if (x_due && x_ready()) {
                issue_x();
                x_due = false;
            }
            if (!wait(B.kt, ph) || !wait(B.fv, ph)) break;
            if (x_due && x_ready()) {
                issue_x();
                x_due = false;
            }
            if (update) {                               // U = v^T K~
                if (uphase > 0 && !wait(B.uf, uphase - 1)) break;
                ++uphase;
                tc::fence_after();
                if (tc::elect_one()) {
                    const uint64_t da = tc::sw128_desc(sv, 0);  // 64 rows of v^T, twice
#pragma unroll
                    for (int piece = 0; piece < PIECES; ++piece) {
                        const uint64_t db = tc::sw128_desc(piece == 0 ? skh : piece == 1 ? skm : sk, 16384);
#pragma unroll
                        for (int k = 0; k < C / 16; ++k)
                            tc::mma_ss(tmem + 192, da + 128 * k, db + 128 * k, kIdU, piece + k > 0);
                    }
                    tc::commit(&B.u);
                }
                __syncwarp();
            }
            if (x_due) {
                if (!wait(B.xr, xphase)) break;
                issue_x();
            }
            if (with_x) ++xphase;
            if (next) {                                 // q's tile is read, and k's or nearly
                if (!wait(B.a, ph)) break;
                if (tc::elect_one()) {
                    load_q(nx);
                    if (PIECES < 3) load_k(nx);
                }
                ++loads_a;
                __syncwarp();
            }
            if (!wait(B.pr, ph)) break;
            tc::fence_after();
            if (tc::elect_one()) {                      // O += P v
                const uint64_t db = tc::sw128_desc(sv, 16384);
                const uint32_t acc = with_x ? 1u : 0u;
#pragma unroll
                for (int k = 0; k < C / 16; ++k)
#pragma unroll
                    for (int half = 0; half < 2; ++half)
                        tc::mma_ts(tmem + 128, tmem + 16 * k + 8 * half, db + 128 * k, kIdP, k + half > 0 ? 1u : acc);
                tc::tma_store_wait(false);              // the output tile is free
                tc::commit(&B.o);
            }
            __syncwarp();
            if (!wait(B.o, ph)) break;                  // also: A's columns are free for the next chunk
            if (next) {
                // U has read v's tile and k's third piece (u is the state warps' to follow; uf comes after it)
                if (update && !wait(B.u, uphase - 1)) break;
                if (tc::elect_one()) {
                    if (PIECES == 3) load_k(nx);
                    load_v(nx);
                }
                ++loads_v;
                __syncwarp();
            }
            out_map = cu.it.prob;
            out_h = cu.it.h;
            out_t = cu.it.t0 + cu.first();
            out_b = cu.it.b;
            out_ph = ph;
            cu = nx;
        }
        store_out();
        if (tc::elect_one()) tc::tma_store_wait(true);
        __syncwarp();
        if (*abort) {
            // what was begun ends before the CTA's memory is given back
            const unsigned long long s0 = tc::global_ns();
            while (loads_a > 0 && !(tc::mbar_test(&B.fa, (unsigned)(loads_a - 1) & 1u) &&
                                    tc::mbar_test(&B.fv, (unsigned)(loads_v - 1) & 1u)) &&
                   tc::global_ns() - s0 <= P.wait_ns) {
            }
            __syncwarp();
            if (issued) {
                if (tc::elect_one()) tc::commit(&B.drain);
                __syncwarp();
                while (!tc::mbar_test(&B.drain, 0) && tc::global_ns() - s0 <= 2 * P.wait_ns) {
                }
            }
        }
        __syncwarp();
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    if (warp == 16) tc::tmem_free(S.tmem, 512);
}

}  // namespace decay
}  // namespace vrwkv
