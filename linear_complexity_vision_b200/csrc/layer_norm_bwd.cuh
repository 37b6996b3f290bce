// LayerNorm backward for sm_100a.  With xh = (x - mean) rstd and d = gamma gy per row:
//   gx = rstd (d - mean_c(d) - xh mean_c(d xh)),
//   ggamma = sum_rows gy xh,  gbeta = sum_rows gy.
// Bound by its bytes (x and gy read, gx written once).  Rows of at most 32
// channels a lane go to a warp each (layer_norm_bwd_warp_kernel): a row's two
// sums then cost 10 shuffles and no barrier, and the next row is on its way in
// registers while one is worked on.  Measured in a graph, both kernels of the
// call: 32768 x 1024 bfloat16 45.3 us, 12544 x 768 bfloat16 20.2, 6272 x 384
// float32 10.6, 32768 x 1024 float32 72.4 us (5.6 TB/s).  The same with the rows
// on their way in a ring of shared memory (bulk copies, four CTAs an SM): 46.7,
// 21.2, 11.0 and 78.9; with three CTAs and spills for wide float32 rows 126 us.
// bfloat16 rows of 1024 are bound by latency: 163 registers leave three warps a
// scheduler, which wait for shared memory (gamma) and the sums' shuffles more than
// for DRAM (1.5 and 0.3 of an instruction's stalls), issue 47 %.  Wider rows, or rows that are
// not made of aligned 16-byte vectors, go to a CTA each.  Either way a thread
// keeps the same channels of every row it visits, so their ggamma and gbeta stay
// in its registers; each CTA leaves one partial row of them, and
// layer_norm_wgrad_kernel adds those rows in a fixed order.
#pragma once

#include "common.cuh"
#include "layer_norm.cuh"
#include "passes.cuh"
#include "qshift.cuh"

namespace vrwkv {

struct LayerNormBwdParams {
    const char* x;
    const char* gy;
    char* gx;
    const float* g;
    const float* mean;
    const float* rstd;
    float* part;      // [gridDim.x][2][C], or nullptr without ggamma and gbeta
    long long rows;
    int C;
};

// One vector of N channels: 16 bytes, or a single element where rows are not
// made of aligned 16-byte vectors.
template <typename IO, bool VEC>
struct LnVec {
    static constexpr int N = VEC ? Vec16<IO>::N : 1;
    __device__ __forceinline__ static void load(const char* p, float (&f)[N]) {
        if constexpr (VEC) Vec16<IO>::unpack(*reinterpret_cast<const uint4*>(p), f);
        else f[0] = Io<IO>::ld1(p);
    }
    __device__ __forceinline__ static void store(char* p, const float (&f)[N]) {
        if constexpr (VEC) *reinterpret_cast<uint4*>(p) = Vec16<IO>::pack(f);
        else Io<IO>::st1(p, f[0]);
    }
};

// The N channels of a 16-byte vector as float pairs (paired FP32 instructions).
__device__ __forceinline__ void ln_pairs(const uint4& r, float2 (&f)[2], float) {
    f[0] = f2(__uint_as_float(r.x), __uint_as_float(r.y));
    f[1] = f2(__uint_as_float(r.z), __uint_as_float(r.w));
}
__device__ __forceinline__ void ln_pairs(const uint4& r, float2 (&f)[4], __nv_bfloat16) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = f2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
}

constexpr int kLnBwdWarps = 4;
// CTAs of an SM, by registers: the row at hand, the next one and the sums of
// gradients are 16 VPL + 2 E of them, and there are about 40 others.
template <typename IO>
constexpr int ln_bwd_ctas(int vpl) {
    const int regs = 40 + 16 * vpl + 2 * vpl * Vec16<IO>::N, fit = 65536 / (32 * kLnBwdWarps * regs);
    return fit < 6 ? fit : 6;
}

template <typename IO, int VPL>
__global__ void __launch_bounds__(32 * kLnBwdWarps, ln_bwd_ctas<IO>(VPL)) layer_norm_bwd_warp_kernel(const LayerNormBwdParams p) {
    using V = Vec16<IO>;
    constexpr int N = V::N, N2 = N / 2, E = VPL * N;  // channels of a lane: vectors lane + 32 k
    next_pass();
    extern __shared__ __align__(16) float sg[];  // gamma, then the CTA's partial rows: max(1, 2) * C floats
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int nv = p.C / N;
    for (int c = tid; c < p.C; c += 32 * kLnBwdWarps) sg[c] = __ldg(p.g + c);
    __syncthreads();
    float2 dg[E / 2], db[E / 2];
#pragma unroll
    for (int e = 0; e < E / 2; ++e) dg[e] = db[e] = f2(0.f);
    const float invC = 1.0f / (float)p.C;
    const size_t rowb = (size_t)p.C * sizeof(IO);
    const long long step = (long long)gridDim.x * kLnBwdWarps;
    long long row = (long long)blockIdx.x * kLnBwdWarps + warp;
    uint4 nx[VPL], ng[VPL];
    float nmean = 0.f, nrs = 0.f;
    auto fetch = [&](long long r) {
#pragma unroll
        for (int k = 0; k < VPL; ++k) {
            const int v = lane + 32 * k;
            nx[k] = ng[k] = make_uint4(0u, 0u, 0u, 0u);
            if (v < nv) {
                nx[k] = __ldcs(reinterpret_cast<const uint4*>(p.x + r * rowb) + v);
                ng[k] = __ldcs(reinterpret_cast<const uint4*>(p.gy + r * rowb) + v);
            }
        }
        nmean = __ldg(p.mean + r);
        nrs = __ldg(p.rstd + r);
    };
    if (row < p.rows) fetch(row);
    for (; row < p.rows; row += step) {
        uint4 cx[VPL], cg[VPL];
#pragma unroll
        for (int k = 0; k < VPL; ++k) {
            cx[k] = nx[k];
            cg[k] = ng[k];
        }
        const float mean = nmean, rs = nrs;
        if (row + step < p.rows) fetch(row + step);
        float2 a2 = f2(0.f), b2 = f2(0.f);
#pragma unroll
        for (int k = 0; k < VPL; ++k) {
            const int v = lane + 32 * k;
            if (v >= nv) continue;
            const float2* gg = reinterpret_cast<const float2*>(sg + v * N);
            float2 x[N2], y[N2];
            ln_pairs(cx[k], x, IO{});
            ln_pairs(cg[k], y, IO{});
#pragma unroll
            for (int e = 0; e < N2; ++e) {
                const float2 xh = mul2(add2(x[e], f2(-mean)), f2(rs)), d = mul2(gg[e], y[e]);
                a2 = add2(a2, d);
                b2 = fma2(d, xh, b2);
                dg[k * N2 + e] = fma2(y[e], xh, dg[k * N2 + e]);
                db[k * N2 + e] = add2(db[k * N2 + e], y[e]);
            }
        }
        const float a = warp_sum(a2.x + a2.y) * invC, b = warp_sum(b2.x + b2.y) * invC;
        // rs (g y - mean(d) - (x - mean) rs mean(d xh)), the row's constants joined
        const float c1 = -rs * rs * b, c0 = -rs * a;
#pragma unroll
        for (int k = 0; k < VPL; ++k) {
            const int v = lane + 32 * k;
            if (v >= nv) continue;
            const float2* gg = reinterpret_cast<const float2*>(sg + v * N);
            float2 x[N2], y[N2];
            float o[N];
            ln_pairs(cx[k], x, IO{});
            ln_pairs(cg[k], y, IO{});
#pragma unroll
            for (int e = 0; e < N2; ++e) {
                const float2 r = fma2(add2(x[e], f2(-mean)), f2(c1), fma2(mul2(f2(rs), gg[e]), y[e], f2(c0)));
                o[2 * e] = r.x;
                o[2 * e + 1] = r.y;
            }
            reinterpret_cast<uint4*>(p.gx + row * rowb)[v] = V::pack(o);
        }
    }
    if (!p.part) return;
    // the warps' sums, in order of the warps
    for (int w = 0; w < kLnBwdWarps; ++w) {
        __syncthreads();
        if (warp != w) continue;
#pragma unroll
        for (int k = 0; k < VPL; ++k) {
            const int v = lane + 32 * k;
            if (v >= nv) continue;
#pragma unroll
            for (int e = 0; e < N; ++e) {
                const int c = v * N + e;
                const float2 g2 = dg[k * N2 + e / 2], b2 = db[k * N2 + e / 2];
                sg[c] = (e & 1 ? g2.y : g2.x) + (w ? sg[c] : 0.f);
                sg[p.C + c] = (e & 1 ? b2.y : b2.x) + (w ? sg[p.C + c] : 0.f);
            }
        }
    }
    __syncthreads();
    for (int c = tid; c < 2 * p.C; c += 32 * kLnBwdWarps) p.part[(size_t)blockIdx.x * 2 * p.C + c] = sg[c];
}

template <typename IO, bool VEC, int NV>
__global__ void __launch_bounds__(1024) layer_norm_bwd_kernel(const LayerNormBwdParams p) {
    using V = LnVec<IO, VEC>;
    constexpr int N = V::N;
    next_pass();
    __shared__ float red[2][32][2];
    const int tid = threadIdx.x, nt = blockDim.x, warp = tid >> 5, lane = tid & 31, nw = nt >> 5;
    const int nv = p.C / N;
    const float invC = 1.0f / (float)p.C;
    float g[NV][N], dg[NV][N], db[NV][N];
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int e = 0; e < N; ++e) {
            const int v = tid + nt * k;
            g[k][e] = v < nv ? __ldg(p.g + v * N + e) : 0.f;
            dg[k][e] = db[k][e] = 0.f;
        }
    int buf = 0;
    for (long long row = blockIdx.x; row < p.rows; row += gridDim.x, buf ^= 1) {
        float xh[NV][N], gy[NV][N];
        const float rs = __ldg(p.rstd + row), mean = __ldg(p.mean + row);
        float a = 0.f, b = 0.f;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int v = tid + nt * k;
#pragma unroll
            for (int e = 0; e < N; ++e) xh[k][e] = gy[k][e] = 0.f;
            if (v >= nv) continue;
            const size_t o = ((size_t)row * p.C + (size_t)v * N) * sizeof(IO);
            V::load(p.x + o, xh[k]);
            V::load(p.gy + o, gy[k]);
#pragma unroll
            for (int e = 0; e < N; ++e) {
                xh[k][e] = (xh[k][e] - mean) * rs;
                const float d = g[k][e] * gy[k][e];
                a += d;
                b = fmaf(d, xh[k][e], b);
                dg[k][e] = fmaf(gy[k][e], xh[k][e], dg[k][e]);
                db[k][e] += gy[k][e];
            }
        }
        a = warp_sum(a);
        b = warp_sum(b);
        if (nw > 1) {
            // two buffers: the next row's sums cannot overtake this row's readers
            if (lane == 0) {
                red[buf][warp][0] = a;
                red[buf][warp][1] = b;
            }
            __syncthreads();
            a = b = 0.f;
            for (int q = 0; q < nw; ++q) {
                a += red[buf][q][0];
                b += red[buf][q][1];
            }
        }
        a *= invC;
        b *= invC;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int v = tid + nt * k;
            if (v >= nv) continue;
            float o[N];
#pragma unroll
            for (int e = 0; e < N; ++e) o[e] = rs * (fmaf(g[k][e], gy[k][e], -a) - xh[k][e] * b);
            V::store(p.gx + ((size_t)row * p.C + (size_t)v * N) * sizeof(IO), o);
        }
    }
    if (!p.part) return;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int v = tid + nt * k;
        if (v >= nv) continue;
        float* dst = p.part + (size_t)blockIdx.x * 2 * p.C + (size_t)v * N;
#pragma unroll
        for (int e = 0; e < N; ++e) {
            dst[e] = dg[k][e];
            dst[p.C + e] = db[k][e];
        }
    }
}

// ggamma[c], gbeta[c]: the sums of n partial rows of 2C floats.  A CTA takes 8
// of the 2C columns (a 32-byte sector of each row), its 128 groups of 8 threads
// every 128th row: the few hundred rows there are take one or two round trips
// to L2.
constexpr int kLnWgradCols = 8;

__global__ void __launch_bounds__(1024) layer_norm_wgrad_kernel(const float* part, int n, int C, float* ggamma,
                                                                float* gbeta) {
    __shared__ float sm[32][kLnWgradCols];
    const int tid = threadIdx.x, col = tid % kLnWgradCols, group = tid / kLnWgradCols;
    const int c = blockIdx.x * kLnWgradCols + col;
    float s = 0.f;
    last_pass();
    if (c < 2 * C) {
#pragma unroll 8
        for (int i = group; i < n; i += 1024 / kLnWgradCols) s += __ldcg(part + (size_t)i * 2 * C + c);
    }
    s += __shfl_xor_sync(0xffffffffu, s, 8);
    s += __shfl_xor_sync(0xffffffffu, s, 16);
    if ((tid & 31) < kLnWgradCols) sm[tid >> 5][col] = s;
    __syncthreads();
    if (tid >= 32 * kLnWgradCols) return;
    const int of = tid >> 5, cw = blockIdx.x * kLnWgradCols + of;
    const float t = warp_sum(sm[tid & 31][of]);  // column of of the CTA's 8
    if ((tid & 31) == 0 && cw < C) ggamma[cw] = t;
    else if ((tid & 31) == 0 && cw < 2 * C) gbeta[cw - C] = t;
}

}  // namespace vrwkv
