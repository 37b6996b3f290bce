// LayerNorm backward for sm_100a.  With xh = (x - mean) rstd and d = gamma gy per row:
//   gx = rstd (d - mean_c(d) - xh mean_c(d xh)),
//   ggamma = sum_rows gy xh,  gbeta = sum_rows gy.
// Bound by its bytes (x and gy read, gx written once).  A CTA holds RB whole
// rows in registers (each thread the same NV vectors of every row, so the
// columns' sums stay in its registers over all rows it visits), reduces the
// rows' two sums together, and leaves one partial row of ggamma and gbeta;
// layer_norm_wgrad_kernel adds the partial rows in a fixed order.
#pragma once

#include "common.cuh"
#include "layer_norm.cuh"
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

template <typename IO, bool VEC, int NV, int RB, int MAXT>
__global__ void __launch_bounds__(MAXT) layer_norm_bwd_kernel(const LayerNormBwdParams p) {
    using V = LnVec<IO, VEC>;
    constexpr int N = V::N;
    __shared__ float red[2][32][2 * RB];
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
    for (long long r0 = (long long)blockIdx.x * RB; r0 < p.rows; r0 += (long long)gridDim.x * RB, buf ^= 1) {
        float xh[RB][NV][N], gy[RB][NV][N], rs[RB], s[2 * RB];
#pragma unroll
        for (int r = 0; r < RB; ++r)
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int v = tid + nt * k;
#pragma unroll
                for (int e = 0; e < N; ++e) xh[r][k][e] = gy[r][k][e] = 0.f;
                if (r0 + r < p.rows && v < nv) {
                    const size_t o = ((size_t)(r0 + r) * p.C + (size_t)v * N) * sizeof(IO);
                    V::load(p.x + o, xh[r][k]);
                    V::load(p.gy + o, gy[r][k]);
                }
            }
#pragma unroll
        for (int r = 0; r < RB; ++r) {
            const bool live = r0 + r < p.rows;
            rs[r] = live ? __ldg(p.rstd + r0 + r) : 0.f;
            const float mean = live ? __ldg(p.mean + r0 + r) : 0.f;
            float a = 0.f, b = 0.f;
#pragma unroll
            for (int k = 0; k < NV; ++k)
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    xh[r][k][e] = (xh[r][k][e] - mean) * rs[r];
                    const float d = g[k][e] * gy[r][k][e];
                    a += d;
                    b = fmaf(d, xh[r][k][e], b);
                    dg[k][e] = fmaf(gy[r][k][e], xh[r][k][e], dg[k][e]);
                    db[k][e] += gy[r][k][e];
                }
            s[2 * r] = warp_sum(a);
            s[2 * r + 1] = warp_sum(b);
        }
        if (nw > 1) {
            // two buffers: the next rows' sums cannot overtake this row's readers
            if (lane == 0)
#pragma unroll
                for (int i = 0; i < 2 * RB; ++i) red[buf][warp][i] = s[i];
            __syncthreads();
#pragma unroll
            for (int i = 0; i < 2 * RB; ++i) {
                s[i] = 0.f;
                for (int q = 0; q < nw; ++q) s[i] += red[buf][q][i];
            }
        }
#pragma unroll
        for (int r = 0; r < RB; ++r) {
            if (r0 + r >= p.rows) break;
            const float a = s[2 * r] * invC, b = s[2 * r + 1] * invC;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int v = tid + nt * k;
                if (v >= nv) continue;
                float o[N];
#pragma unroll
                for (int e = 0; e < N; ++e) o[e] = rs[r] * (fmaf(g[k][e], gy[r][k][e], -a) - xh[r][k][e] * b);
                V::store(p.gx + ((size_t)(r0 + r) * p.C + (size_t)v * N) * sizeof(IO), o);
            }
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

// ggamma[c], gbeta[c]: the sums of n partial rows of 2C floats.  A CTA takes
// 32 of the 2C columns; its 32 warps take every 32nd row.
__global__ void __launch_bounds__(1024) layer_norm_wgrad_kernel(const float* part, int n, int C, float* ggamma,
                                                                float* gbeta) {
    __shared__ float sm[32][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    float s = 0.f;
    if (c < 2 * C)
        for (int i = warp; i < n; i += 32) s += part[(size_t)i * 2 * C + c];
    sm[warp][lane] = s;
    __syncthreads();
    const float t = warp_sum(sm[lane][warp]);  // column warp of the CTA's 32
    const int cw = blockIdx.x * 32 + warp;
    if (lane == 0 && cw < C) ggamma[cw] = t;
    else if (lane == 0 && cw < 2 * C) gbeta[cw - C] = t;
}

}  // namespace vrwkv
