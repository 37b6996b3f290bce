// bfloat16 heads whose channels are not whole 16-byte vectors cannot be read by
// TMA.  For wider ones and longer sequences their rows are first spread to heads
// of W channels, zeros past D, in the workspace, and the outputs gathered from
// there afterwards; the tcgen05 kernels see heads of W.  Element by element on
// the narrow side, a warp four heads' rows at a time, two channels a lane: bound
// by those loads' and stores' number.  Measured at 3 x 7518, 15 heads of 89, the
// whole forward call: 369 us, as they are 1.74 ms (floor 37).
#pragma once

#include "common.cuh"

namespace vrwkv {
namespace decay {

struct PackParams {
    const char* src[4];
    char* dst[4];
    long long ld[4];        // row strides of the narrow side, in elements
    long long heads;        // B * T * H
    int H, D, W;
};

// TO_WIDE: src rows of ld elements -> dst (rows, H, W); else src (rows, H, W) -> dst rows of ld elements.
template <bool TO_WIDE>
__global__ void __launch_bounds__(256) decay_pack_kernel(const PackParams p) {
    using U = unsigned short;
    using U2 = ushort2;
    constexpr int R = 4;  // heads' rows of a warp at a time
    const int lane = threadIdx.x & 31, which = blockIdx.y;
    const U* src = reinterpret_cast<const U*>(p.src[which]);
    U* dst = reinterpret_cast<U*>(p.dst[which]);
    const long long ld = p.ld[which];
    for (long long i0 = (blockIdx.x * 8LL + (threadIdx.x >> 5)) * R; i0 < p.heads; i0 += gridDim.x * 8LL * R) {
        long long row = p.heads < (1LL << 31) ? (long long)((unsigned)i0 / (unsigned)p.H) : i0 / p.H;
        int h = (int)(i0 - row * p.H);
        long long narrow[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            narrow[r] = i0 + r < p.heads ? row * ld + (long long)h * p.D : -1;
            if (++h == p.H) h = 0, ++row;
        }
        for (int c = 2 * lane; c < p.W; c += 64) {
            U2 v[R];
#pragma unroll
            for (int r = 0; r < R; ++r) {
                v[r].x = v[r].y = 0;
                if (narrow[r] < 0) continue;
                if (!TO_WIDE) {
                    v[r] = __ldg(reinterpret_cast<const U2*>(src + (i0 + r) * p.W + c));
                } else {
                    if (c < p.D) v[r].x = __ldg(src + narrow[r] + c);
                    if (c + 1 < p.D) v[r].y = __ldg(src + narrow[r] + c + 1);
                }
            }
#pragma unroll
            for (int r = 0; r < R; ++r) {
                if (narrow[r] < 0) continue;
                if (TO_WIDE) {
                    *reinterpret_cast<U2*>(dst + (i0 + r) * p.W + c) = v[r];
                } else {
                    if (c < p.D) dst[narrow[r] + c] = v[r].x;
                    if (c + 1 < p.D) dst[narrow[r] + c + 1] = v[r].y;
                }
            }
        }
    }
}

}  // namespace decay
}  // namespace vrwkv
