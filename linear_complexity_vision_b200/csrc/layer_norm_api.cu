// C ABI of LayerNorm (declared in include/vrwkv.h): host-side argument
// validation and kernel launches.  Validation happens before any CUDA call.
#include <algorithm>
#include <cstdint>

#include "api_internal.h"
#include "layer_norm.cuh"
#include "layer_norm_bwd.cuh"

namespace vrwkv {
namespace api {

vrwkv_status launch_layer_norm(const LayerNormParams& in, vrwkv_dtype dtype, cudaStream_t s) {
    LayerNormParams p = in;
    const size_t row = (size_t)p.C * elem_bytes(dtype);
    p.vec = row % 16 == 0 && aligned(p.x, 16) && aligned(p.y, 16);
    const unsigned blocks = (unsigned)((p.rows + 7) / 8);
    // 16-byte vectors per lane of the register-resident kernel (0: three-pass)
    const int vpl = (p.vec && aligned(p.g, 16) && aligned(p.b, 16)) ? (int)((row / 16 + 31) / 32) : 0;
    auto launch_ln = [&](auto io) {
        using IO = decltype(io);
        if (vpl >= 1 && vpl <= 1) layer_norm_reg_kernel<IO, 1><<<blocks, 256, 0, s>>>(p);
        else if (vpl == 2) layer_norm_reg_kernel<IO, 2><<<blocks, 256, 0, s>>>(p);
        else if (vpl >= 3 && vpl <= 4) layer_norm_reg_kernel<IO, 4><<<blocks, 256, 0, s>>>(p);
        else if (vpl >= 5 && vpl <= 8) layer_norm_reg_kernel<IO, 8><<<blocks, 256, 0, s>>>(p);
        else layer_norm_kernel<IO><<<blocks, 256, 0, s>>>(p);
    };
    if (dtype == VRWKV_F32) launch_ln(float{});
    else launch_ln(__nv_bfloat16{});
    return cuda_status(cudaGetLastError(), "layer_norm_kernel launch");
}

}  // namespace api
}  // namespace vrwkv

namespace {

using namespace vrwkv;
using namespace vrwkv::api;

constexpr int kLnMaxC = 1 << 30;  // a lane's steps of 32 channels stay an int
constexpr int kLnBwdMaxC = 8192;

// Geometry of the backward pass: a warp per row (vpl vectors a lane) or, with
// vpl = 0, a CTA per row (nv vectors a thread); threads of a CTA; CTAs.
struct LnBwdPlan {
    bool vec;
    int vpl, nv, threads, grid;
};

LnBwdPlan ln_bwd_plan(long long rows, int C, int es, bool vec) {
    LnBwdPlan pl = {};
    pl.vec = vec && ((size_t)C * es) % 16 == 0;
    const int vectors = pl.vec ? C * es / 16 : C;
    if (pl.vec && (vectors + 31) / 32 * (16 / es) <= 32) {
        pl.vpl = (vectors + 31) / 32;
        if (pl.vpl > 4) pl.vpl = (pl.vpl + 1) / 2 * 2;  // float32 alone: 6 or 8, the widths there are
        pl.threads = 32 * kLnBwdWarps;
        const int ctas = es == 4 ? ln_bwd_ctas<float>(pl.vpl) : ln_bwd_ctas<__nv_bfloat16>(pl.vpl);  // resident on an SM
        pl.grid = (int)std::min<long long>((rows + kLnBwdWarps - 1) / kLnBwdWarps, (long long)ctas * sm_count());
        return pl;
    }
    pl.nv = vectors <= 1024 ? 1 : vectors <= 2048 ? 2 : 8;
    const int per = (vectors + pl.nv - 1) / pl.nv;
    pl.threads = std::min(1024, (per + 31) / 32 * 32);
    // as many CTAs as stay resident with 64 registers a thread
    pl.grid = (int)std::min<long long>(rows, (long long)sm_count() * std::max(1, 1024 / pl.threads));
    return pl;
}

// Partial rows are sized for the most CTAs any alignment of the tensors uses.
size_t ln_bwd_ws_bytes(long long rows, int C, int es) {
    const int g = std::max(ln_bwd_plan(rows, C, es, true).grid, ln_bwd_plan(rows, C, es, false).grid);
    return ((size_t)g * 2 * C * 4 + 255) / 256 * 256;
}

template <typename IO, int VPL>
void launch_ln_bwd_warp(const LayerNormBwdParams& p, const LnBwdPlan& pl, cudaStream_t s) {
    layer_norm_bwd_warp_kernel<IO, VPL><<<pl.grid, pl.threads, 2 * p.C * 4, s>>>(p);  // at most 8 KB
}

template <typename IO>
void launch_ln_bwd(const LayerNormBwdParams& p, const LnBwdPlan& pl, cudaStream_t s) {
    switch (pl.vpl) {
    case 1: return launch_ln_bwd_warp<IO, 1>(p, pl, s);
    case 2: return launch_ln_bwd_warp<IO, 2>(p, pl, s);
    case 3: return launch_ln_bwd_warp<IO, 3>(p, pl, s);
    case 4: return launch_ln_bwd_warp<IO, 4>(p, pl, s);
    default: break;
    }
    if constexpr (sizeof(IO) == 4) {  // vectors of 4 channels: up to 8 a lane
        if (pl.vpl == 6) return launch_ln_bwd_warp<IO, 6>(p, pl, s);
        if (pl.vpl == 8) return launch_ln_bwd_warp<IO, 8>(p, pl, s);
    }
    if (pl.vec) {
        if (pl.nv == 1) layer_norm_bwd_kernel<IO, true, 1><<<pl.grid, pl.threads, 0, s>>>(p);
        else if constexpr (sizeof(IO) == 4)  // bfloat16 rows of kLnBwdMaxC channels are 1024 vectors
            layer_norm_bwd_kernel<IO, true, 2><<<pl.grid, pl.threads, 0, s>>>(p);
    } else {
        if (pl.nv == 1) layer_norm_bwd_kernel<IO, false, 1><<<pl.grid, pl.threads, 0, s>>>(p);
        else if (pl.nv == 2) layer_norm_bwd_kernel<IO, false, 2><<<pl.grid, pl.threads, 0, s>>>(p);
        else layer_norm_bwd_kernel<IO, false, 8><<<pl.grid, pl.threads, 0, s>>>(p);
    }
}

vrwkv_status check_ln(long long rows, int C, vrwkv_dtype dtype) {
    if (dtype != VRWKV_F32 && dtype != VRWKV_BF16)
        return fail(VRWKV_ERR_INVALID_ARG, "unknown dtype %d", (int)dtype);
    if (rows <= 0 || C <= 0)
        return fail(VRWKV_ERR_INVALID_ARG, "rows and C must be positive (got %lld, %d)", rows, C);
    if (C > kLnMaxC) return fail(VRWKV_ERR_UNSUPPORTED, "C = %d exceeds 2^30", C);
    if (rows > 0x7fffffffLL) return fail(VRWKV_ERR_UNSUPPORTED, "rows must be below 2^31");
    return ok();
}

}  // namespace

extern "C" {

vrwkv_status vrwkv_layer_norm_fwd(const void* x, const float* gamma, const float* beta, float eps, void* y,
                                  float* mean, float* rstd, long long rows, int C, vrwkv_dtype dtype,
                                  void* stream) {
    vrwkv_status st = check_ln(rows, C, dtype);
    if (st != VRWKV_OK) return st;
    if (!x || !gamma || !beta || !y) return fail(VRWKV_ERR_INVALID_ARG, "required pointer is NULL");
    if (!mean != !rstd) return fail(VRWKV_ERR_INVALID_ARG, "mean and rstd come together or not at all");
    if (!(eps >= 0.0f)) return fail(VRWKV_ERR_INVALID_ARG, "eps must be >= 0");
    const int es = elem_bytes(dtype);
    if (!aligned(x, es) || !aligned(y, es)) return fail(VRWKV_ERR_INVALID_ARG, "token tensor misaligned");
    const float* vecs[4] = {gamma, beta, mean, rstd};
    for (const float* f : vecs)
        if (f && !aligned(f, 4)) return fail(VRWKV_ERR_INVALID_ARG, "float32 vector misaligned");
    const size_t nb = (size_t)rows * C * es, nr = (size_t)rows * 4, nc = (size_t)C * 4;
    struct Span { const void* p; size_t n; };
    const Span ins[3] = {{x, nb}, {gamma, nc}, {beta, nc}};
    const Span outs[3] = {{y, nb}, {mean, nr}, {rstd, nr}};
    for (int i = 0; i < 3; ++i) {
        for (const Span& in : ins)
            if (overlaps(outs[i].p, outs[i].n, in.p, in.n))
                return fail(VRWKV_ERR_INVALID_ARG, "an output overlaps an input");
        for (int j = i + 1; j < 3; ++j)
            if (overlaps(outs[i].p, outs[i].n, outs[j].p, outs[j].n))
                return fail(VRWKV_ERR_INVALID_ARG, "outputs overlap");
    }
    LayerNormParams p;
    p.x = static_cast<const char*>(x);
    p.y = static_cast<char*>(y);
    p.g = gamma;
    p.b = beta;
    p.rows = rows;
    p.C = C;
    p.eps = eps;
    p.mean = mean;
    p.rstd = rstd;
    st = launch_layer_norm(p, dtype, static_cast<cudaStream_t>(stream));
    if (st == VRWKV_OK) set_last_kernel("layer_norm_kernel");
    return st;
}

size_t vrwkv_layer_norm_bwd_workspace_bytes(long long rows, int C, vrwkv_dtype dtype) {
    if (rows <= 0 || rows > 0x7fffffffLL || C <= 0 || C > kLnBwdMaxC || (dtype != VRWKV_F32 && dtype != VRWKV_BF16))
        return 0;
    return ln_bwd_ws_bytes(rows, C, elem_bytes(dtype));
}

vrwkv_status vrwkv_layer_norm_bwd(const void* x, const float* gamma, const float* mean, const float* rstd,
                                  const void* gy, void* gx, float* ggamma, float* gbeta, long long rows, int C,
                                  vrwkv_dtype dtype, void* workspace, size_t workspace_bytes, void* stream) {
    vrwkv_status st = check_ln(rows, C, dtype);
    if (st != VRWKV_OK) return st;
    if (C > kLnBwdMaxC) return fail(VRWKV_ERR_UNSUPPORTED, "C = %d exceeds %d", C, kLnBwdMaxC);
    if (!x || !gamma || !mean || !rstd || !gy || !gx) return fail(VRWKV_ERR_INVALID_ARG, "required pointer is NULL");
    if (!ggamma != !gbeta) return fail(VRWKV_ERR_INVALID_ARG, "ggamma and gbeta come together or not at all");
    const int es = elem_bytes(dtype);
    const void* toks[3] = {x, gy, gx};
    for (const void* t : toks)
        if (!aligned(t, es)) return fail(VRWKV_ERR_INVALID_ARG, "token tensor misaligned");
    const float* vecs[5] = {gamma, mean, rstd, ggamma, gbeta};
    for (const float* f : vecs)
        if (f && !aligned(f, 4)) return fail(VRWKV_ERR_INVALID_ARG, "float32 vector misaligned");
    const size_t need = ggamma ? ln_bwd_ws_bytes(rows, C, es) : 0;
    if (need && !workspace) return fail(VRWKV_ERR_INVALID_ARG, "required pointer is NULL (workspace)");
    if (need && !aligned(workspace, 256)) return fail(VRWKV_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
    if (workspace_bytes < need)
        return fail(VRWKV_ERR_INVALID_ARG, "workspace of %zu bytes is smaller than the %zu needed", workspace_bytes,
                    need);
    const size_t nb = (size_t)rows * C * es, nr = (size_t)rows * 4, nc = (size_t)C * 4;
    struct Span { const void* p; size_t n; };
    const Span ins[5] = {{x, nb}, {gy, nb}, {gamma, nc}, {mean, nr}, {rstd, nr}};
    const Span outs[4] = {{gx, nb}, {ggamma, nc}, {gbeta, nc}, {workspace, need}};
    for (int i = 0; i < 4; ++i) {
        for (const Span& in : ins)
            if (overlaps(outs[i].p, outs[i].n, in.p, in.n))
                return fail(VRWKV_ERR_INVALID_ARG, "an output or the workspace overlaps an input");
        for (int j = i + 1; j < 4; ++j)
            if (overlaps(outs[i].p, outs[i].n, outs[j].p, outs[j].n))
                return fail(VRWKV_ERR_INVALID_ARG, "outputs or the workspace overlap");
    }
    LayerNormBwdParams p;
    p.x = static_cast<const char*>(x);
    p.gy = static_cast<const char*>(gy);
    p.gx = static_cast<char*>(gx);
    p.g = gamma;
    p.mean = mean;
    p.rstd = rstd;
    p.part = ggamma ? static_cast<float*>(workspace) : nullptr;
    p.rows = rows;
    p.C = C;
    const bool vec = aligned(x, 16) && aligned(gy, 16) && aligned(gx, 16);
    const LnBwdPlan pl = ln_bwd_plan(rows, C, es, vec);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (dtype == VRWKV_F32) launch_ln_bwd<float>(p, pl, s);
    else launch_ln_bwd<__nv_bfloat16>(p, pl, s);
    st = cuda_status(cudaGetLastError(), "layer_norm_bwd_kernel launch");
    if (st != VRWKV_OK) return st;
    if (ggamma) {
        st = launch(layer_norm_wgrad_kernel, "layer_norm_wgrad_kernel launch",
                    dim3((unsigned)((2 * C + kLnWgradCols - 1) / kLnWgradCols)), 1024, 0, true, s, (const float*)p.part, pl.grid, C,
                    ggamma, gbeta);
        if (st != VRWKV_OK) return st;
    }
    set_last_kernel("layer_norm_bwd_kernel");
    return ok();
}

}  // extern "C"
