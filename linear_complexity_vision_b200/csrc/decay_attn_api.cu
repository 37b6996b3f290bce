// C ABI of the multi-head decay attention (declared in include/vrwkv.h):
// host-side argument validation, the cut into segments and kernel launches.
// Validation happens before any CUDA call.
#include <algorithm>
#include <climits>
#include <cstdint>
#include <cstdlib>

#include "api_internal.h"
#include "decay_attn.cuh"
#include "decay_attn_tc.cuh"
#include "decay_attn_tc64.cuh"
#include "decay_attn_tcf.cuh"
#include "decay_pack.cuh"

namespace {

using namespace vrwkv;
using namespace vrwkv::api;

constexpr int kMaxD = 128;
constexpr int kMaxT = 1 << 30;  // a segment's end stays an int
constexpr int kSegUnit = 128;  // segments are multiples of this many tokens

struct Span {
    const void* p;
    size_t n;
};

// Bytes a (B, T, C) tensor spans whose rows lie ld elements apart.
size_t span_bytes(int B, int T, int C, long long ld, int es) {
    return (((size_t)B * T - 1) * (size_t)ld + C) * es;
}

vrwkv_status check_sizes(int B, int T, int H, int D, vrwkv_dtype dtype) {
    if (dtype != VRWKV_F32 && dtype != VRWKV_BF16)
        return fail(VRWKV_ERR_INVALID_ARG, "unknown dtype %d", (int)dtype);
    if (B <= 0 || T <= 0 || H <= 0 || D <= 0)
        return fail(VRWKV_ERR_INVALID_ARG, "B, T, H and D must be positive (got %d, %d, %d, %d)", B, T, H, D);
    if (D > kMaxD) return fail(VRWKV_ERR_UNSUPPORTED, "head size D = %d exceeds %d", D, kMaxD);
    if (T > kMaxT) return fail(VRWKV_ERR_UNSUPPORTED, "T = %d exceeds 2^30", T);
    if ((long long)B * T > INT_MAX || (long long)H * D > INT_MAX)
        return fail(VRWKV_ERR_UNSUPPORTED, "B*T and H*D must be below 2^31");
    return ok();
}

// Every output against every input and every other output.
vrwkv_status check_overlaps(const Span* outs, int no, const Span* ins, int ni) {
    for (int i = 0; i < no; ++i) {
        for (int j = 0; j < ni; ++j)
            if (overlaps(outs[i].p, outs[i].n, ins[j].p, ins[j].n))
                return fail(VRWKV_ERR_INVALID_ARG, "an output or the workspace overlaps an input");
        for (int j = i + 1; j < no; ++j)
            if (overlaps(outs[i].p, outs[i].n, outs[j].p, outs[j].n))
                return fail(VRWKV_ERR_INVALID_ARG, "outputs or the workspace overlap");
    }
    return ok();
}

vrwkv_status check_workspace(const void* ws, size_t have, size_t need) {
    if (!need) return ok();
    if (!ws) return fail(VRWKV_ERR_INVALID_ARG, "required pointer is NULL (workspace)");
    if (!aligned(ws, 256)) return fail(VRWKV_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
    if (have < need)
        return fail(VRWKV_ERR_INVALID_ARG, "workspace of %zu bytes is smaller than the %zu needed", have, need);
    return ok();
}

// ---- the cut into segments ----
int padded_d(int D) { return D <= 32 ? 32 : D <= 64 ? 64 : 128; }

// One head's chunks run one after the other; segments let more CTAs than heads
// work, for a pass over k and v that forms the states at the cuts and two more
// launches.  The cut is the one of least estimated time, from what the kernels
// measured alone on an SM, in us for a unit of 128 tokens (and how much of
// that each further CTA on the same SM adds):
//                         outputs          states only      CTAs of an SM
//   tcgen05, D <= 64      2.15             2.0 (+ 0.5)      1 (persistent), 2
//            D <= 128     4.2              3.0              1
//            float32      6.5              4.5              1
//   any size, DP = 32     9 (+ 0.6)        4 (+ 0.6)        3
//             DP = 64     23 (+ 0.6)       9 (+ 0.6)        3
//             DP = 128    45               18               1
// Both sides measured: B = 1, T = 4096, 16 heads of 64, bfloat16: one segment
// 69 us, eight 24 us; B = 3: one 70, three 54; B = 8: one 73 us, two 120 us.
struct Cut {
    int seg_tokens, nseg;
};
Cut cut_into(int T, int want) {
    const int units = (T + kSegUnit - 1) / kSegUnit;
    const int per = (units + std::max(1, std::min(want, units)) - 1) / std::max(1, std::min(want, units));
    return Cut{per * kSegUnit, (units + per - 1) / per};
}

struct PassCost {
    double unit, share;
    int resident;
};
double pass_us(long long ctas, int units, const PassCost& c) {
    const long long per_sm = (ctas + sm_count() - 1) / sm_count(), rounds = per_sm / c.resident;
    const int rest = (int)(per_sm % c.resident);
    const double round = 1.0 + c.share * (c.resident - 1), last = rest ? 1.0 + c.share * (rest - 1) : 0.0;
    return units * c.unit * (rounds * round + last) + 4.5;
}

Cut plan(int B, int T, int H, int D, vrwkv_dtype dtype, int nprob, bool tc) {
    static const PassCost kOut[6] = {{2.15, 0, 1}, {4.2, 0, 1}, {9, 0.6, 3}, {23, 0.6, 3}, {45, 0, 1}, {6.5, 0, 1}};
    static const PassCost kState[6] = {{2.0, 0.5, 2}, {3.0, 0, 1}, {4, 0.6, 3}, {9, 0.6, 3}, {18, 0, 1}, {4.5, 0, 1}};
    const int kind = tc ? (dtype == VRWKV_F32 ? 5 : D <= 64 ? 0 : 1) : (D <= 32 ? 2 : D <= 64 ? 3 : 4);
    const int units = (T + kSegUnit - 1) / kSegUnit;
    const long long heads = (long long)B * H;
    Cut best = cut_into(T, 1);
    double least = pass_us(heads * nprob, units, kOut[kind]);
    static const int kWays[] = {2, 3, 4, 6, 8, 12, 16, 24, 32, 48, 64, 96, 128};
    for (int want : kWays) {
        if (want > units) break;
        const Cut c = cut_into(T, want);
        const int per = c.seg_tokens / kSegUnit, states = nprob == 1 ? 1 : 2;
        const double us = pass_us(heads * nprob * c.nseg, per, kOut[kind]) +
                          pass_us(heads * states * c.nseg, per, kState[kind]) + 5.0 +
                          1e-6 * heads * states * c.nseg * D * D * 4;
        if (us < 0.95 * least) {
            least = us;
            best = c;
        }
    }
    return best;
}

// The tcgen05 kernels take heads of whole 16-byte vectors, bfloat16 ones of up
// to 128 channels, float32 ones of 33 to 64, and work on 128 tokens however few
// there are; the kernel for any size works on 32.  Both measured, us, forward
// (tcgen05 : any size), for 8, 160 and 1024 heads:
//   bfloat16, D = 64   T = 16  5.6 : 5.8    8.3 : 6.2    19.1 : 16.1
//                      T = 32  5.8 : 6.8    8.3 : 7.6    19.2 : 20.8
//                      T = 128 6.0 : 25     8.9 : 28     20.4 : 93
//             D = 32   T = 32  5.9 : 4.4    8.3 : 4.8    19.1 : 12.4
//                      T = 64  5.8 : 7.2    8.4 : 8.1    19.4 : 22.3
//             D = 128  T = 8   5.9 : 6.3    11.0 : 11.1  35.9 : 37.8
//   float32,  D = 64   T = 64  10.2 : 11.5  19.1 : 14.1  67.0 : 43.9
//                      T = 96  11.0 : 17.2  20.5 : 21.0  78.0 : 70.0
//                      T = 128 11.6 : 22.6  21.7 : 28.2  83.4 : 95.4
//             D = 32   T = 128 10.7 : 10.8  20.1 : 13.1  70.9 : 41.2
// VRWKV_DECAY_TC=0 keeps them on the kernel for any size (diagnostics and tests).
bool tc_sizes(int T, int D, vrwkv_dtype dtype) {
    if (dtype == VRWKV_F32) return D % 4 == 0 && D > 32 && D <= 64 && T > 96;
    return D % 8 == 0 && T > (D <= 32 ? 32 : 16);
}
bool tc_disabled() {
    const char* e = getenv("VRWKV_DECAY_TC");
    return e && e[0] == '0' && e[1] == 0;
}

size_t state_floats(int B, int H, int D, int nseg) { return (size_t)B * H * nseg * D * D; }

// bfloat16 heads that are spread to whole 16-byte vectors first (decay_pack.cuh):
// how wide, or 0.  Measured, us, forward (spread : as they are), for 8, 160 and
// 1024 heads:
//   D = 27  T = 200  13.7 : 25.6  35.7 : 27.5  118 : 78
//   D = 45  T = 64   11.1 : 15.7  19.2 : 17.0  53.1 : 49.8
//           T = 96   11.4 : 23.9  22.3 : 26.3  68.4 : 76.4
//   D = 89  T = 32   12.0 : 8.9   20.2 : 16.4  67.6 : 56.0
//           T = 48   12.1 : 18.2  21.4 : 34.4  81.0 : 119
// (float32, D = 45, T = 200: 23.1 : 41.7, 60.8 : 50.7, 240 : 172, as they are.)
int spread_width(int T, int D, vrwkv_dtype dtype) {
    return dtype == VRWKV_BF16 && D > 32 && D % 8 != 0 && T > (D <= 64 ? 64 : 32) ? (D + 7) / 8 * 8 : 0;
}
size_t spread_bytes(int B, int T, int H, int W) {  // of a tensor
    return ((size_t)B * T * H * W * 2 + 255) / 256 * 256;
}

// What the cut needs of the kernel that the sizes go to.
size_t state_bytes(int B, int T, int H, int D, vrwkv_dtype dtype, bool backward) {
    const int W = spread_width(T, D, dtype);
    const Cut c = plan(B, T, H, D, dtype, backward ? 3 : 1, W || tc_sizes(T, D, dtype));
    return c.nseg > 1 ? ((backward ? 2 : 1) * state_floats(B, H, D, c.nseg) * 4 + 255) / 256 * 256 : 0;
}
// The states, then the spread inputs and outputs.
size_t ws_bytes(int B, int T, int H, int D, vrwkv_dtype dtype, bool backward) {
    const int W = spread_width(T, D, dtype);
    return state_bytes(B, T, H, D, dtype, backward) + (W ? (backward ? 7 : 4) * spread_bytes(B, T, H, W) : 0);
}
// The cut of the kernel that runs: where alignment keeps it from the one of the
// sizes, in as many segments as the workspace has room for.
Cut cut_for(int B, int T, int H, int D, vrwkv_dtype dtype, bool backward, bool tc, size_t workspace) {
    const Cut c = plan(B, T, H, D, dtype, backward ? 3 : 1, tc);
    const size_t most = workspace / ((backward ? 2 : 1) * state_floats(B, H, D, 1) * 4);
    return (size_t)c.nseg <= most ? c : cut_into(T, (int)std::max<size_t>(most, 1));
}

// ---- launches ----
template <typename IO, int DP>
vrwkv_status launch_dp(const decay::Params& p, long long ctas, bool follows, cudaStream_t s) {
    static SmemGrants granted;
    constexpr int smem = decay::Cfg<DP>::kSmemFloats * 4;
    const cudaError_t e = ensure_smem(decay::decay_attn_kernel<IO, DP>, granted, smem);
    if (e != cudaSuccess) return cuda_status(e, "cudaFuncSetAttribute");
    return launch(decay::decay_attn_kernel<IO, DP>, "decay_attn_kernel launch", dim3((unsigned)ctas),
                  decay::Cfg<DP>::kThreads, smem, follows, s, p);
}

template <typename IO>
vrwkv_status launch_io(const decay::Params& p, bool follows, cudaStream_t s) {
    const long long ctas = (long long)p.B * p.H * p.nseg * p.nprob;
    if (ctas > INT_MAX / 4) return fail(VRWKV_ERR_UNSUPPORTED, "too many heads (B*H = %lld)", (long long)p.B * p.H);
    switch (padded_d(p.D)) {
    case 32: return launch_dp<IO, 32>(p, ctas, follows, s);
    case 64: return launch_dp<IO, 64>(p, ctas, follows, s);
    default: return launch_dp<IO, 128>(p, ctas, follows, s);
    }
}

// ---- tensor cores ----
// A token tensor as TMA reads it: (D, H, T, B) with rows ld elements apart, in
// boxes of 64 channels of a head x 128 tokens (channels past D and rows past T
// arrive as zeros and are not stored).
bool encode_tokens(CUtensorMap* m, const void* x, long long ld, int B, int T, int H, int D) {
    const EncodeTiledFn enc = encode_fn();
    const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)H, (cuuint64_t)T, (cuuint64_t)B};
    const cuuint64_t strides[3] = {(cuuint64_t)D * 2, (cuuint64_t)ld * 2, (cuuint64_t)T * ld * 2};
    const cuuint32_t box[4] = {64, 1, decay::kTcChunk, 1}, estr[4] = {1, 1, 1, 1};
    return enc && enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(x), dims, strides, box, estr,
                      CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// Rows that start on 16-byte boundaries (and a stride that TMA can hold).
bool rows16(const void* x, long long ld, int es) { return aligned(x, 16) && ld * es % 16 == 0 && ld < (1LL << 36); }

template <int D, bool OUT, int PIECES, bool PAD>
vrwkv_status launch_tc_pad(const decay::TcParams& p, unsigned ctas, bool follows, cudaStream_t s) {
    static SmemGrants granted;
    constexpr int smem = decay::tc_smem_bytes<D, OUT>();
    const cudaError_t e = ensure_smem(decay::decay_attn_tc_kernel<D, OUT, PIECES, PAD>, granted, smem);
    if (e != cudaSuccess) return cuda_status(e, "cudaFuncSetAttribute");
    return launch(decay::decay_attn_tc_kernel<D, OUT, PIECES, PAD>, "decay_attn_tc_kernel launch", dim3(ctas),
                  decay::tc_threads<D>(), smem, follows, s, p);
}
template <int D, bool OUT, int PIECES>
vrwkv_status launch_tc(const decay::TcParams& p, unsigned ctas, bool follows, cudaStream_t s) {
    return OUT && p.p.D == D && p.p.S == D ? launch_tc_pad<D, OUT, PIECES, !OUT>(p, ctas, follows, s)
                             : launch_tc_pad<D, OUT, PIECES, true>(p, ctas, follows, s);
}
template <int PIECES>
vrwkv_status launch_tc64(decay::TcParams& p, bool follows, cudaStream_t s) {
    static SmemGrants granted;
    constexpr int smem = decay::t64_smem_bytes();
    const cudaError_t e = ensure_smem(decay::decay_attn_tc64_kernel<PIECES>, granted, smem);
    if (e != cudaSuccess) return cuda_status(e, "cudaFuncSetAttribute");
    const unsigned ctas = (unsigned)std::min(p.nitems, sm_count());
    int left = (int)ctas;
    const int radix[3] = {p.p.nprob, p.p.nseg, p.p.H};
    for (int i = 0; i < 3; ++i) {
        p.step[i] = left % radix[i];
        left /= radix[i];
    }
    p.step[3] = left;
    return launch(decay::decay_attn_tc64_kernel<PIECES>, "decay_attn_tc64_kernel launch", dim3(ctas),
                  decay::kT64Threads, smem, follows, s, p);
}
template <bool OUT>
vrwkv_status launch_tcf(const decay::TcParams& p, bool follows, cudaStream_t s) {
    static SmemGrants granted;
    constexpr int smem = decay::tf_smem_bytes<OUT>();
    const cudaError_t e = ensure_smem(decay::decay_attn_tcf_kernel<OUT>, granted, smem);
    if (e != cudaSuccess) return cuda_status(e, "cudaFuncSetAttribute");
    return launch(decay::decay_attn_tcf_kernel<OUT>, "decay_attn_tcf_kernel launch", dim3((unsigned)p.nitems),
                  decay::kTfThreads, smem, follows, s, p);
}

vrwkv_status launch_tc_any(decay::TcParams& p, bool exact, bool follows, cudaStream_t s) {
    const unsigned n = (unsigned)p.nitems;
    if (p.p.pr[0].out && p.p.D <= 64) return exact ? launch_tc64<3>(p, follows, s) : launch_tc64<2>(p, follows, s);
    if (p.p.pr[0].out) return exact ? launch_tc<128, true, 3>(p, n, follows, s) : launch_tc<128, true, 2>(p, n, follows, s);
    if (p.p.D <= 64) return exact ? launch_tc<64, false, 3>(p, n, follows, s) : launch_tc<64, false, 2>(p, n, follows, s);
    return exact ? launch_tc<128, false, 3>(p, n, follows, s) : launch_tc<128, false, 2>(p, n, follows, s);
}

// Launch p's problems; with `tc`, on the tensor cores with its maps.
struct Launcher {
    vrwkv_dtype dtype;
    bool tc;
    bool exact;         // a state leaves the call: three pieces (decay_attn_tc.cuh)
    decay::TcParams t;  // maps, error word, wait limit
    const void* src[4]; // the tensors behind the maps, and their row strides
    long long ld[4];

    const char* kernel(int D) const {
        return !tc ? "decay_attn_kernel" : dtype == VRWKV_F32 ? "decay_attn_tcf_kernel"
                   : D <= 64 ? "decay_attn_tc64_kernel" : "decay_attn_tc_kernel";
    }
    int map_of(const char* x, long long row) const {
        for (int i = 0; i < 4; ++i)
            if (src[i] == x && ld[i] == row) return i;
        return 0;  // no q: the state alone
    }
    // follows: behind the call's chain kernel
    vrwkv_status run(const decay::Params& p, bool follows, cudaStream_t s) {
        if (!tc) return dtype == VRWKV_F32 ? launch_io<float>(p, follows, s) : launch_io<__nv_bfloat16>(p, follows, s);
        const long long ctas = (long long)p.B * p.H * p.nseg * p.nprob;
        if (ctas > INT_MAX) return fail(VRWKV_ERR_UNSUPPORTED, "too many heads (B*H = %lld)", (long long)p.B * p.H);
        t.p = p;
        for (int i = 0; i < p.nprob; ++i) {
            t.mq[i] = map_of(p.pr[i].q, p.pr[i].ldq);
            t.mk[i] = map_of(p.pr[i].k, p.pr[i].ldk);
            t.mv[i] = map_of(p.pr[i].v, p.pr[i].ldv);
        }
        t.nitems = (int)ctas;
        if (dtype == VRWKV_F32) return p.pr[0].out ? launch_tcf<true>(t, follows, s) : launch_tcf<false>(t, follows, s);
        return launch_tc_any(t, exact, follows, s);
    }
};

// The tcgen05 kernel where the sizes, alignments and row strides of all
// n <= 4 tensors and of the states read allow, else the kernel for any size.
Launcher make_launcher(vrwkv_dtype dtype, const void* const* x, const long long* ld, int n, const void* const* outs,
                       int no, const float* state, const float* gstate, bool state_leaves, int B, int T, int H, int D) {
    Launcher l = {};
    l.dtype = dtype;
    l.exact = state_leaves;
    l.tc = tc_sizes(T, D, dtype) && !tc_disabled() && aligned(state, 16) && aligned(gstate, 16);
    const int es = elem_bytes(dtype);
    l.t.wide_out = D * es % 32 == 0;
    for (int i = 0; i < no; ++i) {
        l.tc = l.tc && aligned(outs[i], 16);
        if (!aligned(outs[i], 32)) l.t.wide_out = 0;
    }
    for (int i = 0; i < n && l.tc; ++i) l.tc = rows16(x[i], ld[i], es);
    if (!l.tc) return l;
    l.t.err = device_error_word();
    l.t.wait_ns = wait_limit_ns();
    l.tc = l.t.err != nullptr;
    if (dtype == VRWKV_F32) return l;  // reads and writes without TMA
    for (int i = 0; i < n && l.tc; ++i) {
        l.src[i] = x[i];
        l.ld[i] = ld[i];
        l.tc = encode_tokens(&l.t.map[i], x[i], ld[i], B, T, H, D);
    }
    for (int i = 0; i < no && l.tc && D <= 64; ++i)
        l.tc = encode_tokens(&l.t.omap[i], outs[i], (long long)H * D, B, T, H, D);
    return l;
}

// A call's tensors spread to heads of W channels in the workspace.
struct Spread {
    int W, ni, no;
    decay::PackParams in, out;
    long long ld;  // of the spread rows

    void init(int W_, char* ws, const void* const* x, const long long* lds, int n, void* const* y, int m, int B,
              int T, int H, int D) {
        W = W_;
        ni = n;
        no = m;
        ld = (long long)H * W;
        const size_t each = spread_bytes(B, T, H, W);
        in = {};
        in.heads = (long long)B * T * H;
        in.H = H;
        in.D = D;
        in.W = W;
        out = in;
        for (int i = 0; i < n; ++i, ws += each) {
            in.src[i] = static_cast<const char*>(x[i]);
            in.dst[i] = ws;
            in.ld[i] = lds[i];
        }
        for (int i = 0; i < m; ++i, ws += each) {
            out.src[i] = ws;
            out.dst[i] = static_cast<char*>(y[i]);
            out.ld[i] = (long long)H * D;
        }
    }
    vrwkv_status run(bool to_wide, cudaStream_t s) const {
        const unsigned x = (unsigned)std::min<long long>((in.heads + 31) / 32, 8LL * sm_count());
        return to_wide ? launch(decay::decay_pack_kernel<true>, "decay_pack_kernel launch", dim3(x, (unsigned)ni), 256, 0, false, s, in)
                       : launch(decay::decay_pack_kernel<false>, "decay_pack_kernel launch", dim3(x, (unsigned)no), 256, 0, false, s, out);
    }
};

vrwkv_status launch_chain(const decay::ChainParams& p, int bh, int nprob, cudaStream_t s) {
    const int per = p.dd % 4 == 0 ? 1024 : 256;  // elements of a CTA
    return launch(decay::decay_chain_kernel, "decay_chain_kernel launch",
                  dim3((unsigned)bh, (unsigned)((p.dd + per - 1) / per), (unsigned)nprob), 256, 0, true, s, p);
}

bool vec_ok(const void* p, long long ld, int es) { return aligned(p, 4 * es) && ld % 4 == 0; }

}  // namespace

extern "C" {

size_t vrwkv_decay_attn_workspace_bytes(int B, int T, int H, int D, vrwkv_dtype dtype, int backward) {
    if (B <= 0 || T <= 0 || T > kMaxT || H <= 0 || D <= 0 || D > kMaxD || (dtype != VRWKV_F32 && dtype != VRWKV_BF16)) return 0;
    return ws_bytes(B, T, H, D, dtype, backward != 0);
}

vrwkv_status vrwkv_decay_attn_fwd(const void* q, const void* k, const void* v, long long ldq, long long ldk,
                                  long long ldv, const float* w, const float* state, const int* lengths, float scale,
                                  void* out, float* state_out, int B, int T, int H, int D, vrwkv_dtype dtype,
                                  void* workspace, size_t workspace_bytes, void* stream) {
    vrwkv_status st = check_sizes(B, T, H, D, dtype);
    if (st != VRWKV_OK) return st;
    if (!q || !k || !v || !w || !out) return fail(VRWKV_ERR_INVALID_ARG, "required pointer is NULL");
    const int es = elem_bytes(dtype), C = H * D;
    if (ldq < C || ldk < C || ldv < C) return fail(VRWKV_ERR_INVALID_ARG, "a row stride is below H*D = %d", C);
    const void* toks[4] = {q, k, v, out};
    for (const void* t : toks)
        if (!aligned(t, es)) return fail(VRWKV_ERR_INVALID_ARG, "token tensor misaligned");
    const void* words[4] = {w, state, lengths, state_out};
    for (const void* f : words)
        if (f && !aligned(f, 4)) return fail(VRWKV_ERR_INVALID_ARG, "float32 or int32 array misaligned");
    const size_t need = ws_bytes(B, T, H, D, dtype, false);
    st = check_workspace(workspace, workspace_bytes, need);
    if (st != VRWKV_OK) return st;
    const size_t nb = span_bytes(B, T, C, C, es), ns = state_floats(B, H, D, 1) * 4;
    const bool in_place = state_out && state_out == state;
    const Span ins[6] = {{q, span_bytes(B, T, C, ldq, es)}, {k, span_bytes(B, T, C, ldk, es)},
                         {v, span_bytes(B, T, C, ldv, es)}, {w, (size_t)H * 4},
                         {lengths, (size_t)B * 4},          {in_place ? nullptr : state, ns}};
    const Span outs[3] = {{out, nb}, {state_out, ns}, {workspace, need}};
    st = check_overlaps(outs, 3, ins, 6);
    if (st != VRWKV_OK) return st;

    const void* srcs[3] = {q, k, v};
    const void* dsts[1] = {out};
    const long long lds[3] = {ldq, ldk, ldv};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const size_t for_states = state_bytes(B, T, H, D, dtype, false);
    Spread wide = {};
    Launcher attn;
    if (const int W = spread_width(T, D, dtype)) {
        void* const outs_[1] = {out};
        wide.init(W, static_cast<char*>(workspace) + for_states, srcs, lds, 3, outs_, 1, B, T, H, D);
        const long long wlds[3] = {wide.ld, wide.ld, wide.ld};
        attn = make_launcher(dtype, (const void* const*)wide.in.dst, wlds, 3, (const void* const*)wide.out.src, 1, state, nullptr,
                             state_out != nullptr, B, T, H, W);
        if (!attn.tc) wide.W = 0;
    }
    if (!wide.W) attn = make_launcher(dtype, srcs, lds, 3, dsts, 1, state, nullptr, state_out != nullptr, B, T, H, D);
    const Cut cut = cut_for(B, T, H, D, dtype, false, attn.tc, for_states);
    const char *Q = static_cast<const char*>(q), *K = static_cast<const char*>(k), *V = static_cast<const char*>(v);
    char* O = static_cast<char*>(out);
    if (wide.W) {
        st = wide.run(true, s);
        if (st != VRWKV_OK) return st;
        Q = wide.in.dst[0], K = wide.in.dst[1], V = wide.in.dst[2];
        O = const_cast<char*>(wide.out.src[0]);
        ldq = ldk = ldv = wide.ld;
    }
    decay::Params p = {};
    p.w = w;
    p.lengths = lengths;
    p.B = B;
    p.T = T;
    p.H = H;
    p.D = wide.W ? wide.W : D;
    p.S = D;
    p.seg_tokens = cut.seg_tokens;
    p.nseg = cut.nseg;
    p.nprob = 1;
    p.vec = D % 4 == 0 && vec_ok(q, ldq, es) && vec_ok(k, ldk, es) && vec_ok(v, ldv, es) && vec_ok(out, C, es);
    decay::Problem& pr = p.pr[0];
    pr.q = Q;
    pr.k = K;
    pr.v = V;
    pr.ldq = ldq;
    pr.ldk = ldk;
    pr.ldv = ldv;
    pr.scale_intra = pr.scale_inter = scale;
    pr.scale_upd = 1.0f;
    float* ws = static_cast<float*>(workspace);
    if (cut.nseg > 1) {
        pr.x_out = ws;
        pr.skip = state_out ? -1 : cut.nseg - 1;
        st = attn.run(p, false, s);
        if (st != VRWKV_OK) return st;
        decay::ChainParams c = {};
        c.pr[0] = {ws, state, state_out, 0};
        c.w = w;
        c.lengths = lengths;
        c.T = T;
        c.H = H;
        c.dd = D * D;
        c.seg_tokens = cut.seg_tokens;
        c.nseg = cut.nseg;
        st = launch_chain(c, B * H, 1, s);
        if (st != VRWKV_OK) return st;
        pr.x_in = ws;
        pr.x_out = nullptr;
        attn.exact = false;  // the chain handed the state out
    } else {
        pr.x_in = state;
        pr.x_out = state_out;
    }
    pr.out = O;
    st = attn.run(p, cut.nseg > 1, s);
    if (st == VRWKV_OK && wide.W) st = wide.run(false, s);
    if (st == VRWKV_OK) set_last_kernel(attn.kernel(D));
    return st;
}

vrwkv_status vrwkv_decay_attn_bwd(const void* q, const void* k, const void* v, const void* gy, long long ldq,
                                  long long ldk, long long ldv, long long ldg, const float* w, const float* state,
                                  const float* gstate, const int* lengths, float scale, void* gq, void* gk, void* gv,
                                  float* gstate_in, int B, int T, int H, int D, vrwkv_dtype dtype, void* workspace,
                                  size_t workspace_bytes, void* stream) {
    vrwkv_status st = check_sizes(B, T, H, D, dtype);
    if (st != VRWKV_OK) return st;
    if (!q || !k || !v || !gy || !w || !gq || !gk || !gv)
        return fail(VRWKV_ERR_INVALID_ARG, "required pointer is NULL");
    const int es = elem_bytes(dtype), C = H * D;
    if (ldq < C || ldk < C || ldv < C || ldg < C)
        return fail(VRWKV_ERR_INVALID_ARG, "a row stride is below H*D = %d", C);
    const void* toks[7] = {q, k, v, gy, gq, gk, gv};
    for (const void* t : toks)
        if (!aligned(t, es)) return fail(VRWKV_ERR_INVALID_ARG, "token tensor misaligned");
    const void* words[5] = {w, state, gstate, lengths, gstate_in};
    for (const void* f : words)
        if (f && !aligned(f, 4)) return fail(VRWKV_ERR_INVALID_ARG, "float32 or int32 array misaligned");
    const size_t need = ws_bytes(B, T, H, D, dtype, true);
    st = check_workspace(workspace, workspace_bytes, need);
    if (st != VRWKV_OK) return st;
    const size_t nb = span_bytes(B, T, C, C, es), ns = state_floats(B, H, D, 1) * 4;
    const Span ins[8] = {{q, span_bytes(B, T, C, ldq, es)}, {k, span_bytes(B, T, C, ldk, es)},
                         {v, span_bytes(B, T, C, ldv, es)}, {gy, span_bytes(B, T, C, ldg, es)},
                         {w, (size_t)H * 4},                {lengths, (size_t)B * 4},
                         {state, ns},                       {gstate, ns}};
    const Span outs[5] = {{gq, nb}, {gk, nb}, {gv, nb}, {gstate_in, ns}, {workspace, need}};
    st = check_overlaps(outs, 5, ins, 8);
    if (st != VRWKV_OK) return st;

    const void* srcs[4] = {q, k, v, gy};
    const void* dsts[3] = {gq, gk, gv};
    const long long lds[4] = {ldq, ldk, ldv, ldg};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const size_t for_states = state_bytes(B, T, H, D, dtype, true);
    Spread wide = {};
    Launcher attn;
    if (const int W = spread_width(T, D, dtype)) {
        void* const outs_[3] = {gq, gk, gv};
        wide.init(W, static_cast<char*>(workspace) + for_states, srcs, lds, 4, outs_, 3, B, T, H, D);
        const long long wlds[4] = {wide.ld, wide.ld, wide.ld, wide.ld};
        attn = make_launcher(dtype, (const void* const*)wide.in.dst, wlds, 4, (const void* const*)wide.out.src, 3, state, gstate,
                             gstate_in != nullptr, B, T, H, W);
        if (!attn.tc) wide.W = 0;
    }
    if (!wide.W) attn = make_launcher(dtype, srcs, lds, 4, dsts, 3, state, gstate, gstate_in != nullptr, B, T, H, D);
    const Cut cut = cut_for(B, T, H, D, dtype, true, attn.tc, for_states);
    const char *Q = static_cast<const char*>(q), *K = static_cast<const char*>(k), *V = static_cast<const char*>(v),
               *G = static_cast<const char*>(gy);
    char* grads[3] = {static_cast<char*>(gq), static_cast<char*>(gk), static_cast<char*>(gv)};
    if (wide.W) {
        st = wide.run(true, s);
        if (st != VRWKV_OK) return st;
        Q = wide.in.dst[0], K = wide.in.dst[1], V = wide.in.dst[2], G = wide.in.dst[3];
        for (int i = 0; i < 3; ++i) grads[i] = const_cast<char*>(wide.out.src[i]);
        ldq = ldk = ldv = ldg = wide.ld;
    }
    decay::Params p = {};
    p.w = w;
    p.lengths = lengths;
    p.B = B;
    p.T = T;
    p.H = H;
    p.D = wide.W ? wide.W : D;
    p.S = D;
    p.seg_tokens = cut.seg_tokens;
    p.nseg = cut.nseg;
    p.vec = D % 4 == 0 && vec_ok(q, ldq, es) && vec_ok(k, ldk, es) && vec_ok(v, ldv, es) && vec_ok(gy, ldg, es) &&
            vec_ok(gq, C, es) && vec_ok(gk, C, es) && vec_ok(gv, C, es);
    const float* s_in = state;   // X_in of the segments: S of the forward pass
    const float* g_in = gstate;  // and dL/dS of the reversed one
    float* g_out = gstate_in;
    if (cut.nseg > 1) {
        float* ws = static_cast<float*>(workspace);
        float* wg = ws + state_floats(B, H, D, cut.nseg);
        decay::Problem& a = p.pr[0];
        a.k = K;
        a.ldk = ldk;
        a.v = V;
        a.ldv = ldv;
        a.x_out = ws;
        a.skip = cut.nseg - 1;
        a.scale_upd = 1.0f;
        decay::Problem& c = p.pr[1];
        c.k = Q;
        c.ldk = ldq;
        c.v = G;
        c.ldv = ldg;
        c.x_out = wg;
        c.skip = gstate_in ? -1 : 0;
        c.scale_upd = scale;
        c.reverse = 1;
        p.nprob = 2;
        st = attn.run(p, false, s);
        if (st != VRWKV_OK) return st;
        decay::ChainParams cp = {};
        cp.pr[0] = {ws, state, nullptr, 0};
        cp.pr[1] = {wg, gstate, gstate_in, 1};
        cp.w = w;
        cp.lengths = lengths;
        cp.T = T;
        cp.H = H;
        cp.dd = D * D;
        cp.seg_tokens = cut.seg_tokens;
        cp.nseg = cut.nseg;
        st = launch_chain(cp, B * H, 2, s);
        if (st != VRWKV_OK) return st;
        s_in = ws;
        g_in = wg;
        g_out = nullptr;
        attn.exact = false;  // the chain handed the state's gradient out
    }
    p.nprob = 3;
    // gq: (g, v, k) forward in time on S^T
    p.pr[0] = {G, V, K, grads[0], ldg, ldv, ldk, s_in, nullptr, 1, 1, 0, scale, scale, 1.0f, -1};
    // gk: (v, g, q) in reversed time on (dL/dS)^T; gv: (k, q, g) on dL/dS
    p.pr[1] = {V, G, Q, grads[1], ldv, ldg, ldq, g_in, nullptr, 1, 1, 1, scale, 1.0f, scale, -1};
    p.pr[2] = {K, Q, G, grads[2], ldk, ldq, ldg, g_in, g_out, 0, 0, 1, scale, 1.0f, scale, -1};
    st = attn.run(p, cut.nseg > 1, s);
    if (st == VRWKV_OK && wide.W) st = wide.run(false, s);
    if (st == VRWKV_OK) set_last_kernel(attn.kernel(D));
    return st;
}

vrwkv_status vrwkv_decay_attn_step(const void* q, const void* k, const void* v, long long ldq, long long ldk,
                                   long long ldv, const float* w, float* state, const int* slots, float scale,
                                   void* out, int B, int N, int H, int D, vrwkv_dtype dtype, void* stream) {
    vrwkv_status st = check_sizes(B, 1, H, D, dtype);
    if (st != VRWKV_OK) return st;
    if (N <= 0) return fail(VRWKV_ERR_INVALID_ARG, "the pool must hold at least one state (got %d)", N);
    if (!slots && N < B)
        return fail(VRWKV_ERR_INVALID_ARG, "without slots the pool must hold B = %d states (got %d)", B, N);
    if (!q || !k || !v || !w || !state || !out) return fail(VRWKV_ERR_INVALID_ARG, "required pointer is NULL");
    if (H > 65535) return fail(VRWKV_ERR_UNSUPPORTED, "H = %d exceeds 65535", H);
    const int es = elem_bytes(dtype), C = H * D;
    if (ldq < C || ldk < C || ldv < C) return fail(VRWKV_ERR_INVALID_ARG, "a row stride is below H*D = %d", C);
    const void* toks[4] = {q, k, v, out};
    for (const void* t : toks)
        if (!aligned(t, es)) return fail(VRWKV_ERR_INVALID_ARG, "token tensor misaligned");
    const void* words[3] = {w, state, slots};
    for (const void* f : words)
        if (f && !aligned(f, 4)) return fail(VRWKV_ERR_INVALID_ARG, "float32 or int32 array misaligned");
    const Span ins[5] = {{q, span_bytes(B, 1, C, ldq, es)}, {k, span_bytes(B, 1, C, ldk, es)},
                         {v, span_bytes(B, 1, C, ldv, es)}, {w, (size_t)H * 4}, {slots, (size_t)B * 4}};
    const Span outs[2] = {{out, (size_t)B * C * es}, {state, state_floats(N, H, D, 1) * 4}};
    st = check_overlaps(outs, 2, ins, 5);
    if (st != VRWKV_OK) return st;
    decay::StepParams p;
    p.q = static_cast<const char*>(q);
    p.k = static_cast<const char*>(k);
    p.v = static_cast<const char*>(v);
    p.out = static_cast<char*>(out);
    p.ldq = ldq;
    p.ldk = ldk;
    p.ldv = ldv;
    p.w = w;
    p.state = state;
    p.slots = slots;
    p.B = B;
    p.N = N;
    p.H = H;
    p.D = D;
    p.scale = scale;
    p.vec = D % 4 == 0 && aligned(state, 16);
    p.err = device_error_word();
    if (!p.err) return fail(VRWKV_ERR_CUDA, "cannot locate the device error word");
    const dim3 grid((unsigned)B, (unsigned)H, (unsigned)((D + decay::kStepCols - 1) / decay::kStepCols));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    auto step = [&](auto io) {
        using IO = decltype(io);
        if (D <= 32) decay::decay_step_kernel<IO, 2><<<grid, decay::kStepThreads, 0, s>>>(p);
        else if (D <= 64) decay::decay_step_kernel<IO, 4><<<grid, decay::kStepThreads, 0, s>>>(p);
        else decay::decay_step_kernel<IO, 8><<<grid, decay::kStepThreads, 0, s>>>(p);
    };
    if (dtype == VRWKV_F32) step(float{});
    else step(__nv_bfloat16{});
    st = cuda_status(cudaGetLastError(), "decay_step_kernel launch");
    if (st == VRWKV_OK) set_last_kernel("decay_step_kernel");
    return st;
}

}  // extern "C"
