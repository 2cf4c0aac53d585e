// C ABI of a speculative step over a tree of drafted tokens (declared in
// include/kda.h): the recurrence, its short convolution, and the verification
// of the drafts.  Attention over the tree is with the cache's other calls.
//
// Host side: validate every argument synchronously and enqueue exactly one
// kernel on the caller's stream.
#include <cuda_runtime.h>

#include <algorithm>
#include <cfloat>
#include <cstddef>
#include <cstdint>

#include "kda.h"
#include "kda_host.cuh"
#include "kda_accept.cuh"
#include "kda_tree.cuh"

namespace {

#if KDA_STATE16
using state_t = __half;
#else
using state_t = float;
#endif

constexpr int kSms = 152;

template <typename QT, int W>
int launch_tree_warps(const kda::StepParams& prm, const uint64_t* tree, int groups, uint32_t flags, cudaStream_t stream) {
    using SM = kda::TreeSmem<state_t>;
    auto kernel = prm.k == kda::KMAX && prm.v == kda::KMAX ? kda::kda_tree_kernel<state_t, QT, W, true>
                                                           : kda::kda_tree_kernel<state_t, QT, W, false>;
    const int64_t grid = (int64_t)prm.n * prm.hv * ((prm.v + groups * kda::TREE_CW - 1) / (groups * kda::TREE_CW));
    if (grid > 0x7fffffffLL) return KDA_ERR_SHAPE;
    int occ = 0, sms = 0;   // raises the kernel's limit to the most that any call takes
    const int rc = occupancy(reinterpret_cast<const void*>(kernel), kda::tree_groups(W) * W * 32,
                             SM::bytes(kda::TREE_MAX, kda::KMAX, kda::tree_groups(W), W), &occ, &sms);
    if (rc != KDA_OK) return rc;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid, 1, 1);
    cfg.blockDim = dim3((unsigned)(32 * W * groups), 1, 1);
    cfg.dynamicSmemBytes = SM::bytes(prm.t, prm.k, groups, W);
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    set_pdl(cfg, &attr, flags);
    return cudaLaunchKernelEx(&cfg, kernel, prm, tree) == cudaSuccess ? KDA_OK : KDA_ERR_LAUNCH;
}

template <typename QT>
int launch_tree(const kda::StepParams& prm, const uint64_t* tree, uint32_t flags, cudaStream_t stream) {
    const int64_t heads = (int64_t)prm.n * prm.hv, all = heads * ((prm.v + kda::TREE_CW - 1) / kda::TREE_CW);
    // Few column groups: four warps each, for the time that a token takes; many: one, for the instructions.  12 heads of
    // 128, four against one, us (fp16 pool, trees of 32): 1 request 31, 61; 2: 35, 64; 4 (384 groups): 41, 49; 8: 64, 53;
    // 16: 104, 70.  (fp32: 31, 63; 35, 64; 45, 53; 70, 61; 115, 96.)  Two warps gain nothing between.
    const bool few = all <= 3 * kSms;
    // Groups of a CTA share the tokens' vectors; fewer while that leaves an SM without a CTA.
    int groups = kda::tree_groups(few ? 4 : 1);
    auto ctas = [&](int g) { return heads * ((prm.v + g * kda::TREE_CW - 1) / (g * kda::TREE_CW)); };
    while (groups > 1 && (ctas(groups) < kSms || (groups / 2) * kda::TREE_CW >= prm.v)) groups /= 2;
    return few ? launch_tree_warps<QT, 4>(prm, tree, groups, flags, stream) : launch_tree_warps<QT, 1>(prm, tree, groups, flags, stream);
}

template <typename ET, int VC, int KWM>
int launch_conv_width(cudaLaunchConfig_t& cfg, const kda::ConvParams& prm, const uint64_t* tree) {
    auto kernel = kda::kda_conv_tree_kernel<ET, VC, KWM>;
    using SM = kda::ConvTreeSmem<ET, VC>;
    int occ = 0, sms = 0;   // raises the kernel's limit to the most that any call takes
    const int rc = occupancy(reinterpret_cast<const void*>(kernel), (int)cfg.blockDim.x, SM::bytes(kda::TREE_MAX), &occ, &sms);
    if (rc != KDA_OK) return rc;
    cfg.dynamicSmemBytes = SM::bytes(prm.t);
    return cudaLaunchKernelEx(&cfg, kernel, prm, tree) == cudaSuccess ? KDA_OK : KDA_ERR_LAUNCH;
}

template <typename ET, int VC>
int launch_conv(const kda::ConvParams& prm, const uint64_t* tree, uint32_t flags, cudaStream_t stream) {
    const int64_t grid = (int64_t)((prm.C / VC + kda::CONV_TREE_CH - 1) / kda::CONV_TREE_CH) * prm.n;
    if (grid > 0x7fffffffLL) return KDA_ERR_SHAPE;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid, 1, 1);
    cfg.blockDim = dim3(kda::CONV_TREE_CH * kda::CONV_TREE_GROUPS, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    set_pdl(cfg, &attr, flags);
    return prm.KW <= 4 ? launch_conv_width<ET, VC, 4>(cfg, prm, tree) : launch_conv_width<ET, VC, 8>(cfg, prm, tree);
}

template <typename T>
cudaError_t launch_accept(const cudaLaunchConfig_t& cfg, const kda::AcceptParams& prm) {
    return prm.q != nullptr ? cudaLaunchKernelEx(&cfg, kda::kda_accept_kernel<T, true>, prm)
                            : cudaLaunchKernelEx(&cfg, kda::kda_accept_kernel<T, false>, prm);
}

}  // namespace

extern "C" {

int kda_step_tree(const kda_pool* pool, const kda_step_args* args, const uint64_t* tree, int32_t* dev_status, uint32_t flags,
                  void* stream) {
    if (args == nullptr) return KDA_ERR_NULL;
    const kda_step_args& g = *args;
    const int rc = check_pool_for_build(pool);
    if (rc != KDA_OK) return rc;
    if (g.n < 0 || g.total < 0 || g.max_t < 0 || g.reserved != 0 || g.in_place != 0) return KDA_ERR_ARG;
    if (flags & ~(uint32_t)KDA_LAUNCH_PDL) return KDA_ERR_ARG;
    if (elem_size(g.qkv_dtype) == 0) return KDA_ERR_DTYPE_UNSUPPORTED;
    if (g.h_qk < 1 || pool->hv % g.h_qk != 0 || g.num_cols < 1 || g.max_t > g.num_cols || g.max_t > KDA_TREE_MAX_TOKENS)
        return KDA_ERR_SHAPE;
    if (g.cu_seqlens == nullptr && (int64_t)g.total != (int64_t)g.n * g.max_t) return KDA_ERR_SHAPE;
    if (g.n == 0 || g.total == 0 || g.max_t == 0) return KDA_OK;
    if (!g.slot_table || !g.q || !g.k || !g.v || !g.a || !g.b || !g.o || !tree || !dev_status) return KDA_ERR_NULL;
    if (!aligned(g.slot_table, 4) || !aligned(dev_status, 4) || !aligned(g.b, 4) || !aligned(g.o, 4) || !aligned(tree, 8) ||
        !aligned(g.a, 16) || !aligned(g.q, 16) || !aligned(g.k, 16) || !aligned(g.v, 16) || !aligned(g.cu_seqlens, 4) ||
        !aligned(g.accepted, 4) || !aligned(g.a_log, 4) || !aligned(g.dt_bias, 4))
        return KDA_ERR_ALIGN;
    kda::StepParams prm = make_params(pool, g.slot_table, g.slot_table, g.reset, g.n, g.max_t, g.q, g.k, g.v, g.a, g.b, g.o,
                                      dev_status, flags);
    prm.hqk = g.h_qk;
    prm.init_stride = g.num_cols;
    prm.snap_stride = g.num_cols;
    prm.num_cols = g.num_cols;
    prm.accepted = g.accepted;
    prm.cu = g.cu_seqlens;
    prm.total = g.total;
    prm.a_log = g.a_log;
    prm.dt_bias = g.dt_bias;
    prm.mode = kda::MODE_PADDING;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    switch (g.qkv_dtype) {
        case KDA_F32: return launch_tree<float>(prm, tree, flags, st);
        case KDA_F16: return launch_tree<__half>(prm, tree, flags, st);
        default: return launch_tree<__nv_bfloat16>(prm, tree, flags, st);
    }
}

int kda_conv_step_tree(const kda_conv_window* win, const kda_conv_args* args, const uint64_t* tree, int32_t* dev_status,
                       uint32_t flags, void* stream) {
    if (win == nullptr || args == nullptr) return KDA_ERR_NULL;
    const kda_conv_args& g = *args;
    const int es = elem_size(win->dtype);
    if (es == 0) return KDA_ERR_DTYPE_UNSUPPORTED;
    if (win->reserved != 0 || g.reserved != 0 || g.n < 0 || g.total < 0 || g.max_t < 0 || (g.activation != 0 && g.activation != 1) ||
        (flags & ~(uint32_t)KDA_LAUNCH_PDL))
        return KDA_ERR_ARG;
    if (win->channels < 1 || g.kernel_width < 1 || g.kernel_width > kda::CONV_KW_MAX || win->state_len < g.kernel_width - 1 ||
        win->state_len > kda::CONV_L_MAX || win->num_slots < 1 || win->slot_stride < (int64_t)win->state_len * win->channels ||
        g.max_t > KDA_TREE_MAX_TOKENS)
        return KDA_ERR_SHAPE;
    if (g.cu_seqlens == nullptr && (int64_t)g.total != (int64_t)g.n * g.max_t) return KDA_ERR_SHAPE;
    if (g.n == 0 || g.total == 0 || g.max_t == 0) return KDA_OK;
    if (!win->base || !g.conv_slot || !g.x || !g.weight || !g.y || !tree || !dev_status) return KDA_ERR_NULL;
    if (!aligned(win->base, es) || !aligned(g.x, es) || !aligned(g.y, es) || !aligned(g.conv_slot, 4) || !aligned(g.weight, 4) ||
        !aligned(dev_status, 4) || !aligned(g.bias, 4) || !aligned(g.cu_seqlens, 4) || !aligned(g.accepted, 4) || !aligned(tree, 8))
        return KDA_ERR_ALIGN;
    kda::ConvParams prm = {};
    prm.window = win->base;
    prm.num_slots = win->num_slots;
    prm.slot_stride = win->slot_stride;
    prm.C = win->channels;
    prm.L = win->state_len;
    prm.KW = g.kernel_width;
    prm.n = g.n;
    prm.t = g.max_t;
    prm.total = g.total;
    prm.cu = g.cu_seqlens;
    prm.conv_slot = g.conv_slot;
    prm.accepted = g.accepted;
    prm.reset = g.reset;
    prm.x = g.x;
    prm.w = g.weight;
    prm.bias = g.bias;
    prm.y = g.y;
    prm.silu = g.activation;
    prm.flags = flags;
    prm.status = dev_status;
    // 16 bytes of channels a thread where the channel count and every address allow it, else one channel
    const int ve = 16 / es;
    const bool vec = win->channels % ve == 0 && win->slot_stride % ve == 0 && aligned(win->base, 16) && aligned(g.x, 16) &&
                     aligned(g.y, 16);
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    switch (win->dtype) {
        case KDA_F32: return vec ? launch_conv<float, 4>(prm, tree, flags, st) : launch_conv<float, 1>(prm, tree, flags, st);
        case KDA_F16: return vec ? launch_conv<__half, 8>(prm, tree, flags, st) : launch_conv<__half, 1>(prm, tree, flags, st);
        default: return vec ? launch_conv<__nv_bfloat16, 8>(prm, tree, flags, st) : launch_conv<__nv_bfloat16, 1>(prm, tree, flags, st);
    }
}

int kda_accept(const kda_accept_args* args, int32_t* dev_status, uint32_t flags, void* stream) {
    if (args == nullptr) return KDA_ERR_NULL;
    const kda_accept_args& g = *args;
    const int es = elem_size(g.dtype);
    if (es == 0) return KDA_ERR_DTYPE_UNSUPPORTED;
    if (g.n < 0 || g.total < 0 || g.max_t < 0 || g.reserved != 0 || (flags & ~(uint32_t)KDA_LAUNCH_PDL)) return KDA_ERR_ARG;
    if (g.vocab < 1 || g.vocab > KDA_ACCEPT_MAX_VOCAB || g.p_stride < g.vocab || (g.q && g.q_stride < g.vocab) ||
        g.max_t > KDA_TREE_MAX_TOKENS || g.n > 0x7fffffff / kda::ACC_CTAS)
        return KDA_ERR_SHAPE;
    if (g.cu_seqlens == nullptr && (int64_t)g.total != (int64_t)g.n * g.max_t) return KDA_ERR_SHAPE;
    if (g.n == 0 || g.max_t == 0) return KDA_OK;
    if (!g.accepted || !g.node || !g.path || !g.token || !dev_status) return KDA_ERR_NULL;
    if (g.total > 0 && (!g.p || !g.tokens || !g.u || !g.u_last)) return KDA_ERR_NULL;
    if (!aligned(g.p, es) || !aligned(g.q, es) || !aligned(g.tokens, 4) || !aligned(g.tree, 8) || !aligned(g.u, 4) ||
        !aligned(g.u_last, 4) || !aligned(g.cu_seqlens, 4) || !aligned(g.accepted, 4) || !aligned(g.node, 4) || !aligned(g.path, 4) ||
        !aligned(g.token, 4) || !aligned(dev_status, 4))
        return KDA_ERR_ALIGN;
    kda::AcceptParams prm;
    prm.p = g.p;
    prm.q = g.q;
    prm.p_stride = g.p_stride;
    prm.q_stride = g.q_stride;
    prm.n = g.n;
    prm.total = g.total;
    prm.max_t = g.max_t;
    prm.vocab = g.vocab;
    prm.cu = g.cu_seqlens;
    prm.tokens = g.tokens;
    prm.tree = g.tree;
    prm.u = g.u;
    prm.u_last = g.u_last;
    prm.accepted = g.accepted;
    prm.node = g.node;
    prm.path = g.path;
    prm.token = g.token;
    prm.status = dev_status;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)g.n * kda::ACC_CTAS, 1, 1);
    cfg.blockDim = dim3(kda::ACC_THREADS, 1, 1);
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr;
    set_pdl(cfg, &attr, flags);
    cudaError_t err;
    switch (g.dtype) {
        case KDA_F32: err = launch_accept<float>(cfg, prm); break;
        case KDA_F16: err = launch_accept<__half>(cfg, prm); break;
        default: err = launch_accept<__nv_bfloat16>(cfg, prm); break;
    }
    return err == cudaSuccess ? KDA_OK : KDA_ERR_LAUNCH;
}

}  // extern "C"
