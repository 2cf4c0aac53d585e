// C ABI of the operators around the recurrence (declared in include/kda.h):
// the 4-bit paged key/value cache and its attention, and the norms.  None of
// them depends on the state pool's dtype; both library builds carry them.
//
// Host side: validate every argument synchronously and enqueue one kernel on
// the caller's stream; the attention of wide trees enqueues a second one behind
// it, which joins parts (if that launch fails, the call says so with the first
// one enqueued).
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "kda.h"
#include "kda_host.cuh"
#include "kda_kv4.cuh"
#include "kda_kv4_tree.cuh"
#include "kda_norm.cuh"

namespace {

int check_cache(const kda_kv4_cache* c) {
    if (c == nullptr) return KDA_ERR_NULL;
    if (c->reserved != 0) return KDA_ERR_ARG;
    int64_t bytes = 0;
    const int rc = kda_kv4_page_bytes(c->page_tokens, c->heads, c->dim, &bytes);
    if (rc != KDA_OK) return rc;
    if (c->num_pages < 1 || c->num_pages > 0x7fffffffLL || c->page_stride < bytes) return KDA_ERR_SHAPE;
    if (!(c->k_scale > 0.f) || !(c->v_scale > 0.f) || std::isinf(c->k_scale) || std::isinf(c->v_scale)) return KDA_ERR_ARG;
    return KDA_OK;
}

// What append and attend share: counts, table, rotation.
struct Common {
    int32_t n, total, max_t, cols, rot, inter, rope_rows;
    const void *cu, *table, *ctx, *cos, *sin;
};

int check_common(const kda_kv4_cache* c, const Common& g) {
    if (g.n < 0 || g.total < 0 || g.max_t < 0 || (g.inter != 0 && g.inter != 1)) return KDA_ERR_ARG;
    // the kernels round requests up to 32 and tokens up to 8 in 32 bits
    if (g.n > KDA_KV4_MAX_COUNT || g.total > KDA_KV4_MAX_COUNT) return KDA_ERR_SHAPE;
    // positions, rounded up to a unit of keys, stay below 2^31
    if (g.cols < 1 || (int64_t)g.cols * c->page_tokens > 0x7fffffffLL - kda::KV4_KEYS || g.rot < 0 || g.rot > c->dim || g.rot % 32 != 0 ||
        (g.rot > 0 && g.rope_rows < 1))
        return KDA_ERR_SHAPE;
    if (g.cu == nullptr && (int64_t)g.total != (int64_t)g.n * g.max_t) return KDA_ERR_SHAPE;
    return KDA_OK;
}

int check_common_pointers(const kda_kv4_cache* c, const Common& g, const int32_t* status) {
    if (!c->base || !g.table || !g.ctx || !status || (g.rot > 0 && (!g.cos || !g.sin))) return KDA_ERR_NULL;
    if (!aligned(c->base, 16) || c->page_stride % 16 != 0 || !aligned(g.table, 4) || !aligned(g.ctx, 4) || !aligned(status, 4) ||
        !aligned(g.cu, 4) || !aligned(g.cos, 16) || !aligned(g.sin, 16))
        return KDA_ERR_ALIGN;
    return KDA_OK;
}

template <int D, int MODE, bool TREE>
int launch_attend(kda::Kv4AttendParams& prm, int64_t list, uint32_t flags, cudaStream_t stream) {
    auto kernel = kda::kda_kv4_attend_kernel<D, MODE, TREE>;
    int occ = 0, sms = 0;
    const int rc = occupancy(reinterpret_cast<const void*>(kernel), kda::Kv4Shape<D, MODE>::THREADS, kda::Kv4Smem<D, MODE>::BYTES, &occ, &sms);
    if (rc != KDA_OK) return rc;
    // every CTA resident, and none without a unit for each of its warps
    int64_t grid = std::min<int64_t>((int64_t)occ * sms, kda::KV4_MAX_CTAS);
    grid = std::max<int64_t>(1, std::min(grid, list / kda::Kv4Shape<D, MODE>::WARPS + 1));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid, 1, 1);
    cfg.blockDim = dim3(kda::Kv4Shape<D, MODE>::THREADS, 1, 1);
    cfg.dynamicSmemBytes = kda::Kv4Smem<D, MODE>::BYTES;
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    set_pdl(cfg, &attr, flags);
    return cudaLaunchKernelEx(&cfg, kernel, prm) == cudaSuccess ? KDA_OK : KDA_ERR_LAUNCH;
}

// The wide tree's kernel and the join of its parts behind it.
template <int D, bool SPLIT>
int launch_tree(kda::Kv4AttendParams& prm, int64_t list, uint32_t flags, cudaStream_t stream) {
    using SM = kda::KvtSmem<D, SPLIT>;
    auto kernel = kda::kda_kv4_tree_kernel<D, SPLIT>;
    int occ = 0, sms = 0;
    const int rc = occupancy(reinterpret_cast<const void*>(kernel), kda::KVT_THREADS, SM::BYTES, &occ, &sms);
    if (rc != KDA_OK) return rc;
    // every CTA resident (the occupancy call does not know how much tensor memory a kernel takes and answers 1); none
    // without four units
    int64_t grid = std::min<int64_t>((int64_t)SM::CTAS * sms, kda::KVT_MAX_CTAS);
    grid = std::max<int64_t>(1, std::min(grid, list / 4));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid, 1, 1);
    cfg.blockDim = dim3(kda::KVT_THREADS, 1, 1);
    cfg.dynamicSmemBytes = SM::BYTES;
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    set_pdl(cfg, &attr, flags);
    if (cudaLaunchKernelEx(&cfg, kernel, prm) != cudaSuccess) return KDA_ERR_LAUNCH;
    if (grid == 1) return KDA_OK;
    cudaLaunchConfig_t join = {};
    join.gridDim = dim3((unsigned)(grid - 1) * kda::KVT_JOIN_GROUPS, 1, 1);
    join.blockDim = dim3(256, 1, 1);
    join.stream = stream;
    cudaLaunchAttribute after;
    set_pdl(join, &after, KDA_LAUNCH_PDL);      // its CTAs wait for the kernel's end themselves
    return cudaLaunchKernelEx(&join, kda::kda_kv4_tree_join_kernel<D>, prm) == cudaSuccess ? KDA_OK : KDA_ERR_LAUNCH;
}

template <bool TREE>
int append(const kda_kv4_cache* cache, const kda_kv4_append_args* args, const uint64_t* tree, int32_t* dev_status, uint32_t flags,
           void* stream) {
    if (args == nullptr) return KDA_ERR_NULL;
    int rc = check_cache(cache);
    if (rc != KDA_OK) return rc;
    const kda_kv4_append_args& g = *args;
    const int es = elem_size(g.dtype);
    if (es == 0 || ((g.k_out || g.v_out) && elem_size(g.out_dtype) == 0)) return KDA_ERR_DTYPE_UNSUPPORTED;
    const Common c = {g.n, g.total, g.max_t, g.table_cols, g.rot_dim, g.interleaved, g.rope_rows,
                      g.cu_seqlens, g.page_table, g.ctx_len, g.cos, g.sin};
    if (flags & ~(uint32_t)KDA_LAUNCH_PDL) return KDA_ERR_ARG;
    rc = check_common(cache, c);
    if (rc != KDA_OK) return rc;
    if (g.reserved != 0) return KDA_ERR_ARG;
    const int64_t row = (int64_t)cache->heads * cache->dim;
    if (g.k_stride < row || g.v_stride < row || (TREE && g.max_t > kda::TREE_MAX)) return KDA_ERR_SHAPE;
    if (g.n == 0 || g.total == 0 || g.max_t == 0) return KDA_OK;
    rc = check_common_pointers(cache, c, dev_status);
    if (rc != KDA_OK) return rc;
    if (!g.k || !g.v || (TREE && !tree)) return KDA_ERR_NULL;
    if (!aligned(tree, 8) || !aligned(g.k, 16) || !aligned(g.v, 16) || g.k_stride * es % 16 != 0 || g.v_stride * es % 16 != 0 ||
        !aligned(g.k_out, 16) || !aligned(g.v_out, 16))
        return KDA_ERR_ALIGN;
    kda::Kv4AppendParams prm;
    prm.pages = static_cast<uint8_t*>(cache->base);
    prm.num_pages = cache->num_pages;
    prm.page_stride = cache->page_stride;
    prm.page_tokens = cache->page_tokens;
    prm.heads = cache->heads;
    prm.n = g.n;
    prm.total = g.total;
    prm.max_t = g.max_t;
    prm.dtype = g.dtype;
    prm.cols = g.table_cols;
    prm.rot = g.rot_dim;
    prm.inter = g.interleaved;
    prm.rope_rows = g.rope_rows;
    prm.k_stride = g.k_stride;
    prm.v_stride = g.v_stride;
    prm.cu = g.cu_seqlens;
    prm.table = g.page_table;
    prm.ctx = g.ctx_len;
    prm.k = g.k;
    prm.v = g.v;
    prm.cos = g.cos;
    prm.sin = g.sin;
    prm.k_out = g.k_out;
    prm.v_out = g.v_out;
    prm.out_dtype = g.out_dtype;
    prm.k_scale = cache->k_scale;
    prm.v_scale = cache->v_scale;
    prm.inv_k = 1.0f / cache->k_scale;
    prm.inv_v = 1.0f / cache->v_scale;
    prm.status = dev_status;
    prm.tree = tree;
    // eight tokens a CTA; few tokens share their heads out over more CTAs
    const int tokens = (int)(((int64_t)g.total + 7) / 8), items = cache->dim == 128 ? cache->heads * 2 : (cache->heads + 1) / 2 * 2;
    const int parts = std::max(1, std::min((items + kda::KV4_APPEND_WARPS - 1) / kda::KV4_APPEND_WARPS, kda::KV4_APPEND_CTAS / tokens));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)tokens, (unsigned)parts, 1);
    cfg.blockDim = dim3(kda::KV4_APPEND_THREADS, 1, 1);
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr;
    set_pdl(cfg, &attr, flags);
    using namespace kda;
    const cudaError_t err =
        cache->dim == 128 ? (es == 2 ? cudaLaunchKernelEx(&cfg, kda_kv4_append_kernel<128, 2, TREE>, prm)
                                     : cudaLaunchKernelEx(&cfg, kda_kv4_append_kernel<128, 4, TREE>, prm))
                          : (es == 2 ? cudaLaunchKernelEx(&cfg, kda_kv4_append_kernel<64, 2, TREE>, prm)
                                     : cudaLaunchKernelEx(&cfg, kda_kv4_append_kernel<64, 4, TREE>, prm));
    return err == cudaSuccess ? KDA_OK : KDA_ERR_LAUNCH;
}

template <bool TREE>
int attend(const kda_kv4_cache* cache, const kda_kv4_attend_args* args, const uint64_t* tree, int32_t* dev_status, uint32_t flags,
           void* stream) {
    if (args == nullptr) return KDA_ERR_NULL;
    int rc = check_cache(cache);
    if (rc != KDA_OK) return rc;
    const kda_kv4_attend_args& g = *args;
    const int es = elem_size(g.dtype);
    if (es == 0) return KDA_ERR_DTYPE_UNSUPPORTED;
    const Common c = {g.n, g.total, g.max_t, g.table_cols, g.rot_dim, g.interleaved, g.rope_rows,
                      g.cu_seqlens, g.page_table, g.ctx_len, g.cos, g.sin};
    if (flags & ~(uint32_t)(KDA_LAUNCH_PDL | KDA_LAUNCH_TEST_WITHHOLD_STATE)) return KDA_ERR_ARG;
    rc = check_common(cache, c);
    if (rc != KDA_OK) return rc;
    if (g.reserved != 0 || g.window < 0 || !std::isfinite(g.scale)) return KDA_ERR_ARG;
    if (g.h_q < 1 || g.h_q % cache->heads != 0 || g.max_t > (TREE ? kda::TREE_MAX : KDA_KV4_MAX_TOKENS) || g.q_stride < (int64_t)g.h_q * cache->dim)
        return KDA_ERR_SHAPE;
    // the wide tree's units of keys, too, end below 2^31
    if (TREE && (int64_t)g.table_cols * cache->page_tokens > 0x7fffffffLL - kda::KVT_KEYS) return KDA_ERR_SHAPE;
    const int grp = g.h_q / cache->heads;
    // rows of a tile and their rounding (kda_kv4.cuh)
    const int mode = g.dtype != KDA_BF16 ? kda::KV4_REST : (int64_t)g.max_t * grp <= 8 ? kda::KV4_8 : kda::KV4_16;
    const int rows = mode == kda::KV4_16 ? 16 : 8;
    const int64_t units = ((int64_t)g.table_cols * cache->page_tokens + kda::KV4_KEYS - 1) / kda::KV4_KEYS;
    const int64_t tiles = ((int64_t)g.max_t * grp + rows - 1) / rows;
    if ((units + kda::KV4_PART) * tiles * cache->heads > 0x7fffffffLL) return KDA_ERR_SHAPE;
    if (g.n == 0 || g.total == 0 || g.max_t == 0) return KDA_OK;
    rc = check_common_pointers(cache, c, dev_status);
    if (rc != KDA_OK) return rc;
    if (!g.q || !g.o || !g.workspace || (TREE && !tree)) return KDA_ERR_NULL;
    if (!aligned(tree, 8) || !aligned(g.q, 16) || g.q_stride * es % 16 != 0 || !aligned(g.o, 16) || !aligned(g.workspace, 16)) return KDA_ERR_ALIGN;
    if (g.workspace_bytes < (TREE ? KDA_KV4_TREE_WORKSPACE_BYTES : KDA_KV4_WORKSPACE_BYTES)) return KDA_ERR_SHAPE;
    kda::Kv4AttendParams prm;
    prm.pages = static_cast<const uint8_t*>(cache->base);
    prm.num_pages = cache->num_pages;
    prm.page_stride = cache->page_stride;
    prm.page_tokens = cache->page_tokens;
    prm.heads = cache->heads;
    prm.n = g.n;
    prm.total = g.total;
    prm.max_t = g.max_t;
    prm.dtype = g.dtype;
    prm.cols = g.table_cols;
    prm.rot = g.rot_dim;
    prm.inter = g.interleaved;
    prm.rope_rows = g.rope_rows;
    prm.h_q = g.h_q;
    prm.grp = grp;
    prm.window = g.window;
    prm.q_stride = g.q_stride;
    prm.cu = g.cu_seqlens;
    prm.table = g.page_table;
    prm.ctx = g.ctx_len;
    prm.q = g.q;
    prm.cos = g.cos;
    prm.sin = g.sin;
    prm.o = g.o;
    const float scale = g.scale == 0.f ? 1.0f / std::sqrt((float)cache->dim) : g.scale;
    prm.scale_log2 = (float)((double)scale * cache->k_scale * 1.4426950408889634);
    prm.v_scale = cache->v_scale;
    prm.counters = static_cast<int32_t*>(g.workspace);
    prm.partials = reinterpret_cast<float*>(static_cast<char*>(g.workspace) + kda::KV4_MAX_CTAS * sizeof(int32_t));
    prm.status = dev_status;
    prm.tree = tree;
    prm.withhold = (flags & KDA_LAUNCH_TEST_WITHHOLD_STATE) != 0;
    static_assert(kda::KV4_MAX_CTAS * (4 + 2 * kda::KV4_ROWS * (128 + 2) * 4) <= KDA_KV4_WORKSPACE_BYTES, "workspace");
    const int64_t list = units * std::min<int64_t>(tiles * cache->heads * g.n, 1 << 20);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    using namespace kda;
    if (TREE && (int64_t)g.max_t * grp > KVT_MIN_ROWS) {
        static_assert(KVT_COUNTERS + KVT_HEAD + 2LL * KVT_MAX_CTAS * KvtPart<128>::FLOATS * 4 <= KDA_KV4_TREE_WORKSPACE_BYTES, "workspace");
        static_assert(KV4_MAX_CTAS * sizeof(int32_t) <= KVT_COUNTERS, "the other kernel's counters stay zero");
        const int64_t wide = ((int64_t)g.table_cols * cache->page_tokens + KVT_KEYS - 1) / KVT_KEYS * cache->heads * g.n *
                             (((int64_t)g.max_t * grp + KVT_ROWS - 1) / KVT_ROWS);
        const bool split = g.dtype != KDA_BF16;
        prm.counters = reinterpret_cast<int32_t*>(static_cast<char*>(g.workspace) + KVT_COUNTERS);
        prm.partials = reinterpret_cast<float*>(static_cast<char*>(g.workspace) + KVT_COUNTERS + KVT_HEAD);
        if (cache->dim == 128) return split ? launch_tree<128, true>(prm, wide, flags, st) : launch_tree<128, false>(prm, wide, flags, st);
        return split ? launch_tree<64, true>(prm, wide, flags, st) : launch_tree<64, false>(prm, wide, flags, st);
    }
    if (cache->dim == 128)
        return mode == KV4_8 ? launch_attend<128, KV4_8, TREE>(prm, list, flags, st)
               : mode == KV4_16 ? launch_attend<128, KV4_16, TREE>(prm, list, flags, st)
                                : launch_attend<128, KV4_REST, TREE>(prm, list, flags, st);
    return mode == KV4_8 ? launch_attend<64, KV4_8, TREE>(prm, list, flags, st)
           : mode == KV4_16 ? launch_attend<64, KV4_16, TREE>(prm, list, flags, st)
                            : launch_attend<64, KV4_REST, TREE>(prm, list, flags, st);
}

template <typename OT, typename T>
cudaError_t launch_head_norm(const cudaLaunchConfig_t& cfg, const kda::HeadNormParams& prm, int lpr_log2) {
    return cudaLaunchKernelEx(&cfg, kda::kda_head_norm_kernel<OT, T>, prm, lpr_log2);
}
template <typename OT>
cudaError_t launch_head_norm_t(const cudaLaunchConfig_t& cfg, const kda::HeadNormParams& prm, int lpr_log2, int32_t dtype) {
    switch (dtype) {
        case KDA_F32: return launch_head_norm<OT, float>(cfg, prm, lpr_log2);
        case KDA_F16: return launch_head_norm<OT, __half>(cfg, prm, lpr_log2);
        default: return launch_head_norm<OT, __nv_bfloat16>(cfg, prm, lpr_log2);
    }
}

// Rows in turn over CTAs that all fit the card at once, eight channels a thread.
template <typename T, typename R, bool SHIFT>
cudaError_t launch_block_norm_rows(cudaLaunchConfig_t& cfg, const kda::BlockNormParams& prm, int units) {
    auto kernel = kda::kda_block_norm_kernel<T, R, SHIFT>;
    const int threads = (units + 31) / 32 * 32;
    int occ = 0, sms = 0;
    const size_t smem = kda::block_norm_smem<T, R>(threads);
    if (occupancy(reinterpret_cast<const void*>(kernel), threads, smem, &occ, &sms) != KDA_OK) return cudaErrorUnknown;
    cfg.dynamicSmemBytes = smem;
    const int most = SHIFT ? occ * sms & ~7 : occ * sms;   // see the kernel
    cfg.gridDim = dim3((unsigned)std::min(prm.total, most));
    cfg.blockDim = dim3(threads);
    return cudaLaunchKernelEx(&cfg, kernel, prm);
}

// vec: buffers start on 16 bytes and every stride is the width apart from a multiple of eight
template <typename T, typename R>
cudaError_t launch_block_norm(cudaLaunchConfig_t& cfg, const kda::BlockNormParams& prm, bool vec) {
    const bool shift = prm.hidden % 8 != 0;
    const int units = shift ? (prm.hidden + 14) / 8 : prm.hidden / 8;   // vectors that a row can touch
    if (vec && units <= 1024)
        return shift ? launch_block_norm_rows<T, R, true>(cfg, prm, units) : launch_block_norm_rows<T, R, false>(cfg, prm, units);
    const int nv = prm.hidden <= 4096 ? 4 : 16;
    cfg.gridDim = dim3((unsigned)prm.total);
    cfg.blockDim = dim3(((prm.hidden + nv - 1) / nv + 31) / 32 * 32);
    return nv == 4 ? cudaLaunchKernelEx(&cfg, kda::kda_block_norm_any_kernel<T, R, 4>, prm)
                   : cudaLaunchKernelEx(&cfg, kda::kda_block_norm_any_kernel<T, R, 16>, prm);
}

}  // namespace

extern "C" {

int kda_kv4_page_bytes(int32_t page_tokens, int32_t heads, int32_t dim, int64_t* bytes) {
    if (bytes == nullptr) return KDA_ERR_NULL;
    if (page_tokens < 16 || page_tokens % 16 != 0 || page_tokens > 65536 || heads < 1 || heads > 65536 ||
        (dim != 64 && dim != 128))
        return KDA_ERR_SHAPE;
    *bytes = (int64_t)page_tokens / 16 * heads * 18 * dim;
    return KDA_OK;
}

int kda_kv4_append(const kda_kv4_cache* cache, const kda_kv4_append_args* args, int32_t* dev_status, uint32_t flags,
                   void* stream) {
    return append<false>(cache, args, nullptr, dev_status, flags, stream);
}

int kda_kv4_append_tree(const kda_kv4_cache* cache, const kda_kv4_append_args* args, const uint64_t* tree, int32_t* dev_status,
                        uint32_t flags, void* stream) {
    return append<true>(cache, args, tree, dev_status, flags, stream);
}

int kda_kv4_attend(const kda_kv4_cache* cache, const kda_kv4_attend_args* args, int32_t* dev_status, uint32_t flags,
                   void* stream) {
    return attend<false>(cache, args, nullptr, dev_status, flags, stream);
}

int kda_kv4_attend_tree(const kda_kv4_cache* cache, const kda_kv4_attend_args* args, const uint64_t* tree, int32_t* dev_status,
                        uint32_t flags, void* stream) {
    return attend<true>(cache, args, tree, dev_status, flags, stream);
}

int kda_head_norm(const kda_head_norm_args* args, uint32_t flags, void* stream) {
    if (args == nullptr) return KDA_ERR_NULL;
    const kda_head_norm_args& g = *args;
    const int eo = elem_size(g.o_dtype), es = elem_size(g.dtype);
    if (eo == 0 || es == 0) return KDA_ERR_DTYPE_UNSUPPORTED;
    if (g.total < 0 || g.activation < 0 || g.activation > 2 || !(g.eps >= 0.f) || g.reserved != 0 ||
        (flags & ~(uint32_t)KDA_LAUNCH_PDL))
        return KDA_ERR_ARG;
    if (g.heads < 1 || g.dim < 8 || g.dim > 256 || g.dim % 8 != 0 ||
        (g.gate && g.gate_stride < (int64_t)g.heads * g.dim))
        return KDA_ERR_SHAPE;
    if (g.total == 0) return KDA_OK;
    if (!g.o || !g.weight || !g.y) return KDA_ERR_NULL;
    if (!aligned(g.o, 16) || !aligned(g.gate, 16) || !aligned(g.weight, 16) || !aligned(g.y, 16) ||
        (g.gate && g.gate_stride * es % 16 != 0))
        return KDA_ERR_ALIGN;
    kda::HeadNormParams prm;
    prm.o = g.o;
    prm.gate = g.gate;
    prm.weight = g.weight;
    prm.y = g.y;
    prm.rows = (int64_t)g.total * g.heads;
    prm.gate_stride = g.gate_stride;
    prm.heads = g.heads;
    prm.dim = g.dim;
    prm.act = g.activation;
    prm.eps = g.eps;
    int lpr_log2 = 0;
    while ((8 << lpr_log2) < g.dim) ++lpr_log2;
    const int64_t per = kda::HEAD_NORM_THREADS >> lpr_log2, ctas = (prm.rows + per - 1) / per;
    if (prm.rows > 0x7fffffffLL) return KDA_ERR_SHAPE;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas, 1, 1);
    cfg.blockDim = dim3(kda::HEAD_NORM_THREADS, 1, 1);
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr;
    set_pdl(cfg, &attr, flags);
    cudaError_t err;
    switch (g.o_dtype) {
        case KDA_F32: err = launch_head_norm_t<float>(cfg, prm, lpr_log2, g.dtype); break;
        case KDA_F16: err = launch_head_norm_t<__half>(cfg, prm, lpr_log2, g.dtype); break;
        default: err = launch_head_norm_t<__nv_bfloat16>(cfg, prm, lpr_log2, g.dtype); break;
    }
    return err == cudaSuccess ? KDA_OK : KDA_ERR_LAUNCH;
}

int kda_block_norm(const kda_block_norm_args* args, uint32_t flags, void* stream) {
    if (args == nullptr) return KDA_ERR_NULL;
    const kda_block_norm_args& g = *args;
    const int es = elem_size(g.dtype), er = elem_size(g.residual_dtype);
    if (es == 0 || (g.residual_dtype != KDA_F32 && g.residual_dtype != g.dtype)) return KDA_ERR_DTYPE_UNSUPPORTED;
    if (g.total < 0 || g.activation < 0 || g.activation > 2 || !(g.eps >= 0.f) ||
        (flags & ~(uint32_t)KDA_LAUNCH_PDL))
        return KDA_ERR_ARG;
    if (g.hidden < 1 || g.hidden > KDA_BLOCK_NORM_MAX || (g.y && g.y_stride < g.hidden) ||
        (g.gate && g.gate_stride < g.hidden))
        return KDA_ERR_SHAPE;
    if (g.total == 0) return KDA_OK;
    if (!g.residual || (!g.y && !g.x) || (g.y && !g.residual_out) || (!g.y && (g.gate || g.w_post || g.scale)))
        return KDA_ERR_NULL;
    const void* typed[4] = {g.y, g.gate, g.x, nullptr};
    const void* res[2] = {g.residual, g.residual_out};
    const void* w[3] = {g.w_post, g.scale, g.w_pre};
    // eight channels an access when buffers start on 16 bytes and rows keep in step (launch_block_norm), else one
    bool vec = (!g.y || (g.y_stride - g.hidden) % 8 == 0) && (!g.gate || (g.gate_stride - g.hidden) % 8 == 0);
    for (const void* t : typed) {
        if (!aligned(t, es)) return KDA_ERR_ALIGN;
        vec = vec && aligned(t, 16);
    }
    for (const void* t : res) {
        if (!aligned(t, er)) return KDA_ERR_ALIGN;
        vec = vec && aligned(t, 16);
    }
    for (const void* t : w) {
        if (!aligned(t, 4)) return KDA_ERR_ALIGN;
        vec = vec && (g.hidden % 8 != 0 || aligned(t, 16));
    }
    kda::BlockNormParams prm;
    prm.residual = g.residual;
    prm.y = g.y;
    prm.gate = g.gate;
    prm.w_post = g.w_post;
    prm.scale = g.scale;
    prm.w_pre = g.w_pre;
    prm.residual_out = g.residual_out;
    prm.x = g.x;
    prm.y_stride = g.y_stride;
    prm.gate_stride = g.gate_stride;
    prm.total = g.total;
    prm.hidden = g.hidden;
    prm.act = g.activation;
    prm.eps = g.eps;
    prm.residual_scale = g.residual_scale;
    prm.branch_scale = g.branch_scale;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)g.total, 1, 1);
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr;
    set_pdl(cfg, &attr, flags);
    cudaError_t err;
    if (g.dtype == KDA_F32) err = launch_block_norm<float, float>(cfg, prm, vec);
    else if (g.dtype == KDA_F16)
        err = g.residual_dtype == KDA_F32 ? launch_block_norm<__half, float>(cfg, prm, vec)
                                          : launch_block_norm<__half, __half>(cfg, prm, vec);
    else
        err = g.residual_dtype == KDA_F32 ? launch_block_norm<__nv_bfloat16, float>(cfg, prm, vec)
                                          : launch_block_norm<__nv_bfloat16, __nv_bfloat16>(cfg, prm, vec);
    return err == cudaSuccess ? KDA_OK : KDA_ERR_LAUNCH;
}

}  // extern "C"
