// Host helpers that the library's translation units share.
#pragma once

#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <map>
#include <mutex>
#include <tuple>
#include <utility>

#include "kda.h"
#include "kda_common.cuh"

#ifndef KDA_STATE16
#error "build with -DKDA_STATE16=0 (fp32 pool) or -DKDA_STATE16=1 (fp16 pool)"
#endif

namespace {

constexpr int kBuildDtype = KDA_STATE16 ? KDA_F16 : KDA_F32;


int elem_size(int32_t dtype) {
    switch (dtype) {
        case KDA_F32: return 4;
        case KDA_F16: return 2;
        case KDA_BF16: return 2;
        default: return 0;
    }
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Resident CTAs per SM of `kernel` with `smem` dynamic bytes (also raises the
// kernel's dynamic shared-memory limit); cached per (kernel, device, threads).
int occupancy(const void* kernel, int threads, size_t smem, int* blocks_per_sm, int* sms) try {
    static std::mutex mu;
    static std::map<std::pair<const void*, int>, size_t> limit;
    static std::map<std::tuple<const void*, int, int>, std::pair<int, int>> cache;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return KDA_ERR_LAUNCH;
    std::lock_guard<std::mutex> lock(mu);
    auto it = cache.find({kernel, dev, threads});
    if (it == cache.end()) {
        int occ = 0, count = 0;
        size_t& most = limit[{kernel, dev}];
        if ((smem > most && cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) !=
                                cudaSuccess) ||
            cudaOccupancyMaxActiveBlocksPerMultiprocessor(&occ, kernel, threads, smem) != cudaSuccess ||
            cudaDeviceGetAttribute(&count, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
            occ < 1)
            return KDA_ERR_LAUNCH;
        most = std::max(most, smem);   // only ever raised: the same kernel runs with fewer threads and bytes too
        it = cache.emplace(std::make_tuple(kernel, dev, threads), std::make_pair(occ, count)).first;
    }
    *blocks_per_sm = it->second.first;
    *sms = it->second.second;
    return KDA_OK;
} catch (...) {  // no memory for the cache: nothing leaves a C entry point as an exception
    return KDA_ERR_LAUNCH;
}

// Shape, alignment and dtype of one pool, without the build-dtype rule.
[[maybe_unused]] int check_pool_self(const kda_pool* p) {
    if (p == nullptr) return KDA_ERR_NULL;
    if (p->dtype != KDA_F32 && p->dtype != KDA_F16) return KDA_ERR_DTYPE_UNSUPPORTED;
    if (p->base == nullptr) return KDA_ERR_NULL;
    if (p->hv < 1 || p->num_slots < 1) return KDA_ERR_SHAPE;
    if (p->k < 16 || p->k > kda::KMAX || p->k % 16 != 0) return KDA_ERR_SHAPE;
    if (p->v < 16 || p->v > kda::KMAX || p->v % 16 != 0) return KDA_ERR_SHAPE;
    const int64_t per_slot = (int64_t)p->hv * p->k * p->v;
    if (p->slot_stride < per_slot) return KDA_ERR_SHAPE;
    if (p->num_slots > 0x7fffffffLL) return KDA_ERR_SHAPE;  // slot ids are int32
    const int es = elem_size(p->dtype);
    if (!aligned(p->base, 16) || (p->slot_stride * es) % 16 != 0) return KDA_ERR_ALIGN;
    return KDA_OK;
}

[[maybe_unused]] int check_pool_for_build(const kda_pool* p) {
    const int rc = check_pool_self(p);
    if (rc != KDA_OK) return rc;
    if (p->dtype != kBuildDtype) return KDA_ERR_DTYPE_MISMATCH;
    return KDA_OK;
}

// The parameters of plain decode and verify; the general forms change them.
[[maybe_unused]] kda::StepParams make_params(const kda_pool* pool, const int32_t* init_slot,
                            const int32_t* snap_slot, const uint8_t* reset, int32_t n,
                            int32_t t, const void* q, const void* k, const void* v,
                            const float* a, const float* b, float* o, int32_t* dev_status,
                            uint32_t flags) {
    kda::StepParams prm;
    prm.pool = pool->base;
    prm.num_slots = pool->num_slots;
    prm.slot_stride = pool->slot_stride;
    prm.hv = pool->hv;
    prm.k = pool->k;
    prm.v = pool->v;
    prm.n = n;
    prm.t = t;
    prm.init_slot = init_slot;
    prm.snap_slot = snap_slot;
    prm.reset = reset;
    prm.q = q;
    prm.kk = k;
    prm.vv = v;
    prm.a = a;
    prm.b = b;
    prm.o = o;
    prm.status = dev_status;
    prm.inv_sqrt_k = 1.0f / std::sqrt((float)pool->k);
    prm.flags = flags;
    // plain decode / verify: one q/k head per value head, one slot per request
    // row (init), t snapshot columns, no accepted column, no offsets, plain gate
    prm.hqk = pool->hv;
    prm.init_stride = 1;
    prm.snap_stride = t;
    prm.num_cols = 1;
    prm.accepted = nullptr;
    prm.cu = nullptr;
    prm.a_log = nullptr;
    prm.dt_bias = nullptr;
    prm.mode = 0;
    prm.total = n * t;
    prm.final_slot = nullptr;
    prm.conv = kda::StepParams::Conv{};
    return prm;
}

// Programmatic dependent launch attribute when the caller asked for it.
void set_pdl(cudaLaunchConfig_t& cfg, cudaLaunchAttribute* attr, uint32_t flags) {
    if (flags & KDA_LAUNCH_PDL) {
        attr->id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr->val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
    }
}

}  // namespace
