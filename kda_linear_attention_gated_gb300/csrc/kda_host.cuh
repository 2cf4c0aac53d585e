// Host helpers that the library's translation units share.
#pragma once

#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <map>
#include <mutex>
#include <tuple>
#include <utility>

#include "kda.h"

namespace {

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
