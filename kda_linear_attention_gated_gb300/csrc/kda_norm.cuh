// The norms around a block: the per-head norm and output gate behind the
// recurrence (kda_head_norm), and the norms, gate and scaled residual between
// two blocks (kda_block_norm).  Both read and write every element once; sums
// and products are fp32, each output is rounded once, to nearest even.
#pragma once

#include "kda_common.cuh"

namespace kda {

// Eight elements <-> fp32 registers by 16-byte accesses.
template <typename T> __device__ __forceinline__ void ld8(const T* p, float (&x)[8]) {
    if constexpr (sizeof(T) == 4) {
        const float4 a = __ldcs(reinterpret_cast<const float4*>(p)), b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
        x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    } else {
        const uint4 v = __ldcs(reinterpret_cast<const uint4*>(p));
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float2 f;
            if constexpr (sizeof(T) == 2 && __is_same(T, __half)) f = __half22float2(*reinterpret_cast<const __half2*>(&w[e]));
            else f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[e]));
            x[2 * e] = f.x;
            x[2 * e + 1] = f.y;
        }
    }
}
template <typename T> __device__ __forceinline__ uint32_t pack2(float a, float b) {
    if constexpr (__is_same(T, __half)) {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
}
template <typename T> __device__ __forceinline__ void st8(T* p, const float (&x)[8]) {
    if constexpr (sizeof(T) == 4) {
        reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
        reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
    } else {
        *reinterpret_cast<uint4*>(p) = make_uint4(pack2<T>(x[0], x[1]), pack2<T>(x[2], x[3]), pack2<T>(x[4], x[5]),
                                                  pack2<T>(x[6], x[7]));
    }
}
template <typename T> __device__ __forceinline__ T from_f32(float x) {
    if constexpr (sizeof(T) == 4) return x;
    else if constexpr (__is_same(T, __half)) return __float2half_rn(x);
    else return __float2bfloat16_rn(x);
}

// The gate's factor: 0 the gate itself, 1 sigmoid(x), 2 SiLU x sigmoid(x).
__device__ __forceinline__ float gate_act(float x, int act) {
    if (act == 0) return x;
    const float s = sigmoid_neg(-x);
    return act == 1 ? s : x * s;
}

struct HeadNormParams {
    const void* o;           // [total][heads][dim]
    const void* gate;        // [total] rows gate_stride apart, [heads][dim], or nullptr
    const float* weight;     // [dim]
    void* y;                 // [total][heads][dim]
    int64_t rows, gate_stride;
    int heads, dim, act;
    float eps;
};

constexpr int HEAD_NORM_THREADS = 256;

// y = w o / sqrt(mean o^2 + eps) * act(gate), a row a head.  A row is LPR
// lanes (a power of two) of eight channels each, so a warp takes 32 / LPR rows
// and the sum takes log2 LPR shuffles.
template <typename OT, typename T>
__global__ void __launch_bounds__(HEAD_NORM_THREADS) kda_head_norm_kernel(const HeadNormParams p, int lpr_log2) {
    cudaTriggerProgrammaticLaunchCompletion();
    const int lpr = 1 << lpr_log2, sub = threadIdx.x & (lpr - 1), c = sub * 8;
    const int64_t row = (int64_t)blockIdx.x * (HEAD_NORM_THREADS >> lpr_log2) + (threadIdx.x >> lpr_log2);
    const bool on = row < p.rows && c < p.dim;
    cudaGridDependencySynchronize();
    float x[8] = {}, gt[8] = {}, w[8] = {};
    if (on) {
        ld8(static_cast<const OT*>(p.o) + row * p.dim + c, x);
        if (p.gate != nullptr) {
            const int64_t tok = row / p.heads;
            ld8(static_cast<const T*>(p.gate) + tok * p.gate_stride + (row - tok * p.heads) * p.dim + c, gt);
        }
        const float4 a = __ldg(reinterpret_cast<const float4*>(p.weight + c)), b = __ldg(reinterpret_cast<const float4*>(p.weight + c) + 1);
        w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w; w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
    }
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) s = fmaf(x[e], x[e], s);
    for (int o = lpr >> 1; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (!on) return;
    const float r = rsqrtf(s / (float)p.dim + p.eps);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        x[e] = x[e] * r * w[e];
        if (p.gate != nullptr) x[e] *= gate_act(gt[e], p.act);
    }
    st8(static_cast<T*>(p.y) + row * p.dim + c, x);
}

struct BlockNormParams {
    const void* residual;    // [total][hidden]
    const void* y;           // [total] rows y_stride apart, or nullptr
    const void* gate;        // [total] rows gate_stride apart, or nullptr
    const float *w_post, *scale, *w_pre;   // [hidden] or nullptr
    void* residual_out;      // [total][hidden]
    void* x;                 // [total][hidden] or nullptr
    int64_t y_stride, gate_stride;
    int total, hidden, act;
    float eps, residual_scale, branch_scale;
};

// Sum over the CTA of one value a thread; every thread gets it.  `part` is
// one of two alternating [32] buffers: a single barrier a call.
__device__ __forceinline__ float block_sum(float x, float* part, int warps) {
    x = warp_sum(x);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = x;
    __syncthreads();
    float s = 0.f;
    for (int w = 0; w < warps; ++w) s += part[w];
    return s;
}

// h = a residual + b scale act(gate) [w_post y / rms(y)]; x = w_pre h / rms(h).
// A CTA a row at a time; a thread keeps NV vectors of VEC channels of the row
// in registers across both sums, so memory is touched once.
template <typename T, typename R, int VEC, int NV>
__global__ void __launch_bounds__(1024, NV > 8 ? 0 : 1) kda_block_norm_kernel(const BlockNormParams p) {
    __shared__ float part[2][32];
    const int nt = blockDim.x, warps = nt >> 5;
    cudaTriggerProgrammaticLaunchCompletion();
    cudaGridDependencySynchronize();
    const float inv = 1.f / (float)p.hidden;
    for (int row = blockIdx.x; row < p.total; row += gridDim.x) {
        const R* res = static_cast<const R*>(p.residual) + (int64_t)row * p.hidden;
        float h[NV][VEC], z[NV][VEC];
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * nt + (int)threadIdx.x) * VEC;
#pragma unroll
            for (int e = 0; e < VEC; ++e) h[i][e] = z[i][e] = 0.f;
            if (c < p.hidden) {
                if constexpr (VEC == 8) ld8(res + c, h[i]);
                if (p.y != nullptr) {
                    const T* y = static_cast<const T*>(p.y) + (int64_t)row * p.y_stride + c;
                    if constexpr (VEC == 8) ld8(y, z[i]);
                    else z[i][0] = to_f32(y[0]);
                }
            }
#pragma unroll
            for (int e = 0; e < VEC; ++e) s = fmaf(z[i][e], z[i][e], s);
        }
        float r = 1.f;
        if (p.w_post != nullptr) r = rsqrtf(block_sum(s, part[0], warps) * inv + p.eps);
        s = 0.f;
        if constexpr (VEC == 1) {  // late: with up to 16 channels a thread, both rows at once would not fit its registers
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = i * nt + (int)threadIdx.x;
                if (c < p.hidden) h[i][0] = to_f32(res[c]);
            }
        }
        if (p.y != nullptr) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (i * nt + (int)threadIdx.x) * VEC;
                if (c < p.hidden) {
                    float gt[VEC];
                    if (p.gate != nullptr) {
                        const T* g = static_cast<const T*>(p.gate) + (int64_t)row * p.gate_stride + c;
                        if constexpr (VEC == 8) ld8(g, gt);
                        else gt[0] = to_f32(g[0]);
                    }
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        float v = z[i][e] * r * p.branch_scale;
                        if (p.w_post != nullptr) v *= __ldg(p.w_post + c + e);
                        if (p.scale != nullptr) v *= __ldg(p.scale + c + e);
                        if (p.gate != nullptr) v *= gate_act(gt[e], p.act);
                        h[i][e] = fmaf(p.residual_scale, h[i][e], v);
                    }
                    R* out = static_cast<R*>(p.residual_out) + (int64_t)row * p.hidden + c;
                    if constexpr (VEC == 8) st8(out, h[i]);
                    else out[0] = from_f32<R>(h[i][0]);
                }
            }
        }
        if (p.x != nullptr) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int e = 0; e < VEC; ++e) s = fmaf(h[i][e], h[i][e], s);
            r = rsqrtf(block_sum(s, part[1], warps) * inv + p.eps);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (i * nt + (int)threadIdx.x) * VEC;
                if (c < p.hidden) {
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        h[i][e] *= r;
                        if (p.w_pre != nullptr) h[i][e] *= __ldg(p.w_pre + c + e);
                    }
                    T* out = static_cast<T*>(p.x) + (int64_t)row * p.hidden + c;
                    if constexpr (VEC == 8) st8(out, h[i]);
                    else out[0] = from_f32<T>(h[i][0]);
                }
            }
        }
        if ((p.w_post == nullptr) != (p.x == nullptr)) __syncthreads();  // one buffer only: the next row writes it again
    }
}

}  // namespace kda
