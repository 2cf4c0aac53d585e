// The norms around a block: the per-head norm and output gate behind the
// recurrence (kda_head_norm), and the norms, gate and scaled residual between
// two blocks (kda_block_norm).  Both read and write every element once; sums
// and products are fp32, each output is rounded once, to nearest even.
#pragma once

#include "kda_common.cuh"

namespace kda {

// Eight elements -> fp32 registers by 16-byte accesses.
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

// Eight elements as loaded: 16 bytes, or 32 of fp32.
template <typename T> struct Raw8 { uint4 v[sizeof(T) / 2]; };
template <typename T> __device__ __forceinline__ Raw8<T> raw8(const T* p) {
    Raw8<T> r;
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.v[i] = __ldcs(reinterpret_cast<const uint4*>(p) + i);
    return r;
}
template <typename T> __device__ __forceinline__ void widen8(const Raw8<T>& r, float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) {
        const uint32_t w[4] = {r.v[i].x, r.v[i].y, r.v[i].z, r.v[i].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if constexpr (sizeof(T) == 4) {
                x[4 * i + e] = __uint_as_float(w[e]);
            } else {
                float2 f;
                if constexpr (__is_same(T, __half)) f = __half22float2(*reinterpret_cast<const __half2*>(&w[e]));
                else f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[e]));
                x[2 * e] = f.x;
                x[2 * e + 1] = f.y;
            }
        }
    }
}

// h = a residual + b scale act(gate) [w_post y / rms(y)]; x = w_pre h / rms(h).
// Bound by memory: every element of a row is read and written once, the row
// stays in registers across both sums.  A CTA takes rows in turn, its threads
// NV vectors of eight channels each; the weights stay in registers for all its
// rows (reading them again for every row is half as many bytes again, from
// L2), and the next row is on its way while a row is summed up (but for two
// vectors of fp32, which fill the registers).
template <typename T, typename R, int NV>
__global__ void __launch_bounds__(512) kda_block_norm_kernel(const BlockNormParams p) {
    constexpr bool AHEAD = NV == 1 || sizeof(T) == 2;
    __shared__ float part[2][32];
    const int nt = blockDim.x, warps = nt >> 5;
    cudaTriggerProgrammaticLaunchCompletion();
    cudaGridDependencySynchronize();
    const float inv = 1.f / (float)p.hidden;
    bool on[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) on[i] = (i * nt + (int)threadIdx.x) * 8 < p.hidden;
    float wb[NV][8], wq[NV][8];      // weights of the branch, of the next block's input
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if (!on[i]) continue;
        const int c = (i * nt + (int)threadIdx.x) * 8;
        float f[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            wb[i][e] = p.branch_scale;
            wq[i][e] = 1.f;
        }
        if (p.w_post != nullptr) {
            widen8(raw8(p.w_post + c), f);
#pragma unroll
            for (int e = 0; e < 8; ++e) wb[i][e] *= f[e];
        }
        if (p.scale != nullptr) {
            widen8(raw8(p.scale + c), f);
#pragma unroll
            for (int e = 0; e < 8; ++e) wb[i][e] *= f[e];
        }
        if (p.w_pre != nullptr) widen8(raw8(p.w_pre + c), wq[i]);
    }
    Raw8<T> y[NV], gate[NV];
    Raw8<R> res[NV];
    auto load = [&](int row) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * nt + (int)threadIdx.x) * 8;
            if (!on[i]) continue;
            res[i] = raw8(static_cast<const R*>(p.residual) + (int64_t)row * p.hidden + c);
            if (p.y != nullptr) y[i] = raw8(static_cast<const T*>(p.y) + (int64_t)row * p.y_stride + c);
            if (p.gate != nullptr) gate[i] = raw8(static_cast<const T*>(p.gate) + (int64_t)row * p.gate_stride + c);
        }
    };
    int row = blockIdx.x;
    if (AHEAD && row < p.total) load(row);
    for (; row < p.total; row += gridDim.x) {
        if (!AHEAD) load(row);
        float z[NV][8], h[NV][8], s = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
#pragma unroll
            for (int e = 0; e < 8; ++e) z[i][e] = h[i][e] = 0.f;
            if (!on[i]) continue;
            widen8(res[i], h[i]);
            if (p.y != nullptr) {
                widen8(y[i], z[i]);
#pragma unroll
                for (int e = 0; e < 8; ++e) s = fmaf(z[i][e], z[i][e], s);
                if (p.gate != nullptr) {
                    float f[8];
                    widen8(gate[i], f);
#pragma unroll
                    for (int e = 0; e < 8; ++e) z[i][e] *= gate_act(f[e], p.act);
                }
            }
        }
        const int next = row + gridDim.x;
        if (AHEAD && next < p.total) load(next);
        float r = 1.f;
        if (p.w_post != nullptr) r = rsqrtf(block_sum(s, part[0], warps) * inv + p.eps);
        s = 0.f;
        if (p.y != nullptr) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (!on[i]) continue;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    h[i][e] = fmaf(p.residual_scale, h[i][e], z[i][e] * r * wb[i][e]);
                    s = fmaf(h[i][e], h[i][e], s);
                }
                st8(static_cast<R*>(p.residual_out) + (int64_t)row * p.hidden + (i * nt + (int)threadIdx.x) * 8, h[i]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int e = 0; e < 8; ++e) s = fmaf(h[i][e], h[i][e], s);
        }
        if (p.x != nullptr) {
            r = rsqrtf(block_sum(s, part[1], warps) * inv + p.eps);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (!on[i]) continue;
#pragma unroll
                for (int e = 0; e < 8; ++e) h[i][e] *= r * wq[i][e];
                st8(static_cast<T*>(p.x) + (int64_t)row * p.hidden + (i * nt + (int)threadIdx.x) * 8, h[i]);
            }
        }
        if ((p.w_post == nullptr) != (p.x == nullptr)) __syncthreads();  // one buffer only: the next row writes it again
    }
}

// The same for rows that do not start on 16 bytes, are no multiple of eight
// channels wide, or wider than 8192: one channel an access, NV of them a thread; the weights come
// from L1.  Row after row of an odd width is still contiguous, so a warp's
// loads are whole lines.
template <typename T, typename R, int NV>
__global__ void __launch_bounds__(1024, NV > 8 ? 0 : 1) kda_block_norm_any_kernel(const BlockNormParams p) {
    __shared__ float part[2][32];
    const int nt = blockDim.x, warps = nt >> 5;
    cudaTriggerProgrammaticLaunchCompletion();
    cudaGridDependencySynchronize();
    const float inv = 1.f / (float)p.hidden;
    const int row = blockIdx.x;
    float h[NV], s = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = i * nt + (int)threadIdx.x;
        h[i] = c < p.hidden && p.y != nullptr ? to_f32(static_cast<const T*>(p.y)[(int64_t)row * p.y_stride + c]) : 0.f;
        s = fmaf(h[i], h[i], s);
    }
    float r = 1.f;
    if (p.w_post != nullptr) r = rsqrtf(block_sum(s, part[0], warps) * inv + p.eps);
    s = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = i * nt + (int)threadIdx.x;
        if (c >= p.hidden) continue;
        const float old = to_f32(static_cast<const R*>(p.residual)[(int64_t)row * p.hidden + c]);
        if (p.y != nullptr) {
            float w = p.branch_scale;
            if (p.w_post != nullptr) w *= __ldg(p.w_post + c);
            if (p.scale != nullptr) w *= __ldg(p.scale + c);
            if (p.gate != nullptr) h[i] *= gate_act(to_f32(static_cast<const T*>(p.gate)[(int64_t)row * p.gate_stride + c]), p.act);
            h[i] = fmaf(p.residual_scale, old, h[i] * r * w);
            static_cast<R*>(p.residual_out)[(int64_t)row * p.hidden + c] = from_f32<R>(h[i]);
        } else {
            h[i] = old;
        }
        s = fmaf(h[i], h[i], s);
    }
    if (p.x == nullptr) return;
    r = rsqrtf(block_sum(s, part[1], warps) * inv + p.eps);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = i * nt + (int)threadIdx.x;
        if (c >= p.hidden) continue;
        const float w = p.w_pre != nullptr ? __ldg(p.w_pre + c) : 1.f;
        static_cast<T*>(p.x)[(int64_t)row * p.hidden + c] = from_f32<T>(h[i] * r * w);
    }
}

}  // namespace kda
