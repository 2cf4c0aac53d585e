// The norms around a block: the per-head norm and output gate behind the
// recurrence (kda_head_norm), and the norms, gate and scaled residual between
// two blocks (kda_block_norm).  Both read and write every element once; sums
// and products are fp32, each output is rounded once, to nearest even.
#pragma once

#include <type_traits>

#include "kda_common.cuh"

namespace kda {

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

// sigmoid(x) = 1 / (1 + e^-x).  FINE (an fp32 gate): with t = e^-|x| it is
// 1 / (1 + t) or t / (1 + t), so that nothing overflows and a far negative gate
// goes to 0 through the subnormal numbers; expf and the hardware's approximate
// reciprocal refined by one Newton step as in sigmoid_neg.  Otherwise (a 16-bit
// gate, whose own rounding is 2^-12 or more of it) four instructions.  Their
// relative error is within (1.25 |x| + 7) 2^-24 while the result is a normal
// fp32 number, x >= -87: the rounding of the exponent's product with log2(e) and
// of that constant (1.23 |x| together), the exponential (4), its sum with 1 (1)
// and the reciprocal (2); below it is 0.  Instructions bound the head norm: with
// FINE everywhere 8192 x 12 x 128 took 20.2 us.  A NaN passes through both.
template <bool FINE> __device__ __forceinline__ float sigmoid_f(float x) {
    float r;
    if constexpr (FINE) {
        const float t = expf(-fabsf(x)), y = 1.f + t;
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(y));
        r = fmaf(r, fmaf(-y, r, 1.f), r);
        return x < 0.f ? t * r : r;
    } else {
        float e;
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x * -1.44269504f));
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
        return r;
    }
}

// x[i] *= the gate's factor: 0 the gate itself, 1 sigmoid(g), 2 SiLU g sigmoid(g).
template <typename T, int N> __device__ __forceinline__ void apply_gate(float (&x)[N], const float (&g)[N], int act) {
    if (act == 0) {
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] *= g[i];
        return;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] *= sigmoid_f<sizeof(T) == 4>(g[i]);
    if (act == 2) {
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] *= g[i];
    }
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

// y = w o / sqrt(mean o^2 + eps) * act(gate), a row a head.  A row is LPR lanes (a
// power of two) of eight channels each, so a warp takes 32 / LPR rows and the
// sum takes log2 LPR shuffles.  8192 x 12 x 128, fp32 in, bf16 gate and out: 17.0
// us, 0.87 of the measured copy bandwidth.  Two rows a thread (more loads on
// their way) were no faster: 19.2 against 18.7 us at the time.
template <typename OT, typename T>
__global__ void __launch_bounds__(HEAD_NORM_THREADS) kda_head_norm_kernel(const HeadNormParams p, int lpr_log2) {
    cudaTriggerProgrammaticLaunchCompletion();
    const int lpr = 1 << lpr_log2, c = (threadIdx.x & (lpr - 1)) * 8;
    const int64_t row = (int64_t)blockIdx.x * (HEAD_NORM_THREADS >> lpr_log2) + (threadIdx.x >> lpr_log2);
    const bool on = row < p.rows && c < p.dim;
    cudaGridDependencySynchronize();
    Raw8<OT> o;
    Raw8<T> gate;
    float w[8] = {}, x[8] = {}, s = 0.f;
    if (on) {
        o = raw8(static_cast<const OT*>(p.o) + row * p.dim + c);
        if (p.gate != nullptr) {
            int64_t at = row * p.dim;
            if (p.gate_stride != (int64_t)p.heads * p.dim) {   // tokens apart; the host keeps rows below 2^31
                const unsigned tok = (unsigned)row / (unsigned)p.heads;
                at = tok * p.gate_stride + ((unsigned)row - tok * (unsigned)p.heads) * p.dim;
            }
            gate = raw8(static_cast<const T*>(p.gate) + at + c);
        }
        const float4 a = __ldg(reinterpret_cast<const float4*>(p.weight + c)), b = __ldg(reinterpret_cast<const float4*>(p.weight + c) + 1);
        w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w; w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
        widen8(o, x);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) s = fmaf(x[e], x[e], s);
    for (int i = lpr >> 1; i > 0; i >>= 1) s += __shfl_xor_sync(0xffffffffu, s, i);
    if (!on) return;
    const float r = rsqrtf(s / (float)p.dim + p.eps);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = x[e] * r * w[e];
    if (p.gate != nullptr) {
        float f[8];
        widen8(gate, f);
        apply_gate<T>(x, f, p.act);
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
    const int lane = threadIdx.x & 31;
    return warp_sum(lane < warps ? part[lane] : 0.f);
}

// 16 bytes to shared memory; with `bytes` below 16 only so many are read, the rest is zero.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Rows in shared memory at a time, each its residual, y and gate.  Two: three took
// 86.5 us against 83 for 8192 x 4096 (two CTAs an SM by registers either way) and
// 11.2 against 10.7 for 1021 x 2049 of fp32 (two CTAs an SM instead of three).
constexpr int BLOCK_NORM_STAGES = 2;
template <typename T, typename R> constexpr size_t block_norm_smem(int threads) {
    return (size_t)BLOCK_NORM_STAGES * (8 * sizeof(R) + 16 * sizeof(T)) * threads;
}

// h = a residual + b scale act(gate) [w_post y / rms(y)]; x = w_pre h / rms(h).
// Bound by memory: every element of a row is read and written once, the row
// stays in registers across both sums.  A CTA takes rows in turn, eight channels
// a thread (with two vectors a thread the registers leave half as many warps:
// 2000 x 5001 33 against 30 us); the weights stay in registers for all its rows
// (reading them again for every row is half as many bytes again, from L2).  The
// next row is on its way to shared memory meanwhile: a thread copies and reads
// only its own places, so the copies need no barrier.  8192 x 4096, bf16 with an
// fp32 residual: 83 us, 0.83 of the measured copy bandwidth.
//
// SHIFT: a width that is no multiple of eight.  Vectors then lie on multiples
// of eight in the buffer, not in the row: a row's first one begins up to seven
// channels before it.  The grid is a multiple of eight (or holds every row), so
// a CTA's rows all begin at the same place in a vector and the weights still
// stay in registers; a row's two end vectors are masked, their stores are
// single.  4096 x 1537: 21.5 us, 1536 wide 17.4.
template <typename T, typename R, bool SHIFT>
__global__ void __launch_bounds__(1024) kda_block_norm_kernel(const BlockNormParams p) {
    constexpr int CR = (int)sizeof(R) / 2, CT = (int)sizeof(T) / 2, CH = CR + 2 * CT;   // 16-byte chunks of a vector
    constexpr int STAGES = BLOCK_NORM_STAGES;
    extern __shared__ __align__(16) uint4 norm_ring[];
    __shared__ float part[2][32];
    const int nt = blockDim.x, warps = nt >> 5;
    cudaTriggerProgrammaticLaunchCompletion();
    cudaGridDependencySynchronize();
    const float inv = 1.f / (float)p.hidden;
    const int shift = SHIFT ? (int)((int64_t)blockIdx.x * p.hidden & 7) : 0;
    const int c = (int)threadIdx.x * 8 - shift;      // this thread's channels
    const bool on = c < p.hidden, whole = !SHIFT || (c >= 0 && c + 8 <= p.hidden);
    auto at = [&](int stage, int k) { return norm_ring + (stage * CH + k) * nt + threadIdx.x; };
    // one vector of a buffer whose rows are `stride` apart; nothing behind its last row's end is read
    auto copy = [&](auto* base, int64_t stride, unsigned row, int stage, int k0) {
        using E = std::remove_const_t<std::remove_pointer_t<decltype(base)>>;
        const int64_t from = (int64_t)row * stride + c;
        constexpr int W = 16 / (int)sizeof(E);
#pragma unroll
        for (int k = 0; k < (int)sizeof(E) / 2; ++k) {
            int bytes = 16;
            if constexpr (SHIFT) {
                const int64_t left = ((int64_t)(p.total - 1) * stride + p.hidden - from - k * W) * (int)sizeof(E);
                bytes = left < 0 ? 0 : left < 16 ? (int)left : 16;
            }
            cp_async16(smem_u32(at(stage, k0 + k)), bytes > 0 ? base + from + k * W : base, bytes);
        }
    };
    auto fetch = [&](unsigned row, int stage) {
        if (row < (unsigned)p.total && on) {
            copy(static_cast<const R*>(p.residual), p.hidden, row, stage, 0);
            if (p.y != nullptr) copy(static_cast<const T*>(p.y), p.y_stride, row, stage, CR);
            if (p.gate != nullptr) copy(static_cast<const T*>(p.gate), p.gate_stride, row, stage, CR + CT);
        }
        cp_async_commit();
    };
    auto store = [&](auto* row, const float (&v)[8]) {
        using E = std::remove_pointer_t<decltype(row)>;
        if (whole) {
            st8(row + c, v);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (c + e >= 0 && c + e < p.hidden) row[c + e] = from_f32<E>(v[e]);
        }
    };
#pragma unroll
    for (int k = 0; k < STAGES - 1; ++k) fetch(blockIdx.x + k * gridDim.x, k);

    float wb[8], wq[8];      // weights of the branch, of the next block's input
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        wb[e] = p.branch_scale;
        wq[e] = 1.f;
    }
    if (on) {
        auto weights = [&](const float* w, float (&f)[8]) {
            if constexpr (SHIFT) {
#pragma unroll
                for (int e = 0; e < 8; ++e) f[e] = c + e >= 0 && c + e < p.hidden ? __ldg(w + c + e) : 0.f;
            } else {
                widen8(raw8(w + c), f);
            }
        };
        float f[8];
        if (p.w_post != nullptr) {
            weights(p.w_post, f);
#pragma unroll
            for (int e = 0; e < 8; ++e) wb[e] *= f[e];
        }
        if (p.scale != nullptr) {
            weights(p.scale, f);
#pragma unroll
            for (int e = 0; e < 8; ++e) wb[e] *= f[e];
        }
        if (p.w_pre != nullptr) weights(p.w_pre, wq);
    }
    int stage = 0;
    // unsigned: behind the last of up to 2^31 - 1 rows a grid more must not wrap
    for (unsigned row = blockIdx.x; row < (unsigned)p.total; row += gridDim.x) {
        cp_async_wait<STAGES - 2>();
        float h[8] = {}, z[8] = {}, s = 0.f;
        if (on) {
            Raw8<R> res;
#pragma unroll
            for (int k = 0; k < CR; ++k) res.v[k] = *at(stage, k);
            widen8(res, h);
            float f[8];
            if (p.y != nullptr) {
                Raw8<T> raw;
#pragma unroll
                for (int k = 0; k < CT; ++k) raw.v[k] = *at(stage, CR + k);
                widen8(raw, z);
                if (p.gate != nullptr) {
#pragma unroll
                    for (int k = 0; k < CT; ++k) raw.v[k] = *at(stage, CR + CT + k);
                    widen8(raw, f);
                }
            }
            if (SHIFT && !whole) {       // neighbours' channels
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (c + e < 0 || c + e >= p.hidden) h[e] = z[e] = f[e] = 0.f;
            }
            if (p.y != nullptr) {
#pragma unroll
                for (int e = 0; e < 8; ++e) s = fmaf(z[e], z[e], s);
                if (p.gate != nullptr) apply_gate<T>(z, f, p.act);
            }
        }
        // the stage before this one is free: this thread read it in the last turn
        const int free = stage == 0 ? STAGES - 1 : stage - 1;
        stage = stage == STAGES - 1 ? 0 : stage + 1;
        fetch(row + (STAGES - 1) * gridDim.x, free);
        float r = 1.f;
        if (p.w_post != nullptr) r = rsqrtf(block_sum(s, part[0], warps) * inv + p.eps);
        s = 0.f;
        if (p.y != nullptr && on) {
#pragma unroll
            for (int e = 0; e < 8; ++e) h[e] = fmaf(p.residual_scale, h[e], z[e] * r * wb[e]);
            store(static_cast<R*>(p.residual_out) + (int64_t)row * p.hidden, h);
        }
        if (p.x != nullptr) {
#pragma unroll
            for (int e = 0; e < 8; ++e) s = fmaf(h[e], h[e], s);
            r = rsqrtf(block_sum(s, part[1], warps) * inv + p.eps);
            if (on) {
#pragma unroll
                for (int e = 0; e < 8; ++e) h[e] *= r * wq[e];
                store(static_cast<T*>(p.x) + (int64_t)row * p.hidden, h);
            }
        }
        if ((p.w_post == nullptr) != (p.x == nullptr)) __syncthreads();  // one buffer only: the next row writes it again
    }
    cp_async_wait<0>();
}

// The same for buffers that do not start on 16 bytes, strides that are no
// multiple of eight apart from the width, and rows wider than 8192 (odd widths:
// 8178): one channel an access, NV of them a thread; the weights come from L1.
// Row after row of an odd width is still contiguous, so a warp's loads are
// whole lines.
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
            if (p.gate != nullptr) {
                float v[1] = {h[i]};
                const float f[1] = {to_f32(static_cast<const T*>(p.gate)[(int64_t)row * p.gate_stride + c])};
                apply_gate<T>(v, f, p.act);
                h[i] = v[0];
            }
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
