// The paged key/value cache in 4-bit blocks of the attention layers that stand
// between KDA layers: appending (rotation and rounding on the way) and the
// attention of a decode or speculative step over it.
//
// Format.  A value is code * scale * (the cache's k_scale or v_scale): codes
// are e2m1 (0, .5, 1, 1.5, 2, 3, 4, 6 with a sign), one e4m3 scale serves 16
// neighbouring channels of a token's head.  Sixteen tokens of one head make a
// block of 18 D bytes, contiguous, which one bulk copy moves:
//   [0, 8 D)       key codes, [token][D / 2], two channels a byte (low nibble first)
//   [8 D, 16 D)    value codes in the order a warp's mma fragments take them
//   [16 D, 17 D)   key scales, [token][D / 16]
//   [17 D, 18 D)   value scales, fragment order
// Value order: lane (g, t) of a warp (g = lane / 4, t = lane % 4) multiplies
// tokens 2t, 2t + 1, 2t + 8, 2t + 9 by channels g D / 8 .. (g + 1) D / 8 - 1,
// so its D / 16 code bytes of token 2t and of token 2t + 1 are neighbours, and
// the four lanes of a g follow each other: every read is one 16-byte (D = 128)
// word a lane, in lane order.
#pragma once

#include <cfloat>

#include "kda_common.cuh"
#include "kda_tree.cuh"

namespace kda {

template <int D> struct Kv4 {
    static constexpr int CB = D / 16;        // code bytes of a token in one lane's channels; also scale groups
    static constexpr int NG = D / 16;        // 16-channel groups
    static constexpr int KC = 0, VC = 8 * D, KS = 16 * D, VS = 17 * D;
    static constexpr int BLOCK = 18 * D;     // bytes of a block
};

// Places inside a block of token `w` (0..15).
template <int D> __device__ __forceinline__ int kv4_v_code(int w, int g) {
    return Kv4<D>::VC + (w >> 3) * (64 * Kv4<D>::CB) + (g * 4 + ((w & 7) >> 1)) * (2 * Kv4<D>::CB) + (w & 1) * Kv4<D>::CB;
}
template <int D> __device__ __forceinline__ int kv4_v_scale(int w, int grp) {
    return Kv4<D>::VS + (grp * 4 + ((w & 7) >> 1)) * 4 + (w >> 3) * 2 + (w & 1);
}

// Typed buffers are kda_dtype codes: 0 fp32, 1 fp16, 2 bf16.
// N (1, 2 or 4) neighbouring elements from a multiple of N of a 16-byte aligned buffer.
template <int N, int M> __device__ __forceinline__ void ld_elems(const void* p, int64_t i, int dtype, float (&x)[M]) {
    static_assert(N <= M && (N == 1 || N == 2 || N == 4), "elements");
    if (dtype == 0) {
        const float* f = static_cast<const float*>(p) + i;
        if constexpr (N == 4) {
            const float4 v = __ldg(reinterpret_cast<const float4*>(f));
            x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
        } else if constexpr (N == 2) {
            const float2 v = __ldg(reinterpret_cast<const float2*>(f));
            x[0] = v.x; x[1] = v.y;
        } else {
            x[0] = __ldg(f);
        }
        return;
    }
    const uint16_t* h = static_cast<const uint16_t*>(p) + i;
    uint32_t w[2];
    if constexpr (N == 4) {
        const uint2 v = __ldg(reinterpret_cast<const uint2*>(h));
        w[0] = v.x; w[1] = v.y;
    } else if constexpr (N == 2) {
        w[0] = __ldg(reinterpret_cast<const uint32_t*>(h));
    } else {
        w[0] = __ldg(h);
    }
#pragma unroll
    for (int k = 0; k < (N + 1) / 2; ++k) {
        const float2 f = dtype == 1 ? __half22float2(*reinterpret_cast<const __half2*>(&w[k]))
                                    : __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[k]));
        x[2 * k] = f.x;
        if constexpr (N > 1) x[2 * k + 1] = f.y;
    }
}

// Four elements to a typed buffer, rounded to nearest even; i a multiple of 4
// of a 16-byte aligned buffer.
__device__ __forceinline__ void st_elem4(void* p, int64_t i, int dtype, float a, float b, float c, float d) {
    if (dtype == 0) {
        *reinterpret_cast<float4*>(static_cast<float*>(p) + i) = make_float4(a, b, c, d);
    } else if (dtype == 1) {
        const __half2 x = __floats2half2_rn(a, b), y = __floats2half2_rn(c, d);
        *reinterpret_cast<uint2*>(static_cast<__half*>(p) + i) =
            make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
    } else {
        const __nv_bfloat162 x = __floats2bfloat162_rn(a, b), y = __floats2bfloat162_rn(c, d);
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p) + i) =
            make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
    }
}

// PTX conversions of the 4- and 8-bit types (two values an instruction).
__device__ __forceinline__ uint32_t cvt_e4m3x2_f16x2(uint32_t two) {
    uint32_t r;
    asm("{\n\t.reg .b16 h;\n\tcvt.u16.u32 h, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(r) : "r"(two));
    return r;
}
__device__ __forceinline__ uint32_t cvt_f32_e4m3(float x) {  // to nearest even, at most 448
    uint32_t r;
    asm("{\n\t.reg .b16 h;\n\tcvt.rn.satfinite.e4m3x2.f32 h, %2, %1;\n\tcvt.u32.u16 %0, h;\n\t}"
        : "=r"(r) : "f"(x), "f"(0.f));
    return r & 0xffu;
}
// Eight e2m1 codes from eight floats, the first in the lowest nibble.
__device__ __forceinline__ uint32_t cvt_f32x8_e2m1(const float* y) {
    uint32_t r;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(r) : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7]));
    return r;
}
// The four bytes of a word, two codes each, as f16 pairs.
__device__ __forceinline__ void cvt_e2m1x8_f16(uint32_t w, uint32_t (&r)[4]) {
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(w));
}
__device__ __forceinline__ uint32_t hmul2_u32(uint32_t a, uint32_t b) {
    const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
}
// Both halves of a times the low or the high half of s.
template <bool HIGH> __device__ __forceinline__ uint32_t hmul2_half(uint32_t a, uint32_t s) {
    const __half2 h = *reinterpret_cast<const __half2*>(&s);
    const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), HIGH ? __high2half2(h) : __low2half2(h));
    return *reinterpret_cast<const uint32_t*>(&r);
}
// Transposes an 8 x 8 matrix of 16-bit elements held two a lane (row lane / 4,
// columns 2 (lane % 4) ..).
__device__ __forceinline__ uint32_t movmatrix_t(uint32_t x) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}
// threadIdx.x read again, where a value kept across the main loop would cost a register.
__device__ __forceinline__ int tid_again() {
    int t;
    asm volatile("mov.u32 %0, %%tid.x;" : "=r"(t));
    return t;
}
// As mma_16816_f16, free to be scheduled among its neighbours.
__device__ __forceinline__ void kv4_mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The largest of three; NaN if one is.
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ float ex2f(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// ---------------------------------------------------------------------------
// Append
// ---------------------------------------------------------------------------
struct Kv4AppendParams {
    uint8_t* pages;
    int64_t num_pages, page_stride;      // bytes
    int page_tokens, heads;
    int n, total, max_t, dtype, cols, rot, inter, rope_rows;
    int64_t k_stride, v_stride;          // elements between tokens
    const int32_t *cu, *table, *ctx;
    const void *k, *v;
    const float *cos, *sin;
    void *k_out, *v_out;
    int out_dtype;
    float inv_k, inv_v, k_scale, v_scale;
    int32_t* status;
    const uint64_t* tree;                // [total] masks (TREE)
};

constexpr int KV4_APPEND_THREADS = 128, KV4_APPEND_WARPS = KV4_APPEND_THREADS / 32;
// The heads of eight tokens are shared out over several CTAs while the grid stays below 16 CTAs for each of
// 152 SMs.  8 x 1024 tokens of 8 heads of 128: 22.8 us with half as many, 20.5 with these, 20.9 with twice;
// the same of fp32 26.5, 26.6, 27.5; 64 x 8 tokens and fewer 4 us with any.
constexpr int KV4_APPEND_CTAS = 16 * 152;

// Sixteen elements of 2 or 4 bytes as loaded (the host checks the alignment of
// base and stride), and widened to fp32.
template <int ES> struct Raw16 { uint4 v[ES]; };
template <int ES> __device__ __forceinline__ Raw16<ES> raw16(const void* p, int64_t i) {
    Raw16<ES> r;
    const uint4* q = reinterpret_cast<const uint4*>(static_cast<const char*>(p) + i * ES);
#pragma unroll
    for (int j = 0; j < ES; ++j) r.v[j] = __ldg(q + j);
    return r;
}
template <int ES> __device__ __forceinline__ void widen16(const Raw16<ES>& r, int dtype, float (&x)[16]) {
#pragma unroll
    for (int j = 0; j < ES; ++j) {
        const uint32_t w[4] = {r.v[j].x, r.v[j].y, r.v[j].z, r.v[j].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if constexpr (ES == 4) {
                x[4 * j + e] = __uint_as_float(w[e]);
            } else {
                const float2 f = dtype == 1 ? __half22float2(*reinterpret_cast<const __half2*>(&w[e]))
                                            : __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[e]));
                x[8 * j + 2 * e] = f.x;
                x[8 * j + 2 * e + 1] = f.y;
            }
        }
    }
}

// Rounds a group of 16 channels: the two words of codes and the scale byte.  In fp32
//   t = x / scale of the cache (as a product with the reciprocal, 1 by default),
//   s = e4m3(max|t| / 6), code = e2m1(t / s), each rounded to nearest even.
// The quotients are those of IEEE division, so that a value half way between
// two codes stays half way: the product with a reciprocal, corrected once by
// its exact remainder (Markstein, IBM Journal of Research and Development 34,
// 1990).  A reciprocal right to 2^-22 leaves the corrected quotient within 2^-44
// of the true one, and a quotient by 6 or by a scale (four bits) that is no
// float lies 2^-28 or more from the middle of two floats, so it rounds alike;
// where the remainder may underflow the code is 0 either way.  A group that
// holds a NaN or an infinity gets a NaN scale: it reads back as NaN.
__device__ __forceinline__ uint32_t kv4_round(float* x, float inv, uint2& code) {
    if (inv != 1.f) {
#pragma unroll
        for (int j = 0; j < 16; ++j) x[j] = __fmul_rn(x[j], inv);
    }
    float amax = 0.f;
#pragma unroll
    for (int j = 0; j < 16; j += 2) amax = max3_nan(amax, fabsf(x[j]), fabsf(x[j + 1]));
    constexpr float sixth = 1.f / 6.f;
    const bool fine = amax <= FLT_MAX;
    const uint32_t s8 = fine ? cvt_f32_e4m3(fmaf(-fmaf(amax * sixth, 6.f, -amax), sixth, amax * sixth)) : 0x7fu;
    const uint32_t sh = cvt_e4m3x2_f16x2(s8);
    const float s = __low2float(*reinterpret_cast<const __half2*>(&sh));
    float rs;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(rs) : "f"(s));
    if (!(s > 0.f)) rs = 0.f;
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        // as fma(q, s, -x) and minus its product, so that the sign of a zero stays
        const float q = x[j] * rs;
        x[j] = fmaf(-fmaf(q, s, -x[j]), rs, q);
    }
    code = fine ? make_uint2(cvt_f32x8_e2m1(x), cvt_f32x8_e2m1(x + 8)) : make_uint2(0u, 0u);
    return s8;
}

// The 16 values that codes and a scale byte stand for, times g, to a typed
// buffer at element i.  code * scale has six significant bits: whole in fp16.
__device__ __forceinline__ void kv4_values(void* out, int64_t i, int dtype, uint2 code, uint32_t s8, float g) {
    uint32_t q[8];
    cvt_e2m1x8_f16(code.x, *reinterpret_cast<uint32_t(*)[4]>(q));
    cvt_e2m1x8_f16(code.y, *reinterpret_cast<uint32_t(*)[4]>(q + 4));
    const uint32_t sh = cvt_e4m3x2_f16x2(s8), s2 = __byte_perm(sh, sh, 0x1010);
#pragma unroll
    for (int j = 0; j < 8; ++j) q[j] = hmul2_u32(q[j], s2);
    if (dtype == 1 && g == 1.f) {
        uint4* o = reinterpret_cast<uint4*>(static_cast<__half*>(out) + i);
        o[0] = make_uint4(q[0], q[1], q[2], q[3]);
        o[1] = make_uint4(q[4], q[5], q[6], q[7]);
        return;
    }
    float x[16];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&q[j]));
        x[2 * j] = f.x;
        x[2 * j + 1] = f.y;
    }
    if (g != 1.f) {
#pragma unroll
        for (int j = 0; j < 16; ++j) x[j] *= g;
    }
    if (dtype == 2) {
        uint4* o = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(out) + i);
        uint32_t w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * j], x[2 * j + 1]);
            w[j] = *reinterpret_cast<const uint32_t*>(&h);
        }
        o[0] = make_uint4(w[0], w[1], w[2], w[3]);
        o[1] = make_uint4(w[4], w[5], w[6], w[7]);
        return;
    }
#pragma unroll
    for (int j = 0; j < 16; j += 4) st_elem4(out, i + j, dtype, x[j], x[j + 1], x[j + 2], x[j + 3]);
}

__device__ __forceinline__ void kv4_turn(float& a, float& b, float c, float s) {
    const float u = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
    b = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
    a = u;
}

// Eight tokens a CTA, a whole head of each a warp at a time (two heads of 64
// channels).  A lane rounds two groups of 16 channels: of keys those that the
// rotation pairs, so that every key and every table entry is loaded once.  A
// warp's loads are whole 128-byte lines of a token (16-bit inputs), its key
// codes whole 32-byte sectors, and its value codes 64 contiguous bytes when
// the eight tokens fill half a block.  The loads of a head do not wait for the
// token's place: they are on their way while that is looked up.  Rotation in
// fp32, products and sums rounded one by one (no fused multiply-add).  8192
// tokens of 8 heads of 128, bf16: 20.4 us, 3.8 TB/s.  Bound by latency: 16 warps
// an SM (registers) wait for the look-up and for every head after a warp's
// first, whose loads are not ahead; half of the issue slots go to the about 20
// instructions an element.  TREE: a token's key is rotated as at its depth in
// the request's tree of drafted tokens, and stored at its place in the request.
template <int D, int ES, bool TREE = false>
__global__ void __launch_bounds__(KV4_APPEND_THREADS, ES == 2 ? 5 : 4) kda_kv4_append_kernel(const Kv4AppendParams p) {
    constexpr int NG = Kv4<D>::NG, NP = NG / 2, HW = 4 / NP;     // groups and pairs of a head, heads of a warp
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    cudaTriggerProgrammaticLaunchCompletion();
    cudaGridDependencySynchronize();
    const int tok = (int)blockIdx.x * 8 + (lane >> 2);
    // this lane's two groups: those of a rotated pair of halves, else neighbours
    const int i = (lane & 3) % NP, half = p.rot >> 1, rg = p.rot >> 4;
    const bool halves = !p.inter && 2 * i < rg;
    const int grp[2] = {halves ? i : 2 * i, halves ? i + (rg >> 1) : 2 * i + 1};
    const int items = (p.heads + HW - 1) / HW * 2, step = KV4_APPEND_WARPS * (int)gridDim.y;   // heads of k and of v in turn
    int it = (int)blockIdx.y * KV4_APPEND_WARPS + warp;
    Raw16<ES> raw[2];
    auto load = [&](int at) {
        const int h = (at >> 1) * HW + (lane & 3) / NP;
        if (at >= items || h >= p.heads || tok >= p.total) return;
        const int64_t base = (int64_t)tok * (at & 1 ? p.v_stride : p.k_stride) + h * D;
#pragma unroll
        for (int k = 0; k < 2; ++k) raw[k] = raw16<ES>(at & 1 ? p.v : p.k, base + grp[k] * 16);
    };
    load(it);
    // the request that owns the token: the number of requests that end at or before it, counted
    // for the CTA's first token and from there on
    int r = 0;
    if (p.cu == nullptr) {
        r = tok / p.max_t;
    } else {
        const int tok8 = (int)blockIdx.x * 8;
        for (int b = 0; b < p.n; b += 32) {
            const int32_t end = b + lane < p.n ? __ldg(p.cu + b + lane + 1) : 0x7fffffff;
            r += __popc(__ballot_sync(0xffffffffu, end <= tok8));
        }
        while (r < p.n && tok < p.total && __ldg(p.cu + r + 1) <= tok) ++r;
    }
    int pos = -1, turn = 0;   // the token's position, and the one that its key is rotated by
    uint8_t* blk = nullptr;   // the token's block of head 0
    int where = 0;
    if (tok >= p.total) {
        return;
    } else if (r < p.n) {
        const int tok0 = p.cu ? __ldg(p.cu + r) : r * p.max_t;
        const int t = (p.cu ? __ldg(p.cu + r + 1) : tok0 + p.max_t) - tok0;
        const int64_t at = (int64_t)__ldg(p.ctx + r) + (tok - tok0);
        if (tok0 < 0 || tok < tok0 || t > p.max_t || (TREE && at - (tok - tok0) < 0 && at - (tok - tok0) + t > 0) ||
            (at >= 0 && (at >= (int64_t)p.cols * p.page_tokens || (p.rot && at >= p.rope_rows)))) {
            atomicCAS(p.status, 0, STATUS_ARG);
        } else if (at >= 0) {
            const int pg = (int)at / p.page_tokens, in = (int)at - pg * p.page_tokens;
            const int32_t id = __ldg(p.table + (int64_t)r * p.cols + pg);
            if (id < 0 || id >= p.num_pages) {
                atomicCAS(p.status, 0, STATUS_SLOT_RANGE);
            } else {
                pos = turn = (int)at;
                if constexpr (TREE) turn = pos - (tok - tok0) + __popcll(tree_mask(p.tree, tok, tok - tok0)) - 1;
                where = in & 15;
                blk = p.pages + (int64_t)id * p.page_stride + (int64_t)(in >> 4) * Kv4<D>::BLOCK;
            }
        }
    } else {
        atomicCAS(p.status, 0, STATUS_ARG);
    }
    const int64_t head_bytes = (int64_t)(p.page_tokens >> 4) * Kv4<D>::BLOCK;
    bool late = false;
    for (; it < items; it += step) {
        if (late) load(it);
        late = true;
        const bool is_v = (it & 1) != 0;
        const int h = (it >> 1) * HW + (lane & 3) / NP;
        float x[2][16];
#pragma unroll
        for (int k = 0; k < 2; ++k) widen16<ES>(raw[k], p.dtype, x[k]);
        if (h >= p.heads) continue;
        void* out = is_v ? p.v_out : p.k_out;
        const int64_t row = ((int64_t)tok * p.heads + h) * D;
        if (pos < 0) {
            if (out != nullptr)
#pragma unroll
                for (int k = 0; k < 2; ++k)
#pragma unroll
                    for (int j = 0; j < 16; j += 4) st_elem4(out, row + grp[k] * 16 + j, p.out_dtype, 0.f, 0.f, 0.f, 0.f);
            continue;
        }
        if (!is_v && 2 * i < rg) {
            const float* cs = p.cos + (int64_t)turn * half;
            const float* sn = p.sin + (int64_t)turn * half;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                float c[4], s[4];
                const int e0 = 16 * i + 4 * q;      // table entries of the pair's 16 angles
                ld_elems<4>(cs, e0, 0, c);
                ld_elems<4>(sn, e0, 0, s);
                if (!p.inter) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) kv4_turn(x[0][4 * q + j], x[1][4 * q + j], c[j], s[j]);
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j) kv4_turn(x[q >> 1][8 * (q & 1) + 2 * j], x[q >> 1][8 * (q & 1) + 2 * j + 1], c[j], s[j]);
                }
            }
        }
        uint8_t* b = blk + h * head_bytes;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            uint2 c;
            const uint32_t s8 = kv4_round(x[k], is_v ? p.inv_v : p.inv_k, c);
            if (!is_v) {
                *reinterpret_cast<uint2*>(b + Kv4<D>::KC + where * (D / 2) + grp[k] * 8) = c;
                b[Kv4<D>::KS + where * NG + grp[k]] = (uint8_t)s8;
            } else {
                if constexpr (D == 128) {
                    *reinterpret_cast<uint2*>(b + kv4_v_code<D>(where, grp[k])) = c;
                } else {
                    *reinterpret_cast<uint32_t*>(b + kv4_v_code<D>(where, 2 * grp[k])) = c.x;
                    *reinterpret_cast<uint32_t*>(b + kv4_v_code<D>(where, 2 * grp[k] + 1)) = c.y;
                }
                b[kv4_v_scale<D>(where, grp[k])] = (uint8_t)s8;
            }
            if (out != nullptr) kv4_values(out, row + grp[k] * 16, p.out_dtype, c, s8, is_v ? p.v_scale : p.k_scale);
        }
    }
}

// ---------------------------------------------------------------------------
// Attend
// ---------------------------------------------------------------------------
struct Kv4AttendParams {
    const uint8_t* pages;
    int64_t num_pages, page_stride;      // bytes
    int page_tokens, heads;
    int n, total, max_t, dtype, cols, rot, inter, rope_rows, h_q, grp, window;
    int64_t q_stride;                    // elements between tokens
    const int32_t *cu, *table, *ctx;
    const void* q;
    const float *cos, *sin;
    void* o;
    float scale_log2, v_scale;           // softmax scale * k_scale * log2(e)
    int32_t* counters;                   // [gridDim.x], zero between calls
    float* partials;                     // [2 gridDim.x][KV4_ROWS][D + 2]
    int32_t* status;
    int withhold;                        // the test hook: copies are expected and not issued
    const uint64_t* tree;                // [total] masks (TREE)
};

// What the columns of a query tile hold, see kda_kv4_attend_kernel.
constexpr int KV4_8 = 0, KV4_REST = 1, KV4_16 = 2;
constexpr int KV4_ROWS = 16;             // most rows of a tile
constexpr int KV4_KEYS = 32;             // keys of a unit of work: two blocks
// What beginning and ending a part costs a CTA, in units.  With 12, 16, 20, 24, 28, 32, us:
//   ragged 32 x 8 tokens, bf16, grp 6, D = 128 (KV4_16)  87.7, 71.9, 63.6, 61.2, 61.2, 63.0;  D = 64  58.5, 47.7, 44.9, 41.3, 40.2, 41.6
//   ragged 64 x 1, bf16, grp 4 (KV4_8)  D = 128  41.3, 38.1, 36.1, 35.8, 36.1, 37.7;  D = 64  36.1, 32.4, 30.7, 29.4, 28.6, 28.9
//   ragged 32 x 2, grp 4 (KV4_REST)  fp16, D = 128  25.5, 25.9, 26.8, 26.9, 28.1, 27.9;  fp32, D = 64  19.2, 18.9, 19.2, 19.5, 19.3, 19.2
// One value for all builds: the fp16 and fp32 ones, whose units take longer, would gain 5 % and 3 % with 12 and 16.
constexpr int KV4_PART = 24;
constexpr int KV4_MAX_CTAS = 512;        // counters at the head of the workspace
// Units of a warp whose products with the values (fp16 and fp32 queries) add up
// in one sum of the tensor cores, before that is added to the warp's others in
// fp32.  The tensor cores round towards zero at each of a unit's four additions:
// 2^-17 of a sum here, 2^-13 after 680 units in one.
constexpr int KV4_CHAIN = 32;
constexpr int KV4_AHEAD = 16;            // units whose pages a warp looks up at a time: lanes 2 i, 2 i + 1 a block each
// The running maximum may lag by SLACK powers of two, and probabilities are held times 2^LIFT: at most
// 2^15 in fp16, whose last step then stands for 2^-35 of the maximum's (unlifted, what many keys add behind
// a dominant one was lost).  A smaller slack moves the maximum more often: 32 x 8 ragged tokens 57.9 us
// with 8 and with 5, 58.5 with 3, 59.9 with 2.
constexpr float KV4_SLACK = 5.f, KV4_LIFT = 10.f;

// Warps of a CTA (two CTAs an SM) and units that each has in flight: as many
// warps as the registers of a mode allow.
template <int D, int MODE> struct Kv4Shape {
    static constexpr int WARPS = MODE == KV4_16 || (MODE == KV4_REST && D == 128) ? 6 : 8, THREADS = WARPS * 32;
    static constexpr int STAGES = WARPS == 6 ? 3 : 2;
    static constexpr int ROWS = MODE == KV4_16 ? 16 : 8;
    // A cut in a (request, head, row tile) leaves at least FIRST (a unit a warp behind the fixed
    // cost) before it and LAST after it, or it moves to that end; FIRST + LAST is the least share.
    static constexpr int FIRST = KV4_PART + WARPS, LAST = WARPS;
};

template <int D, int MODE> struct Kv4Smem {
    static constexpr int WARPS = Kv4Shape<D, MODE>::WARPS, STAGES = Kv4Shape<D, MODE>::STAGES;
    static constexpr int RING = WARPS * STAGES * 2 * Kv4<D>::BLOCK;
    static constexpr int MERGE = WARPS * 8 * D * 4;
    // a row of queries in 16-byte pieces (w, t) of lane t's channels 8 w .. 8 w + 7; the pitch keeps a
    // quarter-warp's reads (two rows, four t) on different banks
    static constexpr int QPITCH = D + 32;                    // halves
    static constexpr int Q = KV4_ROWS * QPITCH * 2;
    static constexpr int ML = WARPS * KV4_ROWS * 2 * 4;
    static constexpr int OFF_MERGE = RING, OFF_Q = OFF_MERGE + MERGE, OFF_ML = OFF_Q + Q,
                         OFF_ROW = OFF_ML + ML,              // row factors [16]
                         OFF_BAR = OFF_ROW + KV4_ROWS * 4,   // [warps][stages] barriers
                         OFF_FLAG = OFF_BAR + WARPS * STAGES * 8,
                         OFF_WALK = OFF_FLAG + 16,           // [warps][3] Kv4Walk
                         BYTES = OFF_WALK + WARPS * 3 * 96;
    static_assert(BYTES <= 115712, "two CTAs an SM");
};

// One request's part of the work: its tokens, and the units of 32 keys that
// any of its queries can see.
struct Kv4Req {
    int tok0, t, ctx, first, units, tiles, err;
};

template <bool TREE> __device__ __forceinline__ Kv4Req kv4_request(const Kv4AttendParams& p, int r, int rows) {
    Kv4Req q;
    q.err = 0;
    q.tok0 = p.cu ? __ldg(p.cu + r) : r * p.max_t;
    q.t = (p.cu ? __ldg(p.cu + r + 1) : q.tok0 + p.max_t) - q.tok0;
    q.ctx = __ldg(p.ctx + r);
    q.first = q.units = 0;
    if (q.tok0 < 0 || q.t < 0 || q.t > p.max_t || (int64_t)q.tok0 + q.t > p.total) {
        q.err = STATUS_ARG;
        q.tok0 = q.t = 0;
    }
    q.tiles = (q.t * p.grp + rows - 1) / rows;
    const int64_t end = (int64_t)q.ctx + q.t;
    if (q.t > 0 && end > 0) {
        if (end > (int64_t)p.cols * p.page_tokens || (p.rot && end > p.rope_rows) || (TREE && q.ctx < 0)) {
            q.err = STATUS_ARG;
        } else {
            if (p.window > 0) q.first = max(0, max(q.ctx, 0) - p.window + 1) / KV4_KEYS;
            q.units = (int)((end + KV4_KEYS - 1) / KV4_KEYS) - q.first;
        }
    }
    return q;
}

// Cost of a request: each (head, row tile) its units, behind KV4_PART for its
// beginning and end.
__device__ __forceinline__ int kv4_cost(const Kv4Req& q, int heads) {
    return q.units > 0 ? (q.units + KV4_PART) * q.tiles * heads : 0;   // the host bounds it by the page table
}

// A walk over a CTA's share of the flattened list of costs: each step is the
// part of one (request, head, row tile) whose units lie in the share.
struct Kv4Walk {
    int64_t left;        // of the share, not yet taken
    int64_t end, even;   // where the share ends in the list; an even share
    int r, off;          // request, and what is taken of it
    Kv4Req q;
    int h, i0, b0, b1;   // the current step: head, first row of the tile, units [b0, b1)
    int b;               // (fetching) this warp's next unit not looked up
    template <bool TREE> __device__ __forceinline__ bool next(const Kv4AttendParams& p, int rows) {
        do {
            if (left <= 0) return false;
            while (off >= kv4_cost(q, p.heads)) {
                if (++r >= p.n) return false;
                q = kv4_request<TREE>(p, r, rows);
                off = 0;
            }
            const int each = q.units + KV4_PART;
            const int seg = off / each, u = off - seg * each;
            h = seg / q.tiles;
            i0 = (seg - h * q.tiles) * rows;
            const int take = (int)min((int64_t)(each - u), left);
            b0 = max(0, u - KV4_PART);
            b1 = max(0, u + take - KV4_PART);
            off += take;
            left -= take;
        } while (b0 == b1);
        return true;
    }
};

// Attention over the cache, one pass with a running maximum and sum.
//
// Operands.  Keys and values are the A operand of the mma (m16n8k16, fp16,
// fp32 sums): S^T = K Q^T with 16 keys by 8 query rows, and O^T += V^T P^T with
// 16 channels by 8 rows; the 8 rows are the query heads of one key/value head
// and the request's tokens.  A code times its scale has at most 6 significant
// bits, so keys and values are exact in fp16.  Queries are scaled by a power of
// two a row to below 1 and rounded to fp16.  MODE says what B operands each
// decoded A operand meets:
//   KV4_8     8 rows, queries and probabilities rounded to 11 bits, an eighth of
//             the output's own rounding: bf16 queries with up to 8 rows
//   KV4_REST  8 rows, and again with the fp16 remainders of queries and of
//             probabilities into the same sums, so that products carry 22
//             bits: fp16 and fp32 queries
//   KV4_16    two times 8 rows as KV4_8: bf16 queries with more
// KV4_REST also adds a warp's sums up in fp32 every few units (see KV4_CHAIN); a
// single sum of bf16 queries loses 2^-13 over 131072 keys that six warps share.
// In every mode a probability is also off by up to 2^-35 of the row's largest
// (fp16's smallest steps, see KV4_LIFT).
// P leaves the first product with keys along the lane's rows and enters the
// second with keys along its columns: two 8 x 8 transposes a block.
//
// Channel order.  A product over channels may take them in any order, so lane
// (g, t) takes channels t D / 4 .. of key g: 16 contiguous code bytes (D =
// 128), and at most two scales.
//
// Split.  All (request, head, tile, unit) are one list, cut evenly over the
// CTAs whatever the lengths; a CTA's warps take its units in turn, each with
// its own ring of bulk copies, and join at the end of a part.  Parts of one
// (request, head, tile) in several CTAs go to the workspace, and the CTA that
// arrives last joins them in order (results do not depend on who that is).
//
// Bound by issue: decoding fills half of the ALU pipe, and 16 warps an SM (the
// registers of the sums, the rings) leave 0.4 of the issue slots empty.  A loop
// of decode and mma alone takes 290 cycles a block and scheduler, this kernel
// about 430.  64 requests x 8192 tokens, 32/8 heads of 128: 117 us, 5.2 TB/s of
// cache, 0.76 of the measured copy bandwidth.  Keys and values as the B operand
// (query rows on the 16-row side, half of it idle): 168 us.
//
// TREE: the request's tokens are a tree of drafted tokens behind its ctx keys.
// Token j is rotated as at position ctx + its depth, and of the keys from ctx on
// sees those in its mask: only the units there are masked key by key.
template <int D, int MODE, bool TREE = false>
__global__ void __launch_bounds__(Kv4Shape<D, MODE>::THREADS, 2) kda_kv4_attend_kernel(const Kv4AttendParams p) {
    using F = Kv4<D>;
    using SM = Kv4Smem<D, MODE>;
    using SH = Kv4Shape<D, MODE>;
    constexpr int KV4_WARPS = SH::WARPS, KV4_THREADS = SH::THREADS, KV4_STAGES = SH::STAGES;
    constexpr bool SPLIT = MODE == KV4_REST;
    constexpr int ROWS = SH::ROWS;            // rows of a tile
    constexpr int MT = D / 16;                // m tiles of the output
    constexpr int NB = MODE == KV4_16 ? 2 : 1;   // sets of 8 rows
    extern __shared__ __align__(128) uint8_t smem[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    uint8_t* ring = smem + warp * (KV4_STAGES * 2 * F::BLOCK);
    float* merge = reinterpret_cast<float*>(smem + SM::OFF_MERGE);
    __half* qbuf = reinterpret_cast<__half*>(smem + SM::OFF_Q);
    float* ml = reinterpret_cast<float*>(smem + SM::OFF_ML);          // [warp][16] m, then l
    float* rowf = reinterpret_cast<float*>(smem + SM::OFF_ROW);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + SM::OFF_BAR) + warp * KV4_STAGES;
    volatile int* last_to_come = reinterpret_cast<int*>(smem + SM::OFF_FLAG);

    if (lane == 0) {
#pragma unroll
        for (int s = 0; s < KV4_STAGES; ++s) mbar_init(bars + s, 1);
        fence_mbar_init();
    }
    cudaTriggerProgrammaticLaunchCompletion();
    cudaGridDependencySynchronize();

    // what is being fetched, what comes next, what is being worked on: a warp's own, in shared
    // memory (read seldom; the registers go to the accumulators)
    static_assert(sizeof(Kv4Walk) <= 96, "Kv4Smem::OFF_WALK");
    auto walk = [&](int i) -> Kv4Walk& { return *reinterpret_cast<Kv4Walk*>(smem + SM::OFF_WALK + (3 * warp + i) * 96); };
    Kv4Walk &put = walk(0), &get = walk(1), &cur = walk(2);

    // ---- the share of this CTA: the list between two cuts; every warp finds it for itself ----
    const int cnt = (p.n + 31) / 32;
    int64_t mine = 0;
    bool empty = false;
    Kv4Req own;      // of a lane with one request
#pragma unroll 2
    for (int r = lane * cnt; r < min(p.n, (lane + 1) * cnt); ++r) {
        own = kv4_request<TREE>(p, r, ROWS);
        mine += kv4_cost(own, p.heads);
        empty |= own.t > 0 && own.units == 0;
        if (own.err && blockIdx.x == 0 && warp == 0) atomicCAS(p.status, 0, own.err);
    }
    int64_t before = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t up = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += up;
    }
    const int64_t total = __shfl_sync(0xffffffffu, before, 31);
    before -= mine;
    const int64_t even = max((int64_t)(SH::FIRST + SH::LAST),
                             total <= 0x7fffffff ? (int64_t)(((unsigned)total + gridDim.x - 1) / gridDim.x)
                                                 : (total + gridDim.x - 1) / gridDim.x);
    int64_t cut[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        cut[k] = even * (blockIdx.x + k);
        const bool here = before <= cut[k] && cut[k] < before + mine;
        if (here) {
            int64_t at = cut[k] - before;
            Kv4Req q = own;
            int r = lane * cnt;
            for (;; ++r) {
                if (cnt > 1) q = kv4_request<TREE>(p, r, ROWS);
                const int c = kv4_cost(q, p.heads);
                if (at < c) break;
                at -= c;
            }
            const int each = q.units + KV4_PART, u = (int)at % each;
            const int move = u < SH::FIRST ? -u : each - u < SH::LAST ? each - u : 0;
            cut[k] += move;
            if (k == 0) {
                get.r = r;
                get.off = (int)at + move;
                get.q = q;
            }
        }
        const uint32_t who = __ballot_sync(0xffffffffu, here);
        cut[k] = who ? __shfl_sync(0xffffffffu, cut[k], __ffs(who) - 1) : total;
    }
    if (__any_sync(0xffffffffu, empty)) {  // requests without a visible key: zero rows
        for (int r = blockIdx.x; r < p.n; r += gridDim.x) {
            const Kv4Req q = kv4_request<TREE>(p, r, ROWS);
            if (q.units > 0) continue;
            const int64_t base = (int64_t)q.tok0 * p.h_q * D;
            for (int64_t i = tid * 4; i < (int64_t)q.t * p.h_q * D; i += KV4_THREADS * 4)
                st_elem4(p.o, base + i, p.dtype, 0.f, 0.f, 0.f, 0.f);
        }
    }
    if (cut[0] >= cut[1]) return;
    __syncwarp();
    if (lane == 0) {
        get.left = cut[1] - cut[0];
        get.end = cut[1];
        get.even = even;
    }
    auto step = [&](Kv4Walk& w) {   // lane 0 walks, all lanes see it
        int ok = 0;
        __syncwarp();
        if (lane == 0) ok = w.template next<TREE>(p, ROWS);
        __syncwarp();               // the walk is in shared memory, and a shuffle orders no memory
        return __shfl_sync(0xffffffffu, ok, 0) != 0;
    };

    // ---- queries: R rows a warp; loaded ahead, then rotated, scaled and rounded ----
    constexpr int E = D / 32, R = (ROWS + KV4_WARPS - 1) / KV4_WARPS;
    float x[R][E], y[R][E], cs[R][E], sn[R][E];
    auto load_q = [&]() {
        const int d = lane * E, half = p.rot >> 1, h = get.h, i0 = get.i0;
        const bool first = d < half;
#pragma unroll
        for (int k = 0; k < R; ++k) {
            const int i = i0 + warp + k * KV4_WARPS, j = i / p.grp;
            const int pos = get.q.ctx + (TREE && j < get.q.t ? __popcll(tree_mask(p.tree, get.q.tok0 + j, j)) - 1 : j);
            const int64_t base = (int64_t)(get.q.tok0 + j) * p.q_stride + (int64_t)(h * p.grp + i - j * p.grp) * D;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                x[k][e] = y[k][e] = sn[k][e] = 0.f;
                cs[k][e] = 1.f;
            }
            if (i - i0 >= ROWS || j >= get.q.t || pos < 0) continue;
            ld_elems<E>(p.q, base + d, p.dtype, x[k]);
            if (d < p.rot) {
                const int64_t row = (int64_t)pos * half;
                if (p.inter) {
                    ld_elems<E / 2>(p.cos, row + d / 2, 0, cs[k]);
                    ld_elems<E / 2>(p.sin, row + d / 2, 0, sn[k]);
                } else {
                    ld_elems<E>(p.q, base + (first ? d + half : d - half), p.dtype, y[k]);
                    ld_elems<E>(p.cos, row + (first ? d : d - half), 0, cs[k]);
                    ld_elems<E>(p.sin, row + (first ? d : d - half), 0, sn[k]);
                }
            }
        }
    };
    auto store_q = [&]() {
        const int d = lane * E;
        const bool first = d < p.rot >> 1;
#pragma unroll
        for (int k = 0; k < R; ++k) {
            const int i = warp + k * KV4_WARPS;
            if (d < p.rot) {
                if (p.inter) {
#pragma unroll
                    for (int e = E / 2 - 1; e >= 0; --e) {
                        const float a = x[k][2 * e], b = x[k][2 * e + 1];
                        x[k][2 * e] = a * cs[k][e] - b * sn[k][e];
                        x[k][2 * e + 1] = b * cs[k][e] + a * sn[k][e];
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < E; ++e) x[k][e] = x[k][e] * cs[k][e] + (first ? -y[k][e] : y[k][e]) * sn[k][e];
                }
            }
            float amax = 0.f;
#pragma unroll
            for (int e = 0; e < E; ++e) amax = fmaxf(amax, fabsf(x[k][e]));
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
            // 2^-z with amax 2^-z in [1/2, 1); rows of nothing or below 1e-30 stay as they are; rows of an
            // infinity or past 1e37 become NaN (scores of minus infinity alone would read as keys not seen)
            const int z = amax > 1e-30f && amax < 1e37f ? (int)(__float_as_uint(amax) >> 23) - 126 : 0;
            // the factor is positive (not 0: a masked score times it stays -infinity), queries take the sign
            const float down =
                __uint_as_float(amax < 1e37f ? (uint32_t)(127 - z) << 23 | (__float_as_uint(p.scale_log2) & 0x80000000u) : 0x7fffffffu);
            if (i < ROWS) {
#pragma unroll
                for (int e = 0; e < E; e += 2) {
                    const float u = x[k][e] * down, v = x[k][e + 1] * down;
                    const __half2 hi = __floats2half2_rn(u, v);
                    const int dd = d + e, at = (dd % (D / 4) / 8 * 4 + dd / (D / 4)) * 8 + dd % 8;
                    *reinterpret_cast<__half2*>(qbuf + i * SM::QPITCH + at) = hi;
                    if constexpr (SPLIT) {
                        const float2 f = __half22float2(hi);
                        *reinterpret_cast<__half2*>(qbuf + (i + 8) * SM::QPITCH + at) = __floats2half2_rn(u - f.x, v - f.y);
                    }
                }
                if (lane == 0) rowf[i] = fmaxf(1e-30f, fabsf(p.scale_log2) * __uint_as_float((uint32_t)(127 + z) << 23));
            }
        }
    };
    bool have = step(get);
    if (have) load_q();
    if (lane == 0) {
        put = get;
        put.b = have ? get.b0 + warp : 0;
        if (!have) put.b1 = 0;
    }
    __syncwarp();

    const int bpp = p.page_tokens >> 4;
    // one register of flags: bits 0.. the slots' phase parities, 8.. two bits a slot, its blocks
    // that were not fetched, MORE to fetch, ALIVE until a wait runs out
    constexpr uint32_t MORE = 1u << 16, ALIVE = 1u << 17;
    uint32_t flags = MORE | ALIVE;
    const uint8_t* from = nullptr;      // lanes 2 i and 2 i + 1: the two blocks of the i-th unit looked up
    uint32_t there = 0;                 // blocks that are there, from the next unit's on
    int looked = 0;                     // units looked up and not yet fetched

    // Looks up the pages of this warp's next units; false behind the last.
    auto look = [&]() {
        while (put.b >= put.b1) {
            if (!step(put)) return false;
            if (lane == 0) put.b = put.b0 + warp;
            __syncwarp();
        }
        const int first = put.b, mine = first + KV4_WARPS * (lane >> 1);
        bool ok = false;
        const int b = (put.q.first + mine) * 2 + (lane & 1);
        // a request's last unit may be one block, and so may its first: the page left of a window may be released
        if (mine < put.b1 && b * 16 < put.q.ctx + put.q.t &&
            (p.window <= 0 || max(put.q.ctx, 0) - p.window + 1 < (b + 1) * 16)) {
            const int pg = b / bpp, page = __ldg(p.table + (int64_t)put.r * p.cols + pg);
            ok = page >= 0 && page < p.num_pages;
            if (!ok) atomicCAS(p.status, 0, STATUS_SLOT_RANGE);
            from = p.pages + (int64_t)page * p.page_stride + ((int64_t)put.h * bpp + (b - pg * bpp)) * F::BLOCK;
        }
        there = __ballot_sync(0xffffffffu, ok);
        looked = min(KV4_AHEAD, (put.b1 - first + KV4_WARPS - 1) / KV4_WARPS);
        // the next unit's lanes are 0 and 1 until fetch() turns the lanes
        __syncwarp();
        if (lane == 0) put.b = first + KV4_WARPS * looked;
        __syncwarp();
        return true;
    };
    int turn = 0;                       // lane of the next unit's first block
    // Fetches this warp's next unit into a slot.
    auto fetch = [&](uint32_t slot) {
        if (!(flags & MORE)) return;
        if (looked == 0) {
            turn = 0;
            if (!look()) {
                flags &= ~MORE;
                return;
            }
        }
        const uint32_t two = there & 3u;
        flags = (flags & ~(3u << (8 + 2 * slot))) | (two ^ 3u) << (8 + 2 * slot);
        const int mine = lane - turn;
        if ((mine & ~1) == 0) {         // the copies may complete before they are expected: the phase waits for the arrival
            if (mine == 0 && two != 0) mbar_arrive_expect_tx(bars + slot, two == 3u ? 2 * F::BLOCK : F::BLOCK);
            if ((two >> mine & 1u) && !p.withhold) bulk_load(ring + (2 * slot + mine) * F::BLOCK, from, F::BLOCK, bars + slot);
        }
        there >>= 2;
        turn += 2;
        --looked;
    };
#pragma unroll 1
    for (int s = 0; s < KV4_STAGES; ++s) fetch(s);
    uint32_t slot = 0;                  // the slot to work on, and then to fetch into

    // a row's position and the tile's last one: worked out where they are needed, not kept in
    // registers
    auto row_pos = [&](int i) { return cur.q.ctx + (cur.i0 + i) / p.grp; };
    // (a tree's row may see any token of the request: the last one)
    auto last_row_pos = [&]() {
        if constexpr (TREE) return cur.q.ctx + cur.q.t - 1;
        return cur.q.ctx + min(cur.q.t - 1, (cur.i0 + ROWS - 1) / p.grp);
    };
    // a tree's row sees keys by its mask, of which a window leaves the last ones, and the first key of the context that it sees
    auto tree_row = [&](int i, uint64_t& own, int& low) {
        const int j = (cur.i0 + i) / p.grp;
        own = 0;
        low = 0x7fffffff;
        if (j >= cur.q.t) return;
        own = tree_mask(p.tree, cur.q.tok0 + j, j);
        low = p.window > 0 ? cur.q.ctx + __popcll(own) - p.window : 0;
        if (p.window > 0)
            for (int more = __popcll(own) - p.window; more > 0; --more) own &= own - 1;
    };
    auto sees_tree = [&](uint64_t own, int low, int key) {
        const int at = key - cur.q.ctx;
        return at < 0 ? key >= low : at < TREE_MAX && (own >> at & 1u) != 0;
    };

    while (have) {
        store_q();
#pragma unroll
        for (int k = 0; k < R; ++k)      // not to be kept: the next part loads its own
#pragma unroll
            for (int e = 0; e < E; ++e) x[k][e] = y[k][e] = cs[k][e] = sn[k][e] = 0.f;
        __syncwarp();
        if (lane == 0) cur = get;
        __syncthreads();
        // query fragments of row g and of row g + 8: eight channels, two k steps, a piece
        uint4 qa[D / 32], qb[MODE == KV4_8 ? 1 : D / 32];
        {
            const uint4* qr = reinterpret_cast<const uint4*>(qbuf + g * SM::QPITCH) + t;
#pragma unroll
            for (int w = 0; w < D / 32; ++w) qa[w] = qr[w * 4];
            if constexpr (MODE != KV4_8) {
#pragma unroll
                for (int w = 0; w < D / 32; ++w) qb[w] = qr[8 * SM::QPITCH / 8 + w * 4];
            }
        }
        // this lane's rows: 8 n + 2 t and the next, index 2 n + e
        float m[2 * NB], l[2 * NB];     // running maximum and sum
        float bar[2];                   // the score above which the maximum moves (with two sets of rows worked out each time)
#pragma unroll
        for (int a = 0; a < 2 * NB; ++a) {
            m[a] = -FLT_MAX;    // finite: nothing below is infinity minus infinity
            if constexpr (NB == 1) bar[a] = -FLT_MAX;
            l[a] = 0.f;
        }
        auto row_of = [&](int a) { return 8 * (a >> 1) + 2 * t + (a & 1); };
        // units that every row of the tile sees whole: [see0, see1)
        const int see1 = (TREE ? cur.q.ctx : row_pos(0) + 1) / KV4_KEYS;
        const int see0 = p.window > 0 ? (max(0, last_row_pos() - p.window + 1) + KV4_KEYS - 1) / KV4_KEYS : 0;
        // sums of channels g D / 8 + 2 i (elements 0, 1: the lane's rows) and the next (2, 3)
        float acc[NB][MT][4];
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int j = 0; j < MT; ++j) acc[n][j][0] = acc[n][j][1] = acc[n][j][2] = acc[n][j][3] = 0.f;

        // Sums that are kept lie where the warp's are joined from, with their rows' (maximum, sum of probabilities).
        auto kept_at = [&](int e, int k) {      // 16-byte piece k of this lane's channels of its row e
            return reinterpret_cast<float4*>(merge + (warp * 8 + 2 * t + e) * D + ((g * (D / 32) + k) ^ t) * 4);
        };
        bool kept = false;
        int unit = cur.q.first + cur.b0 + warp;
        const int end = cur.q.first + cur.b1;
#pragma unroll 1
        for (;;) {
#pragma unroll 1
            for (const int stop = SPLIT ? min(end, unit + KV4_CHAIN * KV4_WARPS) : end; unit < stop; unit += KV4_WARPS) {
                bool use = (flags & ALIVE) && (flags >> (8 + 2 * slot) & 3u) != 3u;
                if (use) {
                    // the warp's verdict, not a lane's: a copy may land while some lanes give up
                    use = __all_sync(0xffffffffu, mbar_wait(bars + slot, flags >> slot & 1u));
                    if (use) {
                        flags ^= 1u << slot;
                    } else {
                        flags &= ~(MORE | ALIVE);
                        if (lane == 0) atomicCAS(p.status, 0, STATUS_TIMEOUT);
                    }
                }
                if (use) {
                    const uint8_t* B = ring + slot * (2 * F::BLOCK);
                    // ---- scores: s[blk][n][..] of keys 16 blk + g (0, 1) and g + 8 (2, 3) with the lane's rows ----
                    float s[2][NB][4];
#pragma unroll
                    for (int blk = 0; blk < 2; ++blk) {
                        const uint8_t* K = B + blk * F::BLOCK;
#pragma unroll
                        for (int n = 0; n < NB; ++n) s[blk][n][0] = s[blk][n][1] = s[blk][n][2] = s[blk][n][3] = 0.f;
                        uint32_t code[2][D / 32], sc[2];   // sc: scales of the lane's two groups (D = 64: of its one)
#pragma unroll
                        for (int hf = 0; hf < 2; ++hf) {
                            const int key = hf * 8 + g;
                            if constexpr (D == 128) {
                                const uint4 w = *reinterpret_cast<const uint4*>(K + F::KC + key * 64 + t * 16);
                                code[hf][0] = w.x; code[hf][1] = w.y; code[hf][2] = w.z; code[hf][3] = w.w;
                                sc[hf] = cvt_e4m3x2_f16x2(*reinterpret_cast<const uint16_t*>(K + F::KS + key * 8 + 2 * t));
                            } else {
                                const uint2 w = *reinterpret_cast<const uint2*>(K + F::KC + key * 32 + t * 8);
                                code[hf][0] = w.x; code[hf][1] = w.y;
                                sc[hf] = cvt_e4m3x2_f16x2(K[F::KS + key * 4 + t]);
                            }
                        }
#pragma unroll
                        for (int w = 0; w < D / 32; ++w) {
                            uint32_t k0[4], k1[4];
                            cvt_e2m1x8_f16(code[0][w], k0);
                            cvt_e2m1x8_f16(code[1][w], k1);
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                k0[e] = w < 2 ? hmul2_half<false>(k0[e], sc[0]) : hmul2_half<true>(k0[e], sc[0]);
                                k1[e] = w < 2 ? hmul2_half<false>(k1[e], sc[1]) : hmul2_half<true>(k1[e], sc[1]);
                            }
                            kv4_mma(s[blk][0], k0[0], k1[0], k0[1], k1[1], qa[w].x, qa[w].y);
                            if constexpr (MODE != KV4_8) kv4_mma(s[blk][NB - 1], k0[0], k1[0], k0[1], k1[1], qb[w].x, qb[w].y);
                            kv4_mma(s[blk][0], k0[2], k1[2], k0[3], k1[3], qa[w].z, qa[w].w);
                            if constexpr (MODE != KV4_8) kv4_mma(s[blk][NB - 1], k0[2], k1[2], k0[3], k1[3], qb[w].z, qb[w].w);
                        }
                    }
                    // ---- running softmax ----
                    const uint32_t miss = flags >> (8 + 2 * slot) & 3u;
                    const bool masked = unit < see0 || unit >= see1 || miss != 0;
                    if (masked) {
#pragma unroll
                        for (int a = 0; a < 2 * NB; ++a) {
                            if constexpr (TREE) {
                                uint64_t own;
                                int low;
                                tree_row(row_of(a), own, low);
#pragma unroll
                                for (int i = 0; i < 4; ++i)
                                    if (!sees_tree(own, low, unit * KV4_KEYS + i * 8 + g) || (miss >> (i >> 1) & 1u))
                                        s[i >> 1][a >> 1][2 * (i & 1) + (a & 1)] = -INFINITY;
                                continue;
                            }
                            const int pos = row_pos(row_of(a));
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const int key = unit * KV4_KEYS + i * 8 + g;
                                if (key > pos || (p.window > 0 && key <= pos - p.window) || (miss >> (i >> 1) & 1u))
                                    s[i >> 1][a >> 1][2 * (i & 1) + (a & 1)] = -INFINITY;
                            }
                        }
                    }
                    float top[2 * NB];
                    bool grow = false;
#pragma unroll
                    for (int a = 0; a < 2 * NB; ++a) {
                        const int n = a >> 1, e = a & 1;
                        top[a] = fmaxf(fmaxf(s[0][n][e], s[0][n][2 + e]), fmaxf(s[1][n][e], s[1][n][2 + e]));
                        if constexpr (NB == 1) grow |= top[a] > bar[a];
                        else grow |= top[a] * rowf[row_of(a)] > m[a] + KV4_SLACK;
                    }
                    // rarely: a score above the running maximum by more than its slack
                    if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                        for (int a = 0; a < 2 * NB; ++a) {
#pragma unroll
                            for (int o = 4; o < 32; o <<= 1) top[a] = fmaxf(top[a], __shfl_xor_sync(0xffffffffu, top[a], o));
                            const float c = rowf[row_of(a)];
                            top[a] *= c;
                            if (top[a] > m[a]) {
                                if constexpr (NB == 1) bar[a] = (top[a] + KV4_SLACK) / c;
                                const float f = ex2f(m[a] - top[a]);
                                m[a] = top[a];
                                l[a] *= f;
#pragma unroll
                                for (int j = 0; j < MT; ++j) {
                                    acc[a >> 1][j][a & 1] *= f;
                                    acc[a >> 1][j][2 + (a & 1)] *= f;
                                }
                            }
                        }
                    }
                    uint32_t pf[2][NB][2], pr[SPLIT ? 2 : 1][2];   // B fragments of the probabilities, of their remainders
#pragma unroll
                    for (int n = 0; n < NB; ++n) {
                        // both rows at once (packed fp32)
                        const float2 c = *reinterpret_cast<const float2*>(rowf + row_of(2 * n));
                        const float2 neg = make_float2(KV4_LIFT - m[2 * n], KV4_LIFT - m[2 * n + 1]);
                        float2 sum = make_float2(l[2 * n], l[2 * n + 1]);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float2 e = __ffma2_rn(make_float2(s[i >> 1][n][2 * (i & 1)], s[i >> 1][n][2 * (i & 1) + 1]), c, neg);
                            const float x0 = ex2f(e.x), x1 = ex2f(e.y);
                            sum = __fadd2_rn(sum, make_float2(x0, x1));
                            const __half2 hi = __floats2half2_rn(x0, x1);
                            pf[i >> 1][n][i & 1] = movmatrix_t(*reinterpret_cast<const uint32_t*>(&hi));
                            if constexpr (SPLIT) {
                                const float2 f = __half22float2(hi);
                                const __half2 rest = __floats2half2_rn(x0 - f.x, x1 - f.y);
                                pr[i >> 1][i & 1] = movmatrix_t(*reinterpret_cast<const uint32_t*>(&rest));
                            }
                        }
                        l[2 * n] = sum.x;
                        l[2 * n + 1] = sum.y;
                    }
                    // ---- values ----
#pragma unroll
                    for (int blk = 0; blk < 2; ++blk) {
                        const uint8_t* W = B + blk * F::BLOCK;
                        const int grp = g * (D / 8) / 16;       // the lane's channels are of one scale group
                        uint32_t vs4 = *reinterpret_cast<const uint32_t*>(W + F::VS + (grp * 4 + t) * 4);
                        if (masked) {
                            // A token that some row does not see may hold anything, and 0 * NaN is NaN:
                            // scales behind the end become 0, and so do NaN ones, whose channels of the
                            // rows that do see them are then set by hand (a rare path).
                            const int key0 = unit * KV4_KEYS + blk * 16, to = (miss >> blk & 1u) ? -1 : last_row_pos();
                            bool nan = false;
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const int key = key0 + (e >> 1) * 8 + 2 * t + (e & 1);
                                const bool bad = (vs4 >> (8 * e) & 0x7fu) == 0x7fu;
                                if (key > to || bad) vs4 &= ~(0xffu << (8 * e));
                                nan |= bad && key <= to;
                            }
                            if (__any_sync(0xffffffffu, nan)) {
                                uint32_t hit = 0;
#pragma unroll 1
                                for (int w = 0; w < 16; ++w) {
                                    if ((W[kv4_v_scale<D>(w, grp)] & 0x7f) != 0x7f || key0 + w > to) continue;
#pragma unroll
                                    for (int a = 0; a < 2 * NB; ++a) {
                                        if constexpr (TREE) {
                                            uint64_t own;
                                            int low;
                                            tree_row(row_of(a), own, low);
                                            if (sees_tree(own, low, key0 + w)) hit |= 1u << a;
                                            continue;
                                        }
                                        const int pos = row_pos(row_of(a));
                                        if (key0 + w <= pos && (p.window <= 0 || key0 + w > pos - p.window)) hit |= 1u << a;
                                    }
                                }
#pragma unroll
                                for (int a = 0; a < 2 * NB; ++a)
                                    if (hit >> a & 1u)
#pragma unroll
                                        for (int j = 0; j < MT; ++j) acc[a >> 1][j][a & 1] = acc[a >> 1][j][2 + (a & 1)] = NAN;
                            }
                        }
                        const uint32_t sv[2] = {cvt_e4m3x2_f16x2(vs4 & 0xffffu), cvt_e4m3x2_f16x2(vs4 >> 16)};
                        uint32_t vc[2][2][D / 64];          // [half][token of the pair][word]
#pragma unroll
                        for (int hf = 0; hf < 2; ++hf) {
                            const uint8_t* V = W + F::VC + hf * (64 * F::CB) + lane * (2 * F::CB);
                            if constexpr (D == 128) {
                                const uint4 w = *reinterpret_cast<const uint4*>(V);
                                vc[hf][0][0] = w.x; vc[hf][0][1] = w.y; vc[hf][1][0] = w.z; vc[hf][1][1] = w.w;
                            } else {
                                const uint2 w = *reinterpret_cast<const uint2*>(V);
                                vc[hf][0][0] = w.x; vc[hf][1][0] = w.y;
                            }
                        }
#pragma unroll
                        for (int w = 0; w < D / 64; ++w) {
                            uint32_t ev[2][4], od[2][4];   // pairs (token 2t, token 2t + 1) of the even and of the odd channels
#pragma unroll
                            for (int hf = 0; hf < 2; ++hf) {
                                const uint32_t A = vc[hf][0][w], C = vc[hf][1][w];
                                cvt_e2m1x8_f16((A & 0x0f0f0f0fu) | (C << 4 & 0xf0f0f0f0u), ev[hf]);
                                cvt_e2m1x8_f16((A >> 4 & 0x0f0f0f0fu) | (C & 0xf0f0f0f0u), od[hf]);
                            }
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const uint32_t a0 = hmul2_u32(ev[0][e], sv[0]), a1 = hmul2_u32(od[0][e], sv[0]);
                                const uint32_t a2 = hmul2_u32(ev[1][e], sv[1]), a3 = hmul2_u32(od[1][e], sv[1]);
#pragma unroll
                                for (int n = 0; n < NB; ++n) kv4_mma(acc[n][4 * w + e], a0, a1, a2, a3, pf[blk][n][0], pf[blk][n][1]);
                                if constexpr (SPLIT) kv4_mma(acc[0][4 * w + e], a0, a1, a2, a3, pr[blk][0], pr[blk][1]);
                            }
                        }
                    }
                }
                __syncwarp();
                fetch(slot);
                slot = slot + 1 == KV4_STAGES ? 0 : slot + 1;
            }
            if (!SPLIT || unit >= end) break;
            if constexpr (SPLIT) {
                // the products of the units to come start new sums
                float f[2], lk[2];
#pragma unroll
                for (int a = 0; a < 2; ++a) {
                    const float2 old = kept ? *reinterpret_cast<const float2*>(ml + (warp * KV4_ROWS + row_of(a)) * 2) : make_float2(-FLT_MAX, 0.f);
                    f[a] = ex2f(old.x - m[a]);
#pragma unroll
                    for (int o = 4; o < 32; o <<= 1) l[a] += __shfl_xor_sync(0xffffffffu, l[a], o);
                    lk[a] = fmaf(old.y, f[a], l[a]);
                    l[a] = 0.f;
                }
                __syncwarp();
#pragma unroll
                for (int a = 0; a < 2; ++a) {
                    if (g == 0) *reinterpret_cast<float2*>(ml + (warp * KV4_ROWS + row_of(a)) * 2) = make_float2(m[a], lk[a]);
#pragma unroll
                    for (int k = 0; k < D / 32; ++k) {
                        float4* to = kept_at(a, k);
                        float4 v = make_float4(acc[0][2 * k][a], acc[0][2 * k][2 + a], acc[0][2 * k + 1][a], acc[0][2 * k + 1][2 + a]);
                        if (kept) v = make_float4(fmaf(to->x, f[a], v.x), fmaf(to->y, f[a], v.y), fmaf(to->z, f[a], v.z), fmaf(to->w, f[a], v.w));
                        *to = v;
                        acc[0][2 * k][a] = acc[0][2 * k][2 + a] = acc[0][2 * k + 1][a] = acc[0][2 * k + 1][2 + a] = 0.f;
                    }
                }
                __syncwarp();
                kept = true;
            }
        }

        // ---- the warps' sums of this part, joined in warp order ----
        __syncwarp();
        const int live = min(ROWS, cur.q.t * p.grp - cur.i0);
        const bool whole = cur.b0 == 0 && cur.b1 == cur.q.units;
        float* part = p.partials + (2 * blockIdx.x + (cur.b0 == 0 ? 1 : 0)) * (KV4_ROWS * (D + 2));
#pragma unroll
        for (int a = 0; a < 2 * NB; ++a) {
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) l[a] += __shfl_xor_sync(0xffffffffu, l[a], o);
            if (SPLIT && kept) {
                const float2 old = *reinterpret_cast<const float2*>(ml + (warp * KV4_ROWS + row_of(a)) * 2);
                const float f = ex2f(old.x - m[a]);
                l[a] = fmaf(old.y, f, l[a]);
#pragma unroll
                for (int k = 0; k < D / 32; ++k) {
                    const float4 v = *kept_at(a, k);
                    acc[0][2 * k][a] = fmaf(v.x, f, acc[0][2 * k][a]);
                    acc[0][2 * k][2 + a] = fmaf(v.y, f, acc[0][2 * k][2 + a]);
                    acc[0][2 * k + 1][a] = fmaf(v.z, f, acc[0][2 * k + 1][a]);
                    acc[0][2 * k + 1][2 + a] = fmaf(v.w, f, acc[0][2 * k + 1][2 + a]);
                }
                __syncwarp();
            }
            if (g == 0) {
                ml[(warp * KV4_ROWS + row_of(a)) * 2] = m[a];
                ml[(warp * KV4_ROWS + row_of(a)) * 2 + 1] = l[a];
            }
        }
        auto join = [&](int row, int d, float4 o, float L) {
            const int j = (cur.i0 + row) / p.grp;
            const int64_t out = ((int64_t)(cur.q.tok0 + j) * p.h_q + cur.h * p.grp + (cur.i0 + row) - j * p.grp) * D + d;
            const float f = L == 0.f ? 0.f : p.v_scale / L;
            if (L == 0.f) o = make_float4(0.f, 0.f, 0.f, 0.f);
            st_elem4(p.o, out, p.dtype, o.x * f, o.y * f, o.z * f, o.w * f);
        };
        constexpr int CH = D / 4;             // 16-byte pieces of a row
#pragma unroll
        for (int a = 0; a < NB; ++a) {
            if (8 * a < live) {
                if (a > 0) __syncthreads();
                // a row's 16-byte pieces, each at its place xor (row / 2) % 4: eight lanes' stores fall on
                // different banks
                const int tid3 = tid_again(), g3 = (tid3 & 31) >> 2, t3 = tid3 & 3;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float* row = merge + ((tid3 >> 5) * 8 + 2 * t3 + e) * D;
#pragma unroll
                    for (int k = 0; k < D / 32; ++k)
                        *reinterpret_cast<float4*>(row + ((g3 * (D / 32) + k) ^ t3) * 4) =
                            make_float4(acc[a][2 * k][e], acc[a][2 * k][2 + e], acc[a][2 * k + 1][e], acc[a][2 * k + 1][2 + e]);
                }
                if (live <= 8 * (a + 1)) {     // the sums are written: their registers take the next part's queries
                    have = step(get);
                    if (have) load_q();
                }
                __syncthreads();
                const int tid2 = tid_again(), ch = tid2 % CH;
                for (int row = tid2 / CH; row < min(8, live - 8 * a); row += KV4_THREADS / CH) {
                    const int sw = ch ^ (row >> 1 & 3);
                    float M = -FLT_MAX, L = 0.f;
                    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                    for (int w = 0; w < KV4_WARPS; ++w) M = fmaxf(M, ml[(w * KV4_ROWS + row + 8 * a) * 2]);
#pragma unroll 2
                    for (int w = 0; w < KV4_WARPS; ++w) {
                        const float mw = ml[(w * KV4_ROWS + row + 8 * a) * 2], lw = ml[(w * KV4_ROWS + row + 8 * a) * 2 + 1];
                        const float f = ex2f(mw - M);   // a warp that saw no key: sums of 0 (a NaN stays one)
                        const float4 v = *reinterpret_cast<const float4*>(merge + (w * 8 + row) * D + sw * 4);
                        L += f * lw;
                        o.x += f * v.x; o.y += f * v.y; o.z += f * v.z; o.w += f * v.w;
                    }
                    if (whole) {
                        join(row + 8 * a, ch * 4, o, L);
                    } else {
                        __stcg(reinterpret_cast<float4*>(part + (row + 8 * a) * D + ch * 4), o);
                        if (ch == 0) __stcg(reinterpret_cast<float2*>(part + KV4_ROWS * D) + row + 8 * a, make_float2(M, L));
                    }
                }
            }
        }
        if (!whole) {
            // CTAs that share this (request, head, tile): those between the cuts that stayed inside it
            const int64_t seg0 = cur.end - cur.left - cur.b1 - KV4_PART, share = cur.even;
            const int c0 = (int)((seg0 + SH::FIRST + share - 1) / share) - 1;
            const int c1 = (int)((seg0 + cur.q.units + KV4_PART - SH::LAST) / share);
            __syncthreads();
            if (tid == 0) {
                // releases the CTA's stores (ordered before by the barrier), acquires the other CTAs'
                int old;
                asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;" : "=r"(old) : "l"(p.counters + c0) : "memory");
                if (old == c1 - c0) p.counters[c0] = 0;
                *last_to_come = old == c1 - c0;
            }
            __syncthreads();
            if (*last_to_come) {
                // Thread groups a row wide; where there are more groups than rows, several share a
                // row's parts and their sums meet in shared memory.
                constexpr int GROUPS = KV4_THREADS / CH;
                const int tid2 = tid_again(), np = c1 - c0 + 1, ch = tid2 % CH, grp = tid2 / CH;
                const int share = max(1, GROUPS / live), rows = GROUPS / share;   // groups of a row, rows at a time
                auto slot = [&](int k) {
                    return p.partials + (2 * (c0 + k) + (k == 0 ? 1 : 0)) * (KV4_ROWS * (D + 2));
                };
#pragma unroll 1
                for (int row0 = 0; row0 < live; row0 += rows) {
                    const int row = row0 + grp / share, kk = grp % share;
                    const bool on = grp < rows * share && row < live;
                    // one pass with a running maximum: the loads of several parts are on their way together
                    float M = -FLT_MAX, L = 0.f;
                    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
                    auto add = [&](float m, float l, const float4& v) {
                        const float top = fmaxf(M, m), f = ex2f(M - top), w = ex2f(m - top);
                        M = top;
                        L = L * f + l * w;
                        o.x = o.x * f + v.x * w;
                        o.y = o.y * f + v.y * w;
                        o.z = o.z * f + v.z * w;
                        o.w = o.w * f + v.w * w;
                    };
                    if (on) {
#pragma unroll 8
                        for (int k = kk; k < np; k += share) {
                            const float* s = slot(k);
                            const float2 x = __ldcg(reinterpret_cast<const float2*>(s + KV4_ROWS * D) + row);
                            const float4 v = __ldcg(reinterpret_cast<const float4*>(s + row * D + ch * 4));
                            add(x.x, x.y, v);
                        }
                    }
                    if (share > 1) {
                        __syncthreads();
                        reinterpret_cast<float4*>(merge)[tid2] = o;
                        if (ch == 0) {
                            ml[2 * grp] = M;
                            ml[2 * grp + 1] = L;
                        }
                        __syncthreads();
                        for (int k = 1; k < share && kk == 0; ++k)
                            add(ml[2 * (grp + k)], ml[2 * (grp + k) + 1], reinterpret_cast<const float4*>(merge)[tid2 + k * CH]);
                    }
                    if (on && kk == 0) join(row, ch * 4, o, L);
                }
            }
        }
    }
    // after a wait that ran out: the copies still in flight end (or time out) before the CTA does
    if (!(flags & ALIVE)) {
        for (int s = 0; s < KV4_STAGES; ++s)
            if ((flags >> (8 + 2 * s) & 3u) != 3u) (void)mbar_wait(bars + s, flags >> s & 1u);
    }
}

}  // namespace kda
