// The recurrence and its short convolution over a tree of drafted tokens.
//
// A request's tokens form a tree behind its context (a forest: a token without
// ancestors stands directly behind the context).  Token j's mask has bit i for
// its ancestor i and bit j for itself; parents come before their children, so
// only bits up to j are looked at.
#pragma once

#include "kda_common.cuh"
#include "kda_conv.cuh"

namespace kda {

constexpr int TREE_MAX = 64;     // tokens of a request: the bits of a mask

// Token j's ancestors and itself; without masks a chain.
__device__ __forceinline__ uint64_t tree_mask(const uint64_t* tree, int64_t row, int j) {
    const uint64_t self = 1ull << j, below = self - 1;
    return ((tree != nullptr ? __ldg(reinterpret_cast<const unsigned long long*>(tree + row)) : below) & below) | self;
}
// The highest token of a mask; the mask is not zero.
__device__ __forceinline__ int tree_top(uint64_t m) { return 63 - __clzll((long long)m); }

// ---------------------------------------------------------------------------
// Convolution
// ---------------------------------------------------------------------------
constexpr int CONV_TREE_THREADS = 64;

// y_j = act(bias + sum_i weight[i] z_i) over the last KW inputs z on token j's
// path: its ancestors', and before the first of them the window's history.
// The same fmaf chain as kda_conv_kernel's (taps in ascending order, the input
// last), so that a chain gives its bits.  The window is not written: what is
// kept are the accepted tokens, which the caller passes to kda_conv_step.
//
// VC channels a thread (16 bytes, or 1), `chunk` tokens of a request a CTA, the
// weights and the history loaded once for them; an ancestor's row comes out of
// L1 or L2.
template <typename ET, int VC, int KWM>
__global__ void __launch_bounds__(CONV_TREE_THREADS) kda_conv_tree_kernel(const ConvParams p, const uint64_t* tree, int chunk) {
    using IO = ConvIO<ET, VC>;
    using R = typename IO::R;
    const int cblocks = (p.C / VC + CONV_TREE_THREADS - 1) / CONV_TREE_THREADS, chunks = (p.t + chunk - 1) / chunk;
    const int cb = (int)blockIdx.x % cblocks, rc = (int)blockIdx.x / cblocks, r = rc / chunks, j0 = (rc - r * chunks) * chunk;
    const int c = (cb * CONV_TREE_THREADS + (int)threadIdx.x) * VC;
    cudaTriggerProgrammaticLaunchCompletion();
    cudaGridDependencySynchronize();
    if (c >= p.C) return;
    int tb = r * p.t, T = p.t;
    if (p.cu != nullptr) {
        tb = __ldg(p.cu + r);
        T = __ldg(p.cu + r + 1) - tb;
    }
    const int32_t slot = __ldg(p.conv_slot + r);
    const int acc = p.accepted != nullptr ? __ldg(p.accepted + r) - 1 : 0, KW = p.KW;
    const bool rst = p.reset != nullptr && __ldg(p.reset + r) != 0;
    if (tb < 0 || T < 0 || T > p.t || tb > p.total - T) {
        if (threadIdx.x == 0) atomicCAS(p.status, 0, STATUS_ARG);
        return;
    }
    const int j1 = min(T, j0 + chunk);
    if (j0 >= j1) return;
    ET* y = static_cast<ET*>(p.y) + (int64_t)tb * p.C + c;
    if (slot < 0) {
        float zero[VC] = {};
        for (int j = j0; j < j1; ++j) IO::st(y + (int64_t)j * p.C, IO::narrow(zero));
        return;
    }
    if (slot >= p.num_slots || acc < 0 || acc > p.L - (KW - 1)) {
        if (threadIdx.x == 0) atomicCAS(p.status, 0, slot >= p.num_slots ? STATUS_SLOT_RANGE : STATUS_ARG);
        return;
    }
    const ET* x = static_cast<const ET*>(p.x) + (int64_t)tb * p.C + c;
    const ET* W = static_cast<const ET*>(p.window) + (int64_t)slot * p.slot_stride + (int64_t)acc * p.C + c;
    // taps right-aligned: place i of KWM holds tap i - (KWM - KW)
    const int pad = KWM - KW;
    float w[KWM][VC], bias[VC];
    R hist[KWM - 1], none;
    {
        float zero[VC] = {};
        none = IO::narrow(zero);
    }
#pragma unroll
    for (int i = 0; i < KWM - 1; ++i) hist[i] = i >= pad && !rst ? IO::ld(W + (int64_t)(i - pad) * p.C) : none;
#pragma unroll
    for (int v = 0; v < VC; ++v) {
        bias[v] = p.bias != nullptr ? __ldg(p.bias + c + v) : 0.f;
#pragma unroll
        for (int i = 0; i < KWM; ++i) w[i][v] = i >= pad ? __ldg(p.w + (int64_t)(c + v) * KW + i - pad) : 0.f;
    }
    for (int j = j0; j < j1; ++j) {
        uint64_t m = tree_mask(tree, tb + j, j);
        R z[KWM];
#pragma unroll
        for (int i = KWM - 1; i >= 0; --i) {
            // m == 0: the place KWM - 1 - d lies d - (tokens on the path) before the history's end; both
            // the path's length and the place are the CTA's, and the select has constant indexes
            if (m != 0) {
                const int at = tree_top(m);
                m ^= 1ull << at;
                z[i] = i >= pad ? IO::ld(x + (int64_t)at * p.C) : none;
            } else {
                z[i] = none;
            }
        }
        const int depth = min(KWM, __popcll(tree_mask(tree, tb + j, j)));   // places that the path fills
        // place i < KWM - depth: history entry i + depth - 1 of the right-aligned KWM - 1
#pragma unroll
        for (int i = 0; i < KWM - 1; ++i)
#pragma unroll
            for (int d = 1; d < KWM - i; ++d)
                if (depth == d) z[i] = hist[i + d - 1];
        float s[VC];
#pragma unroll
        for (int v = 0; v < VC; ++v) s[v] = bias[v];
#pragma unroll
        for (int i = 0; i < KWM; ++i) {
            if (i < pad) continue;
            float f[VC];
            IO::widen(z[i], f);
#pragma unroll
            for (int v = 0; v < VC; ++v) s[v] = fmaf(w[i][v], f[v], s[v]);
        }
        if (p.silu) {
#pragma unroll
            for (int v = 0; v < VC; ++v) s[v] = silu_fast(s[v]);
        }
        IO::st(y + (int64_t)j * p.C, IO::narrow(s));
    }
}

// ---------------------------------------------------------------------------
// Recurrence
// ---------------------------------------------------------------------------
constexpr int TREE_WARPS_MAX = 4;

// Shared memory of a CTA of `warps` warps with at most t tokens a request.
template <typename ST> struct TreeSmem {
    static constexpr int VEC = StateVec<ST>::VEC, CW = 2 * VEC;   // columns of a lane, of a warp
    static __host__ __device__ constexpr int vecs(int t) { return 3 * t * KMAX * 4; }              // k, alpha, q of each token
    static __host__ __device__ constexpr int delta(int t, int warps) { return t * warps * CW * 4; }
    static __host__ __device__ constexpr int bytes(int t, int warps) {
        return vecs(t) + delta(t, warps) + warps * 32 * 8 * 16 + t * (8 + 8 + 4) + 16;
    }
};

// One CTA: one request, one value head, `warps` times 32 bytes' worth of state
// columns.  A warp owns its columns whole: lane l holds rows 8 (l / 2) .. + 7
// of VEC columns, so the sums over K are shuffles within the warp and nothing
// waits for another warp once the tokens' vectors are in shared memory.
//
// A token's state is S_j = diag(alpha_j) S_parent + khat_j delta_j^T with
// delta_j = beta_j (v_j - S_parent^T diag(alpha_j) khat_j).  Token j - 1's
// state is in registers; where that is j's parent, j goes on from it.  Else the
// parent's is built again from the initial state (kept on chip as it was
// loaded: its slot may be one of the snapshots') with the ancestors' deltas,
// which are kept: two operations an element and ancestor, no sums, the same
// bits as on the way there.  So states carry fp32 along every path whatever
// the pool's type, and siblings do not depend on their order.
template <typename ST, typename QT>
__global__ void __launch_bounds__(TREE_WARPS_MAX * 32) kda_tree_kernel(const StepParams p, const uint64_t* tree) {
    using SV = StateVec<ST>;
    constexpr int VEC = SV::VEC, CW = 2 * VEC, NV = 2 * VEC, P2 = VEC / 2;
    extern __shared__ __align__(16) uint8_t smem[];
    const int warps = blockDim.x >> 5, BV = warps * CW;
    float* kh = reinterpret_cast<float*>(smem);
    float* al = kh + p.t * KMAX;
    float* qh = al + p.t * KMAX;
    float* du = qh + p.t * KMAX;                                            // [t][BV]
    uint4* stash = reinterpret_cast<uint4*>(du + p.t * BV);                 // [8][threads]
    uint64_t* masks = reinterpret_cast<uint64_t*>(stash + 8 * blockDim.x);
    float2* sc = reinterpret_cast<float2*>(masks + p.t);                    // beta, khat . qhat
    int32_t* snaps = reinterpret_cast<int32_t*>(sc + p.t);

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int cblocks = (p.v + BV - 1) / BV;
    const int cb = (int)blockIdx.x % cblocks, nh = (int)blockIdx.x / cblocks, n = nh / p.hv, h = nh - n * p.hv;
    cudaTriggerProgrammaticLaunchCompletion();
    cudaGridDependencySynchronize();
    int tb = n * p.t, T = p.t;
    if (p.cu != nullptr) {
        tb = __ldg(p.cu + n);
        T = __ldg(p.cu + n + 1) - tb;
    }
    const int col = p.accepted != nullptr ? __ldg(p.accepted + n) - 1 : 0;
    bool ok = tb >= 0 && T >= 0 && T <= p.t && tb <= p.total - T;
    if (ok && T == 0) return;
    ok = ok && col >= 0 && col < p.num_cols;
    if (!ok) {
        if (tid == 0) atomicCAS(p.status, 0, STATUS_ARG);
        return;
    }
    const int32_t* row = p.snap_slot + (int64_t)n * p.snap_stride;
    const int32_t slot = __ldg(row + col);
    bool range = slot >= p.num_slots;
    for (int j = lane; j < T; j += 32) {
        const int32_t s = __ldg(row + j);
        if (warp == 0) snaps[j] = s;
        range |= s >= p.num_slots;
    }
    if (__any_sync(0xffffffffu, range)) {
        if (tid == 0) atomicCAS(p.status, 0, STATUS_SLOT_RANGE);
        return;
    }
    const int c0 = cb * BV + warp * CW + (lane & 1) * VEC;                  // the lane's first column
    const int r0 = (lane >> 1) * 8;                                         // and row
    const bool mine = c0 < p.v;
    if (slot < 0) {     // a padding request
        for (int i = tid; i < T * BV; i += blockDim.x) {
            const int j = i / BV, c = cb * BV + i - j * BV;
            if (c < p.v) p.o[((int64_t)(tb + j) * p.hv + h) * p.v + c] = 0.f;
        }
        return;
    }
    const bool rst = p.reset != nullptr && __ldg(p.reset + n) != 0;
    ST* pool = static_cast<ST*>(p.pool);
    const int64_t tile = (int64_t)r0 * p.v + c0;
    uint4 raw[8];
    {
        const ST* from = pool + state_at(p, slot, h) + tile;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            raw[i] = mine && !rst && r0 + i < p.k ? *reinterpret_cast<const uint4*>(from + (int64_t)i * p.v) : make_uint4(0, 0, 0, 0);
    }
    // ---- the tokens' vectors, a token a warp at a time ----
    const int hq = h / (p.hv / p.hqk);
    const bool scaled = p.a_log != nullptr;
    const float gate = scaled ? expf(__ldg(p.a_log + h)) : 1.f;
    for (int j = warp; j < T; j += warps) {
        const int d = 4 * lane;
        const bool on = d < p.k;
        const int64_t at = ((int64_t)(tb + j) * p.hqk + hq) * p.k + d;
        float k4[4] = {}, q4[4] = {};
        float4 a4 = make_float4(0.f, 0.f, 0.f, 0.f);
        if (on) {
            ConvIO<QT, 4>::widen(ConvIO<QT, 4>::ld(static_cast<const QT*>(p.kk) + at), k4);
            ConvIO<QT, 4>::widen(ConvIO<QT, 4>::ld(static_cast<const QT*>(p.q) + at), q4);
            a4 = __ldg(reinterpret_cast<const float4*>(p.a + ((int64_t)(tb + j) * p.hv + h) * p.k + d));
        }
        float kk = 0.f, qq = 0.f, kq = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            kk = fmaf(k4[e], k4[e], kk);
            qq = fmaf(q4[e], q4[e], qq);
            kq = fmaf(k4[e], q4[e], kq);
        }
        kk = warp_sum(kk);
        qq = warp_sum(qq);
        kq = warp_sum(kq);
        const float rk = __frsqrt_rn(kk + L2_EPS), rq = __frsqrt_rn(qq + L2_EPS);
        float bias[4] = {};
        if (on && scaled && p.dt_bias != nullptr) {
#pragma unroll
            for (int e = 0; e < 4; ++e) bias[e] = __ldg(p.dt_bias + h * p.k + d + e);
        }
        const float a[4] = {a4.x, a4.y, a4.z, a4.w};
        float g[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) g[e] = gate_alpha(a[e], scaled, gate, bias[e]);
        *reinterpret_cast<float4*>(kh + j * KMAX + d) = make_float4(k4[0] * rk, k4[1] * rk, k4[2] * rk, k4[3] * rk);
        *reinterpret_cast<float4*>(qh + j * KMAX + d) = make_float4(q4[0] * rq, q4[1] * rq, q4[2] * rq, q4[3] * rq);
        *reinterpret_cast<float4*>(al + j * KMAX + d) = make_float4(g[0], g[1], g[2], g[3]);
        if (lane == 0) {
            sc[j] = make_float2(sigmoid_neg(-__ldg(p.b + (int64_t)(tb + j) * p.hv + h)), kq * rk * rq);
            masks[j] = tree_mask(tree, tb + j, j);
        }
    }
    float2 S[8][P2];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        SV::widen2(raw[i], S[i]);
        stash[i * blockDim.x + tid] = raw[i];
    }
    __syncthreads();

    // which of the warp's sums this lane ends up with: lane bits 4.. down to SB count columns, bit SB is
    // 0 for S^T khat and 1 for S^T qhat, bit 0 the column half
    constexpr int SB = VEC == 4 ? 2 : 1;
    const int vc = lane >> (SB + 1), second = lane >> SB & 1;
    const int my_col = cb * BV + warp * CW + (lane & 1) * VEC + vc;
    const bool live_col = my_col < p.v;
    const QT* vv = static_cast<const QT*>(p.vv) + ((int64_t)tb * p.hv + h) * p.v + my_col;
    const int64_t v_step = (int64_t)p.hv * p.v;
    float v_next = live_col ? to_f32(vv[0]) : 0.f;
    // S <- diag(alpha_i) S + khat_i delta_i^T of an earlier token
    auto again = [&](int i) {
        const float4 a0 = *reinterpret_cast<const float4*>(al + i * KMAX + r0), a1 = *reinterpret_cast<const float4*>(al + i * KMAX + r0 + 4);
        const float4 k0 = *reinterpret_cast<const float4*>(kh + i * KMAX + r0), k1 = *reinterpret_cast<const float4*>(kh + i * KMAX + r0 + 4);
        const float a[8] = {a0.x, a0.y, a0.z, a0.w, a1.x, a1.y, a1.z, a1.w};
        const float k[8] = {k0.x, k0.y, k0.z, k0.w, k1.x, k1.y, k1.z, k1.w};
        float2 d[P2];
#pragma unroll
        for (int x = 0; x < P2; ++x) d[x] = *reinterpret_cast<const float2*>(du + i * BV + warp * CW + (lane & 1) * VEC + 2 * x);
#pragma unroll
        for (int r = 0; r < 8; ++r)
#pragma unroll
            for (int x = 0; x < P2; ++x) S[r][x] = __ffma2_rn(make_float2(k[r], k[r]), d[x], __fmul2_rn(S[r][x], make_float2(a[r], a[r])));
    };
    for (int j = 0; j < T; ++j) {
        uint64_t above = masks[j] ^ (1ull << j);
        if (j > 0 && above != masks[j - 1]) {
#pragma unroll
            for (int i = 0; i < 8; ++i) SV::widen2(stash[i * blockDim.x + tid], S[i]);
            for (; above != 0; above &= above - 1) again(__ffsll((long long)above) - 1);
        }
        const float v_now = v_next;
        if (j + 1 < T && live_col) v_next = to_f32(vv[(j + 1) * v_step]);
        const float4 a0 = *reinterpret_cast<const float4*>(al + j * KMAX + r0), a1 = *reinterpret_cast<const float4*>(al + j * KMAX + r0 + 4);
        const float4 k0 = *reinterpret_cast<const float4*>(kh + j * KMAX + r0), k1 = *reinterpret_cast<const float4*>(kh + j * KMAX + r0 + 4);
        const float4 q0 = *reinterpret_cast<const float4*>(qh + j * KMAX + r0), q1 = *reinterpret_cast<const float4*>(qh + j * KMAX + r0 + 4);
        const float a[8] = {a0.x, a0.y, a0.z, a0.w, a1.x, a1.y, a1.z, a1.w};
        const float k[8] = {k0.x, k0.y, k0.z, k0.w, k1.x, k1.y, k1.z, k1.w};
        const float q[8] = {q0.x, q0.y, q0.z, q0.w, q1.x, q1.y, q1.z, q1.w};
        float2 su[P2], sq[P2];
#pragma unroll
        for (int x = 0; x < P2; ++x) su[x] = sq[x] = make_float2(0.f, 0.f);
#pragma unroll
        for (int r = 0; r < 8; ++r)
#pragma unroll
            for (int x = 0; x < P2; ++x) {
                S[r][x] = __fmul2_rn(S[r][x], make_float2(a[r], a[r]));
                su[x] = __ffma2_rn(S[r][x], make_float2(k[r], k[r]), su[x]);
                sq[x] = __ffma2_rn(S[r][x], make_float2(q[r], q[r]), sq[x]);
            }
        // sums over the 16 row groups (lane bits 4 .. 1), scattered: value 2 c + s of column c
        float f[NV];
#pragma unroll
        for (int x = 0; x < P2; ++x) {
            f[4 * x] = su[x].x;
            f[4 * x + 1] = sq[x].x;
            f[4 * x + 2] = su[x].y;
            f[4 * x + 3] = sq[x].y;
        }
        int m = 16;
#pragma unroll
        for (int cnt = NV; cnt > 1; cnt >>= 1, m >>= 1) {
            const bool upper = (lane & m) != 0;
#pragma unroll
            for (int x = 0; x < cnt / 2; ++x) {
                const float send = upper ? f[x] : f[x + cnt / 2], keep = upper ? f[x + cnt / 2] : f[x];
                f[x] = keep + __shfl_xor_sync(0xffffffffu, send, m);
            }
        }
        if constexpr (VEC == 4) f[0] += __shfl_xor_sync(0xffffffffu, f[0], 2);
        const float other = __shfl_xor_sync(0xffffffffu, f[0], 1 << SB);
        const float u = second ? other : f[0], pq = second ? f[0] : other;
        const float2 bs = sc[j];
        const float delta = bs.x * (v_now - u);
        if (!second && (VEC == 8 || (lane & 2) == 0)) du[j * BV + warp * CW + (lane & 1) * VEC + vc] = delta;
        if (second && live_col && (VEC == 8 || (lane & 2) == 0))
            p.o[((int64_t)(tb + j) * p.hv + h) * p.v + my_col] = fmaf(bs.y, delta, pq) * p.inv_sqrt_k;
        __syncwarp();
        float2 d[P2];
#pragma unroll
        for (int x = 0; x < P2; ++x) d[x] = *reinterpret_cast<const float2*>(du + j * BV + warp * CW + (lane & 1) * VEC + 2 * x);
        const int32_t snap = snaps[j];
        ST* to = pool + state_at(p, snap, h) + tile;
#pragma unroll
        for (int r = 0; r < 8; ++r) {
#pragma unroll
            for (int x = 0; x < P2; ++x) S[r][x] = __ffma2_rn(make_float2(k[r], k[r]), d[x], S[r][x]);
            if (snap >= 0 && mine && r0 + r < p.k) *reinterpret_cast<uint4*>(to + (int64_t)r * p.v) = SV::narrow2(S[r]);
        }
    }
}

}  // namespace kda
