// The recurrence and its short convolution over a tree of drafted tokens.
//
// A request's tokens form a tree behind its context (a forest: a token without
// ancestors stands directly behind the context).  Token j's mask has bit i for
// its ancestor i and bit j for itself; parents come before their children, so
// only bits up to j are looked at.
#pragma once

#include <type_traits>

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
constexpr int CONV_TREE_CH = 64;        // channel vectors of a CTA
constexpr int CONV_TREE_GROUPS = 4;     // threads of a channel vector, which share the tokens

// Shared memory of a CTA: a row for each history entry and token, and the rows
// of each token's taps.
template <typename ET, int VC> struct ConvTreeSmem {
    static constexpr int ROW = CONV_TREE_CH * VC * (int)sizeof(ET);
    static __host__ __device__ constexpr int bytes(int t) { return (CONV_KW_MAX - 1 + t) * ROW + t * 8; }
};

// silu_fast in five instructions: the exponential and the reciprocal without
// their steps for subnormal numbers, which come to the same (e^-s below 2^-126
// vanishes beside 1, and above 2^126 both divide to -0).
__device__ __forceinline__ float silu_short(float s) {
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(s * -1.4426950408889634f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
    return s * r;
}

// y_j = act(bias + sum_i weight[i] z_i) over the last KW inputs z on token j's
// path: its ancestors', and before the first of them the window's history.
// The same fmaf chain as kda_conv_kernel's (taps in ascending order, the input
// last), so that a chain gives its bits.  The window is not written: what is
// kept are the accepted tokens, which the caller passes to kda_conv_step.
//
// A CTA takes a request and 64 vectors of channels (16 bytes, or one channel)
// and loads the history and all inputs to shared memory at once, where a token
// finds its ancestors' wherever they stand; four threads a vector share the
// tokens.  A token's taps are row numbers, a byte each, worked out by one thread.
template <typename ET, int VC, int KWM>
__global__ void __launch_bounds__(CONV_TREE_CH * CONV_TREE_GROUPS) kda_conv_tree_kernel(const ConvParams p, const uint64_t* tree) {
    using IO = ConvIO<ET, VC>;
    using R = typename IO::R;
    extern __shared__ __align__(128) uint8_t smem[];
    R* rows = reinterpret_cast<R*>(smem);       // [KW - 1 + T][64]
    const int cblocks = (p.C / VC + CONV_TREE_CH - 1) / CONV_TREE_CH;
    const int cb = (int)blockIdx.x % cblocks, r = (int)blockIdx.x / cblocks;
    const int ch = threadIdx.x % CONV_TREE_CH, grp = threadIdx.x / CONV_TREE_CH, tid = threadIdx.x;
    const int c = (cb * CONV_TREE_CH + ch) * VC, KW = p.KW;
    uint64_t* taps = reinterpret_cast<uint64_t*>(rows + (KW - 1 + p.t) * CONV_TREE_CH);   // rows are multiples of 128 bytes
    cudaTriggerProgrammaticLaunchCompletion();
    cudaGridDependencySynchronize();
    int tb = r * p.t, T = p.t;
    if (p.cu != nullptr) {
        tb = __ldg(p.cu + r);
        T = __ldg(p.cu + r + 1) - tb;
    }
    const int32_t slot = __ldg(p.conv_slot + r);
    const int acc = p.accepted != nullptr ? __ldg(p.accepted + r) - 1 : 0;
    const bool rst = p.reset != nullptr && __ldg(p.reset + r) != 0, on = c < p.C;
    if (tb < 0 || T < 0 || T > p.t || tb > p.total - T) {
        if (tid == 0) atomicCAS(p.status, 0, STATUS_ARG);
        return;
    }
    if (T == 0) return;
    ET* y = static_cast<ET*>(p.y) + (int64_t)tb * p.C + c;
    float zero[VC] = {};
    if (slot < 0) {
        for (int j = grp; on && j < T; j += CONV_TREE_GROUPS) IO::st(y + (int64_t)j * p.C, IO::narrow(zero));
        return;
    }
    if (slot >= p.num_slots || acc < 0 || acc > p.L - (KW - 1)) {
        if (tid == 0) atomicCAS(p.status, 0, slot >= p.num_slots ? STATUS_SLOT_RANGE : STATUS_ARG);
        return;
    }
    if (on) {
        const ET* x = static_cast<const ET*>(p.x) + (int64_t)tb * p.C + c;
        const ET* W = static_cast<const ET*>(p.window) + (int64_t)slot * p.slot_stride + (int64_t)acc * p.C + c;
        for (int i = grp; i < KW - 1; i += CONV_TREE_GROUPS) rows[i * CONV_TREE_CH + ch] = rst ? IO::narrow(zero) : IO::ld(W + (int64_t)i * p.C);
        constexpr int U = 8;
        int j = grp;
        for (; j + (U - 1) * CONV_TREE_GROUPS < T; j += U * CONV_TREE_GROUPS) {
            R v[U];
#pragma unroll
            for (int i = 0; i < U; ++i) v[i] = IO::ld(x + (int64_t)(j + i * CONV_TREE_GROUPS) * p.C);
#pragma unroll
            for (int i = 0; i < U; ++i) rows[(KW - 1 + j + i * CONV_TREE_GROUPS) * CONV_TREE_CH + ch] = v[i];
        }
        for (; j < T; j += CONV_TREE_GROUPS) rows[(KW - 1 + j) * CONV_TREE_CH + ch] = IO::ld(x + (int64_t)j * p.C);
    }
    if (tid < T) {
        // byte i: the row of tap i
        uint64_t m = tree_mask(tree, tb + tid, tid), packed = 0;
        int hist = KW - 2;
        for (int i = KW - 1; i >= 0; --i) {
            int row = hist;
            if (m != 0) {
                const int at = tree_top(m);
                m ^= 1ull << at;
                row = KW - 1 + at;
            } else {
                --hist;
            }
            packed |= (uint64_t)row << (8 * i);
        }
        taps[tid] = packed;
    }
    // taps right-aligned: place i of KWM holds tap i - (KWM - KW)
    const int pad = KWM - KW;
    float w[KWM][VC], bias[VC];
    if (on) {
        const float* wp = p.w + (int64_t)c * KW;
        if (VC % 4 == 0 && KWM == 4 && KW == 4 && (reinterpret_cast<uintptr_t>(p.w) & 15u) == 0) {
#pragma unroll
            for (int v = 0; v < VC; ++v) {
                const float4 f = __ldg(reinterpret_cast<const float4*>(wp) + v);
                w[0][v] = f.x;
                w[1 % KWM][v] = f.y;
                w[2 % KWM][v] = f.z;
                w[3 % KWM][v] = f.w;
            }
        } else {
#pragma unroll
            for (int v = 0; v < VC; ++v)
#pragma unroll
                for (int i = 0; i < KWM; ++i) w[i][v] = i >= pad ? __ldg(wp + v * KW + i - pad) : 0.f;
        }
#pragma unroll
        for (int v = 0; v < VC; ++v) bias[v] = p.bias != nullptr ? __ldg(p.bias + c + v) : 0.f;
    }
    __syncthreads();
    if (!on) return;
    for (int j = grp; j < T; j += CONV_TREE_GROUPS) {
        const uint64_t packed = taps[j] << (8 * pad);
        R z[KWM];
#pragma unroll
        for (int i = 0; i < KWM; ++i)
            if (i >= pad) z[i] = rows[(int)(packed >> (8 * i) & 0xffu) * CONV_TREE_CH + ch];
        float s[VC];
#pragma unroll
        for (int v = 0; v < VC; ++v) s[v] = bias[v];
#pragma unroll
        for (int i = 0; i < KWM; ++i) {
            if (i < pad) continue;
            float f[VC];
            IO::widen(z[i], f);
            if constexpr (VC % 2 == 0) {    // two at a time, each as fmaf rounds
#pragma unroll
                for (int v = 0; v < VC; v += 2) {
                    const float2 t = __ffma2_rn(make_float2(w[i][v], w[i][v + 1]), make_float2(f[v], f[v + 1]), make_float2(s[v], s[v + 1]));
                    s[v] = t.x;
                    s[v + 1] = t.y;
                }
            } else {
#pragma unroll
                for (int v = 0; v < VC; ++v) s[v] = fmaf(w[i][v], f[v], s[v]);
            }
        }
        if (p.silu) {
#pragma unroll
            for (int v = 0; v < VC; ++v) s[v] = silu_short(s[v]);
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
    static __host__ __device__ constexpr int vecs(int t, int k) { return 3 * t * k * 4; }          // k, alpha, q of each token
    static __host__ __device__ constexpr int delta(int t, int warps) { return t * warps * CW * 4; }
    static __host__ __device__ constexpr int bytes(int t, int k, int warps) {
        return vecs(t, k) + delta(t, warps) + warps * 32 * 8 * 16 + t * (8 + 8 + 8 + 4);
    }
};

// One CTA: one request, one value head, `warps` times 32 bytes' worth of state
// columns.  A warp owns its columns whole: lane l holds VEC columns of the rows
// 4 (l / 2) .. + 3 and 64 more, so the sums over K are shuffles within the
// warp and nothing waits for another warp once the tokens' vectors are in
// shared memory.
//
// A token's state is S_j = diag(alpha_j) S_parent + khat_j delta_j^T with
// delta_j = beta_j (v_j - S_parent^T diag(alpha_j) khat_j), and both of its sums
// are over the parent's state, which is in registers.  Tokens are taken depth
// first: of a token's children first the leaves, whose states only pass
// through on their way out, then the first of the others, in place.  Where
// another branch begins its parent's state is built again from the initial
// state (kept on chip as it was loaded: its slot may be one of the
// snapshots') with the ancestors' deltas, which are kept: two operations an
// element and ancestor, no sums, the same bits as on the way there.  So states
// carry fp32 along every path whatever the pool's type, and do not depend on
// the order of siblings.
//
// FULL: K = V = 128, so that every lane has all its rows and columns and the
// places of a tile are constants.
template <typename ST, typename QT, bool FULL>
__global__ void __launch_bounds__(TREE_WARPS_MAX * 32, 3) kda_tree_kernel(const StepParams p, const uint64_t* tree) {
    using SV = StateVec<ST>;
    constexpr int VEC = SV::VEC, CW = 2 * VEC, NV = 2 * VEC, P2 = VEC / 2;
    extern __shared__ __align__(128) uint8_t smem[];
    const int KD = FULL ? KMAX : p.k, VD = FULL ? KMAX : p.v;
    const int warps = blockDim.x >> 5, BV = warps * CW;
    float* kh = reinterpret_cast<float*>(smem);
    float* al = kh + p.t * KD;
    float* qh = al + p.t * KD;
    float* du = qh + p.t * KD;                                             // [t][BV]: v, then delta
    uint4* stash = reinterpret_cast<uint4*>(du + p.t * BV);                 // [8][threads]
    unsigned long long* masks = reinterpret_cast<unsigned long long*>(stash + 8 * blockDim.x);
    unsigned long long* child = masks + p.t;
    float2* sc = reinterpret_cast<float2*>(child + p.t);                    // beta, khat . qhat
    int32_t* snaps = reinterpret_cast<int32_t*>(sc + p.t);

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int cblocks = (VD + BV - 1) / BV;
    const int cb = (int)blockIdx.x % cblocks, nh = (int)blockIdx.x / cblocks, n = nh / p.hv, h = nh - n * p.hv;
    for (int j = tid; j < p.t; j += blockDim.x) child[j] = 0;
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
    const int r0 = (lane >> 1) * 4;                                         // and row; its i-th is r0 + i % 4 + 64 (i / 4)
    const bool mine = c0 < VD;
    if (slot < 0) {     // a padding request
        for (int i = tid; i < T * BV; i += blockDim.x) {
            const int j = i / BV, c = cb * BV + i - j * BV;
            if (c < VD) p.o[((int64_t)(tb + j) * p.hv + h) * VD + c] = 0.f;
        }
        return;
    }
    const bool rst = p.reset != nullptr && __ldg(p.reset + n) != 0;
    // half 0 and half 1 of the lane's rows are in the state
    const bool live[2] = {FULL || (mine && r0 < KD), FULL || (mine && r0 + 64 < KD)};
    ST* pool = static_cast<ST*>(p.pool);
    const int64_t tile = (int64_t)r0 * VD + c0;
    auto at_row = [&](int i) { return (int64_t)((i & 3) + 64 * (i >> 2)) * VD; };
    uint4 raw[8];
    {
        const ST* from = pool + state_at(p, slot, h) + tile;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            raw[i] = live[i >> 2] && !rst ? *reinterpret_cast<const uint4*>(from + at_row(i)) : make_uint4(0, 0, 0, 0);
    }
    __syncthreads();    // child is zero
    // ---- the tokens' vectors, a token a warp at a time ----
    const int hq = h / (p.hv / p.hqk);
    const bool scaled = p.a_log != nullptr;
    const float gate = scaled ? expf(__ldg(p.a_log + h)) : 1.f;
    constexpr int AHEAD = 4;        // tokens whose loads a warp has on their way
    const int d = 4 * lane;
    const bool on = d < KD;
    float bias[4] = {};
    if (on && scaled && p.dt_bias != nullptr) {
#pragma unroll
        for (int e = 0; e < 4; ++e) bias[e] = __ldg(p.dt_bias + h * KD + d + e);
    }
    using QIO = ConvIO<QT, 4>;
    for (int j0 = warp; j0 < T; j0 += AHEAD * warps) {
        typename QIO::R kr[AHEAD], qr[AHEAD];
        float4 ar[AHEAD];
        float br[AHEAD], vr[AHEAD], vr2[AHEAD];      // a CTA has at most 64 columns
        static_assert(TREE_WARPS_MAX * CW <= 64, "columns");
        unsigned long long mr[AHEAD];
#pragma unroll
        for (int x = 0; x < AHEAD; ++x) {
            const int j = min(j0 + x * warps, T - 1);
            const int64_t tok = tb + j, at = (tok * p.hqk + hq) * KD + (on ? d : 0);
            kr[x] = QIO::ld(static_cast<const QT*>(p.kk) + at);
            qr[x] = QIO::ld(static_cast<const QT*>(p.q) + at);
            ar[x] = __ldg(reinterpret_cast<const float4*>(p.a + (tok * p.hv + h) * KD + (on ? d : 0)));
            br[x] = __ldg(p.b + tok * p.hv + h);
            mr[x] = tree_mask(tree, tok, j) ^ (1ull << j);
const QT* vt = static_cast<const QT*>(p.vv) + (tok * p.hv + h) * VD + cb * BV + lane;
            vr[x] = lane < BV && cb * BV + lane < VD ? to_f32(vt[0]) : 0.f;
            vr2[x] = lane + 32 < BV && cb * BV + lane + 32 < VD ? to_f32(vt[32]) : 0.f;
        }
        // step by step for all of them, so that their latencies overlap; behind the last token it is done again
        float k4[AHEAD][4], q4[AHEAD][4], kk[AHEAD], qq[AHEAD], kq[AHEAD];
#pragma unroll
        for (int x = 0; x < AHEAD; ++x) {
            QIO::widen(kr[x], k4[x]);
            QIO::widen(qr[x], q4[x]);
            kk[x] = qq[x] = kq[x] = 0.f;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (!on) k4[x][e] = q4[x][e] = 0.f;
                kk[x] = fmaf(k4[x][e], k4[x][e], kk[x]);
                qq[x] = fmaf(q4[x][e], q4[x][e], qq[x]);
                kq[x] = fmaf(k4[x][e], q4[x][e], kq[x]);
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
#pragma unroll
            for (int x = 0; x < AHEAD; ++x) {
                kk[x] += __shfl_xor_sync(0xffffffffu, kk[x], o);
                qq[x] += __shfl_xor_sync(0xffffffffu, qq[x], o);
                kq[x] += __shfl_xor_sync(0xffffffffu, kq[x], o);
            }
        float g[AHEAD][4];
        if (scaled) {       // one branch for all
#pragma unroll
            for (int x = 0; x < AHEAD; ++x) {
                const float a[4] = {ar[x].x, ar[x].y, ar[x].z, ar[x].w};
#pragma unroll
                for (int e = 0; e < 4; ++e) g[x][e] = gate_alpha(a[e], true, gate, bias[e]);
            }
        } else {
#pragma unroll
            for (int x = 0; x < AHEAD; ++x) {
                const float a[4] = {ar[x].x, ar[x].y, ar[x].z, ar[x].w};
#pragma unroll
                for (int e = 0; e < 4; ++e) g[x][e] = gate_alpha(a[e], false, gate, bias[e]);
            }
        }
#pragma unroll
        for (int x = 0; x < AHEAD; ++x) {
            const int j = min(j0 + x * warps, T - 1);
            const float rk = __frsqrt_rn(kk[x] + L2_EPS), rq = __frsqrt_rn(qq[x] + L2_EPS);
            if (FULL || on) {
                *reinterpret_cast<float4*>(kh + j * KD + d) = make_float4(k4[x][0] * rk, k4[x][1] * rk, k4[x][2] * rk, k4[x][3] * rk);
                *reinterpret_cast<float4*>(qh + j * KD + d) = make_float4(q4[x][0] * rq, q4[x][1] * rq, q4[x][2] * rq, q4[x][3] * rq);
                *reinterpret_cast<float4*>(al + j * KD + d) = make_float4(g[x][0], g[x][1], g[x][2], g[x][3]);
            }
            if (lane < BV) du[j * BV + lane] = vr[x];
            if (lane + 32 < BV) du[j * BV + lane + 32] = vr2[x];
            if (lane == 0) {
                sc[j] = make_float2(sigmoid_neg(-br[x]), kq[x] * rk * rq);
                masks[j] = mr[x];
                if (mr[x] != 0) atomicOr(child + tree_top(mr[x]), 1ull << j);
            }
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
    // 0 for the sum with khat and 1 for the one with qhat, bit 0 the column half
    constexpr int SB = VEC == 4 ? 2 : 1;
    const int vc = lane >> (SB + 1), second = lane >> SB & 1;
    const int my_col = warp * CW + (lane & 1) * VEC + vc;
    const bool first_of = VEC == 8 || (lane & 2) == 0, live_col = cb * BV + my_col < VD && first_of;
    // a lane without rows there reads other rows', and k as zero: its states stay zero
    const int at0 = r0 < KD ? r0 : 0, at1 = r0 + 64 < KD ? r0 + 64 : 0;
    auto vec8 = [&](const float* v, int j, float (&x)[8]) {
        const float4 lo = *reinterpret_cast<const float4*>(v + j * KD + at0), hi = *reinterpret_cast<const float4*>(v + j * KD + at1);
        x[0] = lo.x; x[1] = lo.y; x[2] = lo.z; x[3] = lo.w;
        x[4] = hi.x; x[5] = hi.y; x[6] = hi.z; x[7] = hi.w;
    };
    auto key8 = [&](int j, float (&x)[8]) {
        vec8(kh, j, x);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (!FULL && r0 + 64 * (i >> 2) >= KD) x[i] = 0.f;
    };
    auto deltas = [&](int j, float2 (&d)[P2]) {
#pragma unroll
        for (int x = 0; x < P2; x += 2) {
            const float4 f = *reinterpret_cast<const float4*>(du + j * BV + warp * CW + (lane & 1) * VEC + 2 * x);
            d[x] = make_float2(f.x, f.y);
            d[x + 1] = make_float2(f.z, f.w);
        }
    };
    // S <- diag(alpha_i) S + khat_i delta_i^T of an earlier token
    auto again = [&](int i) {
        float a[8], k[8];
        float2 d[P2];
        vec8(al, i, a);
        key8(i, k);
        deltas(i, d);
#pragma unroll
        for (int r = 0; r < 8; ++r)
#pragma unroll
            for (int x = 0; x < P2; ++x) S[r][x] = __ffma2_rn(make_float2(k[r], k[r]), d[x], __fmul2_rn(S[r][x], make_float2(a[r], a[r])));
    };
    // Tokens j[0 .. N), children of the token whose state S is: their outputs, and their deltas to du.  Step by step
    // for all of them, so that their latencies overlap.
    auto sums = [&](auto n_of, const int* j) {
        constexpr int N = decltype(n_of)::value;
        float f[N][NV], v[N];
        float2 bs[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float a[8], k[8], q[8];
            vec8(al, j[i], a);
            vec8(kh, j[i], k);
            vec8(qh, j[i], q);
            v[i] = du[j[i] * BV + my_col];
            bs[i] = sc[j[i]];
            float2 su[P2], sq[P2];
#pragma unroll
            for (int x = 0; x < P2; ++x) su[x] = sq[x] = make_float2(0.f, 0.f);
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                const float ak = a[r] * k[r], aq = a[r] * q[r];
#pragma unroll
                for (int x = 0; x < P2; ++x) {
                    su[x] = __ffma2_rn(S[r][x], make_float2(ak, ak), su[x]);
                    sq[x] = __ffma2_rn(S[r][x], make_float2(aq, aq), sq[x]);
                }
            }
#pragma unroll
            for (int x = 0; x < P2; ++x) {
                f[i][4 * x] = su[x].x;
                f[i][4 * x + 1] = sq[x].x;
                f[i][4 * x + 2] = su[x].y;
                f[i][4 * x + 3] = sq[x].y;
            }
        }
        // over the 16 row groups (lane bits 4 .. 1), scattered: value 2 c + s of column c
        int m = 16;
#pragma unroll
        for (int cnt = NV; cnt > 1; cnt >>= 1, m >>= 1) {
            const bool upper = (lane & m) != 0;
#pragma unroll
            for (int x = 0; x < cnt / 2; ++x)
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const float send = upper ? f[i][x] : f[i][x + cnt / 2], keep = upper ? f[i][x + cnt / 2] : f[i][x];
                    f[i][x] = keep + __shfl_xor_sync(0xffffffffu, send, m);
                }
        }
        if constexpr (VEC == 4) {
#pragma unroll
            for (int i = 0; i < N; ++i) f[i][0] += __shfl_xor_sync(0xffffffffu, f[i][0], 2);
        }
        float other[N];
#pragma unroll
        for (int i = 0; i < N; ++i) other[i] = __shfl_xor_sync(0xffffffffu, f[i][0], 1 << SB);
        __syncwarp();       // v is read
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float u = second ? other[i] : f[i][0], pq = second ? f[i][0] : other[i], delta = bs[i].x * (v[i] - u);
            if (!second && first_of) du[j[i] * BV + my_col] = delta;
            if (second && live_col) p.o[((int64_t)(tb + j[i]) * p.hv + h) * VD + cb * BV + my_col] = fmaf(bs[i].y, delta, pq) * p.inv_sqrt_k;
        }
        __syncwarp();
    };
    // Token j's state, from its parent's in S, to its snapshot; keep: and to S.
    auto store = [&](int j, bool keep) {
        float a[8], k[8];
        float2 d[P2];
        vec8(al, j, a);
        key8(j, k);
        deltas(j, d);
        const int32_t snap = snaps[j];
        ST* to = pool + state_at(p, snap, h) + tile;
        if (keep) {
#pragma unroll
            for (int r = 0; r < 8; ++r) {
#pragma unroll
                for (int x = 0; x < P2; ++x) S[r][x] = __ffma2_rn(make_float2(k[r], k[r]), d[x], __fmul2_rn(S[r][x], make_float2(a[r], a[r])));
                if (snap >= 0 && live[r >> 2]) *reinterpret_cast<uint4*>(to + at_row(r)) = SV::narrow2(S[r]);
            }
        } else if (snap >= 0) {
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                float2 out[P2];
#pragma unroll
                for (int x = 0; x < P2; ++x) out[x] = __ffma2_rn(make_float2(k[r], k[r]), d[x], __fmul2_rn(S[r][x], make_float2(a[r], a[r])));
                if (live[r >> 2]) *reinterpret_cast<uint4*>(to + at_row(r)) = SV::narrow2(out);
            }
        }
    };
    // ---- depth first ----
    unsigned long long todo, leaves, kids;      // kids: of the token whose state S is (at first the context)
    {
        const bool in0 = lane < T, in1 = lane + 32 < T;
        auto both = [&](bool b0, bool b1) {
            return __ballot_sync(0xffffffffu, b0) | (unsigned long long)__ballot_sync(0xffffffffu, b1) << 32;
        };
        todo = both(in0, in1);
        leaves = both(in0 && child[lane] == 0, in1 && child[lane + 32] == 0);
        kids = both(in0 && masks[lane] == 0, in1 && masks[lane + 32] == 0);
    }
    while (todo != 0) {
        kids &= todo;
        if (kids == 0) {
            // another branch: the lowest token left, whose parent is done
            const int j = __ffsll((long long)todo) - 1;
#pragma unroll
            for (int i = 0; i < 8; ++i) SV::widen2(stash[i * blockDim.x + tid], S[i]);
            const unsigned long long above = masks[j];
            for (unsigned long long m = above; m != 0; m &= m - 1) again(__ffsll((long long)m) - 1);
            kids = above != 0 ? child[tree_top(above)] & todo : 1ull << j;
        }
        // leaves two at a time, then an inner child; a leaf and the inner child go together too
        const unsigned long long ends = kids & leaves, inner = kids & ~leaves;
        int j[2];
        j[0] = __ffsll((long long)(ends != 0 ? ends : inner)) - 1;
        const unsigned long long left = ends & (ends - 1);
        const bool down = ends == 0 || (left == 0 && inner != 0);       // the last of this token's children that are taken from S
        j[1] = left != 0 ? __ffsll((long long)left) - 1 : inner != 0 && ends != 0 ? __ffsll((long long)inner) - 1 : -1;
        if (j[1] >= 0) {
            sums(std::integral_constant<int, 2>{}, j);
            store(j[0], false);
            store(j[1], down);
            todo &= ~(1ull << j[1]);
        } else {
            sums(std::integral_constant<int, 1>{}, j);
            store(j[0], down);
        }
        todo &= ~(1ull << j[0]);
        if (down) kids = child[j[1] >= 0 ? j[1] : j[0]];
    }
}

}  // namespace kda
