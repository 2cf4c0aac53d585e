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
constexpr int CONV_TREE_CH = 32;        // channel vectors of a CTA
constexpr int CONV_TREE_GROUPS = 4;     // threads of a channel vector, which share the tokens

// Shared memory of a CTA: a row for each history entry and token, and the rows
// of each token's taps.
template <typename ET, int VC> struct ConvTreeSmem {
    static constexpr int ROW = CONV_TREE_CH * VC * (int)sizeof(ET);
    static constexpr int WEIGHTS = CONV_TREE_CH * VC * 16;       // four taps a channel
    static __host__ __device__ constexpr int bytes(int t) { return WEIGHTS + (CONV_KW_MAX - 1 + t) * ROW + t * 8; }
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
// A CTA takes a request and 32 vectors of channels (16 bytes, or one channel)
// and loads the history and all inputs to shared memory at once, where a token
// finds its ancestors' wherever they stand; four threads a vector share the
// tokens.  A token's taps are row numbers, a byte each, worked out by one thread.
//
// Measured: 32 requests of 64 tokens, 4608 bf16 channels, 15.0 us, where its 39
// MB take 5.7 us at the copy rate: a CTA's loads all go out before its first
// sum and its stores come after, so memory waits for the sums and the sums for
// memory (issue slots in use in 37 of 100 cycles).  1 x 8 tokens: 3.1 us in a
// graph, 9.5 to 11 through a call.  Vectors by threads of each, the first size: 64 x 4
// 15.1, 64 x 2 20.4.  Every tap loaded from global memory as it is needed: 39;
// weights fetched a channel a thread and rows through registers: 18.5.
template <typename ET, int VC, int KWM>
__global__ void __launch_bounds__(CONV_TREE_CH * CONV_TREE_GROUPS) kda_conv_tree_kernel(const ConvParams p, const uint64_t* tree) {
    using IO = ConvIO<ET, VC>;
    using R = typename IO::R;
    extern __shared__ __align__(128) uint8_t smem[];
    float4* wide = reinterpret_cast<float4*>(smem);     // [vectors][VC]: a channel's four taps, at their place xor the vector's
    R* rows = reinterpret_cast<R*>(smem + ConvTreeSmem<ET, VC>::WEIGHTS);       // [KW - 1 + T][vectors]
    const int cblocks = (p.C / VC + CONV_TREE_CH - 1) / CONV_TREE_CH;
    const int cb = (int)blockIdx.x % cblocks, r = (int)blockIdx.x / cblocks;
    const int ch = threadIdx.x % CONV_TREE_CH, grp = threadIdx.x / CONV_TREE_CH, tid = threadIdx.x;
    const int c = (cb * CONV_TREE_CH + ch) * VC, KW = p.KW;
    uint64_t* taps = reinterpret_cast<uint64_t*>(rows + (KW - 1 + p.t) * CONV_TREE_CH);
    cudaTriggerProgrammaticLaunchCompletion();
    cudaGridDependencySynchronize();
    // a channel's weights are 16 bytes: fetched in order, read back by vector
    const bool four = VC % 4 == 0 && KWM == 4 && KW == 4 && (reinterpret_cast<uintptr_t>(p.w) & 15u) == 0;
    auto place = [](int v, int c) { return v * VC + (c ^ (VC == 8 ? v & 7 : v >> 1 & 3)); };
    auto copy16 = [](void* to, const void* from) {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(to)), "l"(from) : "memory");
    };
    if (four) {
        for (int i = tid; i < CONV_TREE_CH * VC; i += CONV_TREE_CH * CONV_TREE_GROUPS)
            if (cb * CONV_TREE_CH * VC + i < p.C) copy16(wide + place(i / VC, i % VC), reinterpret_cast<const float4*>(p.w) + cb * CONV_TREE_CH * VC + i);
    }
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
        auto copy = [&](int to, const ET* from) {
            if constexpr (sizeof(R) == 16) copy16(rows + to * CONV_TREE_CH + ch, from);
            else rows[to * CONV_TREE_CH + ch] = IO::ld(from);
        };
        for (int i = grp; i < KW - 1; i += CONV_TREE_GROUPS) {
            if (rst) rows[i * CONV_TREE_CH + ch] = IO::narrow(zero);
            else copy(i, W + (int64_t)i * p.C);
        }
#pragma unroll 8
        for (int j = grp; j < T; j += CONV_TREE_GROUPS) copy(KW - 1 + j, x + (int64_t)j * p.C);
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
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
    if (!on) return;
    // taps right-aligned: place i of KWM holds tap i - (KWM - KW)
    const int pad = KWM - KW;
    float w[KWM][VC], bias[VC];
    if (four) {
#pragma unroll
        for (int v = 0; v < VC; ++v) {
            const float4 f = wide[place(ch, v)];
            w[0][v] = f.x;
            w[1 % KWM][v] = f.y;
            w[2 % KWM][v] = f.z;
            w[3 % KWM][v] = f.w;
        }
    } else {
#pragma unroll
        for (int v = 0; v < VC; ++v)
#pragma unroll
            for (int i = 0; i < KWM; ++i) w[i][v] = i >= pad ? __ldg(p.w + (int64_t)(c + v) * KW + i - pad) : 0.f;
    }
    if (VC % 4 == 0 && p.bias != nullptr && (reinterpret_cast<uintptr_t>(p.bias) & 15u) == 0) {
#pragma unroll
        for (int v = 0; v < VC; v += 4) {
            const float4 f = __ldg(reinterpret_cast<const float4*>(p.bias + c + v));
            bias[v] = f.x;
            bias[(v + 1) % VC] = f.y;
            bias[(v + 2) % VC] = f.z;
            bias[(v + 3) % VC] = f.w;
        }
    } else {
#pragma unroll
        for (int v = 0; v < VC; ++v) bias[v] = p.bias != nullptr ? __ldg(p.bias + c + v) : 0.f;
    }
    // two tokens at a time, step by step, so that their latencies overlap
    constexpr int N = VC * KWM <= 32 ? 2 : 1;
    for (int j = grp; j < T; j += N * CONV_TREE_GROUPS) {
        R z[N][KWM];
#pragma unroll
        for (int x = 0; x < N; ++x) {
            const uint64_t packed = taps[min(j + x * CONV_TREE_GROUPS, T - 1)] << (8 * pad);
#pragma unroll
            for (int i = 0; i < KWM; ++i)
                if (i >= pad) z[x][i] = rows[(int)(packed >> (8 * i) & 0xffu) * CONV_TREE_CH + ch];
        }
        float s[N][VC];
#pragma unroll
        for (int x = 0; x < N; ++x)
#pragma unroll
            for (int v = 0; v < VC; ++v) s[x][v] = bias[v];
#pragma unroll
        for (int i = 0; i < KWM; ++i) {
            if (i < pad) continue;
#pragma unroll
            for (int x = 0; x < N; ++x) {
                float f[VC];
                IO::widen(z[x][i], f);
                if constexpr (VC % 2 == 0) {    // two channels at a time, each as fmaf rounds
#pragma unroll
                    for (int v = 0; v < VC; v += 2) {
                        const float2 t = __ffma2_rn(make_float2(w[i][v], w[i][v + 1]), make_float2(f[v], f[v + 1]), make_float2(s[x][v], s[x][v + 1]));
                        s[x][v] = t.x;
                        s[x][v + 1] = t.y;
                    }
                } else {
#pragma unroll
                    for (int v = 0; v < VC; ++v) s[x][v] = fmaf(w[i][v], f[v], s[x][v]);
                }
            }
        }
        if (p.silu) {
#pragma unroll
            for (int x = 0; x < N; ++x)
#pragma unroll
                for (int v = 0; v < VC; ++v) s[x][v] = silu_short(s[x][v]);
        }
#pragma unroll
        for (int x = 0; x < N; ++x)
            if (j + x * CONV_TREE_GROUPS < T) IO::st(y + (int64_t)(j + x * CONV_TREE_GROUPS) * p.C, IO::narrow(s[x]));
    }
}

// ---------------------------------------------------------------------------
// Recurrence
// ---------------------------------------------------------------------------
// Most column groups of a CTA, of W = 1 or 4 warps each.
__host__ __device__ constexpr int tree_groups(int w) { return w == 4 ? 2 : 4; }
constexpr int TREE_CW = 16;             // columns of a group

// Four neighbouring state elements of a row.
template <typename ST> struct TreeVec;
template <> struct TreeVec<float> {
    using R = uint4;
    static __device__ __forceinline__ void widen(const R& r, float2 (&x)[2]) {
        x[0] = make_float2(__uint_as_float(r.x), __uint_as_float(r.y));
        x[1] = make_float2(__uint_as_float(r.z), __uint_as_float(r.w));
    }
    static __device__ __forceinline__ R narrow(const float2 (&x)[2]) {
        return make_uint4(__float_as_uint(x[0].x), __float_as_uint(x[0].y), __float_as_uint(x[1].x), __float_as_uint(x[1].y));
    }
    static __device__ __forceinline__ R zero() { return make_uint4(0, 0, 0, 0); }
};
template <> struct TreeVec<__half> {
    using R = uint2;
    static __device__ __forceinline__ void widen(const R& r, float2 (&x)[2]) {      // exact
        x[0] = StateVec<__half>::w2(r.x);
        x[1] = StateVec<__half>::w2(r.y);
    }
    static __device__ __forceinline__ R narrow(const float2 (&x)[2]) {              // to nearest even
        return make_uint2(StateVec<__half>::n2(x[0].x, x[0].y), StateVec<__half>::n2(x[1].x, x[1].y));
    }
    static __device__ __forceinline__ R zero() { return make_uint2(0, 0); }
};

// Shared memory of a CTA of `groups` column groups with at most t tokens a request.
template <typename ST> struct TreeSmem {
    static __host__ __device__ constexpr int bytes(int t, int k, int groups, int w) {
        return 3 * t * k * 4                                                        // khat, alpha, qhat of each token
               + t * groups * TREE_CW * 4                                           // v, then delta
               + groups * KMAX * 4 * (int)sizeof(typename TreeVec<ST>::R)           // the initial state
               + 2 * 2 * groups * w * 2 * TREE_CW * 4                               // the warps' sums
               + t * (8 + 8 + 8 + 4);                                               // masks, children, beta and khat . qhat, slots
    }
};

// One CTA: one request, one value head, `groups` times 16 state columns.  W
// warps share a group's columns, 128 / W rows each; lane l of a warp holds 4
// columns (l % 4) of 16 / W rows, four neighbouring ones (l / 4) of every 32.
// The sums over K are three shuffles in a warp and W terms over the warps,
// through shared memory behind a barrier of the group: more warps shorten a
// token's way, fewer save instructions.
//
// A token's state is S_j = diag(alpha_j) S_parent + khat_j delta_j^T with
// delta_j = beta_j (v_j - S_parent^T diag(alpha_j) khat_j), and both of its sums
// are over the parent's state, which is in registers.  Tokens are taken depth
// first: of a token's children first the leaves, whose states only pass
// through on their way out, then the first of the others, in place; two
// children at a time.  Where another branch begins its parent's state is built
// again from the initial state (kept on chip as it was loaded: its slot may be
// one of the snapshots') with the ancestors' deltas, which are kept: two
// operations an element and ancestor, no sums, the same bits as on the way
// there.  So states carry fp32 along every path whatever the pool's type, and
// do not depend on the order of siblings.
//
// FULL: K = V = 128, so that every lane has all its rows and columns and the
// places of a tile are constants.
//
// Measured, us: 16 requests of 32 tokens, 12 heads of 128 x 128, fp16 pool,
// every state stored: 67.6, where its 219 MB take 32.3 at the copy rate.
// Without its stores 51: twelve warps an SM (168 registers) issue in 45 of 100
// cycles, a token's way being sums, shuffles and the next state one behind the
// other.  One request of 8, fp32 pool: 10.6 to 12 (8.2 on the GPU alone, the
// loads and three tokens in a row).  13 requests of up to 48, 6 heads of 96 x 80:
// 56.3.  A child at a time, every tile as if it were ragged: 72 and 74 for the
// first and the last; leaves like any other token, too: 92 and 89.
template <typename ST, typename QT, int W, bool FULL>
__global__ void __launch_bounds__(tree_groups(W) * W * 32, W == 1 ? 3 : 2) kda_tree_kernel(const StepParams p, const uint64_t* tree) {
    using SV = TreeVec<ST>;
    using R = typename SV::R;
    extern __shared__ __align__(128) uint8_t smem[];
    const int KD = FULL ? KMAX : p.k, VD = FULL ? KMAX : p.v;
    constexpr int RL = 16 / W;              // rows of a lane: r0 + i % 4 + 32 (i / 4)
    const int groups = blockDim.x / (32 * W), BV = groups * TREE_CW;
    float* kh = reinterpret_cast<float*>(smem);
    float* al = kh + p.t * KD;
    float* qh = al + p.t * KD;
    float* du = qh + p.t * KD;                                              // [t][BV]: v, then delta
    R* stash = reinterpret_cast<R*>(du + p.t * BV);                         // [RL][threads]
    float* red = reinterpret_cast<float*>(stash + RL * blockDim.x);         // [2][2][groups][W][2][16]
    unsigned long long* masks = reinterpret_cast<unsigned long long*>(red + 2 * 2 * groups * W * 2 * TREE_CW);
    unsigned long long* child = masks + p.t;
    float2* sc = reinterpret_cast<float2*>(child + p.t);                    // beta, khat . qhat
    int32_t* snaps = reinterpret_cast<int32_t*>(sc + p.t);

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, grp = warp / W, share = warp % W;
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
    const int lc = grp * TREE_CW + (lane & 3) * 4, c0 = cb * BV + lc;       // the lane's first column: of the CTA's, of all
    const int r0 = share * (KMAX / W) + (lane >> 2) * 4;                    // its first row
    if (slot < 0) {     // a padding request
        for (int i = tid; i < T * BV; i += blockDim.x) {
            const int j = i / BV, c = cb * BV + i - j * BV;
            if (c < VD) p.o[((int64_t)(tb + j) * p.hv + h) * VD + c] = 0.f;
        }
        return;
    }
    const bool rst = p.reset != nullptr && __ldg(p.reset + n) != 0;
    // its rows and columns are in the state
    auto row_at = [](int i) { return (i & 3) + 32 * (i >> 2); };
    auto has = [&](int i) { return FULL || r0 + 32 * (i >> 2) < KD; };
    auto live = [&](int i) { return FULL || (has(i) && c0 < VD); };
    ST* pool = static_cast<ST*>(p.pool);
    const int64_t tile = (int64_t)r0 * VD + c0;
    // the initial state goes straight to shared memory, each thread's own
    {
        const ST* from = pool + state_at(p, slot, h) + tile;
#pragma unroll
        for (int i = 0; i < RL; ++i) {
            R* to = stash + i * blockDim.x + tid;
            if (live(i) && !rst)
                asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(smem_u32(to)), "l"(from + row_at(i) * VD), "n"(sizeof(R)) : "memory");
            else
                *to = SV::zero();
        }
    }
    __syncthreads();    // child is zero
    // ---- the tokens' vectors, two tokens a warp at a time ----
    const int hq = h / (p.hv / p.hqk), warps = blockDim.x >> 5;
    const bool scaled = p.a_log != nullptr;
    const float gate = scaled ? expf(__ldg(p.a_log + h)) : 1.f;
    constexpr int AHEAD = 2;
    const int d = 4 * lane;
    const bool on = FULL || d < KD;
    const float* bias = scaled && p.dt_bias != nullptr ? p.dt_bias + h * KD + (on ? d : 0) : nullptr;
    using QIO = ConvIO<QT, 4>;
    for (int j0 = warp; j0 < T; j0 += AHEAD * warps) {
        typename QIO::R kr[AHEAD], qr[AHEAD];
        float4 ar[AHEAD];
        float br[AHEAD], vr[AHEAD][2];          // a CTA has at most 64 columns
        static_assert(tree_groups(W) * TREE_CW <= 64, "columns");
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
#pragma unroll
            for (int y = 0; y < 2; ++y) vr[x][y] = lane + 32 * y < BV && cb * BV + lane + 32 * y < VD ? to_f32(vt[32 * y]) : 0.f;
        }
        // step by step for both, so that their latencies overlap; behind the last token it is done again
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
#pragma unroll
        for (int x = 0; x < AHEAD; ++x) {
            const float a[4] = {ar[x].x, ar[x].y, ar[x].z, ar[x].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) g[x][e] = gate_alpha(a[e], scaled, gate, bias != nullptr ? __ldg(bias + e) : 0.f);
        }
#pragma unroll
        for (int x = 0; x < AHEAD; ++x) {
            const int j = min(j0 + x * warps, T - 1);
            const float rk = __frsqrt_rn(kk[x] + L2_EPS), rq = __frsqrt_rn(qq[x] + L2_EPS);
            if (on) {
                *reinterpret_cast<float4*>(kh + j * KD + d) = make_float4(k4[x][0] * rk, k4[x][1] * rk, k4[x][2] * rk, k4[x][3] * rk);
                *reinterpret_cast<float4*>(qh + j * KD + d) = make_float4(q4[x][0] * rq, q4[x][1] * rq, q4[x][2] * rq, q4[x][3] * rq);
                *reinterpret_cast<float4*>(al + j * KD + d) = make_float4(g[x][0], g[x][1], g[x][2], g[x][3]);
            }
#pragma unroll
            for (int y = 0; y < 2; ++y)
                if (lane + 32 * y < BV) du[j * BV + lane + 32 * y] = vr[x][y];
            if (lane == 0) {
                sc[j] = make_float2(sigmoid_neg(-br[x]), kq[x] * rk * rq);
                masks[j] = mr[x];
                if (mr[x] != 0) atomicOr(child + tree_top(mr[x]), 1ull << j);
            }
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    float2 S[RL][2];
#pragma unroll
    for (int i = 0; i < RL; ++i) SV::widen(stash[i * blockDim.x + tid], S[i]);
    __syncthreads();

    // rows r0 + 32 i .. + 3 of a vector; a lane without them reads the first ones, and k as zero: its states stay zero
    auto vec4 = [&](const float* v, int j, int i) {
        return *reinterpret_cast<const float4*>(v + j * KD + (has(4 * i) ? r0 + 32 * i : 0));
    };
    auto key4 = [&](int j, int i) {
        const float4 k = vec4(kh, j, i);
        return has(4 * i) ? k : make_float4(0.f, 0.f, 0.f, 0.f);
    };
    auto times = [&](float2 x, float f) { return __fmul2_rn(x, make_float2(f, f)); };
    auto plus = [&](float f, float2 y, float2 x) { return __ffma2_rn(make_float2(f, f), y, x); };
    auto part = [](const float4& v, int r) { return r == 0 ? v.x : r == 1 ? v.y : r == 2 ? v.z : v.w; };
    // row r of diag(alpha) S + khat delta^T, a and k of its four rows
    auto next_row = [&](int r, const float4& a, const float4& k, const float2 (&dl)[2], float2 (&out)[2]) {
#pragma unroll
        for (int x = 0; x < 2; ++x) out[x] = plus(part(k, r & 3), dl[x], times(S[r][x], part(a, r & 3)));
    };
    // an earlier token's step again
    auto again = [&](int j) {
        const float4 f = *reinterpret_cast<const float4*>(du + j * BV + lc);
        const float2 dl[2] = {make_float2(f.x, f.y), make_float2(f.z, f.w)};
#pragma unroll
        for (int i = 0; i < RL / 4; ++i) {
            const float4 a = vec4(al, j, i), k = key4(j, i);
#pragma unroll
            for (int r = 4 * i; r < 4 * i + 4; ++r) next_row(r, a, k, dl, S[r]);
        }
    };
    int turn = 0;       // which half of `red`
    // Tokens j[0 .. N), children of the token whose state S is: outputs, deltas, states to their snapshots; keep: the
    // last one's to S.  Step by step for all of them, so that their latencies overlap.
    auto step = [&](auto n_of, const int* j, bool keep) {
        constexpr int N = decltype(n_of)::value;
        float f[N][8];
        float4 v[N];
#pragma unroll
        for (int x = 0; x < N; ++x) {
            v[x] = *reinterpret_cast<const float4*>(du + j[x] * BV + lc);
            float2 su[2], sq[2];
#pragma unroll
            for (int i = 0; i < RL / 4; ++i) {
                const float4 a = vec4(al, j[x], i), k = key4(j[x], i), q = vec4(qh, j[x], i);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float ak = part(a, r) * part(k, r), aq = part(a, r) * part(q, r);
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        su[y] = i + r == 0 ? times(S[0][y], ak) : plus(ak, S[4 * i + r][y], su[y]);
                        sq[y] = i + r == 0 ? times(S[0][y], aq) : plus(aq, S[4 * i + r][y], sq[y]);
                    }
                }
            }
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                f[x][2 * y] = su[y].x;
                f[x][2 * y + 1] = su[y].y;
                f[x][4 + 2 * y] = sq[y].x;
                f[x][4 + 2 * y + 1] = sq[y].y;
            }
        }
        // over the 8 row groups (lane bits 4 .. 2), scattered: lane bit 4 tells the sum, bits 3 and 2 the column
        int m = 16;
#pragma unroll
        for (int cnt = 8; cnt > 1; cnt >>= 1, m >>= 1) {
            const bool upper = (lane & m) != 0;
#pragma unroll
            for (int y = 0; y < cnt / 2; ++y)
#pragma unroll
                for (int x = 0; x < N; ++x) {
                    const float send = upper ? f[x][y] : f[x][y + cnt / 2], mine = upper ? f[x][y + cnt / 2] : f[x][y];
                    f[x][y] = mine + __shfl_xor_sync(0xffffffffu, send, m);
                }
        }
        float* sums = red + (turn * 2 * groups + grp) * W * 2 * TREE_CW;        // token x: x * groups * W * 2 * 16 on
        turn ^= 1;
#pragma unroll
        for (int x = 0; x < N; ++x)
            sums[(x * groups * W + share) * 2 * TREE_CW + (lane >> 4) * TREE_CW + (lane & 3) * 4 + (lane >> 2 & 3)] = f[x][0];
        if constexpr (W == 1) __syncwarp();
        else asm volatile("bar.sync %0, %1;" ::"r"(1 + grp), "n"(32 * W) : "memory");
        // the group's sums are there, and its v read
        float2 dl[N][2];
#pragma unroll
        for (int x = 0; x < N; ++x) {
            const float* of = sums + x * groups * W * 2 * TREE_CW + (lane & 3) * 4;
            auto over_warps = [&](const float* y) {
                float4 s = *reinterpret_cast<const float4*>(y);
#pragma unroll
                for (int z = 1; z < W; ++z) {
                    const float4 t = *reinterpret_cast<const float4*>(y + z * 2 * TREE_CW);
                    s.x += t.x; s.y += t.y; s.z += t.z; s.w += t.w;
                }
                return s;
            };
            const float4 u = over_warps(of);
            const float2 bs = sc[j[x]];
            const float4 dt = make_float4(bs.x * (v[x].x - u.x), bs.x * (v[x].y - u.y), bs.x * (v[x].z - u.z), bs.x * (v[x].w - u.w));
            dl[x][0] = make_float2(dt.x, dt.y);
            dl[x][1] = make_float2(dt.z, dt.w);
            if (lane < 4 && share == x % W) {       // one lane of the columns
                *reinterpret_cast<float4*>(du + j[x] * BV + lc) = dt;
                const float4 pq = over_warps(of + TREE_CW);
                float* o = p.o + ((int64_t)(tb + j[x]) * p.hv + h) * VD + c0;
                const float4 out = make_float4(fmaf(bs.y, dt.x, pq.x) * p.inv_sqrt_k, fmaf(bs.y, dt.y, pq.y) * p.inv_sqrt_k,
                                               fmaf(bs.y, dt.z, pq.z) * p.inv_sqrt_k, fmaf(bs.y, dt.w, pq.w) * p.inv_sqrt_k);
                if (FULL || c0 < VD) {              // o has the alignment of floats
                    o[0] = out.x;
                    o[1] = out.y;
                    o[2] = out.z;
                    o[3] = out.w;
                }
            }
        }
#pragma unroll
        for (int x = 0; x < N; ++x) {
            const int32_t snap = snaps[j[x]];
            const bool stay = x == N - 1 && keep;
            ST* to = pool + state_at(p, snap, h) + tile;
#pragma unroll
            for (int i = 0; i < RL / 4; ++i) {
                const float4 a = vec4(al, j[x], i), k = key4(j[x], i);
#pragma unroll
                for (int r = 4 * i; r < 4 * i + 4; ++r) {
                    float2 out[2];
                    next_row(r, a, k, dl[x], out);
                    if (snap >= 0 && live(r)) *reinterpret_cast<R*>(to + row_at(r) * VD) = SV::narrow(out);
                    if (stay) {
                        S[r][0] = out[0];
                        S[r][1] = out[1];
                    }
                }
            }
        }
        if constexpr (W == 1) __syncwarp();     // du is written for all lanes
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
            // another branch: the lowest token left, whose parent is done (two steps ago or more: its delta is there)
            const int j = __ffsll((long long)todo) - 1;
#pragma unroll
            for (int i = 0; i < RL; ++i) SV::widen(stash[i * blockDim.x + tid], S[i]);
            const unsigned long long above = masks[j];
            for (unsigned long long m = above; m != 0; m &= m - 1) again(__ffsll((long long)m) - 1);
            kids = above != 0 ? child[tree_top(above)] & todo : 1ull << j;
        }
        // leaves two at a time, then an inner child; the last leaf and the inner child go together
        const unsigned long long ends = kids & leaves, inner = kids & ~leaves, left = ends & (ends - 1);
        const bool down = ends == 0 || (left == 0 && inner != 0);       // the last of these is the one to go on from
        int j[2];
        j[0] = __ffsll((long long)(ends != 0 ? ends : inner)) - 1;
        j[1] = left != 0 ? __ffsll((long long)left) - 1 : inner != 0 && ends != 0 ? __ffsll((long long)inner) - 1 : -1;
        if (j[1] >= 0) {
            step(std::integral_constant<int, 2>{}, j, down);
            todo &= ~(1ull << j[1]);
        } else {
            step(std::integral_constant<int, 1>{}, j, down);
        }
        todo &= ~(1ull << j[0]);
        if (down) kids = child[j[1] >= 0 ? j[1] : j[0]];
    }
}

}  // namespace kda
