// Verification of drafted tokens: the walk down a request's tree by rejection
// sampling with given random numbers, and the draw of the token behind it.
#pragma once

#include <cfloat>
#include <cstddef>
#include <utility>

#include <cooperative_groups.h>

#include "kda_tree.cuh"

namespace kda {

struct AcceptParams {
    const void *p, *q;              // q: nullptr for drafts that were given, not drawn
    int64_t p_stride, q_stride;     // elements between rows
    int n, total, max_t, vocab;
    const int32_t *cu, *tokens;
    const uint64_t* tree;
    const float *u, *u_last;
    int32_t *accepted, *node, *path, *token, *status;
};

constexpr int ACC_CTAS = 8;         // CTAs of a request: one cluster
constexpr int ACC_THREADS = 256, ACC_WARPS = ACC_THREADS / 32;
constexpr int ACC_SEGS = ACC_CTAS * ACC_WARPS;      // 64 pieces of the vocabulary, a warp each
static_assert(ACC_SEGS == 64, "two pieces a lane");

// A sum of two floats, hi + lo with |lo| at most half a step of hi: 48 bits.
// fp64 runs at a 64th of the fp32 rate here (a version with the tests and the
// scans in fp64: 70 us for 64 chains of 8 over 131072 tokens, where this takes
// 26), and 32 bits lose the places next to a border between two tokens.
struct Pair { float hi, lo; };
// s += x (Knuth's exact sum of two floats; the errors add up in lo).  lo is a
// plain float: a run of these has to be brought back into order by pair_norm
// every few steps, or lo outgrows hi's step and loses its own last places (after
// 1000 steps 2^-41 of the sum, 2^-30 for weights that all round the same way).
__device__ __forceinline__ void pair_add(Pair& s, float x, float x_lo) {
    const float t = s.hi + x, b = t - s.hi;
    s.lo += ((s.hi - (t - b)) + (x - b)) + x_lo;
    s.hi = t;
}
__device__ __forceinline__ Pair pair_norm(Pair s) {
    const float t = s.hi + s.lo;
    return {t, s.lo - (t - s.hi)};
}
__device__ __forceinline__ Pair operator+(Pair a, const Pair& b) {
    pair_add(a, b.hi, b.lo);
    return pair_norm(a);
}
__device__ __forceinline__ Pair operator-(Pair a, const Pair& b) {
    pair_add(a, -b.hi, -b.lo);
    return pair_norm(a);
}
__device__ __forceinline__ Pair operator*(const Pair& a, float f) {
    const float h = __fmul_rn(a.hi, f);     // never fused into the sums that it goes into: its error is added apart
    return pair_norm({h, fmaf(a.hi, f, -h) + a.lo * f});
}
__device__ __forceinline__ bool operator<(const Pair& a, const Pair& b) { return a.hi < b.hi || (a.hi == b.hi && a.lo < b.lo); }
__device__ __forceinline__ Pair pair_shfl(const Pair& a, int lane) {
    return {__shfl_sync(0xffffffffu, a.hi, lane), __shfl_sync(0xffffffffu, a.lo, lane)};
}
// Running sums over the lanes of a warp.
__device__ __forceinline__ Pair pair_scan(Pair a, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const Pair up = {__shfl_up_sync(0xffffffffu, a.hi, o), __shfl_up_sync(0xffffffffu, a.lo, o)};
        if (lane >= o) a = up + a;
    }
    return a;
}

// What every CTA of a request walks by, written by the cluster's first CTA.
struct AcceptInfo {
    int tb, t;                      // t: 0 nothing to do, -1 bad offsets
    int tok[TREE_MAX];
    float p[TREE_MAX], q[TREE_MAX], u[TREE_MAX];    // of the token in its parent's rows; p < 0: not a token
    unsigned long long child[TREE_MAX];
    Pair sum[2][ACC_WARPS];         // a pass's sums, in turn
    Pair part[ACC_WARPS];
    int vote[2][ACC_WARPS];
};

__device__ __forceinline__ float acc_weight(float x) { return x > 0.f ? x : 0.f; }   // NaN: 0

// One row's weights W_k (see kda_accept_kernel) as they are walked over.
template <typename T, bool DRAWN> struct AcceptRow {
    static constexpr int VE = 16 / (int)sizeof(T);
    const T *p, *q;
    int vocab, shift, vecs;         // elements before the row in its first 16-byte vector; vectors
    bool together;                  // q's row lies on its vectors as p's does
    int k;                          // rejections with q
    Pair c;                         // and the sum of their Z: W = max(p - c q, 0)
    unsigned long long gone;        // rejected siblings (without q)
    const AcceptInfo* info;

    __device__ __forceinline__ void set(const T* pr, const T* qr, int v) {
        p = pr;
        q = qr;
        vocab = v;
        shift = (int)((reinterpret_cast<uintptr_t>(pr) & 15u) / sizeof(T));
        vecs = (int)(((int64_t)v + shift + VE - 1) / VE);
        together = DRAWN && ((reinterpret_cast<uintptr_t>(pr) ^ reinterpret_cast<uintptr_t>(qr)) & 15u) == 0;
    }
    struct Raw { uint4 p, q; };
    // A vector's elements; those outside the row are zero.
    __device__ __forceinline__ uint4 edge(const T* row, int i0) const {
        T e[VE];
#pragma unroll
        for (int x = 0; x < VE; ++x) {
            const int i = i0 + x;
            conv_round(0.f, e[x]);
            if (i >= 0 && i < vocab) e[x] = row[i];
        }
        uint4 r;
        memcpy(&r, e, 16);
        return r;
    }
    __device__ __forceinline__ Raw load(int vec) const {
        const int i0 = vec * VE - shift;
        const bool whole = i0 >= 0 && i0 <= vocab - VE;
        Raw r;
        r.p = whole ? __ldg(reinterpret_cast<const uint4*>(p + i0)) : edge(p, i0);
        r.q = make_uint4(0, 0, 0, 0);
        if (DRAWN && k > 0) r.q = whole && together ? __ldg(reinterpret_cast<const uint4*>(q + i0)) : edge(q, i0);
        return r;
    }
    // A vector's weights, as exact sums of two floats, in order.
    template <typename F> __device__ __forceinline__ void weights(const Raw& r, int vec, F&& use) const {
        T pe[VE], qe[VE];
        memcpy(pe, &r.p, 16);
        memcpy(qe, &r.q, 16);
        uint32_t out = 0;           // given drafts: the vector's rejected tokens
        if constexpr (!DRAWN) {
            const int i0 = vec * VE - shift;
            for (unsigned long long g = gone; g != 0; g &= g - 1) {
                const int at = info->tok[__ffsll((long long)g) - 1] - i0;
                if (at >= 0 && at < VE) out |= 1u << at;
            }
        }
#pragma unroll
        for (int x = 0; x < VE; ++x) {
            Pair w = {acc_weight(conv_f32(pe[x])), 0.f};
            if constexpr (DRAWN) {
                const float qf = acc_weight(conv_f32(qe[x]));
                if (k == 1) {       // c = 1: p - q and its error, exact for p > q
                    const float d = w.hi - qf;
                    w = w.hi > qf ? Pair{d, (w.hi - d) - qf} : Pair{0.f, 0.f};
                } else if (k > 1) {
                    const float h = __fmul_rn(c.hi, qf);
                    pair_add(w, -h, -(fmaf(c.hi, qf, -h) + c.lo * qf));
                    w = pair_norm(w);
                    if (!(w.hi > 0.f)) w = {0.f, 0.f};
                }
            } else {
                if (out >> x & 1u) w = {0.f, 0.f};
            }
            use(w, x);
        }
    }
};

// The walk.  cur is the last token accepted (at first token 0), W_0 = p(. | cur),
// Z_0 = 1.  Its children x in order, with W, Z of the rejections so far:
//   drafts drawn from q:  accepted if u q(x) Z < W(x), else W <- max(W - Z q, 0), Z <- sum W
//   drafts given:         accepted if u Z < W(x),      else W(x) <- 0,            Z <- Z - W(x)
// (W / Z is the distribution that is left; nothing is divided, and W = max(p - c q,
// 0) with c the sum of the Z so far, as W only falls).  An accepted
// child becomes cur.  Where no child is left the next token is drawn from W by
// its inverse distribution function: the first i with W(i) > 0 whose running
// sum passes u_last sum W.
//
// A cluster of eight CTAs shares a request's row, 64 warps a piece each.  The
// first CTA gathers what the tests need and gives it to the others, so all
// walk alike; a rejection with q and the draw take one pass over the row's
// pieces and a sum over the cluster, the draw then a second look at one piece
// by its whole CTA.
//
// Measured, us: a chain of 5, fp32, vocabulary 32000: 10.3 (8.7 on the GPU
// alone: the launch, the barriers of the cluster, the draw's second look at a
// piece); 64 chains of 8, 131072: 26.2, of which the 67 MB of the rows looked
// at are 9.9 at the copy rate; 13 trees of up to 37, bf16, 50021: 24, passes
// one behind the other.  Warps mostly stand at barriers (the chain of a walk:
// gather, pass, sum, pass, draw); the issue slots are used in 31 of 100 cycles.
// Eight CTAs are the most that every cluster launch is granted.
template <typename T, bool DRAWN>
__global__ void __cluster_dims__(ACC_CTAS, 1, 1) __launch_bounds__(ACC_THREADS, 4) kda_accept_kernel(const AcceptParams a) {
    namespace cg = cooperative_groups;
    using Row = AcceptRow<T, DRAWN>;
    constexpr int VE = Row::VE;
    __shared__ AcceptInfo info;
    const cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank(), r = (int)blockIdx.x / ACC_CTAS;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const T* P = static_cast<const T*>(a.p);
    const T* Q = static_cast<const T*>(a.q);
    auto begun = cluster.barrier_arrive();      // shared memory of a CTA that has not begun is not written to
    cudaTriggerProgrammaticLaunchCompletion();
    cudaGridDependencySynchronize();

    if (rank == 0) {
        int tb = r * a.max_t, t = a.max_t;
        if (a.cu != nullptr) {
            tb = __ldg(a.cu + r);
            t = __ldg(a.cu + r + 1) - tb;
        }
        if (tb < 0 || t < 0 || t > a.max_t || tb > a.total - t) t = -1;
        if (tid < TREE_MAX) info.child[tid] = 0;
        if (tid == 0) {
            info.tb = tb;
            info.t = t;
        }
        __syncthreads();
        if (tid < t) {
            const unsigned long long m = tree_mask(a.tree, tb + tid, tid) ^ (1ull << tid);
            const int tok = __ldg(a.tokens + tb + tid);
            float pv = -1.f, qv = 1.f;
            if (m != 0) {
                const int up = tree_top(m);
                if (tok >= 0 && tok < a.vocab) {
                    pv = acc_weight(conv_f32(P[(int64_t)(tb + up) * a.p_stride + tok]));
                    if (DRAWN) qv = acc_weight(conv_f32(Q[(int64_t)(tb + up) * a.q_stride + tok]));
                } else {
                    atomicCAS(a.status, 0, STATUS_ARG);
                }
                atomicOr(&info.child[up], 1ull << tid);
            }
            info.tok[tid] = tok;
            info.p[tid] = pv;
            info.q[tid] = qv;
            info.u[tid] = __ldg(a.u + tb + tid);
        }
        __syncthreads();
    }
    cluster.barrier_wait(std::move(begun));
    if (rank == 0) {
        // what the others walk by: the words before the sums
        constexpr int WORDS = offsetof(AcceptInfo, sum) / 4;
        for (int i = tid; i < WORDS * (ACC_CTAS - 1); i += ACC_THREADS) {
            uint32_t* to = reinterpret_cast<uint32_t*>(cluster.map_shared_rank(&info, 1 + i / WORDS));
            to[i % WORDS] = reinterpret_cast<const uint32_t*>(&info)[i % WORDS];
        }
    }
    cluster.sync();
    const int T_ = info.t, tb = info.tb;
    const bool writer = rank == 0 && tid == 0;
    int32_t* path = a.path + (int64_t)r * a.max_t;
    if (T_ <= 0) {      // no tokens: nothing accepted, nothing drawn
        if (rank == 0 && tid < a.max_t) path[tid] = -1;
        if (writer) {
            a.accepted[r] = a.node[r] = 0;
            a.token[r] = -1;
            if (T_ < 0) atomicCAS(a.status, 0, STATUS_ARG);
        }
        return;
    }

    Row row;
    row.info = &info;
    int cur = 0, count = 1, turn = 0;
    Pair z = {1.f, 0.f}, s0, s1, upto, total;
    int v0 = 0, v1 = 0, each = 0;       // this warp's vectors
    auto use = [&](int node) {
        row.set(P + (int64_t)(tb + node) * a.p_stride, DRAWN ? Q + (int64_t)(tb + node) * a.q_stride : nullptr, a.vocab);
        row.k = 0;
        row.c = {0.f, 0.f};
        row.gone = 0;
        each = (row.vecs + ACC_SEGS - 1) / ACC_SEGS;
        v0 = min(row.vecs, (rank * ACC_WARPS + warp) * each);
        v1 = min(row.vecs, v0 + each);
    };
    // sum W over the cluster; lane l then holds the sums s0, s1 of pieces 2 l and 2 l + 1 and the running sum `upto`
    auto sum = [&]() {
        Pair s[2] = {{0.f, 0.f}, {0.f, 0.f}};
        auto add = [&](const Pair& w, int x) { pair_add(s[x & 1], w.hi, w.lo); };
        constexpr int U = 4;
        int v = v0 + lane;
        for (; v < v1; v += 32 * U) {
            typename Row::Raw raw[U];
#pragma unroll
            for (int x = 0; x < U; ++x)
                if (v + 32 * x < v1) raw[x] = row.load(v + 32 * x);
#pragma unroll
            for (int x = 0; x < U; ++x)
                if (v + 32 * x < v1) {
                    row.weights(raw[x], v + 32 * x, add);
                    s[0] = pair_norm(s[0]);
                    s[1] = pair_norm(s[1]);
                }
        }
        Pair d = s[0] + s[1];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            // the lower lane's first: both get the same sum
            const Pair to = {__shfl_xor_sync(0xffffffffu, d.hi, o), __shfl_xor_sync(0xffffffffu, d.lo, o)};
            d = lane & o ? to + d : d + to;
        }
        if (lane == 0) info.sum[turn][warp] = d;
        cluster.sync();
        const Pair* of = &cluster.map_shared_rank(&info, (2 * lane) / ACC_WARPS)->sum[turn][(2 * lane) % ACC_WARPS];
        s0 = of[0];
        s1 = of[1];
        upto = pair_scan(s0 + s1, lane);
        total = pair_shfl(upto, 31);
        turn ^= 1;      // the other half: a CTA may still read this one
    };
    use(0);
    bool summed = false;
    if (writer) path[0] = tb;
    for (unsigned long long rest = info.child[0]; rest != 0;) {
        const int i = __ffsll((long long)rest) - 1;
        rest &= rest - 1;
        if (info.p[i] < 0.f) continue;
        Pair w = {info.p[i], 0.f};
        const float qx = DRAWN ? info.q[i] : 1.f;
        if constexpr (DRAWN) {
            if (row.k > 0) w = w - row.c * qx;      // not above zero: not accepted
        } else {
            for (unsigned long long g = row.gone; g != 0; g &= g - 1)
                if (info.tok[__ffsll((long long)g) - 1] == info.tok[i]) w = {0.f, 0.f};
        }
        // The first child's test is exact: u q is 48 bits, a pair down to 2^-100 (below it the lower half would leave fp32's
        // range, and such a test is made in fp64).
        const float u = info.u[i], uq = u * qx;
        const bool first = row.k == 0 && row.gone == 0;
        const Pair bar = first ? Pair{uq, fmaf(u, qx, -uq)} : (z * qx) * u;
        if (first && uq < 0x1p-100f ? (double)u * (double)qx < (double)w.hi : bar < w) {
            cur = i;
            if (writer) path[count] = tb + i;
            ++count;
            use(i);
            z = {1.f, 0.f};
            summed = false;
            rest = info.child[i];
        } else if constexpr (DRAWN) {
            ++row.k;
            row.c = row.c + z;
            sum();
            z = total;
            summed = true;
        } else {
            row.gone |= 1ull << i;
            z = z - w;
        }
    }
    if (!summed) sum();
    if (!(total.hi > 0.f) && (row.k > 0 || row.gone != 0)) {    // nothing left: from the target's own
        row.k = 0;
        row.gone = 0;
        sum();
    }
    const bool draw = total.hi > 0.f && total.hi <= FLT_MAX;
    if (writer) {
        a.accepted[r] = count;
        a.node[r] = cur + 1;
        if (!draw) {
            a.token[r] = -1;
            atomicCAS(a.status, 0, STATUS_ARG);
        }
    }
    if (rank == 0)
        for (int j = count + tid; j < a.max_t; j += ACC_THREADS) path[j] = -1;
    if (draw) {
        // the piece where the running sum passes u_last of the whole, else the last that has weight
        const Pair target = total * __ldg(a.u_last + r), before = {__shfl_up_sync(0xffffffffu, upto.hi, 1), __shfl_up_sync(0xffffffffu, upto.lo, 1)};
        const Pair base0 = lane == 0 ? Pair{0.f, 0.f} : before, base1 = base0 + s0;
        const bool in0 = s0.hi > 0.f && target < base1, in1 = s1.hi > 0.f && target < upto;
        const uint32_t hit = __ballot_sync(0xffffffffu, in0 || in1), some = __ballot_sync(0xffffffffu, s0.hi > 0.f || s1.hi > 0.f);
        const int who = hit != 0 ? __ffs(hit) - 1 : 31 - __clz(some);
        const int odd = __shfl_sync(0xffffffffu, (int)(hit != 0 ? !in0 : s1.hi > 0.f), who), seg = 2 * who + odd;
        if (seg / ACC_WARPS == rank) {
            // a thread takes neighbouring vectors of the piece
            const Pair base = pair_shfl(odd ? base1 : base0, who);
            const int g0 = min(row.vecs, seg * each), g1 = min(row.vecs, g0 + each), per = (each + ACC_THREADS - 1) / ACC_THREADS;
            const int a0 = min(g1, g0 + tid * per), a1 = min(g1, a0 + per);
            Pair mine = {0.f, 0.f};
            for (int v = a0; v < a1; ++v) {
                row.weights(row.load(v), v, [&](const Pair& w, int) { pair_add(mine, w.hi, w.lo); });
                mine = pair_norm(mine);
            }
            const Pair run = pair_scan(mine, lane);
            if (lane == 31) info.part[warp] = run;
            __syncthreads();
            Pair left = base;
            for (int x = 0; x < warp; ++x) left = left + info.part[x];
            const Pair end = left + run;
            // the first thread that passes the target, else the last with weight; a vote over the CTA
            const bool over = mine.hi > 0.f && target < end;
            const uint32_t o = __ballot_sync(0xffffffffu, over), h = __ballot_sync(0xffffffffu, mine.hi > 0.f);
            if (lane == 0) {
                info.vote[0][warp] = o != 0 ? 32 * warp + __ffs(o) - 1 : 0x7fffffff;
                info.vote[1][warp] = h != 0 ? 32 * warp + 31 - __clz(h) : -1;
            }
            __syncthreads();
            int first = 0x7fffffff, last = -1;
#pragma unroll
            for (int x = 0; x < ACC_WARPS; ++x) {
                first = min(first, info.vote[0][x]);
                last = max(last, info.vote[1][x]);
            }
            if (tid == (first != 0x7fffffff ? first : last)) {
                Pair cum = left + (run - mine);
                int at = -1;
                bool stop = false;
                for (int v = a0; v < a1 && !stop; ++v)
                    row.weights(row.load(v), v, [&](const Pair& w, int x) {
                        if (stop || !(w.hi > 0.f)) return;
                        cum = cum + w;
                        at = v * VE - row.shift + x;
                        stop = first != 0x7fffffff && target < cum;
                    });
                a.token[r] = at;
            }
        }
    }
    cluster.sync();     // a CTA's sums are read by the others until here
}

}  // namespace kda
