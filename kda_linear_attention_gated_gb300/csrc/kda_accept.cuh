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
// fp64 runs at a 64th of the fp32 rate here, and 32 bits lose the places next
// to a border between two tokens.
struct Pair { float hi, lo; };
// s += x (Knuth's exact sum of two floats; the errors add up in lo)
__device__ __forceinline__ void pair_add(Pair& s, float x, float x_lo) {
    const float t = s.hi + x, b = t - s.hi;
    s.lo += ((s.hi - (t - b)) + (x - b)) + x_lo;
    s.hi = t;
}
__device__ __forceinline__ double pair_f64(const Pair& s) { return (double)s.hi + (double)s.lo; }
__device__ __forceinline__ Pair f64_pair(double x) {
    const float hi = (float)x;
    return {hi, isfinite(hi) ? (float)(x - (double)hi) : 0.f};
}

// What every CTA of a request walks by, written by the cluster's first CTA.
struct AcceptInfo {
    int tb, t;                      // t: 0 nothing to do, -1 bad offsets
    int tok[TREE_MAX];
    float p[TREE_MAX], q[TREE_MAX], u[TREE_MAX];    // of the token in its parent's rows; p < 0: not a token
    unsigned long long child[TREE_MAX];
    double sum[2][ACC_WARPS];       // a pass's sums, in turn
    Pair z[TREE_MAX];               // Z_k of the current node
    int found;
};

__device__ __forceinline__ float acc_weight(float x) { return x > 0.f ? x : 0.f; }   // NaN: 0

// One row's weights W_k (see kda_accept_kernel) as they are walked over.
template <typename T, bool DRAWN> struct AcceptRow {
    static constexpr int VE = 16 / (int)sizeof(T);
    const T *p, *q;
    int vocab, shift, vecs;         // elements before the row in its first 16-byte vector; vectors
    bool together;                  // q's row lies on its vectors as p's does
    int k;                          // rejections
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
    // The weights of a vector, as exact sums of two floats.
    __device__ __forceinline__ void weights(const Raw& r, int vec, Pair (&w)[VE]) const {
        T pe[VE], qe[VE];
        memcpy(pe, &r.p, 16);
        memcpy(qe, &r.q, 16);
#pragma unroll
        for (int x = 0; x < VE; ++x) w[x] = {acc_weight(conv_f32(pe[x])), 0.f};
        if constexpr (DRAWN) {
            if (k > 0) {
#pragma unroll
                for (int x = 0; x < VE; ++x) {      // Z_0 = 1: p - q and its error, exact for p > q
                    const float pf = w[x].hi, qf = acc_weight(conv_f32(qe[x])), d = pf - qf;
                    w[x] = pf > qf ? Pair{d, (pf - d) - qf} : Pair{0.f, 0.f};
                }
                for (int j = 1; j < k; ++j) {
                    const Pair z = info->z[j];
#pragma unroll
                    for (int x = 0; x < VE; ++x) {
                        const float qf = acc_weight(conv_f32(qe[x]));
                        const float h = z.hi * qf, e = fmaf(z.hi, qf, -h) + z.lo * qf;
                        Pair s = w[x];
                        pair_add(s, -h, -e);
                        const float hi = s.hi + s.lo;
                        w[x] = hi > 0.f && w[x].hi > 0.f ? Pair{hi, s.lo - (hi - s.hi)} : Pair{0.f, 0.f};
                    }
                }
            }
        } else {
            const int i0 = vec * VE - shift;
            for (unsigned long long g = gone; g != 0; g &= g - 1) {
                const int at = info->tok[__ffsll((long long)g) - 1] - i0;
                if (at >= 0 && at < VE)
#pragma unroll
                    for (int x = 0; x < VE; ++x)
                        if (x == at) w[x] = {0.f, 0.f};
            }
        }
    }
};

// The walk.  cur is the last token accepted (at first token 0), W_0 = p(. | cur),
// Z_0 = 1.  Its children x in order, with W, Z of the rejections so far:
//   drafts drawn from q:  accepted if u q(x) Z < W(x), else W <- max(W - Z q, 0), Z <- sum W
//   drafts given:         accepted if u Z < W(x),      else W(x) <- 0,            Z <- Z - W(x)
// (W / Z is the distribution that is left; nothing is divided).  An accepted
// child becomes cur.  Where no child is left the next token is drawn from W by
// its inverse distribution function: the first i with W(i) > 0 whose running
// sum passes u_last sum W.
//
// A cluster of eight CTAs shares a request's row, 64 warps a piece each.  The
// first CTA gathers what the tests need and gives it to the others, so all
// walk alike; a rejection with q and the draw take one pass over the row's
// pieces and a sum over the cluster, the draw then one warp's second look at its
// piece.  Bound by memory: a row of p and one of q.
template <typename T, bool DRAWN>
__global__ void __cluster_dims__(ACC_CTAS, 1, 1) __launch_bounds__(ACC_THREADS) kda_accept_kernel(const AcceptParams a) {
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
    double z = 1.0, s0 = 0.0, s1 = 0.0, upto = 0.0, total = 0.0;
    int v0 = 0, v1 = 0;         // this warp's vectors
    auto use = [&](int node) {
        row.set(P + (int64_t)(tb + node) * a.p_stride, DRAWN ? Q + (int64_t)(tb + node) * a.q_stride : nullptr, a.vocab);
        row.k = 0;
        row.gone = 0;
        const int each = (row.vecs + ACC_SEGS - 1) / ACC_SEGS, seg = rank * ACC_WARPS + warp;
        v0 = min(row.vecs, seg * each);
        v1 = min(row.vecs, v0 + each);
    };
    // sum W over the cluster; lane l then holds the sums s0, s1 of pieces 2 l and 2 l + 1
    auto sum = [&]() {
        Pair s[2] = {{0.f, 0.f}, {0.f, 0.f}};
        constexpr int U = 4;
        int v = v0 + lane;
        for (; v + 32 * (U - 1) < v1; v += 32 * U) {
            typename Row::Raw raw[U];
#pragma unroll
            for (int x = 0; x < U; ++x) raw[x] = row.load(v + 32 * x);
#pragma unroll
            for (int x = 0; x < U; ++x) {
                Pair w[VE];
                row.weights(raw[x], v + 32 * x, w);
#pragma unroll
                for (int e = 0; e < VE; ++e) pair_add(s[e & 1], w[e].hi, w[e].lo);
            }
        }
        for (; v < v1; v += 32) {
            const typename Row::Raw raw = row.load(v);
            Pair w[VE];
            row.weights(raw, v, w);
#pragma unroll
            for (int e = 0; e < VE; ++e) pair_add(s[e & 1], w[e].hi, w[e].lo);
        }
        double d = pair_f64(s[0]) + pair_f64(s[1]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
        if (lane == 0) info.sum[turn][warp] = d;
        cluster.sync();
        const double* of = &cluster.map_shared_rank(&info, (2 * lane) / ACC_WARPS)->sum[turn][(2 * lane) % ACC_WARPS];
        s0 = of[0];
        s1 = of[1];
        upto = s0 + s1;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const double up = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += up;
        }
        total = __shfl_sync(0xffffffffu, upto, 31);
        turn ^= 1;      // the other half: a CTA may still read this one
    };
    use(0);
    bool summed = false;
    if (writer) path[0] = tb;
    for (unsigned long long rest = info.child[0]; rest != 0;) {
        const int i = __ffsll((long long)rest) - 1;
        rest &= rest - 1;
        if (info.p[i] < 0.f) continue;
        double w = info.p[i];
        const double qx = DRAWN ? info.q[i] : 1.0;
        if constexpr (DRAWN) {
            for (int j = 0; j < row.k; ++j) {
                w -= (j == 0 ? 1.0 : pair_f64(info.z[j])) * qx;
                if (!(w > 0.0)) w = 0.0;
            }
        } else {
            for (unsigned long long g = row.gone; g != 0; g &= g - 1)
                if (info.tok[__ffsll((long long)g) - 1] == info.tok[i]) w = 0.0;
        }
        if ((double)info.u[i] * qx * z < w) {
            cur = i;
            if (writer) path[count] = tb + i;
            ++count;
            use(i);
            z = 1.0;
            summed = false;
            rest = info.child[i];
        } else if constexpr (DRAWN) {
            ++row.k;
            sum();
            z = total;
            summed = true;
            __syncthreads();
            if (tid == 0 && row.k < TREE_MAX) info.z[row.k] = f64_pair(total);
            __syncthreads();
        } else {
            row.gone |= 1ull << i;
            z -= w;
        }
    }
    if (!summed) sum();
    if (!(total > 0.0) && (row.k > 0 || row.gone != 0)) {    // nothing left: from the target's own
        row.k = 0;
        row.gone = 0;
        sum();
    }
    if (writer) {
        a.accepted[r] = count;
        a.node[r] = cur + 1;
        if (!(total > 0.0) || !(total <= DBL_MAX)) {
            a.token[r] = -1;
            atomicCAS(a.status, 0, STATUS_ARG);
        }
    }
    if (rank == 0)
        for (int j = count + tid; j < a.max_t; j += ACC_THREADS) path[j] = -1;
    if (total > 0.0 && total <= DBL_MAX) {
        // the piece where the running sum passes u_last of the whole, else the last that has weight
        const double target = (double)__ldg(a.u_last + r) * total, before = upto - (s0 + s1);
        const bool in0 = s0 > 0.0 && before + s0 > target, in1 = s1 > 0.0 && before + s0 + s1 > target;
        const uint32_t hit = __ballot_sync(0xffffffffu, in0 || in1), some = __ballot_sync(0xffffffffu, s0 > 0.0 || s1 > 0.0);
        const int who = hit != 0 ? __ffs(hit) - 1 : 31 - __clz(some);
        const bool odd = hit != 0 ? !in0 : s1 > 0.0;
        const int seg = 2 * who + (int)__shfl_sync(0xffffffffu, (int)odd, who);
        if (seg == rank * ACC_WARPS + warp) {
            double base = __shfl_sync(0xffffffffu, before, who);
            if (seg & 1) base += __shfl_sync(0xffffffffu, s0, who);
            int last = -1;
            bool done = false;
            for (int v = v0; v < v1 && !done; v += 32) {
                Pair w[VE];
                double mine = 0.0;
                const int vec = v + lane;
                if (vec < v1) {
                    const typename Row::Raw raw = row.load(vec);
                    row.weights(raw, vec, w);
#pragma unroll
                    for (int e = 0; e < VE; ++e) mine += pair_f64(w[e]);
                }
                double run = mine;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const double up = __shfl_up_sync(0xffffffffu, run, o);
                    if (lane >= o) run += up;
                }
                const uint32_t over = __ballot_sync(0xffffffffu, mine > 0.0 && base + run > target);
                const uint32_t has = __ballot_sync(0xffffffffu, mine > 0.0);
                if (has != 0) {
                    const int l = over != 0 ? __ffs(over) - 1 : 31 - __clz(has);
                    int at = -1;
                    if (lane == l) {
                        double cum = base + (run - mine);
                        bool stop = false;
#pragma unroll
                        for (int e = 0; e < VE; ++e) {
                            if (stop || !(w[e].hi > 0.f)) continue;
                            cum += pair_f64(w[e]);
                            at = vec * VE - row.shift + e;
                            stop = over != 0 && cum > target;
                        }
                    }
                    last = __shfl_sync(0xffffffffu, at, l);
                }
                done = over != 0;
                base += __shfl_sync(0xffffffffu, run, 31);
            }
            if (lane == 0) a.token[r] = last;
        }
    }
    cluster.sync();     // a CTA's sums are read by the others until here
}

}  // namespace kda
