// Attention of wide trees of drafted tokens over the 4-bit cache: many query
// rows of a key/value head, on the 5th-generation tensor cores.  The format, the
// scores' units and the softmax's constants are those of kda_kv4.cuh.
#pragma once

#include "kda_kv4.cuh"

namespace kda {

// ---------------------------------------------------------------------------
// tcgen05
// ---------------------------------------------------------------------------
__device__ __forceinline__ void tmem_alloc(uint32_t* where, uint32_t cols) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(where)), "r"(cols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t base, uint32_t cols) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(base), "r"(cols) : "memory");
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// Everything issued so far, done: one arrival on `bar`.
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
// A descriptor `bytes` further on.
__device__ __forceinline__ uint64_t tc_step(uint64_t desc, uint32_t bytes) { return desc + (bytes >> 4); }
// One lane of a converged warp.
__device__ __forceinline__ bool tc_elect() {
    uint32_t yes;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(yes));
    return yes != 0;
}
// d (fp32 in tensor memory) = a b, or += with `more`; fp16 operands in shared memory, 16 deep.
__device__ __forceinline__ void tc_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool more) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
        ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)more) : "memory");
}
// The same with a in tensor memory: a row a lane, two of its elements a column.
__device__ __forceinline__ void tc_mma_ta(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool more) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
        ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)more) : "memory");
}
// A phase that is most likely complete: one test without the scheduler's help first.
__device__ __forceinline__ bool mbar_poll(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok) : "r"(smem_u32(bar)), "r"(parity) : "memory");
    return ok != 0 || mbar_wait(bar, parity);
}
// 32 columns of the warp's 32 lanes.
__device__ __forceinline__ void tmem_ld32(uint32_t addr, float (&x)[32]) {
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
          "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
          "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
          "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr) : "memory");
#pragma unroll
    for (int i = 0; i < 32; ++i) x[i] = __uint_as_float(r[i]);
}
// 16 columns, out and back.
__device__ __forceinline__ void tmem_ld16(uint32_t addr, float (&x)[16]) {
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
          "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(addr) : "memory");
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};\n\t"
        "tcgen05.wait::st.sync.aligned;"
        ::"r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
          "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(addr) : "memory");
}
__device__ __forceinline__ void tmem_st16f(uint32_t addr, const float (&x)[16]) {
    uint32_t r[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(x[i]);
    tmem_st16(addr, r);
}
// Descriptor of a tile of 128-byte rows in shared memory, 16-byte pieces at
// their place xor (row % 8) (the 128-byte swizzle), groups of eight rows 1024
// bytes apart.  `lead`: bytes between 64-element stretches of the other
// dimension, for operands whose rows run along it.
__device__ __forceinline__ uint64_t tc_desc(uint32_t addr, uint32_t lead) {
    return (uint64_t)((addr & 0x3ffffu) >> 4) | (uint64_t)(lead >> 4) << 16 | (uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46 |
           (uint64_t)2 << 61;
}
// fp16 operands, fp32 sums; B_ROWS: b's rows run along N (else along K).
__host__ __device__ constexpr uint32_t tc_idesc(int m, int n, bool b_rows) {
    return 1u << 4 | (b_rows ? 1u << 16 : 0u) | (uint32_t)(n / 8) << 17 | (uint32_t)(m / 16) << 24;
}

// ---------------------------------------------------------------------------
// Attention
// ---------------------------------------------------------------------------
constexpr int KVT_ROWS = 128;            // query rows of a tile: the tensor cores' M
constexpr int KVT_KEYS = 64;             // keys of a unit of work: four blocks
constexpr int KVT_WARPS = 8;              // that compute; one more fetches the codes and starts the products
constexpr int KVT_THREADS = 32 * (KVT_WARPS + 1);
constexpr int KVT_STAGES = 3;            // units of codes: one read for its values, one for its keys, one on its way; a
                                         // fourth would leave an SM's second CTA without shared memory
// What beginning and ending a part costs a CTA, in units.  3, 6, 10, us: 32
// requests of up to 16 tokens, 16383 keys 123, 94, 92; 8 of 64 tokens, 8192
// keys 135, 133, 135; 4 of 32, 4000 keys 46, 46, 49; 1 of 64, 20000 67.6, 64.5,
// 65.5.
constexpr int KVT_PART = 6;
constexpr int KVT_FIRST = KVT_PART + 2, KVT_LAST = 2;   // what a cut leaves before and after it in a tile (see Kv4Shape)
constexpr int KVT_MAX_CTAS = 304;        // two for each of 152 SMs
// Calls with at most so many query rows a head (tokens times query heads of a
// key/value head) go to kda_kv4_attend_kernel, whose time grows with the rows;
// this one's is nearly that of 128 rows.  That kernel / this one at 32, 48, 64
// and 128 rows, us: 16 requests, 8192 keys, 8 heads of 128, bf16 101/111,
// 139/117, 177/117, 330/129; fp16 (two products) 156/207, 222/207, 291/207,
// 559/213; heads of 64, bf16 70/92, 96/97, 121/98, 222/104; fp32 101/102,
// 143/113, 186/113, 354/123; one request, 8 heads of 128, bf16, 100000 keys
// 80/96, 113/100, 131/100, 242/109; 8192 keys 31/35, 33/35, 35/35, 43/38; 500
// keys 22/30, 22/30, 31/34, 30/36.  At 48 rows short contexts gain by staying
// there and long ones lose; their lengths are on the device.
constexpr int KVT_MIN_ROWS = 48;
// CTAs that join a tile.  1, 4, 16, us: one request of 24 tokens, 131071 keys
// (76 CTAs a tile) 381, 146, 88; 32 of up to 16, 16383 keys 128, 99, 94.
constexpr int KVT_JOIN_GROUPS = 16;
// Units whose products with the values add up in one sum of the tensor cores,
// before that is added to the part's others in fp32 (and a thread's sum of
// probabilities likewise).  The tensor cores round towards zero at each
// addition, 4 a unit and 8 with remainders, and a sum that grows evenly loses
// up to 2^-24 of itself at each: 2^-10 after 2000 units in one sum, where here
// it is 2^-17, 2^-15 and 2^-14 at most for fp32, fp16 and bf16 queries.  One sum
// / these, us: 16 requests of 16 tokens, 8192 keys, 8 query heads on each of 8
// heads of 128, fp32 212/215, fp16 209/209, bf16 127/127; heads of 64, fp32
// 121/121; 64 of 32, 30000 keys, 4 on each of 8 of 128, fp16 2587/2611, bf16
// 1342/1344.
__host__ __device__ constexpr int kvt_chain(int dtype) { return dtype == 0 ? 16 : dtype == 1 ? 64 : 256; }
constexpr int KVT_COUNTERS = 4096;       // bytes at the head of the workspace that kda_kv4_attend_kernel's counters take

template <int D, bool SPLIT> struct KvtSmem {
    static constexpr int SLABS = D / 64;                         // 64-channel stretches, 128 bytes a row
    static constexpr int Q = SLABS * KVT_ROWS * 128, K = SLABS * KVT_KEYS * 128;
    static constexpr int STAGE = 4 * Kv4<D>::BLOCK;
    static constexpr int OFF_Q = 0, OFF_K = OFF_Q + Q * (SPLIT ? 2 : 1), OFF_V = OFF_K + 2 * K,       // keys of even and odd units
                         OFF_RAW = OFF_V + K, OFF_ROWF = OFF_RAW + KVT_STAGES * STAGE,
                         OFF_MAX = OFF_ROWF + KVT_ROWS * 4,      // [2][128] halves' maxima, then sums
                         OFF_ROWNAN = OFF_MAX + 2 * KVT_ROWS * 4,     // [128] value groups in which a row has seen a NaN
                         OFF_NAN = OFF_ROWNAN + KVT_ROWS * 4,    // [2][8] tokens of an even or odd unit whose value group is NaN
                         OFF_BAR = OFF_NAN + 2 * 8 * 8,              // raw [stages], scores, sums
                         OFF_MISC = OFF_BAR + 8 * 8,             // tensor memory base, blocks not there [stages]
                         OFF_WALK = OFF_MISC + 32,
                         OFF_KEPT = OFF_WALK + 2 * 128,          // [256] a thread's (maximum, sum) that were kept
                         BYTES = OFF_KEPT + 32 * KVT_WARPS * 8 + 1024;      // and 1024 to align
    // rows of a tile's queries that are fetched together, as they come, to where keys and values will be
    static __host__ __device__ constexpr int fetched(int es) { return KVT_ROWS * D * es <= OFF_RAW - OFF_K ? KVT_ROWS : KVT_ROWS / 2; }
    static_assert(KVT_ROWS / 2 * D * (SPLIT ? 4 : 2) <= OFF_RAW - OFF_K && KVT_ROWS * D * 4 <= OFF_RAW, "queries in, sums out");
    // CTAs an SM (228 KB of shared memory, 1 KB of it taken for each)
    static constexpr int CTAS = 2 * (BYTES + 1024) <= 228 * 1024 ? 2 : 1;
    // columns of tensor memory, of which an SM has 512: scores, sums, probabilities (two a column, SPLIT: and their
    // remainders), and the sums that are kept apart where there is room for them
    static constexpr int TMEM = 512 / CTAS, USED = KVT_KEYS + D + (SPLIT ? 2 : 1) * KVT_KEYS / 2;
    static constexpr bool KEEP = USED + D <= TMEM;
    static_assert(USED <= TMEM, "tensor memory");
};

// N (2 or 4) neighbouring elements of a typed array in shared memory, from a multiple of N.
template <int N> __device__ __forceinline__ void ld_shared(const void* p, int i, int dtype, float (&x)[N]) {
    if (dtype == 0) {
#pragma unroll
        for (int e = 0; e < N; e += 2) {
            const float2 f = *reinterpret_cast<const float2*>(static_cast<const float*>(p) + i + e);
            x[e] = f.x;
            x[e + 1] = f.y;
        }
        return;
    }
#pragma unroll
    for (int e = 0; e < N; e += 2) {
        const uint32_t w = *reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(p) + i + e);
        const float2 f = dtype == 1 ? __half22float2(*reinterpret_cast<const __half2*>(&w)) : __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w));
        x[e] = f.x;
        x[e + 1] = f.y;
    }
}

// Whether any thread of two warps says so; barrier `id` is theirs.
__device__ __forceinline__ bool pair_any(int id, bool yes) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %2, 0;\n\tbarrier.red.or.pred q, %1, 64, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r) : "r"(id), "r"((uint32_t)yes) : "memory");
    return r != 0;
}

// One request's part of the work (see Kv4Req), units of 64 keys.
__device__ __forceinline__ Kv4Req kvt_request(const Kv4AttendParams& p, int r) {
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
    q.tiles = (q.t * p.grp + KVT_ROWS - 1) / KVT_ROWS;
    const int64_t end = (int64_t)q.ctx + q.t;
    if (q.t > 0 && end > 0) {
        if (end > (int64_t)p.cols * p.page_tokens || (p.rot && end > p.rope_rows) || q.ctx < 0) {
            q.err = STATUS_ARG;
        } else {
            if (p.window > 0) q.first = max(0, q.ctx - p.window + 1) / KVT_KEYS;
            q.units = (int)((end + KVT_KEYS - 1) / KVT_KEYS) - q.first;
        }
    }
    return q;
}
__device__ __forceinline__ int64_t kvt_cost(const Kv4Req& q, int heads) {
    return q.units > 0 ? (int64_t)(q.units + KVT_PART) * q.tiles * heads : 0;
}

// The list of all (request, head, row tile, unit), cut evenly: CTA c's share
// begins at cut c, moved to a tile's end where too little of the tile would be
// left on one side (as in kda_kv4_attend_kernel).
__device__ __forceinline__ int64_t kvt_even(int64_t total, int ctas) {
    return max((int64_t)(KVT_FIRST + KVT_LAST), (total + ctas - 1) / ctas);
}

// A CTA's share: thread 0 walks it, from part to part.
struct KvtWalk {
    int64_t at, end;     // in the list: the next place, the share's end
    int64_t r0;          // where request r begins
    int64_t s0;          // and the current tile
    int r, h, i0, b0, b1;
    int valid;           // there is a part
    Kv4Req q;
    __device__ __forceinline__ bool next(const Kv4AttendParams& p) {
        for (;;) {
            if (at >= end) return false;
            while (at >= r0 + kvt_cost(q, p.heads)) {
                r0 += kvt_cost(q, p.heads);
                if (++r >= p.n) return false;
                q = kvt_request(p, r);
            }
            const int each = q.units + KVT_PART;
            const uint32_t off = (uint32_t)(at - r0);       // the host bounds a request's cost
            const int seg = (int)(off / (uint32_t)each), u = (int)(off - (uint32_t)seg * each);
            h = seg / q.tiles;
            i0 = (seg - h * q.tiles) * KVT_ROWS;
            s0 = at - u;
            const int take = (int)min((int64_t)(each - u), end - at);
            b0 = max(0, u - KVT_PART);
            b1 = max(0, u + take - KVT_PART);
            at += take;
            if (b0 < b1) return true;
        }
    }
};

// Where cut c falls (moved as above), by a warp: lanes share the requests.
// `own`: the lane's request where there are at most 32.  `walk` (of the lane
// that finds it): the request there.
__device__ __forceinline__ int64_t kvt_cut(const Kv4AttendParams& p, int64_t even, int64_t total, int c, int lane, const Kv4Req& own,
                                           KvtWalk* walk) {
    const int64_t cut = even * c;
    if (cut >= total) return total;
    int64_t begin = 0;
#pragma unroll 1
    for (int base = 0; base < p.n; base += 32) {
        Kv4Req q = own;
        if (p.n > 32) {
            q = Kv4Req{};
            if (base + lane < p.n) q = kvt_request(p, base + lane);
        }
        const int64_t mine = kvt_cost(q, p.heads);
        int64_t upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t up = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += up;
        }
        upto += begin;
        const uint32_t who = __ballot_sync(0xffffffffu, cut < upto);
        if (who != 0) {
            const int l = __ffs(who) - 1;
            int64_t moved = cut;
            if (lane == l) {
                const int each = q.units + KVT_PART, u = (int)((uint32_t)(cut - (upto - mine)) % (uint32_t)each);
                moved += u < KVT_FIRST ? -u : each - u < KVT_LAST ? each - u : 0;
                if (walk != nullptr) {
                    walk->r = base + l;
                    walk->r0 = upto - mine;
                    walk->q = q;
                }
            }
            return __shfl_sync(0xffffffffu, moved, l);
        }
        begin = __shfl_sync(0xffffffffu, upto, 31);
    }
    return total;
}

// What CTA c leaves for the join at the head of the workspace: the tile that its
// share begins inside, if it is the second of the CTAs that share it.
struct KvtJoin {
    int32_t last;        // the last CTA of the tile; 0: nothing to join here
    int32_t row0, rows;  // the tile's rows: query head h * grp + i % grp of token tok0 + i / grp, i from row0 on
    int32_t tok0, h, pad[3];
};
static_assert(sizeof(KvtJoin) == 32, "workspace");
constexpr int KVT_HEAD = 16384;          // bytes of the workspace before the partial sums
static_assert(KVT_MAX_CTAS * sizeof(KvtJoin) <= KVT_HEAD, "workspace");

// Partial sums of a part: [rows][D] sums, [rows] (maximum, sum).
template <int D> struct KvtPart {
    static constexpr int FLOATS = KVT_ROWS * (D + 2);
};

// S = Q K^T and O += P V on the tensor cores (M 128 query rows of a key/value
// head, fp16 operands, fp32 sums in tensor memory), one pass with a running
// maximum and sum.  Codes times scales are exact in fp16; queries are scaled by a
// power of two a row and rounded as in kda_kv4_attend_kernel, SPLIT: with their
// remainders, and probabilities with theirs, as second operands into the same
// sums.  The tensor cores' sums are added up in fp32 every few units (see
// kvt_chain): in columns of tensor memory that are left, or, for bf16 queries
// and heads of 128, in the part's place in the workspace.
//
// A unit of 64 keys is a step between two barriers of the CTA.  Behind the
// first the control warp starts the last unit's P V and the unit's scores;
// meanwhile the eight others write the next unit's keys to shared memory in the
// tensor cores' layout (two places, in turn) and, once P V is done, this unit's
// values.  They then take the scores to probabilities, a thread half a row, back
// into tensor memory, where the tensor cores read them.  V is used as it lies, keys by
// channels (its rows run along N).  A running maximum moves only past a slack of
// KV4_SLACK, so O is seldom scaled.  The other CTA of the SM fills what one
// leaves idle.
//
// Measured, us: 8 requests of 64 tokens, 8192 keys, 4 query heads on each of 8
// heads of 128, bf16: 126, where the products take 36.2 at the measured rate
// and the codes 12.5; 32 of up to 16 tokens, 6 query heads on each of 8, 16383
// keys at most: 88 (8.7 and 12.7; most of the 128 rows are empty, and warps
// without any skip the softmax); 1 of 24, 131071 keys, 4 heads of 64, fp16: 84
// (6.8 and 5.6).  The two CTAs of an SM issue in 48 of 100 cycles, 460
// instructions a warp and unit, and the tensor cores are busy in 24: bound by a
// unit's chain.  Of its 3300 cycles (heads of 128) a warp spends 600 at the
// barrier, 780 on the next keys, 350 waiting for the last P V, 350 on values,
// 180 waiting for scores, 430 on fetching and comparing them, 430 on
// probabilities.  A CTA's 54 units of the first size are 90 of its 126 us, the
// rest its parts' beginnings and ends and the join.  The first size on the way here: warp products of 16 rows 324;
// tensor cores, a barrier between any two steps 259; one barrier a unit, a warp
// for copies and products 141; probabilities in tensor memory and two places for
// keys 135; queries four rows at a time 131; P V before the scores, values
// between them, keys' stores without bank conflicts 126.  Codes loaded ahead of
// the wait for P V, scores fetched while values are written: the same.
//
// Parts of a (request, head, tile) that several CTAs share go to the
// workspace, and kda_kv4_tree_join_kernel adds them in order.
template <int D, bool SPLIT>
__global__ void __launch_bounds__(KVT_THREADS, KvtSmem<D, SPLIT>::CTAS) kda_kv4_tree_kernel(const Kv4AttendParams p) {
    using F = Kv4<D>;
    using SM = KvtSmem<D, SPLIT>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    uint8_t *Q = smem + SM::OFF_Q, *K = smem + SM::OFF_K, *V = smem + SM::OFF_V, *raw = smem + SM::OFF_RAW;
    float* rowf = reinterpret_cast<float*>(smem + SM::OFF_ROWF);
    uint32_t* row_nan = reinterpret_cast<uint32_t*>(smem + SM::OFF_ROWNAN);
    float* half_max = reinterpret_cast<float*>(smem + SM::OFF_MAX);
    unsigned long long* nan_tok = reinterpret_cast<unsigned long long*>(smem + SM::OFF_NAN);
    uint64_t *bar_raw = reinterpret_cast<uint64_t*>(smem + SM::OFF_BAR), *bar_s = bar_raw + KVT_STAGES, *bar_o = bar_s + 1;
    uint32_t* misc = reinterpret_cast<uint32_t*>(smem + SM::OFF_MISC);
    volatile uint32_t* missing = misc + 1;      // [stages] blocks of a unit that are not there
    volatile int *any_empty = reinterpret_cast<int*>(misc + 4), *nan_any = any_empty + 1;     // nan_any: [2], as nan_tok
    auto walk = [&](int i) -> KvtWalk& { return *reinterpret_cast<KvtWalk*>(smem + SM::OFF_WALK + 128 * i); };   // this part's, the next's
    static_assert(sizeof(KvtWalk) <= 128 && KVT_STAGES == 3, "KvtSmem");

    if (tid == 0) {
        for (int i = 0; i < KVT_STAGES + 2; ++i) mbar_init(bar_raw + i, 1);
        fence_mbar_init();
        nan_any[0] = nan_any[1] = 0;
    }
    if (tid < 16) nan_tok[tid] = 0;
    cudaTriggerProgrammaticLaunchCompletion();
    cudaGridDependencySynchronize();
    // behind the wait: tensor memory that a CTA held there, a CTA of the launch before could be waiting for
    if (warp == 1) tmem_alloc(misc, SM::TMEM);

    // ---- this CTA's share ----
    if (warp == 0) {
        int64_t total = 0;
        bool empty = false;
        Kv4Req own = {};
#pragma unroll 1
        for (int r = lane; r < p.n; r += 32) {
            own = kvt_request(p, r);
            total += kvt_cost(own, p.heads);
            if (own.err && blockIdx.x == 0) atomicCAS(p.status, 0, own.err);
            empty |= own.t > 0 && own.units == 0;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
        empty = __any_sync(0xffffffffu, empty);
        const int64_t even = kvt_even(total, gridDim.x);
        KvtWalk& w = walk(0);
        const int64_t c0 = kvt_cut(p, even, total, blockIdx.x, lane, own, &w), c1 = kvt_cut(p, even, total, blockIdx.x + 1, lane, own, nullptr);
        __syncwarp();
        if (lane == 0) {
            w.at = c0;
            w.end = c1;
            w.valid = c0 < c1 && w.next(p);
            *any_empty = empty;
            KvtJoin j = {};
            if (w.valid && w.b0 > 0) {   // the CTAs of a tile: those between the cuts that stayed inside it
                const int first = (int)((w.s0 + KVT_FIRST + even - 1) / even) - 1;
                if (first + 1 == (int)blockIdx.x) {
                    j.last = (int)((w.s0 + w.q.units + KVT_PART - KVT_LAST) / even);
                    j.row0 = w.i0;
                    j.rows = min(KVT_ROWS, w.q.t * p.grp - w.i0);
                    j.tok0 = w.q.tok0;
                    j.h = w.h;
                }
            }
            reinterpret_cast<KvtJoin*>(p.counters)[blockIdx.x] = j;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // read again where it is needed: registers are short
    auto tm_s = [&]() { return *static_cast<volatile uint32_t*>(misc); };
    auto tm_o = [&]() { return tm_s() + KVT_KEYS; };
    auto tm_p = [&]() { return tm_o() + D; };       // probabilities, two a column, and with SPLIT their remainders
    auto tm_k = [&]() { return tm_s() + SM::USED; };        // KEEP: sums that are kept apart
    if (*any_empty) {   // requests without a visible key: zero rows
        for (int r = blockIdx.x; r < p.n; r += gridDim.x) {
            const Kv4Req q = kvt_request(p, r);
            if (q.units > 0) continue;
            const int64_t base = (int64_t)q.tok0 * p.h_q * D;
            for (int64_t i = tid * 4; i < (int64_t)q.t * p.h_q * D; i += KVT_THREADS * 4) st_elem4(p.o, base + i, p.dtype, 0.f, 0.f, 0.f, 0.f);
        }
    }

    const int bpp = p.page_tokens >> 4;
    uint32_t phases = 0;                // bits: raw stages, then scores, then sums
    auto phase = [&](int i) { return phases >> i & 1u; };
    bool alive = true;
    // this thread's row of a tile (a lane of tensor memory) and half of a unit's keys
    const int row = 32 * (warp & 3) + lane, half = warp >> 2;
    const uint32_t lane_base = (uint32_t)(32 * (warp & 3)) << 16;
    // a part's output or its place in the workspace
    auto part_at = [&](const KvtWalk& w) { return p.partials + (int64_t)(2 * blockIdx.x + (w.b0 == 0 ? 1 : 0)) * KvtPart<D>::FLOATS; };
    auto is_whole = [](const KvtWalk& w) { return w.b0 == 0 && w.b1 == w.q.units; };
    auto out_at = [&](const KvtWalk& w, int i) {        // of row i of the tile
        const int x = w.i0 + i, j = x / p.grp;
        return ((int64_t)(w.q.tok0 + j) * p.h_q + w.h * p.grp + x - j * p.grp) * D;
    };
    int cur = 0;

    for (; walk(cur).valid; cur ^= 1) {
        const KvtWalk& w = walk(cur);
        const Kv4Req& req = w.q;        // read from shared memory where it is needed
        if (warp == KVT_WARPS) {
            // ---- codes fetched and products started: a lane a block, its page looked up a unit ahead ----
            const int b0 = w.b0, b1 = w.b1, last = req.ctx + req.t;
            const int32_t* table = p.table + (int64_t)w.r * p.cols;
            const uint8_t* base = p.pages + (int64_t)w.h * bpp * F::BLOCK;
            // the lane's next block, by page and place in it
            int blk = (req.first + b0) * 4 + lane, pg = blk / bpp, in = blk - pg * bpp, stage = 0, page = 0;
            bool wanted = false;
            const int low_end = p.window > 0 ? req.ctx - p.window + 1 : -1;     // blocks that end there are in no window
            auto look = [&](int b) {
                wanted = b < b1 && lane < 4 && blk * 16 < last && low_end < (blk + 1) * 16;
                if (wanted) page = __ldg(table + pg);
            };
            auto fetch = [&](int b) {
                const bool ok = wanted && page >= 0 && page < p.num_pages;
                if (wanted && !ok) atomicCAS(p.status, 0, STATUS_SLOT_RANGE);
                const uint32_t there = __ballot_sync(0xffffffffu, ok);
                if (lane == 0) {
                    missing[stage] = there ^ 15u;
                    if (there != 0) mbar_arrive_expect_tx(bar_raw + stage, __popc(there) * F::BLOCK);
                    else mbar_arrive(bar_raw + stage);
                }
                __syncwarp();
                if (ok && !p.withhold)
                    bulk_load(raw + stage * SM::STAGE + lane * F::BLOCK, base + (int64_t)page * p.page_stride + in * F::BLOCK, F::BLOCK, bar_raw + stage);
                stage = stage + 1 == KVT_STAGES ? 0 : stage + 1;
                blk += 4;
                for (in += 4; in >= bpp; in -= bpp) ++pg;
                look(b + 1);
            };
            look(b0);
            for (int b = b0; b < min(b1, b0 + 2); ++b) fetch(b);
            if (lane == 0) {            // what comes behind this part
                KvtWalk& n = walk(cur ^ 1);
                n = w;
                n.valid = n.next(p);
            }
            __syncwarp();
            constexpr uint32_t id_s = tc_idesc(KVT_ROWS, KVT_KEYS, false), id_o = tc_idesc(KVT_ROWS, D, true);
            const uint32_t s_at = tm_s(), o_at = tm_o(), p_at = tm_p();
            const uint64_t dQ = tc_desc(smem_u32(Q), 16), dK = tc_desc(smem_u32(K), 16), dV = tc_desc(smem_u32(V), KVT_KEYS * 128);
            auto add_values = [&](bool more) {
#pragma unroll
                for (int part = 0; part < (SPLIT ? 2 : 1); ++part)
#pragma unroll
                    for (int k = 0; k < KVT_KEYS / 16; ++k)
                        tc_mma_ta(o_at, p_at + part * (KVT_KEYS / 2) + k * 8, tc_step(dV, k * 2048), id_o, more || part + k > 0);
                tc_commit(bar_o);
            };
            const int chain = SPLIT ? kvt_chain(p.dtype) : kvt_chain(2);
            int ready = 0;              // the stage of unit b + 1
            for (int b = b0 - 1; b <= b1; ++b) {
                bool ok = true;         // codes b + 1 are there
                if (b + 1 < b1) {
                    ok = mbar_wait(bar_raw + ready, phase(ready));
                    if (ok) phases ^= 1u << ready;
                    ready = ready + 1 == KVT_STAGES ? 0 : ready + 1;
                }
                alive = __syncthreads_and(ok);
                if (!alive) break;
                const bool rare = nan_any[(b - 1) & 1] != 0;
                if (tc_elect()) {
                    tc_fence_after();
                    if (b > b0) add_values(((b - 1 - b0) & (chain - 1)) != 0);
                    if (b >= b0 && b < b1) {
                        const uint64_t dKb = tc_step(dK, (b & 1) * SM::K);
#pragma unroll
                        for (int part = 0; part < (SPLIT ? 2 : 1); ++part)
#pragma unroll
                            for (int k = 0; k < D / 16; ++k)
                                tc_mma(s_at, tc_step(dQ, part * SM::Q + k / 4 * (KVT_ROWS * 128) + k % 4 * 32),
                                       tc_step(dKb, k / 4 * (KVT_KEYS * 128) + k % 4 * 32), id_s, part + k > 0);
                        tc_commit(bar_s);
                    }
                }
                __syncwarp();
                if (b >= b0 && b + 2 < b1) fetch(b + 2);        // into the stage of unit b - 1
                if (rare) __syncthreads();                      // the others look through that unit's tokens
            }
            alive = __syncthreads_and(alive);
        } else {
            const int &b0 = w.b0, &b1 = w.b1;
            const int rows = min(KVT_ROWS, req.t * p.grp - w.i0);
            // rows of the warps that have any; what the others' are is seen nowhere, since a row is a row in both products
            const int live = (rows + 31) & ~31;
            // ---- queries: fetched together, where keys, values and probabilities will be; then rotated, scaled to
            // below 1 by a power of two, rounded: 16 neighbouring rows a warp, a row at a time ----
            {
                const int es = p.dtype == 0 ? 4 : 2, chunks = D * es / 16;       // 16-byte pieces of a row
                const uint32_t hold = smem_u32(K);
                const int most = SM::fetched(es), hr = p.rot >> 1;
                constexpr int E = D / 32;
                const int d = lane * E;
                const bool first = d < hr;
#pragma unroll 1
                for (int from = 0; from < KVT_ROWS; from += most) {
#pragma unroll 4
                    for (int i = tid; i < min(most, rows - from) * chunks; i += 32 * KVT_WARPS) {
                        const int x = i / chunks, c = i - x * chunks, y = w.i0 + from + x, j = y / p.grp;
                        const int64_t at = (int64_t)(req.tok0 + j) * p.q_stride + (int64_t)(w.h * p.grp + y - j * p.grp) * D;
                        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;"
                                     ::"r"(hold + i * 16), "l"(static_cast<const char*>(p.q) + at * es + c * 16) : "memory");
                    }
                    const int each = most / KVT_WARPS, w0 = from + warp * each;
                    int pos = 0;            // of the lane's row of the warp's
                    if (lane < each && w0 + lane < rows) {
                        const int j = (w.i0 + w0 + lane) / p.grp;
                        pos = req.ctx + __popcll(tree_mask(p.tree, req.tok0 + j, j)) - 1;
                    }
                    // the rotation's rows into the first-level cache, a line a load, all at once
                    const int lines = 2 * ((hr + 31) / 32);
                    for (int e0 = 0; e0 < each * lines; e0 += 32) {
                        const int e = min(e0 + lane, each * lines - 1), k = e / lines, line = e - k * lines;
                        const float* entry = (line & 1 ? p.sin : p.cos) + (int64_t)__shfl_sync(0xffffffffu, pos, k) * hr + (line >> 1) * 32;
                        float x;
                        asm volatile("ld.global.ca.f32 %0, [%1];" : "=f"(x) : "l"(entry));
                    }
                    asm volatile("cp.async.wait_all;" ::: "memory");
                    asm volatile("bar.sync 5, 256;" ::: "memory");
                    // four rows at a time, step by step, so that their latencies overlap
                    constexpr int G = 4;
                    const int dtype = SPLIT ? p.dtype : 2;
                    const bool turns = d < p.rot;
#pragma unroll 1
                    for (int k = 0; k < each && w0 + k < live; k += G) {
                        float x[G][E];
#pragma unroll
                        for (int r = 0; r < G; ++r) {
                            ld_shared<E>(K, (w0 + k + r - from) * D + d, dtype, x[r]);
                            if (w0 + k + r >= rows)
#pragma unroll
                                for (int e = 0; e < E; ++e) x[r][e] = 0.f;
                        }
                        int64_t at[G];
#pragma unroll
                        for (int r = 0; r < G; ++r) at[r] = (int64_t)__shfl_sync(0xffffffffu, pos, k + r) * hr;
                        if (turns && p.inter) {
                            float cs[G][E / 2], sn[G][E / 2];
#pragma unroll
                            for (int r = 0; r < G; ++r) {
                                ld_elems<E / 2>(p.cos, at[r] + d / 2, 0, cs[r]);
                                ld_elems<E / 2>(p.sin, at[r] + d / 2, 0, sn[r]);
                            }
#pragma unroll
                            for (int r = 0; r < G; ++r)
#pragma unroll
                                for (int e = 0; e < E / 2; ++e) {
                                    const float a = x[r][2 * e], b = x[r][2 * e + 1];
                                    x[r][2 * e] = a * cs[r][e] - b * sn[r][e];
                                    x[r][2 * e + 1] = b * cs[r][e] + a * sn[r][e];
                                }
                        } else if (turns) {
                            float cs[G][E], sn[G][E], y[G][E];
                            const int pair = first ? d + hr : d - hr, entry = first ? d : d - hr;
#pragma unroll
                            for (int r = 0; r < G; ++r) {
                                ld_elems<E>(p.cos, at[r] + entry, 0, cs[r]);
                                ld_elems<E>(p.sin, at[r] + entry, 0, sn[r]);
                                ld_shared<E>(K, (w0 + k + r - from) * D + pair, dtype, y[r]);
                            }
#pragma unroll
                            for (int r = 0; r < G; ++r)
#pragma unroll
                                for (int e = 0; e < E; ++e) {
                                    const float v = x[r][e] * cs[r][e] + (first ? -y[r][e] : y[r][e]) * sn[r][e];
                                    x[r][e] = w0 + k + r < rows ? v : 0.f;
                                }
                        }
                        float amax[G];
#pragma unroll
                        for (int r = 0; r < G; ++r) {
                            amax[r] = 0.f;
#pragma unroll
                            for (int e = 0; e < E; ++e) amax[r] = fmaxf(amax[r], fabsf(x[r][e]));
                        }
#pragma unroll
                        for (int o = 16; o > 0; o >>= 1)
#pragma unroll
                            for (int r = 0; r < G; ++r) amax[r] = fmaxf(amax[r], __shfl_xor_sync(0xffffffffu, amax[r], o));
#pragma unroll
                        for (int r = 0; r < G; ++r) {
                            // as in kda_kv4_attend_kernel
                            const int i = w0 + k + r, z = amax[r] > 1e-30f && amax[r] < 1e37f ? (int)(__float_as_uint(amax[r]) >> 23) - 126 : 0;
                            const float down = __uint_as_float(
                                amax[r] < 1e37f ? (uint32_t)(127 - z) << 23 | (__float_as_uint(p.scale_log2) & 0x80000000u) : 0x7fffffffu);
                            uint8_t* to = Q + (d / 64) * (KVT_ROWS * 128) + i * 128 + (((d % 64 / 8) ^ (i & 7)) << 4) + d % 8 * 2;
#pragma unroll
                            for (int e = 0; e < E; e += 2) {
                                const float u = x[r][e] * down, v = x[r][e + 1] * down;
                                const __half2 hi = __floats2half2_rn(u, v);
                                *reinterpret_cast<__half2*>(to + e * 2) = hi;
                                if constexpr (SPLIT) {
                                    const float2 f = __half22float2(hi);
                                    *reinterpret_cast<__half2*>(to + SM::Q + e * 2) = __floats2half2_rn(u - f.x, v - f.y);
                                }
                            }
                            if (lane == 0) rowf[i] = fmaxf(1e-30f, fabsf(p.scale_log2) * __uint_as_float((uint32_t)(127 + z) << 23));
                        }
                    }
                    asm volatile("bar.sync 5, 256;" ::: "memory");      // other queries, or keys, go there
                }
            }
            // ---- what this thread's row sees of the tree and of the context ----
            uint64_t own = 0;
            int low = 0x7fffffff;
            if (row < rows) {
                const int j = (w.i0 + row) / p.grp;
                own = tree_mask(p.tree, req.tok0 + j, j);
                low = p.window > 0 ? req.ctx + __popcll(own) - p.window : 0;
                if (p.window > 0)
                    for (int more = __popcll(own) - p.window; more > 0; --more) own &= own - 1;
            }
            auto sees = [&](int key) {
                const int at = key - req.ctx;
                return at < 0 ? key >= low : at < TREE_MAX && (own >> at & 1u) != 0;
            };
            float m = -FLT_MAX, l = 0.f;
            // sums that are kept: this thread's columns in tensor memory, or else in the part's place in the workspace; its
            // row's maximum then and the sum of probabilities until then
            const int chain = SPLIT ? kvt_chain(p.dtype) : kvt_chain(2);
            float2* kept_ml = reinterpret_cast<float2*>(smem + SM::OFF_KEPT) + tid;
            auto kept_at = [&](int k) { return tm_k() + lane_base + half * (D / 2) + 16 * k; };
            auto kept_mem = [&](int k) { return reinterpret_cast<float4*>(part_at(w)) + tid + 4 * k * (32 * KVT_WARPS); };
            auto add_kept = [&](int k, float g, float (&o)[16]) {       // o += g times 16 columns that were kept
                if constexpr (SM::KEEP) {
                    float old[16];
                    tmem_ld16(kept_at(k), old);
#pragma unroll
                    for (int i = 0; i < 16; ++i) o[i] = fmaf(old[i], g, o[i]);
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float4 old = __ldcg(kept_mem(k) + i * (32 * KVT_WARPS));
                        o[4 * i] = fmaf(old.x, g, o[4 * i]);
                        o[4 * i + 1] = fmaf(old.y, g, o[4 * i + 1]);
                        o[4 * i + 2] = fmaf(old.z, g, o[4 * i + 2]);
                        o[4 * i + 3] = fmaf(old.w, g, o[4 * i + 3]);
                    }
                }
            };
            auto keep = [&](int k, const float (&o)[16]) {
                if constexpr (SM::KEEP) {
                    tmem_st16f(kept_at(k), o);
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        __stcg(kept_mem(k) + i * (32 * KVT_WARPS), make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]));
                }
            };
            if (half == 0) row_nan[row] = 0;
            const float c = rowf[row];
            const bool idle = 32 * (warp & 3) >= live;
            bool ok = true;
            int st = 0;                 // the stage of unit b + 1, whose keys are next

            // NaN among unit b's values that not all rows see, behind the barrier that ends it: the flags of even and odd
            // units lie apart, and are set again two barriers on.
            auto find_nan = [&](int b) {
                if (nan_any[b & 1] == 0) return;
#pragma unroll 1
                for (int g = 0; g < D / 16; ++g)
                    for (unsigned long long t = nan_tok[(b & 1) * 8 + g]; t != 0; t &= t - 1)
                        if (half == 0 && sees((req.first + b) * KVT_KEYS + __ffsll((long long)t) - 1)) row_nan[row] |= 1u << g;
                __syncthreads();
                if (tid < 8) nan_tok[(b & 1) * 8 + tid] = 0;
                if (tid == 0) nan_any[b & 1] = 0;
            };

            // Unit b + 1's keys and unit b's values while the tensor cores are on, then unit b's scores; every `chain` units the
            // sums so far are kept apart.  (Two loops, so that the inner one's registers know nothing of it: in one, 3 % slower.)
            int b = b0 - 1, next = b0 + chain + 1;
#pragma unroll 1
            for (;;) {
#pragma unroll 1
                for (const int stop = min(b1, next); b < stop; ++b) {
                    fence_proxy_async_smem();
                    tc_fence_before();
                    // keys b, probabilities and values b - 1 are written, codes b - 1 read, codes b + 1 there
                    alive = __syncthreads_and(ok);
                    if (!alive) break;
                    if (b > b0) find_nan(b - 1);
                    // ---- keys: a token's quarter a thread ----
                    if (b + 1 < b1) {
                        {
                            const int key = tid >> 2, q = tid & 3;
                            const uint8_t* B = raw + st * SM::STAGE + (key >> 4) * F::BLOCK;
                            const bool gone = missing[st] >> (key >> 4) & 1u;
                            if constexpr (D == 128) {
                                const uint4 c = *reinterpret_cast<const uint4*>(B + F::KC + (key & 15) * 64 + q * 16);
                                uint32_t s2 = *reinterpret_cast<const uint16_t*>(B + F::KS + (key & 15) * 8 + 2 * q);
                                if (gone) s2 = 0;
                                // every other quarter takes its words from the middle on, so that eight lanes' stores fall on
                                // different banks
                                const bool swap = (q & 2) != 0;
                                const uint32_t two = cvt_e4m3x2_f16x2(s2), sc = swap ? __byte_perm(two, two, 0x1032) : two;
                                const uint32_t code[4] = {swap ? c.z : c.x, swap ? c.w : c.y, swap ? c.x : c.z, swap ? c.y : c.w};
                                uint8_t* to = K + ((b + 1) & 1) * SM::K + (q >> 1) * (KVT_KEYS * 128) + key * 128;
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    uint32_t v[4];
                                    cvt_e2m1x8_f16(code[i], v);
#pragma unroll
                                    for (int e = 0; e < 4; ++e) v[e] = i < 2 ? hmul2_half<false>(v[e], sc) : hmul2_half<true>(v[e], sc);
                                    *reinterpret_cast<uint4*>(to + ((((q & 1) * 4 + i) ^ (q & 2) ^ (key & 7)) << 4)) =
                                        make_uint4(v[0], v[1], v[2], v[3]);
                                }
                            } else {
                                const uint2 c = *reinterpret_cast<const uint2*>(B + F::KC + (key & 15) * 32 + q * 8);
                                uint32_t s2 = B[F::KS + (key & 15) * 4 + q];
                                if (gone) s2 = 0;
                                const uint32_t sc = cvt_e4m3x2_f16x2(s2);
                                const uint32_t code[2] = {c.x, c.y};
#pragma unroll
                                for (int i = 0; i < 2; ++i) {
                                    uint32_t v[4];
                                    cvt_e2m1x8_f16(code[i], v);
#pragma unroll
                                    for (int e = 0; e < 4; ++e) v[e] = hmul2_half<false>(v[e], sc);
                                    *reinterpret_cast<uint4*>(K + ((b + 1) & 1) * SM::K + key * 128 + (((q * 2 + i) ^ (key & 7)) << 4)) =
                                        make_uint4(v[0], v[1], v[2], v[3]);
                                }
                            }
                        }
                    }
                    st = st + 1 == KVT_STAGES ? 0 : st + 1;
                    if (b < b0) continue;
                    const int sv = st >= 2 ? st - 2 : st + 1;               // the stage of unit b
                    const int key0 = (req.first + b) * KVT_KEYS;
                    const uint32_t miss = missing[sv];
                    // keys that every row sees: [ctx + t - window, ctx)
                    const bool masked = key0 + KVT_KEYS > req.ctx || (p.window > 0 && key0 < req.ctx + req.t - p.window) || miss != 0;
                    // ---- values, when the last unit's products are done with: 16 channels (64: 8) of two tokens a thread ----
                    if (b > b0) {
                        ok = mbar_poll(bar_o, phase(KVT_STAGES + 1));
                        if (ok) phases ^= 1u << (KVT_STAGES + 1);
                    }
                    if (ok) {
                        const int bk = tid >> 6, hf = tid >> 5 & 1, g = lane >> 2, tp = lane & 3;
                        const uint8_t* B = raw + sv * SM::STAGE + bk * F::BLOCK;
                        const int key = bk * 16 + hf * 8 + 2 * tp, grp = D == 128 ? g : g >> 1;     // its first token, its scale group
                        uint32_t s2 = *reinterpret_cast<const uint16_t*>(B + F::VS + (grp * 4 + tp) * 4 + hf * 2);
                        if (masked) {
                            // tokens behind the end hold anything, and 0 * NaN is NaN: their scales become 0, and so do NaN
                            // ones, whose groups of the rows that see them are then set by hand (a rare path)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const bool out = (miss >> bk & 1u) || key0 + key + e >= req.ctx + req.t, nan = (s2 >> (8 * e) & 0x7fu) == 0x7fu;
                                if (nan && !out) {
                                    nan_any[b & 1] = 1;
                                    atomicOr(nan_tok + (b & 1) * 8 + grp, 1ull << (key + e));
                                }
                                if (nan || out) s2 &= ~(0xffu << (8 * e));
                            }
                        }
                        const uint32_t sc = cvt_e4m3x2_f16x2(s2);
                        constexpr int W = D / 64;           // words of a token's
                        uint32_t code[2 * W];
                        if constexpr (D == 128) {
                            const uint4 cw = *reinterpret_cast<const uint4*>(B + F::VC + hf * 512 + lane * 16);
                            code[0] = cw.x; code[1] = cw.y; code[2] = cw.z; code[3] = cw.w;
                        } else {
                            const uint2 cw = *reinterpret_cast<const uint2*>(B + F::VC + hf * 256 + lane * 8);
                            code[0] = cw.x; code[1] = cw.y;
                        }
#pragma unroll
                        for (int i = 0; i < 2 * W; ++i) {
                            // channels 8 ch ..; at D = 128 every other lane's two pieces change places, so that eight lanes' stores
                            // fall on different banks
                            const int kk = key + i / W, piece = D == 128 ? (i ^ g) & 1 : 0, ch = D == 128 ? (g & 3) * 2 + piece : g;
                            const uint32_t word = D == 128 ? (piece ? code[(i & 2) + 1] : code[i & 2]) : code[i];
                            uint32_t v[4];
                            cvt_e2m1x8_f16(word, v);
#pragma unroll
                            for (int e = 0; e < 4; ++e) v[e] = i < W ? hmul2_half<false>(v[e], sc) : hmul2_half<true>(v[e], sc);
                            *reinterpret_cast<uint4*>(V + (D == 128 ? g >> 2 : 0) * (KVT_KEYS * 128) + kk * 128 + ((ch ^ (kk & 7)) << 4)) =
                                make_uint4(v[0], v[1], v[2], v[3]);
                        }
                    }
                    // ---- scores to probabilities ----
                    if (ok) {
                        ok = mbar_poll(bar_s, phase(KVT_STAGES));
                        if (ok) phases ^= 1u << KVT_STAGES;
                    }
                    // the warp's verdict, not a lane's; the two warps of a row meet whatever it is
                    ok = __all_sync(0xffffffffu, ok);
                    tc_fence_after();
                    if (!idle) {
                        float s[32], top = -INFINITY;
                        if (ok) {
                            tmem_ld32(tm_s() + lane_base + 32 * half, s);
                            if (masked) {
#pragma unroll
                                for (int i = 0; i < 32; ++i) {
                                    const int at = 32 * half + i;
                                    if (!sees(key0 + at) || (miss >> (at >> 4) & 1u)) s[i] = -INFINITY;
                                }
                            }
#pragma unroll
                            for (int i = 0; i < 32; i += 2) top = fmaxf(fmaxf(s[i], s[i + 1]), top);
                        }
                        top *= c;
                        // seldom: a score above its row's running maximum by more than the slack, in either half
                        if (pair_any(1 + (warp & 3), top > m + KV4_SLACK)) {
                            half_max[half * KVT_ROWS + row] = top;
                            asm volatile("bar.sync %0, 64;" ::"r"(1 + (warp & 3)) : "memory");
                            top = fmaxf(top, half_max[(half ^ 1) * KVT_ROWS + row]);
                            const bool grow = top > m + KV4_SLACK;
                            const float f = grow ? ex2f(m - top) : 1.f;
                            if (grow) m = top;
                            l *= f;
                            if (ok && b > b0) {
#pragma unroll 1
                                for (int k = 0; k < D / 32; ++k) {
                                    const uint32_t at = tm_o() + lane_base + half * (D / 2) + 16 * k;
                                    float o[16];
                                    tmem_ld16(at, o);
#pragma unroll
                                    for (int i = 0; i < 16; ++i) o[i] *= f;
                                    tmem_st16f(at, o);
                                }
                            }
                            asm volatile("bar.sync %0, 64;" ::"r"(1 + (warp & 3)) : "memory");      // half_max is read
                        }
                        if (ok) {
                            const float neg = KV4_LIFT - m;
                            float2 sum = make_float2(l, 0.f);
                            uint32_t hi[16];
#pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                const float2 x = __ffma2_rn(make_float2(s[2 * i], s[2 * i + 1]), make_float2(c, c), make_float2(neg, neg));
                                const float x0 = ex2f(x.x), x1 = ex2f(x.y);
                                sum = __fadd2_rn(sum, make_float2(x0, x1));
                                const __half2 hh = __floats2half2_rn(x0, x1);
                                hi[i] = *reinterpret_cast<const uint32_t*>(&hh);
                                if constexpr (SPLIT) {
                                    const float2 f = __half22float2(hh);
                                    s[2 * i] = x0 - f.x;
                                    s[2 * i + 1] = x1 - f.y;
                                }
                            }
                            tmem_st16(tm_p() + lane_base + 16 * half, hi);
                            if constexpr (SPLIT) {
#pragma unroll
                                for (int i = 0; i < 16; ++i) {
                                    const __half2 rest = __floats2half2_rn(s[2 * i], s[2 * i + 1]);
                                    hi[i] = *reinterpret_cast<const uint32_t*>(&rest);
                                }
                                tmem_st16(tm_p() + lane_base + KVT_KEYS / 2 + 16 * half, hi);
                            }
                            l = sum.x + sum.y;
                        }
                    }
                }
                if (!alive || b != next) break;
                // The products of the last unit, not begun yet, start new sums; those so far are kept.
                if (ok && !idle) {
                    const bool more = next > b0 + chain + 1;
                    const float2 ml = more ? *kept_ml : make_float2(-FLT_MAX, 0.f);
                    const float g = ex2f(ml.x - m);
#pragma unroll 1
                    for (int k = 0; k < D / 32; ++k) {
                        float o[16];
                        tmem_ld16(tm_o() + lane_base + half * (D / 2) + 16 * k, o);
                        if (more) add_kept(k, g, o);
                        keep(k, o);
                    }
                    *kept_ml = make_float2(m, fmaf(ml.y, g, l));
                    l = 0.f;
                }
                next += chain;
            }
            if (alive) {                // the last unit's
                fence_proxy_async_smem();
                tc_fence_before();
                alive = __syncthreads_and(ok);
                if (alive) find_nan(b1 - 1);
            }
            // ---- the part's sums ----
            if (alive) {
                ok = mbar_wait(bar_o, phase(KVT_STAGES + 1));
                if (ok) phases ^= 1u << (KVT_STAGES + 1);
            }
            const float2 ml_kept = b1 - b0 > chain ? *kept_ml : make_float2(-FLT_MAX, 0.f);
            const float g = ex2f(ml_kept.x - m);
            l = fmaf(ml_kept.y, g, l);
            half_max[half * KVT_ROWS + row] = l;
            alive = __syncthreads_and(alive && ok);
            tc_fence_after();
            if (alive) {
                l += half_max[(half ^ 1) * KVT_ROWS + row];
            } else {                    // a wait ran out: nothing of this part
                m = -FLT_MAX;
                l = 0.f;
            }
            if (b1 - b0 > chain && !idle) {
#pragma unroll 1
                for (int k = 0; k < D / 32; ++k) {
                    const uint32_t at = tm_o() + lane_base + half * (D / 2) + 16 * k;
                    float o[16];
                    tmem_ld16(at, o);
                    add_kept(k, g, o);
                    tmem_st16f(at, o);
                }
            }
            // through shared memory (queries to probabilities are done with), 16-byte pieces at their place xor (row % 8)
            const bool whole = is_whole(w);
            float4* tile = reinterpret_cast<float4*>(smem);
            {
                const uint32_t nan_groups = row_nan[row];
                const float f = whole ? (l == 0.f ? 0.f : p.v_scale / l) : 1.f;
#pragma unroll
                for (int k = 0; k < D / 32; ++k) {
                    if (idle) break;
                    float o[16];
                    const int d0 = half * (D / 2) + 16 * k;
                    tmem_ld16(tm_o() + lane_base + d0, o);
#pragma unroll
                    for (int i = 0; i < 16; i += 4) {
                        float4 v = make_float4(o[i] * f, o[i + 1] * f, o[i + 2] * f, o[i + 3] * f);
                        if (l == 0.f) v = make_float4(0.f, 0.f, 0.f, 0.f);
                        if (nan_groups >> (d0 >> 4) & 1u) v = make_float4(NAN, NAN, NAN, NAN);
                        tile[row * (D / 4) + (((d0 + i) / 4) ^ (row & 7))] = v;
                    }
                }
            }
            float* part = part_at(w);
            if (!whole && half == 0 && row < rows) __stcg(reinterpret_cast<float2*>(part + KVT_ROWS * D) + row, make_float2(m, l));
            asm volatile("bar.sync 5, 256;" ::: "memory");
            for (int i = tid; i < rows * (D / 4); i += 32 * KVT_WARPS) {
                const int x = i / (D / 4), c = i % (D / 4);
                const float4 v = tile[x * (D / 4) + (c ^ (x & 7))];
                if (whole) st_elem4(p.o, out_at(w, x) + 4 * c, p.dtype, v.x, v.y, v.z, v.w);
                else __stcg(reinterpret_cast<float4*>(part) + i, v);
            }
        }
        if (!alive && tid == 0) atomicCAS(p.status, 0, STATUS_TIMEOUT);
        if (!alive) {
            // copies and products in flight end (or time out) before their memory is used again; nothing more is begun
            if (warp == KVT_WARPS) {
                for (int i = 0; i < KVT_STAGES; ++i) (void)mbar_wait(bar_raw + i, phase(i));
            } else {
                (void)mbar_wait(bar_s, phase(KVT_STAGES));
                (void)mbar_wait(bar_o, phase(KVT_STAGES + 1));
            }
        }
        tc_fence_before();
        __syncthreads();                // tensor memory, queries and this part's walk are free
        tc_fence_after();
        if (!alive) break;
    }
    if (!alive) {                       // the share's other parts: as if they saw no key
        KvtWalk& w = walk(cur);
        for (;;) {
            if (tid == 0) w.valid = w.next(p);
            __syncthreads();
            if (!w.valid) break;
            const int rows = min(KVT_ROWS, w.q.t * p.grp - w.i0);
            float* part = part_at(w);
            for (int i = tid; i < rows * (D / 4); i += KVT_THREADS) {
                const int x = i / (D / 4), d = i % (D / 4) * 4;
                if (is_whole(w)) st_elem4(p.o, out_at(w, x) + d, p.dtype, 0.f, 0.f, 0.f, 0.f);
                else __stcg(reinterpret_cast<float4*>(part + x * D + d), make_float4(0.f, 0.f, 0.f, 0.f));
                if (!is_whole(w) && d == 0) __stcg(reinterpret_cast<float2*>(part + KVT_ROWS * D) + x, make_float2(-FLT_MAX, 0.f));
            }
            __syncthreads();
        }
    }
    __syncthreads();
    if (warp == 1) tmem_free(tm_s(), SM::TMEM);
}

// Joins the parts of the tiles that more than one CTA of kda_kv4_tree_kernel
// worked on, in order; several CTAs a tile, found by its second CTA there.
template <int D>
__global__ void __launch_bounds__(256) kda_kv4_tree_join_kernel(const Kv4AttendParams p) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    cudaTriggerProgrammaticLaunchCompletion();
    cudaGridDependencySynchronize();
    constexpr int GROUPS = KVT_JOIN_GROUPS, each = KVT_ROWS / 8 / GROUPS;     // rows of a warp
    const int c1 = (int)blockIdx.x / GROUPS + 1, g = (int)blockIdx.x % GROUPS;
    const KvtJoin j = reinterpret_cast<const KvtJoin*>(p.counters)[c1];
    if (j.last == 0) return;
    constexpr int E = D / 32;
    for (int row = (g * 8 + warp) * each, end = min(j.rows, row + each); row < end; ++row) {
        float M = -FLT_MAX, L = 0.f, o[E] = {};
#pragma unroll 4
        for (int c = c1 - 1; c <= j.last; ++c) {
            const float* part = p.partials + (int64_t)(2 * c + (c == c1 - 1 ? 1 : 0)) * KvtPart<D>::FLOATS;
            const float2 ml = __ldcg(reinterpret_cast<const float2*>(part + KVT_ROWS * D) + row);
            float v[E];
            if constexpr (E == 4) {
                const float4 f = __ldcg(reinterpret_cast<const float4*>(part + row * D) + lane);
                v[0] = f.x; v[1] = f.y; v[2] = f.z; v[3] = f.w;
            } else {
                const float2 f = __ldcg(reinterpret_cast<const float2*>(part + row * D) + lane);
                v[0] = f.x; v[1] = f.y;
            }
            const float top = fmaxf(M, ml.x), a = ex2f(M - top), b = ex2f(ml.x - top);
            M = top;
            L = L * a + ml.y * b;
#pragma unroll
            for (int e = 0; e < E; ++e) o[e] = o[e] * a + v[e] * b;
        }
        const int i = j.row0 + row, t = i / p.grp;
        const int64_t out = ((int64_t)(j.tok0 + t) * p.h_q + j.h * p.grp + i - t * p.grp) * D + lane * E;
        const float f = L == 0.f ? 0.f : p.v_scale / L;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = L == 0.f ? 0.f : o[e] * f;
        if constexpr (E == 4) {
            st_elem4(p.o, out, p.dtype, o[0], o[1], o[2], o[3]);
        } else if (p.dtype == 0) {
            *reinterpret_cast<float2*>(static_cast<float*>(p.o) + out) = make_float2(o[0], o[1]);
        } else if (p.dtype == 1) {
            *reinterpret_cast<__half2*>(static_cast<__half*>(p.o) + out) = __floats2half2_rn(o[0], o[1]);
        } else {
            *reinterpret_cast<__nv_bfloat162*>(static_cast<__nv_bfloat16*>(p.o) + out) = __floats2bfloat162_rn(o[0], o[1]);
        }
    }
}

}  // namespace kda
