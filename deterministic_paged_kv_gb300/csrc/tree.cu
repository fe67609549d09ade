// tree.cu -- attention of a tree of drafted tokens behind each row's prefix, on the 5th-gen
// tensor cores (tcgen05 MMA into TMEM, TMA), RoPE applied to K as it is read.
//
// Mathematics: o_n = sum_t softmax_t(q_n . k_t / sqrt D) v_t over the prefix, n's ancestors and n
// itself; keys and queries rotated at their positions, a node's position being the prefix's length
// plus its depth.  The R = G T queries of a row's KV head (its G query heads x T nodes, one run of
// memory) are the rows of the accumulator, 128 to a q-tile, so every K and V byte serves them all.
//
// Keys: whole pages of the prefix in tiles of 128, then one tile of the tree: the prefix's last
// partly filled page and the nodes (at most 79 keys, 5 pages).  Only that tile needs masks (an
// ancestor set of 64 bits a node) and other angles than t's, and only there can a slot hold what some
// query must not touch: rows past the end and unused nodes are zeroed in V, and a node whose K or V is
// not finite fails the queries that see it.
//
// Splits: a row's prefix is cut at fixed tokens (TreeArgs::zone), the tree's tile belongs to the last
// part; a part leaves O / l and a log2-domain LSE in FP32, and the merge adds the parts up in an
// order that their number sets.  A row of one part writes its results itself.
// Work: items (row, KV head, block of 128 queries, part) on a persistent grid of one CTA per SM.  A head's
// items are dealt to its CTAs in runs of equal numbers of tiles (TrItems); a CTA keeps its queries over
// the parts of a row.  Which CTA runs an item never changes how.
//
// RR = 32, 64 or 128 is the number of queries that an item is padded to.  S = Q K^T has a query to each of
// the 128 lanes of tensor memory: 128 / RR copies of the queries, so that with two warpgroups 256 / RR threads
// share a query's row and each has RR / 2 of the tile's columns (a single copy of 32 queries took 5200
// cycles a tile in the one warp that had rows, where the tile's bytes take 3034).  P^T goes to shared memory
// as the N operand of O^T = V^T P^T, whose lanes are the output dims.
//
// Roles (512 threads):
//   warps 0-3    transform: rotate new queries and each K tile in place in shared memory (FP32, angles
//                from exact anchors and steps), FP16 for the score MMA;
//   warps 4-11   softmax: online, in the log2 domain; the running maximum moves when some query's grows by
//                more than 8 (a vote of the 256 threads says so; then the maxima are exchanged and O^T is
//                rescaled); P as BF16; epilogue, a thread one dim of RR / 2 queries;
//   warps 12, 14 TMA producers of K and V pages; warp 14 cleans the tree's V tile;
//   warp 13      MMA issuer: S of the next tile before PV of this one (S, and O^T by item, have two buffers);
//   warp 15      scheduler: walks the items, checks their metadata, publishes them.
// Four warps transform: with 8 (640 threads, 96 registers) 64 rows of 4096 took 202 us where they take 199, with 16 270; 4
// softmax warps instead of 8 took 197 there, and 128 instead of 113 for 104 queries a head.
// Loops are rolled: sixteen warps in six roles go through their code once a tile, and code of some hundred
// instructions in a row was fetched anew each time (an MMA issued every 150 cycles, a wait on a barrier that had
// completed took 300).
//
// Roundings: q and K to FP16 after the rotation (2^-11, as in the other BF16 calls; lse moves by 1e-5 to 1e-4), weights to BF16
// for P V (2^-9 each, and their sum is of the unrounded ones), out once to BF16; scores, maxima, sums, O and parts FP32.
//
// What bounds it (one GB300, in a replayed graph, merge included): 64 rows of 4096 and 8 nodes, 32 queries a head, 199 us =
// 5.45 TB/s, 80% of a copy's; 2 rows past 100000 and 64 queries 160 us, 80%: DRAM, the first load after 7000 cycles
// (3.7 us; instructions fetched for the first time, 170 cycles to a line of 8) and the merge (84 MB written and read, 12 us).
// 20 rows of 90 to 9001 and 104 queries 113 us, 8 rows of 2048 and 256 queries 55.5 us: the chain of a tile, 3200 cycles: S
// 300, its first half 880, PV of the tile before 230, the second half 1000 to 1100, the vote 200 to 600 (the last warp's share is the
// larger one), to the next wait 350; the rotation of its keys takes four warps 2000 to 2400 of them, and shared memory moves
// 288 KB (2300 cycles).  53% of the issue slots are used.  One row of 777 15 us: latency, 3.3 to the first load, 4 tiles of 1.2,
// merge.
#include <algorithm>
#include <atomic>
#include <cstring>

#include "q8_device.cuh"
#include "tree_args.h"

namespace rk {

namespace {

constexpr int TR_XW = 4, TR_SW = 8;                       // transform and softmax warps
constexpr int TR_SOFTMAX = TR_SW * 32;
constexpr int WARP_S0 = TR_XW, WARP_K = WARP_S0 + TR_SW, WARP_MMA = WARP_K + 1, WARP_V = WARP_K + 2, WARP_SCHED = WARP_K + 3;
constexpr int TR_THREADS = (WARP_SCHED + 1) * 32;
constexpr int TR_SPAN = 128;                              // queries of an item at most
constexpr int TR_BN = 128;                                // keys of a prefix tile
constexpr int TR_TILE_BYTES = TR_BN * HEAD_DIM * 2;       // 32 KiB
constexpr int TR_KSTAGES = 3, TR_VSTAGES = 2;
constexpr int TR_TREE_ROWS = 80;                          // keys of the tree's tile: 15 + 64, whole pages
constexpr float TR_SLACK = 8.0f;                          // the running max moves when it grows by more (log2)
constexpr int TR_SLOTS = 3;                               // items published ahead
constexpr int TR_ROW_STEP = TR_XW * 4;                    // rows between a transform thread's rows
constexpr int TR_ANCHOR = 4;                              // tiles between exact angles
constexpr int TR_GROUPS = 32;                             // row groups of the item search
// Sets of queries whose flags are kept.  The transform writes a set's in the set's first item e, after r_empty of item
// e - 1, which says that the results of items up to e - 3 are written.  Items e - 2 and e - 1, whose flags may still be
// read (with one tile each their scores, and so q_empty, run two items ahead of their results), hold at most the two
// sets before it.
constexpr int TR_QSETS = 3;

template <int RR>
struct TrShape {
    static constexpr int COPIES = TR_SPAN / RR;           // of the queries, in the lanes of S
    static constexpr int PARTS = 2 * COPIES;              // threads of a query's row of S
    static constexpr int COLS = TR_BN / PARTS;            // columns of each: RR / 2, and its queries in the epilogue
    static constexpr int PBUF = RR == 128 ? 1 : 2;        // buffers of P^T, as room allows
    static constexpr int P_BYTES = RR * TR_BN * 2;
    static constexpr int OFF_K = TR_TILE_BYTES;           // queries first
    static constexpr int OFF_V = OFF_K + TR_KSTAGES * TR_TILE_BYTES;
    static constexpr int OFF_P = OFF_V + TR_VSTAGES * TR_TILE_BYTES;
    static constexpr int OFF_CTRL = OFF_P + PBUF * P_BYTES;
    // tensor memory: S at 0 and 128, O^T at 256 and 256 + RR
    static constexpr uint32_t TMEM_COLS = 512;
};

// An item as the scheduler publishes it.
struct TrUnit {
    int end;                 // 1: no further item
    int b, kvh, block, split;
    int t0, n_keys;          // its prefix keys [t0, t0 + n_keys), whole pages
    int tree;                // 1: the tree's tile follows them
    int prefix;              // tokens before the tree
    int newq, nq;            // first item of its queries, their number in this CTA
    int direct;              // 1: the row has one part
    int rows;                // live queries of the item
};
struct TrSlot {
    TrUnit u;
    int8_t up[TREE_MAX];       // parents of the nodes (below 0: none)
    uint8_t depth[TREE_MAX];   // 255: unused
};

// A whole warp waits for a barrier's phase.  The first try suspends the warp as long as any later one; what follows it is
// a call, not code at each of the forty places that wait.
__device__ __noinline__ bool wait_longer(uint32_t bar, uint32_t parity, PipeCtl* pc) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, pc)) != 0;
}
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, PipeCtl* pc) {
    return __all_sync(0xffffffffu, mbar_try_wait(bar, parity)) || wait_longer(bar, parity, pc);
}

// ------------------------------------------------------------ geometry ----

// A row's prefix in whole pages, and why the row has none (status bits; kv_len 0: -1 and no bit).
template <class A>
__device__ __forceinline__ int row_pages16(const A& a, int b, int& kv, int& bad) {
    kv = a.kv_lens[b];
    bad = kv < 0 || kv > a.W * PAGE || (kv > 0 && kv < a.T) ? RK_STATUS_KVLEN : 0;
    return bad || kv == 0 ? -1 : (kv - a.T) & ~(PAGE - 1);
}
// Parts of a row with n prefix keys in whole pages (one where there are none).
template <class A>
__device__ __forceinline__ int parts_of(const A& a, int n) {
    if (n <= 0) return 1;
    const int z = n > a.zone[1].token;
    return a.zone[z].split + ((n - a.zone[z].token + (1 << a.zone[z].shift) - 1) >> a.zone[z].shift);
}
template <class A>
__device__ __forceinline__ int part_start(const A& a, int s) {
    const int z = s >= a.zone[1].split;
    return a.zone[z].token + ((s - a.zone[z].split) << a.zone[z].shift);
}
// Tiles of a row: its prefix's and the tree's (one for a row without keys, which is an item too).
__device__ __forceinline__ int row_tiles(int n) { return n < 0 ? 1 : (n + TR_BN - 1) / TR_BN + 1; }

// The items of a KV head and block of 128 queries are its rows' parts in order of row and part; they are dealt
// to `members` runs of equal numbers of tiles (a part belongs to the run that its first tile lies in), the same
// for every head, so that the CTAs of a row's heads read its pages, in which a token's heads are
// neighbours, at about the same time.  Run v of all is run v / heads of head v % heads; CTA c has the runs
// c, c + grid, ...
struct TrItems {
    int v, m, kvh, block;   // run: the m-th of its head and block of queries
    int b, s;               // row, part
    int kv, n, ns, bad;     // the row's length, prefix keys in whole pages, parts, status
    int at, hi;             // the part's first tile, the run's end
    __device__ __forceinline__ bool valid(const TreeArgs& a, int heads) const { return v < heads * a.members; }
    // (divisions that need no metadata)
    __device__ __forceinline__ void place(int run, int heads, int blocks) {
        v = run;
        m = v / heads;
        const int h = v - m * heads;
        kvh = blocks == 1 ? h : h / blocks;
        block = h - kvh * blocks;
    }
    __device__ __forceinline__ void row(const TreeArgs& a) {
        if (b < a.B) {
            n = row_pages16(a, b, kv, bad);
            ns = parts_of(a, n);
        }
    }
    // The first part of run v that there is, or of a later run of this CTA.
    __device__ __forceinline__ void find(const TreeArgs& a, int total, const int* pre, int heads, int blocks) {
#pragma unroll 1
        for (; valid(a, heads); place(v + (int)gridDim.x, heads, blocks)) {
            at = min(total, (int)((uint64_t)(unsigned)total * (a.share * (unsigned)m) >> 32));
            hi = min(total, (int)((uint64_t)(unsigned)total * (a.share * (unsigned)(m + 1)) >> 32));
            if (at >= hi) continue;
            const int per = (a.B + TR_GROUPS - 1) / TR_GROUPS;
            int lo = 0;  // the last group that begins at or before the tile (those without rows begin at the total)
#pragma unroll 1
            for (int half = TR_GROUPS / 2; half; half >>= 1)
                if (pre[lo + half] <= at) lo += half;
            b = lo * per;
            int base = pre[lo], rt;
#pragma unroll 1
            for (;; base += rt, ++b) {
                row(a);
                rt = row_tiles(n);
                if (at - base < rt || b + 1 >= a.B) break;
            }
            const int tile = at - base;
            s = tile ? parts_of(a, min(max(n, 0), tile * TR_BN)) : 0;  // the first part that starts at this tile or later
            if (s < ns) {
                at = base + part_start(a, s) / TR_BN;
            } else {
                at = base + rt;
                s = 0;
                ++b;
                row(a);
            }
            if (b < a.B && at < hi) return;
        }
    }
    // To the next part; true: of another run, to be found.
    __device__ __forceinline__ bool next(const TreeArgs& a, int heads, int blocks) {
        at -= part_start(a, s) / TR_BN;
        if (++s == ns) {
            at += row_tiles(n);
            s = 0;
            ++b;
            row(a);
        } else {
            at += part_start(a, s) / TR_BN;
        }
        const bool over = b >= a.B || at >= hi;
        if (over) place(v + (int)gridDim.x, heads, blocks);
        return over;
    }
};

struct TrCtrl {
    uint64_t q_ready, q_empty;
    uint64_t k_full[TR_KSTAGES], k_ready[TR_KSTAGES], k_empty[TR_KSTAGES];
    uint64_t v_full[TR_VSTAGES], v_empty[TR_VSTAGES], v_land;
    uint64_t s_full[2], s_free[2], p_ready[2], pv_done[2], o_done[2], o_free[2];
    uint64_t u_full[TR_SLOTS], u_empty[TR_SLOTS];
    uint64_t r_full[2], r_empty[2];
    uint64_t never;
    uint32_t tmem_base;
    PipeCtl pipe;
    int total;                        // tiles of the batch's rows (of one KV head and block)
    int pre[TR_GROUPS];               // tiles before each group of rows
    uint64_t vbad[2];                 // nodes whose V is not finite, by item parity
    alignas(4) uint8_t xbad[2][TR_XW];  // a transform warp met a prefix key out of range
    uint8_t kbad[2][TR_TREE_ROWS];    // keys of the tree's tile out of range
    uint8_t qbad[TR_QSETS][TR_SPAN / 4];  // queries out of range, four to a byte, by the set of queries
    alignas(16) TrSlot slot[TR_SLOTS];
    // exchange of the softmax threads: maxima, or scales of O^T, or an item's factors (its sums, of all parts
    // but the first, lie behind this block)
    alignas(16) float ex[TR_SOFTMAX];
};
template <int RR>
constexpr int tr_smem_bytes() {
    constexpr int bytes = TrShape<RR>::OFF_CTRL + (int)sizeof(TrCtrl) + (TrShape<RR>::PARTS - 1) * RR * 4;
    static_assert(bytes <= 232448, "tree attention shared memory above the 227 KiB opt-in limit");
    return bytes;
}

// First query of (row b, KV head kvh) in q, out and lse: its G heads x T nodes follow one another.
__device__ __forceinline__ size_t first_row(const TreeArgs& a, int b, int kvh) { return ((size_t)b * a.Hkv + kvh) * (size_t)(a.G * a.T); }

// An item that nothing is computed for (count threads, i of them): a part that says NaN or -inf,
// or the results themselves.
__device__ __noinline__ void write_nothing(const TreeArgs& a, int b, int kvh, int block, int split, bool direct, float lse, int i, int count) {
    const int R = a.G * a.T, r0 = block * TR_SPAN, rows = min(TR_SPAN, R - r0);
    if (!direct) {
        float* lp = a.lse_part + ((first_row(a, b, kvh) + r0) * a.n_splits + split);
        for (int r = i; r < rows; r += count) lp[(size_t)r * a.n_splits] = lse;
        return;
    }
    uint4* o = reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(a.out) + (first_row(a, b, kvh) + r0) * HEAD_DIM);
    for (int k = i; k < rows * (HEAD_DIM / 8); k += count) o[k] = make_uint4(0, 0, 0, 0);
    for (int r = i; r < rows; r += count) a.lse[first_row(a, b, kvh) + r0 + r] = lse * 0.693147180559945309f;
}

// D[tmem] (+)= A[smem] * B[smem], the first kn of 4 k-steps of 16 values, accumulating from the second on, and at
// the first iff acc0.  Called by a whole converged warp with uniform operands; one elected lane issues.  a_lo, b_lo:
// low descriptor words of the first k-step; A_STEP, B_STEP (16-byte units) lead to the next.
template <uint32_t A_STEP, uint32_t B_STEP>
__device__ __forceinline__ void mma_f16_x4(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, uint32_t acc0, int kn) {
    asm volatile(
        "{\n\t.reg .pred p, e, t, k;\n\t.reg .b32 al, bl;\n\t.reg .b64 da, db;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "setp.ne.b32 p, %5, 0;\n\tsetp.eq.b32 t, %5, %5;\n\t"
        "mov.b64 da, {%1, %3};\n\tmov.b64 db, {%2, %3};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %4, p;\n\t"
        "add.u32 al, %1, %7;\n\tadd.u32 bl, %2, %8;\n\tmov.b64 da, {al, %3};\n\tmov.b64 db, {bl, %3};\n\t"
        "setp.gt.and.s32 k, %6, 1, e;\n\t"
        "@k tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %4, t;\n\t"
        "add.u32 al, al, %7;\n\tadd.u32 bl, bl, %8;\n\tmov.b64 da, {al, %3};\n\tmov.b64 db, {bl, %3};\n\t"
        "setp.gt.and.s32 k, %6, 2, e;\n\t"
        "@k tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %4, t;\n\t"
        "add.u32 al, al, %7;\n\tadd.u32 bl, bl, %8;\n\tmov.b64 da, {al, %3};\n\tmov.b64 db, {bl, %3};\n\t"
        "setp.gt.and.s32 k, %6, 3, e;\n\t"
        "@k tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %4, t;\n\t}" ::"r"(d),
        "r"(a_lo), "r"(b_lo), "r"(DESC_HI), "r"(idesc), "r"(acc0), "r"(kn), "n"(A_STEP), "n"(B_STEP)
        : "memory");
}

// One box of a 4-D map, by one elected lane of a converged warp, operands uniform.
__device__ __forceinline__ void tma_load_4d_elect(uint32_t dst, const CUtensorMap* m, uint32_t bar, int c0, int c1, int c2, int c3, uint64_t policy) {
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%3, %4, %5, %6}], [%2], %7;\n\t}" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "l"(policy)
        : "memory");
}

__device__ __forceinline__ float2 fsub2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 ra, rb, rd;\n\t"
        "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
        "sub.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
// Angles of eight rotation pairs as (cos, -sin): with the sine's sign turned a step needs no negation, and a rotation one
// difference.
struct Turn {
    float2 c[4], n[4];
    // by a fixed step of (dc, -ds = dn, ds): c' = c dc - s ds, -s' = -s dc - c ds
    __device__ __forceinline__ void step(const float2 (&dc)[4], const float2 (&dn)[4], const float2 (&ds)[4]) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float2 cn = ffma2(n[k], ds[k], fmul2(c[k], dc[k]));
            n[k] = ffma2(c[k], dn[k], fmul2(n[k], dc[k]));
            c[k] = cn;
        }
    }
};
// Eight rotation pairs (16 bf16) in FP32, to FP16 in place: (lo, hi) -> (lo c - hi s, hi c + lo s).  rs, ru: running
// signed and unsigned maxima of the inputs' bits, the largest positive and (if any is below 0) negative one.
__device__ __forceinline__ void rotate(uint4& a, uint4& b, const Turn& t, uint32_t& rs, uint32_t& ru) {
    uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        rs = __vimax3_s16x2(rs, x[k], y[k]);
        ru = __vimax3_u16x2(ru, x[k], y[k]);
        const float2 lo = make_float2(bf16lo(x[k]), bf16hi(x[k])), hi = make_float2(bf16lo(y[k]), bf16hi(y[k]));
        const float2 u = ffma2(hi, t.n[k], fmul2(lo, t.c[k])), v = fsub2(fmul2(hi, t.c[k]), fmul2(lo, t.n[k]));
        x[k] = pack_f16x2(u.x, u.y);
        y[k] = pack_f16x2(v.x, v.y);
    }
    a = make_uint4(x[0], x[1], x[2], x[3]);
    b = make_uint4(y[0], y[1], y[2], y[3]);
}
// Did an input reach 2^15 (or was it no number)?
__device__ __forceinline__ bool too_large(uint32_t rs, uint32_t ru) {
    return max((int16_t)rs, (int16_t)(rs >> 16)) >= (int)RANGE_LIMIT_BF16 || max(ru & 0xffffu, ru >> 16) >= (RANGE_LIMIT_BF16 | 0x8000u);
}

// Keys of tile i of an item (whole pages).
__device__ __forceinline__ int tile_keys(int i, int n_keys, int prefix, int T) {
    const int left = n_keys - i * TR_BN;
    return left > 0 ? min(TR_BN, left) : ((prefix & (PAGE - 1)) + T + PAGE - 1) & ~(PAGE - 1);
}

template <int RR>
__global__ void __launch_bounds__(TR_THREADS, 1)
    tree_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap, const __grid_constant__ TreeArgs a) {
    extern __shared__ __align__(1024) uint8_t sm[];
    using Sh = TrShape<RR>;
    TrCtrl* c = reinterpret_cast<TrCtrl*>(sm + Sh::OFF_CTRL);
    const uint32_t s_base = smem_u32(sm);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int T = a.T, R = a.G * T;
    const int blocks = (R + TR_SPAN - 1) / TR_SPAN, heads = a.Hkv * blocks;
    griddep_launch_dependents();                          // the merge may become resident; it waits for this grid's end

    if (tid == 0) {
        c->pipe.abort = 0;
        c->pipe.limit_ns = wait_limit(a.wait_limit_ns);
        mbar_init(smem_u32(&c->never), 1);
        mbar_init(smem_u32(&c->q_ready), TR_XW);
        mbar_init(smem_u32(&c->q_empty), 1);
        for (int k = 0; k < TR_KSTAGES; ++k) {
            mbar_init(smem_u32(&c->k_full[k]), 1);
            mbar_init(smem_u32(&c->k_ready[k]), TR_XW);
            mbar_init(smem_u32(&c->k_empty[k]), 1);
        }
        for (int k = 0; k < TR_VSTAGES; ++k) {
            mbar_init(smem_u32(&c->v_full[k]), 1);
            mbar_init(smem_u32(&c->v_empty[k]), 1);
        }
        mbar_init(smem_u32(&c->v_land), 1);
        for (int j = 0; j < 2; ++j) {
            mbar_init(smem_u32(&c->s_full[j]), 1);
            mbar_init(smem_u32(&c->s_free[j]), TR_SW);
            mbar_init(smem_u32(&c->p_ready[j]), TR_SW);
            mbar_init(smem_u32(&c->pv_done[j]), 1);
            mbar_init(smem_u32(&c->o_done[j]), 1);
            mbar_init(smem_u32(&c->o_free[j]), TR_SW);
            mbar_init(smem_u32(&c->r_full[j]), TR_XW + 1);
            mbar_init(smem_u32(&c->r_empty[j]), TR_SW);
        }
        for (int k = 0; k < TR_SLOTS; ++k) {
            mbar_init(smem_u32(&c->u_full[k]), 1);
            mbar_init(smem_u32(&c->u_empty[k]), 3 + TR_XW + TR_SW);  // producers, issuer, transform, softmax warps
        }
        fence_mbar_init();
    }
    if (warp == WARP_MMA) {
        tmem_alloc(smem_u32(&c->tmem_base), Sh::TMEM_COLS);
        tmem_relinquish();
    }
    TrItems it;                                           // the scheduler's
    if (warp == WARP_SCHED) it.place((int)blockIdx.x, heads, blocks);
    {
        // Tiles before each group of `per` rows: a group to sixteen threads.
        const int per = (a.B + TR_GROUPS - 1) / TR_GROUPS;
        int cnt = 0;
        for (int i = tid & 15, b = (tid >> 4) * per + i; i < per && b < a.B; i += 16, b += 16) {
            int kv, bad;
            cnt += row_tiles(row_pages16(a, b, kv, bad));
        }
#pragma unroll
        for (int o = 1; o < 16; o <<= 1) cnt += __shfl_xor_sync(0xffffffffu, cnt, o);
        if ((tid & 15) == 0 && (tid >> 4) < TR_GROUPS) c->pre[tid >> 4] = cnt;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = c->tmem_base;
    PipeCtl* pc = &c->pipe;
    int done = 0;                                         // softmax: items written

    auto wait_all = [&](uint64_t& bar, int parity) { return wait_warp(smem_u32(&bar), (uint32_t)(parity & 1), pc); };

    if (warp >= WARP_K) {
        if (warp == WARP_SCHED) {
            // ============================================== scheduler ====
            {
                // Sums to offsets, by the warp that needs them: nothing else waits for them.
                const int own = c->pre[lane];
                int sum = own;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int t = __shfl_up_sync(0xffffffffu, sum, o);
                    if (lane >= o) sum += t;
                }
                c->pre[lane] = sum - own;
                if (lane == 31) c->total = sum;
                __syncwarp();
            }
            int k = 0, nq = -1, tree_row = -1;            // published items, queries; row whose tree is in registers
            int up0[2] = {-1, -1}, deep[2] = {255, 255};  // of nodes lane, lane + 32
            int tree_bad = 0;
            int lb = -1, lv = -1;                         // queries of the item before
            bool ok = true, past = false;                 // past: `it` is done with
            // checks the item `it`; 0: to be published
            auto judge = [&]() -> int {
                int bad = it.bad;
                if (bad || it.n < 0) return bad;
                // page ids of the item's keys (up to 69; most on their way while the tree is looked at)
                const int t0 = part_start(a, it.s), end = it.s + 1 < it.ns ? part_start(a, it.s + 1) : it.kv;
                const int32_t* bt = a.block_table + (size_t)it.b * a.W;
                const int p0 = t0 / PAGE + lane, p1 = (end + PAGE - 1) / PAGE;
                const int first = p0 < p1 ? __ldg(bt + p0) : 0, second = p0 + 32 < p1 ? __ldg(bt + p0 + 32) : 0;
                if (tree_row != it.b) {
                    tree_row = it.b;
                    int p[2], up[2];
                    const int32_t* par = a.parents + (size_t)it.b * T;
#pragma unroll
                    for (int e = 0; e < 2; ++e) p[e] = lane + 32 * e < T ? par[lane + 32 * e] : TREE_UNUSED;
                    auto of = [&](const int (&x)[2], int n) {  // node n's value
                        const int lo = __shfl_sync(0xffffffffu, x[0], n & 31), hi = __shfl_sync(0xffffffffu, x[1], n & 31);
                        return n & 32 ? hi : lo;
                    };
                    int wrong = 0;
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int n = lane + 32 * e;
                        wrong |= p[e] < TREE_UNUSED || (p[e] >= n && p[e] >= 0);
                        const int pp = of(p, p[e] & 63);
                        wrong |= p[e] >= 0 && pp == TREE_UNUSED;
                        up[e] = up0[e] = p[e];
                        deep[e] = p[e] >= 0 ? 1 : 0;
                    }
                    tree_bad = __any_sync(0xffffffffu, wrong) ? RK_STATUS_TREE : 0;
                    // depths: steps to `up`, twice as far up with every turn
#pragma unroll 1
                    for (int turn = 0; turn < 6 && !tree_bad && __any_sync(0xffffffffu, up[0] >= 0 || up[1] >= 0); ++turn) {
                        int add[2], far[2];
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            add[e] = of(deep, up[e] & 63);
                            far[e] = of(up, up[e] & 63);
                        }
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            deep[e] += up[e] >= 0 ? add[e] : 0;
                            up[e] = up[e] >= 0 ? far[e] : -1;
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        if (p[e] == TREE_UNUSED) deep[e] = 255;
                }
                bad |= tree_bad;
                int oob = (unsigned)first >= (unsigned)a.num_pages || (unsigned)second >= (unsigned)a.num_pages;
                for (int i = p0 + 64; i < p1; i += 32) oob |= (unsigned)__ldg(bt + i) >= (unsigned)a.num_pages;
                if (__any_sync(0xffffffffu, oob)) bad |= RK_STATUS_PAGE_OOB;
                return bad;
            };
#pragma unroll 1
            while (ok) {
                // the next item that has something to compute; those that have not are written here
#pragma unroll 1
                for (;; past = true) {
                    if (!past || it.next(a, heads, blocks)) it.find(a, c->total, c->pre, heads, blocks);
                    if (!it.valid(a, heads)) break;
                    const int bad = judge();
                    if (!bad && it.n >= 0) break;
                    if (bad && lane == 0 && a.status) atomicOr(a.status, bad);
                    write_nothing(a, it.b, it.kvh, it.block, it.s, it.ns == 1, bad ? __int_as_float(0x7fc00000) : -INFINITY, lane, 32);
                }
                past = true;
                TrUnit u;
                std::memset(&u, 0, sizeof u);
                u.end = !it.valid(a, heads);
                const int u0 = up0[0], u1 = up0[1], d0 = deep[0], d1 = deep[1];
                if (!u.end) {
                    u.b = it.b;
                    u.kvh = it.kvh;
                    u.block = it.block;
                    u.split = it.s;
                    u.t0 = part_start(a, it.s);
                    u.tree = it.s + 1 == it.ns;
                    u.n_keys = (u.tree ? it.n : part_start(a, it.s + 1)) - u.t0;
                    u.prefix = it.kv - T;
                    u.direct = it.ns == 1;
                    u.rows = min(TR_SPAN, R - u.block * TR_SPAN);
                    u.newq = it.b != lb || it.v != lv;
                    nq += u.newq;
                    u.nq = nq;
                    lb = it.b;
                    lv = it.v;
                }
                TrSlot* s = &c->slot[k % TR_SLOTS];
                const int use = k / TR_SLOTS;
                if (!(ok = wait_all(c->u_empty[k % TR_SLOTS], use + 1))) break;
                s->up[lane] = (int8_t)u0;
                s->up[lane + 32] = (int8_t)u1;
                s->depth[lane] = (uint8_t)d0;
                s->depth[lane + 32] = (uint8_t)d1;
                if (lane == 0) s->u = u;
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&c->u_full[k % TR_SLOTS]));
                ++k;
                if (u.end) break;
            }
        } else if (warp == WARP_K || warp == WARP_V) {
            // ========================================= producers ====
            // The whole warp, converged: the copies' operands stay in uniform registers, one elected lane issues.
            const bool is_k = warp == WARP_K;
            if (lane == 0) prefetch_tmap(is_k ? &kmap : &vmap);
            const int stages = is_k ? TR_KSTAGES : TR_VSTAGES;
            uint64_t* full = is_k ? c->k_full : c->v_full;
            uint64_t* empty = is_k ? c->k_empty : c->v_empty;
            const uint32_t ring = s_base + (is_k ? Sh::OFF_K : Sh::OFF_V);
            const uint64_t once = evict_first_policy();  // the cache passes by; the parts stay in L2 for the merge
            int n = 0, st = 0, nl = 0;  // tiles issued, their stage, tree tiles that went through v_land
            uint32_t phase = 1;
            bool land_open = false, ok = true;
#pragma unroll 1
            for (int k = 0; ok; ++k) {
                TrSlot* s = &c->slot[k % TR_SLOTS];
                if (!(ok = wait_all(c->u_full[k % TR_SLOTS], k / TR_SLOTS))) break;
                const TrUnit u = s->u;
                if (u.end) break;
                const int npt = (u.n_keys + TR_BN - 1) / TR_BN, n_tiles = npt + u.tree;
                const int32_t* bt = a.block_table + (size_t)u.b * a.W + u.t0 / PAGE;
                auto page_ids = [&](int i) {  // lane p: page p of tile i (the tree's begins where the prefix's whole pages end)
                    const int np = tile_keys(i, u.n_keys, u.prefix, T) / PAGE, p0 = i < npt ? i * (TR_BN / PAGE) : u.n_keys / PAGE;
                    return i < n_tiles && lane < np ? __ldg(bt + p0 + lane) : 0;
                };
                int ids = page_ids(0);
#pragma unroll 1
                for (int i = 0; i < n_tiles; ++i, ++n) {
                    const int keys = tile_keys(i, u.n_keys, u.prefix, T), np = __shfl_sync(0xffffffffu, keys / PAGE, 0);
                    const int next = page_ids(i + 1);
                    if (!(ok = wait_warp(smem_u32(&empty[st]), phase, pc))) break;
                    const bool clean = !is_k && i >= npt;
                    const uint32_t lb = smem_u32(clean ? &c->v_land : &full[st]);
                    arrive_expect_tx_elect(lb, (uint32_t)np * 4096);
                    uint32_t dst = ring + st * TR_TILE_BYTES;
                    const int head = __shfl_sync(0xffffffffu, u.kvh, 0);
                    if (is_k) {  // two 16 x 64 boxes per page: the K-major tile layout
#pragma unroll 1
                        for (int p = 0; p < np; ++p, dst += 2048) {
                            const int row = __shfl_sync(0xffffffffu, ids, p) * PAGE;
                            tma_load_3d_elect(dst, &kmap, lb, 0, head, row, once);
                            tma_load_3d_elect(dst + 16384, &kmap, lb, 64, head, row, once);
                        }
                    } else {     // one 4 KiB box per page: [page][half][16 rows][128 B]
#pragma unroll 1
                        for (int p = 0; p < np; ++p, dst += 4096)
                            tma_load_4d_elect(dst, &vmap, lb, 0, __shfl_sync(0xffffffffu, ids, p) * PAGE, 0, head, once);
                    }
                    ids = next;
                    const int here = st;
                    if (++st == stages) {
                        st = 0;
                        phase ^= 1;
                    }
                    if (!clean) continue;
                    // The tree's V: rows past the last node and unused nodes hold anything, and 0 times that need not
                    // be 0; a node whose V is not finite is zeroed too and fails who sees it.
                    if (!(ok = wait_all(c->v_land, nl))) {
                        land_open = true;
                        break;
                    }
                    ++nl;
                    const int off = u.prefix & (PAGE - 1);
                    uint8_t* vt = sm + Sh::OFF_V + here * TR_TILE_BYTES;
                    uint64_t bad = 0;
                    if (!(ok = wait_all(c->r_empty[k & 1], (k >> 1) + 1))) break;
#pragma unroll 1
                    for (int r0 = off; r0 < keys; r0 += 2) {  // two rows a turn, 16 bytes a lane
                        const int r = r0 + (lane >> 4), ch = lane & 15, node = r - off;
                        uint4* x = reinterpret_cast<uint4*>(vt + (r >> 4) * 4096 + (ch >> 3) * 2048 + (r & 15) * 128 + (((ch & 7) ^ (r & 7)) << 4));
                        const bool in = r < keys, real = in && node < T && s->depth[node & 63] != 255;
                        uint32_t m = 0;
                        if (real) {
                            const uint4 y = *x;
                            m = __vmaxu2(__vmaxu2(y.x & 0x7fff7fffu, y.y & 0x7fff7fffu), __vmaxu2(y.z & 0x7fff7fffu, y.w & 0x7fff7fffu));
                        }
                        const bool off_range = (m & 0xffffu) >= 0x7f80u || (m >> 16) >= 0x7f80u;
                        const uint32_t hit = __ballot_sync(0xffffffffu, off_range);
                        const bool mine = (hit >> (lane & 16)) & 0xffffu;
                        if (in && (!real || mine)) *x = make_uint4(0, 0, 0, 0);
                        if (hit & 0xffffu) bad |= 1ull << ((r0 - off) & 63);
                        if (hit >> 16) bad |= 1ull << ((r0 + 1 - off) & 63);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        c->vbad[k & 1] = bad;
                        mbar_arrive(smem_u32(&c->v_full[here]));
                    }
                }
                if (!ok) break;
                if (!is_k && !u.tree && !(ok = wait_all(c->r_empty[k & 1], (k >> 1) + 1))) break;
                if (lane == 0) {
                    if (!is_k) mbar_arrive(smem_u32(&c->r_full[k & 1]));
                    mbar_arrive(smem_u32(&c->u_empty[k % TR_SLOTS]));
                }
            }
            if (lane == 0 && pipe_aborted(pc)) {
                // copies in flight land before the CTA's shared memory is released
                if (land_open) mbar_wait_drain(smem_u32(&c->v_land), (uint32_t)(nl & 1));
                for (int i = max(0, n - stages); i < n; ++i) mbar_wait_drain(smem_u32(&full[i % stages]), (uint32_t)((i / stages) & 1));
            }
        } else if (warp == WARP_MMA) {
            // ============================================= MMA issuer ====
            // The whole warp, converged, so that the operands stay in uniform registers; one elected lane issues.
            constexpr uint32_t idO = idesc_bf16_f32(HEAD_DIM, RR, 1, 0);
            constexpr uint32_t TILE_DESC = TR_TILE_BYTES >> 4;
            const uint32_t dQ = desc_lo(s_base, 16), dK0 = desc_lo(s_base + Sh::OFF_K, 16);
            const uint32_t dV0 = desc_lo(s_base + Sh::OFF_V, 2048), dP0 = desc_lo(s_base + Sh::OFF_P, 16);
            int g = 0, freed = 0;  // tiles so far, sets of queries given back
            bool ok = !a.timeout_drill || __all_sync(0xffffffffu, drill_wait(smem_u32(&c->never), pc));
            for (int k = 0; ok; ++k) {
                if (!(ok = wait_all(c->u_full[k % TR_SLOTS], k / TR_SLOTS))) break;
                const volatile TrUnit* su = &c->slot[k % TR_SLOTS].u;
                auto uni = [](int x) { return __shfl_sync(0xffffffffu, x, 0); };
                const int end = uni(su->end), n_keys = uni(su->n_keys), tree = uni(su->tree), prefix = uni(su->prefix);
                const int newq = uni(su->newq), nq = uni(su->nq);
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&c->u_empty[k % TR_SLOTS]));
                if (end) break;
                const int n_tiles = (n_keys + TR_BN - 1) / TR_BN + tree;
                if (newq) {
                    if (nq > freed) {  // the queries before have been read
                        umma_commit_elect(smem_u32(&c->q_empty));
                        freed = nq;
                    }
                    if (!(ok = wait_all(c->q_ready, nq))) break;
                }
                // PV of tile i, number x of the CTA
                auto issue_pv = [&](int i, int x) -> bool {
                    if (i == 0 && !wait_all(c->o_free[k & 1], (k >> 1) + 1)) return false;  // the buffer's item before has been read
                    if (!wait_all(c->p_ready[x % Sh::PBUF], x / Sh::PBUF)) return false;
                    if (!wait_all(c->v_full[x % TR_VSTAGES], x / TR_VSTAGES)) return false;
                    tc_fence_after();
                    const int pages = tile_keys(i, n_keys, prefix, T) / PAGE;
                    const uint32_t dv = dV0 + (uint32_t)(x % TR_VSTAGES) * TILE_DESC, dp = dP0 + (uint32_t)(x % Sh::PBUF) * (Sh::P_BYTES >> 4);
                    // O^T[dims x RR] += V^T P^T, a page to a k-step: V as the pages lie there (MN-major), P^T's rows as
                    // two blocks of 64 keys (K-major)
#pragma unroll 1
                    for (int h = 0; 4 * h < pages; ++h)
                        mma_f16_x4<256, 2>(tmem + 256 + (k & 1) * RR, dv + h * 1024, dp + h * (RR * 128 >> 4), idO, i > 0 || h > 0, pages - 4 * h);
                    umma_commit_elect(smem_u32(&c->pv_done[x & 1]));
                    umma_commit_elect(smem_u32(&c->v_empty[x % TR_VSTAGES]));
                    if (i == n_tiles - 1) umma_commit_elect(smem_u32(&c->o_done[k & 1]));
                    return true;
                };
#pragma unroll 1
                for (int i = 0; i <= n_tiles; ++i, ++g) {
                    if (i < n_tiles) {
                        const uint32_t idS = idesc_f16_f32(128, tile_keys(i, n_keys, prefix, T));
                        if (!(ok = wait_all(c->k_ready[g % TR_KSTAGES], g / TR_KSTAGES))) break;
                        if (!(ok = wait_all(c->s_free[g & 1], (g >> 1) + 1))) break;
                        tc_fence_after();
#pragma unroll 1
                        for (int h = 0; h < 2; ++h)
                            mma_f16_x4<2, 2>(tmem + (g & 1) * 128, dQ + h * 1024, dK0 + (uint32_t)(g % TR_KSTAGES) * TILE_DESC + h * 1024, idS, h, 4);
                        umma_commit_elect(smem_u32(&c->s_full[g & 1]));
                        umma_commit_elect(smem_u32(&c->k_empty[g % TR_KSTAGES]));
                        if (i == n_tiles - 1 &&
                            __all_sync(0xffffffffu, mbar_test(smem_u32(&c->u_full[(k + 1) % TR_SLOTS]), (uint32_t)((k + 1) / TR_SLOTS) & 1u))) {
                            // the next item is known: if it has other queries, these have been read by the scores so far
                            const volatile TrUnit* nu = &c->slot[(k + 1) % TR_SLOTS].u;
                            const int other = uni(nu->newq), num = uni(nu->nq), none = uni(nu->end);
                            if (!none && other) {
                                umma_commit_elect(smem_u32(&c->q_empty));
                                freed = num;
                            }
                        }
                    }
                    if (i > 0 && !(ok = issue_pv(i - 1, g - 1))) break;
                }
                --g;  // the last turn had no tile
            }
            if (!ok) {  // issued MMAs drain before tensor memory is released
                const uint64_t t0 = global_timer_ns();
                while (global_timer_ns() - t0 < 1000000ull) {
                }
            }
        }
        __syncwarp();
    } else if (warp < TR_XW) {
        // ================================================ transform ====
        // thread: pair-chunk u8 (8 rotation pairs: 16 bytes of each 64-dim half) of rows r0 + ROW_STEP * m
        const int u8 = tid & 7, r0 = tid >> 3;
        constexpr int ROWS = TR_BN / TR_ROW_STEP;
        auto angles = [&](uint32_t pos, Turn& t) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                rope_cos_sin(pos, a.rope_turns[8 * u8 + 2 * e], t.c[e].x, t.n[e].x);
                rope_cos_sin(pos, a.rope_turns[8 * u8 + 2 * e + 1], t.c[e].y, t.n[e].y);
                t.n[e] = make_float2(-t.n[e].x, -t.n[e].y);
            }
        };
        Turn step;
        angles((uint32_t)TR_ROW_STEP, step);
        float2 dsn[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) dsn[e] = make_float2(-step.n[e].x, -step.n[e].y);
        // a row's verdict from the eight threads that hold it
        auto any8 = [&](bool x) {
            const uint32_t b = __ballot_sync(0xffffffffu, x);
            return ((b >> (lane & 24)) & 0xffu) != 0;
        };
        bool ok = true;
        int g = 0;
        for (int k = 0; ok; ++k) {
            TrSlot* s = &c->slot[k % TR_SLOTS];
            if (!(ok = wait_all(c->u_full[k % TR_SLOTS], k / TR_SLOTS))) break;
            const volatile TrUnit* u = &s->u;
            if (u->end) break;
            const int n_keys = u->n_keys, prefix = u->prefix, t0 = u->t0, tree = u->tree;
            const int npt = (n_keys + TR_BN - 1) / TR_BN;
            Turn at;
            if (u->newq) {
                // new queries, once the score MMAs have read the ones before: COPIES of them, zeros behind the last
                const int nq = u->nq, rows = u->rows, base = u->block * TR_SPAN;
                const uint4* q = reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(a.q) +
                                                                (first_row(a, u->b, u->kvh) + base) * HEAD_DIM);
                // (a row's data is asked for while the row before is rotated)
                uint4 lo = make_uint4(0, 0, 0, 0), hi = lo;
                auto row = [&](int r) {
                    if (r < rows) {
                        lo = __ldg(q + r * 16 + u8);
                        hi = __ldg(q + r * 16 + 8 + u8);
                    } else {
                        lo = hi = make_uint4(0, 0, 0, 0);
                    }
                };
                row(r0);
                if (!(ok = wait_all(c->q_empty, nq + 1))) break;
#pragma unroll 1
                for (int r = r0; r < RR; r += TR_ROW_STEP) {
                    uint4 x = lo, y = hi;
                    row(r + TR_ROW_STEP);
                    const int d = r < rows ? s->depth[(base + r) % T] : 255;
                    angles((uint32_t)(prefix + (d == 255 ? 0 : d)), at);
                    uint32_t rs = 0, ru = 0;
                    rotate(x, y, at, rs, ru);
#pragma unroll
                    for (int e = 0; e < Sh::COPIES; ++e) {
                        uint8_t* qt = sm + sw128_off(e * RR + r, u8);
                        *reinterpret_cast<uint4*>(qt) = x;
                        *reinterpret_cast<uint4*>(qt + 16384) = y;
                    }
                    const uint32_t bad = __ballot_sync(0xffffffffu, too_large(rs, ru));
                    if (lane == 0)
                        c->qbad[nq % TR_QSETS][r >> 2] = (uint8_t)(((bad & 0xffu) != 0) | ((bad & 0xff00u) != 0) << 1 | ((bad & 0xff0000u) != 0) << 2 | (bad >> 24 != 0) << 3);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&c->q_ready));
            }
            uint32_t rs = 0, ru = 0;       // largest positive, largest negative input (bits) of the prefix's keys
            if (!(ok = wait_all(c->r_empty[k & 1], (k >> 1) + 1))) break;
            for (int i = 0; i < npt; ++i, ++g) {
                const int kst = g % TR_KSTAGES;
                if ((i & (TR_ANCHOR - 1)) == 0) angles((uint32_t)(t0 + i * TR_BN + r0), at);
                if (!(ok = wait_all(c->k_full[kst], g / TR_KSTAGES))) break;
                uint8_t* kt = sm + Sh::OFF_K + kst * TR_TILE_BYTES;
                const int keys = min(TR_BN, n_keys - i * TR_BN);
                // row r0 + 16 m is chunk u8 ^ (r0 & 7) of its 128 bytes for every m
                uint8_t* row = kt + sw128_off(r0, u8);
                uint4 lo = *reinterpret_cast<const uint4*>(row), hi = *reinterpret_cast<const uint4*>(row + 16384);
#pragma unroll 2
                for (int m = 0; m < ROWS; ++m, row += TR_ROW_STEP * 128) {
                    uint4 x = lo, y = hi;
                    if (m + 1 < ROWS) {  // the next row is read while this one is rotated
                        lo = *reinterpret_cast<const uint4*>(row + TR_ROW_STEP * 128);
                        hi = *reinterpret_cast<const uint4*>(row + TR_ROW_STEP * 128 + 16384);
                    }
                    if (r0 + TR_ROW_STEP * m < keys) {
                        rotate(x, y, at, rs, ru);
                        *reinterpret_cast<uint4*>(row) = x;
                        *reinterpret_cast<uint4*>(row + 16384) = y;
                    }
                    at.step(step.c, step.n, dsn);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&c->k_ready[kst]));
            }
            if (!ok) break;
            if (tree) {
                // the prefix's last page at its positions, the nodes at theirs; unused ones stay as they are (masked)
                const int kst = g % TR_KSTAGES, off0 = prefix & (PAGE - 1), last = off0 + T;
                if (!(ok = wait_all(c->k_full[kst], g / TR_KSTAGES))) break;
                uint8_t* kt = sm + Sh::OFF_K + kst * TR_TILE_BYTES;
#pragma unroll 1
                for (int rr = 0; rr < last; rr += TR_ROW_STEP) {
                    const int r = rr + r0, node = r - off0;
                    // (d: how far from the end of the prefix; the page's own keys lie before it)
                    const int d = node < 0 ? node : r < last ? s->depth[node] : 255;
                    uint32_t ns = 0, nu = 0;
                    if (d != 255) {
                        angles((uint32_t)(prefix + d), at);
                        const uint32_t off = sw128_off(r, u8);
                        uint4 lo = *reinterpret_cast<const uint4*>(kt + off), hi = *reinterpret_cast<const uint4*>(kt + 16384 + off);
                        rotate(lo, hi, at, ns, nu);
                        *reinterpret_cast<uint4*>(kt + off) = lo;
                        *reinterpret_cast<uint4*>(kt + 16384 + off) = hi;
                    }
                    const bool bad = any8(node >= 0 && too_large(ns, nu));
                    if (node < 0) {
                        rs = __vmaxs2(rs, ns);
                        ru = __vmaxu2(ru, nu);
                    }
                    if (u8 == 0 && r < TR_TREE_ROWS) c->kbad[k & 1][r] = bad;
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&c->k_ready[kst]));
                ++g;
            }
            const bool bad = __any_sync(0xffffffffu, too_large(rs, ru));
            if (lane == 0) {
                c->xbad[k & 1][warp] = bad;
                mbar_arrive(smem_u32(&c->r_full[k & 1]));
                mbar_arrive(smem_u32(&c->u_empty[k % TR_SLOTS]));
            }
        }
    } else {
        // ================================================== softmax ====
        constexpr int COLS = Sh::COLS, PARTS = Sh::PARTS, CH = 16;    // CH: columns at a time
        const int t = tid - 32 * WARP_S0, wg = t >> 7, ln = t & 127;  // warpgroup, lane of tensor memory
        const int r = ln % RR, part = wg * Sh::COPIES + ln / RR;      // the thread's query, which of its threads it is
        const uint32_t lane_addr = (uint32_t)((warp & 3) * 32) << 16;
        const float scl = a.qk_scale_log2;
        int g = 0;                                        // tiles so far
        bool ok = true;
        // The warps leave together: one whose wait gave up goes on to the next barrier, where all of them learn it, and
        // no way out lies anywhere but behind one.
        auto wait = [&](uint64_t& bar, int parity) {
            if (ok) ok = wait_all(bar, parity);
        };
        auto failed = [&]() -> bool {
            if (named_bar_or(1, TR_SOFTMAX, !ok)) ok = false;
            return !ok;
        };
        uint64_t sees = 0;                                // the query's node and its ancestors (0: unused)
#pragma unroll 1
        for (int k = 0;; ++k) {
            TrSlot* s = &c->slot[k % TR_SLOTS];
            wait(c->u_full[k % TR_SLOTS], k / TR_SLOTS);
            if (failed()) break;
            const volatile TrUnit* u = &s->u;
            if (u->end) break;
            const int n_keys = u->n_keys, prefix = u->prefix, tree = u->tree, rows = u->rows;
            const int npt = (n_keys + TR_BN - 1) / TR_BN, n_tiles = npt + tree;
            if (u->newq) {
                sees = 0;
                const int node = (u->block * TR_SPAN + r) % T;
                for (int n = r < rows && s->depth[node] != 255 ? node : -1; n >= 0; n = s->up[n]) sees |= 1ull << n;
            }
            const uint32_t tO = tmem + 256 + (k & 1) * RR + wg * COLS + lane_addr;
            float m = -INFINITY, l = 0.0f;
            bool gone = false;                            // all of them leave
#pragma unroll 1
            for (int i = 0; i < n_tiles; ++i, ++g) {
                const uint32_t tS = tmem + (g & 1) * 128 + part * COLS + lane_addr;
                const bool whole = i < npt && n_keys - i * TR_BN >= TR_BN;  // every column is a key that all see
                wait(c->s_full[g & 1], g >> 1);
                tc_fence_after();
                uint32_t xr[CH];
                auto take = [&](int c0) {  // 16 columns from c0 of the thread on, what is hidden at -inf
                    tmem_ld16(tS + c0, xr);
                    tmem_ld_wait();
                    if (whole) return;
                    c0 += part * COLS;
                    uint32_t see;
                    if (i < npt) {         // whole pages of the prefix
                        see = n_keys - i * TR_BN > c0 ? 0xffffu : 0u;
                    } else {               // the prefix's keys and the nodes that the query sees
                        const int at = c0 - (prefix & (PAGE - 1));  // the node of the first column (before 0: prefix)
                        see = at >= 64 ? 0u : at >= 0 ? (uint32_t)(sees >> at) : (uint32_t)(sees << -at) | ((1u << -at) - 1u);
                    }
#pragma unroll
                    for (int x = 0; x < CH; ++x) xr[x] = (see >> x) & 1u ? xr[x] : 0xff800000u;
                };
                auto largest = [&](float mx) {
                    float m0 = mx, m1 = __uint_as_float(xr[1]);
#pragma unroll
                    for (int x = 0; x < CH; x += 4) {
                        m0 = fmaxf(fmaxf(m0, __uint_as_float(xr[x])), __uint_as_float(xr[x + 2]));
                        m1 = fmaxf(fmaxf(m1, __uint_as_float(xr[x + 1])), __uint_as_float(xr[x + 3]));
                    }
                    return fmaxf(m0, m1);
                };
                // A tile's weights are made with the maximum as it is.  Where some query's has grown by too much (and
                // at an item's first tile, which has none yet) the maxima are exchanged and the tile is done again.
                float sum = 0.0f;
                bool again = i == 0;
                float mt = -INFINITY;
                if (i == 0 && ok) {
#pragma unroll 1
                    for (int h = 0; h < COLS; h += CH) {
                        take(h);
                        mt = largest(mt);
                    }
                    mt *= scl;
                }
                while (true) {
                    if (again) {
                        c->ex[part * RR + r] = mt;
                        if ((gone = failed())) break;
#pragma unroll
                        for (int x = 0; x < PARTS; ++x) mt = fmaxf(mt, c->ex[x * RR + r]);
                        float alpha = 1.0f;
                        if (mt > m + TR_SLACK) {
                            alpha = ex2(m - mt);  // 0 for the first
                            m = mt;
                        }
                        l *= alpha;
                        if (i > 0) {              // O^T, once PV of the tile before is in it: dim ln of COLS queries
                            wait(c->pv_done[(g - 1) & 1], (g - 1) >> 1);
                            if ((gone = failed())) break;  // (the maxima have been read)
                            if (part == 0) c->ex[r] = alpha;
                            named_bar_sync(1, TR_SOFTMAX);
                            tc_fence_after();
#pragma unroll 1
                            for (int h = 0; h < COLS; h += CH) {
                                uint32_t rr[CH];
                                tmem_ld16(tO + h, rr);
                                tmem_ld_wait();
#pragma unroll
                                for (int x = 0; x < CH; ++x) rr[x] = __float_as_uint(__uint_as_float(rr[x]) * c->ex[wg * COLS + h + x]);
                                tmem_st16(tO + h, rr);
                            }
                            tmem_st_wait();
                        }
                    }
                    const float nm = m == -INFINITY ? 0.0f : -m;
                    const float2 sc2 = make_float2(scl, scl), nm2 = make_float2(nm, nm);
                    float2 acc0 = make_float2(0.0f, 0.0f), acc1 = acc0;
                    mt = -INFINITY;
                    constexpr int CW = COLS < 32 ? COLS : 32;  // columns whose weights wait in registers for P^T's buffer
#pragma unroll 1
                    for (int h = 0; ok && h < COLS; h += CW) {
                        uint32_t pr[CW / 2];
#pragma unroll
                        for (int e = 0; e < CW; e += CH) {
                            take(h + e);
                            mt = largest(mt);
#pragma unroll
                            for (int x = 0; x < CH; x += 4) {
                                const float2 t0 = ffma2(make_float2(__uint_as_float(xr[x]), __uint_as_float(xr[x + 1])), sc2, nm2);
                                const float2 t1 = ffma2(make_float2(__uint_as_float(xr[x + 2]), __uint_as_float(xr[x + 3])), sc2, nm2);
                                const float2 e0 = make_float2(ex2(t0.x), ex2(t0.y)), e1 = make_float2(ex2(t1.x), ex2(t1.y));
                                acc0 = fadd2(acc0, e0);
                                acc1 = fadd2(acc1, e1);
                                pr[(e + x) >> 1] = pack_bf16x2(e0.x, e0.y);
                                pr[((e + x) >> 1) + 1] = pack_bf16x2(e1.x, e1.y);
                            }
                        }
                        // P^T's buffer: read by PV of the tile PBUF before this one
                        if (h == 0 && g >= Sh::PBUF) wait(c->pv_done[(g - Sh::PBUF) & 1], (g - Sh::PBUF) >> 1);
                        const int col = part * COLS + h;   // chunks of 8 keys of the query's row
                        uint8_t* prow = sm + Sh::OFF_P + (g % Sh::PBUF) * Sh::P_BYTES + (col >> 6) * (RR * 128);
                        if (ok) {
#pragma unroll
                            for (int x = 0; x < CW / 8; ++x)
                                *reinterpret_cast<uint4*>(prow + sw128_off(r, ((col & 63) >> 3) + x)) =
                                    make_uint4(pr[4 * x], pr[4 * x + 1], pr[4 * x + 2], pr[4 * x + 3]);
                        }
                    }
                    sum = (acc0.x + acc0.y) + (acc1.x + acc1.y);
                    mt *= scl;
                    again = named_bar_or(1, TR_SOFTMAX, mt > m + TR_SLACK || !ok);
                    if (!again) break;
                }
                if (gone) break;
                l += sum;
                tc_fence_before();
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(smem_u32(&c->s_free[g & 1]));
                    mbar_arrive(smem_u32(&c->p_ready[g % Sh::PBUF]));
                }
            }
            if (gone) break;
            // ---- the item's results ----
            float* ex_sum = reinterpret_cast<float*>(c + 1);
            if (part) ex_sum[(part - 1) * RR + r] = l;
            wait(c->r_full[k & 1], k >> 1);
            if (failed()) break;
            const size_t row0 = first_row(a, u->b, u->kvh) + u->block * TR_SPAN;
            const int direct = u->direct, split = u->split;
            if (t < RR) {  // part 0 of query t, whole warps
                float sum = l, inv = 0.0f;
#pragma unroll
                for (int x = 1; x < PARTS; ++x) sum += ex_sum[(x - 1) * RR + r];
                bool fail = *reinterpret_cast<const uint32_t*>(c->xbad[k & 1]) != 0;
                if (tree) {
                    const int off = prefix & (PAGE - 1);
                    const uint32_t b0 = __ballot_sync(0xffffffffu, lane < T && c->kbad[k & 1][off + min(lane, TREE_MAX - 1)]);
                    const uint32_t b1 = __ballot_sync(0xffffffffu, lane + 32 < T && c->kbad[k & 1][off + min(lane + 32, TREE_MAX - 1)]);
                    fail |= (sees & (((uint64_t)b1 << 32) | b0 | c->vbad[k & 1])) != 0;
                }
                fail |= (c->qbad[u->nq % TR_QSETS][r >> 2] >> (r & 3)) & 1;
                const bool empty = sees == 0;
                if (!empty && !fail && sum > 0.0f) inv = 1.0f / sum;
                c->ex[r] = inv;  // (the maxima have been read)
                if (r < rows) {
                    const float lse2 = empty ? -INFINITY : fail ? __int_as_float(0x7fc00000) : m + log2f(sum);
                    if (direct) a.lse[row0 + r] = lse2 * 0.693147180559945309f;
                    else a.lse_part[(row0 + r) * a.n_splits + split] = lse2;
                    if (fail && !empty && a.status) atomicOr(a.status, RK_STATUS_RANGE);
                }
            }
            wait(c->o_done[k & 1], k >> 1);
            if (failed()) break;
            tc_fence_after();
            // thread: dim ln of queries wg * COLS ..
            const size_t step = direct ? HEAD_DIM : (size_t)a.n_splits * HEAD_DIM;
            float* part_o = a.o_part + (row0 * a.n_splits + split) * HEAD_DIM + wg * COLS * step + ln;
            __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(a.out) + (row0 + wg * COLS) * HEAD_DIM + ln;
#pragma unroll 1
            for (int h = 0; h < COLS; h += CH) {
                uint32_t rr[CH];
                tmem_ld16(tO + h, rr);
                tmem_ld_wait();
                const int left = rows - wg * COLS - h;
#pragma unroll
                for (int x = 0; x < CH; ++x) {
                    const float f = c->ex[wg * COLS + h + x];
                    const float y = f == 0.0f ? 0.0f : __uint_as_float(rr[x]) * f;  // (a failed query's O may be NaN)
                    if (x < left) {
                        if (direct) *out = __float2bfloat16_rn(y);
                        else *part_o = y;
                    }
                    out += HEAD_DIM;
                    part_o += step;
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(smem_u32(&c->o_free[k & 1]));
                mbar_arrive(smem_u32(&c->r_empty[k & 1]));
                mbar_arrive(smem_u32(&c->u_empty[k % TR_SLOTS]));
            }
            ++done;
        }
    }

    // ---- every role has left its loop; no MMA, copy or TMEM access is in flight ----
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == WARP_MMA) {
        tc_fence_after();
        tmem_dealloc(tmem, Sh::TMEM_COLS);
    }
    if (pipe_aborted(pc)) {
        // A wait gave up.  What the softmax warps have not written of this CTA's items is written as failed,
        // rows without keys among them.
        if (tid == 32 * WARP_S0) *reinterpret_cast<int*>(c->ex) = done;
        __syncthreads();
        int skip = *reinterpret_cast<const int*>(c->ex);
        it.place((int)blockIdx.x, heads, blocks);
        bool found = false;
#pragma unroll 1
        for (;; found = true) {
            if (!found || it.next(a, heads, blocks)) it.find(a, c->total, c->pre, heads, blocks);
            if (!it.valid(a, heads)) break;
            const bool publishes = it.n >= 0 && !it.bad;
            if (publishes && skip > 0) {
                --skip;
                continue;
            }
            write_nothing(a, it.b, it.kvh, it.block, it.s, it.ns == 1, __int_as_float(0x7fc00000), tid, TR_THREADS);
        }
        if (tid == 0 && a.status) atomicOr(a.status, RK_STATUS_TIMEOUT);
    }
}

// Merge of a query's parts: weights 2^(lse_s - max lse), eight sums over the parts s = e, e + 8, ... in
// ascending order, added up in order of e: fixed by the row's number of parts.  A NaN part fails the query, no
// visible key gives out = 0, lse = -inf.  WIDE = false: a warp has a query and all eight sums, four dims to a
// lane; WIDE = true: a block has a query and a warp a sum.  Both add in the same order.
template <bool WIDE>
__global__ void __launch_bounds__(256) tree_merge_kernel(const __grid_constant__ TreeArgs a) {
    constexpr int SUMS = WIDE ? 1 : 8;
    __shared__ float4 acc_s[WIDE ? 8 : 1][32];
    __shared__ float sum_s[8];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, e0 = WIDE ? warp : 0;
    const size_t row = WIDE ? blockIdx.x : (size_t)blockIdx.x * 8 + warp, all = (size_t)a.B * a.Hq * a.T;
    int kv, bad0;
    const int ns = row < all ? parts_of(a, row_pages16(a, (int)(row / ((size_t)a.Hq * a.T)), kv, bad0)) : 1;
    griddep_wait();  // the parts are complete and visible
    if (ns <= 1) return;
    const float* lp = a.lse_part + row * a.n_splits;
    const float4* op = reinterpret_cast<const float4*>(a.o_part + row * a.n_splits * HEAD_DIM) + lane;
    const float4 zero = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    float4 x[SUMS];
    float wt[SUMS];
    auto load = [&](int s0) {
#pragma unroll
        for (int e = 0; e < SUMS; ++e) {
            const int s = s0 + e0 + e;
            x[e] = s < ns ? op[(size_t)s * 32] : zero;
            wt[e] = s < ns ? lp[s] : -INFINITY;
        }
    };
    load(0);
    float m = -INFINITY;
    bool bad = false;
    for (int s = lane; s < ns; s += 32) {
        const float v = lp[s];
        bad |= v != v;
        m = fmaxf(m, v);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    bad = __any_sync(0xffffffffu, bad);
    uint2* out = reinterpret_cast<uint2*>(reinterpret_cast<__nv_bfloat16*>(a.out) + row * HEAD_DIM) + lane;
    if (bad || m == -INFINITY) {  // (the same in every warp of a block)
        if (e0 == 0) {
            *out = make_uint2(0, 0);
            if (lane == 0) a.lse[row] = bad ? __int_as_float(0x7fc00000) : -INFINITY;
        }
        return;
    }
    float4 acc[SUMS];
    float sum[SUMS];
#pragma unroll
    for (int e = 0; e < SUMS; ++e) {
        acc[e] = zero;
        sum[e] = 0.0f;
    }
    for (int s0 = 0; s0 < ns;) {
#pragma unroll
        for (int e = 0; e < SUMS; ++e) {
            const float w = ex2(wt[e] - m);
            sum[e] += w;
            acc[e].x = fmaf(w, x[e].x, acc[e].x);
            acc[e].y = fmaf(w, x[e].y, acc[e].y);
            acc[e].z = fmaf(w, x[e].z, acc[e].z);
            acc[e].w = fmaf(w, x[e].w, acc[e].w);
        }
        s0 += 8;
        if (s0 < ns) load(s0);
    }
    float4 y = acc[0];
    float l = sum[0];
    if constexpr (WIDE) {
        acc_s[e0][lane] = acc[0];
        if (lane == 0) sum_s[e0] = sum[0];
        __syncthreads();
        if (e0) return;
    }
#pragma unroll
    for (int e = 1; e < 8; ++e) {
        const float4 z = WIDE ? acc_s[WIDE ? e : 0][lane] : acc[e % SUMS];
        y.x += z.x;
        y.y += z.y;
        y.z += z.z;
        y.w += z.w;
        l += WIDE ? sum_s[e] : sum[e % SUMS];
    }
    const float inv = 1.0f / l;
    *out = make_uint2(pack_bf16x2(y.x * inv, y.y * inv), pack_bf16x2(y.z * inv, y.w * inv));
    if (lane == 0) a.lse[row] = (m + log2f(l)) * 0.693147180559945309f;
}

std::atomic<uint64_t> g_configured{0};
std::atomic<int> g_sms[64];

}  // namespace

cudaError_t launch_tree(const CUtensorMap& km, const CUtensorMap& vm, const TreeArgs& a, cudaStream_t stream) {
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? (1ull << dev) : 0;
    if (!bit || !(g_configured.load() & bit)) {
        if ((e = cudaFuncSetAttribute(tree_kernel<32>, cudaFuncAttributeMaxDynamicSharedMemorySize, tr_smem_bytes<32>())) != cudaSuccess) return e;
        if ((e = cudaFuncSetAttribute(tree_kernel<64>, cudaFuncAttributeMaxDynamicSharedMemorySize, tr_smem_bytes<64>())) != cudaSuccess) return e;
        if ((e = cudaFuncSetAttribute(tree_kernel<128>, cudaFuncAttributeMaxDynamicSharedMemorySize, tr_smem_bytes<128>())) != cudaSuccess) return e;
        if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
        if (bit) g_sms[dev].store(sms);
        g_configured.fetch_or(bit);
    } else {
        sms = g_sms[dev].load();
    }
    // as many runs to a KV head and block of queries as SMs, and no more than it can have parts
    const int R = a.G * a.T, heads = a.Hkv * ((R + TR_SPAN - 1) / TR_SPAN);
    TreeArgs r = a;
    r.members = (int)std::min<long long>(std::max(1, sms / heads), (long long)a.B * a.n_splits);
    r.share = ((1ull << 32) + r.members - 1) / r.members;
    const unsigned grid = (unsigned)std::min(sms, heads * r.members);
    if (R <= 32) tree_kernel<32><<<grid, TR_THREADS, tr_smem_bytes<32>(), stream>>>(km, vm, r);
    else if (R <= 64) tree_kernel<64><<<grid, TR_THREADS, tr_smem_bytes<64>(), stream>>>(km, vm, r);
    else tree_kernel<128><<<grid, TR_THREADS, tr_smem_bytes<128>(), stream>>>(km, vm, r);
    if ((e = cudaGetLastError()) != cudaSuccess || a.n_splits <= 1) return e;
    const long long rows = (long long)a.B * a.Hq * a.T;
    const bool wide = a.n_splits > 32;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(wide ? rows : (rows + 7) / 8));
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return wide ? cudaLaunchKernelEx(&cfg, tree_merge_kernel<true>, a) : cudaLaunchKernelEx(&cfg, tree_merge_kernel<false>, a);
}

}  // namespace rk
