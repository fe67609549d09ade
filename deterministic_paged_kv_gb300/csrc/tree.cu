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
// Work: the items (row, KV head, pair of q-tiles, part) in that order are dealt to a persistent grid of
// one CTA per SM in runs of equal numbers of tiles; a CTA keeps its queries over the items of one row
// and head.  Which CTA runs an item never changes how.
//
// Roles (512 threads), R <= 128 (TILES = 1) / R > 128 (TILES = 2, two q-tiles to an item):
//   warpgroups 0-1 / 0   transform: rotate new queries and each K tile in place in shared memory
//                        (FP32, angles from exact anchors and steps), FP16 for the score MMA;
//   warpgroup  2 / 1-2   softmax, one thread per accumulator row: online softmax in the log2 domain,
//                        P as BF16 into tensor memory over S; epilogue;
//   warps 12, 14         TMA producers of K and V pages; warp 14 cleans the tree's V tile;
//   warp 13              MMA issuer.  TILES = 1: S has two buffers, S of the next tile is issued before
//                        PV of this one.  TILES = 2: a buffer to each q-tile;
//   warp 15              scheduler: walks the items, checks their metadata, publishes them.
#include <atomic>
#include <cstring>

#include "rk_device.cuh"
#include "tree_args.h"

namespace rk {

namespace {

constexpr int TR_THREADS = 512;
constexpr int WARP_K = 12, WARP_MMA = 13, WARP_V = 14, WARP_SCHED = 15;
constexpr int TR_BN = 128;                                // keys of a prefix tile
constexpr int TR_TILE_BYTES = TR_BN * HEAD_DIM * 2;       // 32 KiB
constexpr int TR_KSTAGES = 3;
constexpr int TR_TREE_ROWS = 80;                          // keys of the tree's tile: 15 + 64, whole pages
constexpr uint32_t TR_TMEM_COLS = 512;                    // S buffers at 0 and 128, O at 256 and 384
constexpr float TR_SLACK = 8.0f;                          // the running max moves when it grows by more (log2)
constexpr int TR_SLOTS = 2;                               // items published ahead
constexpr int TR_ANCHOR = 8;                              // tiles between exact angles
constexpr int TR_GROUPS = 1024;                           // row groups of the item search

template <int TILES>
struct TrShape {
    static constexpr int VSTAGES = TILES == 1 ? 3 : 2;
    static constexpr int XW = TILES == 1 ? 8 : 4;         // transform warps
    static constexpr int ROW_STEP = XW * 4;               // rows between a transform thread's rows
    static constexpr int SW = 4 * TILES;                  // softmax warps
    static constexpr int REG_X = TILES == 1 ? 104 : 88, REG_S = TILES == 1 ? 208 : 184, REG_C = 56;
    static constexpr int OFF_K = TILES * TR_TILE_BYTES;
    static constexpr int OFF_V = OFF_K + TR_KSTAGES * TR_TILE_BYTES;
    static constexpr int OFF_CTRL = OFF_V + VSTAGES * TR_TILE_BYTES;
};
static_assert(2 * TrShape<1>::REG_X + TrShape<1>::REG_S + TrShape<1>::REG_C <= 512, "register split above the launch's");
static_assert(TrShape<2>::REG_X + 2 * TrShape<2>::REG_S + TrShape<2>::REG_C <= 512, "register split above the launch's");

// An item as the scheduler publishes it.
struct TrUnit {
    int end;                 // 1: no further item
    int b, kvh, pair, split;
    int t0, n_keys;          // its prefix keys [t0, t0 + n_keys), whole pages
    int tree;                // 1: the tree's tile follows them
    int prefix;              // tokens before the tree
    int newq, endq, nq;      // first / last item of its queries, their number in this CTA
    int direct;              // 1: the row has one part
    int rows;                // live accumulator rows of the item
};
struct TrSlot {
    TrUnit u;
    uint64_t sees[TREE_MAX];   // node's ancestors and itself
    uint8_t depth[TREE_MAX];   // 255: unused
};

// ------------------------------------------------------------ geometry ----

// A row's prefix in whole pages, and why the row has none (status bits; kv_len 0: -1 and no bit).
__device__ __forceinline__ int row_pages16(const TreeArgs& a, int b, int& kv, int& bad) {
    kv = a.kv_lens[b];
    bad = kv < 0 || kv > a.W * PAGE || (kv > 0 && kv < a.T) ? RK_STATUS_KVLEN : 0;
    return bad || kv == 0 ? -1 : (kv - a.T) & ~(PAGE - 1);
}
// Parts of a row with n prefix keys in whole pages (one where there are none).
__device__ __forceinline__ int parts_of(const TreeArgs& a, int n) {
    if (n <= 0) return 1;
    const int z = n > a.zone[1].token;
    return a.zone[z].split + (n - a.zone[z].token + a.zone[z].size - 1) / a.zone[z].size;
}
__device__ __forceinline__ int part_start(const TreeArgs& a, int s) {
    const int z = s >= a.zone[1].split;
    return a.zone[z].token + (s - a.zone[z].split) * a.zone[z].size;
}
// Tiles of a row: its prefix's and the tree's (one for a row without keys, which is an item too).
__device__ __forceinline__ int row_tiles(int n) { return n < 0 ? 1 : (n + TR_BN - 1) / TR_BN + 1; }

// A CTA's items: the parts whose first tile, in the order of row, KV head and pair, part, lies in
// the CTA's share of all tiles.
struct TrItems {
    int b, h, s;            // row, KV head * pairs + pair, part
    int kv, n, ns, bad;     // the row's length, prefix keys in whole pages, parts, status
    int at, hi;             // the item's first tile, the share's end
    __device__ __forceinline__ bool valid(const TreeArgs& a) const { return b < a.B && at < hi; }
    __device__ __forceinline__ void row(const TreeArgs& a) {
        if (b < a.B) {
            n = row_pages16(a, b, kv, bad);
            ns = parts_of(a, n);
        }
    }
    __device__ void start(const TreeArgs& a, int total, const int* pre, int heads) {
        const unsigned all = (unsigned)(total * heads), each = all / gridDim.x, rest = all % gridDim.x;
        at = (int)(each * blockIdx.x + rest * blockIdx.x / gridDim.x);
        hi = (int)(each * (blockIdx.x + 1) + rest * (blockIdx.x + 1) / gridDim.x);
        const int per = (a.B + TR_GROUPS - 1) / TR_GROUPS, groups = (a.B + per - 1) / per;
        int lo = 0, top = groups;
        while (top - lo > 1) {
            const int mid = (lo + top) >> 1;
            if (pre[mid] * heads <= at) lo = mid;
            else top = mid;
        }
        b = lo * per;
        int base = pre[lo] * heads;
        while (true) {
            row(a);
            const int rt = row_tiles(n), in = at - base;
            if (in < rt * heads || b + 1 >= a.B) {
                h = in / rt;
                const int tile = in % rt;
                // the first part that starts at this tile or later
                for (s = tile ? parts_of(a, min(max(n, 0), tile * TR_BN)) : 0; s < ns && part_start(a, s) < tile * TR_BN; ++s) {
                }
                if (s < ns) {
                    at = base + h * rt + part_start(a, s) / TR_BN;
                } else {
                    at = base + (h + 1) * rt;
                    wrap(a, heads);
                }
                return;
            }
            base += rt * heads;
            ++b;
        }
    }
    __device__ __forceinline__ void wrap(const TreeArgs& a, int heads) {
        s = 0;
        if (++h == heads) {
            h = 0;
            ++b;
            row(a);
        }
    }
    __device__ __forceinline__ void next(const TreeArgs& a, int heads) {
        const int from = part_start(a, s) / TR_BN;
        if (++s == ns) {
            at += row_tiles(n) - from;
            wrap(a, heads);
        } else {
            at += part_start(a, s) / TR_BN - from;
        }
    }
};

struct TrCtrl {
    uint64_t q_ready, q_empty;
    uint64_t k_full[TR_KSTAGES], k_ready[TR_KSTAGES], k_empty[TR_KSTAGES];
    uint64_t v_full[3], v_empty[3], v_land;
    uint64_t s_full[2], p_ready[2], pv_done[2], o_done[2], o_free[2];
    uint64_t u_full[TR_SLOTS], u_empty[TR_SLOTS];
    uint64_t r_full[2], r_empty[2];
    uint64_t never;
    uint32_t tmem_base;
    PipeCtl pipe;
    int total;                        // tiles of the batch's rows (of one KV head and pair)
    int first[sizeof(TrItems) / 4];   // the CTA's first item, for the way out after a failure
    int scan[TR_THREADS / 32];
    uint64_t vbad[2];                 // nodes whose V is not finite, by item parity
    uint8_t xbad[2][8];               // a transform warp met a prefix key out of range
    uint8_t kbad[2][TR_TREE_ROWS];    // keys of the tree's tile out of range
    uint8_t qbad[2][256];             // queries out of range, by the queries' parity
    alignas(16) TrSlot slot[TR_SLOTS];
};
template <int TILES>
constexpr int tr_smem_bytes() {
    static_assert(TrShape<TILES>::OFF_CTRL + sizeof(TrCtrl) <= 232448, "tree attention shared memory above the 227 KiB opt-in limit");
    return TrShape<TILES>::OFF_CTRL + (int)sizeof(TrCtrl);
}
static_assert(TR_GROUPS * 4 <= TR_TILE_BYTES, "the item search's sums lie in a V stage");

// First accumulator row of (row b, KV head kvh) in q, out and lse.
__device__ __forceinline__ size_t first_row(const TreeArgs& a, int b, int kvh) { return ((size_t)b * a.Hkv + kvh) * (size_t)(a.G * a.T); }

// An item that nothing is computed for (count threads, i of them): a part that says NaN or -inf,
// or the results themselves.
__device__ void write_nothing(const TreeArgs& a, int b, int kvh, int pair, int split, bool direct, float lse, int i, int count, int span) {
    const int R = a.G * a.T, r0 = pair * span, rows = min(span, R - r0);
    if (!direct) {
        float* lp = a.lse_part + (((size_t)b * a.Hkv + kvh) * a.n_splits + split) * a.Rp + r0;
        for (int r = i; r < rows; r += count) lp[r] = lse;
        return;
    }
    uint4* o = reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(a.out) + (first_row(a, b, kvh) + r0) * HEAD_DIM);
    for (int k = i; k < rows * (HEAD_DIM / 8); k += count) o[k] = make_uint4(0, 0, 0, 0);
    for (int r = i; r < rows; r += count) a.lse[first_row(a, b, kvh) + r0 + r] = lse * 0.693147180559945309f;
}

// PV of a tile: one k-step per page (P from tensor memory, V from shared memory).
template <int KS>
__device__ __forceinline__ void pv_steps(uint32_t d, uint32_t p, uint32_t v, uint32_t idesc, uint32_t acc0, int pages) {
    if (KS < pages) {
        mma_ts_steps<KS, KS + 1, MN_MAJOR_PAGE>(d, p, v, idesc, acc0);
        if constexpr (KS + 1 < TR_BN / PAGE) pv_steps<KS + 1>(d, p, v, idesc, acc0, pages);
    }
}

// Keys of tile i of an item (whole pages).
__device__ __forceinline__ int tile_keys(int i, int n_keys, int prefix, int T) {
    const int left = n_keys - i * TR_BN;
    return left > 0 ? min(TR_BN, left) : ((prefix & (PAGE - 1)) + T + PAGE - 1) & ~(PAGE - 1);
}

template <int TILES>
__global__ void __launch_bounds__(TR_THREADS, 1)
    tree_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap, const __grid_constant__ TreeArgs a) {
    extern __shared__ __align__(1024) uint8_t sm[];
    using Sh = TrShape<TILES>;
    constexpr int VSTAGES = Sh::VSTAGES;
    TrCtrl* c = reinterpret_cast<TrCtrl*>(sm + Sh::OFF_CTRL);
    int* pre = reinterpret_cast<int*>(sm + Sh::OFF_V + (VSTAGES - 1) * TR_TILE_BYTES);
    const uint32_t s_base = smem_u32(sm);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, wg = warp >> 2;
    const int T = a.T, R = a.G * T;
    constexpr int SPAN = 128 * TILES;                     // accumulator rows of an item
    const int pairs = (R + SPAN - 1) / SPAN, heads = a.Hkv * pairs;
    griddep_launch_dependents();                          // the merge may become resident; it waits for this grid's end

    if (tid == 0) {
        c->pipe.abort = 0;
        c->pipe.limit_ns = wait_limit(a.wait_limit_ns);
        mbar_init(smem_u32(&c->never), 1);
        mbar_init(smem_u32(&c->q_ready), Sh::XW);
        mbar_init(smem_u32(&c->q_empty), 1);
        for (int k = 0; k < TR_KSTAGES; ++k) {
            mbar_init(smem_u32(&c->k_full[k]), 1);
            mbar_init(smem_u32(&c->k_ready[k]), Sh::XW);
            mbar_init(smem_u32(&c->k_empty[k]), 1);
        }
        for (int k = 0; k < VSTAGES; ++k) {
            mbar_init(smem_u32(&c->v_full[k]), 1);
            mbar_init(smem_u32(&c->v_empty[k]), 1);
        }
        mbar_init(smem_u32(&c->v_land), 1);
        for (int j = 0; j < 2; ++j) {
            mbar_init(smem_u32(&c->s_full[j]), 1);
            mbar_init(smem_u32(&c->p_ready[j]), 4);
            mbar_init(smem_u32(&c->pv_done[j]), 1);
            mbar_init(smem_u32(&c->o_done[j]), 1);
            mbar_init(smem_u32(&c->o_free[j]), 4);
            mbar_init(smem_u32(&c->r_full[j]), Sh::XW + 1);
            mbar_init(smem_u32(&c->r_empty[j]), Sh::SW);
        }
        for (int k = 0; k < TR_SLOTS; ++k) {
            mbar_init(smem_u32(&c->u_full[k]), 1);
            mbar_init(smem_u32(&c->u_empty[k]), 3 + Sh::XW + Sh::SW);  // producers, issuer, transform, softmax warps
        }
        fence_mbar_init();
    }
    if (warp == WARP_MMA) {
        tmem_alloc(smem_u32(&c->tmem_base), TR_TMEM_COLS);
        tmem_relinquish();
    }
    {
        // Tiles before each group of `per` rows, a group to a thread and pass.
        const int per = (a.B + TR_GROUPS - 1) / TR_GROUPS, groups = (a.B + per - 1) / per;
        int base = 0;
        for (int g0 = 0; g0 < groups; g0 += TR_THREADS) {
            const int gr = g0 + tid;
            int cnt = 0;
            for (int b = gr * per; gr < groups && b < min(a.B, gr * per + per); ++b) {
                int kv, bad;
                cnt += row_tiles(row_pages16(a, b, kv, bad));
            }
            int v = cnt;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int t = __shfl_up_sync(0xffffffffu, v, o);
                if (lane >= o) v += t;
            }
            __syncthreads();
            if (lane == 31) c->scan[warp] = v;
            __syncthreads();
            int before = base;
            for (int w = 0; w < TR_THREADS / 32; ++w) {
                before += w < warp ? c->scan[w] : 0;
                base += c->scan[w];
            }
            if (gr < groups) pre[gr] = before + v - cnt;
        }
        if (tid == 0) c->total = base;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = c->tmem_base;
    PipeCtl* pc = &c->pipe;
    if (warp == WARP_SCHED) {
        TrItems first;
        first.start(a, c->total, pre, heads);
        if (lane == 0) *reinterpret_cast<TrItems*>(c->first) = first;
        fence_proxy_async_smem();                         // the sums' memory is a V stage from here on
    }
    __syncthreads();
    int done = 0;                                         // softmax: published items written

    auto wait_all = [&](uint64_t& bar, int parity) {
        return __all_sync(0xffffffffu, mbar_wait(smem_u32(&bar), (uint32_t)(parity & 1), pc)) != 0;
    };

    if (wg == 3) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Sh::REG_C));
        if (warp == WARP_SCHED) {
            // ============================================== scheduler ====
            TrItems it = *reinterpret_cast<const TrItems*>(c->first);
            int k = 0, nq = -1, tree_row = -1;            // published items, queries; row whose tree is in registers
            uint64_t sees[2] = {0, 0};                    // of nodes lane, lane + 32
            int deep[2] = {255, 255}, tree_bad = 0;
            int lb = -1, lh = -1;                         // queries of the item before
            bool ok = true;
            // checks the item `it`; 0: to be published
            auto judge = [&]() -> int {
                int bad = it.bad;
                if (bad || it.n < 0) return bad;
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
                        up[e] = p[e];
                        sees[e] = p[e] == TREE_UNUSED ? 0ull : 1ull << n;
                    }
                    tree_bad = __any_sync(0xffffffffu, wrong) ? RK_STATUS_TREE : 0;
                    // ancestors: twice as far up with every step
#pragma unroll 1
                    for (int step = 0; step < 6 && !tree_bad; ++step) {
                        uint64_t add[2];
                        int far[2];
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int n = up[e] & 63;
                            const uint64_t lo = __shfl_sync(0xffffffffu, sees[0], n & 31), hi = __shfl_sync(0xffffffffu, sees[1], n & 31);
                            add[e] = up[e] >= 0 ? (n & 32 ? hi : lo) : 0ull;
                            far[e] = of(up, n);
                        }
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            sees[e] |= add[e];
                            up[e] = up[e] >= 0 ? far[e] : -1;
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 2; ++e) deep[e] = sees[e] ? __popcll(sees[e]) - 1 : 255;
                }
                bad |= tree_bad;
                // page ids of the item's keys
                const int t0 = part_start(a, it.s), end = it.s + 1 < it.ns ? part_start(a, it.s + 1) : it.kv;
                const int32_t* bt = a.block_table + (size_t)it.b * a.W;
                int oob = 0;
                for (int i = t0 / PAGE + lane; i < (end + PAGE - 1) / PAGE; i += 32) {
                    const int pg = __ldg(bt + i);
                    oob |= (pg < 0) | (pg >= a.num_pages);
                }
                if (__any_sync(0xffffffffu, oob)) bad |= RK_STATUS_PAGE_OOB;
                return bad;
            };
            // goes on to the next item that has something to compute, writing those that have not
            auto settle = [&]() {
                while (it.valid(a)) {
                    const int bad = judge();
                    if (!bad && it.n >= 0) return;
                    if (bad && lane == 0 && a.status) atomicOr(a.status, bad);
                    write_nothing(a, it.b, it.h / pairs, it.h % pairs, it.s, it.ns == 1, bad ? __int_as_float(0x7fc00000) : -INFINITY, lane, 32, SPAN);
                    it.next(a, heads);
                }
            };
            settle();
            while (ok) {
                TrUnit u;
                std::memset(&u, 0, sizeof u);
                u.end = !it.valid(a);
                uint64_t s0 = sees[0], s1 = sees[1];
                const int d0 = deep[0], d1 = deep[1];
                if (!u.end) {
                    u.b = it.b;
                    u.kvh = it.h / pairs;
                    u.pair = it.h % pairs;
                    u.split = it.s;
                    u.t0 = part_start(a, it.s);
                    u.tree = it.s + 1 == it.ns;
                    u.n_keys = (u.tree ? it.n : part_start(a, it.s + 1)) - u.t0;
                    u.prefix = it.kv - T;
                    u.direct = it.ns == 1;
                    u.rows = min(SPAN, R - u.pair * SPAN);
                    u.newq = it.b != lb || it.h != lh;
                    nq += u.newq;
                    u.nq = nq;
                    lb = it.b;
                    lh = it.h;
                    it.next(a, heads);
                    settle();
                    u.endq = !it.valid(a) || it.b != lb || it.h != lh;
                }
                TrSlot* s = &c->slot[k % TR_SLOTS];
                const int use = k / TR_SLOTS;
                int good = 1;
                if (lane == 0) good = mbar_wait(smem_u32(&c->u_empty[k % TR_SLOTS]), (uint32_t)((use & 1) ^ 1), pc);
                if (!(ok = __shfl_sync(0xffffffffu, good, 0) != 0)) break;
                s->sees[lane] = s0;
                s->sees[lane + 32] = s1;
                s->depth[lane] = (uint8_t)d0;
                s->depth[lane + 32] = (uint8_t)d1;
                if (lane == 0) s->u = u;
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&c->u_full[k % TR_SLOTS]));
                ++k;
                if (u.end) break;
            }
        } else if (warp == WARP_K || warp == WARP_V) {
            // ======================================= TMA producers ====
            const bool is_k = warp == WARP_K;
            const CUtensorMap* map = is_k ? &kmap : &vmap;
            if (lane == 0) prefetch_tmap(map);
            const int nst = is_k ? TR_KSTAGES : VSTAGES;
            int n = 0, nl = 0;          // tiles issued, tree tiles that went through v_land
            bool land_open = false, ok = true;
            for (int k = 0; ok; ++k) {
                TrSlot* s = &c->slot[k % TR_SLOTS];
                if (!(ok = wait_all(c->u_full[k % TR_SLOTS], k / TR_SLOTS))) break;
                const TrUnit u = s->u;
                if (u.end) break;
                const int npt = (u.n_keys + TR_BN - 1) / TR_BN, n_tiles = npt + u.tree;
                const int32_t* bt = a.block_table + (size_t)u.b * a.W + u.t0 / PAGE;
                int st = n % nst;
                for (int i = 0; i < n_tiles; ++i, ++n) {
                    const int keys = tile_keys(i, u.n_keys, u.prefix, T), np = keys / PAGE;
                    // (the tree's tile begins where the prefix's whole pages end)
                    const int p0 = i < npt ? i * (TR_BN / PAGE) : u.n_keys / PAGE;
                    const int pg = lane < np ? __ldg(bt + p0 + lane) : 0;
                    const uint32_t eb = smem_u32(is_k ? &c->k_empty[st] : &c->v_empty[st]);
                    const uint32_t fb = smem_u32(is_k ? &c->k_full[st] : &c->v_full[st]);
                    int good = 1;
                    if (lane == 0) good = mbar_wait(eb, (uint32_t)((n / nst) & 1) ^ 1u, pc);
                    if (!(ok = __shfl_sync(0xffffffffu, good, 0) != 0)) break;
                    const bool clean = !is_k && i >= npt;
                    const uint32_t lb = clean ? smem_u32(&c->v_land) : fb;
                    if (lane == 0) mbar_arrive_expect_tx(lb, (uint32_t)np * 4096);
                    __syncwarp();
                    if (lane < np) {
                        if (is_k) {  // two 16 x 64 boxes per page: the K-major tile layout
                            const uint32_t t = s_base + Sh::OFF_K + st * TR_TILE_BYTES + lane * 2048;
                            tma_load_3d(t, map, lb, 0, u.kvh, pg * PAGE);
                            tma_load_3d(t + 16384, map, lb, 64, u.kvh, pg * PAGE);
                        } else {     // one 4 KiB box per page: [page][half][16 rows][128 B]
                            tma_load_4d(s_base + Sh::OFF_V + st * TR_TILE_BYTES + lane * 4096, map, lb, 0, pg * PAGE, 0, u.kvh);
                        }
                    }
                    __syncwarp();
                    if (clean) {
                        // The tree's V: rows past the last node and unused nodes hold anything, and 0 times that need not
                        // be 0; a node whose V is not finite is zeroed too and fails who sees it.
                        int landed = 1;
                        if (lane == 0) landed = mbar_wait(lb, (uint32_t)(nl & 1), pc);
                        ++nl;
                        if (!(ok = __shfl_sync(0xffffffffu, landed, 0) != 0)) {
                            land_open = true;
                            break;
                        }
                        const int off = u.prefix & (PAGE - 1);
                        uint8_t* vt = sm + Sh::OFF_V + st * TR_TILE_BYTES;
                        uint64_t bad = 0;
                        if (lane == 0) ok = mbar_wait(smem_u32(&c->r_empty[k & 1]), (uint32_t)((k >> 1) & 1) ^ 1u, pc);
                        if (!(ok = __shfl_sync(0xffffffffu, (int)ok, 0) != 0)) break;
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
                            mbar_arrive(fb);
                        }
                    }
                    if (++st == nst) st = 0;
                }
                if (!ok) break;
                if (!is_k && lane == 0) {
                    if (!u.tree && !(ok = mbar_wait(smem_u32(&c->r_empty[k & 1]), (uint32_t)((k >> 1) & 1) ^ 1u, pc))) {
                    } else {
                        mbar_arrive(smem_u32(&c->r_full[k & 1]));
                    }
                }
                ok = __shfl_sync(0xffffffffu, (int)ok, 0) != 0;
                if (lane == 0) mbar_arrive(smem_u32(&c->u_empty[k % TR_SLOTS]));
            }
            if (lane == 0 && pipe_aborted(pc)) {
                // copies in flight land before the CTA's shared memory is released
                if (land_open) mbar_wait_drain(smem_u32(&c->v_land), (uint32_t)((nl - 1) & 1));
                for (int i = max(0, n - nst); i < n; ++i)
                    mbar_wait_drain(smem_u32(is_k ? &c->k_full[i % nst] : &c->v_full[i % nst]), (uint32_t)((i / nst) & 1));
            }
        } else if (warp == WARP_MMA && lane == 0) {
            // ============================================= MMA issuer ====
            const uint32_t idO = idesc_bf16_f32(128, HEAD_DIM, 0, 1);
            constexpr uint32_t TILE_DESC = TR_TILE_BYTES >> 4;
            const uint32_t dQ0 = desc_lo(s_base, 16), dK0 = desc_lo(s_base + Sh::OFF_K, 16), dV0 = desc_lo(s_base + Sh::OFF_V, 2048);
            auto wait = [&](uint64_t& bar, int parity) { return mbar_wait(smem_u32(&bar), (uint32_t)(parity & 1), pc); };
            int g0 = 0, nu[2] = {0, 0}, np[2] = {0, 0};  // tiles before the item; per q-tile: items, tiles
            bool ok = !a.timeout_drill || drill_wait(smem_u32(&c->never), pc);
            for (int k = 0; ok; ++k) {
                if (!(ok = wait(c->u_full[k % TR_SLOTS], k / TR_SLOTS))) break;
                const volatile TrUnit* su = &c->slot[k % TR_SLOTS].u;
                const int end = su->end, n_keys = su->n_keys, tree = su->tree, prefix = su->prefix;
                const int newq = su->newq, endq = su->endq, nq = su->nq, live = TILES == 2 && su->rows > 128 ? 2 : 1;
                mbar_arrive(smem_u32(&c->u_empty[k % TR_SLOTS]));
                if (end) break;
                const int npt = (n_keys + TR_BN - 1) / TR_BN, n_tiles = npt + tree;
                if (newq && !(ok = wait(c->q_ready, nq))) break;
                auto issue_s = [&](int j, int i) {
                    const int g = g0 + i, keys = tile_keys(i, n_keys, prefix, T);
                    const uint32_t idS = (1u << 4) | ((uint32_t)(keys >> 3) << 17) | (128u >> 4 << 24);
                    const int buf = TILES == 1 ? g & 1 : j;
                    mma_ss_steps<0, 8, K_MAJOR_128, K_MAJOR_128>(tmem + buf * 128, dQ0 + (uint32_t)j * TILE_DESC,
                                                                 dK0 + (uint32_t)(g % TR_KSTAGES) * TILE_DESC, idS, 0u);
                    umma_commit(smem_u32(&c->s_full[buf]));
                };
                // PV of tile i and q-tile j
                auto issue_pv = [&](int j, int i) -> bool {
                    const int g = g0 + i, buf = TILES == 1 ? g & 1 : j;
                    if (i == 0 && !wait(c->o_free[j], nu[j] + 1)) return false;  // the item before has been read
                    if (!wait(c->p_ready[buf], TILES == 1 ? g >> 1 : np[j] + i)) return false;
                    if (!wait(c->v_full[g % VSTAGES], g / VSTAGES)) return false;
                    tc_fence_after();
                    pv_steps<0>(tmem + 256 + j * 128, tmem + buf * 128, dV0 + (uint32_t)(g % VSTAGES) * TILE_DESC, idO, i > 0 ? 1u : 0u,
                                tile_keys(i, n_keys, prefix, T) / PAGE);
                    if constexpr (TILES == 1) umma_commit(smem_u32(&c->pv_done[buf]));
                    if (i == n_tiles - 1) umma_commit(smem_u32(&c->o_done[j]));
                    return true;
                };
                for (int i = 0; i < n_tiles; ++i) {
                    const int g = g0 + i;
                    if (!(ok = wait(c->k_ready[g % TR_KSTAGES], g / TR_KSTAGES))) break;
                    tc_fence_after();
                    if constexpr (TILES == 1) {
                        issue_s(0, i);
                    } else {
                        for (int j = 0; j < live; ++j) {
                            if (i > 0 && !(ok = issue_pv(j, i - 1))) break;
                            issue_s(j, i);
                        }
                        if (!ok) break;
                    }
                    umma_commit(smem_u32(&c->k_empty[g % TR_KSTAGES]));
                    if (endq && i == n_tiles - 1) umma_commit(smem_u32(&c->q_empty));
                    if (TILES == 1 && i > 0 && !(ok = issue_pv(0, i - 1))) break;
                    if (i > 0) umma_commit(smem_u32(&c->v_empty[(g - 1) % VSTAGES]));
                }
                for (int j = 0; j < live && ok; ++j) ok = issue_pv(j, n_tiles - 1);
                if (!ok) break;
                umma_commit(smem_u32(&c->v_empty[(g0 + n_tiles - 1) % VSTAGES]));
                g0 += n_tiles;
                for (int j = 0; j < live; ++j) {
                    ++nu[j];
                    np[j] += n_tiles;
                }
            }
            if (!ok) {  // issued MMAs drain before tensor memory is released
                const uint64_t t0 = global_timer_ns();
                while (global_timer_ns() - t0 < 1000000ull) {
                }
            }
        }
        __syncwarp();
    } else if (warp < Sh::XW) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Sh::REG_X));
        // ================================================ transform ====
        // thread: pair-chunk u8 (8 rotation pairs: 16 bytes of each 64-dim half) of rows r0 + ROW_STEP * m
        const int u8 = tid & 7, r0 = tid >> 3;
        constexpr int ROWS = TR_BN / Sh::ROW_STEP;
        float2 dcs[4], dsn[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            rope_cos_sin((uint32_t)Sh::ROW_STEP, a.rope_turns[8 * u8 + 2 * e], dcs[e].x, dsn[e].x);
            rope_cos_sin((uint32_t)Sh::ROW_STEP, a.rope_turns[8 * u8 + 2 * e + 1], dcs[e].y, dsn[e].y);
        }
        auto angles = [&](uint32_t pos, float2 (&cs)[4], float2 (&sn)[4]) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                rope_cos_sin(pos, a.rope_turns[8 * u8 + 2 * e], cs[e].x, sn[e].x);
                rope_cos_sin(pos, a.rope_turns[8 * u8 + 2 * e + 1], cs[e].y, sn[e].y);
            }
        };
        // a row's verdict from the eight threads that hold it
        auto any8 = [&](bool x) {
            const uint32_t b = __ballot_sync(0xffffffffu, x);
            return ((b >> (lane & 24)) & 0xffu) != 0;
        };
        int g = 0;
        bool ok = true;
        for (int k = 0; ok; ++k) {
            TrSlot* s = &c->slot[k % TR_SLOTS];
            if (!(ok = wait_all(c->u_full[k % TR_SLOTS], k / TR_SLOTS))) break;
            const volatile TrUnit* u = &s->u;
            if (u->end) break;
            const int n_keys = u->n_keys, prefix = u->prefix, t0 = u->t0, tree = u->tree;
            const int npt = (n_keys + TR_BN - 1) / TR_BN;
            float2 cs[4], sn[4];
            if (u->newq) {
                // new queries, once the score MMAs have read the ones before
                const int nq = u->nq, rows = u->rows;
                const uint4* q = reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(a.q) +
                                                                (first_row(a, u->b, u->kvh) + u->pair * SPAN) * HEAD_DIM);
                if (!(ok = wait_all(c->q_empty, nq + 1))) break;
#pragma unroll 1
                for (int rr = 0; rr < SPAN && rr < ((rows + 31) & ~31); rr += Sh::ROW_STEP) {
                    const int r = rr + r0, n = (u->pair * SPAN + r) % T;
                    const bool in = r < rows;
                    uint32_t range = 0;
                    if (in) {
                        uint4 lo = __ldg(q + r * 16 + u8), hi = __ldg(q + r * 16 + 8 + u8);
                        const int d = s->depth[n];
                        angles((uint32_t)(prefix + (d == 255 ? 0 : d)), cs, sn);
                        range = rotate_regs_f16(lo, hi, cs, sn, 0);
                        uint8_t* qt = sm + (r >> 7) * TR_TILE_BYTES + sw128_off(r & 127, u8);
                        *reinterpret_cast<uint4*>(qt) = lo;
                        *reinterpret_cast<uint4*>(qt + 16384) = hi;
                    }
                    const bool bad = any8(in && range_exceeded(range));
                    if (in && u8 == 0) c->qbad[nq & 1][r] = bad;
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&c->q_ready));
            }
            uint32_t range = 0;
            if (!(ok = wait_all(c->r_empty[k & 1], (k >> 1) + 1))) break;
            for (int i = 0; i < npt; ++i, ++g) {
                const int kst = g % TR_KSTAGES;
                if ((i & (TR_ANCHOR - 1)) == 0) angles((uint32_t)(t0 + i * TR_BN + r0), cs, sn);
                if (!(ok = wait_all(c->k_full[kst], g / TR_KSTAGES))) break;
                uint8_t* kt = sm + Sh::OFF_K + kst * TR_TILE_BYTES;
                const int keys = min(TR_BN, n_keys - i * TR_BN);
#pragma unroll
                for (int m0 = 0; m0 < ROWS; m0 += 4) {  // four rows are read before any is rotated
                    uint4 lo[4], hi[4];
#pragma unroll
                    for (int m = 0; m < 4; ++m) {
                        const uint32_t off = sw128_off(r0 + Sh::ROW_STEP * (m0 + m), u8);
                        lo[m] = *reinterpret_cast<const uint4*>(kt + off);
                        hi[m] = *reinterpret_cast<const uint4*>(kt + 16384 + off);
                    }
#pragma unroll
                    for (int m = 0; m < 4; ++m) {
                        const int r = r0 + Sh::ROW_STEP * (m0 + m);
                        if (r < keys) {
                            range = rotate_regs_f16(lo[m], hi[m], cs, sn, range);
                            const uint32_t off = sw128_off(r, u8);
                            *reinterpret_cast<uint4*>(kt + off) = lo[m];
                            *reinterpret_cast<uint4*>(kt + 16384 + off) = hi[m];
                        }
                        rope_step(cs, sn, dcs, dsn);
                    }
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
                for (int rr = 0; rr < last; rr += Sh::ROW_STEP) {
                    const int r = rr + r0, node = r - off0;
                    const int d = node < 0 ? node : r < last ? s->depth[node] : 255;
                    bool bad = false;
                    if (d != 255) {
                        angles((uint32_t)(prefix + d), cs, sn);
                        const uint32_t off = sw128_off(r, u8);
                        const uint32_t rg = rotate_chunk_f16(kt + off, kt + 16384 + off, cs, sn, 0);
                        if (node < 0) range = __vmaxu2(range, rg);
                        else bad = range_exceeded(rg);
                    }
                    bad = any8(bad);
                    if (u8 == 0 && r < TR_TREE_ROWS) c->kbad[k & 1][r] = bad;
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&c->k_ready[kst]));
                ++g;
            }
            const bool bad = __any_sync(0xffffffffu, range_exceeded(range));
            if (lane == 0) {
                c->xbad[k & 1][warp] = bad;
                mbar_arrive(smem_u32(&c->r_full[k & 1]));
                mbar_arrive(smem_u32(&c->u_empty[k % TR_SLOTS]));
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(Sh::REG_S));
        // ================================================== softmax ====
        const int j = TILES == 1 ? 0 : wg - 1;
        const int rt = tid & 127, rj = 128 * j + rt;      // row of the q-tile (TMEM lane), of the item
        const uint32_t lane_addr = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t tO = tmem + 256 + j * 128 + lane_addr;
        const float scl = a.qk_scale_log2;
        int g0 = 0, nu = 0, np = 0;                       // tiles before the item (CTA), items and tiles of this q-tile
        bool ok = true;
        for (int k = 0; ok; ++k) {
            TrSlot* s = &c->slot[k % TR_SLOTS];
            if (!(ok = wait_all(c->u_full[k % TR_SLOTS], k / TR_SLOTS))) break;
            const volatile TrUnit* u = &s->u;
            if (u->end) break;
            const int n_keys = u->n_keys, prefix = u->prefix, tree = u->tree, rows = u->rows;
            const int npt = (n_keys + TR_BN - 1) / TR_BN, n_tiles = npt + tree;
            if (128 * j >= rows) {  // this q-tile has no rows (the other one has)
                ok = wait_all(c->r_full[k & 1], k >> 1);
                if (lane == 0) {
                    mbar_arrive(smem_u32(&c->r_empty[k & 1]));
                    mbar_arrive(smem_u32(&c->u_empty[k % TR_SLOTS]));
                }
                g0 += n_tiles;
                ++done;
                continue;
            }
            const bool live_warp = 128 * j + (warp & 3) * 32 < rows;
            const int node = (u->pair * SPAN + rj) % T;
            const uint64_t sees = rj < rows ? s->sees[node] : 0ull;
            float m = -INFINITY, l = 0.0f;
            for (int i = 0; i < n_tiles; ++i) {
                const int g = g0 + i, buf = TILES == 1 ? g & 1 : j;
                if (!(ok = wait_all(c->s_full[buf], TILES == 1 ? g >> 1 : np + i))) break;
                if (live_warp) {
                    tc_fence_after();
                    const uint32_t tS = tmem + buf * 128 + lane_addr;
                    uint32_t xr[128];
#pragma unroll
                    for (int c4 = 0; c4 < 4; ++c4) tmem_ld32(tS + c4 * 32, *reinterpret_cast<uint32_t(*)[32]>(&xr[c4 * 32]));
                    tmem_ld_wait();
                    if (i >= npt) {  // the tree's tile: the prefix's keys, then the nodes that this one sees
                        const int off = prefix & (PAGE - 1);
                        const uint32_t w0 = (uint32_t)((sees << off) | ((1ull << off) - 1ull)), w1 = (uint32_t)((sees << off) >> 32);
                        const uint32_t w2 = off ? (uint32_t)(sees >> (64 - off)) : 0u;
#pragma unroll
                        for (int x = 0; x < 128; ++x) {
                            const uint32_t w = x < 32 ? w0 : x < 64 ? w1 : x < 96 ? w2 : 0u;
                            xr[x] = (w >> (x & 31)) & 1u ? xr[x] : 0xff800000u;
                        }
                    } else {
                        const int lim = n_keys - i * TR_BN;
                        if (lim < TR_BN) {
#pragma unroll
                            for (int x = 0; x < 128; ++x) xr[x] = x < lim ? xr[x] : 0xff800000u;
                        }
                    }
                    float mx0 = -INFINITY, mx1 = -INFINITY, mx2 = -INFINITY, mx3 = -INFINITY;
#pragma unroll
                    for (int x = 0; x < 128; x += 4) {
                        mx0 = fmaxf(mx0, __uint_as_float(xr[x]));
                        mx1 = fmaxf(mx1, __uint_as_float(xr[x + 1]));
                        mx2 = fmaxf(mx2, __uint_as_float(xr[x + 2]));
                        mx3 = fmaxf(mx3, __uint_as_float(xr[x + 3]));
                    }
                    const float mt = fmaxf(fmaxf(mx0, mx1), fmaxf(mx2, mx3)) * scl;
                    float alpha = 1.0f;
                    bool resc = false;
                    if (mt > m + TR_SLACK) {
                        alpha = ex2(m - mt);
                        m = mt;
                        resc = true;
                    }
                    const float nm = m == -INFINITY ? 0.0f : -m;
                    const float2 sc2 = make_float2(scl, scl), nm2 = make_float2(nm, nm);
                    float2 acc2 = make_float2(0.0f, 0.0f);
#pragma unroll
                    for (int x = 0; x < 128; x += 2) {
                        const float2 t = ffma2(make_float2(__uint_as_float(xr[x]), __uint_as_float(xr[x + 1])), sc2, nm2);
                        const float2 e = make_float2(ex2(t.x), ex2(t.y));
                        acc2 = fadd2(acc2, e);
                        xr[x >> 1] = pack_bf16x2(e.x, e.y);
                    }
                    l = l * alpha + (acc2.x + acc2.y);
                    if (i > 0 && __any_sync(0xffffffffu, resc)) {
                        // PV of the tile before has to be in O (TILES = 2: S of this tile was issued behind it)
                        if (TILES == 1 && !(ok = wait_all(c->pv_done[(g - 1) & 1], (g - 1) >> 1))) break;
                        tc_fence_after();
#pragma unroll 1
                        for (int c4 = 0; c4 < 4; ++c4) {
                            uint32_t rr[32];
                            tmem_ld32(tO + c4 * 32, rr);
                            tmem_ld_wait();
#pragma unroll
                            for (int x = 0; x < 32; ++x) rr[x] = __float_as_uint(__uint_as_float(rr[x]) * alpha);
                            tmem_st32(tO + c4 * 32, rr);
                        }
                    }
                    tmem_st32(tS, *reinterpret_cast<uint32_t(*)[32]>(&xr[0]));
                    tmem_st32(tS + 32, *reinterpret_cast<uint32_t(*)[32]>(&xr[32]));
                    tmem_st_wait();
                    tc_fence_before();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&c->p_ready[buf]));
            }
            if (ok) ok = wait_all(c->o_done[j], nu);
            if (ok) ok = wait_all(c->r_full[k & 1], k >> 1);
            if (!ok) break;
            // ---- the item's results ----
            tc_fence_after();
            bool fail = false;
            {
                const uint64_t xb = *reinterpret_cast<const uint64_t*>(c->xbad[k & 1]);
                fail = (TILES == 1 ? xb : xb & 0xffffffffull) != 0;
                if (tree) {
                    const int off = prefix & (PAGE - 1);
                    const uint32_t b0 = __ballot_sync(0xffffffffu, lane < T && c->kbad[k & 1][off + lane]);
                    const uint32_t b1 = __ballot_sync(0xffffffffu, lane + 32 < T && c->kbad[k & 1][off + min(lane + 32, TREE_MAX - 1)]);
                    fail |= (sees & (((uint64_t)b1 << 32) | b0 | c->vbad[k & 1])) != 0;
                }
                if (rj < rows) fail |= c->qbad[u->nq & 1][rj] != 0;
            }
            const bool empty = sees == 0, direct = u->direct;
            const size_t row = first_row(a, u->b, u->kvh) + u->pair * SPAN + rj;
            const bool zero = empty || fail || !(l > 0.0f);
            const float inv = zero ? 0.0f : 1.0f / l;
            if (live_warp) {
                const bool in = rj < rows;
                const float lse2 = empty ? -INFINITY : fail ? __int_as_float(0x7fc00000) : m + log2f(l);
                float* part = nullptr;
                if (!direct) {
                    const size_t p = ((size_t)u->b * a.Hkv + u->kvh) * a.n_splits + u->split;
                    const int r = u->pair * SPAN + rj;
                    if (in) a.lse_part[p * a.Rp + r] = lse2;
                    part = a.o_part + p * a.Rp * HEAD_DIM + r;
                } else if (in) {
                    a.lse[row] = lse2 * 0.693147180559945309f;
                }
                if (in && fail && !empty && a.status) atomicOr(a.status, RK_STATUS_RANGE);
                uint4* o = reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(a.out) + row * HEAD_DIM);
#pragma unroll 1
                for (int c4 = 0; c4 < 4; ++c4) {
                    uint32_t rr[32];
                    tmem_ld32(tO + c4 * 32, rr);
                    tmem_ld_wait();
                    if (!in) continue;
                    float f[32];
#pragma unroll
                    for (int x = 0; x < 32; ++x) f[x] = zero ? 0.0f : __uint_as_float(rr[x]) * inv;
                    if (direct) {
#pragma unroll
                        for (int x = 0; x < 32; x += 8)
                            o[(c4 * 32 + x) / 8] = make_uint4(pack_bf16x2(f[x], f[x + 1]), pack_bf16x2(f[x + 2], f[x + 3]),
                                                              pack_bf16x2(f[x + 4], f[x + 5]), pack_bf16x2(f[x + 6], f[x + 7]));
                    } else {  // a row to a lane: the warp writes a run of 32 rows of each dim
#pragma unroll
                        for (int x = 0; x < 32; ++x) part[(size_t)(c4 * 32 + x) * a.Rp] = f[x];
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(smem_u32(&c->o_free[j]));
                mbar_arrive(smem_u32(&c->r_empty[k & 1]));
                mbar_arrive(smem_u32(&c->u_empty[k % TR_SLOTS]));
            }
            g0 += n_tiles;
            np += n_tiles;
            ++nu;
            ++done;
        }
    }

    // ---- every role has left its loop; no MMA, copy or TMEM access is in flight ----
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == WARP_MMA) {
        tc_fence_after();
        tmem_dealloc(tmem, TR_TMEM_COLS);
    }
    if (pipe_aborted(pc)) {
        // A wait gave up.  What the first softmax warp has not written of this CTA's items (the others may
        // be one further) is written as failed by all of it, rows without keys among them.
        if (tid == 128 * (TILES == 1 ? 2 : 1)) c->total = done;
        __syncthreads();
        int skip = c->total;
        for (TrItems it = *reinterpret_cast<const TrItems*>(c->first); it.valid(a); it.next(a, heads)) {
            const bool publishes = it.n >= 0 && !it.bad;
            if (publishes && skip > 0) {
                --skip;
                continue;
            }
            write_nothing(a, it.b, it.h / pairs, it.h % pairs, it.s, it.ns == 1, __int_as_float(0x7fc00000), tid, TR_THREADS, SPAN);
        }
        if (tid == 0 && a.status) atomicOr(a.status, RK_STATUS_TIMEOUT);
    }
}

// Merge of the parts of 32 accumulator rows (a row to a lane) for 16 of the dims: weights
// 2^(lse_s - max lse), eight sums over the parts s = w, w + 8, ... (one to a warp) in ascending
// order, added up in order of w: fixed by the row's number of parts.  A NaN part fails the row, no visible
// key gives out = 0, lse = -inf.
constexpr int MG_DIMS = 16;
__global__ void __launch_bounds__(256) tree_merge_kernel(const __grid_constant__ TreeArgs a) {
    __shared__ float acc_s[8][MG_DIMS][33], sum_s[8][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int R = a.G * a.T, groups = (R + 31) / 32;
    const int d0 = (int)(blockIdx.x % (HEAD_DIM / MG_DIMS)) * MG_DIMS;
    const int grp = (int)(blockIdx.x / (HEAD_DIM / MG_DIMS)) % groups;
    const size_t bh = blockIdx.x / (HEAD_DIM / MG_DIMS) / groups;
    int kv, bad0;
    const int ns = parts_of(a, row_pages16(a, (int)(bh / a.Hkv), kv, bad0));
    griddep_wait();  // the parts are complete and visible
    if (ns <= 1) return;
    const int r = grp * 32 + lane;
    const bool in = r < R;
    const float* lp = a.lse_part + bh * a.n_splits * a.Rp + (in ? r : 0);
    const float* op = a.o_part + (bh * a.n_splits * HEAD_DIM + d0) * (size_t)a.Rp + (in ? r : 0);
    float m = -INFINITY;
    bool bad = false;
#pragma unroll 8
    for (int s = 0; s < ns; ++s) {
        const float v = lp[(size_t)s * a.Rp];
        bad |= v != v;
        m = fmaxf(m, v);
    }
    float acc[MG_DIMS], sum = 0.0f;
#pragma unroll
    for (int d = 0; d < MG_DIMS; ++d) acc[d] = 0.0f;
    if (!bad && m > -INFINITY) {
        for (int s = warp; s < ns; s += 8) {
            const float w = ex2(lp[(size_t)s * a.Rp] - m);
            const float* o = op + (size_t)s * HEAD_DIM * a.Rp;
            float x[MG_DIMS];
#pragma unroll
            for (int d = 0; d < MG_DIMS; ++d) x[d] = o[(size_t)d * a.Rp];
            sum += w;
#pragma unroll
            for (int d = 0; d < MG_DIMS; ++d) acc[d] = fmaf(w, x[d], acc[d]);
        }
    }
#pragma unroll
    for (int d = 0; d < MG_DIMS; ++d) acc_s[warp][d][lane] = acc[d];
    sum_s[warp][lane] = sum;
    __syncthreads();
    float l = 0.0f;
#pragma unroll
    for (int w = 0; w < 8; ++w) l += sum_s[w][lane];
    const float inv = bad || m == -INFINITY ? 0.0f : 1.0f / l;
    // warp w: dims 2 w, 2 w + 1
    float y[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < 8; ++w) v += acc_s[w][2 * warp + e][lane];
        y[e] = v * inv;
    }
    if (!in) return;
    const size_t row = bh * R + r;
    reinterpret_cast<uint32_t*>(a.out)[(row * HEAD_DIM + d0) / 2 + warp] = pack_bf16x2(y[0], y[1]);
    if (d0 == 0 && warp == 0) a.lse[row] = bad ? __int_as_float(0x7fc00000) : m == -INFINITY ? m : (m + log2f(l)) * 0.693147180559945309f;
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
        if ((e = cudaFuncSetAttribute(tree_kernel<1>, cudaFuncAttributeMaxDynamicSharedMemorySize, tr_smem_bytes<1>())) != cudaSuccess) return e;
        if ((e = cudaFuncSetAttribute(tree_kernel<2>, cudaFuncAttributeMaxDynamicSharedMemorySize, tr_smem_bytes<2>())) != cudaSuccess) return e;
        if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
        if (bit) g_sms[dev].store(sms);
        g_configured.fetch_or(bit);
    } else {
        sms = g_sms[dev].load();
    }
    const int R = a.G * a.T, tiles = R > 128 ? 2 : 1;
    const long long most = (long long)a.B * a.Hkv * ((R + 128 * tiles - 1) / (128 * tiles)) * a.n_splits;
    const unsigned grid = (unsigned)(most < sms ? most : sms);
    if (tiles == 1) tree_kernel<1><<<grid, TR_THREADS, tr_smem_bytes<1>(), stream>>>(km, vm, a);
    else tree_kernel<2><<<grid, TR_THREADS, tr_smem_bytes<2>(), stream>>>(km, vm, a);
    if ((e = cudaGetLastError()) != cudaSuccess || a.n_splits <= 1) return e;
    const long long blocks = (long long)a.B * a.Hkv * ((R + 31) / 32) * (HEAD_DIM / MG_DIMS);
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, tree_merge_kernel, a);
}

}  // namespace rk
