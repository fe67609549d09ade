// decode_q8.cu -- one-query attention over the 8-bit page cache (tcgen05, TMA).
//
// Operation: the paged decode of "flashinfer_fa2 backend for Ada (SM89)" with a
// fixed split of each row's keys ("WS2 PR7 Fused Attention Backend Alignment",
// "Split-KV Policy", fixed:<N> in logical tokens), over e4m3 codes whose K was
// rotated when it was written.
//
// What bounds it: the cache's bytes (256 a token and KV head).  At half the
// bytes of a BF16 cache there is no time to convert codes, so none is converted:
// K and V go by TMA from the cache into swizzled shared memory and from there
// into kind::f8f6f4 MMAs as they are.  What multiplies them is split into e4m3
// parts instead, which is cheap because it is small:
//   q, rotated and scaled to below 362 by a power of two per head, is four parts
//   (two at 1, two at 2^-8), the G heads' parts being columns of one operand;
//   the softmax weights, scaled to at most 256, are three parts at 1, 2^-5 and 2^-10.
// Products of e4m3 values are exact and the sums are FP32, so a score has the
// precision of q in about 16 bits.  A weight (with V's page scale in it) is good to 2^-14 of itself
// or 2^-28 of its step's largest, whichever is more: a key that takes nearly all of a row's weight
// for a value of nothing, or a page with an outlier in V, leave the other keys their bits.  (Three
// parts at 1 are good to 2^-12 or 2^-18: a weight 2^-10 of the largest to 2^-8 only.)
//
// With S^T = K q^T [128 tokens x 4 G] and O^T = V^T p^T [128 dims x 3 G] both
// operands that come from the cache are A operands in the layout they land in:
// K K-major, V MN-major.  V's page scale enters as an addition to the exponent,
//   w_t = z_t + log2(vs_t),  p'_t = 2^(w_t - max w),  l = sum p'_t / vs_t,
//   o = sum p'_t vcode_t,  out = o / l,
// with z_t the score in the log2 domain.
//
// Work: an item is a split of a row for a bundle of H neighbouring KV heads (2, or 1 where
// Hkv is odd).  A TMA copy takes a page's blocks of the whole bundle: 64 x 4096 takes 125 us head
// by head (copies of 2 KiB, which is what an odd Hkv has: 123 us for the same bytes with Hkv 1 or 3 and
// four queries a KV head, 134 with eight), 90 in bundles of two, 93 in bundles of four, whose items are
// coarser (20 ragged rows of 8 heads a KV head: 54 us, 48 in twos then, 44 now).  A step is 512 / H tokens
// of the bundle, four tiles of 128 tokens and one head; in it the softmax is plain (one
// maximum over its tokens), steps and splits are joined with the running maximum in FP32.  The
// copies leave the bundle as [page][half][head][8 tokens][128 B] in shared memory, so that
// the 16 groups of 8 tokens of a head's tile lie at one stride and make one operand.
// The items in order of row, bundle, split are dealt to a persistent grid of one CTA per
// SM in runs of equal numbers of steps, so a CTA changes its queries a few times only.
// (Dealt in turn, with four heads to a bundle, CTAs of 64 x 4096 ended between 78 and 98 us.)
// The copies carry an evict-first hint: the cache is read once and passes by, while the
// partials of many splits stay in L2 until the merge (64 x 4096: 8 us less).
// Roles (20 warps):
//   warp 0      TMA producer: a step's K, then its V, 64 KiB each, in a ring of three;
//   warp 1      MMA issuer: S and PV of each step;
//   warp 2      q: rotates the query heads of the next row and bundle, splits them into parts
//               (the softmax warps do the first ones, together: they have nothing else to do);
//   warp 3      metadata: walks the items, page ids and scales of each step, and how far V's scales of
//               an item lie apart;
//   warps 4-19  softmax: warpgroup j has tile j of a step, a thread one token, and
//               in the accumulation its share of that KV head's queries, a thread one
//               output dim.
// S and O have two buffers, by the parity of the step; O of step k is added up after
// the weights of step k + 1 are out.  (With a step's four tiles in one thread each
// warp ran through 1000 straight instructions a step and waited for instruction
// fetches a third of its time.)
// Nothing depends on B, W or the grid.
#include <atomic>
#include <cstring>

#include "q8_device.cuh"

namespace rk {

namespace {

constexpr int DQ_SOFTMAX = 512;                   // softmax threads
constexpr int DQ_THREADS = 128 + DQ_SOFTMAX;
constexpr int DQ_TILE = 128;                      // tokens of a tile
constexpr int DQ_TILES = 4;                       // tiles of a step
constexpr int DQ_STEP_BYTES = DQ_TILES * DQ_TILE * HEAD_DIM;  // K (or V) of a step: 64 KiB
constexpr int DQ_SLOTS = 4;                       // steps the metadata runs ahead
constexpr int DQ_PRE = 1024;                      // row groups of the item list

template <int G, int H>
struct DqShape {
    static constexpr int NS = 4 * G < 16 ? 16 : 4 * G;  // columns of S: part * G + query
    static constexpr int NP = 3 * G <= 16 ? 16 : 32;    // columns of O: part * G + query
    static constexpr int TOKENS = DQ_TILES * DQ_TILE / H;  // of a step
    static constexpr int SHARE = 4 / H;                 // warpgroups to a KV head
    static constexpr int OWN = G > SHARE ? G / SHARE : 1;  // queries that one of them adds up
    // tensor memory: two buffers of S (4 tiles) and of O (H heads)
    static constexpr int TMEM_S = DQ_TILES * NS, TMEM_O = 2 * TMEM_S, TMEM_OBUF = H * NP;
    static constexpr int TMEM_COLS = TMEM_O + 2 * TMEM_OBUF <= 256 ? 256 : 512;
    // shared memory: the ring (a step's K or V to a stage), two buffers of q operands (one per
    // head of the bundle), weights (one per tile: 16 columns of O to a 16-byte row per token,
    // MN-major without swizzle)
    static constexpr int STAGES = G == 8 && H == 2 ? 2 : 3;  // as room allows (three, and one buffer of q: 48.5 us of the ragged rows, not 44)
    static constexpr int Q_BYTES = NS * 128, P_BYTES = NP * DQ_TILE;
    static constexpr int OFF_Q = STAGES * DQ_STEP_BYTES;
    static constexpr int OFF_P = OFF_Q + 2 * H * Q_BYTES;
    static constexpr int OFF_CTRL = OFF_P + DQ_TILES * P_BYTES;
};

// Step flags: first and last of its item, first and last of its queries, no step any more.
constexpr int DQ_FIRST = 1, DQ_LAST = 2, DQ_NEWQ = 4, DQ_ENDQ = 8, DQ_END = 16;

struct DqStep {
    int b, h, split;   // row, bundle of KV heads, split
    int cnt;           // tokens of the step (0: nothing to compute)
    int flags;         // DQ_*
    int bad;           // RK_STATUS_* bits of the row
};

struct DqCtrl {
    uint64_t full[3], empty[3];      // the ring
    uint64_t id_full[DQ_SLOTS], sc_full[DQ_SLOTS], slot_empty[DQ_SLOTS];
    uint64_t q_full[2], q_empty[2];
    uint64_t s_full[2], p_ready[2], o_full[2], o_read[2];  // by the parity of the step
    uint64_t never;
    uint32_t tmem_base;
    PipeCtl pipe;
    int total;                       // steps of the batch's rows (of one bundle)
    int scan[DQ_THREADS / 32];
    DqStep step[DQ_SLOTS];
    int ids[DQ_SLOTS][32];           // page of lane p's block: page p / H, head p % H of the step
    uint32_t odd[DQ_SLOTS];          // blocks whose scale is not one
    uint32_t wide[DQ_SLOTS];         // blocks of the heads whose scales of V lie too far apart in the item so far
    alignas(16) float4 sc[DQ_SLOTS][32];  // k scale, log2 of v's, 1 / v's of those blocks
    float qscale[2][16];             // score factor of each query head (log2 domain)
    uint32_t qbad[2];                // query heads out of range
    float red[2][16][8];             // a step's maximum of each softmax warp, by parity
    float lred[2][16][8];            // an item's sums of each softmax warp, by parity
    float2 ab[2][2][8];              // a step's scales of the sum so far and of its O, by parity, head, query
    float top[2][2][8];              // an item's maximum, by parity, head, query
    uint32_t fred[2][16];            // queries out of range; bit 31: a scale
    int pre[DQ_PRE];                 // steps before each group of rows
};
template <int G, int H>
constexpr int dq_smem_bytes() {
    static_assert(DqShape<G, H>::OFF_CTRL + sizeof(DqCtrl) <= 232448, "8-bit decode shared memory above the 227 KiB opt-in limit");
    return DqShape<G, H>::OFF_CTRL + (int)sizeof(DqCtrl);
}

// Visible keys of a row (0 where its metadata is unsafe) and its status bits.
__device__ __forceinline__ int row_keys(const AttnQ8Args& a, int b, int& bad) {
    const int kv = a.kv_lens[b], pos = a.position_ids[b];
    bad = (kv < 0 || kv > a.W * PAGE) ? RK_STATUS_KVLEN : 0;
    if (pos < 0) bad |= RK_STATUS_POSITION;
    return bad ? 0 : (pos < kv ? pos + 1 : kv);
}
// ---- split geometry: one or two zones of equal splits (AttnQ8Args::zone) ----

// Splits of a row of n keys (one for an empty row).
__device__ __forceinline__ int splits_of(const AttnQ8Args& a, int n) {
    if (n <= 0) return 1;
    const int z = n > a.zone[1].token;
    return a.zone[z].split + (n - a.zone[z].token + a.zone[z].size - 1) / a.zone[z].size;
}
// Tokens [first, end) of split s.
__device__ __forceinline__ void split_range(const AttnQ8Args& a, int s, int n, int& first, int& end) {
    const int z = s >= a.zone[1].split;
    first = a.zone[z].token + (s - a.zone[z].split) * a.zone[z].size;
    end = min(n, first + a.zone[z].size);
}
// Steps of T tokens of a row (one for an empty row).
template <int T>
__device__ __forceinline__ int row_steps(const AttnQ8Args& a, int n) {
    if (n <= 0) return 1;
    const int z = n > a.zone[1].token;
    const int len = n - a.zone[z].token, full = len / a.zone[z].size;
    return a.zone[z].step + full * a.zone[z].steps + (len - full * a.zone[z].size + T - 1) / T;
}
// First split of a row that starts at its step r or later; r becomes that split's first step.
__device__ __forceinline__ int split_at(const AttnQ8Args& a, int& r) {
    const int z = r >= a.zone[1].step;
    const int k = (r - a.zone[z].step + a.zone[z].steps - 1) / a.zone[z].steps;
    r = a.zone[z].step + k * a.zone[z].steps;
    return a.zone[z].split + k;
}

// A CTA's items: the splits whose first step, in the order of row, bundle, split, lies in the
// CTA's share of all steps.
template <int T>
struct DqItems {
    int b, h, s, n, ns, bad;  // the item: row, bundle, split; the row's keys, splits, status
    int at, hi;               // its first step, the share's end (the host bounds all steps by INT32_MAX)

    __device__ __forceinline__ bool valid(const AttnQ8Args& a) const { return b < a.B && at < hi; }
    __device__ __forceinline__ void row(const AttnQ8Args& a) {
        if (b < a.B) {
            n = row_keys(a, b, bad);
            ns = splits_of(a, n);
        }
    }
    __device__ void start(const AttnQ8Args& a, const DqCtrl* c, int bundles) {
        const unsigned all = (unsigned)(c->total * bundles), each = all / gridDim.x, rest = all % gridDim.x;
        at = (int)(each * blockIdx.x + rest * blockIdx.x / gridDim.x);
        hi = (int)(each * (blockIdx.x + 1) + rest * (blockIdx.x + 1) / gridDim.x);
        const int per = (a.B + DQ_PRE - 1) / DQ_PRE, groups = (a.B + per - 1) / per;
        int lo = 0, top = groups;
        while (top - lo > 1) {
            const int mid = (lo + top) >> 1;
            if (c->pre[mid] * bundles <= at) lo = mid;
            else top = mid;
        }
        b = lo * per;
        int base = c->pre[lo] * bundles;
        while (true) {
            row(a);
            const int sr = row_steps<T>(a, n);
            const int in = at - base;
            if (in < sr * bundles || b + 1 >= a.B) {
                h = in / sr;
                int r = in % sr;
                s = split_at(a, r);
                at = base + h * sr + min(r, sr);
                if (s >= ns) wrap(a, bundles);
                return;
            }
            base += sr * bundles;
            ++b;
        }
    }
    __device__ __forceinline__ void wrap(const AttnQ8Args& a, int bundles) {  // the row's next bundle, or the next row
        s = 0;
        if (++h == bundles) {
            h = 0;
            ++b;
            row(a);
        }
    }
    __device__ __forceinline__ void next(const AttnQ8Args& a, int bundles) {
        int t0, t1;
        split_range(a, s, n, t0, t1);
        at += max(1, (t1 - t0 + T - 1) / T);
        if (++s == ns) wrap(a, bundles);
    }
};

// One query head of a row (a warp): rotated, over a power of two, as four e4m3 parts in rows
// part * G + g of the operand qt.  wl, wh: dims 2 lane, 2 lane + 1 and the 64 above.
// Returns whether it is out of range (then zeros).
template <int G>
__device__ __forceinline__ bool prepare_query(uint8_t* qt, int g, uint32_t wl, uint32_t wh, float c0, float s0, float c1, float s1,
                                              float scale, float* factor, int lane) {
    uint32_t m = __vmaxu2(wl & 0x7fff7fffu, wh & 0x7fff7fffu);
    m = __reduce_max_sync(0xffffffffu, max(m & 0xffffu, m >> 16));
    const bool bad = m >= Q8_LIMIT_BF16;
    const int e = bad ? 0 : q8_exponent(m);
    const float inv = pow2(-e);
    const float2 l = make_float2(bf16lo(wl) * inv, bf16hi(wl) * inv), u = make_float2(bf16lo(wh) * inv, bf16hi(wh) * inv);
    float2 x = make_float2(l.x * c0 - u.x * s0, l.y * c1 - u.y * s1);
    float2 y = make_float2(u.x * c0 + l.x * s0, u.y * c1 + l.y * s1);
    if (bad) x = y = make_float2(0.0f, 0.0f);
    qt += 2 * lane & 15;
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        if (p == 2) {
            x = make_float2(x.x * 256.0f, x.y * 256.0f);
            y = make_float2(y.x * 256.0f, y.y * 256.0f);
        }
        const uint32_t at = sw128_off(p * G + g, lane >> 3);
        *reinterpret_cast<uint16_t*>(qt + at) = (uint16_t)take_part(x);
        *reinterpret_cast<uint16_t*>(qt + (at ^ 64)) = (uint16_t)take_part(y);  // chunk + 4
    }
    if (lane == 0) *factor = scale * pow2(e);
    return bad;
}

template <int G, int H>
__global__ void __launch_bounds__(DQ_THREADS, 1)
    decode_q8_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                     const __grid_constant__ AttnQ8Args a) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* sm = smem_raw;
    using Sh = DqShape<G, H>;
    DqCtrl* c = reinterpret_cast<DqCtrl*>(sm + Sh::OFF_CTRL);
    const uint32_t s_base = smem_u32(sm);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    constexpr int NS = Sh::NS, NP = Sh::NP, STAGES = Sh::STAGES;
    griddep_launch_dependents();  // the merge may become resident; it waits for this grid's end

    // ---- set-up: barriers, tensor memory, operands that stay zero, the item list ----
    if (tid == 0) {
        c->pipe.abort = 0;
        c->qbad[0] = 0;
        c->pipe.limit_ns = wait_limit(a.wait_limit_ns);
        for (int i = 0; i < Sh::STAGES; ++i) {
            mbar_init(smem_u32(&c->full[i]), 1);
            mbar_init(smem_u32(&c->empty[i]), 1);
        }
        for (int i = 0; i < DQ_SLOTS; ++i) {
            mbar_init(smem_u32(&c->id_full[i]), 1);
            mbar_init(smem_u32(&c->sc_full[i]), 1);
            mbar_init(smem_u32(&c->slot_empty[i]), 19);  // producer, issuer, q, softmax warps
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&c->q_full[i]), 16);      // lanes of the q warp, or the softmax warps
            mbar_init(smem_u32(&c->q_empty[i]), 17);     // issuer's commit, softmax warps
            mbar_init(smem_u32(&c->s_full[i]), 1);
            mbar_init(smem_u32(&c->p_ready[i]), 16);
            mbar_init(smem_u32(&c->o_full[i]), 1);
            mbar_init(smem_u32(&c->o_read[i]), 16);
        }
        mbar_init(smem_u32(&c->never), 1);
        fence_mbar_init();
    }
    for (int i = tid; i < (Sh::OFF_CTRL - Sh::OFF_Q) / 16; i += DQ_THREADS)
        reinterpret_cast<uint4*>(sm + Sh::OFF_Q)[i] = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
    if (warp == 1) {
        tmem_alloc(smem_u32(&c->tmem_base), Sh::TMEM_COLS);
        tmem_relinquish();
    }
    {
        // Steps before each group of `per` rows, a group to a thread and pass.
        const int per = (a.B + DQ_PRE - 1) / DQ_PRE, groups = (a.B + per - 1) / per;
        int base = 0;
        for (int g0 = 0; g0 < groups; g0 += DQ_THREADS) {
            const int gr = g0 + tid;
            int cnt = 0;
            for (int b = gr * per; gr < groups && b < min(a.B, gr * per + per); ++b) {
                int bad;
                const int n = row_keys(a, b, bad);
                cnt += row_steps<Sh::TOKENS>(a, n);
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
            int x = lane < DQ_THREADS / 32 ? c->scan[lane] : 0;
            const int own = x;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int t = __shfl_up_sync(0xffffffffu, x, o);
                if (lane >= o) x += t;
            }
            const int before = base + __shfl_sync(0xffffffffu, x - own, warp);
            base += __shfl_sync(0xffffffffu, x, 31);
            if (gr < groups) c->pre[gr] = before + v - cnt;
        }
        if (tid == 0) c->total = base;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = c->tmem_base;
    PipeCtl* pc = &c->pipe;
    const int bundles = a.Hkv / H;
    using Items = DqItems<Sh::TOKENS>;

    if (warp == 3) {
        // ==================================================== metadata ====
        // lane p: block p of the step, page p / H and head p % H of the bundle
        int slot = 0, use = 0;  // ring position and how often it went round
        bool ok = true;
        DqStep st{};
        Items it;
        it.start(a, c, bundles);
        int t = 0, t1 = 0, id = 0;  // the step's first token, the item's end, the lane's page id
        const int my_page = lane / H;
        bool newq = true;
        VSpan span;  // of the lane's blocks of the item
        auto page_id = [&]() {
            return my_page * PAGE < t1 - t ? __ldg(a.block_table + (size_t)st.b * a.W + t / PAGE + my_page) : 0;
        };
        auto item = [&]() {  // the first step of the item `it` and its page ids
            st = DqStep{};
            st.flags = DQ_END;
            t = t1 = 0;
            if (it.valid(a)) {
                st.b = it.b;
                st.h = it.h;
                st.split = it.s;
                st.bad = it.bad;
                st.flags = DQ_FIRST | (newq ? DQ_NEWQ : 0);
                split_range(a, it.s, it.n, t, t1);
            }
            id = page_id();
        };
        item();
        while (ok) {
            const int cnt = max(0, min(Sh::TOKENS, t1 - t));
            const bool mine = my_page * PAGE < cnt;
            const bool oob = mine && (id < 0 || id >= a.num_pages);
            const bool end = st.flags & DQ_END, last = t + Sh::TOKENS >= t1;
            if (last && !end) {  // the next item, before this step is told: it may have the same queries
                const int b = it.b, h = it.h;
                it.next(a, bundles);
                newq = !it.valid(a) || it.b != b || it.h != h;
                st.flags |= DQ_LAST | (newq ? DQ_ENDQ : 0);
            }
            st.cnt = cnt;
            if (__any_sync(0xffffffffu, oob)) {
                st.bad |= RK_STATUS_PAGE_OOB;
                st.cnt = 0;
            }
            int good = 1;
            if (lane == 0) good = mbar_wait(smem_u32(&c->slot_empty[slot]), (uint32_t)((use & 1) ^ 1), pc);
            if (!(ok = __shfl_sync(0xffffffffu, good, 0) != 0)) break;
            c->ids[slot][lane] = id;
            if (lane == 0) c->step[slot] = st;
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&c->id_full[slot]));
            float ks = 1.0f, vs = 1.0f;
            if (mine && st.cnt > 0) {
                const size_t block = (size_t)id * a.Hkv + st.h * H + lane % H;
                ks = __ldg(a.k_scale + block);
                vs = __ldg(a.v_scale + block);
            }
            if (st.flags & DQ_FIRST) span = VSpan();
            // the next step's page ids travel while this step's scales do
            const bool scaled = mine && st.cnt > 0;
            st.bad = st.flags = 0;  // said once
            if (last) {
                if (!end) item();
            } else {
                t += Sh::TOKENS;
                id = page_id();
            }
            const bool odd = !scale_ok(ks) || !scale_ok(vs);
            if (odd) ks = vs = 1.0f;
            if (scaled) span.add(vs);
            uint32_t wide = 0;
            if (__any_sync(0xffffffffu, span.outside())) {
                VSpan all = span;
                all.join<H, 32>();
                wide = __ballot_sync(0xffffffffu, all.too_wide());
            }
            c->sc[slot][lane] = make_float4(ks, __log2f(vs), rcp(vs), 0.0f);
            const uint32_t odds = __ballot_sync(0xffffffffu, odd);
            if (lane == 0) {
                c->odd[slot] = odds;
                c->wide[slot] = wide;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&c->sc_full[slot]));
            if (++slot == DQ_SLOTS) {
                slot = 0;
                ++use;
            }
            if (end) break;
        }
    } else if (warp == 0) {
        // ==================================================== producer ====
        if (lane == 0) {
            prefetch_tmap(&kmap);
            prefetch_tmap(&vmap);
        }
        // The whole warp, converged: the copies' operands stay in uniform registers and one
        // elected lane issues.  Loops stay rolled: a step's worth of straight code is
        // fetched anew each time, and that, not the copies, set the pace (450 ns for 16 KiB).
        int slot = 0, use = 0, n = 0;  // n: stages filled
        uint32_t stg = 0, phase = 1;
        const uint64_t once = evict_first_policy();  // the cache passes by; the partials stay in L2 for the merge
        bool ok = true;
#pragma unroll 1
        while (ok) {
            if (!(ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&c->id_full[slot]), (uint32_t)(use & 1), pc)))) break;
            const int cnt = __shfl_sync(0xffffffffu, c->step[slot].cnt, 0), head = __shfl_sync(0xffffffffu, c->step[slot].h, 0) * H;
            const int id = c->ids[slot][lane];
            if (__any_sync(0xffffffffu, c->step[slot].flags & DQ_END)) break;
            if (lane == 0) mbar_arrive(smem_u32(&c->slot_empty[slot]));
            if (++slot == DQ_SLOTS) {
                slot = 0;
                ++use;
            }
            if (cnt == 0) continue;
            const int pages = (cnt + PAGE - 1) / PAGE;
#pragma unroll 1
            for (int kv = 0; kv < 2; ++kv, ++n) {
                const uint32_t fb = smem_u32(&c->full[stg]);
                if (!(ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&c->empty[stg]), phase, pc)))) break;
                arrive_expect_tx_elect(fb, (uint32_t)pages * H * Q8_BLOCK_BYTES);
                uint32_t dst = s_base + stg * DQ_STEP_BYTES;
                const CUtensorMap* map = kv ? &vmap : &kmap;
#pragma unroll 1
                for (int p = 0; p < pages; ++p, dst += H * Q8_BLOCK_BYTES)
                    if constexpr (H == 1) tma_load_3d_elect(dst, map, fb, 0, 0, __shfl_sync(0xffffffffu, id, p) * a.Hkv + head, once);
                    else tma_load_5d_elect(dst, map, fb, 0, 0, head, 0, __shfl_sync(0xffffffffu, id, p * H), once);
                if (++stg == STAGES) {
                    stg = 0;
                    phase ^= 1;
                }
            }
        }
        if (lane == 0 && pipe_aborted(pc))  // copies in flight land before the CTA's shared memory is released
            for (int i = max(0, n - STAGES); i < n; ++i)
                mbar_wait_drain(smem_u32(&c->full[i % STAGES]), (uint32_t)((i / STAGES) & 1));
    } else if (warp == 2) {
        // =========================================================== q ====
        int slot = 0, use = 0, nq = 0;
        bool ok = true;
        const uint64_t turn0 = a.rope_turns[2 * lane], turn1 = a.rope_turns[2 * lane + 1];
#pragma unroll 1
        while (ok) {
            if (!(ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&c->id_full[slot]), (uint32_t)(use & 1), pc)))) break;
            const volatile DqStep* st = &c->step[slot];
            const int b = st->b, h = st->h, flags = st->flags;
            if (flags & DQ_END) break;
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&c->slot_empty[slot]));
            if (++slot == DQ_SLOTS) {
                slot = 0;
                ++use;
            }
            if (!(flags & DQ_NEWQ)) continue;
            if (nq == 0) {  // the softmax warps'
                ++nq;
                continue;
            }
            const int buf = nq & 1;
            const uint32_t pos = (uint32_t)max(0, a.position_ids[b]);
            // A query head per turn of a rolled loop (100 instructions that stay in the
            // instruction buffer; four heads unrolled took 5.5 us a bundle of 16), the next
            // four on the way.
            constexpr int N = H * G, AHEAD = 4;
            const uint32_t* q = reinterpret_cast<const uint32_t*>(a.q) + ((size_t)b * a.Hq + h * N) * (HEAD_DIM / 2) + lane;
            uint32_t lo[AHEAD], hi[AHEAD];
#pragma unroll
            for (int i = 0; i < N * 2; i += 32)  // all of it on its way to L2, 128 bytes a lane
                if (i + lane < N * 2) asm volatile("prefetch.global.L2 [%0];" ::"l"(q - lane + (i + lane) * 32));
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) {
                lo[i] = i < N ? __ldg(q + i * 64) : 0;
                hi[i] = i < N ? __ldg(q + i * 64 + 32) : 0;
            }
            float c0, s0, c1, s1;
            rope_cos_sin(pos, turn0, c0, s0);
            rope_cos_sin(pos, turn1, c1, s1);
            if (!(ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&c->q_empty[buf]), (uint32_t)(((nq >> 1) & 1) ^ 1), pc)))) break;
            uint32_t badq = 0;
            uint8_t* qt = sm + Sh::OFF_Q + buf * H * Sh::Q_BYTES;
            int g = 0;
#pragma unroll 1
            for (int i = 0; i < N; ++i) {
                const uint32_t wl = lo[0], wh = hi[0];
#pragma unroll
                for (int e = 0; e + 1 < AHEAD; ++e) {
                    lo[e] = lo[e + 1];
                    hi[e] = hi[e + 1];
                }
                if (i + AHEAD < N) {
                    lo[AHEAD - 1] = __ldg(q + (i + AHEAD) * 64);
                    hi[AHEAD - 1] = __ldg(q + (i + AHEAD) * 64 + 32);
                }
                if (prepare_query<G>(qt, g, wl, wh, c0, s0, c1, s1, a.qk_scale_log2, &c->qscale[buf][i], lane)) badq |= 1u << i;
                if (++g == G) {
                    g = 0;
                    qt += Sh::Q_BYTES;
                }
            }
            if (lane == 0) c->qbad[buf] = badq;
            fence_proxy_async_smem();
            __syncwarp();
            if (lane < 16) mbar_arrive(smem_u32(&c->q_full[buf]));
            ++nq;
        }
    } else if (warp == 1) {
        // ================================================== MMA issuer ====
        // The whole warp, converged, so that the operands stay in uniform registers
        // (one lane alone took 130 cycles an MMA, most of it moving descriptors).
        constexpr uint32_t idS = idesc_e4m3_f32(DQ_TILE, NS, 0, 0);
        constexpr uint32_t idO = idesc_e4m3_f32(HEAD_DIM, NP, 1, 1);
        // operands from the cache: a head's groups of 8 tokens are H KiB apart
        constexpr uint32_t HI_KV = ((H * 1024u) >> 4) | (1u << 14) | (2u << 29);
        const uint32_t dT = desc_lo(s_base, 16);
        const uint32_t dQ = desc_lo(s_base + Sh::OFF_Q, 16), dP = desc_lo(s_base + Sh::OFF_P, 128);
        int slot = 0, use = 0, nq = 0, ks = 0;  // items, steps (S; a step fills two stages)
        int pv_cnt = 0;                         // tokens of the step whose PV is due
        auto wait = [&](uint64_t& bar, int parity) {
            return __all_sync(0xffffffffu, mbar_wait(smem_u32(&bar), (uint32_t)(parity & 1), pc)) != 0;
        };
        bool ok = !a.timeout_drill || __all_sync(0xffffffffu, drill_wait(smem_u32(&c->never), pc));
        // PV of step k
        auto issue_pv = [&](int k) -> bool {
            const int buf = k & 1, n = 2 * k + 1, stg = n % STAGES;
            if (!wait(c->o_read[buf], (k >> 1) + 1)) return false;  // step k - 2's result is read
            if (!wait(c->p_ready[buf], k >> 1)) return false;
            if (!wait(c->full[stg], n / STAGES)) return false;
            tc_fence_after();
#pragma unroll 1
            for (int j = 0; j < DQ_TILES; ++j) {
                const int left = pv_cnt - (j / H) * DQ_TILE, kn = (left + 31) / 32;  // k-steps that hold tokens
                if (left <= 0) break;
                const uint32_t d = tmem + Sh::TMEM_O + buf * Sh::TMEM_OBUF + (j % H) * NP;
                const uint32_t dv = dT + stg * (DQ_STEP_BYTES >> 4) + (j / H) * H * 1024 + (j % H) * 64;
                const uint32_t dp = dP + j * (Sh::P_BYTES >> 4);
                // a k-step is 4 groups of 8 tokens
                mma_f8_x4<256 * H, 32>(d, dv, dp, HI_KV, DESC_HI_ROWS16, idO, j >= H, kn);
            }
            umma_commit_elect(smem_u32(&c->empty[stg]));
            umma_commit_elect(smem_u32(&c->o_full[buf]));
            pv_cnt = 0;
            return true;
        };
#pragma unroll 1
        while (ok) {
            if (!(ok = wait(c->id_full[slot], use))) break;
            const int cnt = __shfl_sync(0xffffffffu, c->step[slot].cnt, 0);
            const int flags = __shfl_sync(0xffffffffu, c->step[slot].flags, 0);
            if (!(flags & DQ_END)) {
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&c->slot_empty[slot]));
                if (++slot == DQ_SLOTS) {
                    slot = 0;
                    ++use;
                }
            }
            // The PV that is due goes before this step's S.  (S first, where this step's K is
            // here before the weights are, gained nothing.)
            if (pv_cnt > 0 && !(ok = issue_pv(ks - 1))) break;
            if (flags & DQ_END) break;
            if ((flags & DQ_NEWQ) && !(ok = wait(c->q_full[nq & 1], nq >> 1))) break;
            if (cnt > 0) {
                const int n = 2 * ks, stg = n % STAGES, kb = ks & 1;
                if (!(ok = wait(c->full[stg], n / STAGES))) break;
                tc_fence_after();
#pragma unroll 1
                for (int j = 0; j < DQ_TILES && (j / H) * DQ_TILE < cnt; ++j)
                    mma_f8_x4<2, 2>(tmem + kb * Sh::TMEM_S + j * NS, dT + stg * (DQ_STEP_BYTES >> 4) + (j / H) * H * 1024 + (j % H) * 64,
                                    dQ + ((nq & 1) * H + j % H) * (Sh::Q_BYTES >> 4), HI_KV, DESC_HI, idS, 0u, 4);
                umma_commit_elect(smem_u32(&c->s_full[kb]));
                umma_commit_elect(smem_u32(&c->empty[stg]));
                pv_cnt = cnt;
                ++ks;
            }
            if (flags & DQ_ENDQ) {
                umma_commit_elect(smem_u32(&c->q_empty[nq & 1]));
                ++nq;
            }
        }
        if (!ok) {  // issued MMAs drain before tensor memory is released
            const uint64_t t0 = global_timer_ns();
            while (global_timer_ns() - t0 < 1000000ull) {
            }
        }
    } else {
        // ===================================================== softmax ====
        const int sw = warp - 4, wg = sw >> 2;         // softmax warp, warpgroup (tile)
        const int hj = wg % H, blk = wg / H;           // KV head of the bundle, token block of the step
        const int t = tid & 127;                       // token of the tile, output dim
        const uint32_t lane_addr = (uint32_t)((warp & 3) * 32) << 16;
        constexpr int OWN = Sh::OWN, SHARE = Sh::SHARE;  // queries blk, blk + SHARE, ... are this warpgroup's
        int slot = 0, use = 0, ni = 0, nq = 0, ks = 0;  // items, queries, steps so far
        // the running maximum of each query; from four on a query's in the lanes lane % G
        constexpr bool SPREAD = G >= 4;
        float M[SPREAD ? 1 : G], l[G];
        int bad = 0;         // the item's status bits
        uint32_t range = 0;  // queries that met a value FP32 cannot hold; bit 31: a scale that is none
        float o[OWN];
        // the step whose O is due
        int due = 0;
        DqStep dst{};
        int dbad = 0, dpar = 0;
        int done = 0;        // items written
        // The warps leave the loop together: one whose wait gave up goes on to the
        // next barrier, which tells the others.
        bool ok = true;
        auto wait = [&](uint64_t& bar, int parity) {
            if (ok) ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&bar), (uint32_t)(parity & 1), pc));
        };
        // Results of an item from the warps' sums (behind a barrier): a query's verdict and sum
        // in lane g of each warp, its dims by the threads.  (Each thread on its own for every
        // query took 300 ns a query, 2.4 us of an item of eight.)
        auto finish = [&](const DqStep& st, int par, int status, bool none) {
            // softmax warp i of this head: the head's warpgroups are hj, hj + H, ...
            auto of_head = [&](int i) { return ((i >> 2) * H + hj) * 4 + (i & 3); };
            uint32_t any = __reduce_or_sync(0xffffffffu, c->fred[par][of_head(lane % (16 / H))]);
            if (status == RK_STATUS_TIMEOUT) any = 0;  // nothing was summed up
            if (any >> 31) status |= RK_STATUS_SCALE;
            const int mine = lane % G;
            float sum = 0.0f;
#pragma unroll 4
            for (int w = 0; w < 16 / H; ++w) sum += c->lred[par][of_head(w)][mine];
            const bool over = !none && (((any >> mine) & 1u) || !(sum > 0.0f && sum < INFINITY));
            const bool fail = status || over, zero = fail || none;
            const float inv = zero ? 0.0f : rcp(sum);
            const uint32_t zeros = __ballot_sync(0xffffffffu, zero);
            const size_t row = (size_t)st.b * a.Hq + (st.h * H + hj) * G;
            if ((warp & 3) == 0 && lane < G && lane % SHARE == blk) {
                const float lse2 = fail ? __int_as_float(0x7fc00000) : none ? -INFINITY : c->top[par][hj][lane] - 8.0f + __log2f(sum);
                if (a.n_splits > 1) a.lse_part[(row + lane) * a.n_splits + st.split] = lse2;
                else a.lse[row + lane] = lse2 * 0.693147180559945309f;
                if (fail && a.status) atomicOr(a.status, status ? status : RK_STATUS_RANGE);
            }
            float* part = a.o_part + ((row + blk) * a.n_splits + st.split) * HEAD_DIM + t;
            __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(a.out) + (row + blk) * HEAD_DIM + t;
#pragma unroll
            for (int i = 0; i < OWN; ++i) {
                const int g = blk + SHARE * i;
                const float x = (zeros >> (g & 31)) & 1u ? 0.0f : o[i] * __shfl_sync(0xffffffffu, inv, g & 31);
                if (g < G) {
                    if (a.n_splits > 1) part[(size_t)(SHARE * i) * a.n_splits * HEAD_DIM] = x;
                    else out[SHARE * i * HEAD_DIM] = __float2bfloat16_rn(x);
                }
            }
            ++done;
        };
        // the first queries, a head to a warp
        wait(c->id_full[0], 0);
        {
            const int qrow = c->step[0].b, qh = c->step[0].h;
            if (ok && !(c->step[0].flags & DQ_END)) {
                constexpr int N = H * G;
                float c0, s0, c1, s1;
                const uint32_t pos = (uint32_t)max(0, a.position_ids[qrow]);
                const uint32_t* q = reinterpret_cast<const uint32_t*>(a.q) + ((size_t)qrow * a.Hq + qh * N) * (HEAD_DIM / 2) + lane;
#pragma unroll 1
                for (int i = sw; i < N; i += 16) {
                    const uint32_t wl = __ldg(q + i * 64), wh = __ldg(q + i * 64 + 32);
                    rope_cos_sin(pos, a.rope_turns[2 * lane], c0, s0);
                    rope_cos_sin(pos, a.rope_turns[2 * lane + 1], c1, s1);
                    if (prepare_query<G>(sm + Sh::OFF_Q + i / G * Sh::Q_BYTES, i % G, wl, wh, c0, s0, c1, s1, a.qk_scale_log2,
                                         &c->qscale[0][i], lane) &&
                        lane == 0)
                        atomicOr(&c->qbad[0], 1u << i);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&c->q_full[0]));
            }
        }
        while (true) {
            wait(c->id_full[slot], use);
            wait(c->sc_full[slot], use);
            DqStep st{};
            float4 ps = make_float4(1.0f, 0.0f, 1.0f, 0.0f);
            float sc[G];
            if (ok) {
                const volatile DqStep* s = &c->step[slot];
                st.b = s->b;
                st.h = s->h;
                st.split = s->split;
                st.cnt = s->cnt;
                st.flags = s->flags;
                st.bad = s->bad;
                ps = c->sc[slot][(8 * blk + (t >> 4)) * H + hj];
                const uint32_t odd = c->odd[slot], wide = c->wide[slot];
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&c->slot_empty[slot]));
                if (++slot == DQ_SLOTS) {
                    slot = 0;
                    ++use;
                }
                const int qb = nq & 1;
                if (st.flags & DQ_NEWQ) wait(c->q_full[qb], nq >> 1);
                if (st.flags & DQ_FIRST) {
#pragma unroll
                    for (int g = 0; g < G; ++g) {
                        M[SPREAD ? 0 : g] = -INFINITY;
                        l[g] = 0.0f;
                    }
                    bad = 0;
                    range = (c->qbad[qb] >> (hj * G)) & ((1u << G) - 1u);
                }
#pragma unroll
                for (int g = 0; g < G; ++g) sc[g] = c->qscale[qb][hj * G + g];
                constexpr uint32_t EACH = H == 1 ? 0xffffffffu : 0x55555555u;
                if (odd & (EACH << hj)) range |= 0x80000000u;
                if (wide & (EACH << hj)) range |= (1u << G) - 1u;
                if (st.flags & DQ_ENDQ) {
                    __syncwarp();
                    if (ok && lane == 0) mbar_arrive(smem_u32(&c->q_empty[qb]));
                    ++nq;
                }
                ni += (st.flags & DQ_LAST) != 0;
            }
            const int par = ks & 1;
            const bool have = blk * DQ_TILE < st.cnt;  // the tile holds tokens
            // scores of the thread's token: w = z + log2 vs (-inf past the last one)
            float w[G];
            if (st.cnt > 0) {
#pragma unroll
                for (int g = 0; g < G; ++g) w[g] = -INFINITY;
                wait(c->s_full[par], ks >> 1);
                tc_fence_after();
                if (have) {
                    uint32_t r[NS];
                    const uint32_t ts = tmem + lane_addr + par * Sh::TMEM_S + wg * NS;
                    if constexpr (NS == 16) tmem_ld16(ts, r);
                    else tmem_ld32(ts, r);
                    tmem_ld_wait();
                    if (blk * DQ_TILE + t < st.cnt) {
#pragma unroll
                        for (int g = 0; g < G; ++g) {
                            const float hi = __uint_as_float(r[g]) + __uint_as_float(r[G + g]);
                            const float lo = __uint_as_float(r[2 * G + g]) + __uint_as_float(r[3 * G + g]);
                            const float z = fmaf(lo, 1.0f / 256.0f, hi) * (ps.x * sc[g]);
                            if (!(fabsf(z) < INFINITY)) range |= 1u << g;
                            w[g] = z + ps.y;
                        }
                    }
                }
#pragma unroll
                for (int g = 0; g < G; ++g) {
                    const float x = warp_max(w[g]);
                    if (lane == 0) c->red[par][sw][g] = x;
                }
            }
            if (named_bar_or(1, DQ_SOFTMAX, !ok)) {
                ok = false;
                break;
            }
            if (st.cnt > 0) {
                float p[G];
                if constexpr (SPREAD) {  // a query to a lane, then to all lanes
                    float m = -INFINITY;
#pragma unroll
                    for (int i = 0; i < 16 / H; i += 32 / G) {  // softmax warp i of this head
                        const int sw_i = i + lane / G;
                        m = fmaxf(m, c->red[par][((sw_i >> 2) * H + hj) * 4 + (sw_i & 3)][lane % G]);
                    }
#pragma unroll
                    for (int k = G; k < 32; k <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, k));
                    m = fabsf(m) < INFINITY ? m : 0.0f;  // otherwise the query fails (range)
                    const float top = fmaxf(M[0], m);
                    const float alpha = ex2(M[0] - top), beta = ex2(m - top);
                    M[0] = top;
                    if (blk == 0 && t < G) c->ab[par][hj][t] = make_float2(alpha, beta);
#pragma unroll
                    for (int g = 0; g < G; ++g) {
                        p[g] = ex2(w[g] - __shfl_sync(0xffffffffu, m, g) + 8.0f);
                        l[g] = fmaf(l[g], __shfl_sync(0xffffffffu, alpha, g), p[g] * ps.z * __shfl_sync(0xffffffffu, beta, g));
                    }
                } else {
                    const int rw = ((lane & 15) >> 2) % H == hj ? lane & 15 : 4 * hj;  // a warp of this head
#pragma unroll
                    for (int g = 0; g < G; ++g) {
                        float m = warp_max(c->red[par][rw][g]);
                        m = fabsf(m) < INFINITY ? m : 0.0f;
                        const float top = fmaxf(M[g], m);
                        const float alpha = ex2(M[g] - top), beta = ex2(m - top);
                        M[g] = top;
                        p[g] = ex2(w[g] - m + 8.0f);
                        l[g] = fmaf(l[g], alpha, p[g] * ps.z * beta);
                        if (blk == 0 && t == 0) c->ab[par][hj][g] = make_float2(alpha, beta);
                    }
                }
                // the weights' buffer is free once the PV of the step before is done
                if (ks > 0) wait(c->o_full[par ^ 1], (ks - 1) >> 1);
                if (have) {
                    // p' = 2^(w - m + 8) as three e4m3 parts at 1, 2^-5, 2^-10: part * G + query of the token's row
                    uint32_t wd[NP / 4];
#pragma unroll
                    for (int i = 0; i < NP / 4; ++i) wd[i] = 0;
#pragma unroll
                    for (int g = 0; g < G; g += 2) {
                        float2 x = make_float2(p[g], g + 1 < G ? p[g + 1 < G ? g + 1 : g] : 0.0f);
#pragma unroll
                        for (int e = 0; e < 3; ++e) {
                            const int col = e * G + g;
                            wd[col >> 2] |= take_part(x) << (8 * (col & 3));
                            x = fmul2(x, make_float2(32.0f, 32.0f));  // at most 2^8 again: a part leaves 8 of 2^8
                        }
                    }
                    uint8_t* pt = sm + Sh::OFF_P + wg * Sh::P_BYTES + t * 16;
#pragma unroll
                    for (int i = 0; i < NP / 16; ++i)
                        *reinterpret_cast<uint4*>(pt + i * DQ_TILE * 16) = make_uint4(wd[4 * i], wd[4 * i + 1], wd[4 * i + 2], wd[4 * i + 3]);
                }
                if (st.cnt & 31) {
                    // the k-step that the last token is in: V rows behind it hold anything, and 0 times a NaN
                    // is not 0.  (The stage's use before this one is known to be over.)
                    const int nv = 2 * ks + 1, stg = nv % STAGES;
                    wait(c->full[stg], nv / STAGES);
                    const int r1 = (st.cnt + 31) & ~31;
                    uint8_t* vt = sm + stg * DQ_STEP_BYTES;
                    for (int i = tid - 128; ok && i < (r1 - st.cnt) * H * 8; i += DQ_SOFTMAX) {
                        const int tok = st.cnt + i / (8 * H), rest = i % (8 * H);
                        *reinterpret_cast<uint4*>(vt + (tok >> 3) * H * 1024 + (rest >> 3) * 1024 + (tok & 7) * 128 + (rest & 7) * 16) =
                            make_uint4(0, 0, 0, 0);
                    }
                }
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&c->p_ready[par]));
            }
            // the item's sums, at its last step
            const int ipar = (ni + 1) & 1;
            bad |= st.bad;
            if (st.flags & DQ_LAST) {
                if constexpr (SPREAD) {
                    if (blk == 0 && t < G) c->top[ipar][hj][t] = M[0];
                } else if (blk == 0 && t == 0) {
#pragma unroll
                    for (int g = 0; g < G; ++g) c->top[ipar][hj][g] = M[g];
                }
                // the lanes' sums: half of the queries to each half of the lanes, until a lane has one
                float x[G];
#pragma unroll
                for (int g = 0; g < G; ++g) x[g] = l[g];
                int mine = 0;
#pragma unroll
                for (int k = 1, m = G / 2; k < 32; k <<= 1, m >>= 1) {
                    const bool up = lane & k;
#pragma unroll
                    for (int g = 0; g < m; ++g) {
                        const float give = up ? x[g] : x[g + m];
                        x[g] = (up ? x[g + m] : x[g]) + __shfl_xor_sync(0xffffffffu, give, k);
                    }
                    if (m == 0) x[0] += __shfl_xor_sync(0xffffffffu, x[0], k);
                    else if (up) mine += m;
                }
                if (lane < G) c->lred[ipar][sw][mine] = x[0];
                range = __reduce_or_sync(0xffffffffu, range);
                if (lane == 0) c->fred[ipar][sw] = range;
            }
            // O of the step before
            if (due) {
                const int k = ks - 1, db = k & 1;
                wait(c->o_full[db], k >> 1);
                tc_fence_after();
                uint32_t r[OWN][3];
                const uint32_t to = tmem + lane_addr + Sh::TMEM_O + db * Sh::TMEM_OBUF + hj * NP;
#pragma unroll
                for (int i = 0; i < OWN; ++i)
#pragma unroll
                    for (int e = 0; e < 3; ++e) tmem_ld1(to + e * G + min(blk + SHARE * i, G - 1), r[i][e]);
                tmem_ld_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&c->o_read[db]));
                uint32_t over = 0;
#pragma unroll
                for (int i = 0; i < OWN; ++i) {
                    const float x = fmaf(fmaf(__uint_as_float(r[i][2]), 1.0f / 32.0f, __uint_as_float(r[i][1])), 1.0f / 32.0f, __uint_as_float(r[i][0]));
                    const float2 ab = c->ab[db][hj][min(blk + SHARE * i, G - 1)];
                    o[i] = fmaf(x, ab.y, o[i] * ab.x);
                    if (!(fabsf(o[i]) < INFINITY) && blk + SHARE * i < G) over |= 1u << (blk + SHARE * i);
                }
                if (dst.flags & DQ_LAST) {
                    // o may be beyond FP32 (a NaN code in V) in a dim only; the head's 128 threads agree on it
                    over = __reduce_or_sync(0xffffffffu, over);
                    if (over && lane == 0) atomicOr(&c->fred[dpar][sw], over);
                    if (named_bar_or(1, DQ_SOFTMAX, !ok)) {
                        ok = false;
                        break;
                    }
                    finish(dst, dpar, dbad, false);
                }
                due = 0;
            }
            if (st.flags & DQ_END) break;
            if (st.cnt > 0) {
                due = 1;
                dst = st;
                dbad = bad;
                dpar = ipar;
#pragma unroll
                for (int i = 0; i < OWN; ++i) {
                    if (st.flags & DQ_FIRST) o[i] = 0.0f;
                }
                ++ks;
            } else if (st.flags & DQ_LAST) {
                // nothing in this step: an empty row, or one that fails
                if (named_bar_or(1, DQ_SOFTMAX, !ok)) {
                    ok = false;
                    break;
                }
                finish(st, ipar, bad, M[0] == -INFINITY);
            }
        }
        if (!ok) {  // a wait gave up: this CTA's items from here on are written as failed
            Items it;
            it.start(a, c, bundles);
            for (int i = 0, skip = done; it.valid(a); ++i, it.next(a, bundles)) {
                if (i < skip) continue;
                DqStep st{};
                st.b = it.b;
                st.h = it.h;
                st.split = it.s;
                finish(st, 0, RK_STATUS_TIMEOUT, false);
            }
            if (tid == 128 && a.status) atomicOr(a.status, RK_STATUS_TIMEOUT);
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, Sh::TMEM_COLS);
    }
}

// Merge of the split partials of one (row, query head): weights 2^(lse_s - max lse), eight
// sums over the splits s = e, e + 8, ... in ascending order, added up in order of e: fixed by
// the row's split count alone.  A NaN partial fails the row, no visible key gives out = 0,
// lse = -inf.  MANY = false: a warp has a row, four dims to a lane and all eight sums (four rows
// to a block).  MANY = true: a block of two warps has a quarter of a row's dims, eight lanes to
// a sum, and asks for sixteen splits of each sum at a time.  Both add in the same order, so which
// one runs (a choice by the table and the number of rows) does not show in the result.  Bound by latency: the
// row's length, a round or two of loads, one of stores.
template <bool MANY>
__global__ void __launch_bounds__(MANY ? 64 : 128) merge_q8_kernel(const __grid_constant__ AttnQ8Args a) {
    constexpr int SUMS = MANY ? 1 : 8, AHEAD = MANY ? 16 : 1;
    __shared__ float4 acc_s[MANY ? 8 : 1][8];
    __shared__ float sum_s[8];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const size_t bh = MANY ? blockIdx.x >> 2 : (size_t)blockIdx.x * 4 + warp;
    if (!MANY && bh >= (size_t)a.B * a.Hq) return;
    const int e0 = MANY ? (int)(threadIdx.x >> 3) : 0;                     // this thread's (first) sum
    const int d4 = MANY ? (int)((blockIdx.x & 3) * 8) + (lane & 7) : lane;  // its four dims
    int bad0;
    const int ns = splits_of(a, row_keys(a, (int)(bh / a.Hq), bad0));
    griddep_wait();  // the partials are complete and visible
    const float* lp = a.lse_part + bh * a.n_splits;
    const float4* op = reinterpret_cast<const float4*>(a.o_part + bh * a.n_splits * HEAD_DIM) + d4;
    const float4 zero = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    float4 x[AHEAD][SUMS];
    float wt[AHEAD][SUMS];
    auto load = [&](int s0) {  // AHEAD rounds of eight splits from s0 on
#pragma unroll
        for (int r = 0; r < AHEAD; ++r)
#pragma unroll
            for (int e = 0; e < SUMS; ++e) {
                const int s = s0 + 8 * r + e0 + e;
                x[r][e] = s < ns ? op[(size_t)s * 32] : zero;
                wt[r][e] = s < ns ? lp[s] : -INFINITY;
            }
    };
    load(0);
    float m = -INFINITY;
    bool bad = false;
#pragma unroll 4
    for (int s = lane; s < ns; s += 32) {
        const float v = lp[s];
        bad |= v != v;
        m = fmaxf(m, v);
    }
    m = warp_max(m);
    bad = __any_sync(0xffffffffu, bad);
    __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(a.out) + bh * HEAD_DIM;
    const bool first = !MANY || (blockIdx.x & 3) == 0;  // says the row's lse
    if (bad || m == -INFINITY) {
        if (!MANY || e0 == 0) {
            reinterpret_cast<uint2*>(out)[d4] = make_uint2(0, 0);
            if (first && lane == 0) a.lse[bh] = bad ? __int_as_float(0x7fc00000) : -INFINITY;
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
        for (int r = 0; r < AHEAD; ++r)
#pragma unroll
            for (int e = 0; e < SUMS; ++e) {
                const float w = ex2(wt[r][e] - m);
                sum[e] += w;
                acc[e].x = fmaf(w, x[r][e].x, acc[e].x);
                acc[e].y = fmaf(w, x[r][e].y, acc[e].y);
                acc[e].z = fmaf(w, x[r][e].z, acc[e].z);
                acc[e].w = fmaf(w, x[r][e].w, acc[e].w);
            }
        s0 += 8 * AHEAD;
        if (s0 < ns) load(s0);
    }
    float4 r = acc[0];
    float l = sum[0];
    if constexpr (MANY) {
        acc_s[e0][lane & 7] = acc[0];
        if ((lane & 7) == 0) sum_s[e0] = sum[0];
        __syncthreads();
        if (e0) return;
    }
#pragma unroll
    for (int e = 1; e < 8; ++e) {
        const float4 y = MANY ? acc_s[MANY ? e : 0][lane & 7] : acc[e % SUMS];
        r.x += y.x;
        r.y += y.y;
        r.z += y.z;
        r.w += y.w;
        l += MANY ? sum_s[e] : sum[e % SUMS];
    }
    const float inv = 1.0f / l;
    reinterpret_cast<uint2*>(out)[d4] = make_uint2(pack_bf16x2(r.x * inv, r.y * inv), pack_bf16x2(r.z * inv, r.w * inv));
    if (first && lane == 0) a.lse[bh] = (m + log2f(l)) * 0.693147180559945309f;
}

std::atomic<uint64_t> g_configured{0};
std::atomic<int> g_sms[64];

template <int G, int H>
cudaError_t launch_one(const CUtensorMap& km, const CUtensorMap& vm, const AttnQ8Args& a, unsigned grid, cudaStream_t stream,
                       bool configure) {
    if (configure)
        return cudaFuncSetAttribute(decode_q8_kernel<G, H>, cudaFuncAttributeMaxDynamicSharedMemorySize, dq_smem_bytes<G, H>());
    decode_q8_kernel<G, H><<<grid, DQ_THREADS, dq_smem_bytes<G, H>(), stream>>>(km, vm, a);
    return cudaGetLastError();
}
template <int G>
cudaError_t launch_bundle(int bundle, const CUtensorMap& km, const CUtensorMap& vm, const AttnQ8Args& a, unsigned grid,
                          cudaStream_t stream, bool configure) {
    return bundle == 2 ? launch_one<G, 2>(km, vm, a, grid, stream, configure) : launch_one<G, 1>(km, vm, a, grid, stream, configure);
}
cudaError_t launch_any(int group, int bundle, const CUtensorMap& km, const CUtensorMap& vm, const AttnQ8Args& a, unsigned grid,
                       cudaStream_t stream, bool configure) {
    switch (group) {
        case 1: return launch_bundle<1>(bundle, km, vm, a, grid, stream, configure);
        case 2: return launch_bundle<2>(bundle, km, vm, a, grid, stream, configure);
        case 4: return launch_bundle<4>(bundle, km, vm, a, grid, stream, configure);
        default: return launch_bundle<8>(bundle, km, vm, a, grid, stream, configure);
    }
}

}  // namespace

// KV heads to an item (and to a TMA box).
int decode_q8_bundle(int Hkv) { return Hkv % 2 == 0 ? 2 : 1; }

cudaError_t launch_decode_q8(const CUtensorMap& km, const CUtensorMap& vm, const AttnQ8Args& a, cudaStream_t stream) {
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const int bundle = decode_q8_bundle(a.Hkv);
    const uint64_t bit = dev < 64 ? (1ull << dev) : 0;
    if (!bit || !(g_configured.load() & bit)) {
        for (int g = 1; g <= 8; g *= 2)
            for (int h = 1; h <= 2; ++h)
                if ((e = launch_any(g, h, km, vm, a, 0, stream, true)) != cudaSuccess) return e;
        if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
        if (bit) g_sms[dev].store(sms);
        g_configured.fetch_or(bit);
    } else {
        sms = g_sms[dev].load();
    }
    const long long most = (long long)a.B * (a.Hkv / bundle) * a.n_splits;
    const unsigned grid = (unsigned)(most < sms ? most : sms);
    e = launch_any(a.G, bundle, km, vm, a, grid, stream, false);
    if (e != cudaSuccess || a.n_splits <= 1) return e;
    const long long rows = (long long)a.B * a.Hq;
    // Rows in quarters where the table holds long ones, unless there are so many rows and heads that the
    // quarters queue.  Whole calls in us, quarters / whole rows: 32 rows and heads past 100000 87.0 / 96.8,
    // 128 of 20000 74.7 / 78.8, 512 of 16000 90.2 / 91.8; 1024 of 8000 91.9 / 89.6, 2048 of 4096 in a table of
    // 131072 96.4 / 89.4, 2048 of 100 to 600 there 29.2 / 21.8.
    const bool many = a.n_splits > 32 && rows <= 512;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(many ? rows * 4 : (rows + 3) / 4));
    cfg.blockDim = dim3(many ? 64 : 128);
    cfg.stream = stream;
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return many ? cudaLaunchKernelEx(&cfg, merge_q8_kernel<true>, a) : cudaLaunchKernelEx(&cfg, merge_q8_kernel<false>, a);
}

}  // namespace rk
