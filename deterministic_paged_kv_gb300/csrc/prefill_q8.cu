// prefill_q8.cu -- causal chunked prefill over the 8-bit page cache (tcgen05).
//
// Operation: the paged prefill of "WS2 PR7 Fused Attention Backend Alignment",
// "Current Implementation", over e4m3 codes whose K was rotated when it was written.
// Work units (two q-tiles of one row and KV head), their heaviest-first order, the
// persistent grid and the online softmax are those of the BF16 prefill kernel.
//
// Operands: the codes of K and V become FP16 (exact) on their way into shared memory; q is
// rotated, scaled to below 362 by a power of two per query, and rounded to FP16 (2^-11 at
// most, the precision of the BF16 kernel's scores); P is FP16, scaled to at most 2^15 (it
// keeps 2^-11 of a weight down to 2^-21 of the largest).  A page's scales are constants of
// 16 columns: the softmax folds K's into its multiplier and V's into the exponent,
// w = z + log2(vs), and divides the row sum's page partials by vs, some 40 instructions of 600
// a tile and row.
// (K as it is, in fp8 MMAs against q in three e4m3 parts, needs no conversion and keeps q to
// 2^-16, but its 12 MMAs a tile read 96 KiB of operands where 8 of FP16 read 64, took 125
// cycles each, and left the copies no room in the shared memory's bandwidth: 925 us for
// S = 8192, 137 us for the chunk.)
// What bounds it: the chain softmax (1760 cycles) -> hand-over (250) -> PV and S of the next
// tile (16 MMAs of 108 cycles) of each q-tile, two of which overlap: 3700 cycles a KV tile.  The
// MMAs would take 64 each, but S reads both operands from shared memory at all of its bandwidth,
// and the conversions take 40% of what they leave.  (An issuer to each q-tile: 538 us, as the
// MMAs of the two then share the pipe and both chains grow; a maximum found along with the
// exponentials and the tile done again where it rose: 500 us.)
// S = 8192 of 32 heads: 474 us, tensor pipe 49% active; 4 chunks of 512 behind 1536: 72 us
// (256 units on 152 CTAs: two units where 1.68 would be even); 33 queries: 22 us.
// Roles (512 threads, registers rebalanced with setmaxnreg):
//   warp 15      scheduler: each unit's metadata, published as a descriptor (two slots);
//   warpgroup 0  transform: K and V tiles from the cache to FP16 operands (V zero past the last
//                key), scales; q of both q-tiles of a unit, as soon as the unit before has read
//                its own (the CTA's first are made by the softmax warpgroups, which have nothing
//                to do yet: 2 us of a call).  Codes come by cp.async, a thread's own 16 bytes of
//                each page, a tile ahead, and are converted two pages to a turn of a loop (with
//                the codes in registers and all unrolled the code pushed the softmax's out of
//                the instruction cache: 615 us of S = 8192 where the loop took 468);
//   warpgroups 1, 2  softmax of q-tile 0, 1: a thread per accumulator row;
//   warp 13      MMA issuer (converged);
//   warp 14      how far V's scales of a unit lie apart (in the transform warps this took 3%: they have
//                no register left);
//   warp 12      nothing.
// Nothing depends on B, W or the grid.
#include <atomic>

#include "q8_device.cuh"

namespace rk {

namespace {

constexpr int PQ_THREADS = 512;
constexpr int WARP_MMA = 13, WARP_SPAN = 14, WARP_SCHED = 15;
constexpr int KST = 2, VST = 2;                 // K stages, V stages
constexpr int SCST = 4;                         // scale slots: one more than K stages at least
constexpr uint32_t TMEM_COLS = 512;             // S0 [0,128) S1 [128,256) O0 [256,384) O1 [384,512)
constexpr float RESCALE_SLACK = 8.0f, P_BIAS = 7.0f;
// A running maximum from here on (log2 domain; one FP32 step is 1/8) is subtracted before the bias is
// added: in one sum with it the bias and log2(vs) drown, and a weight may pass FP16's 2^16.  Below, the
// sum's roundings are under 1/4 and a weight stays under 2^15.25.
constexpr float FAR_MAX = 1048576.0f;

// A page's factor of raw scores (log2 domain) for one query.  Not 0 where the product underflows, as
// masked scores are -inf: a raw score is below 2^25, so 2^-126 of it is as good as nothing.  NaN (a
// query out of range) stays.
__device__ __forceinline__ float score_factor(float k_scale, float q_scale) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(k_scale * q_scale), "f"(1.17549435e-38f));
    return r;
}
constexpr uint32_t UNIT_READERS = 32 + 32 + 128 + 256;

// setmaxnreg split (sum 4 x 128 = the 512 x 128 registers the CTA launches with)
constexpr int REG_XFORM = 96, REG_SOFTMAX = 184, REG_CTRL = 48;
static_assert(REG_XFORM + 2 * REG_SOFTMAX + REG_CTRL == 4 * 128, "register split must sum to the launch budget");

constexpr int OFF_Q = 0;                             // [q-tile][64-dim half][128 rows][128 B]
constexpr int OFF_K = OFF_Q + 2 * PF_TILE_BYTES;     // [64-dim half][128 rows][128 B]
constexpr int OFF_V = OFF_K + KST * PF_TILE_BYTES;   // [page][64-dim half][16 rows][128 B]
constexpr int OFF_C = OFF_V + VST * PF_TILE_BYTES;   // codes of the next tile: K, V (128 rows of 128 B each)
constexpr int OFF_BAR = OFF_C + 2 * PF_BN * HEAD_DIM;

struct PqUnit {
    int end, b, kvh, pair;
    int kv_len, nt0, nt1, n_keys;  // keys, KV tiles of q-tile 0 / 1, keys that the pair reads
    int bad;
};

constexpr int Q_BAD = -128;
struct PqBars {
    uint64_t q_ready[2], q_empty;
    uint64_t k_full[KST], k_empty[KST], v_full[VST], v_empty[VST], sc_full[SCST];
    uint64_t s_full[2], p_ready[2], o_done[2], o_free[2];
    uint64_t u_full[2], u_empty[2];
    uint64_t r_full[2], r_empty[2];      // a unit's verdict: transform threads and warp 14 -> softmax
    uint64_t never;
    uint32_t tmem_base;
    PipeCtl pipe;
    PqUnit unit[2];
    alignas(16) uint8_t r_flag[2][128];  // 1: NaN code in V, 2: a scale that is none
    int r_wide[2];                       // V's scales too far apart
    alignas(16) float4 sc[SCST][PF_PAGES_PER_TILE];  // k scale, log2 of v's, 1 / v's
    int8_t qexp[2][PF_BM];               // exponent of a query's power of two; Q_BAD: out of range
    float qscale[2][PF_BM];              // score factor of each query (log2 domain); NaN: out of range
};
constexpr int PQ_SMEM_BYTES = OFF_BAR + (int)sizeof(PqBars);
static_assert(PQ_SMEM_BYTES <= 232448, "8-bit prefill shared memory above the 227 KiB opt-in limit");

// Unit k of this CTA in the heaviest-first order (positions c, 2 G - 1 - c, 2 G + c, ...).
__device__ __forceinline__ long long cta_unit(int k, int c, int g) {
    return (k & 1) ? (long long)(k + 1) * g - 1 - c : (long long)k * g + c;
}
__device__ __forceinline__ void unit_place(const AttnQ8Args& a, int n_qtiles, long long u, int& b, int& kvh, int& pair) {
    const int units = a.B * a.Hkv;
    pair = (n_qtiles + 1) / 2 - 1 - (int)(u / units);
    const int rem = (int)(u % units);
    b = rem / a.Hkv;
    kvh = rem % a.Hkv;
}

// Row r of a q-tile from query s0 on: query head kvh * G + r / rph, query s0 + (r & (rph - 1)), with
// rph = 128 / G = 1 << rsh queries to a tile.
__device__ __forceinline__ size_t query_row(const AttnQ8Args& a, int b, int kvh, int rsh, int s0, int r) {
    return ((size_t)b * a.Hq + kvh * a.G + (r >> rsh)) * a.Sq + s0 + (r & ((1 << rsh) - 1));
}

__device__ __forceinline__ void write_row(const AttnQ8Args& a, size_t row, float lse) {
    uint4* o = reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(a.out) + row * HEAD_DIM);
#pragma unroll 1
    for (int d = 0; d < HEAD_DIM / 8; ++d) o[d] = make_uint4(0, 0, 0, 0);
    a.lse[row] = lse;
}

// Unit k's metadata checks (one warp): kv_len, positions (the largest of each q-tile sets
// the keys it reads), every page id of the row's keys.
__device__ __forceinline__ PqUnit unit_meta(const AttnQ8Args& a, int n_qtiles, int rph, int k, int cta, int grid, long long total,
                                            int lane) {
    PqUnit d;
    d.b = d.kvh = d.pair = d.kv_len = d.nt0 = d.nt1 = d.n_keys = d.bad = 0;
    const long long u = cta_unit(k, cta, grid);
    d.end = u >= total;
    if (d.end) return d;
    unit_place(a, n_qtiles, u, d.b, d.kvh, d.pair);
    const int kv_len = a.kv_lens[d.b];
    int bad = (kv_len < 0 || kv_len > a.W * PAGE) ? RK_STATUS_KVLEN : 0;
    const int32_t* pos = a.position_ids + (size_t)d.b * a.Sq;
    const int s00 = 2 * d.pair * rph;
    int pm0 = -1, pm1 = -1, neg = 0;
#pragma unroll 1
    for (int r = lane; r < rph; r += 32) {
        if (s00 + r < a.Sq) {
            const int p = pos[s00 + r];
            neg |= p < 0;
            pm0 = max(pm0, p);
        }
        if (s00 + rph + r < a.Sq) {
            const int p = pos[s00 + rph + r];
            neg |= p < 0;
            pm1 = max(pm1, p);
        }
    }
    pm0 = __reduce_max_sync(0xffffffffu, pm0);
    pm1 = __reduce_max_sync(0xffffffffu, pm1);
    if (__reduce_or_sync(0xffffffffu, (unsigned)neg)) bad |= RK_STATUS_POSITION;
    const int row_pages = (bad & RK_STATUS_KVLEN) ? 0 : (kv_len + PAGE - 1) / PAGE;
    const int32_t* bt = a.block_table + (size_t)d.b * a.W;
    int oob = 0;
#pragma unroll 4
    for (int i = lane; i < row_pages; i += 32) {
        const int pg = __ldg(bt + i);
        oob |= (pg < 0) | (pg >= a.num_pages);
    }
    if (__reduce_or_sync(0xffffffffu, (unsigned)oob)) bad |= RK_STATUS_PAGE_OOB;
    const int nk0 = (bad || pm0 < 0) ? 0 : (pm0 >= kv_len ? kv_len : pm0 + 1);
    const int nk1 = (bad || pm1 < 0) ? 0 : (pm1 >= kv_len ? kv_len : pm1 + 1);
    d.kv_len = kv_len;
    d.nt0 = (nk0 + PF_BN - 1) / PF_BN;
    d.nt1 = (nk1 + PF_BN - 1) / PF_BN;
    d.n_keys = max(nk0, nk1);
    d.bad = bad;
    return d;
}

__device__ __forceinline__ bool read_unit(PqBars* bars, int k, PipeCtl* pc, PqUnit& u) {
    const int slot = k & 1;
    if (!mbar_wait(smem_u32(&bars->u_full[slot]), (uint32_t)((k >> 1) & 1), pc)) return false;
    const volatile PqUnit* src = &bars->unit[slot];
    u.end = src->end;
    u.b = src->b;
    u.kvh = src->kvh;
    u.pair = src->pair;
    u.kv_len = src->kv_len;
    u.nt0 = src->nt0;
    u.nt1 = src->nt1;
    u.n_keys = src->n_keys;
    u.bad = src->bad;
    mbar_arrive(smem_u32(&bars->u_empty[slot]));
    return true;
}

// Transpose of 16-byte elements among lanes 4 k .. 4 k + 3: lane i's element q becomes lane
// q's element i.
__device__ __forceinline__ void transpose4(uint32_t (&w)[4][4], int i) {
#pragma unroll
    for (int b = 1; b < 4; b <<= 1)
#pragma unroll
        for (int q = 0; q < 4; ++q)
            if (!(q & b)) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const bool up = i & b;  // keeps q | b, gives q
                    const uint32_t give = up ? w[q][e] : w[q | b][e];
                    const uint32_t got = __shfl_xor_sync(0xffffffffu, give, b);
                    if (up) w[q][e] = got;
                    else w[q | b][e] = got;
                }
            }
}

// q-tile `tile` of a row and KV head into the operand j by cp.async (a warpgroup; rows past the
// last query as zeros), as it is.
__device__ __forceinline__ void load_q(const AttnQ8Args& a, uint32_t s_base, int b, int kvh, int tile, int j, int rsh, int t) {
    const int rph = 1 << rsh, s0 = tile * rph, ch = t & 15;  // 16-byte chunk ch of rows t / 16 + 8 i
    const __nv_bfloat16* src = reinterpret_cast<const __nv_bfloat16*>(a.q) + query_row(a, b, kvh, rsh, s0, 0) * HEAD_DIM + ch * 8;
    const uint32_t dst = s_base + OFF_Q + j * PF_TILE_BYTES + (ch >> 3) * 16384;
#pragma unroll 4
    for (int r = t >> 4; r < PF_BM; r += 8) {
        const int si = r & (rph - 1);
        const bool in = s0 + si < a.Sq;
        cp_async16_or_zero(dst + sw128_off(r, ch & 7), src + (in ? ((size_t)(r >> rsh) * a.Sq + si) * HEAD_DIM : 0), in);
    }
    cp_async_commit();
}

// The operand j from bf16 to rotated FP16 in place (the warpgroup behind named barrier `bar`); its
// threads arrive at q_ready.
__device__ __forceinline__ void rotate_q(const AttnQ8Args& a, uint8_t* sm, PqBars* bars, int b, int tile, int j, int rsh, int t, int bar) {
    const int rph = 1 << rsh, s0 = tile * rph;
    uint8_t* qt = sm + OFF_Q + j * PF_TILE_BYTES;
    {   // the largest element of row t
        uint32_t m = 0;
#pragma unroll 4
        for (int i = 0; i < 16; ++i) {
            const uint4 w = *reinterpret_cast<const uint4*>(qt + (i >> 3) * 16384 + sw128_off(t, i & 7));
            m = __vmaxu2(m, __vmaxu2(__vmaxu2(w.x & 0x7fff7fffu, w.y & 0x7fff7fffu), __vmaxu2(w.z & 0x7fff7fffu, w.w & 0x7fff7fffu)));
        }
        m = max(m & 0xffffu, m >> 16);
        const bool bad = m >= Q8_LIMIT_BF16;
        const int e = bad ? 0 : q8_exponent(m);
        bars->qexp[j][t] = (int8_t)(bad ? Q_BAD : e);
        bars->qscale[j][t] = bad ? __int_as_float(0x7fc00000) : a.qk_scale_log2 * pow2(e);
    }
    named_bar_sync(bar, 128);
    // A thread has a position and 8 rotation pairs (dims 8 ch .. and 64 + 8 ch ..) of its G query
    // heads, so an angle is computed once for all of them.
    const int si = t & (rph - 1);
    const uint32_t pos = s0 + si < a.Sq ? (uint32_t)a.position_ids[(size_t)b * a.Sq + s0 + si] : 0;
#pragma unroll 1
    for (int ch = t >> rsh; ch < 8; ch += a.G) {
        float2 cs[4], sn[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            rope_cos_sin(pos, a.rope_turns[8 * ch + 2 * i], cs[i].x, sn[i].x);
            rope_cos_sin(pos, a.rope_turns[8 * ch + 2 * i + 1], cs[i].y, sn[i].y);
        }
#pragma unroll 2
        for (int r = si; r < PF_BM; r += rph) {
            uint4* pl = reinterpret_cast<uint4*>(qt + sw128_off(r, ch));
            uint4* ph = reinterpret_cast<uint4*>(qt + 16384 + sw128_off(r, ch));
            const uint4 lo = *pl, hi = *ph;
            const uint32_t lw[4] = {lo.x, lo.y, lo.z, lo.w}, hw[4] = {hi.x, hi.y, hi.z, hi.w};
            const int e = bars->qexp[j][r];
            const bool zero = e == Q_BAD;
            const float inv = zero ? 0.0f : pow2(-e);
            const float2 inv2 = make_float2(inv, inv);
            uint32_t ol[4], oh[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 l = fmul2(make_float2(bf16lo(lw[i]), bf16hi(lw[i])), inv2);
                const float2 h = fmul2(make_float2(bf16lo(hw[i]), bf16hi(hw[i])), inv2);
                const float2 x = ffma2(make_float2(-h.x, -h.y), sn[i], fmul2(l, cs[i]));
                const float2 y = ffma2(l, sn[i], fmul2(h, cs[i]));
                ol[i] = pack_f16x2(x.x, x.y);
                oh[i] = pack_f16x2(y.x, y.y);
            }
            // a row that is out of range has 0 times what may be infinite: zeros instead
            *pl = zero ? make_uint4(0, 0, 0, 0) : make_uint4(ol[0], ol[1], ol[2], ol[3]);
            *ph = zero ? make_uint4(0, 0, 0, 0) : make_uint4(oh[0], oh[1], oh[2], oh[3]);
        }
    }
    fence_proxy_async_smem();
    mbar_arrive(smem_u32(&bars->q_ready[j]));
}

__global__ void __launch_bounds__(PQ_THREADS, 1)
    prefill_q8_kernel(const __grid_constant__ AttnQ8Args a) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* sm = smem_raw;
    PqBars* bars = reinterpret_cast<PqBars*>(sm + OFF_BAR);
    const uint32_t s_base = smem_u32(sm);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, wg = warp >> 2;
    const int rph = PF_BM / a.G, rsh = 31 - __clz(rph), n_qtiles = (a.Sq + rph - 1) >> rsh;
    const int cta = (int)blockIdx.x, grid = (int)gridDim.x;
    const long long total = (long long)a.B * a.Hkv * ((n_qtiles + 1) / 2);
    PqUnit first{};
    if (warp == WARP_SCHED) first = unit_meta(a, n_qtiles, rph, 0, cta, grid, total, lane);
    if (tid == 0) {
        bars->pipe.abort = 0;
        bars->pipe.limit_ns = wait_limit(a.wait_limit_ns);
        mbar_init(smem_u32(&bars->never), 1);
        mbar_init(smem_u32(&bars->q_empty), 1 + 8);  // issuer's commit, softmax warps
        for (int k = 0; k < KST; ++k) {
            mbar_init(smem_u32(&bars->k_full[k]), 128);
            mbar_init(smem_u32(&bars->k_empty[k]), 1);
        }
        for (int k = 0; k < SCST; ++k) mbar_init(smem_u32(&bars->sc_full[k]), 1);
        for (int k = 0; k < VST; ++k) {
            mbar_init(smem_u32(&bars->v_full[k]), 128);
            mbar_init(smem_u32(&bars->v_empty[k]), 1);
        }
        for (int j = 0; j < 2; ++j) {
            mbar_init(smem_u32(&bars->q_ready[j]), 128);
            mbar_init(smem_u32(&bars->s_full[j]), 1);
            mbar_init(smem_u32(&bars->p_ready[j]), 128);
            mbar_init(smem_u32(&bars->o_done[j]), 1);
            mbar_init(smem_u32(&bars->o_free[j]), 128);
            mbar_init(smem_u32(&bars->u_full[j]), 1);
            mbar_init(smem_u32(&bars->u_empty[j]), UNIT_READERS);
            mbar_init(smem_u32(&bars->r_full[j]), 128 + 1);
            mbar_init(smem_u32(&bars->r_empty[j]), 256);
        }
        fence_mbar_init();
    }
    if (warp == WARP_MMA) {
        tmem_alloc(smem_u32(&bars->tmem_base), TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars->tmem_base;
    PipeCtl* pc = &bars->pipe;

    if (wg == 3) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REG_CTRL));
        if (warp == WARP_SCHED) {
            // ============================================== scheduler ====
            bool ok = true;
#pragma unroll 1
            for (int k = 0; ok; ++k) {
                const int slot = k & 1;
                const PqUnit m = k == 0 ? first : unit_meta(a, n_qtiles, rph, k, cta, grid, total, lane);
                ok = __shfl_sync(0xffffffffu,
                                 lane == 0 ? (int)mbar_wait(smem_u32(&bars->u_empty[slot]), (uint32_t)(((k >> 1) & 1) ^ 1), pc) : 0,
                                 0) != 0;
                if (!ok) break;
                if (lane == 0) {
                    bars->unit[slot] = m;
                    if (m.bad && a.status) atomicOr(a.status, m.bad);
                    mbar_arrive(smem_u32(&bars->u_full[slot]));
                }
                if (m.end) break;
            }
        } else if (warp == WARP_SPAN) {
            // ===================================== distance of V's scales ====
            bool ok = true;
            int wu = 0;  // work units
#pragma unroll 1
            for (int kk = 0; ok; ++kk) {
                PqUnit u;
                if (!(ok = __all_sync(0xffffffffu, read_unit(bars, kk, pc, u))) || __any_sync(0xffffffffu, u.end)) break;
                if (u.bad || max(u.nt0, u.nt1) == 0) continue;
                const int32_t* bt = a.block_table + (size_t)u.b * a.W;
                VSpan span;
#pragma unroll 1
                for (int p = lane; p < (u.n_keys + PAGE - 1) / PAGE; p += 32) {
                    const float vs = __ldg(a.v_scale + (size_t)__ldg(bt + p) * a.Hkv + u.kvh);
                    if (scale_ok(vs)) span.add(vs);
                }
                span.join<1, 32>();
                const int slot = wu & 1;
                ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&bars->r_empty[slot]), (uint32_t)(((wu >> 1) & 1) ^ 1), pc)) != 0;
                if (ok && lane == 0) {
                    bars->r_wide[slot] = span.too_wide();
                    mbar_arrive(smem_u32(&bars->r_full[slot]));
                }
                ++wu;
            }
        } else if (warp == WARP_MMA) {
            // ============================================= MMA issuer ====
            constexpr uint32_t idS = idesc_f16_f32(PF_BM, PF_BN);
            constexpr uint32_t idO = idesc_f16_f32(PF_BM, HEAD_DIM) | (1u << 16);  // FP16, V MN-major
            const uint32_t dQ = desc_lo(s_base + OFF_Q, 16), dK = desc_lo(s_base + OFF_K, 16), dV = desc_lo(s_base + OFF_V, 2048);
            constexpr uint32_t TILE = PF_TILE_BYTES >> 4;
            // g0: KV tiles before the unit; ph bit 0 work units, bits 2 + j s_full / p_ready of
            // q-tile j, bits 4 + j o_free
            int g0 = 0;
            uint32_t ph = 0;
            auto wait = [&](uint64_t& bar, uint32_t parity) {
                return __all_sync(0xffffffffu, mbar_wait(smem_u32(&bar), parity & 1u, pc)) != 0;
            };
            bool ok = !a.timeout_drill || __all_sync(0xffffffffu, drill_wait(smem_u32(&bars->never), pc));
#pragma unroll 1
            for (int kk = 0; ok; ++kk) {
                PqUnit u;
                if (!(ok = __all_sync(0xffffffffu, read_unit(bars, kk, pc, u))) || __any_sync(0xffffffffu, u.end)) break;
                const int nt0 = __shfl_sync(0xffffffffu, u.nt0, 0), nt1 = __shfl_sync(0xffffffffu, u.nt1, 0);
                const int n_tiles = max(nt0, nt1);
                if (__any_sync(0xffffffffu, u.bad != 0) || n_tiles == 0) continue;
                // O_j (+)= P_j(i) V(i); the unit's first PV into O_j waits for the epilogue before it.
                // P comes last: what follows it (PV, then S of the next tile) is the q-tile's chain,
                // and K and V are there long before.
                auto issue_pv = [&](int j, int i) -> bool {
                    if (i == 0 && !wait(bars->o_free[j], (ph >> (4 + j)) ^ 1u)) return false;
                    if (!wait(bars->p_ready[j], (ph >> (2 + j)) ^ (uint32_t)i)) return false;
                    tc_fence_after();
                    mma_ts_steps<0, 8, MN_MAJOR_PAGE, true>(tmem + 256 + j * 128, tmem + j * 128, dV + (uint32_t)((g0 + i) % VST) * TILE,
                                                            idO, i > 0 ? 1u : 0u);
                    return true;
                };
#pragma unroll 1
                for (int i = 0; i < n_tiles && ok; ++i) {
                    const int g = g0 + i;
                    if (i > 0 && !(ok = wait(bars->v_full[(g - 1) % VST], (uint32_t)((g - 1) / VST)))) break;
                    bool have_k = false;
#pragma unroll 1
                    for (int j = 0; j < 2 && ok; ++j) {
                        const int nt = j ? nt1 : nt0;
                        if (i > nt || nt == 0) continue;
                        if (i == 0 && !(ok = wait(bars->q_ready[j], ph))) break;
                        if (i > 0 && !(ok = issue_pv(j, i - 1))) break;
                        if (i == nt) {
                            umma_commit_elect(smem_u32(&bars->o_done[j]));
                            continue;
                        }
                        if (!have_k) {  // (not before PV, which does without)
                            if (!(ok = wait(bars->k_full[g % KST], (uint32_t)(g / KST)))) break;
                            have_k = true;
                        }
                        tc_fence_after();
                        mma_ss_steps<0, 8, K_MAJOR_128, K_MAJOR_128, true>(tmem + j * 128, dQ + (uint32_t)j * TILE,
                                                                           dK + (uint32_t)(g % KST) * TILE, idS, 0u);
                        umma_commit_elect(smem_u32(&bars->s_full[j]));
                    }
                    if (!ok) break;
                    umma_commit_elect(smem_u32(&bars->k_empty[g % KST]));                       // K(i) read by S(i)
                    if (i > 0) umma_commit_elect(smem_u32(&bars->v_empty[(g - 1) % VST]));      // V(i-1) read by PV(i-1)
                    if (i == n_tiles - 1) umma_commit_elect(smem_u32(&bars->q_empty));          // the unit's last S read q
                }
                if (!ok || !(ok = wait(bars->v_full[(g0 + n_tiles - 1) % VST], (uint32_t)((g0 + n_tiles - 1) / VST)))) break;
                tc_fence_after();
#pragma unroll 1
                for (int j = 0; j < 2 && ok; ++j) {
                    if ((j ? nt1 : nt0) != n_tiles) continue;
                    if (!(ok = issue_pv(j, n_tiles - 1))) break;
                    umma_commit_elect(smem_u32(&bars->o_done[j]));
                }
                if (!ok) break;
                umma_commit_elect(smem_u32(&bars->v_empty[(g0 + n_tiles - 1) % VST]));
                ph ^= 1u | ((uint32_t)(nt0 & 1) << 2) | ((uint32_t)(nt1 & 1) << 3) | (nt0 > 0 ? 16u : 0u) | (nt1 > 0 ? 32u : 0u);
                g0 += n_tiles;
            }
            if (!ok) {  // issued MMAs drain before tensor memory is released
                const uint64_t t0 = global_timer_ns();
                while (global_timer_ns() - t0 < 1000000ull) {
                }
            }
        }
        __syncwarp();
        named_bar_sync(2, PQ_THREADS);
    } else if (wg == 0) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REG_XFORM));
        // ================================================ transform WG ====
        // Tiles: the thread has 16 codes (chunk c) of rows r0 + 16 e, a row of each page.
        const int c = tid & 7, r0 = tid >> 3;
        int g0 = 0, wu = 0;  // KV tiles before the unit, work units
        // The warpgroup leaves the loop together: a warp whose wait gave up goes on to the next
        // barrier, which tells the others.
        bool ok = true;
        auto wait = [&](uint64_t& bar, int parity) {
            if (ok) ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&bar), (uint32_t)(parity & 1), pc));
            return ok;
        };
#pragma unroll 1
        for (int kk = 0;; ++kk) {
            PqUnit u;
            if (ok) ok = __all_sync(0xffffffffu, read_unit(bars, kk, pc, u));
            if (named_bar_or(3, 128, !ok)) {
                ok = false;
                break;
            }
            if (u.end) break;
            const int n_tiles = max(u.nt0, u.nt1);
            if (u.bad || n_tiles == 0) continue;
            const int32_t* bt = a.block_table + (size_t)u.b * a.W;
            const int n_pages = (u.n_keys + PAGE - 1) / PAGE;
            const size_t in_block = (size_t)u.kvh * Q8_BLOCK_BYTES + r0 * HEAD_DIM + c * 16, page_bytes = (size_t)a.Hkv * Q8_BLOCK_BYTES;
            auto page_ids = [&](int i) {  // lane e (of 8): page e of tile i, -1 past the last
                const int p = i * PF_PAGES_PER_TILE + (lane & 7);
                return p < n_pages ? __ldg(bt + p) : -1;
            };
            uint32_t odd = 0;  // 1: NaN code in V, 2: a scale that is none
            float ks = 1.0f, vs = 1.0f;
            uint8_t* codes = sm + OFF_C + r0 * HEAD_DIM + c * 16;  // the thread's chunk of page 0, K; pages 2 KiB, V 16 KiB on
            const uint32_t codes_s = smem_u32(codes);
            auto load_part = [&](int ids, int part) {  // K (0) or V (1) codes of a tile
                const uint8_t* cache = part ? a.v_cache : a.k_cache;
                const uint32_t dst = codes_s + part * PF_BN * HEAD_DIM;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int id = __shfl_sync(0xffffffffu, ids, e);
                    if (id >= 0) cp_async16(dst + e * Q8_BLOCK_BYTES, cache + (size_t)id * page_bytes + in_block);
                }
                cp_async_commit();
            };
            auto load_scales = [&](int ids) {
                ks = vs = 1.0f;
                if (tid < 8 && ids >= 0) {
                    ks = __ldg(a.k_scale + (size_t)ids * a.Hkv + u.kvh);
                    vs = __ldg(a.v_scale + (size_t)ids * a.Hkv + u.kvh);
                }
            };
            // Tile i of the unit from its codes to its operands; `next`: the pages of the tile after it,
            // whose codes are fetched as soon as this tile's have been read.
            auto convert = [&](int i, int next) {
                const int g = g0 + i, kst = g % KST, vst = g % VST;
                if (!wait(bars->k_empty[kst], (g / KST) ^ 1)) return;
                cp_async_wait<1>();  // K is here (V, committed after it, may not be)
                uint8_t* kt = sm + OFF_K + kst * PF_TILE_BYTES + (c >> 2) * 16384 + r0 * 128;
                // The 16 codes are chunks 2 c, 2 c + 1 (of 16 bytes, swizzled) of a half's row; lanes of the
                // upper half store theirs the other way round, so that 8 lanes meet 8 chunks.
                const bool up = c >= 4;
                const uint32_t c0 = (((2 * c & 7) ^ (r0 & 7)) << 4) ^ (up ? 16u : 0u), c1 = c0 ^ 16;
                uint4 ahead = *reinterpret_cast<const uint4*>(codes);
#pragma unroll 2
                for (int e = 0; e < 8; ++e) {
                    const uint4 w = up ? make_uint4(ahead.z, ahead.w, ahead.x, ahead.y) : ahead;
                    ahead = *reinterpret_cast<const uint4*>(codes + min(e + 1, 7) * Q8_BLOCK_BYTES);
                    *reinterpret_cast<uint4*>(kt + e * 2048 + c0) =
                        make_uint4(e4m3x2_to_f16x2(w.x), e4m3x2_to_f16x2(w.x >> 16), e4m3x2_to_f16x2(w.y), e4m3x2_to_f16x2(w.y >> 16));
                    *reinterpret_cast<uint4*>(kt + e * 2048 + c1) =
                        make_uint4(e4m3x2_to_f16x2(w.z), e4m3x2_to_f16x2(w.z >> 16), e4m3x2_to_f16x2(w.w), e4m3x2_to_f16x2(w.w >> 16));
                }
                if (tid < 8) {
                    // The slot's readers of SCST tiles ago are done: the stage of K was free, so S of tile
                    // g - KST is, and with it the softmax of the tile before that.
                    const bool none = !scale_ok(ks) || !scale_ok(vs);
                    if (none) odd |= 2;
                    bars->sc[g % SCST][tid] = none ? make_float4(1.0f, 0.0f, 1.0f, 0.0f) : make_float4(ks, __log2f(vs), rcp(vs), 0.0f);
                }
                if (warp == 0) {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&bars->sc_full[g % SCST]));
                }
                fence_proxy_async_smem();
                mbar_arrive(smem_u32(&bars->k_full[kst]));
                load_part(next, 0);
                load_scales(next);
                if (!wait(bars->v_empty[vst], (g / VST) ^ 1)) return;
                cp_async_wait<1>();
                uint8_t* vt = sm + OFF_V + vst * PF_TILE_BYTES + (c >> 2) * 2048 + r0 * 128;
                uint32_t nan = 0;
                ahead = *reinterpret_cast<const uint4*>(codes + PF_BN * HEAD_DIM);
#pragma unroll 2
                for (int e = 0; e < 8; ++e) {
                    uint4 w = up ? make_uint4(ahead.z, ahead.w, ahead.x, ahead.y) : ahead;
                    ahead = *reinterpret_cast<const uint4*>(codes + PF_BN * HEAD_DIM + min(e + 1, 7) * Q8_BLOCK_BYTES);
                    if (i * PF_BN + 16 * e + r0 >= u.n_keys) w = make_uint4(0, 0, 0, 0);  // 0 times a NaN is not 0
                    // a byte of 0x7f or 0xff: NaN
                    nan |= ((w.x & 0x7f7f7f7fu) + 0x01010101u) | ((w.y & 0x7f7f7f7fu) + 0x01010101u) |
                           ((w.z & 0x7f7f7f7fu) + 0x01010101u) | ((w.w & 0x7f7f7f7fu) + 0x01010101u);
                    *reinterpret_cast<uint4*>(vt + e * 4096 + c0) =
                        make_uint4(e4m3x2_to_f16x2(w.x), e4m3x2_to_f16x2(w.x >> 16), e4m3x2_to_f16x2(w.y), e4m3x2_to_f16x2(w.y >> 16));
                    *reinterpret_cast<uint4*>(vt + e * 4096 + c1) =
                        make_uint4(e4m3x2_to_f16x2(w.z), e4m3x2_to_f16x2(w.z >> 16), e4m3x2_to_f16x2(w.w), e4m3x2_to_f16x2(w.w >> 16));
                }
                if (nan & 0x80808080u) odd |= 1;
                fence_proxy_async_smem();
                mbar_arrive(smem_u32(&bars->v_full[vst]));
                load_part(next, 1);
            };
            int next = page_ids(0);
            load_part(next, 0);
            load_part(next, 1);
            load_scales(next);
            next = page_ids(1);
#pragma unroll 1
            for (int i = 0; i < n_tiles; ++i) {
                const int after = next;
                next = page_ids(i + 2);
                convert(i, after);
                if (i > 0 && !ok) break;
                if (i > 0) continue;
                // ---- q, with the unit's first tile done while the unit before was still at work
                // (the CTA's first: the softmax warpgroups') ----
                if (kk == 0) continue;
                wait(bars->q_empty, wu ^ 1);
                if (named_bar_or(3, 128, !ok)) {
                    ok = false;
                    break;
                }
#pragma unroll 1
                for (int j = 0; j < 2; ++j) load_q(a, s_base, u.b, u.kvh, 2 * u.pair + j, j, rsh, tid);
                cp_async_wait_all();  // (the next tile's codes too)
                named_bar_sync(3, 128);
#pragma unroll 1
                for (int j = 0; j < 2; ++j) rotate_q(a, sm, bars, u.b, 2 * u.pair + j, j, rsh, tid, 3);
            }
            cp_async_wait_all();
            const int slot = wu & 1;
            if (wait(bars->r_empty[slot], (wu >> 1) ^ 1)) {
                bars->r_flag[slot][tid] = (uint8_t)odd;
                mbar_arrive(smem_u32(&bars->r_full[slot]));
            }
            g0 += n_tiles;
            ++wu;
        }
        named_bar_sync(2, PQ_THREADS);
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REG_SOFTMAX));
        // =========================================== softmax WG j ======
        const int j = wg - 1;
        const int r = tid - 128 * wg;  // accumulator row == TMEM lane
        const uint32_t lane_addr = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t tS = tmem + j * 128, tO = tmem + 256 + j * 128;
        const float nanv = __int_as_float(0x7fc00000);
        // A wait gave up: the rows of this q-tile from the CTA's unit k on are written as failed.
        auto fail_from = [&](int k) {
#pragma unroll 1
            for (;; ++k) {
                const long long u = cta_unit(k, cta, grid);
                if (u >= total) break;
                int b, kvh, pair;
                unit_place(a, n_qtiles, u, b, kvh, pair);
                const int t0 = (2 * pair + j) * rph;
                if (t0 + (r & (rph - 1)) < a.Sq) write_row(a, query_row(a, b, kvh, rsh, t0, r), nanv);
            }
            if (r == 0 && a.status) atomicOr(a.status, RK_STATUS_TIMEOUT);
        };
        int g0 = 0;        // KV tiles before the unit
        uint32_t ph = 0;   // bit 0 s_full (this q-tile's tiles), bit 1 o_done, bits 2-3 work units
        bool ok = true;
#pragma unroll 1
        for (int kk = 0;; ++kk) {
            const int uslot = kk & 1;
            ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&bars->u_full[uslot]), (uint32_t)((kk >> 1) & 1), pc)) != 0;
            // (at the first unit the warpgroup's warps go on or leave together: it makes its own operand)
            if (kk == 0 && named_bar_or(4 + j, 128, !ok)) ok = false;
            if (!ok) {
                fail_from(kk);
                break;
            }
            const volatile PqUnit* un = &bars->unit[uslot];
            if (un->end) break;
            const int s0 = (2 * un->pair + j) * rph, s = s0 + (r & (rph - 1));
            const bool valid = s < a.Sq;
            const int n_tiles = max(un->nt0, un->nt1), nt = j ? un->nt1 : un->nt0;
            const size_t row = query_row(a, un->b, un->kvh, rsh, s0, r);
            if (un->bad || n_tiles == 0) {
                if (valid) write_row(a, row, un->bad ? nanv : -INFINITY);
                mbar_arrive(smem_u32(&bars->u_empty[uslot]));
                continue;
            }
            int n_vis;
            {
                const int p = valid ? a.position_ids[(size_t)un->b * a.Sq + s] : -1, kv_len = un->kv_len;
                n_vis = p < 0 ? 0 : (p >= kv_len ? kv_len : p + 1);
            }
            if (kk == 0) {
                load_q(a, s_base, un->b, un->kvh, 2 * un->pair + j, j, rsh, r);
                cp_async_wait_all();
                named_bar_sync(4 + j, 128);
                rotate_q(a, sm, bars, un->b, 2 * un->pair + j, j, rsh, r, 4 + j);
            }
            ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&bars->q_ready[j]), (ph >> 2) & 1u, pc));
            const float scr = bars->qscale[j][r];
            // The next unit's q may take the operand and the factors once every softmax warp has passed this
            // point, those of a q-tile without keys too: no S waits for those, so nothing else would
            // keep q_ready from completing twice before they look (a wait by parity then misses it), or q
            // from being made where they still make the CTA's first.
            __syncwarp();
            if (ok && lane == 0) mbar_arrive(smem_u32(&bars->q_empty));
            float m = -INFINITY, l = 0.0f;
#pragma unroll 1
            for (int i = 0; i < nt && ok; ++i) {
                const int g = g0 + i;
                if (!(ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&bars->s_full[j]), (ph ^ (uint32_t)i) & 1u, pc)))) break;
                // (behind s_full: the scales of every tile before this one are told, so the slot is in
                // this use or the one before, as a wait by parity needs)
                if (!(ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&bars->sc_full[g % SCST]), (uint32_t)((g / SCST) & 1), pc)))) break;
                tc_fence_after();
                const float4* sc = bars->sc[g % SCST];
                uint32_t xr[128];
#pragma unroll
                for (int c4 = 0; c4 < 4; ++c4) tmem_ld32(tS + lane_addr + c4 * 32, *reinterpret_cast<uint32_t(*)[32]>(&xr[c4 * 32]));
                tmem_ld_wait();
                const int lim = n_vis - i * PF_BN;  // columns < lim are visible
                if (__any_sync(0xffffffffu, lim < PF_BN)) {
#pragma unroll
                    for (int c = 0; c < 128; ++c) xr[c] = c < lim ? xr[c] : 0xff800000u;  // -inf
                }
                // Row max of w = z + log2(vs): per page on the raw scores (its factor is positive).
                float mt = -INFINITY;
#pragma unroll
                for (int p = 0; p < PF_PAGES_PER_TILE; ++p) {
                    float x0 = -INFINITY, x1 = -INFINITY;
#pragma unroll
                    for (int c = 0; c < 16; c += 2) {
                        x0 = fmaxf(x0, __uint_as_float(xr[16 * p + c]));
                        x1 = fmaxf(x1, __uint_as_float(xr[16 * p + c + 1]));
                    }
                    const float4 f = sc[p];
                    mt = fmaxf(mt, fmaf(fmaxf(x0, x1), score_factor(f.x, scr), f.y));
                }
                float alpha = 1.0f;
                bool resc = false;
                if (mt - m > RESCALE_SLACK) {  // (m + 8 may round up to mt)
                    alpha = ex2(m - mt);  // 0 when m = -inf
                    m = mt;
                    resc = true;
                }
                // p' = 2^(w - m + 7), packed as FP16 pairs into xr[0..63]; the sum divides vs out
                const float base = (m == -INFINITY) ? 0.0f : m;
                const bool far = fabsf(base) >= FAR_MAX;
                float rs = 0.0f;
                if (__builtin_expect(!__any_sync(0xffffffffu, far), 1)) {
#pragma unroll
                    for (int p = 0; p < PF_PAGES_PER_TILE; ++p) {
                        const float4 f = sc[p];
                        const float mul = score_factor(f.x, scr), add = f.y + (P_BIAS - base);
                        const float2 mul2 = make_float2(mul, mul), add2 = make_float2(add, add);
                        float2 acc2 = make_float2(0.0f, 0.0f);
#pragma unroll
                        for (int c = 16 * p; c < 16 * p + 16; c += 2) {
                            const float2 t = ffma2(make_float2(__uint_as_float(xr[c]), __uint_as_float(xr[c + 1])), mul2, add2);
                            const float2 e = make_float2(ex2(t.x), ex2(t.y));
                            acc2 = fadd2(acc2, e);
                            xr[c >> 1] = pack_f16x2(e.x, e.y);
                        }
                        rs = fmaf(acc2.x + acc2.y, f.z, rs);
                    }
                } else {
                    // the same with the maximum subtracted apart, in the rows that are far: a row's bits are its
                    // own, whatever the rows beside it are
#pragma unroll
                    for (int p = 0; p < PF_PAGES_PER_TILE; ++p) {
                        const float4 f = sc[p];
                        const float mul = score_factor(f.x, scr), add = far ? f.y : f.y + (P_BIAS - base);
                        const float less = far ? base : 0.0f, more = far ? P_BIAS : 0.0f;
                        float2 acc2 = make_float2(0.0f, 0.0f);
#pragma unroll
                        for (int c = 16 * p; c < 16 * p + 16; c += 2) {
                            const float2 e = make_float2(ex2(fmaf(__uint_as_float(xr[c]), mul, add) - less + more),
                                                         ex2(fmaf(__uint_as_float(xr[c + 1]), mul, add) - less + more));
                            acc2 = fadd2(acc2, e);
                            xr[c >> 1] = pack_f16x2(e.x, e.y);
                        }
                        rs = fmaf(acc2.x + acc2.y, f.z, rs);
                    }
                }
                l = fmaf(l, alpha, rs);
                // S_j(i) complete implies PV_j(i-1) complete (MMAs of one issuer retire in order), so O_j is
                // stable and S_j's columns may take P_j(i).
                if (i > 0 && __any_sync(0xffffffffu, resc)) {
#pragma unroll 1
                    for (int c4 = 0; c4 < 4; ++c4) {
                        uint32_t rr[32];
                        tmem_ld32(tO + lane_addr + c4 * 32, rr);
                        tmem_ld_wait();
#pragma unroll
                        for (int q = 0; q < 32; ++q) rr[q] = __float_as_uint(__uint_as_float(rr[q]) * alpha);
                        tmem_st32(tO + lane_addr + c4 * 32, rr);
                    }
                }
                tmem_st32(tS + lane_addr, *reinterpret_cast<uint32_t(*)[32]>(&xr[0]));
                tmem_st32(tS + lane_addr + 32, *reinterpret_cast<uint32_t(*)[32]>(&xr[32]));
                tmem_st_wait();
                tc_fence_before();
                mbar_arrive(smem_u32(&bars->p_ready[j]));
            }
            // ---- epilogue ----
            if (ok && nt > 0) ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&bars->o_done[j]), (ph >> 1) & 1u, pc));
            int unit_bad = 0;
            if (ok) {  // the verdict on the unit's V codes and scales
                const int slot = (ph >> 2) & 1;
                ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&bars->r_full[slot]), (ph >> 3) & 1u, pc));
                if (ok) {
                    const uint4* f = reinterpret_cast<const uint4*>(bars->r_flag[slot]);
                    uint32_t any = 0;
#pragma unroll
                    for (int q = 0; q < 8; ++q) any |= f[q].x | f[q].y | f[q].z | f[q].w;
                    unit_bad = (any & 0x01010101u || bars->r_wide[slot] ? RK_STATUS_RANGE : 0) | (any & 0x02020202u ? RK_STATUS_SCALE : 0);
                    mbar_arrive(smem_u32(&bars->r_empty[slot]));
                }
            }
            if (!ok) {
                fail_from(kk);
                break;
            }
            // a query that sees a key fails if its unit does or its sum is beyond FP32 (which a NaN
            // code in K, a query out of range or an overflowing score make it)
            const bool seen = n_vis > 0;
            const int fail = !valid || !seen ? 0 : unit_bad ? unit_bad : (l > 0.0f && l < INFINITY) ? 0 : RK_STATUS_RANGE;
            if (nt > 0) {
                tc_fence_after();
                const float inv_l = fail || !seen ? 0.0f : 1.0f / l;
                // A thread has a row, so its 16-byte stores would meet 32 lines a warp; four lanes swap their
                // four chunks of 32 columns first and write 64 bytes of a row at a time.
                const int l4 = lane & 3;
                size_t rows[4];
                bool in[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int re = (r & ~3) + e;
                    in[e] = s0 + (re & (rph - 1)) < a.Sq;
                    rows[e] = in[e] ? query_row(a, un->b, un->kvh, rsh, s0, re) : 0;
                }
#pragma unroll 1
                for (int c4 = 0; c4 < 4; ++c4) {
                    uint32_t rr[32];
                    tmem_ld32(tO + lane_addr + c4 * 32, rr);
                    tmem_ld_wait();
                    uint32_t w[4][4];  // [chunk][word], after the swap [row of the four][word]
#pragma unroll
                    for (int q = 0; q < 4; ++q)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            w[q][e] = fail || !seen ? 0u
                                                    : pack_bf16x2(__uint_as_float(rr[8 * q + 2 * e]) * inv_l,
                                                                  __uint_as_float(rr[8 * q + 2 * e + 1]) * inv_l);
                    transpose4(w, l4);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (in[e])
                            *reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(a.out) + rows[e] * HEAD_DIM + c4 * 32 + l4 * 8) =
                                make_uint4(w[e][0], w[e][1], w[e][2], w[e][3]);
                }
                // O_j has been read: the next unit's first PV may overwrite it
                tc_fence_before();
                mbar_arrive(smem_u32(&bars->o_free[j]));
                if (valid) a.lse[row] = fail ? nanv : seen ? (m - P_BIAS + log2f(l)) * 0.693147180559945309f : -INFINITY;
            } else if (valid) {
                write_row(a, row, fail ? nanv : -INFINITY);
            }
            const unsigned any_fail = __reduce_or_sync(0xffffffffu, (unsigned)fail);
            if (any_fail && lane == 0 && a.status) atomicOr(a.status, (int)any_fail);
            mbar_arrive(smem_u32(&bars->u_empty[uslot]));
            g0 += n_tiles;
            ph ^= (uint32_t)(nt & 1) | (nt > 0 ? 2u : 0u);
            ph = (ph & 3u) | ((((ph >> 2) + 1u) & 3u) << 2);
        }
        named_bar_sync(2, PQ_THREADS);
    }

    // ---- teardown: every role has passed barrier 2; no MMA or TMEM access is in flight ----
    if (warp == WARP_MMA) {
        tc_fence_after();
        tmem_dealloc(tmem, TMEM_COLS);
    }
}

}  // namespace

cudaError_t launch_prefill_q8(const AttnQ8Args& a, cudaStream_t stream) {
    static std::atomic<uint64_t> configured{0};
    static std::atomic<int> sm_count[64];
    int dev = 0, nsm = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? (1ull << dev) : 0;
    if (!bit || !(configured.load() & bit)) {
        e = cudaFuncSetAttribute(prefill_q8_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, PQ_SMEM_BYTES);
        if (e == cudaSuccess) e = cudaDeviceGetAttribute(&nsm, cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess) return e;
        if (bit) sm_count[dev].store(nsm);
        configured.fetch_or(bit);
    } else {
        nsm = sm_count[dev].load();
    }
    const int rph = PF_BM / a.G, n_qtiles = (a.Sq + rph - 1) / rph;
    const long long units = (long long)a.B * a.Hkv * ((n_qtiles + 1) / 2);
    if (units <= 0) return cudaSuccess;
    prefill_q8_kernel<<<(unsigned)(units < nsm ? units : nsm), PQ_THREADS, PQ_SMEM_BYTES, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace rk
