// append_q8.cu -- quantise new tokens' K and V into the 8-bit page cache.
//
// A block of the cache is the 16 tokens of a page and one KV head: 2 KiB of
// e4m3 codes and one scale 2^E, value = code * 2^E.
//   E of a token = floor(log2 max_d |x_d|) - 7 of its bf16 inputs, at least
//   -64; E of a block = the largest of its tokens so far.
//   y = x (V), or x rotated at the token's position (K; rotate-half RoPE of
//   "WS2 PR7 Fused Attention Backend Alignment", "FlashInfer RoPE Fusion", done
//   once here rather than at each read).  |y| <= sqrt(2) |x| < 2^8.5 2^E, so a
//   code is at most 362 of 448.
//   code = y 2^-E rounded to 4 significant bits (half to even), 0 where that is
//   below 2^-6 (e4m3's smallest normal number).
// No code is subnormal, so growth of E only lowers the exponents of the block's
// old codes (those that fall below 2^-6 become 0): the result is the same
// whether the tokens come in one call or in many, and bit for bit a function
// of the block's tokens.  Leaving subnormals out costs at most 2^-7 2^E, below
// 2^-14 of the block's largest value; the 4-bit rounding of that value is 2^-5.
// E comes from the inputs' exponent bits, never from a rounded product.
// The rotation is in FP32; a pair with a result that FP32 cannot place on one
// side of a rounding border is done again with 44 bits, so that codes are those of
// the rotation by the plan's rates (a few in a million would be one step off otherwise).
// The rates are doubles, so that at position 131071 an angle is the real number's to
// some 2^-35: one code in 2^30 may still be the neighbour of the real number's.
//
// Work: a run is the tokens of one call on one page (slots that follow one another).  The
// runs that start in a window of tokens belong to one warp (window 4) or to the four warps of a
// CTA (window 16), for one KV head: lane t of each warp has slot, position and exponent of the
// window's t-th token (a run goes on for 15 past the window at most), the values go by 8 lanes
// to a token, four tokens to a warp's turn, once for the exponents and once more (mostly still
// in registers, else out of L1) for the codes.
// 64 single tokens x 8 heads: 4.8 us a launch (latency, and a longer chain of it than a copy has: slots,
// runs, values, exponents by shuffles, scales, codes; the BF16 append of as many tokens takes 1.9); 2048
// tokens in runs of 16: 6.8 us; 12700 tokens of 24 ragged rows: 29 us (bound by instructions, a quarter of
// them for the borders: the bytes alone would take 12).
#include "q8_device.cuh"

namespace rk {

namespace {

constexpr int AQ_THREADS = 128, AQ_WARPS = AQ_THREADS / 32;
// Four warps to a window once there is a CTA of them per SM: the warps of a long run then work
// side by side (2048 tokens of 8 heads: 6.8 us, 15.9 with a warp to each run); below, a warp
// alone needs no barrier and spreads single tokens wider (64 tokens: 4.7 us, 5.2 in fours).
constexpr long long AQ_MANY = 152;

__device__ __forceinline__ float flush_code(float v) { return fabsf(v) < 31.0f / 2048.0f ? 0.0f : v; }

// Lower the exponent of four codes by `by` > 0; below the smallest normal: 0.
__device__ __forceinline__ uint32_t lower4(uint32_t w, int by) {
    uint32_t r = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t c = (w >> (8 * i)) & 0xffu;
        const int e = (int)((c >> 3) & 15u) - by;
        const uint32_t x = (c & 0x7fu) == 0x7fu ? c : (e >= 1 ? (c & 0x87u) | ((uint32_t)e << 3) : 0u);
        r |= x << (8 * i);
    }
    return r;
}

// Largest |x| of the token as a bf16 bit pattern (the 8 lanes of a group agree).
__device__ __forceinline__ uint32_t token_amax(const uint4& lo, const uint4& hi) {
    const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = __vmaxu2(m, w[i] & 0x7fff7fffu);
    m = max(m & 0xffffu, m >> 16);
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    return m;
}

// What FP32 may be off by in a rotated value, relative to |lo| + |hi|.  The angle: rounded as
// an integer and as a product, 2 2^-24 of itself and 2^-25 for the constant, 4.7e-7 at pi, and
// 2 pi 2^-32.  __sincosf on [-pi, pi]: 2^-21.19 by CUDA's documentation, 4.2e-7.  The product, the
// fused sum and the border's own distance: 3 2^-24, 1.8e-7.
constexpr float ROT_ERR = 1.1e-6f;

// A value as the unevaluated sum of two floats, about 47 bits; sums and products after
// Dekker ("A floating-point technique for extending the available precision", 1971).
struct Two {
    float h, l;
};
// x z + c for |c| >= |x z|
__device__ __forceinline__ Two two_fma(Two x, Two z, float ch, float cl) {
    const float m = __fmul_rn(x.h, z.h);
    const float e = __fmaf_rn(x.h, z.h, -m) + fmaf(x.h, z.l, x.l * z.h);
    const float h = __fadd_rn(ch, m);
    return {h, __fsub_rn(m, __fsub_rn(h, ch)) + (e + cl)};
}
// a x + b y for floats a, b, as one float that rounds to fewer bits as the sum does: the
// neighbour with its last bit set, on the side that the rest points to.
__device__ __forceinline__ float two_dot(float a, Two x, float b, Two y) {
    const float p = __fmul_rn(a, x.h), q = __fmul_rn(b, y.h);
    const float e = (__fmaf_rn(a, x.h, -p) + a * x.l) + (__fmaf_rn(b, y.h, -q) + b * y.l);
    const float s = __fadd_rn(p, q), t = __fsub_rn(s, p);
    const float r = __fadd_rn(__fadd_rn(__fsub_rn(p, __fsub_rn(s, t)), __fsub_rn(q, t)), e);
    const float h = __fadd_rn(s, r), l = __fsub_rn(r, __fsub_rn(h, s));
    const int bits = __float_as_int(h);
    return l != 0.0f && !(bits & 1) ? __int_as_float(bits + ((l > 0.0f) == (h > 0.0f) ? 1 : -1)) : h;
}
// Taylor coefficients of sin and cos of pi / 4 t, |t| <= 1, in powers of t^2; the next is below 2^-49.
struct TurnSeries {
    float sin2[5][2], cos2[5][2], sin1[3], cos1[3];
};
__constant__ TurnSeries turn_series = {
    {{7.853981853e-01f, -2.185569414e-08f}, {-8.074551076e-02f, -1.431311292e-09f}, {2.490394516e-03f, 5.427601424e-11f}, {-3.657620255e-05f, -1.635465201e-12f}, {3.133616815e-07f, 7.545715084e-15f}},
    {{1.000000000e+00f, 0.000000000e+00f}, {-3.084251285e-01f, -9.074112128e-09f}, {1.585434377e-02f, 4.718809787e-10f}, {-3.259918885e-04f, 1.603162373e-12f}, {3.590860388e-06f, 6.088822480e-14f}},
    {-1.757247681e-09f, 6.948453098e-12f, -2.041026345e-14f},
    {-2.461136894e-08f, 1.150115905e-10f, -3.898073270e-13f}};

// The rotation of one pair, to about 2^-44 of its length (in FP64 the same took 3 us; that
// pipe is slow here): a quarter turn's share of the angle by the two series, the rest by swaps.
__device__ __noinline__ float2 rotate_exact(float lo, float hi, uint32_t pos, uint64_t turns) {
    const uint64_t frac = pos * turns;
    const uint32_t quarter = (uint32_t)((frac + (1ull << 61)) >> 62);
    const long long r = (long long)(frac - ((uint64_t)quarter << 62));  // of [-2^61, 2^61)
    Two t;
    t.h = (float)r;
    t.l = (float)(r - (long long)t.h) * 0x1p-61f;
    t.h *= 0x1p-61f;
    Two z;
    z.h = __fmul_rn(t.h, t.h);
    z.l = fmaf(2.0f * t.h, t.l, __fmaf_rn(t.h, t.h, -z.h));
    const TurnSeries& c = turn_series;
    Two sn = {fmaf(fmaf(c.sin1[2], z.h, c.sin1[1]), z.h, c.sin1[0]), 0.0f};
    Two cn = {fmaf(fmaf(c.cos1[2], z.h, c.cos1[1]), z.h, c.cos1[0]), 0.0f};
#pragma unroll
    for (int k = 4; k >= 0; --k) {
        sn = two_fma(sn, z, c.sin2[k][0], c.sin2[k][1]);
        cn = two_fma(cn, z, c.cos2[k][0], c.cos2[k][1]);
    }
    const float m = __fmul_rn(sn.h, t.h);
    sn = {m, __fmaf_rn(sn.h, t.h, -m) + fmaf(sn.h, t.l, sn.l * t.h)};
    if (quarter & 1) {  // a quarter turn on: (cos, sin) -> (-sin, cos)
        const Two x = sn;
        sn = cn;
        cn = {-x.h, -x.l};
    }
    if (quarter & 2) {
        lo = -lo;
        hi = -hi;
    }
    return make_float2(two_dot(lo, cn, -hi, sn), two_dot(hi, cn, lo, sn));
}

// Whether two values y may have other codes than what is known of them says: they lie from y0 to y1.
__device__ __forceinline__ bool near_border(float2 y0, float2 y1) {
    return cvt_e4m3x2(flush_code(y0.x), flush_code(y0.y)) != cvt_e4m3x2(flush_code(y1.x), flush_code(y1.y));
}
// The cheap half of it: whether a border of 4 bits (the upper 12 of the word, half up) lies
// between them, at any size.
__device__ __forceinline__ bool maybe_border(float2 y0, float2 y1) {
    const uint32_t h = 0x80000u;
    return (((__float_as_uint(y0.x) + h) ^ (__float_as_uint(y1.x) + h)) | ((__float_as_uint(y0.y) + h) ^ (__float_as_uint(y1.y) + h))) &
           0xfff00000u;
}

__device__ __forceinline__ uint2 pack8(const float (&y)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = cvt_e4m3x2(flush_code(y[2 * i]), flush_code(y[2 * i + 1]));
    return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}

// The codes of one token's 16 dims lo / hi (8 each, dims 8u .. and 64 + 8u ..).
__device__ __forceinline__ void store_codes(uint8_t* row, int u, uint2 lo, uint2 hi) {
    *reinterpret_cast<uint2*>(row + 8 * u) = lo;
    *reinterpret_cast<uint2*>(row + 64 + 8 * u) = hi;
}
__device__ __forceinline__ void unpack8(const uint4& w, float (&x)[8]) {
    const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = (i & 1) ? bf16hi(v[i >> 1]) : bf16lo(v[i >> 1]);
}

// Move the codes of slots [0, n) of a block to a scale 2^by larger (a warp's work).
__device__ __forceinline__ void lower_block(uint8_t* block, int n, int lane, int by) {
#pragma unroll 1
    for (int i = lane; i < n * (HEAD_DIM / 16); i += 32) {
        uint4* c = reinterpret_cast<uint4*>(block) + i;
        const uint4 x = *c;
        *c = make_uint4(lower4(x.x, by), lower4(x.y, by), lower4(x.z, by), lower4(x.w, by));
    }
}

// TEAM: the CTA's warps share one window of 16 tokens, turn by turn; else each has its own of 4.
template <bool TEAM>
__global__ void __launch_bounds__(AQ_THREADS) append_q8_kernel(const __grid_constant__ AppendQ8Args a) {
    const int lane = threadIdx.x & 31, g = lane >> 3, u = lane & 7;
    constexpr int STEP = TEAM ? AQ_WARPS : 1, WINDOW = 4 * STEP;
    const int wid = TEAM ? threadIdx.x >> 5 : 0;
    const long long work = TEAM ? blockIdx.x : (long long)blockIdx.x * AQ_WARPS + (threadIdx.x >> 5);
    const int h = (int)(work % a.Hkv);
    const long long w0 = work / a.Hkv * WINDOW;  // first token of the window
    if (w0 >= a.n) return;

    __shared__ uint32_t s_raw[TEAM ? 32 : 1];
    struct Token {
        uint4 kl, kh, vl, vh;
    };
    auto load = [&](long long i, Token& x) {
        const size_t at = ((size_t)i * a.Hkv + h) * HEAD_DIM + 8 * u;
        const uint4* ks = reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(a.k_new) + at);
        const uint4* vs = reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(a.v_new) + at);
        x.kl = __ldg(ks);
        x.kh = __ldg(ks + 8);
        x.vl = __ldg(vs);
        x.vh = __ldg(vs + 8);
    };
    // The window's first tokens travel while the slots do (in a decode step they are the work).
    Token x;
    x.kl = x.kh = x.vl = x.vh = make_uint4(0, 0, 0, 0);
    if (w0 + 4 * wid + g < a.n) load(w0 + 4 * wid + g, x);

    // ---- lane = token: slots, positions, where runs start and end ----
    const long long i = w0 + lane;
    int slot = -1, pos = -1, prev = -1, bad = 0;
    const int slots = a.num_pages * PAGE;
    if (i < a.n) {
        slot = a.slot_map[i];
        pos = a.position_ids[i];
        if (lane == 0 && w0 > 0) {
            prev = a.slot_map[i - 1];
            if (prev < -1 || prev >= slots || a.position_ids[i - 1] < 0) prev = -1;
        }
        if (slot < -1 || slot >= slots) bad = RK_STATUS_PAGE_OOB;
        else if (slot >= 0 && pos < 0) bad = RK_STATUS_POSITION;
        if (bad) slot = -1;
    }
    if (bad && lane < WINDOW && h == 0 && wid == 0 && a.status) atomicOr(a.status, bad);
    // the token before, as the run rule sees it: a refused one starts no run and carries none on
    const int up = __shfl_up_sync(0xffffffffu, slot, 1);
    if (lane > 0) prev = up;
    const uint32_t live = __ballot_sync(0xffffffffu, slot >= 0);
    const uint32_t lead = __ballot_sync(0xffffffffu, slot >= 0 && !(prev >= 0 && slot == prev + 1 && slot % PAGE != 0));
    const uint32_t ours = lead & ((1u << WINDOW) - 1u);
    if (ours == 0) return;  // no run starts here
    const uint32_t after = ~((2u << lane) - 1u);  // the lanes behind this one
    const int first = __ffs(ours) - 1, last = 31 - __clz(ours);
    const int start = (lead & ~after) ? 31 - __clz(lead & ~after) : 0;  // of this lane's run
    const uint32_t next = (lead | ~live) & after;
    const int close = next ? __ffs(next) - 2 : 31;  // its last token
    const int end = __shfl_sync(0xffffffffu, close, last) + 1;
    const int turns = (end - first + 3) >> 2;

    // ---- the block's scales, where it had tokens before this call ----
    const bool head = (ours >> lane) & 1u;
    const int off = slot % PAGE;
    const size_t block = (size_t)(max(slot, 0) / PAGE) * a.Hkv + h;
    int sk = 0, sv = 0;
    if (head && off > 0) {
        sk = __float_as_int(a.k_scale[block]);
        sv = __float_as_int(a.v_scale[block]);
    }
    // ---- exponents: K in bits 0-7, V in bits 16-23 (plus 128); bits 8 and 24: out of range ----
    uint32_t raw = 0;
#pragma unroll 1
    for (int r = wid; r < turns; r += STEP) {
        const int t = first + 4 * r + g;
        if (r > wid || first > 0) {
            if (t < end && ((live >> t) & 1u)) load(w0 + t, x);
        }
        const uint32_t mk = token_amax(x.kl, x.kh), mv = token_amax(x.vl, x.vh);
        const uint32_t e = (mk >= Q8_LIMIT_BF16 ? 0x100u + (uint32_t)(128 + Q8_E_MIN) : (uint32_t)(q8_exponent(mk) + 128)) |
                           (mv >= Q8_LIMIT_BF16 ? 0x100u + (uint32_t)(128 + Q8_E_MIN) : (uint32_t)(q8_exponent(mv) + 128)) << 16;
        const uint32_t v = __shfl_sync(0xffffffffu, e, ((lane - first) & 3) * 8);
        if (lane - first >= 4 * r && lane - first < 4 * r + 4) raw = v;
    }
    if constexpr (TEAM) {  // each token's exponents from the warp that has them
        if (lane >= first && lane < end && ((lane - first) >> 2) % AQ_WARPS == wid) s_raw[lane] = raw;
        __syncthreads();
        raw = s_raw[lane];
    }
    // largest of the run: up to its last token, and back from there
    uint32_t m = raw & 0x00ff00ffu;
#pragma unroll
    for (int o = 1; o < PAGE; o <<= 1) {
        const uint32_t v = __shfl_up_sync(0xffffffffu, m, o);
        if (lane - o >= start) m = __vmaxu2(m, v);
    }
    m = __shfl_sync(0xffffffffu, m, close);
    int ek = (int)(m & 0xff) - 128, ev = (int)(m >> 16) - 128;
    bool ok = true;
    int up_k = 0, up_v = 0;
    if (head) {
        if (off > 0) {
            const int ek_old = (sk >> 23) - 127, ev_old = (sv >> 23) - 127;
            // not a power of two that this kernel writes: the block's codes cannot be moved to another scale
            ok = !((sk | sv) & 0x7fffff) && ek_old >= Q8_E_MIN && ek_old <= Q8_E_MAX && ev_old >= Q8_E_MIN && ev_old <= Q8_E_MAX;
            up_k = max(0, ek - ek_old);
            up_v = max(0, ev - ev_old);
            ek = max(ek, ek_old);
            ev = max(ev, ev_old);
        }
        if (wid > 0) {
        } else if (ok) {
            a.k_scale[block] = pow2(ek);
            a.v_scale[block] = pow2(ev);
        } else if (a.status) {
            atomicOr(a.status, RK_STATUS_SCALE);
        }
    }
    // earlier codes of the block move along
    uint32_t grown = __ballot_sync(0xffffffffu, head && ok && (up_k | up_v));
    while (wid == 0 && grown) {
        const int src = __ffs(grown) - 1;
        grown &= grown - 1;
        const int n = __shfl_sync(0xffffffffu, off, src);
        const int bk = __shfl_sync(0xffffffffu, up_k, src), bv = __shfl_sync(0xffffffffu, up_v, src);
        const size_t at = ((size_t)(__shfl_sync(0xffffffffu, slot, src) / PAGE) * a.Hkv + h) * Q8_BLOCK_BYTES;
        if (bk) lower_block(a.k_cache + at, n, lane, bk);
        if (bv) lower_block(a.v_cache + at, n, lane, bv);
    }
    // the run's exponents to each of its tokens, with the token's own two bits
    m = (uint32_t)(ek + 128) | (uint32_t)(ev + 128) << 16 | (ok ? 0u : 1u << 31);
    m = __shfl_sync(0xffffffffu, m, start);
    m |= raw & 0x01000100u;
    if (slot >= 0 && lane >= first && lane < end && !(m >> 31) && (m & 0x01000100u) && wid == 0 && a.status) atomicOr(a.status, RK_STATUS_RANGE);

    // ---- codes; the last turn's values are still here ----
    const int top = wid + (turns - 1 - wid) / STEP * STEP;
#pragma unroll 1
    for (int r = top; r >= wid && turns > wid; r -= STEP) {
        const int t = first + 4 * r + g;
        const uint32_t e = __shfl_sync(0xffffffffu, m, t & 31);
        const int at = __shfl_sync(0xffffffffu, slot, t & 31);
        const uint32_t p = (uint32_t)__shfl_sync(0xffffffffu, pos, t & 31);
        if (t >= end || at < 0 || (e >> 31)) continue;
        if (r < top) load(w0 + t, x);
        const size_t row = ((size_t)(at / PAGE) * a.Hkv + h) * Q8_BLOCK_BYTES + (at % PAGE) * HEAD_DIM;
        const uint2 nan8 = make_uint2(0x7f7f7f7fu, 0x7f7f7f7fu);
        {
            float lo[8], hi[8], yl[8], yh[8];
            unpack8(x.kl, lo);
            unpack8(x.kh, hi);
            const float inv = pow2(128 - (int)(e & 0xff));
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float c, s;
                rope_cos_sin(p, a.rope_turns[8 * u + i], c, s);
                float2 y = fmul2(make_float2(lo[i], hi[i]), make_float2(c, c));
                y = fmul2(ffma2(make_float2(-hi[i], lo[i]), make_float2(s, s), y), make_float2(inv, inv));
                const float d = (fabsf(lo[i]) + fabsf(hi[i])) * (ROT_ERR * inv);
                const float2 y0 = fadd2(y, make_float2(-d, -d)), y1 = fadd2(y, make_float2(d, d));
                if (maybe_border(y0, y1) && near_border(y0, y1)) {
                    y = rotate_exact(lo[i], hi[i], p, a.rope_turns[8 * u + i]);
                    y = fmul2(y, make_float2(inv, inv));
                }
                yl[i] = y.x;
                yh[i] = y.y;
            }
            const bool good = !(e & 0x100u);
            store_codes(a.k_cache + row, u, good ? pack8(yl) : nan8, good ? pack8(yh) : nan8);
        }
        {
            float lo[8], hi[8];
            unpack8(x.vl, lo);
            unpack8(x.vh, hi);
            const float inv = pow2(128 - (int)((e >> 16) & 0xff));
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                lo[i] *= inv;
                hi[i] *= inv;
            }
            const bool good = !(e & 0x1000000u);
            store_codes(a.v_cache + row, u, good ? pack8(lo) : nan8, good ? pack8(hi) : nan8);
        }
    }
}

}  // namespace

cudaError_t launch_append_q8(const AppendQ8Args& a, cudaStream_t stream) {
    if (a.n <= 0) return cudaSuccess;
    const long long teams = ((long long)a.n + 4 * AQ_WARPS - 1) / (4 * AQ_WARPS) * a.Hkv;
    const bool team = teams >= AQ_MANY;
    const long long blocks = team ? teams : (((long long)a.n + 3) / 4 * a.Hkv + AQ_WARPS - 1) / AQ_WARPS;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    if (team) append_q8_kernel<true><<<(unsigned)blocks, AQ_THREADS, 0, stream>>>(a);
    else append_q8_kernel<false><<<(unsigned)blocks, AQ_THREADS, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace rk
