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
// side of a rounding border is done again in FP64, so that codes are those of
// the real number (a few in a million would be one step off otherwise).
//
// Work: a run is the tokens of one call on one page (slots that follow one
// another).  A CTA takes one KV head of the runs that start in a window of 16
// tokens: 8 threads to a token, each with 8 rotation pairs (dims 8u .. 8u+7 and
// 64 + 8u ..), so a thread's loads are 16 bytes and 8 lanes cover 128.  A run
// may go on for 15 tokens past the window, in a second pass.  Bound by latency at
// decode sizes, by bytes (512 in, 256 out a token and head) at chunk sizes.
#include "q8_device.cuh"

namespace rk {

namespace {

constexpr int AQ_THREADS = 128;
constexpr int AQ_WINDOW = 16;

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

// What a token's 8 threads hold of one tensor: dims 8u .. 8u+7 and 64+8u ..
struct Half8 {
    uint4 lo, hi;
};

// Largest |x| of the token as a bf16 bit pattern (the 8 lanes of a group agree).
__device__ __forceinline__ uint32_t token_amax(const Half8& x) {
    const uint32_t w[8] = {x.lo.x, x.lo.y, x.lo.z, x.lo.w, x.hi.x, x.hi.y, x.hi.z, x.hi.w};
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = __vmaxu2(m, w[i] & 0x7fff7fffu);
    m = max(m & 0xffffu, m >> 16);
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    return m;
}

// What FP32 may be off by in a rotated value, relative to |lo| + |hi|: the angle
// of rope_cos_sin is off by at most 2 pi 2^-32 and 2^-24 of itself (2^-22.3 at
// pi), its sine and cosine by 2^-21.2, the two products and the sum by 2^-23.
constexpr float ROT_ERR = 1.0f / (1 << 19);

// A double as a float that rounds to 4 bits as the double does: cut off, and the
// last bit set if something was lost.
__device__ __forceinline__ float to_odd(double x) {
    const float r = __double2float_rz(x);
    return (double)r != x ? __int_as_float(__float_as_int(r) | 1) : r;
}

// The rotation of one pair in FP64 (angle in turns from the 0.64 fixed-point rate).
__device__ __noinline__ float2 rotate_exact(float lo, float hi, uint32_t pos, uint64_t turns) {
    double sn, c;
    sincospi(ldexp((double)(long long)(pos * turns), -63), &sn, &c);
    return make_float2(to_odd((double)lo * c - (double)hi * sn), to_odd((double)hi * c + (double)lo * sn));
}

// Whether codes of v 2^-E and of a value up to d away may differ.
__device__ __forceinline__ bool near_border(float v0, float v1, float d) {
    return cvt_e4m3x2(flush_code(v0 - d), flush_code(v1 - d)) != cvt_e4m3x2(flush_code(v0 + d), flush_code(v1 + d));
}

__device__ __forceinline__ uint2 pack8(const float (&y)[8], float inv) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = cvt_e4m3x2(flush_code(y[2 * i] * inv), flush_code(y[2 * i + 1] * inv));
    return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}

__global__ void __launch_bounds__(AQ_THREADS) append_q8_kernel(const __grid_constant__ AppendQ8Args a) {
    __shared__ int s_slot[32], s_pos[32];
    __shared__ uint32_t s_lead, s_live;
    __shared__ int s_ek[32], s_ev[32];
    const int tid = threadIdx.x, g = tid >> 3, u = tid & 7;
    const int h = (int)(blockIdx.x % a.Hkv);
    const long long w0 = (long long)(blockIdx.x / a.Hkv) * AQ_WINDOW;  // first token of the window

    // ---- the window's slots and the 15 after it; which of them start a run ----
    if (tid < 32) {
        const long long i = w0 + tid;
        int slot = -1, pos = -1, bad = 0;
        if (i < a.n) {
            slot = a.slot_map[i];
            pos = a.position_ids[i];
            if (slot < -1 || slot >= a.num_pages * PAGE) bad |= RK_STATUS_PAGE_OOB;
            else if (slot >= 0 && pos < 0) bad |= RK_STATUS_POSITION;
            if (bad) slot = -1;
        }
        if (bad && tid < AQ_WINDOW && h == 0 && a.status) atomicOr(a.status, bad);
        // the token before: as the run rule sees it (a refused one starts no run and carries none on)
        int prev = __shfl_up_sync(0xffffffffu, slot, 1);
        if (tid == 0) {
            prev = -1;
            if (w0 > 0) {
                prev = a.slot_map[w0 - 1];
                if (prev < -1 || prev >= a.num_pages * PAGE || a.position_ids[w0 - 1] < 0) prev = -1;
            }
        }
        const bool live = slot >= 0;
        const bool lead = live && !(prev >= 0 && slot == prev + 1 && slot % PAGE != 0);
        s_slot[tid] = slot;
        s_pos[tid] = pos;
        const uint32_t ml = __ballot_sync(0xffffffffu, lead), mv = __ballot_sync(0xffffffffu, live);
        if (tid == 0) {
            s_lead = ml;
            s_live = mv;
        }
    }
    __syncthreads();
    const uint32_t lead = s_lead, live = s_live;
    if ((lead & 0xffffu) == 0) return;  // no run starts here
    // the last run that starts in the window may reach past it
    const int last = 31 - __clz(lead & 0xffffu);
    const uint32_t stop = (lead | ~live) & ~((2u << last) - 1u);  // first token after `last` that is not of its run
    const int end = stop ? __ffs(stop) - 1 : 32;                  // a run has at most 16 tokens: <= 31
    const bool two = end > AQ_WINDOW;

    Half8 k[2], v[2];
    int run[2];   // the run's first token, -1: not ours
    int ok_k = 1, ok_v = 1;  // per pass, bits
#pragma unroll
    for (int p = 0; p < 2; ++p) {
        const int t = g + AQ_WINDOW * p;
        run[p] = -1;
        const uint32_t before = lead & ((2u << t) - 1u) & 0xffffu;
        if ((p == 0 || two) && t < end && ((live >> t) & 1u) && before) run[p] = 31 - __clz(before);
        uint32_t mk = 0, mv = 0;
        k[p].lo = k[p].hi = v[p].lo = v[p].hi = make_uint4(0, 0, 0, 0);
        if (run[p] >= 0) {
            const size_t at = ((size_t)(w0 + t) * a.Hkv + h) * HEAD_DIM + 8 * u;
            const uint4* ks = reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(a.k_new) + at);
            const uint4* vs = reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(a.v_new) + at);
            k[p].lo = __ldcs(ks);
            k[p].hi = __ldcs(ks + 8);
            v[p].lo = __ldcs(vs);
            v[p].hi = __ldcs(vs + 8);
        }
        if (p == 0 || two) {
            mk = token_amax(k[p]);
            mv = token_amax(v[p]);
            const bool bk = mk >= Q8_LIMIT_BF16, bv = mv >= Q8_LIMIT_BF16;
            if (bk) ok_k &= ~(1 << p); else ok_k |= 1 << p;
            if (bv) ok_v &= ~(1 << p); else ok_v |= 1 << p;
            if (u == 0) {
                s_ek[t] = bk ? Q8_E_MIN : q8_exponent(mk);
                s_ev[t] = bv ? Q8_E_MIN : q8_exponent(mv);
                if ((bk || bv) && a.status) atomicOr(a.status, RK_STATUS_RANGE);
            }
        }
    }
    // the scales of pages that had tokens before this call, read before any is written
    float sk[2] = {1.0f, 1.0f}, sv[2] = {1.0f, 1.0f};
    int off[2];  // the run's first slot in its page
#pragma unroll
    for (int p = 0; p < 2; ++p) {
        off[p] = 0;
        if (run[p] < 0) continue;
        const int slot = s_slot[run[p]];
        off[p] = slot % PAGE;
        if (off[p] > 0) {
            const size_t at = (size_t)(slot / PAGE) * a.Hkv + h;
            sk[p] = a.k_scale[at];
            sv[p] = a.v_scale[at];
        }
    }
    __syncthreads();

#pragma unroll
    for (int p = 0; p < 2; ++p) {
        if (run[p] < 0) continue;
        const int t = g + AQ_WINDOW * p, first = run[p];
        const int page = s_slot[first] / PAGE;
        const size_t block = (size_t)page * a.Hkv + h;
        int ek = Q8_E_MIN, ev = Q8_E_MIN;
        for (int j = first; j < 32 && ((live >> j) & 1u) && (j == first || !((lead >> j) & 1u)); ++j) {
            ek = max(ek, s_ek[j]);
            ev = max(ev, s_ev[j]);
        }
        int ek_old = ek, ev_old = ev;
        if (off[p] > 0) {
            const int bk = __float_as_int(sk[p]), bv = __float_as_int(sv[p]);
            ek_old = (bk >> 23) - 127;
            ev_old = (bv >> 23) - 127;
            // not a power of two that this kernel writes: the block's codes cannot be moved to another scale
            if ((bk & 0x7fffff) || (bv & 0x7fffff) || ek_old < Q8_E_MIN || ek_old > Q8_E_MAX || ev_old < Q8_E_MIN ||
                ev_old > Q8_E_MAX) {
                if (u == 0 && a.status) atomicOr(a.status, RK_STATUS_SCALE);
                continue;
            }
            ek = max(ek, ek_old);
            ev = max(ev, ev_old);
        }
        uint8_t* kb = a.k_cache + block * Q8_BLOCK_BYTES;
        uint8_t* vb = a.v_cache + block * Q8_BLOCK_BYTES;
        if (t == first) {
            if (off[p] == 0 || ek > ek_old || ev > ev_old) {
                if (u == 0) {
                    a.k_scale[block] = pow2(ek);
                    a.v_scale[block] = pow2(ev);
                }
                for (int s = 0; s < off[p]; ++s) {  // old codes: lane u has 16 bytes of each slot
                    if (ek > ek_old) {
                        uint4* c = reinterpret_cast<uint4*>(kb + s * HEAD_DIM) + u;
                        uint4 x = *c;
                        x = make_uint4(lower4(x.x, ek - ek_old), lower4(x.y, ek - ek_old), lower4(x.z, ek - ek_old),
                                       lower4(x.w, ek - ek_old));
                        *c = x;
                    }
                    if (ev > ev_old) {
                        uint4* c = reinterpret_cast<uint4*>(vb + s * HEAD_DIM) + u;
                        uint4 x = *c;
                        x = make_uint4(lower4(x.x, ev - ev_old), lower4(x.y, ev - ev_old), lower4(x.z, ev - ev_old),
                                       lower4(x.w, ev - ev_old));
                        *c = x;
                    }
                }
            }
        }
        const int s = s_slot[t] % PAGE;
        const uint32_t pos = (uint32_t)s_pos[t];
        const uint2 nan8 = make_uint2(0x7f7f7f7fu, 0x7f7f7f7fu);
        {
            const uint32_t lw[4] = {k[p].lo.x, k[p].lo.y, k[p].lo.z, k[p].lo.w};
            const uint32_t hw[4] = {k[p].hi.x, k[p].hi.y, k[p].hi.z, k[p].hi.w};
            float yl[8], yh[8];
            const float inv = pow2(-ek);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float lo = (i & 1) ? bf16hi(lw[i >> 1]) : bf16lo(lw[i >> 1]);
                const float hi = (i & 1) ? bf16hi(hw[i >> 1]) : bf16lo(hw[i >> 1]);
                float c, sn;
                rope_cos_sin(pos, a.rope_turns[8 * u + i], c, sn);
                yl[i] = fmaf(-hi, sn, lo * c);
                yh[i] = fmaf(lo, sn, hi * c);
                const float d = (fabsf(lo) + fabsf(hi)) * ROT_ERR * inv;
                if (near_border(yl[i] * inv, yh[i] * inv, d)) {
                    const float2 y = rotate_exact(lo, hi, pos, a.rope_turns[8 * u + i]);
                    yl[i] = y.x;
                    yh[i] = y.y;
                }
            }
            const bool good = (ok_k >> p) & 1;
            *reinterpret_cast<uint2*>(kb + s * HEAD_DIM + 8 * u) = good ? pack8(yl, inv) : nan8;
            *reinterpret_cast<uint2*>(kb + s * HEAD_DIM + 64 + 8 * u) = good ? pack8(yh, inv) : nan8;
        }
        {
            const uint32_t lw[4] = {v[p].lo.x, v[p].lo.y, v[p].lo.z, v[p].lo.w};
            const uint32_t hw[4] = {v[p].hi.x, v[p].hi.y, v[p].hi.z, v[p].hi.w};
            float yl[8], yh[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                yl[i] = (i & 1) ? bf16hi(lw[i >> 1]) : bf16lo(lw[i >> 1]);
                yh[i] = (i & 1) ? bf16hi(hw[i >> 1]) : bf16lo(hw[i >> 1]);
            }
            const float inv = pow2(-ev);
            const bool good = (ok_v >> p) & 1;
            *reinterpret_cast<uint2*>(vb + s * HEAD_DIM + 8 * u) = good ? pack8(yl, inv) : nan8;
            *reinterpret_cast<uint2*>(vb + s * HEAD_DIM + 64 + 8 * u) = good ? pack8(yh, inv) : nan8;
        }
    }
}

}  // namespace

cudaError_t launch_append_q8(const AppendQ8Args& a, cudaStream_t stream) {
    if (a.n <= 0) return cudaSuccess;
    const long long blocks = (((long long)a.n + AQ_WINDOW - 1) / AQ_WINDOW) * a.Hkv;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    append_q8_kernel<<<(unsigned)blocks, AQ_THREADS, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace rk
