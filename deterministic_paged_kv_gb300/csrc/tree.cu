// tree.cu -- attention of a tree of drafted tokens behind each row's prefix.
//
// Mathematics: o_n = sum_t softmax_t(q_n . k_t / sqrt D) v_t over the prefix, n's ancestors and n
// itself; keys and queries rotated at their positions, a node's position being the prefix's length
// plus its depth.
#include "rk_device.cuh"
#include "tree_args.h"

namespace rk {

namespace {

constexpr int TR_THREADS = 128;
constexpr int TR_ROWS = 8;   // accumulator rows (query head, node) of a CTA
constexpr int TR_KEYS = 32;  // keys of a tile

__global__ void __launch_bounds__(TR_THREADS) tree_kernel(const __grid_constant__ TreeArgs a) {
    __shared__ float qs[TR_ROWS][HEAD_DIM], ks[TR_KEYS][HEAD_DIM + 1], vs[TR_KEYS][HEAD_DIM];
    __shared__ int par[TREE_MAX], depth[TREE_MAX];
    __shared__ unsigned long long sees[TREE_MAX];
    __shared__ int kbad[TR_KEYS], qbad[TR_ROWS];
    const int R = a.T * a.G, blocks = (R + TR_ROWS - 1) / TR_ROWS;
    const int blk = blockIdx.x % blocks, kvh = (blockIdx.x / blocks) % a.Hkv, b = blockIdx.x / blocks / a.Hkv;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int kv = a.kv_lens[b], prefix = kv - a.T;
    int bad = kv < 0 || kv > a.W * PAGE || (kv > 0 && kv < a.T) ? RK_STATUS_KVLEN : 0;
    if (tid < a.T) par[tid] = a.parents[(size_t)b * a.T + tid];
    __syncthreads();
    if (tid < a.T) {
        const int p = par[tid];
        if (p < TREE_UNUSED || p >= tid || (p >= 0 && par[p] == TREE_UNUSED)) bad |= RK_STATUS_TREE;
    }
    if (__syncthreads_or(bad & RK_STATUS_TREE)) bad |= RK_STATUS_TREE;
    else if (tid < a.T) {
        unsigned long long m = 0;
        int d = 0;
        for (int n = par[tid] == TREE_UNUSED ? -1 : tid; n >= 0; n = par[n]) {
            m |= 1ull << n;
            ++d;
        }
        sees[tid] = m;
        depth[tid] = max(d - 1, 0);
    }
    int oob = 0;
    if (!bad)
        for (int i = tid; i < (kv + PAGE - 1) / PAGE; i += TR_THREADS) {
            const int pg = a.block_table[(size_t)b * a.W + i];
            oob |= pg < 0 || pg >= a.num_pages;
        }
    if (__syncthreads_or(oob)) bad |= RK_STATUS_PAGE_OOB;
    const bool none = !bad && kv == 0;
    if (bad && tid == 0 && a.status) atomicOr(a.status, bad);
    auto at = [&](int r) { return ((size_t)b * a.Hq + kvh * a.G + r / a.T) * a.T + r % a.T; };
    if (bad || none) {
        for (int i = tid; i < TR_ROWS * HEAD_DIM; i += TR_THREADS) {
            const int r = blk * TR_ROWS + i / HEAD_DIM;
            if (r < R) reinterpret_cast<__nv_bfloat16*>(a.out)[at(r) * HEAD_DIM + i % HEAD_DIM] = __float2bfloat16_rn(0.0f);
            if (r < R && i % HEAD_DIM == 0) a.lse[at(r)] = bad ? NAN : -INFINITY;
        }
        return;
    }
    if (tid < TR_ROWS) qbad[tid] = 0;
    __syncthreads();
    for (int i = tid; i < TR_ROWS * ROPE_PAIRS; i += TR_THREADS) {
        const int r = blk * TR_ROWS + i / ROPE_PAIRS, e = i % ROPE_PAIRS;
        float x = 0.0f, y = 0.0f;
        if (r < R) {
            const __nv_bfloat16* q = reinterpret_cast<const __nv_bfloat16*>(a.q) + at(r) * HEAD_DIM;
            const float lo = __bfloat162float(q[e]), hi = __bfloat162float(q[e + ROPE_PAIRS]);
            if (!(fabsf(lo) < 32768.0f && fabsf(hi) < 32768.0f)) qbad[i / ROPE_PAIRS] = 1;
            float c, s;
            rope_cos_sin((uint32_t)(prefix + depth[r % a.T]), a.rope_turns[e], c, s);
            x = lo * c - hi * s;
            y = hi * c + lo * s;
        }
        qs[i / ROPE_PAIRS][e] = x;
        qs[i / ROPE_PAIRS][e + ROPE_PAIRS] = y;
    }
    constexpr int PER = TR_ROWS / 4;
    float m[PER], l[PER], o[PER][4];
    bool fail[PER];
    for (int i = 0; i < PER; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.0f;
        fail[i] = false;
        for (int e = 0; e < 4; ++e) o[i][e] = 0.0f;
    }
    for (int t0 = 0; t0 < kv; t0 += TR_KEYS) {
        __syncthreads();
        if (tid < TR_KEYS) kbad[tid] = 0;
        __syncthreads();
        for (int i = tid; i < TR_KEYS * ROPE_PAIRS; i += TR_THREADS) {
            const int t = t0 + i / ROPE_PAIRS, e = i % ROPE_PAIRS;
            float x = 0.0f, y = 0.0f, u = 0.0f, w = 0.0f;
            if (t < kv && !(t >= prefix && par[t - prefix] == TREE_UNUSED)) {
                const int pg = a.block_table[(size_t)b * a.W + t / PAGE];
                const size_t k0 = (((size_t)pg * PAGE + t % PAGE) * a.Hkv + kvh) * HEAD_DIM + e;
                const __nv_bfloat16 *kc = reinterpret_cast<const __nv_bfloat16*>(a.k_cache) + k0, *vc = reinterpret_cast<const __nv_bfloat16*>(a.v_cache) + k0;
                const float lo = __bfloat162float(kc[0]), hi = __bfloat162float(kc[ROPE_PAIRS]);
                u = __bfloat162float(vc[0]);
                w = __bfloat162float(vc[ROPE_PAIRS]);
                float c, s;
                rope_cos_sin((uint32_t)(t < prefix ? t : prefix + depth[t - prefix]), a.rope_turns[e], c, s);
                x = lo * c - hi * s;
                y = hi * c + lo * s;
                bool out = !(fabsf(lo) < 32768.0f && fabsf(hi) < 32768.0f);
                if (t >= prefix && !(fabsf(u) < INFINITY && fabsf(w) < INFINITY)) out = true;
                if (out) {
                    kbad[i / ROPE_PAIRS] = 1;
                    x = y = 0.0f;
                    if (t >= prefix) u = w = 0.0f;
                }
            }
            ks[i / ROPE_PAIRS][e] = x;
            ks[i / ROPE_PAIRS][e + ROPE_PAIRS] = y;
            vs[i / ROPE_PAIRS][e] = u;
            vs[i / ROPE_PAIRS][e + ROPE_PAIRS] = w;
        }
        __syncthreads();
        for (int i = 0; i < PER; ++i) {
            const int rr = warp * PER + i, r = blk * TR_ROWS + rr;
            if (r >= R) break;
            const int t = t0 + lane;
            const unsigned long long mask = sees[r % a.T];
            const bool vis = t < kv && mask != 0 && (t < prefix || ((mask >> (t - prefix)) & 1));
            float s = 0.0f;
            for (int d = 0; d < HEAD_DIM; ++d) s = fmaf(qs[rr][d], ks[lane][d], s);
            s = vis ? s * a.qk_scale_log2 : -INFINITY;
            fail[i] |= __any_sync(0xffffffffu, vis && kbad[lane]);
            float top = s;
            for (int k = 16; k; k >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, k));
            if (top == -INFINITY) continue;
            const float mn = fmaxf(m[i], top), alpha = ex2(m[i] - mn), p = ex2(s - mn);
            m[i] = mn;
            float sum = p;
            for (int k = 16; k; k >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, k);
            l[i] = l[i] * alpha + sum;
            for (int e = 0; e < 4; ++e) o[i][e] *= alpha;
            for (int k = 0; k < TR_KEYS; ++k) {
                const float pk = __shfl_sync(0xffffffffu, p, k);
                for (int e = 0; e < 4; ++e) o[i][e] = fmaf(pk, vs[k][lane + 32 * e], o[i][e]);
            }
        }
    }
    for (int i = 0; i < PER; ++i) {
        const int rr = warp * PER + i, r = blk * TR_ROWS + rr;
        if (r >= R) break;
        const bool empty = sees[r % a.T] == 0, out = !empty && (fail[i] || qbad[rr]);
        const float inv = empty || out ? 0.0f : 1.0f / l[i];
        for (int e = 0; e < 4; ++e)
            reinterpret_cast<__nv_bfloat16*>(a.out)[at(r) * HEAD_DIM + lane + 32 * e] = __float2bfloat16_rn(empty || out ? 0.0f : o[i][e] * inv);
        if (lane == 0) {
            a.lse[at(r)] = out ? NAN : empty ? -INFINITY : (m[i] + log2f(l[i])) * 0.693147180559945309f;
            if (out && a.status) atomicOr(a.status, RK_STATUS_RANGE);
        }
    }
}

}  // namespace

cudaError_t launch_tree(const TreeArgs& a, cudaStream_t stream) {
    const long long blocks = (long long)a.B * a.Hkv * ((a.T * a.G + TR_ROWS - 1) / TR_ROWS);
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    tree_kernel<<<(unsigned)blocks, TR_THREADS, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace rk
