// compact.cu -- after a speculative step: the accepted nodes' K and V move to the slots
// behind the prefix.
//
// The cache holds K pre-RoPE ("WS2 PR7 Fused Attention Backend Alignment", "FlashInfer RoPE
// Fusion": RoPE is applied when K is read), so a token at another slot is the same bits and a
// move is a copy.  Slot prefix + i takes node path[i] >= i of an ascending path; a slot that is
// written may be the source of no later token only, so a block holds all of a row's tokens for its
// 512 bytes of a token's K and V before it writes any.
//
// Bound by latency: metadata, pages, one round of loads, one of stores.
#include "rk_device.cuh"
#include "tree_args.h"

namespace rk {

namespace {

constexpr int CP_THREADS = 256;
constexpr int CP_DEPTH = TREE_MAX / (CP_THREADS / 32);  // tokens of a warp

__global__ void __launch_bounds__(CP_THREADS) kv_compact_kernel(const __grid_constant__ CompactArgs a) {
    __shared__ int32_t from[TREE_MAX], to[TREE_MAX];  // slots of the cache, -1 for a token that stays
    const int cols = a.Hkv * 32, groups = cols / 32;  // 16-byte columns of a token: K's, then V's
    const int b = blockIdx.x / groups, col = (int)(blockIdx.x % groups) * 32 + (threadIdx.x & 31);
    const int warp = threadIdx.x >> 5, i = threadIdx.x;
    const int n = a.n_keep[b], kv = a.kv_lens[b];
    int bad = 0;
    if (n < 0 || n > a.T) bad = RK_STATUS_TREE;
    else if (n > 0 && (kv < a.T || kv > a.W * PAGE)) bad = RK_STATUS_KVLEN;
    if (!bad && i < n) {
        const int p = a.path[(size_t)b * a.T + i], before = i ? a.path[(size_t)b * a.T + i - 1] : -1;
        if (p <= before || p >= a.T || before < i - 1) {
            bad = RK_STATUS_TREE;
        } else {
            const int s = kv - a.T + p, d = kv - a.T + i;
            const int ps = a.block_table[(size_t)b * a.W + s / PAGE], pd = a.block_table[(size_t)b * a.W + d / PAGE];
            if (ps < 0 || ps >= a.num_pages || pd < 0 || pd >= a.num_pages) bad = RK_STATUS_PAGE_OOB;
            from[i] = p == i ? -1 : ps * PAGE + s % PAGE;
            to[i] = pd * PAGE + d % PAGE;
        }
    }
    if (bad && a.status) atomicOr(a.status, bad);
    if (__syncthreads_or(bad)) return;  // the row stays as it is
    const size_t row = (size_t)a.Hkv * 16;  // 16-byte chunks of a token in one cache
    uint4* cache = reinterpret_cast<uint4*>(col < a.Hkv * 16 ? a.k_cache : a.v_cache) + (col < a.Hkv * 16 ? col : col - a.Hkv * 16);
    uint4 x[CP_DEPTH];
#pragma unroll
    for (int e = 0; e < CP_DEPTH; ++e) {
        const int t = warp + e * (CP_THREADS / 32);
        if (t < n && from[t] >= 0) x[e] = cache[(size_t)from[t] * row];
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < CP_DEPTH; ++e) {
        const int t = warp + e * (CP_THREADS / 32);
        if (t < n && from[t] >= 0) cache[(size_t)to[t] * row] = x[e];
    }
}

}  // namespace

cudaError_t launch_kv_compact(const CompactArgs& a, cudaStream_t stream) {
    const long long blocks = (long long)a.B * a.Hkv;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    kv_compact_kernel<<<(unsigned)blocks, CP_THREADS, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace rk
