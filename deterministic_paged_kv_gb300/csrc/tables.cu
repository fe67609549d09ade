// tables.cu -- a step's tables on the device: new pages from a pool of free
// ones, block table entries, lengths, indptr, positions and slot map, from the
// rows' lengths and token counts alone, so that a captured graph of steps
// advances without the host.  The tables are those that the attention calls
// walk ("WS2 PR7 Fused Attention Backend Alignment", "Current Implementation":
// logical page order, canonical -1 padding, trailing query positions).
//
// Mathematics: two prefix sums over the rows, of the tokens (qo_indptr) and of
// the new pages ceil((len + n) / 16) - ceil(len / 16); then each token finds
// its row by bisection of qo_indptr, and everything else is arithmetic.
//
// Up to 4096 tokens one CTA does all of it.  Beyond, that CTA leaves the tokens to a second
// launch, which has all it needs in the first one's outputs: every CTA of it sums the rows'
// pages once more (a few loads per thread) and takes a share of the tokens.  (kv_lens and taken
// may be updated in place, so the CTAs of one launch could not read them and write them
// without a barrier over all; a cluster of 8 CTAs has one, and took 36 us where this takes
// 8.7.)  Bound by latency: launch, one round of loads, the scan, one round of stores; 64 rows of one
// token 4.5 us, 1024 rows of 520000 tokens 8.7 us.
#include <algorithm>
#include <atomic>

#include "q8_args.h"
#include "rk_device.cuh"

namespace rk {

namespace {

// Exclusive prefix sums over the block of two values per thread (all threads
// call it); totals in *ta, *tb.
__device__ void scan2(long long& a, long long& b, long long* ta, long long* tb, long long* sh) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long a0 = a, b0 = b;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, a, o), y = __shfl_up_sync(0xffffffffu, b, o);
        if (lane >= o) {
            a += x;
            b += y;
        }
    }
    __syncthreads();  // sh may still be read by a scan before this one
    if (lane == 31) {
        sh[warp] = a;
        sh[32 + warp] = b;
    }
    __syncthreads();
    const bool there = lane < (int)blockDim.x / 32;
    long long wa = there ? sh[lane] : 0, wb = there ? sh[32 + lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, wa, o), y = __shfl_up_sync(0xffffffffu, wb, o);
        if (lane >= o) {
            wa += x;
            wb += y;
        }
    }
    *ta = __shfl_sync(0xffffffffu, wa, 31);
    *tb = __shfl_sync(0xffffffffu, wb, 31);
    const long long pa = __shfl_sync(0xffffffffu, wa, (warp + 31) & 31), pb = __shfl_sync(0xffffffffu, wb, (warp + 31) & 31);
    a += (warp ? pa : 0) - a0;
    b += (warp ? pb : 0) - b0;
}

__device__ __forceinline__ int pages_of(int n) { return (int)(((unsigned)n + PAGE - 1) / PAGE); }

// What the rows' part leaves in shared memory, [B] each: a row's first token, its first new
// page's place in the pool, its length before.
struct Rows {
    int32_t *tok, *page, *len;
};

// This CTA's share of the tokens, four neighbours to a thread.  Returns status bits.
__device__ int fill_tokens(const TablesArgs& a, const Rows& rows, int total) {
    int bad = 0;
    const bool wide = ((reinterpret_cast<uintptr_t>(a.position_ids) | reinterpret_cast<uintptr_t>(a.slot_map)) & 15) == 0;
    const long long step = 4ll * (int)blockDim.x * gridDim.x;
    for (long long i0 = 4ll * ((long long)blockIdx.x * (int)blockDim.x + threadIdx.x); i0 < a.cap; i0 += step) {
        int pos[4], slot[4];
        int r = -1, next = -1, start = 0, len = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const long long i = i0 + k;
            pos[k] = slot[k] = -1;
            if (i >= total) continue;
            if (i >= next) {  // the last row that starts at or before token i (rows without tokens share a start)
                int lo = r < 0 ? 0 : r, hi = a.B;
                while (hi - lo > 1) {
                    const int mid = (lo + hi) >> 1;
                    if (rows.tok[mid] <= i) lo = mid;
                    else hi = mid;
                }
                r = lo;
                start = rows.tok[r];
                len = rows.len[r];
                next = r + 1 < a.B ? rows.tok[r + 1] : total;
            }
            const int p = len + (int)i - start, j = p / PAGE, have = pages_of(len);
            const int page = j < have ? a.block_table[(size_t)r * a.W + j] : a.pool[rows.page[r] + j - have];
            if (j >= have && (p % PAGE) == 0) a.block_table[(size_t)r * a.W + j] = page;
            pos[k] = p;
            if (page < 0 || page >= a.num_pages) bad |= RK_STATUS_PAGE_OOB;
            else slot[k] = page * PAGE + p % PAGE;
        }
        if (wide && i0 + 4 <= a.cap) {
            *reinterpret_cast<int4*>(a.position_ids + i0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
            *reinterpret_cast<int4*>(a.slot_map + i0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
        } else {
            for (int k = 0; k < 4 && i0 + k < a.cap; ++k) {
                a.position_ids[i0 + k] = pos[k];
                a.slot_map[i0 + k] = slot[k];
            }
        }
    }
    return bad;
}

// The rows; ALL: and the tokens.
template <bool ALL>
__global__ void __launch_bounds__(TAB_THREADS) tables_kernel(const __grid_constant__ TablesArgs a) {
    extern __shared__ int32_t rows[];
    __shared__ long long sh[64];
    int32_t* s_tok = rows;
    int32_t* s_page = rows + a.B;
    int32_t* s_len = rows + 2 * a.B;
    if constexpr (!ALL) griddep_launch_dependents();
    const int tid = threadIdx.x;
    const int per = (a.B + (int)blockDim.x - 1) / (int)blockDim.x;
    const int r0 = min(a.B, tid * per), r1 = min(a.B, r0 + per);
    const int taken = *a.taken;
    const bool taken_ok = taken >= 0 && taken <= a.n_pool;
    const long long avail = taken_ok ? a.n_pool - taken : 0;
    int bad = taken_ok ? 0 : RK_STATUS_POOL;

    // ---- the rows' demands.  s_page holds a row's token count until it is known where its pages start. ----
    long long tok = 0, pg = 0;
    for (int r = r0; r < r1; ++r) {
        const int len = a.kv_lens[r];
        int n = a.n_new[r];
        if (len < 0 || n < 0 || (long long)len + n > (long long)a.W * PAGE) {
            bad |= RK_STATUS_KVLEN;
            n = 0;
        }
        s_len[r] = len;
        s_page[r] = n;
        tok += n;
        if (n > 0) pg += pages_of(len + n) - pages_of(len);
    }
    long long tok_all, pg_all;
    scan2(tok, pg, &tok_all, &pg_all, sh);
    if (tok_all > a.cap || pg_all > avail) {
        // Something does not fit (the same verdict in every thread).  A row is
        // refused if the tokens up to it pass the arrays' capacity, then if the
        // new pages of the rows left up to it pass the pool; rows that need
        // nothing of what ran out stay.
        bad |= RK_STATUS_POOL;
        long long run = tok;
        pg = 0;
        for (int r = r0; r < r1; ++r) {
            const int n = s_page[r];
            run += n;
            if (run > a.cap) s_page[r] = 0;
            if (s_page[r] > 0) pg += pages_of(s_len[r] + s_page[r]) - pages_of(s_len[r]);
        }
        long long none = 0, t0;
        scan2(none, pg, &t0, &pg_all, sh);
        run = pg;
        tok = pg = 0;
        for (int r = r0; r < r1; ++r) {
            if (s_page[r] <= 0) continue;
            const int need = pages_of(s_len[r] + s_page[r]) - pages_of(s_len[r]);
            run += need;
            if (need > 0 && run > avail) {
                s_page[r] = 0;
            } else {
                pg += need;
                tok += s_page[r];
            }
        }
        scan2(tok, pg, &tok_all, &pg_all, sh);
    }
    {
        int t = (int)tok, p = taken + (int)pg;
        for (int r = r0; r < r1; ++r) {
            const int n = s_page[r];
            s_tok[r] = t;
            s_page[r] = p;
            t += n;
            if (n > 0) p += pages_of(s_len[r] + n) - pages_of(s_len[r]);
        }
    }
    __syncthreads();
    const int total = (int)tok_all;
    for (int r = tid; r < a.B; r += (int)blockDim.x) {
        const int t = s_tok[r], e = r + 1 < a.B ? s_tok[r + 1] : total;
        a.qo_indptr[r] = t;
        a.kv_lens_out[r] = s_len[r] + (e - t);
    }
    if (tid == 0) {
        a.qo_indptr[a.B] = total;
        *a.taken_out = taken + (int)pg_all;
    }

    if constexpr (ALL) {
        bad |= fill_tokens(a, {s_tok, s_page, s_len}, total);
    }
    if (bad && a.status) atomicOr(a.status, bad);
}

// The tokens, after tables_kernel<false>: lengths and pages of the rows from its outputs.
__global__ void __launch_bounds__(TAB_THREADS) tokens_kernel(const __grid_constant__ TablesArgs a) {
    extern __shared__ int32_t rows[];
    __shared__ long long sh[64];
    const Rows s = {rows, rows + a.B, rows + 2 * a.B};
    const int per = (a.B + (int)blockDim.x - 1) / (int)blockDim.x;
    const int r0 = min(a.B, (int)threadIdx.x * per), r1 = min(a.B, r0 + per);
    griddep_wait();
    const int total = a.qo_indptr[a.B];
    int t = r0 < r1 ? a.qo_indptr[r0] : total;
    long long pg = 0, none = 0, pg_all, t0;
    for (int r = r0; r < r1; ++r) {
        const int e = a.qo_indptr[r + 1], n = e - t, len = a.kv_lens_out[r] - n;
        s.tok[r] = t;
        s.len[r] = len;
        s.page[r] = n > 0 ? pages_of(len + n) - pages_of(len) : 0;
        pg += s.page[r];
        t = e;
    }
    scan2(none, pg, &t0, &pg_all, sh);
    int p = *a.taken_out - (int)pg_all + (int)pg;
    for (int r = r0; r < r1; ++r) {
        const int need = s.page[r];
        s.page[r] = p;
        p += need;
    }
    __syncthreads();
    const int bad = fill_tokens(a, s, total);
    if (bad && a.status) atomicOr(a.status, bad);
}

}  // namespace

cudaError_t launch_tables(const TablesArgs& a, cudaStream_t stream) {
    const int smem = 3 * a.B * 4;
    static std::atomic<uint64_t> configured{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? (1ull << dev) : 0;
    if (!bit || !(configured.load() & bit)) {
        for (const void* f : {(const void*)tables_kernel<true>, (const void*)tables_kernel<false>, (const void*)tokens_kernel}) {
            e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, 3 * TAB_MAX_ROWS * 4);
            if (e != cudaSuccess) return e;
        }
        configured.fetch_or(bit);
    }
    if (a.cap <= 4 * TAB_THREADS) {
        // (a small step: 64 rows of one token 4.5 us with 128 threads, 5.2 with 1024)
        tables_kernel<true><<<1, a.cap <= 512 && a.B <= 128 ? 128 : TAB_THREADS, smem, stream>>>(a);
        return cudaGetLastError();
    }
    tables_kernel<false><<<1, TAB_THREADS, smem, stream>>>(a);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)std::min<long long>(152, (a.cap + 4ll * TAB_THREADS - 1) / (4ll * TAB_THREADS)));
    cfg.blockDim = dim3(TAB_THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, tokens_kernel, a);
}

}  // namespace rk
