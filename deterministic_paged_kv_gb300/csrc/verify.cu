// verify.cu -- the walk down a row's tree of drafted tokens: which nodes the target's
// distribution accepts, the token behind them, and the tokens' log-probabilities.
//
// Mathematics.  With w(v) = 2^((l(v) - max l) log2(e) / temperature) and Z = sum w, p = w / Z.  After
// rejections the residual r is, up to a factor, (p - a q)+ for one number a: a starts at 0, and a
// rejection adds S(a) = sum (p - a q)+ to it, since with r = (p - a q)+ and S = sum r
//   (r - S q)+ = (p - a q - S q)+      (where r = 0, p - (a + S) q <= 0 as well)
// so a node's state is a number, and each further child one pass over p and q.  Drafts without
// probabilities: the residual is p without the rejected tokens.  The pass over p leaves the children's tokens out
// of its sum; what is left when child n is tried is that sum and the weights of the children from n on, added
// up from the last (sums of positive numbers: nothing cancels), so one pass settles a node.
// The last token is argmax r(v) / race(v): of independent exponential draws of rates r(v) the first to ring, which
// has the distribution r; unlike an inverse of the cumulative sum it does not depend on an order of summation.
//
// Its keys are compared as logarithms, log2 w - log2 race, at a node without children in the same pass as the sum, so that
// a walk that accepts a whole path needs no second pass there.  (Drafts without probabilities: run along at every node it
// saved a pass of 2 to 4 us where the walk ends early, and cost 0.6 to 3 us a node where it does not: 64 x 131072, 8
// accepted nodes 87 us, and 63 without; 20 trees of 13 x 100003 in FP32 44, and 34.)
//
// Work: a cluster of 1 to 16 CTAs (by the batch) walks a row, reading only the nodes that the walk
// reaches.  A pass deals the vocabulary in chunks of 8 to the lanes of 64 virtual warps, a lane's chunks in
// ascending order (in groups of one, two or four, with the lane's running maximum), and joins lanes and warps in a fixed tree, so a
// row's results depend on its data, type and V alone: not on the cluster, nor on how a row lies in memory (a row that does
// not start at 16 bytes is read in whole vectors and shifted, and its ends value by value).  A warp pushes its partial results into every CTA's
// shared memory; behind one cluster barrier a pass every warp joins them and decides for itself.
//
// What bounds it: for few rows the chain of passes, 2.2 us each at V = 32000 (a load, two joins, a cluster barrier, and the
// node's own numbers): a row of 4 nodes 11 us.  For many rows what the warps of a pass wait for, and its exponentials:
// 64 rows of 8 accepted nodes at V = 131072 59 us (63 without probabilities), 7 us a pass, whose 17 MB take 2.5 and whose exponentials take as
// much.  Of a pass's 12700 cycles the first chunks' way is 1500, a group of four chunks 1100 (four of them), the joins and
// pushes of two virtual warps 1200, the barrier 1300, the last join 750, the decision 1200.  With rows that end early and
// draft probabilities 36 us (43 with nothing of it in L2).  FP32 logits with draft probabilities, all nodes accepted: 64 x 8 x 131072
// 94 us and 20 x 13 x 100003 102, of which their bytes take 40 and 15.  Measured against that: chunks asked for only when the
// ones before are summed 71 and 42; 128 virtual warps 20% slower, 32 in FP32 40%; rows fetched to L2 ahead, no change.
#include <algorithm>
#include <atomic>

#include "rk_device.cuh"
#include "tree_args.h"

namespace rk {

namespace {

constexpr int VF_WARPS = 64;            // virtual warps of a pass
constexpr int VF_STEP = VF_WARPS * 32;  // chunks that they take in one round
constexpr int VF_MAX_THREADS = 256;

struct alignas(32) VfPart {
    float m, s;    // largest logit and sum of weights relative to it; or a sum alone
    int v;         // first token of the chunk that has the largest logit
    int bad;       // a value that is none was met
    float key;     // largest key of the race (relative to m, as the weights)
    int kv;        // its token, or its chunk's first
    int pad[2];
};
struct VfShared {
    VfPart part[2][VF_WARPS];
    int par[64], tok[64];  // the row's tree
    float coin[64];
    int path[64], took[64];  // the walk's nodes and the tokens behind them; those tokens' logits, the maxima and sums
    float l[64], top[64], sum[64];
};

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_barrier() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Into the same place of another CTA of the cluster.
__device__ __forceinline__ void push(const VfPart* at, uint32_t rank, const VfPart& x) {
    asm volatile(
        "{\n\t.reg .b32 ra;\n\tmapa.shared::cluster.u32 ra, %0, %1;\n\t"
        "st.shared::cluster.v4.b32 [ra], {%2, %3, %4, %5};\n\t"
        "st.shared::cluster.v2.b32 [ra + 16], {%6, %7};\n\t}" ::"r"(smem_u32(at)),
        "r"(rank), "r"(__float_as_uint(x.m)), "r"(__float_as_uint(x.s)), "r"(x.v), "r"(x.bad), "r"(__float_as_uint(x.key)), "r"(x.kv)
        : "memory");
}

__device__ __forceinline__ float lg2(float x) {
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Largest of a warp's values (a NaN is left out), in every lane.
__device__ __forceinline__ float warp_max(float x) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
    return r;
}

// Eight values of a row from element 8 j on, those past the end as `fill`: asked for, and then taken apart.  (A row
// that does not start at 16 bytes is put together as it arrives, from whole vectors where these lie within the row and
// value by value at its ends, so that nothing outside the caller's array is read; other rows' chunks can be on their way
// several at a time.)
// EVEN: every row starts at 16 bytes and is whole chunks.
template <bool F32, bool EVEN>
struct Chunk {
    static constexpr int VECS = F32 ? 2 : 1;
    uint32_t w[VECS * 4];
    __device__ __forceinline__ void fetch(const char* row, unsigned j, int V, float x) {
        if constexpr (EVEN) {
            if (j < (unsigned)V / 8) load(row, j);
            else fill(x);
        } else {
            fetch_any(row, j, V, x);
        }
    }
    __device__ __forceinline__ void fetch_any(const char* row, unsigned j, int V, float fill) {
        constexpr int SIZE = F32 ? 4 : 2;
        const size_t v0 = (size_t)j * 8;
        const char* at = row + v0 * SIZE;
        const uint32_t off = (uint32_t)reinterpret_cast<uintptr_t>(row) & 15u;  // the same for every chunk
        if (j + (off != 0) >= (unsigned)V / 8 || (off != 0 && j == 0)) {  // (a shifted chunk's vectors reach into both neighbours)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const bool in = v0 + e < (size_t)V;
                if constexpr (F32) {
                    w[e] = in ? __ldg(reinterpret_cast<const uint32_t*>(at) + e) : __float_as_uint(fill);
                } else {
                    const uint32_t x = in ? __ldg(reinterpret_cast<const unsigned short*>(at) + e) : __float_as_uint(fill) >> 16;
                    w[e / 2] = e & 1 ? w[e / 2] | x << 16 : x;
                }
            }
        } else if (off == 0) {
#pragma unroll
            for (int e = 0; e < VECS; ++e) reinterpret_cast<uint4*>(w)[e] = __ldg(reinterpret_cast<const uint4*>(at) + e);
        } else {
            uint32_t x[VECS * 4 + 4];
#pragma unroll
            for (int e = 0; e <= VECS; ++e) reinterpret_cast<uint4*>(x)[e] = __ldg(reinterpret_cast<const uint4*>(at - off) + e);
            if (off & 4)
#pragma unroll
                for (int e = 0; e + 1 < VECS * 4 + 4; ++e) x[e] = x[e + 1];
            if (off & 8)
#pragma unroll
                for (int e = 0; e + 2 < VECS * 4 + 4; ++e) x[e] = x[e + 2];
#pragma unroll
            for (int e = 0; e < VECS * 4; ++e) w[e] = __funnelshift_r(x[e], x[e + 1], (off & 2) * 8);
        }
    }
    // (whole and at 16 bytes)
    __device__ __forceinline__ void load(const char* row, unsigned j) {
        const uint4* at = reinterpret_cast<const uint4*>(row) + (size_t)j * VECS;
#pragma unroll
        for (int e = 0; e < VECS; ++e) reinterpret_cast<uint4*>(w)[e] = __ldg(at + e);
    }
    __device__ __forceinline__ void fill(float x) {
#pragma unroll
        for (int e = 0; e < VECS * 4; ++e) w[e] = F32 ? __float_as_uint(x) : __float_as_uint(x) >> 16 | (__float_as_uint(x) & 0xffff0000u);
    }
    // The largest (a NaN is left out).
    __device__ __forceinline__ float max() const {
        if constexpr (F32) {
            float x = __uint_as_float(w[0]);
#pragma unroll
            for (int e = 1; e < 8; ++e) x = fmaxf(x, __uint_as_float(w[e]));
            return x;
        } else {
            uint32_t x = w[0];
#pragma unroll
            for (int e = 1; e < 4; ++e) asm("max.bf16x2 %0, %0, %1;" : "+r"(x) : "r"(w[e]));
            return fmaxf(bf16lo(x), bf16hi(x));
        }
    }
    __device__ __forceinline__ void take(float2 (&x)[4]) const {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if constexpr (F32) x[e] = make_float2(__uint_as_float(w[2 * e]), __uint_as_float(w[2 * e + 1]));
            else x[e] = make_float2(bf16lo(w[e]), bf16hi(w[e]));
        }
    }
};

// All of a row's walk (see the head of the file).  GROUP: chunks asked for at a time; EVEN: every row of the arrays starts
// at 16 bytes and is whole chunks.
template <bool F32, int GROUP, bool EVEN>
__global__ void __launch_bounds__(VF_MAX_THREADS, 2) verify_kernel(const __grid_constant__ VerifyArgs a) {
    __shared__ VfShared sh;
    const uint32_t rank = cluster_rank();
    const int ctas = a.cluster, b = blockIdx.x / ctas, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int warps = blockDim.x >> 5, mine = VF_WARPS / ctas;  // virtual warps rank * mine .. of this CTA
    const int T = a.T, V = a.V;
    constexpr int SIZE = F32 ? 4 : 2;
    const size_t node0 = (size_t)b * T;
    const char* logits = reinterpret_cast<const char*>(a.logits);
    const char* race = reinterpret_cast<const char*>(a.race + (size_t)b * V);
    const unsigned chunks = ((unsigned)V + 7) / 8;
    const bool probs = a.draft_probs != nullptr;

    // (no CTA writes into another before that one runs)
    if (ctas > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;");
    // ---- the row's tree ----
    if (tid < 64) {
        sh.par[tid] = tid < T ? a.parents[node0 + tid] : TREE_UNUSED;
        sh.tok[tid] = tid < T ? a.draft_tokens[node0 + tid] : 0;
        sh.coin[tid] = tid < T ? a.coins[node0 + tid] : 0.0f;
    }
    const float temp = a.temperature[b];
    const bool greedy = temp == 0.0f;
    __syncthreads();
    if (ctas > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    // (nodes lane and lane + 32 are a lane's)
    auto of = [&](float lo, float hi, int n) {  // node n's value
        lo = __shfl_sync(0xffffffffu, lo, n & 31);
        hi = __shfl_sync(0xffffffffu, hi, n & 31);
        return n & 32 ? hi : lo;
    };
    auto ballot = [&](bool lo, bool hi) {
        const uint64_t y = __ballot_sync(0xffffffffu, hi);
        return y << 32 | __ballot_sync(0xffffffffu, lo);
    };
    // (a row without a root has no use for a temperature)
    int bad = !(greedy || (temp >= 5.421010862427522e-20f && temp < INFINITY) || sh.par[0] == TREE_UNUSED) ? RK_STATUS_RANGE : 0;
    {
        bool wrong[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int n = lane + 32 * e, p = sh.par[n];
            wrong[e] = p < TREE_UNUSED || p >= n || (p >= 0 && sh.par[p] == TREE_UNUSED) ||
                       (n > 0 && p != TREE_UNUSED && (sh.tok[n] < 0 || sh.tok[n] >= V));
        }
        if (ballot(wrong[0], wrong[1])) bad |= RK_STATUS_TREE;
    }
    const bool rootless = !bad && sh.par[0] == TREE_UNUSED;
    const float scale = greedy ? 1.0f : temp, chi = (float)(1.4426950408889634074 / (double)scale);
    const bool writes = rank == 0 && warp == 0;

    const unsigned first_chunk = ((unsigned)rank * mine + warp) * 32;  // of this warp
    const int end = ((int)rank + 1) * mine;
    // ---- a pass: f(warp, part) for the lanes of a virtual warp, join(x, y) of two parts, and all(x) of a warp's; the
    // result in every lane ----
    int pass = 0;
    auto sweep = [&](VfPart zero, auto f, auto join, auto all) {
        VfPart* buf = sh.part[pass & 1];
        ++pass;
#pragma unroll 1
        for (int w = warp; w < mine; w += warps) {
            const int vw = (int)rank * mine + w;
            VfPart x = zero;
            f(vw, x);
            all(x);
            if (ctas == 1) {
                if (lane == 0) buf[vw] = x;
            } else if (lane < ctas) {
                push(&buf[vw], lane, x);
            }
        }
        if (ctas == 1) __syncthreads();
        else cluster_barrier();
        VfPart x = buf[lane];
        join(x, buf[lane + 32]);
        all(x);
        return x;
    };
    auto first_of = [](float& m, int& v, float m2, int v2) {  // the larger, the lower token of equal ones
        if (m2 > m || (m2 == m && v2 < v)) {
            m = m2;
            v = v2;
        }
    };
    auto first_of_all = [](float& m, int& v) {
        const float x = warp_max(m);
        v = __reduce_min_sync(0xffffffffu, m == x ? v : INT32_MAX);
        m = x;
    };
    auto sum_of_all = [](float& s) {
#pragma unroll
        for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    };
    int at = 0, n_acc = 0;
    while (!bad && !rootless) {
        const char* row = logits + (node0 + at) * V * SIZE;
        const char* q = reinterpret_cast<const char*>(a.draft_probs + (probs ? (node0 + at) * V : 0));
        auto logit = [&](int v) {  // (of a token that there is)
            v = min(v, V - 1);
            return F32 ? __ldg(reinterpret_cast<const float*>(row) + v) : bf16lo(__ldg(reinterpret_cast<const unsigned short*>(row) + v));
        };
        auto at16 = [](const char* row) { return (reinterpret_cast<uintptr_t>(row) & 15u) == 0; };
        auto whole = [&](unsigned j) { return j - lane + 32 <= (unsigned)V / 8; };  // a warp's chunks up to lane 31's
        auto ask = [&](auto& c, const char* from, unsigned j, float fill) {
            constexpr int N = sizeof(c) / sizeof(c[0]);
            if constexpr (EVEN) {
#pragma unroll
                for (int u = 0; u < N; ++u) c[u].fetch(from, j + u * VF_STEP, V, fill);
            } else if (at16(from) && whole(j + (N - 1) * VF_STEP)) {
#pragma unroll
                for (int u = 0; u < N; ++u) c[u].load(from, j + u * VF_STEP);
            } else {
#pragma unroll
                for (int u = 0; u < N; ++u) {
                    if (at16(from) && whole(j + u * VF_STEP)) c[u].load(from, j + u * VF_STEP);
                    else if (u == 0 || j + u * VF_STEP - lane < chunks) c[u].fetch(from, j + u * VF_STEP, V, fill);
                    else c[u].fill(fill);
                }
            }
        };
        Chunk<F32, EVEN> next[GROUP];  // the row's first chunks, and then those behind the ones that are summed, on their way
        if (first_chunk < chunks) ask(next, row, first_chunk + lane, -INFINITY);
        // ---- the children: their logits and draft probabilities (on their way while the row is read) ----
        bool kid[2];
        uint32_t lraw[2];  // (asked for unconditionally, of some token: a branch would wait for them)
        float qraw[2];
        const float* from = probs ? reinterpret_cast<const float*>(q) : reinterpret_cast<const float*>(race);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int x = max(0, min(sh.tok[lane + 32 * e], V - 1));
            kid[e] = sh.par[lane + 32 * e] == at;
            lraw[e] = F32 ? __ldg(reinterpret_cast<const uint32_t*>(row) + x) : __ldg(reinterpret_cast<const unsigned short*>(row) + x);
            qraw[e] = __ldg(from + x);
        }
        uint64_t kids = ballot(kid[0], kid[1]);
        const bool leave = !greedy && !probs && kids;  // the sum goes without the children's tokens
        const bool run = !greedy && !kids;             // the race is run along
        bool dup[2] = {false, false};                  // has a child before it the same token
        if (leave) {
            for (uint64_t rest = kids; rest; rest &= rest - 1) {
                const int n = __ffsll((long long)rest) - 1, x = sh.tok[n];
#pragma unroll
                for (int e = 0; e < 2; ++e) dup[e] |= kid[e] && lane + 32 * e > n && sh.tok[lane + 32 * e] == x;
            }
        }
        // Whether the lanes of virtual warp vw meet a child's token at all, and the tokens of chunk j that
        // are children's, as eight bits (whole warps call the first).
        auto meets = [&](int vw) {
            bool hit = false;
#pragma unroll
            for (int e = 0; e < 2; ++e) hit |= kid[e] && (unsigned)sh.tok[lane + 32 * e] / 8 % VF_STEP / 32 == (unsigned)vw;
            return leave && __any_sync(0xffffffffu, hit);
        };
        auto taken = [&](unsigned j) -> uint32_t {
            uint32_t hit = 0;
            for (uint64_t rest = kids; rest; rest &= rest - 1) {
                const int x = sh.tok[__ffsll((long long)rest) - 1];
                if ((unsigned)x / 8 == j) hit |= 1u << (x & 7);
            }
            return hit;
        };
        // ---- the row's maximum (greedy: the first chunk that has it), the sum, and the race ----
        VfPart z = sweep(
            {-INFINITY, 0.0f, INT32_MAX, 0, -INFINITY, INT32_MAX},
            [&](int vw, VfPart& x) {
                const bool some = meets(vw);
#pragma unroll 1
                for (unsigned j0 = vw * 32 + lane; j0 - lane < chunks; j0 += GROUP * VF_STEP) {
                    Chunk<F32, EVEN> c[GROUP];
#pragma unroll
                    for (int u = 0; u < GROUP; ++u) c[u] = next[u];
                    {
                        unsigned j = j0 + GROUP * VF_STEP;
                        if (j - lane >= chunks) j = vw + warps < end ? (vw + warps) * 32 + lane : ~0u;
                        if (j < chunks + 31 && j - lane < chunks) ask(next, row, j, -INFINITY);
                    }
                    float big = x.m;
#pragma unroll
                    for (int u = 0; u < GROUP; ++u) big = fmaxf(big, c[u].max());
                    if (big > x.m) {
                        const float g = __fmul_rn(x.m - big, chi);
                        x.s *= ex2(g);
                        x.key = fmaxf(x.key + g, -INFINITY);  // (never NaN)
                        x.m = big;
                        if (greedy)
#pragma unroll
                            for (int u = GROUP - 1; u >= 0; --u)
                                if (c[u].max() == big) x.v = (int)(j0 + u * VF_STEP) * 8;
                    }
                    const float m = big == -INFINITY ? 0.0f : big;
                    float2 s2 = make_float2(0.0f, 0.0f);
#pragma unroll
                    for (int u = 0; u < GROUP; ++u) {
                        const unsigned j = j0 + u * VF_STEP;
                        if (j - lane >= chunks) break;
                        Chunk<true, EVEN> rc;
                        if (run) {
                            if (!EVEN && at16(race) && whole(j)) rc.load(race, j);
                            else rc.fetch(race, j, V, 1.0f);
                        }
                        float2 d[4];
                        c[u].take(d);
#pragma unroll
                        for (int e = 0; e < 4; ++e) d[e] = fmul2(fadd2(d[e], make_float2(-m, -m)), make_float2(chi, chi));
                        if (some) {
                            const uint32_t hit = taken(j);
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                if ((hit >> (2 * e)) & 1u) d[e].x = -INFINITY;
                                if ((hit >> (2 * e)) & 2u) d[e].y = -INFINITY;
                            }
                        }
#pragma unroll
                        for (int e = 0; e < 4; ++e) s2 = fadd2(s2, make_float2(ex2(d[e].x), ex2(d[e].y)));
                        if (run) {
                            float2 r[4];
                            rc.take(r);
                            float key = -INFINITY;
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                d[e] = make_float2(d[e].x - lg2(r[e].x), d[e].y - lg2(r[e].y));
                                key = fmaxf(key, fmaxf(d[e].x, d[e].y));
                            }
                            if (key > x.key) {  // (seldom)
                                x.key = key;
                                int at8 = 7;
#pragma unroll
                                for (int e = 3; e >= 0; --e) {
                                    if (d[e].y == key) at8 = 2 * e + 1;
                                    if (d[e].x == key) at8 = 2 * e;
                                }
                                x.kv = (int)(j * 8) + at8;
                            }
                        }
                    }
                    x.s += s2.x + s2.y;
                }
            },
            [&](VfPart& x, const VfPart& y) {
                const float top = fmaxf(x.m, y.m);
                const float gx = x.m == top ? 0.0f : __fmul_rn(x.m - top, chi), gy = y.m == top ? 0.0f : __fmul_rn(y.m - top, chi);
                x.s = __fadd_rn(__fmul_rn(x.s, ex2(gx)), __fmul_rn(y.s, ex2(gy)));
                if (greedy) first_of(x.m, x.v, y.m, y.v);
                x.m = top;
                if (run) {
                    x.key = fmaxf(x.key + gx, -INFINITY);
                    first_of(x.key, x.kv, fmaxf(y.key + gy, -INFINITY), y.kv);
                }
            },
            [&](VfPart& x) {
                const float own = x.m;
                if (greedy) first_of_all(x.m, x.v);
                else x.m = warp_max(x.m);
                const float g = own == x.m ? 0.0f : __fmul_rn(own - x.m, chi);
                x.s *= ex2(g);
                sum_of_all(x.s);
                if (run) {
                    x.key = fmaxf(x.key + g, -INFINITY);
                    first_of_all(x.key, x.kv);
                }
            });
        const float top = z.m;
        auto weight = [&](float l) { return ex2(__fmul_rn(__fsub_rn(l, top), chi)); };
        // ---- what is left when each child is tried, if the ones before it were rejected (drafts without probabilities) ----
        float lx[2], w[2], left[2] = {1.0f, 1.0f};
#pragma unroll
        for (int e = 0; e < 2; ++e) lx[e] = F32 ? __uint_as_float(lraw[e]) : bf16lo(lraw[e]);
        const float* qx = qraw;
#pragma unroll
        for (int e = 0; e < 2; ++e) w[e] = kid[e] ? weight(lx[e]) : 0.0f;
        float Z = z.s;
        if (leave) {
            for (uint64_t rest = kids; rest;) {
                const int n = 63 - __clzll((long long)rest);
                rest ^= 1ull << n;
                Z += of(dup[0] ? 0.0f : w[0], dup[1] ? 0.0f : w[1], n);
                if (n == lane) left[0] = Z;
                if (n == lane + 32) left[1] = Z;
            }
        }
        if (!(Z > 0.0f && Z < INFINITY)) {  // a NaN, an infinity, or no token at all
            bad |= RK_STATUS_RANGE;
            break;
        }
        const float inv = probs ? 1.0f / Z : 0.0f;
        const int here = n_acc++;
        auto note = [&](int token, float l) {
            if (writes && lane == 0) {
                sh.path[here] = at;
                sh.took[here] = token;
                sh.l[here] = l;
                sh.top[here] = top;
                sh.sum[here] = Z;
            }
        };
        // A sweep says in which chunk its token lies; the token is the first of those that have the chunk's value again, from
        // the same operations (none of them: no token, which fails the row).
        auto token_of = [&](int first, bool has) {
            const uint32_t hit = __ballot_sync(0xffffffffu, lane < 8 && first + lane < V && has);
            return hit ? first + __ffs(hit) - 1 : INT32_MAX;
        };
        int best = 0;
        if (greedy) best = token_of(z.v, logit(z.v + (lane & 7)) == top);
        if (best >= V) {
            bad |= RK_STATUS_RANGE;
            break;
        }
        auto race_at = [&](int v) { return __ldg(reinterpret_cast<const float*>(race) + min(v, V - 1)); };
        // ---- the children in order ----
        int took = -1;
        float aq = 0.0f, S = 1.0f;
        // the key of a token of what is left, or by p's own weights; -inf where it has no part in it.  (Rounded as written: the
        // token is found by its key, so no compiler may join a product and a difference at one place and not at the other.)
        auto own_key = [&](float l, float r) {
            const float t = __fmul_rn(__fsub_rn(l, top), chi);
            return ex2(t) > 0.0f ? __fsub_rn(t, lg2(r)) : -INFINITY;
        };
        auto left_key = [&](float l, float d, float r) {
            const float k = fmaf(weight(l), inv, __fmul_rn(-aq, d));
            return k > 0.0f ? __fsub_rn(lg2(k), lg2(r)) : -INFINITY;
        };
        if (!probs || greedy) {
            bool yes[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) yes[e] = kid[e] && (greedy ? sh.tok[lane + 32 * e] == best : !dup[e] && sh.coin[lane + 32 * e] * left[e] < w[e]);
            const uint64_t hit = ballot(yes[0], yes[1]);
            if (hit) took = __ffsll((long long)hit) - 1;
        } else {
            for (uint64_t rest = kids; rest && took < 0 && !bad;) {
                const int n = __ffsll((long long)rest) - 1;
                rest &= rest - 1;
                bool yes[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) yes[e] = lane + 32 * e == n && sh.coin[n] * qx[e] * S < fmaxf(fmaf(w[e], inv, -aq * qx[e]), 0.0f);
                if (ballot(yes[0], yes[1])) {
                    took = n;
                    break;
                }
                aq += S;
                if (!rest) break;
                const VfPart y = sweep(
                    {0.0f, 0.0f, 0, 0, 0.0f, 0},
                    [&](int vw, VfPart& x) {
#pragma unroll 1
                        for (unsigned j0 = vw * 32 + lane; j0 - lane < chunks; j0 += GROUP * VF_STEP) {
                            Chunk<F32, EVEN> c[GROUP];
                            Chunk<true, EVEN> qc[GROUP];
                            ask(c, row, j0, -INFINITY);
                            ask(qc, q, j0, 0.0f);
#pragma unroll
                            for (int u = 0; u < GROUP; ++u) {
                                if (j0 + u * VF_STEP - lane >= chunks) break;
                                float2 l[4], d[4], s = make_float2(0.0f, 0.0f), none = s;
                                c[u].take(l);
                                qc[u].take(d);
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    const float2 r = ffma2(make_float2(weight(l[e].x), weight(l[e].y)), make_float2(inv, inv),
                                                           fmul2(d[e], make_float2(-aq, -aq)));
                                    s = fadd2(s, make_float2(fmaxf(r.x, 0.0f), fmaxf(r.y, 0.0f)));
                                    none = ffma2(r, make_float2(0.0f, 0.0f), none);  // NaN where q is none or infinite
                                }
                                s = fadd2(s, none);
                                x.s += s.x + s.y;
                            }
                        }
                    },
                    [](VfPart& x, const VfPart& y) { x.s += y.s; }, [&](VfPart& x) { sum_of_all(x.s); });
                S = y.s;
                if (!(S >= 0.0f)) bad |= RK_STATUS_RANGE;
            }
            if (bad) break;
        }
        if (took >= 0) {
            note(sh.tok[took], of(lx[0], lx[1], took));
            at = took;
            continue;
        }
        // ---- the last token: of what is left, or of p where that is nothing ----
        int last = greedy ? best : INT32_MAX;
        // (the race along with the sum compares tokens with their lanes' maxima, so one that weighs nothing can win it
        // where its draw is 0; then it is run again)
        if (run && z.kv < V && weight(logit(z.kv)) > 0.0f) last = z.kv;
        for (int all = !kids; last >= V && all < 2; ++all) {
            const bool own = all || !probs;
            const VfPart y = sweep(
                {0.0f, 0.0f, 0, 0, -INFINITY, INT32_MAX},
                [&](int vw, VfPart& x) {
                    const bool some = !all && meets(vw);
#pragma unroll 1
                    for (unsigned j0 = vw * 32 + lane; j0 - lane < chunks; j0 += 2 * VF_STEP) {
                        Chunk<F32, EVEN> c[2];
                        Chunk<true, EVEN> rc[2], qc[2];
                        ask(c, row, j0, -INFINITY);
                        ask(rc, race, j0, 1.0f);
                        if (!own) ask(qc, q, j0, 0.0f);
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            if (j0 + u * VF_STEP - lane >= chunks) break;
                            float2 l[4], r[4], d[4];
                            c[u].take(l);
                            rc[u].take(r);
                            if (!own) qc[u].take(d);
                            float key = -INFINITY;
                            if (own) {
                                if (some) {
                                    const uint32_t hit = taken(j0 + u * VF_STEP);
#pragma unroll
                                    for (int e = 0; e < 4; ++e) {
                                        if ((hit >> (2 * e)) & 1u) l[e].x = -INFINITY;
                                        if ((hit >> (2 * e)) & 2u) l[e].y = -INFINITY;
                                    }
                                }
#pragma unroll
                                for (int e = 0; e < 4; ++e) key = fmaxf(key, fmaxf(own_key(l[e].x, r[e].x), own_key(l[e].y, r[e].y)));
                            } else {
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    key = fmaxf(key, fmaxf(left_key(l[e].x, d[e].x, r[e].x), left_key(l[e].y, d[e].y, r[e].y)));
                                    if (!(fabsf(d[e].x) < INFINITY && fabsf(d[e].y) < INFINITY)) x.bad = 1;
                                }
                            }
                            if (key > x.key) {
                                x.key = key;
                                x.kv = (int)((j0 + u * VF_STEP) * 8);
                            }
                        }
                    }
                },
                [&](VfPart& x, const VfPart& y) {
                    first_of(x.key, x.kv, y.key, y.kv);
                    x.bad |= y.bad;
                },
                [&](VfPart& x) {
                    first_of_all(x.key, x.kv);
                    x.bad = __any_sync(0xffffffffu, x.bad);
                });
            if (y.bad) bad |= RK_STATUS_RANGE;
            if (bad) break;
            if (y.kv < V) {
                const int v = min(y.kv + (lane & 7), V - 1);
                const float d = own ? 0.0f : __ldg(reinterpret_cast<const float*>(q) + v);
                const uint32_t hit = !all && leave ? taken((unsigned)y.kv / 8) : 0u;
                last = token_of(y.kv, !((hit >> (lane & 7)) & 1u) &&
                                          (own ? own_key(logit(v), race_at(v)) : left_key(logit(v), d, race_at(v))) == y.key);
                if (last >= V) break;
            }
        }
        if (bad || last >= V) {  // (no draw of the race is a number that is not negative)
            bad |= RK_STATUS_RANGE;
            break;
        }
        note(last, logit(last));
        break;
    }
    if (writes) {
        if (bad && lane == 0 && a.status) atomicOr(a.status, bad);
        const int n = bad || rootless ? 0 : n_acc;
        __syncwarp();
        for (int i = lane; i < T; i += 32) {
            a.path[node0 + i] = i < n ? sh.path[i] : -1;
            a.tokens[node0 + i] = i < n ? sh.took[i] : -1;
            a.logprobs[node0 + i] = i < n ? (sh.l[i] - sh.top[i]) / scale - logf(sh.sum[i]) : bad ? NAN : 0.0f;
        }
        if (lane == 0) {
            a.n_accepted[b] = n;
            a.n_drop[b] = rootless ? 0 : T - n;
        }
    }
    if (ctas > 1) cluster_barrier();  // no CTA leaves while another may still write into it
}

}  // namespace

cudaError_t launch_verify(const VerifyArgs& a, cudaStream_t stream) {
    static std::atomic<uint64_t> configured{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? (1ull << dev) : 0;
    if (!bit || !(configured.load() & bit)) {
        for (const void* f : {(const void*)verify_kernel<false, 2, false>, (const void*)verify_kernel<false, 4, false>,
                              (const void*)verify_kernel<true, 1, false>, (const void*)verify_kernel<false, 2, true>,
                              (const void*)verify_kernel<false, 4, true>, (const void*)verify_kernel<true, 1, true>})
            if ((e = cudaFuncSetAttribute(f, cudaFuncAttributeNonPortableClusterSizeAllowed, 1)) != cudaSuccess) return e;
        configured.fetch_or(bit);
    }
    VerifyArgs r = a;
    // As many CTAs to a row as have room at two to an SM, all at once.  Chains of 8 accepted nodes, at most 152 CTAs / 304
    // / 608: 64 x 131072 86 / 59 / 78 us, 20 x 131072 44 / 33 / 33, 64 x 32000 36 / 29 / 45; rows of mixed lengths,
    // where a waiting cluster takes the room of one that is done, 54 / 37 / 37.
    r.cluster = 16;
    while (r.cluster > 1 && (long long)a.B * r.cluster > 304) r.cluster /= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.B * r.cluster));
    cfg.blockDim = dim3((unsigned)std::min(VF_MAX_THREADS, 32 * VF_WARPS / r.cluster));
    cfg.stream = stream;
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (unsigned)r.cluster;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    // Chunks of a lane, asked for at a time: in BF16 up to two where that is all (two rounds of VF_STEP chunks).  64 rows of 8
    // accepted nodes by 2 / by 4 in us: V = 16384 27.5 / 28.8, 32768 32.3 / 33.9, 40000 40.4 / 36.5, 65536 44.5 / 42.1, 98304
    // 57.5 / 54.6, 131072 70.0 / 62.2; one row 32768 19.4 / 20.1, 40000 20.9 / 20.8, 131072 30.1 / 29.4.  In FP32 20 x 100003
    // 30.1 with 1, 30.8 with 2.
    // Rows that all start at 16 bytes and are whole chunks do without the code for the ends of others: one row of 8 x 32000
    // 12.4 us a call, 13.6 with it; 64 x 8 x 131072 45.8 and 46.3.  (Every product that is added to is rounded by itself, so
    // that both have the same bits.)
    const bool two = a.V <= 2 * 8 * VF_STEP;
    const bool even = a.V % 8 == 0 && ((reinterpret_cast<uintptr_t>(a.logits) | reinterpret_cast<uintptr_t>(a.draft_probs) |
                                        reinterpret_cast<uintptr_t>(a.race)) & 15u) == 0;
    if (even) {
        if (a.f32) return cudaLaunchKernelEx(&cfg, verify_kernel<true, 1, true>, r);
        return two ? cudaLaunchKernelEx(&cfg, verify_kernel<false, 2, true>, r) : cudaLaunchKernelEx(&cfg, verify_kernel<false, 4, true>, r);
    }
    if (a.f32) return cudaLaunchKernelEx(&cfg, verify_kernel<true, 1, false>, r);
    return two ? cudaLaunchKernelEx(&cfg, verify_kernel<false, 2, false>, r) : cudaLaunchKernelEx(&cfg, verify_kernel<false, 4, false>, r);
}

}  // namespace rk
