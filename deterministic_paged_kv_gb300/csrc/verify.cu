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
// Work: a cluster of 1 to 16 CTAs (by the batch) walks a row, reading only the nodes that the walk
// reaches.  A pass deals the vocabulary in chunks of 8 to the lanes of 64 virtual warps, a lane's chunks in
// ascending order (running maximum and sum), and adds the warps up in a fixed tree, so a row's results depend on
// its data and V alone: not on the cluster, nor on how a row lies in memory (a row that does not start at 16
// bytes is read in whole vectors and shifted).  A warp pushes its partial results into every CTA's
// shared memory; behind one cluster barrier a pass every warp adds them up and decides for itself.
// Bound by bytes for many rows and by the chain of passes for few: a round trip to memory, a barrier and
// a few shuffles each.
#include <algorithm>
#include <atomic>

#include "rk_device.cuh"
#include "tree_args.h"

namespace rk {

namespace {

constexpr int VF_WARPS = 64;                 // virtual warps of a pass
constexpr int VF_BLOCK = VF_WARPS * 32 * 8;  // tokens that they take in one round
constexpr int VF_MAX_THREADS = 512;
constexpr int VF_BITS = 8192;                // chunks with a child's token, by number modulo this

struct VfPart {
    float m, s;   // largest logit and sum of weights relative to it; or a sum; or the largest key
    int v, bad;   // a token that has the largest, or its chunk's first; a value that is none was met
};
struct VfShared {
    VfPart part[2][VF_WARPS];
    uint32_t child[VF_BITS / 32];
};

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_barrier() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// 16 bytes into the same place of another CTA of the cluster.
__device__ __forceinline__ void push(const void* at, uint32_t rank, const VfPart& x) {
    asm volatile(
        "{\n\t.reg .b32 ra;\n\tmapa.shared::cluster.u32 ra, %0, %1;\n\t"
        "st.shared::cluster.v4.b32 [ra], {%2, %3, %4, %5};\n\t}" ::"r"(smem_u32(at)),
        "r"(rank), "r"(__float_as_uint(x.m)), "r"(__float_as_uint(x.s)), "r"(x.v), "r"(x.bad)
        : "memory");
}

// Eight values of a row from element 8 j on, those past the end as `fill`.
template <bool F32>
__device__ __forceinline__ void load8(const char* row, unsigned j, int V, float fill, float (&x)[8]) {
    constexpr int SIZE = F32 ? 4 : 2, VECS = F32 ? 2 : 1;
    const size_t v0 = (size_t)j * 8;
    const char* at = row + v0 * SIZE;
    if (v0 + 8 > (size_t)V) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            x[e] = fill;
            if (v0 + e < (size_t)V)
                x[e] = F32 ? __ldg(reinterpret_cast<const float*>(at) + e) : bf16lo(__ldg(reinterpret_cast<const unsigned short*>(at) + e));
        }
        return;
    }
    const uint32_t off = (uint32_t)reinterpret_cast<uintptr_t>(at) & 15u;  // the same for every chunk of the row
    const uint4* vec = reinterpret_cast<const uint4*>(at - off);
    uint32_t w[VECS * 4 + 4];
#pragma unroll
    for (int e = 0; e <= VECS; ++e) {
        // (the vector behind the last holds some of the chunk where there is an offset, so it may be read)
        const uint4 y = e < VECS || off ? __ldg(vec + e) : make_uint4(0, 0, 0, 0);
        w[4 * e] = y.x;
        w[4 * e + 1] = y.y;
        w[4 * e + 2] = y.z;
        w[4 * e + 3] = y.w;
    }
    if (off & 4)
#pragma unroll
        for (int e = 0; e + 1 < VECS * 4 + 4; ++e) w[e] = w[e + 1];
    if (off & 8)
#pragma unroll
        for (int e = 0; e + 2 < VECS * 4 + 4; ++e) w[e] = w[e + 2];
    if constexpr (F32) {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = __uint_as_float(w[e]);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t u = __funnelshift_r(w[e], w[e + 1], (off & 2) * 8);
            x[2 * e] = bf16lo(u);
            x[2 * e + 1] = bf16hi(u);
        }
    }
}

// All of a row's walk (see the head of the file).
template <bool F32>
__global__ void __launch_bounds__(VF_MAX_THREADS) verify_kernel(const __grid_constant__ VerifyArgs a) {
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

    // ---- the row's tree: nodes lane and lane + 32 of every warp ----
    int par[2], tok[2];
    float coin[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int n = lane + 32 * e;
        par[e] = n < T ? a.parents[node0 + n] : TREE_UNUSED;
        tok[e] = n < T ? a.draft_tokens[node0 + n] : 0;
        coin[e] = n < T ? a.coins[node0 + n] : 0.0f;
    }
    const float temp = a.temperature[b];
    const bool greedy = temp == 0.0f;
    for (int i = tid; i < VF_BITS / 32; i += blockDim.x) sh.child[i] = 0;
    {
        // The last draw's numbers on their way to L2, and in a small batch the nodes' logits (each CTA its share).
        auto fetch = [&](const char* p, size_t bytes) {
            for (size_t i = ((size_t)rank * blockDim.x + tid) * 128; i < bytes; i += (size_t)ctas * blockDim.x * 128)
                asm volatile("prefetch.global.L2 [%0];" ::"l"(p + i));
        };
        if (a.prefetch_nodes) fetch(logits + node0 * V * SIZE, (size_t)T * V * SIZE);
        if (!greedy) fetch(race, (size_t)V * 4);
    }
    auto of = [&](const int (&x)[2], int n) {  // node n's value
        const int lo = __shfl_sync(0xffffffffu, x[0], n & 31), hi = __shfl_sync(0xffffffffu, x[1], n & 31);
        return n & 32 ? hi : lo;
    };
    auto ballot = [&](bool lo, bool hi) {
        const uint64_t y = __ballot_sync(0xffffffffu, hi);
        return y << 32 | __ballot_sync(0xffffffffu, lo);
    };
    int bad = !(greedy || (temp >= 5.421010862427522e-20f && temp < INFINITY)) ? RK_STATUS_RANGE : 0;
    {
        bool wrong[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int n = lane + 32 * e, up = of(par, par[e] & 63);
            wrong[e] = par[e] < TREE_UNUSED || par[e] >= n || (par[e] >= 0 && up == TREE_UNUSED) ||
                       (n > 0 && par[e] != TREE_UNUSED && (tok[e] < 0 || tok[e] >= V));
        }
        if (ballot(wrong[0], wrong[1])) bad |= RK_STATUS_TREE;
    }
    const bool rootless = !bad && of(par, 0) == TREE_UNUSED;
    const float scale = greedy ? 1.0f : temp, chi = (float)(1.4426950408889634074 / (double)scale);
    const bool writes = rank == 0 && warp == 0;

    // ---- a pass: f(chunk, part) for a lane's chunks, join(x, y) of two parts; the result in every lane ----
    int pass = 0;
    auto sweep = [&](VfPart zero, auto f, auto join) {
        VfPart* buf = sh.part[pass & 1];
        ++pass;
#pragma unroll 1
        for (int w = warp; w < mine; w += warps) {
            const int vw = (int)rank * mine + w;
            VfPart x = zero;
            f(vw, x);
#pragma unroll
            for (int o = 16; o; o >>= 1) {
                VfPart y;
                y.m = __shfl_xor_sync(0xffffffffu, x.m, o);
                y.s = __shfl_xor_sync(0xffffffffu, x.s, o);
                y.v = __shfl_xor_sync(0xffffffffu, x.v, o);
                y.bad = __shfl_xor_sync(0xffffffffu, x.bad, o);
                join(x, y);
            }
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
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            VfPart y;
            y.m = __shfl_xor_sync(0xffffffffu, x.m, o);
            y.s = __shfl_xor_sync(0xffffffffu, x.s, o);
            y.v = __shfl_xor_sync(0xffffffffu, x.v, o);
            y.bad = __shfl_xor_sync(0xffffffffu, x.bad, o);
            join(x, y);
        }
        return x;
    };
    // the largest key, the lowest token of equal ones
    auto join_max = [](VfPart& x, const VfPart& y) {
        if (y.m > x.m || (y.m == x.m && y.v < x.v)) {
            x.m = y.m;
            x.v = y.v;
        }
        x.bad |= y.bad;
    };
    auto join_sum = [](VfPart& x, const VfPart& y) { x.s += y.s; };

    int at = 0, n_acc = 0;
    while (!bad && !rootless) {
        const char* row = logits + (node0 + at) * V * SIZE;
        const char* q = reinterpret_cast<const char*>(a.draft_probs + (probs ? (node0 + at) * V : 0));
        auto logit = [&](int v) {
            return F32 ? __ldg(reinterpret_cast<const float*>(row) + v) : bf16lo(__ldg(reinterpret_cast<const unsigned short*>(row) + v));
        };
        // ---- the children: their logits and draft probabilities (on their way while the row is read) ----
        bool kid[2];
        float lx[2], qx[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            kid[e] = par[e] == at;
            lx[e] = kid[e] ? logit(tok[e]) : 0.0f;
            qx[e] = kid[e] && probs && !greedy ? __ldg(reinterpret_cast<const float*>(q) + tok[e]) : 1.0f;
        }
        uint64_t kids = ballot(kid[0], kid[1]);
        const bool leave = !greedy && !probs && kids;  // the sum goes without the children's tokens
        bool dup[2] = {false, false};                  // has a child before it the same token
        if (leave) {
            if (warp == 0) {
                for (int e = 0; e < 2; ++e)
                    if (kid[e]) atomicOr(&sh.child[(tok[e] / 8 % VF_BITS) / 32], 1u << (tok[e] / 8 % 32));
            }
            for (uint64_t left = kids; left; left &= left - 1) {
                const int n = __ffsll((long long)left) - 1, x = of(tok, n);
#pragma unroll
                for (int e = 0; e < 2; ++e) dup[e] |= kid[e] && lane + 32 * e > n && tok[e] == x;
            }
            __syncthreads();
        }
        // tokens of chunk j that children have, as eight bits
        auto taken = [&](unsigned j) -> uint32_t {
            uint32_t hit = 0;
            for (uint64_t left = kids; left; left &= left - 1) {
                const int x = of(tok, __ffsll((long long)left) - 1);
                if ((unsigned)x / 8 == j) hit |= 1u << (x & 7);
            }
            return hit;
        };
        // (whole warps call it: the lists of children lie in lanes)
        auto out_of = [&](unsigned j) -> uint32_t {
            const bool maybe = leave && ((sh.child[(j % VF_BITS) / 32] >> (j % 32)) & 1u);
            return __any_sync(0xffffffffu, maybe) ? taken(j) : 0u;
        };
        // ---- the row's maximum, where it is, and the sum ----
        VfPart z = sweep({-INFINITY, 0.0f, INT32_MAX, 0},
                         [&](int vw, VfPart& x) {
#pragma unroll 2
                             for (unsigned j0 = vw * 32; j0 < chunks; j0 += VF_WARPS * 32) {
                                 const unsigned j = j0 + lane;
                                 float l[8];
                                 load8<F32>(row, j, V, -INFINITY, l);  // (past the end: no address is formed beyond the row)
                                 const float top = fmaxf(fmaxf(fmaxf(l[0], l[1]), fmaxf(l[2], l[3])), fmaxf(fmaxf(l[4], l[5]), fmaxf(l[6], l[7])));
                                 if (top > x.m) {
                                     x.s *= ex2((x.m - top) * chi);
                                     x.m = top;
                                     x.v = (int)(j * 8);
                                 }
                                 const float m = x.m == -INFINITY ? 0.0f : x.m;
                                 const uint32_t hit = out_of(j);
                                 float s = 0.0f;
#pragma unroll
                                 for (int e = 0; e < 8; ++e) {
                                     const float w = ex2((l[e] - m) * chi);
                                     s += (hit >> e) & 1u ? 0.0f : w;
                                 }
                                 x.s += s;
                             }
                         },
                         [&](VfPart& x, const VfPart& y) {
                             const float top = fmaxf(x.m, y.m);
                             const float fx = x.m == -INFINITY ? 0.0f : ex2((x.m - top) * chi), fy = y.m == -INFINITY ? 0.0f : ex2((y.m - top) * chi);
                             const float sx = x.s * fx, sy = y.s * fy;
                             x.s = __fadd_rn(sx, sy);
                             if (y.m > x.m || (y.m == x.m && y.v < x.v)) x.v = y.v;
                             x.m = top;
                         });
        const float top = z.m;
        auto weight = [&](float l) { return ex2((l - top) * chi); };
        // ---- what is left when each child is tried, if the ones before it were rejected (drafts without probabilities) ----
        float w[2], left[2] = {1.0f, 1.0f};
#pragma unroll
        for (int e = 0; e < 2; ++e) w[e] = kid[e] ? weight(lx[e]) : 0.0f;
        float Z = z.s;
        if (leave) {
            for (uint64_t rest = kids; rest;) {
                const int n = 63 - __clzll((long long)rest);
                rest ^= 1ull << n;
                const float lo = __shfl_sync(0xffffffffu, dup[0] ? 0.0f : w[0], n & 31), hi = __shfl_sync(0xffffffffu, dup[1] ? 0.0f : w[1], n & 31);
                Z += n & 32 ? hi : lo;
                if (n == lane) left[0] = Z;
                if (n == lane + 32) left[1] = Z;
            }
        }
        if (!(Z > 0.0f && Z < INFINITY)) {  // a NaN, an infinity, or no token at all
            bad |= RK_STATUS_RANGE;
            break;
        }
        const float lnZ = logf(Z), inv = 1.0f / Z;
        auto logp = [&](float l) { return (l - top) / scale - lnZ; };
        if (n_acc == 0 && writes && lane == 0) a.path[node0] = 0;
        const int here = n_acc++;
        int best = z.v;  // the first token of the chunk that has the maximum
        if (greedy) {
            const bool hit = lane < 8 && best + lane < V && logit(min(best + lane, V - 1)) == top;
            best += __ffs(__ballot_sync(0xffffffffu, hit)) - 1;
        }
        // ---- the children in order ----
        int took = -1;
        float aq = 0.0f, S = 1.0f;
        if (!probs || greedy) {
            bool yes[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) yes[e] = kid[e] && (greedy ? tok[e] == best : !dup[e] && coin[e] * left[e] < w[e]);
            const uint64_t hit = ballot(yes[0], yes[1]);
            if (hit) took = __ffsll((long long)hit) - 1;
        } else {
            for (uint64_t rest = kids; rest && took < 0 && !bad;) {
                const int n = __ffsll((long long)rest) - 1;
                rest &= rest - 1;
                bool yes[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) yes[e] = lane + 32 * e == n && coin[e] * qx[e] * S < fmaxf(fmaf(w[e], inv, -aq * qx[e]), 0.0f);
                if (ballot(yes[0], yes[1])) {
                    took = n;
                    break;
                }
                aq += S;
                if (!rest) break;
                const VfPart y = sweep({0.0f, 0.0f, 0, 0},
                                       [&](int vw, VfPart& x) {
#pragma unroll 2
                                           for (unsigned j0 = vw * 32; j0 < chunks; j0 += VF_WARPS * 32) {
                                               float l[8], d[8];
                                               load8<F32>(row, j0 + lane, V, -INFINITY, l);
                                               load8<true>(q, j0 + lane, V, 0.0f, d);
                                               float s = 0.0f;
#pragma unroll
                                               for (int e = 0; e < 8; ++e) {
                                                   const float r = fmaf(weight(l[e]), inv, -aq * d[e]);
                                                   s += fmaf(r, 0.0f, fmaxf(r, 0.0f));  // NaN where q is none or infinite
                                               }
                                               x.s += s;
                                           }
                                       },
                                       join_sum);
                S = y.s;
                if (!(S >= 0.0f)) bad |= RK_STATUS_RANGE;
            }
            if (bad) break;
        }
        if (took >= 0) {
            if (leave && warp == 0) {  // the bits of these children go (the pass that read them lies behind a barrier)
                for (int e = 0; e < 2; ++e)
                    if (kid[e]) sh.child[(tok[e] / 8 % VF_BITS) / 32] = 0;
            }
            const int x = of(tok, took);
            const float lo = __shfl_sync(0xffffffffu, lx[0], took & 31), hi = __shfl_sync(0xffffffffu, lx[1], took & 31);
            if (writes && lane == 0) {
                a.tokens[node0 + here] = x;
                a.logprobs[node0 + here] = logp(took & 32 ? hi : lo);
                a.path[node0 + here + 1] = took;
            }
            at = took;
            continue;
        }
        // ---- the last token: of what is left, or of p where that is nothing ----
        int last = best;
        for (int all = 0; !greedy && all < 2; ++all) {
            const VfPart y = sweep({-1.0f, 0.0f, INT32_MAX, 0},
                                   [&](int vw, VfPart& x) {
#pragma unroll 2
                                       for (unsigned j0 = vw * 32; j0 < chunks; j0 += VF_WARPS * 32) {
                                           const unsigned j = j0 + lane;
                                           float l[8], r[8], d[8];
                                           load8<F32>(row, j, V, -INFINITY, l);
                                           load8<true>(race, j, V, 1.0f, r);
                                           const bool minus = probs && !all && aq > 0.0f;
                                           if (minus) load8<true>(q, j, V, 0.0f, d);
                                           const uint32_t hit = all ? 0u : out_of(j);
#pragma unroll
                                           for (int e = 0; e < 8; ++e) {
                                               float k = weight(l[e]);
                                               if (minus) {
                                                   k = fmaf(k, inv, -aq * d[e]);
                                                   if (!(fabsf(k) < INFINITY)) x.bad = 1;
                                               }
                                               if ((hit >> e) & 1u) k = 0.0f;
                                               if (k > 0.0f) {
                                                   k = __fdividef(k, r[e]);
                                                   if (k > x.m) {
                                                       x.m = k;
                                                       x.v = (int)(j * 8) + e;
                                                   }
                                               }
                                           }
                                       }
                                   },
                                   join_max);
            if (y.bad) bad |= RK_STATUS_RANGE;
            if (y.v < V || bad) {
                last = y.v;
                break;
            }
        }
        if (bad) break;
        if (last >= V || last < 0) last = best;
        if (writes && lane == 0) {
            a.tokens[node0 + here] = last;
            a.logprobs[node0 + here] = logp(logit(last));
        }
        break;
    }
    if (writes) {
        if (bad && lane == 0 && a.status) atomicOr(a.status, bad);
        const int n = bad || rootless ? 0 : n_acc;
        for (int i = n + lane; i < T; i += 32) {
            a.path[node0 + i] = -1;
            a.tokens[node0 + i] = -1;
            a.logprobs[node0 + i] = bad ? NAN : 0.0f;
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
        if ((e = cudaFuncSetAttribute(verify_kernel<false>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1)) != cudaSuccess) return e;
        if ((e = cudaFuncSetAttribute(verify_kernel<true>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1)) != cudaSuccess) return e;
        configured.fetch_or(bit);
    }
    VerifyArgs r = a;
    r.cluster = 16;
    while (r.cluster > 1 && (long long)a.B * r.cluster > 304) r.cluster /= 2;
    r.prefetch_nodes = (double)a.B * a.T * a.V * (a.f32 ? 4 : 2) <= 16e6;
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
    return a.f32 ? cudaLaunchKernelEx(&cfg, verify_kernel<true>, r) : cudaLaunchKernelEx(&cfg, verify_kernel<false>, r);
}

}  // namespace rk
