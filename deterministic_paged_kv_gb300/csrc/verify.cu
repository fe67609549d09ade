// verify.cu -- the walk down a row's tree of drafted tokens: which nodes the target's
// distribution accepts, the token behind them, and the tokens' log-probabilities.
//
// Mathematics.  With w(v) = e^((l(v) - max l) / temperature) and Z = sum w, p = w / Z.  After
// rejections the residual r is, up to a factor, (p - a q)+ for one number a: a starts at 0, and a
// rejection adds S(a) = sum (p - a q)+ to it, since with r = (p - a q)+ and S = sum r
//   (r - S q)+ = (p - a q - S q)+      (where r = 0, p - (a + S) q <= 0 as well)
// so a node's state is a number, and each further child one pass over p and q.  Drafts without
// probabilities: the residual is p without the children's tokens, so one pass that leaves them out
// gives what remains for every child (their own weights are added back one by one: sums of positive
// numbers, nothing cancels).  The last token is argmax r(v) / race(v): of independent exponential
// draws of rates r(v) the first to ring, which has the distribution r; unlike an inverse of the
// cumulative sum it does not depend on an order of summation.
#include "rk_device.cuh"
#include "tree_args.h"

namespace rk {

namespace {

constexpr int VF_THREADS = 512;

struct VfCtl {
    int32_t parent[TREE_MAX], token[TREE_MAX];
    float coin[TREE_MAX];
    int32_t path[TREE_MAX], out[TREE_MAX];
    float logp[TREE_MAX];
    float red[VF_THREADS / 32];
    int redi[VF_THREADS / 32];
};

__device__ __forceinline__ float logit_at(const VerifyArgs& a, size_t row, int v) {
    if (a.f32) return reinterpret_cast<const float*>(a.logits)[row * a.V + v];
    return __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(a.logits)[row * a.V + v]);
}

// e^((x - top) / temperature), c = log2(e) / temperature in two parts.  NaN for a NaN, for x = top =
// -inf, and for x = +inf.
__device__ __forceinline__ float weight(float x, float top, float chi, float clo) {
    const float d = x - top, e = d * chi;
    return e <= -150.0f ? 0.0f : ex2(fmaf(d, chi, d * clo));
}

__device__ float block_sum(float x, VfCtl* c) {
#pragma unroll
    for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) c->red[threadIdx.x >> 5] = x;
    __syncthreads();
    float s = 0.0f;
    for (int i = 0; i < VF_THREADS / 32; ++i) s += c->red[i];
    return s;
}
// The largest key and the lowest index of equal ones (index INT_MAX: none).
__device__ int block_argmax(float& key, int idx, VfCtl* c) {
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        const float k = __shfl_xor_sync(0xffffffffu, key, o);
        const int i = __shfl_xor_sync(0xffffffffu, idx, o);
        if (k > key || (k == key && i < idx)) {
            key = k;
            idx = i;
        }
    }
    __syncthreads();
    if ((threadIdx.x & 31) == 0) {
        c->red[threadIdx.x >> 5] = key;
        c->redi[threadIdx.x >> 5] = idx;
    }
    __syncthreads();
    key = c->red[0];
    idx = c->redi[0];
    for (int w = 1; w < VF_THREADS / 32; ++w)
        if (c->red[w] > key || (c->red[w] == key && c->redi[w] < idx)) {
            key = c->red[w];
            idx = c->redi[w];
        }
    return idx;
}

__global__ void __launch_bounds__(VF_THREADS) verify_kernel(const __grid_constant__ VerifyArgs a) {
    __shared__ VfCtl c;
    const int b = blockIdx.x, tid = threadIdx.x, T = a.T, V = a.V;
    const size_t node0 = (size_t)b * T;
    const float temp = a.temperature[b];
    const bool greedy = temp == 0.0f;
    int bad = !(temp == 0.0f || (temp >= 5.421010862427522e-20f && temp < INFINITY)) ? RK_STATUS_RANGE : 0;
    if (tid < T) {
        c.parent[tid] = a.parents[node0 + tid];
        c.token[tid] = a.draft_tokens[node0 + tid];
        c.coin[tid] = a.coins[node0 + tid];
        c.path[tid] = -1;
        c.out[tid] = -1;
        c.logp[tid] = 0.0f;
    }
    __syncthreads();
    int tree = 0;
    if (tid < T) {
        const int p = c.parent[tid];
        tree = p < TREE_UNUSED || p >= tid || (p >= 0 && c.parent[p] == TREE_UNUSED);
        if (tid > 0 && p != TREE_UNUSED && (c.token[tid] < 0 || c.token[tid] >= V)) tree = 1;
    }
    if (__syncthreads_or(tree)) bad |= RK_STATUS_TREE;
    const bool rootless = !bad && c.parent[0] == TREE_UNUSED;
    int at = 0, n_acc = 0;
    const float scale = greedy ? 1.0f : temp;
    const double cl = 1.4426950408889634074 / (double)scale;
    const float chi = (float)cl, clo = (float)(cl - (double)chi);
    while (!bad && !rootless) {
        const size_t row = node0 + at;
        float top = -INFINITY;
        int best = INT32_MAX;
        for (int v = tid; v < V; v += VF_THREADS) {
            const float x = logit_at(a, row, v);
            if (x > top || best == INT32_MAX) {
                top = x;
                best = v;
            }
        }
        best = block_argmax(top, best, &c);
        float z = 0.0f;
        for (int v = tid; v < V; v += VF_THREADS) z += weight(logit_at(a, row, v), top, chi, clo);
        const float Z = block_sum(z, &c);
        if (!(Z > 0.0f && Z < INFINITY)) {
            bad |= RK_STATUS_RANGE;
            break;
        }
        const float lnZ = logf(Z);
        auto logp = [&](int v) { return (logit_at(a, row, v) - top) / scale - lnZ; };
        if (n_acc == 0) c.path[0] = 0;
        const int here = n_acc++;
        int took = -1;
        float aq = 0.0f, S = 1.0f;
        // what is left of Z without the children's tokens
        float rest = 0.0f;
        if (!greedy && !a.draft_probs) {
            for (int v = tid; v < V; v += VF_THREADS) {
                bool out = false;
                for (int n = at + 1; n < T; ++n) out |= c.parent[n] == at && c.token[n] == v;
                if (!out) rest += weight(logit_at(a, row, v), top, chi, clo);
            }
            rest = block_sum(rest, &c);
        }
        for (int n = at + 1; n < T && took < 0; ++n) {
            if (c.parent[n] != at) continue;
            const int x = c.token[n];
            if (greedy) {
                if (x == best) took = n;
                continue;
            }
            const float w = weight(logit_at(a, row, x), top, chi, clo);
            if (!a.draft_probs) {
                bool gone = false;
                float left = rest;
                for (int m = T - 1; m > at; --m) {  // tokens of the children that are not tried yet, each once
                    if (c.parent[m] != at) continue;
                    bool first = true;
                    for (int k = at + 1; k < m; ++k) first &= !(c.parent[k] == at && c.token[k] == c.token[m]);
                    if (m < n && c.token[m] == x) gone = true;
                    if (m >= n && first) left += weight(logit_at(a, row, c.token[m]), top, chi, clo);
                }
                if (!gone && c.coin[n] * left < w) took = n;
            } else {
                const float* q = a.draft_probs + row * V;
                const float qx = q[x];
                if (c.coin[n] * qx * S < fmaxf(w / Z - aq * qx, 0.0f)) {
                    took = n;
                    continue;
                }
                aq += S;
                float s = 0.0f;
                for (int v = tid; v < V; v += VF_THREADS) {
                    const float qv = q[v];
                    const float r = weight(logit_at(a, row, v), top, chi, clo) / Z - aq * qv;
                    s += qv < INFINITY ? fmaxf(r, 0.0f) : NAN;
                }
                S = block_sum(s, &c);
                if (!(S >= 0.0f)) bad |= RK_STATUS_RANGE;
            }
        }
        if (bad) break;
        if (took >= 0) {
            if (tid == 0) {
                c.out[here] = c.token[took];
                c.logp[here] = logp(c.token[took]);
                c.path[here + 1] = took;
            }
            at = took;
            continue;
        }
        // the last token
        int last = best;
        if (!greedy) {
            for (int pass = 0; pass < 2; ++pass) {  // the second where nothing is left
                float key = -1.0f;
                int idx = INT32_MAX;
                for (int v = tid; v < V; v += VF_THREADS) {
                    float r = weight(logit_at(a, row, v), top, chi, clo);
                    if (pass == 0 && a.draft_probs) {
                        r = r / Z - aq * (aq > 0.0f ? a.draft_probs[row * V + v] : 0.0f);
                    } else if (pass == 0) {
                        for (int n = at + 1; n < T; ++n)
                            if (c.parent[n] == at && c.token[n] == v) r = 0.0f;
                    }
                    if (r > 0.0f) {
                        const float k = r / a.race[(size_t)b * V + v];
                        if (k > key) {
                            key = k;
                            idx = v;
                        }
                    }
                }
                last = block_argmax(key, idx, &c);
                if (last < V) break;
            }
            if (last >= V) last = best;
        }
        if (tid == 0) {
            c.out[here] = last;
            c.logp[here] = logp(last);
        }
        break;
    }
    __syncthreads();
    if (bad && tid == 0 && a.status) atomicOr(a.status, bad);
    if (tid < T) {
        a.path[node0 + tid] = bad ? -1 : c.path[tid];
        a.tokens[node0 + tid] = bad ? -1 : c.out[tid];
        a.logprobs[node0 + tid] = bad ? NAN : c.logp[tid];
    }
    if (tid == 0) {
        a.n_accepted[b] = bad ? 0 : n_acc;
        a.n_drop[b] = rootless ? 0 : T - (bad ? 0 : n_acc);
    }
}

}  // namespace

cudaError_t launch_verify(const VerifyArgs& a, cudaStream_t stream) {
    verify_kernel<<<(unsigned)a.B, VF_THREADS, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace rk
