// attn_q8.cu -- causal attention over the 8-bit page cache, one block per query
// and query head: the simplest kernel that serves every case.  Keys in chunks
// of 128, one key's score per thread, one pass with the running maximum and
// sum, then one output dimension per thread.
#include "q8_device.cuh"

namespace rk {

namespace {

__global__ void __launch_bounds__(128) attn_q8_kernel(const __grid_constant__ AttnQ8Args a) {
    __shared__ float qs[HEAD_DIM], ps[128], red[4];
    __shared__ int pg[8];
    __shared__ int s_bad;  // status bits of the block
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const long long id = blockIdx.x;
    const int s = (int)(id % a.Sq), hq = (int)(id / a.Sq % a.Hq), b = (int)(id / a.Sq / a.Hq);
    const int hk = hq / a.G;
    const size_t row = ((size_t)b * a.Hq + hq) * a.Sq + s;
    __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(a.out) + row * HEAD_DIM;
    const int kv_len = a.kv_lens[b], pos = a.position_ids[(size_t)b * a.Sq + s];
    if (tid == 0) s_bad = 0;
    __syncthreads();
    int bad = (kv_len < 0 || kv_len > a.W * PAGE) ? RK_STATUS_KVLEN : 0;
    if (pos < 0) bad |= RK_STATUS_POSITION;
    const int n = bad ? 0 : min(kv_len, pos + 1);
    if (n > 0 && tid < 64) {
        const __nv_bfloat16* q = reinterpret_cast<const __nv_bfloat16*>(a.q) + row * HEAD_DIM;
        const float lo = __bfloat162float(q[tid]), hi = __bfloat162float(q[tid + 64]);
        if (!(fabsf(lo) < 18446744073709551616.0f) || !(fabsf(hi) < 18446744073709551616.0f)) bad |= RK_STATUS_RANGE;
        float c, sn;
        rope_cos_sin((uint32_t)max(pos, 0), a.rope_turns[tid], c, sn);
        qs[tid] = lo * c - hi * sn;
        qs[tid + 64] = hi * c + lo * sn;
    }
    float m = -INFINITY, l = 0.0f, o = 0.0f;
    for (int t0 = 0; t0 < n; t0 += 128) {
        const int t = t0 + tid;
        __syncthreads();
        if (tid < 8) pg[tid] = t0 + tid * PAGE < n ? a.block_table[(size_t)b * a.W + t0 / PAGE + tid] : 0;
        __syncthreads();
        float x = -INFINITY;
        if (t < n) {
            const int page = pg[tid / PAGE];
            if (page < 0 || page >= a.num_pages) {
                bad |= RK_STATUS_PAGE_OOB;
            } else {
                const size_t block = (size_t)page * a.Hkv + hk;
                const float ks = a.k_scale[block], vs = a.v_scale[block];
                if (!(ks >= 1.17549435e-38f && ks < INFINITY && vs >= 1.17549435e-38f && vs < INFINITY)) bad |= RK_STATUS_SCALE;
                else {
                const uint4* kc = reinterpret_cast<const uint4*>(a.k_cache + block * Q8_BLOCK_BYTES + (t % PAGE) * HEAD_DIM);
                float acc = 0.0f;
                for (int c = 0; c < 8; ++c) {
                    const uint4 w = kc[c];
                    const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float2 p0 = e4m3x2_to_float2(ww[e]), p1 = e4m3x2_to_float2(ww[e] >> 16);
                        const float* qq = qs + c * 16 + e * 4;
                        acc += qq[0] * p0.x + qq[1] * p0.y + qq[2] * p1.x + qq[3] * p1.y;
                    }
                }
                x = acc * ks * a.qk_scale_log2;
                if (!(fabsf(x) < INFINITY)) bad |= RK_STATUS_RANGE;
                }
            }
        }
        float mt = x;
        for (int k = 16; k; k >>= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, k));
        if (lane == 0) red[warp] = mt;
        if (bad) atomicOr(&s_bad, bad);
        __syncthreads();
        bad = s_bad;
        if (bad) break;
        mt = fmaxf(fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])), m);
        const float alpha = ex2(m - mt);
        m = mt;
        ps[tid] = ex2(x - m);
        __syncthreads();
        l *= alpha;
        o *= alpha;
        const int cnt = min(128, n - t0);
        for (int j = 0; j < cnt; ++j) {
            const size_t block = (size_t)pg[j / PAGE] * a.Hkv + hk;
            const uint16_t c = a.v_cache[block * Q8_BLOCK_BYTES + (j % PAGE) * HEAD_DIM + tid];
            const float p = ps[j];
            l += p;
            o += p * (e4m3x2_to_float2(c).x * a.v_scale[block]);
        }
    }
    if (n > 0 && !(fabsf(o) < INFINITY)) bad |= RK_STATUS_RANGE;
    if (bad) atomicOr(&s_bad, bad);
    __syncthreads();
    if (s_bad) {
        if (tid == 0 && a.status) atomicOr(a.status, s_bad);
        if (tid == 0) a.lse[row] = __int_as_float(0x7fc00000);
        out[tid] = __float2bfloat16(0.0f);
        return;
    }
    out[tid] = __float2bfloat16(n > 0 ? o / l : 0.0f);
    if (tid == 0) a.lse[row] = n > 0 ? (m + log2f(l)) * 0.693147180559945309f : -INFINITY;
}

}  // namespace

cudaError_t launch_attn_q8(const AttnQ8Args& a, cudaStream_t stream) {
    const long long blocks = (long long)a.B * a.Hq * a.Sq;
    if (blocks <= 0) return cudaSuccess;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    attn_q8_kernel<<<(unsigned)blocks, 128, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace rk
