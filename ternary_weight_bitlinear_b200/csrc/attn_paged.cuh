// attn_paged.cuh -- attention of the new rows of a batch over the paged
// key/value cache (kvcache.cuh has the batch's description).
//
//   out[r, h] = sum_j p_j v_j,  p = softmax_j(scale q[r, h] . k_j),
// j over the positions of r's sequence (up to r's own when causal), key/value
// head h / (H / H_kv).  A row that sees no position gets zeros.
#pragma once

#include <cuda_bf16.h>

#include "attn.cuh"
#include "common.cuh"
#include "kvcache.cuh"

namespace bl {

struct PagedAttnArgs {
    KvCacheArgs c;
    KvBatchArgs b;
    const uint16_t* q;   // bf16 [T, heads, D], rows q_stride apart
    uint16_t* out;       // bf16 [T, heads, D], rows o_stride apart
    int64_t q_stride, o_stride;
    int heads;
    int group;           // heads / kv_heads
    int causal;
    float qscale;        // scale * log2(e)
};

// One warp per (row, head); a lane holds D/32 dimensions of the query and of
// the running output, and every position costs one dot product over the warp.
template <int D, bool I8>
__global__ void __launch_bounds__(128) attn_paged_row_kernel(const PagedAttnArgs a) {
    constexpr int DL = D / 32;
    const int lane = threadIdx.x & 31;
    const int64_t w = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    pdl_wait();
    pdl_launch_dependents();
    if (w >= (int64_t)a.b.T * a.heads) return;
    const int t = (int)(w / a.heads), h = (int)(w % a.heads), g = h / a.group;
    const int b = kv_seq_of_row(a.b, t, lane);
    if (b >= a.b.batch) return;
    const KvSeq s = kv_seq(a.b, b);
    if (t < s.q0) return;
    const int end = a.causal ? min(s.len, s.len - s.n + (t - s.q0) + 1) : s.len;
    float q[DL], o[DL], m = -INFINITY, l = 0.0f;
#pragma unroll
    for (int e = 0; e < DL; ++e) {
        q[e] = bf16_bits_to_float(__ldcg(a.q + t * a.q_stride + h * D + lane * DL + e)) * a.qscale;
        o[e] = 0.0f;
    }
    for (int j = 0; j < end; ++j) {
        const int page = kv_page(a.c, a.b, b, j), slot = j % a.c.page_size;
        if (page < 0) continue;
        const int64_t off = page * a.c.sp + slot * a.c.ss + g * a.c.sh + lane * DL;
        const int64_t so = ((int64_t)page * a.c.kv_heads + g) * a.c.page_size + slot;
        float x = 0.0f, v[DL];
#pragma unroll
        for (int e = 0; e < DL; ++e) {
            float kk;
            if constexpr (I8) {
                kk = (float)__ldcg(static_cast<const int8_t*>(a.c.k) + off + e) * __ldcg(a.c.k_step + so);
                v[e] = (float)__ldcg(static_cast<const int8_t*>(a.c.v) + off + e) * __ldcg(a.c.v_step + so);
            } else {
                kk = bf16_bits_to_float(__ldcg(static_cast<const uint16_t*>(a.c.k) + off + e));
                v[e] = bf16_bits_to_float(__ldcg(static_cast<const uint16_t*>(a.c.v) + off + e));
            }
            x = fmaf(q[e], kk, x);
        }
        x = warp_sum_f(x);
        const float mn = fmaxf(m, x);
        const float alpha = mn == -INFINITY ? 1.0f : exp2f(m - mn), p = exp2f(x - mn);
        l = fmaf(l, alpha, p);
#pragma unroll
        for (int e = 0; e < DL; ++e) o[e] = fmaf(o[e], alpha, p * v[e]);
        m = mn;
    }
#pragma unroll
    for (int e = 0; e < DL; ++e)
        a.out[t * a.o_stride + h * D + lane * DL + e] = float_to_bf16_bits(end > 0 ? o[e] / l : 0.0f);
}

}  // namespace bl
