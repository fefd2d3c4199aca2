// attn_paged_simple.cuh - attention of new tokens over a paged cache, in its
// plainest form: one block per query row, fp32 throughout.
#pragma once
#include <cuda_bf16.h>
#include <math_constants.h>

#include <cstdint>

namespace attn_sm100 {

struct PagedSimpleParams {
    const __nv_bfloat16 *q;               // [B, H, T, dk]
    const __nv_bfloat16 *k, *v;           // pages
    int64_t page_stride, head_stride, token_stride;
    const int *table, *lens;
    __nv_bfloat16 *o;                     // [B, H, T, dv]
    float *lse;                           // [B, H, T]
    int H, Hkv, T, num_pages, page_size, max_pages, window, dk, dv;
    float scale;
};

constexpr int SIMPLE_THREADS = 256;

__global__ void __launch_bounds__(SIMPLE_THREADS) attn_paged_simple_kernel(const PagedSimpleParams p)
{
    __shared__ float qs[1024], prob[SIMPLE_THREADS], red[SIMPLE_THREADS / 32];
    __shared__ int64_t where[SIMPLE_THREADS];
    const int row = blockIdx.x, u = row % p.T, h = (row / p.T) % p.H, b = row / p.T / p.H;
    const int tid = threadIdx.x;
    const int64_t cap = static_cast<int64_t>(p.max_pages) * p.page_size;
    const int len = static_cast<int>(min(static_cast<int64_t>(max(p.lens[b], 0)), cap));
    const int last = len - p.T + u;
    const int first = p.window >= 0 ? max(0, last - p.window) : 0;
    const int64_t head = (h / (p.H / p.Hkv)) * p.head_stride;
    for (int i = tid; i < p.dk; i += SIMPLE_THREADS) qs[i] = __bfloat162float(p.q[static_cast<int64_t>(row) * p.dk + i]);
    float m = -CUDART_INF_F, l = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
    for (int base = first; base <= last; base += SIMPLE_THREADS) {
        __syncthreads();
        const int at = base + tid;
        float s = -CUDART_INF_F;
        int64_t src = -1;
        if (at <= last) {
            const int page = p.table[static_cast<int64_t>(b) * p.max_pages + at / p.page_size];
            if (static_cast<unsigned>(page) < static_cast<unsigned>(p.num_pages)) {
                src = page * p.page_stride + head + (at % p.page_size) * p.token_stride;
                float d = 0.f;
                for (int i = 0; i < p.dk; ++i) d = fmaf(qs[i], __bfloat162float(p.k[src + i]), d);
                s = d * p.scale;
            }
        }
        where[tid] = src;
        float mx = s;
        for (int o = 16; o >= 1; o /= 2) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        if (tid % 32 == 0) red[tid / 32] = mx;
        __syncthreads();
        float m_new = m;
        for (int w = 0; w < SIMPLE_THREADS / 32; ++w) m_new = fmaxf(m_new, red[w]);
        const float ref = m_new == -CUDART_INF_F ? 0.f : m_new;
        const float alpha = expf(m - ref);
        const float e = src >= 0 ? expf(s - ref) : 0.f;
        prob[tid] = e;
        __syncthreads();
        l *= alpha;
        for (int j = 0; j < SIMPLE_THREADS; ++j) l += prob[j];
        for (int i = 0; i < 4; ++i) {
            const int c = tid + i * SIMPLE_THREADS;
            if (c >= p.dv) break;
            acc[i] *= alpha;
            for (int j = 0; j < SIMPLE_THREADS; ++j)
                if (where[j] >= 0) acc[i] = fmaf(prob[j], __bfloat162float(p.v[where[j] + c]), acc[i]);
        }
        m = m_new;
    }
    for (int i = 0; i < 4; ++i) {
        const int c = tid + i * SIMPLE_THREADS;
        if (c < p.dv) p.o[static_cast<int64_t>(row) * p.dv + c] = __float2bfloat16_rn(l > 0.f ? acc[i] / l : 0.f);
    }
    if (tid == 0) p.lse[row] = l > 0.f ? m + logf(l) : -CUDART_INF_F;
}

}  // namespace attn_sm100
