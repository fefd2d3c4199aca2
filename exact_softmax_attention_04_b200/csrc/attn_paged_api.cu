// attn_paged_api.cu - host side of attention over a paged cache: argument
// checks, workspace layout, launches. Contracts in include/attn.h.
#include <cuda.h>
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>

#include "attn.h"
#include "attn_host.h"
#include "attn_paged_simple.cuh"

namespace {

using namespace attn_host;

// What both forms ask of the cache's shape.
int check_cache(int B, int T, int num_pages, int page_size, int max_pages, float scale)
{
    if (B <= 0 || T <= 0 || num_pages <= 0 || page_size <= 0 || max_pages <= 0) return ATTN_ERR_INVALID;
    if (!std::isfinite(scale) || !(scale > 0.f)) return ATTN_ERR_INVALID;
    // a tile of the kernels is a whole number of pages, or lies inside one
    if (page_size < 8 || (page_size & (page_size - 1)) != 0) return ATTN_ERR_UNSUPPORTED;
    // positions are 32-bit
    if (static_cast<int64_t>(max_pages) * page_size > (1 << 30)) return ATTN_ERR_UNSUPPORTED;
    return ATTN_OK;
}

int check_paged(int B, int H, int Hkv, int T, int num_pages, int page_size, int max_pages, int d, float scale)
{
    const int rc = check_cache(B, T, num_pages, page_size, max_pages, scale);
    if (rc != ATTN_OK) return rc;
    if (H <= 0 || Hkv <= 0 || d <= 0 || H % Hkv != 0) return ATTN_ERR_INVALID;
    if (d != 64 && d != 128) return ATTN_ERR_UNSUPPORTED;
    if (static_cast<int64_t>(B) * H > INT_MAX / T / d) return ATTN_ERR_UNSUPPORTED;
    if (static_cast<int64_t>(H / Hkv) * T > 256) return ATTN_ERR_UNSUPPORTED;
    return ATTN_OK;
}

int check_latent(int B, int H, int T, int num_pages, int page_size, int max_pages, int rank, float scale)
{
    const int rc = check_cache(B, T, num_pages, page_size, max_pages, scale);
    if (rc != ATTN_OK) return rc;
    if (H <= 0 || rank <= 0) return ATTN_ERR_INVALID;
    if (rank != 256 && rank != 512) return ATTN_ERR_UNSUPPORTED;
    if (static_cast<int64_t>(B) * H > INT_MAX / T / (rank + 64)) return ATTN_ERR_UNSUPPORTED;
    if (static_cast<int64_t>(H) * T > 1024) return ATTN_ERR_UNSUPPORTED;
    return ATTN_OK;
}

// Strides (page, head, token) in elements: positive multiples of 8, a row's
// length at least.
int take_strides(const int64_t *given, int64_t Hkv, int64_t page_size, int64_t d, int64_t out[3])
{
    const int64_t packed[3] = {Hkv * page_size * d, page_size * d, d};
    for (int i = 0; i < 3; ++i) {
        out[i] = given ? given[i] : packed[i];
        if (out[i] < d || out[i] % 8 != 0) return ATTN_ERR_INVALID;
    }
    return ATTN_OK;
}

int launch_simple(attn_sm100::PagedSimpleParams &p, int rows, cudaStream_t st)
{
    attn_sm100::attn_paged_simple_kernel<<<static_cast<unsigned>(rows), attn_sm100::SIMPLE_THREADS, 0, st>>>(p);
    return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

}  // namespace

extern "C" int64_t attn_decode_paged_workspace_bytes(int B, int H, int Hkv, int T, int max_pages, int page_size,
                                                     int d)
{
    if (check_paged(B, H, Hkv, T, 1, page_size, max_pages, d, 1.f) != ATTN_OK) return -1;
    return 16;
}

extern "C" int attn_decode_paged(const void *q, const void *k_pages, const void *v_pages, const int64_t *kv_strides,
                                 const int *page_table, const int *lens, void *o, float *lse, void *workspace,
                                 size_t workspace_bytes, int B, int H, int Hkv, int T, int num_pages, int page_size,
                                 int max_pages, int window, int d, float scale, void *stream)
{
    if (!q || !k_pages || !v_pages || !page_table || !lens || !o || !lse || !workspace) return ATTN_ERR_INVALID;
    const int rc = check_paged(B, H, Hkv, T, num_pages, page_size, max_pages, d, scale);
    if (rc != ATTN_OK) return rc;
    for (const void *ptr : {q, k_pages, v_pages, static_cast<const void *>(o), static_cast<const void *>(workspace)})
        if (!aligned(ptr, 16)) return ATTN_ERR_INVALID;
    if (!aligned(page_table, 4) || !aligned(lens, 4) || !aligned(lse, 4)) return ATTN_ERR_INVALID;
    int64_t s[3];
    if (take_strides(kv_strides, Hkv, page_size, d, s) != ATTN_OK) return ATTN_ERR_INVALID;
    if (workspace_bytes < 16) return ATTN_ERR_INVALID;
    attn_sm100::PagedSimpleParams p = {
        static_cast<const __nv_bfloat16 *>(q), static_cast<const __nv_bfloat16 *>(k_pages),
        static_cast<const __nv_bfloat16 *>(v_pages), s[0], s[1], s[2], page_table, lens,
        static_cast<__nv_bfloat16 *>(o), lse, H, Hkv, T, num_pages, page_size, max_pages, window, d, d, scale};
    return launch_simple(p, B * H * T, static_cast<cudaStream_t>(stream));
}

extern "C" int64_t attn_decode_latent_workspace_bytes(int B, int H, int T, int max_pages, int page_size, int rank)
{
    if (check_latent(B, H, T, 1, page_size, max_pages, rank, 1.f) != ATTN_OK) return -1;
    return 16;
}

extern "C" int attn_decode_latent(const void *q, const void *pages, const int64_t *strides, const int *page_table,
                                  const int *lens, void *o, float *lse, void *workspace, size_t workspace_bytes,
                                  int B, int H, int T, int num_pages, int page_size, int max_pages, int rank,
                                  float scale, void *stream)
{
    if (!q || !pages || !page_table || !lens || !o || !lse || !workspace) return ATTN_ERR_INVALID;
    const int rc = check_latent(B, H, T, num_pages, page_size, max_pages, rank, scale);
    if (rc != ATTN_OK) return rc;
    for (const void *ptr : {q, pages, static_cast<const void *>(o), static_cast<const void *>(workspace)})
        if (!aligned(ptr, 16)) return ATTN_ERR_INVALID;
    if (!aligned(page_table, 4) || !aligned(lens, 4) || !aligned(lse, 4)) return ATTN_ERR_INVALID;
    const int64_t given[3] = {strides ? strides[0] : 0, strides ? strides[0] : 0, strides ? strides[1] : 0};
    int64_t s[3];
    if (take_strides(strides ? given : nullptr, 1, page_size, rank + 64, s) != ATTN_OK) return ATTN_ERR_INVALID;
    if (workspace_bytes < 16) return ATTN_ERR_INVALID;
    attn_sm100::PagedSimpleParams p = {
        static_cast<const __nv_bfloat16 *>(q), static_cast<const __nv_bfloat16 *>(pages),
        static_cast<const __nv_bfloat16 *>(pages), s[0], s[1], s[2], page_table, lens,
        static_cast<__nv_bfloat16 *>(o), lse, H, 1, T, num_pages, page_size, max_pages, -1, rank + 64, rank, scale};
    return launch_simple(p, B * H * T, static_cast<cudaStream_t>(stream));
}
