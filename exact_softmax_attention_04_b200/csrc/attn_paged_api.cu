// attn_paged_api.cu - host side of attention over a paged cache: argument
// checks, workspace layout, launches. Contracts in include/attn.h.
#include <cuda.h>
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>
#include <mutex>

#include "attn.h"
#include "attn_host.h"
#include "attn_latent_kernel.cuh"
#include "attn_paged_kernel.cuh"

namespace {

using namespace attn_host;

// What both forms ask of the cache's shape.
int check_cache(int B, int T, int num_pages, int page_size, int max_pages, float scale)
{
    if (B <= 0 || T <= 0 || num_pages <= 0 || page_size <= 0 || max_pages <= 0) return ATTN_ERR_INVALID;
    if (!std::isfinite(scale) || !(scale > 0.f)) return ATTN_ERR_INVALID;
    // a tile of the kernels is a whole number of pages, or lies inside one
    if (page_size < 8 || (page_size & (page_size - 1)) != 0) return ATTN_ERR_UNSUPPORTED;
    // positions, and the tiles of all sequences, are counted in 32 bits
    const int64_t cap = static_cast<int64_t>(max_pages) * page_size;
    if (cap > (1 << 30) || cap > (int64_t(1) << 36) / B) return ATTN_ERR_UNSUPPORTED;
    return ATTN_OK;
}

int check_paged(int B, int H, int Hkv, int T, int num_pages, int page_size, int max_pages, int d, float scale)
{
    const int rc = check_cache(B, T, num_pages, page_size, max_pages, scale);
    if (rc != ATTN_OK) return rc;
    if (H <= 0 || Hkv <= 0 || d <= 0 || H % Hkv != 0) return ATTN_ERR_INVALID;
    if (d != 64 && d != 128) return ATTN_ERR_UNSUPPORTED;
    if (static_cast<int64_t>(B) * H > INT_MAX / T / d) return ATTN_ERR_UNSUPPORTED;
    if (static_cast<int64_t>(H / Hkv) * T > 256 || Hkv > 4096) return ATTN_ERR_UNSUPPORTED;
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

// ---------------------------------------------------------------- the split

constexpr int kSMs = 148;

// How the work is laid out on the device: `ranges` runs of tiles for each of
// `units` (heads or blocks of heads), and the workspace that takes.
struct Layout {
    int ranges, units;
    int64_t before, ml, o, bytes;  // workspace offsets
};

// Runs per unit: as many as one wave of resident blocks holds, or two or three
// waves where that evens out a poor fit by an eighth at least. (A wave more costs
// every SM a block's start and end: 11 sequences x 3 heads of 17,000 tokens at d 64
// take 37 us in three waves, which fit 0.7% better, and 31 in one. But 80 key/value
// heads of 32 columns, 2 sequences of 8000 tokens at d 128, take 211 us in one wave,
// which leaves 68 SMs idle, and 153 in two.) There are no more runs than tiles.
Layout make_layout(int B, int units, int64_t max_tiles, int resident, int nc, int dv)
{
    Layout l;
    l.units = units;
    int64_t best = 1, best_waves = (units + resident - 1) / resident;
    for (int64_t waves = 1; waves <= 3; ++waves) {
        const int64_t r = waves * resident / units < max_tiles ? waves * resident / units : max_tiles;
        if (r >= 1 && 8 * waves * best < 7 * best_waves * r) {
            best = r;
            best_waves = waves;
        }
    }
    l.ranges = static_cast<int>(best);
    const int64_t cols = static_cast<int64_t>(l.ranges) * units * 2 * nc;
    l.before = 0;
    l.ml = B > attn_sm100::COMBINE_SCAN ? (static_cast<int64_t>(B) * 4 + 4 + 15) / 16 * 16 : 0;
    l.o = l.ml + cols * 8;
    l.bytes = l.o + cols * dv * 4;
    return l;
}

template <int TK, int DV, int NC>
int launch_combine(attn_sm100::PagedCombine a, cudaStream_t st)
{
    // a block of 256 threads for each column while there are few, up to 16
    // columns a block where that still leaves two blocks an SM (13 sequences of
    // 2000 tokens x 3 heads x 32 columns at d 128: 15.5 us in all, with one block
    // an SM 15.8, with four 17.8; 23 latent sequences of 6000 x 16 heads of rank 256:
    // 25.7, with one 26.8; 128 sequences of 500 to 4000 x 8 heads at d 64: 33.0, with
    // one 31.1, with four 34.8)
    const int gt = a.H / a.Hkv * a.split.T, cols = gt < NC ? gt : NC;
    const int64_t rows = static_cast<int64_t>(a.split.B) * a.H * a.split.T;
    a.per_block = 1;
    while (a.per_block < 16 && a.per_block < cols && rows / (2 * a.per_block) >= 2 * kSMs) a.per_block *= 2;
    const int64_t blocks = static_cast<int64_t>(a.split.B) * a.Hkv * a.nblk * ((cols + a.per_block - 1) / a.per_block);
    // A row's columns over several blocks while there are few rows: more groups of
    // lanes then share its segments (one latent sequence of 60000 x 16 heads of
    // rank 512: 31.0 -> 22.8 us; keys and values of 131072 and 65500 tokens, 16
    // columns at d 128: 41.2 -> 40.2). More blocks cost more than they share: with
    // up to five an SM, 4 sequences of 2000 tokens x 28 heads of 128 go from 9.2 to
    // 11.1 us, 23 latent sequences of 6000 x 16 heads of rank 256 from 25.7 to 28.4.
    constexpr int DC = DV > 128 ? 128 : 32;
    auto launch = [&](auto *kernel, int dc) {
        return launch_behind(kernel, dim3(static_cast<unsigned>(blocks), static_cast<unsigned>(DV / dc)),
                             attn_sm100::COMBINE_THREADS, 0, st, a);
    };
    if (DV > 128 ? rows <= 2 * kSMs : rows * (DV / DC) <= 2 * kSMs)
        return launch(attn_sm100::attn_paged_combine_kernel<TK, DV, DC, NC>, DC);
    return launch(attn_sm100::attn_paged_combine_kernel<TK, DV, DV, NC>, DV);
}

// Rows of `cols` elements, boxes of 64 columns x `box_rows`.
bool encode_rows(PFN_cuTensorMapEncodeTiled_v12000 enc, CUtensorMap *m, const void *ptr, int64_t rows, int cols,
                 int box_rows)
{
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(cols) * 2};
    const cuuint32_t box[2] = {64, static_cast<cuuint32_t>(box_rows)};
    const cuuint32_t estr[2] = {1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(ptr), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A pool as [page][head][token][column], boxes of 64 columns x `box_rows`
// tokens. Strides (page, head, token) in elements.
bool encode_pool(PFN_cuTensorMapEncodeTiled_v12000 enc, CUtensorMap *m, const void *ptr, int64_t num_pages,
                 int heads, int page_size, int cols, const int64_t s[3], int box_rows)
{
    const cuuint64_t dims[4] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(page_size),
                                static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(num_pages)};
    const cuuint64_t strides[3] = {static_cast<cuuint64_t>(s[2]) * 2, static_cast<cuuint64_t>(s[1]) * 2,
                                   static_cast<cuuint64_t>(s[0]) * 2};
    const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(box_rows), 1, 1};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(ptr), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int log2_of(int x)
{
    int n = 0;
    while ((1 << n) < x) ++n;
    return n;
}

// -------------------------------------------------------- keys and values

// Columns a block handles: a group's G * T, rounded up.
int paged_columns(int gt) { return gt <= 4 ? 4 : gt <= 8 ? 8 : gt <= 16 ? 16 : 32; }

Layout paged_layout(int B, int H, int Hkv, int T, int max_pages, int page_size, int d)
{
    const int gt = H / Hkv * T, nc = paged_columns(gt);
    const int64_t cap = static_cast<int64_t>(max_pages) * page_size;
    const int64_t tiles = B * ((cap + attn_sm100::PAGED_TK - 1) / attn_sm100::PAGED_TK);
    return make_layout(B, Hkv * ((gt + nc - 1) / nc), tiles, kSMs * (nc == 32 ? 1 : 2), nc, d);
}

struct PagedCall {
    const void *q, *k, *v;
    int64_t s[3];
    attn_sm100::PagedParams p;
    Layout l;
    uint8_t *workspace;
    int dev, page_size;
    cudaStream_t st;
};

template <int D, int NC>
int launch_paged(PagedCall &a)
{
    using C = attn_sm100::PagedCfg<D, NC>;
    static bool set[kMaxDevices] = {};
    auto enc = encoder();
    if (!enc) return ATTN_ERR_CUDA;
    attn_sm100::PagedParams &p = a.p;
    CUtensorMap mq, mk, mv;
    const int rows = p.split.B * p.H * p.split.T, box = a.page_size < 128 ? a.page_size : 128;
    if (!encode_rows(enc, &mq, a.q, rows, D, C::N) ||
        !encode_pool(enc, &mk, a.k, p.pages.num_pages, p.Hkv, a.page_size, D, a.s, box) ||
        !encode_pool(enc, &mv, a.v, p.pages.num_pages, p.Hkv, a.page_size, D, a.s, box))
        return ATTN_ERR_CUDA;
    {
        std::lock_guard<std::mutex> lk(g_mu);
        if (!set[a.dev]) {
            if (cudaFuncSetAttribute(attn_sm100::attn_paged_kernel<D, NC>,
                                     cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES) != cudaSuccess)
                return ATTN_ERR_CUDA;
            set[a.dev] = true;
        }
    }
    p.nblk = a.l.units / p.Hkv;
    p.split.ranges = a.l.ranges;
    p.split.before = reinterpret_cast<int *>(a.workspace + a.l.before);
    p.part_ml = reinterpret_cast<float2 *>(a.workspace + a.l.ml);
    p.part_o = reinterpret_cast<float *>(a.workspace + a.l.o);
    const dim3 grid(static_cast<unsigned>(a.l.ranges), static_cast<unsigned>(a.l.units));
    if (launch_behind(attn_sm100::attn_paged_kernel<D, NC>, grid, C::THREADS, C::SMEM_BYTES, a.st, mq, mk,
                      mv, p) != ATTN_OK)
        return ATTN_ERR_CUDA;
    // a sequence of one tile is never split
    if (p.split.cap <= attn_sm100::PAGED_TK) return ATTN_OK;
    const attn_sm100::PagedCombine c = {p.split, p.part_o, p.part_ml, p.o, p.lse, p.H, p.Hkv, p.nblk, 1};
    return launch_combine<attn_sm100::PAGED_TK, D, NC>(c, a.st);
}

template <int D>
int launch_paged_nc(PagedCall &a, int nc)
{
    if (nc == 4) return launch_paged<D, 4>(a);
    if (nc == 8) return launch_paged<D, 8>(a);
    if (nc == 16) return launch_paged<D, 16>(a);
    return launch_paged<D, 32>(a);
}

// ---------------------------------------------------------- latent vectors

// Columns a block handles: the query rows H * T, rounded up.
int latent_columns(int gt) { return gt <= 16 ? 16 : gt <= 32 ? 32 : 64; }

Layout latent_layout(int B, int gt, int max_pages, int page_size, int rank)
{
    const int nc = latent_columns(gt);
    const int64_t cap = static_cast<int64_t>(max_pages) * page_size;
    const int64_t tiles = B * ((cap + attn_sm100::LATENT_TK - 1) / attn_sm100::LATENT_TK);
    return make_layout(B, (gt + nc - 1) / nc, tiles, kSMs, nc, rank);
}

struct LatentCall {
    const void *q, *pages;
    int64_t page_stride, token_stride;
    attn_sm100::LatentParams p;
    Layout l;
    uint8_t *workspace;
    int H, dev, page_size;
    cudaStream_t st;
};

// A pool as [page][8 tokens][64-column group][token of the 8][column]: boxes of
// a page's tokens (a tile's at most) and `boxes` column groups.
bool encode_latent(PFN_cuTensorMapEncodeTiled_v12000 enc, CUtensorMap *m, const LatentCall &a, int groups, int boxes)
{
    const cuuint64_t dims[5] = {64, 8, static_cast<cuuint64_t>(groups), static_cast<cuuint64_t>(a.page_size / 8),
                                static_cast<cuuint64_t>(a.p.pages.num_pages)};
    const cuuint64_t strides[4] = {static_cast<cuuint64_t>(a.token_stride) * 2, 128,
                                   static_cast<cuuint64_t>(a.token_stride) * 16,
                                   static_cast<cuuint64_t>(a.page_stride) * 2};
    const int rows = a.page_size < attn_sm100::LATENT_TK ? a.page_size : attn_sm100::LATENT_TK;
    const cuuint32_t box[5] = {64, 8, static_cast<cuuint32_t>(boxes), static_cast<cuuint32_t>(rows / 8), 1};
    const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void *>(a.pages), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int R, int NC>
int launch_latent(LatentCall &a)
{
    using C = attn_sm100::LatentCfg<R, NC>;
    static bool set[kMaxDevices] = {};
    auto enc = encoder();
    if (!enc) return ATTN_ERR_CUDA;
    attn_sm100::LatentParams &p = a.p;
    CUtensorMap mq, mc, ml;
    const int rows = p.split.B * p.GT;
    if (!encode_rows(enc, &mq, a.q, rows, R + 64, NC) || !encode_latent(enc, &mc, a, C::BOXES, 2) ||
        !encode_latent(enc, &ml, a, C::BOXES, 1))
        return ATTN_ERR_CUDA;
    {
        std::lock_guard<std::mutex> lk(g_mu);
        if (!set[a.dev]) {
            if (cudaFuncSetAttribute(attn_sm100::attn_latent_kernel<R, NC>,
                                     cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES) != cudaSuccess)
                return ATTN_ERR_CUDA;
            set[a.dev] = true;
        }
    }
    p.split.ranges = a.l.ranges;
    p.split.before = reinterpret_cast<int *>(a.workspace + a.l.before);
    p.part_ml = reinterpret_cast<float2 *>(a.workspace + a.l.ml);
    p.part_o = reinterpret_cast<float *>(a.workspace + a.l.o);
    const dim3 grid(static_cast<unsigned>(a.l.ranges), static_cast<unsigned>(a.l.units));
    if (launch_behind(attn_sm100::attn_latent_kernel<R, NC>, grid, C::THREADS, C::SMEM_BYTES, a.st, mq, mc, ml, p) !=
        ATTN_OK)
        return ATTN_ERR_CUDA;
    // a sequence of one tile is never split
    if (p.split.cap <= attn_sm100::LATENT_TK) return ATTN_OK;
    const attn_sm100::PagedCombine c = {p.split, p.part_o, p.part_ml, p.o, p.lse, a.H, 1, a.l.units, 1};
    return launch_combine<attn_sm100::LATENT_TK, R, NC>(c, a.st);
}

template <int R>
int launch_latent_nc(LatentCall &a, int nc)
{
    if (nc == 16) return launch_latent<R, 16>(a);
    if (nc == 32) return launch_latent<R, 32>(a);
    return launch_latent<R, 64>(a);
}

}  // namespace

extern "C" int64_t attn_decode_paged_workspace_bytes(int B, int H, int Hkv, int T, int max_pages, int page_size,
                                                     int d)
{
    if (check_paged(B, H, Hkv, T, 1, page_size, max_pages, d, 1.f) != ATTN_OK) return -1;
    return paged_layout(B, H, Hkv, T, max_pages, page_size, d).bytes;
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
    PagedCall a;
    a.l = paged_layout(B, H, Hkv, T, max_pages, page_size, d);
    if (workspace_bytes < static_cast<size_t>(a.l.bytes)) return ATTN_ERR_INVALID;
    if (current_device(&a.dev) != ATTN_OK) return ATTN_ERR_CUDA;
    attn_sm100::PagedParams &p = a.p;
    p.status = status_word(a.dev);
    if (!p.status) return ATTN_ERR_CUDA;
    a.q = q;
    a.k = k_pages;
    a.v = v_pages;
    for (int i = 0; i < 3; ++i) a.s[i] = s[i];
    a.workspace = static_cast<uint8_t *>(workspace);
    a.page_size = page_size;
    a.st = static_cast<cudaStream_t>(stream);
    // (a window past every position is none; kept small, it cannot overflow)
    p.split = {lens, B, T, max_pages * page_size, window < 0 || window >= (1 << 30) ? -1 : window, 0, nullptr};
    p.pages = {page_table, num_pages, max_pages, log2_of(page_size)};
    p.o = static_cast<__nv_bfloat16 *>(o);
    p.lse = lse;
    p.H = H;
    p.Hkv = Hkv;
    p.scale_log2 = scale * 1.4426950408889634f;
    const int nc = paged_columns(H / Hkv * T);
    return d == 64 ? launch_paged_nc<64>(a, nc) : launch_paged_nc<128>(a, nc);
}

extern "C" int64_t attn_decode_latent_workspace_bytes(int B, int H, int T, int max_pages, int page_size, int rank)
{
    if (check_latent(B, H, T, 1, page_size, max_pages, rank, 1.f) != ATTN_OK) return -1;
    return latent_layout(B, H * T, max_pages, page_size, rank).bytes;
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
    LatentCall a;
    a.l = latent_layout(B, H * T, max_pages, page_size, rank);
    if (workspace_bytes < static_cast<size_t>(a.l.bytes)) return ATTN_ERR_INVALID;
    if (current_device(&a.dev) != ATTN_OK) return ATTN_ERR_CUDA;
    attn_sm100::LatentParams &p = a.p;
    p.status = status_word(a.dev);
    if (!p.status) return ATTN_ERR_CUDA;
    a.q = q;
    a.pages = pages;
    a.page_stride = s[0];
    a.token_stride = s[2];
    a.workspace = static_cast<uint8_t *>(workspace);
    a.H = H;
    a.page_size = page_size;
    a.st = static_cast<cudaStream_t>(stream);
    p.split = {lens, B, T, max_pages * page_size, -1, 0, nullptr};
    p.pages = {page_table, num_pages, max_pages, log2_of(page_size)};
    p.o = static_cast<__nv_bfloat16 *>(o);
    p.lse = lse;
    p.GT = H * T;
    p.scale_log2 = scale * 1.4426950408889634f;
    const int nc = latent_columns(H * T);
    return rank == 256 ? launch_latent_nc<256>(a, nc) : launch_latent_nc<512>(a, nc);
}
