// attn_pages_api.cu - host side of the paged cache's upkeep: argument checks,
// workspace layout, launches. Contracts in include/attn.h.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cstdint>

#include "attn.h"
#include "attn_host.h"
#include "attn_pages_kernel.cuh"

namespace {

using namespace attn_host;
using namespace attn_sm100;

int check_pools(PagePools *p, const void *k_pages, const void *v_pages, const int64_t *strides, int Hkv,
                int num_pages, int page_size, int d)
{
    if (!k_pages || !aligned(k_pages, 16) || !aligned(v_pages, 16)) return ATTN_ERR_INVALID;
    if (Hkv <= 0 || num_pages <= 0 || page_size <= 0 || d <= 0) return ATTN_ERR_INVALID;
    if (d % 8 != 0 || d > 1024 || num_pages > PLAN_MAX_PAGES) return ATTN_ERR_UNSUPPORTED;
    // a page's 16-byte units are counted in 32 bits
    if (static_cast<int64_t>(2) * Hkv * page_size > INT_MAX / (d / 8)) return ATTN_ERR_UNSUPPORTED;
    const int64_t packed[3] = {static_cast<int64_t>(Hkv) * page_size * d, static_cast<int64_t>(page_size) * d, d};
    const int64_t *const s = strides ? strides : packed;
    for (int i = 0; i < 3; ++i)
        if (s[i] < d || s[i] % 8 != 0) return ATTN_ERR_INVALID;
    p->pool[0] = static_cast<uint4 *>(const_cast<void *>(k_pages));
    p->pool[1] = static_cast<uint4 *>(const_cast<void *>(v_pages));
    p->npools = v_pages ? 2 : 1;
    p->page_stride = s[0] / 8;
    p->head_stride = s[1] / 8;
    p->token_stride = s[2] / 8;
    p->heads = Hkv;
    p->vecs = d / 8;
    p->num_pages = num_pages;
    p->page_size = page_size;
    return ATTN_OK;
}

// A page as the copies see it (see PageShape).
PageShape page_shape(const PagePools &p)
{
    PageShape g;
    const bool side_by_side = p.heads == 1 || p.head_stride == p.vecs;
    g.parts = side_by_side ? 1 : p.heads;
    g.part_stride = p.head_stride;
    g.row_stride = p.token_stride;
    g.row = FastDiv(static_cast<uint32_t>(side_by_side ? p.heads * p.vecs : p.vecs));
    return g;
}

constexpr int kSMs = 148;

int check_ints(std::initializer_list<const void *> ptrs)
{
    for (const void *p : ptrs)
        if (!p || !aligned(p, 4)) return ATTN_ERR_INVALID;
    return ATTN_OK;
}

// The plans step through requests, rows and a row's entries in 32 bits, up to
// 1024 at a time.
constexpr int kMaxCount = 1 << 30;

bool countable(int n, int num_rows, int max_pages)
{
    return n <= kMaxCount && num_rows <= kMaxCount && max_pages <= kMaxCount;
}

// Workspace in ints: owners by row, two values and a page per request (or per
// page for reserve and compact), ranks, a few scalars.
int64_t workspace_ints(int n, int num_rows, int num_pages)
{
    return static_cast<int64_t>(num_rows) + 2 * static_cast<int64_t>(n) + 3 * static_cast<int64_t>(num_pages) + 64;
}

}  // namespace

extern "C" int64_t attn_pages_workspace_bytes(int n, int num_rows, int num_pages)
{
    if (n < 0 || num_rows <= 0 || num_pages <= 0 || num_pages > PLAN_MAX_PAGES) return -1;
    if (n > 0 && !countable(n, num_rows, 1)) return -1;  // (compact, n = 0, has no such limit)
    return 4 * workspace_ints(n, num_rows, num_pages);
}

extern "C" int attn_pages_append(const void *k, const void *v, const int64_t *k_strides, const int64_t *v_strides,
                                 void *k_pages, void *v_pages, const int64_t *kv_strides, const int *page_table,
                                 const int *pos, const int *count, int B, int Hkv, int T, int num_pages,
                                 int page_size, int max_pages, int d, void *stream)
{
    AppendParams a;
    int rc = check_pools(&a.p, k_pages, v_pages, kv_strides, Hkv, num_pages, page_size, d);
    if (rc != ATTN_OK) return rc;
    if (!k || !aligned(k, 16) || !aligned(v, 16) || (v == nullptr) != (v_pages == nullptr)) return ATTN_ERR_INVALID;
    if (B <= 0 || T <= 0 || max_pages <= 0) return ATTN_ERR_INVALID;
    rc = check_ints({page_table, pos});
    if (rc != ATTN_OK || !aligned(count, 4)) return ATTN_ERR_INVALID;
    if (B > 65535 || static_cast<int64_t>(Hkv) * T > INT_MAX / d) return ATTN_ERR_UNSUPPORTED;
    if (static_cast<int64_t>(Hkv) * d > (1 << 25)) return ATTN_ERR_UNSUPPORTED;  // (65535 blocks of 1024 in z)
    const int64_t packed[3] = {static_cast<int64_t>(Hkv) * T * d, static_cast<int64_t>(T) * d, d};
    for (int i = 0; i < 2; ++i) {
        const int64_t *s = i == 0 ? k_strides : v_strides;
        if (!s) s = packed;
        for (int j = 0; j < 3; ++j)
            if (s[j] < 0 || s[j] % 8 != 0) return ATTN_ERR_INVALID;
        a.src[i] = static_cast<const uint4 *>(i == 0 ? k : v);
        a.sb[i] = s[0] / 8;
        a.sh[i] = s[1] / 8;
        a.st[i] = s[2] / 8;
    }
    a.table = page_table;
    a.pos = pos;
    a.count = count;
    a.T = T;
    a.max_pages = max_pages;
    a.vecs = FastDiv(static_cast<uint32_t>(a.p.vecs));
    a.page = FastDiv(static_cast<uint32_t>(page_size));
    // Eight loads a lane in flight: one token of two pools, or two of one (27,000
    // latent rows of 576: 8.5 us out of L2, one token a warp 10.0; keys and values
    // of 8 heads x 128, two tokens a warp: 34.4 us instead of 33.5 for 25,000, 23.7
    // instead of 21.5 for 16,000).
    const int tokens = (v ? 1 : 2) * (APPEND_THREADS / 32), units = 32 * APPEND_COLS;
    const dim3 grid(static_cast<unsigned>((T + tokens - 1) / tokens), static_cast<unsigned>(B),
                    static_cast<unsigned>((Hkv * a.p.vecs + units - 1) / units));
    return launch_behind(v ? pages_append_kernel<1, 2> : pages_append_kernel<2, 1>, grid, APPEND_THREADS, 0,
                         static_cast<cudaStream_t>(stream), a);
}

extern "C" int attn_pages_reserve(int *page_table, int *refs, const int *rows, const int *want, int *granted,
                                  void *workspace, size_t workspace_bytes, int n, int num_rows, int num_pages,
                                  int page_size, int max_pages, void *stream)
{
    if (n < 0 || num_rows <= 0 || num_pages <= 0 || page_size <= 0 || max_pages <= 0) return ATTN_ERR_INVALID;
    if (num_pages > PLAN_MAX_PAGES || !countable(n, num_rows, max_pages)) return ATTN_ERR_UNSUPPORTED;
    if (n == 0) return ATTN_OK;
    if (check_ints({page_table, refs, rows, want, granted, workspace}) != ATTN_OK) return ATTN_ERR_INVALID;
    if (workspace_bytes < static_cast<size_t>(4 * workspace_ints(n, num_rows, num_pages))) return ATTN_ERR_INVALID;
    ReserveParams a;
    a.t = {page_table, nullptr, refs, num_rows, max_pages};
    a.rows = rows;
    a.want = want;
    a.granted = granted;
    a.owner = static_cast<int *>(workspace);
    a.need = a.owner + num_rows;
    a.first = a.need + n;
    a.list = a.first + n;
    a.n = n;
    a.num_pages = num_pages;
    a.page_size = page_size;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (n <= RESERVE_FEW) return launch_behind(pages_reserve_kernel, dim3(1), PLAN_THREADS, 0, st, a);
    const unsigned blocks = static_cast<unsigned>((static_cast<int64_t>(n) * 32 + RESERVE_THREADS - 1) / RESERVE_THREADS);
    int rc = launch_behind(pages_reserve_count_kernel, dim3(blocks), RESERVE_THREADS, 0, st, a);
    if (rc == ATTN_OK) rc = launch_behind(pages_reserve_kernel, dim3(1), PLAN_THREADS, 0, st, a);
    if (rc == ATTN_OK) rc = launch_behind(pages_reserve_fill_kernel, dim3(blocks), RESERVE_THREADS, 0, st, a);
    return rc;
}

extern "C" int attn_pages_fork(void *k_pages, void *v_pages, const int64_t *kv_strides, int *page_table, int *lens,
                               int *refs, const int *parents, const int *children, int *fresh, int *granted,
                               void *workspace, size_t workspace_bytes, int n, int num_rows, int Hkv, int num_pages,
                               int page_size, int max_pages, int d, void *stream)
{
    ForkParams a;
    const int rc = check_pools(&a.p, k_pages, v_pages, kv_strides, Hkv, num_pages, page_size, d);
    if (rc != ATTN_OK) return rc;
    if (n < 0 || num_rows <= 0 || max_pages <= 0) return ATTN_ERR_INVALID;
    if (!countable(n, num_rows, max_pages)) return ATTN_ERR_UNSUPPORTED;
    if (n == 0) return ATTN_OK;
    if (check_ints({page_table, lens, refs, parents, children, fresh, granted, workspace}) != ATTN_OK)
        return ATTN_ERR_INVALID;
    if (workspace_bytes < static_cast<size_t>(4 * workspace_ints(n, num_rows, num_pages))) return ATTN_ERR_INVALID;
    a.g = page_shape(a.p);
    a.t = {page_table, lens, refs, num_rows, max_pages};
    a.parents = parents;
    a.children = children;
    a.fresh = fresh;
    a.granted = granted;
    a.owner = static_cast<int *>(workspace);
    a.length = a.owner + num_rows;
    a.list = a.length + n;
    a.n = n;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (launch_behind(pages_fork_plan_kernel, dim3(1), PLAN_THREADS, 0, st, a) != ATTN_OK) return ATTN_ERR_CUDA;
    // eight blocks an SM in all, each with a share of a fork's copy
    const int split = std::max(1, std::min(8 * kSMs / n, 64));
    return launch_behind(pages_fork_kernel, dim3(static_cast<unsigned>(n), static_cast<unsigned>(split)), COPY_THREADS,
                         0, st, a);
}

extern "C" int attn_pages_free(int *page_table, int *lens, int *refs, const int *rows, int n, int num_rows,
                               int num_pages, int max_pages, void *stream)
{
    if (n < 0 || num_rows <= 0 || num_pages <= 0 || max_pages <= 0) return ATTN_ERR_INVALID;
    if (!countable(n, num_rows, max_pages)) return ATTN_ERR_UNSUPPORTED;
    if (n == 0) return ATTN_OK;
    if (check_ints({page_table, lens, refs, rows}) != ATTN_OK) return ATTN_ERR_INVALID;
    const PageTables t = {page_table, lens, refs, num_rows, max_pages};
    return launch_behind(pages_free_kernel, dim3(static_cast<unsigned>(n)), FREE_THREADS, 0,
                         static_cast<cudaStream_t>(stream), t, rows, num_pages);
}

extern "C" int attn_pages_compact(void *k_pages, void *v_pages, const int64_t *kv_strides, const int *page_table,
                                  const int *refs, int *table_out, int *refs_out, int *live, void *workspace,
                                  size_t workspace_bytes, int num_rows, int Hkv, int num_pages, int page_size,
                                  int max_pages, int d, void *stream)
{
    CompactParams a;
    const int rc = check_pools(&a.p, k_pages, v_pages, kv_strides, Hkv, num_pages, page_size, d);
    if (rc != ATTN_OK) return rc;
    if (num_rows <= 0 || max_pages <= 0) return ATTN_ERR_INVALID;
    if (check_ints({page_table, refs, table_out, refs_out, live, workspace}) != ATTN_OK) return ATTN_ERR_INVALID;
    if (workspace_bytes < static_cast<size_t>(4 * workspace_ints(0, num_rows, num_pages))) return ATTN_ERR_INVALID;
    a.g = page_shape(a.p);
    if (a.g.row_stride == a.g.row.d && a.g.parts > 1 && a.p.head_stride == page_size * a.p.token_stride) {
        a.g.parts = 1;
        a.g.row_stride = Hkv * a.p.vecs;
        a.g.row = FastDiv(static_cast<uint32_t>(Hkv * a.p.vecs));
    }
    a.table = page_table;
    a.refs = refs;
    a.table_out = table_out;
    a.refs_out = refs_out;
    a.live = live;
    a.holes = static_cast<int *>(workspace);
    a.movers = a.holes + num_pages;
    a.rank = a.movers + num_pages;
    a.moves = a.rank + num_pages;
    a.cells = static_cast<int64_t>(num_rows) * max_pages;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (launch_behind(pages_compact_plan_kernel, dim3(1), PLAN_THREADS, 0, st, a) != ATTN_OK) return ATTN_ERR_CUDA;
    return launch_behind(pages_compact_kernel, dim3(8 * kSMs), COPY_THREADS, 0, st, a);
}
