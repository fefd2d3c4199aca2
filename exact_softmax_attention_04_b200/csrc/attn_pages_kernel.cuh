// attn_pages_kernel.cuh - upkeep of a paged key/value cache.
//
// The state, all on the device:
//   pool(s)      pages of `page_size` token rows per key/value head, d bf16
//                each; one pool (latent vectors) or two (K and V) of one layout
//   page_table   [num_rows, max_pages]: row r's position p lies in page
//                table[r, p / page_size], slot p % page_size; -1: no page
//   lens         [num_rows]: cached tokens of each row
//   refs         [num_pages]: rows that hold the page; <= 0: the page is free
//
// Everything here moves bytes or small integers: nothing is computed in
// floating point, and every result is a function of its inputs alone (the
// lowest free pages are taken, in the order of the requests).
#pragma once
#include <cstdint>

namespace attn_sm100 {

// One or two pools of one layout. Strides in 16-byte units.
struct PagePools {
    uint4 *pool[2];
    int npools;
    int64_t page_stride, head_stride, token_stride;
    int heads;      // key/value heads
    int vecs;       // 16-byte units per row (d / 8)
    int num_pages;
    int page_size;
};

struct PageTables {
    int *table;     // [num_rows, max_pages]
    int *lens;      // [num_rows]
    int *refs;      // [num_pages]
    int num_rows, max_pages;
};

// ------------------------------------------------------------------- append

struct AppendParams {
    PagePools p;
    const uint4 *src[2];
    int64_t sb[2], sh[2], st[2];  // source strides (sequence, head, token), 16-byte units
    const int *table;             // [B, max_pages]
    const int *pos;               // [B]
    const int *count;             // [B] or null
    int T, max_pages;
};

constexpr int APPEND_THREADS = 256;

// New token u of sequence b goes to position pos[b] + u. A block takes
// `tokens_per_block` tokens of one sequence; a thread keeps its 16-byte column
// of a token's heads * d row and walks the tokens, so the only divisions in
// the loop are those by the page size.
__global__ void __launch_bounds__(APPEND_THREADS) pages_append_kernel(const AppendParams a, int tokens_per_block)
{
    const PagePools &p = a.p;
    const int b = blockIdx.y;
    const int row_vecs = p.heads * p.vecs;
    const int n = a.count ? min(max(a.count[b], 0), a.T) : a.T;
    const int u0 = blockIdx.x * tokens_per_block;
    const int u1 = min(u0 + tokens_per_block, n);
    const int64_t pos = a.pos[b];
    const int *const table = a.table + static_cast<int64_t>(b) * a.max_pages;
    for (int i = threadIdx.x; i < row_vecs * (u1 - u0); i += APPEND_THREADS) {
        const int u = u0 + i / row_vecs, r = i % row_vecs;
        const int h = r / p.vecs, c = r % p.vecs;
        const int64_t at = pos + u;
        if (at < 0 || at >= static_cast<int64_t>(a.max_pages) * p.page_size) continue;
        const int page = table[at / p.page_size];
        if (static_cast<unsigned>(page) >= static_cast<unsigned>(p.num_pages)) continue;
        const int64_t dst = page * p.page_stride + h * p.head_stride + (at % p.page_size) * p.token_stride + c;
        for (int k = 0; k < p.npools; ++k) p.pool[k][dst] = a.src[k][b * a.sb[k] + h * a.sh[k] + u * a.st[k] + c];
    }
}

// ----------------------------------------------------------- planning (1 CTA)

constexpr int PLAN_THREADS = 1024;

// Inclusive sum over the block of one int per thread; `total` to all threads.
__device__ __forceinline__ int plan_scan(int v, int *warp_sums, int &total)
{
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const int t = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += t;
    }
    if (lane == 31) warp_sums[warp] = v;
    __syncthreads();
    if (warp == 0) {
        int s = warp_sums[lane];
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const int t = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += t;
        }
        warp_sums[lane] = s;
    }
    __syncthreads();
    if (warp > 0) v += warp_sums[warp - 1];
    total = warp_sums[31];
    __syncthreads();
    return v;
}

// The lowest `wanted` free pages, ascending, into list[]; returns how many
// there are (all threads).
__device__ __forceinline__ int plan_free_pages(const int *refs, int num_pages, int wanted, int *list, int *warp_sums)
{
    int found = 0;
    for (int base = 0; base < num_pages && found < wanted; base += PLAN_THREADS) {
        const int page = base + threadIdx.x;
        const int is_free = (page < num_pages && refs[page] <= 0) ? 1 : 0;
        int total;
        const int rank = found + plan_scan(is_free, warp_sums, total) - is_free;
        if (is_free && rank < wanted) list[rank] = page;
        found += total;
    }
    return min(found, wanted);
}

// owner[row] = the first request that names the row (num requests: nobody).
__device__ __forceinline__ void plan_owners(const int *rows, int n, int *owner, int num_rows)
{
    for (int i = threadIdx.x; i < num_rows; i += PLAN_THREADS) owner[i] = n;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += PLAN_THREADS) {
        const int r = rows[i];
        if (static_cast<unsigned>(r) < static_cast<unsigned>(num_rows)) atomicMin(&owner[r], i);
    }
    __syncthreads();
}

struct ReserveParams {
    PageTables t;
    const int *rows;  // [n]
    const int *want;  // [n]: tokens each row needs room for
    int *granted;     // [n]
    int *owner;       // workspace [num_rows]
    int *first;       // workspace [n]
    int *list;        // workspace [num_pages]
    int n, num_pages, page_size;
};

// Entries of row r that a request for `want` tokens has to fill: those below
// ceil(want / page_size) that hold no page. -1: the request cannot be met.
__device__ __forceinline__ int reserve_need(const ReserveParams &a, int i)
{
    const int r = a.rows[i], want = a.want[i];
    if (static_cast<unsigned>(r) >= static_cast<unsigned>(a.t.num_rows) || a.owner[r] != i) return -1;
    if (want <= 0) return 0;
    const int pages = (want - 1) / a.page_size + 1;
    if (pages > a.t.max_pages) return -1;
    const int *const row = a.t.table + static_cast<int64_t>(r) * a.t.max_pages;
    int need = 0;
    for (int j = 0; j < pages; ++j) need += row[j] < 0 ? 1 : 0;
    return need;
}

__global__ void __launch_bounds__(PLAN_THREADS) pages_reserve_kernel(const ReserveParams a)
{
    __shared__ int warp_sums[32];
    plan_owners(a.rows, a.n, a.owner, a.t.num_rows);
    int64_t before = 0;
    for (int base = 0; base < a.n; base += PLAN_THREADS) {
        const int i = base + threadIdx.x;
        const int need = i < a.n ? reserve_need(a, i) : -1;
        int total;
        // sums beyond the pool stay beyond it
        const int upto = plan_scan(min(max(need, 0), a.num_pages), warp_sums, total);
        if (i < a.n) a.first[i] = need < 0 ? -1 : static_cast<int>(min(before + upto - need, int64_t(a.num_pages) + 1));
        before += total;
    }
    const int wanted = static_cast<int>(min(before, static_cast<int64_t>(a.num_pages)));
    const int found = plan_free_pages(a.t.refs, a.num_pages, wanted, a.list, warp_sums);
    __syncthreads();
    for (int i = threadIdx.x; i < a.n; i += PLAN_THREADS) {
        const int first = a.first[i];
        const int need = first < 0 ? -1 : reserve_need(a, i);
        const bool ok = need >= 0 && (need == 0 || first + need <= found);
        a.granted[i] = ok ? 1 : 0;
        if (ok && need > 0) {
            int *const row = a.t.table + static_cast<int64_t>(a.rows[i]) * a.t.max_pages;
            for (int j = 0, k = first; k < first + need; ++j) {
                if (row[j] >= 0) continue;
                const int page = a.list[k++];
                row[j] = page;
                a.t.refs[page] = 1;
            }
        }
    }
}

// --------------------------------------------------------------------- fork

struct ForkParams {
    PagePools p;
    PageTables t;
    const int *parents, *children;  // [n]
    int *fresh, *granted;           // [n]
    int *owner;                     // workspace [num_rows]
    int *length;                    // workspace [n]: tokens the child gets, -1: not granted
    int *list;                      // workspace [n]
    int n;
};

__global__ void __launch_bounds__(PLAN_THREADS) pages_fork_plan_kernel(const ForkParams a)
{
    __shared__ int warp_sums[32];
    plan_owners(a.children, a.n, a.owner, a.t.num_rows);
    const unsigned rows = static_cast<unsigned>(a.t.num_rows);
    int before = 0;
    for (int base = 0; base < a.n; base += PLAN_THREADS) {
        const int i = base + threadIdx.x;
        int len = -1, need = 0;
        if (i < a.n) {
            const int from = a.parents[i], to = a.children[i];
            const bool named = static_cast<unsigned>(from) < rows && static_cast<unsigned>(to) < rows &&
                               a.owner[to] == i;
            // the child holds nothing yet
            if (named && a.t.lens[to] == 0 && a.t.table[static_cast<int64_t>(to) * a.t.max_pages] < 0) {
                len = max(a.t.lens[from], 0);
                if (len > static_cast<int64_t>(a.t.max_pages) * a.p.page_size) len = -1;
            }
            if (len > 0 && len % a.p.page_size != 0) {
                const int last = a.t.table[static_cast<int64_t>(from) * a.t.max_pages + len / a.p.page_size];
                need = static_cast<unsigned>(last) < static_cast<unsigned>(a.p.num_pages) ? 1 : 0;
            }
        }
        int total;
        const int upto = before + plan_scan(need, warp_sums, total);
        if (i < a.n) {
            a.length[i] = len;
            a.fresh[i] = need ? upto - 1 : -1;  // the page's rank for now
        }
        before += total;
    }
    const int found = plan_free_pages(a.t.refs, a.p.num_pages, before, a.list, warp_sums);
    __syncthreads();
    for (int i = threadIdx.x; i < a.n; i += PLAN_THREADS) {
        const int rank = a.fresh[i];
        const bool ok = a.length[i] >= 0 && (rank < 0 || rank < found);
        const int page = (ok && rank >= 0) ? a.list[rank] : -1;
        a.fresh[i] = page;
        a.granted[i] = ok ? 1 : 0;
        if (!ok) a.length[i] = -1;
        if (page >= 0) a.t.refs[page] = 1;
    }
}

constexpr int FORK_THREADS = 256;

// Fork i: blockIdx.x; its rows are spread over gridDim.y blocks. The first of
// them also writes the child's table row and length and raises the counts of
// the shared pages. (Lengths come from the plan: a child's own length may be
// another fork's source only while it is 0.)
__global__ void __launch_bounds__(FORK_THREADS) pages_fork_kernel(const ForkParams a)
{
    const PagePools &p = a.p;
    const int i = blockIdx.x;
    const int len = a.length[i];
    if (len < 0) return;
    const int full = len / p.page_size, part = len % p.page_size;
    const int *const from = a.t.table + static_cast<int64_t>(a.parents[i]) * a.t.max_pages;
    if (blockIdx.y == 0) {
        int *const to = a.t.table + static_cast<int64_t>(a.children[i]) * a.t.max_pages;
        for (int j = threadIdx.x; j < full; j += FORK_THREADS) {
            const int page = from[j];
            to[j] = page;
            if (static_cast<unsigned>(page) < static_cast<unsigned>(p.num_pages)) atomicAdd(&a.t.refs[page], 1);
        }
        for (int j = full + threadIdx.x; j < a.t.max_pages; j += FORK_THREADS) to[j] = j == full ? a.fresh[i] : -1;
        if (threadIdx.x == 0) a.t.lens[a.children[i]] = len;
    }
    const int page = a.fresh[i];
    if (page < 0) return;
    const int64_t src = from[full] * p.page_stride, dst = page * p.page_stride;
    const int per_head = part * p.vecs;
    for (int e = blockIdx.y * FORK_THREADS + threadIdx.x; e < p.npools * p.heads * per_head;
         e += gridDim.y * FORK_THREADS) {
        const int hp = e / per_head, r = e % per_head;
        const int64_t at = (hp % p.heads) * p.head_stride + (r / p.vecs) * p.token_stride + r % p.vecs;
        uint4 *const pool = p.pool[hp / p.heads];
        pool[dst + at] = pool[src + at];
    }
}

// --------------------------------------------------------------------- free

constexpr int FREE_THREADS = 256;

// A row named twice gives its pages back once: each entry is taken out of the
// table by an exchange.
__global__ void __launch_bounds__(FREE_THREADS) pages_free_kernel(const PageTables t, const int *rows, int num_pages)
{
    const int r = rows[blockIdx.x];
    if (static_cast<unsigned>(r) >= static_cast<unsigned>(t.num_rows)) return;
    int *const row = t.table + static_cast<int64_t>(r) * t.max_pages;
    for (int j = threadIdx.x; j < t.max_pages; j += FREE_THREADS) {
        const int page = atomicExch(&row[j], -1);
        if (static_cast<unsigned>(page) < static_cast<unsigned>(num_pages)) atomicSub(&t.refs[page], 1);
    }
    if (threadIdx.x == 0) t.lens[r] = 0;
}

// ------------------------------------------------------------------ compact
//
// With L live pages, the holes are the free pages below L and the movers the
// live pages at L or above: equally many. The k-th mover goes to the k-th
// hole (both ascending). No mover's old place is a hole, so all of them move
// at once.

struct CompactParams {
    PagePools p;
    const int *table;
    const int *refs;
    int *table_out, *refs_out;  // may be table and refs themselves
    int *live;                  // [1]
    int *holes;                 // workspace [num_pages]: k-th hole
    int *movers;                // workspace [num_pages]: k-th mover
    int *rank;                  // workspace [num_pages]: a page's number as a mover, -1: it stays
    int *moves;                 // workspace [1]
    int64_t cells;              // num_rows * max_pages
};

__global__ void __launch_bounds__(PLAN_THREADS) pages_compact_plan_kernel(const CompactParams a)
{
    __shared__ int warp_sums[32];
    const int P = a.p.num_pages;
    int live = 0, total;
    for (int base = 0; base < P; base += PLAN_THREADS) {
        const int page = base + threadIdx.x;
        plan_scan((page < P && a.refs[page] > 0) ? 1 : 0, warp_sums, total);
        live += total;
    }
    int holes = 0, movers = 0;
    for (int base = 0; base < P; base += PLAN_THREADS) {
        const int page = base + threadIdx.x;
        const bool is_live = page < P && a.refs[page] > 0;
        const int hole = (page < live && !is_live) ? 1 : 0, mover = (page >= live && is_live) ? 1 : 0;
        const int h = holes + plan_scan(hole, warp_sums, total);
        holes += total;
        const int m = movers + plan_scan(mover, warp_sums, total);
        movers += total;
        if (hole) a.holes[h - 1] = page;
        if (mover) a.movers[m - 1] = page;
        if (page < P) a.rank[page] = mover ? m - 1 : -1;
    }
    if (threadIdx.x == 0) {
        *a.live = live;
        *a.moves = movers;
    }
}

constexpr int COMPACT_THREADS = 256;

__global__ void __launch_bounds__(COMPACT_THREADS) pages_compact_kernel(const CompactParams a)
{
    const PagePools &p = a.p;
    const int moves = *a.moves;
    const int64_t tid = static_cast<int64_t>(blockIdx.x) * COMPACT_THREADS + threadIdx.x;
    const int64_t step = static_cast<int64_t>(gridDim.x) * COMPACT_THREADS;
    for (int64_t i = tid; i < a.cells; i += step) {
        const int page = a.table[i];
        const int r = static_cast<unsigned>(page) < static_cast<unsigned>(p.num_pages) ? a.rank[page] : -1;
        a.table_out[i] = r < 0 ? page : a.holes[r];
    }
    // a mover's count goes to its hole; every other page's stays where it is
    // (holes are written by their movers alone)
    for (int64_t i = tid; i < p.num_pages; i += step) {
        const int r = a.rank[i], n = a.refs[i];
        if (r >= 0) {
            a.refs_out[a.holes[r]] = n;
            a.refs_out[i] = 0;
        } else if (n > 0 || i >= *a.live) {
            a.refs_out[i] = max(n, 0);
        }
    }
    const int per_head = p.page_size * p.vecs, per_page = p.npools * p.heads * per_head;
    for (int k = blockIdx.x; k < moves; k += gridDim.x) {
        const int64_t src = a.movers[k] * p.page_stride, dst = a.holes[k] * p.page_stride;
        for (int e = threadIdx.x; e < per_page; e += COMPACT_THREADS) {
            const int hp = e / per_head, r = e % per_head;
            const int64_t at = (hp % p.heads) * p.head_stride + (r / p.vecs) * p.token_stride + r % p.vecs;
            uint4 *const pool = p.pool[hp / p.heads];
            pool[dst + at] = pool[src + at];
        }
    }
}

}  // namespace attn_sm100
