// attn_pages_kernel.cuh - upkeep of a paged key/value cache.
//
// The state, all on the device:
//   pool(s)      pages of `page_size` token rows per key/value head, d bf16
//                each; one pool (latent vectors) or two (K and V) of one layout
//   page_table   [num_rows, max_pages]: row r's position p lies in page
//                table[r, p / page_size], slot p % page_size; see is_page
//   lens         [num_rows]: cached tokens of each row
//   refs         [num_pages]: rows that hold the page; <= 0: the page is free
//
// Everything here moves bytes or small integers: nothing is computed in
// floating point, and every result is a function of its inputs alone (the
// lowest free pages are taken, in the order of the requests).
//
// What bounds it: HBM for the copies (8 x 2048 to 4096 tokens of 8 heads x 128
// appended: 33.2 us for 201 MB read and written, 6.1 TB/s; 3676 of 16384 latent pages
// compacted: 91 us for 542 MB, 6.0 TB/s, the copy itself 6.7), and for everything
// small the launches, 2 to 3 us each. Plans are made by one block; its running
// sums take eight counts a thread or, for compacting, words of 32 pages' bits (the
// ranks of 16384 pages: 18 -> 8 us).
#pragma once
#include <cstdint>

#include "sm100.cuh"

namespace attn_sm100 {

// n / d for n below 2^31 by a multiplication: with s = ceil(log2 d) and
// m = floor(2^32 (2^s - d) / d) + 1, n / d = (mulhi(m, n) + n) >> s (Granlund
// and Montgomery, division by invariant integers; the sum stays below 2^32).
struct FastDiv {
    uint32_t d, m, s;

    __host__ __device__ FastDiv() : d(1), m(1), s(0) {}
    explicit FastDiv(uint32_t by) : d(by), m(1), s(0)
    {
        while ((1ull << s) < d) ++s;
        m = static_cast<uint32_t>(((1ull << 32) * ((1ull << s) - d)) / d + 1);
    }
    __device__ __forceinline__ uint32_t div(uint32_t n) const { return (__umulhi(m, n) + n) >> s; }
};

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

// How the copies see a page: `parts` blocks `part_stride` apart, each of rows
// (tokens) of `row` units `row_stride` apart. Heads are the parts, unless they
// lie side by side in a token's row, or whole pages without gaps are copied
// (then there is one part).
struct PageShape {
    int parts;
    int64_t part_stride, row_stride;
    FastDiv row;
};

struct PageTables {
    int *table;     // [num_rows, max_pages]
    int *lens;      // [num_rows]
    int *refs;      // [num_pages]
    int num_rows, max_pages;
};

// Any other table entry is no page: nothing is read or written through it.
__device__ __forceinline__ bool is_page(int entry, int num_pages)
{
    return static_cast<unsigned>(entry) < static_cast<unsigned>(num_pages);
}

// Units [at, end) of a part, counted row after row, from src to dst by THREADS
// threads with UNROLL loads in flight each (one at a time, a copy ran at half
// the memory's rate).
constexpr int COPY_THREADS = 256;

template <int THREADS, int UNROLL>
__device__ __forceinline__ void copy_units(uint4 *dst, const uint4 *src, const PageShape &g, int at, int end, int tid)
{
    const bool dense = g.row_stride == g.row.d;
    for (int e = at + tid; e < end; e += THREADS * UNROLL) {
        uint4 v[UNROLL];
        int64_t off[UNROLL];
#pragma unroll
        for (int i = 0; i < UNROLL; ++i) {
            const int n = e + i * THREADS;
            off[i] = n;
            if (!dense) {
                const uint32_t r = g.row.div(n);
                off[i] = r * g.row_stride + (n - r * g.row.d);
            }
            if (n < end) v[i] = src[off[i]];
        }
#pragma unroll
        for (int i = 0; i < UNROLL; ++i)
            if (e + i * THREADS < end) dst[off[i]] = v[i];
    }
}

// Every kernel here is launched so that it may start while the one before it
// in the stream still runs: it waits for that one first, and lets the next one
// do the same. (Then a call's launches cost about a microsecond less each.)
__device__ __forceinline__ void begin_behind()
{
    grid_dependency_wait();
    grid_dependents_launch();
}

// ------------------------------------------------------------------- append

struct AppendParams {
    PagePools p;
    const uint4 *src[2];
    int64_t sb[2], sh[2], st[2];  // source strides (sequence, head, token), 16-byte units
    const int *table;             // [B, max_pages]
    const int *pos;               // [B]
    const int *count;             // [B] or null
    int T, max_pages;
    FastDiv vecs, page;
};

constexpr int APPEND_THREADS = 256;
constexpr int APPEND_COLS = 4;  // 16-byte units a lane takes of a token's row

// New token u of sequence b goes to position pos[b] + u. A warp takes TOK
// tokens of one sequence (blockIdx.x) and 128 units of their heads * d rows
// (blockIdx.z): all its loads are issued before the table's answer is waited
// for, and then the stores.
template <int TOK, int POOLS>
__global__ void __launch_bounds__(APPEND_THREADS) pages_append_kernel(const AppendParams a)
{
    begin_behind();
    const PagePools &p = a.p;
    const int b = blockIdx.y, lane = threadIdx.x % 32;
    const int u0 = (blockIdx.x * (APPEND_THREADS / 32) + threadIdx.x / 32) * TOK;
    const int n = a.count ? min(max(a.count[b], 0), a.T) : a.T;
    if (u0 >= n) return;
    const int64_t first = static_cast<int64_t>(a.pos[b]) + u0;
    const int row_units = p.heads * p.vecs;
    uint4 v[TOK][APPEND_COLS][POOLS];
    int64_t to[APPEND_COLS];
#pragma unroll
    for (int i = 0; i < APPEND_COLS; ++i) {
        const int r = (blockIdx.z * APPEND_COLS + i) * 32 + lane;
        const int h = a.vecs.div(r), c = r - h * p.vecs;
        to[i] = r < row_units ? h * p.head_stride + c : -1;
#pragma unroll
        for (int t = 0; t < TOK; ++t) {
#pragma unroll
            for (int k = 0; k < POOLS; ++k)
                if (r < row_units && u0 + t < n)
                    v[t][i][k] = a.src[k][b * a.sb[k] + h * a.sh[k] + (u0 + t) * a.st[k] + c];
        }
    }
    const int64_t cap = static_cast<int64_t>(a.max_pages) * p.page_size;
#pragma unroll
    for (int t = 0; t < TOK; ++t) {
        const int64_t at = first + t;
        if (u0 + t >= n || at < 0 || at >= cap) continue;
        const int64_t slot_page = cap <= INT32_MAX ? a.page.div(static_cast<uint32_t>(at)) : at / p.page_size;
        const int page = a.table[static_cast<int64_t>(b) * a.max_pages + slot_page];
        if (!is_page(page, p.num_pages)) continue;
        const int64_t dst = page * p.page_stride + (at - slot_page * p.page_size) * p.token_stride;
#pragma unroll
        for (int i = 0; i < APPEND_COLS; ++i) {
            if (to[i] < 0) continue;
#pragma unroll
            for (int k = 0; k < POOLS; ++k) p.pool[k][dst + to[i]] = v[t][i][k];
        }
    }
}

// ----------------------------------------------------------- planning (1 CTA)

constexpr int PLAN_THREADS = 1024;
constexpr int PLAN_WARPS = PLAN_THREADS / 32;
constexpr int PLAN_PAGES = 8;          // pages a thread looks at in one go
constexpr int PLAN_MAX_PAGES = (1 << 21) - 1;  // pages of a pool, so that a block's sums fit in 32 bits
constexpr int PLAN_SMEM_ROWS = 8192;   // owners of this many rows fit in shared memory

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
    // every warp sums up the warps for itself
    int s = warp_sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const int t = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += t;
    }
    total = __shfl_sync(0xffffffffu, s, 31);
    const int before = __shfl_sync(0xffffffffu, s, warp == 0 ? 0 : warp - 1);
    __syncthreads();
    return v + (warp == 0 ? 0 : before);
}

// Which of this thread's PLAN_PAGES pages from `base` on are live, as bits.
__device__ __forceinline__ uint32_t plan_live(const int *refs, int num_pages, int base)
{
    const int at = base + static_cast<int>(threadIdx.x) * PLAN_PAGES;
    uint32_t live = 0;
#pragma unroll
    for (int i = 0; i < PLAN_PAGES; ++i)
        if (at + i < num_pages && refs[at + i] > 0) live |= 1u << i;
    return live;
}

// The lowest `wanted` free pages, ascending, into list[]; returns how many
// there are (all threads).
__device__ __forceinline__ int plan_free_pages(const int *refs, int num_pages, int wanted, int *list, int *warp_sums)
{
    int found = 0;
    for (int base = 0; base < num_pages && found < wanted; base += PLAN_THREADS * PLAN_PAGES) {
        const int at = base + static_cast<int>(threadIdx.x) * PLAN_PAGES;
        const int have = min(max(num_pages - at, 0), PLAN_PAGES);
        const uint32_t free = ~plan_live(refs, num_pages, base) & ((1u << have) - 1u);
        int total;
        int rank = found + plan_scan(__popc(free), warp_sums, total) - __popc(free);
        for (uint32_t f = free; f && rank < wanted; f &= f - 1) list[rank++] = at + __ffs(f) - 1;
        found += total;
    }
    return min(found, wanted);
}

// owner[row] = the first request that names the row (n: nobody). Kept in
// shared memory where it fits; returns where.
__device__ __forceinline__ int *plan_owners(const int *rows, int n, int *scratch, int *owner_s, int num_rows)
{
    int *const owner = num_rows <= PLAN_SMEM_ROWS ? owner_s : scratch;
    for (int i = threadIdx.x; i < num_rows; i += PLAN_THREADS) owner[i] = n;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += PLAN_THREADS) {
        const int r = rows[i];
        if (static_cast<unsigned>(r) < static_cast<unsigned>(num_rows)) atomicMin(&owner[r], i);
    }
    __syncthreads();
    return owner;
}

struct ReserveParams {
    PageTables t;
    const int *rows;  // [n]
    const int *want;  // [n]: tokens each row needs room for
    int *granted;     // [n]
    int *owner;       // workspace [num_rows]
    int *need;        // workspace [n]: pages a request asks for, -1: not valid
    int *first;       // workspace [n]: and asked for before it
    int *list;        // workspace [num_pages]
    int n, num_pages, page_size;
};

// A warp looks at a request's table entries, 32 at a time: `each` is called by
// all lanes with (entry index, whether the entry is one to fill).
template <class F>
__device__ __forceinline__ void reserve_entries(const int *row, int pages, int num_pages, F each)
{
    for (int j0 = 0; j0 < pages; j0 += 32) {
        const int j = j0 + static_cast<int>(threadIdx.x % 32);
        each(j, j < pages && !is_page(row[j], num_pages));
    }
}

// What request i asks for: how many of the entries below ceil(want / page_size)
// hold no page; -1: its row is out of range, or the table too narrow. A warp.
__device__ __forceinline__ void reserve_count(const ReserveParams &a, int i)
{
    const int r = a.rows[i], want = a.want[i];
    const int pages = want <= 0 ? 0 : (want - 1) / a.page_size + 1;
    int need = -1;
    if (static_cast<unsigned>(r) < static_cast<unsigned>(a.t.num_rows) && pages <= a.t.max_pages) {
        need = 0;
        reserve_entries(a.t.table + static_cast<int64_t>(r) * a.t.max_pages, pages, a.num_pages,
                        [&](int, bool fill) { need += __popc(__ballot_sync(0xffffffffu, fill)); });
    }
    if (threadIdx.x % 32 == 0) a.need[i] = need;
}

// Gives request i its pages, if it was granted them. A warp.
__device__ __forceinline__ void reserve_fill(const ReserveParams &a, int i)
{
    const int need = a.need[i], lane = threadIdx.x % 32;
    if (need <= 0 || !a.granted[i]) return;
    int *const row = a.t.table + static_cast<int64_t>(a.rows[i]) * a.t.max_pages;
    int k = a.first[i];
    reserve_entries(row, (a.want[i] - 1) / a.page_size + 1, a.num_pages, [&](int j, bool fill) {
        const uint32_t fills = __ballot_sync(0xffffffffu, fill);
        if (fill) {
            const int page = a.list[k + __popc(fills & ((1u << lane) - 1u))];
            row[j] = page;
            a.t.refs[page] = 1;
        }
        k += __popc(fills);
    });
}

// The plan's arithmetic. A request counts as its need, or as the whole pool where
// that is less: it cannot be met then, and what follows begins behind all pages.
// So the sum of a block's requests fits in 32 bits.
__host__ __device__ constexpr int reserve_ask(int need, int num_pages)
{
    return need < 0 ? 0 : need < num_pages ? need : num_pages;
}
static_assert(int64_t(PLAN_THREADS) * reserve_ask(INT32_MAX, PLAN_MAX_PAGES) <= INT32_MAX, "a block's sum");

// Where the pages of a request begin that `before` are asked for in front of.
__host__ __device__ constexpr int reserve_first(int64_t before, int num_pages)
{
    return static_cast<int>(before < num_pages ? before : num_pages);
}

// With `found` free pages, is the request met?
__host__ __device__ constexpr bool reserve_met(int need, int first, int found)
{
    return need == 0 || (need > 0 && first <= found && need <= found - first);
}

// The middle part, by one block: which requests are met, and where their pages
// begin in the list of the lowest free ones.
__device__ __forceinline__ void reserve_plan(const ReserveParams &a, int *warp_sums, int *owner_s)
{
    const int *const owner = plan_owners(a.rows, a.n, a.owner, owner_s, a.t.num_rows);
    int64_t before = 0;
    for (int base = 0; base < a.n; base += PLAN_THREADS) {
        const int i = base + threadIdx.x;
        int need = i < a.n ? a.need[i] : -1;
        if (need >= 0 && owner[a.rows[i]] != i) a.need[i] = need = -1;
        int total;
        const int ask = reserve_ask(need, a.num_pages);
        const int upto = plan_scan(ask, warp_sums, total);
        if (i < a.n) a.first[i] = reserve_first(before + upto - ask, a.num_pages);
        before += total;
    }
    const int wanted = static_cast<int>(min(before, static_cast<int64_t>(a.num_pages)));
    const int found = plan_free_pages(a.t.refs, a.num_pages, wanted, a.list, warp_sums);
    for (int i = threadIdx.x; i < a.n; i += PLAN_THREADS) {
        a.granted[i] = reserve_met(a.need[i], a.first[i], found) ? 1 : 0;
    }
}

// A block has a warp for each of up to RESERVE_FEW requests and does all of it;
// with more (a warp would go through several rows, one memory latency after
// another: 40 us for 512 rows), grids of warps count and fill around the plan.
constexpr int RESERVE_FEW = PLAN_WARPS;

__global__ void __launch_bounds__(PLAN_THREADS) pages_reserve_kernel(const ReserveParams a)
{
    __shared__ int warp_sums[PLAN_WARPS];
    __shared__ int owner_s[PLAN_SMEM_ROWS];
    const int warp = threadIdx.x / 32;
    begin_behind();
    if (a.n <= RESERVE_FEW) {
        if (warp < a.n) reserve_count(a, warp);
        __syncthreads();
    }
    reserve_plan(a, warp_sums, owner_s);
    if (a.n <= RESERVE_FEW) {
        __syncthreads();
        if (warp < a.n) reserve_fill(a, warp);
    }
}

constexpr int RESERVE_THREADS = 256;

__global__ void __launch_bounds__(RESERVE_THREADS) pages_reserve_count_kernel(const ReserveParams a)
{
    begin_behind();
    const int i = blockIdx.x * (RESERVE_THREADS / 32) + threadIdx.x / 32;
    if (i < a.n) reserve_count(a, i);
}

__global__ void __launch_bounds__(RESERVE_THREADS) pages_reserve_fill_kernel(const ReserveParams a)
{
    begin_behind();
    const int i = blockIdx.x * (RESERVE_THREADS / 32) + threadIdx.x / 32;
    if (i < a.n) reserve_fill(a, i);
}

// --------------------------------------------------------------------- fork

struct ForkParams {
    PagePools p;
    PageShape g;
    PageTables t;
    const int *parents, *children;  // [n]
    int *fresh, *granted;           // [n]
    int *owner;                     // workspace [num_rows]
    int *length;                    // workspace [n]: tokens the child gets, -1: not granted
    int *list;                      // workspace [num_pages]
    int n;
};

__global__ void __launch_bounds__(PLAN_THREADS) pages_fork_plan_kernel(const ForkParams a)
{
    __shared__ int warp_sums[PLAN_WARPS];
    __shared__ int owner_s[PLAN_SMEM_ROWS];
    begin_behind();
    int *const owner = plan_owners(a.children, a.n, a.owner, owner_s, a.t.num_rows);
    const unsigned rows = static_cast<unsigned>(a.t.num_rows);
    int before = 0;
    for (int base = 0; base < a.n; base += PLAN_THREADS) {
        const int i = base + threadIdx.x;
        int len = -1, need = 0;
        if (i < a.n) {
            const int from = a.parents[i], to = a.children[i];
            const bool named = static_cast<unsigned>(from) < rows && static_cast<unsigned>(to) < rows &&
                               owner[to] == i;
            // the child holds nothing yet
            if (named && a.t.lens[to] <= 0 &&
                !is_page(a.t.table[static_cast<int64_t>(to) * a.t.max_pages], a.p.num_pages)) {
                len = max(a.t.lens[from], 0);
                if (len > static_cast<int64_t>(a.t.max_pages) * a.p.page_size) len = -1;
            }
            if (len > 0 && len % a.p.page_size != 0) {
                const int last = a.t.table[static_cast<int64_t>(from) * a.t.max_pages + len / a.p.page_size];
                need = is_page(last, a.p.num_pages) ? 1 : 0;
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
    const int found = plan_free_pages(a.t.refs, a.p.num_pages, min(before, a.p.num_pages), a.list, warp_sums);
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

// Fork i: blockIdx.x; the copy of its last page is spread over gridDim.y
// blocks. The first of them also writes the child's table row and length and
// raises the counts of the shared pages. (Lengths come from the plan: a child's
// own length may be another fork's source only while it is 0.)
__global__ void __launch_bounds__(COPY_THREADS) pages_fork_kernel(const ForkParams a)
{
    begin_behind();
    const PagePools &p = a.p;
    const int i = blockIdx.x;
    const int len = a.length[i], page = a.fresh[i];
    if (len < 0) return;
    const int full = len / p.page_size, part = len % p.page_size;
    const int *const from = a.t.table + static_cast<int64_t>(a.parents[i]) * a.t.max_pages;
    if (page >= 0) {
        const int64_t src = from[full] * p.page_stride, dst = page * p.page_stride;
        // a warp takes up to 512 units of a (pool, part) pair at a time
        constexpr int CHUNK = 512;
        const int units = part * a.g.row.d, spans = p.npools * a.g.parts;
        const int chunks = (units + CHUNK - 1) / CHUNK;
        const int warps = gridDim.y * (COPY_THREADS / 32);
        for (int item = blockIdx.y * (COPY_THREADS / 32) + threadIdx.x / 32; item < spans * chunks; item += warps) {
            const int span = item / chunks, chunk = item % chunks;
            uint4 *const pool = p.pool[span / a.g.parts] + span % a.g.parts * a.g.part_stride;
            copy_units<32, 8>(pool + dst, pool + src, a.g, chunk * CHUNK, min(units, (chunk + 1) * CHUNK), threadIdx.x % 32);
        }
    }
    if (blockIdx.y == 0) {
        int *const to = a.t.table + static_cast<int64_t>(a.children[i]) * a.t.max_pages;
        for (int j = threadIdx.x; j < full; j += COPY_THREADS) {
            const int shared = from[j];
            to[j] = shared;
            if (is_page(shared, p.num_pages)) atomicAdd(&a.t.refs[shared], 1);
        }
        for (int j = full + threadIdx.x; j < a.t.max_pages; j += COPY_THREADS) to[j] = j == full ? page : -1;
        if (threadIdx.x == 0) a.t.lens[a.children[i]] = len;
    }
}

// --------------------------------------------------------------------- free

constexpr int FREE_THREADS = 256;

// A row named twice gives its pages back once: each entry is taken out of the
// table by an exchange.
__global__ void __launch_bounds__(FREE_THREADS) pages_free_kernel(const PageTables t, const int *rows, int num_pages)
{
    begin_behind();
    const int r = rows[blockIdx.x];
    if (static_cast<unsigned>(r) >= static_cast<unsigned>(t.num_rows)) return;
    int *const row = t.table + static_cast<int64_t>(r) * t.max_pages;
    for (int j = threadIdx.x; j < t.max_pages; j += FREE_THREADS) {
        const int page = atomicExch(&row[j], -1);
        if (is_page(page, num_pages)) atomicSub(&t.refs[page], 1);
    }
    if (threadIdx.x == 0) t.lens[r] = 0;
}

// ------------------------------------------------------------------ compact
//
// With L live pages, the holes are the free pages below L and the movers the
// live pages at L or above: equally many. The k-th mover goes to the k-th
// hole (both ascending). No mover's old place is a hole, so all of them move
// at once. A page's rank needs one running sum only, of the live pages before
// it: page - live_before(page) holes come before a hole, and
// live_before(page) - live_before(L) movers before a mover.

struct CompactParams {
    PagePools p;
    PageShape g;
    const int *table;
    const int *refs;
    int *table_out, *refs_out;  // may be table and refs themselves
    int *live;                  // [1]
    int *holes;                 // workspace [num_pages]: k-th hole
    int *movers;                // workspace [num_pages]: k-th mover
    int *rank;                  // workspace [num_pages]: from page L on, a mover's number, or -1
    int *moves;                 // workspace [1]
    int64_t cells;              // num_rows * max_pages
};

// Live pages as bits, a warp reading 32 in a row: up to 32 words a warp.
constexpr int COMPACT_STEP = PLAN_THREADS * 32;

__device__ __forceinline__ void compact_bits(const int *refs, int num_pages, int base, int words, uint32_t *bits_s)
{
    constexpr int AHEAD = 8;  // loads in flight
    const int lane = threadIdx.x % 32;
    if (static_cast<int>(threadIdx.x) >= words) bits_s[threadIdx.x] = 0;
    for (int w0 = threadIdx.x / 32; w0 < words; w0 += AHEAD * PLAN_WARPS) {
        int n[AHEAD];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const int page = base + (w0 + i * PLAN_WARPS) * 32 + lane;
            n[i] = w0 + i * PLAN_WARPS < words && page < num_pages ? refs[page] : 0;
        }
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const uint32_t word = __ballot_sync(0xffffffffu, n[i] > 0);
            if (lane == 0 && w0 + i * PLAN_WARPS < words) bits_s[w0 + i * PLAN_WARPS] = word;
        }
    }
    __syncthreads();
}

__global__ void __launch_bounds__(PLAN_THREADS) pages_compact_plan_kernel(const CompactParams a)
{
    __shared__ int warp_sums[PLAN_WARPS];
    __shared__ uint32_t bits_s[PLAN_THREADS];
    __shared__ int first_s[PLAN_THREADS];  // live pages before the word
    begin_behind();
    const int P = a.p.num_pages, lane = threadIdx.x % 32;
    auto words_at = [&](int base) { return min((P - base + 31) / 32, PLAN_THREADS); };
    int mine = 0, live, total;
    for (int base = 0; base < P; base += COMPACT_STEP) {
        if (base > 0) __syncthreads();
        compact_bits(a.refs, P, base, words_at(base), bits_s);
        mine += __popc(bits_s[threadIdx.x]);
    }
    plan_scan(mine, warp_sums, live);
    int before = 0, below = live;  // below: live pages below L (P == L: all)
    for (int base = 0; base < P; base += COMPACT_STEP) {
        const int words = words_at(base);
        if (P > COMPACT_STEP) compact_bits(a.refs, P, base, words, bits_s);
        const int n = __popc(bits_s[threadIdx.x]);
        first_s[threadIdx.x] = before + plan_scan(n, warp_sums, total) - n;
        before += total;
        __syncthreads();
        if (live < P && live >= base && live < base + COMPACT_STEP) {
            const int w = (live - base) / 32;
            below = first_s[w] + __popc(bits_s[w] & ((1u << (live - base) % 32) - 1u));
        }
#pragma unroll 4
        for (int w = threadIdx.x / 32; w < words; w += PLAN_WARPS) {
            const int page = base + w * 32 + lane;
            const uint32_t word = bits_s[w];
            const bool is_live = (word >> lane) & 1u;
            const int rank = first_s[w] + __popc(word & ((1u << lane) - 1u));
            if (page < P) {
                if (page < live && !is_live) a.holes[page - rank] = page;
                if (page >= live) {
                    if (is_live) a.movers[rank - below] = page;
                    a.rank[page] = is_live ? rank - below : -1;
                }
            }
        }
        __syncthreads();
    }
    if (threadIdx.x == 0) {
        *a.live = live;
        *a.moves = live - below;
    }
}

__global__ void __launch_bounds__(COPY_THREADS) pages_compact_kernel(const CompactParams a)
{
    begin_behind();
    const PagePools &p = a.p;
    const int moves = *a.moves, live = *a.live;
    // a warp takes up to 512 units of a (pool, part) pair at a time
    constexpr int CHUNK = 512;
    const uint32_t units = a.g.row.d * p.page_size, spans = p.npools * a.g.parts;
    const uint32_t chunks = (units + CHUNK - 1) / CHUNK, per_page = spans * chunks;
    const int64_t warps = static_cast<int64_t>(gridDim.x) * (COPY_THREADS / 32);
    for (int64_t item = static_cast<int64_t>(blockIdx.x) * (COPY_THREADS / 32) + threadIdx.x / 32;
         item < static_cast<int64_t>(moves) * per_page; item += warps) {
        const uint32_t k = item / per_page, rest = item - static_cast<int64_t>(k) * per_page;
        const uint32_t span = rest / chunks, chunk = rest - span * chunks;
        uint4 *const pool = p.pool[span / a.g.parts] + span % a.g.parts * a.g.part_stride;
        copy_units<32, 8>(pool + a.holes[k] * p.page_stride, pool + a.movers[k] * p.page_stride, a.g, chunk * CHUNK,
                          min(units, (chunk + 1) * CHUNK), threadIdx.x % 32);
    }
    const int64_t tid = static_cast<int64_t>(blockIdx.x) * COPY_THREADS + threadIdx.x;
    const int64_t step = static_cast<int64_t>(gridDim.x) * COPY_THREADS;
    for (int64_t i = tid; i < a.cells; i += step) {
        const int page = a.table[i];
        const int r = page >= live && page < p.num_pages ? a.rank[page] : -1;
        a.table_out[i] = r < 0 ? page : a.holes[r];
    }
    // a mover's count goes to its hole; every other page's stays where it is
    // (holes are written by their movers alone)
    for (int64_t i = tid; i < p.num_pages; i += step) {
        const int n = a.refs[i];
        if (i >= live) {
            const int r = a.rank[i];
            if (r >= 0) a.refs_out[a.holes[r]] = n;
            a.refs_out[i] = 0;
        } else if (n > 0) {
            a.refs_out[i] = n;
        }
    }
}

}  // namespace attn_sm100
