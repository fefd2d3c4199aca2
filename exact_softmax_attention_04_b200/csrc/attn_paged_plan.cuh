// attn_paged_plan.cuh - how the work of attention over a paged cache is split,
// and how the parts are joined. Shared by the kernels for pages of keys and
// values and for pages of latent vectors.
//
// The positions a sequence's new tokens see are cut into tiles of TK; the
// tiles of all sequences, in order, are dealt out as `ranges` contiguous runs
// that differ by one tile at most, one to each block of the grid's x (the y
// blocks take the heads of the same run). So every block has the same amount
// to read whatever the lengths are, and the host need not know them. Within a
// run, the tiles of one sequence are a segment. A segment that is the whole
// sequence is finished by its block. Others leave their unnormalised O, maximum
// and sum in the workspace: a block has two such segments at most, its first
// and its last, so it has two places there; `attn_paged_combine_kernel` joins
// them (about 3 us at a call's end, most of it latency). A sequence without a
// position counts as one tile, so that its (empty) answer is written like any other.
#pragma once
#include "attn_fwd_kernel.cuh"

namespace attn_sm100 {

struct PagedSplit {
    const int *lens;      // [B]
    int B, T, cap;        // cap: positions that the table holds
    int window;           // -1: none
    int ranges;           // gridDim.x
    int *before;          // workspace [B + 1]: tiles before each sequence, then all (B > COMBINE_SCAN)
};

// Up to this many sequences, the joining kernel sums their tiles itself, while
// the kernel before it still runs; with more it reads what block (0, 0) wrote
// (4 heads a key/value head at d 64: 1000 sequences of up to 600 tokens 24.0 us
// summing, 23.3 reading; 300 of 500 to 4000 x 2 heads 65.9 and 65.5; 128 of them 32.9
// and 33.4; one latent sequence of 60000 x 16 heads of rank 512 22.8 and 24.0).
constexpr int COMBINE_SCAN = 128;

// The tiles of one sequence: positions first * TK up to len - 1.
struct PagedSeq {
    int len, first, ntiles;
};

template <int TK>
__device__ __forceinline__ PagedSeq paged_seq_of(const PagedSplit &p, int len)
{
    PagedSeq s;
    s.len = min(max(len, 0), p.cap);
    s.first = p.window >= 0 ? max(0, s.len - p.T - p.window) / TK : 0;
    s.ntiles = max(s.len - 1, 0) / TK - s.first + 1;
    return s;
}

// (Plain loads of lengths and tables, not read-only ones: the block may have
// started before the kernel that writes them ended.)
template <int TK>
__device__ __forceinline__ PagedSeq paged_seq(const PagedSplit &p, int b)
{
    return paged_seq_of<TK>(p, p.lens[b]);
}

// `total` tiles dealt out to n runs: the first total % n have one more.
struct PagedDeal {
    int each, more;

    __device__ __forceinline__ PagedDeal(int total, int n) : each(total / n), more(total % n) {}
    __device__ __forceinline__ int start(int r) const { return r * each + min(r, more); }
    __device__ __forceinline__ int run_of(int tile) const
    {
        const int large = more * (each + 1);
        return tile < large ? tile / (each + 1) : more + (tile - large) / each;
    }
};

// A place in the order of all tiles: tile j of sequence b.
template <int TK>
struct PagedWalk {
    int b, j;
    PagedSeq s;

    // (the caller does not step past the last tile)
    __device__ __forceinline__ void step(const PagedSplit &p)
    {
        if (++j == s.ntiles) {
            ++b;
            j = 0;
            s = paged_seq<TK>(p, b);
        }
    }
    __device__ __forceinline__ int base() const { return (s.first + j) * TK; }
    __device__ __forceinline__ bool last() const { return j + 1 == s.ntiles; }
};

struct PagedTable {
    const int *table;  // [B, max_pages]
    int num_pages, max_pages;
    int page_log2;
};

// The page that holds positions [at, at + 2^page_log2) of sequence b, `at` a
// multiple of the page size; -1 if no token sees one of them or the entry is
// no page.
__device__ __forceinline__ int paged_page(const PagedSplit &p, const PagedTable &t, const PagedSeq &s, int b, int at)
{
    const int lo = p.window >= 0 ? max(0, s.len - p.T - p.window) : 0;
    if (at >= s.len || at + (1 << t.page_log2) <= lo) return -1;
    const int page = t.table[static_cast<int64_t>(b) * t.max_pages + (at >> t.page_log2)];
    return static_cast<unsigned>(page) < static_cast<unsigned>(t.num_pages) ? page : -1;
}

struct PagedRun {
    int b, j, count, len;  // first tile, number of tiles (0: none), the sequence's length

    template <int TK>
    __device__ __forceinline__ PagedWalk<TK> walk(const PagedSplit &p) const
    {
        return {b, j, paged_seq_of<TK>(p, len)};
    }
};

// The block's run, for all its NT threads; `scratch`: PLAN_SCRATCH bytes of
// shared memory, 16-byte aligned.
constexpr int PLAN_SCRATCH = 96;

template <int TK, int NT>
__device__ __forceinline__ PagedRun paged_run(const PagedSplit &p, int r, void *scratch)
{
    static_assert(NT / 32 * 4 + 16 <= PLAN_SCRATCH, "scratch");
    PagedRun &run = *static_cast<PagedRun *>(scratch);
    int *const sums = static_cast<int *>(scratch) + 4;
    const int tid = threadIdx.x, lane = tid % 32;
    const int per = (p.B + NT - 1) / NT;
    const int b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);
    // (the thread's one sequence is read once; with more than NT sequences,
    // its several are read again)
    const int len0 = b0 < b1 ? p.lens[b0] : 0;
    int mine = b0 < b1 ? paged_seq_of<TK>(p, len0).ntiles : 0;
    for (int b = b0 + 1; b < b1; ++b) mine += paged_seq<TK>(p, b).ntiles;
    int upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const int t = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += t;
    }
    if (lane == 31) sums[tid / 32] = upto;
    if (tid == 0) run.count = 0;
    __syncthreads();
    int total = 0;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) {
        if (w < tid / 32) upto += sums[w];
        total += sums[w];
    }
    if (p.B > COMBINE_SCAN && blockIdx.x == 0 && blockIdx.y == 0) {
        int at = upto - mine;
        for (int b = b0; b < b1; ++b) {
            p.before[b] = at;
            at += paged_seq<TK>(p, b).ntiles;
        }
        if (tid == 0) p.before[p.B] = total;
    }
    const int n = min(p.ranges, total);
    if (r < n) {
        const PagedDeal deal(total, n);
        const int t0 = deal.start(r);
        int at = upto - mine;
        if (t0 >= at && t0 < upto) {
            int b = b0, len = len0, tiles = paged_seq_of<TK>(p, len).ntiles;
            while (t0 >= at + tiles) {
                at += tiles;
                len = p.lens[++b];
                tiles = paged_seq_of<TK>(p, len).ntiles;
            }
            run.b = b;
            run.j = t0 - at;
            run.len = len;
            run.count = deal.start(r + 1) - t0;
        }
    }
    __syncthreads();
    return run;
}

// The segments' results in the workspace: for slot s (two for each block: x,
// then y, then which) and column c of NC, O at o[(s * NC + c) * DV] and the
// maximum (log2 units) and sum at ml[s * NC + c].
__device__ __forceinline__ int64_t paged_slot(int x, int y, int ranges, bool first)
{
    return (static_cast<int64_t>(y) * ranges + x) * 2 + (first ? 0 : 1);
}

struct PagedCombine {
    PagedSplit split;
    const float *part_o;
    const float2 *part_ml;
    __nv_bfloat16 *o;  // [B, H, T, DV]
    float *lse;        // [B, H, T]
    int H, Hkv, nblk;  // heads; column blocks of a group
    int per_block;     // columns a block joins
};

constexpr int COMBINE_THREADS = 256;

// Joins the segments of `per_block` columns of one (sequence, y) pair:
//   M = max_s m_s, l = sum_s l_s 2^(m_s - M), O = sum_s O_s 2^(m_s - M) / l.
// DC of the DV columns of O a block (grid y), DC / 4 lanes with 16 bytes each of
// a segment. With few segments the groups of
// lanes take the columns in turn, with many they take the segments, so that a
// hundred segments of a long sequence are a dozen loads deep. Which segments
// there are follows from the lengths alone and is worked out while the kernel
// before is still running.
template <int TK, int DV, int DC, int NC>
__global__ void __launch_bounds__(COMBINE_THREADS) attn_paged_combine_kernel(const PagedCombine a)
{
    constexpr int LANES = DC / 4, GROUPS = COMBINE_THREADS / LANES;
    constexpr int FEW = 6;
    __shared__ int red[2][COMBINE_THREADS / 32];
    __shared__ float4 acc_s[GROUPS][LANES];
    __shared__ float l_s[GROUPS];
    grid_dependents_launch();
    const PagedSplit &p = a.split;
    const int tid = threadIdx.x;
    const int G = a.H / a.Hkv, GT = G * p.T, units = a.Hkv * a.nblk;
    const int per_unit = (min(GT, NC) + a.per_block - 1) / a.per_block;
    const int b = blockIdx.x / per_unit / units, y = blockIdx.x / per_unit % units;
    const int head = y / a.nblk, c0 = y % a.nblk * NC;
    const int c_begin = blockIdx.x % per_unit * a.per_block;
    const int c_end = min(c_begin + a.per_block, min(GT - c0, NC));

    int before = 0, total = 0;
    if (p.B <= COMBINE_SCAN) {
        for (int i = tid; i < p.B; i += COMBINE_THREADS) {
            const int n = paged_seq<TK>(p, i).ntiles;
            total += n;
            before += i < b ? n : 0;
        }
#pragma unroll
        for (int o = 16; o >= 1; o /= 2) {
            total += __shfl_xor_sync(0xffffffffu, total, o);
            before += __shfl_xor_sync(0xffffffffu, before, o);
        }
        if (tid % 32 == 0) {
            red[0][tid / 32] = total;
            red[1][tid / 32] = before;
        }
        __syncthreads();
        total = before = 0;
#pragma unroll
        for (int w = 0; w < COMBINE_THREADS / 32; ++w) {
            total += red[0][w];
            before += red[1][w];
        }
    } else {
        grid_dependency_wait();
        before = p.before[b];
        total = p.before[p.B];
    }
    const int end = before + paged_seq<TK>(p, b).ntiles - 1;  // the last tile
    const int n = min(p.ranges, total);
    // the runs that hold the first and the last tile
    const PagedDeal deal(total, n);
    const int r0 = deal.run_of(before), r1 = deal.run_of(end);
    const int nseg = r1 - r0 + 1;
    // run r0 may begin before the sequence; then this is its last segment
    const bool r0_first = deal.start(r0) >= before;
    auto slot = [&](int s, int c) { return paged_slot(r0 + s, y, p.ranges, s > 0 || r0_first) * NC + c; };
    const int g = tid / LANES, e = tid % LANES, col = blockIdx.y * DC + 4 * e;
    const int64_t row0 = (static_cast<int64_t>(b) * a.H + head * G) * p.T + c0;

    auto add = [](float4 &acc, float &l, const float2 &ml, const float4 &v, float ref) {
        const float f = ex2_approx(ml.x - ref);  // 0 for a segment without a position
        l = fmaf(ml.y, f, l);
        acc.x = fmaf(v.x, f, acc.x);
        acc.y = fmaf(v.y, f, acc.y);
        acc.z = fmaf(v.z, f, acc.z);
        acc.w = fmaf(v.w, f, acc.w);
    };
    auto write = [&](const float4 &acc, float l, float M, int c) {
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const __nv_bfloat162 lo = __floats2bfloat162_rn(acc.x * inv, acc.y * inv);
        const __nv_bfloat162 hi = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
        uint2 w;
        w.x = *reinterpret_cast<const uint32_t *>(&lo);
        w.y = *reinterpret_cast<const uint32_t *>(&hi);
        *reinterpret_cast<uint2 *>(a.o + (row0 + c) * DV + col) = w;
        if (col == 0) a.lse[row0 + c] = l == 0.f ? -CUDART_INF_F : (M + __log2f(l)) * 0.69314718055994531f;
    };

    grid_dependency_wait();
    if (nseg == 1) return;  // one block had the whole sequence

    if (nseg <= FEW) {
        // all of a column's loads before the first sum (45 latent sequences of 100
        // to 3000 tokens x 128 heads of rank 512: 56 us; by the form below, 72)
        for (int c = c_begin + g; c < c_end; c += GROUPS) {
            float2 ml[FEW];
            float4 v[FEW];
#pragma unroll
            for (int s = 0; s < FEW; ++s) {
                ml[s] = make_float2(-CUDART_INF_F, 0.f);
                v[s] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (s < nseg) {
                    const int64_t at = slot(s, c);
                    ml[s] = a.part_ml[at];
                    v[s] = *reinterpret_cast<const float4 *>(a.part_o + at * DV + col);
                }
            }
            float M = -CUDART_INF_F, l = 0.f;
#pragma unroll
            for (int s = 0; s < FEW; ++s) M = fmaxf(M, ml[s].x);
            const float ref = M == -CUDART_INF_F ? 0.f : M;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int s = 0; s < FEW; ++s)
                if (s < nseg) add(acc, l, ml[s], v[s], ref);
            write(acc, l, M, c);
        }
        return;
    }
    for (int c = c_begin; c < c_end; ++c) {
        float M = -CUDART_INF_F;
        for (int s = tid % 32; s < nseg; s += 32) M = fmaxf(M, a.part_ml[slot(s, c)].x);
        M = redux_max(M);
        const float ref = M == -CUDART_INF_F ? 0.f : M;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        float l = 0.f;
#pragma unroll 8
        for (int s = g; s < nseg; s += GROUPS) {
            const int64_t at = slot(s, c);
            add(acc, l, a.part_ml[at], *reinterpret_cast<const float4 *>(a.part_o + at * DV + col), ref);
        }
        acc_s[g][e] = acc;
        if (e == 0) l_s[g] = l;
        __syncthreads();
        if (g == 0) {
#pragma unroll
            for (int i = 1; i < GROUPS; ++i) {
                const float4 v = acc_s[i][e];
                acc.x += v.x;
                acc.y += v.y;
                acc.z += v.z;
                acc.w += v.w;
                l += l_s[i];
            }
            write(acc, l, M, c);
        }
        __syncthreads();
    }
}

}  // namespace attn_sm100
