// attn_paged_kernel.cuh - attention of each sequence's newest tokens over
// pages of keys and values.
//
// The mathematics and the MMAs are those of attn_decode_kernel.cuh: a key/value
// head's G * T query rows are the columns of S^T = K q^T and O^T += V^T P^T over
// tiles of 128 positions, both on the tensor cores, because the step is bound
// by reading each key and value once and has a few hundred instructions per
// tile to spare. What differs:
//   - a tile is a gather: lane l of the producer warp loads page l of the tile
//     (or the whole tile out of one larger page) as TMA boxes of 64 columns x
//     min(page, 128) rows. Eight rows are one 128-byte-swizzle atom, so pages
//     of 8 and more stack into the operand layout that the MMAs read.
//   - lengths are on the device and differ: the work is dealt out in equal runs
//     of tiles (attn_paged_plan.cuh). A block goes through the segments of its
//     run without draining the pipeline: the ring of K and V tiles runs on
//     across them, q is double-buffered.
//   - more than 16 columns use N = 32, with two groups of softmax warps for 16
//     columns each, and beyond 32 blocks of 32.
//   - the four warps exchange a tile's maxima, and O^T in TMEM is rescaled, only
//     when a vote says that a column's maximum grew. (It is followed exactly, as
//     there: a row's largest weight is then 1 and exact in bf16. A maximum that
//     may lag by 2^8 rounds it, which for peaked rows is the product's whole
//     error: 1.2e-3 instead of 0.4e-3 at scores of standard deviation 6. It saves
//     nothing where the memory bounds the call; the chunks of 64 tokens below
//     take 264 us with it and 301 without.)
// What bounds it: HBM. 64 ragged sequences of 1000 to 8192 tokens (8 key/value
// heads, 4 query heads each, d = 128, 16-token pages): 179 us for 1.21 GB, 6.7
// TB/s (a plain copy reads and writes at 6.55). Two sequences of 131072 and 65500
// tokens, 16 columns: 40 us for 201 MB, of which a quarter is what every call has,
// start, pipeline fill and joining (5 us for one sequence of 77 tokens). At d = 64
// a tile is half the bytes at the same cost of barriers and votes: the ragged batch
// takes 101 us for 603 MB, 6.0 TB/s, 11 sequences x 3 heads of 17,000 tokens 31 for
// 144 MB. Beyond 32 columns blocks of 32 take the pages again, out of L2, and a
// tile's softmax, one after the other with its products, is what counts: the 64
// newest tokens of 8192 x 4 heads for 8 key/value heads, 8 sequences, take 301 us,
// 0.23 PFLOP/s. The ring of 96 KB and two blocks an SM keep 192 KB of loads in
// flight, four times what the latency asks for. One warp issues both kinds of
// MMAs: with a warp for each, S(i + 1) no longer waits in front of PV(i), but the
// ragged batch took 193 us instead of 181.
// A tile's positions that no token sees (before the window, behind the length,
// or whose table entry is no page, which are not loaded at all) have their
// scores replaced and their V rows zeroed before the products.
#pragma once
#include "attn_paged_plan.cuh"

namespace attn_sm100 {

struct PagedParams {
    PagedSplit split;
    __nv_bfloat16 *o;         // [B, H, T, D]
    float *lse;               // [B, H, T]
    float *part_o;            // see paged_slot
    float2 *part_ml;
    int *status;
    int H, Hkv, nblk;         // heads; column blocks of a group (gridDim.y = Hkv * nblk)
    PagedTable pages;
    float scale_log2;         // scale * log2(e)
};

constexpr int PAGED_TK = 128;  // positions per tile

// NC: columns the softmax handles.
template <int D, int NC>
struct PagedCfg {
    static_assert(D == 64 || D == 128, "head size 64 or 128");
    static_assert(NC == 4 || NC == 8 || NC == 16 || NC == 32, "columns");
    static constexpr int N = NC <= 16 ? 16 : 32;               // MMA N
    static constexpr int CTAS = NC <= 16 ? 2 : 1;              // blocks per SM
    static constexpr int GROUPS = NC <= 16 ? 1 : 2;            // softmax warpgroups, which share out the columns
    static constexpr int CG = NC / GROUPS;                     // columns of each
    static constexpr int THREADS = 64 + 128 * GROUPS;
    static constexpr int BOXES = D / BOX_COLS;                 // 64-column boxes per row
    static constexpr int BOX_BYTES_T = PAGED_TK * 128;         // [128 positions x 64 columns] bf16
    static constexpr int TILE_BYTES = BOXES * BOX_BYTES_T;     // one K or V tile
    static constexpr int NST = (CTAS == 2 ? 3 : 6) * 128 / D;  // ring stages (each one K or one V tile)
    static constexpr int OPB_BOX = N * 128;                    // N rows x 64 elements, 128-byte swizzle
    static constexpr int Q_BYTES = BOXES * OPB_BOX;            // N rows x D elements
    static constexpr int P_BYTES = 2 * OPB_BOX;                // N rows x 128 positions
    static constexpr int Q_OFF = NST * TILE_BYTES;             // two q buffers
    static constexpr int P_OFF = Q_OFF + 2 * Q_BYTES;          // P^T
    static constexpr int RED_OFF = P_OFF + P_BYTES;            // fp32, by group [3][CG][4 warps]
    static constexpr int COL_OFF = RED_OFF + 3 * 4 * NC * 4;   // float2 [NC]: reciprocal of the sum, maximum
    static constexpr int BAR_OFF = COL_OFF + NC * 8;
    // full[NST], empty[NST], q_full[2], q_empty[2], s_full[2], s_free[2], p_full, pv_done, mma_drain
    static constexpr int NBAR = 2 * NST + 11;
    static constexpr int MISC_OFF = BAR_OFF + NBAR * 8;        // TMEM base, abort flag
    static constexpr int PLAN_OFF = (MISC_OFF + 8 + 15) / 16 * 16;
    static constexpr int SMEM_BYTES = PLAN_OFF + PLAN_SCRATCH + 1024;  // + slack to align the base to 1 KB
    static constexpr uint32_t TMEM_COLS = N == 16 ? 64 : 128;
    static constexpr uint32_t S_COL = 0;                       // + N * buffer
    static constexpr uint32_t O_COL = 2 * N;
    static_assert(Q_OFF % 1024 == 0 && P_OFF % 1024 == 0 && Q_BYTES % 1024 == 0 && P_BYTES % 1024 == 0,
                  "operand alignment");
    static_assert(CTAS * (SMEM_BYTES + 1024) <= 233472, "blocks per SM");
};

template <int CG>
__device__ __forceinline__ void paged_tmem_ld(uint32_t taddr, uint32_t (&r)[CG < 8 ? 8 : CG])
{
    if constexpr (CG <= 8) {
        tmem_ld8(taddr, r);
    } else {
        tmem_ld16(taddr, r);
    }
}

template <int CG>
__device__ __forceinline__ void paged_tmem_st(uint32_t taddr, const uint32_t (&r)[CG < 8 ? 8 : CG])
{
    if constexpr (CG <= 8) {
        tmem_st8(taddr, r);
    } else {
        tmem_st16(taddr, r);
    }
}

template <int D, int NC>
__global__ void __launch_bounds__((PagedCfg<D, NC>::THREADS), (PagedCfg<D, NC>::CTAS))
    attn_paged_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ CUtensorMap tmV, const PagedParams p)
{
    using C = PagedCfg<D, NC>;
    using Walk = PagedWalk<PAGED_TK>;
    constexpr int N = C::N;
    constexpr int NST = C::NST;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *const base_ptr = smem_raw + (base - raw);
    auto ring = [&](int st) { return base + st * C::TILE_BYTES; };
    auto sQ = [&](int qb) { return base + C::Q_OFF + qb * C::Q_BYTES; };
    const uint32_t sP = base + C::P_OFF;
    float4 *const red_all = reinterpret_cast<float4 *>(base_ptr + C::RED_OFF);
    float2 *const col_all = reinterpret_cast<float2 *>(base_ptr + C::COL_OFF);
    const uint32_t bars = base + C::BAR_OFF;
    auto full = [&](int st) { return bars + 8u * st; };
    auto empty = [&](int st) { return bars + 8u * (NST + st); };
    auto bar2 = [&](int which, int i) { return bars + 8u * (2 * NST + 2 * which + i); };
    auto q_full = [&](int i) { return bar2(0, i); };
    auto q_empty = [&](int i) { return bar2(1, i); };
    auto s_full = [&](int i) { return bar2(2, i); };
    auto s_free = [&](int i) { return bar2(3, i); };
    const uint32_t p_full = bar2(4, 0), pv_done = bar2(4, 1), mma_drain = bar2(5, 0);
    uint32_t *const tmem_slot = reinterpret_cast<uint32_t *>(base_ptr + C::MISC_OFF);
    volatile int *const abort_flag = reinterpret_cast<volatile int *>(base_ptr + C::MISC_OFF + 4);

    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x / 32), 0);
    const int lane = static_cast<int>(threadIdx.x % 32);
    const int T = p.split.T;
    const int G = p.H / p.Hkv;
    const int head = blockIdx.y / p.nblk;            // key/value head
    const int c0 = (blockIdx.y % p.nblk) * NC;       // first column of this block
    // first q row of sequence b's columns: row c0 of its group
    auto first_row = [&](int b) { return (b * p.H + head * G) * T + c0; };

    if (warp == 0) {
        // (a barrier a lane: one thread would take half a microsecond for them)
        for (int i = lane; i < C::NBAR; i += 32) {
            const uint32_t bar = bars + 8u * i;
            const bool by_softmax = bar == s_free(0) || bar == s_free(1) || bar == p_full;
            mbar_init(bar, by_softmax ? C::GROUPS * 128 : 1);
        }
        if (lane == 0) *abort_flag = 0;
        fence_mbar_init();
        if (lane < 3) tma_prefetch_desc(lane == 0 ? &tmQ : lane == 1 ? &tmK : &tmV);
        __syncwarp();
    }
    if (warp == 1) {
        tmem_alloc(smem_addr(tmem_slot), C::TMEM_COLS);
        tmem_relinquish();
    }
    // rows >= NC of P^T meet columns of O^T that nobody reads; NaN there is
    // harmless, but let them be defined
    if constexpr (NC < N) {
        for (int i = threadIdx.x; i < C::P_BYTES / 16; i += C::THREADS)
            st_shared_v4(sP + i * 16, 0u, 0u, 0u, 0u);
        fence_proxy_async_smem();
    }
    tc_fence_before();
    // Nothing of the inputs or the workspace is touched before. (The joining
    // kernel may start once every block is here: it reads the lengths at once.)
    grid_dependency_wait();
    grid_dependents_launch();
    // (synchronises the block)
    const PagedRun run = paged_run<PAGED_TK, C::THREADS>(p.split, blockIdx.x, base_ptr + C::PLAN_OFF);
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const Waiter wt{abort_flag, p.status};
    const int count = run.count;

    if (count == 0) {
        // fewer tiles than blocks: nothing to do
    } else if (warp == 0) {
        // ------------------------------------------------------------ TMA producer
        const uint32_t leader = elect_one();
        const int page = 1 << p.pages.page_log2;
        const int npg = max(1, PAGED_TK >> p.pages.page_log2);  // pages per tile, one per lane
        const int rows = min(page, PAGED_TK);
        Walk w = run.walk<PAGED_TK>(p.split);
        auto lane_page = [&]() {
            const int at = w.base() + lane * page;
            return lane < npg ? paged_page(p.split, p.pages, w.s, w.b, npg == 1 ? at & ~(page - 1) : at) : -1;
        };
        int id = lane_page();
        int items = 0, segs = 0;
        bool ok = true;
        for (int i = 0; ok && i < count; ++i) {
            const int cur = id, b = w.b;
            const int row = npg == 1 ? w.base() & (page - 1) : 0;  // within the page
            const bool starts = i == 0 || w.j == 0;
            // the next tile's table entries travel while this one is issued
            if (i + 1 < count) {
                w.step(p.split);
                id = lane_page();
            }
            if (starts) {
                const int qb = segs % 2;
                if (segs >= 2) ok = __all_sync(0xffffffffu, wt.wait(q_empty(qb), ((segs / 2) - 1) & 1u));
                if (!ok) break;
                if (leader) {
                    mbar_arrive_expect_tx(q_full(qb), C::Q_BYTES);
                    for (int bx = 0; bx < C::BOXES; ++bx)
                        tma_load_2d(sQ(qb) + bx * C::OPB_BOX, &tmQ, q_full(qb), bx * BOX_COLS, first_row(b));
                }
                ++segs;
            }
            const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, cur >= 0)) * rows * (128 * C::BOXES);
            for (int kv = 0; kv < 2; ++kv, ++items) {
                const int st = items % NST;
                if (items >= NST) ok = __all_sync(0xffffffffu, wt.wait(empty(st), ((items / NST) - 1) & 1u));
                if (!ok) break;
                if (leader) mbar_arrive_expect_tx(full(st), bytes);
                __syncwarp();
                if (cur >= 0) {
                    const CUtensorMap *const map = kv ? &tmV : &tmK;
                    const uint32_t dst = ring(st) + lane * rows * 128;
#pragma unroll
                    for (int bx = 0; bx < C::BOXES; ++bx)
                        tma_load_4d(dst + bx * C::BOX_BYTES_T, map, full(st), bx * BOX_COLS, row, head, cur);
                }
                __syncwarp();
            }
        }
        // copies still in flight must land before the CTA exits
        for (int st = 0; st < NST; ++st) {
            if (items > st) wt.drain(full(st), ((items - 1 - st) / NST) & 1u);
        }
        for (int qb = 0; qb < 2; ++qb) {
            if (segs > qb) wt.drain(q_full(qb), ((segs - 1 - qb) / 2) & 1u);
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer
        const uint32_t leader = elect_one();
        constexpr uint32_t idesc_s = idesc_bf16_f32(PAGED_TK, N, 0, 0);  // K, q both K-major
        constexpr uint32_t idesc_o = idesc_bf16_f32(D, N, 1, 0);         // V^T MN-major, P^T K-major
        // where the next scores and the next products are
        Walk ws = run.walk<PAGED_TK>(p.split), wo = ws;
        int segs = 0;  // segments whose q has been waited for
        // S(i) = K_i q^T into S buffer i % 2
        auto issue_s = [&](int i) -> bool {
            if (i == 0 || ws.j == 0) {
                if (!__all_sync(0xffffffffu, wt.wait(q_full(segs % 2), (segs / 2) & 1u))) return false;
                ++segs;
            }
            const int qb = (segs - 1) % 2;
            const int item = 2 * i, st = item % NST;
            if (!__all_sync(0xffffffffu, wt.wait(full(st), (item / NST) & 1u))) return false;
            // the softmax must have read S(i - 2) out of this buffer
            if (i >= 2 && !__all_sync(0xffffffffu, wt.wait(s_free(i % 2), ((i - 2) / 2) & 1u))) return false;
            tc_fence_after();
            const uint64_t kdesc = smem_desc_sw128(ring(st), 16, 1024);
            const uint64_t qdesc = smem_desc_sw128(sQ(qb), 16, 1024);
            const uint32_t d_col = tmem + C::S_COL + N * (i % 2);
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                const uint64_t koff = static_cast<uint64_t>(((k / 4) * C::BOX_BYTES_T + (k % 4) * 32) >> 4);
                const uint64_t qoff = static_cast<uint64_t>(((k / 4) * C::OPB_BOX + (k % 4) * 32) >> 4);
                mma_bf16_ss_if(leader, d_col, kdesc + koff, qdesc + qoff, idesc_s, k > 0 ? 1u : 0u);
            }
            mma_commit_if(leader, s_full(i % 2));
            mma_commit_if(leader, empty(st));
            if (ws.last()) mma_commit_if(leader, q_empty(qb));
            if (i + 1 < count) ws.step(p.split);
            return true;
        };
        // O^T += V_i^T P_i^T; a segment's first tile starts from zero
        auto issue_pv = [&](int i) -> bool {
            const int item = 2 * i + 1, st = item % NST;
            if (!__all_sync(0xffffffffu, wt.wait(full(st), (item / NST) & 1u))) return false;
            if (!__all_sync(0xffffffffu, wt.wait(p_full, i & 1u))) return false;
            tc_fence_after();
            const uint32_t more = (i == 0 || wo.j == 0) ? 0u : 1u;
            const uint64_t vdesc = smem_desc_sw128(ring(st), C::BOX_BYTES_T, 1024);
            const uint64_t pdesc = smem_desc_sw128(sP, 16, 1024);
#pragma unroll
            for (int k = 0; k < PAGED_TK / 16; ++k) {
                const uint64_t poff = static_cast<uint64_t>(((k / 4) * C::OPB_BOX + (k % 4) * 32) >> 4);
                mma_bf16_ss_if(leader, tmem + C::O_COL, vdesc + static_cast<uint64_t>(k * 128), pdesc + poff,
                               idesc_o, k > 0 ? 1u : more);
            }
            mma_commit_if(leader, pv_done);
            mma_commit_if(leader, empty(st));
            if (i + 1 < count) wo.step(p.split);
            return true;
        };
        bool ok = issue_s(0);
        for (int i = 0; ok && i < count; ++i) {
            if (i + 1 < count) ok = issue_s(i + 1);
            if (ok) ok = issue_pv(i);
        }
        // every MMA this warp issued must finish before TMEM is freed
        mma_commit_if(leader, mma_drain);
        wt.drain(mma_drain, 0);
    } else {
        // ------------------------------------------------------------ softmax
        constexpr int CG = C::CG;
        constexpr int NR = CG < 8 ? 8 : CG;         // TMEM columns read per load
        const int grp = C::GROUPS == 1 ? 0 : (warp - 2) / 4, g0 = grp * CG;  // the group's first column
        const int cg0 = c0 + g0, ncol = min(G * T - cg0, CG);
        float4 *const red = red_all + grp * 3 * CG;  // [3][CG]: the four warps
        float2 *const col_s = col_all + g0;
        const int sw = warp % 4;                    // TMEM subpartition of this warp
        const int r = sw * 32 + lane;               // position in the tile (= TMEM lane)
        // column of d that O^T holds in this thread's lane (d = 64: lanes
        // 16-31 of each quarter hold none)
        const int dcol = (D == 128) ? r : 16 * sw + lane;
        const bool has_dcol = (D == 128) || lane < 16;
        const uint32_t lane_base = tmem + (static_cast<uint32_t>(sw * 32) << 16);
        const float sc = p.scale_log2;
        const int window = p.split.window;
        Walk w = run.walk<PAGED_TK>(p.split);
        auto slot_page = [&]() { return paged_page(p.split, p.pages, w.s, w.b, (w.base() + r) & ~((1 << p.pages.page_log2) - 1)); };
        int id = slot_page();
        float m_run[CG], l_part[CG];
        bool ok = true;
        int seg_j = run.j;  // where the segment began
        for (int i = 0; i < count; ++i) {
            const int sb = i % 2;
            const Walk cur = w;
            // (by votes, here and below: branches that the compiler knows to be
            // taken by whole warps)
            const bool starts = __any_sync(0xffffffffu, i == 0 || cur.j == 0);
            const bool ends = __any_sync(0xffffffffu, i + 1 == count || cur.last());
            const int at = cur.base() + r;           // this thread's position
            const int len = cur.s.len;
            // Seen by a token at all, and by all of them? (id >= 0 says that
            // some position of its page is.)
            const int oldest = window >= 0 ? max(0, len - T - window) : 0;
            const bool seen = id >= 0 && at < len && at >= oldest;
            const bool by_all = seen && at <= len - T && (window < 0 || at >= len - 1 - window);
            const bool plain = __all_sync(0xffffffffu, by_all);
            if (i + 1 < count) {
                w.step(p.split);
                id = slot_page();
            }
            if (starts) {
#pragma unroll
                for (int c = 0; c < CG; ++c) {
                    m_run[c] = -CUDART_INF_F;
                    l_part[c] = 0.f;
                }
                seg_j = cur.j;
            }
            bool okw = __all_sync(0xffffffffu, wt.wait(s_full(sb), (i / 2) & 1u));
            float s[CG];
            if (okw) {
                tc_fence_after();
                uint32_t sv[NR];
                paged_tmem_ld<CG>(lane_base + C::S_COL + N * sb + g0, sv);
                tc_fence_before();
                mbar_arrive(s_free(sb));
                if (plain) {
#pragma unroll
                    for (int c = 0; c < CG; ++c) s[c] = __uint_as_float(sv[c]) * sc;
                } else {
#pragma unroll
                    for (int c = 0; c < CG; ++c) s[c] = seen ? __uint_as_float(sv[c]) * sc : -CUDART_INF_F;
                    if (T > 1) {
                        // (at = len - T + t: seen by the tokens t .. t + window)
                        const int t0 = at - (len - T), t1 = window < 0 ? T : t0 + window;
#pragma unroll
                        for (int c = 0; c < CG; ++c) {
                            const int u = (cg0 + c) % T;
                            s[c] = u >= t0 && u <= t1 ? s[c] : -CUDART_INF_F;
                        }
                    }
                }
            }
            // Does a score exceed its column's maximum so far? Then the warps
            // take the tile's maxima.
            bool above = false;
            if (okw) {
#pragma unroll
                for (int c = 0; c < CG; ++c) above = above || s[c] > m_run[c];
            }
            bool raised = false;
            float alpha[CG];
            // (ok carries a wait that gave up later in the previous tile)
            if (!__all_sync(0xffffffffu, named_bar_and(1 + grp, 4 * 32, okw && ok && !above))) {
                if (okw) {
                    float mine = -CUDART_INF_F;  // lane c holds column c's maximum
#pragma unroll
                    for (int c = 0; c < CG; ++c) {
                        const float mx = redux_max(s[c]);
                        mine = lane == c ? mx : mine;
                    }
                    if (lane < CG) reinterpret_cast<float *>(&red[sb * CG + lane])[sw] = mine;
                    __syncwarp();
                }
                ok = __all_sync(0xffffffffu, named_bar_and(1 + grp, 4 * 32, okw && ok));
                if (!ok) break;
#pragma unroll
                for (int c = 0; c < CG; ++c) {
                    const float4 m4 = red[sb * CG + c];
                    const float tmax = fmaxf(fmaxf(m4.x, m4.y), fmaxf(m4.z, m4.w));
                    const bool up = tmax > m_run[c];
                    alpha[c] = up ? ex2_approx(m_run[c] - tmax) : 1.f;
                    l_part[c] *= alpha[c];
                    m_run[c] = up ? tmax : m_run[c];
                    raised = raised || up;
                }
                raised = __any_sync(0xffffffffu, raised);
            }
            float pr[CG];
#pragma unroll
            for (int c = 0; c < CG; ++c) {
                // measure from 0 while there is no position, so that no
                // (-inf) - (-inf) arises; masked positions give 0
                const float m_ref = (m_run[c] == -CUDART_INF_F) ? 0.f : m_run[c];
                pr[c] = ex2_approx(s[c] - m_ref);
                l_part[c] += pr[c];
            }
            // P^T was last read by PV(i - 1), and O^T then holds the segment's
            // tiles before i (every thread decides alike whether to rescale it:
            // all read the same maxima)
            if (i >= 1) okw = __all_sync(0xffffffffu, wt.wait(pv_done, (i - 1) & 1u));
            if (okw && !starts && raised) {
                tc_fence_after();
                uint32_t o[NR];
                paged_tmem_ld<CG>(lane_base + C::O_COL + g0, o);
#pragma unroll
                for (int c = 0; c < CG; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * alpha[c]);
                paged_tmem_st<CG>(lane_base + C::O_COL + g0, o);
                tmem_wait_st();
            }
            // Positions no token sees: their V rows may hold anything (slots
            // nothing was written to, or what the ring held before), and
            // 0 * NaN would reach O. Each warp zeroes its own rows.
            if (okw && __any_sync(0xffffffffu, !seen)) {
                const int item = 2 * i + 1, st = item % NST;
                okw = __all_sync(0xffffffffu, wt.wait(full(st), (item / NST) & 1u));
                if (okw && !seen) {
#pragma unroll
                    for (int bx = 0; bx < C::BOXES; ++bx)
#pragma unroll
                        for (int e = grp * (8 / C::GROUPS); e < (grp + 1) * (8 / C::GROUPS); ++e)  // (in an order that spreads the rows over the banks)
                            st_shared_v4(ring(st) + bx * C::BOX_BYTES_T + r * 128 + ((e ^ (r & 7)) * 16), 0u, 0u, 0u, 0u);
                }
                __syncwarp();
            }
            if (okw) {
                // P^T: row c, column r; rounded to bf16 for the product, as the
                // forward's weights are
                const uint32_t col = sP + (r / 64) * C::OPB_BOX +
                                     ((static_cast<uint32_t>((r % 64) / 8)) * 16) + (r % 8) * 2;
#pragma unroll
                for (int c = 0; c < CG; ++c) {
                    const uint32_t addr = (col + (g0 + c) * 128) ^ (static_cast<uint32_t>(c & 7) << 4);
                    const unsigned short h = __bfloat16_as_ushort(__float2bfloat16_rn(pr[c]));
                    asm volatile("st.shared.u16 [%0], %1;" ::"r"(addr), "h"(h) : "memory");
                }
                fence_proxy_async_smem();
                tc_fence_before();
                mbar_arrive(p_full);
            }
            ok = okw;
            if (ends) {
                // ---------------------------------------------------- the segment's results
                float mine = 0.f;
#pragma unroll
                for (int c = 0; c < CG; ++c) {
                    float sum = l_part[c];
#pragma unroll
                    for (int o = 16; o >= 1; o /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                    mine = lane == c ? sum : mine;
                }
                if (lane < CG) reinterpret_cast<float *>(&red[2 * CG + lane])[sw] = mine;
                if (r == 0) {
#pragma unroll
                    for (int c = 0; c < CG; ++c) col_s[c].y = m_run[c];
                }
                __syncwarp();
                if (ok) ok = __all_sync(0xffffffffu, wt.wait(pv_done, i & 1u));
                ok = __all_sync(0xffffffffu, named_bar_and(1 + grp, 4 * 32, ok));
                if (!ok) break;
                tc_fence_after();
                const bool whole = __any_sync(0xffffffffu, seg_j == 0 && cur.last());
                const int64_t row = first_row(cur.b) + g0;
                const int64_t slot = paged_slot(blockIdx.x, blockIdx.y, p.split.ranges, cur.b == run.b) * NC + g0;
                if (r < CG) {
                    const float4 l4 = red[2 * CG + r];
                    const float l = (l4.x + l4.y) + (l4.z + l4.w), m = col_s[r].y;
                    if (whole) {
                        col_s[r].x = l == 0.f ? 0.f : 1.f / l;
                        if (r < ncol) p.lse[row + r] = l == 0.f ? -CUDART_INF_F : (m + __log2f(l)) * 0.69314718055994531f;
                    } else {
                        p.part_ml[slot + r] = make_float2(m, l);
                    }
                }
                __syncwarp();
                named_bar_sync(1 + grp, 4 * 32);
                // (a short loop: this runs once a segment, and what it costs is
                // above all fetching its instructions)
#pragma unroll 1
                for (int c8 = 0; c8 < CG; c8 += 8) {
                    uint32_t o[8];
                    tmem_ld8(lane_base + C::O_COL + g0 + c8, o);
                    __nv_bfloat16 *const out = p.o + (row + c8) * D + dcol;
                    float *const part = p.part_o + (slot + c8) * D + dcol;
#pragma unroll
                    for (int c = 0; c < (CG < 8 ? CG : 8); ++c) {
                        const float v = __uint_as_float(o[c]);
                        if (whole) {
                            const float x = v * col_s[c8 + c].x;
                            if (has_dcol && c8 + c < ncol) out[c * D] = __float2bfloat16_rn(x);
                        } else if (has_dcol) {
                            part[c * D] = v;  // (the slot has room for columns not in use)
                        }
                    }
                }
                tc_fence_before();
                // (the next segment's sums and factors are written behind the
                // barrier of its first tile)
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, C::TMEM_COLS);
    }
}

}  // namespace attn_sm100
