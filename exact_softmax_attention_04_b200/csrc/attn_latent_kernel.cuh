// attn_latent_kernel.cuh - attention of each sequence's newest tokens over
// pages of latent vectors, shared by all heads.
//
// A row of the cache, R + 64 elements, is the key of every head and its first R
// elements are the value. The H * T query rows of a sequence are the columns
// of (tile: 64 positions, C its rows)
//   S^T  = C q^T            M = 64 positions, K = R + 64: C K-major;
//   O^T += C[:, :R]^T P^T   M = R, as blocks of 128, K = 64 positions: the same
//                           bytes of shared memory as an MN-major operand,
// so a tile is loaded once and used twice: up to 242 operations a byte at 128
// heads, where the tensor cores' rate and the memory's are both near. 64 columns
// a block is the most that O^T (R x 64 in fp32: half of TMEM at R = 512), q (72 KB)
// and two tiles of 72 KB leave room for; 128 heads are two blocks that read the
// same tiles at the same time, the second out of L2.
//
// What bounds it. Up to 16 columns HBM: 48 ragged sequences of 1500 to 16384
// tokens, 16 heads, R = 512: 95 us for 496 MB, 5.2 TB/s.
// At 64 columns the two places for tiles: an M = 64 instruction takes 31 cycles
// at N = 64 (23 at N = 16: its operands' 2 to 4 KB of shared memory a step), an
// M = 128 one 47, so a tile's 36 + 16 instructions take 2100 cycles, but load,
// scores, softmax, rescaling and products in turn take a place for some 8000, 4000 a
// tile: 32 sequences x 128 heads of 2000 to 8192 tokens take 90 us against 30 at
// the rates of the memory and of the tensor cores. Hence the parts of a tile that are
// freed and loaded one by one, a softmax group for each 16 columns (94 us with two
// groups of 32, whose chains are longer; R = 256: 62 instead of 70), a warp for each
// kind of MMAs, and two producers (33 -> 27 us for 23 sequences of 2000 to 8192 tokens
// in 8-token pages, 32 columns, R = 256). The maximum is followed exactly, so that a
// row's largest weight is 1 and exact in bf16 (see attn_paged_kernel.cuh): O^T is
// rescaled in nearly every tile of a short sequence, and one that may lag by 2^8
// takes 80 us here. Bringing the next tile into L2 by TMA ahead of time made it
// slower.
//
// Roles as in attn_paged_kernel.cuh. With M = 64, S^T lies in the lower 16 lanes
// of each quarter of TMEM; read as 8 x 8 blocks, all 32 threads of a warp get a
// share of them, and P^T goes to shared memory by transposing stores. A thread
// has 2 positions of a quarter of the columns; maxima over a tile go through three
// shuffles and then between the four warps. The groups of four warps, 16 columns
// each, need nothing of one another.
#pragma once
#include "attn_paged_plan.cuh"

namespace attn_sm100 {

struct LatentParams {
    PagedSplit split;
    PagedTable pages;
    __nv_bfloat16 *o;         // [B, H, T, R]
    float *lse;               // [B, H, T]
    float *part_o;            // see paged_slot
    float2 *part_ml;
    int *status;
    int GT;                   // query rows of a sequence, H * T
    float scale_log2;         // scale * log2(e)
};

constexpr int LATENT_TK = 64;  // positions per tile

template <int R, int NC>
struct LatentCfg {
    static_assert(R == 256 || R == 512, "rank 256 or 512");
    static_assert(NC == 16 || NC == 32 || NC == 64, "columns");
    static constexpr int CG = 16;                              // columns of a softmax warpgroup
    static constexpr int GROUPS = NC / CG;
    static constexpr int THREADS = 128 + 128 * GROUPS;         // two producers, two MMA warps, the groups
    static constexpr int BOXES = R / 64 + 1;                   // 64-column boxes per row
    static constexpr int BLOCKS = R / 128;                     // blocks of O^T
    // A tile's parts, loaded, used and freed one by one: for each block of O^T
    // its two boxes, and last the box that is no value. In a part, eight rows of
    // its first box are followed by the same rows of the second, so that a page
    // is one TMA copy a part whatever its size.
    static constexpr int PARTS = BLOCKS + 1;
    static constexpr int PART_BYTES = 2 * LATENT_TK * 128;
    static constexpr int BOX_BYTES_T = LATENT_TK * 128;        // [64 positions x 64 columns] bf16
    static constexpr int TILE_BYTES = BOXES * BOX_BYTES_T;
    static constexpr int OPB_BOX = NC * 128;                   // NC rows x 64 elements
    static constexpr int Q_BYTES = BOXES * OPB_BOX;
    static constexpr int P_BYTES = OPB_BOX;                    // NC rows x 64 positions
    static constexpr int TAIL = 2 * 4 * NC * 4 + NC * 8 + 512; // what follows the operands, at most
    static constexpr int NST = (232448 - Q_BYTES - P_BYTES - TAIL) / TILE_BYTES;
    static constexpr int Q_OFF = NST * TILE_BYTES;
    static constexpr int P_OFF = Q_OFF + Q_BYTES;
    static constexpr int RED_OFF = P_OFF + P_BYTES;            // fp32 [2][4 warps][NC]
    static constexpr int COL_OFF = RED_OFF + 2 * 4 * NC * 4;   // float2 [NC]: reciprocal of the sum, maximum
    static constexpr int BAR_OFF = COL_OFF + NC * 8;
    // full[NST][PARTS], empty[NST][PARTS], s_full[2], s_free[2], q_full, q_empty, p_full, pv_done, mma_drain[2]
    static constexpr int NBAR = 2 * NST * PARTS + 10;
    static constexpr int PLAN_OFF = (BAR_OFF + NBAR * 8 + 15) / 16 * 16;
    static constexpr int MISC_OFF = PLAN_OFF + PLAN_SCRATCH;   // TMEM base, abort flag
    // (no slack for alignment: the kernel has no other shared memory, and
    // checks that its base is a multiple of 1 KB)
    static constexpr int SMEM_BYTES = MISC_OFF + 16;
    static constexpr uint32_t O_COL = 2 * NC;                  // behind two S buffers
    static constexpr uint32_t TMEM_NEED = 2 * NC + BLOCKS * NC;
    static constexpr uint32_t TMEM_COLS = TMEM_NEED <= 128 ? 128 : TMEM_NEED <= 256 ? 256 : 512;
    static_assert(NST >= 2 && SMEM_BYTES <= 232448, "shared memory");
    static_assert(Q_OFF % 1024 == 0 && P_OFF % 1024 == 0, "operand alignment");
};

template <int R, int NC>
__global__ void __launch_bounds__((LatentCfg<R, NC>::THREADS), 1)
    attn_latent_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmC,
                       const __grid_constant__ CUtensorMap tmLast, const LatentParams p)
{
    using C = LatentCfg<R, NC>;
    using Walk = PagedWalk<LATENT_TK>;
    constexpr int NST = C::NST;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t base = smem_addr(smem_raw);
    auto ring = [&](int st) { return base + st * C::TILE_BYTES; };
    const uint32_t sQ = base + C::Q_OFF, sP = base + C::P_OFF;
    float *const red_all = reinterpret_cast<float *>(smem_raw + C::RED_OFF);
    float2 *const col_all = reinterpret_cast<float2 *>(smem_raw + C::COL_OFF);
    const uint32_t bars = base + C::BAR_OFF;
    auto full = [&](int st, int part) { return bars + 8u * (st * C::PARTS + part); };
    auto empty = [&](int st, int part) { return bars + 8u * ((NST + st) * C::PARTS + part); };
    auto bar1 = [&](int i) { return bars + 8u * (2 * NST * C::PARTS + i); };
    auto s_full = [&](int i) { return bar1(i); };
    auto s_free = [&](int i) { return bar1(2 + i); };
    const uint32_t q_full = bar1(4), q_empty = bar1(5), p_full = bar1(6), pv_done = bar1(7);
    auto mma_drain = [&](int i) { return bar1(8 + i); };
    uint32_t *const tmem_slot = reinterpret_cast<uint32_t *>(smem_raw + C::MISC_OFF);
    volatile int *const abort_flag = reinterpret_cast<volatile int *>(smem_raw + C::MISC_OFF + 4);

    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x / 32), 0);
    const int lane = static_cast<int>(threadIdx.x % 32);
    const int T = p.split.T;
    const int c0 = blockIdx.y * NC;                  // first column of this block

#ifdef ATTN_FAULT_LATENT_SMEM_BASE
    const bool usable = false;
#else
    const bool usable = base % 1024 == 0;  // (the operands' swizzle needs it)
#endif
    if (!usable) {
        // nothing is computed, but the joining kernel finds its plan
        if (threadIdx.x == 0) atomicOr(p.status, STATUS_SMEM_ALIGN);
        grid_dependency_wait();
        paged_run<LATENT_TK, C::THREADS>(p.split, blockIdx.x, smem_raw + C::PLAN_OFF);
        return;
    }
    if (warp == 0) {
        // (a barrier a lane: one thread would take half a microsecond for them)
        for (int i = lane; i < C::NBAR; i += 32) {
            const uint32_t bar = bars + 8u * i;
            const bool by_softmax = bar == s_free(0) || bar == s_free(1) || bar == p_full;
            mbar_init(bar, by_softmax ? C::GROUPS * 128 : 1);
        }
        if (lane == 0) *abort_flag = 0;
        fence_mbar_init();
        if (lane < 3) tma_prefetch_desc(lane == 0 ? &tmQ : lane == 1 ? &tmC : &tmLast);
        __syncwarp();
    }
    if (warp == 1) {
        tmem_alloc(smem_addr(tmem_slot), C::TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    // Nothing of the inputs or the workspace is touched before. (The joining
    // kernel may start once every block is here: it reads the lengths at once.)
    grid_dependency_wait();
    grid_dependents_launch();
    // (synchronises the block)
    const PagedRun run = paged_run<LATENT_TK, C::THREADS>(p.split, blockIdx.x, smem_raw + C::PLAN_OFF);
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const Waiter wt{abort_flag, p.status};
    const int count = run.count;

    if (count == 0) {
        // fewer tiles than blocks: nothing to do
    } else if (warp == 0 || warp == 3 + 4 * C::GROUPS) {
        // ------------------------------------------------------------ TMA producers
        // The parts in turn by two warps: a copy costs its warp some 100 cycles,
        // and pages of 8 tokens make 24 (R = 256) or 40 of them a tile.
        const int producer = warp == 0 ? 0 : 1;
        const uint32_t leader = elect_one();
        const int page = 1 << p.pages.page_log2;
        const int npg = max(1, LATENT_TK >> p.pages.page_log2);  // pages per tile, one per lane
        const int rows = min(page, LATENT_TK);
        Walk w = run.walk<LATENT_TK>(p.split);
        auto lane_page = [&]() {
            const int at = w.base() + lane * page;
            return lane < npg ? paged_page(p.split, p.pages, w.s, w.b, npg == 1 ? at & ~(page - 1) : at) : -1;
        };
        int id = lane_page();
        int items = 0, segs = 0;
        int issued[C::PARTS];  // tiles of which this part was asked for
#pragma unroll
        for (int part = 0; part < C::PARTS; ++part) issued[part] = 0;
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
            const uint32_t have = __ballot_sync(0xffffffffu, cur >= 0);  // pages of the tile that there are
            const uint32_t bytes = __popc(have) * rows * 128;            // of a box
            const int st = items % NST;
            // (the part that is no value was freed first)
#pragma unroll
            for (int n = 0; n < C::PARTS; ++n) {
                constexpr int LAST = C::BLOCKS;
                const int part = n == 0 ? LAST : n - 1, boxes = n == 0 ? 1 : 2;
                if (n % 2 != producer) continue;
                if (items >= NST)
                    ok = ok && __all_sync(0xffffffffu, wt.wait(empty(st, part), ((items / NST) - 1) & 1u));
                if (!ok) break;
                mbar_arrive_expect_tx_if(leader, full(st, part), bytes * boxes);
                for (int pg = 0; pg < npg; ++pg) {
                    if (!((have >> pg) & 1u)) continue;
                    const int page_id = __shfl_sync(0xffffffffu, cur, pg);
                    tma_load_5d_if(leader, ring(st) + part * C::PART_BYTES + pg * rows * (128 * boxes), n == 0 ? &tmLast : &tmC,
                                   full(st, part), 0, 0, 2 * part, row / 8, page_id);
                }
                issued[part] = items + 1;
            }
            if (!ok) break;
            ++items;
            if (starts && producer == 0) {
                if (segs >= 1) ok = __all_sync(0xffffffffu, wt.wait(q_empty, (segs - 1) & 1u));
                if (!ok) break;
                if (leader) {
                    mbar_arrive_expect_tx(q_full, C::Q_BYTES);
                    for (int bx = 0; bx < C::BOXES; ++bx)
                        tma_load_2d(sQ + bx * C::OPB_BOX, &tmQ, q_full, bx * BOX_COLS, b * p.GT + c0);
                }
                ++segs;
            }
        }
        // copies still in flight must land before the CTA exits
#pragma unroll
        for (int part = 0; part < C::PARTS; ++part) {
            for (int st = 0; st < NST && st < issued[part]; ++st)
                wt.drain(full(st, part), ((issued[part] - 1 - st) / NST) & 1u);
        }
        if (segs > 0) wt.drain(q_full, (segs - 1) & 1u);
    } else if (warp == 1) {
        // ------------------------------------------------------------ scores' MMAs
        const uint32_t leader = elect_one();
        constexpr uint32_t idesc_s = idesc_bf16_f32(LATENT_TK, NC, 0, 0);  // C, q both K-major
        const uint64_t qdesc = smem_desc_sw128(sQ, 16, 1024);
        Walk w = run.walk<LATENT_TK>(p.split);
        int segs = 0;  // segments whose q has been waited for
        bool ok = true;
        // S(i) = C_i q^T into S buffer i % 2, part by part as they land
        for (int i = 0; ok && i < count; ++i) {
            const int st = i % NST;
            if (i == 0 || w.j == 0) ok = __all_sync(0xffffffffu, wt.wait(q_full, segs++ & 1u));
            // the softmax must have read S(i - 2) out of this buffer
            if (ok && i >= 2) ok = __all_sync(0xffffffffu, wt.wait(s_free(i % 2), ((i - 2) / 2) & 1u));
            const uint64_t kdesc = smem_desc_sw128(ring(st), 16, 2048), ldesc = smem_desc_sw128(ring(st), 16, 1024);
            const uint32_t d_col = tmem + NC * (i % 2);
#pragma unroll
            for (int n = 0; n < C::PARTS; ++n) {
                const int part = n == 0 ? C::BLOCKS : n - 1;
                ok = ok && __all_sync(0xffffffffu, wt.wait(full(st, part), (i / NST) & 1u));
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int k = 0; k < (part < C::BLOCKS ? 8 : 4); ++k) {
                    const uint64_t koff = static_cast<uint64_t>((part * C::PART_BYTES + (k / 4) * 1024 + (k % 4) * 32) >> 4);
                    const uint64_t qoff = static_cast<uint64_t>(((2 * part + k / 4) * C::OPB_BOX + (k % 4) * 32) >> 4);
                    mma_bf16_ss_if(leader, d_col, (part < C::BLOCKS ? kdesc : ldesc) + koff, qdesc + qoff, idesc_s, n > 0 || k > 0 ? 1u : 0u);
                }
                if (n == 0) mma_commit_if(leader, empty(st, part));  // (not read again)
            }
            if (!ok) break;
            mma_commit_if(leader, s_full(i % 2));
            if (w.last()) mma_commit_if(leader, q_empty);
            if (i + 1 < count) w.step(p.split);
        }
        // every MMA this warp issued must finish before TMEM is freed
        mma_commit_if(leader, mma_drain(0));
        wt.drain(mma_drain(0), 0);
    } else if (warp == 2 + 4 * C::GROUPS) {
        // ------------------------------------------------------------ products' MMAs
        // A warp of their own: S(i + 1) waits for its tile, PV(i) for the
        // softmax, and neither may hold up the other (PV(i) frees the tile that
        // the load after next waits for).
        const uint32_t leader = elect_one();
        constexpr uint32_t idesc_o = idesc_bf16_f32(128, NC, 1, 0);  // C^T MN-major, P^T K-major
        const uint64_t pdesc = smem_desc_sw128(sP, 16, 1024);
        Walk w = run.walk<LATENT_TK>(p.split);
        // O^T += C_i[:, :R]^T P_i^T by blocks of rows; a segment's first tile
        // starts from zero
        for (int i = 0; i < count; ++i) {
            const int st = i % NST;
            const uint32_t more = (i == 0 || w.j == 0) ? 0u : 1u;
            if (i + 1 < count) w.step(p.split);
            if (!__all_sync(0xffffffffu, wt.wait(p_full, i & 1u))) break;
            tc_fence_after();
            const uint64_t vdesc = smem_desc_sw128(ring(st), 1024, 2048);
#pragma unroll
            for (int blk = 0; blk < C::BLOCKS; ++blk) {
#pragma unroll
                for (int k = 0; k < LATENT_TK / 16; ++k)
                    mma_bf16_ss_if(leader, tmem + C::O_COL + blk * NC,
                                   vdesc + static_cast<uint64_t>((blk * C::PART_BYTES + k * 4096) >> 4),
                                   pdesc + static_cast<uint64_t>(k * 2), idesc_o, k > 0 ? 1u : more);
                mma_commit_if(leader, empty(st, blk));
            }
            mma_commit_if(leader, pv_done);
        }
        mma_commit_if(leader, mma_drain(1));
        wt.drain(mma_drain(1), 0);
    } else {
        // ------------------------------------------------------------ softmax
        constexpr int CG = C::CG, NK = CG / 8;      // the group's columns, as blocks of 8
        const int grp = C::GROUPS == 1 ? 0 : (warp - 2) / 4, g0 = grp * CG;
        const int sw = warp % 4;                    // TMEM quarter: positions 16 sw + 0..15 of the tile
        const int rank_lane = sw * 32 + lane;       // row of an O^T block
        const uint32_t lane_base = tmem + (static_cast<uint32_t>(sw * 32) << 16);
        const int cc = 2 * (lane % 4);              // this thread's columns: 8 k + cc, 8 k + cc + 1
        const int rr = lane / 4;                    // its positions: 16 sw + rr and 8 further
        const int my_row = 16 * sw + lane % 16;     // the position whose page this lane looks up
        const float sc = p.scale_log2;
        float *const red = red_all + grp * 8 * CG;  // [2][4 warps][CG]
        float2 *const col_s = col_all + g0;
        Walk w = run.walk<LATENT_TK>(p.split);
        auto row_page = [&]() {
            return paged_page(p.split, p.pages, w.s, w.b, (w.base() + my_row) & ~((1 << p.pages.page_log2) - 1));
        };
        int id = row_page();
        float m_run[CG / 4], l_part[CG / 4];
        bool ok = true;
        int seg_j = run.j;  // where the segment began
        for (int i = 0; i < count; ++i) {
            const int sb = i % 2, st = i % NST;
            const Walk cur = w;
            // (by votes, here and below: branches that the compiler knows to be
            // taken by whole warps)
            const bool starts = __any_sync(0xffffffffu, i == 0 || cur.j == 0);
            const bool ends = __any_sync(0xffffffffu, i + 1 == count || cur.last());
            const int len = cur.s.len;
            // Seen by a token at all, and by all of them? Bits by row of the
            // warp's 16.
            const bool seen = id >= 0 && cur.base() + my_row < len;
            const uint32_t seen_rows = __ballot_sync(0xffffffffu, seen) & 0xffffu;
            const bool plain = __all_sync(0xffffffffu, seen && cur.base() + my_row <= len - T);
            if (i + 1 < count) {
                w.step(p.split);
                id = row_page();
            }
            if (starts) {
#pragma unroll
                for (int c = 0; c < CG / 4; ++c) {
                    m_run[c] = -CUDART_INF_F;
                    l_part[c] = 0.f;
                }
                seg_j = cur.j;
            }
            bool okw = __all_sync(0xffffffffu, wt.wait(s_full(sb), (i / 2) & 1u));
            float s[CG / 2];  // [8-column block][position rr, rr + 8][column]
            if (okw) {
                tc_fence_after();
                uint32_t sv[CG / 2];
                tmem_ld_half8(lane_base + NC * sb + g0, sv);
                tc_fence_before();
                mbar_arrive(s_free(sb));
#pragma unroll
                for (int e = 0; e < CG / 2; ++e) s[e] = __uint_as_float(sv[e]) * sc;
                if (!plain) {
                    const bool seen0 = (seen_rows >> rr) & 1u, seen1 = (seen_rows >> (rr + 8)) & 1u;
#pragma unroll
                    for (int e = 0; e < CG / 2; ++e) s[e] = ((e & 2) ? seen1 : seen0) ? s[e] : -CUDART_INF_F;
                    if (T > 1) {
                        // (at = len - T + t: seen by the tokens from t on)
                        const int t0 = cur.base() + 16 * sw + rr - (len - T);
#pragma unroll
                        for (int e = 0; e < CG / 2; ++e) {
                            const int c = c0 + g0 + 8 * (e / 4) + cc + (e & 1);
                            s[e] = c % T >= t0 + ((e & 2) ? 8 : 0) ? s[e] : -CUDART_INF_F;
                        }
                    }
                }
            }
            // Does a score exceed its column's maximum so far? Then the group
            // takes the tile's maxima.
            bool above = false;
            if (okw) {
#pragma unroll
                for (int e = 0; e < CG / 2; ++e)
                    above = above || s[e] > m_run[e / 4 * 2 + (e & 1)];
            }
            bool raised = false;
            float alpha[CG / 4];
            // (ok carries a wait that gave up later in the previous tile)
            if (!__all_sync(0xffffffffu, named_bar_and(1 + grp, 4 * 32, okw && ok && !above))) {
                if (okw) {
#pragma unroll
                    for (int k = 0; k < NK; ++k) {
                        float a = fmaxf(s[4 * k], s[4 * k + 2]), b = fmaxf(s[4 * k + 1], s[4 * k + 3]);
#pragma unroll
                        for (int o = 4; o <= 16; o *= 2) {
                            a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
                            b = fmaxf(b, __shfl_xor_sync(0xffffffffu, b, o));
                        }
                        if (lane < 4)
                            *reinterpret_cast<float2 *>(red + (sb * 4 + sw) * CG + 8 * k + cc) = make_float2(a, b);
                    }
                    __syncwarp();
                }
                ok = __all_sync(0xffffffffu, named_bar_and(1 + grp, 4 * 32, okw && ok));
                if (!ok) break;
#pragma unroll
                for (int c = 0; c < CG / 4; ++c) {
                    float tmax = -CUDART_INF_F;
#pragma unroll
                    for (int v = 0; v < 4; ++v) tmax = fmaxf(tmax, red[(sb * 4 + v) * CG + 8 * (c / 2) + cc + c % 2]);
                    const bool up = tmax > m_run[c];
                    alpha[c] = up ? ex2_approx(m_run[c] - tmax) : 1.f;
                    l_part[c] *= alpha[c];
                    m_run[c] = up ? tmax : m_run[c];
                    raised = raised || up;
                }
                // (a warp's lanes hold every column, with the same values in every warp)
                raised = __any_sync(0xffffffffu, raised);
            }
#pragma unroll
            for (int k = 0; k < NK; ++k) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int c = 2 * k + e;
                    // measure from 0 while there is no position, so that no
                    // (-inf) - (-inf) arises; masked positions give 0
                    const float m_ref = (m_run[c] == -CUDART_INF_F) ? 0.f : m_run[c];
                    const float p0 = ex2_approx(s[4 * k + e] - m_ref), p1 = ex2_approx(s[4 * k + 2 + e] - m_ref);
                    s[4 * k + e] = p0;
                    s[4 * k + 2 + e] = p1;
                    l_part[c] += p0 + p1;
                }
            }
            // P^T was last read by PV(i - 1), and O^T then holds the segment's
            // tiles before i
            if (i >= 1) okw = __all_sync(0xffffffffu, wt.wait(pv_done, (i - 1) & 1u));
            if (raised && !starts) {
                // A warp hands its factors round in its row of the maxima of
                // tile i - 1, which every warp has read by now.
                float *const factor = red + ((sb ^ 1) * 4 + sw) * CG;
                if (lane < 4) {
#pragma unroll
                    for (int c = 0; c < CG / 4; ++c) factor[8 * (c / 2) + cc + c % 2] = alpha[c];
                }
                __syncwarp();
                if (okw) {
                    tc_fence_after();
#pragma unroll 1
                    for (int blk = 0; blk < C::BLOCKS; blk += 2) {
                        const uint32_t at = lane_base + C::O_COL + blk * NC + g0;
                        uint32_t o[2 * CG], lo[CG], hi[CG];
                        tmem_ld16_two(at, at + NC, o);
#pragma unroll
                        for (int c = 0; c < CG; ++c) {
                            const float f = factor[c];
                            lo[c] = __float_as_uint(__uint_as_float(o[c]) * f);
                            hi[c] = __float_as_uint(__uint_as_float(o[CG + c]) * f);
                        }
                        tmem_st16(at, lo);
                        tmem_st16(at + NC, hi);
                    }
                    tmem_wait_st();
                }
            }
            // Positions no token sees may hold anything (see attn_paged_kernel):
            // their values are zeroed, each warp's 16 rows by itself. (S(i), which
            // reads them too, is done.)
            if (seen_rows != 0xffffu) {
                // (16-byte chunks in an order that spreads the rows over the banks)
                const uint32_t row = ring(st) + (my_row / 8) * 2048 + (my_row % 8) * 128;
                for (int blk = grp; okw && blk < C::BLOCKS; blk += C::GROUPS) {
                    okw = __all_sync(0xffffffffu, wt.wait(full(st, blk), (i / NST) & 1u));
                    if (okw && !seen) {
                        const uint32_t box = row + blk * C::PART_BYTES + (lane / 16) * 1024;
#pragma unroll
                        for (int e = 0; e < 8; ++e) st_shared_v4(box + ((e ^ (lane & 7)) * 16), 0u, 0u, 0u, 0u);
                    }
                    __syncwarp();
                }
            }
            if (okw) {
                // P^T, rounded to bf16 for the product: row = column of S^T, 64
                // positions of 2 bytes; the warp's 16 are chunks 2 sw and 2 sw + 1
                // of its 16-byte chunks
                const uint32_t j = lane % 8, chunk = 2 * sw + ((lane / 8) & 1);
                const uint32_t dst = sP + (g0 + 8 * (lane / 16) + j) * 128 + ((chunk ^ j) * 16);
#pragma unroll
                for (int k = 0; k < NK; k += 2) {
                    uint32_t h[4];
#pragma unroll
                    for (int v = 0; v < 4; ++v) {
                        const __nv_bfloat162 x = __floats2bfloat162_rn(s[4 * k + 2 * v], s[4 * k + 2 * v + 1]);
                        h[v] = *reinterpret_cast<const uint32_t *>(&x);
                    }
                    stmatrix_x4_trans(dst + k * 8 * 128, h[0], h[1], h[2], h[3]);
                }
                fence_proxy_async_smem();
                tc_fence_before();
                mbar_arrive(p_full);
            }
            ok = okw;
            if (ends) {
                // ---------------------------------------------------- the segment's results
                // (the sums go where the maxima of tile i - 1 were)
                float *const sums = red + (sb ^ 1) * 4 * CG;
#pragma unroll
                for (int k = 0; k < NK; ++k) {
                    float a = l_part[2 * k], b = l_part[2 * k + 1];
#pragma unroll
                    for (int o = 4; o <= 16; o *= 2) {
                        a += __shfl_xor_sync(0xffffffffu, a, o);
                        b += __shfl_xor_sync(0xffffffffu, b, o);
                    }
                    l_part[2 * k] = a;
                    l_part[2 * k + 1] = b;
                }
                if (lane < 4) {
#pragma unroll
                    for (int c = 0; c < CG / 4; ++c) {
                        sums[sw * CG + 8 * (c / 2) + cc + c % 2] = l_part[c];
                        if (sw == 0) col_s[8 * (c / 2) + cc + c % 2].y = m_run[c];
                    }
                }
                __syncwarp();
                if (ok) ok = __all_sync(0xffffffffu, wt.wait(pv_done, i & 1u));
                ok = __all_sync(0xffffffffu, named_bar_and(1 + grp, 4 * 32, ok));
                if (!ok) break;
                tc_fence_after();
                const int ncol = min(p.GT - c0 - g0, CG);  // the group's columns in use
                const bool whole = __any_sync(0xffffffffu, seg_j == 0 && cur.last());
                const int64_t row = static_cast<int64_t>(cur.b) * p.GT + c0 + g0;
                const int64_t slot = paged_slot(blockIdx.x, blockIdx.y, p.split.ranges, cur.b == run.b) * NC + g0;
                auto sum_of = [&](int c) {
                    return (sums[c] + sums[CG + c]) + (sums[2 * CG + c] + sums[3 * CG + c]);
                };
                if (rank_lane < CG) {
                    const int c = rank_lane;
                    const float l = sum_of(c), m = col_s[c].y;
                    if (whole) {
                        col_s[c].x = l == 0.f ? 0.f : 1.f / l;
                        if (c < ncol) p.lse[row + c] = l == 0.f ? -CUDART_INF_F : (m + __log2f(l)) * 0.69314718055994531f;
                    } else if (c < ncol) {
                        p.part_ml[slot + c] = make_float2(m, l);
                    }
                }
                __syncwarp();
                named_bar_sync(1 + grp, 4 * 32);
                // Short loops on purpose: this runs once a segment, and what it
                // costs is above all fetching its instructions (unrolled over the
                // columns it took 6.8 us' worth of cycles at 64 columns).
#pragma unroll 1
                for (int j = 0; j < C::BLOCKS * CG / 8; ++j) {
                    const int blk = j / (CG / 8), c8 = j % (CG / 8) * 8, at = blk * 128 + rank_lane;
                    uint32_t o[8];
                    tmem_ld8(lane_base + C::O_COL + blk * NC + g0 + c8, o);
                    __nv_bfloat16 *const out = p.o + (row + c8) * R + at;
                    float *const part = p.part_o + (slot + c8) * R + at;
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        const float v = __uint_as_float(o[c]);
                        if (whole) {
                            const float x = v * col_s[c8 + c].x;
                            if (c8 + c < ncol) out[c * R] = __float2bfloat16_rn(x);
                        } else {
                            part[c * R] = v;  // (the slot has room for columns not in use)
                        }
                    }
                }
                tc_fence_before();
                // the sums and maxima have been read before the next tile's
                // maxima, or the next rescaling, overwrite them
                ok = __all_sync(0xffffffffu, named_bar_and(1 + grp, 4 * 32, ok));
                if (!ok) break;
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
