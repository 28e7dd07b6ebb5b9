// Decode attention of one new token per sequence over a paged cache: the schedule shared by
// the bf16 and fp32 kernels (decode_paged_bf16.cu, decode_paged_f32.cu).
//
// For sequence b, kv head j and its g query heads, over the sequence's n_b tokens, token t in
// row t % page of page table[b][t / page] (or over the blocks listed for (b, j)):
//   s_t = scale q . K~_t,  out = sum_t 2^(s_t - M) V~_t / sum_t 2^(s_t - M)   (s in log2 units)
// with K~, V~ one source's rows or the convex mix of two. Bound by HBM: 2 * sources * n_b * d
// elements per (b, j) read once, a few operations per byte.
//
// Split. The units (b, j) laid end to end are sum_b Hkv * tiles_b tiles of TT tokens; the grid's
// warps get equal shares of that line, computed on the device from the lengths, so a batch of
// ragged sequences, one long sequence and many short ones all load every SM alike, whatever
// the host knows of the lengths. A warp streams its share through a private ring of NSW
// shared-memory stages filled by TMA (one box per page piece, the page found in the block
// table 32 entries at a time), keeping the online softmax of the unit it is in. A unit that
// lies inside one warp's share is written out from registers. Otherwise the warps' states meet
// in shared memory, and a unit that spans CTAs is joined by the last of them to arrive, from
// one partial per CTA in L2 (two slots a CTA: the unit it ends and the unit it begins). Short
// shares are rounded to whole CTAs per unit, and where every unit is short and has a CTA of its
// own, it is not split across CTAs at all (launch_paged).
// A call reads K and V once, and its copies are marked evict-first in L2. That gains where the
// next call reads another cache, and costs where calls read one cache again and again (layers
// that share a slot) and it fits L2 (bf16; evict-first against the normal policy):
//   32 requests of up to 2K, 24 caches of 28 MB in turn:      13.2 against 13.9 us
//   7 of up to 8K, 4 caches of 82 MB in turn:                 22.2 against 23.2 us
//   the same, each cache read twice in a row:                 20.8 against 21.6 us
//   one cache of 82 MB again and again:                       22.1 against 19.8 us
//   32 of 2K, one cache of 67 MB again and again:             15.3 against 13.0 us
//   4 of up to 64K, 746 MB:                                   116 to 118 us either way
//
// Measured (one layer; graphs that go through several caches, 400 MB and more together):
//   4 requests of up to 64K tokens, 8 kv heads x 128, bf16:  119 to 122 us, 6.3 to 6.5 TB/s (96 to
//                                                             99 % of the measured copy rate)
//   16 requests of up to 8K, two sources, 4 x 128, bf16:      55 us, 5.6 TB/s
//   32 requests of up to 2K, 4 x 64, bf16:                    13.6 us, 2.6 TB/s (12.3 out of L2)
//   one request of 320 tokens, 4 x 128, bf16:                 6.4 us
// Short calls are bound by the chain launch (2 us) -> lengths -> block table -> first tile (3 us
// together) -> last tile -> joins (3 to 4 us), not by bytes.
//
// A page index outside the pool reads as zeros (a copy that starts outside its tensor) and is
// reported; tokens past a sequence's end are masked and their V rows cleared, so that stale
// pages (NaN included) reach no output.
#pragma once

#include <algorithm>

#include "kvs_device.cuh"
#include "kvs_paged.h"

namespace kvs {

constexpr int PAGED_SMEM_MAX = 224 * 1024;   // dynamic share of an SM's 227 KB (static beside it)

// 4-D tiled bulk tensor load global -> shared with an L2 policy, completion counted on `bar`.
__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, int c0, int c1, int c2, int c3,
                                            uint64_t* bar, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%2, %3, %4, %5}], [%6], %7;" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(smem_u32(bar)), "l"(policy)
        : "memory");
}

__device__ __forceinline__ uint64_t policy_evict_first() {
    uint64_t p;
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
    return p;
}

// Zero rows [r0, r1) of a staged tile: `subs` blocks of `sub_stride` bytes, 128 bytes a row.
__device__ __forceinline__ void zero_rows(uint8_t* base, int subs, int sub_stride, int r0, int r1, int lane) {
    const int per = (r1 - r0) * 8;
    for (int i = lane; i < per * subs; i += 32)
        *reinterpret_cast<uint4*>(base + (i / per) * sub_stride + (r0 + (i % per) / 8) * 128 + (i % 8) * 16) =
            make_uint4(0u, 0u, 0u, 0u);
}

// 1 / l; 0 where no token was attended to
__device__ __forceinline__ float inverse_of(float l) { return l > 0.f ? 1.f / l : 0.f; }

// Add a state's values v (x, z of one head with statistics mx, y, w of another with my) against
// the joint maxima M.
__device__ __forceinline__ void add_state(float4& acc, float2& l, const float4& v, float2 mx, float2 my, float2 M) {
    const float fx = merge_factor(mx.x, M.x), fy = merge_factor(my.x, M.y);
    l.x = fmaf(fx, mx.y, l.x);
    l.y = fmaf(fy, my.y, l.y);
    acc.x = fmaf(fx, v.x, acc.x);
    acc.y = fmaf(fy, v.y, acc.y);
    acc.z = fmaf(fx, v.z, acc.z);
    acc.w = fmaf(fy, v.w, acc.w);
}

// P: the arithmetic of one storage type (see PagedBf16, PagedF32). It fixes D, NSRC, TT, NH
// (padded heads), NW (warps), NSW (stages), SUBW (elements of a 128-byte row), STAGE (bytes)
// and WARP_FLOATS (private scratch), and keeps one unit's state in registers.
template <class P>
struct PagedLayout {
    static constexpr int RING = P::NW * P::NSW * P::STAGE;
    static constexpr int SAVE = P::NW * P::NH * P::D * 4;              // states of units begun by an earlier warp
    static constexpr int SCRATCH = P::NW * P::WARP_FLOATS * 4;
    static constexpr int BYTES = RING + SAVE + SCRATCH + 1024;         // + slack to align the ring
    static_assert(P::NSW * P::STAGE >= P::NH * P::D * 4, "a warp's ring holds its last state");
    static_assert(P::STAGE % 1024 == 0, "swizzled stages stay 1024-byte aligned");
    static_assert(BYTES <= PAGED_SMEM_MAX, "shared memory");
    // the (m, l) of every CTA's partial of a unit lie over the ring in the last join
    static_assert(RING >= 65536, "statistics of up to 512 partials");
};

struct PagedState {
    int head0;      // the unit's first query head, b * Hq + j * g, or -1: no state
    int begin;      // the unit's first tile on the line
    int tiles;      // its tiles
    int started;    // the unit's first tile is in this state
    int ended;      // and its last
};

template <class P>
__global__ void __launch_bounds__(P::NW * 32, 1)
decode_paged_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                    const PagedDecodeArgs a) {
    using L = PagedLayout<P>;
    constexpr int D = P::D, TT = P::TT, NW = P::NW, NSW = P::NSW, NH = P::NH;
    constexpr int BLK = TT / 16;                 // 16-token blocks of a tile, each with its own limit
    constexpr int SUBS = D / P::SUBW;            // 128-byte wide sub-tiles of a tile
    constexpr int TILE_BYTES = SUBS * TT * 128;
    extern __shared__ uint8_t smem_dyn[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_dyn) + 1023) & ~uintptr_t(1023));
    __shared__ __align__(8) uint64_t bars[NW * NSW + 1];
    __shared__ int s_lim[NW * NSW * BLK];
    __shared__ PagedState s_state[NW * 2];
    __shared__ float2 s_ml[NW * 2][NH];          // max and sum of every head of a state
    __shared__ int s_part[2][3];                 // units that continue elsewhere: first head, first CTA, CTAs
    __shared__ unsigned s_last[2];

    const int cta = blockIdx.x;
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int g = a.g;
    const int ps = 1 << a.page_shift;

    if (threadIdx.x == 0) {
        prefetch_tmap(&tmK);
        prefetch_tmap(&tmV);
        for (int i = 0; i < NW * NSW + 1; ++i) mbar_init(&bars[i], 1);
        mbar_init_fence();
    }
    if (threadIdx.x < NW * 2) s_state[threadIdx.x].head0 = -1;
    if (threadIdx.x < 2) s_part[threadIdx.x][0] = -1;
    __syncthreads();
    grid_dep_wait();
    if (threadIdx.x == 0) grid_dep_launch();

    // ---- the line of tiles and this warp's share of it
    auto row_len = [&](int b) {
        const int n = a.lens[b];
        const int cap = a.max_blocks << a.page_shift;
        if (n < 0 || n > cap) {
            atomicOr(a.err, ERR_RANGE);
            return n < 0 ? 0 : cap;
        }
        return n;
    };
    auto row_blocks = [&](int n) {               // blocks of a sequence that are read
        const int p = (n + ps - 1) >> a.page_shift;
        return a.sel != nullptr ? min(p, a.top) : p;
    };
    auto row_tiles = [&](int n) {
        return ((a.sel != nullptr ? row_blocks(n) << a.page_shift : n) + TT - 1) / TT;
    };
    struct Cursor {
        int b, j, t, n, tiles;
    };
    Cursor at = {0, 0, 0, 0, 0};
    // entry i of a unit's block list and its page, unchecked (i within the list)
    auto look_up = [&](int b, int j, int i, int& lg, int& ph) {
        lg = i;
        if (a.sel != nullptr) lg = a.sel[(static_cast<size_t>(b) * a.Hkv + j) * a.top + i];
        ph = lg >= 0 && lg < a.max_blocks ? a.table[static_cast<size_t>(b) * a.max_blocks + lg] : -1;
    };
    const int list = a.sel != nullptr ? min(a.top, a.max_blocks) : a.max_blocks;   // longest block list
    int early_lg = -1, early_ph = -1;
    const bool early = a.aligned != 0 && list <= 32;         // the whole list, fetched beside the length
    unsigned share, more, t0;
    int my_n;
    int unit_c0 = -1, unit_ctas = 0;             // whole CTAs per unit: this unit's first and how many
    if (a.aligned) {
        // one CTA per unit, its tiles dealt to the warps
        at.b = cta / a.Hkv;
        at.j = cta - at.b * a.Hkv;
        if (early && lane < list) look_up(at.b, at.j, lane, early_lg, early_ph);
        at.n = row_len(at.b);
        at.tiles = row_tiles(at.n);
        share = at.tiles / NW;
        more = at.tiles - share * NW;
        t0 = share * warp + min(static_cast<unsigned>(warp), more);
        my_n = share + (warp < more ? 1 : 0);
        at.t = t0;
    } else {
        // 32-bit arithmetic: the caller keeps the line below 2^31 tiles
        const int n_lane = lane < a.B ? row_len(lane) : 0;   // the first 32 sequences, one per lane
        const int tiles_lane = row_tiles(n_lane);
        unsigned total = tiles_lane;
        for (int b = lane + 32; b < a.B; b += 32) total += row_tiles(row_len(b));
        const unsigned W = __reduce_add_sync(0xffffffffu, total) * a.Hkv;
        const unsigned most = static_cast<unsigned>(a.ctas) * NW;
        // Whole CTAs per unit where the shares are short and that costs a warp at most a tile more
        // than an even share, or where few units make long joins: a CTA then joins one unit instead
        // of up to two, one after the other. (5 requests of up to 8K, 4 heads: 19.8 -> 17.7 us; one
        // of 64K, 4 heads: 34.9 -> 32.1; 2 of 5K, 8 heads: 17.0 -> 14.6. With longer shares and more
        // units the uneven ends cost more: 30 of 3K, 4 heads: 26.4 -> 27.2.)
        auto pieces_of = [&](unsigned tiles, unsigned s) {   // CTAs of NW * s tiles; division by a constant at s = 1
            return s == 1 ? (tiles + NW - 1) / NW : (tiles + NW * s - 1) / (NW * s);
        };
        unsigned per_warp = 0;
        const unsigned s0 = W <= most ? 1u : (W + most - 1) / most;
        if (a.B * a.Hkv <= (s0 <= 6 ? a.ctas : a.ctas / 8)) {
            for (unsigned s = s0; s <= (s0 <= 6 ? s0 + 1 : s0) && per_warp == 0; ++s) {
                unsigned n = 0;
                for (int b = lane; b < a.B; b += 32)
                    n += pieces_of(b == lane ? tiles_lane : row_tiles(row_len(b)), s);
                if (__reduce_add_sync(0xffffffffu, n) * a.Hkv <= static_cast<unsigned>(a.ctas)) per_warp = s;
            }
        }
        share = more = t0 = 0;
        my_n = 0;
        if (per_warp == 0) {
            // no more CTAs than tiles: every CTA between a unit's first and last holds a part of it
            const unsigned nc = max(1u, min(static_cast<unsigned>(a.ctas), (W + NW - 1) / NW));
            const unsigned workers = nc * NW;
            share = W / workers;
            more = W - share * workers;          // the first `more` warps take one tile more
            const unsigned id = cta * NW + warp;
            t0 = share * id + min(id, more);
            my_n = id < workers ? share + (id < more ? 1 : 0) : 0;
        }
        // where this CTA or this warp's first tile lies on the line of the rows
        const unsigned target = per_warp > 0 ? cta : t0;
        unsigned base = 0;
        bool found = false;
        for (int r0 = 0; !found && r0 < a.B && (per_warp > 0 || my_n > 0); r0 += 32) {
            const int n = r0 == 0 ? n_lane : r0 + lane < a.B ? row_len(r0 + lane) : 0;
            const int own = r0 == 0 ? tiles_lane : row_tiles(n);
            const unsigned pieces = per_warp > 0 ? pieces_of(own, per_warp) : own;
            unsigned incl = pieces * a.Hkv;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const unsigned x = __shfl_up_sync(0xffffffffu, incl, off);
                if (lane >= off) incl += x;
            }
            const unsigned ahead = __ballot_sync(0xffffffffu, base + incl > target);
            if (ahead != 0u) {
                const int who = __ffs(ahead) - 1;
                at.b = r0 + who;
                at.n = __shfl_sync(0xffffffffu, n, who);
                at.tiles = __shfl_sync(0xffffffffu, own, who);
                const unsigned m = __shfl_sync(0xffffffffu, pieces, who);
                const unsigned in_row = target - (base + __shfl_sync(0xffffffffu, incl, who) - m * a.Hkv);
                at.j = in_row / m;
                at.t = in_row - at.j * m;
                if (per_warp > 0) {              // CTA at.t of the unit's m: its warps' part of the unit
                    unit_c0 = cta - at.t;
                    unit_ctas = m;
                    const unsigned all = m * NW, me = at.t * NW + warp;
                    share = at.tiles / all;
                    more = at.tiles - share * all;
                    t0 = share * me + min(me, more);
                    my_n = share + (me < more ? 1 : 0);
                    at.t = t0;
                }
                found = true;
            }
            base += __shfl_sync(0xffffffffu, incl, 31);
        }
        if (!found) my_n = 0;
    }
    // to the next unit that has tiles (only called while the share holds more)
    auto next_unit = [&](Cursor& c) {
        c.t = 0;
        if (++c.j < a.Hkv) return;
        c.j = 0;
        do {
            ++c.b;
            c.n = row_len(c.b);
            c.tiles = row_tiles(c.n);
        } while (c.tiles == 0 && c.b + 1 < a.B);
    };

    // ---- copies: pages of the unit being requested are looked up 32 at a time
    uint8_t* ring = smem + warp * NSW * P::STAGE;
    uint64_t* wb = &bars[warp * NSW];
    int* lims = &s_lim[warp * NSW * BLK];
    const int rows = min(ps, TT);                // tokens of one copy
    // a copy lands as [sub-tile][rows][128 bytes]: strides of 16-token blocks and of sub-tiles
    const int blk_stride = BLK == 1 || rows == TT ? 16 * 128 : SUBS * 16 * 128;
    const int sub_stride = BLK == 1 ? TT * 128 : rows * 128;
    Cursor ic = at;
    int wbase = 0;                               // window: lane i holds the unit's (wbase + i)-th block
    int wphys = -1, wlog = -1;
    bool wvalid = false;
    auto load_window = [&](int first) {
        wbase = early ? 0 : first;
        wphys = wlog = -1;
        const int held = (ic.n + ps - 1) >> a.page_shift, i = wbase + lane;
        if (i < row_blocks(ic.n)) {
            int lg = early_lg, ph = early_ph;
            if (!early) look_up(ic.b, ic.j, i, lg, ph);
            if (lg >= 0 && lg < held) wlog = lg;
            if (wlog >= 0 && ph >= 0 && ph < a.num_pages) wphys = ph;
            if (wphys < 0) atomicOr(a.err, ERR_RANGE);       // a block or a page that does not exist
        }
        wvalid = true;
    };
    const uint64_t policy = policy_evict_first();
    auto issue = [&](int k) {
        if (ic.t == ic.tiles) {
            next_unit(ic);
            wvalid = false;
        }
        const int tok = ic.t * TT;
        const int blk = tok >> a.page_shift;
        if (!wvalid || blk >= wbase + 32) load_window(blk);
        const int s = k % NSW;
        // lane i looks up 16-token block i of the tile: its page, row and limit
        const int my_tok = tok + (lane % BLK) * 16;
        const int from = (my_tok >> a.page_shift) - wbase;
        const int lg = __shfl_sync(0xffffffffu, wlog, from);
        const int phys = __shfl_sync(0xffffffffu, wphys, from);
        const int in_page = my_tok & (ps - 1);
        if (lane < BLK) lims[s * BLK + lane] = lg < 0 ? 0 : ic.n - (lg << a.page_shift) - in_page;
        if (lane == 0) mbar_arrive_expect_tx(&wb[s], P::STAGE);
        // the first lane of a page piece copies it
        if (lane < BLK && (lane * 16) % rows == 0) {
            uint8_t* dst = ring + s * P::STAGE + lane * blk_stride;
            const int c0 = phys < 0 ? -1 : (a.src0 * a.num_pages + phys) * a.Hkv + ic.j;
            tma_load_4d(dst, &tmK, 0, in_page, 0, c0, &wb[s], policy);
            tma_load_4d(dst + TILE_BYTES, &tmV, 0, in_page, 0, c0, &wb[s], policy);
            if (P::NSRC == 2) {
                const int c1 = phys < 0 ? -1 : (a.src1 * a.num_pages + phys) * a.Hkv + ic.j;
                tma_load_4d(dst + 2 * TILE_BYTES, &tmK, 0, in_page, 0, c1, &wb[s], policy);
                tma_load_4d(dst + 3 * TILE_BYTES, &tmV, 0, in_page, 0, c1, &wb[s], policy);
            }
        }
        ++ic.t;
        __syncwarp();
    };
    for (int k = 0; k < min(NSW, my_n); ++k) issue(k);

    if (a.stall_limit > 0 && threadIdx.x == 0) mbar_wait_bounded(&bars[NW * NSW], 0, a.stall_limit, a.err);
    // ---- sequences without tokens: zero output, lse -inf
    for (int b = cta; b < a.B; b += gridDim.x) {
        if (a.lens[b] > 0) continue;
        for (int i = threadIdx.x; i < a.Hq * D; i += NW * 32) a.out[static_cast<size_t>(b) * a.Hq * D + i] = 0.f;
        if (a.lse != nullptr)
            for (int i = threadIdx.x; i < a.Hq; i += NW * 32) a.lse[static_cast<size_t>(b) * a.Hq + i] = NEG_INF;
    }

    // ---- stream the share
    P p;
    float4* save = reinterpret_cast<float4*>(smem + L::RING) + warp * P::VALS;
    p.setup(reinterpret_cast<float*>(smem + L::RING + L::SAVE) + warp * P::WARP_FLOATS, lane);
    Cursor cc = at;
    int first_tile = at.t;                       // first tile of the current unit in this share
    bool alive = true;
    auto end_unit = [&](int k) {
        p.finish();
        const bool started = first_tile == 0, ended = cc.t == cc.tiles;
        const int head0 = cc.b * a.Hq + cc.j * g;
        if (started && ended) {
            p.values([&](int i, const float4& v) {
                const float2 l = p.sums(i);
                P::emit(a.out + static_cast<size_t>(head0) * D, g, i, v, make_float2(inverse_of(l.x), inverse_of(l.y)));
            });
            if (a.lse != nullptr) p.stats(g, [&](int h, float m, float l) { a.lse[head0 + h] = lse_of(m, l); });
            return;
        }
        const int which = 2 * warp + (started ? 1 : 0);
        float4* dst = started ? reinterpret_cast<float4*>(ring) : save;
        p.values([&](int i, const float4& v) { dst[i] = v; });
        p.stats(g, [&](int h, float m, float l) { s_ml[which][h] = make_float2(m, l); });
        if (lane == 0)
            s_state[which] = {head0, static_cast<int>(t0) + k - cc.t, cc.tiles, started ? 1 : 0, ended ? 1 : 0};
    };
    if (my_n > 0) p.begin(a, cc.b, cc.j);
    for (int k = 0; my_n > 0; ++k) {
        if (k == my_n || cc.t == cc.tiles) {
            end_unit(k);
            if (k == my_n) break;
            next_unit(cc);
            first_tile = 0;
            p.begin(a, cc.b, cc.j);
        }
        const int s = k % NSW;
        if (alive) {
            alive = __all_sync(0xffffffffu, mbar_wait_bounded(&wb[s], (k / NSW) & 1, a.wait_limit, a.err));
            if (!alive)   // give the copies still in flight a bounded chance to land; the units are walked without data
                for (int kk = k + 1; kk < min(my_n, k + NSW); ++kk)
                    mbar_wait_bounded(&wb[kk % NSW], (kk / NSW) & 1, a.wait_limit, a.err);
        }
        if (alive) {
            uint8_t* st = ring + s * P::STAGE;
            bool cut = false;
#pragma unroll
            for (int i = 0; i < BLK; ++i) {
                const int lim = lims[s * BLK + i];
                if (lim >= 16) continue;
                cut = true;
                zero_rows(st + TILE_BYTES + i * blk_stride, SUBS, sub_stride, max(lim, 0), 16, lane);
                if (P::NSRC == 2) zero_rows(st + 3 * TILE_BYTES + i * blk_stride, SUBS, sub_stride, max(lim, 0), 16, lane);
            }
            if (cut) __syncwarp();
            p.tile(a, st, blk_stride, sub_stride, lims + s * BLK, cut);
            if (cut) fence_proxy_async();        // the cleared rows before the next copy into the stage
            __syncwarp();
            if (k + NSW < my_n) issue(k + NSW);
        }
        ++cc.t;
    }
    __syncthreads();

    // ---- join the warps' states, unit by unit. States are in the line's order; every warp
    // finds the units' first states by votes (lane i: state i)
    PagedState mine = {-1, 0, 0, 0, 0};
    if (lane < 2 * NW) mine = s_state[lane];
    const int unit_l = mine.head0, flags_l = mine.started | mine.ended << 1;
    const unsigned valid = __ballot_sync(0xffffffffu, unit_l >= 0);
    const unsigned below = valid & ((1u << lane) - 1u);
    const int prev = __shfl_sync(0xffffffffu, unit_l, below ? 31 - __clz(below) : lane);
    const unsigned firsts = __ballot_sync(0xffffffffu, unit_l >= 0 && (below == 0u || prev != unit_l));
    // states of the unit that begins at state i: those up to the next unit's first
    auto states_from = [&](int i) {
        const unsigned later = firsts & ~((2u << i) - 1u);
        return valid & ~((1u << i) - 1u) & (later ? (later & (0u - later)) - 1u : 0xffffffffu);
    };
    // the last state of this lane's unit says whether the unit ends here
    const unsigned own_states = (firsts >> lane) & 1u ? states_from(lane) : 0u;
    const int last_flags = __shfl_sync(0xffffffffu, flags_l, own_states ? 31 - __clz(own_states) : lane);
    const bool split = own_states != 0u && !((flags_l & 1) && (last_flags & 2));
    const unsigned splits = __ballot_sync(0xffffffffu, split);
    if (split && warp == 0) {
        // the CTA whose share holds a tile
        auto owner = [&](unsigned x) {
            const unsigned big = more * (share + 1);
            return static_cast<int>((x < big ? x / (share + 1) : more + (x - big) / share) / NW);
        };
        int* part = s_part[flags_l & 1];
        part[0] = unit_l;
        part[1] = unit_c0 >= 0 ? unit_c0 : owner(mine.begin);
        part[2] = unit_c0 >= 0 ? unit_ctas : owner(mine.begin + mine.tiles - 1) - part[1] + 1;
    }
    constexpr int per = paged_partial(NH, D), VALS = P::VALS;
    static_assert(VALS * 4 == NH * D, "a state's values");
    const int groups = __popc(firsts);
    for (int k = threadIdx.x; k < groups * VALS; k += NW * 32) {
        const int idx = k % VALS;
        const int2 hd = P::heads(idx);
        if (hd.x >= g) continue;
        unsigned rest = firsts;
        for (int c = k / VALS; c > 0; --c) rest &= rest - 1u;
        const int i = __ffs(rest) - 1;
        const unsigned states = states_from(i);
        // a warp has at most one state of a unit (even: begun by an earlier warp, in the save area;
        // odd: over its ring), so the loop over the warps is static and its loads independent
        float2 M = make_float2(NEG_INF, NEG_INF), mx[NW], my[NW];
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            const unsigned own = (states >> (2 * w)) & 3u;
            mx[w] = s_ml[2 * w + (own >> 1)][hd.x];
            my[w] = s_ml[2 * w + (own >> 1)][hd.y];
            if (own == 0u) mx[w] = my[w] = make_float2(NEG_INF, 0.f);     // whatever was there: no state
            M.x = fmaxf(M.x, mx[w].x);
            M.y = fmaxf(M.y, my[w].x);
        }
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        float2 l = make_float2(0.f, 0.f);
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            const unsigned own = (states >> (2 * w)) & 3u;
            float4 v = reinterpret_cast<const float4*>(smem + (own >= 2u ? w * NSW * P::STAGE : L::RING + w * VALS * 16))[idx];
            if (own == 0u) v = make_float4(0.f, 0.f, 0.f, 0.f);
            add_state(acc, l, v, mx[w], my[w], M);
        }
        if ((splits >> i) & 1u) {
            float* part = a.ws + static_cast<size_t>(2 * cta + s_state[i].started) * per;
            reinterpret_cast<float4*>(part)[idx] = acc;
            // the lanes that hold a head's first channels write its statistics
            if (P::first_of(idx)) {
                float2* ml = reinterpret_cast<float2*>(part + NH * D);
                ml[hd.x] = make_float2(M.x, l.x);
                ml[hd.y] = make_float2(M.y, l.y);
            }
        } else {
            const int head0 = s_state[i].head0;
            P::emit(a.out + static_cast<size_t>(head0) * D, g, idx, acc, make_float2(inverse_of(l.x), inverse_of(l.y)));
            if (a.lse != nullptr && P::first_of(idx)) {
                a.lse[head0 + hd.x] = lse_of(M.x, l.x);
                if (hd.y < g) a.lse[head0 + hd.y] = lse_of(M.y, l.y);
            }
        }
    }
    if (splits == 0u) return;

    // ---- the last CTA of a unit to arrive joins its partials. Its thread's acq_rel atomic,
    // between two block barriers, orders every thread's partial before it and every read after it
    __syncthreads();
    if (threadIdx.x < 2 && s_part[threadIdx.x][0] >= 0) {
        unsigned prev_n;
        asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;"
                     : "=r"(prev_n)
                     : "l"(a.counters + s_part[threadIdx.x][1])
                     : "memory");
        s_last[threadIdx.x] = prev_n == static_cast<unsigned>(s_part[threadIdx.x][2] - 1) ? 1u : 0u;
    }
    __syncthreads();
    float2* stat = reinterpret_cast<float2*>(smem);      // [n][NH] (m, l), over the ring
    for (int which = 0; which < 2; ++which) {
        const int head0 = s_part[which][0];
        if (head0 < 0 || s_last[which] == 0u) continue;  // the same for every thread
        const int c0 = s_part[which][1], n = s_part[which][2];
        // partial i: CTA c0 + i, which began the unit (slot 1) or continued it (slot 0)
        const float* base = a.ws + static_cast<size_t>(2 * c0) * per;
        auto slot = [&](int i) { return base + (2 * i + (i == 0 ? 1 : 0)) * per; };
        // a thread's first values are on their way while the statistics are shared
        constexpr int AHEAD = 8;
        float4 early[AHEAD];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i)
            if (i < n && threadIdx.x < VALS) early[i] = __ldcg(reinterpret_cast<const float4*>(slot(i)) + threadIdx.x);
        for (int i = threadIdx.x; i < n * NH; i += NW * 32)
            stat[i] = __ldcg(reinterpret_cast<const float2*>(slot(i / NH) + NH * D) + i % NH);
        __syncthreads();
        for (int idx = threadIdx.x; idx < VALS; idx += NW * 32) {
            const int2 hd = P::heads(idx);
            if (hd.x >= g) continue;
            float2 M = make_float2(NEG_INF, NEG_INF);
#pragma unroll 4
            for (int i = 0; i < n; ++i) {
                M.x = fmaxf(M.x, stat[i * NH + hd.x].x);
                M.y = fmaxf(M.y, stat[i * NH + hd.y].x);
            }
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            float2 l = make_float2(0.f, 0.f);
            int i = 0;
            if (idx == threadIdx.x) {
#pragma unroll
                for (; i < AHEAD; ++i)
                    if (i < n) add_state(acc, l, early[i], stat[i * NH + hd.x], stat[i * NH + hd.y], M);
            }
#pragma unroll 8
            for (; i < n; ++i)
                add_state(acc, l, __ldcg(reinterpret_cast<const float4*>(slot(i)) + idx), stat[i * NH + hd.x], stat[i * NH + hd.y], M);
            P::emit(a.out + static_cast<size_t>(head0) * D, g, idx, acc, make_float2(inverse_of(l.x), inverse_of(l.y)));
            if (a.lse != nullptr && P::first_of(idx)) {
                a.lse[head0 + hd.x] = lse_of(M.x, l.x);
                if (hd.y < g) a.lse[head0 + hd.y] = lse_of(M.y, l.y);
            }
        }
        if (threadIdx.x == 0) a.counters[c0] = 0u;
        __syncthreads();
    }
}

template <class P>
cudaError_t launch_paged(const CUtensorMap& tmK, const CUtensorMap& tmV, const PagedDecodeArgs& a, cudaStream_t st) {
    auto kern = decode_paged_kernel<P>;
    constexpr int smem = PagedLayout<P>::BYTES;
    static std::atomic<unsigned long long> attr_done{0};
    cudaError_t e = once_per_device(attr_done, [&] {
        return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    });
    if (e != cudaSuccess) return e;
    // One CTA per unit where the units fit the grid and even the longest possible one is short:
    // joining a unit across CTAs costs about as much as 4 tiles of every warp. With most of the
    // multiprocessors busy anyway twice that is worth it. Against the splits of the line (the
    // caches together larger than L2): one 320-token request 7.7 -> 6.5 us; 16 requests of 500
    // tokens, 4 x 128: 11.3 -> 8.9; 32 ragged ones of up to 2K, 4 x 64: 15.8 -> 13.2; 32 of 2K:
    // 16.9 -> 15.3; 2 of 1K: 8.5 -> 7.7. Longer units on a CTA each lose (8 units of 1K tokens at
    // 8 tiles a warp: 19.2 -> 22.0, measured on an earlier build).
    PagedDecodeArgs args = a;
    const int units = a.B * a.Hkv;
    const long long cap = static_cast<long long>(a.sel != nullptr ? std::min(a.top, a.max_blocks) : a.max_blocks) << a.page_shift;
    args.aligned = units <= a.ctas && cap <= static_cast<long long>(P::NW) * P::TT * (2 * units >= a.ctas ? 8 : 4);
    return launch_kernel(kern, dim3(args.aligned ? units : a.ctas), dim3(P::NW * 32), smem, st, true, tmK, tmV, args);
}

// The deepest ring that fits beside the saved states and scratch, at most two stages.
constexpr int paged_stages(int nw, int stage, int nh, int d, int warp_floats) {
    for (int s = 2; s > 1; --s)
        if (nw * (s * stage + nh * d * 4 + warp_floats * 4) + 1024 <= PAGED_SMEM_MAX) return s;
    return 1;
}

}  // namespace kvs
