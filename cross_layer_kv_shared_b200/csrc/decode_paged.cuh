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
// one partial per CTA in L2 (two slots a CTA: the unit it ends and the unit it begins).
//
// A page index outside the pool reads as zeros (a copy that starts outside its tensor) and is
// reported; tokens past a sequence's end are masked and their V rows cleared, so that stale
// pages (NaN included) reach no output.
#pragma once

#include "kvs_device.cuh"
#include "kvs_paged.h"

namespace kvs {

constexpr int PAGED_SMEM_MAX = 232448 - 4096;   // dynamic share of an SM's 227 KB (static beside it)

// Zero rows [r0, r1) of a staged tile: `subs` blocks of `sub_stride` bytes, 128 bytes a row.
__device__ __forceinline__ void zero_rows(uint8_t* base, int subs, int sub_stride, int r0, int r1, int lane) {
    const int per = (r1 - r0) * 8;
    for (int i = lane; i < per * subs; i += 32)
        *reinterpret_cast<uint4*>(base + (i / per) * sub_stride + (r0 + (i % per) / 8) * 128 + (i % 8) * 16) =
            make_uint4(0u, 0u, 0u, 0u);
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
    // merge scratch (factors of up to 2^15 / NH partials) lies over the ring
    static_assert(RING >= 65536, "merge scratch");
};

struct PagedState {
    int unit;       // b * Hkv + j, or -1
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
    constexpr int SUB_BYTES = TT * 128;
    constexpr int TILE_BYTES = SUBS * SUB_BYTES;
    extern __shared__ uint8_t smem_dyn[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_dyn) + 1023) & ~uintptr_t(1023));
    __shared__ __align__(8) uint64_t bars[NW * NSW];
    __shared__ int s_lim[NW * NSW * BLK];
    __shared__ PagedState s_state[NW * 2];
    __shared__ float s_m[NW * 2][NH], s_l[NW * 2][NH];
    __shared__ unsigned s_last[2];

    const int cta = blockIdx.x;
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int g = a.g;
    const int ps = 1 << a.page_shift;

    if (threadIdx.x == 0) {
        prefetch_tmap(&tmK);
        prefetch_tmap(&tmV);
        for (int i = 0; i < NW * NSW; ++i) mbar_init(&bars[i], 1);
        mbar_init_fence();
    }
    if (threadIdx.x < NW * 2) s_state[threadIdx.x].unit = -1;
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
    int total = 0;
    for (int b = lane; b < a.B; b += 32) total += row_tiles(row_len(b));
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) total += __shfl_xor_sync(0xffffffffu, total, off);
    const long long W = static_cast<long long>(total) * a.Hkv;
    // no more CTAs than tiles: every CTA between a unit's first and last holds a part of it
    const int nc = static_cast<int>(min(static_cast<long long>(a.ctas), max(1LL, (W + NW - 1) / NW)));
    const int workers = nc * NW;
    long long t0 = 0, t1 = 0;
    if (cta < nc) {
        t0 = W * (cta * NW + warp) / workers;
        t1 = W * (cta * NW + warp + 1) / workers;
    }
    const int my_n = static_cast<int>(t1 - t0);

    struct Cursor {
        int b, j, t, n, tiles;
    };
    Cursor at = {0, 0, 0, 0, 0};
    if (my_n > 0) {
        long long base = 0;
        for (int r0 = 0; r0 < a.B; r0 += 32) {
            const int n = r0 + lane < a.B ? row_len(r0 + lane) : 0;
            const int own = row_tiles(n);
            long long incl = static_cast<long long>(own) * a.Hkv;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const long long x = __shfl_up_sync(0xffffffffu, incl, off);
                if (lane >= off) incl += x;
            }
            const long long all = __shfl_sync(0xffffffffu, incl, 31);
            if (t0 < base + all) {
                const int who = __ffs(__ballot_sync(0xffffffffu, base + incl > t0)) - 1;
                at.b = r0 + who;
                at.n = __shfl_sync(0xffffffffu, n, who);
                at.tiles = __shfl_sync(0xffffffffu, own, who);
                const long long row0 = base + __shfl_sync(0xffffffffu, incl, who) - static_cast<long long>(at.tiles) * a.Hkv;
                at.j = static_cast<int>((t0 - row0) / at.tiles);
                at.t = static_cast<int>((t0 - row0) % at.tiles);
                break;
            }
            base += all;
        }
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
    Cursor ic = at;
    int wbase = 0;                               // window: lane i holds the unit's (wbase + i)-th block
    int wphys = -1, wlog = -1;
    bool wvalid = false;
    auto load_window = [&](int first) {
        wbase = first;
        wphys = wlog = -1;
        const int held = (ic.n + ps - 1) >> a.page_shift;
        if (first + lane < row_blocks(ic.n)) {
            int lg = first + lane;
            if (a.sel != nullptr) lg = a.sel[(static_cast<size_t>(ic.b) * a.Hkv + ic.j) * a.top + lg];
            if (lg >= 0 && lg < held) {
                wlog = lg;
                const int ph = a.table[static_cast<size_t>(ic.b) * a.max_blocks + lg];
                if (ph >= 0 && ph < a.num_pages)
                    wphys = ph;
                else
                    atomicOr(a.err, ERR_RANGE);
            } else {
                atomicOr(a.err, ERR_RANGE);
            }
        }
        wvalid = true;
    };
    auto issue = [&](int k) {
        if (ic.t == ic.tiles) {
            next_unit(ic);
            wvalid = false;
        }
        const int tok = ic.t * TT;
        const int blk = tok >> a.page_shift;
        if (!wvalid || blk >= wbase + 32) load_window(blk);
        const int s = k % NSW;
        uint8_t* st = ring + s * P::STAGE;
        if (lane == 0) mbar_arrive_expect_tx(&wb[s], P::STAGE);
        for (int r = 0; r < TT; r += rows) {
            const int in_page = (tok + r) & (ps - 1);
            const int from = ((tok + r) >> a.page_shift) - wbase;
            const int phys = __shfl_sync(0xffffffffu, wphys, from);
            const int lg = __shfl_sync(0xffffffffu, wlog, from);
            if (lane == 0) {
                const int lim = lg < 0 ? 0 : ic.n - (lg << a.page_shift) - in_page;
                for (int i = 0; i < rows / 16; ++i) lims[s * BLK + r / 16 + i] = lim - 16 * i;
                const int c0 = phys < 0 ? -1 : (a.src0 * a.num_pages + phys) * a.Hkv + ic.j;
                const int c1 = phys < 0 ? -1 : (a.src1 * a.num_pages + phys) * a.Hkv + ic.j;
#pragma unroll
                for (int h = 0; h < SUBS; ++h) {
                    uint8_t* dst = st + h * SUB_BYTES + r * 128;
                    tma_load_3d(dst, &tmK, h * P::SUBW, in_page, c0, &wb[s]);
                    tma_load_3d(dst + TILE_BYTES, &tmV, h * P::SUBW, in_page, c0, &wb[s]);
                    if (P::NSRC == 2) {
                        tma_load_3d(dst + 2 * TILE_BYTES, &tmK, h * P::SUBW, in_page, c1, &wb[s]);
                        tma_load_3d(dst + 3 * TILE_BYTES, &tmV, h * P::SUBW, in_page, c1, &wb[s]);
                    }
                }
            }
        }
        ++ic.t;
        __syncwarp();
    };
    for (int k = 0; k < min(NSW, my_n); ++k) issue(k);

    // ---- sequences without tokens: zero output, lse -inf
    for (int b = cta; b < a.B; b += gridDim.x) {
        if (a.lens[b] > 0) continue;
        for (int i = threadIdx.x; i < a.Hq * D; i += NW * 32) a.out[static_cast<size_t>(b) * a.Hq * D + i] = 0.f;
        if (a.lse != nullptr)
            for (int i = threadIdx.x; i < a.Hq; i += NW * 32) a.lse[static_cast<size_t>(b) * a.Hq + i] = NEG_INF;
    }

    // ---- stream the share
    P p;
    float* save = reinterpret_cast<float*>(smem + L::RING) + warp * NH * D;
    p.setup(reinterpret_cast<float*>(smem + L::RING + L::SAVE) + warp * P::WARP_FLOATS, lane);
    Cursor cc = at;
    int first_tile = at.t;                       // first tile of the current unit in this share
    bool alive = true;
    auto end_unit = [&](int k) {
        p.finish();
        const bool started = first_tile == 0, ended = cc.t == cc.tiles;
        const size_t head0 = static_cast<size_t>(cc.b) * a.Hq + static_cast<size_t>(cc.j) * g;
        if (started && ended) {
            p.each(g, [&](int h, int e, float v, float l) { a.out[(head0 + h) * D + e] = l > 0.f ? v / l : 0.f; });
            if (a.lse != nullptr) p.stats(g, [&](int h, float m, float l) { a.lse[head0 + h] = lse_of(m, l); });
            return;
        }
        const int which = 2 * warp + (started ? 1 : 0);
        float* dst = started ? reinterpret_cast<float*>(ring) : save;
        p.each(g, [&](int h, int e, float v, float) { dst[h * D + e] = v; });
        p.stats(g, [&](int h, float m, float l) {
            s_m[which][h] = m;
            s_l[which][h] = l;
        });
        if (lane == 0)
            s_state[which] = {cc.b * a.Hkv + cc.j, static_cast<int>(t0 + k) - cc.t, cc.tiles, started ? 1 : 0, ended ? 1 : 0};
    };
    if (my_n > 0) p.begin(a, cc.b, cc.j);
    for (int k = 0; k < my_n; ++k) {
        if (cc.t == cc.tiles) {
            end_unit(k);
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
                zero_rows(st + TILE_BYTES, SUBS, SUB_BYTES, i * 16 + max(lim, 0), i * 16 + 16, lane);
                if (P::NSRC == 2) zero_rows(st + 3 * TILE_BYTES, SUBS, SUB_BYTES, i * 16 + max(lim, 0), i * 16 + 16, lane);
            }
            if (cut) __syncwarp();
            p.tile(a, st, lims + s * BLK, cut);
            if (cut) fence_proxy_async();        // the cleared rows before the next copy into the stage
            __syncwarp();
            if (k + NSW < my_n) issue(k + NSW);
        }
        ++cc.t;
    }
    if (my_n > 0) end_unit(my_n);
    __syncthreads();

    // ---- join the warps' states, unit by unit (states are in the line's order)
    const float* saved = reinterpret_cast<const float*>(smem + L::RING);
    auto state_o = [&](int i) {
        return (i & 1) ? reinterpret_cast<const float*>(smem + (i >> 1) * NSW * P::STAGE) : saved + (i >> 1) * NH * D;
    };
    // a unit that continues in other CTAs: [0] began earlier, [1] goes on later
    int part_unit[2] = {-1, -1}, part_c0[2] = {0, 0}, part_n[2] = {0, 0};
    const int per = paged_partial(g, D);
    for (int i = 0; i < 2 * NW;) {
        const int unit = s_state[i].unit;
        if (unit < 0) {
            ++i;
            continue;
        }
        int last = i, i1 = i + 1;
        for (; i1 < 2 * NW && (s_state[i1].unit < 0 || s_state[i1].unit == unit); ++i1)
            if (s_state[i1].unit == unit) last = i1;
        const bool started = s_state[i].started, ended = s_state[last].ended;
        const bool whole = started && ended;
        const int which = started ? 1 : 0;
        float* part = a.ws + static_cast<size_t>(2 * cta + which) * per;
        if (!whole) {
            // CTA of a tile: the worker with the largest index whose share begins at or before it
            const long long x0 = s_state[i].begin, x1 = x0 + s_state[i].tiles - 1;
            const int c0 = static_cast<int>(((x0 + 1) * workers - 1) / W) / NW;
            const int c1 = static_cast<int>(((x1 + 1) * workers - 1) / W) / NW;
            part_unit[which] = unit;
            part_c0[which] = c0;
            part_n[which] = c1 - c0 + 1;
        }
        const size_t head0 = static_cast<size_t>(unit / a.Hkv) * a.Hq + static_cast<size_t>(unit % a.Hkv) * g;
        for (int idx = threadIdx.x; idx < g * (D / 4); idx += NW * 32) {
            const int h = idx / (D / 4), e = (idx % (D / 4)) * 4;
            float M = NEG_INF;
            for (int s = i; s <= last; ++s)
                if (s_state[s].unit == unit) M = fmaxf(M, s_m[s][h]);
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            float l = 0.f;
            for (int s = i; s <= last; ++s) {
                if (s_state[s].unit != unit) continue;
                const float f = merge_factor(s_m[s][h], M);
                const float4 v = *reinterpret_cast<const float4*>(state_o(s) + h * D + e);
                l = fmaf(f, s_l[s][h], l);
                acc.x = fmaf(f, v.x, acc.x);
                acc.y = fmaf(f, v.y, acc.y);
                acc.z = fmaf(f, v.z, acc.z);
                acc.w = fmaf(f, v.w, acc.w);
            }
            if (whole) {
                float* o = a.out + (head0 + h) * D + e;
                *reinterpret_cast<float4*>(o) = l > 0.f ? make_float4(acc.x / l, acc.y / l, acc.z / l, acc.w / l)
                                                        : make_float4(0.f, 0.f, 0.f, 0.f);
                if (e == 0 && a.lse != nullptr) a.lse[head0 + h] = lse_of(M, l);
            } else {
                *reinterpret_cast<float4*>(part + h * D + e) = acc;
                if (e == 0) {
                    part[g * D + h] = M;
                    part[g * D + g + h] = l;
                }
            }
        }
        i = i1;
    }
    if (part_unit[0] < 0 && part_unit[1] < 0) return;

    // ---- the last CTA of a unit to arrive joins its partials
    __threadfence();
    __syncthreads();
    if (threadIdx.x < 2 && part_unit[threadIdx.x] >= 0) {
        const int c0 = threadIdx.x == 0 ? part_c0[0] : part_c0[1];
        const int n = threadIdx.x == 0 ? part_n[0] : part_n[1];
        unsigned prev;
        asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(prev) : "l"(a.counters + c0) : "memory");
        s_last[threadIdx.x] = prev == static_cast<unsigned>(n - 1) ? 1u : 0u;
    }
    __syncthreads();
    float* fac = reinterpret_cast<float*>(smem);         // [n][g] m, then the factors
    for (int which = 0; which < 2; ++which) {
        const int unit = which == 0 ? part_unit[0] : part_unit[1];
        if (unit < 0 || s_last[which] == 0u) continue;   // the same for every thread
        const int c0 = which == 0 ? part_c0[0] : part_c0[1];
        const int n = which == 0 ? part_n[0] : part_n[1];
        __threadfence();
        // partial i: CTA c0 + i, which began the unit (slot 1) or continued it (slot 0)
        auto slot = [&](int i) { return a.ws + static_cast<size_t>(2 * (c0 + i) + (i == 0 ? 1 : 0)) * per; };
        float* sum = fac + n * g;                        // [g] M, [g] l
        for (int idx = threadIdx.x; idx < n * g; idx += NW * 32) fac[idx] = __ldcg(slot(idx / g) + g * D + idx % g);
        __syncthreads();
        for (int h = warp; h < g; h += NW) {
            float M = NEG_INF;
            for (int i = lane; i < n; i += 32) M = fmaxf(M, fac[i * g + h]);
            M = warp_max(M);
            float l = 0.f;
            for (int i = lane; i < n; i += 32) {
                const float f = merge_factor(fac[i * g + h], M);
                fac[i * g + h] = f;
                l = fmaf(f, __ldcg(slot(i) + g * D + g + h), l);
            }
            l = warp_sum(l);
            if (lane == 0) {
                sum[h] = M;
                sum[g + h] = l;
            }
        }
        __syncthreads();
        const size_t head0 = static_cast<size_t>(unit / a.Hkv) * a.Hq + static_cast<size_t>(unit % a.Hkv) * g;
        for (int idx = threadIdx.x; idx < g * (D / 4); idx += NW * 32) {
            const int h = idx / (D / 4), e = (idx % (D / 4)) * 4;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
            for (int i = 0; i < n; ++i) {
                const float f = fac[i * g + h];
                const float4 v = __ldcg(reinterpret_cast<const float4*>(slot(i) + h * D + e));
                acc.x = fmaf(f, v.x, acc.x);
                acc.y = fmaf(f, v.y, acc.y);
                acc.z = fmaf(f, v.z, acc.z);
                acc.w = fmaf(f, v.w, acc.w);
            }
            const float l = sum[g + h];
            *reinterpret_cast<float4*>(a.out + (head0 + h) * D + e) =
                l > 0.f ? make_float4(acc.x / l, acc.y / l, acc.z / l, acc.w / l) : make_float4(0.f, 0.f, 0.f, 0.f);
            if (e == 0 && a.lse != nullptr) a.lse[head0 + h] = lse_of(sum[h], l);
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
    return launch_kernel(kern, dim3(a.ctas), dim3(P::NW * 32), smem, st, true, tmK, tmV, a);
}

// The deepest ring that fits beside the saved states and scratch, at most three stages.
constexpr int paged_stages(int nw, int stage, int nh, int d, int warp_floats) {
    for (int s = 3; s > 1; --s)
        if (nw * (s * stage + nh * d * 4 + warp_floats * 4) + 1024 <= PAGED_SMEM_MAX) return s;
    return 1;
}

}  // namespace kvs
