// Append new tokens to one slot of a paged cache: K and V rows into the rows the slot map
// names, and, where kept, each written page's key bounds.
//
//   k[page][j][row] = k_new[i][j], v likewise, (page, row) = slot_map[i] / page, % page
//   hi_c = max, lo_c = min over the page's rows 0 .. r of channel c (r: the last row this call
//   writes there), s = fl(1/127) max_c max(|hi_c|, |lo_c|),
//   codes min(127, ceil(hi_c / s)) and max(-127, floor(lo_c / s)): rounded outwards, so that
//   s * code bounds the page's keys up to the rounding of the product.
// Every step is one IEEE fp32 operation, so the codes are reproducible bit for bit.
//
// Bound by HBM for prompts (each row read and written once) and by latency for a decode step.
// One launch, two kinds of blocks. Copy blocks: a thread keeps one 16-byte piece of a token
// (K or V, head, piece) and walks the block's tokens, so its offsets are computed once and
// neighbouring threads write neighbouring bytes. Bound blocks: a warp per (page, head) reads
// the new rows from the input and the earlier ones from the page (which this call does not
// write), so it needs nothing from the copy blocks; theirs is the longer chain, so they come
// first in the grid. 8191 tokens x 8 heads x 128 out of 12 KB rows, six pools and inputs in turn
// (407 MB): 12.5 us for the rows alone (5.4 TB/s; 82 % of the measured copy rate), 15.9 us with
// bounds (7.8 and 12.1 us out of L2, one pool again and again). One fused pass (a block per
// page and two heads, extremes kept while copying) took 20.2 us: it reads the input's wide rows
// in 512-byte pieces at different times.
#include "kvs_device.cuh"
#include "kvs_paged.h"

namespace kvs {
namespace {

constexpr int NT = 256;
constexpr int UNROLL = 8;

struct Grid {
    int bound_blocks, bound_tokens;   // bound blocks (first in the grid: theirs is the longer chain) and the tokens of each
    int copy_tokens;                  // tokens of a copy block
};

__device__ __forceinline__ bool slot_ok(const PagedAppendArgs& a, int slot) {
    if (slot < 0) return false;
    if ((slot >> a.page_shift) >= a.num_pages) {
        atomicOr(a.err, ERR_RANGE);
        return false;
    }
    return true;
}

template <int RB>   // bytes of a row (one head)
__device__ void copy_tokens(const PagedAppendArgs& a, int first, int count) {
    constexpr int P = RB / 16;                          // 16-byte pieces of a row
    const int per = 2 * a.Hkv * P;                      // pieces of a token
    const int es = a.f32 ? 4 : 2;
    const int end = min(first + count, a.tokens);
    for (int c0 = 0; c0 < per; c0 += NT) {
        const int span = min(per - c0, NT);             // pieces in this pass
        const int side = NT / span;                     // tokens taken side by side
        const int mine = threadIdx.x / span;
        if (mine >= side) continue;
        const int c = c0 + threadIdx.x % span;
        const bool is_v = c >= a.Hkv * P;
        const int j = (c - (is_v ? a.Hkv * P : 0)) / P;
        const int piece = c % P;
        const char* src = static_cast<const char*>(is_v ? a.v_new : a.k_new) + j * RB + piece * 16;
        const long long step = (is_v ? a.v_stride : a.k_stride) * es;
        char* dst = static_cast<char*>(is_v ? a.v : a.k) + piece * 16;
        const int mask = (1 << a.page_shift) - 1;
        for (int i0 = first + mine; i0 < end; i0 += side * UNROLL) {
            uint4 x[UNROLL];
            int slot[UNROLL];
#pragma unroll
            for (int u = 0; u < UNROLL; ++u) {
                const int i = i0 + u * side;
                slot[u] = i < end ? a.slot_map[i] : -1;
                if (i < end) x[u] = __ldg(reinterpret_cast<const uint4*>(src + i * step));
            }
#pragma unroll
            for (int u = 0; u < UNROLL; ++u) {
                if (!slot_ok(a, slot[u])) continue;
                const long long row = ((static_cast<long long>(slot[u] >> a.page_shift) * a.Hkv + j) << a.page_shift) + (slot[u] & mask);
                *reinterpret_cast<uint4*>(dst + row * RB) = x[u];
            }
        }
    }
}

// element k of a 16-byte piece, as fp32
template <bool F32>
__device__ __forceinline__ float elem(const uint4& x, int k) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    if (F32) return __uint_as_float(w[k]);
    return (k & 1) ? bf16_hi(w[k >> 1]) : bf16_lo(w[k >> 1]);
}

template <bool F32, int RB>
__device__ void bound_page(const PagedAppendArgs& a, int i, int slot, int j) {
    constexpr int P = RB / 16;                          // lanes of a row
    constexpr int E = F32 ? 4 : 8;                      // elements of a piece
    constexpr int ROWS = 32 / P;                        // rows a warp reads at once
    constexpr int ES = F32 ? 4 : 2;
    const int lane = threadIdx.x & 31;
    const int r1 = slot & ((1 << a.page_shift) - 1);
    // rows of this page that the call writes: the tokens before i that hold the slots before
    int fresh = 0;
    for (int k0 = 0; k0 <= r1; k0 += 32) {
        const int k = k0 + lane;
        const unsigned no = __ballot_sync(0xffffffffu, !(k <= r1 && k <= i && a.slot_map[max(i - k, 0)] == slot - k));
        if (no != 0u) {
            fresh = k0 + __ffs(no) - 1;
            break;
        }
        fresh = k0 + 32;
    }
    const size_t page = slot >> a.page_shift;
    const char* held = static_cast<const char*>(a.k) + (((page * a.Hkv + j) << a.page_shift) * RB) + (lane % P) * 16;
    const char* in = static_cast<const char*>(a.k_new) + j * RB + (lane % P) * 16;
    const int old = r1 + 1 - fresh;
    float hi[E], lo[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
        hi[e] = NEG_INF;
        lo[e] = -NEG_INF;
    }
    constexpr int DEEP = 16;                            // rows of a lane in flight
    for (int r = lane / P; r <= r1; r += ROWS * DEEP) {
        uint4 x[DEEP];
#pragma unroll
        for (int u = 0; u < DEEP; ++u) {
            const int row = min(r + u * ROWS, r1);      // the last row again changes nothing
            const char* at = row < old ? held + static_cast<size_t>(row) * RB
                                       : in + (static_cast<long long>(i - (r1 - row)) * a.k_stride) * ES;
            x[u] = *reinterpret_cast<const uint4*>(at);
        }
#pragma unroll
        for (int u = 0; u < DEEP; ++u)
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const float v = elem<F32>(x[u], e);
                hi[e] = fmaxf(hi[e], v);
                lo[e] = fminf(lo[e], v);
            }
    }
    float top = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
#pragma unroll
        for (int off = P; off < 32; off <<= 1) {
            hi[e] = fmaxf(hi[e], __shfl_xor_sync(0xffffffffu, hi[e], off));
            lo[e] = fminf(lo[e], __shfl_xor_sync(0xffffffffu, lo[e], off));
        }
        top = fmaxf(top, fmaxf(fabsf(hi[e]), fabsf(lo[e])));
    }
    const float scale = __fmul_rn(warp_max(top), INV_127);
    if (lane < P) {
        uint32_t ch[E / 4], cl[E / 4];
#pragma unroll
        for (int w = 0; w < E / 4; ++w) {
            ch[w] = cl[w] = 0u;
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                int x = 0, y = 0;
                if (scale > 0.f) {
                    x = __float2int_rn(fminf(ceilf(__fdiv_rn(hi[4 * w + b], scale)), 127.f));
                    y = __float2int_rn(fmaxf(floorf(__fdiv_rn(lo[4 * w + b], scale)), -127.f));
                }
                ch[w] |= static_cast<uint32_t>(x & 0xff) << (8 * b);
                cl[w] |= static_cast<uint32_t>(y & 0xff) << (8 * b);
            }
        }
        int8_t* out = a.codes + (page * a.Hkv + j) * 2 * a.d + lane * E;
#pragma unroll
        for (int w = 0; w < E / 4; ++w) {
            *reinterpret_cast<uint32_t*>(out + 4 * w) = ch[w];
            *reinterpret_cast<uint32_t*>(out + a.d + 4 * w) = cl[w];
        }
        if (lane == 0) a.scales[page * a.Hkv + j] = scale;
    }
}

template <bool F32, int RB>
__global__ void __launch_bounds__(NT) append_paged_kernel(const PagedAppendArgs a, const Grid gr) {
    grid_dep_wait();
    if (threadIdx.x == 0) grid_dep_launch();
    if (static_cast<int>(blockIdx.x) >= gr.bound_blocks) {
        copy_tokens<RB>(a, (blockIdx.x - gr.bound_blocks) * gr.copy_tokens, gr.copy_tokens);
        return;
    }
    // a page's last written row carries the page: the next token is elsewhere, or it is row page - 1
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int first = blockIdx.x * gr.bound_tokens;
    const int i = first + lane;
    bool ends = false;
    if (lane < gr.bound_tokens && i < a.tokens) {
        const int slot = a.slot_map[i];
        if (slot_ok(a, slot)) {
            const int mask = (1 << a.page_shift) - 1;
            ends = (slot & mask) == mask || i + 1 == a.tokens || a.slot_map[i + 1] != slot + 1;
        }
    }
    unsigned todo = __ballot_sync(0xffffffffu, ends);
    int task = 0;
    while (todo != 0u) {
        const int t = first + __ffs(todo) - 1;
        todo &= todo - 1u;
        const int slot = a.slot_map[t];
        for (int j = 0; j < a.Hkv; ++j, ++task)
            if (task % (NT / 32) == warp) bound_page<F32, RB>(a, t, slot, j);
    }
}

template <bool F32, int RB>
cudaError_t launch(const PagedAppendArgs& a, int sms, cudaStream_t st) {
    Grid gr;
    // copy blocks: every thread has up to UNROLL pieces in flight; fewer when that would leave
    // fewer than two blocks a multiprocessor
    const int per = 2 * a.Hkv * (RB / 16);
    const int side = per >= NT ? 1 : NT / per;
    int tokens = side * UNROLL;
    while (tokens > side && (a.tokens + tokens - 1) / tokens < 2 * sms) tokens = (tokens / side + 1) / 2 * side;
    gr.copy_tokens = tokens;
    int blocks = (a.tokens + tokens - 1) / tokens;
    gr.bound_tokens = 1;
    gr.bound_blocks = 0;
    if (a.codes != nullptr) {
        const int bt = (a.tokens + 4 * sms - 1) / (4 * sms);    // four blocks a multiprocessor, at most 32 tokens each
        gr.bound_tokens = bt > 32 ? 32 : bt;
        gr.bound_blocks = (a.tokens + gr.bound_tokens - 1) / gr.bound_tokens;
        blocks += gr.bound_blocks;
    }
    return launch_kernel(append_paged_kernel<F32, RB>, dim3(blocks), dim3(NT), 0, st, true, a, gr);
}

}  // namespace

cudaError_t launch_append_paged(const PagedAppendArgs& a, int sms, cudaStream_t st) {
    if (a.f32) return a.d == 64 ? launch<true, 256>(a, sms, st) : launch<true, 512>(a, sms, st);
    return a.d == 64 ? launch<false, 128>(a, sms, st) : launch<false, 256>(a, sms, st);
}

}  // namespace kvs
