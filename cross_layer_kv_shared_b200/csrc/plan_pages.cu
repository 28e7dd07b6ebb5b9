// Pages and slots of one step of a paged cache, from the sequences' lengths.
//
// Sequence b has n_b cached tokens and takes m_b more (m_b < 0: it leaves, its pages return).
//   held_b = ceil(n_b / page), need_b = ceil((n_b + m_b) / page) - held_b
//   b is admitted iff need_b = 0 or the pages needed by 0 .. b fit the free ones, and the
//   tokens asked for by 0 .. b fit the token arrays (first come, first served)
//   the k-th new page is free ring entry (head + k) mod num_pages; pages that return follow
//   the ring's last in (sequence, block) order: the two stretches never overlap, so no block
//   of the launch waits for another
//   token i of the step (sequences end to end): position n_b + (i - start_b), slot =
//   page(position / page) * page + position % page; entries behind the last token get -1
// A few loads and prefix sums: bound by latency for a decode step and by the writes of the
// token arrays for prompts. Every block repeats the prefix sums over the sequences (a few
// microseconds at most) and fills its share of the token arrays; the last block to have read
// the lengths writes the new ones, which may take their place.
#include "kvs_device.cuh"
#include "kvs_paged.h"

namespace kvs {
namespace {

constexpr int NT = 1024;
constexpr int E = PLAN_MAX_BATCH / NT;

template <typename T>
__device__ T block_scan(T v, T* warp_sums) {         // exclusive prefix sum over the block
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    T incl = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const T x = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += x;
    }
    if (lane == 31) warp_sums[warp] = incl;
    __syncthreads();
    T base = lane < warp ? warp_sums[lane] : T(0);   // 32 warps: each adds up those before it
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) base += __shfl_xor_sync(0xffffffffu, base, off);
    __syncthreads();
    return base + incl - v;
}

__global__ void __launch_bounds__(NT) plan_pages_kernel(const PagePlanArgs a) {
    extern __shared__ int sm[];
    int* s_start = sm;                    // [B + 1] first token
    int* s_len = s_start + a.B + 1;       // [B] tokens held
    int* s_new = s_len + a.B;             // [B] new pages of earlier sequences
    int* s_back = s_new + a.B;            // [B] returning pages
    int* s_backx = s_back + a.B;          // [B] returning pages of earlier sequences
    __shared__ long long wsum[32];
    __shared__ int wsum32[32];
    __shared__ int s_total[3];            // tokens, new pages, returning pages
    __shared__ bool s_last;
    grid_dep_wait();
    if (threadIdx.x == 0) grid_dep_launch();
    const int ps = 1 << a.page_shift;
    const long long cap = static_cast<long long>(a.max_blocks) << a.page_shift;
    int head = a.ring_state[0], count = a.ring_state[1];
    const bool bad_ring = head < 0 || head >= a.num_pages || count < 0 || count > a.num_pages;
    if (bad_ring) {
        if (threadIdx.x == 0) atomicOr(a.err, ERR_RANGE);
        head = 0;
        count = 0;                        // an unusable ring has no free page
    }
    int n[E], held[E];
    long long want[E], need[E];
    bool leaves[E];
    long long sum_want = 0, sum_need = 0;
    unsigned err = 0u;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const int b = threadIdx.x * E + e;
        n[e] = held[e] = 0;
        want[e] = need[e] = 0;
        leaves[e] = false;
        if (b < a.B) {
            int len = a.lens[b];
            const int m = a.new_tokens[b];
            if (len < 0 || len > cap) {
                err |= ERR_RANGE;
                len = len < 0 ? 0 : static_cast<int>(cap);
            }
            n[e] = len;
            held[e] = (len + ps - 1) >> a.page_shift;
            leaves[e] = m < 0;
            if (m > 0) {
                if (static_cast<long long>(len) + m > cap) {
                    err |= ERR_RANGE;     // longer than its row of the block table
                } else {
                    want[e] = m;
                    need[e] = ((len + m + ps - 1) >> a.page_shift) - held[e];
                }
            }
        }
        sum_want += want[e];
        sum_need += need[e];
    }
    long long at_want = block_scan(sum_want, wsum);      // also: every input of this block is read
    if (gridDim.x > 1 && threadIdx.x == 0) {
        unsigned prev;
        asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(prev) : "l"(a.counter) : "memory");
        s_last = prev == gridDim.x - 1;
        if (s_last) *a.counter = 0u;
    } else if (threadIdx.x == 0) {
        s_last = true;
    }
    long long at_need = block_scan(sum_need, wsum);
    int got[E], sum_got = 0, sum_new = 0, sum_held = 0;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        at_want += want[e];
        at_need += need[e];
        const bool ok = (need[e] == 0 || at_need <= count) && at_want <= a.max_tokens;
        if (!ok && want[e] > 0) err |= ERR_POOL;
        got[e] = ok ? static_cast<int>(want[e]) : 0;
        if (!ok) need[e] = 0;
        sum_got += got[e];
        sum_new += static_cast<int>(need[e]);
        sum_held += leaves[e] ? held[e] : 0;             // at most B * max_blocks, checked by the caller
    }
    int at_got = block_scan(sum_got, wsum32);
    int at_new = block_scan(sum_new, wsum32);
    int at_back = block_scan(sum_held, wsum32);
    const int room = bad_ring ? 0 : a.num_pages - count;
    int sum_back = 0;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const int b = threadIdx.x * E + e;
        if (b >= a.B) continue;
        const int give = leaves[e] ? held[e] : 0;
        const bool fits = give == 0 || at_back + give <= room;   // more pages than the pool has: dropped
        if (!fits) err |= ERR_RANGE;
        s_start[b] = at_got;
        s_len[b] = n[e];
        s_new[b] = at_new;
        s_back[b] = fits ? give : 0;
        s_backx[b] = at_back;
        sum_back += fits ? give : 0;
        at_got += got[e];
        at_new += static_cast<int>(need[e]);
        at_back += give;
        if (b == a.B - 1) {
            s_start[a.B] = at_got;
            s_total[0] = at_got;
            s_total[1] = at_new;
        }
    }
    if (threadIdx.x == 0) s_total[2] = 0;
    __syncthreads();
    if (sum_back > 0) atomicAdd(&s_total[2], sum_back);
    if (err != 0u && blockIdx.x == 0) atomicOr(a.err, err);
    __syncthreads();
    const int tokens = s_total[0];
    // the new lengths and ring state: written once every block has read the old ones
    if (s_last) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int b = threadIdx.x * E + e;
            if (b < a.B) a.lens_out[b] = leaves[e] ? 0 : n[e] + got[e];
        }
        if (threadIdx.x == 0) {
            int h = head + s_total[1];
            a.ring_state_out[0] = h >= a.num_pages ? h - a.num_pages : h;
            a.ring_state_out[1] = count - s_total[1] + s_total[2];
        }
    }
    auto ring_at = [&](int k) {           // k < 2 num_pages from the head
        long long x = static_cast<long long>(head) + k;
        while (x >= a.num_pages) x -= a.num_pages;
        return static_cast<int>(x);
    };
    for (int b = blockIdx.x * NT + threadIdx.x; b <= a.B; b += gridDim.x * NT) a.token_start[b] = s_start[b];
    // ---- token arrays and new block-table entries
    for (int i = blockIdx.x * NT + threadIdx.x; i < a.max_tokens; i += gridDim.x * NT) {
        int pos = 0, slot = -1;
        if (i < tokens) {
            int lo = 0, hi = a.B - 1;     // the last sequence that starts at or before i
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (s_start[mid] <= i) lo = mid;
                else hi = mid - 1;
            }
            pos = s_len[lo] + (i - s_start[lo]);
            const int blk = pos >> a.page_shift;
            const int k = blk - ((s_len[lo] + ps - 1) >> a.page_shift);
            int* entry = a.table + static_cast<size_t>(lo) * a.max_blocks + blk;
            const int page = k < 0 ? *entry : a.ring[ring_at(s_new[lo] + k)];
            if (k >= 0 && (pos & (ps - 1)) == 0) *entry = page;
            slot = page * ps + (pos & (ps - 1));
        }
        a.slot_map[i] = slot;
        a.position[i] = pos;
    }
    // ---- pages that return, a warp per sequence
    const int lane = threadIdx.x & 31;
    for (int b = blockIdx.x * (NT / 32) + (threadIdx.x >> 5); b < a.B; b += gridDim.x * (NT / 32)) {
        const int give = s_back[b];
        for (int i = lane; i < give; i += 32)
            a.ring[ring_at(count + s_backx[b] + i)] = a.table[static_cast<size_t>(b) * a.max_blocks + i];
    }
}

}  // namespace

cudaError_t launch_plan_pages(const PagePlanArgs& a, int sms, cudaStream_t st) {
    const int smem = (5 * a.B + 1) * 4;
    static std::atomic<unsigned long long> attr_done{0};
    cudaError_t e = once_per_device(attr_done, [&] {
        return cudaFuncSetAttribute(plan_pages_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    (5 * PLAN_MAX_BATCH + 1) * 4);
    });
    if (e != cudaSuccess) return e;
    int blocks = (a.max_tokens + NT - 1) / NT;
    if (blocks > sms) blocks = sms;
    if (blocks < 1) blocks = 1;
    return launch_kernel(plan_pages_kernel, dim3(blocks), dim3(NT), smem, st, true, a);
}

}  // namespace kvs
