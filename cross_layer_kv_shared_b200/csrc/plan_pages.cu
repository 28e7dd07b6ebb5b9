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
//   page(position / page) * page + position % page; entries behind the last token get -1, and
//   so do tokens whose page lies outside the pool (reported)
// A few loads and prefix sums: bound by latency for a decode step and by the writes of the
// token arrays for prompts. Every block repeats the prefix sums over the sequences (a few
// microseconds at most) and fills its share of the token arrays; the last block to have read
// the lengths writes the new ones, which may take their place. Measured: 64 sequences of one
// token 3.4 us; 509 sequences, 65536 token entries, a tenth of the sequences leaving 5.0 us
// (9.7 us while a warp returned each sequence's pages by itself).
#include "kvs_device.cuh"
#include "kvs_paged.h"

namespace kvs {
namespace {

constexpr int NT = 1024;

// prefix sums saturate here: they only have to tell what exceeds 32-bit limits
__device__ __forceinline__ unsigned sat(unsigned a, unsigned b) { return min(a + b, 0x7fffffffu); }

// exclusive prefix sums over the block of N values at once; `sums` is [N][32], one per use
template <int N>
__device__ __forceinline__ void block_scan(unsigned (&v)[N], unsigned (*sums)[32]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    unsigned incl[N];
#pragma unroll
    for (int i = 0; i < N; ++i) incl[i] = v[i];
#pragma unroll
    for (int off = 1; off < 32; off <<= 1)
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const unsigned x = __shfl_up_sync(0xffffffffu, incl[i], off);
            if (lane >= off) incl[i] = sat(incl[i], x);
        }
    if (lane == 31)
#pragma unroll
        for (int i = 0; i < N; ++i) sums[i][warp] = incl[i];
    __syncthreads();
    unsigned base[N];
#pragma unroll
    for (int i = 0; i < N; ++i) base[i] = lane < warp ? sums[i][lane] : 0u;    // 32 warps: the sums before this one
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
#pragma unroll
        for (int i = 0; i < N; ++i) base[i] = sat(base[i], __shfl_xor_sync(0xffffffffu, base[i], off));
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const unsigned before = __shfl_up_sync(0xffffffffu, incl[i], 1);
        v[i] = sat(base[i], lane > 0 ? before : 0u);
    }
}

// E: sequences per thread
template <int E>
__global__ void __launch_bounds__(NT) plan_pages_kernel(const PagePlanArgs a) {
    extern __shared__ int sm[];
    int* s_start = sm;                    // [B + 1] first token
    int* s_len = s_start + a.B + 1;       // [B] tokens held
    int* s_new = s_len + a.B;             // [B] new pages of earlier sequences
    int* s_backx = s_new + a.B;           // [B] returning pages of earlier sequences
    __shared__ unsigned s_sum[5][32];
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
    unsigned want[E], need[E];
    bool leaves[E];
    unsigned at[2] = {0u, 0u};            // tokens wanted and pages needed, first of this thread's, then before them
    unsigned err = 0u;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const int b = threadIdx.x * E + e;
        n[e] = held[e] = 0;
        want[e] = need[e] = 0u;
        leaves[e] = false;
        if (b < a.B) {
            int len = a.lens[b];
            const int m = a.new_tokens[b];
            if (len < 0 || len > cap) {
                err |= ERR_RANGE;
                // which pages such a sequence holds is unknown: none returns
                len = m < 0 || len < 0 ? 0 : static_cast<int>(cap);
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
        at[0] = sat(at[0], want[e]);
        at[1] = sat(at[1], need[e]);
    }
    block_scan(at, s_sum);                // its barrier: every input of this block is read
    if (threadIdx.x == 0) {
        s_total[2] = 0;
        s_last = true;
        if (gridDim.x > 1) {
            unsigned prev;
            asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(prev) : "l"(a.counter) : "memory");
            s_last = prev == gridDim.x - 1;
            if (s_last) *a.counter = 0u;
        }
    }
    int got[E];
    unsigned sums[3] = {0u, 0u, 0u};      // tokens taken, new pages, pages of those that leave
#pragma unroll
    for (int e = 0; e < E; ++e) {
        at[0] = sat(at[0], want[e]);
        at[1] = sat(at[1], need[e]);
        const bool ok = (need[e] == 0u || at[1] <= static_cast<unsigned>(count)) && at[0] <= static_cast<unsigned>(a.max_tokens);
        if (!ok && want[e] > 0u) err |= ERR_POOL;
        got[e] = ok ? static_cast<int>(want[e]) : 0;
        if (!ok) need[e] = 0u;
        sums[0] += got[e];
        sums[1] += need[e];
        sums[2] += leaves[e] ? held[e] : 0;              // at most B * max_blocks, checked by the caller
    }
    block_scan(sums, s_sum + 2);
    int at_got = sums[0], at_new = sums[1], at_back = sums[2];
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
    auto exists = [&](int page) {         // reports a page outside the pool
        const bool ok = page >= 0 && page < a.num_pages;
        if (!ok) atomicOr(a.err, ERR_RANGE);
        return ok;
    };
    auto last_at_or_before = [&](const int* from, int x) {   // the last sequence with from[b] <= x
        int lo = 0, hi = a.B - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (from[mid] <= x) lo = mid;
            else hi = mid - 1;
        }
        return lo;
    };
    for (int b = blockIdx.x * NT + threadIdx.x; b <= a.B; b += gridDim.x * NT) a.token_start[b] = s_start[b];
    // ---- token arrays and new block-table entries
    for (int i = blockIdx.x * NT + threadIdx.x; i < a.max_tokens; i += gridDim.x * NT) {
        int pos = 0, slot = -1;
        if (i < tokens) {
            const int lo = last_at_or_before(s_start, i);
            pos = s_len[lo] + (i - s_start[lo]);
            const int blk = pos >> a.page_shift;
            const int k = blk - ((s_len[lo] + ps - 1) >> a.page_shift);
            int* entry = a.table + static_cast<size_t>(lo) * a.max_blocks + blk;
            const int page = k < 0 ? *entry : a.ring[ring_at(s_new[lo] + k)];
            if (k >= 0 && (pos & (ps - 1)) == 0) *entry = page;
            // a page the pool does not have gets no slot: its product with the page size could wrap
            // to another page's row
            if (exists(page)) slot = page * ps + (pos & (ps - 1));
        }
        a.slot_map[i] = slot;
        a.position[i] = pos;
    }
    // ---- pages that return, dealt evenly over the grid
    for (int r = blockIdx.x * NT + threadIdx.x; r < s_total[2]; r += gridDim.x * NT) {
        const int b = last_at_or_before(s_backx, r);
        const int page = a.table[static_cast<size_t>(b) * a.max_blocks + (r - s_backx[b])];
        exists(page);                     // reported; it keeps its place, so the count stands
        a.ring[ring_at(count + r)] = page;
    }
}

}  // namespace

template <int E>
static cudaError_t launch(const PagePlanArgs& a, int blocks, cudaStream_t st) {
    auto kern = plan_pages_kernel<E>;
    static std::atomic<unsigned long long> attr_done{0};
    cudaError_t e = once_per_device(attr_done, [&] {
        return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (4 * NT * E + 1) * 4);
    });
    if (e != cudaSuccess) return e;
    return launch_kernel(kern, dim3(blocks), dim3(NT), (4 * a.B + 1) * 4, st, true, a);
}

cudaError_t launch_plan_pages(const PagePlanArgs& a, int sms, cudaStream_t st) {
    static_assert(PLAN_MAX_BATCH <= 4 * NT, "sequences of a block");
    int blocks = (a.max_tokens + NT - 1) / NT;
    if (blocks > sms) blocks = sms;
    return a.B <= NT ? launch<1>(a, blocks, st) : launch<4>(a, blocks, st);
}

}  // namespace kvs
