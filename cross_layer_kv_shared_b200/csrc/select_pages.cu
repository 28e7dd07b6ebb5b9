// Block selection of a paged decode: a cheap score of every page against the query, and the
// best `top` blocks of each (sequence, kv head).
//
//   query codes of head h:  s_q = fl(1/127) max_c |q_c|, c_q = rint(q / s_q)
//   page p:                 dot = sum_c (c_q > 0 ? c_q hi_c : c_q lo_c), an upper bound of
//                           q . k over the page's keys, in whole numbers
//   score_h = (dot s_q) s_p;  MIX: w score_h1 + (1 - w) score_h2;  score = max over the group
// The dot product is the whole-number product of [max(c_q, 0) | min(c_q, 0)] with [hi | lo]
// (below 2^22, exact in fp32 whatever the order), and every fp32 step after it is one IEEE
// operation, so the selection is reproducible bit for bit.
//
// select_score: bound by the codes' bytes (2 d + 4 per page and head). A warp takes 16 pages
// of a head: each lane reads 16-byte pieces of two pages' codes straight into the fragments
// of mma.sync m16n8k32 s8 (the product's index may be permuted freely as long as the query
// codes are laid out alike), the group's heads are its columns.
// select_top: one block per (sequence, kv head), bound by latency. Scores become ordered
// 32-bit keys in registers; the top-th largest is found bit by bit (a count over the block
// each), then the kept blocks are written in ascending order by a prefix sum. Ties go to the
// lowest block; the first and last blocks asked for are kept whatever their score.
#include "kvs_device.cuh"
#include "kvs_paged.h"

namespace kvs {
namespace {

constexpr int SCORE_WARPS = 8;
constexpr int SCORE_PAGES = SCORE_WARPS * 16;

__device__ __forceinline__ void mma_s8(int (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ int seq_tokens(const PagedSelectArgs& a, int b) {
    const int n = a.lens[b], cap = a.max_blocks << a.page_shift;
    if (n < 0 || n > cap) {
        atomicOr(a.err, ERR_RANGE);
        return n < 0 ? 0 : cap;
    }
    return n;
}

template <int D, bool F32, bool MIX, int NH>
__global__ void __launch_bounds__(SCORE_WARPS * 32) select_score_kernel(const PagedSelectArgs a) {
    constexpr int NB = NH / 8;
    constexpr int PIECES = 2 * D / 64;              // 64-byte steps of a page's codes
    __shared__ __align__(16) int8_t s_code[NH][2 * D];
    __shared__ float s_scale[NH];
    const int b = blockIdx.z, j = blockIdx.y;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    grid_dep_wait();
    if (threadIdx.x == 0) grid_dep_launch();
    const int held = (seq_tokens(a, b) + (1 << a.page_shift) - 1) >> a.page_shift;
    if (static_cast<int>(blockIdx.x) * SCORE_PAGES >= held) return;
    // ---- the group's query codes, positive part then negative part
    for (int h = warp; h < NH; h += SCORE_WARPS) {
        constexpr int PER = D / 32;
        float v[PER];
        float top = 0.f;
        const size_t at = (static_cast<size_t>(b) * a.Hq + static_cast<size_t>(j) * a.g + h) * D + lane * PER;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            v[i] = 0.f;
            if (h < a.g)
                v[i] = F32 ? static_cast<const float*>(a.q)[at + i]
                           : __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(a.q)[at + i]) << 16);
            top = fmaxf(top, fabsf(v[i]));
        }
        const float s = __fmul_rn(warp_max(top), INV_127);
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int c = s > 0.f ? __float2int_rn(__fdiv_rn(v[i], s)) : 0;
            s_code[h][lane * PER + i] = static_cast<int8_t>(max(c, 0));
            s_code[h][D + lane * PER + i] = static_cast<int8_t>(min(c, 0));
        }
        if (lane == 0) s_scale[h] = s;
    }
    __syncthreads();
    const int p0 = blockIdx.x * SCORE_PAGES + warp * 16;
    if (p0 >= held) return;
    // ---- pages p0 + lane / 4 and + 8
    const int r = lane >> 2, c4 = lane & 3;
    int page[2];
    float score[NB][4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int p = p0 + r + 8 * i;
        page[i] = p < held ? a.table[static_cast<size_t>(b) * a.max_blocks + p] : -1;
        if (p < held && (page[i] < 0 || page[i] >= a.num_pages)) {
            atomicOr(a.err, ERR_RANGE);
            page[i] = -1;                           // scores as a page of zeros
        }
    }
#pragma unroll
    for (int src = 0; src < (MIX ? 2 : 1); ++src) {
        const size_t slot = static_cast<size_t>(src == 0 ? a.src0 : a.src1) * a.num_pages;
        uint4 x[2][PIECES];
        float sp[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const size_t row = (slot + max(page[i], 0)) * a.Hkv + j;
            const uint4* at = reinterpret_cast<const uint4*>(a.codes + row * 2 * D) + c4;
            sp[i] = page[i] >= 0 ? a.scales[row] : 0.f;
#pragma unroll
            for (int k = 0; k < PIECES; ++k) x[i][k] = page[i] >= 0 ? __ldg(at + 4 * k) : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            int acc[4] = {0, 0, 0, 0};
            const uint4* qc = reinterpret_cast<const uint4*>(s_code[nb * 8 + r]) + c4;
#pragma unroll
            for (int k = 0; k < PIECES; ++k) {
                const uint4 q = qc[4 * k];
                const uint32_t a0[4] = {x[0][k].x, x[1][k].x, x[0][k].y, x[1][k].y};
                const uint32_t a1[4] = {x[0][k].z, x[1][k].z, x[0][k].w, x[1][k].w};
                mma_s8(acc, a0, q.x, q.y);
                mma_s8(acc, a1, q.z, q.w);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float s = __fmul_rn(__fmul_rn(static_cast<float>(acc[i]), s_scale[nb * 8 + 2 * c4 + (i & 1)]), sp[i >> 1]);
                if (!MIX) {
                    score[nb][i] = s;
                } else {
                    const float w = a.w[j];
                    score[nb][i] = src == 0 ? __fmul_rn(w, s) : __fadd_rn(score[nb][i], __fmul_rn(__fsub_rn(1.f, w), s));
                }
            }
        }
    }
    // ---- the group's largest score of each page
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        float top = NEG_INF;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int k = 0; k < 2; ++k)
                if (nb * 8 + 2 * c4 + k < a.g) top = fmaxf(top, score[nb][2 * i + k]);
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int p = p0 + r + 8 * i;
        if (c4 == 0 && p < held) a.score[(static_cast<size_t>(b) * a.Hkv + j) * a.max_blocks + p] = top;
    }
}

// An unsigned key in the order of the scores; NaN below every number.
__device__ __forceinline__ uint32_t score_key(float s) {
    if (s != s) return 0u;
    const uint32_t u = __float_as_uint(s == 0.f ? 0.f : s);     // -0 and 0 tie
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

template <int NT, int E>
__global__ void __launch_bounds__(NT) select_top_kernel(const PagedSelectArgs a) {
    constexpr int NWARP = NT / 32;
    __shared__ int s_cnt[2][NWARP];
    const int j = blockIdx.x, b = blockIdx.y;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    grid_dep_wait();
    if (threadIdx.x == 0) grid_dep_launch();
    const int held = (seq_tokens(a, b) + (1 << a.page_shift) - 1) >> a.page_shift;
    const size_t row = static_cast<size_t>(b) * a.Hkv + j;
    int* out = a.sel + row * a.top;
    if (held <= a.top) {                             // every block
        for (int i = threadIdx.x; i < a.top; i += NT) out[i] = i < held ? i : -1;
        return;
    }
    // thread t holds blocks t * E .. t * E + E - 1
    const float* score = a.score + row * a.max_blocks;
    uint32_t key[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const int p = threadIdx.x * E + e;
        key[e] = 0u;
        if (p < held) {
            key[e] = max(score_key(__ldcg(score + p)), 1u);     // 0 marks "no block"
            if (p < a.first || p >= held - a.last) key[e] = 0xffffffffu;
        }
    }
    // the largest T with at least `top` keys >= T, bit by bit
    uint32_t T = 0u;
    for (int bit = 31; bit >= 0; --bit) {
        const uint32_t cand = T | (1u << bit);
        int c = 0;
#pragma unroll
        for (int e = 0; e < E; ++e) c += key[e] >= cand ? 1 : 0;
        c = __reduce_add_sync(0xffffffffu, c);
        if (lane == 0) s_cnt[bit & 1][warp] = c;
        __syncthreads();
        int all = lane < NWARP ? s_cnt[bit & 1][lane] : 0;
        all = __reduce_add_sync(0xffffffffu, all);
        if (all >= a.top) T = cand;
    }
    // keep every key above T and the lowest blocks among those equal to it
    int above = 0, equal = 0;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        above += key[e] > T ? 1 : 0;
        equal += key[e] == T ? 1 : 0;
    }
    int ia = above, ie = equal;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, ia, off), y = __shfl_up_sync(0xffffffffu, ie, off);
        if (lane >= off) {
            ia += x;
            ie += y;
        }
    }
    __syncthreads();
    if (lane == 31) {
        s_cnt[0][warp] = ia;
        s_cnt[1][warp] = ie;
    }
    __syncthreads();
    int wa = lane < NWARP ? s_cnt[0][lane] : 0, we = lane < NWARP ? s_cnt[1][lane] : 0;
    const int all_above = __reduce_add_sync(0xffffffffu, wa);
    wa = __reduce_add_sync(0xffffffffu, lane < warp ? wa : 0);
    we = __reduce_add_sync(0xffffffffu, lane < warp ? we : 0);
    const int ties = a.top - all_above;
    int na = wa + ia - above, ne = we + ie - equal;  // kept or tied before this thread's blocks
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const bool up = key[e] > T, eq = key[e] == T;
        if (up || (eq && ne < ties)) out[na + min(ne, ties)] = threadIdx.x * E + e;
        na += up ? 1 : 0;
        ne += eq ? 1 : 0;
    }
}

template <int D, bool F32, bool MIX>
cudaError_t launch_score(const PagedSelectArgs& a, cudaStream_t st) {
    const dim3 grid((a.max_blocks + SCORE_PAGES - 1) / SCORE_PAGES, a.Hkv, a.B);
    return a.g <= 8 ? launch_kernel(select_score_kernel<D, F32, MIX, 8>, grid, dim3(SCORE_WARPS * 32), 0, st, true, a)
                    : launch_kernel(select_score_kernel<D, F32, MIX, 16>, grid, dim3(SCORE_WARPS * 32), 0, st, true, a);
}

template <bool F32, bool MIX>
cudaError_t launch_score_d(const PagedSelectArgs& a, cudaStream_t st) {
    return a.d == 64 ? launch_score<64, F32, MIX>(a, st) : launch_score<128, F32, MIX>(a, st);
}

}  // namespace

int launch_select_pages(const PagedSelectArgs& a, cudaStream_t st) {
    int launched = 0;
    if (a.max_blocks > a.top) {                      // otherwise every block is kept, whatever its score
        const cudaError_t e = a.f32 ? (a.mix ? launch_score_d<true, true>(a, st) : launch_score_d<true, false>(a, st))
                                    : (a.mix ? launch_score_d<false, true>(a, st) : launch_score_d<false, false>(a, st));
        if (e != cudaSuccess) return -1;
        ++launched;
    }
    const dim3 grid(a.Hkv, a.B);
    cudaError_t e;
    if (a.max_blocks <= 1024) e = launch_kernel(select_top_kernel<256, 4>, grid, dim3(256), 0, st, true, a);
    else if (a.max_blocks <= 4096) e = launch_kernel(select_top_kernel<512, 8>, grid, dim3(512), 0, st, true, a);
    else e = launch_kernel(select_top_kernel<1024, 16>, grid, dim3(1024), 0, st, true, a);
    if (e != cudaSuccess) return -1;
    return launched + 1;
}

}  // namespace kvs
