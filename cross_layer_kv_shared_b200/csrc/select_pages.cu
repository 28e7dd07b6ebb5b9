// Block selection of a paged decode: a cheap score of every page against the query, and the
// best `top` blocks of each (sequence, kv head). Ranking pages by per-channel extremes of their
// keys is a published idea (query-aware page selection, Tang et al., 2024).
//
//   query codes of head h:  s_q = fl(1/127) max_c |q_c|, c_q = rint(q / s_q)
//   page p:                 dot = sum_c (c_q > 0 ? c_q hi_c : c_q lo_c): times both scales an
//                           upper bound of q~ . k over the page's keys, q~ = s_q c_q the rounded
//                           query; q . k may lie above it by at most s_q / 2 sum |k|
//   score_h = (dot s_q) s_p;  MIX: w score_h1 + (1 - w) score_h2;  score = max over the group
// The dot product is the whole-number product of [max(c_q, 0) | min(c_q, 0)] with [hi | lo]
// (below 2^22, exact in fp32 whatever the order), and every fp32 step after it is one IEEE
// operation, so the selection is reproducible bit for bit.
//
// One cluster of 1 to 8 CTAs per (sequence, kv head). Scores: bound by the codes' bytes
// (2 d + 4 per page). A warp takes 16 pages: each lane reads 16-byte pieces of two pages' codes
// straight into the fragments of mma.sync m16n8k32 s8 (the product's index may be permuted
// freely as long as the query codes are laid out alike), the group's heads are its columns.
// The scores, as ordered 32-bit keys, go into the first CTA's shared memory (distributed shared
// memory from the others), so they never travel to L2 and no second launch waits for them.
// Choice: bound by latency, in the first CTA. The keys move to registers; the top-th largest is
// found bit by bit from the highest bit that differs, a count over the block each, ending as
// soon as exactly `top` keys are at or above the candidate; the kept blocks are written in
// ascending order by a prefix sum. Ties go to the lowest block; the first and last blocks asked
// for are kept whatever their score. Measured: 8 heads x 512 pages 6.1 us, 64 rows x 1024 pages
// of 128 channels 7.7 us (17 MB of codes), both mostly the chain of dependent steps; a step's
// codes are requested before the query codes are made (9.2 -> 7.7 us). Two CTAs on a
// multiprocessor for twice the cluster: 11.6 us (they do not fit at once), or 9.1 us at 64
// registers, with spills.
#include "kvs_device.cuh"
#include "kvs_paged.h"

namespace kvs {
namespace {

constexpr int NT = 512;
constexpr int NWARP = NT / 32;
constexpr int MAX_CLUSTER = 8;

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

// An unsigned key in the order of the scores, above 0; NaN below every number.
__device__ __forceinline__ uint32_t score_key(float s) {
    if (s != s) return 1u;
    const uint32_t u = __float_as_uint(s == 0.f ? 0.f : s);     // -0 and 0 tie
    return max((u & 0x80000000u) ? ~u : (u | 0x80000000u), 1u);
}

// the address of `p` (own shared memory) in the shared memory of the cluster's CTA 0
__device__ __forceinline__ uint32_t in_first_cta(const void* p) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(smem_u32(p)));
    return r;
}
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// E: keys per thread of the choosing CTA
template <int D, bool F32, bool MIX, int NH, int E>
__global__ void __launch_bounds__(NT) select_pages_kernel(const PagedSelectArgs a) {
    constexpr int NB = NH / 8;
    constexpr int PIECES = 2 * D / 64;              // 64-byte steps of a page's codes
    extern __shared__ uint32_t s_key[];             // [blocks] (CTA 0's is the one used)
    __shared__ __align__(16) int8_t s_code[NH][2 * D];
    __shared__ float s_scale[NH];
    __shared__ uint2 s_cnt[2][NWARP];
    __shared__ uint32_t s_mm[2][NWARP];
    const int C = a.cluster, rank = C > 1 ? static_cast<int>(cluster_rank()) : 0;
    const int unit = blockIdx.x / C, b = unit / a.Hkv, j = unit - b * a.Hkv;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // CTA 0 must run before its memory is written to: arrive now, wait where that begins
    if (C > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    grid_dep_wait();
    if (threadIdx.x == 0) grid_dep_launch();
    // the first step's pages and this warp's query are on their way beside the length
    const int r = lane >> 2, c4 = lane & 3;
    const int* table = a.table + static_cast<size_t>(b) * a.max_blocks;
    int first_page[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int p = (rank * NWARP + warp) * 16 + r + 8 * i;
        first_page[i] = p < a.max_blocks ? table[p] : -1;
    }
    constexpr int PER = D / 32;
    float v[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        v[i] = 0.f;
        const size_t at = (static_cast<size_t>(b) * a.Hq + static_cast<size_t>(j) * a.g + warp) * D + lane * PER + i;
        if (warp < a.g)
            v[i] = F32 ? static_cast<const float*>(a.q)[at]
                       : __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(a.q)[at]) << 16);
    }
    const int held = (seq_tokens(a, b) + (1 << a.page_shift) - 1) >> a.page_shift;
    int* out = a.sel + static_cast<size_t>(unit) * a.top;
    if (held <= a.top) {                            // every block, whatever its score (the whole cluster)
        if (rank == 0)
            for (int i = threadIdx.x; i < a.top; i += NT) out[i] = i < held ? i : -1;
        if (C > 1) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
        return;
    }
    // ---- a step's codes and scales: pages p0 + r and + 8, from each source
    constexpr int NS = MIX ? 2 : 1;
    const int begin = (rank * NWARP + warp) * 16;
    uint4 x[NS][2][PIECES];
    float sp[NS][2];
    auto load = [&](int p0) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int p = p0 + r + 8 * i;
            int page = p >= held ? -1 : p0 == begin ? first_page[i] : table[p];
            if (p < held && (page < 0 || page >= a.num_pages)) {
                atomicOr(a.err, ERR_RANGE);
                page = -1;                          // scores as a page of zeros
            }
#pragma unroll
            for (int src = 0; src < NS; ++src) {
                const size_t row = (static_cast<size_t>(src == 0 ? a.src0 : a.src1) * a.num_pages + max(page, 0)) * a.Hkv + j;
                const uint4* at = reinterpret_cast<const uint4*>(a.codes + row * 2 * D) + c4;
                sp[src][i] = page >= 0 ? a.scales[row] : 0.f;
#pragma unroll
                for (int k = 0; k < PIECES; ++k) x[src][i][k] = page >= 0 ? __ldg(at + 4 * k) : make_uint4(0u, 0u, 0u, 0u);
            }
        }
    };
    if (begin < held) load(begin);
    // ---- the group's query codes, positive part then negative part
    static_assert(NH <= NWARP, "a warp per head");
    if (warp < NH) {
        float top = 0.f;
#pragma unroll
        for (int i = 0; i < PER; ++i) top = fmaxf(top, fabsf(v[i]));
        const float s = __fmul_rn(warp_max(top), INV_127);
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int c = s > 0.f ? __float2int_rn(__fdiv_rn(v[i], s)) : 0;
            s_code[warp][lane * PER + i] = static_cast<int8_t>(max(c, 0));
            s_code[warp][D + lane * PER + i] = static_cast<int8_t>(min(c, 0));
        }
        if (lane == 0) s_scale[warp] = s;
    }
    __syncthreads();
    if (C > 1) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    // ---- scores: 16 pages a warp and step, dealt over the cluster
    const uint32_t keys0 = C > 1 ? in_first_cta(s_key) : smem_u32(s_key);
    for (int p0 = begin; p0 < held;) {
        float score[NB][4];
#pragma unroll
        for (int src = 0; src < NS; ++src) {
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                int acc[4] = {0, 0, 0, 0};
                const uint4* qc = reinterpret_cast<const uint4*>(s_code[nb * 8 + r]) + c4;
#pragma unroll
                for (int k = 0; k < PIECES; ++k) {
                    const uint4 q = qc[4 * k];
                    const uint32_t a0[4] = {x[src][0][k].x, x[src][1][k].x, x[src][0][k].y, x[src][1][k].y};
                    const uint32_t a1[4] = {x[src][0][k].z, x[src][1][k].z, x[src][0][k].w, x[src][1][k].w};
                    mma_s8(acc, a0, q.x, q.y);
                    mma_s8(acc, a1, q.z, q.w);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float s = __fmul_rn(__fmul_rn(static_cast<float>(acc[i]), s_scale[nb * 8 + 2 * c4 + (i & 1)]), sp[src][i >> 1]);
                    if (!MIX) {
                        score[nb][i] = s;
                    } else {
                        const float w = a.w[j];
                        score[nb][i] = src == 0 ? __fmul_rn(w, s) : __fadd_rn(score[nb][i], __fmul_rn(__fsub_rn(1.f, w), s));
                    }
                }
            }
        }
        const int done = p0;
        p0 += C * NWARP * 16;
        if (p0 < held) load(p0);                    // on its way while this step's scores are placed
#pragma unroll
        for (int i = 0; i < 2; ++i) {               // the group's largest score of each page
            float top = NEG_INF;
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    if (nb * 8 + 2 * c4 + k < a.g) top = fmaxf(top, score[nb][2 * i + k]);
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const int p = done + r + 8 * i;
            if (c4 == 0 && p < held) {
                const uint32_t key = p < a.first || p >= held - a.last ? 0xffffffffu : score_key(top);
                asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(keys0 + 4u * p), "r"(key) : "memory");
            }
        }
    }
    if (C > 1) cluster_sync();
    else __syncthreads();
    if (rank != 0) return;
    // ---- thread t holds blocks t * E .. t * E + E - 1; 0: no block
    uint32_t key[E];
    uint32_t hi = 0u, lo = 0xffffffffu;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const int p = threadIdx.x * E + e;
        key[e] = p < held ? s_key[p] : 0u;
        if (p < held) {
            hi = max(hi, key[e]);
            lo = min(lo, key[e]);
        }
    }
    hi = __reduce_max_sync(0xffffffffu, hi);
    lo = __reduce_min_sync(0xffffffffu, lo);
    if (lane == 0) {
        s_mm[0][warp] = hi;
        s_mm[1][warp] = lo;
    }
    __syncthreads();
    hi = __reduce_max_sync(0xffffffffu, lane < NWARP ? s_mm[0][lane] : 0u);
    lo = __reduce_min_sync(0xffffffffu, lane < NWARP ? s_mm[1][lane] : 0xffffffffu);
    // T: at least `top` keys are >= T. The bits above the highest that differs are common
    int bit = hi == lo ? -1 : 31 - __clz(hi ^ lo);
    uint32_t T = hi == lo ? lo : lo & ~((2u << bit) - 1u);
    // two bits a step: the counts of the three candidates, two of them in one word
    bool found = false;
    for (int step = 0; bit >= 0 && !found; bit -= 2, ++step) {
        const int low = bit > 0 ? bit - 1 : 0;
        const uint32_t unit_k = 1u << low, c1 = T + unit_k, c2 = bit > 0 ? T + 2u * unit_k : c1, c3 = bit > 0 ? T + 3u * unit_k : c1;
        unsigned n12 = 0u, n3 = 0u;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            n12 += (key[e] >= c1 ? 1u : 0u) + (key[e] >= c2 ? 0x10000u : 0u);
            n3 += key[e] >= c3 ? 1u : 0u;
        }
        n12 = __reduce_add_sync(0xffffffffu, n12);
        n3 = __reduce_add_sync(0xffffffffu, n3);
        if (lane == 0) s_cnt[step & 1][warp] = make_uint2(n12, n3);
        __syncthreads();
        const uint2 own = lane < NWARP ? s_cnt[step & 1][lane] : make_uint2(0u, 0u);
        const unsigned a12 = __reduce_add_sync(0xffffffffu, own.x), top = a.top;
        const unsigned k1 = a12 & 0xffffu, k2 = a12 >> 16, k3 = __reduce_add_sync(0xffffffffu, own.y);
        const unsigned got = k3 >= top ? k3 : k2 >= top ? k2 : k1;
        T = k3 >= top ? c3 : k2 >= top ? c2 : k1 >= top ? c1 : T;
        found = got == top;                         // exactly the wanted blocks: the same for every thread
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
    if (lane == 31) s_cnt[0][warp] = make_uint2(ia, ie);
    __syncthreads();
    const uint2 per_warp = lane < NWARP ? s_cnt[0][lane] : make_uint2(0u, 0u);
    int wa = per_warp.x, we = per_warp.y;
    const int ties = a.top - __reduce_add_sync(0xffffffffu, wa);
    wa = __reduce_add_sync(0xffffffffu, lane < warp ? wa : 0);
    we = __reduce_add_sync(0xffffffffu, lane < warp ? we : 0);
    int na = wa + ia - above, ne = we + ie - equal;  // kept or tied before this thread's blocks
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const bool up = key[e] > T, eq = key[e] == T;
        if (up || (eq && ne < ties)) out[na + min(ne, ties)] = threadIdx.x * E + e;
        na += up ? 1 : 0;
        ne += eq ? 1 : 0;
    }
}

template <int D, bool F32, bool MIX, int NH, int E>
cudaError_t launch(const PagedSelectArgs& args, int sms, cudaStream_t st) {
    PagedSelectArgs a = args;
    auto kern = select_pages_kernel<D, F32, MIX, NH, E>;
    static std::atomic<unsigned long long> attr_done{0};
    cudaError_t e = once_per_device(attr_done, [&] {
        return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, NT * E * 4);
    });
    if (e != cudaSuccess) return e;
    // CTAs per (sequence, kv head): as many as have a multiprocessor each and the blocks can use
    const int units = a.B * a.Hkv;
    a.cluster = 1;
    while (a.cluster < MAX_CLUSTER && units * a.cluster * 2 <= sms && a.cluster * NWARP * 16 < a.max_blocks) a.cluster *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(units * a.cluster);
    cfg.blockDim = dim3(NT);
    cfg.dynamicSmemBytes = static_cast<size_t>(a.max_blocks) * 4;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = a.cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = a.cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, a);
}

template <int D, bool F32, bool MIX, int NH>
cudaError_t launch_e(const PagedSelectArgs& a, int sms, cudaStream_t st) {
    if (a.max_blocks <= 2 * NT) return launch<D, F32, MIX, NH, 2>(a, sms, st);
    if (a.max_blocks <= 8 * NT) return launch<D, F32, MIX, NH, 8>(a, sms, st);
    return launch<D, F32, MIX, NH, 32>(a, sms, st);
}

template <bool F32, bool MIX>
cudaError_t launch_d(const PagedSelectArgs& a, int sms, cudaStream_t st) {
    if (a.d == 64) return a.g <= 8 ? launch_e<64, F32, MIX, 8>(a, sms, st) : launch_e<64, F32, MIX, 16>(a, sms, st);
    return a.g <= 8 ? launch_e<128, F32, MIX, 8>(a, sms, st) : launch_e<128, F32, MIX, 16>(a, sms, st);
}

}  // namespace

cudaError_t launch_select_pages(const PagedSelectArgs& a, int sms, cudaStream_t st) {
    static_assert(SELECT_MAX_BLOCKS <= 32 * NT, "keys of the longest list");
    if (a.f32) return a.mix ? launch_d<true, true>(a, sms, st) : launch_d<true, false>(a, sms, st);
    return a.mix ? launch_d<false, true>(a, sms, st) : launch_d<false, false>(a, sms, st);
}

}  // namespace kvs
