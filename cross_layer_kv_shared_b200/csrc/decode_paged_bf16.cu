// Paged decode, bf16 storage (schedule: decode_paged.cuh). Tokens are the M rows and the
// group's query heads the N columns of mma.sync m16n8k16, so a group of up to 8 heads wastes
// nothing on padding:
//   S^T = K Q^T;  MIX: S^T = w S1^T + (1 - w) S2^T in fp32
//   P^T = 2^(S^T - max), fp32
//   O^T += V^T P^T;  MIX: O^T += V1^T (w P)^T + V2^T ((1 - w) P)^T
// The outputs are fp32, so P keeps its 24 bits: it enters the product as three bf16 parts
// (p = p1 + p2 + p3 with p2 = bf16(p - p1), ...; the remainder is below 2^-24 p). One part
// would leave 2^-9 in every weight. The two extra products cost tensor issue slots that an
// HBM-bound loop has free. A tile's product starts from zero and is added to the running sum
// by one fp32 FMA (the rescaling FMA), because the tensor core's own accumulation truncates:
// over thousands of tokens that drift would exceed the fp32 rounding of everything else.
#include "decode_paged.cuh"

namespace kvs {
namespace {

template <int D_, bool MIX, int NH_>
struct PagedBf16 {
    static constexpr int D = D_, NH = NH_, NSRC = MIX ? 2 : 1;
    static constexpr int TT = D == 128 ? 16 : 32;
    static constexpr int SUBW = 64;
    static constexpr int STAGE = 2 * NSRC * TT * D * 2;
    // many warps with short rings: a tile's chain of dependent products takes longer than its
    // share of HBM time, so warps hide it (d = 128 mix: 60 us with 4 x 3 stages, 55.5 with 8 x 1;
    // d = 64: 15.1 us with 8 x 3, 14.6 with 8 x 2, 13.9 with 12 x 2; d = 128: 120.5 us with 8 x 2,
    // 125 with 10 x 2, 131 with 8 x 1)
    static constexpr int NW = !MIX && D == 64 && NH == 8 ? 12 : 8;
    static constexpr int WARP_FLOATS = 0;
    static constexpr int NSW = paged_stages(NW, STAGE, NH, D, WARP_FLOATS);
    static constexpr int MT = TT / 16, NB = NH / 8, TILE_BYTES = TT * D * 2;

    uint32_t qb[D / 16][NB][2];      // B fragments of Q^T: column n = head nb*8 + lane/4
    float o[D / 16][NB][4];          // O^T: rows = channels, columns = heads nb*8 + 2(lane%4) (+1)
    float m[NB][2], l[NB][2];        // log2-domain max and sum of those two heads
    float w, w1;
    int lane;

    __device__ void setup(float*, int lane_) { lane = lane_; }

    __device__ void begin(const PagedDecodeArgs& a, int b, int j) {
        const uint16_t* qg = static_cast<const uint16_t*>(a.q) + (static_cast<size_t>(b) * a.Hq + static_cast<size_t>(j) * a.g) * D;
        const int cq = 2 * (lane & 3);
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            const int h = nb * 8 + (lane >> 2);
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
                qb[ks][nb][0] = h < a.g ? *reinterpret_cast<const uint32_t*>(qg + h * D + ks * 16 + cq) : 0u;
                qb[ks][nb][1] = h < a.g ? *reinterpret_cast<const uint32_t*>(qg + h * D + ks * 16 + 8 + cq) : 0u;
            }
            m[nb][0] = m[nb][1] = NEG_INF;
            l[nb][0] = l[nb][1] = 0.f;
#pragma unroll
            for (int i = 0; i < D / 16; ++i) o[i][nb][0] = o[i][nb][1] = o[i][nb][2] = o[i][nb][3] = 0.f;
        }
        w = MIX ? a.w[j] : 1.f;
        w1 = 1.f - w;
    }

    // p0, p1: one row's weights of heads 2(lane%4), +1; the next part of them as a B fragment
    __device__ static uint32_t take_part(float& p0, float& p1) {
        const uint32_t x = pack_bf16(p0, p1);
        p0 -= bf16_lo(x);
        p1 -= bf16_hi(x);
        return movmatrix_t(x);
    }

    __device__ void tile(const PagedDecodeArgs& a, const uint8_t* st, int blk_stride, int sub_stride, const int* lim, bool cut) {
        const uint32_t kb = smem_u32(st), vb = kb + TILE_BYTES;
        const int mi = lane >> 3, ri = lane & 7;     // ldmatrix: matrix and row this lane addresses
        float sc[MT][NB][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            // even and odd channel steps accumulate apart: half the chain of dependent products
            float s1[2][NB][4], s2[2][NB][4];
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int i = 0; i < 4; ++i) s1[0][nb][i] = s1[1][nb][i] = s2[0][nb][i] = s2[1][nb][i] = 0.f;
            const int row = (mi & 1) * 8 + ri;
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
                const int c = ks * 2 + (mi >> 1);
                const uint32_t off = mt * blk_stride + (c >> 3) * sub_stride + swz128(row, c & 7);
                uint32_t af[4];
                ldsm_x4(kb + off, af[0], af[1], af[2], af[3]);
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) mma_bf16(s1[ks & 1][nb], af, qb[ks][nb][0], qb[ks][nb][1]);
                if (MIX) {
                    ldsm_x4(kb + 2 * TILE_BYTES + off, af[0], af[1], af[2], af[3]);
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb) mma_bf16(s2[ks & 1][nb], af, qb[ks][nb][0], qb[ks][nb][1]);
                }
            }
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    sc[mt][nb][i] = s1[0][nb][i] + s1[1][nb][i];
                    if (MIX) sc[mt][nb][i] = fmaf(w, sc[mt][nb][i], w1 * (s2[0][nb][i] + s2[1][nb][i]));
                }
            if (cut) {
                const int end = lim[mt] - (lane >> 2);    // rows r of this lane are tokens iff r < end
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if ((i >> 1) * 8 >= end) sc[mt][nb][i] = NEG_INF;
            }
        }
        // ---- online softmax per head, P^T in three parts
        constexpr int PARTS = 3;
        uint32_t pb[NSRC][MT][NB][PARTS][2];
        float corr[NB][2];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            float mx[2] = {NEG_INF, NEG_INF}, ref[2];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                mx[0] = fmaxf(mx[0], fmaxf(sc[mt][nb][0], sc[mt][nb][2]));
                mx[1] = fmaxf(mx[1], fmaxf(sc[mt][nb][1], sc[mt][nb][3]));
            }
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) {
                mx[0] = fmaxf(mx[0], __shfl_xor_sync(0xffffffffu, mx[0], off));
                mx[1] = fmaxf(mx[1], __shfl_xor_sync(0xffffffffu, mx[1], off));
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float mn = fmaxf(m[nb][i], mx[i] * a.scale_log2);
                ref[i] = mn == NEG_INF ? 0.f : mn;
                corr[nb][i] = ex2_approx(m[nb][i] - ref[i]);
                m[nb][i] = mn;
                l[nb][i] *= corr[nb][i];
            }
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                float pr[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) pr[i] = ex2_approx(fmaf(sc[mt][nb][i], a.scale_log2, -ref[i & 1]));
                l[nb][0] += pr[0] + pr[2];
                l[nb][1] += pr[1] + pr[3];
#pragma unroll
                for (int src = 0; src < NSRC; ++src) {
                    const float f = MIX ? (src == 0 ? w : w1) : 1.f;
                    float x0 = f * pr[0], x1 = f * pr[1], x2 = f * pr[2], x3 = f * pr[3];
#pragma unroll
                    for (int part = 0; part < PARTS; ++part) {
                        pb[src][mt][nb][part][0] = take_part(x0, x1);
                        pb[src][mt][nb][part][1] = take_part(x2, x3);
                    }
                }
            }
        }
        // ---- O^T = corr O^T + V^T P^T
#pragma unroll
        for (int dt = 0; dt < D / 16; ++dt) {
            float acc[NB][4];
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) acc[nb][0] = acc[nb][1] = acc[nb][2] = acc[nb][3] = 0.f;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                const int row = (mi >> 1) * 8 + ri;
                const int c = dt * 2 + (mi & 1);
                const uint32_t off = mt * blk_stride + (c >> 3) * sub_stride + swz128(row, c & 7);
#pragma unroll
                for (int src = 0; src < NSRC; ++src) {
                    uint32_t af[4];
                    ldsm_x4_t(vb + src * 2 * TILE_BYTES + off, af[0], af[1], af[2], af[3]);
#pragma unroll
                    for (int part = PARTS - 1; part >= 0; --part)
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb) mma_bf16(acc[nb], af, pb[src][mt][nb][part][0], pb[src][mt][nb][part][1]);
                }
            }
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[dt][nb][i] = fmaf(o[dt][nb][i], corr[nb][i & 1], acc[nb][i]);
        }
    }

    // sum the lanes' shares of l (each lane summed its own token rows)
    __device__ void finish() {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) {
                l[nb][0] += __shfl_xor_sync(0xffffffffu, l[nb][0], off);
                l[nb][1] += __shfl_xor_sync(0xffffffffu, l[nb][1], off);
            }
    }

    // A state's values as float4s in this order, so that saving and joining are 16-byte moves:
    // value (dt, nb) of lane i holds channels e, e + 8 of heads h, h + 1
    static constexpr int VALS = NB * (D / 16) * 32;
    template <typename F>
    __device__ void values(F f) const {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int dt = 0; dt < D / 16; ++dt)
                f((nb * (D / 16) + dt) * 32 + lane, make_float4(o[dt][nb][0], o[dt][nb][1], o[dt][nb][2], o[dt][nb][3]));
    }
    // the heads of value k: x and z belong to .x, y and w to .y
    __device__ static int2 heads(int k) {
        const int h = k / (32 * (D / 16)) * 8 + 2 * (k & 3);
        return make_int2(h, h + 1);
    }
    __device__ static bool first_of(int k) { return k % (32 * (D / 16)) < 4; }    // channel 0
    __device__ static void emit(float* out, int g, int k, const float4& v, float2 inv) {
        const int h = heads(k).x, e = (k / 32) % (D / 16) * 16 + (k & 31) / 4;
        float* at = out + h * D + e;
        if (h < g) {
            at[0] = v.x * inv.x;
            at[8] = v.z * inv.x;
        }
        if (h + 1 < g) {
            at[D] = v.y * inv.y;
            at[D + 8] = v.w * inv.y;
        }
    }
    __device__ float2 sums(int k) const {
        const int nb = k / (32 * (D / 16));
        return make_float2(l[nb][0], l[nb][1]);
    }

    template <typename F>
    __device__ void stats(int g, F f) {
        if (lane >= 4) return;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int h = nb * 8 + 2 * lane + i;
                if (h < g) f(h, m[nb][i], l[nb][i]);
            }
    }
};

template <int D, bool MIX>
cudaError_t launch_g(const CUtensorMap& tmK, const CUtensorMap& tmV, const PagedDecodeArgs& a, cudaStream_t st) {
    return a.g <= 8 ? launch_paged<PagedBf16<D, MIX, 8>>(tmK, tmV, a, st)
                    : launch_paged<PagedBf16<D, MIX, 16>>(tmK, tmV, a, st);
}

}  // namespace

int decode_paged_box_rows(bool f32, int d, int page_size) {
    const int tt = f32 || d == 128 ? 16 : 32;
    static_assert(PagedBf16<128, true, 8>::TT == 16 && PagedBf16<128, false, 8>::TT == 16 &&
                      PagedBf16<64, true, 8>::TT == 32 && PagedBf16<64, false, 8>::TT == 32,
                  "tile rows");
    return page_size < tt ? page_size : tt;
}

cudaError_t launch_decode_paged_bf16(int d, bool mix, const CUtensorMap& tmK, const CUtensorMap& tmV,
                                     const PagedDecodeArgs& a, cudaStream_t st) {
    if (d == 64) return mix ? launch_g<64, true>(tmK, tmV, a, st) : launch_g<64, false>(tmK, tmV, a, st);
    return mix ? launch_g<128, true>(tmK, tmV, a, st) : launch_g<128, false>(tmK, tmV, a, st);
}

}  // namespace kvs
