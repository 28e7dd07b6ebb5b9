// Paged decode, fp32 storage (schedule: decode_paged.cuh), on the fp32 units. Per 16-token tile:
//   scores: lane = (token t % 8, quarter of d); it holds tokens t and t + 8, so one read of a
//           query chunk from shared memory serves two tokens; the quarters' sums meet by
//           shuffles that leave each quarter with its own NH / 4 heads
//   softmax of those heads, the weights written to shared memory
//   output: lane = four channels (at d = 64 the half warps take alternate tokens); the weights
//           of a token are read as broadcasts
// 128-byte swizzled tiles keep every 16-byte read of K and V free of bank conflicts. At g = 8
// the loop takes about half of the fp32 issue slots that a tile's HBM time leaves; larger
// groups are bound by them.
#include "decode_paged.cuh"

namespace kvs {
namespace {

// Pairs of fp32 in one 64-bit register: one instruction for two multiply-adds (sm_100 on).
typedef unsigned long long pair_t;
__device__ __forceinline__ pair_t pack2(float x, float y) {
    pair_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ float2 unpack2(pair_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ void fma2(pair_t& d, pair_t a, pair_t b) {
    asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(d) : "l"(a), "l"(b));
}
__device__ __forceinline__ pair_t mul2(pair_t a, pair_t b) {
    pair_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

template <int D_, bool MIX, int NH_>
struct PagedF32 {
    static constexpr int D = D_, NH = NH_, NSRC = MIX ? 2 : 1;
    static constexpr int TT = 16;
    static constexpr int SUBW = 32;
    static constexpr int STAGE = 2 * NSRC * TT * D * 4;
    static constexpr int NW = STAGE <= 8192 || (STAGE <= 16384 && NH <= 8) ? 8 : 4;
    // queries of the unit, a head's quarters 16 bytes further apart than their length, so that the
    // four that a warp reads at once lie in different banks
    static constexpr int QQ = D / 4 + 4, QF = NH * 4 * QQ;
    static constexpr int WARP_FLOATS = QF + TT * NH + NH; // + weights [TT][NH] + corrections [NH]
    static constexpr int NSW = paged_stages(NW, STAGE, NH, D, WARP_FLOATS);
    static constexpr int SUB_BYTES = TT * 128, TILE_BYTES = TT * D * 4;
    static constexpr int HQ = NH / 4;                     // heads a quarter owns
    static constexpr int EL = D / 4;                      // lanes of one V row
    static constexpr int TP = 32 / EL;                    // V rows read at once
    static_assert(NH % 4 == 0, "heads are dealt to the quarters");

    pair_t o[NH][2];       // channels 4 (lane % EL) .. + 3; at TP = 2 the share of this half's tokens
    float m[HQ], l[HQ];    // heads quarter * HQ + i
    float w, w1;
    int lane;
    float* sq;
    float* sp;
    float* sc;

    __device__ void setup(float* scratch, int lane_) {
        lane = lane_;
        sq = scratch;
        sp = sq + QF;
        sc = sp + TT * NH;
    }

    __device__ void begin(const PagedDecodeArgs& a, int b, int j) {
        const float* qg = static_cast<const float*>(a.q) + (static_cast<size_t>(b) * a.Hq + static_cast<size_t>(j) * a.g) * D;
        __syncwarp();
        for (int i = lane; i < NH * D / 4; i += 32)
            *reinterpret_cast<float4*>(sq + i / (D / 16) * QQ + i % (D / 16) * 4) = 4 * i < a.g * D ? *reinterpret_cast<const float4*>(qg + 4 * i)
                                                                     : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int h = 0; h < NH; ++h) o[h][0] = o[h][1] = 0ull;
#pragma unroll
        for (int i = 0; i < HQ; ++i) {
            m[i] = NEG_INF;
            l[i] = 0.f;
        }
        w = MIX ? a.w[j] : 1.f;
        w1 = 1.f - w;
        __syncwarp();
    }

    // acc[r][h] = q_h . row (lane % 8 + 8 r) over this lane's quarter of the channels
    __device__ void dots(const uint8_t* kt, float (&acc)[2][NH]) const {
        const int row = lane & 7, quarter = lane >> 3;
        pair_t even_odd[2][NH];                           // sums of the even and of the odd channels
#pragma unroll
        for (int h = 0; h < NH; ++h) even_odd[0][h] = even_odd[1][h] = 0ull;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
            const int chunk = quarter * (D / 16) + i;     // 16-byte chunk of the row
            const uint32_t off = (chunk >> 3) * SUB_BYTES + swz128(row, chunk & 7);
            const ulonglong2 k0 = *reinterpret_cast<const ulonglong2*>(kt + off);
            const ulonglong2 k1 = *reinterpret_cast<const ulonglong2*>(kt + off + 8 * 128);
#pragma unroll
            for (int h = 0; h < NH; ++h) {
                const ulonglong2 q = *reinterpret_cast<const ulonglong2*>(sq + (h * 4 + quarter) * QQ + i * 4);
                fma2(even_odd[0][h], q.x, k0.x);
                fma2(even_odd[1][h], q.x, k1.x);
                fma2(even_odd[0][h], q.y, k0.y);
                fma2(even_odd[1][h], q.y, k1.y);
            }
        }
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int h = 0; h < NH; ++h) {
                const float2 x = unpack2(even_odd[r][h]);
                acc[r][h] = x.x + x.y;
            }
    }

    __device__ void tile(const PagedDecodeArgs& a, const uint8_t* st, int, int, const int* lim, bool cut) {
        const int quarter = lane >> 3;
        float acc[2][NH];
        dots(st, acc);
        if (MIX) {
            float acc2[2][NH];
            dots(st + 2 * TILE_BYTES, acc2);
#pragma unroll
            for (int h = 0; h < NH; ++h) {
                acc[0][h] = fmaf(w, acc[0][h], w1 * acc2[0][h]);
                acc[1][h] = fmaf(w, acc[1][h], w1 * acc2[1][h]);
            }
        }
        // each quarter keeps the sums of its own heads: halve the heads at each exchange
        float s[2][HQ];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            float half[NH / 2];
            const bool up = quarter & 2;
#pragma unroll
            for (int h = 0; h < NH / 2; ++h) {
                const float give = up ? acc[r][h] : acc[r][NH / 2 + h];
                const float keep = up ? acc[r][NH / 2 + h] : acc[r][h];
                half[h] = keep + __shfl_xor_sync(0xffffffffu, give, 16);
            }
            const bool odd = quarter & 1;
#pragma unroll
            for (int h = 0; h < HQ; ++h) {
                const float give = odd ? half[h] : half[HQ + h];
                const float keep = odd ? half[HQ + h] : half[h];
                s[r][h] = keep + __shfl_xor_sync(0xffffffffu, give, 8);
            }
        }
        if (cut) {
            const int end = lim[0];
#pragma unroll
            for (int r = 0; r < 2; ++r)
                if ((lane & 7) + 8 * r >= end)
#pragma unroll
                    for (int h = 0; h < HQ; ++h) s[r][h] = NEG_INF;
        }
        __syncwarp();                                     // the previous tile's weights have been read
#pragma unroll
        for (int h = 0; h < HQ; ++h) {
            float mx = fmaxf(s[0][h], s[1][h]);
#pragma unroll
            for (int off = 1; off < 8; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
            const float mn = fmaxf(m[h], mx * a.scale_log2);
            const float ref = mn == NEG_INF ? 0.f : mn;
            const float corr = ex2_approx(m[h] - ref);
            m[h] = mn;
            const float p0 = ex2_approx(fmaf(s[0][h], a.scale_log2, -ref));
            const float p1 = ex2_approx(fmaf(s[1][h], a.scale_log2, -ref));
            l[h] = fmaf(l[h], corr, p0 + p1);
            const int head = quarter * HQ + h;
            sp[(lane & 7) * NH + head] = p0;
            sp[((lane & 7) + 8) * NH + head] = p1;
            if ((lane & 7) == 0) sc[head] = corr;
        }
        __syncwarp();
#pragma unroll
        for (int h = 0; h < NH; ++h) {
            const pair_t c = pack2(sc[h], sc[h]);
            o[h][0] = mul2(o[h][0], c);
            o[h][1] = mul2(o[h][1], c);
        }
        const int chunk = lane % EL;
        const pair_t ww = pack2(w, w), ww1 = pack2(w1, w1);
#pragma unroll
        for (int i = 0; i < TT / TP; ++i) {
            const int t = i * TP + lane / EL;
            const uint32_t off = (chunk >> 3) * SUB_BYTES + swz128(t, chunk & 7);
            ulonglong2 v = *reinterpret_cast<const ulonglong2*>(st + TILE_BYTES + off);
            if (MIX) {
                const ulonglong2 v2 = *reinterpret_cast<const ulonglong2*>(st + 3 * TILE_BYTES + off);
                pair_t x = mul2(ww1, v2.x), y = mul2(ww1, v2.y);
                fma2(x, ww, v.x);
                fma2(y, ww, v.y);
                v.x = x;
                v.y = y;
            }
#pragma unroll
            for (int h4 = 0; h4 < NH / 4; ++h4) {
                const float4 p = *reinterpret_cast<const float4*>(sp + t * NH + 4 * h4);
                const float pw[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const pair_t pp = pack2(pw[x], pw[x]);
                    fma2(o[4 * h4 + x][0], pp, v.x);
                    fma2(o[4 * h4 + x][1], pp, v.y);
                }
            }
        }
    }

    __device__ void finish() {
#pragma unroll
        for (int h = 0; h < HQ; ++h)
#pragma unroll
            for (int off = 1; off < 8; off <<= 1) l[h] += __shfl_xor_sync(0xffffffffu, l[h], off);
        if (TP == 2)
#pragma unroll
            for (int h = 0; h < NH; ++h)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const float2 own = unpack2(o[h][x]), other = unpack2(__shfl_xor_sync(0xffffffffu, o[h][x], 16));
                    o[h][x] = pack2(own.x + other.x, own.y + other.y);
                }
        __syncwarp();
        if ((lane & 7) == 0)
#pragma unroll
            for (int h = 0; h < HQ; ++h) sc[(lane >> 3) * HQ + h] = l[h];
        __syncwarp();
    }

    // a state's values as float4s: head k / EL, channels 4 (k % EL) ..
    static constexpr int VALS = NH * EL;
    template <typename F>
    __device__ void values(F f) const {
        if (lane >= EL) return;
#pragma unroll
        for (int h = 0; h < NH; ++h) {
            const float2 x = unpack2(o[h][0]), y = unpack2(o[h][1]);
            f(h * EL + lane, make_float4(x.x, x.y, y.x, y.y));
        }
    }
    __device__ static int2 heads(int k) { return make_int2(k / EL, k / EL); }
    __device__ static bool first_of(int k) { return k % EL == 0; }    // channel 0
    __device__ static void emit(float* out, int g, int k, const float4& v, float2 inv) {
        if (k / EL < g) *reinterpret_cast<float4*>(out + 4 * k) = make_float4(v.x * inv.x, v.y * inv.x, v.z * inv.x, v.w * inv.x);
    }
    __device__ float2 sums(int k) const { return make_float2(sc[k / EL], sc[k / EL]); }

    template <typename F>
    __device__ void stats(int g, F f) {
        if ((lane & 7) != 0) return;
#pragma unroll
        for (int i = 0; i < HQ; ++i) {
            const int h = (lane >> 3) * HQ + i;
            if (h < g) f(h, m[i], l[i]);
        }
    }
};

template <int D, bool MIX>
cudaError_t launch_g(const CUtensorMap& tmK, const CUtensorMap& tmV, const PagedDecodeArgs& a, cudaStream_t st) {
    if (a.g <= 4) return launch_paged<PagedF32<D, MIX, 4>>(tmK, tmV, a, st);
    if (a.g <= 8) return launch_paged<PagedF32<D, MIX, 8>>(tmK, tmV, a, st);
    return launch_paged<PagedF32<D, MIX, 16>>(tmK, tmV, a, st);
}

}  // namespace

cudaError_t launch_decode_paged_f32(int d, bool mix, const CUtensorMap& tmK, const CUtensorMap& tmV,
                                    const PagedDecodeArgs& a, cudaStream_t st) {
    if (d == 64) return mix ? launch_g<64, true>(tmK, tmV, a, st) : launch_g<64, false>(tmK, tmV, a, st);
    return mix ? launch_g<128, true>(tmK, tmV, a, st) : launch_g<128, false>(tmK, tmV, a, st);
}

}  // namespace kvs
