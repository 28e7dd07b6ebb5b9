// Paged decode, fp32 storage (schedule: decode_paged.cuh), on the fp32 units. Per 16-token tile:
//   scores: lane = (token t % 8, quarter of d); it holds tokens t and t + 8, so one read of a
//           query chunk from shared memory serves two tokens; the quarters' sums meet by
//           shuffles that leave each quarter with its own NH / 4 heads
//   softmax of those heads, the weights written to shared memory
//   output: lane = four channels (at d = 64 the half warps take alternate tokens); the weights
//           of a token are read as broadcasts
// 128-byte swizzled tiles keep every 16-byte read of K and V free of bank conflicts. 16 requests of
// 4K to 8K tokens, 4 kv heads, share of the measured copy rate by group size (d 64, d 64 two
// sources, d 128, d 128 two sources): up to 4 heads 82, 93, 92, 97 %; 8 heads 63, 81, 74, 59 %;
// 16 heads 41, 31, 27, 33 %. At 8 and 16 the one or two warps that a scheduler has wait on their
// own chains of reads and multiply-adds; short calls lose more (32 us where HBM needs 14, 8 heads,
// 8K tokens; 55 us for 7, 16 heads, 4K tokens).
// Tensor cores with tf32 operands in two parts were hardly faster (30 and 45 us) and lost
// precision (1.5e-6 against 3e-7); paired multiply-adds gained 4 % and spilled at 16.
#include "decode_paged.cuh"

namespace kvs {
namespace {

template <int D_, bool MIX, int NH_>
struct PagedF32 {
    static constexpr int D = D_, NH = NH_, NSRC = MIX ? 2 : 1;
    static constexpr int TT = 16;
    static constexpr int SUBW = 32;
    static constexpr int STAGE = 2 * NSRC * TT * D * 4;
    static constexpr int NW = STAGE <= 8192 || (STAGE <= 16384 && NH <= 8) ? 8 : 4;
    static constexpr int QF = NH * D;                     // queries of the unit
    static constexpr int WARP_FLOATS = QF + TT * NH + NH; // + weights [TT][NH] + corrections [NH]
    static constexpr int NSW = paged_stages(NW, STAGE, NH, D, WARP_FLOATS);
    static constexpr int SUB_BYTES = TT * 128, TILE_BYTES = TT * D * 4;
    static constexpr int HQ = NH / 4;                     // heads a quarter owns
    static constexpr int EL = D / 4;                      // lanes of one V row
    static constexpr int TP = 32 / EL;                    // V rows read at once
    static_assert(NH % 4 == 0, "heads are dealt to the quarters");

    float o[NH][4];        // channels 4 (lane % EL) .. + 3; at TP = 2 the share of this half's tokens
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
            *reinterpret_cast<float4*>(sq + 4 * i) = 4 * i < a.g * D ? *reinterpret_cast<const float4*>(qg + 4 * i)
                                                                     : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int h = 0; h < NH; ++h) o[h][0] = o[h][1] = o[h][2] = o[h][3] = 0.f;
#pragma unroll
        for (int i = 0; i < HQ; ++i) {
            m[i] = NEG_INF;
            l[i] = 0.f;
        }
        w = MIX ? a.w[j] : 1.f;
        w1 = 1.f - w;
        __syncwarp();
    }

    // acc[r][h] += q_h . row (lane % 8 + 8 r) over this lane's quarter of the channels
    __device__ void dots(const uint8_t* kt, float (&acc)[2][NH]) const {
        const int row = lane & 7, quarter = lane >> 3;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
            const int chunk = quarter * (D / 16) + i;     // 16-byte chunk of the row
            const uint32_t off = (chunk >> 3) * SUB_BYTES + swz128(row, chunk & 7);
            const float4 k0 = *reinterpret_cast<const float4*>(kt + off);
            const float4 k1 = *reinterpret_cast<const float4*>(kt + off + 8 * 128);
#pragma unroll
            for (int h = 0; h < NH; ++h) {
                const float4 q = *reinterpret_cast<const float4*>(sq + h * D + chunk * 4);
                acc[0][h] = fmaf(q.w, k0.w, fmaf(q.z, k0.z, fmaf(q.y, k0.y, fmaf(q.x, k0.x, acc[0][h]))));
                acc[1][h] = fmaf(q.w, k1.w, fmaf(q.z, k1.z, fmaf(q.y, k1.y, fmaf(q.x, k1.x, acc[1][h]))));
            }
        }
    }

    __device__ void tile(const PagedDecodeArgs& a, const uint8_t* st, int, int, const int* lim, bool cut) {
        const int quarter = lane >> 3;
        float acc[2][NH];
#pragma unroll
        for (int h = 0; h < NH; ++h) acc[0][h] = acc[1][h] = 0.f;
        dots(st, acc);
        if (MIX) {
            float acc2[2][NH];
#pragma unroll
            for (int h = 0; h < NH; ++h) acc2[0][h] = acc2[1][h] = 0.f;
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
            const float c = sc[h];
            o[h][0] *= c;
            o[h][1] *= c;
            o[h][2] *= c;
            o[h][3] *= c;
        }
        const int chunk = lane % EL;
#pragma unroll
        for (int i = 0; i < TT / TP; ++i) {
            const int t = i * TP + lane / EL;
            const uint32_t off = (chunk >> 3) * SUB_BYTES + swz128(t, chunk & 7);
            float4 v = *reinterpret_cast<const float4*>(st + TILE_BYTES + off);
            if (MIX) {
                const float4 v2 = *reinterpret_cast<const float4*>(st + 3 * TILE_BYTES + off);
                v = make_float4(fmaf(w, v.x, w1 * v2.x), fmaf(w, v.y, w1 * v2.y), fmaf(w, v.z, w1 * v2.z),
                                fmaf(w, v.w, w1 * v2.w));
            }
#pragma unroll
            for (int h4 = 0; h4 < NH / 4; ++h4) {
                const float4 p = *reinterpret_cast<const float4*>(sp + t * NH + 4 * h4);
                const float pw[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    o[4 * h4 + x][0] = fmaf(pw[x], v.x, o[4 * h4 + x][0]);
                    o[4 * h4 + x][1] = fmaf(pw[x], v.y, o[4 * h4 + x][1]);
                    o[4 * h4 + x][2] = fmaf(pw[x], v.z, o[4 * h4 + x][2]);
                    o[4 * h4 + x][3] = fmaf(pw[x], v.w, o[4 * h4 + x][3]);
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
                for (int x = 0; x < 4; ++x) o[h][x] += __shfl_xor_sync(0xffffffffu, o[h][x], 16);
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
        for (int h = 0; h < NH; ++h) f(h * EL + lane, make_float4(o[h][0], o[h][1], o[h][2], o[h][3]));
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
