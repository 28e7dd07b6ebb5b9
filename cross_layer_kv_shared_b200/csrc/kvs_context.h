// The library context and the host-side helpers every entry point uses.
#pragma once

#include "kvshare.h"

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <functional>
#include <unordered_map>
#include <vector>

namespace kvs {

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// cuTensorMapEncodeTiled of the loaded driver, or nullptr
EncodeTiledFn encode_fn();

struct MapKey {
    const void* ptr;
    uint64_t d0, d1, d2;
    uint32_t box0, box1;
    int dtype, swizzle;
    bool operator==(const MapKey& o) const {
        return ptr == o.ptr && d0 == o.d0 && d1 == o.d1 && d2 == o.d2 && box0 == o.box0 && box1 == o.box1 &&
               dtype == o.dtype && swizzle == o.swizzle;
    }
};

struct MapKeyHash {
    size_t operator()(const MapKey& k) const {
        size_t h = reinterpret_cast<uintptr_t>(k.ptr);
        for (uint64_t v : {k.d0, k.d1, k.d2, (uint64_t)k.box0, (uint64_t)k.box1, (uint64_t)k.dtype, (uint64_t)k.swizzle})
            h = h * 1000003u ^ std::hash<uint64_t>()(v);
        return h;
    }
};

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline bool is_device_ptr(const void* p) {
    if (p == nullptr) return false;
    cudaPointerAttributes at;
    if (cudaPointerGetAttributes(&at, p) != cudaSuccess) {
        cudaGetLastError();
        return false;
    }
    return at.type == cudaMemoryTypeDevice || at.type == cudaMemoryTypeManaged;
}

inline bool dev_ok(const void* p) { return p != nullptr && aligned16(p) && is_device_ptr(p); }

inline size_t elem_size(kvshare_dtype t) { return t == KVS_F32 ? 4 : 2; }

}  // namespace kvs

struct kvshare_ctx {
    kvshare_config cfg{};
    int device = 0;
    int sms = 148;
    float scale = 0.f;
    std::vector<kvshare_layer> map;
    bool map_set = false;
    float* w_dev = nullptr;          // [L][Hkv]
    std::vector<float> w_host;
    float* ws = nullptr;             // split partials
    size_t ws_floats = 0;
    unsigned* counters = nullptr;    // [max_batch * Hkv]
    unsigned* err = nullptr;         // status word
    int splits_override = 0;
    int kv_overlap = 0;
    int grid_override = 0;
    std::vector<int> order;          // layer order of decode calls (a permutation of 0..L-1)
    int stall_next = 0;
    long long wait_limit = 4000000000LL;     // ~2 s of SM clock
    long long stall_limit = 20000000LL;      // ~10 ms
    uint64_t launches = 0;
    std::unordered_map<kvs::MapKey, CUtensorMap, kvs::MapKeyHash> maps;
    // kept scores of one layer for the attention statistics [max_batch][Hq][max_context]
    float* sscore = nullptr;
    // projected queries of one low-rank prefill layer [max_batch][Hq][max_context][64] bf16
    uint16_t* qp = nullptr;
    // paged cache: split partials (two per CTA) and arrival counters (one per CTA and one for
    // planning, zero between launches)
    float* pg_ws = nullptr;
    unsigned* pg_counters = nullptr;
    // staging for kvshare_decode_host
    void* q_stage = nullptr;
    float* out_stage = nullptr;
    float* lse_stage = nullptr;
    // kvshare_decode_host: copy streams (host to device, device to host) and events that
    // pipeline chunks of layers (copies of one chunk under the decode of another)
    static constexpr int HOST_CHUNKS = 8;
    cudaStream_t h2d = nullptr, d2h = nullptr;
    cudaEvent_t ev_start = nullptr, ev_done = nullptr;
    cudaEvent_t ev_in[HOST_CHUNKS] = {}, ev_out[HOST_CHUNKS] = {};
};
