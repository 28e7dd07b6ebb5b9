// Internal declarations of the paged cache's kernels (planning, append, block selection,
// decode) shared with their host entry points.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kvs_internal.h"

namespace kvs {

constexpr float INV_127 = 1.0f / 127.0f;   // int8 scales are max |x| times this
constexpr int PAGE_MIN_SHIFT = 4;    // 16 tokens
constexpr int PAGE_MAX_SHIFT = 8;    // 256 tokens

// One layer of a paged decode. Pointers are already offset to the layer.
struct PagedDecodeArgs {
    const void* q;          // [B][Hq][d] config dtype
    float* out;             // [B][Hq][d]
    float* lse;             // [B][Hq] or nullptr
    const int* table;       // [B][max_blocks] page of each block of a sequence
    const int* lens;        // [B] tokens of each sequence
    const int* sel;         // [B][Hkv][top] block indices to attend to, or nullptr: every block
    const float* w;         // [Hkv] mix weights of this layer, MIX only
    int src0, src1;         // slots
    int B, Hq, Hkv, g;
    int num_pages, max_blocks, page_shift, top;
    float scale_log2;       // softmax scale * log2(e)
    float* ws;              // split partials: two slots per CTA (paged_partial floats each)
    unsigned* counters;     // [CTAs] arrival counters, zero between launches
    unsigned* err;
    long long wait_limit;
    int ctas;               // grid: at most one CTA per SM
    int aligned;            // one CTA per unit (set by the launcher)
    long long stall_limit;  // test hook: > 0: one thread waits that long on a barrier nothing arrives on
};
// rows of the K/V tensor-map boxes (tokens per copy)
int decode_paged_box_rows(bool f32, int d, int page_size);
cudaError_t launch_decode_paged_bf16(int d, bool mix, const CUtensorMap& tmK, const CUtensorMap& tmV,
                                     const PagedDecodeArgs& a, cudaStream_t st);
cudaError_t launch_decode_paged_f32(int d, bool mix, const CUtensorMap& tmK, const CUtensorMap& tmV,
                                    const PagedDecodeArgs& a, cudaStream_t st);
// floats of one partial: nh (padded) heads' o, then their (m, l) pairs; slots stay 16-byte aligned
__host__ __device__ constexpr int paged_partial(int nh, int d) { return nh * (d + 2); }
// floats one CTA may need in PagedDecodeArgs::ws
inline size_t paged_ws_floats(int g, int d) { return 2 * static_cast<size_t>(paged_partial(g <= 8 ? 8 : 16, d)); }

// Block selection of one layer.
struct PagedSelectArgs {
    const void* q;              // [B][Hq][d] config dtype
    const int8_t* codes;        // [slots][num_pages][Hkv][2][d]
    const float* scales;        // [slots][num_pages][Hkv]
    const int* table;
    const int* lens;
    const float* w;             // [Hkv], MIX only
    int* sel;                   // [B][Hkv][top]
    int src0, src1;
    int B, Hq, Hkv, g, d;
    int num_pages, max_blocks, page_shift, top, first, last;
    int cluster;                // CTAs per (sequence, kv head), set by the launcher
    bool f32, mix;
    unsigned* err;
};
constexpr int SELECT_MAX_BLOCKS = 16384;
cudaError_t launch_select_pages(const PagedSelectArgs& a, int sms, cudaStream_t st);

// Append of new tokens to one slot.
struct PagedAppendArgs {
    const void* k_new; const void* v_new;   // token i, head j at i * stride + j * d elements
    long long k_stride, v_stride;
    const int* slot_map;                    // [tokens]
    void* k; void* v;                       // the slot's [num_pages][Hkv][page][d]
    int8_t* codes; float* scales;           // the slot's [num_pages][Hkv][2][d], [num_pages][Hkv], or nullptr
    int tokens, Hkv, d, page_shift, num_pages;
    bool f32;
    unsigned* err;
};
cudaError_t launch_append_paged(const PagedAppendArgs& a, int sms, cudaStream_t st);

// Pages and slots of a step.
struct PagePlanArgs {
    const int* lens; const int* new_tokens;     // [B]
    int* table;                                 // [B][max_blocks]
    int* ring;                                  // [num_pages]
    const int* ring_state;                      // {head, count}
    int* lens_out; int* ring_state_out;         // [B], [2]
    int* token_start;                           // [B + 1]
    int* slot_map; int* position;               // [max_tokens]
    int B, max_blocks, num_pages, max_tokens, page_shift;
    unsigned* counter;                          // arrival counter, zero between launches
    unsigned* err;
};
constexpr int PLAN_MAX_BATCH = 4096;
cudaError_t launch_plan_pages(const PagePlanArgs& a, int sms, cudaStream_t st);

}  // namespace kvs
