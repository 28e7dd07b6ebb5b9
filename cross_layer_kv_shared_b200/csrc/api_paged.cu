// Host side of the paged cache's entry points: argument validation, tensor maps, launches.
// See include/kvshare.h.
#include <cstring>

#include "kvs_context.h"
#include "kvs_internal.h"
#include "kvs_paged.h"

using namespace kvs;

namespace {

constexpr long long INT_LIMIT = 1LL << 31;
constexpr long long TOKEN_LIMIT = 1LL << 30;   // tokens of a sequence or of one call, counted in int with room to round up

// Makes the context's device current for a call and the caller's current again after it.
struct DeviceScope {
    int prev = -1;
    bool ok;
    explicit DeviceScope(int device) {
        ok = cudaGetDevice(&prev) == cudaSuccess && (prev == device || cudaSetDevice(device) == cudaSuccess);
        moved = ok && prev != device;
    }
    ~DeviceScope() {
        if (moved) cudaSetDevice(prev);
    }
    bool moved = false;
};

// memory of the context's device (or managed), aligned to `align` bytes
bool on_device(const kvshare_ctx* c, const void* p, unsigned align) {
    if (p == nullptr || (reinterpret_cast<uintptr_t>(p) & (align - 1u))) return false;
    cudaPointerAttributes at;
    if (cudaPointerGetAttributes(&at, p) != cudaSuccess) {
        cudaGetLastError();
        return false;
    }
    return (at.type == cudaMemoryTypeDevice && at.device == c->device) || at.type == cudaMemoryTypeManaged;
}

// log2 of a supported page size, or -1
int page_shift(int page_size) {
    for (int s = PAGE_MIN_SHIFT; s <= PAGE_MAX_SHIFT; ++s)
        if (page_size == 1 << s) return s;
    return -1;
}

// what every call over a pool needs of it (not the table and lengths)
kvshare_status check_pool(const kvshare_ctx* c, const kvshare_pages* p) {
    if (p == nullptr || p->slots < 1 || p->num_pages < 1 || page_shift(p->page_size) < 0) return KVS_EINVAL;
    if (static_cast<long long>(p->num_pages) * p->page_size >= INT_LIMIT) return KVS_EINVAL;
    const long long rows = static_cast<long long>(p->num_pages) * c->cfg.num_kv_heads;
    if (rows >= INT_LIMIT || rows * p->slots >= INT_LIMIT) return KVS_EINVAL;
    if (!on_device(c, p->k, 16) || !on_device(c, p->v, 16)) return KVS_EINVAL;
    return KVS_OK;
}

kvshare_status check_tables(const kvshare_ctx* c, const kvshare_pages* p) {
    if (p->batch < 1 || p->batch > c->cfg.max_batch || p->max_blocks < 1) return KVS_EINVAL;
    if ((static_cast<long long>(p->max_blocks) - 1) * p->page_size >= c->cfg.max_context) return KVS_EINVAL;
    // tokens of a sequence, and 16-token tiles of the batch, counted in 32 bits
    if (static_cast<long long>(p->max_blocks) * p->page_size > TOKEN_LIMIT) return KVS_EINVAL;
    if (static_cast<long long>(p->batch) * p->max_blocks * (p->page_size / 16) >= INT_LIMIT / c->cfg.num_kv_heads)
        return KVS_EUNSUPPORTED;
    if (!on_device(c, p->block_table, 4) || !on_device(c, p->lengths, 4)) return KVS_EINVAL;
    return KVS_OK;
}

// the layers of a decode or selection call
kvshare_status check_layers(const kvshare_ctx* c, const kvshare_pages* p, int l0, int l1) {
    if (l0 < 0 || l1 > c->cfg.num_layers || l0 > l1) return KVS_EINVAL;
    for (int l = l0; l < l1; ++l) {
        const kvshare_layer& e = c->map[l];
        if (e.kind == KVS_SRC_LOWRANK) return KVS_EUNSUPPORTED;
        if (e.src0 < 0 || e.src0 >= p->slots) return KVS_EINVAL;
        if (e.kind == KVS_SRC_MIX && (e.src1 < 0 || e.src1 >= p->slots)) return KVS_EINVAL;
    }
    return KVS_OK;
}

// [rows][page][d] of a pool as [rows][128-byte column block][page][columns]: a box of
// `box_rows` tokens and every column block lands in shared memory block by block, each
// 128-byte swizzled, in one copy
bool pool_map(const kvshare_ctx* c, const kvshare_pages* p, const void* base, int box_rows, CUtensorMap* out) {
    EncodeTiledFn fn = encode_fn();
    if (fn == nullptr) return false;
    const bool f32 = c->cfg.dtype == KVS_F32;
    const cuuint64_t es = elem_size(c->cfg.dtype), d = c->cfg.head_dim, cols = 128 / es;
    cuuint64_t dims[4] = {cols, static_cast<cuuint64_t>(p->page_size), d / cols,
                          static_cast<cuuint64_t>(p->slots) * p->num_pages * c->cfg.num_kv_heads};
    cuuint64_t strides[3] = {d * es, 128, d * es * p->page_size};
    cuuint32_t box[4] = {static_cast<cuuint32_t>(cols), static_cast<cuuint32_t>(box_rows), static_cast<cuuint32_t>(d / cols), 1u};
    cuuint32_t estr[4] = {1u, 1u, 1u, 1u};
    return fn(out, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
              const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

extern "C" {

kvshare_status kvshare_plan_pages(kvshare_t ctx, const int* lengths, const int* new_tokens, int* block_table, int* ring,
                                  const int* ring_state, int* lengths_out, int* ring_state_out, int* token_start,
                                  int* slot_map, int* position, int batch, int max_blocks, int page_size, int num_pages,
                                  int max_tokens, void* stream) {
    if (ctx == nullptr) return KVS_EINVAL;
    const int shift = page_shift(page_size);
    if (batch < 1 || max_blocks < 1 || shift < 0 || num_pages < 1 || max_tokens < 1) return KVS_EINVAL;
    if (static_cast<long long>(batch) * max_blocks >= INT_LIMIT ||
        static_cast<long long>(max_blocks) * page_size > TOKEN_LIMIT || max_tokens > TOKEN_LIMIT ||
        static_cast<long long>(num_pages) * page_size >= INT_LIMIT)
        return KVS_EINVAL;
    if (batch > PLAN_MAX_BATCH) return KVS_EUNSUPPORTED;
    const void* ps[] = {lengths, new_tokens, block_table, ring, ring_state, lengths_out, ring_state_out,
                        token_start, slot_map, position};
    for (const void* p : ps)
        if (!on_device(ctx, p, 4)) return KVS_EINVAL;
    DeviceScope scope(ctx->device);
    if (!scope.ok) return KVS_ECUDA;
    PagePlanArgs a;
    std::memset(&a, 0, sizeof(a));
    a.lens = lengths;
    a.new_tokens = new_tokens;
    a.table = block_table;
    a.ring = ring;
    a.ring_state = ring_state;
    a.lens_out = lengths_out;
    a.ring_state_out = ring_state_out;
    a.token_start = token_start;
    a.slot_map = slot_map;
    a.position = position;
    a.B = batch;
    a.max_blocks = max_blocks;
    a.num_pages = num_pages;
    a.max_tokens = max_tokens;
    a.page_shift = shift;
    a.counter = ctx->pg_counters + ctx->sms;
    a.err = ctx->err;
    if (launch_plan_pages(a, ctx->sms, static_cast<cudaStream_t>(stream)) != cudaSuccess) return KVS_ECUDA;
    ++ctx->launches;
    return KVS_OK;
}

kvshare_status kvshare_append_paged(kvshare_t ctx, const kvshare_pages* pages, int slot, const void* k_new,
                                    const void* v_new, long long k_stride, long long v_stride, const int* slot_map,
                                    int tokens, void* stream) {
    if (ctx == nullptr) return KVS_EINVAL;
    kvshare_status s = check_pool(ctx, pages);
    if (s != KVS_OK) return s;
    const kvshare_config& cf = ctx->cfg;
    if (slot < 0 || slot >= pages->slots || tokens < 0 || tokens > TOKEN_LIMIT) return KVS_EINVAL;
    if (tokens == 0) return KVS_OK;
    const long long es = static_cast<long long>(elem_size(cf.dtype)), row = static_cast<long long>(cf.num_kv_heads) * cf.head_dim;
    if (k_stride < row || v_stride < row || (k_stride * es) % 16 != 0 || (v_stride * es) % 16 != 0) return KVS_EINVAL;
    if (!on_device(ctx, k_new, 16) || !on_device(ctx, v_new, 16) || !on_device(ctx, slot_map, 4)) return KVS_EINVAL;
    const bool bounds = pages->bound_codes != nullptr;
    if (bounds && (!on_device(ctx, pages->bound_codes, 16) || !on_device(ctx, pages->bound_scale, 4))) return KVS_EINVAL;
    DeviceScope scope(ctx->device);
    if (!scope.ok) return KVS_ECUDA;
    PagedAppendArgs a;
    std::memset(&a, 0, sizeof(a));
    const size_t heads = static_cast<size_t>(slot) * pages->num_pages * cf.num_kv_heads;   // (page, head) rows before the slot
    const size_t at = heads * pages->page_size * cf.head_dim * es;
    a.k_new = k_new;
    a.v_new = v_new;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.slot_map = slot_map;
    // the pool the decode reads is the one the append writes
    a.k = static_cast<char*>(const_cast<void*>(pages->k)) + at;
    a.v = static_cast<char*>(const_cast<void*>(pages->v)) + at;
    a.codes = bounds ? const_cast<int8_t*>(pages->bound_codes) + heads * 2 * cf.head_dim : nullptr;
    a.scales = bounds ? const_cast<float*>(pages->bound_scale) + heads : nullptr;
    a.tokens = tokens;
    a.Hkv = cf.num_kv_heads;
    a.d = cf.head_dim;
    a.page_shift = page_shift(pages->page_size);
    a.num_pages = pages->num_pages;
    a.f32 = cf.dtype == KVS_F32;
    a.err = ctx->err;
    if (launch_append_paged(a, ctx->sms, static_cast<cudaStream_t>(stream)) != cudaSuccess) return KVS_ECUDA;
    ++ctx->launches;
    return KVS_OK;
}

kvshare_status kvshare_decode_paged(kvshare_t ctx, const kvshare_pages* pages, const void* q, float* out, float* lse,
                                    const int* selected, int top, int l0, int l1, void* stream) {
    if (ctx == nullptr || !ctx->map_set) return KVS_EINVAL;
    kvshare_status s = check_pool(ctx, pages);
    if (s == KVS_OK) s = check_tables(ctx, pages);
    if (s == KVS_OK) s = check_layers(ctx, pages, l0, l1);
    if (s != KVS_OK) return s;
    if (!on_device(ctx, q, 16) || !on_device(ctx, out, 16) || (lse != nullptr && !on_device(ctx, lse, 4)))
        return KVS_EINVAL;
    if (selected != nullptr && (top < 1 || !on_device(ctx, selected, 4))) return KVS_EINVAL;
    DeviceScope scope(ctx->device);
    if (!scope.ok) return KVS_ECUDA;
    const kvshare_config& cf = ctx->cfg;
    const bool f32 = cf.dtype == KVS_F32;
    const int D = cf.head_dim, B = pages->batch, Hq = cf.num_q_heads, Hkv = cf.num_kv_heads;
    const int rows = decode_paged_box_rows(f32, D, pages->page_size);
    CUtensorMap tmK, tmV;
    if (!pool_map(ctx, pages, pages->k, rows, &tmK) || !pool_map(ctx, pages, pages->v, rows, &tmV)) return KVS_ECUDA;
    for (int l : ctx->order) {
        if (l < l0 || l >= l1) continue;
        const kvshare_layer& e = ctx->map[l];
        const bool mix = e.kind == KVS_SRC_MIX;
        const size_t lbh = static_cast<size_t>(l) * B * Hq;
        PagedDecodeArgs a;
        std::memset(&a, 0, sizeof(a));
        a.q = static_cast<const char*>(q) + lbh * D * elem_size(cf.dtype);
        a.out = out + lbh * D;
        a.lse = lse ? lse + lbh : nullptr;
        a.table = pages->block_table;
        a.lens = pages->lengths;
        a.sel = selected ? selected + static_cast<size_t>(l) * B * Hkv * top : nullptr;
        a.w = ctx->w_dev + static_cast<size_t>(l) * Hkv;
        a.src0 = e.src0;
        a.src1 = mix ? e.src1 : e.src0;
        a.B = B;
        a.Hq = Hq;
        a.Hkv = Hkv;
        a.g = Hq / Hkv;
        a.num_pages = pages->num_pages;
        a.max_blocks = pages->max_blocks;
        a.page_shift = page_shift(pages->page_size);
        a.top = top;
        a.scale_log2 = ctx->scale * 1.4426950408889634f;
        a.ws = ctx->pg_ws;
        a.counters = ctx->pg_counters;
        a.err = ctx->err;
        a.wait_limit = ctx->wait_limit;
        a.ctas = ctx->sms;
        a.stall_limit = ctx->stall_next ? ctx->stall_limit : 0;
        ctx->stall_next = 0;
        const cudaStream_t st = static_cast<cudaStream_t>(stream);
        const cudaError_t err = f32 ? launch_decode_paged_f32(D, mix, tmK, tmV, a, st)
                                    : launch_decode_paged_bf16(D, mix, tmK, tmV, a, st);
        if (err != cudaSuccess) return KVS_ECUDA;
        ++ctx->launches;
    }
    return KVS_OK;
}

kvshare_status kvshare_select_pages(kvshare_t ctx, const kvshare_pages* pages, const void* q, int* selected, int top,
                                    int first, int last, int l0, int l1, void* stream) {
    if (ctx == nullptr || !ctx->map_set) return KVS_EINVAL;
    kvshare_status s = check_pool(ctx, pages);
    if (s == KVS_OK) s = check_tables(ctx, pages);
    if (s == KVS_OK) s = check_layers(ctx, pages, l0, l1);
    if (s != KVS_OK) return s;
    if (first < 0 || last < 1 || top < 1 || first > top || last > top - first) return KVS_EINVAL;
    if (pages->max_blocks > SELECT_MAX_BLOCKS) return KVS_EUNSUPPORTED;
    if (!on_device(ctx, q, 16) || !on_device(ctx, selected, 4) || !on_device(ctx, pages->bound_codes, 16) ||
        !on_device(ctx, pages->bound_scale, 4))
        return KVS_EINVAL;
    DeviceScope scope(ctx->device);
    if (!scope.ok) return KVS_ECUDA;
    const kvshare_config& cf = ctx->cfg;
    const int B = pages->batch, Hq = cf.num_q_heads, Hkv = cf.num_kv_heads;
    for (int l : ctx->order) {
        if (l < l0 || l >= l1) continue;
        const kvshare_layer& e = ctx->map[l];
        PagedSelectArgs a;
        std::memset(&a, 0, sizeof(a));
        a.q = static_cast<const char*>(q) + static_cast<size_t>(l) * B * Hq * cf.head_dim * elem_size(cf.dtype);
        a.codes = pages->bound_codes;
        a.scales = pages->bound_scale;
        a.table = pages->block_table;
        a.lens = pages->lengths;
        a.w = ctx->w_dev + static_cast<size_t>(l) * Hkv;
        a.sel = selected + static_cast<size_t>(l) * B * Hkv * top;
        a.mix = e.kind == KVS_SRC_MIX;
        a.src0 = e.src0;
        a.src1 = a.mix ? e.src1 : e.src0;
        a.B = B;
        a.Hq = Hq;
        a.Hkv = Hkv;
        a.g = Hq / Hkv;
        a.d = cf.head_dim;
        a.num_pages = pages->num_pages;
        a.max_blocks = pages->max_blocks;
        a.page_shift = page_shift(pages->page_size);
        a.top = top;
        a.first = first;
        a.last = last;
        a.f32 = cf.dtype == KVS_F32;
        a.err = ctx->err;
        if (launch_select_pages(a, ctx->sms, static_cast<cudaStream_t>(stream)) != cudaSuccess) return KVS_ECUDA;
        ++ctx->launches;
    }
    return KVS_OK;
}

}  // extern "C"
