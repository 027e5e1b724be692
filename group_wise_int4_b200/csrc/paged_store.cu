// Store and load of a paged compressed KV cache.
//
// store: q = the codec's quantiser (quant.cuh) of the new rows, into the slots behind
// ctx_len; load: the codec's value of a run of slots, into rows. Both are a stream: every
// value is read once and written once, so HBM bounds them. A thread owns 8 values (16
// bytes of fp16, 4 or 8 bytes of codes); a block's threads lie along a token's row (heads,
// then dims), so rows are read and written in whole lines and each head's slot is one
// 32- to 128-byte piece. TOKENS tokens a thread keep that many loads in flight.
#include "paged.cuh"

namespace flexq {
namespace {

constexpr int PS_THREADS = 256;

template <int BITS, int GS, int TOKENS>
__global__ void __launch_bounds__(PS_THREADS) paged_store_kernel(PagedView c, RowsOf rows, const __half* __restrict__ k_new,
                                                                 const __half* __restrict__ v_new, int64_t row_stride,
                                                                 const int32_t* __restrict__ pos0, int dim) {
    constexpr int L = GS / 8;                       // lanes of a group
    pdl_wait();
    pdl_trigger();
    const int b = blockIdx.z;
    int first;
    const int n = rows_of(rows, b, first, c.status);
    const int t0 = blockIdx.x * TOKENS;
    if (t0 >= n) return;
    const int vecs = c.heads * dim / 8;             // vectors of one row
    const int col = blockIdx.y * PS_THREADS + threadIdx.x;
    const bool live = col < 2 * vecs;               // keys, then values
    const int which = live && col >= vecs;
    const int e = live ? (col - which * vecs) * 8 : 0;
    const int head = e / dim, d = e % dim;
    const __half* src = (which ? v_new : k_new) + e;
    uint4 v[TOKENS];
#pragma unroll
    for (int i = 0; i < TOKENS; ++i) {
        v[i] = make_uint4(0, 0, 0, 0);
        if (live && t0 + i < n) v[i] = *reinterpret_cast<const uint4*>(src + static_cast<int64_t>(first + t0 + i) * row_stride);
    }
    const int ctx = slots_of(c, b), cap = paged_capacity(c);
    const int start = pos0 ? __ldg(pos0 + b) : ctx;
    const int kb = dim * BITS / 8, ng = dim / GS;
#pragma unroll
    for (int i = 0; i < TOKENS; ++i) {
        __half2 hmn, hmx;
        float mn, mx;
        minmax8(v[i], hmn, hmx);
        group_minmax<L>(hmn, hmx, mn, mx);
        const __half s16 = group_scale16<BITS>(mn, mx);
        const float s = __half2float(s16);
        if (!live || t0 + i >= n) continue;
        const int slot = ctx + t0 + i;
        if (slot >= cap) {
            paged_bad(c);
            continue;
        }
        const int page = page_of(c, b, slot);
        if (page < 0) continue;
        const int64_t row = slot_row(c, page, head, slot);
        uint8_t* codes = (which ? c.vc : c.kc) + row * kb + d * BITS / 8;
        if (BITS == 4)
            *reinterpret_cast<uint32_t*>(codes) = quant8_4bit(v[i], mn, s);
        else
            *reinterpret_cast<uint2*>(codes) = quant8_8bit(v[i], mn, s);
        if (d % GS == 0) (which ? c.vm : c.km)[row * ng + d / GS] = pack_half2_bits(stored_min16(mn), s16);
        if (c.slot_pos && !which && d == 0) c.slot_pos[row] = start + t0 + i;
    }
}

template <int BITS, int GS, int TOKENS>
__global__ void __launch_bounds__(PS_THREADS) paged_load_kernel(PagedView c, RowsOf rows, __half* __restrict__ k_out,
                                                                __half* __restrict__ v_out, int64_t row_stride,
                                                                const int32_t* __restrict__ from, int dim) {
    pdl_wait();
    pdl_trigger();
    const int b = blockIdx.z;
    int first;
    const int n = rows_of(rows, b, first, c.status);
    const int t0 = blockIdx.x * TOKENS;
    if (t0 >= n) return;
    const int vecs = c.heads * dim / 8;
    const int col = blockIdx.y * PS_THREADS + threadIdx.x;
    if (col >= 2 * vecs) return;
    const int which = col >= vecs;
    const int e = (col - which * vecs) * 8;
    const int head = e / dim, d = e % dim;
    const int start = from ? __ldg(from + b) : 0, cap = paged_capacity(c);
    const int kb = dim * BITS / 8, ng = dim / GS;
    uint2 q[TOKENS];
    uint32_t meta[TOKENS];
    int64_t row[TOKENS];
#pragma unroll
    for (int i = 0; i < TOKENS; ++i) {
        row[i] = -1;
        if (t0 + i >= n) continue;
        const int64_t slot = static_cast<int64_t>(start) + t0 + i;
        if (slot < 0 || slot >= cap) {
            paged_bad(c);
            continue;
        }
        const int page = page_of(c, b, static_cast<int>(slot));
        if (page >= 0) row[i] = slot_row(c, page, head, static_cast<int>(slot));
    }
#pragma unroll
    for (int i = 0; i < TOKENS; ++i) {
        if (row[i] < 0) continue;
        const uint8_t* codes = (which ? c.vc : c.kc) + row[i] * kb + d * BITS / 8;
        q[i] = BITS == 4 ? make_uint2(*reinterpret_cast<const uint32_t*>(codes), 0u) : *reinterpret_cast<const uint2*>(codes);
        meta[i] = (which ? c.vm : c.km)[row[i] * ng + d / GS];
    }
#pragma unroll
    for (int i = 0; i < TOKENS; ++i) {
        if (row[i] < 0) continue;
        const float mn = h2f_lo(meta[i]), step = group_step(__ushort_as_half(static_cast<unsigned short>(meta[i] >> 16)));
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            uint32_t a, z;
            if (BITS == 4) {
                a = (q[i].x >> (8 * k)) & 15u;
                z = (q[i].x >> (8 * k + 4)) & 15u;
            } else {
                const uint32_t x = k < 2 ? q[i].x : q[i].y;
                a = (x >> (16 * (k & 1))) & 255u;
                z = (x >> (16 * (k & 1) + 8)) & 255u;
            }
            w[k] = dequant_two(a, z, step, mn);     // a constant group: step 0 and codes 0 give min
        }
        __half* dst = (which ? v_out : k_out) + static_cast<int64_t>(first + t0 + i) * row_stride + e;
        *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

}  // namespace

int validate_paged(const flex_paged_cache* c, bool codes) {
    FLEX_REQUIRE(c != nullptr, FLEX_ERR_INVALID_ARG);
    FLEX_REQUIRE(c->page_table && c->ctx_len, FLEX_ERR_INVALID_ARG);
    FLEX_REQUIRE(!codes || (c->k_codes && c->k_meta && c->v_codes && c->v_meta), FLEX_ERR_INVALID_ARG);
    FLEX_REQUIRE(c->num_pages > 0 && c->max_pages > 0 && c->batch > 0 && c->n_kv_heads > 0, FLEX_ERR_INVALID_ARG);
    FLEX_REQUIRE(c->head_dim == 64 || c->head_dim == 128, FLEX_ERR_UNSUPPORTED);
    FLEX_REQUIRE(c->page_size >= 16 && c->page_size <= 1024 && (c->page_size & (c->page_size - 1)) == 0,
                 FLEX_ERR_UNSUPPORTED);
    FLEX_REQUIRE(c->cfg.symmetric == 0, FLEX_ERR_UNSUPPORTED);
    FLEX_REQUIRE(c->cfg.num_bits == 4 || c->cfg.num_bits == 8, FLEX_ERR_UNSUPPORTED);
    FLEX_REQUIRE(c->cfg.group_size == 32 || c->cfg.group_size == 64, FLEX_ERR_UNSUPPORTED);
    FLEX_REQUIRE(c->cfg.group_dim == 3 || c->cfg.group_dim == -1, FLEX_ERR_UNSUPPORTED);
    // batch and heads are grid dimensions; slots and their rows are ints
    FLEX_REQUIRE(c->batch <= 65535 && c->n_kv_heads <= 65535, FLEX_ERR_UNSUPPORTED);
    FLEX_REQUIRE(static_cast<int64_t>(c->max_pages) * c->page_size <= (1LL << 30), FLEX_ERR_SHAPE);
    FLEX_REQUIRE(static_cast<int64_t>(c->num_pages) * c->page_size <= ((1LL << 31) - 1) / c->n_kv_heads, FLEX_ERR_SHAPE);
    FLEX_REQUIRE(aligned16(c->k_codes) && aligned16(c->k_meta) && aligned16(c->v_codes) && aligned16(c->v_meta) &&
                     aligned16(c->weight) && aligned16(c->slot_pos),
                 FLEX_ERR_ALIGN);
    FLEX_REQUIRE(((reinterpret_cast<uintptr_t>(c->page_table) | reinterpret_cast<uintptr_t>(c->ctx_len)) & 3u) == 0,
                 FLEX_ERR_ALIGN);
    return FLEX_OK;
}

PagedView paged_view(const flex_paged_cache* c) {
    PagedView v{};
    v.kc = static_cast<uint8_t*>(c->k_codes);
    v.vc = static_cast<uint8_t*>(c->v_codes);
    v.km = static_cast<uint32_t*>(c->k_meta);
    v.vm = static_cast<uint32_t*>(c->v_meta);
    v.weight = c->weight;
    v.slot_pos = c->slot_pos;
    v.table = c->page_table;
    v.ctx_len = c->ctx_len;
    v.num_pages = c->num_pages;
    while ((1 << v.shift) < c->page_size) ++v.shift;
    v.max_pages = c->max_pages;
    v.heads = c->n_kv_heads;
    v.status = status_word();
    return v;
}

int validate_rows(const flex_paged_cache* c, const int32_t* cu, int32_t batch, int32_t total, int32_t most) {
    FLEX_REQUIRE(batch > 0 && batch <= c->batch, FLEX_ERR_INVALID_ARG);
    FLEX_REQUIRE(total >= 0 && most >= 0, FLEX_ERR_INVALID_ARG);
    FLEX_REQUIRE(most <= (1 << 24), FLEX_ERR_UNSUPPORTED);
    FLEX_REQUIRE(cu != nullptr || static_cast<int64_t>(batch) * most == total, FLEX_ERR_INVALID_ARG);
    FLEX_REQUIRE((reinterpret_cast<uintptr_t>(cu) & 3u) == 0, FLEX_ERR_ALIGN);
    return FLEX_OK;
}

namespace {

int validate_kv_rows(const flex_paged_cache* c, const void* k, const void* v, int64_t row_stride) {
    FLEX_REQUIRE(k && v, FLEX_ERR_INVALID_ARG);
    FLEX_REQUIRE(row_stride >= static_cast<int64_t>(c->n_kv_heads) * c->head_dim, FLEX_ERR_INVALID_ARG);
    FLEX_REQUIRE(aligned16(k) && aligned16(v) && row_stride % 8 == 0, FLEX_ERR_ALIGN);
    return FLEX_OK;
}

inline dim3 paged_copy_grid(const flex_paged_cache* c, int batch, int most, int tokens) {
    const int64_t vecs = 2LL * c->n_kv_heads * c->head_dim / 8;
    return dim3((most + tokens - 1) / tokens, static_cast<unsigned>((vecs + PS_THREADS - 1) / PS_THREADS), batch);
}

}  // namespace
}  // namespace flexq

using namespace flexq;

// One token a thread where there is one (a decode step), four otherwise.
#define PAGED_COPY(KERNEL, ...)                                                                                   \
    do {                                                                                                          \
        const int B = cache->cfg.num_bits, G = cache->cfg.group_size;                                             \
        const cudaStream_t st = as_stream(stream);                                                                \
        if (most == 1) {                                                                                          \
            const dim3 grid = paged_copy_grid(cache, batch, most, 1);                                             \
            if (B == 4 && G == 32) launch_k(KERNEL<4, 32, 1>, grid, dim3(PS_THREADS), 0, st, true, __VA_ARGS__);  \
            else if (B == 4) launch_k(KERNEL<4, 64, 1>, grid, dim3(PS_THREADS), 0, st, true, __VA_ARGS__);        \
            else if (G == 32) launch_k(KERNEL<8, 32, 1>, grid, dim3(PS_THREADS), 0, st, true, __VA_ARGS__);       \
            else launch_k(KERNEL<8, 64, 1>, grid, dim3(PS_THREADS), 0, st, true, __VA_ARGS__);                    \
        } else {                                                                                                  \
            const dim3 grid = paged_copy_grid(cache, batch, most, 4);                                             \
            if (B == 4 && G == 32) launch_k(KERNEL<4, 32, 4>, grid, dim3(PS_THREADS), 0, st, true, __VA_ARGS__);  \
            else if (B == 4) launch_k(KERNEL<4, 64, 4>, grid, dim3(PS_THREADS), 0, st, true, __VA_ARGS__);        \
            else if (G == 32) launch_k(KERNEL<8, 32, 4>, grid, dim3(PS_THREADS), 0, st, true, __VA_ARGS__);       \
            else launch_k(KERNEL<8, 64, 4>, grid, dim3(PS_THREADS), 0, st, true, __VA_ARGS__);                    \
        }                                                                                                         \
        return launch_status();                                                                                   \
    } while (0)

extern "C" int flex_paged_store_kv(const flex_paged_cache* cache, const void* k_new, const void* v_new, int64_t row_stride,
                                   const int32_t* cu_new, int32_t batch, int32_t total, int32_t most, const int32_t* pos0,
                                   void* stream) {
    int rc = validate_paged(cache, true);
    if (rc == FLEX_OK) rc = validate_rows(cache, cu_new, batch, total, most);
    if (rc == FLEX_OK) rc = validate_kv_rows(cache, k_new, v_new, row_stride);
    if (rc != FLEX_OK) return rc;
    FLEX_REQUIRE((reinterpret_cast<uintptr_t>(pos0) & 3u) == 0, FLEX_ERR_ALIGN);
    if (most == 0 || total == 0) return FLEX_OK;
    const PagedView view = paged_view(cache);
    PAGED_COPY(paged_store_kernel, view, (RowsOf{cu_new, most, total}), static_cast<const __half*>(k_new),
               static_cast<const __half*>(v_new), row_stride, pos0, cache->head_dim);
}

extern "C" int flex_paged_load_kv(const flex_paged_cache* cache, void* k_out, void* v_out, int64_t row_stride,
                                  const int32_t* cu_rows, int32_t batch, int32_t total, int32_t most, const int32_t* start,
                                  void* stream) {
    int rc = validate_paged(cache, true);
    if (rc == FLEX_OK) rc = validate_rows(cache, cu_rows, batch, total, most);
    if (rc == FLEX_OK) rc = validate_kv_rows(cache, k_out, v_out, row_stride);
    if (rc != FLEX_OK) return rc;
    FLEX_REQUIRE((reinterpret_cast<uintptr_t>(start) & 3u) == 0, FLEX_ERR_ALIGN);
    if (most == 0 || total == 0) return FLEX_OK;
    const PagedView view = paged_view(cache);
    PAGED_COPY(paged_load_kernel, view, (RowsOf{cu_rows, most, total}), static_cast<__half*>(k_out),
               static_cast<__half*>(v_out), row_stride, start, cache->head_dim);
}
