// Store and load of a paged compressed KV cache.
//
// store: q = the codec's quantiser (quant.cuh) of the new rows, into the slots behind
// ctx_len; load: the codec's value of a run of slots, into rows. Both are a stream: every
// value is read once and written once, so HBM bounds them as long as the instructions are
// few: a thread owns 16 values (32 bytes of fp16, 8 or 16 bytes of codes), so that a
// group's extremes, scale and step are worked out by few lanes, and TOKENS tokens, whose
// rows it requests first and whose slots lie in two pages at most. A block's threads lie
// along a token's row (heads, then dims): rows are read and written in whole lines, each
// head's slot in one piece of 32 to 128 bytes. Prompts of 301 to 1024 tokens at 96 heads of
// 128, 4 bits: 35 us each way, 69% of the measured copy bandwidth (8 values a thread: 47).
#include "paged.cuh"

namespace flexq {
namespace {

constexpr int PS_THREADS = 256;

// The pages of TOKENS slots from `slot` on: the first one's and the last one's.
template <int TOKENS>
struct SlotRows {
    int entry0, entry1, base;
    __device__ __forceinline__ SlotRows(const PagedView& c, int b, int64_t slot, int count) {
        const int32_t* row = c.table + static_cast<int64_t>(b) * c.max_pages;
        const int cap = paged_capacity(c);
        const int64_t end = slot + count - 1;
        base = slot < 0 || slot >= cap ? INT32_MIN : static_cast<int>(slot);
        entry0 = page_entry(c, row, base, base != INT32_MIN);
        entry1 = TOKENS == 1 ? entry0 : page_entry(c, row, static_cast<int>(end), end >= 0 && end < cap);
        if (base == INT32_MIN || end >= cap) paged_bad(c);
    }
    // row of the i-th slot and this head; -1 where it lies outside the table or its page outside the pool
    __device__ __forceinline__ int row(const PagedView& c, int head, int i) const {
        if (base == INT32_MIN || base + i >= paged_capacity(c)) return -1;
        const int slot = base + i;
        return entry_row(c, (slot >> c.shift) == (base >> c.shift) ? entry0 : entry1, head, slot);
    }
};

// Which tokens a block has. search == 0: sequence blockIdx.z, tokens from blockIdx.x * TOKENS on.
// Otherwise `search` sequences of very unequal lengths have their pieces one after the other
// along blockIdx.x, and every warp finds its block's by counting (one long prompt among single tokens
// would leave nearly all blocks of a rectangle empty).
struct Span {
    int b, first, n, t0;
};
template <int TOKENS>
__device__ __forceinline__ Span find_span(const RowsOf& rows, int search, int* status) {
    Span s{static_cast<int>(blockIdx.z), 0, 0, static_cast<int>(blockIdx.x) * TOKENS};
    if (search == 0) {
        s.n = rows_of(rows, s.b, s.first, status);
        return s;
    }
    const int lane = threadIdx.x & 31;
    int left = blockIdx.x;                          // pieces still to pass
    for (int b0 = 0; b0 < search; b0 += 32) {
        int first = 0, n = 0;
        if (b0 + lane < search) n = rows_of(rows, b0 + lane, first, status);
        const int pieces = (n + TOKENS - 1) / TOKENS;           // at most 2^24
        const int sum = __reduce_add_sync(0xffffffffu, pieces);
        if (left >= sum) {
            left -= sum;
            continue;
        }
        int x = pieces;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        const int l = __ffs(__ballot_sync(0xffffffffu, left < x)) - 1;
        s.b = b0 + l;
        s.first = __shfl_sync(0xffffffffu, first, l);
        s.n = __shfl_sync(0xffffffffu, n, l);
        s.t0 = (left - __shfl_sync(0xffffffffu, x - pieces, l)) * TOKENS;
        return s;
    }
    return s;                                       // n = 0: nothing
}

template <int D, int BITS, int GS, int TOKENS>
__global__ void __launch_bounds__(PS_THREADS) paged_store_kernel(PagedView c, RowsOf rows, const __half* __restrict__ k_new,
                                                                 const __half* __restrict__ v_new, int64_t row_stride,
                                                                 const int32_t* __restrict__ pos0, int search) {
    constexpr int L = GS / 16, V = D / 16, KB = D * BITS / 8, NG = D / GS;      // lanes of a group, threads of a head
    pdl_wait();
    pdl_trigger();
    const Span span = find_span<TOKENS>(rows, search, c.status);
    const int b = span.b, first = span.first, n = span.n, t0 = span.t0;
    if (t0 >= n) return;
    const int vecs = c.heads * V;                   // threads of one row's keys
    const int col = blockIdx.y * PS_THREADS + threadIdx.x;
    const bool live = col < 2 * vecs;               // keys, then values
    const int which = live && col >= vecs, e = live ? col - which * vecs : 0, head = e / V, d = e % V * 16;
    const __half* src = (which ? v_new : k_new) + static_cast<int64_t>(first + t0) * row_stride + e * 16;
    const int count = min(TOKENS, n - t0);
    uint4 v[TOKENS][2];
#pragma unroll
    for (int i = 0; i < TOKENS; ++i) {
        v[i][0] = v[i][1] = make_uint4(0, 0, 0, 0);
        if (live && i < count) {
            const uint4* p = reinterpret_cast<const uint4*>(src + i * row_stride);
            v[i][0] = ld_stream_v4(p);
            v[i][1] = ld_stream_v4(p + 1);
        }
    }
    const int ctx = slots_of(c, b);
    if (ctx < 0) return;
    const int start = pos0 ? __ldg(pos0 + b) : ctx;
    const SlotRows<TOKENS> slots(c, b, static_cast<int64_t>(ctx) + t0, count);
    uint8_t* const codes = (which ? c.vc : c.kc) + d * BITS / 8;
    uint32_t* const meta = (which ? c.vm : c.km) + d / GS;
#pragma unroll
    for (int i = 0; i < TOKENS; ++i) {
        __half2 hmn, hmx, hmn1, hmx1;
        float mn, mx;
        minmax8(v[i][0], hmn, hmx);
        minmax8(v[i][1], hmn1, hmx1);
        group_minmax<L>(__hmin2(hmn, hmn1), __hmax2(hmx, hmx1), mn, mx);
        const __half s16 = group_scale16<BITS>(mn, mx);
        const float s = __half2float(s16);
        if (!live || i >= count) continue;
        const int row = slots.row(c, head, i);
        if (row < 0) continue;
        uint8_t* const to = codes + static_cast<int64_t>(row) * KB;
        if (BITS == 4) {
            *reinterpret_cast<uint2*>(to) = make_uint2(quant8_4bit(v[i][0], mn, s), quant8_4bit(v[i][1], mn, s));
        } else {
            const uint2 a = quant8_8bit(v[i][0], mn, s), z = quant8_8bit(v[i][1], mn, s);
            *reinterpret_cast<uint4*>(to) = make_uint4(a.x, a.y, z.x, z.y);
        }
        if (d % GS == 0) meta[static_cast<int64_t>(row) * NG] = pack_half2_bits(stored_min16(mn), s16);
        if (c.slot_pos && !which && d == 0) c.slot_pos[row] = start + t0 + i;
    }
}

template <int D, int BITS, int GS, int TOKENS>
__global__ void __launch_bounds__(PS_THREADS) paged_load_kernel(PagedView c, RowsOf rows, __half* __restrict__ k_out,
                                                                __half* __restrict__ v_out, int64_t row_stride,
                                                                const int32_t* __restrict__ from, int search) {
    constexpr int V = D / 16, KB = D * BITS / 8, NG = D / GS;
    pdl_wait();
    pdl_trigger();
    const Span span = find_span<TOKENS>(rows, search, c.status);
    const int b = span.b, first = span.first, n = span.n, t0 = span.t0;
    if (t0 >= n) return;
    const int vecs = c.heads * V;
    const int col = blockIdx.y * PS_THREADS + threadIdx.x;
    if (col >= 2 * vecs) return;
    const int which = col >= vecs, e = col - which * vecs, head = e / V, d = e % V * 16;
    const int count = min(TOKENS, n - t0);
    const SlotRows<TOKENS> slots(c, b, static_cast<int64_t>(from ? __ldg(from + b) : 0) + t0, count);
    const uint8_t* const codes = (which ? c.vc : c.kc) + d * BITS / 8;
    const uint32_t* const metas = (which ? c.vm : c.km) + d / GS;
    uint4 q[TOKENS];
    uint32_t meta[TOKENS];
    bool ok[TOKENS];
#pragma unroll
    for (int i = 0; i < TOKENS; ++i) {
        const int row = i < count ? slots.row(c, head, i) : -1;
        ok[i] = row >= 0;
        if (row < 0) continue;
        const uint8_t* at = codes + static_cast<int64_t>(row) * KB;
        if (BITS == 4) {
            const uint2 x = *reinterpret_cast<const uint2*>(at);
            q[i] = make_uint4(x.x, x.y, 0u, 0u);
        } else {
            q[i] = *reinterpret_cast<const uint4*>(at);
        }
        meta[i] = metas[static_cast<int64_t>(row) * NG];
    }
    __half* const dst = (which ? v_out : k_out) + static_cast<int64_t>(first + t0) * row_stride + e * 16;
#pragma unroll
    for (int i = 0; i < TOKENS; ++i) {
        if (!ok[i]) continue;
        // a constant group: step 0 and codes 0 give min
        const float mn = h2f_lo(meta[i]), step = group_step(__ushort_as_half(static_cast<unsigned short>(meta[i] >> 16)));
        uint32_t w[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {                  // values 2k and 2k + 1
            uint32_t a, z;
            if (BITS == 4) {
                const uint32_t x = (k < 4 ? q[i].x : q[i].y) >> (8 * (k & 3));
                a = x & 15u;
                z = (x >> 4) & 15u;
            } else {
                const uint32_t x = (k < 2 ? q[i].x : k < 4 ? q[i].y : k < 6 ? q[i].z : q[i].w) >> (16 * (k & 1));
                a = x & 255u;
                z = (x >> 8) & 255u;
            }
            w[k] = dequant_two(a, z, step, mn);
        }
        uint4* to = reinterpret_cast<uint4*>(dst + i * row_stride);
        to[0] = make_uint4(w[0], w[1], w[2], w[3]);
        to[1] = make_uint4(w[4], w[5], w[6], w[7]);
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

// A rectangle of the longest sequence's pieces times the batch, or (search) the pieces alone: at
// most total / tokens + batch. us for the rectangle / the
// pieces, storing at 96 heads of 128: 1024 tokens and 143 single ones 241 / 21, four of 300 to
// 1024 tokens 33.9 / 35.0, 20 of 200 47.2 / 51.3.
struct CopyGrid {
    dim3 grid;
    int search;
};
inline CopyGrid paged_copy_grid(const flex_paged_cache* c, int batch, int total, int most, int tokens) {
    const int64_t vecs = 2LL * c->n_kv_heads * c->head_dim / 16;
    const unsigned y = static_cast<unsigned>((vecs + PS_THREADS - 1) / PS_THREADS);
    const int64_t wide = (most + tokens - 1) / tokens, pieces = total / tokens + batch;
    if (wide * batch > 4 * pieces) return CopyGrid{dim3(static_cast<unsigned>(pieces), y, 1), batch};
    return CopyGrid{dim3(static_cast<unsigned>(wide), y, batch), 0};
}

}  // namespace
}  // namespace flexq

using namespace flexq;

// One token a thread where there is one (a decode step), four otherwise.
#define PAGED_COPY(KERNEL, ...)                                                                                     \
    do {                                                                                                            \
        const int D = cache->head_dim, B = cache->cfg.num_bits, G = cache->cfg.group_size;                          \
        const cudaStream_t st = as_stream(stream);                                                                  \
        const CopyGrid g = paged_copy_grid(cache, batch, total, most, most == 1 ? 1 : 4);                           \
        const dim3 block(PS_THREADS);                                                                               \
        if (D == 64) {                                                                                              \
            if (B == 4 && G == 32) PAGED_RUN(KERNEL, 64, 4, 32, __VA_ARGS__);                                       \
            else if (B == 4) PAGED_RUN(KERNEL, 64, 4, 64, __VA_ARGS__);                                             \
            else if (G == 32) PAGED_RUN(KERNEL, 64, 8, 32, __VA_ARGS__);                                            \
            else PAGED_RUN(KERNEL, 64, 8, 64, __VA_ARGS__);                                                         \
        } else {                                                                                                    \
            if (B == 4 && G == 32) PAGED_RUN(KERNEL, 128, 4, 32, __VA_ARGS__);                                      \
            else if (B == 4) PAGED_RUN(KERNEL, 128, 4, 64, __VA_ARGS__);                                            \
            else if (G == 32) PAGED_RUN(KERNEL, 128, 8, 32, __VA_ARGS__);                                           \
            else PAGED_RUN(KERNEL, 128, 8, 64, __VA_ARGS__);                                                        \
        }                                                                                                           \
        return launch_status();                                                                                     \
    } while (0)
#define PAGED_RUN(KERNEL, D_, B_, G_, ...)                                            \
    do {                                                                              \
        if (most == 1) launch_k(KERNEL<D_, B_, G_, 1>, g.grid, block, 0, st, true, __VA_ARGS__, g.search); \
        else launch_k(KERNEL<D_, B_, G_, 4>, g.grid, block, 0, st, true, __VA_ARGS__, g.search);  \
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
               static_cast<const __half*>(v_new), row_stride, pos0);
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
               static_cast<__half*>(v_out), row_stride, start);
}
