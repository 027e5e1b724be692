// Paged compressed KV cache: what its kernels share (store, load, attention, eviction).
//
// Layout: page p holds page_size slots of every key head, [page][kv head][slot][...], so a
// head's slots of one page are one contiguous run. A slot's row index
// (page * heads + head) * page_size + slot fits an int (checked on the host); every byte
// offset is formed in 64 bits.
//
// What the device finds wrong (a page id outside the pool, lengths outside the table,
// row offsets that do not fit the call) is reported through the status word as
// FLEX_ERR_INVALID_ARG and the access is skipped: nothing is read or written through it.
#pragma once

#include "quant.cuh"

namespace flexq {

struct PagedView {
    uint8_t *kc, *vc;
    uint32_t *km, *vm;
    float* weight;
    int32_t* slot_pos;
    const int32_t* table;
    const int32_t* ctx_len;
    int num_pages, shift, max_pages, heads;
    int* status;
};

// The new rows of a ragged batch: rows [cu[b], cu[b+1]) belong to sequence b; cu == nullptr:
// `most` rows each.
struct RowsOf {
    const int32_t* cu;
    int most, total;
};

int validate_paged(const flex_paged_cache* c, bool codes);
PagedView paged_view(const flex_paged_cache* c);
int validate_rows(const flex_paged_cache* c, const int32_t* cu, int32_t batch, int32_t total, int32_t most);

__device__ __forceinline__ void paged_bad(const PagedView& c) { set_status(c.status, FLEX_ERR_INVALID_ARG); }

// First row and number of rows of sequence b; none, reported, where they do not fit.
__device__ __forceinline__ int rows_of(const RowsOf& r, int b, int& first, int* status) {
    if (r.cu == nullptr) {
        first = b * r.most;
        return r.most;
    }
    const int lo = __ldg(r.cu + b), hi = __ldg(r.cu + b + 1);
    first = lo;
    if (lo < 0 || hi < lo || hi > r.total || hi - lo > r.most) {
        set_status(status, FLEX_ERR_INVALID_ARG);
        first = 0;
        return 0;
    }
    return hi - lo;
}

__device__ __forceinline__ int paged_capacity(const PagedView& c) { return c.max_pages << c.shift; }

// Slots that sequence b holds; -1, reported, where ctx_len is no length of the table: nothing of
// such a sequence is read or written, since what it holds is not known.
__device__ __forceinline__ int slots_of(const PagedView& c, int b) {
    const int n = __ldg(c.ctx_len + b);
    if (static_cast<unsigned>(n) > static_cast<unsigned>(paged_capacity(c))) {
        paged_bad(c);
        return -1;
    }
    return n;
}

// Page of slot s of sequence b (s within the table); -1, reported, where the id is not a
// page of the pool.
__device__ __forceinline__ int page_of(const PagedView& c, int b, int s) {
    const int p = __ldg(c.table + static_cast<int64_t>(b) * c.max_pages + (s >> c.shift));
    if (static_cast<unsigned>(p) >= static_cast<unsigned>(c.num_pages)) {
        paged_bad(c);
        return -1;
    }
    return p;
}

// The same in two steps, so that the table's entry is on its way while other work is done:
// the entry itself (kNoPage where `there` is false), then its check and the row of slot s.
constexpr int kNoPage = INT32_MIN;
__device__ __forceinline__ int page_entry(const PagedView& c, const int32_t* table_row, int s, bool there) {
    return there ? __ldg(table_row + (s >> c.shift)) : kNoPage;
}
__device__ __forceinline__ int entry_row(const PagedView& c, int entry, int head, int s) {
    if (static_cast<unsigned>(entry) >= static_cast<unsigned>(c.num_pages)) {
        if (entry != kNoPage) paged_bad(c);
        return -1;
    }
    return ((entry * c.heads + head) << c.shift) + (s & ((1 << c.shift) - 1));
}

// Row index of slot s of a page (page >= 0) and head.
__device__ __forceinline__ int slot_row(const PagedView& c, int page, int head, int s) {
    return ((page * c.heads + head) << c.shift) + (s & ((1 << c.shift) - 1));
}

// ---- the attention's form of a code: fp16(c * fp16(1/scale) + min), one fused
// multiply-add, as the products with compressed weights take it. Two rounded steps (the
// codec's value) cost four more instructions a value and change it by at most one unit of
// the last fp16 place; with the fused form the values are exact fp16 operands of the
// matrix instructions, so scores carry only fp32 summation error.
//
// fp16(rcp.approx(s)) is the correctly rounded fp16(1/s): with s = S 2^e (S an 11-bit
// integer) and a rounding boundary M 2^f (M an odd integer of at most 12 bits), S M is
// never a power of two, so 1/s is at least 2^-23 (relative) from every boundary, and the
// approximation's error of one unit in the last fp32 place does not reach it: equality of
// the roundings is checked over every fp16 scale by the tests.
__device__ __forceinline__ __half step16_of(uint32_t meta) {
    const float s = h2f_hi(meta);
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
    return s > 0.0f ? __float2half_rn(r) : __ushort_as_half(0);
}

__device__ __forceinline__ uint32_t h2_sub(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t h2_fma(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t r;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
    return r;
}
// Codes in the low nibbles of bits 0-3 and 16-19: with the exponent of 1024 behind them they
// are 1024 + c; in bits 4-7 and 20-23, with that of 64, 64 + c. Both differences are exact.
__device__ __forceinline__ uint32_t and_or(uint32_t x, uint32_t mask, uint32_t bits) {
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(x), "r"(mask), "r"(bits));
    return r;
}
__device__ __forceinline__ uint32_t codes_lo(uint32_t x) { return h2_sub(and_or(x, 0x000F000Fu, 0x64006400u), 0x64006400u); }
__device__ __forceinline__ uint32_t codes_hi(uint32_t x) { return h2_sub(and_or(x, 0x00F000F0u, 0x54005400u), 0x54005400u); }
__device__ __forceinline__ uint32_t byte_perm(uint32_t a, uint32_t b, uint32_t sel) {
    uint32_t r;
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(sel));
    return r;
}
// Bytes (lo, hi) of x, each 0..255, as two fp16 values.
__device__ __forceinline__ uint32_t codes_b01(uint32_t x) {
    return h2_sub(byte_perm(x, 0x64646464u, 0x4140u), 0x64006400u);
}
__device__ __forceinline__ uint32_t codes_b23(uint32_t x) {
    return h2_sub(byte_perm(x, 0x64646464u, 0x4342u), 0x64006400u);
}
__device__ __forceinline__ uint32_t dup16(__half h) {
    const uint32_t u = __half_as_ushort(h);
    return u | (u << 16);
}
__device__ __forceinline__ uint32_t dup_lo(uint32_t x) { return byte_perm(x, x, 0x1010u); }
__device__ __forceinline__ uint32_t dup_hi(uint32_t x) { return byte_perm(x, x, 0x3232u); }

__device__ __forceinline__ float exp2_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

}  // namespace flexq
