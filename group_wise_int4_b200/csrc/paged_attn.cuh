// What the attention kernels over a paged cache share: operands from codes, the split of
// the work and its plan.
#pragma once

#include <float.h>

#include "paged.cuh"

namespace flexq {

__device__ __forceinline__ void cp16(uint32_t s, const void* g, bool ok) {
    const int n = ok ? 16 : 0;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(s), "l"(g), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// D (16 x 8, fp32) += A (16 x 16) B (16 x 8), fp16 operands
__device__ __forceinline__ void mma168(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t mat_trans(uint32_t x) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}
__device__ __forceinline__ uint32_t half2_of(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t smem_addr(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }

// ---- operands -------------------------------------------------------------------------
//
// Scores are S^T = K Q^T: keys are the rows of the 16 x 8 products, query rows the columns.
// Lane (g, t) of a quad row takes the dims [t D/4, (t+1) D/4) of its keys, so a key's codes
// are one contiguous piece per lane; the product does not care which dims a k-step holds
// as long as both operands agree. At 4 bits the nibble pairs of a word are (d, d+4),
// (d+1, d+5), ..., at 8 bits the byte pairs are neighbours; the query is laid out to match.

// Query operand of row g of an 8-row tile: D/16 k-steps of two registers.
template <int D, int BITS>
__device__ __forceinline__ void load_query(uint32_t (&bq)[D / 16][2], const __half* row, int t, bool ok) {
#pragma unroll
    for (int u = 0; u < D / 32; ++u) {                 // 8 dims: two k-steps
        uint4 x = make_uint4(0, 0, 0, 0);
        if (ok) x = __ldg(reinterpret_cast<const uint4*>(row + t * (D / 4)) + u);
        if (BITS == 4) {
            bq[2 * u][0] = byte_perm(x.x, x.z, 0x5410u);
            bq[2 * u][1] = byte_perm(x.x, x.z, 0x7632u);
            bq[2 * u + 1][0] = byte_perm(x.y, x.w, 0x5410u);
            bq[2 * u + 1][1] = byte_perm(x.y, x.w, 0x7632u);
        } else {
            bq[2 * u][0] = x.x;
            bq[2 * u][1] = x.y;
            bq[2 * u + 1][0] = x.z;
            bq[2 * u + 1][1] = x.w;
        }
    }
}

// Key operand of two k-steps (8 dims) from 8 codes: at 4 bits one word, at 8 bits two.
template <int BITS>
__device__ __forceinline__ void key_pairs(uint32_t (&a)[4], uint32_t w0, uint32_t w1, uint32_t step, uint32_t mn) {
    if (BITS == 4) {
        const uint32_t y = w0 >> 8;
        a[0] = h2_fma(codes_lo(w0), step, mn);
        a[1] = h2_fma(codes_hi(w0), step, mn);
        a[2] = h2_fma(codes_lo(y), step, mn);
        a[3] = h2_fma(codes_hi(y), step, mn);
    } else {
        a[0] = h2_fma(codes_b01(w0), step, mn);
        a[1] = h2_fma(codes_b23(w0), step, mn);
        a[2] = h2_fma(codes_b01(w1), step, mn);
        a[3] = h2_fma(codes_b23(w1), step, mn);
    }
}
// The same from 8 fresh fp16 values.
template <int BITS>
__device__ __forceinline__ void key_pairs_fresh(uint32_t (&a)[4], uint4 x) {
    if (BITS == 4) {
        a[0] = byte_perm(x.x, x.z, 0x5410u);
        a[1] = byte_perm(x.x, x.z, 0x7632u);
        a[2] = byte_perm(x.y, x.w, 0x5410u);
        a[3] = byte_perm(x.y, x.w, 0x7632u);
    } else {
        a[0] = x.x;
        a[1] = x.y;
        a[2] = x.z;
        a[3] = x.w;
    }
}

// Pairs of fp16 values: does one have the largest exponent (infinity or NaN), and the same
// with those taken for 0.
__device__ __forceinline__ uint32_t wild_halves(uint32_t x) { return __vcmpeq2(x & 0x7C007C00u, 0x7C007C00u); }
__device__ __forceinline__ bool any_wild(uint4 x) {
    return (wild_halves(x.x) | wild_halves(x.y) | wild_halves(x.z) | wild_halves(x.w)) != 0u;
}
__device__ __forceinline__ uint4 without_wild(uint4 x) {
    return make_uint4(x.x & ~wild_halves(x.x), x.y & ~wild_halves(x.y), x.z & ~wild_halves(x.z), x.w & ~wild_halves(x.w));
}

// ---- work split -------------------------------------------------------------------------
//
// A unit is (sequence, tile of R query rows, part of the key length); one block per unit
// and key head. The key length of all sequences together is cut into parts of `per`
// blocks of KEYS keys, so that about `target` blocks share it whatever its distribution:
// every warp finds its block's unit by itself from ctx_len and cu (a few loads and
// shuffles), so nothing has to be planned on the host or in another launch.
//
// Bounds that the workspace relies on, with work = sum of row tiles times key blocks and
// per >= work * heads / target (target: of units times heads): tiles are at most total * share / R + batch; the parts
// beyond each tile's first at most work / per <= target / heads; and the units of tiles
// that are split (ceil(blocks / per) < 2 blocks / per, as blocks > per) fewer than
// 2 target / heads: only those have a slot for partial results.
struct RowsPlan {
    int batch, share, target, heads;
    uint32_t share_inverse;             // floor(2^32 / share) + 1 where rows * share < 2^32; else 0
};

// Row / share: with r (share_inverse * share - 2^32) <= r share < 2^32 the high product is the
// quotient. A division takes some 20 instructions, and rows are divided all the time.
__device__ __forceinline__ int token_of(const RowsPlan& p, int r) {
    if (p.share == 1) return r;
    return p.share_inverse ? static_cast<int>(__umulhi(static_cast<uint32_t>(r), p.share_inverse)) : r / p.share;
}

struct Unit {
    int b, tile, part, parts, per;      // per: key blocks in a part
    int plan_per;                       // the whole batch's, before the parts of a tile are made even
    int slot;                           // of this unit's partial result, where parts > 1
    int first, n, ctx;
    bool live;
};

// MIN: blocks of keys that a part has at least; less costs more to join than it saves.
// FULL: where the tiles alone take more than half of the target, parts are as long as FULL
// times an even share of the work: short enough to level the blocks' ends, and 1 or 2 by
// what starting and joining a part costs beside its keys. SORT: the units of a batch of up
// to 32 are in descending order of their keys, so that short blocks fill the end.
template <int R, int KEYS, int MIN, int FULL, bool SORT>
__device__ __forceinline__ Unit find_unit(const PagedView& c, const RowsOf& rows, const RowsPlan& p, int unit) {
    const int lane = threadIdx.x & 31;
    struct Seq {
        int n, ctx, first, tiles;
    };
    auto load = [&](int b) {
        Seq s{};
        if (b < p.batch) {
            s.n = rows_of(rows, b, s.first, c.status);
            s.ctx = slots_of(c, b);
            if (s.ctx < 0) s.n = s.ctx = 0;             // no rows
            s.tiles = static_cast<int>((static_cast<int64_t>(s.n) * p.share + R - 1) / R);
        }
        return s;
    };
    // work of the whole batch, in key blocks times row tiles, and the row tiles
    Seq q = load(lane);                                 // a batch of up to 32 is read once
    int64_t work = 0, all = 0;
    for (int b = lane;; b += 32) {
        const Seq s = b < 32 ? q : load(b);
        work += static_cast<int64_t>(s.tiles) * ((s.ctx + KEYS - 1) / KEYS);
        all += s.tiles;
        if (b - lane + 32 >= p.batch) break;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        work += __shfl_xor_sync(0xffffffffu, work, o);
        all += __shfl_xor_sync(0xffffffffu, all, o);
    }
    // With room for every tile's first part beside them the parts fit the target: they run at once.
    const int64_t fit = p.target - all * p.heads;
    const int64_t room = fit > p.target / 2 ? fit : (p.target + FULL - 1) / FULL;
    const int64_t even = (work * p.heads + room - 1) / room;
    Unit u{};
    u.plan_per = static_cast<int>(even < MIN ? MIN : even > (1 << 30) ? (1 << 30) : even);
    // the unit is the at-th of lane l's sequence, whose partial slots begin at `slots`
    auto found = [&](int l, int at, int b0, int parts, int slots) {
        u.b = b0 + l;
        u.n = __shfl_sync(0xffffffffu, q.n, l);
        u.ctx = __shfl_sync(0xffffffffu, q.ctx, l);
        u.first = __shfl_sync(0xffffffffu, q.first, l);
        u.parts = __shfl_sync(0xffffffffu, parts, l);
        u.per = max(1, ((u.ctx + KEYS - 1) / KEYS + u.parts - 1) / u.parts);     // even parts
        u.slot = slots + at;
        u.tile = at / u.parts;
        u.part = at % u.parts;
        u.live = true;
        return u;
    };
    int64_t before = 0, split = 0;                      // units, and units of split tiles, of the sequences passed
    for (int b0 = 0; b0 < p.batch; b0 += 32) {
        if (b0 > 0) q = load(b0 + lane);
        const int parts = max(1, ((q.ctx + KEYS - 1) / KEYS + u.plan_per - 1) / u.plan_per);
        // (more units than 2^25 of one sequence would be more than a launch has)
        const int mine = static_cast<int>(min(static_cast<int64_t>(q.tiles) * parts, static_cast<int64_t>(1 << 25)));
        const int mine2 = parts > 1 ? mine : 0;
        const int sum = __reduce_add_sync(0xffffffffu, mine), sum2 = __reduce_add_sync(0xffffffffu, mine2);
        if (unit >= before + sum) {
            before += sum;
            split += sum2;
            continue;
        }
        if (SORT && p.batch <= 32) {
            const int cost = (q.ctx + KEYS - 1) / KEYS / parts + q.n / KEYS;
            int x = 0, y = 0;                           // units of the sequences in front of b
            for (int i = 0; i < p.batch; ++i) {
                const int c2 = __shfl_sync(0xffffffffu, cost, i), m = __shfl_sync(0xffffffffu, mine, i),
                          m2 = __shfl_sync(0xffffffffu, mine2, i);
                const bool front = c2 > cost || (c2 == cost && i < lane);
                x += front ? m : 0;
                y += front ? m2 : 0;
            }
            const int l = __ffs(__ballot_sync(0xffffffffu, unit >= x && unit < x + mine)) - 1;
            return found(l, unit - __shfl_sync(0xffffffffu, x, l), b0, parts, __shfl_sync(0xffffffffu, y, l));
        }
        int x = mine, y = mine2;                        // up to and with b
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int xx = __shfl_up_sync(0xffffffffu, x, o), yy = __shfl_up_sync(0xffffffffu, y, o);
            if (lane >= o) {
                x += xx;
                y += yy;
            }
        }
        const int want = static_cast<int>(unit - before);
        const int l = __ffs(__ballot_sync(0xffffffffu, want < x)) - 1;
        const int at = want - __shfl_sync(0xffffffffu, x - mine, l);
        return found(l, at, b0, parts, static_cast<int>(split) + __shfl_sync(0xffffffffu, y - mine2, l));
    }
    return u;
}

// What a split unit tells the joining launch, at its partial slot.
struct SplitRecord {
    int b, tile, part, parts;
};

// What a launch of either attention kernel gets. Partial results: [slot][head][row of the
// tile][D + 4]: the output, then the maximum and the sum.
struct AttnArgs {
    PagedView c;
    RowsOf rows;
    RowsPlan plan;
    const __half* q;
    int64_t q_stride;
    const __half *k_new, *v_new;
    int64_t kv_stride;
    __half* o;
    float* lse;
    float2* stats;              // weights wanted: maximum and log2 of the sum of each row and head; else nullptr
    float* parts;
    float *scores, *fresh;      // one row a sequence and key head, weights wanted: its scores, by slot's row and
                                // of its own token [batch][heads]; else nullptr
    int* split_units;           // how many partial slots are in use
    SplitRecord* records;       // [slots]
    int slots;                  // of partial results
};

// Exponent (base 2) of a score's weight relative to m. The difference comes first: it is exact
// near the maximum and 0 at it, however large the scores are.
__device__ __forceinline__ float exponent_of(float score, float m) { return (score - m) * kLog2e; }
// Weights are 2^kLift times exp(score - m), and the maximum m may be passed by kSlack: up to 2^14,
// which fp16 holds, as it does in full precision what is 2^-20 of them (without the
// lift weights below 2^-14 would be subnormal, and lose bits, in long histories).
constexpr float kLift = 6.f, kSlack = 8.f * kLn2;

// A row's statistics, at [row][head]: sum = 2^left times the sum of exp(score - top).
__device__ __forceinline__ void put_stats(const AttnArgs& A, int64_t at, float top, float sum, float left = 0.f) {
    const float l = log2f(sum) - left;
    if (A.lse) A.lse[at] = sum == 0.f ? -INFINITY : fmaf(l, kLn2, top);
    if (A.stats) A.stats[at] = make_float2(top, sum == 0.f ? INFINITY : l);
}
// The probability of a score, by these statistics; 1 at most. A score that was summed again, in
// another order, is off by roundings of its magnitude (by whole units above 2^23), which would make
// "probabilities" of any size, infinity among them, and one of those would stay in the running
// weights for good. NaN stays NaN.
__device__ __forceinline__ float prob_of(float score, float2 stats) {
    const float x = fmaf(score - stats.x, kLog2e, -stats.y);
    return exp2_fast(x > 0.f ? 0.f : x);
}

// Called by one warp of every unit and head: unit 0 says how many partial slots there are, a
// split unit where it belongs.
template <int R, int KEYS>
__device__ __forceinline__ void record_split(const AttnArgs& A, const Unit& u, int unit, int head) {
    const int lane = threadIdx.x & 31;
    if (head != 0) return;
    if (unit == 0) {
        int64_t units = 0;
        for (int b = lane; b < A.plan.batch; b += 32) {
            int first;
            const int n = rows_of(A.rows, b, first, A.c.status);
            const int64_t tiles = (static_cast<int64_t>(n) * A.plan.share + R - 1) / R;
            const int parts = ((max(slots_of(A.c, b), 0) + KEYS - 1) / KEYS + u.plan_per - 1) / u.plan_per;
            if (parts > 1) units += tiles * parts;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) units += __shfl_xor_sync(0xffffffffu, units, o);
        if (lane == 0) *A.split_units = static_cast<int>(min(units, static_cast<int64_t>(A.slots)));
    }
    if (lane == 0 && u.live && u.parts > 1 && u.slot < A.slots) A.records[u.slot] = SplitRecord{u.b, u.tile, u.part, u.parts};
}

// Joins the parts of split tiles. A block goes through slots and heads; the rows of a slot's
// tile are shared out evenly over its parts' slots and over z.
template <int D, int R>
__global__ void __launch_bounds__(128) paged_join_kernel(AttnArgs A) {
    pdl_wait();
    pdl_trigger();
    const RowsPlan& plan = A.plan;
    const int items = min(*A.split_units, A.slots) * plan.heads;
    for (int item = blockIdx.x; item < items; item += gridDim.x) {
        const int head = item % plan.heads, slot = item / plan.heads;
        const SplitRecord rec = A.records[slot];
        // offsets that overlap (cu out of order) can leave a record unset: whatever it holds, nothing
        // outside the slots and the sequence's rows is touched
        if (static_cast<unsigned>(rec.b) >= static_cast<unsigned>(plan.batch) || rec.part < 0 || rec.part > slot || rec.tile < 0 ||
            rec.parts <= rec.part || rec.parts > A.slots || slot - rec.part > A.slots - rec.parts)
            continue;
        int first;
        const int row_end = rows_of(A.rows, rec.b, first, A.c.status) * plan.share;
        if (rec.tile >= (row_end + R - 1) / R) continue;
        const int row0 = rec.tile * R, rows = min(R, row_end - row0);
        const int chunks = rec.parts * gridDim.y, chunk = rec.part * gridDim.y + blockIdx.y, per = (rows + chunks - 1) / chunks;
        constexpr int L = D / 4, G = 128 / L;               // threads of a row, groups of them
        const int d = (threadIdx.x % L) * 4, group = threadIdx.x / L;
        const int64_t step = static_cast<int64_t>(plan.heads) * R * (D + 4);
        const int begin = chunk * per, end = min(rows, begin + per);
        if (begin >= end) continue;
        // enough rows: one a group; few (long sequences with many parts): the groups share a row's parts
        const bool share_row = end - begin < G;
        __shared__ float4 part_out[G][L];
        __shared__ float2 part_stat[G];
        for (int r = begin + (share_row ? 0 : group); r < end; r += share_row ? 1 : G) {
            const float* p = A.parts + ((static_cast<int64_t>(slot - rec.part) * plan.heads + head) * R + r) * (D + 4);
            float top = -FLT_MAX, sum = 0.f;
            float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
            // (not 0: an infinite value of a part with a far smaller maximum stays what it is, and what is
            // finite of it is below every last place; NaN stays NaN)
            auto factor = [](float m, float t) {
                const float f = exp2_fast(exponent_of(m, t));
                return f < FLT_MIN ? FLT_MIN : f;
            };
            auto add = [&](float2 ml, float4 x) {
                const float t = fmaxf(top, ml.x), f0 = factor(top, t), f = factor(ml.x, t);
                top = t;
                sum = fmaf(sum, f0, f * ml.y);
                a.x = fmaf(a.x, f0, f * x.x);
                a.y = fmaf(a.y, f0, f * x.y);
                a.z = fmaf(a.z, f0, f * x.z);
                a.w = fmaf(a.w, f0, f * x.w);
            };
            const int by = share_row ? G : 1;
            for (int k0 = share_row ? group : 0; k0 < rec.parts; k0 += 8 * by) {
                float2 ml[8];
                float4 x[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int k = k0 + i * by;
                    if (k >= rec.parts) break;
                    ml[i] = __ldg(reinterpret_cast<const float2*>(p + k * step + D));
                    x[i] = __ldg(reinterpret_cast<const float4*>(p + k * step + d));
                }
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (k0 + i * by < rec.parts) add(ml[i], x[i]);
            }
            if (share_row) {
                __syncthreads();                            // (the row before is read)
                part_out[group][threadIdx.x % L] = a;
                if (d == 0) part_stat[group] = make_float2(top, sum);
                __syncthreads();
                if (group != 0) continue;
#pragma unroll
                for (int i = 1; i < G; ++i) add(part_stat[i], part_out[i][threadIdx.x]);
            }
            const int tok = token_of(plan, row0 + r), h = head * plan.share + row0 + r - tok * plan.share;
            const int64_t at = static_cast<int64_t>(first + tok) * (plan.heads * plan.share) + h;
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
            *reinterpret_cast<uint2*>(A.o + at * D + d) = make_uint2(half2_of(a.x * inv, a.y * inv), half2_of(a.z * inv, a.w * inv));
            if (d == 0) put_stats(A, at, top, sum);
        }
    }
}

// A part has at least MIN blocks of keys, so a table of no more splits nothing and needs no
// joining launch.
template <int D, int R, int KEYS, int MIN>
void launch_join(const AttnArgs& a, cudaStream_t st) {
    if (static_cast<int64_t>(a.c.max_pages) << a.c.shift <= static_cast<int64_t>(MIN) * KEYS) return;
    const int64_t items = static_cast<int64_t>(a.slots) * a.plan.heads;
    const int fill = 8 * sm_count();                    // blocks of a device that is full
    launch_k(paged_join_kernel<D, R>, dim3(static_cast<unsigned>(items < fill ? items : fill), R <= 16 ? 1 : R / 64), dim3(128), 0, st,
             true, a);
}

// The tcgen05 kernel over tiles of paged_tile_rows() query rows; `units` blocks per key head.
int paged_tile_rows(int rows);
int paged_tile_target(int row_tile);
void launch_paged_tile(const AttnArgs& a, int head_dim, int bits, int group, int row_tile, int64_t units, cudaStream_t st);

}  // namespace flexq
