// Attention of many new tokens over a paged compressed KV cache, on the tensor cores with
// accumulators in tensor memory (tcgen05).
//
// A block holds TILES tiles of 128 query rows (tokens of a sequence times the heads that
// share a key head) and walks over its keys, 64 at a time. The keys' codes become fp16
// operands once per block of keys and serve all of the block's rows.
//
//   dequant warps   codes -> registers (a block of keys ahead) -> fp16 K and V in shared
//                   memory; a thread takes a key or a value and works out its steps once
//   matrix warps    two a tile: S_t = Q_t K^T (both from shared memory), O_t += P_t V (P_t from tensor
//                   memory, over S_t's columns; V as an MN-major operand, so K and V
//                   have the same layout and neither is transposed)
//   softmax warps   one row a thread: maximum, exp2, sum, P_t
//
// S_t has two buffers, so that the products of one block of keys run while the
// exponentials of the one before are taken, and the next S is there when they are done.
// That is why blocks have 64 keys: at head_dim 128 two tiles take 2 (2 * 64 + 128) = 512
// columns, all there are. With 128 keys and one buffer each step waited for the other
// (wait, S, softmax, P V in turn): 5100 cycles per 128 keys and 256 rows. One warp that
// issues all products: 1745 us for 2000 tokens over 8 and 16 thousand slots at 32 heads of
// 128, one a tile 1169, one for each kind and tile 1018, with the stages' release off its
// path to the next scores 966 us, scores of any magnitude 980 to 990 captured and replayed
// (0.88 PFLOP/s, 53% of the measured fp16 rate) and 1000 to 1070 a call, by the device's
// clock. What bounds
// it now is the softmax warps: 2080 cycles a block of 64 keys, of which the exponential
// unit is busy 1024. Tried and slower: the two tiles' exponentials in turns (1040), a
// quarter of them as polynomials (1125), two threads a row.
//
// One tile: two blocks a multiprocessor leave 96 registers, and all forms spill 56 to 88 bytes (142
// to 214 loaded); of two tiles only 8 bits with groups of 64 at 128 dims does (12).
// Probabilities are rounded to fp16, as operands of the value product: o's error against 64
// bits is 1.2 to 1.4 times that of fp32 probabilities, below one fp16 step; what the
// rounding leaves would take a second product and as many conversions again in the softmax
// warps, which bound the kernel.
//
// The running maximum m only moves when a score passes it by kSlack: until then the weights grow
// instead of O being rescaled (fp16 holds them with the same relative error). The final
// quotient does not depend on m.
#include <type_traits>

#include "paged_attn.cuh"
#include "tc.cuh"

namespace flexq {
namespace {

constexpr int kTileMin = 4;        // blocks of keys that a part has at least

constexpr int NK = 64;             // keys of a block

template <int D, int TILES>
struct TileShape {
    static constexpr int ST = TILES == 1 && D == 128 ? 2 : 4;      // stages of K and of V: two blocks an SM at 1 tile
    static constexpr int QB = 128 * D * 2, BLOCK = NK * D * 2;     // bytes of a tile's queries, of a block of keys
    static constexpr int SMEM = TILES * QB + 2 * ST * BLOCK + 1024;
    static constexpr int COLS = TILES == 1 ? 256 : 512;            // tensor memory: TILES * (2 * NK + D) columns
    static constexpr int SOFT = TILES * 4;                         // softmax warps, then 4 dequant warps, two matrix warps a tile
    static constexpr int THREADS = SOFT * 32 + 128 + 64 * TILES;
};

__device__ __forceinline__ void sts16(uint32_t at, const uint32_t (&a)[4]) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]) : "memory");
}

// Two fp32 values in one register pair: one instruction for both.
__device__ __forceinline__ uint64_t f32x2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void f32x2_get(uint64_t x, float& a, float& b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x));
}
__device__ __forceinline__ uint64_t f32x2_fma(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t f32x2_add(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t f32x2_scale(uint64_t a, float f) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(f32x2(f, f)));
    return r;
}

// 16-byte piece c (8 dims) of row r of an operand: blocks of 64 dims (ROWS rows each), rows
// of 128 bytes, the hardware's 128-byte swizzle. 8 threads that write one piece of consecutive rows hit
// 8 different bank groups.
template <int ROWS>
__device__ __forceinline__ uint32_t piece_at(uint32_t base, int r, int c) {
    return base + (c >> 3) * (ROWS * 128) + r * 128 + ((c & 7) ^ (r & 7)) * 16;
}

// Exponents are score * log2 e + shift_of(m), one fused multiply-add for each score, so that
// weights are 2^lift_of(m) times exp(score - m): kLift but for what rounding the shift left. A
// maximum of 2^23 or more would leave factors that overflow: such rows' scores have m
// subtracted in tensor memory first.
__device__ __forceinline__ bool is_big(float m) { return fabsf(m) >= 8388608.f && m != -FLT_MAX; }
// (No maximum yet: every score so far is -infinity, and its exponent is to stay that.)
__device__ __forceinline__ float shift_of(float m) {
    return m == -FLT_MAX || is_big(m) ? kLift : kLift - __fmul_rn(m, kLog2e);
}
__device__ __forceinline__ float lift_of(float m) {
    return m == -FLT_MAX || is_big(m) ? kLift : fmaf(m, kLog2e, shift_of(m));
}

template <int D, int BITS, int GS, int TILES>
__global__ void __launch_bounds__(TileShape<D, TILES>::THREADS, TILES == 1 ? 2 : 1)
    paged_tile_kernel(AttnArgs A, uint64_t wait_ns, const volatile int* gate) {
    using T = TileShape<D, TILES>;
    constexpr int ST = T::ST, KB = D * BITS / 8, NG = D / GS, R = TILES * 128, NX = KB / 16, SOFT = T::SOFT;
    extern __shared__ unsigned char raw[];
    __shared__ __align__(8) uint64_t bars[4 * ST + 1 + 6 * TILES];
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag, wild_flag;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const PagedView& c = A.c;
    pdl_wait();
    const int head = blockIdx.x % A.plan.heads;
    const Unit u = find_unit<R, 128, kTileMin, 2, true>(c, A.rows, A.plan, blockIdx.x / A.plan.heads);
    if (warp == 0) record_split<R, 128>(A, u, blockIdx.x / A.plan.heads, head);
    if (!u.live) return;
    const int share = A.plan.share;
    const int blocks = (u.ctx + 127) / 128;
    const int key0 = min(blocks, u.part * u.per) * 128;
    const int key1 = min(u.ctx, min(blocks, (u.part + 1) * u.per) * 128);
    const int nc = (key1 - key0 + NK - 1) / NK;               // blocks of cached keys
    const int row_end = u.n * share, row0 = u.tile * R;
    // fresh tokens that any of the rows sees, by the last part
    const int last = A.k_new != nullptr && u.part == u.parts - 1 ? (min(row_end, row0 + R) - 1) / share + 1 : 0;
    const int nb = nc + (last + NK - 1) / NK;
    const int tiles = min(TILES, (row_end - row0 + 127) / 128);

    const uint32_t bar0 = tc::smem_u32(bars);
    const uint32_t k_full = bar0, k_empty = k_full + 8 * ST, v_full = k_empty + 8 * ST, v_empty = v_full + 8 * ST,
                   q_full = v_empty + 8 * ST, s_full = q_full + 8, p_full = s_full + 16 * TILES, o_done = p_full + 16 * TILES;
    const uint32_t sq = (tc::smem_u32(raw) + 1023u) & ~1023u, sk = sq + TILES * T::QB, sv = sk + ST * T::BLOCK;
    volatile int* abort = &abort_flag;
    int* const status = c.status;
    if (tid == 0) {
        for (int i = 0; i < ST; ++i) {
            tc::bar_init(k_full + 8 * i, 2);          // one arrival a warp
            // S_j has read its keys: the softmax warps know first, the score warps with (P V)_j, which is
            // soon enough with 4 stages and takes nothing from the softmax
            tc::bar_init(k_empty + 8 * i, ST > 2 ? tiles : 4 * tiles);
            tc::bar_init(v_full + 8 * i, 2);
            tc::bar_init(v_empty + 8 * i, tiles);       // from the score warps, which see (P V)_j
        }
        tc::bar_init(q_full, 4 * tiles);
        for (int t = 0; t < TILES; ++t) {
            // one for each S buffer: softmax may be a block ahead of the products, and they of it
            for (int i = 0; i < 2; ++i) {
                tc::bar_init(s_full + 16 * t + 8 * i, 1);
                tc::bar_init(p_full + 16 * t + 8 * i, 4);
                tc::bar_init(o_done + 16 * t + 8 * i, 1);
            }
        }
        tc::bar_fence_init();
        abort_flag = 0;
        wild_flag = 0;
    }
    if (warp == SOFT + 4) {
        tc::tmem_alloc(tc::smem_u32(&tmem_slot), T::COLS);
        tc::tmem_relinquish();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    // Dependents may start from here on, not earlier: a GEMM allocates all tensor memory of a
    // multiprocessor before it waits for this kernel, and a block that had signalled without
    // having its own would wait for that GEMM's end, which waits for the block's.
    pdl_trigger();
    const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_slot, 0);

    // a warp's threads wait and arrive as one: an abort leaves no part of it behind
    auto wait = [&](uint32_t bar, uint32_t parity) {
        return __all_sync(0xffffffffu, tc::bar_wait(bar, parity, abort, status, wait_ns)) != 0;
    };
    auto arrive = [&](uint32_t bar) {
        __syncwarp();
        if (lane == 0) tc::bar_arrive(bar);
    };

    if (warp < SOFT) {
        // ---- softmax: one row a thread
        const int tile = warp >> 2, r = tid & 127, row = row0 + tile * 128 + r;
        const bool live = row < row_end;
        const int token = live ? token_of(A.plan, row) : 0, h = head * share + (live ? row - token * share : 0);
        const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;
        const uint32_t ts = tmem + tile * 128 + lanes, to = tmem + TILES * 128 + tile * D + lanes;
        bool ok = tile < tiles;
        // the running maximum; the score from which it moves; what the fused exponent adds
        float m = -FLT_MAX, limit = -FLT_MAX, shift = kLift;
        uint64_t l = 0;                                          // two partial sums
        if (ok) {
            const uint4* qr = reinterpret_cast<const uint4*>(A.q + static_cast<int64_t>(u.first + token) * A.q_stride + h * D);
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
                uint32_t a[4];
                key_pairs_fresh<BITS>(a, live ? __ldg(qr + i) : make_uint4(0, 0, 0, 0));
                sts16(piece_at<128>(sq + tile * T::QB, r, i), a);
            }
            tc::fence_proxy_async_smem();
            arrive(q_full);
            for (int j = 0; j < nb; ++j) {
                if (!(ok = wait(s_full + 16 * tile + 8 * (j & 1), (j >> 1) & 1))) break;
                if (ST <= 2 && j + ST < nb) arrive(k_empty + 8 * (j % ST));
                tc::fence_after_sync();
                // keys of the block that this row sees: the first `lim`
                const int lim = j < nc ? key1 - key0 - j * NK : token + 1 - (j - nc) * NK;
                const uint32_t tj = ts + (j & 1) * NK;
                uint32_t x[2][32];
                tc::tmem_ld32(tj, x[0]);
                tc::tmem_ld32(tj + 32, x[1]);
                tc::tmem_wait_ld(x[0]);
                tc::tmem_wait_ld(x[1]);
                auto block = [&](auto whole_c) {
                    constexpr bool WHOLE = decltype(whole_c)::value;
                    auto score = [&](int i) {
                        const float v = __uint_as_float(x[i >> 5][i & 31]);
                        return WHOLE || i < lim ? v : -INFINITY;
                    };
                    float tops[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int i = 0; i < NK; i += 2)
                        tops[(i >> 1) & 3] = fmaxf(fmaxf(tops[(i >> 1) & 3], score(i)), score(i + 1));
                    const float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
                    if (__any_sync(0xffffffffu, top > limit)) {
                        const bool moves = top > m + kSlack;    // a row's result depends on no other row
                        const float was = m, lift = lift_of(m);
                        m = moves ? top : m;
                        const float f = moves ? exp2_fast(fmaf(was - m, kLog2e, lift_of(m) - lift)) : 1.f;
                        l = f32x2_scale(l, f);
                        limit = is_big(m) ? -INFINITY : m + kSlack;
                        shift = shift_of(m);
                        if (j > 0 && __any_sync(0xffffffffu, moves)) {
                            if (!(ok = wait(o_done + 16 * tile + 8 * ((j - 1) & 1), ((j - 1) >> 1) & 1))) return;
                            tc::fence_after_sync();
#pragma unroll 1
                            for (int i = 0; i < D; i += 16) {
                                uint32_t y[16];
                                tc::tmem_ld16(to + i, y);
#pragma unroll
                                for (int k = 0; k < 16; ++k) y[k] = __float_as_uint(__uint_as_float(y[k]) * f);
                                tc::tmem_st16(to + i, y);
                            }
                        }
                        if (__any_sync(0xffffffffu, is_big(m))) {
                            // S becomes S - m
#pragma unroll 1
                            for (int i = 0; i < NK; i += 16) {
                                uint32_t y[16];
                                tc::tmem_ld16(tj + i, y);
#pragma unroll
                                for (int k = 0; k < 16; ++k)
                                    if (is_big(m)) y[k] = __float_as_uint(__uint_as_float(y[k]) - m);
                                tc::tmem_st16(tj + i, y);
                            }
                            tc::tmem_wait_st();
                            tc::tmem_ld32(tj, x[0]);
                            tc::tmem_ld32(tj + 32, x[1]);
                            tc::tmem_wait_ld(x[0]);
                            tc::tmem_wait_ld(x[1]);
                        }
                    }
                    const uint64_t scale2 = f32x2(kLog2e, kLog2e), shift2 = f32x2(shift, shift);
                    uint64_t sums[2] = {l, 0};
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        uint32_t p[16];
#pragma unroll
                        for (int i = 0; i < 32; i += 2) {
                            float y0, y1;
                            f32x2_get(f32x2_fma(f32x2(score(half * 32 + i), score(half * 32 + i + 1)), scale2, shift2), y0, y1);
                            const float p0 = exp2_fast(y0), p1 = exp2_fast(y1);
                            sums[(i >> 1) & 1] = f32x2_add(sums[(i >> 1) & 1], f32x2(p0, p1));
                            const __half2 hp = __floats2half2_rn(p0, p1);
                            p[i >> 1] = *reinterpret_cast<const uint32_t*>(&hp);
                        }
                        tc::tmem_st16(tj + half * 16, p);
                    }
                    l = f32x2_add(sums[0], sums[1]);
                };
                if (__all_sync(0xffffffffu, lim >= NK))
                    block(std::true_type{});
                else
                    block(std::false_type{});
                if (!ok) break;
                tc::tmem_wait_st();
                tc::fence_before_sync();
                arrive(p_full + 16 * tile + 8 * (j & 1));
            }
            // (both: the values' products are whole)
            if (ok && nb > 1) ok = wait(o_done + 16 * tile + 8 * (nb & 1), ((nb - 2) >> 1) & 1);
            if (ok && nb > 0) ok = wait(o_done + 16 * tile + 8 * ((nb - 1) & 1), ((nb - 1) >> 1) & 1);
            tc::fence_after_sync();
        }
        float l0, sum;
        f32x2_get(l, l0, sum);
        sum += l0;
        if (ok) {
            // partial results are relative to m itself
            const float inv = sum == 0.f ? 0.f : 1.f / sum, even = exp2_fast(-lift_of(m));
            const int64_t at = static_cast<int64_t>(u.first + token) * (A.plan.heads * share) + h;
            float* part = A.parts + ((static_cast<int64_t>(u.slot) * A.plan.heads + head) * R + tile * 128 + r) * (D + 4);
            const bool wild = wild_flag != 0;
#pragma unroll 1
            for (int i = 0; i < D; i += 32) {
                uint32_t y[32];
                __syncwarp();                                    // rows that are not there have gone ahead
                if (nb > 0) {
                    tc::tmem_ld32(to + i, y);
                    tc::tmem_wait_ld(y);
                } else {
#pragma unroll
                    for (int k = 0; k < 32; ++k) y[k] = 0u;
                }
                if (!live) continue;
                float v[32];                                     // in the order of the dims
#pragma unroll
                for (int k = 0; k < 32; ++k) {
                    const int e = k & 7;
                    v[BITS == 4 ? (k & ~7) + (e >> 1) + (e & 1) * 4 : k] = __uint_as_float(y[k]);
                }
                if (wild) {
                    // infinities and NaN that the products left out, for the rows that see them:
                    // whatever their weight, which is positive, the sum is what they make it
                    for (int j = 0; j <= token && j < last; ++j) {
                        const __half* vr = A.v_new + static_cast<int64_t>(u.first + j) * A.kv_stride + head * D + i;
#pragma unroll
                        for (int k = 0; k < 32; ++k) {
                            const float z = __half2float(vr[k]);
                            if (!isfinite(z)) v[k] += z;
                        }
                    }
                }
                if (u.parts == 1) {
                    uint32_t w[16];
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        const __half2 hp = __floats2half2_rn(v[2 * k] * inv, v[2 * k + 1] * inv);
                        w[k] = *reinterpret_cast<const uint32_t*>(&hp);
                    }
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        *reinterpret_cast<uint4*>(A.o + at * D + i + 8 * k) = make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
                } else if (u.slot < A.slots) {
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        *reinterpret_cast<float4*>(part + i + 4 * k) = make_float4(v[4 * k] * even, v[4 * k + 1] * even, v[4 * k + 2] * even, v[4 * k + 3] * even);
                }
            }
            if (live) {
                if (u.parts > 1) {
                    if (u.slot < A.slots) *reinterpret_cast<float2*>(part + D) = make_float2(m, sum * even);
                } else {
                    put_stats(A, at, m, sum, lift_of(m));
                }
            }
        }
    } else if (warp < SOFT + 4) {
        // ---- codes to operands: two warps take the keys, two the values, one key a thread
        const int key = tid & (NK - 1);
        const bool second = warp >= SOFT + 2;
        const uint8_t* codes = second ? c.vc : c.kc;
        const uint32_t* metas = second ? c.vm : c.km;
        const uint32_t dst = second ? sv : sk, full = second ? v_full : k_full, empty = second ? v_empty : k_empty;
        // the table's entry, the codes and their conversion: each a block of keys after the other
        const int32_t* const table_row = c.table + static_cast<int64_t>(u.b) * c.max_pages;
        auto find_page = [&](int j) {
            const int k = key0 + j * NK + key;
            return page_entry(c, table_row, k, k < key1);
        };
        auto find_row = [&](int page, int j) { return entry_row(c, page, head, key0 + j * NK + key); };
        auto load = [&](uint4 (&x)[NX], uint32_t (&meta)[NG], int row) {
            const uint4* src = reinterpret_cast<const uint4*>(codes + static_cast<int64_t>(row < 0 ? 0 : row) * KB);
#pragma unroll
            for (int i = 0; i < NX; ++i) x[i] = row < 0 ? make_uint4(0, 0, 0, 0) : __ldg(src + i);
#pragma unroll
            for (int i = 0; i < NG; ++i) meta[i] = row < 0 ? 0u : __ldg(metas + static_cast<int64_t>(row) * NG + i);
        };
        // absent keys have minimum and step 0: their values are 0
        auto convert = [&](const uint4 (&x)[NX], const uint32_t (&meta)[NG], uint32_t at) {
            uint32_t step[NG], mn[NG];
#pragma unroll
            for (int i = 0; i < NG; ++i) {
                step[i] = dup16(step16_of(meta[i]));
                mn[i] = dup_lo(meta[i]);
            }
            auto word = [&](int w) {
                const uint4& v = x[w / 4];
                return w % 4 == 0 ? v.x : w % 4 == 1 ? v.y : w % 4 == 2 ? v.z : v.w;
            };
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
                uint32_t a[4];
                if (BITS == 4)
                    key_pairs<BITS>(a, word(i), 0u, step[i * 8 / GS], mn[i * 8 / GS]);
                else
                    key_pairs<BITS>(a, word(2 * i % (NX * 4)), word((2 * i + 1) % (NX * 4)), step[i * 8 / GS], mn[i * 8 / GS]);
                sts16(piece_at<NK>(at, key, i), a);
            }
        };
        bool ok = true;
        auto slot_free = [&](int j) {
            return j < ST || wait(empty + 8 * (j % ST), ((j / ST) - 1) & 1);
        };
        auto publish = [&](int j) {
            tc::fence_proxy_async_smem();
            arrive(full + 8 * (j % ST));
        };
        // (flex_set_gemm_gate: the values are held back, so that the scores are on their way meanwhile)
        if (second && gate != nullptr) ok = __all_sync(0xffffffffu, tc::gate_wait(gate, abort, status, wait_ns));
        uint4 x[2][NX];
        uint32_t meta[2][NG];
        const int page0 = find_page(0);
        int page = find_page(1);
        load(x[0], meta[0], find_row(page0, 0));
        auto step = [&](int j, auto now_c) {
            constexpr int NOW = decltype(now_c)::value;
            load(x[1 - NOW], meta[1 - NOW], find_row(page, j + 1));
            page = find_page(j + 2);
            if (!(ok = slot_free(j))) return;
            convert(x[NOW], meta[NOW], dst + (j % ST) * T::BLOCK);
            publish(j);
        };
        for (int j = 0; j < nc && ok; j += 2) {
            step(j, std::integral_constant<int, 0>{});
            if (j + 1 < nc && ok) step(j + 1, std::integral_constant<int, 1>{});
        }
        for (int j = nc; j < nb && ok; ++j) {
            const int tok = (j - nc) * NK + key;
            const bool there = tok < last;
            const uint4* src = reinterpret_cast<const uint4*>((second ? A.v_new : A.k_new) +
                                                              static_cast<int64_t>(u.first + (there ? tok : 0)) * A.kv_stride + head * D);
            if (!(ok = slot_free(j))) break;
#pragma unroll 4
            for (int i = 0; i < D / 8; ++i) {
                uint4 v = there ? __ldg(src + i) : make_uint4(0, 0, 0, 0);
                // a hidden key's probability is 0, and 0 * infinity would be NaN
                if (second && any_wild(v)) {
                    v = without_wild(v);
                    wild_flag = 1;
                }
                uint32_t a[4];
                key_pairs_fresh<BITS>(a, v);
                sts16(piece_at<NK>(dst + (j % ST) * T::BLOCK, key, i), a);
            }
            publish(j);
        }
    } else if ((warp - SOFT - 4) / 2 < tiles) {
        // ---- the matrix products, two warps a tile: the scores S_j, which take the columns of
        // P_(j-2), and P_j V. Waiting for a barrier and committing cost 100 to 300 cycles each while
        // the products load the shared memory; with a warp for each kind they hide behind products.
        const int t = (warp - SOFT - 4) / 2;
        const bool value = (warp - SOFT - 4) & 1;
        const uint32_t leader = lane == 0, td = tmem + t * 128;
        bool ok = true;
        int issued = 0;                                         // blocks of keys committed; buffer j & 1 has the j-th
        auto wait1 = [&](uint32_t bar, uint32_t parity) {
            ok = ok && wait(bar, parity);
            return ok;
        };
        if (!value) {
            constexpr uint32_t idesc = tc::idesc_f16_f32(128, NK);
            // descriptors hold addresses in units of 16 bytes: offsets are added
            const uint64_t a = tc::desc_k_sw128(sq + t * T::QB), dk = tc::desc_k_sw128(sk);
            ok = nb == 0 || wait(q_full, 0);
            for (int j = 0; j < nb && ok; ++j) {
                const int s = j % ST, h = j & 1;
                if (!wait1(k_full + 8 * s, (j / ST) & 1)) break;
                if (j > 1 && !wait1(o_done + 16 * t + 8 * h, ((j - 2) >> 1) & 1)) break;
                tc::fence_after_sync();
                const uint64_t b = dk + s * (T::BLOCK >> 4);
#pragma unroll
                for (int k = 0; k < D / 16; ++k)                // 16 dims a step: 32 bytes of a swizzled row
                    tc::mma_f16_if(leader, td + h * NK, a + (((k >> 2) * 16384 + (k & 3) * 32) >> 4),
                                   b + (((k >> 2) * (NK * 128) + (k & 3) * 32) >> 4), idesc, k > 0);
                tc::mma_commit_if(leader, s_full + 16 * t + 8 * h);
                issued = j + 1;
                if (j > 1 && j - 2 + ST < nb) {                 // (P V)_(j-2) has read its values
                    arrive(v_empty + 8 * ((j - 2) % ST));
                    if (ST > 2) arrive(k_empty + 8 * ((j - 2) % ST));
                }
            }
        } else {
            constexpr uint32_t idesc = tc::idesc_f16_f32(128, D) | tc::kIdescBMnMajor;
            const uint64_t dv = tc::desc_mn_sw128(sv, NK * 128);
            for (int j = 0; j < nb && ok; ++j) {
                const int s = j % ST, h = j & 1;
                if (!wait1(v_full + 8 * s, (j / ST) & 1) || !wait1(p_full + 16 * t + 8 * h, (j >> 1) & 1)) break;
                tc::fence_after_sync();
                const uint64_t b = dv + s * (T::BLOCK >> 4);
#pragma unroll
                for (int k = 0; k < NK / 16; ++k)               // 16 keys a step
                    tc::mma_f16_ts_if(leader, tmem + TILES * 128 + t * D, td + h * NK + k * 8, b + k * (2048 >> 4), idesc,
                                      j > 0 || k > 0);
                tc::mma_commit_if(leader, o_done + 16 * t + 8 * h);
                issued = j + 1;
            }
        }
        // What was issued (each time with a commit) reads shared memory, writes tensor memory and
        // arrives at barriers: it ends before the block does, whoever has given up. (This warp may
        // have issued its last products and be content while the softmax warps no longer wait
        // for them.) Not with the caller's limit, which may be the one that ran out.
        volatile int never = 0;
        const uint32_t done = (value ? o_done : s_full) + 16 * t;
        for (int j = max(0, issued - 2); j < issued; ++j)
            tc::bar_wait(done + 8 * (j & 1), (j >> 1) & 1, &never, status, tc::kWaitLimitNs);
        __syncwarp();
    }
    tc::fence_before_sync();
    __syncthreads();
    if (warp == SOFT + 4) {
        __syncwarp();
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, T::COLS);
    }
}

template <int D, int BITS, int GS, int TILES>
void launch_one(const AttnArgs& a, int64_t units, cudaStream_t st) {
    using T = TileShape<D, TILES>;
    set_smem_once(paged_tile_kernel<D, BITS, GS, TILES>, T::SMEM);
    launch_k(paged_tile_kernel<D, BITS, GS, TILES>, dim3(static_cast<unsigned>(units * a.plan.heads)), dim3(T::THREADS),
             T::SMEM, st, true, a, pipeline_wait_ns(), reinterpret_cast<const volatile int*>(gemm_gate()));
    launch_join<D, 128 * TILES, 128, kTileMin>(a, st);
}

}  // namespace

// Rows of a sequence and key head -> rows of a block. One tile and two blocks an SM, or two
// tiles that share the operands. us with 128 / 256 rows a block for the shapes named at
// attn_plan and for 64 sequences of 700 slots at 8 heads of 64: 64 rows 33 / 32, 164 / 171,
// 91 / 88, 50 / 60; 129 rows 53 / 43, 365 / 253, 164 / 99, 99 / 86.
int paged_tile_rows(int rows) { return rows <= 128 ? 128 : 256; }

// Blocks that the device holds at once.
int paged_tile_target(int row_tile) { return sm_count() * (row_tile == 128 ? 2 : 1); }

void launch_paged_tile(const AttnArgs& a, int head_dim, int bits, int group, int row_tile, int64_t units, cudaStream_t st) {
#define TILE(D_, B_, G_) row_tile == 128 ? launch_one<D_, B_, G_, 1>(a, units, st) : launch_one<D_, B_, G_, 2>(a, units, st)
    if (head_dim == 64) {
        if (bits == 4 && group == 32) TILE(64, 4, 32); else if (bits == 4) TILE(64, 4, 64);
        else if (group == 32) TILE(64, 8, 32); else TILE(64, 8, 64);
    } else {
        if (bits == 4 && group == 32) TILE(128, 4, 32); else if (bits == 4) TILE(128, 4, 64);
        else if (group == 32) TILE(128, 8, 32); else TILE(128, 8, 64);
    }
#undef TILE
}

}  // namespace flexq
