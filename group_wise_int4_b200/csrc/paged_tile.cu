// Attention of many new tokens over a paged compressed KV cache, on the tensor cores with
// accumulators in tensor memory (tcgen05).
//
// A block holds TILES tiles of 128 query rows (tokens of a sequence times the heads that
// share a key head) and walks over its keys, 128 at a time. The keys' codes become fp16
// operands once per block of keys and serve all of the block's rows: at 256 rows that is
// about 1.9 K warp instructions beside 2048 cycles of matrix products, so dequantising in
// the kernel costs less than writing the fp16 values to memory and reading them again.
//
//   dequant warps   codes -> registers (a block of keys ahead) -> fp16 K and V in shared
//                   memory, one key a thread: its steps and minima are worked out once
//   matrix warp     S_t = Q_t K^T (both from shared memory), O_t += P_t V (P_t from tensor
//                   memory, over S_t's columns; V as an MN-major operand, so K and V
//                   have the same layout and neither is transposed)
//   softmax warps   one row a thread: maximum, exp2, sum, P_t; with two tiles the products
//                   of one run while the exponentials of the other are taken
//
// The running maximum m only moves when a score passes it by more than 2^8 (in base 2, 8
// steps): until then the probabilities are up to 256 instead of 1, which fp16 holds with
// the same relative error, and O is not rescaled. The final quotient does not depend on m.
#include <type_traits>

#include "paged_attn.cuh"
#include "tc.cuh"

namespace flexq {
namespace {

template <int D, int TILES>
struct TileShape {
    static constexpr int ST = (TILES == 1 && D == 128) ? 1 : 2;    // stages of K and of V: two blocks an SM at 1 tile
    static constexpr int BLOCK = 128 * D * 2;                      // bytes of 128 fp16 rows
    static constexpr int SMEM = (TILES + 2 * ST) * BLOCK + 1024;
    static constexpr int COLS = TILES == 1 ? 256 : 512;            // tensor memory: TILES * (128 + D) columns
    static constexpr int THREADS = TILES * 128 + 128 + 32;
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

// 16-byte piece c (8 dims) of row r of an operand: halves of 64 dims, rows of 128 bytes,
// the hardware's 128-byte swizzle. 8 threads that write one piece of consecutive rows hit
// 8 different bank groups.
__device__ __forceinline__ uint32_t piece_at(uint32_t base, int r, int c) {
    return base + (c >> 3) * 16384 + r * 128 + ((c & 7) ^ (r & 7)) * 16;
}

template <int D, int BITS, int GS, int TILES>
__global__ void __launch_bounds__(TileShape<D, TILES>::THREADS, TILES == 1 ? 2 : 1)
    paged_tile_kernel(AttnArgs A, uint64_t wait_ns) {
    using T = TileShape<D, TILES>;
    constexpr int ST = T::ST, KB = D * BITS / 8, NG = D / GS, R = TILES * 128, NX = KB / 16;
    extern __shared__ unsigned char raw[];
    __shared__ __align__(8) uint64_t bars[4 * ST + 1 + 3 * TILES + 1];
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag, wild_flag;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const PagedView& c = A.c;
    pdl_wait();
    pdl_trigger();
    const int head = blockIdx.x % A.plan.heads;
    const Unit u = find_unit<R, 128, 4>(c, A.rows, A.plan, blockIdx.x / A.plan.heads);
    if (!u.live) return;
    const int share = A.plan.share;
    const int blocks = (u.ctx + 127) / 128;
    const int key0 = min(blocks, u.part * u.per) * 128;
    const int key1 = min(u.ctx, min(blocks, (u.part + 1) * u.per) * 128);
    const int nc = (key1 - key0 + 127) / 128;                 // blocks of cached keys
    const int row_end = u.n * share, row0 = u.tile * R;
    // fresh tokens that any of the rows sees, by the last part
    const int last = A.k_new != nullptr && u.part == u.parts - 1 ? (min(row_end, row0 + R) - 1) / share + 1 : 0;
    const int nb = nc + (last + 127) / 128;
    const int tiles = min(TILES, (row_end - row0 + 127) / 128);

    const uint32_t bar0 = tc::smem_u32(bars);
    const uint32_t k_full = bar0, k_empty = k_full + 8 * ST, v_full = k_empty + 8 * ST, v_empty = v_full + 8 * ST,
                   q_full = v_empty + 8 * ST, s_full = q_full + 8, p_full = s_full + 8 * TILES, o_done = p_full + 8 * TILES,
                   drain = o_done + 8 * TILES;
    const uint32_t sq = (tc::smem_u32(raw) + 1023u) & ~1023u, sk = sq + TILES * T::BLOCK, sv = sk + ST * T::BLOCK;
    volatile int* abort = &abort_flag;
    int* const status = c.status;
    if (tid == 0) {
        for (int i = 0; i < ST; ++i) {
            tc::bar_init(k_full + 8 * i, 128);
            tc::bar_init(k_empty + 8 * i, 1);
            tc::bar_init(v_full + 8 * i, 128);
            tc::bar_init(v_empty + 8 * i, 1);
        }
        tc::bar_init(q_full, 128 * tiles);
        for (int t = 0; t < TILES; ++t) {
            tc::bar_init(s_full + 8 * t, 1);
            tc::bar_init(p_full + 8 * t, 128);
            tc::bar_init(o_done + 8 * t, 1);
        }
        tc::bar_init(drain, 1);
        tc::bar_fence_init();
        abort_flag = 0;
        wild_flag = 0;
    }
    if (warp == TILES * 4 + 4) {
        tc::tmem_alloc(tc::smem_u32(&tmem_slot), T::COLS);
        tc::tmem_relinquish();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = tmem_slot;

    if (warp < TILES * 4) {
        // ---- softmax: one row a thread
        const int tile = warp >> 2, r = tid & 127, row = row0 + tile * 128 + r;
        const bool live = row < row_end;
        const int token = live ? row / share : 0, h = head * share + (live ? row % share : 0);
        const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;
        const uint32_t ts = tmem + tile * 128 + lanes, to = tmem + TILES * 128 + tile * D + lanes;
        bool ok = tile < tiles;
        float m = -FLT_MAX;
        uint64_t l = 0;                                          // two partial sums
        if (ok) {
            const uint4* qr = reinterpret_cast<const uint4*>(A.q + static_cast<int64_t>(u.first + token) * A.q_stride + h * D);
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
                uint32_t a[4];
                key_pairs_fresh<BITS>(a, live ? __ldg(qr + i) : make_uint4(0, 0, 0, 0));
                sts16(piece_at(sq + tile * T::BLOCK, r, i), a);
            }
            tc::fence_proxy_async_smem();
            tc::bar_arrive(q_full);
            for (int j = 0; j < nb; ++j) {
                if (!tc::bar_wait(s_full + 8 * tile, j & 1, abort, status, wait_ns)) {
                    ok = false;
                    break;
                }
                tc::fence_after_sync();
                // keys of the block that this row sees: the first `lim`
                const int lim = j < nc ? key1 - key0 - j * 128 : token + 1 - (j - nc) * 128;
                uint32_t x[2][32];
                auto load = [&](int half) {
                    tc::tmem_ld32(ts + half * 64, x[0]);
                    tc::tmem_ld32(ts + half * 64 + 32, x[1]);
                    tc::tmem_wait_ld(x[0]);
                    tc::tmem_wait_ld(x[1]);
                };
                auto block = [&](auto whole_c) {
                    constexpr bool WHOLE = decltype(whole_c)::value;
                    auto score = [&](int half, int i) {
                        const float v = __uint_as_float(x[i >> 5][i & 31]);
                        return WHOLE || half * 64 + i < lim ? v : -INFINITY;
                    };
                    float tops[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int half = 1; half >= 0; --half) {      // the first half stays in registers
                        load(half);
#pragma unroll
                        for (int i = 0; i < 64; i += 2)
                            tops[(i >> 1) & 3] = fmaxf(fmaxf(tops[(i >> 1) & 3], score(half, i)), score(half, i + 1));
                    }
                    const float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3])) * kLog2e;
                    if (__any_sync(0xffffffffu, top > m + 8.f)) {
                        // O may be changed: S_j was issued after P_(j-1) V was done
                        const bool moves = top > m + 8.f;       // a row's result depends on no other row
                        const float f = moves ? exp2_fast(m - top) : 1.f;
                        m = moves ? top : m;
                        l = f32x2_scale(l, f);
                        if (j > 0) {
#pragma unroll 1
                            for (int i = 0; i < D; i += 32) {
                                uint32_t y[32];
                                tc::tmem_ld32(to + i, y);
                                tc::tmem_wait_ld(y);
#pragma unroll
                                for (int k = 0; k < 32; ++k) y[k] = __float_as_uint(__uint_as_float(y[k]) * f);
                                tc::tmem_st32(to + i, y);
                            }
                            load(0);
                        }
                    }
                    const uint64_t scale = f32x2(kLog2e, kLog2e), shift = f32x2(-m, -m);
                    uint64_t sums[2] = {l, 0};
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        if (half == 1) load(1);
                        uint32_t p[32];
#pragma unroll
                        for (int i = 0; i < 64; i += 2) {
                            float y0, y1;
                            f32x2_get(f32x2_fma(f32x2(score(half, i), score(half, i + 1)), scale, shift), y0, y1);
                            const float p0 = exp2_fast(y0), p1 = exp2_fast(y1);
                            sums[(i >> 1) & 1] = f32x2_add(sums[(i >> 1) & 1], f32x2(p0, p1));
                            const __half2 hp = __floats2half2_rn(p0, p1);
                            p[i >> 1] = *reinterpret_cast<const uint32_t*>(&hp);
                        }
                        tc::tmem_st32(ts + half * 32, p);
                    }
                    l = f32x2_add(sums[0], sums[1]);
                };
                if (__all_sync(0xffffffffu, lim >= 128))
                    block(std::true_type{});
                else
                    block(std::false_type{});
                tc::tmem_wait_st();
                tc::fence_before_sync();
                tc::bar_arrive(p_full + 8 * tile);
            }
            if (ok && nb > 0) ok = tc::bar_wait(o_done + 8 * tile, (nb - 1) & 1, abort, status, wait_ns);
            tc::fence_after_sync();
        }
        if (tile < tiles && __all_sync(0xffffffffu, ok)) {
            float l0, sum;
            f32x2_get(l, l0, sum);
            sum += l0;
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
            const int64_t at = static_cast<int64_t>(u.first + token) * (A.plan.heads * share) + h;
            float* part = A.parts + ((static_cast<int64_t>(u.slot) * A.plan.heads + head) * R + tile * 128 + r) * (D + 4);
            const bool wild = wild_flag != 0;
#pragma unroll 1
            for (int i = 0; i < D; i += 32) {
                uint32_t y[32];
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
                        *reinterpret_cast<float4*>(part + i + 4 * k) = make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
                }
            }
            if (live) {
                if (u.parts > 1) {
                    if (u.slot < A.slots) *reinterpret_cast<float2*>(part + D) = make_float2(m, sum);
                } else if (A.lse) {
                    A.lse[at] = sum == 0.f ? -INFINITY : (m + log2f(sum)) * kLn2;
                }
            }
            if (r == 0 && tile == 0 && u.part == 0)
                A.records[static_cast<int64_t>(u.b * A.most_tiles + u.tile) * A.plan.heads + head] = TileRecord{u.parts, u.slot};
        }
    } else if (warp < TILES * 4 + 4) {
        // ---- codes to operands: one key a thread
        const int key = tid - TILES * 128;
        auto row_index = [&](int j) {
            const int k = key0 + j * 128 + key;
            if (j >= nc || k >= key1) return -1;
            const int p = page_of(c, u.b, k);
            return p < 0 ? -1 : slot_row(c, p, head, k);
        };
        auto load = [&](uint4 (&x)[NX], uint32_t (&meta)[NG], const uint8_t* codes, const uint32_t* metas, int row) {
            const uint4* src = reinterpret_cast<const uint4*>(codes + static_cast<int64_t>(row < 0 ? 0 : row) * KB);
#pragma unroll
            for (int i = 0; i < NX; ++i) x[i] = row < 0 ? make_uint4(0, 0, 0, 0) : __ldg(src + i);
#pragma unroll
            for (int i = 0; i < NG; ++i) meta[i] = row < 0 ? 0u : __ldg(metas + static_cast<int64_t>(row) * NG + i);
        };
        // absent keys have minimum and step 0: their values are 0
        auto convert = [&](const uint4 (&x)[NX], const uint32_t (&meta)[NG], uint32_t dst) {
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
                sts16(piece_at(dst, key, i), a);
            }
        };
        bool ok = true;
        auto slot_free = [&](uint32_t bar, int j) {
            if (j < ST) return true;
            return tc::bar_wait(bar + 8 * (j % ST), ((j / ST) - 1) & 1, abort, status, wait_ns);
        };
        auto publish = [&](uint32_t bar, int j) {
            tc::fence_proxy_async_smem();
            tc::bar_arrive(bar + 8 * (j % ST));
        };
        uint4 xk[NX], xv[NX];
        uint32_t mk[NG], mv[NG];
        int row = row_index(0);
        load(xk, mk, c.kc, c.km, row);
        for (int j = 0; j < nc && ok; ++j) {
            load(xv, mv, c.vc, c.vm, row);
            row = row_index(j + 1);
            if (!(ok = slot_free(k_empty, j))) break;
            convert(xk, mk, sk + (j % ST) * T::BLOCK);
            publish(k_full, j);
            load(xk, mk, c.kc, c.km, row);
            if (!(ok = slot_free(v_empty, j))) break;
            convert(xv, mv, sv + (j % ST) * T::BLOCK);
            publish(v_full, j);
        }
        for (int j = nc; j < nb && ok; ++j) {
            const int tok = (j - nc) * 128 + key;
            const bool there = tok < last;
            const int64_t off = static_cast<int64_t>(u.first + (there ? tok : 0)) * A.kv_stride + head * D;
            const uint4* xk4 = reinterpret_cast<const uint4*>(A.k_new + off);
            const uint4* xv4 = reinterpret_cast<const uint4*>(A.v_new + off);
            if (!(ok = slot_free(k_empty, j))) break;
#pragma unroll 4
            for (int i = 0; i < D / 8; ++i) {
                uint32_t a[4];
                key_pairs_fresh<BITS>(a, there ? __ldg(xk4 + i) : make_uint4(0, 0, 0, 0));
                sts16(piece_at(sk + (j % ST) * T::BLOCK, key, i), a);
            }
            publish(k_full, j);
            if (!(ok = slot_free(v_empty, j))) break;
#pragma unroll 4
            for (int i = 0; i < D / 8; ++i) {
                uint4 v = there ? __ldg(xv4 + i) : make_uint4(0, 0, 0, 0);
                // a hidden key's probability is 0, and 0 * infinity would be NaN
                if (any_wild(v)) {
                    v = without_wild(v);
                    wild_flag = 1;
                }
                uint32_t a[4];
                key_pairs_fresh<BITS>(a, v);
                sts16(piece_at(sv + (j % ST) * T::BLOCK, key, i), a);
            }
            publish(v_full, j);
        }
    } else if (lane == 0) {
        // ---- the matrix products
        constexpr uint32_t idesc_s = tc::idesc_f16_f32(128, 128), idesc_o = tc::idesc_f16_f32(128, D) | tc::kIdescBMnMajor;
        auto scores = [&](int t, int j) {
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {                  // 16 dims a step: 32 bytes of a swizzled row
                const uint32_t off = (k >> 2) * 16384 + (k & 3) * 32;
                tc::mma_f16(tmem + t * 128, tc::desc_k_sw128(sq + t * T::BLOCK + off),
                            tc::desc_k_sw128(sk + (j % ST) * T::BLOCK + off), idesc_s, k > 0);
            }
            tc::mma_commit(s_full + 8 * t);
        };
        bool ok = nb == 0 || tc::bar_wait(q_full, 0, abort, status, wait_ns);
        if (ok && nb > 0) {
            ok = tc::bar_wait(k_full, 0, abort, status, wait_ns);
            if (ok) {
                tc::fence_after_sync();
                for (int t = 0; t < tiles; ++t) scores(t, 0);
                if (nb > ST) tc::mma_commit(k_empty);
            }
        }
        for (int j = 0; j < nb && ok; ++j) {
            for (int t = 0; t < tiles && ok; ++t) {
                if (t == 0) ok = tc::bar_wait(v_full + 8 * (j % ST), (j / ST) & 1, abort, status, wait_ns);
                ok = ok && tc::bar_wait(p_full + 8 * t, j & 1, abort, status, wait_ns);
                if (!ok) break;
                tc::fence_after_sync();
#pragma unroll
                for (int k = 0; k < 8; ++k)                     // 16 keys a step
                    tc::mma_f16_ts(tmem + TILES * 128 + t * D, tmem + t * 128 + k * 8,
                                   tc::desc_mn_sw128(sv + (j % ST) * T::BLOCK + k * 2048, 16384), idesc_o, j > 0 || k > 0);
                tc::mma_commit(o_done + 8 * t);
                if (t == tiles - 1 && j + ST < nb) tc::mma_commit(v_empty + 8 * (j % ST));
                if (j + 1 < nb) {
                    if (t == 0) ok = tc::bar_wait(k_full + 8 * ((j + 1) % ST), ((j + 1) / ST) & 1, abort, status, wait_ns);
                    // S takes the columns that P V reads
                    ok = ok && tc::bar_wait(o_done + 8 * t, j & 1, abort, status, wait_ns);
                    if (!ok) break;
                    tc::fence_after_sync();
                    scores(t, j + 1);
                    if (t == tiles - 1 && j + 1 + ST < nb) tc::mma_commit(k_empty + 8 * ((j + 1) % ST));
                }
            }
        }
        if (!ok) {                                              // what was issued reads shared memory: let it end
            tc::mma_commit(drain);
            tc::bar_wait(drain, 0, abort, status, wait_ns);
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    if (warp == TILES * 4 + 4) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, T::COLS);
    }
}

template <int D, int BITS, int GS, int TILES>
void launch_one(const AttnArgs& a, int64_t units, cudaStream_t st) {
    using T = TileShape<D, TILES>;
    set_smem_once(paged_tile_kernel<D, BITS, GS, TILES>, T::SMEM);
    launch_k(paged_tile_kernel<D, BITS, GS, TILES>, dim3(static_cast<unsigned>(units * a.plan.heads)), dim3(T::THREADS),
             T::SMEM, st, true, a, pipeline_wait_ns());
}

}  // namespace

// Rows of a sequence and key head -> rows of a tile.
int paged_tile_rows(int rows) { return rows <= 128 ? 128 : 256; }

// Blocks wanted: a few for every one that the device holds at once.
int paged_tile_target(int row_tile, int) { return sm_count() * (row_tile == 128 ? 2 : 1) * 2; }

void launch_paged_tile(const AttnArgs& a, int head_dim, int bits, int group, int row_tile, int64_t units, cudaStream_t st) {
#define TILE(D_, B_, G_)                                                  \
    do {                                                                  \
        if (row_tile == 128) launch_one<D_, B_, G_, 1>(a, units, st);     \
        else launch_one<D_, B_, G_, 2>(a, units, st);                     \
    } while (0)
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
