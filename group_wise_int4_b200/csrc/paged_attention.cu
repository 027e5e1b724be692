// Attention of new tokens over a paged compressed KV cache.
//
// For row r (token i of sequence b, query head h, key head g = h / share):
//   s_j = q_r . k_j over the slots j < ctx_len[b] and the fresh tokens 0..i,
//   lse_r = log sum_j exp(s_j),  o_r = sum_j exp(s_j - lse_r) v_j,
// in one pass over the keys with a running maximum and sum; statistics are fp32. Probabilities
// are fp16 operands of the value product: rounding them costs o about as much as its own
// rounding does (1.2 to 1.4 times the error against 64 bits, below one fp16 step of o), which
// up to 4 rows is avoided (TWICE below); above, the second product would be half as many
// again of all, for what the output's type mostly cannot show.
// k_j and v_j are the fp16 values of paged.cuh, so the products are exact and summed in fp32.
#include <type_traits>

#include "paged_attn.cuh"

namespace flexq {
namespace {

// ---- few rows: one warp's 16 keys against 8 or 16 query rows ------------------------------
//
// mma.sync m16n8k16 with the keys as its 16 rows: a decode step has 1 to 16 query rows per
// key head, and a 128-row tcgen05 tile would be all padding. A warp is on its own: it
// streams the codes of one unit and key head through its part of a cp.async ring,
// dequantises in registers and keeps the maximum, the sum and the output (transposed: 16
// dims x 8 rows a tile). The value product O^T = V^T P^T needs P^T as its 8-column operand,
// which movmatrix makes of the score tile; V^T comes from byte permutations of four keys'
// codes, two keys to a register. Metadata goes through registers: the lane of a key turns
// its scales into steps once, for all lanes that use them.
//
// Three instructions for two values (extract, subtract the exponent's offset, one fused
// multiply-add) make about 220 of the 450 that 16 keys of 128 dims take at 4 bits: 144
// sequences of 512 to 543 slots at 96 heads take 307 us (3.5 TB/s, 53% of the measured copy
// bandwidth) with 66% of the issue slots busy and 12 warps a multiprocessor, so latency is
// part of it. It is no lower bound: the contiguous cache's kernel multiplies raw codes and
// applies step and minimum to each group's sums, 370 instructions and 257 us for the same
// sizes, with values rounded otherwise than here. 8-bit codes of four sequences of 3001 to
// 60001 slots shared by 8 heads each: 65 us (75%).
// Warps of a multiprocessor, by registers: at 128 dims the kernel takes 160 to 168 at 8 rows and
// up to 235 at 16 without spilling (16 warps of 128 registers spill, and took 440 us instead
// of 338 for the 144 sequences); at 64 dims 96 and 128 registers spill 20 to 92 bytes.
// At 64 dims and 8 bits shared memory holds 16 of the 20 warps.
constexpr int rows_warps(int dim, int rows) { return dim == 64 ? (rows == 8 ? 20 : 16) : (rows == 8 ? 12 : 8); }

template <int D, int BITS, int GS, int NR>
struct RowsShape {
    static constexpr int KB = D * BITS / 8, NG = D / GS;   // bytes of a key's codes, groups
    static constexpr int KW = KB >= 128 ? 16 : 32;         // keys of a stage
    static constexpr int STAGES = 3;                       // two requested ahead
    static constexpr int CODE = KW * KB, META = KW * NG * 4;
    static constexpr int WARP = STAGES * 2 * CODE + 2 * 2 * META;      // shared bytes of a warp
    static constexpr int WARPS = 2;                        // of a block
    static constexpr int BLOCKS = rows_warps(D, 8 * NR) / WARPS;
};
constexpr int kRowsKeys = 32, kRowsMin = 8;        // a part's granule of keys; a part has at least MIN of them

// 16-byte piece c of key `key` of a stage. Keys: pieces in order, except that the odd keys of
// 128 bytes have theirs swapped in pairs: lanes (g, t) read pieces 2t and 2t + 1 of key g.
template <int KB>
__device__ __forceinline__ int key_piece(int key, int c) {
    return key * (KB / 16) + (KB == 128 ? c ^ (key & 1) : c);
}
// Values: lanes (g, t) read piece(s) g of keys 2t, 2t + 1, ... without bank conflicts.
template <int KB>
__device__ __forceinline__ int value_piece(int key, int c) {
    if (KB == 128) return key * 8 + (c ^ (((key >> 1) & 3) << 1));
    if (KB == 64) return (key ^ ((key >> 1) & 1)) * 4 + (c ^ (((key >> 2) & 1) << 1));
    return (key ^ ((key >> 2) & 1)) * 2 + c;
}

// TWICE (up to 4 rows): columns r and r + 4 hold the same query, and as the value product's
// operands the rounded probabilities and what the rounding left. Their sum has the weights
// in full precision for 3% of the instructions; the error of o falls by 1.4, to that of its own rounding.
template <int D, int BITS, int GS, int NR, bool TWICE>
__global__ void __launch_bounds__(RowsShape<D, BITS, GS, NR>::WARPS * 32, RowsShape<D, BITS, GS, NR>::BLOCKS)
    paged_rows_kernel(AttnArgs A) {
    using S = RowsShape<D, BITS, GS, NR>;
    constexpr int KB = S::KB, KW = S::KW, ST = S::STAGES, NG = S::NG, R = 8 * NR, KT = KW / 16, CODE = S::CODE;
    constexpr int COL = TWICE ? 3 : 7;                      // column -> row of the tile
    extern __shared__ __align__(16) unsigned char ring[];
    pdl_wait();
    pdl_trigger();
    const PagedView& c = A.c;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int item = blockIdx.x * S::WARPS + warp, share = A.plan.share;
    const int head = item % A.plan.heads;
    const Unit u = find_unit<R, kRowsKeys, kRowsMin, 1, false>(c, A.rows, A.plan, item / A.plan.heads);
    record_split<R, kRowsKeys>(A, u, item / A.plan.heads, head);
    if (!u.live) return;
    const int blocks = (u.ctx + kRowsKeys - 1) / kRowsKeys;
    const int key0 = min(blocks, u.part * u.per) * kRowsKeys;
    const int key1 = min(u.ctx, min(blocks, (u.part + 1) * u.per) * kRowsKeys);
    const int stages = (key1 - key0 + KW - 1) / KW;
    const int row_end = u.n * share, row0 = u.tile * R;

    unsigned char* const mine = ring + warp * S::WARP;
    uint32_t* const meta = reinterpret_cast<uint32_t*>(mine + ST * 2 * CODE);      // [2][keys, values][KW][NG]
    const uint32_t my_ring = smem_addr(mine);
    // Pages hold at least 16 keys: each run of 16 is one contiguous piece of a pool. Runs have a
    // page (the entry of the table), then a row, one stage after the other, so that nothing
    // waits for the table.
    const int32_t* const table_row = c.table + static_cast<int64_t>(u.b) * c.max_pages;
    auto find_pages = [&](int (&page)[KT], int s) {
#pragma unroll
        for (int k = 0; k < KT; ++k) {
            const int j = key0 + s * KW + k * 16;
            page[k] = page_entry(c, table_row, j, j < key1);
        }
    };
    auto find_rows = [&](int (&row)[KT], const int (&page)[KT], int s) {
#pragma unroll
        for (int k = 0; k < KT; ++k) row[k] = entry_row(c, page[k], head, key0 + s * KW + k * 16);
    };
    // Whole runs: keys behind the last one lie in the page too, and where there is no page the
    // stage keeps what it held. Their minimum and step are 0, and so are their values.
    const uint8_t *const kc = c.kc + lane * 16, *const vc = c.vc + lane * 16;
    auto load_codes = [&](uint32_t at, const int (&row)[KT]) {
#pragma unroll
        for (int k = 0; k < KT; ++k) {
            if (row[k] < 0) continue;
            const int64_t off = static_cast<int64_t>(row[k]) * KB;
#pragma unroll
            for (int i = 0; i < KB / 32; ++i) {
                const int piece = lane + i * 32, key = k * 16 + piece / (KB / 16), part = piece % (KB / 16);
                cp16(at + key_piece<KB>(key, part) * 16, kc + off + i * 512, true);
                cp16(at + CODE + value_piece<KB>(key, part) * 16, vc + off + i * 512, true);
            }
        }
        cp_commit();
    };
    // metadata of this lane's key, as {min, scale}: at 32 keys a stage of the key and the value, at 16
    // of the key (lanes 0-15) or the value
    constexpr int MS = KW == 32 ? 2 : 1;
    auto load_meta = [&](uint32_t (&w)[MS][NG], int s, const int (&row)[KT]) {
        const int key = lane & (KW - 1), r = key < 16 ? row[0] : row[KT - 1];
        const bool ok = r >= 0 && key0 + s * KW + key < key1;
        const int64_t off = static_cast<int64_t>(ok ? r + (key & 15) : 0) * NG;
#pragma unroll
        for (int k = 0; k < MS; ++k) {
            const uint32_t* src = (MS == 2 ? k == 1 : lane >= 16) ? c.vm : c.km;
#pragma unroll
            for (int i = 0; i < NG; ++i) w[k][i] = ok ? __ldg(src + off + i) : 0u;
        }
    };
    // {min, scale} -> {min, step} in shared memory
    auto put_meta = [&](const uint32_t (&w)[MS][NG], int s) {
        uint32_t* dst = meta + (s & 1) * 2 * KW * NG;
#pragma unroll
        for (int k = 0; k < MS; ++k) {
#pragma unroll
            for (int i = 0; i < NG; ++i)
                dst[(MS == 2 ? k * KW + lane : lane) * NG + i] =
                    (w[k][i] & 0xFFFFu) | (static_cast<uint32_t>(__half_as_ushort(step16_of(w[k][i]))) << 16);
        }
    };

    int row[KT], page[KT];                                  // of the next stage, of the one whose codes are requested next
    int before[KT];                                         // rows of the stage before that
    uint32_t mw[MS][NG];
    {
        int p0[KT], p1[KT], r0[KT];
        find_pages(p0, 0);
        find_pages(p1, 1);
        find_pages(page, 2);
        find_rows(r0, p0, 0);
        load_codes(my_ring, r0);
        load_meta(mw, 0, r0);
#pragma unroll
        for (int k = 0; k < KT; ++k) before[k] = r0[k];
        find_rows(row, p1, 1);
        load_codes(my_ring + 2 * CODE, row);
    }

    // queries; the tokens of this lane's score columns (rows 2t, 2t + 1 of each tile)
    uint32_t bq[NR][D / 16][2];
    int token[NR][2];
#pragma unroll
    for (int n = 0; n < NR; ++n) {
        const int r = row0 + n * 8 + (g & COL);
        const bool ok = r < row_end;
        const int i = ok ? token_of(A.plan, r) : 0, h = ok ? head * share + r - i * share : 0;
        load_query<D, BITS>(bq[n], A.q + static_cast<int64_t>(u.first + i) * A.q_stride + h * D, t, ok);
#pragma unroll
        for (int e = 0; e < 2; ++e) token[n][e] = token_of(A.plan, row0 + n * 8 + ((2 * t + e) & COL));
    }

    float m[NR][2], l[NR][2], acc[D / 16][NR][4];
#pragma unroll
    for (int n = 0; n < NR; ++n) {
        m[n][0] = m[n][1] = -FLT_MAX;
        l[n][0] = l[n][1] = 0.f;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) acc[i][n][0] = acc[i][n][1] = acc[i][n][2] = acc[i][n][3] = 0.f;
    }

    // Scores of T tiles of 16 keys (-inf where hidden) -> running maximum, sum, and the
    // probabilities as the value product's operand. The maximum moves only when a score passes it
    // by kSlack: until then nothing is rescaled.
    auto softmax = [&](auto& sc, auto& pb, auto tiles_c) {
        constexpr int T = decltype(tiles_c)::value;
#pragma unroll
        for (int n = 0; n < NR; ++n) {
            float top[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                top[e] = fmaxf(sc[0][n][e], sc[0][n][2 + e]);
#pragma unroll
                for (int k = 1; k < T; ++k) top[e] = fmaxf(top[e], fmaxf(sc[k][n][e], sc[k][n][2 + e]));
            }
            if (__any_sync(0xffffffffu, top[0] > m[n][0] + kSlack || top[1] > m[n][1] + kSlack)) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
#pragma unroll
                    for (int w = 4; w < 32; w <<= 1) top[e] = fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], w));
                    const bool moves = top[e] > m[n][e] + kSlack;      // a row's result depends on no other row
                    const float f = moves ? exp2_fast(exponent_of(m[n][e], top[e])) : 1.f;
                    m[n][e] = moves ? top[e] : m[n][e];
                    l[n][e] *= f;
#pragma unroll
                    for (int i = 0; i < D / 16; ++i) {
                        acc[i][n][e] *= f;
                        acc[i][n][2 + e] *= f;
                    }
                }
            }
#pragma unroll
            for (int k = 0; k < T; ++k) {
                float p[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) p[e] = exp2_fast(fmaf(sc[k][n][e] - m[n][e & 1], kLog2e, kLift));
                l[n][0] += p[0] + p[2];
                l[n][1] += p[1] + p[3];
                uint32_t h[2] = {half2_of(p[0], p[1]), half2_of(p[2], p[3])};     // (rounded: at the top of the file)
                if (TWICE) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const uint32_t left = half2_of(p[2 * e] - h2f_lo(h[e]), p[2 * e + 1] - h2f_hi(h[e]));
                        h[e] = t < 2 ? h[e] : left;
                    }
                }
                pb[k][n][0] = mat_trans(h[0]);
                pb[k][n][1] = mat_trans(h[1]);
            }
        }
    };

    // ---- fresh keys, by the last part
    bool wild = false;                                      // one of their values is infinite or NaN
    if (A.k_new != nullptr && u.part == u.parts - 1) {
        const int last = (min(row_end, row0 + R) - 1) / share + 1;          // keys any row sees
        const int64_t kv_stride = A.kv_stride;
        const __half* kf = A.k_new + static_cast<int64_t>(u.first) * kv_stride + head * D;
        const __half* vf = A.v_new + static_cast<int64_t>(u.first) * kv_stride + head * D;
        for (int j0 = 0; j0 < last; j0 += 16) {
            float sc[1][NR][4];
#pragma unroll
            for (int n = 0; n < NR; ++n) sc[0][n][0] = sc[0][n][1] = sc[0][n][2] = sc[0][n][3] = 0.f;
            const bool ok0 = j0 + g < last, ok8 = j0 + g + 8 < last;
            const uint4* x0 = reinterpret_cast<const uint4*>(kf + static_cast<int64_t>(ok0 ? j0 + g : 0) * kv_stride + t * (D / 4));
            const uint4* x8 = reinterpret_cast<const uint4*>(kf + static_cast<int64_t>(ok8 ? j0 + g + 8 : 0) * kv_stride + t * (D / 4));
#pragma unroll
            for (int w = 0; w < D / 32; ++w) {
                uint32_t a[4], z[4];
                key_pairs_fresh<BITS>(a, ok0 ? __ldg(x0 + w) : make_uint4(0, 0, 0, 0));
                key_pairs_fresh<BITS>(z, ok8 ? __ldg(x8 + w) : make_uint4(0, 0, 0, 0));
                const uint32_t a0[4] = {a[0], z[0], a[1], z[1]}, a1[4] = {a[2], z[2], a[3], z[3]};
#pragma unroll
                for (int n = 0; n < NR; ++n) {
                    mma168(sc[0][n], a0, bq[n][2 * w][0], bq[n][2 * w][1]);
                    mma168(sc[0][n], a1, bq[n][2 * w + 1][0], bq[n][2 * w + 1][1]);
                }
            }
#pragma unroll
            for (int n = 0; n < NR; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int j = j0 + g + (e >> 1) * 8;
                    if (j >= last || j > token[n][e & 1]) sc[0][n][e] = -INFINITY;
                }
            if (NR == 1 && A.fresh != nullptr && lane == 0) A.fresh[u.b * A.plan.heads + head] = sc[0][0][0];
            uint32_t pb[1][NR][2];
            softmax(sc, pb, std::integral_constant<int, 1>{});
            uint4 x[4][D / 64];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int j = j0 + 2 * t + (k & 1) + 8 * (k >> 1);
#pragma unroll
                for (int w = 0; w < D / 64; ++w)
                    x[k][w] = j < last ? __ldg(reinterpret_cast<const uint4*>(vf + static_cast<int64_t>(j) * kv_stride + g * (D / 8)) + w)
                                       : make_uint4(0, 0, 0, 0);
            }
            // A hidden key's probability is 0, and 0 * infinity would be NaN: infinities and
            // NaN leave the product and are added, at the end, for the rows that see them.
            bool here = false;
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int w = 0; w < D / 64; ++w) here |= any_wild(x[k][w]);
            if (__any_sync(0xffffffffu, here)) {
                wild = true;
#pragma unroll
                for (int k = 0; k < 4; ++k)
#pragma unroll
                    for (int w = 0; w < D / 64; ++w) x[k][w] = without_wild(x[k][w]);
            }
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
                auto word = [&](int k) {
                    const uint4& v = x[k][i / 4];
                    return i % 4 == 0 ? v.x : i % 4 == 1 ? v.y : i % 4 == 2 ? v.z : v.w;
                };
                const uint32_t a[4] = {byte_perm(word(0), word(1), 0x5410u), byte_perm(word(0), word(1), 0x7632u),
                                       byte_perm(word(2), word(3), 0x5410u), byte_perm(word(2), word(3), 0x7632u)};
#pragma unroll
                for (int n = 0; n < NR; ++n) mma168(acc[i][n], a, pb[0][n][0], pb[0][n][1]);
            }
        }
    }

    // ---- cached keys
    const int kgrp = t * (D / 4) / GS, vgrp = g * (D / 8) / GS;     // group of this lane's dims
    int now = 0, ahead = 2 * 2 * CODE;    // stages in the ring: this one, the one requested
    for (int s = 0; s < stages; ++s) {
        put_meta(mw, s);
        cp_wait<ST - 2>();
        __syncwarp();                     // the stage has landed for, and the one before it is read by, every lane
        int here[KT];                     // rows of this stage
#pragma unroll
        for (int k = 0; k < KT; ++k) {
            here[k] = before[k];
            before[k] = row[k];
        }
        load_meta(mw, s + 1, row);
        find_rows(row, page, s + 2);
        load_codes(my_ring + ahead, row);
        find_pages(page, s + 3);
        const int j0 = key0 + s * KW;
        const unsigned char* st = mine + now;
        now = now == 2 * 2 * CODE ? 0 : now + 2 * CODE;
        ahead = ahead == 2 * 2 * CODE ? 0 : ahead + 2 * CODE;
        const uint32_t* kmeta = meta + (s & 1) * 2 * KW * NG;
        const uint32_t* vmeta = kmeta + KW * NG;
        float sc[KT][NR][4];
#pragma unroll
        for (int k = 0; k < KT; ++k) {
#pragma unroll
            for (int n = 0; n < NR; ++n) sc[k][n][0] = sc[k][n][1] = sc[k][n][2] = sc[k][n][3] = 0.f;
            uint32_t x0[KB / 16], x8[KB / 16];
#pragma unroll
            for (int w = 0; w < KB / 16; w += (KB >= 64 ? 4 : 2)) {
                if (KB >= 64) {
                    constexpr int PER = KB / 64;           // pieces of a lane
                    const uint4 a = *reinterpret_cast<const uint4*>(st + key_piece<KB>(k * 16 + g, t * PER + w / 4) * 16);
                    const uint4 z = *reinterpret_cast<const uint4*>(st + key_piece<KB>(k * 16 + g + 8, t * PER + w / 4) * 16);
                    x0[w] = a.x; x0[(w + 1) % (KB / 16)] = a.y; x0[(w + 2) % (KB / 16)] = a.z; x0[(w + 3) % (KB / 16)] = a.w;
                    x8[w] = z.x; x8[(w + 1) % (KB / 16)] = z.y; x8[(w + 2) % (KB / 16)] = z.z; x8[(w + 3) % (KB / 16)] = z.w;
                } else {
                    const unsigned char* kc = st + (k * 16 + g) * KB + t * (KB / 4);
                    const uint2 a = *reinterpret_cast<const uint2*>(kc + w * 4), z = *reinterpret_cast<const uint2*>(kc + 8 * KB + w * 4);
                    x0[w] = a.x; x0[(w + 1) % (KB / 16)] = a.y;
                    x8[w] = z.x; x8[(w + 1) % (KB / 16)] = z.y;
                }
            }
            const uint32_t m0 = kmeta[(k * 16 + g) * NG + kgrp], m8 = kmeta[(k * 16 + g + 8) * NG + kgrp];
            const uint32_t st0 = dup_hi(m0), st8 = dup_hi(m8), mn0 = dup_lo(m0), mn8 = dup_lo(m8);
#pragma unroll
            for (int w = 0; w < D / 32; ++w) {
                uint32_t a[4], z[4];
                constexpr int W = BITS / 4;
                key_pairs<BITS>(a, x0[w * W], x0[w * W + W - 1], st0, mn0);
                key_pairs<BITS>(z, x8[w * W], x8[w * W + W - 1], st8, mn8);
                const uint32_t a0[4] = {a[0], z[0], a[1], z[1]}, a1[4] = {a[2], z[2], a[3], z[3]};
#pragma unroll
                for (int n = 0; n < NR; ++n) {
                    mma168(sc[k][n], a0, bq[n][2 * w][0], bq[n][2 * w][1]);
                    mma168(sc[k][n], a1, bq[n][2 * w + 1][0], bq[n][2 * w + 1][1]);
                }
            }
            if (NR == 1 && A.scores != nullptr && t == 0 && here[k] >= 0) {
                A.scores[here[k] + g] = sc[k][0][0];         // (a whole run lies in the page)
                A.scores[here[k] + g + 8] = sc[k][0][2];
            }
            if (j0 + KW > key1) {
                const bool in0 = j0 + k * 16 + g < key1, in8 = j0 + k * 16 + g + 8 < key1;
#pragma unroll
                for (int n = 0; n < NR; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (!(e < 2 ? in0 : in8)) sc[k][n][e] = -INFINITY;
            }
        }
        uint32_t pb[KT][NR][2];
        softmax(sc, pb, std::integral_constant<int, KT>{});
#pragma unroll
        for (int k = 0; k < KT; ++k) {
            constexpr int VW = KB / 32;                    // words a lane takes of a key
            uint32_t x[4][VW];
            uint32_t step[2], mn[2];
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                const int key = k * 16 + 2 * t + 8 * p;
                const uint32_t ma = vmeta[key * NG + vgrp], mz = vmeta[(key + 1) * NG + vgrp];
                step[p] = byte_perm(ma, mz, 0x7632u);
                mn[p] = byte_perm(ma, mz, 0x5410u);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int key = k * 16 + 2 * t + (i & 1) + 8 * (i >> 1);
                const int off = g * (KB / 8);
                const unsigned char* vp = st + CODE + value_piece<KB>(key, off / 16) * 16 + off % 16;
                if (VW == 4) {
                    const uint4 a = *reinterpret_cast<const uint4*>(vp);
                    x[i][0] = a.x; x[i][1 % VW] = a.y; x[i][2 % VW] = a.z; x[i][3 % VW] = a.w;
                } else if (VW == 2) {
                    const uint2 a = *reinterpret_cast<const uint2*>(vp);
                    x[i][0] = a.x; x[i][1 % VW] = a.y;
                } else {
                    x[i][0] = *reinterpret_cast<const uint32_t*>(vp);
                }
            }
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {             // dims 2i and 2i + 1 of this lane's D/8
                uint32_t a[4];
                if (BITS == 4) {
                    const uint32_t sel = (i % 4) * 0x11u + (4 + i % 4) * 0x1100u;
                    const uint32_t y0 = byte_perm(x[0][i / 4 % VW], x[1][i / 4 % VW], sel);
                    const uint32_t y1 = byte_perm(x[2][i / 4 % VW], x[3][i / 4 % VW], sel);
                    a[0] = h2_fma(codes_lo(y0), step[0], mn[0]);
                    a[1] = h2_fma(codes_hi(y0), step[0], mn[0]);
                    a[2] = h2_fma(codes_lo(y1), step[1], mn[1]);
                    a[3] = h2_fma(codes_hi(y1), step[1], mn[1]);
                } else {
                    const int w = i / 2 % VW, b0 = (i % 2) * 2;
                    // bytes b0, b0 + 1 of both keys: [k0.b0, k1.b0, k0.b1, k1.b1]
                    const uint32_t sel = b0 | ((4u + b0) << 4) | ((1u + b0) << 8) | ((5u + b0) << 12);
                    const uint32_t y0 = byte_perm(x[0][w], x[1][w], sel), y1 = byte_perm(x[2][w], x[3][w], sel);
                    a[0] = h2_fma(codes_b01(y0), step[0], mn[0]);
                    a[1] = h2_fma(codes_b23(y0), step[0], mn[0]);
                    a[2] = h2_fma(codes_b01(y1), step[1], mn[1]);
                    a[3] = h2_fma(codes_b23(y1), step[1], mn[1]);
                }
#pragma unroll
                for (int n = 0; n < NR; ++n) mma168(acc[i][n], a, pb[k][n][0], pb[k][n][1]);
            }
        }
    }
    cp_wait<0>();

    if (TWICE) {
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[i][0][e] += __shfl_xor_sync(0xffffffffu, acc[i][0][e], 2);
    }
    // lane (g, t): rows 2t, 2t + 1 of each tile, dims [g D/8, (g + 1) D/8)
#pragma unroll
    for (int n = 0; n < NR; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float sum = l[n][e];
#pragma unroll
            for (int w = 4; w < 32; w <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
            const int r = n * 8 + 2 * t + e;
            if (row0 + r >= row_end) continue;
            // whatever their weight, which is positive, the sum is what they make it
            if (wild) {
                for (int j = 0; j <= token[n][e]; ++j) {
                    const __half* vr = A.v_new + static_cast<int64_t>(u.first + j) * A.kv_stride + head * D + g * (D / 8);
#pragma unroll
                    for (int i = 0; i < D / 16; ++i) {
                        const float v0 = __half2float(vr[2 * i]), v1 = __half2float(vr[2 * i + 1]);
                        if (!isfinite(v0)) acc[i][n][e] += v0;
                        if (!isfinite(v1)) acc[i][n][2 + e] += v1;
                    }
                }
            }
            if (u.parts == 1) {
                const int64_t at = static_cast<int64_t>(u.first + token[n][e]) * (A.plan.heads * share) + head * share + row0 + r - token[n][e] * share;
                const float inv = sum == 0.f ? 0.f : 1.f / sum;
                uint32_t w[D / 16];
#pragma unroll
                for (int i = 0; i < D / 16; ++i) w[i] = half2_of(acc[i][n][e] * inv, acc[i][n][2 + e] * inv);
#pragma unroll
                for (int i = 0; i < D / 16; i += 4)
                    *reinterpret_cast<uint4*>(A.o + at * D + g * (D / 8) + 2 * i) = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
                if (g == 0) put_stats(A, at, m[n][e], sum, kLift);
            } else if (u.slot < A.slots) {
                const float down = 0.015625f;                  // 2^-kLift
                float* p = A.parts + ((static_cast<int64_t>(u.slot) * A.plan.heads + head) * R + r) * (D + 4);
#pragma unroll
                for (int i = 0; i < D / 16; i += 2)
                    *reinterpret_cast<float4*>(p + g * (D / 8) + 2 * i) =
                        make_float4(acc[i][n][e] * down, acc[i][n][2 + e] * down, acc[i + 1][n][e] * down, acc[i + 1][n][2 + e] * down);
                if (g == 0) *reinterpret_cast<float2*>(p + D) = make_float2(m[n][e], sum * down);
            }
        }
}

// ---- accumulated weights ------------------------------------------------------------------
//
// weight[slot] += sum over rows of exp(s - lse), with the rows' final statistics.
//
// One row (a decode step without shared heads): the attention kernel leaves its scores, 4
// bytes a slot, and this pass reads them and updates the weights: 12 bytes a slot instead
// of the codes and their conversion again (32 sequences of 500 to 1999 slots, 32 heads of
// 64: 72 us with the kernel below).
template <bool LOOP>
__global__ void __launch_bounds__(128) paged_weight_one_kernel(AttnArgs A) {
    const PagedView& c = A.c;
    const int head = blockIdx.y, b = blockIdx.z;
    int first;
    const int n = rows_of(A.rows, b, first, c.status);
    const int ctx = slots_of(c, b), held = n > 0 && ctx >= 0 ? ctx + (A.k_new != nullptr) : 0, cap = paged_capacity(c);
    // four slots of one page at a time; their row, -1: none
    auto find_row = [&](int s0) {
        if (s0 >= held) return -1;
        if (s0 >= cap) {
            paged_bad(c);                                     // no slot for the new token
            return -1;
        }
        const int p = page_of(c, b, s0);
        return p < 0 ? -1 : slot_row(c, p, head, s0);
    };
    int s0 = (blockIdx.x * 128 + threadIdx.x) * 4, row = find_row(s0);
    pdl_wait();                                               // the attention kernel writes what follows
    pdl_trigger();
    if (LOOP ? s0 >= held : row < 0) return;
    const float2 stats = A.stats[static_cast<int64_t>(first) * A.plan.heads + head];
    for (;;) {
        if (!LOOP || row >= 0) {
            const float fresh = s0 + 4 > ctx && held > ctx ? prob_of(A.fresh[b * A.plan.heads + head], stats) : 0.f;
            const float4 sc = *reinterpret_cast<const float4*>(A.scores + row);
            float4 w = *reinterpret_cast<const float4*>(c.weight + row);
            auto one = [&](float& x, float score, int s) {
                if (s < ctx) x += prob_of(score, stats);
                else if (s < held) x = fresh;
            };
            one(w.x, sc.x, s0);
            one(w.y, sc.y, s0 + 1);
            one(w.z, sc.z, s0 + 2);
            one(w.w, sc.w, s0 + 3);
            *reinterpret_cast<float4*>(c.weight + row) = w;
        }
        s0 += gridDim.x * 512;
        if (!LOOP || s0 >= held) break;
        row = find_row(s0);
    }
}

// Any number of rows: the scores again (about 25 of the 71 us of 12 sequences with 1 to 97 new
// tokens over up to 1500 slots, 32 heads of 64: latency of the first loads, 49% of the issue slots;
// 28 of 62 us of a decode step with 2 heads sharing 16 key heads). A warp holds 32 keys as
// operands in registers and goes through all query rows of the sequence, so every key's sum
// stays in its lanes and is added in one fixed order; no atomics. Query rows pass through
// shared memory, 32 at a time, for 4 warps. The registers that fit 7 (64 dims) and 4 blocks
// spill 4 to 24 bytes.
template <int D, int BITS, int GS, bool LOOP>
__global__ void __launch_bounds__(128, D == 64 ? 7 : 4) paged_weight_kernel(AttnArgs A) {
    const PagedView& c = A.c;
    const RowsPlan& plan = A.plan;
    const __half *q = A.q, *k_new = A.k_new;
    const int64_t q_stride = A.q_stride, kv_stride = A.kv_stride;
    constexpr int KB = D * BITS / 8, NG = D / GS, QR = 32, LD = D + 8;
    __shared__ __align__(16) __half sq[2][QR * LD];
    __shared__ float2 sl[2][QR];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int head = blockIdx.y, b = blockIdx.z;
    int first;
    const int n = rows_of(A.rows, b, first, c.status), ctx = slots_of(c, b), cap = paged_capacity(c);
    const int old_blocks = (ctx + 127) / 128, blocks = n == 0 || ctx < 0 ? 0 : old_blocks + (k_new ? (n + 127) / 128 : 0);
    bool waited = false;
    for (int block = blockIdx.x; block < blocks; block += gridDim.x) {
        const bool fresh = block >= old_blocks;
        const int j0 = (block - (fresh ? old_blocks : 0)) * 128 + warp * 32;     // slot, or fresh token
        const int jend = fresh ? n : ctx;
        // rows of the tokens that see any of the block's keys
        const int row_lo = fresh ? (j0 - warp * 32) * plan.share : 0, row_end = n * plan.share;
        const int tiles = (row_end - row_lo + QR - 1) / QR;
        auto load_q = [&](int s) {
            for (int i = tid; i < QR * (D / 8); i += 128) {
                const int r = row_lo + s * QR + i / (D / 8), d = (i % (D / 8)) * 8;
                const bool ok = r < row_end;
                const int tok = ok ? token_of(plan, r) : 0, h = ok ? head * plan.share + r - tok * plan.share : 0;
                cp16(smem_addr(&sq[s & 1][(i / (D / 8)) * LD + d]), q + static_cast<int64_t>(first + tok) * q_stride + h * D + d, ok);
            }
            cp_commit();
        };
        auto load_stats = [&](int s) {
            if (tid < QR) {
                const int r = row_lo + s * QR + tid;
                const int tok = token_of(plan, r), h = head * plan.share + r - tok * plan.share;
                sl[s & 1][tid] = r < row_end ? A.stats[static_cast<int64_t>(first + tok) * (plan.heads * plan.share) + h] : make_float2(0.f, 0.f);
            }
        };
        // All that the attention kernel does not write is requested before it is waited for: the
        // first queries, and the keys, which become operands (in the order of the dims, as the
        // queries' are) meanwhile.
        load_q(0);
        int row[4];                                         // pool rows of keys j0 + g + 8 i, -1: none
        uint32_t a[2][D / 16][4];
        const int kgrp = t * (D / 4) / GS;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int j = j0 + g + 8 * i, slot = fresh ? ctx + j : j;
            row[i] = -1;
            if (j < jend) {
                if (slot >= cap) {
                    paged_bad(c);
                } else {
                    const int p = page_of(c, b, slot);
                    if (p >= 0) row[i] = slot_row(c, p, head, slot);
                }
            }
            uint32_t pr[D / 32][4];
            if (!fresh) {
                const int64_t r = row[i] < 0 ? 0 : row[i];
                const uint32_t meta = row[i] < 0 ? 0u : __ldg(c.km + r * NG + kgrp);
                const uint32_t step = dup16(step16_of(meta)), mn = dup_lo(meta);
                const uint8_t* kc = c.kc + r * KB + t * (KB / 4);
                uint32_t x[KB / 16];
#pragma unroll
                for (int w = 0; w < KB / 16; w += 2) {
                    const uint2 v = row[i] < 0 ? make_uint2(0, 0) : __ldg(reinterpret_cast<const uint2*>(kc + w * 4));
                    x[w] = v.x;
                    x[w + 1] = v.y;
                }
#pragma unroll
                for (int w = 0; w < D / 32; ++w) {
                    uint32_t z[4];
                    key_pairs<BITS>(z, x[w * (BITS / 4)], x[w * (BITS / 4) + BITS / 4 - 1], step, mn);
                    // at 4 bits the pairs are (d, d + 4): neighbours again
                    pr[w][0] = BITS == 4 ? byte_perm(z[0], z[1], 0x5410u) : z[0];
                    pr[w][1] = BITS == 4 ? byte_perm(z[2], z[3], 0x5410u) : z[1];
                    pr[w][2] = BITS == 4 ? byte_perm(z[0], z[1], 0x7632u) : z[2];
                    pr[w][3] = BITS == 4 ? byte_perm(z[2], z[3], 0x7632u) : z[3];
                }
            } else {
                const uint4* x = reinterpret_cast<const uint4*>(k_new + static_cast<int64_t>(first + (j < jend ? j : 0)) * kv_stride +
                                                                head * D + t * (D / 4));
#pragma unroll
                for (int w = 0; w < D / 32; ++w) key_pairs_fresh<8>(pr[w], j < jend ? __ldg(x + w) : make_uint4(0, 0, 0, 0));
            }
#pragma unroll
            for (int w = 0; w < D / 32; ++w) {
                a[i / 2][2 * w][i % 2] = pr[w][0];
                a[i / 2][2 * w][2 + i % 2] = pr[w][1];
                a[i / 2][2 * w + 1][i % 2] = pr[w][2];
                a[i / 2][2 * w + 1][2 + i % 2] = pr[w][3];
            }
        }
        if (!waited) {
            pdl_wait();
            pdl_trigger();
        }
        waited = true;
        load_stats(0);
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
        // 8 rows and the warp's 32 keys; ALL: every row sees every key
        auto rows8 = [&](int s, int u, auto all_c) {
            constexpr bool ALL = decltype(all_c)::value;
            const int r0 = row_lo + s * QR + u * 8;
            float sc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
            const __half* qr = &sq[s & 1][(u * 8 + g) * LD + t * (D / 4)];
#pragma unroll
            for (int w = 0; w < D / 32; ++w) {
                const uint4 z = *reinterpret_cast<const uint4*>(qr + w * 8);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    mma168(sc[k], a[k][2 * w], z.x, z.y);
                    mma168(sc[k], a[k][2 * w + 1], z.z, z.w);
                }
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = r0 + 2 * t + e;
                const float2 stats = sl[s & 1][u * 8 + 2 * t + e];
                // the last key that the row sees; a row behind the last one sees none
                const int seen = ALL ? 0 : r >= row_end ? -1 : fresh ? token_of(plan, r) : INT32_MAX;
#pragma unroll
                for (int k = 0; k < 2; ++k)
#pragma unroll
                    for (int hh = 0; hh < 2; ++hh) {
                        const float p = prob_of(sc[k][2 * hh + e], stats);
                        if (ALL || j0 + k * 16 + hh * 8 + g <= seen) sum[2 * k + hh] += p;
                    }
            }
        };
        for (int s = 0; s < tiles; ++s) {
            if (s + 1 < tiles) {
                load_q(s + 1);
                load_stats(s + 1);
            } else {
                cp_commit();
            }
            cp_wait<1>();
            __syncthreads();
            if (!fresh && row_lo + (s + 1) * QR <= row_end) {
#pragma unroll
                for (int u = 0; u < QR / 8; ++u) rows8(s, u, std::true_type{});
            } else {
                for (int u = 0; u < QR / 8 && row_lo + s * QR + u * 8 < row_end; ++u) rows8(s, u, std::false_type{});
            }
            __syncthreads();
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 1);
            sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 2);
            if (t == 0 && row[i] >= 0) c.weight[row[i]] = fresh ? sum[i] : c.weight[row[i]] + sum[i];
        }
        if (!LOOP) break;
    }
    if (!waited) pdl_wait();        // (a launch that ends is one whose predecessors have ended)
}

// ---- host -----------------------------------------------------------------------------------

struct AttnPlan {
    int share, row_tile, target, slots;
    int64_t units, records_bytes, parts_bytes, stats_bytes, fresh_bytes, score_bytes;
    int64_t bytes() const { return records_bytes + parts_bytes + stats_bytes + fresh_bytes + score_bytes; }
};

inline int64_t up256(int64_t v) { return (v + 255) / 256 * 256; }

// Blocks along a sequence's keys of the weights' kernels. A table may be far longer than what its
// sequences hold: above 256 blocks a multiprocessor no more are launched than fill the
// device twice, and each goes on to the keys that are left (LOOP). Below, a block for
// every piece: the loop's registers cost 2 of the ragged chunks' 70 us.
struct WeightGrid {
    dim3 grid;
    bool loop;
};
WeightGrid weight_grid(int64_t most, int heads, int batch) {
    const int64_t pairs = static_cast<int64_t>(heads) * batch, fill = (32LL * sm_count() + pairs - 1) / pairs;
    const bool loop = most > fill && most * pairs > 256LL * sm_count();
    return WeightGrid{dim3(static_cast<unsigned>(loop ? fill : most), heads, batch), loop};
}

AttnPlan attn_plan(const flex_paged_cache* c, int n_heads, int batch, int total, int most, bool accumulate) {
    AttnPlan p{};
    p.share = n_heads / c->n_kv_heads;
    const int64_t rows = static_cast<int64_t>(most) * p.share;
    // Row tiles of 16 up to 32 rows, though each of two turns the codes into operands by itself, tcgen05
    // tiles above. us with 16-row / 128-row tiles for 8 sequences of 2000 slots at 16 heads of 64, 32 of
    // 1000 at 32 of 128, 4 of 16000 at 8 of 128 and 8 bits: 17 rows 30 / 35, 123 / 160, 62 / 88; 32 rows
    // 33 / 32, 126 / 161, 64 / 89; 33 rows 43 / 36, 185 / 161, 89 / 91.
    p.row_tile = rows <= 8 ? 8 : rows <= 32 ? 16 : paged_tile_rows(rows > 1024 ? 1024 : static_cast<int>(rows));
    // units times heads wanted: what the device holds at once
    p.target = p.row_tile <= 16 ? rows_warps(c->head_dim, p.row_tile) * sm_count() : paged_tile_target(p.row_tile);
    // every sequence's row tiles, and what their parts add (the bounds stand at find_unit)
    const int64_t more = (p.target + c->n_kv_heads - 1) / c->n_kv_heads;
    p.units = (static_cast<int64_t>(total) * p.share) / p.row_tile + batch + more;
    p.slots = static_cast<int>(2 * more);
    p.records_bytes = 256 + up256(static_cast<int64_t>(p.slots) * sizeof(SplitRecord));
    p.parts_bytes = up256(static_cast<int64_t>(p.slots) * c->n_kv_heads * p.row_tile * (c->head_dim + 4) * 4);
    const bool one = accumulate && rows == 1;
    p.fresh_bytes = one ? up256(static_cast<int64_t>(batch) * n_heads * 4) : 0;
    p.score_bytes = one ? up256(static_cast<int64_t>(c->num_pages) * c->page_size * c->n_kv_heads * 4) : 0;
    p.stats_bytes = accumulate ? up256(static_cast<int64_t>(total) * n_heads * 8) : 0;
    return p;
}

}  // namespace
}  // namespace flexq

using namespace flexq;

namespace {

int validate_attention(const flex_paged_cache* c, int32_t n_heads, int32_t accumulate) {
    const int rc = validate_paged(c, true);
    if (rc != FLEX_OK) return rc;
    FLEX_REQUIRE(n_heads > 0 && n_heads % c->n_kv_heads == 0, FLEX_ERR_INVALID_ARG);
    FLEX_REQUIRE(n_heads <= 65535, FLEX_ERR_UNSUPPORTED);
    FLEX_REQUIRE(!accumulate || c->weight, FLEX_ERR_INVALID_ARG);
    return FLEX_OK;
}

}  // namespace

extern "C" int64_t flex_paged_attention_ws_bytes(const flex_paged_cache* cache, int32_t n_heads, int32_t batch, int32_t total,
                                                 int32_t most, int32_t accumulate) {
    int rc = validate_attention(cache, n_heads, accumulate);
    if (rc != FLEX_OK) return rc;
    FLEX_REQUIRE(batch > 0 && batch <= cache->batch && total >= 0 && most >= 0, FLEX_ERR_INVALID_ARG);
    FLEX_REQUIRE(most <= (1 << 24), FLEX_ERR_UNSUPPORTED);
    return attn_plan(cache, n_heads, batch, total, most, accumulate != 0).bytes();
}

extern "C" int flex_paged_attention(const flex_paged_cache* cache, const void* q, int64_t q_stride, int32_t n_heads,
                                    const void* k_new, const void* v_new, int64_t kv_stride, void* o, float* lse,
                                    const int32_t* cu_new, int32_t batch, int32_t total, int32_t most, int32_t accumulate,
                                    void* ws, int64_t ws_bytes, void* stream) {
    int rc = validate_attention(cache, n_heads, accumulate);
    if (rc == FLEX_OK) rc = validate_rows(cache, cu_new, batch, total, most);
    if (rc != FLEX_OK) return rc;
    FLEX_REQUIRE(q && o && (k_new == nullptr) == (v_new == nullptr), FLEX_ERR_INVALID_ARG);
    FLEX_REQUIRE(q_stride >= static_cast<int64_t>(n_heads) * cache->head_dim, FLEX_ERR_INVALID_ARG);
    FLEX_REQUIRE(k_new == nullptr || kv_stride >= static_cast<int64_t>(cache->n_kv_heads) * cache->head_dim,
                 FLEX_ERR_INVALID_ARG);
    FLEX_REQUIRE(q_stride % 8 == 0 && (k_new == nullptr || kv_stride % 8 == 0), FLEX_ERR_ALIGN);
    FLEX_REQUIRE(aligned16(q) && aligned16(k_new) && aligned16(v_new) && aligned16(o), FLEX_ERR_ALIGN);
    FLEX_REQUIRE((reinterpret_cast<uintptr_t>(lse) & 3u) == 0, FLEX_ERR_ALIGN);
    const AttnPlan p = attn_plan(cache, n_heads, batch, total, most, accumulate != 0);
    FLEX_REQUIRE(ws != nullptr && ws_bytes >= p.bytes(), FLEX_ERR_WORKSPACE);
    FLEX_REQUIRE(aligned16(ws), FLEX_ERR_ALIGN);
    if (most == 0 || total == 0) return FLEX_OK;
    const int kvh = cache->n_kv_heads;
    FLEX_REQUIRE(p.units * kvh < (1LL << 31), FLEX_ERR_UNSUPPORTED);
    FLEX_REQUIRE(static_cast<int64_t>(most) * p.share < (1LL << 31) - 512, FLEX_ERR_UNSUPPORTED);

    AttnArgs a{};
    a.c = paged_view(cache);
    a.rows = RowsOf{cu_new, most, total};
    a.plan = RowsPlan{batch, p.share, p.target, kvh, 0u};
    if (p.share > 1 && (static_cast<int64_t>(most) * p.share + 512) * p.share < (1LL << 32))     // (+ 512: rows of a last tile)
        a.plan.share_inverse = static_cast<uint32_t>((1ULL << 32) / p.share + 1);
    a.q = static_cast<const __half*>(q);
    a.q_stride = q_stride;
    a.k_new = static_cast<const __half*>(k_new);
    a.v_new = static_cast<const __half*>(v_new);
    a.kv_stride = kv_stride;
    a.o = static_cast<__half*>(o);
    unsigned char* w = static_cast<unsigned char*>(ws);
    a.split_units = reinterpret_cast<int*>(w);
    a.records = reinterpret_cast<SplitRecord*>(w + 256);
    a.parts = reinterpret_cast<float*>(w + p.records_bytes);
    a.lse = lse;
    a.stats = accumulate ? reinterpret_cast<float2*>(w + p.records_bytes + p.parts_bytes) : nullptr;
    a.slots = p.slots;
    if (p.score_bytes > 0) {
        w += p.records_bytes + p.parts_bytes + p.stats_bytes;
        a.fresh = reinterpret_cast<float*>(w);
        a.scores = reinterpret_cast<float*>(w + p.fresh_bytes);
    }
    const cudaStream_t st = as_stream(stream);
    const int D = cache->head_dim, B = cache->cfg.num_bits, G = cache->cfg.group_size;
    if (p.row_tile > 16) {
        launch_paged_tile(a, D, B, G, p.row_tile, p.units, st);
    } else {
#define ROWS(D_, B_, G_, N_, T_)                                                                                        \
    do {                                                                                                            \
        using S = RowsShape<D_, B_, G_, N_>;                                                             \
        constexpr int smem = S::WARPS * S::WARP;                                                         \
        set_smem_once(paged_rows_kernel<D_, B_, G_, N_, T_>, smem);                                          \
        const int64_t items = p.units * kvh;                                                             \
        launch_k(paged_rows_kernel<D_, B_, G_, N_, T_>, dim3(static_cast<unsigned>((items + S::WARPS - 1) / S::WARPS)), \
                 dim3(S::WARPS * 32), smem, st, true, a);                                                \
        launch_join<D_, 8 * N_, kRowsKeys, kRowsMin>(a, st);                                             \
    } while (0)
#define ROWS_N(D_, B_, G_) \
    do {                                                                                 \
        if (p.row_tile == 16) ROWS(D_, B_, G_, 2, false);                                \
        else if (static_cast<int64_t>(most) * p.share <= 4) ROWS(D_, B_, G_, 1, true);   \
        else ROWS(D_, B_, G_, 1, false);                                                 \
    } while (0)
        if (D == 64) {
            if (B == 4 && G == 32) ROWS_N(64, 4, 32); else if (B == 4) ROWS_N(64, 4, 64);
            else if (G == 32) ROWS_N(64, 8, 32); else ROWS_N(64, 8, 64);
        } else {
            if (B == 4 && G == 32) ROWS_N(128, 4, 32); else if (B == 4) ROWS_N(128, 4, 64);
            else if (G == 32) ROWS_N(128, 8, 32); else ROWS_N(128, 8, 64);
        }
#undef ROWS_N
#undef ROWS
    }
    if (a.scores != nullptr) {
        const int64_t cap = static_cast<int64_t>(cache->max_pages) * cache->page_size;
        const WeightGrid w = weight_grid((cap + (k_new ? 1 : 0) + 511) / 512, kvh, batch);        // every 512 slots
        if (w.loop)
            launch_k(paged_weight_one_kernel<true>, w.grid, dim3(128), 0, st, true, a);
        else
            launch_k(paged_weight_one_kernel<false>, w.grid, dim3(128), 0, st, true, a);
    } else if (accumulate) {
        const int64_t cap = static_cast<int64_t>(cache->max_pages) * cache->page_size;
        const WeightGrid w = weight_grid((cap + 127) / 128 + (k_new ? (most + 127) / 128 : 0), kvh, batch);      // every 128 keys
#define WEIGHT(D_, B_, G_)                                                                              \
    do {                                                                                                \
        if (w.loop) launch_k(paged_weight_kernel<D_, B_, G_, true>, w.grid, dim3(128), 0, st, true, a); \
        else launch_k(paged_weight_kernel<D_, B_, G_, false>, w.grid, dim3(128), 0, st, true, a);       \
    } while (0)
        if (D == 64) {
            if (B == 4 && G == 32) WEIGHT(64, 4, 32); else if (B == 4) WEIGHT(64, 4, 64);
            else if (G == 32) WEIGHT(64, 8, 32); else WEIGHT(64, 8, 64);
        } else {
            if (B == 4 && G == 32) WEIGHT(128, 4, 32); else if (B == 4) WEIGHT(128, 4, 64);
            else if (G == 32) WEIGHT(128, 8, 32); else WEIGHT(128, 8, 64);
        }
#undef WEIGHT
    }
    return launch_status();
}
