// Eviction from a paged compressed KV cache by accumulated attention weight.
//
// Per (sequence, key head) the cache keeps `budget` of its n > budget slots: first the slots
// whose position lies within `recent` of the head's latest one, then those with the
// largest accumulated weight; equal weights go to the lower slot. Kept slots do not move
// unless they lie behind the budget: the i-th slot given up below it takes the i-th kept
// slot behind it (both in slot order). A cache that is a few tokens over its budget thus
// moves a few slots instead of shifting half of the cache, which is why a slot's position
// is stored beside it and its order in the cache means nothing to attention.
//
// Tables of up to 2048 slots: one launch, a block per (sequence, head) that holds 8
// consecutive slots a thread (one page lookup, two wide loads each of weights and positions),
// finds the budget-th largest key bit by bit with counts over the block, lists the moves
// with two block scans and copies. Nothing passes through memory but what has to; latency
// and the search's barriers bound it: 32 sequences of 1000 to 1040 slots cut to 1024 at 32
// heads 12 us, 4 prompts of 500 to 2048 cut to 512 at 56 heads 13 (the two launches below,
// by a table of a few more pages: 20 and 23). Longer tables, whatever their sequences hold:
// select and move below.
//
// select: one block per (sequence, head). The keys (an order-preserving integer of the
// weight, the largest value for the recent slots) go to shared memory once, the
// budget-th largest is found digit by digit from histograms (11 + 11 + 10 bits), and one
// ordered pass lists what is given up and what moves. Weights and positions are read
// once (8 bytes a slot); the block's few synchronised passes over shared memory bound it:
// 8 sequences of 6000 slots cut to 4096 at 32 heads of 128 take 82 us (floor 17), 2 of
// 40000 cut to 8192 at 8 heads 152 (16 blocks on the whole device).
// move: 8 lanes copy one slot (codes, metadata, weight, position) to its place.
#include "paged.cuh"

namespace flexq {
namespace {

constexpr int PE_THREADS = 512;
constexpr int PE_CACHE = 32768;        // keys held in shared memory; the rest is read again
constexpr int PE_BINS = 2048;

// Larger weights have larger keys, below the recent slots' 0xFFFFFFFF. -0 counts as +0 and
// a NaN as -infinity.
__device__ __forceinline__ uint32_t weight_key(float w) {
    uint32_t u = __float_as_uint(w);
    if (w != w) u = 0xFF800000u;
    if (u == 0x80000000u) u = 0u;
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

constexpr int PS_T = 256, PS_PER = 8, PS_SLOTS = PS_T * PS_PER;      // threads, slots a thread, slots at most

// U: moves that 8 lanes have under way at once; few of them leave registers for more blocks.
template <int KB, int U>
__global__ void __launch_bounds__(PS_T, U == 1 ? 7 : 4) evict_small_kernel(PagedView c, int budget, int recent, int ng,
                                                              int32_t* __restrict__ new_len) {
    constexpr int WARPS = PS_T / 32, PL = KB >= 64 ? KB / 64 : 1;    // 16-byte pieces of a lane: keys', then values'
    __shared__ int pages[PS_SLOTS / 16];
    __shared__ uint16_t from[PS_SLOTS / 2], to[PS_SLOTS / 2];        // moves: at most half of the slots
    __shared__ int red[2][WARPS], moved_count;
    pdl_wait();
    pdl_trigger();
    const int head = blockIdx.x, b = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int n = slots_of(c, b);
    if (head == 0 && tid == 0) new_len[b] = n < 0 ? __ldg(c.ctx_len + b) : min(n, budget);      // (a wrong length stays one)
    if (n <= budget) return;
    for (int i = tid; i < (n + (1 << c.shift) - 1) >> c.shift; i += PS_T) pages[i] = page_of(c, b, i << c.shift);
    __syncthreads();
    // warps without a slot wait for the moves; the others meet at a barrier of their own
    const int active = (n + 32 * PS_PER - 1) / (32 * PS_PER);
    auto meet = [&] { asm volatile("bar.sync 1, %0;" ::"r"(active * 32) : "memory"); };
    int total = 0;
    if (warp < active) {
        const int j0 = tid * PS_PER;                                     // 8 slots lie in one page
        const int page = j0 < n ? pages[j0 >> c.shift] : -1;
        const int64_t row = page < 0 ? 0 : slot_row(c, page, head, j0);
        // a slot behind a bad page id counts as the oldest, with no weight, and never moves
        uint32_t key[PS_PER];
        {
            int pos[PS_PER];
            float w[PS_PER];
#pragma unroll
            for (int i = 0; i < PS_PER; i += 4) {
                const int4 p4 = page < 0 ? make_int4(0, 0, 0, 0) : *reinterpret_cast<const int4*>(c.slot_pos + row + i);
                const float4 w4 = page < 0 ? make_float4(0.f, 0.f, 0.f, 0.f) : *reinterpret_cast<const float4*>(c.weight + row + i);
                pos[i] = p4.x, pos[i + 1] = p4.y, pos[i + 2] = p4.z, pos[i + 3] = p4.w;
                w[i] = w4.x, w[i + 1] = w4.y, w[i + 2] = w4.z, w[i + 3] = w4.w;
            }
            int latest = INT32_MIN;
#pragma unroll
            for (int i = 0; i < PS_PER; ++i)
                if (page >= 0 && j0 + i < n) latest = max(latest, pos[i]);
            latest = __reduce_max_sync(0xffffffffu, latest);
            if (lane == 0) red[0][warp] = latest;
            meet();
            for (int i = 0; i < active; ++i) latest = max(latest, red[0][i]);
            const int64_t after = static_cast<int64_t>(latest) - recent;
#pragma unroll
            for (int i = 0; i < PS_PER; ++i)
                key[i] = page < 0 || j0 + i >= n ? 0u : pos[i] > after ? 0xFFFFFFFFu : weight_key(w[i]);
        }
        // the budget-th largest key: the largest T with at least `budget` keys >= T. Where exactly that
        // many are, they are the kept ones and the search is over.
        uint32_t T = 0;
        int need = 0;                                                    // of the keys equal to T; 0: not known yet
        int side = 1, above = 0;
        auto count = [&](uint32_t bound) {                               // keys >= bound, of the block
            int v = 0;
#pragma unroll
            for (int i = 0; i < PS_PER; ++i) v += key[i] >= bound;
            v = __reduce_add_sync(0xffffffffu, v);
            if (lane == 0) red[side][warp] = v;
            meet();
            v = __reduce_add_sync(0xffffffffu, lane < active ? red[side][lane] : 0);
            side ^= 1;
            return v;
        };
        for (int bit = 31; bit >= 0; --bit) {
            const uint32_t bound = T | (1u << bit);
            const int v = count(bound);
            if (v >= budget) T = bound;
            if (v == budget) {
                need = PS_SLOTS;
                break;
            }
            if (v < budget) above = v;                                   // in the end: the keys > T
        }
        if (need == 0) need = budget - above;
        // kept: keys above T, and the first `need` of those equal to it
        auto scan = [&](int v, int& total) {                             // exclusive prefix over the block
            int x = v;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, x, o);
                if (lane >= o) x += y;
            }
            if (lane == 31) red[side][warp] = x;
            meet();
            const int other = lane < active ? red[side][lane] : 0;
            total = __reduce_add_sync(0xffffffffu, other);
            side ^= 1;
            return __reduce_add_sync(0xffffffffu, lane < warp ? other : 0) + x - v;
        };
        int ties = 0;
#pragma unroll
        for (int i = 0; i < PS_PER; ++i) ties += j0 + i < n && key[i] == T;
        int rank = scan(ties, total);
        int keep = 0, moves = 0;                                         // bits: kept; counts: holes, moved << 16
#pragma unroll
        for (int i = 0; i < PS_PER; ++i) {
            if (j0 + i >= n) continue;
            const bool tie = key[i] == T, k = key[i] > T || (tie && rank < need);
            rank += tie;
            keep |= k << i;
            if (j0 + i < budget) moves += !k;
            else moves += k << 16;
        }
        int at = scan(moves, total);
#pragma unroll
        for (int i = 0; i < PS_PER; ++i) {
            if (j0 + i >= n) continue;
            const bool k = keep >> i & 1;
            if (j0 + i < budget) {
                if (!k) to[at++ & 0xFFFF] = static_cast<uint16_t>(j0 + i);
            } else if (k) {
                from[at >> 16] = static_cast<uint16_t>(j0 + i);
                at += 1 << 16;
            }
        }
        if (tid == 0) moved_count = total & 0xFFFF;
    }
    __syncthreads();
    // 8 lanes a move, U moves at once. No slot is both read and written: what is given up lies
    // below the budget, what moves behind it.
    const int moved = moved_count, l = tid & 7;
    for (int i0 = tid >> 3; i0 < moved; i0 += U * (PS_T / 8)) {
        uint4 x[U][PL];
        uint32_t meta[U], other[U];
        int64_t dst[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + u * (PS_T / 8);
            dst[u] = -1;
            if (i >= moved) continue;
            const int sj = from[i], dj = to[i], sp = pages[sj >> c.shift], dp = pages[dj >> c.shift];
            if (sp < 0 || dp < 0) continue;
            const int64_t s = slot_row(c, sp, head, sj);
            dst[u] = slot_row(c, dp, head, dj);
#pragma unroll
            for (int k = 0; k < PL; ++k) {
                const int piece = l + k * 8;
                if (piece < KB / 8)
                    x[u][k] = *reinterpret_cast<const uint4*>((piece < KB / 16 ? c.kc : c.vc) + s * KB + piece % (KB / 16) * 16);
            }
            if (l < 2 * ng) meta[u] = (l < ng ? c.km : c.vm)[s * ng + (l < ng ? l : l - ng)];
            if (l == 6) other[u] = __float_as_uint(c.weight[s]);
            if (l == 7) other[u] = static_cast<uint32_t>(c.slot_pos[s]);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (dst[u] < 0) continue;
#pragma unroll
            for (int k = 0; k < PL; ++k) {
                const int piece = l + k * 8;
                if (piece < KB / 8)
                    *reinterpret_cast<uint4*>((piece < KB / 16 ? c.kc : c.vc) + dst[u] * KB + piece % (KB / 16) * 16) = x[u][k];
            }
            if (l < 2 * ng) (l < ng ? c.km : c.vm)[dst[u] * ng + (l < ng ? l : l - ng)] = meta[u];
            if (l == 6) c.weight[dst[u]] = __uint_as_float(other[u]);
            if (l == 7) c.slot_pos[dst[u]] = static_cast<int32_t>(other[u]);
        }
    }
}

// Workspace of one (sequence, head): the number of moves, then from[] and to[].
__device__ __forceinline__ int32_t* moves_of(int32_t* ws, int pair, int most) {
    return ws + static_cast<int64_t>(pair) * (4 + 2 * static_cast<int64_t>(most));
}

__device__ __forceinline__ int block_max(int v, int* red) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, o));
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    int m = red[0];
#pragma unroll
    for (int i = 1; i < PE_THREADS / 32; ++i) m = max(m, red[i]);
    __syncthreads();
    return m;
}

// Exclusive prefix of v over the block, and the total.
__device__ __forceinline__ int block_scan(int v, int* red, int& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) red[warp] = x;
    __syncthreads();
    int before = 0;
    total = 0;
#pragma unroll
    for (int i = 0; i < PE_THREADS / 32; ++i) {
        if (i < warp) before += red[i];
        total += red[i];
    }
    __syncthreads();
    return before + x - v;
}

__global__ void __launch_bounds__(PE_THREADS) evict_select_kernel(PagedView c, int budget, int recent, int most,
                                                                  int cached, int32_t* __restrict__ ws,
                                                                  int32_t* __restrict__ new_len) {
    extern __shared__ uint32_t keys[];                 // [cached], then the histogram
    __shared__ int red[PE_THREADS / 32];
    __shared__ int s_bin, s_above;
    uint32_t* hist = keys + cached;
    pdl_wait();
    pdl_trigger();
    const int head = blockIdx.x, b = blockIdx.y, tid = threadIdx.x;
    int32_t* list = moves_of(ws, b * c.heads + head, most);
    const int n = slots_of(c, b);
    if (head == 0 && tid == 0) new_len[b] = n < 0 ? __ldg(c.ctx_len + b) : min(n, budget);
    if (n <= budget) {
        if (tid == 0) list[0] = 0;
        return;
    }
    // A slot behind a bad page id counts as the oldest, with no weight, and never moves.
    auto row_of = [&](int j) {
        const int p = page_of(c, b, j);
        return p < 0 ? -1 : slot_row(c, p, head, j);
    };
    int latest = INT32_MIN;
    for (int j = tid; j < n; j += PE_THREADS) {
        const int r = row_of(j);
        if (r >= 0) latest = max(latest, c.slot_pos[r]);
    }
    latest = block_max(latest, red);
    const int64_t after = static_cast<int64_t>(latest) - recent;
    auto make_key = [&](int j) {
        const int r = row_of(j);
        if (r < 0) return 0u;
        return c.slot_pos[r] > after ? 0xFFFFFFFFu : weight_key(c.weight[r]);
    };
    for (int j = tid; j < min(n, cached); j += PE_THREADS) keys[j] = make_key(j);
    auto key_of = [&](int j) { return j < cached ? keys[j] : make_key(j); };
    __syncthreads();

    // the budget-th largest key, from its highest digit down
    uint32_t prefix = 0;
    int need = budget;                                  // among the keys that match the prefix
    int equal = 0;                                      // keys equal to it
#pragma unroll
    for (int d = 0; d < 3; ++d) {
        const int low = d == 0 ? 21 : d == 1 ? 10 : 0;
        const int bits = d == 2 ? 10 : 11;
        for (int i = tid; i < PE_BINS; i += PE_THREADS) hist[i] = 0;
        __syncthreads();
        for (int j = tid; j < n; j += PE_THREADS) {
            const uint32_t k = key_of(j);
            if (d == 0 || (k >> (low + bits)) == prefix) atomicAdd(&hist[(k >> low) & ((1u << bits) - 1u)], 1u);
        }
        __syncthreads();
        // thread t sums the bins that are the t-th from the top
        constexpr int PER = PE_BINS / PE_THREADS;
        const int top = PE_BINS - 1 - tid * PER;
        int sum = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i) sum += static_cast<int>(hist[top - i]);
        int total;
        int above = block_scan(sum, red, total);
        if (above < need && above + sum >= need) {
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const int h = static_cast<int>(hist[top - i]);
                if (above < need && above + h >= need) {
                    s_bin = top - i;
                    s_above = above;
                }
                above += h;
            }
        }
        __syncthreads();
        prefix = d == 0 ? static_cast<uint32_t>(s_bin) : (prefix << bits) | static_cast<uint32_t>(s_bin);
        need -= s_above;
        equal = static_cast<int>(hist[s_bin]);
        __syncthreads();
    }
    // kept: keys above `prefix`, and the first `need` of those equal to it
    int seen = 0, holes = 0, movers = 0;
    int32_t *from = list + 4, *to = list + 4 + most;
    for (int j0 = 0; j0 < n; j0 += PE_THREADS) {
        const int j = j0 + tid;
        const uint32_t k = j < n ? key_of(j) : 0u;
        bool keep = j < n && k > prefix;
        if (j < n && k == prefix && need == equal) keep = true;
        if (need != equal) {                            // the same for the whole block
            const bool tie = j < n && k == prefix;
            int total;
            const int rank = seen + block_scan(tie, red, total);
            if (tie && rank < need) keep = true;
            seen += total;
        }
        const bool hole = j < budget && !keep, mover = j >= budget && keep;
        int total;
        const int at = block_scan((hole ? 1 : 0) | (mover ? 1 << 16 : 0), red, total);
        if (hole) to[holes + (at & 0xFFFF)] = j;
        if (mover) from[movers + (at >> 16)] = j;
        holes += total & 0xFFFF;
        movers += total >> 16;
    }
    if (tid == 0) list[0] = holes;                      // as many as movers: budget slots are kept
}

// 8 lanes per moved slot. No slot is both read and written: holes lie below the budget,
// moved slots behind it.
__global__ void __launch_bounds__(256) evict_move_kernel(PagedView c, int most, const int32_t* __restrict__ ws, int kb,
                                                         int ng) {
    pdl_wait();
    pdl_trigger();
    const int pair = blockIdx.x, b = pair / c.heads, head = pair % c.heads;
    const int32_t* list = moves_of(const_cast<int32_t*>(ws), pair, most);
    const int count = list[0];
    const int lane = threadIdx.x & 7;
    for (int i = blockIdx.y * 32 + (threadIdx.x >> 3); i < count; i += gridDim.y * 32) {
        const int src = list[4 + i], dst = list[4 + most + i];
        const int sp = page_of(c, b, src), dp = page_of(c, b, dst);
        if (sp < 0 || dp < 0) continue;
        const int64_t s = slot_row(c, sp, head, src), d = slot_row(c, dp, head, dst);
        for (int w = lane; w < kb / 8; w += 8) {        // kb / 16 pieces of the key, then of the value
            uint8_t* pool = w < kb / 16 ? c.kc : c.vc;
            const int o = (w % (kb / 16)) * 16;
            *reinterpret_cast<uint4*>(pool + d * kb + o) = *reinterpret_cast<const uint4*>(pool + s * kb + o);
        }
        if (lane < ng)
            c.km[d * ng + lane] = c.km[s * ng + lane];
        else if (lane < 2 * ng)
            c.vm[d * ng + lane - ng] = c.vm[s * ng + lane - ng];
        if (lane == 6) c.weight[d] = c.weight[s];
        if (lane == 7) c.slot_pos[d] = c.slot_pos[s];
    }
}

// Moves of one (sequence, head): at most the budget, and at most what lies behind it.
int64_t evict_most(const flex_paged_cache* c, int budget) {
    const int64_t cap = static_cast<int64_t>(c->max_pages) * c->page_size;
    const int64_t behind = cap > budget ? cap - budget : 0;
    const int64_t m = behind < budget ? behind : budget;
    return (m + 3) / 4 * 4;
}

int64_t evict_ws_bytes(const flex_paged_cache* c, int budget) {
    return static_cast<int64_t>(c->batch) * c->n_kv_heads * (4 + 2 * evict_most(c, budget)) * 4;
}

}  // namespace
}  // namespace flexq

using namespace flexq;

extern "C" int64_t flex_paged_evict_ws_bytes(const flex_paged_cache* cache, int32_t budget) {
    const int rc = validate_paged(cache, true);
    if (rc != FLEX_OK) return rc;
    FLEX_REQUIRE(budget > 0, FLEX_ERR_INVALID_ARG);
    return evict_ws_bytes(cache, budget);
}

extern "C" int flex_paged_evict(const flex_paged_cache* cache, int32_t budget, int32_t recent, int32_t* new_len, void* ws,
                                int64_t ws_bytes, void* stream) {
    const int rc = validate_paged(cache, true);
    if (rc != FLEX_OK) return rc;
    FLEX_REQUIRE(cache->weight && cache->slot_pos && new_len, FLEX_ERR_INVALID_ARG);
    FLEX_REQUIRE(budget > 0 && recent >= 0 && recent <= budget, FLEX_ERR_INVALID_ARG);
    // every head reads ctx_len while new_len is written
    FLEX_REQUIRE(new_len + cache->batch <= cache->ctx_len || cache->ctx_len + cache->batch <= new_len,
                 FLEX_ERR_INVALID_ARG);
    FLEX_REQUIRE((reinterpret_cast<uintptr_t>(new_len) & 3u) == 0, FLEX_ERR_ALIGN);
    FLEX_REQUIRE(static_cast<int64_t>(cache->batch) * cache->n_kv_heads <= (1LL << 31) - 1, FLEX_ERR_UNSUPPORTED);
    FLEX_REQUIRE(ws != nullptr && ws_bytes >= evict_ws_bytes(cache, budget), FLEX_ERR_WORKSPACE);
    FLEX_REQUIRE(aligned16(ws), FLEX_ERR_ALIGN);
    const PagedView view = paged_view(cache);
    const cudaStream_t st = as_stream(stream);
    const int most = static_cast<int>(evict_most(cache, budget));
    const int cap = cache->max_pages * cache->page_size;
    if (cap <= PS_SLOTS) {
        const int kb = cache->head_dim * cache->cfg.num_bits / 8, ng = cache->head_dim / cache->cfg.group_size;
        const dim3 grid(cache->n_kv_heads, cache->batch);
#define SMALL(KB_, U_) launch_k(evict_small_kernel<KB_, U_>, grid, dim3(PS_T), 0, st, true, view, budget, recent, ng, new_len)
        // up to 64 moves a head (a cache a few tokens over its budget) are two rounds of one move a lane group
        if (most <= 64) {
            if (kb == 32) SMALL(32, 1); else if (kb == 64) SMALL(64, 1); else SMALL(128, 1);
        } else {
            if (kb == 32) SMALL(32, 4); else if (kb == 64) SMALL(64, 4); else SMALL(128, 4);
        }
#undef SMALL
        return launch_status();
    }
    const int cached = cap < PE_CACHE ? cap : PE_CACHE;
    const int smem = (cached + PE_BINS) * 4;
    set_smem_once(evict_select_kernel, (PE_CACHE + PE_BINS) * 4);
    launch_k(evict_select_kernel, dim3(cache->n_kv_heads, cache->batch), dim3(PE_THREADS), smem, st, true, view, budget,
             recent, most, cached, static_cast<int32_t*>(ws), new_len);
    if (most > 0) {
        // enough blocks for the longest list at 4 slots a lane group, no more than fill the device
        const int pairs = cache->batch * cache->n_kv_heads;
        int parts = (most + 127) / 128;
        const int fill = (16 * sm_count() + pairs - 1) / pairs;
        if (parts > fill) parts = fill;
        launch_k(evict_move_kernel, dim3(pairs, parts), dim3(256), 0, st, true, view, most,
                 static_cast<const int32_t*>(ws), cache->head_dim * cache->cfg.num_bits / 8,
                 cache->head_dim / cache->cfg.group_size);
    }
    return launch_status();
}
