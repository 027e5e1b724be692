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
// select: one block per (sequence, head). The keys (an order-preserving integer of the
// weight, the largest value for the recent slots) go to shared memory once, the
// budget-th largest is found digit by digit from histograms (11 + 11 + 10 bits), and one
// ordered pass lists what is given up and what moves. Weights and positions are read
// once (8 bytes a slot); the block's few synchronised passes over shared memory bound it.
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
    if (head == 0 && tid == 0) new_len[b] = min(n, budget);
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
