// attention.cuh: attention of new tokens over the paged cache on the tensor cores.
//
// Page "vllm.models.beam.nvidia.dflash2", DFlash2BeamAttention: the query block attends to keys
// and values in a paged cache, inside a sliding window. For a row (a new token and a query head)
// and its visible keys j:
//   s_j = scale <q, k_j> (capped), out = sum_j e^{s_j} v_j / sum_j e^{s_j}, lse = log sum_j e^{s_j}.
// One pass over the keys keeps a running maximum m, the sum l of e^{s_j - m} and the output O
// relative to m.
//
// Rows. The g = q_heads / kv_heads query heads of a key head share its keys, so a row tile is
// tpt = floor(128 / g) tokens x g heads of one request and key head: at most 128 rows, one
// tensor-memory lane each. A work item is two row tiles (2 tpt tokens) that walk the same key
// tiles of 128 tokens, or, where a request has no more than tpt tokens left, one row tile whose
// even and odd key tiles go to the two halves of the CTA.
//
// Few rows. Row tiles of at most 32 rows (single tokens, small blocks) would keep one softmax warp
// of each half busy and the others idle. They have a build of their own, with tpt = floor(32 / g)
// and one row tile an item. The queries go into all four quarters of the tile's lanes: S then has
// four copies, and each warp takes 32 of the 128 keys of every row. The warps agree on a row's
// maximum through shared memory, and P meets there too: it is the A operand from shared memory in
// place of tensor memory. S is free again once it is in registers, so the next scores are taken
// while the weights are.
//
// One CTA per SM, 16 warps (13-15 work for 8-bit caches only):
//   * warps 0 and 12: TMA producers, of keys (and queries) and of values. Each lane looks up one page
//     of a tile; the pages' boxes (a page's rows x 64 values, 128-byte swizzle) are issued one after
//     another by the warp together. Keys and values go through a ring of stages each. Two warps,
//     because a box takes some 60 ns to issue whatever its size, and a tile of 16-token pages has
//     16.
//   * warps 1 and 2, one for each half: issue the tcgen05.mma: S = Q K^T into tensor memory, and
//     O += P V with P in tensor memory (over S, in 16 bits) and V transposed by its descriptor.
//     Two warps, because the tensor cores idle through the waits of one (16001-token prompt: 810 us,
//     833 us with one).
//   * warp 3: walks the items of this CTA's range and hands them to the others through a ring in
//     shared memory; then looks through the value tiles that some row must not see all of, and
//     clears what is not finite there (0 x infinity would reach the rows that do not see it). See
//     Item::v_odd.
//   * warps 12-15, for 8-bit caches: widen tiles to fp16. With few rows they widen the keys, the
//     softmax warps the values, and warp 3 loads the values and scales bf16 queries to fp16.
//   * warps 4-7 and 8-11: one softmax each, a thread per row. S comes from tensor memory, P goes
//     back over it. O stays in tensor memory and is scaled there only when the row's maximum has
//     grown by more than 2^8 since it was last scaled; until then P is taken relative to the old
//     maximum, which changes nothing but the common factor of P, l and O. With few rows it is scaled
//     whenever the maximum has grown: the largest weight is a power of two then, which no rounding
//     changes.
// While one half's softmax runs, the tensor cores work for the other half.
//
// What bounds it. Single tokens and small blocks read each cached key and value once: 96 single
// tokens over 500 to 16000 (16-bit, 8 key heads of 128) take 285 us, 6.2 TB/s. From an 8-bit cache
// it is shared memory: per value a byte lands, is read, is written as two and read by the MMA (128
// tokens over 200 to 20000: 156 us, 3.7 TB/s). Long prompts are bound by the tensor cores and the
// softmax between two products (16001 tokens, 16 heads of 128, causal: 806 us, 1.3 PFLOP/s). A
// call's plan, launch and first loads take some 20 us (one token over 332, with the join skipped).
//
// Rounding. P is rounded to the type of V (fp16 over an 8-bit cache), since one MMA's operands have
// one type; S, m, l and O are fp32. fp16 weights are lifted by a power of two (weight_lift), so that
// many small ones still count. Where many keys weigh alike that adds as much error as the
// rounding of the output does; where few keys do, a largest weight that is exact keeps it smaller
// (two single tokens over 142 to 428, bf16: 1.3 times the output's rounding, 1.5 with the maximum
// left behind; 1% of the time).
//
// Work split. The flat list of (request, key head, item, key tile) is cut into one equal range
// per SM, wherever that falls. Every CTA takes the running cost over the requests itself (their
// lengths are a few bytes each) and finds its own range in it. An item cut by a range's end leaves
// (O, m, l) of its pieces in the workspace, and a joining kernel weighs them together. No CTA waits
// for another. Every mbarrier wait is bounded; one that runs out sets kStatusTimeout, its warp goes
// to the end of its item without further waits, and takes no other.
#pragma once

#include "common.cuh"
#include "ptx.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <mutex>

namespace dflash {

// A call of the tensor-core kernel.
struct AttentionProblem {
    int D, T, q_heads, kv_heads, g;
    int tpt, tpi;                       // tokens per row tile, per item
    int over;                           // an item's fixed cost, in its steps
    int whole;                          // key tiles up to which items are not worth cutting
    int R, max_pages, num_pages, page_size;
    int left, right;
    float softcap, scale, v_scale;      // scale includes the keys' scale
    const int32_t *block_table, *query_start, *kv_lens;
    int page_shift;
    void* out;
    float* lse;
    const void* value;
    long long page_stride, token_stride, head_stride;
    // workspace
    int4* bound;                        // [G + 1]: request, key head, item, first step
    float* part;                        // [2 G][part_floats]
    int G;
    bool join;                          // items may be cut
};

// The call with a 16-bit cache (attention_16bit.cu) and with an e4m3 cache (attention_e4m3.cu). few:
// the build for row tiles of few rows.
cudaError_t launch_attention_16bit(const DeviceInfo& dev, const AttentionArgs& a,
                                   const AttentionProblem& p, bool few, uint32_t* status,
                                   cudaStream_t stream);
cudaError_t launch_attention_e4m3(const DeviceInfo& dev, const AttentionArgs& a,
                                  const AttentionProblem& p, bool few, uint32_t* status,
                                  cudaStream_t stream);

namespace {

using namespace ptx;
using Problem = AttentionProblem;

constexpr unsigned kFull = 0xffffffffu;
constexpr int BM = 128;                 // rows of a row tile: tensor-memory lanes
constexpr int BN = 128;                 // keys of a key tile
constexpr int kThreads = 512;
constexpr int kJoinThreads = 256;
constexpr int kMaxRanges = 1024;
constexpr int kJoinSlices = 8;          // CTAs that share one cut item's join
constexpr int kFew = 32;                // rows of a tile that is copied to all quarters
constexpr int kItems = 4;               // slots of the item ring
constexpr int kSerialItems = 8;         // items of a request that one thread adds up
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kGrowth = 8.f;          // log2 growth of a maximum before O is scaled

// fp16 weights are taken times 2^lift: the largest is then 2^14 with few rows, 2^15 at most otherwise
// (by 2^kGrowth above a maximum left behind), and weights of 2^-38, or 2^-31, of it still count. (At
// 1, a key 18 above 20000 others would lose them all.) P, l and O have the factor in common; only
// the log-sum-exp takes it out. bf16 weights have fp32's range and none.
__host__ __device__ constexpr float weight_lift(bool half_weights, bool few_rows) {
    return !half_weights ? 0.f : (few_rows ? 14.f : 15.f - kGrowth);
}

__host__ __device__ inline size_t part_floats(int D) { return 2 * (size_t)BM * (D + 2); }

// The keys [first_key, keys_end) that the token at position pos of L sees (pos < 0 sees none to its
// left). No sum here leaves 32 bits: pos < L.
__device__ __forceinline__ int first_key(const Problem& p, int pos) {
    return p.left < 0 || pos <= p.left ? 0 : pos - p.left;
}
__device__ __forceinline__ int keys_end(const Problem& p, int L, int pos) {
    return p.right < 0 || p.right >= L - pos ? L : max(0, pos + p.right + 1);
}

// Key tiles [begin, end) that tokens tok0 .. tok0 + ntok - 1 of a request see any key of.
__device__ __forceinline__ void key_tiles(const Problem& p, int n, int L, int tok0, int ntok,
                                          int& begin, int& end) {
    const int first = L - n + tok0;
    const int lo = first_key(p, first), hi = keys_end(p, L, first + ntok - 1);
    begin = lo / BN;
    end = hi > lo ? (hi - 1) / BN + 1 : begin;
}

__device__ __forceinline__ int item_count(const Problem& p, int n) {
    return (n + p.tpi - 1) / p.tpi;
}

// Cost of an item in half steps of the two-tile kind, which is what the split makes equal.
__device__ __forceinline__ int step_cost(const Problem& p, int ntok) { return ntok > p.tpt ? 2 : 1; }

__device__ __forceinline__ int item_cost(const Problem& p, int n, int L, int t) {
    const int tok0 = t * p.tpi, ntok = min(p.tpi, n - tok0);
    int b, e;
    key_tiles(p, n, L, tok0, ntok, b, e);
    return step_cost(p, ntok) * (p.over + e - b);
}

// A request's new and cached tokens; n = 0 where query_start is refused, bad where kv_lens is.
struct Request {
    int t0, n, L;
    bool bad, rows_ok;
};

__device__ __forceinline__ Request request_of(const Problem& p, int r) {
    Request q;
    q.t0 = p.query_start[r];
    const int t1 = p.query_start[r + 1];
    q.L = p.kv_lens[r];
    q.rows_ok = q.t0 >= 0 && t1 >= q.t0 && t1 <= p.T;
    q.bad = q.L < 0 || (long long)q.L > (long long)p.max_pages * p.page_size;
    q.n = q.rows_ok ? t1 - q.t0 : 0;
    if (q.bad) q.L = 0;
    return q;
}

// ---------------------------------------------------------------- plan

// a / b for a >= 0, b > 0; a 64-bit division takes several times a 32-bit one.
__device__ __forceinline__ long long quotient(long long a, long long b) {
    return ((a | b) >> 32) == 0 ? (long long)((unsigned)a / (unsigned)b) : a / b;
}

// The start of range b of G: x = b W / G falls on a request, a key head, an item and a step of
// it; a start inside an item's last step moves to the next item. Called by a whole warp.
__device__ __forceinline__ int4 range_start(const Problem& p, const long long* cost, bool flat,
                                            int b) {
    const int lane = threadIdx.x & 31;
    const long long W = cost[p.R];
    const long long each = quotient(W, p.G);
    const long long x = each * b + quotient((W - each * p.G) * b, p.G);
    int4 at = make_int4(p.R, 0, 0, 0);
    if (x >= W) return at;
    int lo = 0, hi = p.R;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cost[mid] <= x) lo = mid;
        else hi = mid;
    }
    const Request q = request_of(p, lo);
    const int items = item_count(p, q.n);
    const long long head = quotient(cost[lo + 1] - cost[lo], p.kv_heads);
    const int h = (int)quotient(x - cost[lo], head);
    long long off = (x - cost[lo]) - (long long)h * head;
    if (flat) return make_int4(lo, h, (int)off, 0);
    for (int t0 = 0; t0 < items; t0 += 32) {
        const int t = t0 + lane;
        const int c = t < items ? item_cost(p, q.n, q.L, t) : 0;
        long long upto = c;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const long long o = __shfl_up_sync(kFull, upto, d);
            if (lane >= d) upto += o;
        }
        const unsigned past = __ballot_sync(kFull, upto > off);
        if (!past) {
            off -= __shfl_sync(kFull, upto, 31);
            continue;
        }
        const int k = __ffs(past) - 1;
        const int ck = __shfl_sync(kFull, c, k);
        off -= __shfl_sync(kFull, upto, k) - ck;
        const int tk = t0 + k;
        const int w = step_cost(p, min(p.tpi, q.n - tk * p.tpi));
        const int step = max(0, (w == 2 ? ((int)off + 1) >> 1 : (int)off) - p.over);
        at = make_int4(lo, h, tk, step);
        if (step * w >= ck - p.over * w && step > 0) {       // past the last step: the next item
            at.w = 0;
            if (++at.z == items) {
                at.z = 0;
                if (++at.y == p.kv_heads) {
                    at.y = 0;
                    do ++at.x;
                    while (at.x < p.R && request_of(p, at.x).n == 0);
                }
            }
        }
        break;
    }
    return at;
}

// Every thread of the CTA: the running cost over the requests in cost[R + 1] (shared memory),
// then this CTA's range. Where there are no more items than SMs and none is long, the cost of
// each is 1, so that ranges fall on whole items and nothing has to be joined.
__device__ __forceinline__ void plan_ranges(const Problem& p, long long* cost, int4* range,
                                            uint32_t* status) {
    __shared__ long long warp_sum[kThreads / 32], warp_items[kThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    long long my_items = 0;
    int first_items = 0;                 // of request tid
    bool big = false, is_long = false;
    for (int r = tid; r < p.R; r += kThreads) {
        const Request q = request_of(p, r);
        if (blockIdx.x == 0 && (q.bad || !q.rows_ok)) atomicOr(status, kStatusBadLength);
        const int items = item_count(p, q.n);
        my_items += items;
        if (r == tid) first_items = items;
        long long c = -1;                                    // left to a warp
        if (items <= kSerialItems) {
            c = 0;
            for (int t = 0; t < items; ++t) {
                const int k = item_cost(p, q.n, q.L, t);
                is_long |= k > p.over + p.whole;
                c += k;
            }
        } else {
            big = true;
        }
        cost[r] = c * (c < 0 ? 1 : p.kv_heads);
    }
    if (__syncthreads_or(big)) {
        for (int r = warp; r < p.R; r += kThreads / 32) {
            if (cost[r] >= 0) continue;
            const Request q = request_of(p, r);
            long long c = 0;
            for (int t = lane; t < item_count(p, q.n); t += 32) c += item_cost(p, q.n, q.L, t);
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) c += __shfl_xor_sync(kFull, c, d);
            if (lane == 0) cost[r] = c * p.kv_heads;
        }
        is_long = true;
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) my_items += __shfl_xor_sync(kFull, my_items, d);
    if (lane == 0) warp_items[warp] = my_items;
    bool flat = __syncthreads_or(is_long) == 0;
    if (flat) {
        long long all = 0;
        for (int w = 0; w < kThreads / 32; ++w) all += warp_items[w];
        flat = all * p.kv_heads <= p.G;
    }
    const int per = (p.R + kThreads - 1) / kThreads;
    const int r0 = min(tid * per, p.R), r1 = min(r0 + per, p.R);
    long long sum = 0;
    for (int r = r0; r < r1; ++r) {
        if (flat) {
            const int items = per == 1 ? first_items : item_count(p, request_of(p, r).n);
            cost[r] = (long long)items * p.kv_heads;
        }
        sum += cost[r];
    }
    long long incl = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long o = __shfl_up_sync(kFull, incl, d);
        if (lane >= d) incl += o;
    }
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    long long base = incl - sum;
    for (int w = 0; w < warp; ++w) base += warp_sum[w];
    for (int r = r0; r < r1; ++r) {
        const long long c = cost[r];
        cost[r] = base;
        base += c;
    }
    if (tid == kThreads - 1) cost[p.R] = base;
    __syncthreads();
    if (warp < 2) {
        const int b = (int)blockIdx.x + warp;
        const int4 at = range_start(p, cost, flat, b);
        if (lane == 0) {
            range[warp] = at;
            if (warp == 0 || b == p.G) p.bound[b] = at;      // for the join
        }
    }
    __syncthreads();
}

// ---------------------------------------------------------------- items of a range

// One item, or the part [lo, hi) of its steps that lies in this CTA's range.
struct __align__(16) Item {
    int r, h;            // request (-1: no more items) and key head
    int tok0, ntok;      // tokens of the request
    int t0, n, L, bad;   // the request's first row, new and cached tokens; refused
    int begin, steps;    // the item's first key tile, and their number
    int lo, hi;          // this CTA's steps
    int from, to;        // key tiles that every row of the item sees all of
    int v_odd;           // a value that is not finite was cleared
    int bad_page;        // some row sees a key in a page whose id lies outside the pool
    __device__ __forceinline__ bool pair(const Problem& p) const { return ntok > p.tpt; }
    __device__ __forceinline__ bool whole() const { return lo == 0 && hi == steps; }
};

// Key tiles that all of the tokens tok0 .. tok0 + ntok - 1 of a request see all of: [from, to).
// Others are masked row by row, and their values are looked through.
__device__ __forceinline__ void clear_tiles(const Problem& p, int n, int L, int tok0, int ntok,
                                            int& from, int& to) {
    const int first = L - n + tok0;
    from = (first_key(p, first + ntok - 1) + BN - 1) / BN;
    to = keys_end(p, L, first) / BN;
}

// Waits until the shared counter is past q. Gives up after kWaitLimitNs.
__device__ __forceinline__ bool count_past(const volatile uint32_t* count, uint32_t q) {
    if ((int32_t)(*count - q) > 0) return true;
    const unsigned long long t0 = globaltimer();
    while ((int32_t)(*count - q) <= 0) {
        if (globaltimer() - t0 > kWaitLimitNs) return false;
        __nanosleep(64);
    }
    return true;
}

template <int D, bool kSmall, bool kFewRows>
struct Layout {
    static constexpr int kReaders = kSmall ? 15 : 12;            // warps that wait for items
    static constexpr uint32_t kChunk = BN * 128;                 // 128 rows x 64 values
    static constexpr uint32_t kTile = kChunk * (D / 64);
    static constexpr uint32_t kRaw = BN * D;                     // a tile in 8 bits
    // Raw tiles of an 8-bit cache: one ring of keys and values; or, of few rows, one of keys and one
    // of values, which the softmax warps widen: their half has the tile to itself, and four warps
    // would take longer over keys and values than everything else (128 single tokens over 200 to
    // 20000: 226 us, 241 us by four warps).
    static constexpr bool kSpread = kSmall && kFewRows;
    static constexpr int kRawStages = kSmall ? (kSpread ? (D == 128 ? 2 : 4) : (D == 128 ? 2 : 8)) : 0;
    static constexpr int kRawV = kSpread ? (D == 128 ? 2 : 4) : 0;
    // Stages of keys and values.
    static constexpr int kK = kSmall ? (D == 128 ? (kSpread ? 1 : 2) : 3) : (D == 128 ? 2 : 5);
    static constexpr int kV = kSmall ? (D == 128 ? 2 : (kSpread ? 4 : 3)) : (D == 128 ? 3 : 5);
    static_assert(!kSpread || kV % 2 == 0, "within an item a half's stages are its own");
    // Two row tiles; or four copies of one of few rows, and behind them for each half P, 4 KB for 64
    // keys, and a row's maxima and sums. (The MMA reads on behind P for the lanes of no row.)
    static constexpr uint32_t q = 0;
    static constexpr uint32_t pKeys = kFew * 128, pShare = 2 * pKeys, pHalf = pShare + 2 * 4 * kFew * 4;
    static constexpr uint32_t p = kTile;
    static constexpr uint32_t keys = p + (kFewRows ? 2 * pHalf : kTile);
    static constexpr uint32_t values = keys + kK * kTile;
    static constexpr uint32_t raw = values + kV * kTile;
    static constexpr uint32_t bars = raw + (kRawStages + kRawV) * kRaw;
    static constexpr int kBars = 3 * kK + 4 * kV + 2 * kRawStages + 3 * kRawV + 20 + 2 * kItems;
    static constexpr uint32_t ml = (bars + kBars * 8 + 15) / 16 * 16;   // [128] float2
    static constexpr uint32_t undo = ml + BM * 8;                // [kItems][kFew] float
    static constexpr uint32_t items = undo + (kSpread ? kItems * kFew * 4 : 0);               // [kItems] Item
    static constexpr uint32_t slot = items + kItems * 64;        // tensor memory's base
    static constexpr uint32_t issued = slot + 4;                 // value tiles issued
    static constexpr uint32_t total = slot + 16;
    static_assert(bars - keys >= (kMaxTableRequests + 1) * 8, "the plan's running costs lie in the rings");
    static_assert(total + 1024 + 288 <= 232448, "a block's shared memory, with its alignment and the plan's own");
};

__device__ __forceinline__ uint32_t pack16(bool half_type, float lo, float hi) {
    if (half_type) {
        const __half2 v = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&v);
    }
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ float unpack16(bool half_type, uint32_t w) {
    return half_type ? __half2float(__ushort_as_half((unsigned short)w))
                     : __uint_as_float(w << 16);
}

// Bit per 16-bit half of w that is an infinity or a NaN.
template <bool kHalf>
__device__ __forceinline__ uint32_t odd_halves(uint32_t w) {
    constexpr uint32_t e = kHalf ? 0x7C00u : 0x7F80u;
    return ((w & e) == e ? 1u : 0u) | (((w >> 16) & e) == e ? 2u : 0u);
}

// Clears the infinities and NaNs of a value tile in shared memory; whether one of them was at a
// cached token (one of the first `cached` rows of the tile). By one warp.
template <int D, bool kHalf>
__device__ __forceinline__ bool clear_odd(uint8_t* tile, int lane, int cached) {
    constexpr int kVecs = (int)(Layout<D, false, false>::kTile / 16), kRun = 8;
    uint4* v = reinterpret_cast<uint4*>(tile);
    bool found = false;
    for (int i0 = lane; i0 < kVecs; i0 += 32 * kRun) {
        // x * 0 summed over a run of vectors is NaN if any value is not finite.
        uint4 x[kRun];
#pragma unroll
        for (int r = 0; r < kRun; ++r) x[r] = v[i0 + 32 * r];
        bool odd;
        if constexpr (kHalf) {
            const __half2 z = __float2half2_rn(0.f);
            __half2 a = z;
#pragma unroll
            for (int r = 0; r < kRun; ++r) {
                const __half2* e = reinterpret_cast<const __half2*>(&x[r]);
#pragma unroll
                for (int i = 0; i < 4; ++i) a = __hfma2(e[i], z, a);
            }
            odd = __hisnan(a.x) || __hisnan(a.y);
        } else {
            const __nv_bfloat162 z = __float2bfloat162_rn(0.f);
            __nv_bfloat162 a = z;
#pragma unroll
            for (int r = 0; r < kRun; ++r) {
                const __nv_bfloat162* e = reinterpret_cast<const __nv_bfloat162*>(&x[r]);
#pragma unroll
                for (int i = 0; i < 4; ++i) a = __hfma2(e[i], z, a);
            }
            odd = __hisnan(a.x) || __hisnan(a.y);
        }
        if (!odd) continue;
#pragma unroll 1
        for (int r = 0; r < kRun; ++r) {
            const int at = i0 + 32 * r;
            const uint4 y = v[at];
            uint32_t word[4] = {y.x, y.y, y.z, y.w};
            bool hit = false;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t bits = odd_halves<kHalf>(word[i]);
                hit |= bits != 0;
                word[i] &= (bits & 1 ? 0u : 0xFFFFu) | (bits & 2 ? 0u : 0xFFFF0000u);
            }
            if (!hit) continue;
            v[at] = make_uint4(word[0], word[1], word[2], word[3]);
            found |= (at * 16 % (int)Layout<D, false, false>::kChunk) / 128 < cached;
        }
    }
    return found;
}

// Add back to the columns d_begin .. d_end of a row's output (16-bit `out`, or fp32 `part` where
// out is null) the values that are not finite and that the row sees, of the tiles in which they
// have been cleared: weights are positive, so each gives an infinity of its sign or a NaN. By the
// thread that has written the row; taken only by items in which such a value was found.
template <bool kHalf, bool kSmall>
__device__ __noinline__ void refill_values(const Problem& p, const Item& c, int row_lo, int row_hi,
                                           int d_begin, int d_end, uint16_t* out, float* part) {
    for (int tile = c.begin + c.lo; tile < c.begin + c.hi; ++tile) {
        if (tile >= c.from && tile < c.to) continue;
        const int a = max(row_lo, tile * BN), b = min(row_hi - tile * BN, BN) + tile * BN;
        for (int j = a; j < b; ++j) {
            const int id = p.block_table[(long long)c.r * p.max_pages + (j >> p.page_shift)];
            if (id < 0 || id >= p.num_pages) continue;
            const long long at = id * p.page_stride + (j & (p.page_size - 1)) * p.token_stride +
                                 c.h * p.head_stride;
            for (int d = d_begin; d < d_end; ++d) {
                float v = 0.f;
                if constexpr (kSmall) {
                    const uint8_t x = static_cast<const uint8_t*>(p.value)[at + d];
                    if ((x & 0x7F) == 0x7F) v = NAN;
                } else {
                    const uint16_t x = static_cast<const uint16_t*>(p.value)[at + d];
                    if (odd_halves<kHalf>(x)) v = unpack16(kHalf, x);
                }
                if (v == 0.f) continue;
                if (out) {
                    out[d] = (uint16_t)pack16(kHalf, unpack16(kHalf, out[d]) + v, 0.f);
                } else {
                    part[(size_t)(d / 4) * BM * 4 + d % 4] += v;
                }
            }
        }
    }
}

// An id outside the pool for an item's keys tok .. tok + box - 1: recorded if some row sees one of
// them.
__device__ __noinline__ void note_bad_page(const Problem& p, Item& c, int tok, int box,
                                           uint32_t* status) {
    const int first = c.L - c.n + c.tok0;
    if (tok > first_key(p, first) - box && tok < keys_end(p, c.L, first + c.ntok - 1)) {
        c.bad_page = 1;
        atomicOr(status, kStatusBadId);
    }
}

// Whether a row that sees the keys [row_lo, row_hi) sees one, among this CTA's tiles of the item,
// in a page whose id lies outside the pool. Taken only by items that have met such a page.
__device__ __noinline__ bool sees_bad_page(const Problem& p, const Item& c, int row_lo, int row_hi) {
    const int start = (c.begin + c.lo) * BN;
    const int a = max(row_lo, start), b = min(row_hi - start, (c.hi - c.lo) * BN) + start;
    if (a >= b) return false;
    for (int page = a >> p.page_shift; page <= (b - 1) >> p.page_shift; ++page) {
        const int id = p.block_table[(long long)c.r * p.max_pages + page];
        if (id < 0 || id >= p.num_pages) return true;
    }
    return false;
}

// ---------------------------------------------------------------- 8-bit caches
//
// An e4m3 value is an fp16 value, so tiles of an 8-bit cache are widened to fp16 in shared memory,
// and queries of either type meet them as fp16. A bf16 query row is scaled by a power of two so
// that its largest value lies in [2^14, 2^15); what that pushes below fp16's smallest step is less
// than 2^-39 of the row's largest value. (The power stops at 2^100, so that its inverse is a normal
// number: rows below 2^-86 lose more.) The inverse goes into the row's score scale.

// This thread's row of a query tile (128-byte rows, 128-byte swizzle): bf16 to scaled fp16, in
// place and into the copies 32 rows on. Returns the factor that undoes the scaling.
template <int D, int kCopies>
__device__ __forceinline__ float widen_query_row(uint8_t* tile, int row) {
    constexpr uint32_t kChunk = BN * 128;
    uint32_t top = 0;                                        // largest |x| of each half, as bits
#pragma unroll
    for (int i = 0; i < D / 8; ++i) {
        const uint4 x = *reinterpret_cast<const uint4*>(tile + (i / 8) * kChunk + row * 128 +
                                                        ((i % 8) ^ (row & 7)) * 16);
        top = __vmaxu2(top, x.x & 0x7FFF7FFFu);
        top = __vmaxu2(top, x.y & 0x7FFF7FFFu);
        top = __vmaxu2(top, x.z & 0x7FFF7FFFu);
        top = __vmaxu2(top, x.w & 0x7FFF7FFFu);
    }
    const int e = (int)(max(top & 0xFFFFu, top >> 16) >> 7);   // biased exponent
    const int shift = (e == 0 || e == 255) ? 0 : min(141 - e, 100);
    const float by = __uint_as_float((uint32_t)(127 + shift) << 23);
#pragma unroll
    for (int i = 0; i < D / 8; ++i) {
        uint4* at = reinterpret_cast<uint4*>(tile + (i / 8) * kChunk + row * 128 +
                                             ((i % 8) ^ (row & 7)) * 16);
        uint4 x = *at;
        uint32_t* word = reinterpret_cast<uint32_t*>(&x);
#pragma unroll
        for (int k = 0; k < 4; ++k)
            word[k] = pack16(true, __uint_as_float(word[k] << 16) * by,
                             __uint_as_float(word[k] & 0xFFFF0000u) * by);
#pragma unroll
        for (int copy = 0; copy < kCopies; ++copy) at[copy * kFew * 128 / 16] = x;
    }
    return __uint_as_float((uint32_t)(127 - shift) << 23);
}

__device__ __forceinline__ uint32_t widen2(uint32_t two) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((unsigned short)two));
    return r;
}

// A raw tile (128 rows of D bytes) to fp16 in 128-byte rows with the 128-byte swizzle, by 128
// threads. With `look`, NaNs become 0; returns whether one was at a cached token.
template <int D>
__device__ __forceinline__ bool widen_tile(const uint8_t* raw, uint8_t* tile, int t, bool look,
                                           int cached) {
    constexpr uint32_t kChunk = BN * 128;
    constexpr int kAcross = D / 16, kDown = 128 / kAcross, kRounds = BN / kDown, kRun = 4;
    // Eight lanes that store together: at D = 128 they take the left halves of one row and the right
    // halves of its neighbour, whose pieces the swizzle puts into other banks.
    const int c = t % kAcross, row_t = (t / kAcross) ^ (D == 128 ? (t >> 2) & 1 : 0);
    const uint8_t* from = raw + row_t * D + c * 16;
    uint8_t* to = tile + (c / 4) * kChunk + row_t * 128;
    const int at0 = ((2 * c) % 8 ^ (row_t & 7)) * 16, at1 = ((2 * c + 1) % 8 ^ (row_t & 7)) * 16;
    bool found = false;
#pragma unroll
    for (int n0 = 0; n0 < kRounds; n0 += kRun) {
        uint4 x[kRun];
#pragma unroll
        for (int r = 0; r < kRun; ++r)
            x[r] = *reinterpret_cast<const uint4*>(from + (n0 + r) * kDown * D);
#pragma unroll
        for (int r = 0; r < kRun; ++r) {
            uint32_t* word = reinterpret_cast<uint32_t*>(&x[r]);
            if (look) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t odd = __vcmpeq4(word[i] & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
                    word[i] &= ~odd;
                    found |= odd != 0 && row_t + (n0 + r) * kDown < cached;
                }
            }
            uint4 y[2];
            uint32_t* wide = reinterpret_cast<uint32_t*>(y);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                wide[2 * i] = widen2(word[i] & 0xFFFFu);
                wide[2 * i + 1] = widen2(word[i] >> 16);
            }
            *reinterpret_cast<uint4*>(to + at0 + (n0 + r) * kDown * 128) = y[0];
            *reinterpret_cast<uint4*>(to + at1 + (n0 + r) * kDown * 128) = y[1];
        }
    }
    return found;
}

// The lowest n bits, for any n.
__device__ __forceinline__ uint32_t below(int n) {
    return n <= 0 ? 0u : (n >= 32 ? 0xFFFFFFFFu : (1u << n) - 1u);
}

// cap tanh(s / cap) = cap - 2 cap / (1 + e^(2 s / cap)), in log2 units; in = 2 log2(e) scale / cap.
// Two nearly equal numbers meet in it where s is small beside the cap, so it is off by up to 2^-21
// cap: taken for caps up to kQuickCap, where that is 3e-5, less than an fp32 dot product is sure of.
constexpr float kQuickCap = 64.f;
__device__ __forceinline__ uint32_t capped(uint32_t s, float in, float cap) {
    return __float_as_uint(fmaf(rcp(1.f + ex2(__uint_as_float(s) * in)), -2.f * cap, cap));
}

// The same for any cap, to 2^-19 of the result: below s / cap = 1/4 by tanh's series, whose next term
// is 2^-26 of it there. With y = s in, tanh's argument is y ln 2 / 2, and half the cap times y is
// the uncapped score.
__device__ __forceinline__ uint32_t capped_wide(uint32_t s, float in, float cap) {
    const float y = __uint_as_float(s) * in, x = y * (0.5f * kLn2), x2 = x * x;
    float t = fmaf(x2, 62.f / 2835.f, -17.f / 315.f);
    t = fmaf(x2, t, 2.f / 15.f);
    t = fmaf(x2, t, -1.f / 3.f);
    t = fmaf(x2, t, 1.f);
    const float low = y * (0.5f * kLn2 * cap) * t;
    const float high = fmaf(rcp(1.f + ex2(y)), -2.f * cap, cap);
    return __float_as_uint(fabsf(x) < 0.25f ? low : high);
}

// Builds without a cap, with one up to kQuickCap, and with any. (A branch between the two forms in
// one build costs windowed blocks with a cap of 50 8 us of 205.)
enum : int { kNoCap = 0, kQuick = 1, kWide = 2 };

// 16 columns of this thread's lane times `by`.
__device__ __forceinline__ void scale_columns(uint32_t taddr, float by) {
    uint32_t o[16];
    tmem_ld_issue_x16(taddr, o);
    tmem_ld_wait_x16(o);
#pragma unroll
    for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * by);
    tmem_st_x16(taddr, o);
}

// A 4 x 4 transpose of 16-byte pieces over groups of four lanes: before, lane l holds pieces 0..3
// of its row; after, piece l % 4 of the group's rows 0..3.
__device__ __forceinline__ void turn_pieces(uint32_t (&piece)[4][4], int lane) {
#pragma unroll
    for (int step = 1; step < 4; step <<= 1) {
        const bool up = (lane & step) != 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (i & step) continue;
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                // The upper lane gives its lower piece for the lower lane's upper one.
                const uint32_t give = up ? piece[i][x] : piece[i | step][x];
                const uint32_t take = __shfl_xor_sync(kFull, give, step);
                if (up) piece[i][x] = take;
                else piece[i | step][x] = take;
            }
        }
    }
}

template <int D, bool kHalf, int kCap, bool kSmall, bool kFewRows>
__global__ void __launch_bounds__(kThreads, 1)
attention_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                 const __grid_constant__ CUtensorMap map_v, const __grid_constant__ Problem p,
                 uint32_t* status) {
    using L = Layout<D, kSmall, kFewRows>;
    constexpr bool kMmaHalf = kHalf || kSmall;               // the tensor cores' operands are fp16
    constexpr bool kScaleQ = kSmall && !kHalf;               // bf16 queries are scaled to fp16
    constexpr int kChunks = kSmall ? 1 : D / 64;             // boxes across a row
    constexpr uint32_t kK = L::kK, kV = L::kV;
    constexpr bool kSpread = L::kSpread;                     // the softmax warps widen the values
    constexpr float kLift = weight_lift(kMmaHalf, kFewRows);
    extern __shared__ uint8_t smem_raw[];
    __shared__ int4 range[2];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const uint32_t base = smem_u32(smem);
    const uint32_t bars = base + L::bars;
    // Two barriers a stage for its landings, for its uses by turns: a half that skips the other
    // half's tiles may look at a barrier before the use in front of the one it wants has landed,
    // never before the one in front of that (the tile it used last was issued after that one had
    // been freed), so with two the parity cannot be mistaken.
    const uint32_t k_full = bars, k_empty = k_full + 16 * kK;            // [2 kK], [kK]
    const uint32_t v_full = k_empty + 8 * kK, v_empty = v_full + 16 * kV;   // [2 kV], [kV]
    const uint32_t v_fix = v_empty + 8 * kV;                             // [kV]
    const uint32_t q_full = v_fix + 8 * kV, q_empty = q_full + 8;
    // by half: S there, P of the upper and of the lower 64 keys there, O has the tile
    const uint32_t s_full = q_full + 16, p_up = q_full + 32, p_low = q_full + 48;
    const uint32_t o_done = q_full + 64;
    const uint32_t ml_there = q_full + 80, ml_back = q_full + 88, halves_done = q_full + 96;
    const uint32_t drained = q_full + 104, q_ready = q_full + 120;   // drained: [2]
    const uint32_t s_read = q_full + 128, share = q_full + 144;          // by half
    const uint32_t item_full = q_full + 160, item_empty = item_full + 8 * kItems;
    const uint32_t raw_full = item_empty + 8 * kItems, raw_empty = raw_full + 8 * L::kRawStages;
    const uint32_t rv_full = raw_empty + 8 * L::kRawStages, rv_empty = rv_full + 16 * L::kRawV;   // [2 kRawV]
    float2* ml = reinterpret_cast<float2*>(smem + L::ml);
    float* undo_of = reinterpret_cast<float*>(smem + L::undo);
    Item* items = reinterpret_cast<Item*>(smem + L::items);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::slot);
    volatile uint32_t* issued = reinterpret_cast<volatile uint32_t*>(smem + L::issued);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        // Landings: the producer, or the four widening warps. Releases: both halves' warps.
        for (uint32_t s = 0; s < 2 * kK; ++s) mbar_init(k_full + 8 * s, kSmall ? 4 : 1);
        for (uint32_t s = 0; s < 2 * kV; ++s) mbar_init(v_full + 8 * s, kSmall ? 4 : 1);
        for (uint32_t s = 0; s < kK; ++s) mbar_init(k_empty + 8 * s, kFewRows ? 1 : 2);
        for (uint32_t s = 0; s < kV; ++s) {
            mbar_init(v_empty + 8 * s, kFewRows ? 1 : 2);
            mbar_init(v_fix + 8 * s, 1);
        }
        mbar_init(q_full, 1);
        mbar_init(q_empty, 2);
        for (int w = 0; w < 2; ++w) {
            mbar_init(s_full + 8 * w, 1);
            mbar_init(p_up + 8 * w, 4);          // warps
            mbar_init(p_low + 8 * w, 4);
            mbar_init(o_done + 8 * w, 1);
        }
        mbar_init(ml_there, 4);
        mbar_init(ml_back, 4);
        mbar_init(halves_done, 8);
        mbar_init(drained, 1);
        mbar_init(drained + 8, 1);
        mbar_init(q_ready, kFewRows ? 1 : 8);
        for (int i = 0; i < 2; ++i) {
            mbar_init(s_read + 8 * i, 4);
            mbar_init(share + 8 * i, 4);
        }
        for (int s = 0; s < L::kRawStages; ++s) {
            mbar_init(raw_full + 8 * s, 1);
            mbar_init(raw_empty + 8 * s, 4);
        }
        for (int s = 0; s < 2 * L::kRawV; ++s) mbar_init(rv_full + 8 * s, 1);
        for (int s = 0; s < L::kRawV; ++s) mbar_init(rv_empty + 8 * s, 4);
        for (int i = 0; i < kItems; ++i) {
            mbar_init(item_full + 8 * i, 1);
            mbar_init(item_empty + 8 * i, L::kReaders);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        *issued = 0;
        asm volatile("prefetch.tensormap [%0];" ::"l"(&map_q) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(&map_k) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(&map_v) : "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(tmem_slot)), "r"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    grid_dependents_launch();
    // The running costs use the ring's memory before the first tile does.
    plan_ranges(p, reinterpret_cast<long long*>(smem + L::keys), range, status);
    // Generic writes to the ring come before the first asynchronous ones.
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    uint32_t tries = kWaitTries;         // 0 once a wait of this thread has run out
    auto wait = [&](uint32_t bar, uint32_t parity) { mbar_wait_tries(bar, parity, tries); };
    bool ok = true;                      // no wait of this warp has run out, as of its last item

    // Item k of the range lies in slot k % kItems. get_item waits for it; done_with frees it, by
    // one lane of each reading warp.
    uint32_t k = 0;
    auto get_item = [&]() -> const Item* {
        const uint32_t s = k % kItems;
        wait(item_full + 8 * s, (k / kItems) & 1);
        ok = __all_sync(kFull, tries != 0);
        return ok && items[s].r >= 0 ? &items[s] : nullptr;
    };
    auto done_with = [&]() {
        __syncwarp();
        if (lane == 0) mbar_arrive(item_empty + 8 * (k % kItems));
        ++k;
    };

    // One tile of keys or values of this range: tile g of its ring. `id`: this lane's page, -1 behind
    // the last token.
    auto issue_tile = [&](const CUtensorMap* map, uint32_t to, uint32_t full, int h, int row0, int id) {
        const int box = min(p.page_size, BN);
        const int n = __popc(__ballot_sync(kFull, id >= 0));
        if (lane == 0) mbar_expect_tx(full, (uint32_t)(n * box * D * (kSmall ? 1 : 2)));
        __syncwarp();
        int next = __shfl_sync(kFull, id, 0);
#pragma unroll 1
        for (int i = 0; i < n; ++i, to += box * (kSmall ? D : 128)) {
            const int page = next;
            next = __shfl_sync(kFull, id, i + 1);
#pragma unroll
            for (int x = 0; x < kChunks; ++x)
                tma_load_4d_warp(to + x * L::kChunk, map, full, x * 64, row0, h, page);
        }
    };
    // This lane's page of an item's tile: -1 behind the last token. Ids outside the pool are not
    // followed: page 0 takes their place, and rows that see a key there become NaN. Where no row
    // does (a window has left the page, and it may have been given back), nothing is wrong.
    auto page_of = [&](const Item* c, int step) -> int {
        const int box = min(p.page_size, BN);
        const unsigned tok = (unsigned)(c->begin + step) * BN + lane * box;
        if (lane >= BN / box || step >= c->hi || tok >= (unsigned)c->L) return -1;
        int id = p.block_table[(long long)c->r * p.max_pages + (tok >> p.page_shift)];
        if (id < 0 || id >= p.num_pages) {
            note_bad_page(p, items[k % kItems], (int)tok, box, status);
            id = 0;
        }
        return id;
    };
    auto row_of = [&](const Item* c, int step) {             // of its page, where the tile begins
        return ((c->begin + step) * BN) & (p.page_size - 1);
    };

    // Registers: the block is launched with 128 a thread, 512 for threads of the four warpgroups;
    // the softmax threads, which hold half a row of S, take 184 each, the others keep 72.
    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        if (warp == 0) {
            // ---- TMA producer of queries and keys; of an 8-bit cache's raw tiles, keys and values
            uint32_t g = 0, nq = 0;      // tiles issued, items with steps
            auto free_stage = [&](uint32_t empty, uint32_t n) {
                if (g >= n) wait(empty + 8 * (g % n), (g / n - 1) & 1);
                return ok = __all_sync(kFull, tries != 0);
            };
            while (const Item* c = get_item()) {
                const int lo = c->lo, hi = c->hi, h = c->h;
                if (lo < hi) {
                    if (nq > 0) wait(q_empty, (nq - 1) & 1);
                    if (!(ok = __all_sync(kFull, tries != 0))) break;
                    ++nq;
                    const bool pair = c->pair(p);
                    if (lane == 0) {
                        const int tiles = kFewRows ? (kScaleQ ? 1 : 4) : (pair ? 2 : 1);   // (copies follow)
                        constexpr uint32_t apart = kFewRows ? kFew * 128 : L::kTile;
                        mbar_expect_tx(q_full, (uint32_t)(tiles * p.g * p.tpt) * D * 2);
                        for (int s = 0; s < tiles; ++s)
                            for (int i = 0; i < D / 64; ++i)
                                tma_load_4d(base + L::q + s * apart + i * L::kChunk, &map_q, q_full,
                                            i * 64, 0, h, c->t0 + c->tok0 + (pair ? s * p.tpt : 0));
                    }
                    __syncwarp();
                    if constexpr (kSmall) {
                        // K_0, K_1, V_0, K_2, V_1, ..., K_n-1, V_n-2, V_n-1; with few rows warp 3 loads
                        // the values
                        constexpr uint32_t n = L::kRawStages;
                        auto load = [&](const CUtensorMap* map, int step, int id) {
                            if (!free_stage(raw_empty, n)) return;
                            issue_tile(map, base + L::raw + (g % n) * L::kRaw, raw_full + 8 * (g % n),
                                       h, row_of(c, step), id);
                            ++g;
                        };
                        int id = page_of(c, lo), id_next = page_of(c, lo + 1);
                        load(&map_k, lo, id);
                        for (int j = lo; j < hi && ok; ++j) {
                            const int id_after = page_of(c, j + 2);
                            if (j + 1 < hi) load(&map_k, j + 1, id_next);
                            if (!kSpread && ok) load(&map_v, j, id);
                            id = id_next;
                            id_next = id_after;
                        }
                    } else {
                        int id = page_of(c, lo);
                        for (int j = lo; j < hi; ++j, ++g) {
                            const int id_next = page_of(c, j + 1);
                            if (!free_stage(k_empty, kK)) break;
                            issue_tile(&map_k, base + L::keys + (g % kK) * L::kTile,
                                       k_full + 8 * (g % (2 * kK)), h, row_of(c, j), id);
                            id = id_next;
                        }
                    }
                }
                if (!ok) break;
                done_with();
            }
            if (!ok && lane == 0) atomicOr(status, kStatusTimeout);
            // The last loads land before this CTA leaves, whatever has become of those who use them.
            constexpr uint32_t n = kSmall ? L::kRawStages : kK;
            for (uint32_t t = g > n ? g - n : 0; t < g; ++t)
                (void)(kSmall ? mbar_wait(raw_full + 8 * (t % n), (t / n) & 1)
                              : mbar_wait(k_full + 8 * (t % (2 * n)), (t / (2 * n)) & 1));
            if (nq > 0) (void)mbar_wait(q_full, (nq - 1) & 1);
        } else if (warp <= 2) {
            // ---- MMA issuer of half w: the warp together, an elected lane issues
            const int w = warp - 1;
            const uint32_t idesc_s = f16_idesc_of(kMmaHalf, false, BM, BN);
            const uint32_t idesc_o = f16_idesc_of(kMmaHalf, true, BM, D);
            const uint32_t ubase = __shfl_sync(kFull, base, 0), utmem = __shfl_sync(kFull, tmem, 0);
            const uint64_t dq = sw128_desc(ubase + L::q), dk = sw128_desc(ubase + L::keys);
            const uint64_t dv = sw128_mn_desc(ubase + L::values, L::kChunk);
            const uint64_t dp = sw128_desc(ubase + L::p + w * L::pHalf);
            const uint32_t acc = utmem + 256 + w * 128, st = utmem + w * BN, pt = st + 64;
            uint32_t g = 0, nq = 0;      // steps of earlier items; items with steps
            uint32_t np = 0;             // P tiles waited for
            uint32_t fixed = 0;          // phase bit of each stage's v_fix
            while (const Item* c = get_item()) {
                const int steps = __shfl_sync(kFull, c->hi - c->lo, 0);
                if (steps > 0) {
                    const bool pair =
                        !kFewRows && __shfl_sync(kFull, c->pair(p) ? 1 : 0, 0) != 0;
                    // Steps whose values need no look.
                    const int from = __shfl_sync(kFull, c->from - c->begin - c->lo, 0);
                    const int to = __shfl_sync(kFull, c->to - c->begin - c->lo, 0);
                    auto k_landed = [&](int j) {
                        wait(k_full + 8 * ((g + j) % (2 * kK)), ((g + j) / (2 * kK)) & 1);
                    };
                    // A tile of a pair is freed by both halves, another by its half alone.
                    auto release = [&](uint32_t empty) {
                        umma_commit_warp(empty);
                        if (!kFewRows && !pair) umma_commit_warp(empty);
                    };
                    const int stride = pair ? 1 : 2, j0 = pair ? 0 : w;
                    auto scores = [&](int j) {               // S of step j; its keys have landed
                        const uint32_t s = (g + j) % kK;
                        const uint64_t a = dq + (pair ? w : 0) * (L::kTile >> 4);
                        const uint64_t b = dk + s * (L::kTile >> 4);
                        tc_fence_after();
#pragma unroll
                        for (int i = 0; i < D / 16; ++i) {
                            const uint32_t o = ((i / 4) * L::kChunk + (i % 4) * 32) >> 4;
                            umma_f16_warp(st, a + o, b + o, idesc_s, i != 0);
                        }
                        umma_commit_warp(s_full + 8 * w);
                        release(k_empty + 8 * s);
                        if (j + stride >= steps) umma_commit_warp(q_empty);
                    };
                    wait(kScaleQ ? q_ready : q_full, nq & 1);
                    ++nq;
                    if (j0 < steps) {
                        k_landed(j0);
                        scores(j0);
                    } else if (lane == 0) {
                        mbar_arrive(q_empty);
                    }
#pragma unroll 1
                    for (int j = 0; j < steps; ++j) {
                        const uint32_t t = g + j, s = t % kV;
                        const bool mine = pair || (j & 1) == w;
                        const bool look = !kSmall && !(j >= from && j < to);
                        if (mine) {
                            const int next = j + stride;
                            const uint64_t b = dv + s * (L::kTile >> 4);
                            const uint32_t more = j != j0;
                            if constexpr (kFewRows) {
                                // The next scores start once these are in the softmax's registers.
                                if (next < steps) {
                                    k_landed(next);
                                    wait(s_read + 8 * w, np & 1);
                                    scores(next);
                                }
                            }
                            // The values have landed, and been looked through where they must be.
                            wait(v_full + 8 * (t % (2 * kV)), (t / (2 * kV)) & 1);
                            if (look) wait(v_fix + 8 * s, (fixed >> s) & 1);
                            wait(p_up + 8 * w, np & 1);
                            tc_fence_after();
                            if constexpr (kFewRows) {
#pragma unroll
                                for (int x = 0; x < 8; ++x)
                                    umma_f16_warp(acc, dp + (((x / 4) * L::pKeys + (x % 4) * 32) >> 4),
                                                  b + x * (2048 >> 4), idesc_o, x > 0 ? 1u : more);
                            } else {
#pragma unroll
                                for (int x = 4; x < 8; ++x)
                                    umma_f16_tmem_a_warp(acc, pt + x * 8, b + x * (2048 >> 4), idesc_o,
                                                         x > 4 ? 1u : more);
                                if (next < steps) k_landed(next);
                                wait(p_low + 8 * w, np & 1);
                                tc_fence_after();
#pragma unroll
                                for (int x = 0; x < 4; ++x)
                                    umma_f16_tmem_a_warp(acc, pt + x * 8, b + x * (2048 >> 4), idesc_o,
                                                         1u);
                            }
                            ++np;
                            umma_commit_warp(o_done + 8 * w);
                            release(v_empty + 8 * s);
                            if (!kFewRows && next < steps) scores(next);
                        }
                        if (look) fixed ^= 1u << s;
                    }
                    g += steps;
                }
                done_with();
            }
            if (!ok && lane == 0) atomicOr(status, kStatusTimeout);
            umma_commit_warp(drained + 8 * w);       // all MMAs and arrivals end before the CTA does
            (void)mbar_wait(drained + 8 * w, 0);
        } else {
            // ---- the items of this CTA's range, and the look through their value tiles. Items are
            // handed out two ahead of the one whose tiles are looked through.
            int4 at = range[0];
            const int4 end = range[1];
            int loaded = -1;
            Request q = {};
            bool over = false;
            auto hand_out = [&](uint32_t n) {
                const uint32_t s = n % kItems;
                if (n >= kItems) wait(item_empty + 8 * s, (n / kItems - 1) & 1);
                const bool last = at.x == end.x && at.y == end.y && at.z == end.z;
                over = at.x >= p.R || (last && at.w >= end.w);
                if (!over && at.x != loaded) {
                    q = request_of(p, at.x);
                    loaded = at.x;
                }
                if (lane == 0) {
                    Item& c = items[s];
                    c.r = over ? -1 : at.x;
                    if (!over) {
                        c.h = at.y;
                        c.tok0 = at.z * p.tpi;
                        c.ntok = min(p.tpi, q.n - c.tok0);
                        c.t0 = q.t0;
                        c.n = q.n;
                        c.L = q.L;
                        c.bad = q.bad;
                        int b, e, from, to;
                        key_tiles(p, q.n, q.L, c.tok0, c.ntok, b, e);
                        clear_tiles(p, q.n, q.L, c.tok0, c.ntok, from, to);
                        c.begin = b;
                        c.steps = e - b;
                        c.lo = at.w;
                        c.hi = last ? end.w : e - b;
                        c.from = from;
                        c.to = to;
                        c.v_odd = 0;
                        c.bad_page = 0;
                    }
                }
                mbar_arrive_warp(item_full + 8 * s);
                if (last) {
                    at = end;
                } else if (!over) {
                    at.w = 0;
                    if (++at.z == item_count(p, q.n)) {
                        at.z = 0;
                        if (++at.y == p.kv_heads) {
                            at.y = 0;
                            do ++at.x;
                            while (at.x < p.R && request_of(p, at.x).n == 0);
                        }
                    }
                }
            };
            uint32_t handed = 0, g = 0, nq = 0;
            for (;; ++k) {
                while (!over && handed < k + 3) hand_out(handed++);
                const Item* c = &items[k % kItems];
                if (c->r < 0 || !__all_sync(kFull, tries != 0)) break;
                const int steps = c->hi - c->lo;
                if constexpr (kScaleQ && kFewRows) {
                    // The queries, which are few. (By the softmax warps the scores of an item could
                    // not begin before the item in front of it has ended: 30 us of 226.)
                    if (steps > 0) {
                        wait(q_full, nq++ & 1);
                        undo_of[(k % kItems) * kFew + lane] = widen_query_row<D, 4>(smem + L::q, lane);
                        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                        mbar_arrive_warp(q_ready);
                    }
                }
                if constexpr (kSpread) {
                    // The raw value tiles, as warp 12 loads those of 16-bit caches (pages of 64
                    // tokens 183 us, 187 us by the warp that loads the keys; of 16, 192 and 239).
                    constexpr uint32_t n = L::kRawV;
                    int id = steps > 0 ? page_of(c, c->lo) : -1;
                    for (int j = c->lo; j < c->hi; ++j, ++g) {
                        const int id_next = page_of(c, j + 1);
                        if (g >= n) wait(rv_empty + 8 * (g % n), (g / n - 1) & 1);
                        if (!__all_sync(kFull, tries != 0)) break;
                        issue_tile(&map_v, base + L::raw + (L::kRawStages + g % n) * L::kRaw,
                                   rv_full + 8 * (g % (2 * n)), c->h, row_of(c, j), id);
                        id = id_next;
                    }
                } else if constexpr (!kSmall) {
                    for (int j = 0; j < steps; ++j) {
                        const int tile = c->begin + c->lo + j;
                        if (tile >= c->from && tile < c->to) continue;
                        const uint32_t t = g + j, s = t % kV;
                        // This warp may be any number of tiles ahead: only once the tile is issued does a
                        // parity say which use has landed.
                        if (!__all_sync(kFull, count_past(issued, t))) tries = 0;
                        wait(v_full + 8 * (t % (2 * kV)), (t / (2 * kV)) & 1);
                        if (clear_odd<D, kMmaHalf>(smem + L::values + s * L::kTile, lane, c->L - tile * BN))
                            items[k % kItems].v_odd = 1;
                        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                        mbar_arrive_warp(v_fix + 8 * s);
                    }
                    g += max(steps, 0);
                }
            }
            if (!__all_sync(kFull, tries != 0) && lane == 0) atomicOr(status, kStatusTimeout);
            if constexpr (kSpread) {                         // the last loads land
                constexpr uint32_t n = L::kRawV;
                for (uint32_t t = g > n ? g - n : 0; t < g; ++t)
                    (void)mbar_wait(rv_full + 8 * (t % (2 * n)), (t / (2 * n)) & 1);
            }
        }
    } else if (warp >= 12) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        if constexpr (kSmall) {
            // ---- 8-bit tiles to fp16
            const int t = threadIdx.x - 384;
            uint32_t g = 0, raw = 0;     // steps of earlier items; raw tiles taken
            while (const Item* c = get_item()) {
                const int steps = max(c->hi - c->lo, 0);
                for (int i = 0; i < (kSpread ? 1 : 2) * steps; ++i, ++raw) {
                    // K_0, K_1, V_0, K_2, V_1, ..., K_n-1, V_n-2, V_n-1
                    const bool value = !kSpread && (i == 2 * steps - 1 || (i > 0 && (i & 1) == 0));
                    const int j = kSpread ? i : (value ? (i - 1) / 2 : (i + 1) / 2);
                    const int tile = c->begin + c->lo + j;
                    const bool look = value && !(tile >= c->from && tile < c->to);
                    const uint32_t n = value ? kV : kK, u = g + j, r = raw % L::kRawStages;
                    wait(raw_full + 8 * r, (raw / L::kRawStages) & 1);
                    if (u >= n) wait((value ? v_empty : k_empty) + 8 * (u % n), (u / n - 1) & 1);
                    uint8_t* to = smem + (value ? L::values : L::keys) + (u % n) * L::kTile;
                    if (widen_tile<D>(smem + L::raw + r * L::kRaw, to, t, look, c->L - tile * BN))
                        items[k % kItems].v_odd = 1;
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    mbar_arrive_warp(raw_empty + 8 * r);
                    mbar_arrive_warp((value ? v_full : k_full) + 8 * (u % (2 * n)));
                }
                g += steps;
                done_with();
            }
            if (!ok && lane == 0) atomicOr(status, kStatusTimeout);
        } else if (warp == 12) {
            // ---- TMA producer of values
            uint32_t g = 0;
            while (const Item* c = get_item()) {
                const int hi = c->hi, h = c->h;
                int id = page_of(c, c->lo);
                for (int j = c->lo; j < hi; ++j, ++g) {
                    const int id_next = page_of(c, j + 1);
                    if (g >= kV) wait(v_empty + 8 * (g % kV), (g / kV - 1) & 1);
                    if (!(ok = __all_sync(kFull, tries != 0))) break;
                    if (lane == 0) *issued = g + 1;
                    issue_tile(&map_v, base + L::values + (g % kV) * L::kTile,
                               v_full + 8 * (g % (2 * kV)), h, row_of(c, j), id);
                    id = id_next;
                }
                if (!ok) break;
                done_with();
            }
            if (!ok && lane == 0) atomicOr(status, kStatusTimeout);
            for (uint32_t t = g > kV ? g - kV : 0; t < g; ++t)
                (void)mbar_wait(v_full + 8 * (t % (2 * kV)), (t / (2 * kV)) & 1);
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
        // ---- softmax: thread = row = tensor-memory lane
        const int w = (warp - 4) >> 2;                       // half
        const int row = (warp & 3) * 32 + lane;
        const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t ts = lane_base + w * BN;
        const uint32_t to_ = lane_base + 256 + w * 128;
        const int quarter = warp & 3;
        const float cap = p.softcap * kLog2e;
        // S tiles of this half; items of one row tile, with steps; times that few rows were shared
        uint32_t ns = 0, nb = 0, nq = 0, nshare = 0;
        uint32_t g = 0;                                      // steps of earlier items
        bool both = false;                                   // halves_done is still to be waited for
        auto settle = [&]() {
            if (both) wait(halves_done, (nb - 1) & 1);
            both = false;
        };
        while (const Item* c = get_item()) {
            const int steps = c->hi - c->lo;
            const bool pair = !kFewRows && c->pair(p);
            const int sub0 = c->tok0 + (pair ? w : 0) * p.tpt;   // the row tile's first token
            const int nsub = min(p.tpt, c->n - sub0);            // and its tokens
            const int row_token = (kFewRows ? lane : row) / p.g;
            bool live = row_token < nsub;
            const int pos = c->L - c->n + sub0 + row_token;
            const int row_lo = first_key(p, pos);
            const int row_hi = live ? keys_end(p, c->L, pos) : 0;
            bool warp_live = __any_sync(kFull, live);
            const int first = c->begin + c->lo;
            int from, to;
            clear_tiles(p, c->n, c->L, sub0, nsub, from, to);
            from -= first;
            to -= first;
            float unit = kCap ? 1.f : p.scale * kLog2e;      // S to log2 of a weight
            float cap_in = kCap ? 2.f * kLog2e * p.scale / p.softcap : 0.f;
            if constexpr (kScaleQ && !kFewRows) {
                // Half w scales the row tile it will read the scores of; one row tile is half 0's,
                // which leaves the factors for half 1.
                if (steps > 0) {
                    wait(q_full, nq++ & 1);
                    settle();                            // the factors there have been read
                    if (pair || w == 0) {
                        const float undo = widen_query_row<D, 1>(smem + L::q + w * L::kTile, row);
                        if (!pair) ml[row].x = undo;
                        if (kCap) cap_in *= undo;
                        else unit *= undo;
                        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    }
                    mbar_arrive_warp(q_ready);
                }
            }
            float m = -INFINITY, l = 0.f;
            bool any = false;                                // this half has had a tile
#pragma unroll 1
            for (int j = pair ? 0 : w; j < steps; j += pair ? 1 : 2) {
                wait(s_full + 8 * w, ns & 1);
                if constexpr (kScaleQ && !kFewRows) {
                    if (!pair && w == 1 && !any) {           // S of half 1 follows the scaling
                        if (kCap) cap_in *= ml[row].x;
                        else unit *= ml[row].x;
                    }
                }
                ++ns;
                if (!any) {
                    // Neither half's O is written again before both halves have read it.
                    settle();
                    if constexpr (kScaleQ && kFewRows) {
                        const float undo = undo_of[(k % kItems) * kFew + lane];
                        if (kCap) cap_in *= undo;
                        else unit *= undo;
                    }
                    any = true;
                }
                if constexpr (kFewRows) {
                    // This warp's 32 keys of all rows, which lie in every quarter's lanes.
                    uint32_t v[32];
                    const uint32_t shared = base + L::p + w * L::pHalf;
                    tc_fence_after();
                    tmem_ld_issue_x32(ts + 32 * quarter, v);
                    tmem_ld_wait_x32(v);
                    tc_fence_before();
                    mbar_arrive_warp(s_read + 8 * w);
                    if constexpr (kCap != kNoCap) {
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            v[i] = kCap == kWide ? capped_wide(v[i], cap_in, cap)
                                                 : capped(v[i], cap_in, cap);
                    }
                    if (j < from || j >= to) {
                        const int k0 = (first + j) * BN + 32 * quarter;
                        const uint32_t seen = below(row_hi - k0) & ~below(row_lo - k0);
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (!(seen & (1u << i))) v[i] = 0xFF800000u;
                    }
                    float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
                    for (int i = 0; i < 32; i += 4)
#pragma unroll
                        for (int x = 0; x < 2; ++x)
                            top[x] = fmaxf(fmaxf(top[x], __uint_as_float(v[i + 2 * x])),
                                           __uint_as_float(v[i + 2 * x + 1]));
                    // The tile's maximum of the row, from all four warps.
                    // In two buffers by turns: P of the tile before the last has been waited for by all.
                    float* maxima = reinterpret_cast<float*>(smem + L::p + w * L::pHalf + L::pShare) +
                                    (ns & 1) * 4 * kFew;
                    maxima[quarter * kFew + lane] = fmaxf(top[0], top[1]);
                    mbar_arrive_warp(share + 8 * w);
                    wait(share + 8 * w, nshare++ & 1);
                    const float most = fmaxf(fmaxf(maxima[lane], maxima[kFew + lane]),
                                             fmaxf(maxima[2 * kFew + lane], maxima[3 * kFew + lane])) *
                                       unit;
                    const bool grown = live && most > m;
                    const float keep = grown && m > -INFINITY ? ex2(m - most) : 1.f;
                    if (grown) m = most;
                    // The tile before this one is in O, and its P has been read.
                    wait(o_done + 8 * w, ns & 1);
                    if (__any_sync(kFull, keep != 1.f)) {
                        l *= keep;
                        if (quarter == 0) {              // O lies in the first quarter's lanes
                            tc_fence_after();
#pragma unroll 1
                            for (int d = 0; d < D; d += 16) scale_columns(to_ + d, keep);
                        }
                    }
                    const float off = m == -INFINITY ? 0.f : kLift - m;
                    const uint64_t unit2 = pair_of(unit, unit), off2 = pair_of(off, off);
                    uint64_t add[2] = {0, 0};
                    const uint32_t to_p = shared + (quarter >> 1) * L::pKeys + lane * 128;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t pk[4];
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            const int at = 8 * i + 2 * x;
                            const float2 y = halves_of(
                                fma_pair(pair_of(__uint_as_float(v[at]), __uint_as_float(v[at + 1])),
                                         unit2, off2));
                            const float lo = ex2(y.x), hi = ex2(y.y);
                            add[x & 1] = add_pair(add[x & 1], pair_of(lo, hi));
                            pk[x] = pack16(kMmaHalf, lo, hi);
                        }
                        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                                         to_p + ((((quarter & 1) * 4 + i) ^ (lane & 7)) * 16)),
                                     "r"(pk[0]), "r"(pk[1]), "r"(pk[2]), "r"(pk[3])
                                     : "memory");
                    }
                    const float2 sums = halves_of(add_pair(add[0], add[1]));
                    l += sums.x + sums.y;
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    tmem_st_wait();
                    tc_fence_before();
                    mbar_arrive_warp(p_up + 8 * w);
                    if constexpr (kSpread) {
                        const uint32_t u = g + j, r = u % L::kRawV, to_stage = u % kV;
                        wait(rv_full + 8 * (u % (2 * L::kRawV)), (u / (2 * L::kRawV)) & 1);
                        if (u >= kV) wait(v_empty + 8 * to_stage, (u / kV - 1) & 1);
                        if (widen_tile<D>(smem + L::raw + (L::kRawStages + r) * L::kRaw,
                                          smem + L::values + to_stage * L::kTile, row,
                                          j < from || j >= to, c->L - (first + j) * BN))
                            items[k % kItems].v_odd = 1;
                        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                        mbar_arrive_warp(rv_empty + 8 * r);
                        mbar_arrive_warp(v_full + 8 * (u % (2 * kV)));
                    }
                } else {
                    if (!warp_live) {
                        mbar_arrive_warp(p_up + 8 * w);
                        mbar_arrive_warp(p_low + 8 * w);
                        continue;
                    }
                    tc_fence_after();
                    uint32_t va[32], vb[32];
                    const bool masked = j < from || j >= to;
                    if (kCap || masked) {
                        // Caps and masks first, in tensor memory, in quarters of 32 keys: the steps that
                        // every tile takes stay short.
                        const int k0 = (first + j) * BN;
                        auto prepare = [&](uint32_t (&v)[32], int c0) {
                            if constexpr (kCap != kNoCap) {
#pragma unroll
                                for (int i = 0; i < 32; ++i)
                                    v[i] = kCap == kWide ? capped_wide(v[i], cap_in, cap)
                                                         : capped(v[i], cap_in, cap);
                            }
                            if (masked) {
                                const uint32_t seen =
                                    below(row_hi - k0 - c0) & ~below(row_lo - k0 - c0);
#pragma unroll
                                for (int i = 0; i < 32; ++i)
                                    if (!(seen & (1u << i))) v[i] = 0xFF800000u;
                            }
                            tmem_st_x32(ts + c0, v);
                        };
#pragma unroll 1
                        for (int c0 = 0; c0 < BN; c0 += 64) {
                            tmem_ld_issue_x32(ts + c0, va);
                            tmem_ld_issue_x32(ts + c0 + 32, vb);
                            tmem_ld_wait_x32(va);
                            tmem_ld_wait_x32(vb);
                            prepare(va, c0);
                            prepare(vb, c0 + 32);
                        }
                        tmem_st_wait();
                    }
                    // S in quarters, first for the maximum, then, from the top, for the weights. P of a
                    // quarter overwrites S that has been read for good: quarter c goes to columns
                    // 64 + 16 c.
                    float top[2] = {-INFINITY, -INFINITY};
                    auto raise = [&](const uint32_t (&v)[32]) {
#pragma unroll
                        for (int i = 0; i < 32; i += 4)
#pragma unroll
                            for (int x = 0; x < 2; ++x)
                                top[x] = fmaxf(fmaxf(top[x], __uint_as_float(v[i + 2 * x])),
                                               __uint_as_float(v[i + 2 * x + 1]));
                    };
                    tmem_ld_issue_x32(ts, va);
                    tmem_ld_issue_x32(ts + 32, vb);
                    tmem_ld_wait_x32(va);
                    tmem_ld_wait_x32(vb);
                    raise(va);
                    tmem_ld_issue_x32(ts + 64, va);
                    raise(vb);
                    tmem_ld_issue_x32(ts + 96, vb);
                    tmem_ld_wait_x32(va);
                    tmem_ld_wait_x32(vb);
                    raise(va);
                    raise(vb);
                    const float most = fmaxf(top[0], top[1]) * unit;
                    const bool grown = most > m + kGrowth;       // also when m is still -inf
                    const float keep = grown && m > -INFINITY ? ex2(m - most) : 1.f;
                    if (grown) m = most;
                    if (__any_sync(kFull, keep != 1.f)) {
                        // O holds the tiles before this one: wait for the last of them.
                        wait(o_done + 8 * w, ns & 1);
                        tc_fence_after();
                        l *= keep;
#pragma unroll 1
                        for (int d = 0; d < D; d += 16) scale_columns(to_ + d, keep);
                    }
                    const float off = m == -INFINITY ? 0.f : kLift - m;
                    const uint64_t unit2 = pair_of(unit, unit), off2 = pair_of(off, off);
                    uint64_t add[2] = {0, 0};
                    // The weights of one quarter, from its scores.
                    auto weigh = [&](const uint32_t (&v)[32], int quarter) {
                        uint32_t pk[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const float2 x = halves_of(
                                fma_pair(pair_of(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1])),
                                         unit2, off2));
                            const float lo = ex2(x.x), hi = ex2(x.y);
                            add[i & 1] = add_pair(add[i & 1], pair_of(lo, hi));
                            pk[i] = pack16(kMmaHalf, lo, hi);
                        }
                        tmem_st_x16(ts + 64 + 16 * quarter, pk);
                    };
                    weigh(vb, 3);
                    tmem_ld_issue_x32(ts + 32, vb);
                    weigh(va, 2);
                    tmem_ld_wait_x32(vb);
                    tmem_ld_issue_x32(ts, va);
                    tmem_st_wait();
                    tc_fence_before();
                    mbar_arrive_warp(p_up + 8 * w);
                    weigh(vb, 1);
                    tmem_ld_wait_x32(va);
                    weigh(va, 0);
                    tmem_st_wait();
                    tc_fence_before();
                    mbar_arrive_warp(p_low + 8 * w);
                    const float2 sums = halves_of(add_pair(add[0], add[1]));
                    l += sums.x + sums.y;
                }
            }
            g += max(steps, 0);
            // Epilogue, once this half's last tile is in O.
            if (any) wait(o_done + 8 * w, (ns - 1) & 1);
            else settle();
            if constexpr (kFewRows) {
                // The four warps' sums; O and the rest of the item are the first one's.
                if (any) {
                    float* sums = reinterpret_cast<float*>(smem + L::p + w * L::pHalf + L::pShare);
                    sums[quarter * kFew + lane] = l;
                    mbar_arrive_warp(share + 8 * w);
                    wait(share + 8 * w, nshare++ & 1);
                    l = (sums[lane] + sums[kFew + lane]) + (sums[2 * kFew + lane] + sums[3 * kFew + lane]);
                }
                live &= quarter == 0;
                warp_live &= quarter == 0;
            }
            const bool whole = c->whole();
            auto finish = [&]() {                            // the factor that ends the quotient
                if (c->bad || (c->bad_page && sees_bad_page(p, *c, row_lo, row_hi))) {
                    m = 0.f;
                    l = NAN;
                }
                return !whole ? 1.f : (l == 0.f ? 0.f : p.v_scale / l);
            };
            float f0, f1 = 0.f;                              // factors of the halves' O
            bool has0 = any, has1 = false;
            int d_begin = 0, d_end = D;
            uint32_t o0 = to_;
            if (pair) {
                f0 = finish();
            } else {
                // One row tile: half 1 passes (m, l) over, half 0 returns the factors of both
                // halves' O, and each half writes half of the columns. A half 1 without a tile has
                // nothing to pass, and must not: it has not waited for the scores, which follow half
                // 0's factors in ml, so its write could land on either side of theirs.
                has0 = steps > 0;
                has1 = steps > 1;
                if (w == 1) {
                    if (has1) ml[row] = make_float2(m, l);
                    mbar_arrive_warp(ml_there);
                    wait(ml_back, nb & 1);
                    f0 = ml[row].x;
                    f1 = ml[row].y;
                } else {
                    wait(ml_there, nb & 1);
                    const float2 other = has1 ? ml[row] : make_float2(-INFINITY, 0.f);
                    const float top = fmaxf(m, other.x);
                    const float at = top == -INFINITY ? 0.f : top;
                    f0 = ex2(m - at);
                    f1 = ex2(other.x - at);
                    l = l * f0 + other.y * f1;
                    m = top;
                    const float norm = finish();
                    f0 *= norm;
                    f1 *= norm;
                    ml[row] = make_float2(f0, f1);
                    mbar_arrive_warp(ml_back);
                }
                o0 = lane_base + 256;
                d_begin = w * (D / 2);
                d_end = d_begin + D / 2;
            }
            tc_fence_after();
            if (warp_live) {
                float4* part = reinterpret_cast<float4*>(
                    p.part + (size_t)(2 * blockIdx.x + (c->lo > 0 ? 0 : 1)) * part_floats(D) +
                    (size_t)(pair ? w : 0) * BM * (D + 2));
                const long long out_row = ((long long)c->t0 + sub0 + row_token) * p.q_heads +
                                          c->h * p.g + ((kFewRows ? lane : row) - row_token * p.g);
                uint16_t* out = static_cast<uint16_t*>(p.out) + out_row * D;
                // The rows whose output this lane stores: 16-byte pieces pass through groups of four
                // lanes, so that a store covers 8 rows x 64 bytes and not 32 rows x 16.
                int rows_out[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    rows_out[i] = __shfl_sync(kFull, live ? (int)out_row : -1, (lane & ~3) + i);
#pragma unroll 1
                for (int d = d_begin; d < d_end; d += 32) {
                    uint32_t x[32] = {}, y[32] = {};
                    if (has0) tmem_ld_issue_x32(o0 + d, x);
                    if (has1) tmem_ld_issue_x32(lane_base + 384 + d, y);
                    if (has0) tmem_ld_wait_x32(x);
                    if (has1) tmem_ld_wait_x32(y);
                    float o[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        o[i] = has0 ? __uint_as_float(x[i]) * f0 : f0 * 0.f;
                        if (has1) o[i] = fmaf(__uint_as_float(y[i]), f1, o[i]);
                    }
                    if (whole) {
                        uint32_t piece[4][4];
#pragma unroll
                        for (int i = 0; i < 4; ++i)
#pragma unroll
                            for (int x = 0; x < 4; ++x)
                                piece[i][x] = pack16(kHalf, o[8 * i + 2 * x], o[8 * i + 2 * x + 1]);
                        turn_pieces(piece, lane);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (rows_out[i] >= 0)
                                *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) +
                                                          (long long)rows_out[i] * D + d +
                                                          8 * (lane & 3)) =
                                    make_uint4(piece[i][0], piece[i][1], piece[i][2], piece[i][3]);
                    } else if (live) {
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            part[(d / 4 + i) * BM + row] =
                                make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
                    }
                }
                if (c->v_odd != 0) __syncwarp();             // the rows are written by other lanes
                if (c->v_odd != 0 && live)
                    refill_values<kHalf, kSmall>(p, *c, row_lo, row_hi, d_begin, d_end,
                                                 whole ? out : nullptr,
                                                 reinterpret_cast<float*>(part) + row * 4);
                if (live && (pair || w == 0)) {
                    if (!whole)
                        reinterpret_cast<float2*>(part + BM * (D / 4))[row] = make_float2(m, l);
                    else if (p.lse)
                        p.lse[out_row] = l == 0.f ? -INFINITY : (m + (log2f(l) - kLift)) * kLn2;
                }
            }
            tc_fence_before();
            if (!pair) {
                mbar_arrive_warp(halves_done);
                both = true;
                ++nb;
            }
            done_with();
        }
        if (!ok && lane == 0) atomicOr(status, kStatusTimeout);
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512)
                     : "memory");
    }
}

// ---------------------------------------------------------------- join
//
// For each range start that cuts an item, and is the first to: out = sum_i w_i O_i / sum_i w_i l_i
// over the item's pieces, w_i = 2^(m_i - max m). blockIdx.x: the range start - 1; blockIdx.y: a
// slice of the item's rows and columns. Bound by latency, so pieces are found by all threads at
// once, `ways` threads share an element's pieces, and each loads four at a time (one token over
// 6775 keys, 53 pieces: a call of 86 us with one thread walking them, 27 us so).
template <int D>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const __grid_constant__ Problem p, bool half_type, float lift) {
    __shared__ int slot[kMaxRanges + 1];                     // each piece's place, -1: no steps
    __shared__ float2 sum_ml[kJoinThreads];
    __shared__ float4 sum_o[kJoinThreads];
    grid_dependency_wait();
    const int b = blockIdx.x + 1, tid = threadIdx.x;
    const int4 at = p.bound[b], before = p.bound[b - 1];
    if (at.x >= p.R || at.w == 0) return;
    if (before.x == at.x && before.y == at.y && before.z == at.z && before.w > 0) return;
    const Request q = request_of(p, at.x);
    const int tok0 = at.z * p.tpi, ntok = min(p.tpi, q.n - tok0);
    int begin, end;
    key_tiles(p, q.n, q.L, tok0, ntok, begin, end);
    const int steps = end - begin;
    // The item's pieces: range b - 1 from step 0, and the ranges that start in it.
    int pieces = 1;
    for (int m0 = b; m0 <= p.G; m0 += kJoinThreads) {
        const int m = m0 + tid;
        const int4 x = p.bound[min(m, p.G)];
        const int4 next = p.bound[min(m + 1, p.G)];
        const bool in = m <= p.G && x.x == at.x && x.y == at.y && x.z == at.z;
        const bool ends = !(m < p.G && next.x == at.x && next.y == at.y && next.z == at.z);
        if (in) slot[m - b + 1] = x.w < (ends ? steps : next.w) ? 2 * m : -1;
        pieces += __syncthreads_count(in);
    }
    if (tid == 0) slot[0] = 2 * (b - 1) + 1;
    __syncthreads();
    const int ways = pieces >= 32 ? 8 : (pieces >= 8 ? 4 : (pieces >= 4 ? 2 : 1));
    const int per = kJoinThreads / ways, way = tid / per;
    const int rows = ntok * p.g;                             // of both row tiles
    const int in_tile = p.tpt * p.g, total = rows * (D / 4);
    for (int e0 = blockIdx.y * per; e0 < total; e0 += kJoinSlices * per) {
        const int e = min(e0 + tid % per, total - 1);
        const int col = e / rows, row = e - col * rows;
        const int sub = row >= in_tile ? 1 : 0, r = row - sub * in_tile;
        const float* tile = p.part + (size_t)sub * BM * (D + 2);
        float top = -INFINITY, l = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        auto add = [&](float2 s, float4 x, float ref) {
            const float wt = ex2(s.x - ref);
            l = fmaf(s.y, wt, l);
            o.x = fmaf(x.x, wt, o.x);
            o.y = fmaf(x.y, wt, o.y);
            o.z = fmaf(x.z, wt, o.z);
            o.w = fmaf(x.w, wt, o.w);
        };
        auto follow = [&](float most) -> float {             // the reference from here on
            const float ref = most == -INFINITY ? 0.f : most, by = ex2(top - ref);
            top = most;
            l *= by;
            o = make_float4(o.x * by, o.y * by, o.z * by, o.w * by);
            return ref;
        };
        for (int i = way; i < pieces; i += 4 * ways) {
            float2 s[4];
            float4 x[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int at_slot = i + u * ways < pieces ? slot[i + u * ways] : -1;
                s[u] = make_float2(-INFINITY, 0.f);
                x[u] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (at_slot >= 0) {
                    const float* o_ml = tile + (size_t)at_slot * part_floats(D);
                    s[u] = reinterpret_cast<const float2*>(o_ml + BM * D)[r];
                    x[u] = reinterpret_cast<const float4*>(o_ml)[col * BM + r];
                }
            }
            const float ref = follow(fmaxf(top, fmaxf(fmaxf(s[0].x, s[1].x), fmaxf(s[2].x, s[3].x))));
#pragma unroll
            for (int u = 0; u < 4; ++u) add(s[u], x[u], ref);
        }
        if (ways > 1) {
            sum_ml[tid] = make_float2(top, l);
            sum_o[tid] = o;
            __syncthreads();
            if (way == 0) {
                for (int y = 1; y < ways; ++y) {
                    const float2 s = sum_ml[tid + y * per];
                    add(s, sum_o[tid + y * per], follow(fmaxf(top, s.x)));
                }
            }
            __syncthreads();
        }
        if (way > 0 || e0 + tid >= total) continue;
        const float norm = l == 0.f ? 0.f : p.v_scale / l;
        const long long out_row = ((long long)q.t0 + tok0 + row / p.g) * p.q_heads + at.y * p.g +
                                  row % p.g;
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + out_row * D + col * 4) =
            make_uint2(pack16(half_type, o.x * norm, o.y * norm),
                       pack16(half_type, o.z * norm, o.w * norm));
        if (col == 0 && p.lse)
            p.lse[out_row] = l == 0.f ? -INFINITY : (top + (log2f(l) - lift)) * kLn2;
    }
}

// ---------------------------------------------------------------- host

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
    static std::once_flag once;
    static EncodeTiledFn fn = nullptr;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                             &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(p);
        else
            (void)cudaGetLastError();
    });
    return fn;
}

// A rank-4 tensor: dims and strides innermost first (strides in elements, of dimensions 1 to 3),
// boxes of 128 bytes x box1 x 1 x box3 with the 128-byte swizzle for 16-bit types, and of whole
// rows, unswizzled, for e4m3.
bool encode_4d(CUtensorMap* map, int dtype, const void* base, const long long (&dim)[4],
               const long long (&stride)[3], int box1, int box3) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const int size = dtype == kE4m3 ? 1 : 2;
    cuuint64_t dims[4], strides[3];
    for (int i = 0; i < 4; ++i) dims[i] = (cuuint64_t)dim[i];
    // A dimension of one element is never stepped along; its stride only has to be encodable.
    for (int i = 0; i < 3; ++i)
        strides[i] = (cuuint64_t)((dim[i + 1] == 1 ? dim[0] : stride[i]) * size);
    const cuuint32_t box[4] = {dtype == kE4m3 ? (cuuint32_t)dim[0] : 64u, (cuuint32_t)box1, 1,
                               (cuuint32_t)box3};
    const cuuint32_t step[4] = {1, 1, 1, 1};
    const CUtensorMapDataType type = dtype == kE4m3   ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                     : dtype == kFp16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                      : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    return fn(map, type, 4, const_cast<void*>(base), dims, strides, box, step,
              CU_TENSOR_MAP_INTERLEAVE_NONE,
              dtype == kE4m3 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B,
              dtype == kE4m3 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B : CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool kHalf, int kCap, bool kSmall, bool kFewRows>
cudaError_t launch_on_tensor_cores(const DeviceInfo& dev, const AttentionArgs& a, const Problem& p,
                                   uint32_t* status, cudaStream_t stream) {
    static std::once_flag once[64];
    static cudaError_t attr_err[64];
    if (dev.device < 0 || dev.device >= 64) return cudaErrorInvalidDevice;
    using L = Layout<D, kSmall, kFewRows>;
    auto kernel = attention_kernel<D, kHalf, kCap, kSmall, kFewRows>;
    const size_t smem = 1024 + L::total;
    std::call_once(once[dev.device], [&] {
        attr_err[dev.device] = cudaFuncSetAttribute(
            kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    });
    if (attr_err[dev.device] != cudaSuccess) return attr_err[dev.device];
    const KvCache& c = a.cache;
    CUtensorMap map_q, map_k, map_v;
    const int box = std::min(c.page_size, BN);
    if (!encode_4d(&map_q, a.dtype, a.query, {D, p.g, c.kv_heads, a.T},
                   {a.q_head_stride, p.g * a.q_head_stride, a.q_token_stride}, p.g, p.tpt) ||
        !encode_4d(&map_k, c.dtype, c.key, {D, c.page_size, c.kv_heads, c.num_pages},
                   {c.token_stride, c.head_stride, c.page_stride}, box, 1) ||
        !encode_4d(&map_v, c.dtype, c.value, {D, c.page_size, c.kv_heads, c.num_pages},
                   {c.token_stride, c.head_stride, c.page_stride}, box, 1))
        return cudaErrorInvalidValue;
    kernel<<<p.G, kThreads, smem, stream>>>(map_q, map_k, map_v, p, status);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !p.join) return e;
    // The join may be set up before the attention has ended, and waits for it before it reads.
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3((unsigned)(p.G - 1), kJoinSlices);
    cfg.blockDim = dim3(kJoinThreads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, join_kernel<D>, p, kHalf, weight_lift(kHalf || kSmall, kFewRows));
}

template <int D, bool kHalf, bool kSmall>
cudaError_t launch_build(const DeviceInfo& dev, const AttentionArgs& a, const Problem& p, bool few,
                         uint32_t* status, cudaStream_t stream) {
    if (p.softcap == 0.f)
        return few ? launch_on_tensor_cores<D, kHalf, kNoCap, kSmall, true>(dev, a, p, status, stream)
                   : launch_on_tensor_cores<D, kHalf, kNoCap, kSmall, false>(dev, a, p, status, stream);
    if (p.softcap <= kQuickCap)
        return few ? launch_on_tensor_cores<D, kHalf, kQuick, kSmall, true>(dev, a, p, status, stream)
                   : launch_on_tensor_cores<D, kHalf, kQuick, kSmall, false>(dev, a, p, status, stream);
    return few ? launch_on_tensor_cores<D, kHalf, kWide, kSmall, true>(dev, a, p, status, stream)
               : launch_on_tensor_cores<D, kHalf, kWide, kSmall, false>(dev, a, p, status, stream);
}

template <bool kSmall>
cudaError_t launch_for_cache(const DeviceInfo& dev, const AttentionArgs& a, const Problem& p, bool few,
                             uint32_t* status, cudaStream_t stream) {
    const bool half_type = a.dtype == kFp16;
    if (p.D == 64)
        return half_type ? launch_build<64, true, kSmall>(dev, a, p, few, status, stream)
                         : launch_build<64, false, kSmall>(dev, a, p, few, status, stream);
    return half_type ? launch_build<128, true, kSmall>(dev, a, p, few, status, stream)
                     : launch_build<128, false, kSmall>(dev, a, p, few, status, stream);
}

}  // namespace
}  // namespace dflash
