// verify.cu: verification of drafted tokens against the target model's logits.
//
// Page "vllm.v1.worker.gpu.spec_decode.dflash.speculator": propose() hands its draft tokens to the
// target model, which looks at them in its next step; the pages do not show how it takes or leaves
// them. This is the standard rule, which keeps the target's distribution whatever the drafter's is.
// With p_i = softmax(logits of row i / T) and the draft's distribution q_i over its K candidates:
//
//   draft i is taken iff u_i q_i(x_i) < p_i(x_i), for i = 0, 1, ... until one is not;
//   in the row of the first that is not, a token is drawn from max(p_i - q_i, 0), normalised;
//   if all are taken, from p in the row behind the last;
//   drawn: the smallest v with sum_{j<=v} weight_j > u sum_j weight_j.
//
// The tokens are those of exact arithmetic, but for borders nearer than about 2^-38 of a row's sum: every
// choice is made with fp32 sums first, whose error is bounded, and once more with sums of twice the
// precision where the bound does not settle it. (Where the border falls among many unlikely tokens it
// seldom does.)
//
// Three kernels, each the next one's programmatic predecessor:
// - row_sums reads the logits: of each tile of a row (4 KB) the largest, m, and the sum of
//   exp((x - m) / T).
// - choose, a CTA a request, joins the tiles' sums, takes the drafts in order, and draws the last token:
//   the tile from the sums, then the place in it from the tile's logits, read again. Draws that are not
//   settled go on a list.
// - settle takes the list's rows' sums again in twice the precision, all SMs on all tiles, and the CTA that
//   finishes a row draws its token.
// Bounds: row_sums is to be bound by memory, and reads more than it needs, since a row's draft is judged while the
// next positions' rows stream in; choose and settle by the latency of their steps. 64 requests of 16 rows of 151936
// bf16 logits: 86 us on an idle GPU with nothing in L2, of which sums 42, choose 15, settle 22 (8 requests have a draw
// that fp32 does not settle); 94.5 MB are needed, 14 us. 512 requests, greedy: 223 us, sums 205, 961 MB needed, 144 us.
// 256 of 262144 fp32 logits: 322 us, sums 268, 1657 MB needed, 248 us: 93% of what a copy reaches. One request: 20 us.
//
// Rows behind the first rejected draft are not needed. Where the batch is large, row_sums goes through
// the requests' first rows, then their second ones, and so on; the warp that finishes a row looks whether
// its draft is surely rejected, and later rows of that request are passed over. (64 requests of 16 rows of 151936 bf16
// logits, all but 50 of a row masked and the first drafts among the masked: 68 of 315 MB are read, in 46 us.)
#include "common.cuh"
#include "ptx.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cfloat>
#include <climits>
#include <cmath>
#include <mutex>
#include <type_traits>

namespace dflash {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr float kLog2e = 1.4426950408889634f;

// ---------------------------------------------------------------- logits

template <typename T>
struct Vec;   // a 16-byte vector of logits
template <>
struct Vec<float> {
    static constexpr int kN = 4;
    static __device__ __forceinline__ void widen(const uint4& v, float* x) {
        x[0] = __uint_as_float(v.x);
        x[1] = __uint_as_float(v.y);
        x[2] = __uint_as_float(v.z);
        x[3] = __uint_as_float(v.w);
    }
};
template <>
struct Vec<__nv_bfloat16> {
    static constexpr int kN = 8;
    static __device__ __forceinline__ void widen(const uint4& v, float* x) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
};
template <>
struct Vec<__half> {
    static constexpr int kN = 8;
    static __device__ __forceinline__ void widen(const uint4& v, float* x) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
        }
    }
};

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }

// A row's tiles. The row starts `head` elements before its first 16-byte boundary; tile 0 also has
// those, and tile t has the elements from first(t) to first(t + 1), so every other tile starts on one.
constexpr int kVecs = 8;                         // 16-byte vectors of a tile a lane holds
template <typename T>
struct Row {
    static constexpr int kN = Vec<T>::kN;
    static constexpr int kTile = kVecs * 32 * kN;
    // -inf
    static constexpr uint32_t kLow = sizeof(T) == 4 ? 0xff800000u
                                                    : std::is_same<T, __half>::value ? 0xfc00fc00u : 0xff80ff80u;
    const T* x;
    int V, head;
    __device__ __forceinline__ Row(const VerifyArgs& a, long long row) {
        x = static_cast<const T*>(a.logits) + row * a.row_stride;
        V = a.V;
        head = (int)((16 - (reinterpret_cast<uintptr_t>(x) & 15)) & 15) / (int)sizeof(T);
    }
    __device__ __forceinline__ int first(int t) const {
        return t == 0 ? 0 : (int)min((long long)head + (long long)t * kTile, (long long)V);
    }
    // the tile of element v
    __device__ __forceinline__ int tile_of(int v) const { return v < head ? 0 : (v - head) / kTile; }

    // Elements of tile t that start on a boundary: from, and how many.
    __device__ __forceinline__ int body(int t, int& n) const {
        const int hi = first(t + 1), from = t == 0 ? min(head, hi) : first(t);
        n = hi - from;
        return from;
    }
    // Tile t's whole vectors, a warp's lanes side by side, -inf where there are none. from: the first, in
    // the row or in a copy of it.
    __device__ __forceinline__ void load(int t, int lane, const uint4* from, uint4 (&v)[kVecs]) const {
        int n;
        body(t, n);
        from += lane;
        if (n == kTile) {
#pragma unroll
            for (int k = 0; k < kVecs; ++k) v[k] = from[32 * k];
            return;
        }
#pragma unroll
        for (int k = 0; k < kVecs; ++k) {
            v[k] = make_uint4(kLow, kLow, kLow, kLow);
            if ((k * 32 + lane) * kN + kN <= n) v[k] = from[32 * k];
        }
    }
    // Of the elements of tile t that are in no whole vector, at most one a lane, or -inf.
    __device__ __forceinline__ float edge(int t, int lane) const {
        int n;
        const int from = body(t, n), rest = n & (kN - 1);
        if (t == 0 && lane < head && lane < from) return to_float(x[lane]);
        if (lane >= 16 && lane - 16 < rest) return to_float(x[from + n - rest + lane - 16]);
        return -INFINITY;
    }
};

// Rows that no request can have.
__device__ __forceinline__ bool bad_rows(const VerifyArgs& a, int start, int end) {
    return start < 0 || end < start || end > a.T || end - start > a.S + 1;
}

// Temperatures: a request is greedy at 0 (and below, and at NaN); else weights are exp2((x - m) * c).
struct Temperature {
    float t, c;
    bool greedy;
    __device__ __forceinline__ Temperature(const VerifyArgs& a, int r) {
        t = a.temperatures ? a.temperatures[r] : a.temperature;
        greedy = !(t > 0.f);
        // Between 2^-99 and 2^100, so that no product with 1 / T turns 0 or a difference of -inf to NaN.
        t = greedy ? 0.f : fminf(fmaxf(t, 0x1p-99f), 0x1p100f);
        c = greedy ? 1.f : kLog2e / t;
    }
};

// A draw that fp32 sums do not settle.
struct Unsettled {
    int r, i;          // row i of request r
    float M;           // its largest logit
    unsigned arrived;  // CTAs that are done with their tiles
};

// Quotients by a fixed divisor, of numbers below 2^31: with l = ceil(log2 d) and m = floor(2^32 (2^l - d)
// / d) + 1, n / d is the upper half of m n, plus n, shifted by l.
struct Divisor {
    unsigned m;
    int l;
    Divisor(unsigned d = 1) {
        for (l = 0; (1ull << l) < d;) ++l;
        m = (unsigned)(((1ull << 32) * ((1ull << l) - d)) / d + 1);
    }
    __device__ __forceinline__ unsigned of(unsigned n) const { return (__umulhi(m, n) + n) >> l; }
};

struct VerifyPlan {
    VerifyArgs a;
    int tiles;                // of a row
    int chunks;               // items of a row: kSumWarps tiles each
    float2* sums;             // [T][tiles]: the largest logit, the sum of exp((x - it) / T); a listed row's: a Two
    Unsettled* list;          // [R]
    unsigned* listed;         // how many
    // Where rows may be passed over (else null), by position and request, [S + 1][padded]:
    int* alive;               // [padded] the request's last row that may be needed, -1: none
    int* handed;              // groups of items that were handed out, less one
    int padded;               // R, to a multiple of 4
    int group, groups;        // items that are handed out at a time, and such groups in a row
    int window;               // rows that items are taken of at a time
    Divisor by_chunks, by_R, by_padded;
};

// NaN is passed over.
__device__ __forceinline__ float warp_max(float x) {
    float y;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(kFull, x, d);
    return x;
}

// A tile's sum, as other CTAs may be writing it: whole, or as it was before.
__device__ __forceinline__ float2 tile_sum(const float2* at) {
    const uint64_t v = ptx::load_shared_by_all(static_cast<const void*>(at));
    return ptx::halves_of(v);
}

// The largest logit of a row and the sum of its weights relative to it, from the tiles' sums, by a
// warp. The sum is NaN where the row has a NaN or +inf, and 0 where all of it is -inf. False if a tile's
// is not there yet.
__device__ __forceinline__ bool join_tiles(const float2* sums, int tiles, float c, int lane, float& M,
                                           float& Z) {
    bool there = true;
    M = -INFINITY;
#pragma unroll 4
    for (int t = lane; t < tiles; t += 32) {
        const float m = tile_sum(&sums[t]).x;
        there &= __float_as_uint(m) != 0xffffffffu;
        M = fmaxf(M, m);
    }
    if (!__all_sync(kFull, there)) return false;
    M = warp_max(M);
    Z = 0.f;
#pragma unroll 4
    for (int t = lane; t < tiles; t += 32) {
        const float2 x = tile_sum(&sums[t]);
        Z += x.y * (x.x == -INFINITY ? (x.y == x.y ? 0.f : 1.f) : ptx::ex2((x.x - M) * c));
    }
    Z = warp_sum(Z);
    return true;
}

// q of token x in row (r, i), by a warp.
__device__ __forceinline__ float draft_probability(const VerifyArgs& a, long long at, int x, int lane) {
    if (!a.cand_ids) return 1.f;
    float q = 0.f;
    if (lane < a.K && a.cand_ids[at * a.K + lane] == x) q = a.draft_probs[at * a.K + lane];
    return warp_sum(q);
}

// ---------------------------------------------------------------- sums of tiles

// Error of the fp32 sums, relative to a row's sum, in units of 2^-24 and for V <= 2^20: the exponents' roundings
// 2.5 |z| (log2(e) / T is 1.5 off), and sum p |z| <= ln V + 1, so 37; ex2, twice, 4 each; a tile's additions, 16 in
// a lane and 7 across, 23, and what takes mc's rounding back 5; joining up to 1024 tiles, 32 additions in a lane, 5
// across and a product, 38: 111, below 2^-17. A border is a difference of two such sums, and inside a tile exponents
// are rounded once more: below 240, 2^-16.
constexpr float kSlack = 0x1p-16f;
// A draft's u q Z against its weight 2^z: one such sum, the sum of up to 32 equal candidates' q (5) and two products,
// 118, 2^-17; and ex2, 4, with an exponent rounded three times, 2.5 |z| ln 2. Drafts within it, one in a hundred
// thousand, are looked at again by their request's CTA alone, 120 us for 262144 logits: a wider bound would be dear.
// z is taken as -150 below that, where w is 0: a masked draft's is -inf, whose product with 0 would be no bound.
__device__ __forceinline__ float draft_slack(float uq, float w, float z) {
    return 0x1p-17f * uq + (0x1p-21f - fmaxf(z, -150.f) * 0x1p-22f) * w;
}

enum : int { kTaken = 0, kRejected = 1, kUnsure = 2, kBad = 3 };   // drafts

constexpr int kSumWarps = 8;
constexpr int kSumBlocks = 2;                    // CTAs of an SM
constexpr int kSumThreads = 32 * (kSumWarps + 2);

template <typename T>
__device__ __forceinline__ float largest(const uint4 (&v)[kVecs]);
template <>
__device__ __forceinline__ float largest<float>(const uint4 (&v)[kVecs]) {
    float m = -INFINITY;
#pragma unroll
    for (int k = 0; k < kVecs; ++k)
        m = fmaxf(m, fmaxf(fmaxf(__uint_as_float(v[k].x), __uint_as_float(v[k].y)),
                           fmaxf(__uint_as_float(v[k].z), __uint_as_float(v[k].w))));
    return m;
}
template <typename T2>
__device__ __forceinline__ T2 largest_pair(const uint4 (&v)[kVecs]) {
    T2 m = *reinterpret_cast<const T2*>(&v[0].x);
#pragma unroll
    for (int k = 0; k < kVecs; ++k) {
        m = __hmax2(m, __hmax2(*reinterpret_cast<const T2*>(&v[k].x), *reinterpret_cast<const T2*>(&v[k].y)));
        m = __hmax2(m, __hmax2(*reinterpret_cast<const T2*>(&v[k].z), *reinterpret_cast<const T2*>(&v[k].w)));
    }
    return m;
}
template <>
__device__ __forceinline__ float largest<__nv_bfloat16>(const uint4 (&v)[kVecs]) {
    const float2 m = __bfloat1622float2(largest_pair<__nv_bfloat162>(v));
    return fmaxf(m.x, m.y);
}
template <>
__device__ __forceinline__ float largest<__half>(const uint4 (&v)[kVecs]) {
    const float2 m = __half22float2(largest_pair<__half2>(v));
    return fmaxf(m.x, m.y);
}

template <typename T>
__device__ __forceinline__ float weight_sum(const uint4 (&v)[kVecs], float m, float c) {
    constexpr int kN = Vec<T>::kN;
    const float mc = __fmul_rn(m, c);
    if (fabsf(mc) < 0x1p22f) {
        // x c - mc in one rounding, two at a time; mc's own, at most 1/8, is taken back at the end.
        const uint64_t cc = ptx::pair_of(c, c), mm = ptx::pair_of(-mc, -mc);
        uint64_t s[2] = {0, 0};
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            float x[kN];
            Vec<T>::widen(v[i], x);
#pragma unroll
            for (int e = 0; e < kN; e += 2) {
                const float2 z = ptx::halves_of(ptx::fma_pair(ptx::pair_of(x[e], x[e + 1]), cc, mm));
                s[e / 2 & 1] = ptx::add_pair(s[e / 2 & 1], ptx::pair_of(ptx::ex2(z.x), ptx::ex2(z.y)));
            }
        }
        const float2 both = ptx::halves_of(ptx::add_pair(s[0], s[1]));
        return (both.x + both.y) * ptx::ex2(-fmaf(m, c, -mc));
    }
    float s[4] = {0.f, 0.f, 0.f, 0.f};
    const float ref = fmaxf(m, -FLT_MAX);
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
        float x[kN];
        Vec<T>::widen(v[i], x);
#pragma unroll
        for (int e = 0; e < kN; ++e) s[e & 3] += ptx::ex2((x[e] - ref) * c);
    }
    return (s[0] + s[1]) + (s[2] + s[3]);
}

// Whether draft i of request r is surely rejected; kUnsure if not all of its row's sums are there. A warp.
// Sums are 8 bytes, written and read in one access, and are all ones before: each tells by itself that it is there,
// and no order between them is needed.
template <typename T>
__device__ __noinline__ int judge(const VerifyPlan& p, int r, int i, long long row, const volatile bool* over) {
    const VerifyArgs& a = p.a;
    const int lane = threadIdx.x & 31;
    if (__any_sync(kFull, ptx::load_shared_by_all(&p.alive[r]) < i)) return kTaken;   // an earlier draft is rejected: no matter
    const Temperature temp(a, r);
    const float2* sums = p.sums + row * p.tiles;
    float M, Z;
    if (!join_tiles(sums, p.tiles, temp.c, lane, M, Z) || __any_sync(kFull, *over)) return kUnsure;
    if (!(Z > 0.f)) return kRejected;                // no distribution: the request ends here
    const long long draft = (long long)r * a.S + i;
    const int token = a.draft_tokens[draft];
    if ((unsigned)token >= (unsigned)a.V) return kRejected;
    const float l = to_float(Row<T>(a, row).x[token]);
    if (temp.greedy) return l < M ? kRejected : kTaken;
    const float q = draft_probability(a, draft, token, lane);
    const float z = (l - M) * temp.c;
    const float w = ptx::ex2(z), uq = a.accept_uniforms[draft] * q * Z;
    return uq - w >= draft_slack(uq, w, z) ? kRejected : kTaken;
}

// Slots: two are not enough (batches of 64 and 256 as above: 104 and 355 us instead of 86 and 322); items of half the
// size, four CTAs on an SM: 101 and 337.
// An item is kSumWarps tiles of a row, 32 KB in one piece, and goes through a ring of kSlots in shared memory.
// A CTA has a warp that finds the next item and starts its copy, eight that take a tile of it each, and one
// that judges rows' drafts.
//
// Rows go by position in the requests, then by request. Where rows may be passed over, a CTA looks at the
// next 256 of them, and takes items of one that is alive and has some left; of several such rows not all CTAs
// take the first, which would have them all ask at one address. (In a fixed assignment, CTAs that pass over
// many rows run ahead, into rows that nothing is known of yet: a batch of 64 x 16 rows of 1 MB read 683 MB, of
// which it needed 414. With one counter of items for all it read 479 MB, at half of the bandwidth.)
struct Item {
    long long row;
    int r, i, chunk;
    bool drafted;       // not the request's last row
};

struct Handout {
    const VerifyPlan& p;
    const int lane;
    long long at;       // rows are not passed over: the next item; else the first row with anything left
    int look = 0;       // the first of the rows that are looked at, at or behind `at`
    int turn;
    int more = 0;       // items in hand behind the last
    Item last;
    int4 alive[2], handed[2];   // of the 8 rows that this lane looks at

    __device__ Handout(const VerifyPlan& plan)
        : p(plan), lane(threadIdx.x & 31), at(plan.alive ? 0 : blockIdx.x), turn(blockIdx.x) {
        if (p.alive) ask();
    }

    // Asks for the rows from `look` on; the answers are first needed when the next item is.
    __device__ __forceinline__ void ask() {
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            const int x = look + 128 * g + 4 * lane;
            alive[g] = handed[g] = make_int4(-1, -1, -1, -1);
            if (x >= (p.a.S + 1) * p.padded) continue;
            alive[g] = ptx::load_shared_by_all(
                reinterpret_cast<const int4*>(p.alive + (x - (int)p.by_padded.of(x) * p.padded)));
            handed[g] = ptx::load_shared_by_all(reinterpret_cast<const int4*>(p.handed + x));
        }
    }

    // The next item, chunk -1 if there is none. One warp.
    __device__ Item next() {
        if (more > 0) {
            --more;
            ++last.chunk;
        } else if (p.alive) {
            of_the_living();
        } else {
            in_order();
        }
        return last;
    }

    __device__ void in_order() {
        const VerifyArgs& a = p.a;
        const long long items = (long long)(a.S + 1) * a.R * p.chunks;
        const bool narrow = items < 1ll << 31;
        last.chunk = -1;
        for (; at < items && last.chunk < 0; at += gridDim.x) {
            const long long x = narrow ? p.by_chunks.of((unsigned)at) : at / p.chunks;
            const int i = narrow ? (int)p.by_R.of((unsigned)x) : (int)(x / a.R), r = (int)(x - (long long)i * a.R);
            const int start = a.query_start[r], end = a.query_start[r + 1];
            if (bad_rows(a, start, end) || i >= end - start) continue;
            last = Item{(long long)start + i, r, i, (int)(at - x * p.chunks), false};
        }
    }

    // The next rows to look at: up to a position further on, else from the first again. (Without it CTAs try the same
    // few rows that are left, again and again: 1024 requests of 16 rows of 32768 bf16 logits 235 us, with it 194.)
    __device__ __forceinline__ void further() {
        look = look + 256 - (int)at <= p.a.R && look + 256 < (p.a.S + 1) * p.padded ? look + 256 : (int)at;
    }

    // Looks at 256 rows, 8 a lane; takes of the turn-th of the first `window` that have anything left.
    __device__ void of_the_living() {
        const int rows = (p.a.S + 1) * p.padded;
        last.chunk = -1;
        for (; at < rows; ask()) {
            unsigned left = 0;                                       // a bit for each of the lane's rows
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                const int i = (int)p.by_padded.of(look + 128 * g + 4 * lane);
                left |= ((alive[g].x >= i && handed[g].x + 1 < p.groups) |
                         (alive[g].y >= i && handed[g].y + 1 < p.groups) << 1 |
                         (alive[g].z >= i && handed[g].z + 1 < p.groups) << 2 |
                         (alive[g].w >= i && handed[g].w + 1 < p.groups) << 3) << 4 * g;
            }
            // How many such rows lanes below have, of the first 128 and of the others.
            const int n0 = __popc(left & 15u), n1 = __popc(left >> 4);
            int below0 = 0, below1 = 0, total0 = 0, total1 = 0;
#pragma unroll
            for (int k = 0; k < 3; ++k) {
                const unsigned b0 = __ballot_sync(kFull, n0 >> k & 1), b1 = __ballot_sync(kFull, n1 >> k & 1);
                const unsigned lower = (1u << lane) - 1;
                below0 += __popc(b0 & lower) << k;
                below1 += __popc(b1 & lower) << k;
                total0 += __popc(b0) << k;
                total1 += __popc(b1) << k;
            }
            if (total0 + total1 == 0) {
                if (look == (int)at) look = (int)(at += 256);
                else further();
                continue;
            }
            const int pick = turn % min(total0 + total1, p.window);
            ++turn;
            int row = -1, count = 0, start = 0, end = 0;
            if (pick < total0 ? pick >= below0 && pick < below0 + n0
                              : pick - total0 >= below1 && pick - total0 < below1 + n1) {
                const int g = pick < total0 ? 0 : 1;
                unsigned bits = g ? left >> 4 : left & 15u;
                for (int k = g ? pick - total0 - below1 : pick - below0; k > 0; --k) bits &= bits - 1;
                row = look + 128 * g + 4 * lane + __ffs(bits) - 1;
                count = (int)(atomicAdd(&p.handed[row], 1) + 1);
                const int r = row - (int)p.by_padded.of(row) * p.padded;
                start = p.a.query_start[r];
                end = p.a.query_start[r + 1];
            }
            const int from = __ffs(__ballot_sync(kFull, row >= 0)) - 1;
            if (total0 == 0 && look == (int)at) look = (int)(at += 128);
            count = __shfl_sync(kFull, count, from);
            if (count >= p.groups) {                                 // others were quicker
                further();
                continue;
            }
            row = __shfl_sync(kFull, row, from);
            start = __shfl_sync(kFull, start, from);
            end = __shfl_sync(kFull, end, from);
            const int i = (int)p.by_padded.of(row), r = row - i * p.padded;
            last = Item{(long long)start + i, r, i, count * p.group, i < end - start - 1};
            more = min(p.group, p.chunks - last.chunk) - 1;
            ask();
            return;
        }
    }
};

constexpr int kSlots = 3;
constexpr int kSlotBytes = kSumWarps * kVecs * 32 * 16;

constexpr int kQueue = 32;

struct SumShared {
    uint64_t full[kSlots];     // the item's copy has landed
    uint64_t done[kSlots];     // its tiles' sums are written
    Item items[kSlots];
    // Rows whose last item this CTA has, to be judged.
    Item queue[kQueue];
    volatile unsigned pushed, popped;
    volatile bool over;
};

template <typename T>
__global__ void __launch_bounds__(kSumThreads, kSumBlocks)
row_sums_kernel(const __grid_constant__ VerifyPlan p, uint32_t* status) {
    extern __shared__ __align__(128) uint8_t ring[];                 // [kSlots][kSlotBytes]
    __shared__ SumShared sh;
    constexpr int kN = Vec<T>::kN;
    const VerifyArgs& a = p.a;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        if (blockIdx.x == 0 && !p.alive) *p.listed = 0;
        for (int k = 0; k < kSlots; ++k) {
            ptx::mbar_init(ptx::smem_u32(&sh.full[k]), 1);
            ptx::mbar_init(ptx::smem_u32(&sh.done[k]), kSumWarps);
        }
        sh.pushed = sh.popped = 0;
        sh.over = false;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    ptx::grid_dependents_launch();
    if (p.alive) ptx::grid_dependency_wait();
    __syncthreads();
    int slot = 0;
    uint32_t parity = 0;
    auto advance = [&]() {
        if (++slot == kSlots) {
            slot = 0;
            parity ^= 1;
        }
    };
    auto await = [&](uint64_t* bar, uint32_t phase) {
        if (ptx::mbar_wait(ptx::smem_u32(bar), phase)) return true;
        if (lane == 0) atomicOr(status, kStatusTimeout);
        return false;
    };
    if (warp == kSumWarps) {                                         // finds and copies
        Handout handout(p);
        for (int n = 0;; ++n) {
            const Item item = handout.next();                        // while the slot is still in use
            if (n >= kSlots && !await(&sh.done[slot], parity ^ 1)) break;
            if (lane == 0) {
                sh.items[slot] = item;
                const uint32_t bar = ptx::smem_u32(&sh.full[slot]);
                uint32_t bytes = 0;
                if (item.chunk >= 0) {
                    const Row<T> x(a, item.row);
                    const int t = item.chunk * kSumWarps;
                    const int hi = x.first(min(t + kSumWarps, p.tiles));
                    const int body = t == 0 ? min(x.head, hi) : x.first(t);
                    bytes = (uint32_t)((hi - body) / kN) * 16;
                    if (bytes) {
                        ptx::mbar_expect_tx(bar, bytes);
                        ptx::bulk_load(ptx::smem_u32(ring + slot * kSlotBytes), x.x + body, bytes, bar);
                    }
                }
                if (!bytes) ptx::mbar_arrive(bar);
                // (With a full queue nobody looks at the row, and the next ones are read.)
                if (p.alive && item.drafted && item.chunk == p.chunks - 1 && sh.pushed - sh.popped < kQueue) {
                    sh.queue[sh.pushed % kQueue] = item;
                    __threadfence_block();
                    sh.pushed = sh.pushed + 1;
                }
            }
            if (item.chunk < 0) break;
            advance();
        }
        if (lane == 0) sh.over = true;
        return;
    }
    if (warp > kSumWarps) {                                          // judges
        // Looks at a row until all of its sums are there. Ends with the warp that finds items, which ends.
        if (!p.alive) return;
        for (;;) {
            if (__any_sync(kFull, sh.over)) return;                  // what is left decides nothing any more
            const unsigned popped = sh.popped;
            if (!__any_sync(kFull, sh.pushed != popped)) {
                __nanosleep(200);
                continue;
            }
            __threadfence_block();
            const Item row = sh.queue[popped % kQueue];
            const int state = judge<T>(p, row.r, row.i, row.row, &sh.over);
            if (state == kRejected && lane == 0) atomicMin(&p.alive[row.r], row.i);
            __threadfence_block();                                   // the item is read before its place is free
            __syncwarp();
            if (lane == 0 && state != kUnsure) sh.popped = popped + 1;
            __syncwarp();
        }
    }
    for (;; advance()) {                                             // sums
        if (!await(&sh.full[slot], parity)) return;
        const Item now = sh.items[slot];
        if (now.chunk < 0) return;
        const int t = now.chunk * kSumWarps + warp;
        if (t < p.tiles) {
            const Row<T> x(a, now.row);
            uint4 v[kVecs];
            const float edge = x.edge(t, lane);
            x.load(t, lane, reinterpret_cast<const uint4*>(ring + slot * kSlotBytes) + warp * kVecs * 32, v);
            const float c = Temperature(a, now.r).c;
            const float m = warp_max(fmaxf(edge, largest<T>(v)));
            float s = weight_sum<T>(v, m, c);
            if (__any_sync(kFull, edge > -INFINITY || edge != edge)) s += ptx::ex2((edge - fmaxf(m, -FLT_MAX)) * c);
            s = warp_sum(s);
            if (lane == 0) ptx::store_shared_by_all(&p.sums[now.row * p.tiles + t], m, s);
        }
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&sh.done[slot]));
    }
}

// What row_sums starts from where rows may be passed over.
constexpr int kStartThreads = 256;
__global__ void __launch_bounds__(kStartThreads) start_kernel(const __grid_constant__ VerifyPlan p) {
    const VerifyArgs& a = p.a;
    ptx::grid_dependents_launch();
    const long long at = (long long)blockIdx.x * kStartThreads + threadIdx.x, step = (long long)gridDim.x * kStartThreads;
    if (at == 0) *p.listed = 0;
    for (long long r = at; r < p.padded; r += step) {
        const int start = r < a.R ? a.query_start[r] : 0, end = r < a.R ? a.query_start[r + 1] : 0;
        p.alive[r] = bad_rows(a, start, end) ? -1 : end - start - 1;
    }
    for (long long k = at; k < (long long)(a.S + 1) * p.padded; k += step) p.handed[k] = -1;
    const uint4 ones = make_uint4(~0u, ~0u, ~0u, ~0u);
    uint4* sums = reinterpret_cast<uint4*>(p.sums);                  // room for a whole number of these
    for (long long k = at; k < ((long long)a.T * p.tiles + 1) / 2; k += step) sums[k] = ones;
}

// ---------------------------------------------------------------- sums of twice the precision

// A value as the sum of two floats, the second at most half a step of the first.
struct Two {
    float h, l;
};
__device__ __forceinline__ Two two_sum(float a, float b) {        // exact
    const float s = __fadd_rn(a, b), bb = __fsub_rn(s, a);
    return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, bb)), __fsub_rn(b, bb))};
}

__device__ __forceinline__ Two quick_sum(float a, float b) {      // exact where |a| >= |b|
    const float s = __fadd_rn(a, b);
    return {s, __fsub_rn(b, __fsub_rn(s, a))};
}
// Sums and products are within about 2^-46 of the larger operand, or of the product. (fp64 would be a few hundred
// clocks an operation here.)
__device__ __forceinline__ Two operator+(Two a, Two b) {
    const Two s = two_sum(a.h, b.h);
    return quick_sum(s.h, __fadd_rn(s.l, __fadd_rn(a.l, b.l)));
}
__device__ __forceinline__ Two operator-(Two a, Two b) { return a + Two{-b.h, -b.l}; }
__device__ __forceinline__ Two operator*(Two a, Two b) {
    const float p = __fmul_rn(a.h, b.h);
    return quick_sum(p, __fmaf_rn(a.l, b.h, __fmaf_rn(a.h, b.l, __fmaf_rn(a.h, b.h, -p))));
}
__device__ __forceinline__ bool operator>(Two a, Two b) { return a.h > b.h || (a.h == b.h && a.l > b.l); }

// What the choice needs of its numbers, float or Two.
template <typename F>
__device__ __forceinline__ F number(float x);
template <>
__device__ __forceinline__ float number<float>(float x) { return x; }
template <>
__device__ __forceinline__ Two number<Two>(float x) { return {x, 0.f}; }
__device__ __forceinline__ float rounded(float x) { return x; }
__device__ __forceinline__ float rounded(Two x) { return x.h; }
__device__ __forceinline__ float shift_up(float x, int d) { return __shfl_up_sync(kFull, x, d); }
__device__ __forceinline__ Two shift_up(Two x, int d) {
    return {__shfl_up_sync(kFull, x.h, d), __shfl_up_sync(kFull, x.l, d)};
}
__device__ __forceinline__ Two warp_sum(Two x) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
        x = x + Two{__shfl_xor_sync(kFull, x.h, d), __shfl_xor_sync(kFull, x.l, d)};
    return x;
}

// 2^(j / 64) in two floats.
__device__ const Two kPowers[64] = {
    {0x1.0000000000000p+0f, 0x0.0p+0f}, {0x1.02c9a40000000p+0f, -0x1.887fa00000000p-28f}, {0x1.059b0e0000000p+0f, -0x1.9d4f520000000p-25f},
    {0x1.0874520000000p+0f, -0x1.e2990e0000000p-26f}, {0x1.0b55860000000p+0f, 0x1.9f31220000000p-25f}, {0x1.0e3ec40000000p+0f, -0x1.a585cc0000000p-25f},
    {0x1.11301e0000000p+0f, -0x1.fdb4960000000p-25f}, {0x1.1429aa0000000p+0f, 0x1.d525bc0000000p-25f}, {0x1.172b840000000p+0f, -0x1.c157420000000p-27f},
    {0x1.1a35be0000000p+0f, 0x1.6df96e0000000p-25f}, {0x1.1d48740000000p+0f, -0x1.d2e8ca0000000p-25f}, {0x1.2063b80000000p+0f, 0x1.0c519a0000000p-25f},
    {0x1.2387a60000000p+0f, 0x1.ceac480000000p-25f}, {0x1.26b4560000000p+0f, 0x1.789f380000000p-26f}, {0x1.29e9e00000000p+0f, -0x1.5c04240000000p-25f},
    {0x1.2d285a0000000p+0f, 0x1.b900c20000000p-26f}, {0x1.306fe00000000p+0f, 0x1.4636e20000000p-25f}, {0x1.33c08c0000000p+0f, -0x1.b37d200000000p-25f},
    {0x1.371a740000000p+0f, -0x1.18aac60000000p-25f}, {0x1.3a7db40000000p+0f, -0x1.634c020000000p-25f}, {0x1.3dea640000000p+0f, 0x1.8246840000000p-25f},
    {0x1.4160a20000000p+0f, 0x1.f72e2a0000000p-28f}, {0x1.44e0860000000p+0f, 0x1.8624b40000000p-30f}, {0x1.486a2c0000000p+0f, -0x1.47d8660000000p-25f},
    {0x1.4bfdae0000000p+0f, -0x1.593abc0000000p-25f}, {0x1.4f9b280000000p+0f, -0x1.2c5a6c0000000p-25f}, {0x1.5342b60000000p+0f, -0x1.2c56100000000p-25f},
    {0x1.56f4740000000p+0f, -0x1.295b040000000p-25f}, {0x1.5ab07e0000000p+0f, -0x1.5bd5ec0000000p-27f}, {0x1.5e76f20000000p+0f, -0x1.4a5bd60000000p-25f},
    {0x1.6247ec0000000p+0f, -0x1.f8b5500000000p-25f}, {0x1.6623880000000p+0f, 0x1.2a91120000000p-27f}, {0x1.6a09e60000000p+0f, 0x1.9fcef40000000p-26f},
    {0x1.6dfb240000000p+0f, -0x1.cd72e80000000p-27f}, {0x1.71f75e0000000p+0f, 0x1.1d8bee0000000p-25f}, {0x1.75feb60000000p+0f, -0x1.37b3060000000p-25f},
    {0x1.7a11480000000p+0f, -0x1.829fd00000000p-25f}, {0x1.7e2f340000000p+0f, -0x1.2616340000000p-25f}, {0x1.82589a0000000p+0f, -0x1.accc7c0000000p-26f},
    {0x1.868d9a0000000p+0f, -0x1.2edb440000000p-26f}, {0x1.8ace540000000p+0f, 0x1.15506e0000000p-27f}, {0x1.8f1aea0000000p+0f, -0x1.baa2320000000p-26f},
    {0x1.93737c0000000p+0f, -0x1.e647440000000p-25f}, {0x1.97d82a0000000p+0f, -0x1.0d8d840000000p-31f}, {0x1.9c49180000000p+0f, 0x1.51f8480000000p-27f},
    {0x1.a0c6680000000p+0f, -0x1.2886a60000000p-26f}, {0x1.a5503c0000000p+0f, -0x1.b83b540000000p-25f}, {0x1.a9e6b60000000p+0f, -0x1.50c0480000000p-25f},
    {0x1.ae89fa0000000p+0f, -0x1.a94b140000000p-26f}, {0x1.b33a2c0000000p+0f, -0x1.ec3a820000000p-26f}, {0x1.b7f7700000000p+0f, -0x1.a094380000000p-25f},
    {0x1.bcc1ea0000000p+0f, -0x1.f687c60000000p-25f}, {0x1.c199be0000000p+0f, -0x1.3d56b20000000p-27f}, {0x1.c67f120000000p+0f, 0x1.cafa2a0000000p-25f},
    {0x1.cb720e0000000p+0f, -0x1.8837cc0000000p-27f}, {0x1.d072d40000000p+0f, 0x1.40f1300000000p-25f}, {0x1.d5818e0000000p+0f, -0x1.822dbc0000000p-27f},
    {0x1.da9e600000000p+0f, 0x1.ed99420000000p-27f}, {0x1.dfc9740000000p+0f, -0x1.908c940000000p-25f}, {0x1.e502ee0000000p+0f, 0x1.e2cffe0000000p-26f},
    {0x1.ea4afa0000000p+0f, 0x1.52486c0000000p-27f}, {0x1.efa1be0000000p+0f, 0x1.cc2b440000000p-25f}, {0x1.f507660000000p+0f, -0x1.246eb00000000p-26f},
    {0x1.fa7c180000000p+0f, 0x1.9e90d80000000p-28f},
};

// 1 / T in two floats: within 2^-47 of it.
__device__ __forceinline__ Two inverse(float t) {
    const float h = 1.f / t;
    return {h, h * __fmaf_rn(-t, h, 1.f)};
}

// Two of them, which the pipes take in one instruction.
struct TwoPair {
    uint64_t h, l;
};
__device__ __forceinline__ uint64_t both(float x) { return ptx::pair_of(x, x); }
__device__ __forceinline__ uint64_t minus(uint64_t a, uint64_t b) { return ptx::fma_pair(b, both(-1.f), a); }   // a - b
__device__ __forceinline__ TwoPair two_sum(uint64_t a, uint64_t b) {
    const uint64_t s = ptx::add_pair(a, b), bb = minus(s, a);
    return {s, ptx::add_pair(minus(a, minus(s, bb)), minus(b, bb))};
}

// exp((x - M) / T), within about 2^-39 of it; 0 below e^-87. With y = (x - M) / T = n ln 2 / 64 + s,
// |s| < 0.0055: e^y = 2^(n / 64) e^s, e^s by Taylor's series to s^4 (s^5 / 120 is below 2^-44), whose terms
// from s^2 on are below 2^-16 and need one float. powers: kPowers, in shared memory. Two logits at a time.
__device__ __forceinline__ TwoPair exp_two(uint64_t x, float M, Two inv_t, const Two* powers) {
    using namespace ptx;
    const TwoPair d = two_sum(x, both(-M));
    const uint64_t ih = both(inv_t.h), p = mul_pair(d.h, ih);
    const uint64_t e = fma_pair(d.l, ih, fma_pair(d.h, both(inv_t.l), fma_pair(d.h, ih, mul_pair(p, both(-1.f)))));
    const uint64_t magic = fma_pair(p, both(0x1.715476p+6f), both(12582912.f));   // 64 / ln 2; rounds to a whole
    const uint64_t n = add_pair(magic, both(-12582912.f));
    const uint64_t sh = fma_pair(n, both(-0x1.62e43p-7f), p);                // exact: ln 2 / 64 has 21 bits here
    const uint64_t sl = fma_pair(n, both(0x1.05c61p-35f), e);
    const uint64_t s = add_pair(sh, sl);
    const uint64_t tail =
        fma_pair(mul_pair(s, s), fma_pair(s, fma_pair(s, both(1.f / 24.f), both(1.f / 6.f)), both(0.5f)), sl);
    const uint64_t one = add_pair(both(1.f), sh);
    const uint64_t low = add_pair(minus(sh, add_pair(one, both(-1.f))), tail);
    const float2 m = halves_of(magic), q = halves_of(p);
    const int k0 = __float_as_int(m.x) - 0x4b400000, k1 = __float_as_int(m.y) - 0x4b400000;
    const Two b0 = powers[k0 & 63], b1 = powers[k1 & 63];
    const uint64_t bh = pair_of(b0.h, b1.h), bl = pair_of(b0.l, b1.l);
    const uint64_t h = mul_pair(one, bh);
    const uint64_t rest =
        fma_pair(low, bh, fma_pair(one, bl, fma_pair(one, bh, mul_pair(h, both(-1.f)))));
    const uint64_t scale =
        pair_of(__int_as_float(((k0 >> 6) + 127) << 23), __int_as_float(((k1 >> 6) + 127) << 23));
    const uint64_t w = add_pair(h, rest);
    const float2 wh = halves_of(mul_pair(w, scale)), wl = halves_of(mul_pair(minus(rest, minus(w, h)), scale));
    return {pair_of(q.x > -87.f ? wh.x : 0.f, q.y > -87.f ? wh.y : 0.f),
            pair_of(q.x > -87.f ? wl.x : 0.f, q.y > -87.f ? wl.y : 0.f)};
}
__device__ __forceinline__ Two exp_two(float x, float M, Two inv_t, const Two* powers) {
    const TwoPair w = exp_two(both(x), M, inv_t, powers);
    return {ptx::halves_of(w.h).x, ptx::halves_of(w.l).x};
}

// The sum of the weights of half of a tile, by a warp. stage: room for it in shared memory.
template <typename T>
__device__ __noinline__ Two exact_half(const Row<T>& x, int t, int half, float M, Two inv_t, const Two* powers,
                                       uint4* stage) {
    constexpr int kHalf = kVecs / 2, kN = Vec<T>::kN;
    const int lane = threadIdx.x & 31;
    int n;
    const uint4* from = reinterpret_cast<const uint4*>(x.x + x.body(t, n)) + half * kHalf * 32 + lane;
    uint4 v[kHalf];
#pragma unroll
    for (int k = 0; k < kHalf; ++k) {
        v[k] = make_uint4(Row<T>::kLow, Row<T>::kLow, Row<T>::kLow, Row<T>::kLow);
        if (((half * kHalf + k) * 32 + lane) * kN + kN <= n) v[k] = from[32 * k];
    }
    const float edge = half == 0 ? x.edge(t, lane) : -INFINITY;
    __syncwarp();
#pragma unroll
    for (int k = 0; k < kHalf; ++k) stage[32 * k + lane] = v[k];
    __syncwarp();
    const T* f = reinterpret_cast<const T*>(stage);
    TwoPair sum = {0, 0};
    // (Not unrolled further: the code runs once or twice, and is fetched from far.)
#pragma unroll 1
    for (int e = lane - 64; e < Row<T>::kTile / 2; e += 64) {
        const uint64_t v = e < 0 ? ptx::pair_of(edge, -INFINITY) : ptx::pair_of(to_float(f[e]), to_float(f[e + 32]));
        const TwoPair w = exp_two(v, M, inv_t, powers), to = two_sum(sum.h, w.h);
        sum = {to.h, ptx::add_pair(sum.l, ptx::add_pair(to.l, w.l))};
    }
    const float2 h = ptx::halves_of(sum.h), l = ptx::halves_of(sum.l);
    return warp_sum(Two{h.x, l.x} + Two{h.y, l.y});
}

// ---------------------------------------------------------------- the choice

constexpr int kChooseThreads = 256;
constexpr int kWarps = kChooseThreads / 32;
constexpr int kMaxK = 32;
constexpr int kTiles = kWarps / 2;                   // that the block sums exactly at a time
constexpr int kRoom = 9 * kChooseThreads * 8;        // a tile's weights, or half a tile for each warp
static_assert(kRoom >= kWarps * kVecs / 2 * 32 * 16, "half a tile for each warp");

struct ChooseShared {
    uint4 room[kRoom / 16];
    Two powers[64];
    float M[kMaxDrafts + 1], Z[kMaxDrafts + 1], logprob[kMaxDrafts + 1];
    uint8_t state[kMaxDrafts + 1];
    Two warp[kWarps];
    int owner[kWarps];
    // what the draft's distribution takes away: places and probabilities, each token once
    int n_less, less_at[kMaxK];
    Two less_q[kMaxK], less[kMaxK];
    // answers that one thread has for all
    int tile, found, unsure, taken;
    Two before;
    bool last;
};

// Inclusive running sum over the block's threads, and the sum of all.
template <typename F>
__device__ __forceinline__ F block_scan(F x, ChooseShared& sh, F& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    F* warps = reinterpret_cast<F*>(sh.warp);
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const F o = shift_up(x, d);
        if (lane >= d) x = x + o;
    }
    __syncthreads();
    if (lane == 31) warps[warp] = x;
    __syncthreads();
    F below = number<F>(0.f);
    total = number<F>(0.f);
#pragma unroll 1
    for (int w = 0; w < kWarps; ++w) {
        if (w == warp) below = total;
        total = total + warps[w];
    }
    return below + x;
}

// The first thread of the block where `here` holds, or -1.
__device__ __forceinline__ int first_thread(bool here, ChooseShared& sh) {
    const unsigned b = __ballot_sync(kFull, here);
    if ((threadIdx.x & 31) == 0) sh.owner[threadIdx.x >> 5] = b ? (int)(threadIdx.x & ~31u) + __ffs(b) - 1 : INT_MAX;
    __syncthreads();
    int owner = INT_MAX;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) owner = min(owner, sh.owner[w]);
    return owner == INT_MAX ? -1 : owner;
}

// The tile to look in after `tile` where `from` has nothing to draw: the nearest behind it with any weight, then the
// nearest before it; -1: none is left. sums: the row's tiles', each a Two. The whole block.
__device__ __forceinline__ int next_tile(const float2* sums, int tiles, int from, int tile, ChooseShared& sh) {
    const int tid = threadIdx.x;
    if (tile >= from) {
        for (int t0 = tile + 1; t0 < tiles; t0 += kChooseThreads) {
            __syncthreads();
            const int at = first_thread(t0 + tid < tiles && __ldcg(&sums[min(t0 + tid, tiles - 1)]).x > 0.f, sh);
            if (at >= 0) return t0 + at;
        }
        tile = from;
    }
    for (int t0 = tile - 1; t0 >= 0; t0 -= kChooseThreads) {
        __syncthreads();
        const int at = first_thread(t0 - tid >= 0 && __ldcg(&sums[max(t0 - tid, 0)]).x > 0.f, sh);
        if (at >= 0) return t0 - at;
    }
    return -1;
}

// Where an exact draw's tile has no weight: the first token with some in the next tile that has any, into sh.found; in
// a tile before it the last one. The whole block. (Apart from the draw, which it would slow down: seldom in need.)
template <typename T>
__device__ __noinline__ void draw_elsewhere(const VerifyPlan& p, long long row, float M, float t, ChooseShared& sh) {
    const Row<T> x(p.a, row);
    const Two inv_t = inverse(t);
    const float2* sums = p.sums + row * p.tiles;
    const int tid = threadIdx.x, from = sh.tile, taken = sh.taken;
    int found = -1;
    for (int tile = from; found < 0 && (tile = next_tile(sums, p.tiles, from, tile, sh)) >= 0;) {
        const bool behind = tile > from;
        const int lo = x.first(tile), hi = x.first(tile + 1);
        unsigned best = 0;                                           // the nearer, the larger; 0: none
        for (int v = lo + tid; v < hi; v += kChooseThreads) {
            Two w = exp_two(to_float(x.x[v]), M, inv_t, sh.powers);
            for (int k = 0; k < taken; ++k)
                if (sh.less_at[k] == v) w = w > sh.less[k] ? w - sh.less[k] : Two{0.f, 0.f};
            if (w > Two{0.f, 0.f}) best = max(best, (unsigned)(behind ? hi - v : v - lo + 1));
        }
        best = __reduce_max_sync(kFull, best);
        __syncthreads();
        if ((tid & 31) == 0) sh.owner[tid >> 5] = (int)best;
        __syncthreads();
        for (int k = 0; k < kWarps; ++k) best = max(best, (unsigned)sh.owner[k]);
        if (best) found = behind ? hi - (int)best : lo + (int)best - 1;
    }
    __syncthreads();
    if (tid == 0) sh.found = found >= 0 ? found : min(x.first(from), p.a.V - 1);
    __syncthreads();
}

template <typename T>
struct Chooser {
    const VerifyPlan& p;
    ChooseShared& sh;
    const int r;
    const Temperature temp;

    // Weight of a logit relative to the row's largest, in fp32 (F: float) or twice that.
    template <typename F>
    __device__ __forceinline__ F weight(float x, float M, Two inv_t) const {
        if constexpr (std::is_same<F, Two>::value) return exp_two(x, M, inv_t, sh.powers);
        else return x > -INFINITY ? ptx::ex2((x - M) * temp.c) : 0.f;
    }

    // Weight of a tile.
    template <typename F>
    __device__ __forceinline__ F tile_weight(long long row, int t, float M) const {
        const float2 s = __ldcg(&p.sums[row * p.tiles + t]);
        if constexpr (std::is_same<F, Two>::value) return Two{s.x, s.y};
        else return s.x == -INFINITY ? 0.f : s.y * ptx::ex2((s.x - M) * temp.c);
    }

    __device__ __forceinline__ float uniform() const {
        // numbers outside [0, 1) count as the nearer end, NaN as 0
        return fminf(fmaxf(p.a.sample_uniforms[r], 0.f), 1.f - 0x1p-24f);
    }

    // The draft's distribution in row i, each token once; ids outside the vocabulary are left out.
    __device__ void gather_less(int i, bool residual, uint32_t* status) {
        const VerifyArgs& a = p.a;
        const int lane = threadIdx.x & 31;
        if (threadIdx.x < 32) {
            int n = 0;
            if (residual) {
                const long long at = (long long)r * a.S + i;
                const int k_all = a.cand_ids ? a.K : 1;
                int id = -1;
                float q = 0.f;
                if (lane < k_all) {
                    id = a.cand_ids ? a.cand_ids[at * a.K + lane] : a.draft_tokens[at];
                    q = a.cand_ids ? a.draft_probs[at * a.K + lane] : 1.f;
                }
                const bool in = (unsigned)id < (unsigned)a.V;
                if (lane < k_all && !in && status) atomicOr(status, kStatusBadId);
                // Lanes of one id; the first of them has the sum of their q.
                const unsigned same = __match_any_sync(kFull, id);
                const bool first = in && (int)__ffs(same) - 1 == lane;
                Two sum = {q, 0.f};
                if (__any_sync(kFull, in && same != (1u << lane)))
#pragma unroll 1
                    for (int k = 0; k < 32; ++k) {
                        const float oq = __shfl_sync(kFull, q, k);
                        if ((same >> k & 1) && k != lane) sum = sum + Two{oq, 0.f};
                    }
                const unsigned firsts = __ballot_sync(kFull, first);
                if (first) {
                    const int to = __popc(firsts & ((1u << lane) - 1));
                    sh.less_at[to] = id;
                    sh.less_q[to] = sum;
                }
                n = __popc(firsts);
            }
            if (lane == 0) sh.n_less = n;
        }
        __syncthreads();
    }

    // Draws a token of the row, into sh.found; whether fp32 sums settle it. Z: the sum of weights.
    template <typename F>
    __device__ bool draw(long long row, float M, F Z) {
        constexpr bool kExact = std::is_same<F, Two>::value;
        const F zero = number<F>(0.f);
        const Row<T> x(p.a, row);
        const int tid = threadIdx.x;
        const Two inv_t = kExact ? inverse(temp.t) : Two{0.f, 0.f};
        F* less = reinterpret_cast<F*>(sh.less);
        const int n_less = sh.n_less;
        // Tiles: each thread a run of them.
        const int per = (p.tiles + kChooseThreads - 1) / kChooseThreads;
        const int t0 = min(tid * per, p.tiles), t1 = min(t0 + per, p.tiles);
        const float less_x = tid < n_less ? to_float(x.x[sh.less_at[tid]]) : 0.f;
        F run = zero, total;
#pragma unroll 1
        for (int t = t0; t < t1; ++t) run = run + tile_weight<F>(row, t, M);
        // What each candidate loses.
        if (tid < n_less) {
            const F w = weight<F>(less_x, M, inv_t);
            F qz;
            if constexpr (kExact) qz = sh.less_q[tid] * Z;
            else qz = sh.less_q[tid].h * Z;
            less[tid] = w > qz ? qz : w;
        }
        if (tid == 0) {
            sh.found = -1;
            sh.unsure = 1;
            sh.tile = p.tiles - 1;
            *reinterpret_cast<F*>(&sh.before) = zero;
        }
        __syncthreads();
        F lost = zero;
#pragma unroll 1
        for (int k = 0; k < n_less; ++k) lost = lost + less[k];
        const bool any = n_less == 0 || rounded(Z - lost) > (kExact ? 0x1p-36f : kSlack) * rounded(Z);
        if (!kExact && !any) return false;
        const int taken = any ? n_less : 0;          // nothing left over: from p itself
        if (kExact && tid == 0) sh.taken = taken;
#pragma unroll 1
        for (int k = 0; k < taken; ++k) {
            const int t = x.tile_of(sh.less_at[k]);
            if (t >= t0 && t < t1) run = run - less[k];
        }
        // The first run whose running sum passes the border has the tile.
        const F upto = block_scan(run, sh, total);
        const F border = number<F>(uniform()) * total;
        const int owner = first_thread(upto > border, sh);
        if (tid == owner) {
            F before = upto - run;
            int pick = t0;
            if (t1 - t0 > 1) {
#pragma unroll 1
                for (int t = t0; t < t1; ++t) {
                    F w = tile_weight<F>(row, t, M);
                    for (int k = 0; k < taken; ++k)
                        if (x.tile_of(sh.less_at[k]) == t) w = w - less[k];
                    pick = t;
                    if (before + w > border || t == t1 - 1) break;
                    before = before + w;
                }
            }
            sh.tile = pick;
            *reinterpret_cast<F*>(&sh.before) = before;
        }
        __syncthreads();
        // Inside the tile: its elements' weights, what the candidates lose taken away, then each thread a
        // run of them.
        constexpr int kN = Row<T>::kN;
        constexpr int kEach = ((Row<T>::kTile + kN - 1 + kChooseThreads - 1) / kChooseThreads) | 1;   // odd: no bank conflicts
        static_assert(kEach * kChooseThreads * sizeof(F) <= kRoom, "a tile's weights fit");
        F* w = reinterpret_cast<F*>(sh.room);
        const int tile = sh.tile;
        const F before = *reinterpret_cast<F*>(&sh.before);
        const int lo = x.first(tile), n = x.first(tile + 1) - lo;
        {
            // A vector a thread; what is in none, one by one; 0 behind the end.
            int whole;
            const int skip = x.body(tile, whole) - lo;               // elements before the first vector
            float l[kN];
            const bool full = (tid + 1) * kN <= whole;
            if (full) Vec<T>::widen(reinterpret_cast<const uint4*>(x.x + lo + skip)[tid], l);
#pragma unroll 1
            for (int e = tid; e < kEach * kChooseThreads; e += kChooseThreads) {
                const bool outside = e < skip || (e >= skip + (whole & -kN) && e < n);
                if (outside) w[e] = weight<F>(to_float(x.x[lo + e]), M, inv_t);
                else if (e >= n) w[e] = zero;
            }
            if (full) {
#pragma unroll
                for (int k = 0; k < kN; ++k) w[skip + tid * kN + k] = weight<F>(l[k], M, inv_t);
            }
        }
        __syncthreads();
        if (tid < taken) {
            const int e = sh.less_at[tid] - lo;
            if (e >= 0 && e < n) w[e] = w[e] > less[tid] ? w[e] - less[tid] : zero;
        }
        __syncthreads();
        const F* own = w + tid * kEach;
        run = zero;
#pragma unroll 1
        for (int e = 0; e < kEach; ++e) run = run + own[e];
        F in_tile;
        const F here = before + block_scan(run, sh, in_tile);
        int holder = first_thread(run > zero && here > border, sh);
        // The tile's sum and its elements' may differ by a rounding: then the last with any weight. (The tile may have
        // none: where the candidates took all of it, rounding may have left some of its sum.)
        if (holder < 0) {
            if (!kExact) return false;
            __syncthreads();
            const unsigned b = __ballot_sync(kFull, run > zero);
            if ((tid & 31) == 0) sh.owner[tid >> 5] = b ? tid + 31 - __clz(b) : -1;
            __syncthreads();
            for (int k = 0; k < kWarps; ++k) holder = max(holder, sh.owner[k]);
        }
        if (tid == holder) {
            F at = here - run, after = at;
            int pick = -1;
#pragma unroll 1
            for (int e = 0; e < kEach && !(pick >= 0 && after > border); ++e) {
                if (!(own[e] > zero)) continue;
                if (pick >= 0) at = after;
                pick = e;
                after = at + own[e];
            }
            if (pick >= 0) sh.found = lo + tid * kEach + pick;
            const float slack = kSlack * rounded(Z);
            sh.unsure = pick < 0 || rounded(border - at) < slack || rounded(after - border) < slack;
        }
        __syncthreads();
        return kExact || !sh.unsure;
    }

    // The first of a row's largest logits. One warp.
    __device__ int argmax(long long row, float M) const {
        const Row<T> x(p.a, row);
        const int lane = threadIdx.x & 31;
        const float2* sums = p.sums + row * p.tiles;
        unsigned tile = INT_MAX;
        for (int t0 = 0; t0 < p.tiles && tile == INT_MAX; t0 += 128) {
            float m[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int t = t0 + 32 * k + lane;
                m[k] = t < p.tiles ? __ldcg(&sums[t].x) : -INFINITY;
            }
#pragma unroll
            for (int k = 3; k >= 0; --k) {
                const unsigned b = __ballot_sync(kFull, m[k] == M && t0 + 32 * k + lane < p.tiles);
                if (b) tile = t0 + 32 * k + __ffs(b) - 1;
            }
        }
        if (tile == INT_MAX) return -1;                              // no tile has it (not so for a row's M)
        uint4 v[kVecs];
        int n;
        const int body = x.body((int)tile, n);
        const float edge = x.edge((int)tile, lane);
        x.load((int)tile, lane, reinterpret_cast<const uint4*>(x.x + body), v);
        unsigned best = UINT_MAX;
        constexpr int kN = Vec<T>::kN;
#pragma unroll
        for (int k = 0; k < kVecs; ++k) {
            float f[kN];
            Vec<T>::widen(v[k], f);
#pragma unroll
            for (int e = kN - 1; e >= 0; --e)
                if (f[e] == M) best = min(best, (unsigned)(body + (k * 32 + lane) * kN + e));
        }
        if (edge == M) best = min(best, (unsigned)(lane < 16 ? lane : body + n - (n & (kN - 1)) + lane - 16));
        return (int)__reduce_min_sync(kFull, best);
    }

    // Looks at row i of the request, one of n; one warp.
    __device__ void look(long long row, int i, int n) {
        const VerifyArgs& a = p.a;
        const int lane = threadIdx.x & 31;
        float M, Z;
        const bool drafted = i < n - 1;
        const long long at = (long long)r * a.S + i;
        const int token = drafted ? a.draft_tokens[at] : -1;
        const bool in = (unsigned)token < (unsigned)a.V;
        const float l = in ? to_float(Row<T>(a, row).x[token]) : 0.f;
        const float u = drafted ? a.accept_uniforms[at] : 0.f;
        const float q = drafted ? draft_probability(a, at, token, lane) : 0.f;
        join_tiles(p.sums + row * p.tiles, p.tiles, temp.c, lane, M, Z);
        int state = kRejected;
        float logprob = 0.f;
        if (!(Z > 0.f)) {
            state = kBad;
        } else if (in) {
            if (temp.greedy) {
                state = l == M && argmax(row, M) == token ? kTaken : kRejected;
            } else {
                const float z = (l - M) * temp.c, w = ptx::ex2(z), uq = u * q * Z;
                // (Both are 0 where a draft is masked and u or q is 0: 0 < 0 does not hold.)
                state = fabsf(uq - w) < draft_slack(uq, w, z) ? kUnsure : uq < w ? kTaken : kRejected;
                logprob = (l - M) / temp.t - logf(Z);
            }
        }
        if (lane == 0) {
            sh.M[i] = M;
            sh.Z[i] = Z;
            sh.state[i] = (uint8_t)state;
            sh.logprob[i] = logprob;
        }
    }

    // Whether draft i, in doubt, is taken: its row's sum again in twice the precision. The whole block.
    __device__ __noinline__ bool taken_exactly(long long row, int i) {
        const VerifyArgs& a = p.a;
        const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
        const Row<T> x(a, row);
        const float M = sh.M[i];
        for (int k = tid; k < 64; k += kChooseThreads) sh.powers[k] = kPowers[k];
        __syncthreads();
        const Two inv_t = inverse(temp.t);
        Two mine = {0.f, 0.f}, Z;
        for (int t = warp >> 1; t < p.tiles; t += kTiles) {
            const Two sum = exact_half<T>(x, t, warp & 1, M, inv_t, sh.powers, sh.room + warp * kVecs / 2 * 32);
            if (lane == 0) mine = mine + sum;
        }
        block_scan(mine, sh, Z);
        const long long at = (long long)r * a.S + i;
        const int token = a.draft_tokens[at];
        const Two w = weight<Two>(to_float(x.x[token]), M, inv_t);
        Two q = {1.f, 0.f};
        if (a.cand_ids) {
            const bool here = lane < a.K && a.cand_ids[at * a.K + lane] == token;
            q = warp_sum(Two{here ? a.draft_probs[at * a.K + lane] : 0.f, 0.f});
        }
        return w > Two{a.accept_uniforms[at], 0.f} * q * Z;
    }

    __device__ void run(uint32_t* status) {
        const VerifyArgs& a = p.a;
        const int tid = threadIdx.x, warp = tid >> 5;
        const int start = a.query_start[r], end = a.query_start[r + 1];
        int32_t* tokens = a.tokens + (long long)r * (a.S + 1);
        float* logprobs = a.logprobs ? a.logprobs + (long long)r * (a.S + 1) : nullptr;
        const bool bad = bad_rows(a, start, end);
        const int n = bad ? 0 : end - start;
        const int rows = p.alive && n > 0 ? p.alive[r] + 1 : n;
        for (int i = warp; i < rows; i += kWarps) look(start + i, i, n);
        __syncthreads();
        // The drafts in order.
        int i = 0;
        for (; i < rows; ++i) {
            const int state = sh.state[i];
            if (state == kTaken || (state == kUnsure && taken_exactly(start + i, i))) continue;
            break;
        }
        int count = i, drawn = -1;
        float last_logprob = 0.f;
        if (i < rows && sh.state[i] != kBad) {
            const long long row = start + i;
            const float M = sh.M[i], Z = sh.Z[i];
            count = i + 1;
            if (temp.greedy) {
                drawn = argmax(row, M);
            } else {
                gather_less(i, i < n - 1, status);
                if (draw<float>(row, M, Z)) {
                    drawn = sh.found;
                    last_logprob = (to_float(Row<T>(a, row).x[drawn]) - M) / temp.t - logf(Z);
                } else if (tid == 0) {
                    p.list[atomicAdd(p.listed, 1u)] = Unsettled{r, i, M, 0u};
                }
            }
        }
        for (int k = tid; k <= a.S; k += kChooseThreads) {
            tokens[k] = k < i ? a.draft_tokens[(long long)r * a.S + k] : k < count ? drawn : -1;
            if (logprobs) logprobs[k] = k < i ? sh.logprob[k] : k < count ? last_logprob : 0.f;
        }
        if (tid == 0) {
            a.counts[r] = count;
            if (bad) atomicOr(status, kStatusBadLength);
            if (i < rows && sh.state[i] == kBad) atomicOr(status, kStatusBadLogits);
            // a draft that was looked at and is no token
            if (i < n - 1 && i < rows && (unsigned)a.draft_tokens[(long long)r * a.S + i] >= (unsigned)a.V)
                atomicOr(status, kStatusBadId);
        }
    }

    // Writes the token that a listed row's exact sums draw.
    __device__ void settle(const Unsettled& u) {
        const VerifyArgs& a = p.a;
        const int tid = threadIdx.x;
        const int start = a.query_start[r], n = a.query_start[r + 1] - start;
        const long long row = start + u.i;
        Two mine = {0.f, 0.f}, Z;
        for (int t = tid; t < p.tiles; t += kChooseThreads) mine = mine + tile_weight<Two>(row, t, u.M);
        block_scan(mine, sh, Z);
        gather_less(u.i, u.i < n - 1, nullptr);
        draw<Two>(row, u.M, Z);
        if (sh.found < 0) draw_elsewhere<T>(p, row, u.M, temp.t, sh);
        if (tid == 0) {
            const long long at = (long long)r * (a.S + 1) + u.i;
            a.tokens[at] = sh.found;
            if (a.logprobs)
                a.logprobs[at] = (to_float(Row<T>(a, row).x[sh.found]) - u.M) / temp.t - logf(Z.h);
        }
    }
};

template <typename T>
__global__ void __launch_bounds__(kChooseThreads)
choose_kernel(const __grid_constant__ VerifyPlan p, uint32_t* status) {
    __shared__ ChooseShared sh;
    ptx::grid_dependents_launch();
    ptx::grid_dependency_wait();
    const int r = blockIdx.x;
    Chooser<T> chooser{p, sh, r, Temperature(p.a, r)};
    chooser.run(status);
}

// Items are kTiles tiles of a listed row, two warps a tile; the CTA that finishes a row's last draws its token. 8 rows
// of 151936 bf16 logits: 22 us, 12 of them until the tiles' sums are there and 8 for the draw, each a chain of steps
// that wait for one another. (With fp64 sums 37. To run the code once before the wait, for the instructions: no gain.)
template <typename T>
__global__ void __launch_bounds__(kChooseThreads) settle_kernel(const __grid_constant__ VerifyPlan p) {
    __shared__ ChooseShared sh;
    ptx::grid_dependency_wait();
    const int tid = threadIdx.x, warp = tid >> 5;
    const unsigned n = __ldcg(p.listed);
    if (n == 0) return;
    if (tid < 64) sh.powers[tid] = kPowers[tid];
    const int chunks = (p.tiles + kTiles - 1) / kTiles;
    for (long long item = blockIdx.x; item < (long long)n * chunks; item += gridDim.x) {
        const int at = (int)(item / chunks), first = (int)(item - (long long)at * chunks) * kTiles;
        const Unsettled u{__ldcg(&p.list[at].r), __ldcg(&p.list[at].i), __ldcg(&p.list[at].M), 0u};
        const Temperature temp(p.a, u.r);
        const long long row = p.a.query_start[u.r] + u.i;
        __syncthreads();
        const int t = first + (warp >> 1);
        if (t < p.tiles) {
            const Two half = exact_half<T>(Row<T>(p.a, row), t, warp & 1, u.M, inverse(temp.t), sh.powers,
                                           sh.room + warp * kVecs / 2 * 32);
            if ((tid & 31) == 0) sh.warp[warp] = half;
        }
        __syncthreads();
        if (tid < kTiles && first + tid < p.tiles) {
            const Two sum = sh.warp[2 * tid] + sh.warp[2 * tid + 1];
            __stcg(&p.sums[row * p.tiles + first + tid], make_float2(sum.h, sum.l));
        }
        __syncwarp();
        if (tid == 0) {
            __threadfence();
            sh.last = atomicAdd(&p.list[at].arrived, 1u) + 1u == (unsigned)chunks;
            __threadfence();
        }
        __syncthreads();
        if (sh.last) {
            Chooser<T> chooser{p, sh, u.r, temp};
            chooser.settle(u);
        }
    }
}

// The workspace: the list's length, the list, requests' and rows' counters, the tiles' sums.
size_t padded_bytes(size_t n) { return (n + 255) & ~(size_t)255; }
size_t list_bytes(int R) { return padded_bytes(16 + (size_t)R * sizeof(Unsettled)); }
// (Counters are by position and request, (S + 1) R of them, of which at most T + R are of use: where they are more
// than 4 (T + R), because few requests have many rows, rows are not passed over. 512 requests of up to 16 rows of 151936
// bf16 logits, 1535 and 1536 rows in all, read whole and passed over: 218 and 189 us; 68 and 69 of them with 16 rows, the others
// with one: 255 and 239. Read whole, each empty place is looked at: 512 single rows 200 us with S = 0, 233 with S = 15.)
size_t counter_bytes(int R, int T) { return padded_bytes((4 * ((size_t)T + R) + R + 8) * 4); }

int tiles_of(int V, int size) {
    const int tile = kVecs * 32 * 16 / size;
    return (int)(((long long)V + tile - 1) / tile);
}

// dependent: as the programmatic dependent of the kernel before it.
template <typename Kernel, typename... Args>
cudaError_t launch_kernel(Kernel kernel, unsigned blocks, int threads, int smem, bool dependent,
                          cudaStream_t stream, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = dependent ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <typename T>
cudaError_t launch(const DeviceInfo& dev, const VerifyArgs& a, void* workspace, uint32_t* status,
                   cudaStream_t stream) {
    VerifyPlan p{};
    p.a = a;
    p.tiles = tiles_of(a.V, (int)sizeof(T));
    p.chunks = (p.tiles + kSumWarps - 1) / kSumWarps;
    p.padded = (a.R + 3) & ~3;
    p.by_chunks = Divisor((unsigned)p.chunks);
    p.by_R = Divisor((unsigned)a.R);
    p.by_padded = Divisor((unsigned)p.padded);
    char* at = static_cast<char*>(workspace);
    p.listed = reinterpret_cast<unsigned*>(at);
    p.list = reinterpret_cast<Unsettled*>(at + 16);
    p.sums = reinterpret_cast<float2*>(at + list_bytes(a.R) + counter_bytes(a.R, a.T));
    const long long items = (long long)(a.S + 1) * a.R * p.chunks;
    const long long most = (long long)kSumBlocks * dev.sm_count;
    const long long rows = (long long)(a.S + 1) * p.padded;
    // Rows are passed over where they are many to each CTA: that costs a launch and the looks for items, 3 to 6 us,
    // and saves what is not read. (151936 logits of 2 bytes, without and with it: 8 requests of 8 rows 26 and 30 us,
    // 32 of 8 38 and 43, 48 of 8 (items = 12.6 most) 64 and 63, 24 of 16 67 and 63, 64 of 16 108 and 86.)
    const bool pass_over = items > 12 * most && a.S > 0 && rows <= 4 * ((long long)a.T + a.R) && rows < 1 << 30;
    if (pass_over) {
        p.alive = reinterpret_cast<int*>(at + list_bytes(a.R));
        p.handed = p.alive + p.padded;
        // To find an item takes about 2500 clocks, much of it waiting for other SMs' counts, and all CTAs ask at few
        // addresses: up to 5 at a time (160 KB), a row in equal parts, where a position has 1.5 such groups for each
        // CTA. (One at a time / 2 / 5 / 8 / whole rows of 10: 512 greedy requests 298, 259, 234, 239 and 226 us, 256 of
        // them 167, 153, 146, 151 and 145; 64 sampled ones 87, 89, 94, 99 and 101, and over rows of 32 items 130, 126, 134,
        // 147 and 160: more is read that is not needed.)
        const int most_group = (int)std::min(5LL, std::max(1LL, (long long)a.R * p.chunks * 2 / (3 * most)));
        p.groups = (p.chunks + most_group - 1) / most_group;
        p.group = (p.chunks + p.groups - 1) / p.groups;
        p.window = (int)std::min(256LL, std::max(1LL, 2 * most / p.groups));
        const long long most_start = (long long)a.T * p.tiles / (2 * 8 * kStartThreads) + 1;
        start_kernel<<<(unsigned)std::min(most_start, 4LL * dev.sm_count), kStartThreads, 0, stream>>>(p);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    const unsigned blocks = (unsigned)std::min(items, most);
    constexpr int smem = kSlots * kSlotBytes;
    static std::once_flag once[64];
    static cudaError_t attr_err[64];
    if (dev.device < 0 || dev.device >= 64) return cudaErrorInvalidDevice;
    std::call_once(once[dev.device], [&] {
        attr_err[dev.device] =
            cudaFuncSetAttribute(row_sums_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    });
    if (attr_err[dev.device] != cudaSuccess) return attr_err[dev.device];
    cudaError_t e = launch_kernel(row_sums_kernel<T>, blocks, kSumThreads, smem, pass_over, stream, p, status);
    if (e != cudaSuccess) return e;
    e = launch_kernel(choose_kernel<T>, (unsigned)a.R, kChooseThreads, 0, true, stream, p, status);
    if (e != cudaSuccess) return e;
    // More CTAs than fit at once, since the last ones of a row also draw (512 requests of 8 rows of 262144 fp32 logits:
    // 456, 425 and 412 us with 3, 5 and 8 an SM).
    const long long chunks = (long long)a.R * ((p.tiles + kTiles - 1) / kTiles);
    return launch_kernel(settle_kernel<T>, (unsigned)std::min(chunks, 8LL * dev.sm_count), kChooseThreads, 0,
                         true, stream, p);
}

}  // namespace

size_t verify_workspace_bytes(int R, int T, int V) {
    return list_bytes(R) + counter_bytes(R, T) + padded_bytes((size_t)T * tiles_of(V, 4) * sizeof(float2));
}

cudaError_t launch_verify(const DeviceInfo& dev, const VerifyArgs& a, void* workspace,
                          uint32_t* status_word, cudaStream_t stream) {
    if (a.dtype == kFp32) return launch<float>(dev, a, workspace, status_word, stream);
    if (a.dtype == kBf16) return launch<__nv_bfloat16>(dev, a, workspace, status_word, stream);
    return launch<__half>(dev, a, workspace, status_word, stream);
}

}  // namespace dflash
