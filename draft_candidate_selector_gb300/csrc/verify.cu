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
// Rows behind the first rejected draft are not needed. Where the batch is large, row_sums goes through
// the requests' first rows, then their second ones, and so on; the warp that finishes a row looks whether
// its draft is surely rejected, and later rows of that request are passed over.
// Bound by HBM: the rows up to the first rejected draft are read once.
#include "common.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cfloat>
#include <climits>
#include <cmath>
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

// 2^x, within 2^-22 of it; results below 2^-126 are 0.
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// A row's tiles. The row starts `head` elements before its first 16-byte boundary; tile 0 also has
// those, and tile t has the elements from first(t) to first(t + 1), so every other tile starts on one.
constexpr int kVecs = 8;                         // 16-byte vectors of a tile a lane holds
template <typename T>
struct Row {
    static constexpr int kN = Vec<T>::kN;
    static constexpr int kTile = kVecs * 32 * kN;
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

    // Tile t's whole vectors, a warp's lanes side by side, -inf where there are none; and of the elements
    // at its ends that are in none, at most one a lane, or -inf.
    __device__ __forceinline__ void load(int t, int lane, uint4 (&v)[kVecs], float& edge) const {
        const int hi = first(t + 1), body = t == 0 ? min(head, hi) : first(t), n = hi - body;
        const uint32_t low = sizeof(T) == 4 ? 0xff800000u
                                            : std::is_same<T, __half>::value ? 0xfc00fc00u : 0xff80ff80u;
        const T* base = x + body;
#pragma unroll
        for (int k = 0; k < kVecs; ++k) {
            const int e = (k * 32 + lane) * kN;
            v[k] = make_uint4(low, low, low, low);
            if (e + kN <= n) v[k] = __ldcs(reinterpret_cast<const uint4*>(base + e));
        }
        edge = -INFINITY;
        const int rest = n & (kN - 1);
        if (t == 0 && lane < head && lane < hi) edge = to_float(x[lane]);
        if (lane >= 16 && lane - 16 < rest) edge = to_float(base[n - rest + lane - 16]);
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

struct VerifyPlan {
    VerifyArgs a;
    int tiles;                // of a row
    float2* sums;             // [T][tiles]: the largest logit, the sum of exp((x - it) / T); settle: a double
    Unsettled* list;          // [R]
    unsigned* listed;         // how many
    uint32_t* dead;           // [R] a row at and before the first rejected; null: rows are not left out
    uint32_t* arrived;        // [T] tiles of the row that are done, less one (as a wrapped number)
};

__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) x = fmaxf(x, __shfl_xor_sync(kFull, x, d));
    return x;
}
template <typename F>
__device__ __forceinline__ F warp_sum(F x) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(kFull, x, d);
    return x;
}

// The largest logit of a row and the sum of its weights relative to it, from the tiles' sums, by a
// warp. The sum is NaN where the row has a NaN or +inf, and 0 where all of it is -inf.
__device__ __forceinline__ void join_tiles(const float2* sums, int tiles, float c, int lane, float& M,
                                           float& Z) {
    constexpr int kHeld = 8;
    float2 s[kHeld];
    M = -INFINITY;
#pragma unroll
    for (int k = 0; k < kHeld; ++k) {
        s[k] = make_float2(-INFINITY, 0.f);
        if (k * 32 + lane < tiles) s[k] = __ldcg(&sums[k * 32 + lane]);
    }
    for (int t = kHeld * 32 + lane; t < tiles; t += 32) M = fmaxf(M, __ldcg(&sums[t].x));
#pragma unroll
    for (int k = 0; k < kHeld; ++k) M = fmaxf(M, s[k].x);
    M = warp_max(M);
    Z = 0.f;
    auto part = [&](float2 x) {
        return x.y * (x.x == -INFINITY ? (x.y == x.y ? 0.f : 1.f) : exp2_fast((x.x - M) * c));
    };
#pragma unroll
    for (int k = 0; k < kHeld; ++k) Z += part(s[k]);
    for (int t = kHeld * 32 + lane; t < tiles; t += 32) Z += part(__ldcg(&sums[t]));
    Z = warp_sum(Z);
}

// q of token x in row (r, i), by a warp.
template <typename F>
__device__ __forceinline__ F draft_probability(const VerifyArgs& a, long long at, int x, int lane) {
    if (!a.cand_ids) return F(1);
    F q = 0;
    if (lane < a.K && a.cand_ids[at * a.K + lane] == x) q = a.draft_probs[at * a.K + lane];
    return warp_sum(q);
}

// ---------------------------------------------------------------- sums of tiles

// Error of the fp32 sums, relative to a row's sum: an element's exponent is rounded once in the
// difference and its T 2^-22.4 off, so the sum is within 2^-22 sum p |z| <= 2^-22 (ln V + 1); ex2 is within
// 2^-22, at most 24 additions in a row within 24 * 2^-24, joining the tiles (a difference, a product,
// an exponential, additions) no more than that again. In all below 2^-17 for V < 2^31.
constexpr float kSlack = 0x1p-16f;

constexpr int kSumThreads = 256;
constexpr int kSumWarps = kSumThreads / 32;

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
    float s[4] = {0.f, 0.f, 0.f, 0.f};
    const float mc = __fmul_rn(m, c);
    if (fabsf(mc) < 0x1p60f) {
        // x c - mc in one rounding; mc's own is taken back at the end.
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            float x[kN];
            Vec<T>::widen(v[i], x);
#pragma unroll
            for (int e = 0; e < kN; ++e) s[e & 3] += exp2_fast(fmaf(x[e], c, -mc));
        }
        return ((s[0] + s[1]) + (s[2] + s[3])) * exp2_fast(-fmaf(m, c, -mc));
    }
    const float ref = fmaxf(m, -FLT_MAX);
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
        float x[kN];
        Vec<T>::widen(v[i], x);
#pragma unroll
        for (int e = 0; e < kN; ++e) s[e & 3] += exp2_fast((x[e] - ref) * c);
    }
    return (s[0] + s[1]) + (s[2] + s[3]);
}

// Whether draft i of request r, in a row whose tiles are all done, is surely rejected. A warp.
template <typename T>
__device__ __noinline__ bool surely_rejected(const VerifyPlan& p, int r, int i, long long row) {
    const VerifyArgs& a = p.a;
    const int lane = threadIdx.x & 31;
    const Temperature temp(a, r);
    float M, Z;
    join_tiles(p.sums + row * p.tiles, p.tiles, temp.c, lane, M, Z);
    if (!(Z > 0.f)) return true;                     // no distribution: the request ends here
    const long long draft = (long long)r * a.S + i;
    const int token = a.draft_tokens[draft];
    if ((unsigned)token >= (unsigned)a.V) return true;
    const float l = to_float(Row<T>(a, row).x[token]);
    if (temp.greedy) return l < M;
    const float q = draft_probability<float>(a, draft, token, lane);
    const float z = (l - M) * temp.c;
    const float w = exp2_fast(z), uq = a.accept_uniforms[draft] * q * Z;
    return uq > w * (1.f + kSlack - z * 0x1p-20f) + kSlack * uq;
}

// A warp takes tiles at the distance of all warps, rows of the requests' first drafts first. Whether a
// tile completed its row is looked at a tile later, when the count has long come back.
template <typename T>
__global__ void __launch_bounds__(kSumThreads, 4) row_sums_kernel(const __grid_constant__ VerifyPlan p) {
    const VerifyArgs& a = p.a;
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.listed = 0;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int lane = threadIdx.x & 31;
    const int warps = gridDim.x * kSumWarps;
    const int step_t = warps % p.tiles, step_at = warps / p.tiles;
    const int w = blockIdx.x * kSumWarps + (threadIdx.x >> 5);
    int t = w % p.tiles, i = w / p.tiles / a.R, r = w / p.tiles - i * a.R;
    long long judge = -1;                            // the row before: its last arrival is under way
    int judge_r = 0, judge_i = 0;
    unsigned arrival = 0;
    auto judge_last = [&]() {
        if (judge < 0) return;
        const long long row = judge;
        judge = -1;
        if (__shfl_sync(kFull, arrival, 0) + 2u != (uint32_t)p.tiles) return;
        __syncwarp();
        const bool rejected = surely_rejected<T>(p, judge_r, judge_i, row);
        if (rejected && lane == 0) atomicMin(&p.dead[judge_r], (uint32_t)judge_i);
    };
    while (i <= a.S) {
        const int start = a.query_start[r], end = a.query_start[r + 1];
        // lengths that the choice refuses, and rows that the request does not have
        bool here = !bad_rows(a, start, end) && i < end - start;
        if (here && p.dead) here = __shfl_sync(kFull, lane == 0 ? __ldcg(&p.dead[r]) : 0u, 0) >= (uint32_t)i;
        if (here) {
            const long long row = start + i;
            const Row<T> x(a, row);
            uint4 v[kVecs];
            float edge;
            x.load(t, lane, v, edge);
            const float c = Temperature(a, r).c;
            const float m = warp_max(fmaxf(edge, largest<T>(v)));
            float s = weight_sum<T>(v, m, c);
            s += exp2_fast((edge - fmaxf(m, -FLT_MAX)) * c);
            s = warp_sum(s);
            judge_last();
            if (lane == 0) __stcg(&p.sums[row * p.tiles + t], make_float2(m, s));
            if (p.dead && i < end - start - 1) {
                if (lane == 0)
                    asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;"
                                 : "=r"(arrival) : "l"(&p.arrived[row]) : "memory");
                judge = row;
                judge_r = r;
                judge_i = i;
            }
        } else {
            judge_last();
        }
        t += step_t;
        r += step_at;
        if (t >= p.tiles) {
            t -= p.tiles;
            ++r;
        }
        if (r >= a.R) {
            const int q = r / a.R;
            i += q;
            r -= q * a.R;
        }
    }
    judge_last();
}

// ---------------------------------------------------------------- sums of twice the precision

// A value as the sum of two floats.
struct Two {
    float h, l;
};
__device__ __forceinline__ Two two_sum(float a, float b) {        // exact
    const float s = __fadd_rn(a, b), bb = __fsub_rn(s, a);
    return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, bb)), __fsub_rn(b, bb))};
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

// exp((x - M) / T), within about 2^-39 of it; 0 below e^-87. With y = (x - M) / T = n ln 2 / 64 + s,
// |s| < 0.0055: e^y = 2^(n / 64) e^s, e^s by Taylor's series to s^4 (s^5 / 120 is below 2^-44), whose terms
// from s^2 on are below 2^-16 and need one float. powers: kPowers, in shared memory.
__device__ __forceinline__ Two exp_two(float x, float M, Two inv_t, const Two* powers) {
    const Two d = two_sum(x, -M);
    const float p = __fmul_rn(d.h, inv_t.h);
    const float e = __fmaf_rn(d.l, inv_t.h, __fmaf_rn(d.h, inv_t.l, __fmaf_rn(d.h, inv_t.h, -p)));
    const float magic = __fmaf_rn(p, 0x1.715476p+6f, 12582912.f);          // 64 / ln 2; rounds to a whole
    const float n = __fsub_rn(magic, 12582912.f);
    const int k = __float_as_int(magic) - 0x4b400000;
    const float sh = __fmaf_rn(n, -0x1.62e43p-7f, p);                       // exact: ln 2 / 64 has 21 bits here
    const float sl = __fmaf_rn(n, 0x1.05c61p-35f, e);
    const float s = __fadd_rn(sh, sl);
    const float tail = __fmaf_rn(__fmul_rn(s, s), __fmaf_rn(s, __fmaf_rn(s, 1.f / 24.f, 1.f / 6.f), 0.5f), sl);
    const float one = __fadd_rn(1.f, sh);
    const float low = __fadd_rn(__fsub_rn(sh, __fsub_rn(one, 1.f)), tail);
    const Two b = powers[k & 63];
    const float h = __fmul_rn(one, b.h);
    const float l = __fmaf_rn(low, b.h, __fmaf_rn(one, b.l, __fmaf_rn(one, b.h, -h)));
    const float scale = __int_as_float(((k >> 6) + 127) << 23);
    const bool some = p > -87.f;
    return {some ? h * scale : 0.f, some ? l * scale : 0.f};
}

// The sum of a tile's weights, by a warp.
template <typename T>
__device__ __noinline__ double exact_tile(const Row<T>& x, int t, float M, Two inv_t, const Two* powers) {
    constexpr int kN = Vec<T>::kN;
    const int lane = threadIdx.x & 31;
    const int hi = x.first(t + 1), body = t == 0 ? min(x.head, hi) : x.first(t), n = hi - body;
    const T* base = x.x + body;
    Two sum[2] = {{0.f, 0.f}, {0.f, 0.f}};
    auto add = [&](float f, int to) {
        const Two w = exp_two(f, M, inv_t, powers), s = two_sum(sum[to].h, w.h);
        sum[to] = {s.h, sum[to].l + (s.l + w.l)};
    };
    const int rest = n & (kN - 1);
    if (t == 0 && lane < x.head && lane < hi) add(to_float(x.x[lane]), 0);
    if (lane >= 16 && lane - 16 < rest) add(to_float(base[n - rest + lane - 16]), 0);
    uint4 next = make_uint4(0, 0, 0, 0);
    if (lane * kN + kN <= n) next = *reinterpret_cast<const uint4*>(base + lane * kN);
#pragma unroll 1
    for (int e = lane * kN; e + kN <= n; e += 32 * kN) {
        float f[kN];
        Vec<T>::widen(next, f);
        if (e + 33 * kN <= n) next = *reinterpret_cast<const uint4*>(base + e + 32 * kN);
#pragma unroll
        for (int k = 0; k < kN; ++k) add(f[k], k & 1);
    }
    return warp_sum(((double)sum[0].h + (double)sum[1].h) + ((double)sum[0].l + (double)sum[1].l));
}

// ---------------------------------------------------------------- the choice

constexpr int kChooseThreads = 256;
constexpr int kWarps = kChooseThreads / 32;
constexpr int kMaxK = 32;
enum : int { kTaken = 0, kRejected = 1, kUnsure = 2, kBad = 3 };

struct ChooseShared {
    Two powers[64];
    float M[kMaxDrafts + 1], Z[kMaxDrafts + 1], logprob[kMaxDrafts + 1];
    uint8_t state[kMaxDrafts + 1];
    double warp[kWarps];
    int owner[kWarps];
    // what the draft's distribution takes away: places and probabilities, each token once
    int n_less, less_at[kMaxK];
    double less_q[kMaxK], less[kMaxK];
    // answers that one thread has for all
    int tile, found, unsure;
    double before;
    double total;
    bool last;
};

// Inclusive running sum over the block's threads, and the sum of all.
template <typename F>
__device__ __forceinline__ F block_scan(F x, ChooseShared& sh, F& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    F* warps = reinterpret_cast<F*>(sh.warp);
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const F o = __shfl_up_sync(kFull, x, d);
        if (lane >= d) x += o;
    }
    __syncthreads();
    if (lane == 31) warps[warp] = x;
    __syncthreads();
    if (sizeof(F) == 8) {                            // fp64 is slow here: one warp takes the warps' sums
        if (warp == 0) {
            F s = lane < kWarps ? warps[lane] : F(0);
#pragma unroll
            for (int d = 1; d < kWarps; d <<= 1) {
                const F o = __shfl_up_sync(kFull, s, d);
                if (lane >= d) s += o;
            }
            __syncwarp();
            if (lane < kWarps) warps[lane] = s;
        }
        __syncthreads();
        total = warps[kWarps - 1];
        return warp ? warps[warp - 1] + x : x;
    }
    F below = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w == warp) below = total;
        total += warps[w];
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

template <typename T>
struct Chooser {
    const VerifyPlan& p;
    ChooseShared& sh;
    const int r;
    const Temperature temp;

    // Weight of a logit relative to the row's largest, in fp32 (F: float) or twice that.
    template <typename F>
    __device__ __forceinline__ F weight(float x, float M) const {
        if (sizeof(F) == 8) {
            const Two w = exp_two(x, M, inverse(temp.t), sh.powers);
            return (F)w.h + (F)w.l;
        }
        return (F)exp2_fast((x - M) * temp.c);
    }

    // Weight of a tile.
    template <typename F>
    __device__ __forceinline__ F tile_weight(long long row, int t, float M) const {
        const float2* sums = p.sums + row * p.tiles;
        if (sizeof(F) == 8) return (F)__ldcg(reinterpret_cast<const double*>(sums) + t);
        const float2 s = __ldcg(&sums[t]);
        return s.x == -INFINITY ? (F)0 : (F)(s.y * exp2_fast((s.x - M) * temp.c));
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
                double sum = q;
                if (__any_sync(kFull, in && same != (1u << lane)))
                    for (int k = 0; k < 32; ++k) {
                        const float oq = __shfl_sync(kFull, q, k);
                        if ((same >> k & 1) && k != lane) sum += oq;
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
        constexpr bool kExact = sizeof(F) == 8;
        const Row<T> x(p.a, row);
        const int tid = threadIdx.x;
        F* less = reinterpret_cast<F*>(sh.less);
        const int n_less = sh.n_less;
        // What each candidate loses.
        if (tid < n_less) {
            const F w = weight<F>(to_float(x.x[sh.less_at[tid]]), M), qz = (F)sh.less_q[tid] * Z;
            less[tid] = w < qz ? w : qz;
        }
        if (tid == 0) {
            sh.found = -1;
            sh.unsure = 1;
            sh.tile = p.tiles - 1;
            sh.before = 0;
        }
        __syncthreads();
        F lost = 0;
        for (int k = 0; k < n_less; ++k) lost += less[k];
        const bool any = n_less == 0 || Z - lost > (kExact ? (F)0x1p-36 : (F)kSlack) * Z;
        if (!kExact && !any) return false;
        const int taken = any ? n_less : 0;          // nothing left over: from p itself
        // Tiles: each thread a run of them; the first whose running sum passes the border has the tile.
        const int per = (p.tiles + kChooseThreads - 1) / kChooseThreads;
        const int t0 = min(tid * per, p.tiles), t1 = min(t0 + per, p.tiles);
        F run = 0, total;
        for (int t = t0; t < t1; ++t) run += tile_weight<F>(row, t, M);
        for (int k = 0; k < taken; ++k) {
            const int t = x.tile_of(sh.less_at[k]);
            if (t >= t0 && t < t1) run -= less[k];
        }
        const F upto = block_scan(run, sh, total);
        const F border = (F)uniform() * total;
        const int owner = first_thread(upto > border, sh);
        if (tid == owner) {
            F before = upto - run;
            int pick = t0;
            for (int t = t0; t < t1; ++t) {
                F w = tile_weight<F>(row, t, M);
                for (int k = 0; k < taken; ++k)
                    if (x.tile_of(sh.less_at[k]) == t) w -= less[k];
                pick = t;
                if (before + w > border || t == t1 - 1) break;
                before += w;
            }
            sh.tile = pick;
            *reinterpret_cast<F*>(&sh.before) = before;
        }
        __syncthreads();
        // Inside the tile: each thread a run of its elements.
        constexpr int kEach = (Row<T>::kTile + Row<T>::kN - 1 + kChooseThreads - 1) / kChooseThreads;
        const int tile = sh.tile;
        const F before = *reinterpret_cast<F*>(&sh.before);
        const int lo = x.first(tile), n = x.first(tile + 1) - lo, e0 = tid * kEach;
        float l[kEach];
        F w[kEach];
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
            l[e] = -INFINITY;
            if (e0 + e < n) l[e] = to_float(x.x[lo + e0 + e]);
        }
        run = 0;
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
            w[e] = l[e] > -INFINITY ? weight<F>(l[e], M) : (F)0;
            for (int k = 0; k < taken; ++k)
                if (sh.less_at[k] == lo + e0 + e) w[e] = w[e] > less[k] ? w[e] - less[k] : (F)0;
            run += w[e];
        }
        F in_tile;
        const F here = before + block_scan(run, sh, in_tile);
        int holder = first_thread(here > border, sh);
        // The tile's sum and its elements' may differ by a rounding: then the last with any weight.
        if (holder < 0) {
            if (!kExact) return false;
            __syncthreads();
            const unsigned b = __ballot_sync(kFull, run > (F)0);
            if ((tid & 31) == 0) sh.owner[tid >> 5] = b ? tid + 31 - __clz(b) : -1;
            __syncthreads();
            for (int k = 0; k < kWarps; ++k) holder = max(holder, sh.owner[k]);
            if (holder < 0 && tid == 0) sh.found = min(lo, p.a.V - 1);
        }
        if (tid == holder) {
            F at = here - run, after = at;
            int pick = -1;
#pragma unroll
            for (int e = 0; e < kEach; ++e) {
                if (pick >= 0 && after > border) continue;
                if (!(w[e] > (F)0)) continue;
                if (pick >= 0) at = after;
                pick = e;
                after = at + w[e];
            }
            if (pick >= 0) sh.found = lo + e0 + pick;
            const F slack = (F)kSlack * Z;
            sh.unsure = pick < 0 || border - at < slack || after - border < slack;
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
        float edge;
        x.load((int)tile, lane, v, edge);
        const int hi = x.first(tile + 1), body = tile == 0 ? min(x.head, hi) : x.first(tile);
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
        if (edge == M) best = min(best, (unsigned)(lane < 16 ? lane : hi - ((hi - body) & (kN - 1)) + lane - 16));
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
        const float q = drafted ? draft_probability<float>(a, at, token, lane) : 0.f;
        join_tiles(p.sums + row * p.tiles, p.tiles, temp.c, lane, M, Z);
        int state = kRejected;
        float logprob = 0.f;
        if (!(Z > 0.f)) {
            state = kBad;
        } else if (in) {
            if (temp.greedy) {
                state = l == M && argmax(row, M) == token ? kTaken : kRejected;
            } else {
                const float z = (l - M) * temp.c, w = exp2_fast(z), uq = u * q * Z;
                const float slack = kSlack * uq + (kSlack - z * 0x1p-20f) * w;
                state = fabsf(uq - w) <= slack ? kUnsure : uq < w ? kTaken : kRejected;
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
        double mine = 0.0, Z;
        for (int t = warp; t < p.tiles; t += kWarps) {
            const double s = exact_tile<T>(x, t, M, inverse(temp.t), sh.powers);
            if (lane == 0) mine += s;
        }
        block_scan(mine, sh, Z);
        const long long at = (long long)r * a.S + i;
        const int token = a.draft_tokens[at];
        const double w = weight<double>(to_float(x.x[token]), M);
        const double q = draft_probability<double>(a, at, token, lane);
        return (double)a.accept_uniforms[at] * q * Z < w;
    }

    __device__ void run(uint32_t* status) {
        const VerifyArgs& a = p.a;
        const int tid = threadIdx.x, warp = tid >> 5;
        const int start = a.query_start[r], end = a.query_start[r + 1];
        int32_t* tokens = a.tokens + (long long)r * (a.S + 1);
        float* logprobs = a.logprobs ? a.logprobs + (long long)r * (a.S + 1) : nullptr;
        const bool bad = bad_rows(a, start, end);
        const int n = bad ? 0 : end - start;
        const uint32_t dead = p.dead ? p.dead[r] : 0xffffffffu;
        const int rows = dead < (uint32_t)n ? (int)dead + 1 : n;
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
        double mine = 0.0, Z;
        for (int t = tid; t < p.tiles; t += kChooseThreads) mine += tile_weight<double>(row, t, u.M);
        block_scan(mine, sh, Z);
        gather_less(u.i, u.i < n - 1, nullptr);
        draw<double>(row, u.M, Z);
        if (tid == 0) {
            const long long at = (long long)r * (a.S + 1) + u.i;
            a.tokens[at] = sh.found;
            if (a.logprobs && sh.found >= 0)
                a.logprobs[at] = (to_float(Row<T>(a, row).x[sh.found]) - u.M) / temp.t - logf((float)Z);
        }
    }
};

template <typename T>
__global__ void __launch_bounds__(kChooseThreads)
choose_kernel(const __grid_constant__ VerifyPlan p, uint32_t* status) {
    __shared__ ChooseShared sh;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int r = blockIdx.x;
    Chooser<T> chooser{p, sh, r, Temperature(p.a, r)};
    chooser.run(status);
}

// Items are kWarps tiles of a listed row; the CTA that finishes a row's last draws its token.
template <typename T>
__global__ void __launch_bounds__(kChooseThreads) settle_kernel(const __grid_constant__ VerifyPlan p) {
    __shared__ ChooseShared sh;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int tid = threadIdx.x, lane = tid & 31;
    const unsigned n = __ldcg(p.listed);
    if (n == 0) return;
    if (tid < 64) sh.powers[tid] = kPowers[tid];
    const int chunks = (p.tiles + kWarps - 1) / kWarps;
    for (long long item = blockIdx.x; item < (long long)n * chunks; item += gridDim.x) {
        const int at = (int)(item / chunks), t = (int)(item - (long long)at * chunks) * kWarps + (tid >> 5);
        const Unsettled u{__ldcg(&p.list[at].r), __ldcg(&p.list[at].i), __ldcg(&p.list[at].M), 0u};
        const Temperature temp(p.a, u.r);
        const long long row = p.a.query_start[u.r] + u.i;
        __syncthreads();
        if (t < p.tiles) {
            const double s = exact_tile<T>(Row<T>(p.a, row), t, u.M, inverse(temp.t), sh.powers);
            if (lane == 0) __stcg(reinterpret_cast<double*>(p.sums + row * p.tiles) + t, s);
        }
        __syncthreads();
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

// The workspace: the list's length and the rows' counters, the list, the tiles' sums.
size_t counter_bytes(int R, int T) { return (16 + ((size_t)R + T) * 4 + 255) & ~(size_t)255; }
size_t list_bytes(int R) { return ((size_t)R * sizeof(Unsettled) + 255) & ~(size_t)255; }

int tiles_of(int V, int size) {
    const int tile = kVecs * 32 * 16 / size;
    return (int)(((long long)V + tile - 1) / tile);
}

template <typename Kernel, typename... Args>
cudaError_t launch_dependent(Kernel kernel, unsigned blocks, int threads, cudaStream_t stream, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(threads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <typename T>
cudaError_t launch(const DeviceInfo& dev, const VerifyArgs& a, void* workspace, uint32_t* status,
                   cudaStream_t stream) {
    VerifyPlan p{};
    p.a = a;
    p.tiles = tiles_of(a.V, (int)sizeof(T));
    char* at = static_cast<char*>(workspace);
    p.listed = reinterpret_cast<unsigned*>(at);
    p.list = reinterpret_cast<Unsettled*>(at + counter_bytes(a.R, a.T));
    p.sums = reinterpret_cast<float2*>(at + counter_bytes(a.R, a.T) + list_bytes(a.R));
    const long long items = (long long)(a.S + 1) * a.R * p.tiles;
    const long long most = 4LL * dev.sm_count;
    if (items > 2 * most * kSumWarps && a.S > 0) {
        p.dead = reinterpret_cast<uint32_t*>(at + 16);
        p.arrived = p.dead + a.R;
        const cudaError_t e = cudaMemsetAsync(p.dead, 0xff, ((size_t)a.R + a.T) * 4, stream);
        if (e != cudaSuccess) return e;
    }
    const unsigned blocks = (unsigned)std::min((items + kSumWarps - 1) / kSumWarps, most);
    row_sums_kernel<T><<<blocks, kSumThreads, 0, stream>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    e = launch_dependent(choose_kernel<T>, (unsigned)a.R, kChooseThreads, stream, p, status);
    if (e != cudaSuccess) return e;
    const long long chunks = (long long)a.R * ((p.tiles + kWarps - 1) / kWarps);
    return launch_dependent(settle_kernel<T>, (unsigned)std::min(chunks, 3LL * dev.sm_count), kChooseThreads,
                            stream, p);
}

}  // namespace

size_t verify_workspace_bytes(int R, int T, int V) {
    return counter_bytes(R, T) + list_bytes(R) + (size_t)T * tiles_of(V, 4) * sizeof(float2);
}

cudaError_t launch_verify(const DeviceInfo& dev, const VerifyArgs& a, void* workspace,
                          uint32_t* status_word, cudaStream_t stream) {
    if (a.dtype == kFp32) return launch<float>(dev, a, workspace, status_word, stream);
    if (a.dtype == kBf16) return launch<__nv_bfloat16>(dev, a, workspace, status_word, stream);
    return launch<__half>(dev, a, workspace, status_word, stream);
}

}  // namespace dflash
