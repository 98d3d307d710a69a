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
// The tokens are those of exact arithmetic, but for borders nearer than about 2^-40 of a row's sum: every
// choice is made with fp32 sums first, whose error is bounded, and once more with sums of twice the
// precision where the bound does not settle it.
//
// Two kernels. row_sums reads logits: of each tile of a row (8 KB) the largest, m, and the sum of
// exp((x - m) / T). choose, a CTA for each request, joins the tiles' sums, takes the drafts in order, and
// draws the last token: the tile from the sums, then the place in it from the tile's logits, read again.
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
constexpr int kVecs = 16;                        // 16-byte vectors of a tile a lane holds
template <typename T>
struct Row {
    static constexpr int kTile = kVecs * 32 * Vec<T>::kN;
    const T* x;
    int V, head;
    __device__ __forceinline__ Row(const VerifyArgs& a, long long row) {
        x = static_cast<const T*>(a.logits) + row * a.row_stride;
        V = a.V;
        head = (int)((16 - (reinterpret_cast<uintptr_t>(x) & 15)) & 15) / (int)sizeof(T);
    }
    __device__ __forceinline__ long long first(int t) const {
        return t == 0 ? 0 : min((long long)head + (long long)t * kTile, (long long)V);
    }
    // the tile of element v
    __device__ __forceinline__ int tile_of(int v) const { return v < head ? 0 : (v - head) / kTile; }
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
        // Within [2^-100, 2^100], so that no product with it turns 0 or a difference of -inf to NaN.
        c = greedy ? 1.f : fminf(fmaxf(kLog2e / t, 0x1p-100f), 0x1p100f);
    }
};

struct VerifyPlan {
    VerifyArgs a;
    int tiles;                // of a row
    float2* sums;             // [T][tiles]: the largest logit, the sum of exp((x - it) / T)
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
    M = -INFINITY;
    for (int t = lane; t < tiles; t += 32) M = fmaxf(M, __ldcg(&sums[t].x));
    M = warp_max(M);
    Z = 0.f;
    for (int t = lane; t < tiles; t += 32) {
        const float2 s = __ldcg(&sums[t]);
        Z += s.y * (s.x == -INFINITY ? (s.y == s.y ? 0.f : 1.f) : exp2_fast((s.x - M) * c));
    }
    Z = warp_sum(Z);
}

// q of token x in row (r, i), by a warp.
__device__ __forceinline__ double draft_probability(const VerifyArgs& a, long long at, int x, int lane) {
    if (!a.cand_ids) return 1.0;
    double q = 0.0;
    if (lane < a.K && a.cand_ids[at * a.K + lane] == x) q = a.draft_probs[at * a.K + lane];
    return warp_sum(q);
}

// ---------------------------------------------------------------- sums of tiles

// Error of the fp32 sums, relative to a row's sum: an element's exponent is rounded once in the
// difference and its T 2^-22.4 off, so the sum is within 2^-22 sum p |z| <= 2^-22 (ln V + 1); ex2 is within
// 2^-22, at most 24 additions in a row within 24 * 2^-24, joining the tiles (a difference, a product,
// an exponential, additions) no more than that again. In all below 2^-17 for V < 2^31.
constexpr double kSlack = 0x1p-16;

constexpr int kSumThreads = 256;

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

template <typename T>
__global__ void __launch_bounds__(kSumThreads, 2) row_sums_kernel(VerifyPlan p) {
    const VerifyArgs& a = p.a;
    constexpr int kN = Vec<T>::kN;
    const int lane = threadIdx.x & 31;
    const long long warps = (long long)gridDim.x * (kSumThreads / 32);
    const long long items = (long long)(a.S + 1) * a.R * p.tiles;
    for (long long item = (long long)blockIdx.x * (kSumThreads / 32) + (threadIdx.x >> 5); item < items;
         item += warps) {
        const long long at = item / p.tiles;
        const int t = (int)(item - at * p.tiles);
        const int i = (int)(at / a.R), r = (int)(at - (long long)i * a.R);
        const int start = a.query_start[r], end = a.query_start[r + 1];
        // lengths that the choice refuses, and rows that the request does not have
        if (bad_rows(a, start, end) || i >= end - start) continue;
        if (p.dead && __shfl_sync(kFull, lane == 0 ? __ldcg(&p.dead[r]) : 0u, 0) < (uint32_t)i) continue;
        const long long row = start + i;
        const Row<T> x(a, row);
        const Temperature temp(a, r);
        const long long lo = x.first(t), hi = x.first(t + 1);
        const long long body = t == 0 ? min((long long)x.head, hi) : lo;     // on a 16-byte boundary
        const int n = (int)(hi - body);
        uint4 v[kVecs];
        const uint32_t low = sizeof(T) == 4 ? 0xff800000u
                                            : sizeof(T) == 2 && Vec<T>::kN == 8 && a.dtype == kBf16
                                                  ? 0xff80ff80u : 0xfc00fc00u;   // -inf
        const T* base = x.x + body;
#pragma unroll
        for (int k = 0; k < kVecs; ++k) {
            const int e = (k * 32 + lane) * kN;
            v[k] = make_uint4(low, low, low, low);
            if (e + kN <= n) v[k] = __ldcs(reinterpret_cast<const uint4*>(base + e));
        }
        // what is left of the ends: the row's elements before its first boundary, and behind the tile's
        // last whole vector
        float edge = -INFINITY;
        if (t == 0 && lane < x.head && lane < (int)hi) edge = to_float(x.x[lane]);
        const int rest = n & (kN - 1);
        if (lane >= 16 && lane - 16 < rest) edge = to_float(base[n - rest + lane - 16]);
        float m = edge;
#pragma unroll
        for (int k = 0; k < kVecs; ++k) {
            float f[kN];
            Vec<T>::widen(v[k], f);
#pragma unroll
            for (int e = 0; e < kN; ++e) m = fmaxf(m, f[e]);
        }
        m = warp_max(m);
        float s = weight_sum<T>(v, m, temp.c);
        s += exp2_fast((edge - fmaxf(m, -FLT_MAX)) * temp.c);
        s = warp_sum(s);
        float2* sums = p.sums + row * p.tiles;
        if (lane == 0) __stcg(&sums[t], make_float2(m, s));
        if (!p.dead || i == end - start - 1) continue;
        // The warp that completes a row before the last looks whether its draft is surely rejected.
        unsigned done = 0;
        if (lane == 0) {
            __threadfence();
            done = atomicAdd(&p.arrived[row], 1u) + 2u == (uint32_t)p.tiles;
            __threadfence();
        }
        if (!__shfl_sync(kFull, done, 0)) continue;
        __syncwarp();
        float M, Z;
        join_tiles(sums, p.tiles, temp.c, lane, M, Z);
        const long long draft = (long long)r * a.S + i;
        const int token = a.draft_tokens[draft];
        bool rejected = !(Z > 0.f);
        if (!rejected) {
            if ((unsigned)token >= (unsigned)a.V) {
                rejected = true;
            } else if (temp.greedy) {
                rejected = to_float(x.x[token]) < M;
            } else {
                const float q = (float)draft_probability(a, draft, token, lane);
                const float z = (to_float(x.x[token]) - M) * temp.c;
                const float w = exp2_fast(z), uq = a.accept_uniforms[draft] * q * Z;
                rejected = uq > w * (1.f + (float)kSlack - z * 0x1p-20f) + (float)kSlack * uq;
            }
        }
        if (rejected && lane == 0) atomicMin(&p.dead[r], (uint32_t)i);
    }
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
__device__ __forceinline__ Two operator*(Two a, Two b) {          // within 2^-46
    const float p = __fmul_rn(a.h, b.h);
    float e = __fmaf_rn(a.h, b.h, -p);
    e = __fmaf_rn(a.h, b.l, e);
    e = __fmaf_rn(a.l, b.h, e);
    return quick_sum(p, e);
}
__device__ __forceinline__ Two operator+(Two a, Two b) {
    const Two s = two_sum(a.h, b.h);
    return quick_sum(s.h, __fadd_rn(s.l, __fadd_rn(a.l, b.l)));
}
__device__ __forceinline__ Two two_of(double x) {
    const float h = (float)x;
    return {h, (float)(x - (double)h)};
}

// exp((x - M) / T) within about 2^-41. With y = (x - M) log2(e) / T = n / 16 + f, |f| <= 1/32:
// 2^y = 2^(n / 16) e^g, g = f ln 2, |g| < 0.0217, by Taylor's series to g^6 (g^7 / 5040 is below 2^-50),
// the first two powers in two floats. powers: 2^(j/16).
__device__ __forceinline__ Two exp_two(float x, float M, Two c, const Two* powers) {
    const Two d = two_sum(x, -M);
    if (!(d.h * c.h > -126.f)) return {0.f, 0.f};
    const Two y = d * c;
    const float n = rintf(__fmul_rn(y.h, 16.f));
    const Two f = two_sum(__fmaf_rn(n, -0.0625f, y.h), y.l);
    const Two ln2 = {0.693147182464599609375f, -1.9046542999577679e-09f};   // ln 2
    const Two g = f * ln2;
    const Two g2 = g * g;
    const float tail = __fmul_rn(__fmul_rn(g2.h, g.h),
                                 __fmaf_rn(g.h, __fmaf_rn(g.h, __fmaf_rn(g.h, 1.f / 720.f, 1.f / 120.f),
                                                          1.f / 24.f), 1.f / 6.f));
    Two e = quick_sum(__fmul_rn(0.5f, g2.h), __fmaf_rn(0.5f, g2.l, tail));
    e = g + e;
    e = Two{1.f, 0.f} + e;
    const int k = (int)n;
    e = e * powers[k & 15];
    const float scale = __uint_as_float((uint32_t)(127 + (k >> 4)) << 23);
    return {e.h * scale, e.l * scale};
}

// ---------------------------------------------------------------- the choice

constexpr int kChooseThreads = 512;
constexpr int kWarps = kChooseThreads / 32;
constexpr int kMaxK = 32;
enum : int { kTaken = 0, kRejected = 1, kUnsure = 2, kBad = 3 };

struct ChooseShared {
    Two powers[16];
    float M[kMaxDrafts + 1], Z[kMaxDrafts + 1], logprob[kMaxDrafts + 1];
    uint8_t state[kMaxDrafts + 1];
    double warp[kWarps];
    // what the draft's distribution takes away: places, tiles and probabilities, each token once
    int n_less, less_at[kMaxK];
    double less[kMaxK], less_q[kMaxK];
    // answers that one thread has for all
    int row, found, found_tile, unsure;
    double before, border;
};

// Inclusive running sum over the block's threads; total is the sum of all.
__device__ __forceinline__ double block_scan(double x, ChooseShared& sh, double& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const double o = __shfl_up_sync(kFull, x, d);
        if (lane >= d) x += o;
    }
    __syncthreads();
    if (lane == 31) sh.warp[warp] = x;
    __syncthreads();
    double below = 0.0;
    total = 0.0;
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) below += sh.warp[w];
        total += sh.warp[w];
    }
    return below + x;
}

template <typename T>
struct Chooser {
    const VerifyPlan& p;
    ChooseShared& sh;
    const int r;
    const Temperature temp;
    Two c2;

    // Weight of a logit relative to the row's largest.
    template <bool kCareful>
    __device__ __forceinline__ double weight(float x, float M) const {
        if (kCareful) {
            const Two w = exp_two(x, M, c2, sh.powers);
            return (double)w.h + (double)w.l;
        }
        return (double)exp2_fast((x - M) * temp.c);
    }

    // Sums of a row's tiles in twice the precision, as doubles in the place of the fp32 ones; returns
    // the sum of all. The whole block.
    __device__ double careful_sums(long long row, float M) {
        const Row<T> x(p.a, row);
        const int lane = threadIdx.x & 31;
        double* sums = reinterpret_cast<double*>(p.sums + row * p.tiles);
        double mine = 0.0, total;
        for (int t = threadIdx.x >> 5; t < p.tiles; t += kWarps) {
            const long long lo = x.first(t), hi = x.first(t + 1);
            Two s = {0.f, 0.f};
            for (long long e = lo + lane; e < hi; e += 32)
                s = s + exp_two(to_float(x.x[e]), M, c2, sh.powers);
            const double w = warp_sum((double)s.h + (double)s.l);
            if (lane == 0) {
                sums[t] = w;
                mine += w;
            }
        }
        block_scan(mine, sh, total);       // its barriers also make the sums visible to the block
        return total;
    }

    // Weight of a tile.
    template <bool kCareful>
    __device__ __forceinline__ double tile_weight(long long row, int t, float M) const {
        const float2* sums = p.sums + row * p.tiles;
        if (kCareful) return reinterpret_cast<const volatile double*>(sums)[t];
        const float2 s = __ldcg(&sums[t]);
        return s.x == -INFINITY ? 0.0 : (double)(s.y * exp2_fast((s.x - M) * temp.c));
    }

    // Draws a token of the row: whether it is certain, in sh.unsure; the token in sh.found. Z: the sum of
    // weights. residual: the draft's distribution is taken away. The whole block.
    template <bool kCareful>
    __device__ void draw(long long row, float M, double Z, bool residual, double u) {
        const Row<T> x(p.a, row);
        const int tid = threadIdx.x;
        // What each candidate loses.
        __syncthreads();
        const int n_less = residual ? sh.n_less : 0;
        if (tid < n_less)
            sh.less[tid] = fmin(weight<kCareful>(to_float(x.x[sh.less_at[tid]]), M), sh.less_q[tid] * Z);
        __syncthreads();
        double lost = 0.0;
        for (int k = 0; k < n_less; ++k) lost += sh.less[k];
        // (kCareful draws have an exact Z; a fast one's is the sum below, up to its error.)
        const bool any = n_less == 0 || Z - lost > (kCareful ? 0x1p-40 : kSlack) * Z;
        if (!kCareful && !any) {
            if (tid == 0) sh.unsure = 1;
            __syncthreads();
            return;
        }
        const int taken = any ? n_less : 0;          // nothing left over: from p itself
        // Tiles: each thread a run of them, then the run with the border, then the tile.
        const int per = (p.tiles + kChooseThreads - 1) / kChooseThreads;
        const int t0 = min(tid * per, p.tiles), t1 = min(t0 + per, p.tiles);
        double run = 0.0, total;
        for (int t = t0; t < t1; ++t) run += tile_weight<kCareful>(row, t, M);
        for (int k = 0; k < taken; ++k) {
            const int t = x.tile_of(sh.less_at[k]);
            if (t >= t0 && t < t1) run -= sh.less[k];
        }
        const double upto = block_scan(run, sh, total);
        const double border = u * total;
        if (tid == 0) {
            sh.found_tile = -1;
            sh.found = -1;
            sh.unsure = 0;
        }
        __syncthreads();
        // The first thread whose running sum passes the border.
        if (upto > border) atomicMin(reinterpret_cast<unsigned*>(&sh.found_tile), (unsigned)tid);
        __syncthreads();
        const int owner = sh.found_tile;
        __syncthreads();
        if (owner < 0 ? tid == kChooseThreads - 1 : tid == owner) {
            double before = upto - run;
            int pick = -1;
            double pick_before = before;
            for (int t = t0; t < t1; ++t) {
                double w = tile_weight<kCareful>(row, t, M);
                for (int k = 0; k < taken; ++k)
                    if (x.tile_of(sh.less_at[k]) == t) w -= sh.less[k];
                if (w > 0.0) {
                    pick = t;
                    pick_before = before;
                }
                before += w;
                if (pick == t && before > border) break;
            }
            // none by rounding: the last tile, which the search below ends in
            sh.found_tile = pick < 0 ? p.tiles - 1 : pick;
            sh.before = pick < 0 ? before : pick_before;
            sh.border = border;
        }
        __syncthreads();
        // Inside the tile.
        const int tile = sh.found_tile;
        const double before = sh.before;
        const long long lo = x.first(tile), hi = x.first(tile + 1);
        const int each = (int)((hi - lo + kChooseThreads - 1) / kChooseThreads);
        const long long e0 = min(lo + (long long)tid * each, hi), e1 = min(e0 + each, hi);
        auto left = [&](long long e) {
            double w = weight<kCareful>(to_float(x.x[e]), M);
            for (int k = 0; k < taken; ++k)
                if (sh.less_at[k] == e) w = fmax(w - sh.less[k], 0.0);
            return w;
        };
        run = 0.0;
        for (long long e = e0; e < e1; ++e) run += left(e);
        double in_tile;
        const double here = block_scan(run, sh, in_tile);
        // Past every border by rounding: the last element with any weight.
        if (before + here > border && before + here - run <= border) {
            double at = before + here - run;
            for (long long e = e0; e < e1; ++e) {
                const double w = left(e);
                if (at + w > border) {
                    sh.found = (int)e;
                    const double slack = kSlack * Z;
                    if (!kCareful && (border - at < slack || at + w - border < slack)) sh.unsure = 1;
                    break;
                }
                at += w;
            }
        }
        __syncthreads();
        if (sh.found < 0) {
            if (!kCareful) {
                if (tid == 0) sh.unsure = 1;
            } else {
                int last = -1;
                for (long long e = e0; e < e1; ++e)
                    if (left(e) > 0.0) last = (int)e;
                if (last >= 0) atomicMax(&sh.found, last);
            }
        }
        __syncthreads();
    }

    // The first of a row's largest logits. One warp.
    __device__ int argmax(long long row, float M) const {
        const Row<T> x(p.a, row);
        const int lane = threadIdx.x & 31;
        const float2* sums = p.sums + row * p.tiles;
        int tile = INT_MAX;
        for (int t = lane; t < p.tiles && tile == INT_MAX; t += 32)
            if (__ldcg(&sums[t].x) == M) tile = t;
        tile = (int)__reduce_min_sync(kFull, (unsigned)tile);
        long long best = INT_MAX;
        for (long long e = x.first(tile) + lane; e < x.first(tile + 1) && best == INT_MAX; e += 32)
            if (to_float(x.x[e]) == M) best = e;
        return (int)__reduce_min_sync(kFull, (unsigned)best);
    }

    // Looks at row i of the request, one of n; one warp.
    __device__ void look(long long row, int i, int n) {
        const VerifyArgs& a = p.a;
        const int lane = threadIdx.x & 31;
        float M, Z;
        join_tiles(p.sums + row * p.tiles, p.tiles, temp.c, lane, M, Z);
        int state = kRejected;
        float logprob = 0.f;
        if (!(Z > 0.f) || M == -INFINITY) {
            state = kBad;
        } else if (i < n - 1) {
            const Row<T> x(a, row);
            const long long at = (long long)r * a.S + i;
            const int token = a.draft_tokens[at];
            if ((unsigned)token < (unsigned)a.V) {
                const float l = to_float(x.x[token]);
                if (temp.greedy) {
                    state = l == M && argmax(row, M) == token ? kTaken : kRejected;
                } else {
                    const float z = (l - M) * temp.c;
                    const double w = exp2_fast(z);
                    const double uq = (double)a.accept_uniforms[at] * draft_probability(a, at, token, lane) * Z;
                    const double slack = kSlack * uq + (kSlack - (double)z * 0x1p-20) * w;
                    state = fabs(uq - w) <= slack ? kUnsure : uq < w ? kTaken : kRejected;
                    logprob = (l - M) / temp.t - logf(Z);
                }
            }
        }
        if (lane == 0) {
            sh.M[i] = M;
            sh.Z[i] = Z;
            sh.state[i] = (uint8_t)state;
            sh.logprob[i] = logprob;
        }
    }

    // Whether draft i, in doubt, is taken; Z: its row's exact sum.
    __device__ bool taken(long long row, int i, double Z) const {
        const VerifyArgs& a = p.a;
        const long long at = (long long)r * a.S + i;
        const int token = a.draft_tokens[at];
        const double w = weight<true>(to_float(Row<T>(a, row).x[token]), sh.M[i]);
        const double q = draft_probability(a, at, token, threadIdx.x & 31);
        return (double)a.accept_uniforms[at] * q * Z < w;
    }

    __device__ void run(uint32_t* status) {
        const VerifyArgs& a = p.a;
        const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
        const int start = a.query_start[r], end = a.query_start[r + 1];
        int32_t* tokens = a.tokens + (long long)r * (a.S + 1);
        float* logprobs = a.logprobs ? a.logprobs + (long long)r * (a.S + 1) : nullptr;
        const bool bad = bad_rows(a, start, end);
        const int n = bad ? 0 : end - start;
        const uint32_t dead = p.dead ? p.dead[r] : 0xffffffffu;
        const int rows = dead < (uint32_t)n ? (int)dead + 1 : n;
        for (int i = warp; i < rows; i += kWarps) look(start + i, i, n);
        if (!temp.greedy) {
            c2 = two_of(fmin(fmax(1.4426950408889634074 / (double)temp.t, 0x1p-100), 0x1p100));
            if (tid < 16) sh.powers[tid] = two_of(exp2((double)tid / 16.0));
        }
        __syncthreads();
        // The drafts in order.
        int i = 0, count = 0, drawn = -1;
        float last_logprob = 0.f;
        bool careful = false;
        double Z = 0.0;
        for (; i < rows; ++i) {
            const int state = sh.state[i];
            if (state == kTaken) continue;
            careful = false;
            if (state == kUnsure) {
                Z = careful_sums(start + i, sh.M[i]);
                careful = true;
                if (taken(start + i, i, Z)) continue;
            }
            break;
        }
        const long long row = start + i;
        if (i < rows && sh.state[i] != kBad) {
            const bool residual = i < n - 1;
            const float M = sh.M[i];
            count = i + 1;
            if (temp.greedy) {
                drawn = argmax(row, M);
            } else {
                // The draft's distribution, each token once; ids outside the vocabulary are left out.
                if (tid == 0) sh.n_less = 0;
                __syncthreads();
                if (residual && warp == 0) {
                    const long long at = (long long)r * a.S + i;
                    const int k_all = a.cand_ids ? a.K : 1;
                    const int id = lane < k_all ? (a.cand_ids ? a.cand_ids[at * a.K + lane] : a.draft_tokens[at]) : -1;
                    const double q = lane < k_all ? (a.cand_ids ? (double)a.draft_probs[at * a.K + lane] : 1.0) : 0.0;
                    const bool in = (unsigned)id < (unsigned)a.V;
                    if (lane < k_all && !in) atomicOr(status, kStatusBadId);
                    double sum = 0.0;
                    bool first = in;
                    for (int k = 0; k < 32; ++k) {
                        const int other = __shfl_sync(kFull, id, k);
                        const double oq = __shfl_sync(kFull, q, k);
                        if (other == id) {
                            sum += oq;
                            if (k < lane) first = false;
                        }
                    }
                    const unsigned firsts = __ballot_sync(kFull, first);
                    if (first) {
                        const int to = __popc(firsts & ((1u << lane) - 1));
                        sh.less_at[to] = id;
                        sh.less_q[to] = sum;
                    }
                    if (lane == 0) sh.n_less = __popc(firsts);
                }
                __syncthreads();
                // numbers outside [0, 1) count as the nearer end, NaN as 0
                const double u = fminf(fmaxf(a.sample_uniforms[r], 0.f), 1.f - 0x1p-24f);
                bool settled = false;
                if (!careful) {
                    draw<false>(row, M, (double)sh.Z[i], residual, u);
                    settled = sh.unsure == 0;
                    if (!settled) Z = careful_sums(row, M);
                }
                if (!settled) draw<true>(row, M, Z, residual, u);
                drawn = sh.found;
                const Row<T> x(a, row);
                if (drawn >= 0)
                    last_logprob = (to_float(x.x[drawn]) - M) / temp.t -
                                   logf(settled ? sh.Z[i] : (float)Z);
            }
        } else if (i < rows) {
            count = i;
        }
        for (int k = tid; k <= a.S; k += kChooseThreads) {
            tokens[k] = k < i ? a.draft_tokens[(long long)r * a.S + k] : k == i && k < count ? drawn : -1;
            if (logprobs) logprobs[k] = k < i ? sh.logprob[k] : k == i && k < count ? last_logprob : 0.f;
        }
        if (tid == 0) {
            a.counts[r] = count;
            if (bad) atomicOr(status, kStatusBadLength);
            if (i < rows && sh.state[i] == kBad) atomicOr(status, kStatusBadLogits);
            // drafts that were looked at and are no tokens
            if (i < n - 1 && (unsigned)a.draft_tokens[(long long)r * a.S + i] >= (unsigned)a.V)
                atomicOr(status, kStatusBadId);
        }
    }
};

template <typename T>
__global__ void __launch_bounds__(kChooseThreads) choose_kernel(VerifyPlan p, uint32_t* status) {
    __shared__ ChooseShared sh;
    const int r = blockIdx.x;
    Chooser<T> chooser{p, sh, r, Temperature(p.a, r), Two{0.f, 0.f}};
    chooser.run(status);
}

// Bytes of the row counters, in front of the tiles' sums.
size_t counter_bytes(int R, int T) { return ((size_t)R + T) * 4 + 255 & ~(size_t)255; }

int tiles_of(int V, int size) {
    const int tile = kVecs * 32 * 16 / size;
    return (int)(((long long)V + tile - 1) / tile);
}

template <typename T>
cudaError_t launch(const DeviceInfo& dev, const VerifyArgs& a, void* workspace, uint32_t* status,
                   cudaStream_t stream) {
    VerifyPlan p{a, tiles_of(a.V, (int)sizeof(T)), nullptr, nullptr, nullptr};
    const size_t counters = counter_bytes(a.R, a.T);
    p.sums = reinterpret_cast<float2*>(static_cast<char*>(workspace) + counters);
    const long long items = (long long)(a.S + 1) * a.R * p.tiles;
    const long long per_wave = 2LL * dev.sm_count * (kSumThreads / 32);
    if (items > 4 * per_wave && a.S > 0) {
        p.dead = static_cast<uint32_t*>(workspace);
        p.arrived = p.dead + a.R;
        const cudaError_t e = cudaMemsetAsync(workspace, 0xff, ((size_t)a.R + a.T) * 4, stream);
        if (e != cudaSuccess) return e;
    }
    const unsigned blocks = (unsigned)std::min((items + kSumThreads / 32 - 1) / (kSumThreads / 32),
                                               2LL * dev.sm_count);
    row_sums_kernel<T><<<blocks, kSumThreads, 0, stream>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    choose_kernel<T><<<(unsigned)a.R, kChooseThreads, 0, stream>>>(p, status);
    return cudaGetLastError();
}

}  // namespace

size_t verify_workspace_bytes(int R, int T, int V) {
    return counter_bytes(R, T) + (size_t)T * tiles_of(V, 4) * sizeof(float2);
}

cudaError_t launch_verify(const DeviceInfo& dev, const VerifyArgs& a, void* workspace,
                          uint32_t* status_word, cudaStream_t stream) {
    if (a.dtype == kFp32) return launch<float>(dev, a, workspace, status_word, stream);
    if (a.dtype == kBf16) return launch<__nv_bfloat16>(dev, a, workspace, status_word, stream);
    return launch<__half>(dev, a, workspace, status_word, stream);
}

}  // namespace dflash
