// rope.cu: the norm of each query and key head and its rotation by position, in one pass, with the
// keys and values stored in the paged cache in the same pass where a cache is given.
//
// Page "vllm.models.beam.nvidia.dflash2", DFlash2BeamAttention: beam_qk_norm_rope norms queries and
// keys, rotates them and can write keys and values into the cache by slot; in
// precompute_and_store_context_kv the keys of the context are normed, rotated and stored without
// queries. The pages show the calls; the arithmetic is the standard one:
//
//   y = x * w / sqrt(mean(x^2) + eps)                          (each head by itself)
//   (y_a, y_b) -> scale * (y_a cos t - y_b sin t, y_b cos t + y_a sin t),  t = position * f_j
//
// for pair j of the first rotary_dim values: (j, j + rotary_dim / 2), or (2j, 2j + 1) interleaved.
//
// Angles: f_j is kept in turns, as a whole number of 2^-64, so position * f_j modulo one turn is
// the low 64 bits of an integer product, exact for the f_j that is kept. That one is made in doubles, off by a
// few 2^-53 of itself, and rounded to 2^-64: within 2^-25.5 of a turn at position 2^31 for base 10^4, 2^-24.3 for 10^6.
#include "common.cuh"
#include "ptx.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <algorithm>
#include <cfloat>
#include <climits>
#include <cmath>

namespace dflash {
namespace {

// A head row (one head of one token) belongs to a group of `lanes` threads, the power of two at or
// above head_dim / 16; a thread holds 16 values of it, eight a and eight b, chosen so that both values of a
// pair are in one thread: its pairs are 8j to 8j + 7. Interleaved, those are the 16 values from 16 j on. Else
// they come in units of kUnit pairs, kUnit the largest of 8, 4, 2, 1 that divides the halves: a unit is kUnit
// values of the first half and the same of the second, or two such pieces of what is not rotated. Pieces are
// loaded and stored at once: 16 bytes where the halves are multiples of 8 values.
//
// A CTA takes a run of tokens: all of their query rows, then key rows, then value rows, so that addresses
// and weights are found once for a kind. A row is loaded while the one before is worked on, the first ones
// while the threads take the tokens' cosines and sines, once each, into shared memory.
constexpr int kThreads = 256;
constexpr int kBlocks = 3;          // CTAs of an SM
enum : int { kQuery = 0, kKey = 1, kValue = 2, kNone = 3 };

template <typename T>
__device__ __forceinline__ float2 widen(uint32_t v);
template <>
__device__ __forceinline__ float2 widen<__nv_bfloat16>(uint32_t v) {
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}
template <>
__device__ __forceinline__ float2 widen<__half>(uint32_t v) {
    return __half22float2(*reinterpret_cast<__half2*>(&v));
}

template <typename T>
__device__ __forceinline__ uint32_t narrow(float x, float y);
template <>
__device__ __forceinline__ uint32_t narrow<__nv_bfloat16>(float x, float y) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&v);
}
template <>
__device__ __forceinline__ uint32_t narrow<__half>(float x, float y) {
    const __half2 v = __floats2half2_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// kN 16-bit values at p, as kN / 2 words (one, its lower half, for a single value), and back.
template <int kN>
__device__ __forceinline__ void get(const uint16_t* p, uint32_t* w) {
    if constexpr (kN == 8) {
        const uint4 v = __ldcs(reinterpret_cast<const uint4*>(p));
        w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    } else if constexpr (kN == 4) {
        const uint2 v = __ldcs(reinterpret_cast<const uint2*>(p));
        w[0] = v.x, w[1] = v.y;
    } else if constexpr (kN == 2) {
        w[0] = __ldcs(reinterpret_cast<const uint32_t*>(p));
    } else {
        w[0] = __ldcs(p);
    }
}
template <int kN>
__device__ __forceinline__ void set(uint16_t* p, const uint32_t* w) {
    if constexpr (kN == 8) *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    else if constexpr (kN == 4) *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    else if constexpr (kN == 2) *reinterpret_cast<uint32_t*>(p) = w[0];
    else *p = (uint16_t)w[0];
}

// Quotients by a fixed divisor d, of n with n d < 2^32: by the divisor's reciprocal, rounded up, in 32 bits.
struct Divisor {
    uint32_t m, d;
    Divisor(uint32_t divisor = 1) : m((uint32_t)((0x100000000ull + divisor - 1) / divisor)), d(divisor) {}
    __device__ __forceinline__ int of(int n) const { return d == 1 ? n : (int)__umulhi(m, (uint32_t)n); }
};

struct RopePlan {
    NormRopeArgs a;
    int per;             // threads of a group that hold any of a head: ceil(head_dim / 16)
    int lanes;           // the group
    int pairs_shift;     // log2(8 per), where that is a whole number
    int tokens;          // of a CTA
    int page_shift;      // -1: page_size is no power of two
    float k_mul, v_mul;  // inverses of the scales, where a product with them is exact; else 0
    float inv_dim;       // 1 / head_dim
    // Of queries, keys and values: strides in bytes, of tokens and of heads; and of the first two's outputs.
    uint32_t token_bytes[3], head_bytes[3], out_token_bytes[2], out_head_bytes[2];
    Divisor by_q, by_kv;
};

// kFull: head_dim is 16 times a power of two, so that every thread has all of its values (40001 tokens of 128: 175 us,
// 179 with checks; units of 4 pairs instead of 8 also 179).
template <typename T, bool kInterleaved, int kUnit, bool kFull>
struct Rows {
    static constexpr int kUnits = 8 / kUnit;             // of a thread
    static constexpr int kWords = (kUnit + 1) / 2;       // of a piece
    const RopePlan& p;
    uint32_t* status;
    const float4* table;       // [tokens][4][per] chunks of two pairs: (cos, cos, sin, sin)
    long long token0;
    int tokens, j, group, groups;
    int dim[2][kUnits];        // first value of each of the thread's pieces; head_dim or more: none

    __device__ __forceinline__ Rows(const RopePlan& plan, uint32_t* word, const float4* cs)
        : p(plan), status(word), table(cs) {
        j = threadIdx.x & (p.lanes - 1);
        group = threadIdx.x / p.lanes;
        groups = kThreads / p.lanes;
        token0 = (long long)blockIdx.x * p.tokens;
        tokens = (int)min((long long)p.tokens, p.a.T - token0);
        const int half = p.a.rotary_dim / 2;
#pragma unroll
        for (int k = 0; k < kUnits; ++k) {
            const int pair = 8 * j + k * kUnit;
#pragma unroll
            for (int b = 0; b < 2; ++b)
                dim[b][k] = kInterleaved || pair >= half ? 2 * pair + b * kUnit : pair + b * half;
        }
    }

    template <int kKind>
    __device__ __forceinline__ int heads() const {
        return kKind == kQuery ? p.a.q_heads : p.a.kv_heads;
    }
    template <int kKind>
    __device__ __forceinline__ int rows() const {
        if (kKind == kNone || (kKind == kValue && !p.a.slots)) return 0;
        return tokens * heads<kKind>();
    }
    // (Runs of several tokens have at most 2048 rows of a kind.)
    template <int kKind>
    __device__ __forceinline__ int token_of(int row) const {
        return p.tokens == 1 ? 0 : (kKind == kQuery ? p.by_q : p.by_kv).of(row);
    }
    __device__ __forceinline__ bool has(int b, int k) const { return kFull || dim[b][k] < p.a.head_dim; }

    // The thread's 16 values of a row, as they are: eight a, eight b.
    template <int kKind>
    __device__ __forceinline__ void load(int row, uint32_t (&x)[2][kUnits][kWords]) const {
        const NormRopeArgs& a = p.a;
        if (rows<kKind>() == 0) return;
        row = min(row, rows<kKind>() - 1);                           // past the end: anything, it is not used
        const int t = token_of<kKind>(row), h = row - t * heads<kKind>();
        const void* from = kKind == kQuery ? a.query : kKind == kKey ? a.key : a.value;
        const uint32_t ts = p.token_bytes[kKind % 3], hs = p.head_bytes[kKind % 3];
        const uint16_t* src = reinterpret_cast<const uint16_t*>(
            static_cast<const uint8_t*>(from) + (uint64_t)token0 * ts + (uint64_t)(uint32_t)t * ts +
            (uint64_t)(uint32_t)h * hs);
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int k = 0; k < kUnits; ++k) {
#pragma unroll
                for (int w = 0; w < kWords; ++w) x[b][k][w] = 0;
                if (has(b, k)) get<kUnit>(src + dim[b][k], x[b][k]);
            }
    }

    // The same as pairs of floats: 0 to 3 are the a, 4 to 7 the b.
    __device__ __forceinline__ void widened(const uint32_t (&raw)[2][kUnits][kWords], uint64_t (&x)[8]) const {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int b = k >> 2, at = 2 * (k & 3);                  // values at, at + 1
            float2 f;
            if constexpr (kUnit == 1) f = make_float2(widen<T>(raw[b][at][0]).x, widen<T>(raw[b][at + 1][0]).x);
            else f = widen<T>(raw[b][at / kUnit][at % kUnit / 2]);
            x[k] = ptx::pair_of(f.x, f.y);
        }
    }

    // The thread's 16 weights.
    __device__ __forceinline__ void weights(const void* from, uint64_t (&w)[8]) const {
        if (p.a.weight_dtype == kFp32) {
            float f[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                const int b = k >> 3, unit = (k & 7) / kUnit;
                f[k] = has(b, unit) ? static_cast<const float*>(from)[dim[b][unit] + (k & 7) % kUnit] : 0.f;
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) w[k] = ptx::pair_of(f[2 * k], f[2 * k + 1]);
        } else {
            uint32_t raw[2][kUnits][kWords];
#pragma unroll
            for (int k = 0; k < 2 * kUnits; ++k) {
                const int b = k / kUnits, unit = k % kUnits;
#pragma unroll
                for (int u = 0; u < kWords; ++u) raw[b][unit][u] = 0;
                if (has(b, unit)) get<kUnit>(static_cast<const uint16_t*>(from) + dim[b][unit], raw[b][unit]);
            }
            widened(raw, w);
        }
    }

    // Writes a row's values: as T, or as e4m3 of x / scale (mul: its exact inverse, or 0).
    __device__ __forceinline__ void put(void* out, long long to, const uint64_t (&x)[8], bool small, float scale,
                                        float mul) const {
        if (!small) {
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int k = 0; k < kUnits; ++k) {
                    if (!has(b, k)) continue;
                    uint32_t w[kWords];
#pragma unroll
                    for (int u = 0; u < kWords; ++u) {
                        const int at = k * kUnit + 2 * u;
                        const float2 f = ptx::halves_of(x[4 * b + at / 2]);
                        w[u] = kUnit == 1 ? narrow<T>(at & 1 ? f.y : f.x, 0.f) : narrow<T>(f.x, f.y);
                    }
                    set<kUnit>(static_cast<uint16_t*>(out) + to + dim[b][k], w);
                }
            return;
        }
        uint16_t two[8];                                             // two e4m3 values each
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            float2 f = ptx::halves_of(x[k]);
            f = mul == 0.f ? make_float2(__fdiv_rn(f.x, scale), __fdiv_rn(f.y, scale))
                           : make_float2(f.x * mul, f.y * mul);
            two[k] = __nv_cvt_float2_to_fp8x2(f, __NV_SATFINITE, __NV_E4M3);
        }
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int k = 0; k < kUnits; ++k) {
                if (!has(b, k)) continue;
                uint8_t* dst = static_cast<uint8_t*>(out) + to + dim[b][k];
                const uint16_t* v = two + 4 * b + k * kUnit / 2;
                if constexpr (kUnit == 8)
                    *reinterpret_cast<uint2*>(dst) = make_uint2(v[0] | (uint32_t)v[1] << 16, v[2] | (uint32_t)v[3] << 16);
                else if constexpr (kUnit == 4) *reinterpret_cast<uint32_t*>(dst) = v[0] | (uint32_t)v[1] << 16;
                else if constexpr (kUnit == 2) *reinterpret_cast<uint16_t*>(dst) = v[0];
                else *dst = (uint8_t)(k & 1 ? v[0] >> 8 : v[0]);
            }
    }

    // The sum of squares of a group's row. Every lane of the warp takes part.
    __device__ __forceinline__ float squares(const uint64_t (&x)[8]) const {
        uint64_t sum[2] = {0, 0};
#pragma unroll
        for (int k = 0; k < 8; ++k) sum[k & 1] = ptx::fma_pair(x[k], x[k], sum[k & 1]);
        const float2 f = ptx::halves_of(ptx::add_pair(sum[0], sum[1]));
        float s = f.x + f.y;
        for (int d = p.lanes / 2; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
        return s;
    }

    // Norms row x in place, by weights w.
    __device__ __forceinline__ void norm(uint64_t (&x)[8], const uint64_t (&w)[8]) const {
        float sum = squares(x), eps = p.a.eps, of = fmaf(sum, p.inv_dim, eps);
        // Where fp32's range ends: squares past it (bf16 values from 2^60 on) once more with the head 2^-72 as large; and
        // where the root is of less than 2^-100, with it 2^72 as large, since squares below 2^-126 lose bits (from
        // 2^-100 on, 2^-150 for each of them does not show). eps goes with the squares.
        if (__any_sync(0xffffffffu, !(of >= 0x1p-100f && of <= FLT_MAX))) {
            const float by = of > FLT_MAX ? 0x1p-72f : of < 0x1p-100f ? 0x1p72f : 1.f;
#pragma unroll
            for (int k = 0; k < 8; ++k) x[k] = ptx::mul_pair(x[k], ptx::pair_of(by, by));
            sum = squares(x);
            eps = eps * by * by;
            of = fmaf(sum, p.inv_dim, eps);
        }
        const float r = rsqrtf(of);
        const uint64_t rr = ptx::pair_of(r, r);
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = ptx::mul_pair(x[k], ptx::mul_pair(w[k], rr));
    }

    // Pairs 2c and 2c + 1 of the thread's, rotated.
    __device__ __forceinline__ void rotated(const uint64_t (&x)[8], int c, const float4& f, uint64_t& u, uint64_t& v) const {
        if constexpr (!kInterleaved) {
            const uint64_t cc = ptx::pair_of(f.x, f.y), ss = ptx::pair_of(f.z, f.w);
            const uint64_t minus = ptx::pair_of(-f.z, -f.w);
            u = ptx::fma_pair(x[c + 4], minus, ptx::mul_pair(x[c], cc));
            v = ptx::fma_pair(x[c], ss, ptx::mul_pair(x[c + 4], cc));
        } else {
            const float2 a = ptx::halves_of(x[2 * c]), b = ptx::halves_of(x[2 * c + 1]);
            u = ptx::pair_of(a.x * f.x - a.y * f.z, a.y * f.x + a.x * f.z);
            v = ptx::pair_of(b.x * f.y - b.y * f.w, b.y * f.y + b.x * f.w);
        }
    }

    // Rotates row x of token t in place. Pairs behind rotary_dim are left alone (by a cosine of 1 and a sine of 0 an
    // infinity would make its partner NaN, and -0 would turn 0). Pairs of a unit are rotated together or not at all:
    // units of 4 by a way out between them, of 2 by choosing between results (20001 tokens of 40 heads of 80, rotated by 40
    // and by 20: 71 and 86 us by ways out, 73 and 81 by choosing; 69 and 79 without a difference).
    __device__ __forceinline__ void rotate(uint64_t (&x)[8], int t) const {
        constexpr int kTogether = kInterleaved ? 1 : kUnit;
        constexpr int kStep = kInterleaved ? 1 : 4;
        const int turn = p.a.rotary_dim / 2 - 8 * j;                 // so many of the thread's pairs, all where 8 or more
        if (kTogether != 2 && turn <= 0) return;
        const float4* cs = table + (size_t)t * 4 * p.per + j;
        if (kTogether > 1 || turn >= 8) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                if (kTogether == 4 && c == 2 && turn <= 4) return;
                const bool on = kTogether != 2 || 2 * c < turn;
                const int at = kInterleaved ? 2 * c : c;
                uint64_t u, v;
                rotated(x, c, cs[c * p.per], u, v);
                x[at] = on ? u : x[at];
                x[at + kStep] = on ? v : x[at + kStep];
            }
            return;
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            if (2 * c >= turn) return;
            const int at = kInterleaved ? 2 * c : c;
            const bool both = 2 * c + 1 < turn;
            uint64_t u, v;
            rotated(x, c, cs[c * p.per], u, v);
            if constexpr (kInterleaved) {                            // u is the first pair, v the second
                x[at] = u;
                if (both) x[at + kStep] = v;
            } else {                                                 // the pairs' a and their b
                x[at] = both ? u : ptx::pair_of(ptx::halves_of(u).x, ptx::halves_of(x[at]).y);
                x[at + kStep] = both ? v : ptx::pair_of(ptx::halves_of(v).x, ptx::halves_of(x[at + kStep]).y);
            }
        }
    }

    // All of the CTA's rows of a kind; next: the thread's first, loaded, and then the next kind's.
    template <int kKind, int kNext>
    __device__ __forceinline__ void run(uint32_t (&next)[2][kUnits][kWords]) const {
        const NormRopeArgs& a = p.a;
        const int n = rows<kKind>();
        const void* from = kKind == kQuery ? a.q_weight : a.k_weight;
        uint64_t w[8];
        if (kKind != kValue && from) weights(from, w);
        for (int row0 = 0; row0 < n; row0 += groups) {               // the warp stays together
            const int row = row0 + group;
            const bool live = row < n;
            const int t = token_of<kKind>(min(row, n - 1)), h = row - t * heads<kKind>();
            long long slot = -1;
            if (kKind != kQuery && a.slots && live) slot = a.slots[token0 + t];
            const bool small = a.cache.dtype == kE4m3;
            uint32_t bits[2][kUnits][kWords];
            if (kKind == kValue && !small) {
#pragma unroll
                for (int k = 0; k < 2 * kUnits * kWords; ++k) (&bits[0][0][0])[k] = (&next[0][0][0])[k];
            }
            uint64_t x[8];
            widened(next, x);
            if (row0 + groups < n) load<kKind>(row + groups, next);
            else load<kNext>(group, next);
            if (kKind != kValue && from) norm(x, w);
            if (!live || (!kFull && j >= p.per)) continue;
            if (kKind != kValue && a.rotary_dim > 0) rotate(x, t);
            if (kKind == kQuery || !a.slots) {
                const uint32_t ts = p.out_token_bytes[kKind & 1], hs = p.out_head_bytes[kKind & 1];
                uint8_t* out = static_cast<uint8_t*>(kKind == kQuery ? a.query_out : a.key_out);
                put(out + (uint64_t)token0 * ts + (uint64_t)(uint32_t)t * ts + (uint64_t)(uint32_t)h * hs, 0, x,
                    false, 1.f, 1.f);
                continue;
            }
            if (slot >= (long long)a.cache.num_pages * a.cache.page_size) {
                if (j == 0) atomicOr(status, kStatusBadId);
                continue;
            }
            if (slot < 0) continue;
            const long long page = p.page_shift >= 0 ? slot >> p.page_shift : slot / a.cache.page_size;
            const long long to = page * a.cache.page_stride +
                                 (slot - page * a.cache.page_size) * a.cache.token_stride + h * a.cache.head_stride;
            if (kKind == kValue && !small) {                         // the bits as they are
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int k = 0; k < kUnits; ++k)
                        if (has(b, k)) set<kUnit>(static_cast<uint16_t*>(a.cache.value) + to + dim[b][k], bits[b][k]);
                continue;
            }
            put(kKind == kValue ? a.cache.value : a.cache.key, to, x, small,
                kKind == kValue ? a.cache.v_scale : a.cache.k_scale, kKind == kValue ? p.v_mul : p.k_mul);
        }
    }
};

// Bound by memory and, into an e4m3 cache, as much by instructions: 55 to 64% of the issue slots go to 235
// instructions for every four rows of 128. 40001 tokens of 32 + 8 + 8 heads of 128: with a bf16 cache 175 us, 984 MB,
// 5.6 TB/s; with an e4m3 cache 174 us, 902 MB, 5.2 TB/s. 16411 tokens of 48 heads of 64, rotated by halves: 39 us, 202 MB.
// 8 key and 8 value heads of 128 of 20001 tokens, without queries: 42 us, 164 MB. One token: 5 us. An e4m3 scale that is
// no power of two is divided by: 201 us for both scales of that kind, 188 for one of them, 176 for none (the same bits).
// (Two rows loaded ahead instead of one, 80 registers: 171 and 190 us for the first two, 181 in CTAs of
// 128 threads; two CTAs an SM: 196 and 204; single floats instead of pairs: 5 us more.)
template <typename T, bool kInterleaved, int kUnit, bool kFull>
__global__ void __launch_bounds__(kThreads, kBlocks)
norm_rope_kernel(const __grid_constant__ RopePlan p, uint32_t* status) {
    extern __shared__ __align__(16) float4 table[];
    const NormRopeArgs& a = p.a;
    Rows<T, kInterleaved, kUnit, kFull> rows(p, status, table);
    uint32_t first[2][8 / kUnit][(kUnit + 1) / 2];
    if (a.q_heads > 0) rows.template load<kQuery>(rows.group, first);
    else rows.template load<kKey>(rows.group, first);
    if (a.rotary_dim > 0) {
        // Cosines and sines (of pairs behind rotary_dim none are used).
        const int pairs = 8 * p.per;
        for (int e = threadIdx.x; e < rows.tokens * pairs; e += kThreads) {
            const int t = kFull ? e >> p.pairs_shift : e / pairs, pair = e - t * pairs;
            float c = 1.f, s = 0.f;
            if (pair < a.rotary_dim / 2) {
                const unsigned long long turn = (unsigned long long)a.frequencies[pair] *
                                                (unsigned long long)(long long)a.positions[rows.token0 + t];
                // The nearest quarter turn, and the rest, at most an eighth, in half turns to fp32's precision.
                const unsigned long long near = turn + (1ull << 61);
                const int rest = (int)((long long)(turn - (near & (3ull << 62))) >> 30);
                float sn, cs;
                sincospif((float)rest * 0x1p-33f, &sn, &cs);
                const int quarter = (int)(near >> 62);
                c = quarter & 1 ? sn : cs;
                s = quarter & 1 ? cs : sn;
                c = ((quarter + 1) & 2 ? -c : c) * a.rope_scale;
                s = (quarter & 2 ? -s : s) * a.rope_scale;
            }
            // thread pair / 8, chunk (pair % 8) / 2: threads of a group read neighbouring chunks
            float* to = reinterpret_cast<float*>(table + ((size_t)t * 4 + ((pair & 7) >> 1)) * p.per + (pair >> 3));
            to[pair & 1] = c;
            to[2 + (pair & 1)] = s;
        }
        __syncthreads();
    }
    rows.template run<kQuery, kKey>(first);
    rows.template run<kKey, kValue>(first);
    rows.template run<kValue, kNone>(first);
}

// 1 / x where multiplying by it is the same as dividing by x: x a power of two, and 1 / x one too.
float exact_inverse(float x) {
    int e;
    return frexpf(x, &e) == 0.5f && e > -120 && e < 120 ? 1.f / x : 0.f;
}

template <typename T, bool kInterleaved, int kUnit>
cudaError_t launch(const RopePlan& p, uint32_t* status, cudaStream_t stream) {
    const size_t smem = (size_t)p.tokens * 4 * p.per * sizeof(float4);
    const long long blocks = ((long long)p.a.T + p.tokens - 1) / p.tokens;
    if (p.per == p.lanes && p.a.head_dim % 16 == 0)
        norm_rope_kernel<T, kInterleaved, kUnit, true><<<(unsigned)blocks, kThreads, smem, stream>>>(p, status);
    else
        norm_rope_kernel<T, kInterleaved, kUnit, false><<<(unsigned)blocks, kThreads, smem, stream>>>(p, status);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_pairs(const RopePlan& p, uint32_t* status, cudaStream_t stream) {
    if (p.a.interleaved) return launch<T, true, 8>(p, status, stream);
    if (p.a.rotary_dim % 16 == 0) return launch<T, false, 8>(p, status, stream);
    if (p.a.rotary_dim % 8 == 0) return launch<T, false, 4>(p, status, stream);
    if (p.a.rotary_dim % 4 == 0) return launch<T, false, 2>(p, status, stream);
    return launch<T, false, 1>(p, status, stream);
}

}  // namespace

cudaError_t launch_norm_rope(const DeviceInfo& dev, const NormRopeArgs& a, uint32_t* status_word,
                             cudaStream_t stream) {
    RopePlan p{};
    p.a = a;
    p.per = (a.head_dim + 15) / 16;
    for (p.lanes = 1; p.lanes < p.per;) p.lanes *= 2;
    for (p.pairs_shift = 3; (1 << p.pairs_shift) < 8 * p.per;) ++p.pairs_shift;
    p.k_mul = exact_inverse(a.cache.k_scale);
    p.v_mul = exact_inverse(a.cache.v_scale);
    p.inv_dim = 1.f / (float)a.head_dim;
    const long long strides[10] = {a.qt, a.kt, a.vt, a.qh, a.kh, a.vh, a.qot, a.kot, a.qoh, a.koh};
    uint32_t* const bytes[10] = {&p.token_bytes[0], &p.token_bytes[1], &p.token_bytes[2], &p.head_bytes[0],
                                 &p.head_bytes[1], &p.head_bytes[2], &p.out_token_bytes[0],
                                 &p.out_token_bytes[1], &p.out_head_bytes[0], &p.out_head_bytes[1]};
    for (int k = 0; k < 10; ++k) *bytes[k] = 2u * (uint32_t)strides[k];
    p.by_q = Divisor((uint32_t)std::max(1, a.q_heads));
    p.by_kv = Divisor((uint32_t)std::max(1, a.kv_heads));
    // Tokens of a CTA, up to 16 KB of cosines and sines: the number that makes waves times a CTA's time
    // least, which is its rounds of rows, each kind's rounded up, and about kFixed rounds for cosines, sines and
    // weights. (Without kFixed 183 us instead of 175 for 40001 tokens of 48 heads of 128, 80 instead of 69 at
    // head_dim 80; kFixed = 8 the same as 2; one token a CTA 350 us, and 116 instead of 18 with one query and one key head
    // of 128 of 20001 tokens.)
    constexpr int kFixed = 2;
    const long long groups = kThreads / p.lanes, resident = (long long)kBlocks * dev.sm_count;
    long long least = LLONG_MAX;
    for (int n = 1; n <= std::min(a.T, 256 / p.per); ++n) {
        const long long blocks = (a.T + (long long)n - 1) / n;
        const long long rounds = (n * (long long)a.q_heads + groups - 1) / groups +
                                 (a.slots ? 2 : 1) * ((n * (long long)a.kv_heads + groups - 1) / groups);
        const long long cost = (blocks + resident - 1) / resident * (rounds + kFixed);
        if (n > 1 && n * (long long)std::max(a.q_heads, a.kv_heads) > 2048) break;
        if (cost < least) {
            least = cost;
            p.tokens = n;
        }
    }
    p.page_shift = -1;
    if (a.slots && (a.cache.page_size & (a.cache.page_size - 1)) == 0)
        for (p.page_shift = 0; (1 << p.page_shift) < a.cache.page_size;) ++p.page_shift;
    return a.dtype == kBf16 ? launch_pairs<__nv_bfloat16>(p, status_word, stream)
                            : launch_pairs<__half>(p, status_word, stream);
}

}  // namespace dflash
