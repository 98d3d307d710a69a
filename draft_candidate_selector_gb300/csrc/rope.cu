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
// the low 64 bits of an integer product: what is left of f_j's own rounding is 2^-33 of a turn at
// position 2^31.
#include "common.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <algorithm>
#include <cfloat>
#include <cmath>
#include <mutex>

namespace dflash {
namespace {

// A head row (one head of one token) belongs to a group of kLanes threads, the power of two at or
// above head_dim / 16; a thread holds 16 values of it, as two 16-byte vectors a and b, chosen so
// that both values of a pair are in one thread: vectors j and j + rotary_dim / 16 of the halves, or
// 2j and 2j + 1. Its eight pairs are 8j to 8j + 7 either way. (Halves that are no multiple of 8
// values long exchange the normed row through shared memory instead.)
//
// A CTA takes a run of consecutive head rows (query, key and value heads of one token, then of the
// next), kRows of them a thread, all loaded before anything else; while they travel, its threads take
// the cosines and sines of the tokens that the run touches, once each, into shared memory.
constexpr int kThreads = 256;
enum : int { kHalves = 0, kInterleaved = 1, kOddHalves = 2 };

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

// Eight values at dst (element address), as T or as e4m3 of x / scale (mul: its exact inverse, or 0).
template <typename T>
__device__ __forceinline__ void put(void* base, long long at, const float* x, bool small, float scale,
                                    float mul) {
    if (small) {
        uint32_t o[4];
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            float2 f = make_float2(x[2 * w], x[2 * w + 1]);
            f.x = mul != 0.f ? f.x * mul : __fdiv_rn(f.x, scale);
            f.y = mul != 0.f ? f.y * mul : __fdiv_rn(f.y, scale);
            o[w] = __nv_cvt_float2_to_fp8x2(f, __NV_SATFINITE, __NV_E4M3);
        }
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(base) + at) =
            make_uint2(o[0] | (o[1] << 16), o[2] | (o[3] << 16));
    } else {
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + at) =
            make_uint4(narrow<T>(x[0], x[1]), narrow<T>(x[2], x[3]), narrow<T>(x[4], x[5]),
                       narrow<T>(x[6], x[7]));
    }
}

struct RopePlan {
    NormRopeArgs a;
    long long rows;      // T * heads
    int heads;           // query, key and value heads of a token
    int vecs;            // vectors of 8 in a head
    int per;             // threads of a group that hold any: ceil(vecs / 2)
    int lanes;           // the group
    int run;             // head rows a CTA
    int tokens;          // tokens that a run touches at most
    int page_shift;      // -1: page_size is no power of two
    float k_mul, v_mul;  // inverses of the scales, where a product with them is exact; else 0
};

// Vector of a thread j's first (b: second) half; vecs or more if there is none.
template <int kMode>
__device__ __forceinline__ int vector_of(int j, int b, int rotary_dim) {
    if (kMode != kHalves) return 2 * j + b;
    const int half = rotary_dim / 16;
    return j < half ? j + b * half : 2 * j + b;
}

template <typename T, int kMode, int kRows>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(RopePlan p, uint32_t* status) {
    extern __shared__ __align__(16) float rope_smem[];
    const NormRopeArgs& a = p.a;
    // [tokens][4][per] chunks of two (cos, sin), [2][4][per] chunks of four weights, odd halves: rows
    float4* table = reinterpret_cast<float4*>(rope_smem);
    float4* weights = table + (size_t)p.tokens * 4 * p.per;
    float* exchange = reinterpret_cast<float*>(weights + 8 * p.per);
    const int tid = threadIdx.x;
    const int j = tid & (p.lanes - 1), group = tid / p.lanes, groups = kThreads / p.lanes;
    const long long row0 = (long long)blockIdx.x * p.run;
    const int token0 = (int)(row0 / p.heads), head0 = (int)(row0 - (long long)token0 * p.heads);
    const int rows = (int)min((long long)p.run, p.rows - row0);
    const int va = vector_of<kMode>(j, 0, a.rotary_dim), vb = vector_of<kMode>(j, 1, a.rotary_dim);
    const bool has_a = j < p.per, has_b = has_a && vb < p.vecs;

    uint4 xa[kRows], xb[kRows];
    long long slot[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int local = i * groups + group;
        xa[i] = xb[i] = make_uint4(0, 0, 0, 0);
        slot[i] = -1;
        if (local >= rows) continue;
        const unsigned at = head0 + local;
        const unsigned skip = at / p.heads;
        const int h = (int)(at - skip * p.heads);
        const long long t = token0 + (long long)skip;
        const uint16_t* src;
        if (h < a.q_heads)
            src = static_cast<const uint16_t*>(a.query) + t * a.qt + h * a.qh;
        else if (h < a.q_heads + a.kv_heads)
            src = static_cast<const uint16_t*>(a.key) + t * a.kt + (h - a.q_heads) * a.kh;
        else
            src = static_cast<const uint16_t*>(a.value) + t * a.vt + (h - a.q_heads - a.kv_heads) * a.vh;
        if (has_a) xa[i] = *reinterpret_cast<const uint4*>(src + 8 * va);
        if (has_b) xb[i] = *reinterpret_cast<const uint4*>(src + 8 * vb);
        if (a.slots && h >= a.q_heads) slot[i] = a.slots[t];
    }

    // Cosines and sines; pairs past rotary_dim stay as they are.
    const int pairs = 8 * p.per;
    const int touched = (head0 + rows - 1) / p.heads + 1;
    for (int e = tid; e < touched * pairs; e += kThreads) {
        const int skip = e / pairs, pair = e - skip * pairs;
        float c = 1.f, s = 0.f;
        if (pair < a.rotary_dim / 2) {
            const unsigned long long turn = (unsigned long long)a.frequencies[pair] *
                                            (unsigned long long)(long long)a.positions[token0 + skip];
            // The nearest quarter turn, and the rest, at most an eighth, in half turns to fp32's precision.
            const unsigned long long near = turn + (1ull << 61);
            const int rest = (int)((long long)(turn - (near & (3ull << 62))) >> 30);
            float sn, cs;
            sincospif((float)rest * 0x1p-33f, &sn, &cs);
            const int quarter = (int)(near >> 62);
            c = quarter & 1 ? sn : cs;
            s = quarter & 1 ? cs : sn;
            c = (quarter + 1) & 2 ? -c : c;
            s = quarter & 2 ? -s : s;
            c *= a.rope_scale;
            s *= a.rope_scale;
        }
        // thread pair / 8, chunk (pair % 8) / 2: threads of a group read neighbouring chunks
        float2* to = reinterpret_cast<float2*>(table + ((size_t)skip * 4 + (pair & 7) / 2) * p.per +
                                               (pair >> 3));
        to[pair & 1] = make_float2(c, s);
    }
    for (int e = tid; e < 2 * 16 * p.per; e += kThreads) {
        const int of = e / (16 * p.per), x = e - of * 16 * p.per;
        const int chunk = x / (4 * p.per), y = x - chunk * 4 * p.per;
        const int dim = 8 * vector_of<kMode>(y >> 2, chunk >> 1, a.rotary_dim) + 4 * (chunk & 1) + (y & 3);
        const void* w = of ? a.k_weight : a.q_weight;
        float v = 1.f;
        if (w && dim < a.head_dim)
            v = a.weight_dtype == kFp32 ? static_cast<const float*>(w)[dim]
                                        : widen<T>(static_cast<const uint16_t*>(w)[dim]).x;
        reinterpret_cast<float*>(weights)[e] = v;
    }
    __syncthreads();

#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int local = i * groups + group;
        const unsigned at = head0 + local;
        const unsigned skip = at / p.heads;
        const int h = (int)(at - skip * p.heads);
        const long long t = token0 + (long long)skip;
        const bool live = local < rows;
        const bool is_key = h >= a.q_heads, is_value = h >= a.q_heads + a.kv_heads;
        float x[16];
        const uint32_t raw[8] = {xa[i].x, xa[i].y, xa[i].z, xa[i].w, xb[i].x, xb[i].y, xb[i].z, xb[i].w};
#pragma unroll
        for (int w = 0; w < 8; ++w) {
            const float2 f = widen<T>(raw[w]);
            x[2 * w] = f.x;
            x[2 * w + 1] = f.y;
        }
        const bool normed = !is_value && (is_key ? a.k_weight : a.q_weight) != nullptr;
        if (a.q_weight || a.k_weight) {                      // every lane takes part in the exchanges
            float sum = 0.f;
#pragma unroll
            for (int w = 0; w < 16; ++w) sum = fmaf(x[w], x[w], sum);
            for (int d = p.lanes / 2; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
            // Squares past fp32's range (bf16 values from 2^60 on): once more, 2^-72 as large.
            if (__any_sync(0xffffffffu, sum > FLT_MAX && normed)) {
                const float down = sum > FLT_MAX && normed ? 0x1p-72f : 1.f;
                sum = 0.f;
#pragma unroll
                for (int w = 0; w < 16; ++w) {
                    x[w] *= down;
                    sum = fmaf(x[w], x[w], sum);
                }
                for (int d = p.lanes / 2; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
            }
            if (normed) {
                const float r = rsqrtf(sum / (float)a.head_dim + a.eps);
                const float4* w4 = weights + (is_key ? 4 * p.per : 0) + (has_a ? j : 0);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const float4 w = w4[c * p.per];
                    x[4 * c] *= r * w.x;
                    x[4 * c + 1] *= r * w.y;
                    x[4 * c + 2] *= r * w.z;
                    x[4 * c + 3] *= r * w.w;
                }
            }
        }
        if constexpr (kMode == kOddHalves) {
            float* row = exchange + group * a.head_dim;
            __syncwarp();
            if (live && !is_value) {
                for (int w = 0; w < 8; ++w) {
                    if (has_a) row[8 * va + w] = x[w];
                    if (has_b) row[8 * vb + w] = x[8 + w];
                }
            }
            __syncwarp();
            if (live && !is_value && has_a) {
                const int half = a.rotary_dim / 2;
                const float4* cs = table + (size_t)skip * 4 * p.per;
                for (int w = 0; w < 16; ++w) {
                    const int dim = 16 * j + w;
                    if (dim >= a.rotary_dim) continue;
                    const int pair = dim < half ? dim : dim - half;
                    const float2 f = reinterpret_cast<const float2*>(
                        cs + (size_t)((pair & 7) / 2) * p.per + (pair >> 3))[pair & 1];
                    x[w] = dim < half ? x[w] * f.x - row[dim + half] * f.y
                                      : x[w] * f.x + row[dim - half] * f.y;
                }
            }
        } else if (live && !is_value && has_a && a.rotary_dim > 0) {
            const float4* cs = table + (size_t)skip * 4 * p.per + j;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const float4 f = cs[c * p.per];          // two pairs
                const int u0 = kMode == kHalves ? 2 * c : 4 * c, u1 = kMode == kHalves ? u0 + 8 : u0 + 1;
                const int w0 = kMode == kHalves ? u0 + 1 : u0 + 2, w1 = kMode == kHalves ? u1 + 1 : u1 + 2;
                const float x0 = x[u0], x1 = x[u1], y0 = x[w0], y1 = x[w1];
                x[u0] = x0 * f.x - x1 * f.y;
                x[u1] = x1 * f.x + x0 * f.y;
                x[w0] = y0 * f.z - y1 * f.w;
                x[w1] = y1 * f.z + y0 * f.w;
            }
        }
        if (!live || !has_a) continue;
        if (!is_key) {
            const long long to = t * a.qot + h * a.qoh;
            put<T>(a.query_out, to + 8 * va, x, false, 1.f, 1.f);
            if (has_b) put<T>(a.query_out, to + 8 * vb, x + 8, false, 1.f, 1.f);
        } else if (!a.slots) {
            const long long to = t * a.kot + (h - a.q_heads) * a.koh;
            put<T>(a.key_out, to + 8 * va, x, false, 1.f, 1.f);
            if (has_b) put<T>(a.key_out, to + 8 * vb, x + 8, false, 1.f, 1.f);
        } else if (slot[i] >= (long long)a.cache.num_pages * a.cache.page_size) {
            if (j == 0) atomicOr(status, kStatusBadId);
        } else if (slot[i] >= 0) {
            const long long page = p.page_shift >= 0 ? slot[i] >> p.page_shift : slot[i] / a.cache.page_size;
            const int head = is_value ? h - a.q_heads - a.kv_heads : h - a.q_heads;
            const long long to = page * a.cache.page_stride +
                                 (slot[i] - page * a.cache.page_size) * a.cache.token_stride +
                                 head * a.cache.head_stride;
            const bool small = a.cache.dtype == kE4m3;
            void* base = is_value ? a.cache.value : a.cache.key;
            const float scale = is_value ? a.cache.v_scale : a.cache.k_scale;
            const float mul = is_value ? p.v_mul : p.k_mul;
            if (is_value && !small) {                        // the bits as they are
                uint16_t* copy = static_cast<uint16_t*>(base) + to;
                *reinterpret_cast<uint4*>(copy + 8 * va) = xa[i];
                if (has_b) *reinterpret_cast<uint4*>(copy + 8 * vb) = xb[i];
                continue;
            }
            put<T>(base, to + 8 * va, x, small, scale, mul);
            if (has_b) put<T>(base, to + 8 * vb, x + 8, small, scale, mul);
        }
    }
}

// 1 / x where multiplying by it is the same as dividing by x: x a power of two, and 1 / x one too.
float exact_inverse(float x) {
    int e;
    return frexpf(x, &e) == 0.5f && e > -120 && e < 120 ? 1.f / x : 0.f;
}

template <typename T, int kMode, int kRows>
cudaError_t launch(const DeviceInfo& dev, RopePlan p, uint32_t* status, cudaStream_t stream) {
    const int groups = kThreads / p.lanes;
    p.run = groups * kRows;
    p.tokens = (p.run - 1) / p.heads + 2;
    const size_t smem = ((size_t)p.tokens * 4 * p.per + 8 * p.per) * sizeof(float4) +
                        (kMode == kOddHalves ? (size_t)groups * p.a.head_dim * sizeof(float) : 0);
    static std::once_flag once[64];
    static cudaError_t err[64];
    if (dev.device < 0 || dev.device >= 64) return cudaErrorInvalidDevice;
    std::call_once(once[dev.device], [&] {
        err[dev.device] = cudaFuncSetAttribute(norm_rope_kernel<T, kMode, kRows>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, 100 * 1024);
    });
    if (err[dev.device] != cudaSuccess) return err[dev.device];
    const long long blocks = (p.rows + p.run - 1) / p.run;
    norm_rope_kernel<T, kMode, kRows><<<(unsigned)blocks, kThreads, smem, stream>>>(p, status);
    return cudaGetLastError();
}

template <typename T, int kMode>
cudaError_t launch_rows(const DeviceInfo& dev, const RopePlan& p, uint32_t* status,
                        cudaStream_t stream) {
    return launch<T, kMode, 1>(dev, p, status, stream);
}

template <typename T>
cudaError_t launch_mode(const DeviceInfo& dev, const RopePlan& p, uint32_t* status,
                        cudaStream_t stream) {
    if (p.a.interleaved) return launch_rows<T, kInterleaved>(dev, p, status, stream);
    if (p.a.rotary_dim % 16 == 0) return launch_rows<T, kHalves>(dev, p, status, stream);
    return launch_rows<T, kOddHalves>(dev, p, status, stream);
}

}  // namespace

cudaError_t launch_norm_rope(const DeviceInfo& dev, const NormRopeArgs& a, uint32_t* status_word,
                             cudaStream_t stream) {
    RopePlan p{};
    p.a = a;
    p.heads = a.q_heads + (a.slots ? 2 : 1) * a.kv_heads;
    p.rows = (long long)a.T * p.heads;
    p.vecs = a.head_dim / 8;
    p.per = (p.vecs + 1) / 2;
    for (p.lanes = 1; p.lanes < p.per;) p.lanes *= 2;
    p.k_mul = exact_inverse(a.cache.k_scale);
    p.v_mul = exact_inverse(a.cache.v_scale);
    p.page_shift = -1;
    if (a.slots && (a.cache.page_size & (a.cache.page_size - 1)) == 0)
        for (p.page_shift = 0; (1 << p.page_shift) < a.cache.page_size;) ++p.page_shift;
    return a.dtype == kBf16 ? launch_mode<__nv_bfloat16>(dev, p, status_word, stream)
                            : launch_mode<__half>(dev, p, status_word, stream);
}

}  // namespace dflash
