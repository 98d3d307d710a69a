// kvcache.cu: the paged key-value cache's bookkeeping (block tables, positions, slots) and the
// store of new keys and values.
//
// Page "vllm.v1.worker.gpu.spec_decode.dflash.speculator", DFlashSpeculator.propose:
// prepare_dflash_inputs builds positions and slot mappings per request on the GPU; page
// "vllm.models.beam.nvidia.dflash2", precompute_and_store_context_kv: store_context_kv scatters
// keys and values by slot, optionally to fp8 with a scale per layer.
#include "common.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <mutex>

namespace dflash {
namespace {

// ---------------------------------------------------------------- block tables
//
//   need_r = max(0, ceil((ctx_r + n_r) / P) - held_r),  f_r = sum_{s<r} need_s,
//   start_r = sum_{s<r} n_s;  table[r, held_r + i] = free[f_r + i] for i < need_r;
//   token t of request r (i = t - start_r): position ctx_r + i, slot = page * P + position % P.
//
// One launch. Every CTA takes both running sums over all R requests itself (R * 12 bytes, read
// from L2 by all but the first) and keeps them in shared memory, so no CTA waits for another; then
// the CTAs share the tokens, the fresh pages and the rows evenly, whatever the requests' lengths
// are. A token's page is read from the old table or from the free list directly, so the slots
// do not depend on the table's new entries having been written. Bound by latency: two passes over
// the lengths, a scan and a search. 64 requests of 16 tokens take 4.8 us in a graph, 700 prompts
// of 31 to 2500 tokens 9.7 us; a call from Python takes 27 and 32 us, which is the host's.

constexpr int kTableThreads = 256;
constexpr int kTokensPerThread = 4;   // consecutive tokens: one search, then steps

// The request that owns item x: the largest r in [0, R) with sum[r] <= x. sum is non-decreasing,
// sum[0] = 0 and x < sum[R], so requests with no items are passed over.
__device__ __forceinline__ int owner_of(const int* sum, int R, int x) {
    int lo = 0, hi = R;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (sum[mid] <= x) lo = mid;
        else hi = mid;
    }
    return lo;
}

// new tokens and pages of request r; need < 0 marks a request whose lengths are refused.
__device__ __forceinline__ void request_sizes(const BlockTableArgs& a, int r, int& n, int& need) {
    const long long ctx = a.context_lens[r], add = a.new_lens[r], held = a.held_pages[r];
    n = (int)(add > 0 ? add : 0);
    const long long pages = (ctx + add + a.page_size - 1) / a.page_size;
    const bool good = ctx >= 0 && add >= 0 && held >= 0 && held <= a.max_pages &&
                      ctx <= held * a.page_size && pages <= a.max_pages &&
                      ctx + add <= (long long)INT_MAX;
    need = good ? (int)(pages > held ? pages - held : 0) : -1;
}

__global__ void __launch_bounds__(kTableThreads) block_tables_kernel(BlockTableArgs a,
                                                                     uint32_t* status) {
    extern __shared__ int table_smem[];
    int* start = table_smem;             // [R + 1] tokens before each request
    int* first = table_smem + a.R + 1;   // [R + 1] pages before each request
    __shared__ long long warp_n[kTableThreads / 32], warp_p[kTableThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

    // Running sums: each thread its own run of requests, then a scan over the threads. 64-bit,
    // so that no sum of lengths wraps; stored cut off at INT_MAX.
    const int per = (a.R + kTableThreads - 1) / kTableThreads;
    const int r0 = min(tid * per, a.R), r1 = min(r0 + per, a.R);
    long long sn = 0, sp = 0;
    bool bad = false;
    for (int r = r0; r < r1; ++r) {
        int n, need;
        request_sizes(a, r, n, need);
        bad |= need < 0;
        sn += n;
        sp += max(need, 0);
    }
    long long in = sn, ip = sp;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long on = __shfl_up_sync(0xffffffffu, in, d);
        const long long op = __shfl_up_sync(0xffffffffu, ip, d);
        if (lane >= d) {
            in += on;
            ip += op;
        }
    }
    if (lane == 31) {
        warp_n[warp] = in;
        warp_p[warp] = ip;
    }
    __syncthreads();
    long long base_n = in - sn, base_p = ip - sp;
    for (int w = 0; w < warp; ++w) {
        base_n += warp_n[w];
        base_p += warp_p[w];
    }
    for (int r = r0; r < r1; ++r) {
        int n, need;
        request_sizes(a, r, n, need);
        start[r] = (int)min(base_n, (long long)INT_MAX);
        first[r] = (int)min(base_p, (long long)INT_MAX);
        base_n += n;
        base_p += max(need, 0);
    }
    if (r1 == a.R && r0 < r1) {
        start[a.R] = (int)min(base_n, (long long)INT_MAX);
        first[a.R] = (int)min(base_p, (long long)INT_MAX);
    }
    __syncthreads();
    const int tokens = start[a.R], fresh = first[a.R];
    if (blockIdx.x == 0) {
        if (bad) atomicOr(status, kStatusBadLength);
        if (tid == 0) {
            a.pages_needed[0] = fresh;
            if (tokens > a.T) atomicOr(status, kStatusBadLength);
            if (fresh > a.n_free) atomicOr(status, kStatusNoPages);
        }
    }

    const int stride = gridDim.x * kTableThreads;
    const int at = blockIdx.x * kTableThreads + tid;
    for (int r = at; r <= a.R; r += stride) {
        a.query_start[r] = start[r];
        if (r == a.R) break;
        int n, need;
        request_sizes(a, r, n, need);
        const bool granted = need >= 0 && (need == 0 || first[r] + (long long)need <= a.n_free);
        a.kv_lens[r] = granted ? a.context_lens[r] + n : 0;
        a.held_out[r] = a.held_pages[r] + (granted ? need : 0);
    }
    for (long long j = at; j < min(fresh, a.n_free); j += stride) {   // 64 bits: j + stride may pass 2^31
        const int r = owner_of(first, a.R, (int)j);
        if (first[r + 1] > a.n_free) continue;               // refused: the list ends inside it
        a.block_table[(long long)r * a.max_pages + a.held_pages[r] + (j - first[r])] =
            a.free_pages[j];
    }
    for (long long t0 = (long long)at * kTokensPerThread; t0 < a.T;
         t0 += (long long)stride * kTokensPerThread) {
        int r = -1, end = 0, held = 0, pos = 0, row = 0, block = 0;
        long long page = 0;
        bool granted = false;
        for (int k = 0; k < kTokensPerThread; ++k) {
            const int t = (int)t0 + k;
            if (t >= a.T) break;
            if (t >= tokens) {
                a.positions[t] = 0;
                a.slots[t] = -1;
                continue;
            }
            bool look = false;
            if (t >= end) {                                  // the next request with tokens
                r = owner_of(start, a.R, t);
                end = start[r + 1];
                held = a.held_pages[r];
                int n, need;
                request_sizes(a, r, n, need);
                granted = need >= 0 && (need == 0 || first[r] + (long long)need <= a.n_free);
                pos = (int)((unsigned)a.context_lens[r] + (unsigned)(t - start[r]));
                block = granted ? pos / a.page_size : 0;
                row = granted ? pos - block * a.page_size : 0;
                look = true;
            } else {
                ++pos;
                if (++row == a.page_size) {
                    row = 0;
                    ++block;
                    look = true;
                }
            }
            if (look && granted)
                page = block < held ? a.block_table[(long long)r * a.max_pages + block]
                                    : a.free_pages[first[r] + (block - held)];
            a.positions[t] = pos;
            a.slots[t] = granted ? page * a.page_size + row : -1;
        }
    }
}

// ---------------------------------------------------------------- store
//
// A thread moves 8 elements of a key or value row at a time: 16 bytes in, 16 or 8 out. The threads of
// a block lie along a token's vectors and over tokens, so that a thread keeps its head and vector
// and finds a token's place in the cache once for several, with all of their loads in flight. The
// rows are streamed once; bound by HBM: 40001 tokens of 8 heads of 128 from bf16 to e4m3 take 43 us,
// 5.7 TB/s (with 256 threads a block, one vector of a token's 256 each, 53 us; 90 us with one token
// in flight besides).

template <typename T>
__device__ __forceinline__ float to_float(T x);
template <>
__device__ __forceinline__ float to_float<__nv_bfloat16>(__nv_bfloat16 x) {
    return __bfloat162float(x);
}
template <>
__device__ __forceinline__ float to_float<__half>(__half x) {
    return __half2float(x);
}

// x / scale in e4m3: an IEEE division, then one rounding to the nearest, clamped to 448. Where scale
// is a power of two (and its inverse one too) the product with the inverse is the same value.
template <typename T, bool kDivide>
__device__ __forceinline__ uint2 to_e4m3(const uint4& v, float scale) {
    const T* x = reinterpret_cast<const T*>(&v);
    uint32_t o[4];
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        float2 f = make_float2(to_float(x[2 * w]), to_float(x[2 * w + 1]));
        f.x = kDivide ? __fdiv_rn(f.x, scale) : f.x * scale;
        f.y = kDivide ? __fdiv_rn(f.y, scale) : f.y * scale;
        o[w] = __nv_cvt_float2_to_fp8x2(f, __NV_SATFINITE, __NV_E4M3);
    }
    return make_uint2(o[0] | (o[1] << 16), o[2] | (o[3] << 16));
}

struct StoreArgs {
    const uint16_t *key, *value;
    long long kt, kh, vt, vh;      // strides in elements
    const int64_t* slots;
    int T, vecs;                   // 8-element vectors per head row
    int across;                    // threads along a token's vectors; a divisor of the block
    int page_shift;                // -1: page_size is no power of two
    float k_mul, v_mul;            // scales, or their inverses
    KvCache cache;
};

constexpr int kStoreThreads = 128;
constexpr int kStoreTokens = 4;    // tokens a thread has in flight

template <typename T, bool kSmall, bool kDivide>
__global__ void __launch_bounds__(kStoreThreads) store_kv_kernel(StoreArgs a, uint32_t* status) {
    const int row = a.cache.kv_heads * a.vecs;               // vectors of one token's keys
    const int down = kStoreThreads / a.across;               // tokens of a block at a time
    const int x0 = threadIdx.x % a.across, y = threadIdx.x / a.across;
    const long long slots_in_pool = (long long)a.cache.num_pages * a.cache.page_size;
    const long long first = (long long)blockIdx.x * down * kStoreTokens + y;
    long long to[kStoreTokens];                              // the token's row in the cache, or -1
#pragma unroll
    for (int i = 0; i < kStoreTokens; ++i) {
        const long long t = first + (long long)i * down;
        const long long slot = t < a.T ? a.slots[t] : -1;
        to[i] = -1;
        if (slot >= slots_in_pool) {
            if (x0 == 0) atomicOr(status, kStatusBadId);
        } else if (slot >= 0) {
            const long long page = a.page_shift >= 0 ? slot >> a.page_shift : slot / a.cache.page_size;
            to[i] = page * a.cache.page_stride +
                    (slot - page * a.cache.page_size) * a.cache.token_stride;
        }
    }
    for (int x = x0; x < 2 * row; x += a.across) {
        const bool is_value = x >= row;
        const int at = is_value ? x - row : x;
        const int head = at / a.vecs, vec = at - head * a.vecs;
        const uint16_t* src = is_value ? a.value + head * a.vh : a.key + head * a.kh;
        const long long step = is_value ? a.vt : a.kt;
        const long long in_row = head * a.cache.head_stride + vec * 8;
        void* base = is_value ? a.cache.value : a.cache.key;
        uint4 v[kStoreTokens];
#pragma unroll
        for (int i = 0; i < kStoreTokens; ++i)
            if (to[i] >= 0)
                v[i] = __ldcs(reinterpret_cast<const uint4*>(
                    src + (first + (long long)i * down) * step + vec * 8));
#pragma unroll
        for (int i = 0; i < kStoreTokens; ++i) {
            if (to[i] < 0) continue;
            if constexpr (kSmall)
                *reinterpret_cast<uint2*>(static_cast<uint8_t*>(base) + to[i] + in_row) =
                    to_e4m3<T, kDivide>(v[i], is_value ? a.v_mul : a.k_mul);
            else
                *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + to[i] + in_row) = v[i];
        }
    }
}

// Whether x is a power of two with one as its inverse.
bool exact_inverse(float x) {
    int e;
    return frexpf(x, &e) == 0.5f && e > -120 && e < 120;
}

template <typename T>
void store_small(const StoreArgs& a, bool divide, unsigned blocks, uint32_t* status,
                 cudaStream_t stream) {
    if (divide) store_kv_kernel<T, true, true><<<blocks, kStoreThreads, 0, stream>>>(a, status);
    else store_kv_kernel<T, true, false><<<blocks, kStoreThreads, 0, stream>>>(a, status);
}

}  // namespace

cudaError_t launch_block_tables(const DeviceInfo& dev, const BlockTableArgs& a,
                                uint32_t* status_word, cudaStream_t stream) {
    const size_t smem = 2 * ((size_t)a.R + 1) * sizeof(int);
    static std::once_flag once[64];
    static cudaError_t attr_err[64];
    if (dev.device < 0 || dev.device >= 64) return cudaErrorInvalidDevice;
    std::call_once(once[dev.device], [&] {
        attr_err[dev.device] = cudaFuncSetAttribute(
            block_tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
            (int)(2 * ((size_t)kMaxTableRequests + 1) * sizeof(int)));
    });
    if (attr_err[dev.device] != cudaSuccess) return attr_err[dev.device];
    const long long items = std::max({((long long)a.T + kTokensPerThread - 1) / kTokensPerThread,
                                      (long long)a.R + 1, 1LL});
    const int blocks = (int)std::min<long long>((items + kTableThreads - 1) / kTableThreads,
                                                2LL * dev.sm_count);
    block_tables_kernel<<<blocks, kTableThreads, smem, stream>>>(a, status_word);
    return cudaGetLastError();
}

cudaError_t launch_store_kv(const DeviceInfo& dev, const void* key, const void* value, int dtype,
                            const int64_t* slots, int T, long long key_token_stride,
                            long long key_head_stride, long long value_token_stride,
                            long long value_head_stride, const KvCache& cache,
                            uint32_t* status_word, cudaStream_t stream) {
    const bool divide = !exact_inverse(cache.k_scale) || !exact_inverse(cache.v_scale);
    StoreArgs a{static_cast<const uint16_t*>(key), static_cast<const uint16_t*>(value),
                key_token_stride, key_head_stride, value_token_stride, value_head_stride,
                slots, T, cache.head_dim / 8, 1, -1,
                divide ? cache.k_scale : 1.f / cache.k_scale,
                divide ? cache.v_scale : 1.f / cache.v_scale, cache};
    while (a.across < kStoreThreads && a.across < 2 * cache.kv_heads * a.vecs) a.across *= 2;
    if ((cache.page_size & (cache.page_size - 1)) == 0)
        for (a.page_shift = 0; (1 << a.page_shift) < cache.page_size;) ++a.page_shift;
    const long long per_block = (long long)(kStoreThreads / a.across) * kStoreTokens;
    const unsigned blocks = (unsigned)((T + per_block - 1) / per_block);
    if (cache.dtype != kE4m3)
        store_kv_kernel<__nv_bfloat16, false, false><<<blocks, kStoreThreads, 0, stream>>>(a, status_word);
    else if (dtype == kBf16)
        store_small<__nv_bfloat16>(a, divide, blocks, status_word, stream);
    else
        store_small<__half>(a, divide, blocks, status_word, stream);
    return cudaGetLastError();
}

}  // namespace dflash
