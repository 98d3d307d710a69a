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
// do not depend on the table's new entries having been written.

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
    for (int j = at; j < min(fresh, a.n_free); j += stride) {
        const int r = owner_of(first, a.R, j);
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
// One thread moves 8 elements of a key or value row: 16 bytes in, 16 or 8 out. The rows are
// streamed once; nothing is reused. Bound by HBM.

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

// x / scale in e4m3: an IEEE division, then one rounding to the nearest, clamped to 448.
template <typename T>
__device__ __forceinline__ uint2 to_e4m3(const uint4& v, float scale) {
    const T* x = reinterpret_cast<const T*>(&v);
    uint32_t o[2];
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        uint32_t lo = __nv_cvt_float2_to_fp8x2(
            make_float2(__fdiv_rn(to_float(x[4 * w]), scale),
                        __fdiv_rn(to_float(x[4 * w + 1]), scale)), __NV_SATFINITE, __NV_E4M3);
        uint32_t hi = __nv_cvt_float2_to_fp8x2(
            make_float2(__fdiv_rn(to_float(x[4 * w + 2]), scale),
                        __fdiv_rn(to_float(x[4 * w + 3]), scale)), __NV_SATFINITE, __NV_E4M3);
        o[w] = lo | (hi << 16);
    }
    return make_uint2(o[0], o[1]);
}

struct StoreArgs {
    const uint16_t *key, *value;
    long long kt, kh, vt, vh;      // strides in elements
    const int64_t* slots;
    int T, vecs;                   // 8-element vectors per head row
    KvCache cache;
};

constexpr int kStoreThreads = 256;

template <typename T, bool kSmall>
__global__ void __launch_bounds__(kStoreThreads) store_kv_kernel(StoreArgs a, uint32_t* status) {
    const int row = a.cache.kv_heads * a.vecs;               // vectors of one token's keys
    const long long n = 2LL * a.T * row;
    const long long slots_in_pool = (long long)a.cache.num_pages * a.cache.page_size;
    for (long long i = (long long)blockIdx.x * kStoreThreads + threadIdx.x; i < n;
         i += (long long)gridDim.x * kStoreThreads) {
        const int token = (int)(i / (2 * row));
        int at = (int)(i - (long long)token * 2 * row);
        const bool is_value = at >= row;
        at -= is_value ? row : 0;
        const int head = at / a.vecs, vec = at - head * a.vecs;
        const long long slot = a.slots[token];
        if (slot < 0) continue;
        if (slot >= slots_in_pool) {
            atomicOr(status, kStatusBadId);
            continue;
        }
        const uint16_t* src = is_value ? a.value + token * a.vt + head * a.vh
                                       : a.key + token * a.kt + head * a.kh;
        const uint4 v = __ldcs(reinterpret_cast<const uint4*>(src + vec * 8));
        const long long page = slot / a.cache.page_size;
        const long long to = page * a.cache.page_stride +
                             (slot - page * a.cache.page_size) * a.cache.token_stride +
                             head * a.cache.head_stride + vec * 8;
        void* base = is_value ? a.cache.value : a.cache.key;
        if constexpr (kSmall)
            *reinterpret_cast<uint2*>(static_cast<uint8_t*>(base) + to) =
                to_e4m3<T>(v, is_value ? a.cache.v_scale : a.cache.k_scale);
        else
            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + to) = v;
    }
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
    StoreArgs a{static_cast<const uint16_t*>(key), static_cast<const uint16_t*>(value),
                key_token_stride, key_head_stride, value_token_stride, value_head_stride,
                slots, T, cache.head_dim / 8, cache};
    const long long n = 2LL * T * cache.kv_heads * a.vecs;
    const int blocks = (int)std::min<long long>((n + kStoreThreads - 1) / kStoreThreads,
                                                16LL * dev.sm_count);
    if (cache.dtype != kE4m3)
        store_kv_kernel<__nv_bfloat16, false><<<blocks, kStoreThreads, 0, stream>>>(a, status_word);
    else if (dtype == kBf16)
        store_kv_kernel<__nv_bfloat16, true><<<blocks, kStoreThreads, 0, stream>>>(a, status_word);
    else
        store_kv_kernel<__half, true><<<blocks, kStoreThreads, 0, stream>>>(a, status_word);
    return cudaGetLastError();
}

}  // namespace dflash
