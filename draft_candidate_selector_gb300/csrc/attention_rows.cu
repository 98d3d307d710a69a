// attention_rows.cu: attention of new tokens over the paged cache, one warp per (token, query
// head), on the CUDA cores.
//
// Page "vllm.models.beam.nvidia.dflash2", DFlash2BeamAttention: the query block attends to keys
// and values in a paged cache, inside a sliding window. For a row's visible keys j:
//   s_j = scale <q, k_j> (capped), out = sum_j e^{s_j} v_j / sum_j e^{s_j}, lse = log sum_j e^{s_j}.
//
// The warp takes 32 keys at a time. Each lane forms one key's score; the warp's maximum updates
// the running maximum m, and the sum and output so far are scaled by e^{m_old - m}. Then the 32
// values are added in turn, each lane holding 8 of the output's dimensions. Everything is fp32.
// A NaN score is passed over by the maximum and reaches the sum, and so the outputs.
#include "common.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

namespace dflash {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kWarps = 4;
constexpr int kMaxDim = 256;

template <int kType>
__device__ __forceinline__ void load8(const void* base, long long at, float (&x)[8]) {
    if constexpr (kType == kE4m3) {
        const uint2 v = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(base) + at);
        const uint32_t w[2] = {v.x, v.y};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
                (__nv_fp8x2_storage_t)(w[i >> 1] >> (16 * (i & 1))), __NV_E4M3);
            const float2 f = __half22float2(__half2(h));
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
        }
    } else {
        const uint4 v = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + at);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float2 f;
            if constexpr (kType == kBf16)
                f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]));
            else
                f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
        }
    }
}

template <int kType>
__device__ __forceinline__ void store8(void* base, long long at, const float (&x)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (kType == kBf16) {
            const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&v);
        } else {
            const __half2 v = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&v);
        }
    }
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + at) = make_uint4(w[0], w[1], w[2], w[3]);
}

template <int kQ, int kC>
__global__ void __launch_bounds__(kWarps * 32) attention_rows_kernel(AttentionArgs a,
                                                                     uint32_t* status) {
    __shared__ float q_smem[kWarps][kMaxDim];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long item = (long long)blockIdx.x * kWarps + warp;
    if (item >= (long long)a.T * a.q_heads) return;          // warps are independent
    const int token = (int)(item / a.q_heads), head = (int)(item - (long long)token * a.q_heads);
    const int D = a.cache.head_dim;
    const int kvh = head / (a.q_heads / a.cache.kv_heads);

    // The request: the last one that starts at or before the token.
    int lo = 0, hi = a.R;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a.query_start[mid] <= token) lo = mid;
        else hi = mid;
    }
    const int r = lo, t0 = a.query_start[r], t1 = a.query_start[r + 1], L = a.kv_lens[r];
    if (token < t0 || token >= t1) return;                   // behind the last request
    bool bad = L < 0 || t1 > a.T || (long long)L > (long long)a.max_pages * a.cache.page_size;
    if (bad && lane == 0) atomicOr(status, kStatusBadLength);

    float* q = q_smem[warp];
    for (int d = lane * 8; d < D; d += 256) {
        float x[8];
        load8<kQ>(a.query, token * a.q_token_stride + head * a.q_head_stride + d, x);
#pragma unroll
        for (int i = 0; i < 8; ++i) q[d + i] = x[i];
    }
    __syncwarp();

    const long long pos = (long long)L - (t1 - t0) + (token - t0);
    const long long first = a.window_left < 0 ? 0 : (pos > a.window_left ? pos - a.window_left : 0);
    const long long last = a.window_right < 0 ? L : min((long long)L, pos + a.window_right + 1);
    const int32_t* table = a.block_table + (long long)r * a.max_pages;
    const float scale = a.scale * a.cache.k_scale;
    float m = -INFINITY, sum = 0.f, o[8] = {};
    for (long long j0 = first; j0 < last && !bad; j0 += 32) {
        const long long j = j0 + lane;
        float s = -INFINITY;
        long long row = 0;
        bool off = false;
        if (j < last) {
            const int page = table[j / a.cache.page_size];
            off = page < 0 || page >= a.cache.num_pages;
            row = (off ? 0 : page) * a.cache.page_stride +
                  (j % a.cache.page_size) * a.cache.token_stride + kvh * a.cache.head_stride;
            if (!off) {
                float acc = 0.f;
                for (int d = 0; d < D; d += 8) {
                    float x[8];
                    load8<kC>(a.cache.key, row + d, x);
#pragma unroll
                    for (int i = 0; i < 8; ++i) acc = fmaf(q[d + i], x[i], acc);
                }
                s = acc * scale;
                if (a.softcap > 0.f) s = a.softcap * tanhf(s / a.softcap);
            }
        }
        if (__any_sync(kFull, off)) {
            if (lane == 0) atomicOr(status, kStatusBadId);
            bad = true;
            break;
        }
        float top = s;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, d));
        const float m_new = fmaxf(m, top);
        const float base = m_new == -INFINITY ? 0.f : m_new;
        const float keep = expf(m - base);
        const float p = j < last ? expf(s - base) : 0.f;
        float add = p;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) add += __shfl_xor_sync(kFull, add, d);
        sum = sum * keep + add;
        m = m_new;
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] *= keep;
        const int n = (int)min(32LL, last - j0);
        for (int k = 0; k < n; ++k) {
            const float pk = __shfl_sync(kFull, p, k);
            const long long rk = __shfl_sync(kFull, row, k);
            if (lane * 8 < D) {
                float x[8];
                load8<kC>(a.cache.value, rk + lane * 8, x);
#pragma unroll
                for (int i = 0; i < 8; ++i) o[i] = fmaf(pk, x[i], o[i]);
            }
        }
    }
    const float norm = bad ? NAN : (sum == 0.f ? 0.f : a.cache.v_scale / sum);
    if (lane * 8 < D) {
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = o[i] * norm;
        store8<kQ>(a.out, ((long long)token * a.q_heads + head) * D + lane * 8, x);
    }
    if (lane == 0 && a.lse)
        a.lse[(long long)token * a.q_heads + head] = bad ? NAN : (sum == 0.f ? -INFINITY
                                                                            : m + logf(sum));
}

}  // namespace

cudaError_t launch_attention_rows(const DeviceInfo&, const AttentionArgs& a, uint32_t* status_word,
                                  cudaStream_t stream) {
    const long long rows = (long long)a.T * a.q_heads;
    const unsigned blocks = (unsigned)((rows + kWarps - 1) / kWarps);
    const bool half_q = a.dtype == kFp16;
    if (a.cache.dtype == kE4m3) {
        if (half_q) attention_rows_kernel<kFp16, kE4m3><<<blocks, kWarps * 32, 0, stream>>>(a, status_word);
        else attention_rows_kernel<kBf16, kE4m3><<<blocks, kWarps * 32, 0, stream>>>(a, status_word);
    } else {
        if (half_q) attention_rows_kernel<kFp16, kFp16><<<blocks, kWarps * 32, 0, stream>>>(a, status_word);
        else attention_rows_kernel<kBf16, kBf16><<<blocks, kWarps * 32, 0, stream>>>(a, status_word);
    }
    return cudaGetLastError();
}

}  // namespace dflash
