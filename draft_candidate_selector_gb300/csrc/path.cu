// path.cu: paths through each request's edge scores: the best one, and one drawn at random.
//
// Reading (the pages show no consumer of the edge scores): page
// "vllm.models.beam.nvidia.dflash2", module docstring: the selector rescores the top-k tokens
// at each block position against the token before it. The best path picks one candidate per
// step so that the sum over p of E[r,p,c_{p-1},c_p] is largest; at p = 0 the predecessor row is
// q = 0 (every q row there is the anchor's). Max-sum dynamic programming over the steps in
// fp32, in a fixed order with a fixed tie rule, so the choice is exactly reproducible:
//   V_0[c] = E[r,0,0,c];
//   V_p[c] = running maximum over q = 0..K-1 of V_{p-1}[q] + E[r,p,q,c], replaced only by a
//            strictly larger sum (ties keep the lower q; a NaN neither replaces nor is
//            replaced);
//   the last step's candidate is the running maximum of V_{S-1} (same rule), and the path
//   follows the kept predecessors back.
//
// Design: one 128-thread CTA per request. Thread (c, g), c = 0..31 the candidate column and
// g = 0..3 a quarter of the predecessors (q = 8g .. 8g+7), forms its 8 sums V_{p-1}[q] +
// E[r,p,q,c], reduces them with a 3-level tree, and two ordered shuffle levels combine the
// four quarters; every combine keeps exactly the running maximum's choice (scan_combine). The
// CTA stages the K x K blocks of the next steps in a shared-memory ring with cp.async
// (16-byte copies when K is even and the scores are 16-byte aligned, 4-byte ones otherwise), so a step's update runs while
// later steps' blocks are in flight; one barrier per step. V_{p-1} is double-buffered in
// shared memory, and the kept predecessors go to shared memory (S x 32 bytes). Thread 0
// takes the last step's choice and walks the kept predecessors back; the threads then write
// the path and its token ids in parallel. Reads R*S*K*K*4 bytes of E once. No waits on other
// CTAs.
//
// The drawn path takes the edge scores as the drafter's own distribution of each token given the
// one before it, softmax over c of E[r,p,c_{p-1},c] / T, and inverts its running sum at a number that
// the caller drew.
#include "common.cuh"
#include "ptx.cuh"

#include <algorithm>
#include <cfloat>
#include <cmath>

namespace dflash {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kThreads = 128;
constexpr int kDepth = 8;                // ring stages (steps in flight: kDepth - 1)
constexpr int kMaxK = 32;
constexpr int kQuarter = kMaxK / 4;      // predecessors per thread

// Shared bytes: the ring [kDepth][K*K] floats, V [2][32] floats, the kept predecessors
// [S][32] and the path [S], 16-byte rounded.
__host__ __device__ inline size_t path_ring_bytes(int K) { return (size_t)kDepth * K * K * 4; }
__host__ __device__ inline size_t path_smem_bytes(int S, int K) {
    return path_ring_bytes(K) + 2 * kMaxK * 4 + (((size_t)S * 33 + 15) & ~(size_t)15);
}

__device__ __forceinline__ void cp_async4(void* dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(
                     (uint32_t)__cvta_generic_to_shared(dst)),
                 "l"(src)
                 : "memory");
}
__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                     (uint32_t)__cvta_generic_to_shared(dst)),
                 "l"(src)
                 : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
    asm volatile("cp.async.commit_group;" ::: "memory");
}
// All but the newest kDepth - 2 groups of this thread have landed.
__device__ __forceinline__ void cp_async_wait_ring() {
    asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 2) : "memory");
}

// This thread's share of the copy of step p's K x K block into ring stage p % kDepth. When
// every block starts on a 16-byte boundary (K even and a 16-byte aligned base; `wide`), the
// copy moves 16 bytes per thread and instruction; otherwise 4.
__device__ __forceinline__ void stage_step(float* ring, const float* E, int p, int K, int tid,
                                           bool wide) {
    const int n = K * K;
    float* dst = ring + (size_t)(p % kDepth) * n;
    const float* src = E + (size_t)p * n;
    if (wide) {
        for (int i = tid * 4; i < n; i += kThreads * 4) cp_async16(dst + i, src + i);
    } else {
        for (int i = tid; i < n; i += kThreads) cp_async4(dst + i, src + i);
    }
}

// Combine two pieces of a left-to-right running maximum: (av, ai) covers lower indices than
// (bv, bi). The result is what the scan keeps over both: a strictly larger value replaces;
// ties keep the lower index; a NaN at index 0 sticks (nothing compares larger than it), and
// any other NaN is passed over (it never compares larger). Associative for adjacent pieces,
// so a tree over the indices gives exactly the scan's choice.
__device__ __forceinline__ void scan_combine(float& av, int& ai, float bv, int bi) {
    const bool a_nan = av != av;
    const bool take_b = a_nan ? (ai != 0) : (bv > av);
    if (take_b) {
        av = bv;
        ai = bi;
    }
}

// One ordered level across lanes lane and lane ^ m: the lane whose bit m is clear holds the
// lower indices. Both lanes end with the combined piece.
__device__ __forceinline__ void lane_combine(float& v, int& i, int lane, int m) {
    const float ov = __shfl_xor_sync(kFull, v, m);
    const int oi = __shfl_xor_sync(kFull, i, m);
    if (lane & m) {
        float lv = ov;
        int li = oi;
        scan_combine(lv, li, v, i);
        v = lv;
        i = li;
    } else {
        scan_combine(v, i, ov, oi);
    }
}

__global__ void __launch_bounds__(kThreads)
best_path_kernel(const float* __restrict__ edges, const int32_t* __restrict__ cand, int R, int S,
                 int K, int32_t* __restrict__ path, int32_t* __restrict__ tokens,
                 float* __restrict__ score) {
    extern __shared__ __align__(16) uint8_t path_smem[];
    const int tid = threadIdx.x;
    const int lane = tid & 31;
    const int c = (tid >> 5) * 8 + (lane >> 2);          // candidate column
    const int g = lane & 3;                              // predecessor quarter
    const long long r = blockIdx.x;
    float* ring = reinterpret_cast<float*>(path_smem);                   // [kDepth][K*K]
    float* vbuf = reinterpret_cast<float*>(path_smem + path_ring_bytes(K));   // [2][32]
    uint8_t* keep = reinterpret_cast<uint8_t*>(vbuf + 2 * kMaxK);        // [S][32]
    uint8_t* chosen = keep + (size_t)S * 32;                             // [S]
    const float* E = edges + (size_t)r * S * K * K;
    const bool live = c < K;
    const bool wide = (K & 1) == 0 && (reinterpret_cast<uintptr_t>(edges) & 15) == 0;

    for (int p = 0; p < kDepth; ++p) {                   // prologue: steps 0 .. kDepth-1
        if (p < S) stage_step(ring, E, p, K, tid, wide);
        cp_async_commit();
    }
    for (int p = 0; p < S; ++p) {
        cp_async_wait_ring();                            // step p has landed (this thread's part)
        __syncthreads();                                 // ... everyone's; step p-1 is finished
        if (p >= 1) {
            // Refill the stage step p-1 used. One group per step, empty past the last step,
            // so that before step p's wait exactly p + kDepth - 1 groups are committed and
            // waiting for all but the newest kDepth - 2 covers step p.
            if (p - 1 + kDepth < S) stage_step(ring, E, p - 1 + kDepth, K, tid, wide);
            cp_async_commit();
        }
        const float* Ep = ring + (size_t)(p % kDepth) * K * K;
        if (p == 0) {
            if (g == 0 && live) vbuf[c] = Ep[c];         // predecessor row q = 0
            continue;
        }
        const float* vprev = vbuf + ((p - 1) & 1) * kMaxK;
        float s[kQuarter];
        int at[kQuarter];
#pragma unroll
        for (int j = 0; j < kQuarter; ++j) {
            const int q = g * kQuarter + j;
            at[j] = q;
            s[j] = (live && q < K) ? vprev[q] + Ep[q * K + c] : -INFINITY;
        }
#pragma unroll
        for (int w = 1; w < kQuarter; w <<= 1) {
#pragma unroll
            for (int j = 0; j + w < kQuarter; j += 2 * w) scan_combine(s[j], at[j], s[j + w], at[j + w]);
        }
        float v = s[0];
        int bq = at[0];
        lane_combine(v, bq, lane, 1);                    // quarters 0+1 and 2+3
        lane_combine(v, bq, lane, 2);                    // then the halves
        if (g == 0 && live) {
            vbuf[(p & 1) * kMaxK + c] = v;
            keep[p * 32 + c] = (uint8_t)bq;
        }
    }
    __syncthreads();
    if (tid == 0) {
        // The last step's choice: the running maximum over c, then the kept predecessors.
        const float* vl = vbuf + ((S - 1) & 1) * kMaxK;
        int cur = 0;
        float vb = vl[0];
        for (int j = 1; j < K; ++j) {
            if (vl[j] > vb) {
                vb = vl[j];
                cur = j;
            }
        }
        score[r] = vb;
        for (int p = S - 1; p >= 0; --p) {
            chosen[p] = (uint8_t)cur;
            if (p > 0) cur = keep[p * 32 + cur];
        }
    }
    __syncthreads();
    for (int p = tid; p < S; p += kThreads) {
        const int cc = chosen[p];
        path[(size_t)r * S + p] = cc;
        tokens[(size_t)r * S + p] = cand[((size_t)r * S + p) * K + cc];
    }
}

// ---------------------------------------------------------------- a drawn path
//
//   w_c = exp((E[p, c_{p-1}, c] - max) / T),  c_p = the smallest c with sum_{j<=c} w_j > u_p sum_j w_j
//
// The choice is the one that exact sums give. Sums are taken in fp32 first, and where u_p sum_j w_j
// lies within kSlack of the sum from one of the borders, again in fp64. The fp32 error: exponents are
// rounded four times (difference, log2(e) / T twice, product), 2^-22 of |z|, and sum p |z| <= ln 32 + 1; ex2
// is within 2^-22, 32 additions within 2^-19: in all below 2^-18 of the sum. A choice in about ten thousand is
// taken again.
//
// A CTA a request. Every row's choice is made, a thread a row, whether the path comes through it or not: following
// the path is then a look-up for each step. (One warp that made the choices along the path, a maximum, an
// exponential and a scan for each, took 15 us for 15 steps, this 5.) Rows lie in shared memory at a distance that
// spreads threads over the banks. The distributions are then taken for the path's rows, a warp a step.
// Bound by latency; 512 requests of 15 steps of 32 also read 31 MB of edges, 4.7 us at the copy rate.
constexpr float kSlack = 0x1p-17f;
constexpr int kSampleThreads = 256;
constexpr float kLog2e = 1.4426950408889634f;

// The order of floats as unsigned numbers; NaN lowest.
__device__ __forceinline__ uint32_t order_of(float x) {
    const uint32_t b = __float_as_uint(x);
    return x != x ? 0u : (b & 0x80000000u) ? ~b : b | 0x80000000u;
}

// The first lane with w > 0 whose running sum of w passes u times the sum of all; the last with w > 0 if none does.
__device__ __forceinline__ int invert(double w, double u, int lane) {
    double run = w;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const double other = __shfl_up_sync(kFull, run, d);
        if (lane >= d) run += other;
    }
    const double total = __shfl_sync(kFull, run, 31);
    // (Lanes add in different orders, so one without weight may be a rounding past the lane before it.)
    const unsigned past = __ballot_sync(kFull, w > 0.0 && run > u * total), any = __ballot_sync(kFull, w > 0.0);
    return past ? __ffs(past) - 1 : 31 - __clz(any | 1u);
}

// T, its inverse in two floats, and whether it is greedy.
struct PathTemperature {
    float t, inv, inv_low;
    bool greedy;
    __device__ __forceinline__ explicit PathTemperature(float x) {
        greedy = !(x > 0.f);                             // NaN too
        t = fmaxf(x, 0x1p-100f);
        inv = greedy ? 0.f : 1.f / t;
        inv_low = t < 0x1p60f ? inv * fmaf(-t, inv, 1.f) : 0.f;
    }
};

// The choice in a row of K scores at `row`, and 0x80 if fp32 sums do not settle it. One thread. Weights take the
// scores' place.
template <int kVec>
__device__ __forceinline__ uint32_t choose(float* row, int K, float u, const PathTemperature& t) {
    float m = -INFINITY;
    int first = -1;
    auto each = [&](bool back, auto&& f) {
        for (int c = 0; c < K; c += kVec) {
            float e[kVec];
            if constexpr (kVec == 4) {
                const float4 v = *reinterpret_cast<const float4*>(row + c);
                e[0] = v.x, e[1] = v.y, e[2] = v.z, e[3] = v.w;
            } else {
                e[0] = row[c];
            }
#pragma unroll
            for (int k = 0; k < kVec; ++k) f(c + k, e[k]);
            if (!back) continue;
            if constexpr (kVec == 4) *reinterpret_cast<float4*>(row + c) = make_float4(e[0], e[1], e[2], e[3]);
            else row[c] = e[0];
        }
    };
    each(false, [&](int c, float e) {
        if (e > m || (first < 0 && e == e)) {            // -0 equals 0
            m = e;
            first = c;
        }
    });
    if (t.greedy || !(fabsf(m) < INFINITY)) return max(first, 0);
    const float scale = kLog2e * t.inv;
    float total = 0.f;
    each(true, [&](int, float& e) {
        e = e > -INFINITY ? ptx::ex2(fmaxf(e - m, -FLT_MAX) * scale) : 0.f;
        total += e;
    });
    const float border = u * total;
    float run = 0.f, near = INFINITY;
    int pick = -1, last = 0;
    each(false, [&](int c, float w) {
        run += w;
        near = fminf(near, fabsf(run - border));
        if (w > 0.f) last = c;
        if (pick < 0 && run > border) pick = c;
    });
    return (uint32_t)(pick < 0 ? last : pick) | (near <= kSlack * total ? 0x80u : 0u);
}

// chunk: steps that are in shared memory at a time; stride: floats from row to row there.
template <int kVec>
__global__ void __launch_bounds__(kSampleThreads) sample_path_kernel(SamplePathArgs a, int chunk, int stride) {
    extern __shared__ __align__(16) uint8_t path_smem[];
    const int tid = threadIdx.x, lane = tid & 31, K = a.K, S = a.S;
    const long long r = blockIdx.x;
    float* rows = reinterpret_cast<float*>(path_smem);                        // [chunk * K][stride]
    float* u = rows + (size_t)chunk * K * stride;                             // [S]
    uint8_t* picks = reinterpret_cast<uint8_t*>(u + S);                       // [chunk * K]
    uint8_t* chosen = picks + chunk * K;                                      // [S]
    const float* E = a.edges + (size_t)r * S * K * K;
    // numbers outside [0, 1) count as the nearer end, NaN as 0
    for (int p = tid; p < S; p += kSampleThreads)
        u[p] = fminf(fmaxf(a.uniforms[(size_t)r * S + p], 0.f), 1.f - 0x1p-24f);
    const PathTemperature t(a.temperatures ? a.temperatures[r] : a.temperature);
    int before = 0;                                      // the row of step 0 is q = 0
    for (int p0 = 0; p0 < S; p0 += chunk) {
        const int steps = min(chunk, S - p0), n = steps * K;
        const float* from = E + (size_t)p0 * K * K;
        // A run of threads copies a row.
        const int across = K / kVec, down = kSampleThreads / across;
        const int x = tid % across * kVec, y = tid / across;
        if (y < down)
            for (int i = y; i < n; i += down) {
                if constexpr (kVec == 4) cp_async16(rows + i * stride + x, from + (size_t)i * K + x);
                else cp_async4(rows + i * stride + x, from + (size_t)i * K + x);
            }
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncthreads();
        for (int i = tid; i < n; i += kSampleThreads)
            if (p0 > 0 || i == 0 || i >= K) picks[i] = (uint8_t)choose<kVec>(rows + i * stride, K, u[p0 + i / K], t);
        __syncthreads();
        if (tid < 32) {
            for (int p = 0; p < steps; ++p) {
                const int i = p * K + before;
                int pick = picks[i] & 0x7f;
                if (picks[i] & 0x80) {
                    const float e = lane < K ? from[(size_t)i * K + lane] : NAN;
                    const uint32_t order = order_of(e), top = __reduce_max_sync(kFull, order);
                    const float m = __shfl_sync(kFull, e, __ffs(__ballot_sync(kFull, order == top)) - 1);
                    const double w = e > -INFINITY ? exp(((double)e - (double)m) / (double)t.t) : 0.0;
                    pick = invert(w, (double)u[p0 + p], lane);
                }
                if (lane == 0) chosen[p0 + p] = (uint8_t)pick;
                before = pick;
            }
        }
        __syncthreads();
        // The distributions along the path.
        for (int p = tid >> 5; p < steps; p += kSampleThreads / 32) {
            const int at = p0 + p, i = p * K + (at > 0 ? chosen[at - 1] : 0);
            const float e = lane < K ? from[(size_t)i * K + lane] + 0.f : NAN;   // no -0
            const uint32_t order = order_of(e), top = __reduce_max_sync(kFull, order);
            // the largest score (of a row with one): its first lane
            const int first = __ffs(__ballot_sync(kFull, order == top)) - 1;
            const float m = __shfl_sync(kFull, e, first);
            float prob = lane == first ? 1.f : 0.f;
            if (!t.greedy && fabsf(m) < INFINITY) {      // else nothing to draw from: the largest
                float w = 0.f;
                if (e > -INFINITY) {
                    // z in two floats; exp(z_low) = 1 + z_low
                    const float d = fmaxf(__fsub_rn(e, m), -FLT_MAX), back = __fsub_rn(d, e);
                    const float d_low = __fsub_rn(__fsub_rn(e, __fsub_rn(d, back)), __fadd_rn(m, back));
                    const float z = __fmul_rn(d, t.inv);
                    const float z_low = fmaf(d, t.inv_low, fmaf(d_low, t.inv, fmaf(d, t.inv, -z)));
                    w = expf(z);
                    if (z > -100.f) w = fmaf(w, z_low, w);
                }
                float total = w;
#pragma unroll
                for (int d = 16; d > 0; d >>= 1) total += __shfl_xor_sync(kFull, total, d);
                prob = w / total;
            }
            if (lane < K) a.probs[((size_t)r * S + at) * K + lane] = prob;
        }
        __syncthreads();
    }
    for (int p = tid; p < S; p += kSampleThreads) {
        const int c = chosen[p];
        a.path[(size_t)r * S + p] = c;
        a.tokens[(size_t)r * S + p] = a.cand_ids[((size_t)r * S + p) * K + c];
    }
}

}  // namespace

cudaError_t launch_sample_path(const SamplePathArgs& a, cudaStream_t stream) {
    // Rows of whole 16-byte pieces lie 16 bytes apart, which spreads 8 threads' pieces over the banks (K = 4: two
    // at a time); others at an odd distance.
    const bool wide = a.K % 4 == 0 && (reinterpret_cast<uintptr_t>(a.edges) & 15) == 0;
    const int stride = wide ? a.K + 4 : a.K | 1;
    // (512 requests of 15 steps of 32: 22 us, 28 with single floats.)
    constexpr int kRoom = 40 * 1024;                     // five CTAs an SM, and no more than 48 KB in all; half: 26 us
    const int most = kRoom / (a.K * stride * 4), chunks = (a.S + most - 1) / most;
    const int chunk = (a.S + chunks - 1) / chunks;
    const size_t smem = (size_t)chunk * a.K * stride * 4 + (size_t)a.S * 5 + (size_t)chunk * a.K;
    if (wide) sample_path_kernel<4><<<(unsigned)a.R, kSampleThreads, smem, stream>>>(a, chunk, stride);
    else sample_path_kernel<1><<<(unsigned)a.R, kSampleThreads, smem, stream>>>(a, chunk, stride);
    return cudaGetLastError();
}

cudaError_t launch_best_path(const float* edges, const int32_t* cand_ids, int R, int S, int K,
                             int32_t* path, int32_t* tokens, float* score, cudaStream_t stream) {
    // At most 32 KB of ring + 8.5 KB (S = 256): under the default 48 KB, no opt-in needed.
    const size_t smem = path_smem_bytes(S, K);
    best_path_kernel<<<(unsigned)R, kThreads, smem, stream>>>(edges, cand_ids, R, S, K, path,
                                                             tokens, score);
    return cudaGetLastError();
}

}  // namespace dflash
