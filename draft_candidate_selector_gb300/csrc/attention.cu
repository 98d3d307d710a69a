// attention.cu: which attention kernel a call takes, its workspace and its launch. The tensor-core
// kernel is in attention.cuh; its builds are in attention_16bit.cu and attention_e4m3.cu.
#include "attention.cuh"

namespace dflash {
namespace {

size_t align256(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace

size_t attention_workspace_bytes(const DeviceInfo& dev, int D) {
    return align256((size_t)(dev.sm_count + 1) * sizeof(int4)) +
           2 * (size_t)dev.sm_count * part_floats(D) * sizeof(float);
}

bool attention_may_use_tensor_cores(int head_dim, int g, int R) {
    return (head_dim == 64 || head_dim == 128) && g <= BM && R <= kMaxTableRequests;
}

bool attention_on_tensor_cores(const AttentionArgs& a) {
    const KvCache& c = a.cache;
    const auto fits = [](long long stride, long long dim) {   // a tensor map's stride
        return dim == 1 || (stride > 0 && stride < (1LL << 38));
    };
    return attention_may_use_tensor_cores(c.head_dim, a.q_heads / c.kv_heads, a.R) &&
           c.page_size >= 8 && (c.page_size & (c.page_size - 1)) == 0 &&
           fits(c.token_stride, c.page_size) && fits(c.head_stride, c.kv_heads) &&
           fits(c.page_stride, c.num_pages) && fits(a.q_head_stride, a.q_heads) &&
           fits(a.q_token_stride, a.T);
}

cudaError_t launch_attention(const DeviceInfo& dev, const AttentionArgs& a, void* workspace,
                             uint32_t* status_word, cudaStream_t stream) {
    const KvCache& c = a.cache;
    const int D = c.head_dim;
    Problem p = {};
    p.D = D;
    p.T = a.T;
    p.q_heads = a.q_heads;
    p.kv_heads = c.kv_heads;
    p.g = a.q_heads / c.kv_heads;
    p.R = a.R;
    p.max_pages = a.max_pages;
    p.num_pages = c.num_pages;
    p.page_size = c.page_size;
    while ((1 << p.page_shift) < c.page_size) ++p.page_shift;
    p.left = a.window_left;
    p.right = a.window_right;
    // Beyond 2^64 a cap changes no score that fp32 tells from its neighbours, below 2^-64 it makes all
    // of them 0; between, nothing in the cap's arithmetic overflows.
    p.softcap = a.softcap > 0.f ? std::min(std::max(a.softcap, 0x1p-64f), 0x1p64f) : 0.f;
    p.scale = a.scale * c.k_scale;
    p.v_scale = c.v_scale;
    p.block_table = a.block_table;
    p.query_start = a.query_start;
    p.kv_lens = a.kv_lens;
    p.out = a.out;
    p.lse = a.lse;
    p.value = c.value;
    p.page_stride = c.page_stride;
    p.token_stride = c.token_stride;
    p.head_stride = c.head_stride;
    char* w = static_cast<char*>(workspace);
    p.bound = reinterpret_cast<int4*>(w);
    w += align256((size_t)(dev.sm_count + 1) * sizeof(int4));
    p.part = reinterpret_cast<float*>(w);
    p.G = std::min(dev.sm_count, kMaxRanges);
    // Two builds. Where a request has few rows of a key head on average, the one whose row tiles
    // have few rows and use all softmax warps (windowed, capped blocks of 32 rows: 199 us, 389 us
    // without; a longer request among them takes more items); the others are spared its code
    // (16001-token prompt: 806 us, 890 us with both).
    const bool few = p.g <= kFew && (long long)a.T * p.g <= (long long)kFew * a.R;
    p.tpt = (few ? kFew : BM) / p.g;
    p.tpi = few ? p.tpt : 2 * p.tpt;
    // What an item costs besides its steps, in steps: more where a step is short, which it is with few
    // rows and 32 KB or less of keys and values. Microseconds at 1 / 2 / 3: windowed blocks of
    // D = 64 233 / 215 / 203 (uncapped 209 / 195 / 184), single tokens from an 8-bit cache 191 / 176 /
    // 164 at D = 128, 147 / 137 / 129 at 64, windowed blocks over one 80 / 76 / 70; 16-bit single tokens
    // of D = 128 299 / 297 / 297, of D = 64 246 / 245 / 247, a 16001-token prompt 819 / 792 / 797.
    const long long step_bytes = 2LL * BN * D * (c.dtype == kE4m3 ? 1 : 2);
    p.over = few && step_bytes <= 32768 ? 3 : 2;
    // Nothing is cut, and no join is launched, where the table's width and the number of tokens alone
    // say that plan_ranges will take whole items (about 2 us of a short call).
    const long long steps = ((long long)a.max_pages * c.page_size + BN - 1) / BN;
    const long long per_request = ((long long)a.T + p.tpi - 1) / p.tpi;
    const long long items = (a.R + (long long)a.T / p.tpi) * c.kv_heads;
    // Single tokens of few requests gain from SMs that have no item of their own (a call in a graph, 8
    // items of 9 tiles: 14 us cut, 20 us whole; cold, 22 and 28, and 16 items of 8 tiles 24 and 26); 100
    // tokens over 400 are joined dearly (35 us, 26 us whole), and so are items that nearly fill the SMs
    // (128 items of 6 tiles: 33 us, 27 us whole; 144 of 11: 43 and 39).
    p.whole = few && 2 * items <= p.G ? 4 : 12;
    p.join = p.G > 1 && ((a.T > p.tpt && !few ? 2 : 1) * (p.over + steps) > p.over + p.whole ||
                         per_request > kSerialItems || items > p.G);
    return (c.dtype == kE4m3 ? launch_attention_e4m3 : launch_attention_16bit)(dev, a, p, few,
                                                                              status_word, stream);
}

}  // namespace dflash
