// C ABI of the serving step's operators: argument checks and launches of the norms and rotations,
// of the 4- and 8-bit key-value caches' calls and of sampling.
#include "api_internal.cuh"
#include "kv4.cuh"
#include "kv8.cuh"
#include "rope.cuh"
#include "sample.cuh"
#include "w4a16.h"

#include <math.h>
#include <stdint.h>

#include <atomic>

namespace {

using namespace w4a16;

std::atomic<int> g_kv4_path{0}, g_kv8_path{0};   // forced attention kernel, for tests and ablations

constexpr float kLog2E = 1.44269504088896340736f;

bool aligned(const void* p, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

bool valid_page(int page_size) { return page_size >= 16 && page_size <= 256 && (page_size & (page_size - 1)) == 0; }

bool valid_dim(int head_dim) { return head_dim == 64 || head_dim == 128; }

// The stride of `count` items (that of one item is never used).
bool valid_stride(int64_t stride, int head_dim, int count)
{
    return count <= 1 || (stride >= head_dim && stride % 8 == 0);
}

// The stride of rows that are only read: 0 where all of them are one row.
bool valid_row_stride(int64_t stride, int length) { return stride == 0 || stride >= length; }

// The arguments that append and read share.
bool valid_rows(const void* cache, int pages, const int64_t* slots, int tokens, int kv_heads, int head_dim,
                int page_size, int dtype, int dtypes)
{
    if (tokens < 0 || kv_heads <= 0 || pages < 0 || !valid_dim(head_dim) || !valid_page(page_size)) return false;
    if (dtype < 0 || dtype >= dtypes) return false;
    // the kernels count rows (K and V of a token and head) in 32 bits, a last block past them too
    if ((int64_t)tokens * kv_heads >= ((int64_t)1 << 31) - 256) return false;
    return tokens == 0 || (cache && slots && aligned(cache, 16) && aligned(slots, 8));
}

// A rotation's arguments; without a table there is none.
bool valid_rope(const int32_t* positions, const float* rope, int rows, int rot, int interleaved, int head_dim)
{
    if (!rope) return !positions;
    return positions && rows > 0 && rot > 0 && rot <= head_dim && rot % 8 == 0 && (interleaved == 0 || interleaved == 1) &&
           aligned(positions, 4) && aligned(rope, 16);
}

int rope_mode(const float* rope, int interleaved) { return !rope ? kRopeNone : interleaved ? kRopePairs : kRopeHalves; }

// Attention over a cache of either kind.
struct CacheKind {
    size_t (*partial_bytes)(int sms);
    cudaError_t (*launch)(const Kv4AttnParams& p, int head_dim, int max_q, int path, int sms, cudaStream_t stream);
    std::atomic<int>* path;
};
const CacheKind kFourBits{kv4_partial_bytes, launch_kv4_attention, &g_kv4_path};
const CacheKind kEightBits{kv8_partial_bytes, launch_kv8_attention, &g_kv8_path};

size_t attention_workspace(const CacheKind& kind)
{
    DeviceInfo dev;
    if (device_info(&dev) != W4A16_OK) return 0;
    return kWsPartialsOff + kind.partial_bytes(dev.sms);
}

w4a16_status attention(const CacheKind& kind, const void* q, int64_t q_token_stride, int64_t q_head_stride, const uint8_t* cache,
                       int pages, const int32_t* block_table, int64_t table_stride, int table_cols,
                       const int32_t* seq_lens, const int32_t* starts, void* out, int64_t out_token_stride,
                       int64_t out_head_stride, float* lse, int batch, int tokens, int q_heads, int kv_heads,
                       int head_dim, int page_size, int max_q, float scale, int window, int dtype,
                       void* workspace, size_t ws_bytes, w4a16_stream_t stream)
{
    if (batch < 0 || tokens < 0 || q_heads <= 0 || kv_heads <= 0 || q_heads % kv_heads != 0 || pages < 0 || max_q < 0 ||
        table_cols < 0 || window < 0 || !valid_dim(head_dim) || !valid_page(page_size))
        return W4A16_ERR_INVALID_ARG;
    if ((dtype != W4A16_FP16 && dtype != W4A16_BF16) || !(fabsf(scale) <= 3.0e38f)) return W4A16_ERR_INVALID_ARG;
    // rows (query token, head) and tiles of them are counted in 31 bits
    if ((int64_t)tokens * q_heads + (int64_t)batch * kv_heads >= ((int64_t)1 << 31)) return W4A16_ERR_INVALID_ARG;
    if (batch == 0 || tokens == 0) return W4A16_OK;
    if (!q || !out || !seq_lens || !starts || (pages > 0 && !cache) || (table_cols > 0 && !block_table))
        return W4A16_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(cache, 16) || !aligned(block_table, 4) || !aligned(seq_lens, 4) ||
        !aligned(starts, 4) || !aligned(lse, 4))
        return W4A16_ERR_INVALID_ARG;
    if (!valid_stride(q_token_stride, head_dim, tokens) || !valid_stride(q_head_stride, head_dim, q_heads) ||
        !valid_stride(out_token_stride, head_dim, tokens) || !valid_stride(out_head_stride, head_dim, q_heads) ||
        (batch > 1 && !valid_row_stride(table_stride, table_cols)))
        return W4A16_ERR_INVALID_ARG;
    if (workspace && !aligned(workspace, 256)) return W4A16_ERR_INVALID_ARG;
    DeviceInfo dev;
    w4a16_status rc = device_info(&dev);
    if (rc != W4A16_OK) return rc;
    if (!workspace) {
        rc = library_workspace(&workspace, &ws_bytes);
        if (rc != W4A16_OK) return rc;
    }
    if (ws_bytes < kWsPartialsOff + kind.partial_bytes(dev.sms)) return W4A16_ERR_WORKSPACE;
    char* ws = static_cast<char*>(workspace);
    Kv4AttnParams p = {};
    p.q = q;
    p.out = out;
    p.lse = lse;
    p.cache = cache;
    p.table = block_table;
    p.seq_lens = seq_lens;
    p.starts = starts;
    p.q_token = q_token_stride;
    p.q_head = q_head_stride;
    p.o_token = out_token_stride;
    p.o_head = out_head_stride;
    p.table_stride = table_stride;
    p.status = reinterpret_cast<int*>(ws);
    p.counters = reinterpret_cast<int*>(ws + kWsCountersOff);
    p.partials = reinterpret_cast<float*>(ws + kWsPartialsOff);
    p.wait_limit_ns = dev.wait_limit_ns;
    p.scale_log2 = scale * kLog2E;
    p.batch = batch;
    p.tokens = tokens;
    p.q_heads = q_heads;
    p.kv_heads = kv_heads;
    p.group = q_heads / kv_heads;
    p.pages = pages;
    p.page_size = page_size;
    p.table_cols = table_cols;
    p.window = window;
    p.bf16 = dtype == W4A16_BF16;
    return report_cuda(kind.launch(p, head_dim, max_q, kind.path->load(), dev.sms, stream));
}

}  // namespace

namespace w4a16 {

cudaError_t setup_kv4()
{
    const cudaError_t e = setup_kv4_attention();
    return e != cudaSuccess ? e : setup_kv8_attention();
}

}  // namespace w4a16

extern "C" {

size_t w4a16_kv4_page_bytes(int kv_heads, int head_dim, int page_size)
{
    if (kv_heads <= 0 || !valid_dim(head_dim) || !valid_page(page_size)) return 0;
    return (size_t)kv_heads * page_size * (head_dim + 6);
}

w4a16_status w4a16_kv4_tables(const int32_t* seq_lens, const int32_t* new_lens, int batch, const int32_t* free_pages,
                              int n_free, const int32_t* taken_in, int32_t* taken_out, int32_t* block_table,
                              int max_pages, int page_size, int64_t* slots, int32_t* positions, int max_tokens,
                              int32_t* starts, w4a16_stream_t stream)
{
    if (batch < 0 || n_free < 0 || max_pages <= 0 || max_tokens < 0 || !valid_page(page_size)) return W4A16_ERR_INVALID_ARG;
    if (!taken_out || !starts || taken_in == taken_out) return W4A16_ERR_INVALID_ARG;
    if (batch > 0 && (!seq_lens || !new_lens || !block_table)) return W4A16_ERR_INVALID_ARG;
    if ((n_free > 0 && !free_pages) || (max_tokens > 0 && (!slots || !positions))) return W4A16_ERR_INVALID_ARG;
    if (!aligned(seq_lens, 4) || !aligned(new_lens, 4) || !aligned(free_pages, 4) || !aligned(taken_in, 4) ||
        !aligned(taken_out, 4) || !aligned(block_table, 4) || !aligned(positions, 4) || !aligned(starts, 4) ||
        !aligned(slots, 8))
        return W4A16_ERR_INVALID_ARG;
    DeviceInfo dev;
    const w4a16_status rc = device_info(&dev);
    if (rc != W4A16_OK) return rc;
    const Kv4TablesParams p{seq_lens, new_lens, free_pages, taken_in, taken_out, block_table, slots,
                            positions, starts, batch, n_free, max_pages, page_size, max_tokens};
    return report_cuda(launch_kv4_tables(p, stream));
}

w4a16_status w4a16_kv4_append(const void* k, int64_t k_token_stride, int64_t k_head_stride, const void* v,
                              int64_t v_token_stride, int64_t v_head_stride, const int64_t* slots, uint8_t* cache,
                              int pages, int tokens, int kv_heads, int head_dim, int page_size, int dtype,
                              w4a16_stream_t stream)
{
    if (!valid_rows(cache, pages, slots, tokens, kv_heads, head_dim, page_size, dtype, W4A16_FP32))
        return W4A16_ERR_INVALID_ARG;
    if (tokens == 0) return W4A16_OK;
    if (!k || !v || !aligned(k, 16) || !aligned(v, 16)) return W4A16_ERR_INVALID_ARG;
    if (!valid_stride(k_token_stride, head_dim, tokens) || !valid_stride(k_head_stride, head_dim, kv_heads) ||
        !valid_stride(v_token_stride, head_dim, tokens) || !valid_stride(v_head_stride, head_dim, kv_heads))
        return W4A16_ERR_INVALID_ARG;
    DeviceInfo dev;
    const w4a16_status rc = device_info(&dev);
    if (rc != W4A16_OK) return rc;
    Kv4RowsParams p = {};
    p.k = k;
    p.v = v;
    p.k_token = k_token_stride;
    p.k_head = k_head_stride;
    p.v_token = v_token_stride;
    p.v_head = v_head_stride;
    p.slots = slots;
    p.cache = cache;
    p.n_slots = (long long)pages * page_size;
    p.tokens = tokens;
    p.kv_heads = kv_heads;
    p.head_dim = head_dim;
    p.page_size = page_size;
    p.dtype = dtype;
    p.per_head = 0xffffffffu / (uint32_t)kv_heads;
    return report_cuda(launch_kv4_append(p, stream));
}

w4a16_status w4a16_kv4_read(const uint8_t* cache, int pages, const int64_t* slots, void* k, void* v, int tokens,
                            int kv_heads, int head_dim, int page_size, int dtype, w4a16_stream_t stream)
{
    if (!valid_rows(cache, pages, slots, tokens, kv_heads, head_dim, page_size, dtype, W4A16_FP32 + 1))
        return W4A16_ERR_INVALID_ARG;
    if (tokens == 0) return W4A16_OK;
    if (!k || !v || !aligned(k, 16) || !aligned(v, 16)) return W4A16_ERR_INVALID_ARG;
    DeviceInfo dev;
    const w4a16_status rc = device_info(&dev);
    if (rc != W4A16_OK) return rc;
    Kv4RowsParams p = {};
    p.k_out = k;
    p.v_out = v;
    p.slots = slots;
    p.cache = const_cast<uint8_t*>(cache);
    p.n_slots = (long long)pages * page_size;
    p.tokens = tokens;
    p.kv_heads = kv_heads;
    p.head_dim = head_dim;
    p.page_size = page_size;
    p.dtype = dtype;
    p.per_head = 0xffffffffu / (uint32_t)kv_heads;
    return report_cuda(launch_kv4_read(p, stream));
}

size_t w4a16_kv4_workspace_bytes(void)
{
    return attention_workspace(kFourBits);
}

w4a16_status w4a16_kv4_attention(const void* q, int64_t q_token_stride, int64_t q_head_stride, const uint8_t* cache,
                                 int pages, const int32_t* block_table, int64_t table_stride, int table_cols,
                                 const int32_t* seq_lens, const int32_t* starts, void* out, int64_t out_token_stride,
                                 int64_t out_head_stride, float* lse, int batch, int tokens, int q_heads, int kv_heads,
                                 int head_dim, int page_size, int max_q, float scale, int window, int dtype,
                                 void* workspace, size_t ws_bytes, w4a16_stream_t stream)
{
    return attention(kFourBits, q, q_token_stride, q_head_stride, cache, pages, block_table, table_stride, table_cols, seq_lens,
                     starts, out, out_token_stride, out_head_stride, lse, batch, tokens, q_heads, kv_heads, head_dim, page_size,
                     max_q, scale, window, dtype, workspace, ws_bytes, stream);
}

int w4a16_kv4_force_path(int path)
{
    if (path < 0 || path > 2) return -1;
    return g_kv4_path.exchange(path);
}

w4a16_status w4a16_rope_table(float* table, int rows, int rot, double base, w4a16_stream_t stream)
{
    if (rows < 0 || rot <= 0 || rot % 8 != 0 || rot > 65536 || !(base > 0.0) || !(base <= 1.0e300)) return W4A16_ERR_INVALID_ARG;
    if (rows == 0) return W4A16_OK;
    if (!table || !aligned(table, 16)) return W4A16_ERR_INVALID_ARG;
    DeviceInfo dev;
    const w4a16_status rc = device_info(&dev);
    if (rc != W4A16_OK) return rc;
    return report_cuda(launch_rope_table(table, rows, rot, base, stream));
}

w4a16_status w4a16_qk_norm_rope(const void* q, int64_t q_token_stride, int64_t q_head_stride, void* q_out,
                                int64_t q_out_token_stride, int64_t q_out_head_stride, const void* k, int64_t k_token_stride,
                                int64_t k_head_stride, void* k_out, int64_t k_out_token_stride, int64_t k_out_head_stride,
                                const void* q_weight, const void* k_weight, float eps, const int32_t* positions,
                                const float* rope, int rope_rows, int rot, int interleaved, int tokens, int q_heads,
                                int kv_heads, int head_dim, int dtype, w4a16_stream_t stream)
{
    if (tokens < 0 || q_heads < 0 || kv_heads < 0 || !valid_dim(head_dim) || (dtype != W4A16_FP16 && dtype != W4A16_BF16) ||
        !(eps >= 0.0f) || !(eps <= 3.0e38f) || !valid_rope(positions, rope, rope_rows, rot, interleaved, head_dim))
        return W4A16_ERR_INVALID_ARG;
    const int64_t heads = (int64_t)q_heads + kv_heads;
    // warps of eight rows of queries or of keys, and more, counted in 31 bits, as is the head behind a warp's last pass
    if (heads > INT32_MAX - 256 || (int64_t)tokens * (((int64_t)q_heads + 7) / 8 + ((int64_t)kv_heads + 7) / 8) >= ((int64_t)1 << 31) - 8)
        return W4A16_ERR_INVALID_ARG;
    if (tokens == 0 || heads == 0) return W4A16_OK;
    NormRopeParams p = {};
    const void* x[2] = {q, k};
    void* out[2] = {q_out, k_out};
    const void* weight[2] = {q_weight, k_weight};
    const int64_t strides[2][4] = {{q_token_stride, q_head_stride, q_out_token_stride, q_out_head_stride},
                                   {k_token_stride, k_head_stride, k_out_token_stride, k_out_head_stride}};
    const int counts[2] = {q_heads, kv_heads};
    for (int i = 0; i < 2; ++i) {
        if (counts[i] > 0 && (!x[i] || !out[i] || !aligned(x[i], 16) || !aligned(out[i], 16) || !aligned(weight[i], 16) ||
                              !valid_stride(strides[i][0], head_dim, tokens) || !valid_stride(strides[i][1], head_dim, counts[i]) ||
                              !valid_stride(strides[i][2], head_dim, tokens) || !valid_stride(strides[i][3], head_dim, counts[i])))
            return W4A16_ERR_INVALID_ARG;
        p.x[i] = x[i];
        p.out[i] = out[i];
        p.weight[i] = counts[i] > 0 ? weight[i] : nullptr;
        p.token[i] = strides[i][0];
        p.head[i] = strides[i][1];
        p.out_token[i] = strides[i][2];
        p.out_head[i] = strides[i][3];
        p.heads[i] = counts[i];
    }
    DeviceInfo dev;
    const w4a16_status rc = device_info(&dev);
    if (rc != W4A16_OK) return rc;
    p.rope = Rope{positions, rope, rope_rows, rope ? rot : 0};
    p.eps = eps;
    p.tokens = tokens;
    p.head_dim = head_dim;
    p.dtype = dtype;
    p.mode = rope_mode(rope, interleaved);
    return report_cuda(launch_norm_rope(p, dev.sms, stream));
}

size_t w4a16_kv8_page_bytes(int kv_heads, int head_dim, int page_size)
{
    if (kv_heads <= 0 || !valid_dim(head_dim) || !valid_page(page_size)) return 0;
    return (size_t)kv_heads * (page_size / 16) * kv8_tile_bytes(head_dim);
}

w4a16_status w4a16_kv8_append(const void* k, int64_t k_token_stride, int64_t k_head_stride, const void* v,
                              int64_t v_token_stride, int64_t v_head_stride, const int64_t* slots,
                              const int32_t* positions, const float* rope, int rope_rows, int rot, int interleaved,
                              uint8_t* cache, int pages, int tokens, int kv_heads, int head_dim, int page_size, int dtype,
                              w4a16_stream_t stream)
{
    if (!valid_rows(cache, pages, slots, tokens, kv_heads, head_dim, page_size, dtype, W4A16_FP32) ||
        !valid_rope(positions, rope, rope_rows, rot, interleaved, head_dim))
        return W4A16_ERR_INVALID_ARG;
    if (kv_heads > 1 << 29) return W4A16_ERR_INVALID_ARG;   // CTAs are counted in 31 bits, two and more for each head
    if (tokens == 0) return W4A16_OK;
    if (!k || !v || !aligned(k, 16) || !aligned(v, 16)) return W4A16_ERR_INVALID_ARG;
    if (!valid_stride(k_token_stride, head_dim, tokens) || !valid_stride(k_head_stride, head_dim, kv_heads) ||
        !valid_stride(v_token_stride, head_dim, tokens) || !valid_stride(v_head_stride, head_dim, kv_heads))
        return W4A16_ERR_INVALID_ARG;
    DeviceInfo dev;
    const w4a16_status rc = device_info(&dev);
    if (rc != W4A16_OK) return rc;
    Kv8RowsParams p = {};
    p.k = k;
    p.v = v;
    p.k_token = k_token_stride;
    p.k_head = k_head_stride;
    p.v_token = v_token_stride;
    p.v_head = v_head_stride;
    p.slots = slots;
    p.rope = Rope{positions, rope, rope_rows, rope ? rot : 0};
    p.cache = cache;
    p.n_slots = (long long)pages * page_size;
    p.tokens = tokens;
    p.kv_heads = kv_heads;
    p.head_dim = head_dim;
    p.page_size = page_size;
    p.dtype = dtype;
    p.mode = rope_mode(rope, interleaved);
    return report_cuda(launch_kv8_append(p, stream));
}

w4a16_status w4a16_kv8_read(const uint8_t* cache, int pages, const int64_t* slots, void* k, void* v, int tokens,
                            int kv_heads, int head_dim, int page_size, int dtype, w4a16_stream_t stream)
{
    if (!valid_rows(cache, pages, slots, tokens, kv_heads, head_dim, page_size, dtype, W4A16_FP32 + 1))
        return W4A16_ERR_INVALID_ARG;
    if (tokens == 0) return W4A16_OK;
    if (!k || !v || !aligned(k, 16) || !aligned(v, 16)) return W4A16_ERR_INVALID_ARG;
    DeviceInfo dev;
    const w4a16_status rc = device_info(&dev);
    if (rc != W4A16_OK) return rc;
    Kv8RowsParams p = {};
    p.k_out = k;
    p.v_out = v;
    p.slots = slots;
    p.cache = const_cast<uint8_t*>(cache);
    p.n_slots = (long long)pages * page_size;
    p.tokens = tokens;
    p.kv_heads = kv_heads;
    p.head_dim = head_dim;
    p.page_size = page_size;
    p.dtype = dtype;
    return report_cuda(launch_kv8_read(p, stream));
}

size_t w4a16_kv8_workspace_bytes(void)
{
    return attention_workspace(kEightBits);
}

w4a16_status w4a16_kv8_attention(const void* q, int64_t q_token_stride, int64_t q_head_stride, const uint8_t* cache,
                                 int pages, const int32_t* block_table, int64_t table_stride, int table_cols,
                                 const int32_t* seq_lens, const int32_t* starts, void* out, int64_t out_token_stride,
                                 int64_t out_head_stride, float* lse, int batch, int tokens, int q_heads, int kv_heads,
                                 int head_dim, int page_size, int max_q, float scale, int window, int dtype,
                                 void* workspace, size_t ws_bytes, w4a16_stream_t stream)
{
    return attention(kEightBits, q, q_token_stride, q_head_stride, cache, pages, block_table, table_stride, table_cols, seq_lens,
                     starts, out, out_token_stride, out_head_stride, lse, batch, tokens, q_heads, kv_heads, head_dim, page_size,
                     max_q, scale, window, dtype, workspace, ws_bytes, stream);
}

int w4a16_kv8_force_path(int path)
{
    if (path < 0 || path > 2) return -1;
    return g_kv8_path.exchange(path);
}

w4a16_status w4a16_sample(const void* logits, int64_t row_stride, const float* u, const float* temperature,
                          const int32_t* top_k, const float* top_p, const float* min_p, int32_t* token, float* prob,
                          int batch, int vocab, int dtype, w4a16_stream_t stream)
{
    if (batch < 0 || vocab <= 0 || vocab > kSampleMaxVocab || dtype < 0 || dtype > W4A16_FP32) return W4A16_ERR_INVALID_ARG;
    if (batch > (1 << 27)) return W4A16_ERR_INVALID_ARG;   // CTAs are counted in 31 bits, up to eight a row
    if (batch == 0) return W4A16_OK;
    if (!logits || !u || !token || !valid_row_stride(row_stride, vocab)) return W4A16_ERR_INVALID_ARG;
    if (!aligned(logits, dtype == W4A16_FP32 ? 4 : 2) || !aligned(u, 4) || !aligned(temperature, 4) || !aligned(top_k, 4) ||
        !aligned(top_p, 4) || !aligned(min_p, 4) || !aligned(token, 4) || !aligned(prob, 4))
        return W4A16_ERR_INVALID_ARG;
    DeviceInfo dev;
    const w4a16_status rc = device_info(&dev);
    if (rc != W4A16_OK) return rc;
    SampleParams p = {};
    p.logits = logits;
    p.stride = row_stride;
    p.u = u;
    p.temperature = temperature;
    p.top_k = top_k;
    p.top_p = top_p;
    p.min_p = min_p;
    p.token = token;
    p.prob = prob;
    p.batch = batch;
    p.vocab = vocab;
    p.dtype = dtype;
    return report_cuda(launch_sample(p, dev.sms, stream));
}

}  // extern "C"
