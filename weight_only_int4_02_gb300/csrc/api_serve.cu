// C ABI of the serving step's operators: argument checks and launches of the 4-bit
// key-value cache's calls and of sampling.
#include "api_internal.cuh"
#include "kv4.cuh"
#include "sample.cuh"
#include "w4a16.h"

#include <math.h>

#include <atomic>

namespace {

using namespace w4a16;

std::atomic<int> g_kv4_path{0};   // forced attention kernel, for tests and ablations

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

}  // namespace

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
    DeviceInfo dev;
    if (device_info(&dev) != W4A16_OK) return 0;
    return kWsPartialsOff + kv4_partial_bytes(dev.sms);
}

w4a16_status w4a16_kv4_attention(const void* q, int64_t q_token_stride, int64_t q_head_stride, const uint8_t* cache,
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
    if (ws_bytes < kWsPartialsOff + kv4_partial_bytes(dev.sms)) return W4A16_ERR_WORKSPACE;
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
    return report_cuda(launch_kv4_attention(p, head_dim, max_q, g_kv4_path.load(), dev.sms, stream));
}

int w4a16_kv4_force_path(int path)
{
    if (path < 0 || path > 2) return -1;
    return g_kv4_path.exchange(path);
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
