// The paged key-value cache held in 4 bits: its layout, and the parameters and
// launches of the kernels that build its tables, write it, read it and attend over it.
//
// cache: uint8 [pages][kv_heads][page_size / 16][16 * (D + 6)]. A tile of 16 tokens:
//   K codes  [16][D/2]               byte j of a token: d = 2j low nibble, 2j + 1 high nibble
//   V codes  [2][8][4][D/32][2] u16  word (h, n, c, w, e), nibble i: d = n*D/8 + 4w + i of
//                                    token 8h + 2c + e
//   K scales binary16 [16], V scales binary16 [16], K zero-points u8 [16], V zero-points u8 [16]
// A value is (code - zero) * scale. Why this layout:
//  - a tile is contiguous and a multiple of 16 bytes, so any run of tiles of a page is one
//    bulk copy, whatever the page size;
//  - a lane's share of a K fragment (one token, D/4 values of d) and of a V fragment (two
//    tokens, D/8 values of d) is one contiguous 8- or 16-byte word, and a warp's 32 shares
//    are contiguous: shared-memory loads without bank conflicts;
//  - the two 16-bit halves of a 32-bit word hold values that an MMA register pairs (two d of
//    one token for K, one d of two tokens for V), so `word & 0x000f000f` is a register of two
//    binary16 subnormals, code * 2^-24, and `word & 0x00f000f0` one of code * 2^-20: one
//    logic operation unpacks two codes, exactly.
#pragma once
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace w4a16 {

constexpr int kKv4Tile = 16;   // tokens per tile

__host__ __device__ constexpr int kv4_tile_bytes(int D) { return kKv4Tile * (D + 6); }
__host__ __device__ constexpr int kv4_v_off(int D) { return 8 * D; }
__host__ __device__ constexpr int kv4_k_scale_off(int D) { return 16 * D; }
__host__ __device__ constexpr int kv4_v_scale_off(int D) { return 16 * D + 32; }
__host__ __device__ constexpr int kv4_k_zero_off(int D) { return 16 * D + 64; }
__host__ __device__ constexpr int kv4_v_zero_off(int D) { return 16 * D + 80; }

struct Kv4TablesParams {
    const int32_t* seq_lens;     // [batch]
    const int32_t* new_lens;     // [batch]
    const int32_t* free_pages;   // [n_free]
    const int32_t* taken_in;     // or null: none taken
    int32_t* taken_out;
    int32_t* table;              // [batch][max_pages]
    int64_t* slots;              // [max_tokens]
    int32_t* positions;          // [max_tokens]
    int32_t* starts;             // [batch + 1]
    int batch, n_free, max_pages, page_size, max_tokens;
};
cudaError_t launch_kv4_tables(const Kv4TablesParams& p, cudaStream_t stream);

struct Kv4RowsParams {
    const void* k;               // append: [tokens][kv_heads][D] at the strides below
    const void* v;
    void* k_out;                 // read: [tokens][kv_heads][D], contiguous
    void* v_out;
    long long k_token, k_head, v_token, v_head;   // strides in elements
    const int64_t* slots;        // [tokens]
    uint8_t* cache;
    long long n_slots;           // pages * page_size
    int tokens, kv_heads, head_dim, page_size;
    int dtype;                   // w4a16_dtype
    uint32_t per_head;           // (2^32 - 1) / kv_heads
};
cudaError_t launch_kv4_append(const Kv4RowsParams& p, cudaStream_t stream);
cudaError_t launch_kv4_read(const Kv4RowsParams& p, cudaStream_t stream);

struct Kv4AttnParams {
    const void* q;               // [tokens][q_heads][D]
    void* out;                   // [tokens][q_heads][D]
    float* lse;                  // [tokens][q_heads] or null
    const uint8_t* cache;
    const int32_t* table;        // [batch][table_stride], table_cols valid
    const int32_t* seq_lens;     // [batch]
    const int32_t* starts;       // [batch + 1]
    long long q_token, q_head, o_token, o_head, table_stride;
    int* status;
    int* counters;
    float* partials;
    long long wait_limit_ns;
    float scale_log2;            // softmax scale * log2(e)
    int batch, tokens, q_heads, kv_heads, group, pages, page_size, table_cols, window;
    int few_rows;                // requests of at most this many rows a KV head are the stream-K kernel's
    int bf16;
    int splits;                  // CTAs that a pair of row tiles may have (tcgen05 kernel)
};
// path: 0 as measured, 1 the stream-K kernel, 2 the tcgen05 kernel for every request of more than 32 rows.
cudaError_t launch_kv4_attention(const Kv4AttnParams& p, int head_dim, int max_q, int path, int sms, cudaStream_t stream);
// The tcgen05 kernel, for requests of more than few_rows rows.
cudaError_t setup_kv4_prompt();
cudaError_t launch_kv4_prompt(const Kv4AttnParams& p, int head_dim, int sms, cudaStream_t stream);
size_t kv4_prompt_partial_bytes(int sms);
// Bytes of partial sums that launch_kv4_attention may use.
size_t kv4_partial_bytes(int sms);

}  // namespace w4a16
