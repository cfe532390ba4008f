// The paged key-value cache held in 8 bits: its layout, and the parameters and launches of the kernels that write it, read
// it and attend over it. Block tables and slots are those of the 4-bit cache.
//
// cache: uint8 [pages][kv_heads][page_size / 16][32 D + 16]. A tile of 16 tokens:
//   K codes  [D/64][16][64]              byte i of token t in slab p: d = 64p + i
//   V codes  [D/64][2][8][4][4][2][2]    byte (p, h, n, c, j, e, i): d = 64p + 8n + 2j + i of token 8h + 2c + e
//   K scale, V scale  float32, of all 16 tokens; 8 bytes unused
// A value is (code - 128) * scale. Why this layout: as in the 4-bit cache a tile is one bulk copy and the shares of an MMA's
// lanes (16 bytes of one token for K, of two tokens for V) lie one behind the other, without bank conflicts; bytes 0 and 2
// of a word (one prmt or logic operation apart from bytes 1 and 3) are a pair of an MMA's operand, two d of one token
// for K and one d of two tokens for V, as two binary16 subnormals code * 2^-24, exact.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "kv4.cuh"
#include "rope.cuh"

namespace w4a16 {

__host__ __device__ constexpr int kv8_tile_bytes(int D) { return 32 * D + 16; }
__host__ __device__ constexpr int kv8_v_off(int D) { return 16 * D; }
__host__ __device__ constexpr int kv8_k_scale_off(int D) { return 32 * D; }
__host__ __device__ constexpr int kv8_v_scale_off(int D) { return 32 * D + 4; }

struct Kv8RowsParams {
    const void* k;               // append: [tokens][kv_heads][D] at the strides below
    const void* v;
    void* k_out;                 // read: [tokens][kv_heads][D], contiguous
    void* v_out;
    long long k_token, k_head, v_token, v_head;   // strides in elements
    const int64_t* slots;        // [tokens]
    Rope rope;
    uint8_t* cache;
    long long n_slots;           // pages * page_size
    int tokens, kv_heads, head_dim, page_size;
    int dtype, mode;             // w4a16_dtype, RopeMode
    int window;                  // list places of a warp (set by the launch)
};
cudaError_t launch_kv8_append(const Kv8RowsParams& p, cudaStream_t stream);
cudaError_t launch_kv8_read(const Kv8RowsParams& p, cudaStream_t stream);

// path: 0 as measured, 1 the stream-K kernel, 2 the tcgen05 kernel for every request of more than 32 rows.
cudaError_t launch_kv8_attention(const Kv4AttnParams& p, int head_dim, int max_q, int path, int sms, cudaStream_t stream);
cudaError_t setup_kv8_attention();   // attributes of the attention kernels
// The tcgen05 kernel, for requests of more than few_rows rows.
cudaError_t setup_kv8_prompt();
cudaError_t launch_kv8_prompt(const Kv4AttnParams& p, int head_dim, int sms, cudaStream_t stream);
size_t kv8_prompt_partial_bytes(int sms);
// Bytes of partial sums that launch_kv8_attention may use.
size_t kv8_partial_bytes(int sms);

}  // namespace w4a16
