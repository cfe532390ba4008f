// The 4-bit cache's bookkeeping and rows: block tables and slot maps from request
// lengths, quantisation of new keys and values into their slots, and the read back.
#include <cuda_bf16.h>

#include "kv4.cuh"
#include "w4a16.h"

namespace w4a16 {
namespace {

// ---------------------------------------------------------------- tables
// Request b holds old = ceil((seq - new) / P) pages and needs want = ceil(seq / P), both at
// most max_pages; its want - old fresh pages come from the free list behind those of the
// requests before it. Two prefix sums over the requests (new tokens, fresh pages) fix
// everything, so one launch does it all: a CTA owns a run of requests, sums over the
// requests before it by itself (8 bytes a request out of L2), and its warps write their
// requests' table rows, slots and positions with no word between CTAs. Bound by
// latency: the launch, two dependent reads and the stores. A warp per request, so that
// a thousand requests fill the GPU and a chunk of 512 tokens is 16 steps of its warp.
constexpr int kTabWarps = 8;

struct Need {
    int fresh, tokens;
};

__device__ __forceinline__ int pages_of(int tokens, const Kv4TablesParams& p)
{
    const int n = tokens <= 0 ? 0 : (tokens - 1) / p.page_size + 1;
    return n < p.max_pages ? n : p.max_pages;
}

__device__ __forceinline__ Need need_of(int seq, int fresh_tokens, const Kv4TablesParams& p)
{
    const int n = fresh_tokens > 0 ? fresh_tokens : 0;
    const int pages = pages_of(seq, p) - pages_of(seq - n, p);
    return {pages > 0 ? pages : 0, n};
}

__global__ void __launch_bounds__(kTabWarps * 32) kv4_tables_kernel(const Kv4TablesParams p)
{
    __shared__ int part[2][kTabWarps], own[2][kTabWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int b0 = blockIdx.x * kTabWarps, b = b0 + warp;
    int seq = 0, fresh_tokens = 0;
    if (b < p.batch) {
        seq = p.seq_lens[b];
        fresh_tokens = p.new_lens[b];
    }
    const int taken = p.taken_in ? *p.taken_in : 0;
    int f = 0, t = 0;
    for (int i = threadIdx.x; i < b0; i += kTabWarps * 32) {
        const Need n = need_of(p.seq_lens[i], p.new_lens[i], p);
        f += n.fresh;
        t += n.tokens;
    }
    f = __reduce_add_sync(0xffffffffu, f);
    t = __reduce_add_sync(0xffffffffu, t);
    const Need mine = need_of(seq, fresh_tokens, p);
    if (lane == 0) {
        part[0][warp] = f;
        part[1][warp] = t;
        own[0][warp] = mine.fresh;
        own[1][warp] = mine.tokens;
    }
    __syncthreads();
    int page0 = taken, start = 0, all_pages = taken, all_tokens = 0;
#pragma unroll
    for (int i = 0; i < kTabWarps; ++i) {
        const int a = part[0][i] + own[0][i], c = part[1][i] + own[1][i];
        all_pages += a;
        all_tokens += c;
        page0 += i < warp ? a : part[0][i];
        start += i < warp ? c : part[1][i];
    }
    const bool last = b0 + kTabWarps >= p.batch;
    if (last) {
        // places past the batch's tokens
        for (int i = all_tokens + threadIdx.x; i < p.max_tokens; i += kTabWarps * 32) {
            p.slots[i] = -1;
            p.positions[i] = -1;
        }
        if (threadIdx.x == 0) {
            p.starts[p.batch] = all_tokens;
            *p.taken_out = all_pages;
        }
    }
    if (b >= p.batch) return;
    if (lane == 0) p.starts[b] = start;
    const int old = pages_of(seq - mine.tokens, p), want = pages_of(seq, p);
    int32_t* row = p.table + (long long)b * p.max_pages;
    auto fresh_page = [&](int col) {
        const long long at = (long long)page0 + (col - old);
        return at >= 0 && at < p.n_free ? p.free_pages[at] : -1;
    };
    int col = old + lane;
    for (; col < want; col += 32) row[col] = fresh_page(col);
    // columns past the request's pages: 16-byte stores once aligned
    const int from = old > want ? old : want;
    const int head = from + (int)(((16 - (reinterpret_cast<uintptr_t>(row + from) & 15)) & 15) >> 2);
    if (from + lane < head && from + lane < p.max_pages) row[from + lane] = -1;
    int c4 = head + 4 * lane;
    for (; c4 + 3 < p.max_pages; c4 += 128) *reinterpret_cast<int4*>(row + c4) = make_int4(-1, -1, -1, -1);
    for (; c4 < p.max_pages; ++c4) row[c4] = -1;
    for (int i = lane; i < mine.tokens; i += 32) {
        const long long at = (long long)start + i;
        if (at >= p.max_tokens) break;
        const int pos = seq - mine.tokens + i;
        long long slot = -1;
        if (pos >= 0) {
            const int c = pos / p.page_size;
            int page = -1;
            if (c < p.max_pages) page = c >= old ? fresh_page(c) : row[c];
            if (page >= 0) slot = (long long)page * p.page_size + (pos - c * p.page_size);
        }
        p.slots[at] = slot;
        p.positions[at] = pos;
    }
}

// ---------------------------------------------------------------- rows
template <int DTYPE>
__device__ __forceinline__ void unpack2(uint32_t w, float& a, float& b)
{
    if constexpr (DTYPE == W4A16_BF16) {
        a = __uint_as_float(w << 16);
        b = __uint_as_float(w & 0xffff0000u);
    } else {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
        a = f.x;
        b = f.y;
    }
}

template <int DTYPE>
__device__ __forceinline__ uint32_t pack2(float a, float b)
{
    if constexpr (DTYPE == W4A16_BF16) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    } else {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
}

// Address of the tile that holds a slot, and the slot's token in it; null for a slot outside the cache.
__device__ __forceinline__ uint8_t* tile_of(const Kv4RowsParams& p, int token, int head, int D, int* tok)
{
    const long long slot = p.slots[token];
    if (slot < 0 || slot >= p.n_slots) return nullptr;
    const long long page = slot / p.page_size;
    const int in_page = (int)(slot - page * p.page_size);
    *tok = in_page & 15;
    return p.cache + ((page * p.kv_heads + head) * (p.page_size >> 4) + (in_page >> 4)) * (long long)kv4_tile_bytes(D);
}

// One row (token, KV head, K or V) per group of D/8 lanes, eight values a lane: the row's
// extremes by shuffles, then
//   s = fp16(min((hi - lo) / 15, 65504)), z = clamp(rint(-lo / s), 0, 15),
//   code = clamp(rint(x / s) + z, 0, 15)        (lo = min(x, 0), hi = max(x, 0))
// with 1 / s rounded once to FP32; every operation is an IEEE one (no contraction, no
// approximate division), so the codes are the same wherever the formula is evaluated. A row
// that holds an infinity or a NaN gets scale NaN, so that it shows in whatever reads it.
// Reads 4 D bytes a token and head and writes D + 6: bound by bandwidth for a prompt,
// by latency for a decode step.
template <int D, int DTYPE>
__global__ void __launch_bounds__(256) kv4_append_kernel(const Kv4RowsParams p)
{
    constexpr int L = D / 8;   // lanes per row
    const long long rows = (long long)p.tokens * p.kv_heads * 2;
    const long long row = (long long)blockIdx.x * (256 / L) + threadIdx.x / L;
    const int j = threadIdx.x % L;
    const bool live = row < rows;
    int token = 0, head = 0, tok = 0;
    bool is_v = false;
    uint8_t* tile = nullptr;
    uint4 raw = make_uint4(0, 0, 0, 0);
    if (live) {
        // K rows of a token, then its V rows
        token = (int)(row / (2 * p.kv_heads));
        const int r = (int)(row - (long long)token * 2 * p.kv_heads);
        is_v = r >= p.kv_heads;
        head = is_v ? r - p.kv_heads : r;
        const uint16_t* src = is_v ? (const uint16_t*)p.v + token * p.v_token + head * p.v_head
                                   : (const uint16_t*)p.k + token * p.k_token + head * p.k_head;
        raw = *reinterpret_cast<const uint4*>(src + 8 * j);
        tile = tile_of(p, token, head, D, &tok);
    }
    float x[8];
    unpack2<DTYPE>(raw.x, x[0], x[1]);
    unpack2<DTYPE>(raw.y, x[2], x[3]);
    unpack2<DTYPE>(raw.z, x[4], x[5]);
    unpack2<DTYPE>(raw.w, x[6], x[7]);
    float lo = 0.0f, hi = 0.0f;
    bool fine = true;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        lo = fminf(lo, x[i]);
        hi = fmaxf(hi, x[i]);
        fine = fine && isfinite(x[i]);
    }
    int odd = fine ? 0 : 1;
#pragma unroll
    for (int d = L / 2; d > 0; d >>= 1) {
        lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, d));
        hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, d));
        odd |= __shfl_xor_sync(0xffffffffu, odd, d);
    }
    if (tile == nullptr) return;
    const __half s = odd ? __ushort_as_half(0x7fff)
                         : __float2half_rn(fminf(__fdiv_rn(__fsub_rn(hi, lo), 15.0f), 65504.0f));
    const float sf = __half2float(s);
    const float inv = !odd && sf > 0.0f ? __frcp_rn(sf) : 0.0f;
    const float z = odd ? 0.0f : fminf(rintf(__fmul_rn(-lo, inv)), 15.0f);
    uint32_t code[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float c = odd ? 0.0f : fminf(fmaxf(rintf(__fmul_rn(x[i], inv)) + z, 0.0f), 15.0f);
        code[i] = (uint32_t)c;
    }
    const uint32_t w0 = code[0] | code[1] << 4 | code[2] << 8 | code[3] << 12;
    const uint32_t w1 = code[4] | code[5] << 4 | code[6] << 8 | code[7] << 12;
    if (is_v) {
        // d = 8j .. 8j+7 of token 8h + 2c + e: two 16-bit words
        constexpr int PER = D / 8;   // d per n
        const int n = 8 * j / PER, w = (8 * j % PER) / 4;
        const int h = tok >> 3, c = (tok & 7) >> 1, e = tok & 1;
        uint16_t* dst = reinterpret_cast<uint16_t*>(tile + kv4_v_off(D)) + ((((h * 8 + n) * 4 + c) * (D / 32) + w) * 2 + e);
        dst[0] = (uint16_t)w0;
        dst[2] = (uint16_t)w1;
    } else {
        *reinterpret_cast<uint32_t*>(tile + tok * (D / 2) + 4 * j) = w0 | w1 << 16;
    }
    if (j == 0) {
        *reinterpret_cast<__half*>(tile + (is_v ? kv4_v_scale_off(D) : kv4_k_scale_off(D)) + 2 * tok) = s;
        tile[(is_v ? kv4_v_zero_off(D) : kv4_k_zero_off(D)) + tok] = (uint8_t)z;
    }
}

// The values that slots stand for, (code - zero) * scale in FP32, rounded once. Lanes as above.
template <int D, int DTYPE>
__global__ void __launch_bounds__(256) kv4_read_kernel(const Kv4RowsParams p)
{
    constexpr int L = D / 8;
    const long long rows = (long long)p.tokens * p.kv_heads * 2;
    const long long row = (long long)blockIdx.x * (256 / L) + threadIdx.x / L;
    const int j = threadIdx.x % L;
    if (row >= rows) return;
    const int token = (int)(row / (2 * p.kv_heads));
    const int r = (int)(row - (long long)token * 2 * p.kv_heads);
    const bool is_v = r >= p.kv_heads;
    const int head = is_v ? r - p.kv_heads : r;
    int tok = 0;
    const uint8_t* tile = tile_of(p, token, head, D, &tok);
    uint32_t w = 0;
    float s = 0.0f, z = 0.0f;
    if (tile) {
        if (is_v) {
            constexpr int PER = D / 8;
            const int n = 8 * j / PER, wi = (8 * j % PER) / 4;
            const int h = tok >> 3, c = (tok & 7) >> 1, e = tok & 1;
            const uint16_t* src = reinterpret_cast<const uint16_t*>(tile + kv4_v_off(D)) +
                                  ((((h * 8 + n) * 4 + c) * (D / 32) + wi) * 2 + e);
            w = src[0] | (uint32_t)src[2] << 16;
        } else {
            w = *reinterpret_cast<const uint32_t*>(tile + tok * (D / 2) + 4 * j);
        }
        s = __half2float(*reinterpret_cast<const __half*>(tile + (is_v ? kv4_v_scale_off(D) : kv4_k_scale_off(D)) + 2 * tok));
        z = (float)tile[(is_v ? kv4_v_zero_off(D) : kv4_k_zero_off(D)) + tok];
    }
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = ((float)((w >> (4 * i)) & 15u) - z) * s;
    const long long at = ((long long)token * p.kv_heads + head) * D + 8 * j;
    if constexpr (DTYPE == W4A16_FP32) {
        float4* dst = reinterpret_cast<float4*>((float*)(is_v ? p.v_out : p.k_out) + at);
        dst[0] = make_float4(x[0], x[1], x[2], x[3]);
        dst[1] = make_float4(x[4], x[5], x[6], x[7]);
    } else {
        *reinterpret_cast<uint4*>((uint16_t*)(is_v ? p.v_out : p.k_out) + at) =
            make_uint4(pack2<DTYPE>(x[0], x[1]), pack2<DTYPE>(x[2], x[3]), pack2<DTYPE>(x[4], x[5]),
                       pack2<DTYPE>(x[6], x[7]));
    }
}

unsigned row_blocks(const Kv4RowsParams& p)
{
    const long long per = 256 / (p.head_dim / 8);
    return (unsigned)(((long long)p.tokens * p.kv_heads * 2 + per - 1) / per);
}

}  // namespace

cudaError_t launch_kv4_tables(const Kv4TablesParams& p, cudaStream_t stream)
{
    const unsigned blocks = p.batch > 0 ? (unsigned)((p.batch - 1) / kTabWarps + 1) : 1u;   // an empty batch still has ends to write
    kv4_tables_kernel<<<blocks, kTabWarps * 32, 0, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_kv4_append(const Kv4RowsParams& p, cudaStream_t stream)
{
    const unsigned g = row_blocks(p);
    if (p.head_dim == 128) {
        if (p.dtype == W4A16_BF16) kv4_append_kernel<128, W4A16_BF16><<<g, 256, 0, stream>>>(p);
        else kv4_append_kernel<128, W4A16_FP16><<<g, 256, 0, stream>>>(p);
    } else {
        if (p.dtype == W4A16_BF16) kv4_append_kernel<64, W4A16_BF16><<<g, 256, 0, stream>>>(p);
        else kv4_append_kernel<64, W4A16_FP16><<<g, 256, 0, stream>>>(p);
    }
    return cudaGetLastError();
}

cudaError_t launch_kv4_read(const Kv4RowsParams& p, cudaStream_t stream)
{
    const unsigned g = row_blocks(p);
    if (p.head_dim == 128) {
        if (p.dtype == W4A16_BF16) kv4_read_kernel<128, W4A16_BF16><<<g, 256, 0, stream>>>(p);
        else if (p.dtype == W4A16_FP16) kv4_read_kernel<128, W4A16_FP16><<<g, 256, 0, stream>>>(p);
        else kv4_read_kernel<128, W4A16_FP32><<<g, 256, 0, stream>>>(p);
    } else {
        if (p.dtype == W4A16_BF16) kv4_read_kernel<64, W4A16_BF16><<<g, 256, 0, stream>>>(p);
        else if (p.dtype == W4A16_FP16) kv4_read_kernel<64, W4A16_FP16><<<g, 256, 0, stream>>>(p);
        else kv4_read_kernel<64, W4A16_FP32><<<g, 256, 0, stream>>>(p);
    }
    return cudaGetLastError();
}

}  // namespace w4a16
