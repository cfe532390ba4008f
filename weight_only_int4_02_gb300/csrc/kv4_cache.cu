// The 4-bit cache's bookkeeping and rows: block tables and slot maps from request
// lengths, quantisation of new keys and values into their slots, and the read back.
#include <cuda_bf16.h>
#include <cuda_fp16.h>


#include "kv4.cuh"
#include "launch.cuh"
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
// a thousand requests fill the GPU and a chunk of 512 tokens is 16 steps of its warp, four of
// whose page lookups are in flight together (8 requests 2.3 us; 1000 requests with 56061
// new tokens 4.4 us, 7.8 with one lookup at a time). A long chunk is one warp's all the same: 8191 tokens 26 us.
constexpr int kTabWarps = 8;

struct Need {
    int fresh, tokens;
};

__device__ __forceinline__ int pages_of(int tokens, const Kv4TablesParams& p)
{
    const int n = tokens <= 0 ? 0 : ((tokens - 1) >> (__ffs(p.page_size) - 1)) + 1;   // a power of two
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
    chained_kernel();
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
    const int shift = __ffs(p.page_size) - 1;   // a power of two
    const int count = (long long)p.max_tokens - start < mine.tokens ? p.max_tokens - start : mine.tokens;
    for (int i0 = lane; i0 < count; i0 += 128) {   // four tokens' pages are looked up together
        int page[4], pos[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            pos[q] = seq - mine.tokens + i0 + 32 * q;
            const int c = pos[q] >> shift;
            page[q] = -1;
            if (i0 + 32 * q < count && pos[q] >= 0 && c < p.max_pages) page[q] = c >= old ? fresh_page(c) : row[c];
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            if (i0 + 32 * q >= count) break;
            const long long at = (long long)start + i0 + 32 * q;
            p.slots[at] = page[q] >= 0 ? (long long)page[q] << shift | (pos[q] & (p.page_size - 1)) : -1;
            p.positions[at] = pos[q];
        }
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

__device__ __forceinline__ uint32_t negate2(uint32_t w) { return w ^ 0x80008000u; }

// The larger (smaller) of each pair; a NaN on either side gives a NaN.
template <int DTYPE>
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b)
{
    if constexpr (DTYPE == W4A16_BF16) {
        const __nv_bfloat162 m = __hmax2_nan(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
        return *reinterpret_cast<const uint32_t*>(&m);
    } else {
        const __half2 m = __hmax2_nan(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
        return *reinterpret_cast<const uint32_t*>(&m);
    }
}

template <int DTYPE>
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b)
{
    if constexpr (DTYPE == W4A16_BF16) {
        const __nv_bfloat162 m = __hmin2_nan(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
        return *reinterpret_cast<const uint32_t*>(&m);
    } else {
        const __half2 m = __hmin2_nan(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
        return *reinterpret_cast<const uint32_t*>(&m);
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
    const int shift = __ffs(p.page_size) - 1;   // a power of two
    const int in_page = (int)slot & (p.page_size - 1);
    *tok = in_page & 15;
    return p.cache + ((((slot >> shift) * p.kv_heads + head) << (shift - 4)) + (in_page >> 4)) * (long long)kv4_tile_bytes(D);
}

// The rows of a group of D/8 lanes: K and V of a token and KV head.
struct Rows {
    int token, head;
    bool live;
};

template <int D>
__device__ __forceinline__ Rows rows_of(const Kv4RowsParams& p)
{
    const uint32_t i = blockIdx.x * (256u / (D / 8)) + threadIdx.x / (D / 8);   // below 2^32: checked on the host
    Rows r;
    // i / kv_heads by the reciprocal, rounded down: right or one too small
    uint32_t token = __umulhi(i, p.per_head), head = i - token * (uint32_t)p.kv_heads;
    if (head >= (uint32_t)p.kv_heads) {
        ++token;
        head -= (uint32_t)p.kv_heads;
    }
    r.token = (int)token;
    r.head = (int)head;
    r.live = r.token < p.tokens;
    return r;
}

// What a row is stored with: 1 / s as a number, and s as binary16 bits below the zero-point and a poisoned row's flag.
struct Stored {
    float inv;
    uint32_t word;
    __device__ __forceinline__ uint32_t zero() const { return word >> 16 & 15u; }
    __device__ __forceinline__ bool poisoned() const { return word >> 31; }
};

// The extremes of eight values as a pair (max x, max -x) of the inputs' own type, exact; a NaN stays one.
template <int DTYPE>
__device__ __forceinline__ uint32_t extremes(const uint4& raw)
{
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
    uint32_t up = w[0], dn = w[0];
#pragma unroll
    for (int i = 1; i < 4; ++i) {
        up = max2<DTYPE>(up, w[i]);
        dn = min2<DTYPE>(dn, w[i]);
    }
    dn = negate2(dn);
    return max2<DTYPE>(__byte_perm(up, dn, 0x5410), __byte_perm(up, dn, 0x7632));
}

// rint by adding 1.5 * 2^23, whose last bit is 1: the sum's low bits are the whole number
constexpr float kRound = 12582912.0f;
__device__ __forceinline__ int whole(float v, float inv)
{
    return __float_as_int(__fadd_rn(__fmul_rn(v, inv), kRound)) - __float_as_int(kRound);
}

// From a row's extremes
//   s = fp16(min((hi - lo) / 15, 65504)), z = clamp(rint(-lo / s), 0, 15),
// with hi - lo formed from max(x, 0) and max(-x, 0), and 1 / s rounded once to FP32; every
// operation is an IEEE one (no contraction, no approximate division), so the codes are the same
// wherever the formula is evaluated. A row that holds an infinity or a NaN gets scale NaN, so
// that it shows in whatever reads it.
template <int DTYPE>
__device__ __forceinline__ Stored stored_of(uint32_t ext)
{
    float hi, neg;   // max(x, 0) and max(-x, 0)
    unpack2<DTYPE>(max2<DTYPE>(ext, 0u), hi, neg);
    if (!isfinite(hi) || !isfinite(neg)) return {0.0f, 0x80007fffu};
    const __half scale = __float2half_rn(fminf(__fdiv_rn(__fadd_rn(hi, neg), 15.0f), 65504.0f));
    const float s = __half2float(scale);
    Stored r;
    r.inv = s > 0.0f ? __frcp_rn(s) : 0.0f;
    r.word = (uint32_t)__half_as_ushort(scale) | (uint32_t)min(whole(neg, r.inv), 15) << 16;
    return r;
}

// Eight codes, four to a 16-bit word: clamp(rint(x / s) + z, 0, 15). Where the scale stays at 65504, a bfloat16 value may lie
// so many scales below 0 that the integer sum would pass its range; below -2^20, which no row of a smaller scale reaches,
// every code is 0, so such values stop there (four instructions more for eight values). Above 0 the sum cannot overflow.
template <int DTYPE>
__device__ __forceinline__ uint32_t codes_of(const uint4& raw, const Stored& r)
{
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
    const int z = (int)r.zero() - __float_as_int(kRound);
    uint32_t code[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float a, b;
        unpack2<DTYPE>(DTYPE == W4A16_BF16 ? max2<DTYPE>(w[i], 0xc980c980u) : w[i], a, b);
        // one by one: a packed product and sum are made one operation with one rounding
        code[2 * i] = (uint32_t)__viaddmin_s32_relu(__float_as_int(__fadd_rn(__fmul_rn(a, r.inv), kRound)), z, 15);
        code[2 * i + 1] = (uint32_t)__viaddmin_s32_relu(__float_as_int(__fadd_rn(__fmul_rn(b, r.inv), kRound)), z, 15);
    }
    uint32_t out = code[7];
#pragma unroll
    for (int i = 6; i >= 0; --i) out = out * 16u + code[i];
    return r.poisoned() ? 0u : out;
}

// Index of the 16-bit word of V's codes that holds d = 8j .. 8j + 3 of a token; the next four are two words on.
template <int D>
__device__ __forceinline__ int v_word(int tok, int j)
{
    const int n = 8 * j / (D / 8), w = (8 * j % (D / 8)) / 4;   // token 8h + 2c + e
    return ((((tok >> 3) * 8 + n) * 4 + ((tok & 7) >> 1)) * (D / 32) + w) * 2 + (tok & 1);
}

// Quantises the new rows into their slots. Reads 4 D bytes a token and head and writes
// 2 (D + 6): bound by bandwidth for a long prompt, by latency for a decode step. A thread has its K and
// its V load in flight together (8191 tokens of eight heads of 128: 12.6 us against 16.2 with one
// row a thread), and every lane goes on with one row's extremes and scale (now 11.0 us). Half of that
// time is the bytes', the rest instructions (issue slots 77% busy) and the launch; V's 2-byte stores are 0.5 us of it.
template <int D, int DTYPE>
__global__ void __launch_bounds__(256) kv4_append_kernel(const Kv4RowsParams p)
{
    chained_kernel();
    const Rows r = rows_of<D>(p);
    const int j = threadIdx.x % (D / 8);
    uint4 k = make_uint4(0, 0, 0, 0), v = k;
    uint8_t* tile = nullptr;
    int tok = 0;
    if (r.live) {
        k = __ldg(reinterpret_cast<const uint4*>((const uint16_t*)p.k + r.token * p.k_token + r.head * p.k_head + 8 * j));
        v = __ldg(reinterpret_cast<const uint4*>((const uint16_t*)p.v + r.token * p.v_token + r.head * p.v_head + 8 * j));
        tile = tile_of(p, r.token, r.head, D, &tok);
    }
    // Even lanes go on with K's row and odd ones with V's: extremes, scale and zero-point once a lane, not twice.
    const uint32_t ek = extremes<DTYPE>(k), ev = extremes<DTYPE>(v);
    const bool odd = j & 1;
    uint32_t ext = max2<DTYPE>(odd ? ev : ek, __shfl_xor_sync(0xffffffffu, odd ? ek : ev, 1));
#pragma unroll
    for (int d = 2; d < D / 8; d <<= 1) ext = max2<DTYPE>(ext, __shfl_xor_sync(0xffffffffu, ext, d));
    const Stored mine = stored_of<DTYPE>(ext);
    const Stored other = {__shfl_xor_sync(0xffffffffu, mine.inv, 1), __shfl_xor_sync(0xffffffffu, mine.word, 1)};
    const uint32_t a = codes_of<DTYPE>(k, odd ? other : mine), b = codes_of<DTYPE>(v, odd ? mine : other);
    if (tile == nullptr) return;
    *reinterpret_cast<uint32_t*>(tile + tok * (D / 2) + 4 * j) = a;
    uint16_t* const dst = reinterpret_cast<uint16_t*>(tile + kv4_v_off(D)) + v_word<D>(tok, j);
    dst[0] = (uint16_t)b;
    dst[2] = (uint16_t)(b >> 16);
    if (j < 2) {   // lane 0 writes K's scale and zero-point, lane 1 V's
        *reinterpret_cast<uint16_t*>(tile + (j ? kv4_v_scale_off(D) : kv4_k_scale_off(D)) + 2 * tok) = (uint16_t)mine.word;
        tile[(j ? kv4_v_zero_off(D) : kv4_k_zero_off(D)) + tok] = (uint8_t)mine.zero();
    }
}

// The values that slots stand for, (code - zero) * scale in FP32, rounded once. Lanes as above. Bound by its instructions
// and the loads' latency: 8191 tokens of eight heads of 128 in 7.4 us (8.5 with a shift a code and scalar sums).
template <int D, int DTYPE>
__global__ void __launch_bounds__(256) kv4_read_kernel(const Kv4RowsParams p)
{
    chained_kernel();
    const Rows r = rows_of<D>(p);
    const int j = threadIdx.x % (D / 8);
    if (!r.live) return;
    int tok = 0;
    const uint8_t* tile = tile_of(p, r.token, r.head, D, &tok);
    uint32_t w[2] = {0, 0};
    float s[2] = {0.0f, 0.0f}, z[2] = {0.0f, 0.0f};
    if (tile) {
        w[0] = *reinterpret_cast<const uint32_t*>(tile + tok * (D / 2) + 4 * j);
        const uint16_t* src = reinterpret_cast<const uint16_t*>(tile + kv4_v_off(D)) + v_word<D>(tok, j);
        w[1] = src[0] | (uint32_t)src[2] << 16;
        s[0] = __half2float(*reinterpret_cast<const __half*>(tile + kv4_k_scale_off(D) + 2 * tok));
        s[1] = __half2float(*reinterpret_cast<const __half*>(tile + kv4_v_scale_off(D) + 2 * tok));
        z[0] = (float)tile[kv4_k_zero_off(D) + tok];
        z[1] = (float)tile[kv4_v_zero_off(D) + tok];
    }
    const long long at = ((long long)r.token * p.kv_heads + r.head) * D + 8 * j;
#pragma unroll
    for (int o = 0; o < 2; ++o) {
        void* const out = o ? p.v_out : p.k_out;
        float x[8];
        const float from = -8388608.0f - z[o];
        const uint64_t from2 = pack_f32x2(from, from), s2 = pack_f32x2(s[o], s[o]);
        const uint32_t even = w[o] & 0x0f0f0f0fu, odd = w[o] >> 4 & 0x0f0f0f0fu;
#pragma unroll
        for (int i = 0; i < 4; ++i)   // 2^23 + code, exact, less 2^23 + zero
            unpack_f32x2(mul_f32x2(add_f32x2(pack_f32x2(__uint_as_float(__byte_perm(even, 0x4b000000u, 0x7440 | i)),
                                                        __uint_as_float(__byte_perm(odd, 0x4b000000u, 0x7440 | i))), from2), s2),
                         x[2 * i], x[2 * i + 1]);
        if constexpr (DTYPE == W4A16_FP32) {
            float4* dst = reinterpret_cast<float4*>((float*)out + at);
            dst[0] = make_float4(x[0], x[1], x[2], x[3]);
            dst[1] = make_float4(x[4], x[5], x[6], x[7]);
        } else {
            *reinterpret_cast<uint4*>((uint16_t*)out + at) =
                make_uint4(pack2<DTYPE>(x[0], x[1]), pack2<DTYPE>(x[2], x[3]), pack2<DTYPE>(x[4], x[5]), pack2<DTYPE>(x[6], x[7]));
        }
    }
}

unsigned row_blocks(const Kv4RowsParams& p)
{
    const long long per = 256 / (p.head_dim / 8);
    return (unsigned)(((long long)p.tokens * p.kv_heads + per - 1) / per);
}

}  // namespace

cudaError_t launch_kv4_tables(const Kv4TablesParams& p, cudaStream_t stream)
{
    const unsigned blocks = p.batch > 0 ? (unsigned)((p.batch - 1) / kTabWarps + 1) : 1u;   // an empty batch still has ends to write
    return launch_chained(kv4_tables_kernel, blocks, kTabWarps * 32, 0, 1, stream, p);
}

cudaError_t launch_kv4_append(const Kv4RowsParams& p, cudaStream_t stream)
{
    const bool bf = p.dtype == W4A16_BF16;
    auto* const kernel = p.head_dim == 128 ? (bf ? kv4_append_kernel<128, W4A16_BF16> : kv4_append_kernel<128, W4A16_FP16>)
                                           : (bf ? kv4_append_kernel<64, W4A16_BF16> : kv4_append_kernel<64, W4A16_FP16>);
    return launch_chained(kernel, row_blocks(p), 256, 0, 1, stream, p);
}

cudaError_t launch_kv4_read(const Kv4RowsParams& p, cudaStream_t stream)
{
    auto* kernel = p.head_dim == 128 ? kv4_read_kernel<128, W4A16_FP32> : kv4_read_kernel<64, W4A16_FP32>;
    if (p.dtype == W4A16_BF16) kernel = p.head_dim == 128 ? kv4_read_kernel<128, W4A16_BF16> : kv4_read_kernel<64, W4A16_BF16>;
    if (p.dtype == W4A16_FP16) kernel = p.head_dim == 128 ? kv4_read_kernel<128, W4A16_FP16> : kv4_read_kernel<64, W4A16_FP16>;
    return launch_chained(kernel, row_blocks(p), 256, 0, 1, stream, p);
}

}  // namespace w4a16
