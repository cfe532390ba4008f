// The 8-bit cache's rows: keys rotated on the way and quantised with their values into their slots, and the read back.
#include "kv8.cuh"
#include "launch.cuh"
#include "pairs.cuh"
#include "w4a16.h"

#include <math_constants.h>

namespace w4a16 {
namespace {

constexpr int kWarps = 8;
constexpr float kLeastScale = 0x1p-40f, kMostScale = 0x1p40f;
constexpr uint32_t kFull = 0xffffffffu;

// Address of the tile that holds a slot.
__device__ __forceinline__ uint8_t* tile_of(const Kv8RowsParams& p, long long slot, int head, int D)
{
    const int shift = __ffs(p.page_size) - 1;   // a power of two
    const int in_page = (int)slot & (p.page_size - 1);
    return p.cache + ((((slot >> shift) * p.kv_heads + head) << (shift - 4)) + (in_page >> 4)) * (long long)kv8_tile_bytes(D);
}

template <int DTYPE>
__device__ __forceinline__ void unpack8(const uint4& raw, float (&x)[8])
{
    unpack2<DTYPE>(raw.x, x[0], x[1]);
    unpack2<DTYPE>(raw.y, x[2], x[3]);
    unpack2<DTYPE>(raw.z, x[4], x[5]);
    unpack2<DTYPE>(raw.w, x[6], x[7]);
}

// A word of four low bytes.
__device__ __forceinline__ uint32_t bytes4(uint32_t a, uint32_t b, uint32_t c, uint32_t d)
{
    return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

// clamp(rint(x * inv), -127, 127) + 128 in the low byte: rint by adding 1.5 * 2^23, whose last bits are 0, and 128.
__device__ __forceinline__ uint32_t code_of(float x, float inv)
{
    const float v = fminf(fmaxf(__fmul_rn(x, inv), -127.0f), 127.0f);
    return __float_as_uint(__fadd_rn(v, 12582912.0f + 128.0f));
}

// The code of what four codes stand for, with a scale 1 / f times as large.
__device__ __forceinline__ uint32_t less4(uint32_t w, float f)
{
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = code_of((float)(int)(w >> (8 * i) & 255u) - 128.0f, f);
    return bytes4(c[0], c[1], c[2], c[3]);
}

// What a tile is stored with from now on. top: bits of the largest magnitude of the new rows.
struct Scale {
    float now, inv, less;   // the scale, its reciprocal or 0, and what earlier codes are multiplied by (1: they stay)
};

__device__ __forceinline__ Scale scale_of(uint32_t top, float old)
{
    float a = __fdiv_rn(__uint_as_float(top), 127.0f);
    a = a < kLeastScale ? 0.0f : fminf(a, kMostScale);
    if (top >= 0x7f800000u || old != old) return {CUDART_NAN_F, 0.0f, 1.0f};
    Scale s;
    s.now = fmaxf(old, a);
    s.inv = s.now > 0.0f ? __frcp_rn(s.now) : 0.0f;
    s.less = a > old ? __fmul_rn(old, s.inv) : 1.0f;
    return s;
}

// A lane's dims of a row of K, and where their codes begin in a token's slabs.
template <int D, int MODE>
struct KeyLane {
    LaneDims at;
    int byte[2];
    __device__ __forceinline__ KeyLane(int j, int rot) : at(lane_dims<MODE>(j, rot))
    {
        byte[0] = (at.a >> 6) * 1024 + (at.a & 63);
        byte[1] = (at.b >> 6) * 1024 + (at.b & 63);
    }
};

// A run: neighbours in the list whose slots are neighbours in one tile. One warp stores a run's keys or values of one head.
struct Run {
    uint8_t* tile;
    int token, off, count;   // first token, its place in the tile, tokens
};

template <int D, int DTYPE, int MODE>
__device__ __forceinline__ void store_keys(const Kv8RowsParams& p, const Run& run, int head)
{
    constexpr int kLanes = D / 8, kTogether = 32 / kLanes, kSteps = 16 / kTogether;
    const int lane = threadIdx.x & 31, sub = lane / kLanes;
    const KeyLane<D, MODE> my(lane % kLanes, p.rope.rot);
    float x[kSteps][8];
    uint2 raw[kSteps][2];
    const int end = run.off + run.count;
    const uint16_t* const from = (const uint16_t*)p.k + head * p.k_head;
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
        const int tok = i * kTogether + sub;
        raw[i][0] = raw[i][1] = make_uint2(0, 0);
        if (tok >= run.off && tok < end) {
            const uint16_t* const row = from + (run.token + tok - run.off) * p.k_token;
            raw[i][0] = __ldg(reinterpret_cast<const uint2*>(row + my.at.a));
            raw[i][1] = __ldg(reinterpret_cast<const uint2*>(row + my.at.b));
        }
    }
    const float old = run.off > 0 ? *reinterpret_cast<const float*>(run.tile + kv8_k_scale_off(D)) : 0.0f;
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
        const int tok = i * kTogether + sub;
        unpack8<DTYPE>(make_uint4(raw[i][0].x, raw[i][0].y, raw[i][1].x, raw[i][1].y), x[i]);
        if constexpr (MODE != kRopeNone) {
            if (tok >= run.off && tok < end) {
                const int pos = __ldg(p.rope.positions + run.token + tok - run.off);
                if (pos < 0 || pos >= p.rope.rows) {
                    x[i][0] = CUDART_NAN_F;   // a position that the table does not have poisons the tile
                } else if (my.at.turned) {
                    const float* const row = p.rope.table + (long long)pos * p.rope.rot + 4 * (lane % kLanes);
                    rotate<MODE>(x[i], __ldg(reinterpret_cast<const float4*>(row)),
                                 __ldg(reinterpret_cast<const float4*>(row + p.rope.rot / 2)));
                }
            }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(x[i][e]) & 0x7fffffffu);
    }
    const Scale s = scale_of(__reduce_max_sync(kFull, top), old);
    const bool again = s.less != 1.0f;
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
        const int tok = i * kTogether + sub;
#pragma unroll
        for (int o = 0; o < 2; ++o) {
            uint32_t* const at = reinterpret_cast<uint32_t*>(run.tile + tok * 64 + my.byte[o]);
            if (tok >= run.off && tok < end) {
                uint32_t c[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) c[e] = code_of(x[i][4 * o + e], s.inv);
                *at = s.inv > 0.0f ? bytes4(c[0], c[1], c[2], c[3]) : 0x80808080u;
            } else if (again && tok < run.off) {
                *at = less4(*at, s.less);
            }
        }
    }
    __syncwarp();   // every lane has the old scale
    if (lane == 0) *reinterpret_cast<float*>(run.tile + kv8_k_scale_off(D)) = s.now;
}

// Values: a lane has eight d of two neighbouring tokens, 16 bytes of codes.
template <int D, int DTYPE>
__device__ __forceinline__ void store_values(const Kv8RowsParams& p, const Run& run, int head)
{
    constexpr int kLanes = D / 8, kTogether = 32 / kLanes, kSteps = 8 / kTogether;   // pairs of tokens
    const int lane = threadIdx.x & 31, sub = lane / kLanes, j = lane % kLanes;
    const int end = run.off + run.count;
    const uint16_t* const from = (const uint16_t*)p.v + head * p.v_head + 8 * j;
    uint4 raw[kSteps][2];
#pragma unroll
    for (int i = 0; i < kSteps; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int tok = 2 * (i * kTogether + sub) + e;
            raw[i][e] = make_uint4(0, 0, 0, 0);
            if (tok >= run.off && tok < end) raw[i][e] = __ldg(reinterpret_cast<const uint4*>(from + (run.token + tok - run.off) * p.v_token));
        }
    const float old = run.off > 0 ? *reinterpret_cast<const float*>(run.tile + kv8_v_scale_off(D)) : 0.0f;
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < kSteps; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float x[8];
            unpack8<DTYPE>(raw[i][e], x);
#pragma unroll
            for (int d = 0; d < 8; ++d) top = max(top, __float_as_uint(x[d]) & 0x7fffffffu);
        }
    const Scale s = scale_of(__reduce_max_sync(kFull, top), old);
    const bool again = s.less != 1.0f;
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
        const int pair = i * kTogether + sub;
        uint8_t* const at = run.tile + kv8_v_off(D) + (((j >> 3) * 2 + (pair >> 2)) * 8 + (j & 7)) * 64 + (pair & 3) * 16;
        if (again && 2 * pair < run.off) {   // bytes of tokens that follow are written below, or hold nothing
            uint4 w = *reinterpret_cast<const uint4*>(at);
            w = make_uint4(less4(w.x, s.less), less4(w.y, s.less), less4(w.z, s.less), less4(w.w, s.less));
            *reinterpret_cast<uint4*>(at) = w;
        }
        uint32_t half[2][4];   // two codes each
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float x[8];
            unpack8<DTYPE>(raw[i][e], x);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const uint32_t two = __byte_perm(code_of(x[2 * q], s.inv), code_of(x[2 * q + 1], s.inv), 0x0040);
                half[e][q] = s.inv > 0.0f ? two : 0x8080u;
            }
        }
        const bool first = 2 * pair >= run.off && 2 * pair < end, second = 2 * pair + 1 >= run.off && 2 * pair + 1 < end;
        if (first && second) {
            *reinterpret_cast<uint4*>(at) = make_uint4(__byte_perm(half[0][0], half[1][0], 0x5410), __byte_perm(half[0][1], half[1][1], 0x5410),
                                                       __byte_perm(half[0][2], half[1][2], 0x5410), __byte_perm(half[0][3], half[1][3], 0x5410));
        } else if (first || second) {
#pragma unroll
            for (int q = 0; q < 4; ++q) *reinterpret_cast<uint16_t*>(at + 4 * q + (second ? 2 : 0)) = (uint16_t)(second ? half[1][q] : half[0][q]);
        }
    }
    __syncwarp();
    if (lane == 0) *reinterpret_cast<float*>(run.tile + kv8_v_scale_off(D)) = s.now;
}

// Quantises new rows into their slots, K rotated on the way, with a scale for a tile of 16 tokens and head:
//   s = max(old, max |x| / 127), code = clamp(rint(x / s), -127, 127) + 128,
// old being 0 where the run begins at the tile's first token; codes stored before are rounded again where s grew. Reads 4 D bytes
// a token and head and writes 2 D. A warp looks at `window` places of the list, finds the runs that begin there
// and stores one head's K or V of each. A tile belongs to one warp, so there is no word between warps and no
// order of theirs that shows.
template <int D, int DTYPE, int MODE>
__global__ void __launch_bounds__(kWarps * 32) kv8_append_kernel(const Kv8RowsParams p)
{
    chained_kernel();
    const int lane = threadIdx.x & 31;
    const long long item = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
    const int per = 2 * p.kv_heads;
    const long long place = item / per;
    const int rest = (int)(item - place * per), head = rest >> 1;
    const long long w0 = place * p.window;
    if (w0 >= p.tokens) return;
    // lane l: place w0 - 1 + l; runs that begin in the window end 15 places past it at most
    const long long t = w0 - 1 + lane;
    const long long slot = t >= 0 && t < p.tokens ? p.slots[t] : -2;
    const bool live = slot >= 0 && slot < p.n_slots;
    const long long before = __shfl_up_sync(kFull, slot, 1);
    const bool follows = live && (slot & 15) != 0 && before == slot - 1;
    const uint32_t chain = __ballot_sync(kFull, follows);
    uint32_t begins = __ballot_sync(kFull, live && !follows && lane >= 1 && lane <= p.window && t < p.tokens);
    while (begins) {
        const int l = __ffs(begins) - 1;
        begins &= begins - 1;
        const long long s = __shfl_sync(kFull, slot, l);
        Run run;
        run.tile = tile_of(p, s, head, D);
        run.token = (int)(w0 - 1 + l);
        run.off = (int)(s & 15);
        run.count = __ffs(~(l < 31 ? chain >> (l + 1) : 0u));   // itself and what follows it
        if (rest & 1) store_values<D, DTYPE>(p, run, head);
        else store_keys<D, DTYPE, MODE>(p, run, head);
    }
}

// The values that slots stand for, (code - 128) * scale in FP32, rounded once. D / 8 lanes a token and head.
template <int D, int DTYPE>
__global__ void __launch_bounds__(256) kv8_read_kernel(const Kv8RowsParams p)
{
    chained_kernel();
    constexpr int kLanes = D / 8;
    const long long i = (long long)blockIdx.x * (256 / kLanes) + threadIdx.x / kLanes;
    const int j = threadIdx.x % kLanes;
    const uint32_t token = (uint32_t)i / (uint32_t)p.kv_heads, head = (uint32_t)i - token * (uint32_t)p.kv_heads;   // below 2^32: checked on the host
    if (token >= (uint32_t)p.tokens) return;
    const long long slot = p.slots[token];
    uint32_t w[2][2] = {{0x80808080u, 0x80808080u}, {0x80808080u, 0x80808080u}};
    float s[2] = {0.0f, 0.0f};
    if (slot >= 0 && slot < p.n_slots) {
        const uint8_t* const tile = tile_of(p, slot, (int)head, D);
        const int tok = (int)slot & 15;
        const uint2 k = *reinterpret_cast<const uint2*>(tile + ((j >> 3) * 16 + tok) * 64 + 8 * (j & 7));
        const uint4 v = *reinterpret_cast<const uint4*>(tile + kv8_v_off(D) + (((j >> 3) * 2 + (tok >> 3)) * 8 + (j & 7)) * 64 +
                                                        (tok >> 1 & 3) * 16);
        const float2 both = *reinterpret_cast<const float2*>(tile + kv8_k_scale_off(D));
        s[0] = both.x;
        s[1] = both.y;
        w[0][0] = k.x;
        w[0][1] = k.y;
        const uint32_t pick = tok & 1 ? 0x7632u : 0x5410u;
        w[1][0] = __byte_perm(v.x, v.y, pick);
        w[1][1] = __byte_perm(v.z, v.w, pick);
    }
    const long long at = ((long long)token * p.kv_heads + head) * D + 8 * j;
#pragma unroll
    for (int o = 0; o < 2; ++o) {
        void* const out = o ? p.v_out : p.k_out;
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)   // 2^23 + code, exact, less 2^23 + 128
            x[e] = __fmul_rn(__uint_as_float(__byte_perm(w[o][e >> 2], 0x4b000000u, 0x7440 | (e & 3))) - 8388736.0f, s[o]);
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

template <int D, int DTYPE>
auto* append_of(int mode)
{
    return mode == kRopeNone ? kv8_append_kernel<D, DTYPE, kRopeNone>
                             : mode == kRopeHalves ? kv8_append_kernel<D, DTYPE, kRopeHalves> : kv8_append_kernel<D, DTYPE, kRopePairs>;
}

}  // namespace

cudaError_t launch_kv8_append(const Kv8RowsParams& in, cudaStream_t stream)
{
    Kv8RowsParams p = in;
    p.window = p.tokens <= 1024 ? 1 : 16;
    const long long items = ((long long)p.tokens + p.window - 1) / p.window * 2 * p.kv_heads, blocks = (items + kWarps - 1) / kWarps;
    if (blocks >= 1LL << 31) return cudaErrorInvalidValue;
    const bool bf = p.dtype == W4A16_BF16;
    auto* const kernel = p.head_dim == 128 ? (bf ? append_of<128, W4A16_BF16>(p.mode) : append_of<128, W4A16_FP16>(p.mode))
                                           : (bf ? append_of<64, W4A16_BF16>(p.mode) : append_of<64, W4A16_FP16>(p.mode));
    return launch_chained(kernel, (unsigned)blocks, kWarps * 32, 0, 1, stream, p);
}

cudaError_t launch_kv8_read(const Kv8RowsParams& p, cudaStream_t stream)
{
    auto* kernel = p.head_dim == 128 ? kv8_read_kernel<128, W4A16_FP32> : kv8_read_kernel<64, W4A16_FP32>;
    if (p.dtype == W4A16_BF16) kernel = p.head_dim == 128 ? kv8_read_kernel<128, W4A16_BF16> : kv8_read_kernel<64, W4A16_BF16>;
    if (p.dtype == W4A16_FP16) kernel = p.head_dim == 128 ? kv8_read_kernel<128, W4A16_FP16> : kv8_read_kernel<64, W4A16_FP16>;
    const long long per = 256 / (p.head_dim / 8);
    return launch_chained(kernel, (unsigned)(((long long)p.tokens * p.kv_heads + per - 1) / per), 256, 0, 1, stream, p);
}

}  // namespace w4a16
