// The 8-bit cache's rows: keys rotated on the way and quantised with their values into their slots, and the read back.
#include "kv8.cuh"
#include "launch.cuh"
#include "pairs.cuh"
#include "w4a16.h"

#include <math_constants.h>

#include <type_traits>

namespace w4a16 {
namespace {

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

// clamp(rint(x * inv), -127, 127) + 128 in the low byte: rint by adding 1.5 * 2^23, whose last bits are 0, and 128. Product and
// sum one by one: packed ones are made one operation with one rounding. Without CLAMP |x * inv| is to be below 127.5.
template <bool CLAMP>
__device__ __forceinline__ uint32_t code_of(float x, float inv)
{
    float v = __fmul_rn(x, inv);
    if (CLAMP) v = fminf(fmaxf(v, -127.0f), 127.0f);
    return __float_as_uint(__fadd_rn(v, 12582912.0f + 128.0f));
}

// The code of what four codes stand for, with a scale 1 / f times as large.
__device__ __forceinline__ uint32_t less4(uint32_t w, float f)
{
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = code_of<true>((float)(int)(w >> (8 * i) & 255u) - 128.0f, f);
    return bytes4(c[0], c[1], c[2], c[3]);
}

// What a tile is stored with from now on. top: bits of the largest magnitude of the new rows.
struct Scale {
    float now, inv, less;   // the scale, its reciprocal or 0, and what earlier codes are multiplied by (1: they stay)
};

// Calls f with whether codes have to be clamped: rows have no magnitude above 127 scales, but for two roundings, unless the scale
// stays at its largest.
template <typename F>
__device__ __forceinline__ void with_clamp(const Scale& s, F f)
{
    if (s.now >= kMostScale) f(std::true_type());
    else f(std::false_type());
}

__device__ __forceinline__ Scale scale_of(uint32_t top, float old)
{
    float a = __fmul_rn(__uint_as_float(top), 1.0f / 127.0f);
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

// A lane's values of a key, rotated by its position; one that the table does not have poisons the tile.
template <int MODE>
__device__ __forceinline__ void turn(const Kv8RowsParams& p, float (&x)[8], int pos, int j, bool turned)
{
    if ((unsigned)pos >= (unsigned)p.rope.rows) {
        x[0] = CUDART_NAN_F;
    } else if (turned) {
        const float* const row = p.rope.table + (long long)pos * p.rope.rot + 4 * j;
        rotate<MODE>(x, __ldg(reinterpret_cast<const float4*>(row)), __ldg(reinterpret_cast<const float4*>(row + p.rope.rot / 2)));
    }
}

// A run: neighbours in the list whose slots are neighbours in one tile.
struct Run {
    uint8_t* tile;
    int token, off, end;   // first token; its place in the tile, and that behind the last
    int lane, pos;         // the lane that holds the first token's position; this lane's
    __device__ __forceinline__ bool has(int tok) const { return tok >= off && tok < end; }
};

// Two warps store a run's keys or values of one head, eight of the tile's places each; the larger of their maxima is
// both's. top: bits of this warp's largest magnitude. Two runs that follow each other use different words.
__device__ __forceinline__ uint32_t both_tops(uint32_t (&shared)[2], int half, uint32_t top)
{
    if ((threadIdx.x & 31) == 0) shared[half] = top;
    __syncthreads();
    return max(shared[0], shared[1]);
}

// The largest of top and two magnitudes; a NaN stays one.
__device__ __forceinline__ float top3(float top, float a, float b)
{
    float y;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(top), "f"(fabsf(a)), "f"(fabsf(b)));
    return y;
}

__device__ __forceinline__ float top_of(const float (&x)[8], float top)
{
#pragma unroll
    for (int e = 0; e < 8; e += 2) top = top3(top, x[e], x[e + 1]);
    return top;
}

// Over a warp, as bits: of numbers that are not negative they are in the numbers' order, a NaN's are the greatest.
__device__ __forceinline__ uint32_t warp_top(float top) { return __reduce_max_sync(kFull, __float_as_uint(top) & 0x7fffffffu); }

// WHOLE: the run is all of its tile.
template <int D, int DTYPE, int MODE, bool WHOLE>
__device__ __forceinline__ void store_keys(const Kv8RowsParams& p, const Run& run, int head, int half, uint32_t (&shared)[2])
{
    constexpr int kLanes = D / 8, kTogether = 32 / kLanes, kSteps = 8 / kTogether;
    const int lane = threadIdx.x & 31, place0 = 8 * half + lane / kLanes;
    const KeyLane<D, MODE> my(lane % kLanes, p.rope.rot);
    float x[kSteps][8];
    const uint16_t* const from = (const uint16_t*)p.k + head * p.k_head;
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
        const int tok = place0 + i * kTogether;
        uint2 a = make_uint2(0, 0), b = a;
        if (WHOLE || run.has(tok)) {
            const uint16_t* const row = from + (run.token + tok - run.off) * p.k_token;
            a = __ldg(reinterpret_cast<const uint2*>(row + my.at.a));
            b = __ldg(reinterpret_cast<const uint2*>(row + my.at.b));
        }
        unpack8<DTYPE>(make_uint4(a.x, a.y, b.x, b.y), x[i]);
    }
    const float old = !WHOLE && run.off > 0 ? *reinterpret_cast<const float*>(run.tile + kv8_k_scale_off(D)) : 0.0f;
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
        if constexpr (MODE != kRopeNone) {
            const int tok = place0 + i * kTogether, pos = __shfl_sync(kFull, run.pos, run.lane + tok - run.off & 31);
            if (WHOLE || run.has(tok)) turn<MODE>(p, x[i], pos, lane % kLanes, my.at.turned);
        }
        top = top_of(x[i], top);
    }
    const Scale s = scale_of(both_tops(shared, half, warp_top(top)), old);
    const bool again = !WHOLE && s.less != 1.0f;
    with_clamp(s, [&](auto clamp) {
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            const int tok = place0 + i * kTogether;
#pragma unroll
            for (int o = 0; o < 2; ++o) {
                uint32_t* const at = reinterpret_cast<uint32_t*>(run.tile + tok * 64 + my.byte[o]);
                if (WHOLE || run.has(tok)) {
                    uint32_t c[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) c[e] = code_of<clamp.value>(x[i][4 * o + e], s.inv);
                    *at = s.inv > 0.0f ? bytes4(c[0], c[1], c[2], c[3]) : 0x80808080u;
                } else if (again && tok < run.off) {
                    *at = less4(*at, s.less);
                }
            }
        }
    });
    if (half == 0 && lane == 0) *reinterpret_cast<float*>(run.tile + kv8_k_scale_off(D)) = s.now;
}

// Values: a lane has eight d of two neighbouring tokens, 16 bytes of codes.
template <int D, int DTYPE, bool WHOLE>
__device__ __forceinline__ void store_values(const Kv8RowsParams& p, const Run& run, int head, int half, uint32_t (&shared)[2])
{
    constexpr int kLanes = D / 8, kTogether = 32 / kLanes, kSteps = 4 / kTogether;   // pairs of tokens
    const int lane = threadIdx.x & 31, j = lane % kLanes, two0 = 4 * half + lane / kLanes;
    const uint16_t* const from = (const uint16_t*)p.v + head * p.v_head + 8 * j;
    uint4 raw[kSteps][2];
#pragma unroll
    for (int i = 0; i < kSteps; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int tok = 2 * (two0 + i * kTogether) + e;
            raw[i][e] = make_uint4(0, 0, 0, 0);
            if (WHOLE || run.has(tok)) raw[i][e] = __ldg(reinterpret_cast<const uint4*>(from + (run.token + tok - run.off) * p.v_token));
        }
    const float old = !WHOLE && run.off > 0 ? *reinterpret_cast<const float*>(run.tile + kv8_v_scale_off(D)) : 0.0f;
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < kSteps; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float x[8];
            unpack8<DTYPE>(raw[i][e], x);
            top = top_of(x, top);
        }
    const Scale s = scale_of(both_tops(shared, half, warp_top(top)), old);
    const bool again = !WHOLE && s.less != 1.0f;
    with_clamp(s, [&](auto clamp) {
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            const int two = two0 + i * kTogether;
            uint8_t* const at = run.tile + kv8_v_off(D) + (((j >> 3) * 2 + (two >> 2)) * 8 + (j & 7)) * 64 + (two & 3) * 16;
            if (again && 2 * two < run.off) {   // the second token's bytes, where it is a new one, are written below
                uint4 w = *reinterpret_cast<const uint4*>(at);
                w = make_uint4(less4(w.x, s.less), less4(w.y, s.less), less4(w.z, s.less), less4(w.w, s.less));
                *reinterpret_cast<uint4*>(at) = w;
            }
            const bool first = WHOLE || run.has(2 * two), second = WHOLE || run.has(2 * two + 1);
            if (!first && !second) continue;
            float x[2][8];
            unpack8<DTYPE>(raw[i][0], x[0]);
            unpack8<DTYPE>(raw[i][1], x[1]);
            uint32_t word[4];   // two d of both tokens
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                word[q] = bytes4(code_of<clamp.value>(x[0][2 * q], s.inv), code_of<clamp.value>(x[0][2 * q + 1], s.inv),
                                 code_of<clamp.value>(x[1][2 * q], s.inv), code_of<clamp.value>(x[1][2 * q + 1], s.inv));
                if (!(s.inv > 0.0f)) word[q] = 0x80808080u;
            }
            if (first && second) {
                *reinterpret_cast<uint4*>(at) = make_uint4(word[0], word[1], word[2], word[3]);
            } else {
#pragma unroll
                for (int q = 0; q < 4; ++q) *reinterpret_cast<uint16_t*>(at + 4 * q + (second ? 2 : 0)) = (uint16_t)(second ? word[q] >> 16 : word[q]);
            }
        }
    });
    if (half == 0 && lane == 0) *reinterpret_cast<float*>(run.tile + kv8_v_scale_off(D)) = s.now;
}

// The largest of D / 8 lanes' numbers, as warp_top.
template <int D>
__device__ __forceinline__ uint32_t lanes_top(float top)
{
    uint32_t t = __float_as_uint(top) & 0x7fffffffu;
#pragma unroll
    for (int d = 1; d < D / 8; d <<= 1) t = max(t, __shfl_xor_sync(kFull, t, d));
    return t;
}

// Runs of one token, as batches of decoding requests have them: D / 8 lanes a run. `fine`: these lanes have one.
template <int D, int DTYPE, int MODE>
__device__ __forceinline__ void store_key(const Kv8RowsParams& p, bool fine, long long slot, int token, int pos, int head)
{
    const int j = threadIdx.x % (D / 8), off = (int)slot & 15;
    const KeyLane<D, MODE> my(j, p.rope.rot);
    uint8_t* const tile = tile_of(p, fine ? slot : 0, head, D);
    float x[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f}, old = 0.0f;
    if (fine) {
        const uint16_t* const row = (const uint16_t*)p.k + head * p.k_head + token * p.k_token;
        const uint2 a = __ldg(reinterpret_cast<const uint2*>(row + my.at.a)), b = __ldg(reinterpret_cast<const uint2*>(row + my.at.b));
        if (off > 0) old = *reinterpret_cast<const float*>(tile + kv8_k_scale_off(D));
        unpack8<DTYPE>(make_uint4(a.x, a.y, b.x, b.y), x);
        if constexpr (MODE != kRopeNone) turn<MODE>(p, x, pos, j, my.at.turned);
    }
    const Scale s = scale_of(lanes_top<D>(top_of(x, 0.0f)), old);
    if (!fine) return;
    with_clamp(s, [&](auto clamp) {
#pragma unroll
        for (int o = 0; o < 2; ++o) {
            uint32_t c[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) c[e] = code_of<clamp.value>(x[4 * o + e], s.inv);
            *reinterpret_cast<uint32_t*>(tile + off * 64 + my.byte[o]) = s.inv > 0.0f ? bytes4(c[0], c[1], c[2], c[3]) : 0x80808080u;
        }
    });
    if (s.less != 1.0f)
        for (int t = 0; t < off; ++t)
#pragma unroll
            for (int o = 0; o < 2; ++o) {
                uint32_t* const at = reinterpret_cast<uint32_t*>(tile + t * 64 + my.byte[o]);
                *at = less4(*at, s.less);
            }
    if (j == 0) *reinterpret_cast<float*>(tile + kv8_k_scale_off(D)) = s.now;
}

template <int D, int DTYPE>
__device__ __forceinline__ void store_value(const Kv8RowsParams& p, bool fine, long long slot, int token, int head)
{
    const int j = threadIdx.x % (D / 8), off = (int)slot & 15;
    uint8_t* const tile = tile_of(p, fine ? slot : 0, head, D);
    float x[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f}, old = 0.0f;
    if (fine) {
        const uint4 raw = __ldg(reinterpret_cast<const uint4*>((const uint16_t*)p.v + head * p.v_head + token * p.v_token + 8 * j));
        if (off > 0) old = *reinterpret_cast<const float*>(tile + kv8_v_scale_off(D));
        unpack8<DTYPE>(raw, x);
    }
    const Scale s = scale_of(lanes_top<D>(top_of(x, 0.0f)), old);
    if (!fine) return;
    auto at = [&](int two) { return tile + kv8_v_off(D) + (((j >> 3) * 2 + (two >> 2)) * 8 + (j & 7)) * 64 + (two & 3) * 16; };
    if (s.less != 1.0f)
        for (int two = 0; 2 * two < off; ++two) {   // the new token's bytes, where it shares the last 16, are written below
            uint4 w = *reinterpret_cast<const uint4*>(at(two));
            w = make_uint4(less4(w.x, s.less), less4(w.y, s.less), less4(w.z, s.less), less4(w.w, s.less));
            *reinterpret_cast<uint4*>(at(two)) = w;
        }
    with_clamp(s, [&](auto clamp) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const uint32_t c = __byte_perm(code_of<clamp.value>(x[2 * q], s.inv), code_of<clamp.value>(x[2 * q + 1], s.inv), 0x0040);
            *reinterpret_cast<uint16_t*>(at(off >> 1) + 4 * q + 2 * (off & 1)) = (uint16_t)(s.inv > 0.0f ? c : 0x8080u);
        }
    });
    if (j == 0) *reinterpret_cast<float*>(tile + kv8_v_scale_off(D)) = s.now;
}

// Quantises new rows into their slots, K rotated on the way, with a scale for a tile of 16 tokens and head:
//   s = max(old, max |x| * (1 / 127)), code = clamp(rint(x * (1 / s)), -127, 127) + 128, each operation rounded,
// old being 0 where the run begins at the tile's first token; codes stored before are rounded again where s grew. Reads 4 D bytes
// a token and head and writes 2 D. A CTA's two warps look at `window` places of the list, find the runs that begin there and store
// one head's K or V of each: runs of one token several at a time, longer ones one after the other, all lanes together. A tile
// belongs to one CTA, so there is no word between CTAs and no order of theirs that shows. Bound by the latency of a tile's steps (slots,
// rows and angles, the maximum, codes): 8191 tokens of eight heads of 128, rotated, 11 us, 67% of a copy's rate (16 us with CTAs of
// eight warps, for whose last ones the GPU waits); a token each of 16 requests with 32 heads 2.3 us.
template <int D, int DTYPE, int MODE>
__global__ void __launch_bounds__(64, 16) kv8_append_kernel(const Kv8RowsParams p)
{
    __shared__ uint32_t tops[2][2];   // [run, in turns][warp]
    chained_kernel();
    const int lane = threadIdx.x & 31, half = threadIdx.x >> 5;
    const uint32_t place = blockIdx.x / (uint32_t)(2 * p.kv_heads);
    const int rest = (int)(blockIdx.x - place * (uint32_t)(2 * p.kv_heads)), head = rest >> 1;
    const long long w0 = (long long)place * p.window;
    if (w0 >= p.tokens) return;
    // lane l: place w0 - 1 + l; runs that begin in the window end 15 places past it at most
    const long long t = w0 - 1 + lane;
    const long long slot = t >= 0 && t < p.tokens ? p.slots[t] : -2;
    int pos = 0;
    if (MODE != kRopeNone && !(rest & 1) && t >= 0 && t < p.tokens) pos = p.rope.positions[t];
    const bool live = slot >= 0 && slot < p.n_slots;
    const long long before = __shfl_up_sync(kFull, slot, 1);
    const bool follows = live && (slot & 15) != 0 && before == slot - 1;
    const uint32_t chain = __ballot_sync(kFull, follows);
    uint32_t begins = __ballot_sync(kFull, live && !follows && lane >= 1 && lane <= p.window);
    // runs of one token: as many at a time as the CTA has rows of lanes
    uint32_t single = begins & ~(chain >> 1);
    begins &= ~single;
    while (single) {
        uint32_t left = single;
        for (int i = 0; i < (int)threadIdx.x / (D / 8); ++i) left &= left - 1;
        const int l = left ? __ffs(left) - 1 : 0;
        const long long s = __shfl_sync(kFull, slot, l);
        const int at = __shfl_sync(kFull, pos, l);
        if (rest & 1) store_value<D, DTYPE>(p, left != 0, s, (int)(w0 - 1 + l), head);
        else store_key<D, DTYPE, MODE>(p, left != 0, s, (int)(w0 - 1 + l), at, head);
        for (int i = 0; i < 64 / (D / 8); ++i) single &= single - 1;
    }
    for (int turn = 0; begins; turn ^= 1) {
        const int l = __ffs(begins) - 1;
        begins &= begins - 1;
        const long long s = __shfl_sync(kFull, slot, l);
        Run run;
        run.tile = tile_of(p, s, head, D);
        run.token = (int)(w0 - 1 + l);
        run.lane = l;
        run.pos = pos;
        run.off = (int)(s & 15);
        run.end = run.off + __ffs(~(l < 31 ? chain >> (l + 1) : 0u));   // itself and what follows it
        const bool whole = run.off == 0 && run.end == 16;
        if (rest & 1) {
            if (whole) store_values<D, DTYPE, true>(p, run, head, half, tops[turn]);
            else store_values<D, DTYPE, false>(p, run, head, half, tops[turn]);
        } else {
            if (whole) store_keys<D, DTYPE, MODE, true>(p, run, head, half, tops[turn]);
            else store_keys<D, DTYPE, MODE, false>(p, run, head, half, tops[turn]);
        }
    }
}

// The values that slots stand for, (code - 128) * scale in FP32, rounded once. D / 8 lanes a token and head, kRead rows of a
// lane in flight; neighbouring lanes' rows are neighbouring tokens, two of which share each 16 bytes of V's codes. Bound by the loads'
// latency and its instructions: 8191 tokens of eight heads of 128 in 9.6 us (four rows in flight 11.6, one 9.9), 80% of a copy's rate.
constexpr int kRead = 2, kReadThreads = 256;
template <int D, int DTYPE>
__global__ void __launch_bounds__(kReadThreads) kv8_read_kernel(const Kv8RowsParams p)
{
    chained_kernel();
    constexpr int kLanes = D / 8, kRows = kReadThreads / kLanes;
    const int j = threadIdx.x % kLanes;
    uint32_t w[kRead][2][2];
    float s[kRead][2];
    long long row[kRead];
#pragma unroll
    for (int r = 0; r < kRead; ++r) {
        row[r] = ((long long)blockIdx.x * kRead + r) * kRows + threadIdx.x / kLanes;
        // neighbours are tokens of one head, which share sectors; rows are below 2^32: checked on the host
        const uint32_t head = (uint32_t)row[r] / (uint32_t)p.tokens, token = (uint32_t)row[r] - head * (uint32_t)p.tokens;
        const bool live = head < (uint32_t)p.kv_heads;
        const long long slot = live ? p.slots[token] : -1;
        row[r] = live ? (long long)token * p.kv_heads + head : -1;
        w[r][0][0] = w[r][0][1] = w[r][1][0] = w[r][1][1] = 0;
        s[r][0] = s[r][1] = 0.0f;
        if (slot >= 0 && slot < p.n_slots) {
            const uint8_t* const tile = tile_of(p, slot, (int)head, D);
            const int tok = (int)slot & 15;
            const uint2 k = *reinterpret_cast<const uint2*>(tile + ((j >> 3) * 16 + tok) * 64 + 8 * (j & 7));
            const uint4 v = *reinterpret_cast<const uint4*>(tile + kv8_v_off(D) + (((j >> 3) * 2 + (tok >> 3)) * 8 + (j & 7)) * 64 +
                                                            (tok >> 1 & 3) * 16);
            const float2 both = *reinterpret_cast<const float2*>(tile + kv8_k_scale_off(D));
            s[r][0] = both.x;
            s[r][1] = both.y;
            w[r][0][0] = k.x;
            w[r][0][1] = k.y;
            const uint32_t pick = tok & 1 ? 0x7632u : 0x5410u;
            w[r][1][0] = __byte_perm(v.x, v.y, pick);
            w[r][1][1] = __byte_perm(v.z, v.w, pick);
        }
    }
#pragma unroll
    for (int r = 0; r < kRead; ++r) {
        if (row[r] < 0) continue;
        const long long at = row[r] * D + 8 * j;
#pragma unroll
        for (int o = 0; o < 2; ++o) {
            void* const out = o ? p.v_out : p.k_out;
            const uint64_t from2 = pack_f32x2(-8388736.0f, -8388736.0f), s2 = pack_f32x2(s[r][o], s[r][o]);
            float x[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) {   // 2^23 + code, exact, less 2^23 + 128
                const uint32_t four = w[r][o][e >> 1];
                unpack_f32x2(mul_f32x2(add_f32x2(pack_f32x2(__uint_as_float(__byte_perm(four, 0x4b000000u, 0x7440 | (2 * (e & 1)))),
                                                            __uint_as_float(__byte_perm(four, 0x4b000000u, 0x7441 | (2 * (e & 1))))), from2), s2),
                             x[2 * e], x[2 * e + 1]);
            }
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
    // Places of a CTA: few make long chunks slow (CTAs that find no run still take their turn), many make small batches wait for runs
    // stored one after the other. Chunks / single tokens with 4 and 16 places, D = 128, rotated: 64 tokens of 8 heads 3.2 / 2.4,
    // 5.0 / 4.7 us; 1024 5.4 / 7.1, 5.2 / 8.7; 4096 17.8 / 19.9, 7.0 / 22.1 (with one place 3.3 / 2.5, 17 / 17, 67 / 66; and single
    // tokens by the whole CTA, as longer runs are, 1024 with 4 places 16.6).
    p.window = (long long)p.tokens * p.kv_heads <= 8192 ? 4 : 16;
    const long long blocks = ((long long)p.tokens + p.window - 1) / p.window * 2 * p.kv_heads;   // below 2^28 + 2^30: rows are below 2^31, heads at most 2^29
    const bool bf = p.dtype == W4A16_BF16;
    auto* const kernel = p.head_dim == 128 ? (bf ? append_of<128, W4A16_BF16>(p.mode) : append_of<128, W4A16_FP16>(p.mode))
                                           : (bf ? append_of<64, W4A16_BF16>(p.mode) : append_of<64, W4A16_FP16>(p.mode));
    return launch_chained(kernel, (unsigned)blocks, 64, 0, 1, stream, p);
}

cudaError_t launch_kv8_read(const Kv8RowsParams& p, cudaStream_t stream)
{
    auto* kernel = p.head_dim == 128 ? kv8_read_kernel<128, W4A16_FP32> : kv8_read_kernel<64, W4A16_FP32>;
    if (p.dtype == W4A16_BF16) kernel = p.head_dim == 128 ? kv8_read_kernel<128, W4A16_BF16> : kv8_read_kernel<64, W4A16_BF16>;
    if (p.dtype == W4A16_FP16) kernel = p.head_dim == 128 ? kv8_read_kernel<128, W4A16_FP16> : kv8_read_kernel<64, W4A16_FP16>;
    const long long per = kRead * kReadThreads / (p.head_dim / 8);
    return launch_chained(kernel, (unsigned)(((long long)p.tokens * p.kv_heads + per - 1) / per), kReadThreads, 0, 1, stream, p);
}

}  // namespace w4a16
