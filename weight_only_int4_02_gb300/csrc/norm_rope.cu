// Norms of queries and keys for each head and the rotation by their positions, in one pass over the rows; and the
// rotation's table.
#include "launch.cuh"
#include "pairs.cuh"
#include "rope.cuh"
#include "w4a16.h"

#include <math_constants.h>

namespace w4a16 {
namespace {

constexpr int kWarps = 2;       // of a CTA: larger ones leave the GPU waiting for their last warps (eight 54.6 us where two took 52.0, as below)
constexpr int kRowsAhead = 4;   // rows of a lane group that are loaded together
constexpr int kMostPasses = 4;

// Four neighbours as two pairs.
struct Four {
    uint64_t a, b;
};

template <int DTYPE>
__device__ __forceinline__ Four four_of(const uint2& w)
{
    float x[4];
    unpack2<DTYPE>(w.x, x[0], x[1]);
    unpack2<DTYPE>(w.y, x[2], x[3]);
    return {pack_f32x2(x[0], x[1]), pack_f32x2(x[2], x[3])};
}

__device__ __forceinline__ Four four_of(const float4& v) { return {pack_f32x2(v.x, v.y), pack_f32x2(v.z, v.w)}; }
__device__ __forceinline__ Four operator*(const Four& x, const Four& y) { return {mul_f32x2(x.a, y.a), mul_f32x2(x.b, y.b)}; }
__device__ __forceinline__ Four operator*(const Four& x, uint64_t f) { return {mul_f32x2(x.a, f), mul_f32x2(x.b, f)}; }
__device__ __forceinline__ Four fma4(const Four& x, const Four& y, const Four& z) { return {fma_f32x2(x.a, y.a, z.a), fma_f32x2(x.b, y.b, z.b)}; }

template <int DTYPE>
__device__ __forceinline__ uint2 packed(const Four& x)
{
    float v[4];
    unpack_f32x2(x.a, v[0], v[1]);
    unpack_f32x2(x.b, v[2], v[3]);
    return make_uint2(pack2<DTYPE>(v[0], v[1]), pack2<DTYPE>(v[2], v[3]));
}

// Neighbours in each pair swapped.
__device__ __forceinline__ uint64_t swapped(uint64_t v)
{
    float a, b;
    unpack_f32x2(v, a, b);
    return pack_f32x2(b, a);
}

// y = x / sqrt(mean(x^2) + eps) * weight, then the rotation, rounded once; sums and factors are FP32. With the weights w and the
// angles of a token fixed, a row's outputs are r (x A + x' B), x' the partners and r = 1 / sqrt(mean(x^2) + eps), with A = w cos
// and B = -+ w' sin. A warp has one token and some of its query or key heads, so that A and B are made once for them,
// takes them in passes of which the next one's rows are on their way, and works on pairs of numbers. Bound by bandwidth: a row
// is read once and written once. 8191 tokens of 64 and 8 heads of 128: 50.8 us, 6.0 TB/s, 89% of a copy's rate; with scalar arithmetic
// and one pass 67. 16 tokens of 40 heads take 2.4 us. Fourteen CTAs an SM leave 72 registers, of which the forms that rotate want a few more (8 to 24
// bytes spilled): sixteen, with 64, spilled 52 to 92 and took 51.8; twelve spill none, 52.7 (1003 tokens of 32 heads of 64, 32 of them
// turned: 3.8, 4.4 and 3.4 us).
template <int D, int DTYPE, int MODE>
__global__ void __launch_bounds__(kWarps * 32, 14) norm_rope_kernel(const NormRopeParams p)
{
    chained_kernel();
    constexpr int kLanes = D / 8, kTogether = 32 / kLanes;
    const uint32_t item = blockIdx.x * kWarps + (threadIdx.x >> 5);   // below 2^31 + 8: checked on the host
    const int all = p.groups[0] + p.groups[1];
    const int token = (int)(item / (uint32_t)all), group = (int)(item - (uint32_t)token * (uint32_t)all);
    if (token >= p.tokens) return;
    const int which = group >= p.groups[0];
    const int lane = threadIdx.x & 31, j = lane % kLanes;
    const LaneDims at = lane_dims<MODE>(j, p.rope.rot);
    const int heads = which ? p.heads[1] : p.heads[0];
    constexpr int kPass = kTogether * kRowsAhead;   // heads of a pass
    int h = (which ? group - p.groups[0] : group) * kPass * p.passes + lane / kLanes;
    const int end = min(heads, h - lane / kLanes + kPass * p.passes);
    // plain loads: the outputs may be the inputs
    const long long step = (which ? p.head[1] : p.head[0]) * kTogether;
    const uint16_t* x = (const uint16_t*)(which ? p.x[1] : p.x[0]) + token * (which ? p.token[1] : p.token[0]) +
                        h * (which ? p.head[1] : p.head[0]);
    uint2 raw[kRowsAhead][2];
    auto load = [&](int from) {
#pragma unroll
        for (int i = 0; i < kRowsAhead; ++i) {
            raw[i][0] = raw[i][1] = make_uint2(0, 0);
            if (from + i * kTogether < end) {
                raw[i][0] = *reinterpret_cast<const uint2*>(x + at.a);
                raw[i][1] = *reinterpret_cast<const uint2*>(x + at.b);
            }
            x += step;
        }
    };
    load(h);
    const uint16_t* const weight = (const uint16_t*)(which ? p.weight[1] : p.weight[0]);
    const uint64_t one = pack_f32x2(1.0f, 1.0f);
    Four w[2] = {{one, one}, {one, one}};
    if (weight) {
        w[0] = four_of<DTYPE>(__ldg(reinterpret_cast<const uint2*>(weight + at.a)));
        w[1] = four_of<DTYPE>(__ldg(reinterpret_cast<const uint2*>(weight + at.b)));
    }
    Four A[2] = {w[0], w[1]}, B[2] = {{0, 0}, {0, 0}};
    if constexpr (MODE != kRopeNone) {
        const int pos = p.rope.positions[token];
        if (pos < 0) return;   // padding: its rows stay as they were
        if (pos >= p.rope.rows) {   // an error that shows
            const uint64_t nan = pack_f32x2(CUDART_NAN_F, CUDART_NAN_F);
            A[0] = A[1] = {nan, nan};
        } else if (at.turned) {
            const float* const row = p.rope.table + (long long)pos * p.rope.rot + 4 * j;
            const float4 c = __ldg(reinterpret_cast<const float4*>(row));
            // rot / 2 is a multiple of 4, so these are 16-byte aligned too
            const float4 s = __ldg(reinterpret_cast<const float4*>(row + p.rope.rot / 2));
            if constexpr (MODE == kRopeHalves) {
                const Four cos4 = four_of(c), sin4 = four_of(s);
                A[0] = w[0] * cos4;
                A[1] = w[1] * cos4;
                B[0] = w[1] * sin4 * pack_f32x2(-1.0f, -1.0f);
                B[1] = w[0] * sin4;
            } else {
                const Four cos4[2] = {{pack_f32x2(c.x, c.x), pack_f32x2(c.y, c.y)}, {pack_f32x2(c.z, c.z), pack_f32x2(c.w, c.w)}};
                const Four sin4[2] = {{pack_f32x2(-s.x, s.x), pack_f32x2(-s.y, s.y)}, {pack_f32x2(-s.z, s.z), pack_f32x2(-s.w, s.w)}};
#pragma unroll
                for (int o = 0; o < 2; ++o) {
                    A[o] = w[o] * cos4[o];
                    B[o] = Four{swapped(w[o].a), swapped(w[o].b)} * sin4[o];
                }
            }
        }
    }
    const long long out_step = (which ? p.out_head[1] : p.out_head[0]) * kTogether;
    uint16_t* y = (uint16_t*)(which ? p.out[1] : p.out[0]) + token * (which ? p.out_token[1] : p.out_token[0]) +
                  h * (which ? p.out_head[1] : p.out_head[0]);
#pragma unroll 1
    for (;;) {
        uint2 now[kRowsAhead][2];
#pragma unroll
        for (int i = 0; i < kRowsAhead; ++i) {
            now[i][0] = raw[i][0];
            now[i][1] = raw[i][1];
        }
        const bool more = h - lane / kLanes + kPass < end;   // the same for the whole warp
        if (more) load(h + kPass);
#pragma unroll
        for (int i = 0; i < kRowsAhead; ++i) {
            const Four u = four_of<DTYPE>(now[i][0]), v = four_of<DTYPE>(now[i][1]);
            uint64_t r2 = one;
            if (weight) {
                float s0, s1;
                unpack_f32x2(fma_f32x2(v.b, v.b, fma_f32x2(v.a, v.a, fma_f32x2(u.b, u.b, mul_f32x2(u.a, u.a)))), s0, s1);
                float sum = s0 + s1;
#pragma unroll
                for (int d = 1; d < kLanes; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
                const float r = rsqrtf(sum * (1.0f / D) + p.eps);
                r2 = pack_f32x2(r, r);
            }
            Four lo = u * A[0], hi = v * A[1];
            if (MODE != kRopeNone && at.turned) {   // what is not turned has no partner, whose infinity times 0 would show
                lo = fma4(MODE == kRopeHalves ? v : Four{swapped(u.a), swapped(u.b)}, B[0], lo);
                hi = fma4(MODE == kRopeHalves ? u : Four{swapped(v.a), swapped(v.b)}, B[1], hi);
            }
            if (h + i * kTogether < end) {
                *reinterpret_cast<uint2*>(y + at.a) = packed<DTYPE>(lo * r2);
                *reinterpret_cast<uint2*>(y + at.b) = packed<DTYPE>(hi * r2);
            }
            y += out_step;
        }
        if (!more) break;
        h += kPass;
    }
}

// cos and sin of p * base^(-2i / rot), in 64 bits (angles of far positions lose their fraction in 32), rounded once. Made once for
// a model.
__global__ void __launch_bounds__(256) rope_table_kernel(float* out, int rows, int rot, double base)
{
    chained_kernel();
    const long long n = (long long)rows * (rot / 2), step = (long long)gridDim.x * blockDim.x;
    for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += step) {
        const long long row = i / (rot / 2);
        const int k = (int)(i - row * (rot / 2));
        double s, c;
        sincos((double)row * pow(base, -2.0 * k / rot), &s, &c);
        out[row * rot + k] = (float)c;
        out[row * rot + rot / 2 + k] = (float)s;
    }
}

template <int D, int DTYPE>
auto* kernel_of(int mode)
{
    return mode == kRopeNone ? norm_rope_kernel<D, DTYPE, kRopeNone>
                             : mode == kRopeHalves ? norm_rope_kernel<D, DTYPE, kRopeHalves> : norm_rope_kernel<D, DTYPE, kRopePairs>;
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeParams& in, int sms, cudaStream_t stream)
{
    NormRopeParams p = in;
    // More passes a warp where that leaves enough warps, three times what an SM holds: A and B cost as much as a pass (8191 tokens
    // of 64 and 8 heads of 128, in CTAs of eight warps: one pass 68.9 us, two 57.4, four 55.3, eight 55.3).
    const long long pass = 32 / (p.head_dim / 8) * kRowsAhead;
    auto groups_of = [&](int i) { return (p.heads[i] + pass * p.passes - 1) / (pass * p.passes); };
    long long groups = 0;
    for (p.passes = kMostPasses; ; p.passes /= 2) {
        groups = groups_of(0) + groups_of(1);
        if (p.passes == 1 || groups * p.tokens >= 96LL * sms) break;
    }
    for (int i = 0; i < 2; ++i) p.groups[i] = (int)groups_of(i);
    if (groups * p.tokens >= 1LL << 31) return cudaErrorInvalidValue;
    const unsigned blocks = (unsigned)((groups * p.tokens + kWarps - 1) / kWarps);
    const bool bf = p.dtype == W4A16_BF16;
    auto* const kernel = p.head_dim == 128 ? (bf ? kernel_of<128, W4A16_BF16>(p.mode) : kernel_of<128, W4A16_FP16>(p.mode))
                                           : (bf ? kernel_of<64, W4A16_BF16>(p.mode) : kernel_of<64, W4A16_FP16>(p.mode));
    return launch_chained(kernel, blocks, kWarps * 32, 0, 1, stream, p);
}

cudaError_t launch_rope_table(float* out, int rows, int rot, double base, cudaStream_t stream)
{
    const long long n = (long long)rows * (rot / 2), blocks = (n + 255) / 256;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(blocks < 4096 ? blocks : 4096));
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, rope_table_kernel, out, rows, rot, base);
}

}  // namespace w4a16
