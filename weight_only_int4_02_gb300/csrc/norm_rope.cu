// Norms of queries and keys for each head and the rotation by their positions, in one pass over the rows; and the
// rotation's table.
#include "launch.cuh"
#include "pairs.cuh"
#include "rope.cuh"
#include "w4a16.h"

#include <math_constants.h>

namespace w4a16 {
namespace {

constexpr int kWarps = 8;
constexpr int kRowsAhead = 4;   // rows of a lane group in flight

// y = x / sqrt(mean(x^2) + eps) * weight, then the rotation, rounded once; sums and factors are FP32.
// Bound by bandwidth: a row is read once and written once. A warp has one token and 32 / (D / 8) * kRowsAhead of its heads, so that
// the token's angles and the weights are loaded once for them.
template <int D, int DTYPE, int MODE>
__global__ void __launch_bounds__(kWarps * 32) norm_rope_kernel(const NormRopeParams p)
{
    chained_kernel();
    constexpr int kLanes = D / 8, kTogether = 32 / kLanes;
    const uint32_t item = blockIdx.x * kWarps + (threadIdx.x >> 5);   // below 2^31 + 8: checked on the host
    const int token = (int)(item / (uint32_t)p.groups), group = (int)(item - (uint32_t)token * (uint32_t)p.groups);
    if (token >= p.tokens) return;
    const int lane = threadIdx.x & 31, j = lane % kLanes;
    const LaneDims at = lane_dims<MODE>(j, p.rope.rot);
    const int first = group * kTogether * kRowsAhead + lane / kLanes, all = p.heads[0] + p.heads[1];

    uint2 raw[kRowsAhead][2];
#pragma unroll
    for (int i = 0; i < kRowsAhead; ++i) {
        const int h = first + i * kTogether;
        raw[i][0] = raw[i][1] = make_uint2(0, 0);
        if (h < all) {
            const int which = h >= p.heads[0], hh = which ? h - p.heads[0] : h;
            // plain loads: the outputs may be the inputs
            const uint16_t* const x = (const uint16_t*)p.x[which] + token * p.token[which] + hh * p.head[which];
            raw[i][0] = *reinterpret_cast<const uint2*>(x + at.a);
            raw[i][1] = *reinterpret_cast<const uint2*>(x + at.b);
        }
    }
    uint2 w[2][2];
#pragma unroll
    for (int o = 0; o < 2; ++o) {
        const uint16_t* const weight = (const uint16_t*)p.weight[o];
        w[o][0] = weight ? __ldg(reinterpret_cast<const uint2*>(weight + at.a)) : make_uint2(0, 0);
        w[o][1] = weight ? __ldg(reinterpret_cast<const uint2*>(weight + at.b)) : make_uint2(0, 0);
    }
    float4 cos4 = make_float4(1, 1, 1, 1), sin4 = make_float4(0, 0, 0, 0);
    bool past = false;
    if constexpr (MODE != kRopeNone) {
        const int pos = p.rope.positions[token];
        if (pos < 0) return;   // padding: its rows stay as they were
        past = pos >= p.rope.rows;
        if (!past && at.turned) {
            const float* const row = p.rope.table + (long long)pos * p.rope.rot + 4 * j;
            cos4 = __ldg(reinterpret_cast<const float4*>(row));
            // rot / 2 is a multiple of 4, so these are 16-byte aligned too
            sin4 = __ldg(reinterpret_cast<const float4*>(row + p.rope.rot / 2));
        }
    }
#pragma unroll
    for (int i = 0; i < kRowsAhead; ++i) {
        const int h = first + i * kTogether;
        const int which = h >= p.heads[0], hh = which ? h - p.heads[0] : h;
        float x[8];
        unpack2<DTYPE>(raw[i][0].x, x[0], x[1]);
        unpack2<DTYPE>(raw[i][0].y, x[2], x[3]);
        unpack2<DTYPE>(raw[i][1].x, x[4], x[5]);
        unpack2<DTYPE>(raw[i][1].y, x[6], x[7]);
        float sum = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) sum = fmaf(x[e], x[e], sum);
#pragma unroll
        for (int d = 1; d < kLanes; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        if (p.weight[which]) {
            const float r = rsqrtf(sum * (1.0f / D) + p.eps);
            const uint2 lo = which ? w[1][0] : w[0][0], hi = which ? w[1][1] : w[0][1];
            const uint32_t words[4] = {lo.x, lo.y, hi.x, hi.y};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float u, v;
                unpack2<DTYPE>(words[e], u, v);
                x[2 * e] *= r * u;
                x[2 * e + 1] *= r * v;
            }
        }
        if (MODE != kRopeNone && at.turned) rotate<MODE == kRopeNone ? kRopeHalves : MODE>(x, cos4, sin4);
        if (past) {   // a position that the table does not have: an error that shows
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = CUDART_NAN_F;
        }
        if (h < all) {
            uint16_t* const y = (uint16_t*)p.out[which] + token * p.out_token[which] + hh * p.out_head[which];
            *reinterpret_cast<uint2*>(y + at.a) = make_uint2(pack2<DTYPE>(x[0], x[1]), pack2<DTYPE>(x[2], x[3]));
            *reinterpret_cast<uint2*>(y + at.b) = make_uint2(pack2<DTYPE>(x[4], x[5]), pack2<DTYPE>(x[6], x[7]));
        }
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

cudaError_t launch_norm_rope(const NormRopeParams& in, cudaStream_t stream)
{
    NormRopeParams p = in;
    const long long rows = 32 / (p.head_dim / 8) * kRowsAhead, heads = (long long)p.heads[0] + p.heads[1];
    const long long groups = (heads + rows - 1) / rows;
    if (groups * p.tokens >= 1LL << 31) return cudaErrorInvalidValue;
    p.groups = (int)groups;
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
