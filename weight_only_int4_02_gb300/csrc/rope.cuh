// Rotation of a head's row by its position, and the operator that norms and rotates queries and keys.
//
// The table float32 [rows][rot] holds a position's rot / 2 cosines, then its sines. Of the first rot values of a row, pair i is
// (x[i], x[i + rot / 2]), or (x[2i], x[2i + 1]) where pairs are interleaved: (a, b) -> (a cos - b sin, b cos + a sin).
// D / 8 lanes hold a row, each of them two runs of four neighbours that are each other's partners: x[4j ..] and
// x[rot / 2 + 4j ..], or x[8j ..] and x[8j + 4 ..]. So no value changes lanes, and either way a lane wants the
// angles 4j .. 4j + 3: one 16-byte load of cosines and one of sines.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

namespace w4a16 {

enum RopeMode { kRopeNone = 0, kRopeHalves = 1, kRopePairs = 2 };

struct Rope {
    const int32_t* positions;    // [tokens], or null: no rotation
    const float* table;          // [rows][rot]
    int rows, rot;
};

// Where a lane's two runs of four begin; `turned`: they are rotated, by the angles from 4 j on.
struct LaneDims {
    int a, b;
    bool turned;
};

template <int MODE>
__device__ __forceinline__ LaneDims lane_dims(int j, int rot)
{
    if (MODE == kRopeHalves && j < rot / 8) return {4 * j, rot / 2 + 4 * j, true};
    return {8 * j, 8 * j + 4, MODE == kRopePairs && j < rot / 8};
}

// x[0..3] and x[4..7]: the two runs. Every product and sum is rounded by itself, so that what is quantised afterwards has the
// same codes wherever the formula is evaluated.
template <int MODE>
__device__ __forceinline__ void rotate(float (&x)[8], const float4& cos4, const float4& sin4)
{
    const float c[4] = {cos4.x, cos4.y, cos4.z, cos4.w}, s[4] = {sin4.x, sin4.y, sin4.z, sin4.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float& p = x[MODE == kRopePairs ? 2 * i : i];
        float& q = x[MODE == kRopePairs ? 2 * i + 1 : i + 4];
        const float a = __fsub_rn(__fmul_rn(p, c[i]), __fmul_rn(q, s[i]));
        q = __fadd_rn(__fmul_rn(q, c[i]), __fmul_rn(p, s[i]));
        p = a;
    }
}

struct NormRopeParams {
    const void* x[2];            // queries and keys, [tokens][heads][D] at the strides below; null: none
    void* out[2];
    const void* weight[2];       // [D], or null: no norm
    long long token[2], head[2], out_token[2], out_head[2];   // strides in elements
    Rope rope;
    float eps;
    int tokens, heads[2], head_dim, dtype, mode;
    int groups[2], passes;       // warps that a token's queries and keys take, and their passes (set by the launch)
};
cudaError_t launch_norm_rope(const NormRopeParams& p, int sms, cudaStream_t stream);
cudaError_t launch_rope_table(float* out, int rows, int rot, double base, cudaStream_t stream);

}  // namespace w4a16
