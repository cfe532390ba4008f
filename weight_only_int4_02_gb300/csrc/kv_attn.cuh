// What the attention kernels for few query rows share, whatever the cache's bits: the batch's work as one line of units dealt to
// the CTAs in equal runs, and the joining of a segment's parts.
#pragma once
#include "api_internal.cuh"
#include "kv4.cuh"
#include "ptx.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <limits.h>
#include <math_constants.h>

namespace w4a16 {

constexpr int kAttnWarps = 4;
constexpr int kAttnThreads = kAttnWarps * 32;
constexpr int kAttnGrow = 8;       // log2 of how far probabilities may grow before their reference moves

__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8(uint32_t x)
{
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float pow2i(int e) { return __int_as_float((e + 127) << 23); }   // e in -126 .. 127

__device__ __forceinline__ uint32_t half2_bits(float a, float b)
{
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ float2 bits_half2(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2*>(&w)); }

// One request as the kernel sees it: every length clamped to what the buffers hold.
struct Request {
    int seq, q0, nq, rows, tiles;   // cached tokens that the table can hold, first query token, query tokens, rows, row tiles
    int pos0;                       // the first query's position: of all cached tokens, also those past the table's columns
    int base, units;                // first cached token looked at (a multiple of UNIT), units a segment
    long long work;                 // cost of all its segments: OVERHEAD, then the units, of each
};

// A: the kernel's ROWS of a segment, UNIT cached tokens and OVERHEAD, what starting and ending a segment costs, in units.
template <class A>
__device__ __forceinline__ Request request_of(const Kv4AttnParams& p, int b)
{
    Request r;
    const long long held = (long long)p.table_cols * p.page_size;
    int s = p.seq_lens[b];
    s = s < 0 ? 0 : s;
    r.seq = s < held ? s : (int)held;
    int a = p.starts[b], e = p.starts[b + 1];
    a = a < 0 ? 0 : a > p.tokens ? p.tokens : a;
    e = e < a ? a : e > p.tokens ? p.tokens : e;
    r.q0 = a;
    r.nq = e - a;
    r.pos0 = s - r.nq;
    r.rows = r.nq * p.group;
    r.tiles = r.rows > p.few_rows ? 0 : (r.rows + A::ROWS - 1) / A::ROWS;
    // first token that a query's window holds (a query at a negative position sees nothing; none of them: no overflow
    // whatever the window)
    const int first = (r.pos0 > 0 ? r.pos0 : 0) - p.window + 1;
    r.base = (p.window > 0 && first > 0) ? first / A::UNIT * A::UNIT : 0;
    r.units = r.seq > r.base ? (r.seq - r.base + A::UNIT - 1) / A::UNIT : 1;   // an empty segment still writes its rows
    r.work = (long long)r.tiles * p.kv_heads * (r.units + A::OVERHEAD);
    return r;
}

// In shared memory beside a kernel's own.
template <int ROWS>
struct RunShared {
    float m[kAttnWarps][ROWS], l[kAttnWarps][ROWS];   // each warp's maxima and sums
    float weight[kAttnWarps][ROWS];
    long long scan[kAttnWarps];
    long long start_off, total;   // of the run, and all units
    Request start;
    int start_b, ctas, abort_flag, last;
};

// floor(total * n / of) for n up to `of`, at most kWsMaxGrid: 64-bit divisions take a warp a hundred instructions each.
__device__ __forceinline__ long long share_of(long long total, int n, int of)
{
    if (total >> 32) return total * n / of;
    const uint32_t q = (uint32_t)total / (uint32_t)of, rest = (uint32_t)total - q * (uint32_t)of;
    return (long long)q * n + rest * (uint32_t)n / (uint32_t)of;
}

// One more of a segment's parts is there: what was written before by this CTA (behind a barrier) is seen by whoever counts later.
__device__ __forceinline__ int count_part(int* counter)
{
    int before;
    asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;" : "=r"(before) : "l"(counter) : "memory");
    return before;
}

// A CTA's run of units: u0 .. u1 of all of the batch's, from `off` on in request b's. Requests without a CTA of this launch (b past
// the batch) have none. Every thread of the CTA calls it; the lengths stay on the device, so every CTA sums them by itself.
struct Units {
    long long u0, u1, off;
    int b;
    Request r;      // request b
};

template <class A>
__device__ __forceinline__ Units units_of(const Kv4AttnParams& p, typename A::Shared& sh)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    Units u = {};
    u.b = p.batch;
    long long sum = 0;
    const int per = (p.batch + kAttnThreads - 1) / kAttnThreads;
    const int bl = tid * per, bh = bl + per < p.batch ? bl + per : p.batch;
    for (int b = bl; b < bh; ++b) sum += request_of<A>(p, b).work;
    long long incl = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long o = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += o;
    }
    if (lane == 31) sh.scan[warp] = incl;
    if (tid == 0) {
        sh.abort_flag = 0;
        sh.start_b = p.batch;
    }
    __syncthreads();
    long long excl = incl - sum, total = 0;
#pragma unroll
    for (int w = 0; w < kAttnWarps; ++w) {
        if (w < warp) excl += sh.scan[w];
        total += sh.scan[w];
    }
    // as many CTAs as give each warp a unit (two, where there are few: a request of 1000 tokens over 4 bits 9.9 -> 12.0 us)
    const long long want = (total + kAttnWarps - 1) / kAttnWarps;
    const int ctas = (int)(want < gridDim.x ? want : gridDim.x);
    if ((int)blockIdx.x >= ctas) return u;
    if (tid == 0) {
        sh.total = total;
        sh.ctas = ctas;
    }
    u.u0 = share_of(total, blockIdx.x, ctas), u.u1 = share_of(total, blockIdx.x + 1, ctas);
    if (u.u0 >= excl && u.u0 < excl + sum) {
        long long at = excl;
        for (int b = bl; b < bh; ++b) {
            const Request r = request_of<A>(p, b);
            if (u.u0 < at + r.work) {
                sh.start_b = b;
                sh.start_off = u.u0 - at;
                sh.start = r;
                break;
            }
            at += r.work;
        }
    }
    __syncthreads();
    u.b = sh.start_b;
    u.off = sh.start_off;
    u.r = sh.start;
    return u;
}

// The end of a segment's share: the warps' outputs, each in its own ring [row][D], their maxima and sums in sh, are joined; a whole
// segment's rows are written, and of a segment cut by a run's end the last CTA to arrive joins the parts, in the CTAs' order.
// pos, take: the share's first unit and its units; seg_u: the segment's place among all.
template <class A>
__device__ __forceinline__ void finish_segment(const Kv4AttnParams& p, uint8_t* smem, typename A::Shared& sh, const Request& r, int head, int row0,
                                               int pos, int take, long long seg_u)
{
    constexpr int ROWS = A::ROWS, D = A::DIM;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    __syncthreads();
    const int live = r.rows - row0 < ROWS ? r.rows - row0 : ROWS;
    const bool whole = pos == 0 && take == r.units;
    // joined maximum, sum and the warps' weights of each row
    float* const part = p.partials + (long long)(2 * blockIdx.x + (pos == 0 ? 1 : 0)) * A::PART;
    if (tid < live) {
        float mm = -CUDART_INF_F, ll = 0.0f;
#pragma unroll
        for (int w = 0; w < kAttnWarps; ++w) mm = fmaxf(mm, sh.m[w][tid]);
#pragma unroll
        for (int w = 0; w < kAttnWarps; ++w) {
            const float f = sh.m[w][tid] == mm ? 1.0f : ex2(sh.m[w][tid] - mm);
            ll += sh.l[w][tid] * f;
            sh.weight[w][tid] = f;
        }
        if (whole) {
            const float inv = ll == 0.0f ? 0.0f : 1.0f / ll;
#pragma unroll
            for (int w = 0; w < kAttnWarps; ++w) sh.weight[w][tid] *= inv;
            if (p.lse) {
                const int rr = row0 + tid, qi = rr / p.group;
                p.lse[(long long)(r.q0 + qi) * p.q_heads + head * p.group + rr - qi * p.group] =
                    ll == 0.0f ? -CUDART_INF_F : (mm + log2f(ll)) * CUDART_LN2_F;
            }
        } else {
            __stcg(part + ROWS * D + tid, mm);
            __stcg(part + ROWS * D + ROWS + tid, ll);
        }
    }
    __syncthreads();
    auto store_row = [&](int row, int d, const float4& x) {
        const int rr = row0 + row, qi = rr / p.group;
        uint16_t* dst = (uint16_t*)p.out + (long long)(r.q0 + qi) * p.o_token +
                        (long long)(head * p.group + rr - qi * p.group) * p.o_head + d;
        uint2 w;
        if (p.bf16) {
            const __nv_bfloat162 a = __floats2bfloat162_rn(x.x, x.y), bb = __floats2bfloat162_rn(x.z, x.w);
            w = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&bb));
        } else {
            w = make_uint2(half2_bits(x.x, x.y), half2_bits(x.z, x.w));
        }
        *reinterpret_cast<uint2*>(dst) = w;
    };
    for (int i = tid; i < live * (D / 4); i += kAttnThreads) {
        const int row = i / (D / 4), d = i % (D / 4) * 4;
        float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int w = 0; w < kAttnWarps; ++w) {
            const float f = sh.weight[w][row];
            const float4 y = *reinterpret_cast<const float4*>(smem + w * A::RING + (row * D + d) * 4);
            x.x += f * y.x;
            x.y += f * y.y;
            x.z += f * y.z;
            x.w += f * y.w;
        }
        if (whole) store_row(row, d, x);
        else __stcg(reinterpret_cast<float4*>(part + row * D + d), x);
    }
    if (!whole) {
        // ---- the last CTA of the segment to arrive joins the partial results, in the CTAs' order
        const long long g0 = seg_u + A::OVERHEAD;   // the place of the segment's first unit
        const long long total = sh.total;
        const int ctas = sh.ctas;
        const int ca = (int)(((g0 + 1) * ctas - 1) / total), cb = (int)(((g0 + r.units) * ctas - 1) / total);
        __syncthreads();
        if (tid == 0) {
            sh.last = count_part(p.counters + ca) == cb - ca;
            if (sh.last) p.counters[ca] = 0;   // ready for the next launch
        }
        __syncthreads();
        if (sh.last) {
            // every part's weight, kept where the rings were, then the sums
            const int parts = cb - ca + 1;
            float* const wt = reinterpret_cast<float*>(smem);
            const float* const first = p.partials + (long long)(2 * ca) * A::PART;   // the first CTA's last part, the others' first
            auto part_of = [&](int k) { return first + (2 * k + (k == 0)) * A::PART; };
            for (int row = warp; row < live; row += kAttnWarps) {
                float mm = -CUDART_INF_F, ll = 0.0f;
                // a lane's first parts stay in registers: their maxima and sums are loaded together
                constexpr int kMine = 4;
                float mk[kMine], lk[kMine];
#pragma unroll
                for (int j = 0; j < kMine; ++j) {
                    const int k = lane + 32 * j;
                    mk[j] = k < parts ? __ldcg(part_of(k) + ROWS * D + row) : -CUDART_INF_F;
                    lk[j] = k < parts ? __ldcg(part_of(k) + ROWS * D + ROWS + row) : 0.0f;
                    mm = fmaxf(mm, mk[j]);
                }
                for (int k = lane + 32 * kMine; k < parts; k += 32) mm = fmaxf(mm, __ldcg(part_of(k) + ROWS * D + row));
#pragma unroll
                for (int d = 16; d > 0; d >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, d));
                auto weigh = [&](int k, float m_k, float l_k) {
                    const float f = m_k == mm ? 1.0f : ex2(m_k - mm);
                    wt[k * live + row] = f;
                    ll += f * l_k;
                };
#pragma unroll
                for (int j = 0; j < kMine; ++j)
                    if (lane + 32 * j < parts) weigh(lane + 32 * j, mk[j], lk[j]);
                for (int k = lane + 32 * kMine; k < parts; k += 32)
                    weigh(k, __ldcg(part_of(k) + ROWS * D + row), __ldcg(part_of(k) + ROWS * D + ROWS + row));
#pragma unroll
                for (int d = 16; d > 0; d >>= 1) ll += __shfl_xor_sync(0xffffffffu, ll, d);
                if (lane == 0) {
                    sh.l[0][row] = ll == 0.0f ? 0.0f : 1.0f / ll;
                    if (p.lse) {
                        const int rr = row0 + row, qi = rr / p.group;
                        p.lse[(long long)(r.q0 + qi) * p.q_heads + head * p.group + rr - qi * p.group] =
                            ll == 0.0f ? -CUDART_INF_F : (mm + log2f(ll)) * CUDART_LN2_F;
                    }
                }
            }
            __syncthreads();
            for (int i = tid; i < live * (D / 4); i += kAttnThreads) {
                const int row = i / (D / 4), d = i % (D / 4) * 4;
                float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                const float* const at = first + row * D + d;
                for (int k0 = 0; k0 < parts; k0 += A::JOIN) {   // JOIN parts' loads together; past the last part they count nothing
                    float4 y[A::JOIN];
#pragma unroll
                    for (int k = 0; k < A::JOIN; ++k) {
                        const int part = k0 + k < parts ? k0 + k : parts - 1;
                        y[k] = __ldcg(reinterpret_cast<const float4*>(at + (2 * part + (part == 0)) * A::PART));
                    }
#pragma unroll
                    for (int k = 0; k < A::JOIN; ++k) {
                        const float f = k0 + k < parts ? wt[(k0 + k) * live + row] : 0.0f;
                        x.x += f * y[k].x;
                        x.y += f * y[k].y;
                        x.z += f * y[k].z;
                        x.w += f * y[k].w;
                    }
                }
                const float inv = sh.l[0][row];
                store_row(row, d, make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv));
            }
        }
    }
    // the rings are read: bulk copies may follow the plain accesses
    fence_proxy_async_smem();
    __syncthreads();
}

}  // namespace w4a16
