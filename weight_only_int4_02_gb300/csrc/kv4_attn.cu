// Attention over the 4-bit paged cache for few query rows (a decode step, drafted
// tokens): O = softmax(scale * Q K^T) V with K, V = (code - zero) * scale.
//
// A segment is one request's KV head and up to 8 NR rows, or four (query token, query head of
// the group); its cached tokens are cut into units of 32, and the units of all segments,
// laid end to end, are dealt to the CTAs in equal runs (stream-K), so ragged lengths, one
// long request and a thousand short ones fill the GPU alike. The lengths stay on the
// device: every CTA sums them by itself. A segment cut by a run's end is joined through
// the workspace by the last of its CTAs to arrive, in the CTAs' order.
//
// In a CTA, four warps take a run's units in turn, each with its own ring of bulk copies
// and barriers (no CTA barrier in the loop), and keep their own running maximum, sum and
// output. Mathematics, with c the code, z the zero-point, s the scale of a token:
//   score = s_k (q . c_k - z_k sum(q)) * scale,   out = sum_t p_t s_v (c_v - z_v) / sum_t p_t
// so the MMAs multiply by the bare codes: an unpacked register is one logic operation (two
// codes as binary16 subnormals, exact), K's scale and zero-point act on scores and V's scale on
// probabilities, once a (token, row). V's zero-points are taken off the running sums unit by unit, from MMAs of their
// own: an MMA rounds towards zero, and in sums of codes alone, some hundred times what is left of them in
// the end, these roundings added up (over 2^20 tokens to 0.8% of the output, 0.1% for 128 requests of 16384; now
// nothing beside a binary16 output's rounding, for 4% of the time). Tokens are the MMA's M for K (A = 16 tokens x
// 16 d) and d is for V (A = 16 d x 16 tokens), so that eight rows are the MMA's N and cost
// eight columns. Q is scaled per row by a power of two into binary16's range (exact
// for binary16 and bfloat16 inputs). Probabilities times V's scale are fed as a high
// and a low binary16 part, 22 bits: one part alone would add a rounding as large as that of
// a binary16 output, for 5% of the time (62.8 us against 66.3 below). Where four rows are enough they stand twice
// in the eight columns: the second four's lanes, which know the same probabilities, feed the low parts, so
// that V takes half the MMAs (one request of 131072 tokens 43.2 -> 42.3 us). Scores, sums, maxima and outputs
// are FP32.
//
// Measured, D = 128: 64 requests of 257 to 16384 cached tokens 71 us, 3.6 TB/s, 53% of a copy's rate; one of
// 131072 tokens 44 us; D = 64, 48 requests of 1 to 5 drafted tokens and a window of 4096 17.6 us; one of 1000
// tokens 10.9 us, most of it latency. Four CTAs an SM (128 registers a thread) keep the issue slots busy for 52% of the
// time and the tensor pipe for 33%: a unit is about 640 warp instructions (the integer pipe is busy
// for 47%), which wait for one another more than for memory. Eight or two warps a CTA, five CTAs an SM
// (fewer registers) and tokens' scales through shared memory were slower.
#include "api_internal.cuh"
#include "kv4.cuh"
#include "launch.cuh"
#include "ptx.cuh"

#include <float.h>
#include <limits.h>
#include <math_constants.h>

namespace w4a16 {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kUnit = 32;      // tokens of a unit: two tiles
constexpr int kOverhead = 12;  // what starting and ending a segment costs, in units
constexpr int kGrow = 8;       // log2 of how far probabilities may grow before their reference moves
constexpr uint32_t kLow = 0x000f000fu, kHigh = 0x00f000f0u;

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
    int base, units;                // first cached token looked at (a multiple of kUnit), units a segment
    long long work;                 // cost of all its segments: kOverhead, then the units, of each
};

template <int ROWS>
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
    r.tiles = r.rows > p.few_rows ? 0 : (r.rows + ROWS - 1) / ROWS;
    // first token that a query's window holds (a query at a negative position sees nothing; none of them: no overflow
    // whatever the window)
    const int first = (r.pos0 > 0 ? r.pos0 : 0) - p.window + 1;
    r.base = (p.window > 0 && first > 0) ? first / kUnit * kUnit : 0;
    r.units = r.seq > r.base ? (r.seq - r.base + kUnit - 1) / kUnit : 1;   // an empty segment still writes its rows
    r.work = (long long)r.tiles * p.kv_heads * (r.units + kOverhead);
    return r;
}

template <int D, int NR>
struct Attn {
    static constexpr bool FOUR = NR == 0;       // four rows, twice in an MMA's eight columns
    static constexpr int G = FOUR ? 1 : NR;     // columns, in eights
    static constexpr int ROWS = FOUR ? 4 : 8 * NR;
    static constexpr int CTAS = NR <= 1 ? 4 : D == 64 ? 3 : 2;   // on an SM, as registers and rings allow
    static constexpr int STAGES = D == 128 ? 3 : 4;   // units in flight per warp
    static constexpr int TB = kv4_tile_bytes(D);
    static constexpr int STAGE = 2 * TB;
    static constexpr int RING = STAGES * STAGE;
    static constexpr int W = D / 32;            // words of a lane's share
    static constexpr int PART = ROWS * (D + 2); // floats of one partial: O, then m and l
    static_assert(RING >= ROWS * D * 4, "a warp's ring holds its output");
    struct Shared {
        uint64_t bar[kWarps][STAGES];
        float m[kWarps][ROWS], l[kWarps][ROWS];
        float weight[kWarps][ROWS];
        long long scan[kWarps];
        long long start_off;
        int start_b, abort_flag, last;
    };
    static constexpr int SMEM = kWarps * RING + sizeof(Shared);
};

template <int W>
__device__ __forceinline__ void lds_share(const uint8_t* at, uint32_t (&w)[W])
{
    if constexpr (W == 4) {
        const uint4 v = *reinterpret_cast<const uint4*>(at);
        w[0] = v.x;
        w[1] = v.y;
        w[2] = v.z;
        w[3] = v.w;
    } else {
        const uint2 v = *reinterpret_cast<const uint2*>(at);
        w[0] = v.x;
        w[1] = v.y;
    }
}

template <int D, int NR>
__global__ void __launch_bounds__(kThreads, Attn<D, NR>::CTAS) kv4_attn_kernel(const Kv4AttnParams p)
{
    using A = Attn<D, NR>;
    constexpr int W = A::W, ROWS = A::ROWS, G = A::G;
    constexpr bool FOUR = A::FOUR;
    extern __shared__ __align__(128) uint8_t smem[];
    typename A::Shared& sh = *reinterpret_cast<typename A::Shared*>(smem + kWarps * A::RING);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int n = lane >> 2, c = lane & 3;
    uint8_t* const ring = smem + warp * A::RING;
    chained_kernel();

    // ---- this CTA's run of units
    long long sum = 0;
    const int per = (p.batch + kThreads - 1) / kThreads;
    const int bl = tid * per, bh = bl + per < p.batch ? bl + per : p.batch;
    for (int b = bl; b < bh; ++b) sum += request_of<ROWS>(p, b).work;
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
    if (lane < A::STAGES) mbar_init(smem_addr(&sh.bar[warp][lane]), 1);
    fence_mbar_init();
    __syncthreads();
    long long excl = incl - sum, total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) excl += sh.scan[w];
        total += sh.scan[w];
    }
    // as many CTAs as give each warp a unit
    const long long want = (total + kWarps - 1) / kWarps;
    const long long ctas = want < gridDim.x ? want : gridDim.x;
    if (blockIdx.x >= ctas) return;
    const long long u0 = total * blockIdx.x / ctas, u1 = total * (blockIdx.x + 1) / ctas;
    if (u0 >= excl && u0 < excl + sum) {
        long long at = excl;
        for (int b = bl; b < bh; ++b) {
            const long long w = request_of<ROWS>(p, b).work;
            if (u0 < at + w) {
                sh.start_b = b;
                sh.start_off = u0 - at;
                break;
            }
            at += w;
        }
    }
    __syncthreads();
    int b = sh.start_b;
    long long off = sh.start_off;
    if (b >= p.batch) return;   // cannot happen: u0 < total

    const WaitCtl ctl{&sh.abort_flag, p.status, p.wait_limit_ns};
    // the ring: stage and phase of the next unit to issue and to use; two bits a stage: tiles present
    int s_issue = 0, s_use = 0;
    uint32_t phase = 0, pending = 0, ok_bits = 0;
    bool dead = false;
    const int tpp_shift = __ffs(p.page_size) - 5;   // log2(tiles per page)

    Request r = request_of<ROWS>(p, b);
    for (long long u = u0; u < u1;) {
        while (off >= r.work) {   // next request with work
            off -= r.work;
            r = request_of<ROWS>(p, ++b);
        }
        const int cost = r.units + kOverhead;
        const long long seg = off / cost;
        const int at = (int)(off - seg * cost);                                  // this run's first place in the segment
        const int end = (int)(cost - at < u1 - u ? cost : at + (u1 - u));        // and its end
        const long long seg_u = u - at;                                          // the segment's place among all
        u += end - at;
        off += end - at;
        if (end <= kOverhead) continue;                                          // no unit of it is this run's
        const int pos = at > kOverhead ? at - kOverhead : 0, take = end - kOverhead - pos;
        const int head = (int)(seg / r.tiles), rt = (int)(seg - (long long)head * r.tiles);
        const int row0 = rt * ROWS;
        // a unit needs no mask if it lies below the first row's position and inside the last row's window;
        // units that no row of the tile sees are left out: [first, last) of the run are looked at
        const int last_row = (row0 + ROWS < r.rows ? row0 + ROWS : r.rows) - 1;
        const int pos_min = r.pos0 + row0 / p.group, pos_max = r.pos0 + last_row / p.group;
        const int seen = pos_max >= r.base ? (pos_max - r.base) / kUnit + 1 : 0;
        const int low_at = (pos_min > 0 ? pos_min : 0) - p.window + 1;   // as in request_of
        const int low = p.window > 0 && low_at > r.base ? (low_at - r.base) / kUnit : 0;
        const int first = low > pos ? low : pos, last = seen < pos + take ? seen : pos + take;

        // ---- copies: a batch of 16 units at a time, lanes 2j and 2j + 1 own the tiles of its unit j
        const int32_t* const trow = p.table + (long long)b * p.table_stride;
        const int mine_n = last > first + warp ? (last - first - warp + kWarps - 1) / kWarps : 0;   // units of this warp: first + warp, + kWarps, ...
        auto page_of = [&](int k) {   // page of this lane's tile of the batch from unit k on, or -1
            const int t = first + warp + (k + (lane >> 1)) * kWarps;
            const int tile = ((r.base + t * kUnit) >> 4) + (lane & 1);
            return (k + (lane >> 1) < mine_n && tile * kKv4Tile < r.seq) ? trow[tile >> tpp_shift] : -1;
        };
        int k_issue = 0, page = page_of(0);
        uint32_t present = 0;
        const uint8_t* src = nullptr;
        uint32_t len = 0;
        auto issue_next = [&]() {
            if (k_issue >= mine_n || dead) return;
            const int j = k_issue & 15;
            if (j == 0) {
                const int t = first + warp + (k_issue + (lane >> 1)) * kWarps;
                const int in_page = (((r.base + t * kUnit) >> 4) + (lane & 1)) & ((1 << tpp_shift) - 1);
                const bool ok = page >= 0 && page < p.pages;
                present = __ballot_sync(0xffffffffu, ok);
                const int other = __shfl_xor_sync(0xffffffffu, page, 1);
                // a unit's two tiles in one page are one copy, the even lane's
                const bool pair = (present >> (lane & 30) & 3u) == 3u && other == page && (in_page | 1) < (1 << tpp_shift);
                len = !ok ? 0u : !pair ? (uint32_t)A::TB : (lane & 1) ? 0u : (uint32_t)A::STAGE;
                src = p.cache + ((((long long)page * p.kv_heads + head) << tpp_shift) + in_page) * A::TB;
                page = page_of(k_issue + 16);
            }
            const uint32_t bits = present >> (2 * j) & 3u;
            ok_bits = (ok_bits & ~(3u << (2 * s_issue))) | bits << (2 * s_issue);
            const uint32_t bar = smem_addr(&sh.bar[warp][s_issue]);
            if (lane == 0) mbar_arrive_expect_tx(bar, __popc(bits) * A::TB);
            if ((lane >> 1) == j && len) bulk_load(smem_addr(ring + s_issue * A::STAGE + (lane & 1) * A::TB), src, len, bar);
            ++k_issue;
            ++pending;
            s_issue = s_issue + 1 == A::STAGES ? 0 : s_issue + 1;
        };
        auto next_stage = [&]() {
            --pending;
            if (++s_use == A::STAGES) {
                s_use = 0;
                phase ^= 1;
            }
        };
#pragma unroll 1
        for (int i = 0; i < A::STAGES; ++i) issue_next();

        // ---- Q fragments, scaled per row by a power of two; row constants of the columns 2c, 2c + 1
        uint32_t ql[G][W][2], qh[G][W][2];
        float row_a[G][2], row_z[G][2];   // score = row_a * s_k * (MMA + z_k * row_z), in powers of two
        int row_pos[G][2];
#pragma unroll
        for (int g = 0; g < G; ++g) {
            const int row = row0 + g * 8 + (FOUR ? n & 3 : n);
            uint32_t raw[4 * W];
#pragma unroll
            for (int i = 0; i < 4 * W; ++i) raw[i] = 0;
            if (row < r.rows) {
                const int qi = row / p.group, h = row - qi * p.group;
                const uint16_t* q = (const uint16_t*)p.q + (long long)(r.q0 + qi) * p.q_token +
                                    (long long)(head * p.group + h) * p.q_head + c * (D / 4);
#pragma unroll
                for (int i = 0; i < W; ++i) {
                    const uint4 v = *reinterpret_cast<const uint4*>(q + 8 * i);
                    raw[4 * i] = v.x;
                    raw[4 * i + 1] = v.y;
                    raw[4 * i + 2] = v.z;
                    raw[4 * i + 3] = v.w;
                }
            }
            auto lo_of = [&](uint32_t x) { return p.bf16 ? __uint_as_float(x << 16) : bits_half2(x).x; };
            auto hi_of = [&](uint32_t x) { return p.bf16 ? __uint_as_float(x & 0xffff0000u) : bits_half2(x).y; };
            float top = 0.0f;
#pragma unroll
            for (int i = 0; i < 4 * W; ++i) top = fmaxf(top, fmaxf(fabsf(lo_of(raw[i])), fabsf(hi_of(raw[i]))));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            // largest magnitude into [2^13, 2^14); an infinity or a NaN stays one
            int e = ((__float_as_int(top) >> 23) & 255) - 127 - 13;
            e = (top == 0.0f || !(top <= FLT_MAX)) ? 0 : e < -120 ? -120 : e;
            // a negative softmax scale goes into Q, so that the largest score is that of the largest product
            const float f = p.scale_log2 < 0.0f ? -pow2i(-e) : pow2i(-e);
            float qsum = 0.0f;
#pragma unroll
            for (int w = 0; w < W; ++w) {
                float x[8];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x[2 * i] = lo_of(raw[4 * w + i]) * f;
                    x[2 * i + 1] = hi_of(raw[4 * w + i]) * f;
                }
                ql[g][w][0] = half2_bits(x[0], x[4]);
                ql[g][w][1] = half2_bits(x[2], x[6]);
                // codes in the high nibbles come times 16
                qh[g][w][0] = half2_bits(x[1] * 0.0625f, x[5] * 0.0625f);
                qh[g][w][1] = half2_bits(x[3] * 0.0625f, x[7] * 0.0625f);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float2 a = bits_half2(ql[g][w][i]), bb = bits_half2(qh[g][w][i]);
                    qsum += (a.x + a.y) + 16.0f * (bb.x + bb.y);
                }
            }
            qsum += __shfl_xor_sync(0xffffffffu, qsum, 1);
            qsum += __shfl_xor_sync(0xffffffffu, qsum, 2);
            // codes come as c * 2^-24
            const float unit = fabsf(p.scale_log2) * pow2i(e > 103 ? 103 : e) * 16777216.0f;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float un = __shfl_sync(0xffffffffu, unit, (2 * c + i) * 4);
                row_a[g][i] = un > 0.0f ? un : FLT_MIN;   // scale 0: all scores nearly equal, masked ones stay -infinity
                row_z[g][i] = __shfl_sync(0xffffffffu, qsum, (2 * c + i) * 4) * -0x1p-24f;
                const int rr = row0 + g * 8 + (FOUR ? 2 * (c & 1) + i : 2 * c + i);
                row_pos[g][i] = rr < r.rows ? r.pos0 + rr / p.group : -1;
            }
        }
        float m[G][2], l[G][2], bad[G][2], o[G][2 * W][4];   // bad: NaN where a row sees a poisoned V, else 0
        int ev = -40;   // V's scales seen so far are at most 2^ev
#pragma unroll
        for (int g = 0; g < G; ++g) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                m[g][i] = -CUDART_INF_F;
                l[g][i] = 0.0f;
                bad[g][i] = 0.0f;
            }
#pragma unroll
            for (int w = 0; w < 2 * W; ++w)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[g][w][i] = 0.0f;
        }

#pragma unroll 1
        for (int t = first + warp; t < last && !dead; t += kWarps) {
            if (!wait_warp(smem_addr(&sh.bar[warp][s_use]), phase, ctl)) {
                dead = true;
                break;
            }
            const uint8_t* const st = ring + s_use * A::STAGE;
            const uint32_t have = (ok_bits >> (2 * s_use)) & 3u;
            const int t0 = r.base + t * kUnit;
            const bool full = have == 3u && t0 + kUnit - 1 <= pos_min && (p.window <= 0 || t0 > pos_max - p.window);

            // s_k times the products of the unit's two tiles: tokens n and n + 8 of each, rows 2c and 2c + 1
            float sc[2][G][4];
            float vs[2][2];
#pragma unroll
            for (int tl = 0; tl < 2; ++tl) {
                const uint8_t* const tile = st + tl * A::TB;
                uint32_t ka[W], kb[W];
                lds_share<W>(tile + lane * (4 * W), ka);
                lds_share<W>(tile + 8 * (D / 2) + lane * (4 * W), kb);
                float ks[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int tok = n + 8 * j;
                    ks[j] = __half2float(*reinterpret_cast<const __half*>(tile + kv4_k_scale_off(D) + 2 * tok));
                    const float kz = (float)tile[kv4_k_zero_off(D) + tok];
                    vs[tl][j] = __half2float(*reinterpret_cast<const __half*>(tile + kv4_v_scale_off(D) + 2 * tok));
                    // the sums start from the zero-points' share
#pragma unroll
                    for (int g = 0; g < G; ++g) {
                        sc[tl][g][2 * j] = kz * row_z[g][0];
                        sc[tl][g][2 * j + 1] = kz * row_z[g][1];
                    }
                }
                // low and high nibbles in sums of their own: two short chains of MMAs instead of a long one
                float sh4[G][4];
#pragma unroll
                for (int g = 0; g < G; ++g)
#pragma unroll
                    for (int i = 0; i < 4; ++i) sh4[g][i] = 0.0f;
#pragma unroll
                for (int w = 0; w < W; ++w) {
                    const uint32_t ka8 = ka[w] >> 8, kb8 = kb[w] >> 8;
#pragma unroll
                    for (int g = 0; g < G; ++g)
                        mma_16816(sc[tl][g], ka[w] & kLow, kb[w] & kLow, ka8 & kLow, kb8 & kLow, ql[g][w][0], ql[g][w][1]);
#pragma unroll
                    for (int g = 0; g < G; ++g)
                        mma_16816(sh4[g], ka[w] & kHigh, kb[w] & kHigh, ka8 & kHigh, kb8 & kHigh, qh[g][w][0], qh[g][w][1]);
                }
#pragma unroll
                for (int g = 0; g < G; ++g)
#pragma unroll
                    for (int i = 0; i < 4; ++i) sc[tl][g][i] = (sc[tl][g][i] + sh4[g][i]) * ks[i >> 1];
            }
            if (!full) {
#pragma unroll
                for (int tl = 0; tl < 2; ++tl)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int key = t0 + tl * kKv4Tile + n + 8 * j;
                        const bool there = (have >> tl & 1) && key < r.seq;
                        const bool odd = there && vs[tl][j] != vs[tl][j];   // a poisoned row of V
                        if (!there || odd) vs[tl][j] = 0.0f;
#pragma unroll
                        for (int g = 0; g < G; ++g)
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                const bool see = there && key <= row_pos[g][i] &&
                                                 (p.window <= 0 || key > row_pos[g][i] - p.window);
                                if (!see) sc[tl][g][2 * j + i] = -CUDART_INF_F;
                                else if (odd) bad[g][i] = CUDART_NAN_F;     // shows in the rows that see it alone
                            }
                    }
            }
            // the references of the running sums move if a score passes its row's by 2^kGrow, or a scale 2^ev
            float vf = pow2i(15 - kGrow - ev);
            bool grow = false;
#pragma unroll
            for (int g = 0; g < G; ++g)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float x = fmaxf(fmaxf(sc[0][g][i], sc[0][g][2 + i]), fmaxf(sc[1][g][i], sc[1][g][2 + i]));
                    grow = grow || x * row_a[g][i] > m[g][i] + (float)kGrow;
                }
            const float vmax = fmaxf(fmaxf(vs[0][0], vs[0][1]), fmaxf(vs[1][0], vs[1][1]));   // drops NaN
            grow = grow || vmax * vf > (float)(1 << (15 - kGrow));
            if (__any_sync(0xffffffffu, grow)) {
                const uint32_t vbits = __reduce_max_sync(0xffffffffu, vmax > 0.0f && vmax <= 65504.0f ? __float_as_uint(vmax) : 0u);
                const int ev_new = vbits == 0u ? ev : (int)(vbits >> 23) - 126;   // scale < 2^ev_new
                const int en = ev_new > ev ? ev_new : ev;
                const float shift = pow2i(ev - en);
#pragma unroll
                for (int g = 0; g < G; ++g) {
                    float f[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        float x = fmaxf(fmaxf(sc[0][g][i], sc[0][g][2 + i]), fmaxf(sc[1][g][i], sc[1][g][2 + i]));
                        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
                        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
                        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16)) * row_a[g][i];
                        x = fmaxf(x, m[g][i]);
                        f[i] = x == m[g][i] ? 1.0f : ex2(m[g][i] - x);
                        m[g][i] = x;
                        l[g][i] *= f[i];
                        f[i] *= shift;
                    }
#pragma unroll
                    for (int w = 0; w < 2 * W; ++w)
#pragma unroll
                        for (int i = 0; i < 4; ++i) o[g][w][i] *= f[i & 1];
                }
                ev = en;
                vf = pow2i(15 - kGrow - ev);   // probabilities are fed below 2^15, clear of subnormals
            }
            float ref[G][2];
#pragma unroll
            for (int g = 0; g < G; ++g)
#pragma unroll
                for (int i = 0; i < 2; ++i) ref[g][i] = m[g][i] == -CUDART_INF_F ? 0.0f : m[g][i];
            // The first tile adds p c and the second -p (15 - c), so that neither leaves the sums far from where they were; zo is
            // the zero-points' share of that (MMAs with V's zero-points in every row of A): o - zo gains p (c - z)
            float zo[G][4];
#pragma unroll
            for (int g = 0; g < G; ++g)
#pragma unroll
                for (int i = 0; i < 4; ++i) zo[g][i] = 0.0f;
#pragma unroll
            for (int tl = 0; tl < 2; ++tl) {
                uint32_t ph[G][2], pl[G][2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float v = vs[tl][j] * (tl ? -vf : vf);
#pragma unroll
                    for (int g = 0; g < G; ++g) {
                        float pv[2];
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const float e = ex2(fmaf(sc[tl][g][2 * j + i], row_a[g][i], -ref[g][i]));
                            l[g][i] += e;
                            pv[i] = e * v;
                        }
                        const uint32_t h = half2_bits(pv[0], pv[1]);
                        const float2 back = bits_half2(h);
                        const uint32_t low = half2_bits(pv[0] - back.x, pv[1] - back.y);
                        if constexpr (FOUR) {
                            ph[g][j] = transpose8(c < 2 ? h : low);   // the second four columns are the low parts
                        } else {
                            ph[g][j] = transpose8(h);
                            pl[g][j] = transpose8(low);
                        }
                    }
                }
                const uint8_t* const tile = st + tl * A::TB + kv4_v_off(D);
                uint32_t va[W], vb[W];
                lds_share<W>(tile + lane * (4 * W), va);
                lds_share<W>(tile + 4 * D + lane * (4 * W), vb);
                const uint16_t* const vz = reinterpret_cast<const uint16_t*>(st + tl * A::TB + kv4_v_zero_off(D));
                const uint32_t flip = tl ? 0xffffffffu : 0u;   // 15 - c is c with every bit turned
                const uint32_t za = __byte_perm(vz[c] ^ (flip & 0x0f0fu), 0, 0x4140);       // of tokens 2c and 2c + 1
                const uint32_t zb = __byte_perm(vz[c + 4] ^ (flip & 0x0f0fu), 0, 0x4140);   // of tokens 8 + 2c and 9 + 2c
#pragma unroll
                for (int g = 0; g < G; ++g) {
                    mma_16816(zo[g], za, za, zb, zb, ph[g][0], ph[g][1]);
                    if constexpr (!FOUR) mma_16816(zo[g], za, za, zb, zb, pl[g][0], pl[g][1]);
                }
#pragma unroll
                for (int w = 0; w < W; ++w) {
                    const uint32_t v1 = va[w] ^ flip, v2 = vb[w] ^ flip, v1s = v1 >> 8, v2s = v2 >> 8;
#pragma unroll
                    for (int g = 0; g < G; ++g) {
                        mma_16816(o[g][2 * w], v1 & kLow, v1s & kLow, v2 & kLow, v2s & kLow, ph[g][0], ph[g][1]);
                        mma_16816(o[g][2 * w + 1], v1 & kHigh, v1s & kHigh, v2 & kHigh, v2s & kHigh, ph[g][0], ph[g][1]);
                        if constexpr (!FOUR) {
                            mma_16816(o[g][2 * w], v1 & kLow, v1s & kLow, v2 & kLow, v2s & kLow, pl[g][0], pl[g][1]);
                            mma_16816(o[g][2 * w + 1], v1 & kHigh, v1s & kHigh, v2 & kHigh, v2s & kHigh, pl[g][0], pl[g][1]);
                        }
                    }
                }
            }
            // The unit's sums less the zero-points' share: running sums of code - zero. An MMA rounds towards zero, so the
            // roundings of sums that grow without end would all point one way, and show where what is left of them is small.
#pragma unroll
            for (int g = 0; g < G; ++g) {
                const uint64_t low2 = pack_f32x2(-zo[g][0], -zo[g][1]), high2 = mul_f32x2(low2, pack_f32x2(16.0f, 16.0f));
#pragma unroll
                for (int w = 0; w < 2 * W; ++w)
#pragma unroll
                    for (int i = 0; i < 4; i += 2)
                        unpack_f32x2(add_f32x2(pack_f32x2(o[g][w][i], o[g][w][i + 1]), w & 1 ? high2 : low2), o[g][w][i], o[g][w][i + 1]);
            }
            next_stage();
            fence_proxy_async_smem();
            __syncwarp();
            issue_next();
        }
        // copies in flight after a wait gave up
        while (pending != 0) {
            wait_drain(smem_addr(&sh.bar[warp][s_use]), phase, p.wait_limit_ns);
            next_stage();
        }
        __syncwarp();

        // ---- the four warps' shares: into shared memory, each in its own ring
        float* const mine = reinterpret_cast<float*>(ring);
        const float o_unit = pow2i(ev - (15 - kGrow));
#pragma unroll
        for (int g = 0; g < G; ++g) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) {
                    l[g][i] += __shfl_xor_sync(0xffffffffu, l[g][i], d);
                    bad[g][i] += __shfl_xor_sync(0xffffffffu, bad[g][i], d);
                }
                if (n == 0 && (!FOUR || c < 2)) {
                    sh.m[warp][g * 8 + 2 * c + i] = m[g][i];
                    sh.l[warp][g * 8 + 2 * c + i] = l[g][i];
                }
            }
            if constexpr (FOUR) {   // low and high parts of the probabilities
#pragma unroll
                for (int w = 0; w < 2 * W; ++w)
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[g][w][i] += __shfl_xor_sync(0xffffffffu, o[g][w][i], 2);
            }
#pragma unroll
            for (int w = 0; w < W; ++w)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    if (FOUR && c >= 2) continue;
                    // codes in low nibbles come as c * 2^-24, in high ones as c * 2^-20
                    float4 x;
                    x.x = o[g][2 * w][i] * 16777216.0f * o_unit + bad[g][i];
                    x.y = o[g][2 * w + 1][i] * 1048576.0f * o_unit + bad[g][i];
                    x.z = o[g][2 * w][2 + i] * 16777216.0f * o_unit + bad[g][i];
                    x.w = o[g][2 * w + 1][2 + i] * 1048576.0f * o_unit + bad[g][i];
                    *reinterpret_cast<float4*>(mine + (g * 8 + 2 * c + i) * D + n * (D / 8) + 4 * w) = x;
                }
        }
        __syncthreads();
        const int live = r.rows - row0 < ROWS ? r.rows - row0 : ROWS;
        const bool whole = pos == 0 && take == r.units;
        // joined maximum, sum and the warps' weights of each row
        float* const part = p.partials + (long long)(2 * blockIdx.x + (pos == 0 ? 1 : 0)) * A::PART;
        if (tid < live) {
            float mm = -CUDART_INF_F, ll = 0.0f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, sh.m[w][tid]);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float f = sh.m[w][tid] == mm ? 1.0f : ex2(sh.m[w][tid] - mm);
                ll += sh.l[w][tid] * f;
                sh.weight[w][tid] = f;
            }
            if (whole) {
                const float inv = ll == 0.0f ? 0.0f : 1.0f / ll;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) sh.weight[w][tid] *= inv;
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
        for (int i = tid; i < live * (D / 4); i += kThreads) {
            const int row = i / (D / 4), d = i % (D / 4) * 4;
            float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
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
            const long long g0 = seg_u + kOverhead;   // the place of the segment's first unit
            const int ca = (int)(((g0 + 1) * ctas - 1) / total), cb = (int)(((g0 + r.units) * ctas - 1) / total);
            __threadfence();
            __syncthreads();
            if (tid == 0) {
                const int before = atomicAdd(p.counters + ca, 1);
                sh.last = before == cb - ca;
                if (sh.last) p.counters[ca] = 0;   // ready for the next launch
                __threadfence();
            }
            __syncthreads();
            if (sh.last) {
                // first every partial's weight (all rows and CTAs at once, kept where the rings were), then the sums
                const int parts = cb - ca + 1;
                float* const wt = reinterpret_cast<float*>(smem);
                auto part_of = [&](int k) { return p.partials + (long long)(2 * (ca + k) + (k == 0)) * A::PART; };
                for (int i = tid; i < parts * live; i += kThreads) wt[i] = __ldcg(part_of(i / live) + ROWS * D + i % live);
                __syncthreads();
                if (warp < live) {
                    for (int row = warp; row < live; row += kWarps) {
                        float mm = -CUDART_INF_F, ll = 0.0f;
                        for (int k = lane; k < parts; k += 32) mm = fmaxf(mm, wt[k * live + row]);
#pragma unroll
                        for (int d = 16; d > 0; d >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, d));
                        for (int k = lane; k < parts; k += 32) {
                            const float mk = wt[k * live + row], f = mk == mm ? 1.0f : ex2(mk - mm);
                            wt[k * live + row] = f;
                            ll += f * __ldcg(part_of(k) + ROWS * D + ROWS + row);
                        }
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
                }
                __syncthreads();
                for (int i = tid; i < live * (D / 4); i += kThreads) {
                    const int row = i / (D / 4), d = i % (D / 4) * 4;
                    float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
                    for (int k = 0; k < parts; ++k) {
                        const float4 y = __ldcg(reinterpret_cast<const float4*>(part_of(k) + row * D + d));
                        const float f = wt[k * live + row];
                        x.x += f * y.x;
                        x.y += f * y.y;
                        x.z += f * y.z;
                        x.w += f * y.w;
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
}

template <int D, int NR>
struct Launch {
    static inline int per_sm = 1;   // CTAs an SM holds

    // CTAs of a launch: what the GPU holds, the workspace counts, and a join's weights in the rings leave room for
    static int grid_of(int sms)
    {
        const int most = (int)(kWarps * Attn<D, NR>::RING / (Attn<D, NR>::ROWS * sizeof(float)));
        const int fit = most < kWsMaxGrid ? most : kWsMaxGrid;
        return sms * per_sm < fit ? sms * per_sm : fit;
    }

    static cudaError_t setup()
    {
        cudaError_t e = cudaFuncSetAttribute(kv4_attn_kernel<D, NR>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             Attn<D, NR>::SMEM);
        if (e != cudaSuccess) return e;
        return cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kv4_attn_kernel<D, NR>, kThreads, Attn<D, NR>::SMEM);
    }

    static cudaError_t run(const Kv4AttnParams& p, int sms, cudaStream_t stream)
    {
        const int grid = grid_of(sms);
        return launch_chained(kv4_attn_kernel<D, NR>, grid, kThreads, Attn<D, NR>::SMEM, 1, stream, p);
    }
};
}  // namespace

size_t kv4_partial_bytes(int sms)
{
    size_t need = kv4_prompt_partial_bytes(sms);
    auto most = [&](int grid, int part) {
        const size_t bytes = (size_t)2 * grid * part * sizeof(float);
        need = bytes > need ? bytes : need;
    };
    most(Launch<64, 0>::grid_of(sms), Attn<64, 0>::PART);
    most(Launch<64, 1>::grid_of(sms), Attn<64, 1>::PART);
    most(Launch<64, 2>::grid_of(sms), Attn<64, 2>::PART);
    most(Launch<128, 0>::grid_of(sms), Attn<128, 0>::PART);
    most(Launch<128, 1>::grid_of(sms), Attn<128, 1>::PART);
    most(Launch<128, 2>::grid_of(sms), Attn<128, 2>::PART);
    return need;
}

cudaError_t setup_kv4()
{
    cudaError_t e;
    if ((e = Launch<64, 0>::setup()) != cudaSuccess || (e = Launch<128, 0>::setup()) != cudaSuccess ||
        (e = Launch<64, 1>::setup()) != cudaSuccess || (e = Launch<64, 2>::setup()) != cudaSuccess ||
        (e = Launch<128, 1>::setup()) != cudaSuccess || (e = Launch<128, 2>::setup()) != cudaSuccess)
        return e;
    return setup_kv4_prompt();
}

// The tcgen05 kernel takes requests of more than kFewRows rows a KV head where the batch's rows (query
// tokens times query heads) fill the GPU with its tiles of 256; which request is which is known on
// the device, so such a batch gets both kernels. With fewer rows the stream-K kernel takes everything:
// it cuts the cached tokens too. Measured for one request, D = 128, tcgen05 and stream-K in us:
// 800 rows over 1000 tokens 34 / 17; 2048 over 4000 50 / 41; 4096 50 / 64; 8192 53 / 105; 16384
// 64 / 192; 3200 over 300 14 / 21; 8400 over 300 14 / 31. D = 64: 8192 over 4000 42 / 71; 16384
// 53 / 126; 5120 over 500 16 / 25. (How many tokens are cached is not known on the host.)
// The rule does not look at the rows of one request, and a tile computes 256: many requests of 33 to 64 rows a KV
// head would be better off with the stream-K kernel. 48 requests over 4000 tokens, 4 KV heads, D = 128, tcgen05 and
// stream-K: 36 rows 174 / 116, 64 rows 175 / 155, 72 rows 175 / 186, 128 rows 175 / 288; D = 64: 166 / 80, 166 / 102,
// 166 / 122, 166 / 188.
constexpr int kFewRows = 32;
// Segments of 16 rows cost 1.75 times those of 8, and half as many CTAs fit an SM: 8 where they are fewer than 1.75
// times as many (9 to 16 rows of 64 requests over 4000 tokens, D = 128, 112 / 126 us with 16 / 8; 17 to 24 rows 199 / 178;
// 32 rows 201 / 232; D = 64, where an SM holds three of their CTAs, 75 / 88; 131 / 123; 134 / 160), and where the rows are too
// few for throughput to count (one request of 16 rows over 8000 tokens 29 / 21; eight of 16 over 1000 21 / 17; eight of 32
// over 8000 65 / 70).
constexpr int kNarrowRows = 1024;
constexpr long long prompt_rows(int head_dim) { return head_dim == 128 ? 3200 : 4096; }

cudaError_t launch_kv4_attention(const Kv4AttnParams& in, int head_dim, int max_q, int path, int sms, cudaStream_t stream)
{
    Kv4AttnParams p = in;
    const long long rows = (long long)max_q * p.group;
    const bool prompt = rows > kFewRows && path != 1 &&
                        (path == 2 || (long long)p.tokens * p.q_heads >= prompt_rows(head_dim));
    if (prompt && p.batch == 1) {   // one request is one kernel's, whatever its rows turn out to be
        p.few_rows = 0;
        return launch_kv4_prompt(p, head_dim, sms, stream);
    }
    p.few_rows = prompt ? kFewRows : INT_MAX;
    const long long held = prompt && rows > kFewRows ? kFewRows : rows;   // of a request that is this kernel's, at most
    const bool wide = 4 * ((held + 7) / 8) >= 7 * ((held + 15) / 16) && (long long)p.tokens * p.q_heads > kNarrowRows;
    cudaError_t e;
    if (head_dim == 128)
        e = held <= 4 ? Launch<128, 0>::run(p, sms, stream) : wide ? Launch<128, 2>::run(p, sms, stream) : Launch<128, 1>::run(p, sms, stream);
    else
        e = held <= 4 ? Launch<64, 0>::run(p, sms, stream) : wide ? Launch<64, 2>::run(p, sms, stream) : Launch<64, 1>::run(p, sms, stream);
    if (e != cudaSuccess || !prompt) return e;
    return launch_kv4_prompt(p, head_dim, sms, stream);
}

}  // namespace w4a16
