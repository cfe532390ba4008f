// Attention over the 4-bit paged cache for many query rows (prompt chunks): the
// mathematics of kv4_attn.cu on the tcgen05 tensor cores.
//
// A CTA owns 256 rows (query token, query head of the group) of one request's KV head, as
// two tiles of 128, and walks the cached tokens in blocks of 128, scored by halves of 64:
//   S = Q (c_k - z_k)^T          both operands in shared memory, S in tensor memory
//   P = 2^(a s_k S - m) s_v      by the rows' threads, written over S as binary16
//   O += P (c_v - z_v)           P from tensor memory, V from shared memory
// Codes less their zero-points are whole numbers of -15 .. 15, exact in binary16; the
// scales act on scores and probabilities in FP32, so the one rounding of the chain is P's to
// binary16. For bfloat16 outputs it is an eighth of theirs; for binary16 outputs it would be as
// large as theirs, so there P is fed as a high and a low part (half as many products again).
// V's scales are fed relative to the largest seen so far and P below 2^15, clear of
// overflow and of subnormals.
//
// Warps: 0-3 and 4-7 the softmax of a tile each, one thread a row (no word between threads),
// a half's 64 scores in registers; 8-11 unpack K (one thread a token) and V (one thread 8
// tokens x D/8 values of d), reading codes straight from HBM or L2 into registers most of a
// block ahead, so that there is no staging of packed data; 12 issues the MMAs. A tile's S has two
// halves in tensor memory, so the scores of the next half are there when the softmax of one ends,
// and the products run under the other half's and the other tile's softmax:
//   O_A(h), S_A(h+2), O_B(h), S_B(h+2), ...
// O is rescaled only when a row's maximum grew by more than 2^8 (its P stays below 2^15 until then).
//
// Queries and outputs go between registers and memory by way of shared memory, so that 16 (D = 64: 8) lanes
// read or write a row together; a row a lane cost a CTA 4 us more.
//
// Where the pairs of row tiles leave SMs idle, each pair's cached tokens are split over several CTAs (the
// host allows as many as fit, the device takes parts of four blocks or more), and the last of them to finish
// joins them through the workspace, in their order: 8192 rows over 4000 tokens 81 -> 53 us, 41 of D = 64.
//
// Three requests' chunks of 839 to 4000 tokens behind 5690 to 8200 cached ones, 32 query heads over
// 8, D = 128, bfloat16: 909 us, 898 TFLOP/s, 47% of what a plain bf16 matrix product reaches. (Scores
// by whole blocks, one S a tile: 1000 us.) The tensor pipe is busy for 42% of the time, the issue slots for
// 51%, shared memory for 93% (55% for the warps, 38% for the MMAs' operands), which is the nearest to a limit: without
// the exponentials, the scales or the unpacking the kernel takes 0 to 5% less, with an eighth of the products 12%.
// Of a CTA's 110 us its start and end, which nothing overlaps, are about 9; CTAs that stay and
// take the next rows themselves gained nothing there (929 us).
#include "api_internal.cuh"
#include "kv4.cuh"
#include "launch.cuh"
#include "ptx.cuh"

#include <float.h>
#include <math_constants.h>

namespace w4a16 {
namespace {

constexpr int kRows = 128;            // rows of a tile
constexpr int kBlock = 128;           // cached tokens of a block: what is unpacked together
constexpr int kHalf = 64;             // and of a half: what is scored together
constexpr int kMmaWarp = 12;
constexpr int kThreads = 512;         // four warpgroups, of the last the MMA warp alone at work
// Registers a thread: 128 at launch, moved to the softmax from the warps that need fewer. Each
// of the SM's four quarters holds one warp of every warpgroup and a quarter of the registers.
// Below 160 the softmax spills (152/112/96: 933 us where this takes 905).
constexpr int kLaunchRegs = 128, kSoftmaxRegs = 168, kUnpackRegs = 96, kIssueRegs = 80;
static_assert(2 * kSoftmaxRegs + kUnpackRegs + kIssueRegs <= 4 * kLaunchRegs, "registers of the block");
constexpr int kScaleStages = 4;       // K's scales live until the softmax has read them: two blocks past K itself
constexpr int kMaxSplits = 8;
constexpr int kLeast = 4;             // blocks of a CTA where a request's cached tokens are split over several
constexpr int kGrow = 8;              // log2 of how far P may grow before O is rescaled

template <int D>
struct Prompt {
    static constexpr int TB = kv4_tile_bytes(D);
    static constexpr int QT = kRows * D * 2;       // bytes of a Q tile, of a K block, of a V block
    static constexpr int OFF_K = 2 * QT;
    static constexpr int OFF_V = OFF_K + 2 * QT;
    static constexpr int OFF_MISC = OFF_V + 2 * QT;
    static constexpr int S_COL = 0, O_COL = 2 * kBlock;   // tensor memory columns: S of both tiles (P over it), O of both
    struct Misc {
        float sk[kScaleStages][kBlock];
        float sv[2][kBlock];
        uint32_t valid[kScaleStages][4];     // tokens that are stored and inside the request
        uint32_t odd[2][4];                  // tokens whose V scale is NaN
        uint32_t vred[2][4];
        int exponent[2][kRows];              // of the queries' rows
        int ev[2];                           // V's scales so far are below 2^ev
        uint64_t qfull, kfull[2], kempty[2], vfull[2], vempty[2], skfull[kScaleStages], sfull[2][2], pfull[2][2], odone[2][2], teardown;
        uint32_t tmem;
        int abort_flag, b, rt, last;
    };
    // one CTA an SM: it holds all of the SM's tensor memory
    static constexpr int SMEM = (OFF_MISC + (int)sizeof(Misc) > 120 * 1024 ? OFF_MISC + (int)sizeof(Misc) : 120 * 1024) + 1024;
    static_assert(SMEM <= 227 * 1024, "shared memory");
};

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

__device__ __forceinline__ __half2 as_half2(uint32_t w) { return *reinterpret_cast<const __half2*>(&w); }

__device__ __forceinline__ uint32_t sub2(uint32_t a, uint32_t b)
{
    const __half2 h = __hsub2(as_half2(a), as_half2(b));
    return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ uint32_t fma2(uint32_t a, uint32_t b, uint32_t c)
{
    const __half2 h = __hfma2(as_half2(a), as_half2(b), as_half2(c));
    return *reinterpret_cast<const uint32_t*>(&h);
}

// Four registers of code - zero from a word: nibbles (0,4), (1,5), (2,6), (3,7). A nibble in the
// mantissa of 1024.0 is 1024 + c, or 1024 + 16 c for the high one of a byte, exactly; lo = 1024 + z and
// hi = -(64 + z), in the halves' order.
__device__ __forceinline__ void unpack4(uint32_t w, uint32_t lo, uint32_t hi, uint32_t (&r)[4])
{
    constexpr uint32_t kLow = 0x000f000fu, kHigh = 0x00f000f0u, kMagic = 0x64006400u, kSixteenth = 0x2c002c00u;
    const uint32_t w8 = w >> 8;
    r[0] = sub2(and_or(w, kLow, kMagic), lo);
    r[1] = fma2(and_or(w, kHigh, kMagic), kSixteenth, hi);
    r[2] = sub2(and_or(w8, kLow, kMagic), lo);
    r[3] = fma2(and_or(w8, kHigh, kMagic), kSixteenth, hi);
}

// Byte offset of a 16-byte chunk of a K-major tile in 128-byte swizzle: blocks of 64 columns, rows of 128 bytes.
__device__ __forceinline__ uint32_t swizzled(int row, int chunk, int block_rows)
{
    return (uint32_t)((chunk >> 3) * block_rows * 128 + row * 128 + (((chunk & 7) ^ (row & 7)) << 4));
}

__device__ __forceinline__ void sts128(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d)
{
    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

template <int D, bool BF>
__global__ void __launch_bounds__(kThreads, 1) kv4_prompt_kernel(const Kv4AttnParams p)
{
    using C = Prompt<D>;
    constexpr int W = D / 32;
    extern __shared__ __align__(16) uint8_t raw_smem[];
    uint8_t* const smem = raw_smem + ((1024u - (smem_addr(raw_smem) & 1023u)) & 1023u);
    const uint32_t sbase = smem_addr(smem);
    typename C::Misc& sh = *reinterpret_cast<typename C::Misc*>(smem + C::OFF_MISC);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

    chained_kernel();
    // ---- this CTA's rows: CTAs count KV heads fastest, then row tiles, the last rows of a request
    // (which see the most tokens) first
    const int pair = blockIdx.x / p.splits, split = blockIdx.x - pair * p.splits;
    const int head = pair % p.kv_heads;
    if (warp == 0) {
        const int want = pair / p.kv_heads;
        int at = 0;
        if (lane == 0) sh.b = -1;
        for (int b0 = 0; b0 < p.batch; b0 += 32) {
            int tiles = 0;
            if (b0 + lane < p.batch) {
                int a = p.starts[b0 + lane], e = p.starts[b0 + lane + 1];
                a = a < 0 ? 0 : a > p.tokens ? p.tokens : a;
                e = e < a ? a : e > p.tokens ? p.tokens : e;
                const int rows = (e - a) * p.group;
                tiles = rows > p.few_rows ? (rows + 2 * kRows - 1) / (2 * kRows) : 0;
            }
            int incl = tiles;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int o = __shfl_up_sync(0xffffffffu, incl, d);
                if (lane >= d) incl += o;
            }
            if (want >= at + incl - tiles && want < at + incl) {
                sh.b = b0 + lane;
                sh.rt = at + incl - 1 - want;
            }
            at += __shfl_sync(0xffffffffu, incl, 31);
            if (want < at) break;
        }
        __syncwarp();
        if (lane == 0) {
            sh.abort_flag = 0;
            mbar_init(smem_addr(&sh.qfull), 2 * kRows);
            mbar_init(smem_addr(&sh.teardown), 1);
            for (int s = 0; s < 2; ++s) {
                mbar_init(smem_addr(&sh.kfull[s]), kBlock);
                mbar_init(smem_addr(&sh.vfull[s]), kBlock);
                mbar_init(smem_addr(&sh.kempty[s]), 1);
                mbar_init(smem_addr(&sh.vempty[s]), 1);
                for (int h = 0; h < 2; ++h) {
                    mbar_init(smem_addr(&sh.sfull[s][h]), 1);
                    mbar_init(smem_addr(&sh.pfull[s][h]), kRows);
                    mbar_init(smem_addr(&sh.odone[s][h]), 1);
                }
            }
            for (int s = 0; s < kScaleStages; ++s) mbar_init(smem_addr(&sh.skfull[s]), 4);
            fence_mbar_init();
        }
    }
    __syncthreads();
    const int b = sh.b;
    if (b < 0) return;   // more CTAs than row tiles
    const long long held = (long long)p.table_cols * p.page_size;
    const int len = p.seq_lens[b] < 0 ? 0 : p.seq_lens[b];   // cached tokens, of which the table holds the first `seq`
    const int seq = len < held ? len : (int)held;
    int q0 = p.starts[b], q1 = p.starts[b + 1];
    q0 = q0 < 0 ? 0 : q0 > p.tokens ? p.tokens : q0;
    q1 = q1 < q0 ? q0 : q1 > p.tokens ? p.tokens : q1;
    const int nq = q1 - q0, rows = nq * p.group, row0 = sh.rt * 2 * kRows;
    const int end_row = row0 + 2 * kRows < rows ? row0 + 2 * kRows : rows;
    // cached tokens that some row here sees: from base to end
    const int pos0 = len - nq;   // the first query's position
    const int pos_first = pos0 + row0 / p.group, pos_last = pos0 + (end_row - 1) / p.group;
    const int last_seen = pos_last < seq ? pos_last : seq - 1;
    // (a row at a negative position sees nothing; none of them: no overflow whatever the window)
    const int low = p.window > 0 ? (pos_first > 0 ? pos_first : 0) - p.window + 1 : 0;
    int base = low > 0 ? low / kBlock * kBlock : 0;
    int halves = last_seen >= base ? (last_seen - base) / kHalf + 1 : 0, blocks = (halves + 1) / 2;
    // of them this CTA's part; parts of fewer than kLeast blocks are not worth joining
    const int most = blocks / kLeast, parts = most < 1 ? 1 : most < p.splits ? most : p.splits;
    if (split >= parts) return;
    if (parts > 1) {
        const int from = (int)((long long)blocks * split / parts), to = (int)((long long)blocks * (split + 1) / parts);
        halves = (2 * to < halves ? 2 * to : halves) - 2 * from;
        base += from * kBlock;
        blocks = to - from;
    }
    if (warp == kMmaWarp) {
        tmem_alloc(smem_addr(&sh.tmem), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem;
    const WaitCtl ctl{&sh.abort_flag, p.status, p.wait_limit_ns};

    if (warp < 8) {
        // ------------------------------------------------------------ softmax: one thread a row
        setmaxnreg_inc<kSoftmaxRegs>();
        const int tile = warp >> 2;
        const int row = row0 + tile * kRows + (warp & 3) * 32 + lane;
        const bool live = row < rows;
        const int qi = row / p.group, hq = row - qi * p.group;
        const int pos = live ? pos0 + qi : -1;
        // lanes that move a row between memory and shared memory together, and rows of a warp's access
        constexpr int kLanes = D / 8, kTogether = 32 / kLanes;
        const int warp_row = (warp & 3) * 32;   // of the tile's rows
        const long long q_off = live ? (long long)(q0 + qi) * p.q_token + (long long)(head * p.group + hq) * p.q_head : -1;
        const long long o_off = live ? (long long)(q0 + qi) * p.o_token + (long long)(head * p.group + hq) * p.o_head : -1;
        float a;   // score = a * (s_k S) in powers of two
        {
            auto lo_of = [&](uint32_t x) { return BF ? __uint_as_float(x << 16) : __low2float(as_half2(x)); };
            auto hi_of = [&](uint32_t x) { return BF ? __uint_as_float(x & 0xffff0000u) : __high2float(as_half2(x)); };
            // kLanes lanes read a row together, so that a warp's load is of few lines
            uint4 raw[kLanes];
#pragma unroll
            for (int i = 0; i < kLanes; ++i) {
                const long long off = __shfl_sync(0xffffffffu, q_off, i * kTogether + lane / kLanes);
                raw[i] = off < 0 ? make_uint4(0, 0, 0, 0) : __ldg(reinterpret_cast<const uint4*>((const uint16_t*)p.q + off) + lane % kLanes);
            }
            const uint32_t qb = sbase + tile * C::QT;
#pragma unroll
            for (int i = 0; i < kLanes; ++i) {
                const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
                float top = 0.0f;
#pragma unroll
                for (int c = 0; c < 4; ++c) top = fmaxf(top, fmaxf(fabsf(lo_of(w[c])), fabsf(hi_of(w[c]))));
#pragma unroll
                for (int d = 1; d < kLanes; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
                // largest magnitude into [2^9, 2^10), by a power of two; an infinity or a NaN stays one
                int e = ((__float_as_int(top) >> 23) & 255) - 127 - 9;
                e = (top == 0.0f || !(top <= FLT_MAX)) ? 0 : e < -120 ? -120 : e;
                // a negative softmax scale goes into Q, so that the largest score is that of the largest product
                const float f = p.scale_log2 < 0.0f ? -pow2i(-e) : pow2i(-e);
                float x[8];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    x[2 * c] = lo_of(w[c]) * f;
                    x[2 * c + 1] = hi_of(w[c]) * f;
                }
                const int r = warp_row + i * kTogether + lane / kLanes;
                if (lane % kLanes == 0) sh.exponent[tile][r] = e;
                // the order in which a word of K's codes unpacks
                sts128(qb + swizzled(r, lane % kLanes, kRows), half2_bits(x[0], x[4]), half2_bits(x[1], x[5]),
                       half2_bits(x[2], x[6]), half2_bits(x[3], x[7]));
            }
            __syncwarp();
            a = fabsf(p.scale_log2) * pow2i(sh.exponent[tile][warp_row + lane]);
            a = a > 0.0f ? a : FLT_MIN;   // scale 0: all scores nearly equal, and masked ones stay -infinity
        }
        fence_proxy_async_smem();
        mbar_arrive(smem_addr(&sh.qfull));

        const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t s_at = lanes + C::S_COL + tile * kBlock, o_at = lanes + C::O_COL + tile * D;
        const int t_row0 = row0 + tile * kRows;
        const int t_last = t_row0 + kRows < rows ? t_row0 + kRows : rows;
        const int pos_min = t_row0 < rows ? pos0 + t_row0 / p.group : -1;
        const int pos_max = t_row0 < rows ? pos0 + (t_last - 1) / p.group : -1;
        float m = -CUDART_INF_F;   // of s_k S
        uint64_t l2 = 0;           // sums of even and odd columns
        const uint64_t a2 = pack_f32x2(a, a);
        int ev = -126;
        bool ok = true, poisoned = false;
        // the products of all halves before h > 0 (those of two halves may be outstanding, so each half has a barrier)
        auto wait_outputs = [&](int h) { return wait_warp(smem_addr(&sh.odone[tile][(h - 1) & 1]), ((h - 1) >> 1) & 1, ctl); };
#pragma unroll 1
        for (int h = 0; h < halves; ++h) {
            const int i = h >> 1, half = h & 1, s4 = i % kScaleStages, s2 = i & 1;
            if (!wait_warp(smem_addr(&sh.skfull[s4]), (i / kScaleStages) & 1, ctl) ||
                !wait_warp(smem_addr(&sh.sfull[tile][half]), i & 1, ctl)) {
                ok = false;
                break;
            }
            tc_fence_after();
            const uint32_t sh_at = s_at + half * kHalf;
            // x: s_k times the products, then the exponent, pairs of columns
            uint64_t x[kHalf / 2];
            {
                uint32_t r[64];
                tmem_ld64(sh_at, r);
#pragma unroll
                for (int j = 0; j < kHalf / 2; ++j)
                    x[j] = pack_f32x2(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1]));
            }
#pragma unroll
            for (int j = 0; j < kHalf / 2; j += 2) {
                const ulonglong2 k = *reinterpret_cast<const ulonglong2*>(&sh.sk[s4][half * kHalf + 2 * j]);
                x[j] = mul_f32x2(x[j], k.x);
                x[j + 1] = mul_f32x2(x[j + 1], k.y);
            }
            const int t0 = base + h * kHalf;
            const uint2 vw = *reinterpret_cast<const uint2*>(&sh.valid[s4][2 * half]);
            const bool full = (vw.x & vw.y) == 0xffffffffu && t0 + kHalf - 1 <= pos_min &&
                              (p.window <= 0 || t0 > pos_max - p.window);
            // this row's visible columns of the half, where stored: word w's bits
            auto see = [&](int w) -> uint32_t {
                const int hi = pos - t0 + 1 - 32 * w, lo = p.window > 0 && hi > 0 ? hi - p.window : 0;
                const uint32_t upto = hi <= 0 ? 0u : hi >= 32 ? 0xffffffffu : (1u << hi) - 1u;
                const uint32_t below = lo <= 0 ? 0u : lo >= 32 ? 0xffffffffu : (1u << lo) - 1u;
                return (w ? vw.y : vw.x) & upto & ~below;
            };
            if (!full) {
                // selected, not added: what a row does not see may be any memory
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    const uint32_t bits = see(w);
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        float u, v;
                        unpack_f32x2(x[16 * w + j], u, v);
                        u = bits >> (2 * j) & 1u ? u : -CUDART_INF_F;
                        v = bits >> (2 * j + 1) & 1u ? v : -CUDART_INF_F;
                        x[16 * w + j] = pack_f32x2(u, v);
                    }
                }
            }
            float tops[4] = {-CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F};
#pragma unroll
            for (int j = 0; j < kHalf / 2; ++j) {
                float u, v;
                unpack_f32x2(x[j], u, v);
                tops[j & 3] = fmaxf(tops[j & 3], fmaxf(u, v));
            }
            const float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
            if (half == 0 && !wait_warp(smem_addr(&sh.vfull[s2]), (i >> 1) & 1, ctl)) {
                ok = false;
                break;
            }
            const int en = sh.ev[s2];
            const uint2 ow = *reinterpret_cast<const uint2*>(&sh.odd[s2][2 * half]);
            if (ow.x | ow.y)   // a NaN in V's scales shows in the rows that see it
                poisoned = poisoned || ((ow.x & see(0)) | (ow.y & see(1))) != 0u;
            float f = 1.0f;
            if (top > m) {
                if (m == -CUDART_INF_F) {
                    m = top;       // nothing so far: l and O are zero
                } else if ((top - m) * a > (float)kGrow) {
                    f = ex2((m - top) * a);
                    m = top;
                    l2 = mul_f32x2(l2, pack_f32x2(f, f));
                }
            }
            if (en != ev) {
                if (ev > -126) f *= pow2i(ev - en > -126 ? ev - en : -126);
                ev = en;
            }
            if (h > 0 && __any_sync(0xffffffffu, f != 1.0f)) {
                if (!wait_outputs(h)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
#pragma unroll 1
                for (int c = 0; c < D; c += 16) {
                    float y[16];
                    uint32_t r[16];
                    tmem_ld_f32<16>(o_at + c, y);
#pragma unroll
                    for (int j = 0; j < 16; ++j) r[j] = __float_as_uint(y[j] * f);
                    tmem_st16(o_at + c, r);
                }
            }
            const float ma = m == -CUDART_INF_F ? 0.0f : m * a;
            const uint64_t ma2 = pack_f32x2(-ma, -ma);
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                uint32_t hi[16], lo[16];
#pragma unroll
                for (int j = 0; j < 16; j += 2) {
                    const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(&sh.sv[s2][half * kHalf + 32 * c + 2 * j]);
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        float u0, u1;
                        unpack_f32x2(fma_f32x2(x[16 * c + j + q], a2, ma2), u0, u1);
                        const uint64_t e = pack_f32x2(ex2(u0), ex2(u1));
                        l2 = add_f32x2(l2, e);
                        float p0, p1;
                        unpack_f32x2(mul_f32x2(e, q ? v.y : v.x), p0, p1);
                        hi[j + q] = half2_bits(p0, p1);
                        if constexpr (!BF) {
                            const float2 back = __half22float2(as_half2(hi[j + q]));
                            lo[j + q] = half2_bits(p0 - back.x, p1 - back.y);
                        }
                    }
                }
                // the high parts of 32 columns over the first 16 of them, the low parts over the others
                tmem_st16_async(sh_at + 32 * c, hi);
                if constexpr (!BF) tmem_st16_async(sh_at + 32 * c + 16, lo);
            }
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(smem_addr(&sh.pfull[tile][half]));
        }
        float l, l_odd;
        unpack_f32x2(l2, l, l_odd);
        l += l_odd;
        if (ok && halves > 0) {
            ok = wait_outputs(halves);
            tc_fence_after();
        }
        if (parts > 1) {
            // ---- O, not divided, with its maximum and sum; the last of the parts to be written joins them all
            float* const first = p.partials + (long long)pair * p.splits * (2 * kRows * (D + 2));
            float* const mine = first + (long long)split * (2 * kRows * (D + 2));
            const int r = tile * kRows + warp_row + lane;
            if (ok) {
                const float unit = poisoned ? CUDART_NAN_F : pow2i(ev - 7 > -126 ? ev - 7 : -126);
#pragma unroll
                for (int c = 0; c < D; c += 16) {
                    float x[16];
                    if (halves > 0) tmem_ld_f32<16>(o_at + c, x);
#pragma unroll
                    for (int j = 0; j < 16; j += 4) {
                        const float4 y = l == 0.0f ? make_float4(0.0f, 0.0f, 0.0f, 0.0f)
                                                   : make_float4(x[j] * unit, x[j + 1] * unit, x[j + 2] * unit, x[j + 3] * unit);
                        __stcg(reinterpret_cast<float4*>(mine + r * D + c + j), y);
                    }
                }
                __stcg(mine + 2 * kRows * D + r, l == 0.0f ? -CUDART_INF_F : m * a);
                __stcg(mine + 2 * kRows * (D + 1) + r, l);
            }
            __threadfence();
            named_bar_sync(2, 2 * kRows);
            if (tid == 0) {
                const int before = atomicAdd(p.counters + pair, 1);
                sh.last = before == parts - 1;
                if (sh.last) p.counters[pair] = 0;   // ready for the next launch
                __threadfence();
            }
            named_bar_sync(2, 2 * kRows);
            if (sh.last) {
                // this row's maximum and sum over the parts, and their weights where the tile's queries were
                float* const weight = reinterpret_cast<float*>(smem) + tile * kMaxSplits * kRows + warp_row;   // [part][row of the tile]
                constexpr long long kPart = 2 * kRows * (D + 2);
                float top = -CUDART_INF_F, sum = 0.0f, mk[kMaxSplits];
#pragma unroll
                for (int k = 0; k < kMaxSplits; ++k)
                    if (k < parts) mk[k] = __ldcg(first + k * kPart + 2 * kRows * D + r);
#pragma unroll
                for (int k = 0; k < kMaxSplits; ++k)
                    if (k < parts) top = fmaxf(top, mk[k]);
#pragma unroll
                for (int k = 0; k < kMaxSplits; ++k)
                    if (k < parts) {
                        const float f = mk[k] == top ? 1.0f : ex2(mk[k] - top);
                        sum += f * __ldcg(first + k * kPart + 2 * kRows * (D + 1) + r);
                        weight[k * kRows + lane] = f;
                    }
                const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
                if (live && p.lse)
                    p.lse[(long long)(q0 + qi) * p.q_heads + head * p.group + hq] =
                        sum == 0.0f ? -CUDART_INF_F : (top + log2f(sum)) * CUDART_LN2_F;
                __syncwarp();
                // D / 8 lanes a row, eight values each, as the outputs are written
#pragma unroll 2
                for (int i = 0; i < kLanes; ++i) {
                    const int q = i * kTogether + lane / kLanes;
                    const float by = __shfl_sync(0xffffffffu, inv, q);
                    const long long off = __shfl_sync(0xffffffffu, o_off, q);
                    float o[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
                    if (off >= 0) {
                        const float4* at = reinterpret_cast<const float4*>(first + (long long)(tile * kRows + warp_row + q) * D) + 2 * (lane % kLanes);
#pragma unroll 4
                        for (int k = 0; k < parts; ++k) {
                            const float4 x = __ldcg(at + k * (kPart / 4)), y = __ldcg(at + k * (kPart / 4) + 1);
                            const float f = weight[k * kRows + q];
                            o[0] += f * x.x, o[1] += f * x.y, o[2] += f * x.z, o[3] += f * x.w;
                            o[4] += f * y.x, o[5] += f * y.y, o[6] += f * y.z, o[7] += f * y.w;
                        }
                        uint32_t w[4];
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            const float u = by == 0.0f ? 0.0f : o[2 * c] * by, v = by == 0.0f ? 0.0f : o[2 * c + 1] * by;
                            if constexpr (BF) {
                                const __nv_bfloat162 h = __floats2bfloat162_rn(u, v);
                                w[c] = *reinterpret_cast<const uint32_t*>(&h);
                            } else {
                                w[c] = half2_bits(u, v);
                            }
                        }
                        *(reinterpret_cast<uint4*>((uint16_t*)p.out + off) + lane % kLanes) = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                }
            }
        } else if (ok) {
            const float inv = l == 0.0f ? 0.0f : poisoned ? CUDART_NAN_F : pow2i(ev - 7 > -126 ? ev - 7 : -126) / l;
            // through the tile's queries, which have been read, so that kLanes lanes write a row together
            const uint32_t qb = sbase + tile * C::QT;
#pragma unroll
            for (int c = 0; c < D; c += 16) {
                float x[16];
                if (halves > 0) tmem_ld_f32<16>(o_at + c, x);
                uint32_t r[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float u = l == 0.0f ? 0.0f : x[2 * j] * inv, v = l == 0.0f ? 0.0f : x[2 * j + 1] * inv;
                    if constexpr (BF) {
                        const __nv_bfloat162 h = __floats2bfloat162_rn(u, v);
                        r[j] = *reinterpret_cast<const uint32_t*>(&h);
                    } else {
                        r[j] = half2_bits(u, v);
                    }
                }
                sts128(qb + swizzled(warp_row + lane, c / 8, kRows), r[0], r[1], r[2], r[3]);
                sts128(qb + swizzled(warp_row + lane, c / 8 + 1, kRows), r[4], r[5], r[6], r[7]);
            }
            __syncwarp();
#pragma unroll
            for (int i = 0; i < kLanes; ++i) {
                const int r = i * kTogether + lane / kLanes;
                const long long off = __shfl_sync(0xffffffffu, o_off, r);
                const uint4 v = *reinterpret_cast<const uint4*>(smem + tile * C::QT + swizzled(warp_row + r, lane % kLanes, kRows));
                if (off >= 0) *(reinterpret_cast<uint4*>((uint16_t*)p.out + off) + lane % kLanes) = v;
            }
            __syncwarp();
            if (live && p.lse)
                p.lse[(long long)(q0 + qi) * p.q_heads + head * p.group + hq] =
                    l == 0.0f ? -CUDART_INF_F : (m * a + log2f(l)) * CUDART_LN2_F;
        }
    } else if (warp < kMmaWarp) {
        // ------------------------------------------------------------ unpack
        setmaxnreg_dec<kUnpackRegs>();
        const int t = tid - 8 * 32;   // 0 .. 127
        const int32_t* const trow = p.table + (long long)b * p.table_stride;
        const int tpp_shift = __ffs(p.page_size) - 1 - 4;
        // K: token t, of tile t / 16. V: tokens 8 vh .. 8 vh + 7 of tile vt, values vn D/8 .. of d, so
        // that the eight 16-byte chunks of a swizzled row are written by eight neighbouring lanes
        const int vh = t & 1, vt = (t >> 6) * 4 + ((t >> 1) & 3), vn = (t >> 3) & 7;
        auto page_of = [&](int i, int tile) {   // the page that holds a tile of block i, or -1
            const int g = (base + i * kBlock) / kKv4Tile + tile;
            if (i >= blocks || g * kKv4Tile >= seq) return -1;
            const int page = trow[g >> tpp_shift];
            return page >= 0 && page < p.pages ? page : -1;
        };
        auto tile_at = [&](int i, int tile, int page) {
            const int g = (base + i * kBlock) / kKv4Tile + tile;
            return p.cache + ((((long long)page * p.kv_heads + head) << tpp_shift) + (g & ((1 << tpp_shift) - 1))) * C::TB;
        };
        constexpr uint32_t kNotStored = 0x10000u;
        uint4 kw[W], vw[W];
        uint2 vz;
        uint32_t kz, ks, vs;   // scales: binary16 bits of token t's, or kNotStored
        auto load_k = [&](int i, int page) {
#pragma unroll
            for (int j = 0; j < W; ++j) kw[j] = make_uint4(0, 0, 0, 0);
            kz = 0;
            ks = vs = kNotStored;
            if (page >= 0) {
                const uint8_t* const tile = tile_at(i, t >> 4, page);
                const uint4* at = reinterpret_cast<const uint4*>(tile + (t & 15) * (D / 2));
#pragma unroll
                for (int j = 0; j < W; ++j) kw[j] = __ldg(at + j);
                kz = __ldg(tile + kv4_k_zero_off(D) + (t & 15));
                if (base + i * kBlock + t < seq) {
                    ks = __ldg(reinterpret_cast<const uint16_t*>(tile + kv4_k_scale_off(D)) + (t & 15));
                    vs = __ldg(reinterpret_cast<const uint16_t*>(tile + kv4_v_scale_off(D)) + (t & 15));
                }
            }
        };
        auto load_v = [&](int i, int page) {
#pragma unroll
            for (int j = 0; j < W; ++j) vw[j] = make_uint4(0, 0, 0, 0);
            vz = make_uint2(0, 0);
            if (page >= 0) {
                const uint8_t* const tile = tile_at(i, vt, page);
                const uint4* at = reinterpret_cast<const uint4*>(tile + kv4_v_off(D) + (vh * 8 + vn) * (16 * W));
#pragma unroll
                for (int j = 0; j < W; ++j) vw[j] = __ldg(at + j);
                vz = __ldg(reinterpret_cast<const uint2*>(tile + kv4_v_zero_off(D) + 8 * vh));
            }
        };
        load_k(0, page_of(0, t >> 4));
        load_v(0, page_of(0, vt));
        int kpage = page_of(1, t >> 4), vpage = page_of(1, vt);
        int ev = -126;
#pragma unroll 1
        for (int i = 0; i < blocks; ++i) {
            const int s2 = i & 1, s4 = i % kScaleStages;
            if (!wait_warp(smem_addr(&sh.kempty[s2]), ((i >> 1) & 1) ^ 1, ctl)) sh.abort_flag = 1;
            {
                const bool stored = ks != kNotStored;
                sh.sk[s4][t] = stored ? __half2float(__ushort_as_half((uint16_t)ks)) : 0.0f;
                const uint32_t bits = __ballot_sync(0xffffffffu, stored);
                if (lane == 0) sh.valid[s4][warp & 3] = bits;
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_addr(&sh.skfull[s4]));
                const uint32_t z = kz & 255u;
                const uint32_t lo = (0x6400u + z) * 0x00010001u, hi = (0xd400u + (z << 4)) * 0x00010001u;
                const uint32_t kb = sbase + C::OFF_K + s2 * C::QT;
#pragma unroll
                for (int j = 0; j < W; ++j) {
                    const uint32_t w[4] = {kw[j].x, kw[j].y, kw[j].z, kw[j].w};
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        uint32_t r[4];
                        unpack4(w[q], lo, hi, r);
                        sts128(kb + swizzled(t, 4 * j + q, kBlock), r[0], r[1], r[2], r[3]);
                    }
                }
            }
            fence_proxy_async_smem();
            mbar_arrive(smem_addr(&sh.kfull[s2]));
            const uint32_t my_vs = vs;
            load_k(i + 1, kpage);
            kpage = page_of(i + 2, t >> 4);

            const bool ready = wait_warp(smem_addr(&sh.vempty[s2]), ((i >> 1) & 1) ^ 1, ctl);
            {
                // the exponent that bounds V's scales so far
                const bool stored = my_vs != kNotStored;
                float scale = stored ? __half2float(__ushort_as_half((uint16_t)my_vs)) : 0.0f;
                const uint32_t odd = __ballot_sync(0xffffffffu, scale != scale);
                if (scale != scale) scale = 0.0f;
                const uint32_t wmax = __reduce_max_sync(0xffffffffu, scale <= 65504.0f ? __float_as_uint(scale) & 0x7fffffffu : 0u);
                if (lane == 0) {
                    sh.odd[s2][warp & 3] = odd;
                    sh.vred[s2][warp & 3] = wmax;
                }
                if (named_bar_or(1, kBlock, !ready)) break;   // all of these warps or none
                const uint4 red = *reinterpret_cast<const uint4*>(sh.vred[s2]);
                uint32_t top = red.x > red.y ? red.x : red.y;
                top = red.z > top ? red.z : top;
                top = red.w > top ? red.w : top;
                const int en = top == 0u ? -126 : (int)(top >> 23) - 126;
                ev = en > ev ? en : ev;
                sh.sv[s2][t] = scale * (ev <= -126 ? 0.0f : pow2i(15 - kGrow - ev));
                if (t == 0) sh.ev[s2] = ev;
                uint32_t lo[4], hi[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const uint32_t zz = (c < 2 ? vz.x : vz.y) >> (16 * (c & 1));
                    const uint32_t z2 = (zz & 255u) | (zz >> 8 & 255u) << 16;   // tokens 2c and 2c + 1
                    lo[c] = 0x64006400u + z2;
                    hi[c] = 0xd400d400u + (z2 << 4);
                }
                uint32_t w[4][W];   // [pair of tokens][word]
                if constexpr (W == 4) {
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        w[c][0] = vw[c].x;
                        w[c][1] = vw[c].y;
                        w[c][2] = vw[c].z;
                        w[c][3] = vw[c].w;
                    }
                } else {
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        w[2 * c][0] = vw[c].x;
                        w[2 * c][1] = vw[c].y;
                        w[2 * c + 1][0] = vw[c].z;
                        w[2 * c + 1][1] = vw[c].w;
                    }
                }
                const uint32_t vb = sbase + C::OFF_V + s2 * C::QT;
                const int chunk = vt * 2 + vh;
#pragma unroll
                for (int j = 0; j < W; ++j) {
                    uint32_t r[4][4];
#pragma unroll
                    for (int c = 0; c < 4; ++c) unpack4(w[c][j], lo[c], hi[c], r[c]);
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        sts128(vb + swizzled(vn * (D / 8) + 4 * j + q, chunk, D), r[0][q], r[1][q], r[2][q], r[3][q]);
                }
            }
            fence_proxy_async_smem();
            mbar_arrive(smem_addr(&sh.vfull[s2]));
            load_v(i + 1, vpage);
            vpage = page_of(i + 2, vt);
        }
    } else {
        // ------------------------------------------------------------ MMA issue
        setmaxnreg_dec<kIssueRegs>();
        if (warp == kMmaWarp) {
        constexpr uint32_t idesc_s = idesc_f16_f32(128, kHalf), idesc_o = idesc_f16_f32(128, D);
        // S of a tile for half h: K's tokens 64 (h mod 2) .. of its block
        auto scores = [&](int tile, int h) {
            const uint64_t qd = smem_desc_k_sw128(sbase + tile * C::QT);
            const uint64_t kd = smem_desc_k_sw128(sbase + C::OFF_K + (h >> 1 & 1) * C::QT + (h & 1) * kHalf * 128);
            const uint32_t d = tmem + C::S_COL + tile * kBlock + (h & 1) * kHalf;
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                const uint64_t off = (uint64_t)((k >> 2) * (kRows * 8) + (k & 3) * 2);
                mma_f16_ss(d, qd + off, kd + off, idesc_s, k > 0 ? 1u : 0u);
            }
        };
        auto outputs = [&](int tile, int h) {
            const uint64_t vd = smem_desc_k_sw128(sbase + C::OFF_V + (h >> 1 & 1) * C::QT + (h & 1) * D * 128);
            const uint32_t d = tmem + C::O_COL + tile * D, a = tmem + C::S_COL + tile * kBlock + (h & 1) * kHalf;
            // 32 columns of P lie in the first 16 of S's columns for them, their low parts in the others
#pragma unroll
            for (int k = 0; k < kHalf / 16; ++k)
                mma_f16_ts(d, a + (k >> 1) * 32 + (k & 1) * 8, vd + (uint64_t)(k * 2), idesc_o, (h > 0 || k > 0) ? 1u : 0u);
            if constexpr (!BF) {
#pragma unroll
                for (int k = 0; k < kHalf / 16; ++k)
                    mma_f16_ts(d, a + (k >> 1) * 32 + 16 + (k & 1) * 8, vd + (uint64_t)(k * 2), idesc_o, 1u);
            }
        };
        bool ok = halves > 0 && wait_warp(smem_addr(&sh.qfull), 0, ctl) && wait_warp(smem_addr(&sh.kfull[0]), 0, ctl);
        if (ok) {
            tc_fence_after();
            if (elect_one()) {
                for (int h = 0; h < 2 && h < halves; ++h)
                    for (int tile = 0; tile < 2; ++tile) {
                        scores(tile, h);
                        mma_commit(smem_addr(&sh.sfull[tile][h]));
                    }
                mma_commit(smem_addr(&sh.kempty[0]));
            }
            __syncwarp();
        }
        for (int h = 0; ok && h < halves; ++h) {
            const int half = h & 1, i = h >> 1, s2 = i & 1, n = i + 1;   // h + 2 is of block n
            const bool more = h + 2 < halves;
            if (half == 0) {
                if (!wait_warp(smem_addr(&sh.vfull[s2]), (i >> 1) & 1, ctl)) break;
                if (more && !wait_warp(smem_addr(&sh.kfull[n & 1]), (n >> 1) & 1, ctl)) break;
            }
#pragma unroll 1
            for (int tile = 0; tile < 2; ++tile) {
                if (ok && !wait_warp(smem_addr(&sh.pfull[tile][half]), i & 1, ctl)) ok = false;
                if (!ok) continue;
                tc_fence_after();
                if (elect_one()) {
                    outputs(tile, h);
                    mma_commit(smem_addr(&sh.odone[tile][half]));
                    if (tile == 1 && half == 1) mma_commit(smem_addr(&sh.vempty[s2]));
                    if (more) {
                        scores(tile, h + 2);
                        mma_commit(smem_addr(&sh.sfull[tile][half]));
                        if (tile == 1 && half == 1) mma_commit(smem_addr(&sh.kempty[n & 1]));
                    }
                }
                __syncwarp();
            }
        }
        // every MMA issued so far completes before the tensor memory is freed
        if (elect_one()) {
            mma_commit(smem_addr(&sh.teardown));
            wait_drain(smem_addr(&sh.teardown), 0, 1000000000LL);
        }
        __syncwarp();
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

}  // namespace

namespace {

template <int D, bool BF>
cudaError_t setup_one()
{
    cudaFuncAttributes attr;
    cudaError_t e = cudaFuncGetAttributes(&attr, kv4_prompt_kernel<D, BF>);
    if (e != cudaSuccess) return e;
    // the warpgroups' shares have to fit the registers the block is launched with
    if (attr.numRegs < kLaunchRegs) return cudaErrorInvalidConfiguration;
    return cudaFuncSetAttribute(kv4_prompt_kernel<D, BF>, cudaFuncAttributeMaxDynamicSharedMemorySize, Prompt<D>::SMEM);
}

template <int D, bool BF>
cudaError_t launch_one(const Kv4AttnParams& p, unsigned grid, cudaStream_t stream)
{
    return launch_chained(kv4_prompt_kernel<D, BF>, grid, kThreads, Prompt<D>::SMEM, 1, stream, p);
}

}  // namespace

size_t kv4_prompt_partial_bytes(int sms) { return (size_t)sms * 2 * kRows * (128 + 2) * sizeof(float); }

cudaError_t setup_kv4_prompt()
{
    cudaError_t e;
    if ((e = setup_one<64, false>()) != cudaSuccess || (e = setup_one<64, true>()) != cudaSuccess ||
        (e = setup_one<128, false>()) != cudaSuccess || (e = setup_one<128, true>()) != cudaSuccess)
        return e;
    return cudaSuccess;
}

cudaError_t launch_kv4_prompt(const Kv4AttnParams& in, int head_dim, int sms, cudaStream_t stream)
{
    Kv4AttnParams p = in;
    // the row tiles of any split of the tokens over the requests
    const long long tiles = (long long)p.tokens * p.group / (2 * kRows) + p.batch;
    const long long pairs = tiles * p.kv_heads;
    // where they leave SMs idle, each pair's cached tokens are split over several CTAs
    p.splits = pairs * 2 > sms ? 1 : (int)(sms / pairs < kMaxSplits ? sms / pairs : kMaxSplits);
    const long long grid = pairs * p.splits;
    if (grid >= (1LL << 31)) return cudaErrorInvalidValue;
    if (head_dim == 128) return p.bf16 ? launch_one<128, true>(p, (unsigned)grid, stream) : launch_one<128, false>(p, (unsigned)grid, stream);
    return p.bf16 ? launch_one<64, true>(p, (unsigned)grid, stream) : launch_one<64, false>(p, (unsigned)grid, stream);
}

}  // namespace w4a16
