// Attention over the 8-bit paged cache for few query rows (a decode step, drafted tokens): O = softmax(scale * Q K^T) V with
// K, V = (code - 128) * scale, one scale for 16 tokens of a head.
//
// Work is dealt and joined as in the 4-bit cache's kernel (segments of up to 8 NR rows, or four, their cached tokens in units of 32,
// stream-K over the CTAs). In a CTA, four warps take a run's units in turn, each with its own ring of bulk copies. With c the code
// and s the scale of a tile:
//   score = s_k (q . c_k - 128 sum(q)) * scale,   out = sum_tiles s_v sum_t p_t (c_v - 128) / sum_t p_t
// The MMAs multiply by the bare codes (two binary16 subnormals from a word by one operation, exact), from accumulators that
// start at the share of the 128s: -128 sum(q) for the scores, -128 sum(p), itself an MMA, for the outputs. V's scale acts on
// a tile's sums, which go into the running output by an FP32 multiply-add: roundings of the MMAs (towards zero) do
// not add up over the tiles, and scales of any size keep all of P's bits. P is fed as a high and a low binary16 part, 22 bits. Where four
// rows are enough they stand twice in the MMA's eight columns, the second time with the low parts.
//
// Measured, D = 128: 64 requests of 257 to 16384 cached tokens 97 us, 5.6 TB/s, 83% of a copy's rate; one of 131072 tokens 51 us,
// 5.2 TB/s; D = 64, 48 requests of 1 to 5 drafted tokens and a window of 4096 19 us; one of 1000 tokens 9.2 us, most of it latency.
// The bytes bound it while all CTAs are at work; the rest is their ends: SMs finish 15% apart at equal work (of 64 ragged requests
// after 79 to 108 us, 94 on average), a segment's end takes 2 us, under load 6. Units of one tile took 102, 53.5 and 22 us; four CTAs an SM (128
// registers, spills) 107, 57 and, D = 64, what they take now. More CTAs than the GPU holds, with shorter runs, took 108 and 69 us;
// parts counted at the end of a CTA's run instead of at once 100 and 53.
#include "api_internal.cuh"
#include "kv8.cuh"
#include "kv_attn.cuh"
#include "launch.cuh"
#include "ptx.cuh"

#include <float.h>

namespace w4a16 {
namespace {

constexpr int kWarps = kAttnWarps, kThreads = kAttnThreads, kGrow = kAttnGrow;
constexpr uint32_t kEven = 0x00ff00ffu;          // bytes 0 and 2 of a word
constexpr uint32_t kMiddle = 0x80808080u;        // -128 * 2^-24, twice

__device__ __forceinline__ uint32_t odd_bytes(uint32_t w) { return __byte_perm(w, 0, 0x4341); }   // bytes 1 and 3

// d = a * b + c
__device__ __forceinline__ void mma_from(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1,
                                         const float (&c)[4])
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}

template <int D_, int NR>
struct Attn {
    static constexpr int DIM = D_;
    static constexpr int JOIN = D_ == 128 ? 16 : 8;   // parts whose outputs a join loads together
    static constexpr bool FOUR = NR == 0;       // four rows, twice in an MMA's eight columns
    static constexpr int G = FOUR ? 1 : NR;     // columns, in eights
    static constexpr int ROWS = FOUR ? 4 : 8 * NR;
    static constexpr int TILES = 2;             // of a unit
    static constexpr int UNIT = 16 * TILES;     // tokens
    static constexpr int OVERHEAD = 12;         // what starting and ending a segment costs, in units (4: 64 ragged requests 105 us, 8: 98, 18: 97)
    static constexpr int CTAS = D_ == 128 ? (NR <= 1 ? 3 : 2) : NR <= 1 ? 4 : 3;   // on an SM, as registers and rings allow
    static constexpr int STAGES = 2;            // units in a warp's ring: one in use and one on its way
    static constexpr int TB = kv8_tile_bytes(D_);
    static constexpr int STAGE = TILES * TB;
    static constexpr int RING = STAGES * STAGE;
    static constexpr int SLABS = D_ / 64;
    static constexpr int PART = ROWS * (D_ + 2); // floats of one partial: O, then m and l
    static_assert(RING >= ROWS * D_ * 4, "a warp's ring holds its output");
    struct Shared : RunShared<ROWS> {
        uint64_t bar[kWarps][STAGES];
    };
    static constexpr int SMEM = kWarps * RING + sizeof(Shared);
};

template <int D, int NR>
__global__ void __launch_bounds__(kThreads, Attn<D, NR>::CTAS) kv8_attn_kernel(const __grid_constant__ Kv4AttnParams p)
{
    using A = Attn<D, NR>;
    constexpr int ROWS = A::ROWS, G = A::G, SLABS = A::SLABS, TILES = A::TILES, UNIT = A::UNIT, OVERHEAD = A::OVERHEAD;
    constexpr bool FOUR = A::FOUR;
    extern __shared__ __align__(128) uint8_t smem[];
    typename A::Shared& sh = *reinterpret_cast<typename A::Shared*>(smem + kWarps * A::RING);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int n = lane >> 2, c = lane & 3;
    uint8_t* const ring = smem + warp * A::RING;
    chained_kernel();

    // ---- this CTA's run of units
    if (lane < A::STAGES) mbar_init(smem_addr(&sh.bar[warp][lane]), 1);
    fence_mbar_init();
    const Units un = units_of<A>(p, sh);
    int b = un.b;
    long long off = un.off;
    if (b >= p.batch) return;   // more CTAs than units
    const long long u0 = un.u0, u1 = un.u1;

    const WaitCtl ctl{&sh.abort_flag, p.status, p.wait_limit_ns};
    // the ring: stage and phase of the next unit to issue and to use; TILES bits a stage: its tiles are stored
    int s_issue = 0, s_use = 0;
    uint32_t phase = 0, pending = 0, ok_bits = 0;
    bool dead = false;
    const int tpp_shift = __ffs(p.page_size) - 5;   // log2(tiles per page)

    Request r = un.r;
    for (long long u = u0; u < u1;) {
        while (off >= r.work) {   // next request with work
            off -= r.work;
            r = request_of<A>(p, ++b);
        }
        const int cost = r.units + OVERHEAD;
        const long long seg = off / cost;
        const int at = (int)(off - seg * cost);                                  // this run's first place in the segment
        const int end = (int)(cost - at < u1 - u ? cost : at + (u1 - u));        // and its end
        const long long seg_u = u - at;                                          // the segment's place among all
        u += end - at;
        off += end - at;
        if (end <= OVERHEAD) continue;                                           // no unit of it is this run's
        const int pos = at > OVERHEAD ? at - OVERHEAD : 0, take = end - OVERHEAD - pos;
        const int head = (int)(seg / r.tiles), rt = (int)(seg - (long long)head * r.tiles);
        const int row0 = rt * ROWS;
        // a unit needs no mask if it lies below the first row's position and inside the last row's window;
        // units that no row of the tile sees are left out: [first, last) of the run are looked at
        const int last_row = (row0 + ROWS < r.rows ? row0 + ROWS : r.rows) - 1;
        const int pos_min = r.pos0 + row0 / p.group, pos_max = r.pos0 + last_row / p.group;
        const int seen = pos_max >= r.base ? (pos_max - r.base) / UNIT + 1 : 0;
        const int low_at = (pos_min > 0 ? pos_min : 0) - p.window + 1;   // as in request_of
        const int low = p.window > 0 && low_at > r.base ? (low_at - r.base) / UNIT : 0;
        const int first = low > pos ? low : pos, last = seen < pos + take ? seen : pos + take;

        // ---- copies: a batch of 32 tiles at a time, a lane each
        constexpr int BATCH = 32 / TILES;   // units
        const int32_t* const trow = p.table + (long long)b * p.table_stride;
        const int mine_n = last > first + warp ? (last - first - warp + kWarps - 1) / kWarps : 0;   // units of this warp: first + warp, + kWarps, ...
        const int tile0 = (r.base >> 4) + (first + warp + lane / TILES * kWarps) * TILES + lane % TILES;   // this lane's of the first batch
        auto page_of = [&](int k) {   // page of this lane's tile of the batch from unit k on, or -1
            const int tile = tile0 + k * kWarps * TILES;
            return (k + lane / TILES < mine_n && tile * kKv4Tile < r.seq) ? trow[tile >> tpp_shift] : -1;
        };
        int k_issue = 0, page = page_of(0);
        uint32_t present = 0;
        const uint8_t* src = nullptr;
        auto issue_next = [&]() {
            if (k_issue >= mine_n || dead) return;
            const int j = k_issue % BATCH;
            if (j == 0) {
                const int in_page = (tile0 + k_issue * kWarps * TILES) & ((1 << tpp_shift) - 1);
                present = __ballot_sync(0xffffffffu, page >= 0 && page < p.pages);
                src = p.cache + ((((long long)page * p.kv_heads + head) << tpp_shift) + in_page) * A::TB;
                page = page_of(k_issue + BATCH);
            }
            constexpr uint32_t MASK = (1u << TILES) - 1u;
            const uint32_t bits = present >> (j * TILES) & MASK;
            ok_bits = (ok_bits & ~(MASK << (s_issue * TILES))) | bits << (s_issue * TILES);
            const uint32_t bar = smem_addr(&sh.bar[warp][s_issue]);
            if (lane == 0) mbar_arrive_expect_tx(bar, __popc(bits) * A::TB);
            if (lane / TILES == j && (bits >> (lane % TILES) & 1u))
                bulk_load(smem_addr(ring + s_issue * A::STAGE + lane % TILES * A::TB), src, A::TB, bar);
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

        // ---- Q fragments, scaled per row by a power of two; row constants of the columns 2c, 2c + 1. Word w of slab s of a
        // token's share are its d = 64 s + 16 c + 4 w + 0 .. 3, even ones first
        uint32_t qf[G][SLABS * 4][2];
        float row_a[G][2], row_z[G][2];   // score = row_a * s_k * (MMA from row_z), in powers of two
#pragma unroll
        for (int g = 0; g < G; ++g) {
            const int row = row0 + g * 8 + (FOUR ? n & 3 : n);
            uint32_t raw[8 * SLABS];
#pragma unroll
            for (int i = 0; i < 8 * SLABS; ++i) raw[i] = 0;
            if (row < r.rows) {
                const int qi = row / p.group, h = row - qi * p.group;
                const uint16_t* q = (const uint16_t*)p.q + (long long)(r.q0 + qi) * p.q_token +
                                    (long long)(head * p.group + h) * p.q_head + c * 16;
#pragma unroll
                for (int i = 0; i < 2 * SLABS; ++i) {
                    const uint4 v = *reinterpret_cast<const uint4*>(q + (i >> 1) * 64 + (i & 1) * 8);
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
            for (int i = 0; i < 8 * SLABS; ++i) top = fmaxf(top, fmaxf(fabsf(lo_of(raw[i])), fabsf(hi_of(raw[i]))));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            // largest magnitude into [2^13, 2^14); an infinity or a NaN stays one
            int e = ((__float_as_int(top) >> 23) & 255) - 127 - 13;
            e = (top == 0.0f || !(top <= FLT_MAX)) ? 0 : e < -120 ? -120 : e;
            // a negative softmax scale goes into Q, so that the largest score is that of the largest product
            const float f = p.scale_log2 < 0.0f ? -pow2i(-e) : pow2i(-e);
            float qsum = 0.0f;
#pragma unroll
            for (int w = 0; w < 4 * SLABS; ++w) {
                qf[g][w][0] = half2_bits(lo_of(raw[2 * w]) * f, lo_of(raw[2 * w + 1]) * f);
                qf[g][w][1] = half2_bits(hi_of(raw[2 * w]) * f, hi_of(raw[2 * w + 1]) * f);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float2 a = bits_half2(qf[g][w][i]);
                    qsum += a.x + a.y;
                }
            }
            qsum += __shfl_xor_sync(0xffffffffu, qsum, 1);
            qsum += __shfl_xor_sync(0xffffffffu, qsum, 2);
            // codes come as c * 2^-24
            const float unit = fabsf(p.scale_log2) * pow2i(e > 103 ? 103 : e) * 16777216.0f;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float un_i = __shfl_sync(0xffffffffu, unit, (2 * c + i) * 4);
                row_a[g][i] = un_i > 0.0f ? un_i : FLT_MIN;   // scale 0: all scores nearly equal, masked ones stay -infinity
                row_z[g][i] = __shfl_sync(0xffffffffu, qsum, (2 * c + i) * 4) * -0x1p-17f;   // 128 * 2^-24
            }
        }
        float m[G][2], l[G][2], o[G][4 * SLABS][4];
#pragma unroll
        for (int g = 0; g < G; ++g) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                m[g][i] = -CUDART_INF_F;
                l[g][i] = 0.0f;
            }
#pragma unroll
            for (int w = 0; w < 4 * SLABS; ++w)
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
            const uint32_t have = ok_bits >> (s_use * TILES) & ((1u << TILES) - 1u);
            const int t0 = r.base + t * UNIT;
            const bool full = have == (1u << TILES) - 1u && t0 + UNIT - 1 <= pos_min && (p.window <= 0 || t0 > pos_max - p.window);

            // scores in powers of two: of each tile tokens n and n + 8, rows 2c and 2c + 1; two chains of MMAs, of even and odd words.
            // They are rounded before a reference is taken off, which is one of them, so that the largest weight is one however large they are
            float sc[TILES][G][4], sv[TILES];
#pragma unroll
            for (int tl = 0; tl < TILES; ++tl) {
                const uint8_t* const tile = st + tl * A::TB;
                const float2 scales = *reinterpret_cast<const float2*>(tile + kv8_k_scale_off(D));
                sv[tl] = scales.y;
                float odd_sc[G][4];
#pragma unroll
                for (int g = 0; g < G; ++g)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        sc[tl][g][i] = row_z[g][i & 1];
                        odd_sc[g][i] = 0.0f;
                    }
#pragma unroll
                for (int s = 0; s < SLABS; ++s) {
                    const uint4 ka4 = *reinterpret_cast<const uint4*>(tile + s * 1024 + lane * 16);
                    const uint4 kb4 = *reinterpret_cast<const uint4*>(tile + s * 1024 + 512 + lane * 16);
                    const uint32_t ka[4] = {ka4.x, ka4.y, ka4.z, ka4.w}, kb[4] = {kb4.x, kb4.y, kb4.z, kb4.w};
#pragma unroll
                    for (int w = 0; w < 4; ++w)
#pragma unroll
                        for (int g = 0; g < G; ++g)
                            mma_16816(w & 1 ? odd_sc[g] : sc[tl][g], ka[w] & kEven, kb[w] & kEven, odd_bytes(ka[w]), odd_bytes(kb[w]),
                                      qf[g][4 * s + w][0], qf[g][4 * s + w][1]);
                }
#pragma unroll
                for (int g = 0; g < G; ++g)
#pragma unroll
                    for (int i = 0; i < 4; ++i) sc[tl][g][i] = (sc[tl][g][i] + odd_sc[g][i]) * (scales.x * row_a[g][i & 1]);
            }
            if (!full) {
#pragma unroll
                for (int tl = 0; tl < TILES; ++tl) {
                    const bool there = have >> tl & 1u, odd = there && sv[tl] != sv[tl];   // a poisoned tile of V
                    if (!there || odd) sv[tl] = 0.0f;
#pragma unroll
                    for (int g = 0; g < G; ++g)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int row = row0 + g * 8 + (FOUR ? 2 * (c & 1) + i : 2 * c + i);
                            const int row_pos = row < r.rows ? r.pos0 + row / p.group : -1;
                            bool sees = false;
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                const int key = t0 + 16 * tl + n + 8 * j;
                                const bool see = there && key < r.seq && key <= row_pos && (p.window <= 0 || key > row_pos - p.window);
                                if (!see) sc[tl][g][2 * j + i] = -CUDART_INF_F;
                                sees = sees || see;
                            }
                            // a poisoned tile shows in the rows that see some of it alone
                            if (odd && (__ballot_sync(0xffffffffu, sees) >> c & 0x11111111u))
#pragma unroll
                                for (int w = 0; w < 4 * SLABS; ++w) o[g][w][i] = o[g][w][2 + i] = CUDART_NAN_F;
                        }
                }
            }
            auto largest = [&](int g, int i) {
                static_assert(TILES == 2, "both tiles' scores");
                return fmaxf(fmaxf(sc[0][g][i], sc[0][g][2 + i]), fmaxf(sc[1][g][i], sc[1][g][2 + i]));
            };
            // the references of the running sums move if a score passes its row's by 2^kGrow
            bool grow = false;
#pragma unroll
            for (int g = 0; g < G; ++g)
#pragma unroll
                for (int i = 0; i < 2; ++i) grow = grow || largest(g, i) - m[g][i] > (float)kGrow;
            if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                for (int g = 0; g < G; ++g) {
                    float f[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        float x = largest(g, i);
                        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
                        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
                        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
                        x = fmaxf(x, m[g][i]);
                        f[i] = x == m[g][i] ? 1.0f : ex2(m[g][i] - x);
                        m[g][i] = x;
                        l[g][i] *= f[i];
                    }
#pragma unroll
                    for (int w = 0; w < 4 * SLABS; ++w)
#pragma unroll
                        for (int i = 0; i < 4; ++i) o[g][w][i] *= f[i & 1];
                }
            }
            float ref[G][2];
#pragma unroll
            for (int g = 0; g < G; ++g)
#pragma unroll
                for (int i = 0; i < 2; ++i) ref[g][i] = m[g][i] == -CUDART_INF_F ? 0.0f : m[g][i];
#pragma unroll
            for (int tl = 0; tl < TILES; ++tl) {
                // probabilities, fed below 2^15, clear of subnormals, and -128 times their sum, the same in every row of d
                uint32_t ph[G][2], pl[G][2];
                float z[G][4];
#pragma unroll
                for (int g = 0; g < G; ++g) {
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        float pv[2];
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const float e = ex2(sc[tl][g][2 * j + i] - ref[g][i]);
                            l[g][i] += e;
                            pv[i] = e * (float)(1 << (15 - kGrow));
                        }
                        const uint32_t h = half2_bits(pv[0], pv[1]);
                        const float2 back = bits_half2(h);
                        const uint32_t rest = half2_bits(pv[0] - back.x, pv[1] - back.y);
                        if constexpr (FOUR) {
                            ph[g][j] = transpose8(c < 2 ? h : rest);   // the second four columns are the low parts
                        } else {
                            ph[g][j] = transpose8(h);
                            pl[g][j] = transpose8(rest);
                        }
                    }
                    const float none[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                    mma_from(z[g], kMiddle, kMiddle, kMiddle, kMiddle, ph[g][0], ph[g][1], none);
                    if constexpr (!FOUR) mma_16816(z[g], kMiddle, kMiddle, kMiddle, kMiddle, pl[g][0], pl[g][1]);
                }
                const uint64_t sv2 = pack_f32x2(sv[tl], sv[tl]);
                const uint8_t* const vt = st + tl * A::TB + kv8_v_off(D) + lane * 16;
#pragma unroll
                for (int s = 0; s < SLABS; ++s) {
                    const uint4 va4 = *reinterpret_cast<const uint4*>(vt + s * 1024);
                    const uint4 vb4 = *reinterpret_cast<const uint4*>(vt + s * 1024 + 512);
                    const uint32_t va[4] = {va4.x, va4.y, va4.z, va4.w}, vb[4] = {vb4.x, vb4.y, vb4.z, vb4.w};
#pragma unroll
                    for (int w = 0; w < 4; ++w)
#pragma unroll
                        for (int g = 0; g < G; ++g) {
                            float d[4];
                            mma_from(d, va[w] & kEven, odd_bytes(va[w]), vb[w] & kEven, odd_bytes(vb[w]), ph[g][0], ph[g][1], z[g]);
                            if constexpr (!FOUR) mma_16816(d, va[w] & kEven, odd_bytes(va[w]), vb[w] & kEven, odd_bytes(vb[w]), pl[g][0], pl[g][1]);
                            float(&to)[4] = o[g][4 * s + w];
#pragma unroll
                            for (int i = 0; i < 4; i += 2)
                                unpack_f32x2(fma_f32x2(pack_f32x2(d[i], d[i + 1]), sv2, pack_f32x2(to[i], to[i + 1])), to[i], to[i + 1]);
                        }
                }
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
        constexpr float kOut = 16777216.0f / (1 << (15 - kGrow));   // codes come as c * 2^-24
#pragma unroll
        for (int g = 0; g < G; ++g) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) l[g][i] += __shfl_xor_sync(0xffffffffu, l[g][i], d);
                if (n == 0 && (!FOUR || c < 2)) {
                    sh.m[warp][g * 8 + 2 * c + i] = m[g][i];
                    sh.l[warp][g * 8 + 2 * c + i] = l[g][i];
                }
            }
            if constexpr (FOUR) {   // low and high parts of the probabilities
#pragma unroll
                for (int w = 0; w < 4 * SLABS; ++w)
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[g][w][i] += __shfl_xor_sync(0xffffffffu, o[g][w][i], 2);
            }
#pragma unroll
            for (int w = 0; w < 4 * SLABS; w += 2)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    if (FOUR && c >= 2) continue;
                    float4 x;   // d = 64 s + 8 n + 2 w .. of the slab's words w and w + 1
                    x.x = o[g][w][i] * kOut;
                    x.y = o[g][w][2 + i] * kOut;
                    x.z = o[g][w + 1][i] * kOut;
                    x.w = o[g][w + 1][2 + i] * kOut;
                    *reinterpret_cast<float4*>(mine + (g * 8 + 2 * c + i) * D + (w >> 2) * 64 + n * 8 + 2 * (w & 3)) = x;
                }
        }
        __syncthreads();
        finish_segment<A>(p, smem, sh, r, head, row0, pos, take, seg_u);
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
        cudaError_t e = cudaFuncSetAttribute(kv8_attn_kernel<D, NR>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             Attn<D, NR>::SMEM);
        if (e != cudaSuccess) return e;
        return cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kv8_attn_kernel<D, NR>, kThreads, Attn<D, NR>::SMEM);
    }

    static cudaError_t run(const Kv4AttnParams& p, int sms, cudaStream_t stream)
    {
        return launch_chained(kv8_attn_kernel<D, NR>, grid_of(sms), kThreads, Attn<D, NR>::SMEM, 1, stream, p);
    }
};
}  // namespace

size_t kv8_partial_bytes(int sms)
{
    size_t need = kv8_prompt_partial_bytes(sms);
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
    most(Launch<128, 3>::grid_of(sms), Attn<128, 3>::PART);
    return need;
}

cudaError_t setup_kv8_attention()
{
    cudaError_t e;
    if ((e = Launch<64, 0>::setup()) != cudaSuccess || (e = Launch<128, 0>::setup()) != cudaSuccess ||
        (e = Launch<64, 1>::setup()) != cudaSuccess || (e = Launch<64, 2>::setup()) != cudaSuccess ||
        (e = Launch<128, 1>::setup()) != cudaSuccess || (e = Launch<128, 2>::setup()) != cudaSuccess ||
        (e = Launch<128, 3>::setup()) != cudaSuccess)
        return e;
    return setup_kv8_prompt();
}

// The tcgen05 kernel takes requests of more than kFewRows rows a KV head where the batch's rows fill the GPU with its tiles of 256, but
// no batch whose requests all have few enough rows that such a tile is mostly empty. Which request has how many is known on the
// device, so other batches get both kernels. tcgen05 and stream-K, us: one request, D = 128, over 4000 tokens, 2048 rows 49 / 43,
// 2400 49 / 47, 2816 49 / 51, 4096 48 / 69, 8192 47 / 112; over 300 tokens 3200 13 / 24, over 1000 33 / 31; D = 64, 2048 over 4000 26 / 28,
// 2400 27 / 29, 4096 31 / 44, 8192 36 / 70; over 300 tokens 3200 11 / 15, over 1000 23 / 20. 48 requests over 4000 tokens of 4 KV heads,
// 36, 48, 64, 72, 128 rows a KV head: D = 128 154 / 128, 130, 161, 183, 297; D = 64 142 / 75, 80, 103, 125, 190. (How many tokens are
// cached is not known on the host: 2048 rows over 16000 would be 70 / 108, D = 64 47 / 67.)
// Between these, requests of 8 KV heads, over 400, 1000 and 4000 tokens, D = 128: four of 96 rows 17 / 25, 37 / 30, 53 / 54, of
// 128 17 / 24, 37 / 30, 53 / 63; eight of 40 18 / 24, 37 / 30, 64 / 53, of 64 18 / 24, 27 / 30, 79 / 63, of 96 18 / 32, 28 /
// 43, 80 / 92; 16 of 40 18 / 31, 28 / 41, 85 / 92, of 64 18 / 33, 28 / 45, 84 / 113. D = 64: four of 128 14 / 16, 25 / 23, 41 /
// 45; eight of 64 15 / 18, 24 / 22, 75 / 45, of 96 15 / 22, 24 / 26, 75 / 57, of 128 15 / 23, 24 / 31, 75 / 71; 16 of 96 16 /
// 29, 25 / 41, 76 / 102. So the rule takes the slower kernel by up to 1.26 times where it takes tcgen05 (eight of 64 over 4000;
// one or two requests of few blocks over 1000), and by up to 1.8 where it does not (16 of 40 rows, or of 96 with D = 64, over
// 400). Both limits are times alone, and they decide a precision: with bfloat16 outputs the tcgen05 kernel feeds weights in 11
// bits, the stream-K kernel in 22 (errors against 64 bits 1% larger, of which an output's rounding is the rest).
constexpr int kFewRows = 32;
constexpr int sparse_rows(int head_dim) { return head_dim == 128 ? 60 : 96; }
constexpr long long kPromptRows = 2400;

// Rows of a segment, in eights (0: four), where requests have up to `held` rows a KV head and the batch has `all`. Of few rows segments
// of eight are the fastest: latency counts. Otherwise what the segments cost together decides. 64 requests over 4000 tokens of 4
// KV heads, segments of 8 / 16 / 24 rows, us: D = 128, 16 rows 68 / 65 / 88, 24 rows 126 / 111 / 94, 32 rows 140 / 114 / 161;
// D = 64, 16 rows 46 / 47, 24 rows 63 / 71, 32 rows 81 / 73 (24 rows gained 5% at 24 and lost elsewhere). Eight requests of 32 rows
// over 4000 tokens: 27 / 32 / 42 and 19 / 21.
int segment_rows(long long held, int head_dim, long long all)
{
    if (held <= 4) return 0;
    const long long eights = (held + 7) / 8;
    if (all <= 1024 || eights == 1) return 1;
    if (head_dim == 64) return 36 * ((eights + 1) / 2) < 19 * eights ? 2 : 1;
    const long long cost[3] = {35 * eights, 57 * ((eights + 1) / 2), 78 * ((eights + 2) / 3)};
    return cost[2] < cost[0] && cost[2] < cost[1] ? 3 : cost[1] < cost[0] ? 2 : 1;
}

cudaError_t launch_kv8_attention(const Kv4AttnParams& in, int head_dim, int max_q, int path, int sms, cudaStream_t stream)
{
    Kv4AttnParams p = in;
    const long long rows = (long long)max_q * p.group;
    const bool prompt = path != 1 && (path == 2 ? rows > kFewRows
                                                : rows > sparse_rows(head_dim) && (long long)p.tokens * p.q_heads >= kPromptRows);
    if (prompt && p.batch == 1) {   // one request is one kernel's, whatever its rows turn out to be
        p.few_rows = 0;
        return launch_kv8_prompt(p, head_dim, sms, stream);
    }
    p.few_rows = prompt ? kFewRows : INT_MAX;
    // of a request that is this kernel's, at most; beside prompts it is a single token's more often than not (two prompts of 800 new
    // tokens behind 1200 with 30 single tokens over 8000, 8 KV heads, four query heads to each: 182 -> 172 us, D = 64 131 -> 114; 154 and 103
    // since the prompt kernel is faster. The single tokens' bytes are 73 us of it, the prompts' products 22)
    const long long held = !prompt ? rows : p.group < 8 ? 8 : p.group < kFewRows ? p.group : kFewRows;
    const int nr = segment_rows(held, head_dim, (long long)p.tokens * p.q_heads);
    cudaError_t e;
    if (head_dim == 128)
        e = nr == 0 ? Launch<128, 0>::run(p, sms, stream) : nr == 1 ? Launch<128, 1>::run(p, sms, stream)
          : nr == 2 ? Launch<128, 2>::run(p, sms, stream) : Launch<128, 3>::run(p, sms, stream);
    else
        e = nr == 0 ? Launch<64, 0>::run(p, sms, stream) : nr == 1 ? Launch<64, 1>::run(p, sms, stream) : Launch<64, 2>::run(p, sms, stream);
    if (e != cudaSuccess || !prompt) return e;
    return launch_kv8_prompt(p, head_dim, sms, stream);
}

}  // namespace w4a16
