// Sampling of one token per row of logits with temperature, top-k, top-p and min-p, from
// given uniform numbers.
//
// With m the row's maximum and r = 1 / T, a token's weight is the whole number
//   w = rint(2^31 exp((x - m) r)),
// so every sum below is exact in 64 bits and the same in any order, and a row's token
// depends neither on the launch shape nor on a race between atomics. Tokens are ranked by
// (x descending, index ascending). top-k keeps ranks below k; top-p keeps a token
// if the weight ranked before it is below p times the weight of the top-k set; min-p
// keeps exp((x - m) r) >= min_p; rank 0 is always kept. The token is the first, in index
// order, whose running kept weight passes floor(u * total).
//
// A cluster of CTAs shares one row, each CTA a slice, which it reads once from HBM and then
// from L2: a slice kept in shared memory leaves room for too few CTAs on an SM to hide
// the barriers between a row's steps (256 x 100003 FP32 with slices in shared memory took 193 us
// where it took 93 otherwise). Once the first CTA has what the others found, they leave.
// The kept set is a prefix of the ranking, so it is one cut: the last kept token's
// logit and index. Ways to the cut, by what a row asks for:
//  - top-k of up to kListMax / 2: the k-th largest of the maxima of groups of tokens (four a
//    thread; found by a histogram of them) is below at least k tokens and, as a group has few
//    tokens, not many more; those are listed, and one CTA does the rest on the list;
//  - top-p alone: a histogram of the weights over 1024 bins of (m - x) r, which spreads logits
//    evenly where their bits would not (fewer conflicts of shared atomics), finds the bin that
//    holds the cut, and the tokens of that bin are listed and cut by one CTA;
//  - a larger k, or a bin with more tokens than a list holds (many equal logits): histograms
//    of counts and weights over the keys inside the bin, ten bits at a time.
// A list is never sorted: up to 128 entries are compared with each other; of more, the entry at
// which a running count or weight crosses a limit is found by histograms over its keys, which are
// all different (logit, then index), and so is the drawn token of a top-k row (keys: indices). Every other row sums the kept weights of each
// warp's segment, in index order, and the segment that holds the drawn place looks it up.
// Vectors whose largest logit is below what a pass looks for are skipped, at about one
// instruction a token; a weight takes about 20.
//
// Bound by the chain of a row's steps (barriers of the CTA and the cluster, about 1 us each under load), a
// weight's instructions where weights are summed, and shared atomics where they are binned: 128 rows of 131072
// bfloat16 logits take 17 us greedy, 33 with no filter or top-k 50, 42 with top-k 500, 84 with top-p 0.95 alone,
// and 45 mixed; one row of 32000 9.6 us.
#include "launch.cuh"
#include "ptx.cuh"
#include "sample.cuh"
#include "w4a16.h"

#include <cooperative_groups.h>
#include <float.h>
#include <math_constants.h>

namespace w4a16 {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 1024;
constexpr int kPer = kBins / kThreads;   // bins a thread adds up
constexpr int kMaxCluster = 8;
constexpr int kMaxSlice = 65536;         // tokens of a CTA's slice
constexpr float kSpan = 22.2f;           // exp(-22.2) * 2^31 rounds to 0

constexpr int kListMax = 2048;           // tokens of a list
constexpr int kListMine = kListMax / 2;  // of them, one CTA's share at most
constexpr int kListPer = kListMax / kThreads;
constexpr int kIndexBits = 18;
constexpr uint32_t kIndexTop = (1u << kIndexBits) - 1u;
static_assert(kSampleMaxVocab <= 1 << kIndexBits, "an entry holds a token's index");
constexpr int kFew = kThreads / 4;       // entries that are compared with each other, four threads an entry
constexpr int kGroups = 4;               // groups of a thread's tokens, each with its maximum

struct Histogram {
    uint32_t cnt[kBins], part[2][kBins];   // a bin's count, and its weights' bits 0..15 and 16..31 summed
};

struct Shared {
    Histogram bins;                      // over (m - x) r
    Histogram keys;                      // over keys
    unsigned long long list[kListMine];  // key, then the index from the top of kIndexBits down: greater is ranked before
    unsigned long long best[kWarps];
    unsigned long long range;            // what this CTA shows to the cluster: least and greatest key,
    float top;                           // its maximum,
    uint32_t listed;                     // the length of its list,
    unsigned long long cut;              // and, of the first CTA, the cut
    unsigned long long scan_mass[kWarps];
    uint32_t scan_cnt[kWarps];
    unsigned long long warp_mass[kWarps];   // kept weight of each warp's segment
    unsigned long long all_mass[kMaxCluster * kWarps];
    // results of a search
    int bin;
    uint32_t base_cnt, bin_cnt;
    unsigned long long base_mass, bin_mass, total;
    unsigned long long limit;            // what a search compares with
    unsigned long long picked, picked_before;
    uint32_t picked_weight;
    uint32_t few;                        // entries of a bin that a warp looks through
    // the chosen segment
    int seg;
    unsigned long long seg_target;
};

// A 16-byte vector's elements: their type, bits as a float, and the largest of them (NaN aside).
template <int DTYPE>
struct Elem;
template <>
struct Elem<W4A16_FP32> {
    using T = float;
    static constexpr int kShift = 0;
    static __device__ __forceinline__ float get(uint32_t bits) { return __uint_as_float(bits); }
    static __device__ __forceinline__ float largest(const uint4& v)
    {
        return fmaxf(fmaxf(__uint_as_float(v.x), __uint_as_float(v.y)), fmaxf(__uint_as_float(v.z), __uint_as_float(v.w)));
    }
};
template <>
struct Elem<W4A16_FP16> {
    using T = uint16_t;
    static constexpr int kShift = 13;
    static __device__ __forceinline__ float get(uint32_t bits) { return __half2float(__ushort_as_half((uint16_t)bits)); }
    static __device__ __forceinline__ float largest(const uint4& v)
    {
        auto h = [](const uint32_t& w) { return *reinterpret_cast<const __half2*>(&w); };
        const __half2 m = __hmax2(__hmax2(h(v.x), h(v.y)), __hmax2(h(v.z), h(v.w)));
        return __half2float(__hmax(__low2half(m), __high2half(m)));
    }
};
template <>
struct Elem<W4A16_BF16> {
    using T = uint16_t;
    static constexpr int kShift = 16;
    static __device__ __forceinline__ float get(uint32_t bits) { return __uint_as_float(bits << 16); }
    static __device__ __forceinline__ float largest(const uint4& v)
    {
        auto h = [](const uint32_t& w) { return *reinterpret_cast<const __nv_bfloat162*>(&w); };
        const __nv_bfloat162 m = __hmax2(__hmax2(h(v.x), h(v.y)), __hmax2(h(v.z), h(v.w)));
        return fmaxf(__low2float(m), __high2float(m));
    }
};

// Whole numbers in the order of x (-inf lowest among numbers); equal exactly where x is equal.
template <int DTYPE>
__device__ __forceinline__ uint32_t key_of(float x)
{
    const uint32_t b = __float_as_uint(x + 0.0f);   // -0 as +0
    return (b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u)) >> Elem<DTYPE>::kShift;
}

struct Row {
    float top, inv, min_p;
};

__device__ __forceinline__ float scaled(float x, const Row& r) { return __fmul_rn(__fsub_rn(x, r.top), r.inv); }

__device__ __forceinline__ float exp_of(float x, const Row& r)
{
    const float e = expf(scaled(x, r));
    return x == r.top ? 1.0f : e;
}

__device__ __forceinline__ uint32_t weight_of(float e) { return __float2uint_rn(e * 2147483648.0f); }

// A logit's bin, before truncation: kBins or more past kSpan.
__device__ __forceinline__ float place(float x, const Row& r) { return x == r.top ? 0.0f : scaled(x, r) * (-kBins / kSpan); }

// The whole part of a number in 0 .. kBins, without the conversion unit that the weights keep busy.
__device__ __forceinline__ int whole(float at) { return (int)(__float_as_uint(__fadd_rz(at, 8388608.0f)) & (2u * kBins - 1u)); }

__device__ __forceinline__ int bin_of(float x, const Row& r) { return whole(fminf(place(x, r), (float)(kBins - 1))); }

// Sums of 64-bit numbers over a warp.
__device__ __forceinline__ unsigned long long warp_sum(unsigned long long v)
{
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    return v;
}

template <typename T>
__device__ __forceinline__ T warp_incl(T v, int lane)
{
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const T o = __shfl_up_sync(0xffffffffu, v, d);
        if (lane >= d) v += o;
    }
    return v;
}

__device__ __forceinline__ void clear(Histogram& h)
{
    uint4* const at = reinterpret_cast<uint4*>(&h);
    for (int i = threadIdx.x; i < (int)(sizeof(Histogram) / 16); i += kThreads) at[i] = make_uint4(0, 0, 0, 0);
}

// 32 bits hold the low parts of kMaxSlice weights, and as many high parts: a weight is at most 2^31.
__device__ __forceinline__ void add_mass(Histogram& h, int bin, uint32_t w)
{
    atomicAdd(&h.part[0][bin], w & 0xffffu);
    if (w >= 1u << 16) atomicAdd(&h.part[1][bin], w >> 16);
}

__device__ __forceinline__ unsigned long long mass_of(uint32_t a, uint32_t b) { return a + ((unsigned long long)b << 16); }

// The least whole number that is not below a share of a weight: m < limit_of(...) is (double)m < (double)total * share.
// 64-bit floating point is slow here, so one thread does it for a search, and the search compares whole numbers.
__device__ __forceinline__ unsigned long long limit_of(unsigned long long total, float share)
{
    return __double2ull_ru((double)total * (double)share);
}

// Finds the first bin with done(count, weight of every bin up to and with it, limit), from each thread's two bins;
// base counts come on top. MASS: weights count, else only counts do. The limit is bound(weight of all bins). Leaves
// bin = -1 if there is none; sh.bin is -1 on entry, and a barrier lies between that and here.
template <bool MASS, typename F, typename B>
__device__ __forceinline__ void scan_bins(Shared& sh, const uint32_t (&cnt)[kPer], const unsigned long long (&mass)[kPer],
                                          uint32_t base_cnt, unsigned long long base_mass, F done, B bound)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t ic = warp_incl(cnt[0] + cnt[1], lane);
    const unsigned long long im = MASS ? warp_incl(mass[0] + mass[1], lane) : 0ull;
    if (lane == 31) {
        sh.scan_cnt[warp] = ic;
        if (MASS) sh.scan_mass[warp] = im;
    }
    __syncthreads();
    static_assert(kWarps <= 32, "a warp scans the warps' sums");
    const uint32_t wc = warp_incl(lane < kWarps ? sh.scan_cnt[lane] : 0u, lane);
    uint32_t c = base_cnt + __shfl_sync(0xffffffffu, wc, warp > 0 ? warp - 1 : 0) * (warp > 0) + ic - cnt[0] - cnt[1];
    unsigned long long m = base_mass, all = base_mass;
    if (MASS) {
        const unsigned long long wm = warp_incl(lane < kWarps ? sh.scan_mass[lane] : 0ull, lane);
        const unsigned long long upto = __shfl_sync(0xffffffffu, wm, warp > 0 ? warp - 1 : 0);
        m += (warp > 0 ? upto : 0ull) + im - mass[0] - mass[1];
        all += __shfl_sync(0xffffffffu, wm, 31);
        if (threadIdx.x == 0) sh.total = all;
    }
    const unsigned long long limit = bound(all);
    bool before = done(c, m, limit);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const bool now = done(c + cnt[i], m + mass[i], limit);
        if (now && !before) {
            sh.bin = threadIdx.x * kPer + i;
            sh.base_cnt = c;
            sh.base_mass = m;
            sh.bin_cnt = cnt[i];
            sh.bin_mass = mass[i];
        }
        before = now;
        c += cnt[i];
        m += mass[i];
    }
    __syncthreads();
}

// scan_bins over the sum of the cluster's histograms; every CTA finds the same. A cluster barrier before
// (the histograms are complete) is in here; the caller keeps one between this and the next use of the histogram.
template <bool MASS, typename F, typename B>
__device__ __forceinline__ void search(cg::cluster_group& cl, Shared& sh, Histogram& hist, uint32_t base_cnt,
                                       unsigned long long base_mass, F done, B bound)
{
    if (threadIdx.x == 0) sh.bin = -1;
    cl.sync();
    static_assert(kPer == 2, "two bins a thread");
    uint32_t cnt[kPer] = {0, 0};
    unsigned long long mass[kPer] = {0, 0};
    const int ctas = (int)cl.num_blocks();
    const int at = threadIdx.x * kPer;
#pragma unroll
    for (int two = 0; two < kMaxCluster; two += 2) {   // two CTAs' loads in flight at a time
        if (two >= ctas) break;
        uint2 a[2], b[2][2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            a[k] = b[k][0] = b[k][1] = make_uint2(0, 0);
            if (two + k < ctas) {
                const Histogram* o = cl.map_shared_rank(&hist, two + k);
                a[k] = *reinterpret_cast<const uint2*>(&o->cnt[at]);
#pragma unroll
                for (int q = 0; q < 2; ++q)
                    if (MASS) b[k][q] = *reinterpret_cast<const uint2*>(&o->part[q][at]);
            }
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            cnt[0] += a[k].x;
            cnt[1] += a[k].y;
            if (MASS) {
                mass[0] += mass_of(b[k][0].x, b[k][1].x);
                mass[1] += mass_of(b[k][0].y, b[k][1].y);
            }
        }
    }
    scan_bins<MASS>(sh, cnt, mass, base_cnt, base_mass, done, bound);
}

// In one CTA: of this thread's entries (0: none; all others different and in kmin .. kmax), the one at which
// done(count, weight of every entry from the greatest key down to it, limit) becomes true, in sh.picked (0 if there is
// none), with what is before it and its weight; the limit is bound(), by one thread. Ten bits of the keys' range at a time, until a bin has one entry.
template <typename F, typename B>
__device__ __forceinline__ void pick(Shared& sh, const unsigned long long (&key)[kListPer], const uint32_t (&w)[kListPer],
                                     unsigned long long kmin, unsigned long long kmax, unsigned long long base_mass, F done, B bound)
{
    const int tid = threadIdx.x;
    __syncthreads();   // what was picked before has been read
    if (tid == 0) {
        sh.picked = 0;
        sh.limit = bound();
    }
    uint32_t base_cnt = 0;
    for (int level = 0; level < 7; ++level) {
        const unsigned long long range = kmax - kmin;
        const int bits = 64 - __clzll((long long)range);
        const int shift = bits > 10 ? bits - 10 : 0;
#pragma unroll
        for (int b = tid; b < kBins; b += kThreads)
            sh.keys.cnt[b] = sh.keys.part[0][b] = sh.keys.part[1][b] = 0;
        if (tid == 0) {
            sh.bin = -1;
            sh.few = 0;
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kListPer; ++i)
            if (key[i] != 0 && key[i] >= kmin && key[i] <= kmax) {
                const int b = (int)((kmax - key[i]) >> shift);
                atomicAdd(&sh.keys.cnt[b], 1u);
                add_mass(sh.keys, b, w[i]);
            }
        __syncthreads();
        uint32_t cnt[kPer];
        unsigned long long mass[kPer];
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int b = tid * kPer + i;
            cnt[i] = sh.keys.cnt[b];
            mass[i] = mass_of(sh.keys.part[0][b], sh.keys.part[1][b]);
        }
        scan_bins<true>(sh, cnt, mass, base_cnt, base_mass, done, [&](unsigned long long) { return sh.limit; });
        if (sh.bin < 0) break;
        base_cnt = sh.base_cnt;
        base_mass = sh.base_mass;
        kmax -= (unsigned long long)sh.bin << shift;
        const unsigned long long low = kmax - ((1ull << shift) - 1ull);
        kmin = low > kmin && low <= kmax ? low : kmin;
        const uint32_t left = sh.bin_cnt;
        if (left > 32) {
            __syncthreads();
            continue;
        }
        // few entries in the bin: a warp ranks them
        unsigned long long* const keys = reinterpret_cast<unsigned long long*>(sh.keys.part[0]);   // the bins have been read
        uint32_t* const ws = sh.keys.part[1];
#pragma unroll
        for (int i = 0; i < kListPer; ++i)
            if (key[i] != 0 && key[i] >= kmin && key[i] <= kmax) {
                const uint32_t at = left > 1 ? atomicAdd(&sh.few, 1u) : 0u;
                keys[at] = key[i];
                ws[at] = w[i];
            }
        __syncthreads();
        if (tid < 32) {
            const int lane = tid;
            const unsigned long long own = lane < (int)left ? keys[lane] : 0ull;
            const uint32_t own_w = lane < (int)left ? ws[lane] : 0u;
            const unsigned long long limit = sh.limit;
            uint32_t c = base_cnt;
            unsigned long long m = base_mass;
            for (int o = 0; o < (int)left; ++o) {
                const bool ahead = keys[o] > own;
                c += ahead;
                m += ahead ? ws[o] : 0u;
            }
            if (own != 0 && done(c + 1, m + own_w, limit) && !done(c, m, limit)) {
                sh.picked = own;
                sh.picked_before = m;
                sh.picked_weight = own_w;
            }
        }
        break;
    }
    __syncthreads();
}

template <int DTYPE>
__device__ __forceinline__ float float_of(uint32_t key)
{
    const uint32_t k = key << Elem<DTYPE>::kShift;
    // positive numbers had their top bit set, negative ones were complemented
    return (k & 0x80000000u) ? __uint_as_float(k & 0x7fffffffu)
                             : __uint_as_float(~(k | ((1u << Elem<DTYPE>::kShift) - 1u)));
}

// What a row asks for.
struct Settings {
    float temp, top_p, min_p;
    int k;
    __device__ __forceinline__ bool greedy() const { return !(temp > 0.0f) || k == 1 || !(top_p > 0.0f) || !(min_p <= 1.0f); }
    __device__ __forceinline__ bool need_k(int vocab) const { return k > 0 && k < vocab; }
    __device__ __forceinline__ bool need_p() const { return top_p < 1.0f; }
    // The longest first: a cut without a list of top-k's, a long list, a short one or the sum of all weights, the maximum.
    __device__ __forceinline__ int turn(int vocab) const
    {
        return greedy() ? 3 : need_k(vocab) ? (k > kListMax / 2 ? 0 : k > kFew / 2 ? 1 : 2) : need_p() ? 0 : 2;
    }
};

__device__ __forceinline__ Settings settings_of(const SampleParams& p, int row)
{
    return {p.temperature ? p.temperature[row] : 1.0f, p.top_p ? p.top_p[row] : 1.0f, p.min_p ? p.min_p[row] : 0.0f,
            p.top_k ? p.top_k[row] : 0};
}

// The row that is number `at` when rows are taken in order of their turns (batches of more than a wave:
// a long row begun last would leave the GPU waiting for it; 128 x 131072: 66 -> 55 us when it came in).
__device__ __forceinline__ int row_in_turn(const SampleParams& p, Shared& sh, int at)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (p.batch <= kThreads) {   // a row a thread: its place is the rows of earlier turns, and those of its own before it
        constexpr int kTurns = 4;
        static_assert(kTurns * kWarps == 64, "two counts a lane");
        const int turn = tid < p.batch ? settings_of(p, tid).turn(p.vocab) : kTurns;
        uint32_t* const counts = sh.keys.cnt;   // [turn][warp]
        int place = 0;
#pragma unroll
        for (int q = 0; q < kTurns; ++q) {
            const uint32_t bits = __ballot_sync(0xffffffffu, turn == q);
            if (lane == 0) counts[q * kWarps + warp] = __popc(bits);
            if (turn == q) place = __popc(bits & ((1u << lane) - 1u));
        }
        __syncthreads();
        const uint32_t even = counts[2 * lane], both = even + counts[2 * lane + 1];
        const uint32_t before = warp_incl(both, lane) - both;
        const int e = turn * kWarps + warp, from = e >> 1 & 31;
        const uint32_t upto = __shfl_sync(0xffffffffu, before, from) + __shfl_sync(0xffffffffu, even, from) * (e & 1);
        if (turn < kTurns && (int)upto + place == at) sh.bin = tid;
        __syncthreads();
        return sh.bin;   // not written before the next barrier
    }
    unsigned long long counts = 0;   // of each turn, sixteen bits
    for (int i = tid; i < p.batch; i += kThreads) counts += 1ull << (16 * settings_of(p, i).turn(p.vocab));
    counts = warp_sum(counts);
    if (lane == 0) sh.best[warp] = counts;
    __syncthreads();
    counts = warp_sum(lane < kWarps ? sh.best[lane] : 0ull);
    int turn = 0;
    for (; turn < 3 && at >= (int)(counts >> (16 * turn) & 0xffffu); ++turn) at -= (int)(counts >> (16 * turn) & 0xffffu);
    for (int base = 0; base < p.batch; base += kThreads) {
        const int i = base + tid;
        const bool mine = i < p.batch && settings_of(p, i).turn(p.vocab) == turn;
        const uint32_t bits = __ballot_sync(0xffffffffu, mine);
        __syncthreads();
        if (lane == 0) sh.scan_cnt[warp] = __popc(bits);
        __syncthreads();
        const uint32_t upto = warp_incl(lane < kWarps ? sh.scan_cnt[lane] : 0u, lane);
        const int before = (int)__shfl_sync(0xffffffffu, upto, warp > 0 ? warp - 1 : 0) * (warp > 0) + __popc(bits & ((1u << lane) - 1u));
        if (mine && before == at) sh.bin = i;
        at -= (int)__shfl_sync(0xffffffffu, upto, kWarps - 1);
        if (at < 0) break;
    }
    __syncthreads();
    const int row = sh.bin;
    __syncthreads();
    return row;
}

template <int DTYPE>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const SampleParams p)
{
    using T = typename Elem<DTYPE>::T;
    constexpr int VEC = 16 / sizeof(T);
    __shared__ __align__(16) Shared sh;
    chained_kernel();
    cg::cluster_group cl = cg::this_cluster();
    const int rank = (int)cl.block_rank(), ctas = (int)cl.num_blocks();
    const int row = p.in_turn ? row_in_turn(p, sh, blockIdx.x / ctas) : blockIdx.x / ctas;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

    // ---- the slice: places are counted from the 16-byte boundary at or before the row's first logit
    const T* const src = static_cast<const T*>(p.logits) + (long long)row * p.stride;
    const int mis = (int)((reinterpret_cast<uintptr_t>(src) & 15) / sizeof(T));
    const int first = rank * p.slice - mis;           // the token at this slice's first place (may be below 0)
    const int slice = p.slice;                        // a multiple of VEC * kThreads
    auto load = [&](int v) {                          // 16 bytes from place v on; -infinity outside the row
        const int at = first + v;
        if (at >= 0 && at + VEC <= p.vocab) return __ldg(reinterpret_cast<const uint4*>(src + at));
        uint32_t b[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            const bool in = at + i >= 0 && at + i < p.vocab;
            if constexpr (sizeof(T) == 4) b[i] = in ? __float_as_uint(src[at + i]) : 0xff800000u;
            else b[i] = in ? src[at + i] : DTYPE == W4A16_FP16 ? 0xfc00u : 0xff80u;
        }
        if constexpr (sizeof(T) == 4) return make_uint4(b[0], b[1], b[2], b[3]);
        else return make_uint4(b[0] | b[1] << 16, b[2] | b[3] << 16, b[4] | b[5] << 16, b[6] | b[7] << 16);
    };
    // a NaN never compares above anything and weighs nothing
    auto expand = [](const uint4& raw, float (&x)[VEC]) {
        const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
        for (int i = 0; i < VEC; ++i)
            x[i] = Elem<DTYPE>::get(sizeof(T) == 4 ? w[i * 4 / VEC] : (w[i / 2] >> (16 * (i & 1))) & 0xffffu);
    };
    // runs f(place, x) over the vectors from place a on, `step` apart, below b, that hold an x >= low
    auto sweep = [&](int a, int b, int step, float low, auto f) {
        for (int v0 = a; v0 < b; v0 += 4 * step) {   // four loads in flight
            uint4 raw[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (v0 + i * step < b) raw[i] = load(v0 + i * step);
#pragma unroll 1
            for (int i = 0; i < 4 && v0 + i * step < b; ++i) {
                const uint4 now = raw[0];
                raw[0] = raw[1];
                raw[1] = raw[2];
                raw[2] = raw[3];
                if (!(Elem<DTYPE>::largest(now) >= low)) continue;
                float x[VEC];
                expand(now, x);
#pragma unroll
                for (int e = 0; e < VEC; ++e) f(v0 + i * step + e, x[e]);
            }
        }
    };
    auto each = [&](float low, auto f) { sweep(tid * VEC, slice, kThreads * VEC, low, f); };

    float tops[kGroups], mine = -CUDART_INF_F;        // maxima of this thread's groups of tokens, and of all
#pragma unroll
    for (int i = 0; i < kGroups; ++i) tops[i] = -CUDART_INF_F;
    for (int v0 = tid * VEC; v0 < slice; v0 += 2 * kGroups * kThreads * VEC) {   // eight loads in flight
        uint4 raw[2 * kGroups];
#pragma unroll
        for (int i = 0; i < 2 * kGroups; ++i)
            if (v0 + i * kThreads * VEC < slice) raw[i] = load(v0 + i * kThreads * VEC);
#pragma unroll
        for (int i = 0; i < 2 * kGroups; ++i)
            if (v0 + i * kThreads * VEC < slice) tops[i % kGroups] = fmaxf(tops[i % kGroups], Elem<DTYPE>::largest(raw[i]));
    }
#pragma unroll
    for (int i = 0; i < kGroups; ++i) mine = fmaxf(mine, tops[i]);
    float wtop = mine;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) wtop = fmaxf(wtop, __shfl_xor_sync(0xffffffffu, wtop, d));
    float* const wtops = reinterpret_cast<float*>(sh.best);
    if (lane == 0) wtops[warp] = wtop;
    clear(sh.bins);
    __syncthreads();
    if (warp == 0) {
        float t = lane < kWarps ? wtops[lane] : -CUDART_INF_F;
#pragma unroll
        for (int d = kWarps / 2; d > 0; d >>= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, d));
        if (lane == 0) {
            sh.top = t;
            sh.listed = 0;
        }
    }
    const Settings s = settings_of(p, row);
    const float temp = s.temp, top_p = s.top_p, u = p.u[row];
    const int k = s.k;
    Row r;
    r.min_p = s.min_p;
    r.inv = __frcp_rn(temp);
    cl.sync();
    r.top = cl.map_shared_rank(&sh, lane < ctas ? lane : 0)->top;
#pragma unroll
    for (int d = kMaxCluster / 2; d > 0; d >>= 1) r.top = fmaxf(r.top, __shfl_xor_sync(0xffffffffu, r.top, d));
    r.top = __shfl_sync(0xffffffffu, r.top, 0);

    auto result = [&](int token, double share) {
        p.token[row] = token;
        if (p.prob) p.prob[row] = (float)share;
    };
    // the place of the draw in a kept weight
    auto target_of = [&](unsigned long long total) {
        const unsigned long long t = (unsigned long long)((double)total * (double)u);
        return t < total ? t : total - 1;
    };
    const bool none = r.top == -CUDART_INF_F;
    if (none || s.greedy()) {
        // the lowest index of the maximum
        uint32_t at = 0xffffffffu;
        if (!none && mine == r.top)
            each(r.top, [&](int v, float x) {
                if (x == r.top) at = min(at, (uint32_t)(first + v));
            });
        at = __reduce_min_sync(0xffffffffu, at);
        if (lane == 0) sh.best[warp] = at;
        __syncthreads();
        if (warp == 0) {
            at = __reduce_min_sync(0xffffffffu, lane < kWarps ? (uint32_t)sh.best[lane] : 0xffffffffu);
            if (lane == 0) sh.range = at;
        }
        cl.sync();
        if (rank == 0 && warp == 0) {
            at = __reduce_min_sync(0xffffffffu, lane < ctas ? (uint32_t)cl.map_shared_rank(&sh, lane)->range : 0xffffffffu);
            if (lane == 0) result(none ? -1 : (int)at, none ? 0.0 : 1.0);
        }
        cl.sync();   // no CTA leaves while another may read its shared memory
        return;
    }

    // ---- the cut: kept are logits above cut_x, and those equal to it up to index cut_at
    float cut_x = -CUDART_INF_F;
    int cut_at = -1;
    const bool need_k = s.need_k(p.vocab), need_p = s.need_p();
    const float to_bin = kBins / kSpan;
    // a logit below every one that is at most d below the maximum, whatever the roundings of either side
    auto below = [&](float d) { return r.top <= FLT_MAX ? r.top - d * 1.00001f - 1e-6f * fabsf(r.top) : r.top; };
    // and one at or above every one that is at least d below it
    auto above = [&](float d) { return r.top <= FLT_MAX ? fminf(r.top - fminf(d, FLT_MAX) * 0.99999f + 1e-6f * fabsf(r.top), r.top) : r.top; };
    const float weightless = below(22.5f * temp);   // lower ones weigh nothing
    auto entry_of = [](float x, uint32_t low) { return (unsigned long long)key_of<DTYPE>(x) << kIndexBits | low; };
    auto list_it = [&](int v, float x) {
        const uint32_t at = atomicAdd(&sh.listed, 1u);
        if (at < kListMine)
            sh.list[at] = entry_of(x, kIndexTop - (uint32_t)(first + v));
    };
    auto logit_of = [](unsigned long long e) { return float_of<DTYPE>((uint32_t)(e >> kIndexBits)); };
    auto token_of = [](unsigned long long e) { return (int)(kIndexTop - ((uint32_t)e & kIndexTop)); };
    // The cluster's lists in the first CTA's registers, kListPer entries a thread (0: none), with their weights.
    // Returns the number of entries, or -1 (everywhere) where they do not fit.
    unsigned long long key[kListPer];
    uint32_t w[kListPer];
    auto gather = [&]() {
        cl.sync();
        const int len = lane < ctas ? (int)cl.map_shared_rank(&sh, lane)->listed : 0;
        const int upto = warp_incl(len, lane), n = __shfl_sync(0xffffffffu, upto, 31);
        if (__any_sync(0xffffffffu, len > kListMine) || n > kListMax) return -1;
        if (rank == 0) {
#pragma unroll
            for (int i = 0; i < kListPer; ++i) {
                const int at = i * kThreads + tid;
                int c = 0, from = 0;   // the CTA that holds the entry
                for (int o = 0; o < kMaxCluster; ++o) {
                    const int e = __shfl_sync(0xffffffffu, upto, o);
                    if (at >= e && o + 1 < ctas) {
                        c = o + 1;
                        from = e;
                    }
                }
                key[i] = at < n ? cl.map_shared_rank(&sh, c)->list[at - from] : 0ull;
                w[i] = at < n ? weight_of(exp_of(logit_of(key[i]), r)) : 0u;
            }
        }
        return n;
    };
    // this CTA's sum of 64-bit numbers
    auto block_sum = [&](unsigned long long v) {
        v = warp_sum(v);
        __syncthreads();
        if (lane == 0) sh.best[warp] = v;
        __syncthreads();
        v = lane < kWarps ? sh.best[lane] : 0ull;
        return warp_sum(v);
    };

    const uint32_t kk = (uint32_t)k;
    auto by_count = [kk](uint32_t c, unsigned long long, unsigned long long) { return c >= kk; };
    auto by_mass = [](uint32_t, unsigned long long m, unsigned long long limit) { return m >= limit; };
    auto no_bound = [](unsigned long long) { return 0ull; };
    if (need_k && k <= kListMax / 2) {
        // a bound below at least k tokens: the bin of the k-th largest of the groups' maxima
#pragma unroll
        for (int i = 0; i < kGroups; ++i) {
            const float b = place(tops[i], r);
            if (tops[i] > -CUDART_INF_F && b < (float)kBins) atomicAdd(&sh.bins.cnt[whole(b)], 1u);
        }
        search<false>(cl, sh, sh.bins, 0u, 0ull, by_count, no_bound);
        if (sh.bin >= 0) {
            // down to the bin's lower end, and a few tokens more
            const float low = below((float)(sh.bin + 1) / to_bin * temp);
            if (mine >= low)   // else this thread has none
                each(low, [&](int v, float x) {
                    if (x >= low && x > -CUDART_INF_F) list_it(v, x);
                });
            const int n = gather();
            if (n >= 0) {
                cl.sync();   // the first CTA has read the lists: the others leave their place to another row
                if (rank == 0 && n <= kFew) {
                    // few entries: each counts and weighs those ranked before it, then the kept ones of lower index
                    unsigned long long* const keys = sh.list;   // the lists have been gathered
                    uint32_t* const ws = sh.keys.cnt;
                    __syncthreads();
                    if (tid < n) {
                        keys[tid] = key[0];
                        ws[tid] = w[0];
                    }
                    __syncthreads();
                    const int i = tid >> 2;
                    const unsigned long long own = i < n ? keys[i] : 0ull;
                    const uint32_t own_w = i < n ? ws[i] : 0u;
                    int ahead = 0;
                    unsigned long long before = 0;
                    for (int j = tid & 3; j < n; j += 4)
                        if (keys[j] > own) {
                            ++ahead;
                            before += ws[j];
                        }
#pragma unroll
                    for (int d = 1; d < 4; d *= 2) {
                        ahead += __shfl_xor_sync(0xffffffffu, ahead, d);
                        before += __shfl_xor_sync(0xffffffffu, before, d);
                    }
                    bool keep = i < n && ahead < k;
                    unsigned long long total = block_sum(keep && (tid & 3) == 0 ? own_w : 0u);
                    if (tid == 0) sh.limit = need_p ? limit_of(total, top_p) : ~0ull;
                    __syncthreads();
                    const float x = logit_of(own);
                    keep = keep && (ahead == 0 || before < sh.limit) && (ahead == 0 || exp_of(x, r) >= r.min_p || x == r.top);
                    total = block_sum(keep && (tid & 3) == 0 ? own_w : 0u);
                    if (!keep && i < n) ws[i] = 0u;
                    if (tid == 0) sh.limit = target_of(total);
                    __syncthreads();
                    const unsigned long long target = sh.limit;
                    before = 0;
                    for (int j = tid & 3; j < n; j += 4)
                        if (((uint32_t)keys[j] & kIndexTop) > ((uint32_t)own & kIndexTop)) before += ws[j];
#pragma unroll
                    for (int d = 1; d < 4; d *= 2) before += __shfl_xor_sync(0xffffffffu, before, d);
                    if (keep && (tid & 3) == 0 && target >= before && target < before + own_w)
                        result(token_of(own), (double)own_w / (double)total);
                } else if (rank == 0) {
                    unsigned long long least = entry_of(low, 0), greatest = entry_of(r.top, kIndexTop);
                    // the k-th entry, the entry at which top-p's limit is passed, and the drawn one among the kept
                    if (n > k) {
                        pick(sh, key, w, least, greatest, 0ull, by_count, [] { return 0ull; });
                        least = sh.picked;
#pragma unroll
                        for (int i = 0; i < kListPer; ++i)
                            if (key[i] < least) key[i] = 0, w[i] = 0;
                    }
                    unsigned long long sum = 0;
#pragma unroll
                    for (int i = 0; i < kListPer; ++i) sum += w[i];
                    unsigned long long total = block_sum(sum);
                    if (need_p) {
                        pick(sh, key, w, least, greatest, 0ull, by_mass, [&] { return limit_of(total, top_p); });
                        const unsigned long long last = sh.picked;
#pragma unroll
                        for (int i = 0; i < kListPer; ++i)
                            if (key[i] < last) key[i] = 0, w[i] = 0;
                    }
                    if (r.min_p > 0.0f) {
#pragma unroll
                        for (int i = 0; i < kListPer; ++i)
                            if (key[i] && !(exp_of(logit_of(key[i]), r) >= r.min_p)) key[i] = 0, w[i] = 0;
                    }
                    if (need_p || r.min_p > 0.0f) {
                        sum = 0;
#pragma unroll
                        for (int i = 0; i < kListPer; ++i) sum += w[i];
                        total = block_sum(sum);
                    }
                    // by index now: the low bits, greatest first, are ascending indices (one bit on top, as 0 is no entry)
#pragma unroll
                    for (int i = 0; i < kListPer; ++i) key[i] = key[i] ? 1ull << kIndexBits | (key[i] & kIndexTop) : 0ull;
                    pick(sh, key, w, 1ull << kIndexBits, (2ull << kIndexBits) - 1ull, 0ull,
                         [](uint32_t, unsigned long long m, unsigned long long target) { return m > target; },
                         [&] { return target_of(total); });
                    if (tid == 0) result(token_of(sh.picked), (double)sh.picked_weight / (double)total);
                }
                return;
            }
        }
        cl.sync();
        clear(sh.bins);
        __syncthreads();
    }

    const int seg_len = slice / kWarps;               // a warp's segment: a multiple of 32 VEC
    const int s0 = warp * seg_len;
    auto kept = [&](float x, int v) -> uint32_t {
        // evaluated for every token of a vector: cheaper than a branch around it
        const float e = exp_of(x, r);
        const bool in = (x > cut_x || (x == cut_x && first + v <= cut_at)) && (e >= r.min_p || x == r.top);
        return in ? weight_of(e) : 0u;
    };
    // the segment that holds the draw, from sh.all_mass
    auto choose = [&](int segs) {
        if (warp != 0) return;
        constexpr int PER = kMaxCluster * kWarps / 32;
        unsigned long long ms[PER], msum = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int s = lane * PER + i;
            ms[i] = s < segs ? sh.all_mass[s] : 0ull;
            msum += ms[i];
        }
        const unsigned long long mi = warp_incl(msum, lane);
        const unsigned long long total = __shfl_sync(0xffffffffu, mi, 31);
        const unsigned long long target = target_of(total);
        unsigned long long b = mi - msum;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            if (target >= b && target < b + ms[i]) {
                sh.seg = lane * PER + i;
                sh.seg_target = target - b;
            }
            b += ms[i];
        }
        if (lane == 0) sh.total = total;
    };
    // the drawn token, by all threads of a CTA
    auto locate = [&](int seg, unsigned long long target, unsigned long long total) {
        const int from = seg % kWarps * seg_len + (seg / kWarps - rank) * slice;   // counted in this CTA's places
        unsigned long long before = 0;
        for (int v0 = from; v0 < from + seg_len; v0 += kThreads * VEC) {
            const int v = v0 + tid * VEC;
            uint32_t weight[VEC];
            unsigned long long sum = 0;
            float x[VEC];
            if (v < from + seg_len) expand(load(v), x);
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                weight[i] = v < from + seg_len ? kept(x[i], v + i) : 0u;
                sum += weight[i];
            }
            const unsigned long long incl = warp_incl(sum, lane);
            __syncthreads();
            if (lane == 31) sh.best[warp] = incl;
            __syncthreads();
            const unsigned long long wm = warp_incl(lane < kWarps ? sh.best[lane] : 0ull, lane);
            const unsigned long long upto = __shfl_sync(0xffffffffu, wm, warp > 0 ? warp - 1 : 0);
            unsigned long long b = before + (warp > 0 ? upto : 0ull) + incl - sum;
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                if (target >= b && target < b + weight[i]) result(first + v + i, (double)weight[i] / (double)total);
                b += weight[i];
            }
            before += __shfl_sync(0xffffffffu, wm, 31);
        }
    };

    // The cut inside a bin found by search(), where a list would not hold it: the bin's range of keys, then
    // histograms over the keys until one is left; n(count before, weight before, ties, a tie's weight) of that
    // key's tokens are kept, the first by index.
    auto refine = [&](auto done, unsigned long long limit, auto n) {
        const int bin = sh.bin;
        uint32_t cnt0 = sh.base_cnt;
        unsigned long long mass0 = sh.base_mass;
        uint32_t kmin = 0xffffffffu, kmax = 0u;
        each(weightless, [&](int, float x) {
            if (!(x > -CUDART_INF_F) || bin_of(x, r) != bin || weight_of(exp_of(x, r)) == 0) return;
            const uint32_t key = key_of<DTYPE>(x);
            kmin = key < kmin ? key : kmin;
            kmax = key > kmax ? key : kmax;
        });
        kmin = __reduce_min_sync(0xffffffffu, kmin);
        kmax = __reduce_max_sync(0xffffffffu, kmax);
        if (lane == 0) sh.best[warp] = (unsigned long long)kmax << 32 | kmin;
        __syncthreads();
        if (tid == 0) {
            for (int i = 0; i < kWarps; ++i) {
                const uint32_t a = (uint32_t)sh.best[i], b = (uint32_t)(sh.best[i] >> 32);
                kmin = a < kmin ? a : kmin;
                kmax = b > kmax ? b : kmax;
            }
            sh.range = (unsigned long long)kmax << 32 | kmin;
        }
        cl.sync();
        for (int c = 0; c < ctas; ++c) {
            const unsigned long long o = cl.map_shared_rank(&sh, c)->range;
            kmin = (uint32_t)o < kmin ? (uint32_t)o : kmin;
            kmax = (uint32_t)(o >> 32) > kmax ? (uint32_t)(o >> 32) : kmax;
        }
        for (int level = 0; level < 4; ++level) {   // ten bits of the range a level
            cl.sync();                              // the last level's counts are read
            clear(sh.keys);
            __syncthreads();
            const uint32_t range = kmax - kmin;
            const int bits = range ? 32 - __clz(range) : 0;
            const int shift = bits > 10 ? bits - 10 : 0;
            each(float_of<DTYPE>(kmin), [&](int, float x) {
                const uint32_t key = key_of<DTYPE>(x);
                if (x > -CUDART_INF_F && key >= kmin && key <= kmax) {
                    const int at = (int)((kmax - key) >> shift);
                    atomicAdd(&sh.keys.cnt[at], 1u);
                    add_mass(sh.keys, at, weight_of(exp_of(x, r)));
                }
            });
            search<true>(cl, sh, sh.keys, cnt0, mass0, done, [limit](unsigned long long) { return limit; });
            cnt0 = sh.base_cnt;
            mass0 = sh.base_mass;
            if (shift == 0) break;
            kmax -= (uint32_t)sh.bin << shift;
            const uint32_t low = kmax - ((1u << shift) - 1u);
            kmin = low > kmin && low <= kmax ? low : kmin;
        }
        // the key's kept tokens end at an index: that of the last, by counts of the warps' segments
        const uint32_t ties = sh.bin_cnt;
        const uint32_t keep = n(cnt0, mass0, ties, (uint32_t)(sh.bin_mass / ties));
        cut_x = float_of<DTYPE>(kmax - (uint32_t)sh.bin);
        cut_at = 0x7fffffff;
        if (keep < ties) {
            auto tie_at = [&](int v) {
                const int at = first + v;
                if (at < 0 || at >= p.vocab) return false;
                if constexpr (sizeof(T) == 4) return src[at] == cut_x;
                else return Elem<DTYPE>::get(src[at]) == cut_x;
            };
            uint32_t here = 0;
            for (int v = warp * seg_len + lane; v < (warp + 1) * seg_len; v += 32) here += tie_at(v);
            here = __reduce_add_sync(0xffffffffu, here);
            if (lane == 0) sh.scan_cnt[warp] = here;
            __syncthreads();
            if (tid == 0) {
                uint32_t sum = 0;
                for (int i = 0; i < kWarps; ++i) sum += sh.scan_cnt[i];
                sh.listed = sum;
            }
            cl.sync();
            uint32_t before = 0;
            for (int c = 0; c < rank; ++c) before += cl.map_shared_rank(&sh, c)->listed;
            for (int i = 0; i < warp; ++i) before += sh.scan_cnt[i];
            if (before < keep && keep <= before + here) {   // one warp of the cluster
                for (int v = warp * seg_len + lane; v < (warp + 1) * seg_len; v += 32) {
                    const bool tie = tie_at(v);
                    const uint32_t bits = __ballot_sync(0xffffffffu, tie);
                    const uint32_t at = before + __popc(bits & ((2u << lane) - 1u));
                    if (tie && at == keep) cl.map_shared_rank(&sh, 0)->cut = 0xffffffffu - (uint32_t)(first + v);
                    before += __popc(bits);
                }
            }
            cl.sync();
            cut_at = (int)(0xffffffffu - (uint32_t)cl.map_shared_rank(&sh, 0)->cut);
        }
        __syncthreads();
    };
    // how many of a key's tokens top-p keeps
    auto kept_ties = [](double limit, unsigned long long m, uint32_t ties, uint32_t weight) {
        uint32_t n = (uint32_t)fmin((limit - (double)m) / (double)weight, 4294967040.0);
        n = n > ties ? ties : n;
        while (n > 0 && !((double)(m + (unsigned long long)(n - 1) * weight) < limit)) --n;
        while (n < ties && (double)(m + (unsigned long long)n * weight) < limit) ++n;
        return n > 0u ? n : 1u;
    };

    if (need_k) {
        each(weightless, [&](int, float x) {
            const uint32_t weight = weight_of(exp_of(x, r));
            if (weight) {
                const int b = bin_of(x, r);
                atomicAdd(&sh.bins.cnt[b], 1u);
                add_mass(sh.bins, b, weight);
            }
        });
        search<true>(cl, sh, sh.bins, 0u, 0ull, by_count, no_bound);
        unsigned long long total = sh.total;
        if (sh.bin >= 0)
            refine(by_count, 0ull, [&](uint32_t c, unsigned long long m, uint32_t, uint32_t weight) {
                total = m + (unsigned long long)(kk - c) * weight;
                return kk - c;
            });
        __syncthreads();
        if (need_p) {
            // both cuts are prefixes of one ranking: the shorter one holds
            const float k_x = cut_x;
            const int k_at = cut_at;
            const double limit = (double)total * (double)top_p;
            const unsigned long long least = limit_of(total, top_p);
            search<true>(cl, sh, sh.bins, 0u, 0ull, by_mass, [least](unsigned long long) { return least; });
            if (sh.bin >= 0) {
                refine(by_mass, least, [&](uint32_t, unsigned long long m, uint32_t ties, uint32_t weight) {
                    return kept_ties(limit, m, ties, weight);
                });
                if (k_x > cut_x || (k_x == cut_x && k_at < cut_at)) {
                    cut_x = k_x;
                    cut_at = k_at;
                }
            }
            __syncthreads();
        }
    } else if (need_p) {
        each(weightless, [&](int, float x) {
            const uint32_t weight = weight_of(exp_of(x, r));
            if (weight) add_mass(sh.bins, whole(place(x, r)), weight);   // a token that weighs lies inside the bins
        });
        // the bin past which the weight before a token is no longer below top_p times the whole
        search<true>(cl, sh, sh.bins, 0u, 0ull, by_mass, [&](unsigned long long all) {
            if (tid == 0) sh.limit = limit_of(all, top_p);
            __syncthreads();
            return sh.limit;
        });
        if (sh.bin >= 0) {
            const unsigned long long limit = sh.limit, total = sh.total, base = sh.base_mass;
            const int bin = sh.bin;
            // one pass sums what lies above the bin, by segments, and lists the bin's tokens
            unsigned long long mass = 0;
            const float low = below((float)(bin + 1) / to_bin * temp);
            sweep(s0 + lane * VEC, s0 + seg_len, 32 * VEC, low, [&](int v, float x) {
                const float e = exp_of(x, r), at = place(x, r);   // NaN: no bin
                mass += at < (float)bin && (e >= r.min_p || x == r.top) ? weight_of(e) : 0u;
                if (at >= (float)bin && at < (float)(bin + 1) && x > -CUDART_INF_F) list_it(v, x);
            });
            mass = warp_sum(mass);
            if (lane == 0) sh.warp_mass[warp] = mass;
            const int n = gather();
            if (n >= 0) {
                const int segs = ctas * kWarps;
                if (rank == 0 && tid < segs) sh.all_mass[tid] = cl.map_shared_rank(&sh, tid / kWarps)->warp_mass[tid % kWarps];
                cl.sync();   // the others leave, as above
                if (rank == 0) {
                    // the first bin begins at the maximum, whatever the temperature (0 times an infinite one is no distance)
                    const float high = bin == 0 ? r.top : above((float)bin / to_bin * temp);
                    pick(sh, key, w, entry_of(low, 0), entry_of(high, kIndexTop), base, by_mass, [limit] { return limit; });
#pragma unroll
                    for (int i = 0; i < kListPer; ++i)
                        if (key[i] != 0 && key[i] >= sh.picked && (exp_of(logit_of(key[i]), r) >= r.min_p || logit_of(key[i]) == r.top)) {
                            const int at = token_of(key[i]) + mis;   // place in the row
                            atomicAdd(&sh.all_mass[at / p.slice * kWarps + at % p.slice / seg_len], (unsigned long long)w[i]);
                        }
                    cut_x = logit_of(sh.picked);
                    cut_at = token_of(sh.picked);
                    __syncthreads();
                    choose(segs);
                    __syncthreads();
                    locate(sh.seg, sh.seg_target, sh.total);
                }
                return;
            }
            const double share = (double)total * (double)top_p;
            refine(by_mass, limit, [&](uint32_t, unsigned long long m, uint32_t ties, uint32_t weight) {
                return kept_ties(share, m, ties, weight);
            });
        }
    }

    // ---- the kept weight of each warp's segment, in index order
    unsigned long long mass = 0;
    if (cut_x == -CUDART_INF_F && !(r.min_p > 0.0f))   // nothing is cut
        sweep(s0 + lane * VEC, s0 + seg_len, 32 * VEC, weightless, [&](int, float x) { mass += weight_of(exp_of(x, r)); });
    else
        sweep(s0 + lane * VEC, s0 + seg_len, 32 * VEC, fmaxf(cut_x, weightless), [&](int v, float x) { mass += kept(x, v); });
    mass = warp_sum(mass);
    if (lane == 0) sh.warp_mass[warp] = mass;
    cl.sync();
    const int segs = ctas * kWarps;
    if (tid < segs) sh.all_mass[tid] = cl.map_shared_rank(&sh, tid / kWarps)->warp_mass[tid % kWarps];
    cl.sync();   // no CTA leaves while another may read its shared memory
    choose(segs);
    __syncthreads();
    if (sh.seg / kWarps == rank) locate(sh.seg, sh.seg_target, sh.total);
}

}  // namespace

cudaError_t launch_sample(const SampleParams& in, int sms, cudaStream_t stream)
{
    SampleParams p = in;
    const int size = p.dtype == W4A16_FP32 ? 4 : 2;
    const int step = 16 / size * kThreads;   // a slice is whole rounds of 16-byte loads
    // As many CTAs a row as give every SM the two it holds, while a slice is more than a round of loads; up
    // to the portable cluster of eight. A row's steps are a chain, so that fewer, longer slices leave it waiting
    // (256 x 100003 FP32: 243 us with one CTA a row, 77 with two, 96 with four; 128 x 131072 bfloat16: 65 with
    // two, 55 with four, 84 with eight; now 69 and 45). More where a slice would pass kMaxSlice.
    auto slice_of = [&](int n) { return ((p.vocab + 16 / size + n - 1) / n + step - 1) / step * step; };
    int ctas = 1;
    while (ctas < kMaxCluster && (((long long)p.batch * ctas < 2 * sms && p.vocab / ctas > step) || slice_of(ctas) > kMaxSlice)) ctas *= 2;
    p.in_turn = (long long)p.batch * ctas > 2 * sms && p.batch <= 16384;
    p.slice = slice_of(ctas);
    const unsigned grid = (unsigned)(p.batch * ctas);
    switch (p.dtype) {
        case W4A16_FP32: return launch_chained(sample_kernel<W4A16_FP32>, grid, kThreads, 0, (unsigned)ctas, stream, p);
        case W4A16_FP16: return launch_chained(sample_kernel<W4A16_FP16>, grid, kThreads, 0, (unsigned)ctas, stream, p);
        default: return launch_chained(sample_kernel<W4A16_BF16>, grid, kThreads, 0, (unsigned)ctas, stream, p);
    }
}

}  // namespace w4a16
