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
// A cluster of CTAs holds one row, each CTA a slice of it in shared memory (read from HBM
// once). The kept set is a prefix of the ranking, so it is one cut: a key, and how many of
// the tokens that tie with it (by index). The cut is found by histograms of counts and
// weights: first over 1024 bins of (m - x) r, which spreads logits evenly where their bits
// would not (fewer conflicts of shared atomics), then, inside the bin that holds the cut,
// over the keys. Every CTA adds up the cluster's histograms for itself.
#include "ptx.cuh"
#include "sample.cuh"
#include "w4a16.h"

#include <cooperative_groups.h>
#include <math_constants.h>

namespace w4a16 {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 1024;
constexpr int kPer = kBins / kThreads;   // bins a thread adds up
constexpr int kMaxCluster = 8;
constexpr float kSpan = 22.2f;           // exp(-22.2) * 2^31 rounds to 0

struct Shared {
    uint32_t cnt[3][kBins], lo[3][kBins], hi[3][kBins];   // a bin's count, and its weight's low and high 16 bits summed
    unsigned long long best[kWarps];
    unsigned long long mine[4];          // what this CTA shows to the cluster: maximum; least and greatest key
    unsigned long long scan_mass[kWarps];
    uint32_t scan_cnt[kWarps];
    unsigned long long warp_mass[kWarps];   // kept weight above the cut's key, of each warp's segment
    uint32_t warp_ties[kWarps];
    unsigned long long all_mass[kMaxCluster * kWarps];
    uint32_t all_ties[kMaxCluster * kWarps];
    // results of a search
    int bin;
    uint32_t base_cnt, bin_cnt;
    unsigned long long base_mass, bin_mass;
    // the chosen segment
    int seg;
    uint32_t seg_ties;
    unsigned long long seg_target, total;
};

template <int DTYPE>
struct Elem;
template <>
struct Elem<W4A16_FP32> {
    using T = float;
    static constexpr int kShift = 0;
    static __device__ __forceinline__ float get(uint32_t bits) { return __uint_as_float(bits); }
};
template <>
struct Elem<W4A16_FP16> {
    using T = uint16_t;
    static constexpr int kShift = 13;
    static __device__ __forceinline__ float get(uint32_t bits) { return __half2float(__ushort_as_half((uint16_t)bits)); }
};
template <>
struct Elem<W4A16_BF16> {
    using T = uint16_t;
    static constexpr int kShift = 16;
    static __device__ __forceinline__ float get(uint32_t bits) { return __uint_as_float(bits << 16); }
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

__device__ __forceinline__ float exp_of(float x, const Row& r)
{
    return x == r.top ? 1.0f : expf(__fmul_rn(__fsub_rn(x, r.top), r.inv));
}

__device__ __forceinline__ uint32_t weight_of(float e) { return __float2uint_rn(e * 2147483648.0f); }

__device__ __forceinline__ int bin_of(float x, const Row& r)
{
    const int b = (int)(__fmul_rn(__fsub_rn(r.top, x), r.inv) * (kBins / kSpan));
    return b < kBins - 1 ? b : kBins - 1;
}

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

__device__ __forceinline__ void clear_bins(Shared& sh, int h)
{
    for (int i = threadIdx.x; i < kBins; i += kThreads) sh.cnt[h][i] = sh.lo[h][i] = sh.hi[h][i] = 0;
}

__device__ __forceinline__ void count_in(Shared& sh, int h, int bin, uint32_t w)
{
    atomicAdd(&sh.cnt[h][bin], 1u);
    atomicAdd(&sh.lo[h][bin], w & 0xffffu);
    if (w >> 16) atomicAdd(&sh.hi[h][bin], w >> 16);
}

// Adds up the cluster's histograms h and finds the first bin with done(count, mass of every bin up to
// and with it); base counts come on top. Leaves bin = -1 if there is none. Every CTA finds the same.
// A cluster barrier before (the histograms are complete) is in here; the caller keeps one between this
// and the next use of the same histogram.
template <typename F>
__device__ __forceinline__ void search(cg::cluster_group& cl, Shared& sh, int h, uint32_t base_cnt,
                                       unsigned long long base_mass, F done)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) sh.bin = -1;
    cl.sync();
    uint32_t cnt[kPer];
    unsigned long long mass[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        cnt[i] = 0;
        mass[i] = 0;
    }
    const int ctas = (int)cl.num_blocks();
    for (int k = 0; k < ctas; ++k) {
        const Shared* o = cl.map_shared_rank(&sh, k);
        const int at = threadIdx.x * kPer;
        const uint2 a = *reinterpret_cast<const uint2*>(&o->cnt[h][at]);
        const uint2 b = *reinterpret_cast<const uint2*>(&o->lo[h][at]);
        const uint2 c = *reinterpret_cast<const uint2*>(&o->hi[h][at]);
        cnt[0] += a.x;
        cnt[1] += a.y;
        mass[0] += b.x + ((unsigned long long)c.x << 16);
        mass[1] += b.y + ((unsigned long long)c.y << 16);
    }
    static_assert(kPer == 2, "two bins a thread");
    const uint32_t my_cnt = cnt[0] + cnt[1];
    const unsigned long long my_mass = mass[0] + mass[1];
    const uint32_t ic = warp_incl(my_cnt, lane);
    const unsigned long long im = warp_incl(my_mass, lane);
    if (lane == 31) {
        sh.scan_cnt[warp] = ic;
        sh.scan_mass[warp] = im;
    }
    __syncthreads();
    uint32_t c = base_cnt + ic - my_cnt;
    unsigned long long m = base_mass + im - my_mass;
    unsigned long long all = base_mass;
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) {
            c += sh.scan_cnt[w];
            m += sh.scan_mass[w];
        }
        all += sh.scan_mass[w];
    }
    if (threadIdx.x == 0) sh.total = all;
    bool before = done(c, m);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const bool now = done(c + cnt[i], m + mass[i]);
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

struct Cut {
    uint32_t key, ties;           // kept: greater keys, and the first `ties` tokens with this key
    unsigned long long mass;      // weight of what is greater
    uint32_t weight;              // weight of a token with this key
    uint32_t cnt;                 // tokens with greater keys
};

template <int DTYPE>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const SampleParams p)
{
    using T = typename Elem<DTYPE>::T;
    constexpr int VEC = 16 / sizeof(T);
    extern __shared__ __align__(16) uint8_t dyn[];
    Shared& sh = *reinterpret_cast<Shared*>(dyn);
    T* const xs = reinterpret_cast<T*>(dyn + (sizeof(Shared) + 15) / 16 * 16);
    cg::cluster_group cl = cg::this_cluster();
    const int rank = (int)cl.block_rank(), ctas = (int)cl.num_blocks();
    const int row = blockIdx.x / ctas;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

    // ---- the slice: positions are counted from the 16-byte boundary at or before the row's first logit
    const T* const src = static_cast<const T*>(p.logits) + (long long)row * p.stride;
    const int mis = (int)((reinterpret_cast<uintptr_t>(src) & 15) / sizeof(T));
    const int first = rank * p.slice;                 // this slice's first position; token = position - mis
    const int slice = p.slice;                        // a multiple of VEC * kThreads
    unsigned long long best = 0;
    for (int v = tid * VEC; v < slice; v += kThreads * VEC) {
        uint4 raw;
        const int at = first + v - mis;               // token of the first element
        if (at >= 0 && at + VEC <= p.vocab) {
            raw = __ldg(reinterpret_cast<const uint4*>(src + at));
        } else {
            uint32_t b[VEC];
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const bool in = at + i >= 0 && at + i < p.vocab;
                if constexpr (sizeof(T) == 4) b[i] = in ? __float_as_uint(src[at + i]) : 0xff800000u;
                else b[i] = in ? src[at + i] : DTYPE == W4A16_FP16 ? 0xfc00u : 0xff80u;
            }
            if constexpr (sizeof(T) == 4) raw = make_uint4(b[0], b[1], b[2], b[3]);
            else raw = make_uint4(b[0] | b[1] << 16, b[2] | b[3] << 16, b[4] | b[5] << 16, b[6] | b[7] << 16);
        }
        uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            uint32_t bits = sizeof(T) == 4 ? w[i] : (w[i / 2] >> (16 * (i & 1))) & 0xffffu;
            float x = Elem<DTYPE>::get(bits);
            if (x != x) {                              // NaN: never sampled
                x = -CUDART_INF_F;
                if constexpr (sizeof(T) == 4) w[i] = 0xff800000u;
                else {
                    const uint32_t inf = DTYPE == W4A16_FP16 ? 0xfc00u : 0xff80u;
                    w[i / 2] = (w[i / 2] & (0xffff0000u >> (16 * (i & 1)))) | inf << (16 * (i & 1));
                }
            }
            const unsigned long long k = (unsigned long long)key_of<DTYPE>(x) << 32 | (0xffffffffu - (uint32_t)(at + i));
            if (at + i >= 0 && at + i < p.vocab) best = k > best ? k : best;
        }
        *reinterpret_cast<uint4*>(xs + v) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    auto at = [&](int v) {
        if constexpr (sizeof(T) == 4) return xs[v];
        else return Elem<DTYPE>::get(xs[v]);
    };
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        const unsigned long long o = __shfl_xor_sync(0xffffffffu, best, d);
        best = o > best ? o : best;
    }
    if (lane == 0) sh.best[warp] = best;
    clear_bins(sh, 0);
    __syncthreads();
    if (tid == 0) {
        for (int w = 1; w < kWarps; ++w) best = sh.best[w] > best ? sh.best[w] : best;
        sh.mine[0] = best;
    }
    cl.sync();
    best = 0;
    for (int k = 0; k < ctas; ++k) {
        const unsigned long long o = cl.map_shared_rank(&sh, k)->mine[0];
        best = o > best ? o : best;
    }
    const int top_token = (int)(0xffffffffu - (uint32_t)best);

    Row r;
    {
        const uint32_t k = (uint32_t)(best >> 32) << Elem<DTYPE>::kShift;
        // back from the key: positive numbers had their top bit set, negative ones were complemented
        r.top = (k & 0x80000000u) ? __uint_as_float(k & 0x7fffffffu)
                                  : __uint_as_float(~(k | ((1u << Elem<DTYPE>::kShift) - 1u)));
    }
    const float temp = p.temperature ? p.temperature[row] : 1.0f;
    const float top_p = p.top_p ? p.top_p[row] : 1.0f;
    const int k = p.top_k ? p.top_k[row] : 0;
    r.min_p = p.min_p ? p.min_p[row] : 0.0f;
    const bool none = r.top == -CUDART_INF_F;
    if (none || !(temp > 0.0f) || k == 1 || !(top_p > 0.0f) || !(r.min_p <= 1.0f)) {
        if (rank == 0 && tid == 0) {
            p.token[row] = none ? -1 : top_token;
            if (p.prob) p.prob[row] = none ? 0.0f : 1.0f;
        }
        cl.sync();   // no CTA leaves while another may read its shared memory
        return;
    }
    r.inv = __frcp_rn(temp);

    // ---- the cut
    const bool need_k = k > 0 && k < p.vocab, need_p = top_p < 1.0f;
    Cut cut = {0u, 0xffffffffu, 0ull, 0u, 0u};
    int h = 1;   // histogram in turn: 1 and 2; 0 keeps the bins of (m - x) r
    if (need_k || need_p) {
        for (int v = tid; v < slice; v += kThreads) {
            const float x = at(v);
            const uint32_t w = weight_of(exp_of(x, r));
            if (w) count_in(sh, 0, bin_of(x, r), w);
        }
        // the cut's key inside a bin: its range of keys, then histograms over the keys until one is left
        auto refine = [&](auto done) {
            const int bin = sh.bin;
            uint32_t cnt0 = sh.base_cnt;
            unsigned long long mass0 = sh.base_mass;
            uint32_t kmin = 0xffffffffu, kmax = 0u;
            for (int v = tid; v < slice; v += kThreads) {
                const float x = at(v);
                if (x == -CUDART_INF_F || bin_of(x, r) != bin || weight_of(exp_of(x, r)) == 0) continue;
                const uint32_t key = key_of<DTYPE>(x);
                kmin = key < kmin ? key : kmin;
                kmax = key > kmax ? key : kmax;
            }
            kmin = __reduce_min_sync(0xffffffffu, kmin);
            kmax = __reduce_max_sync(0xffffffffu, kmax);
            if (lane == 0) sh.best[warp] = (unsigned long long)kmax << 32 | kmin;
            __syncthreads();
            if (tid == 0) {
                for (int w = 0; w < kWarps; ++w) {
                    const uint32_t a = (uint32_t)sh.best[w], b = (uint32_t)(sh.best[w] >> 32);
                    kmin = a < kmin ? a : kmin;
                    kmax = b > kmax ? b : kmax;
                }
                sh.mine[1] = (unsigned long long)kmax << 32 | kmin;
            }
            cl.sync();
            for (int c = 0; c < ctas; ++c) {
                const unsigned long long o = cl.map_shared_rank(&sh, c)->mine[1];
                kmin = (uint32_t)o < kmin ? (uint32_t)o : kmin;
                kmax = (uint32_t)(o >> 32) > kmax ? (uint32_t)(o >> 32) : kmax;
            }
            Cut res = {};
            for (int level = 0; level < 4; ++level) {   // ten bits of the range a level
                h ^= 3;
                clear_bins(sh, h);
                __syncthreads();
                const uint32_t range = kmax - kmin;
                const int bits = range ? 32 - __clz(range) : 0;
                const int shift = bits > 10 ? bits - 10 : 0;
                for (int v = tid; v < slice; v += kThreads) {
                    const float x = at(v);
                    const uint32_t key = key_of<DTYPE>(x);
                    if (x != -CUDART_INF_F && key >= kmin && key <= kmax)
                        count_in(sh, h, (int)((kmax - key) >> shift), weight_of(exp_of(x, r)));
                }
                search(cl, sh, h, cnt0, mass0, done);
                cnt0 = sh.base_cnt;
                mass0 = sh.base_mass;
                if (shift == 0) {
                    res.key = kmax - (uint32_t)sh.bin;
                    res.cnt = cnt0;
                    res.mass = mass0;
                    res.ties = sh.bin_cnt;
                    res.weight = (uint32_t)(sh.bin_mass / sh.bin_cnt);
                    break;
                }
                kmax -= (uint32_t)sh.bin << shift;
                const uint32_t low = kmax - ((1u << shift) - 1u);
                kmin = low > kmin && low <= kmax ? low : kmin;
                __syncthreads();   // sh.bin is read before the next search writes it
            }
            __syncthreads();
            return res;
        };
        unsigned long long total = 0;
        if (need_k) {
            const uint32_t kk = (uint32_t)k;
            auto done = [kk](uint32_t c, unsigned long long) { return c >= kk; };
            search(cl, sh, 0, 0u, 0ull, done);
            total = sh.total;
            if (sh.bin >= 0) {
                __syncthreads();
                cut = refine(done);
                cut.ties = kk - cut.cnt;
                total = cut.mass + (unsigned long long)cut.ties * cut.weight;
            }
            __syncthreads();
        }
        if (need_p) {
            if (!need_k) {   // the whole weight
                auto never = [](uint32_t, unsigned long long) { return false; };
                search(cl, sh, 0, 0u, 0ull, never);
                total = sh.total;
                __syncthreads();
            }
            const double limit = (double)total * (double)top_p;
            // the bin past which the weight before a token is no longer below the limit
            auto done = [limit](uint32_t, unsigned long long m) { return !((double)m < limit); };
            search(cl, sh, 0, 0u, 0ull, done);
            if (sh.bin >= 0) {
                __syncthreads();
                Cut c = refine(done);
                // ties kept: those with mass + j * weight below the limit
                uint32_t n = (uint32_t)fmin((limit - (double)c.mass) / (double)c.weight, 4294967040.0);
                n = n > c.ties ? c.ties : n;
                while (n > 0 && !((double)(c.mass + (unsigned long long)(n - 1) * c.weight) < limit)) --n;
                while (n < c.ties && (double)(c.mass + (unsigned long long)n * c.weight) < limit) ++n;
                if (c.cnt == 0 && n == 0) n = 1;   // rank 0
                c.ties = n;
                if (c.key > cut.key || (c.key == cut.key && c.ties < cut.ties)) cut = c;
            }
            __syncthreads();
        }
    }

    // ---- the kept weight of each warp's segment (in index order), ties counted apart
    const int seg_len = slice / kWarps;
    const int s0 = warp * seg_len;
    auto kept = [&](float x, uint32_t key) -> uint32_t {   // weight of a token at or above the cut's key
        if (key < cut.key || x == -CUDART_INF_F) return 0u;
        const float e = exp_of(x, r);
        return e >= r.min_p || x == r.top ? weight_of(e) : 0u;
    };
    unsigned long long mass = 0;
    uint32_t ties = 0;
    for (int v = s0 + lane; v < s0 + seg_len; v += 32) {
        const float x = at(v);
        const uint32_t key = key_of<DTYPE>(x);
        if (key > cut.key) mass += kept(x, key);
        else if (key == cut.key && x != -CUDART_INF_F) ++ties;
    }
    mass = warp_sum(mass);
    ties = __reduce_add_sync(0xffffffffu, ties);
    if (lane == 0) {
        sh.warp_mass[warp] = mass;
        sh.warp_ties[warp] = ties;
    }
    cl.sync();
    const int segs = ctas * kWarps;
    if (tid < segs) {
        const Shared* o = cl.map_shared_rank(&sh, tid / kWarps);
        sh.all_mass[tid] = o->warp_mass[tid % kWarps];
        sh.all_ties[tid] = o->warp_ties[tid % kWarps];
    }
    __syncthreads();
    if (warp == 0) {
        // weight of a tie: that of the cut's key, if min-p lets it
        uint32_t tw = 0;
        if (cut.weight) {
            const uint32_t kb = cut.key << Elem<DTYPE>::kShift;
            const float x = (kb & 0x80000000u) ? __uint_as_float(kb & 0x7fffffffu)
                                               : __uint_as_float(~(kb | ((1u << Elem<DTYPE>::kShift) - 1u)));
            tw = kept(x, cut.key);
        }
        constexpr int PER = kMaxCluster * kWarps / 32;
        uint32_t t[PER], tsum = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int s = lane * PER + i;
            t[i] = s < segs ? sh.all_ties[s] : 0u;
            tsum += t[i];
        }
        uint32_t tb = warp_incl(tsum, lane) - tsum;
        unsigned long long ms[PER], msum = 0;
        uint32_t left[PER];
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int s = lane * PER + i;
            left[i] = tb < cut.ties ? cut.ties - tb : 0u;   // ties that may be kept from this segment on
            const uint32_t n = t[i] < left[i] ? t[i] : left[i];
            ms[i] = (s < segs ? sh.all_mass[s] : 0ull) + (unsigned long long)n * tw;
            msum += ms[i];
            tb += t[i];
        }
        const unsigned long long mi = warp_incl(msum, lane);
        const unsigned long long total = __shfl_sync(0xffffffffu, mi, 31);
        const double want = (double)total * (double)p.u[row];
        unsigned long long target = (unsigned long long)want;
        target = target < total ? target : total - 1;
        unsigned long long b = mi - msum;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            if (target >= b && target < b + ms[i]) {
                sh.seg = lane * PER + i;
                sh.seg_target = target - b;
                sh.seg_ties = left[i];
            }
            b += ms[i];
        }
        if (lane == 0) sh.total = total;
    }
    __syncthreads();
    if (sh.seg == rank * kWarps + warp) {
        unsigned long long run = 0;
        uint32_t seen = 0;
        for (int v = s0 + lane; v < s0 + seg_len; v += 32) {   // seg_len is a multiple of 32
            const float x = at(v);
            const uint32_t key = key_of<DTYPE>(x);
            const bool tie = key == cut.key && x != -CUDART_INF_F && cut.weight != 0;
            const uint32_t ties_here = __ballot_sync(0xffffffffu, tie);
            const uint32_t before = seen + __popc(ties_here & ((1u << lane) - 1u));
            const uint32_t w = key > cut.key || (tie && before < sh.seg_ties) ? kept(x, key) : 0u;
            const unsigned long long incl = run + warp_incl((unsigned long long)w, lane);
            const uint32_t hit = __ballot_sync(0xffffffffu, incl > sh.seg_target);
            if (hit) {
                if (lane == __ffs(hit) - 1) {
                    p.token[row] = first + v - mis;
                    if (p.prob) p.prob[row] = (float)((double)w / (double)sh.total);
                }
                break;
            }
            run = __shfl_sync(0xffffffffu, incl, 31);
            seen += __popc(ties_here);
        }
    }
    cl.sync();   // no CTA leaves while another may read its shared memory
}

constexpr int kSharedBytes = (sizeof(Shared) + 15) / 16 * 16;
constexpr int kMaxSmem = 227 * 1024;

template <int DTYPE>
cudaError_t launch_one(const SampleParams& p, int ctas, cudaStream_t stream)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.batch * ctas));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = (size_t)kSharedBytes + (size_t)p.slice * sizeof(typename Elem<DTYPE>::T);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)ctas;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, sample_kernel<DTYPE>, p);
}

}  // namespace

cudaError_t setup_sample()
{
    cudaError_t e;
    if ((e = cudaFuncSetAttribute(sample_kernel<W4A16_FP32>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem)) !=
            cudaSuccess ||
        (e = cudaFuncSetAttribute(sample_kernel<W4A16_FP16>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem)) !=
            cudaSuccess ||
        (e = cudaFuncSetAttribute(sample_kernel<W4A16_BF16>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem)) !=
            cudaSuccess)
        return e;
    return cudaSuccess;
}

cudaError_t launch_sample(const SampleParams& in, int sms, cudaStream_t stream)
{
    SampleParams p = in;
    const int size = p.dtype == W4A16_FP32 ? 4 : 2;
    const int step = 16 / size * kThreads;   // a slice is whole rounds of 16-byte loads
    // As many CTAs a row as give every SM one, and at least as many as hold the row
    // with two CTAs on an SM; up to the portable cluster of eight.
    int ctas = 1;
    const long long bytes = (long long)p.vocab * size;
    while (ctas < kMaxCluster && ((long long)p.batch * ctas < sms || bytes / ctas > 80 * 1024) &&
           p.vocab / ctas > step)
        ctas *= 2;
    p.slice = ((p.vocab + 16 / size + ctas - 1) / ctas + step - 1) / step * step;
    switch (p.dtype) {
        case W4A16_FP32: return launch_one<W4A16_FP32>(p, ctas, stream);
        case W4A16_FP16: return launch_one<W4A16_FP16>(p, ctas, stream);
        default: return launch_one<W4A16_BF16>(p, ctas, stream);
    }
}

}  // namespace w4a16
