// sample.cu -- the next token of each row of logits, and its C entry point.
//
// A row's tokens are ranked by logit, the lower index first among equals. Each
// filter keeps a prefix of that order: top-k its first k; top-p the shortest one
// with p of the mass that top-k left; min-p those with at least min_p of the
// largest weight. The token drawn is the one whose stretch of the kept mass, laid
// out in that order, holds the point u.
//
// So all that is asked of a row are places in its order, by count or by mass, and
// the row is never sorted. One histogram of 2048 bins, linear in the logit, says
// which bin holds a place. Where no more than 512 tokens lie up to there, they are
// listed, ranked and the row is done by one CTA; otherwise only the bin's own
// tokens are listed, or, if these are too many, told apart by histograms over their
// keys (the logits' bits, made to order as integers), 2048 bins a round: equal
// tokens need no list.
//
// Which token holds a point is a comparison of sums over the whole vocabulary:
// with 100000 tokens kept, an error of 1e-8 in the sums moves one draw in a
// thousand. So weights are computed to about 2^-36 (Weigher) and summed as
// integers of 2^-43, exactly and in any order: results do not depend on how a row
// is split, nor on the order of atomics. (The unit is what 64 bits leave for the sum
// of 2^20 tokens. Weights are rounded to it, to nothing below half of it: 2^-44 a
// token, 2^-24 of the largest weight where 2^20 tokens lie 30.5 temperatures below
// the top and are left out.) That costs about 45 instructions a token,
// which bounds rows of wide nuclei; where top-k or min-p leave few tokens, only
// theirs are computed, and the chain of steps over the cluster bounds the call.
//
// A row is a cluster's: its CTAs hold a slice of it each in shared memory, which
// is read from HBM once, and put their histograms together over distributed
// shared memory.
//
// Measured in a graph. One row of 131072 bf16 logits: top-k 50 and top-p 0.95 15.0
// us, no filter 18.5: a chain of about eight steps over the cluster, 1 to 2 us each.
// 61 rows of 50021 fp32, settings mixed: 61. 128 rows of 131072: greedy 38, top-k 50
// 50, no filter 127, top-p 0.98 of flat logits 154, where 109 million warp
// instructions at 0.66 an SM quarter's cycle are what it takes (the weights of all
// tokens once, 50 instructions each, two atomics, and three or four passes that
// compare).
#include <cooperative_groups.h>

#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "kv.cuh"
#include "moe_cache.h"

namespace moe {

namespace cg = cooperative_groups;

constexpr int kSampleThreads = 512, kSampleWarps = kSampleThreads / 32;
constexpr int kBins = 2048;
constexpr int kMaxCluster = 16;  // 8 where the device has no place for 16
constexpr int kMassBits = 43;                 // of weight 1: 2^20 tokens stay below 2^63
constexpr int kMaxVocab = 1 << 20;
constexpr uint32_t kKeyNegInf = 0x007fffffu;  // of -inf: the keys of numbers are above it
constexpr uint32_t kKeyInf = 0xff800000u;

struct SampleArgs {
    const void* logits;
    int64_t stride;
    int rows, vocab;
    int slice, held;  // values of a CTA's slice (a multiple of 8), and how many of them shared memory holds
    const float *temperature, *top_p, *min_p, *uniform;
    const int* top_k;
    int* tokens;
    float* logprobs;
};

struct Pow2Entry {  // 2^(r / 32), as a sum
    float hi, lo;
};
__device__ const Pow2Entry kPow2[32] = {
    {0x1.0000000000000p+0f, 0x0.0p+0f}, {0x1.059b0e0000000p+0f, -0x1.9d4f520000000p-25f}, {0x1.0b55860000000p+0f, 0x1.9f31220000000p-25f},
    {0x1.11301e0000000p+0f, -0x1.fdb4960000000p-25f}, {0x1.172b840000000p+0f, -0x1.c157420000000p-27f}, {0x1.1d48740000000p+0f, -0x1.d2e8ca0000000p-25f},
    {0x1.2387a60000000p+0f, 0x1.ceac480000000p-25f}, {0x1.29e9e00000000p+0f, -0x1.5c04240000000p-25f}, {0x1.306fe00000000p+0f, 0x1.4636e20000000p-25f},
    {0x1.371a740000000p+0f, -0x1.18aac60000000p-25f}, {0x1.3dea640000000p+0f, 0x1.8246840000000p-25f}, {0x1.44e0860000000p+0f, 0x1.8624b40000000p-30f},
    {0x1.4bfdae0000000p+0f, -0x1.593abc0000000p-25f}, {0x1.5342b60000000p+0f, -0x1.2c56100000000p-25f}, {0x1.5ab07e0000000p+0f, -0x1.5bd5ec0000000p-27f},
    {0x1.6247ec0000000p+0f, -0x1.f8b5500000000p-25f}, {0x1.6a09e60000000p+0f, 0x1.9fcef40000000p-26f}, {0x1.71f75e0000000p+0f, 0x1.1d8bee0000000p-25f},
    {0x1.7a11480000000p+0f, -0x1.829fd00000000p-25f}, {0x1.82589a0000000p+0f, -0x1.accc7c0000000p-26f}, {0x1.8ace540000000p+0f, 0x1.15506e0000000p-27f},
    {0x1.93737c0000000p+0f, -0x1.e647440000000p-25f}, {0x1.9c49180000000p+0f, 0x1.51f8480000000p-27f}, {0x1.a5503c0000000p+0f, -0x1.b83b540000000p-25f},
    {0x1.ae89fa0000000p+0f, -0x1.a94b140000000p-26f}, {0x1.b7f7700000000p+0f, -0x1.a094380000000p-25f}, {0x1.c199be0000000p+0f, -0x1.3d56b20000000p-27f},
    {0x1.cb720e0000000p+0f, -0x1.8837cc0000000p-27f}, {0x1.d5818e0000000p+0f, -0x1.822dbc0000000p-27f}, {0x1.dfc9740000000p+0f, -0x1.908c940000000p-25f},
    {0x1.ea4afa0000000p+0f, 0x1.52486c0000000p-27f}, {0x1.f507660000000p+0f, -0x1.246eb00000000p-26f},
};

// What a CTA tells the others of its cluster, a line per sender.
struct SampleNote {
    uint64_t mass;
    uint32_t a, b, c, d;
};
constexpr int kList = kSampleThreads;  // tokens that a list takes
struct alignas(16) SampleSmem {
    union {
        struct {
            uint32_t lo[kBins], hi[kBins];              // a histogram: counts in lo, or masses as two words
        };
        struct {
            uint64_t mine[kList];                       // the tokens that this CTA lists: key, ~index
            uint64_t list[kList], ranked[kList];        // the cluster's (rank 0)
        };
    };
    SampleNote note[2][kMaxCluster];            // a phase's and the next one's
    SampleNote found;                           // a place, by who found it
    uint64_t wmass[kSampleWarps], wsame[kSampleWarps];
    uint32_t wcnt[kSampleWarps], wa[kSampleWarps], wb[kSampleWarps], wc[kSampleWarps];
    int listed;
    float c, cl;                                // log2 e / temperature
    double least;                               // temperature * log min_p
    // behind it: this CTA's chunk of the cluster's histogram (kBins / CTAs sums), then the values held
};

// Keys order as the values do; -0 is 0.
__device__ __forceinline__ uint32_t key_of(float v) {
    const uint32_t u = __float_as_uint(v + 0.0f);
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t key) {
    return __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key);
}

// 2^(c (v - top)) in units of 2^-kMassBits, c = log2 e / temperature. Whole warps.
//
// v - top is taken as a sum of two floats, and x = c (v - top) as x + xl. With k =
// rint(32 x) and g = x - k / 32 (exact, at most 1/64), 2^x = 2^(k/32) (1 + z), z =
// e^y - 1 for y = (g + xl) ln 2: the first term h = g ln 2 with its rounding, the
// others by the series up to y^5 / 120 (the next term is below 2^-48). The power
// 2^(r/32), r = k mod 32, is held by lane r as hi + lo (a shuffle has no bank
// conflicts, as a table in shared memory has); hi * h keeps its rounding. The
// largest error left is that of the last sums, about 2^-36. (A c below 2^-100 has not all
// of its bits in two floats: off by 2^-150, which v - top from 2^114 on shows.)
struct Weigher {
    float top, c, cl, hi, lo;  // hi, lo: this lane's power
    __device__ __forceinline__ uint64_t operator()(float v) const {
        const float d = v - top, t = d - v, dl = (v - (d - t)) + (-top - t);
        const float x = d * c;
        const bool some = x > -44.f;  // not below half a unit, nor -inf
        const float xl = fmaf(dl, c, fmaf(d, cl, fmaf(d, c, -x)));
        const float j = fmaf(x, 32.f, 12582912.f), kf = j - 12582912.f;  // 1.5 2^23: rint in the last bits
        const int k = __float_as_int(j) - 0x4b400000;
        const float g = fmaf(kf, -0.03125f, x);
        constexpr float kLn2 = 0.693147182f, kLn2Lo = -1.90465421e-9f;
        const float h = g * kLn2;
        const float e = fmaf(xl, kLn2, fmaf(g, kLn2Lo, fmaf(g, kLn2, -h)));
        const float y = h + e;
        const float s = fmaf(y, fmaf(y, fmaf(y, 1.f / 120.f, 1.f / 24.f), 1.f / 6.f), 0.5f);
        const float q = fmaf(y * y, s, e);
        const float p = __shfl_sync(0xffffffffu, hi, k & 31), pl = __shfl_sync(0xffffffffu, lo, k & 31);
        const float a = p * h, b = fmaf(pl, h, fmaf(p, q, fmaf(p, h, -a))) + pl;
        // in units of 2^-36: p is in [1, 2), its bits those of an integer
        const int b2 = __float_as_int(fmaf(b, 0x1p35f, 12582912.f)) - 0x4b400000;  // b is below 2^-13
        const uint64_t m = ((uint64_t)((__float_as_uint(p) & 0x7fffffu) | 0x800000u) << 13) +
                           (uint64_t)(int64_t)(__float2int_rn(a * 0x1p36f) + 2 * b2);
        // 2^(k / 32) = 2^(k >> 5) 2^(r / 32)
        const int down = 63 & -(k >> 5);
        return some ? ((m << (kMassBits - 36)) + ((1ull << down) >> 1)) >> down : 0;
    }
};

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.aligned;\n" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.aligned;\n" ::: "memory"); }

// mass * f for 0 <= f <= 1, exactly: rounded down, or up.
__device__ __forceinline__ uint64_t part_of(uint64_t mass, float f, bool up) {
    const uint32_t bits = __float_as_uint(f), e = bits >> 23;
    const uint64_t mant = (bits & 0x7fffffu) | (e ? 0x800000u : 0u);
    const int down = 150 - (int)max(e, 1u);  // f = mant 2^-down, down >= 23
    const uint64_t lo = mass * mant, hi = __umul64hi(mass, mant);
    if (down >= 64) {
        const int d = down - 64;
        const uint64_t q = d > 63 ? 0 : hi >> d;
        return q + (up && (lo != 0 || (d > 63 ? hi != 0 : (q << d) != hi)));
    }
    const uint64_t q = lo >> down | hi << (64 - down);
    return q + (up && (q << down) != lo);
}

template <class T>
struct Slice {
    const T* smem;
    const T* row;  // of the slice
    int held;
    __device__ __forceinline__ float operator()(int i) const {
        const T v = i < held ? smem[i] : row[i];
        if constexpr (sizeof(T) == 4) return v;
        else return __uint_as_float((uint32_t)v << 16);
    }
};

template <class T>
__global__ void __launch_bounds__(kSampleThreads, 2) k_sample(SampleArgs a) {
    extern __shared__ __align__(16) uint8_t raw[];
    SampleSmem& sm = *reinterpret_cast<SampleSmem*>(raw);
    cg::cluster_group cluster = cg::this_cluster();
    const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int chunk = kBins / C;  // bins that a CTA puts together
    uint64_t* sums = reinterpret_cast<uint64_t*>(raw + sizeof(SampleSmem));
    T* values = reinterpret_cast<T*>(sums + chunk);
    const int row = (int)(blockIdx.x / (unsigned)C), tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int first = min(rank * a.slice, a.vocab), n = min(a.slice, a.vocab - first);  // of this CTA's slice

    cluster_arrive();
    if (tid == 0) sm.listed = 0;
    const Pow2Entry pow2 = kPow2[lane];
    griddep_wait();
    griddep_launch();
    const T* src = (const T*)a.logits + row * a.stride + first;
    const Slice<T> value = {values, src, min(a.held, n)};
    float temp = a.temperature ? a.temperature[row] : 1.f;
    if (temp > 0.f) temp = fmaxf(temp, 0x1p-99f);  // log2 e / temp stays far below fp32's largest
    const float top_p = a.top_p ? a.top_p[row] : 1.f;
    const float min_p = a.min_p ? a.min_p[row] : 0.f, u = a.uniform ? a.uniform[row] : 0.f;
    const int top_k = a.top_k ? a.top_k[row] : 0;
    const bool greedy = !a.uniform || temp == 0.f;
    if (tid == 0) {  // fp64 is slow: one thread's work
        const double c = 1.4426950408889634 / (double)temp;
        sm.c = (float)c;
        sm.cl = (float)(c - (double)sm.c);
        if (min_p > 0.f) sm.least = (double)temp * log((double)min_p);
    }

    // --- the slice into shared memory; its largest key, its smallest of a number, NaN
    float most = -INFINITY, least = INFINITY;
    uint32_t bad = 0;
    auto look = [&](float v) {
        bad |= v != v;
        most = fmaxf(most, v);
        least = fminf(least, v == -INFINITY ? INFINITY : v);
    };
    constexpr int kPer = 16 / sizeof(T);
    auto unpack = [&](const uint4& w, float (&v)[kPer]) {
        const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if constexpr (sizeof(T) == 4) {
                v[e] = __uint_as_float(x[e]);
            } else {
                v[2 * e] = __uint_as_float(x[e] << 16);
                v[2 * e + 1] = __uint_as_float(x[e] & 0xffff0000u);
            }
        }
    };
    {
        const int whole = ((uintptr_t)src & 15u) == 0 ? n / kPer * kPer : 0;
#pragma unroll 4
        for (int i = tid * kPer; i < whole; i += kSampleThreads * kPer) {
            const uint4 w = *reinterpret_cast<const uint4*>(src + i);
            if (i < value.held) *reinterpret_cast<uint4*>(values + i) = w;  // `held` is a multiple of 8, or all
            float v[kPer];
            unpack(w, v);
#pragma unroll
            for (int e = 0; e < kPer; ++e) look(v[e]);
        }
#pragma unroll 8
        for (int i = whole + tid; i < n; i += kSampleThreads) {
            const T v = src[i];
            if (i < value.held) values[i] = v;
            if constexpr (sizeof(T) == 4) look(v);
            else look(__uint_as_float((uint32_t)v << 16));
        }
    }
    // f(value, index) for all of the slice, by whole warps; -inf in the place of what is past it
    auto each = [&](auto f) {
        const int whole = value.held / kPer * kPer;
        for (int i0 = warp * 32 * kPer; i0 < whole; i0 += kSampleThreads * kPer) {
            const int i = i0 + lane * kPer;
            float v[kPer];
            if (i < whole) {
                unpack(*reinterpret_cast<const uint4*>(values + i), v);
            } else {
#pragma unroll
                for (int e = 0; e < kPer; ++e) v[e] = -INFINITY;
            }
#pragma unroll
            for (int e = 0; e < kPer; ++e) f(v[e], i + e);
        }
        for (int i0 = whole + warp * 32; i0 < n; i0 += kSampleThreads) f(i0 + lane < n ? value(i0 + lane) : -INFINITY, i0 + lane);
    };
    int phase = 0;
    // Every CTA's note to every CTA; all of them afterwards in sm.note[...], until the next but one.
    auto tell = [&](const SampleNote& note) -> const SampleNote* {
        phase ^= 1;
        if (tid < C) cluster.map_shared_rank(&sm, tid)->note[phase][rank] = note;
        cluster.sync();
        return sm.note[phase];
    };
    uint32_t kmax = __reduce_max_sync(0xffffffffu, key_of(most)), kmin = __reduce_min_sync(0xffffffffu, key_of(least));
    bad = __reduce_or_sync(0xffffffffu, bad);
    if (lane == 0) sm.wa[warp] = kmax, sm.wb[warp] = kmin, sm.wc[warp] = bad;
    __syncthreads();
    for (int w = 0; w < kSampleWarps; ++w) kmax = max(kmax, sm.wa[w]), kmin = min(kmin, sm.wb[w]), bad |= sm.wc[w];
    cluster_wait();  // the others have started
    {
        const SampleNote* all = tell({0, kmax, kmin, bad, 0});
        for (int r = 0; r < C; ++r) kmax = max(kmax, all[r].a), kmin = min(kmin, all[r].b), bad |= all[r].c;
    }
    bad |= kmax >= kKeyInf || kmax <= kKeyNegInf || !(temp >= 0.f && temp <= 3.4028235e38f) || top_p != top_p ||
           min_p != min_p || u != u;

    auto logprob_of = [&](uint32_t key, uint64_t mass) {
        return (float)(((double)value_of(key) - (double)value_of(kmax)) / (double)temp - log((double)mass * (1.0 / (1ull << kMassBits))));
    };
    // The j-th token (from 0) of a key, in the order of the indexes: the CTA that has it writes it.
    auto pick = [&](uint32_t key, uint64_t j, uint64_t mass) {
        const int per = (n + kSampleThreads - 1) / kSampleThreads * 32;  // a warp's stretch of the slice
        const int from = min(warp * per, n), to = min(from + per, n);
        auto hits = [&](int i) { return __ballot_sync(0xffffffffu, i + lane < to && key_of(value(min(i + lane, n - 1))) == key); };
        unsigned mine = 0;
        for (int i = from; i < to; i += 32) mine += __popc(hits(i));
        __syncthreads();
        if (lane == 0) sm.wcnt[warp] = mine;
        __syncthreads();
        unsigned before = 0, sum = 0;
        for (int w = 0; w < kSampleWarps; ++w) {
            if (w == warp) before = sum;
            sum += sm.wcnt[w];
        }
        const SampleNote* all = tell({0, sum, 0, 0, 0});
        uint64_t at = before;
        for (int r = 0; r < rank; ++r) at += all[r].a;
        if (at > j || j >= at + mine) return;
        for (int i = from; i < to; i += 32) {
            unsigned hit = hits(i);
            if (j < at + __popc(hit)) {
                for (int skip = (int)(j - at); skip; --skip) hit &= hit - 1;
                if (lane == 0) {
                    a.tokens[row] = first + i + __ffs(hit) - 1;
                    if (a.logprobs) a.logprobs[row] = greedy ? 0.f : logprob_of(key, mass);
                }
                return;
            }
            at += __popc(hit);
        }
    };
    auto finish = [&]() { cluster.sync(); };  // no CTA leaves while another may read or write its memory

    if (bad) {
        if (rank == 0 && tid == 0) {
            a.tokens[row] = -1;
            if (a.logprobs) a.logprobs[row] = __int_as_float(0x7fc00000);
        }
        finish();
        return;
    }
    if (greedy) {
        pick(kmax, 0, 0);
        finish();
        return;
    }

    const float top = value_of(kmax);
    const Weigher weigh = {top, sm.c, sm.cl, pow2.hi, pow2.lo};
    auto weight_of = [&](uint32_t key) { return weigh(value_of(key)); };

    // Bins of the histogram over the row: linear in the logit down to where weights are nothing, or to the
    // row's lowest; the last one has all that is lower. The grain stays finite, so that the top is bin 0's.
    const float reach = fminf(top - value_of(kmin), 44.5f / sm.c), grain = (float)(kBins - 1) / fmaxf(reach, 0x1p-110f);
    auto bin_of_value = [&](float v) {  // 1.5 2^23: the nearest whole number in the last bits
        return __float_as_int(fminf((v - top) * -grain, (float)(kBins - 1)) + 12582912.f) - 0x4b400000;
    };
    // The lowest key of bins up to b. (The bins order as the keys do.)
    auto lowest_key = [&](int b) {
        uint32_t lo = kmin, hi = kmax;  // the answer is among them, and hi is one of those bins'
        while (lo < hi) {
            const uint32_t mid = lo + (hi - lo) / 2;
            if (bin_of_value(value_of(mid)) <= b) hi = mid;
            else lo = mid + 1;
        }
        return lo;
    };

    // The histogram by bin(value) (below 0: not in it), put together: this CTA's chunk in sums. few: where a
    // warp often has none in it. (It takes the lists' memory: behind a list comes a barrier of the cluster
    // before the next one.)
    auto histogram = [&](auto bin_of, bool by_count, bool few) {
        for (int b = tid; b < kBins; b += kSampleThreads) sm.lo[b] = sm.hi[b] = 0;
        __syncthreads();
        each([&](float v, int) {
            const int b = bin_of(v);
            if (by_count) {
                if (b >= 0) atomicAdd(&sm.lo[b], 1u);
            } else {
                if (few && !__any_sync(0xffffffffu, b >= 0)) return;
                const uint64_t w = weigh(v);
                if (b >= 0 && w) {
                    const uint32_t old = atomicAdd(&sm.lo[b], (uint32_t)w);
                    const uint32_t high = (uint32_t)(w >> 32) + (old + (uint32_t)w < old);
                    if (high) atomicAdd(&sm.hi[b], high);
                }
            }
        });
        cluster.sync();
        for (int b = tid; b < chunk; b += kSampleThreads) {
            uint64_t sum = 0;
            for (int r = 0; r < C; ++r) {
                const SampleSmem* s = cluster.map_shared_rank(&sm, r);
                const int at = rank * chunk + b;
                sum += (uint64_t)s->hi[at] << 32 | s->lo[at];
            }
            sums[b] = sum;
        }
        __syncthreads();
    };
    // The bin of the histogram put together that holds the point that point_of gives for the total: its number
    // (-1: the point is not below the total), what lies before it, and what up to its end.
    struct Bin {
        int bin;
        uint64_t before, upto;
    };
    auto find_bin = [&](auto point_of) -> Bin {
        // each thread a stretch of the chunk
        const int per = (chunk + kSampleThreads - 1) / kSampleThreads, b0 = min(tid * per, chunk), b1 = min(b0 + per, chunk);
        uint64_t size = 0;
        for (int b = b0; b < b1; ++b) size += sums[b];
        uint64_t upto = size;
        for (int off = 1; off < 32; off <<= 1) {
            const uint64_t v = __shfl_up_sync(0xffffffffu, upto, off);
            if (lane >= off) upto += v;
        }
        __syncthreads();
        if (lane == 31) sm.wmass[warp] = upto;
        __syncthreads();
        uint64_t here = 0, at = upto - size;
        for (int w = 0; w < kSampleWarps; ++w) {
            if (w < warp) at += sm.wmass[w];
            here += sm.wmass[w];
        }
        const SampleNote* all = tell({here, 0, 0, 0, 0});
        uint64_t total = 0;
        for (int r = 0; r < C; ++r) {
            if (r < rank) at += all[r].mass;
            total += all[r].mass;
        }
        const uint64_t point = point_of(total);
        if (point < total && at <= point && point < at + size) {
            int b = b0;
            while (point >= at + sums[b]) at += sums[b++];
            const uint64_t end = at + sums[b];
            for (int r = 0; r < C; ++r)
                cluster.map_shared_rank(&sm, r)->found = {at, (uint32_t)(rank * chunk + b), (uint32_t)end, (uint32_t)(end >> 32), 0};
        }
        cluster.sync();
        if (point >= total) return {-1, 0, 0};
        return {(int)sm.found.a, sm.found.mass, (uint64_t)sm.found.c << 32 | sm.found.b};
    };
    // The tokens of values lo .. hi, in rank 0's list if there are at most kList; their number, and their
    // lowest and highest key.
    uint32_t listed_lo, listed_hi;
    auto gather = [&](float lo, float hi) -> int {
        float least = INFINITY, most = -INFINITY;
        each([&](float v, int i) {
            const bool in = v >= lo && v <= hi;
            const unsigned hit = __ballot_sync(0xffffffffu, in);
            if (!hit) return;
            if (in) least = fminf(least, v), most = fmaxf(most, v);
            int at = 0;
            if (lane == 0) at = atomicAdd(&sm.listed, __popc(hit));
            at = __shfl_sync(0xffffffffu, at, 0) + __popc(hit & ((1u << lane) - 1u));
            if (in && at < kList) sm.mine[at] = (uint64_t)key_of(v) << 32 | (uint32_t)~(first + i);
        });
        listed_lo = __reduce_min_sync(0xffffffffu, key_of(least));
        listed_hi = __reduce_max_sync(0xffffffffu, key_of(most));
        if (lane == 0) sm.wa[warp] = listed_hi, sm.wb[warp] = listed_lo;
        __syncthreads();
        for (int w = 0; w < kSampleWarps; ++w) listed_hi = max(listed_hi, sm.wa[w]), listed_lo = min(listed_lo, sm.wb[w]);
        const SampleNote* all = tell({0, (uint32_t)sm.listed, listed_lo, listed_hi, 0});
        if (tid == 0) sm.listed = 0;
        int sum = 0, from = -1, at = 0;
        for (int r = 0; r < C; ++r) {
            listed_lo = min(listed_lo, all[r].b);
            listed_hi = max(listed_hi, all[r].c);
            const int here = (int)all[r].a;
            if (from < 0 && tid < sum + here) from = r, at = tid - sum;
            sum += here;
        }
        if (rank == 0 && sum <= kList) {
            if (from >= 0) sm.list[tid] = cluster.map_shared_rank(&sm, from)->mine[at];
            else if (tid == sum) sm.list[tid] = 0;  // the list is read in pairs
        }
        __syncthreads();  // and `listed` is 0 again before the next list
        return sum;
    };
    // Rank 0: the list in order. Thread r gets the r-th token (0 past the end), its weight, and what lies before it.
    struct Ranked {
        uint64_t token, weight, before;
    };
    auto rank_list = [&](int count, bool by_count) -> Ranked {
        const uint64_t mine = tid < count ? sm.list[tid] : 0;
        int above = 0;
        if (warp * 32 < count)
#pragma unroll 8
            for (int e = 0; e < count; e += 2) {
                const ulonglong2 two = *reinterpret_cast<const ulonglong2*>(sm.list + e);
                above += (two.x > mine) + (two.y > mine);
            }
        if (tid < count) sm.ranked[above] = mine;
        __syncthreads();
        Ranked r;
        r.token = tid < count ? sm.ranked[tid] : 0;
        const uint64_t w = weigh(tid < count ? value_of((uint32_t)(r.token >> 32)) : -INFINITY);
        r.weight = tid >= count ? 0 : by_count ? 1 : w;
        uint64_t upto = r.weight;
        for (int off = 1; off < 32; off <<= 1) {
            const uint64_t v = __shfl_up_sync(0xffffffffu, upto, off);
            if (lane >= off) upto += v;
        }
        if (lane == 31) sm.wmass[warp] = upto;
        __syncthreads();
        r.before = upto - r.weight;
        for (int w2 = 0; w2 < warp; ++w2) r.before += sm.wmass[w2];
        return r;
    };

    const bool some_p = top_p < 1.f, some_min = min_p > 0.f;
    const uint32_t k_least = some_min ? (min_p > 1.f ? kmax : key_of(__double2float_ru((double)top + sm.least))) : 0;
    // The row, where the list holds all tokens up to the last one kept (and maybe more): the first k of
    // them, p of `mass` (0: of theirs), min-p, and the draw.
    auto finish_list = [&](int count, int k, uint64_t mass) {
        if (rank == 0) {
            const Ranked r = rank_list(count, false);
            const uint64_t upto = r.before + r.weight;
            const int last = min(k, count) - 1;
            if (tid == last) sm.wsame[0] = upto;
            __syncthreads();
            if (mass == 0) mass = sm.wsame[0];
            const uint64_t want = !some_p ? ~0ull : top_p > 0.f ? max(part_of(mass, top_p, true), (uint64_t)1) : 1;
            const bool keep = tid <= last && (tid == 0 || (r.before < want && !(min_p > 1.f) && (uint32_t)(r.token >> 32) >= k_least));
            const int kept = __syncthreads_count(keep);  // a prefix
            if (tid == kept - 1) sm.wsame[1] = upto;
            __syncthreads();
            const uint64_t left = sm.wsame[1], point = min(part_of(left, fminf(fmaxf(u, 0.f), 1.f), false), left - 1);
            if (keep && r.before <= point && point < upto) {
                a.tokens[row] = (int)~(uint32_t)r.token;
                if (a.logprobs) a.logprobs[row] = logprob_of((uint32_t)(r.token >> 32), left);
            }
        }
        finish();
    };
    // A point's place in a bin of the row's histogram: the key, what lies before it, and the number of the
    // token among the key's.
    struct Place {
        uint32_t key;
        uint64_t before, j;
        unsigned same;  // tokens of the key
    };
    auto shift_of = [](uint32_t klo, uint32_t khi) {
        int s = 0;
        while (((khi - klo) >> s) >= (uint32_t)kBins) ++s;
        return s;
    };
    bool fresh = true;  // the row's histogram is still there
    // (Where `draw` and the list holds the token, it is written, and `done`.)
    auto place_in = [&](const Bin& bin, uint32_t from, uint64_t point, bool by_count, uint64_t draw, bool& done) -> Place {
        const uint32_t last = lowest_key(bin.bin);
        uint32_t klo = max(from, last), khi = bin.bin ? lowest_key(bin.bin - 1) - 1 : kmax;
        const int count = gather(value_of(klo), value_of(khi));
        if (count <= kList) {
            if (rank == 0) {
                const Ranked r = rank_list(count, by_count);
                const uint64_t rest = point - bin.before;
                if (r.before <= rest && rest < r.before + r.weight) {
                    const uint32_t key = (uint32_t)(r.token >> 32);
                    if (draw) {
                        a.tokens[row] = (int)~(uint32_t)r.token;
                        if (a.logprobs) a.logprobs[row] = logprob_of(key, draw);
                    } else {
                        int j = 0, to = tid + 1;  // tokens of its key before it, and their end
                        while (j < tid && (uint32_t)(sm.ranked[tid - 1 - j] >> 32) == key) ++j;
                        while (to < count && (uint32_t)(sm.ranked[to] >> 32) == key) ++to;
                        const SampleNote note = {bin.before + r.before - j * r.weight, key, (uint32_t)j, (uint32_t)(to - tid + j), 0};
                        for (int q = 0; q < C; ++q) cluster.map_shared_rank(&sm, q)->found = note;
                    }
                }
            }
            done = draw != 0;
            if (!done) cluster.sync();
            return {sm.found.a, sm.found.mass, sm.found.b, sm.found.c};
        }
        klo = listed_lo;
        khi = listed_hi;
        uint64_t before = bin.before, upto = bin.upto;
        while (klo < khi) {
            fresh = false;
            const int shift = shift_of(klo, khi);
            histogram([&](float v) {
                const uint32_t key = key_of(v);
                return key >= klo && key <= khi ? (int)((khi - key) >> shift) : -1;
            }, by_count, true);
            const Bin b = find_bin([&](uint64_t) { return point - before; });
            upto = before + b.upto;
            before += b.before;
            khi -= (uint32_t)b.bin << shift;
            const uint32_t width = (1u << shift) - 1u;
            klo = khi - klo > width ? khi - width : klo;
        }
        const uint64_t w = by_count ? 1 : weight_of(khi);
        return {khi, before, (point - before) / w, (unsigned)((upto - before) / w)};
    };
    // the mass of the tokens of keys from `from` on
    auto mass_from = [&](uint32_t from) {
        uint64_t mine = 0;
        const float bound = value_of(from);
        each([&](float v, int) {
            if (!__any_sync(0xffffffffu, v >= bound)) return;
            const uint64_t w = weigh(v);
            if (v >= bound) mine += w;
        });
        for (int off = 16; off; off >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, off);
        __syncthreads();
        if (lane == 0) sm.wmass[warp] = mine;
        __syncthreads();
        mine = 0;
        for (int w = 0; w < kSampleWarps; ++w) mine += sm.wmass[w];
        const SampleNote* all = tell({mine, 0, 0, 0, 0});
        mine = 0;
        for (int r = 0; r < C; ++r) mine += all[r].mass;
        return mine;
    };

    constexpr int kNoCut = 0x7fffffff;
    bool done = false;
    // --- top-k: the last key kept, and how many of its tokens
    uint32_t k_keep = kmin;
    uint64_t spare = 0;  // tokens of that key that are not
    bool cut = false;
    if (top_k > 0 && top_k < a.vocab) {
        histogram([&](float v) { return v > -INFINITY ? bin_of_value(v) : -1; }, true, false);
        const Bin b = find_bin([&](uint64_t) { return (uint64_t)(top_k - 1); });
        if (b.bin >= 0 && b.upto <= (uint64_t)kList) {
            finish_list(gather(value_of(lowest_key(b.bin)), top), top_k, 0);
            return;
        }
        if (b.bin >= 0) {
            const Place p = place_in(b, kmin, (uint64_t)(top_k - 1), true, 0, done);
            k_keep = p.key;
            spare = p.same - (p.j + 1);
            cut = true;
        }
    }
    if (!cut && !some_p && some_min && k_least > kmin) {
        // min-p alone
        const int count = gather(value_of(k_least), top);
        if (count <= kList) {
            finish_list(count, kNoCut, 0);
            return;
        }
        k_keep = k_least;
    }
    // --- the masses
    const uint32_t from = k_keep;
    auto masses = [&]() {
        const float bound = value_of(from);
        histogram([&](float v) { return v >= bound ? bin_of_value(v) : -1; }, false, from > kmin);
        fresh = true;
    };
    masses();
    const uint64_t beyond = cut ? spare * weight_of(k_keep) : 0;  // the histogram's, not kept
    uint64_t mass = 0;                                            // 0: all of the histogram's but that
    if (some_p) {
        // the tokens with less than p of the mass before them, the first one among them
        uint64_t last = 0;
        const Bin b = find_bin([&](uint64_t total) {
            mass = total - beyond;
            return last = top_p > 0.f ? max(part_of(mass, top_p, true), (uint64_t)1) - 1 : 0;
        });
        if ((b.before >> kMassBits) < (uint64_t)kList) {  // at least so many tokens come before the bin
            const int count = gather(value_of(max(from, lowest_key(b.bin))), top);
            if (count <= kList) {
                finish_list(count, cut ? top_k : kNoCut, mass);
                return;
            }
        }
        const Place p = place_in(b, from, last, false, 0, done);
        k_keep = p.key;
        mass = p.before + (p.j + 1) * weight_of(p.key);
    }
    if (some_min && min_p > 1.f) {
        pick(kmax, 0, weight_of(kmax));
        finish();
        return;
    }
    if (some_min && k_least > k_keep) {
        k_keep = k_least;
        mass = mass_from(k_keep);
    }
    // --- the draw
    if (!fresh) masses();
    uint64_t point = 0;
    const Bin b = find_bin([&](uint64_t total) {
        if (mass == 0) mass = total - beyond;
        return point = min(part_of(mass, fminf(fmaxf(u, 0.f), 1.f), false), mass - 1);
    });
    const Place p = place_in(b, from, point, false, mass, done);
    if (!done) pick(p.key, p.j, mass);
    finish();
}

template <class T>
static cudaError_t launch_sample(SampleArgs a, int dev, cudaStream_t st) {
    constexpr int kHeldBytes = 68 * 1024;
    static DeviceOnce once;
    const cudaError_t set = once.run(dev, [] {
        const cudaError_t e = cudaFuncSetAttribute(k_sample<T>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
        return cudaFuncSetAttribute(k_sample<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    (int)(sizeof(SampleSmem) + kBins * sizeof(uint64_t)) + kHeldBytes);
    });
    if (set != cudaSuccess) return set;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kSampleThreads);
    cfg.stream = st;
    // A row's CTAs: enough that its slices fit in shared memory with two CTAs on an SM, and more as far as all
    // rows' run at once (61 rows of 50021: 4 CTAs a row 61 us, 8 in two rounds 67). 16 for up to four rows (one
    // of 131072: 14.8 us, 8 CTAs 15.6; without filters 18.5 and 22.4).
    const int sms = sm_count(dev);
    int C = 1;
    auto slice_of = [&](int c) { return ((a.vocab + c - 1) / c + 7) / 8 * 8; };
    while (C < 8 && (size_t)slice_of(C) * sizeof(T) > kHeldBytes) C *= 2;
    while (C < 8 && (int64_t)a.rows * 2 * C <= 2 * sms && slice_of(C) > 2048) C *= 2;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    auto split = [&](int c) {
        C = c;
        a.slice = slice_of(C);
        a.held = (int)std::min<int64_t>(a.slice, kHeldBytes / sizeof(T));
        cfg.gridDim = dim3((unsigned)(a.rows * C));
        cfg.dynamicSmemBytes = sizeof(SampleSmem) + kBins / C * sizeof(uint64_t) + (size_t)a.held * sizeof(T);
        attr[1].val.clusterDim.x = (unsigned)C;
    };
    if (C == 8 && a.rows <= 4 && slice_of(C) > 2048) {
        static std::atomic<int> most[kMaxDevices] = {};  // clusters of 16 that fit the device, + 1
        int known = dev < kMaxDevices ? most[dev].load(std::memory_order_relaxed) : 0;
        if (!known) {
            split(16);
            cfg.dynamicSmemBytes = sizeof(SampleSmem) + kBins / C * sizeof(uint64_t) + kHeldBytes;
            if (cudaOccupancyMaxActiveClusters(&known, k_sample<T>, &cfg) != cudaSuccess) {
                cudaGetLastError();
                known = 0;
            }
            ++known;
            if (dev < kMaxDevices) most[dev].store(known, std::memory_order_relaxed);
        }
        C = known > 4 ? 16 : 8;
    }
    split(C);
    return cudaLaunchKernelEx(&cfg, k_sample<T>, a);
}

}  // namespace moe

namespace {
moe_status_t refuse(const char* msg) {
    moe::set_last_error(msg);
    return MOE_ERR_INVALID;
}
}  // namespace

extern "C" moe_status_t moe_sample(const void* logits, int32_t type, int64_t row_stride, int32_t rows, int32_t vocab,
                                   const moe_sampling_t* settings, int32_t* tokens, float* logprobs, void* stream) {
    if (rows < 0 || rows > (1 << 24)) return refuse("rows must be in 0..2^24");
    if (vocab < 1 || vocab > moe::kMaxVocab) return refuse("vocab must be in 1..2^20");
    if (type != MOE_TYPE_BF16 && type != MOE_TYPE_F32) return refuse("type must be MOE_TYPE_BF16 or MOE_TYPE_F32");
    if (!settings) return refuse("NULL settings");
    if (rows == 0) return MOE_OK;
    if (!logits || !tokens) return refuse("NULL logits or tokens");
    if (row_stride < vocab && rows > 1) return refuse("rows must be at least vocab elements apart");
    if ((uintptr_t)logits % (type == MOE_TYPE_F32 ? 4 : 2) ||
        (((uintptr_t)settings->temperature | (uintptr_t)settings->top_k | (uintptr_t)settings->top_p | (uintptr_t)settings->min_p |
          (uintptr_t)settings->uniform | (uintptr_t)tokens | (uintptr_t)logprobs) & 3u))
        return refuse("an array is not aligned to its type");
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    const moe::SampleArgs a = {logits, row_stride, rows, vocab, 0, 0, settings->temperature, settings->top_p, settings->min_p,
                               settings->uniform, settings->top_k, tokens, logprobs};
    if (e == cudaSuccess)
        e = type == MOE_TYPE_F32 ? moe::launch_sample<float>(a, dev, (cudaStream_t)stream)
                                 : moe::launch_sample<uint16_t>(a, dev, (cudaStream_t)stream);
    if (e == cudaSuccess) return MOE_OK;
    moe::set_last_error(cudaGetErrorString(e));
    return MOE_ERR_CUDA;
}
