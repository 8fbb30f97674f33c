// sample.cu -- the next token of each row of logits, and its C entry point.
//
// A row's tokens are ranked by logit, the lower index first among equals. Each
// filter keeps a prefix of that order: top-k its first k; top-p the shortest one
// with p of the mass that top-k left; min-p those with at least min_p of the
// largest weight. The token drawn is the one whose stretch of the kept mass, laid
// out in that order, holds the point u.
//
// So all that is asked of a row are places in its order, by count or by mass, and
// nothing is sorted: a place is found by a histogram over the keys (the logits'
// bits, made to order as integers), then over the bin that holds it, until a bin
// is a single key. 2048 bins at a time, so bf16 logits take two rounds, fp32 up to
// three.
//
// Which token holds a point is a comparison of sums over the whole vocabulary:
// with 100000 tokens kept, an error of 1e-8 in the sums moves one draw in a
// thousand. So weights are computed to about 2^-36 (weight_of) and summed as
// integers of 2^-43, exactly and in any order: results do not depend on how a row
// is split, nor on the order of atomics.
//
// A row is a cluster's: its CTAs hold a slice of it each in shared memory, which
// is read from HBM once, and put their histograms together over distributed
// shared memory.
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
constexpr int kMaxCluster = 8;
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

struct alignas(16) Pow2Entry {  // 2^(r / 32)
    float hi, lo;               // as a sum
    unsigned long long fixed;   // in units of 2^-36
};
__device__ const Pow2Entry kPow2[32] = {
    {0x1.0000000000000p+0f, 0x0.0p+0f, 68719476736ull}, {0x1.059b0e0000000p+0f, -0x1.9d4f520000000p-25f, 70224237334ull},
    {0x1.0b55860000000p+0f, 0x1.9f31220000000p-25f, 71761947898ull}, {0x1.11301e0000000p+0f, -0x1.fdb4960000000p-25f, 73333329938ull},
    {0x1.172b840000000p+0f, -0x1.c157420000000p-27f, 74939120765ull}, {0x1.1d48740000000p+0f, -0x1.d2e8ca0000000p-25f, 76580073833ull},
    {0x1.2387a60000000p+0f, 0x1.ceac480000000p-25f, 78256959093ull}, {0x1.29e9e00000000p+0f, -0x1.5c04240000000p-25f, 79970563360ull},
    {0x1.306fe00000000p+0f, 0x1.4636e20000000p-25f, 81721690674ull}, {0x1.371a740000000p+0f, -0x1.18aac60000000p-25f, 83511162683ull},
    {0x1.3dea640000000p+0f, 0x1.8246840000000p-25f, 85339819026ull}, {0x1.44e0860000000p+0f, 0x1.8624b40000000p-30f, 87208517730ull},
    {0x1.4bfdae0000000p+0f, -0x1.593abc0000000p-25f, 89118135606ull}, {0x1.5342b60000000p+0f, -0x1.2c56100000000p-25f, 91069568669ull},
    {0x1.5ab07e0000000p+0f, -0x1.5bd5ec0000000p-27f, 93063732552ull}, {0x1.6247ec0000000p+0f, -0x1.f8b5500000000p-25f, 95101562938ull},
    {0x1.6a09e60000000p+0f, 0x1.9fcef40000000p-26f, 97184015999ull}, {0x1.71f75e0000000p+0f, 0x1.1d8bee0000000p-25f, 99312068844ull},
    {0x1.7a11480000000p+0f, -0x1.829fd00000000p-25f, 101486719979ull}, {0x1.82589a0000000p+0f, -0x1.accc7c0000000p-26f, 103708989773ull},
    {0x1.8ace540000000p+0f, 0x1.15506e0000000p-27f, 105979920939ull}, {0x1.93737c0000000p+0f, -0x1.e647440000000p-25f, 108300579022ull},
    {0x1.9c49180000000p+0f, 0x1.51f8480000000p-27f, 110672052900ull}, {0x1.a5503c0000000p+0f, -0x1.b83b540000000p-25f, 113095455294ull},
    {0x1.ae89fa0000000p+0f, -0x1.a94b140000000p-26f, 115571923291ull}, {0x1.b7f7700000000p+0f, -0x1.a094380000000p-25f, 118102618875ull},
    {0x1.c199be0000000p+0f, -0x1.3d56b20000000p-27f, 120688729477ull}, {0x1.cb720e0000000p+0f, -0x1.8837cc0000000p-27f, 123331468528ull},
    {0x1.d5818e0000000p+0f, -0x1.822dbc0000000p-27f, 126032076028ull}, {0x1.dfc9740000000p+0f, -0x1.908c940000000p-25f, 128791819132ull},
    {0x1.ea4afa0000000p+0f, 0x1.52486c0000000p-27f, 131611992741ull}, {0x1.f507660000000p+0f, -0x1.246eb00000000p-26f, 134493920110ull},
};

// What a CTA tells the others of its cluster, a line per sender.
struct SampleNote {
    uint64_t mass;
    uint32_t a, b, c, d;
};
struct alignas(16) SampleSmem {
    uint32_t lo[kBins], hi[kBins];  // a histogram: counts in lo, or masses as two words
    uint64_t sums[kBins];           // this CTA's chunk of the cluster's histogram
    Pow2Entry pow2[32];
    SampleNote note[2][kMaxCluster];             // a phase's and the next one's
    SampleNote found;                            // the bin found, by its owner
    uint64_t wmass[kSampleWarps];
    uint32_t wcnt[kSampleWarps], wa[kSampleWarps], wb[kSampleWarps], wc[kSampleWarps];
    float c, cl;                                 // log2 e / temperature
    double least;                                // temperature * log min_p
};

// Keys order as the values do; -0 is 0.
__device__ __forceinline__ uint32_t key_of(float v) {
    const uint32_t u = __float_as_uint(v + 0.0f);
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t key) {
    return __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key);
}

// 2^(c (v - top)) in units of 2^-kMassBits, c = log2 e / temperature.
//
// v - top is taken as a sum of two floats, and x = c (v - top) as x + xl. With k =
// rint(32 x) and g = x - k / 32 (exact, at most 1/64), 2^x = 2^(k/32) (1 + z), z =
// e^y - 1 for y = (g + xl) ln 2: the first term h = g ln 2 with its rounding, the
// others by the series up to y^5 / 120 (the next term is below 2^-48). The power
// of the table is held as hi + lo and in fixed point; hi * h keeps its rounding. The
// largest error left is that of the last sums, about 2^-36.
struct Weigher {
    float top, c, cl;
    __device__ uint64_t operator()(float v, const Pow2Entry* table) const {
        const float d = v - top, t = d - v, dl = (v - (d - t)) + (-top - t);
        const float x = d * c;
        if (!(x > -44.f)) return 0;  // below half a unit, or -inf
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
        const Pow2Entry p = table[k & 31];
        const float a = p.hi * h, b = fmaf(p.lo, h, fmaf(p.hi, q, fmaf(p.hi, h, -a)));
        const uint64_t m = p.fixed + (uint64_t)(int64_t)(__float2int_rn(a * 0x1p36f) + __float2int_rn(b * 0x1p36f));
        const int down = 36 - kMassBits - (k >> 5);
        if (down <= 0) return m << -down;
        return down > 62 ? 0 : (m + (1ull << (down - 1))) >> down;
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
    T* values = reinterpret_cast<T*>(raw + sizeof(SampleSmem));
    cg::cluster_group cluster = cg::this_cluster();
    const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int row = (int)(blockIdx.x / (unsigned)C), tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int first = min(rank * a.slice, a.vocab), n = min(a.slice, a.vocab - first);  // of this CTA's slice

    cluster_arrive();
    if (tid < 32) sm.pow2[tid] = kPow2[tid];
    griddep_wait();
    griddep_launch();
    const T* src = (const T*)a.logits + row * a.stride + first;
    const Slice<T> value = {values, src, min(a.held, n)};
    const float temp = a.temperature ? a.temperature[row] : 1.f, top_p = a.top_p ? a.top_p[row] : 1.f;
    const float min_p = a.min_p ? a.min_p[row] : 0.f, u = a.uniform ? a.uniform[row] : 0.f;
    const int top_k = a.top_k ? a.top_k[row] : 0;
    const bool greedy = !a.uniform || temp == 0.f;
    if (tid == 0) {  // fp64 is slow: one thread's work
        const double c = fmin(1.4426950408889634 / (double)temp, 0x1p100);
        sm.c = (float)c;
        sm.cl = (float)(c - (double)sm.c);
        if (min_p > 0.f) sm.least = (double)temp * log((double)min_p);
    }

    // --- the slice into shared memory; its largest key, its smallest of a number, NaN
    uint32_t kmax = 0, kmin = 0xffffffffu, bad = 0;
    auto look = [&](float v) {
        if (v != v) bad = 1;
        const uint32_t k = key_of(v);
        kmax = max(kmax, k);
        if (k > kKeyNegInf) kmin = min(kmin, k);
    };
    auto as_float = [&](T v) {
        if constexpr (sizeof(T) == 4) return v;
        else return __uint_as_float((uint32_t)v << 16);
    };
    {
        constexpr int kPer = 16 / sizeof(T);
        const int whole = ((uintptr_t)src & 15u) == 0 ? n / kPer * kPer : 0;
#pragma unroll 4
        for (int i = tid * kPer; i < whole; i += kSampleThreads * kPer) {
            const uint4 w = *reinterpret_cast<const uint4*>(src + i);
            if (i < value.held) *reinterpret_cast<uint4*>(values + i) = w;  // `held` is a multiple of 8, or all
            const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if constexpr (sizeof(T) == 4) {
                    look(__uint_as_float(x[e]));
                } else {
                    look(__uint_as_float(x[e] << 16));
                    look(__uint_as_float(x[e] & 0xffff0000u));
                }
            }
        }
#pragma unroll 4
        for (int i = whole + tid; i < n; i += kSampleThreads) {
            const T v = src[i];
            if (i < value.held) values[i] = v;
            look(as_float(v));
        }
    }
    int phase = 0;
    // Every CTA's note to every CTA; all of them afterwards in sm.note[...], until the next but one.
    auto tell = [&](const SampleNote& note) -> const SampleNote* {
        phase ^= 1;
        if (tid < C) cluster.map_shared_rank(&sm, tid)->note[phase][rank] = note;
        cluster.sync();
        return sm.note[phase];
    };
    kmax = __reduce_max_sync(0xffffffffu, kmax);
    kmin = __reduce_min_sync(0xffffffffu, kmin);
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

    // The j-th token (from 0) of a key, in the order of the indexes: the CTA that has it writes it.
    auto pick = [&](uint32_t key, uint64_t j, uint64_t mass) {
        const int per = (n + kSampleThreads - 1) / kSampleThreads * 32;  // a warp's stretch of the slice
        const int from = min(warp * per, n), to = min(from + per, n);
        unsigned mine = 0;
        for (int i = from; i < to; i += 32) mine += __popc(__ballot_sync(0xffffffffu, i + lane < to && key_of(value(min(i + lane, n - 1))) == key));
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
            const unsigned hit = __ballot_sync(0xffffffffu, i + lane < to && key_of(value(min(i + lane, n - 1))) == key);
            if (j < at + __popc(hit)) {
                unsigned rest = hit;
                for (uint64_t skip = j - at; skip; --skip) rest &= rest - 1;
                if (lane == 0) {
                    a.tokens[row] = first + i + __ffs(rest) - 1;
                    if (a.logprobs)
                        a.logprobs[row] = greedy ? 0.f
                                                 : (float)(((double)value_of(key) - (double)value_of(kmax)) / (double)temp -
                                                           log((double)mass * (1.0 / (1ull << kMassBits))));
                }
                return;
            }
            at += __popc(hit);
        }
    };
    auto finish = [&]() { cluster.sync(); };  // no CTA leaves while another may write to it

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
    const Weigher weigh = {top, sm.c, sm.cl};
    auto weight_of = [&](uint32_t key) { return weigh(value_of(key), sm.pow2); };

    struct Place {
        uint32_t key;
        uint64_t before, in;  // of the point: what lies before the key, and the rest
    };
    const int chunk = kBins / C;  // bins that a CTA puts together
    // The histogram of the keys klo .. khi, by (khi - key) >> shift, put together: this CTA's chunk in
    // sm.sums.
    auto histogram = [&](uint32_t klo, uint32_t khi, int shift, bool by_count) {
        for (int b = tid; b < kBins; b += kSampleThreads) sm.lo[b] = sm.hi[b] = 0;
        __syncthreads();
        for (int i = tid; i < n; i += kSampleThreads) {
            const float v = value(i);
            const uint32_t key = key_of(v);
            if (key < klo || key > khi) continue;
            const uint32_t bin = (khi - key) >> shift;
            if (by_count) {
                atomicAdd(&sm.lo[bin], 1u);
            } else {
                const uint64_t w = weigh(v, sm.pow2);
                const uint32_t old = atomicAdd(&sm.lo[bin], (uint32_t)w), high = (uint32_t)(w >> 32) + (old + (uint32_t)w < old);
                if (high) atomicAdd(&sm.hi[bin], high);
            }
        }
        cluster.sync();
        for (int b = tid; b < chunk; b += kSampleThreads) {
            uint64_t sum = 0;
            for (int r = 0; r < C; ++r) {
                SampleSmem* s = cluster.map_shared_rank(&sm, r);
                const int at = rank * chunk + b;
                sum += (uint64_t)s->hi[at] << 32 | s->lo[at];
            }
            sm.sums[b] = sum;
        }
        __syncthreads();
    };
    // The bin of the histogram put together that holds the point (below the total): what lies before it, and its number.
    auto bin_of = [&](uint64_t point, uint64_t& before, uint64_t& total) -> int {
        // each thread a stretch of the chunk
        const int per = (chunk + kSampleThreads - 1) / kSampleThreads, b0 = min(tid * per, chunk), b1 = min(b0 + per, chunk);
        uint64_t mine = 0;
        for (int b = b0; b < b1; ++b) mine += sm.sums[b];
        uint64_t upto = mine;
        for (int off = 1; off < 32; off <<= 1) {
            const uint64_t v = __shfl_up_sync(0xffffffffu, upto, off);
            if (lane >= off) upto += v;
        }
        if (lane == 31) sm.wmass[warp] = upto;
        __syncthreads();
        uint64_t here = 0, ahead = 0;
        for (int w = 0; w < kSampleWarps; ++w) {
            if (w == warp) ahead = here;
            here += sm.wmass[w];
        }
        const SampleNote* all = tell({here, 0, 0, 0, 0});
        total = 0;
        uint64_t start = 0;
        for (int r = 0; r < C; ++r) {
            if (r == rank) start = total;
            total += all[r].mass;
        }
        uint64_t at = start + ahead + upto - mine;
        if (point < total && at <= point && point < at + mine) {
            int b = b0;
            while (point >= at + sm.sums[b]) at += sm.sums[b++];
            for (int r = 0; r < C; ++r) cluster.map_shared_rank(&sm, r)->found = {at, (uint32_t)(rank * chunk + b), 0, 0, 0};
        }
        cluster.sync();
        before = sm.found.mass;
        return (int)sm.found.a;
    };
    auto shift_of = [](uint32_t klo, uint32_t khi) {
        int s = 0;
        while (((khi - klo) >> s) >= (uint32_t)kBins) ++s;
        return s;
    };
    // The place of a point (by count or by mass) among the keys klo .. khi; total: of all of them.
    auto locate = [&](uint32_t klo, uint32_t khi, uint64_t point, bool by_count, uint64_t& total) -> Place {
        uint64_t before = 0;
        for (bool outer = true;; outer = false) {
            const int shift = shift_of(klo, khi);
            histogram(klo, khi, shift, by_count);
            uint64_t ahead, sum;
            const int bin = bin_of(point - before, ahead, sum);
            if (outer) {
                total = sum;
                if (point >= sum) return {klo, 0, 0};
            }
            before += ahead;
            khi -= (uint32_t)bin << shift;
            if (shift == 0) return {khi, before, point - before};
            const uint32_t width = (1u << shift) - 1u;
            klo = khi - klo > width ? khi - width : klo;
        }
    };

    // --- top-k: the last key kept, and how many of its tokens
    uint64_t total, j_keep = 0xffffffffull;
    uint32_t k_keep = kmin;
    if (top_k > 0 && top_k < a.vocab) {
        const Place p = locate(kmin, kmax, (uint64_t)(top_k - 1), true, total);
        if ((uint64_t)top_k <= total) k_keep = p.key, j_keep = p.in + 1;
    }
    // mass of the tokens of keys klo .. kmax, and of key klo alone
    auto mass_from = [&](uint32_t klo, uint64_t& of_klo) {
        uint64_t mine = 0, same = 0;
        const uint64_t w_klo = weight_of(klo);
        for (int i = tid; i < n; i += kSampleThreads) {
            const float v = value(i);
            const uint32_t key = key_of(v);
            if (key > klo) mine += weigh(v, sm.pow2);
            else if (key == klo) same += w_klo;
        }
        for (int off = 16; off; off >>= 1) {
            mine += __shfl_xor_sync(0xffffffffu, mine, off);
            same += __shfl_xor_sync(0xffffffffu, same, off);
        }
        __syncthreads();
        if (lane == 0) sm.wmass[warp] = mine, sm.sums[warp] = same;
        __syncthreads();
        mine = same = 0;
        for (int w = 0; w < kSampleWarps; ++w) mine += sm.wmass[w], same += sm.sums[w];
        const SampleNote* all = tell({mine, (uint32_t)same, (uint32_t)(same >> 32), 0, 0});
        mine = same = 0;
        for (int r = 0; r < C; ++r) mine += all[r].mass, same += (uint64_t)all[r].b << 32 | all[r].a;
        of_klo = same;
        return mine;
    };
    // the mass kept so far: that above k_keep, and of k_keep's tokens the first j_keep
    auto kept_mass = [&]() {
        uint64_t same;
        const uint64_t above = mass_from(k_keep, same), w = weight_of(k_keep);
        const uint64_t of_key = j_keep == 0xffffffffull ? same : min(same, w * j_keep);
        return above + of_key;
    };
    uint64_t mass = kept_mass();
    if (top_p < 1.f) {
        // the tokens with less than p of the mass before them, the first one among them
        const uint64_t want = top_p > 0.f ? max(part_of(mass, top_p, true), (uint64_t)1) : 1;
        uint64_t all_mass;
        const Place p = locate(k_keep, kmax, want - 1, false, all_mass);
        k_keep = p.key;
        j_keep = p.in / weight_of(p.key) + 1;
        mass = p.before + j_keep * weight_of(p.key);
    }
    if (min_p > 0.f) {
        const uint32_t k_least = key_of(__double2float_ru((double)top + sm.least));
        if (min_p > 1.f) {  // no weight is above 1: the first token only
            k_keep = kmax;
            j_keep = 1;
            mass = weight_of(kmax);
        } else if (k_least > k_keep) {
            k_keep = k_least;
            j_keep = 0xffffffffull;
            mass = kept_mass();
        }
    }
    // --- the draw
    const uint64_t point = min(part_of(mass, fminf(fmaxf(u, 0.f), 1.f), false), mass - 1);
    uint64_t all_mass;
    const Place p = locate(k_keep, kmax, point, false, all_mass);
    pick(p.key, p.in / weight_of(p.key), mass);
    finish();
}

template <class T>
static cudaError_t launch_sample(SampleArgs a, int dev, cudaStream_t st) {
    // A row's CTAs: enough that its slices fit in shared memory beside one another on an SM, more where
    // there are few rows.
    const int sms = sm_count(dev);
    int C = 1;
    auto slice_of = [&](int c) { return ((a.vocab + c - 1) / c + 7) / 8 * 8; };
    constexpr int kHeldBytes = 64 * 1024;
    while (C < kMaxCluster && ((size_t)slice_of(C) * sizeof(T) > kHeldBytes || ((int64_t)a.rows * C < 2 * sms && slice_of(C) > 2048))) C *= 2;
    a.slice = slice_of(C);
    a.held = (int)std::min<int64_t>(a.slice, kHeldBytes / sizeof(T));
    const size_t bytes = sizeof(SampleSmem) + (size_t)a.held * sizeof(T);
    static DeviceOnce once;
    const cudaError_t set = once.run(dev, [] {
        return cudaFuncSetAttribute(k_sample<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(SampleSmem) + kHeldBytes);
    });
    if (set != cudaSuccess) return set;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.rows * C));
    cfg.blockDim = dim3(kSampleThreads);
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)C;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
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
