// attn_prompt.cu -- causal attention over packed sequences of bf16 keys and
// values on the tcgen05 tensor cores, and its C entry point.
//
// Row i of a sequence's lq queries: out = sum_j softmax_j(scale q . k_j) v_j
// over the keys j <= lk - lq + i; 4 * head_dim operations per visible (query,
// key) pair, bound by the tensor cores except for short prompts.
//
// A tile is 128 rows: the query heads of one key/value head for 128 / group
// consecutive tokens, token-major, so grouped heads share every key tile and
// only 128 / group tokens straddle the diagonal. A CTA takes two neighbouring
// tiles (or two halves of one tile's keys, joined at the end) and runs them
// through the tensor cores in turn, so that the softmax of one overlaps the
// products of the other:
//   warps 0-3, 4-7  softmax of tile 0, 1: a thread per row, scores from tensor
//                   memory, weights back to it as bf16 over the scores, 64 keys
//                   at a time
//   warp 8          items and TMA loads: the two query tiles, then K0 V0 K1 V1 ...
//                   into a ring of 128-key stages (128-byte swizzle)
//   warps 9, 10     issue the MMAs of tile 0, 1: S = Q K^T (both from shared
//                   memory), and O += P V (P from tensor memory, V as the
//                   MN-major operand)
// CTAs are persistent: one that has finished its pair of tiles takes the work
// of a CTA that has not started (cluster launch control), so that the next
// pair's loads and scores run under the last one's outputs.
// Values that some row of a CTA does not see are cleaned in shared memory
// before use: those past the sequence's keys are set to zero, and infinities
// and NaN behind the diagonal are replaced by zero (0 * inf would reach every
// row) and added, times their weights, to the rows that do see them at the end.
// Tensor memory: S0 S1 (128 columns each) and O0 O1 (head_dim each), fp32.
// Weights are bf16 (the tensor cores take one type for both operands, and the
// values are bf16): an error of the size of the output's own rounding. Maxima
// and sums are fp32; a row's maximum is raised, and its output rescaled, only
// when a score exceeds it by 2^8.
//
// Measured: 8192 tokens, 32 query heads over 4, head_dim 128: 351 us a call, where
// the power limit lowers the clock, 333 us in a graph (1560 and 1650 TFLOP/s, 0.80
// and 0.85 of cuBLAS's bf16 rate); 2451 tokens 51 us; 512 tokens over a context of
// 4000 37 us; 20 sequences of up to 1500 tokens at head_dim 64 106 us. A key tile of a pair takes 2058 cycles of the tensor cores
// at head_dim 128 and about 2770 here; at 64 it takes 1538 (N = 64 products run at
// half rate) and 2240.
#include <cuda.h>

#include <cmath>

#include "attn_tc.cuh"
#include "kv.cuh"
#include "moe_cache.h"
#include "piece_ring.h"

namespace moe {

constexpr int kPromptThreads = 384;
constexpr float kRaise = 8.0f;       // log2 of the growth a row's weights may reach before a rescale

struct PromptArgs {
    const uint16_t *q, *k, *v;
    int64_t qs, ks, vs;
    const int *cu_q, *cu_k;
    int Tq, Tk, B, hq, hkv;
    float c;  // scale * log2 e
    uint16_t* out;
    int out32;  // out is 32-byte aligned
};

// One item of work: two neighbouring query tiles of a sequence and head (or a
// single one, with two halves of its keys in the place of the tiles).
struct Item {
    int q0, lq;   // the sequence's first query row, and its queries
    int k0, lk;   // its first key row, and its keys
    int i0, head; // the first token of the pair of tiles; the key/value head
    int end;      // no item: the CTA's work is done
};

constexpr int kTable = 256;  // entries of the table of pairs of tiles before a run of sequences

template <int D>
struct PromptSmem {
    static constexpr int kHalves = D / 64;                 // 64-dim halves of a tile: one swizzled row each
    static constexpr int kTileBytes = kTile * D * 2;
    static constexpr int kStages = D == 128 ? 4 : 6;       // (one more of 32 KB: 1 to 5% slower)
    uint8_t q[2][kTileBytes];
    uint8_t kv[kStages][kTileBytes];
    ulonglong2 answer;  // of the launch-control request
    unsigned long long q_full[2], q_empty[2], full[kStages], empty[kStages];
    unsigned long long s_full[2], p_full[2][2], o_full[2];
    // The values of a stage are cleaned. One barrier a stage, so that a stage's
    // next cleaning comes only after both MMA warps have passed this one (they
    // free the stage) and a wait cannot be a phase behind. Halves of one tile's
    // keys have one a slot, in the first two: there the slot's own MMA warp alone
    // waits, and its next scores come after.
    unsigned long long clean[kStages];
    unsigned long long item_full[2], item_empty[2], asked, half_done, half_read, drained[2];
    float half[kTile][2];  // maximum and sum of a row's second half of keys
    Item item[2];
    int flag[2];        // number of the last item (of each parity) with infinities or NaN among its cleaned values, + 1
    int prefix[kTable], total;
    int wsum[kTable / 32];
    int longest;        // key tiles of the longest item put so far
    int dead;           // a wait has given up
    uint32_t tmem;
};

// Launch control: asks for the next CTA of the grid that has not started, to
// run its work here instead. The answer lands in shared memory.
__device__ __forceinline__ void ask_next_cta(uint32_t answer, uint32_t bar) {
    asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];\n" ::"r"(answer),
                 "r"(bar)
                 : "memory");
}
// The CTA that the answer gives, or -1.
__device__ __forceinline__ int next_cta(uint32_t answer) {
    uint32_t yes, x;
    asm volatile(
        "{\n.reg .pred p;\n.reg .b128 r;\nld.shared.b128 r, [%2];\n"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\nselp.u32 %0, 1, 0, p;\nmov.u32 %1, 0;\n"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, r;\n}\n"
        : "=r"(yes), "=r"(x)
        : "r"(answer)
        : "memory");
    return yes ? (int)x : -1;
}

__device__ __forceinline__ void tma_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];\n" ::"r"(dst),
        "l"(map), "r"(bar), "r"(x), "r"(y), "r"(z)
        : "memory");
}
__device__ __forceinline__ void tma_4d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z, int w) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], [%2];\n" ::"r"(dst),
        "l"(map), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(w)
        : "memory");
}

// bf16 operands, fp32 accumulator; b_mn: B is MN-major.
__host__ __device__ constexpr uint32_t idesc_bf16(int M, int N, bool b_mn) {
    return tc_idesc_f16(M, N) | (1u << 7) | (1u << 10) | ((b_mn ? 1u : 0u) << 16);
}
// A value tile [128 keys][64 dims per half] as the MN-major operand: 64 dims
// are a swizzled row, 8 keys an atom (1024 bytes: the stride along K), and the
// halves are 16 KB apart (the stride along N).
__device__ __forceinline__ uint64_t sdesc_mn(uint32_t saddr) {
    uint64_t d = (uint64_t)((saddr >> 4) & 0x3FFFu);
    d |= (uint64_t)((kTile * 128) >> 4) << 16;
    d |= (uint64_t)(1024 >> 4) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)2 << 61;
    return d;
}

__device__ __forceinline__ uint32_t pack_bf(float lo, float hi) {
    __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&p);
}
__device__ __forceinline__ uint32_t drop_nonfinite(uint32_t w) {
    if ((w & 0x7f80u) == 0x7f80u) w &= 0xffff0000u;
    if ((w & 0x7f800000u) == 0x7f800000u) w &= 0xffffu;
    return w;
}

// The values of a key tile that some row of the CTA does not see (keys from
// `from` on): infinities and NaN to zero, and everything from key `end` on. One
// of 128 threads' share; true if it found some. Rows 8 apart have the same
// swizzle, so a thread keeps its 16-byte column and steps through the rows.
template <int D>
__device__ __forceinline__ bool clean_values(uint8_t* tile, int t, int from, int end) {
    constexpr int kChunks = D / 8, kRowsAtOnce = 128 / kChunks;  // chunks of a key's values; keys of a pass
    end = min(max(end, 0), kTile);
    const int cc = t % kChunks;
    int r = max(from, 0) + t / kChunks;
    uint4* at = reinterpret_cast<uint4*>(tile + (cc >> 3) * (kTile * 128) + r * 128 + (((cc ^ r) & 7) << 4));
    bool found = false, wrote = false;
#pragma unroll 4
    for (; r < end; r += kRowsAtOnce, at += kRowsAtOnce * 8) {
        const uint4 u = *at;
        const uint32_t top = __vmaxu2(__vmaxu2(u.x & 0x7f807f80u, u.y & 0x7f807f80u), __vmaxu2(u.z & 0x7f807f80u, u.w & 0x7f807f80u));
        if ((top & 0xffffu) == 0x7f80u || (top >> 16) == 0x7f80u) {  // an exponent of all ones
            found = wrote = true;
            *at = make_uint4(drop_nonfinite(u.x), drop_nonfinite(u.y), drop_nonfinite(u.z), drop_nonfinite(u.w));
        }
    }
    for (; r < kTile; r += kRowsAtOnce, at += kRowsAtOnce * 8) {
        wrote = true;
        *at = make_uint4(0, 0, 0, 0);
    }
    if (wrote) fence_async_smem();
    return found;
}

// Adds the infinities and NaN among the values of keys first .. end - 1, which
// the cleaning took out, to a row that sees them (queries q, mc its maximum),
// each times its weight as the tensor cores would have: infinity, or NaN where
// the weight is 0 in fp32. Out of line: it hardly runs.
template <int D>
__device__ __noinline__ void add_nonfinite(const PromptArgs& a, uint16_t* row, const uint16_t* q, float mc, int k0, int head, int first,
                                           int end) {
    auto value = [](const uint16_t* p) { return __uint_as_float((uint32_t)*p << 16); };
    for (int t = first; t < end; ++t) {
        const uint16_t* v = a.v + (size_t)(k0 + t) * a.vs + (size_t)head * D;
        const uint16_t* k = a.k + (size_t)(k0 + t) * a.ks + (size_t)head * D;
        float weight = -1.f;  // not known yet
        for (int d = 0; d < D; ++d) {
            const float x = value(v + d);
            if (!(fabsf(x) <= 3.4028235e38f)) {
                if (weight < 0.f) {
                    float s = 0.f;
                    for (int e = 0; e < D; ++e) s = fmaf(value(q + e), value(k + e), s);
                    weight = ex2f(fmaf(s, a.c, -mc));
                }
                const __nv_bfloat16 y = __float2bfloat16_rn(__uint_as_float((uint32_t)row[d] << 16) + x * weight);
                row[d] = *reinterpret_cast<const uint16_t*>(&y);
            }
        }
    }
}

// The outputs of rows `row` .. `end` - 1 and a key/value head that no warp works on,
// since a wait gave up: NaN. A warp; out of line: it hardly runs.
template <int D>
__device__ __noinline__ void lose_rows(uint16_t* out, int hq, int group, int head, int row, int end, int lane) {
    const uint4 nan = make_uint4(0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u);
    for (; row < end; ++row) {
        uint4* at = reinterpret_cast<uint4*>(out + ((size_t)row * hq + (size_t)head * group) * D);
        for (int e = lane; e < group * D / 8; e += 32) at[e] = nan;
    }
}

// kSingle: items are one tile, its keys in two halves, in place of two tiles.
template <int D, bool kSingle>
__global__ void __launch_bounds__(kPromptThreads, 1) k_prompt(const __grid_constant__ PromptArgs a,
                                                              const __grid_constant__ CUtensorMap mq,
                                                              const __grid_constant__ CUtensorMap mk,
                                                              const __grid_constant__ CUtensorMap mv) {
    using S = PromptSmem<D>;
    constexpr int kStages = S::kStages, kHalves = S::kHalves, kHalf = kTile * 128;
    extern __shared__ uint8_t raw[];
    S& sm = *reinterpret_cast<S*>(raw + (((gsmem(raw) + 1023u) & ~1023u) - gsmem(raw)));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int group = a.hq / a.hkv, tokens = kTile / group;  // tokens of a tile

    const int reach = kSingle ? tokens : 2 * tokens;  // tokens of an item
    // --- the table: items before sequence t * run
    const int run = (a.B + kTable - 1) / kTable;
    auto pairs_of = [&](int s) {
        const int n = min(max(a.cu_q[s + 1], 0), a.Tq) - min(max(a.cu_q[s], 0), a.Tq);
        return n > 0 ? (n + reach - 1) / reach : 0;
    };
    int incl = 0, mine = 0;
    if (warp < kTable / 32) {
        griddep_wait();
        for (int s = tid * run; s < min((tid + 1) * run, a.B); ++s) mine += pairs_of(s);
        incl = mine;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl, off);
            if (lane >= off) incl += v;
        }
        if (lane == 31) sm.wsum[warp] = incl;
    } else if (warp == 8) {
        tc_alloc(gsmem(&sm.tmem), 512);
        tc_relinquish();
        griddep_wait();
    } else if (warp == 9) {
        if (lane == 0) {
            for (int x = 0; x < 2; ++x) {
                bar_init_n(gsmem(&sm.q_full[x]), 1);
                bar_init_n(gsmem(&sm.q_empty[x]), 1);
                bar_init_n(gsmem(&sm.s_full[x]), 1);
                bar_init_n(gsmem(&sm.p_full[x][0]), 128);
                bar_init_n(gsmem(&sm.p_full[x][1]), 128);
                bar_init_n(gsmem(&sm.o_full[x]), 1);
                bar_init_n(gsmem(&sm.item_full[x]), 1);
                bar_init_n(gsmem(&sm.item_empty[x]), 10);  // the softmax and MMA warps
                sm.flag[x] = 0;
            }
            for (int st = 0; st < kStages; ++st) {
                bar_init_n(gsmem(&sm.full[st]), 1);
                bar_init_n(gsmem(&sm.empty[st]), 2);  // both MMA warps
                bar_init_n(gsmem(&sm.clean[st]), 128);
            }
            bar_init_n(gsmem(&sm.half_done), 128);
            bar_init_n(gsmem(&sm.half_read), 128);
            bar_init_n(gsmem(&sm.asked), 1);
            bar_init_n(gsmem(&sm.drained[0]), 1);
            bar_init_n(gsmem(&sm.drained[1]), 1);
            sm.longest = 0;
            sm.dead = 0;
            asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
        }
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp < kTable / 32) {
        int before = 0, sum = 0;
#pragma unroll
        for (int w = 0; w < kTable / 32; ++w) {
            if (w == warp) before = sum;
            sum += sm.wsum[w];
        }
        sm.prefix[tid] = before + incl - mine;
        if (tid == 0) sm.total = sum;
    }
    __syncthreads();
    const uint32_t tmem = sm.tmem;
    int* dead = &sm.dead;

    // What a pair of tiles asks for: token i of the sequence sees the keys below shift + i + 1.
    struct Span {
        int shift, n0, n1, n;  // key tiles of slot 0, of slot 1, and in the ring
        int seen_by_all;       // keys below this are seen by every row
        int first_masked;      // the first key tile with a value to be cleaned
    };
    auto span_of = [&](const Item& it) {
        Span p;
        p.shift = it.lk - it.lq;
        auto tiles_of = [&](int first) {
            const int last = min(first + tokens, it.lq) - 1;
            const int lim = last < first ? 0 : max(min(p.shift + last + 1, it.lk), 0);
            return (lim + kTile - 1) / kTile;
        };
        p.n0 = tiles_of(it.i0);
        if (kSingle) {  // slot 0 has the first half, slot 1 the rest
            p.n = p.n0;
            p.n1 = p.n / 2;
            p.n0 = p.n - p.n1;
        } else {
            p.n1 = tiles_of(it.i0 + tokens);
            p.n = max(p.n0, p.n1);
        }
        p.seen_by_all = max(min(p.shift + it.i0 + 1, it.lk), 0);
        p.first_masked = p.seen_by_all / kTile;
        return p;
    };
    // What the longest item may take, beyond a wait's 0.2 s: 20 us for each key tile.
    auto at_work = [&]() { return 20000ull * (unsigned)*(volatile int*)&sm.longest; };
    // The next item, for a warp that uses them; false at the end. `number` counts the
    // items taken. The limit is above all that warp 8 may wait for between two items
    // (three waits, two of them of twice the time, and the loads of an item), so that
    // an item that was put is taken, and what is not put is lost to warp 8 alone.
    auto take = [&](int number) {
        return take_piece(
            number,
            [&](int place, uint32_t parity) {
                return warp_wait(gsmem(&sm.item_full[place]), parity, dead, [&] { return 8 * kGWaitNs + 2 * at_work(); });
            },
            [&](int place) { return sm.item[place].end != 0; });
    };
    auto give_back = [&](int number) {
        __syncwarp();
        if (lane == 0) bar_arrive(gsmem(&sm.item_empty[number & 1]));
    };

    // Registers: the launch gives 168 a thread (64512 in all); the softmax
    // warpgroups hold a row of scores each and take 216, the third 72.
    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;\n");
        if (warp == 8) {
            // --- items and loads. The CTA starts with its own and asks for
            // others until none is left. Items are numbered from the last pair
            // of tiles, so that a sequence's longest run first.
            int which = blockIdx.x, number = 0, st = 0;
            uint32_t turn = 1, asks = 0;   // the ring's parity of `empty`; parity of `asked`
            uint32_t q_turn[2] = {1, 1};
            bool open = true;  // false once the wait for a place has given up: no more items
            auto put = [&](const Item& it) {
                open = open && put_piece(
                                   number,
                                   [&](int place, uint32_t parity) {
                                       return warp_wait(gsmem(&sm.item_empty[place]), parity, dead, [&] { return kGWaitNs + at_work(); });
                                   },
                                   [&](int place) {
                                       if (lane == 0) {
                                           sm.item[place] = it;
                                           bar_arrive(gsmem(&sm.item_full[place]));
                                       }
                                       __syncwarp();
                                   });
                ++number;
                return open;
            };
            while (which >= 0) {
                const bool ask = !warp_dead(dead);
                if (ask && lane == 0) {
                    bar_expect(gsmem(&sm.asked), 16);
                    ask_next_cta(gsmem(&sm.answer), gsmem(&sm.asked));
                }
                const int head = which % a.hkv, at = sm.total - 1 - which / a.hkv;
                if (at >= 0) {
                    // the last entry of the table that is not above `at`, then the sequence among its run
                    int below = 0;
#pragma unroll
                    for (int e = 0; e < kTable / 32; ++e) below += sm.prefix[32 * e + lane] <= at;
                    below = __reduce_add_sync(0xffffffffu, below) - 1;
                    int seq = below * run, base = sm.prefix[below];
                    if (run > 1) {
                        for (;; seq += 32) {
                            const int s = seq + lane, w = s < a.B ? pairs_of(s) : 0;
                            int upto = w;
#pragma unroll
                            for (int off = 1; off < 32; off <<= 1) {
                                const int v = __shfl_up_sync(0xffffffffu, upto, off);
                                if (lane >= off) upto += v;
                            }
                            const unsigned hit = __ballot_sync(0xffffffffu, base + upto > at);
                            if (hit) {
                                const int l = __ffs(hit) - 1;
                                seq += l;
                                base += __shfl_sync(0xffffffffu, upto - w, l);
                                break;
                            }
                            base += __shfl_sync(0xffffffffu, upto, 31);
                            if (seq + 32 >= a.B) break;  // not reached: the table has the pair
                        }
                        seq = min(seq, a.B - 1);
                    }
                    const int bound = lane < 2 ? min(max(a.cu_q[seq + lane], 0), a.Tq)
                                      : lane < 4 ? min(max(a.cu_k[seq + lane - 2], 0), a.Tk) : 0;
                    Item it;
                    it.q0 = __shfl_sync(0xffffffffu, bound, 0);
                    it.lq = __shfl_sync(0xffffffffu, bound, 1) - it.q0;
                    it.k0 = __shfl_sync(0xffffffffu, bound, 2);
                    it.lk = max(__shfl_sync(0xffffffffu, bound, 3) - it.k0, 0);
                    it.i0 = (at - base) * reach;
                    it.head = head;
                    it.end = 0;
                    if (put(it)) {
                        const Span p = span_of(it);
                        if (lane == 0) *(volatile int*)&sm.longest = max(sm.longest, p.n);
                        for (int x = 0; x < 2; ++x) {
                            if ((x ? p.n1 : p.n0) == 0) continue;
                            const uint32_t bar = gsmem(&sm.q_full[x]);
                            bar_wait(gsmem(&sm.q_empty[x]), q_turn[x], dead);
                            if (warp_dead(dead)) break;
                            q_turn[x] ^= 1;
                            if (lane == 0) {
                                bar_expect(bar, (uint32_t)(kHalves * 128 * group * tokens));
                                for (int h = 0; h < kHalves; ++h)
                                    tma_4d(gsmem(sm.q[x]) + h * kHalf, &mq, bar, 64 * h, 0, it.head, it.q0 + it.i0 + (kSingle ? 0 : x * tokens));
                            }
                        }
                        for (int e = 0; e < 2 * p.n; ++e) {  // K0 V0 K1 V1 ...; the two halves' in turn
                            const int tile = !kSingle ? e >> 1 : (e & 2) ? p.n0 + (e >> 2) : e >> 2;
                            const uint32_t bar = gsmem(&sm.full[st]);
                            bar_wait(gsmem(&sm.empty[st]), turn, dead);
                            if (warp_dead(dead)) break;
                            if (lane == 0) {
                                bar_expect(bar, S::kTileBytes);
                                for (int h = 0; h < kHalves; ++h)
                                    tma_3d(gsmem(sm.kv[st]) + h * kHalf, (e & 1) ? &mv : &mk, bar, 64 * h, it.head, it.k0 + tile * kTile);
                            }
                            if (++st == kStages) st = 0, turn ^= 1;
                        }
                    } else {
                        lose_rows<D>(a.out, a.hq, group, it.head, it.q0 + it.i0, it.q0 + min(it.i0 + reach, it.lq), lane);
                    }
                    __syncwarp();
                }
                which = -1;
                if (ask) {
                    const bool answered = warp_wait(gsmem(&sm.asked), asks, dead, [] { return 2 * kGWaitNs; });
                    asks ^= 1;
                    if (answered) which = next_cta(gsmem(&sm.answer));
                    fence_async_smem();  // the answer is read before the next one is asked for
                    __syncwarp();
                }
            }
            Item none = {};
            none.end = 1;
            put(none);
            // copies under way land before the CTA leaves, whatever else gave up
            for (int e = 0; e < kStages; ++e) bar_wait(gsmem(&sm.full[e]), e < st ? turn ^ 1 : turn, dead, true);
            for (int x = 0; x < 2; ++x) bar_wait(gsmem(&sm.q_full[x]), q_turn[x], dead, true);
        } else if (warp < 11) {
            // --- the MMAs of tile x. A warp each, so that the tensor cores have
            // the other tile's products while this one waits for its weights. The
            // whole warp walks the loop and one lane issues, so that the operands
            // stay in uniform registers; descriptors are one base each plus
            // constants. Both warps pass every stage of the ring and every
            // cleaning, needed or not: a wait cannot tell a phase from the next
            // but one, and so no barrier may complete twice before both have passed.
            constexpr uint32_t id_s = idesc_bf16(kTile, kTile, false), id_o = idesc_bf16(kTile, D, true);
            const int x = __shfl_sync(0xffffffffu, warp - 9, 0);
            const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
            const uint32_t ts = tm + x * kTile, to = tm + 2 * kTile + x * D;
            const bool leader = elect_one();
            const uint64_t qd = tc_sdesc(gsmem(sm.q[0]) + x * S::kTileBytes), kd = tc_sdesc(gsmem(sm.kv[0])),
                           vd = sdesc_mn(gsmem(sm.kv[0]));
            constexpr uint64_t kTileStep = S::kTileBytes >> 4;  // to the next stage, in a descriptor
            auto scores = [&](int st, bool last) {
                const uint64_t kx = kd + st * kTileStep;
#pragma unroll
                for (int d = 0; d < D / 16; ++d) {
                    const uint32_t off = ((d / 4) * kHalf + (d % 4) * 32) >> 4;
                    tc_mma(ts, qd + off, kx + off, id_s, d != 0);
                }
                tc_commit(gsmem(&sm.s_full[x]));
                if (last) tc_commit(gsmem(&sm.q_empty[x]));
            };
            auto values = [&](int half, int st, bool first) {  // of the tile's keys 64 half ..
                const uint64_t vx = vd + st * kTileStep;
#pragma unroll
                for (int t = half * kTile / 32; t < (half + 1) * kTile / 32; ++t)
                    tc_mma_ta(to, ts + 8 * t, vx + t * (2048 >> 4), id_o, t == 0 ? !first : 1);
            };
            auto free_stage = [&](int st, bool used) {
                if (used) tc_commit(gsmem(&sm.empty[st]));
                else bar_arrive(gsmem(&sm.empty[st]));
            };
            int st = 0;
            uint32_t round = 0, p_turn = 0, q_turn = 0, c_turn = 0;  // c_turn: a bit a stage (halves: a bit)
            auto step = [&]() { if (++st == kStages) st = 0, round ^= 1; };
            for (int number = 0; take(number); ++number) {
                const Span p = span_of(sm.item[number & 1]);
                give_back(number);
                if (p.n == 0) continue;
                const int nx = x ? p.n1 : p.n0;
                int sk, sv;
                if (kSingle) {
                    auto pass = [&]() {  // a key and a value tile of the other half
                        for (int e = 0; e < 2; ++e) {
                            bar_wait(gsmem(&sm.full[st]), round, dead);
                            if (leader) bar_arrive(gsmem(&sm.empty[st]));
                            step();
                        }
                    };
                    if (x) pass();
                    for (int j = 0; j <= nx && nx; ++j) {  // the scores of tile j, after the values of tile j - 1
                        if (j) {
                            sv = st;
                            bar_wait(gsmem(&sm.full[sv]), round, dead);
                            step();
                            if (warp_dead(dead)) break;
                            if ((x ? p.n0 : 0) + j - 1 >= p.first_masked) {
                                bar_wait(gsmem(&sm.clean[x]), c_turn, dead);
                                c_turn ^= 1;
                            }
                            for (int half = 0; half < 2; ++half) {
                                bar_wait(gsmem(&sm.p_full[x][half]), p_turn, dead);
                                __syncwarp();
                                tc_fence_after();
                                if (leader) values(half, sv, j == 1);
                                __syncwarp();
                            }
                            p_turn ^= 1;
                            if (leader) {
                                if (j == nx) tc_commit(gsmem(&sm.o_full[x]));
                                free_stage(sv, true);
                            }
                            __syncwarp();
                            if (2 * j + x - 1 < p.n) pass();
                            if (j == nx) break;
                        }
                        sk = st;
                        bar_wait(gsmem(&sm.full[sk]), round, dead);
                        step();
                        if (j == 0) {
                            bar_wait(gsmem(&sm.q_full[x]), q_turn, dead);
                            q_turn ^= 1;
                        }
                        __syncwarp();
                        tc_fence_after();
                        if (leader) {
                            scores(sk, j + 1 == nx);
                            free_stage(sk, true);
                        }
                        __syncwarp();
                    }
                    if (warp_dead(dead)) break;
                    continue;
                }
                sk = st;
                bar_wait(gsmem(&sm.full[sk]), round, dead);
                step();
                if (nx) {
                    bar_wait(gsmem(&sm.q_full[x]), q_turn, dead);
                    q_turn ^= 1;
                }
                __syncwarp();
                tc_fence_after();
                if (leader) {
                    if (nx) scores(sk, nx == 1);
                    free_stage(sk, nx);
                }
                __syncwarp();
                // The next keys are waited for after the values' products at head_dim
                // 128, whose ring of four stages may not have them any earlier (8192
                // tokens 333 us, before them 349); at 64 before them, so that the next
                // scores follow the values with no other product between (20 sequences
                // of up to 1500 tokens 105 us, after them 110).
                constexpr bool kLate = D == 128;
                for (int j = 0; j < p.n; ++j) {
                    auto next_keys = [&]() {
                        sk = st;
                        if (j + 1 == p.n) return;
                        bar_wait(gsmem(&sm.full[sk]), round, dead);
                        step();
                    };
                    sv = st;
                    bar_wait(gsmem(&sm.full[sv]), round, dead);
                    step();
                    if (!kLate) next_keys();
                    if (warp_dead(dead)) break;
                    if (j >= p.first_masked) {
                        bar_wait(gsmem(&sm.clean[sv]), (c_turn >> sv) & 1, dead);
                        c_turn ^= 1u << sv;
                    }
                    if (j < nx) {
                        bar_wait(gsmem(&sm.p_full[x][0]), p_turn, dead);
                        __syncwarp();
                        tc_fence_after();
                        if (leader) values(0, sv, j == 0);
                        __syncwarp();
                        bar_wait(gsmem(&sm.p_full[x][1]), p_turn, dead);
                        p_turn ^= 1;
                        __syncwarp();
                        tc_fence_after();
                        if (leader) {
                            values(1, sv, false);
                            if (j + 1 == nx) tc_commit(gsmem(&sm.o_full[x]));
                            else if (!kLate) scores(sk, j + 2 == nx);
                        }
                    }
                    if (leader) free_stage(sv, j < nx);
                    if (kLate) {
                        __syncwarp();
                        next_keys();
                        __syncwarp();
                        tc_fence_after();
                        if (leader && j + 1 < nx) scores(sk, j + 2 == nx);
                    }
                    if (leader && j + 1 < p.n) free_stage(sk, j < nx);
                    __syncwarp();
                }
                if (warp_dead(dead)) break;
            }
            // the last arrivals, so that none is under way when the CTA ends: a stage's `empty`
            // completes once for each time it was filled. Where one does not come, the products.
            bool over = true;
            for (int e = 0; e < kStages; ++e) over &= bar_wait(gsmem(&sm.empty[e]), e < st ? round : round ^ 1, dead);
            if (!__all_sync(0xffffffffu, over)) {
                if (leader) tc_commit(gsmem(&sm.drained[x]));
                __syncwarp();
                bar_wait(gsmem(&sm.drained[x]), 0, dead, true);
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 216;\n");
        // --- softmax of tile x, a thread per row
        const int x = warp >> 2, row = tid & 127, tok = row / group;
        const int shifted = kSingle ? 0 : x * tokens;  // of the tile's first token, from the item's
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        const uint32_t ts = tmem + lanes + x * kTile, to = tmem + lanes + 2 * kTile + x * D;
        uint32_t s_turn = 0, o_turn = 0, half_turn = 0;
        int ring = 0;  // stages of the ring used before this item
        for (int number = 0; take(number); ++number) {
            // the item stays in shared memory until the warp gives it back; only
            // what the loop needs is kept in registers
            const Item& it = sm.item[number & 1];
            int nx, lim, lim_tile;  // key tiles; keys this row sees, and the first row of the tile
            int cleans;             // the first key tile whose values this warpgroup cleans
            int t0;                 // its first key tile
            {
                const Span p = span_of(it);
                const int i = it.i0 + shifted + tok;
                nx = x ? p.n1 : p.n0;
                cleans = x && !kSingle ? max(p.first_masked, p.n0) : p.first_masked;
                t0 = x && kSingle ? p.n0 : 0;
                lim = tok < tokens && i < it.lq ? max(min(p.shift + i + 1, it.lk), 0) : 0;
                lim_tile = max(min(p.shift + it.i0 + shifted + 1, it.lk), 0);
            }
            float m = -INFINITY, l = 0.f;
            for (int j = 0; j < nx; ++j) {
                bar_wait(gsmem(&sm.s_full[x]), s_turn, dead);
                s_turn ^= 1;
                const int kt = t0 + j;  // the key tile
                if (kt >= cleans) {
                    // The stage's previous round is over, since these scores came after it.
                    const int e = ring + 1 + (kSingle ? 4 * j + 2 * x : 2 * j), st = e % kStages;
                    bar_wait(gsmem(&sm.full[st]), (e / kStages) & 1, dead);
                    if (clean_values<D>(sm.kv[st], row, span_of(it).seen_by_all - kt * kTile, it.lk - kt * kTile))
                        *(volatile int*)&sm.flag[number & 1] = number + 1;
                    bar_arrive(gsmem(&sm.clean[kSingle ? x : st]));
                }
                __syncwarp();
                tc_fence_after();
                if ((kt + 1) * kTile > lim_tile) hide_scores(ts, lim - kt * kTile);
                uint32_t s[4][32];
                float mx4[4] = {m, m, m, m};
                // half of the row at a time: one half's maximum is found while the other is loaded
#pragma unroll
                for (int h = 0; h < 2; ++h) tc_ld32(ts + 32 * h, s[h]);
#pragma unroll
                for (int b = 0; b < 4; b += 2) {
#pragma unroll
                    for (int h = b; h < b + 2; ++h) tc_ld_wait32(s[h]);
                    if (b == 0) {
#pragma unroll
                        for (int h = 2; h < 4; ++h) tc_ld32(ts + 32 * h, s[h]);
                    }
#pragma unroll
                    for (int h = b; h < b + 2; ++h)
#pragma unroll
                        for (int e = 0; e < 32; e += 2)
                            mx4[(e >> 1) & 3] = max3(mx4[(e >> 1) & 3], __uint_as_float(s[h][e]), __uint_as_float(s[h][e + 1]));
                }
                const float mx = fmaxf(max3(mx4[0], mx4[1], mx4[2]), mx4[3]);
                const bool raise = (mx - m) * a.c > kRaise;
                if (__any_sync(0xffffffffu, raise)) {
                    // S of this step was computed after the last step's O, so O is at rest
                    const float f = raise ? ex2f((m - mx) * a.c) : 1.f;
                    if (raise) m = mx;
                    l *= f;
                    if (j > 0) {
#pragma unroll 1
                        for (int h = 0; h < D / 8; ++h) {  // few registers beside the row's
                            uint32_t o[8];
                            tc_ld8_wait(to + 8 * h, o);
#pragma unroll
                            for (int e = 0; e < 8; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                            tc_st8(to + 8 * h, o);
                        }
                    }
                }
                const float mc = m == -INFINITY ? 0.f : m * a.c;
                const unsigned long long c2 = pair2(a.c, a.c), mc2 = pair2(-mc, -mc);
                unsigned long long sum[4] = {0, 0, 0, 0};
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    uint32_t w[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const unsigned long long y =
                            fma2(pair2(__uint_as_float(s[h][2 * e]), __uint_as_float(s[h][2 * e + 1])), c2, mc2);
                        const float e0 = ex2f(lo2(y)), e1 = ex2f(hi2(y));
                        sum[e & 3] = add2(sum[e & 3], pair2(e0, e1));
                        w[e] = pack_bf(e0, e1);
                    }
                    tc_st16(ts + 16 * h, w);
                    if (h & 1) {  // the products with the first 64 keys begin while the other weights are computed
                        tc_st_wait();
                        tc_fence_before();
                        bar_arrive(gsmem(&sm.p_full[x][h >> 1]));
                    }
                }
                sum[0] = add2(add2(sum[0], sum[1]), add2(sum[2], sum[3]));
                l += lo2(sum[0]) + hi2(sum[0]);
            }
            float scale0 = 1.f;
            // --- out. (The next item's first O comes after its first weights, so O stays until this is done.)
            if (nx) {
                bar_wait(gsmem(&sm.o_full[x]), o_turn, dead);
                o_turn ^= 1;
            }
            __syncwarp();
            tc_fence_after();
            // two halves of the keys: slot 1 leaves its maxima and sums, and slot 0
            // writes out both
            const bool halves = kSingle && (x ? nx > 0 : span_of(it).n1 > 0);
            float scale1 = 0.f;
            if (halves) {
                if (x) {
                    sm.half[row][0] = m;
                    sm.half[row][1] = l;
                    tc_fence_before();
                    bar_arrive(gsmem(&sm.half_done));
                    bar_wait(gsmem(&sm.half_read), half_turn, dead);  // before O is written again
                } else {
                    bar_wait(gsmem(&sm.half_done), half_turn, dead);
                    __syncwarp();
                    tc_fence_after();
                    const float m1 = sm.half[row][0], high = fmaxf(m, m1);
                    const float f = m == -INFINITY ? 0.f : ex2f((m - high) * a.c);
                    scale1 = m1 == -INFINITY ? 0.f : ex2f((m1 - high) * a.c);
                    l = l * f + sm.half[row][1] * scale1;
                    scale0 = f;
                    m = high;
                }
                half_turn ^= 1;
            }
            const bool flag = nx && *(volatile int*)&sm.flag[number & 1] == number + 1;
            const bool lost = *(volatile int*)dead;
            const float inv = lost ? __int_as_float(0x7fc00000) : l == 0.f ? 0.f : 1.0f / l;
            const bool seen = lim > 0 || lost;
            const int i = it.i0 + shifted + tok;
            const bool used = tok < tokens && i < it.lq && !(x && kSingle);
            uint16_t* dst = a.out + ((size_t)(it.q0 + i) * a.hq + it.head * group + (row - tok * group)) * D;
#pragma unroll 1
            for (int h = 0; h < (x && kSingle ? 0 : D / 32); ++h) {
                uint32_t o[32];
                __syncwarp();
                if (nx) {
                    tc_ld32(to + 32 * h, o);
                    tc_ld_wait32(o);
                    if (halves && !x) {
                        uint32_t o1[32];
                        tc_ld32(to + D + 32 * h, o1);
                        tc_ld_wait32(o1);
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            o[e] = __float_as_uint(__uint_as_float(o[e]) * scale0 + __uint_as_float(o1[e]) * scale1);
                    }
                }
                if (used) {
#pragma unroll
                    for (int e = 0; e < 32; e += 16) {
                        uint32_t w[8];
#pragma unroll
                        for (int q = 0; q < 8; ++q)
                            w[q] = seen ? pack_bf(__uint_as_float(o[e + 2 * q]) * inv, __uint_as_float(o[e + 2 * q + 1]) * inv) : 0u;
                        uint16_t* at = dst + 32 * h + e;
                        // a lane's row is a line of its own: whole sectors halve the stores' trips
                        if (a.out32) {
                            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};\n" ::"l"(at), "r"(w[0]), "r"(w[1]),
                                         "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                                         : "memory");
                        } else {
                            *reinterpret_cast<uint4*>(at) = make_uint4(w[0], w[1], w[2], w[3]);
                            *reinterpret_cast<uint4*>(at + 8) = make_uint4(w[4], w[5], w[6], w[7]);
                        }
                    }
                }
            }
            if (flag && used) {
                const Span p = span_of(it);
                add_nonfinite<D>(a, dst, a.q + (size_t)(it.q0 + i) * a.qs + (size_t)(it.head * group + (row - tok * group)) * D,
                                 m == -INFINITY ? 0.f : m * a.c, it.k0, it.head, max(p.first_masked * kTile, p.seen_by_all), lim);
            }
            tc_fence_before();  // the reads of O, before the weights that let it be overwritten
            if (halves && !x) bar_arrive(gsmem(&sm.half_read));
            ring = (ring + 2 * span_of(it).n) % (2 * kStages);
            give_back(number);  // only now: the flag of the next item but one shares this one's place
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 8) {
        tc_fence_after();
        tc_dealloc(tmem, 512);
    }
}

typedef CUresult (*EncodeTiled)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
static EncodeTiled encode_tiled() {
    static EncodeTiled fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &r) != cudaSuccess ||
            r != cudaDriverEntryPointSuccess)
            p = nullptr;
        return (EncodeTiled)p;
    }();
    return fn;
}
static bool encode(CUtensorMap* m, const void* p, int rank, const cuuint64_t* dims, const cuuint64_t* strides, const cuuint32_t* box) {
    const cuuint32_t ones[4] = {1, 1, 1, 1};
    EncodeTiled fn = encode_tiled();
    return fn && fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(p), dims, strides, box, ones,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool kSingle>
static cudaError_t launch_prompt(const PromptArgs& a, const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv,
                                 int dev, int64_t grid, cudaStream_t st) {
    constexpr int bytes = (int)sizeof(PromptSmem<D>) + 1024;
    static DeviceOnce once;
    const cudaError_t set = once.run(dev, [] {
        return cudaFuncSetAttribute(k_prompt<D, kSingle>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    });
    if (set != cudaSuccess) return set;
    return launch_ex(k_prompt<D, kSingle>, dim3((unsigned)grid), dim3(kPromptThreads), bytes, st, true, a, mq, mk, mv);
}

}  // namespace moe

namespace {
moe_status_t refuse(const char* msg) {
    moe::set_last_error(msg);
    return MOE_ERR_INVALID;
}
}  // namespace

extern "C" moe_status_t moe_attn_prompt(const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                                        const void* v, int64_t v_stride, int32_t Tq, int32_t Tk, int32_t num_seqs,
                                        const int32_t* cu_q, const int32_t* cu_k, int32_t q_heads, int32_t kv_heads,
                                        int32_t head_dim, float scale, void* out, void* stream) {
    if (Tq < 0 || Tk < 0) return refuse("Tq and Tk must be >= 0");
    if (num_seqs < 1 || !cu_q || !cu_k) return refuse("num_seqs must be >= 1 and cu_q, cu_k not NULL");
    if (head_dim != 64 && head_dim != 128) return refuse("head_dim must be 64 or 128");
    if (kv_heads < 1 || kv_heads > 1024 || q_heads < 1 || q_heads % kv_heads || q_heads / kv_heads > 128)
        return refuse("kv_heads must be in 1..1024 and q_heads a multiple of it, at most 128 times");
    if (Tq == 0) return MOE_OK;
    if (!q || !out || (Tk > 0 && (!k || !v))) return refuse("NULL q, k, v or out");
    auto rows_ok = [&](const void* p, int64_t stride, int heads) {
        return ((uintptr_t)p & 15u) == 0 && stride % 8 == 0 && stride >= (int64_t)heads * head_dim;
    };
    if (!rows_ok(q, q_stride, q_heads) || (Tk > 0 && (!rows_ok(k, k_stride, kv_heads) || !rows_ok(v, v_stride, kv_heads))) ||
        ((uintptr_t)out & 15u))
        return refuse("q, k, v and out need 16-byte aligned rows: strides multiples of 8 and not below heads * head_dim");
    if (!(scale >= 0.f) || !std::isfinite(scale)) return refuse("scale must be finite and not negative");
    const int group = q_heads / kv_heads, tokens = moe::kTile / group;
    const cuuint64_t D = head_dim;
    CUtensorMap mq, mk, mv;
    const cuuint64_t qd[4] = {D, (cuuint64_t)group, (cuuint64_t)kv_heads, (cuuint64_t)Tq};
    const cuuint64_t qst[3] = {2 * D, 2 * D * group, 2 * (cuuint64_t)q_stride};
    const cuuint32_t qb[4] = {64, (cuuint32_t)group, 1, (cuuint32_t)tokens};
    bool ok = moe::encode(&mq, q, 4, qd, qst, qb);
    mk = mv = mq;
    if (Tk > 0) {
        const cuuint64_t kd[3] = {D, (cuuint64_t)kv_heads, (cuuint64_t)Tk};
        const cuuint64_t kst[2] = {2 * D, 2 * (cuuint64_t)k_stride}, vst[2] = {2 * D, 2 * (cuuint64_t)v_stride};
        const cuuint32_t kb[3] = {64, 1, (cuuint32_t)moe::kTile};
        ok = ok && moe::encode(&mk, k, 3, kd, kst, kb) && moe::encode(&mv, v, 3, kd, vst, kb);
    }
    if (!ok) {
        moe::set_last_error("cuTensorMapEncodeTiled refused the rows");
        return MOE_ERR_CUDA;
    }
    // a scale of zero still hides what is hidden: -inf times a tiny factor is -inf
    const float c = std::fmax(scale * 1.4426950408889634f, 1e-37f);
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    // At most this many items of n tiles, whatever the lengths on the device are.
    auto items = [&](int n) { return (int64_t)Tq / (n * tokens) + std::min(num_seqs, Tq); };
    const bool single = moe::prompt_in_halves(items(2) * kv_heads, head_dim, Tk / num_seqs, moe::sm_count(dev));
    const int64_t ctas = items(single ? 1 : 2) * kv_heads;
    const moe::PromptArgs a = {(const uint16_t*)q, (const uint16_t*)k, (const uint16_t*)v, q_stride, k_stride, v_stride,
                               cu_q, cu_k, Tq, Tk, num_seqs, q_heads, kv_heads, c, (uint16_t*)out, ((uintptr_t)out & 31u) == 0};
    if (ctas > 0x7fffffffll) return refuse("too many rows");
    const auto launch = head_dim == 128 ? (single ? moe::launch_prompt<128, true> : moe::launch_prompt<128, false>)
                                        : (single ? moe::launch_prompt<64, true> : moe::launch_prompt<64, false>);
    if (e == cudaSuccess) e = launch(a, mq, mk, mv, dev, ctas, (cudaStream_t)stream);
    if (e == cudaSuccess) return MOE_OK;
    moe::set_last_error(cudaGetErrorString(e));
    return MOE_ERR_CUDA;
}
