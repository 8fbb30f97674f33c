// kv_shared.cu -- attention over the positions that groups of sequences have in
// common, read once for their group from the paged Q4_0 cache, on the tcgen05
// tensor cores.
//
// A row is one query head of one new token; the rows of a group that share a
// key/value head are taken 256 at a time (two tiles of 128) against the common
// positions. This kernel leaves each row's sum begun; the kernel of kv_attend.cu
// goes on with what the sequences have for themselves, and joins.
//
// Work. The common positions are cut into units of a key tile (128 positions of a
// head), numbered over (group, head, row tiles); every CTA takes an equal run of
// them, whatever the lengths are. The first piece of an item (rows and head) leaves
// its sum with the rows, the others in their CTA's slot: a CTA has one at most.
//
// A CTA's 16 warps:
//   0-3, 4-7  softmax of tile 0, 1: a thread per row, which also brings its query
//             to shared memory (fp16 after the exact power-of-two prescale of its
//             row)
//   8         the run's pieces
//   9, 10     issue the MMAs of tile 0, 1: S = Q K^T, and O += P V with P in
//             tensor memory
//   11        copies a tile's cells, their keys and their values in turn, into a
//             ring of three half tiles as they are (bulk copies)
//   12-15     codes into tiles (they vote on rare cases over a barrier of their own): a
//             warp takes two of a tile's eight cells and writes
//             d (q - 8) as fp16 to a ring K0 V0 K1 V1 ... of tiles in 128-byte
//             swizzle. Keys lie [key][dim], values [dim][key], as the cells hold
//             them; both K-major. The code is kept short: with the cells in
//             registers and all written out, a tile took 6500 cycles, most of them
//             waiting for instructions.
// Where groups fill one tile of rows, or three, both tiles are the same rows and take
// every other key tile (kSingle); their sums are joined at the end.
//
// Arithmetic. d (q - 8) is rounded to fp16 once, by at most 2^-11 of itself (an eighth of
// what a bf16 key or value may be off by), and so are the weights. A row's weights refer
// to an exponent 6 below its maximum when that was raised, which happens when a score
// exceeds it by 2^kRaise: they reach 2^14, keep all bits down to 2^-20 of the largest and
// count down to 2^-30. fp16 does not hold values from 65504 on: keys of a cell with a
// scale of 4096 or more are written 2^-4 times as large, and its scores raised again;
// value blocks with such a scale are left out of their tile and follow in one of their
// own, divided by 8, which is multiplied eight times. A NaN scale makes its block of the
// output NaN for the rows that see it and for no others. Maxima, sums and outputs are
// fp32.
//
// All waits are bounded. Where one gives up, its warp takes no more pieces (piece_ring.h)
// and the CTA says so in parts.failed, for the join to write NaN.
//
// Measured: 32768 common positions, 512 rows for each of 8 heads, head_dim 128: 75 us
// of the call's 116 (916 TFLOP/s, 0.47 of cuBLAS's bf16 rate), about 4400 cycles a key
// tile where the products take 2150 and shared memory's traffic for them and the
// tiles 2500. The chain of a tile is what runs: softmax 2300, then the values'
// products, the next scores and their waits 2100; the tile warps need 3500 beside
// them. One key tile a CTA (2451 positions, 128 rows): 11 us, nearly all of it
// latency (1.5 us to the first piece, cells, tiles, scores, weights, products, 2 us
// for the sums' stores, much of it code fetched for the first time).
#include <algorithm>

#include "attn_tc.cuh"
#include "kv.cuh"
#include "piece_ring.h"

namespace moe {

constexpr int kSharedThreads = 512;
constexpr float kRaise = 8.0f;    // log2 of the growth a row's weights may reach before a rescale
constexpr float kBelow = 6.0f;    // a row's exponent is so far below its maximum when that is raised
constexpr int kPieceStart = 2;    // what beginning a piece costs, in units
constexpr uint32_t kLargeScale = 0x6c00, kNoNumber = 0x7c00;  // fp16 bits of 4096, and of infinity

struct SharedArgs {
    KvDev c;
    KvBatch b;
    KvGroups g;
    SharedParts parts;
    const uint16_t* q;
    int64_t qs;
    int T;
    float scale;        // times log2 e
    FastDiv group_div;  // by the query heads of a key/value head
};

// A piece of an item: key tiles u0 .. u1 - 1.
struct SharedPiece {
    int seq;         // the group's first sequence, whose table is read
    int t0, rows;    // the group's first packed row; its rows (tokens times heads)
    int row0, head;  // the item's first row; the key/value head
    int u0, u1, common;
    int slot, more;  // of an item's first piece: the first slot of the others, and their number
    int end;         // no piece: the CTA's work is done
};

template <int D>
struct SharedSmem {
    static constexpr int kTileBytes = kTile * D * 2;
    static constexpr int kStages = D == 128 ? 4 : 6;
    static constexpr int kRaw = 3;
    uint8_t q[2][kTileBytes];
    uint8_t kv[kStages][kTileBytes];
    uint8_t raw[kRaw][kTile / kCellTokens][Cell<D>::kBytes / 2];  // the cells' keys, or values, with their scales
    unsigned long long raw_full[kRaw], raw_empty[kRaw];
    unsigned long long q_full[2], full[kStages], empty[kStages], s_full[2], p_full[2][2], o_full[2];
    unsigned long long item_full[2], item_empty[2], half_done, half_read, voted, drained[2];
    float half[kTile][2];  // exponent and sum of a row's second half of key tiles
    SharedPiece item[2];
    int meta[kStages];     // of a tile of values: how often it is multiplied; + 256: another one of the same keys follows
    unsigned absent[kRaw]; // the cells that are not there, a bit each
    unsigned long long large[8];  // of a key tile: the cells written 2^-4 times as large, a byte each
    int nan_from[2][4];    // of a piece, for each block of dims: the first position with a NaN scale
    Votes votes;           // on whether a tile of values has large scales
    int longest;           // key tiles of the longest piece put so far
    int dead;              // a wait has given up
    uint32_t tmem;
};

template <int G>
__device__ __forceinline__ void load_words(uint32_t (&r)[G], const uint8_t* p) {
    if constexpr (G == 4) {
        const uint4 v = *reinterpret_cast<const uint4*>(p);
        r[0] = v.x, r[1] = v.y, r[2] = v.z, r[3] = v.w;
    } else if constexpr (G == 2) {
        const uint2 v = *reinterpret_cast<const uint2*>(p);
        r[0] = v.x, r[1] = v.y;
    } else {
        r[0] = *reinterpret_cast<const uint32_t*>(p);
    }
}
__device__ __forceinline__ uint32_t times(uint32_t a, uint32_t b) { return h2_as_u32(__hmul2(u32_as_h2(a), u32_as_h2(b))); }
// The larger magnitude of a word's two fp16 values, as bits.
__device__ __forceinline__ uint32_t larger_half(uint32_t w) { return max(w & 0x7fffu, (w >> 16) & 0x7fffu); }

template <int D, bool kSingle>
__global__ void __launch_bounds__(kSharedThreads, 1) k_shared(const __grid_constant__ SharedArgs a) {
    using S = SharedSmem<D>;
    using C = Cell<D>;
    constexpr int G = D / 32, kStages = S::kStages, kHalf = kTile * 128;  // bytes of 64 dims of a tile of keys
    constexpr int kRows = kSingle ? kTile : 2 * kTile;                    // of an item
    extern __shared__ uint8_t raw[];
    S& sm = *reinterpret_cast<S*>(raw + (((gsmem(raw) + 1023u) & ~1023u) - gsmem(raw)));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int group = a.c.hq / a.c.hkv;

    if (warp == 10) {
        tc_alloc(gsmem(&sm.tmem), 512);
        tc_relinquish();
    } else if (warp == 9 && lane == 0) {
        for (int x = 0; x < 2; ++x) {
            bar_init_n(gsmem(&sm.q_full[x]), 128);
            bar_init_n(gsmem(&sm.s_full[x]), 1);
            bar_init_n(gsmem(&sm.p_full[x][0]), 128);
            bar_init_n(gsmem(&sm.p_full[x][1]), 128);
            bar_init_n(gsmem(&sm.o_full[x]), 1);
            bar_init_n(gsmem(&sm.item_full[x]), 1);
            bar_init_n(gsmem(&sm.item_empty[x]), 15);  // all warps but the pieces' own
        }
        for (int st = 0; st < kStages; ++st) {
            bar_init_n(gsmem(&sm.full[st]), 4);   // the warps that make tiles
            bar_init_n(gsmem(&sm.empty[st]), 2);  // both MMA warps
        }
        for (int r = 0; r < S::kRaw; ++r) {
            bar_init_n(gsmem(&sm.raw_full[r]), 1);
            bar_init_n(gsmem(&sm.raw_empty[r]), 4);  // the warps that make tiles
        }
        bar_init_n(gsmem(&sm.half_done), 128);
        bar_init_n(gsmem(&sm.half_read), 128);
        bar_init_n(gsmem(&sm.voted), 4);  // the warps that make tiles
        bar_init_n(gsmem(&sm.drained[0]), 1);
        bar_init_n(gsmem(&sm.drained[1]), 1);
        sm.longest = 0;
        sm.dead = 0;
        asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    }
    __syncwarp();
    griddep_wait();
    griddep_launch();
    // the pieces' warp: what the groups ask for, while the others set up
    int seq, t0, rows, common, work, total = 0;  // of a lane's group; of all
    auto look = [&](int g) {
        seq = t0 = rows = common = work = 0;
        if (g >= a.g.n) return;
        seq = a.g.cu[g];
        const int last = min(max(a.g.cu[g + 1], 0), a.b.B);
        if (seq < 0 || seq >= last) return;
        t0 = min(max(a.b.cu[seq], 0), a.T);
        rows = max(min(max(a.b.cu[last], 0), a.T) - t0, 0) * group;
        common = common_tokens(a.c, a.b, a.g, g);
        if (rows && common) work = ((common + kTile - 1) / kTile + kPieceStart) * a.c.hkv * ((rows + kRows - 1) / kRows);
    };
    if (warp == 8) {
        for (int g = lane; g - lane < a.g.n; g += 32) {
            look(g);
            total += work;
        }
        total = __reduce_add_sync(0xffffffffu, total);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm.tmem;
    int* dead = &sm.dead;

    // What a wait for a piece has, to be put or to be given back: 20 us for each key tile
    // of the longest one, which may be at work meanwhile, and 0.1 us for each group, which
    // are looked through for the next one (32 at a time, in 0.5 us).
    auto limit = [&]() { return kGWaitNs + 20000ull * (unsigned)*(volatile int*)&sm.longest + 100ull * (unsigned)a.g.n; };
    // The next piece, for whole warps; false at the end. `number` counts the pieces taken.
    auto take = [&](int number) {
        return take_piece(
            number, [&](int place, uint32_t parity) { return warp_wait(gsmem(&sm.item_full[place]), parity, dead, limit); },
            [&](int place) { return sm.item[place].end != 0; });
    };
    auto give_back = [&](int number) {
        __syncwarp();
        if (lane == 0) bar_arrive(gsmem(&sm.item_empty[number & 1]));
    };
    // key tiles of tile x
    auto tiles_of = [&](const SharedPiece& p, int x) {
        const int n = p.u1 - p.u0;
        return kSingle ? (n + 1 - x) / 2 : x == 0 || p.rows - p.row0 > kTile ? n : 0;
    };

    // Registers: the launch gives 128 a thread (65536 in all).
    if (warp >= 12) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;\n");
        // --- codes into tiles. A warp has cells 2w and 2w + 1 of a tile. Keys: lane
        // -> token and quarter of each block, so that eight lanes read and write
        // without conflicts. Values: lane -> cell, half of its tokens, and dims g +
        // 8 j of each block.
        const int w = warp - 12, ki = lane & 3, kp = lane >> 3, kt = lane & 4 ? kp ^ 5 : kp;
        const int vz = lane >> 4, vh = (lane >> 3) & 1, vg = lane & 7;
        int st = 0, raw_st = 0, order = 0;  // stage, half tile; tiles so far
        uint32_t turn = 1, raw_turn = 0;
        auto step = [&]() { if (++st == kStages) st = 0, turn ^= 1; };
        auto next_raw = [&]() {
            bar_wait(gsmem(&sm.raw_full[raw_st]), raw_turn, dead);
            __syncwarp();
        };
        auto free_raw = [&]() {
            __syncwarp();
            if (lane == 0) bar_arrive(gsmem(&sm.raw_empty[raw_st]));
            if (++raw_st == S::kRaw) raw_st = 0, raw_turn ^= 1;
        };
        auto stage_full = [&]() {
            fence_async_smem();
            __syncwarp();
            if (lane == 0) bar_arrive(gsmem(&sm.full[st]));
            step();
        };
        // The scales of the warp's two cells, a word a lane; none in cells that are not there.
        constexpr bool kAll = C::kScales == 128;  // every lane has one
        auto scale_word = [&](int z) { return reinterpret_cast<uint32_t*>(sm.raw[raw_st][2 * w + z] + C::kCodes) + lane; };
        auto put_scales = [&](const uint32_t (&v)[2]) {
            __syncwarp();
#pragma unroll
            for (int z = 0; z < 2; ++z)
                if (kAll || lane < C::kScales / 4) *scale_word(z) = v[z];
            __syncwarp();
        };
        auto get_scales = [&](uint32_t (&v)[2]) {
            const unsigned absent = __shfl_sync(0xffffffffu, sm.absent[raw_st] >> (2 * w) & 3u, 0);
#pragma unroll
            for (int z = 0; z < 2; ++z) v[z] = kAll || lane < C::kScales / 4 ? *scale_word(z) : 0u;
            if (absent) {
#pragma unroll
                for (int z = 0; z < 2; ++z)
                    if (absent >> z & 1u) v[z] = 0;
                put_scales(v);
            }
        };
        for (int number = 0; take(number); ++number) {
            const int u1 = sm.item[number & 1].u1;
#pragma unroll 1
            for (int tile = sm.item[number & 1].u0; tile < u1; ++tile, ++order) {
                uint32_t v[2];
                // --- keys
                next_raw();
                get_scales(v);
                {
                    const bool l0 = __any_sync(0xffffffffu, larger_half(v[0]) >= kLargeScale);
                    const bool l1 = __any_sync(0xffffffffu, larger_half(v[1]) >= kLargeScale);
                    if (lane == 0) reinterpret_cast<uint16_t*>(&sm.large[order & 7])[w] = (uint16_t)((l0 ? 1 : 0) | (l1 ? 256 : 0));
                    if (l0 || l1) {  // 2^-4 times as large
                        if (l0) v[0] = times(v[0], 0x2c002c00u);
                        if (l1) v[1] = times(v[1], 0x2c002c00u);
                        put_scales(v);
                    }
                }
                bar_wait(gsmem(&sm.empty[st]), turn, dead);
#pragma unroll 1
                for (int z = 0; z < 2; ++z) {
                    const uint8_t* cell = sm.raw[raw_st][2 * w + z];
                    uint8_t* to = sm.kv[st] + ((2 * w + z) * kCellTokens + kt) * 128;
                    uint32_t codes[2][G], ds[2][G / 2];
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        load_words<G>(codes[u], cell + C::k_word(kt + 8 * u, ki, 0));
                        load_words<G / 2>(ds[u], cell + C::kCodes + C::k_scale(kt + 8 * u, 0));
                    }
#pragma unroll
                    for (int u = 0; u < 2; ++u)
#pragma unroll
                        for (int b = 0; b < G; ++b) {
                            const uint32_t d = __byte_perm(ds[u][b / 2], 0, b & 1 ? 0x3232 : 0x1010);
                            uint32_t f[4];
                            q4_to_frag(codes[u][b], f);
                            *reinterpret_cast<uint4*>(to + u * 1024 + (b / 2) * kHalf + ((((b & 1) * 4 + ki) ^ kt) << 4)) =
                                make_uint4(times(f[0], d), times(f[1], d), times(f[2], d), times(f[3], d));
                        }
                }
                stage_full();
                free_raw();
                // --- values: once, and where some scales are large a second time
                next_raw();
                get_scales(v);
                const bool any = __any_sync(
                    0xffffffffu,
                    any_of_four(
                        sm.votes, order, w, __any_sync(0xffffffffu, max(larger_half(v[0]), larger_half(v[1])) >= kLargeScale),
                        [&](auto vote) {
                            if (lane == 0) {
                                vote();
                                bar_arrive(gsmem(&sm.voted));
                            }
                        },
                        [&](uint32_t parity) { bar_wait(gsmem(&sm.voted), parity, dead); }));
                uint32_t rest[2] = {0, 0};
                if (any) {  // the small ones first, then an eighth of the large ones
#pragma unroll
                    for (int z = 0; z < 2; ++z) {
                        rest[z] = times(v[z], 0x30003000u);
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const uint32_t bits = (v[z] >> (16 * h)) & 0x7fffu, other = ~(0xffffu << (16 * h));
                            if (bits >= kNoNumber)
                                atomicMin(&sm.nan_from[number & 1][lane % G],
                                          tile * kTile + (2 * w + z) * kCellTokens + 8 * (lane / (4 * G)) + 2 * (lane / G % 4) + h);
                            if (bits < kLargeScale || bits >= kNoNumber) rest[z] &= other;
                            if (bits >= kLargeScale) v[z] &= other;
                        }
                    }
                    put_scales(v);
                }
                const uint8_t* cell = sm.raw[raw_st][2 * w + vz];
                const int chunk = 2 * (2 * w + vz) + vh;  // 8 keys each
#pragma unroll 1
                for (int pass = 0;; ++pass) {
                    bar_wait(gsmem(&sm.empty[st]), turn, dead);
                    uint8_t* to = sm.kv[st] + (chunk >> 3) * (D * 128) + vg * 128 + (((chunk & 7) ^ vg) << 4);
                    uint32_t codes[4][G], scale[4][G];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        load_words<G>(codes[i], cell + ((vh * 32 + vg * 4 + i) * G) * 4);
                        load_words<G>(scale[i], cell + C::kCodes + ((vh * 4 + i) * G) * 4);
                    }
#pragma unroll
                    for (int b = 0; b < G; ++b) {
                        uint32_t f[4][4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) q4_to_frag(codes[i][b], f[i]);
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            *reinterpret_cast<uint4*>(to + (32 * b + 8 * j) * 128) =
                                make_uint4(times(f[0][j], scale[0][b]), times(f[1][j], scale[1][b]), times(f[2][j], scale[2][b]),
                                           times(f[3][j], scale[3][b]));
                    }
                    if (tid == kSharedThreads - 128) sm.meta[st] = pass ? 8 : any ? 1 + 256 : 1;
                    stage_full();
                    if (pass == (int)any) break;
                    put_scales(rest);
                }
                free_raw();
            }
            give_back(number);
        }
    } else if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 40;\n");
        if (warp == 8) {
            // --- the pieces of this CTA's run [lo, hi)
            const int ctas = min(total, (int)gridDim.x), base = ctas ? total / ctas : 0, extra = total - base * ctas;
            auto cta_of = [&](int x) {
                const int wide = extra * (base + 1);
                return x < wide ? x / (base + 1) : extra + (x - wide) / base;
            };
            const bool has = (int)blockIdx.x < ctas;
            const int lo = has ? blockIdx.x * base + min((int)blockIdx.x, extra) : 0;
            const int hi = has ? lo + base + ((int)blockIdx.x < extra) : 0;
            int number = 0, before = 0, x = lo;
            bool open = true;  // false once a wait for a place has given up: no more pieces
            auto put = [&](const SharedPiece& p) {
                open = open && put_piece(
                                   number,
                                   [&](int place, uint32_t parity) {
                                       return warp_wait(gsmem(&sm.item_empty[place]), parity, dead, limit);
                                   },
                                   [&](int place) {
                                       if (lane < 4) sm.nan_from[place][lane] = 0x7fffffff;
                                       __syncwarp();
                                       if (lane == 0) {
                                           sm.longest = max(sm.longest, p.u1 - p.u0);
                                           sm.item[place] = p;
                                           bar_arrive(gsmem(&sm.item_full[place]));
                                       }
                                       __syncwarp();
                                   });
                ++number;
            };
            for (int g0 = 0; g0 < a.g.n && x < hi && open; g0 += 32) {
                if (a.g.n > 32) look(g0 + lane);
                int upto = work;
#pragma unroll
                for (int off = 1; off < 32; off <<= 1) {
                    const int v = __shfl_up_sync(0xffffffffu, upto, off);
                    if (lane >= off) upto += v;
                }
                upto += before;
                before = __shfl_sync(0xffffffffu, upto, 31);
                while (x < hi && x < before && open) {
                    const int l = __ffs(__ballot_sync(0xffffffffu, x < upto)) - 1;  // the group of number x
                    SharedPiece p;
                    p.seq = __shfl_sync(0xffffffffu, seq, l);
                    p.t0 = __shfl_sync(0xffffffffu, t0, l);
                    p.rows = __shfl_sync(0xffffffffu, rows, l);
                    p.common = __shfl_sync(0xffffffffu, common, l);
                    const int start = __shfl_sync(0xffffffffu, upto - work, l);
                    const int units = (p.common + kTile - 1) / kTile, len = units + kPieceStart, tiles = (p.rows + kRows - 1) / kRows;
                    const int item = (x - start) / len, in = x - start - item * len, to = min(len, in + hi - x);
                    p.u0 = max(in - kPieceStart, 0);
                    p.u1 = max(to - kPieceStart, 0);
                    p.head = item / tiles;
                    p.row0 = (item - p.head * tiles) * kRows;
                    p.end = 0;
                    const int first = x - in + kPieceStart, c0 = cta_of(first);
                    p.slot = c0 + 1;
                    p.more = cta_of(first + units - 1) - c0;
                    x += to - in;
                    if (p.u1 > p.u0) put(p);
                }
            }
            SharedPiece none = {};
            none.end = 1;
            put(none);
        } else if (warp < 11) {
            // --- the MMAs of tile x. The whole warp walks the loop and one lane
            // issues. Both warps pass every stage of the ring, needed or not: no
            // barrier may complete twice before both have passed.
            constexpr uint32_t id_s = tc_idesc_f16(kTile, kTile), id_o = tc_idesc_f16(kTile, D);
            const int x = __shfl_sync(0xffffffffu, warp - 9, 0);
            const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
            const uint32_t ts = tm + x * kTile, to = tm + 2 * kTile + x * D;
            const bool leader = elect_one();
            const uint64_t qd = tc_sdesc(gsmem(sm.q[0]) + x * S::kTileBytes), kd = tc_sdesc(gsmem(sm.kv[0]));
            constexpr uint64_t kTileStep = S::kTileBytes >> 4;  // to the next stage, in a descriptor
            auto scores = [&](int st) {
                const uint64_t kx = kd + st * kTileStep;
#pragma unroll
                for (int d = 0; d < D / 16; ++d) {
                    const uint32_t off = ((d / 4) * kHalf + (d % 4) * 32) >> 4;
                    tc_mma(ts, qd + off, kx + off, id_s, d != 0);
                }
                tc_commit(gsmem(&sm.s_full[x]));
            };
            auto values = [&](int half, int st, bool first) {  // of the tile's keys 64 half ..
                const uint64_t vx = kd + st * kTileStep + half * ((D * 128) >> 4);
#pragma unroll
                for (int t = 0; t < kTile / 32; ++t)
                    tc_mma_ta(to, ts + 32 * half + 8 * t, vx + 2 * t, id_o, t == 0 ? !first : 1);
            };
            auto free_stage = [&](int st, bool used) {
                if (!leader) return;
                if (used) tc_commit(gsmem(&sm.empty[st]));
                else bar_arrive(gsmem(&sm.empty[st]));
            };
            auto meta_of = [&](int st) { return __shfl_sync(0xffffffffu, *(volatile int*)&sm.meta[st], 0); };
            int st = 0;
            uint32_t round = 0, p_turn = 0, q_turn = 0;
            auto next_stage = [&]() {  // waits for the stage, and steps on
                const int s = st;
                bar_wait(gsmem(&sm.full[s]), round, dead);
                if (++st == kStages) st = 0, round ^= 1;
                __syncwarp();
                tc_fence_after();
                return s;
            };
            for (int number = 0; take(number); ++number) {
                const int n = sm.item[number & 1].u1 - sm.item[number & 1].u0, nx = tiles_of(sm.item[number & 1], x);
                give_back(number);
                int done = 0;
                for (int i = 0; i < n; ++i) {  // (the whole warp alike, whatever the waits have seen)
                    const bool mine = kSingle ? (i & 1) == x : nx > 0;
                    const int sk = next_stage();
                    if (mine) {
                        if (done == 0) {
                            bar_wait(gsmem(&sm.q_full[x]), q_turn, dead);
                            q_turn ^= 1;
                            __syncwarp();
                            tc_fence_after();
                        }
                        if (leader) scores(sk);
                    }
                    free_stage(sk, mine);
                    __syncwarp();
                    int sv = next_stage();
                    int meta = meta_of(sv);
                    if (mine) {
                        for (int half = 0; half < 2; ++half) {
                            bar_wait(gsmem(&sm.p_full[x][half]), p_turn, dead);
                            __syncwarp();
                            tc_fence_after();
                            if (leader) values(half, sv, done == 0 && half == 0);
                            __syncwarp();
                        }
                        p_turn ^= 1;
                        ++done;
                        if (leader && done == nx && meta < 256) tc_commit(gsmem(&sm.o_full[x]));
                    }
                    free_stage(sv, mine);
                    __syncwarp();
                    while (meta >= 256) {  // the keys' large values
                        sv = next_stage();
                        meta = meta_of(sv);
                        if (mine && leader) {
                            for (int e = 0; e < (meta & 255); ++e) {
                                values(0, sv, false);
                                values(1, sv, false);
                            }
                            if (done == nx && meta < 256) tc_commit(gsmem(&sm.o_full[x]));
                        }
                        free_stage(sv, mine);
                        __syncwarp();
                        if (warp_dead(dead)) break;
                    }
                }
            }
            // the last arrivals, so that none is under way when the CTA ends; where one does not
            // come, the products
            bool over = true;
            for (int e = 0; e < kStages; ++e) over &= bar_wait(gsmem(&sm.empty[e]), e < st ? round : round ^ 1, dead);
            if (!__all_sync(0xffffffffu, over)) {
                if (leader) tc_commit(gsmem(&sm.drained[x]));
                __syncwarp();
                bar_wait(gsmem(&sm.drained[x]), 0, dead, true);
            }
        } else {
            // --- the cells' bytes: lane n has cell n of a tile
            constexpr uint32_t kBytes = C::kBytes / 2;
            int r = 0;
            uint32_t turn = 1;
            for (int number = 0; take(number); ++number) {
                const SharedPiece& p = sm.item[number & 1];
                const int seq = p.seq, head = p.head, u1 = p.u1, cells = p.common / kCellTokens;
#pragma unroll 1
                for (int tile = p.u0; tile < u1; ++tile) {
                    const int n = tile * (kTile / kCellTokens) + lane;
                    const bool inside = lane < kTile / kCellTokens && n < cells;
                    const uint8_t* at = inside ? kv_cell<D>(a.c, a.b, seq, n, head) : nullptr;
                    if (inside && !at) {  // no such page: its values are NaN
                        atomicOr(a.c.err, 1u);
                        for (int b = 0; b < G; ++b) atomicMin(&sm.nan_from[number & 1][b], n * kCellTokens);
                    }
                    const unsigned there = __ballot_sync(0xffffffffu, at != nullptr);
#pragma unroll 1
                    for (int half = 0; half < 2; ++half) {
                        bar_wait(gsmem(&sm.raw_empty[r]), turn, dead);
                        if (warp_dead(dead)) break;  // no more copies: r is the stage after the last one
                        const uint32_t bar = gsmem(&sm.raw_full[r]);
                        if (lane == 0) {
                            sm.absent[r] = ~there;
                            bar_expect(bar, kBytes * __popc(there));
                        }
                        __syncwarp();
                        if (at)
                            asm volatile(
                                "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n" ::"r"(
                                    gsmem(sm.raw[r][lane & 7])),
                                "l"(at + half * kBytes), "r"(kBytes), "r"(bar)
                                : "memory");
                        if (++r == S::kRaw) r = 0, turn ^= 1;
                    }
                }
                give_back(number);
            }
            // copies under way land before the CTA leaves, whatever else gave up
            for (int e = 0; e < S::kRaw; ++e) bar_wait(gsmem(&sm.raw_full[e]), e < r ? turn ^ 1 : turn, dead, true);
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 200;\n");
        // --- softmax of tile x, a thread per row
        const int x = warp >> 2, row = tid & 127;
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        const uint32_t ts = tmem + lanes + x * kTile, to = tmem + lanes + 2 * kTile + x * D;
        uint32_t s_turn = 0, o_turn = 0, half_turn = 0;
        int order = 0;  // key tiles before this piece
        for (int number = 0; take(number); ++number) {
            const SharedPiece& p = sm.item[number & 1];
            const int n = p.u1 - p.u0, nx = tiles_of(p, x), u0 = p.u0;
            const int r = p.row0 + (kSingle ? 0 : x * kTile) + row;  // among the group's rows
            const bool used = r < p.rows;
            const int tok = a.group_div.div(used ? r : 0), head = p.head * group + (used ? r : 0) - tok * group, t = p.t0 + tok;
            int lim = 0;  // positions that the row sees
            float c = 0.f;
            if (nx) {
                // the query as fp16, and its row's factor
                uint32_t w[D / 2];
                if (used) {
                    const uint16_t* src = a.q + (size_t)t * a.qs + (size_t)head * D;
#pragma unroll
                    for (int e = 0; e < D / 8; ++e) load_words<4>(*reinterpret_cast<uint32_t(*)[4]>(w + 4 * e), (const uint8_t*)(src + 8 * e));
                    int seq = min(t, a.b.B - 1);  // in a decode step row t is sequence t's
                    if (!(a.b.cu[seq] <= t && t < a.b.cu[seq + 1])) seq = seq_of_row(a.b.cu, a.b.B, t);
                    if (seq >= 0) lim = max(min(a.b.kv_lens[seq] - (a.b.cu[seq + 1] - t) + 1, p.common), 0);
                } else {
#pragma unroll
                    for (int e = 0; e < D / 2; ++e) w[e] = 0;
                }
                unsigned mx = 0;
#pragma unroll
                for (int e = 0; e < D / 2; ++e) mx = max(mx, bf16x2_absmax(w[e]));
                const int sh = token_shift(mx);
                const float f = pow2f(-sh);
                // a scale of zero still hides what is hidden: -inf times a tiny factor is -inf
                c = fmaxf(a.scale * pow2f(sh), 1e-37f);
#pragma unroll
                for (int e = 0; e < D / 8; ++e) {
                    uint32_t h[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint32_t v = w[4 * e + k];
                        h[k] = h2_as_u32(__floats2half2_rn(__uint_as_float(v << 16) * f, __uint_as_float(v & 0xffff0000u) * f));
                    }
                    *reinterpret_cast<uint4*>(sm.q[x] + (e >> 3) * kHalf + row * 128 + (((e & 7) ^ (row & 7)) << 4)) =
                        make_uint4(h[0], h[1], h[2], h[3]);
                }
                fence_async_smem();
                bar_arrive(gsmem(&sm.q_full[x]));
            }
            const int lim_warp = __reduce_min_sync(0xffffffffu, used ? lim : 0x7fffffff);
            float m = -INFINITY, l = 0.f;
#pragma unroll 1
            for (int j = 0; j < nx; ++j) {
                bar_wait(gsmem(&sm.s_full[x]), s_turn, dead);
                s_turn ^= 1;
                const int tile = kSingle ? 2 * j + x : j, kt = u0 + tile;
                __syncwarp();
                tc_fence_after();
                const unsigned long long large = *(volatile unsigned long long*)&sm.large[(order + tile) & 7];
                if (__any_sync(0xffffffffu, large != 0)) {
                    // scores of cells written 2^-4 times as large
#pragma unroll 1
                    for (int h = 0; h < kTile / 32; ++h) {
                        uint32_t v[32];
                        tc_ld32(ts + 32 * h, v);
                        tc_ld_wait32(v);
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            v[e] = __float_as_uint(__uint_as_float(v[e]) * (large >> (8 * (2 * h + (e >> 4))) & 1u ? 16.f : 1.f));
                        tc_st32(ts + 32 * h, v);
                    }
                    tc_st_wait();
                }
                if ((kt + 1) * kTile > lim_warp) hide_scores(ts, lim - kt * kTile);
                // The row's scores are read twice, 32 at a time and the next ones on their
                // way, in loops that stay short.
                uint32_t s0[32], s1[32];
                float mx4[4] = {m, m, m, m};
                auto most = [&](const uint32_t (&v)[32]) {
#pragma unroll
                    for (int e = 0; e < 32; e += 2)
                        mx4[(e >> 1) & 3] = max3(mx4[(e >> 1) & 3], __uint_as_float(v[e]), __uint_as_float(v[e + 1]));
                };
                tc_ld32(ts, s0);
#pragma unroll 1
                for (int h = 0; h < 4; h += 2) {
                    tc_ld_wait32(s0);
                    tc_ld32(ts + 32 * h + 32, s1);
                    most(s0);
                    tc_ld_wait32(s1);
                    tc_ld32(ts + (h ? 0 : 64), s0);  // the third quarter, then the first again
                    most(s1);
                }
                tc_ld_wait32(s0);
                const float mx = fmaxf(max3(mx4[0], mx4[1], mx4[2]), mx4[3]);
                const bool raise = (mx - m) * c > kRaise;
                if (__any_sync(0xffffffffu, raise)) {
                    // these scores came after the last tile's O, so O is at rest
                    const float f = raise ? ex2f((m - mx) * c) : 1.f;
                    if (raise) m = mx;
                    l *= f;
                    if (j > 0) {
#pragma unroll 1
                        for (int h = 0; h < D / 32; ++h) {
                            uint32_t o[32];
                            tc_ld32(to + 32 * h, o);
                            tc_ld_wait32(o);
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                            tc_st32(to + 32 * h, o);
                        }
                    }
                }
                const float mc = m == -INFINITY ? 0.f : fmaf(m, c, -kBelow);
                const unsigned long long c2 = pair2(c, c), mc2 = pair2(-mc, -mc);
                unsigned long long sum[4] = {0, 0, 0, 0};
                auto weights = [&](const uint32_t (&v)[32], int h) {
                    uint32_t w[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const unsigned long long y =
                            fma2(pair2(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1])), c2, mc2);
                        const float e0 = ex2f(lo2(y)), e1 = ex2f(hi2(y));
                        sum[e & 3] = add2(sum[e & 3], pair2(e0, e1));
                        w[e] = h2_as_u32(__floats2half2_rn(e0, e1));
                    }
                    tc_st16(ts + 16 * h, w);
                };
#pragma unroll 1
                for (int h = 0; h < 4; h += 2) {
                    if (h) tc_ld_wait32(s0);
                    tc_ld32(ts + 32 * h + 32, s1);
                    weights(s0, h);
                    tc_ld_wait32(s1);
                    if (h == 0) tc_ld32(ts + 64, s0);
                    weights(s1, h + 1);
                    // the products with the first 64 keys begin while the other weights are computed
                    tc_st_wait();
                    tc_fence_before();
                    bar_arrive(gsmem(&sm.p_full[x][h >> 1]));
                }
                sum[0] = add2(add2(sum[0], sum[1]), add2(sum[2], sum[3]));
                l += lo2(sum[0]) + hi2(sum[0]);
            }
            float low = m == -INFINITY ? -INFINITY : fmaf(m, c, -kBelow);  // the exponent that the weights refer to
            if (nx) {
                bar_wait(gsmem(&sm.o_full[x]), o_turn, dead);
                o_turn ^= 1;
            }
            __syncwarp();
            tc_fence_after();
            // two halves of the key tiles: slot 1 leaves its exponents and sums, and
            // slot 0 writes out both
            const bool halves = kSingle && n > 1;
            float scale0 = 1.f, scale1 = 0.f;
            if (halves) {
                if (x) {
                    sm.half[row][0] = low;
                    sm.half[row][1] = l;
                    tc_fence_before();
                    bar_arrive(gsmem(&sm.half_done));
                    bar_wait(gsmem(&sm.half_read), half_turn, dead);  // before O is written again
                } else {
                    bar_wait(gsmem(&sm.half_done), half_turn, dead);
                    __syncwarp();
                    tc_fence_after();
                    const float low1 = sm.half[row][0], high = fmaxf(low, low1);
                    scale0 = low == -INFINITY ? 0.f : ex2f(low - high);
                    scale1 = low1 == -INFINITY ? 0.f : ex2f(low1 - high);
                    l = fmaf(l, scale0, sm.half[row][1] * scale1);
                    low = high;
                }
                half_turn ^= 1;
            }
            // --- the row's sum, or a part of it
            const bool first = u0 == 0;
            const size_t place = first ? (size_t)t * a.c.hq + head
                                       : (size_t)blockIdx.x * kSlotRows + (kSingle ? 0 : x * kTile) + row;
            float* dst = (first ? a.parts.o : a.parts.slot_o) + place * D;
            const bool mine = used && nx && !(x && kSingle);
#pragma unroll 1
            for (int h = 0; h < (nx && !(x && kSingle) ? D / 32 : 0); ++h) {
                uint32_t o[32];
                __syncwarp();
                tc_ld32(to + 32 * h, o);
                tc_ld_wait32(o);
                if (halves) {
                    uint32_t o1[32];
                    tc_ld32(to + D + 32 * h, o1);
                    tc_ld_wait32(o1);
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        o[e] = __float_as_uint(__uint_as_float(o[e]) * scale0 + __uint_as_float(o1[e]) * scale1);
                }
                if (*(volatile int*)&sm.nan_from[number & 1][h] < lim) {
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = 0x7fc00000u;
                }
                if (mine) {
#pragma unroll
                    for (int e = 0; e < 32; e += 8)  // a lane's row is a line of its own: whole sectors
                        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};\n" ::"l"(dst + 32 * h + e), "r"(o[e]),
                                     "r"(o[e + 1]), "r"(o[e + 2]), "r"(o[e + 3]), "r"(o[e + 4]), "r"(o[e + 5]), "r"(o[e + 6]),
                                     "r"(o[e + 7])
                                     : "memory");
                }
            }
            if (mine) {
                if (*(volatile int*)dead) l = __int_as_float(0x7fc00000);  // a wait gave up
                const int more = p.more | (r - p.row0) << 16;
                (first ? a.parts.head : a.parts.slot_head)[place] = make_float4(low, l, __int_as_float(p.slot), __int_as_float(more));
            }
            tc_fence_before();  // the reads of O, before the weights that let it be overwritten
            if (halves && !x) bar_arrive(gsmem(&sm.half_read));
            order += n;
            give_back(number);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (tid == 0) a.parts.failed[blockIdx.x] = *(volatile int*)dead;
    if (warp == 10) {
        tc_fence_after();
        tc_dealloc(tmem, 512);
    }
}

static uint64_t dense_rows(int T, int hq) { return (uint64_t)T * hq; }

uint64_t shared_bytes(int device, int T, int hq, int D) {
    const uint64_t ctas = sm_count(device);
    return (2 * dense_rows(T, hq) + ctas * kSlotRows) * (D * sizeof(float) + sizeof(float4)) + ctas * sizeof(int);
}

SharedParts shared_parts(void* workspace, int device, int T, int hq, int D) {
    const uint64_t rows = dense_rows(T, hq), slots = (uint64_t)sm_count(device) * kSlotRows;
    SharedParts p;
    p.o = (float*)workspace;
    p.rest_o = p.o + rows * D;
    p.slot_o = p.rest_o + rows * D;
    p.head = (float4*)(p.slot_o + slots * D);
    p.rest_head = p.head + rows;
    p.slot_head = p.rest_head + rows;
    p.failed = (int*)(p.slot_head + slots);
    p.slots = sm_count(device);
    return p;
}

bool shared_fits(const KvDev& c, const KvBatch& b, int groups, int T) {
    const int64_t rows = (int64_t)T * (c.hq / c.hkv), tiles = rows / kTile + std::min(groups, T);
    const int64_t units = (int64_t)b.table_stride * c.page_tokens / kTile + 1;
    return rows < (1ll << 30) && (double)tiles * (double)(units + kPieceStart) * (double)c.hkv < (double)(1ll << 30);
}

template <int D, bool kSingle>
static cudaError_t launch_k(const SharedArgs& a, int dev, cudaStream_t st) {
    constexpr int bytes = (int)sizeof(SharedSmem<D>) + 1024;
    static DeviceOnce once;
    const cudaError_t set = once.run(dev, [] {
        return cudaFuncSetAttribute(k_shared<D, kSingle>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    });
    if (set != cudaSuccess) return set;
    return launch_ex(k_shared<D, kSingle>, dim3((unsigned)sm_count(dev)), dim3(kSharedThreads), bytes, st, true, a);
}

cudaError_t launch_shared(const KvDev& c, const KvBatch& b, const KvGroups& g, const SharedParts& parts, int D,
                          const uint16_t* q, int64_t q_stride, int T, float scale, cudaStream_t st) {
    int dev = 0;
    if (const cudaError_t e = cudaGetDevice(&dev); e != cudaSuccess) return e;
    const int group = c.hq / c.hkv;
    const SharedArgs a = {c, b, g, parts, q, q_stride, T, scale * 1.4426950408889634f, fast_div((uint32_t)group)};
    const bool single = shared_in_single_tiles((int64_t)T * group, g.n, kTile);
    if (D == 128) return single ? launch_k<128, true>(a, dev, st) : launch_k<128, false>(a, dev, st);
    return single ? launch_k<64, true>(a, dev, st) : launch_k<64, false>(a, dev, st);
}

}  // namespace moe
