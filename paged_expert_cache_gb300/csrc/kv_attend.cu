// kv_attend.cu -- attention of the newest tokens over the paged Q4_0 cache.
//
// A row is one query head of one new token; out = sum_p softmax_p(scale q .
// k_p) v_p over the positions p it sees. The rows that share a key/value head
// (its group of query heads, times the sequence's new tokens) are taken 8 or
// 16 at a time against the cache, so each block is read from HBM once for a
// decode step. The bytes of the cache are the floor: 18 per 32 values, keys
// and values once.
//
// Work. The sequences' contexts are cut into units of kWarps cells (a cell is
// 16 tokens of one head); units are numbered over (sequence, head, row tile)
// and every CTA takes an equal run of them, whatever the lengths are: the
// lengths are read on the device, and a long sequence is spread over the whole
// GPU. A run's pieces that cover an item only in part leave a partial sum
// (maximum, sum, unnormalised output), and a second small kernel, launched
// behind the first, adds an item's pieces in order. (The last CTA to arrive
// doing it instead cost each piece a fence and an atomic, about 2000 cycles, and
// a long sequence one CTA's walk over 76 pieces, about 20000.)
//
// A warp owns every kWarps-th cell of the run: it asks for its cells kStages
// ahead with 16-byte asynchronous copies into a ring of its own, and never waits
// for another warp before the end of an item. A cell is 2304 bytes at head_dim
// 128. (One bulk copy and mbarrier per cell in their place cost a warp about
// 1000 of 3200 cycles for every two cells: the issue alone 760.)
//
// Arithmetic. A 4-bit code q masked out of its word is the fp16 subnormal q *
// 2^-24 (or q * 2^-20 for the upper nibble of a byte), which the tensor cores
// multiply exactly, so codes become operands with one AND.
//  scores: A = key codes (16 tokens), B = q (8 rows; fp16 after the exact
//    power-of-two prescale of its row). The codes keep their 8: a block's sum
//    starts at -8 sum(q) instead (the sums are then within 8e-7 of a random
//    row's score, measured), and is multiplied by the block's scale in fp32.
//  values: A = value codes (32 dims by 16 tokens), here with the 8 subtracted
//    (exact in fp16), since a sum that only cancels would leave a rounding of
//    8 d p where the values met are zero; B = p * d for each block, from the
//    scores' layout by one 8 x 8 transposition, rounded to fp16 twice (p, then
//    the product: 2^-11 each, an eighth of the output's own rounding each).
//    fp16's range does not hold every product. What a row sees of a block of
//    dimensions is `far` from the first product past it on, or from a warp's
//    first step on where its scales there are below kQuiet: such products are
//    formed in fp32 and taken as two bf16 operands (16 bits, fp32's range), in
//    matrix products of their own to which the other rows give zeros. So neither
//    other blocks, nor what other rows see, nor what no row sees touch a bit of it.
//    (One power of two for all of a warp's scales is faster there, 157 us for the
//    64 sequences below with values 20 times as large or 1000 times as small, in
//    place of 169 and 250; but a block 2^11 below the largest one met, hidden or
//    not, loses bits by it.)
// Softmax statistics, sums and outputs are fp32. A row's running maximum is
// raised only when a score exceeds it by 2^kLazy, the outputs being rescaled
// then.
//
// Measured in a graph at head_dim 128: 64 sequences of 4000 to 12000 tokens, 64
// query heads over 8, 120 us (4.9 TB/s, 0.73 of a copy's rate; the warps' issue slots
// and latencies bound it, not the memory). 28 or 32 heads over 4: 32 sequences of up
// to 4095 tokens 19.3 us, one of 100003 tokens 24.0, one of 513 tokens 8.5, where the
// two launches, an item's start and the join are most of it.
#include <algorithm>
#include <type_traits>

#include "kv.cuh"

namespace moe {

constexpr int kWarps = 8;
constexpr int kAttThreads = 32 * kWarps;
constexpr int kStages = 4;
constexpr int kMaxCtas = 304;             // two per SM
// What beginning an item costs, in units: its rows to be fetched and laid out,
// the warps' sums to be joined and written (about 8000 cycles, a unit 1400). Items
// are numbered with so many idle units before their first, so that CTAs with
// many short sequences get fewer cells (2, 4, 6, 9: 20.6, 20.0, 19.7, 20.7 us for
// 32 streams of up to 4095 tokens).
constexpr int kBegin = 6;
// fp16's range for the product p * d. A row's largest weight is 2^kOffset when
// its maximum is set and may grow by 2^kLazy, so with scales below 2 a product is
// below 2^15, and with scales of kQuiet and more weights down to 2^-14 of the
// largest keep all bits and down to 2^-24 count (down to 2^-34 / d for a smaller
// scale d that comes later in a block that is not far). A row that has seen a
// scale of 2 or more raises its maximum at once: its products then hold scales up
// to 2^5 (with values 20 times as large as usual 169 us, 258 if it is as lazy as
// others).
constexpr float kLazy = 4.0f, kOffset = 10.0f;
constexpr uint32_t kMost = 0x7bff, kQuiet = 0x1400;  // fp16's largest value, and 2^-10
constexpr float kLog2e = 1.4426950408889634f;

struct AttendArgs {
    const uint16_t* q;
    int64_t qs;
    int T;
    float scale;
    uint16_t* out;
    FastDiv group_div;
    float* partial;       // [grid][2] records: first and last piece of each CTA
    struct Split* split;  // [grid] the item that starts in a CTA and ends in another
};

// What a CTA leaves for the kernel that joins the pieces of an item: the last
// piece of CTA `from` and the first ones of the next pieces - 1. The CTA where
// the item starts leaves all rows to join or, if there are many pieces, the
// first one, and CTAs in the item's middle the others.
struct alignas(16) Split {
    int pieces;            // 0: none
    int from, row, rows;   // rows `row` to rows - 1
    int t0, head, tile;
};
constexpr int kJoinAhead = 5;  // pieces that a lane of k_join asks for at once
// Whether a block takes a row instead of a warp. (pieces - 2 CTAs are in the item's
// middle, and rows - 1 of them are needed.)
template <int D>
__device__ __forceinline__ bool many_pieces(int pieces, int rows) {
    return pieces > kJoinAhead * (128 / D) && pieces > rows;
}

// (q - 8) 2^-24 of the codes at bits 0-3 and 16-19, (q - 8) 2^-20 of those at 4-7 and 20-23, as fp16 pairs.
__device__ __forceinline__ uint32_t centred_lo(uint32_t w) {
    return h2_as_u32(__hadd2(u32_as_h2(w & 0x000f000fu), u32_as_h2(0x80088008u)));
}
__device__ __forceinline__ uint32_t centred_hi(uint32_t w) {
    return h2_as_u32(__hadd2(u32_as_h2(w & 0x00f000f0u), u32_as_h2(0x80808080u)));
}

// q - 8, or 16 (q - 8), of the codes at bits 0-3 and 16-19 as bf16 pairs: 128 + q
// is a bf16 with the code as its last bits.
__device__ __forceinline__ uint32_t centred_bf16(uint32_t w, float times) {
    const uint32_t u = (w & 0x000f000fu) | 0x43004300u;
    const __nv_bfloat162 r = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&u), __float2bfloat162_rn(times),
                                     __float2bfloat162_rn(-136.0f * times));
    return *reinterpret_cast<const uint32_t*>(&r);
}

// a / b for a >= 0, b > 0: nearly always both fit 32 bits, where a division
// takes a fraction of the 64-bit one's time.
__device__ __forceinline__ long long quotient(long long a, long long b) {
    if ((((unsigned long long)a | (unsigned long long)b) >> 32) == 0) return (unsigned)a / (unsigned)b;
    return a / b;
}

// What a sequence asks for. cells: of its context (one more than the table
// has where the length is past it, so that the missing page is met). end: the row
// after the sequence's last one, which sits at kv - 1, whether the call has all
// of the rows (t0 to t0 + n - 1) or not.
struct SeqWork {
    int t0, n, end, kv, cells, units, tiles, work;
};
template <int NT>
__device__ __forceinline__ SeqWork seq_work(const KvDev& c, const KvBatch& b, int T, int group, int seq) {
    SeqWork s;
    s.t0 = min(max(b.cu[seq], 0), T);
    s.end = b.cu[seq + 1];
    s.n = max(min(max(s.end, 0), T) - s.t0, 0);
    s.kv = b.kv_lens[seq];
    const long long cap = (long long)b.table_stride * c.page_tokens + 1;
    s.cells = (int)((unsigned)((int)min((long long)max(s.kv, 0), cap) + kCellTokens - 1) / kCellTokens);
    s.units = max(1, (s.cells + kWarps - 1) / kWarps);
    s.tiles = (s.n * group + 8 * NT - 1) / (8 * NT);
    s.work = (s.units + kBegin) * c.hkv * s.tiles;
    return s;
}

// A piece of an item: units [u0, u1) of (sequence, head, row tile); none (u0 ==
// u1) where the run ends in the item's idle units.
struct Piece {
    int seq, head, tile, u0, u1;
    SeqWork s;
    int first, next, prefix;  // numbers of the item's first unit, of the one after the piece, of the sequence's first
};

// The piece that starts at number x (x in seq's range), cut at `hi`.
__device__ __forceinline__ void piece_at(Piece& p, int x, int hi) {
    const int len = p.s.units + kBegin;
    const unsigned off = x - p.prefix, item = off / (unsigned)len;
    const int in = (int)(off - item * len), to = min(len, in + (hi - x));
    p.u0 = max(in - kBegin, 0);
    p.u1 = max(to - kBegin, 0);
    p.head = p.s.tiles == 1 ? (int)item : (int)(item / (unsigned)p.s.tiles);
    p.tile = (int)item - p.head * p.s.tiles;
    p.first = x - in + kBegin;
    p.next = x - in + to;
}
// Steps to the next piece; false at `hi`. Whole warps.
template <int NT>
__device__ __forceinline__ bool next_piece(Piece& p, int hi, const KvDev& c, const KvBatch& b, int T, int group, int lane) {
    const int x = p.next;
    if (x >= hi) return false;
    if (x >= p.prefix + p.s.work) {
        p.prefix += p.s.work;
        int s = p.seq + 1;
        for (;; s += 32) {  // the next sequence with new tokens: there is one, since x < hi
            const int e = min(s + lane, b.B - 1);
            const bool has = s + lane < b.B && min(max(b.cu[e + 1], 0), T) > min(max(b.cu[e], 0), T);
            const unsigned any = __ballot_sync(0xffffffffu, has);
            if (any) { s += __ffs(any) - 1; break; }
            if (s + 32 >= b.B) return false;
        }
        p.seq = s;
        p.s = seq_work<NT>(c, b, T, group, s);
    }
    piece_at(p, x, hi);
    return true;
}

// Cells of the piece that fall to warp w: (u0 + k) * kWarps + w, k below this.
__device__ __forceinline__ int warp_cells(const Piece& p, int w) {
    const int last = (p.s.cells - w + kWarps - 1) / kWarps;  // units in which the warp has a cell (cells >= 0)
    return max(0, min(p.u1, last) - p.u0);
}

template <int D, int NT>
struct AttSmem {
    static constexpr int kRows = 8 * NT, kPad = D + 4;
    alignas(128) uint8_t ring[kWarps][kStages][Cell<D>::kBytes];
    float o[kWarps][kRows][kPad];    // the warps' outputs
    float m[kWarps][kRows], l[kWarps][kRows];
    int wsum[kWarps];
    Piece cur[kWarps], ask[kWarps];  // a warp's piece at work and the one it asks for: rarely read, so not in registers
    int prefix, seq;
};

constexpr int kPartFloats(int D) { return 16 * D + 32; }  // output rows, then each row's maximum and sum

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
    return y;
}
// d = a b + c, c kept.
__device__ __forceinline__ void mma_f16_from(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, float c0, float c1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%10,%11};\n"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c0), "f"(c1));
}
// Transposes an 8 x 8 matrix of 16-bit values held two a lane (row lane / 4).
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(r) : "r"(v));
    return r;
}
__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) { return h2_as_u32(__floats2half2_rn(lo, hi)); }

// Four dims of a row's output: sums v of weights times values over the sum l of
// weights (m their maximum).
template <int D>
__device__ __forceinline__ void put_row(const KvDev& c, const AttendArgs& a, int t0, int head, int row, int d, float4 v, float m, float l) {
    const int group = c.hq / c.hkv, tok = a.group_div.div(row);
    const float inv = 1.0f / l;
    float x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = m == -INFINITY && l == 0.f ? 0.f : x[e] * inv;
    __nv_bfloat162 y0 = __floats2bfloat162_rn(x[0], x[1]), y1 = __floats2bfloat162_rn(x[2], x[3]);
    *reinterpret_cast<uint2*>(a.out + ((size_t)(t0 + tok) * c.hq + head * group + row - tok * group) * D + d) =
        make_uint2(*reinterpret_cast<uint32_t*>(&y0), *reinterpret_cast<uint32_t*>(&y1));
}

template <int D, int NT>
__global__ void __launch_bounds__(kAttThreads, NT == 1 ? 2 : 1) k_attend(KvDev c, KvBatch b, AttendArgs a) {
    constexpr int G = D / 32, kRows = 8 * NT;
    using C = Cell<D>;
    extern __shared__ uint8_t raw[];
    AttSmem<D, NT>& sm = *reinterpret_cast<AttSmem<D, NT>*>(raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, i = lane & 3;
    const int group = c.hq / c.hkv;

    griddep_wait();    // the batch's arrays, and the last call's records
    griddep_launch();  // k_join may be set up meanwhile
    // --- this CTA's run of units [lo, hi), and the sequence that lo falls in.
    // CTA x takes base units, the first `extra` CTAs one more.
    int total = 0, ctas = 0, base = 0, extra = 0, lo = 0, hi = 0, seq = -1, prefix = 0;
    auto share = [&]() {
        ctas = min(total, (int)gridDim.x);
        if ((int)blockIdx.x >= ctas) {
            if (tid == 0) a.split[blockIdx.x].pieces = 0;
            return false;
        }
        base = (unsigned)total / (unsigned)ctas;
        extra = total - base * ctas;
        lo = blockIdx.x * base + min((int)blockIdx.x, extra);
        hi = lo + base + ((int)blockIdx.x < extra);
        return true;
    };
    auto cta_of = [&](int x) {
        const int wide = extra * (base + 1);
        return x < wide ? (int)((unsigned)x / (unsigned)(base + 1)) : extra + (int)((unsigned)(x - wide) / (unsigned)base);
    };
    if (b.B <= 8 * 32) {
        // every warp by itself: a lane takes a few neighbouring sequences
        const int per = (b.B + 31) / 32, s0 = min(lane * per, b.B), s1 = min(s0 + per, b.B);
        int mine = 0;
        for (int s = s0; s < s1; ++s) mine += seq_work<NT>(c, b, a.T, group, s).work;
        int upto = mine;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, upto, off);
            if (lane >= off) upto += v;
        }
        total = __shfl_sync(0xffffffffu, upto, 31);
        if (!share()) return;
        const unsigned hit = __ballot_sync(0xffffffffu, lo < upto);
        const int l = __ffs(hit) - 1;
        seq = l * per;
        prefix = __shfl_sync(0xffffffffu, upto - mine, l);
        if (per > 1)
            for (;; ++seq) {
                const int w = seq_work<NT>(c, b, a.T, group, seq).work;
                if (lo < prefix + w) break;
                prefix += w;
            }
    } else {
        auto block_scan = [&](int w, int& incl, int& sum) {
            incl = w;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, incl, off);
                if (lane >= off) incl += v;
            }
            if (lane == 31) sm.wsum[warp] = incl;
            __syncthreads();
            sum = 0;
            int before = 0;
#pragma unroll
            for (int w2 = 0; w2 < kWarps; ++w2) {
                if (w2 == warp) before = sum;
                sum += sm.wsum[w2];
            }
            incl += before;
            __syncthreads();
        };
        int mine = 0, incl, sum, below = 0;
        for (int s = tid; s < b.B; s += kAttThreads) mine += seq_work<NT>(c, b, a.T, group, s).work;
        block_scan(mine, incl, total);
        if (!share()) return;
        for (int s0 = 0; s0 < b.B; s0 += kAttThreads) {
            const int s = s0 + tid, w = s < b.B ? seq_work<NT>(c, b, a.T, group, s).work : 0;
            block_scan(w, incl, sum);
            incl += below;
            if (incl - w <= lo && lo < incl) {
                sm.seq = s;
                sm.prefix = incl - w;
            }
            below += sum;
            if (below > lo) break;
        }
        __syncthreads();
        seq = sm.seq;
        prefix = sm.prefix;
    }

    // --- the warp's ring: sm.ask is the piece being asked for, sm.cur the one at work
    auto keep_piece = [&](Piece& to, const Piece& from) {
        __syncwarp();
        if (lane == 0) to = from;
        __syncwarp();
    };
    // steps a kept piece on; false (and the piece as it was) at the end of the run, an item's idle units among it
    auto step = [&](Piece& at) {
        Piece p = at;
        const bool there = next_piece<NT>(p, hi, c, b, a.T, group, lane) && p.u1 > p.u0;
        if (there) keep_piece(at, p);
        return there;
    };
    // row r of a piece's tile: new token and query head
    auto token_head = [&](const Piece& p, int r, int& tok, int& head) {
        const int row = p.tile * kRows + r;
        tok = a.group_div.div(row);
        head = p.head * group + row - tok * group;
    };
    auto rows_of = [&](const Piece& p) { return min(kRows, p.s.n * group - p.tile * kRows); };
    uint4 u[NT][G];  // this lane's part of q: row 8 nt + g, dims 32 bl + 8 i ..
    auto load_q = [&](const Piece& p) {
        const int rows = rows_of(p);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int r = g + 8 * nt;
            int tok, head;
            token_head(p, r < rows ? r : 0, tok, head);
            const uint16_t* src = a.q + (size_t)(p.s.t0 + tok) * a.qs + (size_t)head * D + 8 * i;
#pragma unroll
            for (int bl = 0; bl < G; ++bl) u[nt][bl] = *reinterpret_cast<const uint4*>(src + 32 * bl);
        }
    };
    int ask_n, ask_k = 0;
    {
        Piece p;
        p.seq = seq;
        p.prefix = prefix;
        p.s = seq_work<NT>(c, b, a.T, group, seq);
        piece_at(p, lo, hi);
        if (p.u1 == p.u0) {  // a run of idle units only
            if (tid == 0) a.split[blockIdx.x].pieces = 0;
            return;
        }
        load_q(p);
        ask_n = warp_cells(p, warp);
        keep_piece(sm.cur[warp], p);
        keep_piece(sm.ask[warp], p);
    }
    unsigned issued = 0, used = 0;
    bool more = true, split_here = false;
    const uint8_t* addr = nullptr;
    const uint32_t ring0 = (uint32_t)__cvta_generic_to_shared(sm.ring[warp][0]) + 16 * lane;
    // Copies the cell whose place lane `from` has into the ring.
    auto copy_cell = [&](int from, int slot) {
        const uint8_t* src = reinterpret_cast<const uint8_t*>(
            __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(addr), from));
        constexpr int kChunks = C::kBytes / 16;
        if (src) {
            const uint8_t* at = src + 16 * lane;
            const uint32_t to = ring0 + slot * C::kBytes;
#pragma unroll
            for (int e = 0; e < kChunks; e += 32)
                if (e + 32 <= kChunks || lane < kChunks - e)
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(to + 16 * e), "l"(at + 16 * e) : "memory");
        } else {  // no such page: its values are NaN
            if (lane == 0) atomicOr(c.err, 1u);
            uint8_t* dst = sm.ring[warp][slot];
            for (int e = lane; e < kChunks; e += 32) {
                const uint32_t w = e < C::kVs / 16 ? 0u : 0x7fff7fffu;
                *reinterpret_cast<uint4*>(dst + 16 * e) = make_uint4(w, w, w, w);
            }
        }
    };
    // Asks for the warp's next `want` cells, as far as there are some, and closes
    // the group of these copies. All groups but the last one hold all but the
    // last one or two of the ring's cells: a step waits for those.
    auto issue = [&](int want) {
        while (want > 0) {
            while (more && ask_k == ask_n) {
                more = step(sm.ask[warp]);
                ask_n = more ? warp_cells(sm.ask[warp], warp) : 0;
                ask_k = 0;
                if (more && warp == 0) {  // the next piece's q on its way to L2
                    const Piece& p = sm.ask[0];
                    const int r = lane / (D / 64);
                    if (r < rows_of(p)) {
                        int tok, head;
                        token_head(p, r, tok, head);
                        asm volatile("prefetch.global.L2 [%0];\n" ::"l"(
                            a.q + (size_t)(p.s.t0 + tok) * a.qs + (size_t)head * D + 64 * (lane % (D / 64))));
                    }
                }
            }
            if (!more) break;
            if ((ask_k & 31) == 0) {  // the next 32 cells' places
                const int k = ask_k + lane;
                const Piece& q = sm.ask[warp];
                addr = k < ask_n ? kv_cell<D>(c, b, q.seq, (q.u0 + k) * kWarps + warp, q.head) : nullptr;
            }
            copy_cell(ask_k & 31, issued % kStages);
            ++issued;
            ++ask_k;
            --want;
        }
        cp_async_commit();
    };
    issue(kStages / 2);
    issue(kStages / 2);

    for (bool first_piece = true;; first_piece = false) {
        if (!first_piece) {
            if (!step(sm.cur[warp])) break;
            load_q(sm.cur[warp]);
        }
        const Piece& p = sm.cur[warp];
        const int rows = rows_of(p);
        uint32_t qb[NT][G][2][2];        // B registers of the scores, row 8 nt + g: k-step, (b0, b1)
        float corr[NT][G][2];            // -8 sum(q) of rows 2i, 2i + 1, for codes of 2^-24
        float rf[NT][2];                 // scores to log2 units, rows 2i, 2i + 1
        int lim[NT][2], lim_row[NT];     // positions seen by rows 2i, 2i + 1, and by row g
        int min_lim = 0x7fffffff;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int r = g + 8 * nt;
            int tok, head;
            token_head(p, r < rows ? r : 0, tok, head);
            lim_row[nt] = p.s.kv - (p.s.end - p.s.t0) + tok + 1;
            min_lim = min(min_lim, lim_row[nt]);
            unsigned mx = 0;
#pragma unroll
            for (int bl = 0; bl < G; ++bl) {
                const uint4 w = u[nt][bl];
                mx = max(max(mx, bf16x2_absmax(w.x)), max(bf16x2_absmax(w.y), max(bf16x2_absmax(w.z), bf16x2_absmax(w.w))));
            }
            mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            const int sh = token_shift(mx);
            const float f = pow2f(-sh);
#pragma unroll
            for (int bl = 0; bl < G; ++bl) {
                const uint32_t w[4] = {u[nt][bl].x, u[nt][bl].y, u[nt][bl].z, u[nt][bl].w};
                float sum = 0.f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float x0 = __uint_as_float(w[j] << 16) * f, x1 = __uint_as_float(w[j] & 0xffff0000u) * f;
                    const float k = (j & 1) ? 0.0625f : 1.0f;  // the upper nibbles' codes are 16 times larger
                    const uint32_t h = pack_h2(x0 * k, x1 * k);
                    const float2 back = __half22float2(u32_as_h2(h));
                    sum += (back.x + back.y) * ((j & 1) ? 16.0f : 1.0f);
                    qb[nt][bl][j >> 1][j & 1] = h;
                }
                sum += __shfl_xor_sync(0xffffffffu, sum, 1);
                sum += __shfl_xor_sync(0xffffffffu, sum, 2);
                sum *= -8.0f / 16777216.0f;
#pragma unroll
                for (int e = 0; e < 2; ++e) corr[nt][bl][e] = __shfl_sync(0xffffffffu, sum, 8 * i + 4 * e);
            }
            // a scale of zero still hides what is hidden: -inf times a tiny factor is -inf
            const float fac = fmaxf(a.scale * kLog2e * 16777216.0f * pow2f(sh), 1e-37f);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                rf[nt][e] = __shfl_sync(0xffffffffu, fac, 8 * i + 4 * e);
                lim[nt][e] = __shfl_sync(0xffffffffu, lim_row[nt], 8 * i + 4 * e);
            }
        }
        min_lim = min(min_lim, __shfl_xor_sync(0xffffffffu, min_lim, 4));
        min_lim = min(min_lim, __shfl_xor_sync(0xffffffffu, min_lim, 8));
        min_lim = min(min_lim, __shfl_xor_sync(0xffffffffu, min_lim, 16));

        float o[G][2][NT][4] = {};   // c0, c1: dim 32 bl + 16 mu + g of rows 2i, 2i + 1; c2, c3: dim + 8, times 16
        float m[NT][2], l[NT][2];    // rows 2i, 2i + 1; l: this lane's tokens
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) m[nt][0] = m[nt][1] = -INFINITY, l[nt][0] = l[nt][1] = 0.f;
        unsigned far = 0;            // bit nt G + bl: row 8 nt + g's products in block bl are
        unsigned loud = 0;           // bit nt: row 8 nt + g has seen a scale of 2 or more

        const int cells = warp_cells(p, warp), first = (p.u0 * kWarps + warp) * kCellTokens;
        auto words = [&](uint32_t (&r)[G], const uint8_t* src) {
            if constexpr (G == 4) {
                const uint4 v = *reinterpret_cast<const uint4*>(src);
                r[0] = v.x, r[1] = v.y, r[2] = v.z, r[3] = v.w;
            } else {
                const uint2 v = *reinterpret_cast<const uint2*>(src);
                r[0] = v.x, r[1] = v.y;
            }
        };
        // The blocks of which row g sees small scales only in the warp's first step
        // (bits of `far`): of this lane's tokens, or of all.
        auto small_blocks = [&](const auto& vs, auto count, bool all) {
            unsigned bits = 0;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                uint32_t x[G] = {};
#pragma unroll
                for (int z = 0; z < decltype(count)::value; ++z)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int t = first + z * (kWarps * kCellTokens) + 8 * h + 2 * i;
                        const uint32_t sees = (t < lim_row[nt] ? 0x7fffu : 0u) | (t + 1 < lim_row[nt] ? 0x7fff0000u : 0u);
#pragma unroll
                        for (int bl = 0; bl < G; ++bl) x[bl] = __vmaxu2(x[bl], vs[z][h][bl] & sees);
                    }
#pragma unroll
                for (int bl = 0; bl < G; ++bl) {
                    uint32_t big = max(x[bl] & 0xffffu, x[bl] >> 16);
                    if (all) {
                        big = max(big, __shfl_xor_sync(0xffffffffu, big, 1));
                        big = max(big, __shfl_xor_sync(0xffffffffu, big, 2));
                    }
                    if (big - 1u < kQuiet - 1u) bits |= 1u << (nt * G + bl);  // not zero, and below
                }
            }
            return bits;
        };
        // Z cells, from the warp's k-th. Until a scale of 2 or more or a small block
        // is met, fp16 holds all products: then nothing is done, and the rest of the
        // piece goes by `wide` steps, which look at each product's range.
        auto cells_step = [&](int k, auto count, auto wide) {
            constexpr int Z = decltype(count)::value;
            constexpr bool kWide = decltype(wide)::value;
            // which of tokens 8h + 2i, + 1 of cell z row 8 nt + g sees
            auto sees = [&](int z, int nt, int h) {
                const int t = first + (k + z) * (kWarps * kCellTokens) + 8 * h + 2 * i;
                return (t < lim_row[nt] ? 0xffffu : 0u) | (t + 1 < lim_row[nt] ? 0xffff0000u : 0u);
            };
            float s[Z][NT][4];       // c0, c1: token g, rows 2i, 2i + 1; c2, c3: token g + 8
            uint32_t vs[Z][2][G];    // value scales
            uint32_t seen = 0;       // their bits
            cp_async_wait_but_last();
            __syncwarp();
#pragma unroll
            for (int z = 0; z < Z; ++z) {
                const uint8_t* cell = sm.ring[warp][(used + z) % kStages];
                uint32_t kw[2][G];
                __half2 ks[2][G / 2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    words(kw[h], cell + (h * 32 + lane) * G * 4);
                    words(vs[z][h], cell + C::kVs + (h * 4 + i) * G * 4);
                    if constexpr (G == 4) {
                        const uint2 v = *reinterpret_cast<const uint2*>(cell + C::kKs + (8 * h + g) * G * 2);
                        ks[h][0] = u32_as_h2(v.x), ks[h][1] = u32_as_h2(v.y);
                    } else {
                        ks[h][0] = *reinterpret_cast<const __half2*>(cell + C::kKs + (8 * h + g) * G * 2);
                    }
                }
#pragma unroll
                for (int bl = 0; bl < G; ++bl) {
                    const uint32_t w0 = kw[0][bl], w1 = kw[1][bl], w08 = w0 >> 8, w18 = w1 >> 8;
                    const uint32_t a0[4] = {w0 & 0x000f000fu, w1 & 0x000f000fu, w0 & 0x00f000f0u, w1 & 0x00f000f0u};
                    const uint32_t a1[4] = {w08 & 0x000f000fu, w18 & 0x000f000fu, w08 & 0x00f000f0u, w18 & 0x00f000f0u};
                    const float d0 = bl & 1 ? __high2float(ks[0][bl / 2]) : __low2float(ks[0][bl / 2]);
                    const float d1 = bl & 1 ? __high2float(ks[1][bl / 2]) : __low2float(ks[1][bl / 2]);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        float acc[4];
                        mma_f16_from(acc, a0, qb[nt][bl][0][0], qb[nt][bl][0][1], corr[nt][bl][0], corr[nt][bl][1]);
                        mma_f16(acc, a1, qb[nt][bl][1][0], qb[nt][bl][1][1]);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float d = e < 2 ? d0 : d1;
                            s[z][nt][e] = bl ? fmaf(acc[e], d, s[z][nt][e]) : acc[e] * d;
                        }
                    }
                    seen |= vs[z][0][bl] | vs[z][1][bl];
                }
                const int pos0 = first + (k + z) * (kWarps * kCellTokens);
                if (pos0 + kCellTokens > min_lim) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (pos0 + g + 8 * (e >> 1) >= lim[nt][e & 1]) s[z][nt][e] = -INFINITY;
                }
            }
            // Do the running maxima and fp16's range still do? A lane looks at its
            // own scores and scales; only if one does not are the maxima shared.
            // (A scale of 2 or more, and NaN, have the top exponent bit.)
            bool raise = !kWide && (seen & 0x40004000u) != 0;
            float mx[NT][2], lazy[NT][2];
            if constexpr (kWide) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int z = 0; z < Z; ++z)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            uint32_t any = 0;
#pragma unroll
                            for (int bl = 0; bl < G; ++bl) any |= vs[z][h][bl];
                            if (any & sees(z, nt, h) & 0x40004000u) loud |= 1u << nt;
                        }
                loud |= __shfl_xor_sync(0xffffffffu, loud, 1);
                loud |= __shfl_xor_sync(0xffffffffu, loud, 2);
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    lazy[nt][e] = kWide && (__shfl_sync(0xffffffffu, loud, 8 * i + 4 * e) >> nt & 1u) ? 0.f : kLazy;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float v = fmaxf(s[0][nt][e], s[0][nt][e + 2]);
                    if (Z == 2) v = fmaxf(v, fmaxf(s[Z - 1][nt][e], s[Z - 1][nt][e + 2]));
                    mx[nt][e] = rf[nt][e] * v;
                    raise |= mx[nt][e] > m[nt][e] + lazy[nt][e];
                }
            if (__any_sync(0xffffffffu, raise)) {
                if (kWide && k == 0) far = small_blocks(vs, count, true);
                if (!kWide && __any_sync(0xffffffffu, (seen & 0x40004000u) != 0 || (k == 0 && small_blocks(vs, count, false) != 0)))
                    return false;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float f[2];
#pragma unroll
                    for (int e2 = 0; e2 < 2; ++e2) {
                        float v = mx[nt][e2];
#pragma unroll
                        for (int off = 4; off < 32; off <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, off));
                        // raised where it is exceeded by enough, so that a row is raised by its own scores alone
                        v = v > m[nt][e2] + lazy[nt][e2] ? v : m[nt][e2];
                        f[e2] = v == m[nt][e2] ? 1.f : ex2(m[nt][e2] - v);
                        m[nt][e2] = v;
                        l[nt][e2] *= f[e2];
                    }
#pragma unroll
                    for (int bl = 0; bl < G; ++bl)
#pragma unroll
                        for (int mu = 0; mu < 2; ++mu)
#pragma unroll
                            for (int c4 = 0; c4 < 4; ++c4) o[bl][mu][nt][c4] *= f[c4 & 1];
                }
            }
            float mm[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) mm[nt][e] = (m[nt][e] == -INFINITY ? 0.f : m[nt][e]) - kOffset;
            // the weights of cell z for the values: row g, tokens 8h + 2i, + 1
            auto weights = [&](int z, uint32_t (&ph)[NT][2]) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float e0 = ex2(fmaf(s[z][nt][2 * h], rf[nt][0], -mm[nt][0]));
                        const float e1 = ex2(fmaf(s[z][nt][2 * h + 1], rf[nt][1], -mm[nt][1]));
                        l[nt][0] += e0;
                        l[nt][1] += e1;
                        ph[nt][h] = transpose8(pack_h2(e0, e1));
                    }
            };
            // values of cell z; `masked`: some row does not see all of it
            auto values = [&](int z, const uint32_t (&ph)[NT][2], auto masked) {
                const uint8_t* cell = sm.ring[warp][(used + z) % kStages];
                uint32_t vw[2][G];
                words(vw[0], cell + C::kV + lane * G * 4);
                words(vw[1], cell + C::kV + (32 + lane) * G * 4);
#pragma unroll
                for (int bl = 0; bl < G; ++bl) {
                    uint32_t pb[NT][2];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            pb[nt][h] = h2_as_u32(__hmul2(u32_as_h2(ph[nt][h]), u32_as_h2(vs[z][h][bl])));
                            if (decltype(masked)::value) pb[nt][h] &= sees(z, nt, h);  // a hidden token's scale may be NaN
                        }
                    const uint32_t w0 = vw[0][bl], w1 = vw[1][bl], w08 = w0 >> 8, w18 = w1 >> 8;
                    const uint32_t v0[4] = {centred_lo(w0), centred_hi(w0), centred_lo(w1), centred_hi(w1)};
                    const uint32_t v1[4] = {centred_lo(w08), centred_hi(w08), centred_lo(w18), centred_hi(w18)};
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        mma_f16(o[bl][0][nt], v0, pb[nt][0], pb[nt][1]);
                        mma_f16(o[bl][1][nt], v1, pb[nt][0], pb[nt][1]);
                    }
                }
            };
            // the same where some rows and blocks are far
            auto far_values = [&](int z, const uint32_t (&ph)[NT][2]) {
                const uint8_t* cell = sm.ring[warp][(used + z) % kStages];
                float pf[NT][4];  // the weights in fp32
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t e0 = __float_as_uint(ex2(fmaf(s[z][nt][2 * h], rf[nt][0], -mm[nt][0])));
                        const uint32_t e1 = __float_as_uint(ex2(fmaf(s[z][nt][2 * h + 1], rf[nt][1], -mm[nt][1])));
                        const uint32_t lo = transpose8(__byte_perm(e0, e1, 0x5410)), hi = transpose8(__byte_perm(e0, e1, 0x7632));
                        pf[nt][2 * h] = __uint_as_float(__byte_perm(lo, hi, 0x5410));
                        pf[nt][2 * h + 1] = __uint_as_float(__byte_perm(lo, hi, 0x7632));
                    }
                uint32_t vw[2][G];
                words(vw[0], cell + C::kV + lane * G * 4);
                words(vw[1], cell + C::kV + (32 + lane) * G * 4);
#pragma unroll
                for (int bl = 0; bl < G; ++bl) {
                    bool is_far = false, is_near = false;
                    uint32_t near[NT][2], hi[NT][2], lo[NT][2];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        const bool f = far & 1u << (nt * G + bl);
                        is_far |= f, is_near |= !f;
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const uint32_t scale = vs[z][h][bl] & sees(z, nt, h);  // a hidden token's may be NaN, or large
                            const float2 d = __half22float2(u32_as_h2(scale));
                            const float x0 = pf[nt][2 * h] * d.x * 0x1p-24f, x1 = pf[nt][2 * h + 1] * d.y * 0x1p-24f;
                            const __nv_bfloat162 b = __floats2bfloat162_rn(x0, x1);
                            const float2 back = __bfloat1622float2(b);
                            const __nv_bfloat162 rest = __floats2bfloat162_rn(x0 - back.x, x1 - back.y);
                            near[nt][h] = f ? 0u : h2_as_u32(__hmul2(u32_as_h2(ph[nt][h]), u32_as_h2(scale)));
                            hi[nt][h] = f ? *reinterpret_cast<const uint32_t*>(&b) : 0u;
                            lo[nt][h] = f ? *reinterpret_cast<const uint32_t*>(&rest) : 0u;
                        }
                    }
                    const uint32_t w0 = vw[0][bl], w1 = vw[1][bl], w08 = w0 >> 8, w18 = w1 >> 8;
                    if (__any_sync(0xffffffffu, is_near)) {
                        const uint32_t v0[4] = {centred_lo(w0), centred_hi(w0), centred_lo(w1), centred_hi(w1)};
                        const uint32_t v1[4] = {centred_lo(w08), centred_hi(w08), centred_lo(w18), centred_hi(w18)};
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            mma_f16(o[bl][0][nt], v0, near[nt][0], near[nt][1]);
                            mma_f16(o[bl][1][nt], v1, near[nt][0], near[nt][1]);
                        }
                    }
                    if (__any_sync(0xffffffffu, is_far)) {
                        const uint32_t v0[4] = {centred_bf16(w0, 1.f), centred_bf16(w0 >> 4, 16.f), centred_bf16(w1, 1.f),
                                                centred_bf16(w1 >> 4, 16.f)};
                        const uint32_t v1[4] = {centred_bf16(w08, 1.f), centred_bf16(w08 >> 4, 16.f), centred_bf16(w18, 1.f),
                                                centred_bf16(w18 >> 4, 16.f)};
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            mma_bf16(o[bl][0][nt], v0, hi[nt][0], hi[nt][1]);
                            mma_bf16(o[bl][1][nt], v1, hi[nt][0], hi[nt][1]);
                            mma_bf16(o[bl][0][nt], v0, lo[nt][0], lo[nt][1]);
                            mma_bf16(o[bl][1][nt], v1, lo[nt][0], lo[nt][1]);
                        }
                    }
                }
            };
            // the same by the products' range
            auto wide_values = [&](int z) {
                uint32_t ph[NT][2];
                weights(z, ph);
                unsigned over = 0;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int bl = 0; bl < G; ++bl) {
                        uint32_t x = 0;
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const uint32_t v = h2_as_u32(__hmul2(u32_as_h2(ph[nt][h]), u32_as_h2(vs[z][h][bl])));
                            x = __vmaxu2(x, v & sees(z, nt, h) & 0x7fff7fffu);
                        }
                        if ((x & 0xffffu) > kMost || (x >> 16) > kMost) over |= 1u << (nt * G + bl);
                    }
                over |= __shfl_xor_sync(0xffffffffu, over, 1);
                far |= over | __shfl_xor_sync(0xffffffffu, over, 2);
                if (__any_sync(0xffffffffu, far != 0)) far_values(z, ph);
                else values(z, ph, std::true_type{});
            };
            auto plain_values = [&](int z, auto masked) {
                uint32_t ph[NT][2];
                weights(z, ph);
                values(z, ph, masked);
            };
            if constexpr (kWide) {
#pragma unroll
                for (int z = 0; z < Z; ++z) wide_values(z);
            } else if (first + (k + Z - 1) * (kWarps * kCellTokens) + kCellTokens > min_lim) {
#pragma unroll
                for (int z = 0; z < Z; ++z) plain_values(z, std::true_type{});
            } else {
#pragma unroll
                for (int z = 0; z < Z; ++z) plain_values(z, std::false_type{});
            }
            used += Z;
            __syncwarp();  // every lane has read the slots
            const int at = ask_k & 31;
            if (at && at + Z <= 32 && ask_k + Z <= ask_n) {
#pragma unroll
                for (int z = 0; z < Z; ++z) copy_cell(at + z, (issued + z) % kStages);
                issued += Z;
                ask_k += Z;
                cp_async_commit();
            } else {
                issue(Z);
            }
            return true;
        };
        int k = 0;
        auto run = [&](auto wide) {
            bool did = true;
#pragma unroll 1
            for (; did && k + 1 < cells; k += did ? 2 : 0) did = cells_step(k, std::integral_constant<int, 2>{}, wide);
            if (did && k + 1 == cells && cells_step(k, std::integral_constant<int, 1>{}, wide)) ++k;
        };
        run(std::false_type{});
        if (k < cells) run(std::true_type{});

        // --- the warps' sums into one
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int off = 4; off < 32; off <<= 1) l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], off);
                if (g == 0) {
                    sm.m[warp][8 * nt + 2 * i + e] = m[nt][e];
                    sm.l[warp][8 * nt + 2 * i + e] = l[nt][e];
                }
            }
#pragma unroll
        for (int bl = 0; bl < G; ++bl)
#pragma unroll
            for (int mu = 0; mu < 2; ++mu)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        sm.o[warp][8 * nt + 2 * i + (e & 1)][32 * bl + 16 * mu + g + 8 * (e >> 1)] =
                            e < 2 ? o[bl][mu][nt][e] : o[bl][mu][nt][e] * 0.0625f;
        __syncthreads();

        // --- out, or to the item's other pieces
        const bool whole = p.u1 - p.u0 == p.s.units;
        float* rec = a.partial + ((size_t)blockIdx.x * 2 + (p.u0 == 0 ? 1 : 0)) * kPartFloats(D);
        for (int e = tid; e < rows * (D / 4); e += kAttThreads) {
            const int r = e / (D / 4), d = 4 * (e % (D / 4));
            float mm = -INFINITY, ll = 0.f;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, sm.m[w][r]);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float wm = sm.m[w][r], wl = sm.l[w][r];
                const float f = wm == -INFINITY ? 0.f : ex2(wm - mm), fu = f * 0x1p24f;  // of the codes
                const float4 x = *reinterpret_cast<const float4*>(&sm.o[w][r][d]);
                ll += f * wl;
                v.x = fmaf(fu, x.x, v.x), v.y = fmaf(fu, x.y, v.y), v.z = fmaf(fu, x.z, v.z), v.w = fmaf(fu, x.w, v.w);
            }
            if (whole) {
                put_row<D>(c, a, p.s.t0, p.head, p.tile * kRows + r, d, v, mm, ll);
            } else {
                __stcg(reinterpret_cast<float4*>(rec + r * D + d), v);
                if (d == 0) {
                    __stcg(reinterpret_cast<float2*>(rec + 16 * D + 2 * r), make_float2(mm, ll));
                }
            }
        }
        if (tid == 0 && p.u1 < p.s.units) {
            const int c0 = cta_of(p.first), c1 = cta_of(p.first + p.s.units - 1), row = (int)blockIdx.x - c0;
            const bool many = many_pieces<D>(c1 - c0 + 1, rows);
            if (row < (many ? rows : 1)) {
                a.split[blockIdx.x] = {c1 - c0 + 1, c0, row, many ? row + 1 : rows, p.s.t0, p.head, p.tile};
                split_here = true;
            }
        }
        __syncthreads();  // o, m and l are free again
    }
    if (tid == 0 && !split_here) a.split[blockIdx.x].pieces = 0;
}

// Joins the pieces of split items, as k_attend's CTA of the same number says: a
// warp takes a row of few pieces, a block one of many. A lane has four dims and
// asks for kJoinAhead pieces at once, each a trip to L2; more of them (8, 10) are
// fewer trips, but also more code, which a kernel this short fetches as it goes:
// one of 513 tokens 8.5 us (8.6, 8.9), one of 100003 25.0 (25.4, 24.5), 32 of up to
// 4095 19.8 (20.2, 20.3). One wave of blocks: with four for each CTA, a quarter of
// the rows each, the last two of these were 26.4 and 20.3 us.
template <int D, int NT>
__global__ void __launch_bounds__(256) k_join(KvDev c, AttendArgs a) {
    constexpr int kLanes = D / 4, kSide = 32 / kLanes;  // lanes of a row's dims; pieces a warp takes side by side
    __shared__ float4 part[8][kSide][kLanes];
    __shared__ float mpart[8][kSide], lpart[8][kSide];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, side = lane / kLanes, d = 4 * (lane % kLanes);
    griddep_wait();
    const int4* at = reinterpret_cast<const int4*>(a.split + blockIdx.x);
    const int4 s0 = __ldcg(at), s1 = __ldcg(at + 1);
    const Split s = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z};
    if (s.pieces == 0) return;
    const bool many = s.row + 1 == s.rows;  // one row: all warps take it (few pieces of a single row as well)
    const float* base = a.partial + (size_t)s.from * 2 * kPartFloats(D);
    const int set = (many ? warp * kSide : 0) + side, sets = many ? 8 * kSide : kSide;
    for (int r = many ? s.row : warp; r < s.rows; r += 8) {
        float m = -INFINITY, l = 0.f;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int q0 = set; q0 < s.pieces; q0 += kJoinAhead * sets) {
            float qm[kJoinAhead], ql[kJoinAhead], high = m;
            float4 x[kJoinAhead];
#pragma unroll
            for (int e = 0; e < kJoinAhead; ++e) {
                // (volatile: left alone, the compiler moves each load to its use, and each use waits)
                const int q = min(q0 + e * sets, s.pieces - 1);
                const float* rec = base + (unsigned)(2 * q + (q == 0)) * kPartFloats(D);
                asm volatile("ld.global.cg.v2.f32 {%0, %1}, [%2];\n" : "=f"(qm[e]), "=f"(ql[e]) : "l"(rec + 16 * D + 2 * r));
                asm volatile("ld.global.cg.v4.f32 {%0, %1, %2, %3}, [%4];\n"
                             : "=f"(x[e].x), "=f"(x[e].y), "=f"(x[e].z), "=f"(x[e].w)
                             : "l"(rec + r * D + d));
            }
#pragma unroll
            for (int e = 0; e < kJoinAhead; ++e) {
                if (q0 + e * sets >= s.pieces) qm[e] = -INFINITY;  // weight 0
                high = fmaxf(high, qm[e]);
            }
            const float f0 = m == high ? 1.f : ex2(m - high);
            m = high;
            l *= f0;
            v.x *= f0, v.y *= f0, v.z *= f0, v.w *= f0;
#pragma unroll
            for (int e = 0; e < kJoinAhead; ++e) {
                const float f = qm[e] == -INFINITY ? 0.f : ex2(qm[e] - m);
                l = fmaf(f, ql[e], l);
                v.x = fmaf(f, x[e].x, v.x), v.y = fmaf(f, x[e].y, v.y), v.z = fmaf(f, x[e].z, v.z), v.w = fmaf(f, x[e].w, v.w);
            }
        }
        if (sets > 1) {
            part[warp][side][lane % kLanes] = v;
            if (lane % kLanes == 0) mpart[warp][side] = m, lpart[warp][side] = l;
            if (many) __syncthreads();
            else __syncwarp();
            if (set == 0) {
                float high = m;
                for (int q = 1; q < sets; ++q) high = fmaxf(high, mpart[warp + q / kSide][q % kSide]);
                const float f0 = m == -INFINITY ? 0.f : ex2(m - high);
                l *= f0;
                v.x *= f0, v.y *= f0, v.z *= f0, v.w *= f0;
                for (int q = 1; q < sets; ++q) {
                    const float qm = mpart[warp + q / kSide][q % kSide], f = qm == -INFINITY ? 0.f : ex2(qm - high);
                    const float4 x = part[warp + q / kSide][q % kSide][lane % kLanes];
                    l = fmaf(f, lpart[warp + q / kSide][q % kSide], l);
                    v.x = fmaf(f, x.x, v.x), v.y = fmaf(f, x.y, v.y), v.z = fmaf(f, x.z, v.z), v.w = fmaf(f, x.w, v.w);
                }
                m = high;
            }
        }
        if (set == 0) put_row<D>(c, a, s.t0, s.head, s.tile * 8 * NT + r, d, v, m, l);
        if (many) break;
        __syncwarp();  // the sums are free again
    }
}

bool attend_fits(const KvDev& c, const KvBatch& b, int T) {
    const int64_t rows = (int64_t)T * (c.hq / c.hkv), tiles = rows / 8 + std::min<int64_t>(b.B, T);
    const int64_t units = ((int64_t)b.table_stride * c.page_tokens + 1) / (kCellTokens * kWarps) + 1;
    return rows < (1ll << 30) && (double)tiles * (double)(units + kBegin) * (double)c.hkv < (double)(1ll << 30);
}

int sm_count(int device) {
    static std::atomic<int> counts[kMaxDevices] = {};
    if (device < 0 || device >= kMaxDevices) return 152;
    int n = counts[device].load(std::memory_order_relaxed);
    if (!n) {
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, device) != cudaSuccess || n < 1) n = 152;
        counts[device].store(n, std::memory_order_relaxed);
    }
    return n;
}
static int max_grid(int device) { return std::min(2 * sm_count(device), kMaxCtas); }

// Partial records, then the split items.
uint64_t attend_scratch_bytes(int device) {
    return (uint64_t)max_grid(device) * (2 * kPartFloats(128) * sizeof(float) + sizeof(Split));
}

template <int D, int NT>
static cudaError_t launch(const KvDev& c, const KvBatch& b, const AttendArgs& a, int dev, int grid, cudaStream_t st) {
    static DeviceOnce once;
    const cudaError_t set = once.run(dev, [] {
        cudaError_t e = cudaFuncSetAttribute(k_attend<D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(AttSmem<D, NT>));
        // the same division of L1 and shared memory for both: an SM is idle while it changes
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(k_attend<D, NT>, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(k_join<D, NT>, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
        return e;
    });
    if (set != cudaSuccess) return set;
    const cudaError_t e = launch_ex(k_attend<D, NT>, dim3(grid), dim3(kAttThreads), sizeof(AttSmem<D, NT>), st, true, c, b, a);
    return e != cudaSuccess ? e : launch_ex(k_join<D, NT>, dim3(grid), dim3(256), 0, st, true, c, a);
}

cudaError_t launch_attend(const KvDev& c, const KvBatch& b, int D, const uint16_t* q, int64_t q_stride, int T, float scale,
                          uint16_t* out, void* scratch, cudaStream_t st) {
    int dev = 0;
    if (const cudaError_t e = cudaGetDevice(&dev); e != cudaSuccess) return e;
    const int n = max_grid(dev);
    AttendArgs a = {q, q_stride, T, scale, out, fast_div((uint32_t)(c.hq / c.hkv)), (float*)scratch,
                    (Split*)((uint8_t*)scratch + (size_t)n * 2 * kPartFloats(128) * sizeof(float))};
    // 16 rows at a time where a head has more than 8 in a step (its group times
    // the new tokens of an average sequence), although only half as many warps
    // fit: 8 streams of 4000 tokens, 4 new ones and 8 heads a group 23.1 us, 8
    // rows at a time 26.4. Not at head_dim 64, where a row's part is smaller: 7
    // streams of 5000-54000 tokens 60.2 and 57.8 us.
    const bool wide = D == 128 && (int64_t)(c.hq / c.hkv) * T > 8 * (int64_t)b.B;
    if (wide) return launch<128, 2>(c, b, a, dev, (n + 1) / 2, st);
    return D == 128 ? launch<128, 1>(c, b, a, dev, n, st) : launch<64, 1>(c, b, a, dev, n, st);
}

}  // namespace moe
