// kv.cuh -- the paged key/value cache in Q4_0 blocks: its layout, and the
// device helpers that its kernels share.
//
// Layout. A page of one layer is [kv_heads][page_tokens / 16] cells; a cell
// holds 16 tokens of one head, in the order in which the lanes of a warp hold
// the operands of mma.sync.m16n8k16, so that attention loads it with 16-byte
// reads and no shuffles. With G = head_dim / 32 blocks per token, lane l,
// g = l / 4 and i = l % 4, a cell is
//   K codes   words [16 tokens][4 i][G]    word (t, i, b): dims 32b + 8i + 2j (bits 4j) and + 1 (bits 16 + 4j)
//   K scales  fp16 [16 tokens][G]
//   V codes   words [2 halves][8 g][4 i][G]  dims 32b + g + 8j of tokens 8 half + 2i (bits 4j) and + 1 (bits 16 + 4j)
//   V scales  fp16x2 [2 halves][4 i][G]    tokens 8 half + 2i, + 1
// 576 G bytes, 18 per block. Every token owns whole 16-bit units, so tokens
// are written without reading their neighbours.
#pragma once

#include "common.cuh"
#include "device_policy.h"

namespace moe {

constexpr int kCellTokens = 16;

template <int D>
struct Cell {
    static constexpr int G = D / 32;
    static constexpr int kCodes = 256 * G, kScales = 32 * G;
    static constexpr int kKs = kCodes, kV = kCodes + kScales, kVs = kV + kCodes, kBytes = kVs + kScales;
    // byte offsets for token t of the cell
    __device__ static int k_word(int t, int i, int b) { return (t * 4 + i) * G * 4 + b * 4; }
    __device__ static int v_half(int t, int g, int b) {
        return (((t >> 3) * 32 + g * 4 + ((t & 7) >> 1)) * G + b) * 4 + (t & 1) * 2;
    }
    __device__ static int k_scale(int t, int b) { return (t * G + b) * 2; }
    __device__ static int v_scale(int t, int b) { return (((t >> 3) * 4 + ((t & 7) >> 1)) * G + b) * 4 + (t & 1) * 2; }
};

// Division of 0 <= x < 2^31 by a divisor fixed on the host (Granlund and
// Montgomery, Division by Invariant Integers using Multiplication, 1994): with
// 2^(l - 1) < d <= 2^l, x / d = (x + hi(x m)) / 2^l for m = 2^32 (2^l - d) / d + 1, rounded
// down.
struct FastDiv {
    uint32_t m, l;
    __device__ int div(int x) const { return (int)((__umulhi((uint32_t)x, m) + (uint32_t)x) >> l); }
};
inline FastDiv fast_div(uint32_t d) {
    uint32_t l = 0;
    while ((1u << l) < d) ++l;
    return {(uint32_t)((((uint64_t)1 << 32) * (((uint64_t)1 << l) - d)) / d + 1), l};
}

// What the kernels need of a handle and a batch, by value. They start before the
// kernel in front of them has ended (griddep_wait waits for it), and that one may
// write the batch's arrays, the rotation table and the queries: so all of these
// are read with ordinary loads, the read-only path being for what does not change
// while a kernel runs.
struct KvDev {
    uint8_t* pool;        // this layer's pages
    unsigned* err;        // sticky: 1 once a position or page was out of range
    uint64_t page_bytes;
    int num_pages, page_tokens, hq, hkv;
    FastDiv cells_div;    // by the cells of a page and head
};
struct KvBatch {
    const int *cu, *kv_lens, *table;
    int B, table_stride;
};

// Groups of neighbouring sequences that have their first positions in common, and
// what the kernels leave of a row's sum for the one that joins it: unnormalised
// outputs, each with a head: the exponent that its weights 2^(score - exponent) refer
// to, the sum of the weights, and two words. Of the common positions they are the first
// of the slots that go on with the sum, and their number with, above 16 bits, its row
// there. Of the rest the third word has the flags kWhole, kPieces and kCommon of
// kv_attend.cu; where the rest is in pieces there is no sum yet, and the first two words
// are the CTA of the first piece and their number, the fourth the row's place there.
struct KvGroups {
    const int *cu, *prefix;
    int n;
};
struct SharedParts {
    float *o, *slot_o, *rest_o;            // [T x q_heads], [CTAs x kSlotRows], [T x q_heads] rows of head_dim
    float4 *head, *slot_head, *rest_head;  // as many
    int* failed;                           // [CTAs] of launch_shared's kernel: whether a wait there gave up
    int slots;                             // CTAs
};
constexpr int kSlotRows = 256;

// The positions that a group has in common, as far as they are read for it as a
// whole: whole cells, held by its first sequence and in reach of its table.
__device__ __forceinline__ int common_tokens(const KvDev& c, const KvBatch& b, const KvGroups& g, int group) {
    const int first = g.cu[group];
    if ((unsigned)first >= (unsigned)b.B) return 0;
    const long long cap = (long long)b.table_stride * c.page_tokens;
    const int p = (int)min((long long)min(g.prefix[group], b.kv_lens[first]), cap);
    return max(p, 0) / kCellTokens * kCellTokens;
}
// The group of a sequence, or -1.
__device__ __forceinline__ int group_of_seq(const KvGroups& g, int seq) {
    if (seq < g.cu[0] || seq >= g.cu[g.n]) return -1;
    int lo = 0, hi = g.n;  // cu[lo] <= seq < cu[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (g.cu[mid] <= seq) lo = mid;
        else hi = mid;
    }
    return lo;
}

// Cell `n` of a sequence (positions 16 n ..) for head `head`, or null where the
// table or the pool has no such page.
template <int D>
__device__ __forceinline__ uint8_t* kv_cell(const KvDev& c, const KvBatch& b, int seq, int n, int head) {
    if (n < 0) return nullptr;
    const int pg = c.cells_div.div(n);
    if (pg >= b.table_stride) return nullptr;
    const int page = b.table[(size_t)seq * b.table_stride + pg];
    if ((unsigned)page >= (unsigned)c.num_pages) return nullptr;
    const int cells = c.page_tokens / kCellTokens, in = n - pg * cells;
    return c.pool + (size_t)page * c.page_bytes + (size_t)(head * cells + in) * Cell<D>::kBytes;
}

// The sequence of packed row t: the last b with cu[b] <= t, or -1 where t is
// before cu[0], or at or past cu[B].
__device__ __forceinline__ int seq_of_row(const int* cu, int B, int t) {
    if (t < cu[0] || t >= cu[B]) return -1;
    int lo = 0, hi = B;  // cu[lo] <= t < cu[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cu[mid] <= t) lo = mid;
        else hi = mid;
    }
    return lo;
}

// SMs of a device (asked for once; a GB300's where that fails).
int sm_count(int device);
// Device scratch of the attention kernel on `device`, zeroed once.
uint64_t attend_scratch_bytes(int device);
// Whether every piece of work of such a call can be numbered in 31 bits.
bool attend_fits(const KvDev& c, const KvBatch& b, int T);
cudaError_t launch_attend(const KvDev& c, const KvBatch& b, int D, const uint16_t* q, int64_t q_stride, int T, float scale,
                          uint16_t* out, void* scratch, cudaStream_t st);
// The same behind launch_shared: over what the groups do not have in common, and
// both joined.
cudaError_t launch_attend_rest(const KvDev& c, const KvBatch& b, const KvGroups& g, const SharedParts& parts, int D,
                               const uint16_t* q, int64_t q_stride, int T, float scale, uint16_t* out, void* scratch,
                               cudaStream_t st);

// Attention over what groups have in common (kv_shared.cu): the workspace of such a
// call and its parts, whether its work can be numbered in 31 bits, and the launch.
uint64_t shared_bytes(int device, int T, int hq, int D);
SharedParts shared_parts(void* workspace, int device, int T, int hq, int D);
bool shared_fits(const KvDev& c, const KvBatch& b, int groups, int T);
cudaError_t launch_shared(const KvDev& c, const KvBatch& b, const KvGroups& g, const SharedParts& parts, int D,
                          const uint16_t* q, int64_t q_stride, int T, float scale, cudaStream_t st);

}  // namespace moe
