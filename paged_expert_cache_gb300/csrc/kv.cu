// kv.cu -- the paged key/value cache: its handle and C entry points, the
// kernel that rotates and stores new tokens, and the one that reads tokens
// back.
#include <algorithm>
#include <new>

#include "kv.cuh"
#include "moe_cache.h"

namespace moe {

constexpr int kAppendThreads = 128;

struct AppendArgs {
    const uint16_t *q, *k, *v;
    int64_t qs, ks, vs;
    int T;
    const float* rope;
    int rope_rows;
    uint16_t *q_out, *k_out;
};

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&p);
}
__device__ __forceinline__ void unpack8(const uint4& u, float (&x)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) { x[2 * j] = bf16_lo(w[j]); x[2 * j + 1] = bf16_hi(w[j]); }
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
    return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
}

// One Q4_0 block held as 8 values in each of a quad's four lanes: this lane's
// eight codes (q - 8, as integers) and the block's scale.
__device__ __forceinline__ void quantise8(const float (&x)[8], int (&q)[8], __half& d) {
    float hi = x[0], lo = x[0];
    bool bad = false;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        hi = fmaxf(hi, x[e]);
        lo = fminf(lo, x[e]);
        bad |= !(fabsf(x[e]) <= 3.4028235e38f);
    }
#pragma unroll
    for (int off = 1; off < 4; off <<= 1) {
        hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, off));
        lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, off));
        bad |= __shfl_xor_sync(0xffffffffu, (int)bad, off) != 0;
    }
    const float m = hi >= -lo ? hi : lo;
    d = __float2half_rn(fminf(fmaxf(m * -0.125f, -65504.0f), 65504.0f));
    if (bad) d = __ushort_as_half(0x7fff);  // the block reads as NaN
    const float f = __half2float(d);
    const float inv = f == 0.0f || bad ? 0.0f : __frcp_rn(f);
    // rint(x / d) without a division for each value. x is a bf16 and d an fp16
    // value, so a quotient that is no tie n + 1/2 is at least 2^-16 away from
    // one (x - d (n + 1/2) is a whole number of units in 8 + 11 + 4 bits), while
    // x * inv is within 2^-20 of it: rounded to multiples of 2^-17 (the spacing
    // of fp32 about 96) ties become exact and nothing else does, and the second
    // rounding is the quotient's own, ties to even.
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float y = __fsub_rn(__fmaf_rn(x[e], inv, 96.0f), 96.0f);
        q[e] = __float2int_rn(bad ? 0.0f : fminf(fmaxf(y, -8.0f), 7.0f));
    }
}

// The position of packed row t, its sequence in `seq` (-1: none). In a decode
// step row t is sequence t's, so that is looked at first: one trip to memory
// instead of a search's several.
__device__ __forceinline__ int row_position(const KvBatch& b, int t, bool live, int& seq) {
    seq = -1;
    if (!live) return -1;
    const int guess = min(t, b.B - 1), c0 = b.cu[guess];
    int c1 = b.cu[guess + 1], len = b.kv_lens[guess];
    seq = guess;
    if (!(c0 <= t && t < c1)) {
        seq = seq_of_row(b.cu, b.B, t);
        if (seq < 0) return -1;
        c1 = b.cu[seq + 1];
        len = b.kv_lens[seq];
    }
    return len - (c1 - t);
}

// ---------------------------------------------------------------------------
// New tokens into the cache.
//
// A row is a head of a token; four lanes (a quad) hold one, lane i the dims 32b
// + 8i .. + 7 of every block b: whole rotation pairs, and a block across the
// quad. Warps of queries have one token and heads in steps of eight, so its
// rotation is read once; warps of keys or values have eight neighbouring tokens
// of one head, so a cell's bytes are written 16 at a time: a key row's words lie
// together, and a value word holds two neighbouring tokens, put together from
// two quads where both are in the warp.
//
// The kernel moves each value once (18 of 64 bytes for keys and values on the
// way to the cache); what bounds a prompt is the queries' bytes, what bounds a
// decode step is the launch and the chain batch -> position -> page. Measured in a
// graph: 13296 tokens of 64 query heads over 8, head_dim 64, 52.5 us (5.1 TB/s, three
// quarters of a copy's rate); 32 heads over 4, head_dim 128: 2451 tokens 10.6 us, one
// token 2.9.
// ---------------------------------------------------------------------------
template <int D>
struct RotaryRow {
    static constexpr int P = D / 64;  // blocks of the lower half
    float c[P][8], s[P][8];
    bool bad;
    __device__ void load(const AppendArgs& a, int pos, int i) {
        bad = pos < 0 || pos >= a.rope_rows;
        const float* row = a.rope + (size_t)(bad ? 0 : pos) * D + 8 * i;
#pragma unroll
        for (int b = 0; b < P; ++b)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float4 x = *reinterpret_cast<const float4*>(row + 32 * b + 4 * h);
                const float4 y = *reinterpret_cast<const float4*>(row + D / 2 + 32 * b + 4 * h);
                c[b][4 * h] = x.x, c[b][4 * h + 1] = x.y, c[b][4 * h + 2] = x.z, c[b][4 * h + 3] = x.w;
                s[b][4 * h] = y.x, s[b][4 * h + 1] = y.y, s[b][4 * h + 2] = y.z, s[b][4 * h + 3] = y.w;
            }
        if (bad) {
#pragma unroll
            for (int b = 0; b < P; ++b)
#pragma unroll
                for (int e = 0; e < 8; ++e) c[b][e] = s[b][e] = __int_as_float(0x7fc00000);
        }
    }
    // rotates a row; products and sum each rounded to fp32, as a program of
    // separate multiplies and adds computes them, then once to bf16
    __device__ void turn(uint4 (&u)[D / 32]) const {
#pragma unroll
        for (int b = 0; b < P; ++b) {
            float x[8], y[8];
            unpack8(u[b], x);
            unpack8(u[b + P], y);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float p = x[e], q = y[e];
                x[e] = __fsub_rn(__fmul_rn(p, c[b][e]), __fmul_rn(q, s[b][e]));
                y[e] = __fadd_rn(__fmul_rn(q, c[b][e]), __fmul_rn(p, s[b][e]));
            }
            u[b] = pack8(x);
            u[b + P] = pack8(y);
        }
    }
};

// HB: steps of eight heads that a warp of queries takes
template <int D, int HB>
__global__ void __launch_bounds__(kAppendThreads) k_kv_append(KvDev c, KvBatch b, AppendArgs a, int q_warps, int q_chunks) {
    constexpr int G = D / 32;
    using C = Cell<D>;
    const int tid = threadIdx.x, lane = tid & 31, quad = lane >> 2, i = lane & 3;
    const int w = blockIdx.x * (kAppendThreads / 32) + (tid >> 5);
    const bool is_q = w < q_warps;
    griddep_wait();
    griddep_launch();
    // --- the rows, asked for before anything about them is known
    int t, head;
    bool live, is_k = false;
    uint4 u[HB][G];
    if (is_q) {
        t = q_chunks == 1 ? w : (int)((unsigned)w / (unsigned)q_chunks);
        head = (w - t * q_chunks) * 8 * HB + quad;
        live = true;
#pragma unroll
        for (int e = 0; e < HB; ++e)
            if (head + 8 * e < c.hq) {
#pragma unroll
                for (int bl = 0; bl < G; ++bl)
                    u[e][bl] = __ldcs(reinterpret_cast<const uint4*>(a.q + (size_t)t * a.qs + (size_t)(head + 8 * e) * D + 32 * bl + 8 * i));
            }
    } else {
        const int v = w - q_warps, kv = (int)((unsigned)v / (unsigned)c.hkv);  // keys and values in turn
        head = v - kv * c.hkv;
        is_k = (kv & 1) == 0;
        t = (kv >> 1) * 8 + quad;
        live = t < a.T;
        const uint16_t* src = is_k ? a.k + (size_t)(live ? t : 0) * a.ks : a.v + (size_t)(live ? t : 0) * a.vs;
#pragma unroll
        for (int bl = 0; bl < G; ++bl)
            u[0][bl] = live ? __ldcs(reinterpret_cast<const uint4*>(src + (size_t)head * D + 32 * bl + 8 * i)) : make_uint4(0, 0, 0, 0);
    }
    if (!is_q && (w - q_warps) >= 2 * c.hkv * ((a.T + 7) / 8)) return;  // past the last warp of work
    int seq;
    const int pos = row_position(b, t, live, seq);
    RotaryRow<D> rot;
    if (a.rope && (is_q || is_k)) {
        rot.load(a, seq >= 0 ? pos : 0, i);
        if (seq >= 0 && rot.bad && i == 0) atomicOr(c.err, 1u);
    }
    if (is_q) {
        if (seq < 0) return;
#pragma unroll
        for (int e = 0; e < HB; ++e)
            if (head + 8 * e < c.hq) {
                if (a.rope) rot.turn(u[e]);
                uint16_t* dst = a.q_out + ((size_t)t * c.hq + head + 8 * e) * D + 8 * i;
#pragma unroll
                for (int bl = 0; bl < G; ++bl) *reinterpret_cast<uint4*>(dst + 32 * bl) = u[e][bl];
            }
        return;
    }
    if (is_k && a.rope) rot.turn(u[0]);
    if (is_k && a.k_out && seq >= 0) {
        uint16_t* dst = a.k_out + ((size_t)t * c.hkv + head) * D + 8 * i;
#pragma unroll
        for (int bl = 0; bl < G; ++bl) *reinterpret_cast<uint4*>(dst + 32 * bl) = u[0][bl];
    }
    uint8_t* cell = seq >= 0 ? kv_cell<D>(c, b, seq, pos >> 4, head) : nullptr;
    if (seq >= 0 && !cell && i == 0) atomicOr(c.err, 1u);
    const int tc = pos & (kCellTokens - 1);
    uint32_t code[G];    // keys: the word of each block; values: nibble e of dim 8i + e
    __half d[G];
#pragma unroll
    for (int bl = 0; bl < G; ++bl) {
        float x[8];
        int q[8];
        unpack8(u[0][bl], x);
        quantise8(x, q, d[bl]);
        uint32_t r = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) r |= (uint32_t)(q[e] + 8) << (is_k ? (e >> 1) * 4 + (e & 1) * 16 : 4 * e);
        code[bl] = r;
    }
    auto store_words = [&](uint8_t* to, const uint32_t (&x)[G]) {
        if constexpr (G == 4) *reinterpret_cast<uint4*>(to) = make_uint4(x[0], x[1], x[2], x[3]);
        else *reinterpret_cast<uint2*>(to) = make_uint2(x[0], x[1]);
    };
    uint32_t scale[G];  // this token's, in the low half
#pragma unroll
    for (int bl = 0; bl < G; ++bl) scale[bl] = __half_as_ushort(d[bl]);
    if (is_k) {
        if (!cell) return;
        store_words(cell + C::k_word(tc, i, 0), code);
        if (i == 0) {
            if constexpr (G == 4)
                *reinterpret_cast<uint2*>(cell + C::kKs + C::k_scale(tc, 0)) = make_uint2(scale[0] | scale[1] << 16, scale[2] | scale[3] << 16);
            else
                *reinterpret_cast<uint32_t*>(cell + C::kKs + C::k_scale(tc, 0)) = scale[0] | scale[1] << 16;
        }
        return;
    }
    // the neighbouring token of this one's value words, if its quad is here
    const bool odd = pos & 1;
    const int other = odd ? lane - 4 : lane + 4, from = other & 31;
    const bool pair = __shfl_sync(0xffffffffu, cell ? seq : -2, from) == seq && (unsigned)other < 32u && cell;
    uint32_t word[G], half[G], swap[G];
#pragma unroll
    for (int bl = 0; bl < G; ++bl) {
        uint32_t h = 0;  // dims g = 2i (low half) and 2i + 1 (high half), + 8j at nibble j
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t v = __shfl_sync(0xffffffffu, code[bl], (lane & 28) + j) >> (8 * i);
            h |= (v & 15u) << (4 * j) | ((v >> 4) & 15u) << (16 + 4 * j);
        }
        half[bl] = h;
        const uint32_t theirs = __shfl_sync(0xffffffffu, h, from);
        word[bl] = odd ? (theirs >> 16) | (h & 0xffff0000u) : (h & 0xffffu) | theirs << 16;
        swap[bl] = __shfl_sync(0xffffffffu, scale[bl], from);
    }
    if (!cell) return;
    uint8_t* vc = cell + C::kV;
    if (pair) {
        store_words(vc + C::v_half(tc & ~1, 2 * i + odd, 0), word);
        if (i == 0 && !odd) {
#pragma unroll
            for (int bl = 0; bl < G; ++bl) scale[bl] |= swap[bl] << 16;
            store_words(cell + C::kVs + C::v_scale(tc, 0), scale);
        }
    } else {
#pragma unroll
        for (int bl = 0; bl < G; ++bl) {
            *reinterpret_cast<uint16_t*>(vc + C::v_half(tc, 2 * i, bl)) = (uint16_t)half[bl];
            *reinterpret_cast<uint16_t*>(vc + C::v_half(tc, 2 * i + 1, bl)) = (uint16_t)(half[bl] >> 16);
            if (i == 0) *reinterpret_cast<uint16_t*>(cell + C::kVs + C::v_scale(tc, bl)) = (uint16_t)scale[bl];
        }
    }
}

template <int D>
static cudaError_t launch_append(const KvDev& d, const KvBatch& b, const AppendArgs& a, int device, cudaStream_t st) {
    const int hq = a.q ? d.hq : 0;
    const bool deep = append_takes_32_heads((int64_t)a.T * ((hq + 31) / 32), sm_count(device));
    const int chunk = deep ? 32 : 8, q_chunks = std::max((hq + chunk - 1) / chunk, 1);
    const int64_t q_warps = hq ? (int64_t)a.T * q_chunks : 0, warps = q_warps + 2 * (int64_t)d.hkv * ((a.T + 7) / 8);
    if (warps > 0x7ffffff0ll) return cudaErrorInvalidValue;
    const unsigned blocks = (unsigned)((warps + kAppendThreads / 32 - 1) / (kAppendThreads / 32));
    return launch_ex(deep ? k_kv_append<D, 4> : k_kv_append<D, 1>, dim3(blocks), dim3(kAppendThreads), 0, st, true, d, b, a,
                     (int)q_warps, q_chunks);
}

// ---------------------------------------------------------------------------
// Tokens of the cache back as bf16: a warp takes eight neighbouring rows of a
// head's keys or values, a quad each, as they were written. d * (q - 8) is exact
// in fp32 (11 + 4 bits), then rounded once. 13296 tokens of 8 heads, head_dim 64:
// 10.8 us in a graph (3.2 TB/s: few bytes for its start and its chain); one token 2.1.
// ---------------------------------------------------------------------------
template <int D>
__global__ void __launch_bounds__(kAppendThreads) k_kv_read(KvDev c, KvBatch b, int T, uint16_t* __restrict__ k_out,
                                                            uint16_t* __restrict__ v_out) {
    constexpr int G = D / 32;
    using C = Cell<D>;
    const int lane = threadIdx.x & 31, quad = lane >> 2, i = lane & 3;
    const int w = blockIdx.x * (kAppendThreads / 32) + (threadIdx.x >> 5);
    griddep_wait();
    griddep_launch();
    if (w >= 2 * c.hkv * ((T + 7) / 8)) return;
    const int kv = (int)((unsigned)w / (unsigned)c.hkv), head = w - kv * c.hkv, t = (kv >> 1) * 8 + quad;
    const bool is_k = (kv & 1) == 0;
    int seq;
    const int pos = row_position(b, t, t < T, seq);
    const uint8_t* cell = seq >= 0 ? kv_cell<D>(c, b, seq, pos >> 4, head) : nullptr;
    if (seq >= 0 && !cell && i == 0) atomicOr(c.err, 1u);
    const int tc = pos & (kCellTokens - 1);
    auto words = [&](uint32_t (&r)[G], const uint8_t* src) {
        if constexpr (G == 4) {
            const uint4 v = *reinterpret_cast<const uint4*>(src);
            r[0] = v.x, r[1] = v.y, r[2] = v.z, r[3] = v.w;
        } else {
            const uint2 v = *reinterpret_cast<const uint2*>(src);
            r[0] = v.x, r[1] = v.y;
        }
    };
    uint32_t code[G] = {};  // keys: the block's word; values: dims g = 2i (low half) and 2i + 1 (high half)
    float d[G];
#pragma unroll
    for (int bl = 0; bl < G; ++bl) d[bl] = __int_as_float(0x7fc00000);
    if (cell && is_k) {
        words(code, cell + C::k_word(tc, i, 0));
#pragma unroll
        for (int bl = 0; bl < G; ++bl) d[bl] = __half2float(*reinterpret_cast<const __half*>(cell + C::kKs + C::k_scale(tc, bl)));
    } else if (cell) {
        uint32_t lo[G], hi[G], sc[G];
        words(lo, cell + C::kV + C::v_half(tc & ~1, 2 * i, 0));
        words(hi, cell + C::kV + C::v_half(tc & ~1, 2 * i + 1, 0));
        words(sc, cell + C::kVs + C::v_scale(tc & ~1, 0));
        const int shift = 16 * (tc & 1);
#pragma unroll
        for (int bl = 0; bl < G; ++bl) {
            code[bl] = ((lo[bl] >> shift) & 0xffffu) | (hi[bl] >> shift) << 16;
            d[bl] = __half2float(__ushort_as_half((unsigned short)(sc[bl] >> shift)));
        }
    }
    uint16_t* dst = (is_k ? k_out : v_out) + ((size_t)t * c.hkv + head) * D + 8 * i;
#pragma unroll
    for (int bl = 0; bl < G; ++bl) {
        float x[8];
        if (is_k) {
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = (float)((code[bl] >> ((e >> 1) * 4 + (e & 1) * 16)) & 15u);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {  // dims 8i + 2j, + 1 are nibble i of lane j's halves
                const uint32_t v = __shfl_sync(0xffffffffu, code[bl], (lane & 28) + j) >> (4 * i);
                x[2 * j] = (float)(v & 15u);
                x[2 * j + 1] = (float)((v >> 16) & 15u);
            }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = d[bl] * (x[e] - 8.0f);
        if (seq >= 0) *reinterpret_cast<uint4*>(dst + 32 * bl) = pack8(x);
    }
}

}  // namespace moe

// ---------------------------------------------------------------------------
// The handle and the C entry points.
// ---------------------------------------------------------------------------
struct moe_kv {
    moe_kv_config_t cfg;
    uint64_t page_bytes, layer_bytes, scratch_bytes;
    uint8_t* pool;
    unsigned* err;
    void* scratch;
};

namespace {

struct CudaDevices {
    static cudaError_t get(int* device) { return cudaGetDevice(device); }
    static cudaError_t set(int device) { return cudaSetDevice(device); }
};
using DeviceScope = moe::DeviceScope<CudaDevices>;

moe_status_t refuse(const char* msg) {
    moe::set_last_error(msg);
    return MOE_ERR_INVALID;
}
moe_status_t cuda_refuse(cudaError_t e) {
    moe::set_last_error(cudaGetErrorString(e));
    return MOE_ERR_CUDA;
}

bool rows_ok(const void* p, int64_t stride, int heads, int dim) {
    return ((uintptr_t)p & 15u) == 0 && stride % 8 == 0 && stride >= (int64_t)heads * dim;
}

const char* batch_problem(const moe_kv_batch_t* b) {
    if (!b || !b->cu_tokens || !b->kv_lens || !b->block_table) return "NULL batch or batch array";
    if (b->num_seqs < 1 || b->table_stride < 1) return "num_seqs and table_stride must be >= 1";
    return nullptr;
}

// What is wrong with a call on the handle, or null.
const char* call_problem(const moe_kv_t* h, int32_t layer, int32_t T, const moe_kv_batch_t* b) {
    if (!h) return "handle is NULL";
    if (layer < 0 || layer >= h->cfg.num_layers) return "layer out of range";
    if (T < 0) return "T must be >= 0";
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess || dev != h->cfg.device) return "the handle's device is not the current one";
    return batch_problem(b);
}

moe::KvDev dev_of(const moe_kv_t* h, int layer) {
    moe::KvDev d;
    d.pool = h->pool + (size_t)layer * h->layer_bytes;
    d.err = h->err;
    d.page_bytes = h->page_bytes;
    d.num_pages = h->cfg.num_pages;
    d.page_tokens = h->cfg.page_tokens;
    d.hq = h->cfg.q_heads;
    d.hkv = h->cfg.kv_heads;
    d.cells_div = moe::fast_div((uint32_t)h->cfg.page_tokens / moe::kCellTokens);
    return d;
}
moe::KvBatch batch_of(const moe_kv_batch_t* b) {
    return {b->cu_tokens, b->kv_lens, b->block_table, b->num_seqs, b->table_stride};
}

}  // namespace

extern "C" {

void moe_kv_config_default(moe_kv_config_t* cfg) {
    if (!cfg) return;
    memset(cfg, 0, sizeof(*cfg));
    cfg->num_layers = 1;
    cfg->num_pages = 1;
    cfg->page_tokens = 64;
    cfg->q_heads = 1;
    cfg->kv_heads = 1;
    cfg->head_dim = 128;
}

moe_status_t moe_kv_create(const moe_kv_config_t* cfg, moe_kv_t** out) {
    if (!out) return refuse("out is NULL");
    *out = nullptr;
    if (!cfg) return refuse("cfg is NULL");
    const moe_kv_config_t& c = *cfg;
    if (c.num_layers < 1 || c.num_pages < 1) return refuse("num_layers and num_pages must be >= 1");
    if (c.page_tokens < 16 || c.page_tokens > 1024 || c.page_tokens % 16)
        return refuse("page_tokens must be a multiple of 16 in 16..1024");
    if (c.head_dim != 64 && c.head_dim != 128) return refuse("head_dim must be 64 or 128");
    if (c.kv_heads < 1 || c.kv_heads > 1024 || c.q_heads < 1 || c.q_heads % c.kv_heads || c.q_heads / c.kv_heads > 128)
        return refuse("kv_heads must be in 1..1024 and q_heads a multiple of it, at most 128 times");
    moe_kv_t* h = new (std::nothrow) moe_kv_t();
    if (!h) { moe::set_last_error("out of host memory"); return MOE_ERR_OOM; }
    h->cfg = c;
    h->page_bytes = (uint64_t)c.page_tokens * c.kv_heads * (c.head_dim / 32) * 36;
    h->layer_bytes = h->page_bytes * (uint64_t)c.num_pages;
    const uint64_t pool = h->layer_bytes <= (1ull << 40) / (uint64_t)c.num_layers ? h->layer_bytes * (uint64_t)c.num_layers : ~0ull;
    const DeviceScope scope(c.device);
    if (scope.status != cudaSuccess) { delete h; return cuda_refuse(scope.status); }
    h->scratch_bytes = moe::attend_scratch_bytes(c.device);
    void *p = nullptr, *s = nullptr;
    if (pool > (1ull << 40) || cudaMalloc(&p, pool) != cudaSuccess ||
        cudaMalloc(&s, h->scratch_bytes + 256) != cudaSuccess) {
        cudaGetLastError();
        cudaFree(p);
        delete h;
        moe::set_last_error("device allocation failed");
        return MOE_ERR_OOM;
    }
    h->pool = (uint8_t*)p;
    h->err = (unsigned*)s;
    h->scratch = (uint8_t*)s + 256;
    cudaError_t e = cudaMemset(p, 0, pool);
    if (e == cudaSuccess) e = cudaMemset(s, 0, h->scratch_bytes + 256);
    if (e == cudaSuccess) e = cudaDeviceSynchronize();
    if (e != cudaSuccess) {
        moe_kv_destroy(h);
        return cuda_refuse(e);
    }
    *out = h;
    return MOE_OK;
}

moe_status_t moe_kv_append(moe_kv_t* h, int32_t layer, const void* q, int64_t q_stride, const void* k,
                           int64_t k_stride, const void* v, int64_t v_stride, int32_t T,
                           const moe_kv_batch_t* batch, const float* rope, int32_t rope_rows, void* q_out,
                           void* k_out, void* stream) {
    if (const char* p = call_problem(h, layer, T, batch)) return refuse(p);
    const moe_kv_config_t& c = h->cfg;
    if (T == 0) return MOE_OK;
    if (!k || !v || (q && !q_out)) return refuse("NULL k, v or q_out");
    if ((q && !rows_ok(q, q_stride, c.q_heads, c.head_dim)) || !rows_ok(k, k_stride, c.kv_heads, c.head_dim) ||
        !rows_ok(v, v_stride, c.kv_heads, c.head_dim))
        return refuse("q, k and v need 16-byte aligned rows: strides multiples of 8 and not below heads * head_dim");
    if (((uintptr_t)q_out | (uintptr_t)k_out | (uintptr_t)rope) & 15u) return refuse("rope and outputs must be 16-byte aligned");
    if (rope && rope_rows < 1) return refuse("rope_rows must be >= 1");
    moe::AppendArgs a = {(const uint16_t*)q, (const uint16_t*)k, (const uint16_t*)v, q_stride, k_stride, v_stride, T,
                         rope, rope_rows, (uint16_t*)q_out, (uint16_t*)k_out};
    const moe::KvDev d = dev_of(h, layer);
    const cudaError_t e = c.head_dim == 128 ? moe::launch_append<128>(d, batch_of(batch), a, c.device, (cudaStream_t)stream)
                                            : moe::launch_append<64>(d, batch_of(batch), a, c.device, (cudaStream_t)stream);
    if (e == cudaErrorInvalidValue) return refuse("T is too large");
    return e == cudaSuccess ? MOE_OK : cuda_refuse(e);
}

moe_status_t moe_kv_attend(moe_kv_t* h, int32_t layer, const void* q, int64_t q_stride, int32_t T,
                           const moe_kv_batch_t* batch, float scale, void* out, void* stream) {
    if (const char* p = call_problem(h, layer, T, batch)) return refuse(p);
    const moe_kv_config_t& c = h->cfg;
    if (T == 0) return MOE_OK;
    if (!q || !out) return refuse("NULL q or out");
    if (!moe::attend_fits(dev_of(h, layer), batch_of(batch), T))
        return refuse("the batch is too large: more than 2^30 units of 128 cache tokens and 8 rows are possible");
    if (!(scale >= 0.f && scale <= 3.4028235e38f)) return refuse("scale must be finite and not negative");
    if (!rows_ok(q, q_stride, c.q_heads, c.head_dim) || ((uintptr_t)out & 15u))
        return refuse("q and out need 16-byte aligned rows: q_stride a multiple of 8 and not below q_heads * head_dim");
    const cudaError_t e = moe::launch_attend(dev_of(h, layer), batch_of(batch), c.head_dim, (const uint16_t*)q, q_stride, T,
                                             scale, (uint16_t*)out, h->scratch, (cudaStream_t)stream);
    return e == cudaSuccess ? MOE_OK : cuda_refuse(e);
}

moe_status_t moe_kv_shared_bytes(const moe_kv_t* h, int32_t T, uint64_t* bytes) {
    if (!h || !bytes) return refuse("NULL argument");
    if (T < 0) return refuse("T must be >= 0");
    *bytes = moe::shared_bytes(h->cfg.device, T, h->cfg.q_heads, h->cfg.head_dim);
    return MOE_OK;
}

moe_status_t moe_kv_attend_shared(moe_kv_t* h, int32_t layer, const void* q, int64_t q_stride, int32_t T,
                                  const moe_kv_batch_t* batch, const moe_kv_groups_t* groups, float scale, void* out,
                                  void* workspace, uint64_t workspace_bytes, void* stream) {
    if (const char* p = call_problem(h, layer, T, batch)) return refuse(p);
    const moe_kv_config_t& c = h->cfg;
    if (!groups || !groups->cu_seqs || !groups->prefix_lens || groups->num_groups < 1)
        return refuse("groups need at least one group, and neither array NULL");
    if (T == 0) return MOE_OK;
    if (!q || !out || !workspace) return refuse("NULL q, out or workspace");
    const moe::KvDev d = dev_of(h, layer);
    const moe::KvBatch b = batch_of(batch);
    if (!moe::attend_fits(d, b, T) || !moe::shared_fits(d, b, groups->num_groups, T))
        return refuse("the batch is too large: more than 2^30 units of 128 cache tokens and 8 rows are possible");
    if (!(scale >= 0.f && scale <= 3.4028235e38f)) return refuse("scale must be finite and not negative");
    if (!rows_ok(q, q_stride, c.q_heads, c.head_dim) || ((uintptr_t)out & 15u))
        return refuse("q and out need 16-byte aligned rows: q_stride a multiple of 8 and not below q_heads * head_dim");
    if ((uintptr_t)workspace & 255u) return refuse("the workspace must be 256-byte aligned");
    if (workspace_bytes < moe::shared_bytes(c.device, T, c.q_heads, c.head_dim))
        return refuse("the workspace is smaller than moe_kv_shared_bytes");
    if (!moe::sharing_pays((int64_t)T * (c.q_heads / c.kv_heads), b.B, (int64_t)b.table_stride * c.page_tokens, c.kv_heads, c.head_dim)) {
        const cudaError_t e = moe::launch_attend(d, b, c.head_dim, (const uint16_t*)q, q_stride, T, scale, (uint16_t*)out, h->scratch,
                                                 (cudaStream_t)stream);
        return e == cudaSuccess ? MOE_OK : cuda_refuse(e);
    }
    const moe::KvGroups g = {groups->cu_seqs, groups->prefix_lens, groups->num_groups};
    const moe::SharedParts parts = moe::shared_parts(workspace, c.device, T, c.q_heads, c.head_dim);
    cudaError_t e = moe::launch_shared(d, b, g, parts, c.head_dim, (const uint16_t*)q, q_stride, T, scale, (cudaStream_t)stream);
    if (e == cudaSuccess)
        e = moe::launch_attend_rest(d, b, g, parts, c.head_dim, (const uint16_t*)q, q_stride, T, scale, (uint16_t*)out,
                                    h->scratch, (cudaStream_t)stream);
    return e == cudaSuccess ? MOE_OK : cuda_refuse(e);
}

moe_status_t moe_kv_read(moe_kv_t* h, int32_t layer, int32_t T, const moe_kv_batch_t* batch, void* k_out,
                         void* v_out, void* stream) {
    if (const char* p = call_problem(h, layer, T, batch)) return refuse(p);
    const moe_kv_config_t& c = h->cfg;
    if (T == 0) return MOE_OK;
    if (!k_out || !v_out || (((uintptr_t)k_out | (uintptr_t)v_out) & 15u))
        return refuse("k_out and v_out must not be NULL, and 16-byte aligned");
    const uint64_t warps = 2 * (uint64_t)c.kv_heads * (((uint64_t)T + 7) / 8), per = moe::kAppendThreads / 32;
    if (warps > 0x7ffffff0ull) return refuse("T is too large");
    const uint64_t blocks = (warps + per - 1) / per;
    const cudaError_t e = moe::launch_ex(c.head_dim == 128 ? moe::k_kv_read<128> : moe::k_kv_read<64>, dim3((unsigned)blocks),
                                         dim3(moe::kAppendThreads), 0, (cudaStream_t)stream, true, dev_of(h, layer),
                                         batch_of(batch), T, (uint16_t*)k_out, (uint16_t*)v_out);
    return e == cudaSuccess ? MOE_OK : cuda_refuse(e);
}

moe_status_t moe_kv_info(const moe_kv_t* h, moe_kv_info_t* out) {
    if (!h || !out) return refuse("NULL argument");
    out->page_bytes = h->page_bytes;
    out->pool_device_bytes = h->layer_bytes * (uint64_t)h->cfg.num_layers;
    out->scratch_device_bytes = h->scratch_bytes + 256;
    return MOE_OK;
}

moe_status_t moe_kv_status(moe_kv_t* h) {
    if (!h) return refuse("handle is NULL");
    unsigned bits = 0;
    const DeviceScope scope(h->cfg.device);
    cudaError_t e = scope.status;
    if (e == cudaSuccess) e = cudaDeviceSynchronize();
    if (e == cudaSuccess) e = cudaMemcpy(&bits, h->err, sizeof bits, cudaMemcpyDeviceToHost);
    if (e == cudaSuccess && bits) e = cudaMemset(h->err, 0, sizeof bits);
    if (e != cudaSuccess) return cuda_refuse(e);
    if (bits) return refuse("a call met a position or page outside its tables");
    return MOE_OK;
}

moe_status_t moe_kv_destroy(moe_kv_t* h) {
    if (!h) return MOE_OK;
    const DeviceScope scope(h->cfg.device);
    cudaDeviceSynchronize();
    cudaFree(h->pool);
    cudaFree(h->err);
    delete h;
    return MOE_OK;
}

}  // extern "C"
