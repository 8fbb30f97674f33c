// kv.cu -- the paged key/value cache: its handle and C entry points, the
// kernel that rotates and stores new tokens, and the one that reads tokens
// back.
#include <new>

#include "kv.cuh"
#include "moe_cache.h"

namespace moe {

constexpr int kAppendThreads = 256;
constexpr int kCuShared = 1024;  // batches up to this many sequences are searched in shared memory

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

// One Q4_0 block held as 8 values in each of four neighbouring lanes: this
// lane's eight codes (nibble e is value e) and the block's scale.
__device__ __forceinline__ uint32_t quantise8(const float (&x)[8], __half& d) {
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
    uint32_t w = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        // the quotient of a bf16 value and an fp16 scale is never within an
        // fp32 rounding of a tie it does not hit, so this is the exact rounding
        const float r = f == 0.0f || bad ? 0.0f : rintf(__fdiv_rn(x[e], f));
        w |= (uint32_t)(int)(fminf(fmaxf(r, -8.0f), 7.0f) + 8.0f) << (4 * e);
    }
    return w;
}

// nibbles 0..7 -> the word of a K cell: nibble 2j at bits 4j, 2j + 1 at 16 + 4j
__device__ __forceinline__ uint32_t spread_pairs(uint32_t w) {
    uint32_t r = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) r |= ((w >> (8 * j)) & 15u) << (4 * j) | ((w >> (8 * j + 4)) & 15u) << (16 + 4 * j);
    return r;
}

// ---------------------------------------------------------------------------
// New tokens into the cache.
//
// One row (a head of q, k or v of a token) is D / 16 lanes: lane c holds
// dims 8c .. 8c + 7 and the same of the upper half, which are whole rotation
// pairs, and four neighbouring lanes hold one Q4_0 block of each half. The
// kernel moves each value once (18 of 32 bytes for k and v on the way out);
// what bounds a prompt is the q rows' bytes, what bounds a decode step is the
// launch and the chain batch -> position -> page.
// ---------------------------------------------------------------------------
template <int D>
__global__ void __launch_bounds__(kAppendThreads) k_kv_append(KvDev c, KvBatch b, AppendArgs a) {
    constexpr int kLanes = D / 16, G = D / 32;
    __shared__ int cu_s[kCuShared + 1];
    const int tid = threadIdx.x;
    const int rows = (a.q ? c.hq : 0) + 2 * c.hkv;
    const unsigned long long item = (unsigned long long)blockIdx.x * (kAppendThreads / kLanes) + tid / kLanes;
    const int lane = tid % kLanes;
    const unsigned long long total = (unsigned long long)a.T * rows;
    const bool live = item < total;
    const int t = !live ? 0 : total <= 0xffffffffull ? (int)((unsigned)item / (unsigned)rows) : (int)(item / rows);
    int r = live ? (int)(item - (unsigned long long)t * rows) : 0;
    int kind = 2, head;  // 0 q, 1 k, 2 v
    if (!a.q) r += c.hq;
    if (r < c.hq) { kind = 0; head = r; }
    else if (r < c.hq + c.hkv) { kind = 1; head = r - c.hq; }
    else head = r - c.hq - c.hkv;
    uint4 ua = make_uint4(0, 0, 0, 0), ub = ua;
    if (live) {
        const uint16_t* src = kind == 0 ? a.q + (size_t)t * a.qs : kind == 1 ? a.k + (size_t)t * a.ks : a.v + (size_t)t * a.vs;
        src += (size_t)head * D + 8 * lane;
        ua = *reinterpret_cast<const uint4*>(src);
        ub = *reinterpret_cast<const uint4*>(src + D / 2);
    }
    const int* cu = b.cu;
    if (b.B <= kCuShared) {
        for (int i = tid; i <= b.B; i += kAppendThreads) cu_s[i] = __ldg(b.cu + i);
        cu = cu_s;
        __syncthreads();
    }
    const int seq = live ? seq_of_row(cu, b.B, t) : -1;
    const int pos = seq >= 0 ? __ldg(b.kv_lens + seq) - (cu[seq + 1] - t) : -1;
    float x[8], y[8];
    unpack8(ua, x);
    unpack8(ub, y);
    bool bad = false;
    if (kind != 2) {
        if (a.rope && seq >= 0) {
            bad = pos < 0 || pos >= a.rope_rows;
            const float4* row = reinterpret_cast<const float4*>(a.rope + (size_t)(bad ? 0 : pos) * D) + 2 * lane;
            const float4 c0 = __ldg(row), c1 = __ldg(row + 1), s0 = __ldg(row + D / 8), s1 = __ldg(row + D / 8 + 1);
            const float cs[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
            const float sn[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                // products and sum each rounded to fp32, as a program of
                // separate multiplies and adds computes them
                const float u = x[e], w = y[e];
                x[e] = __fsub_rn(__fmul_rn(u, cs[e]), __fmul_rn(w, sn[e]));
                y[e] = __fadd_rn(__fmul_rn(w, cs[e]), __fmul_rn(u, sn[e]));
                if (bad) x[e] = y[e] = __int_as_float(0x7fc00000);
            }
            ua = pack8(x);
            ub = pack8(y);
        }
        uint16_t* dst = kind == 0 ? a.q_out : a.k_out;
        if (seq >= 0 && dst) {
            dst += ((size_t)t * (kind == 0 ? c.hq : c.hkv) + head) * D + 8 * lane;
            *reinterpret_cast<uint4*>(dst) = ua;
            *reinterpret_cast<uint4*>(dst + D / 2) = ub;
        }
        unpack8(ua, x);  // the block holds the rounded key
        unpack8(ub, y);
    }
    if (!__any_sync(0xffffffffu, kind != 0)) {  // a warp of q rows is done
        if (bad) atomicOr(c.err, 1u);
        return;
    }
    __half d0, d1;
    const uint32_t w0 = quantise8(x, d0), w1 = quantise8(y, d1);
    uint8_t* cell = seq >= 0 && kind != 0 ? kv_cell<D>(c, b, seq, pos >> 4, head) : nullptr;
    bad |= seq >= 0 && kind != 0 && !cell;
    if (bad) atomicOr(c.err, 1u);
    const int tc = pos & (kCellTokens - 1), i = lane & 3, b0 = lane >> 2, b1 = b0 + G / 2;
    // v: the four lanes' words, of which this lane stores dims g = 2i, 2i + 1 (+ 8j)
    uint32_t h0 = 0, h1 = 0;  // halfwords of g = 2i (low) and 2i + 1 (high)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int from = (threadIdx.x & 28) + j;
        const uint32_t v0 = __shfl_sync(0xffffffffu, w0, from) >> (8 * i), v1 = __shfl_sync(0xffffffffu, w1, from) >> (8 * i);
        h0 |= (v0 & 15u) << (4 * j) | ((v0 >> 4) & 15u) << (16 + 4 * j);
        h1 |= (v1 & 15u) << (4 * j) | ((v1 >> 4) & 15u) << (16 + 4 * j);
    }
    if (!cell) return;
    using C = Cell<D>;
    if (kind == 1) {
        *reinterpret_cast<uint32_t*>(cell + C::k_word(tc, i, b0)) = spread_pairs(w0);
        *reinterpret_cast<uint32_t*>(cell + C::k_word(tc, i, b1)) = spread_pairs(w1);
    } else {
        uint8_t* vc = cell + C::kV;
        *reinterpret_cast<uint16_t*>(vc + C::v_half(tc, 2 * i, b0)) = (uint16_t)h0;
        *reinterpret_cast<uint16_t*>(vc + C::v_half(tc, 2 * i + 1, b0)) = (uint16_t)(h0 >> 16);
        *reinterpret_cast<uint16_t*>(vc + C::v_half(tc, 2 * i, b1)) = (uint16_t)h1;
        *reinterpret_cast<uint16_t*>(vc + C::v_half(tc, 2 * i + 1, b1)) = (uint16_t)(h1 >> 16);
    }
    if (i == 0) {
        *reinterpret_cast<__half*>(cell + (kind == 1 ? C::kKs + C::k_scale(tc, b0) : C::kVs + C::v_scale(tc, b0))) = d0;
        *reinterpret_cast<__half*>(cell + (kind == 1 ? C::kKs + C::k_scale(tc, b1) : C::kVs + C::v_scale(tc, b1))) = d1;
    }
}

// ---------------------------------------------------------------------------
// Tokens of the cache back as bf16: the same rows and lanes, the other way.
// d * (q - 8) is exact in fp32 (11 + 4 bits), then rounded once.
// ---------------------------------------------------------------------------
template <int D>
__global__ void __launch_bounds__(kAppendThreads) k_kv_read(KvDev c, KvBatch b, int T, uint16_t* __restrict__ k_out,
                                                            uint16_t* __restrict__ v_out) {
    constexpr int kLanes = D / 16, G = D / 32;
    using C = Cell<D>;
    __shared__ int cu_s[kCuShared + 1];
    const int tid = threadIdx.x;
    const int rows = 2 * c.hkv;
    const unsigned long long item = (unsigned long long)blockIdx.x * (kAppendThreads / kLanes) + tid / kLanes;
    const int lane = tid % kLanes;
    const unsigned long long total = (unsigned long long)T * rows;
    const bool live = item < total;
    const int t = !live ? 0 : total <= 0xffffffffull ? (int)((unsigned)item / (unsigned)rows) : (int)(item / rows);
    int head = live ? (int)(item - (unsigned long long)t * rows) : 0;
    const bool is_v = head >= c.hkv;
    if (is_v) head -= c.hkv;
    const int* cu = b.cu;
    if (b.B <= kCuShared) {
        for (int i = tid; i <= b.B; i += kAppendThreads) cu_s[i] = __ldg(b.cu + i);
        cu = cu_s;
        __syncthreads();
    }
    const int seq = live ? seq_of_row(cu, b.B, t) : -1;
    const int pos = seq >= 0 ? __ldg(b.kv_lens + seq) - (cu[seq + 1] - t) : -1;
    const uint8_t* cell = seq >= 0 ? kv_cell<D>(c, b, seq, pos >> 4, head) : nullptr;
    if (seq >= 0 && !cell) atomicOr(c.err, 1u);
    const int tc = pos & (kCellTokens - 1), i = lane & 3, b0 = lane >> 2, b1 = b0 + G / 2;
    uint32_t w0 = 0, w1 = 0;  // nibble e: dim 8i + e of the block
    float d0 = __int_as_float(0x7fc00000), d1 = d0;
    if (cell) {
        d0 = __half2float(*reinterpret_cast<const __half*>(cell + (is_v ? C::kVs + C::v_scale(tc, b0) : C::kKs + C::k_scale(tc, b0))));
        d1 = __half2float(*reinterpret_cast<const __half*>(cell + (is_v ? C::kVs + C::v_scale(tc, b1) : C::kKs + C::k_scale(tc, b1))));
        if (!is_v) {
            const uint32_t u0 = *reinterpret_cast<const uint32_t*>(cell + C::k_word(tc, i, b0));
            const uint32_t u1 = *reinterpret_cast<const uint32_t*>(cell + C::k_word(tc, i, b1));
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                w0 |= ((u0 >> (4 * j)) & 15u) << (8 * j) | ((u0 >> (16 + 4 * j)) & 15u) << (8 * j + 4);
                w1 |= ((u1 >> (4 * j)) & 15u) << (8 * j) | ((u1 >> (16 + 4 * j)) & 15u) << (8 * j + 4);
            }
        } else {
            const uint8_t* vc = cell + C::kV;
            w0 = *reinterpret_cast<const uint16_t*>(vc + C::v_half(tc, 2 * i, b0)) |
                 (uint32_t)*reinterpret_cast<const uint16_t*>(vc + C::v_half(tc, 2 * i + 1, b0)) << 16;
            w1 = *reinterpret_cast<const uint16_t*>(vc + C::v_half(tc, 2 * i, b1)) |
                 (uint32_t)*reinterpret_cast<const uint16_t*>(vc + C::v_half(tc, 2 * i + 1, b1)) << 16;
        }
    }
    // v: lane j of the quad holds dims g = 2j, 2j + 1 (+ 8i'); gather dims 8i + g
    uint32_t g0 = 0, g1 = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int from = (threadIdx.x & 28) + j;
        const uint32_t v0 = __shfl_sync(0xffffffffu, w0, from) >> (4 * i), v1 = __shfl_sync(0xffffffffu, w1, from) >> (4 * i);
        g0 |= (v0 & 15u) << (8 * j) | ((v0 >> 16) & 15u) << (8 * j + 4);
        g1 |= (v1 & 15u) << (8 * j) | ((v1 >> 16) & 15u) << (8 * j + 4);
    }
    if (is_v) { w0 = g0; w1 = g1; }
    if (seq < 0) return;
    float x[8], y[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        x[e] = d0 * ((float)((w0 >> (4 * e)) & 15u) - 8.0f);
        y[e] = d1 * ((float)((w1 >> (4 * e)) & 15u) - 8.0f);
    }
    uint16_t* dst = (is_v ? v_out : k_out) + ((size_t)t * c.hkv + head) * D + 8 * lane;
    *reinterpret_cast<uint4*>(dst) = pack8(x);
    *reinterpret_cast<uint4*>(dst + D / 2) = pack8(y);
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
    const uint64_t pool = h->layer_bytes * (uint64_t)c.num_layers;
    if (cudaError_t e = cudaSetDevice(c.device); e != cudaSuccess) { delete h; return cuda_refuse(e); }
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
    if (!h) return refuse("handle is NULL");
    const moe_kv_config_t& c = h->cfg;
    if (layer < 0 || layer >= c.num_layers) return refuse("layer out of range");
    if (T < 0) return refuse("T must be >= 0");
    if (const char* p = batch_problem(batch)) return refuse(p);
    if (T == 0) return MOE_OK;
    if (!k || !v || (q && !q_out)) return refuse("NULL k, v or q_out");
    if ((q && !rows_ok(q, q_stride, c.q_heads, c.head_dim)) || !rows_ok(k, k_stride, c.kv_heads, c.head_dim) ||
        !rows_ok(v, v_stride, c.kv_heads, c.head_dim))
        return refuse("q, k and v need 16-byte aligned rows: strides multiples of 8 and not below heads * head_dim");
    if (((uintptr_t)q_out | (uintptr_t)k_out | (uintptr_t)rope) & 15u) return refuse("rope and outputs must be 16-byte aligned");
    if (rope && rope_rows < 1) return refuse("rope_rows must be >= 1");
    moe::AppendArgs a = {(const uint16_t*)q, (const uint16_t*)k, (const uint16_t*)v, q_stride, k_stride, v_stride, T,
                         rope, rope_rows, (uint16_t*)q_out, (uint16_t*)k_out};
    const uint64_t items = (uint64_t)T * ((q ? c.q_heads : 0) + 2 * c.kv_heads);
    const uint64_t per = moe::kAppendThreads / (c.head_dim / 16), blocks = (items + per - 1) / per;
    if (blocks > 0x7fffffffull) return refuse("T is too large");
    const moe::KvDev d = dev_of(h, layer);
    if (c.head_dim == 128)
        moe::k_kv_append<128><<<(unsigned)blocks, moe::kAppendThreads, 0, (cudaStream_t)stream>>>(d, batch_of(batch), a);
    else
        moe::k_kv_append<64><<<(unsigned)blocks, moe::kAppendThreads, 0, (cudaStream_t)stream>>>(d, batch_of(batch), a);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? MOE_OK : cuda_refuse(e);
}

moe_status_t moe_kv_attend(moe_kv_t* h, int32_t layer, const void* q, int64_t q_stride, int32_t T,
                           const moe_kv_batch_t* batch, float scale, void* out, void* stream) {
    if (!h) return refuse("handle is NULL");
    const moe_kv_config_t& c = h->cfg;
    if (layer < 0 || layer >= c.num_layers) return refuse("layer out of range");
    if (T < 0) return refuse("T must be >= 0");
    if (const char* p = batch_problem(batch)) return refuse(p);
    if (T == 0) return MOE_OK;
    if (!q || !out) return refuse("NULL q or out");
    if (!moe::attend_fits(dev_of(h, layer), batch_of(batch), T))
        return refuse("the batch is too large: more than 2^30 units of 128 cache tokens and 8 rows are possible");
    if (!(scale >= 0.f && scale <= 3.4028235e38f)) return refuse("scale must be finite and not negative");
    if (!rows_ok(q, q_stride, c.q_heads, c.head_dim) || ((uintptr_t)out & 15u))
        return refuse("q and out need 16-byte aligned rows: q_stride a multiple of 8 and not below q_heads * head_dim");
    moe::launch_attend(dev_of(h, layer), batch_of(batch), c.head_dim, (const uint16_t*)q, q_stride, T, scale,
                       (uint16_t*)out, h->scratch, (cudaStream_t)stream);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? MOE_OK : cuda_refuse(e);
}

moe_status_t moe_kv_read(moe_kv_t* h, int32_t layer, int32_t T, const moe_kv_batch_t* batch, void* k_out,
                         void* v_out, void* stream) {
    if (!h) return refuse("handle is NULL");
    const moe_kv_config_t& c = h->cfg;
    if (layer < 0 || layer >= c.num_layers) return refuse("layer out of range");
    if (T < 0) return refuse("T must be >= 0");
    if (const char* p = batch_problem(batch)) return refuse(p);
    if (T == 0) return MOE_OK;
    if (!k_out || !v_out || (((uintptr_t)k_out | (uintptr_t)v_out) & 15u))
        return refuse("k_out and v_out must not be NULL, and 16-byte aligned");
    const uint64_t items = (uint64_t)T * 2 * c.kv_heads;
    const uint64_t per = moe::kAppendThreads / (c.head_dim / 16), blocks = (items + per - 1) / per;
    if (blocks > 0x7fffffffull) return refuse("T is too large");
    const moe::KvDev d = dev_of(h, layer);
    if (c.head_dim == 128)
        moe::k_kv_read<128><<<(unsigned)blocks, moe::kAppendThreads, 0, (cudaStream_t)stream>>>(
            d, batch_of(batch), T, (uint16_t*)k_out, (uint16_t*)v_out);
    else
        moe::k_kv_read<64><<<(unsigned)blocks, moe::kAppendThreads, 0, (cudaStream_t)stream>>>(
            d, batch_of(batch), T, (uint16_t*)k_out, (uint16_t*)v_out);
    const cudaError_t e = cudaGetLastError();
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
    cudaError_t e = cudaSetDevice(h->cfg.device);
    if (e == cudaSuccess) e = cudaDeviceSynchronize();
    if (e == cudaSuccess) e = cudaMemcpy(&bits, h->err, sizeof bits, cudaMemcpyDeviceToHost);
    if (e == cudaSuccess && bits) e = cudaMemset(h->err, 0, sizeof bits);
    if (e != cudaSuccess) return cuda_refuse(e);
    if (bits) return refuse("a call met a position or page outside its tables");
    return MOE_OK;
}

moe_status_t moe_kv_destroy(moe_kv_t* h) {
    if (!h) return MOE_OK;
    cudaSetDevice(h->cfg.device);
    cudaDeviceSynchronize();
    cudaFree(h->pool);
    cudaFree(h->err);
    delete h;
    return MOE_OK;
}

}  // extern "C"
