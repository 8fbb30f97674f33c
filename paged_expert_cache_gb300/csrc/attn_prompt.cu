// attn_prompt.cu -- causal attention over packed sequences of bf16 keys and
// values, and its C entry point.
//
// Row i of a sequence's lq queries: out = sum_j softmax_j(scale q . k_j) v_j
// over the keys j <= lk - lq + i.
#include "kv.cuh"
#include "moe_cache.h"

namespace moe {

struct PromptArgs {
    const uint16_t *q, *k, *v;
    int64_t qs, ks, vs;
    const int *cu_q, *cu_k;
    int Tq, Tk, B, hq, hkv;
    float scale;
    uint16_t* out;
};

constexpr int kPromptWarps = 4;

// One warp per (row, query head): 32 keys at a time, a lane each for the
// scores, then a lane per D / 32 dims for the values.
template <int D>
__global__ void __launch_bounds__(32 * kPromptWarps) k_prompt(PromptArgs a) {
    constexpr int G = D / 32;
    __shared__ float q_s[kPromptWarps][D];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t = blockIdx.x, h = blockIdx.y * kPromptWarps + warp;
    const int seq = seq_of_row(a.cu_q, a.B, t);
    if (seq < 0 || h >= a.hq) return;
    for (int d = lane; d < D; d += 32)
        q_s[warp][d] = a.scale * __uint_as_float((uint32_t)a.q[(size_t)t * a.qs + (size_t)h * D + d] << 16);
    __syncwarp();
    const int k0 = max(__ldg(a.cu_k + seq), 0), k1 = min(__ldg(a.cu_k + seq + 1), a.Tk);
    const int seen = min(k1 - k0, k1 - k0 - (__ldg(a.cu_q + seq + 1) - t) + 1);
    const int head = h / (a.hq / a.hkv);
    float m = -INFINITY, l = 0.f, o[G] = {};
    for (int p0 = 0; p0 < seen; p0 += 32) {
        const int p = p0 + lane;
        float s = -INFINITY;
        if (p < seen) {
            s = 0.f;
            const uint16_t* kr = a.k + (size_t)(k0 + p) * a.ks + (size_t)head * D;
            for (int d = 0; d < D; d += 2) {
                const uint32_t w = *reinterpret_cast<const uint32_t*>(kr + d);
                s += q_s[warp][d] * __uint_as_float(w << 16) + q_s[warp][d + 1] * __uint_as_float(w & 0xffff0000u);
            }
        }
        float mx = s;
        for (int off = 16; off; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
        const float mn = fmaxf(m, mx);
        const float base = mn == -INFINITY ? 0.f : mn;
        const float f = expf(m - base);
        const float e = p < seen ? expf(s - base) : 0.f;
        float sum = e;
        for (int off = 16; off; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        l = l * f + sum;
        m = mn;
        for (int g = 0; g < G; ++g) o[g] *= f;
        for (int j = 0; j < 32 && p0 + j < seen; ++j) {
            const float pj = __shfl_sync(0xffffffffu, e, j);
            const uint16_t* vr = a.v + (size_t)(k0 + p0 + j) * a.vs + (size_t)head * D;
            for (int g = 0; g < G; ++g) o[g] += pj * __uint_as_float((uint32_t)vr[32 * g + lane] << 16);
        }
    }
    for (int g = 0; g < G; ++g) {
        __nv_bfloat16 v = __float2bfloat16_rn(l > 0.f || l != l ? o[g] / l : 0.f);
        a.out[((size_t)t * a.hq + h) * D + 32 * g + lane] = *reinterpret_cast<uint16_t*>(&v);
    }
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
    const moe::PromptArgs a = {(const uint16_t*)q, (const uint16_t*)k, (const uint16_t*)v, q_stride, k_stride, v_stride,
                               cu_q, cu_k, Tq, Tk, num_seqs, q_heads, kv_heads, scale, (uint16_t*)out};
    const dim3 grid((unsigned)Tq, (unsigned)((q_heads + moe::kPromptWarps - 1) / moe::kPromptWarps));
    if (head_dim == 128) moe::k_prompt<128><<<grid, 32 * moe::kPromptWarps, 0, (cudaStream_t)stream>>>(a);
    else moe::k_prompt<64><<<grid, 32 * moe::kPromptWarps, 0, (cudaStream_t)stream>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) return MOE_OK;
    moe::set_last_error(cudaGetErrorString(e));
    return MOE_ERR_CUDA;
}
