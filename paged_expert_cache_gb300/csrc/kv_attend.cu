// kv_attend.cu -- attention of the newest tokens over the paged Q4_0 cache.
//
// out = sum_p softmax_p(scale q . k_p) v_p over the positions p a row sees.
#include "kv.cuh"

namespace moe {

constexpr int kWarps = 4;

// One warp per (row, query head): 32 positions at a time, a lane each for the
// scores, then a lane per D / 32 dims for the values; running maximum and sum
// in fp32.
template <int D>
__global__ void __launch_bounds__(32 * kWarps) k_attend(KvDev c, KvBatch b, const uint16_t* __restrict__ q, int64_t qs,
                                                        int T, float scale, uint16_t* __restrict__ out) {
    constexpr int G = D / 32;
    using C = Cell<D>;
    __shared__ float q_s[kWarps][D];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t = blockIdx.x, h = blockIdx.y * kWarps + warp;
    const int seq = seq_of_row(b.cu, b.B, t);
    if (seq < 0 || h >= c.hq) return;
    for (int d = lane; d < D; d += 32)
        q_s[warp][d] = scale * __uint_as_float((uint32_t)q[(size_t)t * qs + (size_t)h * D + d] << 16);
    __syncwarp();
    const int seen = __ldg(b.kv_lens + seq) - (__ldg(b.cu + seq + 1) - t) + 1;
    const int head = h / (c.hq / c.hkv);
    float m = -INFINITY, l = 0.f, o[G] = {};
    bool bad = false;
    for (int p0 = 0; p0 < seen; p0 += 32) {
        const int p = p0 + lane, tc = p & (kCellTokens - 1);
        const uint8_t* cell = p < seen ? kv_cell<D>(c, b, seq, p, head) : nullptr;
        bad |= p < seen && !cell;
        float s = -INFINITY;
        if (cell) {
            s = 0.f;
            for (int bl = 0; bl < G; ++bl) {
                float a = 0.f;
                for (int i = 0; i < 4; ++i) {
                    const uint32_t w = *reinterpret_cast<const uint32_t*>(cell + C::k_word(tc, i, bl));
                    for (int j = 0; j < 4; ++j) {
                        const float* qq = &q_s[warp][32 * bl + 8 * i + 2 * j];
                        a += qq[0] * ((float)((w >> (4 * j)) & 15u) - 8.f) + qq[1] * ((float)((w >> (16 + 4 * j)) & 15u) - 8.f);
                    }
                }
                s += a * __half2float(*reinterpret_cast<const __half*>(cell + C::kKs + C::scale(tc, bl)));
            }
        }
        float mx = s;
        for (int off = 16; off; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
        const float mn = fmaxf(m, mx);
        const float base = mn == -INFINITY ? 0.f : mn;
        const float f = expf(m - base);
        const float e = cell ? expf(s - base) : 0.f;
        float sum = e;
        for (int off = 16; off; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        l = l * f + sum;
        m = mn;
        for (int bl = 0; bl < G; ++bl) o[bl] *= f;
        for (int j = 0; j < 32 && p0 + j < seen; ++j) {
            const float pj = __shfl_sync(0xffffffffu, e, j);
            const uint8_t* cj = kv_cell<D>(c, b, seq, p0 + j, head);
            if (!cj) continue;
            const int tj = (p0 + j) & (kCellTokens - 1);
            for (int bl = 0; bl < G; ++bl) {  // dim 32 bl + lane = 32 bl + g + 8 i
                const uint32_t w = *reinterpret_cast<const uint16_t*>(cj + C::kV + C::v_half(tj, lane & 7, bl));
                const float d = __half2float(*reinterpret_cast<const __half*>(cj + C::kVs + C::scale(tj, bl)));
                o[bl] += pj * (d * ((float)((w >> (4 * (lane >> 3))) & 15u) - 8.f));
            }
        }
    }
    bad = __any_sync(0xffffffffu, bad);
    if (bad && lane == 0) atomicOr(c.err, 1u);
    for (int bl = 0; bl < G; ++bl) {
        float r = l > 0.f || l != l ? o[bl] / l : 0.f;
        if (bad) r = __int_as_float(0x7fc00000);
        __nv_bfloat16 v = __float2bfloat16_rn(r);
        out[((size_t)t * c.hq + h) * D + 32 * bl + lane] = *reinterpret_cast<uint16_t*>(&v);
    }
}

uint64_t attend_scratch_bytes(int) { return 0; }

void launch_attend(const KvDev& c, const KvBatch& b, int D, const uint16_t* q, int64_t q_stride, int T, float scale,
                   uint16_t* out, void*, cudaStream_t st) {
    const dim3 grid((unsigned)T, (unsigned)((c.hq + kWarps - 1) / kWarps));
    if (D == 128) k_attend<128><<<grid, 32 * kWarps, 0, st>>>(c, b, q, q_stride, T, scale, out);
    else k_attend<64><<<grid, 32 * kWarps, 0, st>>>(c, b, q, q_stride, T, scale, out);
}

}  // namespace moe
