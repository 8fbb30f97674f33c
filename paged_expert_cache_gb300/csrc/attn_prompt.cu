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
// tiles and runs them through the tensor cores in turn, so that the softmax of
// one overlaps the products of the other:
//   warps 0-3, 4-7  softmax of tile 0, 1: a thread per row, scores from tensor
//                   memory, weights back to it as bf16 over the scores
//   warp 8          TMA loads: the two query tiles, then K0 V0 K1 V1 ... into a
//                   ring of 128-key stages (128-byte swizzle)
//   warp 9          issues the MMAs: S = Q K^T (both from shared memory), and
//                   O += P V (P from tensor memory, V as the MN-major operand)
//   warps 10, 11    the values that some row of the CTA does not see: those past
//                   the sequence's keys are set to zero, and infinities and NaN
//                   behind the diagonal are replaced by zero (0 * inf would
//                   reach every row) and added to the rows that do see them at
//                   the end
// Tensor memory: S0 S1 (128 columns each) and O0 O1 (head_dim each), fp32.
// Weights are bf16 (the tensor cores take one type for both operands, and the
// values are bf16): an error of the size of the output's own rounding. Maxima
// and sums are fp32; a row's maximum is raised, and its output rescaled, only
// when a score exceeds it by 2^8.
#include <cuda.h>

#include <cmath>

#include "kv.cuh"
#include "moe_cache.h"
#include "tc.cuh"

namespace moe {

constexpr int kTile = 128;           // rows of a query tile, keys of a key tile
constexpr int kPromptThreads = 384;
constexpr float kRaise = 8.0f;       // log2 of the growth a row's weights may reach before a rescale

struct PromptArgs {
    const uint16_t* v;
    int64_t vs;
    const int *cu_q, *cu_k;
    int Tq, Tk, B, hq, hkv;
    float c;  // scale * log2 e
    uint16_t* out;
};

template <int D>
struct PromptSmem {
    static constexpr int kHalves = D / 64;                 // 64-dim halves of a tile: one swizzled row each
    static constexpr int kTileBytes = kTile * D * 2;
    static constexpr int kStages = D == 128 ? 5 : 8;
    uint8_t q[2][kTileBytes];
    uint8_t kv[kStages][kTileBytes];
    unsigned long long q_full[2], full[kStages], empty[kStages];
    unsigned long long s_full[2], p_full[2], o_full[2], dirty, clean;
    int seq_sum[kPromptThreads / 32];
    int total, seq, pair, flag, dead;
    uint32_t tmem;
};

__device__ __forceinline__ void bar_init_n(uint32_t bar, int n) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;\n" ::"r"(bar), "r"(n) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint32_t bar) {
    asm volatile("{\n.reg .b64 st;\nmbarrier.arrive.shared::cta.b64 st, [%0];\n}\n" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void bar_expect(uint32_t bar, uint32_t bytes) {
    asm volatile("{\n.reg .b64 st;\nmbarrier.arrive.expect_tx.shared::cta.b64 st, [%0], %1;\n}\n" ::"r"(bar), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n.reg .pred p;\nmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok;
}
// Waits for the phase; a wait that gives up marks the CTA, whose rows come out
// as NaN and whose other waits give up at once.
__device__ __forceinline__ void bar_wait(uint32_t bar, uint32_t parity, int* dead) {
    if (bar_try(bar, parity)) return;
    const unsigned long long t0 = globaltimer_ns();
    while (!bar_try(bar, parity)) {
        if (*(volatile int*)dead) return;
        if (globaltimer_ns() - t0 > kGWaitNs) *(volatile int*)dead = 1;
    }
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

// D[tmem] (+)= A[tmem] * B[smem], kind::f16.
__device__ __forceinline__ void tc_mma_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\ntcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d_tmem),
        "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// 32 columns of this thread's tensor-memory lane.
__device__ __forceinline__ void tc_st32(uint32_t taddr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
        "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};\n" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}
__device__ __forceinline__ void tc_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory"); }

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

// One lane of a converged warp, the same each time.
__device__ __forceinline__ bool elect_one() {
    uint32_t yes;
    asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}\n" : "=r"(yes));
    return yes;
}

__device__ __forceinline__ float ex2f(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
    return y;
}
// Two fp32 operations in one instruction (pairs in 64-bit registers).
__device__ __forceinline__ unsigned long long pair2(float lo, float hi) {
    return (unsigned long long)__float_as_uint(hi) << 32 | __float_as_uint(lo);
}
__device__ __forceinline__ unsigned long long fma2(unsigned long long a, unsigned long long b, unsigned long long c) {
    unsigned long long d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ unsigned long long add2(unsigned long long a, unsigned long long b) {
    unsigned long long d;
    asm("add.rn.f32x2 %0, %1, %2;\n" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ float lo2(unsigned long long v) { return __uint_as_float((uint32_t)v); }
__device__ __forceinline__ float hi2(unsigned long long v) { return __uint_as_float((uint32_t)(v >> 32)); }
__device__ __forceinline__ uint32_t pack_bf(float lo, float hi) {
    __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&p);
}
__device__ __forceinline__ bool any_nonfinite(uint32_t w) {  // of two bf16
    return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
}
__device__ __forceinline__ uint32_t drop_nonfinite(uint32_t w) {
    if ((w & 0x7f80u) == 0x7f80u) w &= 0xffff0000u;
    if ((w & 0x7f800000u) == 0x7f800000u) w &= 0xffffu;
    return w;
}

template <int D>
__global__ void __launch_bounds__(kPromptThreads, 1) k_prompt(PromptArgs a, const __grid_constant__ CUtensorMap mq,
                                                              const __grid_constant__ CUtensorMap mk,
                                                              const __grid_constant__ CUtensorMap mv) {
    using S = PromptSmem<D>;
    constexpr int kStages = S::kStages, kHalves = S::kHalves, kHalf = kTile * 128;
    extern __shared__ uint8_t raw[];
    S& sm = *reinterpret_cast<S*>(raw + (((gsmem(raw) + 1023u) & ~1023u) - gsmem(raw)));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int group = a.hq / a.hkv, tokens = kTile / group;  // tokens of a tile
    const int head = blockIdx.x % a.hkv, which = blockIdx.x / a.hkv;

    if (warp == 8) {
        tc_alloc(gsmem(&sm.tmem), 512);
        tc_relinquish();
    }
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            bar_init_n(gsmem(&sm.q_full[i]), 1);
            bar_init_n(gsmem(&sm.s_full[i]), 1);
            bar_init_n(gsmem(&sm.p_full[i]), 128);
            bar_init_n(gsmem(&sm.o_full[i]), 1);
        }
        for (int i = 0; i < kStages; ++i) {
            bar_init_n(gsmem(&sm.full[i]), 1);
            bar_init_n(gsmem(&sm.empty[i]), 1);
        }
        bar_init_n(gsmem(&sm.dirty), 1);
        bar_init_n(gsmem(&sm.clean), 64);
        sm.flag = 0;
        sm.dead = 0;
        asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    }
    // --- which pair of tiles: the sequences' pairs are numbered in order, and
    // the CTAs take them from the last, so that a sequence's longest run first
    auto pairs_of = [&](int s) {
        const int n = min(max(__ldg(a.cu_q + s + 1), 0), a.Tq) - min(max(__ldg(a.cu_q + s), 0), a.Tq);
        return n > 0 ? (n + 2 * tokens - 1) / (2 * tokens) : 0;
    };
    auto scan = [&](int w, int& incl, int& sum) {
        incl = w;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl, off);
            if (lane >= off) incl += v;
        }
        if (lane == 31) sm.seq_sum[warp] = incl;
        __syncthreads();
        sum = 0;
        int before = 0;
#pragma unroll
        for (int w2 = 0; w2 < kPromptThreads / 32; ++w2) {
            if (w2 == warp) before = sum;
            sum += sm.seq_sum[w2];
        }
        incl += before;
        __syncthreads();
    };
    int total = 0, mine = -1, seq = -1, pair = 0;
    if (a.B > kPromptThreads) {
        int w = 0, incl;
        for (int s = tid; s < a.B; s += kPromptThreads) w += pairs_of(s);
        scan(w, incl, total);
    }
    if (tid == 0) sm.seq = -1;
    for (int s0 = 0, base = 0; s0 < a.B; s0 += kPromptThreads) {
        const int w = s0 + tid < a.B ? pairs_of(s0 + tid) : 0;
        int incl, sum;
        scan(w, incl, sum);
        if (a.B <= kPromptThreads) total = sum;
        mine = total - 1 - which;
        incl += base;
        if (mine >= 0 && incl - w <= mine && mine < incl) {
            sm.seq = s0 + tid;
            sm.pair = mine - (incl - w);
        }
        base += sum;
        if (base > mine) break;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    seq = sm.seq;
    pair = sm.pair;
    const uint32_t tmem = sm.tmem;
    int* dead = &sm.dead;

    if (seq >= 0) {
        const int q0 = min(max(__ldg(a.cu_q + seq), 0), a.Tq), q1 = min(max(__ldg(a.cu_q + seq + 1), 0), a.Tq);
        const int k0 = min(max(__ldg(a.cu_k + seq), 0), a.Tk);
        const int lk = max(min(max(__ldg(a.cu_k + seq + 1), 0), a.Tk) - k0, 0), lq = q1 - q0, shift = lk - lq;
        // tile x: tokens i0[x] .. ; token i sees the keys below shift + i + 1
        const int i0 = pair * 2 * tokens;
        auto tiles_of = [&](int x) {  // key tiles of tile x
            const int first = i0 + x * tokens, last = min(first + tokens, lq) - 1;
            const int lim = last < first ? 0 : max(min(shift + last + 1, lk), 0);
            return (lim + kTile - 1) / kTile;
        };
        const int n0 = tiles_of(0), n1 = tiles_of(1), n = max(n0, n1);
        const int seen_by_all = max(min(shift + i0 + 1, lk), 0);  // keys below this are seen by every row
        const int first_masked = seen_by_all / kTile;             // first key tile with a value to be cleaned

        // Registers: the launch gives 168 a thread (64512 in all); the softmax
        // warpgroups hold a row of scores each and take 208, the third 88.
        if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 88;\n");
        if (warp == 8) {
            if (lane == 0) {
                for (int x = 0; x < 2; ++x) {
                    if ((x ? n1 : n0) == 0) continue;
                    const uint32_t bar = gsmem(&sm.q_full[x]);
                    bar_expect(bar, (uint32_t)(kHalves * 128 * group * tokens));
                    for (int h = 0; h < kHalves; ++h)
                        tma_4d(gsmem(sm.q[x]) + h * kHalf, &mq, bar, 64 * h, 0, head, q0 + i0 + x * tokens);
                }
                for (int e = 0; e < 2 * n; ++e) {  // K0 V0 K1 V1 ...
                    const int st = e % kStages;
                    const uint32_t bar = gsmem(&sm.full[st]);
                    if (e >= kStages) bar_wait(gsmem(&sm.empty[st]), (e / kStages - 1) & 1, dead);
                    if (*(volatile int*)dead) break;
                    bar_expect(bar, S::kTileBytes);
                    for (int h = 0; h < kHalves; ++h)
                        tma_3d(gsmem(sm.kv[st]) + h * kHalf, (e & 1) ? &mv : &mk, bar, 64 * h, head, k0 + (e >> 1) * kTile);
                }
            }
        } else if (warp == 9) {
            // The whole warp walks the loop and one lane issues, so that the
            // operands stay in uniform registers; descriptors are one base each
            // plus constants.
            if (n > 0) {
                constexpr uint32_t id_s = idesc_bf16(kTile, kTile, false), id_o = idesc_bf16(kTile, D, true);
                const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
                const bool leader = elect_one();
                const uint64_t qd = tc_sdesc(gsmem(sm.q[0])), kd = tc_sdesc(gsmem(sm.kv[0])), vd = sdesc_mn(gsmem(sm.kv[0]));
                constexpr uint64_t kTileStep = S::kTileBytes >> 4;  // to the next tile, in a descriptor
                auto scores = [&](int x, int st) {
                    const uint64_t qx = qd + x * kTileStep, kx = kd + st * kTileStep;
#pragma unroll
                    for (int d = 0; d < D / 16; ++d) {
                        const uint32_t off = ((d / 4) * kHalf + (d % 4) * 32) >> 4;
                        tc_mma(tm + x * kTile, qx + off, kx + off, id_s, d != 0);
                    }
                    tc_commit(gsmem(&sm.s_full[x]));
                };
                auto values = [&](int x, int st, bool first) {
                    const uint64_t vx = vd + st * kTileStep;
#pragma unroll
                    for (int t = 0; t < kTile / 16; ++t)
                        tc_mma_ta(tm + 2 * kTile + x * D, tm + x * kTile + 8 * t, vx + t * (2048 >> 4), id_o, t == 0 ? !first : 1);
                };
                bar_wait(gsmem(&sm.full[0]), 0, dead);
                for (int x = 0; x < 2; ++x) {
                    if ((x ? n1 : n0) == 0) continue;
                    bar_wait(gsmem(&sm.q_full[x]), 0, dead);
                    __syncwarp();
                    tc_fence_after();
                    if (leader) scores(x, 0);
                }
                if (leader) tc_commit(gsmem(&sm.empty[0]));
                int sv = 1, sk = 2;               // stages of V_j and K_(j + 1), and their rounds' parities
                uint32_t pv = 0, pk = 0;
                for (int j = 0; j < n; ++j) {
                    bar_wait(gsmem(&sm.full[sv]), pv, dead);
                    // the cleaning warps cannot tell the ring's rounds apart
                    if (j >= first_masked && leader) bar_arrive(gsmem(&sm.dirty));
                    if (j + 1 < n) bar_wait(gsmem(&sm.full[sk]), pk, dead);
                    if (*(volatile int*)dead) break;
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const int nx = x ? n1 : n0;
                        if (j < nx) {
                            bar_wait(gsmem(&sm.p_full[x]), j & 1, dead);
                            if (j >= first_masked) bar_wait(gsmem(&sm.clean), (j - first_masked) & 1, dead);
                            __syncwarp();
                            tc_fence_after();
                            if (leader) {
                                values(x, sv, j == 0);
                                if (j + 1 == nx) tc_commit(gsmem(&sm.o_full[x]));
                                else scores(x, sk);
                            }
                        }
                    }
                    if (leader) {
                        tc_commit(gsmem(&sm.empty[sv]));
                        if (j + 1 < n) tc_commit(gsmem(&sm.empty[sk]));
                    }
                    sv += 2, sk += 2;
                    if (sv >= kStages) sv -= kStages, pv ^= 1;
                    if (sk >= kStages) sk -= kStages, pk ^= 1;
                }
                // the last arrivals, so that none is under way when the CTA ends
                const int e = 2 * n - 1;
                bar_wait(gsmem(&sm.empty[e % kStages]), (e / kStages) & 1, dead);
            }
        } else {
            for (int j = first_masked; j < n; ++j) {
                const int e = 2 * j + 1, st = e % kStages;
                bar_wait(gsmem(&sm.dirty), (j - first_masked) & 1, dead);
                bar_wait(gsmem(&sm.full[st]), (e / kStages) & 1, dead);
                const int r0 = max(seen_by_all - j * kTile, 0);
                bool found = false;
                constexpr int kChunks = D / 8;  // 16-byte chunks of a key's values
                for (int w = tid - 320 + r0 * kChunks; w < kTile * kChunks; w += 64) {
                    const int r = w / kChunks, cc = w % kChunks;
                    uint4* at = reinterpret_cast<uint4*>(sm.kv[st] + (cc >> 3) * kHalf + r * 128 + (((cc ^ r) & 7) << 4));
                    if (j * kTile + r >= lk) {
                        *at = make_uint4(0, 0, 0, 0);
                    } else {
                        const uint4 u = *at;
                        if (any_nonfinite(u.x) || any_nonfinite(u.y) || any_nonfinite(u.z) || any_nonfinite(u.w)) {
                            found = true;
                            *at = make_uint4(drop_nonfinite(u.x), drop_nonfinite(u.y), drop_nonfinite(u.z), drop_nonfinite(u.w));
                        }
                    }
                }
                if (found) sm.flag = 1;
                fence_async_smem();
                bar_arrive(gsmem(&sm.clean));
            }
        }
        } else {
            asm volatile("setmaxnreg.inc.sync.aligned.u32 208;\n");
            // --- softmax of tile x, a thread per row
            const int x = warp >> 2, nx = x ? n1 : n0, row = tid & 127;
            const int tok = row / group, i = i0 + x * tokens + tok;
            const bool used = tok < tokens && i < lq;
            const int lim = used ? max(min(shift + i + 1, lk), 0) : 0;   // keys this row sees
            const int lim_tile = max(min(shift + i0 + x * tokens + 1, lk), 0);
            const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
            const uint32_t ts = tmem + lanes + x * kTile, to = tmem + lanes + 2 * kTile + x * D;
            float m = -INFINITY, l = 0.f;
            for (int j = 0; j < nx; ++j) {
                bar_wait(gsmem(&sm.s_full[x]), j & 1, dead);
                __syncwarp();
                tc_fence_after();
                uint32_t s[4][32];
#pragma unroll
                for (int h = 0; h < 4; ++h) tc_ld32(ts + 32 * h, s[h]);
                tc_ld_wait();
                if ((j + 1) * kTile > lim_tile) {
                    const int left = lim - j * kTile;  // columns from here on are hidden
#pragma unroll
                    for (int h = 0; h < 4; ++h)
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (32 * h + e >= left) s[h][e] = 0xff800000u;
                }
                float mx4[4] = {m, m, m, m};
#pragma unroll
                for (int h = 0; h < 4; ++h)
#pragma unroll
                    for (int e = 0; e < 32; e += 2)
                        mx4[(e >> 1) & 3] = fmaxf(mx4[(e >> 1) & 3], fmaxf(__uint_as_float(s[h][e]), __uint_as_float(s[h][e + 1])));
                const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3]));
                const bool raise = (mx - m) * a.c > kRaise;
                if (__any_sync(0xffffffffu, raise)) {
                    // S of this step was computed after the last step's O, so O is at rest
                    const float f = raise ? ex2f((m - mx) * a.c) : 1.f;
                    if (raise) m = mx;
                    l *= f;
                    if (j > 0) {
#pragma unroll
                        for (int h = 0; h < D / 32; ++h) {
                            uint32_t o[32];
                            tc_ld32(to + 32 * h, o);
                            tc_ld_wait();
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                            tc_st32(to + 32 * h, o);
                        }
                    }
                }
                const float mc = m == -INFINITY ? 0.f : m * a.c;
                const unsigned long long c2 = pair2(a.c, a.c), mc2 = pair2(-mc, -mc);
                unsigned long long sum[4] = {0, 0, 0, 0};
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t p[32];
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        const uint32_t* z = &s[2 * h + (e >> 4)][(2 * e) & 31];
                        const unsigned long long y = fma2(pair2(__uint_as_float(z[0]), __uint_as_float(z[1])), c2, mc2);
                        const float e0 = ex2f(lo2(y)), e1 = ex2f(hi2(y));
                        sum[e & 3] = add2(sum[e & 3], pair2(e0, e1));
                        p[e] = pack_bf(e0, e1);
                    }
                    tc_st32(ts + 32 * h, p);
                }
                sum[0] = add2(add2(sum[0], sum[1]), add2(sum[2], sum[3]));
                l += lo2(sum[0]) + hi2(sum[0]);
                tc_st_wait();
                tc_fence_before();
                bar_arrive(gsmem(&sm.p_full[x]));
            }
            // --- out
            if (nx) bar_wait(gsmem(&sm.o_full[x]), 0, dead);
            __syncwarp();
            tc_fence_after();
            const bool flag = nx && *(volatile int*)&sm.flag;
            const bool lost = *(volatile int*)dead;
            const float inv = l == 0.f ? 0.f : 1.0f / l;
            uint16_t* dst = a.out + ((size_t)(q0 + i) * a.hq + head * group + (row - tok * group)) * D;
#pragma unroll
            for (int h = 0; h < D / 32; ++h) {
                uint32_t o[32];
                __syncwarp();
                if (nx) {
                    tc_ld32(to + 32 * h, o);
                    tc_ld_wait();
                }
                float y[32];
#pragma unroll
                for (int e = 0; e < 32; ++e) y[e] = lim > 0 ? __uint_as_float(o[e]) * inv : 0.f;
                if (flag) {  // infinities and NaN that the cleaning took out, where this row sees them
                    for (int t = first_masked * kTile; t < lim; ++t) {
                        if (t < seen_by_all) continue;
                        const uint16_t* vr = a.v + (size_t)(k0 + t) * a.vs + (size_t)head * D + 32 * h;
#pragma unroll
                        for (int e = 0; e < 32; ++e) {
                            const float w = __uint_as_float((uint32_t)__ldg(vr + e) << 16);
                            if (!(fabsf(w) <= 3.4028235e38f)) y[e] += w;
                        }
                    }
                }
                if (used) {
#pragma unroll
                    for (int e = 0; e < 32; e += 8) {
                        uint4 u = make_uint4(pack_bf(y[e], y[e + 1]), pack_bf(y[e + 2], y[e + 3]), pack_bf(y[e + 4], y[e + 5]),
                                             pack_bf(y[e + 6], y[e + 7]));
                        if (lost) u = make_uint4(0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u);
                        *reinterpret_cast<uint4*>(dst + 32 * h + e) = u;
                    }
                }
            }
        }
        __syncwarp();
        if (*(volatile int*)dead && warp == 8 && lane == 0) {
            // copies under way land before the CTA leaves
            for (int e = 0; e < min(2 * n, kStages); ++e) gbar_wait(gsmem(&sm.full[e]), 0);
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

template <int D>
static cudaError_t launch_prompt(const PromptArgs& a, const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv,
                                 int64_t grid, cudaStream_t st) {
    constexpr int bytes = (int)sizeof(PromptSmem<D>) + 1024;
    static const cudaError_t set = cudaFuncSetAttribute(k_prompt<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (set != cudaSuccess) return set;
    k_prompt<D><<<(unsigned)grid, kPromptThreads, bytes, st>>>(a, mq, mk, mv);
    return cudaGetLastError();
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
    const moe::PromptArgs a = {(const uint16_t*)v, v_stride, cu_q, cu_k, Tq, Tk, num_seqs, q_heads, kv_heads, c, (uint16_t*)out};
    // at most this many pairs of tiles, whatever the lengths on the device are
    const int64_t pairs = (int64_t)Tq / (2 * tokens) + std::min(num_seqs, Tq);
    if (pairs * kv_heads > 0x7fffffffll) return refuse("too many rows");
    const cudaError_t e = head_dim == 128 ? moe::launch_prompt<128>(a, mq, mk, mv, pairs * kv_heads, (cudaStream_t)stream)
                                          : moe::launch_prompt<64>(a, mq, mk, mv, pairs * kv_heads, (cudaStream_t)stream);
    if (e == cudaSuccess) return MOE_OK;
    moe::set_last_error(cudaGetErrorString(e));
    return MOE_ERR_CUDA;
}
