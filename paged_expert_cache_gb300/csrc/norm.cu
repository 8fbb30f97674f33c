// norm.cu -- what stands between the two halves of a decoder layer: a block's
// output goes into the residual stream, and the sum, normed, is the next
// block's input; and its C entry point.
//
//   s = x + scale * gate * (post_weight ? rms(y) * post_weight : y)
//   x_out = s,  out = rms(s) * weight,  rms(v) = v / sqrt(mean(v^2) + eps)
//
// Bytes bound it: x, y in and x_out, out once each, and the weights from L2 for
// every row. A row stays in its threads' registers between the two sums: eight
// values a thread where rows are aligned (16-byte loads). A row of at most 256
// values is a warp's (four rows a CTA, no barrier), a longer one a CTA's, up to
// 1024 threads; so a call of one row has all its loads on the way at once.
//
// Everything is fp32: the sums of squares too, which fp32 holds unless values
// pass 2^63 or all are below 2^-50. A row whose sum left that range is summed
// again with its values times 2^-80 or 2^64, exact factors.
#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "kv.cuh"
#include "moe_cache.h"

namespace moe {

struct NormArgs {
    const void *x, *y, *weight, *post, *gate;
    void *x_out, *out;
    int64_t xs, ys, xos, os, gs;  // elements between rows
    int rows, hidden, gate_wide;
    float scale, eps, inv_h;
};

template <class T>
__device__ __forceinline__ float to_float(T v);
template <>
__device__ __forceinline__ float to_float(float v) { return v; }
template <>
__device__ __forceinline__ float to_float(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }

__device__ __forceinline__ uint32_t norm_pack(float lo, float hi) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&p);
}
// V consecutive values: one, or eight from a 16-byte boundary.
template <int V, class T>
__device__ __forceinline__ void load_values(float (&v)[V], const T* p) {
    if constexpr (V == 1) {
        v[0] = to_float(*p);
    } else if constexpr (sizeof(T) == 4) {
        const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
        const uint4 a = *reinterpret_cast<const uint4*>(p);
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) v[2 * e] = __uint_as_float(w[e] << 16), v[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
    }
}
template <int V, class T>
__device__ __forceinline__ void store_values(T* p, const float (&v)[V]) {
    if constexpr (V == 1) {
        if constexpr (sizeof(T) == 4) {
            *p = v[0];
        } else {
            const __nv_bfloat16 b = __float2bfloat16_rn(v[0]);
            *p = *reinterpret_cast<const uint16_t*>(&b);
        }
    } else if constexpr (sizeof(T) == 4) {
        *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
        *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
    } else {
        *reinterpret_cast<uint4*>(p) =
            make_uint4(norm_pack(v[0], v[1]), norm_pack(v[2], v[3]), norm_pack(v[4], v[5]), norm_pack(v[6], v[7]));
    }
}

// V values as they are in memory, on their way.
template <class T, int V>
struct Raw {
    uint32_t r[V == 1 ? 1 : V * sizeof(T) / 4];
    __device__ __forceinline__ void load(const T* p) {
        if constexpr (V == 1) {
            if constexpr (sizeof(T) == 4) r[0] = *reinterpret_cast<const uint32_t*>(p);
            else r[0] = *p;
        } else {
#pragma unroll
            for (int e = 0; e < (int)(V * sizeof(T) / 16); ++e) {
                const uint4 v = *(reinterpret_cast<const uint4*>(p) + e);
                r[4 * e] = v.x, r[4 * e + 1] = v.y, r[4 * e + 2] = v.z, r[4 * e + 3] = v.w;
            }
        }
    }
    __device__ __forceinline__ void get(float (&v)[V]) const {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int e = 0; e < V; ++e) v[e] = __uint_as_float(r[e]);
        } else if constexpr (V == 1) {
            v[0] = __uint_as_float(r[0] << 16);
        } else {
#pragma unroll
            for (int e = 0; e < V / 2; ++e) v[2 * e] = __uint_as_float(r[e] << 16), v[2 * e + 1] = __uint_as_float(r[e] & 0xffff0000u);
        }
    }
};

// The sum over a row's threads: a warp (`group` 32), or the CTA. Each call of a
// CTA has a line of `part` of its own, so that one barrier does.
__device__ __forceinline__ float row_sum(float v, int group, float* part) {
#pragma unroll
    for (int off = 16; off; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    if (group == 32) return v;
    const int lane = threadIdx.x & 31;
    if (lane == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    v = lane < group / 32 ? part[lane] : 0.f;
#pragma unroll
    for (int off = 16; off; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

// 1 / sqrt(mean v^2 + eps) is first * second (the factors apart, since their
// product may leave fp32's range). The values past the row's end are 0.
template <int E>
__device__ __forceinline__ float2 inverse_rms(const float (&v)[E], const NormArgs& a, int group, float (*part)[32]) {
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) s = fmaf(v[e], v[e], s);
    s = row_sum(s, group, part[0]);
    float f = 1.f;
    if (!(s <= 3.4028235e38f)) f = 0x1p-80f;
    else if (s < 0x1p-100f && a.eps < 0x1p-100f) f = 0x1p64f;
    if (f != 1.f) {  // the same for all of the row's threads
        s = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) s = fmaf(v[e] * f, v[e] * f, s);
        s = row_sum(s, group, part[1]);
    }
    return make_float2(f, 1.0f / sqrtf(fmaf(s, a.inv_h, a.eps * f * f)));
}

// V values at a time, N times a thread; `group` threads a row.
template <class X, class Y, class W, int V, int N>
__global__ void __launch_bounds__(1024) k_norm(NormArgs a, int group) {
    __shared__ float part[4][32];
    const int row = group == 32 ? blockIdx.x * (blockDim.x / 32) + (threadIdx.x >> 5) : blockIdx.x;
    const int t = group == 32 ? threadIdx.x & 31 : threadIdx.x;
    griddep_wait();
    griddep_launch();
    if (row >= a.rows) return;  // whole warps, and only where rows are warps'
    auto at = [&](int n) { return (n * group + t) * V; };
    float x[N * V], y[N * V];
    const X* xr = (const X*)a.x + row * a.xs;
    auto each = [&](auto f) {
#pragma unroll
        for (int n = 0; n < N; ++n)
            if (at(n) < a.hidden) f(n);
    };
#pragma unroll
    for (int e = 0; e < N * V; ++e) x[e] = y[e] = 0.f;
    each([&](int n) { load_values<V>(*reinterpret_cast<float(*)[V]>(x + n * V), xr + at(n)); });
    if (a.y) {
        const Y* yr = (const Y*)a.y + row * a.ys;
        each([&](int n) { load_values<V>(*reinterpret_cast<float(*)[V]>(y + n * V), yr + at(n)); });
        const W* gate = a.gate ? (const W*)a.gate + row * a.gs : nullptr;
        float one = a.scale;
        if (gate && !a.gate_wide) one *= to_float(*gate);
        if (a.post) {
            const float2 r = inverse_rms(y, a, group, part);
            each([&](int n) {
                float w[V];
                load_values<V>(w, (const W*)a.post + at(n));
#pragma unroll
                for (int e = 0; e < V; ++e) y[n * V + e] = y[n * V + e] * r.x * r.y * w[e];
            });
        }
        each([&](int n) {
            float g[V];
            if (a.gate_wide) load_values<V>(g, gate + at(n));
#pragma unroll
            for (int e = 0; e < V; ++e) x[n * V + e] = fmaf(a.gate_wide ? one * g[e] : one, y[n * V + e], x[n * V + e]);
        });
        if (a.x_out) {
            X* dst = (X*)a.x_out + row * a.xos;
            each([&](int n) { store_values<V>(dst + at(n), *reinterpret_cast<float(*)[V]>(x + n * V)); });
        }
    }
    if (!a.out) return;
    const float2 r = inverse_rms(x, a, group, part + 2);
    uint16_t* dst = (uint16_t*)a.out + row * a.os;
    each([&](int n) {
        float w[V], o[V];
        if (a.weight) load_values<V>(w, (const W*)a.weight + at(n));
#pragma unroll
        for (int e = 0; e < V; ++e) o[e] = x[n * V + e] * r.x * r.y * (a.weight ? w[e] : 1.f);
        store_values<V>(dst + at(n), o);
    });
}

// The same for many rows: a CTA takes every gridDim-th one. Its threads keep their
// columns' weights in registers (the post norm's times the gate's and the scale),
// and a row's loads are on the way while the row before it is done.
template <class X, class Y, class W, int V, int N>
__global__ void __launch_bounds__(512, 2) k_norm_rows(NormArgs a, int group) {
    constexpr int E = N * V;
    __shared__ float part[2][4][32];
    const int t = threadIdx.x;
    griddep_wait();
    griddep_launch();
    auto at = [&](int n) { return (n * group + t) * V; };
    auto each = [&](auto f) {
#pragma unroll
        for (int n = 0; n < N; ++n)
            if (at(n) < a.hidden) f(n);
    };
    float w[E], pw[E];  // of out; of y
    float one = a.scale;
#pragma unroll
    for (int e = 0; e < E; ++e) w[e] = 1.f, pw[e] = 1.f;
    each([&](int n) {
        if (a.weight) load_values<V>(*reinterpret_cast<float(*)[V]>(w + n * V), (const W*)a.weight + at(n));
        if (a.post) load_values<V>(*reinterpret_cast<float(*)[V]>(pw + n * V), (const W*)a.post + at(n));
        if (a.gate_wide) {
            float g[V];
            load_values<V>(g, (const W*)a.gate + at(n));
#pragma unroll
            for (int e = 0; e < V; ++e) pw[n * V + e] *= g[e];
        }
    });
    Raw<X, V> xr[N];
    Raw<Y, V> yr[N];
    float gate = 1.f;
    auto fetch = [&](int row) {
        each([&](int n) {
            xr[n].load((const X*)a.x + row * a.xs + at(n));
            if (a.y) yr[n].load((const Y*)a.y + row * a.ys + at(n));
        });
        if (a.gate && !a.gate_wide) gate = to_float(*((const W*)a.gate + row * a.gs));
    };
    fetch(blockIdx.x);
    int turn = 0;
    for (int row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1) {
        float x[E], y[E];
#pragma unroll
        for (int e = 0; e < E; ++e) x[e] = y[e] = 0.f;
        each([&](int n) {
            xr[n].get(*reinterpret_cast<float(*)[V]>(x + n * V));
            if (a.y) yr[n].get(*reinterpret_cast<float(*)[V]>(y + n * V));
        });
        const float here = one * gate;
        if (row + gridDim.x < (unsigned)a.rows) fetch(row + gridDim.x);
        if (a.y) {
            float2 r = make_float2(1.f, 1.f);
            if (a.post) r = inverse_rms(y, a, group, part[turn]);
#pragma unroll
            for (int e = 0; e < E; ++e) x[e] = fmaf(here, y[e] * r.x * r.y * pw[e], x[e]);
            if (a.x_out) {
                X* dst = (X*)a.x_out + row * a.xos;
                each([&](int n) { store_values<V>(dst + at(n), *reinterpret_cast<float(*)[V]>(x + n * V)); });
            }
        }
        if (!a.out) continue;
        const float2 r = inverse_rms(x, a, group, part[turn] + 2);
        uint16_t* dst = (uint16_t*)a.out + row * a.os;
        each([&](int n) {
            float o[V];
#pragma unroll
            for (int e = 0; e < V; ++e) o[e] = x[n * V + e] * r.x * r.y * w[n * V + e];
            store_values<V>(dst + at(n), o);
        });
    }
}

template <class X, class Y, class W>
static cudaError_t launch_norm(const NormArgs& a, bool aligned, int sms, cudaStream_t st) {
    const int per = 8, threads = std::min(1024, std::max(32, (a.hidden + per * 32 - 1) / (per * 32) * 32));
    const int n = (a.hidden + per * threads - 1) / (per * threads);  // eights a thread: 1, 2 or 4
    const int rows_a_cta = threads == 32 ? 4 : 1;
    if (threads > 32 && threads <= 512 && n == 1 && !(a.gate_wide && a.gs) && a.rows >= 8 * sms) {
        const int per_sm = 1024 / threads;
        return launch_ex(aligned ? k_norm_rows<X, Y, W, 8, 1> : k_norm_rows<X, Y, W, 1, 8>, dim3((unsigned)(sms * per_sm)), dim3(threads),
                         0, st, true, a, threads);
    }
    const dim3 grid((unsigned)((a.rows + rows_a_cta - 1) / rows_a_cta)), block(threads * rows_a_cta);
    if (aligned)
        return launch_ex(n == 1 ? k_norm<X, Y, W, 8, 1> : n == 2 ? k_norm<X, Y, W, 8, 2> : k_norm<X, Y, W, 8, 4>, grid, block, 0,
                         st, true, a, threads);
    return launch_ex(n == 1 ? k_norm<X, Y, W, 1, 8> : n == 2 ? k_norm<X, Y, W, 1, 16> : k_norm<X, Y, W, 1, 32>, grid, block, 0, st,
                     true, a, threads);
}

}  // namespace moe

namespace {
moe_status_t refuse(const char* msg) {
    moe::set_last_error(msg);
    return MOE_ERR_INVALID;
}
}  // namespace

extern "C" moe_status_t moe_residual_norm(const moe_norm_t* n, void* stream) {
    if (!n) return refuse("NULL argument");
    if (n->rows < 0) return refuse("rows must be >= 0");
    if (n->hidden < 1 || n->hidden > 32768) return refuse("hidden must be in 1..32768");
    for (int t : {n->x_type, n->y_type, n->w_type})
        if (t != MOE_TYPE_BF16 && t != MOE_TYPE_F32) return refuse("types must be MOE_TYPE_BF16 or MOE_TYPE_F32");
    if (!std::isfinite(n->scale) || !std::isfinite(n->eps) || n->eps < 0.f)
        return refuse("scale must be finite, eps finite and not negative");
    if (n->gate_wide != 0 && n->gate_wide != 1) return refuse("gate_wide must be 0 or 1");
    if (n->rows == 0) return MOE_OK;
    if (!n->y && (n->x_out || n->post_weight || n->gate)) return refuse("x_out, post_weight and gate need y");
    if (!n->out && !n->x_out) return refuse("neither out nor x_out");
    if (!n->x) return refuse("NULL x");
    const int H = n->hidden;
    bool aligned = H % 8 == 0;
    const char* problem = nullptr;
    auto look = [&](const void* p, int type, int64_t stride, bool repeats) {
        if (!p) return;
        const uintptr_t size = type == MOE_TYPE_F32 ? 4 : 2;
        if ((uintptr_t)p % size) problem = "a tensor is not aligned to its type";
        if (stride < H && !(repeats && stride == 0) && n->rows > 1) problem = "rows must be at least hidden elements apart";
        aligned = aligned && (uintptr_t)p % 16 == 0 && (stride * size) % 16 == 0;
    };
    look(n->x, n->x_type, n->x_stride, false);
    look(n->y, n->y_type, n->y_stride, false);
    look(n->x_out, n->x_type, n->x_out_stride, false);
    look(n->out, MOE_TYPE_BF16, n->out_stride, false);
    look(n->weight, n->w_type, 0, true);
    look(n->post_weight, n->w_type, 0, true);
    if (n->gate_wide) {
        look(n->gate, n->w_type, n->gate_stride, true);
    } else if (n->gate) {
        if (n->gate_stride < 0) problem = "gate_stride must be >= 0";
        if ((uintptr_t)n->gate % (n->w_type == MOE_TYPE_F32 ? 4 : 2)) problem = "a tensor is not aligned to its type";
    }
    if (problem) return refuse(problem);
    const moe::NormArgs a = {n->x, n->y, n->weight, n->post_weight, n->gate, n->x_out, n->out, n->x_stride, n->y_stride,
                             n->x_out_stride, n->out_stride, n->gate_stride, n->rows, H, n->gate ? n->gate_wide : 0, n->scale,
                             n->eps, 1.0f / (float)H};
    using F = float;
    using B = uint16_t;
    const int which = n->x_type * 4 + (n->y ? n->y_type : n->x_type) * 2 + n->w_type;
    auto* launch = moe::launch_norm<B, B, B>;
    switch (which) {
    case 1: launch = moe::launch_norm<B, B, F>; break;
    case 2: launch = moe::launch_norm<B, F, B>; break;
    case 3: launch = moe::launch_norm<B, F, F>; break;
    case 4: launch = moe::launch_norm<F, B, B>; break;
    case 5: launch = moe::launch_norm<F, B, F>; break;
    case 6: launch = moe::launch_norm<F, F, B>; break;
    case 7: launch = moe::launch_norm<F, F, F>; break;
    default: break;
    }
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = launch(a, aligned, moe::sm_count(dev), (cudaStream_t)stream);
    if (e == cudaSuccess) return MOE_OK;
    moe::set_last_error(cudaGetErrorString(e));
    return MOE_ERR_CUDA;
}
