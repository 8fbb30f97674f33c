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
// 1024 threads; so a call of one row has all its loads on the way at once (k_norm).
// From 8193 values on a thread has 16 or 32 of x and as many of y, more than its
// registers hold: part of them go through local memory, most of them where rows past
// 16384 are not aligned.
// From two rows an SM on, and up to 4096 values, CTAs take several rows, the next
// one's loads under the last one's sums: k_norm_rows where rows are aligned, and two
// more kernels for rows that are not. (Rows of 4096 bf16 with both norms, of 4001, and of
// 2048 fp32 with one norm and y bf16, two sets of inputs in turn: 320 rows 4.0, 5.4 and 2.9
// us, a row a CTA 4.7, 8.3 and 2.7; 2451 rows 17.0, 18.9 and 10.6, a row a CTA 27.7, 44.8
// and 11.2, their bytes 12.0, 11.7 and 9.0.)
//
// Measured in a graph: one row of 2048 1.9 us, 61 of 4096 with both norms 2.9, 2451
// of 2048 8.9 (6.8 TB/s, part of it from L2), 15013 of 4000 with both norms 94 (6.4
// TB/s, 0.95 of a copy), of 4001 103. Past 4096 values, a row a CTA: 7500 rows of 5120 bf16
// with both norms 86, of 8192 174, of 16384 252, of 16391 3520 (bytes 46, 74, 147 and 147).
//
// Everything is fp32: the sums of squares too, which fp32 holds unless values
// pass 2^63 or all are below 2^-50. A row whose sum left that range is summed
// again with its values times 2^-80 or 2^64, exact factors.
#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "kv.cuh"
#include "moe_cache.h"
#include "row_piece.h"

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
    // elements lo .. hi - 1 only, 0 for the others
    __device__ __forceinline__ void load_some(const T* p, int lo, int hi) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const bool in = e >= lo && e < hi;
            if constexpr (sizeof(T) == 4) {
                r[e] = in ? *reinterpret_cast<const uint32_t*>(p + e) : 0u;
            } else {
                const uint32_t v = in ? (uint32_t)p[e] << (16 * (e & 1)) : 0u;
                r[e / 2] = e & 1 ? r[e / 2] | v : v;
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

// 1 / sqrt(mean v^2 + eps). Where the sum of squares leaves fp32's range, v is taken
// times a power of two, and so is the result, whose product with v stays the same.
// The values past the row's end are 0.
template <int E>
__device__ __forceinline__ float inverse_rms(float (&v)[E], const NormArgs& a, int group, float (*part)[32]) {
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
        for (int e = 0; e < E; ++e) {
            v[e] *= f;
            s = fmaf(v[e], v[e], s);
        }
        s = row_sum(s, group, part[1]);
    }
    return 1.0f / sqrtf(fmaf(s, a.inv_h, a.eps * f * f));
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
            const float r = inverse_rms(y, a, group, part);
            each([&](int n) {
                float w[V];
                load_values<V>(w, (const W*)a.post + at(n));
#pragma unroll
                for (int e = 0; e < V; ++e) y[n * V + e] = y[n * V + e] * r * w[e];
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
    const float r = inverse_rms(x, a, group, part + 2);
    uint16_t* dst = (uint16_t*)a.out + row * a.os;
    each([&](int n) {
        float w[V], o[V];
        if (a.weight) load_values<V>(w, (const W*)a.weight + at(n));
#pragma unroll
        for (int e = 0; e < V; ++e) o[e] = x[n * V + e] * r * (a.weight ? w[e] : 1.f);
        store_values<V>(dst + at(n), o);
    });
}

// The same for many rows: a CTA takes every gridDim-th one. Its threads keep their
// columns' weights in registers (the post norm's times the gate's and the scale),
// and a row's loads are on the way while the row before it is done.
template <class X, class Y, class W>
__global__ void __launch_bounds__(512, 2) k_norm_rows(NormArgs a, int group) {
    constexpr int V = 8, N = 1, E = N * V;
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
    if ((int)blockIdx.x >= a.rows) return;  // the whole CTA
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
            float r = 1.f;
            if (a.post) r = inverse_rms(y, a, group, part[turn]);
#pragma unroll
            for (int e = 0; e < E; ++e) x[e] = fmaf(here, y[e] * r * pw[e], x[e]);
            if (a.x_out) {
                X* dst = (X*)a.x_out + row * a.xos;
                each([&](int n) { store_values<V>(dst + at(n), *reinterpret_cast<float(*)[V]>(x + n * V)); });
            }
        }
        if (!a.out) continue;
        const float r = inverse_rms(x, a, group, part[turn] + 2);
        uint16_t* dst = (uint16_t*)a.out + row * a.os;
        each([&](int n) {
            float o[V];
#pragma unroll
            for (int e = 0; e < V; ++e) o[e] = x[n * V + e] * r * w[n * V + e];
            store_values<V>(dst + at(n), o);
        });
    }
}

// The same for rows of any width whose tensors have one phase: element 0 of a row
// lies as many elements behind a multiple of eight in each of them (dense tensors of
// one odd width). A thread takes eight elements from a 16-byte boundary on, which
// start at 8 t - phase. The phase changes from row to row, but over eight rows it
// comes back, and the grid is a multiple of eight: a CTA's rows have one, and its
// threads' columns stay as they are. The pieces at a row's edges are read whole, but
// for the tensor's first and last row, and written element by element.
// 15013 rows of 4001, both norms: 103 us (5.8 TB/s, 0.87 of a copy; weights in shared
// memory and edges read element by element, whose packing waits for them, 147; through
// k_norm_lines 182). What is left over the aligned rows' 94 is mostly the edges' stores.
template <class X, class Y, class W>
__global__ void __launch_bounds__(512, 2) k_norm_phase(NormArgs a, int group, int phase0) {
    constexpr int V = 8;
    __shared__ float part[2][4][32];
    const int H = a.hidden, i = 8 * (int)threadIdx.x - (int)(((unsigned)phase0 + blockIdx.x * (unsigned)(a.xs & 7)) & 7u);
    const bool edge = i < 0 || i + V > H;
    auto in = [&](int e) { return i + e >= 0 && i + e < H; };
    griddep_wait();
    griddep_launch();
    float w[V], pw[V];  // of out; of y. Past the row's ends they are 0, and so are the values there made
#pragma unroll
    for (int e = 0; e < V; ++e) {
        w[e] = !in(e) ? 0.f : a.weight ? to_float(((const W*)a.weight)[i + e]) : 1.f;
        pw[e] = !in(e) ? 0.f : a.post ? to_float(((const W*)a.post)[i + e]) : 1.f;
        if (a.gate_wide && in(e)) pw[e] *= to_float(((const W*)a.gate)[i + e]);
    }
    Raw<X, V> xr;
    Raw<Y, V> yr;
    float gate = 1.f;
    auto fetch = [&](int row) {
        const X* x = (const X*)a.x + row * a.xs + i;
        const Y* y = (const Y*)a.y + row * a.ys + i;
        const bool inner = row > 0 && row + 1 < a.rows;  // what lies beside the row is the tensor's as well
        if (inner || !edge) {
            if (i < H) {
                xr.load(x);
                if (a.y) yr.load(y);
            }
        } else {
            xr.load_some(x, -i, H - i);
            if (a.y) yr.load_some(y, -i, H - i);
        }
        if (a.gate && !a.gate_wide) gate = to_float(((const W*)a.gate)[row * a.gs]);
    };
    auto put = [&](auto* to, const float (&v)[V]) {
        if (!edge) {
            store_values<V>(to, v);
        } else if (i < H) {
#pragma unroll
            for (int e = 0; e < V; ++e)
                if (in(e)) {
                    const float one[1] = {v[e]};
                    store_values<1>(to + e, one);
                }
        }
    };
    if ((int)blockIdx.x >= a.rows) return;  // the whole CTA
    fetch(blockIdx.x);
    int turn = 0;
    for (int row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1) {
        float x[V], y[V];
        xr.get(x);
        if (a.y) yr.get(y);
        if (edge) {
#pragma unroll
            for (int e = 0; e < V; ++e)
                if (!in(e)) x[e] = y[e] = 0.f;
        }
        const float here = a.scale * gate;
        if (row + gridDim.x < (unsigned)a.rows) fetch(row + gridDim.x);
        if (a.y) {
            float r = 1.f;
            if (a.post) r = inverse_rms(y, a, group, part[turn]);
#pragma unroll
            for (int e = 0; e < V; ++e) x[e] = fmaf(here, y[e] * r * pw[e], x[e]);
            if (a.x_out) put((X*)a.x_out + row * a.xos + i, x);
        }
        if (!a.out) continue;
        const float r = inverse_rms(x, a, group, part[turn] + 2);
        float o[V];
#pragma unroll
        for (int e = 0; e < V; ++e) o[e] = x[e] * r * w[e];
        put((uint16_t*)a.out + row * a.os + i, o);
    }
}

// A row that need not start on a 16-byte boundary, between memory and shared
// memory: there its bytes lie from the row's own phase on, so that aligned 16-byte
// pieces go over as they are. The pieces that the row shares with its neighbours are
// read whole, but for the tensor's first and last one, and written element by element.
template <class T>
struct Line {
    static constexpr int kPieces = sizeof(T) / 2 + 1;  // of a thread, at most: a row of n has n sizeof(T) / 16 + 2
    uint4 piece[kPieces];
    // whole: the row's first and last piece lie in the tensor as well
    __device__ __forceinline__ void fetch(const T* row, int n, bool whole, int t, int group) {
        const int phase = (int)((uintptr_t)row & 15u), bytes = phase + n * (int)sizeof(T), pieces = (bytes + 15) / 16;
        const uint4* from = reinterpret_cast<const uint4*>((const uint8_t*)row - phase);
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const int k = t + i * group;
            if (k >= pieces) break;
            if (whole || (k > 0 && 16 * k + 16 <= bytes)) {
                piece[i] = from[k];
            } else {  // only what is the row's
                uint32_t w[4];
                row_piece(w, row, (16 * k - phase) / (int)sizeof(T), n);
                piece[i] = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
    }
    __device__ __forceinline__ void put(uint8_t* to, int phase, int n, int t, int group) const {
        const int pieces = (phase + n * (int)sizeof(T) + 15) / 16;
#pragma unroll
        for (int i = 0; i < kPieces; ++i)
            if (t + i * group < pieces) *reinterpret_cast<uint4*>(to + 16 * (t + i * group)) = piece[i];
    }
    static __device__ __forceinline__ void out(T* row, const uint8_t* from, int n, int t, int group) {
        const int phase = (int)((uintptr_t)row & 15u), bytes = phase + n * (int)sizeof(T);
        uint4* to = reinterpret_cast<uint4*>((uint8_t*)row - phase);
        const int first = (phase + 15) / 16, end = bytes / 16;
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const int k = first + t + i * group;
            if (k < end) to[k] = *reinterpret_cast<const uint4*>(from + 16 * k);
        }
        if (t < 16) {  // fewer than 8 elements before them, and behind them
            const int at = t < 8 ? t : (16 * end - phase) / (int)sizeof(T) + t - 8;
            if (t < 8 ? at < (16 * first - phase) / (int)sizeof(T) : at < n) row[at] = reinterpret_cast<const T*>(from + phase)[at];
        }
    }
    // of a line in shared memory that holds n elements and is read up to 8 `group`
    static __host__ __device__ constexpr int bytes(int group) { return 8 * group * (int)sizeof(T) + 32; }
};

// k_norm_rows for rows of any width, each tensor with a phase of its own. Its
// instructions bound it (3.1 TB/s).
template <class X, class Y, class W>
__global__ void __launch_bounds__(512, 2) k_norm_lines(NormArgs a, int group) {
    constexpr int E = 8;
    extern __shared__ __align__(16) uint8_t lines[];
    __shared__ float part[2][4][32];
    const int t = threadIdx.x, H = a.hidden;
    uint8_t *lx = lines, *ly = lx + Line<X>::bytes(group), *lo = ly + Line<Y>::bytes(group), *lxo = lo + Line<uint16_t>::bytes(group);
    griddep_wait();
    griddep_launch();
    float w[E], pw[E];  // of out; of y. Past the row's end they are 0, and so are the values there made
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const int i = e * group + t;
        w[e] = i >= H ? 0.f : a.weight ? to_float(((const W*)a.weight)[i]) : 1.f;
        pw[e] = i >= H ? 0.f : a.post ? to_float(((const W*)a.post)[i]) : 1.f;
        if (a.gate_wide && i < H) pw[e] *= to_float(((const W*)a.gate)[i]);
    }
    Line<X> xl;
    Line<Y> yl;
    float gate = 1.f;
    auto x_row = [&](int row) { return (const X*)a.x + row * a.xs; };
    auto y_row = [&](int row) { return (const Y*)a.y + row * a.ys; };
    auto fetch = [&](int row) {
        const bool inner = row > 0 && row + 1 < a.rows;
        xl.fetch(x_row(row), H, inner, t, group);
        if (a.y) yl.fetch(y_row(row), H, inner, t, group);
        if (a.gate && !a.gate_wide) gate = to_float(((const W*)a.gate)[row * a.gs]);
    };
    if ((int)blockIdx.x >= a.rows) return;  // the whole CTA
    fetch(blockIdx.x);
    const int last = H - 1 - t;  // element e * group + t is the row's where e * group <= last
    int turn = 0;
    for (int row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1) {
        const int px = (int)((uintptr_t)x_row(row) & 15u), py = (int)((uintptr_t)y_row(row) & 15u);
        xl.put(lx, px, H, t, group);
        if (a.y) yl.put(ly, py, H, t, group);
        const float here = a.scale * gate;
        if (row + gridDim.x < (unsigned)a.rows) fetch(row + gridDim.x);
        __syncthreads();  // the row is there, and the last one's outputs have left
        const X* xs = reinterpret_cast<const X*>(lx + px) + t;
        float x[E];
#pragma unroll
        for (int e = 0; e < E; ++e) x[e] = e * group <= last ? to_float(xs[e * group]) : 0.f;
        X* xo = (X*)a.x_out + row * a.xos;
        uint16_t* o = (uint16_t*)a.out + row * a.os;
        if (a.y) {
            const Y* ys = reinterpret_cast<const Y*>(ly + py) + t;
            float y[E];
#pragma unroll
            for (int e = 0; e < E; ++e) y[e] = e * group <= last ? to_float(ys[e * group]) : 0.f;
            float r = 1.f;
            if (a.post) r = inverse_rms(y, a, group, part[turn]);
#pragma unroll
            for (int e = 0; e < E; ++e) x[e] = fmaf(here, y[e] * r * pw[e], x[e]);
            if (a.x_out) {
                X* to = reinterpret_cast<X*>(lxo + ((uintptr_t)xo & 15u)) + t;
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const float v[1] = {x[e]};
                    store_values<1>(to + e * group, v);
                }
            }
        }
        if (a.out) {
            const float r = inverse_rms(x, a, group, part[turn] + 2);
            uint16_t* to = reinterpret_cast<uint16_t*>(lo + ((uintptr_t)o & 15u)) + t;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const float v[1] = {x[e] * r * w[e]};
                store_values<1>(to + e * group, v);
            }
        }
        __syncthreads();
        if (a.x_out) Line<X>::out(xo, lxo, H, t, group);
        if (a.out) Line<uint16_t>::out(o, lo, H, t, group);
    }
}

template <class X, class Y, class W>
static cudaError_t launch_norm(const NormArgs& a, bool aligned, int dev, cudaStream_t st) {
    const int sms = sm_count(dev);
    const int per = 8, threads = std::min(1024, std::max(32, (a.hidden + per * 32 - 1) / (per * 32) * 32));
    const int n = (a.hidden + per * threads - 1) / (per * threads);  // eights a thread: 1, 2 or 4
    const int rows_a_cta = threads == 32 ? 4 : 1;
    if (threads > 32 && threads <= 512 && n == 1 && !(a.gate_wide && a.gs) && a.rows >= 2 * sms) {
        auto ctas = [&](int per) { return dim3((unsigned)std::min(a.rows, sms * (1024 / per))); };  // 1024 threads an SM
        const dim3 grid = ctas(threads);
        if (aligned) return launch_ex(k_norm_rows<X, Y, W>, grid, dim3(threads), 0, st, true, a, threads);
        // the phase that all rows of all tensors have, if there is one
        const int sx = sizeof(X), sy = sizeof(Y), phase = (int)((uintptr_t)a.x / sx & 7u);
        const bool one = (!a.y || ((int)((uintptr_t)a.y / sy & 7u) == phase && ((a.ys - a.xs) & 7) == 0)) &&
                         (!a.x_out || ((int)((uintptr_t)a.x_out / sx & 7u) == phase && ((a.xos - a.xs) & 7) == 0)) &&
                         (!a.out || ((int)((uintptr_t)a.out / 2 & 7u) == phase && ((a.os - a.xs) & 7) == 0));
        if (one && a.hidden + 7 <= 8 * 512) {
            const int wider = std::max(64, (a.hidden + 7 + 255) / 256 * 32);  // 8 threads' elements, and the phase
            dim3 eights = ctas(wider);
            eights.x = std::max(8u, eights.x & ~7u);  // rows 8 n apart have one phase
            return launch_ex(k_norm_phase<X, Y, W>, eights, dim3(wider), 0, st, true, a, wider, phase);
        }
        const int bytes = 2 * Line<X>::bytes(threads) + Line<Y>::bytes(threads) + Line<uint16_t>::bytes(threads);
        static DeviceOnce once;
        const cudaError_t set = once.run(dev, [] {
            return cudaFuncSetAttribute(k_norm_lines<X, Y, W>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        2 * Line<X>::bytes(512) + Line<Y>::bytes(512) + Line<uint16_t>::bytes(512));
        });
        if (set != cudaSuccess) return set;
        return launch_ex(k_norm_lines<X, Y, W>, grid, dim3(threads), bytes, st, true, a, threads);
    }
    const dim3 grid((unsigned)((a.rows - 1) / rows_a_cta + 1)), block(threads * rows_a_cta);
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
    if (e == cudaSuccess) e = launch(a, aligned, dev, (cudaStream_t)stream);
    if (e == cudaSuccess) return MOE_OK;
    moe::set_last_error(cudaGetErrorString(e));
    return MOE_ERR_CUDA;
}
