// rope_axes.cuh -- rotary positions with several axes (time, height, width of
// images and video, or any other), on the queries and keys of one layer.
//
// Pair i of a row (x_i, x_{i+d/2}) belongs to one axis a(i) and turns by
//   angle = pos[a(i)][b][t] * frequency(i) / factor,
// rotate-half form, as the single-axis kernel of rope.cuh; `sign` = -1 turns
// back (the rotation's transpose, which carries gradients).
//
// Angles are counted in whole turns in fp64, x = pos * frequency / (2 pi
// factor): rint(x) drops out exactly, and what is left, |r| <= 1/2, goes to
// the fp32 sincospi, whose argument's rounding is made good to first order
// (cos(a + e) = cos a - e sin a): no range reduction of a large angle, and an
// error of the order of fp32's own rounding at any 32-bit position.
//
// One CTA per `rows` consecutive tokens (flattened over the sequences) and
// slice of heads: the tokens' cosines and sines are computed once and shared by
// the slice's heads; each thread turns 16-byte pieces of a row's two halves,
// four rows' loads in flight.  HBM-bound: one read and one write of the
// tensors.
#pragma once

#include "device.cuh"

namespace ssa {

constexpr int kRopeAxesRows = 16;     // most tokens per CTA
constexpr int kRopeAxesThreads = 256;
constexpr int kRopeMaxAxes = 4;

struct RopeAxesTable {
    double turns[64];  // turns per unit of position of every pair
    uint8_t axis[64];
};

// One tensor [B, heads, T, d]: element strides of batch, head and token (elements of a row are adjacent).
struct RopeAxesTensor {
    const void *in;
    void *out;
    int64_t is[3], os[3];
    int heads;  // 0: no such tensor
};

template <typename T>
__device__ __forceinline__ void rope_load(const T *x, float (&v)[16 / sizeof(T)]) {
    const uint4 w = *reinterpret_cast<const uint4 *>(x);
    const uint32_t p[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        if constexpr (sizeof(T) == 2) {
            v[2 * q] = __uint_as_float(p[q] << 16);
            v[2 * q + 1] = __uint_as_float(p[q] & 0xFFFF0000u);
        } else {
            v[q] = __uint_as_float(p[q]);
        }
    }
}

template <typename T>
__device__ __forceinline__ void rope_store(T *x, const float (&v)[16 / sizeof(T)]) {
    uint32_t p[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        if constexpr (sizeof(T) == 2)
            p[q] = pack_bf16x2(v[2 * q], v[2 * q + 1]);
        else
            p[q] = __float_as_uint(v[q]);
    }
    *reinterpret_cast<uint4 *>(x) = make_uint4(p[0], p[1], p[2], p[3]);
}

// Rows [head h0 .. h1) x [the CTA's nt tokens] of one tensor.  `in` may be `out`: a thread reads both
// pieces of a row before it writes them, and no other thread touches them.
template <typename T>
__device__ __forceinline__ void rope_axes_rows(const RopeAxesTensor &X, const float2 (*cs)[64], const int64_t *in_at,
                                               const int64_t *out_at, int h0, int h1, int nt, int half) {
    constexpr int V = 16 / sizeof(T), U = 4;
    const int units = half / V, rpp = kRopeAxesThreads / units;
    const int u = threadIdx.x % units, rr = threadIdx.x / units;
    const int rows = (h1 - h0) * nt;
    for (int row0 = rr; row0 < rows; row0 += U * rpp) {
        float a[U][V], c[U][V];
        int64_t to[U];
        int tok[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int row = row0 + i * rpp;
            if (row < rows) {
                const int h = h0 + row / nt;
                tok[i] = row % nt;
                const T *x = static_cast<const T *>(X.in) + in_at[tok[i]] + h * X.is[1] + u * V;
                to[i] = out_at[tok[i]] + h * X.os[1] + u * V;
                rope_load<T>(x, a[i]);
                rope_load<T>(x + half, c[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
            if (row0 + i * rpp < rows) {
                float y0[V], y1[V];
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const float2 t = cs[tok[i]][u * V + v];
                    y0[v] = a[i][v] * t.x - c[i][v] * t.y;
                    y1[v] = a[i][v] * t.y + c[i][v] * t.x;
                }
                T *y = static_cast<T *>(X.out) + to[i];
                rope_store<T>(y, y0);
                rope_store<T>(y + half, y1);
            }
        }
    }
}

// grid (ceil(B*T / rows), head slices); heads_per = query heads, then key heads, of one slice.
template <typename T>
__global__ void __launch_bounds__(kRopeAxesThreads) rope_axes_kernel(
    const __grid_constant__ RopeAxesTable tab, const int32_t *__restrict__ pos, int64_t BT, int T_len, int half,
    int rows, int heads_per, float sign, const __grid_constant__ RopeAxesTensor Q,
    const __grid_constant__ RopeAxesTensor K) {
    __shared__ float2 cs[kRopeAxesRows][64];
    __shared__ int64_t at[4][kRopeAxesRows];  // element offsets of the tokens: Q in, Q out, K in, K out
    const int64_t f0 = static_cast<int64_t>(blockIdx.x) * rows;
    const int nt = static_cast<int>(min(static_cast<int64_t>(rows), BT - f0));
    for (int e = threadIdx.x; e < nt * half; e += kRopeAxesThreads) {
        const int tt = e / half, i = e % half;
        const double p = static_cast<double>(__ldg(pos + tab.axis[i] * BT + f0 + tt));
        const double r = fma(p, tab.turns[i], -rint(p * tab.turns[i]));  // turns, in [-1/2, 1/2]
        const float rf = static_cast<float>(r);
        const float e1 = static_cast<float>((r - static_cast<double>(rf)) * 6.283185307179586);
        float s, c;
        sincospif(2.f * rf, &s, &c);
        cs[tt][i] = make_float2(fmaf(-e1, s, c), sign * fmaf(e1, c, s));
    }
    if (threadIdx.x < nt) {
        const int64_t f = f0 + threadIdx.x, b = f / T_len, t = f % T_len;
        at[0][threadIdx.x] = b * Q.is[0] + t * Q.is[2];
        at[1][threadIdx.x] = b * Q.os[0] + t * Q.os[2];
        at[2][threadIdx.x] = b * K.is[0] + t * K.is[2];
        at[3][threadIdx.x] = b * K.os[0] + t * K.os[2];
    }
    __syncthreads();
    const int h0 = blockIdx.y * heads_per, h1 = min(h0 + heads_per, Q.heads + K.heads);
    if (h0 < Q.heads) rope_axes_rows<T>(Q, cs, at[0], at[1], h0, min(h1, Q.heads), nt, half);
    if (h1 > Q.heads) rope_axes_rows<T>(K, cs, at[2], at[3], max(h0 - Q.heads, 0), h1 - Q.heads, nt, half);
}

}  // namespace ssa
