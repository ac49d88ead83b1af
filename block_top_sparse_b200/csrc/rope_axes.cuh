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
// One CTA per `rows` consecutive tokens (flattened over the sequences): the
// tokens' cosines and sines are computed once, while the
// first heads' rows are on their way.  A thread keeps those of one token's
// 16-byte piece in registers and walks down the heads with them, four heads'
// loads (both halves of the row) in flight.
// HBM-bound: one read and one write of the tensors.
#pragma once

#include "device.cuh"

namespace ssa {

constexpr int kRopeAxesRows = 8;      // most tokens per CTA (a power of two)
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

// Elements of a 16-byte piece.
template <typename T>
__device__ __forceinline__ void rope_unpack(const uint4 &w, float (&v)[16 / sizeof(T)]) {
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
__device__ __forceinline__ uint4 rope_pack(const float (&v)[16 / sizeof(T)]) {
    uint32_t p[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        if constexpr (sizeof(T) == 2)
            p[q] = pack_bf16x2(v[2 * q], v[2 * q + 1]);
        else
            p[q] = __float_as_uint(v[q]);
    }
    return make_uint4(p[0], p[1], p[2], p[3]);
}

// grid ceil(B*T / rows).  Three CTAs per SM: 80 registers, 40 bytes of which spill for bf16, 113.7 us for a 32K prompt of
// 40 heads; two without a spill 149 us.
template <typename T>
__global__ void __launch_bounds__(kRopeAxesThreads, 3) rope_axes_kernel(
    const __grid_constant__ RopeAxesTable tab, const int32_t *__restrict__ pos, int64_t BT, int T_len, int half,
    int rows, float sign, const __grid_constant__ RopeAxesTensor Q,
    const __grid_constant__ RopeAxesTensor K) {
    constexpr int V = 16 / sizeof(T), U = 4;
    __shared__ float2 cs[kRopeAxesRows][64];
    const int64_t f0 = static_cast<int64_t>(blockIdx.x) * rows;
    const int nt = static_cast<int>(min(static_cast<int64_t>(rows), BT - f0));
    // thread: 16-byte piece u of token tt, heads h, h + step, .. (rows * units divides the CTA); the queries'
    // heads come first, then the keys'
    const int units = half / V, u = threadIdx.x % units, tt = threadIdx.x / units % rows;
    const int step = kRopeAxesThreads / units / rows;
    const int h1 = Q.heads + K.heads;
    int h = threadIdx.x / units / rows;
    if (tt >= nt) h = h1;
    const int64_t f = f0 + tt, b = f / T_len, t = f % T_len;
    const T *q_in = static_cast<const T *>(Q.in) + b * Q.is[0] + t * Q.is[2] + u * V;
    const T *k_in = static_cast<const T *>(K.in) + b * K.is[0] + t * K.is[2] + u * V;
    // The outputs may be the inputs: a thread reads both halves of a row before it writes them, and no other
    // thread touches them.
    uint4 a[U], c[U];
    auto load = [&]() {
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int hi = h + i * step;
            if (hi < h1) {
                const T *x = hi < Q.heads ? q_in + hi * Q.is[1] : k_in + (hi - Q.heads) * K.is[1];
                a[i] = *reinterpret_cast<const uint4 *>(x);
                c[i] = *reinterpret_cast<const uint4 *>(x + half);
            }
        }
    };
    // (bf16: 115 -> 113.6 us for a 32K prompt of 40 heads; fp32 has no registers left for it: 46 -> 49 us for 16K
    // tokens of 32 heads of 64)
    constexpr bool kAhead = sizeof(T) == 2;
    if (kAhead) load();
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
    __syncthreads();
    if (tt >= nt) return;
    float2 mine[V];
#pragma unroll
    for (int v = 0; v < V; ++v) mine[v] = cs[tt][u * V + v];
    T *q_out = static_cast<T *>(Q.out) + b * Q.os[0] + t * Q.os[2] + u * V;
    T *k_out = static_cast<T *>(K.out) + b * K.os[0] + t * K.os[2] + u * V;
    while (h < h1) {
        if (!kAhead) load();
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int hi = h + i * step;
            if (hi < h1) {
                float x0[V], x1[V], y0[V], y1[V];
                rope_unpack<T>(a[i], x0);
                rope_unpack<T>(c[i], x1);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    y0[v] = x0[v] * mine[v].x - x1[v] * mine[v].y;
                    y1[v] = x0[v] * mine[v].y + x1[v] * mine[v].x;
                }
                T *y = hi < Q.heads ? q_out + hi * Q.os[1] : k_out + (hi - Q.heads) * K.os[1];
                *reinterpret_cast<uint4 *>(y) = rope_pack<T>(y0);
                *reinterpret_cast<uint4 *>(y + half) = rope_pack<T>(y1);
            }
        }
        h += U * step;
        if (kAhead) load();
    }
}

}  // namespace ssa
