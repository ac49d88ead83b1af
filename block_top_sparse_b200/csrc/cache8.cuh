// cache8.cuh -- the 8-bit key/value cache: writing tokens into it and dropping
// blocks from it (attention over it: cache_decode.cuh).
//
// A cache row holds d = 128 e4m3 codes; every block of s tokens of a key/value
// head has one fp32 scale for its keys and one for its values, and the element
// is code * scale.  Scales are powers of two: dividing by one is exact, so a
// stored element carries the one rounding to e4m3 (4 significant bits, at most
// 2^-4 of the value; multiples of 2^-9 scale below 2^-6 scale) and
// code * scale is again exact in bf16.  The scale of a block is the smallest
// 2^p >= 2^-126 that brings the largest finite element to 448 (e4m3's largest)
// or less, so that the block's largest element lies in (224, 448] codes.
//
// cache_append_kernel writes new tokens.  A block that is begun keeps its scale
// until a larger element arrives; then its older codes are moved to the larger
// scale (exact but for codes that fall below 2^-6, which are rounded a second
// time).  When a block's last token arrives, the mean of its keys as the cache
// holds them joins the pooled keys.  One CTA per (sequence and key head, touched
// block, keys or values): the block's new rows stay in registers between the
// maximum and the conversion, so they are read once.  HBM-bound for prompts
// (4 d bytes read, 2 d written per token and key head), latency-bound for single
// tokens.
//
// cache_evict_*_kernel drops blocks by accumulated attention weight.  The kept
// blocks and the one begun move down in order, in place.  Every 16-byte column
// of a head's blocks is moved by one thread, ascending: a block's new place is
// never behind its old one, so what a thread overwrites it has already read,
// and no thread waits for another.  Bound by reading and writing the moved
// blocks once.
#pragma once

#include "device.cuh"
#include "top_blocks.cuh"

namespace ssa {

constexpr int kCacheD = 128;  // head size: a row of codes is 128 bytes

enum : unsigned { ERR_CACHE_INPUT = 6u };  // SSA_ERR_BAD_INPUT

// Smallest power of two >= 2^-126 that brings |a| (finite, >= 0) to 448 = 1.75 * 2^8 or less.
__device__ __forceinline__ float e4m3_scale(float a) {
    const uint32_t u = __float_as_uint(a);
    const int e = static_cast<int>(u >> 23) - 127;  // a = 1.m * 2^e (subnormals: below every scale)
    int p = (u & 0x7FFFFFu) <= 0x600000u ? e - 8 : e - 7;
    p = max(p, -126);
    return __uint_as_float(static_cast<uint32_t>(p + 127) << 23);
}

// 1 / 2^p for p in [-126, 126] (exact).
__device__ __forceinline__ float pow2_inverse(float s) {
    return __uint_as_float((254u << 23) - __float_as_uint(s));
}

// New rows [B, Hkv, n, d]: element strides of batch, head and token.
struct CacheRows {
    const __nv_bfloat16 *p;
    int64_t st[3];
};

// grid (B * Hk, blocks that n rows can touch, 2: keys, values): 16 threads of 8 elements per row, kAppendPasses
// passes over the block's rows, all of them in flight at once.  (A 32K prompt of 8 heads, blocks of 128, and
// ragged pieces of 16 heads, blocks of 64, in a captured graph: 33.6 and 13.7 us; with 4 passes by twice the threads
// 46.4 and 17.0 us, with 16 by half of them 49.0 and 20.0 us.  The launch bounds keep 1024 threads on an SM at 64
// registers, 40 and 52 bytes of which spill; at 512 threads and 96 registers nothing does: 43.9 and 15.1 us.)
constexpr int kAppendPasses = 8;
constexpr int append_threads(int s) { return 16 * s / kAppendPasses; }

template <int S>
__global__ void __launch_bounds__(append_threads(S), 1024 / append_threads(S)) cache_append_kernel(
    const int32_t *__restrict__ cache_len, const int32_t *__restrict__ n_new, int n, const CacheRows K,
    const CacheRows V, uint8_t *K8, float *Kscale, uint8_t *V8, float *Vscale, float *Kbar, int Hk, int T) {
    constexpr int P = kAppendPasses, kRows = S / P, kThreads = append_threads(S), kWarps = kThreads / 32;
    __shared__ uint32_t red[kWarps];
    __shared__ float col[kRows][kCacheD];
    const int bh = blockIdx.x, b = bh / Hk, hk = bh % Hk;
    const int L = __ldg(cache_len + b), nn = n_new ? __ldg(n_new + b) : n;
    if (L < -1 || nn < 0 || nn > n || nn > T - L) {  // nothing is written for this sequence
        if (threadIdx.x == 0) record_error(ERR_CACHE_INPUT, 0x701);
        return;
    }
    if (L < 0) return;  // an idle row
    const int j = L / S + blockIdx.y;
    const int64_t u0 = static_cast<int64_t>(j) * S;                      // the block's first token
    const int r0 = static_cast<int>(max(static_cast<int64_t>(L), u0) - u0);  // new rows [r0, r1)
    const int r1 = static_cast<int>(min(static_cast<int64_t>(L) + nn, u0 + S) - u0);
    if (r1 <= r0) return;
    const bool keys = blockIdx.z == 0;
    const CacheRows &X = keys ? K : V;
    const size_t block = static_cast<size_t>(bh) * (T / S) + j;
    uint8_t *codes = (keys ? K8 : V8) + block * S * kCacheD;
    float *scale = (keys ? Kscale : Vscale) + block;
    const int u = threadIdx.x & 15, rr = threadIdx.x >> 4, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const __nv_bfloat16 *x = X.p + b * X.st[0] + hk * X.st[1] + (u0 - L) * X.st[2] + u * 8;
    uint4 v[P];
    uint32_t top2 = 0;  // largest magnitude bits, even and odd elements
#pragma unroll
    for (int p = 0; p < P; ++p) {
        const int r = rr + kRows * p;
        v[p] = make_uint4(0u, 0u, 0u, 0u);
        if (r >= r0 && r < r1) v[p] = __ldg(reinterpret_cast<const uint4 *>(x + r * X.st[2]));
    }
    const float old = r0 > 0 ? *scale : 0.f;
#pragma unroll
    for (int p = 0; p < P; ++p) {
        const uint32_t a = __vmaxu2(v[p].x & 0x7FFF7FFFu, v[p].y & 0x7FFF7FFFu);
        const uint32_t c = __vmaxu2(v[p].z & 0x7FFF7FFFu, v[p].w & 0x7FFF7FFFu);
        top2 = __vmaxu2(top2, __vmaxu2(a, c));
    }
    auto block_max = [&](uint32_t m) {
        m = __reduce_max_sync(0xffffffffu, m);
        __syncthreads();
        if (lane == 0) red[warp] = m;
        __syncthreads();
        m = red[0];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) m = max(m, red[w]);
        return m;
    };
    uint32_t top = block_max(max(top2 & 0xFFFFu, top2 >> 16));
    const bool special = top >= 0x7F80u;  // (uniform) an infinity or a NaN among the new rows
    if (special) {  // the scale goes by the finite elements; infinities become NaN
        uint32_t m = 0;
#pragma unroll
        for (int p = 0; p < P; ++p) {
            uint32_t w[4] = {v[p].x, v[p].y, v[p].z, v[p].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t lo = w[i] & 0x7FFFu, hi = (w[i] >> 16) & 0x7FFFu;
                if (lo < 0x7F80u)
                    m = max(m, lo);
                else
                    w[i] |= 0x7FFFu;
                if (hi < 0x7F80u)
                    m = max(m, hi);
                else
                    w[i] |= 0x7FFF0000u;
            }
            v[p] = make_uint4(w[0], w[1], w[2], w[3]);
        }
        top = block_max(m);
    }
    const float want = fmaxf(e4m3_scale(__uint_as_float(top << 16)), old);
    const float inv = pow2_inverse(want);
    const bool pool = keys && Kbar && r1 == S;  // the block is complete: its mean key (uniform)
    uint64_t sum[4] = {0, 0, 0, 0};  // of this thread's eight columns, in pairs
    auto add = [&](const uint2 &w) {
        const uint32_t q[2] = {w.x, w.y};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            sum[2 * i] = fadd2(sum[2 * i], unpack_e4m3x2_f2(static_cast<uint16_t>(q[i])));
            sum[2 * i + 1] = fadd2(sum[2 * i + 1], unpack_e4m3x2_f2(static_cast<uint16_t>(q[i] >> 16)));
        }
    };
    const uint64_t inv2 = f2_pack(inv, inv);
    if (r0 > 0 && (want > old || pool)) {  // older rows: moved to a larger scale, or summed
        const float ratio = old * inv;
        for (int r = rr; r < r0; r += kRows) {
            uint2 *q = reinterpret_cast<uint2 *>(codes + r * kCacheD + u * 8);
            uint2 w = *q;
            if (want > old) {
                uint32_t c[2] = {w.x, w.y};
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float2 a = unpack_e4m3x2(static_cast<uint16_t>(c[i]));
                    const float2 d = unpack_e4m3x2(static_cast<uint16_t>(c[i] >> 16));
                    c[i] = pack_e4m3x2(a.x * ratio, a.y * ratio) |
                           static_cast<uint32_t>(pack_e4m3x2(d.x * ratio, d.y * ratio)) << 16;
                }
                w = make_uint2(c[0], c[1]);
                *q = w;
            }
            if (pool) add(w);
        }
    }
#pragma unroll
    for (int p = 0; p < P; ++p) {
        const int r = rr + kRows * p;
        if (r < r0 || r >= r1) continue;
        const uint32_t w[4] = {v[p].x, v[p].y, v[p].z, v[p].w};
        uint32_t c[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float lo, hi;
            f2_unpack(fmul2(f2_pack(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u)), inv2), lo, hi);
            c[i] = pack_e4m3x2(lo, hi);
        }
        const uint2 q = make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
        *reinterpret_cast<uint2 *>(codes + r * kCacheD + u * 8) = q;
        if (pool) add(q);
    }
    if (threadIdx.x == 0) *scale = want;
    if (pool) {  // sums of codes are multiples of 2^-9 and mostly exact in fp32
#pragma unroll
        for (int i = 0; i < 4; ++i) f2_unpack(sum[i], col[rr][u * 8 + 2 * i], col[rr][u * 8 + 2 * i + 1]);
        __syncthreads();
        for (int c = threadIdx.x; c < kCacheD; c += kThreads) {
            float a = 0.f;
#pragma unroll
            for (int r = 0; r < kRows; ++r) a += col[r][c];
            Kbar[block * kCacheD + c] = a / static_cast<float>(S) * want;  // (both powers of two)
        }
    }
}

// One new token per sequence (n = 1): a warp per (sequence, key head), lanes 0-15 the key, lanes 16-31 the
// value, no barrier; grid ceil(B * Hk / 4).  The decode step's form: its time is that of the loads after one
// another (length, row and scale, store); kernel time for 64 sequences, 8 key heads: 2.1 us, 6.2 us with a CTA per
// block.  A step in which some token outgrows its block's scale, as most steps of a batch of this size have one, waits for
// the older rows of that block to be moved, eight per round trip: 4 us more with 43 older rows, 10 us more with 126; a
// step that completes every block 3 us more.
template <int S>
__global__ void __launch_bounds__(128) cache_append_token_kernel(
    const int32_t *__restrict__ cache_len, const int32_t *__restrict__ n_new, const CacheRows K, const CacheRows V,
    uint8_t *K8, float *Kscale, uint8_t *V8, float *Vscale, float *Kbar, int pairs, int Hk, int T) {
    const int bh = blockIdx.x * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31, side = lane >> 4, u = lane & 15;
    if (bh >= pairs) return;
    const int b = bh / Hk, hk = bh % Hk;
    const CacheRows &X = side ? V : K;
    // the row does not depend on the length: both are asked for at once
    const uint4 v = __ldg(reinterpret_cast<const uint4 *>(X.p + b * X.st[0] + hk * X.st[1] + u * 8));
    const int L = __ldg(cache_len + b), nn = n_new ? __ldg(n_new + b) : 1;
    if (L < -1 || nn < 0 || nn > 1 || nn > T - L) {
        if (lane == 0) record_error(ERR_CACHE_INPUT, 0x704);
        return;
    }
    if (L < 0 || nn == 0) return;
    const int j = L / S, r0 = L % S;
    const size_t block = static_cast<size_t>(bh) * (T / S) + j;
    uint8_t *codes = (side ? V8 : K8) + block * S * kCacheD + u * 8;
    float *scale = (side ? Vscale : Kscale) + block;
    const float old = r0 > 0 ? *scale : 0.f;
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t finite = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t lo = w[i] & 0x7FFFu, hi = (w[i] >> 16) & 0x7FFFu;
        if (lo < 0x7F80u) finite = max(finite, lo);
        if (hi < 0x7F80u) finite = max(finite, hi);
    }
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) finite = max(finite, __shfl_xor_sync(0xffffffffu, finite, o));
    const float want = fmaxf(e4m3_scale(__uint_as_float(finite << 16)), old), inv = pow2_inverse(want);
    if (r0 > 0 && want > old) {  // the older rows move to the larger scale
        const float ratio = old * inv;
#pragma unroll 8
        for (int r = 0; r < r0; ++r) {
            uint2 *q = reinterpret_cast<uint2 *>(codes + r * kCacheD);
            uint32_t c[2] = {q->x, q->y};
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float2 a = unpack_e4m3x2(static_cast<uint16_t>(c[i]));
                const float2 d = unpack_e4m3x2(static_cast<uint16_t>(c[i] >> 16));
                c[i] = pack_e4m3x2(a.x * ratio, a.y * ratio) |
                       static_cast<uint32_t>(pack_e4m3x2(d.x * ratio, d.y * ratio)) << 16;
            }
            *q = make_uint2(c[0], c[1]);
        }
    }
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float lo = __uint_as_float(w[i] << 16) * inv, hi = __uint_as_float(w[i] & 0xFFFF0000u) * inv;
        lo = fabsf(lo) < INFINITY ? lo : NAN, hi = fabsf(hi) < INFINITY ? hi : NAN;  // (-0 stays -0)
        c[i] = pack_e4m3x2(lo, hi);
    }
    *reinterpret_cast<uint2 *>(codes + r0 * kCacheD) = make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
    if (u == 0) *scale = want;
    if (Kbar && r0 == S - 1) {  // the block is complete: the whole warp sums its keys, two rows at a time
        __syncwarp();           // the rows just written
        const float key_scale = __shfl_sync(0xffffffffu, want, 0);
        const uint8_t *rows = K8 + block * S * kCacheD + side * kCacheD + u * 8;
        float sum[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[i] = 0.f;
#pragma unroll 16
        for (int r = 0; r < S; r += 2) {
            const uint2 q = *reinterpret_cast<const uint2 *>(rows + r * kCacheD);
            const uint32_t p[2] = {q.x, q.y};
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float2 a = unpack_e4m3x2(static_cast<uint16_t>(p[i]));
                const float2 d = unpack_e4m3x2(static_cast<uint16_t>(p[i] >> 16));
                sum[4 * i] += a.x, sum[4 * i + 1] += a.y, sum[4 * i + 2] += d.x, sum[4 * i + 3] += d.y;
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 16);
        if (side == 0) {
            float4 *to = reinterpret_cast<float4 *>(Kbar + block * kCacheD + u * 8);
#pragma unroll
            for (int i = 0; i < 2; ++i)
                to[i] = make_float4(sum[4 * i] / S * key_scale, sum[4 * i + 1] / S * key_scale,
                                    sum[4 * i + 2] / S * key_scale, sum[4 * i + 3] / S * key_scale);
        }
    }
}

// ---------------------------------------------------------------------------
// Eviction
// ---------------------------------------------------------------------------
// The move list of one head in the workspace: blocks in use after the call, the sequence's new length, the
// first place whose block changes, then the old place of the block that goes to every place.
constexpr int kEvictHead = 4;
__host__ __device__ __forceinline__ size_t evict_list_ints(int nb) { return static_cast<size_t>(nb) + kEvictHead; }

// One CTA per (sequence, key head).  Shared memory: nb weights, nb keys, keep + 1 list entries.
__global__ void __launch_bounds__(kTopThreads) cache_evict_select_kernel(
    const int32_t *__restrict__ cache_len, const float *weight_in, float *weight_out, float *Kscale, float *Vscale,
    int32_t *__restrict__ kept, int32_t *__restrict__ lists, int Hk, int T, int s, int nb, int keep, int sink,
    int recent) {
    grid_dependents_launch();
    extern __shared__ uint32_t evict_sm[];
    __shared__ TopScratch sc;
    __shared__ int first_sm;
    float *w = reinterpret_cast<float *>(evict_sm);
    uint32_t *key = evict_sm + nb;
    int32_t *list = reinterpret_cast<int32_t *>(evict_sm + 2 * nb);
    const int bh = blockIdx.x, b = bh / Hk, tid = threadIdx.x;
    int L = __ldg(cache_len + b);
    const int given = L;
    if (L < 0 || L > T) {  // the sequence stays as it is; -1 is an idle row, others are reported
        if (L != -1 && tid == 0) record_error(ERR_CACHE_INPUT, 0x702);
        L = 0;
    }
    const int whole = L / s, begun = L % s > 0 ? 1 : 0;
    const float *win = weight_in + static_cast<size_t>(bh) * nb;
    for (int j = tid; j < nb; j += kTopThreads) {
        w[j] = win[j];
        // blocks that always stay come before every weight
        key[j] = (j < sink || j >= whole - recent) ? 0xFFFFFFFFu : score_key(w[j]);
    }
    if (tid == 0) first_sm = nb;
    __syncthreads();
    const int left = min(whole, keep), used = left + begun;
    if (whole > keep) {
        top_blocks(key, whole, keep, list, sc);
    } else {
        for (int r = tid; r < left; r += kTopThreads) list[r] = r;
    }
    if (tid == 0 && begun) list[left] = whole;
    __syncthreads();
    int32_t *out = lists + bh * evict_list_ints(nb);
    for (int r = tid; r < keep; r += kTopThreads)
        kept[static_cast<size_t>(bh) * keep + r] = r < left ? list[r] : -1;
    for (int r = tid; r < used; r += kTopThreads) {
        out[kEvictHead + r] = list[r];
        if (list[r] != r) atomicMin(&first_sm, r);
    }
    __syncthreads();
    if (tid == 0) {
        out[0] = used;
        out[1] = given == L ? left * s + L % s : given;
        out[2] = first_sm;
    }
    if (weight_out)
        for (int j = tid; j < nb; j += kTopThreads)
            weight_out[static_cast<size_t>(bh) * nb + j] = given != L ? w[j] : j < used ? w[list[j]] : 0.f;
    // scales move as the blocks do: a step's reads come before its writes, and later steps read further on
    float *ks = Kscale + static_cast<size_t>(bh) * nb, *vs = Vscale + static_cast<size_t>(bh) * nb;
    for (int r0 = first_sm; r0 < used; r0 += kTopThreads) {
        const int r = r0 + tid;
        const float a = r < used ? ks[list[r]] : 0.f, c = r < used ? vs[list[r]] : 0.f;
        __syncthreads();
        if (r < used) ks[r] = a, vs[r] = c;
    }
}

constexpr int kMoveThreads = 128;

// grid (B * Hk, column groups): a thread owns one 16-byte column of every block of a head (first the keys'
// s * 8 columns, then the values', then the pooled keys' 32) and moves it down the list.
__global__ void __launch_bounds__(kMoveThreads) cache_evict_move_kernel(uint8_t *K8, uint8_t *V8, float *Kbar,
                                                                        int32_t *new_len, const int32_t *lists, int Hk,
                                                                        int s, int nb) {
    extern __shared__ int32_t list[];  // [nb]
    grid_dependency_wait();
    const int bh = blockIdx.x;
    const int32_t *head = lists + bh * evict_list_ints(nb);
    const int used = __ldcg(head), first = __ldcg(head + 2);
    if (new_len && blockIdx.y == 0 && threadIdx.x == 0 && bh % Hk == 0) new_len[bh / Hk] = __ldcg(head + 1);
    if (first >= used) return;
    for (int r = first + threadIdx.x; r < used; r += kMoveThreads) list[r] = __ldcg(head + kEvictHead + r);
    __syncthreads();
    const int per = s * (kCacheD / 16);
    int c = blockIdx.y * kMoveThreads + threadIdx.x;
    uint8_t *base;
    size_t step;
    if (c < 2 * per) {
        step = static_cast<size_t>(s) * kCacheD;
        base = c < per ? K8 : V8;
        c = c < per ? c : c - per;
    } else {
        step = kCacheD * 4;
        base = reinterpret_cast<uint8_t *>(Kbar);
        c -= 2 * per;
        if (!base || c >= kCacheD * 4 / 16) return;
    }
    uint8_t *col = base + static_cast<size_t>(bh) * nb * step + static_cast<size_t>(c) * 16;
    constexpr int U = 16;
    for (int r0 = first; r0 < used; r0 += U) {
        uint4 v[U];
#pragma unroll
        for (int i = 0; i < U; ++i)
            if (r0 + i < used) v[i] = *reinterpret_cast<const uint4 *>(col + list[r0 + i] * step);
#pragma unroll
        for (int i = 0; i < U; ++i)
            if (r0 + i < used) *reinterpret_cast<uint4 *>(col + (r0 + i) * step) = v[i];
    }
}

}  // namespace ssa
