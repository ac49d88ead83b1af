// top_blocks.cuh -- the kk largest of n scores of one row, by one CTA: which
// blocks a query attends and which blocks stay in a cache.
//
// Scores become 32-bit keys whose unsigned order is theirs (NaN lowest, both
// zeros equal).  Four passes over the key's bytes, highest first, each a
// 256-bin count in shared memory among the keys that share the bytes found so
// far, give the kk-th largest key; the chosen indices are those above it and
// the first ones equal to it, written in ascending order from ballots.  The
// counts do not depend on the order of the additions, so neither does the
// result; the cost is 4n / 256 steps of the CTA, whatever kk.  Below 1024 keys one
// warp searches them in its registers instead.
#pragma once

#include "device.cuh"

namespace ssa {

constexpr int kTopThreads = 256;
constexpr int kTopMaxBlocks = 8192;  // keys of a row in 32 KB of shared memory

struct TopScratch {
    int hist[256];
    int warp_gt[kTopThreads / 32], warp_eq[kTopThreads / 32];
    uint32_t prefix;
    int left;
};

__device__ __forceinline__ uint32_t score_key(float x) {
    if (x != x) return 0u;
    const uint32_t u = __float_as_uint(x + 0.f);  // -0 -> +0
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Indices of the kk largest of keys[0, n), 1 <= kk < n, ascending, into out[0, kk) (shared or global
// memory).  All kTopThreads threads take part; keys must be visible to all of them on entry, and out is
// not to be read before the next barrier.
__device__ __forceinline__ void top_ascending(const uint32_t *keys, int n, int kk, int32_t *out, TopScratch &sc) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint32_t prefix = 0;
    int left = kk;  // how many of the keys that share the prefix are still to be chosen
#pragma unroll 1
    for (int shift = 24; shift >= 0; shift -= 8) {
        sc.hist[tid] = 0;
        __syncthreads();
        const uint32_t mask = shift == 24 ? 0u : (0xFFFFFFFFu << (shift + 8));
        for (int i = tid; i < n; i += kTopThreads) {
            const uint32_t key = keys[i];
            if ((key & mask) == prefix) atomicAdd(&sc.hist[(key >> shift) & 255u], 1);
        }
        __syncthreads();
        if (warp == 0) {  // lane l: digits 255 - 8l .. 248 - 8l, counted from the top
            int c[8], sum = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                c[i] = sc.hist[255 - 8 * lane - i];
                sum += c[i];
            }
            int upto = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto += v;
            }
            int before = upto - sum;
            if (before < left && upto >= left) {  // exactly one lane
                int digit = 0;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if (before < left && before + c[i] >= left) {
                        digit = 255 - 8 * lane - i;
                        sc.left = left - before;
                    }
                    before += c[i];
                }
                sc.prefix = prefix | (static_cast<uint32_t>(digit) << shift);
            }
        }
        __syncthreads();
        prefix = sc.prefix;
        left = sc.left;
    }
    // prefix = the kk-th largest key; `left` of the keys equal to it are chosen, lowest index first
    int at = 0, eq_at = 0;
    for (int i0 = 0; i0 < n; i0 += kTopThreads) {
        const int i = i0 + tid;
        const uint32_t key = i < n ? keys[i] : 0u;
        const bool gt = i < n && key > prefix, eq = i < n && key == prefix;
        const unsigned bg = __ballot_sync(0xffffffffu, gt), be = __ballot_sync(0xffffffffu, eq);
        __syncthreads();  // the last step's counts have been read
        if (lane == 0) {
            sc.warp_gt[warp] = __popc(bg);
            sc.warp_eq[warp] = __popc(be);
        }
        __syncthreads();
        int gt_before = 0, eq_before = 0, gt_all = 0, eq_all = 0;
#pragma unroll
        for (int w = 0; w < kTopThreads / 32; ++w) {
            const int g = sc.warp_gt[w], e = sc.warp_eq[w];
            if (w < warp) gt_before += g, eq_before += e;
            gt_all += g, eq_all += e;
        }
        const unsigned below = (1u << lane) - 1u;
        gt_before += __popc(bg & below);
        eq_before += __popc(be & below);
        // chosen before this index: all larger keys, and of the equal ones at most `left`
        const int rank = at + gt_before + min(eq_at + eq_before, left) - min(eq_at, left);
        if (gt || (eq && eq_at + eq_before < left)) out[rank] = i;
        at += gt_all + min(eq_at + eq_all, left) - min(eq_at, left);
        eq_at += eq_all;
    }
}

// The same for n < 1024 by one warp, the keys in its registers (KPL per lane, n <= 32 * KPL): the kk-th
// largest key is found two bits at a time from the first bit in which the keys differ (three candidates'
// counts, 11 bits each, in one warp sum), stopping early at a candidate with exactly kk keys at or above it.
// No barrier.  (Calls in a captured graph: eviction of one of 17 blocks 7.6 us, sparse decode of 64 caches with 16 of
// up to 256 blocks 66.2 us, of 64 caches with 16 of up to 128 40.5 us; with the CTA's counts 9.1, 66.7 and 41.6 us.)
template <int KPL>
__device__ __forceinline__ void top_ascending_warp(const uint32_t *keys, int n, int kk, int32_t *out, int lane) {
    uint32_t key[KPL], hi = 0u, lo = 0xFFFFFFFFu;
#pragma unroll
    for (int i = 0; i < KPL; ++i) {
        const int j = 32 * i + lane;
        key[i] = j < n ? keys[j] : 0u;  // never at or above a candidate
        if (j < n) hi = max(hi, key[i]), lo = min(lo, key[i]);
    }
    hi = __reduce_max_sync(0xffffffffu, hi);
    lo = __reduce_min_sync(0xffffffffu, lo);
    uint32_t tau = hi;
    bool exact = false;
    if (hi != lo) {
        int b = (31 - __clz(hi ^ lo)) | 1;
        tau = b == 31 ? 0u : hi & (0xFFFFFFFFu << (b + 1));  // at least kk keys are >= tau throughout
#pragma unroll 1
        for (; b > 0 && !exact; b -= 2) {
            const uint32_t c1 = tau + (1u << (b - 1)), c2 = tau + (2u << (b - 1)), c3 = tau + (3u << (b - 1));
            uint32_t k1 = 0, k2 = 0, k3 = 0;  // (chains of their own: one sum of all would be three times as long)
#pragma unroll
            for (int i = 0; i < KPL; ++i) {
                k1 += key[i] >= c1 ? 1u : 0u;
                k2 += key[i] >= c2 ? 1u << 11 : 0u;
                k3 += key[i] >= c3 ? 1u << 22 : 0u;
            }
            const uint32_t cnt = __reduce_add_sync(0xffffffffu, k1 + k2 + k3);
            const int n1 = cnt & 2047, n2 = (cnt >> 11) & 2047, n3 = cnt >> 22;
            int m = n;
            if (n3 >= kk)
                tau = c3, m = n3;
            else if (n2 >= kk)
                tau = c2, m = n2;
            else if (n1 >= kk)
                tau = c1, m = n1;
            exact = m == kk;
        }
    }
    int left = 0;  // of the keys equal to tau, lowest index first
    if (!exact) {
        unsigned gt = 0;
#pragma unroll
        for (int i = 0; i < KPL; ++i) gt += key[i] > tau ? 1u : 0u;
        left = kk - static_cast<int>(__reduce_add_sync(0xffffffffu, gt));
    }
    const unsigned below = (1u << lane) - 1u;
    int at = 0, eq_at = 0;
#pragma unroll
    for (int i = 0; i < KPL; ++i) {
        if (32 * i >= n) break;
        const bool in = 32 * i + lane < n, eq = !exact && in && key[i] == tau;
        const unsigned be = __ballot_sync(0xffffffffu, eq);
        const bool chosen = in && (exact ? key[i] >= tau : key[i] > tau || (eq && eq_at + __popc(be & below) < left));
        const unsigned bc = __ballot_sync(0xffffffffu, chosen);
        if (chosen) out[at + __popc(bc & below)] = 32 * i + lane;
        at += __popc(bc);
        eq_at += __popc(be);
    }
}

// Either of the two, by the number of keys (uniform over the CTA).
__device__ __forceinline__ void top_blocks(const uint32_t *keys, int n, int kk, int32_t *out, TopScratch &sc) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (n <= 256) {
        if (warp == 0) top_ascending_warp<8>(keys, n, kk, out, lane);
    } else if (n < 1024) {
        if (warp == 0) top_ascending_warp<32>(keys, n, kk, out, lane);
    } else {
        top_ascending(keys, n, kk, out, sc);
    }
}

}  // namespace ssa
