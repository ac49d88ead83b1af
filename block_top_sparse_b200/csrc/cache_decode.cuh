// cache_decode.cuh -- attention of one new token per sequence over the 8-bit
// cache of cache8.cuh, over all blocks (k = 0) or over the own block and the
// k - 1 highest-scoring ones before it.
//
//   logit_u = scale * q . (Kscale * K8_u),  p = softmax over u <= L,
//   o = sum_u p_u * (Vscale * V8_u),        lse = log sum_u exp(logit_u)
// and, on demand, the attention weight of every block, sum_h sum_{u in j} p_hu.
//
// Bound by reading the cache: 2 d bytes per key and key head, half of what a
// bf16 cache costs.  A group of G query heads shares each key, so on CUDA cores
// the conversions and 4 d G operations per key would take longer than the read
// from G = 4 on; both products therefore run on the tensor cores on the codes
// as they are (tcgen05 kind::f8f6f4, nothing is converted or copied), and the
// other operand is brought to e4m3 without losing its precision, as a sum of
// terms of 4 significant bits each:
//   q = 2^e (t0 + t1/16):          8 significant bits (bf16) in two terms, or 2^-22 of the
//                                  head's largest element,
//   p = (t0 + t1/16 + t2/256 + t3/4096)/256: 16 bits, error <= 2^-16 p (four roundings,
//                                  each at most 2^-4 of what is left) + 2^-30 of a tile's largest.
// (Three terms, 12 bits, showed where values cancel: of two weights 2^-10 apart, the difference was off by up to 9 %,
// with four by 0.24 %, less than its rounding to bf16.)
// The terms are extra columns (N) of the same product, and its results are put
// together in fp32; N is small and the tensor cores have time to spare.
//
//   cache_select_kernel    one CTA per (sequence, key head): block scores and
//                          the top k - 1 (top_blocks.cuh).  Scores are summed
//                          in fp64 and rounded to fp32 once, so which blocks
//                          are chosen does not depend on the order of summation;
//   cache_attend_kernel    a fixed grid; every CTA takes an equal share of all
//                          the tiles of 128 keys of all (sequence, key head)
//                          pairs, so long and short sequences balance, and
//                          writes an unnormalised partial output, maximum and
//                          sum for each pair that it touches;
//   cache_combine_kernel   joins a pair's partials in a fixed order; block weights
//                          from the blocks' own maxima and sums.
// Atomics only where their order does not matter (maxima, counts): results are the same from run to run.
#pragma once

#include <cooperative_groups.h>

#include "cache8.cuh"
#include "device.cuh"
#include "top_blocks.cuh"

namespace ssa {

constexpr int kCacheMaxGroup = 32;  // query heads per key head
constexpr int kCacheSms = 148;

// Blocks attended and tiles of 128 keys of one key head whose newest token is at position L.
__device__ __forceinline__ int cache_slots(int L, int T, int s, int k) {
    if (L < 0 || L >= T) return 0;
    const int nblk = L / s + 1;
    return k > 0 ? min(k, nblk) : nblk;
}
__device__ __forceinline__ int cache_tiles(int L, int T, int s, int k) {
    const int n = cache_slots(L, T, s, k);
    return s == 128 ? n : (n + 1) >> 1;
}

// ---------------------------------------------------------------------------
// Selection
// ---------------------------------------------------------------------------
// A cluster of CTAs per (sequence, key head), one where there are many pairs: the CTAs share the rows and put
// their scores into the first one's shared memory (nb keys), which chooses.  k >= 1.
__global__ void __launch_bounds__(kTopThreads, 4) cache_select_kernel(const int32_t *__restrict__ cache_len,
                                                                   const __nv_bfloat16 *__restrict__ q,
                                                                   const float *__restrict__ Kbar,
                                                                   int32_t *__restrict__ idx, int Hk, int G, int T,
                                                                   int s, int k, int nb) {
    extern __shared__ uint32_t select_key[];
    __shared__ TopScratch sc;
    __shared__ double qs[kCacheD];
    grid_dependents_launch();
    namespace cg = cooperative_groups;
    const int parts = static_cast<int>(cg::this_cluster().num_blocks()), part_id = static_cast<int>(cg::this_cluster().block_rank());
    const int bh = blockIdx.x / parts, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    constexpr int R = 8, kWarps = kTopThreads / 32;  // rows in flight per warp, four elements per lane
    const int first = R * (part_id * kWarps + warp), stride = R * kWarps * parts;
    const int L = __ldg(cache_len + bh / Hk);
    int32_t *out = idx + static_cast<size_t>(bh) * k;
    // the first rows (whether they count or not) and the query are asked for before the length is known
    float4 v[R];
    const float4 *kb = reinterpret_cast<const float4 *>(Kbar + static_cast<size_t>(bh) * nb * kCacheD) + lane;
    auto load = [&](int i, int j, int n) {
        v[i] = j < n ? __ldg(kb + static_cast<size_t>(j) * (kCacheD / 4)) : make_float4(0.f, 0.f, 0.f, 0.f);
    };
    if (k > 1) {
#pragma unroll
        for (int i = 0; i < R; ++i) load(i, first + i, nb);
        if (tid < kCacheD) {
            double sum = 0.0;
            const __nv_bfloat16 *qr = q + static_cast<size_t>(bh) * G * kCacheD + tid;
#pragma unroll 4
            for (int h = 0; h < G; ++h) sum += static_cast<double>(__bfloat162float(qr[h * kCacheD]));
            qs[tid] = sum;
        }
    }
    if (L < 0 || L >= T) {  // (the cluster's CTAs go the same way here and below)
        if (part_id == 0)
            for (int i = tid; i < k; i += kTopThreads) out[i] = -1;
        return;
    }
    const int bt = L / s, want = min(k - 1, bt);
    if (part_id > 0 && (want == bt || want == 0)) return;
    if (want == bt) {
        for (int i = tid; i < want; i += kTopThreads) out[i] = i;
    } else if (want > 0) {
        if (parts > 1)
            cg::this_cluster().sync();  // the first CTA runs: its shared memory may be written
        else
            __syncthreads();
        double q4[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) q4[i] = qs[4 * lane + i];
        uint32_t *keys = parts > 1 ? cg::this_cluster().map_shared_rank(select_key, 0) : select_key;
        for (int j0 = first; j0 < bt; j0 += stride) {
#pragma unroll
            for (int half = 0; half < R; half += 4) {
                double part[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float4 x = v[half + i];
                    part[i] = fma(q4[0], static_cast<double>(x.x), q4[1] * static_cast<double>(x.y)) +
                              fma(q4[2], static_cast<double>(x.z), q4[3] * static_cast<double>(x.w));
                    load(half + i, j0 + half + i + stride, bt);  // the next rows arrive during the sums
                }
                // butterfly: two steps hand each lane the sum of one row over 8 lanes, three more the whole sum
#pragma unroll
                for (int off = 16, n = 2; n >= 1; off >>= 1, n >>= 1) {
                    const bool up = (lane & off) != 0;
#pragma unroll
                    for (int i = 0; i < n; ++i) {
                        const double send = up ? part[i] : part[i + n], mine = up ? part[i + n] : part[i];
                        part[i] = mine + __shfl_xor_sync(0xffffffffu, send, off);
                    }
                }
#pragma unroll
                for (int off = 4; off > 0; off >>= 1) part[0] += __shfl_xor_sync(0xffffffffu, part[0], off);
                const int j = j0 + half + (lane >> 3);  // lane bit 4: row bit 1, lane bit 3: row bit 0
                if ((lane & 7) == 0 && j < bt) keys[j] = score_key(static_cast<float>(part[0]));
            }
        }
        if (parts > 1)
            cg::this_cluster().sync();
        else
            __syncthreads();
        if (part_id > 0) return;
        top_blocks(select_key, bt, want, out, sc);
    }
    for (int i = want + tid; i < k; i += kTopThreads) out[i] = i == want ? bt : -1;
}

// ---------------------------------------------------------------------------
// Attention
// ---------------------------------------------------------------------------
// Workspace: partial outputs, one slot for every (CTA, pair) that can meet (slot = CTA + pair, distinct since
// either grows along the tiles), their (maximum in log2 units, sum); per query head and attended block the
// same pair for the block alone.
__host__ __device__ __forceinline__ size_t cache_partials(size_t ctas, size_t pairs) { return ctas + pairs; }

// Position in the sequence of tiles: pair (b, hk), tile t of its nt.
struct TilePos {
    int b, hk, t, nt, L;
    __device__ __forceinline__ void next(const int32_t *cache_len, int B, int Hk, int T, int s, int k) {
        if (++t < nt) return;
        t = 0;
        if (++hk < Hk) return;
        hk = 0;
        for (++b; b < B; ++b) {
            L = __ldg(cache_len + b);
            nt = cache_tiles(L, T, s, k);
            if (nt > 0) return;
        }
    }
};

// Tiles of all sequences (times Hk: of all pairs), counted by one warp.
__device__ __forceinline__ int64_t cache_total_tiles(const int32_t *cache_len, int B, int Hk, int T, int s, int k,
                                                     int lane) {
    int64_t n = 0;
    for (int b = lane; b < B; b += 32) n += cache_tiles(__ldg(cache_len + b), T, s, k);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
    return n * Hk;
}

// Tiles of the sequences before b, by one warp.
__device__ __forceinline__ int64_t cache_tiles_before(const int32_t *cache_len, int b, int T, int s, int k, int lane) {
    int64_t n = 0;
    for (int i = lane; i < b; i += 32) n += cache_tiles(__ldg(cache_len + i), T, s, k);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
    return n;
}

// The pair and tile of global tile g, by one warp.
__device__ __forceinline__ TilePos cache_locate(const int32_t *cache_len, int64_t g, int B, int Hk, int T, int s, int k,
                                                int lane) {
    TilePos p;
    int64_t before = 0;
    for (int b0 = 0; b0 < B; b0 += 32) {
        const int L = b0 + lane < B ? __ldg(cache_len + b0 + lane) : -1;
        const int nt = cache_tiles(L, T, s, k);
        int64_t upto = static_cast<int64_t>(nt) * Hk;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t v = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += v;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, before + upto > g);
        if (hit) {
            const int l = __ffs(hit) - 1;
            p.b = b0 + l;
            p.nt = __shfl_sync(0xffffffffu, nt, l);
            p.L = __shfl_sync(0xffffffffu, L, l);
            const int64_t start = before + __shfl_sync(0xffffffffu, upto, l) - static_cast<int64_t>(p.nt) * Hk;
            const int at = static_cast<int>(g - start);
            p.hk = at / p.nt;
            p.t = at % p.nt;
            return p;
        }
        before += __shfl_sync(0xffffffffu, upto, 31);
    }
    p.b = B;  // not reached: g is below the total
    p.hk = p.t = p.L = 0;
    p.nt = 1;
    return p;
}

// Query heads per key head are padded to NH = 4, 8, 16 or 32.
template <int NH>
struct CacheAttend {
    static constexpr int kTile = 128 * kCacheD;                      // 16 KB: keys or values of one tile
    static constexpr int kNS = NH < 8 ? 16 : 2 * NH;                 // columns of the logits' product (term * NH + head)
    static constexpr int kNP = 4 * NH;                               // columns of the output's product
    static constexpr int kQ = 2 * kTile;                             // [kNS][128 B]
    static constexpr int kP = kQ + kNS * 128;                        // [kNP / 16][128 keys][16 B]
    static constexpr int kRed = kP + kNP * 128;                      // two of: [NH][4 warps] sums
    static constexpr int kHead = kRed + 2 * NH * 16;                 // [3][NH] factors, [3][2][NH] maxima
    static constexpr int kBar = kHead + 9 * NH * 4;
    static constexpr int kBytes = kBar + 64 + 1024;                  // + alignment of the dynamic base to 1024 B
    // the logits' columns may be written again while the outputs are read, except at NH = 32, where both
    // products would take 192 columns a CTA (256 allocated) and the outputs take the logits' place
    static constexpr bool kApart = NH < 32;
    static constexpr int kTmemO = kApart ? kNS : 0;                  // first column of the output's product
    static constexpr int kCols = kTmemO + kNP;
    static constexpr int kTmemCols = kCols <= 32 ? 32 : kCols <= 64 ? 64 : 128;
    // CTAs per SM.  64 caches of 16K to 32K tokens, 8 key heads, G = 4: 461 us with three, 453 us with four, 475 us
    // with five; 16 ragged ones, G = 8, blocks of 64: 45, 35 and 35 us.  NH = 32, 64 caches of 8K to 16K tokens, one key
    // head, blocks of 128 and 64: 75 and 86 us with three (168 registers, 124 and 164 bytes spilled), 78 and 94 us with
    // two (nothing spilled).
    static constexpr int kPerSm = NH <= 16 ? 4 : 3;
};

// Tile of 128 keys (one block of 128 or two of 64):
//   S^T [128 keys x 2 NH] = K8 . (q terms)^T      A: keys as loaded (K-major), thread = key
//   weights of the thread's key against the tile's maxima, split into four terms
//   O^T [128 dims x 4 NH] = V8^T . (p terms)^T    A: values as loaded (M-major), thread = dim
// A tile's weights are relative to its own maximum, so their 2^-30 is of the tile's largest weight, however much
// larger another tile's is; where the values of two blocks of 64 in a tile have scales more than 2^6 apart, it is
// of the largest product of weight and scale.  The outputs stay in registers, brought to the running maximum tile
// by tile; only O^T of one tile is in tensor memory.  A tile is a chain of dependent steps (product, maximum, weights, product, output), so the CTA is
// kept small -- one tile of keys and one of values, each loaded again as soon as its product has read it --
// and up to four CTAs per SM run their chains beside one another's loads: 128 KB in flight or in use per SM.
// (Two tiles of each and three CTAs per SM: 784 us instead of 481 us for 64 caches of 16K to 32K tokens, 8 key
// heads, G = 4; 458 us, 7.0 TB/s, with the steps since.)
template <int NH, int S>
__global__ void __launch_bounds__(128, CacheAttend<NH>::kPerSm) cache_attend_kernel(
    const __grid_constant__ CUtensorMap mapK, const __grid_constant__ CUtensorMap mapV,
    const int32_t *__restrict__ cache_len, const __nv_bfloat16 *__restrict__ q, const float *__restrict__ Kscale,
    const float *__restrict__ Vscale, const int32_t *idx, float *__restrict__ opart, float2 *__restrict__ mlpart,
    float2 *__restrict__ block_ml, int B, int Hk, int G, int T, int k, int nb, float scale_log2) {
    using SM = CacheAttend<NH>;
    constexpr int kPer = 128 / S;  // blocks of a tile
    extern __shared__ __align__(1024) uint8_t cad_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(cad_raw) + 1023) & ~uintptr_t(1023));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t sK = smem_u32(smem), sV = sK + SM::kTile, sQ = sK + SM::kQ, sP = sK + SM::kP;
    // per head: logit factor; what a tile multiplies the outputs so far by, and its own
    float *head_f = reinterpret_cast<float *>(smem + SM::kHead), *head_old = head_f + NH, *head_new = head_f + 2 * NH;
    // maxima of a tile per block and head, raised by the warps; three in turn, the one after the next being reset
    // while others may already raise the next
    float *tile_m = head_f + 3 * NH;
    // maximum of no key: below every finite logit, so that a masked or overflowing one (-inf) weighs 0
    constexpr float kLowest = -3.4e38f;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + SM::kBar);
    uint64_t *bar_k = bars, *bar_v = bars + 1, *bar_s = bars + 2, *bar_o = bars + 3;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 4);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(bars + 5);

    // Tensor memory first: the SM starts its next CTA only when this one has given up the right to allocate
    // (measured with five: with the allocation behind the search below the fifth CTA of an SM started 7.4 us after
    // the first, now 2.2 us; 16 ragged sequences of up to 32K tokens 38 -> 36 us in all).
    if (warp == 1) {
        tmem_alloc(tmem_slot, SM::kTmemCols);
        tmem_relinquish();
    }
    grid_dependents_launch();  // (takes effect once every CTA of this grid has started)

    // this CTA's share of the tiles
    const int64_t total = cache_total_tiles(cache_len, B, Hk, T, S, k, lane);
    if (blockIdx.x == 0)
        for (int b = tid; b < B; b += 128) {
            const int L = __ldg(cache_len + b);
            if (L < -1 || L >= T) record_error(ERR_CACHE_INPUT, 0x703);
        }
    const int64_t ctas = min(static_cast<int64_t>(gridDim.x), total);
    if (static_cast<int64_t>(blockIdx.x) >= ctas) {
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
        if (warp == 1) tmem_dealloc(*tmem_slot, SM::kTmemCols);
        grid_dependency_wait();
        return;
    }
    const int64_t g0 = blockIdx.x * total / ctas;
    const int n_tiles = static_cast<int>((blockIdx.x + 1) * total / ctas - g0);
    TilePos cur = cache_locate(cache_len, g0, B, Hk, T, S, k, lane);

    struct Blocks {
        int v[kPer];  // -1: none
    };
    auto blocks_of = [&](const TilePos &p) {
        Blocks r;
        const int bt = p.L / S;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int slot = p.t * kPer + i;
            if (k > 0)
                r.v[i] = slot < k ? __ldcg(idx + (static_cast<size_t>(p.b) * Hk + p.hk) * k + slot) : -1;
            else
                r.v[i] = slot;
            if (r.v[i] > bt) r.v[i] = -1;
        }
        return r;
    };
    // (one thread) the keys or values of one tile
    auto load = [&](const CUtensorMap *map, uint64_t *bar, uint32_t off, const TilePos &p, const Blocks &r) {
        uint32_t bytes = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (r.v[i] >= 0) bytes += S * kCacheD;
        mbar_arrive_expect_tx(bar, bytes);
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (r.v[i] >= 0)  // (the host keeps B * Hkv * T below 2^31)
                tma_load_2d(map, bar, smem + off + i * S * kCacheD, 0, (p.b * Hk + p.hk) * T + r.v[i] * S);
    };
    struct Scales {
        float k, v[2];  // of this key's block; of the tile's blocks (0: none)
    };
    auto scales_of = [&](const TilePos &p, const Blocks &r) {
        const size_t at = (static_cast<size_t>(p.b) * Hk + p.hk) * nb;
        Scales c{0.f, {0.f, 0.f}};
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (r.v[i] >= 0) {
                c.v[i] = __ldg(Vscale + at + r.v[i]);
                if (i == tid / S) c.k = __ldg(Kscale + at + r.v[i]);
            }
        return c;
    };

    constexpr int kLoader = 96;  // the thread that issues the loads (thread 0 issues the products)
    if (tid == kLoader) {
        for (int i = 0; i < 4; ++i) mbar_init(bars + i, 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    grid_dependency_wait();  // the selection (k > 0) has been written
    Blocks blk = blocks_of(cur), blk1 = blk, blk2 = blk;
    int loads_k = 0, loads_v = 0, products_s = 0, products_o = 0;  // issued by this thread
    if (tid == kLoader) {
        load(&mapK, bar_k, 0, cur, blk);
        load(&mapV, bar_v, SM::kTile, cur, blk);
        loads_k = loads_v = 1;
    }
    // rows of heads past G stay zero: logits 0, nothing of them is written
    for (int e = tid; e < SM::kNS * 8; e += 128)
        *reinterpret_cast<uint4 *>(smem + SM::kQ + e * 16) = make_uint4(0u, 0u, 0u, 0u);
    if (tid < NH) head_f[tid] = 0.f;
    for (int e = tid; e < 6 * NH; e += 128) tile_m[e] = kLowest;
    Scales sc = scales_of(cur, blk), sc1 = sc;
    TilePos pos1 = cur, pos2;
    if (n_tiles > 1) {
        pos1.next(cache_len, B, Hk, T, S, k);
        blk1 = blocks_of(pos1);
    }
    pos2 = pos1;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    auto leave = [&](bool failed) {
        if (failed) {  // let the loads and products in flight finish
            if (loads_k) mbar_drain(bar_k, (loads_k - 1) & 1);
            if (loads_v) mbar_drain(bar_v, (loads_v - 1) & 1);
            if (products_s) mbar_drain(bar_s, (products_s - 1) & 1);
            if (products_o) mbar_drain(bar_o, (products_o - 1) & 1);
        }
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
        if (warp == 1) tmem_dealloc(tmem, SM::kTmemCols);
    };
    auto product_s = [&]() {  // (thread 0) the keys have landed
        tc_fence_after();
        constexpr uint32_t id = idesc_e4m3(128, SM::kNS, false, false);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
            mma_e4m3_ss(tmem, smem_desc_sw128(sK + kk * 32, 16), smem_desc_sw128(sQ + kk * 32, 16), id, kk > 0 ? 1u : 0u);
        mma_commit(bar_s);
        ++products_s;
    };

    // rows of the next group's queries, asked for one tile ahead (up to 16 heads: registers)
    constexpr int kQRows = NH <= 16 ? NH / 4 : 1;
    uint2 q_next[kQRows];
    auto load_q = [&](int bh) {
#pragma unroll
        for (int i = 0; i < kQRows; ++i)
            if (warp + 4 * i < G)
                q_next[i] = __ldg(reinterpret_cast<const uint2 *>(
                                      q + (static_cast<size_t>(bh) * G + warp + 4 * i) * kCacheD) + lane);
    };
    if (NH <= 16) load_q(cur.b * Hk + cur.hk);

    uint64_t o[NH / 2];  // outputs of heads 2 i and 2 i + 1, this thread's dim
    float m_run = kLowest, l_run = 0.f;  // (threads below NH) the head's maximum and sum
    int pair = -1, turn = 0;
    bool failed = false;
    for (int it = 0; it < n_tiles; ++it) {
        const uint32_t ph = it & 1;
        const int bh = cur.b * Hk + cur.hk;
        const bool last = it + 1 == n_tiles || pos1.b * Hk + pos1.hk != bh;  // of this pair
        // the next tile's scales and the one after's blocks arrive during this tile
        if (it + 1 < n_tiles) sc1 = scales_of(pos1, blk1);
        if (it + 2 < n_tiles) {
            pos2.next(cache_len, B, Hk, T, S, k);
            blk2 = blocks_of(pos2);
        }
        if (bh != pair) {  // a new group of query heads: two terms per element, two rows per head
            pair = bh;
#pragma unroll
            for (int i = 0; i < NH / 4; ++i) {
                const int h = warp + 4 * i;
                if (h >= G) break;
                const uint2 w = NH <= 16 ? q_next[i < kQRows ? i : 0]
                                         : __ldg(reinterpret_cast<const uint2 *>(
                                                     q + (static_cast<size_t>(bh) * G + h) * kCacheD) + lane);
                const float x[4] = {__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u),
                                    __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xFFFF0000u)};
                uint32_t top = 0;
#pragma unroll
                for (int e = 0; e < 4; ++e) top = max(top, __float_as_uint(x[e]) & 0x7FFFFFFFu);
                top = __reduce_max_sync(0xffffffffu, top);
                const bool finite = top < 0x7F800000u;
                const float unit = finite ? e4m3_scale(__uint_as_float(top)) : 1.f, inv = pow2_inverse(unit);
                uint32_t t0 = 0, t1 = 0;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float a = x[2 * e] * inv, c = x[2 * e + 1] * inv;
                    const uint16_t hi = pack_e4m3x2(a, c);
                    const float2 f = unpack_e4m3x2(hi);
                    t0 |= static_cast<uint32_t>(hi) << (16 * e);
                    t1 |= static_cast<uint32_t>(pack_e4m3x2((a - f.x) * 16.f, (c - f.y) * 16.f)) << (16 * e);
                }
                const int unit16 = lane >> 2, in16 = (lane & 3) * 4, h1 = NH + h;
                *reinterpret_cast<uint32_t *>(smem + SM::kQ + h * 128 + ((unit16 ^ (h & 7)) << 4) + in16) = t0;
                *reinterpret_cast<uint32_t *>(smem + SM::kQ + h1 * 128 + ((unit16 ^ (h1 & 7)) << 4) + in16) = t1;
                if (lane == 0) {
                    // an infinity or NaN in the query makes the row's results NaN, not large
                    head_f[h] = finite ? unit * scale_log2 : __int_as_float(0x7FC00000);
                }
            }
#pragma unroll
            for (int i = 0; i < NH / 2; ++i) o[i] = 0;
            m_run = kLowest, l_run = 0.f;
            fence_proxy_async_smem();
            __syncthreads();
        }
        if (NH <= 16 && last && it + 1 < n_tiles) load_q(pos1.b * Hk + pos1.hk);
        bool ok = true;
        if (tid == 0 && products_s == it) {
            ok = mbar_wait(bar_k, ph, abort_flag, 0x711);
            if (ok) product_s();
        }
        ok = ok && mbar_wait(bar_s, ph, abort_flag, 0x712);
        tc_fence_after();
        if (tid == kLoader && ok && it + 1 < n_tiles) {  // the keys have been read
            load(&mapK, bar_k, 0, pos1, blk1);
            ++loads_k;
        }
        const int my_blk = kPer == 1 ? blk.v[0] : (tid < S ? blk.v[0] : blk.v[kPer - 1]);
        const bool valid = my_blk >= 0 && my_blk * S + tid % S <= cur.L;
        float *red_l = reinterpret_cast<float *>(smem + SM::kRed + (it & 1) * NH * 16);
        float *now_m = tile_m + turn * 2 * NH;  // block, head
        uint64_t p[NH / 2];  // logits, then weights, of heads 2 i and 2 i + 1
        {
            const uint32_t row = tmem + (static_cast<uint32_t>(warp * 32) << 16);
            const uint64_t sixteenth = f2_pack(0.0625f, 0.0625f);
            auto join = [&](const float *t0, const float *t1) {
#pragma unroll
                for (int i = 0; i < NH / 2; ++i)
                    p[i] = ffma2(f2_pack(t1[2 * i], t1[2 * i + 1]), sixteenth, f2_pack(t0[2 * i], t0[2 * i + 1]));
            };
            if constexpr (NH <= 8) {
                float v[16];
                tmem_ld16(row, v);
                join(v, v + NH);
            } else if constexpr (NH == 16) {
                float v[32];
                tmem_ld32(row, v);
                join(v, v + 16);
            } else {
                float v[32], w[32];
                tmem_ld32(row, v);
                tmem_ld32(row + 32, w);
                join(v, w);
            }
        }
        {
            const uint64_t kk = f2_pack(sc.k, sc.k);
            float mine = 0.f;  // the warp's maximum of head `lane`
#pragma unroll
            for (int i = 0; i < NH / 2; ++i) {
                p[i] = fmul2(p[i], fmul2(kk, *reinterpret_cast<const uint64_t *>(head_f + 2 * i)));
                float a, c;
                f2_unpack(p[i], a, c);
                a = valid ? a : -INFINITY;
                c = valid ? c : -INFINITY;
                p[i] = f2_pack(a, c);
                const float ma = warp_max(a), mc = warp_max(c);
                mine = lane == 2 * i ? ma : lane == 2 * i + 1 ? mc : mine;
            }
            if (lane < NH) atomic_max_shared(now_m + tid / S * NH + lane, mine);
        }
        tc_fence_before();
        __syncthreads();
        // weights against the tile's maximum; for the product with the values in units of 1/256 of the tile's
        // largest value scale, or (wide) of its largest product of weight and scale
        float sum[NH];
        const float top = fmaxf(sc.v[0], sc.v[1]), low = fminf(sc.v[0], sc.v[1]);
        const bool wide = kPer == 2 && low > 0.f && top > 64.f * low;  // (uniform)
        auto tile_max = [&](int i) {  // of heads 4 i ..
            float4 m = *reinterpret_cast<const float4 *>(now_m + 4 * i);
            if (kPer == 2) {
                const float4 n = *reinterpret_cast<const float4 *>(now_m + NH + 4 * i);
                m.x = fmaxf(m.x, n.x), m.y = fmaxf(m.y, n.y), m.z = fmaxf(m.z, n.z), m.w = fmaxf(m.w, n.w);
            }
            return m;
        };
        // (wide) log2 of the largest product of weight and value scale of head h, weights against maximum m
        const float log0 = wide ? __log2f(sc.v[0]) : 0.f, log1 = wide ? __log2f(sc.v[1]) : 0.f;
        auto largest = [&](int h, float m) { return fmaxf(log0 + (now_m[h] - m), log1 + (now_m[NH + h] - m)); };
        {
            const float unit = kPer == 1 ? 256.f : top > 0.f ? 256.f * ((tid < S ? sc.v[0] : sc.v[1]) / top) : 0.f;
            const uint64_t unit2 = f2_pack(unit, unit);
#pragma unroll
            for (int i = 0; i < NH / 4; ++i) {
                const float4 m = tile_max(i);
                float a[4];
                f2_unpack(fadd2(p[2 * i], f2_pack(-m.x, -m.y)), a[0], a[1]);
                f2_unpack(fadd2(p[2 * i + 1], f2_pack(-m.z, -m.w)), a[2], a[3]);
#pragma unroll
                for (int e = 0; e < 4; ++e) sum[4 * i + e] = fast_exp2(a[e]);  // 0 for a masked key
                if (!wide) {
                    p[2 * i] = fmul2(f2_pack(sum[4 * i], sum[4 * i + 1]), unit2);
                    p[2 * i + 1] = fmul2(f2_pack(sum[4 * i + 2], sum[4 * i + 3]), unit2);
                } else {
                    const float mm[4] = {m.x, m.y, m.z, m.w}, own = (tid < S ? log0 : log1) + 8.f;
#pragma unroll
                    for (int e = 0; e < 4; ++e) a[e] = fast_exp2(a[e] + (own - largest(4 * i + e, mm[e])));
                    p[2 * i] = f2_pack(a[0], a[1]);
                    p[2 * i + 1] = f2_pack(a[2], a[3]);
                }
            }
        }
        float m_tile = 0.f, own_f = 0.f, old_f = 0.f;  // (threads below NH)
        if (tid < NH) {
            m_tile = kPer == 2 ? fmaxf(now_m[tid], now_m[NH + tid]) : now_m[tid];
            const float m = fmaxf(m_run, m_tile);
            old_f = fast_exp2(m_run - m);
            own_f = fast_exp2(m_tile - m);
            m_run = m;
            head_old[tid] = old_f;
            head_new[tid] = wide ? fast_exp2(m_tile - m + (largest(tid, m_tile) - 8.f)) : own_f * (top * (1.f / 256.f));
        }
        // sums over the warp: each step hands a lane half of the heads it holds
        {
            int n = NH / 2, off = 16;
#pragma unroll
            for (; n >= 1; n >>= 1, off >>= 1) {
                const bool up = (lane & off) != 0;
#pragma unroll
                for (int i = 0; i < NH / 2; ++i) {
                    if (i < n) {
                        const float send = up ? sum[i] : sum[i + n], mine = up ? sum[i + n] : sum[i];
                        sum[i] = mine + __shfl_xor_sync(0xffffffffu, send, off);
                    }
                }
            }
#pragma unroll
            for (; off >= 1; off >>= 1) sum[0] += __shfl_xor_sync(0xffffffffu, sum[0], off);
            constexpr int kLanes = 32 / NH;  // lanes that end up with the same head
            if (lane % kLanes == 0) red_l[lane / kLanes * 4 + warp] = sum[0];
        }
        // four terms of every weight into the N-major operand: byte term * NH + h of the key's row, rows of 16
        // bytes in groups of 2 KB (one 16-byte store per 16 bytes; key by key, single bytes would go to rows of
        // their own)
        {
            uint32_t w[SM::kNP / 4];
#pragma unroll
            for (int i = 0; i < SM::kNP / 4; ++i) w[i] = 0u;
#pragma unroll
            for (int h = 0; h < NH; h += 2) {
                uint64_t rest = p[h / 2];
#pragma unroll
                for (int term = 0; term < 4; ++term) {
                    float a, c;
                    f2_unpack(rest, a, c);
                    const uint16_t e = pack_e4m3x2(a, c);
                    w[(term * NH + h) / 4] |= static_cast<uint32_t>(e) << (h % 4 * 8);
                    // 16 (rest - e), exact
                    if (term < 3) rest = ffma2(unpack_e4m3x2_f2(e), f2_pack(-16.f, -16.f), fmul2(rest, f2_pack(16.f, 16.f)));
                }
            }
#pragma unroll
            for (int g = 0; g < SM::kNP / 16; ++g)
                *reinterpret_cast<uint4 *>(smem + SM::kP + g * 2048 + tid * 16) =
                    make_uint4(w[4 * g], w[4 * g + 1], w[4 * g + 2], w[4 * g + 3]);
        }
        ok = ok && mbar_wait(bar_v, ph, abort_flag, 0x713);
        if (ok && !valid) {  // whatever the cache holds behind the newest token must not meet even a weight of 0
            uint4 *row = reinterpret_cast<uint4 *>(smem + SM::kTile + tid * kCacheD);
#pragma unroll
            for (int i = 0; i < 8; ++i) row[i] = make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();
        tc_fence_before();
        if (__syncthreads_or(!ok || failed)) {
            leave(true);
            return;
        }
        if (tid == 0) {
            tc_fence_after();
            constexpr uint32_t id = idesc_e4m3(128, SM::kNP, true, true);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
                mma_e4m3_ss(tmem + SM::kTmemO, smem_desc_sw128(sV + kk * 4096, 16), smem_desc_mn8(sP + kk * 512, 128, 2048),
                            id, kk > 0 ? 1u : 0u);
            mma_commit(bar_o);
            ++products_o;
            // the next tile's logits follow at once where its keys are there and the query heads are the same
            if (SM::kApart && !last && mbar_test_wait(bar_k, ph ^ 1)) product_s();
        }
        // meanwhile: the head's running maximum and sum, and the blocks' own
        if (tid < NH) {
            const float4 rl = *reinterpret_cast<const float4 *>(red_l + tid * 4);
            const float l = (rl.x + rl.y) + (rl.z + rl.w);
            l_run = l_run * old_f + l * own_f;
            float *later = tile_m + (turn == 0 ? 2 : turn - 1) * 2 * NH + tid;  // those of the tile after the next
            later[0] = later[NH] = kLowest;
            if (block_ml && tid < G) {
                float2 *to = block_ml + (static_cast<size_t>(bh) * G + tid) * (k > 0 ? k : nb) + cur.t * kPer;
                if (kPer == 1) {
                    to[0] = make_float2(m_tile, l);
                } else {
                    to[0] = make_float2(m_tile, rl.x + rl.y);
                    if (blk.v[kPer - 1] >= 0) to[1] = make_float2(m_tile, rl.z + rl.w);
                }
            }
        }
        ok = mbar_wait(bar_o, ph, abort_flag, 0x714);
        failed = !ok;  // (met at the next tile's barrier, or at the end)
        tc_fence_after();
        if (tid == kLoader && ok && it + 1 < n_tiles) {  // the values have been read
            load(&mapV, bar_v, SM::kTile, pos1, blk1);
            ++loads_v;
        }
        {
            const uint32_t row = tmem + SM::kTmemO + (static_cast<uint32_t>(warp * 32) << 16);
            const uint64_t sixteenth = f2_pack(0.0625f, 0.0625f);
            auto factor = [&](const float *f, int i) { return *reinterpret_cast<const uint64_t *>(f + 2 * i); };
            uint64_t acc[NH / 2];  // the terms so far, the smallest first
            auto add = [&](const float *t, bool first) {
#pragma unroll
                for (int i = 0; i < NH / 2; ++i) {
                    const uint64_t x = f2_pack(t[2 * i], t[2 * i + 1]);
                    acc[i] = first ? x : ffma2(acc[i], sixteenth, x);
                }
            };
            if constexpr (NH == 4) {
                float v[16];
                tmem_ld16(row, v);
#pragma unroll
                for (int term = 3; term >= 0; --term) add(v + 4 * term, term == 3);
            } else {
                constexpr int kTerms = 32 / NH;  // of 32 columns
#pragma unroll
                for (int part = 4 / kTerms - 1; part >= 0; --part) {
                    float v[32];
                    tmem_ld32(row + 32 * part, v);
#pragma unroll
                    for (int term = kTerms - 1; term >= 0; --term)
                        add(v + NH * term, part * kTerms + term == 3);
                }
            }
#pragma unroll
            for (int i = 0; i < NH / 2; ++i) o[i] = ffma2(acc[i], factor(head_new, i), fmul2(o[i], factor(head_old, i)));
            tc_fence_before();
        }
        if (last) {
            const size_t slot = static_cast<size_t>(blockIdx.x) + bh;
            float *to = opart + slot * G * kCacheD + tid;
#pragma unroll
            for (int i = 0; i < NH / 2; ++i) {
                float a, c;
                f2_unpack(o[i], a, c);
                if (2 * i < G) to[2 * i * kCacheD] = a;
                if (2 * i + 1 < G) to[(2 * i + 1) * kCacheD] = c;
            }
            if (tid < G) mlpart[slot * G + tid] = make_float2(m_run, l_run);
        } else if (!SM::kApart) {
            __syncthreads();  // every warp has read its outputs before the next logits take their place
        }
        cur = pos1;
        pos1 = pos2;
        blk = blk1;
        blk1 = blk2;
        sc = sc1;
        turn = turn == 2 ? 0 : turn + 1;
    }
    leave(__syncthreads_or(failed) != 0);
}

// ---------------------------------------------------------------------------
// Joining the partials: M = max m_i, l = sum 2^(m_i - M) l_i, o = sum 2^(m_i - M) o_i / l, in the order of the
// CTAs; the attention weight of the blocks from their own maxima and sums.  Where there are many pairs of few
// partials a CTA takes eight heads of a pair, a warp each, then its share of the pair's blocks (SPLIT = 0).  Where a pair is
// split over many CTAs, the first head_ctas CTAs take one head (SPLIT = 1) or a quarter of one head's dims (4)
// each, and every CTA after them 256 blocks of one pair.  The whole call for B caches of 16K to 32K tokens, one key
// head, in a captured graph (us; 592 / B partials a pair), by form:
//   partials a pair       8     12     16     20     33     49     66     99    148
//   G = 4, form 0       77.7   57.7   47.1   42.2   35.4   34.7   36.8   40.8   55.3
//          form 1       76.1   54.9   42.6   36.5   25.8   20.9   18.4   15.8   14.0
//          form 4       84.5   59.8   46.4   38.9   25.7   20.4   17.0   13.9   12.3
//   G = 16, form 0      81.0   61.4   51.2   45.4   38.2   38.3   40.8   46.3   59.2
//           form 1      88.0   62.4   49.8   42.0   28.8   23.9   21.6   19.0   16.4
//           form 4     120.3   82.5   63.5   52.4   34.6   26.5   23.0   17.8   15.4
// Hence 1 from 16 partials a pair on and 4 from 64 on.  (At G = 16 form 1 is still ahead at 66, with block weights by
// 25.6 to 28.8 us, and there by 21.0 to 21.4 us at 148.)
// ---------------------------------------------------------------------------
struct CachePartials {
    int n;
    size_t slot0;
};

// The CTAs c with tiles of a pair: c * total / ctas <= tile < (c + 1) * total / ctas.
__device__ __forceinline__ CachePartials cache_partials_of(int64_t total, int64_t first, int nt, int grid, int bh) {
    const int64_t ctas = min(static_cast<int64_t>(grid), total);
    // (quotients of integers below 2^53 by one below 2^31 round down correctly in fp64, at a fraction of the
    // cost of a 64-bit division)
    const double per = static_cast<double>(total);
    const int c0 = static_cast<int>(static_cast<double>((first + 1) * ctas - 1) / per);
    const int c1 = static_cast<int>(static_cast<double>((first + nt) * ctas - 1) / per);
    return CachePartials{c1 - c0 + 1, static_cast<size_t>(c0) + bh};
}

// Joins (m2, l2) into (m, l).
__device__ __forceinline__ void cache_join(float &m, float &l, float m2, float l2) {
    const float top = fmaxf(m, m2);
    l = l * (m == top ? 1.f : fast_exp2(m - top)) + l2 * (m2 == top ? 1.f : fast_exp2(m2 - top));
    m = top;
}

// Maximum and sum over n partials of one head, by `threads` threads of which this is number t (a multiple of a
// warp); the result is that of the thread's warp alone.
__device__ __forceinline__ float2 cache_join_partials(const float2 *ml, int n, int G, int h, int t, int threads) {
    constexpr int U = 4;
    float m = -INFINITY, l = 0.f;
    for (int i0 = t; i0 < n; i0 += U * threads) {
        float2 a[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + u * threads;
            a[u] = i < n ? __ldcg(ml + static_cast<size_t>(i) * G + h) : make_float2(-INFINITY, 0.f);
        }
        float top = m;
#pragma unroll
        for (int u = 0; u < U; ++u) top = fmaxf(top, a[u].x);
        l *= m == top ? 1.f : fast_exp2(m - top);
#pragma unroll
        for (int u = 0; u < U; ++u) l += a[u].y * (a[u].x == top ? 1.f : fast_exp2(a[u].x - top));
        m = top;
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
        cache_join(m, l, __shfl_xor_sync(0xffffffffu, m, off), __shfl_xor_sync(0xffffffffu, l, off));
    return make_float2(m, l);
}

// Adds partial i of a head, 16 bytes of its outputs.
__device__ __forceinline__ void cache_add(float4 &a, float f, const float4 &v) {
    a.x = fmaf(f, v.x, a.x), a.y = fmaf(f, v.y, a.y), a.z = fmaf(f, v.z, a.z), a.w = fmaf(f, v.w, a.w);
}

// Four outputs of one query head (t: its maximum and sum; tokens = false: o = 0, lse = -inf).
__device__ __forceinline__ void cache_write(__nv_bfloat16 *o, float *lse, int row, int piece, const float4 &a,
                                            const float2 &t, bool tokens) {
    const float inv = tokens ? 1.f / t.y : 0.f;
    reinterpret_cast<uint2 *>(o + static_cast<size_t>(row) * kCacheD)[piece] =
        make_uint2(pack_bf16x2(a.x * inv, a.y * inv), pack_bf16x2(a.z * inv, a.w * inv));
    if (piece == 0) lse[row] = tokens ? fmaf(t.x, kLn2, logf(t.y)) : -INFINITY;
}

template <int SPLIT>
__global__ void __launch_bounds__(256) cache_combine_kernel(const int32_t *__restrict__ cache_len,
                                                            const float *opart, const float2 *mlpart,
                                                            const float2 *block_ml, const int32_t *idx,
                                                            __nv_bfloat16 *__restrict__ o, float *__restrict__ lse,
                                                            const float *weight_in, float *weight_out, int B, int Hk,
                                                            int G, int T, int s, int k, int nb, int grid,
                                                            int head_ctas) {
    constexpr int kSplit = SPLIT ? SPLIT : 1;
    __shared__ float2 head[kCacheMaxGroup];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const bool heads = SPLIT == 0 || static_cast<int>(blockIdx.x) < head_ctas;
    const int chunks = (nb + 255) / 256, w = blockIdx.x - head_ctas;
    const int parts = SPLIT == 0 ? (G + 7) / 8 : 1, part = SPLIT == 0 ? blockIdx.x % parts : 0;  // CTAs of a pair
    const int bh = SPLIT == 0 ? blockIdx.x / parts : heads ? blockIdx.x / kSplit / G : w / chunks, b = bh / Hk;
    const int L = __ldg(cache_len + b), nt = cache_tiles(L, T, s, k), ns = cache_slots(L, T, s, k);
    const int64_t total = cache_total_tiles(cache_len, B, Hk, T, s, k, lane);
    const int64_t first = cache_tiles_before(cache_len, b, T, s, k, lane) * Hk + static_cast<int64_t>(bh % Hk) * nt;
    CachePartials P{0, 0};
    if (nt > 0) P = cache_partials_of(total, first, nt, grid, bh);
    const float2 *ml = mlpart + P.slot0 * G;
    const size_t step = static_cast<size_t>(G) * (kCacheD / 4);
    constexpr int U = 4;  // the first outputs are asked for along with the maxima
    grid_dependency_wait();
    if constexpr (SPLIT == 0) {
        for (int h = warp; weight_out && h < G; h += blockDim.x >> 5)  // the other CTAs' heads, for the weights
            if (h / 8 != part) {
                const float2 t = cache_join_partials(ml, P.n, G, h, lane, 32);
                if (lane == 0) head[h] = t;
            }
        for (int h = 8 * part + warp; h < min(G, 8 * part + 8); h += blockDim.x >> 5) {
            const float4 *op = reinterpret_cast<const float4 *>(opart + (P.slot0 * G + h) * kCacheD) + lane;
            float4 a = make_float4(0.f, 0.f, 0.f, 0.f), v0[U];
            float m0[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (u < P.n) {
                    v0[u] = __ldcg(op + u * step);
                    m0[u] = __ldcg(ml + static_cast<size_t>(u) * G + h).x;
                }
            const float2 t = cache_join_partials(ml, P.n, G, h, lane, 32);
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (u < P.n) cache_add(a, fast_exp2(m0[u] - t.x), v0[u]);
#pragma unroll 4
            for (int i = U; i < P.n; ++i)
                cache_add(a, fast_exp2(__ldcg(ml + static_cast<size_t>(i) * G + h).x - t.x), __ldcg(op + i * step));
            cache_write(o, lse, bh * G + h, lane, a, t, nt > 0);
            if (lane == 0) head[h] = t;
        }
    } else if (heads) {
        constexpr int kLanes = 32 / kSplit, kGroups = 256 / kLanes;  // take partials in turn
        __shared__ float2 part_ml[8];
        __shared__ float4 part_o[8][kLanes];
        const int row = blockIdx.x / kSplit, h = row % G, group = tid / kLanes;
        const int piece = blockIdx.x % kSplit * kLanes + tid % kLanes;
        const float4 *op = reinterpret_cast<const float4 *>(opart + (P.slot0 * G + h) * kCacheD) + piece;
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f), v0[U];
        float m0[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = group + u * kGroups;
            if (i < P.n) {
                v0[u] = __ldcg(op + i * step);
                m0[u] = __ldcg(ml + static_cast<size_t>(i) * G + h).x;
            }
        }
        const float2 own = cache_join_partials(ml, P.n, G, h, tid, 256);
        if (lane == 0) part_ml[warp] = own;
        __syncthreads();
        float2 t = part_ml[0];
#pragma unroll
        for (int i = 1; i < 8; ++i) cache_join(t.x, t.y, part_ml[i].x, part_ml[i].y);
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (group + u * kGroups < P.n) cache_add(a, fast_exp2(m0[u] - t.x), v0[u]);
#pragma unroll 8
        for (int i = group + U * kGroups; i < P.n; i += kGroups)
            cache_add(a, fast_exp2(__ldcg(ml + static_cast<size_t>(i) * G + h).x - t.x), __ldcg(op + i * step));
#pragma unroll
        for (int off = kLanes; off < 32; off <<= 1) {
            a.x += __shfl_xor_sync(0xffffffffu, a.x, off), a.y += __shfl_xor_sync(0xffffffffu, a.y, off);
            a.z += __shfl_xor_sync(0xffffffffu, a.z, off), a.w += __shfl_xor_sync(0xffffffffu, a.w, off);
        }
        if (lane < kLanes) part_o[warp][lane] = a;
        __syncthreads();
        if (tid < kLanes) {
#pragma unroll
            for (int i = 1; i < 8; ++i) cache_add(a, 1.f, part_o[i][tid]);
            cache_write(o, lse, row, piece, a, t, nt > 0);
        }
        return;
    } else if (nt > 0) {
        for (int h = warp; h < G; h += 8) {
            const float2 t = cache_join_partials(ml, P.n, G, h, lane, 32);
            if (lane == 0) head[h] = t;
        }
    }
    if (!weight_out) return;
    // attention weight of blocks [j0, j1)
    const int share = SPLIT == 0 ? (nb + parts - 1) / parts : 256;
    const int j0 = SPLIT == 0 ? part * share : w % chunks * 256, j1 = min(j0 + share, nb);
    const float *win = weight_in ? weight_in + static_cast<size_t>(bh) * nb : nullptr;
    float *wout = weight_out + static_cast<size_t>(bh) * nb;
    auto mass = [&](int slot, int slots) {  // of one attended block
        float sum = 0.f;
        const float2 *bl = block_ml + static_cast<size_t>(bh) * G * slots + slot;
#pragma unroll 4
        for (int h = 0; h < G; ++h) {
            const float2 a = __ldcg(bl + static_cast<size_t>(h) * slots);
            sum += a.y * fast_exp2(a.x - head[h].x) / head[h].y;
        }
        return sum;
    };
    if (k == 0) {
        __syncthreads();
        for (int j = j0 + tid; j < j1; j += blockDim.x) wout[j] = (win ? win[j] : 0.f) + (j < ns ? mass(j, nb) : 0.f);
    } else {
        // every block first, then the attended ones, which are distinct (weight_in may be weight_out: the first
        // writes leave its values)
        for (int j = j0 + tid; j < j1; j += blockDim.x) wout[j] = win ? win[j] : 0.f;
        __syncthreads();
        for (int i = tid; i < ns; i += blockDim.x) {
            const int j = __ldcg(idx + static_cast<size_t>(bh) * k + i);
            if (j >= j0 && j < j1) wout[j] = (win ? win[j] : 0.f) + mass(i, k);
        }
    }
}

}  // namespace ssa
