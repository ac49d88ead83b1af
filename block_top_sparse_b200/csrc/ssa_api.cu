// ssa_api.cu -- the C ABI of libssa (declared in include/ssa.h): argument
// validation, workspace carving, TMA descriptor set-up and kernel launches.
// All kernels are compiled into this one translation unit.

#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstring>
#include <type_traits>

#include "ssa.h"

#include "device.cuh"
#include "pool_select.cuh"
#include "aux_kernels.cuh"
#include "attn_simt.cuh"
#include "attn_tc.cuh"
#include "attn_bwd.cuh"
#include "decode.cuh"
#include "rope.cuh"
#include "rope_axes.cuh"
#include "cache8.cuh"
#include "cache_decode.cuh"

using namespace ssa;

namespace {

struct Shape {
    int B, H, T, d, s, k, dtype;
    float scale;
    int Hk, G;         // key/value heads, query heads per key/value head
    size_t BH, rows;   // query heads B*H, query rows B*H*T
    size_t BHk, krows; // key/value heads B*Hk, key rows B*Hk*T
    int nb;
    size_t esz;       // element size in bytes
    bool tc;          // tensor-core path (bf16, d == 128)
};

ssa_status_t check_dims(const ssa_dims_t *dims, Shape &S, bool need_k) {
    if (!dims) return SSA_ERR_INVALID_ARG;
    S.B = dims->B;
    S.H = dims->H;
    S.T = dims->T;
    S.d = dims->d;
    S.s = dims->s;
    S.k = dims->k;
    S.dtype = dims->dtype;
    S.scale = dims->scale;
    if (S.B < 1 || S.H < 1 || S.T < 1 || S.d < 1 || S.s < 1) return SSA_ERR_INVALID_ARG;
    if (S.dtype != SSA_DT_BF16 && S.dtype != SSA_DT_FP32) return SSA_ERR_INVALID_ARG;
    if (!(std::isfinite(S.scale) && S.scale > 0.f)) return SSA_ERR_INVALID_ARG;
    if (S.d != 64 && S.d != 128) return SSA_ERR_UNSUPPORTED;
    if (S.s != 64 && S.s != 128) return SSA_ERR_UNSUPPORTED;
    if (S.T % S.s != 0) return SSA_ERR_UNSUPPORTED;
    S.Hk = dims->Hkv ? dims->Hkv : S.H;
    if (S.Hk < 1 || S.H % S.Hk != 0) return SSA_ERR_INVALID_ARG;
    S.G = S.H / S.Hk;
    S.BH = static_cast<size_t>(S.B) * S.H;
    S.rows = S.BH * S.T;
    S.BHk = static_cast<size_t>(S.B) * S.Hk;
    S.krows = S.BHk * S.T;
    if (S.rows > 0x7FFFFFFFull) return SSA_ERR_UNSUPPORTED;  // TMA row coordinates are int32
    S.nb = S.T / S.s;
    if (need_k) {
        if (S.k < 1 || S.k > S.nb) return SSA_ERR_INVALID_ARG;
        if (static_cast<int64_t>(S.T) * S.k > 0x7FFFFFFFll) return SSA_ERR_UNSUPPORTED;
    }
    S.esz = S.dtype == SSA_DT_BF16 ? 2 : 4;
    S.tc = S.dtype == SSA_DT_BF16 && S.d == 128;
    // a tensor-core tile holds 128 / G list entries for each of the G heads of a group
    if (S.tc && 128 % S.G != 0) return SSA_ERR_UNSUPPORTED;
    // the sparse index packs (t << 8) | slot into an int32
    if (need_k && S.tc && (S.k > 256 || S.T >= (1 << 23))) return SSA_ERR_UNSUPPORTED;
    // list positions of the whole index (and TMA row coordinates of the G partial rows per entry) fit an int32
    if (need_k && S.tc && S.BHk * list_stride(S.T, S.k, S.nb) * S.G >= (size_t(1) << 31)) return SSA_ERR_UNSUPPORTED;
    // one warp's staging of the index fill must fit in shared memory
    if (need_k && S.tc && index_fill_warp_ints(S.nb, S.k) * 4 > 227 * 1024) return SSA_ERR_UNSUPPORTED;
    return SSA_OK;
}

// Shapes of the 8-bit cache's calls: H query heads (any multiple of Hkv), T = capacity, k = 0 or blocks attended.
ssa_status_t check_cache_dims(const ssa_dims_t *dims, Shape &S) {
    if (!dims) return SSA_ERR_INVALID_ARG;
    S.B = dims->B;
    S.H = dims->H;
    S.T = dims->T;
    S.d = dims->d;
    S.s = dims->s;
    S.k = dims->k;
    S.dtype = dims->dtype;
    S.scale = dims->scale;
    if (S.B < 1 || S.H < 1 || S.T < 1 || S.d < 1 || S.s < 1) return SSA_ERR_INVALID_ARG;
    if (S.dtype != SSA_DT_BF16 && S.dtype != SSA_DT_FP32) return SSA_ERR_INVALID_ARG;
    if (!(std::isfinite(S.scale) && S.scale > 0.f)) return SSA_ERR_INVALID_ARG;
    S.Hk = dims->Hkv ? dims->Hkv : S.H;
    if (S.Hk < 1 || S.H % S.Hk != 0) return SSA_ERR_INVALID_ARG;
    if (S.dtype != SSA_DT_BF16 || S.d != kCacheD) return SSA_ERR_UNSUPPORTED;
    if (S.s != 64 && S.s != 128) return SSA_ERR_UNSUPPORTED;
    if (S.T % S.s != 0) return SSA_ERR_UNSUPPORTED;
    S.nb = S.T / S.s;
    if (S.k < 0 || S.k > S.nb) return SSA_ERR_INVALID_ARG;
    if (S.nb > kTopMaxBlocks) return SSA_ERR_UNSUPPORTED;
    S.G = S.H / S.Hk;
    S.BH = static_cast<size_t>(S.B) * S.H;
    S.BHk = static_cast<size_t>(S.B) * S.Hk;
    S.krows = S.BHk * S.T;
    if (S.krows > 0x7FFFFFFFull || S.BH > 0x7FFFFFFFull) return SSA_ERR_UNSUPPORTED;  // TMA row coordinates are int32
    return SSA_OK;
}

// Query heads per key head padded to a kernel's, and the grid of cache_attend_kernel: the CTAs that its shared
// memory lets reside at once.
inline int cache_heads(int G) { return G <= 4 ? 4 : G <= 8 ? 8 : G <= 16 ? 16 : 32; }
inline unsigned cache_grid(int G) {
    const int NH = cache_heads(G);
    return kCacheSms * (NH == 4   ? CacheAttend<4>::kPerSm
                        : NH == 8 ? CacheAttend<8>::kPerSm
                        : NH == 16 ? CacheAttend<16>::kPerSm
                                   : CacheAttend<32>::kPerSm);
}

inline size_t align_up(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

// Layout of the inverse selection index (the `index` buffer of ssa_sparse_index, or
// the head of a sparse call's workspace when the caller passes none).
struct IndexWs {
    int *cnt, *lstart, *llen;
    int32_t *entries;  // per head: list_stride(T, k, nb) entries, block lists on 128-entry boundaries
    int32_t *pos;      // [B*H*T, k] list position of every (query, slot), -1 when unused
    int32_t *order;    // [B*Hk*nb] launch order of the (head, block) units, heaviest first
    int nch;
};

size_t index_bytes(const Shape &S) {
    if (!S.tc) return 0;
    const size_t nch = (S.T + kIdxChunk - 1) / kIdxChunk;
    return align_up(S.BHk * nch * S.nb * 4) + 3 * align_up(S.BHk * S.nb * 4) +
           align_up(S.BHk * list_stride(S.T, S.k, S.nb) * 4) + align_up(S.krows * S.k * 4);
}

IndexWs carve_index(const Shape &S, const void *base) {
    IndexWs W;
    uint8_t *p = static_cast<uint8_t *>(const_cast<void *>(base));
    W.nch = (S.T + kIdxChunk - 1) / kIdxChunk;
    W.cnt = reinterpret_cast<int *>(p);
    p += align_up(S.BHk * W.nch * S.nb * 4);
    W.lstart = reinterpret_cast<int *>(p);
    p += align_up(S.BHk * S.nb * 4);
    W.llen = reinterpret_cast<int *>(p);
    p += align_up(S.BHk * S.nb * 4);
    W.entries = reinterpret_cast<int32_t *>(p);
    p += align_up(S.BHk * list_stride(S.T, S.k, S.nb) * 4);
    W.pos = reinterpret_cast<int32_t *>(p);
    p += align_up(S.krows * S.k * 4);
    W.order = reinterpret_cast<int32_t *>(p);
    return W;
}

// Layout of ssa_cache_decode's workspace.
struct CacheWs {
    size_t ml, blocks, bytes;  // byte offsets behind the partial outputs; size
};
CacheWs cache_ws(const Shape &S) {
    CacheWs W;
    const size_t slots = cache_partials(cache_grid(S.G), S.BHk) * S.G;
    W.ml = align_up(slots * kCacheD * 4);
    W.blocks = W.ml + align_up(slots * 8);
    W.bytes = W.blocks + align_up(S.BH * (S.k > 0 ? S.k : S.nb) * 8);
    return W;
}

size_t cache_ws_bytes(const Shape &S, int op) {
    if (op == SSA_OP_CACHE_EVICT) return align_up(S.BHk * evict_list_ints(S.nb) * 4);
    return S.G <= kCacheMaxGroup ? cache_ws(S).bytes : 0;
}

size_t ws_bytes_for(const Shape &S, int op) {
    switch (op) {
        case SSA_OP_SPARSE_INDEX:
            return index_bytes(S);
        case SSA_OP_SPARSE_FWD:
            if (!S.tc) return 0;
            // index (used when the caller passes none) | fp16 partial outputs and fp32 partial lse,
            // G rows per list position | range exponent of every key block, then a flag word
            return index_bytes(S) + align_up(S.BHk * list_stride(S.T, S.k, S.nb) * S.G * (128 * 2 + 4)) +
                   align_up(S.BHk * S.nb * 4 + 4);
        case SSA_OP_SPARSE_BWD:
            // D | index (used when the caller passes none) | fp32 dQ accumulator
            if (S.tc) return align_up(S.rows * 4) + index_bytes(S) + align_up(S.rows * S.d * 4);
            [[fallthrough]];
        case SSA_OP_FULL_BWD: {
            size_t b = align_up(S.rows * 4) + align_up(S.rows * S.d * 4);  // D, dQacc
            if (!S.tc) b += 2 * align_up(S.krows * S.d * 4);               // dKacc, dVacc
            return b;
        }
        case SSA_OP_FULL_FWD:
            return 0;
        case SSA_OP_ALIGN_FWD:
            return align_up(kAlignBlocks * 4);
        case SSA_OP_DECODE:
            // per (sequence, query head, slot): fp32 partial output and log-sum-exp
            return align_up(S.BH * S.k * S.d * 4) + align_up(S.BH * S.k * 4);
        default:
            return 0;
    }
}

ssa_status_t check_ws(const Shape &S, int op, const void *ws, size_t ws_bytes) {
    const size_t need = ws_bytes_for(S, op);
    if (need == 0) return SSA_OK;
    if (!ws || ws_bytes < need || (reinterpret_cast<uintptr_t>(ws) & 15u)) return SSA_ERR_WORKSPACE;
    return SSA_OK;
}

// Bits of a backward call's `accumulate`; fp32 gradients are written with 16-byte accesses and
// reduced into by the TMA unit, so their base addresses must be 16-byte aligned.
ssa_status_t check_grads(int accumulate, const void *dQ, const void *dK, const void *dV) {
    if (accumulate & ~static_cast<int>(SSA_BWD_ACCUMULATE | SSA_BWD_GRAD_FP32)) return SSA_ERR_INVALID_ARG;
    if ((accumulate & SSA_BWD_GRAD_FP32) &&
        ((reinterpret_cast<uintptr_t>(dQ) | reinterpret_cast<uintptr_t>(dK) | reinterpret_cast<uintptr_t>(dV)) & 15u))
        return SSA_ERR_INVALID_ARG;
    return SSA_OK;
}

ssa_status_t launch_status() {
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? SSA_OK : SSA_ERR_CUDA;
}

// ---------------------------------------------------------------------------
// TMA descriptors: 2D view [rows, 128] of a bf16 tensor, box 64 columns x box_rows.
// ---------------------------------------------------------------------------
typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                  const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
    static EncodeTiledFn fn = nullptr;
    if (!fn) {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(p);
    }
    return fn;
}

bool make_tmap(CUtensorMap *m, const void *base, size_t rows, int box_rows) {
    EncodeTiledFn f = encode_fn();
    if (!f) return false;
    const cuuint64_t gdim[2] = {128, rows};
    const cuuint64_t gstride[1] = {128 * 2};
    const cuuint32_t box[2] = {64, static_cast<cuuint32_t>(box_rows)};
    const cuuint32_t estride[2] = {1, 1};
    return f(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(base), gdim, gstride, box, estride,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// fp32 view [rows, 128] of the dQ accumulator, box 32 columns x 128 rows (128-byte rows, swizzled).
bool make_tmap_f32(CUtensorMap *m, const void *base, size_t rows) {
    EncodeTiledFn f = encode_fn();
    if (!f) return false;
    const cuuint64_t gdim[2] = {128, rows};
    const cuuint64_t gstride[1] = {128 * 4};
    const cuuint32_t box[2] = {32, 128};
    const cuuint32_t estride[2] = {1, 1};
    return f(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, const_cast<void *>(base), gdim, gstride, box, estride,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename K>
bool set_smem(K kernel, size_t bytes) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes)) ==
           cudaSuccess;
}

// Launch of a kernel that may start while the one before it on the stream still runs (it waits for that one
// with grid_dependency_wait before it touches what that one writes or reads).
template <typename... P, typename... A>
bool launch_dependent(void (*kernel)(P...), dim3 grid, unsigned threads, size_t smem, cudaStream_t st, A... args) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...) == cudaSuccess) return true;
    cudaGetLastError();  // reported by this call, not by the next one
    return false;
}

// e4m3 rows of 128 bytes, boxes of one block.
bool make_tmap_codes(CUtensorMap *m, const void *base, size_t rows, int box_rows) {
    EncodeTiledFn f = encode_fn();
    if (!f) return false;
    const cuuint64_t gdim[2] = {kCacheD, rows};
    const cuuint64_t gstride[1] = {kCacheD};
    const cuuint32_t box[2] = {kCacheD, static_cast<cuuint32_t>(box_rows)};
    const cuuint32_t estride[2] = {1, 1};
    return f(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), gdim, gstride, box, estride,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

unsigned grid_for(size_t n, unsigned per_block) {
    size_t g = (n + per_block - 1) / per_block;
    if (g > 148u * 32u) g = 148u * 32u;
    return static_cast<unsigned>(g ? g : 1);
}

template <typename T, int KPL>
ssa_status_t launch_select(const Shape &S, const void *Q, const float *Kbar, int32_t *idx, size_t sm, cudaStream_t st) {
    if (!set_smem(select_kernel<T, KPL>, sm)) return SSA_ERR_CUDA;
    select_kernel<T, KPL><<<dim3(S.T / kSelQ, S.BHk), 256, sm, st>>>((const T *)Q, Kbar, idx, S.T, S.d, S.s, S.k, S.nb,
                                                                      S.G);
    return SSA_OK;
}

// Inverse selection index: entries of block j of head bh (query order) and the list
// position of every (query, slot).
ssa_status_t build_index(const Shape &S, const int32_t *idx, const IndexWs &W, cudaStream_t st) {
    const size_t hbytes = static_cast<size_t>(S.nb) * 4;
    if (!set_smem(index_count_kernel, hbytes)) return SSA_ERR_CUDA;
    index_count_kernel<<<dim3(W.nch, S.BHk), 256, hbytes, st>>>(idx, W.cnt, S.T, S.k, S.nb, W.nch);
    index_scan_kernel<<<S.BHk, 1024, 0, st>>>(W.cnt, W.lstart, W.llen, S.nb, W.nch);
    // four warps (chunks) per CTA while their staging fits comfortably, else one
    const size_t wbytes = index_fill_warp_ints(S.nb, S.k) * 4;
    const int wpc = wbytes * 4 <= 160 * 1024 ? 4 : 1;
    if (!set_smem(index_fill_kernel, wbytes * wpc)) return SSA_ERR_CUDA;
    index_fill_kernel<<<dim3((W.nch + wpc - 1) / wpc, S.BHk), 32 * wpc, wbytes * wpc, st>>>(
        idx, W.cnt, W.entries, W.pos, S.T, S.k, S.nb, W.nch);
    unit_order_kernel<<<1, 1024, 0, st>>>(W.llen, W.order, static_cast<int>(S.BHk) * S.nb, kTileQ / S.G);
    return launch_status();
}

template <typename T>
void launch_simt_fwd(const Shape &S, const void *Q, const void *K, const void *V, const int32_t *idx, void *O,
                     void *O_lo, float *lse, cudaStream_t st) {
    const unsigned g = static_cast<unsigned>((S.rows + 7) / 8);
    T *lo = sizeof(T) == 2 ? (T *)O_lo : nullptr;  // the residual is only kept for bf16 outputs
    if (S.d == 64)
        simt_fwd_kernel<T, 2><<<g, 256, 0, st>>>((const T *)Q, (const T *)K, (const T *)V, idx, (T *)O, lo, lse,
                                                 S.rows, S.T, S.s, S.k, S.scale, S.G);
    else
        simt_fwd_kernel<T, 4><<<g, 256, 0, st>>>((const T *)Q, (const T *)K, (const T *)V, idx, (T *)O, lo, lse,
                                                 S.rows, S.T, S.s, S.k, S.scale, S.G);
}

template <typename T>
ssa_status_t simt_bwd(const Shape &S, const void *Q, const void *K, const void *V, const void *O, const void *O_lo,
                      const float *lse, const void *dO, const int32_t *idx, void *dQ, void *dK, void *dV,
                      int accumulate, void *ws, cudaStream_t st) {
    uint8_t *p = static_cast<uint8_t *>(ws);
    float *Dvec = reinterpret_cast<float *>(p);
    p += align_up(S.rows * 4);
    float *dQacc = reinterpret_cast<float *>(p);
    p += align_up(S.rows * S.d * 4);
    float *dKacc = reinterpret_cast<float *>(p);
    p += align_up(S.krows * S.d * 4);
    float *dVacc = reinterpret_cast<float *>(p);
    const size_t n = S.rows * S.d, nk = S.krows * S.d;
    if (cudaMemsetAsync(dKacc, 0, nk * 4, st) != cudaSuccess || cudaMemsetAsync(dVacc, 0, nk * 4, st) != cudaSuccess)
        return SSA_ERR_CUDA;
    const unsigned g = static_cast<unsigned>((S.rows + 7) / 8);
    bwd_prep_kernel<T><<<g, 256, 0, st>>>((const T *)dO, (const T *)O, sizeof(T) == 2 ? (const T *)O_lo : nullptr,
                                          Dvec, dQacc, S.rows, S.d);
    if (S.d == 64)
        simt_bwd_kernel<T, 2><<<g, 256, 0, st>>>((const T *)Q, (const T *)K, (const T *)V, (const T *)dO, idx, lse,
                                                 Dvec, dQacc, dKacc, dVacc, S.rows, S.T, S.s, S.k, S.scale, S.G);
    else
        simt_bwd_kernel<T, 4><<<g, 256, 0, st>>>((const T *)Q, (const T *)K, (const T *)V, (const T *)dO, idx, lse,
                                                 Dvec, dQacc, dKacc, dVacc, S.rows, S.T, S.s, S.k, S.scale, S.G);
    const unsigned ge = grid_for(n, 256), gk = grid_for(nk, 256);
    const int acc = accumulate & SSA_BWD_ACCUMULATE;
    if ((accumulate & SSA_BWD_GRAD_FP32) || sizeof(T) == 4) {
        acc_to_out_kernel<float><<<ge, 256, 0, st>>>(dQacc, (float *)dQ, n, acc);
        acc_to_out_kernel<float><<<gk, 256, 0, st>>>(dKacc, (float *)dK, nk, acc);
        acc_to_out_kernel<float><<<gk, 256, 0, st>>>(dVacc, (float *)dV, nk, acc);
    } else {
        acc_to_out_kernel<T><<<ge, 256, 0, st>>>(dQacc, (T *)dQ, n, acc);
        acc_to_out_kernel<T><<<gk, 256, 0, st>>>(dKacc, (T *)dK, nk, acc);
        acc_to_out_kernel<T><<<gk, 256, 0, st>>>(dVacc, (T *)dV, nk, acc);
    }
    return launch_status();
}

// Tensor-core backward shared by both streams.
ssa_status_t tc_bwd(const Shape &S, const void *Q, const void *K, const void *V, const void *O, const void *O_lo,
                    const float *lse, const void *dO, const int32_t *idx, const void *index, void *dQ, void *dK,
                    void *dV, int accumulate, void *ws, cudaStream_t st) {
    uint8_t *p = static_cast<uint8_t *>(ws);
    float *Dvec = reinterpret_cast<float *>(p);
    p += align_up(S.rows * 4);
    const bool sparse = idx != nullptr;
    IndexWs W{};
    if (sparse) {
        // the caller's index, or one built here in the workspace
        W = carve_index(S, index ? index : p);
        p += index_bytes(S);
        if (!index) {
            const ssa_status_t e = build_index(S, idx, W, st);
            if (e != SSA_OK) return e;
        }
    }
    // fp32 dQ accumulator: TMA reduce-adds of whole tiles (full) or vector reductions of gathered
    // rows (sparse); zeroed by the prep kernel, converted (and added to dQ when accumulating) after.
    // With fp32 gradients the caller's dQ is the accumulator itself (zeroed unless accumulating).
    const bool acc = (accumulate & SSA_BWD_ACCUMULATE) != 0, g32 = (accumulate & SSA_BWD_GRAD_FP32) != 0;
    float *dQacc = g32 ? static_cast<float *>(dQ) : reinterpret_cast<float *>(p);
    float *zero_acc = (g32 && acc) ? nullptr : dQacc;
    if (((reinterpret_cast<uintptr_t>(O) | reinterpret_cast<uintptr_t>(O_lo)) & 7u) == 0) {  // 8-byte row loads
        const unsigned g = static_cast<unsigned>((S.rows + 8 * kPrepRows - 1) / (8 * kPrepRows));
        bwd_prep_bf16_kernel<<<g, 256, 0, st>>>((const __nv_bfloat16 *)dO, (const __nv_bfloat16 *)O,
                                                (const __nv_bfloat16 *)O_lo, Dvec, zero_acc, S.rows);
    } else {
        const unsigned g = static_cast<unsigned>((S.rows + 7) / 8);
        bwd_prep_kernel<__nv_bfloat16><<<g, 256, 0, st>>>((const __nv_bfloat16 *)dO, (const __nv_bfloat16 *)O,
                                                           (const __nv_bfloat16 *)O_lo, Dvec, zero_acc, S.rows, S.d);
    }
    const int nkv = sparse ? S.s : 128;
    CUtensorMap tmK, tmV, tmQ, tmdO, tmdQ;
    if (!make_tmap(&tmK, K, S.krows, nkv) || !make_tmap(&tmV, V, S.krows, nkv) || !make_tmap(&tmQ, Q, S.rows, 128) ||
        !make_tmap(&tmdO, dO, S.rows, 128) || !make_tmap_f32(&tmdQ, dQacc, S.rows))
        return SSA_ERR_CUDA;
    BwdArgs a{};
    a.Q = (const __nv_bfloat16 *)Q;
    a.dO = (const __nv_bfloat16 *)dO;
    a.lse = lse;
    a.Dvec = Dvec;
    a.dQacc = dQacc;
    a.dK = dK;
    a.dV = dV;
    a.entries = W.entries;
    a.lstart = W.lstart;
    a.llen = W.llen;
    a.order = sparse ? W.order : nullptr;
    a.BH = static_cast<int>(S.BHk);
    a.G = S.G;
    a.T = S.T;
    a.k = S.k;
    a.nb = S.nb;
    a.sparse = sparse ? 1 : 0;
    a.accumulate = acc ? 1 : 0;
    a.grad_fp32 = g32 ? 1 : 0;
    a.scale = S.scale;
    a.scale_log2 = S.scale * kLog2e;
    const unsigned units = static_cast<unsigned>(S.BHk * (sparse ? S.nb : (S.T + 127) / 128));
    const bool gq = S.G > 1;
    // the grouped-head instantiations carry the group arithmetic; one query head per key head does not
    auto run = [&](auto kernel, size_t sm) {
        if (!set_smem(kernel, sm)) return false;
        kernel<<<units, kBwdThreads, sm, st>>>(tmK, tmV, tmQ, tmdO, tmdQ, a);
        return true;
    };
    const size_t sm128 = BwdSmem<128>::kTotal + 1024, sm64 = BwdSmem<64>::kTotal + 1024;
    const bool launched = nkv == 128 ? (gq ? run(attn_bwd_kernel<128, true>, sm128) : run(attn_bwd_kernel<128, false>, sm128))
                                     : (gq ? run(attn_bwd_kernel<64, true>, sm64) : run(attn_bwd_kernel<64, false>, sm64));
    if (!launched) return SSA_ERR_CUDA;
    if (!g32) {
        const size_t n = S.rows * S.d;
        acc_to_out_kernel<__nv_bfloat16><<<grid_for(n, 256), 256, 0, st>>>(dQacc, (__nv_bfloat16 *)dQ, n, acc);
    }
    return launch_status();
}

}  // namespace

extern "C" {

size_t ssa_workspace_size(const ssa_dims_t *dims, int op) {
    Shape S;
    if (op == SSA_OP_CACHE_DECODE || op == SSA_OP_CACHE_EVICT)
        return check_cache_dims(dims, S) == SSA_OK ? cache_ws_bytes(S, op) : 0;
    const bool need_k = op == SSA_OP_SPARSE_FWD || op == SSA_OP_SPARSE_BWD;
    if (check_dims(dims, S, need_k) != SSA_OK) return 0;
    return ws_bytes_for(S, op);
}

ssa_status_t ssa_block_pool(const ssa_dims_t *dims, const void *K, float *Kbar, ssa_stream_t stream) {
    Shape S;
    ssa_status_t e = check_dims(dims, S, false);
    if (e != SSA_OK) return e;
    if (!K || !Kbar) return SSA_ERR_INVALID_ARG;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const size_t units = S.BHk * S.nb;  // one warp per (key/value head, block)
    const unsigned g = static_cast<unsigned>((units + kPoolWarps - 1) / kPoolWarps);
    const int blk = kPoolWarps * 32;
    if (S.dtype == SSA_DT_BF16) {
        if (S.d == 128)
            pool_kernel<__nv_bfloat16, 128><<<g, blk, 0, st>>>((const __nv_bfloat16 *)K, Kbar, S.T, S.s, S.nb, units);
        else
            pool_kernel<__nv_bfloat16, 64><<<g, blk, 0, st>>>((const __nv_bfloat16 *)K, Kbar, S.T, S.s, S.nb, units);
    } else {
        if (S.d == 128)
            pool_kernel<float, 128><<<g, blk, 0, st>>>((const float *)K, Kbar, S.T, S.s, S.nb, units);
        else
            pool_kernel<float, 64><<<g, blk, 0, st>>>((const float *)K, Kbar, S.T, S.s, S.nb, units);
    }
    return launch_status();
}

ssa_status_t ssa_block_select(const ssa_dims_t *dims, const void *Q, const float *Kbar, int32_t *idx,
                              unsigned flags, ssa_stream_t stream) {
    Shape S;
    ssa_status_t e = check_dims(dims, S, true);
    if (e != SSA_OK) return e;
    if (!Q || !Kbar || !idx) return SSA_ERR_INVALID_ARG;
    if (!(flags & SSA_SEL_FORCE_CURRENT) || (flags & ~static_cast<unsigned>(SSA_SEL_FORCE_CURRENT)))
        return SSA_ERR_UNSUPPORTED;
    const size_t sm = select_smem_bytes(S.d, S.nb);
    if (S.nb > 1024 || sm > 227 * 1024) return SSA_ERR_UNSUPPORTED;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (S.tc && S.nb <= kSelTcMaxBlocks) {
        // scores on the tensor cores
        const size_t smt = SelTcSmem::kTotal + 1024;
        if (!set_smem(select_tc_kernel, smt)) return SSA_ERR_CUDA;
        select_tc_kernel<<<dim3((S.T + kSelTcRows - 1) / kSelTcRows, S.BHk), kSelTcThreads, smt, st>>>(
            (const __nv_bfloat16 *)Q, Kbar, idx, S.T, S.s, S.k, S.nb, S.G);
        return launch_status();
    }
    if (S.dtype == SSA_DT_BF16) {
        if (S.nb <= 256)
            e = launch_select<__nv_bfloat16, 8>(S, Q, Kbar, idx, sm, st);
        else if (S.nb <= 512)
            e = launch_select<__nv_bfloat16, 16>(S, Q, Kbar, idx, sm, st);
        else
            e = launch_select<__nv_bfloat16, 32>(S, Q, Kbar, idx, sm, st);
    } else {
        if (S.nb <= 256)
            e = launch_select<float, 8>(S, Q, Kbar, idx, sm, st);
        else if (S.nb <= 512)
            e = launch_select<float, 16>(S, Q, Kbar, idx, sm, st);
        else
            e = launch_select<float, 32>(S, Q, Kbar, idx, sm, st);
    }
    if (e != SSA_OK) return e;
    return launch_status();
}

ssa_status_t ssa_sparse_index(const ssa_dims_t *dims, const int32_t *idx, void *index, size_t index_bytes_,
                              ssa_stream_t stream) {
    Shape S;
    ssa_status_t e = check_dims(dims, S, true);
    if (e != SSA_OK) return e;
    if (!idx) return SSA_ERR_INVALID_ARG;
    if (!S.tc) return SSA_OK;  // the CUDA-core kernels read idx directly
    if ((e = check_ws(S, SSA_OP_SPARSE_INDEX, index, index_bytes_)) != SSA_OK) return e;
    return build_index(S, idx, carve_index(S, index), reinterpret_cast<cudaStream_t>(stream));
}

ssa_status_t ssa_sparse_attn_fwd(const ssa_dims_t *dims, const void *Q, const void *K, const void *V,
                                 const int32_t *idx, const void *index, void *O, void *O_lo, float *lse, void *ws,
                                 size_t ws_bytes, ssa_stream_t stream) {
    Shape S;
    ssa_status_t e = check_dims(dims, S, true);
    if (e != SSA_OK) return e;
    if (!Q || !K || !V || !idx || !O || !lse) return SSA_ERR_INVALID_ARG;
    if ((e = check_ws(S, SSA_OP_SPARSE_FWD, ws, ws_bytes)) != SSA_OK) return e;
    if (index && (reinterpret_cast<uintptr_t>(index) & 15u)) return SSA_ERR_WORKSPACE;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (!S.tc) {
        if (S.dtype == SSA_DT_BF16)
            launch_simt_fwd<__nv_bfloat16>(S, Q, K, V, idx, O, O_lo, lse, st);
        else
            launch_simt_fwd<float>(S, Q, K, V, idx, O, O_lo, lse, st);
        return launch_status();
    }
    uint8_t *p = static_cast<uint8_t *>(ws);
    const IndexWs W = carve_index(S, index ? index : p);
    p += index_bytes(S);
    if (!index && (e = build_index(S, idx, W, st)) != SSA_OK) return e;
    const size_t nprow = S.BHk * list_stride(S.T, S.k, S.nb) * S.G;  // partial rows: G per list position
    __half *Opart = reinterpret_cast<__half *>(p);
    float *lsepart = reinterpret_cast<float *>(p + nprow * 128 * 2);
    p += align_up(nprow * (128 * 2 + 4));
    int32_t *bexp = reinterpret_cast<int32_t *>(p);  // [BHk * nb] exponents, then the "any set" flag
    if (cudaMemsetAsync(bexp + S.BHk * S.nb, 0, 4, st) != cudaSuccess) return SSA_ERR_CUDA;
    CUtensorMap tmK, tmV, tmO;
    // the fp16 partials are stored through a 16-bit tensor map (no conversion happens in a store)
    if (!make_tmap(&tmK, K, S.krows, S.s) || !make_tmap(&tmV, V, S.krows, S.s) ||
        !make_tmap(&tmO, Opart, nprow, 32))
        return SSA_ERR_CUDA;
    const unsigned units = static_cast<unsigned>(S.BHk * S.nb);
    const float sl2 = S.scale * kLog2e;
    auto run = [&](auto kernel, size_t sm) {
        if (!set_smem(kernel, sm)) return false;
        kernel<<<units, kSparseFwdThreads, sm, st>>>(tmK, tmV, tmO, (const __nv_bfloat16 *)Q, W.entries, W.lstart,
                                                     W.llen, W.order, lsepart, bexp, static_cast<int>(S.BHk), S.T, S.k, S.nb,
                                                     S.G, sl2);
        return true;
    };
    const bool gq = S.G > 1;
    const size_t sm128 = SparseFwdSmem<128>::kTotal + 1024, sm64 = SparseFwdSmem<64>::kTotal + 1024;
    const bool launched = S.s == 128 ? (gq ? run(sparse_fwd_kernel<128, true>, sm128) : run(sparse_fwd_kernel<128, false>, sm128))
                                     : (gq ? run(sparse_fwd_kernel<64, true>, sm64) : run(sparse_fwd_kernel<64, false>, sm64));
    if (!launched) return SSA_ERR_CUDA;
    const unsigned mg = static_cast<unsigned>((S.rows + 7) / 8);
    auto merge = [&](auto kernel) {
        kernel<<<mg, 256, 0, st>>>(W.pos, idx, bexp, Opart, lsepart, (__nv_bfloat16 *)O, (__nv_bfloat16 *)O_lo, lse,
                                   S.rows, S.T, S.k, S.nb, S.G);
    };
    if (S.k <= 8)
        merge(sparse_merge_kernel<1>);
    else if (S.k <= 16)
        merge(sparse_merge_kernel<2>);
    else if (S.k <= 32)
        merge(sparse_merge_kernel<4>);
    else
        merge(sparse_merge_kernel<0>);
    return launch_status();
}

ssa_status_t ssa_sparse_attn_bwd(const ssa_dims_t *dims, const void *Q, const void *K, const void *V,
                                 const void *O, const void *O_lo, const float *lse, const void *dO,
                                 const int32_t *idx, const void *index, void *dQ, void *dK, void *dV, int accumulate,
                                 void *ws, size_t ws_bytes, ssa_stream_t stream) {
    Shape S;
    ssa_status_t e = check_dims(dims, S, true);
    if (e != SSA_OK) return e;
    if (!Q || !K || !V || !O || !lse || !dO || !idx || !dQ || !dK || !dV) return SSA_ERR_INVALID_ARG;
    if ((e = check_grads(accumulate, dQ, dK, dV)) != SSA_OK) return e;
    if ((e = check_ws(S, SSA_OP_SPARSE_BWD, ws, ws_bytes)) != SSA_OK) return e;
    if (index && (reinterpret_cast<uintptr_t>(index) & 15u)) return SSA_ERR_WORKSPACE;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (S.tc) return tc_bwd(S, Q, K, V, O, O_lo, lse, dO, idx, index, dQ, dK, dV, accumulate, ws, st);
    if (S.dtype == SSA_DT_BF16)
        return simt_bwd<__nv_bfloat16>(S, Q, K, V, O, O_lo, lse, dO, idx, dQ, dK, dV, accumulate, ws, st);
    return simt_bwd<float>(S, Q, K, V, O, O_lo, lse, dO, idx, dQ, dK, dV, accumulate, ws, st);
}

ssa_status_t ssa_full_attn_fwd(const ssa_dims_t *dims, const void *Q, const void *K, const void *V, void *O,
                               void *O_lo, float *lse, void *ws, size_t ws_bytes, ssa_stream_t stream) {
    Shape S;
    ssa_status_t e = check_dims(dims, S, false);
    if (e != SSA_OK) return e;
    if (!Q || !K || !V || !O || !lse) return SSA_ERR_INVALID_ARG;
    (void)ws;
    (void)ws_bytes;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (!S.tc) {
        if (S.dtype == SSA_DT_BF16)
            launch_simt_fwd<__nv_bfloat16>(S, Q, K, V, nullptr, O, O_lo, lse, st);
        else
            launch_simt_fwd<float>(S, Q, K, V, nullptr, O, O_lo, lse, st);
        return launch_status();
    }
    CUtensorMap tmQ, tmK, tmV;
    if (!make_tmap(&tmQ, Q, S.rows, 128) || !make_tmap(&tmK, K, S.krows, 128) || !make_tmap(&tmV, V, S.krows, 128))
        return SSA_ERR_CUDA;
    const size_t sm = FullFwdSmem::kTotal + 1024;
    if (!set_smem(full_fwd_kernel, sm)) return SSA_ERR_CUDA;
    const unsigned grid = static_cast<unsigned>(S.BH * ((S.T + 255) / 256));
    full_fwd_kernel<<<grid, kFullFwdThreads, sm, st>>>(tmQ, tmK, tmV, (__nv_bfloat16 *)O, (__nv_bfloat16 *)O_lo, lse,
                                                      static_cast<int>(S.BH), S.T, S.G, S.scale * kLog2e);
    return launch_status();
}

ssa_status_t ssa_full_attn_bwd(const ssa_dims_t *dims, const void *Q, const void *K, const void *V,
                               const void *O, const void *O_lo, const float *lse, const void *dO, void *dQ, void *dK,
                               void *dV, int accumulate, void *ws, size_t ws_bytes, ssa_stream_t stream) {
    Shape S;
    ssa_status_t e = check_dims(dims, S, false);
    if (e != SSA_OK) return e;
    if (!Q || !K || !V || !O || !lse || !dO || !dQ || !dK || !dV) return SSA_ERR_INVALID_ARG;
    if ((e = check_grads(accumulate, dQ, dK, dV)) != SSA_OK) return e;
    if ((e = check_ws(S, SSA_OP_FULL_BWD, ws, ws_bytes)) != SSA_OK) return e;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (S.tc) return tc_bwd(S, Q, K, V, O, O_lo, lse, dO, nullptr, nullptr, dQ, dK, dV, accumulate, ws, st);
    if (S.dtype == SSA_DT_BF16)
        return simt_bwd<__nv_bfloat16>(S, Q, K, V, O, O_lo, lse, dO, nullptr, dQ, dK, dV, accumulate, ws, st);
    return simt_bwd<float>(S, Q, K, V, O, O_lo, lse, dO, nullptr, dQ, dK, dV, accumulate, ws, st);
}

ssa_status_t ssa_align_loss_fwd(const ssa_dims_t *dims, const void *Of, const void *Os, int kind, float beta,
                                float w_sparsity, float w_commit, float *loss_dev, void *ws, size_t ws_bytes,
                                ssa_stream_t stream) {
    Shape S;
    ssa_status_t e = check_dims(dims, S, false);
    if (e != SSA_OK) return e;
    if (!Of || !Os || !loss_dev) return SSA_ERR_INVALID_ARG;
    if (kind != SSA_ALIGN_SMOOTH_L1 && kind != SSA_ALIGN_L2) return SSA_ERR_INVALID_ARG;
    if (!(beta > 0.f) || !std::isfinite(beta) || !std::isfinite(w_sparsity) || !std::isfinite(w_commit))
        return SSA_ERR_INVALID_ARG;
    if ((e = check_ws(S, SSA_OP_ALIGN_FWD, ws, ws_bytes)) != SSA_OK) return e;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    float *partial = static_cast<float *>(ws);
    const size_t n = S.rows * S.d;
    if (S.dtype == SSA_DT_BF16)
        align_fwd_partial_kernel<__nv_bfloat16><<<kAlignBlocks, 256, 0, st>>>(
            (const __nv_bfloat16 *)Of, (const __nv_bfloat16 *)Os, partial, n, kind, beta);
    else
        align_fwd_partial_kernel<float><<<kAlignBlocks, 256, 0, st>>>((const float *)Of, (const float *)Os, partial,
                                                                      n, kind, beta);
    align_fwd_final_kernel<<<1, 32, 0, st>>>(partial, kAlignBlocks, loss_dev,
                                             (static_cast<double>(w_sparsity) + w_commit) / static_cast<double>(n));
    return launch_status();
}

ssa_status_t ssa_align_loss_bwd(const ssa_dims_t *dims, const void *Of, const void *Os, int kind, float beta,
                                float w_sparsity, float w_commit, const float *dloss_dev, void *dOf, void *dOs,
                                int accumulate, ssa_stream_t stream) {
    Shape S;
    ssa_status_t e = check_dims(dims, S, false);
    if (e != SSA_OK) return e;
    if (!Of || !Os || !dloss_dev || !dOf || !dOs) return SSA_ERR_INVALID_ARG;
    if (kind != SSA_ALIGN_SMOOTH_L1 && kind != SSA_ALIGN_L2) return SSA_ERR_INVALID_ARG;
    if (!(beta > 0.f) || !std::isfinite(beta) || !std::isfinite(w_sparsity) || !std::isfinite(w_commit))
        return SSA_ERR_INVALID_ARG;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const size_t n = S.rows * S.d;
    if (S.dtype == SSA_DT_BF16)
        align_bwd_kernel<__nv_bfloat16><<<grid_for(n, 256), 256, 0, st>>>(
            (const __nv_bfloat16 *)Of, (const __nv_bfloat16 *)Os, dloss_dev, (__nv_bfloat16 *)dOf,
            (__nv_bfloat16 *)dOs, n, kind, beta, w_sparsity, w_commit, accumulate);
    else
        align_bwd_kernel<float><<<grid_for(n, 256), 256, 0, st>>>((const float *)Of, (const float *)Os, dloss_dev,
                                                                  (float *)dOf, (float *)dOs, n, kind, beta,
                                                                  w_sparsity, w_commit, accumulate);
    return launch_status();
}

ssa_status_t ssa_dropped_mass(const ssa_dims_t *dims, const float *lse_sparse, const float *lse_full, float *delta,
                              ssa_stream_t stream) {
    Shape S;
    ssa_status_t e = check_dims(dims, S, false);
    if (e != SSA_OK) return e;
    if (!lse_sparse || !lse_full || !delta) return SSA_ERR_INVALID_ARG;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    dropped_mass_kernel<<<grid_for(S.rows, 256), 256, 0, st>>>(lse_sparse, lse_full, delta, S.rows);
    return launch_status();
}

}  // extern "C"

// ---------------------------------------------------------------------------
// Allocation-free full attention backward: scratch in a static device array.
// In host code the array's name is only a stand-in; its device address comes
// from cudaGetSymbolAddress, looked up with the caller's device current.
// ---------------------------------------------------------------------------
static __device__ __align__(256) unsigned char g_noalloc_scratch[SSA_NOALLOC_SCRATCH_BYTES];

namespace {
// Device address of the scratch array in the current device's context.  Looked up on
// every call (the lookup allocates nothing): an address cached across calls would be
// stale after the context is torn down and the module loaded again.
ssa_status_t noalloc_scratch(void **out) {
    void *p = nullptr;
    if (cudaGetSymbolAddress(&p, g_noalloc_scratch) != cudaSuccess || !p) return SSA_ERR_CUDA;
    *out = p;
    return SSA_OK;
}

// One slot's block of the decode against the G query heads, for G padded to GP.
template <int GP>
bool launch_decode_attend(const Shape &S, cudaStream_t st, const int32_t *cache_len, const void *q, const void *Kc,
                          const void *Vc, const int32_t *idx, float *opart, float *lsepart) {
    const size_t sm = dec_attend_smem(S.s, GP);
    if (!set_smem(decode_attend_kernel<GP>, sm)) return false;
    decode_attend_kernel<GP><<<dim3(static_cast<unsigned>(S.BHk), S.k), kDecThreads, sm, st>>>(
        cache_len, (const __nv_bfloat16 *)q, (const __nv_bfloat16 *)Kc, (const __nv_bfloat16 *)Vc, idx, opart, lsepart,
        S.Hk, S.G, S.T, S.s, S.k, S.scale);
    return true;
}
}  // namespace

extern "C" {

ssa_status_t ssa_full_attn_bwd_noalloc(const ssa_dims_t *dims, const void *Q, const void *K, const void *V,
                                       const void *O, const void *O_lo, const float *lse, const void *dO, void *dQ,
                                       void *dK, void *dV, int accumulate, ssa_stream_t stream) {
    Shape S;
    ssa_status_t e = check_dims(dims, S, false);
    if (e != SSA_OK) return e;
    if (!Q || !K || !V || !O || !lse || !dO || !dQ || !dK || !dV) return SSA_ERR_INVALID_ARG;
    const size_t need = ws_bytes_for(S, SSA_OP_FULL_BWD);
    if (need > SSA_NOALLOC_SCRATCH_BYTES) return SSA_ERR_WORKSPACE;
    void *ws = nullptr;
    if ((e = noalloc_scratch(&ws)) != SSA_OK) return e;
    return ssa_full_attn_bwd(dims, Q, K, V, O, O_lo, lse, dO, dQ, dK, dV, accumulate, ws, SSA_NOALLOC_SCRATCH_BYTES,
                             stream);
}

ssa_status_t ssa_sparse_decode(const ssa_dims_t *dims, const int32_t *cache_len, const void *q, const void *Kcache,
                               const void *Vcache, float *Kbar_cache, int32_t *idx, void *o, float *lse, void *ws,
                               size_t ws_bytes, ssa_stream_t stream) {
    Shape S;
    ssa_status_t e = check_dims(dims, S, true);
    if (e != SSA_OK) return e;
    if (!cache_len || !q || !Kcache || !Vcache || !Kbar_cache || !idx || !o || !lse) return SSA_ERR_INVALID_ARG;
    if (S.dtype != SSA_DT_BF16 || S.d != 128 || S.nb > kDecMaxBlocks || S.G > kDecMaxGroup) return SSA_ERR_UNSUPPORTED;
    // the selected blocks are bulk-copied and the query rows read in 16-byte units: 16-byte aligned bases
    if ((reinterpret_cast<uintptr_t>(Kcache) | reinterpret_cast<uintptr_t>(Vcache) | reinterpret_cast<uintptr_t>(q)) &
        15u)
        return SSA_ERR_INVALID_ARG;
    if ((e = check_ws(S, SSA_OP_DECODE, ws, ws_bytes)) != SSA_OK) return e;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    float *opart = static_cast<float *>(ws);
    float *lsepart = reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + align_up(S.BH * S.k * S.d * 4));
    const unsigned bhk = static_cast<unsigned>(S.BHk);
    const size_t sm = (128 + (S.nb > 256 ? S.nb : 256)) * sizeof(float);
    // the warp search holds ceil(nb / 32) scores per lane (8, 16 or 32)
    auto sel = S.nb <= 256 ? decode_select_kernel<8> : S.nb <= 512 ? decode_select_kernel<16> : decode_select_kernel<32>;
    sel<<<bhk, kDecThreads, sm, st>>>(cache_len, (const __nv_bfloat16 *)q, (const __nv_bfloat16 *)Kcache, Kbar_cache,
                                      idx, S.Hk, S.G, S.T, S.s, S.k, S.nb);
    if (S.s == 128) {  // tensor-core attend: blocks brought in by TMA, both products on tcgen05
        CUtensorMap tmK, tmV;
        if (!make_tmap(&tmK, Kcache, S.krows, 128) || !make_tmap(&tmV, Vcache, S.krows, 128)) return SSA_ERR_CUDA;
        if (!set_smem(decode_attend_tc_kernel, DecTcSmem::kTotal)) return SSA_ERR_CUDA;
        decode_attend_tc_kernel<<<dim3(bhk, S.k), 128, DecTcSmem::kTotal, st>>>(
            tmK, tmV, cache_len, (const __nv_bfloat16 *)q, idx, opart, lsepart, S.Hk, S.G, S.T, S.k,
            S.scale * 1.4426950408889634f);
    } else {  // blocks of 64 keys: CUDA-core attend, the group padded to a power of two
        auto launch = S.G <= 1   ? launch_decode_attend<1>
                      : S.G <= 2 ? launch_decode_attend<2>
                      : S.G <= 4 ? launch_decode_attend<4>
                      : S.G <= 8 ? launch_decode_attend<8>
                                 : launch_decode_attend<16>;
        if (!launch(S, st, cache_len, q, Kcache, Vcache, idx, opart, lsepart)) return SSA_ERR_CUDA;
    }
    const unsigned rows = static_cast<unsigned>(S.BH);
    decode_combine_kernel<<<(rows + kDecThreads / 32 - 1) / (kDecThreads / 32), kDecThreads, 0, st>>>(
        opart, lsepart, (__nv_bfloat16 *)o, lse, static_cast<int>(rows), S.k);
    return launch_status();
}

ssa_status_t ssa_rope(const ssa_dims_t *dims, void *X, int heads, int pos0, float base, float factor, int transpose,
                      ssa_stream_t stream) {
    Shape S;
    ssa_status_t e = check_dims(dims, S, false);
    if (e != SSA_OK) return e;
    if (!X || heads < 1 || pos0 < 0 || !(base > 1.f) || !std::isfinite(base) || !(factor > 0.f) ||
        !std::isfinite(factor))
        return SSA_ERR_INVALID_ARG;
    if (static_cast<size_t>(S.B) * heads * S.T > 0x7FFFFFFFull) return SSA_ERR_UNSUPPORTED;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const dim3 grid((S.T + kRopeRows - 1) / kRopeRows, S.B);
    const double l2b = std::log2(static_cast<double>(base)), inv = 1.0 / static_cast<double>(factor);
    if (S.dtype == SSA_DT_BF16)
        rope_kernel<__nv_bfloat16><<<grid, 256, 0, st>>>((__nv_bfloat16 *)X, heads, S.T, S.d, pos0, l2b, inv,
                                                         transpose ? 1 : 0);
    else
        rope_kernel<float><<<grid, 256, 0, st>>>((float *)X, heads, S.T, S.d, pos0, l2b, inv, transpose ? 1 : 0);
    return launch_status();
}

ssa_status_t ssa_rope_axes(const ssa_dims_t *dims, const int32_t *pos, int axes, const int32_t *sections,
                           unsigned flags, float base, float factor, const void *Q, const int64_t *q_strides, void *Qr,
                           const int64_t *qr_strides, const void *K, const int64_t *k_strides, void *Kr,
                           const int64_t *kr_strides, ssa_stream_t stream) {
    if (!dims || !pos || !sections || (!Q && !K) || !Q != !Qr || !K != !Kr) return SSA_ERR_INVALID_ARG;
    const int B = dims->B, T = dims->T, d = dims->d, H = dims->H, Hk = dims->Hkv ? dims->Hkv : dims->H;
    if (B < 1 || T < 1 || d < 1 || H < 1 || Hk < 1 || axes < 1 || axes > kRopeMaxAxes) return SSA_ERR_INVALID_ARG;
    if (dims->dtype != SSA_DT_BF16 && dims->dtype != SSA_DT_FP32) return SSA_ERR_INVALID_ARG;
    if (flags & ~static_cast<unsigned>(SSA_ROPE_TRANSPOSE | SSA_ROPE_INTERLEAVED | SSA_ROPE_OWN_LADDER))
        return SSA_ERR_INVALID_ARG;
    if (!(base > 1.f) || !std::isfinite(base) || !(factor > 0.f) || !std::isfinite(factor)) return SSA_ERR_INVALID_ARG;
    if (d != 64 && d != 128) return SSA_ERR_UNSUPPORTED;
    const int half = d / 2;
    int left[kRopeMaxAxes];
    int64_t sum = 0;
    for (int a = 0; a < axes; ++a) {
        if (sections[a] < 1) return SSA_ERR_INVALID_ARG;
        sum += sections[a];
        left[a] = sections[a];
    }
    if (sum != half) return SSA_ERR_INVALID_ARG;
    const int64_t BT = static_cast<int64_t>(B) * T;
    if (BT > 0x7FFFFFFFll || H > 65536 || Hk > 65536) return SSA_ERR_UNSUPPORTED;
    const int esz = dims->dtype == SSA_DT_BF16 ? 2 : 4;
    // strides: rows of one tensor must not share elements when it is written; 16-byte accesses
    auto tensor = [&](RopeAxesTensor &X, const void *in, const int64_t *is, void *out, const int64_t *os, int heads) {
        X.in = in;
        X.out = out;
        X.heads = in ? heads : 0;
        const int64_t contiguous[3] = {static_cast<int64_t>(heads) * T * d, static_cast<int64_t>(T) * d, d};
        const int64_t extent[3] = {B, heads, T};
        for (int i = 0; i < 3; ++i) {
            X.is[i] = is ? is[i] : contiguous[i];
            X.os[i] = os ? os[i] : contiguous[i];
            if (extent[i] == 1) X.is[i] = X.os[i] = 0;
        }
        if (!in) return true;
        int order[3] = {0, 1, 2};
        for (int i = 0; i < 3; ++i) {
            if (X.is[i] < 0 || X.is[i] * esz % 16 || X.os[i] * esz % 16) return false;
            if (in == out && X.is[i] != X.os[i]) return false;
            for (int j = i; j > 0 && X.os[order[j]] < X.os[order[j - 1]]; --j) {
                const int a = order[j];
                order[j] = order[j - 1];
                order[j - 1] = a;
            }
        }
        int64_t span = d;  // elements that the dimensions of smaller strides cover
        for (int i = 0; i < 3; ++i) {
            const int a = order[i];
            if (extent[a] == 1) continue;
            if (X.os[a] < span) return false;
            span += X.os[a] * (extent[a] - 1);
        }
        return ((reinterpret_cast<uintptr_t>(in) | reinterpret_cast<uintptr_t>(out)) & 15u) == 0;
    };
    RopeAxesTensor XQ, XK;
    if (!tensor(XQ, Q, q_strides, Qr, qr_strides, H) || !tensor(XK, K, k_strides, Kr, kr_strides, Hk))
        return SSA_ERR_INVALID_ARG;
    RopeAxesTable tab;
    const double l2b = std::log2(static_cast<double>(base));
    const double per = 1.0 / (6.283185307179586476925 * static_cast<double>(factor));
    for (int i = 0, a = 0; i < half; ++i) {  // contiguous sections, or pairs dealt out in turn
        while (left[a] == 0) a = (a + 1) % axes;
        const int rank = sections[a] - left[a]--;
        const double power = (flags & SSA_ROPE_OWN_LADDER) ? static_cast<double>(rank) / sections[a]
                                                           : static_cast<double>(i) / half;
        tab.axis[i] = static_cast<uint8_t>(a);
        tab.turns[i] = std::exp2(-power * l2b) * per;
        if (flags & SSA_ROPE_INTERLEAVED) a = (a + 1) % axes;
    }
    for (int i = half; i < 64; ++i) tab.axis[i] = 0, tab.turns[i] = 0.0;
    // tokens per CTA: 8 where there are many (16: 118 and 49 us instead of 115 and 46 us for 32K tokens of 40 bf16
    // heads of 128 and 16K of 32 fp32 heads of 64, whose last wave is longer), down to one, so that at
    // least two CTAs per SM share the work
    int rows = 1;
    while (rows < kRopeAxesRows && BT > static_cast<int64_t>(rows) * 2 * kCacheSms) rows *= 2;
    const unsigned grid = static_cast<unsigned>((BT + rows - 1) / rows);
    const float sign = (flags & SSA_ROPE_TRANSPOSE) ? -1.f : 1.f;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (dims->dtype == SSA_DT_BF16)
        rope_axes_kernel<__nv_bfloat16><<<grid, kRopeAxesThreads, 0, st>>>(tab, pos, BT, T, half, rows, sign, XQ, XK);
    else
        rope_axes_kernel<float><<<grid, kRopeAxesThreads, 0, st>>>(tab, pos, BT, T, half, rows, sign, XQ, XK);
    return launch_status();
}

ssa_status_t ssa_cache_append(const ssa_dims_t *dims, int n, const int32_t *cache_len, const int32_t *n_new,
                              const void *K, const int64_t *k_strides, const void *V, const int64_t *v_strides,
                              void *K8, float *Kscale, void *V8, float *Vscale, float *Kbar, ssa_stream_t stream) {
    Shape S;
    const ssa_status_t e = check_cache_dims(dims, S);
    if (e != SSA_OK) return e;
    if (!cache_len || !K || !V || !K8 || !Kscale || !V8 || !Vscale || n < 1 || n > S.T) return SSA_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(K) | reinterpret_cast<uintptr_t>(V) | reinterpret_cast<uintptr_t>(K8) |
         reinterpret_cast<uintptr_t>(V8) | reinterpret_cast<uintptr_t>(Kbar)) & 15u)
        return SSA_ERR_INVALID_ARG;
    CacheRows X[2];
    for (int i = 0; i < 2; ++i) {
        const int64_t *st = i ? v_strides : k_strides;
        X[i].p = static_cast<const __nv_bfloat16 *>(i ? V : K);
        const int64_t contiguous[3] = {static_cast<int64_t>(S.Hk) * n * S.d, static_cast<int64_t>(n) * S.d, S.d};
        const int64_t extent[3] = {S.B, S.Hk, n};
        for (int a = 0; a < 3; ++a) {
            X[i].st[a] = extent[a] == 1 ? 0 : st ? st[a] : contiguous[a];
            if (X[i].st[a] < 0 || X[i].st[a] % 8) return SSA_ERR_INVALID_ARG;  // 16-byte reads
        }
    }
    cudaStream_t cst = reinterpret_cast<cudaStream_t>(stream);
    if (n == 1) {
        auto token = S.s == 128 ? cache_append_token_kernel<128> : cache_append_token_kernel<64>;
        token<<<static_cast<unsigned>((S.BHk + 3) / 4), 128, 0, cst>>>(
            cache_len, n_new, X[0], X[1], static_cast<uint8_t *>(K8), Kscale, static_cast<uint8_t *>(V8), Vscale, Kbar,
            static_cast<int>(S.BHk), S.Hk, S.T);
        return launch_status();
    }
    int blocks = (n + S.s - 2) / S.s + 1;
    if (blocks > S.nb) blocks = S.nb;
    const dim3 grid(static_cast<unsigned>(S.BHk), blocks, 2);
    auto kernel = S.s == 128 ? cache_append_kernel<128> : cache_append_kernel<64>;
    kernel<<<grid, append_threads(S.s), 0, cst>>>(
        cache_len, n_new, n, X[0], X[1], static_cast<uint8_t *>(K8), Kscale, static_cast<uint8_t *>(V8), Vscale, Kbar,
        S.Hk, S.T);
    return launch_status();
}

ssa_status_t ssa_cache_decode(const ssa_dims_t *dims, const int32_t *cache_len, const void *q, const void *K8,
                              const float *Kscale, const void *V8, const float *Vscale, const float *Kbar, int32_t *idx,
                              void *o, float *lse, const float *weight_in, float *weight_out, void *ws, size_t ws_bytes,
                              ssa_stream_t stream) {
    Shape S;
    const ssa_status_t e = check_cache_dims(dims, S);
    if (e != SSA_OK) return e;
    if (!cache_len || !q || !K8 || !Kscale || !V8 || !Vscale || !o || !lse) return SSA_ERR_INVALID_ARG;
    if ((S.k > 0 && !idx) || (S.k > 1 && !Kbar) || (weight_in && !weight_out)) return SSA_ERR_INVALID_ARG;
    if (S.G > kCacheMaxGroup) return SSA_ERR_UNSUPPORTED;
    if ((reinterpret_cast<uintptr_t>(K8) | reinterpret_cast<uintptr_t>(V8) | reinterpret_cast<uintptr_t>(q) |
         reinterpret_cast<uintptr_t>(o) | reinterpret_cast<uintptr_t>(Kbar)) & 15u)
        return SSA_ERR_INVALID_ARG;
    const CacheWs W = cache_ws(S);
    if (!ws || ws_bytes < W.bytes || (reinterpret_cast<uintptr_t>(ws) & 15u)) return SSA_ERR_WORKSPACE;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    float *opart = static_cast<float *>(ws);
    float2 *ml = reinterpret_cast<float2 *>(static_cast<uint8_t *>(ws) + W.ml);
    float2 *block_ml = weight_out ? reinterpret_cast<float2 *>(static_cast<uint8_t *>(ws) + W.blocks) : nullptr;
    const unsigned bhk = static_cast<unsigned>(S.BHk);
    const __nv_bfloat16 *qb = static_cast<const __nv_bfloat16 *>(q);
    CUtensorMap tmK, tmV;
    if (!make_tmap_codes(&tmK, K8, S.krows, S.s) || !make_tmap_codes(&tmV, V8, S.krows, S.s)) return SSA_ERR_CUDA;
    if (S.k > 0) {
        // CTAs per pair: a second one only from 128 blocks on (each scores 64 at a time), while SMs are idle.  The whole
        // call, k = 16, s = 128, G = 4, with 1, 2, 4 and 8 (us): 1024 blocks, 8 pairs 28.1, 22.8, 20.5, 18.7 and 37
        // pairs 34.1, 27.9, 23.9, 22.8; 256 blocks, 37 pairs 18.0, 17.2, 16.4, 17.1, 74 pairs 23.7, 22.5, 22.4, 24.6
        // and 512 pairs 67.5, 70.5, 76.9, 90.4; 128 blocks, 74 pairs 21.0, 21.0, 21.1, 23.4
        unsigned parts = 1;
        while (parts < 8 && parts * 2 * bhk <= 2u * kCacheSms && static_cast<unsigned>(S.nb) >= 128 * parts) parts *= 2;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = parts;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(bhk * parts);
        cfg.blockDim = dim3(kTopThreads);
        cfg.dynamicSmemBytes = static_cast<size_t>(S.nb) * 4;
        cfg.stream = st;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        if (cudaLaunchKernelEx(&cfg, cache_select_kernel, cache_len, qb, Kbar, idx, S.Hk, S.G, S.T, S.s, S.k, S.nb) !=
            cudaSuccess) {
            cudaGetLastError();
            return SSA_ERR_CUDA;
        }
    }
    // no more CTAs than the caches can have tiles
    const size_t most = S.BHk * ((static_cast<size_t>(S.k > 0 ? S.k : S.nb) * S.s + 127) / 128);
    const unsigned grid = static_cast<unsigned>(most < cache_grid(S.G) ? most : cache_grid(S.G));
    auto attend = [&](auto kernel, size_t smem) {
        if (!set_smem(kernel, smem)) return false;
        const float scale_log2 = static_cast<float>(S.scale * 1.4426950408889634);
        if (S.k > 0)
            return launch_dependent(kernel, grid, 128, smem, st, tmK, tmV, cache_len, qb, Kscale, Vscale, idx, opart, ml,
                                    block_ml, S.B, S.Hk, S.G, S.T, S.k, S.nb, scale_log2);
        kernel<<<grid, 128, smem, st>>>(tmK, tmV, cache_len, qb, Kscale, Vscale, idx, opart, ml, block_ml, S.B, S.Hk, S.G,
                                        S.T, S.k, S.nb, scale_log2);
        return true;
    };
    auto heads = [&](auto nh) {
        constexpr int NH = decltype(nh)::value;
        return S.s == 128 ? attend(cache_attend_kernel<NH, 128>, CacheAttend<NH>::kBytes)
                          : attend(cache_attend_kernel<NH, 64>, CacheAttend<NH>::kBytes);
    };
    const int NH = cache_heads(S.G);
    const bool ok = NH == 4    ? heads(std::integral_constant<int, 4>())
                    : NH == 8  ? heads(std::integral_constant<int, 8>())
                    : NH == 16 ? heads(std::integral_constant<int, 16>())
                               : heads(std::integral_constant<int, 32>());
    if (!ok) return SSA_ERR_CUDA;
    // partials per pair: about grid / pairs, each of 128 values per head
    const unsigned split = grid < 16 * bhk ? 0 : grid < 64 * bhk ? 1 : 4;
    auto combine = split == 0   ? cache_combine_kernel<0>
                   : split == 1 ? cache_combine_kernel<1>
                                : cache_combine_kernel<4>;
    const unsigned head_ctas = split ? split * static_cast<unsigned>(S.BH) : bhk * ((S.G + 7) / 8);
    const size_t weight_ctas = split && weight_out ? S.BHk * ((S.nb + 255) / 256) : 0;
    if (!launch_dependent(combine, dim3(static_cast<unsigned>(head_ctas + weight_ctas)), 256, 0, st, cache_len, opart, ml,
                          block_ml, idx, static_cast<__nv_bfloat16 *>(o), lse, weight_in, weight_out, S.B, S.Hk, S.G, S.T,
                          S.s, S.k, S.nb, static_cast<int>(grid), static_cast<int>(head_ctas)))
        return SSA_ERR_CUDA;
    return launch_status();
}

ssa_status_t ssa_cache_evict(const ssa_dims_t *dims, int keep, int sink, int recent, const int32_t *cache_len,
                             int32_t *new_len, const float *weight_in, float *weight_out, void *K8, float *Kscale,
                             void *V8, float *Vscale, float *Kbar, int32_t *kept, void *ws, size_t ws_bytes,
                             ssa_stream_t stream) {
    Shape S;
    const ssa_status_t e = check_cache_dims(dims, S);
    if (e != SSA_OK) return e;
    if (!cache_len || !weight_in || !K8 || !Kscale || !V8 || !Vscale || !kept) return SSA_ERR_INVALID_ARG;
    if (keep < 1 || keep > S.nb || sink < 0 || recent < 0 || sink > keep || recent > keep - sink)
        return SSA_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(K8) | reinterpret_cast<uintptr_t>(V8) | reinterpret_cast<uintptr_t>(Kbar)) & 15u)
        return SSA_ERR_INVALID_ARG;
    if (!ws || ws_bytes < cache_ws_bytes(S, SSA_OP_CACHE_EVICT) || (reinterpret_cast<uintptr_t>(ws) & 15u))
        return SSA_ERR_WORKSPACE;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    int32_t *lists = static_cast<int32_t *>(ws);
    const unsigned bhk = static_cast<unsigned>(S.BHk);
    const size_t sm = (2 * static_cast<size_t>(S.nb) + keep + 1) * 4, sm_move = static_cast<size_t>(S.nb) * 4;
    if (!set_smem(cache_evict_select_kernel, sm)) return SSA_ERR_CUDA;
    cache_evict_select_kernel<<<bhk, kTopThreads, sm, st>>>(cache_len, weight_in, weight_out, Kscale, Vscale, kept, lists,
                                                            S.Hk, S.T, S.s, S.nb, keep, sink, recent);
    const int columns = 2 * S.s * (kCacheD / 16) + (Kbar ? kCacheD * 4 / 16 : 0);
    if (!launch_dependent(cache_evict_move_kernel, dim3(bhk, (columns + kMoveThreads - 1) / kMoveThreads), kMoveThreads,
                          sm_move, st, static_cast<uint8_t *>(K8), static_cast<uint8_t *>(V8), Kbar, new_len, lists, S.Hk,
                          S.s, S.nb))
        return SSA_ERR_CUDA;
    return launch_status();
}

ssa_status_t ssa_wait_probe(uint64_t limit_ns, ssa_stream_t stream) {
    if (limit_ns < 1000u || limit_ns > 1000000000u) return SSA_ERR_INVALID_ARG;
    wait_probe_kernel<<<1, 32, 0, reinterpret_cast<cudaStream_t>(stream)>>>(limit_ns);
    return launch_status();
}

ssa_status_t ssa_get_device_error(ssa_stream_t stream) {
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (cudaStreamSynchronize(st) != cudaSuccess) return SSA_ERR_CUDA;
    unsigned int w = 0;
    if (cudaMemcpyFromSymbol(&w, g_error_word, sizeof(w)) != cudaSuccess) return SSA_ERR_CUDA;
    if (w == 0) return SSA_OK;
    const unsigned int zero = 0;
    if (cudaMemcpyToSymbol(g_error_word, &zero, sizeof(zero)) != cudaSuccess) return SSA_ERR_CUDA;
    return (w >> 24) == ERR_BAD_INPUT ? SSA_ERR_BAD_INPUT : SSA_ERR_TIMEOUT;
}

const char *ssa_status_string(ssa_status_t s) {
    switch (s) {
        case SSA_OK: return "SSA_OK";
        case SSA_ERR_INVALID_ARG: return "SSA_ERR_INVALID_ARG";
        case SSA_ERR_UNSUPPORTED: return "SSA_ERR_UNSUPPORTED";
        case SSA_ERR_WORKSPACE: return "SSA_ERR_WORKSPACE";
        case SSA_ERR_CUDA: return "SSA_ERR_CUDA";
        case SSA_ERR_TIMEOUT: return "SSA_ERR_TIMEOUT";
        case SSA_ERR_BAD_INPUT: return "SSA_ERR_BAD_INPUT";
    }
    return "SSA_ERR_UNKNOWN";
}

}  // extern "C"
