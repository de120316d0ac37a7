// api.cu -- the C ABI of libforge_attn.so (declared in include/forge_attn.h):
// argument validation, TMA tensor maps, workspace layout and kernel dispatch.
// Single translation unit: every kernel header is included here.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <mutex>

#include "forge_attn.h"

#include "bwd_aux.cuh"
#include "bwd_dkv.cuh"
#include "bwd_tc.cuh"
#include "decode.cuh"
#include "decode_paged.cuh"
#include "fwd2_tc.cuh"
#include "fwd_tc.cuh"
#include "paged.cuh"
#include "simt.cuh"
#include "sm100.cuh"
#include "varlen.cuh"
#include "varlen_f32.cuh"
#include "varlen_fwd.cuh"

namespace forge {
namespace {

// ------------------------------------------------------------------ validation
bool aligned16(const void *p) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned32(const void *p) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & 31u) == 0; }
bool aligned4(const void *p) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

forge_status check_sizes(int B, int Hq, int Hkv, int T, int D, forge_dtype dtype) {
    if (B < 1 || Hq < 1 || Hkv < 1 || T < 1 || D < 1) return FORGE_ERR_INVALID_ARG;
    if (Hq % Hkv != 0) return FORGE_ERR_INVALID_ARG;  // n_heads % n_kv_heads == 0
    if (D % 2 != 0) return FORGE_ERR_INVALID_ARG;     // head_dim even
    if (dtype != FORGE_DTYPE_F32 && dtype != FORGE_DTYPE_BF16) return FORGE_ERR_INVALID_ARG;
    if (D != 64 && D != 128 && D != 256) return FORGE_ERR_UNSUPPORTED;
    // index arithmetic limits: grid sizes and per-tensor element counts
    const long long rows = (long long)B * Hq * T;
    if ((long long)B * Hq > (1ll << 24) || T > (1 << 30) || rows * D > (1ll << 40)) return FORGE_ERR_INVALID_ARG;
    const long long ntiles = (long long)((T + 127) / 128) * B * Hq;
    if (ntiles > 0x7fffffffll) return FORGE_ERR_INVALID_ARG;
    return FORGE_OK;
}

forge_status check_scalars(float scale, int window, float softcap) {
    if (!(scale > 0.0f) || !isfinite(scale)) return FORGE_ERR_INVALID_ARG;
    if (window < 0) return FORGE_ERR_INVALID_ARG;
    if (!(softcap >= 0.0f) || !isfinite(softcap)) return FORGE_ERR_INVALID_ARG;
    return FORGE_OK;
}

int effective_window(int window, int T) { return (window >= T) ? 0 : window; }

// Grid for kernels that take one (batch, head) pair per block row: the pairs go
// on y, and past the 65535 that y allows, on z (the kernels' `pair_index`); x
// is the kernel's own split of the rows or keys.
dim3 pair_grid(unsigned x, long long pairs) {
    const long long y = pairs < 65535 ? pairs : 65535;
    return dim3(x, (unsigned)y, (unsigned)((pairs + y - 1) / y));
}

// ------------------------------------------------------------- workspace layout
// [ delta: B*Hq*T f32, 256-aligned ][ dq accumulator: B*Hq*Tpad*D f32 (bf16 only) ]
size_t round256(size_t x) { return (x + 255) & ~size_t(255); }
int tpad_of(int T) { return (T + 127) / 128 * 128; }
size_t delta_bytes(int B, int Hq, int T) { return round256(sizeof(float) * (size_t)B * Hq * T); }
size_t acc_bytes(int B, int Hq, int T, int D) { return round256(sizeof(float) * (size_t)B * Hq * tpad_of(T) * D); }

// Blocks of bwd_preprocess for `rows` rows of head dim D: 8 warps a block, each
// warp 32 / min(32, D / 8) rows.
unsigned preprocess_grid(long rows, int D) {
    const int lpr = D / 8 < 32 ? D / 8 : 32;
    const long per_block = 8L * (32 / lpr);
    return (unsigned)((rows + per_block - 1) / per_block);
}

// ----------------------------------------------------------------- tensor maps
typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                  const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
    static EncodeTiledFn fn = nullptr;
    if (fn == nullptr) {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(ptr);
    }
    return fn;
}

// [BH][T][D] bf16 viewed as a 3D tensor (D innermost); box = 64 columns x rows x 1,
// 128-byte swizzle (the layout the tcgen05 descriptors describe). Rows past T
// read as zeros.
bool make_map(CUtensorMap *map, const void *base, int D, int T, long long BH, int box_rows) {
    EncodeTiledFn enc = encode_fn();
    if (enc == nullptr) return false;
    cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)T, (cuuint64_t)BH};
    cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)D * 2 * (cuuint64_t)T};
    cuuint32_t box[3] = {64, (cuuint32_t)box_rows, 1};
    cuuint32_t estr[3] = {1, 1, 1};
    CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, estr,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS;
}

// A packed [rows][H][D] bf16 tensor whose rows are `stride` elements apart, viewed as
// [H][rows][D] (same box and swizzle): a head's rows are `stride` apart, so a box holds
// box_rows consecutive tokens of one head. Rows past `rows` read as zeros.
bool make_map_rows(CUtensorMap *map, const void *base, int D, int rows, int H, size_t stride, int box_rows) {
    EncodeTiledFn enc = encode_fn();
    if (enc == nullptr) return false;
    cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)rows, (cuuint64_t)H};
    cuuint64_t strides[2] = {(cuuint64_t)stride * 2, (cuuint64_t)D * 2};
    cuuint32_t box[3] = {64, (cuuint32_t)box_rows, 1};
    cuuint32_t estr[3] = {1, 1, 1};
    CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, estr,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS;
}

// [BH][Tpad][D] f32 accumulator as a 3D tensor; box = 32 columns (128 bytes) x
// rows x 1 with the 128-byte swizzle, the layout of the dQ staging tiles.
bool make_map_acc(CUtensorMap *map, const float *base, int D, int Tpad, long long BH, int box_rows) {
    EncodeTiledFn enc = encode_fn();
    if (enc == nullptr) return false;
    cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)Tpad, (cuuint64_t)BH};
    cuuint64_t strides[2] = {(cuuint64_t)D * 4, (cuuint64_t)D * 4 * (cuuint64_t)Tpad};
    cuuint32_t box[3] = {32, (cuuint32_t)box_rows, 1};
    cuuint32_t estr[3] = {1, 1, 1};
    CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, const_cast<float *>(base), dims, strides, box, estr,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS;
}

// Text of the last CUDA error a call of this thread ran into (for diagnostics).
thread_local const char *t_last_cuda_error = "no error";

forge_status cuda_status(cudaError_t e) {
    if (e == cudaSuccess) return FORGE_OK;
    t_last_cuda_error = cudaGetErrorString(e);
    return FORGE_ERR_CUDA;
}

forge_status launch_status() { return cuda_status(cudaGetLastError()); }

// SM count of the current device (cached per device), for persistent grids.
int sm_count() {
    static int cache[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 148;
    if (cache[dev] == 0) {
        int n = 0;
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) n = 148;
        cache[dev] = n;
    }
    return cache[dev];
}

// L2 size of the current device in bytes (cached per device)
long long l2_bytes() {
    static long long cache[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 126LL << 20;
    if (cache[dev] == 0) {
        int n = 0;
        if (cudaDeviceGetAttribute(&n, cudaDevAttrL2CacheSize, dev) != cudaSuccess || n < 1) n = 126 << 20;
        cache[dev] = n;
    }
    return cache[dev];
}

// Launch with programmatic stream serialization: the kernel may start while the
// previous kernel on the stream finishes (its prologue overlaps that kernel's
// tail); the kernels launched this way call griddep_wait before touching global
// memory, so the stream order of all memory effects is kept.
template <typename... KArgs, typename... Args>
forge_status launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t st,
                        Args &&...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cuda_status(cudaLaunchKernelEx(&cfg, kernel, static_cast<Args &&>(args)...));
}

template <typename K>
forge_status set_smem(K kernel, size_t bytes) {
    if (bytes <= 48 * 1024) return FORGE_OK;
    return cuda_status(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes));
}

// ----------------------------------------------------------------- dispatchers
template <int D>
forge_status fwd_tc(const void *q, const void *k, const void *v, void *o, float *lse, int B, int Hq, int Hkv, int T,
                    float scale, int window, float softcap, const float *sink, float *max_logit, cudaStream_t st) {
    using C = FwdTc<D>;
    CUtensorMap mq, mk, mv;
    if (!make_map(&mq, q, D, T, (long long)B * Hq, 128) || !make_map(&mk, k, D, T, (long long)B * Hkv, 128) ||
        !make_map(&mv, v, D, T, (long long)B * Hkv, 128))
    {
        t_last_cuda_error = "cuTensorMapEncodeTiled failed";
        return FORGE_ERR_CUDA;
    }
    FwdParams p;
    p.o = static_cast<__nv_bfloat16 *>(o);
    p.lse = lse;
    p.B = B; p.Hq = Hq; p.Hkv = Hkv; p.T = T; p.window = window;
    p.num_qt = (T + 127) / 128;
    p.scale_log2 = scale * kLog2e;
    p.softcap = softcap;
    p.cap_in = softcap > 0.0f ? scale / softcap : 0.0f;
    p.cap_out = softcap * kLog2e;
    p.sink = sink;
    p.max_logit = max_logit;
    if constexpr (D == 256) {
        // one query tile per CTA: S0, S1 and the 256-column O fill TMEM
        if (set_smem(fwd_tc_kernel<D>, C::SMEM) != FORGE_OK) return FORGE_ERR_CUDA;
        const unsigned grid = (unsigned)(p.num_qt * B * Hq);
        fwd_tc_kernel<D><<<grid, C::THREADS, C::SMEM, st>>>(mq, mk, mv, p);
    } else {
        // two query tiles per CTA
        using C2 = Fwd2Tc<D>;
        CUtensorMap mo;
        if (!make_map(&mo, o, D, T, (long long)B * Hq, 128)) {
            t_last_cuda_error = "cuTensorMapEncodeTiled failed";
            return FORGE_ERR_CUDA;
        }
        if (set_smem(fwd2_tc_kernel<D, true>, C2::SMEM) != FORGE_OK ||
            set_smem(fwd2_tc_kernel<D, false>, C2::SMEM) != FORGE_OK)
            return FORGE_ERR_CUDA;
        // Persistent (one CTA per SM, the most shared memory and TMEM allow) for
        // short sequences, whose items are too light to amortise a CTA's start;
        // one CTA per item otherwise, where the hardware's dynamic placement
        // balances the uneven items better than a static order (measured forward
        // times: 16K global layer 2.57 ms persistent against 2.40 ms one CTA per
        // item; T = 512, head dim 64: 0.039 ms persistent against 0.045 ms).
        const long long items = (long long)((p.num_qt + 1) / 2) * B * Hq;
        const bool persistent = p.num_qt <= 8;
        const unsigned grid = (unsigned)(persistent && items > sm_count() ? sm_count() : items);
        // (the persistent form with grid = items takes the same items; the flag
        // only removes the work-item loop from the one-item-per-CTA code)
        if (persistent)
            return launch_pdl(fwd2_tc_kernel<D, true>, dim3(grid), dim3(C2::THREADS), C2::SMEM, st, mq, mk, mv, mo, p);
        return launch_pdl(fwd2_tc_kernel<D, false>, dim3(grid), dim3(C2::THREADS), C2::SMEM, st, mq, mk, mv, mo, p);
    }
    return launch_status();
}

// Single-tile tensor-core forward with separate key and value head dims.
template <int DK, int DV>
forge_status fwd_tc_dkv(const void *q, const void *k, const void *v, void *o, float *lse, int B, int Hq, int Hkv,
                        int T, float scale, int window, float softcap, cudaStream_t st) {
    using C = FwdTc<DK, DV>;
    CUtensorMap mq, mk, mv;
    if (!make_map(&mq, q, DK, T, (long long)B * Hq, 128) || !make_map(&mk, k, DK, T, (long long)B * Hkv, 128) ||
        !make_map(&mv, v, DV, T, (long long)B * Hkv, 128)) {
        t_last_cuda_error = "cuTensorMapEncodeTiled failed";
        return FORGE_ERR_CUDA;
    }
    FwdParams p;
    p.o = static_cast<__nv_bfloat16 *>(o);
    p.lse = lse;
    p.B = B; p.Hq = Hq; p.Hkv = Hkv; p.T = T; p.window = window;
    p.num_qt = (T + 127) / 128;
    p.scale_log2 = scale * kLog2e;
    p.softcap = softcap;
    p.cap_in = softcap > 0.0f ? scale / softcap : 0.0f;
    p.cap_out = softcap * kLog2e;
    p.sink = nullptr;
    p.max_logit = nullptr;
    if (set_smem(fwd_tc_kernel<DK, DV>, C::SMEM) != FORGE_OK) return FORGE_ERR_CUDA;
    fwd_tc_kernel<DK, DV><<<(unsigned)(p.num_qt * B * Hq), C::THREADS, C::SMEM, st>>>(mq, mk, mv, p);
    return launch_status();
}

template <typename T_, int DK, int DV = DK>
forge_status fwd_simt(const void *q, const void *k, const void *v, void *o, float *lse, int B, int Hq, int Hkv, int T,
                      float scale, int window, float softcap, const float *sink, float *max_logit, cudaStream_t st) {
    const size_t sm = simt_fwd_smem<DK, DV>();
    if (set_smem(simt_fwd<T_, DK, DV>, sm) != FORGE_OK) return FORGE_ERR_CUDA;
    const dim3 grid = pair_grid((unsigned)((T + kSimtRows - 1) / kSimtRows), (long long)B * Hq);
    simt_fwd<T_, DK, DV><<<grid, kSimtThreads, sm, st>>>(static_cast<const T_ *>(q), static_cast<const T_ *>(k),
                                                     static_cast<const T_ *>(v), static_cast<T_ *>(o), lse, Hq, Hkv,
                                                     T, scale, window, softcap, sink, max_logit, B * Hq);
    return launch_status();
}

template <typename T_, int DK, int DV = DK>
forge_status bwd_simt(const void *q, const void *k, const void *v, const float *lse, const void *dO,
                      const float *delta, void *dq, void *dk, void *dv, int B, int Hq, int Hkv, int T, float scale,
                      int window, float softcap, cudaStream_t st) {
    const size_t sm1 = simt_bwd_dq_smem<DK, DV>(), sm2 = simt_bwd_dkdv_smem<DK, DV>();
    if (set_smem(simt_bwd_dq<T_, DK, DV>, sm1) != FORGE_OK || set_smem(simt_bwd_dkdv<T_, DK, DV>, sm2) != FORGE_OK)
        return FORGE_ERR_CUDA;
    const dim3 g1 = pair_grid((unsigned)((T + kSimtRows - 1) / kSimtRows), (long long)B * Hq);
    simt_bwd_dq<T_, DK, DV><<<g1, kSimtThreads, sm1, st>>>(
        static_cast<const T_ *>(q), static_cast<const T_ *>(k), static_cast<const T_ *>(v), lse,
        static_cast<const T_ *>(dO), delta, static_cast<T_ *>(dq), Hq, Hkv, T, scale, window, softcap, B * Hq);
    forge_status s = launch_status();
    if (s != FORGE_OK) return s;
    const dim3 g2 = pair_grid((unsigned)((T + kSimtRows - 1) / kSimtRows), (long long)B * Hkv);
    simt_bwd_dkdv<T_, DK, DV><<<g2, kSimtThreads, sm2, st>>>(
        static_cast<const T_ *>(q), static_cast<const T_ *>(k), static_cast<const T_ *>(v), lse,
        static_cast<const T_ *>(dO), delta, static_cast<T_ *>(dk), static_cast<T_ *>(dv), Hq, Hkv, T, scale, window,
        softcap, B * Hkv);
    return launch_status();
}

template <int D>
forge_status bwd_tc(const void *q, const void *k, const void *v, const float *lse, const void *dO,
                    const float *delta, float *acc, void *dk, void *dv, int B, int Hq, int Hkv, int T, float scale,
                    int window, float softcap, cudaStream_t st) {
    using C = BwdTc<D>;
    CUtensorMap mq, mk, mv, mdo, macc;
    if (!make_map(&mq, q, D, T, (long long)B * Hq, C::BM) || !make_map(&mk, k, D, T, (long long)B * Hkv, 128) ||
        !make_map(&mv, v, D, T, (long long)B * Hkv, 128) || !make_map(&mdo, dO, D, T, (long long)B * Hq, C::BM) ||
        !make_map_acc(&macc, acc, D, tpad_of(T), (long long)B * Hq, C::BM)) {
        t_last_cuda_error = "cuTensorMapEncodeTiled failed";
        return FORGE_ERR_CUDA;
    }
    BwdParams p;
    p.lse = lse;
    p.delta = delta;
    p.dq_acc = acc;
    p.dk = static_cast<__nv_bfloat16 *>(dk);
    p.dv = static_cast<__nv_bfloat16 *>(dv);
    p.B = B; p.Hq = Hq; p.Hkv = Hkv; p.T = T; p.Tpad = tpad_of(T); p.window = window;
    p.num_kt = (T + 127) / 128;
    p.scale = scale;
    p.scale_log2 = scale * kLog2e;
    p.softcap = softcap;
    p.cap_in = softcap > 0.0f ? scale / softcap : 0.0f;
    p.cap_out = softcap * kLog2e;
    // descending query tiles where it measured faster: global causal attention at
    // head dim <= 128, T <= 8192, with Q, dO and the f32 dq accumulator larger
    // than L2 (bwd_step in bwd_tc.cuh)
    const double operand_bytes = (double)B * Hq * T * D * (2 + 2 + 4);
    p.q_desc = window == 0 && D <= 128 && T <= 8192 && operand_bytes > (double)l2_bytes() ? 1 : 0;
    if (set_smem(bwd_tc_kernel<D>, C::SMEM) != FORGE_OK) return FORGE_ERR_CUDA;
    // persistent: one CTA per SM (the kernel's shared memory and TMEM allow no
    // more), each walking its share of the work items
    const long long items = (long long)p.num_kt * B * Hkv * C::NSPLIT;
    const unsigned grid = (unsigned)(items < sm_count() ? items : sm_count());
    return launch_pdl(bwd_tc_kernel<D>, dim3(grid), dim3(C::THREADS), C::SMEM, st, mq, mk, mv, mdo, macc, p);
}

// bf16 backward with separate key and value head dims: the dK/dV kernel (one CTA
// per key tile and KV head), then the dQ kernel (one CTA per query tile and
// query head). Both read Delta from the workspace and write their outputs.
template <int DK, int DV>
forge_status bwd_tc_dkv(const void *q, const void *k, const void *v, const float *lse, const void *dO,
                        const float *delta, void *dq, void *dk, void *dv, int B, int Hq, int Hkv, int T, float scale,
                        int window, float softcap, cudaStream_t st) {
    using CA = BwdKvTc<DK, DV>;
    using CQ = BwdQTc<DK, DV>;
    CUtensorMap mq, mk, mv, mdo, mk64, mv64;
    if (!make_map(&mq, q, DK, T, (long long)B * Hq, 128) || !make_map(&mk, k, DK, T, (long long)B * Hkv, 128) ||
        !make_map(&mv, v, DV, T, (long long)B * Hkv, 128) || !make_map(&mdo, dO, DV, T, (long long)B * Hq, 128) ||
        !make_map(&mk64, k, DK, T, (long long)B * Hkv, CQ::BN) || !make_map(&mv64, v, DV, T, (long long)B * Hkv, CQ::BN)) {
        t_last_cuda_error = "cuTensorMapEncodeTiled failed";
        return FORGE_ERR_CUDA;
    }
    BwdParams p;
    p.lse = lse;
    p.delta = delta;
    p.dq_acc = nullptr;
    p.dk = static_cast<__nv_bfloat16 *>(dk);
    p.dv = static_cast<__nv_bfloat16 *>(dv);
    p.B = B; p.Hq = Hq; p.Hkv = Hkv; p.T = T; p.Tpad = tpad_of(T); p.window = window;
    p.num_kt = (T + 127) / 128;
    p.scale = scale;
    p.scale_log2 = scale * kLog2e;
    p.softcap = softcap;
    p.cap_in = softcap > 0.0f ? scale / softcap : 0.0f;
    p.cap_out = softcap * kLog2e;
    p.q_desc = 0;
    if (set_smem(bwd_dkdv_tc_kernel<DK, DV>, CA::SMEM) != FORGE_OK) return FORGE_ERR_CUDA;
    bwd_dkdv_tc_kernel<DK, DV><<<(unsigned)(p.num_kt * B * Hkv), CA::THREADS, CA::SMEM, st>>>(mq, mk, mv, mdo, p);
    forge_status s = launch_status();
    if (s != FORGE_OK) return s;
    BwdQParams pq;
    pq.lse = lse;
    pq.delta = delta;
    pq.dq = static_cast<__nv_bfloat16 *>(dq);
    pq.B = B; pq.Hq = Hq; pq.Hkv = Hkv; pq.T = T; pq.window = window;
    pq.num_qt = (T + 127) / 128;
    pq.scale = p.scale; pq.scale_log2 = p.scale_log2; pq.softcap = p.softcap; pq.cap_in = p.cap_in;
    pq.cap_out = p.cap_out;
    if (set_smem(bwd_dq_tc_kernel<DK, DV>, CQ::SMEM) != FORGE_OK) return FORGE_ERR_CUDA;
    bwd_dq_tc_kernel<DK, DV><<<(unsigned)(pq.num_qt * B * Hq), CQ::THREADS, CQ::SMEM, st>>>(mq, mk64, mv64, mdo, pq);
    return launch_status();
}

// ------------------------------------------------------------ packed sequences
// Arguments of the two packed entry points that the dispatchers share.
struct VarArgs {
    const void *q, *k, *v;
    const int *cu;
    int num_seqs, rows, Hq, Hkv, D;
    size_t q_stride, k_stride, v_stride;
    float scale;
    int window;
    float softcap;
    const float *sink;
    forge_dtype dtype;
    cudaStream_t st;
};

// Rows of a tile of the schedule: pairs of 128-row query tiles for the two-tile
// forward, single ones at head dim 256, 128 keys in the backward, 64 rows in f32.
int var_unit(int D, forge_dtype dtype, bool backward) {
    if (dtype == FORGE_DTYPE_F32) return kVfRows;
    return !backward && D != 256 ? 256 : 128;
}
// Upper bounds that need no lengths: a sequence of n > 0 rows has at most
// n / unit + 1 tiles and n + 127 padded rows.
int var_max_items(int rows, int num_seqs, int unit) {
    const long long n = (long long)rows / unit + num_seqs;
    return (int)(n < rows ? n : rows);
}
int var_pad_rows(int rows, int num_seqs) {
    const long long n = rows + 127ll * (num_seqs < rows ? num_seqs : rows);
    return (int)((n + 127) / 128 * 128);
}

// Slots for the parts of key tiles that varlen_plan cuts. A part has about S per / (ctas
// kPlanParts) query tiles or more (S: all query tiles over the key tiles; per: items of a
// key tile), so the parts of cut tiles, which have more than that each, are at most
// 2 S / that = 2 ctas kPlanParts / per; and a sequence of n tiles has n (n + 1) / 2 query
// tiles in all.
int var_per_tile(int Hkv, int D) { return Hkv * (D == 256 ? 2 : 1); }
int var_max_slots(int rows, int tiles, int Hkv, int D) {
    const long long a = 2ll * sm_count() * kPlanParts / var_per_tile(Hkv, D) + 2;
    const long long most = rows / 128 + 1, b = tiles * (most < 64 ? most : 64);
    return (int)(a < b ? a : b);
}

forge_status check_var_sizes(int num_seqs, int rows, int Hq, int Hkv, int D, forge_dtype dtype) {
    forge_status s = check_sizes(1, Hq, Hkv, rows, D, dtype);
    if (s != FORGE_OK) return s;
    if (num_seqs < 1 || num_seqs > (1 << 20)) return FORGE_ERR_INVALID_ARG;
    // items (with the parts of cut tiles, at most var_max_slots) times heads: grids and 32-bit counts
    if (((long long)rows / 64 + num_seqs + 1188) * Hq > 0x7fffffffll) return FORGE_ERR_INVALID_ARG;
    return FORGE_OK;
}

forge_status check_var_args(const VarArgs &a) {
    forge_status s = check_var_sizes(a.num_seqs, a.rows, a.Hq, a.Hkv, a.D, a.dtype);
    if (s != FORGE_OK) return s;
    if ((s = check_scalars(a.scale, a.window, a.softcap)) != FORGE_OK) return s;
    if (!aligned16(a.q) || !aligned16(a.k) || !aligned16(a.v) || !aligned4(a.cu)) return FORGE_ERR_INVALID_ARG;
    if (a.sink != nullptr && !aligned4(a.sink)) return FORGE_ERR_INVALID_ARG;
    // rows 16 bytes apart or a multiple, under the tensor maps' 2^40 bytes, and
    // not overlapping
    const size_t es = a.dtype == FORGE_DTYPE_BF16 ? 2 : 4, most = (size_t)1 << 36;
    if (a.q_stride < (size_t)a.Hq * a.D || a.k_stride < (size_t)a.Hkv * a.D || a.v_stride < (size_t)a.Hkv * a.D ||
        a.q_stride > most || a.k_stride > most || a.v_stride > most || a.q_stride * es % 16 != 0 ||
        a.k_stride * es % 16 != 0 || a.v_stride * es % 16 != 0)
        return FORGE_ERR_INVALID_ARG;
    return FORGE_OK;
}

// Workspace: [ count ][ items ][ backward: Delta [Hq][rows] f32 ][ bf16: dq accumulator [Hq][pad_rows][D] f32 ]
//   bf16 backward:      [ cut list ][ parts [slots][Hkv][dk, dv][128][D] f32 ]
struct VarLayout {
    size_t items, delta, acc, cut, parts, bytes;
    int max_items, slots;
};
VarLayout var_layout(int num_seqs, int rows, int Hq, int Hkv, int D, forge_dtype dtype, bool backward) {
    VarLayout l;
    const int tiles = var_max_items(rows, num_seqs, var_unit(D, dtype, backward));
    const bool cuts = backward && dtype == FORGE_DTYPE_BF16;
    l.slots = cuts ? var_max_slots(rows, tiles, Hkv, D) : 0;
    // a tile cut into n parts takes n slots and is n items
    l.max_items = tiles + l.slots;
    l.items = 256;
    l.delta = l.items + round256(sizeof(VarItem) * (size_t)l.max_items);
    l.acc = l.delta + (backward ? delta_bytes(1, Hq, rows) : 0);
    l.cut = l.acc + (cuts ? round256(sizeof(float) * (size_t)Hq * var_pad_rows(rows, num_seqs) * D) : 0);
    l.parts = l.cut + (cuts ? round256(16 * ((size_t)l.slots / 2 + 1)) : 0);
    l.bytes = l.parts + sizeof(float) * (size_t)l.slots * Hkv * 256 * D;
    return l;
}

VarSched var_sched(const VarArgs &a, const VarLayout &l, void *ws, bool backward) {
    VarSched v;
    char *base = static_cast<char *>(ws);
    v.items = reinterpret_cast<const VarItem *>(base + l.items);
    v.count = static_cast<const int *>(ws);
    v.next = static_cast<int *>(ws) + 32;  // another 128-byte line than the count, which every CTA reads
    v.max_slots = l.slots;
    v.max_items = l.max_items;
    v.cut = l.slots > 0 ? reinterpret_cast<const int *>(base + l.cut) : nullptr;
    v.parts = reinterpret_cast<float *>(base + l.parts);
    v.unit = var_unit(a.D, a.dtype, backward);
    v.rows = a.rows;
    v.pad_rows = var_pad_rows(a.rows, a.num_seqs);
    return v;
}

bool sink_is_fixed(int flags) { return flags > 0 && (flags & FORGE_VARLEN_SINK_FIXED) != 0; }
bool clears_tail(int flags) { return (sink_is_fixed(flags) ? flags & ~FORGE_VARLEN_SINK_FIXED : flags) != 0; }

// Launches varlen_plan; tail: up to three tensors of `heads` x D elements a row
// whose rows behind the last sequence are cleared.
forge_status run_plan(const VarArgs &a, const VarSched &v, bool backward, void *const (&tail)[3],
                      const int (&tail_heads)[3], float *tail_lse, bool clear) {
    VarPlanParams p;
    p.cu = a.cu;
    p.num_seqs = a.num_seqs;
    p.rows = a.rows;
    p.unit = v.unit;
    p.window = a.window;
    p.backward = backward;
    p.items = const_cast<VarItem *>(v.items);
    p.count = const_cast<int *>(v.count);
    p.next = v.next;
    p.max_items = v.max_items;
    p.ctas = v.cut != nullptr ? sm_count() : 0;
    p.per_tile = var_per_tile(a.Hkv, a.D);
    // at least six steps a part, below which its loads and its epilogue cost more
    // than the balance gains
    const int G = a.Hq / a.Hkv;
    p.min_part = G >= 3 ? 2 : (6 + G - 1) / G;
    p.max_slots = v.max_slots;
    p.cut = const_cast<int *>(v.cut);
    for (int i = 0; i < 3; i++) {
        p.tail[i] = clear ? static_cast<uint4 *>(tail[i]) : nullptr;
        p.tail_chunks[i] = tail_heads[i] * a.D * (a.dtype == FORGE_DTYPE_BF16 ? 2 : 4) / 16;
    }
    p.tail_lse = clear ? tail_lse : nullptr;
    p.heads = a.Hq;
    return launch_pdl(varlen_plan, dim3(clear ? 33 : 1), dim3(kPlanThreads), 0, a.st, p);
}

FwdParams var_fwd_params(const VarArgs &a, const VarSched &v, void *o, void *o_res, float *lse, bool sink_fixed) {
    FwdParams p = {};
    p.o = static_cast<__nv_bfloat16 *>(o);
    p.lse = lse;
    p.B = 1; p.Hq = a.Hq; p.Hkv = a.Hkv; p.window = a.window;
    p.scale_log2 = a.scale * kLog2e;
    p.softcap = a.softcap;
    p.cap_in = a.softcap > 0.0f ? a.scale / a.softcap : 0.0f;
    p.cap_out = a.softcap * kLog2e;
    p.sink = a.sink;
    p.var = v;
    p.o_res = static_cast<__nv_bfloat16 *>(o_res);
    // a forward whose backward will want dsink
    p.for_dsink = a.sink != nullptr && o_res != nullptr && !sink_fixed;
    return p;
}

template <int D>
forge_status var_fwd_tc(const VarArgs &a, const VarSched &v, void *o, void *o_res, float *lse, bool sink_fixed) {
    CUtensorMap mq, mk, mv, mo;
    if (!make_map_rows(&mq, a.q, D, a.rows, a.Hq, a.q_stride, 128) ||
        !make_map_rows(&mk, a.k, D, a.rows, a.Hkv, a.k_stride, 128) ||
        !make_map_rows(&mv, a.v, D, a.rows, a.Hkv, a.v_stride, 128) ||
        !make_map_rows(&mo, o, D, a.rows, a.Hq, (size_t)a.Hq * D, 128)) {
        t_last_cuda_error = "cuTensorMapEncodeTiled failed";
        return FORGE_ERR_CUDA;
    }
    const FwdParams p = var_fwd_params(a, v, o, o_res, lse, sink_fixed);
    const long long items = (long long)v.max_items * a.Hq;
    if constexpr (D == 256) {
        using C = FwdTc<D>;
        if (set_smem(fwd_tc_kernel<D, D, true>, C::SMEM) != FORGE_OK) return FORGE_ERR_CUDA;
        return launch_pdl(fwd_tc_kernel<D, D, true>, dim3((unsigned)items), dim3(C::THREADS), C::SMEM, a.st, mq, mk, mv,
                          p);
    } else {
        using C = VarFwdTc<D>;
        const bool cap = a.softcap > 0.0f, win = a.window > 0;
        auto *kernel = p.for_dsink ? (cap ? varlen_fwd_tc<D, true, true, true> : varlen_fwd_tc<D, true, false, true>)
                       : cap ? (win ? varlen_fwd_tc<D, false, true, true> : varlen_fwd_tc<D, false, true, false>)
                             : (win ? varlen_fwd_tc<D, false, false, true> : varlen_fwd_tc<D, false, false, false>);
        if (set_smem(kernel, C::SMEM) != FORGE_OK) return FORGE_ERR_CUDA;
        // one CTA an SM for every length: its items are handed out as CTAs get done
        return launch_pdl(kernel, dim3((unsigned)(items < sm_count() ? items : sm_count())), dim3(C::THREADS), C::SMEM,
                          a.st, mq, mk, mv, mo, p);
    }
}

VfParams var_f32_params(const VarArgs &a, const VarSched &v) {
    VfParams p = {};
    p.q = static_cast<const float *>(a.q);
    p.k = static_cast<const float *>(a.k);
    p.v = static_cast<const float *>(a.v);
    p.q_row = (long long)a.q_stride;
    p.k_row = (long long)a.k_stride;
    p.v_row = (long long)a.v_stride;
    p.Hq = a.Hq; p.Hkv = a.Hkv; p.window = a.window;
    p.scale = a.scale;
    p.softcap = a.softcap;
    p.sink = a.sink;
    p.var = v;
    return p;
}

template <int D>
forge_status var_fwd_f32(const VarArgs &a, const VarSched &v, void *o, float *lse) {
    VfParams p = var_f32_params(a, v);
    p.o = static_cast<float *>(o);
    p.lse = lse;
    if (set_smem(varlen_f32_fwd<D>, vf_fwd_smem<D>()) != FORGE_OK) return FORGE_ERR_CUDA;
    const unsigned grid = (unsigned)v.max_items * (unsigned)a.Hq;
    return launch_pdl(varlen_f32_fwd<D>, dim3(grid), dim3(kVfThreads), vf_fwd_smem<D>(), a.st, p);
}

// The backward after the schedule: Delta (and the cleared accumulator), dsink, the
// main kernels, dq.
template <typename T_, int D>
forge_status var_bwd(const VarArgs &a, const VarSched &v, const void *o, const void *o_res, const float *lse, const void *dO, void *dq,
                     void *dk, void *dv, float *dsink, float *delta, float *acc) {
    const int items = v.max_items;
    // the stages around the main kernels: as many blocks as the SMs hold, each taking its share
    const long long pairs = (long long)items * a.Hq;
    const unsigned wave = (unsigned)(pairs < 8ll * sm_count() ? pairs : 8ll * sm_count());
    forge_status s = launch_pdl(varlen_preprocess<T_, D>, dim3(wave), dim3(256), 0, a.st,
                                static_cast<const T_ *>(o), static_cast<const T_ *>(o_res), static_cast<const T_ *>(dO),
                                delta, acc, a.Hq, v);
    if (s != FORGE_OK) return s;
    if (dsink != nullptr) {
        s = launch_pdl(varlen_sink_grad, dim3((unsigned)a.Hq), dim3(512), 0, a.st, lse, static_cast<const float *>(delta),
                       a.sink, dsink, a.cu, a.num_seqs, a.rows);
        if (s != FORGE_OK) return s;
    }
    if constexpr (sizeof(T_) == 4) {
        VfParams p = var_f32_params(a, v);
        p.dO = static_cast<const float *>(dO);
        p.lse = const_cast<float *>(lse);
        p.delta = delta;
        p.dq = static_cast<float *>(dq);
        p.dk = static_cast<float *>(dk);
        p.dv = static_cast<float *>(dv);
        if (set_smem(varlen_f32_bwd_dq<D>, vf_bwd_dq_smem<D>()) != FORGE_OK ||
            set_smem(varlen_f32_bwd_dkdv<D>, vf_bwd_dkdv_smem<D>()) != FORGE_OK)
            return FORGE_ERR_CUDA;
        s = launch_pdl(varlen_f32_bwd_dq<D>, dim3((unsigned)items * (unsigned)a.Hq), dim3(kVfThreads),
                       vf_bwd_dq_smem<D>(), a.st, p);
        if (s != FORGE_OK) return s;
        return launch_pdl(varlen_f32_bwd_dkdv<D>, dim3((unsigned)items * (unsigned)a.Hkv), dim3(kVfThreads),
                          vf_bwd_dkdv_smem<D>(), a.st, p);
    } else {
        using C = BwdTc<D>;
        CUtensorMap mq, mk, mv, mdo, macc;
        if (!make_map_rows(&mq, a.q, D, a.rows, a.Hq, a.q_stride, C::BM) ||
            !make_map_rows(&mk, a.k, D, a.rows, a.Hkv, a.k_stride, 128) ||
            !make_map_rows(&mv, a.v, D, a.rows, a.Hkv, a.v_stride, 128) ||
            !make_map_rows(&mdo, dO, D, a.rows, a.Hq, (size_t)a.Hq * D, C::BM) ||
            !make_map_acc(&macc, acc, D, v.pad_rows, a.Hq, C::BM)) {
            t_last_cuda_error = "cuTensorMapEncodeTiled failed";
            return FORGE_ERR_CUDA;
        }
        BwdParams p = {};
        p.lse = lse;
        p.delta = delta;
        p.dq_acc = acc;
        p.dk = static_cast<__nv_bfloat16 *>(dk);
        p.dv = static_cast<__nv_bfloat16 *>(dv);
        p.B = 1; p.Hq = a.Hq; p.Hkv = a.Hkv; p.window = a.window;
        p.scale = a.scale;
        p.scale_log2 = a.scale * kLog2e;
        p.softcap = a.softcap;
        p.cap_in = a.softcap > 0.0f ? a.scale / a.softcap : 0.0f;
        p.cap_out = a.softcap * kLog2e;
        p.var = v;
        auto *kernel = a.softcap > 0.0f || a.window > 0 ? bwd_tc_kernel<D, true, false> : bwd_tc_kernel<D, true, true>;
        if (set_smem(kernel, C::SMEM) != FORGE_OK) return FORGE_ERR_CUDA;
        const long long work = (long long)items * a.Hkv * C::NSPLIT;
        s = launch_pdl(kernel, dim3((unsigned)(work < sm_count() ? work : sm_count())), dim3(C::THREADS),
                       C::SMEM, a.st, mq, mk, mv, mdo, macc, p);
        if (s != FORGE_OK) return s;
        return launch_pdl(varlen_finalize<D>, dim3(wave), dim3(256), 0, a.st,
                          static_cast<const float *>(acc), static_cast<__nv_bfloat16 *>(dq), p.dk, p.dv, a.Hq, a.Hkv, v);
    }
}

// ---------------------------------------------------------------- paged cache
// CTAs of the split pass: one wave of what fits an SM.
template <typename T_, int D>
int pd_workers() {
    return PdCfg<T_, D>::PER_SM * sm_count();
}
int pd_workers_of(int D, forge_dtype dtype) {
    const bool bf = dtype == FORGE_DTYPE_BF16;
    switch (D) {
        case 64: return bf ? pd_workers<__nv_bfloat16, 64>() : pd_workers<float, 64>();
        case 128: return bf ? pd_workers<__nv_bfloat16, 128>() : pd_workers<float, 128>();
        default: return bf ? pd_workers<__nv_bfloat16, 256>() : pd_workers<float, 256>();
    }
}

// Workspace: [ part [2 workers][G][D] f32 ][ stat [2 workers][G] float2 ][ cut [B][Hkv] int2 ]
struct PdLayout {
    size_t stat, cut, bytes;
};
PdLayout pd_layout(int B, int Hq, int Hkv, int D, forge_dtype dtype) {
    PdLayout l;
    const size_t slots = (size_t)2 * pd_workers_of(D, dtype) * (Hq / Hkv);
    l.stat = round256(slots * D * sizeof(float));
    l.cut = l.stat + round256(slots * sizeof(float2));
    l.bytes = l.cut + round256((size_t)B * Hkv * sizeof(int2));
    return l;
}

template <typename T_, int D, class W>
forge_status pd_launch(const PdParams &p, cudaStream_t st) {
    using C = PdCfg<T_, D>;
    if (set_smem(decode_paged_split<T_, D, W>, C::SMEM) != FORGE_OK) return FORGE_ERR_CUDA;
    forge_status s = launch_pdl(decode_paged_split<T_, D, W>, dim3((unsigned)p.workers), dim3(kPdThreads), C::SMEM, st, p);
    if (s != FORGE_OK) return s;
    return launch_pdl(decode_paged_join<T_, D>, dim3((unsigned)(p.B * p.Hq)), dim3(D), 0, st, p);
}

template <int D>
forge_status pd_run(const PdParams &p, forge_dtype dtype, cudaStream_t st) {
    if (dtype == FORGE_DTYPE_BF16) return pd_launch<__nv_bfloat16, D, PdWarpBf<D>>(p, st);
    const int G = p.Hq / p.Hkv;
    if (G <= 4) return pd_launch<float, D, PdWarpF32<D, 4>>(p, st);
    if (G <= 8) return pd_launch<float, D, PdWarpF32<D, 8>>(p, st);
    return pd_launch<float, D, PdWarpF32<D, 16>>(p, st);
}

// A pool of pages: [num_pages][Hkv][page_size][D], pages page_stride elements apart.
forge_status check_pool(const void *k, const void *v, int Hkv, int D, int num_pages, int page_size, size_t page_stride,
                        forge_dtype dtype) {
    if (Hkv < 1 || D < 1 || num_pages < 1 || page_size < 1) return FORGE_ERR_INVALID_ARG;
    if (dtype != FORGE_DTYPE_F32 && dtype != FORGE_DTYPE_BF16) return FORGE_ERR_INVALID_ARG;
    if (D != 64 && D != 128 && D != 256) return D % 2 ? FORGE_ERR_INVALID_ARG : FORGE_ERR_UNSUPPORTED;
    if (page_size % 16 != 0) return FORGE_ERR_UNSUPPORTED;
    if (Hkv > (1 << 16) || page_size > (1 << 20)) return FORGE_ERR_INVALID_ARG;
    const size_t es = dtype == FORGE_DTYPE_BF16 ? 2 : 4;
    if (page_stride < (size_t)Hkv * page_size * D || page_stride * es % 16 != 0 ||
        page_stride > ((size_t)1 << 44) / (size_t)num_pages)
        return FORGE_ERR_INVALID_ARG;
    if (!aligned16(k) || !aligned16(v)) return FORGE_ERR_INVALID_ARG;
    return FORGE_OK;
}

// A set of page numbers on the stack, for the pairs of one copy launch.
struct PageSet {
    static constexpr int N = 2048;  // slots; at most kCopyPairs used
    int slot[N];
    void clear() { memset(slot, 0xff, sizeof(slot)); }
    int find(int page) const {
        int i = (int)((unsigned)page * 2654435761u % N);
        while (slot[i] >= 0 && slot[i] != page) i = (i + 1) % N;
        return i;
    }
    bool has(int page) const { return slot[find(page)] == page; }
    void add(int page) { slot[find(page)] = page; }
};

// out[i] = value for i < n
__global__ void fill_f32_kernel(float *out, long n, float value) {
    const long i = (long)blockIdx.x * blockDim.x + threadIdx.x;
    if (i < n) out[i] = value;
}

// dsink[hq] = -sum over b, t of exp(sink[hq] - lse[b][hq][t]) * delta[b][hq][t]:
// the gradient of a per-head sink logit (its softmax column times (0 - Delta),
// the sink having no value vector). One block per query head, deterministic.
__global__ void __launch_bounds__(256) sink_grad_kernel(const float *lse, const float *delta, const float *sink,
                                                        float *dsink, int B, int Hq, int T) {
    __shared__ float part[8];
    const int hq = blockIdx.x;
    const float sg = sink[hq];
    float acc = 0.0f;
    for (long idx = threadIdx.x; idx < (long)B * T; idx += blockDim.x) {
        const long b = idx / T, t = idx % T;
        const size_t row = ((size_t)b * Hq + hq) * T + t;
        acc -= expf(sg - lse[row]) * delta[row];
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = acc;
    __syncthreads();
    if (threadIdx.x == 0) {
        float sum = 0.0f;
        for (int w = 0; w < 8; w++) sum += part[w];
        dsink[hq] = sum;
    }
}

// Keys per decode chunk, multiples of 64: enough chunks for about 16 CTAs per SM.
// The warp-pipelined split kernel keeps six CTAs resident per SM at head dim 128,
// so this gives several waves with a short tail (measured on B 16, Hkv 8, 16K
// keys: 5.40 TB/s at 16 per SM, 5.36 at 24, 5.32 at 32, 5.03 at 8).
constexpr long kDecCtasPerSm = 16;
int decode_chunk(int B, int Hkv, int T) {
    const long per = (long)B * Hkv;
    const long splits = (kDecCtasPerSm * 148 + per - 1) / per;
    long chunk = ((T + splits - 1) / splits + 63) / 64 * 64;
    return (int)(chunk < 64 ? 64 : chunk);
}

template <typename T_, int D, int MG>
forge_status decode_split_launch(const void *q, const void *kc, const void *vc, const DecParams &p, cudaStream_t st) {
    using C = DecCfg<T_, D>;
    if (set_smem(decode_split<T_, D, MG>, C::smem(MG)) != FORGE_OK) return FORGE_ERR_CUDA;
    decode_split<T_, D, MG><<<pair_grid((unsigned)p.nsplit, (long long)p.B * p.Hkv), kDecThreads,
                              C::smem(p.Hq / p.Hkv), st>>>(static_cast<const T_ *>(q), static_cast<const T_ *>(kc),
                                                           static_cast<const T_ *>(vc), p);
    return launch_status();
}

// The warp-pipelined kernel serves groups whose queries and outputs fit a lane's
// registers (MG * D <= 1024) with steps of at most 8 KB of K rows; decode_split
// the others.
template <typename T_, int D, int MG>
constexpr bool decode_warp_fits() {
    return MG * D <= 1024 && (32 / MG) * D * (int)sizeof(T_) <= 8192;
}

template <typename T_, int D, int MG>
forge_status decode_pick(const void *q, const void *kc, const void *vc, const DecParams &p, cudaStream_t st) {
    if constexpr (decode_warp_fits<T_, D, MG>()) {
        using C = DecWCfg<T_, D, MG>;
        if (set_smem(decode_split_warp<T_, D, MG>, C::SMEM) != FORGE_OK) return FORGE_ERR_CUDA;
        decode_split_warp<T_, D, MG><<<pair_grid((unsigned)p.nsplit, (long long)p.B * p.Hkv), kDecWarps * 32, C::SMEM,
                                       st>>>(static_cast<const T_ *>(q), static_cast<const T_ *>(kc),
                                             static_cast<const T_ *>(vc), p);
        return launch_status();
    } else {
        return decode_split_launch<T_, D, (MG < 4 ? 4 : MG)>(q, kc, vc, p, st);
    }
}

template <typename T_, int D>
forge_status decode_run(const void *q, const void *kc, const void *vc, void *o, DecParams p, cudaStream_t st) {
    const int G = p.Hq / p.Hkv;
    forge_status s = G <= 1   ? decode_pick<T_, D, 1>(q, kc, vc, p, st)
                     : G <= 2 ? decode_pick<T_, D, 2>(q, kc, vc, p, st)
                     : G <= 4 ? decode_pick<T_, D, 4>(q, kc, vc, p, st)
                     : G <= 8 ? decode_pick<T_, D, 8>(q, kc, vc, p, st)
                              : decode_pick<T_, D, 16>(q, kc, vc, p, st);
    if (s != FORGE_OK) return s;
    decode_combine<T_, D><<<(unsigned)(p.B * p.Hq), D, 0, st>>>(static_cast<T_ *>(o), p);
    return launch_status();
}

#define FORGE_DISPATCH_D(D, ...)                               \
    switch (D) {                                               \
        case 64: { constexpr int kD = 64; __VA_ARGS__ } break;   \
        case 128: { constexpr int kD = 128; __VA_ARGS__ } break; \
        case 256: { constexpr int kD = 256; __VA_ARGS__ } break; \
        default: return FORGE_ERR_UNSUPPORTED;                 \
    }

}  // namespace

// Timeout self-test: waits on a barrier nothing completes.
__global__ void selftest_timeout_kernel(unsigned long long limit_ns) {
    __shared__ __align__(8) uint64_t barrier;
    __shared__ int abort_flag;
    if (threadIdx.x == 0) {
        abort_flag = 0;
        mbar_init(smem_u32(&barrier), 1);
        fence_mbar_init();
    }
    __syncthreads();
    if (threadIdx.x == 0) mbar_wait(smem_u32(&barrier), 0, &abort_flag, limit_ns);
    __syncthreads();
}

// exp2 self-test: the kernels' FMA-pipe exp2 next to CUDA's exp2f.
__global__ void selftest_exp2_kernel(const float *x, float *y, float *y_ref, int n) {
    const int i = blockIdx.x * blockDim.x + threadIdx.x;
    if (i < n) {
        y[i] = exp2_poly(x[i]);
        y_ref[i] = exp2f(x[i]);
    }
}

}  // namespace forge

// ---------------------------------------------------------------------------
// Backward without caller-provided workspace.
//
// Some callers cannot allocate device memory at all: a host program that only
// receives device buffers from another runtime and has no allocator of its own
// (plain C or a foreign-language binding), or a process whose memory pool owns
// the whole device and forbids allocations outside it. forge_attn_bwd_noalloc
// serves them with scratch that lives in this fixed-size device array instead
// of a caller workspace. Every GPU that loads the library holds the array until
// the process exits. Its device address belongs to the device's current
// context: it is looked up on the first call made with that device current and
// cached together with the context's unique id, and looked up again when the
// id has changed (a cudaDeviceReset ends the old context, and the module and
// its array get a new address in the next one).
namespace {
constexpr size_t kNoAllocScratchBytes = size_t(32) << 20;  // 32 MiB
static __device__ __align__(256) unsigned char g_noalloc_scratch[kNoAllocScratchBytes];
constexpr int kNoAllocMaxDevices = 64;
std::mutex g_noalloc_mutex;
struct NoAllocEntry {
    unsigned long long ctx_id;  // id of the context the address belongs to
    void *ptr;
};
NoAllocEntry g_noalloc[kNoAllocMaxDevices] = {};

typedef CUresult (*CtxGetCurrentFn)(CUcontext *);
typedef CUresult (*CtxGetIdFn)(CUcontext, unsigned long long *);

template <typename F>
F driver_fn(const char *name) {
    void *ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint(name, &ptr, cudaEnableDefault, &q) == cudaSuccess && q == cudaDriverEntryPointSuccess)
        return reinterpret_cast<F>(ptr);
    return nullptr;
}

// Unique id of the calling thread's current context (never reused within the
// process), or 0 when there is none or the driver cannot say.
unsigned long long current_context_id() {
    static CtxGetCurrentFn get_current = driver_fn<CtxGetCurrentFn>("cuCtxGetCurrent");
    static CtxGetIdFn get_id = driver_fn<CtxGetIdFn>("cuCtxGetId");
    if (get_current == nullptr || get_id == nullptr) return 0;
    CUcontext ctx = nullptr;
    unsigned long long id = 0;
    if (get_current(&ctx) != CUDA_SUCCESS || ctx == nullptr) return 0;
    if (get_id(ctx, &id) != CUDA_SUCCESS) return 0;
    return id;
}

forge_status noalloc_scratch_for_current_device(void **out) {
    int dev = -1;
    forge_status s = forge::cuda_status(cudaGetDevice(&dev));
    if (s != FORGE_OK) return s;
    if (dev < 0 || dev >= kNoAllocMaxDevices) return FORGE_ERR_UNSUPPORTED;
    std::lock_guard<std::mutex> lock(g_noalloc_mutex);
    NoAllocEntry &e = g_noalloc[dev];
    const unsigned long long id = current_context_id();
    if (e.ptr == nullptr || id == 0 || id != e.ctx_id) {
        // first call on this device, a context without a readable id (looked up
        // every time then), or a new context since the last lookup
        void *p = nullptr;
        s = forge::cuda_status(cudaGetSymbolAddress(&p, g_noalloc_scratch));
        if (s != FORGE_OK) return s;
        e.ptr = p;
        e.ctx_id = current_context_id();  // the lookup may have created the context
    }
    *out = e.ptr;
    return FORGE_OK;
}
}  // namespace

using namespace forge;

extern "C" {

forge_status forge_attn_fwd_ext(const void *q, const void *k, const void *v, void *o, float *lse, int B, int Hq,
                                int Hkv, int T, int D, float scale, int window, float softcap, const float *sink,
                                float *max_logit, forge_dtype dtype, void *stream) {
    forge_status s = check_sizes(B, Hq, Hkv, T, D, dtype);
    if (s != FORGE_OK) return s;
    if ((s = check_scalars(scale, window, softcap)) != FORGE_OK) return s;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(lse))
        return FORGE_ERR_INVALID_ARG;
    if ((sink != nullptr && !aligned4(sink)) || (max_logit != nullptr && !aligned4(max_logit)))
        return FORGE_ERR_INVALID_ARG;
    window = effective_window(window, T);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (max_logit != nullptr) {
        const long n = (long)B * Hq;
        fill_f32_kernel<<<(unsigned)((n + 255) / 256), 256, 0, st>>>(max_logit, n, -INFINITY);
        if ((s = launch_status()) != FORGE_OK) return s;
    }
    if (dtype == FORGE_DTYPE_BF16) {
        FORGE_DISPATCH_D(D, return fwd_tc<kD>(q, k, v, o, lse, B, Hq, Hkv, T, scale, window, softcap, sink,
                                               max_logit, st);)
    } else {
        FORGE_DISPATCH_D(D, return fwd_simt<float, kD>(q, k, v, o, lse, B, Hq, Hkv, T, scale, window, softcap, sink,
                                                        max_logit, st);)
    }
    return FORGE_ERR_UNSUPPORTED;
}

forge_status forge_attn_fwd(const void *q, const void *k, const void *v, void *o, float *lse, int B, int Hq,
                            int Hkv, int T, int D, float scale, int window, float softcap, forge_dtype dtype,
                            void *stream) {
    return forge_attn_fwd_ext(q, k, v, o, lse, B, Hq, Hkv, T, D, scale, window, softcap, nullptr, nullptr, dtype,
                              stream);
}

size_t forge_attn_bwd_workspace_size(int B, int Hq, int Hkv, int T, int D, forge_dtype dtype) {
    if (check_sizes(B, Hq, Hkv, T, D, dtype) != FORGE_OK) return 0;
    size_t n = delta_bytes(B, Hq, T);
    if (dtype == FORGE_DTYPE_BF16) n += acc_bytes(B, Hq, T, D);
    return n;
}

static forge_status check_workspace(void *ws, size_t bytes, int B, int Hq, int Hkv, int T, int D, forge_dtype dtype) {
    if (ws == nullptr || (reinterpret_cast<uintptr_t>(ws) & 255u) != 0) return FORGE_ERR_WORKSPACE;
    if (bytes < forge_attn_bwd_workspace_size(B, Hq, Hkv, T, D, dtype)) return FORGE_ERR_WORKSPACE;
    return FORGE_OK;
}

forge_status forge_attn_bwd_preprocess(const void *o, const void *dO, int B, int Hq, int Hkv, int T, int D,
                                       forge_dtype dtype, void *workspace, size_t workspace_bytes, void *stream) {
    forge_status s = check_sizes(B, Hq, Hkv, T, D, dtype);
    if (s != FORGE_OK) return s;
    if (!aligned16(o) || !aligned16(dO)) return FORGE_ERR_INVALID_ARG;
    if ((s = check_workspace(workspace, workspace_bytes, B, Hq, Hkv, T, D, dtype)) != FORGE_OK) return s;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    float *delta = static_cast<float *>(workspace);
    const long rows = (long)B * Hq * T;
    const unsigned grid = preprocess_grid(rows, D);
    if (dtype == FORGE_DTYPE_BF16) {
        // the dq accumulator receives reductions: zero it in the same pass
        float *acc = reinterpret_cast<float *>(static_cast<char *>(workspace) + delta_bytes(B, Hq, T));
        FORGE_DISPATCH_D(D, return launch_pdl(bwd_preprocess<__nv_bfloat16, kD>, dim3(grid), dim3(256), 0, st,
                                              static_cast<const __nv_bfloat16 *>(o),
                                              static_cast<const __nv_bfloat16 *>(dO), delta, acc, rows, T,
                                              tpad_of(T));)
    }
    FORGE_DISPATCH_D(D, return launch_pdl(bwd_preprocess<float, kD>, dim3(grid), dim3(256), 0, st,
                                          static_cast<const float *>(o), static_cast<const float *>(dO), delta,
                                          static_cast<float *>(nullptr), rows, T, tpad_of(T));)
    return FORGE_ERR_UNSUPPORTED;
}

forge_status forge_attn_bwd_main(const void *q, const void *k, const void *v, const float *lse, const void *dO,
                                 void *dq, void *dk, void *dv, int B, int Hq, int Hkv, int T, int D, float scale,
                                 int window, float softcap, forge_dtype dtype, void *workspace,
                                 size_t workspace_bytes, void *stream) {
    forge_status s = check_sizes(B, Hq, Hkv, T, D, dtype);
    if (s != FORGE_OK) return s;
    if ((s = check_scalars(scale, window, softcap)) != FORGE_OK) return s;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(lse) || !aligned16(dO) || !aligned16(dq) ||
        !aligned16(dk) || !aligned16(dv))
        return FORGE_ERR_INVALID_ARG;
    if ((s = check_workspace(workspace, workspace_bytes, B, Hq, Hkv, T, D, dtype)) != FORGE_OK) return s;
    window = effective_window(window, T);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const float *delta = static_cast<const float *>(workspace);
    if (dtype == FORGE_DTYPE_BF16) {
        float *acc = reinterpret_cast<float *>(static_cast<char *>(workspace) + delta_bytes(B, Hq, T));
        FORGE_DISPATCH_D(D, return bwd_tc<kD>(q, k, v, lse, dO, delta, acc, dk, dv, B, Hq, Hkv, T, scale, window,
                                              softcap, st);)
    }
    FORGE_DISPATCH_D(D, return bwd_simt<float, kD>(q, k, v, lse, dO, delta, dq, dk, dv, B, Hq, Hkv, T, scale, window,
                                                   softcap, st);)
    return FORGE_ERR_UNSUPPORTED;
}

forge_status forge_attn_bwd_finalize(void *dq, int B, int Hq, int Hkv, int T, int D, forge_dtype dtype,
                                     void *workspace, size_t workspace_bytes, void *stream) {
    forge_status s = check_sizes(B, Hq, Hkv, T, D, dtype);
    if (s != FORGE_OK) return s;
    if (!aligned16(dq)) return FORGE_ERR_INVALID_ARG;
    if ((s = check_workspace(workspace, workspace_bytes, B, Hq, Hkv, T, D, dtype)) != FORGE_OK) return s;
    if (dtype != FORGE_DTYPE_BF16) return FORGE_OK;  // f32: dq already written by the main stage
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const float *acc = reinterpret_cast<const float *>(static_cast<char *>(workspace) + delta_bytes(B, Hq, T));
    const long long total = (long long)B * Hq * T * (D / 8);
    const unsigned grid = (unsigned)((total + 255) / 256);
    FORGE_DISPATCH_D(D, return launch_pdl(bwd_finalize_dq<kD>, dim3(grid), dim3(256), 0, st, acc,
                                          static_cast<__nv_bfloat16 *>(dq), (long)B * Hq, T, tpad_of(T));)
    return FORGE_ERR_UNSUPPORTED;
}

forge_status forge_attn_bwd_ext(const void *q, const void *k, const void *v, const void *o, const float *lse,
                                const void *dO, void *dq, void *dk, void *dv, int B, int Hq, int Hkv, int T, int D,
                                float scale, int window, float softcap, const float *sink, float *dsink,
                                forge_dtype dtype, void *workspace, size_t workspace_bytes, void *stream) {
    forge_status s = check_sizes(B, Hq, Hkv, T, D, dtype);
    if (s != FORGE_OK) return s;
    if ((s = check_scalars(scale, window, softcap)) != FORGE_OK) return s;
    // validate everything before the first launch: on error nothing runs
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(lse) || !aligned16(dO) ||
        !aligned16(dq) || !aligned16(dk) || !aligned16(dv))
        return FORGE_ERR_INVALID_ARG;
    if (dsink != nullptr && (!aligned4(dsink) || !aligned4(sink))) return FORGE_ERR_INVALID_ARG;
    if (sink != nullptr && !aligned4(sink)) return FORGE_ERR_INVALID_ARG;
    if ((s = check_workspace(workspace, workspace_bytes, B, Hq, Hkv, T, D, dtype)) != FORGE_OK) return s;
    s = forge_attn_bwd_preprocess(o, dO, B, Hq, Hkv, T, D, dtype, workspace, workspace_bytes, stream);
    if (s != FORGE_OK) return s;
    if (dsink != nullptr) {
        // the sink enters dq, dk, dv only through lse; its own gradient needs Delta
        sink_grad_kernel<<<(unsigned)Hq, 256, 0, static_cast<cudaStream_t>(stream)>>>(
            lse, static_cast<const float *>(workspace), sink, dsink, B, Hq, T);
        if ((s = launch_status()) != FORGE_OK) return s;
    }
    s = forge_attn_bwd_main(q, k, v, lse, dO, dq, dk, dv, B, Hq, Hkv, T, D, scale, window, softcap, dtype, workspace,
                            workspace_bytes, stream);
    if (s != FORGE_OK) return s;
    return forge_attn_bwd_finalize(dq, B, Hq, Hkv, T, D, dtype, workspace, workspace_bytes, stream);
}

forge_status forge_attn_bwd(const void *q, const void *k, const void *v, const void *o, const float *lse,
                            const void *dO, void *dq, void *dk, void *dv, int B, int Hq, int Hkv, int T, int D,
                            float scale, int window, float softcap, forge_dtype dtype, void *workspace,
                            size_t workspace_bytes, void *stream) {
    return forge_attn_bwd_ext(q, k, v, o, lse, dO, dq, dk, dv, B, Hq, Hkv, T, D, scale, window, softcap, nullptr,
                              nullptr, dtype, workspace, workspace_bytes, stream);
}

forge_status forge_attn_bwd_noalloc(const void *q, const void *k, const void *v, const void *o, const float *lse,
                                    const void *dO, void *dq, void *dk, void *dv, int B, int Hq, int Hkv, int T, int D,
                                    float scale, int window, float softcap, forge_dtype dtype, void *stream) {
    forge_status s = check_sizes(B, Hq, Hkv, T, D, dtype);
    if (s != FORGE_OK) return s;
    if (forge_attn_bwd_workspace_size(B, Hq, Hkv, T, D, dtype) > kNoAllocScratchBytes) {
        t_last_cuda_error = "problem too large for forge_attn_bwd_noalloc's 32 MiB scratch";
        return FORGE_ERR_WORKSPACE;
    }
    void *scratch = nullptr;
    if ((s = noalloc_scratch_for_current_device(&scratch)) != FORGE_OK) return s;
    // the preprocess stage zeroes the dq accumulator rows and overwrites Delta,
    // so whatever the previous call left in the array does not matter
    return forge_attn_bwd(q, k, v, o, lse, dO, dq, dk, dv, B, Hq, Hkv, T, D, scale, window, softcap, dtype, scratch,
                          kNoAllocScratchBytes, stream);
}

// d_k != d_v at (d_k, d_v) = (192, 128), the decompressed multi-head latent
// attention of the DeepSeek V3 family: on the tensor cores (bf16) or the CUDA
// cores (f32), forward and backward.
static bool dkv_supported(int Dk, int Dv, forge_dtype dtype) {
    return (dtype == FORGE_DTYPE_F32 || dtype == FORGE_DTYPE_BF16) && Dk == 192 && Dv == 128;
}
static bool dkv_fwd_supported(int Dk, int Dv, forge_dtype dtype) { return dkv_supported(Dk, Dv, dtype); }

size_t forge_attn_bwd_workspace_size_dkv(int B, int Hq, int Hkv, int T, int Dk, int Dv, forge_dtype dtype) {
    if (Dk == Dv) return forge_attn_bwd_workspace_size(B, Hq, Hkv, T, Dk, dtype);
    if (!dkv_supported(Dk, Dv, dtype) || check_sizes(B, Hq, Hkv, T, Dv, dtype) != FORGE_OK) return 0;
    return delta_bytes(B, Hq, T);  // Delta only: both paths write dq directly
}

forge_status forge_attn_fwd_dkv(const void *q, const void *k, const void *v, void *o, float *lse, int B, int Hq,
                                int Hkv, int T, int Dk, int Dv, float scale, int window, float softcap,
                                forge_dtype dtype, void *stream) {
    if (Dk == Dv) return forge_attn_fwd(q, k, v, o, lse, B, Hq, Hkv, T, Dk, scale, window, softcap, dtype, stream);
    forge_status s = check_sizes(B, Hq, Hkv, T, Dv, dtype);
    if (s != FORGE_OK) return s;
    if (!dkv_fwd_supported(Dk, Dv, dtype)) return FORGE_ERR_UNSUPPORTED;
    if ((s = check_scalars(scale, window, softcap)) != FORGE_OK) return s;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(lse))
        return FORGE_ERR_INVALID_ARG;
    window = effective_window(window, T);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (dtype == FORGE_DTYPE_BF16) return fwd_tc_dkv<192, 128>(q, k, v, o, lse, B, Hq, Hkv, T, scale, window, softcap, st);
    return fwd_simt<float, 192, 128>(q, k, v, o, lse, B, Hq, Hkv, T, scale, window, softcap, nullptr, nullptr, st);
}

forge_status forge_attn_bwd_dkv(const void *q, const void *k, const void *v, const void *o, const float *lse,
                                const void *dO, void *dq, void *dk, void *dv, int B, int Hq, int Hkv, int T, int Dk,
                                int Dv, float scale, int window, float softcap, forge_dtype dtype, void *workspace,
                                size_t workspace_bytes, void *stream) {
    if (Dk == Dv)
        return forge_attn_bwd(q, k, v, o, lse, dO, dq, dk, dv, B, Hq, Hkv, T, Dk, scale, window, softcap, dtype,
                              workspace, workspace_bytes, stream);
    forge_status s = check_sizes(B, Hq, Hkv, T, Dv, dtype);
    if (s != FORGE_OK) return s;
    if (!dkv_supported(Dk, Dv, dtype)) return FORGE_ERR_UNSUPPORTED;
    if ((s = check_scalars(scale, window, softcap)) != FORGE_OK) return s;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(lse) || !aligned16(dO) ||
        !aligned16(dq) || !aligned16(dk) || !aligned16(dv))
        return FORGE_ERR_INVALID_ARG;
    if (workspace == nullptr || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0 ||
        workspace_bytes < forge_attn_bwd_workspace_size_dkv(B, Hq, Hkv, T, Dk, Dv, dtype))
        return FORGE_ERR_WORKSPACE;
    window = effective_window(window, T);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    float *delta = static_cast<float *>(workspace);
    const long rows = (long)B * Hq * T;
    if (dtype == FORGE_DTYPE_BF16) {
        bwd_preprocess<__nv_bfloat16, 128><<<preprocess_grid(rows, 128), 256, 0, st>>>(
            static_cast<const __nv_bfloat16 *>(o), static_cast<const __nv_bfloat16 *>(dO), delta, nullptr, rows, T,
            tpad_of(T));
        if ((s = launch_status()) != FORGE_OK) return s;
        return bwd_tc_dkv<192, 128>(q, k, v, lse, dO, delta, dq, dk, dv, B, Hq, Hkv, T, scale, window, softcap, st);
    }
    bwd_preprocess<float, 128><<<preprocess_grid(rows, 128), 256, 0, st>>>(
        static_cast<const float *>(o), static_cast<const float *>(dO), delta, nullptr, rows, T, tpad_of(T));
    if ((s = launch_status()) != FORGE_OK) return s;
    return bwd_simt<float, 192, 128>(q, k, v, lse, dO, delta, dq, dk, dv, B, Hq, Hkv, T, scale, window, softcap, st);
}

size_t forge_attn_decode_workspace_size(int B, int Hq, int Hkv, int T, int D) {
    if (check_sizes(B, Hq, Hkv, T, D, FORGE_DTYPE_BF16) != FORGE_OK) return 0;
    const int chunk = decode_chunk(B, Hkv, T);
    const long nsplit = (T + chunk - 1) / chunk;
    return ((size_t)B * Hq * nsplit * (size_t)(D + 2) * sizeof(float) + 255) / 256 * 256;
}

forge_status forge_attn_decode(const void *q, const void *k_cache, const void *v_cache, void *o, float *lse,
                               const int *seq_lens, int B, int Hq, int Hkv, int T, int Tmax, int D, float scale,
                               int window, float softcap, const float *sink, forge_dtype dtype, void *workspace,
                               size_t workspace_bytes, void *stream) {
    forge_status s = check_sizes(B, Hq, Hkv, T, D, dtype);
    if (s != FORGE_OK) return s;
    if ((s = check_scalars(scale, window, softcap)) != FORGE_OK) return s;
    if (Tmax < T || (long)Tmax * D * B * Hkv > (1L << 40)) return FORGE_ERR_INVALID_ARG;
    if (Hq / Hkv > kDecMaxG) return FORGE_ERR_UNSUPPORTED;
    if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(o)) return FORGE_ERR_INVALID_ARG;
    if ((lse && !aligned4(lse)) || (seq_lens && !aligned4(seq_lens)) || (sink && !aligned4(sink)))
        return FORGE_ERR_INVALID_ARG;
    const size_t need = forge_attn_decode_workspace_size(B, Hq, Hkv, T, D);
    if (!aligned16(workspace) || workspace_bytes < need) return FORGE_ERR_WORKSPACE;
    DecParams p;
    p.seq_lens = seq_lens;
    p.sink = sink;
    p.part = static_cast<float *>(workspace);
    p.lse = lse;
    p.B = B; p.Hq = Hq; p.Hkv = Hkv; p.T = T; p.Tmax = Tmax;
    p.window = effective_window(window, T);
    p.chunk = decode_chunk(B, Hkv, T);
    p.nsplit = (T + p.chunk - 1) / p.chunk;
    p.qscale = softcap > 0.0f ? scale / softcap : scale * kLog2e;
    p.cap_out = softcap > 0.0f ? softcap * kLog2e : 0.0f;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (dtype == FORGE_DTYPE_BF16) {
        FORGE_DISPATCH_D(D, return decode_run<__nv_bfloat16, kD>(q, k_cache, v_cache, o, p, st);)
    } else {
        FORGE_DISPATCH_D(D, return decode_run<float, kD>(q, k_cache, v_cache, o, p, st);)
    }
    return FORGE_ERR_UNSUPPORTED;
}

size_t forge_attn_varlen_fwd_workspace_size(int num_seqs, int rows, int Hq, int Hkv, int D, forge_dtype dtype) {
    if (check_var_sizes(num_seqs, rows, Hq, Hkv, D, dtype) != FORGE_OK) return 0;
    return var_layout(num_seqs, rows, Hq, Hkv, D, dtype, false).bytes;
}

size_t forge_attn_varlen_bwd_workspace_size(int num_seqs, int rows, int Hq, int Hkv, int D, forge_dtype dtype) {
    if (check_var_sizes(num_seqs, rows, Hq, Hkv, D, dtype) != FORGE_OK) return 0;
    return var_layout(num_seqs, rows, Hq, Hkv, D, dtype, true).bytes;
}

forge_status forge_attn_varlen_fwd(const void *q, const void *k, const void *v, void *o, void *o_res, float *lse,
                                   const int *cu_seqlens, int num_seqs, int rows, int Hq, int Hkv, int D,
                                   size_t q_stride, size_t k_stride, size_t v_stride, float scale, int window,
                                   float softcap, const float *sink, int flags, forge_dtype dtype,
                                   void *workspace, size_t workspace_bytes, void *stream) {
    VarArgs a = {q, k, v, cu_seqlens, num_seqs, rows, Hq, Hkv, D, q_stride, k_stride, v_stride, scale, window, softcap,
                 sink, dtype, static_cast<cudaStream_t>(stream)};
    forge_status s = check_var_args(a);
    if (s != FORGE_OK) return s;
    if (!aligned16(o) || !aligned16(lse) || (o_res != nullptr && !aligned32(o_res))) return FORGE_ERR_INVALID_ARG;
    if (workspace == nullptr || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0 ||
        workspace_bytes < forge_attn_varlen_fwd_workspace_size(num_seqs, rows, Hq, Hkv, D, dtype))
        return FORGE_ERR_WORKSPACE;
    a.window = effective_window(window, rows);
    const VarSched sched = var_sched(a, var_layout(num_seqs, rows, Hq, Hkv, D, dtype, false), workspace, false);
    void *const tail[3] = {o, nullptr, nullptr};
    const int heads[3] = {Hq, 0, 0};
    if ((s = run_plan(a, sched, false, tail, heads, lse, clears_tail(flags))) != FORGE_OK) return s;
    if (dtype == FORGE_DTYPE_BF16) {
        FORGE_DISPATCH_D(D, return var_fwd_tc<kD>(a, sched, o, o_res, lse, sink_is_fixed(flags));)
    } else {
        FORGE_DISPATCH_D(D, return var_fwd_f32<kD>(a, sched, o, lse);)
    }
    return FORGE_ERR_UNSUPPORTED;
}

forge_status forge_attn_varlen_bwd(const void *q, const void *k, const void *v, const void *o, const void *o_res,
                                   const float *lse, const void *dO, void *dq, void *dk, void *dv, const int *cu_seqlens, int num_seqs,
                                   int rows, int Hq, int Hkv, int D, size_t q_stride, size_t k_stride, size_t v_stride,
                                   float scale, int window, float softcap, const float *sink, float *dsink,
                                   int flags, forge_dtype dtype, void *workspace, size_t workspace_bytes,
                                   void *stream) {
    VarArgs a = {q, k, v, cu_seqlens, num_seqs, rows, Hq, Hkv, D, q_stride, k_stride, v_stride, scale, window, softcap,
                 sink, dtype, static_cast<cudaStream_t>(stream)};
    forge_status s = check_var_args(a);
    if (s != FORGE_OK) return s;
    if (!aligned16(o) || !aligned16(lse) || !aligned16(dO) || !aligned16(dq) || !aligned16(dk) || !aligned16(dv))
        return FORGE_ERR_INVALID_ARG;
    if (o_res != nullptr && !aligned32(o_res)) return FORGE_ERR_INVALID_ARG;
    if (dsink != nullptr && (!aligned4(dsink) || !aligned4(sink))) return FORGE_ERR_INVALID_ARG;
    if (dtype == FORGE_DTYPE_F32) o_res = nullptr;  // an f32 o has no residual
    if (workspace == nullptr || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0 ||
        workspace_bytes < forge_attn_varlen_bwd_workspace_size(num_seqs, rows, Hq, Hkv, D, dtype))
        return FORGE_ERR_WORKSPACE;
    a.window = effective_window(window, rows);
    const VarLayout l = var_layout(num_seqs, rows, Hq, Hkv, D, dtype, true);
    const VarSched sched = var_sched(a, l, workspace, true);
    float *delta = reinterpret_cast<float *>(static_cast<char *>(workspace) + l.delta);
    float *acc = dtype == FORGE_DTYPE_BF16 ? reinterpret_cast<float *>(static_cast<char *>(workspace) + l.acc) : nullptr;
    void *const tail[3] = {dq, dk, dv};
    const int heads[3] = {Hq, Hkv, Hkv};
    if ((s = run_plan(a, sched, true, tail, heads, nullptr, clears_tail(flags))) != FORGE_OK) return s;
    if (dtype == FORGE_DTYPE_BF16) {
        FORGE_DISPATCH_D(D, return var_bwd<__nv_bfloat16, kD>(a, sched, o, o_res, lse, dO, dq, dk, dv, dsink, delta, acc);)
    } else {
        FORGE_DISPATCH_D(D, return var_bwd<float, kD>(a, sched, o, o_res, lse, dO, dq, dk, dv, dsink, delta, acc);)
    }
    return FORGE_ERR_UNSUPPORTED;
}

size_t forge_attn_decode_paged_workspace_size(int B, int Hq, int Hkv, int D, forge_dtype dtype) {
    if (check_sizes(B, Hq, Hkv, 1, D, dtype) != FORGE_OK || Hq / Hkv > kPdMaxG) return 0;
    return pd_layout(B, Hq, Hkv, D, dtype).bytes;
}

forge_status forge_attn_decode_paged(const void *q, const void *k_pages, const void *v_pages, void *o, float *lse,
                                     const int *page_table, const int *seq_lens, int B, int Hq, int Hkv, int D,
                                     int num_pages, int page_size, int table_width, size_t page_stride, float scale,
                                     int window, float softcap, const float *sink, forge_dtype dtype, void *workspace,
                                     size_t workspace_bytes, void *stream) {
    forge_status s = check_sizes(B, Hq, Hkv, 1, D, dtype);
    if (s != FORGE_OK) return s;
    if ((s = check_scalars(scale, window, softcap)) != FORGE_OK) return s;
    if ((s = check_pool(k_pages, v_pages, Hkv, D, num_pages, page_size, page_stride, dtype)) != FORGE_OK) return s;
    if (Hq / Hkv > kPdMaxG) return FORGE_ERR_UNSUPPORTED;
    if (table_width < 1 || (long long)table_width * page_size > (1 << 30)) return FORGE_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(o) || !aligned4(page_table) || !aligned4(seq_lens) || (lse && !aligned4(lse)) ||
        (sink && !aligned4(sink)))
        return FORGE_ERR_INVALID_ARG;
    if (workspace == nullptr || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0 ||
        workspace_bytes < forge_attn_decode_paged_workspace_size(B, Hq, Hkv, D, dtype))
        return FORGE_ERR_WORKSPACE;
    PdParams p;
    p.q = q;
    p.k = k_pages;
    p.v = v_pages;
    p.o = o;
    p.lse = lse;
    p.table = page_table;
    p.seq_lens = seq_lens;
    p.sink = sink;
    const PdLayout l = pd_layout(B, Hq, Hkv, D, dtype);
    p.part = static_cast<float *>(workspace);
    p.stat = reinterpret_cast<float2 *>(static_cast<char *>(workspace) + l.stat);
    p.cut = reinterpret_cast<int2 *>(static_cast<char *>(workspace) + l.cut);
    p.page_stride = (long long)page_stride;
    p.B = B; p.Hq = Hq; p.Hkv = Hkv; p.width = table_width; p.page = page_size; p.num_pages = num_pages;
    p.window = effective_window(window, table_width * page_size);
    p.qscale = softcap > 0.0f ? scale / softcap : scale * kLog2e;
    p.cap_out = softcap > 0.0f ? softcap * kLog2e : 0.0f;
    // no more CTAs than units of 32 keys that the tables could hold
    const long long most = (long long)B * Hkv * ((long long)table_width * page_size / 32 + 1);
    const int workers = pd_workers_of(D, dtype);
    p.workers = most < workers ? (int)most : workers;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    FORGE_DISPATCH_D(D, return pd_run<kD>(p, dtype, st);)
    return FORGE_ERR_UNSUPPORTED;
}

forge_status forge_attn_paged_append(const void *k, const void *v, void *k_pages, void *v_pages, const int *page_table,
                                     const int *starts, const int *cu_seqlens, int num_seqs, int rows, int Hkv, int D,
                                     int num_pages, int page_size, int table_width, size_t k_stride, size_t v_stride,
                                     size_t page_stride, forge_dtype dtype, void *stream) {
    forge_status s = check_pool(k_pages, v_pages, Hkv, D, num_pages, page_size, page_stride, dtype);
    if (s != FORGE_OK) return s;
    if (num_seqs < 1 || rows < 1 || rows > (1 << 30) || table_width < 1 || (long long)table_width * page_size > (1 << 30))
        return FORGE_ERR_INVALID_ARG;
    if (cu_seqlens == nullptr && rows != num_seqs) return FORGE_ERR_INVALID_ARG;
    if (!aligned16(k) || !aligned16(v) || !aligned4(page_table) || !aligned4(starts) ||
        (cu_seqlens && !aligned4(cu_seqlens)))
        return FORGE_ERR_INVALID_ARG;
    const size_t es = dtype == FORGE_DTYPE_BF16 ? 2 : 4, most = (size_t)1 << 36;
    if (k_stride < (size_t)Hkv * D || v_stride < (size_t)Hkv * D || k_stride > most || v_stride > most ||
        k_stride * es % 16 != 0 || v_stride * es % 16 != 0)
        return FORGE_ERR_INVALID_ARG;
    AppendParams p;
    p.src[0] = static_cast<const uint8_t *>(k);
    p.src[1] = static_cast<const uint8_t *>(v);
    p.dst[0] = static_cast<uint8_t *>(k_pages);
    p.dst[1] = static_cast<uint8_t *>(v_pages);
    p.src_stride[0] = (long long)(k_stride * es);
    p.src_stride[1] = (long long)(v_stride * es);
    p.page_stride = (long long)(page_stride * es);
    p.table = page_table;
    p.starts = starts;
    p.cu = cu_seqlens;
    p.num_seqs = num_seqs; p.rows = rows; p.width = table_width; p.page = page_size; p.num_pages = num_pages;
    p.Hkv = Hkv;
    p.chunks = (int)(D * es / 16);
    // few tokens: one a block, so that they spread over the SMs
    const int per_sm = rows / (4 * sm_count());
    p.tokens = per_sm < 1 ? 1 : per_sm > kAppendTokens ? kAppendTokens : per_sm;
    const unsigned blocks = (unsigned)((rows + p.tokens - 1) / p.tokens) + (cu_seqlens != nullptr ? 1 : 0);
    return launch_pdl(paged_append, dim3(blocks), dim3(kAppendThreads), 0,
                      static_cast<cudaStream_t>(stream), p);
}

forge_status forge_attn_paged_copy(void *k_pages, void *v_pages, const int *src, const int *dst, int n, int num_layers,
                                   size_t layer_stride, int num_pages, int Hkv, int page_size, int D,
                                   size_t page_stride, forge_dtype dtype, void *stream) {
    forge_status s = check_pool(k_pages, v_pages, Hkv, D, num_pages, page_size, page_stride, dtype);
    if (s != FORGE_OK) return s;
    const size_t es = dtype == FORGE_DTYPE_BF16 ? 2 : 4;
    if (n < 0 || num_layers < 1 || num_layers > 65535 || layer_stride * es % 16 != 0 ||
        layer_stride > ((size_t)1 << 44) / (size_t)num_layers)
        return FORGE_ERR_INVALID_ARG;
    if (n > 0 && (src == nullptr || dst == nullptr)) return FORGE_ERR_INVALID_ARG;
    for (int i = 0; i < n; i++)
        if (src[i] < 0 || src[i] >= num_pages || dst[i] < 0 || dst[i] >= num_pages) return FORGE_ERR_INVALID_ARG;
    CopyParams p;
    p.pool[0] = static_cast<uint8_t *>(k_pages);
    p.pool[1] = static_cast<uint8_t *>(v_pages);
    p.page_stride = (long long)(page_stride * es);
    p.layer_stride = (long long)(layer_stride * es);
    p.page_bytes = (long long)((size_t)Hkv * page_size * D * es);
    const long long per = (long long)kCopyThreads * kCopyUnroll * 16;
    const long long splits = (p.page_bytes + per - 1) / per;
    p.splits = (int)(splits < 1024 ? splits : 1024);
    PageSet read, written;
    int at = 0;
    while (at < n) {
        // the longest run whose copies do not depend on one another: the next run
        // starts at a page that this one writes, or that it would have to read first
        read.clear();
        written.clear();
        p.pairs = 0;
        for (; at < n && p.pairs < kCopyPairs; at++) {
            if (src[at] == dst[at]) continue;
            if (written.has(src[at]) || written.has(dst[at]) || read.has(dst[at])) break;
            read.add(src[at]);
            written.add(dst[at]);
            p.src[p.pairs] = src[at];
            p.dst[p.pairs++] = dst[at];
        }
        if (p.pairs == 0) continue;  // only pages copied onto themselves were left
        s = launch_pdl(paged_copy, dim3((unsigned)(p.pairs * p.splits), (unsigned)num_layers, 2), dim3(kCopyThreads), 0,
                       static_cast<cudaStream_t>(stream), p);
        if (s != FORGE_OK) return s;
    }
    return FORGE_OK;
}

forge_status forge_attn_check(void *stream) {
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    forge_status s = cuda_status(cudaStreamSynchronize(st));
    if (s != FORGE_OK) return s;
    int h = 0;
    if ((s = cuda_status(cudaMemcpyFromSymbol(&h, g_status, sizeof(int)))) != FORGE_OK) return s;
    if (h != 0) {
        const int zero = 0;
        if ((s = cuda_status(cudaMemcpyToSymbol(g_status, &zero, sizeof(int)))) != FORGE_OK) return s;
        return static_cast<forge_status>(h);
    }
    return FORGE_OK;
}

const char *forge_attn_status_string(forge_status s) {
    switch (s) {
        case FORGE_OK: return "FORGE_OK";
        case FORGE_ERR_INVALID_ARG: return "FORGE_ERR_INVALID_ARG: invalid argument";
        case FORGE_ERR_UNSUPPORTED: return "FORGE_ERR_UNSUPPORTED: unsupported configuration";
        case FORGE_ERR_WORKSPACE: return "FORGE_ERR_WORKSPACE: workspace missing, misaligned or too small";
        case FORGE_ERR_CUDA: return "FORGE_ERR_CUDA: CUDA runtime or launch failure";
        case FORGE_ERR_TIMEOUT: return "FORGE_ERR_TIMEOUT: a bounded wait inside a kernel ran out";
    }
    return "FORGE_ERR_UNKNOWN";
}

forge_status forge_attn_selftest_timeout(unsigned int limit_us, void *stream) {
    if (limit_us < 1 || limit_us > 2000000u) return FORGE_ERR_INVALID_ARG;
    selftest_timeout_kernel<<<1, 32, 0, static_cast<cudaStream_t>(stream)>>>(1000ull * limit_us);
    return launch_status();
}

forge_status forge_attn_selftest_exp2(const float *x, float *y, float *y_ref, int n, void *stream) {
    if (n < 0 || (n > 0 && (x == nullptr || y == nullptr || y_ref == nullptr))) return FORGE_ERR_INVALID_ARG;
    if (n == 0) return FORGE_OK;
    selftest_exp2_kernel<<<(n + 255) / 256, 256, 0, static_cast<cudaStream_t>(stream)>>>(x, y, y_ref, n);
    return launch_status();
}

const char *forge_attn_last_cuda_error(void) { return t_last_cuda_error; }

forge_status forge_attn_timeout_info(unsigned int *info4) {
    if (info4 == nullptr) return FORGE_ERR_INVALID_ARG;
    forge_status s = cuda_status(cudaMemcpyFromSymbol(info4, g_timeout_info, 4 * sizeof(unsigned)));
    if (s != FORGE_OK) return s;
    const unsigned zero[4] = {0, 0, 0, 0};
    return cuda_status(cudaMemcpyToSymbol(g_timeout_info, zero, sizeof(zero)));
}

const char *forge_attn_version(void) { return "forge_attn 0.1.0 sm_100a"; }

}  // extern "C"
