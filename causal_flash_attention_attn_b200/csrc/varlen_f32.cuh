// varlen_f32.cuh -- f32 attention over packed sequences on the CUDA cores (exact
// f32 FMAs, as simt.cuh, for the 1e-4 parity bar), register-tiled.
//
// A block of 256 threads (16 x 16) owns 64 rows of one head and streams BK rows of
// the other operand through shared memory. Thread (ty, tx) computes the products of
// rows 4 ty .. 4 ty + 3 with streamed rows tx, tx + 16, ..: a step over four head
// dims takes 4 + BK / 16 16-byte shared loads (the four broadcast over tx) for
// 4 * BK FMAs per 16 lanes, so the FMA pipe, not the shared-memory port, is the
// bound. Rows are D + 4 floats apart, which puts the 16-byte loads of eight lanes on
// eight rows into 32 different banks. The second products (P V, dS K, P^T dO,
// dS^T Q) read P or dS back from shared memory as broadcasts; thread (ty, tx) owns
// columns 4 tx + 64 j of its four output rows.
//  - varlen_f32_fwd:      rows = queries, streams K, V; o and lse.
//  - varlen_f32_bwd_dq:   rows = queries, streams K, V; dq.
//  - varlen_f32_bwd_dkdv: rows = keys, streams Q, dO of every head of the group; dk, dv.
// No atomics: one writer per output element, in a fixed order.
#pragma once

#include "simt.cuh"
#include "varlen_item.cuh"

namespace forge {

constexpr int kVfRows = 64;  // rows of a tile (the schedule's unit)
constexpr int kVfThreads = 256;

// Streamed rows per step: as many as leave two blocks an SM (one at head dim 256).
template <int D>
constexpr int vf_bk() {
    return D == 64 ? 64 : 32;
}

struct VfParams {
    const float *q, *k, *v, *dO;
    long long q_row, k_row, v_row;  // floats between rows; dO and the outputs are dense
    float *o, *lse, *dq, *dk, *dv;
    const float *delta;
    int Hq, Hkv, window;
    float scale, softcap;
    const float *sink;
    VarSched var;
};

// Rows [r0, r0 + N) of a [.. rows ..][D] tensor (row stride `ld` floats) into shared
// memory rows of D + 4 floats; rows at or past `end` become zeros.
template <int D, int N>
__device__ __forceinline__ void vf_load(float *dst, const float *src, long long ld, int r0, int end) {
#pragma unroll 4
    for (int i = threadIdx.x; i < N * (D / 4); i += kVfThreads) {
        const int r = i / (D / 4), c = i % (D / 4);
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r0 + r < end) x = *reinterpret_cast<const float4 *>(src + (long long)(r0 + r) * ld + c * 4);
        *reinterpret_cast<float4 *>(dst + r * (D + 4) + c * 4) = x;
    }
}

// s[i][j] = sum_d A[4 ty + i][d] B[tx + 16 j][d]
template <int D, int BK>
__device__ __forceinline__ void vf_dots(const float *A, const float *B, float (&s)[4][BK / 16]) {
    const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
#pragma unroll
    for (int i = 0; i < 4; i++)
#pragma unroll
        for (int j = 0; j < BK / 16; j++) s[i][j] = 0.0f;
#pragma unroll 4
    for (int d = 0; d < D; d += 4) {
        float4 a[4], b[BK / 16];
#pragma unroll
        for (int i = 0; i < 4; i++) a[i] = *reinterpret_cast<const float4 *>(A + (4 * ty + i) * (D + 4) + d);
#pragma unroll
        for (int j = 0; j < BK / 16; j++) b[j] = *reinterpret_cast<const float4 *>(B + (tx + 16 * j) * (D + 4) + d);
#pragma unroll
        for (int i = 0; i < 4; i++)
#pragma unroll
            for (int j = 0; j < BK / 16; j++) {
                s[i][j] = fmaf(a[i].x, b[j].x, s[i][j]);
                s[i][j] = fmaf(a[i].y, b[j].y, s[i][j]);
                s[i][j] = fmaf(a[i].z, b[j].z, s[i][j]);
                s[i][j] = fmaf(a[i].w, b[j].w, s[i][j]);
            }
    }
}

// acc[i][.] += sum_j P[4 ty + i][j] B[j][4 tx + 64 ..], P rows BK + 4 floats apart
template <int D, int BK>
__device__ __forceinline__ void vf_accumulate(const float *P, const float *B, float (&acc)[4][D / 16]) {
    const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
#pragma unroll 2
    for (int j = 0; j < BK; j += 4) {
        float4 p[4];
#pragma unroll
        for (int i = 0; i < 4; i++) p[i] = *reinterpret_cast<const float4 *>(P + (4 * ty + i) * (BK + 4) + j);
#pragma unroll
        for (int e = 0; e < 4; e++) {
#pragma unroll
            for (int c = 0; c < D / 64; c++) {
                const float4 b = *reinterpret_cast<const float4 *>(B + (j + e) * (D + 4) + 4 * tx + 64 * c);
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const float x = e == 0 ? p[i].x : e == 1 ? p[i].y : e == 2 ? p[i].z : p[i].w;
                    acc[i][4 * c + 0] = fmaf(x, b.x, acc[i][4 * c + 0]);
                    acc[i][4 * c + 1] = fmaf(x, b.y, acc[i][4 * c + 1]);
                    acc[i][4 * c + 2] = fmaf(x, b.z, acc[i][4 * c + 2]);
                    acc[i][4 * c + 3] = fmaf(x, b.w, acc[i][4 * c + 3]);
                }
            }
        }
    }
}

// Row r of this thread's four output rows, `f` times the accumulator.
template <int D>
__device__ __forceinline__ void vf_store(float *row, const float (&acc)[D / 16], float f) {
    const int tx = threadIdx.x % 16;
#pragma unroll
    for (int c = 0; c < D / 64; c++)
        *reinterpret_cast<float4 *>(row + 4 * tx + 64 * c) =
            make_float4(acc[4 * c] * f, acc[4 * c + 1] * f, acc[4 * c + 2] * f, acc[4 * c + 3] * f);
}

template <int D>
constexpr size_t vf_fwd_smem() {
    return sizeof(float) * (size_t)((kVfRows + 2 * vf_bk<D>()) * (D + 4) + kVfRows * (vf_bk<D>() + 4));
}
template <int D>
constexpr size_t vf_bwd_dq_smem() {
    return sizeof(float) * (size_t)((2 * kVfRows + 2 * vf_bk<D>()) * (D + 4) + kVfRows * (vf_bk<D>() + 4));
}
template <int D>
constexpr size_t vf_bwd_dkdv_smem() {
    return sizeof(float) *
           (size_t)((2 * kVfRows + 2 * vf_bk<D>()) * (D + 4) + 2 * kVfRows * (vf_bk<D>() + 4) + 2 * vf_bk<D>());
}

template <int D>
__global__ void __launch_bounds__(kVfThreads, 1) varlen_f32_fwd(const VfParams p) {
    constexpr int BK = vf_bk<D>(), NJ = BK / 16;
    extern __shared__ __align__(16) float sm[];
    float *sQ = sm, *sK = sQ + kVfRows * (D + 4), *sV = sK + BK * (D + 4), *sP = sV + BK * (D + 4);
    griddep_launch_dependents();
    griddep_wait();
    const int w = blockIdx.x, h = w % p.Hq, hk = h / (p.Hq / p.Hkv);
    if (w / p.Hq >= var_count(p.var)) return;
    const VarItem it = var_item(p.var, w / p.Hq);
    const int q0 = it.tile * kVfRows, W = p.window >= it.len ? 0 : p.window;
    const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
    const float *K = p.k + (long long)it.row0 * p.k_row + (long long)hk * D;
    const float *V = p.v + (long long)it.row0 * p.v_row + (long long)hk * D;
    vf_load<D, kVfRows>(sQ, p.q + (long long)it.row0 * p.q_row + (long long)h * D, p.q_row, q0, it.len);
    // a sink (natural units) starts each row's (max, sum) at (sink, 1)
    float m[4], l[4], acc[4][D / 16];
#pragma unroll
    for (int i = 0; i < 4; i++) {
        m[i] = p.sink ? p.sink[h] : -INFINITY;
        l[i] = p.sink ? 1.0f : 0.0f;
#pragma unroll
        for (int c = 0; c < D / 16; c++) acc[i][c] = 0.0f;
    }
    const int last = min(q0 + kVfRows, it.len) - 1;
    for (int k0 = W > 0 ? max(0, q0 - W + 1) / BK * BK : 0; k0 <= last; k0 += BK) {
        __syncthreads();
        vf_load<D, BK>(sK, K, p.k_row, k0, it.len);
        vf_load<D, BK>(sV, V, p.v_row, k0, it.len);
        __syncthreads();
        float s[4][NJ];
        vf_dots<D, BK>(sQ, sK, s);
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const int qi = q0 + 4 * ty + i;
            float mx = -INFINITY;
#pragma unroll
            for (int j = 0; j < NJ; j++) {
                const int kj = k0 + tx + 16 * j;
                s[i][j] = visible(qi, kj, W) ? simt_capped(s[i][j] * p.scale, p.softcap) : -INFINITY;
                mx = fmaxf(mx, s[i][j]);
            }
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            const float m_new = fmaxf(m[i], mx);
            const float m0 = m_new == -INFINITY ? 0.0f : m_new;
            const float corr = expf(m[i] - m0);  // 0 while the row has seen nothing
            float sum = 0.0f;
#pragma unroll
            for (int j = 0; j < NJ; j++) {
                const float e = expf(s[i][j] - m0);
                sum += e;
                sP[(4 * ty + i) * (BK + 4) + tx + 16 * j] = e;
            }
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            l[i] = l[i] * corr + sum;
            m[i] = m_new;
#pragma unroll
            for (int c = 0; c < D / 16; c++) acc[i][c] *= corr;
        }
        __syncwarp();  // a warp reads back only the P rows that it wrote
        vf_accumulate<D, BK>(sP, sV, acc);
        __syncwarp();
    }
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const int qi = q0 + 4 * ty + i;
        if (qi >= it.len) continue;
        const size_t row = (size_t)it.row0 + qi;
        vf_store<D>(p.o + (row * p.Hq + h) * D, acc[i], 1.0f / l[i]);
        if (tx == 0) p.lse[(size_t)h * p.var.rows + row] = m[i] + logf(l[i]);
    }
}

// P and dS of one score: P = exp(s - lse), dS = P (dP - Delta) [* (1 - tanh^2)],
// both 0 where the pair is not visible.
__device__ __forceinline__ void vf_pds(float dot, float dp, float lse, float delta, bool ok, const VfParams &p,
                                       float &pr, float &ds) {
    const float sc = simt_capped(dot * p.scale, p.softcap);
    pr = ok ? expf(sc - lse) : 0.0f;
    const float t = p.softcap > 0.0f ? sc / p.softcap : 0.0f;
    ds = ok ? pr * (dp - delta) * (1.0f - t * t) : 0.0f;
}

template <int D>
__global__ void __launch_bounds__(kVfThreads, 1) varlen_f32_bwd_dq(const VfParams p) {
    constexpr int BK = vf_bk<D>(), NJ = BK / 16;
    extern __shared__ __align__(16) float sm[];
    float *sQ = sm, *sO = sQ + kVfRows * (D + 4), *sK = sO + kVfRows * (D + 4), *sV = sK + BK * (D + 4),
          *sS = sV + BK * (D + 4);
    griddep_launch_dependents();
    griddep_wait();
    const int w = blockIdx.x, h = w % p.Hq, hk = h / (p.Hq / p.Hkv);
    if (w / p.Hq >= var_count(p.var)) return;
    const VarItem it = var_item(p.var, w / p.Hq);
    const int q0 = it.tile * kVfRows, W = p.window >= it.len ? 0 : p.window;
    const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
    const float *K = p.k + (long long)it.row0 * p.k_row + (long long)hk * D;
    const float *V = p.v + (long long)it.row0 * p.v_row + (long long)hk * D;
    vf_load<D, kVfRows>(sQ, p.q + (long long)it.row0 * p.q_row + (long long)h * D, p.q_row, q0, it.len);
    vf_load<D, kVfRows>(sO, p.dO + ((long long)it.row0 * p.Hq + h) * D, (long long)p.Hq * D, q0, it.len);
    float acc[4][D / 16], L[4], Dl[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const size_t at = (size_t)h * p.var.rows + it.row0 + min(q0 + 4 * ty + i, it.len - 1);
        L[i] = p.lse[at];
        Dl[i] = p.delta[at];
#pragma unroll
        for (int c = 0; c < D / 16; c++) acc[i][c] = 0.0f;
    }
    const int last = min(q0 + kVfRows, it.len) - 1;
    for (int k0 = W > 0 ? max(0, q0 - W + 1) / BK * BK : 0; k0 <= last; k0 += BK) {
        __syncthreads();
        vf_load<D, BK>(sK, K, p.k_row, k0, it.len);
        vf_load<D, BK>(sV, V, p.v_row, k0, it.len);
        __syncthreads();
        float s[4][NJ], dp[4][NJ];
        vf_dots<D, BK>(sQ, sK, s);
        vf_dots<D, BK>(sO, sV, dp);
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const int qi = q0 + 4 * ty + i;
#pragma unroll
            for (int j = 0; j < NJ; j++) {
                float pr, ds;
                vf_pds(s[i][j], dp[i][j], L[i], Dl[i], qi < it.len && visible(qi, k0 + tx + 16 * j, W), p, pr, ds);
                sS[(4 * ty + i) * (BK + 4) + tx + 16 * j] = ds;
            }
        }
        __syncwarp();
        vf_accumulate<D, BK>(sS, sK, acc);
        __syncwarp();
    }
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const int qi = q0 + 4 * ty + i;
        if (qi < it.len) vf_store<D>(p.dq + (((size_t)it.row0 + qi) * p.Hq + h) * D, acc[i], p.scale);
    }
}

template <int D>
__global__ void __launch_bounds__(kVfThreads, 1) varlen_f32_bwd_dkdv(const VfParams p) {
    constexpr int BK = vf_bk<D>(), NJ = BK / 16;
    extern __shared__ __align__(16) float sm[];
    float *sK = sm, *sV = sK + kVfRows * (D + 4), *sQ = sV + kVfRows * (D + 4), *sO = sQ + BK * (D + 4),
          *sP = sO + BK * (D + 4), *sS = sP + kVfRows * (BK + 4), *sL = sS + kVfRows * (BK + 4), *sD = sL + BK;
    griddep_launch_dependents();
    griddep_wait();
    const int w = blockIdx.x, hk = w % p.Hkv, G = p.Hq / p.Hkv;
    if (w / p.Hkv >= var_count(p.var)) return;
    const VarItem it = var_item(p.var, w / p.Hkv);
    const int k0 = it.tile * kVfRows, W = p.window >= it.len ? 0 : p.window;
    const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
    vf_load<D, kVfRows>(sK, p.k + (long long)it.row0 * p.k_row + (long long)hk * D, p.k_row, k0, it.len);
    vf_load<D, kVfRows>(sV, p.v + (long long)it.row0 * p.v_row + (long long)hk * D, p.v_row, k0, it.len);
    float adk[4][D / 16], adv[4][D / 16];
#pragma unroll
    for (int i = 0; i < 4; i++)
#pragma unroll
        for (int c = 0; c < D / 16; c++) adk[i][c] = adv[i][c] = 0.0f;
    const int last = W > 0 ? (int)min((long long)it.len - 1, (long long)k0 + kVfRows - 1 + W - 1) : it.len - 1;
    for (int g = 0; g < G; g++) {
        const int h = hk * G + g;
        const float *Q = p.q + (long long)it.row0 * p.q_row + (long long)h * D;
        const float *dO = p.dO + ((long long)it.row0 * p.Hq + h) * D;
        for (int q0 = k0; q0 <= last; q0 += BK) {
            __syncthreads();
            vf_load<D, BK>(sQ, Q, p.q_row, q0, it.len);
            vf_load<D, BK>(sO, dO, (long long)p.Hq * D, q0, it.len);
            if (threadIdx.x < BK) {
                const size_t at = (size_t)h * p.var.rows + it.row0 + min(q0 + (int)threadIdx.x, it.len - 1);
                sL[threadIdx.x] = p.lse[at];
                sD[threadIdx.x] = p.delta[at];
            }
            __syncthreads();
            float s[4][NJ], dp[4][NJ];
            vf_dots<D, BK>(sK, sQ, s);
            vf_dots<D, BK>(sV, sO, dp);
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const int kj = k0 + 4 * ty + i;
#pragma unroll
                for (int j = 0; j < NJ; j++) {
                    const int c = tx + 16 * j, qi = q0 + c;
                    float pr, ds;
                    vf_pds(s[i][j], dp[i][j], sL[c], sD[c], qi < it.len && visible(qi, kj, W), p, pr, ds);
                    sP[(4 * ty + i) * (BK + 4) + c] = pr;
                    sS[(4 * ty + i) * (BK + 4) + c] = ds;
                }
            }
            __syncwarp();
            vf_accumulate<D, BK>(sP, sO, adv);
            vf_accumulate<D, BK>(sS, sQ, adk);
        }
    }
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const int kj = k0 + 4 * ty + i;
        if (kj >= it.len) continue;
        const size_t at = (((size_t)it.row0 + kj) * p.Hkv + hk) * D;
        vf_store<D>(p.dk + at, adk[i], p.scale);
        vf_store<D>(p.dv + at, adv[i], 1.0f);
    }
}

}  // namespace forge
