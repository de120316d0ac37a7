// decode_paged.cuh -- one-query attention against a paged KV cache.
//
// A layer's cache is a pool of pages, [num_pages][Hkv][page][D] for K and for V;
// position t of sequence b is row t % page of page page_table[b][t / page], so one
// head's rows of a page are contiguous. HBM-bound: each cache byte is read once, for
// all G query heads of its KV head.
//
// Work split: the visible keys of every (sequence, KV head) pair are cut into units of
// four warp steps (KS keys each, one page), all units of the batch are numbered in
// order, and CTA c of nw takes units [U c / nw, U (c + 1) / nw): equal shares whatever
// the lengths, read from seq_lens on the device. A CTA whose share covers a whole pair
// writes o and lse itself; a pair cut between CTAs leaves (max, sum, o) per CTA in
// the workspace, at most two per CTA (its first and its last pair), the CTA that holds
// the pair's first unit writes down where, and decode_paged_join merges them. Nothing
// depends on a maximum length.
//
// Inside a CTA the four warps take the four steps of each unit, each with its own ring
// of 16-byte asynchronous copies and its own online softmax, and merge when the CTA
// leaves a pair; the copies run ahead across pairs. Rows outside the visible range
// (past the length, before the window, the rest of a sequence's last page) are
// filled with zeros and never read from the pool.
//  - bf16: the G heads are the rows of m16n8k16 products (mma.sync, f32 accumulation):
//    scores Q K^T, then P V with P rounded to bf16 as in the prefill kernels. The tensor
//    cores are idle 90 % of the time; they are used to keep the issue slots free for the
//    copies (the CUDA-core form spends 2 G FMAs an element).
//  - f32: FMAs on the CUDA cores, 32 / KS lanes a key.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "decode.cuh"
#include "simt.cuh"
#include "sm100.cuh"

namespace forge {

constexpr int kPdWarps = 4, kPdThreads = 32 * kPdWarps;
constexpr int kPdMaxG = 16;

template <typename T_, int D>
struct PdCfg {
    static constexpr bool BF = sizeof(T_) == 2;
    static constexpr int KS = BF ? 16 : (D == 256 ? 8 : 16);  // keys of a warp step; divides the page size
    static constexpr int UNIT = KS * kPdWarps;
    static constexpr int ROWB = D * (int)sizeof(T_);
    static constexpr int CPR = ROWB / 16;         // 16-byte chunks a row
    static constexpr int STEP = KS * ROWB;        // bytes of K (or V) of a step
    static constexpr int STAGES = 2 * STEP <= 4096 ? 4 : (!BF && D == 256 ? 2 : 3);  // what shared memory holds
    static constexpr int RING = STAGES * 2 * STEP;  // bytes of one warp's ring
    static constexpr int MERGE = 2 * kPdMaxG * D * 4;  // two warps' o
    static constexpr int STATS = 2 * kPdWarps * kPdMaxG * 4 + 64;
    static constexpr int QB = BF ? 0 : kPdMaxG * D * 4;                 // f32: the group's queries
    static constexpr int PB = BF ? 0 : kPdWarps * KS * kPdMaxG * 4;     // f32: a step's probabilities
    static constexpr int SMEM = kPdWarps * RING + MERGE + STATS + QB + PB;
    // CTAs an SM that shared memory admits (228 KB, 1 KB of it reserved per CTA)
    static constexpr int PER_SM = 233472 / (SMEM + 1024) < 4 ? 233472 / (SMEM + 1024) : 4;
    static_assert(SMEM <= 232448, "shared memory");
};

struct PdParams {
    const void *q, *k, *v;
    void *o;
    float *lse;                // [B][Hq], may be nullptr
    const int *table;          // [B][width]
    const int *seq_lens;       // [B]
    const float *sink;
    float *part;               // [2 nw][G][D]: unnormalised o of a cut pair's pieces
    float2 *stat;              // [2 nw][G]: (max, sum) of those
    int2 *cut;                 // [B][Hkv]: (first piece's slot, pieces; 0 = the pair was not cut)
    long long page_stride;     // elements between pages
    int B, Hq, Hkv, width, page, num_pages, window, workers;
    float qscale;              // scale * log2(e), or scale / softcap with a cap
    float cap_out;             // softcap * log2(e), 0 = no cap
};

// The visible keys of a sequence: [first, len), and the units that hold them.
struct PdSeq {
    int len, first, u0, nu;
};
template <int UNIT>
__device__ __forceinline__ PdSeq pd_seq(const PdParams &p, int b) {
    PdSeq s;
    s.len = p.seq_lens[b];
    if (s.len < 0 || (long long)s.len > (long long)p.width * p.page) {
        record_status(kStatusInvalidArg);  // such a sequence is taken as empty
        s.len = 0;
    }
    s.first = p.window > 0 ? max(0, s.len - p.window) : 0;
    s.u0 = s.first / UNIT;
    s.nu = (int)(((long long)s.len + UNIT - 1) / UNIT) - s.u0;
    return s;
}

// First unit of share c of n.
__device__ __forceinline__ long long pd_share(long long U, int c, int n) {
    if (U < (1 << 20) && n <= 2048) return (unsigned)U * (unsigned)c / (unsigned)n;  // below 2^31
    return U * c / n;
}

// Walks units: sequence b, KV head hk, unit j of the pair's nu.
struct PdIter {
    int b, hk, j;
    PdSeq s;
    template <int UNIT>
    __device__ __forceinline__ void next(const PdParams &p) {
        if (++j < s.nu) return;
        j = 0;
        if (++hk < p.Hkv) return;
        hk = 0;
        do {
            b++;
            if (b < p.B) s = pd_seq<UNIT>(p, b);
        } while (b < p.B && s.nu == 0);
    }
};

__device__ __forceinline__ void pd_copy16(uint32_t dst, const void *src, bool live) {
    const int n = live ? 16 : 0;  // 0: nothing is read, the 16 bytes become zeros
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void pd_copy16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Score of a dot product in log2 units.
__device__ __forceinline__ float pd_score(float x, const PdParams &p) {
    return p.cap_out > 0.0f ? p.cap_out * tanh_via_ex2(x * p.qscale) : x * p.qscale;
}

// One warp's softmax over the group's heads and its share of the keys, bf16 on
// mma.sync: rows (heads) lane / 4 and lane / 4 + 8.
template <int D>
struct PdWarpBf {
    using C = PdCfg<__nv_bfloat16, D>;
    uint32_t q[D / 16][4];
    float o[D / 8][4], m[2], l[2];

    __device__ __forceinline__ void begin(const PdParams &p, int b, int hk, int G, float *) {
        const int lane = threadIdx.x % 32, r = lane / 4;
        const __nv_bfloat16 *Q = static_cast<const __nv_bfloat16 *>(p.q) + ((size_t)b * p.Hq + (size_t)hk * G) * D;
#pragma unroll
        for (int kk = 0; kk < D / 16; kk++)
#pragma unroll
            for (int e = 0; e < 4; e++) {
                const int row = r + 8 * (e & 1), col = 16 * kk + 8 * (e >> 1) + 2 * (lane % 4);
                q[kk][e] = row < G ? *reinterpret_cast<const uint32_t *>(Q + row * D + col) : 0u;
            }
#pragma unroll
        for (int i = 0; i < D / 8; i++)
#pragma unroll
            for (int e = 0; e < 4; e++) o[i][e] = 0.0f;
        m[0] = m[1] = -INFINITY;
        l[0] = l[1] = 0.0f;
    }

    // keys [key0, key0 + 16) in shared memory at sK, sV; visible: [lo, hi)
    __device__ __forceinline__ void step(const PdParams &p, uint32_t sK, uint32_t sV, int key0, int lo, int hi, int G,
                                         float *, const float *) {
        const int lane = threadIdx.x % 32;
        float s[2][4], s2[2][4];  // two chains of products each: even and odd slices of the head dim
#pragma unroll
        for (int i = 0; i < 2; i++)
#pragma unroll
            for (int e = 0; e < 4; e++) s[i][e] = s2[i][e] = 0.0f;
        const int kr = (lane / 16) * 8 + lane % 8, kc = (lane / 8) % 2;
#pragma unroll
        for (int kk = 0; kk < D / 16; kk++) {
            uint32_t b[4];
            ldsm4(sK + (uint32_t)(kr * C::ROWB + (((2 * kk + kc) ^ (kr & 7)) << 4)), b);
            mma16816(kk % 2 ? s2[0] : s[0], q[kk], b[0], b[1]);
            mma16816(kk % 2 ? s2[1] : s[1], q[kk], b[2], b[3]);
        }
#pragma unroll
        for (int i = 0; i < 2; i++)
#pragma unroll
            for (int e = 0; e < 4; e++) s[i][e] += s2[i][e];
        const bool part = key0 < lo || key0 + C::KS > hi;
        float f[2];
        bool moved = false;
#pragma unroll
        for (int h = 0; h < 2; h++) {  // row halves
            float mx = -INFINITY;
#pragma unroll
            for (int i = 0; i < 2; i++)
#pragma unroll
                for (int e = 0; e < 2; e++) {
                    const int key = key0 + 8 * i + 2 * (lane % 4) + e;
                    float y = pd_score(s[i][2 * h + e], p);
                    if (part && (key < lo || key >= hi)) y = -INFINITY;
                    s[i][2 * h + e] = y;
                    mx = fmaxf(mx, y);
                }
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            // the running max moves only when a step exceeds it by a factor 2^8
            const float m_new = mx > m[h] + 8.0f ? mx : m[h];
            f[h] = m_new != m[h] ? ex2_approx(m[h] - m_new) : 1.0f;
            moved |= m_new != m[h];
            m[h] = m_new;
            const float m0 = m_new == -INFINITY ? 0.0f : m_new;
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < 2; i++)
#pragma unroll
                for (int e = 0; e < 2; e++) {
                    const float x = ex2_approx(s[i][2 * h + e] - m0);
                    s[i][2 * h + e] = x;
                    sum += x;
                }
            l[h] = l[h] * f[h] + sum;
        }
        if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
            for (int i = 0; i < D / 8; i++)
#pragma unroll
                for (int e = 0; e < 4; e++) o[i][e] *= f[e >> 1];
        }
        // the scores' accumulator layout is the A operand's: keys are its columns
        const uint32_t a[4] = {pack_bf16x2(s[0][0], s[0][1]), pack_bf16x2(s[0][2], s[0][3]),
                               pack_bf16x2(s[1][0], s[1][1]), pack_bf16x2(s[1][2], s[1][3])};
        const int vr = ((lane / 8) % 2) * 8 + lane % 8, vc = lane / 16;
#pragma unroll
        for (int t = 0; t < D / 16; t++) {
            uint32_t b[4];
            ldsm4_t(sV + (uint32_t)(vr * C::ROWB + (((2 * t + vc) ^ (vr & 7)) << 4)), b);
            mma16816(o[2 * t], a, b[0], b[1]);
            mma16816(o[2 * t + 1], a, b[2], b[3]);
        }
    }
    // row sums over the quad; afterwards lane % 4 == 0 of a row holds (m, l)
    __device__ __forceinline__ void finish() {
#pragma unroll
        for (int h = 0; h < 2; h++) {
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
        }
    }
    __device__ __forceinline__ void put_stats(float *sm, float *sl, int) {
        const int lane = threadIdx.x % 32;
        if (lane % 4 == 0) {
#pragma unroll
            for (int h = 0; h < 2; h++) {
                sm[lane / 4 + 8 * h] = m[h];
                sl[lane / 4 + 8 * h] = l[h];
            }
        }
    }
    // o rows times 2^(m - M[row]) into (add: onto) the [16][D] buffer
    __device__ __forceinline__ void put_o(float *buf, const float *M, int G, bool add) {
        const int lane = threadIdx.x % 32;
#pragma unroll
        for (int h = 0; h < 2; h++) {
            const int row = lane / 4 + 8 * h;
            if (row >= G) continue;
            const float f = m[h] == -INFINITY ? 0.0f : ex2_approx(m[h] - M[row]);
#pragma unroll
            for (int i = 0; i < D / 8; i++) {
                float2 *at = reinterpret_cast<float2 *>(buf + row * D + 8 * i + 2 * (lane % 4));
                float2 x = make_float2(o[i][2 * h] * f, o[i][2 * h + 1] * f);
                if (add) {
                    const float2 y = *at;
                    x.x += y.x;
                    x.y += y.y;
                }
                *at = x;
            }
        }
    }
    __device__ static __forceinline__ int swizzle(int row) { return row & 7; }
};

// f32 on the CUDA cores: LPK lanes share a key's dot products (chunks c with
// c % LPK = lane % LPK), every lane owns D / 32 output dims. MG >= G heads.
template <int D, int MG>
struct PdWarpF32 {
    using C = PdCfg<float, D>;
    static constexpr int LPK = 32 / C::KS, DPL = D / 32;
    float o[MG][DPL], m[MG], l[MG];

    __device__ __forceinline__ void begin(const PdParams &p, int b, int hk, int G, float *sQ) {
        // the block's queries: the caller brackets this with barriers
        const float *Q = static_cast<const float *>(p.q) + ((size_t)b * p.Hq + (size_t)hk * G) * D;
        for (int i = threadIdx.x; i < MG * D; i += kPdThreads) sQ[i] = i < G * D ? Q[i] : 0.0f;
#pragma unroll
        for (int g = 0; g < MG; g++) {
#pragma unroll
            for (int i = 0; i < DPL; i++) o[g][i] = 0.0f;
            m[g] = -INFINITY;
            l[g] = 0.0f;
        }
    }
    __device__ static __forceinline__ int swizzle(int row) { return (row * LPK) & 7; }

    __device__ __forceinline__ void step(const PdParams &p, uint32_t sK, uint32_t sV, int key0, int lo, int hi, int G,
                                         float *sP, const float *sQ) {
        const int lane = threadIdx.x % 32, kr = lane / LPK, sub = lane % LPK;
        float s[MG];
#pragma unroll
        for (int g = 0; g < MG; g++) s[g] = 0.0f;
#pragma unroll 4
        for (int c = 0; c < D / 4; c += LPK) {
            float4 k;
            asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                         : "=f"(k.x), "=f"(k.y), "=f"(k.z), "=f"(k.w)
                         : "r"(sK + (uint32_t)(kr * C::ROWB + (((c + sub) ^ swizzle(kr)) << 4))));
#pragma unroll
            for (int g = 0; g < MG; g++) {
                const float4 x = *reinterpret_cast<const float4 *>(sQ + g * D + (c + sub) * 4);
                s[g] = fmaf(x.x, k.x, s[g]);
                s[g] = fmaf(x.y, k.y, s[g]);
                s[g] = fmaf(x.z, k.z, s[g]);
                s[g] = fmaf(x.w, k.w, s[g]);
            }
        }
        const bool ok = key0 + kr >= lo && key0 + kr < hi;
        __syncwarp();  // the previous step's probabilities have been read
#pragma unroll
        for (int g = 0; g < MG; g++) {
#pragma unroll
            for (int x = 1; x < LPK; x <<= 1) s[g] += __shfl_xor_sync(0xffffffffu, s[g], x);
            const float y = ok ? pd_score(s[g], p) : -INFINITY;
            float mx = y;
#pragma unroll
            for (int x = LPK; x < 32; x <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
            if (mx > m[g] + 8.0f) {  // warp-uniform
                const float f = ex2_approx(m[g] - mx);
                m[g] = mx;
                l[g] *= f;
#pragma unroll
                for (int i = 0; i < DPL; i++) o[g][i] *= f;
            }
            const float e = ex2_approx(y - (m[g] == -INFINITY ? 0.0f : m[g]));
            if (sub == 0) {
                l[g] += e;
                sP[kr * MG + g] = e;
            }
        }
        __syncwarp();
#pragma unroll 2
        for (int k = 0; k < C::KS; k++) {
            float v[DPL];
            const uint32_t row = sV + (uint32_t)(k * C::ROWB);
            if constexpr (DPL == 2) {
                asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];"
                             : "=f"(v[0]), "=f"(v[1])
                             : "r"(row + (uint32_t)((((lane / 2) ^ swizzle(k)) << 4) + (lane % 2) * 8)));
            } else {
#pragma unroll
                for (int i = 0; i < DPL; i += 4)  // chunks lane, lane + 32
                    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                                 : "=f"(v[i]), "=f"(v[i + 1]), "=f"(v[i + 2]), "=f"(v[i + 3])
                                 : "r"(row + (uint32_t)(((lane + 8 * i) ^ swizzle(k)) << 4)));
            }
#pragma unroll
            for (int g = 0; g < MG; g++) {
                const float e = sP[k * MG + g];
#pragma unroll
                for (int i = 0; i < DPL; i++) o[g][i] = fmaf(e, v[i], o[g][i]);
            }
        }
    }
    __device__ __forceinline__ void finish() {
#pragma unroll
        for (int g = 0; g < MG; g++) l[g] = warp_sum(l[g]);
    }
    __device__ __forceinline__ void put_stats(float *sm, float *sl, int) {
        if (threadIdx.x % 32 == 0) {
#pragma unroll
            for (int g = 0; g < MG; g++) {
                sm[g] = m[g];
                sl[g] = l[g];
            }
        }
    }
    __device__ __forceinline__ void put_o(float *buf, const float *M, int G, bool add) {
        const int lane = threadIdx.x % 32;
#pragma unroll
        for (int g = 0; g < MG; g++) {
            if (g >= G) break;
            const float f = m[g] == -INFINITY ? 0.0f : ex2_approx(m[g] - M[g]);
#pragma unroll
            for (int i = 0; i < DPL; i++) {
                float *at = buf + g * D + (DPL == 2 ? lane * 2 + i : (lane + 8 * (i & ~3)) * 4 + (i & 3));
                *at = o[g][i] * f + (add ? *at : 0.0f);
            }
        }
    }
};

// o and lse of one (sequence, head) from the unnormalised o, the max (log2 units)
// and the sum; the sink (natural units) joins the sum here, once. A sum of 0: nothing is
// visible. A NaN among the visible scores makes the sum, and so both results, NaN.
__device__ __forceinline__ float pd_total(float M, float l, const PdParams &p, int hq, float &scale_o, float &lse) {
    if (p.sink != nullptr) {
        const float sk = p.sink[hq] * kLog2e;
        const float M2 = fmaxf(M, sk);
        const float f = M == -INFINITY ? 0.0f : ex2_approx(M - M2);
        l = l * f + (sk == -INFINITY ? 0.0f : ex2_approx(sk - M2));
        scale_o = l != 0.0f ? f / l : 0.0f;
        lse = l != 0.0f ? (M2 + __log2f(l)) * kLn2 : -INFINITY;
    } else {
        scale_o = l != 0.0f ? 1.0f / l : 0.0f;
        lse = l != 0.0f ? (M + __log2f(l)) * kLn2 : -INFINITY;
    }
    return l;
}

template <typename T_, int D, class W>
__global__ void __launch_bounds__(kPdThreads, PdCfg<T_, D>::PER_SM) decode_paged_split(const PdParams p) {
    using C = PdCfg<T_, D>;
    extern __shared__ __align__(128) uint8_t smem[];
    float *sO = reinterpret_cast<float *>(smem + kPdWarps * C::RING);  // [2][16][D]
    float *sM = sO + 2 * kPdMaxG * D, *sL = sM + kPdWarps * kPdMaxG;   // [warps][16]
    long long *red = reinterpret_cast<long long *>(sL + kPdWarps * kPdMaxG);
    float *sQ = reinterpret_cast<float *>(red + 8);                    // f32: [16][D]
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, G = p.Hq / p.Hkv;
    float *sP = sQ + C::QB / 4 + warp * (C::PB / 4 / kPdWarps);
    const uint32_t ring = smem_u32(smem) + (uint32_t)(warp * C::RING);
    griddep_launch_dependents();
    griddep_wait();

    // this CTA's units, and the sequence that holds the first: prefix sums over the
    // sequences, 128 at a time (after a pass for the total, if there are more)
    long long U = 0, lo = 0, hi = 0;
    int nw = 1;
    PdIter ld;
    long long pair0 = 0;  // first unit of the iterator's pair
    {
        if (p.B > kPdThreads) {
            long long n = 0;
            for (int b = threadIdx.x; b < p.B; b += kPdThreads) n += pd_seq<C::UNIT>(p, b).nu;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
            if (lane == 0) red[warp] = n;
            __syncthreads();
            for (int w = 0; w < kPdWarps; w++) U += red[w] * p.Hkv;
        }
        long long before = 0;
        for (int b0 = 0; b0 < p.B; b0 += kPdThreads) {
            const int b = b0 + (int)threadIdx.x;
            const int nu = b < p.B ? pd_seq<C::UNIT>(p, b).nu : 0;
            long long s = nu;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long y = __shfl_up_sync(0xffffffffu, s, o);
                if (lane >= o) s += y;
            }
            __syncthreads();
            if (lane == 31) red[warp] = s;
            __syncthreads();
            long long chunk = 0;
            for (int w = 0; w < kPdWarps; w++) {
                if (w < warp) s += red[w];
                chunk += red[w];
            }
            if (p.B <= kPdThreads) U = chunk * p.Hkv;
            if (b0 == 0) {
                if (U == 0) return;  // every sequence is empty: the join writes them
                nw = (int)min((long long)gridDim.x, U);
                if ((int)blockIdx.x >= nw) return;
                lo = pd_share(U, (int)blockIdx.x, nw);
                hi = pd_share(U, (int)blockIdx.x + 1, nw);
            }
            const long long u = (before + s - nu) * p.Hkv;  // first unit of sequence b
            if (nu > 0 && u <= lo && lo < u + (long long)nu * p.Hkv) {
                red[4] = b;
                red[5] = u;
            }
            before += chunk;
        }
        __syncthreads();
        ld.b = (int)red[4];
        ld.s = pd_seq<C::UNIT>(p, ld.b);
        const long long r = lo - red[5];
        ld.hk = (int)(r / ld.s.nu);
        ld.j = (int)(r % ld.s.nu);
        pair0 = lo - ld.j;
    }
    PdIter at = ld;

    // The page of this warp's step of the iterator's unit; -1 = nothing visible there, or a
    // page outside the pool, which is reported and taken as holding no visible key.
    auto page_of = [&](const PdIter &i) -> int {
        const int key0 = (i.s.u0 + i.j) * C::UNIT + warp * C::KS;
        if (key0 >= i.s.len || key0 + C::KS <= i.s.first) return -1;
        const int pg = p.table[(long long)i.b * p.width + key0 / p.page];
        if ((unsigned)pg >= (unsigned)p.num_pages) {
            record_status(kStatusInvalidArg);
            return -1;
        }
        return pg;
    };
    auto load = [&](const PdIter &i, int pg, int stage) {
        const int key0 = (i.s.u0 + i.j) * C::UNIT + warp * C::KS;
        const long long base = pg < 0 ? 0 : (long long)pg * p.page_stride + ((long long)i.hk * p.page + key0 % p.page) * D;
        const uint8_t *K = reinterpret_cast<const uint8_t *>(static_cast<const T_ *>(p.k) + base);
        const uint8_t *V = reinterpret_cast<const uint8_t *>(static_cast<const T_ *>(p.v) + base);
        const uint32_t dst = ring + (uint32_t)(stage * 2 * C::STEP);
        if (pg >= 0 && key0 >= i.s.first && key0 + C::KS <= i.s.len) {  // every row visible
#pragma unroll
            for (int e = 0; e < C::KS * C::CPR / 32; e++) {
                const int c = e * 32 + lane, r = c / C::CPR;
                const uint32_t to = (uint32_t)(r * C::ROWB + (((c % C::CPR) ^ W::swizzle(r)) << 4));
                pd_copy16(dst + to, K + c * 16);
                pd_copy16(dst + C::STEP + to, V + c * 16);
            }
        } else {
#pragma unroll 1
            for (int e = 0; e < C::KS * C::CPR / 32; e++) {
                const int c = e * 32 + lane, r = c / C::CPR, key = key0 + r;
                const bool live = pg >= 0 && key >= i.s.first && key < i.s.len;
                const uint32_t to = (uint32_t)(r * C::ROWB + (((c % C::CPR) ^ W::swizzle(r)) << 4));
                const size_t from = live ? (size_t)c * 16 : 0;
                pd_copy16(dst + to, K + from, live);
                pd_copy16(dst + C::STEP + to, V + from, live);
            }
        }
    };
    long long to_load = hi - lo;
    int pg = page_of(ld);
    unsigned held = 0;  // bit s: stage s holds keys of a page (not just zeros)
    auto issue = [&](int stage) {
        if (to_load > 0) {
            const PdIter now = ld;
            const int page_now = pg;
            if (--to_load > 0) {
                ld.next<C::UNIT>(p);
                pg = page_of(ld);  // one step ahead of its use
            }
            load(now, page_now, stage);
            held = (held & ~(1u << stage)) | ((unsigned)(page_now >= 0) << stage);
        }
        cp_async_commit();  // an empty group keeps the count
    };
#pragma unroll
    for (int s = 0; s < C::STAGES - 1; s++) issue(s);

    W acc;
    bool fresh = true;
    bool first_pair = true;
    bool whole = at.j == 0;  // the CTA holds the current pair from its first unit on
    int stage = 0;
    for (long long u = lo; u < hi; u++) {
        if (fresh) {
            if (!C::BF) __syncthreads();  // the previous pair's queries have been read
            acc.begin(p, at.b, at.hk, G, sQ);
            if (!C::BF) __syncthreads();
            fresh = false;
        }
        const int end = (held >> stage) & 1u ? at.s.len : 0;  // no page: no visible key
        cp_async_wait<C::STAGES - 2>();
        __syncwarp();  // every lane's copies of this stage, and all reads of the stage refilled next
        issue(stage == 0 ? C::STAGES - 1 : stage - 1);
        const int key0 = (at.s.u0 + at.j) * C::UNIT + warp * C::KS;
        const uint32_t sK = ring + (uint32_t)(stage * 2 * C::STEP);
        acc.step(p, sK, sK + C::STEP, key0, at.s.first, end, G, sP, sQ);
        stage = stage + 1 == C::STAGES ? 0 : stage + 1;

        const bool pair_end = at.j + 1 == at.s.nu;
        if (pair_end || u + 1 == hi) {
            // the four warps' results: a common max, then o summed in a fixed order
            const bool done = pair_end && whole;
            acc.finish();
            acc.put_stats(sM + warp * kPdMaxG, sL + warp * kPdMaxG, G);
            __syncthreads();
            if (threadIdx.x < kPdMaxG) {
                const int r = threadIdx.x;
                float M = -INFINITY, l = 0.0f;
                for (int w = 0; w < kPdWarps; w++) M = fmaxf(M, sM[w * kPdMaxG + r]);
                for (int w = 0; w < kPdWarps; w++) {
                    // (a maximum of -inf: the sum is 0, or NaN if all of the warp's scores were)
                    const float mw = sM[w * kPdMaxG + r], lw = sL[w * kPdMaxG + r];
                    l += mw == -INFINITY ? lw : lw * ex2_approx(mw - M);
                }
                sM[r] = M;  // rows of warp 0: read by this thread alone
                sL[r] = l;
            }
            __syncthreads();
            if (warp >= 2) acc.put_o(sO + (warp - 2) * kPdMaxG * D, sM, G, false);
            __syncthreads();
            if (warp < 2) acc.put_o(sO + warp * kPdMaxG * D, sM, G, true);
            __syncthreads();
            if (done) {
                T_ *O = static_cast<T_ *>(p.o) + ((size_t)at.b * p.Hq + (size_t)at.hk * G) * D;
                for (int i = threadIdx.x; i < G * D; i += kPdThreads) {
                    const int r = i / D;
                    float f, lse;
                    pd_total(sM[r], sL[r], p, at.hk * G + r, f, lse);
                    from_f32(O + i, (sO[i] + sO[kPdMaxG * D + i]) * f);
                    if (p.lse != nullptr && i % D == 0) p.lse[(size_t)at.b * p.Hq + at.hk * G + r] = lse;
                }
            } else {
                const size_t slot = 2 * (size_t)blockIdx.x + (first_pair ? 0 : 1);
                for (int i = threadIdx.x; i < G * D; i += kPdThreads) p.part[slot * G * D + i] = sO[i] + sO[kPdMaxG * D + i];
                if ((int)threadIdx.x < G) p.stat[slot * G + threadIdx.x] = make_float2(sM[threadIdx.x], sL[threadIdx.x]);
            }
            if (whole && threadIdx.x == 0) {
                // where the join finds the pair's pieces: this CTA's, then the first one
                // of each of the CTAs up to the one that holds the pair's last unit
                int2 cut = make_int2(2 * (int)blockIdx.x + (first_pair ? 0 : 1), 0);
                if (!done) {
                    // share c ends past unit x: c < (x + 1) nw / U
                    const long long x = pair0 + at.s.nu - 1;
                    cut.y = (int)(((x + 1) * nw - 1) / U) - (int)blockIdx.x + 1;
                }
                p.cut[(size_t)at.b * p.Hkv + at.hk] = cut;
            }
            fresh = true;
            first_pair = false;
            whole = true;
            pair0 = u + 1;
            __syncthreads();  // sM, sL are read before the next pair's are written
        }
        if (u + 1 < hi) at.next<C::UNIT>(p);
    }
    cp_async_wait<0>();
}

// One block per (sequence, query head), a thread per head dim: merges the pieces of
// a pair that was cut between CTAs; writes the empty sequences.
template <typename T_, int D>
__global__ void __launch_bounds__(D) decode_paged_join(const PdParams p) {
    using C = PdCfg<T_, D>;
    griddep_launch_dependents();
    griddep_wait();
    const int b = blockIdx.x / p.Hq, hq = blockIdx.x % p.Hq, G = p.Hq / p.Hkv, hk = hq / G, r = hq % G;
    const int d = threadIdx.x, lane = threadIdx.x % 32;
    const PdSeq s = pd_seq<C::UNIT>(p, b);
    const int2 cut = p.cut[(size_t)b * p.Hkv + hk];  // of an earlier call if the sequence is empty
    if (s.nu > 0 && cut.y == 0) return;
    float M = -INFINITY, l = 0.0f, acc = 0.0f;
    if (s.nu > 0) {
        auto slot = [&](int c) -> size_t { return c == 0 ? (size_t)cut.x : 2 * ((size_t)cut.x / 2 + c); };
        for (int c0 = 0; c0 < cut.y; c0 += 32) {  // 32 pieces at a time
            const int n = min(32, cut.y - c0);
            const float2 x = lane < n ? p.stat[slot(c0 + lane) * G + r] : make_float2(-INFINITY, 0.0f);
            const float M2 = fmaxf(M, warp_max(x.x));
            const float M0 = M2 == -INFINITY ? 0.0f : M2;
            const float f = ex2_approx(x.x - M0), keep = ex2_approx(M - M0);
            l = l * keep + warp_sum(x.y * f);
            acc *= keep;
            M = M2;
#pragma unroll 8
            for (int c = 0; c < n; c++)
                acc = fmaf(p.part[(slot(c0 + c) * G + r) * D + d], __shfl_sync(0xffffffffu, f, c), acc);
        }
    }
    float f, lse;
    pd_total(M, l, p, hq, f, lse);
    from_f32(static_cast<T_ *>(p.o) + ((size_t)b * p.Hq + hq) * D + d, s.nu > 0 ? acc * f : 0.0f);
    if (p.lse != nullptr && d == 0) p.lse[(size_t)b * p.Hq + hq] = lse;
}

}  // namespace forge
