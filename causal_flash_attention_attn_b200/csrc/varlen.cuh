// varlen.cuh -- attention over packed sequences: the schedule, and the HBM-bound
// stages around the backward.
//
// Sequences of different lengths lie one after the other along the row axis of
// [rows][heads][D] tensors; cu_seqlens[b] is the first row of sequence b and
// cu_seqlens[num_seqs] the first row behind the last one. Query and key tiles
// start at their sequence's first row, so a tile never mixes two sequences and
// one sequence's values (an infinity, a NaN) never reach another's results.
//
// The lengths are read on the device: varlen_plan writes the list of tiles that
// the attention kernels walk, heaviest first (a tile's weight is the span of keys,
// or of queries in the backward, that it has to visit), with the number of tiles
// in front. Launches are sized by an upper bound that needs only `rows` and
// `num_seqs`.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "bwd_aux.cuh"
#include "simt.cuh"
#include "sm100.cuh"
#include "varlen_item.cuh"

namespace forge {

constexpr int kPlanParts = 2;
constexpr int kPlanThreads = 1024;  // also the weight classes, and the sequences held in shared memory at once

struct VarPlanParams {
    const int *cu;  // [num_seqs + 1]
    int num_seqs, rows;
    int unit;      // rows of a tile
    int window;    // 0 = none
    int backward;  // weights: 0 = keys a query tile sees, 1 = queries that see a key tile
    VarItem *items;
    int *count, *next;
    int max_items;
    // backward on the tensor cores: key tiles with many query tiles are cut into parts
    // (0 = never): of about 1 / kPlanParts of a CTA's share, which is all (key tile, KV
    // head, head-dim half) items over `ctas`, and at least min_part query tiles
    int ctas, per_tile, min_part, max_slots;
    int *cut;
    // tensors whose rows behind the last sequence are set to zero (nullptr = none):
    // [rows][row_chunks * 16 bytes]
    uint4 *tail[3];
    int tail_chunks[3];
    float *tail_lse;  // [heads][rows], set to -inf there
    int heads;
};

// Exclusive prefix sum over the block's 1024 threads; `total` gets the sum.
__device__ __forceinline__ int plan_scan(int x, int &total, int *warp_sums) {
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    int s = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += y;
    }
    __syncthreads();  // the previous scan's warp_sums have been read
    if (lane == 31) warp_sums[warp] = s;
    __syncthreads();
    int w = warp_sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += y;
    }
    total = __shfl_sync(0xffffffffu, w, 31);
    const int before = __shfl_sync(0xffffffffu, w, (warp + 31) % 32);
    return (warp ? before : 0) + s - x;
}

// Block 0 writes the schedule: a counting sort of the tiles by weight class, one
// warp per sequence, one lane per tile. The other blocks clear the rows behind the
// last sequence. Lengths that do not ascend from 0 or that leave the tensors are
// reported as FORGE_ERR_INVALID_ARG, and no tile is scheduled.
__global__ void __launch_bounds__(kPlanThreads) varlen_plan(const VarPlanParams p) {
    griddep_launch_dependents();
    griddep_wait();
    if (blockIdx.x > 0) {
        const int end = min(max(p.cu[p.num_seqs], 0), p.rows);
        const size_t t0 = (size_t)(blockIdx.x - 1) * blockDim.x + threadIdx.x;
        const size_t nt = (size_t)(gridDim.x - 1) * blockDim.x;
#pragma unroll
        for (int i = 0; i < 3; i++) {
            if (p.tail[i] == nullptr) continue;
            const size_t c = (size_t)p.tail_chunks[i];
            for (size_t j = (size_t)end * c + t0; j < (size_t)p.rows * c; j += nt) p.tail[i][j] = make_uint4(0, 0, 0, 0);
        }
        const size_t left = (size_t)(p.rows - end);
        if (p.tail_lse != nullptr)
            for (size_t j = t0; j < left * p.heads; j += nt)
                p.tail_lse[(j / left) * p.rows + end + j % left] = -INFINITY;
        return;
    }
    __shared__ int cls[kPlanThreads], first[kPlanThreads], length[kPlanThreads], padded[kPlanThreads], sums[32];
    __shared__ int slots, cuts, part_tiles;
    __shared__ unsigned long long steps;
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    const int gran = max(128, (p.rows + kPlanThreads - 1) / kPlanThreads);
    const int most = p.window > 0 ? (int)min((long long)p.window + p.unit, (long long)p.rows) : p.rows;
    // query tiles that see key tile t
    auto q_tiles = [&](int len, int t) -> int {
        const int k1 = (t + 1) * p.unit - 1;
        const int last = p.window > 0 ? (int)min((long long)len - 1, (long long)k1 + p.window - 1) : len - 1;
        return last / p.unit - t + 1;
    };
    auto klass = [&](int span) -> int { return min(min(span, most) / gran, kPlanThreads - 1); };
    bool bad = tid == 0 && p.cu[0] != 0;
    cls[tid] = 0;
    if (tid == 0) {
        slots = cuts = 0;
        part_tiles = 0x7fffffff;
        steps = 0;
    }
    int total = 0;
    // pass 0 (with cutting): all query tiles; pass 1: class sizes; pass 2: the list
    for (int pass = p.ctas > 0 ? 0 : 1; pass < 3; pass++) {
        const bool loads = pass == (p.ctas > 0 ? 0 : 1) || p.num_seqs > kPlanThreads;
        int pad = 0;
        for (int c0 = 0; c0 < p.num_seqs; c0 += kPlanThreads) {
            if (loads) {
                const int b = c0 + tid;
                int s = 0, len = 0;
                if (b < p.num_seqs) {
                    s = p.cu[b];
                    const int e = p.cu[b + 1];
                    if (s >= 0 && s <= e && e <= p.rows) len = e - s;
                    else bad = true;
                }
                int sum;
                __syncthreads();  // the previous chunk has been read
                const int at = plan_scan((len + 127) / 128 * 128, sum, sums);
                first[tid] = s;
                length[tid] = len;
                padded[tid] = pad + at;
                pad += sum;
            }
            __syncthreads();
            for (int i = warp; i < min(kPlanThreads, p.num_seqs - c0); i += 32) {
                const int len = length[i];
                unsigned long long n = 0;
                for (int t = lane; t * p.unit < len; t += 32) {
                    if (pass == 0) {
                        n += q_tiles(len, t);
                        continue;
                    }
                    if (p.backward) {
                        const int nm = q_tiles(len, t);
                        int parts = nm > part_tiles ? (nm + part_tiles - 1) / part_tiles : 1, slot = 0;
                        if (pass == 2 && parts > 1) {
                            // the host's bound on the slots covers every cut
                            slot = atomicAdd(&slots, parts);
                            int *c = p.cut + 4 + 4 * atomicAdd(&cuts, 1);
                            c[0] = first[i] + t * p.unit;
                            c[1] = min(p.unit, len - t * p.unit);
                            c[2] = slot;
                            c[3] = parts;
                        }
                        for (int x = 0; x < parts; x++) {
                            // the first nm % parts parts have one query tile more
                            const int m0 = nm / parts * x + min(nm % parts, x), m1 = m0 + nm / parts + (x < nm % parts);
                            const int at = atomicAdd(&cls[klass((m1 - m0) * p.unit)], 1);
                            if (pass == 2 && at < p.max_items)
                                p.items[at] = VarItem{first[i], len, t, padded[i], m0, m1 - m0, slot + x, parts};
                        }
                    } else {
                        const int at = atomicAdd(&cls[klass(min(len, (t + 1) * p.unit))], 1);
                        if (pass == 2 && at < p.max_items) p.items[at] = VarItem{first[i], len, t, padded[i], 0, 0, 0, 1};
                    }
                }
                if (pass == 0) {
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
                    if (lane == 0) atomicAdd(&steps, n);
                }
            }
        }
        __syncthreads();
        // lengths that do not add up could overlap: nothing is scheduled then
        if (pass < 2 && __syncthreads_or(bad)) {
            if (tid == 0) {
                *p.count = *p.next = 0;
                if (p.ctas > 0) p.cut[0] = 0;
                record_status(kStatusInvalidArg);
            }
            return;
        }
        if (pass == 0) {
            if (tid == 0) {
                const unsigned long long n = (steps * p.per_tile + p.ctas * kPlanParts - 1) / (p.ctas * kPlanParts);
                part_tiles = max((int)min(n, (unsigned long long)p.rows), p.min_part);
            }
            __syncthreads();
        }
        if (pass == 1) {
            // class sizes -> first place of each class, the heaviest class first
            const int n = cls[kPlanThreads - 1 - tid];
            const int at = plan_scan(n, total, sums);
            __syncthreads();
            cls[kPlanThreads - 1 - tid] = at;
            __syncthreads();
        }
    }
    if (tid == 0) {
        *p.count = min(total, p.max_items);
        *p.next = 0;
        if (p.ctas > 0) p.cut[0] = cuts;
    }
}

// Delta_i = rowsum(dO_i * o_i) of a tile of one head (o + o_res, where the forward
// wrote o's rounding residual), and (acc != nullptr)
// the tile's rows of the padded dq accumulator set to zero. The blocks take the (item,
// head) pairs in turn, heads innermost; LPR lanes a row as in bwd_preprocess.
template <typename T, int D>
__global__ void __launch_bounds__(256) varlen_preprocess(const T *__restrict__ o, const T *__restrict__ o_res,
                                                         const T *__restrict__ dO, float *__restrict__ delta, float *__restrict__ acc, int Hq,
                                                         const VarSched var) {
    constexpr int LPR = D / 8 < 32 ? D / 8 : 32;  // lanes per row
    constexpr int RPB = 256 / LPR;                // rows per pass of the block
    constexpr int NR = sizeof(T) == 2 ? 4 : 2;
    griddep_launch_dependents();
    griddep_wait();
    const int work = var_count(var) * Hq, sub = threadIdx.x % LPR;
    for (int idx = blockIdx.x; idx < work; idx += gridDim.x) {
        const int item = idx / Hq, h = idx % Hq;
        const VarItem it = var_item_part(var, item);
        if (it.m0 > 0) continue;  // the tile comes once more as another part
        const int n = min(var.unit, it.len - it.tile * var.unit);
        const size_t row0 = (size_t)it.row0 + (size_t)it.tile * var.unit;
        float *arow0 = acc == nullptr ? nullptr : acc + ((size_t)h * var.pad_rows + it.pad0 + (size_t)it.tile * var.unit) * D;
        // NR rows a lane at once, all their loads issued before the first is used
        for (int r0 = threadIdx.x / LPR; r0 - (int)(threadIdx.x / LPR) < n; r0 += NR * RPB) {
            float sum[NR];
#pragma unroll
            for (int e = 0; e < NR; e++) sum[e] = 0.0f;
#pragma unroll
            for (int c = sub * 8; c < D; c += 8 * LPR) {
                float a[NR][8], b[NR][8], x[NR][8];
#pragma unroll
                for (int e = 0; e < NR; e++) {
                    // every lane takes part in the shuffles below; rows past the end repeat the first
                    const size_t at = ((row0 + (r0 + e * RPB < n ? r0 + e * RPB : 0)) * Hq + h) * D + c;
                    load8(o + at, a[e]);
                    load8(dO + at, b[e]);
                    if (o_res != nullptr) load8(o_res + at, x[e]);
                }
#pragma unroll
                for (int e = 0; e < NR; e++)
#pragma unroll
                    for (int i = 0; i < 8; i++) sum[e] = fmaf(o_res != nullptr ? a[e][i] + x[e][i] : a[e][i], b[e][i], sum[e]);
            }
#pragma unroll
            for (int e = 0; e < NR; e++) {
                const int r = r0 + e * RPB;
#pragma unroll
                for (int off = LPR / 2; off > 0; off >>= 1) sum[e] += __shfl_xor_sync(0xffffffffu, sum[e], off);
                if (r >= n) continue;
                if (sub == 0) delta[(size_t)h * var.rows + row0 + r] = sum[e];
                if (acc != nullptr)
#pragma unroll
                    for (int c = sub * 4; c < D; c += 4 * LPR)
                        *reinterpret_cast<float4 *>(arow0 + (size_t)r * D + c) = make_float4(0.f, 0.f, 0.f, 0.f);
            }
        }
    }
}

// The last stage of the bf16 backward: dk and dv of the key tiles that were cut, the
// parts' sums added in their order, and dq rows from the padded accumulator, 128-row
// tiles of one head. The blocks take the units of both in turn.
template <int D>
__global__ void __launch_bounds__(256) varlen_finalize(const float *__restrict__ acc, __nv_bfloat16 *__restrict__ dq,
                                                       __nv_bfloat16 *__restrict__ dk, __nv_bfloat16 *__restrict__ dv,
                                                       int Hq, int Hkv, const VarSched var) {
    constexpr int CH = D / 8;  // 8-element chunks per row
    griddep_launch_dependents();
    griddep_wait();
    {
        // units of 256 chunks: 256 / CH rows of one of (dk, dv), KV head, cut tile
        constexpr int RPU = 256 / CH, UPT = 128 / RPU;
        const int units = var.cut[0] * Hkv * 2 * UPT;
        for (int u = blockIdx.x; u < units; u += gridDim.x) {
            const int r = u % UPT * RPU + (int)threadIdx.x / CH, c = (int)threadIdx.x % CH * 8;
            const int which = u / UPT % 2, h = u / (UPT * 2) % Hkv;
            const int4 t = *reinterpret_cast<const int4 *>(var.cut + 4 + 4 * (u / (UPT * 2 * Hkv)));
            if (r >= t.y) continue;
            float sum[8] = {};
            for (int x = 0; x < t.w; x++) {
                float f[8];
                load8(var.parts + ((((size_t)(t.z + x) * Hkv + h) * 2 + which) * 128 + r) * D + c, f);
#pragma unroll
                for (int e = 0; e < 8; e++) sum[e] += f[e];
            }
            uint4 o;
            uint32_t *w = reinterpret_cast<uint32_t *>(&o);
#pragma unroll
            for (int e = 0; e < 4; e++) w[e] = pack_bf16x2(sum[2 * e], sum[2 * e + 1]);
            *reinterpret_cast<uint4 *>((which ? dv : dk) + ((size_t)(t.x + r) * Hkv + h) * D + c) = o;
        }
    }
    const int work = var_count(var) * Hq;
    for (int idx = blockIdx.x; idx < work; idx += gridDim.x) {
        const int item = idx / Hq, h = idx % Hq;
        const VarItem it = var_item_part(var, item);
        if (it.m0 > 0) continue;  // the tile comes once more as another part
        const int n = min(var.unit, it.len - it.tile * var.unit);
        const size_t row0 = (size_t)it.row0 + (size_t)it.tile * var.unit;
        const float *arow0 = acc + ((size_t)h * var.pad_rows + it.pad0 + (size_t)it.tile * var.unit) * D;
        constexpr int NC = 4;  // chunks a thread loads at once
        for (int i0 = threadIdx.x; i0 < n * CH; i0 += NC * 256) {
            float f[NC][8];
#pragma unroll
            for (int k = 0; k < NC; k++)
                if (i0 + k * 256 < n * CH) load8(arow0 + (size_t)(i0 + k * 256) * 8, f[k]);
#pragma unroll
            for (int k = 0; k < NC; k++) {
                const int i = i0 + k * 256, r = i / CH, c = i % CH;
                if (i >= n * CH) break;
                uint4 u;
                uint32_t *w = reinterpret_cast<uint32_t *>(&u);
#pragma unroll
                for (int e = 0; e < 4; e++) w[e] = pack_bf16x2(f[k][2 * e], f[k][2 * e + 1]);
                *reinterpret_cast<uint4 *>(dq + ((row0 + r) * Hq + h) * D + c * 8) = u;
            }
        }
    }
}

// dsink[h] = -sum over the rows of all sequences of exp(sink[h] - lse) * Delta. One
// block per head, in a fixed order.
__global__ void __launch_bounds__(512) varlen_sink_grad(const float *lse, const float *delta, const float *sink,
                                                        float *dsink, const int *cu, int num_seqs, int rows) {
    __shared__ float part[16];
    griddep_launch_dependents();
    griddep_wait();
    const int h = blockIdx.x, end = min(max(cu[num_seqs], 0), rows);
    const float sg = sink[h];
    float acc = 0.0f;
    for (int t = threadIdx.x; t < end; t += 512) {
        const size_t at = (size_t)h * rows + t;
        acc -= expf(sg - lse[at]) * delta[at];
    }
    acc = warp_sum(acc);
    if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = acc;
    __syncthreads();
    if (threadIdx.x == 0) {
        float sum = 0.0f;
        for (int w = 0; w < 16; w++) sum += part[w];
        dsink[h] = sum;
    }
}

}  // namespace forge
