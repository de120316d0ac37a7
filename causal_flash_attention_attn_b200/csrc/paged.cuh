// paged.cuh -- writing into a paged KV cache: new tokens appended to their sequences'
// pages, and pages copied to other pages. Both move bytes only: HBM-bound, every byte
// read once and written once in 16-byte accesses.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "sm100.cuh"

namespace forge {

constexpr int kAppendThreads = 256;
constexpr int kAppendTokens = 16;  // tokens of one block, at most

struct AppendParams {
    const uint8_t *src[2];   // K, V: [rows][Hkv][row bytes], rows src_stride bytes apart
    uint8_t *dst[2];         // pools: [num_pages][Hkv][page][row bytes], pages page_stride bytes apart
    long long src_stride[2], page_stride;
    const int *table;        // [num_seqs][width]
    const int *starts;       // [num_seqs] tokens that each sequence holds already
    const int *cu;           // [num_seqs + 1], or nullptr: token i belongs to sequence i
    int num_seqs, rows, width, page, num_pages, Hkv;
    int chunks;              // 16-byte chunks of one row of one head
    int tokens;              // tokens of one block
};

// A block first finds the place of each of its tokens (one thread a token: the
// sequence by bisection of cu, then its page), then copies their Hkv rows of K and V.
__global__ void __launch_bounds__(kAppendThreads) paged_append(const AppendParams p) {
    __shared__ long long place[kAppendTokens];  // byte offset of the token's row of head 0; -1 = none
    griddep_launch_dependents();
    griddep_wait();
    const int t0 = blockIdx.x * p.tokens, n = min(p.tokens, p.rows - t0);
    const long long head = (long long)p.page * p.chunks * 16;  // bytes between a page's heads
    if ((int)threadIdx.x < n) {
        const int t = t0 + threadIdx.x;
        int b = t, i = 0;
        bool live = t < p.num_seqs, bad = false;
        if (p.cu != nullptr) {
            // the last sequence that starts at or before t: cu[b] <= t < cu[b + 1]
            int lo = 0, hi = p.num_seqs;
            while (lo < hi) {
                const int mid = (lo + hi) / 2;
                if (p.cu[mid + 1] <= t) lo = mid + 1;
                else hi = mid;
            }
            b = lo;
            live = b < p.num_seqs;  // rows behind the last sequence go nowhere
            if (live) {
                i = t - p.cu[b];
                bad = i < 0;
            }
        }
        long long at = -1;
        if (live) {
            const long long start = p.starts[b], pos = start + i;
            bad |= start < 0 || pos >= (long long)p.width * p.page;
            if (!bad) {
                const int pg = p.table[(long long)b * p.width + pos / p.page];
                bad = (unsigned)pg >= (unsigned)p.num_pages;
                if (!bad) at = pg * p.page_stride + (pos % p.page) * p.chunks * 16;
            }
            if (bad) record_status(kStatusInvalidArg);
        }
        place[threadIdx.x] = at;
    }
    __syncthreads();
    const int per = p.Hkv * p.chunks;  // chunks of one token's K (or V)
    for (int i = threadIdx.x; i < n * per * 2; i += kAppendThreads) {
        const int t = i / (2 * per), r = i % (2 * per), kv = r / per, c = r % per;
        if (place[t] < 0) continue;
        const uint4 x = *reinterpret_cast<const uint4 *>(p.src[kv] + (long long)(t0 + t) * p.src_stride[kv] + (long long)c * 16);
        *reinterpret_cast<uint4 *>(p.dst[kv] + place[t] + (c / p.chunks) * head + (long long)(c % p.chunks) * 16) = x;
    }
}

// Page copies of one launch: the (source, destination) pairs travel as kernel
// parameters, so the host's lists need no device copy of their own and may be
// reused as soon as the call returns.
constexpr int kCopyPairs = 496;  // 4 KB of parameters
constexpr int kCopyThreads = 256, kCopyUnroll = 8;
struct CopyParams {
    uint8_t *pool[2];
    long long page_stride, layer_stride;  // bytes
    long long page_bytes;
    int pairs, splits;                    // blocks of one page
    int src[kCopyPairs], dst[kCopyPairs];
};

// Block: (split of a page, pair) x layer x {K, V}. No page of a launch is both read
// and written, and none is written twice (the host cuts the list where one would be).
__global__ void __launch_bounds__(kCopyThreads) paged_copy(const __grid_constant__ CopyParams p) {
    griddep_launch_dependents();
    griddep_wait();
    const int pair = blockIdx.x / p.splits, split = blockIdx.x % p.splits;
    uint8_t *base = p.pool[blockIdx.z] + blockIdx.y * p.layer_stride;
    const uint4 *src = reinterpret_cast<const uint4 *>(base + p.src[pair] * p.page_stride);
    uint4 *dst = reinterpret_cast<uint4 *>(base + p.dst[pair] * p.page_stride);
    const long long n = p.page_bytes / 16;
    const long long per = (long long)kCopyThreads * kCopyUnroll;
    for (long long c0 = split * per; c0 < n; c0 += p.splits * per) {
        uint4 x[kCopyUnroll];
#pragma unroll
        for (int i = 0; i < kCopyUnroll; i++) {
            const long long c = c0 + i * kCopyThreads + threadIdx.x;
            if (c < n) x[i] = src[c];
        }
#pragma unroll
        for (int i = 0; i < kCopyUnroll; i++) {
            const long long c = c0 + i * kCopyThreads + threadIdx.x;
            if (c < n) dst[c] = x[i];
        }
    }
}

}  // namespace forge
