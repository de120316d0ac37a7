// paged.cuh -- writing into a paged KV cache: new tokens appended to their sequences'
// pages, and pages copied to other pages. Both move bytes only: HBM-bound, every byte
// read once and written once in 16-byte accesses.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "sm100.cuh"

namespace forge {

constexpr int kAppendThreads = 256;
constexpr int kAppendTokens = 4;  // tokens of one block, at most
constexpr int kAppendUnroll = 4;

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

// A token has 2 Hkv rows (K's heads, then V's) of `chunks` 16-byte chunks. A thread keeps
// its chunk of its row over the block's tokens (tokens smaller than the block are taken
// several at a time), so that a copy needs no division. It loads its first kAppendUnroll
// tokens' chunks at once; while they are on their way the block finds where its tokens
// go, one thread a token: the sequence by bisection of cu, then its page, a chain of
// dependent loads as long as the copy itself. 16384 tokens of 8 heads of 128 in bf16 (134 MB
// moved): 23.8 us, 86 % of the measured copy rate; places first, then copies took 35 us,
// eight tokens a block 24.6-26.4.
__global__ void __launch_bounds__(kAppendThreads, 6) paged_append(const __grid_constant__ AppendParams p) {
    __shared__ long long place[kAppendTokens];  // byte offset of the token's row of head 0; -1 = none
    griddep_launch_dependents();
    griddep_wait();
    const int t0 = blockIdx.x * p.tokens, n = min(p.tokens, p.rows - t0);
    if (n <= 0) {
        // a block of its own (cu != nullptr) looks all lengths over: they have to ascend from 0 and
        // not pass `rows`, or tokens would be left out or taken for another sequence's
        for (int b = threadIdx.x; b <= p.num_seqs; b += kAppendThreads) {
            const int at = p.cu[b], next = b < p.num_seqs ? p.cu[b + 1] : p.rows;
            if (at > next || (b == 0 && at != 0)) record_status(kStatusInvalidArg);
        }
        return;
    }
    const long long head = (long long)p.page * p.chunks * 16;  // bytes between a page's heads
    const int per = 2 * p.Hkv * p.chunks, side = max(1, kAppendThreads / per);
    const int t1 = (int)threadIdx.x / per;  // which of the tokens side by side
    int i = t1 < side ? (int)threadIdx.x % per : per, t = t1;
    const uint8_t *src = nullptr;
    uint8_t *dst = nullptr;
    long long step = 0;
    auto row = [&]() {  // this thread's chunk i of a token
        if (i >= per) return;
        const bool v = i >= per / 2;
        const int h = (v ? i - per / 2 : i) / p.chunks, c = i % p.chunks;
        step = v ? p.src_stride[1] : p.src_stride[0];
        src = (v ? p.src[1] : p.src[0]) + t0 * step + ((long long)h * p.chunks + c) * 16;
        dst = (v ? p.dst[1] : p.dst[0]) + h * head + (long long)c * 16;
    };
    uint4 x[kAppendUnroll];
    auto load = [&]() {
#pragma unroll
        for (int e = 0; e < kAppendUnroll; e++)
            if (i < per && t + e * side < n) x[e] = *reinterpret_cast<const uint4 *>(src + (t + e * side) * step);
    };
    row();
    load();
    if ((int)threadIdx.x < n) {
        const int tok = t0 + threadIdx.x;
        int b = tok, first = tok;
        bool live = tok < p.num_seqs;
        if (p.cu != nullptr) {
            // the last sequence that starts at or before the token: cu[b] <= tok < cu[b + 1]
            int lo = 0, hi = p.num_seqs;
            while (lo < hi) {
                const int mid = (lo + hi) / 2;
                if (p.cu[mid + 1] <= tok) lo = mid + 1;
                else hi = mid;
            }
            b = lo;
            live = b < p.num_seqs;  // rows behind the last sequence go nowhere
            if (live) first = p.cu[b];
        }
        long long at = -1;
        if (live) {
            const long long start = p.starts[b], pos = start + tok - first;
            bool bad = tok < first || start < 0 || pos >= (long long)p.width * p.page;
            if (!bad) {
                const int pg = p.table[(long long)b * p.width + (int)pos / p.page];
                bad = (unsigned)pg >= (unsigned)p.num_pages;
                if (!bad) at = pg * p.page_stride + ((int)pos % p.page) * p.chunks * 16;
            }
            if (bad) record_status(kStatusInvalidArg);
        }
        place[threadIdx.x] = at;
    }
    __syncthreads();
    while (i < per) {
#pragma unroll
        for (int e = 0; e < kAppendUnroll; e++) {
            const int u = t + e * side;
            if (u < n && place[u] >= 0) *reinterpret_cast<uint4 *>(dst + place[u]) = x[e];
        }
        t += side * kAppendUnroll;
        if (t >= n) {
            t = t1;
            i += kAppendThreads;
            row();
        }
        load();
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
