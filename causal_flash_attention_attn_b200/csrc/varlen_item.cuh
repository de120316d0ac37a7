// varlen_item.cuh -- one tile of a packed batch, as the kernels for packed
// sequences read it from the schedule that varlen_plan (varlen.cuh) writes.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace forge {

// One lane of a converged warp, always the same.
__device__ __forceinline__ bool elect_one() {
    uint32_t x;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(x));
    return x != 0;
}

struct alignas(16) VarItem {
    int row0;  // first row of the sequence in the packed tensors
    int len;   // rows of the sequence
    int tile;  // tile index within the sequence
    int pad0;  // first row of the sequence in tensors whose sequences are padded to 128 rows
    // backward: this item walks the query tiles m0 .. m0 + nm - 1 (of 128 rows, counted from
    // the key tile's own), and is one of `parts` that share the key tile: part
    // number `slot` of the partial sums if parts > 1
    int m0, nm, slot, parts;
};

// The schedule of one call, in device memory. Both are written by an earlier
// kernel of the same stream, so they are read with plain (not read-only-cache)
// loads, after griddep_wait.
struct VarSched {
    const VarItem *items;
    const int *count;  // tiles in `items`
    int *next;         // items handed out so far (var_next), set to 0 by the schedule's kernel
    float *parts;      // backward: partial [slot][Hkv][dk, dv][128][D] of key tiles cut into parts
    int max_items, max_slots;
    const int *cut;        // [0]: key tiles cut; then 4 ints each: row0 + first key, keys, first slot, parts
    int unit;          // rows of a tile
    int rows;          // rows of the packed tensors
    int pad_rows;      // rows of the padded tensors (an upper bound)
};

__device__ __forceinline__ VarItem var_item(const VarSched &v, int i) {
    VarItem t;
    asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(t.row0), "=r"(t.len), "=r"(t.tile), "=r"(t.pad0)
                 : "l"(v.items + i)
                 : "memory");
    return t;  // m0 .. parts are read by var_item_part
}
__device__ __forceinline__ VarItem var_item_part(const VarSched &v, int i) {
    VarItem t = var_item(v, i);
    asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(t.m0), "=r"(t.nm), "=r"(t.slot), "=r"(t.parts)
                 : "l"(&v.items[i].m0)
                 : "memory");
    return t;
}

// Work items handed out one at a time in the schedule's order, heaviest first: a CTA
// that gets done early takes more (a fixed order would leave it idle: the lengths are
// not known at launch). The first item is the CTA's own number; while it loads an item,
// one thread takes the next one's number and publishes it in a ring of kVarRing shared
// words, each with a barrier on which every role waits (pass p >= 1: word and barrier
// p % kVarRing, phase (p / kVarRing) & 1, the barriers of pass 0 completed at the start).
// No role releases a word. The thread publishes pass p + 1 when it has issued the first
// loads of pass p, for which the buffers of pass p - 2 (or p - 1) must have been freed. By
// then the products of pass p - 2 are done, and with them every role has finished pass p - 3:
// in the backward each step waits for all of its warps; in the forward the last commit of
// a pass (O_FINAL) waits until all warps of both tiles have left the pass before it
// (O_EMPTY), whether or not the pass has a tile B. So the word to be written, last used for
// pass p + 1 - kVarRing = p - 7, has been read.
constexpr int kVarRing = 8;
__device__ __forceinline__ int var_count(const VarSched &v) {
    int n;
    asm volatile("ld.global.b32 %0, [%1];" : "=r"(n) : "l"(v.count) : "memory");
    return n;
}

// 32 bytes, one whole sector, to global memory (32-byte aligned). Where each lane
// writes a row of its own, the store unit takes one cycle per lane and instruction, so
// that half as many instructions of twice the width take half the time.
__device__ __forceinline__ void st_global_v8(void *at, const uint32_t *w) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(at), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

// Rows [valid, ROWS) of a tile of NCB swizzled column blocks (128 bytes a row, `cb`
// bytes a block) set to zero by NT threads, t = 0 .. NT - 1. A TMA box that runs past a sequence's
// end brings rows of the next sequence: they are replaced by the zeros that a
// box past the tensor's end would have brought, so that a product summed over
// the tile's rows never multiplies them (zero times an infinity is NaN). Zeros
// are the same under the swizzle, which permutes the 16-byte chunks of a row.
template <int ROWS, int NCB, int NT>
__device__ __forceinline__ void zero_tail_rows(uint32_t tile, uint32_t cb, int valid, int t) {
    for (int r = valid + t / 8; r < ROWS; r += NT / 8) {
#pragma unroll
        for (int c = 0; c < NCB; c++)
            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(tile + c * cb + (uint32_t)r * 128u +
                                                                         (uint32_t)(t % 8) * 16u),
                         "r"(0)
                         : "memory");
    }
}

}  // namespace forge
