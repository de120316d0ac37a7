// varlen_fwd.cuh -- tensor-core forward over packed sequences at head dims 64 and 128 (head
// dim 256: the VAR instance of fwd_tc_kernel).
//
// Work item: a pair of consecutive 128-row query tiles A, B of one sequence and head, from the
// schedule (varlen_plan). As in fwd2_tc_kernel a CTA streams each K/V tile once for both
// tiles, and while one tile's scores are in softmax the tensor cores work on the other tile.
// There a KV step of a tile is a chain: its softmax (one warpgroup, 2400 cycles), then P V
// and the next Q K^T behind the other tile's. The two tiles' S and O fill TMEM, so the chain
// cannot be overlapped with itself; what can be cut is the softmax. So four softmax warpgroups
// here: two share a tile's rows and split its 128 columns, 64 scores a thread, four warps on
// each SM sub-partition instead of two for the exponentials. The halves exchange only the
// row's maximum (shared memory, one barrier of 64 threads a tile) and, at the end, its sum.
// Then the products pace the tile pair, and how they are issued matters (see the MMA issuer).
// P is handed over in two chunks, the first 32 keys of both halves and the other 32, so that
// half of P V runs under the second chunk's exponentials.
// 16,384 tokens, 32 / 8 heads, D 128, window 4096, at 1965 MHz: two softmax warpgroups 775 us, four
// 764, with the products issued by an elected lane 700, with P in two chunks 687, now 689-694
// (1.03 PFLOP/s of the entries needed); back to back, at 1000 W and 1695 MHz, 786. A tile's chain is now, in cycles: row maximum 440, exchange 250,
// exponentials 1250, store and hand-off 400, products 1024, commit 400, with the tensor cores
// busy for 2048 of 3800 a pair. Forming the first chunk's exponentials before the other half's
// maximum is there, and again if it moved a row, measured slower (687 -> 728: spills).
//
// Roles (640 threads): warps 0-15 softmax (tile warp / 8, column half warp / 4 % 2, TMEM lanes
// 32 (warp % 4)..), warp 16 TMA producer, warp 17 MMA issuer and TMEM owner, warps 18-19 idle
// (they complete the fifth warpgroup). TMEM: S_A, S_B (128 columns each; the P of each column
// half overwrites that half's own scores as bf16, so neither half waits for the other to have
// read its scores), O_A, O_B (D columns each). MMA order per KV tile j:
// PV_A(j) in its two chunks, QK_A(j+1), PV_B(j), QK_B(j+1); QK_x(j+1) is committed after
// PV_x(j), so that a softmax warp that sees S_x(j+1) may rescale O_x.
//
// Rows of the next sequence that a sequence's last tiles bring along are kept out: K's by the
// causal mask (and out of the choice of the cap's tanh, see tanh_poly.cuh), V's by zeroing them in
// shared memory (the softmax warps of the last tile, before they hand its P to the MMA warp),
// O's by storing that tile row by row.
//
// SPLIT: O += P V with P as two bf16 terms (P lo beside P hi in S's columns), so that
// O, and with its residual the backward's Delta, are accurate to ~2^-17 instead of
// carrying P's rounding. dsink, an f32 gradient that is a sum of Delta over all rows, needs
// that: 1.6e-3 of its norm off without, 7e-6 with it (1000 + 700 + 333 rows).
// CAP, WIN: compiled with or without the score cap and the window, whose code beside the plain
// path costs the plain one (7 % on 8K mixed rows with both).
#pragma once

#include "fwd2_tc.cuh"
#include "tanh_poly.cuh"
#include "varlen_item.cuh"

namespace forge {

template <int D>
struct VarFwdTc {
    static constexpr int BM = 128, BN = 128;
    static constexpr int NCB = D / 64;
    static constexpr uint32_t CB = 128 * 128;  // column block of a 128-row tile
    static constexpr uint32_t TILE = NCB * CB;  // one 128 x D bf16 tile
    static constexpr int NSTAGE = 4;            // K/V ring, as in Fwd2Tc
    static constexpr int NQB = D == 64 ? 2 : 1;  // buffers of (Q_A, Q_B)
    static constexpr uint32_t CTRL = 1024;
    // after the tiles: row maxima [tile][parity][half][128] and row sums [tile][half][128]
    static constexpr uint32_t XCH = (2 * 2 * 2 + 2 * 2) * 128 * 4;
    static constexpr uint32_t SMEM = CTRL + TILE * (2 * NQB + NSTAGE) + 1024 + XCH;
    static constexpr int THREADS = 640, W_LOAD = 16, W_MMA = 17;
    // launched at 96 registers a thread; the fifth warpgroup gives back down to REG_CTRL
    static constexpr int REG_LAUNCH = 96, REG_CTRL = 64, REG_SOFTMAX = 104;
    static_assert(4 * (REG_LAUNCH - REG_CTRL) >= 16 * (REG_SOFTMAX - REG_LAUNCH), "register split");
    static constexpr uint32_t TMEM_COLS = 512;
    static constexpr uint32_t col_s(int x) { return (uint32_t)(x * 128); }
    // P of keys [16 kk, 16 kk + 16): each column half's P over its own scores (low parts 32 on)
    static constexpr uint32_t col_p(int x, int kk) { return col_s(x) + (uint32_t)(64 * (kk / 4) + 8 * (kk % 4)); }
    static constexpr uint32_t col_o(int x) { return (uint32_t)(256 + x * D); }
    static constexpr int B_Q_FULL = 0;                    // [NQB]
    static constexpr int B_Q_EMPTY = NQB;                 // [NQB] both tiles' O stores have read the buffer
    static constexpr int B_KV_FULL = 2 * NQB;             // [NSTAGE]
    static constexpr int B_KV_EMPTY = B_KV_FULL + NSTAGE;
    static constexpr int B_S_FULL = B_KV_EMPTY + NSTAGE;  // [2]
    static constexpr int B_P_FULL = B_S_FULL + 2;         // [2] eight warps
    static constexpr int B_P_HALF = B_P_FULL + 2;         // [2] the first 32 keys of each column half: eight warps
    static constexpr int B_O_FINAL = B_P_HALF + 2;        // [2]
    static constexpr int B_O_EMPTY = B_O_FINAL + 2;       // [2] O_x read out of TMEM, eight warps
    static constexpr int B_ITEM = B_O_EMPTY + 2;          // [kVarRing] the next item's number is there
    static constexpr int NBAR = B_ITEM + kVarRing;
    static constexpr uint32_t OFF_TMEM_SLOT = 512, OFF_ABORT = 516, OFF_ITEM = 528;
    static constexpr int EMU_MASK = 7;  // column pairs with (c & 7) == 7 use the FMA-pipe exp2
    static_assert(NBAR * 8 <= 512, "control block");
    static_assert(SMEM <= 232448, "shared memory");
    static_assert(256 + 2 * D <= 512, "tensor memory");
};

// Query tiles tA = 2 pr and tB = 2 pr + 1 of head bh of a sequence (heads innermost); tile A
// sees KV tiles [loA, tA], tile B [loB, tB].
struct VarFwdItem {
    int bh, bkv, tA, tB, qA0, qB0, loA, loB, lo, hi;
    int row0, T;  // the sequence's first row in the tensors and its length
    bool hasB;
};
__device__ __forceinline__ VarFwdItem varlen_fwd_item(int w, const FwdParams &p) {
    VarFwdItem I;
    const VarItem it = var_item(p.var, w / p.Hq);
    I.bh = w % p.Hq;
    I.bkv = I.bh / (p.Hq / p.Hkv);
    I.row0 = it.row0;
    I.T = it.len;
    I.tA = 2 * it.tile;
    I.tB = 2 * it.tile + 1;
    I.qA0 = I.tA * 128;
    I.qB0 = I.tB * 128;
    I.hasB = I.qB0 < it.len;
    I.loA = p.window > 0 ? max(0, I.qA0 - p.window + 1) / 128 : 0;
    I.loB = p.window > 0 ? max(0, I.qB0 - p.window + 1) / 128 : 0;
    I.lo = I.loA;
    I.hi = I.hasB ? I.tB : I.tA;
    return I;
}

// Exponentials of 32 scores with P split into two bf16 terms, P = hi + lo (lo = bf16(P -
// hi)); every exponential by MUFU (2^-22; the FMA-pipe one is within 3e-6 only).
template <bool CAP>
__device__ __forceinline__ void exp_chunk32_split(const uint32_t (&s)[32], uint64_t sl2x2, uint64_t negm2,
                                                  uint64_t (&rs)[2], uint32_t (&hi)[16], uint32_t (&lo)[16]) {
#pragma unroll
    for (int c = 0; c < 16; c++) {
        const uint64_t x2 = f2_make(__uint_as_float(s[2 * c]), __uint_as_float(s[2 * c + 1]));
        float y0, y1;
        f2_split(CAP ? f2_add(x2, negm2) : f2_fma(x2, sl2x2, negm2), y0, y1);
        const float p0 = ex2_approx(y0), p1 = ex2_approx(y1);
        rs[c & 1] = f2_add(rs[c & 1], f2_make(p0, p1));
        hi[c] = pack_bf16x2(p0, p1);
        const float2 h = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&hi[c]));
        lo[c] = pack_bf16x2(p0 - h.x, p1 - h.y);
    }
}

template <int D, bool SPLIT, bool CAP, bool WIN>
__global__ void __launch_bounds__(640, 1)
    varlen_fwd_tc(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                  const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmO, const FwdParams p) {
    using C = VarFwdTc<D>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t sbase = smem_u32(smem_raw);
    const uint32_t tiles = (sbase + C::CTRL + 1023u) & ~1023u;
    const uint32_t sQ0 = tiles;                          // NQB x (Q_A, Q_B)
    const uint32_t sKV = tiles + 2 * C::NQB * C::TILE;  // NSTAGE K/V tiles
    float *xmax = reinterpret_cast<float *>(smem_raw + (sKV - sbase) + C::NSTAGE * C::TILE);  // [2][2][2][128]
    float *xsum = xmax + 2 * 2 * 2 * 128;                                                     // [2][2][128]
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem_raw + C::OFF_ABORT);
    volatile int *sItem = reinterpret_cast<volatile int *>(smem_raw + C::OFF_ITEM);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem_raw + C::OFF_TMEM_SLOT);
    auto bar = [&](int i) -> uint32_t { return sbase + 8u * (uint32_t)i; };

    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    // the item of a pass, which the producer took; nitems or more: none left, -1: abort
    // (item_of: by one thread; item_of_warp: by a whole warp, with one answer)
    auto item_of = [&](int pass) -> int {
        if (pass == 0) return (int)blockIdx.x;
        if (!mbar_wait(bar(C::B_ITEM + pass % kVarRing), (uint32_t)((pass / kVarRing) & 1), abort_flag)) return -1;
        return sItem[pass % kVarRing];
    };
    auto item_of_warp = [&](int pass) -> int {
        if (pass == 0) return (int)blockIdx.x;
        if (!mbar_wait_warp(bar(C::B_ITEM + pass % kVarRing), (uint32_t)((pass / kVarRing) & 1), abort_flag)) return -1;
        return sItem[pass % kVarRing];
    };

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::NQB; s++) {
            mbar_init(bar(C::B_Q_FULL + s), 1);
            mbar_init(bar(C::B_Q_EMPTY + s), 2);
        }
        for (int s = 0; s < C::NSTAGE; s++) {
            mbar_init(bar(C::B_KV_FULL + s), 1);
            mbar_init(bar(C::B_KV_EMPTY + s), 1);
        }
        for (int x = 0; x < 2; x++) {
            mbar_init(bar(C::B_S_FULL + x), 1);
            mbar_init(bar(C::B_P_FULL + x), 8);
            mbar_init(bar(C::B_P_HALF + x), 8);
            mbar_init(bar(C::B_O_FINAL + x), 1);
            mbar_init(bar(C::B_O_EMPTY + x), 8);
        }
        for (int s = 0; s < kVarRing; s++) mbar_init(bar(C::B_ITEM + s), 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == C::W_LOAD && lane == 0) {
        tma_prefetch_desc(&tmQ);
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmV);
        tma_prefetch_desc(&tmO);
    }
    if (warp == C::W_MMA) {
        tmem_alloc(smem_u32(tmem_slot), C::TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    griddep_wait();  // the schedule and, behind it, q, k and v are visible
    const int nitems = var_count(p.var) * p.Hq;

    if (warp >= C::W_LOAD) {
        setmaxnreg_dec<C::REG_CTRL>();
        if (warp == C::W_LOAD) {
            // ------------------------------------------------------------ producer
            if (lane == 0) {
                const uint64_t keep = policy_evict_last();
                int issued = 0, q_issued = 0;  // ring slots and Q buffers loaded (for the abort drain)
                bool ok = true;
                mbar_arrive(bar(C::B_ITEM));  // pass 0
                for (int pass = 0; ok; pass++) {
                    const int w = item_of(pass);
                    if (w < 0) {
                        ok = false;
                        break;
                    }
                    if (w >= nitems) break;
                    const VarFwdItem I = varlen_fwd_item(w, p);
                    // the next item's number is on its way while this
                    // one's queries are loaded
                    const int next = (int)gridDim.x + atomicAdd(p.var.next, 1);
                    // the item's queries once both O stores of the item that used this
                    // buffer NQB items ago have read it
                    const int qb = pass % C::NQB;
                    if (!mbar_wait(bar(C::B_Q_EMPTY + qb), (uint32_t)(((pass / C::NQB) & 1) ^ 1), abort_flag)) {
                        ok = false;
                        break;
                    }
                    const uint32_t sQ = sQ0 + (uint32_t)qb * 2 * C::TILE;
                    mbar_arrive_expect_tx(bar(C::B_Q_FULL + qb), I.hasB ? 2 * C::TILE : C::TILE);
                    for (int c = 0; c < C::NCB; c++) {
                        tma_load_3d(sQ + c * C::CB, &tmQ, bar(C::B_Q_FULL + qb), c * 64, I.row0 + I.qA0, I.bh);
                        if (I.hasB)
                            tma_load_3d(sQ + C::TILE + c * C::CB, &tmQ, bar(C::B_Q_FULL + qb), c * 64, I.row0 + I.qB0,
                                        I.bh);
                    }
                    q_issued++;
                    sItem[(pass + 1) % kVarRing] = next;
                    mbar_arrive(bar(C::B_ITEM + (pass + 1) % kVarRing));
                    if (next >= nitems) griddep_launch_dependents();  // this CTA's last item
                    // ring slots in order K(lo), V(lo), K(lo+1), V(lo+1), ...
                    for (int j = I.lo; ok && j <= I.hi; j++) {
                        for (int kv = 0; kv < 2 && ok; kv++) {
                            const int st = issued % C::NSTAGE;
                            const uint32_t ph = (uint32_t)((issued / C::NSTAGE) & 1);
                            if (!mbar_wait(bar(C::B_KV_EMPTY + st), ph ^ 1u, abort_flag)) {
                                ok = false;
                                break;
                            }
                            mbar_arrive_expect_tx(bar(C::B_KV_FULL + st), C::TILE);
                            for (int c = 0; c < C::NCB; c++)
                                tma_load_3d_hint(sKV + st * C::TILE + c * C::CB, kv ? &tmV : &tmK,
                                                 bar(C::B_KV_FULL + st), c * 64, I.row0 + j * C::BN, I.bkv, keep);
                            issued++;
                        }
                    }
                }
                if (!ok) {
                    for (int back = 1; back <= min(q_issued, C::NQB); back++) {
                        const int L = q_issued - back;
                        mbar_wait_drain(bar(C::B_Q_FULL + L % C::NQB), (uint32_t)((L / C::NQB) & 1), 200000000ull);
                    }
                    for (int back = 1; back <= min(issued, C::NSTAGE); back++) {
                        const int L = issued - back;
                        mbar_wait_drain(bar(C::B_KV_FULL + L % C::NSTAGE), (uint32_t)((L / C::NSTAGE) & 1), 200000000ull);
                    }
                }
            }
        } else if (warp == C::W_MMA) {
            // ---------------------------------------------------------- MMA issuer
            // The whole warp walks the schedule and one elected lane issues, so that addresses
            // and descriptors are known to be equal across the warp. Inside a branch that only
            // lane 0 enters they are not, and issuing a 128 x 128 x 16 product took 90-110
            // cycles against the 64 that it computes (16K windowed prompt 793 -> 707 us, 8K
            // mixed rows 194 -> 174 us).
            {
                const bool lead = elect_one();
                const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
                constexpr uint32_t ID_QK = idesc_bf16_f32(128, 128, false, false);
                constexpr uint32_t ID_PV = idesc_bf16_f32(128, D, false, true);
                auto wait_full = [&](int slot) -> bool {
                    return mbar_wait_warp(bar(C::B_KV_FULL + slot % C::NSTAGE), (uint32_t)((slot / C::NSTAGE) & 1), abort_flag);
                };
                auto release = [&](int slot) {
                    if (lead) tc_commit(bar(C::B_KV_EMPTY + slot % C::NSTAGE));
                };
                int slot0 = 0;          // ring slot of the current item's K(lo)
                int cnt0 = 0, cnt1 = 0;  // PVs issued per tile over the whole run (P_FULL phases)
                bool ok = true;
                int pass = 0;
                for (; ok; pass++) {
                    const int w = item_of_warp(pass);
                    if (w < 0) {
                        ok = false;
                        break;
                    }
                    if (w >= nitems) break;
                    const VarFwdItem I = varlen_fwd_item(w, p);
                    const int qb = pass % C::NQB;
                    const uint32_t sQ = sQ0 + (uint32_t)qb * 2 * C::TILE;
                    // KV range of each tile ([lo_x, hi_x]; empty for a missing tile B)
                    const int lo0 = I.loA, hi0 = I.tA, lo1 = I.loB, hi1 = I.hasB ? I.tB : -1;
                    auto issue_qk = [&](int x, int slot) {
                        const uint64_t dq = sdesc_sw128(sQ + (uint32_t)x * C::TILE, 16, 1024);
                        const uint64_t dk = sdesc_sw128(sKV + (uint32_t)(slot % C::NSTAGE) * C::TILE, 16, 1024);
                        if (lead) {
#pragma unroll
                            for (int kk = 0; kk < D / 16; kk++) {
                                const uint32_t off = (kk >> 2) * C::CB + (kk & 3) * 32;
                                mma_ss(tm + C::col_s(x), sdesc_step(dq, off), sdesc_step(dk, off), ID_QK, kk > 0);
                            }
                            tc_commit(bar(C::B_S_FULL + x));
                        }
                        __syncwarp();
                    };
                    // P V over the keys of chunk c (0 or 1) of both column halves
                    auto issue_pv = [&](int x, int slot, int c, bool acc) {
                        const uint64_t dv = sdesc_sw128(sKV + (uint32_t)(slot % C::NSTAGE) * C::TILE, C::CB, 1024);
                        if (lead) {
#pragma unroll
                            for (int i = 0; i < 4; i++) {
                                const int kk = (i >> 1) * 4 + 2 * c + (i & 1);
                                mma_ts(tm + C::col_o(x), tm + C::col_p(x, kk), sdesc_step(dv, kk * 2048), ID_PV,
                                       (acc || c > 0 || i > 0) ? 1u : 0u);
                            }
                            if (SPLIT && c == 1) {
#pragma unroll
                                for (int kk = 0; kk < C::BN / 16; kk++)
                                    mma_ts(tm + C::col_o(x), tm + C::col_p(x, kk) + 32, sdesc_step(dv, kk * 2048), ID_PV,
                                           1u);
                            }
                        }
                        __syncwarp();
                    };
                    if (!(ok = mbar_wait_warp(bar(C::B_Q_FULL + qb), (uint32_t)((pass / C::NQB) & 1), abort_flag))) break;
                    if (!(ok = wait_full(slot0))) break;
                    tc_fence_after();
                    if (I.lo >= lo0 && I.lo <= hi0) issue_qk(0, slot0);
                    if (I.lo >= lo1 && I.lo <= hi1) issue_qk(1, slot0);
                    release(slot0);
                    bool first0 = true, first1 = true;
                    for (int j = I.lo; ok && j <= I.hi; j++) {
                        const int slotV = slot0 + 2 * (j - I.lo) + 1, slotK = slotV + 1;
                        if (!(ok = wait_full(slotV))) break;
                        bool k_ready = false;
#pragma unroll
                        for (int x = 0; x < 2; x++) {
                            const int lox = x ? lo1 : lo0, hix = x ? hi1 : hi0;
                            bool &first = x ? first1 : first0;
                            int &cx = x ? cnt1 : cnt0;
                            if (ok && j >= lox && j <= hix) {
                                if (!(ok = mbar_wait_warp(bar(C::B_P_HALF + x), (uint32_t)(cx & 1), abort_flag))) break;
                                tc_fence_after();
                                // the first PV of an item overwrites O_x: the previous
                                // item's O_x must have been read out
                                if (first && pass > 0) {
                                    if (!(ok = mbar_wait_warp(bar(C::B_O_EMPTY + x), (uint32_t)((pass - 1) & 1), abort_flag)))
                                        break;
                                    tc_fence_after();
                                }
                                issue_pv(x, slotV, 0, !first);
                                if (!(ok = mbar_wait_warp(bar(C::B_P_FULL + x), (uint32_t)(cx & 1), abort_flag))) break;
                                tc_fence_after();
                                issue_pv(x, slotV, 1, true);
                                first = false;
                                cx++;
                            }
                            if (ok && j < I.hi && j + 1 >= lox && j + 1 <= hix) {
                                if (!k_ready) {
                                    if (!(ok = wait_full(slotK))) break;
                                    tc_fence_after();
                                    k_ready = true;
                                }
                                issue_qk(x, slotK);
                            }
                        }
                        if (!ok) break;
                        release(slotV);
                        if (j < I.hi) release(slotK);
                    }
                    if (!ok) break;
                    slot0 += 2 * (I.hi - I.lo + 1);
                    // Every O_FINAL phase of a tile comes behind its O_EMPTY of the item before, as the
                    // first PV sees to where there is one: else tile B's warps, which have nothing
                    // to do in a run of items without a tile B, could fall two phases behind, and a
                    // wait by parity would not see the phase that it waits for.
                    if (!I.hasB && pass > 0 &&
                        !(ok = mbar_wait_warp(bar(C::B_O_EMPTY + 1), (uint32_t)((pass - 1) & 1), abort_flag)))
                        break;
                    // O_FINAL fires once every MMA of the item (and before) has completed
                    if (lead) {
                        tc_commit(bar(C::B_O_FINAL + 0));
                        tc_commit(bar(C::B_O_FINAL + 1));
                    }
                }
                if (!ok && lead) {
                    tc_commit(bar(C::B_O_FINAL + 0));
                    mbar_wait_drain(bar(C::B_O_FINAL + 0), (uint32_t)(pass & 1), 200000000ull);
                }
            }
        }
    } else {
        setmaxnreg_inc<C::REG_SOFTMAX>();
        // ------------------------------------------------------------ softmax
        const int x = warp / 8, hf = (warp / 4) % 2;  // tile, column half
        const int row = threadIdx.x % 128, t = threadIdx.x % 256;
        const uint32_t lane_base = (uint32_t)((warp % 4) * 32) << 16;
        const uint32_t tS = tmem + lane_base + C::col_s(x) + 64 * (uint32_t)hf;  // this half's scores
        const uint32_t tO = tmem + lane_base + C::col_o(x);
        const uint32_t pair_bar = 1 + (uint32_t)(x * 4 + warp % 4);  // the two warps of these rows
        const uint32_t tile_bar = 9 + (uint32_t)x;                   // the tile's eight warps
        const uint64_t sl2x2 = f2_make(p.scale_log2, p.scale_log2);
        int cnt = 0;    // KV tiles of this tile slot over the whole run (S_FULL phases)
        int slot0 = 0;  // ring slot of the current item's K(lo)
        // The warps of a tile go through the same items and leave together: a wait that ran
        // out for one of them travels in `ok` to the pair's barriers and from there to the
        // tile's, which ends every item.
        for (int pass = 0, w = (int)blockIdx.x; w < nitems; pass++, w = sItem[pass % kVarRing]) {
            const VarFwdItem I = varlen_fwd_item(w, p);
            const int qb = pass % C::NQB;
            const bool has = (x == 0) || I.hasB;
            bool ok = true;
            // a window that hides nothing is none
            const int W = !WIN || p.window >= I.T ? 0 : p.window;
            const int q0 = x ? I.qB0 : I.qA0;
            const int lox = x ? I.loB : I.loA, hix = x ? I.tB : I.tA;
            const int qi = q0 + row;
            const int r0 = q0 + 32 * (warp % 4);
            float m = p.sink ? p.sink[I.bh] * kLog2e : -INFINITY;
            float l = p.sink && hf == 0 ? 1.0f : 0.0f;  // the sink's 1 counts once
            for (int j = lox; has && j <= hix; j++, cnt++) {
                const int k0 = j * C::BN + 64 * hf;  // first key of this half
                if (!mbar_wait_warp(bar(C::B_S_FULL + x), (uint32_t)(cnt & 1), abort_flag)) {
                    ok = named_barrier_all(pair_bar, 64, false);
                    break;
                }
                tc_fence_after();
                // classes of the two 32-key chunks for this warp's 32 rows (warp-uniform):
                // bit q of `dead` = no key of chunk q is visible to any of the rows, bit q
                // of `part` = some are
                unsigned dead = 0, part = 0;
                if (k0 + 63 > r0 || (WIN && W > 0 && k0 <= r0 + 31 - W)) {
#pragma unroll
                    for (int q2 = 0; q2 < 2; q2++) {
                        const int c0 = k0 + 32 * q2;
                        const bool all_vis = (c0 + 31 <= r0) && (W == 0 || c0 > r0 + 31 - W);
                        const bool none = (c0 > r0 + 31) || (W > 0 && c0 + 31 <= r0 - W);
                        dead |= (unsigned)none << q2;
                        part |= (unsigned)(!all_vis && !none) << q2;
                    }
                }
                // scores of chunk q2 as the softmax sees them
                auto finish = [&](uint32_t(&s)[32], int q2) {
                    uint32_t vm = ~0u;
                    if (dead | part) {
                        // bit c of vm: key k0 + 32 q2 + c is visible to row qi, i.e. lo_c < c <= hi_c
                        const int hi_c = qi - (k0 + 32 * q2);
                        vm = hi_c < 0 ? 0u : (hi_c >= 31 ? ~0u : (~0u >> (31 - hi_c)));
                        if (W > 0) {
                            const int lo_c = hi_c - W;
                            vm &= lo_c < 0 ? ~0u : (lo_c >= 31 ? 0u : (~0u << (lo_c + 1)));
                        }
                    }
                    if constexpr (CAP) {
                        // the warp's scores choose the tanh's form together: masked ones and
                        // those of rows past the end, which may hold another sequence's values,
                        // have no say in it
                        if (dead | part) {
#pragma unroll
                            for (int c = 0; c < 32; c++)
                                if (!((vm >> c) & 1u)) s[c] = 0u;
                        }
                        cap_scores(s, p.cap_in, p.cap_out, qi < I.T);
                    }
                    if (dead | part) {
#pragma unroll
                        for (int c = 0; c < 32; c++)
                            if (!((vm >> c) & 1u)) s[c] = __float_as_uint(-INFINITY);
                    }
                };
                float best;
                {
                    uint32_t s[2][32];
                    tmem_ld32(tS, s[0]);
                    tmem_ld32(tS + 32, s[1]);
                    tmem_ld_wait(s[0]);
                    tmem_ld_wait(s[1]);
                    finish(s[0], 0);
                    finish(s[1], 1);
                    float mx[4];
#pragma unroll
                    for (int i = 0; i < 4; i++)
                        mx[i] = fmaxf(__uint_as_float(s[0][2 * i]), __uint_as_float(s[0][2 * i + 1]));
#pragma unroll
                    for (int c = 8; c < 64; c += 8)
#pragma unroll
                        for (int i = 0; i < 4; i++) {
                            const int a = c + 2 * i;
                            mx[i] = fmax3(mx[i], __uint_as_float(s[a >> 5][a & 31]), __uint_as_float(s[a >> 5][(a & 31) + 1]));
                        }
                    best = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                }
                // the row's maximum over both halves. A slot is written again two tiles on,
                // behind the next barrier.
                float *xm = xmax + (x * 2 + (cnt & 1)) * 256 + row;
                xm[128 * hf] = best;
                if (!(ok = named_barrier_all(pair_bar, 64, true))) break;
                best = fmaxf(best, xm[128 * (hf ^ 1)]);
                if constexpr (!CAP) best *= p.scale_log2;
                const float m_new = (best > m + 8.0f) ? best : m;
                const bool moved = (m_new != m);
                const float factor = moved ? ex2_approx(m - m_new) : 1.0f;
                const bool later = j > lox;  // O_x holds PVs of this item
                if (__any_sync(0xffffffffu, moved && later)) {
                    // O_x already holds every PV of this tile's earlier KV tiles; this half's columns
                    const float f = (moved && later) ? factor : 1.0f;
                    const uint64_t f2 = f2_make(f, f);
#pragma unroll 1
                    for (int c0 = hf * (D / 2); c0 < (hf + 1) * (D / 2); c0 += 32) {
                        uint32_t o[32];
                        tmem_ld32(tO + c0, o);
                        tmem_ld_wait(o);
#pragma unroll
                        for (int i = 0; i < 32; i += 2) {
                            float a, bb;
                            f2_split(f2_mul(f2_make(__uint_as_float(o[i]), __uint_as_float(o[i + 1])), f2), a, bb);
                            o[i] = __float_as_uint(a);
                            o[i + 1] = __float_as_uint(bb);
                        }
                        tmem_st32(tO + c0, o);
                    }
                }
                m = m_new;
                const float msub = (m == -INFINITY) ? 0.0f : m;
                const uint64_t negm2 = f2_make(-msub, -msub);
                uint64_t rs[2] = {f2_make(0.0f, 0.0f), f2_make(0.0f, 0.0f)};
                // the sequence's last V tile: its rows past the end become zeros. Only this
                // tile slot (the pair's last tile) reads it, and it is not released before
                // the PV that waits for these warps.
                const int end = I.T - j * C::BN;
                if (end < C::BN) {
                    const int slotV = slot0 + 2 * (j - I.lo) + 1;
                    if (!mbar_wait_warp(bar(C::B_KV_FULL + slotV % C::NSTAGE), (uint32_t)((slotV / C::NSTAGE) & 1),
                                        abort_flag)) {
                        // (behind the last tile the pair's next barrier is the one below)
                        ok = j < hix && named_barrier_all(pair_bar, 64, false);
                        break;
                    }
                    zero_tail_rows<128, C::NCB, 256>(sKV + (uint32_t)(slotV % C::NSTAGE) * C::TILE, C::CB, end, t);
                    fence_proxy_async_smem();
                }
                // The scores again from TMEM, chunk by chunk (64 held over the exchange would
                // not fit the registers). Masked scores are -inf and need the MUFU exp2 (the
                // FMA-pipe one is only valid for finite arguments); chunks no row sees are 0.
                uint32_t lo16[16];
#pragma unroll
                for (int q2 = 0; q2 < 2; q2++) {
                    uint32_t s[32], pk[16];
                    tmem_ld32(tS + 32 * q2, s);
                    tmem_ld_wait(s);
                    finish(s, q2);
                    // chunk 0's low parts go over chunk 1's scores, just read
                    if (SPLIT && q2 == 1) tmem_st16(tS + 32, lo16);
                    if constexpr (SPLIT) {
                        exp_chunk32_split<CAP>(s, sl2x2, negm2, rs, pk, lo16);
                        if (q2 == 1) tmem_st16(tS + 48, lo16);
                    } else if (dead | part) {
                        if ((dead >> q2) & 1u) {
#pragma unroll
                            for (int c = 0; c < 16; c++) pk[c] = 0u;
                        } else {
                            exp_chunk32<CAP, false, C::EMU_MASK>(s, sl2x2, negm2, rs, pk);
                        }
                    } else {
                        exp_chunk32<CAP, true, C::EMU_MASK>(s, sl2x2, negm2, rs, pk);
                    }
                    tmem_st16(tS + 16 * q2, pk);
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar((q2 ? C::B_P_FULL : C::B_P_HALF) + x));
                }
                float a0, a1, a2, a3;
                f2_split(rs[0], a0, a1);
                f2_split(rs[1], a2, a3);
                l = l * factor + ((a0 + a1) + (a2 + a3));
            }
            // (the next item's number, read by the loop's step, was published behind this one's queries)
            ok = ok && item_of_warp(pass + 1) >= 0 &&
                 mbar_wait_warp(bar(C::B_O_FINAL + x), (uint32_t)(pass & 1), abort_flag);
            tc_fence_after();
            // Stage this tile's O (bf16) in its Q buffer, which every MMA of the item has
            // finished reading once O_FINAL fired, in the 128-byte-swizzled layout of the O
            // tensor map, then store it with TMA.
            const uint32_t sO = sQ0 + (uint32_t)qb * 2 * C::TILE + (uint32_t)x * C::TILE;
            if (has) {
                xsum[(x * 2 + hf) * 128 + row] = l;
                ok = named_barrier_all(pair_bar, 64, ok);
                l += xsum[(x * 2 + (hf ^ 1)) * 128 + row];
                const float inv_l = 1.0f / l;
                const uint64_t inv2 = f2_make(inv_l, inv_l);
#pragma unroll 1
                for (int c0 = hf * (D / 2); c0 < (hf + 1) * (D / 2); c0 += 32) {
                    uint32_t o[32];
                    tmem_ld32(tO + c0, o);
                    tmem_ld_wait(o);
                    uint32_t w16[16];
                    if (p.o_res != nullptr) {
                        uint32_t lo16[16];
                        o_pairs32(o, inv_l, w16, lo16);
                        if (qi < I.T) {
                            __nv_bfloat16 *dst = p.o_res + ((size_t)(I.row0 + qi) * p.Hq + I.bh) * D + c0;
                            st_global_v8(dst, lo16);
                            st_global_v8(dst + 16, lo16 + 8);
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 16; i++) {
                            float a, bb;
                            f2_split(f2_mul(f2_make(__uint_as_float(o[2 * i]), __uint_as_float(o[2 * i + 1])), inv2), a,
                                     bb);
                            w16[i] = pack_bf16x2(a, bb);
                        }
                    }
                    const uint32_t rowaddr = sO + (uint32_t)(c0 / 64) * C::CB + (uint32_t)row * 128u;
                    const uint32_t ch0 = (uint32_t)((c0 % 64) / 8);
#pragma unroll
                    for (int i = 0; i < 4; i++)
                        st_shared_v4(rowaddr + ((((ch0 + i) ^ (uint32_t)(row & 7))) << 4), w16[4 * i], w16[4 * i + 1],
                                     w16[4 * i + 2], w16[4 * i + 3]);
                }
            }
            // O_x is in registers / shared memory: the next item's PVs may overwrite it
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(C::B_O_EMPTY + x));
            if (has) fence_proxy_async_smem();
            if (!named_barrier_all(tile_bar, 256, ok)) break;
            if (has) {
                if (q0 + C::BM > I.T) {
                    // a box would write into the next sequence: the rows up to the end,
                    // D / 8 chunks of 16 bytes each, one chunk a thread at a time
                    for (int i = t; i < (I.T - q0) * (D / 8); i += 256) {
                        const int r = i / (D / 8), ch = i % (D / 8);
                        uint4 w4;
                        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                                     : "=r"(w4.x), "=r"(w4.y), "=r"(w4.z), "=r"(w4.w)
                                     : "r"(sO + (uint32_t)(ch / 8) * C::CB + (uint32_t)r * 128u +
                                           (((uint32_t)(ch % 8) ^ (uint32_t)(r & 7)) << 4)));
                        *reinterpret_cast<uint4 *>(p.o + ((size_t)(I.row0 + q0 + r) * p.Hq + I.bh) * D + ch * 8) = w4;
                    }
                    named_barrier_sync(tile_bar, 256);  // the buffer is read before it is released below
                } else if (t == 0) {
                    for (int cb = 0; cb < C::NCB; cb++)
                        tma_store_3d(&tmO, sO + cb * C::CB, cb * 64, I.row0 + q0, I.bh);
                    bulk_commit();
                    bulk_wait_read<0>();
                }
                if (hf == 0 && qi < I.T) p.lse[(size_t)I.bh * p.var.rows + I.row0 + qi] = (m + __log2f(l)) * kLn2;
            }
            // the Q buffer is free for the item NQB ahead once both tiles' stores read it
            if (t == 0) mbar_arrive(bar(C::B_Q_EMPTY + qb));
            slot0 += 2 * (I.hi - I.lo + 1);
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == C::W_MMA) {
        tc_fence_after();
        tmem_dealloc(tmem, C::TMEM_COLS);
    }
}

}  // namespace forge
