// tanh_poly.cuh -- the score cap's tanh on the FMA pipe, for the packed kernels.
//
// tanh_via_ex2 takes an exponential and a reciprocal, so that a capped score costs the
// MUFU unit (16 results a cycle and SM) three operations and the softmax is bound by it. Scores
// are mostly far below the cap (|s / cap| < 0.4 for scores of standard deviation 4 and a cap of
// 50): for |y| <= 3/4, tanh(y) = y P(y^2) with P of degree 5, minimax in relative error
// (Remez exchange; coefficients and their f32 error, 1.6e-7, from gen_tanh_poly.py), nine packed
// f32x2 operations a pair. A warp takes it for a group of scores when none of its lanes
// has one beyond 3/4, and tanh_via_ex2 for the whole group otherwise. Scores that may belong to
// another sequence are kept out of that choice, so that its values never reach a result: the
// callers set masked ones to 0, and lanes whose row lies past the sequence's end have no vote (what
// comes out of a score beyond the limit there is not used).
#pragma once

#include "sm100.cuh"

namespace forge {

constexpr float kTanhPolyLimit = 0.75f;

// tanh of the pair y2, both within the limit
__device__ __forceinline__ uint64_t tanh_poly2(uint64_t y2) {
    const uint64_t u = f2_mul(y2, y2);
    uint64_t p = f2_fma(u, f2_make(-4.716257099e-03f, -4.716257099e-03f), f2_make(1.958290860e-02f, 1.958290860e-02f));
    p = f2_fma(p, u, f2_make(-5.334442854e-02f, -5.334442854e-02f));
    p = f2_fma(p, u, f2_make(1.332540661e-01f, 1.332540661e-01f));
    p = f2_fma(p, u, f2_make(-3.333295882e-01f, -3.333295882e-01f));
    p = f2_fma(p, u, f2_make(1.0f, 1.0f));
    return f2_mul(p, y2);
}

// Whether the N raw scores of every lane with a vote, times `in` (positive), are within the
// limit. A NaN does not count: it comes out as NaN either way.
template <int N>
__device__ __forceinline__ bool tanh_poly_fits(const uint32_t (&s)[N], float in, bool votes = true) {
    float m = 0.0f;
#pragma unroll
    for (int c = 0; c < N; c += 2) m = fmax3(m, fabsf(__uint_as_float(s[c])), fabsf(__uint_as_float(s[c + 1])));
    return __all_sync(0xffffffffu, m * in <= kTanhPolyLimit || !votes);
}

// s = out * tanh(in * s) for N raw scores
template <int N>
__device__ __forceinline__ void cap_scores(uint32_t (&s)[N], float in, float out, bool votes) {
    if (tanh_poly_fits<N>(s, in, votes)) {
        const uint64_t in2 = f2_make(in, in), out2 = f2_make(out, out);
#pragma unroll
        for (int c = 0; c < N; c += 2) {
            const uint64_t t = tanh_poly2(f2_mul(f2_make(__uint_as_float(s[c]), __uint_as_float(s[c + 1])), in2));
            float a, b;
            f2_split(f2_mul(t, out2), a, b);
            s[c] = __float_as_uint(a);
            s[c + 1] = __float_as_uint(b);
        }
    } else {
#pragma unroll
        for (int c = 0; c < N; c++) s[c] = __float_as_uint(out * tanh_via_ex2(__uint_as_float(s[c]) * in));
    }
}

}  // namespace forge
