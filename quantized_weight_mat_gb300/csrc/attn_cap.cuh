// The cap of pq_attn_mod's scores, for the kernels and for a test on the host.
#pragma once

#include <cmath>

namespace pqk {

// A capped score's constants: `top`, the cap times log2 e, and `to_unit`, from a score times log2 e to one over the cap.
inline void cap_constants(float cap, float &top, float &to_unit) {
    top = (float)(cap * 1.4426950408889634);
    to_unit = (float)(1 / (cap * 1.4426950408889634));
}

// x = score * log2 e -> cap * tanh(score / cap) * log2 e, from tanh y = 1 - 2 / (1 + e^2y): the exponential's and the
// quotient's errors are absolute ones, cap * 2^-20 of the score (with 2^-22 and 2^-23 for theirs), which 16-bit rows do not
// see up to caps of 256 (at 10^6 it is 0.1 and more). EXACT, for f32 rows and larger caps: a relative one, 2^-21, below
// |y| = 0.8 by y + y^3 Q(y^2), Q fitted there for the least largest error (2^-23.9; 2^-22.8 evaluated in f32); from there on
// by the first form of |y|, where 2 / (1 + e^2y) is a third of the unit at most: of a negative y it is nearly 2, and its
// rounding 1.8 times as much. (The Taylor series to 0.4 instead: one f32 row over 4096 tokens up to 1.1e-6 off.)
template <bool EXACT, class Ex2, class Rcp> __device__ inline float cap_score(float x, float to_unit, float top, Ex2 ex2, Rcp rcp) {
    const float y = x * to_unit, u = EXACT ? fabsf(y) : y;
    const float far = fmaf(rcp(1.f + ex2(u * (2.f * 1.4426950408889634f))), -2.f * top, top);
    if (!EXACT) return far;
    const float z = y * y;
    float s = fmaf(z, -0.00441088624f, 0.0191907637f);
    s = fmaf(z, s, -0.0531763146f);
    s = fmaf(z, s, 0.133227658f);
    s = fmaf(z, s, -0.33332867f);
    s = fmaf(z * y, s, y) * top;
    return u < 0.8f ? s : copysignf(far, y);
}

}  // namespace pqk
