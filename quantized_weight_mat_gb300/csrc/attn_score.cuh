// Scores and views of pq_attn_mod: the cap, the bias by distance, a row's first token and prefix.
#pragma once

#include "kv_device.cuh"

namespace pqk {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// x = score * log2 e -> cap * tanh(score / cap) * log2 e, from tanh y = 1 - 2 / (1 + e^2y): the exponential's and the
// quotient's errors are absolute ones, cap * 2^-21 of the score, which 16-bit rows do not see up to caps of 256 (at 10^6 it
// is 0.1 and more). EXACT, for f32 rows and larger caps: a relative one, 2^-22,
// below y = 0.8 by y + y^3 Q(y^2), Q fitted there for the least largest error (2^-23.9; 2^-22.8 evaluated in f32); from
// there on the first form is as good. (The Taylor series to 0.4 instead: one f32 row over 4096 tokens up to 1.1e-6 off.)
template <bool EXACT> __device__ __forceinline__ float capped(float x, const AttnMod &m) {
    const float y = x * m.to_unit;
    const float far = fmaf(rcp(1.f + ex2(y * (2.f * kLog2e))), -2.f * m.top, m.top);
    if (!EXACT) return far;
    const float z = y * y;
    float s = fmaf(z, -0.00441088624f, 0.0191907637f);
    s = fmaf(z, s, -0.0531763146f);
    s = fmaf(z, s, 0.133227658f);
    s = fmaf(z, s, -0.33332867f);
    s = fmaf(z * y, s, y) * m.top;
    return fabsf(y) < 0.8f ? s : far;
}

// What a row sees beside what its position says: tokens from `first` on, and all below `prefix` (kept below len).
struct RowView {
    int first, prefix;
    // near: causality aside, whether window and first tokens show it
    __device__ __forceinline__ bool sees(int t, int pos, bool near) const { return t >= first && (t < prefix || (t <= pos && near)); }
};
// Of a row at a position of 0 or more.
__device__ __forceinline__ RowView row_view(const AttnArgs &p, int r, int len) {
    RowView v;
    v.first = p.mod.first ? max(p.mod.first[r], 0) : 0;
    v.prefix = p.mod.prefix ? min(max(p.mod.prefix[r], 0), len) : 0;
    return v;
}

}  // namespace
}  // namespace pqk
