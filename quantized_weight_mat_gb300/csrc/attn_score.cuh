// Scores and views of pq_attn_mod: the cap, the bias by distance, a row's first token and prefix.
#pragma once

#include "attn_cap.cuh"
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

template <bool EXACT> __device__ __forceinline__ float capped(float x, const AttnMod &m) {
    return cap_score<EXACT>(x, m.to_unit, m.top, [](float v) { return ex2(v); }, [](float v) { return rcp(v); });
}

// The slope of a query head in log2 units; MAYBE: 0 if there are none. An infinite one is NaN, so that every score that a row sees is: of
// tokens all ahead of a row the prompt kernel would otherwise take none, and give zeros. A finite one counts up to 2^96: times
// the largest distance (below 2^31) and log2 e it stays below 2^128, where a bias of -infinity would make NaN of warps that
// see no nearer token; between tokens at different distances nothing but the nearer one counts either way.
template <bool MAYBE> __device__ __forceinline__ float slope_of(const AttnArgs &p, int head) {
    if (MAYBE && !p.mod.slope) return 0.f;
    const float s = p.mod.slope[head];
    return fmaf(fminf(fmaxf(s, -0x1p96f), 0x1p96f), kLog2e, s - s);      // s - s: 0, or NaN
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
