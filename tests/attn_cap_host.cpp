// Host build of the cap that the attention kernels put on scores (attn_cap.cuh), for a CPU test: its two hardware
// functions rounded to nearest, or off by what the PTX documentation allows them (2^-22 for ex2.approx.ftz.f32, one
// last bit for rcp.approx.ftz.f32).
#define __device__
#include "attn_cap.cuh"

// n scores times log2 e; `e` and `r`: the sign of the two functions' errors, 0 for none.
extern "C" void cap_host(int exact, float cap, int e, int r, int n, const float *x, float *out) {
    float top, to_unit;
    pqk::cap_constants(cap, top, to_unit);
    auto ex2 = [&](float v) { return (float)(std::exp2((double)v) * (1 + e * 0x1p-22)); };
    auto rcp = [&](float v) {
        const float y = (float)(1 / (double)v);
        return r == 0 ? y : std::nextafterf(y, r > 0 ? INFINITY : 0.f);
    };
    for (int i = 0; i < n; ++i)
        out[i] = exact ? pqk::cap_score<true>(x[i], to_unit, top, ex2, rcp) : pqk::cap_score<false>(x[i], to_unit, top, ex2, rcp);
}
