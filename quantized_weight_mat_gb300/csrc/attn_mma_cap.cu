// The decode-step attention kernel with the capped scores, views and biases of pq_attn_mod.

#define PQ_ATTN_MOD
#include "attn_mma.cu"

namespace pqk {

unsigned attn_mma_cap_wait_timeouts(bool reset) {
    unsigned v = 0;
    if (cudaMemcpyFromSymbol(&v, g_wait_timeouts, sizeof(v)) != cudaSuccess) return 0;
    if (reset) {
        const unsigned z = 0;
        cudaMemcpyToSymbol(g_wait_timeouts, &z, sizeof(z));
    }
    return v;
}

cudaError_t launch_attn_mma_cap(int dt, const AttnArgs &a, int rows, cudaStream_t s, const DeviceInfo &dev) {
    if (a.mod.large && dt == PQ_F16) return launch_t<__half, kExact>(a, rows, s, dev);
    if (a.mod.large && dt == PQ_BF16) return launch_t<__nv_bfloat16, kExact>(a, rows, s, dev);
    return a.mod.slope ? launch_dt<kViews | kCap | kBias>(dt, a, rows, s, dev) : launch_dt<kViews | kCap>(dt, a, rows, s, dev);
}

}  // namespace pqk
