// The prompt attention kernel with the capped scores, views and biases of pq_attn_mod.

#define PQ_ATTN_MOD
#include "attn_tc.cu"

namespace pqk {

unsigned attn_tc_cap_wait_timeouts(bool reset) {
    unsigned v = 0;
    if (cudaMemcpyFromSymbol(&v, g_wait_timeouts, sizeof(v)) != cudaSuccess) return 0;
    if (reset) {
        const unsigned z = 0;
        cudaMemcpyToSymbol(g_wait_timeouts, &z, sizeof(z));
    }
    return v;
}

cudaError_t launch_attn_tc_cap(int dt, const AttnArgs &a, cudaStream_t s, const DeviceInfo &dev) {
    if (a.mod.large) return launch_dt<kExact>(dt, a, s, dev);
    return a.mod.slope ? launch_dt<kViews | kCap | kBias>(dt, a, s, dev) : launch_dt<kViews | kCap>(dt, a, s, dev);
}

}  // namespace pqk
