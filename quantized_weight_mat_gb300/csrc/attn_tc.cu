// The prompt attention kernel as pq_attn runs it.

#include "attn_tc.cuh"

namespace pqk {

unsigned attn_tc_wait_timeouts(bool reset) {
    unsigned v = 0;
    if (cudaMemcpyFromSymbol(&v, g_wait_timeouts, sizeof(v)) != cudaSuccess) return 0;
    if (reset) {
        const unsigned z = 0;
        cudaMemcpyToSymbol(g_wait_timeouts, &z, sizeof(z));
    }
    return v;
}

size_t attn_tc_ws_bytes(int d) { return attn_splits_bytes() + 2 * kTcGrid * attn_part_floats(RT, d) * 4; }

cudaError_t launch_attn_tc(int dt, const AttnArgs &a, cudaStream_t s, const DeviceInfo &dev) { return launch_dt<0>(dt, a, s, dev); }

}  // namespace pqk
