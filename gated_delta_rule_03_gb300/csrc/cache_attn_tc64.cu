// cache_attn_tc64.cu -- the many-row kernels of cache_attn_tc.cuh for heads of 64.
#include "cache_attn_tc.cuh"

namespace gdr {
namespace cattn {

int launch_tc64(const Attn &a, int codes, int dtype, void *ws, cudaStream_t s) {
    return launch_tc_d<64>(a, codes, dtype, ws, s);
}
size_t tc_bytes64(const Attn &a, int dtype) { return tc_bytes_d<64>(a, dtype); }

}  // namespace cattn
}  // namespace gdr
