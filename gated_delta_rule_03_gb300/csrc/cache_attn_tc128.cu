// cache_attn_tc128.cu -- the many-row kernels of cache_attn_tc.cuh for heads of 128.
#include "cache_attn_tc.cuh"

namespace gdr {
namespace cattn {

int launch_tc128(const Attn &a, int codes, int dtype, void *ws, cudaStream_t s) {
    return launch_tc_d<128>(a, codes, dtype, ws, s);
}
size_t tc_bytes128(const Attn &a, int dtype) { return tc_bytes_d<128>(a, dtype); }

}  // namespace cattn
}  // namespace gdr
