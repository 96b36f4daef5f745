// The paged attention over the 8-bit cache with block scales, many query rows.
#include "attend_many.cuh"

namespace dkv {

template cudaError_t launch_attend_many<kE4M3, __nv_bfloat16, 64>(const AttendParams&, int, cudaStream_t);
template cudaError_t launch_attend_many<kE4M3, __nv_bfloat16, 128>(const AttendParams&, int, cudaStream_t);
template cudaError_t launch_attend_many<kE4M3, __half, 64>(const AttendParams&, int, cudaStream_t);
template cudaError_t launch_attend_many<kE4M3, __half, 128>(const AttendParams&, int, cudaStream_t);

}  // namespace dkv
