// moeop_attend_hf.cu -- attention over a cache of type MOEOP_FP16.
#include "moeop_attend.cuh"

namespace moe {
namespace op {

cudaError_t launch_attend_hf(const AttendParams &p, int dim, cudaStream_t st) {
    return attend::launch_type<MOEOP_FP16>(p, dim, st);
}

}  // namespace op
}  // namespace moe
