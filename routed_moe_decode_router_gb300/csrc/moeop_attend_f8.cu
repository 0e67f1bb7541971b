// moeop_attend_f8.cu -- attention over a cache of type MOEOP_E4M3.
#include "moeop_attend.cuh"

namespace moe {
namespace op {

cudaError_t launch_attend_f8(const AttendParams &p, int dim, cudaStream_t st) {
    return attend::launch_type<MOEOP_E4M3>(p, dim, st);
}

}  // namespace op
}  // namespace moe
