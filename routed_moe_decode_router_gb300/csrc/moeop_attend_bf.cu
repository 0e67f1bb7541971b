// moeop_attend_bf.cu -- attention over a cache of type MOEOP_BF16.
#include "moeop_attend.cuh"

namespace moe {
namespace op {

cudaError_t launch_attend_bf(const AttendParams &p, int dim, cudaStream_t st) {
    return attend::launch_type<MOEOP_BF16>(p, dim, st);
}

}  // namespace op
}  // namespace moe
