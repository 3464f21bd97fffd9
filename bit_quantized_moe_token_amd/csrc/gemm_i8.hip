// Instantiation of the expert-sorted products for 8-bit codes (see gemm.hpp).
#include "gemm_kernels.hpp"

namespace moeq {

moeq_status launch_gemm_i8(const GemmArgs &a, hipStream_t s) {
  return launch_staged<kI8, kFwd, 128, 128, 2, 2>(a, s, "gemm_i8");
}

}  // namespace moeq
