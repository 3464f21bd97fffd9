// Instantiation of the expert-sorted products for 8-bit codes (see gemm.hpp).
#include "gemm_kernels.hpp"

namespace moeq {

moeq_status launch_gemm_i8(const GemmArgs &a, hipStream_t s) {
  return launch_mode<kI8, kFwd>(a, s, "gemm_i8");
}

}  // namespace moeq
