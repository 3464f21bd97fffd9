// Instantiation of the expert-sorted products for f16 (see gemm.hpp).
#include "gemm_kernels.hpp"

namespace moeq {

moeq_status launch_gemm_f16(const GemmArgs &a, GemmMode mode, hipStream_t s) {
  return launch_gemm_16bit<MOEQ_F16>(a, mode, s);
}

}  // namespace moeq
