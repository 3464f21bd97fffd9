// Instantiation of the expert-sorted products for bf16 (see gemm.hpp).
#include "gemm_kernels.hpp"

namespace moeq {

moeq_status launch_gemm_bf16(const GemmArgs &a, GemmMode mode, hipStream_t s) {
  return launch_gemm_16bit<MOEQ_BF16>(a, mode, s);
}

}  // namespace moeq
