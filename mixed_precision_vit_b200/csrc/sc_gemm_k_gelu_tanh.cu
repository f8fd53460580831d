// The matrix product's kernels with this activation in the epilogue.
#include "sc_gemm_dev.cuh"

namespace scb {
namespace gemm {

GemmKernels gemm_kernels_gelu_tanh() { return gemm_kernels<SC_ACT_GELU_TANH>(); }

}  // namespace gemm
}  // namespace scb
