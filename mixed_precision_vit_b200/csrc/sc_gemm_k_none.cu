// The matrix product's kernels with this activation in the epilogue.
#include "sc_gemm_dev.cuh"

namespace scb {
namespace gemm {

GemmKernels gemm_kernels_none() { return gemm_kernels<SC_ACT_NONE>(); }

}  // namespace gemm
}  // namespace scb
