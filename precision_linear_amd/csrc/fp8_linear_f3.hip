// Kernels of the FP8 scaled multiply with the linear layer's epilogue for A in
// e5m2 and B in e5m2.
#include "fp8_gemm_kernels.h"

FP8MM_DEFINE_LINEAR_TABLE(kLinearF3, 3)
