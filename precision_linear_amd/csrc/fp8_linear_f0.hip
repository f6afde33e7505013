// Kernels of the FP8 scaled multiply with the linear layer's epilogue for A in
// e4m3fn and B in e4m3fn.
#include "fp8_gemm_kernels.h"

FP8MM_DEFINE_LINEAR_TABLE(kLinearF0, 0)
