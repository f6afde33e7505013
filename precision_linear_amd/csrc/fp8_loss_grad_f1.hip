// Kernels of the FP8 multiply with the codes of the cross entropy's gradient in its
// epilogue, for A in e5m2 and B in e4m3fn.
#include "fp8_gemm_kernels.h"

FP8MM_DEFINE_LOSS_TABLE(kCodesF1, kEpiCodes, 1)
