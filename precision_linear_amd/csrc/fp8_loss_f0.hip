// Kernels of the FP8 multiply with the cross entropy's softmax statistics in its
// epilogue, for A and B in e4m3fn.
#include "fp8_gemm_kernels.h"

FP8MM_DEFINE_LOSS_TABLE(kStatsF0, kEpiStats, 0)
