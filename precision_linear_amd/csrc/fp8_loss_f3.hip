// Kernels of the FP8 multiply with the cross entropy's softmax statistics in its
// epilogue, for A and B in e5m2.
#include "fp8_gemm_kernels.h"

FP8MM_DEFINE_LOSS_TABLE(kStatsF3, kEpiStats, 3)
