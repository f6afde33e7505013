// Kernels of the FP8 multiply with the cross entropy's softmax statistics in its
// epilogue, for A in e4m3fn and B in e5m2.
#include "fp8_gemm_kernels.h"

FP8MM_DEFINE_LOSS_TABLE(kStatsF2, kEpiStats, 2)
