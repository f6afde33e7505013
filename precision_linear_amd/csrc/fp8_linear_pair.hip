// Kernels of two products in one launch for A in e5m2 and B in e4m3fn: the
// linear layer's gradient, dx and dw.
#include "fp8_gemm_kernels.h"

#define FP8MM_PAIR_ENTRY(name, BM, BN, BK, WMW, WNW, ST, MI, GM) \
    &launch_pair<BM, BN, BK, WMW, WNW, ST, MI, GM, 1>,

namespace fp8mm {
PairLaunch kPairF1[kNumGenericConfigs] = {FP8MM_GENERIC_CONFIGS(FP8MM_PAIR_ENTRY)};
}
