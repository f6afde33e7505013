// The ping-pong kernel of a product whose K range comes in pieces, for A in e5m2
// (the codes of the cross entropy's gradient) and B in either format.
#include "fp8_gemm_kernels.h"

namespace fp8mm {
Launch kSum[2] = {&launch_pp<8, 1, kEpiSum>, &launch_pp<8, 3, kEpiSum>};
}
