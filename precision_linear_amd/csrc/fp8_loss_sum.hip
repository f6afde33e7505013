// The ping-pong kernel of a product whose sums stay in fp32 (kEpiSum), for A in e5m2
// (the codes of the cross entropy's gradient) and B in either format, and the kernel
// that joins the sums of its work units.
#include "fp8_gemm_kernels.h"

namespace {

// out = bf16(scale_a scale_b sum over the units of a tile).  Workgroup: 16 rows of a
// wave's 128 x 64 sums; each of its waves 16 of the columns, as the accumulators
// lie.  1001 x
// 2048 of 8 units a tile, 67 MB: 12.7 us.
__global__ void __launch_bounds__(256) join_sums_kernel(SumParams p) {
    constexpr int PER_WAVE = 128 * 64, kAhead = 8;
    const int j = blockIdx.x % pp::FM, wave = blockIdx.x / pp::FM % pp::WAVES;
    const int t = blockIdx.x / (pp::FM * pp::WAVES);
    const int i = threadIdx.x / kWave, lane = threadIdx.x % kWave;
    int pm, pn;
    tile_coords(t, p.tiles_m, p.tiles_n, 8, pm, pn);
    const int m = pm * pp::BM + wave / 4 * 128 + j * pp::MI + lane % pp::MI;
    const int n = pn * pp::BN + wave % 4 * 64 + epi_col<pp::MI>(i, 0, lane);
    if (m >= p.M || n >= p.N) return;   // N is a multiple of 16
    const v4f* at = reinterpret_cast<const v4f*>(p.partials) + ((size_t)t * pp::WAVES + wave) * (PER_WAVE / 4) +
                    (i * pp::FM + j) * kWave + lane;
    const size_t unit = (size_t)p.num_tiles * pp::WAVES * (PER_WAVE / 4);   // [unit][tile]
    v4f sum{};
    for (int s = 0; s < p.splits; s += kAhead) {
        v4f v[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) v[k] = s + k < p.splits ? at[(s + k) * unit] : v4f{};
#pragma unroll
        for (int k = 0; k < kAhead; ++k) sum += v[k];
    }
    const float sa = p.scale_a[m];
    const v4f sb{p.scale_b[n], p.scale_b[n + 1], p.scale_b[n + 2], p.scale_b[n + 3]};
    uint2 w;
    w.x = pack_bf16x2(sum[0] * (sa * sb[0]), sum[1] * (sa * sb[1]));
    w.y = pack_bf16x2(sum[2] * (sa * sb[2]), sum[3] * (sa * sb[3]));
    uint16_t* out = p.out + (size_t)m * p.N + n;
    if (p.vec_store) {
        *reinterpret_cast<uint2*>(out) = w;
    } else {
        out[0] = (uint16_t)w.x;
        out[1] = (uint16_t)(w.x >> 16);
        out[2] = (uint16_t)w.y;
        out[3] = (uint16_t)(w.y >> 16);
    }
}

}  // namespace

namespace fp8mm {

Launch kSum[2] = {&launch_pp<8, 1, kEpiSum>, &launch_pp<8, 3, kEpiSum>};

void join_sums(const SumParams& p, hipStream_t stream) {
    hipLaunchKernelGGL(join_sums_kernel, dim3((unsigned)(p.num_tiles * pp::WAVES * pp::FM)), dim3(256), 0, stream, p);
}

}  // namespace fp8mm
