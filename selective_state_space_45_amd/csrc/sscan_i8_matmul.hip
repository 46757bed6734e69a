// Products of rows in 8-bit integers with the scales of both sides.
#include "sscan_layer.h"

namespace sscan {

typedef int i32x4 __attribute__((ext_vector_type(4)));

// A workgroup of four waves has a tile of 64 x 64 sums; k goes through LDS 64 bytes at a time.
// Lane l of a matrix instruction holds row l % 16 of either side, bytes 16 (l / 16) .. + 15,
// and of the result column l % 16, rows 4 (l / 16) .. + 3.
template <typename Tout>
__global__ __launch_bounds__(256) void i8_matmul_kernel(MatmulParams p, int ntn) {
  constexpr int kPitch = 80;
  __shared__ __attribute__((aligned(16))) int8_t la[64 * kPitch];
  __shared__ __attribute__((aligned(16))) int8_t lb[64 * kPitch];
  const int64_t tile = workgroup<256>();
  const int64_t m0 = tile / ntn * 64, n0 = tile % ntn * 64;
  if (m0 >= p.m) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  i32x4 acc[4] = {};
  for (int k0 = 0; k0 < p.k; k0 += 64) {
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const int at = j * 256 + threadIdx.x, r = at >> 6, c = at & 63;
      const bool in = k0 + c < p.k;
      la[r * kPitch + c] = in && m0 + r < p.m ? p.a[(m0 + r) * p.sa + k0 + c] : 0;
      lb[r * kPitch + c] = in && n0 + r < p.n ? p.b[(n0 + r) * p.sb + k0 + c] : 0;
    }
    __syncthreads();
    const int at = (lane & 15) * kPitch + (lane >> 4) * 16;
    const i32x4 a = *reinterpret_cast<const i32x4*>(la + wave * 16 * kPitch + at);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      acc[j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(a, *reinterpret_cast<const i32x4*>(lb + j * 16 * kPitch + at), acc[j], 0, 0, 0);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int64_t n = n0 + j * 16 + (lane & 15);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t m = m0 + wave * 16 + (lane >> 4) * 4 + i;
      if (m < p.m && n < p.n)
        store_val(static_cast<Tout*>(p.out) + m * p.so + n,
                  fmaf(static_cast<float>(acc[j][i]), p.as[m] * p.bs[n], p.bias ? p.bias[n] : 0.f));
    }
  }
}

size_t i8_matmul_workspace_bytes(int64_t, int64_t, int64_t) { return 0; }

hipError_t launch_i8_matmul(const MatmulParams& p, size_t, bool bf16, hipStream_t s) {
  const int ntn = (p.n + 63) / 64;
  const int64_t tiles = static_cast<int64_t>(ntn) * ((p.m + 63) / 64);
  if (bf16) hipLaunchKernelGGL((i8_matmul_kernel<bf16_t>), grid_of<256>(tiles), dim3(256), 0, s, p, ntn);
  else hipLaunchKernelGGL((i8_matmul_kernel<float>), grid_of<256>(tiles), dim3(256), 0, s, p, ntn);
  return hipGetLastError();
}

}  // namespace sscan
