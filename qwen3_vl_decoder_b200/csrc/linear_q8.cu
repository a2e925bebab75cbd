// Product of 8-bit rows and an 8-bit weight with block scales (q8.cuh):
//   out[m][n] = sum_j 2^(xs[m][j] + ws[n / 128][j] - 254) sum_{k in block j} xq[m][k] wq[n][k]
// (+ resid[m][n]), in fp32.
#include "q3vl_internal.h"
#include "q8.cuh"

namespace q3vl {
namespace {

// One warp per output: lanes stride over the k-blocks' words.
template <typename T>
__global__ void __launch_bounds__(256)
linear_q8_kernel(const uint8_t* __restrict__ xq, const uint8_t* __restrict__ xs, int64_t M,
                 const uint8_t* __restrict__ wq, const uint8_t* __restrict__ ws, int64_t N,
                 int64_t K, const T* resid, T* out) {
  const int lane = threadIdx.x & 31;
  const int64_t idx = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (idx >= M * N) return;
  const int64_t m = idx / N, n = idx % N, kblk = (K + 127) / 128;
  float acc = 0.f;
  for (int64_t k = 4 * lane; k < K; k += 128) {
    const float4 a = unpack_e4m3x4(*reinterpret_cast<const uint32_t*>(xq + m * K + k));
    const float4 b = unpack_e4m3x4(*reinterpret_cast<const uint32_t*>(wq + n * K + k));
    const float s = e8m0_scale(xs[m * kblk + k / 128]) * e8m0_scale(ws[n / 128 * kblk + k / 128]);
    acc = fmaf(s, a.x * b.x + a.y * b.y + a.z * b.z + a.w * b.w, acc);
  }
  acc = warp_sum(acc);
  if (lane == 0) {
    if (resid != nullptr) acc += static_cast<float>(resid[idx]);
    out[idx] = static_cast<T>(acc);
  }
}

}  // namespace

cudaError_t launch_linear_q8(const uint8_t* xq, const uint8_t* xs, int64_t M, const uint8_t* wq,
                             const uint8_t* ws, int64_t N, int64_t K, const void* resid, void* out,
                             bool out_bf16, cudaStream_t st) {
  const int64_t blocks = (M * N + 7) / 8;
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  if (out_bf16)
    linear_q8_kernel<<<static_cast<unsigned>(blocks), 256, 0, st>>>(
        xq, xs, M, wq, ws, N, K, static_cast<const __nv_bfloat16*>(resid),
        static_cast<__nv_bfloat16*>(out));
  else
    linear_q8_kernel<<<static_cast<unsigned>(blocks), 256, 0, st>>>(
        xq, xs, M, wq, ws, N, K, static_cast<const float*>(resid), static_cast<float*>(out));
  return counted_launch(1);
}

}  // namespace q3vl
