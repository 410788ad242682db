// Product of 8-bit rows with 8-bit weights, a scale for each token and each
// output channel:
//   y[m, n] = (sum_k xq[m, k] wq[n, k]) * (x_scale[m] * w_scale[n]) + bias[n]
// The sum is exact in 32-bit integers (128^2 K < 2^31 up to kMaxK), so it
// does not depend on its order; the scales and the bias are applied in fp32
// and y is rounded once.
//
// A wave owns a 32 x 32 tile of y as 2 x 2 tiles of v_mfma_i32_16x16x64_i8 and
// reads its operands straight from memory: both are row-major along K, so a
// lane's 16 bytes of a row are one load.
#include "common.h"

namespace bllm {
namespace {

typedef int intx4 __attribute__((ext_vector_type(4)));

constexpr int64_t kMaxK = (1 << 17) - 16;  // 128 * 128 * kMaxK < 2^31

struct LinArgs {
  const int8_t* xq;
  const float* sx;
  const int8_t* wq;
  const float* sw;
  const float* bias;  // or null
  void* y;
  int64_t m, n;
  int k;
};

// element r of a lane's 16 x 16 accumulator: row 4 (lane / 16) + r, column lane % 16
template <int DT>
__device__ inline void store_y(const LinArgs& a, int64_t row, int64_t col, int acc) {
  float v = static_cast<float>(acc) * (a.sx[row] * a.sw[col]);
  if (a.bias) v += a.bias[col];
  if (DT == BLLM_F32)
    static_cast<float*>(a.y)[row * a.n + col] = v;
  else
    static_cast<uint16_t*>(a.y)[row * a.n + col] = f32_to_bf16(v);
}

template <int DT>
__global__ __launch_bounds__(256) void linear_direct(LinArgs a) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t row0 = static_cast<int64_t>(blockIdx.y) * 64 + (wave >> 1) * 32;
  const int64_t col0 = static_cast<int64_t>(blockIdx.x) * 64 + (wave & 1) * 32;
  const int kk = (lane >> 4) * 16;
  const int8_t* pa[2];
  const int8_t* pb[2];
  for (int i = 0; i < 2; ++i) {
    const int64_t r = row0 + 16 * i + (lane & 15), c = col0 + 16 * i + (lane & 15);
    pa[i] = a.xq + (r < a.m ? r : a.m - 1) * a.k;
    pb[i] = a.wq + (c < a.n ? c : a.n - 1) * a.k;
  }
  intx4 acc[2][2] = {};
  for (int k0 = 0; k0 < a.k; k0 += 64) {
    intx4 fa[2] = {}, fb[2] = {};
    if (k0 + kk < a.k) {
      for (int i = 0; i < 2; ++i) {
        fa[i] = *reinterpret_cast<const intx4*>(pa[i] + k0 + kk);
        fb[i] = *reinterpret_cast<const intx4*>(pb[i] + k0 + kk);
      }
    }
    for (int i = 0; i < 2; ++i)
      for (int j = 0; j < 2; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fa[i], fb[j], acc[i][j], 0, 0, 0);
  }
  for (int i = 0; i < 2; ++i)
    for (int j = 0; j < 2; ++j)
      for (int r = 0; r < 4; ++r) {
        const int64_t row = row0 + 16 * i + 4 * (lane >> 4) + r, col = col0 + 16 * j + (lane & 15);
        if (row < a.m && col < a.n) store_y<DT>(a, row, col, acc[i][j][r]);
      }
}

}  // namespace
}  // namespace bllm

using namespace bllm;

extern "C" size_t bllm_linear_i8_workspace(int64_t m, int64_t n, int64_t k) { return 0; }

extern "C" int bllm_linear_i8(const int8_t* xq, const float* x_scale, const int8_t* wq, const float* w_scale,
                              const float* bias, int dtype, int64_t m, int64_t n, int64_t k, void* y_out,
                              void* ws, size_t ws_bytes, void* stream) {
  if (m < 0 || n < 1 || k < 1 || !wq || !w_scale || (m > 0 && (!xq || !x_scale || !y_out))) return BLLM_E_INVAL;
  if (!valid_dtype(dtype) || k % 16 != 0 || k > kMaxK || m >= (int64_t(1) << 31) || n >= (int64_t(1) << 31) ||
      !aligned16(xq) || !aligned16(wq) || !aligned16(y_out))
    return BLLM_E_NOTSUP;
  if (m == 0) return BLLM_OK;
  LinArgs a{xq, x_scale, wq, w_scale, bias, y_out, m, n, static_cast<int>(k)};
  const int64_t gy = ceil_div(m, 64), gx = ceil_div(n, 64);
  if (gy > 65535) return BLLM_E_NOTSUP;
  hipStream_t st = static_cast<hipStream_t>(stream);
  const dim3 grid(static_cast<unsigned>(gx), static_cast<unsigned>(gy));
  if (dtype == BLLM_F32)
    hipLaunchKernelGGL(linear_direct<BLLM_F32>, grid, dim3(256), 0, st, a);
  else
    hipLaunchKernelGGL(linear_direct<BLLM_BF16>, grid, dim3(256), 0, st, a);
  return launch_status();
}
