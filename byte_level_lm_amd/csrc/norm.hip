// RMS norm of rows with the residual's addition, in the activations' type or
// as 8-bit rows with a scale; rows to 8 bits without a norm.
//
//   s = x + residual (fp32),  r = 1 / sqrt(mean(s^2) + eps),  y = (s w) r
//   8 bits: t = s w,  a = max |t|,  q = rne(t * (127 * (1 / a))),  scale = a r / 127
// r divides out of q, so q depends on no sum's order: it is the same whole
// number whatever the split of the row over threads.
//
// One workgroup per row, two passes over it: the sum of squares and the
// largest |t|, then the outputs.
#include "common.h"

namespace bllm {
namespace {

constexpr float kTiny = 1e-30f;  // a row whose largest |t| is below this becomes zeros with scale 0

// what one call computes
struct NormArgs {
  const void* x;
  const void* res;   // or null
  const void* w;     // or null (no norm: r = 1, w = 1)
  void* res_out;     // or null
  void* y;           // or null
  int8_t* q;         // or null
  float* scale;
  int64_t rows;
  int d;
  float eps;
};

// 127 (1 / a) and the row's scale; zeros for rows that are too small to divide by
__device__ inline void quant_scales(float a, float r, float* inv, float* scale) {
  const bool some = !(a < kTiny);
  *inv = some ? 127.0f * (1.0f / a) : 0.0f;
  *scale = some ? a * r / 127.0f : 0.0f;
}

__device__ inline int quant1(float t, float inv) {
  const float v = rintf(t * inv);
  return static_cast<int>(fminf(fmaxf(v, -127.0f), 127.0f));
}

template <int DT>
__global__ __launch_bounds__(256) void norm_rows(NormArgs a) {
  constexpr int N = Vec<DT>::N;
  __shared__ float sSum[4], sMax[4];
  const int64_t base = static_cast<int64_t>(blockIdx.x) * a.d;
  float ss = 0.0f, top = 0.0f;
  for (int c = threadIdx.x * N; c < a.d; c += 256 * N) {
    float s[N], r[N], w[N];
    Vec<DT>::load(a.x, base + c, s);
    if (a.res) Vec<DT>::load(a.res, base + c, r);
    if (a.w) Vec<DT>::load(a.w, c, w);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (a.res) s[i] += r[i];
      ss += s[i] * s[i];
      top = fmaxf(top, fabsf(a.w ? s[i] * w[i] : s[i]));
    }
  }
  ss = wave_sum(ss);
  for (int off = 32; off >= 1; off >>= 1) top = fmaxf(top, __shfl_xor(top, off, kWave));
  if ((threadIdx.x & 63) == 0) {
    sSum[threadIdx.x >> 6] = ss;
    sMax[threadIdx.x >> 6] = top;
  }
  __syncthreads();
  ss = sSum[0] + sSum[1] + sSum[2] + sSum[3];
  top = fmaxf(fmaxf(sMax[0], sMax[1]), fmaxf(sMax[2], sMax[3]));
  // a NaN in the row is lost by the maximum but not by the sum: it reaches r, y and the scale
  const float r1 = a.w ? 1.0f / sqrtf(ss / static_cast<float>(a.d) + a.eps) : (ss == ss ? 1.0f : ss);
  float inv, scale;
  quant_scales(top, r1, &inv, &scale);
  for (int c = threadIdx.x * N; c < a.d; c += 256 * N) {
    float s[N], r[N], w[N];
    Vec<DT>::load(a.x, base + c, s);
    if (a.res) Vec<DT>::load(a.res, base + c, r);
    if (a.w) Vec<DT>::load(a.w, c, w);
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (a.res) s[i] += r[i];
    if (a.res_out) Vec<DT>::store(a.res_out, base + c, s);
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (a.w) s[i] *= w[i];
    if (a.q) {
#pragma unroll
      for (int i = 0; i < N; ++i) a.q[base + c + i] = static_cast<int8_t>(quant1(s[i], inv));
    }
    if (a.y) {
#pragma unroll
      for (int i = 0; i < N; ++i) s[i] *= r1;
      Vec<DT>::store(a.y, base + c, s);
    }
  }
  if (a.q && threadIdx.x == 0) a.scale[blockIdx.x] = scale;
}

int norm_launch(const NormArgs& a, int dtype, void* stream) {
  if (a.rows == 0) return BLLM_OK;
  const dim3 grid(static_cast<unsigned>(a.rows));
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (dtype == BLLM_F32)
    hipLaunchKernelGGL(norm_rows<BLLM_F32>, grid, dim3(256), 0, st, a);
  else
    hipLaunchKernelGGL(norm_rows<BLLM_BF16>, grid, dim3(256), 0, st, a);
  return launch_status();
}

// arguments shared by the three entry points; `eps` only matters with a norm
int norm_check(const void* x, int dtype, int64_t rows, int64_t d, bool outputs) {
  if (rows < 0 || d < 1 || (rows > 0 && (!x || !outputs))) return BLLM_E_INVAL;
  if (!valid_dtype(dtype) || (d * elem_size(dtype)) % 16 != 0 || d >= (int64_t(1) << 24) ||
      rows >= (int64_t(1) << 31))
    return BLLM_E_NOTSUP;
  return BLLM_OK;
}

bool norm_aligned(const NormArgs& a) {
  return aligned16(a.x) && aligned16(a.res) && aligned16(a.w) && aligned16(a.res_out) && aligned16(a.y) &&
         aligned16(a.q) && (reinterpret_cast<uintptr_t>(a.scale) & 3u) == 0;
}

}  // namespace
}  // namespace bllm

using namespace bllm;

extern "C" int bllm_rmsnorm(const void* x, const void* residual, const void* w, int dtype, int64_t rows,
                            int64_t d, double eps, void* residual_out, void* y_out, void* stream) {
  if (!(eps >= 0.0) || !w || (residual_out && !residual)) return BLLM_E_INVAL;
  const int rc = norm_check(x, dtype, rows, d, y_out != nullptr);
  if (rc != BLLM_OK) return rc;
  NormArgs a{x, residual, w, residual_out, y_out, nullptr, nullptr, rows, static_cast<int>(d),
             static_cast<float>(eps)};
  return norm_aligned(a) ? norm_launch(a, dtype, stream) : BLLM_E_NOTSUP;
}

extern "C" int bllm_rmsnorm_q8(const void* x, const void* residual, const void* w, int dtype, int64_t rows,
                               int64_t d, double eps, void* residual_out, int8_t* q_out, float* scale_out,
                               void* stream) {
  if (!(eps >= 0.0) || !w || (residual_out && !residual)) return BLLM_E_INVAL;
  const int rc = norm_check(x, dtype, rows, d, q_out && scale_out);
  if (rc != BLLM_OK) return rc;
  NormArgs a{x, residual, w, residual_out, nullptr, q_out, scale_out, rows, static_cast<int>(d),
             static_cast<float>(eps)};
  return norm_aligned(a) ? norm_launch(a, dtype, stream) : BLLM_E_NOTSUP;
}

extern "C" int bllm_quant_rows_q8(const void* x, int dtype, int64_t rows, int64_t d, int8_t* q_out,
                                  float* scale_out, void* stream) {
  const int rc = norm_check(x, dtype, rows, d, q_out && scale_out);
  if (rc != BLLM_OK) return rc;
  NormArgs a{x, nullptr, nullptr, nullptr, nullptr, q_out, scale_out, rows, static_cast<int>(d), 0.0f};
  return norm_aligned(a) ? norm_launch(a, dtype, stream) : BLLM_E_NOTSUP;
}
