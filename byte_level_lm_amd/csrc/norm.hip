// RMS norm of rows with the residual's addition, in the activations' type or
// as 8-bit rows with a scale; rows to 8 bits without a norm.
//
//   s = x + residual (fp32),  r = 1 / sqrt(mean(s^2) + eps),  y = (s w) r
//   8 bits: t = s w,  a = max |t|,  q = rne(t * (127 * (1 / a))),  scale = a r / 127
// r divides out of q, so q depends on no sum's order: it is the same whole
// number whatever the split of the row over threads.  a is the maximum of the
// bits of |t|: in that order infinity lies above every finite value and NaN
// above infinity, so neither can leave a row with a finite scale.
//
// Bound by the bytes: x and the residual are read once, held in registers as
// they came (a row's 16-byte pieces over the lanes) and the outputs written
// once.  A group of G lanes has a row, with P pieces each: part of a wave for
// short rows (several rows a wave keep its loads in flight), a wave, or a
// workgroup whose waves add up in LDS.  Rows of more than 64 KB are read twice.
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

template <int DT>
__device__ inline void unpack(const uint4& v, float* x) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (DT == BLLM_F32) {
      x[i] = __uint_as_float(u[i]);
    } else {
      x[2 * i] = __uint_as_float(u[i] << 16);
      x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    }
  }
}
__device__ inline uint4 piece(const void* p, int64_t i) { return static_cast<const uint4*>(p)[i]; }

// |t| as the maximum takes it
__device__ inline uint32_t magnitude(float t) { return __float_as_uint(t) & 0x7FFFFFFFu; }

// 1 / sqrt(v), rounded once: the quotient of a rounded root is off by up to a unit in the last place, which
// one step of Newton's iteration takes away (1 - v r^2 from exact products).  0 and infinity stay as they are.
__device__ inline float inverse_root(float v) {
  const float r = 1.0f / sqrtf(v), h = v * r;
  const float e = fmaf(-h, r, 1.0f) - fmaf(v, r, -h) * r;
  return fabsf(e) < 1.0f ? fmaf(0.5f * r, e, r) : r;
}

// the row's divisor and 8-bit scales from its sum of squares and the bits of its largest |t|
struct RowScale {
  float r, inv, scale;
};
__device__ inline RowScale row_scale(const NormArgs& a, float ss, uint32_t bits) {
  RowScale s;
  const float top = __uint_as_float(bits);
  s.r = a.w ? inverse_root(ss / static_cast<float>(a.d) + a.eps) : 1.0f;
  const bool some = !(top < kTiny);  // also where top is NaN, which then is the scale
  s.inv = some ? 127.0f * (1.0f / top) : 0.0f;
  s.scale = some ? top * s.r / 127.0f : 0.0f;
  return s;
}

// s of one piece: x (+ residual)
template <int DT, bool RES>
__device__ inline void sum_piece(const uint4& x, const uint4& res, float* s) {
  constexpr int N = Vec<DT>::N;
  unpack<DT>(x, s);
  if (RES) {
    float r[N];
    unpack<DT>(res, r);
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] += r[i];
  }
}

// writes one piece's outputs; i is the piece's number in the arrays
template <int DT, bool RES, bool Q8>
__device__ inline void put_piece(const NormArgs& a, int64_t i, float* s, const float* w, const RowScale& rs) {
  constexpr int N = Vec<DT>::N;
  if (RES && a.res_out) Vec<DT>::store(a.res_out, i * N, s);
  if (Q8) {
    uint32_t q[N / 4];
#pragma unroll
    for (int j = 0; j < N / 4; ++j) {
      uint32_t u = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float v = rintf(s[4 * j + e] * w[4 * j + e] * rs.inv);
        const int c = static_cast<int>(fminf(fmaxf(v, -127.0f), 127.0f));
        u |= static_cast<uint32_t>(c & 0xFF) << (8 * e);
      }
      q[j] = u;
    }
    uint32_t* to = reinterpret_cast<uint32_t*>(a.q + i * N);
    if constexpr (N == 8)
      *reinterpret_cast<uint2*>(to) = make_uint2(q[0], q[1]);
    else
      *to = q[0];
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j) s[j] = s[j] * w[j] * rs.r;
    Vec<DT>::store(a.y, i * N, s);
  }
}

template <int DT>
__device__ inline void weights(const NormArgs& a, int64_t c, float* w) {
  if (a.w) {
    unpack<DT>(piece(a.w, c), w);
  } else {
#pragma unroll
    for (int i = 0; i < Vec<DT>::N; ++i) w[i] = 1.0f;
  }
}

template <int G>
__device__ inline uint32_t group_max(uint32_t v) {
#pragma unroll
  for (int off = G / 2; off >= 1; off >>= 1) v = max(v, __shfl_xor(v, off, kWave));
  return v;
}

// G <= 64: lanes of a wave, rows side by side.  G > 64: G threads, one row a workgroup.
template <int DT, bool RES, bool Q8, int G, int P>
__global__ __launch_bounds__(G > 256 ? G : 256) void norm_rows(NormArgs a) {
  constexpr int N = Vec<DT>::N, NT = G > 256 ? G : 256, GW = G < 64 ? G : 64;
  __shared__ float sSum[16];
  __shared__ uint32_t sMax[16];
  const int pieces = a.d / N, in = threadIdx.x % G;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (NT / G) + threadIdx.x / G;
  if (G <= 64 && row >= a.rows) return;
  const int64_t base = row * pieces;
  uint4 x[P], r[P];
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const int c = in + p * G;
    x[p] = r[p] = make_uint4(0, 0, 0, 0);
    if (c < pieces) {
      x[p] = piece(a.x, base + c);
      if (RES) r[p] = piece(a.res, base + c);
    }
  }
  float ss = 0.0f;
  uint32_t top = 0;
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const int c = in + p * G;
    if (c >= pieces) break;
    float s[N], w[N];
    sum_piece<DT, RES>(x[p], r[p], s);
    if (Q8) weights<DT>(a, c, w);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      ss = fmaf(s[i], s[i], ss);
      if (Q8) top = max(top, magnitude(s[i] * w[i]));
    }
  }
  ss = group_sum<GW>(ss);
  if (Q8) top = group_max<GW>(top);
  if (G > 64) {
    if ((threadIdx.x & 63) == 0) {
      sSum[threadIdx.x >> 6] = ss;
      sMax[threadIdx.x >> 6] = top;
    }
    __syncthreads();
    ss = 0.0f;
    top = 0;
#pragma unroll
    for (int i = 0; i < G / 64; ++i) {
      ss += sSum[i];
      top = max(top, sMax[i]);
    }
  }
  const RowScale rs = row_scale(a, ss, top);
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const int c = in + p * G;
    if (c >= pieces) break;
    float s[N], w[N];
    sum_piece<DT, RES>(x[p], r[p], s);
    weights<DT>(a, c, w);
    put_piece<DT, RES, Q8>(a, base + c, s, w, rs);
  }
  if (Q8 && in == 0) a.scale[row] = rs.scale;
}

// rows too long for registers: two passes over memory
template <int DT, bool RES, bool Q8>
__global__ __launch_bounds__(1024) void norm_long(NormArgs a) {
  constexpr int N = Vec<DT>::N;
  __shared__ float sSum[16];
  __shared__ uint32_t sMax[16];
  const int pieces = a.d / N;
  const int64_t base = static_cast<int64_t>(blockIdx.x) * pieces;
  float ss = 0.0f;
  uint32_t top = 0;
  for (int c = threadIdx.x; c < pieces; c += 1024) {
    float s[N], w[N];
    sum_piece<DT, RES>(piece(a.x, base + c), RES ? piece(a.res, base + c) : uint4{}, s);
    weights<DT>(a, c, w);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      ss = fmaf(s[i], s[i], ss);
      top = max(top, magnitude(s[i] * w[i]));
    }
  }
  ss = group_sum<64>(ss);
  top = group_max<64>(top);
  if ((threadIdx.x & 63) == 0) {
    sSum[threadIdx.x >> 6] = ss;
    sMax[threadIdx.x >> 6] = top;
  }
  __syncthreads();
  ss = 0.0f;
  top = 0;
  for (int i = 0; i < 16; ++i) {
    ss += sSum[i];
    top = max(top, sMax[i]);
  }
  const RowScale rs = row_scale(a, ss, top);
  for (int c = threadIdx.x; c < pieces; c += 1024) {
    float s[N], w[N];
    sum_piece<DT, RES>(piece(a.x, base + c), RES ? piece(a.res, base + c) : uint4{}, s);
    weights<DT>(a, c, w);
    put_piece<DT, RES, Q8>(a, base + c, s, w, rs);
  }
  if (Q8 && threadIdx.x == 0) a.scale[blockIdx.x] = rs.scale;
}

constexpr int64_t kFewRows = 4096;
constexpr int64_t kMaxThreads = (int64_t(1) << 32) - 1;  // of one launch, along x

// a call's rows in slices of `most` of them, as many as one launch has threads for
template <int DT, typename Launch>
void in_slices(NormArgs a, int64_t most, const Launch& launch) {
  for (int64_t left = a.rows; left > 0; left -= a.rows) {
    a.rows = left < most ? left : most;
    launch(a);
    const int64_t n = a.rows * a.d, bytes = n * elem_size(DT);
    a.x = static_cast<const char*>(a.x) + bytes;
    if (a.res) a.res = static_cast<const char*>(a.res) + bytes;
    if (a.res_out) a.res_out = static_cast<char*>(a.res_out) + bytes;
    if (a.y) a.y = static_cast<char*>(a.y) + bytes;
    if (a.q) a.q += n;
    if (a.scale) a.scale += a.rows;
  }
}

template <int DT, bool RES, bool Q8, int G, int P>
void rows_launch(const NormArgs& a, hipStream_t st) {
  constexpr int NT = G > 256 ? G : 256, R = NT / G;  // rows of a workgroup
  in_slices<DT>(a, kMaxThreads / NT * R, [st](const NormArgs& a) {
    const dim3 grid(static_cast<unsigned>(ceil_div(a.rows, R)));
    hipLaunchKernelGGL((norm_rows<DT, RES, Q8, G, P>), grid, dim3(NT), 0, st, a);
  });
}

// The smallest group whose lanes hold the row in four pieces or fewer: more rows
// a wave, more loads in flight (262144 x 512 in bf16 with the residual: 173 us).
// A few rows only wait for their own chain, which a piece a lane makes shortest.
template <int DT, bool RES, bool Q8>
void norm_launch_as(const NormArgs& a, hipStream_t st) {
  const int pieces = a.d / Vec<DT>::N;
  if (a.rows <= kFewRows && pieces > 16 && pieces <= 64)
    rows_launch<DT, RES, Q8, 64, 1>(a, st);
  else if (pieces <= 16)
    rows_launch<DT, RES, Q8, 16, 1>(a, st);
  else if (pieces <= 32)
    rows_launch<DT, RES, Q8, 16, 2>(a, st);
  else if (pieces <= 64)
    rows_launch<DT, RES, Q8, 16, 4>(a, st);
  else if (pieces <= 128)
    rows_launch<DT, RES, Q8, 64, 2>(a, st);
  else if (pieces <= 256)
    rows_launch<DT, RES, Q8, 64, 4>(a, st);
  else if (pieces <= 1024)
    rows_launch<DT, RES, Q8, 256, 4>(a, st);
  else if (pieces <= 4096)
    rows_launch<DT, RES, Q8, 1024, 4>(a, st);
  else
    in_slices<DT>(a, kMaxThreads / 1024, [st](const NormArgs& a) {
      hipLaunchKernelGGL((norm_long<DT, RES, Q8>), dim3(static_cast<unsigned>(a.rows)), dim3(1024), 0, st, a);
    });
}

template <int DT>
void norm_launch_type(const NormArgs& a, hipStream_t st) {
  if (a.res)
    a.q ? norm_launch_as<DT, true, true>(a, st) : norm_launch_as<DT, true, false>(a, st);
  else
    a.q ? norm_launch_as<DT, false, true>(a, st) : norm_launch_as<DT, false, false>(a, st);
}

int norm_launch(const NormArgs& a, int dtype, void* stream) {
  if (a.rows == 0) return BLLM_OK;
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (dtype == BLLM_F32)
    norm_launch_type<BLLM_F32>(a, st);
  else
    norm_launch_type<BLLM_BF16>(a, st);
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
