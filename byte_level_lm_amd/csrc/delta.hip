// Gated delta rule: a head's state S [dk x dv] decays, loses what it holds
// under the key and takes the new value there,
//   u_t = beta_t (v_t - a_t S_{t-1}^T k_t),  S_t = a_t S_{t-1} + k_t u_t^T,
//   o_t = scale S_t^T q_t,                   a_t = exp(g_t),
// with q and k scaled to unit length on request (x / sqrt(|x|^2 + 1e-6)).
// States, gates and every sum are fp32.
//
// Recurrent form.  A wave owns 32 columns of one head's state: lane (i, c),
// i = lane / 8, c = lane % 8, holds rows R i .. R i + R - 1 of columns
// 4 c .. 4 c + 3 in registers.  Both sums over dk that a token needs are taken
// from the state before it,
//   S_t^T q = a_t S_{t-1}^T q + (k.q) u_t,
// so a token costs one reduction over the eight lane groups.
#include "common.h"

namespace bllm {
namespace {

constexpr float kL2Eps = 1e-6f;

// one call's arguments; rows of q, k and v lie q_stride, k_stride, v_stride elements apart
struct DeltaArgs {
  const uint16_t *q, *k, *v;
  const float *g, *beta;
  const int64_t* offsets;   // [nseq + 1], or null: sequence s is the one token s
  const int32_t* slots;     // [nseq] rows of the states, or null: row s
  const float* state_in;    // or null: zero
  float* state_out;         // or null
  uint16_t* o;
  int64_t total, qs, ks, vs, nslots;
  int nseq, hk, hv, dk, dv;
  float scale;
  int unit;
};

// sum over the lanes that hold the same columns (lane % 8)
__device__ inline float column_sum(float x) {
  x += __shfl_xor(x, 8, kWave);
  x += __shfl_xor(x, 16, kWave);
  return x + __shfl_xor(x, 32, kWave);
}

// R = ceil(dk / 8) rounded up to 2, 4, 8 or 16 rows for each lane
template <int R>
__global__ __launch_bounds__(256) void delta_recurrent(DeltaArgs a) {
  const int lane = threadIdx.x & 63;
  const int col = (blockIdx.x * 4 + (threadIdx.x >> 6)) * 32 + 4 * (lane & 7);
  const int h = blockIdx.y, s = blockIdx.z, kh = h / (a.hv / a.hk);
  const int r0 = (lane >> 3) * R;
  if (col - 4 * (lane & 7) >= a.dv) return;
  int64_t t0 = s, t1 = s + 1, slot = s;
  if (a.offsets) {
    t0 = min(max(a.offsets[s], int64_t(0)), a.total);
    t1 = min(max(a.offsets[s + 1], t0), a.total);
  }
  if (a.slots) slot = a.slots[s];
  const bool held = slot >= 0 && slot < a.nslots, in = col < a.dv;
  const int64_t at = ((held ? slot : 0) * a.hv + h) * a.dk * static_cast<int64_t>(a.dv) + col;
  float4 S[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    S[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (a.state_in && held && in && r0 + i < a.dk)
      S[i] = *reinterpret_cast<const float4*>(a.state_in + at + static_cast<int64_t>(r0 + i) * a.dv);
  }
  for (int64_t t = t0; t < t1; ++t) {
    float q[R], k[R];
    float kk = 0.0f, qq = 0.0f, kq = 0.0f;
    float4 xk = make_float4(0, 0, 0, 0), xq = make_float4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const bool row = r0 + i < a.dk;
      q[i] = row ? bf16_to_f32(a.q[t * a.qs + static_cast<int64_t>(kh) * a.dk + r0 + i]) : 0.0f;
      k[i] = row ? bf16_to_f32(a.k[t * a.ks + static_cast<int64_t>(kh) * a.dk + r0 + i]) : 0.0f;
      kk += k[i] * k[i];
      qq += q[i] * q[i];
      kq += k[i] * q[i];
      xk.x += S[i].x * k[i]; xk.y += S[i].y * k[i]; xk.z += S[i].z * k[i]; xk.w += S[i].w * k[i];
      xq.x += S[i].x * q[i]; xq.y += S[i].y * q[i]; xq.z += S[i].z * q[i]; xq.w += S[i].w * q[i];
    }
    kq = column_sum(kq);
    float rk = 1.0f, rq = 1.0f;
    if (a.unit) {
      rk = 1.0f / sqrtf(column_sum(kk) + kL2Eps);
      rq = 1.0f / sqrtf(column_sum(qq) + kL2Eps);
    }
    xk.x = column_sum(xk.x); xk.y = column_sum(xk.y); xk.z = column_sum(xk.z); xk.w = column_sum(xk.w);
    xq.x = column_sum(xq.x); xq.y = column_sum(xq.y); xq.z = column_sum(xq.z); xq.w = column_sum(xq.w);
    const float al = expf(a.g[t * a.hv + h]), be = a.beta[t * a.hv + h];
    float vv[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (in) {
      const uint2 p = *reinterpret_cast<const uint2*>(a.v + t * a.vs + static_cast<int64_t>(h) * a.dv + col);
      vv[0] = bf16_to_f32(p.x & 0xFFFFu); vv[1] = bf16_to_f32(p.x >> 16);
      vv[2] = bf16_to_f32(p.y & 0xFFFFu); vv[3] = bf16_to_f32(p.y >> 16);
    }
    const float ak = al * rk;
    const float u[4] = {be * (vv[0] - ak * xk.x), be * (vv[1] - ak * xk.y), be * (vv[2] - ak * xk.z),
                        be * (vv[3] - ak * xk.w)};
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const float kr = k[i] * rk;
      S[i].x = al * S[i].x + kr * u[0]; S[i].y = al * S[i].y + kr * u[1];
      S[i].z = al * S[i].z + kr * u[2]; S[i].w = al * S[i].w + kr * u[3];
    }
    if (in && lane < 8) {
      const float c = a.scale * rq, d = kq * rk;
      uint2 p;
      p.x = f32_to_bf16(c * (al * xq.x + d * u[0])) |
            static_cast<uint32_t>(f32_to_bf16(c * (al * xq.y + d * u[1]))) << 16;
      p.y = f32_to_bf16(c * (al * xq.z + d * u[2])) |
            static_cast<uint32_t>(f32_to_bf16(c * (al * xq.w + d * u[3]))) << 16;
      *reinterpret_cast<uint2*>(a.o + (t * a.hv + h) * a.dv + col) = p;
    }
  }
  if (!a.state_out || !held || !in) return;
#pragma unroll
  for (int i = 0; i < R; ++i)
    if (r0 + i < a.dk) *reinterpret_cast<float4*>(a.state_out + at + static_cast<int64_t>(r0 + i) * a.dv) = S[i];
}

void recurrent_launch(const DeltaArgs& a, hipStream_t st) {
  const dim3 grid(static_cast<unsigned>(ceil_div(a.dv, 128)), static_cast<unsigned>(a.hv),
                  static_cast<unsigned>(a.nseq));
  if (a.dk <= 16)
    hipLaunchKernelGGL(delta_recurrent<2>, grid, dim3(256), 0, st, a);
  else if (a.dk <= 32)
    hipLaunchKernelGGL(delta_recurrent<4>, grid, dim3(256), 0, st, a);
  else if (a.dk <= 64)
    hipLaunchKernelGGL(delta_recurrent<8>, grid, dim3(256), 0, st, a);
  else
    hipLaunchKernelGGL(delta_recurrent<16>, grid, dim3(256), 0, st, a);
}

// sizes, strides and alignment shared by the prompt and the step
int delta_check(const DeltaArgs& a, int dtype, int64_t nseq, int64_t hk, int64_t hv, int64_t dk, int64_t dv) {
  if (nseq < 1 || a.total < 0 || hk < 1 || hv < hk || hv % hk != 0 || dk < 1 || dv < 1 || a.qs < hk * dk ||
      a.ks < hk * dk || a.vs < hv * dv || !(a.scale == a.scale))
    return BLLM_E_INVAL;
  if (a.total > 0 && (!a.q || !a.k || !a.v || !a.g || !a.beta || !a.o)) return BLLM_E_INVAL;
  if (dtype != BLLM_BF16 || dk % 8 != 0 || dk > 128 || dv % 8 != 0 || dv > 1024 || hv > 1024 || nseq > 65535 ||
      a.total >= (int64_t(1) << 31) || a.qs % 8 != 0 || a.ks % 8 != 0 || a.vs % 8 != 0 || !aligned16(a.q) ||
      !aligned16(a.k) || !aligned16(a.v) || !aligned16(a.o) || !aligned16(a.state_in) || !aligned16(a.state_out))
    return BLLM_E_NOTSUP;
  return BLLM_OK;
}

}  // namespace
}  // namespace bllm

using namespace bllm;

extern "C" size_t bllm_gated_delta_workspace(int64_t nseq, int64_t total, int64_t hv, int64_t dk, int64_t dv) {
  if (nseq < 1 || total < 0 || hv < 1 || dk < 1 || dv < 1) return 0;
  return 256;
}

extern "C" int bllm_gated_delta(const void* q, const void* k, const void* v, const float* g, const float* beta,
                                int dtype, const int64_t* offsets, int64_t nseq, int64_t total, int64_t hk,
                                int64_t hv, int64_t dk, int64_t dv, int64_t q_stride, int64_t k_stride,
                                int64_t v_stride, double scale, int unit_qk, const float* state_in,
                                float* state_out, void* o_out, void* ws, size_t ws_bytes, void* stream) {
  if (!offsets) return BLLM_E_INVAL;
  DeltaArgs a{static_cast<const uint16_t*>(q), static_cast<const uint16_t*>(k), static_cast<const uint16_t*>(v),
              g, beta, offsets, nullptr, state_in, state_out, static_cast<uint16_t*>(o_out), total, q_stride,
              k_stride, v_stride, nseq, static_cast<int>(nseq), static_cast<int>(hk), static_cast<int>(hv),
              static_cast<int>(dk), static_cast<int>(dv), static_cast<float>(scale), unit_qk != 0};
  const int rc = delta_check(a, dtype, nseq, hk, hv, dk, dv);
  if (rc != BLLM_OK) return rc;
  if (!ws || ws_bytes < bllm_gated_delta_workspace(nseq, total, hv, dk, dv) || !aligned16(ws)) return BLLM_E_WS;
  recurrent_launch(a, static_cast<hipStream_t>(stream));
  return launch_status();
}

extern "C" int bllm_gated_delta_step(const void* q, const void* k, const void* v, const float* g,
                                     const float* beta, int dtype, int64_t nseq, int64_t hk, int64_t hv,
                                     int64_t dk, int64_t dv, int64_t q_stride, int64_t k_stride,
                                     int64_t v_stride, double scale, int unit_qk, const float* state_in,
                                     float* state_out, const int32_t* slots, int64_t nslots, void* o_out,
                                     void* stream) {
  if (!state_in || !state_out || nslots < 1 || (!slots && nslots < nseq)) return BLLM_E_INVAL;
  DeltaArgs a{static_cast<const uint16_t*>(q), static_cast<const uint16_t*>(k), static_cast<const uint16_t*>(v),
              g, beta, nullptr, slots, state_in, state_out, static_cast<uint16_t*>(o_out), nseq, q_stride,
              k_stride, v_stride, nslots, static_cast<int>(nseq), static_cast<int>(hk), static_cast<int>(hv),
              static_cast<int>(dk), static_cast<int>(dv), static_cast<float>(scale), unit_qk != 0};
  const int rc = delta_check(a, dtype, nseq, hk, hv, dk, dv);
  if (rc != BLLM_OK) return rc;
  recurrent_launch(a, static_cast<hipStream_t>(stream));
  return launch_status();
}
