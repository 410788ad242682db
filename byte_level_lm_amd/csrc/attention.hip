// Softmax attention: packed prompts, and one new token of each stream over its pages.
//
//   s_ij = scale q_i.k_j (capped, lowered by distance),  o_i = sum_j e^{s_ij - m} v_j / sum_j e^{s_ij - m}
//
// in one pass over the keys with the running maximum m and sum.  A wave has a
// query of a head: a lane a key of 64 for the scores, then a lane four columns of v.
#include "attention.h"

namespace bllm {
namespace {

constexpr int kWaves = 4;

struct AttArgs {
  const uint16_t *q, *k, *v;            // dense keys and values
  const void *k_pages, *v_pages;        // or pages
  const float *k_scale, *v_scale;
  Pages pages;
  const int64_t *offsets, *k_offsets;
  const int32_t* lengths;
  uint16_t* o;
  int64_t total, total_k, q_stride, k_stride, v_stride;
  int nseq, hq, hkv, d;
  Mask mask;
};

template <bool PAGED, bool Q8>
__global__ __launch_bounds__(64 * kWaves) void attend(AttArgs a) {
  __shared__ float sQ[kWaves][256], sP[kWaves][64];
  __shared__ int64_t sRow[kWaves][64];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, group = a.hq / a.hkv;
  const int64_t work = a.total * a.hq;
  for (int64_t i = int64_t(blockIdx.x) * kWaves + w; i < work; i += int64_t(gridDim.x) * kWaves) {
    const int64_t row = i / a.hq;
    const int h = static_cast<int>(i - row * a.hq), kh = h / group;
    int s, keys, t;
    int64_t k0 = 0;
    if (PAGED) {
      s = static_cast<int>(row);
      keys = min(max(a.lengths[s], 0), a.pages.cols << a.pages.shift);
      t = keys - 1;
    } else {
      s = wave_find(a.nseq, row, [&](int j) { return a.offsets[j]; });
      int64_t t0, t1, k1;
      seq_rows(a.offsets, s, a.total, &t0, &t1);
      seq_rows(a.k_offsets, s, a.total_k, &k0, &k1);
      if (row < t0 || row >= t1) continue;
      keys = static_cast<int>(k1 - k0);
      t = static_cast<int>(row - t0 + keys - (t1 - t0));
    }
    const int prefix = a.mask.prefix ? a.mask.prefix[s] : 0;
    const float slope = a.mask.slopes ? a.mask.slopes[h] : 0.0f;
    for (int c = lane; c < 256; c += 64)
      sQ[w][c] = c < a.d ? bf16_to_f32(a.q[row * a.q_stride + h * a.d + c]) : 0.0f;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "workgroup");
    float m = -INFINITY, l = 0.0f, o[4] = {};
    for (int j0 = 0; j0 < keys; j0 += 64) {
      const int j = j0 + lane;
      bool seen = j < keys && (j < prefix || ((!a.mask.causal || j <= t) && (!a.mask.window || abs(t - j) < a.mask.window)));
      int64_t r = k0 + j;
      if (PAGED) {
        r = seen ? a.pages.row(s, j) : -1;
        seen = r >= 0;
        r += static_cast<int64_t>(kh) << a.pages.shift;
      }
      float x = -INFINITY;
      if (seen) {
        x = 0.0f;
        for (int c = 0; c < a.d; ++c) {
          float k;
          if (!PAGED) k = bf16_to_f32(a.k[r * a.k_stride + kh * a.d + c]);
          else if (Q8) k = static_cast<const int8_t*>(a.k_pages)[r * a.d + c];
          else k = bf16_to_f32(static_cast<const uint16_t*>(a.k_pages)[r * a.d + c]);
          x = fmaf(sQ[w][c], k, x);
        }
        if (Q8) x *= a.k_scale[r];
        x *= a.mask.scale;
        if (a.mask.cap > 0.0f) x = a.mask.cap * tanhf(x / a.mask.cap);
        if (a.mask.slopes) x -= slope * static_cast<float>(abs(t - j));
      }
      if (!__ballot(seen)) continue;
      float top = x;
      for (int off = 32; off; off >>= 1) top = fmaxf(top, __shfl_xor(top, off, 64));
      const float m2 = fmaxf(m, top), safe = m2 == -INFINITY ? 0.0f : m2;
      const float p = seen ? expf(x - safe) : 0.0f, fall = expf(m - safe);
      l = l * fall + wave_sum(p);
      m = m2;
      sP[w][lane] = p;
      sRow[w][lane] = seen ? r : -1;
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "workgroup");
      for (int e = 0; e < 4; ++e) o[e] *= fall;
      for (int n = 0; n < 64; ++n) {
        const int64_t rn = sRow[w][n];
        if (rn < 0) continue;
        float pn = sP[w][n];
        if (Q8) pn *= a.v_scale[rn];
        for (int e = 0; e < 4; ++e) {
          const int c = 4 * lane + e;
          if (c >= a.d) continue;
          float v;
          if (!PAGED) v = bf16_to_f32(a.v[rn * a.v_stride + kh * a.d + c]);
          else if (Q8) v = static_cast<const int8_t*>(a.v_pages)[rn * a.d + c];
          else v = bf16_to_f32(static_cast<const uint16_t*>(a.v_pages)[rn * a.d + c]);
          o[e] = fmaf(pn, v, o[e]);
        }
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "workgroup");
    }
    for (int e = 0; e < 4; ++e)
      if (4 * lane + e < a.d)
        a.o[(row * a.hq + h) * a.d + 4 * lane + e] = l == 0.0f ? 0 : f32_to_bf16(o[e] / l);
  }
}

unsigned grid_of(int64_t work) {
  const int64_t n = ceil_div(work, kWaves);
  return static_cast<unsigned>(n < (1 << 20) ? n : 1 << 20);
}

}  // namespace
}  // namespace bllm

using namespace bllm;

extern "C" size_t bllm_attention_workspace(int64_t nseq, int64_t total, int64_t total_k, int64_t hq, int64_t hkv,
                                           int64_t d) {
  return nseq < 1 || total < 0 || total_k < 0 || hq < 1 || hkv < 1 || d < 1 ? 0 : 16;
}

extern "C" int bllm_attention(const void* q, const void* k, const void* v, int dtype, const int64_t* offsets,
                              const int64_t* k_offsets, int64_t nseq, int64_t total, int64_t total_k, int64_t hq,
                              int64_t hkv, int64_t d, int64_t q_stride, int64_t k_stride, int64_t v_stride,
                              double scale, int causal, int64_t window, double cap, const float* slopes,
                              const int32_t* prefix, void* o_out, void* ws, size_t ws_bytes, void* stream) {
  AttArgs a{};
  int rc = heads_check(hq, hkv, d);
  if (rc == BLLM_E_INVAL || nseq < 1 || total < 0 || total_k < 0 || !offsets || (!k_offsets && total != total_k) ||
      (total > 0 && (!q || !o_out)) || (total_k > 0 && (!k || !v)) || q_stride < hq * d || k_stride < hkv * d ||
      v_stride < hkv * d || mask_make(scale, causal, window, cap, slopes, prefix, &a.mask) != BLLM_OK)
    return BLLM_E_INVAL;
  if (rc != BLLM_OK || dtype != BLLM_BF16 || nseq > kMaxSeqs || total > kMaxTokens || total_k > kMaxTokens ||
      !stride_ok(q_stride) || !stride_ok(k_stride) || !stride_ok(v_stride) || !aligned16(q) || !aligned16(k) ||
      !aligned16(v) || !aligned16(o_out))
    return BLLM_E_NOTSUP;
  if (!ws || ws_bytes < bllm_attention_workspace(nseq, total, total_k, hq, hkv, d)) return BLLM_E_WS;
  if (total == 0) return BLLM_OK;
  a.q = static_cast<const uint16_t*>(q);
  a.k = static_cast<const uint16_t*>(k);
  a.v = static_cast<const uint16_t*>(v);
  a.offsets = offsets;
  a.k_offsets = k_offsets ? k_offsets : offsets;
  a.o = static_cast<uint16_t*>(o_out);
  a.total = total;
  a.total_k = total_k;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.nseq = static_cast<int>(nseq);
  a.hq = static_cast<int>(hq);
  a.hkv = static_cast<int>(hkv);
  a.d = static_cast<int>(d);
  hipLaunchKernelGGL((attend<false, false>), dim3(grid_of(total * hq)), dim3(64 * kWaves), 0,
                     static_cast<hipStream_t>(stream), a);
  return launch_status();
}
