// Softmax attention of packed prompts.
//
//   s_ij = scale q_i.k_j (capped, lowered by distance),  o_i = sum_j 2^{x_ij - m_i} v_j / sum_j 2^{x_ij - m_i},  x = s log2 e
//
// Bound by the matrix cores, with the exponentials close behind: 32 keys cost a
// wave 32 exponentials' issue beside 16 instructions of 32 x 32 x 16.  A
// workgroup has 128 queries of a head, a wave 32 of them; tiles of BN keys go through LDS, two
// buffers of them filled without registers, in one pass with the running maximum and sum.
//
// Registers: scores come as S^T = K Q^T, of which a lane (half h of the wave)
// has its query lane % 32 and keys 8 (r / 4) + 4 h + r % 4 of each 32.  The second product
// O^T = V^T P^T takes 16 keys in the order 4 h + {0..3}, 8 + 4 h + {0..3}: the
// weights as the lane has them, and V's columns by transposing LDS reads.  So
// weights never leave their lane, and maximum, sum and the factor of O are one number a lane.
#include "attention.h"

namespace bllm {
namespace {

typedef float floatx16 __attribute__((ext_vector_type(16)));
typedef short shortx4 __attribute__((ext_vector_type(4)));
typedef __amdgpu_buffer_rsrc_t Buffer;

constexpr int kRows = 128;       // queries of a workgroup
constexpr int kWaves = 4;
constexpr int kXcds = 8;
constexpr int kRun = 64;         // neighbouring workgroups that one XCD takes in a row
constexpr uint32_t kOutside = 0x7FFFFFF0u;  // an offset past every buffer: reads as zero
constexpr float kSlack = 8.0f;   // how far (log2) scores may pass the maximum that weights are taken against

struct AttArgs {
  const uint16_t *q, *k, *v;
  const int64_t *offsets, *k_offsets;
  uint16_t* o;
  int64_t total, total_k, q_stride, k_stride, v_stride;
  int64_t first, units, slots;   // this launch's first unit of work, all of them, 128-query slots
  int nseq, hq, hkv, group, d;
  Mask mask;
};

__device__ inline void to_lds(Buffer b, uint32_t at, void* lds) {
  typedef __attribute__((address_space(3))) void lds_void;
  __builtin_amdgcn_raw_ptr_buffer_load_lds(b, (lds_void*)lds, 16, at, 0, 0, 0);
}
// all of the wave's loads have landed, then the workgroup's
__device__ inline void landed_barrier() {
  __asm__ volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0x0070);  // vmcnt(0) lgkmcnt(0)
  __builtin_amdgcn_s_barrier();
  __asm__ volatile("" ::: "memory");
}
__device__ inline uint2 read_tr(const uint16_t* p) {
  typedef __attribute__((address_space(3))) shortx4 lds_s4;
  const shortx4 v = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4*)p);
  return __builtin_bit_cast(uint2, v);
}

// 16-byte piece p of row r of a tile lies at piece p ^ exchange(r): sixteen rows' pieces p lie in all the banks
// (K's reads), and so do four neighbouring rows' four pieces 4 i .. 4 i + 3 (V's transposing reads)
template <int D>
__device__ inline int exchange(int r) {
  return D == 64 ? 4 * (r >> 1 & 1) | (r >> 2 & 3) : 4 * (r & 3) | (r >> 2 & 3);
}

// What one query sees: keys lo .. hi and those below front.
struct Sight {
  int lo, hi, front;
  __device__ inline bool has(int j) const { return (j >= lo && j <= hi) || j < front; }
};
__device__ inline Sight sight(const Mask& m, int t, int keys, int front) {
  Sight s;
  s.lo = m.window ? t - m.window + 1 : 0;
  s.hi = min(m.causal ? t : m.window ? t + m.window - 1 : keys - 1, keys - 1);
  s.front = front;
  return s;
}

// A query on its own, where v has values that are not finite: products with a
// weight of zero would carry them to queries that do not see their keys.  A
// wave takes 64 keys at a time, a lane a key, then a lane four columns of v.
__device__ inline void query_alone(const AttArgs& a, int64_t row, int h, int64_t k0, int t, Sight see,
                                                      float slope) {
  const int lane = lane_id(), kh = h / a.group, d = a.d;
  const uint16_t* q = a.q + row * a.q_stride + static_cast<int64_t>(h) * d;
  float m = -INFINITY, l = 0.0f, o[4] = {};
  for (int j0 = 0; j0 <= max(see.hi, see.front - 1); j0 += kWave) {
    const int j = j0 + lane;
    const bool has = see.has(j);
    if (!__ballot(has)) continue;
    float x = -INFINITY;
    if (has) {
      const uint16_t* k = a.k + (k0 + j) * a.k_stride + static_cast<int64_t>(kh) * d;
      x = 0.0f;
      for (int c = 0; c < d; ++c) x = fmaf(bf16_to_f32(q[c]), bf16_to_f32(k[c]), x);
      x *= a.mask.scale;
      if (a.mask.cap > 0.0f) x = capped(x, a.mask.cap, 2.0f * kLog2e / a.mask.cap);
      x = (x - slope * static_cast<float>(abs(t - j))) * kLog2e;
    }
    float top = x;
    for (int off = 32; off >= 1; off >>= 1) top = fmaxf(top, __shfl_xor(top, off, kWave));
    const float now = fmaxf(m, top), base = now == -INFINITY ? 0.0f : now, fall = exp2_fast(m - base);
    const float p = exp2_fast(x - base);
    l = l * fall + wave_sum(p);
    m = now;
    for (int e = 0; e < 4; ++e) o[e] *= fall;
    for (int n = 0; n < kWave; ++n) {
      if (!see.has(j0 + n)) continue;
      const float w = __shfl(p, n, kWave);
      const uint16_t* v = a.v + (k0 + j0 + n) * a.v_stride + static_cast<int64_t>(kh) * d + 4 * lane;
      if (4 * lane < d)
        for (int e = 0; e < 4; ++e) o[e] = fmaf(w, bf16_to_f32(v[e]), o[e]);
    }
  }
  if (4 * lane < d)
    *reinterpret_cast<uint2*>(a.o + (row * a.hq + h) * d + 4 * lane) =
        make_uint2(pack2(o[0] / l, o[1] / l), pack2(o[2] / l, o[3] / l));
}

// GEN: with a cap or slopes
template <int D, int BN, bool GEN>
__global__ __launch_bounds__(64 * kWaves, 2) void prompt_tiles(AttArgs a) {
  constexpr int NS = D / 16;               // steps of the first product
  constexpr int NB = D / 32;               // 32-column blocks of the second
  constexpr int NK = BN / 32;              // 32-key blocks of a tile
  constexpr int RPI = 512 / D;             // rows of a 1 KB load
  constexpr int U = BN / RPI / kWaves;     // loads a wave makes for K, and for V
  __shared__ __align__(1024) uint16_t sK[2][BN * D], sV[2][BN * D];
  const int lane = threadIdx.x & 63, qi = lane & 31, half = lane >> 5;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);

  // Unit of work: kRun neighbours go to one XCD.  Units of a key head follow
  // each other, of these a sequence's, the last queries (with the most keys) first.
  int64_t unit = a.first + blockIdx.x;
  {
    const int64_t full = a.units / (kRun * kXcds) * (kRun * kXcds);
    if (unit < full) {
      const int64_t in = unit % (kRun * kXcds);
      unit += (in % kXcds) * kRun + in / kXcds - in;
    }
  }
  const int64_t per = a.slots * a.group;
  const int kh = static_cast<int>(unit / per);
  const int64_t slot = unit % per / a.group;
  const int h = kh * a.group + static_cast<int>(unit % a.group);
  const int s = wave_find(a.nseq, slot, [&](int i) { return min(max(a.offsets[i], int64_t(0)), a.total) / kRows + i; });
  int64_t t0, t1, k0, k1;
  seq_rows(a.offsets, s, a.total, &t0, &t1);
  seq_rows(a.k_offsets, s, a.total_k, &k0, &k1);
  const int n = static_cast<int>(t1 - t0), keys = static_cast<int>(k1 - k0);
  const int back = static_cast<int>(slot - (t0 / kRows + s)), blocks = (n + kRows - 1) / kRows;
  if (back < 0 || back >= blocks) return;
  const int first = (blocks - 1 - back) * kRows;
  const int shift = keys - n;                            // position of query 0
  const int front = a.mask.prefix ? min(max(a.mask.prefix[s], 0), keys) : 0;

  // the tiles that some query of the workgroup sees: [0, b) then [e, f)
  const Sight low = sight(a.mask, first + shift, keys, front), high = sight(a.mask, min(first + kRows, n) - 1 + shift, keys, front);
  int from = max(low.lo, 0), to = high.hi + 1, ahead = front;
  if (ahead >= from) {
    from = 0;
    to = max(to, ahead);
    ahead = 0;
  }
  const int tb = (ahead + BN - 1) / BN, te = max(from / BN, tb), tiles = tb + max((to + BN - 1) / BN - te, 0);
  const auto key_of = [&](int i) { return (i < tb ? i : i - tb + te) * BN; };
  // the wave's own queries
  const int i0 = first + 32 * w, p0 = i0 + shift, p1 = min(i0 + 32, n) - 1 + shift;
  const bool some = i0 < n;
  const Sight w0 = sight(a.mask, p0, keys, front), w1 = sight(a.mask, p1, keys, front);
  const int t = p0 + qi;
  const Sight see = sight(a.mask, t, keys, front);

  // queries: 8 values of each 16, negated for a negative scale, so that the largest product has the largest score
  uint4 fq[NS];
  {
    const uint16_t* q = a.q + (t0 + i0 + qi) * a.q_stride + static_cast<int64_t>(h) * a.d + 8 * half;
    const uint32_t sign = a.mask.scale < 0.0f ? 0x80008000u : 0u;
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      uint4 x = i0 + qi < n && 16 * i + 8 * half < a.d ? *reinterpret_cast<const uint4*>(q + 16 * i) : make_uint4(0, 0, 0, 0);
      fq[i] = make_uint4(x.x ^ sign, x.y ^ sign, x.z ^ sign, x.w ^ sign);
    }
  }
  // x = c1 times the product; with GEN the product becomes x itself
  const float size = fabsf(a.mask.scale), c1 = GEN ? 1.0f : fmaxf(size * kLog2e, 1e-30f);
  const float c2 = GEN && a.mask.cap > 0.0f ? 2.0f * kLog2e / a.mask.cap : 0.0f;
  const float slope = GEN && a.mask.slopes ? a.mask.slopes[h] : 0.0f;

  // loads: where the lane's piece of each 1 KB lies
  uint32_t ko[U], vo[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int r = (u * kWaves + w) * RPI + lane / (D / 8), p = (lane % (D / 8)) ^ exchange<D>(r);
    const bool in = 8 * p < a.d;
    ko[u] = in ? static_cast<uint32_t>(2 * (r * a.k_stride + 8 * p)) : kOutside;
    vo[u] = in ? static_cast<uint32_t>(2 * (r * a.v_stride + 8 * p)) : kOutside;
  }
  const uint16_t* kb = a.k + k0 * a.k_stride + static_cast<int64_t>(kh) * a.d;
  const uint16_t* vb = a.v + k0 * a.v_stride + static_cast<int64_t>(kh) * a.d;
  const auto load = [&](int j0, uint16_t* K, uint16_t* V) __attribute__((always_inline)) {
    const int rows = min(keys - j0, BN);  // rows past the end read as zero
    const Buffer bk = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(kb + j0 * a.k_stride), 0,
                                                        static_cast<int>(2 * rows * a.k_stride), 0x00027000);
    const Buffer bv = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(vb + j0 * a.v_stride), 0,
                                                        static_cast<int>(2 * rows * a.v_stride), 0x00027000);
#pragma unroll
    for (int u = 0; u < U; ++u) to_lds(bk, ko[u], K + (u * kWaves + w) * 512);
#pragma unroll
    for (int u = 0; u < U; ++u) to_lds(bv, vo[u], V + (u * kWaves + w) * 512);
  };

  // reads: K's row qi of 32, pieces 2 i + half; V's rows 4 half + (lane % 16) / 4 of 8, columns by lane / 16 % 2 and lane % 4
  const int kx = half ^ exchange<D>(qi), kat = qi * D;
  const int vr = 4 * half + (lane >> 2 & 3), vp = 2 * (lane >> 4 & 1) + (lane >> 1 & 1);
  const int vat = vr * D + 4 * (lane & 1);
  const int vx0 = vp ^ exchange<D>(vr), vx1 = vp ^ exchange<D>(vr + 8);

  float m = -INFINITY, l = 0.0f;
  floatx16 o[NB] = {};
  const auto step = [&](int i, uint16_t* nK, uint16_t* nV, const uint16_t* __restrict__ cK,
                        const uint16_t* __restrict__ cV) __attribute__((always_inline)) {
    landed_barrier();
    const int j0 = key_of(i);
    if (i + 1 < tiles) load(key_of(i + 1), nK, nV);
    // no query of the wave sees a key of the tile
    if (!some || (j0 >= front && (j0 > w1.hi || j0 + BN <= w0.lo))) return;
    floatx16 x[NK] = {};
#pragma unroll
    for (int e = 0; e < NS; ++e)
#pragma unroll
      for (int b = 0; b < NK; ++b) {
        const uint4 f = *reinterpret_cast<const uint4*>(cK + 32 * b * D + kat + 8 * (kx ^ 2 * e));
        x[b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(as_frag(f), as_frag(fq[e]), x[b], 0, 0, 0);
      }
    if (GEN) {
#pragma unroll
      for (int b = 0; b < NK; ++b)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          float y = x[b][r] * size;
          if (c2 != 0.0f) y = capped(y, a.mask.cap, c2);
          x[b][r] = (y - slope * static_cast<float>(abs(t - (j0 + 32 * b + 8 * (r / 4) + 4 * half + r % 4)))) * kLog2e;
        }
    }
    // every query of the wave sees every key of the tile?
    const bool whole = j0 + BN <= front || (j0 >= w1.lo && j0 + BN - 1 <= w0.hi);
    if (!whole) {
#pragma unroll
      for (int b = 0; b < NK; ++b)
#pragma unroll
        for (int r = 0; r < 16; ++r)
          x[b][r] = see.has(j0 + 32 * b + 8 * (r / 4) + 4 * half + r % 4) ? x[b][r] : -INFINITY;
    }
    float top = x[0][0];
#pragma unroll
    for (int b = 0; b < NK; ++b)
#pragma unroll
      for (int r = 0; r < 16; ++r) top = fmaxf(top, x[b][r]);
    top = max_xor32(top) * c1;
    if (__any(top > m + kSlack)) {
      const float now = fmaxf(m, top), fall = exp2_fast(m - (now == -INFINITY ? 0.0f : now));
      m = now;
      l *= fall;
#pragma unroll
      for (int b = 0; b < NB; ++b) o[b] *= fall;
    }
    const float base = m == -INFINITY ? 0.0f : m;
    uint32_t p[NK][8];
#pragma unroll
    for (int b = 0; b < NK; ++b)
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        const float y0 = exp2_fast(fmaf(x[b][2 * r], c1, -base)), y1 = exp2_fast(fmaf(x[b][2 * r + 1], c1, -base));
        p[b][r] = pack2(y0, y1);
        l += low_half(p[b][r]) + high_half(p[b][r]);
      }
#pragma unroll
    for (int e = 0; e < 2 * NK; ++e) {  // 16 keys
      const bf16x8 fp = as_frag(make_uint4(p[e / 2][4 * (e % 2)], p[e / 2][4 * (e % 2) + 1], p[e / 2][4 * (e % 2) + 2],
                                           p[e / 2][4 * (e % 2) + 3]));
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const uint2 f0 = read_tr(cV + 16 * e * D + vat + 8 * (vx0 ^ 4 * b));
        const uint2 f1 = read_tr(cV + 16 * e * D + 8 * D + vat + 8 * (vx1 ^ 4 * b));
        o[b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(as_frag(make_uint4(f0.x, f0.y, f1.x, f1.y)), fp, o[b], 0, 0, 0);
      }
    }
  };
  if (tiles > 0) load(key_of(0), sK[0], sV[0]);
  for (int i = 0; i < tiles; i += 2) {
    step(i, sK[1], sV[1], sK[0], sV[0]);
    if (i + 1 < tiles) step(i + 1, sK[0], sV[0], sK[1], sV[1]);
  }
  if (!some) return;

  l = sum_xor32(l);
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  float odd = 0.0f;
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int r = 0; r < 16; ++r) odd = fmaf(o[b][r], 0.0f, odd);  // 0 x infinity and 0 x NaN are NaN
  odd = sum_xor32(odd);
  // lanes of the lower half take columns 0 .. 7 of each 16, of the upper half 8 .. 15
  const int64_t row = t0 + i0 + qi;
  uint16_t* out = a.o + (row * a.hq + h) * a.d + 8 * half;
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      uint32_t y[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) y[r] = pack2(o[b][8 * e + 2 * r] * inv, o[b][8 * e + 2 * r + 1] * inv);
      const auto u = __builtin_amdgcn_permlane32_swap(y[0], y[2], false, false);
      const auto v = __builtin_amdgcn_permlane32_swap(y[1], y[3], false, false);
      if (i0 + qi < n && 32 * b + 16 * e + 8 * half < a.d)
        *reinterpret_cast<uint4*>(out + 32 * b + 16 * e) = make_uint4(u[0], v[0], u[1], v[1]);
    }
  // scores were finite and outputs are not: those queries once more, one by one
  uint64_t again = __ballot(half == 0 && i0 + qi < n && odd != 0.0f && fabsf(l) < INFINITY);
  if (again) __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "workgroup");  // behind the stores above
  while (again) {
    const int i = __builtin_ctzll(again);
    again &= again - 1;
    query_alone(a, t0 + i0 + i, h, k0, p0 + i, sight(a.mask, p0 + i, keys, front), a.mask.slopes ? a.mask.slopes[h] : 0.0f);
  }
}

template <int D, int BN>
void launch(AttArgs a, hipStream_t st) {
  constexpr int64_t kMost = (int64_t(1) << 32) / (64 * kWaves) - 1;  // workgroups that one launch has threads for
  for (a.first = 0; a.first < a.units; a.first += kMost) {
    const dim3 grid(static_cast<unsigned>(a.units - a.first < kMost ? a.units - a.first : kMost)), block(64 * kWaves);
    if (a.mask.cap > 0.0f || a.mask.slopes)
      hipLaunchKernelGGL((prompt_tiles<D, BN, true>), grid, block, 0, st, a);
    else
      hipLaunchKernelGGL((prompt_tiles<D, BN, false>), grid, block, 0, st, a);
  }
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
  const int rc = heads_check(hq, hkv, d);
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
  a.slots = total / kRows + nseq;  // sequence s has slots offsets[s] / 128 + s and on
  a.units = a.slots * hq;
  a.nseq = static_cast<int>(nseq);
  a.hq = static_cast<int>(hq);
  a.hkv = static_cast<int>(hkv);
  a.group = static_cast<int>(hq / hkv);
  a.d = static_cast<int>(d);
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (d <= 64)
    launch<64, 64>(a, st);
  else if (d <= 128)
    launch<128, 64>(a, st);
  else
    launch<256, 32>(a, st);
  return launch_status();
}
