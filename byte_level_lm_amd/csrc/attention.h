// What the calls around attention share: the pages of a cache of keys and
// values, ragged batches, and which keys a query sees.
#pragma once

#include "common.h"

namespace bllm {

constexpr int64_t kMaxTokens = int64_t(1) << 30;  // positions and distances then fit 32 bits
constexpr int64_t kMaxHeads = 1024, kMaxSeqs = 65535, kMaxStride = int64_t(1) << 22;

// the pages of a call: rows of d values, [npages x hkv x page]
struct Pages {
  const int32_t* table;  // [nseq x cols]
  int cols, npages;
  int shift;             // page == 1 << shift
  int hkv, d;
  // row of position p of stream s for head 0, or -1 where it has no page (head h: + h << shift)
  __device__ inline int64_t row(int s, int64_t p) const {
    const int64_t c = p >> shift;
    if (p < 0 || c >= cols) return -1;
    const int id = table[static_cast<int64_t>(s) * cols + c];
    if (id < 0 || id >= npages) return -1;
    return ((static_cast<int64_t>(id) * hkv) << shift) + (p & ((1 << shift) - 1));
  }
};

__device__ inline int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ inline int64_t uniform64(int64_t v) {
  const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v));
  const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v >> 32));
  return static_cast<int64_t>(static_cast<uint64_t>(hi) << 32 | lo);
}

// rows of sequence s, cut at the arrays' `total` rows
__device__ inline void seq_rows(const int64_t* offsets, int s, int64_t total, int64_t* t0, int64_t* t1) {
  *t0 = uniform64(min(max(offsets[s], int64_t(0)), total));
  *t1 = uniform64(min(max(offsets[s + 1], *t0), total));
}

// Last s in [0, n) for which slot(s) <= t (slot ascending, slot(0) <= t), by a
// whole wave: every lane asks about one of 64 places at once, one trip to
// memory for up to 64 sequences, two for up to 4096.
template <typename Slot>
__device__ inline int wave_find(int n, int64_t t, const Slot& slot) {
  int lo = 0, hi = n;
  for (;;) {
    const int step = (hi - lo + kWave - 1) / kWave, at = lo + lane_id() * step;
    const bool before = at < hi && slot(min(at, n - 1)) <= t;
    const int k = max(static_cast<int>(__popcll(__ballot(before))) - 1, 0);
    lo += k * step;
    if (step == 1) return lo;
    hi = min(hi, lo + step);
  }
}

// ---------------------------------------------------------------- matrix instructions and lanes

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float floatx4 __attribute__((ext_vector_type(4)));

__device__ inline bf16x8 as_frag(uint4 v) { return __builtin_bit_cast(bf16x8, v); }
// two values to bf16, rounded to nearest even, the first in the lower half
__device__ inline uint32_t pack2(float a, float b) {
  bf16x2 v;
  v[0] = static_cast<__bf16>(a);
  v[1] = static_cast<__bf16>(b);
  return __builtin_bit_cast(uint32_t, v);
}
__device__ inline float low_half(uint32_t v) { return __uint_as_float(v << 16); }
__device__ inline float high_half(uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); }

// maximum and sum with the lane 32 away, and with the lane 16 away
__device__ inline float max_xor32(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ inline float max_xor16(float x) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ inline float sum_xor32(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
__device__ inline float sum_xor16(float x) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

constexpr float kLog2e = 1.4426950408889634f;
__device__ inline float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }  // v_exp_f32: 1 ulp, tiny results are zero

// scores and visibility, as the entry points take them
struct Mask {
  float scale;
  float cap;             // 0: none
  const float* slopes;   // or null
  const int32_t* prefix; // or null
  int window;            // 0: none
  int causal;
};

// cap * tanh(x / cap) as cap - 2 cap / (e^{2 x / cap} + 1): off by about 2^-22 cap
__device__ inline float capped(float x, float cap, float two_over_cap_log2e) {
  return cap - 2.0f * cap * __builtin_amdgcn_rcpf(exp2_fast(x * two_over_cap_log2e) + 1.0f);
}

// ---------------------------------------------------------------- shares of a query's keys

constexpr int kMaxSplits = 256;  // the lanes of a workgroup, which joins them

// What each of a query's shares of keys gave (queries: row * hq + head)
struct Shares {
  float* part;      // [queries x splits x d], not yet divided by the sum
  float2* stat;     // [queries x splits]: maximum and sum of the weights against it
  int splits;
};
inline size_t shares_bytes(int64_t queries, int64_t splits, int64_t d) {
  return 16 + (splits > 1 ? static_cast<size_t>(queries * splits) * (sizeof(float) * d + sizeof(float2)) : 0);
}
inline Shares shares_at(void* ws, int64_t queries, int64_t splits) {
  float2* stat = static_cast<float2*>(ws);
  return {reinterpret_cast<float*>(stat + (queries * splits + 1) / 2 * 2), stat, static_cast<int>(splits)};
}

__host__ __device__ inline int join_lanes(int d) { return d <= 32 ? 8 : d <= 64 ? 16 : d <= 128 ? 32 : 64; }  // of four values each

// Joins a query's shares.  Up to kFewSplits of them: join_lanes(d) lanes of a wave, with all
// their loads in flight at once (beside those of the wave's other queries).  More: WAVES waves, whose groups of
// lanes take the shares in turn; one has up to 64 of them, four are the workgroup.  Each of threads_to_join's
// sides: 61 streams of 5 shares, 8 heads of 64: 18.4 us in lanes, 19.9 in waves; 4 pieces of 64 to 512 queries of 8
// heads of 64 behind 8192 keys, 11 shares: 41 in waves, 54 in workgroups; 8 queries of 256 shares (262144 positions, one
// key head): 31 in workgroups, 71 in the 64 shares that a wave can join.
constexpr int kFewSplits = 8;

__device__ inline void join_few(const Shares& sh, int64_t query, bool mine, int d, uint16_t* o) {
  const int lanes = join_lanes(d), in = lane_id() & (lanes - 1), col = 4 * in, first = lane_id() - in;
  if (!mine) query = 0;
  const float2 st = in < sh.splits ? sh.stat[query * sh.splits + in] : make_float2(-INFINITY, 0.0f);
  const float* part = sh.part + query * sh.splits * d + (col < d ? col : 0);
  float4 v[kFewSplits];
#pragma unroll
  for (int i = 0; i < kFewSplits; ++i)
    if (i < sh.splits) v[i] = *reinterpret_cast<const float4*>(part + i * d);
  float top = st.y == 0.0f ? -INFINITY : st.x;
#pragma unroll
  for (int off = 4; off >= 1; off >>= 1) top = fmaxf(top, __shfl_xor(top, off, kWave));
  const float weight = st.y == 0.0f ? 0.0f : exp2_fast(st.x - (top == -INFINITY ? 0.0f : top));
  float sum = weight * st.y;
#pragma unroll
  for (int off = 4; off >= 1; off >>= 1) sum += __shfl_xor(sum, off, kWave);
  sum = __shfl(sum, first, kWave);
  float y[4] = {};
#pragma unroll
  for (int i = 0; i < kFewSplits; ++i)
    if (i < sh.splits) {
      const float w = __shfl(weight, first + i, kWave);
      const bool some = __shfl(st.y, first + i, kWave) != 0.0f;  // a share without keys has written no values
      y[0] = some ? fmaf(w, v[i].x, y[0]) : y[0];
      y[1] = some ? fmaf(w, v[i].y, y[1]) : y[1];
      y[2] = some ? fmaf(w, v[i].z, y[2]) : y[2];
      y[3] = some ? fmaf(w, v[i].w, y[3]) : y[3];
    }
#pragma unroll
  for (int e = 0; e < 4; ++e) y[e] = sum == 0.0f ? 0.0f : y[e] / sum;
  if (mine && col < d) *reinterpret_cast<uint2*>(o + query * d + col) = make_uint2(pack2(y[0], y[1]), pack2(y[2], y[3]));
}

template <int WAVES>
__device__ inline void join_many(const Shares& sh, int64_t query, int d, uint16_t* o) {
  __shared__ float sO[WAVES][256];
  __shared__ float2 sStat[WAVES];
  // a wave's share i is share w + WAVES i of the query's
  const int lane = lane_id(), w = WAVES > 1 ? uniform(threadIdx.x >> 6) : 0, lanes = join_lanes(d), col = 4 * (lane & (lanes - 1));
  const int n = (sh.splits - w + WAVES - 1) / WAVES;
  const float2* stat = sh.stat + query * sh.splits + w;
  const float2 st = lane < n ? stat[WAVES * lane] : make_float2(-INFINITY, 0.0f);
  float top = st.y == 0.0f ? -INFINITY : st.x;
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) top = fmaxf(top, __shfl_xor(top, off, kWave));
  const float weight = st.y == 0.0f ? 0.0f : exp2_fast(st.x - (top == -INFINITY ? 0.0f : top));
  const float sum = wave_sum(weight * st.y);
  const bool mine = col < d;
  const float* part = sh.part + (query * sh.splits + w) * d + (mine ? col : 0);
  float y[4] = {};
  for (int i0 = 0; i0 < n; i0 += 8 * kWave / lanes) {
    float4 v[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int i = i0 + u * (kWave / lanes) + lane / lanes;
      v[u] = *reinterpret_cast<const float4*>(part + static_cast<int64_t>(WAVES * min(i, n - 1)) * d);
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int i = i0 + u * (kWave / lanes) + lane / lanes;
      const float f = __shfl(weight, i & 63, kWave);
      const bool some = __shfl(st.y, i & 63, kWave) != 0.0f && i < n;
      y[0] = some ? fmaf(f, v[u].x, y[0]) : y[0];
      y[1] = some ? fmaf(f, v[u].y, y[1]) : y[1];
      y[2] = some ? fmaf(f, v[u].z, y[2]) : y[2];
      y[3] = some ? fmaf(f, v[u].w, y[3]) : y[3];
    }
  }
  for (int off = lanes; off < kWave; off <<= 1)
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] += __shfl_xor(y[e], off, kWave);
  float l = sum;
  if (WAVES > 1) {
    if (mine && lane < lanes) *reinterpret_cast<float4*>(&sO[w][col]) = make_float4(y[0], y[1], y[2], y[3]);
    if (lane == 0) sStat[w] = make_float2(top, sum);
    __syncthreads();
    if (w > 0) return;
    float all = -INFINITY;
#pragma unroll
    for (int i = 0; i < WAVES; ++i) all = sStat[i].y == 0.0f ? all : fmaxf(all, sStat[i].x);
    l = y[0] = y[1] = y[2] = y[3] = 0.0f;
#pragma unroll
    for (int i = 0; i < WAVES; ++i) {
      if (sStat[i].y == 0.0f || !mine) continue;
      const float f = exp2_fast(sStat[i].x - (all == -INFINITY ? 0.0f : all));
      const float4 v = *reinterpret_cast<const float4*>(&sO[i][col]);
      l = fmaf(f, sStat[i].y, l);
      y[0] = fmaf(f, v.x, y[0]);
      y[1] = fmaf(f, v.y, y[1]);
      y[2] = fmaf(f, v.z, y[2]);
      y[3] = fmaf(f, v.w, y[3]);
    }
  }
  if (!mine || lane >= lanes) return;
#pragma unroll
  for (int e = 0; e < 4; ++e) y[e] = l == 0.0f ? 0.0f : y[e] / l;
  *reinterpret_cast<uint2*>(o + query * d + col) = make_uint2(pack2(y[0], y[1]), pack2(y[2], y[3]));
}

// Threads for each query of a join: join_lanes(d) of them, a wave or a workgroup of 256.
inline int threads_to_join(const Shares& sh, int64_t queries, int d) {
  return sh.splits <= kFewSplits ? join_lanes(d) : sh.splits > kWave || queries <= 2048 ? 256 : kWave;
}
// In a kernel of 256 threads with THREADS of them a query (0: join_lanes(d)): the thread's query, and its join.
template <int THREADS>
__device__ inline int64_t joined_query(int d) {
  return (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) / (THREADS ? THREADS : join_lanes(d));
}
template <int THREADS>
__device__ inline void join(const Shares& sh, int64_t query, bool there, int d, uint16_t* o) {
  if (THREADS == 0)
    join_few(sh, query, there, d, o);
  else if (there)
    join_many<THREADS == 256 ? 4 : 1>(sh, query, d, o);
}

// A launch by its function, without the call configuration of <<<>>>, which costs the host 0.2 of 3.4 us.  Arguments cost
// it too, 0.35 us for 100 bytes, and 256 more of them go along where a kernel asks for gridDim.  False where it failed:
// then the call launches nothing more.
template <typename Args>
inline bool launch_kernel(void (*kernel)(Args), int64_t groups, int64_t rows, int threads, hipStream_t st, Args a) {
  void* args[] = {&a};
  return hipLaunchKernel(reinterpret_cast<const void*>(kernel), dim3(static_cast<unsigned>(groups), static_cast<unsigned>(rows)),
                         dim3(static_cast<unsigned>(threads)), args, 0, st) == hipSuccess;
}
// a call's result; the runtime's error is taken either way
inline int launched(bool all) {
  const int status = launch_status();
  return all ? status : BLLM_E_HIP;
}

inline bool page_shift(int64_t page, int* shift) {
  for (*shift = 4; *shift <= 8; ++*shift)
    if (page == int64_t(1) << *shift) return true;
  return false;
}

// arguments that the calls on pages share
inline int pages_check(const void* k_pages, const void* v_pages, const float* k_scale, const float* v_scale,
                       int pages_dtype, int64_t npages, int64_t page, int64_t hkv, int64_t d, const int32_t* table,
                       int64_t cols, int64_t nseq, Pages* p) {
  const bool q8 = pages_dtype == BLLM_I8;
  if (!k_pages || !v_pages || !table || npages < 1 || page < 1 || hkv < 1 || d < 1 || cols < 1 || nseq < 1 ||
      q8 != (k_scale != nullptr) || q8 != (v_scale != nullptr))
    return BLLM_E_INVAL;
  if ((!q8 && pages_dtype != BLLM_BF16) || !page_shift(page, &p->shift) || d % (q8 ? 16 : 8) != 0 || d > 256 ||
      hkv > kMaxHeads || nseq > kMaxSeqs || npages >= int64_t(1) << 31 || cols > kMaxTokens / page ||
      !aligned16(k_pages) || !aligned16(v_pages) || (reinterpret_cast<uintptr_t>(k_scale) & 3u) ||
      (reinterpret_cast<uintptr_t>(v_scale) & 3u))
    return BLLM_E_NOTSUP;
  p->table = table;
  p->cols = static_cast<int>(cols);
  p->npages = static_cast<int>(npages);
  p->hkv = static_cast<int>(hkv);
  p->d = static_cast<int>(d);
  return BLLM_OK;
}

inline int mask_make(double scale, int causal, int64_t window, double cap, const float* slopes, const int32_t* prefix,
                     Mask* m) {
  if (scale != scale || window < 0 || !(cap >= 0.0 && cap <= 3.0e38)) return BLLM_E_INVAL;
  if (cap != 0.0 && !(cap >= 0.0009765625 && cap <= 1024.0)) return BLLM_E_NOTSUP;  // capped() is off by 2^-22 cap
  // a window past every distance is none
  *m = Mask{static_cast<float>(scale), static_cast<float>(cap), slopes, prefix,
            static_cast<int>(window > kMaxTokens ? 0 : window), causal != 0};
  return BLLM_OK;
}

inline int heads_check(int64_t hq, int64_t hkv, int64_t d) {
  if (hq < 1 || hkv < 1 || d < 1 || hq % hkv != 0) return BLLM_E_INVAL;
  return hq > kMaxHeads || d % 8 != 0 || d > 256 ? BLLM_E_NOTSUP : BLLM_OK;
}

inline bool stride_ok(int64_t stride) { return stride % 8 == 0 && stride < kMaxStride; }

}  // namespace bllm
