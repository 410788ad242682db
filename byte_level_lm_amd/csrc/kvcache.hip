// Rows of keys and values into the pages of a cache and back, as bf16 or as
// 8-bit codes with a scale for each row:
//   a = max |x|,  code = rne(x * (127 * (1 / a))),  scale = a / 127
// (the arithmetic of the rows of norm.hip).
//
// Bound by the bytes: 65536 tokens of 4 heads of 128 in bf16 45 us (6.0 TB/s) written, 44 read; in
// 8 bits written and read back 82 (43 and 39; the vector instructions of the codes take 3/4 of the cycles).  A group of G lanes has a row, one 16-byte piece of bf16
// a lane; a workgroup finds the places of its tokens once, then moves all
// their rows, several loads a lane in flight.
#include "attention.h"

namespace bllm {
namespace {

constexpr float kTiny = 1e-30f;  // a row whose largest value is below this becomes zeros with scale 0
constexpr int kThreads = 256;
constexpr int kFlight = 4;       // rows a lane has in flight (131072 8-bit rows read: 2 take 111 us, 4 94, 8 106)
constexpr int kMaxTile = 64;     // tokens of a workgroup

struct KvArgs {
  Pages pages;
  uint16_t *k, *v;               // packed rows
  int k_stride, v_stride;        // between tokens
  void *k_pages, *v_pages;
  float *k_scale, *v_scale;      // or null
  const int64_t* offsets;        // or null: one row of each stream
  const int32_t* start;          // or null
  int total, nseq;
  int tile, groups;              // tokens of a workgroup, workgroups
};

__device__ inline uint4 codes_to_bf16(uint2 c, float scale) {
  float x[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[i] = static_cast<float>(static_cast<int8_t>(c.x >> (8 * i))) * scale;
    x[4 + i] = static_cast<float>(static_cast<int8_t>(c.y >> (8 * i))) * scale;
  }
  return Vec<BLLM_BF16>::pack(x);
}

// |x| as bits: NaN lies above infinity, which lies above every finite value
template <int G>
__device__ inline uint32_t group_top(uint32_t v) {
#pragma unroll
  for (int off = G / 2; off >= 1; off >>= 1) v = max(v, static_cast<uint32_t>(__shfl_xor(v, off, kWave)));
  return v;
}

template <bool WRITE, bool Q8, int G>
__global__ __launch_bounds__(kThreads) void kv_move(KvArgs a) {
  __shared__ int64_t sRow[kMaxTile];  // the page row of each token (head 0), -1: none, -2: not a sequence's
  const int hkv = a.pages.hkv, rows = 2 * hkv * a.tile, group = threadIdx.x / G, in = threadIdx.x % G;
  const bool mine = in * 8 < a.pages.d;
  const int tiles = (a.total + a.tile - 1) / a.tile;
  for (int tile = blockIdx.x; tile < tiles; tile += a.groups) {
    const int64_t first = static_cast<int64_t>(tile) * a.tile;
    if (threadIdx.x < kWave) {
      const int64_t t = first + threadIdx.x;
      int s = static_cast<int>(t);
      int64_t at = 0, there = -2;
      bool has = threadIdx.x < a.tile && t < a.total;
      if (a.offsets) {
        const auto slot = [&](int i) { return a.offsets[i]; };
        const int64_t last = min(first + a.tile, static_cast<int64_t>(a.total)) - 1;
        const int s0 = wave_find(a.nseq, first, slot), s1 = max(s0, wave_find(a.nseq, last, slot));
        s = s0 + upper_seq(a.offsets + s0, s1 - s0 + 1, t);
        at = t - a.offsets[s];
        has = has && at >= 0 && t < a.offsets[s + 1];
      }
      if (has) {
        there = a.pages.row(s, at + (a.start ? a.start[s] : 0));
      }
      if (threadIdx.x < a.tile) sRow[threadIdx.x] = there;
    }
    __syncthreads();
    for (int r0 = group; r0 < rows; r0 += kFlight * (kThreads / G)) {
      uint4 x[kFlight];
      float scale[kFlight];
      int64_t to[kFlight], packed[kFlight];
      bool val[kFlight];
#pragma unroll
      for (int i = 0; i < kFlight; ++i) {
        const int r = r0 + i * (kThreads / G), t = r / (2 * hkv), h = r - t * 2 * hkv;
        val[i] = h >= hkv;
        const int head = val[i] ? h - hkv : h;
        to[i] = -2;
        x[i] = make_uint4(0, 0, 0, 0);
        scale[i] = 0.0f;
        if (r < rows) {
          to[i] = sRow[t];
          packed[i] = (first + t) * (val[i] ? a.v_stride : a.k_stride) + head * a.pages.d + 8 * in;
          if (to[i] >= 0) to[i] += static_cast<int64_t>(head) << a.pages.shift;
        }
        if (to[i] >= 0 && mine) {
          if (WRITE) {
            x[i] = *reinterpret_cast<const uint4*>((val[i] ? a.v : a.k) + packed[i]);
          } else {
            const int64_t at = to[i] * a.pages.d + 8 * in;
            const void* p = val[i] ? a.v_pages : a.k_pages;
            if (Q8) {
              const uint2 c = *reinterpret_cast<const uint2*>(static_cast<const int8_t*>(p) + at);
              x[i].x = c.x;
              x[i].y = c.y;
              scale[i] = (val[i] ? a.v_scale : a.k_scale)[to[i]];
            } else {
              x[i] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + at);
            }
          }
        }
      }
#pragma unroll
      for (int i = 0; i < kFlight; ++i) {
        if (!WRITE) {
          if (to[i] >= -1 && mine)
            *reinterpret_cast<uint4*>((val[i] ? a.v : a.k) + packed[i]) = Q8 ? codes_to_bf16(make_uint2(x[i].x, x[i].y), scale[i]) : x[i];
          continue;
        }
        const int64_t at = to[i] * a.pages.d + 8 * in;
        void* p = val[i] ? a.v_pages : a.k_pages;
        if (!Q8) {
          if (to[i] >= 0 && mine) *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + at) = x[i];
          continue;
        }
        float f[8];
        const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          f[2 * j] = __uint_as_float(w[j] << 16);
          f[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
          top = max(top, max(w[j] << 16 & 0x7FFFFFFFu, w[j] & 0x7FFF0000u));
        }
        const float m = __uint_as_float(group_top<G>(top));
        const bool some = !(m < kTiny);  // also where m is NaN, which then is the scale
        const float inv = some ? 127.0f * (1.0f / m) : 0.0f;
        uint32_t c[2] = {0, 0};
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int v = static_cast<int>(fminf(fmaxf(rintf(f[j] * inv), -127.0f), 127.0f));
          c[j / 4] |= static_cast<uint32_t>(v & 0xFF) << (8 * (j % 4));
        }
        if (to[i] < 0) continue;
        if (mine) *reinterpret_cast<uint2*>(static_cast<int8_t*>(p) + at) = make_uint2(c[0], c[1]);
        if (in == 0) (val[i] ? a.v_scale : a.k_scale)[to[i]] = some ? m / 127.0f : 0.0f;
      }
    }
    __syncthreads();
  }
}

template <bool WRITE, bool Q8>
bool launch_as(KvArgs a, hipStream_t st) {
  const int pieces = a.pages.d / 8, g = pieces <= 8 ? 8 : pieces <= 16 ? 16 : 32;
  // tokens of a workgroup: two rounds of its loads (131072 tokens of 8-bit rows read: 95 us, one round
  // 96, four 100), less where that leaves CUs idle (32 tokens written: 3.5 us alone, 4.7 without this)
  const int64_t round = kFlight * (kThreads / g);
  int64_t tile = 2 * round / (2 * a.pages.hkv);
  const int64_t spread = a.total / 1024;
  tile = tile > spread ? spread : tile;
  a.tile = static_cast<int>(tile < 1 ? 1 : tile > kMaxTile ? kMaxTile : tile);
  const int64_t tiles = ceil_div(a.total, a.tile);
  a.groups = static_cast<int>(tiles < (1 << 20) ? tiles : 1 << 20);
  return launch_kernel(g == 8 ? kv_move<WRITE, Q8, 8> : g == 16 ? kv_move<WRITE, Q8, 16> : kv_move<WRITE, Q8, 32>, a.groups, 1,
                       kThreads, st, a);
}

template <bool WRITE>
int launch(const KvArgs& a, void* stream) {
  if (a.total == 0) return BLLM_OK;
  hipStream_t st = static_cast<hipStream_t>(stream);
  return launched(a.k_scale ? launch_as<WRITE, true>(a, st) : launch_as<WRITE, false>(a, st));
}

}  // namespace
}  // namespace bllm

using namespace bllm;

extern "C" int bllm_kv_write(const void* k, const void* v, int dtype, const int64_t* offsets, int64_t nseq,
                             int64_t total, int64_t hkv, int64_t d, int64_t k_stride, int64_t v_stride,
                             const int32_t* start, const int32_t* table, int64_t cols, int pages_dtype,
                             int64_t npages, int64_t page, void* k_pages, void* v_pages, float* k_scale,
                             float* v_scale, void* stream) {
  KvArgs a{};
  if (total < 0 || (total > 0 && (!k || !v)) || (!offsets && total != nseq)) return BLLM_E_INVAL;
  const int rc = pages_check(k_pages, v_pages, k_scale, v_scale, pages_dtype, npages, page, hkv, d, table, cols, nseq,
                             &a.pages);
  if (rc == BLLM_E_INVAL || k_stride < hkv * d || v_stride < hkv * d) return BLLM_E_INVAL;
  if (rc != BLLM_OK) return rc;
  if (dtype != BLLM_BF16 || total > kMaxTokens || !stride_ok(k_stride) || !stride_ok(v_stride) || !aligned16(k) ||
      !aligned16(v))
    return BLLM_E_NOTSUP;
  a.k = static_cast<uint16_t*>(const_cast<void*>(k));
  a.v = static_cast<uint16_t*>(const_cast<void*>(v));
  a.k_stride = static_cast<int>(k_stride);
  a.v_stride = static_cast<int>(v_stride);
  a.k_pages = k_pages;
  a.v_pages = v_pages;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.offsets = offsets;
  a.start = start;
  a.total = static_cast<int>(total);
  a.nseq = static_cast<int>(nseq);
  return launch<true>(a, stream);
}

extern "C" int bllm_kv_read(const void* k_pages, const void* v_pages, const float* k_scale, const float* v_scale,
                            int pages_dtype, int64_t npages, int64_t page, int64_t hkv, int64_t d,
                            const int32_t* table, int64_t cols, const int64_t* offsets, int64_t nseq, int64_t total,
                            const int32_t* start, int dtype, void* k_out, void* v_out, void* stream) {
  KvArgs a{};
  if (total < 0 || (total > 0 && (!k_out || !v_out)) || !offsets) return BLLM_E_INVAL;
  const int rc = pages_check(k_pages, v_pages, k_scale, v_scale, pages_dtype, npages, page, hkv, d, table, cols, nseq,
                             &a.pages);
  if (rc != BLLM_OK) return rc;
  if (dtype != BLLM_BF16 || total > kMaxTokens || !aligned16(k_out) || !aligned16(v_out)) return BLLM_E_NOTSUP;
  a.k = static_cast<uint16_t*>(k_out);
  a.v = static_cast<uint16_t*>(v_out);
  a.k_stride = a.v_stride = static_cast<int>(hkv * d);
  a.k_pages = const_cast<void*>(k_pages);
  a.v_pages = const_cast<void*>(v_pages);
  a.k_scale = const_cast<float*>(k_scale);
  a.v_scale = const_cast<float*>(v_scale);
  a.offsets = offsets;
  a.start = start;
  a.total = static_cast<int>(total);
  a.nseq = static_cast<int>(nseq);
  return launch<false>(a, stream);
}
