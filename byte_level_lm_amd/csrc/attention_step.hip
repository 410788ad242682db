// Attention of one new token of each stream over its pages.
//
//   s_j = scale q.k_j (capped, lowered by distance),  o = sum_j 2^{x_j - m} v_j / sum_j 2^{x_j - m},  x = s log2 e
//
// Bound by the cache's bytes, each read once (kernels' medians in a trace): 8 streams of 65536 positions, 12 heads on 4 of
// 128, bf16: 184 us and 5 for the join, 5.8 TB/s; 256 streams of 256 to 2048 positions in
// 8 bits: 69 us, 4.7 TB/s (codes to bf16 by vector instructions, 35 % of their cycles); one
// stream of 2048: 5.5 us and 4.4.  The keys that a stream sees are
// cut into `splits` equal shares, each a workgroup of up to 16 query heads of one key
// head; its four waves take tiles of 32 keys in turn, straight from memory
// into the matrix instructions' registers, with a running maximum and sum of
// their own.  They are joined through LDS, the shares by a second launch.
//
// Registers (16 x 16 x 32 instructions; lane = 16 g + c): scores come as
// S^T = K Q^T, of which a lane has its query c and keys 4 g + r of each 16.
// That is how the second product O^T = V^T P^T takes its weights, with the
// 32 keys in the order 4 g + r, 16 + 4 g + r, so weights never leave their lane.  V's side then
// is 8 rows of a lane's VP = D / 16 values c VP + n, read as they lie and
// transposed by byte permutes, and a lane's part of O^T is 4 VP values side by side.
#include "attention.h"

namespace bllm {
namespace {

constexpr int kTile = 32;        // keys of a wave's tile
constexpr int kStepWaves = 4;

struct StepArgs {
  const uint16_t* q;
  const void *k_pages, *v_pages;
  const float *k_scale, *v_scale;
  Pages pages;
  const int32_t* lengths;
  uint16_t* o;
  Shares shares;
  int64_t q_stride;
  int hq, group, blocks;  // query heads, those of a key head, blocks of 16 of these
  Mask mask;
};

// scales lie on 4 bytes, no more; the load is as wide all the same
__device__ inline floatx4 four_floats(const float* p) {
  floatx4 v;
  __builtin_memcpy(&v, p, sizeof(v));
  return v;
}

// The tiles that the last query of a stream sees: those of keys [0, front), then from `skip` on those of [lo, n).
struct Seen {
  int n, lo, front, first, skip, tiles;
  __device__ inline Seen(const StepArgs& a, int s) {
    n = min(max(a.lengths[s], 0), a.pages.cols << a.pages.shift);
    lo = a.mask.window ? max(n - a.mask.window, 0) : 0;
    front = a.mask.prefix ? min(max(a.mask.prefix[s], 0), lo) : 0;
    first = (front + kTile - 1) / kTile;
    skip = max(lo / kTile, first) - first;
    tiles = max((n + kTile - 1) / kTile - skip, 0);
  }
  __device__ inline int key(int tile) const { return (tile < first ? tile : tile + skip) * kTile; }
  // without branches: the selects that use it then stay selects
  __device__ inline bool has(int j) const { return (j < front) | ((j >= lo) & (j < n)); }
  __device__ inline bool all(int j) const { return (j + kTile <= front) | ((j >= lo) & (j + kTile <= n)); }
};

// GEN: with a cap or slopes.  The workgroups of a CU that registers are kept for: the most
// that spill nothing in the loop.  bf16: 4 of them spill (8 x 65536 positions 200 us, with 3
// 189), 2 have too few loads on their way (61 streams with a window of 512 21 us, 18); 8 bits: 256 streams
// 69 us with 4, 76 with 3; d > 128 has room for 2 in LDS (8 bits, 8 x 32768: 107 us, 123 with the registers of one).
template <int D, bool Q8, bool GEN>
__global__ __launch_bounds__(64 * kStepWaves, D > 128 ? 2 : Q8 ? 4 : 3) void step_share(StepArgs a) {
  constexpr int VP = D / 16;               // values of a row that a lane has of V
  constexpr int VW = Q8 ? VP / 4 : VP / 2; // their 32-bit words
  constexpr int KP = Q8 ? D / 64 : D / 32; // 16-byte pieces of a row that a lane has of K
  constexpr int kPitch = D + 4;
  __shared__ float sO[kStepWaves][16 * kPitch];
  __shared__ float sM[kStepWaves][16], sL[kStepWaves][16];
  const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int split = blockIdx.x % a.shares.splits, rest = blockIdx.x / a.shares.splits, kh = rest / a.blocks, block = rest % a.blocks;
  const int s = blockIdx.y, d = a.pages.d, h0 = kh * a.group + 16 * block, heads = min(a.group - 16 * block, 16);
  const Seen seen(a, s);
  const int share = (seen.tiles + a.shares.splits - 1) / a.shares.splits, t0 = split * share, t1 = min(t0 + share, seen.tiles);
  const int h = h0 + min(c, heads - 1), t = seen.n - 1;

  // the queries, 8 values of each 32 (in the order of K's pieces)
  uint4 fq[D / 32];
  const uint16_t* q = a.q + static_cast<int64_t>(s) * a.q_stride + static_cast<int64_t>(h) * d;
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    const int at = Q8 ? 16 * (g + 4 * (i / 2)) + 8 * (i % 2) : 8 * (g + 4 * i);
    fq[i] = c < heads && at < d ? *reinterpret_cast<const uint4*>(q + at) : make_uint4(0, 0, 0, 0);
  }
  const float slope = GEN && a.mask.slopes ? a.mask.slopes[h] : 0.0f;
  const float c1 = GEN ? a.mask.scale : a.mask.scale * kLog2e;
  const float c2 = GEN && a.mask.cap > 0.0f ? 2.0f * kLog2e / a.mask.cap : 0.0f;

  float m = -INFINITY, l = 0.0f;
  floatx4 o[VP] = {};
  const int mask = (1 << a.pages.shift) - 1, elem = Q8 ? 1 : 2;
  // the wave's tiles (twice: the weights' first terms so, no second ones)
  const auto pass = [&](bool twice) __attribute__((always_inline)) {
    for (int tile = t0 + w; tile < t1; tile += kStepWaves) {
      const int j0 = seen.key(tile);
      // each half of a tile lies in one page
      bool page[2];
      int64_t row[2];
      const char *kp[2], *vp[2];
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const int j = j0 + 16 * b, col = min(j >> a.pages.shift, a.pages.cols - 1);
        const int id = __builtin_amdgcn_readfirstlane(a.pages.table[static_cast<int64_t>(s) * a.pages.cols + col]);
        page[b] = id >= 0 && id < a.pages.npages;
        row[b] = ((static_cast<int64_t>(page[b] ? id : 0) * a.pages.hkv + kh) << a.pages.shift) + (j & mask);
        kp[b] = static_cast<const char*>(a.k_pages) + row[b] * d * elem;
        vp[b] = static_cast<const char*>(a.v_pages) + row[b] * d * elem;
      }
      uint4 k[2][KP];
      uint32_t v[8][VW];
      floatx4 ks[2], vs[2];
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int i = 0; i < KP; ++i) {
          const int at = 16 * (g + 4 * i);  // bytes
          k[b][i] = at < d * elem ? *reinterpret_cast<const uint4*>(kp[b] + c * d * elem + at) : make_uint4(0, 0, 0, 0);
        }
      if (Q8) {
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          ks[b] = four_floats(a.k_scale + row[b] + 4 * g);
          vs[b] = four_floats(a.v_scale + row[b] + 4 * g);
        }
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const char* from = vp[e / 4] + ((4 * g + e % 4) * d + c * VP) * elem;
#pragma unroll
        for (int i = 0; i < VW; i += 4) {
          constexpr int N = VW < 4 ? VW : 4;
          if (c * VP + i * 4 / elem < d)
            __builtin_memcpy(&v[e][i], __builtin_assume_aligned(from + 4 * i, 4 * N), 4 * N);
          else
            __builtin_memset(&v[e][i], 0, 4 * N);
        }
      }

      floatx4 x[2] = {};
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int i = 0; i < KP; ++i) {
          if (!Q8) {
            x[b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_frag(k[b][i]), as_frag(fq[i]), x[b], 0, 0, 0);
          } else {
            const uint32_t u[4] = {k[b][i].x, k[b][i].y, k[b][i].z, k[b][i].w};
            uint32_t f[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {  // codes are exact in bf16: the upper halves of their floats
              const float lo = static_cast<float>(static_cast<int8_t>(u[j / 2] >> (16 * (j % 2))));
              const float hi = static_cast<float>(static_cast<int8_t>(u[j / 2] >> (16 * (j % 2) + 8)));
              f[j] = __builtin_amdgcn_perm(__float_as_uint(hi), __float_as_uint(lo), 0x07060302);
            }
            x[b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_frag(make_uint4(f[0], f[1], f[2], f[3])), as_frag(fq[2 * i]), x[b], 0, 0, 0);
            x[b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_frag(make_uint4(f[4], f[5], f[6], f[7])), as_frag(fq[2 * i + 1]), x[b], 0, 0, 0);
          }
        }

      const bool whole = seen.all(j0) && page[0] && page[1];
      float p[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int b = e / 4, r = e % 4, j = j0 + 16 * b + 4 * g + r;
        p[e] = x[b][r] * (Q8 ? c1 * ks[b][r] : c1);
        if (GEN) {
          if (c2 != 0.0f) p[e] = capped(p[e], a.mask.cap, c2);
          p[e] = (p[e] - slope * static_cast<float>(abs(t - j))) * kLog2e;
        }
      }
      if (!whole) {
        // keys that the query does not see: no score, and zeros for what their rows hold
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const bool has = page[e / 4] & seen.has(j0 + 16 * (e / 4) + 4 * g + e % 4);
          p[e] = has ? p[e] : -INFINITY;
          if (Q8) vs[e / 4][e % 4] = has ? vs[e / 4][e % 4] : 0.0f;
#pragma unroll
          for (int i = 0; i < VW; ++i) v[e][i] &= has ? ~0u : 0u;
        }
      }
      float top = p[0];
#pragma unroll
      for (int e = 1; e < 8; ++e) top = fmaxf(top, p[e]);
      top = max_xor16(max_xor32(top));
      if (__any(top > m)) {
        const float now = fmaxf(m, top), fall = exp2_fast(m - (now == -INFINITY ? 0.0f : now));
        m = now;
        l *= fall;
#pragma unroll
        for (int n = 0; n < VP; ++n) o[n] *= fall;
      }
      const float base = m == -INFINITY ? 0.0f : m;
      // weights in two bf16 terms, 16 bits: the second costs no time where the bytes bound (256 streams
      // of 8-bit pages 68 us, 67 with one) and 47 us instead of 44 where rows are the shortest (64 streams, d 64, 8 bits)
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        p[e] = exp2_fast(p[e] - base);
        l += p[e];
        if (Q8) p[e] *= vs[e / 4][e % 4];
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        hi[e] = pack2(p[2 * e], p[2 * e + 1]);
        lo[e] = twice ? hi[e] : pack2(p[2 * e] - low_half(hi[e]), p[2 * e + 1] - high_half(hi[e]));
      }
      const bf16x8 ph = as_frag(make_uint4(hi[0], hi[1], hi[2], hi[3])), pl = as_frag(make_uint4(lo[0], lo[1], lo[2], lo[3]));
#pragma unroll
      for (int n = 0; n < VP; ++n) {
        uint32_t f[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (Q8) {
            const float x0 = static_cast<float>(static_cast<int8_t>(v[2 * e][n / 4] >> (8 * (n % 4))));
            const float x1 = static_cast<float>(static_cast<int8_t>(v[2 * e + 1][n / 4] >> (8 * (n % 4))));
            f[e] = __builtin_amdgcn_perm(__float_as_uint(x1), __float_as_uint(x0), 0x07060302);
          } else {
            f[e] = __builtin_amdgcn_perm(v[2 * e + 1][n / 2], v[2 * e][n / 2], n % 2 ? 0x07060302 : 0x05040100);
          }
        }
        const bf16x8 fv = as_frag(make_uint4(f[0], f[1], f[2], f[3]));
        o[n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fv, ph, o[n], 0, 0, 0);
        o[n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fv, pl, o[n], 0, 0, 0);
      }
    }
    l = sum_xor16(sum_xor32(l));
  };
  pass(false);

  // the waves' parts: lane (c, g) has values (4 g + r) VP + n of query c
#pragma unroll
  for (int r = 0; r < 4; ++r)
#pragma unroll
    for (int n = 0; n < VP; n += 4)
      *reinterpret_cast<floatx4*>(&sO[w][c * kPitch + (4 * g + r) * VP + n]) = floatx4{o[n][r], o[n + 1][r], o[n + 2][r], o[n + 3][r]};
  if (g == 0) {
    sM[w][c] = m;
    sL[w][c] = l;
  }
  // An infinity times a weight's second term, which may be zero or negative, undoes what it gave times the first, and an infinite scale has no
  // second term.  Where scores are finite and outputs are not, the wave takes its tiles once more with the first term twice, for
  // these outputs alone (what the look at them costs: 8 bits, d 128, slopes 72.5 us, 71 without; others up to 1 %).
  float odd = 0.0f;
#pragma unroll
  for (int n = 0; n < VP; ++n)
#pragma unroll
    for (int r = 0; r < 4; ++r) odd = fmaf(o[n][r], 0.0f, odd);  // 0 x infinity and 0 x NaN are NaN
  if (__any(odd != 0.0f && fabsf(l) < INFINITY)) {
    m = -INFINITY;
    l = 0.0f;
#pragma unroll
    for (int n = 0; n < VP; ++n) o[n] = floatx4{};
    pass(true);
    float* part = &sO[w][c * kPitch + 4 * g * VP];
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int n = 0; n < VP; ++n)
        if (!(fabsf(part[r * VP + n]) < INFINITY)) part[r * VP + n] = o[n][r];
  }
  __syncthreads();
  const int qi = threadIdx.x / 16, col = threadIdx.x % 16;  // a query's values in pieces of 8
  if (qi >= heads) return;
  float top = sM[0][qi];
#pragma unroll
  for (int i = 1; i < kStepWaves; ++i) top = fmaxf(top, sM[i][qi]);
  float weight[kStepWaves], sum = 0.0f;
#pragma unroll
  for (int i = 0; i < kStepWaves; ++i) {
    weight[i] = sL[i][qi] == 0.0f ? 0.0f : exp2_fast(sM[i][qi] - top);
    sum += weight[i] * sL[i][qi];
  }
  const int64_t head = static_cast<int64_t>(s) * a.hq + h0 + qi;
  if (a.shares.splits > 1 && col == 0) a.shares.stat[head * a.shares.splits + split] = make_float2(top, sum);
#pragma unroll
  for (int i = 0; i < D / 128 + (D < 128); ++i) {
    const int at = 8 * (col + 16 * i);
    if (at >= d) break;
    float y[8] = {};
#pragma unroll
    for (int n = 0; n < kStepWaves; ++n)
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] += weight[n] * sO[n][qi * kPitch + at + e];
    if (a.shares.splits > 1) {
      float4* to = reinterpret_cast<float4*>(a.shares.part + (head * a.shares.splits + split) * d + at);
      to[0] = make_float4(y[0], y[1], y[2], y[3]);
      to[1] = make_float4(y[4], y[5], y[6], y[7]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = sum == 0.0f ? 0.0f : y[e] / sum;
      Vec<BLLM_BF16>::store(a.o, head * d + at, y);
    }
  }
}

struct JoinArgs {
  Shares shares;
  uint16_t* o;
  int heads, d;
};
template <int THREADS>
__global__ __launch_bounds__(256) void step_join(JoinArgs a) {
  const int64_t head = joined_query<THREADS>(a.d);
  join<THREADS>(a.shares, head, head < a.heads, a.d, a.o);
}

// Shares of a stream, each at least a tile a wave: as many as give a workgroup to each
// place for one (LDS has room for 8, 4 or 2 of them a CU).  8 streams of 65536 positions, d 128:
// 970 us whole, 189 in these 32 shares, 188 in 16, 192 in 64.  8 of 32768, d 256, 8 bits: 626 whole,
// 107 in 16, 110 in 32.  64 streams of 4096 to 16384, d 64, 8 bits, 2 heads, whose longest ones
// end last: 196 whole, 47 in 16, 49 in 8.  One stream of 262144, d 128, one key head: 31 in 256, 71 in 64.
int splits_of(int64_t nseq, int64_t heads, int64_t positions, int64_t d) {
  const int64_t places = 256 * (d > 128 ? 2 : d > 64 ? 4 : 8);
  // few tiles a wave take no longer than a second launch (640 positions, 12 heads on 4 of 128: 13.3 us whole, 15.8 in
  // shares; d 256: 20.5 and 16.0)
  if (positions <= (d > 128 ? 2 : 5) * kTile * kStepWaves) return 1;
  const int64_t most = ceil_div(positions, kTile * kStepWaves), want = ceil_div(places, nseq * heads);
  const int64_t n = want < most ? want : most;
  return static_cast<int>(n < 1 ? 1 : n > kMaxSplits ? kMaxSplits : n);
}

template <int D, bool Q8>
bool step_launch(const StepArgs& a, int64_t groups, int64_t nseq, hipStream_t st) {
  return launch_kernel(a.mask.cap > 0.0f || a.mask.slopes ? step_share<D, Q8, true> : step_share<D, Q8, false>, groups, nseq,
                       64 * kStepWaves, st, a);
}

}  // namespace
}  // namespace bllm

using namespace bllm;

extern "C" size_t bllm_attention_step_workspace(int64_t nseq, int64_t hq, int64_t hkv, int64_t d, int64_t positions) {
  if (nseq < 1 || nseq > kMaxSeqs || heads_check(hq, hkv, d) != BLLM_OK || positions < 1) return 0;
  const int64_t splits = splits_of(nseq, hkv * ceil_div(hq / hkv, 16), positions, d);
  return shares_bytes(nseq * hq, splits, d);
}

extern "C" int bllm_attention_step(const void* q, int dtype, int64_t nseq, int64_t hq, int64_t hkv, int64_t d,
                                   int64_t q_stride, const void* k_pages, const void* v_pages, const float* k_scale,
                                   const float* v_scale, int pages_dtype, int64_t npages, int64_t page,
                                   const int32_t* table, int64_t cols, const int32_t* lengths, double scale,
                                   int64_t window, double cap, const float* slopes, const int32_t* prefix, void* o_out,
                                   void* ws, size_t ws_bytes, void* stream) {
  StepArgs a{};
  const int rc = heads_check(hq, hkv, d);
  const int mc = mask_make(scale, 1, window, cap, slopes, prefix, &a.mask);
  if (rc == BLLM_E_INVAL || mc == BLLM_E_INVAL || !q || !lengths || !o_out || q_stride < hq * d) return BLLM_E_INVAL;
  const int pc = pages_check(k_pages, v_pages, k_scale, v_scale, pages_dtype, npages, page, hkv, d, table, cols, nseq,
                             &a.pages);
  if (pc != BLLM_OK) return pc;
  if (rc != BLLM_OK || mc != BLLM_OK || dtype != BLLM_BF16 || !stride_ok(q_stride) || !aligned16(q) || !aligned16(o_out) || !aligned16(ws))
    return BLLM_E_NOTSUP;
  if (!ws || ws_bytes < bllm_attention_step_workspace(nseq, hq, hkv, d, cols * page)) return BLLM_E_WS;
  a.q = static_cast<const uint16_t*>(q);
  a.k_pages = k_pages;
  a.v_pages = v_pages;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.lengths = lengths;
  a.o = static_cast<uint16_t*>(o_out);
  a.q_stride = q_stride;
  a.hq = static_cast<int>(hq);
  a.group = static_cast<int>(hq / hkv);
  a.blocks = (a.group + 15) / 16;
  // The positions that a query sees: a window bounds them but for a prefix, whose length only the device knows.  It is taken to be
  // short where a row of each workgroup makes 48 KB: whole streams then read a long one at the cache's rate too (window of 512, 488
  // key heads of 64 in bf16, prefixes of 32768: 642 us whole, 663 in shares; of 5: 14.8 and 17.4; ragged streams lose,
  // with prefixes of up to 4096 56 and 49, up to 32768 373 and 265).  With fewer bytes they do not: 256 key heads of 64
  // in 8 bits, prefixes of 32768: 392 whole, 210 in shares, ragged 328 and 117; of 5: 9.0 and 14.8.
  int64_t positions = cols * page;
  const int64_t row_bytes = nseq * hkv * a.blocks * d * (pages_dtype == BLLM_I8 ? 1 : 2);
  if (a.mask.window && (!prefix || row_bytes >= 48 << 10) && window + 2 * kTile < positions) positions = window + 2 * kTile;
  const int splits = splits_of(nseq, hkv * a.blocks, positions, d);
  if (ws_bytes < shares_bytes(nseq * hq, splits, d)) return BLLM_E_WS;  // not so: fewer positions take no more shares
  a.shares = shares_at(ws, nseq * hq, splits);
  const int64_t groups = hkv * a.blocks * a.shares.splits;
  hipStream_t st = static_cast<hipStream_t>(stream);
  const bool q8 = pages_dtype == BLLM_I8;
  bool all;
  if (d <= 64)
    all = q8 ? step_launch<64, true>(a, groups, nseq, st) : step_launch<64, false>(a, groups, nseq, st);
  else if (d <= 128)
    all = q8 ? step_launch<128, true>(a, groups, nseq, st) : step_launch<128, false>(a, groups, nseq, st);
  else
    all = q8 ? step_launch<256, true>(a, groups, nseq, st) : step_launch<256, false>(a, groups, nseq, st);
  const int64_t heads = nseq * hq;
  if (all && a.shares.splits > 1) {
    const int threads = threads_to_join(a.shares, heads, a.pages.d);
    all = launch_kernel(a.shares.splits <= kFewSplits ? step_join<0> : threads == kWave ? step_join<kWave> : step_join<256>,
                        ceil_div(heads * threads, 256), 1, 256, st, JoinArgs{a.shares, a.o, static_cast<int>(heads), a.pages.d});
  }
  return launched(all);
}
