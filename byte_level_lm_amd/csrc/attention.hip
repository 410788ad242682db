// Softmax attention of packed prompts.
//
//   s_ij = scale q_i.k_j (capped, lowered by distance),  o_i = sum_j 2^{x_ij - m_i} v_j / sum_j 2^{x_ij - m_i},  x = s log2 e
//
// Times are medians of a call among others without a profiler; both sides of a choice were taken in one run on one card.
//
// A workgroup has 128 rows, a wave 32 of them: queries with all heads of a key head (29 us for 64 prompts of 75 to 300, 12
// heads on 4; when workgroups had rows of one head it took a tenth longer, 16 x 2048 with d 256 6 %).  Tiles of 32 keys go
// through LDS, two buffers of them filled without registers, in one pass with
// the running maximum and sum.  With d = 128, 32 keys are 16 matrix instructions of
// 32 x 32 x 16 (512 cycles) and 16 exponentials a lane with what they need (some 480) for a
// wave, which three waves a SIMD run beside each other.  What bounds it then is the card's
// power: 32 sequences of 2048 tokens, 12 heads on 4, causal: 440 us, 940 TFLOP/s, the
// matrix cores busy 48 % of the cycles at 1.65 to 1.85 GHz (the same instructions with less to
// move, without the loads, run at 2.3).  With d = 64 vector instructions take 60 % of the cycles beside 38 % of matrix ones (the
// same sequences 258 us, 800 TFLOP/s); a window of 512 over 16 ragged sequences of up to 8192 bytes, 8 heads, 121 us, 620
// TFLOP/s, 52 % and 28 %, the rest a tile's way through a wave.  With d = 256 registers leave two waves a SIMD, which
// wait for half of their time (16 x 2048, 8 heads on 2, 334 us, 820 TFLOP/s).  With cap and slopes, 8 pieces of 64 to 512 queries behind 4096
// keys 118 us, 510 TFLOP/s: 60 us are vector instructions, and units of uneven length leave 1.7 waves a SIMD in the mean of 3.  Tried and
// no faster, each against its kernel of then (438 to 489 us): 256 rows a workgroup (489), 64 rows (514), 64 a wave (registers of one
// wave a SIMD), tiles of 64 keys, the next tile's first product between this one's exponentials, the sum by
// a matrix instruction (480 us), priorities, loads two tiles ahead in three buffers (461 us; without
// any loads 342, so that what they cost is the way into LDS, not its latency).
//
// Registers: scores come as S^T = K Q^T, of which a lane (half h of the wave)
// has its row lane % 32 and keys 8 (r / 4) + 4 h + r % 4 of each 32.  The second product
// O^T = V^T P^T takes 16 keys in the order 4 h + {0..3}, 8 + 4 h + {0..3}: the
// weights as the lane has them, and V's columns by transposing LDS reads.  So
// weights never leave their lane, and maximum, sum and the factor of O are one number a lane.
#include "attention.h"

namespace bllm {
namespace {

typedef float floatx16 __attribute__((ext_vector_type(16)));
typedef short shortx4 __attribute__((ext_vector_type(4)));
typedef __amdgpu_buffer_rsrc_t Buffer;

constexpr int kWaves = 4, kRows = 32 * kWaves;  // rows of a workgroup
constexpr int BN = 32;           // keys of a tile
constexpr int kXcds = 8;
// Neighbouring workgroups that one XCD takes in a row, so that they share its L2: window of 512 121.5 us
// (in order of the grid 125), 32 x 2048 chunks 440 (449); runs of 256 are no better (121).
constexpr int kRun = 64;
constexpr uint32_t kOutside = 0x7FFFFFF0u;  // an offset past every buffer: reads as zero
// How far (log2) scores may pass the maximum that weights are taken against: weights up to 256
// lose nothing, and O is scaled anew seldom (32 x 2048 chunks 440 us, 492 with 0; window of 512 121 and 132).
constexpr float kSlack = 8.0f;

struct AttArgs {
  const uint16_t *q, *k, *v;
  const int64_t *offsets, *k_offsets;
  uint16_t* o;
  int64_t total, total_k, q_stride, k_stride, v_stride;
  int64_t first;                 // this launch's first slot of a workgroup's rows
  uint32_t slots, units;         // its slots and units of work
  double inv_group;              // 1 / group
  uint32_t small_inv;            // 2^21 / group, rounded up
  int nseq, hq, hkv, group, d;
  int ranked;                    // units of work in the order of their rows' place in a sequence, the last first
  Mask mask;
  Shares shares;
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

// Where a tile's 16-byte pieces lie in LDS, so that the sixteen rows of K's
// reads lie in all the banks, and so do the four rows and pieces of V's
// transposing reads.  A load brings a chunk of 1 KB: with D = 128 piece p of a row r
// is exchanged with p ^ 4 (r % 4) and chunks (of four rows) are a piece
// apart, which leaves few address registers; else with p ^ exchange(r).
template <int D>
constexpr int kChunk = D == 128 ? 520 : 512;  // values from chunk to chunk
template <int D>
__device__ inline int exchange(int r) {
  return D == 64 ? 4 * (r >> 1 & 1) | (r >> 2 & 3) : D == 128 ? 4 * (r & 3) : 4 * (r & 3) | (r >> 2 & 3);
}

// sum plus both values of a pair
__device__ inline float dot2_ones(uint32_t pair, float sum) {
  return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, pair), __builtin_bit_cast(bf16x2, 0x3F803F80u), sum, false);
}

// What one query sees: keys lo .. hi and those below front.
struct Sight {
  int lo, hi, front;
  __device__ inline bool has(int j) const { return ((j >= lo) & (j <= hi)) | (j < front); }
};
__device__ inline Sight sight(const Mask& m, int t, int keys, int front) {
  Sight s;
  s.lo = m.window ? t - m.window + 1 : 0;
  s.hi = min(m.causal ? t : m.window ? t + m.window - 1 : keys - 1, keys - 1);
  s.front = front;
  return s;
}

__device__ inline int64_t lane_value(int64_t v, int lane) {
  const uint32_t lo = __builtin_amdgcn_readlane(static_cast<uint32_t>(v), lane);
  const uint32_t hi = __builtin_amdgcn_readlane(static_cast<uint32_t>(v >> 32), lane);
  return static_cast<int64_t>(static_cast<uint64_t>(hi) << 32 | lo);
}

// The sequence that has the slot, and its rows of queries and keys.  Up to 63
// sequences take one trip to memory: their offsets are in the wave's lanes.
__device__ inline int find_rows(const AttArgs& a, int64_t slot, int64_t* t0, int64_t* t1, int64_t* k0, int64_t* k1) {
  const auto cut = [](int64_t v, int64_t most) { return min(max(v, int64_t(0)), most); };
  if (a.nseq < kWave) {
    const int i = min(lane_id(), a.nseq);
    const int64_t off = cut(a.offsets[i], a.total), k_off = cut(a.k_offsets[i], a.total_k);
    const uint64_t before = __ballot(lane_id() < a.nseq && off * a.group / kRows + i <= slot);
    const int s = max(static_cast<int>(__popcll(before)) - 1, 0);
    *t0 = lane_value(off, s);
    *t1 = max(lane_value(off, s + 1), *t0);
    *k0 = lane_value(k_off, s);
    *k1 = max(lane_value(k_off, s + 1), *k0);
    return s;
  }
  const int s = uniform(wave_find(a.nseq, slot, [&](int i) { return cut(a.offsets[i], a.total) * a.group / kRows + i; }));
  seq_rows(a.offsets, s, a.total, t0, t1);
  seq_rows(a.k_offsets, s, a.total_k, k0, k1);
  return s;
}

// The sequence and the block of rows that come at place `at` where the blocks of up to 63
// sequences are ordered by their index, the highest first (-1: no block).  place_of(b) blocks have an index of b or more.
__device__ inline int find_ranked(const AttArgs& a, int64_t at, int* block, int64_t* t0, int64_t* t1, int64_t* k0, int64_t* k1) {
  const auto cut = [](int64_t v, int64_t most) { return min(max(v, int64_t(0)), most); };
  const int i = min(lane_id(), a.nseq), next = min(lane_id() + 1, a.nseq);
  const int64_t off = cut(a.offsets[i], a.total), end = max(cut(a.offsets[next], a.total), off);
  const int64_t k_off = cut(a.k_offsets[i], a.total_k), k_end = max(cut(a.k_offsets[next], a.total_k), k_off);
  const int blocks = static_cast<int>(((end - off) * a.group + kRows - 1) / kRows);
  const auto place_of = [&](int b) {
    int sum;
    wave_incl_scan(max(blocks - b, 0), sum);
    return sum;
  };
  if (at >= place_of(0)) return -1;
  int lo = 0, hi = static_cast<int>(a.slots);  // place_of(lo) > at >= place_of(hi)
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (place_of(mid) > at) lo = mid; else hi = mid;
  }
  // of the sequences with such a block the one that is the rest's; scans and ballots with every lane
  const int64_t rest = at - place_of(lo + 1);
  const uint64_t with = __ballot(blocks > lo);
  const uint64_t its = __ballot((blocks > lo) & (lanes_below(with) == rest));
  if (its == 0) return -1;
  const int s = static_cast<int>(__builtin_ctzll(its));
  *block = lo;
  *t0 = lane_value(off, s);
  *t1 = lane_value(end, s);
  *k0 = lane_value(k_off, s);
  *k1 = lane_value(k_end, s);
  return s;
}

// an infinity or a NaN, of a bf16 value and in a pair of them
__device__ inline bool not_finite(uint32_t v) { return (v & 0x7F80u) == 0x7F80u; }
__device__ inline bool pair_not_finite(uint32_t v) { return not_finite(v) || not_finite(v >> 16); }

// GEN: with a cap or slopes (their branches alone: 32 x 2048 chunks 473 us, 440 without).  SPLIT: a
// share of the tiles, to be joined.  Three workgroups a CU with d = 128 take 440 us, two 479; a fourth has no registers.
template <int D, bool GEN, bool SPLIT>
__global__ __launch_bounds__(64 * kWaves, D == 256 ? 2 : D == 128 ? 3 : 4) void prompt_tiles(AttArgs a) {
  constexpr int NS = D / 16;               // steps of the first product
  constexpr int NB = D / 32;               // 32-column blocks of the second
  constexpr int RPI = 512 / D;             // rows of a 1 KB load
  constexpr int U = BN / RPI / kWaves;     // loads a wave makes for K, and for V
  // four arrays: a fragment's read then waits for no load that fills another one
  constexpr int kTile = BN / RPI * kChunk<D>;
  __shared__ __align__(16) uint16_t sK0[kTile], sK1[kTile], sV0[kTile], sV1[kTile];
  const int lane = threadIdx.x & 63, qi = lane & 31, half = lane >> 5;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);

  // Unit of work: kRun neighbours go to one XCD.  Units of a key head follow
  // each other, of these a sequence's, the last queries (with the most keys) first.
  uint32_t unit = blockIdx.x;
  {
    const uint32_t full = a.ranked ? 0 : a.units / (kRun * kXcds) * (kRun * kXcds);
    if (unit < full) {
      const uint32_t in = unit % (kRun * kXcds);
      unit += (in % kXcds) * kRun + in / kXcds - in;
    }
  }
  const int split = SPLIT ? static_cast<int>(unit % a.shares.splits) : 0;
  if (SPLIT) unit /= a.shares.splits;
  const uint32_t kh = a.ranked ? unit % a.hkv : unit / a.slots;
  const int64_t slot = a.ranked ? unit / a.hkv : a.first + (unit - kh * a.slots);
  int64_t t0, t1, k0, k1;
  int block = 0;
  const int s = a.ranked ? find_ranked(a, slot, &block, &t0, &t1, &k0, &k1) : find_rows(a, slot, &t0, &t1, &k0, &k1);
  if (s < 0) return;
  const int n = static_cast<int>(t1 - t0), keys = static_cast<int>(k1 - k0);
  // the sequence's rows: a query's heads of this key head, then the next query's
  const int64_t rows = static_cast<int64_t>(n) * a.group;
  const int64_t back = slot - (t0 * a.group / kRows + s), blocks = (rows + kRows - 1) / kRows;
  if (!a.ranked && (back < 0 || back >= blocks)) return;
  const int64_t first = (a.ranked ? block : blocks - 1 - back) * kRows;  // below 2^40: the product below is off by less than half of 1 / group
  const int left = static_cast<int>(min(rows - first, int64_t(kRows)));
  const int query0 = uniform(static_cast<int>((static_cast<double>(first) + 0.5) * a.inv_group));
  const int rest = static_cast<int>(first - static_cast<int64_t>(query0) * a.group);
  // query and head of row r, 0 .. kRows - 1 (rest + r < 2^11, so that the product's error stays below 1 / group)
  const auto query_of = [&](int r) { return query0 + static_cast<int>((static_cast<uint32_t>(rest + r) * a.small_inv) >> 21); };
  const auto head_of = [&](int r, int query) { return static_cast<int>(kh) * a.group + rest + r - (query - query0) * a.group; };
  const int shift = keys - n;                            // position of query 0
  const int front = a.mask.prefix ? uniform(min(max(a.mask.prefix[s], 0), keys)) : 0;

  // the keys that some query of the workgroup sees, in tiles: from 0 to `ahead`, then from `from` to `to`
  const Sight low = sight(a.mask, query0 + shift, keys, front), high = sight(a.mask, query_of(left - 1) + shift, keys, front);
  int from = max(low.lo, 0) / BN * BN, ahead = (front + BN - 1) / BN * BN;
  const int to = max(high.hi + 1, front);
  if (ahead >= from) from = ahead;
  from = uniform(from);
  int tiles = max((ahead + to - from + BN - 1) / BN, ahead / BN), begin = 0;
  if (SPLIT) {
    const int share = (tiles + a.shares.splits - 1) / a.shares.splits;
    begin = split * share;
    tiles = max(min(share, tiles - begin), 0);
  }
  // the wave's own rows, and the lane's
  const int r0 = 32 * w, p0 = query_of(r0) + shift, p1 = query_of(min(r0 + 32, left) - 1) + shift;
  const int query = query_of(r0 + qi), h = head_of(r0 + qi, query);
  const bool some = r0 < left, mine = r0 + qi < left;
  const Sight w0 = sight(a.mask, p0, keys, front), w1 = sight(a.mask, p1, keys, front);
  // tiles that every query of the wave sees whole (at least these), and tiles of which some query sees a key
  const int whole0 = uniform(w1.lo <= front ? 0 : w1.lo), whole1 = uniform(max(w0.hi + 1, w1.lo <= front ? front : 0) - BN);
  const int seen0 = uniform(some ? front : 0), seen1 = uniform(w0.lo - BN + 1), seen2 = uniform(some ? w1.hi : -1);

  bf16x8 fq[NS];                                         // queries: 8 values of each 16
  const int t = query + shift;
  const Sight see = sight(a.mask, t, keys, front);
  // x = c1 times the product; with GEN the product becomes x itself
  const float size = fabsf(a.mask.scale), c1 = GEN ? 1.0f : fmaxf(size * kLog2e, 1e-30f);
  const float cap2 = GEN ? a.mask.cap * kLog2e : 0.0f, to_cap = GEN && cap2 != 0.0f ? 2.0f * kLog2e / a.mask.cap * size : 0.0f;
  const float slope2 = GEN && a.mask.slopes && mine ? a.mask.slopes[h] * kLog2e : 0.0f;

  // loads: where the lane's piece of each 1 KB lies
  uint32_t ko[U], vo[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int r = (u * kWaves + w) * RPI + lane / (D / 8), p = (lane % (D / 8)) ^ exchange<D>(r);
    const bool in = 8 * p < a.d;
    ko[u] = in ? static_cast<uint32_t>(2 * (r * a.k_stride + 8 * p)) : kOutside;
    vo[u] = in ? static_cast<uint32_t>(2 * (r * a.v_stride + 8 * p)) : kOutside;
  }
  const int kbytes = static_cast<int>(2 * a.k_stride), vbytes = static_cast<int>(2 * a.v_stride);
  const char* kb = reinterpret_cast<const char*>(a.k + k0 * a.k_stride + static_cast<int64_t>(kh) * a.d);
  const char* vb = reinterpret_cast<const char*>(a.v + k0 * a.v_stride + static_cast<int64_t>(kh) * a.d);
  // rows past the end read as zero
  const auto load = [&](const char* from, int rows, int bytes, const uint32_t (&at)[U], uint16_t* to) __attribute__((always_inline)) {
    const Buffer b = __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(from), 0, rows * bytes, 0x00027000);
#pragma unroll
    for (int u = 0; u < U; ++u) to_lds(b, at[u], to + (u * kWaves + w) * kChunk<D>);
  };

  // reads: K's row qi, pieces 2 e + half; V's rows 4 half + (lane % 16) / 4 of 8, pieces 4 b + vp
  const int kx = half ^ exchange<D>(qi), kat = qi / RPI * kChunk<D> + qi % RPI * D;
  const auto k_at = [&](int e) {
    return D == 128 ? kat + 8 * half + 32 * (e / 2 ^ (qi & 3)) + 16 * (e % 2) : kat + 8 * (kx ^ 2 * e);
  };
  const int vr = 4 * half + (lane >> 2 & 3), vp = 2 * (lane >> 4 & 1) + (lane >> 1 & 1);
  const int vat = vr / RPI * kChunk<D> + vr % RPI * D + 4 * (lane & 1);
  const auto v_at = [&](int r, int b) {  // rows r on, a multiple of 8
    return r / RPI * kChunk<D> + vat + 8 * ((D == 128 ? vp ^ exchange<D>(vr) : vp ^ exchange<D>(vr + r % 16)) ^ 4 * b);
  };

  float m = -INFINITY, base = 0.0f, l = 0.0f;  // weights are 2^(x - base), base = m once there is one
  floatx16 o[NB] = {};
  const auto products = [&](const uint16_t* K, floatx16& x) __attribute__((always_inline)) {
#pragma unroll
    for (int e = 0; e < NS; ++e)
      x = __builtin_amdgcn_mfma_f32_32x32x16_bf16(*reinterpret_cast<const bf16x8*>(K + k_at(e)), fq[e],
                                                  e ? x : floatx16{}, 0, 0, 0);
  };
  // scores of 32 keys made ready, and the maximum that their weights are taken against
  const auto ready = [&](int j0, floatx16& x, float slack) __attribute__((always_inline)) {
    if (GEN) {  // the product becomes x: capped as in capped(), then lowered by the distance
      if (cap2 != 0.0f) {
#pragma unroll
        for (int r = 0; r < 16; ++r) x[r] = fmaf(-2.0f * cap2, __builtin_amdgcn_rcpf(exp2_fast(x[r] * to_cap) + 1.0f), cap2);
      } else {
#pragma unroll
        for (int r = 0; r < 16; ++r) x[r] *= size * kLog2e;
      }
      if (a.mask.slopes) {
        const float far = static_cast<float>(t - j0 - 4 * half);
#pragma unroll
        for (int r = 0; r < 16; ++r) x[r] = fmaf(-slope2, fabsf(far - static_cast<float>(8 * (r / 4) + r % 4)), x[r]);
      }
    }
    if (!(j0 >= whole0 && j0 <= whole1)) {
      const int lo = see.lo - j0 - 4 * half, hi = see.hi - j0 - 4 * half;  // of the keys 8 (r / 4) + r % 4
      if (j0 < front) {
        const int ahead = front - j0 - 4 * half;
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const int j = 8 * (r / 4) + r % 4;
          x[r] = (((j >= lo) & (j <= hi)) | (j < ahead)) ? x[r] : -INFINITY;
        }
      } else {  // one edge or both
        if (j0 + BN - 1 > w0.hi) {
#pragma unroll
          for (int r = 0; r < 16; ++r) x[r] = 8 * (r / 4) + r % 4 <= hi ? x[r] : -INFINITY;
        }
        if (j0 < w1.lo) {
#pragma unroll
          for (int r = 0; r < 16; ++r) x[r] = 8 * (r / 4) + r % 4 >= lo ? x[r] : -INFINITY;
        }
      }
    }
    float z[5];
#pragma unroll
    for (int r = 0; r < 5; ++r) z[r] = fmaxf(fmaxf(x[3 * r], x[3 * r + 1]), x[3 * r + 2]);
    const float top = fmaxf(fmaxf(fmaxf(z[0], z[1]), z[2]), fmaxf(fmaxf(z[3], z[4]), x[15])) * c1;
    if (__any(top > m + slack)) {
      const float now = fmaxf(m, max_xor32(top));
      base = now == -INFINITY ? 0.0f : now;
      const float fall = exp2_fast(m - base);
      m = now;
      l *= fall;
#pragma unroll
      for (int b = 0; b < NB; ++b) o[b] *= fall;
    }
  };
  // their weights, and the second product.  Weights are rounded to bf16, and their sum is of the rounded ones: outputs of 32 x 2048
  // chunks are off by 0.21 % of their norm, 0.16 % of which is their own rounding.  A second bf16 term of each weight, as the step has
  // it, leaves the 0.16 % and takes another product: 621 us, 440 so (window of 512 156 and 119; d 64 370 and 256)
  const auto weigh = [&](const floatx16& x, uint32_t (&p)[8]) __attribute__((always_inline)) {
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      p[r] = pack2(exp2_fast(fmaf(x[2 * r], c1, -base)), exp2_fast(fmaf(x[2 * r + 1], c1, -base)));
      l = dot2_ones(p[r], l);
    }
  };
  const auto apply = [&](const uint32_t (&p)[8], const uint16_t* V) __attribute__((always_inline)) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {  // 16 keys
      const bf16x8 fp = as_frag(make_uint4(p[4 * e], p[4 * e + 1], p[4 * e + 2], p[4 * e + 3]));
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const uint2 f0 = read_tr(V + v_at(16 * e, b));
        const uint2 f1 = read_tr(V + v_at(16 * e + 8, b));
        o[b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(as_frag(make_uint4(f0.x, f0.y, f1.x, f1.y)), fp, o[b], 0, 0, 0);
      }
    }
  };
  // some query of the wave sees a key of the tile?
  const auto sees = [&](int j0) { return j0 < seen0 || (j0 >= seen1 && j0 <= seen2); };
  // the first key of the i-th tile
  const auto tile_at = [&](int i) {
    const int j = (begin + i) * BN;
    return j < ahead ? j : from + j - ahead;
  };
  // the tile that the loads are at; its first row of k and v
  int j1 = tile_at(0);
  const char *kj = kb + static_cast<int64_t>(j1) * kbytes, *vj = vb + static_cast<int64_t>(j1) * vbytes;
  const auto load_next = [&](uint16_t* K, uint16_t* V) __attribute__((always_inline)) {
    const int rows = min(keys - j1, BN);
    load(kj, rows, kbytes, ko, K);
    load(vj, rows, vbytes, vo, V);
    int by = BN;
    if (j1 + BN == ahead) by = from - j1;
    j1 += by;
    kj += static_cast<int64_t>(by) * kbytes;
    vj += static_cast<int64_t>(by) * vbytes;
  };
  int j2 = j1;  // the tile that the products are at
  // one tile, with the loads of the next, if there is one, on their way
  const auto step = [&](bool more, uint16_t* nK, uint16_t* nV, const uint16_t* cK, const uint16_t* cV) __attribute__((always_inline)) {
    const int j0 = j2;
    j2 = j1;
    landed_barrier();
    if (more) load_next(nK, nV);
    if (sees(j0)) {
      floatx16 x;
      uint32_t p[8];
      products(cK, x);
      ready(j0, x, kSlack);
      weigh(x, p);
      apply(p, cV);
    }
  };
  // the queries, negated for a negative scale, so that the largest product has the largest score
  const auto load_queries = [&](int part, int query, int h) __attribute__((always_inline)) {
    const uint16_t* q = a.q + (t0 + query) * a.q_stride + static_cast<int64_t>(h) * a.d + 8 * part;
    const uint32_t sign = a.mask.scale < 0.0f ? 0x80008000u : 0u;
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      const uint4 z = mine && 16 * i + 8 * part < a.d ? *reinterpret_cast<const uint4*>(q + 16 * i) : make_uint4(0, 0, 0, 0);
      fq[i] = as_frag(make_uint4(z.x ^ sign, z.y ^ sign, z.z ^ sign, z.w ^ sign));
    }
  };
  if (tiles > 0) load_next(sK0, sV0);
  load_queries(half, query, h);  // behind the first keys
  for (int i = 0; i < tiles; i += 2) {
    step(i + 1 < tiles, sK1, sV1, sK0, sV0);
    if (i + 1 < tiles) step(i + 2 < tiles, sK0, sV0, sK1, sV1);
  }
  if (!some) return;

  l = sum_xor32(l);
  // Scores were finite and outputs are not: v has values that are not.  In a tile that every query of the wave sees
  // whole they belong in the outputs; in one with an edge they may have met the weight of zero of a
  // query that does not see their key (0 x infinity is NaN).  Then the wave takes its tiles once more by itself,
  // straight from memory (a call of which every wave does 3 to 11 times as long, one with a NaN in its first rows 1.1 to 1.7
  // times), in the same order and with the same weights: queries which do not see such values have the
  // bits that they have without them.  With no such value sums have passed fp32: once more with weights of 1 at most.
  float odd = 0.0f;
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int r = 0; r < 16; ++r) odd = fmaf(o[b][r], 0.0f, odd);  // 0 x infinity and 0 x NaN are NaN
  odd = sum_xor32(odd);
  if (__any(mine && odd != 0.0f && fabsf(l) < INFINITY)) {
    int me = lane;
    __asm__ volatile("" : "+v"(me));  // the loop above keeps no register for what follows, the queries neither (d 256: 335 us, 387 and 421 else)
    const int row = me & 31, part = me >> 5;
    const uint16_t *kr = a.k + k0 * a.k_stride + static_cast<int64_t>(kh) * a.d, *vr0 = a.v + k0 * a.v_stride + static_cast<int64_t>(kh) * a.d;
    bool belong = false, again = false;
    for (int i = 0; i < tiles && !again; ++i) {
      const int j0 = tile_at(i);
      const bool whole = j0 >= whole0 && j0 <= whole1;
      if (!sees(j0) || (whole && belong)) continue;
      bool bad = false;
      for (int c = me; c < BN * a.d / 8; c += 64) {
        const int r = c / (a.d / 8), col = 8 * (c - r * (a.d / 8));
        if (j0 + r >= keys) break;
        const uint4 z = *reinterpret_cast<const uint4*>(vr0 + static_cast<int64_t>(j0 + r) * a.v_stride + col);
        bad = bad || pair_not_finite(z.x) || pair_not_finite(z.y) || pair_not_finite(z.z) || pair_not_finite(z.w);
      }
      if (__any(bad)) (whole ? belong : again) = true;
    }
    if (again || !belong) {
      const int qu = query_of(r0 + row);
      load_queries(part, qu, head_of(r0 + row, qu));
      m = -INFINITY;
      base = l = 0.0f;
#pragma unroll
      for (int b = 0; b < NB; ++b) o[b] = floatx16{};
      for (int i = 0; i < tiles; ++i) {
        const int j0 = tile_at(i);
        if (!sees(j0)) continue;
        int d = a.d, v_stride = static_cast<int>(a.v_stride);
        __asm__ volatile("" : "+s"(d), "+s"(v_stride));  // or every place of a tile's values would be held across the loop
        floatx16 x;
        uint32_t p[8];
        const uint16_t* kt = kr + static_cast<int64_t>(min(j0 + row, keys - 1)) * a.k_stride + 8 * part;
#pragma unroll
        for (int e = 0; e < NS; ++e) {
          const uint4 z = 16 * e + 8 * part < d ? *reinterpret_cast<const uint4*>(kt + 16 * e) : make_uint4(0, 0, 0, 0);
          x = __builtin_amdgcn_mfma_f32_32x32x16_bf16(as_frag(z), fq[e], e ? x : floatx16{}, 0, 0, 0);
        }
        __builtin_amdgcn_sched_barrier(0);
        ready(j0, x, again ? kSlack : 0.0f);
        weigh(x, p);
#pragma unroll
        for (int e = 0; e < 2; ++e) {  // 16 keys, of which the lane has 4 half + {0 .. 3} and 8 more on
          const int jh = j0 + 16 * e + 4 * part;
          const uint16_t* vt = vr0 + static_cast<int64_t>(min(jh, keys - 1)) * a.v_stride;
          const int last = keys - 1 - jh;  // a tile's last keys may not be there
          uint32_t none[4];  // 1 for keys that the query sees with a weight of zero
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int jr = jh + 8 * (r / 2) + 2 * (r % 2);
            none[r] = ((p[4 * e + r] & 0xFFFFu) == 0 && see.has(jr) ? 0x3F80u : 0u) | (p[4 * e + r] >> 16 == 0 && see.has(jr + 1) ? 0x3F800000u : 0u);
          }
          const bf16x8 fp = as_frag(make_uint4(p[4 * e], p[4 * e + 1], p[4 * e + 2], p[4 * e + 3]));
          const bf16x8 fn = as_frag(make_uint4(none[0], none[1], none[2], none[3]));
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            // a column of v in pairs of keys: its finite values, and 1 for those that are up (infinity, NaN), down (-infinity,
            // NaN) and either.  In whole words and with every load made: with branches the registers spill
            const int c = 32 * b + row;
            uint32_t f[4], up[4], down[4], bad[4];
#pragma unroll
            for (int n = 0; n < 4; ++n) {
              const int j = 8 * (n / 2) + 2 * (n % 2), col = min(c, d - 1);
              const uint32_t lo = vt[max(min(j, last), 0) * v_stride + col], hi = vt[max(min(j + 1, last), 0) * v_stride + col];
              const uint32_t in = c < d ? (j <= last ? 0xFFFFu : 0u) | (j + 1 <= last ? 0xFFFF0000u : 0u) : 0u, v = (lo | hi << 16) & in;
              const uint32_t odd = (((v & 0x7F807F80u) + 0x00800080u) >> 15) & 0x00010001u, sign = v >> 15 & 0x00010001u;
              const uint32_t nan = (((v & 0x007F007Fu) + 0x007F007Fu) >> 7) & 0x00010001u;
              f[n] = v & ~(odd * 0xFFFFu);
              up[n] = (odd & (nan | ~sign)) * 0x3F80u;
              down[n] = (odd & (nan | sign)) * 0x3F80u;
              bad[n] = odd * 0x3F80u;
            }
            const auto frag = [](const uint32_t (&z)[4]) { return as_frag(make_uint4(z[0], z[1], z[2], z[3])); };
            o[b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(frag(f), fp, o[b], 0, 0, 0);
            const auto meet = [&](const uint32_t (&z)[4], bf16x8 w, float value) __attribute__((always_inline)) {
              const floatx16 sum = __builtin_amdgcn_mfma_f32_32x32x16_bf16(frag(z), w, floatx16{}, 0, 0, 0);
#pragma unroll
              for (int r = 0; r < 16; ++r) o[b][r] = sum[r] > 0.0f ? o[b][r] + value : o[b][r];
              __builtin_amdgcn_sched_barrier(0);
            };
            meet(up, fp, INFINITY);
            meet(down, fp, -INFINITY);
            meet(bad, fn, NAN);  // zero times it
          }
        }
      }
      l = sum_xor32(l);
    }
  }
  if (SPLIT) {
    if (mine) {
      const int64_t at = ((t0 + query) * a.hq + h) * a.shares.splits + split;
      if (half == 0) a.shares.stat[at] = make_float2(m, l);
      float* out = a.shares.part + at * a.d + 4 * half;
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (32 * b + 8 * e < a.d && l != 0.0f)
            *reinterpret_cast<float4*>(out + 32 * b + 8 * e) = make_float4(o[b][4 * e], o[b][4 * e + 1], o[b][4 * e + 2], o[b][4 * e + 3]);
    }
    return;
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  // lanes of the lower half take columns 0 .. 7 of each 16, of the upper half 8 .. 15
  uint16_t* out = a.o + ((t0 + query) * a.hq + h) * a.d + 8 * half;
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      uint32_t z[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) z[r] = pack2(o[b][8 * e + 2 * r] * inv, o[b][8 * e + 2 * r + 1] * inv);
      const auto u = __builtin_amdgcn_permlane32_swap(z[0], z[2], false, false);
      const auto v = __builtin_amdgcn_permlane32_swap(z[1], z[3], false, false);
      if (mine && 32 * b + 16 * e + 8 * half < a.d)
        *reinterpret_cast<uint4*>(out + 32 * b + 16 * e) = make_uint4(u[0], v[0], u[1], v[1]);
    }
}

template <int THREADS>
__global__ __launch_bounds__(256) void prompt_join(AttArgs a) {
  const int64_t query = joined_query<THREADS>(a.d), row = query / a.hq;
  const bool mine = row < a.total && row >= a.offsets[0] && row < a.offsets[a.nseq];
  join<THREADS>(a.shares, query, mine, a.d, a.o);
}

// Shares of a query's keys, of 384 or more in the mean: as many as the workgroups of whole queries
// find places for on the card (4, 3 or 2 a CU, by registers), since a few that begin late cost a round.
// One piece of 512 queries of 12 heads on 4 of 128 behind 32768 keys: 121 us in 15 shares, 141 in 23; 8 pieces
// of 64 to 512 behind 4096: 168 whole, 118 in 3, 125 in 4, 126 in 6; 3 x 2048, causal: 56 whole, 76 in 2; 16 queries behind
// 65536: 165 in 8, 34 in 64; 64 behind 8192: 24.4 in 16, 22.7 in 21.  Their parts' way to memory and back makes more of them dear, less
// so where rows are short, whose number is rounded (8192 queries of 8 heads of 64: 128 whole, 99 in 2, 155 in 8). Where few
// rows leave most places empty a long sequence among short ones, which the mean hides, has up to 4 (5 of 531 to 2125, 2 heads of
// 32: 35 us, 19 so).  Lengths are the device's, and means hide them: 2048 queries, causal, go in 2 shares, 41 us, 37 in 3; 8 x 3339, 2
// heads of 256, whole, 175, 162 in 2.
int splits_of(int64_t nseq, int64_t total, int64_t keys, int64_t last, int64_t hq, int64_t hkv, int64_t d) {
  const int64_t places = 256 * (d > 128 ? 2 : d > 64 ? 3 : 4);
  // half a workgroup more a sequence, for its last rows
  const int64_t units = (total * (hq / hkv) / kRows + (nseq + 1) / 2) * hkv, want = (places + (d > 64 ? 0 : units / 2)) / units;
  int64_t most = keys / 384;
  if (4 * units <= places && most < 4) most = last / 192 < 4 ? last / 192 : 4;
  const int64_t n = want < most ? want : most;
  return static_cast<int>(n < 1 ? 1 : n > kMaxSplits ? kMaxSplits : n);
}

template <int D, bool SPLIT>
bool launch_as(const AttArgs& a, hipStream_t st) {
  return launch_kernel(a.mask.cap > 0.0f || a.mask.slopes ? prompt_tiles<D, true, SPLIT> : prompt_tiles<D, false, SPLIT>, a.units, 1,
                       64 * kWaves, st, a);
}

template <int D>
bool launch(AttArgs a, hipStream_t st) {
  constexpr int64_t kMost = (int64_t(1) << 32) / (64 * kWaves) - 1;  // workgroups that one launch has threads for
  const int64_t slots = a.total * a.group / kRows + a.nseq;  // sequence s has slots offsets[s] * group / kRows + s and on
  const int64_t each = static_cast<int64_t>(a.hkv) * a.shares.splits, most = kMost / each;
  for (a.first = 0; a.first < slots; a.first += most) {
    a.slots = static_cast<uint32_t>(slots - a.first < most ? slots - a.first : most);
    a.units = static_cast<uint32_t>(a.slots * each);
    // Causal prompts, whose last queries see the most keys, in the order of these, so that none of them begins
    // late and no CU has several: 4 x 2048, 12 heads on 4 of 128, 73 us in order of the sequences, 63 so; 55 of up to 1320, 3 heads of 64,
    // cap and slopes, 68 and 45; 16 x 2048, d 256, 368 and 334.  With more units neighbours' keys in L2 count for more
    // (48 x 2048 chunks 646, 689 so; 60: 797, 937; 32: 440 both), with fewer than CUs the search (2 x 2260, 2 heads of 64: 20.7, 21.2 so), and
    // behind many keys most last equally long (8 of 200 to 256 behind 4096: 8 heads of 64 39.1, 41.4 so; 12 on 4 of 64 45.9, 47.0; but 12 on
    // 4 of 128 84, 71).
    constexpr uint32_t kPlaces = 256 * (D == 256 ? 2 : D == 128 ? 3 : 4);
    a.ranked = a.mask.causal && !a.mask.window && a.nseq < kWave && slots <= most && a.units <= 4096 && 5 * a.units >= 2 * kPlaces &&
               2 * a.total >= a.total_k;
    if (!(a.shares.splits > 1 ? launch_as<D, true>(a, st) : launch_as<D, false>(a, st))) return false;
  }
  if (a.shares.splits == 1) return true;
  // few queries, by the rule of splits_of
  const int threads = threads_to_join(a.shares, a.total * a.hq, a.d);
  return launch_kernel(a.shares.splits <= kFewSplits ? prompt_join<0> : threads == kWave ? prompt_join<kWave> : prompt_join<256>,
                       ceil_div(a.total * a.hq * threads, 256), 1, 256, st, a);
}

}  // namespace
}  // namespace bllm

using namespace bllm;

extern "C" size_t bllm_attention_workspace(int64_t nseq, int64_t total, int64_t total_k, int64_t hq, int64_t hkv,
                                           int64_t d) {
  if (nseq < 1 || nseq > kMaxSeqs || total < 0 || total > kMaxTokens || total_k < 0 || total_k > kMaxTokens ||
      heads_check(hq, hkv, d) != BLLM_OK)
    return 0;
  return shares_bytes(total * hq, splits_of(nseq, total, total_k / nseq, total_k / nseq, hq, hkv, d), d);
}

extern "C" int bllm_attention(const void* q, const void* k, const void* v, int dtype, const int64_t* offsets,
                              const int64_t* k_offsets, int64_t nseq, int64_t total, int64_t total_k, int64_t hq,
                              int64_t hkv, int64_t d, int64_t q_stride, int64_t k_stride, int64_t v_stride,
                              double scale, int causal, int64_t window, double cap, const float* slopes,
                              const int32_t* prefix, void* o_out, void* ws, size_t ws_bytes, void* stream) {
  AttArgs a{};
  const int rc = heads_check(hq, hkv, d), mc = mask_make(scale, causal, window, cap, slopes, prefix, &a.mask);
  if (rc == BLLM_E_INVAL || mc == BLLM_E_INVAL || nseq < 1 || total < 0 || total_k < 0 || !offsets || (!k_offsets && total != total_k) ||
      (total > 0 && (!q || !o_out)) || (total_k > 0 && (!k || !v)) || q_stride < hq * d || k_stride < hkv * d ||
      v_stride < hkv * d)
    return BLLM_E_INVAL;
  if (rc != BLLM_OK || mc != BLLM_OK || dtype != BLLM_BF16 || nseq > kMaxSeqs || total > kMaxTokens || total_k > kMaxTokens ||
      !stride_ok(q_stride) || !stride_ok(k_stride) || !stride_ok(v_stride) || !aligned16(q) || !aligned16(k) ||
      !aligned16(v) || !aligned16(o_out) || !aligned16(ws))
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
  a.group = static_cast<int>(hq / hkv);
  a.d = static_cast<int>(d);
  a.inv_group = 1.0 / a.group;
  a.small_inv = ((1u << 21) + a.group - 1) / a.group;
  // keys that a sequence's last query sees and its queries in the mean; a window alone bounds them, with the workgroup's others
  int64_t last = total_k / nseq;
  if (a.mask.window && !prefix && a.mask.window + kRows < last) last = a.mask.window + kRows;
  int64_t keys = total_k / nseq - (causal ? total / nseq / 2 : 0);
  if (last < keys) keys = last;
  const int splits = splits_of(nseq, total, keys, last, hq, hkv, d);
  if (ws_bytes < shares_bytes(total * hq, splits, d)) return BLLM_E_WS;  // not so: fewer keys take no more shares
  a.shares = shares_at(ws, total * hq, splits);
  hipStream_t st = static_cast<hipStream_t>(stream);
  return launched(d <= 64 ? launch<64>(a, st) : d <= 128 ? launch<128>(a, st) : launch<256>(a, st));
}
