// Product of 8-bit rows with 8-bit weights, a scale for each token and each
// output channel:
//   y[m, n] = (sum_k xq[m, k] wq[n, k]) * (x_scale[m] * w_scale[n]) + bias[n]
// The sum is exact in 32-bit integers (128^2 K < 2^31 up to kMaxK), so it
// does not depend on its order; the scales and the bias are applied in fp32
// and y is rounded once.
//
// Products run on v_mfma_i32_16x16x64_i8 with the weights as its rows and the
// tokens as its columns: a lane then holds one token's consecutive channels.
// The rows of a pair of weight tiles interleave in fours, which makes those
// eight channels, one 16-byte store in bf16.
#include <algorithm>

#include "common.h"

namespace bllm {
namespace {

typedef int intx4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float floatx8 __attribute__((ext_vector_type(8)));
typedef __amdgpu_buffer_rsrc_t Buffer;

constexpr int64_t kMaxK = (1 << 17) - 16;  // 128 * 128 * kMaxK < 2^31
constexpr int64_t kMaxRows = INT32_MAX - 1024, kMaxOut = int64_t(1) << 44;  // tile and row numbers fit 32 bits
constexpr int kCus = 256, kXcds = 8;
constexpr int kBK = 64;            // bytes of K in a step
constexpr int kOutside = 1 << 30;  // a buffer offset that reads as zero

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

// channel of row r of weight tile j: pairs of tiles interleave in fours
__device__ inline int chan(int j, int r) { return 32 * (j >> 1) + 8 * (r >> 2) + 4 * (j & 1) + (r & 3); }

// scales and biases of N channels from col; past the last channel it is repeated
template <int N>
__device__ inline void channel_scales(const LinArgs& a, int64_t col, float* sw, float* bias) {
#pragma unroll
  for (int i = 0; i < N; ++i) sw[i] = a.sw[min(col + i, a.n - 1)];
#pragma unroll
  for (int i = 0; i < N; ++i) bias[i] = 0.0f;
  if (a.bias) {
#pragma unroll
    for (int i = 0; i < N; ++i) bias[i] = a.bias[min(col + i, a.n - 1)];
  }
}

// Eight channels of one token from a lane's two accumulators: one store of 16
// bytes (two in fp32) at any alignment, rows of y may start anywhere.
template <int DT>
__device__ inline void store_whole(const LinArgs& a, int64_t at, float sx, const float* sw, const float* bias,
                                   const intx4& lo, const intx4& hi) {
  typedef uint32_t loose4 __attribute__((ext_vector_type(4), aligned(2)));
  floatx8 v;
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = static_cast<float>(i < 4 ? lo[i] : hi[i - 4]) * (sx * sw[i]) + bias[i];
  loose4 u[2];
  loose4* to;
  if constexpr (DT == BLLM_F32) {
    __builtin_memcpy(u, &v, 32);
    to = reinterpret_cast<loose4*>(static_cast<float*>(a.y) + at);
  } else {
    const bf16x8 b = __builtin_convertvector(v, bf16x8);
    __builtin_memcpy(u, &b, 16);
    to = reinterpret_cast<loose4*>(static_cast<uint16_t*>(a.y) + at);
  }
#pragma unroll
  for (int i = 0; i < (DT == BLLM_F32 ? 2 : 1); ++i) to[i] = u[i];
}
// the same at the right edge, where only `count` of the channels exist
template <int DT>
__device__ inline void store_some(const LinArgs& a, int64_t at, float sx, const float* sw, const float* bias,
                                  const intx4& lo, const intx4& hi, int count) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float u = static_cast<float>(i < 4 ? lo[i] : hi[i - 4]) * (sx * sw[i]) + bias[i];
    if (i < count) {
      if constexpr (DT == BLLM_F32)
        static_cast<float*>(a.y)[at + i] = u;
      else
        static_cast<uint16_t*>(a.y)[at + i] = f32_to_bf16(u);
    }
  }
}

// four fp32 results, of which `count` exist
__device__ inline void store_four(const LinArgs& a, int64_t at, float sx, const float* sw, const float* bias,
                                  const intx4& x, int count) {
  typedef uint32_t loose4 __attribute__((ext_vector_type(4), aligned(4)));
  float u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) u[i] = static_cast<float>(x[i]) * (sx * sw[i]) + bias[i];
  float* y = static_cast<float*>(a.y) + at;
  if (count >= 4) {
    loose4 v;
    __builtin_memcpy(&v, u, 16);
    *reinterpret_cast<loose4*>(y) = v;
  } else {
#pragma unroll
    for (int i = 0; i < 3; ++i)
      if (i < count) y[i] = u[i];
  }
}

// ---------------------------------------------------------------- few tokens

// A workgroup owns 16 MT tokens and 32 channels; its eight waves take K in
// turns of 64 bytes, straight from memory (weights are read once by the chip,
// tokens come from L2), and add their sums in LDS.  Latency bounds it (32 x 1536,
// K 512: 3.6 us, a launch alone takes as long).
template <int DT, int MT>
__global__ __launch_bounds__(512) void linear_few(LinArgs a) {
  constexpr int NW = 8;
  __shared__ intx4 sAcc[NW / 2][2 * MT][64];
  const int lane = threadIdx.x & 63, n = lane & 15, gq = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t row0 = static_cast<int64_t>(blockIdx.y) * 16 * MT;
  const int64_t col0 = (static_cast<int64_t>(blockIdx.z) * gridDim.x + blockIdx.x) * 32;
  if (col0 >= a.n) return;
  const int8_t *pw[2], *px[MT];
#pragma unroll
  for (int j = 0; j < 2; ++j) pw[j] = a.wq + min(col0 + chan(j, n), a.n - 1) * a.k + 16 * gq;
#pragma unroll
  for (int i = 0; i < MT; ++i) px[i] = a.xq + min(row0 + 16 * i + n, a.m - 1) * a.k + 16 * gq;
  intx4 acc[2][MT] = {};
  const int whole = a.k & ~63;
#pragma unroll 2
  for (int k = 64 * w; k < whole; k += 64 * NW) {
    intx4 fw[2], fx[MT];
#pragma unroll
    for (int j = 0; j < 2; ++j) fw[j] = *reinterpret_cast<const intx4*>(pw[j] + k);
#pragma unroll
    for (int i = 0; i < MT; ++i) fx[i] = *reinterpret_cast<const intx4*>(px[i] + k);
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int i = 0; i < MT; ++i) acc[j][i] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fw[j], fx[i], acc[j][i], 0, 0, 0);
  }
  if (whole < a.k && ((whole >> 6) & (NW - 1)) == w) {  // the last, partial 64 bytes
    const bool in = whole + 16 * gq < a.k;
    intx4 fw[2], fx[MT];
#pragma unroll
    for (int j = 0; j < 2; ++j) fw[j] = in ? *reinterpret_cast<const intx4*>(pw[j] + whole) : intx4{};
#pragma unroll
    for (int i = 0; i < MT; ++i) fx[i] = in ? *reinterpret_cast<const intx4*>(px[i] + whole) : intx4{};
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int i = 0; i < MT; ++i) acc[j][i] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fw[j], fx[i], acc[j][i], 0, 0, 0);
  }
  for (int half = NW / 2; half >= 1; half >>= 1) {
    if (w >= half && w < 2 * half) {
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < MT; ++i) sAcc[w - half][j * MT + i][lane] = acc[j][i];
    }
    __syncthreads();
    if (w < half) {
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < MT; ++i) acc[j][i] += sAcc[w][j * MT + i][lane];
    }
    __syncthreads();
  }
  if (w) return;
  const int64_t col = col0 + 8 * gq;
  const int count = static_cast<int>(min(a.n - col, int64_t(8)));
  if (count < 1) return;
  float sw[8], bias[8];
  channel_scales<8>(a, col, sw, bias);
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int64_t row = row0 + 16 * i + n;
    if (row >= a.m) continue;
    if (count == 8)
      store_whole<DT>(a, row * a.n + col, a.sx[row], sw, bias, acc[0][i], acc[1][i]);
    else
      store_some<DT>(a, row * a.n + col, a.sx[row], sw, bias, acc[0][i], acc[1][i], count);
  }
}

// ---------------------------------------------------------------- tiles

// Channel of row r of weight tile j.  For bf16 two tiles interleave in fours of
// rows, so that a lane's two hold eight consecutive channels: either way a store
// is 16 bytes and four lanes' stores 64 in a row (5003 x 1551, K 768 to fp32:
// 25 us with runs of sixteen channels a lane, 19 so).
template <int DT>
__device__ inline int tile_chan(int j, int r) {
  return DT == BLLM_F32 ? 16 * j + r : 32 * (j >> 1) + 8 * (r >> 2) + 4 * (j & 1) + (r & 3);
}

// 16-byte piece p of row r of a staged tile (rows of kBK bytes) lies at piece
// p ^ (-(r / 4) % 4), where tiles interleave at p ^ (-(r / 8) % 4): the sixteen
// lanes that LDS serves together (four rows of one piece and four of another,
// twice) start in different banks
__device__ inline int swz(int row, int p) { return row * kBK + ((p ^ (-(row >> 2) & 3)) << 4); }
__device__ inline int swz_pairs(int row, int p) { return row * kBK + ((p ^ (-(row >> 3) & 3)) << 4); }

__device__ inline void to_lds(Buffer b, int at, int k, int8_t* lds) {
  typedef __attribute__((address_space(3))) void lds_void;
  __builtin_amdgcn_raw_ptr_buffer_load_lds(b, (lds_void*)lds, 16, at, k, 0, 0);
}

// At most N vector memory operations and no LDS operation of this wave are
// outstanding, then the workgroup's barrier.  (A fence would wait for every
// load into LDS, also those for later steps.)
template <int N>
__device__ inline void wait_and_meet() {
  __asm__ volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((N & 15) | 0x70 | (N >> 4) << 14);
  __builtin_amdgcn_s_barrier();
  __asm__ volatile("" ::: "memory");
}

// Tile t of the product: XCD x has the x-th eighth of them, and its workgroups
// take neighbours at a time, token tiles first in groups of kGroup, so that
// what its L2 holds at one time is a few row blocks of either side.
constexpr int kGroup = 8;
struct Where {
  int row, col;
};
__device__ inline Where tile_at(int t, int mt, int nt, int TM, int TN) {
  const int g = t / (kGroup * nt), first = g * kGroup, gm = min(mt - first, kGroup);
  const int in = t - g * kGroup * nt, j = in / gm;
  return {(first + in - j * gm) * TM, j * TN};
}

// Tiles of TM tokens and TN channels, 2 x WN waves.  K goes by in steps
// of kBK bytes through a ring of R LDS buffers, filled without registers
// R - 1 steps ahead.  In a step a wave multiplies weight tile by weight tile;
// once it has read the step's last fragment it meets the others, refills the
// buffer they have all read and reads the next step's fragments under the
// rest of the products.  The loop runs over all steps of all the workgroup's
// tiles, so the next tile's first steps are on their way while one is written.
// The matrix cores bound it (65536 x 6144, K 1536 to bf16: 0.64 to 0.77 ms with the
// card's clock, 1.6 to 1.9 POP/s; 8192 x 8192, K 8192: 2.4 POP/s).
template <int DT, int TM, int TN, int WN, int R>
__global__ __launch_bounds__(128 * WN, 2) void linear_tiles(LinArgs a, int mt, int nt) {
  constexpr int NW = 2 * WN;                              // waves, as 2 x WN
  constexpr int MT = TM / 32, NT = TN / WN / 16;          // 16 x 16 tiles of a wave
  constexpr int UX = TM * kBK / (1024 * NW), U = UX + TN * kBK / (1024 * NW);  // loads of 1 KB a wave makes for a step
  constexpr bool kPairs = DT == BLLM_BF16;                // weight tiles interleave
  constexpr int JB = NT / 2 - 1;                          // the weight tile before which the waves meet
  struct Stage {
    int8_t X[TM * kBK], W[TN * kBK];
  };
  __shared__ __align__(1024) Stage ring[R];
  __shared__ __align__(16) float sScale[TM + 2 * TN];
  const int tid = threadIdx.x, lane = tid & 63, n = lane & 15, gq = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6), wr = w / WN * (TM / 2), wc = w % WN * (TN / WN);
  const int tiles = mt * nt, per = (tiles + kXcds - 1) / kXcds;
  const int group = gridDim.x / kXcds;     // the grid is a multiple of kXcds
  const int lo = (blockIdx.x % kXcds) * per, hi = min(lo + per, tiles);
  int t = lo + blockIdx.x / kXcds;         // this workgroup's tile
  if (t >= hi) return;
  const int steps = (a.k + kBK - 1) / kBK;
  int left = (hi - t + group - 1) / group * steps;  // steps of all its tiles

  // Loads: where the lane's piece of each 1 KB lies, for the tile the loads are at.
  // Sixteen rows of four pieces are one load; rows past the end repeat the last.
  int lt = t, lk = 0, off[U];
  Buffer bx, bw;
  static_assert(NW % 4 == 0, "row / 16 of a wave's loads is w modulo 4");
  const int prow = lane >> 2, pkx = 16 * ((lane & 3) ^ (-(lane >> 4) & 3)), pkw = kPairs ? 16 * ((lane & 3) ^ (-(2 * w + (lane >> 5)) & 3)) : pkx;
  const auto aim = [&]() __attribute__((always_inline)) {
    const Where at = tile_at(lt, mt, nt, TM, TN);
    const int rx = min(static_cast<int>(a.m) - at.row, TM), rw = min(static_cast<int>(a.n) - at.col, TN);
    bx = __builtin_amdgcn_make_buffer_rsrc(const_cast<int8_t*>(a.xq + static_cast<int64_t>(at.row) * a.k), 0, rx * a.k,
                                           0x00027000);
    bw = __builtin_amdgcn_make_buffer_rsrc(const_cast<int8_t*>(a.wq + static_cast<int64_t>(at.col) * a.k), 0, rw * a.k,
                                           0x00027000);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int row = ((u < UX ? u : u - UX) * NW + w) * 16 + prow;
      off[u] = min(row, (u < UX ? rx : rw) - 1) * a.k + (u < UX ? pkx : pkw);
    }
  };
  const auto load = [&](int u, int8_t* X, int8_t* W) __attribute__((always_inline)) {
    const bool x = u < UX;
    const bool out = lk + (x ? pkx : pkw) >= a.k;  // pieces past the end of K read as zero
    to_lds(x ? bx : bw, out ? kOutside : off[u], lk, (x ? X : W) + ((x ? u : u - UX) * NW + w) * 1024);
  };
  const auto advance = [&]() __attribute__((always_inline)) {
    lk += kBK;
    if (lk >= a.k) {
      lk = 0;
      lt += group;
      if (lt < hi) aim();
    }
  };

  intx4 acc[NT][MT] = {};
  intx4 fx[MT], fw[NT];
  const int rx0 = swz(wr + n, gq);
  const int cn = wc + tile_chan<DT>(0, n), rw0 = kPairs ? swz_pairs(cn, gq) : swz(cn, gq);
  const auto read_x = [&](int i, const int8_t* X) __attribute__((always_inline)) {
    return *reinterpret_cast<const intx4*>(X + rx0 + 16 * i * kBK);  // 16 rows on, the pieces are exchanged alike
  };
  const auto read_w = [&](int j, const int8_t* W) __attribute__((always_inline)) {
    return *reinterpret_cast<const intx4*>(W + rw0 + tile_chan<DT>(j, 0) * kBK);  // and so for these
  };
  // One step, with `more` if there is one to load.  The buffers are restrict
  // arguments: no fragment read has to wait for loads that fill another one.
  const auto step = [&](int left, int8_t* dX, int8_t* dW, const int8_t* __restrict__ cW,
                        const int8_t* __restrict__ nX, const int8_t* __restrict__ nW) __attribute__((always_inline)) {
    intx4 gx[MT];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      if (j < JB) {
#pragma unroll
        for (int q = 2 + (NT - 2) * j / JB; q < 2 + (NT - 2) * (j + 1) / JB; ++q) fw[q] = read_w(q, cW);
      }
      if (j == JB) {
        if (left >= R)
          wait_and_meet<(R - 2) * U>();
        else
          wait_and_meet<0>();
      }
      if (j >= JB) {
        constexpr int M = NT - JB;
        if (left > R) {
#pragma unroll
          for (int u = U * (j - JB) / M; u < U * (j - JB + 1) / M; ++u) load(u, dX, dW);
        }
#pragma unroll
        for (int i = MT * (j - JB) / M; i < MT * (j - JB + 1) / M; ++i) gx[i] = read_x(i, nX);
        if (j == JB + 1) fw[0] = read_w(0, nW);
        if (j == JB + 2) fw[1] = read_w(1, nW);
      }
#pragma unroll
      for (int i = 0; i < MT; ++i) acc[j][i] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fw[j], fx[i], acc[j][i], 0, 0, 0);
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int i = 0; i < MT; ++i) fx[i] = gx[i];
    if (left > R) advance();
  };

  aim();
#pragma unroll 1
  for (int i = 0; i < min(R, left); ++i) {
#pragma unroll
    for (int u = 0; u < U; ++u) load(u, ring[i].X, ring[i].W);
    advance();
  }
  if (left >= R)
    wait_and_meet<(R - 1) * U>();
  else
    wait_and_meet<0>();
#pragma unroll
  for (int i = 0; i < MT; ++i) fx[i] = read_x(i, ring[0].X);
  fw[0] = read_w(0, ring[0].W);
  fw[1] = read_w(1, ring[0].W);
#pragma unroll 1
  for (int i = 0, k = 0; left > 0; --left) {
    Stage& c = ring[i];
    i = i + 1 < R ? i + 1 : 0;
    step(left, c.X, c.W, c.W, ring[i].X, ring[i].W);
    if (++k < steps) continue;
    k = 0;
    const Where at = tile_at(t, mt, nt, TM, TN);
    t += group;
    const int m = static_cast<int>(a.m), row0 = at.row + wr + n;
    const bool whole = at.row + TM <= m && at.col + TN <= static_cast<int>(a.n);
    // the tile's scales, through LDS: 16 + 16 + 8 loads a lane from memory would be one or more trips there
    if (tid < TN) {
      sScale[TM + tid] = a.sw[min(at.col + tid, static_cast<int>(a.n) - 1)];
      sScale[TM + TN + tid] = a.bias ? a.bias[min(at.col + tid, static_cast<int>(a.n) - 1)] : 0.0f;
    } else if (tid < TN + TM) {
      sScale[tid - TN] = a.sx[min(at.row + tid - TN, m - 1)];
    }
    __asm__ volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    __asm__ volatile("" ::: "memory");
    static_assert(NT == 4 && TN + TM <= 128 * WN, "a lane has sixteen channels, a thread one scale");
    const int c0 = wc + tile_chan<DT>(0, 4 * gq), count = static_cast<int>(a.n) - at.col - c0;
    float sw[16], bias[16];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int c = TM + c0 + tile_chan<DT>(j, 0);
      *reinterpret_cast<float4*>(sw + 4 * j) = *reinterpret_cast<const float4*>(sScale + c);
      *reinterpret_cast<float4*>(bias + 4 * j) = *reinterpret_cast<const float4*>(sScale + TN + c);
    }
#pragma unroll
    for (int r = 0; r < MT; ++r) {
      const int row = row0 + 16 * r;
      const int64_t to = static_cast<int64_t>(row) * a.n + at.col + c0;
      const float sx = sScale[wr + 16 * r + n];
#pragma unroll
      for (int j = 0; j < 4; j += kPairs ? 2 : 1) {
        const int c = tile_chan<DT>(j, 0);
        if constexpr (kPairs) {
          if (whole || (row < m && count >= c + 8))
            store_whole<DT>(a, to + c, sx, sw + 4 * j, bias + 4 * j, acc[j][r], acc[j + 1][r]);
          else if (row < m && count > c)
            store_some<DT>(a, to + c, sx, sw + 4 * j, bias + 4 * j, acc[j][r], acc[j + 1][r], count - c);
        } else if (row < m) {
          store_four(a, to + c, sx, sw + 4 * j, bias + 4 * j, acc[j][r], count - c);
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[j][r] = intx4{};
      __builtin_amdgcn_sched_barrier(0);
    }
  }
}

template <int MT>
void few_launch(const LinArgs& a, int dtype, hipStream_t st) {
  // one launch has fewer than 2^32 threads along x: beyond, the channels go on along z
  const int64_t cols = ceil_div(a.n, 32), x = std::min(cols, int64_t(1) << 22);
  const dim3 grid(static_cast<unsigned>(x), static_cast<unsigned>(ceil_div(a.m, 16 * MT)),
                  static_cast<unsigned>(ceil_div(cols, x)));
  if (dtype == BLLM_F32)
    hipLaunchKernelGGL((linear_few<BLLM_F32, MT>), grid, dim3(512), 0, st, a);
  else
    hipLaunchKernelGGL((linear_few<BLLM_BF16, MT>), grid, dim3(512), 0, st, a);
}

template <int TM, int TN, int WN, int R>
void tiles_launch(const LinArgs& a, int dtype, hipStream_t st) {
  const int mt = static_cast<int>(ceil_div(a.m, TM)), nt = static_cast<int>(ceil_div(a.n, TN));
  // as many workgroups as the LDS of all CUs holds at once, each with several tiles
  const int64_t most = kCus * (160 * 1024 / (R * (TM + TN) * kBK + 4 * (TM + 2 * TN)));
  const dim3 grid(static_cast<unsigned>(std::min(ceil_div(int64_t(mt) * nt, kXcds) * kXcds, most)));
  if (dtype == BLLM_F32)
    hipLaunchKernelGGL((linear_tiles<BLLM_F32, TM, TN, WN, R>), grid, dim3(128 * WN), 0, st, a, mt, nt);
  else
    hipLaunchKernelGGL((linear_tiles<BLLM_BF16, TM, TN, WN, R>), grid, dim3(128 * WN), 0, st, a, mt, nt);
}

}  // namespace
}  // namespace bllm

using namespace bllm;

extern "C" int bllm_linear_i8(const int8_t* xq, const float* x_scale, const int8_t* wq, const float* w_scale,
                              const float* bias, int dtype, int64_t m, int64_t n, int64_t k, void* y_out,
                              void* stream) {
  if (m < 0 || n < 1 || k < 1 || !wq || !w_scale || (m > 0 && (!xq || !x_scale || !y_out))) return BLLM_E_INVAL;
  if (!valid_dtype(dtype) || k % 16 != 0 || k > kMaxK || m > kMaxRows || n > kMaxRows || m * n > kMaxOut ||
      !aligned16(xq) || !aligned16(wq) || !aligned16(y_out))
    return BLLM_E_NOTSUP;
  if (m == 0) return BLLM_OK;
  LinArgs a{xq, x_scale, wq, w_scale, bias, y_out, m, n, static_cast<int>(k)};
  hipStream_t st = static_cast<hipStream_t>(stream);
  const int64_t col32 = ceil_div(n, 32);
  // Few tokens: the fewest token tiles a workgroup that do not need more
  // workgroups than CUs, so that K's waves are spread widest (us by 16, 32, 64
  // tokens a workgroup: 100 x 1000, K 1024: 4.5, 5.2, 6.9; 300 x 1024, K 4096:
  // 19.2, 17.6, 14.9).  Up to 64 tokens weights are read once whatever n is.
  // Else the largest tile that three quarters of the CUs (all of them for 128 x
  // 128) get one of.  Two LDS buffers where several workgroups share a CU, four
  // where one has it (64 x 128, 128 x 128 with two and with four, 256 x 256; bf16:
  // 1024 x 2048, K 2048: 13.5, 16.3, 16.7, 27.0; 1000 x 6144, K 1536: 20.9, 18.9,
  // 19.5, 25.6; 5003 x 1551, K 768: 22.1, 19.7, 22.2, 23.4; 8192 x 1536, K 1536:
  // 38.1, 28.5, 30.7, 27.0; 4096 x 4096, K 4096: 115, 91, 89, 63).
  if (ceil_div(m, 16) * col32 <= kCus || m <= 16)
    few_launch<1>(a, dtype, st);
  else if (ceil_div(m, 32) * col32 <= kCus || m <= 32)
    few_launch<2>(a, dtype, st);
  else if (ceil_div(m, 64) * col32 <= kCus || m <= 64)
    few_launch<4>(a, dtype, st);
  else if (ceil_div(m, 256) * ceil_div(n, 256) >= kCus / 4 * 3)
    tiles_launch<256, 256, 4, 4>(a, dtype, st);
  else if (ceil_div(m, 128) * ceil_div(n, 128) >= kCus)
    tiles_launch<128, 128, 2, 2>(a, dtype, st);
  else
    tiles_launch<64, 128, 2, 2>(a, dtype, st);
  return launch_status();
}
