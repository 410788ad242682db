// Gated delta rule: a head's state S [dk x dv] decays, loses what it holds
// under the key and takes the new value there,
//   u_t = beta_t (v_t - a_t S_{t-1}^T k_t),  S_t = a_t S_{t-1} + k_t u_t^T,
//   o_t = scale S_t^T q_t,                   a_t = exp(g_t),
// with q and k scaled to unit length on request (x / sqrt(|x|^2 + 1e-6)).
// States, gates and every sum are fp32.
//
// Blocked form, for prompts.  In a block of C = 64 tokens with b_t = g_1 + .. + g_t,
//   (I + A) U = diag(beta) (V - diag(e^b) K S0),  A_ti = beta_t e^(b_t - b_i) k_t.k_i  (i < t),
//   O = scale (diag(e^b) Q S0 + P U),             P_ti = e^(b_t - b_i) q_t.k_i         (i <= t),
//   S = e^(b_C) S0 + K^T diag(e^(b_C - b)) U,
// so the state is read and rounded once a block.  delta_prep, one workgroup for
// each block and head, forms T = (I + A)^-1 diag(beta), P and the decays, all
// blocks at once; a scan walks the blocks of a sequence with the state in
// registers.  That chain is what bounds it: one wave issues an instruction every
// four or five cycles, so the scans leave to a wave on the way from state to state
// what only it can do and give outputs and loads to others.  delta_scan, for many
// heads, has 16 columns and every row on a wave; delta_scan_quarters, for few, a
// quarter of the rows, and takes long sequences in segments at once.  What one product makes the next takes as it lies: a
// 16 x 16 accumulator has a lane's four rows where the next product wants its
// inner index, once the tiles' rows are numbered 8 (r / 4) + r % 4 (+ 4 for the
// second tile of a pair), which costs nothing.
// Matrix products run on bf16 MFMA.  q and k are bf16 as they come (their unit
// lengths are factors of rows); fp32 operands are cut into three bf16 terms
// that hold all 24 bits (S, T, U where they lead to the state), or two (16
// bits) where the result is rounded to bf16 (S, P and U for o).
// A value that is not finite must not reach tokens before its own through a
// zero of T or P: such entries are cut out of the products, and what depends
// on them (its column's later rows and state) is set to NaN afterwards.
//
// Recurrent form, for steps and prompts of a few tokens.  A wave owns 32 columns
// of one head's state: lane (i, c), i = lane / 8, c = lane % 8, holds rows R i .. R i + R - 1 of columns
// 4 c .. 4 c + 3 in registers.  Both sums over dk that a token needs are taken
// from the state before it,
//   S_t^T q = a_t S_{t-1}^T q + (k.q) u_t,
// so a token costs one reduction over the eight lane groups.
#include <algorithm>
#include <cmath>

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

// R bf16 of a lane's rows as pairs; `left` rows exist (8 of 16 at least)
template <int R>
__device__ inline void row_words(const uint16_t* p, int left, uint32_t* w) {
  if constexpr (R >= 8) {
#pragma unroll
    for (int i = 0; i < R; i += 8) {
      if (i && left < 16) break;
      const uint4 v = *reinterpret_cast<const uint4*>(p + i);
      w[i / 2] = v.x; w[i / 2 + 1] = v.y; w[i / 2 + 2] = v.z; w[i / 2 + 3] = v.w;
    }
  } else if constexpr (R == 4) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x; w[1] = v.y;
  } else {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  }
}

// R = ceil(dk / 8) rounded up to 2, 4, 8 or 16 rows for each lane.  Many steps
// are bound by the states' way in and out (8000 of 128 x 128: 1.05 GB in 187 us,
// 5.6 TB/s, more than a copy), one by latency (4 of them: 6.8 us).
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
  // the next token's inputs are on their way while this one's are used
  const int64_t hd = static_cast<int64_t>(kh) * a.dk + r0;
  const bool rows = r0 < a.dk;  // dk is a multiple of 8: R rows of 8 or 16 are whole or end at 8
  uint32_t nq[R / 2] = {}, nk[R / 2] = {};
  uint2 nv = make_uint2(0, 0);
  float ng = 0.0f, nb = 0.0f;
  const auto load = [&](int64_t t) __attribute__((always_inline)) {
    if (rows) {
      row_words<R>(a.q + t * a.qs + hd, a.dk - r0, nq);
      row_words<R>(a.k + t * a.ks + hd, a.dk - r0, nk);
    }
    if (in) nv = *reinterpret_cast<const uint2*>(a.v + t * a.vs + static_cast<int64_t>(h) * a.dv + col);
    ng = a.g[t * a.hv + h];
    nb = a.beta[t * a.hv + h];
  };
  if (t0 < t1) load(t0);
  for (int64_t t = t0; t < t1; ++t) {
    float q[R], k[R];
    const uint2 p = nv;
    const float al = expf(ng), be = nb;
#pragma unroll
    for (int i = 0; i < R; i += 2) {
      q[i] = __uint_as_float(nq[i / 2] << 16);
      q[i + 1] = __uint_as_float(nq[i / 2] & 0xFFFF0000u);
      k[i] = __uint_as_float(nk[i / 2] << 16);
      k[i + 1] = __uint_as_float(nk[i / 2] & 0xFFFF0000u);
    }
    if (t + 1 < t1) load(t + 1);
    float kk = 0.0f, qq = 0.0f, kq = 0.0f;
    float4 xk = make_float4(0, 0, 0, 0), xq = make_float4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < R; ++i) {
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
    const float vv[4] = {__uint_as_float(p.x << 16), __uint_as_float(p.x & 0xFFFF0000u), __uint_as_float(p.y << 16),
                         __uint_as_float(p.y & 0xFFFF0000u)};
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
      uint2 y;
      y.x = f32_to_bf16(c * (al * xq.x + d * u[0])) |
            static_cast<uint32_t>(f32_to_bf16(c * (al * xq.y + d * u[1]))) << 16;
      y.y = f32_to_bf16(c * (al * xq.z + d * u[2])) |
            static_cast<uint32_t>(f32_to_bf16(c * (al * xq.w + d * u[3]))) << 16;
      *reinterpret_cast<uint2*>(a.o + (t * a.hv + h) * a.dv + col) = y;
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

// ---------------------------------------------------------------- blocked form

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short shortx4 __attribute__((ext_vector_type(4)));
typedef float floatx4 __attribute__((ext_vector_type(4)));
typedef float floatx2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

constexpr int kC = 64;            // tokens of a block
// One block and head in the workspace, in 4-byte words: T - I and P, each 6 fragments of 64 lanes x 8
// (16 x 32 entries on or below the diagonal) in three and two bf16 terms, then beta and the decays of the tokens
constexpr int kFragsT = 6 * 768, kFragsP = 6 * 512, kFrags = kFragsT + kFragsP;
constexpr int kRec = kFrags + 256 + 64;
constexpr int kLd = 68;           // pitch of a 64 x 64 fp32 tile in LDS
constexpr float kForget = -1e4f;  // smaller gates decay by e^-10000 = 0 as well, and their sums stay finite

// fragment f of T and P: row tile frag_row(f), inner tokens 32 frag_k(f) .. + 31
__device__ constexpr int frag_row(int f) { return f < 2 ? f : 2 + (f & 1); }
__device__ constexpr int frag_k(int f) { return f < 4 ? 0 : 1; }
// token (or row of the state) of row r of tile i: pairs of tiles interleave in fours
__device__ inline int tile_row(int i, int r) { return 32 * (i >> 1) + 8 * (r >> 2) + 4 * (i & 1) + (r & 3); }

__device__ inline bf16x8 as_frag(const uint32_t* w) {
  bf16x8 v;
  __builtin_memcpy(&v, w, 16);
  return v;
}
__device__ inline bf16x8 as_frag(const uint4& w) {
  bf16x8 v;
  __builtin_memcpy(&v, &w, 16);
  return v;
}
__device__ inline floatx4 mfma_bf(const bf16x8& a, const bf16x8& b, const floatx4& c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ inline uint32_t high_halves(float a, float b) {
  return __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302u);
}
__device__ inline float below_high(float a) { return a - __uint_as_float(__float_as_uint(a) & 0xFFFF0000u); }
// a and b cut into terms of 8 bits each; w[0] + w[1] (+ w[2]) is the value
template <int N>
__device__ inline void cut(float a, float b, uint32_t* w, int stride) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    w[i * stride] = high_halves(a, b);
    if (i + 1 < N) {
      a = below_high(a);
      b = below_high(b);
    }
  }
}
// B operand of 32 inner entries from a pair of accumulators, cut into N terms
template <int N>
__device__ inline void cut_pair(const floatx4& a, const floatx4& b, bf16x8* f) {
  uint32_t w[N * 4];
  cut<N>(a[0], a[1], w + 0, 4);
  cut<N>(a[2], a[3], w + 1, 4);
  cut<N>(b[0], b[1], w + 2, 4);
  cut<N>(b[2], b[3], w + 3, 4);
#pragma unroll
  for (int i = 0; i < N; ++i) f[i] = as_frag(w + 4 * i);
}

// Barrier for what the waves exchange through LDS: waits for the wave's own LDS
// operations, not for loads and stores of memory.
__device__ inline void exchange_barrier() {
  __asm__ volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
  __builtin_amdgcn_s_barrier();
  __asm__ volatile("" ::: "memory");
}

struct Block {
  int64_t first, left;  // its first token; tokens from there to the sequence's end
};

// the same value in every lane, told to the compiler
__device__ inline int64_t uniform(int64_t v) {
  const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<int>(v));
  const int hi = __builtin_amdgcn_readfirstlane(static_cast<int>(v >> 32));
  return static_cast<int64_t>(hi) << 32 | lo;
}

// sequence s of the batch, cut at its rows
__device__ inline void seq_span(const DeltaArgs& a, int s, int64_t* t0, int64_t* t1) {
  *t0 = uniform(min(max(a.offsets[s], int64_t(0)), a.total));
  *t1 = uniform(min(max(a.offsets[s + 1], *t0), a.total));
}

// Block j of the workspace: sequence s has blocks offsets[s] / 64 + s and on,
// which leaves room for every sequence's last, partial block.
__device__ inline bool find_block(const DeltaArgs& a, int64_t j, Block* b) {
  int lo = 0, hi = a.nseq;  // the sequence is in [lo, hi); every lane asks about one of 64 places at once
  for (;;) {
    const int step = (hi - lo + kWave - 1) / kWave, at = min(lo + lane_id() * step, a.nseq);
    const int64_t off = min(max(a.offsets[at], int64_t(0)), a.total);
    const bool before = lo + lane_id() * step < hi && off / kC + at <= j;
    const int k = max(__popcll(__ballot(before)) - 1, 0);
    if (step == 1) {
      const int s = __builtin_amdgcn_readfirstlane(lo + k);
      const int64_t t0 = __shfl(off, k, kWave);
      // the next offset is the next lane's, if there is one
      int64_t t1 = k + 1 < kWave ? __shfl(off, k + 1, kWave) : min(a.offsets[s + 1], a.total);
      t1 = max(t1, t0);
      b->first = uniform(t0 + (j - (t0 / kC + s)) * kC);
      b->left = uniform(t1) - b->first;
      return b->first >= uniform(t0) && b->left > 0;
    }
    lo += k * step;
    hi = min(hi, lo + step);
  }
}

// A block's rows of one head as a buffer: pieces past the last row, and pieces
// whose offset is kOutside, read as zero and are not stored, without a branch.
// Strides below kMaxStride keep every offset of a block under kOutside.
typedef __amdgpu_buffer_rsrc_t Rows;
typedef uint32_t uintx4 __attribute__((ext_vector_type(4)));
constexpr int kOutside = 1 << 30;
constexpr int64_t kMaxStride = 1 << 22;

__device__ inline Rows rows_at(const uint16_t* base, int64_t stride, int left, int width) {
  const int n = min(left, kC);
  const int bytes = __builtin_amdgcn_readfirstlane(n > 0 ? 2 * ((n - 1) * static_cast<int>(stride) + width) : 0);
  const int64_t at = uniform(reinterpret_cast<int64_t>(base));
  return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<uint16_t*>(at), 0, bytes, 0x00027000);
}
__device__ inline Rows rows_of(const uint16_t* base, int64_t stride, const Block& b, int width) {
  return rows_at(base + b.first * stride, stride, static_cast<int>(min(b.left, int64_t(kC))), width);
}
__device__ inline int piece_at(int row, int64_t stride, int col, int width) {
  return col < width ? 2 * (row * static_cast<int>(stride) + col) : kOutside;
}
__device__ inline uint4 piece(Rows r, int at) {
  const uintx4 v = __builtin_amdgcn_raw_buffer_load_b128(r, at, 0, 0);
  return make_uint4(v.x, v.y, v.z, v.w);
}

// 64 lanes' 16-byte pieces straight into 1 KB of LDS, no register in between
__device__ inline void to_lds(Rows r, int at, void* lds) {
  typedef __attribute__((address_space(3))) void lds_void;
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)lds, 16, at, 0, 0, 0);
}

// LDS image of a block's keys or queries: rows of DKP values in 16-byte pieces,
// the pieces of a row exchanged so that neither the sixteen lanes of a fragment
// read that LDS serves together (eight rows at one piece, eight at the next) nor
// the 4 x 4 pieces of a transposing read meet in a bank
template <int DKP>
__device__ inline int swz(int row, int pc) {
  if (DKP == 128) return row * 128 + ((pc ^ ((row & 3) << 2 | (-(row >> 3) & 3))) << 3);
  return row * 64 + ((pc ^ ((row & 2) << 1 | (-(row >> 3) & 3))) << 3);
}

// inclusive sum over the lanes of a wave, in fp64, by row shifts and readlanes
template <int N>
__device__ inline double row_shr(double v) {
  const int64_t u = __double_as_longlong(v);
  const int lo = __builtin_amdgcn_update_dpp(0, static_cast<int>(u), 0x110 + N, 0xF, 0xF, true);
  const int hi = __builtin_amdgcn_update_dpp(0, static_cast<int>(u >> 32), 0x110 + N, 0xF, 0xF, true);
  return __longlong_as_double(static_cast<int64_t>(hi) << 32 | static_cast<uint32_t>(lo));
}
__device__ inline double lane_value(double v, int lane) {
  const int64_t u = __double_as_longlong(v);
  const int lo = __builtin_amdgcn_readlane(static_cast<int>(u), lane);
  const int hi = __builtin_amdgcn_readlane(static_cast<int>(u >> 32), lane);
  return __longlong_as_double(static_cast<int64_t>(hi) << 32 | static_cast<uint32_t>(lo));
}
__device__ inline double wave_sums(double v) {
  v += row_shr<1>(v);
  v += row_shr<2>(v);
  v += row_shr<4>(v);
  v += row_shr<8>(v);
  const double t0 = lane_value(v, 15), t1 = lane_value(v, 31) + t0, t2 = lane_value(v, 47) + t1;
  const int r = lane_id() >> 4;
  return r == 0 ? v : v + (r == 1 ? t0 : r == 2 ? t1 : t2);
}

// products of 16 x 16 fp32 blocks on MFMA: inner index 4 (lane / 16) + r at step r,
// which is how an accumulator already holds it
__device__ inline floatx4 mfma_f32(const float* a, const floatx4& b, floatx4 c) {
  const float4 v = *reinterpret_cast<const float4*>(a);
  c = __builtin_amdgcn_mfma_f32_16x16x4f32(v.x, b[0], c, 0, 0, 0);
  c = __builtin_amdgcn_mfma_f32_16x16x4f32(v.y, b[1], c, 0, 0, 0);
  c = __builtin_amdgcn_mfma_f32_16x16x4f32(v.z, b[2], c, 0, 0, 0);
  return __builtin_amdgcn_mfma_f32_16x16x4f32(v.w, b[3], c, 0, 0, 0);
}
__device__ inline floatx4 column4(const float* t) {  // entries r kLd of a column
  return floatx4{t[0], t[kLd], t[2 * kLd], t[3 * kLd]};
}

// T - I, P and the decays of one block and head, T = (I + A)^-1.
// Waves 0 and 1 form K K^T and from it A in LDS, waves 2 and 3 K Q^T, which
// gives P in the order of its fragments (a lane a row, its accumulator four
// consecutive columns).  The inverse: 8 x 8 blocks on the diagonal by
// substitution, a lane a column, then three doublings [T1 0; -T2 A21 T1 T2] on
// fp32 MFMA, whose accumulators feed the second product as they are.  Gates
// are summed in fp64, in units of ln 2, so that a difference of two sums is as
// good as an fp32 gate however far the block has decayed.  Many blocks run at
// the rate of a copy (128 heads of 128, 8192 tokens: 1.05 GB in 206 us), few are
// bound by the chain of these steps (4 such heads: 512 blocks in 12.4 us).
//
// A decay e^(b_t - b_u) is a quotient that must not be formed from its terms
// (both can underflow).  Between two tiles it is the product of three factors
// below 1, row to tile start, tile to tile and tile end to column, so that only
// the tiles on the diagonal take an exponential an entry.
template <int DKP>
__global__ __launch_bounds__(256, 4) void delta_prep(DeltaArgs a, float* ws) {
  constexpr int NS = DKP / 32;
  constexpr int PR = DKP / 8;          // pieces of a staged row
  constexpr int NK = kC * PR / 256;    // pieces of K (and of Q) a thread loads
  __shared__ __align__(1024) float sA[2 * kC * kLd];  // A and T; before them K and Q
  __shared__ __align__(16) double sB[kC];
  // by token: beta, the factors of its decays, the inverse lengths of k and q
  __shared__ __align__(16) float sBeta[kC], sRow[kC], sCol[kC], sMid[kC], sRk[kC], sRq[kC];
  __shared__ int sBad;
  static_assert(2 * kC * DKP * 2 <= 2 * kC * kLd * 4, "K and Q must fit in the place of A and T");
  float* const sT = sA + kC * kLd;
  uint16_t* const sK = reinterpret_cast<uint16_t*>(sA);
  uint16_t* const sQ = sK + kC * DKP;
  Block blk;
  if (!find_block(a, blockIdx.x, &blk)) return;
  const int tid = threadIdx.x, lane = tid & 63, n = lane & 15, gq = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int h = blockIdx.y, kh = h / (a.hv / a.hk);
  const Rows K = rows_of(a.k + static_cast<int64_t>(kh) * a.dk, a.ks, blk, a.dk);
  const Rows Q = rows_of(a.q + static_cast<int64_t>(kh) * a.dk, a.qs, blk, a.dk);
#pragma unroll
  for (int i = 0; i < NK; ++i) {
    const int row = (i * 256 + tid) / PR, p = (swz<DKP>(row, tid % PR) >> 3) % PR;
    to_lds(K, piece_at(row, a.ks, 8 * p, a.dk), sK + (i * 4 + w) * 512);
    to_lds(Q, piece_at(row, a.qs, 8 * p, a.dk), sQ + (i * 4 + w) * 512);
  }
  if (w == 0) {
    const int64_t mine = (blk.first + min(static_cast<int64_t>(lane), blk.left - 1)) * a.hv + h;
    const float g = a.g[mine], be = lane < blk.left ? a.beta[mine] : 0.0f;
    // a NaN stays
    const double b = wave_sums(lane < blk.left ? (g < kForget ? kForget : g) * 1.4426950408889634 : 0.0);
    const double b15 = lane_value(b, 15), b31 = lane_value(b, 31), b47 = lane_value(b, 47), b63 = lane_value(b, 63);
    const double start = gq == 0 ? 0.0 : gq == 1 ? b15 : gq == 2 ? b31 : b47;
    const double end = gq == 0 ? b15 : gq == 1 ? b31 : gq == 2 ? b47 : b63;
    sB[lane] = b;
    sBeta[lane] = be;
    sRow[lane] = __builtin_amdgcn_exp2f(static_cast<float>(b - start));
    sCol[lane] = __builtin_amdgcn_exp2f(static_cast<float>(end - b));
    sMid[lane] = __builtin_amdgcn_exp2f(static_cast<float>(lane < 32 ? b31 - b : b - b31));
    if (lane == 0) sBad = kC;
  }
  __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0): K and Q have landed
  __syncthreads();
  float* rec = ws + (static_cast<int64_t>(blockIdx.x) * a.hv + h) * kRec;
  // 1 / |x| of the rows of a tile from the diagonal of its square, on the lanes that hold it
  const auto inverse_length = [&](const floatx4& d) {
    const float v = n & 2 ? (n & 1 ? d[3] : d[2]) : (n & 1 ? d[1] : d[0]);
    return a.unit ? 1.0f / sqrtf(v + kL2Eps) : 1.0f;
  };
  const bool diagonal = gq == n >> 2;
  if (w < 2) {
    // rows 16 i of K K^T: wave 0 has i = 3 and 0, wave 1 has i = 2 and 1
    const int i0 = 3 - w, i1 = w;
    floatx4 G0[4] = {}, G1[2] = {};
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      bf16x8 f[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) f[c] = as_frag(*reinterpret_cast<const uint4*>(sK + swz<DKP>(16 * c + n, 4 * s + gq)));
      const bf16x8 f0 = w ? f[2] : f[3], f1 = w ? f[1] : f[0];
#pragma unroll
      for (int c = 0; c < 4; ++c) G0[c] = mfma_bf(f0, f[c], G0[c]);
#pragma unroll
      for (int c = 0; c < 2; ++c) G1[c] = mfma_bf(f1, f[c], G1[c]);
    }
    if (diagonal) {
      sRk[16 * i0 + n] = inverse_length(w ? G0[2] : G0[3]);
      sRk[16 * i1 + n] = inverse_length(w ? G1[1] : G1[0]);
    }
    exchange_barrier();  // K and Q have been read
    float z = 0.0f;
#pragma unroll
    for (int part = 0; part < 2; ++part) {
      const int i = part ? i1 : i0, t = 16 * i + 4 * gq;
      const float4 be = *reinterpret_cast<const float4*>(sBeta + t), rk = *reinterpret_cast<const float4*>(sRk + t);
      const float4 rw = *reinterpret_cast<const float4*>(sRow + t);
      const float row[4] = {be.x * rk.x, be.y * rk.y, be.z * rk.z, be.w * rk.w};
      const float far[4] = {row[0] * rw.x, row[1] * rw.y, row[2] * rw.z, row[3] * rw.w};
#pragma unroll
      for (int c = 0; c < (part ? 2 : 4); ++c) {
        if (c > i) continue;
        const int u = 16 * c + n;
        floatx4& G = part ? G1[c & 1] : G0[c];
        if (c < i) {
          const float f = sCol[u] * sRk[u] *
                          (c + 1 < i ? __builtin_amdgcn_exp2f(static_cast<float>(sB[16 * i - 1] - sB[16 * c + 15])) : 1.0f);
#pragma unroll
          for (int r = 0; r < 4; ++r) G[r] *= far[r] * f;
        } else {
          const double bu = sB[u];
          const float ru = sRk[u];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const float f = __builtin_amdgcn_exp2f(static_cast<float>(sB[t + r] - bu)) * ru;
            G[r] = n < 4 * gq + r ? row[r] * f * G[r] : 0.0f;
          }
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          z = fmaf(G[r], 0.0f, z);
          sA[(t + r) * kLd + u] = G[r];
        }
      }
    }
    if (__builtin_expect(__any(z != 0.0f), 0)) {
      // entries that are not finite: none enters the inverse, rows from the first on are lost
#pragma unroll
      for (int part = 0; part < 2; ++part) {
        const int i = part ? i1 : i0, t = 16 * i + 4 * gq;
#pragma unroll
        for (int c = 0; c < (part ? 2 : 4); ++c) {
          if (c > i) continue;
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (!(fabsf(part ? G1[c & 1][r] : G0[c][r]) < INFINITY)) {
              atomicMin(&sBad, t + r);
              sA[(t + r) * kLd + 16 * c + n] = 0.0f;
            }
        }
      }
    }
  } else {
    // columns of P^T: wave 2 the even row tiles of P, wave 3 the odd ones, each against tiles 0, 1 and then 0 .. 3
    const int odd = w - 2;
    floatx4 P[6] = {}, qq[2] = {};
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      bf16x8 fk[4], fq[2];
#pragma unroll
      for (int c = 0; c < 4; ++c)
        fk[c] = as_frag(*reinterpret_cast<const uint4*>(sK + swz<DKP>(tile_row(c, n), 4 * s + gq)));
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        fq[i] = as_frag(*reinterpret_cast<const uint4*>(sQ + swz<DKP>(tile_row(2 * i, n) + 4 * odd, 4 * s + gq)));
        qq[i] = mfma_bf(fq[i], fq[i], qq[i]);
      }
      P[0] = mfma_bf(fk[0], fq[0], P[0]);
      P[1] = mfma_bf(fk[1], fq[0], P[1]);
#pragma unroll
      for (int c = 0; c < 4; ++c) P[2 + c] = mfma_bf(fk[c], fq[1], P[2 + c]);
    }
    if (diagonal) {
#pragma unroll
      for (int i = 0; i < 2; ++i) sRq[tile_row(2 * i, n) + 4 * odd] = inverse_length(qq[i]);
    }
    exchange_barrier();
#pragma unroll
    for (int f = 0; f < 3; ++f) {  // fragments odd, 2 + odd, 4 + odd
      const int t = tile_row(f ? 2 : 0, n) + 4 * odd, c0 = f == 2 ? 2 : 0;
      const double bt = sB[t];
      const float pt = a.scale * sRq[t] * (f == 1 ? sMid[t] : 1.0f);
      uint32_t p[8];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int u = tile_row(c0 + c, 4 * gq);
        const float4 rk = *reinterpret_cast<const float4*>(sRk + u), mid = *reinterpret_cast<const float4*>(sMid + u);
        const float k[4] = {rk.x, rk.y, rk.z, rk.w}, m[4] = {mid.x, mid.y, mid.z, mid.w};
        float v[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float e = f == 1 ? m[r] : __builtin_amdgcn_exp2f(static_cast<float>(bt - sB[u + r]));
          v[r] = pt * (k[r] * e) * P[2 * f + c][r];
          if (f != 1) v[r] = u + r <= t ? v[r] : 0.0f;
        }
        cut<2>(v[0], v[1], p + 2 * c, 4);
        cut<2>(v[2], v[3], p + 2 * c + 1, 4);
      }
      uint4* to = reinterpret_cast<uint4*>(rec + kFragsT) + 128 * (2 * f + odd) + lane;
      to[0] = make_uint4(p[0], p[1], p[2], p[3]);
      to[64] = make_uint4(p[4], p[5], p[6], p[7]);
    }
    if (w == 3) {
      float* c = rec + kFrags;
      const double b = sB[lane], end = sB[kC - 1];
      const float e = __builtin_amdgcn_exp2f(static_cast<float>(b)), bb = sBeta[lane];
      c[lane] = bb * e * sRk[lane];
      c[64 + lane] = e * sRq[lane] * a.scale;
      c[128 + lane] = __builtin_amdgcn_exp2f(static_cast<float>(end - b)) * sRk[lane];
      c[192 + lane] = bb;
      if (lane == 0) c[256] = __builtin_amdgcn_exp2f(static_cast<float>(end));
    }
  }
  exchange_barrier();
  // rows 16 w .. of the inverse: two 8 x 8 blocks, lane (block, column), zeros between them
  if (lane < 16) {
    const int d = 16 * w + (n & 8);
    const float* A = sA + d * kLd + d;
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float v = i == (n & 7) ? 1.0f : 0.0f;
#pragma unroll
      for (int m = 0; m < i; m += 4) {
        const float4 r = *reinterpret_cast<const float4*>(A + i * kLd + m);
        v = fmaf(-r.x, x[m], v);
        if (m + 1 < i) v = fmaf(-r.y, x[m + 1], v);
        if (m + 2 < i) v = fmaf(-r.z, x[m + 2], v);
        if (m + 3 < i) v = fmaf(-r.w, x[m + 3], v);
      }
      x[i] = v;
    }
    float* T = sT + 16 * w * kLd + 16 * w + n;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      T[(i + (n & 8)) * kLd] = x[i];
      T[(i + 8 - (n & 8)) * kLd] = 0.0f;
    }
  }
  {  // 16 x 16: the wave's own block, so no barrier; A's entries outside the lower left 8 x 8 are left out
    float* T = sT + 16 * w * kLd + 16 * w;
    const float* A = sA + 16 * w * kLd + 16 * w;
    __builtin_amdgcn_wave_barrier();
    floatx4 m = {}, o = {};
    const floatx4 t1 = column4(T + 4 * gq * kLd + n);
    const float4 ar = *reinterpret_cast<const float4*>(A + n * kLd + 4 * gq);
    const bool low = n >= 8 && gq < 2;
    m = __builtin_amdgcn_mfma_f32_16x16x4f32(low ? ar.x : 0.0f, t1[0], m, 0, 0, 0);
    m = __builtin_amdgcn_mfma_f32_16x16x4f32(low ? ar.y : 0.0f, t1[1], m, 0, 0, 0);
    m = __builtin_amdgcn_mfma_f32_16x16x4f32(low ? ar.z : 0.0f, t1[2], m, 0, 0, 0);
    m = __builtin_amdgcn_mfma_f32_16x16x4f32(low ? ar.w : 0.0f, t1[3], m, 0, 0, 0);
    o = mfma_f32(T + n * kLd + 4 * gq, m, o);
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (n < 8 && gq >= 2) T[(4 * gq + r) * kLd + n] = -o[r];
  }
  exchange_barrier();
  if (w < 2) {  // 32 x 32: below the diagonal of pair w
    const int lo = 32 * w, up = 32 * w + 16;
    floatx4 m = {}, o = {};
    m = mfma_f32(sA + (up + n) * kLd + lo + 4 * gq, column4(sT + (lo + 4 * gq) * kLd + lo + n), m);
    o = mfma_f32(sT + (up + n) * kLd + up + 4 * gq, m, o);
#pragma unroll
    for (int r = 0; r < 4; ++r) sT[(up + 4 * gq + r) * kLd + lo + n] = -o[r];
  } else {  // and zeros above it
#pragma unroll
    for (int r = 0; r < 4; ++r) sT[(32 * (w - 2) + 4 * gq + r) * kLd + 32 * (w - 2) + 16 + n] = 0.0f;
  }
  exchange_barrier();
  {  // the lower left 32 x 32 block: wave w has rows 16 (w / 2) and columns 16 (w % 2) of it
    const int c = 16 * (w & 1), p = 32 + 16 * (w >> 1);
    const floatx4 t0 = column4(sT + 4 * gq * kLd + c + n), t1 = column4(sT + (16 + 4 * gq) * kLd + c + n);
    floatx4 m[2] = {}, o[2] = {};
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      m[j] = mfma_f32(sA + (32 + 16 * j + n) * kLd + 4 * gq, t0, m[j]);
      m[j] = mfma_f32(sA + (32 + 16 * j + n) * kLd + 16 + 4 * gq, t1, m[j]);
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) o[j] = mfma_f32(sT + (p + n) * kLd + 32 + 16 * j + 4 * gq, m[j], o[j]);
#pragma unroll
    for (int r = 0; r < 4; ++r) sT[(p + 4 * gq + r) * kLd + c + n] = -o[0][r] - o[1][r];
  }
  exchange_barrier();
  const int bad = sBad;
#pragma unroll
  for (int q = 0; q < 3; ++q) {  // 12 halves of fragments
    const int e = 4 * q + w, f = e >> 1, k = 32 * frag_k(f) + 8 * gq + 4 * (e & 1), t = tile_row(frag_row(f), n);
    const float4 v = *reinterpret_cast<const float4*>(sT + t * kLd + k);
    float x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int r = 0; r < 4; ++r) x[r] = k + r < t ? (t < bad ? x[r] : NAN) : 0.0f;
    uint32_t terms[6];
    cut<3>(x[0], x[1], terms, 2);
    cut<3>(x[2], x[3], terms + 1, 2);
    uint2* to = reinterpret_cast<uint2*>(rec) + (3 * f * 64 + lane) * 2 + (e & 1);
#pragma unroll
    for (int i = 0; i < 3; ++i) to[128 * i] = make_uint2(terms[2 * i], terms[2 * i + 1]);
  }
}

// first token of a lane's column that is not finite, over the lanes of the column; such entries become zero
__device__ inline int cut_out(floatx4* x, int gq) {
  int at = kC;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (!(fabsf(x[i][r]) < INFINITY)) {
        at = min(at, tile_row(i, 4 * gq + r));
        x[i][r] = 0.0f;
      }
  at = min(at, __shfl_xor(at, 16, kWave));
  return min(at, __shfl_xor(at, 32, kWave));
}
__device__ inline bool any_not_finite(const floatx4* x) {
  floatx4 z = {};
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int r = 0; r < 4; ++r) z[r] = fmaf(x[i][r], 0.0f, z[r]);
  return __any((z[0] + z[1]) + (z[2] + z[3]) != 0.0f);  // 0 x infinity and 0 x NaN are NaN
}

__device__ inline uint2 read_tr(const uint16_t* p) {
  typedef __attribute__((address_space(3))) shortx4 lds_s4;
  const shortx4 v = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4*)p);
  uint2 r;
  __builtin_memcpy(&r, &v, 8);
  return r;
}

// waits for all but the wave's N latest loads and stores, then for the workgroup's
template <int N>
__device__ inline void landed_barrier() {
  static_assert(N < 64);
  __builtin_amdgcn_s_waitcnt(0x0F70 | (N & 15) | (N >> 4) << 14);  // vmcnt(N)
  exchange_barrier();
}

// The scan with 16 G columns on 2 G waves.  Wave i < G holds 16 columns of the
// state, every row, on the way from state to state; wave G + i takes the outputs
// of these columns, half a block behind, and the loads.  It gets S and U through
// LDS, cut into the two terms that the outputs take.  Where all CUs are busy the
// products bound it, with the cutting between them (128 heads of 128 x 128, 8192
// tokens: 455 us at the full clock, 860 TFLOP/s on the matrix cores; 580 once the
// card lowers its clock under that load).
template <int DKP, int G>
struct ScanLds {
  uint16_t K[2][kC * DKP], T[2][2 * kFragsT];
  float C[2][256];                         // a block's and the next's
  uint16_t V[kC * 16 * G], Q[kC * DKP], P[2 * kFragsP];
  uint32_t S[G][2 * DKP / 32 * 256], U[G][4 * 256];  // fragments: 64 lanes x 8 terms, 1 KB each
  int lost[16 * G];                         // first token of the column whose u is not finite
};
static_assert(sizeof(ScanLds<128, 4>) <= 160 * 1024, "LDS of a CU");

template <int DKP, int G>
__global__ __launch_bounds__(128 * G) void delta_scan(DeltaArgs a, const float* ws, int cols) {
  constexpr int NS = DKP / 32;         // inner steps of 32 over the state's rows
  constexpr int PR = DKP / 8;          // pieces of a staged row
  constexpr int NK = PR / G;           // pieces of K (and of Q) a thread loads
  __shared__ __align__(1024) ScanLds<DKP, G> L;
  const int lane = threadIdx.x & 63, n = lane & 15, gq = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), w = wave % G, tid = 64 * w + lane;
  // the column parts of a head follow each other on one XCD, whose L2 then holds its K, Q, T and P once
  const int id = blockIdx.y * gridDim.x + blockIdx.x, part = id / 8 % cols, head = id / (8 * cols) * 8 + id % 8;
  if (head >= a.nseq * a.hv) return;
  const int s = head / a.hv, h = head % a.hv, kh = h / (a.hv / a.hk);
  const int wcol = part * 16 * G, col = wcol + 16 * w + n;
  const bool in = col < a.dv;
  int64_t t0, t1;
  seq_span(a, s, &t0, &t1);
  const int blocks = static_cast<int>((t1 - t0 + kC - 1) / kC);
  const float* rec = ws + ((t0 / kC + s) * a.hv + h) * kRec;
  const int64_t next_rec = static_cast<int64_t>(a.hv) * kRec;
  const auto v_at = [](int row, int p) { return row * 16 * G + 8 * (p ^ (row & 2)); };
  const auto frag = [&](const void* f, int i) __attribute__((always_inline)) {
    return as_frag(*(reinterpret_cast<const uint4*>(f) + i * 64 + lane));
  };
  if (wave < G) {
    const int64_t at = static_cast<int64_t>(head) * a.dk * a.dv + col;
    floatx4 S[2 * NS];
#pragma unroll
    for (int i = 0; i < 2 * NS; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int d = tile_row(i, 4 * gq + r);
        S[i][r] = a.state_in && in && d < a.dk ? a.state_in[at + static_cast<int64_t>(d) * a.dv] : 0.0f;
      }
    const auto step = [&](const uint16_t* sK, const uint16_t* sT, const float* sC, float eC) __attribute__((always_inline)) {
      // K S0
      floatx4 X[4] = {};
#pragma unroll
      for (int k = 0; k < NS; ++k) {
        bf16x8 fk[4], f[3];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          fk[i] = as_frag(*reinterpret_cast<const uint4*>(sK + swz<DKP>(tile_row(i, n), 4 * k + gq)));
        cut_pair<3>(S[2 * k], S[2 * k + 1], f);
#pragma unroll
        for (int t = 0; t < 2; ++t) *reinterpret_cast<bf16x8*>(L.S[w] + ((2 * k + t) * 64 + lane) * 4) = f[t];
#pragma unroll
        for (int t = 2; t >= 0; --t)
#pragma unroll
          for (int i = 0; i < 4; ++i) X[i] = mfma_bf(fk[i], f[t], X[i]);
      }
      // X = diag(beta) (V - diag(e^b) K S0)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = tile_row(i, 4 * gq);
        const uint2 v = read_tr(L.V + v_at(t + (n >> 2), 2 * w + ((n >> 1) & 1)) + 4 * (n & 1));
        const float4 c1 = *reinterpret_cast<const float4*>(sC + t), be = *reinterpret_cast<const float4*>(sC + 192 + t);
        X[i][0] = __uint_as_float(v.x << 16) * be.x - c1.x * X[i][0];
        X[i][1] = __uint_as_float(v.x & 0xFFFF0000u) * be.y - c1.y * X[i][1];
        X[i][2] = __uint_as_float(v.y << 16) * be.z - c1.z * X[i][2];
        X[i][3] = __uint_as_float(v.y & 0xFFFF0000u) * be.w - c1.w * X[i][3];
      }
      // U = X + (T - I) X
      floatx4 U[4];
      const auto solve = [&]() __attribute__((always_inline)) {
        bf16x8 f[2][3];
        cut_pair<3>(X[0], X[1], f[0]);
        cut_pair<3>(X[2], X[3], f[1]);
        // six chains, the two of a lower tile added at the end
        floatx4 u[6];
#pragma unroll
        for (int b = 0; b < 6; ++b) u[b] = b < 4 ? X[b] : floatx4{};
#pragma unroll
        for (int j = 2; j >= 0; --j) {  // term j of T with terms 2 - j .. 0 of X, the smallest products first
          bf16x8 t[6];
#pragma unroll
          for (int b = 0; b < 6; ++b) t[b] = frag(sT, b * 3 + j);
#pragma unroll
          for (int i = 2 - j; i >= 0; --i)
#pragma unroll
            for (int b = 0; b < 6; ++b) u[b] = mfma_bf(t[b], f[frag_k(b)][i], u[b]);
        }
        U[0] = u[0];
        U[1] = u[1];
        U[2] = u[2] + u[4];
        U[3] = u[3] + u[5];
      };
      solve();
      int lost = kC;  // first token of this column whose u is not finite
      if (__builtin_expect(any_not_finite(U), 0)) {
        lost = cut_out(X, gq);
        solve();
        lost = min(lost, cut_out(U, gq));
      }
      float4 c3[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) c3[i] = *reinterpret_cast<const float4*>(sC + 128 + tile_row(i, 4 * gq));
      exchange_barrier();  // the outputs of the block before are made
      if (gq == 0) L.lost[16 * w + n] = lost;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        bf16x8 f[2];
        cut_pair<2>(U[2 * k], U[2 * k + 1], f);
#pragma unroll
        for (int t = 0; t < 2; ++t) *reinterpret_cast<bf16x8*>(L.U[w] + ((2 * k + t) * 64 + lane) * 4) = f[t];
      }
      // S = e^(b_C) S0 + K^T diag(e^(b_C - b)) U
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        U[i][0] *= c3[i].x; U[i][1] *= c3[i].y; U[i][2] *= c3[i].z; U[i][3] *= c3[i].w;
      }
      bf16x8 f[2][3];
      cut_pair<3>(U[0], U[1], f[0]);
      cut_pair<3>(U[2], U[3], f[1]);
#pragma unroll
      for (int j = 0; j < 2 * NS; j += 4) {  // four tiles of the state at a time
#pragma unroll
        for (int i = j; i < j + 4; ++i) S[i] *= eC;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          bf16x8 fk[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int row = 32 * k + 8 * gq + (n >> 2), p = 4 * ((j + i) >> 1) + (n & 3);
            const uint2 lo = read_tr(sK + swz<DKP>(row, p) + 4 * (i & 1));
            const uint2 hi = read_tr(sK + swz<DKP>(row + 4, p) + 4 * (i & 1));
            fk[i] = as_frag(make_uint4(lo.x, lo.y, hi.x, hi.y));
          }
#pragma unroll
          for (int t = 2; t >= 0; --t)
#pragma unroll
            for (int i = 0; i < 4; ++i) S[j + i] = mfma_bf(fk[i], f[k][t], S[j + i]);
        }
      }
      if (__builtin_expect(__any(lost < kC), 0)) {
#pragma unroll
        for (int i = 0; i < 2 * NS; ++i)
          if (lost < kC) S[i] = floatx4{NAN, NAN, NAN, NAN};
      }
    };
    if (blocks > 0) {
      float eC = rec[kFrags + 256];
      for (int c = 0; c < blocks; ++c) {
        if (c + 1 < blocks) rec += next_rec;
        exchange_barrier();  // this block is in LDS, the outputs of the one before have taken S
        const float e = eC;
        eC = rec[kFrags + 256];
        step(L.K[c & 1], L.T[c & 1], L.C[c & 1], e);
      }
      exchange_barrier();
    }
    if (!a.state_out || !in) return;
#pragma unroll
    for (int i = 0; i < 2 * NS; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int d = tile_row(i, 4 * gq + r);
        if (d < a.dk) a.state_out[at + static_cast<int64_t>(d) * a.dv] = S[i][r];
      }
    return;
  }
  const int os = a.hv * a.dv;
  // the block whose K, T and decays are loaded next, and its V; the block whose Q and P are; the outputs to store
  const uint16_t* pk = a.k + static_cast<int64_t>(kh) * a.dk + t0 * a.ks;
  const uint16_t* pq = a.q + static_cast<int64_t>(kh) * a.dk + t0 * a.qs;
  const uint16_t* pv = a.v + static_cast<int64_t>(h) * a.dv + t0 * a.vs;
  const float* recp = rec;
  int left = static_cast<int>(t1 - t0), done = 0;  // tokens from the former block to the sequence's end; from the latter
  uint16_t* po = a.o + (t0 * a.hv + h) * a.dv - static_cast<int64_t>(kC) * os;
  // where this lane's pieces lie in a block: piece e of the LDS image holds piece
  // (e % PR) ^ swap(row) of row e / PR
  int ak[NK], aq[NK], av[2];
#pragma unroll
  for (int i = 0; i < NK; ++i) {
    const int row = (i * 64 * G + tid) / PR, p = (swz<DKP>(row, tid % PR) >> 3) % PR;
    ak[i] = piece_at(row, a.ks, 8 * p, a.dk);
    aq[i] = piece_at(row, a.qs, 8 * p, a.dk);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int row = (i * 64 * G + tid) / (2 * G), p = (v_at(row, tid % (2 * G)) >> 3) % (2 * G);
    av[i] = piece_at(row, a.vs, wcol + 8 * p, a.dv);
  }
  constexpr int kTc = 20 / G;
  const auto fetch_ktc = [&](uint16_t* nK, uint16_t* nT, float* nC) __attribute__((always_inline)) {
    const Rows K = rows_at(pk, a.ks, left, a.dk);
    const Rows R = __builtin_amdgcn_make_buffer_rsrc(const_cast<float*>(rec), 0, 4 * kRec, 0x00027000);
#pragma unroll
    for (int i = 0; i < NK; ++i) to_lds(K, ak[i], nK + (i * G + w) * 512);
#pragma unroll
    for (int i = 0; i < kTc; ++i) {  // 18 KB of T, then the decays, twice to keep the waves' loads alike
      const int u = i * G + w;
      to_lds(R, (u < 18 ? u * 1024 : 4 * kFrags) + 16 * lane,
             u < 18 ? static_cast<void*>(nT + u * 512) : static_cast<void*>(nC));
    }
    pk += kC * a.ks;
    if (left > kC) rec += next_rec;
  };
  const auto fetch_v = [&](uint16_t* nV) __attribute__((always_inline)) {
    const Rows V = rows_at(pv, a.vs, left, a.dv);
#pragma unroll
    for (int i = 0; i < 2; ++i) to_lds(V, av[i], nV + (i * G + w) * 512);
    pv += kC * a.vs;
    left -= kC;
  };
  const int o_at = in ? 2 * (8 * gq * os + col) : kOutside;  // row tile_row(0, 4 gq)
  floatx4 O[4] = {};
  // P U and the stores of the block before, from the s buffers
  const auto finish = [&](const uint16_t* __restrict__ sP, const uint32_t* __restrict__ sU,
                          const int* __restrict__ sLost) __attribute__((always_inline)) {
    bf16x8 f[2][2], ph[6], pl[6];
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int t = 0; t < 2; ++t) f[k][t] = frag(sU, 2 * k + t);
#pragma unroll
    for (int b = 0; b < 6; ++b) {
      pl[b] = frag(sP, 2 * b + 1);
      ph[b] = frag(sP, 2 * b);
    }
    const int lost = sLost[16 * w + n];
    floatx4 o[6] = {O[0], O[1], O[2], O[3]};
#pragma unroll
    for (int b = 0; b < 6; ++b) o[b] = mfma_bf(pl[b], f[frag_k(b)][0], o[b]);
#pragma unroll
    for (int b = 0; b < 6; ++b) o[b] = mfma_bf(ph[b], f[frag_k(b)][1], o[b]);
#pragma unroll
    for (int b = 0; b < 6; ++b) o[b] = mfma_bf(ph[b], f[frag_k(b)][0], o[b]);
    o[2] += o[4];
    o[3] += o[5];
    if (__builtin_expect(__any(lost < kC), 0)) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (tile_row(i, 4 * gq + r) >= lost) o[i][r] = NAN;
    }
    const Rows to = rows_at(po, os, done, a.dv);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const floatx4 v = o[i >> 1];
      const bf16x2 b = __builtin_convertvector((i & 1 ? floatx2{v[2], v[3]} : floatx2{v[0], v[1]}), bf16x2);
      uint32_t two;
      __builtin_memcpy(&two, &b, 4);
      const int to_at = o_at + 2 * os * (32 * (i >> 2) + 4 * ((i >> 1) & 1) + 2 * (i & 1));
      __builtin_amdgcn_raw_buffer_store_b16(static_cast<uint16_t>(two), to, to_at, 0, 0);
      __builtin_amdgcn_raw_buffer_store_b16(static_cast<uint16_t>(two >> 16), to, to_at + 2 * os, 0, 0);
    }
  };
  constexpr int kStores = 16;
  // The loads into the n buffers go out beside the products from the s buffers;
  // restrict arguments keep the reads from waiting for the loads.
  const auto first_half = [&](uint16_t* __restrict__ nQ, uint16_t* __restrict__ nK, uint16_t* __restrict__ nT,
                              float* __restrict__ nC, const uint16_t* __restrict__ sP, const uint32_t* __restrict__ sU,
                              const int* __restrict__ sLost) __attribute__((always_inline)) {
    const int tokens = left + kC;
    const Rows Q = rows_at(pq, a.qs, tokens, a.dk);
#pragma unroll
    for (int i = 0; i < NK; ++i) to_lds(Q, aq[i], nQ + (i * G + w) * 512);
    pq += kC * a.qs;
    __asm__ volatile("" ::: "memory");  // Q before the others: they are counted
    fetch_ktc(nK, nT, nC);  // after the last block zeros and that block's T again: no branch around it
    finish(sP, sU, sLost);  // before the first block nothing is stored
    po += static_cast<int64_t>(kC) * os;
    done = tokens;
  };
  const auto second_half = [&](uint16_t* __restrict__ nP, uint16_t* __restrict__ nV, const uint16_t* __restrict__ sQ,
                               const uint32_t* __restrict__ sS,
                               const float* __restrict__ sC) __attribute__((always_inline)) {
    const Rows R = __builtin_amdgcn_make_buffer_rsrc(const_cast<float*>(recp), 0, 4 * kRec, 0x00027000);
#pragma unroll
    for (int i = 0; i < 12 / G; ++i) to_lds(R, 4 * kFragsT + (i * G + w) * 1024 + 16 * lane, nP + (i * G + w) * 512);
    recp += next_rec;
    fetch_v(nV);
#pragma unroll
    for (int i = 0; i < 4; ++i) O[i] = floatx4{};
#pragma unroll
    for (int k = 0; k < NS; ++k) {
      bf16x8 fq[4], f[2];
#pragma unroll
      for (int t = 0; t < 2; ++t) f[t] = frag(sS, 2 * k + t);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        fq[i] = as_frag(*reinterpret_cast<const uint4*>(sQ + swz<DKP>(tile_row(i, n), 4 * k + gq)));
#pragma unroll
      for (int t = 1; t >= 0; --t)
#pragma unroll
        for (int i = 0; i < 4; ++i) O[i] = mfma_bf(fq[i], f[t], O[i]);
    }
    // O = diag(e^b) Q S0 (+ P U; the scale is in both)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 c2 = *reinterpret_cast<const float4*>(sC + 64 + tile_row(i, 4 * gq));
      O[i][0] *= c2.x; O[i][1] *= c2.y; O[i][2] *= c2.z; O[i][3] *= c2.w;
    }
  };
  if (blocks > 0) {
    fetch_ktc(L.K[0], L.T[0], L.C[0]);
    fetch_v(L.V);
    for (int c = 0; c < blocks; ++c) {
      const int i = c & 1;
      landed_barrier<0>();
      first_half(L.Q, L.K[i ^ 1], L.T[i ^ 1], L.C[i ^ 1], L.P, L.U[w], L.lost);
      landed_barrier<NK + kTc + kStores>();  // Q
      second_half(L.P, L.V, L.Q, L.S[w], L.C[i]);
    }
    landed_barrier<0>();  // nothing is on its way into LDS when the workgroup ends
    finish(L.P, L.U[w], L.lost);
  }
}

// Brings a block's lines into L2, a quarter of a kilobyte of LDS taking what nobody reads:
// the way from memory is about as long as a block takes, so the loads into LDS alone,
// a block ahead, come late (the scan of 16 ragged prompts of 8 heads of 64 x 64 at 16 columns a
// workgroup: 360 us without, 334 with; delta_prep's 95 before it are apart).
// NV lines of 64 columns of v; every wave of NW issues kLoads.
template <int DKP, int NV, int NW>
struct Ahead {
  static constexpr int kRows = DKP / 64, kUnits = 4 + 2 * kRows + NV, kLoads = (kUnits + NW - 1) / NW;
  static_assert(kLoads <= 15, "counted by vmcnt's low bits");
  static __device__ inline void touch(int w, const float* rec, const uint16_t* k, const uint16_t* q, const uint16_t* v,
                                      int ks, int qs, int vs, int rows, int dk, int dv, void* unused) {
    typedef __attribute__((address_space(3))) void lds_void;
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
      const int u = w + j * NW, m = u - 4;  // uniform
      int64_t base = reinterpret_cast<int64_t>(rec);
      int stride = 64, line = 8192 * u, width = 0, bytes = 4 * kRec;
      if (m >= 0) {
        base = m < kRows       ? reinterpret_cast<int64_t>(k)
               : m < 2 * kRows ? reinterpret_cast<int64_t>(q)
                               : reinterpret_cast<int64_t>(v);
        stride = m < kRows ? +ks : m < 2 * kRows ? +qs : +vs;
        width = m < 2 * kRows ? +dk : +dv;
        line = 128 * (m < kRows ? m : m < 2 * kRows ? m - kRows : m - 2 * kRows);
        bytes = rows > 0 && u < kUnits ? 2 * ((min(rows, kC) - 1) * stride + width) : 0;
      }
      const Rows r = __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(base), 0,
                                                       __builtin_amdgcn_readfirstlane(bytes), 0x00027000);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)unused, 4, 2 * lane_id() * stride + line, 0, 0, 0);
    }
  }
};

// The scan with 16 columns on eight waves.  Wave i < 4 holds a quarter of the
// state's rows and takes tile i of the block's tokens (16 of them) on the way from
// state to state; wave 4 + i takes that tile's outputs, which nothing waits for,
// and the loads.  What a product needs of other waves (S, X and U, cut into terms
// by the wave that made them) goes through LDS, with three barriers a block.
// The chain from barrier to barrier bounds it: LDS latency, six to twelve products
// and the cutting of a tile or two (4 heads of 128 x 128, 8192 tokens: 203 us,
// 1.6 us a block; with one wave for all of it 3.1 us; in five segments 41 + 50 us).
template <int DKP>
struct QuarterLds {
  struct {
    uint16_t K[kC * DKP], Q[kC * DKP], V[kC * 16], T[2 * kFragsT], P[2 * kFragsP];
    float C[256];
  } in[2];                             // a block and the next
  uint32_t S[3 * DKP / 32 * 256], X[6 * 256], U[10 * 256];   // fragments: 64 lanes x 8 terms, 1 KB each
  int lost[64];                        // [column][wave]: first token whose u is not finite
  uint32_t unused[64];                 // what the loads that only bring lines into L2 leave behind
};
static_assert(sizeof(QuarterLds<128>) <= 160 * 1024, "LDS of a CU");

__device__ inline bool tile_not_finite(const floatx4& x) {
  const float z = fmaf(x[0], 0.0f, x[1] * 0.0f) + fmaf(x[2], 0.0f, x[3] * 0.0f);
  return __any(z != 0.0f);  // 0 x infinity and 0 x NaN are NaN
}
__device__ inline int cut_out_tile(floatx4* x, int t) {  // t: token of (*x)[0]
  int at = kC;
#pragma unroll
  for (int r = 3; r >= 0; --r)
    if (!(fabsf((*x)[r]) < INFINITY)) {
      at = t + r;
      (*x)[r] = 0.0f;
    }
  at = min(at, __shfl_xor(at, 16, kWave));
  return min(at, __shfl_xor(at, 32, kWave));
}
// tile i of an operand's rows, cut into N terms, into its half of the fragments at f (of 32 rows: N of them)
template <int N>
__device__ inline void put_tile(uint32_t* f, int i, int lane, const floatx4& x) {
  uint32_t w[2 * N];
  cut<N>(x[0], x[1], w, 2);
  cut<N>(x[2], x[3], w + 1, 2);
#pragma unroll
  for (int t = 0; t < N; ++t)
    *reinterpret_cast<uint2*>(f + (((i >> 1) * N + t) * 64 + lane) * 4 + 2 * (i & 1)) = make_uint2(w[2 * t], w[2 * t + 1]);
}

// A long sequence of few heads in segments of `len` blocks.  The state after a
// segment is linear in the state before it, S' = M S + N: kTransfer finds [N | M]
// of every segment but the last at once, as the scan from a zero state and, with
// zero values, from the unit columns; the first segment starts from its state
// and needs no M.  kSegments walks these to its segment's first state, then
// scans the segment.  The sequence's state is copied by kTransfer, so that in
// kSegments nobody reads the array to which the last segment may write.
enum Part { kWhole, kTransfer, kSegments };
struct Segments {
  float* m;      // for each segment and head N, DKP rows of 16 ceil(dv / 16) values, and M's fragments in three bf16 terms
  float* first;  // for each sequence and head DKP rows of its state, 16 ceil(dv / 16) values each
  int len;
};
__device__ __host__ constexpr int map_words(int dkp, int pitch) { return dkp * pitch + dkp * dkp * 3 / 2; }
__device__ __host__ inline int64_t segment_slot(int64_t t0, int s, int len) { return t0 / kC / len + s; }

template <int DKP, Part PART>
__global__ __launch_bounds__(512) void delta_scan_quarters(DeltaArgs a, const float* ws, int cols, Segments sg) {
  constexpr int NS = DKP / 32, PR = DKP / 8, NK = PR / 4, TS = DKP / 64;  // TS: tiles of the state a wave holds
  __shared__ __align__(1024) QuarterLds<DKP> L;
  const int lane = threadIdx.x & 63, n = lane & 15, gq = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), w = wave & 3, tid = 64 * w + lane;
  // the column parts of a head and segment follow each other on one XCD
  const int id = blockIdx.x, part = id / 8 % cols, unit = id / (8 * cols) * 8 + id % 8, heads = a.nseq * a.hv;
  const int seg = PART == kWhole ? 0 : unit / heads, head = unit - seg * heads;
  if (PART == kWhole && unit >= heads) return;
  const int s = head / a.hv, h = head % a.hv, kh = h / (a.hv / a.hk);
  const int wcol = part * 16, col = wcol + n;
  const bool in = col < a.dv;
  int64_t t0, t1;
  seq_span(a, s, &t0, &t1);
  const int64_t record = t0 / kC + s + (PART == kWhole ? 0 : int64_t(seg) * sg.len);
  const int pitch = (a.dv + 15) / 16 * 16, next_map = a.hv * map_words(DKP, pitch);
  float *m = nullptr, *first = nullptr;  // [N | M] of the sequence's first segment
  bool last = true;
  if (PART != kWhole) {
    const int segments = max(static_cast<int>((t1 - t0 + int64_t(sg.len) * kC - 1) / (int64_t(sg.len) * kC)), 1);
    last = seg == segments - 1;
    if (PART == kTransfer ? seg >= segments - 1 || (seg == 0 && wcol >= pitch) : seg >= segments) return;
    if (segments > 1) first = sg.first + static_cast<int64_t>(head) * DKP * pitch + col;
    m = sg.m + (segment_slot(t0, s, sg.len) * a.hv + h) * map_words(DKP, pitch);
    t0 += int64_t(seg) * sg.len * kC;
    t1 = min(t1, t0 + int64_t(sg.len) * kC);
  }
  const int blocks = static_cast<int>((t1 - t0 + kC - 1) / kC);
  const float* rec = ws + (record * a.hv + h) * kRec;
  const int64_t next_rec = static_cast<int64_t>(a.hv) * kRec;
  const int t4 = tile_row(w, 4 * gq);  // the lane's tokens: t4 .. t4 + 3
  const auto frag = [&](const void* f, int i) __attribute__((always_inline)) {
    return as_frag(*(reinterpret_cast<const uint4*>(f) + i * 64 + lane));
  };
  if (wave < 4) {
    const int64_t at = static_cast<int64_t>(head) * a.dk * a.dv + col;
    floatx4 S[TS];
#pragma unroll
    for (int i = 0; i < TS; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int d = tile_row(TS * w + i, 4 * gq + r);
        const auto given = [&]() {
          return a.state_in && in && d < a.dk ? a.state_in[at + static_cast<int64_t>(d) * a.dv] : 0.0f;
        };
        if (PART == kTransfer && seg > 0)
          S[i][r] = d == wcol - pitch + n ? 1.0f : 0.0f;
        else if (PART == kTransfer)
          first[d * pitch] = S[i][r] = given();
        else if (PART == kSegments && seg > 0)
          S[i][r] = m[d * pitch + col];
        else if (PART == kSegments && first)
          S[i][r] = first[d * pitch];
        else
          S[i][r] = given();
      }
    const auto put_state = [&]() __attribute__((always_inline)) {
      if constexpr (TS == 2) {
        bf16x8 f[3];
        cut_pair<3>(S[0], S[1], f);
#pragma unroll
        for (int t = 0; t < 3; ++t) *reinterpret_cast<bf16x8*>(L.S + ((w * 3 + t) * 64 + lane) * 4) = f[t];
      } else {
        put_tile<3>(L.S, w, lane, S[0]);
      }
    };
    const auto step = [&](const auto& in, float eC) __attribute__((always_inline)) {
      // K S0 of the wave's tokens, a chain for each term of S0
      floatx4 x[3] = {};
      bf16x8 fk[NS], fs[NS][3];
#pragma unroll
      for (int k = 0; k < NS; ++k) {
        fk[k] = as_frag(*reinterpret_cast<const uint4*>(in.K + swz<DKP>(tile_row(w, n), 4 * k + gq)));
#pragma unroll
        for (int t = 0; t < 3; ++t) fs[k][t] = frag(L.S, 3 * k + t);
      }
      const uint2 v = read_tr(in.V + (t4 + (n >> 2)) * 16 + 4 * (n & 3));
      const float4 c1 = *reinterpret_cast<const float4*>(in.C + t4), c3 = *reinterpret_cast<const float4*>(in.C + 128 + t4),
                   be = *reinterpret_cast<const float4*>(in.C + 192 + t4);
      bf16x8 ft[2][3];
#pragma unroll
      for (int t = 0; t < 3; ++t) {
        ft[0][t] = frag(in.T, 3 * w + t);
        if (w >= 2) ft[1][t] = frag(in.T, 3 * (w + 2) + t);
      }
#pragma unroll
      for (int k = 0; k < NS; ++k)
#pragma unroll
        for (int t = 2; t >= 0; --t) x[t] = mfma_bf(fk[k], fs[k][t], x[t]);
      floatx4 X = (x[2] + x[1]) + x[0];
      X[0] = __uint_as_float(v.x << 16) * be.x - c1.x * X[0];
      X[1] = __uint_as_float(v.x & 0xFFFF0000u) * be.y - c1.y * X[1];
      X[2] = __uint_as_float(v.y << 16) * be.z - c1.z * X[2];
      X[3] = __uint_as_float(v.y & 0xFFFF0000u) * be.w - c1.w * X[3];
      int lost = kC;
      if (__builtin_expect(tile_not_finite(X), 0)) lost = cut_out_tile(&X, t4);
      put_tile<3>(L.X, w, lane, X);
      exchange_barrier();
      // U = X + (T - I) X
      floatx4 u[6] = {X};
      bf16x8 fx[3];
#pragma unroll
      for (int t = 0; t < 3; ++t) fx[t] = frag(L.X, t);
      const auto solve = [&](const bf16x8* ft, floatx4* u) __attribute__((always_inline)) {
        u[2] = mfma_bf(ft[2], fx[0], u[2]);
        u[1] = mfma_bf(ft[1], fx[0], u[1]);
        u[0] = mfma_bf(ft[0], fx[0], u[0]);
        u[2] = mfma_bf(ft[1], fx[1], u[2]);
        u[1] = mfma_bf(ft[0], fx[1], u[1]);
        u[2] = mfma_bf(ft[0], fx[2], u[2]);
      };
      bf16x8 fkt[TS][2];
#pragma unroll
      for (int i = 0; i < TS; ++i)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int ti = TS * w + i, row = 32 * k + 8 * gq + (n >> 2), p = 4 * (ti >> 1) + (n & 3);
          const uint2 lo = read_tr(in.K + swz<DKP>(row, p) + 4 * (ti & 1));
          const uint2 hi = read_tr(in.K + swz<DKP>(row + 4, p) + 4 * (ti & 1));
          fkt[i][k] = as_frag(make_uint4(lo.x, lo.y, hi.x, hi.y));
        }
      solve(ft[0], u);
      if (w >= 2) {
#pragma unroll
        for (int t = 0; t < 3; ++t) fx[t] = frag(L.X, 3 + t);
        solve(ft[1], u + 3);
      }
      floatx4 U = ((u[2] + u[5]) + (u[1] + u[4])) + (u[0] + u[3]);
      if (__builtin_expect(tile_not_finite(U), 0)) lost = min(lost, cut_out_tile(&U, t4));
      if (gq == 0) L.lost[4 * n + w] = lost;
      if (PART != kTransfer) put_tile<2>(L.U, w, lane, U);
      U[0] *= c3.x; U[1] *= c3.y; U[2] *= c3.z; U[3] *= c3.w;
      put_tile<3>(L.U + 4 * 256, w, lane, U);
      exchange_barrier();
      // S = e^(b_C) S0 + K^T diag(e^(b_C - b)) U
      floatx4 z[TS] = {};
      bf16x8 f[2][3];
#pragma unroll
      for (int t = 2; t >= 0; --t)
#pragma unroll
        for (int k = 0; k < 2; ++k) f[k][t] = frag(L.U, 4 + 3 * k + t);
      const int4 all = *reinterpret_cast<const int4*>(L.lost + 4 * n);
#pragma unroll
      for (int i = 0; i < TS; ++i) S[i] *= eC;
#pragma unroll
      for (int t = 2; t >= 0; --t)
#pragma unroll
        for (int i = 0; i < TS; ++i) {
          z[i] = mfma_bf(fkt[i][1], f[1][t], z[i]);
          S[i] = mfma_bf(fkt[i][0], f[0][t], S[i]);
        }
#pragma unroll
      for (int i = 0; i < TS; ++i) S[i] += z[i];
      lost = min(min(all.x, all.y), min(all.z, all.w));
      if (__builtin_expect(__any(lost < kC), 0)) {
#pragma unroll
        for (int i = 0; i < TS; ++i)
          if (lost < kC) S[i] = floatx4{NAN, NAN, NAN, NAN};
      }
      put_state();
    };
    if constexpr (PART == kSegments) {
      for (int j = 1; j < seg; ++j) {  // S = M S + N
        m += next_map;
        bf16x8 fm[TS][NS][3];
        floatx4 c[TS][3];
#pragma unroll
        for (int i = 0; i < TS; ++i) {
#pragma unroll
          for (int k = 0; k < NS; ++k)
#pragma unroll
            for (int t = 0; t < 3; ++t) fm[i][k][t] = frag(m + DKP * pitch, ((TS * w + i) * NS + k) * 3 + t);
#pragma unroll
          for (int r = 0; r < 4; ++r) c[i][0][r] = m[tile_row(TS * w + i, 4 * gq + r) * pitch + col];
          c[i][1] = c[i][2] = floatx4{};
        }
        put_state();
        exchange_barrier();
#pragma unroll
        for (int k = 0; k < NS; ++k) {
          bf16x8 fs[3];
#pragma unroll
          for (int t = 0; t < 3; ++t) fs[t] = frag(L.S, 3 * k + t);
#pragma unroll
          for (int i = 0; i < TS; ++i) {
            c[i][2] = mfma_bf(fm[i][k][2], fs[0], c[i][2]);
            c[i][1] = mfma_bf(fm[i][k][1], fs[0], c[i][1]);
            c[i][0] = mfma_bf(fm[i][k][0], fs[0], c[i][0]);
            c[i][2] = mfma_bf(fm[i][k][1], fs[1], c[i][2]);
            c[i][1] = mfma_bf(fm[i][k][0], fs[1], c[i][1]);
            c[i][2] = mfma_bf(fm[i][k][0], fs[2], c[i][2]);
          }
        }
#pragma unroll
        for (int i = 0; i < TS; ++i) S[i] = (c[i][2] + c[i][1]) + c[i][0];
        exchange_barrier();
      }
    }
    if (blocks > 0) {
      put_state();
      float eC = rec[kFrags + 256];
      for (int c = 0; c < blocks; ++c) {
        if (c + 1 < blocks) rec += next_rec;
        exchange_barrier();  // the other waves' loads of this block have landed
        const float e = eC;
        eC = rec[kFrags + 256];
        step(L.in[c & 1], e);
      }
    }
    if constexpr (PART == kTransfer) {
      m += seg * static_cast<int64_t>(next_map);
      if (wcol < pitch) {
#pragma unroll
        for (int i = 0; i < TS; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r) m[tile_row(TS * w + i, 4 * gq + r) * pitch + col] = S[i][r];
      } else {  // column c of M: value c % 8 of the lanes of its eight columns and this row
        const int c = col - pitch;
        uint16_t* to = reinterpret_cast<uint16_t*>(m + DKP * pitch) +
                       ((TS * w * NS + (c >> 5)) * 192 + ((c & 31) >> 3) * 16 + 4 * gq) * 8 + (c & 7);
#pragma unroll
        for (int i = 0; i < TS; ++i)
#pragma unroll
          for (int r = 0; r < 4; r += 2) {
            uint32_t terms[3];
            cut<3>(S[i][r], S[i][r + 1], terms, 1);
#pragma unroll
            for (int t = 0; t < 3; ++t) {
              uint16_t* at = to + (i * NS * 192 + t * 64 + r) * 8;
              at[0] = static_cast<uint16_t>(terms[t]);
              at[8] = static_cast<uint16_t>(terms[t] >> 16);
            }
          }
      }
      return;
    }
    if (!a.state_out || !in || !last) return;
#pragma unroll
    for (int i = 0; i < TS; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int d = tile_row(TS * w + i, 4 * gq + r);
        if (d < a.dk) a.state_out[at + static_cast<int64_t>(d) * a.dv] = S[i][r];
      }
    return;
  }
  const int os = a.hv * a.dv;
  const uint16_t* pk = a.k + static_cast<int64_t>(kh) * a.dk + t0 * a.ks;
  const uint16_t* pq = a.q + static_cast<int64_t>(kh) * a.dk + t0 * a.qs;
  const uint16_t* pv = a.v + static_cast<int64_t>(h) * a.dv + t0 * a.vs;
  int left = static_cast<int>(t1 - t0), done = 0;
  uint16_t* po = a.o + (t0 * a.hv + h) * a.dv - static_cast<int64_t>(kC) * os;
  int ak[NK], aq[NK];
#pragma unroll
  for (int i = 0; i < NK; ++i) {
    const int row = (i * 256 + tid) / PR, p = (swz<DKP>(row, tid % PR) >> 3) % PR;
    ak[i] = piece_at(row, a.ks, 8 * p, a.dk);
    aq[i] = piece_at(row, a.qs, 8 * p, a.dk);
  }
  const int av = piece_at((tid & 127) >> 1, a.vs, wcol + 8 * (tid & 1), a.dv);
  const auto fetch = [&](uint16_t* nK, uint16_t* nQ, uint16_t* nV, uint16_t* nT, uint16_t* nP,
                         float* nC) __attribute__((always_inline)) {
    const Rows K = rows_at(pk, a.ks, left, a.dk), Q = rows_at(pq, a.qs, left, a.dk);
    const Rows R = __builtin_amdgcn_make_buffer_rsrc(const_cast<float*>(rec), 0, 4 * kRec, 0x00027000);
#pragma unroll
    for (int i = 0; i < NK; ++i) to_lds(K, ak[i], nK + (i * 4 + w) * 512);
    if (w < 2) to_lds(rows_at(pv, a.vs, left, a.dv), av, nV + w * 512);
    if (w == 3) to_lds(R, 4 * kFrags + 16 * lane, nC);
#pragma unroll
    for (int i = 0; i < 5; ++i)
      if (i < 4 || w < 2) to_lds(R, (4 * i + w) * 1024 + 16 * lane, nT + (4 * i + w) * 512);
    if (PART != kTransfer) {
#pragma unroll
      for (int i = 0; i < NK; ++i) to_lds(Q, aq[i], nQ + (i * 4 + w) * 512);
#pragma unroll
      for (int i = 0; i < 3; ++i) to_lds(R, 4 * kFragsT + (4 * i + w) * 1024 + 16 * lane, nP + (4 * i + w) * 512);
    }
    if (left > kC) rec += next_rec;
    pk += kC * a.ks;
    pq += kC * a.qs;
    pv += kC * a.vs;
    left -= kC;
  };
  typedef Ahead<DKP, 1, 4> Next;  // the block after the next
  uint32_t ready[2];  // the outputs of the block before
  const int o_at = in ? 2 * (t4 * os + col) : kOutside;
  const auto store_o = [&]() __attribute__((always_inline)) {
    const Rows to = rows_at(po, os, done, a.dv);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      __builtin_amdgcn_raw_buffer_store_b16(static_cast<uint16_t>(ready[i]), to, o_at + 4 * os * i, 0, 0);
      __builtin_amdgcn_raw_buffer_store_b16(static_cast<uint16_t>(ready[i] >> 16), to, o_at + 4 * os * i + 2 * os, 0, 0);
    }
  };
  // One block, from the s buffers, with the next on its way into the n buffers.
  // The buffers are restrict arguments so that no read of one waits for the
  // loads into the other.
  const auto step = [&](bool first, const uint16_t* __restrict__ sQ, const uint16_t* __restrict__ sP,
                        const float* __restrict__ sC, uint16_t* __restrict__ nK, uint16_t* __restrict__ nQ,
                        uint16_t* __restrict__ nV, uint16_t* __restrict__ nT, uint16_t* __restrict__ nP,
                        float* __restrict__ nC, const uint32_t* __restrict__ xS, const uint32_t* __restrict__ xU,
                        const int* __restrict__ xLost, uint32_t* __restrict__ unused) __attribute__((always_inline)) {
    if (PART != kTransfer && !first) store_o();
    done = left + kC;
    po += static_cast<int64_t>(kC) * os;
    fetch(nK, nQ, nV, nT, nP, nC);  // after the last block zeros and that block's T again: no branch around it
    __asm__ volatile("" ::: "memory");
    Next::touch(w, rec, pk, pq, pv + wcol, static_cast<int>(a.ks), static_cast<int>(a.qs), static_cast<int>(a.vs), left,
                a.dk, a.dv - wcol, unused);
    exchange_barrier();  // leaves the reads of S0 before it to the waves that are waited for
    if constexpr (PART == kTransfer) {
      exchange_barrier();
      return;
    }
    floatx4 o[2] = {};
#pragma unroll
    for (int k = 0; k < NS; ++k) {
      const bf16x8 fq = as_frag(*reinterpret_cast<const uint4*>(sQ + swz<DKP>(tile_row(w, n), 4 * k + gq)));
#pragma unroll
      for (int t = 1; t >= 0; --t) o[t] = mfma_bf(fq, frag(xS, 3 * k + t), o[t]);
    }
    const float4 c2 = *reinterpret_cast<const float4*>(sC + 64 + t4);
    floatx4 O = o[1] + o[0];
    O[0] *= c2.x; O[1] *= c2.y; O[2] *= c2.z; O[3] *= c2.w;
    bf16x8 fp[2][2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      fp[0][t] = frag(sP, 2 * w + t);
      if (w >= 2) fp[1][t] = frag(sP, 2 * (w + 2) + t);
    }
    exchange_barrier();
    // O = diag(e^b) Q S0 + P U (the scale is in both)
    floatx4 z[3] = {};
    bf16x8 f[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) f[t] = frag(xU, t);
    const int4 all = *reinterpret_cast<const int4*>(xLost + 4 * n);
    z[0] = mfma_bf(fp[0][1], f[0], z[0]);
    O = mfma_bf(fp[0][0], f[0], O);
    z[0] = mfma_bf(fp[0][0], f[1], z[0]);
    if (w >= 2) {
#pragma unroll
      for (int t = 0; t < 2; ++t) f[t] = frag(xU, 2 + t);
      z[1] = mfma_bf(fp[1][1], f[0], z[1]);
      z[2] = mfma_bf(fp[1][0], f[0], z[2]);
      z[1] = mfma_bf(fp[1][0], f[1], z[1]);
    }
    O = ((z[0] + z[1]) + z[2]) + O;
    const int lost = min(min(all.x, all.y), min(all.z, all.w));
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (t4 + r >= lost) O[r] = NAN;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const bf16x2 b = __builtin_convertvector((floatx2{O[2 * i], O[2 * i + 1]}), bf16x2);
      __builtin_memcpy(&ready[i], &b, 4);
    }
  };
  if (blocks > 0) {
    fetch(L.in[0].K, L.in[0].Q, L.in[0].V, L.in[0].T, L.in[0].P, L.in[0].C);
    for (int j = 2; PART == kSegments && j < 2 * seg; ++j) exchange_barrier();  // beside M S + N
    for (int c = 0; c < blocks; ++c) {
      const auto& now = L.in[c & 1];
      auto& then = L.in[(c & 1) ^ 1];
      if (c == 0)
        landed_barrier<0>();
      else
        landed_barrier<Next::kLoads>();
      step(c == 0, now.Q, now.P, now.C, then.K, then.Q, then.V, then.T, then.P, then.C, L.S, L.U, L.lost, L.unused);
    }
    if (PART != kTransfer) store_o();
    __builtin_amdgcn_s_waitcnt(0x0F70);  // nothing is on its way into LDS when the workgroup ends
  }
}

int64_t ws_blocks(int64_t nseq, int64_t total) { return total / kC + nseq; }

// Prompts of at most kFew tokens on average go token by token, 1.7 us a token after the first (4 heads of
// 128 x 128, 1 and 64 streams: 4 tokens 11.9 and 14.4 us against 17.4 and 25.8 in a block; 8 tokens 18.7 and 21.3).
// The mean decides, as lengths lie on the device: one long sequence among many of a few tokens goes token by token
// too, and plan_of counts short sequences as it counts long ones.
constexpr int64_t kFew = 6;
constexpr int64_t kCus = 256;

// How a call's blocks are scanned: 4-byte words of the blocks' records, to the end
// of the segments' maps and of the whole workspace, and the segments' length in
// blocks with the most segments that a sequence can have (0: each whole).
struct Plan {
  int64_t records, maps, words;
  int len, most;
};
// Segments where at least three of them find their workgroups a CU each, of [N | M] as of the scan.  A block more
// in each costs 3 us, a segment more 2 to 3: lengths of 1.2 times the root of the blocks, at least 6.  (us with
// delta_prep, whole and in 3, 5, 8, 12 segments: 1 head of 128 x 128, 8192 tokens 210, 142, 99, 82, 76; 4 heads,
// which have CUs for 5, 212, 148, 106, 110, 138; 2048 tokens 63, 54, 47, 57, 78; 1024 tokens 37 either way; 16 heads,
// which have them for 2, 231, 287, 314, 341, 416.)
constexpr int64_t kMinLen = 6, kMinSegments = 3;
Plan plan_of(int64_t nseq, int64_t total, int64_t hv, int64_t dk, int64_t dv) {
  Plan p{ws_blocks(nseq, total) * hv * kRec, 0, 0, 0, 0};
  p.words = p.records;
  const int64_t dkp = dk <= 64 ? 64 : 128, groups = nseq * hv * ceil_div(dv, 16), units = nseq * hv * dkp / 16;
  const int64_t blocks = ceil_div(total, kC), mean = ceil_div(blocks, nseq);
  const int64_t at_once = std::min(kCus / groups, (kCus + groups + 2 * units) / (groups + units));
  if (at_once < kMinSegments) return p;
  const int64_t root = static_cast<int64_t>(std::ceil(1.2 * std::sqrt(static_cast<double>(mean))));
  const int64_t len = std::max({kMinLen, root, ceil_div(mean, at_once)});
  if (mean <= (kMinSegments - 1) * len) return p;
  p.len = static_cast<int>(len);
  p.most = static_cast<int>(ceil_div(blocks, len));
  p.maps = p.records + (p.most + nseq) * hv * map_words(static_cast<int>(dkp), static_cast<int>(ceil_div(dv, 16) * 16));
  p.words = p.maps + nseq * hv * dkp * ceil_div(dv, 16) * 16;
  return p;
}

template <int DKP>
void blocked_launch(const DeltaArgs& a, float* ws, hipStream_t st) {
  const int64_t heads = int64_t(a.nseq) * a.hv;
  const dim3 blocks(static_cast<unsigned>(ws_blocks(a.nseq, a.total)), static_cast<unsigned>(a.hv));
  hipLaunchKernelGGL(delta_prep<DKP>, blocks, dim3(256), 0, st, a, ws);
  // Workgroups of all column parts, in eights.  One launch has fewer than 2^32 threads along x: past 2^22
  // workgroups, which only delta_scan can have, they go on along y.
  const auto grid = [](int64_t units, int64_t cols) {
    const int64_t all = ceil_div(units, 8) * 8 * cols, x = std::min(all, int64_t(1) << 22);
    return dim3(static_cast<unsigned>(x), static_cast<unsigned>(ceil_div(all, x)));
  };
  const int by16 = static_cast<int>(ceil_div(a.dv, 16)), by32 = (by16 + 1) / 2, by64 = (by16 + 3) / 4;
  const Plan plan = plan_of(a.nseq, a.total, a.hv, a.dk, a.dv);
  // The narrowest workgroups that still find a CU each: a block takes a workgroup 1.6 us with 16 columns, 2.3 with
  // 32, 2.7 with 64 (4 heads of 128 x 128), but the CU the same for any (us with delta_prep at 16, 32, 64 columns:
  // 4 heads of 128 x 128, 8192 tokens 215, 311, 360; 32, 64, 128 of them, 2048 tokens 79, 100, 111; 150, 117, 127;
  // 306, 238, 179; 128 heads of 64 x 64, 16 ragged prompts 437, 365, 397).
  if (plan.len) {
    const Segments sg{ws + plan.records, ws + plan.maps, plan.len};
    const int both = by16 + DKP / 16;
    hipLaunchKernelGGL((delta_scan_quarters<DKP, kTransfer>), grid(heads * (plan.most - 1), both), dim3(512), 0, st, a, ws,
                       both, sg);
    hipLaunchKernelGGL((delta_scan_quarters<DKP, kSegments>), grid(heads * plan.most, by16), dim3(512), 0, st, a, ws, by16,
                       sg);
  } else if (heads * by16 <= kCus) {
    hipLaunchKernelGGL((delta_scan_quarters<DKP, kWhole>), grid(heads, by16), dim3(512), 0, st, a, ws, by16, Segments{});
  } else if (heads * by32 <= kCus) {
    hipLaunchKernelGGL((delta_scan<DKP, 2>), grid(heads, by32), dim3(256), 0, st, a, ws, by32);
  } else {
    hipLaunchKernelGGL((delta_scan<DKP, 4>), grid(heads, by64), dim3(512), 0, st, a, ws, by64);
  }
}

// sizes, strides and alignment shared by the prompt and the step
int delta_check(const DeltaArgs& a, int dtype, int64_t nseq, int64_t hk, int64_t hv, int64_t dk, int64_t dv) {
  if (nseq < 1 || a.total < 0 || hk < 1 || hv < hk || hv % hk != 0 || dk < 1 || dv < 1 || a.qs < hk * dk ||
      a.ks < hk * dk || a.vs < hv * dv || !(a.scale == a.scale))
    return BLLM_E_INVAL;
  if (a.total > 0 && (!a.q || !a.k || !a.v || !a.g || !a.beta || !a.o)) return BLLM_E_INVAL;
  if (dtype != BLLM_BF16 || dk % 8 != 0 || dk > 128 || dv % 8 != 0 || dv > 1024 || hv > 1024 || nseq > 65535 ||
      a.total >= (int64_t(1) << 31) || a.qs >= kMaxStride || a.ks >= kMaxStride || a.vs >= kMaxStride ||
      a.qs % 8 != 0 || a.ks % 8 != 0 || a.vs % 8 != 0 || !aligned16(a.q) || !aligned16(a.k) || !aligned16(a.v) || !aligned16(a.o) || !aligned16(a.state_in) || !aligned16(a.state_out))
    return BLLM_E_NOTSUP;
  return BLLM_OK;
}

}  // namespace
}  // namespace bllm

using namespace bllm;

extern "C" size_t bllm_gated_delta_workspace(int64_t nseq, int64_t total, int64_t hv, int64_t dk, int64_t dv) {
  if (nseq < 1 || total < 0 || hv < 1 || dk < 1 || dv < 1) return 0;
  return static_cast<size_t>(plan_of(nseq, total, hv, dk, dv).words) * 4;
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
  hipStream_t st = static_cast<hipStream_t>(stream);
  float* w = static_cast<float*>(ws);
  if (total <= kFew * nseq)
    recurrent_launch(a, st);
  else
    dk <= 64 ? blocked_launch<64>(a, w, st) : blocked_launch<128>(a, w, st);
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
