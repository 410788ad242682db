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
// blocks at once; delta_scan walks the blocks of a sequence with the state in
// registers.  A wave there owns 16 columns and every row, so the waves of a
// workgroup share K, Q, T and P through LDS and never exchange results: a
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
// Recurrent form, for steps and prompts of a few tokens.  A wave owns 32 columns of one head's state: lane (i, c),
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

// ---------------------------------------------------------------- blocked form

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short shortx4 __attribute__((ext_vector_type(4)));
typedef float floatx4 __attribute__((ext_vector_type(4)));

constexpr int kC = 64;            // tokens of a block
constexpr int kTFloats = 6 * 512; // T: 6 fragments of 64 lanes x 8 floats (16 x 32 entries on or below the diagonal)
constexpr int kPWords = 6 * 512;  // P: the same fragments in two bf16 terms
constexpr int kRec = kTFloats + kPWords + 256;  // one block and head in the workspace, in 4-byte words
constexpr int kLd = 68;           // pitch of a 64 x 64 fp32 tile in LDS
constexpr float kForget = -1e4f;  // smaller gates decay by e^-10000 = 0 as well, and their sums stay finite

// fragment f of T and P: row tile kFragRow[f] (0 .. 3), inner index 32 kFragK[f] .. + 31
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

struct Block {
  int64_t first, left;  // its first token; tokens from there to the sequence's end
};

// sequence s of the batch, cut at its rows
__device__ inline void seq_span(const DeltaArgs& a, int s, int64_t* t0, int64_t* t1) {
  *t0 = min(max(a.offsets[s], int64_t(0)), a.total);
  *t1 = min(max(a.offsets[s + 1], *t0), a.total);
}

// Block j of the workspace: sequence s has blocks offsets[s] / 64 + s and on,
// which leaves room for every sequence's last, partial block.
__device__ inline bool find_block(const DeltaArgs& a, int64_t j, Block* b) {
  int lo = 0, hi = a.nseq;
  int64_t t0, t1;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    seq_span(a, mid, &t0, &t1);
    if (t0 / kC + mid <= j) lo = mid; else hi = mid;
  }
  seq_span(a, lo, &t0, &t1);
  b->first = t0 + (j - (t0 / kC + lo)) * kC;
  b->left = t1 - b->first;
  return b->first >= t0 && b->left > 0;
}

// one 16-byte piece of a token's key or query, zero outside the rows or the width
__device__ inline uint4 piece(const uint16_t* base, int64_t stride, const Block& b, int row, int col, int width) {
  if (row < b.left && col < width) return *reinterpret_cast<const uint4*>(base + (b.first + row) * stride + col);
  return make_uint4(0, 0, 0, 0);
}

// T, P and the decays of one block and head.  Wave w has rows 16 w .. 16 w + 15
// of K K^T and Q K^T.  (I + A)^-1: the 16 x 16 blocks on the diagonal by
// substitution (a lane a column), then two doublings,
//   [T1 0; -T2 A21 T1 T2],
// on fp32 MFMA, whose accumulators feed the second product as they are.
template <int DKP>
__global__ __launch_bounds__(256) void delta_prep(DeltaArgs a, float* ws) {
  constexpr int NS = DKP / 32;
  __shared__ float sA[kC * kLd], sT[kC * kLd];
  __shared__ double sB[kC];
  __shared__ float sBeta[kC], sRk[kC], sRq[kC];
  __shared__ int sBad;
  Block blk;
  if (!find_block(a, blockIdx.x, &blk)) return;
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), n = lane & 15, gq = lane >> 4;
  const int h = blockIdx.y, kh = h / (a.hv / a.hk);
  const uint16_t* K = a.k + static_cast<int64_t>(kh) * a.dk;
  const uint16_t* Q = a.q + static_cast<int64_t>(kh) * a.dk;
  if (threadIdx.x == 0) sBad = kC;
  if (w == 0) {
    double b = 0.0;
    float be = 0.0f;
    if (lane < blk.left) {
      const float g = a.g[(blk.first + lane) * a.hv + h];
      b = g < kForget ? kForget : g;  // a NaN stays
      be = a.beta[(blk.first + lane) * a.hv + h];
    }
    for (int off = 1; off < kC; off <<= 1) {
      const double up = __shfl_up(b, off, kWave);
      if (lane >= off) b += up;
    }
    sB[lane] = b;
    sBeta[lane] = be;
  }
  floatx4 G[4] = {}, P[4] = {}, qq = {};
  {
    bf16x8 fk[NS], fq[NS];
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      fk[s] = as_frag(piece(K, a.ks, blk, 16 * w + n, 32 * s + 8 * gq, a.dk));
      fq[s] = as_frag(piece(Q, a.qs, blk, 16 * w + n, 32 * s + 8 * gq, a.dk));
    }
#pragma unroll
    for (int s = 0; s < NS; ++s) qq = mfma_bf(fq[s], fq[s], qq);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      if (c > w) break;
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        const bf16x8 fb = as_frag(piece(K, a.ks, blk, 16 * c + n, 32 * s + 8 * gq, a.dk));
        G[c] = mfma_bf(fk[s], fb, G[c]);
        P[c] = mfma_bf(fq[s], fb, P[c]);
      }
    }
  }
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    if (c != w) continue;
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (n == 4 * gq + r) {
        sRk[16 * w + n] = a.unit ? 1.0f / sqrtf(G[c][r] + kL2Eps) : 1.0f;
        sRq[16 * w + n] = a.unit ? 1.0f / sqrtf(qq[r] + kL2Eps) : 1.0f;
      }
  }
  __syncthreads();
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    if (c > w) break;
    const int i = 16 * c + n;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int t = 16 * w + 4 * gq + r;
      float av = 0.0f, pv = 0.0f;
      if (i <= t) {
        const float f = expf(static_cast<float>(sB[t] - sB[i])) * sRk[i];
        pv = a.scale * sRq[t] * f * P[c][r];
        if (i < t) av = sBeta[t] * sRk[t] * f * G[c][r];
        if (!(fabsf(av) < INFINITY)) {
          atomicMin(&sBad, t);
          av = 0.0f;
        }
      }
      P[c][r] = pv;
      sA[t * kLd + i] = av;
    }
  }
  // a token's own gates reach T through its column and the decays: not finite there counts as well
  if (threadIdx.x < kC && !(fabsf(sBeta[threadIdx.x] * sRk[threadIdx.x]) < INFINITY && fabs(sB[threadIdx.x]) < INFINITY))
    atomicMin(&sBad, static_cast<int>(threadIdx.x));
  __syncthreads();
  {  // diagonal blocks: column n of the inverse of rows 16 w ..
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float v = i == n ? 1.0f : 0.0f;
#pragma unroll
      for (int m = 0; m < i; ++m) v -= sA[(16 * w + i) * kLd + 16 * w + m] * x[m];
      x[i] = v;
    }
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if ((i >> 2) == gq) sT[(16 * w + i) * kLd + 16 * w + n] = x[i];
  }
  __syncthreads();
  if (w < 2) {  // 32 x 32 blocks: below the diagonal of pair w
    const int lo = 32 * w, up = 32 * w + 16;
    floatx4 m = {}, o = {};
#pragma unroll
    for (int r = 0; r < 4; ++r)
      m = __builtin_amdgcn_mfma_f32_16x16x4f32(sA[(up + n) * kLd + lo + 4 * gq + r],
                                               sT[(lo + 4 * gq + r) * kLd + lo + n], m, 0, 0, 0);
#pragma unroll
    for (int r = 0; r < 4; ++r)
      o = __builtin_amdgcn_mfma_f32_16x16x4f32(sT[(up + n) * kLd + up + 4 * gq + r], m[r], o, 0, 0, 0);
#pragma unroll
    for (int r = 0; r < 4; ++r) sT[(up + 4 * gq + r) * kLd + lo + n] = -o[r];
  } else {  // and zeros above it
#pragma unroll
    for (int r = 0; r < 4; ++r) sT[(32 * (w - 2) + 4 * gq + r) * kLd + 32 * (w - 2) + 16 + n] = 0.0f;
  }
  __syncthreads();
  {  // the lower left 32 x 32 block: wave w has rows 16 (w / 2) and columns 16 (w % 2) of it
    const int c = 16 * (w & 1), p = 32 + 16 * (w >> 1);
    floatx4 m[2] = {}, o = {};
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        const int k = 16 * (r >> 2) + 4 * gq + (r & 3);
        m[j] = __builtin_amdgcn_mfma_f32_16x16x4f32(sA[(32 + 16 * j + n) * kLd + k], sT[k * kLd + c + n], m[j], 0, 0, 0);
      }
#pragma unroll
    for (int r = 0; r < 8; ++r)
      o = __builtin_amdgcn_mfma_f32_16x16x4f32(sT[(p + n) * kLd + 32 + 16 * (r >> 2) + 4 * gq + (r & 3)],
                                               m[r >> 2][r & 3], o, 0, 0, 0);
#pragma unroll
    for (int r = 0; r < 4; ++r) sT[(p + 4 * gq + r) * kLd + c + n] = -o[r];
  }
  __syncthreads();
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    if (c > w) break;
#pragma unroll
    for (int r = 0; r < 4; ++r) sA[(16 * w + 4 * gq + r) * kLd + 16 * c + n] = P[c][r];
  }
  float* rec = ws + (static_cast<int64_t>(blockIdx.x) * a.hv + h) * kRec;
  const int bad = sBad;
  for (int f = w; f < 6; f += 4) {
    const int t = tile_row(frag_row(f), n), k0 = 32 * frag_k(f) + 8 * gq;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      float v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int k = k0 + 4 * half + j;
        v[j] = k <= t ? (t < bad ? sT[t * kLd + k] * sBeta[k] : NAN) : 0.0f;
      }
      reinterpret_cast<float4*>(rec)[(2 * f + half) * 64 + lane] = make_float4(v[0], v[1], v[2], v[3]);
    }
  }
  __syncthreads();
  for (int f = w; f < 6; f += 4) {
    const int t = tile_row(frag_row(f), n), k0 = 32 * frag_k(f) + 8 * gq;
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = k0 + j <= t ? sA[t * kLd + k0 + j] : 0.0f;
    uint32_t p[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) cut<2>(v[2 * j], v[2 * j + 1], p + j, 4);
    uint4* to = reinterpret_cast<uint4*>(rec + kTFloats) + 128 * f + lane;
    to[0] = make_uint4(p[0], p[1], p[2], p[3]);
    to[64] = make_uint4(p[4], p[5], p[6], p[7]);
  }
  if (w == 0) {
    float* c = rec + kTFloats + kPWords;
    const float e = expf(static_cast<float>(sB[lane]));
    c[lane] = e * sRk[lane];
    c[64 + lane] = e * sRq[lane] * a.scale;
    c[128 + lane] = expf(static_cast<float>(sB[kC - 1] - sB[lane])) * sRk[lane];
    if (lane == 0) c[192] = expf(static_cast<float>(sB[kC - 1]));
  }
}

// first row of a lane's column that is not finite, over the lanes of the column; such entries become zero
__device__ inline int cut_out(floatx4* x, int gq) {
  int at = kC;
#pragma unroll
  for (int i = 3; i >= 0; --i)
#pragma unroll
    for (int r = 3; r >= 0; --r)
      if (!(fabsf(x[i][r]) < INFINITY)) {
        at = min(at, tile_row(i, 4 * gq + r));
        x[i][r] = 0.0f;
      }
  at = min(at, __shfl_xor(at, 16, kWave));
  return min(at, __shfl_xor(at, 32, kWave));
}
__device__ inline bool any_not_finite(const floatx4* x) {
  float z = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int r = 0; r < 4; ++r) z = fmaf(x[i][r], 0.0f, z);
  return __any(z != 0.0f);  // 0 x infinity and 0 x NaN are NaN
}

// LDS image of a block's keys or queries: rows of DKP values in 16-byte pieces,
// the pieces of a row exchanged so that the sixteen rows of a tile start in
// different banks
template <int DKP>
__device__ inline int swz(int row, int pc) {
  if (DKP == 128) return row * 128 + ((pc ^ ((row & 3) | ((row >> 1) & 12))) << 3);
  return row * 64 + ((pc ^ (((row >> 1) & 1) | ((row >> 2) & 6))) << 3);
}

__device__ inline uint2 read_tr(const uint16_t* p) {
  typedef __attribute__((address_space(3))) shortx4 lds_s4;
  const shortx4 v = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4*)p);
  uint2 r;
  __builtin_memcpy(&r, &v, 8);
  return r;
}

template <int DKP>
__global__ __launch_bounds__(256, DKP == 64 ? 2 : 1) void delta_scan(DeltaArgs a, const float* ws) {
  constexpr int NS = DKP / 32;    // inner steps over dk
  constexpr int NP = DKP / 32;    // pieces of K (and of Q) a thread stages
  constexpr int kLv = 64 + 8;     // pitch of the staged V
  __shared__ __align__(16) uint16_t sK[kC * DKP], sQ[kC * DKP], sV[kC * kLv], sT[6 * 3 * 512], sP[6 * 2 * 512];
  __shared__ __align__(16) float sC[256];
  const int tid = threadIdx.x, lane = tid & 63, n = lane & 15, gq = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int h = blockIdx.y, s = blockIdx.z, kh = h / (a.hv / a.hk);
  const int wcol = blockIdx.x * 64, col = wcol + 16 * w + n;
  const bool in = col < a.dv;
  int64_t t0, t1;
  seq_span(a, s, &t0, &t1);
  const int64_t at = (static_cast<int64_t>(s) * a.hv + h) * a.dk * static_cast<int64_t>(a.dv) + col;
  floatx4 S[2 * NS];
#pragma unroll
  for (int i = 0; i < 2 * NS; ++i)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int d = tile_row(i, 4 * gq + r);
      S[i][r] = a.state_in && in && d < a.dk ? a.state_in[at + static_cast<int64_t>(d) * a.dv] : 0.0f;
    }
  const uint16_t* K = a.k + static_cast<int64_t>(kh) * a.dk;
  const uint16_t* Q = a.q + static_cast<int64_t>(kh) * a.dk;
  const uint16_t* V = a.v + static_cast<int64_t>(h) * a.dv;
  const int64_t rec0 = t0 / kC + s;
  Block blk{t0, t1 - t0};
  uint4 pk[NP], pq[NP], pv[2], pt[3], pp[3];
  float pc = 0.0f;
  auto fetch = [&](int64_t c) {
    const float* rec = ws + ((rec0 + c) * a.hv + h) * kRec;
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      pt[i] = reinterpret_cast<const uint4*>(rec)[i * 256 + tid];
      pp[i] = reinterpret_cast<const uint4*>(rec + kTFloats)[i * 256 + tid];
    }
    if (tid < 193) pc = rec[kTFloats + kPWords + tid];
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const int e = i * 256 + tid, row = e / (DKP / 8), p = e % (DKP / 8);
      pk[i] = piece(K, a.ks, blk, row, 8 * p, a.dk);
      pq[i] = piece(Q, a.qs, blk, row, 8 * p, a.dk);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int e = i * 256 + tid;
      pv[i] = piece(V, a.vs, blk, e >> 3, wcol + 8 * (e & 7), a.dv);
    }
  };
  const int64_t blocks = (t1 - t0 + kC - 1) / kC;
  if (blocks > 0) fetch(0);
  for (int64_t c = 0; c < blocks; ++c) {
    if (c) lds_barrier();
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const int e = i * 256 + tid, row = e / (DKP / 8), p = e % (DKP / 8);
      *reinterpret_cast<uint4*>(sK + swz<DKP>(row, p)) = pk[i];
      *reinterpret_cast<uint4*>(sQ + swz<DKP>(row, p)) = pq[i];
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int e = i * 256 + tid;
      *reinterpret_cast<uint4*>(sV + (e >> 3) * kLv + 8 * (e & 7)) = pv[i];
    }
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      const int e = i * 256 + tid, f = e >> 7, half = (e >> 6) & 1;
      uint32_t t[6];
      cut<3>(__uint_as_float(pt[i].x), __uint_as_float(pt[i].y), t, 2);
      cut<3>(__uint_as_float(pt[i].z), __uint_as_float(pt[i].w), t + 1, 2);
#pragma unroll
      for (int j = 0; j < 3; ++j)
        *reinterpret_cast<uint2*>(sT + ((f * 3 + j) * 64 + lane) * 8 + 4 * half) = make_uint2(t[2 * j], t[2 * j + 1]);
      *reinterpret_cast<uint4*>(sP + e * 8) = pp[i];
    }
    sC[tid] = pc;
    lds_barrier();
    const Block now = blk;
    blk.first += kC;
    blk.left -= kC;
    if (c + 1 < blocks) fetch(c + 1);

    // K S0 and Q S0
    floatx4 X[4] = {}, O[4] = {}, U[4] = {};
#pragma unroll
    for (int k = 0; k < NS; ++k) {
      bf16x8 f[3];
      cut_pair<3>(S[2 * k], S[2 * k + 1], f);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int e = swz<DKP>(tile_row(i, n), 4 * k + gq);
        const bf16x8 fk = as_frag(*reinterpret_cast<const uint4*>(sK + e));
        const bf16x8 fq = as_frag(*reinterpret_cast<const uint4*>(sQ + e));
        X[i] = mfma_bf(fk, f[2], X[i]);
        O[i] = mfma_bf(fq, f[1], O[i]);
        X[i] = mfma_bf(fk, f[1], X[i]);
        O[i] = mfma_bf(fq, f[0], O[i]);
        X[i] = mfma_bf(fk, f[0], X[i]);
      }
    }
    // X = V - diag(e^b) K S0
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = tile_row(i, 4 * gq);
      const uint2 v = read_tr(sV + (t + (n >> 2)) * kLv + 16 * w + 4 * (n & 3));
      const float4 c1 = *reinterpret_cast<const float4*>(sC + t);
      X[i][0] = __uint_as_float(v.x << 16) - c1.x * X[i][0];
      X[i][1] = __uint_as_float(v.x & 0xFFFF0000u) - c1.y * X[i][1];
      X[i][2] = __uint_as_float(v.y << 16) - c1.z * X[i][2];
      X[i][3] = __uint_as_float(v.y & 0xFFFF0000u) - c1.w * X[i][3];
    }
    int lost = kC;  // first token of this column whose u is not finite
    if (any_not_finite(X)) lost = cut_out(X, gq);
    // U = T X
    {
      bf16x8 f[2][3];
      cut_pair<3>(X[0], X[1], f[0]);
      cut_pair<3>(X[2], X[3], f[1]);
#pragma unroll
      for (int b = 0; b < 6; ++b) {
        const int i = frag_row(b), k = frag_k(b);
        bf16x8 t[3];
#pragma unroll
        for (int j = 0; j < 3; ++j) t[j] = as_frag(*reinterpret_cast<const uint4*>(sT + ((b * 3 + j) * 64 + lane) * 8));
        U[i] = mfma_bf(t[2], f[k][0], U[i]);
        U[i] = mfma_bf(t[1], f[k][1], U[i]);
        U[i] = mfma_bf(t[0], f[k][2], U[i]);
        U[i] = mfma_bf(t[1], f[k][0], U[i]);
        U[i] = mfma_bf(t[0], f[k][1], U[i]);
        U[i] = mfma_bf(t[0], f[k][0], U[i]);
      }
    }
    if (any_not_finite(U)) lost = min(lost, cut_out(U, gq));
    // O = diag(e^b) Q S0 + P U (the scale is in both), S = e^(b_C) S0 + K^T diag(e^(b_C - b)) U
    {
      bf16x8 f[2][2];
      cut_pair<2>(U[0], U[1], f[0]);
      cut_pair<2>(U[2], U[3], f[1]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 c2 = *reinterpret_cast<const float4*>(sC + 64 + tile_row(i, 4 * gq));
        O[i][0] *= c2.x; O[i][1] *= c2.y; O[i][2] *= c2.z; O[i][3] *= c2.w;
      }
#pragma unroll
      for (int b = 0; b < 6; ++b) {
        const bf16x8 p = as_frag(*reinterpret_cast<const uint4*>(sP + (b * 128 + lane) * 8));
        const bf16x8 p1 = as_frag(*reinterpret_cast<const uint4*>(sP + (b * 128 + 64 + lane) * 8));
        O[frag_row(b)] = mfma_bf(p1, f[frag_k(b)][0], O[frag_row(b)]);
        O[frag_row(b)] = mfma_bf(p, f[frag_k(b)][1], O[frag_row(b)]);
        O[frag_row(b)] = mfma_bf(p, f[frag_k(b)][0], O[frag_row(b)]);
      }
    }
    const bool poisoned = __any(lost < kC);
    if (poisoned) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (tile_row(i, 4 * gq + r) >= lost) O[i][r] = NAN;
    }
    if (in) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int t = tile_row(i, 4 * gq + r);
          if (t < now.left) a.o[((now.first + t) * a.hv + h) * a.dv + col] = f32_to_bf16(O[i][r]);
        }
    }
    const float eC = sC[192];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 c3 = *reinterpret_cast<const float4*>(sC + 128 + tile_row(i, 4 * gq));
      U[i][0] *= c3.x; U[i][1] *= c3.y; U[i][2] *= c3.z; U[i][3] *= c3.w;
    }
    bf16x8 f[2][3];
    cut_pair<3>(U[0], U[1], f[0]);
    cut_pair<3>(U[2], U[3], f[1]);
#pragma unroll
    for (int i = 0; i < 2 * NS; ++i) {
      S[i] *= eC;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int row = 32 * k + 8 * gq + (n >> 2), p = 4 * (i >> 1) + (n & 3);
        const uint2 lo = read_tr(sK + swz<DKP>(row, p) + 4 * (i & 1));
        const uint2 hi = read_tr(sK + swz<DKP>(row + 4, p) + 4 * (i & 1));
        const bf16x8 fk = as_frag(make_uint4(lo.x, lo.y, hi.x, hi.y));
        S[i] = mfma_bf(fk, f[k][2], S[i]);
        S[i] = mfma_bf(fk, f[k][1], S[i]);
        S[i] = mfma_bf(fk, f[k][0], S[i]);
      }
      if (poisoned && lost < kC) S[i] = floatx4{NAN, NAN, NAN, NAN};
    }
  }
  if (!a.state_out || !in) return;
#pragma unroll
  for (int i = 0; i < 2 * NS; ++i)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int d = tile_row(i, 4 * gq + r);
      if (d < a.dk) a.state_out[at + static_cast<int64_t>(d) * a.dv] = S[i][r];
    }
}

int64_t ws_blocks(int64_t nseq, int64_t total) { return total / kC + nseq; }

// Prompts of at most kFew tokens on average go token by token.
constexpr int64_t kFew = 2;

template <int DKP>
void blocked_launch(const DeltaArgs& a, float* ws, hipStream_t st) {
  const dim3 blocks(static_cast<unsigned>(ws_blocks(a.nseq, a.total)), static_cast<unsigned>(a.hv));
  hipLaunchKernelGGL(delta_prep<DKP>, blocks, dim3(256), 0, st, a, ws);
  const dim3 grid(static_cast<unsigned>(ceil_div(a.dv, 64)), static_cast<unsigned>(a.hv),
                  static_cast<unsigned>(a.nseq));
  hipLaunchKernelGGL(delta_scan<DKP>, grid, dim3(256), 0, st, a, ws);
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
  return static_cast<size_t>(ws_blocks(nseq, total)) * hv * kRec * 4;
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
  if (total <= kFew * nseq)
    recurrent_launch(a, st);
  else if (dk <= 64)
    blocked_launch<64>(a, static_cast<float*>(ws), st);
  else
    blocked_launch<128>(a, static_cast<float*>(ws), st);
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
