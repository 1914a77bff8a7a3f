// Shared pieces of the linear attention kernels (linattn_fwd.cu, linattn_bwd.cu,
// linattn_step.cu): the call's arguments, the decays of a chunk and the plan
// that cuts a long sequence into segments.
//
//   S_t = exp(g_t) S_{t-1} + k_t v_t^T,   o_t = scale * S_t^T q_t       per (batch row, head)
//
// A chunk of C tokens with running log decay c_i = g_first + ... + g_i is
//   o_i   = scale * ( e^{c_i} q_i S_in + sum_{j<=i} e^{c_i - c_j} (q_i.k_j) v_j )
//   S_out = e^{c_last} S_in + sum_j e^{c_last - c_j} k_j v_j^T
// so all its products are matrix products and only S passes from chunk to chunk.
#pragma once

#include <type_traits>

#include "common.cuh"

namespace ssk {

// One call's arguments.  Rows of q, k, v are ld* elements apart (batch rows
// L * ld*); o, dout and the gradients are dense.
struct LinAttn {
  const void *q, *k, *v;
  long long ldq, ldk, ldv;
  const float* g;  // [B, L, H], or [H] with g_head
  int g_head;
  const int* lengths;  // [B] or null: tokens t >= lengths[b] neither decay nor add nor read
  int B, L, H, G, K, V;
  float scale;
  int nck;        // chunks of a row
  int nseg, cps;  // segments of a row and chunks per segment

  __device__ __forceinline__ int len(int b) const {
    if (lengths == nullptr) return L;
    const int n = lengths[b];
    return n < 0 ? 0 : n > L ? L : n;
  }
  __device__ __forceinline__ float gate(int b, int t, int h) const {
    return g_head ? g[h] : g[((size_t)b * L + t) * H + h];
  }
};

// A log decay in units of log2, as an unevaluated sum hi + lo of two floats.
// c_i - c_j of two far tokens is then good to ~2^-45 of c and exp2 of it to the
// hardware's rounding: a single float c would cost |c| * 2^-24 in the exponent,
// which after a few strong decays (c = -200) is 1e-5 of every later product.
// (Two floats, not a double: the running sums of a chunk in fp64 took 8000
// cycles of one warp that the other warps waited for, in two floats 700.)
struct Dec {
  float hi, lo;
};
__device__ __forceinline__ Dec dec_add(Dec a, Dec b) {
  const float s = __fadd_rn(a.hi, b.hi), t = __fsub_rn(s, a.hi);
  const float e = __fadd_rn(__fadd_rn(__fsub_rn(a.hi, __fsub_rn(s, t)), __fsub_rn(b.hi, t)), __fadd_rn(a.lo, b.lo));
  Dec r;
  r.hi = __fadd_rn(s, e);
  r.lo = __fsub_rn(e, __fsub_rn(r.hi, s));
  return r;
}
// Log decays below this empty the state in fp32 anyway (e^-160 = 0); the clamp
// keeps -inf, a reset, from making c_i - c_j = -inf + inf.
constexpr float kMinLogDecay = -160.0f;
__device__ __forceinline__ Dec dec_of_log(float g) {  // g log2(e)
  constexpr float kHi = 1.44269502f, kLo = 1.92596303e-8f;
  if (g < kMinLogDecay) g = kMinLogDecay;
  const float p = __fmul_rn(g, kHi), e = __fmaf_rn(g, kLo, __fmaf_rn(g, kHi, -p));
  Dec r;
  r.hi = __fadd_rn(p, e);
  r.lo = __fsub_rn(e, __fsub_rn(r.hi, p));
  return r;
}
__device__ __forceinline__ float dec_exp(float hi, float lo) { return ex2(hi) * fmaf(lo, kLn2, 1.0f); }
// e^{c_i - c_j}
__device__ __forceinline__ float dec_diff(float hi_i, float lo_i, float hi_j, float lo_j) {
  return ex2((hi_i - hi_j) + (lo_i - lo_j));
}

// The running log2 decays of chunks, by one warp: lane l owns C / 32 consecutive
// tokens.  fetch() reads a chunk's gates (a token past the row's end decays by
// 1), scan() puts their running sums with put(i, c_i); a caller fetches one
// chunk ahead, so that no one waits for the loads.
template <int C>
struct ChunkGates {
  static constexpr int PER = C / 32;
  float g[PER];
  __device__ __forceinline__ void fetch(const LinAttn& p, int b, int h, int t0, int len, int lane) {
#pragma unroll
    for (int e = 0; e < PER; ++e) {
      const int t = t0 + lane * PER + e;
      g[e] = t >= 0 && t < len ? p.gate(b, t, h) : 0.0f;
    }
  }
  // Running sums within groups of `lanes` lanes: x[e] becomes that of the lane's own tokens, `before` that of the
  // group's lanes before it, the result that through the lane's last token.
  __device__ __forceinline__ Dec sums(int lane, int lanes, Dec (&x)[PER], Dec& before) const {
    x[0] = dec_of_log(g[0]);
#pragma unroll
    for (int e = 1; e < PER; ++e) x[e] = dec_add(x[e - 1], dec_of_log(g[e]));
    Dec incl = x[PER - 1];
#pragma unroll
    for (int o = 1; o < lanes; o <<= 1) {
      Dec u;
      u.hi = __shfl_up_sync(0xffffffffu, incl.hi, o);
      u.lo = __shfl_up_sync(0xffffffffu, incl.lo, o);
      const Dec s = dec_add(incl, u);
      if ((lane & (lanes - 1)) >= o) incl = s;
    }
    before.hi = __shfl_up_sync(0xffffffffu, incl.hi, 1);
    before.lo = __shfl_up_sync(0xffffffffu, incl.lo, 1);
    if ((lane & (lanes - 1)) == 0) before.hi = before.lo = 0.0f;
    return incl;
  }
  template <typename Put>
  __device__ __forceinline__ void scan(int lane, Put put) const {
    Dec x[PER], before;
    sums(lane, 32, x, before);
#pragma unroll
    for (int e = 0; e < PER; ++e) put(lane * PER + e, dec_add(before, x[e]));
  }
  // Running sums within blocks of 32 tokens, rel[e] of the lane's own tokens, and in lane n the sum before block n.
  __device__ __forceinline__ Dec scan_rel(int lane, Dec (&rel)[PER]) const {
    constexpr int LB = 32 / PER;  // lanes of a block
    Dec before;
    const Dec incl = sums(lane, LB, rel, before);
#pragma unroll
    for (int e = 0; e < PER; ++e) rel[e] = dec_add(before, rel[e]);
    Dec base = {0.f, 0.f}, own = base;
#pragma unroll
    for (int n = 0; n < 32 / LB; ++n) {
      if (lane == n) own = base;
      Dec u;
      u.hi = __shfl_sync(0xffffffffu, incl.hi, n * LB + LB - 1);
      u.lo = __shfl_sync(0xffffffffu, incl.lo, n * LB + LB - 1);
      base = dec_add(base, u);
    }
    return own;
  }
};

constexpr int kLinMaxHead = 128;  // widest K, V
constexpr int kLinChunkF32 = 64;    // tokens of a chunk: fp32 (FMA pipe)
constexpr int kLinChunkBf16 = 128;  // bf16 (tensor cores: 128 rows of an MMA)

inline int linattn_chunk(int dtype) { return dtype == SS_F32 ? kLinChunkF32 : kLinChunkBf16; }

// Segments: with fewer independent walks (batch rows x heads x column tiles)
// than the GPU holds at once, a row is cut in `nseg` pieces whose end states
// are found first.  Each piece costs a second read of its inputs, so no more
// pieces than fill `slots` walks, and none shorter than four chunks.
inline void linattn_segments(LinAttn& p, int chunk, long long walks, int slots) {
  p.nck = (p.L + chunk - 1) / chunk;
  int n = walks > 0 ? (int)(slots / walks) : 1;
  if (n > p.nck / 4) n = p.nck / 4;
  if (n < 1) n = 1;
  p.cps = (p.nck + n - 1) / n;
  p.nseg = (p.nck + p.cps - 1) / p.cps;
}

inline int linattn_validate(int B, int L, int H, int G, int K, int V, int dtype) {
  if (B <= 0 || L <= 0 || H <= 0 || G <= 0 || K <= 0 || V <= 0) return SS_ERR_DIM;
  if (dtype != SS_F32 && dtype != SS_BF16) return SS_ERR_UNSUPPORTED;
  if (H % G != 0) return SS_ERR_DIM;
  if (K % 8 != 0 || V % 8 != 0) return SS_ERR_ALIGN;
  if (K > kLinMaxHead || V > kLinMaxHead) return SS_ERR_DIM;
  return SS_OK;
}

// a token stride: at least the row it holds, and rows on 16-byte boundaries
inline int linattn_ld_ok(long long ld, int width) {
  if (ld < width) return SS_ERR_DIM;
  return ld % 8 != 0 ? SS_ERR_ALIGN : SS_OK;
}

// an argument as the kernel takes it (untyped activations become its type)
template <typename K, typename A>
inline K lin_arg(A a) {
  if constexpr (std::is_same_v<A, const void*> && std::is_pointer_v<K>) return static_cast<K>(a);
  else return a;
}
template <typename... KArgs, typename... Args>
inline int lin_launch(void (*kern)(KArgs...), unsigned grid, int threads, size_t smem, cudaStream_t s, Args... args) {
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess) return SS_ERR_CUDA;
  kern<<<grid, threads, smem, s>>>(lin_arg<KArgs>(args)...);
  return cudaGetLastError() == cudaSuccess ? SS_OK : SS_ERR_CUDA;
}

// ---------------------------------------------------------------- FP32 tiles
// C += A B from shared memory on the FMA pipe, 256 threads as 16 x 16: thread
// (ty, tx) owns rows ty * M/16 + r and columns tx + 16 c of the M x N product.
// A is stored [M][Kd] (TA false) or [Kd][M]; B is stored [Kd][N] (TB false) or
// [N][Kd].  Every product of a kernel uses the same ownership, so accumulators
// of different products combine element by element in registers.
template <int M, int N, int Kd, bool TA, bool TB, int LDA, int LDB>
__device__ __forceinline__ void mm(const float* __restrict__ A, const float* __restrict__ B, float (&acc)[M / 16][N / 16], int tid) {
  constexpr int RM = M / 16, RN = N / 16;
  const int ty = tid >> 4, tx = tid & 15;
#pragma unroll 2
  for (int k = 0; k < Kd; k += 4) {
    float a[RM][4], b[RN][4];
#pragma unroll
    for (int r = 0; r < RM; ++r) {
      if constexpr (!TA) {
        const float4 v = *reinterpret_cast<const float4*>(A + (ty * RM + r) * LDA + k);
        a[r][0] = v.x; a[r][1] = v.y; a[r][2] = v.z; a[r][3] = v.w;
      }
    }
    if constexpr (TA) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int r = 0; r < RM; r += 4) {
          const float4 v = *reinterpret_cast<const float4*>(A + (k + e) * LDA + ty * RM + r);
          a[r][e] = v.x; a[r + 1][e] = v.y; a[r + 2][e] = v.z; a[r + 3][e] = v.w;
        }
    }
#pragma unroll
    for (int c = 0; c < RN; ++c) {
      if constexpr (TB) {
        const float4 v = *reinterpret_cast<const float4*>(B + (tx + 16 * c) * LDB + k);
        b[c][0] = v.x; b[c][1] = v.y; b[c][2] = v.z; b[c][3] = v.w;
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) b[c][e] = B[(k + e) * LDB + tx + 16 * c];
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
      for (int r = 0; r < RM; ++r)
#pragma unroll
        for (int c = 0; c < RN; ++c) acc[r][c] = fmaf(a[r][e], b[c][e], acc[r][c]);
  }
}

template <int R, int Cn>
__device__ __forceinline__ void zero_acc(float (&acc)[R][Cn]) {
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int c = 0; c < Cn; ++c) acc[r][c] = 0.f;
}

// C tokens x W columns of a strided input into a padded fp32 tile; columns
// past `width` and tokens past `valid` become zero (their memory is not read).
template <int C, int W, int LD>
__device__ __forceinline__ void load_tile(const float* __restrict__ src, long long ld, int valid, int width, float* dst, int tid) {
  for (int i = tid; i < C * (W / 8); i += 256) {
    const int t = i / (W / 8), c = (i % (W / 8)) * 8;
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (t < valid && c < width) ActT<float>::ld8(src + (long long)t * ld + c, v);
    ActT<float>::st8(dst + t * LD + c, v);
  }
}

// Row sums of a per-thread [rows][cols] product over the 16 threads of a row.
__device__ __forceinline__ float row_sum16(float v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

}  // namespace ssk
