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

constexpr int kLinMaxHead = 128;    // widest K, V
constexpr int kLinMaxLen = 2147483136;  // longest row: token numbers up to three chunks past its end are still an int
constexpr int kLinChunkF32 = 64;    // tokens of a chunk: fp32 (its tiles fit shared memory)
constexpr int kLinChunkBf16 = 128;  // bf16 (the 128 rows of an MMA)

inline int linattn_chunk(int dtype) { return dtype == SS_F32 ? kLinChunkF32 : kLinChunkBf16; }

// Segments: with fewer independent walks (batch rows x heads, x column tiles
// for the fp32 forward) than fill the GPU, a row is cut in pieces of at least
// four chunks whose end states are found first, at the price of a second read of
// half the inputs.  The tensor-core kernels hold an SM each: as many pieces as
// leave every one of them its own (16384 tokens of 32 heads of 128 x 64: 152 us,
// 349 uncut, 155 for twice as many; 8192 forward and backward 366, 909, 392).  From
// 77 walks on nothing is cut, so a count a little above the SMs' takes two turns
// of whole rows (4 x 2048 tokens of 32 heads of 128 x 128, 128 walks: 77 us, 5 x 2048,
// 160 walks: 141).  The fp32 kernels share an SM (three forward,
// two backward) and their time is arithmetic: pieces for three CTAs an SM, so that
// no SM is left with far more than its share (a training step of 192 walks of
// 2048 tokens, 64 x 64: 1449 us for three pieces, 1516 for six, 1766 for two, 1741
// uncut).  The sums are taken over the last piece walked too, whose end no one reads.
inline void linattn_segments(LinAttn& p, int dtype, long long walks) {
  const int chunk = linattn_chunk(dtype);
  p.nck = (p.L + chunk - 1) / chunk;
  long long n = dtype == SS_F32 ? (3 * 152 + walks - 1) / walks : 152 / walks;
  if (n > p.nck / 4) n = p.nck / 4;
  if (n < 1) n = 1;
  p.cps = (int)((p.nck + n - 1) / n);
  p.nseg = (p.nck + p.cps - 1) / p.cps;
}

inline int linattn_validate(int B, int L, int H, int G, int K, int V, int dtype) {
  if (B <= 0 || L <= 0 || H <= 0 || G <= 0 || K <= 0 || V <= 0 || L > kLinMaxLen) return SS_ERR_DIM;
  if (dtype != SS_F32 && dtype != SS_BF16) return SS_ERR_UNSUPPORTED;
  if (H % G != 0) return SS_ERR_DIM;
  if (K % 8 != 0 || V % 8 != 0) return SS_ERR_ALIGN;
  if (K > kLinMaxHead || V > kLinMaxHead) return SS_ERR_DIM;
  return SS_OK;
}

// a token stride: at least the row it holds, and rows on 16-byte boundaries
inline int linattn_ld_ok(long long ld, int heads, int width) {
  if (ld < (long long)heads * width) return SS_ERR_DIM;
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
// fp32 products from shared memory on the tensor cores: each operand is split
// in registers into a tf32 value and the tf32 of what that leaves (22 bits), and
// the three products that matter are summed in fp32, the smallest first; what is
// dropped is 2^-22 of a term.  Each step of 8 is summed by itself and added with a
// rounding: the tensor core cuts its sums, which into a state carried over 32
// chunks added up to 1e-5 of it.  The outputs are off by 6e-7 of their root mean square
// over 32 chunks (2e-7 for plain fp32 products).  These take operands from registers
// (mma.sync), so that a tile lies in shared memory once and in fp32, and are split
// again for every product.  tcgen05 reads its operands from shared memory: both
// halves of q, k, v, do and two states are 192 KB for heads of 64 x 64 and do not fit
// for wider ones; that form has not been built.  (On the
// FMA pipe the same kernels were bound by shared memory: 8 x 4 products a thread
// read 16 vectors for every 128 multiplies.)
//
// Warps tile the M x N product; a thread's accumulators acc[r][c] are rows row(r)
// and columns col(c), columns in neighbouring pairs.  Products of the same shape
// have the same owners, so they combine element by element in registers.
template <int NT, int M, int N>
struct Own {
  static constexpr int TM = M * N == 64 * 64 ? 16 : 32, WM = M / TM, WN = NT / 32 / WM, TN = N / WN;
  static constexpr int RM = TM / 8, RN = TN / 4;
  static_assert(WM * WN * 32 == NT && WN * TN == N, "warps tile the product");
  __device__ __forceinline__ static int wn(int tid) { return (tid >> 5) % WN; }
  __device__ __forceinline__ static int row(int tid, int r) {
    return (tid >> 5) / WN * TM + (r >> 1) * 16 + (r & 1) * 8 + ((tid & 31) >> 2);
  }
  __device__ __forceinline__ static int col(int tid, int c) { return wn(tid) * TN + (c >> 1) * 8 + (tid & 3) * 2 + (c & 1); }
  float v[RM][RN];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int r = 0; r < RM; ++r)
#pragma unroll
      for (int c = 0; c < RN; ++c) v[r][c] = 0.f;
  }
  // f(row, column, value pair) over neighbouring columns
  template <typename F>
  __device__ __forceinline__ void pairs(int tid, F f) {
#pragma unroll
    for (int r = 0; r < RM; ++r)
#pragma unroll
      for (int c = 0; c < RN; c += 2) f(row(tid, r), col(tid, c), v[r][c], v[r][c + 1]);
  }
  // every row times f(row)
  template <typename F>
  __device__ __forceinline__ void scale_rows(int tid, F f) {
#pragma unroll
    for (int r = 0; r < RM; ++r) {
      const float e = f(row(tid, r));
#pragma unroll
      for (int c = 0; c < RN; ++c) v[r][c] *= e;
    }
  }
};

__device__ __forceinline__ void tf32_split(float x, uint32_t& hi, uint32_t& lo) {
  asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(hi) : "f"(x));
  lo = __float_as_uint(x - __uint_as_float(hi));
}
__device__ __forceinline__ void mma_tf32(float& c0, float& c1, float& c2, float& c3, const uint32_t (&a)[4], const uint32_t (&b)[2]) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c0), "+f"(c1), "+f"(c2), "+f"(c3)
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}

// acc += A B.  A is stored [M][Kd] (TA false) or [Kd][M]; B is stored [Kd][N] (TB false) or [N][Kd].
template <bool TA, bool TB, int LDA, int LDB, int Kd, int NT, int M, int N>
__device__ __forceinline__ void mm(const float* __restrict__ A, const float* __restrict__ B, Own<NT, M, N>& acc, int tid) {
  using O = Own<NT, M, N>;
  constexpr int MT = O::RM / 2, NL = O::RN / 2;
  const int lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int m0 = (tid >> 5) / O::WN * O::TM + g, n0 = O::wn(tid) * O::TN + g;
#pragma unroll 2
  for (int k = 0; k < Kd; k += 8) {
    uint32_t ah[MT][4], al[MT][4];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int i = m0 + m * 16 + (e & 1) * 8, kk = k + t + (e >> 1) * 4;
        tf32_split(TA ? A[kk * LDA + i] : A[i * LDA + kk], ah[m][e], al[m][e]);
      }
#pragma unroll
    for (int n = 0; n < NL; ++n) {
      uint32_t bh[2], bl[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int j = n0 + n * 8, kk = k + t + e * 4;
        tf32_split(TB ? B[j * LDB + kk] : B[kk * LDB + j], bh[e], bl[e]);
      }
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        float c0 = 0.f, c1 = 0.f, c2 = 0.f, c3 = 0.f;
        mma_tf32(c0, c1, c2, c3, al[m], bh);
        mma_tf32(c0, c1, c2, c3, ah[m], bl);
        mma_tf32(c0, c1, c2, c3, ah[m], bh);
        acc.v[2 * m][2 * n] += c0;
        acc.v[2 * m][2 * n + 1] += c1;
        acc.v[2 * m + 1][2 * n] += c2;
        acc.v[2 * m + 1][2 * n + 1] += c3;
      }
    }
  }
}

// C tokens x W columns of a strided input into a padded fp32 tile; columns
// past `width` and tokens past `valid` become zero (their memory is not read).
template <int NT, int C, int W, int LD>
__device__ __forceinline__ void load_tile(const float* __restrict__ src, long long ld, int valid, int width, float* dst, int tid) {
  for (int i = tid; i < C * (W / 8); i += NT) {
    const int t = i / (W / 8), c = (i % (W / 8)) * 8;
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (t < valid && c < width) ActT<float>::ld8(src + (long long)t * ld + c, v);
    ActT<float>::st8(dst + t * LD + c, v);
  }
}

// Sum over the four threads of a warp that share a row of an Own<>.
__device__ __forceinline__ float row_sum4(float v) {
  v += __shfl_xor_sync(0xffffffffu, v, 1);
  return v + __shfl_xor_sync(0xffffffffu, v, 2);
}
__device__ __forceinline__ void st_pair(float* p, float x, float y) { *reinterpret_cast<float2*>(p) = make_float2(x, y); }

}  // namespace ssk
