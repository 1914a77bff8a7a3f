// Shared pieces of the gated delta rule's kernels (delta_prep.cu, delta_fwd.cu, delta_bwd.cu): the call's arguments,
// operand tiles and the products of a warp.
//
//   r_t = v_t - e^{g_t} S_{t-1}^T k_t,   S_t = e^{g_t} S_{t-1} + beta_t k_t r_t^T,   o_t = scale * S_t^T q_t
//
// A chunk of 64 tokens that starts in state S0, with running log decay c_t and D_ts = e^{c_t - c_s}:
//   A_ts = D_ts k_t.k_s (s < t)      M = (I + A beta)^{-1} A      P_ts = D_ts q_t.k_s (s <= t)
//   R = V - e^c K S0      r = R - M (beta R)      u = beta r
//   o = scale (e^c Q S0 + P u)      S1 = e^{c_last} S0 + K^T (e^{c_last - c} u)
// M and P depend on no state: delta_prep_kernel finds them for all chunks at once.  What passes from chunk to chunk is a
// chain of three products (K S0, M (beta R), K^T u), and every column of V is a chain of its own.
//
// fp32 inputs (this file's tiles and products; bf16 ones: delta_tc.cuh): products run on the tensor cores in fp16 with fp32
// sums, every operand as two fp16 terms (22 bits) scaled by a power of two to the range of fp16; k and q are scaled token by
// token:
//   k'_t = 2^{-e_t} k_t (largest element in [1, 2)),   beta' = 4^{e} beta,   v' = 2^{-e} v,   r' = 2^{-e} r,   u' = 2^{e} u
// leaves every formula above as it is.
#pragma once

#include <cuda_fp16.h>

#include "linattn_common.cuh"

namespace ssk {

constexpr int kDC = 64;        // tokens of a chunk
constexpr int kDVec = 272;     // floats of a chunk's scalars: into, rest, beta', M's row scales (64 each), e^{c_last}
constexpr int kDMBytes = kDC * kDC * 4;  // M of a chunk: two fp16 terms,
constexpr int kDMTerms = kDC * kDC * 6;  // or three of bf16; P alike

// One call's arguments.  a: q, k, v, g (null: no decay), lengths, sizes as in linear attention.
struct Delta {
  LinAttn a;
  const float* beta;  // [B, L, H]
  // what delta_prep_kernel leaves for each (batch row, head, chunk)
  unsigned char *M, *P;  // operand tiles
  float* vec;

  // the room they take, in bytes, and their places in it
  size_t prep_bytes(bool bf16) const { return items() * (2 * tile_bytes(bf16) + kDVec * sizeof(float)); }
  void place(void* at, bool bf16) {
    M = static_cast<unsigned char*>(at);
    P = M + items() * tile_bytes(bf16);
    vec = reinterpret_cast<float*>(P + items() * tile_bytes(bf16));
  }
  size_t items() const { return (size_t)a.B * a.H * a.nck; }
  static size_t tile_bytes(bool bf16) { return bf16 ? kDMTerms : kDMBytes; }
};

template <typename T>
constexpr int kTerms = sizeof(T) == 4 ? 2 : 1;  // fp16 terms of an activation

// What the forward leaves for the backward, floats of one (batch row, head): the state entering each chunk and the last one
// (fp32: [V][K]; bf16: [K / 4][V][4]), then of every chunk r and, in bf16, o, else the state's part of o, all in fp32 (fp32:
// [V][64]; bf16: [16][V][4]).  Behind all heads' lie M, P and the scalars of all chunks, so that the backward need not find them
// again (78 us at 4 x 2048 tokens of 32 heads of 128 x 128, of a training step's 948 then).
__host__ __device__ inline long long delta_ckpt_floats(int nck, int K, int V) {
  return (long long)(nck + 1) * K * V + 2ll * nck * kDC * V;
}

// Launches a kernel that may start while the one before it ends (each CTA of it calls pdl_wait): its first tiles, its barriers
// and its tensor memory are then ready when that is done (3 to 5 us a pair).
template <typename... KArgs, typename... Args>
inline int delta_launch_next(void (*kern)(KArgs...), unsigned grid, int threads, size_t smem, cudaStream_t s, Args... args) {
  if (!allow_smem(kern)) return SS_ERR_CUDA;
  return launch_dependent(kern, dim3(grid), dim3((unsigned)threads), smem, s, args...) == cudaSuccess ? SS_OK : SS_ERR_CUDA;
}

template <typename... KArgs, typename... Args>
inline int delta_launch(void (*kern)(KArgs...), unsigned grid, int threads, size_t smem, cudaStream_t s, Args... args) {
  if (!allow_smem(kern)) return SS_ERR_CUDA;
  kern<<<grid, threads, smem, s>>>(args...);
  return cudaGetLastError() == cudaSuccess ? SS_OK : SS_ERR_CUDA;
}

inline int delta_validate(int B, int L, int H, int G, int K, int V, int dtype) {
  const int rc = linattn_validate(B, L, H, G, K, V, dtype);
  if (rc != SS_OK) return rc;
  return (long long)B * H > (1ll << 24) || (long long)B * H * ((L + kDC - 1) / kDC) > 2147483647ll / 8 ? SS_ERR_DIM : SS_OK;
}

// ---------------------------------------------------------------- operand tiles
// Rows of W columns of fp16 in N terms: 16-byte unit u (8 columns) of term n lies at unit (u N + n) ^ (row & 7) of its
// row, so that the eight rows an ldmatrix reads fall on different banks.  A raw tile (activations as they are in memory)
// takes the same bytes: unit u of bf16, or of fp32 as its two halves.
template <int W, int N>
struct DTile {
  static constexpr int row = W * 2 * N, bytes = kDC * row;
  __device__ __forceinline__ static uint32_t at(int r, int u, int n) { return (uint32_t)(r * row + (((u * N + n) ^ (r & 7)) << 4)); }
};

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool on) {
  const int n = on ? 16 : 0;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void sts128(uint32_t a, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// kDC rows of `width` columns of activations, `ld` elements apart, as a raw tile; rows from `valid` and columns from
// `width` on are zero (their memory is not read)
template <typename T, int W>
__device__ __forceinline__ void tile_load(uint32_t tile, const T* __restrict__ src, long long ld, int valid, int width, int tid, int nt) {
  constexpr int N = kTerms<T>, U = W / 8;
  for (int i = tid; i < kDC * U * N; i += nt) {
    const int r = i / (U * N), x = i % (U * N), u = x / N, n = x % N;
    const bool on = r < valid && u * 8 < width;
    cp16(tile + DTile<W, N>::at(r, u, n), src + (on ? (long long)r * ld + u * 8 + n * 4 : 0), on);
  }
}
// a finished tile of `bytes` bytes from memory
__device__ __forceinline__ void tile_copy(uint32_t tile, const unsigned char* __restrict__ src, int bytes, int tid, int nt) {
  for (int i = tid * 16; i < bytes; i += nt * 16) cp16(tile + i, src + i, true);
}

// 2^-e and 2^e for e = the exponent of m >= 0, kept where both are normal numbers (and e at most 2^60 from 1)
struct Pow2 {
  float down, up;
};
template <int SHIFT, int MIN, int MAX>
__device__ __forceinline__ Pow2 pow2_of(float m) {
  int e = (int)(__float_as_uint(m) >> 23) & 0xff;
  e = e < MIN ? MIN : e > MAX ? MAX : e;
  Pow2 p;
  p.down = __uint_as_float((uint32_t)(254 - e + SHIFT) << 23);
  p.up = __uint_as_float((uint32_t)(e - SHIFT) << 23);
  return p;
}
// an operand of a product: its largest value into [2^13, 2^14)
__device__ __forceinline__ Pow2 operand_scale(float m) { return pow2_of<13, 14, 253>(m); }
// a token's row: its largest element into [1, 2).  A key's scale is squared in beta', so keys have it within 2^60 of 1: elements
// of 2^60 and more overflow, those of keys below 2^-60 lose bits.
template <bool KEY>
__device__ __forceinline__ Pow2 token_scale(float m) {
  return m == 0.f ? Pow2{1.f, 1.f} : KEY ? pow2_of<0, 127 - 60, 127 + 60>(m) : pow2_of<0, 1, 253>(m);
}

__device__ __forceinline__ uint32_t pack_half(float x, float y) {
  const __half2 h = __floats2half2_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 wide_half(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2*>(&w)); }
// x, y as two fp16 terms: the first is off by 2^-11 of the value at most, both by 2^-22
__device__ __forceinline__ void split_half(float x, float y, uint32_t& hi, uint32_t& lo) {
  hi = pack_half(x, y);
  const float2 f = wide_half(hi);
  lo = pack_half(x - f.x, y - f.y);
}
__device__ __forceinline__ void store_terms(uint32_t hi_at, uint32_t lo_at, const float (&x)[8]) {
  uint4 h, l;
  split_half(x[0], x[1], h.x, l.x);
  split_half(x[2], x[3], h.y, l.y);
  split_half(x[4], x[5], h.z, l.z);
  split_half(x[6], x[7], h.w, l.w);
  sts128(hi_at, h);
  sts128(lo_at, l);
}

// Raw fp32 rows become scaled fp16 operands in place; up[r] = the row's 2^e.  W / 8 neighbouring lanes hold a row.
template <int W, bool KEY>
__device__ __forceinline__ void tile_scale(uint32_t tile, float* up, int tid, int nt) {
  constexpr int U = W / 8;
  for (int i = tid; i < kDC * U; i += nt) {  // nt and kDC * U are multiples of 32: whole warps
    const int r = i / U, u = i % U;
    const uint32_t a0 = tile + DTile<W, 2>::at(r, u, 0), a1 = tile + DTile<W, 2>::at(r, u, 1);
    const uint4 p = lds128(a0), q = lds128(a1);
    float x[8] = {__uint_as_float(p.x), __uint_as_float(p.y), __uint_as_float(p.z), __uint_as_float(p.w),
                  __uint_as_float(q.x), __uint_as_float(q.y), __uint_as_float(q.z), __uint_as_float(q.w)};
    float m = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(x[e]));
#pragma unroll
    for (int o = 1; o < U; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const Pow2 s = token_scale<KEY>(m);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] *= s.down;
    store_terms(a0, a1, x);
    if (u == 0) up[r] = s.up;
  }
}

// ---------------------------------------------------------------- a warp's products
// m16n8k16: a warp's accumulators of a 16 x 8 tile are c[0..1] of row lane / 4 and c[2..3] of row lane / 4 + 8, columns
// 2 (lane % 4) and the next.  As the left operand of the next product they are where they have to be: a chain of products
// whose rows are columns of V stays in registers.
__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldsm(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
__device__ __forceinline__ void ldsm_t(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}

// Right operands from a tile, for two neighbouring column tiles of 8: b[0], b[1] of the first, b[2], b[3] of the second.
// The contraction runs along the tile's columns (16 from 16 kb), the product's columns are its rows (16 from 16 np):
template <int W, int N>
__device__ __forceinline__ void right_rows(uint32_t (&b)[4], uint32_t tile, int np, int kb, int n, int lane) {
  const int mi = lane >> 3;
  ldsm(b, tile + DTile<W, N>::at(16 * np + (mi >> 1) * 8 + (lane & 7), 2 * kb + (mi & 1), n));
}
// ... down the tile's rows (16 from 16 kb), the product's columns are its columns (16 from 16 jp):
template <int W, int N>
__device__ __forceinline__ void right_cols(uint32_t (&b)[4], uint32_t tile, int jp, int kb, int n, int lane) {
  const int mi = lane >> 3;
  ldsm_t(b, tile + DTile<W, N>::at(16 * kb + (mi & 1) * 8 + (lane & 7), 2 * jp + (mi >> 1), n));
}
// Left operands: 16 rows from 16 mb, contraction along the columns (16 from 16 kb)
template <int W, int N>
__device__ __forceinline__ void left_rows(uint32_t (&a)[4], uint32_t tile, int mb, int kb, int n, int lane) {
  const int mi = lane >> 3;
  ldsm(a, tile + DTile<W, N>::at(16 * mb + (mi & 1) * 8 + (lane & 7), 2 * kb + (mi >> 1), n));
}
// ... rows are the tile's columns (16 from 16 mb), contraction down its rows (16 from 16 kb)
template <int W, int N>
__device__ __forceinline__ void left_cols(uint32_t (&a)[4], uint32_t tile, int mb, int kb, int n, int lane) {
  const int mi = lane >> 3;
  ldsm_t(a, tile + DTile<W, N>::at(16 * kb + (mi >> 1) * 8 + (lane & 7), 2 * mb + (mi & 1), n));
}

// The scale of each of a thread's two rows of accumulators: [0] row lane / 4, [1] row lane / 4 + 8
struct RowScale {
  Pow2 r[2];
};
template <int N>
__device__ __forceinline__ RowScale row_scale(const float (&x)[N][4]) {
  float m0 = 0.f, m1 = 0.f;
#pragma unroll
  for (int j = 0; j < N; ++j) {
    m0 = fmaxf(m0, fmaxf(fabsf(x[j][0]), fabsf(x[j][1])));
    m1 = fmaxf(m1, fmaxf(fabsf(x[j][2]), fabsf(x[j][3])));
  }
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    m0 = fmaxf(m0, __shfl_xor_sync(0xffffffffu, m0, o));
    m1 = fmaxf(m1, __shfl_xor_sync(0xffffffffu, m1, o));
  }
  return RowScale{{operand_scale(m0), operand_scale(m1)}};
}
// accumulators of two neighbouring column tiles as the left operand of a product that contracts over them, in two terms
__device__ __forceinline__ void left_terms(uint32_t (&h)[4], uint32_t (&l)[4], const float (&x)[4], const float (&y)[4], const RowScale& s) {
  split_half(x[0] * s.r[0].down, x[1] * s.r[0].down, h[0], l[0]);
  split_half(x[2] * s.r[1].down, x[3] * s.r[1].down, h[1], l[1]);
  split_half(y[0] * s.r[0].down, y[1] * s.r[0].down, h[2], l[2]);
  split_half(y[2] * s.r[1].down, y[3] * s.r[1].down, h[3], l[3]);
}

// c0, c1 += (h + l) (b + bl) over one step of 16; the lowest terms' product is dropped (2^-22).  The tensor core cuts its sums, and
// three products a step into one sum left outputs 1.5 to 2.5 times as far off as plain fp32 (1.3e-6 for 5e-7 with beta up to
// 2).  So the low products have sums of their own, d0 and d1, which fold() adds at the end, and c0 and c1 are cut once a step: as far
// off as plain fp32, for 3 % of a training step.
__device__ __forceinline__ void mma_terms(float (&c0)[4], float (&c1)[4], float (&d0)[4], float (&d1)[4], const uint32_t (&h)[4],
                                          const uint32_t (&l)[4], const uint32_t (&b)[4], const uint32_t (&bl)[4]) {
  mma_f16(c0, h, b[0], b[1]);
  mma_f16(c1, h, b[2], b[3]);
  mma_f16(d0, l, b[0], b[1]);
  mma_f16(d1, l, b[2], b[3]);
  mma_f16(d0, h, bl[0], bl[1]);
  mma_f16(d1, h, bl[2], bl[3]);
}
template <int M>
__device__ __forceinline__ void fold(float (&c)[M][4], const float (&d)[M][4]) {
#pragma unroll
  for (int n = 0; n < M; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) c[n][e] += d[n][e];
}
template <int M>
__device__ __forceinline__ void clear(float (&c)[M][4]) {
#pragma unroll
  for (int n = 0; n < M; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) c[n][e] = 0.f;
}

// A warp's own 16 columns of V of a chunk of fp32 (v or do), rows of 80 bytes (banks)
struct DSlice {
  static constexpr int bytes = kDC * 80;
  __device__ __forceinline__ static void load(uint32_t s, const float* __restrict__ src, long long ld, int valid, int width, int lane) {
#pragma unroll
    for (int i = lane; i < kDC * 4; i += 32) {
      const int t = i >> 2, u = i & 3;
      const bool on = t < valid && u * 4 < width;
      cp16(s + t * 80 + u * 16, src + (on ? (long long)t * ld + u * 4 : 0), on);
    }
  }
  __device__ __forceinline__ static float get(uint32_t s, int t, int v) {
    float x;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(x) : "r"(s + t * 80 + v * 4) : "memory");
    return x;
  }
  __device__ __forceinline__ static void read(uint32_t s, int p, int lane, float (&x)[4], float (&y)[4]) {
    const int g = lane >> 2, t = 16 * p + 2 * (lane & 3);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[e] = get(s, t + (e & 1), g + (e >> 1) * 8);
      y[e] = get(s, t + 8 + (e & 1), g + (e >> 1) * 8);
    }
  }
};

// Accumulators (rows = 16 columns of V from v0, columns = 8 tokens from t) to rows of a [.., ld] array
__device__ __forceinline__ void store_tokens(float* __restrict__ dst, long long ld, int t, int rows, int width, const float (&x)[4], int lane) {
  const int g = lane >> 2, r = t + 2 * (lane & 3);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int c = g + (e >> 1) * 8;
    if (r + (e & 1) < rows && c < width) dst[(long long)(r + (e & 1)) * ld + c] = x[e];
  }
}

}  // namespace ssk

namespace ssh {
// Launches delta_prep_kernel for all chunks of a call.
int delta_prep(const ssk::Delta& p, int dtype, cudaStream_t s);
// The chunks' walk in bf16, after delta_prep.
int delta_fwd_bf16(const ssk::Delta& p, const float* h0, void* o, float* ckpt, float* h_last, cudaStream_t s);
// The backward's walk in bf16: dv, dh0, and dS ([K / 4][V][4]) and du ([16][V][4]) of
// every chunk.
int delta_back_bf16(const ssk::Delta& p, const void* dout, const float* dh_last, void* dv, float* dS, float* du, float* dh0, cudaStream_t s);
// The other gradients in bf16, chunk by chunk.  dq, dk: rows of `heads` heads, bf16 or (parts) fp32
int delta_grad_bf16(const ssk::Delta& p, const float* ckpt, const void* dout, const float* dS, const float* du, void* dq, void* dk, bool parts,
                    float* dg, float* dbeta, cudaStream_t s);
}  // namespace ssh
