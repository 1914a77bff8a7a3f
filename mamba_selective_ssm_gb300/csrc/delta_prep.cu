// What the gated delta rule's chunks need and no state enters: M, P and the scalars of every chunk (delta_common.cuh).
// A CTA takes one (batch row, head, chunk): 4096 chunks with K = 128 in bf16 take 78 us, 6144 with K = 64 in fp32 140 us.  What
// bounds it is instructions and their latency at six CTAs of four warps an SM (shared memory) and five (registers): half of the issue
// slots; the substitution a third of the time, the 64 x 64 decays a fifth.  Memory is at a quarter of its rate (150 MB).
#include "delta_common.cuh"

namespace {

using namespace ssk;

constexpr int kPrepThreads = 128;
constexpr int kPrepLA = kDC + 4;  // floats from row to row of A

// M = (I + A beta)^{-1} A in place of A [64][kPrepLA], strictly lower triangular; be[s] = beta_s.  By substitution in fp32 and
// in the order of the tokens, which neither doubles small differences nor needs the powers of A that a product form does (for
// keys that resemble one another those reach 1e18): four diagonal blocks of 16 tokens at once, a column to a lane,
//   m_t = A_t - sum_{s < t} A_ts beta_s m_s,
// then twice the block below two of them in two products: X = A21 - A21 beta M11, M21 = X - M22 beta X.
template <int T>
struct Substitute {
  __device__ __forceinline__ static void go(const float* __restrict__ a, const float* __restrict__ be, float (&m)[16], float (&y)[16]) {
    Substitute<T - 1>::go(a, be, m, y);
    float s0 = m[T], s1 = 0.f, s2 = 0.f, s3 = 0.f;
#pragma unroll
    for (int s = 0; s < T; s += 4) {
      const float4 x = *reinterpret_cast<const float4*>(a + T * kPrepLA + s);
      s0 = fmaf(-x.x, y[s], s0);
      if (s + 1 < T) s1 = fmaf(-x.y, y[s + 1], s1);
      if (s + 2 < T) s2 = fmaf(-x.z, y[s + 2], s2);
      if (s + 3 < T) s3 = fmaf(-x.w, y[s + 3], s3);
    }
    m[T] = (s0 + s1) + (s2 + s3);
    y[T] = be[T] * m[T];
  }
};
template <>
struct Substitute<0> {
  __device__ __forceinline__ static void go(const float*, const float*, float (&m)[16], float (&y)[16]) { m[0] = y[0] = 0.f; }
};
// x[i] -= sum_{s < S} a[i][s] z[s] for R rows and two neighbouring columns, z[s] = be[s] * col[s * kPrepLA]
template <int S, int R>
__device__ __forceinline__ void below(const float* __restrict__ a, const float* __restrict__ be, const float* __restrict__ col, float2 (&x)[R]) {
#pragma unroll 2
  for (int s = 0; s < S; s += 4) {
    const float4 b = *reinterpret_cast<const float4*>(be + s);
    const float bb[4] = {-b.x, -b.y, -b.z, -b.w};
    float2 z[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) z[e] = mul2(bc2(bb[e]), *reinterpret_cast<const float2*>(col + (s + e) * kPrepLA));
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const float4 v = *reinterpret_cast<const float4*>(a + i * kPrepLA + s);
      x[i] = fma2(bc2(v.x), z[0], x[i]);
      x[i] = fma2(bc2(v.y), z[1], x[i]);
      x[i] = fma2(bc2(v.z), z[2], x[i]);
      x[i] = fma2(bc2(v.w), z[3], x[i]);
    }
  }
}
// the S x S block below the diagonal at tokens t0 .. t0 + 2 S: this thread's R rows from r and two columns from c of it
template <int S, int R>
__device__ __forceinline__ void join(float* A, const float* be, int t0, int r, int c) {
  float* d = A + t0 * (kPrepLA + 1);
  float* row = d + (S + r) * kPrepLA;
  float2 x[R];
#pragma unroll
  for (int i = 0; i < R; ++i) x[i] = *reinterpret_cast<const float2*>(row + i * kPrepLA + c);
  below<S, R>(row, be + t0, d + c, x);
  __syncthreads();
#pragma unroll
  for (int i = 0; i < R; ++i) *reinterpret_cast<float2*>(row + i * kPrepLA + c) = x[i];
  __syncthreads();
  below<S, R>(row + S, be + t0 + S, d + S * kPrepLA + c, x);
  __syncthreads();
#pragma unroll
  for (int i = 0; i < R; ++i) *reinterpret_cast<float2*>(row + i * kPrepLA + c) = x[i];
  __syncthreads();
}
__device__ __forceinline__ void solve(float* A, const float* be, int tid) {
  const int warp = tid >> 5, lane = tid & 31;
  if (lane < 16) {
    float* a = A + 16 * warp * (kPrepLA + 1);
    float m[16], y[16];
#pragma unroll
    for (int t = 0; t < 16; ++t) m[t] = a[t * kPrepLA + lane];
    Substitute<15>::go(a, be + 16 * warp, m, y);
    __syncwarp(0xffffu);
#pragma unroll
    for (int t = 0; t < 16; ++t) a[t * kPrepLA + lane] = m[t];
  }
  __syncthreads();
  join<16, 2>(A, be, (tid >> 6) * 32, (tid >> 3 & 7) * 2, (tid & 7) * 2);
  join<32, 4>(A, be, 0, (tid >> 4) * 4, (tid & 15) * 2);
}

template <typename T, int KP>
struct PrepSmem {
  static constexpr int tile = DTile<KP, kTerms<T>>::bytes;
  // A lies where k and q were
  static constexpr int k = 0, q = tile, a = 0, f = 2 * tile > kDC * kPrepLA * 4 ? 2 * tile : kDC * kPrepLA * 4;
  // scalars: running log2 decay (two floats), token scales of k and q, beta'
  static constexpr int bytes = f + 5 * kDC * 4;
};

__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// fp32 activations: k and q are scaled fp16 terms (delta_common.cuh), M and P operand tiles of such, M scaled row by row.
// bf16: everything in true units; M three tiles of bf16 terms, P tiles of such with `scale` in them.
template <typename T, int KP>
__global__ void __launch_bounds__(kPrepThreads) delta_prep_kernel(Delta p) {
  using S = PrepSmem<T, KP>;
  constexpr int N = kTerms<T>;
  extern __shared__ __align__(128) unsigned char raw[];
  const uint32_t sb = smem_u32(raw);
  float* A = reinterpret_cast<float*>(raw + S::a);
  float *chi = reinterpret_cast<float*>(raw + S::f), *clo = chi + kDC, *kup = clo + kDC, *qup = kup + kDC, *bp = qup + kDC;
  const LinAttn& a = p.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const long long item = blockIdx.x, bh = item / a.nck;
  const int ck = (int)(item % a.nck), h = (int)(bh % a.H), b = (int)(bh / a.H), gh = h / (a.H / a.G);
  const int t0 = ck * kDC, left = a.len(b) - t0, valid = left < kDC ? left : kDC;
  pdl_trigger();
  if (valid <= 0) return;  // the chunk is not walked
  const T* q = static_cast<const T*>(a.q) + ((long long)b * a.L + t0) * a.ldq + (long long)gh * a.K;
  const T* k = static_cast<const T*>(a.k) + ((long long)b * a.L + t0) * a.ldk + (long long)gh * a.K;
  tile_load<T, KP>(sb + S::k, k, a.ldk, valid, a.K, tid, kPrepThreads);
  tile_load<T, KP>(sb + S::q, q, a.ldq, valid, a.K, tid, kPrepThreads);
  cp_commit();
  const float beta = tid < valid ? p.beta[((long long)b * a.L + t0 + tid) * a.H + h] : 0.f;
  if (warp == 3) {
    ChunkGates<kDC> gates;
    if (a.g != nullptr) gates.fetch(a, b, h, t0, t0 + valid, lane);
    else gates.g[0] = gates.g[1] = 0.f;
    gates.scan(lane, [&](int i, Dec e) { chi[i] = e.hi; clo[i] = e.lo; });
  }
  cp_wait<0>();
  __syncthreads();
  if constexpr (N == 2) {
    tile_scale<KP, true>(sb + S::k, kup, tid, kPrepThreads);
    tile_scale<KP, false>(sb + S::q, qup, tid, kPrepThreads);
    __syncthreads();
  }
  float* vec = p.vec + item * kDVec;
  if (tid < kDC) {
    bp[tid] = N == 2 ? beta * kup[tid] * kup[tid] : beta;
    vec[tid] = dec_exp(chi[tid], clo[tid]);
    vec[kDC + tid] = dec_diff(chi[kDC - 1], clo[kDC - 1], chi[tid], clo[tid]);
    vec[2 * kDC + tid] = bp[tid];
    if (tid == 0) vec[4 * kDC] = dec_exp(chi[kDC - 1], clo[kDC - 1]);
  }
  // A and P, a warp's 16 rows against the tokens up to its own
  unsigned char* P = p.P + item * (long long)(N == 1 ? kDMTerms : kDMBytes);
  float kk[8][4];
  const int g = lane >> 2, c2 = 2 * (lane & 3);
  const float ps = N == 2 ? 1.f : a.scale;
#pragma unroll
  for (int np = 0; np < 4; ++np) {
    float qk[2][4], kl[2][4], ql[2][4];
    clear(kl);
    clear(ql);
#pragma unroll
    for (int e = 0; e < 4; ++e) kk[2 * np][e] = kk[2 * np + 1][e] = qk[0][e] = qk[1][e] = 0.f;
    if (np > warp) {
      if constexpr (N == 2) {  // (fp32: whole tiles are read; bf16: what is above the diagonal blocks is not)
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int n = 0; n < 2; ++n) *reinterpret_cast<uint32_t*>(P + DTile<kDC, 2>::at(16 * warp + g + 8 * e, 2 * np + i, n) + 2 * c2) = 0u;
      }
      continue;
    }
#pragma unroll 2
    for (int kb = 0; kb < KP / 16; ++kb) {
      uint32_t ka[N][4], qa[N][4], bb[N][4];
#pragma unroll
      for (int n = 0; n < N; ++n) {
        left_rows<KP, N>(ka[n], sb + S::k, warp, kb, n, lane);
        left_rows<KP, N>(qa[n], sb + S::q, warp, kb, n, lane);
        right_rows<KP, N>(bb[n], sb + S::k, np, kb, n, lane);
      }
      if constexpr (N == 1) {
        mma_bf16(kk[2 * np], ka[0], bb[0][0], bb[0][1]);
        mma_bf16(kk[2 * np + 1], ka[0], bb[0][2], bb[0][3]);
        mma_bf16(qk[0], qa[0], bb[0][0], bb[0][1]);
        mma_bf16(qk[1], qa[0], bb[0][2], bb[0][3]);
      } else {
        mma_terms(kk[2 * np], kk[2 * np + 1], kl[0], kl[1], ka[0], ka[N - 1], bb[0], bb[N - 1]);
        mma_terms(qk[0], qk[1], ql[0], ql[1], qa[0], qa[N - 1], bb[0], bb[N - 1]);
      }
    }
    if constexpr (N == 2) {
      fold(qk, ql);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        kk[2 * np][e] += kl[0][e];
        kk[2 * np + 1][e] += kl[1][e];
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int e = 0; e < 4; e += 2) {
        const int n = 2 * np + i, t = 16 * warp + g + (e >> 1) * 8, s = 8 * n + c2;
        const float2 sh = *reinterpret_cast<const float2*>(chi + s), sl = *reinterpret_cast<const float2*>(clo + s);
        const float th = chi[t], tl = clo[t];
        const float d0 = s <= t ? dec_diff(th, tl, sh.x, sl.x) : 0.f, d1 = s + 1 <= t ? dec_diff(th, tl, sh.y, sl.y) : 0.f;
        kk[n][e] = s < t ? kk[n][e] * d0 : 0.f;
        kk[n][e + 1] = s + 1 < t ? kk[n][e + 1] * d1 : 0.f;
        float y0 = s <= t ? qk[i][e] * d0 * ps : 0.f, y1 = s + 1 <= t ? qk[i][e + 1] * d1 * ps : 0.f;
        if constexpr (N == 2) {
          uint32_t hi, lo;
          split_half(y0, y1, hi, lo);
          *reinterpret_cast<uint32_t*>(P + DTile<kDC, 2>::at(t, n, 0) + 2 * c2) = hi;
          *reinterpret_cast<uint32_t*>(P + DTile<kDC, 2>::at(t, n, 1) + 2 * c2) = lo;
        } else {
#pragma unroll
          for (int m = 0; m < 3; ++m) {
            const uint32_t w = ActT<__nv_bfloat16>::pack2(y0, y1);
            *reinterpret_cast<uint32_t*>(P + m * (kDC * kDC * 2) + DTile<kDC, 1>::at(t, n, 0) + 2 * c2) = w;
            y0 -= bf16_lo(w);
            y1 -= bf16_hi(w);
          }
        }
      }
  }
  __syncthreads();  // k and q have been read
#pragma unroll
  for (int n = 0; n < 8; ++n)
#pragma unroll
    for (int e = 0; e < 4; e += 2)
      *reinterpret_cast<float2*>(A + (16 * warp + g + (e >> 1) * 8) * kPrepLA + 8 * n + c2) = make_float2(kk[n][e], kk[n][e + 1]);
  __syncthreads();
  solve(A, bp, tid);
  unsigned char* M = p.M + item * (N == 1 ? kDMTerms : kDMBytes);
  if constexpr (N == 1) {
    for (int i = tid; i < kDC * 8; i += kPrepThreads) {
      const int t = i >> 3, u = i & 7;
      if (u > 2 * (t >> 4) + 1) continue;  // (not read)
      float x[8];
      ActT<float>::ld8(A + t * kPrepLA + u * 8, x);
#pragma unroll
      for (int n = 0; n < 3; ++n) {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          w[e] = ActT<__nv_bfloat16>::pack2(x[2 * e], x[2 * e + 1]);
          x[2 * e] -= bf16_lo(w[e]);
          x[2 * e + 1] -= bf16_hi(w[e]);
        }
        *reinterpret_cast<uint4*>(M + n * (kDC * kDC * 2) + DTile<kDC, 1>::at(t, u, 0)) = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
  } else {
    for (int i = tid; i < kDC * 8; i += kPrepThreads) {  // eight lanes a row
      const int t = i >> 3, u = i & 7;
      float x[8], mx = 0.f;
      ActT<float>::ld8(A + t * kPrepLA + u * 8, x);
#pragma unroll
      for (int e = 0; e < 8; ++e) mx = fmaxf(mx, fabsf(x[e]));
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      const Pow2 s = operand_scale(mx);
      uint4 hi, lo;
      split_half(x[0] * s.down, x[1] * s.down, hi.x, lo.x);
      split_half(x[2] * s.down, x[3] * s.down, hi.y, lo.y);
      split_half(x[4] * s.down, x[5] * s.down, hi.z, lo.z);
      split_half(x[6] * s.down, x[7] * s.down, hi.w, lo.w);
      *reinterpret_cast<uint4*>(M + DTile<kDC, 2>::at(t, u, 0)) = hi;
      *reinterpret_cast<uint4*>(M + DTile<kDC, 2>::at(t, u, 1)) = lo;
      if (u == 0) vec[3 * kDC + t] = s.up;
    }
  }
}

template <typename T, int KP>
int prep(const Delta& p, cudaStream_t s) {
  return delta_launch(delta_prep_kernel<T, KP>, (unsigned)((long long)p.a.B * p.a.H * p.a.nck), kPrepThreads, PrepSmem<T, KP>::bytes, s, p);
}

}  // namespace

int ssh::delta_prep(const Delta& p, int dtype, cudaStream_t s) {
  if (dtype == SS_F32) return p.a.K <= 64 ? prep<float, 64>(p, s) : prep<float, 128>(p, s);
  return p.a.K <= 64 ? prep<__nv_bfloat16, 64>(p, s) : prep<__nv_bfloat16, 128>(p, s);
}
