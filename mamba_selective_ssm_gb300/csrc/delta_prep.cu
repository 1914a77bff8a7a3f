// What the gated delta rule's chunks need and no state enters: M, P and the scalars of every chunk (delta_common.cuh).
// A CTA takes one (batch row, head, chunk).
#include "delta_common.cuh"

namespace {

using namespace ssk;

constexpr int kPrepThreads = 128;

template <typename T, int KP>
struct PrepSmem {
  static constexpr int tile = DTile<KP, kTerms<T>>::bytes, LA = kDC + 4;  // floats from row to row of A
  static constexpr int k = 0, q = tile, a = 2 * tile, f = a + kDC * LA * 4;
  // scalars: running log2 decay (two floats), token scales of k and q, beta'
  static constexpr int bytes = f + 5 * kDC * 4;
};

// M = (I + A beta)^{-1} A by substitution, a column to a thread: M_tj = A_tj - sum_{j<s<t} (A beta)_ts M_sj, in fp32 and in
// the order of the tokens, which neither doubles small differences nor needs the powers of A that a product form does
// (for keys that resemble one another those reach 1e18).
template <int T>
struct Solve {
  __device__ __forceinline__ static void go(const float* __restrict__ ab, int LA, float (&m)[kDC], int j) {
    Solve<T - 1>::go(ab, LA, m, j);
    float s0 = 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
#pragma unroll
    for (int s = 0; s < T; s += 4) {
      const float4 x = *reinterpret_cast<const float4*>(ab + T * LA + s);
      s0 = fmaf(x.x, m[s], s0);
      if (s + 1 < T) s1 = fmaf(x.y, m[s + 1], s1);
      if (s + 2 < T) s2 = fmaf(x.z, m[s + 2], s2);
      if (s + 3 < T) s3 = fmaf(x.w, m[s + 3], s3);
    }
    m[T] = j < T ? m[T] - ((s0 + s1) + (s2 + s3)) : 0.f;
  }
};
template <>
struct Solve<0> {
  __device__ __forceinline__ static void go(const float*, int, float (&m)[kDC], int) { m[0] = 0.f; }
};

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
  if (valid <= 0) return;  // the chunk is not walked
  const T* q = static_cast<const T*>(a.q) + ((long long)b * a.L + t0) * a.ldq + (long long)gh * a.K;
  const T* k = static_cast<const T*>(a.k) + ((long long)b * a.L + t0) * a.ldk + (long long)gh * a.K;
  tile_load<T, KP>(sb + S::k, k, a.ldk, valid, a.K, tid, kPrepThreads);
  tile_load<T, KP>(sb + S::q, q, a.ldq, valid, a.K, tid, kPrepThreads);
  cp_commit();
  if (warp == 0) {
    ChunkGates<kDC> gates;
    if (a.g != nullptr) gates.fetch(a, b, h, t0, t0 + valid, lane);
    else gates.g[0] = gates.g[1] = 0.f;
    gates.scan(lane, [&](int i, Dec e) { chi[i] = e.hi; clo[i] = e.lo; });
  }
  cp_wait<0>();
  __syncthreads();
  tile_scale<T, KP>(sb + S::k, kup, tid, kPrepThreads);
  tile_scale<T, KP>(sb + S::q, qup, tid, kPrepThreads);
  __syncthreads();
  float* vec = p.vec + item * kDVec;
  if (tid < kDC) {
    const float beta = tid < valid ? p.beta[((long long)b * a.L + t0 + tid) * a.H + h] : 0.f;
    bp[tid] = beta * kup[tid] * kup[tid];
    vec[tid] = dec_exp(chi[tid], clo[tid]);
    vec[kDC + tid] = dec_diff(chi[kDC - 1], clo[kDC - 1], chi[tid], clo[tid]);
    vec[2 * kDC + tid] = bp[tid];
    if (tid == 0) vec[4 * kDC] = dec_exp(chi[kDC - 1], clo[kDC - 1]);
  }
  __syncthreads();
  // A and P, a warp's 16 rows against the tokens up to its own
  unsigned char* P = p.P + item * (long long)(kDC * kDC * 2) * p.pterms;
  {
    float kk[8][4], qk[8][4];
#pragma unroll
    for (int n = 0; n < 8; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) kk[n][e] = qk[n][e] = 0.f;
#pragma unroll 2
    for (int kb = 0; kb < KP / 16; ++kb) {
      uint32_t ka[N][4], qa[N][4];
#pragma unroll
      for (int n = 0; n < N; ++n) {
        left_rows<KP, N>(ka[n], sb + S::k, warp, kb, n, lane);
        left_rows<KP, N>(qa[n], sb + S::q, warp, kb, n, lane);
      }
#pragma unroll
      for (int np = 0; np < 4; ++np) {
        if (np > warp) continue;
        uint32_t bb[N][4];
#pragma unroll
        for (int n = 0; n < N; ++n) right_rows<KP, N>(bb[n], sb + S::k, np, kb, n, lane);
        if constexpr (N == 1) {
          mma_f16(kk[2 * np], ka[0], bb[0][0], bb[0][1]);
          mma_f16(kk[2 * np + 1], ka[0], bb[0][2], bb[0][3]);
          mma_f16(qk[2 * np], qa[0], bb[0][0], bb[0][1]);
          mma_f16(qk[2 * np + 1], qa[0], bb[0][2], bb[0][3]);
        } else {
          mma_terms<2>(kk[2 * np], kk[2 * np + 1], ka[0], ka[N - 1], bb[0], bb[N - 1]);
          mma_terms<2>(qk[2 * np], qk[2 * np + 1], qa[0], qa[N - 1], bb[0], bb[N - 1]);
        }
      }
    }
    const int g = lane >> 2;
#pragma unroll
    for (int n = 0; n < 8; ++n) {
#pragma unroll
      for (int e = 0; e < 4; e += 2) {
        const int t = 16 * warp + g + (e >> 1) * 8, s = 8 * n + 2 * (lane & 3);
        float x[2], y[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float d = s + i <= t ? dec_diff(chi[t], clo[t], chi[s + i], clo[s + i]) : 0.f;
          x[i] = s + i < t ? kk[n][e + i] * d : 0.f;
          y[i] = s + i <= t ? qk[n][e + i] * d : 0.f;
        }
        *reinterpret_cast<float2*>(A + t * S::LA + s) = make_float2(x[0], x[1]);
        uint32_t hi, lo;
        split_half(y[0], y[1], hi, lo);
        if (p.pterms == 1) {
          *reinterpret_cast<uint32_t*>(P + DTile<kDC, 1>::at(t, n, 0) + 4 * (lane & 3)) = hi;
        } else {
          *reinterpret_cast<uint32_t*>(P + DTile<kDC, 2>::at(t, n, 0) + 4 * (lane & 3)) = hi;
          *reinterpret_cast<uint32_t*>(P + DTile<kDC, 2>::at(t, n, 1) + 4 * (lane & 3)) = lo;
        }
      }
    }
  }
  __syncthreads();
  float m[kDC];
  if (tid < kDC) {
#pragma unroll
    for (int t = 0; t < kDC; ++t) m[t] = A[t * S::LA + tid];
  }
  __syncthreads();
  for (int i = tid; i < kDC * kDC; i += kPrepThreads) A[i / kDC * S::LA + i % kDC] *= bp[i % kDC];
  __syncthreads();
  if (tid < kDC) Solve<kDC - 1>::go(A, S::LA, m, tid);
  __syncthreads();
  if (tid < kDC) {
#pragma unroll
    for (int t = 0; t < kDC; ++t) A[t * S::LA + tid] = m[t];
  }
  __syncthreads();
  unsigned char* M = p.M + item * kDMBytes;
  for (int i = tid; i < kDC * 8; i += kPrepThreads) {  // eight lanes a row
    const int t = i >> 3, u = i & 7;
    float x[8], mx = 0.f;
    ActT<float>::ld8(A + t * S::LA + u * 8, x);
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

template <typename T, int KP>
int prep(const Delta& p, cudaStream_t s) {
  return lin_launch(delta_prep_kernel<T, KP>, (unsigned)((long long)p.a.B * p.a.H * p.a.nck), kPrepThreads, PrepSmem<T, KP>::bytes, s, p);
}

}  // namespace

int ssh::delta_prep(const Delta& p, int dtype, cudaStream_t s) {
  if (dtype == SS_F32) return p.a.K <= 64 ? prep<float, 64>(p, s) : prep<float, 128>(p, s);
  return p.a.K <= 64 ? prep<__nv_bfloat16, 64>(p, s) : prep<__nv_bfloat16, 128>(p, s);
}
