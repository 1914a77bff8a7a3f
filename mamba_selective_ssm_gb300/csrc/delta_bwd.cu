// The gated delta rule's backward (deltarule_bwd) for sm_103a: its plan, and its kernels for fp32 (bf16: delta_back_tc.cu,
// delta_grad_tc.cu).
//
// With U the gradient of the state leaving a chunk (dS1) and every formula in the scaled tokens of delta_common.cuh:
//   du0 = scale P^T do + e^{c_last - c} K dS1      du = du0 - M^T (beta du0)      dv = dR = beta du      dbeta = <du, r>
//   dS0 = e^{c_last} dS1 + scale (e^c Q)^T do - (e^c K)^T dR                               (the chain from chunk to chunk)
//   dq = scale (e^c do S0^T + E K),   E_ts = D_ts do_t.u_s
//   dk = -e^c dR S0^T + e^{c_last - c} u dS1^T + scale E^T Q - (F + F^T) K,   F_ts = D_ts dR_t.u_s (s < t)
// A log decay multiplies whatever crosses it: what tokens from t on read of the state (a) and of writes before t (X), what writes
// before t leave to the end (b), and the state that passes through:
//   dg_t = sum_{i >= t} a_i + sum_{s < t <= i} X_is + sum_{s < t} b_s + e^{c_last} <S0, dS1>
//   a_i = scale e^{c_i} do_i.S0^T q_i - e^{c_i} dR_i.S0^T k_i      b_s = e^{c_last - c_s} u_s.dS1^T k_s      X_is = E_is q_i.k_s - F_is k_i.k_s
// Each of these terms carries e^{g_t}, so the sum is as good for a head that forgets as for one that remembers.  (The same
// sum is that of do_i.o_i - dv_i.v_i over i >= t and of <S1, dS1>, in which every token's own write cancels: 3e-6 of dg was lost at
// g = -1, all of it at -14.)  do.S0^T q is the forward's; the other products with q and k are taken of the parts of dk.
#include <stddef.h>

#include "delta_common.cuh"

namespace {

using namespace ssk;

// ---------------------------------------------------------------- the chain
// As in the forward, a warp carries 16 columns of dS, transposed, from the last chunk to the first.  It leaves dS1 and du of
// every chunk ([V][K] and [V][64], fp32) and dv.  8 x 2048 tokens of 24 heads of 64 x 64: 348 us.
template <int KP>
struct BackStage {
  static constexpr int k = 0, q = k + DTile<KP, 2>::bytes, m = q + DTile<KP, 2>::bytes, p = m + kDMBytes,
                       vec = p + DTile<kDC, 2>::bytes, up = vec + kDVec * 4, slices = up + 2 * kDC * 4;
  static int bytes(int warps) { return slices + warps * DSlice::bytes; }
};

constexpr int kWalkThreads = 256;

template <int KP>
__global__ void __launch_bounds__(kWalkThreads) delta_bwd_kernel(Delta p, const float* __restrict__ dout, const float* __restrict__ dh_last,
                                                                 float* __restrict__ dv, float* __restrict__ dS, float* __restrict__ du,
                                                                 float* __restrict__ dh0, int stages, int stage_bytes) {
  using St = BackStage<KP>;
  constexpr int N = 2, KT = KP / 8;
  extern __shared__ __align__(128) unsigned char raw[];
  const uint32_t sb = smem_u32(raw);
  const LinAttn& a = p.a;
  const int tid = threadIdx.x, nt = blockDim.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t2 = 2 * (lane & 3);
  const int nvt = (a.V + nt / 2 - 1) / (nt / 2);
  const int vt = (int)(blockIdx.x % nvt);
  const long long bh = blockIdx.x / nvt;
  const int h = (int)(bh % a.H), b = (int)(bh / a.H), gh = h / (a.H / a.G);
  const int v0 = vt * (nt / 2) + warp * 16, vw = a.V - v0;
  const int len = a.len(b), nck = (len + kDC - 1) / kDC;
  const float* q = static_cast<const float*>(a.q) + (long long)b * a.L * a.ldq + (long long)gh * a.K;
  const float* k = static_cast<const float*>(a.k) + (long long)b * a.L * a.ldk + (long long)gh * a.K;
  const long long ldo = (long long)a.H * a.V;
  const long long row0 = ((long long)b * a.L * a.H + h) * a.V + v0;

  auto fetch = [&](int ck) {
    const uint32_t at = sb + (stages == 2 ? (ck & 1) * stage_bytes : 0);
    const long long t0 = (long long)ck * kDC;
    const int valid = len - (int)t0 < kDC ? len - (int)t0 : kDC;
    const long long item = bh * a.nck + ck;
    tile_load<float, KP>(at + St::k, k + t0 * a.ldk, a.ldk, valid, a.K, tid, nt);
    tile_load<float, KP>(at + St::q, q + t0 * a.ldq, a.ldq, valid, a.K, tid, nt);
    tile_copy(at + St::m, p.M + item * kDMBytes, kDMBytes, tid, nt);
    tile_copy(at + St::p, p.P + item * DTile<kDC, 2>::bytes, DTile<kDC, 2>::bytes, tid, nt);
    tile_copy(at + St::vec, reinterpret_cast<const unsigned char*>(p.vec + item * kDVec), kDVec * 4, tid, nt);
    DSlice::load(at + St::slices + warp * DSlice::bytes, dout + row0 + t0 * ldo, ldo, valid, vw, lane);
    cp_commit();
  };

  float U[KT][4];
#pragma unroll
  for (int j = 0; j < KT; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int kk = 8 * j + t2 + (e & 1), vv = g + (e >> 1) * 8;
      U[j][e] = dh_last != nullptr && kk < a.K && vv < vw ? dh_last[(bh * a.K + kk) * a.V + v0 + vv] : 0.f;
    }

  pdl_trigger();
  if (nck > 0) fetch(nck - 1);
  for (int ck = nck - 1; ck >= 0; --ck) {
    const uint32_t off = stages == 2 ? (uint32_t)((ck & 1) * stage_bytes) : 0u, at = sb + off;
    const float* vec = reinterpret_cast<const float*>(raw + off + St::vec);
    float* up = reinterpret_cast<float*>(raw + off + St::up);
    const uint32_t mine = at + St::slices + warp * DSlice::bytes;
    const long long item = bh * a.nck + ck;
    cp_wait<0>();
    __syncthreads();
    tile_scale<KP, true>(at + St::k, up, tid, nt);
    tile_scale<KP, false>(at + St::q, up + kDC, tid, nt);
    __syncthreads();
    if (stages == 2 && ck > 0) fetch(ck - 1);
#pragma unroll
    for (int j = 0; j < KT; ++j)
#pragma unroll
      for (int e = 0; e < 4; e += 2) {
        const int kk = 8 * j + t2, vv = g + (e >> 1) * 8;
        if (kk < a.K && vv < vw)
          *reinterpret_cast<float2*>(dS + (item * a.V + v0 + vv) * a.K + kk) = make_float2(U[j][e], U[j][e + 1]);
      }
    // du0^T = (rest K dS1)^T + scale do^T P
    float D[8][4];
    {
      const RowScale us = row_scale(U);
      float low[8][4];
      clear(D);
      clear(low);
#pragma unroll
      for (int kb = 0; kb < KP / 16; ++kb) {
        uint32_t hi[4], lo[4];
        left_terms(hi, lo, U[2 * kb], U[2 * kb + 1], us);
#pragma unroll
        for (int np = 0; np < 4; ++np) {
          uint32_t bb[N][4];
#pragma unroll
          for (int n = 0; n < N; ++n) right_rows<KP, N>(bb[n], at + St::k, np, kb, n, lane);
          mma_terms(D[2 * np], D[2 * np + 1], low[2 * np], low[2 * np + 1], hi, lo, bb[0], bb[N - 1]);
        }
      }
      fold(D, low);
#pragma unroll
      for (int n = 0; n < 8; ++n) {
        const float2 re = *reinterpret_cast<const float2*>(vec + kDC + 8 * n + t2);
        D[n][0] *= re.x * us.r[0].up;
        D[n][1] *= re.y * us.r[0].up;
        D[n][2] *= re.x * us.r[1].up;
        D[n][3] *= re.y * us.r[1].up;
      }
    }
    uint32_t hi[4][4], lo[4][4];
    {  // scale do^T P
      float x[8][4];
#pragma unroll
      for (int np = 0; np < 4; ++np) DSlice::read(mine, np, lane, x[2 * np], x[2 * np + 1]);
#pragma unroll
      for (int n = 0; n < 8; ++n) {
        const float2 qu = *reinterpret_cast<const float2*>(up + kDC + 8 * n + t2);
        x[n][0] *= qu.x;
        x[n][1] *= qu.y;
        x[n][2] *= qu.x;
        x[n][3] *= qu.y;
      }
      const RowScale xs = row_scale(x);
#pragma unroll
      for (int kb = 0; kb < 4; ++kb) {
        left_terms(hi[kb], lo[kb], x[2 * kb], x[2 * kb + 1], xs);
      }
#pragma unroll
      for (int np = 0; np < 4; ++np) {
        float c[2][4], d[2][4];
        clear(c);
        clear(d);
#pragma unroll
        for (int kb = np; kb < 4; ++kb) {  // tokens from this one on
          uint32_t b0[4], b1[4];
          right_cols<kDC, 2>(b0, at + St::p, np, kb, 0, lane);
          right_cols<kDC, 2>(b1, at + St::p, np, kb, 1, lane);
          mma_terms(c[0], c[1], d[0], d[1], hi[kb], lo[kb], b0, b1);
        }
        fold(c, d);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) D[2 * np + i][e] = fmaf(a.scale * xs.r[e >> 1].up, c[i][e], D[2 * np + i][e]);
      }
    }
    {  // du^T = du0^T - (beta du0)^T M
      float w[8][4];
#pragma unroll
      for (int n = 0; n < 8; ++n) {
        const int t = 8 * n + t2;
        const float2 em = *reinterpret_cast<const float2*>(vec + 3 * kDC + t), be = *reinterpret_cast<const float2*>(vec + 2 * kDC + t);
        w[n][0] = be.x * em.x * D[n][0];
        w[n][1] = be.y * em.y * D[n][1];
        w[n][2] = be.x * em.x * D[n][2];
        w[n][3] = be.y * em.y * D[n][3];
      }
      const RowScale ws = row_scale(w);
#pragma unroll
      for (int kb = 0; kb < 4; ++kb) left_terms(hi[kb], lo[kb], w[2 * kb], w[2 * kb + 1], ws);
#pragma unroll
      for (int np = 0; np < 4; ++np) {
        float c[2][4], d[2][4];
        clear(c);
        clear(d);
#pragma unroll
        for (int kb = np; kb < 4; ++kb) {
          uint32_t b0[4], b1[4];
          right_cols<kDC, 2>(b0, at + St::m, np, kb, 0, lane);
          right_cols<kDC, 2>(b1, at + St::m, np, kb, 1, lane);
          mma_terms(c[0], c[1], d[0], d[1], hi[kb], lo[kb], b0, b1);
        }
        fold(c, d);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) D[2 * np + i][e] = fmaf(-ws.r[e >> 1].up, c[i][e], D[2 * np + i][e]);
      }
    }
    const int t0 = ck * kDC, rows = a.L - t0 < kDC ? a.L - t0 : kDC;
#pragma unroll
    for (int n = 0; n < 8; ++n) {
      const int t = 8 * n + t2;
#pragma unroll
      for (int e = 0; e < 4; e += 2) {
        const int vv = g + (e >> 1) * 8;
        if (vv < vw) *reinterpret_cast<float2*>(du + (item * a.V + v0 + vv) * kDC + t) = make_float2(D[n][e], D[n][e + 1]);
      }
      const float2 be = *reinterpret_cast<const float2*>(vec + 2 * kDC + t), ku = *reinterpret_cast<const float2*>(up + t);
      const float d0 = __frcp_rn(ku.x), d1 = __frcp_rn(ku.y);
      D[n][0] *= be.x;
      D[n][1] *= be.y;
      D[n][2] *= be.x;
      D[n][3] *= be.y;
      const bool on0 = t0 + t < len, on1 = t0 + t + 1 < len;
      const float x[4] = {on0 ? D[n][0] * d0 : 0.f, on1 ? D[n][1] * d1 : 0.f, on0 ? D[n][2] * d0 : 0.f, on1 ? D[n][3] * d1 : 0.f};
      store_tokens(dv + row0 + (long long)t0 * ldo, ldo, 8 * n, rows, vw, x, lane);
    }
    {  // dS0^T = e^{c_last} dS1^T + (scale e^c do)^T Q - (e^c dR)^T K, the two left operands in one scale
      float x[8][4];
#pragma unroll
      for (int np = 0; np < 4; ++np) DSlice::read(mine, np, lane, x[2 * np], x[2 * np + 1]);
#pragma unroll
      for (int n = 0; n < 8; ++n) {
        const int t = 8 * n + t2;
        const float2 in = *reinterpret_cast<const float2*>(vec + t), qu = *reinterpret_cast<const float2*>(up + kDC + t);
        const float f0 = a.scale * in.x * qu.x, f1 = a.scale * in.y * qu.y;
        x[n][0] *= f0;
        x[n][1] *= f1;
        x[n][2] *= f0;
        x[n][3] *= f1;
        D[n][0] *= -in.x;
        D[n][1] *= -in.y;
        D[n][2] *= -in.x;
        D[n][3] *= -in.y;
      }
      RowScale xs = row_scale(x);
      const RowScale ds = row_scale(D);
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (ds.r[i].up > xs.r[i].up) xs.r[i] = ds.r[i];
      uint32_t dh[4][4], dl[4][4];
#pragma unroll
      for (int kb = 0; kb < 4; ++kb) {
        left_terms(hi[kb], lo[kb], x[2 * kb], x[2 * kb + 1], xs);
        left_terms(dh[kb], dl[kb], D[2 * kb], D[2 * kb + 1], xs);
      }
      const float whole = vec[4 * kDC];
#pragma unroll
      for (int jp = 0; jp < KP / 16; ++jp) {
        float c[2][4], d[2][4];
        clear(c);
        clear(d);
#pragma unroll
        for (int kb = 0; kb < 4; ++kb) {
          uint32_t bb[N][4];
#pragma unroll
          for (int n = 0; n < N; ++n) right_cols<KP, N>(bb[n], at + St::q, jp, kb, n, lane);
          mma_terms(c[0], c[1], d[0], d[1], hi[kb], lo[kb], bb[0], bb[N - 1]);
#pragma unroll
          for (int n = 0; n < N; ++n) right_cols<KP, N>(bb[n], at + St::k, jp, kb, n, lane);
          mma_terms(c[0], c[1], d[0], d[1], dh[kb], dl[kb], bb[0], bb[N - 1]);
        }
        fold(c, d);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) U[2 * jp + i][e] = fmaf(U[2 * jp + i][e], whole, c[i][e] * xs.r[e >> 1].up);
      }
    }
    if (stages == 1) {
      __syncthreads();
      if (ck > 0) fetch(ck - 1);
    }
  }
  if (dh0 != nullptr) {
#pragma unroll
    for (int j = 0; j < KT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int kk = 8 * j + t2 + (e & 1), vv = g + (e >> 1) * 8;
        if (kk < a.K && vv < vw) dh0[(bh * a.K + kk) * a.V + v0 + vv] = U[j][e];
      }
  }
  const int w = vw < 16 ? vw : 16;  // tokens of chunks past the row's end
  for (long long i = (long long)nck * kDC * 16 + lane; i < (long long)a.L * 16; i += 32)
    if ((int)(i & 15) < w) dv[row0 + (i >> 4) * ldo + (i & 15)] = 0.f;
}

// ---------------------------------------------------------------- the other gradients, chunk by chunk
// A CTA takes one (batch row, head, chunk).  First its warps take 16 columns of V each (with half of the tokens where V is 64
// and less): what they add to dg and dbeta, from r and the state's part of o (the forward's), du and do.  Then they share the
// products that contract over V, from tiles in shared memory scaled as a whole: u, dR, S0, dS1 lie [V][..].  8 x 2048 tokens of 24
// heads of 64 x 64: 495 us, with decays 600 (tensor pipe 22 %, memory a quarter of its rate: the steps between barriers, at two
// CTAs an SM).
template <int KP, int VP>
struct GradSmem {
  static constexpr int N = 2, tile = DTile<KP, N>::bytes;
  static constexpr int vk = VP * KP * 2 * N, vt = VP * kDC * 2 * N, tt = DTile<kDC, N>::bytes;
  static constexpr int doo = 0, u = doo + DTile<VP, N>::bytes, r = u + vt, k = r + vt, q = k + tile;
  // S0 and dS1 take turns, and where there is no room for one beside k and q these come a second time
  static constexpr bool turns = r + vt + 2 * tile + vk > 220 * 1024;
  static constexpr int st = turns ? k : q + tile, e = doo, f = e + tt;  // (E and F after do, u and dR)
  static constexpr int end = turns ? k + (2 * tile > vk ? 2 * tile : vk) : st + vk;
  static constexpr int vec = end, up = vec + kDVec * 4, red = up + 3 * kDC * 4, bytes = red + (2 * 8 * kDC + 64 + 2 * kDC) * 4;
  static constexpr int ctas = 2 * (bytes + 1024) <= 228 * 1024 ? 2 : 1;
  static_assert(f + tt <= r && vt >= kDC * kDC * 4, "E, F and X where do, u and dR were");
};

constexpr int kGradThreads = 256;

// 2^13 .. 2^14 for the largest of eight warps' maxima
__device__ __forceinline__ Pow2 warps_scale(const float* m, int stride) {
  float x = 0.f;
#pragma unroll
  for (int w = 0; w < 8; ++w) x = fmaxf(x, m[w * stride]);
  return operand_scale(x);
}
__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}
template <int NJ>
__device__ __forceinline__ float abs_max(const float (&x)[NJ][4]) {
  float m = 0.f;
#pragma unroll
  for (int j = 0; j < NJ; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) m = fmaxf(m, fabsf(x[j][e]));
  return warp_max(m);
}
// accumulators to a tile of rows of W columns: rows r0 + lane / 4 (+ 8), column tile j
template <int W>
__device__ __forceinline__ void store_acc(uint32_t tile, int r0, int j, const float (&x)[4], float f, int lane) {
#pragma unroll
  for (int e = 0; e < 4; e += 2) {
    const int r = r0 + (lane >> 2) + (e >> 1) * 8;
    uint32_t hi, lo;
    split_half(x[e] * f, x[e + 1] * f, hi, lo);
    asm volatile("st.shared.b32 [%0], %1;" ::"r"(tile + DTile<W, 2>::at(r, j, 0) + 4 * (lane & 3)), "r"(hi) : "memory");
    asm volatile("st.shared.b32 [%0], %1;" ::"r"(tile + DTile<W, 2>::at(r, j, 1) + 4 * (lane & 3)), "r"(lo) : "memory");
  }
}
// columns 2 (lane % 4) and the next of unit u of a row, from its two terms
template <int W>
__device__ __forceinline__ float2 tile_pair(uint32_t tile, int r, int u, int lane) {
  uint32_t hi, lo;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(hi) : "r"(tile + DTile<W, 2>::at(r, u, 0) + 4 * (lane & 3)) : "memory");
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(lo) : "r"(tile + DTile<W, 2>::at(r, u, 1) + 4 * (lane & 3)) : "memory");
  const float2 h = wide_half(hi), l = wide_half(lo);
  return make_float2(h.x + l.x, h.y + l.y);
}
template <int KP, int VP>
__global__ void __launch_bounds__(kGradThreads, (GradSmem<KP, VP>::ctas)) delta_grad_kernel(Delta p, const float* __restrict__ ckpt,
                                                                  const float* __restrict__ dout,
                                                                  const float* __restrict__ dS, const float* __restrict__ du,
                                                                  float* __restrict__ dq, float* __restrict__ dk, int heads,
                                                                  float* __restrict__ dg, float* __restrict__ dbeta) {
  using Sm = GradSmem<KP, VP>;
  constexpr int N = 2, VB = VP / 16, NC = KP / 16;  // NC: column tiles of a warp's half of K
  constexpr int NW = 8 / VB, KT = KP / 8 / NW, NT = 8 / NW;  // warps of 16 columns of V; a warp's tiles of K, of tokens
  extern __shared__ __align__(128) unsigned char raw[];
  const uint32_t sb = smem_u32(raw);
  const LinAttn& a = p.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t2 = 2 * (lane & 3);
  const long long item = blockIdx.x, bh = item / a.nck;
  const int ck = (int)(item % a.nck), h = (int)(bh % a.H), b = (int)(bh / a.H), gh = h / (a.H / a.G);
  const long long t0 = (long long)ck * kDC;
  const int len = a.len(b), rows = a.L - (int)t0 < kDC ? a.L - (int)t0 : kDC;
  const int valid = len - (int)t0 < 0 ? 0 : len - (int)t0 < kDC ? len - (int)t0 : kDC;
  const long long tok = (long long)b * a.L + t0;
  // rows of dq and dk: `heads` of them to a token (the groups', or every head's own part)
  const long long ldg = (long long)heads * a.K;
  float* dqb = dq + (tok * heads + (heads == a.G ? gh : h)) * a.K;
  float* dkb = dk + (tok * heads + (heads == a.G ? gh : h)) * a.K;
  if (valid == 0) {
    pdl_wait();
    for (int i = tid; i < rows * a.K; i += kGradThreads) {
      dqb[i / a.K * ldg + i % a.K] = 0.f;
      dkb[i / a.K * ldg + i % a.K] = 0.f;
    }
    if (tid < rows) {
      if (dg != nullptr) dg[(tok + tid) * a.H + h] = 0.f;
      dbeta[(tok + tid) * a.H + h] = 0.f;
    }
    return;
  }
  const float* q = static_cast<const float*>(a.q) + tok * a.ldq + (long long)gh * a.K;
  const float* k = static_cast<const float*>(a.k) + tok * a.ldk + (long long)gh * a.K;
  const long long ldo = (long long)a.H * a.V;
  const float* dob = dout + (tok * a.H + h) * a.V;
  float *vec = reinterpret_cast<float*>(raw + Sm::vec), *up = reinterpret_cast<float*>(raw + Sm::up), *red = reinterpret_cast<float*>(raw + Sm::red);
  float* mx = red + 2 * 8 * kDC;  // eight warps' maxima: S0, u, dR, dS1, E, F, and the state's product
  tile_load<float, KP>(sb + Sm::k, k, a.ldk, valid, a.K, tid, kGradThreads);
  tile_load<float, KP>(sb + Sm::q, q, a.ldq, valid, a.K, tid, kGradThreads);
  tile_load<float, VP>(sb + Sm::doo, dob, ldo, valid, a.V, tid, kGradThreads);
  tile_copy(sb + Sm::vec, reinterpret_cast<const unsigned char*>(p.vec + item * kDVec), kDVec * 4, tid, kGradThreads);
  cp_commit();
  float* cc = mx + 64;  // running log2 decays: D_ts = e^{c_t - c_s} from the scalars, e^{c_t} / e^{c_s}, would lose small ones
  if (warp == 7) {
    ChunkGates<kDC> gates;
    if (a.g != nullptr) gates.fetch(a, b, h, (int)t0, (int)t0 + valid, lane);
    else gates.g[0] = gates.g[1] = 0.f;
    gates.scan(lane, [&](int i, Dec e) { cc[i] = e.hi; cc[kDC + i] = e.lo; });
  }
  const int v0 = warp % VB * 16, part = warp / VB, vw = a.V - v0;  // this warp's columns, its part of the other axis
  // a [V][K] state in the order of accumulators
  auto state = [&](const float* src, float (&x)[KT][4]) {
#pragma unroll
    for (int j = 0; j < KT; ++j)
#pragma unroll
      for (int e = 0; e < 4; e += 2) {
        const int kk = 8 * (part * KT + j) + t2, vv = g + (e >> 1) * 8;
        float2 y = make_float2(0.f, 0.f);
        if (kk < a.K && vv < vw) y = *reinterpret_cast<const float2*>(src + (long long)(v0 + vv) * a.K + kk);
        x[j][e] = y.x;
        x[j][e + 1] = y.y;
      }
  };
  // [V][64] values, and rows of do
  auto tokens = [&](const float* src, float (&x)[NT][4]) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; e += 2) {
        const int t = 8 * (part * NT + n) + t2, vv = g + (e >> 1) * 8;
        float2 y = make_float2(0.f, 0.f);
        if (vv < vw) y = *reinterpret_cast<const float2*>(src + (long long)(v0 + vv) * kDC + t);
        x[n][e] = y.x;
        x[n][e + 1] = y.y;
      }
  };
  auto rows_of = [&](const float* src, long long ld, float (&x)[NT][4]) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int t = 8 * (part * NT + n) + t2 + (e & 1), vv = g + (e >> 1) * 8;
        x[n][e] = t < valid && vv < vw ? src[(long long)t * ld + v0 + vv] : 0.f;
      }
  };
  pdl_wait();  // dS and du are delta_bwd_kernel's
  const float* base = ckpt + bh * delta_ckpt_floats(a.nck, a.K, a.V);
  const float* s0 = base + (long long)ck * a.K * a.V;
  const float* ro = base + (long long)(a.nck + 1) * a.K * a.V + (long long)ck * kDC * a.V;
  float R[NT][4], D[NT][4];  // r, then u; du, then dR
  float db[2 * NT], af[2 * NT];
  tokens(ro, R);
  tokens(du + item * kDC * a.V, D);
  {
    float x[NT][4], o[NT][4];
    rows_of(dob, ldo, x);
    tokens(ro + (long long)a.nck * kDC * a.V, o);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int t = 8 * (part * NT + n) + t2;
      af[2 * n] = t < valid ? fmaf(x[n][0], o[n][0], x[n][2] * o[n][2]) : 0.f;
      af[2 * n + 1] = t + 1 < valid ? fmaf(x[n][1], o[n][1], x[n][3] * o[n][3]) : 0.f;
    }
  }
  cp_wait<0>();
  __syncthreads();
  tile_scale<KP, true>(sb + Sm::k, up, tid, kGradThreads);
  tile_scale<KP, false>(sb + Sm::q, up + kDC, tid, kGradThreads);
  tile_scale<VP, false>(sb + Sm::doo, up + 2 * kDC, tid, kGradThreads);
  __syncthreads();
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int t = 8 * (part * NT + n) + t2;
    const float2 be = *reinterpret_cast<const float2*>(vec + 2 * kDC + t);
    db[2 * n] = fmaf(D[n][0], R[n][0], D[n][2] * R[n][2]);
    db[2 * n + 1] = fmaf(D[n][1], R[n][1], D[n][3] * R[n][3]);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      R[n][e] *= e & 1 ? be.y : be.x;
      D[n][e] *= e & 1 ? be.y : be.x;
    }
  }
#pragma unroll
  for (int i = 0; i < 2 * NT; ++i) {
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      db[i] += __shfl_xor_sync(0xffffffffu, db[i], o);
      af[i] += __shfl_xor_sync(0xffffffffu, af[i], o);
    }
    if (g == 0) {
      const int t = 8 * (part * NT + (i >> 1)) + t2 + (i & 1);
      red[warp % VB * kDC + t] = db[i];
      red[(8 + warp % VB) * kDC + t] = af[i];
    }
  }
  // dS1: its largest and <S0, dS1>; S0
  float S[KT][4];
  float dot = 0.f;
  state(dS + item * a.V * a.K, S);
  {
#pragma unroll
    for (int j = 0; j < KT; ++j)
#pragma unroll
      for (int e = 0; e < 4; e += 2) {
        const int kk = 8 * (part * KT + j) + t2, vv = g + (e >> 1) * 8;
        if (kk < a.K && vv < vw) {
          const float2 y = *reinterpret_cast<const float2*>(s0 + (long long)(v0 + vv) * a.K + kk);
          dot = fmaf(y.x, S[j][e], fmaf(y.y, S[j][e + 1], dot));
        }
      }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
  }
  {
    const float mt = abs_max(S);
    state(s0, S);
    const float ms = abs_max(S), mu = abs_max(R), md = abs_max(D);
    if (lane == 0) {
      mx[warp * 8] = ms;
      mx[warp * 8 + 1] = mu;
      mx[warp * 8 + 2] = md;
      mx[warp * 8 + 3] = mt;
      mx[warp * 8 + 6] = dot;
    }
  }
  __syncthreads();
  const Pow2 scS = warps_scale(mx, 8), scU = warps_scale(mx + 1, 8), scR = warps_scale(mx + 2, 8), scT = warps_scale(mx + 3, 8);
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    store_acc<kDC>(sb + Sm::u, v0, part * NT + n, R[n], scU.down, lane);
    store_acc<kDC>(sb + Sm::r, v0, part * NT + n, D[n], scR.down, lane);
  }
  auto put_state = [&](float f) {
#pragma unroll
    for (int j = 0; j < KT; ++j) store_acc<KP>(sb + Sm::st, v0, part * KT + j, S[j], f, lane);
  };
  if (!Sm::turns) put_state(scS.down);
  if (warp == 0) {  // dbeta, and a's part of q
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int t = 2 * lane + i;
      float s = 0.f, d = 0.f;
      for (int w = 0; w < VB; ++w) {
        d += red[w * kDC + t];
        s += red[(8 + w) * kDC + t];
      }
      if (t < rows) dbeta[(tok + t) * a.H + h] = t < valid ? d * up[t] * up[t] : 0.f;
      red[8 * kDC + t] = s;
    }
  }
  // E and F, a warp's 16 tokens t against half of the tokens s
  const int mb = warp & 3, half = warp >> 2, vb = (a.V + 15) / 16;
  float E[4][4], F[4][4], Xr[4][4];
  __syncthreads();  // u and dR
  {
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) E[n][e] = F[n][e] = 0.f;
#pragma unroll
    for (int np = 0; np < 2; ++np) {
      if (2 * half + np > mb) continue;
      float el[2][4], fl[2][4];
      clear(el);
      clear(fl);
      for (int kb = 0; kb < vb; ++kb) {
        uint32_t ea[N][4], fa[N][4], bb[N][4];
#pragma unroll
        for (int n = 0; n < N; ++n) {
          left_rows<VP, N>(ea[n], sb + Sm::doo, mb, kb, n, lane);
          left_cols<kDC, N>(fa[n], sb + Sm::r, mb, kb, n, lane);
          right_cols<kDC, N>(bb[n], sb + Sm::u, 2 * half + np, kb, n, lane);
        }
        mma_terms(E[2 * np], E[2 * np + 1], el[0], el[1], ea[0], ea[1], bb[0], bb[1]);
        mma_terms(F[2 * np], F[2 * np + 1], fl[0], fl[1], fa[0], fa[1], bb[0], bb[1]);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          E[2 * np + i][e] += el[i][e];
          F[2 * np + i][e] += fl[i][e];
        }
    }
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int t = 16 * mb + g + (e >> 1) * 8, s = 32 * half + 8 * n + t2 + (e & 1);
        const float d = s <= t ? dec_diff(cc[t], cc[kDC + t], cc[s], cc[kDC + s]) : 0.f;
        E[n][e] = s <= t ? a.scale * up[kDC + t] * up[2 * kDC + t] * scU.up * d * E[n][e] : 0.f;
        F[n][e] = s < t ? -scR.up * scU.up * d * F[n][e] : 0.f;
      }
    // X: its values wait here for the place of dR (and are made of these, not of E's and F's tiles: in those a token's own values
    // set the scale, and what a strong decay left is lost)
    if (dg != nullptr) {
#pragma unroll
      for (int np = 0; np < 2; ++np) {
        float qk[2][4], kk[2][4], ql[2][4], kl[2][4];
        clear(qk);
        clear(kk);
        clear(ql);
        clear(kl);
        if (2 * half + np <= mb)
#pragma unroll 1
          for (int kb = 0; kb < KP / 16; ++kb) {
            uint32_t qa[N][4], ka[N][4], bb[N][4];
#pragma unroll
            for (int n = 0; n < N; ++n) {
              left_rows<KP, N>(qa[n], sb + Sm::q, mb, kb, n, lane);
              left_rows<KP, N>(ka[n], sb + Sm::k, mb, kb, n, lane);
              right_rows<KP, N>(bb[n], sb + Sm::k, 2 * half + np, kb, n, lane);
            }
            mma_terms(qk[0], qk[1], ql[0], ql[1], qa[0], qa[1], bb[0], bb[1]);
            mma_terms(kk[0], kk[1], kl[0], kl[1], ka[0], ka[1], bb[0], bb[1]);
          }
        fold(qk, ql);
        fold(kk, kl);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int n = 2 * np + i, t = 16 * mb + g + (e >> 1) * 8, s = 32 * half + 8 * n + t2 + (e & 1);
            Xr[n][e] = s < t ? fmaf(E[n][e], qk[i][e], F[n][e] * kk[i][e]) : 0.f;
          }
      }
    }
    const float me = abs_max(E), mf = abs_max(F);
    if (lane == 0) {
      mx[warp * 8 + 4] = me;
      mx[warp * 8 + 5] = mf;
    }
  }
  // dq and dk: a warp's 16 tokens and half of the columns of K
  float Q[NC][4], Kg[NC][4], C[NC][4], Cl[NC][4];
  const int ta = 16 * mb + g, tb = ta + 8;
  auto zero = [&] {
    clear(C);
    clear(Cl);
  };
  auto add = [&](float (&to)[NC][4], float fa, float fb, bool first) {
    fold(C, Cl);
#pragma unroll
    for (int j = 0; j < NC; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) to[j][e] = fmaf(e < 2 ? fa : fb, C[j][e], first ? 0.f : to[j][e]);
  };
  // red[row + half][t] = f C.k of this warp's tokens, over its columns of K, in the tokens' scale
  auto meet = [&](int row, float fa, float fb) {
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int t = i == 0 ? ta : tb;
      const float* kt = k + (long long)(t < valid ? t : 0) * a.ldk;
#pragma unroll
      for (int j = 0; j < NC; ++j) {
        const int c = half * (KP / 2) + 8 * j + t2;
        if (c >= a.K) continue;
        float2 y;
        if constexpr (Sm::turns) y = *reinterpret_cast<const float2*>(kt + c);  // (a state is where k was)
        else y = tile_pair<KP>(sb + Sm::k, t, half * (KP / 16) + j, lane);
        s[i] = fmaf(C[j][2 * i], y.x, fmaf(C[j][2 * i + 1], y.y, s[i]));
      }
      s[i] *= (i == 0 ? fa : fb) * (Sm::turns ? __frcp_rn(up[t]) : 1.f);
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) s[i] += __shfl_xor_sync(0xffffffffu, s[i], o);
      if ((lane & 3) == 0) red[(row + half) * kDC + t] = t < valid ? s[i] : 0.f;
    }
  };
  // C += (left operand at step kb) x (the tile's rows 16 kb .., this warp's columns)
  auto step = [&](uint32_t tile, int kb, const uint32_t (&la)[N][4]) {
#pragma unroll
    for (int jp = 0; jp < NC / 2; ++jp) {
      uint32_t bb[N][4];
#pragma unroll
      for (int n = 0; n < N; ++n) right_cols<KP, N>(bb[n], tile, half * (NC / 2) + jp, kb, n, lane);
      mma_terms(C[2 * jp], C[2 * jp + 1], Cl[2 * jp], Cl[2 * jp + 1], la[0], la[1], bb[0], bb[1]);
    }
  };
  if constexpr (Sm::turns) {
    __syncthreads();  // (k and q have been read by tile_scale and for X)
    put_state(scS.down);
    __syncthreads();
  }
  zero();
  for (int kb = 0; kb < vb; ++kb) {
    uint32_t la[N][4];
#pragma unroll
    for (int n = 0; n < N; ++n) left_rows<VP, N>(la[n], sb + Sm::doo, mb, kb, n, lane);
    step(sb + Sm::st, kb, la);
  }
  const float fs = a.scale * scS.up;
  add(Q, fs * vec[ta] * up[2 * kDC + ta], fs * vec[tb] * up[2 * kDC + tb], true);
  zero();
  for (int kb = 0; kb < vb; ++kb) {
    uint32_t la[N][4];
#pragma unroll
    for (int n = 0; n < N; ++n) left_cols<kDC, N>(la[n], sb + Sm::r, mb, kb, n, lane);
    step(sb + Sm::st, kb, la);
  }
  add(Kg, -vec[ta] * scR.up * scS.up, -vec[tb] * scR.up * scS.up, true);
  if (dg != nullptr) meet(0, -vec[ta] * scR.up * scS.up, -vec[tb] * scR.up * scS.up);
  state(dS + item * a.V * a.K, S);
  __syncthreads();
  put_state(scT.down);
  __syncthreads();
  zero();
  for (int kb = 0; kb < vb; ++kb) {
    uint32_t la[N][4];
#pragma unroll
    for (int n = 0; n < N; ++n) left_cols<kDC, N>(la[n], sb + Sm::u, mb, kb, n, lane);
    step(sb + Sm::st, kb, la);
  }
  add(Kg, vec[kDC + ta] * scU.up * scT.up, vec[kDC + tb] * scU.up * scT.up, false);
  if (dg != nullptr) meet(2, vec[kDC + ta] * scU.up * scT.up, vec[kDC + tb] * scU.up * scT.up);
  __syncthreads();  // do, u, dR and dS1 have been read
  if constexpr (Sm::turns) {
    tile_load<float, KP>(sb + Sm::k, k, a.ldk, valid, a.K, tid, kGradThreads);
    tile_load<float, KP>(sb + Sm::q, q, a.ldq, valid, a.K, tid, kGradThreads);
    cp_commit();
  }
  const Pow2 scE = warps_scale(mx + 4, 8), scF = warps_scale(mx + 5, 8);
#pragma unroll
  for (int n = 0; n < 4; ++n) {
    store_acc<kDC>(sb + Sm::e, 16 * mb, 4 * half + n, E[n], scE.down, lane);
    store_acc<kDC>(sb + Sm::f, 16 * mb, 4 * half + n, F[n], scF.down, lane);
  }
  // X, whose sums over s < t <= i follow between the products
  float* X = reinterpret_cast<float*>(raw + Sm::r);  // [t][s], s's eights turned by t (banks)
  auto xat = [](int t, int s) { return t * kDC + (s ^ ((t & 7) << 3)); };
#pragma unroll
  for (int n = 0; n < 4; ++n)
#pragma unroll
    for (int e = 0; e < 4; e += 2)
      if (dg != nullptr) *reinterpret_cast<float2*>(X + xat(e == 0 ? ta : tb, 32 * half + 8 * n + t2)) = make_float2(Xr[n][e], Xr[n][e + 1]);
  if constexpr (Sm::turns) {
    cp_wait<0>();
    __syncthreads();
    tile_scale<KP, true>(sb + Sm::k, up, tid, kGradThreads);
    tile_scale<KP, false>(sb + Sm::q, up + kDC, tid, kGradThreads);
  }
  __syncthreads();
  if (dg != nullptr) {
    float run = 0.f;  // X[t][s] becomes its sum over the tokens from t to the end of t's 16
#pragma unroll
    for (int t = 15; t >= 0; --t) {
      float* at = X + xat(16 * (tid >> 6) + t, tid & 63);
      run += *at;
      *at = run;
    }
  }
  zero();
#pragma unroll
  for (int kb = 0; kb < 4; ++kb) {
    uint32_t la[N][4];
    if (kb > mb) continue;
#pragma unroll
    for (int n = 0; n < N; ++n) left_rows<kDC, N>(la[n], sb + Sm::e, mb, kb, n, lane);
    step(sb + Sm::k, kb, la);
  }
  add(Q, scE.up * __frcp_rn(up[kDC + ta]), scE.up * __frcp_rn(up[kDC + tb]), false);
  if (dg != nullptr) {
    __syncthreads();
    const int j = tid >> 2;
    float s = 0.f;
#pragma unroll 1
    for (int c = tid & 3; c < j; c += 4) {
      s += X[xat(j, c)];
#pragma unroll 1
      for (int later = (j >> 4) + 1; later < 4; ++later) s += X[xat(16 * later, c)];
    }
    s += __shfl_xor_sync(0xffffffffu, s, 1);
    s += __shfl_xor_sync(0xffffffffu, s, 2);
    if ((tid & 3) == 0) red[9 * kDC + j] = s;
  }
  zero();
#pragma unroll
  for (int kb = 0; kb < 4; ++kb) {
    uint32_t la[N][4];
    if (kb < mb) continue;
#pragma unroll
    for (int n = 0; n < N; ++n) left_cols<kDC, N>(la[n], sb + Sm::e, mb, kb, n, lane);
    step(sb + Sm::q, kb, la);
  }
  add(Kg, scE.up, scE.up, false);
  if (dg != nullptr) {
    __syncthreads();
    if (warp == 0) {
      float x = 0.f, after[2], before[2];
      for (int w = 0; w < 8; ++w) x += mx[w * 8 + 6];
      x *= vec[4 * kDC];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int t = 2 * lane + i;
        after[i] = red[8 * kDC + t] + (red[t] + red[kDC + t]);
        before[i] = red[2 * kDC + t] + red[3 * kDC + t];
      }
      float from = after[0] + after[1], upto = before[0] + before[1];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const float y = __shfl_down_sync(0xffffffffu, from, o), z = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane + o < 32) from += y;
        if (lane >= o) upto += z;
      }
      float rest = __shfl_down_sync(0xffffffffu, from, 1), past = __shfl_up_sync(0xffffffffu, upto, 1);
      if (lane == 31) rest = 0.f;
      if (lane == 0) past = 0.f;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int t = 2 * lane + i;
        const float y = ((i == 0 ? from : after[1] + rest) + (i == 0 ? past : past + before[0])) + (x + red[9 * kDC + t]);
        if (t < rows) dg[(tok + t) * a.H + h] = t < valid ? y : 0.f;
      }
    }
  }
  zero();
#pragma unroll
  for (int kb = 0; kb < 4; ++kb) {
    uint32_t la[N][4];
    if (kb <= mb) {
#pragma unroll
      for (int n = 0; n < N; ++n) left_rows<kDC, N>(la[n], sb + Sm::f, mb, kb, n, lane);
      step(sb + Sm::k, kb, la);
    }
    if (kb >= mb) {
#pragma unroll
      for (int n = 0; n < N; ++n) left_cols<kDC, N>(la[n], sb + Sm::f, mb, kb, n, lane);
      step(sb + Sm::k, kb, la);
    }
  }
  add(Kg, scF.up, scF.up, false);
#pragma unroll
  for (int e = 0; e < 4; e += 2) {
    const int t = e == 0 ? ta : tb;
    if (t >= rows) continue;
    const float f = __frcp_rn(up[t]);
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      const int c = half * (KP / 2) + 8 * j + t2;
      if (c >= a.K) continue;
      const bool on = t < valid;
      *reinterpret_cast<float2*>(dqb + (long long)t * ldg + c) = on ? make_float2(Q[j][e], Q[j][e + 1]) : make_float2(0.f, 0.f);
      *reinterpret_cast<float2*>(dkb + (long long)t * ldg + c) = on ? make_float2(Kg[j][e] * f, Kg[j][e + 1] * f) : make_float2(0.f, 0.f);
    }
  }
}

// dq and dk of a group from its heads' parts, added in order: [tokens, G, R, K] -> [tokens, G, K], four columns a thread
template <typename T>
__global__ void __launch_bounds__(256) delta_share_kernel(const float* __restrict__ pq, const float* __restrict__ pk, T* __restrict__ dq,
                                                          T* __restrict__ dk, long long n4, int R, int K) {
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  if (i >= n4) return;
  const float* src = (blockIdx.y == 0 ? pq : pk) + i * 4 / K * R * K + i * 4 % K;
  T* dst = (blockIdx.y == 0 ? dq : dk) + i * 4;
  float4 s = *reinterpret_cast<const float4*>(src);
  for (int r = 1; r < R; ++r) {
    const float4 x = *reinterpret_cast<const float4*>(src + (long long)r * K);
    s.x += x.x; s.y += x.y; s.z += x.z; s.w += x.w;
  }
  ActT<T>::st2(dst, s.x, s.y);
  ActT<T>::st2(dst + 2, s.z, s.w);
}

struct BwdPlan {
  Delta p;
  size_t ds, du, part, bytes;
};

int bwd_plan(int B, int L, int H, int G, int K, int V, int dtype, BwdPlan& pl) {
  const int rc = delta_validate(B, L, H, G, K, V, dtype);
  if (rc != SS_OK) return rc;
  pl.p = Delta{};
  LinAttn& a = pl.p.a;
  a.B = B; a.L = L; a.H = H; a.G = G; a.K = K; a.V = V;
  a.nck = (L + kDC - 1) / kDC;
  const size_t items = pl.p.items();
  pl.ds = items * K * V * sizeof(float);
  pl.du = items * kDC * V * sizeof(float);
  pl.part = H > G ? (size_t)B * L * H * K * sizeof(float) : 0;
  pl.bytes = pl.ds + pl.du + 2 * pl.part;
  return SS_OK;
}

struct BwdArgs {
  const float *ckpt, *dh_last;
  const void* dout;
  void *dq, *dk, *dv;
  float *dg, *dbeta, *dh0, *dS, *du, *pq, *pk;
};

template <int KP>
int chain(const BwdPlan& pl, const BwdArgs& x, cudaStream_t s) {
  using St = BackStage<KP>;
  const LinAttn& a = pl.p.a;
  const long long bh = (long long)a.B * a.H;
  int warps = (a.V + 15) / 16;
  while (warps > 1 && bh * ((a.V + 16 * warps - 1) / (16 * warps)) < 100) warps = (warps + 1) / 2;
  const int nvt = (a.V + 16 * warps - 1) / (16 * warps);
  // as in the forward (192 heads of 64 x 64: 334 us for 445)
  const int sb = St::bytes(warps), stages = 2 * sb <= 226 * 1024 && bh * nvt <= 152 ? 2 : 1;
  return delta_launch(delta_bwd_kernel<KP>, (unsigned)(bh * nvt), 32 * warps, (size_t)sb * stages, s, pl.p, static_cast<const float*>(x.dout),
                    x.dh_last, static_cast<float*>(x.dv), x.dS, x.du, x.dh0, stages, sb);
}

// a group's dq and dk from its heads' parts
template <typename T>
int share(const BwdPlan& pl, const BwdArgs& x, cudaStream_t s) {
  const LinAttn& a = pl.p.a;
  const long long n4 = (long long)a.B * a.L * a.G * a.K / 4;
  delta_share_kernel<T><<<dim3((unsigned)((n4 + 255) / 256), 2), 256, 0, s>>>(x.pq, x.pk, static_cast<T*>(x.dq), static_cast<T*>(x.dk), n4,
                                                                              a.H / a.G, a.K);
  return cudaGetLastError() == cudaSuccess ? SS_OK : SS_ERR_CUDA;
}

template <int KP, int VP>
int grads(const BwdPlan& pl, const BwdArgs& x, cudaStream_t s) {
  const LinAttn& a = pl.p.a;
  const unsigned grid = (unsigned)((long long)a.B * a.H * a.nck);
  constexpr size_t smem = GradSmem<KP, VP>::bytes;
  static_assert(smem <= 227 * 1024, "a chunk's tiles fit shared memory");
  const bool parts = a.H > a.G;
  const int rc = delta_launch_next(delta_grad_kernel<KP, VP>, grid, kGradThreads, smem, s, pl.p, x.ckpt, static_cast<const float*>(x.dout), x.dS,
                            x.du,
                            parts ? x.pq : static_cast<float*>(x.dq), parts ? x.pk : static_cast<float*>(x.dk), parts ? a.H : a.G, x.dg, x.dbeta);
  return rc != SS_OK || !parts ? rc : share<float>(pl, x, s);
}

template <int KP>
int run(const BwdPlan& pl, const BwdArgs& x, cudaStream_t s) {
  const int rc = chain<KP>(pl, x, s);
  if (rc != SS_OK) return rc;
  return pl.p.a.V <= 64 ? grads<KP, 64>(pl, x, s) : grads<KP, 128>(pl, x, s);
}

int run_bf16(const BwdPlan& pl, const BwdArgs& x, cudaStream_t s) {
  int rc = ssh::delta_back_bf16(pl.p, x.dout, x.dh_last, x.dv, x.dS, x.du, x.dh0, s);
  if (rc != SS_OK) return rc;
  const bool parts = pl.p.a.H > pl.p.a.G;
  rc = ssh::delta_grad_bf16(pl.p, x.ckpt, x.dout, x.dS, x.du, parts ? x.pq : x.dq, parts ? x.pk : x.dk, parts, x.dg, x.dbeta, s);
  return rc != SS_OK || !parts ? rc : share<__nv_bfloat16>(pl, x, s);
}

}  // namespace

extern "C" size_t deltarule_bwd_workspace_size(int B, int L, int H, int G, int K, int V, int dtype) {
  BwdPlan pl;
  return bwd_plan(B, L, H, G, K, V, dtype, pl) == SS_OK ? pl.bytes : 0;
}

extern "C" int deltarule_bwd(const void* q, long long ldq, const void* k, long long ldk, const void* v, long long ldv, const float* g,
                             const float* beta, const int* lengths, const float* ckpt, const void* dout, const float* dh_last, void* dq,
                             void* dk, void* dv, float* dg, float* dbeta, float* dh0, int B, int L, int H, int G, int K, int V, float scale,
                             int dtype, void* workspace, size_t ws_bytes, void* stream) {
  if (!q || !k || !v || !beta || !ckpt || !dout || !dq || !dk || !dv || !dbeta || (g && !dg)) return SS_ERR_NULL;
  BwdPlan pl;
  int rc = bwd_plan(B, L, H, G, K, V, dtype, pl);
  if (rc != SS_OK) return rc;
  if ((rc = linattn_ld_ok(ldq, G, K)) != SS_OK || (rc = linattn_ld_ok(ldk, G, K)) != SS_OK || (rc = linattn_ld_ok(ldv, H, V)) != SS_OK)
    return rc;
  const void* ptrs[] = {q, k, v, ckpt, dout, dh_last, dq, dk, dv, dh0};
  for (const void* x : ptrs)
    if (x != nullptr && !ssh::aligned16(x)) return SS_ERR_ALIGN;
  const void* words[] = {g, beta, lengths, dg, dbeta};
  for (const void* x : words)
    if (reinterpret_cast<uintptr_t>(x) & 3u) return SS_ERR_ALIGN;
  if (workspace == nullptr || ws_bytes < pl.bytes) return SS_ERR_WORKSPACE;
  if (!ssh::aligned16(workspace)) return SS_ERR_ALIGN;
  LinAttn& a = pl.p.a;
  a.q = q; a.k = k; a.v = v;
  a.ldq = ldq; a.ldk = ldk; a.ldv = ldv;
  a.g = g;
  a.lengths = lengths;
  a.scale = scale;
  pl.p.beta = beta;
  char* w = static_cast<char*>(workspace);
  BwdArgs x{ckpt, dh_last, dout, dq, dk, dv, g ? dg : nullptr, dbeta, dh0, nullptr, nullptr, nullptr, nullptr};
  pl.p.place(const_cast<float*>(ckpt) + (long long)B * H * delta_ckpt_floats(a.nck, K, V), dtype == SS_BF16);  // (only read)
  x.dS = reinterpret_cast<float*>(w);
  x.du = reinterpret_cast<float*>(w += pl.ds);
  x.pq = reinterpret_cast<float*>(w += pl.du);
  x.pk = reinterpret_cast<float*>(w += pl.part);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dtype == SS_BF16) return run_bf16(pl, x, s);
  return K <= 64 ? run<64>(pl, x, s) : run<128>(pl, x, s);
}
