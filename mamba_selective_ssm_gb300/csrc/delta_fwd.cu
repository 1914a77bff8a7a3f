// The gated delta rule, chunked forward (deltarule_fwd) for sm_103a: its plan, and the chain for fp32 (bf16: delta_fwd_tc.cu).
#include <stddef.h>

#include "delta_common.cuh"

namespace {

using namespace ssk;

// A warp walks the chunks of one (batch row, head) with 16 columns of the state in registers, transposed: rows are columns
// of V, so that K S0, M (beta R), K^T u and o are products whose left operand is the accumulators of the one before, and the
// warps of a CTA share nothing but the tiles of the chunk (k, q, M, P).  8 x 2048 tokens of 24 heads of 64 x 64: 378 us with r,
// the state's part of o and the states for the backward; the chain's latency bounds it at four warps a CTA (tensor pipe 18 %, issue slots 26 %).
template <int KP>
struct WalkStage {
  static constexpr int k = 0, q = k + DTile<KP, 2>::bytes, m = q + DTile<KP, 2>::bytes, p = m + kDMBytes,
                       vec = p + DTile<kDC, 2>::bytes, up = vec + kDVec * 4, slices = up + 2 * kDC * 4;
  static int bytes(int warps) { return slices + warps * DSlice::bytes; }
};

constexpr int kWalkThreads = 256;

template <int KP>
__global__ void __launch_bounds__(kWalkThreads) delta_fwd_kernel(Delta p, const float* __restrict__ h0, float* __restrict__ o,
                                                                 float* __restrict__ ckpt, float* __restrict__ h_last, int stages,
                                                                 int stage_bytes) {
  using St = WalkStage<KP>;
  constexpr int N = 2, KT = KP / 8;
  extern __shared__ __align__(128) unsigned char raw[];
  const uint32_t sb = smem_u32(raw);
  const LinAttn& a = p.a;
  const int tid = threadIdx.x, nt = blockDim.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t2 = 2 * (lane & 3);
  const int nvt = (a.V + nt / 2 - 1) / (nt / 2);  // CTAs of a head: 16 columns a warp
  const int vt = (int)(blockIdx.x % nvt);
  const long long bh = blockIdx.x / nvt;
  const int h = (int)(bh % a.H), b = (int)(bh / a.H), gh = h / (a.H / a.G);
  const int v0 = vt * (nt / 2) + warp * 16, vw = a.V - v0;  // (a warp past V walks along with zeros)
  const int len = a.len(b), nck = (len + kDC - 1) / kDC;
  const float* q = static_cast<const float*>(a.q) + (long long)b * a.L * a.ldq + (long long)gh * a.K;
  const float* k = static_cast<const float*>(a.k) + (long long)b * a.L * a.ldk + (long long)gh * a.K;
  const float* v = static_cast<const float*>(a.v) + (long long)b * a.L * a.ldv + (long long)h * a.V + v0;
  float* ob = o + ((long long)b * a.L * a.H + h) * a.V + v0;
  const long long ldo = (long long)a.H * a.V;

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
    DSlice::load(at + St::slices + warp * DSlice::bytes, v + t0 * a.ldv, a.ldv, valid, vw, lane);
    cp_commit();
  };

  float S[KT][4];
#pragma unroll
  for (int j = 0; j < KT; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int kk = 8 * j + t2 + (e & 1), vv = g + (e >> 1) * 8;
      S[j][e] = h0 != nullptr && kk < a.K && vv < vw ? h0[(bh * a.K + kk) * a.V + v0 + vv] : 0.f;
    }
  if (ckpt != nullptr) ckpt += bh * delta_ckpt_floats(a.nck, a.K, a.V);
  float* ro = ckpt + (long long)(a.nck + 1) * a.K * a.V;  // r of every chunk, [V][64], and then the state's part of o
  auto keep = [&](float* dst, int t, const float (&x)[4]) {  // two tokens of two columns
#pragma unroll
    for (int e = 0; e < 4; e += 2) {
      const int vv = g + (e >> 1) * 8;
      if (vv < vw) *reinterpret_cast<float2*>(dst + (long long)(v0 + vv) * kDC + t) = make_float2(x[e], x[e + 1]);
    }
  };
  auto save = [&](int ck) {  // the state entering chunk ck: [V][K]
#pragma unroll
    for (int j = 0; j < KT; ++j)
#pragma unroll
      for (int e = 0; e < 4; e += 2) {
        const int kk = 8 * j + t2, vv = g + (e >> 1) * 8;
        if (kk < a.K && vv < vw)
          *reinterpret_cast<float2*>(ckpt + ((long long)ck * a.V + v0 + vv) * a.K + kk) = make_float2(S[j][e], S[j][e + 1]);
      }
  };

  pdl_wait();  // M, P and the scalars are delta_prep_kernel's
  if (nck > 0) fetch(0);
  for (int ck = 0; ck < nck; ++ck) {
    const uint32_t off = stages == 2 ? (uint32_t)((ck & 1) * stage_bytes) : 0u, at = sb + off;
    const float* vec = reinterpret_cast<const float*>(raw + off + St::vec);
    float* up = reinterpret_cast<float*>(raw + off + St::up);
    cp_wait<0>();
    __syncthreads();
    tile_scale<KP, true>(at + St::k, up, tid, nt);
    tile_scale<KP, false>(at + St::q, up + kDC, tid, nt);
    __syncthreads();
    if (stages == 2 && ck + 1 < nck) fetch(ck + 1);  // its place was read in the chunk before
    if (ckpt != nullptr) save(ck);
    const RowScale ss = row_scale(S);
    // R^T = v^T - e^c (K S0)^T
    float R[8][4], low[8][4];
    clear(R);
    clear(low);
#pragma unroll
    for (int kb = 0; kb < KP / 16; ++kb) {
      uint32_t hi[4], lo[4];
      left_terms(hi, lo, S[2 * kb], S[2 * kb + 1], ss);
#pragma unroll
      for (int np = 0; np < 4; ++np) {
        uint32_t bb[N][4];
#pragma unroll
        for (int n = 0; n < N; ++n) right_rows<KP, N>(bb[n], at + St::k, np, kb, n, lane);
        mma_terms(R[2 * np], R[2 * np + 1], low[2 * np], low[2 * np + 1], hi, lo, bb[0], bb[N - 1]);
      }
    }
    fold(R, low);
#pragma unroll
    for (int np = 0; np < 4; ++np) {
      float x[2][4];
      DSlice::read(at + St::slices + warp * DSlice::bytes, np, lane, x[0], x[1]);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int n = 2 * np + i, t = 8 * n + t2;
        const float2 in = *reinterpret_cast<const float2*>(vec + t), ku = *reinterpret_cast<const float2*>(up + t);
        const float d0 = __frcp_rn(ku.x), d1 = __frcp_rn(ku.y);  // powers of two: exact
        R[n][0] = fmaf(-in.x * ss.r[0].up, R[n][0], x[i][0] * d0);
        R[n][1] = fmaf(-in.y * ss.r[0].up, R[n][1], x[i][1] * d1);
        R[n][2] = fmaf(-in.x * ss.r[1].up, R[n][2], x[i][2] * d0);
        R[n][3] = fmaf(-in.y * ss.r[1].up, R[n][3], x[i][3] * d1);
      }
    }
    uint32_t hi[4][4], lo[4][4];
    {  // r^T = R^T - (beta R)^T M^T, u^T = beta r^T
      float w[8][4];
#pragma unroll
      for (int n = 0; n < 8; ++n) {
        const float2 be = *reinterpret_cast<const float2*>(vec + 2 * kDC + 8 * n + t2);
        w[n][0] = be.x * R[n][0];
        w[n][1] = be.y * R[n][1];
        w[n][2] = be.x * R[n][2];
        w[n][3] = be.y * R[n][3];
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
        for (int kb = 0; kb <= np; ++kb) {  // tokens up to this one
          uint32_t b0[4], b1[4];
          right_rows<kDC, 2>(b0, at + St::m, np, kb, 0, lane);
          right_rows<kDC, 2>(b1, at + St::m, np, kb, 1, lane);
          mma_terms(c[0], c[1], d[0], d[1], hi[kb], lo[kb], b0, b1);
        }
        fold(c, d);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int n = 2 * np + i, t = 8 * n + t2;
          const float2 em = *reinterpret_cast<const float2*>(vec + 3 * kDC + t), be = *reinterpret_cast<const float2*>(vec + 2 * kDC + t);
          R[n][0] = fmaf(-em.x * ws.r[0].up, c[i][0], R[n][0]);
          R[n][1] = fmaf(-em.y * ws.r[0].up, c[i][1], R[n][1]);
          R[n][2] = fmaf(-em.x * ws.r[1].up, c[i][2], R[n][2]);
          R[n][3] = fmaf(-em.y * ws.r[1].up, c[i][3], R[n][3]);
          if (ckpt != nullptr) keep(ro + (long long)ck * kDC * a.V, t, R[n]);
          R[n][0] *= be.x;
          R[n][1] *= be.y;
          R[n][2] *= be.x;
          R[n][3] *= be.y;
        }
      }
    }
    {  // o^T = scale (e^c (Q S0)^T + u^T P^T)
      float O[8][4], low[8][4];
      clear(O);
      clear(low);
#pragma unroll
      for (int kb = 0; kb < KP / 16; ++kb) {
        uint32_t sh[4], sl[4];
        left_terms(sh, sl, S[2 * kb], S[2 * kb + 1], ss);
#pragma unroll
        for (int np = 0; np < 4; ++np) {
          uint32_t bb[N][4];
#pragma unroll
          for (int n = 0; n < N; ++n) right_rows<KP, N>(bb[n], at + St::q, np, kb, n, lane);
          mma_terms(O[2 * np], O[2 * np + 1], low[2 * np], low[2 * np + 1], sh, sl, bb[0], bb[N - 1]);
        }
      }
      fold(O, low);
      const RowScale us = row_scale(R);
#pragma unroll
      for (int kb = 0; kb < 4; ++kb) {
        left_terms(hi[kb], lo[kb], R[2 * kb], R[2 * kb + 1], us);
      }
      const int t0 = ck * kDC, rows = a.L - t0 < kDC ? a.L - t0 : kDC;
#pragma unroll
      for (int np = 0; np < 4; ++np) {
        float c[2][4], d[2][4];
        clear(c);
        clear(d);
#pragma unroll
        for (int kb = 0; kb <= np; ++kb) {
          uint32_t bb[N][4];
#pragma unroll
          for (int n = 0; n < N; ++n) right_rows<kDC, N>(bb[n], at + St::p, np, kb, n, lane);
          mma_terms(c[0], c[1], d[0], d[1], hi[kb], lo[kb], bb[0], bb[N - 1]);
        }
        fold(c, d);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int n = 2 * np + i, t = 8 * n + t2;
          const float2 in = *reinterpret_cast<const float2*>(vec + t), qu = *reinterpret_cast<const float2*>(up + kDC + t);
          const float f0 = t0 + t < len ? a.scale * qu.x : 0.f, f1 = t0 + t + 1 < len ? a.scale * qu.y : 0.f;
          if (ckpt != nullptr) {
            const bool on0 = t0 + t < len, on1 = t0 + t + 1 < len;  // (not 0 * NaN)
            const float x0 = f0 * in.x * ss.r[0].up, x1 = f1 * in.y * ss.r[0].up, x2 = f0 * in.x * ss.r[1].up, x3 = f1 * in.y * ss.r[1].up;
            const float st[4] = {on0 ? x0 * O[n][0] : 0.f, on1 ? x1 * O[n][1] : 0.f, on0 ? x2 * O[n][2] : 0.f, on1 ? x3 * O[n][3] : 0.f};
            keep(ro + (long long)(a.nck + ck) * kDC * a.V, t, st);
          }
          O[n][0] = f0 * fmaf(O[n][0], in.x * ss.r[0].up, c[i][0] * us.r[0].up);
          O[n][1] = f1 * fmaf(O[n][1], in.y * ss.r[0].up, c[i][1] * us.r[0].up);
          O[n][2] = f0 * fmaf(O[n][2], in.x * ss.r[1].up, c[i][2] * us.r[1].up);
          O[n][3] = f1 * fmaf(O[n][3], in.y * ss.r[1].up, c[i][3] * us.r[1].up);
          if (t0 + t >= len) O[n][0] = O[n][2] = 0.f;  // (not 0 * NaN)
          if (t0 + t + 1 >= len) O[n][1] = O[n][3] = 0.f;
          store_tokens(ob + (long long)t0 * ldo, ldo, 8 * n, rows, vw, O[n], lane);
        }
      }
    }
    {  // S1^T = e^{c_last} S0^T + (rest u)^T K
#pragma unroll
      for (int n = 0; n < 8; ++n) {
        const float2 re = *reinterpret_cast<const float2*>(vec + kDC + 8 * n + t2);
        R[n][0] *= re.x;
        R[n][1] *= re.y;
        R[n][2] *= re.x;
        R[n][3] *= re.y;
      }
      const RowScale us = row_scale(R);
#pragma unroll
      for (int kb = 0; kb < 4; ++kb) left_terms(hi[kb], lo[kb], R[2 * kb], R[2 * kb + 1], us);
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
          for (int n = 0; n < N; ++n) right_cols<KP, N>(bb[n], at + St::k, jp, kb, n, lane);
          mma_terms(c[0], c[1], d[0], d[1], hi[kb], lo[kb], bb[0], bb[N - 1]);
        }
        fold(c, d);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float(&s)[4] = S[2 * jp + i];
          s[0] = fmaf(s[0], whole, c[i][0] * us.r[0].up);
          s[1] = fmaf(s[1], whole, c[i][1] * us.r[0].up);
          s[2] = fmaf(s[2], whole, c[i][2] * us.r[1].up);
          s[3] = fmaf(s[3], whole, c[i][3] * us.r[1].up);
        }
      }
    }
    if (stages == 1) {
      __syncthreads();
      if (ck + 1 < nck) fetch(ck + 1);
    }
  }
  if (ckpt != nullptr) save(nck);
  if (h_last != nullptr) {
#pragma unroll
    for (int j = 0; j < KT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int kk = 8 * j + t2 + (e & 1), vv = g + (e >> 1) * 8;
        if (kk < a.K && vv < vw) h_last[(bh * a.K + kk) * a.V + v0 + vv] = S[j][e];
      }
  }
  // tokens of chunks past the row's end
  const int w = vw < 16 ? vw : 16;
  for (long long i = (long long)nck * kDC * 16 + lane; i < (long long)a.L * 16; i += 32)
    if ((int)(i & 15) < w) ob[(i >> 4) * ldo + (i & 15)] = 0.f;
}

struct FwdPlan {
  Delta p;
  size_t bytes;
};

int fwd_plan(int B, int L, int H, int G, int K, int V, int dtype, FwdPlan& pl) {
  const int rc = delta_validate(B, L, H, G, K, V, dtype);
  if (rc != SS_OK) return rc;
  pl.p = Delta{};
  LinAttn& a = pl.p.a;
  a.B = B; a.L = L; a.H = H; a.G = G; a.K = K; a.V = V;
  a.nck = (L + kDC - 1) / kDC;
  pl.bytes = pl.p.prep_bytes(dtype == SS_BF16);
  return SS_OK;
}

template <int KP>
int walk(const FwdPlan& pl, const float* h0, void* o, float* ckpt, float* h_last, cudaStream_t s) {
  using St = WalkStage<KP>;
  const LinAttn& a = pl.p.a;
  const long long bh = (long long)a.B * a.H;
  int warps = (a.V + 15) / 16;
  while (warps > 1 && bh * ((a.V + 16 * warps - 1) / (16 * warps)) < 100) warps = (warps + 1) / 2;
  const int nvt = (a.V + 16 * warps - 1) / (16 * warps);
  // A chunk's tiles have two places where these fit and the CTAs are no more than the SMs; with more CTAs two an SM, each with
  // one place, are faster than one with two (192 heads of 64 x 64: 363 us for 497).
  const int sb = St::bytes(warps), stages = 2 * sb <= 226 * 1024 && bh * nvt <= 152 ? 2 : 1;
  return delta_launch_next(delta_fwd_kernel<KP>, (unsigned)(bh * nvt), 32 * warps, (size_t)sb * stages, s, pl.p, h0, static_cast<float*>(o), ckpt,
                           h_last, stages, sb);
}

}  // namespace

extern "C" size_t deltarule_ckpt_size(int L, int K, int V, int dtype) {
  FwdPlan pl;
  if (fwd_plan(1, L, 1, 1, K, V, dtype, pl) != SS_OK) return 0;
  return (size_t)delta_ckpt_floats(pl.p.a.nck, K, V) + pl.bytes / sizeof(float);
}

extern "C" size_t deltarule_fwd_workspace_size(int B, int L, int H, int G, int K, int V, int dtype) {
  FwdPlan pl;
  return fwd_plan(B, L, H, G, K, V, dtype, pl) == SS_OK ? pl.bytes : 0;
}

extern "C" int deltarule_fwd(const void* q, long long ldq, const void* k, long long ldk, const void* v, long long ldv, const float* g,
                             const float* beta, const float* h0, const int* lengths, void* o, float* ckpt, float* h_last, int B, int L,
                             int H, int G, int K, int V, float scale, int dtype, void* workspace, size_t ws_bytes, void* stream) {
  if (!q || !k || !v || !beta || !o) return SS_ERR_NULL;
  FwdPlan pl;
  int rc = fwd_plan(B, L, H, G, K, V, dtype, pl);
  if (rc != SS_OK) return rc;
  if ((rc = linattn_ld_ok(ldq, G, K)) != SS_OK || (rc = linattn_ld_ok(ldk, G, K)) != SS_OK || (rc = linattn_ld_ok(ldv, H, V)) != SS_OK)
    return rc;
  const void* ptrs[] = {q, k, v, o, h0, ckpt, h_last};
  for (const void* x : ptrs)
    if (x != nullptr && !ssh::aligned16(x)) return SS_ERR_ALIGN;
  if ((reinterpret_cast<uintptr_t>(g) & 3u) || (reinterpret_cast<uintptr_t>(beta) & 3u) || (reinterpret_cast<uintptr_t>(lengths) & 3u))
    return SS_ERR_ALIGN;
  if (ckpt == nullptr) {
    if (workspace == nullptr || ws_bytes < pl.bytes) return SS_ERR_WORKSPACE;
    if (!ssh::aligned16(workspace)) return SS_ERR_ALIGN;
  }
  LinAttn& a = pl.p.a;
  a.q = q; a.k = k; a.v = v;
  a.ldq = ldq; a.ldk = ldk; a.ldv = ldv;
  a.g = g;
  a.lengths = lengths;
  a.scale = scale;
  pl.p.beta = beta;
  pl.p.place(ckpt != nullptr ? ckpt + (long long)B * H * delta_ckpt_floats(a.nck, K, V) : workspace, dtype == SS_BF16);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if ((rc = ssh::delta_prep(pl.p, dtype, s)) != SS_OK) return rc;
  if (dtype == SS_F32) return K <= 64 ? walk<64>(pl, h0, o, ckpt, h_last, s) : walk<128>(pl, h0, o, ckpt, h_last, s);
  return ssh::delta_fwd_bf16(pl.p, h0, o, ckpt, h_last, s);
}
