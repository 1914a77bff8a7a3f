// The gated delta rule's other gradients, bf16, chunk by chunk on tcgen05 (delta_tc.cuh).  A CTA takes one (batch row, head,
// chunk) with the state S0 that enters it, its r and o (from the forward), the gradient dS of the state that leaves it and its
// du (from the backward chain); u = beta r, dR = beta du.
//   dbeta = <du, r>      dg_t = sum_{s >= t} (do_s.o_s - dR_s.v_s) + <S1, dS>           along columns of V, in fp32
//   E = scale D do u^T,  F = -D dR u^T (strict)                                          [t, s]
//   dq = scale e^c do S0^T + E K      dk = -e^c dR S0^T + e^{c_last - c} u dS^T + E^T Q + (F + F^T) K
// dq and dk are rounded to bf16; their fp32 operands are two bf16 terms (2^-15).  Products run with the columns of K as the
// 128 rows of an MMA; S0, dS, u and dR lie in shared memory by columns of V, as they come from memory, and are contracted down
// their rows.
#include "delta_tc.cuh"

namespace {

using namespace ssk;

constexpr int kGT = 512;
template <int KP>
struct GradTc {
  static constexpr int NKP = KP / 64, ST = NKP * kPanel;  // bytes of a term of a state
  static constexpr int S = 0, u = S + 2 * ST, r = u + 2 * kPanel, dy = r + 2 * kPanel, k = dy + 2 * kTok, q = k + NKP * kTok, e = q + NKP * kTok,
                       f = e + 2 * kDTerm, vec = f + 2 * kDTerm, dec = vec + kDVec * 4, red = dec + 2 * kDC * 4, bar = red + (16 * 32 + 16) * 4;
  static constexpr int kIn = 0, kM0 = 1, kM1 = 2, nbar = 3, tm = bar + nbar * 8, bytes = tm + 8;
  // tensor memory: do S0^T, dR S0^T, u dS^T, E, F, E K, E^T Q + (F + F^T) K
  static constexpr int G1 = 0, G2 = 64, G3 = 128, E = 192, F = 256, H1 = 320, H2 = 384, cols = 512;
};

struct GradMaps {
  CUtensorMap q, k, dy;
};

template <int KP, typename TO>
__global__ void __launch_bounds__(kGT, 1) delta_grad_tc_kernel(Delta p, const __grid_constant__ GradMaps maps, const float* __restrict__ ckpt,
                                                               const float* __restrict__ dS, const float* __restrict__ du, TO* __restrict__ dq,
                                                               TO* __restrict__ dk, int heads, float* __restrict__ dg, float* __restrict__ dbeta) {
  using L = GradTc<KP>;
  constexpr int SC = KP / 4, TC = kDC / 4;
  extern __shared__ __align__(1024) unsigned char raw[];
  const uint32_t sb = smem_u32(raw);
  uint64_t* bar = reinterpret_cast<uint64_t*>(raw + L::bar);
  uint32_t* tma = reinterpret_cast<uint32_t*>(raw + L::tm);
  const LinAttn& a = p.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const long long item = blockIdx.x, bh = item / a.nck;
  const int ck = (int)(item % a.nck), h = (int)(bh % a.H), b = (int)(bh / a.H), gh = h / (a.H / a.G);
  const int t0 = ck * kDC, len = a.len(b), rows = a.L - t0 < kDC ? a.L - t0 : kDC;
  const int valid = len - t0 < 0 ? 0 : len - t0 < kDC ? len - t0 : kDC;
  const long long tok = (long long)b * a.L + t0, ldg = (long long)heads * a.K;
  TO* dqb = dq + (tok * heads + (heads == a.G ? gh : h)) * a.K;
  TO* dkb = dk + (tok * heads + (heads == a.G ? gh : h)) * a.K;
  if (valid == 0) {
    for (int i = tid; i < rows * a.K; i += kGT) {
      ActT<TO>::st1(dqb + i / a.K * ldg + i % a.K, 0.f);
      ActT<TO>::st1(dkb + i / a.K * ldg + i % a.K, 0.f);
    }
    if (tid < rows) {
      if (dg != nullptr) dg[(tok + tid) * a.H + h] = 0.f;
      dbeta[(tok + tid) * a.H + h] = 0.f;
    }
    return;
  }
  float *vec = reinterpret_cast<float*>(raw + L::vec), *dec = reinterpret_cast<float*>(raw + L::dec), *red = reinterpret_cast<float*>(raw + L::red);
  const int kp = (a.K + 63) / 64, vp = (a.V + 63) / 64, vb = (a.V + 15) / 16;
  if (tid == 0) {
    for (int i = 0; i < L::nbar; ++i) mbar_init(&bar[i], 1);
    fence_barrier_init();
    mbar_arrive_expect_tx(&bar[L::kIn], (2 * kp + vp) * kTok);
    tok_load(sb + L::dy, vp, &maps.dy, &bar[L::kIn], h, t0, b);
    tok_load(sb + L::k, kp, &maps.k, &bar[L::kIn], gh, t0, b);
    tok_load(sb + L::q, kp, &maps.q, &bar[L::kIn], gh, t0, b);
  }
  if (warp == 0) {
    tmem_alloc(tma, L::cols);
    tmem_relinquish();
  }
  if (tid >= kGT - kDVec / 4) reinterpret_cast<float4*>(vec)[tid - (kGT - kDVec / 4)] = __ldcg(reinterpret_cast<const float4*>(p.vec + item * kDVec) + tid - (kGT - kDVec / 4));
  if (warp == 4) {
    ChunkGates<kDC> gates;
    if (a.g != nullptr) gates.fetch(a, b, h, t0, t0 + valid, lane);
    else gates.g[0] = gates.g[1] = 0.f;
    gates.scan(lane, [&](int i, Dec e) { dec[i] = e.hi; dec[kDC + i] = e.lo; });
  }
  const int row = (warp & 3) * 32 + lane, cq = warp >> 2;  // a column of V (or of K, or a token), a quarter of the other axis
  const bool mine = row < a.V;
  const float* base = ckpt + bh * delta_ckpt_floats(a.nck, a.K, a.V, true);
  const float4* s0 = reinterpret_cast<const float4*>(base + (long long)ck * a.K * a.V) + row;
  const float4* s1 = s0 + (long long)a.K * a.V / 4;
  const float4* rr = reinterpret_cast<const float4*>(base + (long long)(a.nck + 1) * a.K * a.V + (long long)ck * kDC * a.V) + (long long)(cq * TC / 4) * a.V + row;
  const float4* oo = rr + (long long)a.nck * kDC * a.V / 4;
  const float4* uu = reinterpret_cast<const float4*>(du + item * kDC * a.V) + (long long)(cq * TC / 4) * a.V + row;
  const __nv_bfloat16* v = static_cast<const __nv_bfloat16*>(a.v) + tok * a.ldv + (long long)h * a.V + row;
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tm = *tma;
  auto state = [&](const float4* src, float4 (&x)[SC / 4]) {
#pragma unroll
    for (int e = 0; e < SC / 4; ++e)
      x[e] = mine && cq * SC + 4 * e < a.K ? __ldcg(src + (long long)(cq * (SC / 4) + e) * a.V) : make_float4(0.f, 0.f, 0.f, 0.f);
  };
  float4 X[SC / 4];
  state(s0, X);
  bool ok = chain_wait(&bar[L::kIn], 0);
  if (valid < kDC && t0 + valid < a.L) {  // the row ends inside the tensor: what follows is not its own
    if (warp == 0) tok_clear(sb + L::dy, vp, valid, lane);
    if (warp == 1) tok_clear(sb + L::k, kp, valid, lane);
    if (warp == 2) tok_clear(sb + L::q, kp, valid, lane);
    __syncthreads();
  }
  // ---- along columns of V: u, dR and the sums
  float sums[32];  // this column's part of dbeta's and dg's 16 tokens
  {
    const uint32_t dcol = col_at(sb + L::dy, row < 64 * vp ? row : 0) + cq * TC * 128, unit = unit_at(kPanel, row, cq * (TC / 8));
    float2 y[TC / 2];
    ColRead<TC>::go(dcol, y);
#pragma unroll
    for (int u = 0; u < TC / 8; ++u) {
      float2 be[4], us[4], ds[4];
      pairs4(vec + 2 * kDC + cq * TC + 8 * u, be);
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        float4 r4 = make_float4(0.f, 0.f, 0.f, 0.f), d4 = r4, o4 = r4;
        if (mine) {
          r4 = __ldcs(rr + (long long)(2 * u + z) * a.V);
          d4 = __ldcs(uu + (long long)(2 * u + z) * a.V);
          o4 = __ldcs(oo + (long long)(2 * u + z) * a.V);
        }
        const float rs[4] = {r4.x, r4.y, r4.z, r4.w}, dd[4] = {d4.x, d4.y, d4.z, d4.w}, os[4] = {o4.x, o4.y, o4.z, o4.w};
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const int e = 8 * u + 4 * z + w, t = cq * TC + e;
          const bool on = mine && t < valid;
          const float bb = w & 1 ? be[2 * z + w / 2].y : be[2 * z + w / 2].x, yy = e & 1 ? y[e / 2].y : y[e / 2].x;
          const float vv = on ? ActT<__nv_bfloat16>::ld(v + (long long)t * a.ldv) : 0.f;
          const float uv = bb * rs[w], dv = bb * dd[w];
          sums[e] = dd[w] * rs[w];
          sums[16 + e] = on ? fmaf(yy, os[w], -dv * vv) : 0.f;
          (w & 1 ? us[2 * z + w / 2].y : us[2 * z + w / 2].x) = uv;
          (w & 1 ? ds[2 * z + w / 2].y : ds[2 * z + w / 2].x) = dv;
        }
      }
      if (row < 16 * vb) {
        put_terms<2>(sb + L::u + (unit ^ (16u * u)), kPanel, us);
        put_terms<2>(sb + L::r + (unit ^ (16u * u)), kPanel, ds);
      }
    }
  }
  auto put_state = [&](const float4 (&x)[SC / 4]) {  // two terms, [V][K]
    if (row >= 16 * vb) return;
#pragma unroll
    for (int e = 0; e < SC / 8; ++e) {
      float2 y[4] = {f2(x[2 * e].x, x[2 * e].y), f2(x[2 * e].z, x[2 * e].w), f2(x[2 * e + 1].x, x[2 * e + 1].y), f2(x[2 * e + 1].z, x[2 * e + 1].w)};
      put_terms<2>(sb + L::S + unit_at(kPanel, row, cq * (SC / 8) + e), L::ST, y);
    }
  };
  // sums over a warp's 32 columns: each step adds a half of the values to the other lane's and keeps the half
#pragma unroll
  for (int n = 16; n > 0; n >>= 1) {
    const bool upper = lane & n;
#pragma unroll
    for (int e = 0; e < n; ++e) {
      const float keep = upper ? sums[e + n] : sums[e], give = upper ? sums[e] : sums[e + n];
      sums[e] = keep + __shfl_xor_sync(0xffffffffu, give, n);
    }
  }
  red[warp * 32 + lane] = sums[0];  // value `lane`: dbeta of token cq * 16 + lane, from 16 on dg's
  put_state(X);
  fence_proxy_async_smem();
  __syncthreads();
  const int ksv = vb;
  if (warp == 0) {
    if (elect_one()) {
      const uint32_t ic = mma_idesc(64, true, false), cc = mma_idesc(64, true, true), rc = mma_idesc(64, false, true);
#pragma unroll 1
      for (int n = 1; n >= 0; --n)
#pragma unroll 1
        for (int s = 0; s < ksv; ++s) {
          mma_ss(tm + L::E, rows_desc(sb + L::dy, kTok, s), cols_desc(sb + L::u + n * kPanel, kPanel, s), rc, n < 1 || s > 0);
          mma_ss(tm + L::G1, cols_desc(sb + L::S + n * L::ST, kPanel, s), rows_desc(sb + L::dy, kTok, s), ic, n < 1 || s > 0);
        }
#pragma unroll 1
      for (int n = 0; n < 3; ++n) {  // (1, 0) (0, 1) (0, 0)
        const int i = n == 0, j = n == 1;
#pragma unroll 1
        for (int s = 0; s < ksv; ++s) {
          mma_ss(tm + L::F, cols_desc(sb + L::r + i * kPanel, kPanel, s), cols_desc(sb + L::u + j * kPanel, kPanel, s), cc, n > 0 || s > 0);
          mma_ss(tm + L::G2, cols_desc(sb + L::S + i * L::ST, kPanel, s), cols_desc(sb + L::r + j * kPanel, kPanel, s), cc, n > 0 || s > 0);
        }
      }
      mma_commit(&bar[L::kM0]);
    }
    __syncwarp();
  }
  // ---- under the products: <S1, dS>, and dg and dbeta
  float dot = 0.f;
  {
    float4 Y[SC / 4];
    state(s1, Y);
    state(reinterpret_cast<const float4*>(dS + item * a.K * a.V) + row, X);
#pragma unroll
    for (int e = 0; e < SC / 4; ++e) dot = fmaf(X[e].x, Y[e].x, fmaf(X[e].y, Y[e].y, fmaf(X[e].z, Y[e].z, fmaf(X[e].w, Y[e].w, dot))));
  }
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
  if (lane == 0) red[16 * 32 + warp] = dot;
  __syncthreads();
  if (warp == 15) {
    float s[2], x = 0.f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int t = 2 * lane + i, w = (t >> 4) * 4, e = t & 15;
      const float d = (red[w * 32 + e] + red[(w + 1) * 32 + e]) + (red[(w + 2) * 32 + e] + red[(w + 3) * 32 + e]);
      s[i] = (red[w * 32 + 16 + e] + red[(w + 1) * 32 + 16 + e]) + (red[(w + 2) * 32 + 16 + e] + red[(w + 3) * 32 + 16 + e]);
      if (t < rows) dbeta[(tok + t) * a.H + h] = t < valid ? d : 0.f;
    }
    for (int w = 0; w < 16; ++w) x += red[16 * 32 + w];
    float incl = s[0] + s[1];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const float y = __shfl_down_sync(0xffffffffu, incl, o);
      if (lane + o < 32) incl += y;
    }
    float after = __shfl_down_sync(0xffffffffu, incl, 1);
    if (lane == 31) after = 0.f;
    if (dg != nullptr) {
      if (2 * lane < rows) dg[(tok + 2 * lane) * a.H + h] = 2 * lane < valid ? x + incl : 0.f;
      if (2 * lane + 1 < rows) dg[(tok + 2 * lane + 1) * a.H + h] = 2 * lane + 1 < valid ? x + (s[1] + after) : 0.f;
    }
  }
  ok = chain_wait(&bar[L::kM0], 0) && ok;
  tc_fence_after_sync();
  put_state(X);  // dS where S0 was
  const uint32_t tl = tm + ((uint32_t)((warp & 3) * 32) << 16);
  if ((warp & 3) < 2) {  // E and F: row = token t, this warp's 16 tokens s
    uint32_t d[16], f[16];
    tmem_ld16(tl + L::E + cq * TC, d);
    tmem_ld16(tl + L::F + cq * TC, f);
    tmem_done(d);
    tmem_done(f);
    const float th = dec[row], tlo = dec[kDC + row];
#pragma unroll
    for (int u = 0; u < TC / 8; ++u) {
      float2 x[4], y[4];
#pragma unroll
      for (int z = 0; z < 8; ++z) {
        const int e = 8 * u + z, s = cq * TC + e;
        const float c = s <= row ? dec_diff(th, tlo, dec[s], dec[kDC + s]) : 0.f;
        const float xe = s <= row ? a.scale * c * __uint_as_float(d[e]) : 0.f, ye = s < row ? -c * __uint_as_float(f[e]) : 0.f;
        (z & 1 ? x[z / 2].y : x[z / 2].x) = xe;
        (z & 1 ? y[z / 2].y : y[z / 2].x) = ye;
      }
      const uint32_t at = unit_at(kTok, row, cq * (TC / 8) + u);
      put_terms<2>(sb + L::e + at, kDTerm, x);
      put_terms<2>(sb + L::f + at, kDTerm, y);
    }
  }
  fence_proxy_async_smem();
  tc_fence_before_sync();
  __syncthreads();
  if (warp == 0) {
    if (elect_one()) {
      tc_fence_after_sync();
      const uint32_t ic = mma_idesc(64, true, false), cc = mma_idesc(64, true, true);
#pragma unroll 1
      for (int n = 1; n >= 0; --n)
#pragma unroll 1
        for (int s = 0; s < 4; ++s) {
          const uint64_t kd = cols_desc(sb + L::k, kTok, s), qd = cols_desc(sb + L::q, kTok, s);
          const uint32_t et = sb + L::e + n * kDTerm, ft = sb + L::f + n * kDTerm;
          mma_ss(tm + L::H1, kd, rows_desc(et, kTok, s), ic, n < 1 || s > 0);
          mma_ss(tm + L::H2, qd, cols_desc(et, kTok, s), cc, n < 1 || s > 0);
          mma_ss(tm + L::H2, kd, rows_desc(ft, kTok, s), ic, true);
          mma_ss(tm + L::H2, kd, cols_desc(ft, kTok, s), cc, true);
        }
#pragma unroll 1
      for (int n = 0; n < 3; ++n) {
        const int i = n == 0, j = n == 1;
#pragma unroll 1
        for (int s = 0; s < ksv; ++s)
          mma_ss(tm + L::G3, cols_desc(sb + L::S + i * L::ST, kPanel, s), cols_desc(sb + L::u + j * kPanel, kPanel, s), cc, n > 0 || s > 0);
      }
      mma_commit(&bar[L::kM1]);
    }
    __syncwarp();
  }
  ok = chain_wait(&bar[L::kM1], 0) && ok;
  tc_fence_after_sync();
  if ((warp & 3) * 32 < a.K) {  // row = column of K, this warp's 16 tokens
#pragma unroll
    for (int c = 0; c < TC; c += 8) {
      uint32_t g1[8], g2[8], g3[8], h1[8], h2[8];
      tmem_ld8u(tl + L::G1 + cq * TC + c, g1);
      tmem_ld8u(tl + L::G2 + cq * TC + c, g2);
      tmem_ld8u(tl + L::G3 + cq * TC + c, g3);
      tmem_ld8u(tl + L::H1 + cq * TC + c, h1);
      tmem_ld8u(tl + L::H2 + cq * TC + c, h2);
      tmem_done(g1);
      tmem_done(g2);
      tmem_done(g3);
      tmem_done(h1);
      tmem_done(h2);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int t = cq * TC + c + e;
        const float in = vec[t], re = vec[kDC + t];
        const float x = fmaf(a.scale * in, __uint_as_float(g1[e]), __uint_as_float(h1[e]));
        const float y = fmaf(re, __uint_as_float(g3[e]), fmaf(-in, __uint_as_float(g2[e]), __uint_as_float(h2[e])));
        if (row < a.K && t < rows) {
          ActT<TO>::st1(dqb + (long long)t * ldg + row, t < valid ? x : 0.f);
          ActT<TO>::st1(dkb + (long long)t * ldg + row, t < valid ? y : 0.f);
        }
      }
    }
  }
  lin_leave(ok, bar, L::nbar, tm, L::cols, warp, lane);
}

template <int KP, typename TO>
int run(const Delta& p, const float* ckpt, const void* dout, const float* dS, const float* du, void* dq, void* dk, int heads, float* dg, float* dbeta,
        cudaStream_t s) {
  const LinAttn& a = p.a;
  GradMaps maps;
  if (!delta_map(&maps.q, a.q, a.ldq, a.B, a.L, a.G, a.K) || !delta_map(&maps.k, a.k, a.ldk, a.B, a.L, a.G, a.K) ||
      !delta_map(&maps.dy, dout, (long long)a.H * a.V, a.B, a.L, a.H, a.V))
    return SS_ERR_CUDA;
  static_assert(GradTc<KP>::bytes <= 227 * 1024, "a chunk's tiles fit shared memory");
  return lin_launch(delta_grad_tc_kernel<KP, TO>, (unsigned)((long long)a.B * a.H * a.nck), kGT, GradTc<KP>::bytes, s, p, maps, ckpt, dS, du,
                    static_cast<TO*>(dq), static_cast<TO*>(dk), heads, dg, dbeta);
}

}  // namespace

int ssh::delta_grad_bf16(const Delta& p, const float* ckpt, const void* dout, const float* dS, const float* du, void* dq, void* dk, bool parts, float* dg,
                         float* dbeta, cudaStream_t s) {
  const int heads = parts ? p.a.H : p.a.G;
  if (p.a.K <= 64)
    return parts ? run<64, float>(p, ckpt, dout, dS, du, dq, dk, heads, dg, dbeta, s) : run<64, __nv_bfloat16>(p, ckpt, dout, dS, du, dq, dk, heads, dg, dbeta, s);
  return parts ? run<128, float>(p, ckpt, dout, dS, du, dq, dk, heads, dg, dbeta, s) : run<128, __nv_bfloat16>(p, ckpt, dout, dS, du, dq, dk, heads, dg, dbeta, s);
}

namespace ssh {
int read_clear_delg_err(cudaStream_t s, unsigned* out) { return read_clear_lin_err(s, out); }
}  // namespace ssh
