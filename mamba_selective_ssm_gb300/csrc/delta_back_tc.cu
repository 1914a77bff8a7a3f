// The gated delta rule's backward chain, bf16, on tcgen05 (delta_tc.cuh): from the last chunk to the first the gradient of the
// state, as the forward carries the state (delta_fwd_tc.cu).  With dS = the gradient of the state leaving the chunk:
//   D2 = do^T P (P holds scale)      D1 = dS K^T       du0 = e^{c_last - c} D1 + D2,  w = beta du0  (three terms)
//   D3 = w M                         du = du0 - D3,  dv = dR = beta du,  -e^c dR  (three terms, w's place)
//   D5 = (scale e^c do)^T Q + (-e^c dR)^T K           dS = e^{c_last} dS + D5  (three terms, tensor memory)
// The product with Q waits for do alone and runs under the others.  Leaves dS and du of every chunk for the other gradients.
// 4 x 2048 tokens of 32 heads of 128 x 128: 170 us, bound as the forward's chain is.
#include "delta_tc.cuh"

namespace {

using namespace ssk;

constexpr int kDW = 16, kDThreads = 32 * (kDW + 1);  // computing warps; one that issues

template <int KP>
struct BackTc {
  static constexpr int NKP = KP / 64;  // panels of K
  static constexpr int kq = 0, place = NKP * kPanel, dy = kq + 2 * place, m = dy + 2 * kTok, p = m + 3 * kDTerm, a1 = p + 3 * kDTerm,
                       w2 = a1 + 3 * kPanel, out = w2 + kPanel, vec = out + 2 * kTok, bar = vec + 2 * kDVec * 4;
  // barriers: k and q (two), do, scalars (two), M, P landed; dS, w / -e^c dR, scale e^c do stored, dv staged; products done
  static constexpr int kK = 0, kV = 2, kX = 3, kMr = 5, kPr = 6, kS = 7, kW = 8, kA = 9, kO = 10, kD1 = 11, kD2 = 12, kD3 = 13, kD5 = 14, nbar = 15;
  static constexpr int tm = bar + nbar * 8, bytes = tm + 8;
  // tensor memory: dS's terms; D1, then D3; D2; D5; two terms of w (the third lies in shared memory)
  static constexpr int S = 0, D1 = 192, D2 = 256, D5 = 320, W = 448, cols = 512;
};

struct BackMaps {
  CUtensorMap q, k, dy, dv;
};

template <int KP>
__global__ void __launch_bounds__(kDThreads, 1) delta_back_tc_kernel(Delta p, const __grid_constant__ BackMaps maps,
                                                                     const float* __restrict__ dh_last,
                                                                     __nv_bfloat16* __restrict__ dv, float* __restrict__ dS, float* __restrict__ du,
                                                                     float* __restrict__ dh0) {
  using L = BackTc<KP>;
  constexpr int SC = KP / 4, TC = kDC / 4;  // a thread's columns of dS, its tokens of a product
  extern __shared__ __align__(1024) unsigned char raw[];
  const uint32_t sb = smem_u32(raw);
  uint64_t* bar = reinterpret_cast<uint64_t*>(raw + L::bar);
  uint32_t* tma = reinterpret_cast<uint32_t*>(raw + L::tm);
  const LinAttn& a = p.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const long long bh = blockIdx.x;
  const int h = (int)(bh % a.H), b = (int)(bh / a.H), gh = h / (a.H / a.G);
  const int len = a.len(b), nck = (len + kDC - 1) / kDC;
  const int quarters = (a.V + 31) / 32;  // of the 128 lanes that hold columns of V
  if (tid == 0) {
    for (int i = 0; i < L::nbar; ++i) mbar_init(&bar[i], i >= L::kS && i <= L::kO ? 4 * quarters : 1);
    fence_barrier_init();
  }
  pdl_trigger();
  if (warp == 0) {
    tmem_alloc(tma, L::cols);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tm = *tma;
  bool ok = true;
  auto wait = [&](int i, uint32_t par) { return ok = chain_wait(&bar[i], par); };

  if (warp == kDW) {  // ---- the issuing warp.  Chunk i of the walk is chunk nck - 1 - i of the row
    const int ks = (a.K + 15) / 16, kp = (a.K + 63) / 64, vp = (a.V + 63) / 64;
    auto item = [&](int i) { return bh * a.nck + (nck - 1 - i); };
    auto load_kq = [&](int i) {
      if (elect_one()) {
        uint64_t* at = &bar[L::kK + (i & 1)];
        mbar_arrive_expect_tx(at, 2 * kp * kTok);
        for (int n = 0; n < kp; ++n) {
          const uint32_t to = sb + L::kq + (i & 1) * L::place + n * kPanel;
          tma_load_4d(to, &maps.k, at, n * 64, gh, (nck - 1 - i) * kDC, b);
          tma_load_4d(to + kTok, &maps.q, at, n * 64, gh, (nck - 1 - i) * kDC, b);
        }
      }
      __syncwarp();
    };
    auto load_dy = [&](int i) {
      if (elect_one()) {
        mbar_arrive_expect_tx(&bar[L::kV], vp * kTok);
        tok_load(sb + L::dy, vp, &maps.dy, &bar[L::kV], h, (nck - 1 - i) * kDC, b);
      }
      __syncwarp();
    };
    auto load = [&](int n, int to, const void* src, int bytes) {
      if (elect_one()) {
        mbar_arrive_expect_tx(&bar[n], bytes);
        bulk_load(raw + to, src, bytes, &bar[n]);
      }
      __syncwarp();
    };
    auto load_m = [&](int i) { load(L::kMr, L::m, p.M + item(i) * kDMTerms, 3 * kDTerm); };
    auto load_p = [&](int i) { load(L::kPr, L::p, p.P + item(i) * 3 * kDTerm, 3 * kDTerm); };
    auto load_x = [&](int i) { load(L::kX + (i & 1), L::vec + (i & 1) * kDVec * 4, p.vec + item(i) * kDVec, kDVec * 4); };
    auto store_dv = [&](int i) {
      if (elect_one()) {
        for (int n = 0; n < vp; ++n) tma_store_4d(&maps.dv, sb + L::out + n * kTok, n * 64, h, (nck - 1 - i) * kDC, b);
        bulk_commit();
      }
      __syncwarp();
    };
    if (nck > 0) {
      load_dy(0);
      load_p(0);
      load_kq(0);
      load_x(0);
      load_m(0);
    }
    for (int i = 0; i < nck; ++i) {
      const uint32_t par = (uint32_t)i & 1u;
      const uint32_t kt = sb + L::kq + par * L::place;
      const int valid = len - (nck - 1 - i) * kDC;
      const bool more = i + 1 < nck, cut = valid < kDC && len < a.L;  // (the row ends inside the tensor: what follows is not its own)
      if (!wait(L::kV, par) || !wait(L::kPr, par)) break;
      if (cut) {
        tok_clear(sb + L::dy, vp, valid, lane);
        fence_proxy_async_smem();
        __syncwarp();
      }
      if (elect_one()) {  // tokens 16 s .. of P reach no token past them
#pragma unroll 1
        for (int n = 2; n >= 0; --n)
#pragma unroll
          for (int s = 3; s >= 0; --s)
            mma_ss(tm + L::D2, cols_desc(sb + L::dy, kTok, s), cols_desc(sb + L::p + n * kDTerm, kTok, s),
                   mma_idesc(16 * (s + 1), true, true), n < 2 || s < 3);
        mma_commit(&bar[L::kD2]);
      }
      __syncwarp();
      if (!wait(L::kK + (int)par, (uint32_t)(i >> 1) & 1u)) break;
      if (cut) {
        for (int n = 0; n < kp; ++n) {
          tok_clear(kt + n * kPanel, 1, valid, lane);
          tok_clear(kt + n * kPanel + kTok, 1, valid, lane);
        }
        fence_proxy_async_smem();
        __syncwarp();
      }
      if (!wait(L::kS, par)) break;
      if (elect_one()) {
        tc_fence_after_sync();
#pragma unroll 1
        for (int n = 2; n >= 0; --n)
#pragma unroll 4
          for (int s = 0; s < ks; ++s)
            mma_ts(tm + L::D1, tm + L::S + n * (KP / 2) + s * 8, rows_desc(kt, kPanel, s), mma_idesc(kDC, false, false), n < 2 || s > 0);
        mma_commit(&bar[L::kD1]);
      }
      __syncwarp();
      if (more) {  // their places were read by the chunk before, whose dS has been stored
        load_kq(i + 1);
        load_x(i + 1);
      }
      if (!wait(L::kA, par)) break;
      if (elect_one()) {
        tc_fence_after_sync();
#pragma unroll 1
        for (int n = 2; n >= 0; --n)
#pragma unroll
          for (int s = 0; s < 4; ++s)
            mma_ss(tm + L::D5, rows_desc(sb + L::a1 + n * kPanel, kPanel, s), cols_desc(kt + kTok, kPanel, s), mma_idesc(KP, false, true),
                   n < 2 || s > 0);
      }
      __syncwarp();
      if (!wait(L::kMr, par) || !wait(L::kW, 0u)) break;
      if (elect_one()) {
        tc_fence_after_sync();
        uint32_t pairs = 0x041852u;  // (w, M): (2, 0) (1, 1) (0, 2) (1, 0) (0, 1) (0, 0)
#pragma unroll 1
        for (int n = 0; n < 6; ++n, pairs >>= 4) {
          const uint32_t l = pairs & 3u, r = sb + L::m + (pairs >> 2 & 3u) * kDTerm;
#pragma unroll
          for (int s = 3; s >= 0; --s) {
            if (l == 2)
              mma_ss(tm + L::D1, rows_desc(sb + L::w2, kPanel, s), cols_desc(r, kTok, s), mma_idesc(16 * (s + 1), false, true), n > 0 || s < 3);
            else mma_ts(tm + L::D1, tm + L::W + l * 32 + s * 8, cols_desc(r, kTok, s), mma_idesc(16 * (s + 1), false, true), n > 0 || s < 3);
          }
        }
        bulk_wait_read();  // dv of the chunk before has left: this one's may be staged once D3 is done
        mma_commit(&bar[L::kD3]);
      }
      __syncwarp();
      if (more) {  // do and P have been read: D2 has been waited for
        load_dy(i + 1);
        load_p(i + 1);
      }
      if (!wait(L::kW, 1u)) break;
      if (elect_one()) {
        tc_fence_after_sync();
#pragma unroll
        for (int s = 0; s < 4; ++s) mma_ss(tm + L::D5, rows_desc(sb + L::w2, kPanel, s), cols_desc(kt, kPanel, s), mma_idesc(KP, false, true), true);
#pragma unroll 1
        for (int n = 1; n >= 0; --n)
#pragma unroll
          for (int s = 0; s < 4; ++s) mma_ts(tm + L::D5, tm + L::W + n * 32 + s * 8, cols_desc(kt, kPanel, s), mma_idesc(KP, false, true), true);
        mma_commit(&bar[L::kD5]);
      }
      __syncwarp();
      if (more) load_m(i + 1);  // (D3 has been read)
      if (!wait(L::kO, par)) break;
      store_dv(i);
    }
    if (elect_one()) bulk_wait();
    __syncwarp();
  } else if ((warp & 3) < quarters) {  // ---- a computing warp
    const int row = (warp & 3) * 32 + lane, cq = warp >> 2;  // this thread's column of V; its quarter of K and of the tokens
    const uint32_t tl = tm + ((uint32_t)((warp & 3) * 32) << 16);
    const bool mine = row < a.V;
    float2 S[SC / 2];
#pragma unroll
    for (int e = 0; e < SC; e += 2) {
      const int kk = cq * SC + e;
      const float* src = dh_last + (bh * a.K + kk) * a.V + row;
      S[e / 2] = dh_last != nullptr && mine && kk < a.K ? f2(src[0], src[a.V]) : f2(0.f, 0.f);
    }
    auto arrive = [&](int i) {
      fence_proxy_async_smem();
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar[i]);
    };
    auto store_s = [&](int c) {  // columns c .. c + 15 of this thread's as three terms, one at a time (registers)
      float2 x[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = S[c / 2 + e];
#pragma unroll
      for (int n = 0; n < 3; ++n) {
        uint32_t w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = n < 2 ? take_pair(x[e]) : last_pair(x[e]);
        tmem_stn(tl + L::S + n * (KP / 2) + (cq * SC + c) / 2, w);
      }
    };
    const uint32_t dcol = col_at(sb + L::dy, row) + cq * TC * 128, ocol = col_at(sb + L::out, row) + cq * TC * 128;
    const uint32_t unit = unit_at(kPanel, row, cq * (TC / 8));  // a unit of 8 tokens; the next is at ^ 16
    auto store_w = [&](int u, float2 (&x)[4]) {  // eight tokens as three terms
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = take_pair(x[e]);
        tmem_st4(tl + L::W + n * 32 + cq * (TC / 2) + 4 * u, w);
      }
      sts16(sb + L::w2 + (unit ^ (16u * u)), make_uint4(last_pair(x[0]), last_pair(x[1]), last_pair(x[2]), last_pair(x[3])));
    };
    if (nck > 0) {
#pragma unroll
      for (int c = 0; c < SC; c += 16) store_s(c);
      tmem_wait_st();
      arrive(L::kS);
    }
    for (int i = 0; i < nck && ok; ++i) {
      const uint32_t par = (uint32_t)i & 1u;
      const int ck = nck - 1 - i, valid = len - ck * kDC;
      const long long item = bh * a.nck + ck;
      const float* vec = reinterpret_cast<const float*>(raw + L::vec + par * kDVec * 4) + cq * TC;
      float2 R[TC / 2];
      if (!wait(L::kX + (int)par, (uint32_t)(i >> 1) & 1u) || !wait(L::kV, par)) break;
      ColRead<TC>::go(dcol, R);
      if (valid < kDC) {
#pragma unroll
        for (int e = 0; e < TC; ++e)
          if (cq * TC + e >= valid) (e & 1 ? R[e / 2].y : R[e / 2].x) = 0.f;
      }
#pragma unroll
      for (int u = 0; u < TC / 8; ++u) {  // (the place was read by D5 of the chunk before, which has been waited for)
        float2 in[4], x[4];
        pairs4(vec + 8 * u, in);
#pragma unroll
        for (int z = 0; z < 4; ++z) x[z] = mul2(mul2(bc2(a.scale), in[z]), R[4 * u + z]);
        put_terms<3>(sb + L::a1 + (unit ^ (16u * u)), kPanel, x);
      }
      arrive(L::kA);
      if (mine) {  // dS, [K / 4][V][4]
        float4* dst = reinterpret_cast<float4*>(dS + item * a.K * a.V) + row;
#pragma unroll
        for (int e = 0; e < SC; e += 4)
          if (cq * SC + e < a.K) dst[(long long)((cq * SC + e) / 4) * a.V] = make_float4(S[e / 2].x, S[e / 2].y, S[e / 2 + 1].x, S[e / 2 + 1].y);
      }
      if (!wait(L::kD2, par) || !wait(L::kD1, par)) break;
      tc_fence_after_sync();
      {
        uint32_t d[16], f[16];
        tmem_ld16(tl + L::D1 + cq * TC, d);
        tmem_ld16(tl + L::D2 + cq * TC, f);
        tmem_done(d);
        tmem_done(f);
#pragma unroll
        for (int u = 0; u < TC / 8; ++u) {
          float2 re[4], be[4], x[4];
          pairs4(vec + kDC + 8 * u, re);
          pairs4(vec + 2 * kDC + 8 * u, be);
#pragma unroll
          for (int z = 0; z < 4; ++z) {
            const int e = 4 * u + z;
            R[e] = fma2(re[z], u2f(d[2 * e], d[2 * e + 1]), u2f(f[2 * e], f[2 * e + 1]));
            x[z] = mul2(be[z], R[e]);
          }
          store_w(u, x);
        }
      }
      tmem_wait_st();
      arrive(L::kW);
      if (!wait(L::kD3, par)) break;
      tc_fence_after_sync();
      {
        uint32_t d[16];
        tmem_ld16(tl + L::D1 + cq * TC, d);
        tmem_done(d);
#pragma unroll
        for (int e = 0; e < TC / 2; ++e) R[e] = fma2(u2f(d[2 * e], d[2 * e + 1]), bc2(-1.f), R[e]);
#pragma unroll
        for (int u = 0; u < TC / 8; ++u) {
          float2 in[4], be[4], x[4];
          pairs4(vec + 8 * u, in);
          pairs4(vec + 2 * kDC + 8 * u, be);
#pragma unroll
          for (int z = 0; z < 4; ++z) x[z] = mul2(mul2(in[z], bc2(-1.f)), mul2(be[z], R[4 * u + z]));
          store_w(u, x);
        }
      }
      tmem_wait_st();
      arrive(L::kW);
      if (mine) {  // du, [16][V][4]
        float4* dst = reinterpret_cast<float4*>(du + item * kDC * a.V) + (long long)(cq * TC / 4) * a.V + row;
#pragma unroll
        for (int e = 0; e < TC / 2; e += 2) dst[(long long)(e / 2) * a.V] = make_float4(R[e].x, R[e].y, R[e + 1].x, R[e + 1].y);
      }
#pragma unroll
      for (int u = 0; u < TC / 8; ++u) {
        float2 be[4];
        pairs4(vec + 2 * kDC + 8 * u, be);
#pragma unroll
        for (int z = 0; z < 4; ++z) R[4 * u + z] = mul2(be[z], R[4 * u + z]);
      }
      if (valid < kDC) {
#pragma unroll
        for (int e = 0; e < TC; ++e)
          if (cq * TC + e >= valid) (e & 1 ? R[e / 2].y : R[e / 2].x) = 0.f;
      }
      ColWrite<TC>::go(ocol, R);
      const float whole = vec[4 * kDC - cq * TC];
      arrive(L::kO);
      if (!wait(L::kD5, par)) break;
      tc_fence_after_sync();
#pragma unroll
      for (int c = 0; c < SC; c += 16) {
        uint32_t d[16];
        tmem_ld16(tl + L::D5 + cq * SC + c, d);
        tmem_done(d);
#pragma unroll
        for (int e = 0; e < 8; ++e) S[c / 2 + e] = fma2(S[c / 2 + e], bc2(whole), u2f(d[2 * e], d[2 * e + 1]));
        if (i + 1 < nck) store_s(c);
      }
      if (i + 1 < nck) {
        tmem_wait_st();
        arrive(L::kS);
      }
    }
    if (ok && mine && dh0 != nullptr) {
#pragma unroll
      for (int e = 0; e < SC; ++e)
        if (cq * SC + e < a.K) dh0[(bh * a.K + cq * SC + e) * a.V + row] = e & 1 ? S[e / 2].y : S[e / 2].x;
    }
  }
  // tokens of chunks past the row's end
  const int n = a.V / 8;
  for (long long i = (long long)nck * kDC * n + tid; i < (long long)a.L * n; i += kDThreads)
    *reinterpret_cast<uint4*>(dv + (((long long)b * a.L + i / n) * a.H + h) * a.V + i % n * 8) = make_uint4(0u, 0u, 0u, 0u);
  lin_leave(ok, bar, L::nbar, tm, L::cols, warp, lane);
}

template <int KP>
int walk(const Delta& p, const __nv_bfloat16* dout, const float* dh_last, __nv_bfloat16* dv, float* dS, float* du, float* dh0, cudaStream_t s) {
  const LinAttn& a = p.a;
  const long long ldo = (long long)a.H * a.V;
  BackMaps maps;
  if (!delta_map(&maps.q, a.q, a.ldq, a.B, a.L, a.G, a.K) || !delta_map(&maps.k, a.k, a.ldk, a.B, a.L, a.G, a.K) ||
      !delta_map(&maps.dy, dout, ldo, a.B, a.L, a.H, a.V) || !delta_map(&maps.dv, dv, ldo, a.B, a.L, a.H, a.V))
    return SS_ERR_CUDA;
  static_assert(BackTc<KP>::bytes <= 227 * 1024, "a chunk's tiles fit shared memory");
  return delta_launch(delta_back_tc_kernel<KP>, (unsigned)((long long)a.B * a.H), kDThreads, BackTc<KP>::bytes, s, p, maps, dh_last, dv, dS, du, dh0);
}

}  // namespace

int ssh::delta_back_bf16(const Delta& p, const void* dout, const float* dh_last, void* dv, float* dS, float* du, float* dh0, cudaStream_t s) {
  const __nv_bfloat16* y = static_cast<const __nv_bfloat16*>(dout);
  __nv_bfloat16* dvb = static_cast<__nv_bfloat16*>(dv);
  return p.a.K <= 64 ? walk<64>(p, y, dh_last, dvb, dS, du, dh0, s) : walk<128>(p, y, dh_last, dvb, dS, du, dh0, s);
}

namespace ssh {
int read_clear_delb_err(cudaStream_t s, unsigned* out) { return read_clear_lin_err(s, out); }
}  // namespace ssh
