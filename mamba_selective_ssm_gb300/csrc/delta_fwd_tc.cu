// The gated delta rule, chunked forward, bf16: the chain on tcgen05 (delta_tc.cuh).  A CTA walks the chunks of one
// (batch row, head) with the state in registers (thread = one column of V and a quarter of K) and, as three bf16 terms, in tensor
// memory, where it is the left operand of K S0 and Q S0.
//   D1 = S K^T       R = v - e^c D1,  w = beta R  (three terms, tensor memory)
//   D3 = w M^T       r = R - D3,  u = beta r,  e^{c_last - c} u (three terms, w's place),  u (three terms, shared memory)
//   D5 = .. K        S = e^{c_last} S + D5  (three terms, tensor memory)
//   D2 = S Q^T, D4 = u P^T:  o = scale e^c D2 + D4, under the next chunk's D1
// Sixteen warps compute, one issues the copies and MMAs; they meet at mbarriers with bounded waits.  With the left operand in
// tensor memory an MMA of 64 columns takes 36 cycles, in shared memory 51.
// 4 x 2048 tokens of 32 heads of 128 x 128: 145 us, with ckpt 192 (128 CTAs of 32 chunks, 4.5 and 6.0 us a chunk; with ckpt tensor
// pipe 27 %, memory 57 %): the chain of a chunk's steps bounds it, reading sums and making terms of operands between the
// products.
#include "delta_tc.cuh"

namespace {

using namespace ssk;

constexpr int kDW = 16, kDThreads = 32 * (kDW + 1);  // computing warps; one that issues

template <int KP>
struct DeltaTc {
  // terms of u and P: with two, o was 2e-4 of its size from the rounded fp32 result, for 4e-5, and had other bits than with ckpt
  static constexpr int UT = 3;
  static constexpr int NKP = KP / 64;  // panels of K
  static constexpr int kq = 0, place = NKP * kPanel, v = kq + 2 * place, m = v + 2 * kTok, p = m + 3 * kDTerm,
                       u = p + UT * kDTerm, vec = u + UT * kPanel, bar = vec + 2 * kDVec * 4;
  // barriers: k and q (two), v, scalars (two), M, P landed; S, w / weighted u, u stored, o staged; products done
  static constexpr int kK = 0, kV = 2, kX = 3, kMr = 5, kPr = 6, kS = 7, kW = 8, kU = 9, kO = 10, kD1 = 11, kD3 = 12, kD4 = 13, kD5 = 14,
                       nbar = 15;
  static constexpr int tm = bar + nbar * 8, bytes = tm + 8;
  // tensor memory: the state's terms; D1, then D3, and with the columns after it D5; D2; w's terms, then D4
  static constexpr int S = 0, D1 = 192, D5 = 192, D2 = 320, W = 384, D4 = 384, cols = 512;
};

struct DeltaMaps {
  CUtensorMap q, k, v, o;
};

template <int KP, bool TRAIN>
__global__ void __launch_bounds__(kDThreads, 1) delta_fwd_tc_kernel(Delta p, const __grid_constant__ DeltaMaps maps, const float* __restrict__ h0,
                                                                    __nv_bfloat16* __restrict__ o, float* __restrict__ ckpt,
                                                                    float* __restrict__ h_last) {
  using L = DeltaTc<KP>;
  constexpr int UT = L::UT;
  constexpr int SC = KP / 4, TC = kDC / 4;  // a thread's columns of the state, its tokens of a product
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
    for (int i = 0; i < L::nbar; ++i)
      mbar_init(&bar[i], i >= L::kS && i <= L::kO ? 4 * quarters : 1);
    fence_barrier_init();
  }
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

  if (warp == kDW) {  // ---- the issuing warp
    const int ks = (a.K + 15) / 16, kp = (a.K + 63) / 64, vp = (a.V + 63) / 64;
    auto load_kq = [&](int ck) {  // panels of 128 rows: the tokens of k, then those of q
      if (elect_one()) {
        uint64_t* at = &bar[L::kK + (ck & 1)];
        mbar_arrive_expect_tx(at, 2 * kp * kTok);
        for (int i = 0; i < kp; ++i) {
          const uint32_t to = sb + L::kq + (ck & 1) * L::place + i * kPanel;
          tma_load_4d(to, &maps.k, at, i * 64, gh, ck * kDC, b);
          tma_load_4d(to + kTok, &maps.q, at, i * 64, gh, ck * kDC, b);
        }
      }
      __syncwarp();
    };
    auto load_v = [&](int ck) {
      if (elect_one()) {
        mbar_arrive_expect_tx(&bar[L::kV], vp * kTok);
        tok_load(sb + L::v, vp, &maps.v, &bar[L::kV], h, ck * kDC, b);
      }
      __syncwarp();
    };
    auto load_m = [&](int ck) {
      if (elect_one()) {
        mbar_arrive_expect_tx(&bar[L::kMr], 3 * kDTerm);
        bulk_load(raw + L::m, p.M + (bh * a.nck + ck) * kDMTerms, 3 * kDTerm, &bar[L::kMr]);
      }
      __syncwarp();
    };
    auto load_p = [&](int ck) {
      if (elect_one()) {
        mbar_arrive_expect_tx(&bar[L::kPr], UT * kDTerm);
        bulk_load(raw + L::p, p.P + (bh * a.nck + ck) * UT * kDTerm, UT * kDTerm, &bar[L::kPr]);
      }
      __syncwarp();
    };
    auto load_x = [&](int ck) {
      if (elect_one()) {
        uint64_t* at = &bar[L::kX + (ck & 1)];
        mbar_arrive_expect_tx(at, kDVec * 4);
        bulk_load(raw + L::vec + (ck & 1) * kDVec * 4, p.vec + (bh * a.nck + ck) * kDVec, kDVec * 4, at);
      }
      __syncwarp();
    };
    auto store_o = [&](int ck) {
      if (elect_one()) {
        for (int i = 0; i < vp; ++i) tma_store_4d(&maps.o, sb + L::u + i * kTok, i * 64, h, ck * kDC, b);
        bulk_commit();
      }
      __syncwarp();
    };
    // a product with M or P, of which the column tiles from 16 s on are not zero (products of whole tiles give the same bits at all
    // sizes of the tests, and take 4 % longer in the forward).  `pairs`: its pairs of terms from the smallest, left in the low and
    // right in the high bits of four
    auto lower = [&](uint32_t right, uint32_t pairs, int n, auto mma) {
#pragma unroll 1
      for (int i = 0; i < n; ++i, pairs >>= 4) {
        const uint32_t l = pairs & 3u, r = right + (pairs >> 2 & 3u) * kDTerm;
#pragma unroll
        for (int s = 0; s < 4; ++s) mma(l, s, rows_desc(r, kTok, s, 16 * s), mma_idesc(kDC - 16 * s, false, false), i > 0 || s > 0);
      }
    };
    if (nck > 0) {
      load_kq(0);
      load_v(0);
    }
    pdl_wait();  // M, P and the scalars are delta_prep_kernel's
    if (nck > 0) {
      load_x(0);
      load_m(0);
      load_p(0);
    }
    for (int ck = 0; ck < nck; ++ck) {
      const uint32_t par = (uint32_t)ck & 1u;
      const uint32_t kt = sb + L::kq + par * L::place;
      const int valid = len - ck * kDC;
      const bool more = ck + 1 < nck;
      if (!wait(L::kK + (int)par, (uint32_t)(ck >> 1) & 1u)) break;
      if (valid < kDC && ck * kDC + valid < a.L) {  // the row ends inside the tensor: what follows is not its own
        for (int i = 0; i < kp; ++i) tok_clear(kt + i * kPanel, 1, valid, lane);
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
      if (more) load_kq(ck + 1);  // its place was read by the chunk before, whose state has been stored
      if (more && ck == 0) load_x(1);
      if (ck > 0) {
        if (!wait(L::kO, par ^ 1u)) break;  // o of the chunk before is staged: its scalars and P have been read
        store_o(ck - 1);
        load_p(ck);
        if (more) load_x(ck + 1);
      }
      if (elect_one()) {
        tc_fence_after_sync();
#pragma unroll 1
        for (int n = UT - 1; n >= 0; --n)
#pragma unroll 4
          for (int s = 0; s < ks; ++s)
            mma_ts(tm + L::D2, tm + L::S + n * (KP / 2) + s * 8, rows_desc(kt, kPanel, s, kDC), mma_idesc(kDC, false, false), n < UT - 1 || s > 0);
      }
      __syncwarp();
      if (!wait(L::kMr, par) || !wait(L::kW, 0u)) break;
      if (elect_one()) {
        tc_fence_after_sync();
        lower(sb + L::m, 0x041852u, 6,  // (left, right): (2, 0) (1, 1) (0, 2) (1, 0) (0, 1) (0, 0)
              [&](uint32_t l, int s, uint64_t r, uint32_t id, bool add) { mma_ts(tm + L::D1 + 16 * s, tm + L::W + l * 32 + s * 8, r, id, add); });
        bulk_wait_read();  // o has left: u may be stored once D3 is done
        mma_commit(&bar[L::kD3]);
      }
      __syncwarp();
      if (more) load_v(ck + 1);
      if (!wait(L::kW, 1u)) break;
      if (more) load_m(ck + 1);  // (D3 has been read)
      if (elect_one()) {
        tc_fence_after_sync();
#pragma unroll 1
        for (int n = 2; n >= 0; --n)
#pragma unroll
          for (int s = 0; s < 4; ++s)
            mma_ts(tm + L::D5, tm + L::W + n * 32 + s * 8, cols_desc(kt, kPanel, s), mma_idesc(KP, false, true), n < 2 || s > 0);
        mma_commit(&bar[L::kD5]);
      }
      __syncwarp();
      // (D4's place is that of w, which D5 reads; the wait costs 0.5 % of 4 x 2048 tokens, 1.7 % of 1 x 16384)
      if (!wait(L::kPr, par) || !wait(L::kU, par) || !wait(L::kD5, par)) break;
      if (elect_one()) {
        tc_fence_after_sync();
        lower(sb + L::p, 0x041852u, 6,
              [&](uint32_t l, int s, uint64_t r, uint32_t id, bool add) {
                mma_ss(tm + L::D4 + 16 * s, rows_desc(sb + L::u + l * kPanel, kPanel, s), r, id, add);
              });
        mma_commit(&bar[L::kD4]);
      }
      __syncwarp();
    }
    if (ok && nck > 0 && wait(L::kO, (uint32_t)(nck - 1) & 1u)) store_o(nck - 1);
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
      const float* src = h0 + (bh * a.K + kk) * a.V + row;
      S[e / 2] = h0 != nullptr && mine && kk < a.K ? f2(src[0], src[a.V]) : f2(0.f, 0.f);
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
    auto save = [&](int ck) {  // the state entering chunk ck: [K / 4][V][4], so that a warp's vectors follow one another
      float4* dst = reinterpret_cast<float4*>(ckpt + (long long)ck * a.K * a.V) + row;
#pragma unroll
      for (int e = 0; e < SC; e += 4)
        if (cq * SC + e < a.K) dst[(long long)((cq * SC + e) / 4) * a.V] = make_float4(S[e / 2].x, S[e / 2].y, S[e / 2 + 1].x, S[e / 2 + 1].y);
    };
    if (nck > 0) {
#pragma unroll
      for (int c = 0; c < SC; c += 16) store_s(c);
      tmem_wait_st();
      arrive(L::kS);
    }
    const uint32_t vcol = col_at(sb + L::v, row) + cq * TC * 128, ocol = col_at(sb + L::u, row) + cq * TC * 128;
    const uint32_t uat = sb + L::u + unit_at(kPanel, row, cq * (TC / 8));  // a unit of 8 tokens; the next is at ^ 16
    auto store_w = [&](int u, float2 (&x)[4]) {  // eight tokens as three terms
#pragma unroll
      for (int n = 0; n < 3; ++n) {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = n < 2 ? take_pair(x[e]) : last_pair(x[e]);
        tmem_st4(tl + L::W + n * 32 + cq * (TC / 2) + 4 * u, w);
      }
    };
    auto arrive_w = [&] {
      tmem_wait_st();
      arrive(L::kW);
    };
    float2 R[TC / 2];
    auto read_v = [&](int ck) {  // v of this thread's column, its tokens
      if (!wait(L::kV, (uint32_t)ck & 1u)) return false;
      ColRead<TC>::go(vcol, R);
      if (len - ck * kDC < kDC) {
#pragma unroll
        for (int e = 0; e < TC; ++e)
          if (cq * TC + e >= len - ck * kDC) (e & 1 ? R[e / 2].y : R[e / 2].x) = 0.f;
      }
      return true;
    };
    // r and o of a chunk, [16][V][4]: this thread's first vector
    float4* keep = nullptr;
    if (TRAIN) {
      ckpt += bh * delta_ckpt_floats(a.nck, a.K, a.V);
      keep = reinterpret_cast<float4*>(ckpt + (long long)(a.nck + 1) * a.K * a.V) + (long long)(cq * TC / 4) * a.V + row;
    }
    if (nck > 0) read_v(0);
    for (int ck = 0; ck < nck && ok; ++ck) {
      const uint32_t par = (uint32_t)ck & 1u;
      const float* vec = reinterpret_cast<const float*>(raw + L::vec + par * kDVec * 4) + cq * TC;
      float4* rs = keep + (long long)ck * (kDC / 4) * a.V;
      if (!wait(L::kX + (int)par, (uint32_t)(ck >> 1) & 1u)) break;
      if (ck > 0 && !wait(L::kO, par ^ 1u)) break;  // D4, in w's place, has been read
      if (!wait(L::kD1, par)) break;
      tc_fence_after_sync();
      {
        uint32_t d[16];
        tmem_ld16(tl + L::D1 + cq * TC, d);
        tmem_done(d);
#pragma unroll
        for (int u = 0; u < TC / 8; ++u) {
          float2 in[4], be[4], x[4];
          pairs4(vec + 8 * u, in);
          pairs4(vec + 2 * kDC + 8 * u, be);
#pragma unroll
          for (int z = 0; z < 4; ++z) {
            const int e = 4 * u + z;
            R[e] = fma2(mul2(in[z], bc2(-1.f)), u2f(d[2 * e], d[2 * e + 1]), R[e]);
            x[z] = mul2(be[z], R[e]);
          }
          store_w(u, x);
        }
      }
      arrive_w();
      if (!wait(L::kD3, par)) break;
      tc_fence_after_sync();
      {
        uint32_t d[16];
        tmem_ld16(tl + L::D1 + cq * TC, d);
        tmem_done(d);
#pragma unroll
        for (int u = 0; u < TC / 8; ++u) {
          float2 re[4], be[4], x[4];
          pairs4(vec + kDC + 8 * u, re);
          pairs4(vec + 2 * kDC + 8 * u, be);
#pragma unroll
          for (int z = 0; z < 4; ++z) {
            const int e = 4 * u + z;
            R[e] = fma2(u2f(d[2 * e], d[2 * e + 1]), bc2(-1.f), R[e]);
            if (TRAIN && mine && (z & 1)) rs[(long long)(2 * u + z / 2) * a.V] = make_float4(R[e - 1].x, R[e - 1].y, R[e].x, R[e].y);
            x[z] = mul2(be[z], R[e]);
            if (z & 1) {
              R[e - 1] = x[z - 1];
              R[e] = x[z];
            }
          }
#pragma unroll
          for (int z = 0; z < 4; ++z) x[z] = mul2(re[z], x[z]);
          store_w(u, x);
        }
      }
      arrive_w();
#pragma unroll
      for (int u = 0; u < TC / 8; ++u) {
        float2 x[4] = {R[4 * u], R[4 * u + 1], R[4 * u + 2], R[4 * u + 3]};
        put_terms<UT>(uat ^ (16u * u), kPanel, x);
      }
      arrive(L::kU);
      if (TRAIN && mine) save(ck);
      const float whole = vec[4 * kDC - cq * TC];
      if (ck + 1 < nck && !read_v(ck + 1)) break;  // (u has been stored)
      if (!wait(L::kD5, par)) break;
      tc_fence_after_sync();
#pragma unroll
      for (int c = 0; c < SC; c += 16) {
        uint32_t d[16];
        tmem_ld16(tl + L::D5 + cq * SC + c, d);
        tmem_done(d);
#pragma unroll
        for (int e = 0; e < 8; ++e) S[c / 2 + e] = fma2(S[c / 2 + e], bc2(whole), u2f(d[2 * e], d[2 * e + 1]));
        if (ck + 1 < nck) store_s(c);
      }
      if (ck + 1 < nck) {
        tmem_wait_st();
        arrive(L::kS);
      }
      if (!wait(L::kD4, par)) break;
      tc_fence_after_sync();
      {  // o into u's place, tokens as rows; the issuing warp sends it from there
        uint32_t d[16], f[16];
        tmem_ld16(tl + L::D2 + cq * TC, d);
        tmem_ld16(tl + L::D4 + cq * TC, f);
        tmem_done(d);
        tmem_done(f);
        float2 y[TC / 2];
#pragma unroll
        for (int u = 0; u < TC / 8; ++u) {
          float2 in[4];
          pairs4(vec + 8 * u, in);
#pragma unroll
          for (int z = 0; z < 4; ++z) {
            const int e = 4 * u + z;
            y[e] = fma2(mul2(bc2(a.scale), in[z]), u2f(d[2 * e], d[2 * e + 1]), u2f(f[2 * e], f[2 * e + 1]));
          }
        }
        if (len - ck * kDC < kDC) {
#pragma unroll
          for (int e = 0; e < TC; ++e)
            if (cq * TC + e >= len - ck * kDC) (e & 1 ? y[e / 2].y : y[e / 2].x) = 0.f;
        }
        ColWrite<TC>::go(ocol, y);
        if (TRAIN && mine) {
          float4* os = rs + (long long)a.nck * (kDC / 4) * a.V;
#pragma unroll
          for (int e = 0; e < TC / 2; e += 2) os[(long long)(e / 2) * a.V] = make_float4(y[e].x, y[e].y, y[e + 1].x, y[e + 1].y);
        }
      }
      arrive(L::kO);
    }
    if (ok && mine) {
      if (TRAIN) save(nck);
      if (h_last != nullptr) {
#pragma unroll
        for (int e = 0; e < SC; ++e)
          if (cq * SC + e < a.K) h_last[(bh * a.K + cq * SC + e) * a.V + row] = e & 1 ? S[e / 2].y : S[e / 2].x;
      }
    }
  }
  // tokens of chunks past the row's end
  const int n = a.V / 8;
  for (long long i = (long long)nck * kDC * n + tid; i < (long long)a.L * n; i += kDThreads)
    *reinterpret_cast<uint4*>(o + (((long long)b * a.L + i / n) * a.H + h) * a.V + i % n * 8) = make_uint4(0u, 0u, 0u, 0u);
  lin_leave(ok, bar, L::nbar, tm, L::cols, warp, lane);
}

template <int KP, bool TRAIN>
int walk(const Delta& p, const float* h0, __nv_bfloat16* o, float* ckpt, float* h_last, cudaStream_t s) {
  const LinAttn& a = p.a;
  DeltaMaps maps;
  if (!delta_map(&maps.q, a.q, a.ldq, a.B, a.L, a.G, a.K) || !delta_map(&maps.k, a.k, a.ldk, a.B, a.L, a.G, a.K) ||
      !delta_map(&maps.v, a.v, a.ldv, a.B, a.L, a.H, a.V) || !delta_map(&maps.o, o, (long long)a.H * a.V, a.B, a.L, a.H, a.V))
    return SS_ERR_CUDA;
  return delta_launch_next(delta_fwd_tc_kernel<KP, TRAIN>, (unsigned)((long long)a.B * a.H), kDThreads, DeltaTc<KP>::bytes, s, p, maps, h0, o,
                    ckpt, h_last);
}

}  // namespace

int ssh::delta_fwd_bf16(const Delta& p, const float* h0, void* o, float* ckpt, float* h_last, cudaStream_t s) {
  __nv_bfloat16* ob = static_cast<__nv_bfloat16*>(o);
  if (ckpt != nullptr) return p.a.K <= 64 ? walk<64, true>(p, h0, ob, ckpt, h_last, s) : walk<128, true>(p, h0, ob, ckpt, h_last, s);
  return p.a.K <= 64 ? walk<64, false>(p, h0, ob, ckpt, h_last, s) : walk<128, false>(p, h0, ob, ckpt, h_last, s);
}

namespace ssh {
int read_clear_delf_err(cudaStream_t s, unsigned* out) { return read_clear_lin_err(s, out); }
}  // namespace ssh
