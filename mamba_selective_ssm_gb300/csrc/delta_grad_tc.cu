// The gated delta rule's other gradients, bf16, chunk by chunk on tcgen05 (delta_tc.cuh).  Each (batch row, head, chunk) has
// the state S0 that enters it, its r and o (from the forward), the gradient dS of the state that leaves it and its du (from
// the backward chain); u = beta r, dR = beta du.
//   dbeta = <du, r>      dg_t = sum_{s >= t} (do_s.o_s - dR_s.v_s) + <S1, dS>           along columns of V, in fp32
// In this dg each token's own write cancels, which leaves an error of 3e-7 of the terms, and dg is e^{g_t} of them.  A token that
// forgets (g_t below kForget) takes the sum of what crosses it instead, as the fp32 kernel does (delta_bwd.cu), of the products
// below: their operands of two terms leave 2 to 4e-6 of dg at any g, the other form 9e-7 at g = -1, 3e-6 at -2, 3e-5 at -4 and
// all at -14.  If every chunk has such a token the kernel takes 505 us for 420; chunks without one skip the work.
//   E = scale D do u^T,  F = -D dR u^T (strict)                                          [t, s]
//   dq = scale e^c do S0^T + E K      dk = -e^c dR S0^T + e^{c_last - c} u dS^T + E^T Q + (F + F^T) K
// dq and dk are rounded to bf16; their fp32 operands are two rounded bf16 terms (2^-16).  Products run with the columns of K as the
// 128 rows of an MMA; S0, dS, u and dR lie in shared memory by columns of V, as they come from memory, and are contracted down
// their rows.  4 x 2048 tokens of 32 heads of 128 x 128: 420 us, 3.2 TB/s.  A CTA an SM (210 KB; tensor memory is taken whole),
// whose steps wait for one another: the sums and operands along V a third of a chunk's time, the states' loads and terms a third.
// A CTA for each chunk took 438 us, and where the heads' parts are added up (32 heads on 4, 128 x 64) 384 for 346.
#include <algorithm>

#include "delta_tc.cuh"

namespace {

using namespace ssk;

constexpr int kGT = 512, kGGrid = 152;  // a CTA an SM, which goes from chunk to chunk
constexpr float kForget = -2.f;  // where the two forms of dg are off by the same
template <int KP>
struct GradTc {
  static constexpr int NKP = KP / 64, ST = NKP * kPanel;  // bytes of a term of a state
  static constexpr int S = 0, u = S + 2 * ST, r = u + 2 * kPanel, dy = r + 2 * kPanel, k = dy + 2 * kTok, q = k + NKP * kTok, e = q + NKP * kTok,
                       f = e + 2 * kDTerm, vec = f + 2 * kDTerm, dec = vec + kDVec * 4, red = dec + 2 * kDC * 4, fg = red + (16 * 8 + 32) * 4,
                       bar = fg + 4 * 4;
  static constexpr int v = e;  // (v's tile, before E and F)
  static constexpr int x = r, cross = r + kPanel;  // X, and the sums of a, b and X, where dR's terms were
  static constexpr int kIn = 0, kM0 = 1, kM1 = 2, nbar = 3, tm = bar + nbar * 8, bytes = tm + 8;
  // tensor memory: do S0^T, dR S0^T, u dS^T, E, F, E K, E^T Q + (F + F^T) K; before the last two in their places q k^T, k k^T
  static constexpr int G1 = 0, G2 = 64, G3 = 128, E = 192, F = 256, H1 = 320, H2 = 384, QK = H1, KK = H2, cols = 512;
};

struct GradMaps {
  CUtensorMap q, k, v, dy, dq, dk;
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
  const long long items = (long long)a.B * a.H * a.nck, ldg = (long long)heads * a.K;
  float *vec = reinterpret_cast<float*>(raw + L::vec), *dec = reinterpret_cast<float*>(raw + L::dec), *red = reinterpret_cast<float*>(raw + L::red);
  const int kp = (a.K + 63) / 64, vp = (a.V + 63) / 64, vb = (a.V + 15) / 16;
  const int row = (warp & 3) * 32 + lane, cq = warp >> 2;  // a column of V (or of K, or a token), a quarter of the other axis
  const bool mine = row < a.V;
  auto valid_of = [&](long long it) {  // tokens of a chunk within their row
    const int n = a.len((int)(it / a.nck / a.H)) - (int)(it % a.nck) * kDC;
    return n < 0 ? 0 : n < kDC ? n : kDC;
  };
  auto following = [&](long long it) {  // this CTA's next chunk that holds a token
    while (it < items && valid_of(it) == 0) it += gridDim.x;
    return it;
  };
  auto load = [&](long long it) {  // one thread: a chunk's do, v, k, q
    const long long bh = it / a.nck;
    const int h = (int)(bh % a.H), b = (int)(bh / a.H), gh = h / (a.H / a.G), t0 = (int)(it % a.nck) * kDC;
    mbar_arrive_expect_tx(&bar[L::kIn], 2 * (kp + vp) * kTok);
    tok_load(sb + L::dy, vp, &maps.dy, &bar[L::kIn], h, t0, b);
    tok_load(sb + L::v, vp, &maps.v, &bar[L::kIn], h, t0, b);
    tok_load(sb + L::k, kp, &maps.k, &bar[L::kIn], gh, t0, b);
    tok_load(sb + L::q, kp, &maps.q, &bar[L::kIn], gh, t0, b);
  };
  auto marks = [&](long long it) {  // the forward's states, and after them r and o, of a chunk's batch row and head
    return ckpt + it / a.nck * delta_ckpt_floats(a.nck, a.K, a.V);
  };
  // r, o and du of a chunk towards L2, a line of 128 bytes at a time, under the first products; its states under the second.  (427 us
  // without the states or with r, o and du asked for earlier, 415 so; all of it before this chunk's own loads: 481.)
  auto states_ahead = [&](long long it) {
    const float* st = marks(it) + it % a.nck * a.K * a.V;
    for (int i = tid; i < a.K * a.V / 32; i += kGT) {
      prefetch_l2(st + i * 32);
      prefetch_l2(dS + it * a.K * a.V + i * 32);
    }
  };
  auto ahead = [&](long long it) {
    const long long ck = it % a.nck;
    const float* ro = marks(it) + (long long)(a.nck + 1) * a.K * a.V + ck * kDC * a.V;
    for (int i = tid; i < kDC * a.V / 32; i += kGT) {
      prefetch_l2(ro + i * 32);
      prefetch_l2(ro + (long long)a.nck * kDC * a.V + i * 32);
      prefetch_l2(du + it * kDC * a.V + i * 32);
    }
    if (tid < kDVec / 32) prefetch_l2(p.vec + it * kDVec + tid * 32);
  };
  if (tid == 0) {
    for (int i = 0; i < L::nbar; ++i) mbar_init(&bar[i], 1);
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
  const uint32_t tl = tm + ((uint32_t)((warp & 3) * 32) << 16);
  bool ok = true;
  {
    const long long first = following(blockIdx.x);
    if (first < items) {
      if (tid == 0) load(first);
      pdl_wait();  // dS and du are delta_back_tc_kernel's
      ahead(first);
    } else {
      pdl_wait();
    }
  }
  uint32_t par = 0;
  uint32_t* forgets = reinterpret_cast<uint32_t*>(raw + L::fg);  // a chunk's tokens that forget: the even ones, the odd ones
  float *X = reinterpret_cast<float*>(raw + L::x), *as = reinterpret_cast<float*>(raw + L::cross), *bs = as + 4 * kDC, *xs = bs + 4 * kDC;
  auto xat = [](int t, int s) { return t * kDC + (s ^ ((t & 7) << 2)); };
  // a warp's sums of sixteen tokens over its lanes: token lane % 16 of them ends in x[0]
  auto lanes_tokens = [&](float (&x)[TC]) {
#pragma unroll
    for (int n = TC / 2; n > 0; n >>= 1) {
      const bool upper = lane & n;
#pragma unroll
      for (int e = 0; e < n; ++e) {
        const float keep = upper ? x[e + n] : x[e], give = upper ? x[e] : x[e + n];
        x[e] = keep + __shfl_xor_sync(0xffffffffu, give, n);
      }
    }
    x[0] += __shfl_xor_sync(0xffffffffu, x[0], TC);
  };
  for (long long item = blockIdx.x; item < items && ok; item += gridDim.x) {
    const long long bh = item / a.nck;
    const int ck = (int)(item % a.nck), h = (int)(bh % a.H), b = (int)(bh / a.H), gh = h / (a.H / a.G);
    const int t0 = ck * kDC, rows = a.L - t0 < kDC ? a.L - t0 : kDC, valid = valid_of(item);
    const long long tok = (long long)b * a.L + t0;
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
      continue;
    }
    const long long next = following(item + gridDim.x);
    const float* base = marks(item);
    const float4* s0 = reinterpret_cast<const float4*>(base + (long long)ck * a.K * a.V) + row;
    const float4* s1 = s0 + (long long)a.K * a.V / 4;
    // r, o and du of this warp's four tokens: [V] vectors of four
    const float4* rr = reinterpret_cast<const float4*>(base + (long long)(a.nck + 1) * a.K * a.V + (long long)ck * kDC * a.V) + warp * a.V;
    const float4* oo = rr + (long long)a.nck * kDC * a.V / 4;
    const float4* uu = reinterpret_cast<const float4*>(du + item * kDC * a.V) + warp * a.V;
    if (const int i = tid - (kGT - kDVec / 4); i >= 0)
      reinterpret_cast<float4*>(vec)[i] = __ldcg(reinterpret_cast<const float4*>(p.vec + item * kDVec) + i);
    if (warp == 4) {
      ChunkGates<kDC> gates;
      if (a.g != nullptr) gates.fetch(a, b, h, t0, t0 + valid, lane);
      else gates.g[0] = gates.g[1] = 0.f;
      gates.scan(lane, [&](int i, Dec e) { dec[i] = e.hi; dec[kDC + i] = e.lo; });
      const uint32_t even = __ballot_sync(0xffffffffu, gates.g[0] < kForget), odd = __ballot_sync(0xffffffffu, gates.g[1] < kForget);
      if (lane == 0) {
        forgets[0] = even;
        forgets[1] = odd;
      }
    }
    __syncthreads();
    const uint32_t forget[2] = {forgets[0], forgets[1]};
    const bool crossing = (forget[0] | forget[1]) != 0u;
    auto state = [&](const float4* src, float4 (&x)[SC / 4]) {
#pragma unroll
      for (int e = 0; e < SC / 4; ++e)
        x[e] = mine && cq * SC + 4 * e < a.K ? __ldcg(src + (long long)(cq * (SC / 4) + e) * a.V) : make_float4(0.f, 0.f, 0.f, 0.f);
    };
    float4 X4[SC / 4];
    state(s0, X4);
    ok = chain_wait(&bar[L::kIn], par);
    if (valid < kDC && t0 + valid < a.L) {  // the row ends inside the tensor: what follows is not its own
      if (warp == 0) tok_clear(sb + L::dy, vp, valid, lane);
      if (warp == 1) tok_clear(sb + L::k, kp, valid, lane);
      if (warp == 2) tok_clear(sb + L::q, kp, valid, lane);
      __syncthreads();
    }
    // ---- along columns of V: u, dR and the sums.  A warp takes four tokens and all of V
    float sums[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};  // dbeta's and dg's of the four
    {
      const float4 be = *reinterpret_cast<const float4*>(vec + 2 * kDC + 4 * warp);
      const bool on[4] = {4 * warp < valid, 4 * warp + 1 < valid, 4 * warp + 2 < valid, 4 * warp + 3 < valid};
#pragma unroll 2
      for (int c = lane; c < 16 * vb; c += 32) {
        const bool in = c < a.V;
        const float4 z4 = make_float4(0.f, 0.f, 0.f, 0.f);
        const float4 r4 = in ? __ldcs(rr + c) : z4, d4 = in ? __ldcs(uu + c) : z4, o4 = in ? __ldcs(oo + c) : z4;
        const uint32_t at = (uint32_t)((c >> 6) * kTok + (((c >> 3) & 7) << 4) + (c & 7) * 2) + warp * 512;
        float y[4], v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {  // tokens 4 warp + e: their rows' swizzle is (4 (warp & 1) + e)
          const uint32_t to = (at ^ ((4 * (warp & 1) + e) << 4)) + e * 128;
          uint16_t p0, p1;
          asm volatile("ld.shared.u16 %0, [%1];" : "=h"(p0) : "r"(sb + L::dy + to) : "memory");
          asm volatile("ld.shared.u16 %0, [%1];" : "=h"(p1) : "r"(sb + L::v + to) : "memory");
          y[e] = bf16_lo(p0);
          v[e] = bf16_lo(p1);
        }
        const float2 u0 = f2(be.x * r4.x, be.y * r4.y), u1 = f2(be.z * r4.z, be.w * r4.w);
        const float2 d0 = f2(be.x * d4.x, be.y * d4.y), d1 = f2(be.z * d4.z, be.w * d4.w);
        sums[0] = fmaf(d4.x, r4.x, sums[0]);
        sums[1] = fmaf(d4.y, r4.y, sums[1]);
        sums[2] = fmaf(d4.z, r4.z, sums[2]);
        sums[3] = fmaf(d4.w, r4.w, sums[3]);
        if (on[0]) sums[4] += fmaf(y[0], o4.x, -d0.x * v[0]);  // (past the row's end v may be anything)
        if (on[1]) sums[5] += fmaf(y[1], o4.y, -d0.y * v[1]);
        if (on[2]) sums[6] += fmaf(y[2], o4.z, -d1.x * v[2]);
        if (on[3]) sums[7] += fmaf(y[3], o4.w, -d1.y * v[3]);
        const uint32_t w = (uint32_t)(c * 128 + (((warp >> 1) ^ (c & 7)) << 4) + (warp & 1) * 8);
        auto put = [&](uint32_t tile, float2 x, float2 z) {
          const uint32_t a0 = round_pair(x), a1 = round_pair(z);
          asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(tile + w), "r"(a0), "r"(a1) : "memory");
          asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(tile + kPanel + w), "r"(pack_bf16(x.x, x.y)), "r"(pack_bf16(z.x, z.y)) : "memory");
        };
        put(sb + L::u, u0, u1);
        put(sb + L::r, d0, d1);
      }
    }
    auto put_state = [&](const float4 (&x)[SC / 4]) {  // two terms, [V][K]
      if (row >= 16 * vb) return;
#pragma unroll
      for (int e = 0; e < SC / 8; ++e) {
        const float4 l = x[2 * e], u = x[2 * e + 1];
        float2 y[4] = {f2(l.x, l.y), f2(l.z, l.w), f2(u.x, u.y), f2(u.z, u.w)};
        put_terms<2>(sb + L::S + unit_at(kPanel, row, cq * (SC / 8) + e), L::ST, y);
      }
    };
    // sums over the lanes: each of the first three steps adds a half of the values to the other lane's and keeps the half
#pragma unroll
    for (int n = 4; n > 0; n >>= 1) {
      const bool upper = lane & n;
#pragma unroll
      for (int e = 0; e < n; ++e) {
        const float keep = upper ? sums[e + n] : sums[e], give = upper ? sums[e] : sums[e + n];
        sums[e] = keep + __shfl_xor_sync(0xffffffffu, give, n);
      }
    }
    sums[0] += __shfl_xor_sync(0xffffffffu, sums[0], 8);
    sums[0] += __shfl_xor_sync(0xffffffffu, sums[0], 16);
    if (lane < 8) red[warp * 8 + lane] = sums[0];
    put_state(X4);
    fence_proxy_async_smem();
    __syncthreads();
    if (warp == 0) {
      if (elect_one()) {
        const uint32_t ic = mma_idesc(64, true, false), cc = mma_idesc(64, true, true), rc = mma_idesc(64, false, true);
#pragma unroll 1
        for (int n = 1; n >= 0; --n)
#pragma unroll 1
          for (int s = 0; s < vb; ++s) {
            mma_ss(tm + L::E, rows_desc(sb + L::dy, kTok, s), cols_desc(sb + L::u + n * kPanel, kPanel, s), rc, n < 1 || s > 0);
            mma_ss(tm + L::G1, cols_desc(sb + L::S + n * L::ST, kPanel, s), rows_desc(sb + L::dy, kTok, s), ic, n < 1 || s > 0);
          }
#pragma unroll 1
        for (int n = 0; n < 3; ++n) {  // (1, 0) (0, 1) (0, 0)
          const int i = n == 0, j = n == 1;
#pragma unroll 1
          for (int s = 0; s < vb; ++s) {
            mma_ss(tm + L::F, cols_desc(sb + L::r + i * kPanel, kPanel, s), cols_desc(sb + L::u + j * kPanel, kPanel, s), cc, n > 0 || s > 0);
            mma_ss(tm + L::G2, cols_desc(sb + L::S + i * L::ST, kPanel, s), cols_desc(sb + L::r + j * kPanel, kPanel, s), cc, n > 0 || s > 0);
          }
        }
        if (crossing) {
          const uint32_t rr = mma_idesc(64, false, false);
#pragma unroll 1
          for (int s = 0; s < (a.K + 15) / 16; ++s) {
            const uint64_t kd = rows_desc(sb + L::k, kTok, s);
            mma_ss(tm + L::QK, rows_desc(sb + L::q, kTok, s), kd, rr, s > 0);
            mma_ss(tm + L::KK, kd, kd, rr, s > 0);
          }
        }
        mma_commit(&bar[L::kM0]);
      }
      __syncwarp();
    }
    // ---- under the products: <S1, dS>, and dg and dbeta
    {
      float4 Y[SC / 4];
      auto dot = [&](int at) {
        float d = 0.f;
#pragma unroll
        for (int e = 0; e < SC / 4; ++e) d = fmaf(X4[e].x, Y[e].x, fmaf(X4[e].y, Y[e].y, fmaf(X4[e].z, Y[e].z, fmaf(X4[e].w, Y[e].w, d))));
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
        if (lane == 0) red[at + warp] = d;
      };
      state(s1, Y);
      state(reinterpret_cast<const float4*>(dS + item * a.K * a.V) + row, X4);
      dot(16 * 8);
      if (crossing) {
        state(s0, Y);
        dot(16 * 8 + 16);
      }
    }
    __syncthreads();
    if (warp == 15) {
      float s[2], x = 0.f;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int t = 2 * lane + i;
        const float d = red[(t >> 2) * 8 + (t & 3)];
        s[i] = red[(t >> 2) * 8 + 4 + (t & 3)];
        if (t < rows) dbeta[(tok + t) * a.H + h] = t < valid ? d : 0.f;
      }
      for (int w = 0; w < 16; ++w) x += red[16 * 8 + w];
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
    if (next < items) ahead(next);
    ok = chain_wait(&bar[L::kM0], par) && ok;
    tc_fence_after_sync();
    put_state(X4);  // dS where S0 was
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
        if (crossing) {
          uint32_t qk[8], kk[8];
          tmem_ld8u(tl + L::QK + cq * TC + 8 * u, qk);
          tmem_ld8u(tl + L::KK + cq * TC + 8 * u, kk);
          tmem_done(qk);
          tmem_done(kk);
          float w[8];
#pragma unroll
          for (int z = 0; z < 8; ++z)
            w[z] = cq * TC + 8 * u + z < row ? fmaf(z & 1 ? x[z / 2].y : x[z / 2].x, __uint_as_float(qk[z]),
                                                    (z & 1 ? y[z / 2].y : y[z / 2].x) * __uint_as_float(kk[z])) : 0.f;
          *reinterpret_cast<float4*>(X + xat(row, cq * TC + 8 * u)) = make_float4(w[0], w[1], w[2], w[3]);
          *reinterpret_cast<float4*>(X + xat(row, cq * TC + 8 * u + 4)) = make_float4(w[4], w[5], w[6], w[7]);
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
          for (int s = 0; s < vb; ++s)
            mma_ss(tm + L::G3, cols_desc(sb + L::S + i * L::ST, kPanel, s), cols_desc(sb + L::u + j * kPanel, kPanel, s), cc, n > 0 || s > 0);
        }
        mma_commit(&bar[L::kM1]);
      }
      __syncwarp();
    }
    if (next < items) states_ahead(next);
    if (crossing) {  // ---- under the products: a, and the sums of X over s < t <= i
      float sa[TC];
#pragma unroll
      for (int e = 0; e < TC; ++e) sa[e] = 0.f;
      if ((warp & 3) * 32 < a.K) {
        float2 qc[TC / 2], kc[TC / 2];
        ColRead<TC>::go(col_at(sb + L::q, row) + cq * TC * 128, qc);
        ColRead<TC>::go(col_at(sb + L::k, row) + cq * TC * 128, kc);
        tc_fence_after_sync();
#pragma unroll
        for (int c = 0; c < TC; c += 8) {
          uint32_t g1[8], g2[8];
          tmem_ld8u(tl + L::G1 + cq * TC + c, g1);
          tmem_ld8u(tl + L::G2 + cq * TC + c, g2);
          tmem_done(g1);
          tmem_done(g2);
          float2 in[4];
          pairs4(vec + cq * TC + c, in);
#pragma unroll
          for (int z = 0; z < 8; ++z) {
            const float qv = z & 1 ? qc[(c + z) / 2].y : qc[(c + z) / 2].x, kv = z & 1 ? kc[(c + z) / 2].y : kc[(c + z) / 2].x;
            sa[c + z] = (z & 1 ? in[z / 2].y : in[z / 2].x) * (a.scale * qv * __uint_as_float(g1[z]) - kv * __uint_as_float(g2[z]));
          }
        }
      }
      lanes_tokens(sa);
      if (lane < TC) as[(warp & 3) * kDC + cq * TC + lane] = sa[0];
      float run = 0.f;  // X[t][s] becomes its sum over the tokens from t to the end of t's eight
#pragma unroll
      for (int t = 7; t >= 0; --t) {
        float* at = X + xat(8 * (tid >> 6) + t, tid & 63);
        run += *at;
        *at = run;
      }
      __syncthreads();
      const int j = tid >> 3;
      float s = 0.f;
#pragma unroll 1  // (unrolled, its instructions cost every chunk 4 %, those that skip them too)
      for (int c = tid & 7; c < j; c += 8) {
        s += X[xat(j, c)];
#pragma unroll 1
        for (int later = (j >> 3) + 1; later < 8; ++later) s += X[xat(8 * later, c)];
      }
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      if ((tid & 7) == 0) xs[j] = s;
    }
    const float whole = vec[4 * kDC];
    ok = chain_wait(&bar[L::kM1], par) && ok;
    tc_fence_after_sync();
    if (crossing) {  // ---- b
      float sw[TC];
#pragma unroll
      for (int e = 0; e < TC; ++e) sw[e] = 0.f;
      if ((warp & 3) * 32 < a.K) {
        float2 kc[TC / 2];
        ColRead<TC>::go(col_at(sb + L::k, row) + cq * TC * 128, kc);
#pragma unroll
        for (int c = 0; c < TC; c += 8) {
          uint32_t g3[8];
          tmem_ld8u(tl + L::G3 + cq * TC + c, g3);
          tmem_done(g3);
          float2 re[4];
          pairs4(vec + kDC + cq * TC + c, re);
#pragma unroll
          for (int z = 0; z < 8; ++z)
            sw[c + z] = (z & 1 ? re[z / 2].y * kc[(c + z) / 2].y : re[z / 2].x * kc[(c + z) / 2].x) * __uint_as_float(g3[z]);
        }
      }
      lanes_tokens(sw);
      if (lane < TC) bs[(warp & 3) * kDC + cq * TC + lane] = sw[0];
      fence_proxy_async_smem();
      __syncthreads();  // (the columns of k and q were read before the copies that follow)
    }
    if (tid == 0 && next < items && ok) load(next);  // (their places have been read)
    par ^= 1u;
    constexpr bool kTile = sizeof(TO) == 2;  // bf16 leaves by TMA from tiles of tokens, where the states were
    if ((warp & 3) * 32 < a.K) {  // row = column of K, this warp's 16 tokens
      const uint32_t qat = col_at(sb + L::S, row) + cq * TC * 128;
      float2 xq[TC / 2], xk[TC / 2];
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
        float2 in[4], re[4];
        pairs4(vec + cq * TC + c, in);
        pairs4(vec + kDC + cq * TC + c, re);
#pragma unroll
        for (int z = 0; z < 4; ++z) {
          const int e = 2 * z;
          xq[c / 2 + z] = fma2(mul2(bc2(a.scale), in[z]), u2f(g1[e], g1[e + 1]), u2f(h1[e], h1[e + 1]));
          xk[c / 2 + z] = fma2(re[z], u2f(g3[e], g3[e + 1]), fma2(mul2(in[z], bc2(-1.f)), u2f(g2[e], g2[e + 1]), u2f(h2[e], h2[e + 1])));
        }
      }
      if (valid < kDC) {
#pragma unroll
        for (int e = 0; e < TC; ++e)
          if (cq * TC + e >= valid) {
            (e & 1 ? xq[e / 2].y : xq[e / 2].x) = 0.f;
            (e & 1 ? xk[e / 2].y : xk[e / 2].x) = 0.f;
          }
      }
      if constexpr (kTile) {
        ColWrite<TC>::go(qat, xq);
        ColWrite<TC>::go(qat + L::NKP * kTok, xk);
      } else if (row < a.K) {
#pragma unroll
        for (int e = 0; e < TC; ++e) {
          const int t = cq * TC + e;
          if (t < rows) {
            ActT<TO>::st1(dqb + (long long)t * ldg + row, e & 1 ? xq[e / 2].y : xq[e / 2].x);
            ActT<TO>::st1(dkb + (long long)t * ldg + row, e & 1 ? xk[e / 2].y : xk[e / 2].x);
          }
        }
      }
    }
    if constexpr (kTile) {
      fence_proxy_async_smem();
      __syncthreads();
      if (tid == 0) {
        for (int i = 0; i < kp; ++i) {
          tma_store_4d(&maps.dq, sb + L::S + i * kTok, i * 64, gh, t0, b);
          tma_store_4d(&maps.dk, sb + L::S + (L::NKP + i) * kTok, i * 64, gh, t0, b);
        }
        bulk_commit();
        bulk_wait_read();
      }
    }
    tc_fence_before_sync();
    ok = __syncthreads_and(ok);  // the sums, the scalars and the tiles have been read; all go on or none does
    tc_fence_after_sync();
    if (crossing && warp == 15) {  // (what it reads is written again behind the next chunk's first barrier)
      float after[2], before[2], x = 0.f;
      for (int w = 0; w < 16; ++w) x += red[16 * 8 + 16 + w];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int t = 2 * lane + i;
        after[i] = (as[t] + as[kDC + t]) + (as[2 * kDC + t] + as[3 * kDC + t]);
        before[i] = (bs[t] + bs[kDC + t]) + (bs[2 * kDC + t] + bs[3 * kDC + t]);
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
        const float y = ((i == 0 ? from : after[1] + rest) + (i == 0 ? past : past + before[0])) + fmaf(whole, x, xs[t]);
        if ((forget[i] >> lane & 1u) && t < valid) dg[(tok + t) * a.H + h] = y;
      }
    }
  }
  if (tid == 0) bulk_wait();
  lin_leave(ok, bar, L::nbar, tm, L::cols, warp, lane);
}

template <int KP, typename TO>
int run(const Delta& p, const float* ckpt, const void* dout, const float* dS, const float* du, void* dq, void* dk, float* dg, float* dbeta,
        cudaStream_t s) {
  const LinAttn& a = p.a;
  constexpr bool kTile = sizeof(TO) == 2;  // a group's own gradients; fp32: each head's parts
  const long long ldg = (long long)a.G * a.K;
  GradMaps maps{};
  if (!delta_map(&maps.q, a.q, a.ldq, a.B, a.L, a.G, a.K) || !delta_map(&maps.k, a.k, a.ldk, a.B, a.L, a.G, a.K) ||
      !delta_map(&maps.v, a.v, a.ldv, a.B, a.L, a.H, a.V) || !delta_map(&maps.dy, dout, (long long)a.H * a.V, a.B, a.L, a.H, a.V))
    return SS_ERR_CUDA;
  if (kTile && (!delta_map(&maps.dq, dq, ldg, a.B, a.L, a.G, a.K) || !delta_map(&maps.dk, dk, ldg, a.B, a.L, a.G, a.K)))
    return SS_ERR_CUDA;
  static_assert(GradTc<KP>::bytes <= 227 * 1024, "a chunk's tiles fit shared memory");
  const unsigned grid = (unsigned)std::min<long long>(kGGrid, (long long)a.B * a.H * a.nck);
  return delta_launch_next(delta_grad_tc_kernel<KP, TO>, grid, kGT, GradTc<KP>::bytes, s, p, maps, ckpt, dS, du, static_cast<TO*>(dq),
                           static_cast<TO*>(dk), kTile ? a.G : a.H, dg, dbeta);
}

}  // namespace

int ssh::delta_grad_bf16(const Delta& p, const float* ckpt, const void* dout, const float* dS, const float* du, void* dq, void* dk, bool parts,
                         float* dg, float* dbeta, cudaStream_t s) {
  auto go = [&](auto run) { return run(p, ckpt, dout, dS, du, dq, dk, dg, dbeta, s); };
  if (p.a.K <= 64) return parts ? go(run<64, float>) : go(run<64, __nv_bfloat16>);
  return parts ? go(run<128, float>) : go(run<128, __nv_bfloat16>);
}

namespace ssh {
int read_clear_delg_err(cudaStream_t s, unsigned* out) { return read_clear_lin_err(s, out); }
}  // namespace ssh
