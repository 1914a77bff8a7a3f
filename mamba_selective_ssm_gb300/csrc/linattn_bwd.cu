// Linear attention with a decay for each head, chunked backward (linattn_bwd) for sm_103a.
//
// With U = dL/dS of the state leaving a chunk, c_i its running log decay, and
//   P_ij = scale e^{c_i-c_j} (q_i.k_j),  dP_ij = scale e^{c_i-c_j} (do_i.v_j)     (j <= i)
// the chunk's gradients are
//   dq_i = sum_j dP_ij k_j + scale e^{c_i} S_in do_i
//   dk_j = sum_i dP_ij q_i + e^{c_last-c_j} U v_j
//   dv_j = sum_i P_ij do_i + e^{c_last-c_j} U^T k_j
//   U_in = e^{c_last} U + scale sum_i e^{c_i} q_i do_i^T
// and the gradient of a log decay counts every path that crosses it, a sum
// without cancelling terms (the difference of running sums of q.dq and k.dk is
// the same number, but loses what the sums have in common):
//   dg_t = sum_{j<t<=i} M_ij + sum_{i>=t} q_i.(scale e^{c_i} S_in do_i)
//        + sum_{j<t} k_j.(e^{c_last-c_j} U v_j) + e^{c_last} <S_in, U>,   M_ij = P_ij (do_i.v_j)
#include <stddef.h>

#include "linattn_tc.cuh"

namespace {

template <int KP, int VP>
struct BwdSmem {
  static constexpr int NT = 256;  // threads
  static constexpr int C = kLinChunkF32, LK = KP + 4, LV = VP + 4, LC = C + 4;
  float q[C * LK], d[C * LV], chi[C], clo[C], into[C], rest[C];
  float k[C * LK], v[C * LV], s[KP * LV], p[C * LC];  // (these not for a sum)
  float a[4 * C], b[4 * C], rect[C], red[8];  // a, b: by the warp columns of a C x KP product
};

struct BwdOut {
  void *dq, *dk, *dv;
  float *dqp, *dkp;  // fp32 per-head parts when heads share q, k (then dq, dk are summed from them)
  float* dg;         // [B, L, H], or per-chunk sums [B * nck, H] with a decay per head
  float* dh0;
};

// ---------------------------------------------------------------- fp32: three-product tf32
// A CTA walks the chunks of one (batch row, head, segment) from the last to the
// first with U in registers.  SUM only finds the segment's U from zero.
// Bound as the forward: 825 us (and 127 for the sums) for 8 x 2048 tokens of 24
// heads of 64 x 64, ten products a chunk for the forward's four.
template <int KP, int VP, bool SUM>
__global__ void __launch_bounds__(256, KP == 64 && VP == 64 ? 2 : 1) linattn_bwd_kernel(LinAttn p, const float* __restrict__ dout,
                                                                          const float* __restrict__ ckpt, const float* __restrict__ u0,
                                                                          BwdOut out, float* __restrict__ uend, Dec* __restrict__ udec) {
  using Sm = BwdSmem<KP, VP>;
  constexpr int C = Sm::C, LK = Sm::LK, LV = Sm::LV, LC = Sm::LC, NT = Sm::NT;
  extern __shared__ __align__(16) unsigned char raw[];
  Sm& sm = *reinterpret_cast<Sm*>(raw);
  const int tid = threadIdx.x;
  long long id = blockIdx.x;
  const int seg = (int)(id % p.nseg);
  id /= p.nseg;
  const int h = (int)(id % p.H), b = (int)(id / p.H);
  const int gh = h / (p.H / p.G);
  const int len = p.len(b);
  const long long bh = (long long)b * p.H + h, kv = (long long)p.K * p.V;
  const float* q = static_cast<const float*>(p.q) + (long long)b * p.L * p.ldq + (long long)gh * p.K;
  const float* k = static_cast<const float*>(p.k) + (long long)b * p.L * p.ldk + (long long)gh * p.K;
  const float* v = static_cast<const float*>(p.v) + (long long)b * p.L * p.ldv + (long long)h * p.V;
  const long long ldo = (long long)p.H * p.V;
  const float* d = dout + (long long)b * p.L * ldo + (long long)h * p.V;

  using State = Own<NT, KP, VP>;
  using TokK = Own<NT, C, KP>;
  using TokV = Own<NT, C, VP>;
  using Score = Own<NT, C, C>;
  State U;
  U.zero();
  if (u0 != nullptr && !SUM) {
    const float* src = u0 + (p.nseg > 1 ? bh * p.nseg + seg : bh) * kv;
    U.pairs(tid, [&](int kk, int vv, float& x, float& y) {
      if (kk < p.K && vv < p.V) {
        x = src[(long long)kk * p.V + vv];
        y = src[(long long)kk * p.V + vv + 1];
      }
    });
  }
  // gradients of q or k: typed when each head has its own, else this head's fp32 part
  auto put_qk = [&](void* typed, float* part, int t0, int rows, int valid, TokK& a) {
    float* dst = part != nullptr ? part : static_cast<float*>(typed);
    a.pairs(tid, [&](int i, int kk, float& x, float& y) {
      if (i < rows && kk < p.K)
        st_pair(dst + (((long long)b * p.L + t0 + i) * p.H + h) * p.K + kk, i < valid ? x : 0.f, i < valid ? y : 0.f);
    });
  };
  // a C x KP product's rows dotted with those of a tile, by warp column
  auto row_dots = [&](TokK& a, const float* tile, float* to) {
#pragma unroll
    for (int r = 0; r < TokK::RM; ++r) {
      const int i = TokK::row(tid, r);
      float s = 0.f;
#pragma unroll
      for (int c = 0; c < TokK::RN; ++c) s = fmaf(tile[i * LK + TokK::col(tid, c)], a.v[r][c], s);
      s = row_sum4(s);
      if ((tid & 3) == 0) to[TokK::wn(tid) * C + i] = s;
    }
  };
  Dec total = {0.f, 0.f};
  ChunkGates<C> gates;
  const int c0 = seg * p.cps, c1 = c0 + p.cps < p.nck ? c0 + p.cps : p.nck;
  if (tid < 32) gates.fetch(p, b, h, (c1 - 1) * C, len, tid);
  for (int ck = c1 - 1; ck >= c0; --ck) {
    const int t0 = ck * C;
    const int rows = p.L - t0 < C ? p.L - t0 : C;
    const int valid = len - t0 < 0 ? 0 : len - t0 < C ? len - t0 : C;
    if (valid == 0) {
      if (!SUM) {
        TokK z;
        z.zero();
        put_qk(out.dq, out.dqp, t0, rows, 0, z);
        put_qk(out.dk, out.dkp, t0, rows, 0, z);
        for (int i = tid; i < rows * p.V; i += NT)
          static_cast<float*>(out.dv)[(((long long)b * p.L + t0 + i / p.V) * p.H + h) * p.V + i % p.V] = 0.f;
        if (p.g_head) {
          if (tid == 0) out.dg[((long long)b * p.nck + ck) * p.H + h] = 0.f;
        } else if (tid < rows) {
          out.dg[((long long)b * p.L + t0 + tid) * p.H + h] = 0.f;
        }
      }
      if (tid < 32) gates.fetch(p, b, h, t0 - C, len, tid);
      continue;
    }
    load_tile<NT, C, KP, LK>(q + t0 * p.ldq, p.ldq, valid, p.K, sm.q, tid);
    load_tile<NT, C, VP, LV>(d + t0 * ldo, ldo, valid, p.V, sm.d, tid);
    if (!SUM) {
      load_tile<NT, C, KP, LK>(k + t0 * p.ldk, p.ldk, valid, p.K, sm.k, tid);
      load_tile<NT, C, VP, LV>(v + t0 * p.ldv, p.ldv, valid, p.V, sm.v, tid);
      const float* src = ckpt + (bh * p.nck + ck) * kv;
      for (int i = tid; i < KP * (VP / 4); i += NT) {
        const int kk = i / (VP / 4), vv = i % (VP / 4) * 4;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (kk < p.K && vv < p.V) x = *reinterpret_cast<const float4*>(src + (long long)kk * p.V + vv);
        *reinterpret_cast<float4*>(sm.s + kk * LV + vv) = x;
      }
    }
    if (tid < 32) {
      gates.scan(tid, [&](int i, Dec e) { sm.chi[i] = e.hi; sm.clo[i] = e.lo; });
      __syncwarp();
      for (int i = tid; i < C; i += 32) {
        sm.into[i] = p.scale * dec_exp(sm.chi[i], sm.clo[i]);
        sm.rest[i] = dec_diff(sm.chi[C - 1], sm.clo[C - 1], sm.chi[i], sm.clo[i]);
      }
      gates.fetch(p, b, h, t0 - C, len, tid);
    }
    __syncthreads();
    const float chi = sm.chi[C - 1], clo = sm.clo[C - 1];
    total = dec_add(total, Dec{chi, clo});
    Score m;  // what dg's rectangle sums are taken from
    if (!SUM) {
      float part = 0.f;  // <S_in, U>
      U.pairs(tid, [&](int kk, int vv, float& x, float& y) {
        const float2 s = *reinterpret_cast<const float2*>(sm.s + kk * LV + vv);
        part = fmaf(s.x, x, fmaf(s.y, y, part));
      });
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) part += __shfl_xor_sync(0xffffffffu, part, o);
      if ((tid & 31) == 0) sm.red[tid >> 5] = part;
      TokK dq;
      dq.zero();
      mm<false, true, LV, LV, VP>(sm.d, sm.s, dq, tid);
      dq.scale_rows(tid, [&](int i) { return sm.into[i]; });
      row_dots(dq, sm.q, sm.a);
      Score pr;
      m.zero();
      pr.zero();
      mm<false, true, LV, LV, VP>(sm.d, sm.v, m, tid);
      mm<false, true, LK, LK, KP>(sm.q, sm.k, pr, tid);
#pragma unroll
      for (int r = 0; r < Score::RM; ++r) {
        const int i = Score::row(tid, r);
        const float hi = sm.chi[i], lo = sm.clo[i];
#pragma unroll
        for (int c = 0; c < Score::RN; c += 2) {
          const int j = Score::col(tid, c);
          float dp[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const bool in = j + e <= i;
            const float w = in ? p.scale * dec_diff(hi, lo, sm.chi[j + e], sm.clo[j + e]) : 0.f;
            float &x = m.v[r][c + e], &y = pr.v[r][c + e];
            y = in ? y * w : 0.f;
            dp[e] = in ? x * w : 0.f;
            x = in ? x * y : 0.f;
          }
          st_pair(sm.p + i * LC + j, dp[0], dp[1]);
        }
      }
      __syncthreads();
      mm<false, false, LC, LK, C>(sm.p, sm.k, dq, tid);
      put_qk(out.dq, out.dqp, t0, rows, valid, dq);
      TokK dk;
      dk.zero();
      mm<true, false, LC, LK, C>(sm.p, sm.q, dk, tid);
      __syncthreads();
      pr.pairs(tid, [&](int i, int j, float& x, float& y) { st_pair(sm.p + i * LC + j, x, y); });
      U.pairs(tid, [&](int kk, int vv, float& x, float& y) { st_pair(sm.s + kk * LV + vv, x, y); });
      __syncthreads();
      {
        TokV dv;
        dv.zero();
        mm<false, false, LK, LV, KP>(sm.k, sm.s, dv, tid);
        dv.scale_rows(tid, [&](int i) { return sm.rest[i]; });
        mm<true, false, LC, LV, C>(sm.p, sm.d, dv, tid);
        dv.pairs(tid, [&](int i, int vv, float& x, float& y) {
          if (i < rows && vv < p.V)
            st_pair(static_cast<float*>(out.dv) + (((long long)b * p.L + t0 + i) * p.H + h) * p.V + vv, i < valid ? x : 0.f, i < valid ? y : 0.f);
        });
      }
      TokK ki;
      ki.zero();
      mm<false, true, LV, LV, VP>(sm.v, sm.s, ki, tid);
      ki.scale_rows(tid, [&](int i) { return sm.rest[i]; });
      row_dots(ki, sm.k, sm.b);
#pragma unroll
      for (int r = 0; r < TokK::RM; ++r)
#pragma unroll
        for (int c = 0; c < TokK::RN; ++c) dk.v[r][c] += ki.v[r][c];
      put_qk(out.dk, out.dkp, t0, rows, valid, dk);
      __syncthreads();
      m.pairs(tid, [&](int i, int j, float& x, float& y) { st_pair(sm.p + i * LC + j, x, y); });
    }
    for (int i = tid; i < C * (KP / 4); i += NT) {  // scale e^{c_i} q_i
      float4* at = reinterpret_cast<float4*>(sm.q + i / (KP / 4) * LK) + i % (KP / 4);
      const float w = sm.into[i / (KP / 4)];
      float4 x = *at;
      x.x *= w; x.y *= w; x.z *= w; x.w *= w;
      *at = x;
    }
    __syncthreads();
    if (!SUM) {
      // row r of M becomes its running sum over j < t, for t <= r; LR lanes a row, CW columns each
      constexpr int LR = NT / C, CW = C / LR;
      const int r = tid / LR, part = tid % LR;
      {
        float* row = sm.p + r * LC + part * CW;
        float run = 0.f;
#pragma unroll
        for (int e = 0; e < CW; ++e) run += row[e];
        float base = 0.f;
#pragma unroll
        for (int o = 1; o < LR; ++o) {
          const float u = __shfl_up_sync(0xffffffffu, run, o, LR);
          if (part >= o) base += u;
        }
#pragma unroll
        for (int e = 0; e < CW; ++e) {
          const float x = row[e];
          row[e] = part * CW + e <= r ? base : 0.f;
          base += x;
        }
      }
      __syncthreads();
      {  // column sums: every path from before t to t or later
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < CW; ++e) s += sm.p[(part * CW + e) * LC + r];
#pragma unroll
        for (int o = 1; o < LR; o <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (part == 0) sm.rect[r] = s;
      }
      __syncthreads();
      if (tid < 32) {  // two consecutive tokens a lane
        float through = 0.f;
#pragma unroll
        for (int w = 0; w < NT / 32; ++w) through += sm.red[w];
        through *= dec_exp(chi, clo);
        float a0 = 0.f, a1 = 0.f, b0 = 0.f, b1 = 0.f;
#pragma unroll
        for (int w = 0; w < TokK::WN; ++w) {
          a0 += sm.a[w * C + 2 * tid];
          a1 += sm.a[w * C + 2 * tid + 1];
          b0 += sm.b[w * C + 2 * tid];
          b1 += sm.b[w * C + 2 * tid + 1];
        }
        float sa = a0 + a1, sb = b0 + b1;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const float ua = __shfl_down_sync(0xffffffffu, sa, o), ub = __shfl_up_sync(0xffffffffu, sb, o);
          if (tid + o < 32) sa += ua;
          if (tid >= o) sb += ub;
        }
        // sums over the tokens after this lane's two, and before them
        float after = __shfl_down_sync(0xffffffffu, sa, 1), before = __shfl_up_sync(0xffffffffu, sb, 1);
        if (tid == 31) after = 0.f;
        if (tid == 0) before = 0.f;
        const float g0 = (after + (a0 + a1)) + before + through + sm.rect[2 * tid];
        const float g1 = (after + a1) + (before + b0) + through + sm.rect[2 * tid + 1];
        if (p.g_head) {
          float s = (2 * tid < valid ? g0 : 0.f) + (2 * tid + 1 < valid ? g1 : 0.f);
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
          if (tid == 0) out.dg[((long long)b * p.nck + ck) * p.H + h] = s;
        } else {
          float* dst = out.dg + ((long long)b * p.L + t0) * p.H + h;
          if (2 * tid < rows) dst[(long long)(2 * tid) * p.H] = 2 * tid < valid ? g0 : 0.f;
          if (2 * tid + 1 < rows) dst[(long long)(2 * tid + 1) * p.H] = 2 * tid + 1 < valid ? g1 : 0.f;
        }
      }
    }
    const float e = dec_exp(chi, clo);
    U.scale_rows(tid, [&](int) { return e; });
    mm<true, false, LK, LV, C>(sm.q, sm.d, U, tid);
    __syncthreads();
  }
  float* dst = nullptr;
  if (SUM) dst = uend + (bh * p.nseg + seg) * kv;
  else if (out.dh0 != nullptr && seg == 0) dst = out.dh0 + bh * kv;
  if (dst != nullptr)
    U.pairs(tid, [&](int kk, int vv, float& x, float& y) {
      if (kk < p.K && vv < p.V) st_pair(dst + (long long)kk * p.V + vv, x, y);
    });
  if (SUM && tid == 0) udec[bh * p.nseg + seg] = total;
}

// ---------------------------------------------------------------- bf16: tensor cores
// A CTA walks the chunks (128 tokens) of a (batch row, head, segment) from the
// last to the first.  U stays in registers in fp32 (thread = row d of K and a
// quarter of the V columns).  Scores are taken transposed (tensor-memory lane =
// key token j), so that P^T and dP^T are A operands where they are made, and one
// shared-memory copy of dP^T serves dq.
//   T0 = k q^T, T1 = v do^T                            -> P^T, dP^T (bf16), M for dg
//   T2 = do S_in^T (three terms)                       -> * scale e^{c_i}, dotted with q for dg
//   T0 = k U (one term), T1 = v U^T (three terms)      -> * e^{c_last-c_j}, T1 dotted with k for dg
//   T0 += P^T do = dv, T1 += dP^T q = dk, T2 += dP k = dq
//   T3 = q^T (scale e^{c_i} do) (three terms)          -> U
// What ends in fp32 (dg, dh0, U) takes its fp32 operands as three bf16 terms;
// a term of dq, dk or dv is rounded to bf16 once on its way.
//
// Sixteen warps compute, one issues the TMA loads and the MMAs, one finds the
// decays; they meet at mbarriers, as in the forward.  dv, dq and dk are copied out
// by way of dP^T's tile, each warp through a part of its own, while the next k and
// do land (sent by TMA from the tiles of do, dP^T and k they held these for 5000
// cycles: 377 us for a training step of 4 x 2048 tokens of 32 heads of 128 x 128).
// Measured: 235 us of that step's 323.  A chunk takes 29000 cycles, its MMAs 8100:
// bound by the chain of operands that the computing warps make for the tensor cores
// (S and U as three terms, the scores, scale e^{c_i} do) and read back, at the 16
// warps that the registers leave; the tiles fill shared memory, so that no second
// chunk or CTA runs beside it.  Five warps on some of the SM's quarters leave a thread
// 96 registers: 188 bytes of it spill with VP = 128, 128 with VP = 64.
template <int VP>
struct BwdTc {
  static constexpr int vt = kTC * VP * 2;  // bytes of a tile VP columns wide
  static constexpr int q = 0, k = q + 2 * kPanel, x = k + 2 * kPanel, v = x + 2 * kPanel, d = v + vt, y0 = d + vt, y1 = y0 + vt;
  // the third term of a state: a tile of its own, or x, which is free then
  static constexpr int y2 = VP == 64 ? y1 + vt : x, dec = VP == 64 ? y2 + vt : y1 + vt;
  // scale e^{c_i - c of the end of the block of 32 before}; column sums of M by (quarter, block of rows up to it); <S_in, U> by
  // warp; dg of a chunk by quarter
  static constexpr int into = dec + DecTile::bytes, rect = into + kTC * 4, thr = rect + 10 * 32 * 4, hsum = thr + kLinWarps * 4;  // hsum: twice
  // barriers: tiles landed, decays stored; MMA groups done; S terms, U terms and scores, last operands stored; accumulators read;
  // parts of dg stored; their sums by quarter, and by chunk (warps 0 .. 3)
  static constexpr int kLd = 0, kDc = 1, kM0 = 2, kM1 = 3, kM2 = 4, kM3 = 5, kM4 = 6, kR1 = 7, kR3 = 8, kR4 = 9, kR6 = 10, kPt = 11, kEx = 12,
                       kEs = 13, nbar = 14;
  static constexpr int bar = hsum + 160, tm = bar + nbar * 8, bytes = tm + 8;
  static_assert(bytes <= 227 * 1024, "shared memory of a CTA");
  static constexpr int T0 = 0, T1 = 128, T2 = 256, T3 = 384, Pb = 384, dPb = 448, cols = 512;
};

struct BwdMaps {
  CUtensorMap q, k, v, d;
};

// the sum over the warp's lanes of x[l & 15], in lane l
__device__ __forceinline__ float col_sums16(float (&x)[16], int lane) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int e = 0; e < o; ++e) {
      const float give = up ? x[e] : x[e + o], keep = up ? x[e + o] : x[e];
      x[e] = keep + __shfl_xor_sync(0xffffffffu, give, o);
    }
  }
  return x[0] + __shfl_xor_sync(0xffffffffu, x[0], 16);
}

template <int VP>
__global__ void __launch_bounds__(kLinThreads, 1) linattn_bwd_tc_kernel(LinAttn p, const __grid_constant__ BwdMaps maps,
                                                                       const float* __restrict__ ckpt,
                                                                       const float* __restrict__ u0, BwdOut out) {
  using L = BwdTc<VP>;
  constexpr int VQ = VP / 4, NU = VQ / 8;  // columns and 16-byte units of a thread's quarter of V
  extern __shared__ __align__(1024) unsigned char raw[];
  const uint32_t sb = smem_u32(raw);
  const DecTile dec{sb + L::dec};
  uint64_t* bar = reinterpret_cast<uint64_t*>(raw + L::bar);
  uint32_t* tma = reinterpret_cast<uint32_t*>(raw + L::tm);
  float* into_block = reinterpret_cast<float*>(raw + L::into);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  long long id = blockIdx.x;
  const int seg = (int)(id % p.nseg);
  id /= p.nseg;
  const int h = (int)(id % p.H), b = (int)(id / p.H), gh = h / (p.H / p.G);
  const int len = p.len(b);
  const long long bh = (long long)b * p.H + h, kv = (long long)p.K * p.V;
  const int c0 = seg * p.cps, c1 = c0 + p.cps < p.nck ? c0 + p.cps : p.nck;
  int cend = (len + kTC - 1) / kTC;
  cend = cend < c0 ? c0 : cend < c1 ? cend : c1;

  if (tid == 0) {
    for (int i = 0; i < L::nbar; ++i) mbar_init(&bar[i], i >= L::kEx ? 4 : i >= L::kR1 ? kLinWarps : 1);
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
  auto wait = [&](int i, uint32_t par) { return ok = lin_wait(&bar[i], par); };

  if (warp == kLinWarps) {  // ---- the issuing warp
    const int ks = (p.K + 15) / 16, vs = (p.V + 15) / 16;  // contraction steps over K and V
    const uint32_t id128 = mma_idesc(128, false, false);
    // a chunk's tiles; their readers have passed a barrier that this warp has waited for, with a proxy fence before it
    auto load_kd = [&](int ck) {
      if (elect_one()) {
        mbar_arrive_expect_tx(&bar[L::kLd], 4 * kPanel + 2 * L::vt);  // q and v follow
        load_panels(sb + L::k, 2, &maps.k, &bar[L::kLd], 0, gh, ck * kTC, b);
        load_panels(sb + L::d, VP / 64, &maps.d, &bar[L::kLd], 0, h, ck * kTC, b);
      }
      __syncwarp();
    };
    auto load_qv = [&](int ck) {
      if (elect_one()) {
        load_panels(sb + L::q, 2, &maps.q, &bar[L::kLd], 0, gh, ck * kTC, b);
        load_panels(sb + L::v, VP / 64, &maps.v, &bar[L::kLd], 0, h, ck * kTC, b);
      }
      __syncwarp();
    };
    if (c0 < cend) {
      load_kd(cend - 1);
      load_qv(cend - 1);
    }
    for (int ck = cend - 1; ck >= c0; --ck) {
      const uint32_t par = (uint32_t)(cend - 1 - ck) & 1u;
      const int valid = len - ck * kTC;
      if (!wait(L::kLd, par)) break;
      if (valid < kTC && ck * kTC + valid < p.L) {  // the row ends inside the tensor: what follows is not its own
        zero_rows(sb + L::q, 4, valid, lane);         // (the tiles' other readers take dead rows as zero)
        zero_rows(sb + L::v, 2 * VP / 64, valid, lane);
        fence_proxy_async_smem();
        __syncwarp();
      }
      if (ck < cend - 1 && !wait(L::kR6, par ^ 1u)) break;  // the accumulators' places take scores next
      if (elect_one()) {
        tc_fence_after_sync();
        mma_steps(tm + L::T0, Rows{sb + L::k}, Rows{sb + L::q}, id128, ks, false);
        mma_steps(tm + L::T1, Rows{sb + L::v}, Rows{sb + L::d}, id128, vs, false);
        mma_commit(&bar[L::kM0]);
        if (ck > c0) {  // the next chunk towards L2
          prefetch_panels((p.K + 63) / 64, &maps.q, 0, gh, (ck - 1) * kTC, b);
          prefetch_panels((p.K + 63) / 64, &maps.k, 0, gh, (ck - 1) * kTC, b);
          prefetch_panels((p.V + 63) / 64, &maps.v, 0, h, (ck - 1) * kTC, b);
          prefetch_panels((p.V + 63) / 64, &maps.d, 0, h, (ck - 1) * kTC, b);
        }
      }
      __syncwarp();
      if (!wait(L::kR1, par)) break;
      if (elect_one()) {
        tc_fence_after_sync();
#pragma unroll
        for (int t = 2; t >= 0; --t)  // the smallest term first
          mma_steps(tm + L::T2, Rows{sb + L::d}, Rows{sb + (t == 0 ? L::y0 : t == 1 ? L::y1 : L::y2)}, id128, vs, t < 2);
        mma_commit(&bar[L::kM1]);
      }
      __syncwarp();
      if (!wait(L::kR3, par)) break;
      if (elect_one()) {
        tc_fence_after_sync();
        mma_steps(tm + L::T0, Rows{sb + L::k}, Cols{sb + L::y0}, mma_idesc(VP, false, true), ks, false);
#pragma unroll
        for (int t = 2; t >= 0; --t)
          mma_steps(tm + L::T1, Rows{sb + L::v}, Rows{sb + (t == 0 ? L::y0 : t == 1 ? L::y1 : L::y2)}, id128, vs, t < 2);
        mma_commit(&bar[L::kM2]);
      }
      __syncwarp();
      if (!wait(L::kR4, par)) break;
      if (elect_one()) {
        tc_fence_after_sync();
#pragma unroll
        for (int s = 0; s < kTC / 16; ++s) mma_ts(tm + L::T0, tm + L::Pb + s * 8, desc_cols(sb + L::d, s), mma_idesc(VP, false, true), true);
#pragma unroll
        for (int s = 0; s < kTC / 16; ++s) mma_ts(tm + L::T1, tm + L::dPb + s * 8, desc_cols(sb + L::q, s), mma_idesc(128, false, true), true);
        mma_steps(tm + L::T2, Cols{sb + L::x}, Cols{sb + L::k}, mma_idesc(128, true, true), kTC / 16, true);
        mma_commit(&bar[L::kM3]);
      }
      __syncwarp();
      if (!wait(L::kM3, par)) break;
      if (elect_one()) {  // into the scores' place, whose readers are done
        tc_fence_after_sync();
#pragma unroll
        for (int t = 2; t >= 0; --t)
          mma_steps(tm + L::T3, Cols{sb + L::q}, Cols{sb + (t == 0 ? L::y0 : t == 1 ? L::y1 : L::v)}, mma_idesc(VP, true, true), kTC / 16, t < 2);
        mma_commit(&bar[L::kM4]);
      }
      __syncwarp();
      if (ck > c0) {
        load_kd(ck - 1);
        if (!wait(L::kM4, par)) break;
        load_qv(ck - 1);
      }
    }
  } else if (warp > kLinWarps) {  // ---- the decays' warp
    DecStage ds;
    ds.g.fetch(p, b, h, (cend - 1) * kTC, len, lane);
    for (int ck = cend - 1; ck >= c0; --ck) {
      ds.scan(lane);
      if (ck < cend - 1 && !wait(L::kR3, (uint32_t)(cend - 2 - ck) & 1u)) break;  // the chunk before is done with its own
      ds.put(dec, lane);
      __syncwarp();
#pragma unroll
      for (int e = 0; e < kTC; e += 32) into_block[e + lane] = p.scale * dec_exp(dec.rel(e + lane));
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar[L::kDc]);
      if (ck > c0) {
        ds.g.fetch(p, b, h, (ck - 1) * kTC, len, lane);
        const float* c = ckpt + (bh * p.nck + ck - 1) * kv;
        for (long long i = lane * 32; i < kv; i += 32 * 32) prefetch_l2(c + i);
      }
    }
  } else {  // ---- a computing warp
    const int row = (warp & 3) * 32 + lane, cq = warp >> 2;  // tensor-memory lane, quarter of the columns
    const uint32_t tl = tm + ((uint32_t)((warp & 3) * 32) << 16);
    float* rect = reinterpret_cast<float*>(raw + L::rect);
    float* thr = reinterpret_cast<float*>(raw + L::thr);
    float U[VQ];
#pragma unroll
    for (int e = 0; e < VQ; ++e) U[e] = 0.f;
    if (u0 != nullptr && row < p.K) {
      const float* src = u0 + ((p.nseg > 1 ? bh * p.nseg + seg : bh) * p.K + row) * p.V + cq * VQ;
#pragma unroll
      for (int e = 0; e < VQ; e += 4)
        if (cq * VQ + e < p.V) {
          const float4 x = *reinterpret_cast<const float4*>(src + e);
          U[e] = x.x; U[e + 1] = x.y; U[e + 2] = x.z; U[e + 3] = x.w;
        }
    }
    auto arrive = [&](int i) {  // this warp's shared- and tensor-memory accesses before are over
      fence_proxy_async_smem();
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar[i]);
    };
    // 32 gradients of q or k of this thread's token (columns cq * 32 ...) as this head's fp32 part, [K/4][token][4]
    auto put_part = [&](float* part, int ck, const uint32_t (&r)[32], bool live) {
      float4* dst = reinterpret_cast<float4*>(part) + (((long long)b * p.nck + ck) * p.H + h) * (p.K / 4) * kTC + row;
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        if (cq * 32 + u * 4 >= p.K) continue;
        dst[(cq * 8 + u) * kTC] = live ? make_float4(__uint_as_float(r[4 * u]), __uint_as_float(r[4 * u + 1]), __uint_as_float(r[4 * u + 2]),
                                                     __uint_as_float(r[4 * u + 3]))
                                       : make_float4(0.f, 0.f, 0.f, 0.f);
      }
    };
    // the three terms of a [K][V] fp32 state, this thread's row and quarter
    auto put_terms = [&](const float (&s)[VQ]) {
#pragma unroll
      for (int u = 0; u < NU; ++u) {
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = s[8 * u + e];
        const uint32_t at = tile_at(row, cq * NU + u);
        sts16(sb + L::y0 + at, take_term(x));
        sts16(sb + L::y1 + at, take_term(x));
        sts16(sb + L::y2 + at, last_term(x));
      }
    };
    // N columns of tensor memory times f, in place, dotted with this token's row of a tile of 128 columns
    auto scale_dot = [&](uint32_t t, uint32_t tile, float f, bool live) {
      uint32_t r[32];
      tmem_ld32(tl + t + cq * 32, r);
      tmem_wait_ld();
      float dot = 0.f;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        float x[8];
        Raw8<__nv_bfloat16>::wide(live ? lds16(sb + tile + tile_at(row, cq * 4 + u)) : make_uint4(0u, 0u, 0u, 0u), x);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float y = __uint_as_float(r[8 * u + e]) * f;
          dot = fmaf(x[e], y, dot);
          r[8 * u + e] = __float_as_uint(y);
        }
      }
      __syncwarp();
      tmem_st32(tl + t + cq * 32, r);
      return dot;
    };
    // typed gradients of this token (this quarter of them), by way of this warp's part of x, whose product is done
    auto put_rows = [&](void* dst, auto& r, int width, int ck, bool live) {
      constexpr int n = sizeof(r) / 32;
#pragma unroll
      for (int u = 0; u < n; ++u) {
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = live ? __uint_as_float(r[8 * u + e]) : 0.f;
        sts16(sb + L::x + tile_at(row, cq * 4 + u), pack8(x));
      }
      __syncwarp();
      store_rows<n>(sb + L::x, static_cast<__nv_bfloat16*>(dst) + (((long long)b * p.L + ck * kTC) * p.H + h) * width, (long long)p.H * width,
                    (warp & 3) * 32, cq * 4, cq * n, p.L - ck * kTC, width, lane);
      __syncwarp();
    };

    // dg of a chunk's tokens t = 32 warp + lane (warps 0 .. 3), from what their warps took when its accumulators were done
    float in = 0.f, th = 0.f, in_e = 0.f, fa = 0.f, fb = 0.f, q1 = 0.f, q2 = 0.f, q3 = 0.f;
    auto sum_dg = [&](int ck) {
      const int t0 = ck * kTC;
      const uint32_t par = (uint32_t)(cend - 1 - ck) & 1u;
      const bool live = row < len - t0;
      float ra = fa, rb = fb + (warp == 0 ? q1 : warp == 1 ? q2 : warp == 2 ? q3 : 0.f);  // running sums within the warp's tokens
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const float ua = __shfl_down_sync(0xffffffffu, ra, o), ub = __shfl_up_sync(0xffffffffu, rb, o);
        if (lane + o < 32) ra += ua;
        if (lane >= o) rb += ub;
      }
      // what other quarters of tokens need of this one: its sum of fa (for those before), of fb and of the paths to quarters after c
      // (for quarter c after it)
      float sa = fa, s2 = fb + q2, s3 = fb + q3, s4 = fb;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        sa += __shfl_xor_sync(0xffffffffu, sa, o);
        s2 += __shfl_xor_sync(0xffffffffu, s2, o);
        s3 += __shfl_xor_sync(0xffffffffu, s3, o);
        s4 += __shfl_xor_sync(0xffffffffu, s4, o);
        th += __shfl_xor_sync(0xffffffffu, th, o);
      }
      float* ex = reinterpret_cast<float*>(raw + L::hsum) + par * 20;  // [quarter][4], then the quarters' dg
      if (lane == 0) {
        ex[warp * 4] = sa; ex[warp * 4 + 1] = s2; ex[warp * 4 + 2] = s3; ex[warp * 4 + 3] = s4;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar[L::kEx]);
      if (!wait(L::kEx, par)) return;
      float after = 0.f, before = 0.f;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        if (w > warp) after += ex[w * 4];
        if (w < warp) before += ex[w * 4 + warp];  // warp 1, 2, 3: the paths that cross into it
      }
      const float up = __shfl_up_sync(0xffffffffu, rb, 1);
      const float g = in + (after + ra) + (before + (lane > 0 ? up : 0.f)) + in_e * th;
      if (!p.g_head) {
        if (t0 + row < p.L) out.dg[((long long)b * p.L + t0 + row) * p.H + h] = live ? g : 0.f;
      } else {
        float s = live ? g : 0.f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (lane == 0) ex[16 + warp] = s;
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar[L::kEs]);
        if (warp == 0 && wait(L::kEs, par) && lane == 0)
          out.dg[((long long)b * p.nck + ck) * p.H + h] = (ex[16] + ex[17]) + (ex[18] + ex[19]);
      }
    };
    for (int ck = cend; ck < c1; ++ck) {  // past the row's end
      const int rows = p.L - ck * kTC < kTC ? p.L - ck * kTC : kTC;
      const long long at = ((long long)b * p.L + ck * kTC) * p.H + h;
      auto clear = [&](void* dst, int width) {  // rows of `width` bf16, H rows apart
        const int n = width / 8;
        uint4* to = static_cast<uint4*>(dst) + at * n;
        for (int i = tid; i < rows * n; i += 32 * kLinWarps) to[(long long)(i / n) * p.H * n + i % n] = make_uint4(0u, 0u, 0u, 0u);
      };
      if (out.dqp != nullptr) {
        const long long n = (long long)(p.K / 4) * kTC, to = (((long long)b * p.nck + ck) * p.H + h) * n;
        for (int i = tid; i < n; i += 32 * kLinWarps)
          reinterpret_cast<float4*>(out.dqp)[to + i] = reinterpret_cast<float4*>(out.dkp)[to + i] = make_float4(0.f, 0.f, 0.f, 0.f);
      } else {
        clear(out.dq, p.K);
        clear(out.dk, p.K);
      }
      clear(out.dv, p.V);
      if (p.g_head) {
        if (tid == 0) out.dg[((long long)b * p.nck + ck) * p.H + h] = 0.f;
      } else if (tid < rows) {
        out.dg[((long long)b * p.L + ck * kTC + tid) * p.H + h] = 0.f;
      }
    }
    for (int ck = cend - 1; ck >= c0; --ck) {
      const uint32_t par = (uint32_t)(cend - 1 - ck) & 1u;
      const int t0 = ck * kTC, valid = len - t0;
      const bool live = row < valid;
      float through = 0.f;  // <S_in, U>, this thread's part
      {
        float S[VQ];
        const float4* src = reinterpret_cast<const float4*>(ckpt + (bh * p.nck + ck) * kv) + row;
#pragma unroll
        for (int e = 0; e < VQ; e += 4) {
          float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
          if (row < p.K && cq * VQ + e < p.V) x = src[(long long)((cq * VQ + e) / 4) * p.K];
          S[e] = x.x; S[e + 1] = x.y; S[e + 2] = x.z; S[e + 3] = x.w;
        }
#pragma unroll
        for (int e = 0; e < VQ; ++e) through = fmaf(S[e], U[e], through);
        put_terms(S);
      }
      arrive(L::kR1);
      if (!wait(L::kDc, par) || !wait(L::kLd, par)) break;
      const Dec last = dec.get(kTC - 1), own = dec.get(row);
      const float elast = dec_exp(last), into = p.scale * dec_exp(own), rest = dec_exp(dec_sub(last, own));
      if (!wait(L::kM0, par)) break;
      tc_fence_after_sync();
      float tot = 0.f;
      if (cq >= (warp & 3)) {  // query tokens of this quarter at or after this warp's key tokens
        const bool diag = cq == (warp & 3);
        const float from = diag ? 0.f : dec_exp(dec_sub(dec.base(cq), own));  // off the diagonal a decay is a product of two
        const Dec orel = dec.rel(row);
        float sums[2];
#pragma unroll
        for (int g = 1; g >= 0; --g) {
          const int i0 = cq * 32 + g * 16;
          uint32_t s[16], t[16], w[8], z[8];
          float m[16];
          tmem_ld16(tl + L::T0 + i0, s);
          tmem_ld16(tl + L::T1 + i0, t);
          tmem_wait_ld();
          if (!diag) {
#pragma unroll
            for (int e = 12; e >= 0; e -= 4) {
              const float4 f = *reinterpret_cast<const float4*>(into_block + i0 + e);
              const float wt[4] = {f.x * from, f.y * from, f.z * from, f.w * from};
              float pp[4], dp[4];
#pragma unroll
              for (int n = 3; n >= 0; --n) {
                const float d = __uint_as_float(t[e + n]);
                pp[n] = __uint_as_float(s[e + n]) * wt[n];
                dp[n] = d * wt[n];
                tot = fmaf(pp[n], d, tot);  // paths from j to this query token or a later one of the quarter
                m[e + n] = tot;
              }
              w[e / 2] = pack_bf16(pp[0], pp[1]);
              w[e / 2 + 1] = pack_bf16(pp[2], pp[3]);
              z[e / 2] = pack_bf16(dp[0], dp[1]);
              z[e / 2 + 1] = pack_bf16(dp[2], dp[3]);
            }
          } else {
#pragma unroll
            for (int e = 12; e >= 0; e -= 4) {
              float hi[4], lo[4], pp[4], dp[4];
              dec.rel4(i0 + e, hi, lo);
#pragma unroll
              for (int n = 3; n >= 0; --n) {
                const int i = g * 16 + e + n;
                const float wt = i >= lane ? p.scale * dec_diff(hi[n], lo[n], orel.hi, orel.lo) : 0.f;
                const float d = i >= lane ? __uint_as_float(t[e + n]) : 0.f;
                pp[n] = (i >= lane ? __uint_as_float(s[e + n]) : 0.f) * wt;
                dp[n] = d * wt;
                tot = fmaf(pp[n], d, tot);
                m[e + n] = i > lane ? tot : 0.f;
              }
              w[e / 2] = pack_bf16(pp[0], pp[1]);
              w[e / 2 + 1] = pack_bf16(pp[2], pp[3]);
              z[e / 2] = pack_bf16(dp[0], dp[1]);
              z[e / 2 + 1] = pack_bf16(dp[2], dp[3]);
            }
          }
          tmem_st8u(tl + L::Pb + i0 / 2, w);
          tmem_st8u(tl + L::dPb + i0 / 2, z);
          sums[g] = col_sums16(m, lane);
        }
        rect[(cq * (cq + 1) / 2 + (warp & 3)) * 32 + lane] = lane < 16 ? sums[0] : sums[1];
      } else {
        uint32_t z[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) z[e] = 0u;
        tmem_st16(tl + L::Pb + cq * 16, z);
        tmem_st16(tl + L::dPb + cq * 16, z);
      }
      if (!wait(L::kM1, par)) break;
      tc_fence_after_sync();
      put_terms(U);
      tmem_wait_st();
      arrive(L::kR3);
      const float dot_a = scale_dot(L::T2, L::q, into, live);  // under the products of U
      if (warp < 4 && ck < cend - 1) sum_dg(ck + 1);
      if (!ok || !wait(L::kM2, par)) break;
      tc_fence_after_sync();
      // operands of the last products: dP^T in shared memory, scale e^{c_i} do in three terms (the third in v's place)
      {
        uint32_t z[16];
        tmem_ld16(tl + L::dPb + cq * 16, z);
        tmem_wait_ld();
#pragma unroll
        for (int u = 0; u < 4; ++u)
          sts16(sb + L::x + tile_at(row, cq * 4 + u), make_uint4(z[4 * u], z[4 * u + 1], z[4 * u + 2], z[4 * u + 3]));
      }
#pragma unroll
      for (int u = 0; u < NU; ++u) {
        const uint32_t at = tile_at(row, cq * NU + u);
        float x[8];
        Raw8<__nv_bfloat16>::wide(live ? lds16(sb + L::d + at) : make_uint4(0u, 0u, 0u, 0u), x);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] *= into;
        sts16(sb + L::y0 + at, take_term(x));
        sts16(sb + L::y1 + at, take_term(x));
        sts16(sb + L::v + at, last_term(x));
      }
      __syncwarp();
      const float dot_b = scale_dot(L::T1, L::k, rest, live);
      tmem_scale<VQ>(tl + L::T0 + cq * VQ, rest);
      tmem_wait_st();
      arrive(L::kR4);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) through += __shfl_xor_sync(0xffffffffu, through, o);
      if (lane == 0) thr[warp] = through;
      if (!wait(L::kM3, par)) break;
      tc_fence_after_sync();
      const bool shared = out.dqp != nullptr;
      {
        uint32_t r[VQ];
        tmem_ldn(tl + L::T0 + cq * VQ, r);
        tmem_wait_ld();
        put_rows(out.dv, r, p.V, ck, live);
      }
      {
        uint32_t r[32];
        tmem_ld32(tl + L::T2 + cq * 32, r);
        tmem_wait_ld();
        if (shared) put_part(out.dqp, ck, r, live);
        else put_rows(out.dq, r, p.K, ck, live);
        {  // this token's parts of dg to the warps that sum it, in the place just read
          const uint32_t e[8] = {__float_as_uint(dot_a), __float_as_uint(dot_b), __float_as_uint(tot), 0u, 0u, 0u, 0u, 0u};
          tmem_st8u(tl + L::T2 + cq * 32, e);
        }
        tmem_ld32(tl + L::T1 + cq * 32, r);
        tmem_wait_ld();
        tmem_wait_st();
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar[L::kPt]);
        if (shared) put_part(out.dkp, ck, r, live);
        else put_rows(out.dk, r, p.K, ck, live);
      }
      if (warp < 4) {  // what dg is summed from; the sums under the next chunk's products
        if (!wait(L::kPt, par)) break;
        tc_fence_after_sync();
        in = 0.f;
        in_e = elast;
#pragma unroll
        for (int w = 0; w < 4; ++w)  // the blocks of rows up to this quarter
          if (w <= warp) in += rect[(warp * (warp + 1) / 2 + w) * 32 + lane];
        th = lane < kLinWarps ? thr[lane] : 0.f;
        uint32_t e[4][8];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld8u(tl + L::T2 + c * 32, e[c]);
        tmem_wait_ld();
        // token `row`'s sums over the quarters of the columns, and its paths to the quarters after 0, 1, 2
        fa = (__uint_as_float(e[0][0]) + __uint_as_float(e[1][0])) + (__uint_as_float(e[2][0]) + __uint_as_float(e[3][0]));
        fb = (__uint_as_float(e[0][1]) + __uint_as_float(e[1][1])) + (__uint_as_float(e[2][1]) + __uint_as_float(e[3][1]));
        q3 = __uint_as_float(e[3][2]);
        q2 = q3 + __uint_as_float(e[2][2]);
        q1 = q2 + __uint_as_float(e[1][2]);
      }
      if (!wait(L::kM4, par)) break;
      tc_fence_after_sync();
      {
        uint32_t r[VQ];
        tmem_ldn(tl + L::T3 + cq * VQ, r);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < VQ; ++e) U[e] = fmaf(U[e], elast, __uint_as_float(r[e]));
      }
      arrive(L::kR6);
    }
    if (ok && cend > c0 && warp < 4) sum_dg(c0);
    if (out.dh0 != nullptr && seg == 0 && row < p.K) {
      float* dst = out.dh0 + (bh * p.K + row) * p.V + cq * VQ;
#pragma unroll
      for (int e = 0; e < VQ; e += 4)
        if (cq * VQ + e < p.V) *reinterpret_cast<float4*>(dst + e) = make_float4(U[e], U[e + 1], U[e + 2], U[e + 3]);
    }
  }
  lin_leave(ok, bar, L::nbar, tm, L::cols, warp, lane);
}

// dq, dk of a shared head: the parts of its R heads added in order, rounded once.
__global__ void __launch_bounds__(256) linattn_share_kernel(const float* __restrict__ pq, const float* __restrict__ pk,
                                                            float* __restrict__ dq, float* __restrict__ dk, long long n, int R, int K) {
  const long long i = ((long long)blockIdx.x * 256 + threadIdx.x) * 4;  // K is a multiple of 8: four elements of one head
  if (i >= n) return;
  const float* src = blockIdx.y ? pk : pq;
  float* dst = blockIdx.y ? dk : dq;
  const long long row = i / K, at = row * R * K + i % K;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int r = 0; r < R; ++r) {
    const float4 x = *reinterpret_cast<const float4*>(src + at + (long long)r * K);
    a.x += x.x; a.y += x.y; a.z += x.z; a.w += x.w;
  }
  *reinterpret_cast<float4*>(dst + i) = a;
}

// The same from parts in blocks of kTC tokens, [K/4][token][4] (the tensor-core kernel's): a warp reads eight tokens of four
// groups of columns, 128 bytes each.
__global__ void __launch_bounds__(256) linattn_share_tc_kernel(const float* __restrict__ pq, const float* __restrict__ pk,
                                                               __nv_bfloat16* __restrict__ dq, __nv_bfloat16* __restrict__ dk, int L,
                                                               int nck, int H, int G, int K) {
  const float4* src = reinterpret_cast<const float4*>(blockIdx.y ? pk : pq);
  __nv_bfloat16* dst = blockIdx.y ? dk : dq;
  const int R = H / G, g = (int)(blockIdx.x % G);
  const long long bc = blockIdx.x / G, b = bc / nck;
  const int ck = (int)(bc % nck), lane = threadIdx.x & 31, n4 = K / 4;
  const long long block = (long long)n4 * kTC;
  for (int i = threadIdx.x >> 5; i < (n4 + 3) / 4 * (kTC / 8); i += 8) {
    const int c4 = i / (kTC / 8) * 4 + (lane >> 3), t = i % (kTC / 8) * 8 + (lane & 7);
    if (c4 >= n4 || ck * kTC + t >= L) continue;
    const float4* at = src + (bc * H + (long long)g * R) * block + (long long)c4 * kTC + t;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int r = 0; r < R; ++r) {
      const float4 x = at[r * block];
      a.x += x.x; a.y += x.y; a.z += x.z; a.w += x.w;
    }
    *reinterpret_cast<uint2*>(dst + ((b * L + ck * kTC + t) * G + g) * K + c4 * 4) = make_uint2(pack_bf16(a.x, a.y), pack_bf16(a.z, a.w));
  }
}

struct AddDg {
  float* out;
  __device__ void put(long long i, float v) const { out[i] += v; }
};

struct BwdPlan {
  LinAttn p;
  size_t states, decs, parts, sums, bytes;  // segment states and decays, dq/dk parts (each), per-chunk dg sums
};

inline size_t up16(size_t n) { return (n + 15) / 16 * 16; }

int bwd_plan(int B, int L, int H, int G, int K, int V, int dtype, int g_head, BwdPlan& pl) {
  const int rc = linattn_validate(B, L, H, G, K, V, dtype);
  if (rc != SS_OK) return rc;
  pl.p = LinAttn{};
  pl.p.B = B; pl.p.L = L; pl.p.H = H; pl.p.G = G; pl.p.K = K; pl.p.V = V;
  const long long walks = (long long)B * H;
  if (walks > (1ll << 24)) return SS_ERR_DIM;
  linattn_segments(pl.p, dtype, walks);
  const int n = pl.p.nseg;
  pl.states = n > 1 ? (size_t)walks * n * K * V * sizeof(float) : 0;
  pl.decs = n > 1 ? up16((size_t)walks * n * sizeof(Dec)) : 0;
  pl.parts = H != G ? (size_t)B * (dtype == SS_F32 ? (size_t)L : (size_t)pl.p.nck * kTC) * H * K * sizeof(float) : 0;
  pl.sums = g_head ? up16((size_t)B * pl.p.nck * H * sizeof(float)) : 0;
  pl.bytes = pl.states + pl.decs + 2 * pl.parts + pl.sums;
  return SS_OK;
}

// The walk (for a row cut in segments after their U), then the sums over heads that share q, k and over chunks.
template <typename T, typename Sum, typename Walk>
int bwd_run(const BwdPlan& pl, const float* dh_last, BwdOut out, float* dg, char* ws, cudaStream_t s, Sum sum, Walk walk) {
  const LinAttn& p = pl.p;
  float* st = reinterpret_cast<float*>(ws);
  Dec* dec = reinterpret_cast<Dec*>(ws + pl.states);
  out.dqp = pl.parts ? reinterpret_cast<float*>(ws + pl.states + pl.decs) : nullptr;
  out.dkp = pl.parts ? reinterpret_cast<float*>(ws + pl.states + pl.decs + pl.parts) : nullptr;
  out.dg = p.g_head ? reinterpret_cast<float*>(ws + pl.states + pl.decs + 2 * pl.parts) : dg;
  int rc;
  if (p.nseg == 1) {
    rc = walk(dh_last, out);
  } else {
    if ((rc = sum(st, dec, out)) != SS_OK) return rc;
    const long long kv = (long long)p.K * p.V;
    linattn_join_kernel<true><<<dim3((unsigned)((kv + 255) / 256), (unsigned)(p.B * p.H)), 256, 0, s>>>(dh_last, st, dec, kv, p.nseg);
    if (cudaGetLastError() != cudaSuccess) return SS_ERR_CUDA;
    rc = walk(st, out);
  }
  if (rc != SS_OK) return rc;
  if (pl.parts && std::is_same_v<T, __nv_bfloat16>) {
    linattn_share_tc_kernel<<<dim3((unsigned)((long long)p.B * p.nck * p.G), 2), 256, 0, s>>>(
        out.dqp, out.dkp, static_cast<__nv_bfloat16*>(out.dq), static_cast<__nv_bfloat16*>(out.dk), p.L, p.nck, p.H, p.G, p.K);
    if (cudaGetLastError() != cudaSuccess) return SS_ERR_CUDA;
  } else if (pl.parts) {
    const long long n = (long long)p.B * p.L * p.G * p.K;
    linattn_share_kernel<<<dim3((unsigned)((n / 4 + 255) / 256), 2), 256, 0, s>>>(out.dqp, out.dkp, static_cast<float*>(out.dq),
                                                                              static_cast<float*>(out.dk), n, p.H / p.G, p.K);
    if (cudaGetLastError() != cudaSuccess) return SS_ERR_CUDA;
  }
  if (p.g_head && colsum(out.dg, p.H, p.B * p.nck, AddDg{dg}, s) != cudaSuccess) return SS_ERR_CUDA;
  return SS_OK;
}

template <int KP, int VP>
int bwd_f32(const BwdPlan& pl, const void* dout, const float* ckpt, const float* dh_last, const BwdOut& out, float* dg, char* ws,
            cudaStream_t s) {
  const unsigned grid = (unsigned)pl.p.B * pl.p.H * pl.p.nseg;
  using Sm = BwdSmem<KP, VP>;
  const size_t smem = sizeof(Sm);
  return bwd_run<float>(
      pl, dh_last, out, dg, ws, s,
      [&](float* st, Dec* dec, const BwdOut& o) {
        return lin_launch(linattn_bwd_kernel<KP, VP, true>, grid, BwdSmem<KP, VP>::NT, offsetof(Sm, k), s, pl.p, dout, ckpt, nullptr, o, st, dec);
      },
      [&](const float* u0, const BwdOut& o) {
        return lin_launch(linattn_bwd_kernel<KP, VP, false>, grid, BwdSmem<KP, VP>::NT, smem, s, pl.p, dout, ckpt, u0, o, nullptr, nullptr);
      });
}

template <int VP>
int bwd_bf16(const BwdPlan& pl, const void* dout, const float* ckpt, const float* dh_last, const BwdOut& out, float* dg, char* ws,
             cudaStream_t s) {
  const LinAttn& p = pl.p;
  const unsigned grid = (unsigned)p.B * p.H * p.nseg;
  BwdMaps maps;
  if (!lin_map(&maps.q, p.q, p.ldq, p.B, p.L, p.G, p.K) || !lin_map(&maps.k, p.k, p.ldk, p.B, p.L, p.G, p.K) ||
      !lin_map(&maps.v, p.v, p.ldv, p.B, p.L, p.H, p.V) || !lin_map(&maps.d, dout, (long long)p.H * p.V, p.B, p.L, p.H, p.V))
    return SS_ERR_CUDA;
  return bwd_run<__nv_bfloat16>(
      pl, dh_last, out, dg, ws, s,
      [&](float* st, Dec* dec, const BwdOut&) {
        return lin_launch(linattn_sum_tc_kernel<true>, grid * ((p.V + 63) / 64), kLinThreads, SumTc::bytes, s, p, maps.q, maps.d, st, dec);
      },
      [&](const float* u0, const BwdOut& o) {
        return lin_launch(linattn_bwd_tc_kernel<VP>, grid, kLinThreads, BwdTc<VP>::bytes, s, p, maps, ckpt, u0, o);
      });
}

}  // namespace

extern "C" size_t linattn_bwd_workspace_size(int B, int L, int H, int G, int K, int V, int g_per_head, int dtype) {
  BwdPlan pl;
  return bwd_plan(B, L, H, G, K, V, dtype, g_per_head, pl) == SS_OK ? pl.bytes : 0;
}

extern "C" int linattn_bwd(const void* q, long long ldq, const void* k, long long ldk, const void* v, long long ldv,
                           const float* g, int g_per_head, const int* lengths, const float* ckpt, const void* dout,
                           const float* dh_last, void* dq, void* dk, void* dv, float* dg, float* dh0, int B, int L, int H,
                           int G, int K, int V, float scale, int dtype, void* workspace, size_t ws_bytes, void* stream) {
  if (!q || !k || !v || !g || !ckpt || !dout || !dq || !dk || !dv || !dg) return SS_ERR_NULL;
  BwdPlan pl;
  int rc = bwd_plan(B, L, H, G, K, V, dtype, g_per_head, pl);
  if (rc != SS_OK) return rc;
  if ((rc = linattn_ld_ok(ldq, G, K)) != SS_OK || (rc = linattn_ld_ok(ldk, G, K)) != SS_OK ||
      (rc = linattn_ld_ok(ldv, H, V)) != SS_OK)
    return rc;
  const void* ptrs[] = {q, k, v, ckpt, dout, dh_last, dq, dk, dv, dh0};
  for (const void* x : ptrs)
    if (x != nullptr && !ssh::aligned16(x)) return SS_ERR_ALIGN;
  if ((reinterpret_cast<uintptr_t>(g) & 3u) || (reinterpret_cast<uintptr_t>(dg) & 3u) || (reinterpret_cast<uintptr_t>(lengths) & 3u))
    return SS_ERR_ALIGN;
  if (pl.bytes > 0) {
    if (workspace == nullptr || ws_bytes < pl.bytes) return SS_ERR_WORKSPACE;
    if (!ssh::aligned16(workspace)) return SS_ERR_ALIGN;
  }
  LinAttn& p = pl.p;
  p.q = q; p.k = k; p.v = v;
  p.ldq = ldq; p.ldk = ldk; p.ldv = ldv;
  p.g = g; p.g_head = g_per_head;
  p.lengths = lengths;
  p.scale = scale;
  BwdOut out = {dq, dk, dv, nullptr, nullptr, nullptr, dh0};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  char* ws = static_cast<char*>(workspace);
  if (dtype == SS_BF16)  // (8192 tokens of 32 heads of 128 x 64, forward and backward: 366 us in tiles of 64 columns, 406 in tiles of 128)
    return V <= 64 ? bwd_bf16<64>(pl, dout, ckpt, dh_last, out, dg, ws, s) : bwd_bf16<128>(pl, dout, ckpt, dh_last, out, dg, ws, s);
  if (K <= 64)  // (24 heads of 64 x 64, forward and backward: 1449 us in tiles of 64 rows, 2352 in tiles of 128)
    return V <= 64 ? bwd_f32<64, 64>(pl, dout, ckpt, dh_last, out, dg, ws, s) : bwd_f32<64, 128>(pl, dout, ckpt, dh_last, out, dg, ws, s);
  return V <= 64 ? bwd_f32<128, 64>(pl, dout, ckpt, dh_last, out, dg, ws, s) : bwd_f32<128, 128>(pl, dout, ckpt, dh_last, out, dg, ws, s);
}

namespace ssh {
int read_clear_linb_err(cudaStream_t s, unsigned* out) { return read_clear_lin_err(s, out); }
}  // namespace ssh
