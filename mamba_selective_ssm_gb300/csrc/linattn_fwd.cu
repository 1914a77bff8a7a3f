// Linear attention with a decay for each head, chunked forward (linattn_fwd) for sm_103a.
#include <stddef.h>

#include "linattn_tc.cuh"

namespace {

// fp32: three-product tf32 (see Own).  A CTA walks the chunks of one (batch row,
// head, 64-column tile of V, segment) in order with the state in registers.
// SUM only finds the segment's end state from zero and its decay (no q, no o).
// Bound by mma.sync and the shared-memory loads and splits that feed it: 367 us (and
// 99 for the sums) for 8 x 2048 tokens of 24 heads of 64 x 64.
constexpr int kVT = 64;

template <int KP>
struct FwdSmem {
  static constexpr int NT = 256;  // threads
  static constexpr int C = kLinChunkF32, LK = KP + 4, LV = kVT + 4, LC = C + 4;
  float k[C * LK], v[C * LV], chi[C], clo[C], rest[C];
  float q[C * LK], s[KP * LV];  // (not for a sum) the scores take q's place
};

template <int KP, bool SUM>
__global__ void __launch_bounds__(FwdSmem<KP>::NT) linattn_fwd_kernel(LinAttn p, const float* __restrict__ s0, float* __restrict__ o,
                                                                      float* __restrict__ ckpt, float* __restrict__ send,
                                                                      Dec* __restrict__ sdec) {
  using Sm = FwdSmem<KP>;
  constexpr int C = Sm::C, LK = Sm::LK, LV = Sm::LV, LC = Sm::LC, NT = Sm::NT;
  extern __shared__ __align__(16) unsigned char raw[];
  Sm& sm = *reinterpret_cast<Sm*>(raw);
  const int tid = threadIdx.x;
  const int nvt = (p.V + kVT - 1) / kVT;
  long long id = blockIdx.x;
  const int seg = (int)(id % p.nseg);
  id /= p.nseg;
  const int vt = (int)(id % nvt);
  id /= nvt;
  const int h = (int)(id % p.H), b = (int)(id / p.H);
  const int gh = h / (p.H / p.G), v0 = vt * kVT, vw = p.V - v0 < kVT ? p.V - v0 : kVT;
  const int len = p.len(b);
  const long long bh = (long long)b * p.H + h;
  const float* q = static_cast<const float*>(p.q) + (long long)b * p.L * p.ldq + (long long)gh * p.K;
  const float* k = static_cast<const float*>(p.k) + (long long)b * p.L * p.ldk + (long long)gh * p.K;
  const float* v = static_cast<const float*>(p.v) + (long long)b * p.L * p.ldv + (long long)h * p.V + v0;

  // the state this segment starts from: what the segments before composed, or h0, or zero
  Own<NT, KP, kVT> S;
  S.zero();
  if (s0 != nullptr && !SUM) {
    const float* src = s0 + (p.nseg > 1 ? bh * p.nseg + seg : bh) * p.K * p.V + v0;
    S.pairs(tid, [&](int kk, int vv, float& x, float& y) {
      if (kk < p.K && vv < vw) {
        x = src[(long long)kk * p.V + vv];
        y = src[(long long)kk * p.V + vv + 1];
      }
    });
  }
  Dec total = {0.f, 0.f};
  ChunkGates<C> gates;
  const int c0 = seg * p.cps, c1 = c0 + p.cps < p.nck ? c0 + p.cps : p.nck;
  if (tid < 32) gates.fetch(p, b, h, c0 * C, len, tid);
  for (int ck = c0; ck < c1; ++ck) {
    const int t0 = ck * C;
    const int rows = p.L - t0 < C ? p.L - t0 : C;
    const int valid = len - t0 < 0 ? 0 : len - t0 < C ? len - t0 : C;
    if (valid == 0) {  // past the row's end: nothing decays, adds or reads
      if (!SUM)
        for (int i = tid; i < rows * vw; i += NT)
          o[(((long long)b * p.L + t0 + i / vw) * p.H + h) * p.V + v0 + i % vw] = 0.f;
      continue;
    }
    if (!SUM) load_tile<NT, C, KP, LK>(q + t0 * p.ldq, p.ldq, valid, p.K, sm.q, tid);
    load_tile<NT, C, KP, LK>(k + t0 * p.ldk, p.ldk, valid, p.K, sm.k, tid);
    load_tile<NT, C, kVT, LV>(v + t0 * p.ldv, p.ldv, valid, vw, sm.v, tid);
    if (tid < 32) {
      gates.scan(tid, [&](int i, Dec e) { sm.chi[i] = e.hi; sm.clo[i] = e.lo; });
      __syncwarp();
      for (int i = tid; i < C; i += 32) sm.rest[i] = dec_diff(sm.chi[C - 1], sm.clo[C - 1], sm.chi[i], sm.clo[i]);
      gates.fetch(p, b, h, t0 + C, len, tid);
    }
    if (!SUM)
      S.pairs(tid, [&](int kk, int vv, float& x, float& y) {
        st_pair(sm.s + kk * LV + vv, x, y);
        if (ckpt != nullptr && kk < p.K && vv < vw) st_pair(ckpt + ((bh * p.nck + ck) * p.K + kk) * p.V + v0 + vv, x, y);
      });
    __syncthreads();
    if (!SUM) {
      Own<NT, C, C> pr;
      Own<NT, C, kVT> a;
      pr.zero();
      mm<false, true, LK, LK, KP>(sm.q, sm.k, pr, tid);
      a.zero();
      mm<false, false, LK, LV, KP>(sm.q, sm.s, a, tid);
      __syncthreads();
      float* sp = sm.q;
      pr.pairs(tid, [&](int i, int j, float& x, float& y) {
        const float hi = sm.chi[i], lo = sm.clo[i];
        st_pair(sp + i * LC + j, j <= i ? x * dec_diff(hi, lo, sm.chi[j], sm.clo[j]) : 0.f,
                j + 1 <= i ? y * dec_diff(hi, lo, sm.chi[j + 1], sm.clo[j + 1]) : 0.f);
      });
      a.scale_rows(tid, [&](int i) { return dec_exp(sm.chi[i], sm.clo[i]); });
      __syncthreads();
      mm<false, false, LC, LV, C>(sp, sm.v, a, tid);
      a.pairs(tid, [&](int i, int vv, float& x, float& y) {
        if (i < rows && vv < vw)
          st_pair(o + (((long long)b * p.L + t0 + i) * p.H + h) * p.V + v0 + vv, i < valid ? p.scale * x : 0.f, i < valid ? p.scale * y : 0.f);
      });
    }
    const float chi = sm.chi[C - 1], clo = sm.clo[C - 1];
    total = dec_add(total, Dec{chi, clo});
    for (int i = tid; i < C * (KP / 4); i += NT) {  // k_j e^{c_last - c_j}
      float4* at = reinterpret_cast<float4*>(sm.k + i / (KP / 4) * LK) + i % (KP / 4);
      const float w = sm.rest[i / (KP / 4)];
      float4 x = *at;
      x.x *= w; x.y *= w; x.z *= w; x.w *= w;
      *at = x;
    }
    const float e = dec_exp(chi, clo);
    S.scale_rows(tid, [&](int) { return e; });
    __syncthreads();
    mm<true, false, LK, LV, C>(sm.k, sm.v, S, tid);
    __syncthreads();
  }
  float* dst = nullptr;
  if (SUM) dst = send + (bh * p.nseg + seg) * p.K * p.V;
  else if (send != nullptr && seg == p.nseg - 1) dst = send + bh * p.K * p.V;
  if (dst != nullptr)
    S.pairs(tid, [&](int kk, int vv, float& x, float& y) {
      if (kk < p.K && vv < vw) st_pair(dst + (long long)kk * p.V + v0 + vv, x, y);
    });
  if (SUM && tid == 0 && vt == 0) sdec[bh * p.nseg + seg] = total;
}

// ---------------------------------------------------------------- bf16: tensor cores
// A CTA walks the chunks (128 tokens) of one (batch row, head, segment).  The
// state stays in registers in fp32 (thread = row d of K and a quarter of the V
// columns) and goes to shared memory as bf16 for the product with q.
//   P  = q k^T               -> scaled by the decays, rounded to bf16, back to tensor memory as an A operand
//   O  = q S_in              -> * e^{c_i} in fp32 (bf16 S_in)
//   Sn = k^T (w v),  w_j = e^{c_last - c_j}: w v as three bf16 terms, an fp32-exact product
//   O += P v
// A term of o is rounded to bf16 once on its way (as a score or as a state).
//
// Sixteen warps compute; one issues the TMA loads and the MMAs (whose issue
// blocks while the tensor cores are behind), one finds the next chunk's decays.
// They meet at mbarriers only: the products of the state run under the scaling
// of the scores, v has two tiles so that the next chunk's w v begins under this
// one's output, and the third term of w v waits in tensor memory for the state's
// tile to be free.  o is staged in the chunk's tile of v and sent from there by
// TMA, behind the next chunk's products (copied out by the computing warps it
// held up the state: 2700 of a chunk's 9100 cycles).
// Measured: 75 us for 4 x 2048 tokens of 32 heads of 128 x 128 with 32 heads of k,
// 54 % of the copy bandwidth; a chunk takes 9100 cycles of which the chain
// w v -> Sn -> S -> its tile -> q S -> o binds 6400.  All of V in one CTA: with 64 columns a CTA and two CTAs an SM
// the scores were made and scaled twice and the narrow products waited for
// shared memory (114 us).  Five warps on some of the SM's quarters leave a thread 96
// registers; with VP = 128 56 bytes of it spill.  Tiles of q and k are 128 columns wide
// whatever K is: with K <= 64 half of the computing threads hold no row of the state
// (8 x 2048 tokens of 24 heads of 64 x 64: 94 us for 30 of copying).
template <int VP>
struct FwdTc {
  static constexpr int vt = kTC * VP * 2;  // bytes of a tile VP columns wide
  static constexpr int q = 0, k = q + 2 * kPanel, v = k + 2 * kPanel, w = v + 2 * vt, s = w + 2 * vt, dec = s + vt;
  // barriers: v (two tiles), q, k landed, decays stored; two terms of w v stored; scores and third term stored and O scaled;
  // state tile stored; O read; P, O, Sn, O + P v done
  static constexpr int kLv = 0, kLq = 2, kLk = 3, kDc = 4, kMp = 5, kMo = 6, kMs = 7, kM1 = 8, kW = 9, kSc = 10, kSt = 11, kRd = 12, nbar = 13;
  static constexpr int bar = dec + DecTile::bytes, tm = bar + nbar * 8, bytes = tm + 8;
  // tensor memory columns.  VP = 64: the first two terms side by side are one product of 128 columns, Sn has three parts
  static constexpr int P = 0, Pb = 128, O = 192, Sn = 192 + VP, Wp = VP == 64 ? Sn + 192 : Sn + 128, cols = 512;
};

struct FwdMaps {
  CUtensorMap q, k, v, o;
};

template <int VP>
__global__ void __launch_bounds__(kLinThreads, 1) linattn_fwd_tc_kernel(LinAttn p, const __grid_constant__ FwdMaps maps,
                                                                        const float* __restrict__ s0, __nv_bfloat16* __restrict__ o,
                                                                        float* __restrict__ ckpt, float* __restrict__ send) {
  using L = FwdTc<VP>;
  constexpr int VQ = VP / 4, NU = VQ / 8;  // columns and 16-byte units of a thread's quarter of V
  extern __shared__ __align__(1024) unsigned char raw[];
  const uint32_t sb = smem_u32(raw);
  const DecTile dec{sb + L::dec};
  uint64_t* bar = reinterpret_cast<uint64_t*>(raw + L::bar);
  uint32_t* tma = reinterpret_cast<uint32_t*>(raw + L::tm);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  long long id = blockIdx.x;
  const int seg = (int)(id % p.nseg);
  id /= p.nseg;
  const int h = (int)(id % p.H), b = (int)(id / p.H), gh = h / (p.H / p.G);
  const int len = p.len(b);
  const long long bh = (long long)b * p.H + h;
  const int c0 = seg * p.cps, c1 = c0 + p.cps < p.nck ? c0 + p.cps : p.nck;
  int cend = (len + kTC - 1) / kTC;  // chunks that hold a token
  cend = cend < c0 ? c0 : cend < c1 ? cend : c1;

  if (tid == 0) {
    for (int i = 0; i < L::nbar; ++i) mbar_init(&bar[i], i >= L::kW ? kLinWarps : 1);
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
    const int ks = (p.K + 15) / 16;  // contraction steps over K
    // a chunk's tiles; their readers have passed a barrier that this warp has waited for, with a proxy fence before it
    auto load_q = [&](int ck) {
      if (elect_one()) {
        mbar_arrive_expect_tx(&bar[L::kLq], 2 * kPanel);
        load_panels(sb + L::q, 2, &maps.q, &bar[L::kLq], 0, gh, ck * kTC, b);
      }
      __syncwarp();
    };
    auto load_k = [&](int ck) {
      if (elect_one()) {
        mbar_arrive_expect_tx(&bar[L::kLk], 2 * kPanel);
        load_panels(sb + L::k, 2, &maps.k, &bar[L::kLk], 0, gh, ck * kTC, b);
      }
      __syncwarp();
    };
    auto load_v = [&](int ck) {
      const int at = (ck - c0) & 1;
      if (elect_one()) {
        mbar_arrive_expect_tx(&bar[L::kLv + at], L::vt);
        load_panels(sb + L::v + at * L::vt, VP / 64, &maps.v, &bar[L::kLv + at], 0, h, ck * kTC, b);
      }
      __syncwarp();
    };
    // (bulk groups belong to the thread that committed them: the elected one is always the same)
    auto store_o = [&](int ck) {  // a chunk's o, staged in its tile of v
      if (elect_one()) {
        for (int i = 0; i < (p.V + 63) / 64; ++i)
          tma_store_4d(&maps.o, sb + L::v + ((ck - c0) & 1) * L::vt + i * kPanel, i * 64, h, ck * kTC, b);
        bulk_commit();
      }
      __syncwarp();
    };
    if (c0 < cend) {
      load_v(c0);
      load_q(c0);
      load_k(c0);
    }
    for (int ck = c0; ck < cend; ++ck) {
      const uint32_t par = (uint32_t)(ck - c0) & 1u;
      const uint32_t vtile = L::v + par * L::vt;
      const int valid = len - ck * kTC;
      const bool more = ck + 1 < cend, cut = valid < kTC && ck * kTC + valid < p.L;
      if (!wait(L::kLq, par) || !wait(L::kLk, par)) break;
      if (cut) {  // the row ends inside the tensor: what follows is not its own
        zero_rows(sb + L::q, 4, valid, lane);
        fence_proxy_async_smem();
        __syncwarp();
      }
      if (elect_one()) {  // the scores of the chunk before have been read: its kSc has been waited for
        tc_fence_after_sync();
        mma_steps(tm + L::P, Rows{sb + L::q}, Rows{sb + L::k}, mma_idesc(kTC, false, false), ks, false);
        mma_commit(&bar[L::kMp]);
      }
      __syncwarp();
      if (!wait(L::kSt, par) || !wait(L::kRd, par)) break;
      if (ck > c0) store_o(ck - 1);
      if (elect_one()) {
        tc_fence_after_sync();
        mma_steps(tm + L::O, Rows{sb + L::q}, Cols{sb + L::s}, mma_idesc(VP, false, true), ks, false);
        mma_commit(&bar[L::kMo]);
      }
      __syncwarp();
      if (!wait(L::kW, par)) break;
      if (cut) {  // (the v tile's other readers take its dead rows as zero)
        zero_rows(sb + vtile, VP / 64, valid, lane);
        fence_proxy_async_smem();
        __syncwarp();
      }
      if (elect_one()) {
        tc_fence_after_sync();
        if constexpr (VP == 64) {
          mma_steps(tm + L::Sn, Cols{sb + L::k}, Cols{sb + L::w}, mma_idesc(128, true, true), kTC / 16, false);
        } else {
          mma_steps(tm + L::Sn, Cols{sb + L::k}, Cols{sb + L::w + L::vt}, mma_idesc(VP, true, true), kTC / 16, false);
          mma_steps(tm + L::Sn, Cols{sb + L::k}, Cols{sb + L::w}, mma_idesc(VP, true, true), kTC / 16, true);
        }
      }
      __syncwarp();
      if (!wait(L::kMo, par)) break;
      if (more) {
        load_q(ck + 1);
        if (elect_one()) bulk_wait_read();  // v's place held the o of the chunk before
        __syncwarp();
        load_v(ck + 1);
      }
      if (!wait(L::kSc, par)) break;
      if (elect_one()) {
        tc_fence_after_sync();
        mma_steps(tm + L::Sn + (VP == 64 ? 128 : 0), Cols{sb + L::k}, Cols{sb + L::s}, mma_idesc(VP, true, true), kTC / 16, VP != 64);
        mma_commit(&bar[L::kMs]);
#pragma unroll
        for (int s = 0; s < kTC / 16; ++s)
          mma_ts(tm + L::O, tm + L::Pb + s * 8, desc_cols(sb + vtile, s), mma_idesc(VP, false, true), true);
        mma_commit(&bar[L::kM1]);
      }
      __syncwarp();
      if (more) {
        if (!wait(L::kMs, par)) break;
        load_k(ck + 1);
        if (ck + 2 < cend && elect_one()) {  // the chunk after it towards L2
          prefetch_panels((p.V + 63) / 64, &maps.v, 0, h, (ck + 2) * kTC, b);
          prefetch_panels((p.K + 63) / 64, &maps.q, 0, gh, (ck + 2) * kTC, b);
          prefetch_panels((p.K + 63) / 64, &maps.k, 0, gh, (ck + 2) * kTC, b);
        }
        __syncwarp();
      }
    }
    if (ok && c0 < cend && wait(L::kRd, (uint32_t)(cend - c0) & 1u)) store_o(cend - 1);
    if (elect_one()) bulk_wait();
    __syncwarp();
  } else if (warp > kLinWarps) {  // ---- the decays' warp: a chunk ahead, stored when the chunk before has read its own
    DecStage ds;
    ds.g.fetch(p, b, h, c0 * kTC, len, lane);
    for (int ck = c0; ck < cend; ++ck) {
      ds.scan(lane);
      if (ck > c0 && !wait(L::kSc, (uint32_t)(ck - 1 - c0) & 1u)) break;
      ds.put(dec, lane);
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar[L::kDc]);
      ds.g.fetch(p, b, h, (ck + 1) * kTC, len, lane);
    }
  } else {  // ---- a computing warp
    const int row = (warp & 3) * 32 + lane, cq = warp >> 2;  // tensor-memory lane and quarter of the columns of this thread
    const uint32_t tl = tm + ((uint32_t)((warp & 3) * 32) << 16);
    float S[VQ];
#pragma unroll
    for (int e = 0; e < VQ; ++e) S[e] = 0.f;
    if (s0 != nullptr && row < p.K) {
      const float* src = s0 + ((p.nseg > 1 ? bh * p.nseg + seg : bh) * p.K + row) * p.V + cq * VQ;
#pragma unroll
      for (int e = 0; e < VQ; e += 4)
        if (cq * VQ + e < p.V) {
          const float4 x = *reinterpret_cast<const float4*>(src + e);
          S[e] = x.x; S[e + 1] = x.y; S[e + 2] = x.z; S[e + 3] = x.w;
        }
    }
    auto arrive = [&](int i) {  // this warp's shared- and tensor-memory accesses before are over
      fence_proxy_async_smem();
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar[i]);
    };
    auto store_s = [&]() {  // S_in as a bf16 tile
#pragma unroll
      for (int u = 0; u < NU; ++u) {
        const float x[8] = {S[8 * u], S[8 * u + 1], S[8 * u + 2], S[8 * u + 3], S[8 * u + 4], S[8 * u + 5], S[8 * u + 6], S[8 * u + 7]};
        sts16(sb + L::s + tile_at(row, cq * NU + u), pack8(x));
      }
    };
    if (c0 < cend) {
      store_s();
      arrive(L::kSt);
      arrive(L::kRd);
    }
    for (int ck = c0; ck < cend; ++ck) {
      const uint32_t par = (uint32_t)(ck - c0) & 1u;
      const int t0 = ck * kTC, valid = len - t0;
      const uint32_t vtile = sb + L::v + par * L::vt;
      if (!wait(L::kDc, par) || !wait(L::kLv + (int)par, (uint32_t)((ck - c0) >> 1) & 1u)) break;
      const Dec last = dec.get(kTC - 1), own = dec.get(row);
      const float elast = dec_exp(last);
      {
        const float wj = dec_exp(dec_sub(last, own));
        uint32_t third[NU * 4];
#pragma unroll
        for (int u = 0; u < NU; ++u) {  // w v of this thread's token
          const uint32_t at = tile_at(row, cq * NU + u);
          float x[8];
          Raw8<__nv_bfloat16>::wide(row < valid ? lds16(vtile + at) : make_uint4(0u, 0u, 0u, 0u), x);
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] *= wj;
          sts16(sb + L::w + at, take_term(x));
          sts16(sb + L::w + L::vt + at, take_term(x));
          const uint4 t = last_term(x);
          third[4 * u] = t.x; third[4 * u + 1] = t.y; third[4 * u + 2] = t.z; third[4 * u + 3] = t.w;
        }
        __syncwarp();
        tmem_stn(tl + L::Wp + cq * NU * 4, third);
        tmem_wait_st();
        arrive(L::kW);
      }
      if (!wait(L::kMp, par)) break;
      tc_fence_after_sync();
      {  // 32 key tokens: all before this warp's tokens, among them, or after them
        uint32_t w[16];
        if (cq <= (warp & 3)) {
          uint32_t r[32];
          tmem_ld32(tl + L::P + cq * 32, r);
          const Dec d = dec_sub(own, dec.base(cq));
          const float x = d.hi + d.lo;
          tmem_wait_ld();
          if (cq < (warp & 3)) {
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              const float4 c = dec.r4(cq * 32 + e);
              w[e / 2] = pack_bf16(__uint_as_float(r[e]) * ex2(x - c.x), __uint_as_float(r[e + 1]) * ex2(x - c.y));
              w[e / 2 + 1] = pack_bf16(__uint_as_float(r[e + 2]) * ex2(x - c.z), __uint_as_float(r[e + 3]) * ex2(x - c.w));
            }
          } else {
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              const float4 c = dec.r4(cq * 32 + e);
              w[e / 2] = pack_bf16(e <= lane ? __uint_as_float(r[e]) * ex2(x - c.x) : 0.f,
                                   e + 1 <= lane ? __uint_as_float(r[e + 1]) * ex2(x - c.y) : 0.f);
              w[e / 2 + 1] = pack_bf16(e + 2 <= lane ? __uint_as_float(r[e + 2]) * ex2(x - c.z) : 0.f,
                                       e + 3 <= lane ? __uint_as_float(r[e + 3]) * ex2(x - c.w) : 0.f);
            }
          }
        } else {
#pragma unroll
          for (int e = 0; e < 16; ++e) w[e] = 0u;
        }
        tmem_st16(tl + L::Pb + cq * 16, w);
      }
      if (!wait(L::kMo, par)) break;
      tc_fence_after_sync();
      {  // the state's tile has been read: the third term takes it
        uint32_t third[NU * 4];
        tmem_ldn(tl + L::Wp + cq * NU * 4, third);
        tmem_wait_ld();
#pragma unroll
        for (int u = 0; u < NU; ++u)
          sts16(sb + L::s + tile_at(row, cq * NU + u), make_uint4(third[4 * u], third[4 * u + 1], third[4 * u + 2], third[4 * u + 3]));
      }
      tmem_scale<VQ>(tl + L::O + cq * VQ, dec_exp(own));
      tmem_wait_st();
      arrive(L::kSc);
      if (ckpt != nullptr && row < p.K) {
        float4* dst = reinterpret_cast<float4*>(ckpt + (bh * p.nck + ck) * p.K * p.V) + row;
#pragma unroll
        for (int e = 0; e < VQ; e += 4)
          if (cq * VQ + e < p.V) dst[(long long)((cq * VQ + e) / 4) * p.K] = make_float4(S[e], S[e + 1], S[e + 2], S[e + 3]);
      }
      if (!wait(L::kMs, par)) break;
      tc_fence_after_sync();
      {
        uint32_t r[VQ];
        if constexpr (VP == 64) {
          uint32_t r1[VQ], r2[VQ];
          tmem_ldn(tl + L::Sn + cq * VQ, r);
          tmem_ldn(tl + L::Sn + 64 + cq * VQ, r1);
          tmem_ldn(tl + L::Sn + 128 + cq * VQ, r2);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < VQ; ++e)
            r[e] = __float_as_uint(__uint_as_float(r[e]) + (__uint_as_float(r1[e]) + __uint_as_float(r2[e])));
        } else {
          tmem_ldn(tl + L::Sn + cq * VQ, r);
          tmem_wait_ld();
        }
#pragma unroll
        for (int e = 0; e < VQ; ++e) S[e] = fmaf(S[e], elast, __uint_as_float(r[e]));
      }
      if (ck + 1 < cend) {
        store_s();
        arrive(L::kSt);
      }
      if (!wait(L::kM1, par)) break;
      tc_fence_after_sync();
      {  // o into v's place (P v is done); the issuing warp sends it from there
        uint32_t r[VQ];
        tmem_ldn(tl + L::O + cq * VQ, r);
        tmem_wait_ld();
#pragma unroll
        for (int u = 0; u < NU; ++u) {
          float x[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = row < valid ? p.scale * __uint_as_float(r[8 * u + e]) : 0.f;
          sts16(vtile + tile_at(row, cq * NU + u), pack8(x));
        }
        arrive(L::kRd);
      }
    }
    if (ok) {
      for (int ck = cend; ck < c1; ++ck) {  // past the row's end
        const int rows = p.L - ck * kTC < kTC ? p.L - ck * kTC : kTC, n = p.V / 8;
        for (int i = tid; i < rows * n; i += 32 * kLinWarps)
          *reinterpret_cast<uint4*>(o + (((long long)b * p.L + ck * kTC + i / n) * p.H + h) * p.V + i % n * 8) = make_uint4(0u, 0u, 0u, 0u);
      }
    }
    if (send != nullptr && seg == p.nseg - 1 && row < p.K) {
      float* dst = send + (bh * p.K + row) * p.V + cq * VQ;
#pragma unroll
      for (int e = 0; e < VQ; e += 4)
        if (cq * VQ + e < p.V) *reinterpret_cast<float4*>(dst + e) = make_float4(S[e], S[e + 1], S[e + 2], S[e + 3]);
    }
  }
  lin_leave(ok, bar, L::nbar, tm, L::cols, warp, lane);
}

struct FwdPlan {
  LinAttn p;
  long long walks;  // (batch row, head) and for fp32 column tile
  size_t states, bytes;
};

int fwd_plan(int B, int L, int H, int G, int K, int V, int dtype, FwdPlan& pl) {
  const int rc = linattn_validate(B, L, H, G, K, V, dtype);
  if (rc != SS_OK) return rc;
  pl.p = LinAttn{};
  pl.p.B = B; pl.p.L = L; pl.p.H = H; pl.p.G = G; pl.p.K = K; pl.p.V = V;
  pl.walks = (long long)B * H * (dtype == SS_F32 ? (V + kVT - 1) / kVT : 1);
  if (pl.walks > (1ll << 24)) return SS_ERR_DIM;
  linattn_segments(pl.p, dtype, pl.walks);
  pl.states = pl.p.nseg > 1 ? (size_t)B * H * pl.p.nseg * K * V * sizeof(float) : 0;
  pl.bytes = pl.p.nseg > 1 ? pl.states + (size_t)B * H * pl.p.nseg * sizeof(Dec) : 0;
  return SS_OK;
}

// The walk; for a row cut in segments first their end states, then the states they start from.
template <typename Sum, typename Walk>
int fwd_run(const FwdPlan& pl, const float* h0, void* ws, cudaStream_t s, Sum sum, Walk walk) {
  const LinAttn& p = pl.p;
  if (p.nseg == 1) return walk(h0);
  float* st = static_cast<float*>(ws);
  Dec* dec = reinterpret_cast<Dec*>(static_cast<char*>(ws) + pl.states);
  const int rc = sum(st, dec);
  if (rc != SS_OK) return rc;
  const long long kv = (long long)p.K * p.V;
  linattn_join_kernel<false><<<dim3((unsigned)((kv + 255) / 256), (unsigned)(p.B * p.H)), 256, 0, s>>>(h0, st, dec, kv, p.nseg);
  if (cudaGetLastError() != cudaSuccess) return SS_ERR_CUDA;
  return walk(st);
}

template <int KP>
int fwd_f32(const FwdPlan& pl, const float* h0, float* o, float* ckpt, float* h_last, void* ws, cudaStream_t s) {
  const unsigned grid = (unsigned)pl.walks * pl.p.nseg;
  const size_t smem = sizeof(FwdSmem<KP>);
  return fwd_run(
      pl, h0, ws, s,
      [&](float* st, Dec* dec) { return lin_launch(linattn_fwd_kernel<KP, true>, grid, FwdSmem<KP>::NT, offsetof(FwdSmem<KP>, q), s, pl.p, nullptr, o, ckpt, st, dec); },
      [&](const float* s0) { return lin_launch(linattn_fwd_kernel<KP, false>, grid, FwdSmem<KP>::NT, smem, s, pl.p, s0, o, ckpt, h_last, nullptr); });
}

template <int VP>
int fwd_bf16(const FwdPlan& pl, const float* h0, __nv_bfloat16* o, float* ckpt, float* h_last, void* ws, cudaStream_t s) {
  const LinAttn& p = pl.p;
  const unsigned grid = (unsigned)pl.walks * p.nseg;
  FwdMaps maps;
  if (!lin_map(&maps.q, p.q, p.ldq, p.B, p.L, p.G, p.K) || !lin_map(&maps.k, p.k, p.ldk, p.B, p.L, p.G, p.K) ||
      !lin_map(&maps.v, p.v, p.ldv, p.B, p.L, p.H, p.V) || !lin_map(&maps.o, o, (long long)p.H * p.V, p.B, p.L, p.H, p.V))
    return SS_ERR_CUDA;
  return fwd_run(
      pl, h0, ws, s,
      [&](float* st, Dec* dec) {
        return lin_launch(linattn_sum_tc_kernel<false>, grid * ((p.V + 63) / 64), kLinThreads, SumTc::bytes, s, p, maps.k, maps.v, st, dec);
      },
      [&](const float* s0) { return lin_launch(linattn_fwd_tc_kernel<VP>, grid, kLinThreads, FwdTc<VP>::bytes, s, p, maps, s0, o, ckpt, h_last); });
}

}  // namespace

extern "C" int linattn_num_chunks(int L, int dtype) {
  if (L <= 0 || L > kLinMaxLen || (dtype != SS_F32 && dtype != SS_BF16)) return 0;
  const int c = linattn_chunk(dtype);
  return (L + c - 1) / c;
}

extern "C" size_t linattn_fwd_workspace_size(int B, int L, int H, int G, int K, int V, int dtype) {
  FwdPlan pl;
  return fwd_plan(B, L, H, G, K, V, dtype, pl) == SS_OK ? pl.bytes : 0;
}

extern "C" int linattn_fwd(const void* q, long long ldq, const void* k, long long ldk, const void* v, long long ldv,
                           const float* g, int g_per_head, const float* h0, const int* lengths, void* o, float* ckpt,
                           float* h_last, int B, int L, int H, int G, int K, int V, float scale, int dtype, void* workspace,
                           size_t ws_bytes, void* stream) {
  if (!q || !k || !v || !g || !o) return SS_ERR_NULL;
  FwdPlan pl;
  int rc = fwd_plan(B, L, H, G, K, V, dtype, pl);
  if (rc != SS_OK) return rc;
  if ((rc = linattn_ld_ok(ldq, G, K)) != SS_OK || (rc = linattn_ld_ok(ldk, G, K)) != SS_OK ||
      (rc = linattn_ld_ok(ldv, H, V)) != SS_OK)
    return rc;
  const void* ptrs[] = {q, k, v, o, h0, ckpt, h_last};
  for (const void* x : ptrs)
    if (x != nullptr && !ssh::aligned16(x)) return SS_ERR_ALIGN;
  if ((reinterpret_cast<uintptr_t>(g) & 3u) || (reinterpret_cast<uintptr_t>(lengths) & 3u)) return SS_ERR_ALIGN;
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
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dtype == SS_F32)  // (24 heads of 64 x 64, forward and backward: 1449 us in tiles of 64 rows, 2051 in tiles of 128)
    return K <= 64 ? fwd_f32<64>(pl, h0, static_cast<float*>(o), ckpt, h_last, workspace, s)
                   : fwd_f32<128>(pl, h0, static_cast<float*>(o), ckpt, h_last, workspace, s);
  // (16384 tokens of 32 heads of 128 x 64: 152 us in tiles of 64 columns, 187 in tiles of 128)
  return V <= 64 ? fwd_bf16<64>(pl, h0, static_cast<__nv_bfloat16*>(o), ckpt, h_last, workspace, s)
                 : fwd_bf16<128>(pl, h0, static_cast<__nv_bfloat16*>(o), ckpt, h_last, workspace, s);
}

namespace ssh {
int read_clear_linf_err(cudaStream_t s, unsigned* out) { return read_clear_lin_err(s, out); }
}  // namespace ssh
