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
#include "linattn_common.cuh"

namespace {

using namespace ssk;

template <int KP, int VP>
struct BwdSmem {
  static constexpr int C = kLinChunkF32, LK = KP + 4, LV = VP + 4, LC = C + 4;
  float q[C * LK], k[C * LK], v[C * LV], d[C * LV], s[KP * LV], p[C * LC], chi[C], clo[C], a[C], b[C], rect[C], red[8];
};

struct BwdOut {
  void *dq, *dk, *dv;
  float *dqp, *dkp;  // fp32 per-head parts when heads share q, k (then dq, dk are summed from them)
  float* dg;         // [B, L, H], or per-chunk sums [B * nck, H] with a decay per head
  float* dh0;
};

// A CTA walks the chunks of one (batch row, head, segment) from the last to the
// first with U in registers.  SUM only finds the segment's U from zero.
template <typename T, int KP, int VP, bool SUM>
__global__ void __launch_bounds__(256) linattn_bwd_kernel(LinAttn p, const T* __restrict__ dout, const float* __restrict__ ckpt,
                                                          const float* __restrict__ u0, BwdOut out, float* __restrict__ uend,
                                                          double* __restrict__ udec) {
  using Sm = BwdSmem<KP, VP>;
  constexpr int C = Sm::C, LK = Sm::LK, LV = Sm::LV, LC = Sm::LC, RK = KP / 16, RV = VP / 16;
  extern __shared__ __align__(16) unsigned char raw[];
  Sm& sm = *reinterpret_cast<Sm*>(raw);
  const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
  long long id = blockIdx.x;
  const int seg = (int)(id % p.nseg);
  id /= p.nseg;
  const int h = (int)(id % p.H), b = (int)(id / p.H);
  const int gh = h / (p.H / p.G);
  const int len = p.len(b);
  const long long bh = (long long)b * p.H + h, kv = (long long)p.K * p.V;
  const T* q = static_cast<const T*>(p.q) + (long long)b * p.L * p.ldq + (long long)gh * p.K;
  const T* k = static_cast<const T*>(p.k) + (long long)b * p.L * p.ldk + (long long)gh * p.K;
  const T* v = static_cast<const T*>(p.v) + (long long)b * p.L * p.ldv + (long long)h * p.V;
  const long long ldo = (long long)p.H * p.V;
  const T* d = dout + (long long)b * p.L * ldo + (long long)h * p.V;

  float U[RK][RV];
  zero_acc(U);
  if (u0 != nullptr && !SUM) {
    const float* src = u0 + (p.nseg > 1 ? bh * p.nseg + seg : bh) * kv;
#pragma unroll
    for (int r = 0; r < RK; ++r)
#pragma unroll
      for (int c = 0; c < RV; ++c) {
        const int kk = ty * RK + r, vv = tx + 16 * c;
        if (kk < p.K && vv < p.V) U[r][c] = src[(long long)kk * p.V + vv];
      }
  }
  // gradients of q or k of token row i: typed when each head has its own, else this head's fp32 part
  auto put_qk = [&](void* typed, float* part, int t0, int rows, int valid, const float (&a)[4][RK]) {
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int c = 0; c < RK; ++c) {
        const int i = ty * 4 + r, kk = tx + 16 * c;
        if (i >= rows || kk >= p.K) continue;
        const long long at = (((long long)b * p.L + t0 + i) * p.H + h) * p.K + kk;
        const float x = i < valid ? a[r][c] : 0.f;
        if (part != nullptr) part[at] = x;
        else ActT<T>::st1(static_cast<T*>(typed) + at, x);
      }
  };
  double total = 0.0;
  const int c0 = seg * p.cps, c1 = c0 + p.cps < p.nck ? c0 + p.cps : p.nck;
  for (int ck = c1 - 1; ck >= c0; --ck) {
    const int t0 = ck * C;
    const int rows = p.L - t0 < C ? p.L - t0 : C;
    const int valid = len - t0 < 0 ? 0 : len - t0 < C ? len - t0 : C;
    if (valid == 0) {
      if (!SUM) {
        float z[4][RK];
        zero_acc(z);
        put_qk(out.dq, out.dqp, t0, rows, 0, z);
        put_qk(out.dk, out.dkp, t0, rows, 0, z);
        for (int i = tid; i < rows * p.V; i += 256)
          ActT<T>::st1(static_cast<T*>(out.dv) + (((long long)b * p.L + t0 + i / p.V) * p.H + h) * p.V + i % p.V, 0.f);
        if (p.g_head) {
          if (tid == 0) out.dg[((long long)b * p.nck + ck) * p.H + h] = 0.f;
        } else if (tid < rows) {
          out.dg[((long long)b * p.L + t0 + tid) * p.H + h] = 0.f;
        }
      }
      continue;
    }
    if (tid < 32) chunk_decays<C>(p, b, h, t0, len, tid, sm.chi, sm.clo);
    load_tile<T, C, KP, LK>(q + t0 * p.ldq, p.ldq, valid, p.K, sm.q, tid);
    load_tile<T, C, VP, LV>(d + t0 * ldo, ldo, valid, p.V, sm.d, tid);
    if (!SUM) {
      load_tile<T, C, KP, LK>(k + t0 * p.ldk, p.ldk, valid, p.K, sm.k, tid);
      load_tile<T, C, VP, LV>(v + t0 * p.ldv, p.ldv, valid, p.V, sm.v, tid);
      const float* src = ckpt + (bh * p.nck + ck) * kv;
#pragma unroll
      for (int r = 0; r < RK; ++r)
#pragma unroll
        for (int c = 0; c < RV; ++c) {
          const int kk = ty * RK + r, vv = tx + 16 * c;
          sm.s[kk * LV + vv] = kk < p.K && vv < p.V ? src[(long long)kk * p.V + vv] : 0.f;
        }
    }
    __syncthreads();
    const float chi = sm.chi[C - 1], clo = sm.clo[C - 1];
    total += (double)chi + (double)clo;
    float m[4][4], pr[4][4];
    if (!SUM) {
      float part = 0.f;  // <S_in, U>
#pragma unroll
      for (int r = 0; r < RK; ++r)
#pragma unroll
        for (int c = 0; c < RV; ++c) part = fmaf(sm.s[(ty * RK + r) * LV + tx + 16 * c], U[r][c], part);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) part += __shfl_xor_sync(0xffffffffu, part, o);
      if ((tid & 31) == 0) sm.red[tid >> 5] = part;
      float dq[4][RK];
      zero_acc(dq);
      mm<C, KP, VP, false, true, LV, LV>(sm.d, sm.s, dq, tid);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int i = ty * 4 + r;
        const float e = p.scale * dec_exp(sm.chi[i], sm.clo[i]);
        float s = 0.f;
#pragma unroll
        for (int c = 0; c < RK; ++c) {
          dq[r][c] *= e;
          s = fmaf(sm.q[i * LK + tx + 16 * c], dq[r][c], s);
        }
        s = row_sum16(s);
        if (tx == 0) sm.a[i] = s;
      }
      zero_acc(m);
      zero_acc(pr);
      mm<C, C, VP, false, true, LV, LV>(sm.d, sm.v, m, tid);
      mm<C, C, KP, false, true, LK, LK>(sm.q, sm.k, pr, tid);
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int i = ty * 4 + r, j = tx + 16 * c;
          const float w = j <= i ? p.scale * dec_diff(sm.chi[i], sm.clo[i], sm.chi[j], sm.clo[j]) : 0.f;
          pr[r][c] = j <= i ? pr[r][c] * w : 0.f;
          sm.p[i * LC + j] = j <= i ? m[r][c] * w : 0.f;
          m[r][c] = j <= i ? m[r][c] * pr[r][c] : 0.f;
        }
      __syncthreads();
      mm<C, KP, C, false, false, LC, LK>(sm.p, sm.k, dq, tid);
      put_qk(out.dq, out.dqp, t0, rows, valid, dq);
      float dk[4][RK];
      zero_acc(dk);
      mm<C, KP, C, true, false, LC, LK>(sm.p, sm.q, dk, tid);
      __syncthreads();
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int c = 0; c < 4; ++c) sm.p[(ty * 4 + r) * LC + tx + 16 * c] = pr[r][c];
#pragma unroll
      for (int r = 0; r < RK; ++r)
#pragma unroll
        for (int c = 0; c < RV; ++c) sm.s[(ty * RK + r) * LV + tx + 16 * c] = U[r][c];
      __syncthreads();
      float dv[4][RV], rest[4];
      zero_acc(dv);
      mm<C, VP, KP, false, false, LK, LV>(sm.k, sm.s, dv, tid);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        rest[r] = dec_diff(chi, clo, sm.chi[ty * 4 + r], sm.clo[ty * 4 + r]);
#pragma unroll
        for (int c = 0; c < RV; ++c) dv[r][c] *= rest[r];
      }
      mm<C, VP, C, true, false, LC, LV>(sm.p, sm.d, dv, tid);
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int c = 0; c < RV; ++c) {
          const int i = ty * 4 + r, vv = tx + 16 * c;
          if (i < rows && vv < p.V)
            ActT<T>::st1(static_cast<T*>(out.dv) + (((long long)b * p.L + t0 + i) * p.H + h) * p.V + vv, i < valid ? dv[r][c] : 0.f);
        }
      float ki[4][RK];
      zero_acc(ki);
      mm<C, KP, VP, false, true, LV, LV>(sm.v, sm.s, ki, tid);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int j = ty * 4 + r;
        float s = 0.f;
#pragma unroll
        for (int c = 0; c < RK; ++c) {
          const float x = ki[r][c] * rest[r];
          s = fmaf(sm.k[j * LK + tx + 16 * c], x, s);
          dk[r][c] += x;
        }
        s = row_sum16(s);
        if (tx == 0) sm.b[j] = s;
      }
      put_qk(out.dk, out.dkp, t0, rows, valid, dk);
    }
    __syncthreads();
    if (!SUM) {
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int c = 0; c < 4; ++c) sm.p[(ty * 4 + r) * LC + tx + 16 * c] = m[r][c];
    }
    for (int i = tid; i < C * KP; i += 256) {  // scale e^{c_i} q_i
      const int t = i / KP;
      sm.q[t * LK + i % KP] *= p.scale * dec_exp(sm.chi[t], sm.clo[t]);
    }
    __syncthreads();
    if (!SUM) {
      // row r of M becomes its running sum over j < t, for t <= r; 4 lanes a row, 16 columns each
      {
        const int r = tid >> 2, s4 = tid & 3;
        float* row = sm.p + r * LC + s4 * 16;
        float x[16], run = 0.f;
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          x[e] = run;
          run += row[e];
        }
        float base = 0.f;
#pragma unroll
        for (int o = 1; o < 4; ++o) {
          const float u = __shfl_up_sync(0xffffffffu, run, o, 4);
          if (s4 >= o) base += u;
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) row[e] = s4 * 16 + e <= r ? base + x[e] : 0.f;
      }
      __syncthreads();
      {  // column sums: every path from before t to t or later
        const int t = tid >> 2, s4 = tid & 3;
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < 16; ++e) s += sm.p[(s4 * 16 + e) * LC + t];
        s += __shfl_xor_sync(0xffffffffu, s, 1);
        s += __shfl_xor_sync(0xffffffffu, s, 2);
        if (s4 == 0) sm.rect[t] = s;
      }
      __syncthreads();
      if (tid < 32) {  // two consecutive tokens a lane
        float through = 0.f;
#pragma unroll
        for (int w = 0; w < 8; ++w) through += sm.red[w];
        through *= dec_exp(chi, clo);
        const float a0 = sm.a[2 * tid], a1 = sm.a[2 * tid + 1], b0 = sm.b[2 * tid], b1 = sm.b[2 * tid + 1];
        double sa = (double)a0 + a1, sb = (double)b0 + b1;
        const double sb_own = sb;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const double ua = __shfl_down_sync(0xffffffffu, sa, o), ub = __shfl_up_sync(0xffffffffu, sb, o);
          if (tid + o < 32) sa += ua;
          if (tid >= o) sb += ub;
        }
        const double before = sb - sb_own;
        float g0 = (float)(sa + before + through + sm.rect[2 * tid]);
        float g1 = (float)((sa - a0) + (before + b0) + through + sm.rect[2 * tid + 1]);
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
#pragma unroll
    for (int r = 0; r < RK; ++r)
#pragma unroll
      for (int c = 0; c < RV; ++c) U[r][c] *= e;
    mm<KP, VP, C, true, false, LK, LV>(sm.q, sm.d, U, tid);
    __syncthreads();
  }
  float* dst = nullptr;
  if (SUM) dst = uend + (bh * p.nseg + seg) * kv;
  else if (out.dh0 != nullptr && seg == 0) dst = out.dh0 + bh * kv;
  if (dst != nullptr) {
#pragma unroll
    for (int r = 0; r < RK; ++r)
#pragma unroll
      for (int c = 0; c < RV; ++c) {
        const int kk = ty * RK + r, vv = tx + 16 * c;
        if (kk < p.K && vv < p.V) dst[(long long)kk * p.V + vv] = U[r][c];
      }
  }
  if (SUM && tid == 0) udec[bh * p.nseg + seg] = total;
}

// In place over the segments of a (batch row, head), last to first: the U found
// from zero becomes the U arriving at the segment's end.
__global__ void __launch_bounds__(256) linattn_bwd_join_kernel(const float* __restrict__ dh_last, float* __restrict__ st,
                                                               const double* __restrict__ dec, long long kv, int nseg) {
  const long long bh = blockIdx.y;
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  if (i >= kv) return;
  float s = dh_last != nullptr ? dh_last[bh * kv + i] : 0.f;
  for (int n = nseg - 1; n >= 0; --n) {
    float* at = st + (bh * nseg + n) * kv + i;
    const Dec d = dec_of(dec[bh * nseg + n]);
    const float end = *at;
    *at = s;
    s = fmaf(dec_exp(d.hi, d.lo), s, end);
  }
}

// dq, dk of a shared head: the parts of its R heads added in order, rounded once.
template <typename T>
__global__ void __launch_bounds__(256) linattn_share_kernel(const float* __restrict__ pq, const float* __restrict__ pk,
                                                            T* __restrict__ dq, T* __restrict__ dk, long long n, int R, int K) {
  const long long i = ((long long)blockIdx.x * 256 + threadIdx.x) * 4;  // K is a multiple of 8: four elements of one head
  if (i >= n) return;
  const float* src = blockIdx.y ? pk : pq;
  T* dst = blockIdx.y ? dk : dq;
  const long long row = i / K, at = row * R * K + i % K;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int r = 0; r < R; ++r) {
    const float4 x = *reinterpret_cast<const float4*>(src + at + (long long)r * K);
    a.x += x.x; a.y += x.y; a.z += x.z; a.w += x.w;
  }
  ActT<T>::st2(dst + i, a.x, a.y);
  ActT<T>::st2(dst + i + 2, a.z, a.w);
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
  linattn_segments(pl.p, linattn_chunk(dtype), walks, 152);
  const int n = pl.p.nseg;
  pl.states = n > 1 ? (size_t)walks * n * K * V * sizeof(float) : 0;
  pl.decs = n > 1 ? up16((size_t)walks * n * sizeof(double)) : 0;
  pl.parts = H != G ? (size_t)B * L * H * K * sizeof(float) : 0;
  pl.sums = g_head ? up16((size_t)B * pl.p.nck * H * sizeof(float)) : 0;
  pl.bytes = pl.states + pl.decs + 2 * pl.parts + pl.sums;
  return SS_OK;
}

template <typename T, int KP, int VP>
int bwd_launch(const BwdPlan& pl, const void* dout, const float* ckpt, const float* dh_last, BwdOut out, float* dg, char* ws,
               cudaStream_t s) {
  const LinAttn& p = pl.p;
  const size_t smem = sizeof(BwdSmem<KP, VP>);
  float* st = reinterpret_cast<float*>(ws);
  double* dec = reinterpret_cast<double*>(ws + pl.states);
  out.dqp = pl.parts ? reinterpret_cast<float*>(ws + pl.states + pl.decs) : nullptr;
  out.dkp = pl.parts ? reinterpret_cast<float*>(ws + pl.states + pl.decs + pl.parts) : nullptr;
  out.dg = p.g_head ? reinterpret_cast<float*>(ws + pl.states + pl.decs + 2 * pl.parts) : dg;
  auto run = [&](auto kern, const float* u0, float* uend, double* udec) -> int {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess) return SS_ERR_CUDA;
    const long long grid = (long long)p.B * p.H * p.nseg;
    kern<<<(unsigned)grid, 256, smem, s>>>(p, static_cast<const T*>(dout), ckpt, u0, out, uend, udec);
    return cudaGetLastError() == cudaSuccess ? SS_OK : SS_ERR_CUDA;
  };
  int rc;
  if (p.nseg == 1) {
    rc = run(linattn_bwd_kernel<T, KP, VP, false>, dh_last, nullptr, nullptr);
  } else {
    if ((rc = run(linattn_bwd_kernel<T, KP, VP, true>, nullptr, st, dec)) != SS_OK) return rc;
    const long long kv = (long long)p.K * p.V;
    linattn_bwd_join_kernel<<<dim3((unsigned)((kv + 255) / 256), (unsigned)(p.B * p.H)), 256, 0, s>>>(dh_last, st, dec, kv, p.nseg);
    if (cudaGetLastError() != cudaSuccess) return SS_ERR_CUDA;
    rc = run(linattn_bwd_kernel<T, KP, VP, false>, st, nullptr, nullptr);
  }
  if (rc != SS_OK) return rc;
  if (pl.parts) {
    const long long n = (long long)p.B * p.L * p.G * p.K;
    linattn_share_kernel<T><<<dim3((unsigned)((n / 4 + 255) / 256), 2), 256, 0, s>>>(out.dqp, out.dkp, static_cast<T*>(out.dq),
                                                                                 static_cast<T*>(out.dk), n, p.H / p.G, p.K);
    if (cudaGetLastError() != cudaSuccess) return SS_ERR_CUDA;
  }
  if (p.g_head && colsum(out.dg, p.H, p.B * p.nck, AddDg{dg}, s) != cudaSuccess) return SS_ERR_CUDA;
  return SS_OK;
}

template <typename T>
int bwd_dispatch(const BwdPlan& pl, const void* dout, const float* ckpt, const float* dh_last, const BwdOut& out, float* dg,
                 char* ws, cudaStream_t s) {
  if (pl.p.K <= 64)
    return pl.p.V <= 64 ? bwd_launch<T, 64, 64>(pl, dout, ckpt, dh_last, out, dg, ws, s)
                        : bwd_launch<T, 64, 128>(pl, dout, ckpt, dh_last, out, dg, ws, s);
  return pl.p.V <= 64 ? bwd_launch<T, 128, 64>(pl, dout, ckpt, dh_last, out, dg, ws, s)
                      : bwd_launch<T, 128, 128>(pl, dout, ckpt, dh_last, out, dg, ws, s);
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
  if ((rc = linattn_ld_ok(ldq, G * K)) != SS_OK || (rc = linattn_ld_ok(ldk, G * K)) != SS_OK ||
      (rc = linattn_ld_ok(ldv, H * V)) != SS_OK)
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
  if (dtype == SS_F32) return bwd_dispatch<float>(pl, dout, ckpt, dh_last, out, dg, ws, s);
  return bwd_dispatch<__nv_bfloat16>(pl, dout, ckpt, dh_last, out, dg, ws, s);
}
