// Linear attention with a decay for each head, chunked forward (linattn_fwd) for sm_103a.
#include "linattn_common.cuh"

namespace {

using namespace ssk;

// FP32 products on the FMA pipe.  A CTA walks the chunks of one (batch row,
// head, 64-column tile of V, segment) in order with the state in registers.
// SUM only finds the segment's end state from zero and its decay (no q, no o).
constexpr int kVT = 64;

template <int KP>
struct FwdSmem {
  static constexpr int C = kLinChunkF32, LK = KP + 4, LV = kVT + 4, LC = C + 4;
  float q[C * LK], k[C * LK], v[C * LV], s[KP * LV], p[C * LC], chi[C], clo[C];
};

template <typename T, int KP, bool SUM>
__global__ void __launch_bounds__(256) linattn_fwd_kernel(LinAttn p, const float* __restrict__ s0, T* __restrict__ o,
                                                          float* __restrict__ ckpt, float* __restrict__ send,
                                                          double* __restrict__ sdec) {
  using Sm = FwdSmem<KP>;
  constexpr int C = Sm::C, LK = Sm::LK, LV = Sm::LV, LC = Sm::LC, RK = KP / 16;
  extern __shared__ __align__(16) unsigned char raw[];
  Sm& sm = *reinterpret_cast<Sm*>(raw);
  const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
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
  const T* q = static_cast<const T*>(p.q) + (long long)b * p.L * p.ldq + (long long)gh * p.K;
  const T* k = static_cast<const T*>(p.k) + (long long)b * p.L * p.ldk + (long long)gh * p.K;
  const T* v = static_cast<const T*>(p.v) + (long long)b * p.L * p.ldv + (long long)h * p.V + v0;

  // the state this segment starts from: what the segments before composed, or h0, or zero
  float S[RK][4];
  zero_acc(S);
  if (s0 != nullptr && !SUM) {
    const float* src = s0 + (p.nseg > 1 ? bh * p.nseg + seg : bh) * p.K * p.V;
#pragma unroll
    for (int r = 0; r < RK; ++r)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int kk = ty * RK + r, vv = tx + 16 * c;
        if (kk < p.K && vv < vw) S[r][c] = src[(long long)kk * p.V + v0 + vv];
      }
  }
  double total = 0.0;
  const int c0 = seg * p.cps, c1 = c0 + p.cps < p.nck ? c0 + p.cps : p.nck;
  for (int ck = c0; ck < c1; ++ck) {
    const int t0 = ck * C;
    const int rows = p.L - t0 < C ? p.L - t0 : C;
    const int valid = len - t0 < 0 ? 0 : len - t0 < C ? len - t0 : C;
    if (valid == 0) {  // past the row's end: nothing decays, adds or reads
      if (!SUM)
        for (int i = tid; i < rows * vw; i += 256)
          ActT<T>::st1(o + (((long long)b * p.L + t0 + i / vw) * p.H + h) * p.V + v0 + i % vw, 0.f);
      continue;
    }
    if (tid < 32) chunk_decays<C>(p, b, h, t0, len, tid, sm.chi, sm.clo);
    if (!SUM) load_tile<T, C, KP, LK>(q + t0 * p.ldq, p.ldq, valid, p.K, sm.q, tid);
    load_tile<T, C, KP, LK>(k + t0 * p.ldk, p.ldk, valid, p.K, sm.k, tid);
    load_tile<T, C, kVT, LV>(v + t0 * p.ldv, p.ldv, valid, vw, sm.v, tid);
    if (!SUM) {
#pragma unroll
      for (int r = 0; r < RK; ++r)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int kk = ty * RK + r, vv = tx + 16 * c;
          sm.s[kk * LV + vv] = S[r][c];
          if (ckpt != nullptr && kk < p.K && vv < vw) ckpt[((bh * p.nck + ck) * p.K + kk) * p.V + v0 + vv] = S[r][c];
        }
    }
    __syncthreads();
    if (!SUM) {
      float a[4][4];
      zero_acc(a);
      mm<C, C, KP, false, true, LK, LK>(sm.q, sm.k, a, tid);
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int i = ty * 4 + r, j = tx + 16 * c;
          sm.p[i * LC + j] = j <= i ? a[r][c] * dec_diff(sm.chi[i], sm.clo[i], sm.chi[j], sm.clo[j]) : 0.f;
        }
      zero_acc(a);
      mm<C, kVT, KP, false, false, LK, LV>(sm.q, sm.s, a, tid);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float e = dec_exp(sm.chi[ty * 4 + r], sm.clo[ty * 4 + r]);
#pragma unroll
        for (int c = 0; c < 4; ++c) a[r][c] *= e;
      }
      __syncthreads();
      mm<C, kVT, C, false, false, LC, LV>(sm.p, sm.v, a, tid);
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int i = ty * 4 + r, vv = tx + 16 * c;
          if (i < rows && vv < vw)
            ActT<T>::st1(o + (((long long)b * p.L + t0 + i) * p.H + h) * p.V + v0 + vv, i < valid ? p.scale * a[r][c] : 0.f);
        }
    }
    __syncthreads();
    const float chi = sm.chi[C - 1], clo = sm.clo[C - 1];
    total += (double)chi + (double)clo;
    for (int i = tid; i < C * KP; i += 256) {  // k_j e^{c_last - c_j}
      const int j = i / KP;
      sm.k[j * LK + i % KP] *= dec_diff(chi, clo, sm.chi[j], sm.clo[j]);
    }
    const float e = dec_exp(chi, clo);
#pragma unroll
    for (int r = 0; r < RK; ++r)
#pragma unroll
      for (int c = 0; c < 4; ++c) S[r][c] *= e;
    __syncthreads();
    mm<KP, kVT, C, true, false, LK, LV>(sm.k, sm.v, S, tid);
    __syncthreads();
  }
  float* dst = nullptr;
  if (SUM) dst = send + (bh * p.nseg + seg) * p.K * p.V;
  else if (send != nullptr && seg == p.nseg - 1) dst = send + bh * p.K * p.V;
  if (dst != nullptr) {
#pragma unroll
    for (int r = 0; r < RK; ++r)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int kk = ty * RK + r, vv = tx + 16 * c;
        if (kk < p.K && vv < vw) dst[(long long)kk * p.V + v0 + vv] = S[r][c];
      }
  }
  if (SUM && tid == 0 && vt == 0) sdec[bh * p.nseg + seg] = total;
}

// In place over the segments of a (batch row, head): the end states found from
// zero become the states entering the segments, S[s+1] = 2^{dec[s]} S[s] + end[s].
__global__ void __launch_bounds__(256) linattn_fwd_join_kernel(const float* __restrict__ h0, float* __restrict__ st,
                                                               const double* __restrict__ dec, long long kv, int nseg) {
  const long long bh = blockIdx.y;
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  if (i >= kv) return;
  float s = h0 != nullptr ? h0[bh * kv + i] : 0.f;
  for (int n = 0; n < nseg; ++n) {
    float* at = st + (bh * nseg + n) * kv + i;
    const Dec d = dec_of(dec[bh * nseg + n]);
    const float end = *at;
    *at = s;
    s = fmaf(dec_exp(d.hi, d.lo), s, end);
  }
}

struct FwdPlan {
  LinAttn p;
  size_t states, bytes;
};

int fwd_plan(int B, int L, int H, int G, int K, int V, int dtype, FwdPlan& pl) {
  const int rc = linattn_validate(B, L, H, G, K, V, dtype);
  if (rc != SS_OK) return rc;
  pl.p = LinAttn{};
  pl.p.B = B; pl.p.L = L; pl.p.H = H; pl.p.G = G; pl.p.K = K; pl.p.V = V;
  const long long walks = (long long)B * H * ((V + kVT - 1) / kVT);
  if (walks > (1ll << 24)) return SS_ERR_DIM;
  linattn_segments(pl.p, linattn_chunk(dtype), walks, (K > 64 ? 1 : 2) * 152);
  pl.states = pl.p.nseg > 1 ? (size_t)B * H * pl.p.nseg * K * V * sizeof(float) : 0;
  pl.bytes = pl.p.nseg > 1 ? pl.states + (size_t)B * H * pl.p.nseg * sizeof(double) : 0;
  return SS_OK;
}

template <typename T, int KP>
int fwd_launch(const FwdPlan& pl, const float* h0, void* o, float* ckpt, float* h_last, void* ws, cudaStream_t s) {
  const LinAttn& p = pl.p;
  const size_t smem = sizeof(FwdSmem<KP>);
  auto run = [&](auto kern, const float* s0, float* send, double* dec) -> int {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess) return SS_ERR_CUDA;
    const long long grid = (long long)p.B * p.H * ((p.V + kVT - 1) / kVT) * p.nseg;
    kern<<<(unsigned)grid, 256, smem, s>>>(p, s0, static_cast<T*>(o), ckpt, send, dec);
    return cudaGetLastError() == cudaSuccess ? SS_OK : SS_ERR_CUDA;
  };
  if (p.nseg == 1) return run(linattn_fwd_kernel<T, KP, false>, h0, h_last, nullptr);
  float* st = static_cast<float*>(ws);
  double* dec = reinterpret_cast<double*>(static_cast<char*>(ws) + pl.states);
  int rc = run(linattn_fwd_kernel<T, KP, true>, nullptr, st, dec);
  if (rc != SS_OK) return rc;
  const long long kv = (long long)p.K * p.V;
  linattn_fwd_join_kernel<<<dim3((unsigned)((kv + 255) / 256), (unsigned)(p.B * p.H)), 256, 0, s>>>(h0, st, dec, kv, p.nseg);
  if (cudaGetLastError() != cudaSuccess) return SS_ERR_CUDA;
  return run(linattn_fwd_kernel<T, KP, false>, st, h_last, nullptr);
}

}  // namespace

extern "C" int linattn_num_chunks(int L, int dtype) {
  if (L <= 0 || (dtype != SS_F32 && dtype != SS_BF16)) return 0;
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
  if ((rc = linattn_ld_ok(ldq, G * K)) != SS_OK || (rc = linattn_ld_ok(ldk, G * K)) != SS_OK ||
      (rc = linattn_ld_ok(ldv, H * V)) != SS_OK)
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
  if (dtype == SS_F32)
    return K <= 64 ? fwd_launch<float, 64>(pl, h0, o, ckpt, h_last, workspace, s)
                   : fwd_launch<float, 128>(pl, h0, o, ckpt, h_last, workspace, s);
  return K <= 64 ? fwd_launch<__nv_bfloat16, 64>(pl, h0, o, ckpt, h_last, workspace, s)
                 : fwd_launch<__nv_bfloat16, 128>(pl, h0, o, ckpt, h_last, workspace, s);
}
