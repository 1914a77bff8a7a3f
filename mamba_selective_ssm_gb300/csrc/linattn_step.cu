// One step of linear attention with a decay for each head (linattn_step), decode:
//   h <- e^{g} h + k v^T,   o = scale * h^T q           per (batch row, head), h in place
//
// All the time goes to reading and writing h ([K, V] fp32).  A CTA takes `cw`
// columns of one head: a thread owns four neighbouring columns of every RP-th
// row, so that a warp's 16-byte vectors follow one another in memory, up to eight
// rows of a thread in flight.  For o each thread leaves its rows' sum in shared
// memory, and one thread for each group of columns adds the RP of them in order
// (8 at V = 128, 128 at V = 8).
// All of V in one CTA when there is a head for every SM (96 sequences of 32 heads of
// 128 x 128: 62 us, 6.5 TB/s, and 82 with 32 columns a CTA; 8 sequences 6.2 and
// 9.7), 32 columns for fewer, whose latency is the number of loads one after
// another (one sequence 4.2 us, and 6.2 with all of V).  The rule was measured at V =
// 128.  Narrower states, 96 sequences of 32 heads: V = 64 31 us for 30 of copying
// their bytes, V = 24 21 for 11, V = 8 21 for 4: there the CTAs count, not the bytes.
#include "linattn_common.cuh"

namespace {

using namespace ssk;

constexpr int kLinStepThreads = 256;

template <typename T>
__global__ void __launch_bounds__(kLinStepThreads) linattn_step_kernel(const T* __restrict__ q, const T* __restrict__ k,
                                                                       const T* __restrict__ v, const float* __restrict__ g, int g_head,
                                                                       float* __restrict__ st, T* __restrict__ o, int H, int G, int K,
                                                                       int V, int cw, float scale) {
  __shared__ float2 kq[kLinMaxHead];
  __shared__ float4 red[kLinStepThreads];
  const int tid = threadIdx.x;
  const long long bh = blockIdx.x;
  const long long b = bh / H;
  const int h = (int)(bh % H), gh = h / (H / G);
  const int c0 = (int)blockIdx.y * cw, n4 = (V - c0 < cw ? V - c0 : cw) / 4;  // this CTA's groups of four columns
  const int RP = kLinStepThreads / n4, c = c0 + tid % n4 * 4, r0 = tid / n4;
  const bool on = r0 < RP;
  float4* at = reinterpret_cast<float4*>(st + (bh * K + r0) * V + c);
  const long long step = (long long)RP * V / 4;
  const float e = expf(g[g_head ? h : bh]);
  if (tid < K) kq[tid] = make_float2(ActT<T>::ld(k + (b * G + gh) * K + tid), ActT<T>::ld(q + (b * G + gh) * K + tid));
  float vv[4] = {0.f, 0.f, 0.f, 0.f};
  if (on) ActT<T>::ld4(v + bh * V + c, vv);
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
  constexpr int U = 8;
  bool first = true;
  for (int r = r0; r < K || first; r += U * RP) {  // (every thread passes the barrier)
    float4 x[U];
#pragma unroll
    for (int u = 0; u < U; ++u) x[u] = on && r + u * RP < K ? __ldcs(at + u * step) : make_float4(0.f, 0.f, 0.f, 0.f);
    if (first) __syncthreads();  // k, q
    first = false;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (!on || r + u * RP >= K) continue;
      const float2 kk = kq[r + u * RP];
      x[u].x = fmaf(e, x[u].x, kk.x * vv[0]);
      x[u].y = fmaf(e, x[u].y, kk.x * vv[1]);
      x[u].z = fmaf(e, x[u].z, kk.x * vv[2]);
      x[u].w = fmaf(e, x[u].w, kk.x * vv[3]);
      __stcs(at + u * step, x[u]);
      a.x = fmaf(kk.y, x[u].x, a.x);
      a.y = fmaf(kk.y, x[u].y, a.y);
      a.z = fmaf(kk.y, x[u].z, a.z);
      a.w = fmaf(kk.y, x[u].w, a.w);
    }
    at += U * step;
  }
  red[tid] = a;
  __syncthreads();
  if (tid < n4) {  // the rows' parts in order
    float4 s = red[tid];
    for (int w = 1; w < RP; ++w) {
      const float4 y = red[w * n4 + tid];
      s.x += y.x; s.y += y.y; s.z += y.z; s.w += y.w;
    }
    ActT<T>::st2(o + bh * V + c, scale * s.x, scale * s.y);
    ActT<T>::st2(o + bh * V + c + 2, scale * s.z, scale * s.w);
  }
}

}  // namespace

extern "C" int linattn_step(const void* q, const void* k, const void* v, const float* g, int g_per_head, float* h, void* o, int B,
                            int H, int G, int K, int V, float scale, int dtype, void* stream) {
  if (!q || !k || !v || !g || !h || !o) return SS_ERR_NULL;
  const int rc = linattn_validate(B, 1, H, G, K, V, dtype);
  if (rc != SS_OK) return rc;
  if ((long long)B * H > 2147483647ll) return SS_ERR_DIM;
  const void* ptrs[] = {q, k, v, h, o};
  for (const void* x : ptrs)
    if (!ssh::aligned16(x)) return SS_ERR_ALIGN;
  if (reinterpret_cast<uintptr_t>(g) & 3u) return SS_ERR_ALIGN;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int cw = B * H >= 152 ? V : 32;
  const dim3 grid((unsigned)(B * H), (unsigned)((V + cw - 1) / cw));
  if (dtype == SS_F32)
    linattn_step_kernel<float><<<grid, kLinStepThreads, 0, s>>>(static_cast<const float*>(q), static_cast<const float*>(k),
                                                    static_cast<const float*>(v), g, g_per_head, h, static_cast<float*>(o), H, G, K, V, cw, scale);
  else
    linattn_step_kernel<__nv_bfloat16><<<grid, kLinStepThreads, 0, s>>>(
        static_cast<const __nv_bfloat16*>(q), static_cast<const __nv_bfloat16*>(k), static_cast<const __nv_bfloat16*>(v), g, g_per_head,
        h, static_cast<__nv_bfloat16*>(o), H, G, K, V, cw, scale);
  return cudaGetLastError() == cudaSuccess ? SS_OK : SS_ERR_CUDA;
}
