// One step of the gated delta rule (deltarule_step), decode:
//   h <- e^{g} h,   r = v - h^T k,   h <- h + beta k r^T,   o = scale * h^T q        per (batch row, head), h in place
//
// All the time goes to reading and writing h ([K, V] fp32), once each: a CTA takes `cw` columns of one head and holds them in
// registers (a thread owns four neighbouring columns of every RP-th row, at most ROWS of them).  Both products over K are taken of
// the decayed state at once, since o = scale * (h^T q + (k.q) beta r); each thread leaves its rows' sums in shared memory,
// and they are added in order.  bf16, 96 sequences of 32 heads of 128 x 128 (8 of q, k): 66 us, 6.2 TB/s; one sequence 4.5 us.
#include "linattn_common.cuh"

namespace {

using namespace ssk;

constexpr int NT = 256;

template <typename T, int ROWS>
__global__ void __launch_bounds__(NT, 4) delta_step_kernel(const T* __restrict__ q, const T* __restrict__ k, const T* __restrict__ v,
                                                           const float* __restrict__ g, const float* __restrict__ beta,
                                                           float* __restrict__ st, T* __restrict__ o, int H, int G, int K, int V, int cw,
                                                           float scale) {
  __shared__ float2 kq[kLinMaxHead];
  __shared__ float4 red[2][NT];
  __shared__ float dots[4];
  const int tid = threadIdx.x;
  const long long bh = blockIdx.x, b = bh / H;
  const int h = (int)(bh % H), gh = h / (H / G);
  const int c0 = (int)blockIdx.y * cw, n4 = (V - c0 < cw ? V - c0 : cw) / 4;  // this CTA's groups of four columns
  const int RP = NT / n4, c = c0 + tid % n4 * 4, r0 = tid / n4;
  const bool on = r0 < RP;
  float4* at = reinterpret_cast<float4*>(st + (bh * K + r0) * V + c);
  const long long step = (long long)RP * V / 4;
  float4 x[ROWS];
#pragma unroll
  for (int u = 0; u < ROWS; ++u) x[u] = on && r0 + u * RP < K ? __ldcs(at + u * step) : make_float4(0.f, 0.f, 0.f, 0.f);
  if (tid < kLinMaxHead) {  // k.q of the token, in four warps
    float2 y = make_float2(0.f, 0.f);
    if (tid < K) y = make_float2(ActT<T>::ld(k + (b * G + gh) * K + tid), ActT<T>::ld(q + (b * G + gh) * K + tid));
    kq[tid] = y;
    float d = y.x * y.y;
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) d += __shfl_xor_sync(0xffffffffu, d, s);
    if ((tid & 31) == 0) dots[tid >> 5] = d;
  }
  const float e = g != nullptr ? expf(g[bh]) : 1.f, be = beta[bh];
  float vv[4] = {0.f, 0.f, 0.f, 0.f};
  if (on) ActT<T>::ld4(v + bh * V + c, vv);
  __syncthreads();
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f), d = a;
#pragma unroll
  for (int u = 0; u < ROWS; ++u) {
    if (r0 + u * RP >= K) continue;
    const float2 y = kq[r0 + u * RP];
    x[u].x *= e; x[u].y *= e; x[u].z *= e; x[u].w *= e;
    a.x = fmaf(y.x, x[u].x, a.x); a.y = fmaf(y.x, x[u].y, a.y); a.z = fmaf(y.x, x[u].z, a.z); a.w = fmaf(y.x, x[u].w, a.w);
    d.x = fmaf(y.y, x[u].x, d.x); d.y = fmaf(y.y, x[u].y, d.y); d.z = fmaf(y.y, x[u].z, d.z); d.w = fmaf(y.y, x[u].w, d.w);
  }
  red[0][tid] = a;
  red[1][tid] = d;
  __syncthreads();
  if (tid < 2 * n4) {  // the rows' parts in order
    float4* part = red[tid >= n4] + (tid >= n4 ? tid - n4 : tid);
    float4 s = part[0];
    for (int w = 1; w < RP; ++w) {
      const float4 y = part[w * n4];
      s.x += y.x; s.y += y.y; s.z += y.z; s.w += y.w;
    }
    part[0] = s;  // (no one else reads this column's parts)
  }
  __syncthreads();
  if (!on) return;
  a = red[0][tid % n4];
  const float u0 = be * (vv[0] - a.x), u1 = be * (vv[1] - a.y), u2 = be * (vv[2] - a.z), u3 = be * (vv[3] - a.w);
#pragma unroll
  for (int u = 0; u < ROWS; ++u) {
    if (r0 + u * RP >= K) continue;
    const float kk = kq[r0 + u * RP].x;
    x[u].x = fmaf(kk, u0, x[u].x); x[u].y = fmaf(kk, u1, x[u].y); x[u].z = fmaf(kk, u2, x[u].z); x[u].w = fmaf(kk, u3, x[u].w);
    __stcs(at + u * step, x[u]);
  }
  if (r0 == 0) {
    d = red[1][tid];
    const float w = (dots[0] + dots[1]) + (dots[2] + dots[3]);
    ActT<T>::st2(o + bh * V + c, scale * fmaf(w, u0, d.x), scale * fmaf(w, u1, d.y));
    ActT<T>::st2(o + bh * V + c + 2, scale * fmaf(w, u2, d.z), scale * fmaf(w, u3, d.w));
  }
}

template <typename T>
int launch(const void* q, const void* k, const void* v, const float* g, const float* beta, float* h, void* o, int B, int H, int G, int K, int V,
           float scale, cudaStream_t s) {
  // 64 columns of 128 rows a CTA where there are many heads (of 128 x 128: 1024 24.1 us, 96 times 32 65.9; with 32 columns 24.7 and
  // 71.5), 32 where there are few (32 heads 4.5 us, 320 10.8; with 64 columns 5.1 and 11.0)
  const bool many = (long long)B * H >= 512;
  const int cw = many ? 64 : 32;
  const dim3 grid((unsigned)(B * H), (unsigned)((V + cw - 1) / cw));
  const auto kernel = many ? delta_step_kernel<T, 8> : delta_step_kernel<T, 4>;
  kernel<<<grid, NT, 0, s>>>(static_cast<const T*>(q), static_cast<const T*>(k), static_cast<const T*>(v), g, beta, h, static_cast<T*>(o), H, G, K, V,
                             cw, scale);
  return cudaGetLastError() == cudaSuccess ? SS_OK : SS_ERR_CUDA;
}

}  // namespace

extern "C" int deltarule_step(const void* q, const void* k, const void* v, const float* g, const float* beta, float* h, void* o, int B, int H, int G,
                              int K, int V, float scale, int dtype, void* stream) {
  if (!q || !k || !v || !beta || !h || !o) return SS_ERR_NULL;
  const int rc = linattn_validate(B, 1, H, G, K, V, dtype);
  if (rc != SS_OK) return rc;
  if ((long long)B * H > 2147483647ll) return SS_ERR_DIM;
  const void* ptrs[] = {q, k, v, h, o};
  for (const void* x : ptrs)
    if (!ssh::aligned16(x)) return SS_ERR_ALIGN;
  if ((reinterpret_cast<uintptr_t>(g) & 3u) || (reinterpret_cast<uintptr_t>(beta) & 3u)) return SS_ERR_ALIGN;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return dtype == SS_F32 ? launch<float>(q, k, v, g, beta, h, o, B, H, G, K, V, scale, s)
                         : launch<__nv_bfloat16>(q, k, v, g, beta, h, o, B, H, G, K, V, scale, s);
}
