// One step of linear attention with a decay for each head (linattn_step), decode:
//   h <- e^{g} h + k v^T,   o = scale * h^T q           per (batch row, head), h in place
//
// All the time goes to reading and writing h ([K, V] fp32).  A CTA takes 16
// columns of one head: thread (ty, tx) owns the four columns 4 tx of the rows
// ty, ty + 64, ... as 16-byte vectors, and the sum over rows for o is a shared-memory tree.
#include "linattn_common.cuh"

namespace {

using namespace ssk;

template <typename T>
__global__ void __launch_bounds__(256) linattn_step_kernel(const T* __restrict__ q, const T* __restrict__ k, const T* __restrict__ v,
                                                           const float* __restrict__ g, int g_head, float* __restrict__ st,
                                                           T* __restrict__ o, int H, int G, int K, int V, float scale) {
  __shared__ float4 red[8][4];
  const int tid = threadIdx.x, ty = tid >> 2, tx = tid & 3;
  const long long bh = blockIdx.x;
  const long long b = bh / H;
  const int h = (int)(bh % H), gh = h / (H / G);
  const int c = (int)blockIdx.y * 16 + 4 * tx;
  const bool ok = c < V;
  float gv = g[g_head ? h : bh];
  const float e = expf(gv);
  const T* qr = q + (b * G + gh) * K;
  const T* kr = k + (b * G + gh) * K;
  float4 x[2];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int r = ty + 64 * u;
    x[u] = ok && r < K ? *reinterpret_cast<const float4*>(st + (bh * K + r) * V + c) : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  float vv[4] = {0.f, 0.f, 0.f, 0.f};
  if (ok) ActT<T>::ld4(v + bh * V + c, vv);
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int r = ty + 64 * u;
    if (!ok || r >= K) continue;
    const float kk = ActT<T>::ld(kr + r), qq = ActT<T>::ld(qr + r);
    x[u].x = fmaf(e, x[u].x, kk * vv[0]);
    x[u].y = fmaf(e, x[u].y, kk * vv[1]);
    x[u].z = fmaf(e, x[u].z, kk * vv[2]);
    x[u].w = fmaf(e, x[u].w, kk * vv[3]);
    *reinterpret_cast<float4*>(st + (bh * K + r) * V + c) = x[u];
    a.x = fmaf(qq, x[u].x, a.x);
    a.y = fmaf(qq, x[u].y, a.y);
    a.z = fmaf(qq, x[u].z, a.z);
    a.w = fmaf(qq, x[u].w, a.w);
  }
#pragma unroll
  for (int s = 4; s < 32; s <<= 1) {
    a.x += __shfl_xor_sync(0xffffffffu, a.x, s);
    a.y += __shfl_xor_sync(0xffffffffu, a.y, s);
    a.z += __shfl_xor_sync(0xffffffffu, a.z, s);
    a.w += __shfl_xor_sync(0xffffffffu, a.w, s);
  }
  if ((tid & 31) < 4) red[tid >> 5][tx] = a;
  __syncthreads();
  if (tid < 4 && ok) {
    float4 s = red[0][tx];
#pragma unroll
    for (int w = 1; w < 8; ++w) {
      const float4 y = red[w][tx];
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
  const dim3 grid((unsigned)(B * H), (unsigned)((V + 15) / 16));
  if (dtype == SS_F32)
    linattn_step_kernel<float><<<grid, 256, 0, s>>>(static_cast<const float*>(q), static_cast<const float*>(k),
                                                    static_cast<const float*>(v), g, g_per_head, h, static_cast<float*>(o), H, G, K, V, scale);
  else
    linattn_step_kernel<__nv_bfloat16><<<grid, 256, 0, s>>>(
        static_cast<const __nv_bfloat16*>(q), static_cast<const __nv_bfloat16*>(k), static_cast<const __nv_bfloat16*>(v), g, g_per_head,
        h, static_cast<__nv_bfloat16*>(o), H, G, K, V, scale);
  return cudaGetLastError() == cudaSuccess ? SS_OK : SS_ERR_CUDA;
}
