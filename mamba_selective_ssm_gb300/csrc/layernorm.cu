// Layer norm forward and backward (layernorm_fwd, layernorm_bwd) for sm_103a.
//
//   mean_r = mean_i x,  rstd_r = 1 / sqrt(mean_i (x - mean_r)^2 + eps),  xh = (x - mean_r) rstd_r
//   y = xh scale + bias
//   w = dy scale;  dx = rstd_r (w - mean_i w - xh mean_i(w xh));  dscale += sum_r dy xh;  dbias += sum_r dy
//
// Both are one pass over memory: a row is held in registers (as loaded, 8
// columns a lane and group) between the sums and the output, so the variance is
// taken around the mean that was found, not as a difference of moments.
//   rows of <= 256 columns    G lanes per row, 32/G rows per warp, U row sets in flight (131072 rows of 256 in bf16:
//                             forward 32 us, backward 50; as wider rows 38 and 59)
//   rows of <= 4096 bytes     forward: one warp per row (16384 rows of 2048 in bf16: 27 us, as wider rows 29; in fp32
//                             51 and 48)
//   wider rows                and the backward's above 256: a CTA's threads share the columns, one row per step
//                             (backward with a warp per row: 16384 rows of 1024 in bf16 55 us for 33).  Its column sums
//                             fit the registers up to 8192 columns (4096 rows of 8192: bf16 70 us, fp32 85); above, they
//                             spill (4096 rows of 16384: 527 and 300)
// The backward's column sums stay in registers over all the rows a thread
// visits; the CTAs' partial rows are added in fixed order by colsum_kernel.
// 1 / sqrt is rsqrtf (2 units in the last place):
// 262144 rows of 128 take 30 us with it, 32 with a square root and a division.
#include <type_traits>

#include "common.cuh"

namespace {

using namespace ssk;

constexpr int kLnMaxDim = 32768;

__device__ __forceinline__ void ld8f(const float* p, bool ok, float* o) {
  const float4 a = ok ? __ldg(reinterpret_cast<const float4*>(p)) : make_float4(0.f, 0.f, 0.f, 0.f);
  const float4 b = ok ? __ldg(reinterpret_cast<const float4*>(p + 4)) : make_float4(0.f, 0.f, 0.f, 0.f);
  o[0] = a.x; o[1] = a.y; o[2] = a.z; o[3] = a.w; o[4] = b.x; o[5] = b.y; o[6] = b.z; o[7] = b.w;
}

template <int G>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
  for (int o = 1; o < G; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// ---------------------------------------------------------------- forward

template <typename T, int G, int U>
__global__ void __launch_bounds__(256) ln_fwd_small_kernel(const T* __restrict__ x, const float* __restrict__ scale,
                                                           const float* __restrict__ bias, float eps, T* __restrict__ y,
                                                           float* __restrict__ mean, float* __restrict__ rstd, int rows, int dim) {
  using R = Raw8<T>;
  constexpr int RW = 32 / G;  // rows of a warp's set
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, slot = lane / G, c = (lane % G) * 8;
  const bool cv = c < dim;
  float sc[8], bi[8];
  ld8f(scale + c, cv, sc);
  ld8f(bias + c, cv && bias != nullptr, bi);
  const float inv_dim = 1.0f / (float)dim;
  const long long step = (long long)gridDim.x * 8 * RW * U;
  for (long long r0 = ((long long)blockIdx.x * 8 + warp) * RW * U; r0 < rows; r0 += step) {
    typename R::V raw[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const long long r = r0 + u * RW + slot;
      raw[u] = cv && r < rows ? R::ld(x + r * dim + c) : R::zero();
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const long long r = r0 + u * RW + slot;
      float v[8], s = 0.f;
      R::wide(raw[u], v);
#pragma unroll
      for (int e = 0; e < 8; ++e) s += v[e];
      const float m = lanes_sum<G>(s) * inv_dim;
      s = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        v[e] -= m;
        s = fmaf(v[e], v[e], s);
      }
      if (!cv) s = 0.f;
      const float rs = rsqrtf(fmaf(lanes_sum<G>(s), inv_dim, eps));
      if (r < rows) {
        if (c == 0) {
          if (mean != nullptr) mean[r] = m;
          if (rstd != nullptr) rstd[r] = rs;
        }
        if (cv) {
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = fmaf(v[e] * rs, sc[e], bi[e]);
          ActT<T>::st8(y + r * dim + c, v);
        }
      }
    }
  }
}

// One warp per row; lane l owns the 8-column groups l, l + 32, ... (VPW of
// them).  scale and bias wait in shared memory, split so that a warp's reads
// follow one another.
template <typename T, int VPW>
__global__ void __launch_bounds__(256) ln_fwd_warp_kernel(const T* __restrict__ x, const float* __restrict__ scale,
                                                          const float* __restrict__ bias, float eps, T* __restrict__ y,
                                                          float* __restrict__ mean, float* __restrict__ rstd, int rows, int dim) {
  using R = Raw8<T>;
  extern __shared__ float4 par[];  // [scale first 4 | scale last 4 | bias first 4 | bias last 4][dim / 8]
  const int ng = dim / 8;
  for (int i = threadIdx.x; i < ng; i += blockDim.x) {
    par[i] = __ldg(reinterpret_cast<const float4*>(scale) + 2 * i);
    par[ng + i] = __ldg(reinterpret_cast<const float4*>(scale) + 2 * i + 1);
    par[2 * ng + i] = bias ? __ldg(reinterpret_cast<const float4*>(bias) + 2 * i) : make_float4(0.f, 0.f, 0.f, 0.f);
    par[3 * ng + i] = bias ? __ldg(reinterpret_cast<const float4*>(bias) + 2 * i + 1) : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  __syncthreads();
  const int lane = threadIdx.x & 31;
  const float inv_dim = 1.0f / (float)dim;
  const long long step = (long long)gridDim.x * 8;
  for (long long r = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); r < rows; r += step) {
    typename R::V raw[VPW];
#pragma unroll
    for (int u = 0; u < VPW; ++u) {
      const int gi = u * 32 + lane;
      raw[u] = gi < ng ? R::ld(x + (size_t)r * dim + gi * 8) : R::zero();
    }
    float s = 0.f;
#pragma unroll
    for (int u = 0; u < VPW; ++u) {
      float v[8];
      R::wide(raw[u], v);
#pragma unroll
      for (int e = 0; e < 8; ++e) s += v[e];
    }
    const float m = lanes_sum<32>(s) * inv_dim;
    s = 0.f;
#pragma unroll
    for (int u = 0; u < VPW; ++u) {
      float v[8], t = 0.f;
      R::wide(raw[u], v);
#pragma unroll
      for (int e = 0; e < 8; ++e) t = fmaf(v[e] - m, v[e] - m, t);
      if (u * 32 + lane < ng) s += t;
    }
    const float rs = rsqrtf(fmaf(lanes_sum<32>(s), inv_dim, eps));
    if (lane == 0) {
      if (mean != nullptr) mean[r] = m;
      if (rstd != nullptr) rstd[r] = rs;
    }
#pragma unroll
    for (int u = 0; u < VPW; ++u) {
      const int gi = u * 32 + lane;
      if (gi < ng) {
        float v[8];
        R::wide(raw[u], v);
        const float4 s0 = par[gi], s1 = par[ng + gi], b0 = par[2 * ng + gi], b1 = par[3 * ng + gi];
        const float sc[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
        const float bi[8] = {b0.x, b0.y, b0.z, b0.w, b1.x, b1.y, b1.z, b1.w};
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = fmaf((v[e] - m) * rs, sc[e], bi[e]);
        ActT<T>::st8(y + (size_t)r * dim + gi * 8, v);
      }
    }
  }
}

// Sum over the CTA of two values at once; buffers alternate with `par`.
__device__ __forceinline__ float2 cta_sum2(float2 v, float2 (*red)[32], int par) {
  const int lane = threadIdx.x & 31, nw = (blockDim.x + 31) >> 5;
  v.x = lanes_sum<32>(v.x);
  v.y = lanes_sum<32>(v.y);
  if (lane == 0) red[par][threadIdx.x >> 5] = v;
  __syncthreads();
  const float2 w = lane < nw ? red[par][lane] : make_float2(0.f, 0.f);
  return make_float2(lanes_sum<32>(w.x), lanes_sum<32>(w.y));
}

// A CTA's threads share a row, the next one in flight.  Two column groups a thread
// halve the warps that meet at the two barriers (8192 rows of 4096 in bf16: one
// group 37 us, two 34; without the next row 39).  HOLD: at most 512 threads, whose
// registers hold scale and bias too; in bf16, where these are four times a row's
// bytes, 30 us, in fp32 52 for 49.
template <typename T, int VPT, bool HOLD>
__global__ void __launch_bounds__(HOLD ? 512 : 1024) ln_fwd_wide_kernel(const T* __restrict__ x, const float* __restrict__ scale,
                                                           const float* __restrict__ bias, float eps, T* __restrict__ y,
                                                           float* __restrict__ mean, float* __restrict__ rstd, int rows, int dim) {
  using R = Raw8<T>;
  __shared__ float2 red[2][32];
  const float inv_dim = 1.0f / (float)dim;
  typename R::V raw[VPT], next[VPT];
  auto load = [&](typename R::V(&v)[VPT], long long r) {
#pragma unroll
    for (int u = 0; u < VPT; ++u) {
      const int c = (u * (int)blockDim.x + (int)threadIdx.x) * 8;
      v[u] = c < dim && r < rows ? R::ld(x + (size_t)r * dim + c) : R::zero();
    }
  };
  float sc[HOLD ? VPT : 1][8], bi[HOLD ? VPT : 1][8];
  auto params = [&](int c, float(&ps)[8], float(&pb)[8]) {
    ld8f(scale + c, c < dim, ps);
    ld8f(bias + c, c < dim && bias != nullptr, pb);
  };
  if constexpr (HOLD) {
#pragma unroll
    for (int u = 0; u < VPT; ++u) params((u * (int)blockDim.x + (int)threadIdx.x) * 8, sc[u], bi[u]);
  }
  load(raw, blockIdx.x);
  for (long long r = blockIdx.x; r < rows; r += gridDim.x) {
    load(next, r + gridDim.x);  // in flight during this row's sums
    float s = 0.f;
#pragma unroll
    for (int u = 0; u < VPT; ++u) {
      float v[8];
      R::wide(raw[u], v);
#pragma unroll
      for (int e = 0; e < 8; ++e) s += v[e];
    }
    const float m = cta_sum2(make_float2(s, 0.f), red, 0).x * inv_dim;
    s = 0.f;
#pragma unroll
    for (int u = 0; u < VPT; ++u) {
      const int c = (u * (int)blockDim.x + (int)threadIdx.x) * 8;
      float v[8], t = 0.f;
      R::wide(raw[u], v);
#pragma unroll
      for (int e = 0; e < 8; ++e) t = fmaf(v[e] - m, v[e] - m, t);
      if (c < dim) s += t;
    }
    const float rs = rsqrtf(fmaf(cta_sum2(make_float2(s, 0.f), red, 1).x, inv_dim, eps));
    if (threadIdx.x == 0) {
      if (mean != nullptr) mean[r] = m;
      if (rstd != nullptr) rstd[r] = rs;
    }
#pragma unroll
    for (int u = 0; u < VPT; ++u) {
      const int c = (u * (int)blockDim.x + (int)threadIdx.x) * 8;
      if (c < dim) {
        float v[8];
        R::wide(raw[u], v);
        constexpr int hold = HOLD ? 1 : 0;
        if (!HOLD) params(c, sc[0], bi[0]);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = fmaf((v[e] - m) * rs, sc[u * hold][e], bi[u * hold][e]);
        ActT<T>::st8(y + (size_t)r * dim + c, v);
      }
      raw[u] = next[u];
    }
  }
}

// ---------------------------------------------------------------- backward

template <typename T, int G, int U>
__global__ void __launch_bounds__(256) ln_bwd_small_kernel(const T* __restrict__ dy, const T* __restrict__ x,
                                                           const float* __restrict__ scale, const float* __restrict__ mean,
                                                           const float* __restrict__ rstd, float* __restrict__ dx,
                                                           float* __restrict__ ws, int rows, int dim) {
  pdl_trigger();  // the column sum of the partials may launch now; it waits for this grid's end
  using R = Raw8<T>;
  constexpr int RW = 32 / G;
  __shared__ float red[2][8][G * 8];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, slot = lane / G, c = (lane % G) * 8;
  const bool cv = c < dim;
  float sc[8], as[8], ab[8];
  ld8f(scale + c, cv, sc);
#pragma unroll
  for (int e = 0; e < 8; ++e) as[e] = ab[e] = 0.f;
  const float inv_dim = 1.0f / (float)dim;
  const long long step = (long long)gridDim.x * 8 * RW * U;
  for (long long r0 = ((long long)blockIdx.x * 8 + warp) * RW * U; r0 < rows; r0 += step) {
    typename R::V gr[U], xr[U];
    float ms[U], rs[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const long long r = r0 + u * RW + slot;
      const bool ok = r < rows;
      gr[u] = cv && ok ? R::ld(dy + r * dim + c) : R::zero();
      xr[u] = cv && ok ? R::ld(x + r * dim + c) : R::zero();
      ms[u] = ok ? __ldg(mean + r) : 0.f;
      rs[u] = ok ? __ldg(rstd + r) : 0.f;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const long long r = r0 + u * RW + slot;
      float g[8], v[8], s1 = 0.f, s2 = 0.f;
      R::wide(gr[u], g);
      R::wide(xr[u], v);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        v[e] = (v[e] - ms[u]) * rs[u];
        ab[e] += g[e];
        as[e] = fmaf(g[e], v[e], as[e]);
        g[e] *= sc[e];
        s1 += g[e];
        s2 = fmaf(g[e], v[e], s2);
      }
      s1 = lanes_sum<G>(s1) * inv_dim;
      s2 = lanes_sum<G>(s2) * inv_dim;
      if (cv && r < rows) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = rs[u] * (g[e] - s1 - v[e] * s2);
        ActT<float>::st8(dx + r * dim + c, v);
      }
    }
  }
  // the warp's row slots in lane order, then the warps in order
#pragma unroll
  for (int e = 0; e < 8; ++e) {
#pragma unroll
    for (int o = G; o < 32; o <<= 1) {
      as[e] += __shfl_xor_sync(0xffffffffu, as[e], o);
      ab[e] += __shfl_xor_sync(0xffffffffu, ab[e], o);
    }
    if (slot == 0) {
      red[0][warp][c + e] = as[e];
      red[1][warp][c + e] = ab[e];
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * dim; i += 256) {
    const int which = i >= dim, col = which ? i - dim : i;
    float a = red[which][0][col];
#pragma unroll
    for (int w = 1; w < 8; ++w) a += red[which][w][col];
    ws[(size_t)blockIdx.x * 2 * dim + i] = a;
  }
}

template <typename T, int VPT>
__global__ void __launch_bounds__(1024) ln_bwd_cols_kernel(const T* __restrict__ dy, const T* __restrict__ x,
                                                           const float* __restrict__ scale, const float* __restrict__ mean,
                                                           const float* __restrict__ rstd, float* __restrict__ dx,
                                                           float* __restrict__ ws, int rows, int dim) {
  pdl_trigger();
  using R = Raw8<T>;
  __shared__ float2 red[2][32];
  float as[VPT][8], ab[VPT][8];
#pragma unroll
  for (int u = 0; u < VPT; ++u)
#pragma unroll
    for (int e = 0; e < 8; ++e) as[u][e] = ab[u][e] = 0.f;
  const float inv_dim = 1.0f / (float)dim;
  typename R::V gr[VPT], xr[VPT], gn[VPT], xn[VPT];
  auto load = [&](typename R::V(&g)[VPT], typename R::V(&v)[VPT], long long r) {
#pragma unroll
    for (int u = 0; u < VPT; ++u) {
      const int c = (u * (int)blockDim.x + (int)threadIdx.x) * 8;
      const bool ok = c < dim && r < rows;
      g[u] = ok ? R::ld(dy + (size_t)r * dim + c) : R::zero();
      v[u] = ok ? R::ld(x + (size_t)r * dim + c) : R::zero();
    }
  };
  int par = 0;
  load(gr, xr, blockIdx.x);
  for (long long r = blockIdx.x; r < rows; r += gridDim.x) {
    load(gn, xn, r + gridDim.x);  // the next row in flight during this one's sums
    const float m = __ldg(mean + r), rs = __ldg(rstd + r);
    float2 s = make_float2(0.f, 0.f);
#pragma unroll
    for (int u = 0; u < VPT; ++u) {
      const int c = (u * (int)blockDim.x + (int)threadIdx.x) * 8;
      float g[8], v[8], sc[8];
      R::wide(gr[u], g);
      R::wide(xr[u], v);
      ld8f(scale + c, c < dim, sc);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float xh = (v[e] - m) * rs, w = g[e] * sc[e];
        ab[u][e] += g[e];
        as[u][e] = fmaf(g[e], xh, as[u][e]);
        s.x += w;
        s.y = fmaf(w, xh, s.y);
      }
    }
    s = cta_sum2(s, red, par);
    par ^= 1;
    s.x *= inv_dim;
    s.y *= inv_dim;
#pragma unroll
    for (int u = 0; u < VPT; ++u) {
      const int c = (u * (int)blockDim.x + (int)threadIdx.x) * 8;
      if (c < dim) {
        float g[8], v[8], sc[8];
        R::wide(gr[u], g);
        R::wide(xr[u], v);
        ld8f(scale + c, true, sc);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = rs * (g[e] * sc[e] - s.x - (v[e] - m) * rs * s.y);
        ActT<float>::st8(dx + (size_t)r * dim + c, v);
      }
      gr[u] = gn[u];
      xr[u] = xn[u];
    }
  }
#pragma unroll
  for (int u = 0; u < VPT; ++u) {
    const int c = (u * (int)blockDim.x + (int)threadIdx.x) * 8;
    if (c < dim) {
      ActT<float>::st8(ws + (size_t)blockIdx.x * 2 * dim + c, as[u]);
      ActT<float>::st8(ws + (size_t)blockIdx.x * 2 * dim + dim + c, ab[u]);
    }
  }
}

struct ScaleBiasOut {
  float *dscale, *dbias;
  int dim, add;
  __device__ void put(long long i, float v) const {
    float* out = i < dim ? dscale + i : dbias + (i - dim);
    *out = (add & (i < dim ? 1 : 2)) ? *out + v : v;
  }
};

// ---------------------------------------------------------------- host

int ln_validate(int rows, int dim, int dtype) {
  if (rows <= 0 || dim <= 0) return SS_ERR_DIM;
  if (dtype != SS_F32 && dtype != SS_BF16) return SS_ERR_UNSUPPORTED;
  if (dim % 8 != 0) return SS_ERR_ALIGN;
  if (dim > kLnMaxDim) return SS_ERR_DIM;
  return SS_OK;
}

// row sets in flight per warp of narrow rows (262144 of 128 in bf16: forward 30 us, backward 49; two sets 30 and 61, eight 35 and 68)
constexpr int kLnU = 4;

// lanes per row: the power of two that covers dim / 8 groups
inline int ln_lanes(int dim) {
  int g = 1;
  while (g * 8 < dim) g <<= 1;
  return g;
}

// f(std::integral_constant-like tag) for the lanes of a narrow row
template <typename F>
int ln_narrow(int lanes, F f) {
  switch (lanes) {
    case 1: return f(std::integral_constant<int, 1>());
    case 2: return f(std::integral_constant<int, 2>());
    case 4: return f(std::integral_constant<int, 4>());
    case 8: return f(std::integral_constant<int, 8>());
    case 16: return f(std::integral_constant<int, 16>());
    default: return f(std::integral_constant<int, 32>());
  }
}

// rows of more than 256 columns: 8-column groups per thread and threads of a CTA that share a row
inline int ln_vpt(int dim) { return dim <= 8192 ? 1 : dim <= 16384 ? 2 : 4; }
inline int ln_threads(int dim, int vpt) { return ((dim / 8 + vpt - 1) / vpt + 31) / 32 * 32; }

// CTAs of the backward = partial rows of the column sums: about 32 warps per SM
inline int ln_bwd_grid(int rows, int dim) {
  long long n;
  if (dim <= 256) {
    const int per = 8 * (32 / ln_lanes(dim)) * kLnU;
    n = ((long long)rows + per - 1) / per;
    return (int)(n < 4 * 152 ? n : 4 * 152);
  }
  const int warps = ln_threads(dim, ln_vpt(dim)) / 32;
  const int cap = 152 * (warps >= 32 ? 1 : 32 / warps);
  return rows < cap ? rows : cap;
}

// CTAs of the warp-per-row forward that the GPU holds at once (8192 rows of 2048 in bf16: 14.4 us; four an SM 15.2, eight
// 16.6).  The driver's answers take longer than the launch, so a thread keeps them for its last device and width.
template <typename T, int VPW>
int ln_warp_ctas(int dim) {
  thread_local int dev = -1, width = 0, n = 0;
  int now = 0;
  if (cudaGetDevice(&now) != cudaSuccess) return 0;
  if (now != dev || dim != width) {
    n = resident_ctas(ln_fwd_warp_kernel<T, VPW>, 256, (size_t)dim * 8) * device_sm_count();
    dev = n > 0 ? now : -1;
    width = dim;
  }
  return n;
}

template <typename T>
int ln_fwd_launch(const T* x, const float* scale, const float* bias, float eps, T* y, float* mean, float* rstd, int rows, int dim,
                  cudaStream_t s) {
  if (dim <= 256) {
    return ln_narrow(ln_lanes(dim), [&](auto tag) -> int {
      constexpr int G = decltype(tag)::value;
      const int per = 8 * (32 / G) * kLnU;
      long long grid = ((long long)rows + per - 1) / per;
      if (grid > 16 * 152) grid = 16 * 152;  // (30 us for 262144 rows of 128; a CTA for every set 32)
      ln_fwd_small_kernel<T, G, kLnU><<<(int)grid, 256, 0, s>>>(x, scale, bias, eps, y, mean, rstd, rows, dim);
      return cudaGetLastError() == cudaSuccess ? SS_OK : SS_ERR_CUDA;
    });
  }
  if (dim * sizeof(T) <= 4096) {
    auto run = [&](auto tag) -> int {
      constexpr int VPW = decltype(tag)::value;
      const int most = ln_warp_ctas<T, VPW>(dim), need = (int)(((long long)rows + 7) / 8);
      if (most < 1) return SS_ERR_CUDA;
      ln_fwd_warp_kernel<T, VPW><<<most < need ? most : need, 256, (size_t)dim * 8, s>>>(x, scale, bias, eps, y, mean, rstd, rows, dim);
      return cudaGetLastError() == cudaSuccess ? SS_OK : SS_ERR_CUDA;
    };
    if (dim <= 512) return run(std::integral_constant<int, 2>());
    if (sizeof(T) == 4 || dim <= 1024) return run(std::integral_constant<int, 4>());
    if constexpr (sizeof(T) == 2) return run(std::integral_constant<int, 8>());
  }
  const int vpt = dim <= 16384 ? 2 : 4, threads = ln_threads(dim, vpt);
  const int cap = 152 * (1024 / threads);
  const int grid = rows < cap ? rows : cap;
  if (vpt == 4) ln_fwd_wide_kernel<T, 4, false><<<grid, threads, 0, s>>>(x, scale, bias, eps, y, mean, rstd, rows, dim);
  else if (sizeof(T) == 2 && threads <= 512) ln_fwd_wide_kernel<T, 2, sizeof(T) == 2><<<grid, threads, 0, s>>>(x, scale, bias, eps, y, mean, rstd, rows, dim);
  else ln_fwd_wide_kernel<T, 2, false><<<grid, threads, 0, s>>>(x, scale, bias, eps, y, mean, rstd, rows, dim);
  return cudaGetLastError() == cudaSuccess ? SS_OK : SS_ERR_CUDA;
}

template <typename T>
int ln_bwd_launch(const T* dy, const T* x, const float* scale, const float* mean, const float* rstd, float* dx, float* dscale,
                  float* dbias, int add, int rows, int dim, float* ws, cudaStream_t s) {
  const int grid = ln_bwd_grid(rows, dim);
  if (dim <= 256) {
    const int rc = ln_narrow(ln_lanes(dim), [&](auto tag) -> int {
      constexpr int G = decltype(tag)::value;
      ln_bwd_small_kernel<T, G, kLnU><<<grid, 256, 0, s>>>(dy, x, scale, mean, rstd, dx, ws, rows, dim);
      return cudaGetLastError() == cudaSuccess ? SS_OK : SS_ERR_CUDA;
    });
    if (rc != SS_OK) return rc;
  } else {
    const int vpt = ln_vpt(dim), threads = ln_threads(dim, vpt);
    if (vpt == 1) ln_bwd_cols_kernel<T, 1><<<grid, threads, 0, s>>>(dy, x, scale, mean, rstd, dx, ws, rows, dim);
    else if (vpt == 2) ln_bwd_cols_kernel<T, 2><<<grid, threads, 0, s>>>(dy, x, scale, mean, rstd, dx, ws, rows, dim);
    else ln_bwd_cols_kernel<T, 4><<<grid, threads, 0, s>>>(dy, x, scale, mean, rstd, dx, ws, rows, dim);
    if (cudaGetLastError() != cudaSuccess) return SS_ERR_CUDA;
  }
  return colsum(ws, 2ll * dim, grid, ScaleBiasOut{dscale, dbias, dim, add}, s) == cudaSuccess ? SS_OK : SS_ERR_CUDA;
}

}  // namespace

extern "C" int layernorm_fwd(const void* x, const float* scale, const float* bias, float eps, void* y, float* mean, float* rstd,
                             int rows, int dim, int dtype, void* stream) {
  if (!x || !scale || !y) return SS_ERR_NULL;
  const int v = ln_validate(rows, dim, dtype);
  if (v != SS_OK) return v;
  if (!(eps >= 0.0f)) return SS_ERR_DIM;  // also rejects NaN
  const void* ptrs[] = {x, scale, bias, y, mean, rstd};
  for (const void* q : ptrs)
    if (q != nullptr && !ssh::aligned16(q)) return SS_ERR_ALIGN;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dtype == SS_F32)
    return ln_fwd_launch(static_cast<const float*>(x), scale, bias, eps, static_cast<float*>(y), mean, rstd, rows, dim, s);
  return ln_fwd_launch(static_cast<const __nv_bfloat16*>(x), scale, bias, eps, static_cast<__nv_bfloat16*>(y), mean, rstd, rows, dim, s);
}

extern "C" size_t layernorm_bwd_workspace_size(int rows, int dim) {
  if (ln_validate(rows, dim, SS_F32) != SS_OK) return 0;
  return (size_t)ln_bwd_grid(rows, dim) * 2 * dim * sizeof(float);
}

extern "C" int layernorm_bwd(const void* dy, const void* x, const float* scale, const float* mean, const float* rstd, float* dx,
                             float* dscale, float* dbias, int accumulate, int rows, int dim, int dtype, void* workspace,
                             size_t ws_bytes, void* stream) {
  if (!dy || !x || !scale || !mean || !rstd || !dx || !dscale || !dbias) return SS_ERR_NULL;
  const int v = ln_validate(rows, dim, dtype);
  if (v != SS_OK) return v;
  const void* ptrs[] = {dy, x, scale, mean, rstd, dx, dscale, dbias};
  for (const void* q : ptrs)
    if (!ssh::aligned16(q)) return SS_ERR_ALIGN;
  if (workspace == nullptr || ws_bytes < layernorm_bwd_workspace_size(rows, dim)) return SS_ERR_WORKSPACE;
  if (!ssh::aligned16(workspace)) return SS_ERR_ALIGN;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  float* ws = static_cast<float*>(workspace);
  if (dtype == SS_F32)
    return ln_bwd_launch(static_cast<const float*>(dy), static_cast<const float*>(x), scale, mean, rstd, dx, dscale, dbias, accumulate,
                         rows, dim, ws, s);
  return ln_bwd_launch(static_cast<const __nv_bfloat16*>(dy), static_cast<const __nv_bfloat16*>(x), scale, mean, rstd, dx, dscale,
                       dbias, accumulate, rows, dim, ws, s);
}
