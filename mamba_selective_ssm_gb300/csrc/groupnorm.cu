// Group norm with an activation, channels last, forward and backward (groupnorm_fwd, groupnorm_bwd) for sm_103a.
//
//   x [N, M, C], C in `groups` groups of cg channels; per sample n and group, over its M * cg values:
//   mean, rstd = 1 / sqrt(mean (x - mean)^2 + eps);   xh = (x - mean) rstd,   t = xh scale + bias,   y = act(t)
//   da = dy act'(t),  w = da scale;   dx = rstd (w - mean w - xh mean(w xh));   dscale += sum da xh;   dbias += sum da
// act is SiLU (t sigmoid(t), derivative p (1 + t (1 - p)) with p = sigmoid(t)) or nothing; t is found again in the backward.
//
// Three forms, by what a group's values are:
//   M = 1, cg <= 256 in eights   G lanes hold a row of a group, 32 / G groups (or rows) a warp, U rows in flight, the
//                                values in registers between the sums and the output: one pass over memory.
//   a sample of few values       a CTA holds one in registers (eight 16-byte units a thread), per-channel sums meet in
//                                shared memory: one pass too.
//   else                         sums by (sample, channels, rows) in fixed parts, a kernel that joins them, and a second
//                                pass for the output, which takes the rows from the last: L2 still holds those.
// The variance is taken around the mean (in parts around the mean of a few rows at a time, joined with their means), never as a
// difference of moments.  The backward's column sums are joined by colsum_kernel in fixed order.
//
// bf16 with SiLU, floors at 6.7 TB/s in brackets: 8192 x 1 x 4096 in 32 groups, forward 29 us (20; latency at four rows in flight a
// lane: 61 % of the issue slots, 38 % of memory), backward 50 + 6 (40); 4 x 2048 x 4096 forward 43 (20; x is read twice, the second time from L2 in
// part).  fp32, 8 x 2048 x 1536 in 24 groups, backward 89 (45; dy and x twice).  The forms at each other's sizes: the first of
// these with a sample in a CTA 105 and 283 us; 4096 x 4 x 512 with a sample in a CTA 34 and 60, in parts 203 and 184;
// 16 x 4 x 512 5.1 and 10, in parts 12.4 and 15; 8000 x 2 x 4096 136 and 410, in parts 1750 and 1890.
#include <algorithm>

#include "common.cuh"

namespace {

using namespace ssk;

constexpr int kGnMaxDim = 32768, kGnNarrow = 256, kGnMaxNarrow = 1 << 20;  // widest samples: in any groups, in groups of at most 256 channels
constexpr int kGnThreads = 256;
constexpr int kGnMost = 2147483647 - (1 << 22);  // samples or positions: a thread's next ones are still an int
constexpr int kGnSampleDim = 8192;  // widest sample of the one-CTA form

template <int G>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
  for (int o = 1; o < G; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ void ld8f(const float* p, bool ok, float* o) {
  const float4 a = ok ? __ldg(reinterpret_cast<const float4*>(p)) : make_float4(0.f, 0.f, 0.f, 0.f);
  const float4 b = ok ? __ldg(reinterpret_cast<const float4*>(p + 4)) : make_float4(0.f, 0.f, 0.f, 0.f);
  o[0] = a.x; o[1] = a.y; o[2] = a.z; o[3] = a.w; o[4] = b.x; o[5] = b.y; o[6] = b.z; o[7] = b.w;
}
// pairs of channels: packed arithmetic halves the instructions, which is what short rows are bound by
__device__ __forceinline__ void ld8p(const float* p, bool ok, float2 (&o)[4]) {
  float x[8];
  ld8f(p, ok, x);
#pragma unroll
  for (int e = 0; e < 4; ++e) o[e] = f2(x[2 * e], x[2 * e + 1]);
}
template <typename T>
__device__ __forceinline__ void wide4(const typename Raw8<T>::V& v, float2 (&o)[4]) {
  float x[8];
  Raw8<T>::wide(v, x);
#pragma unroll
  for (int e = 0; e < 4; ++e) o[e] = f2(x[2 * e], x[2 * e + 1]);
}
template <typename T>
__device__ __forceinline__ void st4p(T* p, const float2 (&o)[4]) {
  const float x[8] = {o[0].x, o[0].y, o[1].x, o[1].y, o[2].x, o[2].y, o[3].x, o[3].y};
  ActT<T>::st8(p, x);
}
// In the second pass of the parts' form x (and dy) are read for the last time and the output is not read again: marked so, more of
// them is still in L2 from the first pass (4 x 2048 x 4096 in bf16: 45.0 -> 42.9 us; backward of 8 x 2048 x 1536 in fp32 90.4 ->
// 88.6).
template <typename T>
__device__ __forceinline__ typename Raw8<T>::V ld_last(const T* p) {
  if constexpr (sizeof(T) == 4) {
    const float4* f = reinterpret_cast<const float4*>(p);
    return typename Raw8<T>::V{__ldcs(f), __ldcs(f + 1)};
  } else {
    return __ldcs(reinterpret_cast<const uint4*>(p));
  }
}
template <typename T>
__device__ __forceinline__ void st4_last(T* p, const float2 (&o)[4]) {
  if constexpr (sizeof(T) == 4) {
    __stcs(reinterpret_cast<float4*>(p), make_float4(o[0].x, o[0].y, o[1].x, o[1].y));
    __stcs(reinterpret_cast<float4*>(p) + 1, make_float4(o[2].x, o[2].y, o[3].x, o[3].y));
  } else {
    using A = ActT<__nv_bfloat16>;
    __stcs(reinterpret_cast<uint4*>(p),
           make_uint4(A::pack2(o[0].x, o[0].y), A::pack2(o[1].x, o[1].y), A::pack2(o[2].x, o[2].y), A::pack2(o[3].x, o[3].y)));
  }
}
__device__ __forceinline__ float2 sigmoid2(float2 t) {
  const float2 e = ex2_2(mul2(t, bc2(-kLog2e))), d = add2(e, bc2(1.f));
  return f2(rcp(d.x), rcp(d.y));
}
template <bool SILU>
__device__ __forceinline__ float2 act2(float2 t) {
  return SILU ? mul2(t, sigmoid2(t)) : t;
}
template <bool SILU>
__device__ __forceinline__ float2 dact2(float2 dy, float2 t) {
  if (!SILU) return dy;
  const float2 p = sigmoid2(t);
  return mul2(mul2(dy, p), fma2(t, fma2(p, bc2(-1.f), bc2(1.f)), bc2(1.f)));
}
__device__ __forceinline__ float sum4p(const float2 (&x)[4]) {
  const float2 s = add2(add2(x[0], x[1]), add2(x[2], x[3]));
  return s.x + s.y;
}

template <bool SILU>
__device__ __forceinline__ float act(float t) {
  return SILU ? t * sigmoid(t) : t;
}
// dy act'(t)
template <bool SILU>
__device__ __forceinline__ float dact(float dy, float t) {
  if (!SILU) return dy;
  const float p = sigmoid(t);
  return dy * (p * fmaf(t, 1.f - p, 1.f));
}

struct Gn {
  int N, M, C, groups, cg;
  float eps;
};

// ---------------------------------------------------------------- rows of a group in lanes (M = 1)

template <typename T, int G, int U, bool SILU>
__global__ void __launch_bounds__(kGnThreads) gn_fwd_lanes_kernel(Gn p, int gp, const T* __restrict__ x, const float* __restrict__ scale,
                                                                  const float* __restrict__ bias, T* __restrict__ y, float* __restrict__ mean,
                                                                  float* __restrict__ rstd) {
  using R = Raw8<T>;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, slot = lane / G, rs = 32 / G / gp;  // rs rows of gp groups a warp
  const int g = (int)blockIdx.y * gp + slot % gp, i = (lane % G) * 8, c = g * p.cg + i;
  const bool cv = g < p.groups && i < p.cg;
  float2 sc[4], bi[4];
  ld8p(scale + c, cv, sc);
  ld8p(bias + c, cv && bias != nullptr, bi);
  const float inv = 1.0f / (float)p.cg;
  const int step = (int)gridDim.x * 8 * rs * U;
  for (int w0 = ((int)blockIdx.x * 8 + warp) * rs * U; w0 < p.N; w0 += step) {  // (a warp goes round together: it shuffles)
    const int r0 = w0 + slot / gp;  // this lane's rows: r0 + u rs
    const T* src = x + (long long)r0 * p.C + c;
    typename R::V raw[U];
#pragma unroll
    for (int u = 0; u < U; ++u) raw[u] = cv && u * rs < p.N - r0 ? R::ld(src + (long long)(u * rs) * p.C) : R::zero();
    T* dst = y + (long long)r0 * p.C + c;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float2 v[4], q[4];
      wide4<T>(raw[u], v);
      const float m = lanes_sum<G>(sum4p(v)) * inv;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[e] = add2(v[e], bc2(-m));
        q[e] = mul2(v[e], v[e]);
      }
      const float rv = rsqrtf(fmaf(lanes_sum<G>(cv ? sum4p(q) : 0.f), inv, p.eps));
      if (cv && u * rs < p.N - r0) {
        if (i == 0) {
          const long long at = (long long)(r0 + u * rs) * p.groups + g;
          if (mean != nullptr) mean[at] = m;
          if (rstd != nullptr) rstd[at] = rv;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = act2<SILU>(fma2(mul2(v[e], bc2(rv)), sc[e], bi[e]));
        st4p<T>(dst + (long long)(u * rs) * p.C, v);
      }
    }
  }
}

template <typename T, int G, int U, bool SILU>
__global__ void __launch_bounds__(kGnThreads, 2) gn_bwd_lanes_kernel(Gn p, int gp, const T* __restrict__ dy, const T* __restrict__ x,
                                                                  const float* __restrict__ scale, const float* __restrict__ bias,
                                                                  const float* __restrict__ mean, const float* __restrict__ rstd,
                                                                  float* __restrict__ dx, float* __restrict__ part) {
  using R = Raw8<T>;
  __shared__ float4 red[4][kGnThreads];
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, slot = lane / G, rs = 32 / G / gp;
  const int g = (int)blockIdx.y * gp + slot % gp, i = (lane % G) * 8, c = g * p.cg + i;
  const bool cv = g < p.groups && i < p.cg;
  float2 sc[4], bi[4], as[4], ab[4];
  ld8p(scale + c, cv, sc);
  ld8p(bias + c, cv && SILU && bias != nullptr, bi);
#pragma unroll
  for (int e = 0; e < 4; ++e) as[e] = ab[e] = f2(0.f, 0.f);
  const float inv = 1.0f / (float)p.cg;
  const int step = (int)gridDim.x * 8 * rs * U;
  for (int w0 = ((int)blockIdx.x * 8 + warp) * rs * U; w0 < p.N; w0 += step) {
    const int r0 = w0 + slot / gp;
    const long long first = (long long)r0 * p.C + c;
    typename R::V rx[U], ry[U];
    float mu[U], rv[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool on = cv && u * rs < p.N - r0;
      const long long at = (long long)(r0 + u * rs) * p.groups + g;
      rx[u] = on ? R::ld(x + first + (long long)(u * rs) * p.C) : R::zero();
      ry[u] = on ? R::ld(dy + first + (long long)(u * rs) * p.C) : R::zero();
      mu[u] = on ? mean[at] : 0.f;
      rv[u] = on ? rstd[at] : 0.f;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float2 xh[4], w[4], q[4];
      wide4<T>(rx[u], xh);
      wide4<T>(ry[u], w);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        xh[e] = mul2(add2(xh[e], bc2(-mu[u])), bc2(rv[u]));
        const float2 da = dact2<SILU>(w[e], fma2(xh[e], sc[e], bi[e]));
        as[e] = fma2(da, xh[e], as[e]);
        ab[e] = add2(ab[e], da);
        w[e] = mul2(da, sc[e]);
        q[e] = mul2(w[e], xh[e]);
      }
      const float s1 = lanes_sum<G>(sum4p(w)) * inv, s2 = lanes_sum<G>(sum4p(q)) * inv;
      if (cv && u * rs < p.N - r0) {
        const float2 k0 = bc2(-s1 * rv[u]), k1 = bc2(-s2 * rv[u]), k2 = bc2(rv[u]);
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = fma2(k2, w[e], fma2(xh[e], k1, k0));
        st4p<float>(dx + first + (long long)(u * rs) * p.C, w);
      }
    }
  }
  red[0][threadIdx.x] = make_float4(as[0].x, as[0].y, as[1].x, as[1].y);
  red[1][threadIdx.x] = make_float4(as[2].x, as[2].y, as[3].x, as[3].y);
  red[2][threadIdx.x] = make_float4(ab[0].x, ab[0].y, ab[1].x, ab[1].y);
  red[3][threadIdx.x] = make_float4(ab[2].x, ab[2].y, ab[3].x, ab[3].y);
  __syncthreads();
  // the block's rows in order: a thread adds one of the four parts of a lane of a group
  const int w = threadIdx.x >> 6, l = threadIdx.x & 63;  // (gp * G <= 32 lanes hold different channels)
  if (l < gp * G && (int)blockIdx.y * gp + l / G < p.groups && (l % G) * 8 < p.cg) {
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int v = 0; v < 8; ++v)
      for (int o = 0; o < rs; ++o) {
        const float4 z = red[w][v * 32 + o * gp * G + l];
        s.x += z.x; s.y += z.y; s.z += z.z; s.w += z.w;
      }
    const int cc = ((int)blockIdx.y * gp + l / G) * p.cg + (l % G) * 8 + (w & 1) * 4;
    *reinterpret_cast<float4*>(part + (size_t)blockIdx.x * 2 * p.C + (w >> 1) * p.C + cc) = s;
  }
}

// ---------------------------------------------------------------- a sample in a CTA

// Which of a sample's units (8 channels of one position) a thread holds.  Up to 256 units a position: one of them, of every
// `lanes`-th position; more: every 256th unit of all positions.  Walked with next(), which divides nothing (with the divisions that
// a unit's place and its channels' groups take otherwise, 4096 samples of 4 x 512 took 124 us).
struct Mine {
  int units, lanes, rl, items;  // units of a position; threads that share one, this one's place among them; units held, at most
  int per, step, m0, u0;        // units of a position held, positions from one to the next
  uint32_t magic;               // 2^26 / cg, rounded up: exact quotients below 2^13 (kGnSampleDim)
  int m, u, k;
  __device__ __forceinline__ Mine(const Gn& p, int n) {
    units = p.C / 8;
    items = n;
    const bool narrow = units < kGnThreads;
    lanes = narrow ? kGnThreads / units : 1;
    rl = narrow ? (int)threadIdx.x / units : 0;
    u0 = narrow ? (int)threadIdx.x % units : (int)threadIdx.x;
    per = narrow ? 1 : (units + kGnThreads - 1) / kGnThreads;
    step = lanes;
    m0 = rl < lanes ? rl : p.M;
    magic = (1u << 26) / (uint32_t)p.cg + 1u;
  }
  __device__ __forceinline__ void first() {
    m = m0;
    u = u0;
    k = 0;
  }
  __device__ __forceinline__ bool on(const Gn& p) const { return m < p.M && u < units; }
  __device__ __forceinline__ void next() {
    u += kGnThreads;
    if (++k == per) {
      k = 0;
      u = u0;
      m += step;
    }
  }
  __device__ __forceinline__ int group(int e) const { return (int)__umulhi((uint32_t)(u * 8 + e) << 6, magic); }
};
inline int gn_sample_items(const Gn& p) {
  const int units = p.C / 8;
  if (units < kGnThreads) return (p.M + kGnThreads / units - 1) / (kGnThreads / units);
  const long long n = (long long)((units + kGnThreads - 1) / kGnThreads) * p.M;
  return n > 1000 ? 1000 : (int)n;
}
template <typename T>
constexpr int kGnItems = 16 / sizeof(T);  // units a thread holds: 128 bytes of x

// A unit goes to its thread's own place in shared memory (registers would have to be indexed by constants: a kernel that
// unrolled its eight units held 230 of them, and one CTA an SM, or spilled).
template <typename V, typename T>
__device__ __forceinline__ void hold_copy(V* dst, const T* src) {
#pragma unroll
  for (int e = 0; e < (int)sizeof(V); e += 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst) + e), "l"(reinterpret_cast<const char*>(src) + e) : "memory");
}
__device__ __forceinline__ void hold_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// dst[g] = f(sum over the group's channels and the `lanes` rows of part), a warp to a group
template <typename F>
__device__ __forceinline__ void group_sums(const Gn& p, const float* part, int lanes, F f) {
  const int lane = threadIdx.x & 31;
  for (int g = threadIdx.x >> 5; g < p.groups; g += kGnThreads / 32) {
    float s = 0.f;
    for (int l = 0; l < lanes; ++l)
      for (int j = lane; j < p.cg; j += 32) s += part[l * p.C + g * p.cg + j];
    s = lanes_sum<32>(s);
    if (lane == 0) f(g, s);
  }
}
// per-channel sums of a thread's units into part[lanes][C]; val(i, e) its values
template <typename V>
__device__ __forceinline__ void channel_sums(const Gn& p, Mine& my, float* part, V val) {
  float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  my.first();
  for (int i = 0; i < my.items; ++i, my.next()) {
    if (my.units < kGnThreads) {  // one unit: summed over its positions
      if (my.on(p)) {
#pragma unroll
        for (int e = 0; e < 8; ++e) s[e] += val(i, e);
      }
    } else if (my.on(p)) {
      float* at = part + my.u * 8;
      if (my.m == 0) {
#pragma unroll
        for (int e = 0; e < 8; ++e) s[e] = val(i, e);
      } else {
        ActT<float>::ld8(at, s);
#pragma unroll
        for (int e = 0; e < 8; ++e) s[e] += val(i, e);
      }
      ActT<float>::st8(at, s);
    }
  }
  if (my.units < kGnThreads && my.rl < my.lanes) ActT<float>::st8(part + my.rl * p.C + my.u0 * 8, s);
}

inline size_t gn_part_floats(const Gn& p) { return p.C < 8 * kGnThreads ? 8 * kGnThreads : p.C; }

template <typename T, bool SILU>
__global__ void __launch_bounds__(kGnThreads, 4) gn_fwd_sample_kernel(Gn p, int items, const T* __restrict__ x, const float* __restrict__ scale,
                                                                   const float* __restrict__ bias, T* __restrict__ y, float* __restrict__ mean,
                                                                   float* __restrict__ rstd) {
  using R = Raw8<T>;
  extern __shared__ float4 sm4[];
  typename R::V* hold = reinterpret_cast<typename R::V*>(sm4) + threadIdx.x;  // this thread's units of x
  float* part = reinterpret_cast<float*>(sm4) + items * kGnThreads * (int)(sizeof(typename R::V) / 4);
  float* st = part + (p.C < 8 * kGnThreads ? 8 * kGnThreads : p.C);  // mean, rstd of each group
  Mine my(p, items);
  const float inv = 1.0f / ((float)p.M * (float)p.cg);
  for (long long n = blockIdx.x; n < p.N; n += gridDim.x) {
    const T* xn = x + n * p.M * p.C;
    my.first();
    for (int i = 0; i < items; ++i, my.next())
      if (my.on(p)) hold_copy(hold + i * kGnThreads, xn + (long long)my.m * p.C + my.u * 8);
    hold_wait();
    float v[8];
    channel_sums(p, my, part, [&](int i, int e) {
      if (e == 0) R::wide(hold[i * kGnThreads], v);
      return v[e];
    });
    __syncthreads();
    group_sums(p, part, my.lanes, [&](int g, float s) { st[g] = s * inv; });
    __syncthreads();
    channel_sums(p, my, part, [&](int i, int e) {
      if (e == 0) R::wide(hold[i * kGnThreads], v);
      const float d = v[e] - st[my.group(e)];
      return d * d;
    });
    __syncthreads();
    group_sums(p, part, my.lanes, [&](int g, float s) {
      const float r = rsqrtf(fmaf(s, inv, p.eps));
      st[p.groups + g] = r;
      if (mean != nullptr) mean[n * p.groups + g] = st[g];
      if (rstd != nullptr) rstd[n * p.groups + g] = r;
    });
    __syncthreads();
    my.first();
    for (int i = 0; i < items; ++i, my.next()) {
      if (!my.on(p)) continue;
      float sc[8], bi[8];
      ld8f(scale + my.u * 8, true, sc);
      ld8f(bias + my.u * 8, bias != nullptr, bi);
      R::wide(hold[i * kGnThreads], v);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int g = my.group(e);
        v[e] = act<SILU>(fmaf((v[e] - st[g]) * st[p.groups + g], sc[e], bi[e]));
      }
      ActT<T>::st8(y + (n * p.M + my.m) * p.C + my.u * 8, v);
    }
    __syncthreads();  // the next sample's sums
  }
}

template <typename T, bool SILU>
__global__ void __launch_bounds__(kGnThreads, 3) gn_bwd_sample_kernel(Gn p, int items, const T* __restrict__ dy, const T* __restrict__ x,
                                                                   const float* __restrict__ scale, const float* __restrict__ bias,
                                                                   const float* __restrict__ mean, const float* __restrict__ rstd,
                                                                   float* __restrict__ dx, float* __restrict__ out) {
  using R = Raw8<T>;
  extern __shared__ float4 sm4[];
  const int pf = p.C < 8 * kGnThreads ? 8 * kGnThreads : p.C;
  typename R::V* hold = reinterpret_cast<typename R::V*>(sm4) + threadIdx.x;  // this thread's units of x, then of dy
  float *part = reinterpret_cast<float*>(sm4) + 2 * items * kGnThreads * (int)(sizeof(typename R::V) / 4), *acc = part + pf, *st = acc + 2 * p.C;
  pdl_trigger();
  for (int c = threadIdx.x; c < 2 * p.C; c += kGnThreads) acc[c] = 0.f;
  Mine my(p, items);
  const float inv = 1.0f / ((float)p.M * (float)p.cg);
  for (long long n = blockIdx.x; n < p.N; n += gridDim.x) {
    my.first();
    for (int i = 0; i < items; ++i, my.next()) {
      if (!my.on(p)) continue;
      const long long at = (n * p.M + my.m) * p.C + my.u * 8;
      hold_copy(hold + i * kGnThreads, x + at);
      hold_copy(hold + (items + i) * kGnThreads, dy + at);
    }
    hold_wait();
    const float *mu = mean + n * p.groups, *rv = rstd + n * p.groups;
    float sc[8], bi[8], xh[8], da[8];
    auto unit = [&](int i) {  // xh and da of a unit
      ld8f(scale + my.u * 8, true, sc);
      ld8f(bias + my.u * 8, SILU && bias != nullptr, bi);
      R::wide(hold[i * kGnThreads], xh);
      R::wide(hold[(items + i) * kGnThreads], da);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int g = my.group(e);
        xh[e] = (xh[e] - mu[g]) * rv[g];
        da[e] = dact<SILU>(da[e], fmaf(xh[e], sc[e], bi[e]));
      }
    };
    // sums of da, then of da xh: per channel into the column sums, per group with the scale
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      channel_sums(p, my, part, [&](int i, int e) {
        if (e == 0) unit(i);
        return k == 0 ? da[e] : da[e] * xh[e];
      });
      __syncthreads();
      for (int c = threadIdx.x; c < p.C; c += kGnThreads) {
        float s = 0.f;
        for (int l = 0; l < my.lanes; ++l) s += part[l * p.C + c];
        acc[(1 - k) * p.C + c] += s;
        part[c] = s * scale[c];
      }
      __syncthreads();
      group_sums(p, part, 1, [&](int g, float s) { st[k * p.groups + g] = s * inv; });
      __syncthreads();
    }
    my.first();
    for (int i = 0; i < items; ++i, my.next()) {
      if (!my.on(p)) continue;
      unit(i);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int g = my.group(e);
        // (w and its mean, each rounded, first: in a group of one value they are the same, and dx is 0)
        da[e] = rv[g] * fmaf(-xh[e], st[p.groups + g], __fsub_rn(__fmul_rn(da[e], sc[e]), st[g]));
      }
      ActT<float>::st8(dx + (n * p.M + my.m) * p.C + my.u * 8, da);
    }
    __syncthreads();
  }
  __syncthreads();
  for (int c = threadIdx.x; c < 2 * p.C; c += kGnThreads) out[(size_t)blockIdx.x * 2 * p.C + c] = acc[c];
}

// ---------------------------------------------------------------- long samples, in parts

// A CTA's part: `ut` units of channels from u0, rows m0 .. m1 of sample n; thread = (unit, row lane)
struct Part {
  int ut, tiles, splits, per;  // units a CTA, CTAs across C, parts of the rows, rows of a part
};
struct Where {
  long long n;
  int split, c, rl, lanes, m0, m1;
  bool on;
  __device__ __forceinline__ Where(const Gn& p, const Part& q) {
    long long id = blockIdx.x;
    const int tile = (int)(id % q.tiles);
    id /= q.tiles;
    split = (int)(id % q.splits);
    n = id / q.splits;
    lanes = kGnThreads / q.ut;
    rl = (int)threadIdx.x / q.ut;
    c = (tile * q.ut + (int)threadIdx.x % q.ut) * 8;
    on = rl < lanes && c < p.C;
    m0 = split * q.per;
    m1 = m0 + q.per < p.M ? m0 + q.per : p.M;
  }
};
// the row lanes' sums, in pairs: red[thread][8] -> the first lane, and there
__device__ __forceinline__ void lanes_add(float4 (*red)[kGnThreads], int ut, int lanes, float2 (&s)[4]) {
  const int tid = threadIdx.x, rl = tid / ut;
  __syncthreads();
  red[0][tid] = make_float4(s[0].x, s[0].y, s[1].x, s[1].y);
  red[1][tid] = make_float4(s[2].x, s[2].y, s[3].x, s[3].y);
  int h = 1;
  while (h < lanes) h *= 2;
  for (h /= 2; h > 0; h /= 2) {
    __syncthreads();
    if (rl < h && rl + h < lanes) {
      const float4 a = red[0][tid + h * ut], b = red[1][tid + h * ut];
      s[0] = add2(s[0], f2(a.x, a.y));
      s[1] = add2(s[1], f2(a.z, a.w));
      s[2] = add2(s[2], f2(b.x, b.y));
      s[3] = add2(s[3], f2(b.z, b.w));
      red[0][tid] = make_float4(s[0].x, s[0].y, s[1].x, s[1].y);
      red[1][tid] = make_float4(s[2].x, s[2].y, s[3].x, s[3].y);
    }
  }
}
template <typename T>
constexpr int kGnAhead = 16 / sizeof(T);  // rows of a thread in flight: 128 bytes

// part[n][split][c] = the rows' sum, and after all of those the sum of squares around their mean.  A thread's rows come in sets
// of a few: a set's squares are taken around its own mean, and sets, then threads, are joined as
//   m2 = m2_a + m2_b + (mean_a - mean_b)^2 n_a n_b / (n_a + n_b),
// sums of squares all, so that no row (a first one of zeros, one far from the others) costs the variance its digits, as it did when
// the squares were taken around the first row: 1e-4 of rstd for 4096 rows a thread's part of deviation 1 and mean 100 behind one of
// zeros.  A thread's sum carries what its additions drop (kahan), since a thread may have most of a long sample.
template <typename T>
__global__ void __launch_bounds__(kGnThreads, 2) gn_stats_kernel(Gn p, Part q, const T* __restrict__ x, float* __restrict__ part) {
  using R = Raw8<T>;
  __shared__ float4 red[2][kGnThreads];
  pdl_trigger();
  const Where w(p, q);
  float2 s[4], lost[4], m2[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) s[e] = lost[e] = m2[e] = f2(0.f, 0.f);
  const T* src = x + w.n * p.M * p.C + w.c;
  constexpr int A = kGnAhead<T>;
  float n = 0.f;  // rows so far
  if (w.on) {
    for (int m = w.m0 + w.rl; m < w.m1; m += A * w.lanes) {
      typename R::V raw[A];
      int rows = 0;
#pragma unroll
      for (int u = 0; u < A; ++u)
        if (m + u * w.lanes < w.m1) {
          raw[u] = R::ld(src + (long long)(m + u * w.lanes) * p.C);
          rows = u + 1;
        }
      float2 b[4], mb[4], sq[4], v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) b[e] = sq[e] = f2(0.f, 0.f);
#pragma unroll
      for (int u = 0; u < A; ++u) {
        if (u >= rows) break;
        wide4<T>(raw[u], v);
#pragma unroll
        for (int e = 0; e < 4; ++e) b[e] = add2(b[e], v[e]);
      }
      const float nb = (float)rows, ib = rows == A ? 1.f / A : __frcp_rn(nb);
#pragma unroll
      for (int e = 0; e < 4; ++e) mb[e] = mul2(b[e], bc2(-ib));
#pragma unroll
      for (int u = 0; u < A; ++u) {
        if (u >= rows) break;
        wide4<T>(raw[u], v);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          v[e] = add2(v[e], mb[e]);
          sq[e] = fma2(v[e], v[e], sq[e]);
        }
      }
      const float in = n > 0.f ? __frcp_rn(n) : 0.f, wt = __fdividef(n * nb, n + nb);
      n += nb;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 d = fma2(s[e], bc2(in), mb[e]);  // (of the rows before, minus the set's)
        m2[e] = add2(m2[e], fma2(mul2(d, bc2(wt)), d, sq[e]));
        const float2 y = fma2(lost[e], bc2(-1.f), b[e]), t = add2(s[e], y);
        lost[e] = fma2(y, bc2(-1.f), fma2(s[e], bc2(-1.f), t));
        s[e] = t;
      }
    }
  }
  float2 own[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) own[e] = s[e];
  lanes_add(red, q.ut, w.lanes, s);
  __syncthreads();
  {
    const float4 a = red[0][threadIdx.x % q.ut], b = red[1][threadIdx.x % q.ut];
    const float2 all[4] = {f2(a.x, a.y), f2(a.z, a.w), f2(b.x, b.y), f2(b.z, b.w)};
    const float inv = -1.f / (float)(w.m1 - w.m0), in = n > 0.f ? __frcp_rn(n) : 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 d = fma2(own[e], bc2(in), mul2(all[e], bc2(inv)));
      m2[e] = fma2(mul2(d, bc2(n)), d, m2[e]);
    }
  }
  lanes_add(red, q.ut, w.lanes, m2);
  if (w.on && w.rl == 0) {
    float* at = part + (w.n * q.splits + w.split) * p.C + w.c;
    st4p<float>(at, s);
    st4p<float>(at + (long long)p.N * q.splits * p.C, m2);
  }
}

__device__ __forceinline__ float block_sum(float* red, float v) {
  v = lanes_sum<32>(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.f;
#pragma unroll
  for (int w = 0; w < kGnThreads / 32; ++w) s += red[w];
  return s;
}

// f(channel of the group, part) over all of them, by the threads of a CTA
template <typename F>
__device__ __forceinline__ void each_part(const Gn& p, const Part& q, F f) {
  const int w = p.cg < kGnThreads ? p.cg : kGnThreads, l = kGnThreads / w, r = (int)threadIdx.x / w;
  if (r < l)
    for (int c = (int)threadIdx.x % w; c < p.cg; c += w)
#pragma unroll 4
      for (int s = r; s < q.splits; s += l) f(c, s);
}

// a CTA joins the parts of one (sample, group)
__global__ void __launch_bounds__(kGnThreads) gn_join_kernel(Gn p, Part q, const float* __restrict__ part, float* __restrict__ mean,
                                                             float* __restrict__ rstd) {
  __shared__ float red[kGnThreads / 32];
  pdl_trigger();
  const long long n = blockIdx.x / p.groups;
  const int g = blockIdx.x % p.groups;
  const float inv = 1.0f / ((float)p.M * (float)p.cg);
  const float* sum = part + n * q.splits * p.C + g * p.cg;
  const float* sq = sum + (long long)p.N * q.splits * p.C;
  const float full = (float)q.per, last = (float)(p.M - (q.splits - 1) * q.per), fi = 1.f / full, li = 1.f / last;
  pdl_wait();
  float s = 0.f;
  each_part(p, q, [&](int c, int i) { s += sum[(long long)i * p.C + c]; });
  const float m = block_sum(red, s) * inv;
  s = 0.f;
  each_part(p, q, [&](int c, int i) {
    const bool end = i == q.splits - 1;
    const float d = fmaf(sum[(long long)i * p.C + c], end ? li : fi, -m);
    s += fmaf(d * d, end ? last : full, sq[(long long)i * p.C + c]);
  });
  s = block_sum(red, s);
  if (threadIdx.x == 0) {
    mean[blockIdx.x] = m;
    rstd[blockIdx.x] = rsqrtf(fmaf(s, inv, p.eps));
  }
}

template <typename T, bool SILU>
__global__ void __launch_bounds__(kGnThreads, 2) gn_apply_kernel(Gn p, Part q, const T* __restrict__ x, const float* __restrict__ scale,
                                                              const float* __restrict__ bias, const float* __restrict__ mean,
                                                              const float* __restrict__ rstd, T* __restrict__ y) {
  using R = Raw8<T>;
  const Where w(p, q);
  if (!w.on) return;
  float2 sc[4], bi[4], mu[4];
  ld8p(scale + w.c, true, sc);
  ld8p(bias + w.c, bias != nullptr, bi);
  pdl_wait();
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const long long g = w.n * p.groups + (w.c + 2 * e) / p.cg, h = w.n * p.groups + (w.c + 2 * e + 1) / p.cg;
    mu[e] = f2(-mean[g], -mean[h]);
    sc[e] = mul2(sc[e], f2(rstd[g], rstd[h]));
  }
  const long long base = w.n * p.M * p.C + w.c;
  constexpr int A = kGnAhead<T> / 2;
  for (int m = w.m1 - 1 - w.rl; m >= w.m0; m -= A * w.lanes) {
    typename R::V raw[A];
#pragma unroll
    for (int u = 0; u < A; ++u)
      if (m - u * w.lanes >= w.m0) raw[u] = ld_last<T>(x + base + (long long)(m - u * w.lanes) * p.C);
#pragma unroll
    for (int u = 0; u < A; ++u) {
      if (m - u * w.lanes < w.m0) break;
      float2 v[4];
      wide4<T>(raw[u], v);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = act2<SILU>(fma2(add2(v[e], mu[e]), sc[e], bi[e]));
      st4_last<T>(y + base + (long long)(m - u * w.lanes) * p.C, v);
    }
  }
}

// part[n][split][2 C]: the rows' sums of da xh and of da
template <typename T, bool SILU>
__global__ void __launch_bounds__(kGnThreads, 2) gn_bwd_sums_kernel(Gn p, Part q, const T* __restrict__ dy, const T* __restrict__ x,
                                                                 const float* __restrict__ scale, const float* __restrict__ bias,
                                                                 const float* __restrict__ mean, const float* __restrict__ rstd,
                                                                 float* __restrict__ part) {
  using R = Raw8<T>;
  __shared__ float4 red[2][kGnThreads];
  pdl_trigger();
  const Where w(p, q);
  float2 s1[4], s2[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) s1[e] = s2[e] = f2(0.f, 0.f);
  if (w.on) {
    float2 sc[4], bi[4], mu[4], rv[4];
    ld8p(scale + w.c, true, sc);
    ld8p(bias + w.c, SILU && bias != nullptr, bi);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const long long g = w.n * p.groups + (w.c + 2 * e) / p.cg, h = w.n * p.groups + (w.c + 2 * e + 1) / p.cg;
      mu[e] = f2(-mean[g], -mean[h]);
      rv[e] = f2(rstd[g], rstd[h]);
    }
    const long long base = w.n * p.M * p.C + w.c;
    constexpr int A = kGnAhead<T> / 2;
    for (int m = w.m0 + w.rl; m < w.m1; m += A * w.lanes) {
      typename R::V rx[A], ry[A];
#pragma unroll
      for (int u = 0; u < A; ++u)
        if (m + u * w.lanes < w.m1) {
          const long long at = base + (long long)(m + u * w.lanes) * p.C;
          rx[u] = R::ld(x + at);
          ry[u] = R::ld(dy + at);
        }
#pragma unroll
      for (int u = 0; u < A; ++u) {
        if (m + u * w.lanes >= w.m1) break;
        float2 xh[4], da[4];
        wide4<T>(rx[u], xh);
        wide4<T>(ry[u], da);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          xh[e] = mul2(add2(xh[e], mu[e]), rv[e]);
          da[e] = dact2<SILU>(da[e], fma2(xh[e], sc[e], bi[e]));
          s1[e] = add2(s1[e], da[e]);
          s2[e] = fma2(da[e], xh[e], s2[e]);
        }
      }
    }
  }
  lanes_add(red, q.ut, w.lanes, s1);
  lanes_add(red, q.ut, w.lanes, s2);
  if (w.on && w.rl == 0) {
    float* at = part + (w.n * q.splits + w.split) * 2 * p.C + w.c;
    st4p<float>(at, s2);
    st4p<float>(at + p.C, s1);
  }
}

// means[n][g] of w and of w xh from the parts
__global__ void __launch_bounds__(kGnThreads) gn_bwd_join_kernel(Gn p, Part q, const float* __restrict__ part, const float* __restrict__ scale,
                                                                 float2* __restrict__ means) {
  __shared__ float red[kGnThreads / 32];
  pdl_trigger();
  const long long n = blockIdx.x / p.groups;
  const int g = blockIdx.x % p.groups;
  const float inv = 1.0f / ((float)p.M * (float)p.cg);
  const float* at = part + n * q.splits * 2 * p.C + g * p.cg;
  pdl_wait();
  float a = 0.f, b = 0.f;
  each_part(p, q, [&](int c, int i) {
    const float s = scale[g * p.cg + c];
    const float* y = at + (long long)i * 2 * p.C + c;
    b = fmaf(y[0], s, b);
    a = fmaf(y[p.C], s, a);
  });
  a = block_sum(red, a);
  b = block_sum(red, b);
  if (threadIdx.x == 0) means[blockIdx.x] = make_float2(a * inv, b * inv);
}

template <typename T, bool SILU>
__global__ void __launch_bounds__(kGnThreads, 2) gn_bwd_apply_kernel(Gn p, Part q, const T* __restrict__ dy, const T* __restrict__ x,
                                                                  const float* __restrict__ scale, const float* __restrict__ bias,
                                                                  const float* __restrict__ mean, const float* __restrict__ rstd,
                                                                  const float2* __restrict__ means, float* __restrict__ dx) {
  using R = Raw8<T>;
  const Where w(p, q);
  if (!w.on) return;
  float2 sc[4], bi[4], mu[4], rv[4], k0[4], k1[4];
  ld8p(scale + w.c, true, sc);
  ld8p(bias + w.c, SILU && bias != nullptr, bi);
  pdl_wait();
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const long long g = w.n * p.groups + (w.c + 2 * e) / p.cg, h = w.n * p.groups + (w.c + 2 * e + 1) / p.cg;
    const float2 a = means[g], b = means[h];
    mu[e] = f2(-mean[g], -mean[h]);
    rv[e] = f2(rstd[g], rstd[h]);
    k0[e] = f2(-a.x, -b.x);
    k1[e] = f2(-a.y, -b.y);
  }
  constexpr int A = kGnAhead<T> / 2;
  const long long base = w.n * p.M * p.C + w.c;
  for (int m = w.m1 - 1 - w.rl; m >= w.m0; m -= A * w.lanes) {
    typename R::V rx[A], ry[A];
#pragma unroll
    for (int u = 0; u < A; ++u)
      if (m - u * w.lanes >= w.m0) {
        const long long at = base + (long long)(m - u * w.lanes) * p.C;
        rx[u] = ld_last<T>(x + at);
        ry[u] = ld_last<T>(dy + at);
      }
#pragma unroll
    for (int u = 0; u < A; ++u) {
      if (m - u * w.lanes < w.m0) break;
      float2 xh[4], da[4];
      wide4<T>(rx[u], xh);
      wide4<T>(ry[u], da);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        xh[e] = mul2(add2(xh[e], mu[e]), rv[e]);
        da[e] = dact2<SILU>(da[e], fma2(xh[e], sc[e], bi[e]));
        // w - mean w first, as above (in scalars: a packed product and sum are made one)
        da[e] = f2(__fadd_rn(__fmul_rn(da[e].x, sc[e].x), k0[e].x), __fadd_rn(__fmul_rn(da[e].y, sc[e].y), k0[e].y));
        da[e] = mul2(rv[e], fma2(xh[e], k1[e], da[e]));
      }
      st4_last<float>(dx + base + (long long)(m - u * w.lanes) * p.C, da);
    }
  }
}

// ---------------------------------------------------------------- host

enum GnForm { kLanes, kSample, kParts };

struct GnPlan {
  Gn p;
  GnForm form;
  int G, gp, segs, grid;  // lanes
  int items;              // a sample's units in a thread
  Part q, qa;             // parts of the sums, and of the forward's second pass
  size_t fwd, bwd;        // workspace
  int rows;               // partial rows of the backward's column sums
};

int gn_plan(int N, int M, int C, int groups, int dtype, GnPlan& pl) {
  if (N <= 0 || M <= 0 || C <= 0 || groups <= 0 || C % groups != 0) return SS_ERR_DIM;
  if (C > (C / groups <= kGnNarrow ? kGnMaxNarrow : kGnMaxDim)) return SS_ERR_DIM;
  if (dtype != SS_F32 && dtype != SS_BF16) return SS_ERR_UNSUPPORTED;
  if (C % 8 != 0) return SS_ERR_ALIGN;
  if (N > kGnMost || M > kGnMost) return SS_ERR_DIM;
  if ((long long)N * groups > 2147483647ll || (long long)N * M > (1ll << 40) / C) return SS_ERR_DIM;
  Gn& p = pl.p;
  p.N = N; p.M = M; p.C = C; p.groups = groups; p.cg = C / groups;
  pl.fwd = pl.bwd = 0;
  const int items = pl.items = gn_sample_items(p);
  if (M == 1 && p.cg % 8 == 0 && p.cg <= 256) {
    pl.form = kLanes;
    pl.G = 1;
    while (pl.G * 8 < p.cg) pl.G *= 2;
    pl.gp = 1;
    while (pl.gp < groups && pl.gp < 32 / pl.G) pl.gp *= 2;
    pl.segs = (groups + pl.gp - 1) / pl.gp;
    const long long sets = ((long long)N + 32 / pl.G / pl.gp * 8 - 1) / (32 / pl.G / pl.gp * 8);  // one set of rows for each warp
    pl.grid = (int)std::min<long long>(sets, std::max(1, 152 * 8 / pl.segs));
    pl.rows = pl.grid;
    pl.bwd = (size_t)pl.rows * 2 * C * sizeof(float);
  } else if (C <= kGnSampleDim && items <= (dtype == SS_F32 ? kGnItems<float> : kGnItems<__nv_bfloat16>)) {
    pl.form = kSample;
    pl.grid = std::min(N, 152 * 8);
    pl.rows = pl.grid;
    pl.bwd = (size_t)pl.rows * 2 * C * sizeof(float);
  } else {
    pl.form = kParts;
    // one turn of two CTAs an SM for the sums (17.8 -> 15.9 us for 4 x 2048 x 4096 in bf16 against two turns), three turns
    // for the forward's output (25 -> 22)
    auto parts = [&](int turns) {
      Part q;
      q.ut = std::min(32, C / 8);
      q.tiles = (C / 8 + q.ut - 1) / q.ut;
      const int lanes = kGnThreads / q.ut;
      const long long want = std::max<long long>(1, 152ll * 2 * turns / ((long long)N * q.tiles));
      const int splits = (int)std::min<long long>(want, std::max(1, M / (lanes * 4)));
      q.per = (M + splits - 1) / splits;
      q.splits = (M + q.per - 1) / q.per;
      return q;
    };
    pl.qa = parts(3);
    pl.q = parts(1);
    const Part& q = pl.q;
    if ((long long)N * pl.qa.splits * q.tiles > 2147483647ll) return SS_ERR_DIM;
    pl.rows = N * q.splits;
    pl.fwd = (size_t)N * q.splits * 2 * C * sizeof(float) + (size_t)N * groups * 2 * sizeof(float);
    pl.bwd = (size_t)N * q.splits * 2 * C * sizeof(float) + (size_t)N * groups * 2 * sizeof(float);
  }
  return SS_OK;
}

template <typename T, int G, bool SILU>
void fwd_lanes(const GnPlan& pl, const T* x, const float* scale, const float* bias, T* y, float* mean, float* rstd, cudaStream_t s) {
  gn_fwd_lanes_kernel<T, G, 4, SILU><<<dim3(pl.grid, pl.segs), kGnThreads, 0, s>>>(pl.p, pl.gp, x, scale, bias, y, mean, rstd);
}
template <typename T, int G, bool SILU>
void bwd_lanes(const GnPlan& pl, const T* dy, const T* x, const float* scale, const float* bias, const float* mean, const float* rstd, float* dx,
               float* part, cudaStream_t s) {
  gn_bwd_lanes_kernel<T, G, 3, SILU><<<dim3(pl.grid, pl.segs), kGnThreads, 0, s>>>(pl.p, pl.gp, dy, x, scale, bias, mean, rstd, dx, part);
}
#define GN_LANES(f, ...)                             \
  switch (pl.G) {                                    \
    case 1: f<T, 1, SILU>(__VA_ARGS__); break;       \
    case 2: f<T, 2, SILU>(__VA_ARGS__); break;       \
    case 4: f<T, 4, SILU>(__VA_ARGS__); break;       \
    case 8: f<T, 8, SILU>(__VA_ARGS__); break;       \
    case 16: f<T, 16, SILU>(__VA_ARGS__); break;     \
    default: f<T, 32, SILU>(__VA_ARGS__); break;     \
  }

template <typename T, bool SILU>
int fwd(const GnPlan& pl, const T* x, const float* scale, const float* bias, T* y, float* mean, float* rstd, void* ws, cudaStream_t s) {
  const Gn& p = pl.p;
  if (pl.form == kLanes) {
    GN_LANES(fwd_lanes, pl, x, scale, bias, y, mean, rstd, s)
  } else if (pl.form == kSample) {
    const size_t smem = pl.items * kGnThreads * sizeof(typename Raw8<T>::V) + (gn_part_floats(p) + 2 * p.groups) * sizeof(float);
    const auto kernel = gn_fwd_sample_kernel<T, SILU>;
    if (!allow_smem(kernel)) return SS_ERR_CUDA;
    kernel<<<pl.grid, kGnThreads, smem, s>>>(p, pl.items, x, scale, bias, y, mean, rstd);
  } else {
    const Part& q = pl.q;
    float* part = static_cast<float*>(ws);
    float* st = part + (size_t)p.N * q.splits * 2 * p.C;
    float* mu = mean != nullptr ? mean : st;
    float* rv = rstd != nullptr ? rstd : st + (size_t)p.N * p.groups;
    const unsigned grid = (unsigned)((long long)p.N * q.splits * q.tiles);
    gn_stats_kernel<T><<<grid, kGnThreads, 0, s>>>(p, q, x, part);
    if (launch_dependent(gn_join_kernel, dim3((unsigned)((long long)p.N * p.groups)), dim3(kGnThreads), 0, s, p, q, (const float*)part, mu, rv) !=
            cudaSuccess ||
        launch_dependent(gn_apply_kernel<T, SILU>, dim3((unsigned)((long long)p.N * pl.qa.splits * q.tiles)), dim3(kGnThreads), 0, s, p, pl.qa, x,
                         scale, bias, (const float*)mu, (const float*)rv, y) !=
            cudaSuccess)
      return SS_ERR_CUDA;
  }
  return cudaGetLastError() == cudaSuccess ? SS_OK : SS_ERR_CUDA;
}

struct StoreColumns {  // [dscale | dbias]
  float *ds, *db;
  int C, add;
  __device__ __forceinline__ void put(long long i, float v) const {
    float* at = i < C ? ds + i : db + (i - C);
    *at = (add & (i < C ? 1 : 2)) ? *at + v : v;
  }
};

template <typename T, bool SILU>
int bwd(const GnPlan& pl, const T* dy, const T* x, const float* scale, const float* bias, const float* mean, const float* rstd, float* dx,
        float* dscale, float* dbias, int accumulate, void* ws, cudaStream_t s) {
  const Gn& p = pl.p;
  float* part = static_cast<float*>(ws);
  const StoreColumns st{dscale, dbias, p.C, accumulate};
  if (pl.form == kLanes) {
    GN_LANES(bwd_lanes, pl, dy, x, scale, bias, mean, rstd, dx, part, s)
  } else if (pl.form == kSample) {
    const size_t smem = 2 * pl.items * kGnThreads * sizeof(typename Raw8<T>::V) + (gn_part_floats(p) + 2 * p.C + 2 * p.groups) * sizeof(float);
    const auto kernel = gn_bwd_sample_kernel<T, SILU>;
    if (!allow_smem(kernel)) return SS_ERR_CUDA;
    kernel<<<pl.grid, kGnThreads, smem, s>>>(p, pl.items, dy, x, scale, bias, mean, rstd, dx, part);
  } else {
    const Part& q = pl.q;
    float2* means = reinterpret_cast<float2*>(part + (size_t)p.N * q.splits * 2 * p.C);
    const unsigned grid = (unsigned)((long long)p.N * q.splits * q.tiles);
    gn_bwd_sums_kernel<T, SILU><<<grid, kGnThreads, 0, s>>>(p, q, dy, x, scale, bias, mean, rstd, part);
    if (launch_dependent(gn_bwd_join_kernel, dim3((unsigned)((long long)p.N * p.groups)), dim3(kGnThreads), 0, s, p, q, (const float*)part, scale,
                         means) != cudaSuccess ||
        launch_dependent(gn_bwd_apply_kernel<T, SILU>, dim3(grid), dim3(kGnThreads), 0, s, p, q, dy, x, scale, bias, mean, rstd,
                         (const float2*)means, dx) != cudaSuccess)
      return SS_ERR_CUDA;
  }
  if (cudaGetLastError() != cudaSuccess) return SS_ERR_CUDA;
  return colsum(part, 2ll * p.C, pl.rows, st, s) == cudaSuccess ? SS_OK : SS_ERR_CUDA;
}

}  // namespace

extern "C" size_t groupnorm_fwd_workspace_size(int N, int M, int C, int groups, int dtype) {
  GnPlan pl;
  return gn_plan(N, M, C, groups, dtype, pl) == SS_OK ? pl.fwd : 0;
}

extern "C" int groupnorm_fwd(const void* x, const float* scale, const float* bias, float eps, void* y, float* mean, float* rstd, int N, int M,
                             int C, int groups, int silu, int dtype, void* workspace, size_t ws_bytes, void* stream) {
  if (!x || !scale || !y) return SS_ERR_NULL;
  GnPlan pl;
  const int rc = gn_plan(N, M, C, groups, dtype, pl);
  if (rc != SS_OK) return rc;
  if (!(eps >= 0.f)) return SS_ERR_DIM;
  const void* ptrs[] = {x, scale, bias, y};
  for (const void* q : ptrs)
    if (!ssh::aligned16(q)) return SS_ERR_ALIGN;
  if ((reinterpret_cast<uintptr_t>(mean) & 3u) || (reinterpret_cast<uintptr_t>(rstd) & 3u)) return SS_ERR_ALIGN;
  if (pl.fwd > 0) {
    if (workspace == nullptr || ws_bytes < pl.fwd) return SS_ERR_WORKSPACE;
    if (!ssh::aligned16(workspace)) return SS_ERR_ALIGN;
  }
  pl.p.eps = eps;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  auto go = [&](auto* t) {
    using T = std::remove_pointer_t<decltype(t)>;
    const T* xt = static_cast<const T*>(x);
    return silu ? fwd<T, true>(pl, xt, scale, bias, static_cast<T*>(y), mean, rstd, workspace, s)
                : fwd<T, false>(pl, xt, scale, bias, static_cast<T*>(y), mean, rstd, workspace, s);
  };
  return dtype == SS_F32 ? go(static_cast<float*>(nullptr)) : go(static_cast<__nv_bfloat16*>(nullptr));
}

extern "C" size_t groupnorm_bwd_workspace_size(int N, int M, int C, int groups, int dtype) {
  GnPlan pl;
  return gn_plan(N, M, C, groups, dtype, pl) == SS_OK ? pl.bwd : 0;
}

extern "C" int groupnorm_bwd(const void* dy, const void* x, const float* scale, const float* bias, const float* mean, const float* rstd, float* dx,
                             float* dscale, float* dbias, int accumulate, int N, int M, int C, int groups, int silu, int dtype, void* workspace,
                             size_t ws_bytes, void* stream) {
  if (!dy || !x || !scale || !mean || !rstd || !dx || !dscale || !dbias) return SS_ERR_NULL;
  GnPlan pl;
  const int rc = gn_plan(N, M, C, groups, dtype, pl);
  if (rc != SS_OK) return rc;
  const void* ptrs[] = {dy, x, scale, bias, dx};
  for (const void* q : ptrs)
    if (!ssh::aligned16(q)) return SS_ERR_ALIGN;
  const void* words[] = {mean, rstd, dscale, dbias};
  for (const void* q : words)
    if (reinterpret_cast<uintptr_t>(q) & 3u) return SS_ERR_ALIGN;
  if (workspace == nullptr || ws_bytes < pl.bwd) return SS_ERR_WORKSPACE;
  if (!ssh::aligned16(workspace)) return SS_ERR_ALIGN;
  pl.p.eps = 0.f;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  auto go = [&](auto* t) {
    using T = std::remove_pointer_t<decltype(t)>;
    const T *yt = static_cast<const T*>(dy), *xt = static_cast<const T*>(x);
    return silu ? bwd<T, true>(pl, yt, xt, scale, bias, mean, rstd, dx, dscale, dbias, accumulate, workspace, s)
                : bwd<T, false>(pl, yt, xt, scale, bias, mean, rstd, dx, dscale, dbias, accumulate, workspace, s);
  };
  return dtype == SS_F32 ? go(static_cast<float*>(nullptr)) : go(static_cast<__nv_bfloat16*>(nullptr));
}
