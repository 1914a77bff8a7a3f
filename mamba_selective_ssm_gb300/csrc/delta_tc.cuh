// Tensor-core pieces of the gated delta rule's bf16 kernels, on top of those of linear attention (linattn_tc.cuh).
//
// Products run transposed, columns of V as the 128 rows of an MMA, so that a head's state lies in the tensor memory's lanes
// and every step of the chain (K S0, M (beta R), K^T u) hands its result on along a lane.  Tiles of tokens are 64 rows of
// 128-byte panels.  bf16 inputs are operands as they are in memory; an fp32 operand is three bf16 terms that together are the
// value (8 + 8 + 8 bits, each the leading ones of what is left), a product of two such operands the six products of terms
// that reach 2^-16 of the largest.
#pragma once

#include "delta_common.cuh"
#include "linattn_tc.cuh"

namespace ssk {

constexpr int kTok = kDC * 128;       // bytes of a panel of 64 tokens (64 columns)
constexpr int kDTerm = kDC * kDC * 2;  // bytes of a 64 x 64 operand

// 16-byte unit u (8 columns) of row r in a tile whose panels have `panel` bytes
__device__ __forceinline__ uint32_t unit_at(int panel, int r, int u) {
  return (uint32_t)((u >> 3) * panel + r * 128 + (((u & 7) ^ (r & 7)) << 4));
}
// contraction along the columns (16 from 16 s), rows of the product from row r0 (a multiple of 8) on
__device__ __forceinline__ uint64_t rows_desc(uint32_t tile, int panel, int s, int r0 = 0) {
  return smem_desc(((tile + r0 * 128) >> 4) + (s >> 2) * (panel >> 4) + (s & 3) * 2 + (1u << 16));
}
// contraction down the rows (16 from 16 s), all 64-column panels
__device__ __forceinline__ uint64_t cols_desc(uint32_t tile, int panel, int s) {
  return smem_desc((tile >> 4) + s * 128 + ((uint32_t)(panel >> 4) << 16));
}

// A whole warp waits for a phase of a barrier and leaves together, as lin_wait does, with two differences that a chain of
// short waits asks for: a warp sleeps in the barrier for up to 20 us instead of asking again, since sixteen that ask use the
// shared memory that the MMAs read, and the timer, whose reading takes longer than most of the waits, is read after 4096
// rounds only (then the limit is the same).
__device__ __forceinline__ bool chain_wait(uint64_t* bar, uint32_t parity) {
  const uint32_t addr = smem_u32(bar);
  uint64_t t0 = 0;
  bool done = false;
  for (uint32_t it = 1;; ++it) {
    uint32_t got;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(got)
        : "r"(addr), "r"(parity), "r"(20000u)
        : "memory");
    if (got) {
      done = true;
      break;
    }
    if ((it & 4095u) == 0) {
      const uint64_t now = globaltimer_ns();
      if (t0 == 0) t0 = now;
      else if (now - t0 > kWaitLimitNs) break;
    }
  }
  return __all_sync(0xffffffffu, done);
}

__device__ __forceinline__ void tmem_done(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]),
                 "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}
__device__ __forceinline__ void tmem_done(uint32_t (&r)[8]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7])
               :
               : "memory");
}

__device__ __forceinline__ void tmem_st4(uint32_t taddr, const uint32_t (&r)[4]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%4], {%0, %1, %2, %3};" ::"r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(taddr) : "memory");
}

// The leading bf16 of a pair, packed; the pair becomes what is left (exactly).  (The half that moves up does so by a
// multiplication: these kernels keep the integer pipe busier than the fp32 one.)
__device__ __forceinline__ uint32_t take_pair(float2& x) {
  const uint32_t w = __byte_perm(__float_as_uint(x.x), __float_as_uint(x.y), 0x7632);
  x = fma2(f2(bf16_lo(w), bf16_hi(w)), bc2(-1.f), x);
  return w;
}
// The nearest bf16 of a pair, packed; the pair becomes what is left.  Of two terms the first is this one: what is left is half as much
// and of either sign, so that the pair is off by 2^-16 at most where a cut one is by 2^-15, and the product of two second terms,
// which is dropped, is 2^-16 of any sign for 2^-14 of one sign (dq and dk were 1.6e-4 and 2e-4 of their size from the rounded
// fp32 result).
__device__ __forceinline__ uint32_t round_pair(float2& x) {
  const uint32_t w = pack_bf16(x.x, x.y);
  x = fma2(f2(bf16_lo(w), bf16_hi(w)), bc2(-1.f), x);
  return w;
}
__device__ __forceinline__ uint32_t last_pair(float2 x) { return __byte_perm(__float_as_uint(x.x), __float_as_uint(x.y), 0x7632); }
// eight values as NT terms to 16-byte units `step` bytes apart.  Three cut terms are the value (what is left after two has
// eight bits); two are rounded.
template <int NT>
__device__ __forceinline__ void put_terms(uint32_t at, int step, float2 (&x)[4]) {
  static_assert(NT == 2 || NT == 3, "two terms or three");
  if constexpr (NT == 3) {
#pragma unroll
    for (int n = 0; n < 2; ++n) sts16(at + n * step, make_uint4(take_pair(x[0]), take_pair(x[1]), take_pair(x[2]), take_pair(x[3])));
    sts16(at + 2 * step, make_uint4(last_pair(x[0]), last_pair(x[1]), last_pair(x[2]), last_pair(x[3])));
  } else {
    sts16(at, make_uint4(round_pair(x[0]), round_pair(x[1]), round_pair(x[2]), round_pair(x[3])));
    sts16(at + step, make_uint4(pack_bf16(x[0].x, x[0].y), pack_bf16(x[1].x, x[1].y), pack_bf16(x[2].x, x[2].y), pack_bf16(x[3].x, x[3].y)));
  }
}
__device__ __forceinline__ float2 u2f(uint32_t a, uint32_t b) { return f2(__uint_as_float(a), __uint_as_float(b)); }

// A tile of tokens read or written along a column (a thread's column of V, a bf16 at a time): token t of the column whose
// token 0 is at `at` (t0 a multiple of 8 is added in bytes) lies at (at ^ ((t & 7) << 4)) + 128 t.
__device__ __forceinline__ uint32_t col_at(uint32_t tile, int c) { return tile + (uint32_t)((c >> 6) * kTok + (((c >> 3) & 7) << 4) + (c & 7) * 2); }
template <int T>
__device__ __forceinline__ float col_get(uint32_t at) {
  uint16_t x;
  asm volatile("ld.shared.u16 %0, [%1+%2];" : "=h"(x) : "r"(at ^ ((T & 7) << 4)), "n"(T * 128) : "memory");
  return bf16_lo(x);
}
template <int T>
__device__ __forceinline__ void col_put2(uint32_t at, float2 v) {  // tokens T and T + 1
  const uint32_t w = pack_bf16(v.x, v.y);
  asm volatile("st.shared.b16 [%0+%1], %2;" ::"r"(at ^ ((T & 7) << 4)), "n"(T * 128), "h"((uint16_t)w) : "memory");
  asm volatile("st.shared.b16 [%0+%1], %2;" ::"r"(at ^ (((T + 1) & 7) << 4)), "n"((T + 1) * 128), "h"((uint16_t)(w >> 16)) : "memory");
}
template <int N>
struct ColRead {
  __device__ __forceinline__ static void go(uint32_t at, float2* x) {
    ColRead<N - 2>::go(at, x);
    x[N / 2 - 1] = f2(col_get<N - 2>(at), col_get<N - 1>(at));
  }
};
template <>
struct ColRead<0> {
  __device__ __forceinline__ static void go(uint32_t, float2*) {}
};
template <int N>
struct ColWrite {
  __device__ __forceinline__ static void go(uint32_t at, const float2* x) {
    ColWrite<N - 2>::go(at, x);
    col_put2<N - 2>(at, x[N / 2 - 1]);
  }
};
template <>
struct ColWrite<0> {
  __device__ __forceinline__ static void go(uint32_t, const float2*) {}
};
// pairs of scalars of neighbouring tokens
__device__ __forceinline__ void pairs4(const float* p, float2 (&x)[4]) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  x[0] = f2(a.x, a.y); x[1] = f2(a.z, a.w); x[2] = f2(b.x, b.y); x[3] = f2(b.z, b.w);
}

// [B, L, heads, width] bf16 as boxes of one panel: 64 columns of one head x 64 tokens
inline bool delta_map(CUtensorMap* m, const void* base, long long ld, int B, int L, int heads, int width) {
  const uint64_t dims[4] = {(uint64_t)width, (uint64_t)heads, (uint64_t)L, (uint64_t)B};
  const uint64_t strides[3] = {(uint64_t)width * 2, (uint64_t)ld * 2, (uint64_t)ld * 2 * (uint64_t)L};
  const uint32_t box[4] = {64, 1, (uint32_t)kDC, 1};
  return ssh::encode_tiled(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, base, dims, strides, box, true);
}
__device__ __forceinline__ void tok_load(uint32_t tile, int panels, const CUtensorMap* m, uint64_t* bar, int head, int t0, int b) {
  for (int i = 0; i < panels; ++i) tma_load_4d(tile + i * kTok, m, bar, i * 64, head, t0, b);
}
// rows from `valid` on become zero (one warp): a row that ends inside the tensor
__device__ __forceinline__ void tok_clear(uint32_t tile, int panels, int valid, int lane) {
  for (int n = 0; n < panels; ++n)
    for (int r = valid + (lane >> 3); r < kDC; r += 4) sts16(tile + n * kTok + r * 128 + (lane & 7) * 16, make_uint4(0u, 0u, 0u, 0u));
}

}  // namespace ssk
