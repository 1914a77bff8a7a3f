// Tensor-core pieces of the bf16 linear attention kernels: shared-memory tiles
// in the 128-byte-swizzled layout that tcgen05.mma reads, their descriptors, and
// tensor-memory access.
//
// A tile of R rows x W columns of bf16 is W / 64 panels of R rows of 128 bytes;
// 16-byte unit u of row r lies at unit u ^ (r & 7) of its row.  One tile serves
// as an operand whose contraction runs along its columns ("rows" below: M or N
// are its rows) and as one whose contraction runs down its rows ("cols": M or N
// are its columns), so q, k, v and do are loaded once for all their products.
#pragma once

#include "linattn_common.cuh"

namespace ssk {

constexpr int kTC = kLinChunkBf16;        // tokens of a chunk = rows of a tile
constexpr int kPanel = kTC * 128;         // bytes of a panel of kTC rows
constexpr int kLinWarps = 16, kLinThreads = 32 * (kLinWarps + 2);  // computing warps, one that issues, one for the decays

// byte offset of 16-byte unit `u` (8 columns) of row r in a tile of kTC rows
__device__ __forceinline__ uint32_t tile_at(int r, int u) {
  return (uint32_t)((u >> 3) * kPanel + r * 128 + (((u & 7) ^ (r & 7)) << 4));
}

// The decays of a chunk in shared memory, each token's c_i relative to the end of
// the 32 tokens before its own 32 (base): r_i = c_i - base as a float and, in
// bf16, what that leaves.  Against tokens of one block of 32 a score's decay is
// 2^(x - r_j) with x = c_i - base taken once, good to 2^-24 |r_j|.
struct DecTile {
  static constexpr int bytes = kTC * 6 + 32;
  uint32_t at;
  __device__ __forceinline__ static float ldf(uint32_t a) {
    float x;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(x) : "r"(a));
    return x;
  }
  __device__ __forceinline__ void put(int i, Dec r) const {
    asm volatile("st.shared.f32 [%0], %1;" ::"r"(at + 4 * i), "f"(r.hi) : "memory");
    const __nv_bfloat16 l = __float2bfloat16_rn(r.lo);
    asm volatile("st.shared.b16 [%0], %1;" ::"r"(at + 4 * kTC + 2 * i), "h"(*reinterpret_cast<const uint16_t*>(&l)) : "memory");
  }
  __device__ __forceinline__ void put_base(int n, Dec b) const {
    asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(at + 6 * kTC + 8 * n), "f"(b.hi), "f"(b.lo) : "memory");
  }
  __device__ __forceinline__ Dec base(int n) const {
    Dec b;
    asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(b.hi), "=f"(b.lo) : "r"(at + 6 * kTC + 8 * n));
    return b;
  }
  __device__ __forceinline__ Dec rel(int i) const {
    Dec d;
    uint16_t l;
    d.hi = ldf(at + 4 * i);
    asm volatile("ld.shared.b16 %0, [%1];" : "=h"(l) : "r"(at + 4 * kTC + 2 * i));
    d.lo = __uint_as_float((uint32_t)l << 16);
    return d;
  }
  __device__ __forceinline__ Dec get(int i) const { return dec_add(base(i >> 5), rel(i)); }
  // r of tokens j .. j + 3 (j a multiple of 4)
  __device__ __forceinline__ float4 r4(int j) const {
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(at + 4 * j));
    return v;
  }
  // both parts of them
  __device__ __forceinline__ void rel4(int j, float (&hi)[4], float (&lo)[4]) const {
    const float4 v = r4(j);
    uint32_t a, b;
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(a), "=r"(b) : "r"(at + 4 * kTC + 2 * j));
    hi[0] = v.x; hi[1] = v.y; hi[2] = v.z; hi[3] = v.w;
    lo[0] = bf16_lo(a); lo[1] = bf16_hi(a); lo[2] = bf16_lo(b); lo[3] = bf16_hi(b);
  }
};
__device__ __forceinline__ Dec dec_sub(Dec a, Dec b) { return dec_add(a, Dec{-b.hi, -b.lo}); }
__device__ __forceinline__ float dec_exp(Dec d) { return dec_exp(d.hi, d.lo); }

// A chunk's decays, in one warp: the gates are read ahead, scan() finds the sums
// in registers, put() stores them once the tile's readers are done.
struct DecStage {
  ChunkGates<kTC> g;
  Dec rel[ChunkGates<kTC>::PER], base;
  __device__ __forceinline__ void scan(int lane) { base = g.scan_rel(lane, rel); }
  __device__ __forceinline__ void put(const DecTile& t, int lane) const {
#pragma unroll
    for (int e = 0; e < ChunkGates<kTC>::PER; ++e) t.put(lane * ChunkGates<kTC>::PER + e, rel[e]);
    if (lane < kTC / 32) t.put_base(lane, base);
  }
};

// One 128-byte line into L2, ahead of the loads that will want it.
__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// ---------------------------------------------------------------- descriptors
// Shared-memory operand descriptor: start address, leading and stride byte
// offsets (all in 16-byte units), version 1, 128-byte swizzle; 8-row groups are
// 1024 bytes apart.  Only the low word changes from step to step of a product.
__device__ __forceinline__ uint64_t smem_desc(uint32_t lo) { return ((uint64_t)((1024u >> 4) | (1u << 14) | (2u << 29)) << 32) | lo; }
// contraction along the columns; step s takes columns 16 s .. 16 s + 15
__device__ __forceinline__ uint64_t desc_rows(uint32_t tile, int s) {
  return smem_desc((tile >> 4) + (s >> 2) * (kPanel >> 4) + (s & 3) * 2 + (1u << 16));
}
// contraction down the rows; step s takes rows 16 s .. 16 s + 15; 64-column panels kPanel apart
__device__ __forceinline__ uint64_t desc_cols(uint32_t tile, int s) {
  return smem_desc((tile >> 4) + s * 128 + ((uint32_t)(kPanel >> 4) << 16));
}

// bf16 x bf16 -> fp32, M = 128; a_cols / b_cols: that operand's contraction runs down its rows
__device__ __forceinline__ uint32_t mma_idesc(int n, bool a_cols, bool b_cols) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((a_cols ? 1u : 0u) << 15) | ((b_cols ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) |
         ((128u >> 4) << 24);
}

// True in one thread of a converged warp.  What that thread then issues takes its
// operands from the warp's uniform registers; behind a test of the lane's number
// the compiler cannot know that one thread is left: an MMA took 100 cycles to
// issue, and operands came to hold other lanes' values.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.b32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

// D (tensor memory) = A B (+ D); one thread issues
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
      : "memory");
}
// the same with A (128 rows, bf16 pairs in columns) in tensor memory
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
      : "memory");
}
// A product of n steps of 16 (n <= 8), unrolled, so that a step costs its issuing thread a few instructions:
// the operands' descriptors as functions of the step
template <typename A, typename B>
__device__ __forceinline__ void mma_steps(uint32_t d, A a, B b, uint32_t idesc, int n, bool add) {
#pragma unroll
  for (int s = 0; s < 8; ++s)
    if (s < n) mma_ss(d, a(s), b(s), idesc, add || s > 0);
}
struct Rows {  // an operand whose contraction runs along the tile's columns
  uint32_t tile;
  __device__ __forceinline__ uint64_t operator()(int s) const { return desc_rows(tile, s); }
};
struct Cols {  // ... down its rows
  uint32_t tile;
  __device__ __forceinline__ uint64_t operator()(int s) const { return desc_cols(tile, s); }
};
// the barrier completes when all MMAs issued before are done
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
               : "r"(taddr)
               : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};" ::"r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(taddr)
               : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
               : "r"(taddr)
               : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};" ::"r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(taddr)
               : "memory");
}
__device__ __forceinline__ void tmem_ld8u(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr)
               : "memory");
}
__device__ __forceinline__ void tmem_st8u(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::"r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(taddr)
               : "memory");
}
__device__ __forceinline__ void tmem_ldn(uint32_t taddr, uint32_t (&r)[32]) { tmem_ld32(taddr, r); }
__device__ __forceinline__ void tmem_ldn(uint32_t taddr, uint32_t (&r)[16]) { tmem_ld16(taddr, r); }
__device__ __forceinline__ void tmem_ldn(uint32_t taddr, uint32_t (&r)[8]) { tmem_ld8u(taddr, r); }
__device__ __forceinline__ void tmem_stn(uint32_t taddr, const uint32_t (&r)[8]) { tmem_st8u(taddr, r); }
__device__ __forceinline__ void tmem_stn(uint32_t taddr, const uint32_t (&r)[32]) { tmem_st32(taddr, r); }
__device__ __forceinline__ void tmem_stn(uint32_t taddr, const uint32_t (&r)[16]) { tmem_st16(taddr, r); }
// N columns of this thread's lane times f, in place (the caller waits for the store)
template <int N>
__device__ __forceinline__ void tmem_scale(uint32_t taddr, float f) {
  uint32_t r[N];
  tmem_ldn(taddr, r);
  tmem_wait_ld();
#pragma unroll
  for (int e = 0; e < N; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * f);
  tmem_stn(taddr, r);
}

// ---------------------------------------------------------------- tiles

// [B, L, heads, width] bf16 with `ld` elements from token to token, as boxes of one panel (64 columns of one head
// x kTC tokens); columns past `width` and tokens past L read as zero
inline bool lin_map(CUtensorMap* m, const void* base, long long ld, int B, int L, int heads, int width) {
  const uint64_t dims[4] = {(uint64_t)width, (uint64_t)heads, (uint64_t)L, (uint64_t)B};
  const uint64_t strides[3] = {(uint64_t)width * 2, (uint64_t)ld * 2, (uint64_t)ld * 2 * (uint64_t)L};
  const uint32_t box[4] = {64, 1, (uint32_t)kTC, 1};
  return ssh::encode_tiled(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, base, dims, strides, box, true);
}
// the panels of a tile of `n` panels
__device__ __forceinline__ void load_panels(uint32_t tile, int n, const CUtensorMap* m, uint64_t* bar, int c, int head, int t0, int b) {
  for (int i = 0; i < n; ++i) tma_load_4d(tile + i * kPanel, m, bar, c + i * 64, head, t0, b);
}
__device__ __forceinline__ void prefetch_panels(int n, const CUtensorMap* m, int c, int head, int t0, int b) {
  for (int i = 0; i < n; ++i) tma_prefetch_4d(m, c + i * 64, head, t0, b);
}
// rows from `valid` on of `panels` panels become zero (one warp): a row that ends inside the tensor
__device__ __forceinline__ void zero_rows(uint32_t tile, int panels, int valid, int lane) {
  for (int n = 0; n < panels; ++n)
    for (int r = valid + (lane >> 3); r < kTC; r += 4)
      asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(tile + n * kPanel + r * 128 + (lane & 7) * 16), "r"(0) : "memory");
}

__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ void sts16(uint32_t a, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) { return ActT<__nv_bfloat16>::pack2(lo, hi); }

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
}

// A warp's part of a tile (32 rows from r0, NU 16-byte units from u0) to units
// from `to` of rows in global memory, up to `rows` rows and `width` columns.  A
// lane's accumulators are one row, so storing them as they are would touch 32
// rows with each instruction; through the tile four lanes share a row (the
// backward's three outputs took 9000 cycles a chunk, so 5500).
template <int NU>  // NU units of each row: 4 or 2
__device__ __forceinline__ void store_rows(uint32_t tile, __nv_bfloat16* __restrict__ dst, long long ld, int r0, int u0, int to, int rows,
                                           int width, int lane) {
#pragma unroll
  for (int i = 0; i < NU; ++i) {
    const int r = r0 + i * (32 / NU) + lane / NU, u = lane % NU;
    if (r < rows && (to + u) * 8 < width) *reinterpret_cast<uint4*>(dst + (long long)r * ld + (to + u) * 8) = lds16(tile + tile_at(r, u0 + u));
  }
}

// An fp32 value as a sum of three bf16 terms: the first is off by 2^-8 of the
// value at most, the first two by 2^-16, all three by 2^-24, the half-step of
// fp32 itself, so that a product of the terms with an exact bf16 operand is an
// fp32 product.  This takes term n of eight values and leaves what is left.
__device__ __forceinline__ uint4 take_term(float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    w[e] = pack_bf16(x[2 * e], x[2 * e + 1]);
    x[2 * e] -= bf16_lo(w[e]);
    x[2 * e + 1] -= bf16_hi(w[e]);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ uint4 last_term(const float (&x)[8]) { return pack8(x); }

}  // namespace ssk

namespace {

using namespace ssk;

__device__ unsigned g_lin_err;  // this translation unit's error word: a wait for its own MMAs ran out

inline int read_clear_lin_err(cudaStream_t s, unsigned* out) {
  return ssk::read_clear_word(g_lin_err, s, out);
}

// A whole warp waits for a phase of a barrier, and leaves together: tensor-memory
// accesses want the warp converged, and a warp's uniform registers (an MMA's
// descriptors, a copy's coordinates) are not a lane's own, so no lane may run on
// while another issues; every block that one lane issues ends with __syncwarp().
__device__ __forceinline__ bool lin_wait(uint64_t* bar, uint32_t par) {
  return __all_sync(0xffffffffu, mbar_wait_bounded(bar, par, kWaitLimitNs));
}

// The end of a kernel of kLinThreads: a wait that ran out is told (the outputs
// are invalid) and whatever is still in flight gets a limited wait, then the
// tensor memory is returned.
__device__ __forceinline__ void lin_leave(bool ok, uint64_t* bar, int nbar, uint32_t tm, uint32_t cols, int warp, int lane) {
  if (!ok && lane == 0) atomicOr(&g_lin_err, kErrTmaTimeout);
  tc_fence_before_sync();
  if (__syncthreads_or(!ok) && warp == 0) {
    for (int i = 0; i < nbar; ++i)
      for (uint32_t ph = 0; ph < 2; ++ph) mbar_wait_bounded(&bar[i], ph, 20000000ull);
  }
  if (warp == 0) tmem_dealloc(tm, cols);
}

// ---------------------------------------------------------------- a segment's state
// The state a segment reaches from zero and its log decay, for both directions:
//   forward   S = e^{c_last} S + sum_j k_j (e^{c_last-c_j} v_j)^T      chunks in order
//   REV       U = e^{c_last} U + sum_i q_i (scale e^{c_i} do_i)^T      chunks from the last
// A CTA takes 64 columns of y (v or do).  The weighted rows of y, as three bf16
// terms side by side, are one product of 192 columns, so that x is read once;
// every tile has two places, and a chunk's weights are under the product before.
struct SumTc {
  static constexpr int x = 0, y = x + 4 * kPanel, w = y + 2 * kPanel, dec = w + 6 * kPanel, bar = dec + 2 * ((DecTile::bytes + 15) / 16 * 16);
  // barriers, two each: tiles landed, decays stored, product done, terms stored
  static constexpr int kLd = 0, kDc = 2, kM = 4, kW = 6, nbar = 8;
  static constexpr int tm = bar + nbar * 8, bytes = tm + 8, cols = 512;
};

template <bool REV>
__global__ void __launch_bounds__(kLinThreads, 1) linattn_sum_tc_kernel(LinAttn p, const __grid_constant__ CUtensorMap mx,
                                                                        const __grid_constant__ CUtensorMap my,
                                                                        float* __restrict__ send, Dec* __restrict__ sdec) {
  using L = SumTc;
  extern __shared__ __align__(1024) unsigned char raw[];
  const uint32_t sb = smem_u32(raw);
  uint64_t* bar = reinterpret_cast<uint64_t*>(raw + L::bar);
  uint32_t* tma = reinterpret_cast<uint32_t*>(raw + L::tm);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int nvt = (p.V + 63) / 64;
  long long id = blockIdx.x;
  const int seg = (int)(id % p.nseg);
  id /= p.nseg;
  const int vt = (int)(id % nvt);
  id /= nvt;
  const int h = (int)(id % p.H), b = (int)(id / p.H), gh = h / (p.H / p.G), v0 = vt * 64, vw = p.V - v0 < 64 ? p.V - v0 : 64;
  const int len = p.len(b);
  const long long bh = (long long)b * p.H + h;
  const int c0 = seg * p.cps, c1 = c0 + p.cps < p.nck ? c0 + p.cps : p.nck;
  int cend = (len + kTC - 1) / kTC;
  cend = cend < c0 ? c0 : cend < c1 ? cend : c1;
  const int n = cend - c0;
  auto chunk = [&](int i) { return REV ? cend - 1 - i : c0 + i; };  // the i-th chunk walked
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
  // barrier pair `i` for its place's turn m: the places take turns, so place m & 1 is at phase (m >> 1) & 1
  auto wait = [&](int i, int m) { return ok = lin_wait(&bar[i + (m & 1)], (uint32_t)(m >> 1) & 1u); };

  if (warp == kLinWarps) {  // ---- the issuing warp
    auto load = [&](int i) {
      if (elect_one()) {
        uint64_t* bl = &bar[L::kLd + (i & 1)];
        mbar_arrive_expect_tx(bl, 3 * kPanel);
        load_panels(sb + L::x + (i & 1) * 2 * kPanel, 2, &mx, bl, 0, gh, chunk(i) * kTC, b);
        load_panels(sb + L::y + (i & 1) * kPanel, 1, &my, bl, v0, h, chunk(i) * kTC, b);
      }
      __syncwarp();
    };
    if (n > 0) load(0);
    if (n > 1) load(1);
    for (int i = 0; i < n; ++i) {
      const uint32_t x = sb + L::x + (i & 1) * 2 * kPanel;
      if (!wait(L::kLd, i)) break;
      const int valid = len - chunk(i) * kTC;
      if (valid < kTC && chunk(i) * kTC + valid < p.L) {  // the row ends inside the tensor (y's readers take dead rows as zero)
        zero_rows(x, 2, valid, lane);
        fence_proxy_async_smem();
        __syncwarp();
      }
      if (!wait(L::kW, i)) break;
      if (elect_one()) {
        tc_fence_after_sync();
        mma_steps(tm + (i & 1) * 256, Cols{x}, Cols{sb + L::w + (i & 1) * 3 * kPanel}, mma_idesc(192, true, true), kTC / 16, false);
        mma_commit(&bar[L::kM + (i & 1)]);
      }
      __syncwarp();
      if (i + 2 < n) {
        if (!wait(L::kM, i)) break;
        load(i + 2);
      }
    }
  } else if (warp > kLinWarps) {  // ---- the decays' warp
    DecStage ds;
    Dec total = {0.f, 0.f};
    if (n > 0) ds.g.fetch(p, b, h, chunk(0) * kTC, len, lane);
    for (int i = 0; i < n; ++i) {
      ds.scan(lane);
      if (i + 1 < n) ds.g.fetch(p, b, h, chunk(i + 1) * kTC, len, lane);
      if (i > 1 && !wait(L::kM, i - 2)) break;  // its readers had stored their terms
      const DecTile dec{sb + L::dec + (i & 1) * ((DecTile::bytes + 15) / 16 * 16)};
      ds.put(dec, lane);
      __syncwarp();
      total = dec_add(total, dec.get(kTC - 1));
      if (lane == 0) mbar_arrive(&bar[L::kDc + (i & 1)]);
    }
    if (lane == 0 && vt == 0) sdec[bh * p.nseg + seg] = total;
  } else {  // ---- a computing warp
    const int row = (warp & 3) * 32 + lane, cq = warp >> 2;
    const uint32_t tl = tm + ((uint32_t)((warp & 3) * 32) << 16);
    float S[16], elast = 0.f;
#pragma unroll
    for (int e = 0; e < 16; ++e) S[e] = 0.f;
    auto add = [&](int i, float f) {  // S = f S + the product of chunk i
      uint32_t a[16], c[16], d[16];
      tmem_ld16(tl + (i & 1) * 256 + cq * 16, a);
      tmem_ld16(tl + (i & 1) * 256 + 64 + cq * 16, c);
      tmem_ld16(tl + (i & 1) * 256 + 128 + cq * 16, d);
      tmem_wait_ld();
#pragma unroll
      for (int e = 0; e < 16; ++e)
        S[e] = fmaf(S[e], f, __uint_as_float(a[e]) + (__uint_as_float(c[e]) + __uint_as_float(d[e])));
    };
    for (int i = 0; i < n; ++i) {
      if (!wait(L::kDc, i) || !wait(L::kLd, i)) break;
      const DecTile dec{sb + L::dec + (i & 1) * ((DecTile::bytes + 15) / 16 * 16)};
      const Dec last = dec.get(kTC - 1), own = dec.get(row);
      const float w = REV ? p.scale * dec_exp(own) : dec_exp(dec_sub(last, own));
      const bool live = row < len - chunk(i) * kTC;
      const uint32_t wt = sb + L::w + (i & 1) * 3 * kPanel;  // read by product i - 2, whose sum has been taken
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const uint32_t at = tile_at(row, cq * 2 + u);
        float x[8];
        Raw8<__nv_bfloat16>::wide(live ? lds16(sb + L::y + (i & 1) * kPanel + at) : make_uint4(0u, 0u, 0u, 0u), x);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] *= w;
        sts16(wt + at, take_term(x));
        sts16(wt + kPanel + at, take_term(x));
        sts16(wt + 2 * kPanel + at, last_term(x));
      }
      fence_proxy_async_smem();
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar[L::kW + (i & 1)]);
      if (i > 0) {  // the product before, under this one
        if (!wait(L::kM, i - 1)) break;
        tc_fence_after_sync();
        add(i - 1, elast);
      }
      elast = dec_exp(last);
    }
    if (ok && n > 0 && wait(L::kM, n - 1)) {
      tc_fence_after_sync();
      add(n - 1, elast);
    }
    if (row < p.K) {
      float* dst = send + ((bh * p.nseg + seg) * p.K + row) * p.V + v0 + cq * 16;
#pragma unroll
      for (int e = 0; e < 16; e += 4)
        if (cq * 16 + e < vw) *reinterpret_cast<float4*>(dst + e) = make_float4(S[e], S[e + 1], S[e + 2], S[e + 3]);
    }
  }
  lin_leave(ok, bar, L::nbar, tm, L::cols, warp, lane);
}

// In place over the segments of a (batch row, head), in walking order: the
// states found from zero become the states the segments start from,
// s[next] = 2^{dec} s + end.
template <bool REV>
__global__ void __launch_bounds__(256) linattn_join_kernel(const float* __restrict__ first, float* __restrict__ st,
                                                           const Dec* __restrict__ dec, long long kv, int nseg) {
  const long long bh = blockIdx.y;
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  if (i >= kv) return;
  float s = first != nullptr ? first[bh * kv + i] : 0.f;
  constexpr int U = 8;  // end states in flight
  for (int m = 0; m < nseg; m += U) {
    float end[U];
    Dec d[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (m + u >= nseg) break;
      const int n = REV ? nseg - 1 - m - u : m + u;
      end[u] = st[(bh * nseg + n) * kv + i];
      d[u] = dec[bh * nseg + n];
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (m + u >= nseg) break;
      const int n = REV ? nseg - 1 - m - u : m + u;
      st[(bh * nseg + n) * kv + i] = s;
      s = fmaf(dec_exp(d[u]), s, end[u]);
    }
  }
}

}  // namespace
