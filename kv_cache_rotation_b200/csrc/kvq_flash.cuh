// Pieces of the tiled attention kernels (sm_100a): the 5th-generation tensor
// core instructions and their descriptors, and the softmax of a 128 x 128
// score tile held in tensor memory.
//
// Tiles of 128 rows x 64 16-bit channels (16 KB, 128-byte rows, 128-byte
// swizzle: 16-byte chunk c of row r at r * 128 + ((c ^ (r & 7)) << 4)) are the
// unit of shared memory; a head of D channels is D / 64 of them. Read along
// the channels (the products q . k) such a tile is K-major, read along the
// rows (p . v) it is MN-major.
#pragma once

#include <cuda_bf16.h>

#include "kvq_device.cuh"

namespace kvq {

constexpr uint32_t kTileBytes = 128 * 128;  // 128 rows x 64 channels

// ---------------------------------------------------------------- tensor memory
__device__ __forceinline__ void tmem_alloc(uint32_t* dst, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst)), "r"(cols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc(uint32_t addr, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols) : "memory");
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// Products are issued by a whole warp in step, one elected lane doing it: with the warp together the
// descriptors stay in uniform registers. In a branch of one lane the same instruction took 74 to 124
// clocks to issue, whatever its size; so it takes 32 (N = 64) or 64 (N = 128), which is the tensor
// cores' own rate. The mbarrier is arrived on when all products issued so far by this warp are done.
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar))
      : "memory");
}
// A wait of a whole warp: every lane has the same answer.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, uint64_t limit_ns, uint32_t* err) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, limit_ns, err));
}

#define KVQ_R4(a, i) "=r"(a[i]), "=r"(a[i + 1]), "=r"(a[i + 2]), "=r"(a[i + 3])
#define KVQ_R32(a) \
  KVQ_R4(a, 0), KVQ_R4(a, 4), KVQ_R4(a, 8), KVQ_R4(a, 12), KVQ_R4(a, 16), KVQ_R4(a, 20), KVQ_R4(a, 24), KVQ_R4(a, 28)
#define KVQ_RW4(a, i) "+r"((a)[i]), "+r"((a)[i + 1]), "+r"((a)[i + 2]), "+r"((a)[i + 3])
#define KVQ_RW32(a) \
  KVQ_RW4(a, 0), KVQ_RW4(a, 4), KVQ_RW4(a, 8), KVQ_RW4(a, 12), KVQ_RW4(a, 16), KVQ_RW4(a, 20), KVQ_RW4(a, 24), KVQ_RW4(a, 28)
#define KVQ_I4(a, i) "r"(a[i]), "r"(a[i + 1]), "r"(a[i + 2]), "r"(a[i + 3])

// 32 columns of this warp's 32 lanes: register i of lane l is column col + i of lane l.
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
      "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : KVQ_R32(r)
      : "r"(addr));
}
// The loads so far are complete; the registers pass through, so no use of them moves above it.
__device__ __forceinline__ void tmem_wait_ld32(uint32_t* r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" : KVQ_RW32(r)::"memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
      "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(addr),
      KVQ_I4(r, 0), KVQ_I4(r, 4), KVQ_I4(r, 8), KVQ_I4(r, 12), KVQ_I4(r, 16), KVQ_I4(r, 20), KVQ_I4(r, 24), KVQ_I4(r, 28)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          addr),
      KVQ_I4(r, 0), KVQ_I4(r, 4), KVQ_I4(r, 8), KVQ_I4(r, 12)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Registers per thread of a warpgroup, every warp of which comes here.
template <int N>
__device__ __forceinline__ void more_regs() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void fewer_regs() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

// ---------------------------------------------------------------- products
// Shared-memory operand descriptor: start address, leading and stride byte
// offsets (in 16-byte units), version 1, 128-byte swizzle. K-major: groups of
// 8 rows are 1024 bytes apart. MN-major: the leading offset steps over 64
// channels, the stride over 8 rows.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lead, uint32_t stride) {
  return static_cast<uint64_t>((addr >> 4) & 0x3fff) | (static_cast<uint64_t>((lead >> 4) & 0x3fff) << 16) |
         (static_cast<uint64_t>((stride >> 4) & 0x3fff) << 32) | (1ull << 46) | (2ull << 61);
}
// Instruction descriptor: fp32 accumulators, A and B both fp16 (0) or both bf16
// (1), B MN-major if bt, M = 128.
__host__ __device__ constexpr uint32_t mma_desc(int type, bool bt, int n) {
  return (1u << 4) | (static_cast<uint32_t>(type) << 7) | (static_cast<uint32_t>(type) << 10) | (bt ? 1u << 16 : 0u) |
         (static_cast<uint32_t>(n >> 3) << 17) | ((128u >> 4) << 24);
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\tsetp.ne.u32 p, %4, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(acc))
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\tsetp.ne.u32 p, %4, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(acc))
      : "memory");
}

template <typename T>
struct Elem;
template <>
struct Elem<__half> {
  static constexpr int kType = 0;
  static constexpr uint32_t kInf = 0x7c00, kToTop = 0x04000400;  // |x| >= kInf: x + kToTop reaches the sign bit
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
  }
};
template <>
struct Elem<__nv_bfloat16> {
  static constexpr int kType = 1;
  static constexpr uint32_t kInf = 0x7f80, kToTop = 0x00800080;
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
  }
};

// D[128 x 128] = A . B^T over D channels: A and B K-major tiles (a, b: shared addresses).
template <typename T, int D>
__device__ __forceinline__ void issue_scores(uint32_t d, uint32_t a, uint32_t b) {
#pragma unroll
  for (int k = 0; k < D / 16; ++k) {
    const uint32_t off = (k / 4) * kTileBytes + (k % 4) * 32;
    mma_ss(d, smem_desc(a, 16, 1024) + (off >> 4), smem_desc(b, 16, 1024) + (off >> 4), mma_desc(Elem<T>::kType, false, 128), k > 0);
  }
}
// O[128 x D] (+)= P . V: P 128 x 128 16-bit in tensor memory, V 128 rows x D channels MN-major.
template <typename T, int D>
__device__ __forceinline__ void issue_values(uint32_t o, uint32_t p, uint32_t v, bool acc) {
#pragma unroll
  for (int k = 0; k < 8; ++k)
    mma_ts(o, p + 8 * k, smem_desc(v, kTileBytes, 1024) + (k * 2048 >> 4), mma_desc(Elem<T>::kType, true, D), acc || k > 0);
}

// ---------------------------------------------------------------- softmax of a tile
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Running statistics of a row in units of log2: p = 2^(s * mul - m). The
// reference m is raised only when a score exceeds it by 2^kRaise, so the sums
// are rescaled rarely; a weight is then at most 2^kRaise, far inside 16 bits.
constexpr float kRaise = 8.0f;
struct RowStat {
  float m = -INFINITY, l = 0.0f;
};

// Columns [0, left) of a tile as bits.
__device__ __forceinline__ uint32_t first_bits(int left, int at) {
  return left >= at + 32 ? 0xffffffffu : left <= at ? 0u : (1u << (left - at)) - 1u;
}

// One score tile of a row (a thread's lane of tensor memory at `s_addr`, 128
// fp32 columns), of which bit c of `seen` allows column c when MASKED: the weights
// go back to the same columns, 16-bit, two to a column, and the sums at
// `o_addr` (D fp32 columns, present when `have_o`) are rescaled if the
// reference rises. Warp-uniform: every lane of the warp calls it. Each weight
// is rounded once to T for the product (relative 2^-12 on average in fp16,
// 2^-9 in bf16, where a sum over many keys averages it out); the row sum takes
// the unrounded weights. The row's 128 scores stay in registers between the
// maximum and the weights: reading them twice, or two threads to a row, was
// slower (562 against 529 us for 16384 tokens of 8 / 2 heads of 128).
template <typename T, int D, bool MASKED>
__device__ __forceinline__ void softmax_tile(uint32_t s_addr, uint32_t o_addr, bool have_o, float mul, RowStat& st,
                                             const uint32_t (&seen)[4]) {
  uint32_t r[128];
  float mx = -INFINITY, mx2 = -INFINITY;
#pragma unroll
  for (int c = 0; c < 4; ++c) tmem_ld32(s_addr + 32 * c, r + 32 * c);
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    uint32_t* x = r + 32 * c;
    tmem_wait_ld32(x);
    if constexpr (MASKED) {
#pragma unroll
      for (int i = 0; i < 32; ++i) x[i] = (seen[c] >> i) & 1u ? x[i] : 0xff800000u;
    }
#pragma unroll
    for (int i = 0; i < 32; i += 4) {
      mx = max3f(mx, __uint_as_float(x[i]), __uint_as_float(x[i + 1]));
      mx2 = max3f(mx2, __uint_as_float(x[i + 2]), __uint_as_float(x[i + 3]));
    }
  }
  mx = fmaxf(mx, mx2) * mul;
  const bool raise = mx > st.m + kRaise;
  if (__any_sync(0xffffffffu, raise)) {
    const float f = raise ? exp2_fast(st.m - mx) : 1.0f;
    if (raise) st.m = mx;
    st.l *= f;
    if (have_o) {
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        uint32_t o[32];
        tmem_ld32(o_addr + 32 * c, o);
        tmem_wait_ld32(o);
#pragma unroll
        for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
        tmem_st32(o_addr + 32 * c, o);
      }
    }
  }
  const float nm = st.m == -INFINITY ? 0.0f : -st.m;
  const float2 mul2v = f2(mul, mul), nm2 = f2(nm, nm);
  float2 sum = f2(0.0f, 0.0f), sum2 = f2(0.0f, 0.0f);
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    uint32_t w[16];
    const uint32_t* x32 = r + 32 * c;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float2 x = fma2(f2(__uint_as_float(x32[2 * i]), __uint_as_float(x32[2 * i + 1])), mul2v, nm2);
      const float2 p = f2(exp2_fast(x.x), exp2_fast(x.y));
      if (i & 1) sum2 = add2(sum2, p); else sum = add2(sum, p);
      w[i] = Elem<T>::pack(p.x, p.y);
    }
    tmem_st16(s_addr + 16 * c, w);
  }
  sum = add2(sum, sum2);
  st.l += sum.x + sum.y;
  tmem_wait_st();
}

// ---------------------------------------------------------------- packed rows
// A tile of rows of one sequence.
struct RowItem {
  int seq, row0;  // its first packed row
  int rows, len;  // its rows in all, and those that are computed (at most max_rows)
  int q0;         // the tile's first row in the sequence
};

// Tile `idx` (of `tile` rows): under a causal mask a sequence's last tiles take longest and come first.
// Up to 32 sequences: all sequences' tiles by their place in the sequence, from the last on. More: from
// the last sequence's last tile backwards, a dependent step per 32 sequences (31 for the first of 1000
// sequences, in every CTA) and without an order by length. One warp; item->len is 0 when there is no such
// tile. Offsets are cut to [0, n_rows] and to ascending order.
__device__ __forceinline__ void find_item(const int32_t* cu_rows, int n_seqs, int n_rows, int max_rows, int tile,
                                          int idx, int lane, RowItem* item) {
  if (lane == 0) item->len = 0;
  __syncwarp();
  if (n_seqs <= 32) {
    int b = 0, rows = 0;
    if (lane < n_seqs) {
      b = min(max(__ldg(cu_rows + lane), 0), n_rows);
      rows = min(max(__ldg(cu_rows + lane + 1), b), n_rows) - b;
    }
    const int len = min(rows, max_rows), nt = (len + tile - 1) / tile;
    // tiles at place p or behind it, over all sequences
    auto behind = [&](int p) { return __reduce_add_sync(0xffffffffu, max(0, nt - p)); };
    int lo = 0, hi = __reduce_max_sync(0xffffffffu, nt);
    if (idx >= behind(0)) return;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (behind(mid) > idx) lo = mid; else hi = mid;
    }
    const int rank = idx - behind(lo + 1);
    const uint32_t has = __ballot_sync(0xffffffffu, nt > lo);
    if (nt > lo && __popc(has & ((1u << lane) - 1u)) == rank) {
      item->seq = lane;
      item->row0 = b;
      item->rows = rows;
      item->len = len;
      item->q0 = lo * tile;
    }
    return;
  }
  for (int s0 = n_seqs - 1; s0 >= 0; s0 -= 32) {
    const int s = s0 - lane;
    int b = 0, rows = 0;
    if (s >= 0) {
      b = min(max(__ldg(cu_rows + s), 0), n_rows);
      rows = min(max(__ldg(cu_rows + s + 1), b), n_rows) - b;
    }
    const int len = min(rows, max_rows), nt = (len + tile - 1) / tile;
    int acc = nt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, acc, o);
      if (lane >= o) acc += y;
    }
    if (idx >= acc - nt && idx < acc) {
      item->seq = s;
      item->row0 = b;
      item->rows = rows;
      item->len = len;
      item->q0 = (nt - 1 - (idx - (acc - nt))) * tile;
    }
    const int total = __shfl_sync(0xffffffffu, acc, 31);
    if (idx < total) break;
    idx -= total;
  }
}

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

}  // namespace kvq
