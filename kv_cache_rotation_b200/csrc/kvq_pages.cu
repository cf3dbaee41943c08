// The paged cache: block tables and slot maps from a batch's lengths
// (k_page_map), and the head-variant encode / decode of packed token rows
// through a slot map (k_encode_rows, k_decode_rows). The transform and the
// quantizer are kvq_encode's, operation by operation ("RotateKV: Accurate and
// Robust 2-Bit KV Cache Quantization for LLMs via Outlier-Aware Adaptive
// Rotations", 关键设计): RoPE in the fma order of rope_fwd, the permutation
// gather, the FWHT's strides in ascending order, min-max per group, so a row
// has the same record here and in a dense cache.
//
// Page p, head h, offset o of the pool is record (p * H + h) * page_size + o:
// a dense cache whose batch is the page and whose t_cap is the page size.
#include <math.h>

#include "kvq_device.cuh"
#include "kvq_internal.h"

namespace kvq {
namespace {

// ---------------------------------------------------------------- page map
// One launch: every CTA scans the S lengths (rows and new pages per sequence)
// into shared memory for itself, which costs less than a second launch, then
// takes its share of the rows, of the new table entries and of the sequences;
// the last CTA takes none and writes the report, whose table reads would
// lengthen the others' chain (1000 sequences, call after call: 7.5 us in one of them, 6.6 beside).
// A row finds its sequence by bisection of the row offsets. What bounds it is
// that chain of dependent steps (two passes over the lengths, the scan, the
// bisection, a table read), then the three words written per row.
constexpr int kMapThreads = 512;
// kMapMaxSeqs sequences take two int32 prefix sums of 64 KB

struct MapArgs {
  int S, n_rows, max_pages, n_free, n_pages;
  FastDiv div_ps;
  const int32_t* ctx_len;
  const int32_t* new_len;
  const int32_t* free_pages;
  const int32_t* free_used;
  int32_t *cu_rows, *kv_len, *block_table, *seq, *pos, *slot, *report;
};

__device__ __forceinline__ int sat32(long long v) { return v > 0x7fffffffll ? 0x7fffffff : static_cast<int>(v); }

// Pages of sequence s: it holds k0 of them, takes `need` more.
__device__ __forceinline__ void seq_pages(const MapArgs& a, int s, int& ctx, int& n, int& k0, int& need) {
  ctx = max(0, __ldg(a.ctx_len + s));
  n = max(0, __ldg(a.new_len + s));
  auto pages = [&](int tokens) {  // rounded up
    const uint32_t t = static_cast<uint32_t>(tokens), q = a.div_ps.div(t);
    return static_cast<int>(q + (a.div_ps.mod(t, q) != 0));
  };
  k0 = pages(ctx);
  need = max(0, min(pages(sat32(static_cast<long long>(ctx) + n)), a.max_pages) - k0);
}

// Largest s in [0, S) with off[s] <= v (off ascending, off[0] <= v < off[S]).
__device__ __forceinline__ int find_seq(const int* off, int S, int v) {
  int lo = 0, hi = S;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (off[mid] <= v) lo = mid; else hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kMapThreads) k_page_map(const MapArgs a) {
  extern __shared__ int map_smem[];
  int* cu = map_smem;                // [S + 1] first row of each sequence
  int* pst = map_smem + a.S + 1;     // [S + 1] first new page of each sequence
  __shared__ long long wrow[kMapThreads / 32], wpage[kMapThreads / 32], wmiss[kMapThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (a.S + kMapThreads - 1) / kMapThreads;  // consecutive sequences of a thread
  const int s0 = min(a.S, tid * per), s1 = min(a.S, s0 + per);
  const bool reports = blockIdx.x == gridDim.x - 1;
  long long rows = 0, pages = 0;
  for (int s = s0; s < s1; ++s) {
    int ctx, n, k0, need;
    seq_pages(a, s, ctx, n, k0, need);
    rows += n;
    pages += need;
  }
  long long r = rows, p = pages;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long r2 = __shfl_up_sync(0xffffffffu, r, o), p2 = __shfl_up_sync(0xffffffffu, p, o);
    if (lane >= o) r += r2, p += p2;
  }
  if (lane == 31) wrow[warp] = r, wpage[warp] = p;
  __syncthreads();
  r -= rows;
  p -= pages;
  long long all_pages = 0, all_rows = 0;
  for (int w = 0; w < kMapThreads / 32; ++w) {
    if (w < warp) r += wrow[w], p += wpage[w];
    all_rows += wrow[w];
    all_pages += wpage[w];
  }
  const long long used = max(0, __ldg(a.free_used));
  long long miss = 0;  // rows without a slot
  for (int s = s0; s < s1; ++s) {
    int ctx, n, k0, need;
    seq_pages(a, s, ctx, n, k0, need);
    cu[s] = sat32(r);
    pst[s] = sat32(p);
    if (reports) {  // past the pool's end or the table's, or going on in a page that an earlier call did not get
      const long long got = max(0ll, min(static_cast<long long>(need), a.n_free - used - p));
      const long long end = min(k0 + got, static_cast<long long>(a.max_pages)) * a.div_ps.d;
      miss += max(0ll, static_cast<long long>(ctx) + n - max(static_cast<long long>(ctx), end));
      const uint32_t part = static_cast<uint32_t>(k0) * a.div_ps.d - static_cast<uint32_t>(ctx);  // left of its last page
      if (n > 0 && part > 0 && k0 <= a.max_pages) {
        const int page = a.block_table[static_cast<size_t>(s) * a.max_pages + k0 - 1];
        if (page < 0 || page >= a.n_pages) miss += min(static_cast<uint32_t>(n), part);
      }
    }
    r += n;
    p += need;
  }
  if (tid == 0) {
    cu[a.S] = sat32(all_rows);
    pst[a.S] = sat32(all_pages);
  }
  if (reports) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) miss += __shfl_xor_sync(0xffffffffu, miss, o);
    if (lane == 0) wmiss[warp] = miss;
  }
  __syncthreads();
  if (reports) {
    if (tid != 0) return;
    long long m = 0;
    for (int w = 0; w < kMapThreads / 32; ++w) m += wmiss[w];
    a.report[0] = cu[a.S];
    a.report[1] = static_cast<int>(min(used + all_pages, static_cast<long long>(a.n_free)));
    a.report[2] = sat32(m);
    a.report[3] = sat32(max(0ll, used + all_pages - a.n_free));
    return;
  }

  const int gtid = blockIdx.x * kMapThreads + tid, gsize = (gridDim.x - 1) * kMapThreads;
  for (int s = gtid; s <= a.S; s += gsize) {
    a.cu_rows[s] = cu[s];
    if (s < a.S) a.kv_len[s] = sat32(static_cast<long long>(max(0, __ldg(a.ctx_len + s))) + max(0, __ldg(a.new_len + s)));
  }
  auto new_page = [&](long long i) { return used + i < a.n_free ? __ldg(a.free_pages + used + i) : -1; };
  for (int e = gtid; e < pst[a.S]; e += gsize) {
    const int s = find_seq(pst, a.S, e);
    int ctx, n, k0, need;
    seq_pages(a, s, ctx, n, k0, need);
    a.block_table[static_cast<size_t>(s) * a.max_pages + k0 + (e - pst[s])] = new_page(e);
  }
  // four consecutive rows per thread: mostly one sequence, one 16-byte store per array
  const int total = cu[a.S];
  for (long long b = 4ll * gtid; b < a.n_rows; b += 4ll * gsize) {
    int sv[4], pv[4], lv[4];
    int s = -1, next = 0, ctx = 0, k0 = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = static_cast<int>(b) + i;
      sv[i] = pv[i] = lv[i] = -1;
      if (row >= a.n_rows || row >= total) continue;
      if (s < 0 || row >= next) {
        int n, need;
        s = find_seq(cu, a.S, row);
        next = cu[s + 1];
        seq_pages(a, s, ctx, n, k0, need);
      }
      const long long ps64 = static_cast<long long>(ctx) + (row - cu[s]);
      sv[i] = s;
      pv[i] = sat32(ps64);
      if (ps64 < 0x7fffffffll) {
        const int k = static_cast<int>(a.div_ps.div(static_cast<uint32_t>(ps64)));
        if (k < a.max_pages) {
          const int page = k < k0 ? a.block_table[static_cast<size_t>(s) * a.max_pages + k]
                                  : new_page(static_cast<long long>(pst[s]) + (k - k0));
          if (page >= 0 && page < a.n_pages) lv[i] = page * static_cast<int>(a.div_ps.d) + static_cast<int>(a.div_ps.mod(static_cast<uint32_t>(ps64), k));
        }
      }
    }
    const int nb = static_cast<int>(b);
    if (nb + 4 <= a.n_rows) {
      *reinterpret_cast<int4*>(a.seq + nb) = make_int4(sv[0], sv[1], sv[2], sv[3]);
      *reinterpret_cast<int4*>(a.pos + nb) = make_int4(pv[0], pv[1], pv[2], pv[3]);
      *reinterpret_cast<int4*>(a.slot + nb) = make_int4(lv[0], lv[1], lv[2], lv[3]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (nb + i < a.n_rows) {
          a.seq[nb + i] = sv[i];
          a.pos[nb + i] = pv[i];
          a.slot[nb + i] = lv[i];
        }
    }
  }
}

// ---------------------------------------------------------------- rows
// L = D / 16 lanes hold a row of one head; lane p has channels 8p .. 8p+7 and
// the same of the upper half, so each half of a row is one run of 16-byte loads
// and both RoPE pairings stay inside a lane. P[i] = (x[8p + i], x[D/2 + 8p + i]).
// FWHT strides in ascending order: 1, 2, 4 on packed pairs, 8 .. D/4 by shuffle
// (every lane computes fma(own, +-1, partner): exactly a + b below and a - b
// above), D/2 inside the pairs. Rows go head-fastest, so the heads of a token
// share its (cos, sin) row in L1. With the permutation the L1 data pipe is the
// bound (75 to 87 % busy: gather, shuffles, (cos, sin) rows; issue 54 to 64 %):
// K and V of 30119 rows of 8 heads in and out, 4 bits, groups of 64, half-split
// RoPE, take 224 us for 318 MB (1.42 TB/s, 22 % of a copy's rate), the table of
// 2940 positions counted once.
constexpr int kRowThreads = 256;

struct RowArgs {
  int H, n_sink, rope, rope_rows, rot, sink_rows, out_fp32;
  int whole, lanes;  // a group is the whole row; else the lanes of a group within a half
  uint32_t n_vec;  // n_rows * H
  int64_t stride;  // elements between the rows of x / out
  FastDiv div_h, div_ps;
  uint32_t n_slots;  // pages * page_size
  float rscale;
  const __half* x;
  void* out;
  const int32_t *seq, *pos, *slot, *sink_slot;
  const int16_t* perm;
  const float* rope_cs;
  uint8_t* codes;
  __half2* sz;
  __half* sink;
};

struct RowPlace {
  bool live, sink;     // the row has a slot; it is a sink position
  int h, m;            // head, position
  size_t rec, row;     // record index, packed row
  size_t sink_at;      // its row in the sink buffer
};

template <int D>
__device__ __forceinline__ RowPlace place(const RowArgs& a, uint32_t v) {
  RowPlace p;
  const uint32_t vv = v < a.n_vec ? v : a.n_vec - 1;
  const uint32_t row = a.div_h.div(vv);
  p.row = row;
  p.h = static_cast<int>(a.div_h.mod(vv, row));
  const int slot = __ldg(a.slot + row);
  const int m = __ldg(a.pos + row);
  p.live = v < a.n_vec && slot >= 0 && static_cast<uint32_t>(slot) < a.n_slots && m >= 0 && !(a.rope && m >= a.rope_rows);
  const uint32_t sl = p.live ? static_cast<uint32_t>(slot) : 0u;
  p.m = p.live ? m : 0;
  const uint32_t page = a.div_ps.div(sl);
  p.rec = (static_cast<size_t>(page) * a.H + p.h) * a.div_ps.d + a.div_ps.mod(sl, page);
  p.sink = p.live && p.m < a.n_sink;
  p.sink_at = 0;
  if (p.sink) {
    const int s = __ldg(a.seq + row);
    const int at = s >= 0 && s < a.sink_rows ? (a.sink_slot ? __ldg(a.sink_slot + s) : s) : -1;
    if (at < 0 || at >= a.sink_rows) p.live = p.sink = false;  // a sink without a place: the row is skipped
    else p.sink_at = ((static_cast<size_t>(at) * a.H + p.h) * a.n_sink + p.m) * D;
  }
  return p;
}

// RoPE of both pairings, in the fma order of rope_fwd.
template <int D, bool INV>
__device__ __forceinline__ void rope_row(const RowArgs& a, int m, int part, float2 (&P)[8]) {
  const float4* cs = reinterpret_cast<const float4*>(a.rope_cs + static_cast<size_t>(m) * D);
  if (a.rope == 1) {  // pairs 4p .. 4p+3 of each half
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float4 u = __ldg(cs + 2 * part + i), v = __ldg(cs + D / 8 + 2 * part + i);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float2 c = e ? f2(u.z, v.z) : f2(u.x, v.x), t = e ? f2(u.w, v.w) : f2(u.y, v.y), n = f2(-t.x, -t.y);
        const float2 x0 = P[4 * i + 2 * e], x1 = P[4 * i + 2 * e + 1];
        P[4 * i + 2 * e] = fma2(x0, c, mul2(x1, INV ? t : n));
        P[4 * i + 2 * e + 1] = fma2(x0, INV ? n : t, mul2(x1, c));
      }
    }
  } else {  // pairs (i, i + D/2), angles 8p .. 8p+7
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 u = __ldg(cs + 4 * part + i);
      rope_fwd(P[2 * i].x, P[2 * i].y, u.x, INV ? -u.y : u.y);
      rope_fwd(P[2 * i + 1].x, P[2 * i + 1].y, u.z, INV ? -u.w : u.w);
    }
  }
}

// Unnormalised FWHT of a row.
template <int D>
__device__ __forceinline__ void fwht_row(int part, float2 (&P)[8]) {
#pragma unroll
  for (int h = 1; h < 8; h <<= 1)
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if ((i & h) == 0) bfly(P[i], P[i + h]);
#pragma unroll
  for (int o = 1; o < D / 16; o <<= 1) {
    const float sg = (part & o) ? -1.0f : 1.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float2 q = f2(__shfl_xor_sync(0xffffffffu, P[k].x, o), __shfl_xor_sync(0xffffffffu, P[k].y, o));
      P[k] = fma2(P[k], f2(sg, sg), q);
    }
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) P[k] = f2(__fadd_rn(P[k].x, P[k].y), __fsub_rn(P[k].x, P[k].y));
}

// Rows of the permutation in shared memory: channel j at j + 4 (j / 32), so that the lanes' 16-byte
// accesses (32 bytes apart) meet different banks.
__device__ __forceinline__ int row_at(int j) { return j + ((j >> 5) << 2); }
template <int D>
__host__ __device__ constexpr int row_words() { return D + D / 8; }
template <int D>
constexpr size_t perm_smem() { return static_cast<size_t>(kRowThreads / 32) * (512 / D) * row_words<D>() * 4; }

// Own channels of a row into the buffer / out of it.
template <int D>
__device__ __forceinline__ void put_own(float* buf, int part, const float2 (&P)[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    *reinterpret_cast<float4*>(buf + row_at(8 * part + 4 * i)) = make_float4(P[4 * i].x, P[4 * i + 1].x, P[4 * i + 2].x, P[4 * i + 3].x);
    *reinterpret_cast<float4*>(buf + row_at(D / 2 + 8 * part + 4 * i)) = make_float4(P[4 * i].y, P[4 * i + 1].y, P[4 * i + 2].y, P[4 * i + 3].y);
  }
}
template <int D>
__device__ __forceinline__ void get_own(const float* buf, int part, float2 (&P)[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float4 u = *reinterpret_cast<const float4*>(buf + row_at(8 * part + 4 * i));
    const float4 v = *reinterpret_cast<const float4*>(buf + row_at(D / 2 + 8 * part + 4 * i));
    P[4 * i] = f2(u.x, v.x), P[4 * i + 1] = f2(u.y, v.y), P[4 * i + 2] = f2(u.z, v.z), P[4 * i + 3] = f2(u.w, v.w);
  }
}
// perm[h][own channels], low and high halves of words in channel order.
template <int D>
__device__ __forceinline__ void own_perm(const RowArgs& a, int h, int part, uint4& lo, uint4& hi) {
  const uint4* pr = reinterpret_cast<const uint4*>(a.perm + static_cast<size_t>(h) * D) + part;
  lo = __ldg(pr);
  hi = __ldg(pr + D / 16);
}
__device__ __forceinline__ int nth16(const uint4& v, int i) {
  const uint32_t w = i < 2 ? v.x : i < 4 ? v.y : i < 6 ? v.z : v.w;
  return static_cast<int>((w >> (16 * (i & 1))) & 0xffffu);
}

// The eight codes of one half of a lane, BITS each, to and from the record. Three bits: four lanes'
// 24-bit runs are three words, which the first three of them hold.
template <int BITS>
__device__ __forceinline__ void store_codes(uint8_t* at, int part, uint32_t w, bool live) {
  if constexpr (BITS == 2) {
    if (live) *reinterpret_cast<uint16_t*>(at + 2 * part) = static_cast<uint16_t>(w);
  } else if constexpr (BITS == 4) {
    if (live) *reinterpret_cast<uint32_t*>(at + 4 * part) = w;
  } else {
    const int k = part & 3;
    const uint32_t up = __shfl_down_sync(0xffffffffu, w, 1);
    if (live && k < 3) *reinterpret_cast<uint32_t*>(at + 12 * (part >> 2) + 4 * k) = (w >> (8 * k)) | (up << (24 - 8 * k));
  }
}
template <int BITS>
__device__ __forceinline__ uint32_t load_codes(const uint8_t* at, int part) {
  if constexpr (BITS == 2) {
    return __ldg(reinterpret_cast<const uint16_t*>(at + 2 * part));
  } else if constexpr (BITS == 4) {
    return __ldg(reinterpret_cast<const uint32_t*>(at + 4 * part));
  } else {
    const int k = part & 3;
    const uint32_t own = k < 3 ? __ldg(reinterpret_cast<const uint32_t*>(at + 12 * (part >> 2) + 4 * k)) : 0u;
    const uint32_t before = __shfl_up_sync(0xffffffffu, own, 1);
    return k == 0 ? own : __funnelshift_r(before, own, 32 - 8 * k);
  }
}

template <int D, int BITS>
__global__ void __launch_bounds__(kRowThreads) k_encode_rows(const RowArgs a) {
  constexpr int L = D / 16, VW = 32 / L;  // lanes per row, rows per warp
  constexpr int RB = D * BITS / 8;
  extern __shared__ __align__(16) float row_smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, part = lane % L;
  float* buf = row_smem + (warp * VW + lane / L) * row_words<D>();
  const uint32_t step = gridDim.x * (kRowThreads / 32) * VW;
  for (uint32_t base = (blockIdx.x * (kRowThreads / 32) + warp) * VW; base < a.n_vec; base += step) {
    const RowPlace p = place<D>(a, base + lane / L);
    const uint4* src = reinterpret_cast<const uint4*>(a.x + static_cast<int64_t>(p.row) * a.stride + p.h * D) + part;
    const uint4 r0 = __ldg(src), r1 = __ldg(src + D / 16);
    float2 P[8];
    {
      float lo[8], hi[8];
      h8_to_f32(r0, lo);
      h8_to_f32(r1, hi);
#pragma unroll
      for (int i = 0; i < 8; ++i) P[i] = f2(lo[i], hi[i]);
    }
    if (p.sink) {
      uint4* dst = reinterpret_cast<uint4*>(a.sink + p.sink_at) + part;
      dst[0] = r0;
      dst[D / 16] = r1;
    }
    if (a.rope) rope_row<D, false>(a, p.m, part, P);
    if (a.perm) {  // p_j = y[perm[j]]
      uint4 lo, hi;
      own_perm<D>(a, p.h, part, lo, hi);
      put_own<D>(buf, part, P);
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 8; ++i)
        P[i] = f2(buf[row_at(nth16(lo, i) & (D - 1))], buf[row_at(nth16(hi, i) & (D - 1))]);
      __syncwarp();
    }
    if (a.rot) {
      fwht_row<D>(part, P);
#pragma unroll
      for (int i = 0; i < 8; ++i) P[i] = mul2(P[i], f2(a.rscale, a.rscale));
    }
    // the halves' ranges, joined where a group is the whole row
    float2 mn = P[0], mx = P[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) {
      mn = f2(fminf(mn.x, P[i].x), fminf(mn.y, P[i].y));
      mx = f2(fmaxf(mx.x, P[i].x), fmaxf(mx.y, P[i].y));
    }
    if (a.whole) {
      mn.x = fminf(mn.x, mn.y);
      mx.x = fmaxf(mx.x, mx.y);
    }
#pragma unroll
    for (int o = 1; o < L; o <<= 1)
      if (o < a.lanes) {
        mn.x = fminf(mn.x, __shfl_xor_sync(0xffffffffu, mn.x, o));
        mx.x = fmaxf(mx.x, __shfl_xor_sync(0xffffffffu, mx.x, o));
        if (!a.whole) {
          mn.y = fminf(mn.y, __shfl_xor_sync(0xffffffffu, mn.y, o));
          mx.y = fmaxf(mx.y, __shfl_xor_sync(0xffffffffu, mx.y, o));
        }
      }
    QParams q0 = minmax_params<BITS>(mn.x, mx.x), q1 = a.whole ? q0 : minmax_params<BITS>(mn.y, mx.y);
    if (p.sink) {  // a sink's record is zero: every value quantizes with Z = R = 0
      q0.Z = q0.R = q1.Z = q1.R = 0.0f;
      q0.sz = q1.sz = __halves2half2(__ushort_as_half(0), __ushort_as_half(0));
    }
    // code = the integer added to the magic constant; its pattern's offset is taken off once per word
    uint32_t w0 = 0, w1 = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 u = fma2(add2(P[i], f2(-q0.Z, -q1.Z)), f2(q0.R, q1.R), f2(kMagicRound, kMagicRound));
      w0 += __float_as_uint(u.x) << (BITS * i);
      w1 += __float_as_uint(u.y) << (BITS * i);
    }
    w0 -= magic_offset<BITS, 8>();
    w1 -= magic_offset<BITS, 8>();
    if constexpr (BITS == 3) w0 &= 0xffffffu, w1 &= 0xffffffu;
    uint8_t* dst = a.codes + p.rec * RB;
    store_codes<BITS>(dst, part, w0, p.live);
    store_codes<BITS>(dst + RB / 2, part, w1, p.live);
    if (p.live) {
      if (a.whole) {
        if (part == 0) a.sz[p.rec] = q0.sz;
      } else if (part % a.lanes == 0) {  // groups of the lower half, then of the upper
        const int per = L / a.lanes;
        __half2* z = a.sz + p.rec * (2 * per) + part / a.lanes;
        z[0] = q0.sz;
        z[per] = q1.sz;
      }
    }
  }
}

template <int D, int BITS>
__global__ void __launch_bounds__(kRowThreads) k_decode_rows(const RowArgs a) {
  constexpr int L = D / 16, VW = 32 / L;
  constexpr int RB = D * BITS / 8;
  constexpr uint32_t MASK = (1u << BITS) - 1u;
  extern __shared__ __align__(16) float row_smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, part = lane % L;
  float* buf = row_smem + (warp * VW + lane / L) * row_words<D>();
  const uint32_t step = gridDim.x * (kRowThreads / 32) * VW;
  for (uint32_t base = (blockIdx.x * (kRowThreads / 32) + warp) * VW; base < a.n_vec; base += step) {
    const RowPlace p = place<D>(a, base + lane / L);
    const uint8_t* src = a.codes + p.rec * RB;
    const uint32_t w0 = load_codes<BITS>(src, part), w1 = load_codes<BITS>(src + RB / 2, part);
    const int per = a.whole ? 0 : L / a.lanes;
    const __half2* z = a.sz + (a.whole ? p.rec : p.rec * (2 * per) + part / a.lanes);
    float2 s0 = __half22float2(z[0]), s1 = __half22float2(z[per]);
    if (a.rot) s0 = mul2(s0, f2(a.rscale, a.rscale)), s1 = mul2(s1, f2(a.rscale, a.rscale));
    float2 P[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 c = f2(__uint_as_float(0x4B000000u | ((w0 >> (BITS * i)) & MASK)),
                          __uint_as_float(0x4B000000u | ((w1 >> (BITS * i)) & MASK)));
      P[i] = fma2(add2(c, f2(-8388608.0f, -8388608.0f)), f2(s0.x, s1.x), f2(s0.y, s1.y));
    }
    if (a.rot) fwht_row<D>(part, P);
    if (a.perm) {  // x[perm[j]] = p_j
      uint4 lo, hi;
      own_perm<D>(a, p.h, part, lo, hi);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        buf[row_at(nth16(lo, i) & (D - 1))] = P[i].x;
        buf[row_at(nth16(hi, i) & (D - 1))] = P[i].y;
      }
      __syncwarp();
      get_own<D>(buf, part, P);
      __syncwarp();
    }
    if (a.rope) rope_row<D, true>(a, p.m, part, P);
    float lo[8], hi[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) lo[i] = P[i].x, hi[i] = P[i].y;
    if (p.sink) {
      const uint4* s = reinterpret_cast<const uint4*>(a.sink + p.sink_at) + part;
      h8_to_f32(s[0], lo);
      h8_to_f32(s[D / 16], hi);
    }
    if (p.live) {
      const int64_t at = static_cast<int64_t>(p.row) * a.stride + p.h * D + 8 * part;
      if (a.out_fp32) {
        float4* o = reinterpret_cast<float4*>(static_cast<float*>(a.out) + at);
        float4* o2 = reinterpret_cast<float4*>(static_cast<float*>(a.out) + at + D / 2);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          o[i] = make_float4(lo[4 * i], lo[4 * i + 1], lo[4 * i + 2], lo[4 * i + 3]);
          o2[i] = make_float4(hi[4 * i], hi[4 * i + 1], hi[4 * i + 2], hi[4 * i + 3]);
        }
      } else {
        *reinterpret_cast<uint4*>(static_cast<__half*>(a.out) + at) = f32_to_h8(lo);
        *reinterpret_cast<uint4*>(static_cast<__half*>(a.out) + at + D / 2) = f32_to_h8(hi);
      }
    }
  }
}

template <int D, int BITS>
kvq_status run_rows(bool enc, const RowArgs& a, const LaunchCtx& ctx, cudaStream_t st) {
  const void* fn = enc ? reinterpret_cast<const void*>(k_encode_rows<D, BITS>)
                       : reinterpret_cast<const void*>(k_decode_rows<D, BITS>);
  const size_t smem = a.perm ? perm_smem<D>() : 0;
  const int per_sm = occupancy_once(fn, kRowThreads, smem);
  const long long per_cta = (kRowThreads / 32) * (512 / D);
  const long long steps = (static_cast<long long>(a.n_vec) + per_cta - 1) / per_cta;
  const long long want = static_cast<long long>(ctx.num_sms) * per_sm;
  const unsigned grid = static_cast<unsigned>(steps < want ? steps : want);
  if (enc)
    k_encode_rows<D, BITS><<<grid, kRowThreads, smem, st>>>(a);
  else
    k_decode_rows<D, BITS><<<grid, kRowThreads, smem, st>>>(a);
  return launch_status();
}

kvq_status launch_rows(bool enc, const kvq_desc& d, const kvq_paged& pg, const kvq_tables& tb, const kvq_packed& c,
                       const void* x, void* out, int64_t stride, int out_fp32, cudaStream_t st, const LaunchCtx& ctx) {
  RowArgs a{};
  a.H = d.heads;
  a.n_sink = d.n_sink;
  a.rope = d.rope;
  a.rope_rows = tb.rope_rows;
  a.rot = d.rot == KVQ_ROT_FWHT_HEAD;
  a.whole = d.group == d.head_dim;
  a.lanes = a.whole ? d.head_dim / 16 : d.group / 8;
  a.sink_rows = pg.sink_rows;
  a.out_fp32 = out_fp32;
  a.n_vec = static_cast<uint32_t>(pg.n_rows) * static_cast<uint32_t>(d.heads);
  a.stride = stride;
  a.div_h = FastDiv(static_cast<uint32_t>(d.heads));
  a.div_ps = FastDiv(static_cast<uint32_t>(d.t_cap));
  a.n_slots = static_cast<uint32_t>(d.batch) * static_cast<uint32_t>(d.t_cap);
  a.rscale = static_cast<float>(1.0 / sqrt(static_cast<double>(d.head_dim)));
  a.x = static_cast<const __half*>(x);
  a.out = out;
  a.seq = pg.seq;
  a.pos = pg.pos;
  a.slot = pg.slot;
  a.sink_slot = pg.sink_slot;
  a.perm = tb.perm;
  a.rope_cs = tb.rope_cs;
  a.codes = c.codes;
  a.sz = static_cast<__half2*>(c.scale_zero);
  a.sink = static_cast<__half*>(c.sink);
#define KVQ_CASE(D_, B_) \
  if (d.head_dim == D_ && d.bits == B_) return run_rows<D_, B_>(enc, a, ctx, st);
  KVQ_CASE(128, 2) KVQ_CASE(128, 3) KVQ_CASE(128, 4) KVQ_CASE(64, 2) KVQ_CASE(64, 3) KVQ_CASE(64, 4)
#undef KVQ_CASE
  return KVQ_ERR_UNSUPPORTED;
}

}  // namespace

kvq_status launch_page_map(const kvq_desc& d, const kvq_paged& pg, const int32_t* ctx_len, const int32_t* new_len,
                           const int32_t* free_pages, int n_free, const int32_t* free_used, int32_t* report,
                           cudaStream_t st, const LaunchCtx& ctx) {
  MapArgs a{};
  a.S = pg.n_seqs;
  a.n_rows = pg.n_rows;
  a.max_pages = pg.max_pages;
  a.n_free = n_free;
  a.n_pages = d.batch;
  a.div_ps = FastDiv(static_cast<uint32_t>(d.t_cap));
  a.ctx_len = ctx_len;
  a.new_len = new_len;
  a.free_pages = free_pages;
  a.free_used = free_used;
  a.cu_rows = pg.cu_rows;
  a.kv_len = pg.kv_len;
  a.block_table = pg.block_table;
  a.seq = pg.seq;
  a.pos = pg.pos;
  a.slot = pg.slot;
  a.report = report;
  // Allowed for on every call, also below 48 KB: that limit covers the kernel's static arrays too, so 6096
  // sequences (48776 bytes, and 384 static) are above it.
  const size_t smem = 2 * (static_cast<size_t>(pg.n_seqs) + 1) * 4;
  if (!set_smem_once(reinterpret_cast<const void*>(k_page_map), smem)) return KVQ_ERR_CUDA;
  long long grid = (static_cast<long long>(pg.n_rows) + 4 * kMapThreads - 1) / (4 * kMapThreads);
  if (grid > ctx.num_sms - 1) grid = ctx.num_sms - 1;
  if (grid < 1) grid = 1;
  k_page_map<<<static_cast<unsigned>(grid + 1), kMapThreads, smem, st>>>(a);
  return launch_status();
}

kvq_status launch_encode_paged(const kvq_desc& d, const void* x, int64_t stride, const kvq_paged& pg,
                               const kvq_tables& tb, const kvq_packed& out, cudaStream_t st, const LaunchCtx& ctx) {
  return launch_rows(true, d, pg, tb, out, x, nullptr, stride, 0, st, ctx);
}

kvq_status launch_decode_paged(const kvq_desc& d, const kvq_packed& in, const kvq_paged& pg, const kvq_tables& tb,
                               void* x_out, int64_t stride, int out_fp32, cudaStream_t st, const LaunchCtx& ctx) {
  return launch_rows(false, d, pg, tb, in, nullptr, x_out, stride, out_fp32, st, ctx);
}

}  // namespace kvq
