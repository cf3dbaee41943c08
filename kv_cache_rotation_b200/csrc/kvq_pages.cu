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
// takes its share of the rows, of the new table entries and of the sequences.
// A row finds its sequence by bisection of the row offsets. What bounds it is
// the scan's latency, then the three words written per row.
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
  const long long ps = a.div_ps.d;
  k0 = static_cast<int>((ctx + ps - 1) / ps);
  const long long k1 = (static_cast<long long>(ctx) + n + ps - 1) / ps;
  need = static_cast<int>(max(0ll, min(k1, static_cast<long long>(a.max_pages)) - k0));
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
  long long miss = 0;  // rows without a slot: past the pool's end or the table's
  for (int s = s0; s < s1; ++s) {
    int ctx, n, k0, need;
    seq_pages(a, s, ctx, n, k0, need);
    cu[s] = sat32(r);
    pst[s] = sat32(p);
    const long long got = max(0ll, min(static_cast<long long>(need), a.n_free - used - p));
    const long long end = min(k0 + got, static_cast<long long>(a.max_pages)) * a.div_ps.d;
    miss += max(0ll, static_cast<long long>(ctx) + n - max(static_cast<long long>(ctx), end));
    r += n;
    p += need;
  }
  if (tid == 0) {
    cu[a.S] = sat32(all_rows);
    pst[a.S] = sat32(all_pages);
  }
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) miss += __shfl_xor_sync(0xffffffffu, miss, o);
  if (lane == 0) wmiss[warp] = miss;
  __syncthreads();

  const int gtid = blockIdx.x * kMapThreads + tid, gsize = gridDim.x * kMapThreads;
  if (gtid == 0) {
    long long m = 0;
    for (int w = 0; w < kMapThreads / 32; ++w) m += wmiss[w];
    a.report[0] = cu[a.S];
    a.report[1] = static_cast<int>(min(used + all_pages, static_cast<long long>(a.n_free)));
    a.report[2] = sat32(m);
    a.report[3] = sat32(max(0ll, used + all_pages - a.n_free));
  }
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
// D / 16 lanes hold a row of one head, 16 consecutive channels each: a lane
// loads 32 contiguous bytes, a warp 1 KB. FWHT strides 1 .. 8 run in registers
// on packed pairs, strides 16 .. D/2 by shuffle (every lane computes
// fma(own, +-1, partner): exactly a + b below and a - b above). Rows go
// head-fastest, so the heads of a token share its (cos, sin) row in L1.
constexpr int kRowThreads = 256;
constexpr int kC = 16;  // channels per lane

struct RowArgs {
  int H, n_sink, rope, rope_rows, rot, lpg, sink_rows, out_fp32;
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

// (cos, sin) of this lane's channels: mode 1 (pairs 2i, 2i+1) 8 pairs, mode 2
// (pairs i, i + D/2) the 16 angles of its channels modulo D/2.
template <int D, bool INV>
__device__ __forceinline__ void rope_rows16(const RowArgs& a, int m, int part, float (&x)[kC]) {
  constexpr int L = D / kC;
  const float4* cs = reinterpret_cast<const float4*>(a.rope_cs + static_cast<size_t>(m) * D);
  if (a.rope == 1) {
#pragma unroll
    for (int i = 0; i < kC / 4; ++i) {
      const float4 c = __ldg(cs + part * (kC / 4) + i);
      float x0 = x[4 * i], x1 = x[4 * i + 1], x2 = x[4 * i + 2], x3 = x[4 * i + 3];
      rope_fwd(x0, x1, c.x, INV ? -c.y : c.y);
      rope_fwd(x2, x3, c.z, INV ? -c.w : c.w);
      x[4 * i] = x0, x[4 * i + 1] = x1, x[4 * i + 2] = x2, x[4 * i + 3] = x3;
    }
  } else {
    const bool up = part >= L / 2;
#pragma unroll
    for (int i = 0; i < kC / 2; ++i) {
      const float4 c = __ldg(cs + (part & (L / 2 - 1)) * (kC / 2) + i);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float own = x[2 * i + e];
        const float oth = __shfl_xor_sync(0xffffffffu, own, L / 2);
        float x0 = up ? oth : own, x1 = up ? own : oth;
        rope_fwd(x0, x1, e ? c.z : c.x, INV ? -(e ? c.w : c.y) : (e ? c.w : c.y));
        x[2 * i + e] = up ? x1 : x0;
      }
    }
  }
}

// Unnormalised FWHT of a row held by D / 16 lanes.
template <int D>
__device__ __forceinline__ void fwht_rows16(int part, float (&x)[kC]) {
  float2 P[kC / 2];  // the register-pair layout of fwht_pairs
#pragma unroll
  for (int g = 0; g < kC / 4; ++g) {
    P[2 * g] = f2(x[4 * g], x[4 * g + 2]);
    P[2 * g + 1] = f2(x[4 * g + 1], x[4 * g + 3]);
  }
  fwht_pairs<kC>(P);
#pragma unroll
  for (int o = 1; o < D / kC; o <<= 1) {
    const float sg = (part & o) ? -1.0f : 1.0f;
#pragma unroll
    for (int k = 0; k < kC / 2; ++k) {
      const float2 q = f2(__shfl_xor_sync(0xffffffffu, P[k].x, o), __shfl_xor_sync(0xffffffffu, P[k].y, o));
      P[k] = fma2(P[k], f2(sg, sg), q);
    }
  }
#pragma unroll
  for (int g = 0; g < kC / 4; ++g) {
    x[4 * g] = P[2 * g].x;
    x[4 * g + 2] = P[2 * g].y;
    x[4 * g + 1] = P[2 * g + 1].x;
    x[4 * g + 3] = P[2 * g + 1].y;
  }
}

// A warp's rows of the permutation: D floats and four of padding each.
template <int D>
__host__ __device__ constexpr int row_words() { return D + 4; }
template <int D>
constexpr size_t perm_smem() { return static_cast<size_t>(kRowThreads / 32) * (32 * kC / D) * row_words<D>() * 4; }

template <int D, int BITS>
__global__ void __launch_bounds__(kRowThreads) k_encode_rows(const RowArgs a) {
  constexpr int L = D / kC, VW = 32 / L;  // lanes per row, rows per warp
  constexpr int RB = D * BITS / 8;
  extern __shared__ __align__(16) float row_smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, part = lane % L;
  float* buf = row_smem + (warp * VW + lane / L) * row_words<D>();
  const uint32_t step = gridDim.x * (kRowThreads / 32) * VW;
  for (uint32_t base = (blockIdx.x * (kRowThreads / 32) + warp) * VW; base < a.n_vec; base += step) {
    const RowPlace p = place<D>(a, base + lane / L);
    const uint4* src = reinterpret_cast<const uint4*>(a.x + static_cast<int64_t>(p.row) * a.stride + p.h * D + part * kC);
    const uint4 r0 = __ldg(src), r1 = __ldg(src + 1);
    float x[kC];
    h8_to_f32(r0, x);
    h8_to_f32(r1, x + 8);
    if (p.sink) {
      uint4* dst = reinterpret_cast<uint4*>(a.sink + p.sink_at + part * kC);
      dst[0] = r0;
      dst[1] = r1;
    }
    if (a.rope) rope_rows16<D, false>(a, p.m, part, x);
    if (a.perm) {
#pragma unroll
      for (int i = 0; i < kC / 4; ++i)
        reinterpret_cast<float4*>(buf + part * kC)[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
      __syncwarp();
      const uint4* pr = reinterpret_cast<const uint4*>(a.perm + static_cast<size_t>(p.h) * D + part * kC);
      const uint4 p0 = __ldg(pr), p1 = __ldg(pr + 1);
      const uint32_t pw[8] = {p0.x, p0.y, p0.z, p0.w, p1.x, p1.y, p1.z, p1.w};
#pragma unroll
      for (int i = 0; i < kC; ++i) x[i] = buf[(pw[i >> 1] >> (16 * (i & 1))) & (D - 1)];
      __syncwarp();
    }
    if (a.rot) {
      fwht_rows16<D>(part, x);
#pragma unroll
      for (int i = 0; i < kC; ++i) x[i] = __fmul_rn(x[i], a.rscale);
    }
    float lo = x[0], hi = x[0];
#pragma unroll
    for (int i = 1; i < kC; ++i) lo = fminf(lo, x[i]), hi = fmaxf(hi, x[i]);
#pragma unroll
    for (int o = 1; o < L; o <<= 1)
      if (o < a.lpg) {
        lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
        hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
      }
    QParams q = minmax_params<BITS>(lo, hi);
    if (p.sink) {
      q.Z = q.R = 0.0f;
      q.sz = __halves2half2(__ushort_as_half(0), __ushort_as_half(0));
    }
    uint64_t w = 0;  // 16 codes: 4, 6 or 8 bytes
#pragma unroll
    for (int i = 0; i < kC; ++i) {
      const float u = __fmaf_rn(__fsub_rn(x[i], q.Z), q.R, kMagicRound);
      // a NaN or overflowed group has no code: whatever bits it gives stay in its own field
      const uint32_t c = (__float_as_uint(u) - kMagicBits) & ((1u << BITS) - 1u);
      w |= static_cast<uint64_t>(p.sink ? 0u : c) << (BITS * i);
    }
    if (p.live) {
      uint8_t* dst = a.codes + p.rec * RB + part * (kC * BITS / 8);
      if constexpr (BITS == 2) {
        *reinterpret_cast<uint32_t*>(dst) = static_cast<uint32_t>(w);
      } else if constexpr (BITS == 4) {
        *reinterpret_cast<uint2*>(dst) = make_uint2(static_cast<uint32_t>(w), static_cast<uint32_t>(w >> 32));
      } else {
#pragma unroll
        for (int i = 0; i < 3; ++i) reinterpret_cast<uint16_t*>(dst)[i] = static_cast<uint16_t>(w >> (16 * i));
      }
      if (part % a.lpg == 0) a.sz[p.rec * (L / a.lpg) + part / a.lpg] = q.sz;
    }
  }
}

template <int D, int BITS>
__global__ void __launch_bounds__(kRowThreads) k_decode_rows(const RowArgs a) {
  constexpr int L = D / kC, VW = 32 / L;
  constexpr int RB = D * BITS / 8;
  extern __shared__ __align__(16) float row_smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, part = lane % L;
  float* buf = row_smem + (warp * VW + lane / L) * row_words<D>();
  const uint32_t step = gridDim.x * (kRowThreads / 32) * VW;
  for (uint32_t base = (blockIdx.x * (kRowThreads / 32) + warp) * VW; base < a.n_vec; base += step) {
    const RowPlace p = place<D>(a, base + lane / L);
    const uint8_t* src = a.codes + p.rec * RB + part * (kC * BITS / 8);
    uint64_t w;
    if constexpr (BITS == 2) {
      w = __ldg(reinterpret_cast<const uint32_t*>(src));
    } else if constexpr (BITS == 4) {
      const uint2 u = __ldg(reinterpret_cast<const uint2*>(src));
      w = u.x | (static_cast<uint64_t>(u.y) << 32);
    } else {
      const uint16_t* h = reinterpret_cast<const uint16_t*>(src);
      w = __ldg(h) | (static_cast<uint64_t>(__ldg(h + 1)) << 16) | (static_cast<uint64_t>(__ldg(h + 2)) << 32);
    }
    const float2 sz = __half22float2(a.sz[p.rec * (L / a.lpg) + part / a.lpg]);
    const float S = a.rot ? __fmul_rn(sz.x, a.rscale) : sz.x, Z = a.rot ? __fmul_rn(sz.y, a.rscale) : sz.y;
    float x[kC];
#pragma unroll
    for (int i = 0; i < kC; ++i)
      x[i] = __fmaf_rn(code_to_float(static_cast<uint32_t>(w >> (BITS * i)) & ((1u << BITS) - 1u)), S, Z);
    if (a.rot) fwht_rows16<D>(part, x);
    if (a.perm) {  // x[perm[j]] = p_j
      const uint4* pr = reinterpret_cast<const uint4*>(a.perm + static_cast<size_t>(p.h) * D + part * kC);
      const uint4 p0 = __ldg(pr), p1 = __ldg(pr + 1);
      const uint32_t pw[8] = {p0.x, p0.y, p0.z, p0.w, p1.x, p1.y, p1.z, p1.w};
#pragma unroll
      for (int i = 0; i < kC; ++i) buf[(pw[i >> 1] >> (16 * (i & 1))) & (D - 1)] = x[i];
      __syncwarp();
#pragma unroll
      for (int i = 0; i < kC / 4; ++i) {
        const float4 f = reinterpret_cast<const float4*>(buf + part * kC)[i];
        x[4 * i] = f.x, x[4 * i + 1] = f.y, x[4 * i + 2] = f.z, x[4 * i + 3] = f.w;
      }
      __syncwarp();
    }
    if (a.rope) rope_rows16<D, true>(a, p.m, part, x);
    if (p.sink) {
      const uint4* s = reinterpret_cast<const uint4*>(a.sink + p.sink_at + part * kC);
      h8_to_f32(s[0], x);
      h8_to_f32(s[1], x + 8);
    }
    if (p.live) {
      const int64_t at = static_cast<int64_t>(p.row) * a.stride + p.h * D + part * kC;
      if (a.out_fp32) {
        float4* o = reinterpret_cast<float4*>(static_cast<float*>(a.out) + at);
#pragma unroll
        for (int i = 0; i < kC / 4; ++i) o[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
      } else {
        uint4* o = reinterpret_cast<uint4*>(static_cast<__half*>(a.out) + at);
        o[0] = f32_to_h8(x);
        o[1] = f32_to_h8(x + 8);
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
  const long long per_cta = (kRowThreads / 32) * (32 * kC / D);
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
  a.lpg = d.group / kC;
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
  const size_t smem = 2 * (static_cast<size_t>(pg.n_seqs) + 1) * 4;
  if (smem > 48 * 1024 && !set_smem_once(reinterpret_cast<const void*>(k_page_map), smem)) return KVQ_ERR_CUDA;
  long long grid = (static_cast<long long>(pg.n_rows) + 4 * kMapThreads - 1) / (4 * kMapThreads);
  if (grid > ctx.num_sms) grid = ctx.num_sms;
  if (grid < 1) grid = 1;
  k_page_map<<<static_cast<unsigned>(grid), kMapThreads, smem, st>>>(a);
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
