// Attention of packed new rows over the pages of a compressed cache
// (kvq_attend_paged). With y the dequantized record and R = P^T H the rotation
// of a head, khat = R y and vhat = R y, so
//   q . khat = (R^T q) . y,   sum_n p_n vhat_n = R (sum_n p_n y_n):
// the query is rotated once, the output once. The sinks' fp16 rows enter in
// their own basis.
#include <math.h>

#include "kvq_device.cuh"
#include "kvq_internal.h"

namespace kvq {
namespace {

struct PagedArgs {
  int S, n_rows, max_pages, sink_rows, H, Hq, g, ps, n_pages, n_sink, rope, rope_rows, rot, group, max_rows;
  int64_t q_stride, out_stride;
  float scale, rscale;
  const __half* q;
  __half* out;
  const int32_t *cu_rows, *kv_len, *block_table, *sink_slot;
  const int16_t *kperm, *vperm;
  const float* rope_cs;
  const uint8_t *kcodes, *vcodes;
  const __half2 *ksz, *vsz;
  const __half *ksink, *vsink;
};

// FWHT of D channels, D / 32 consecutive ones per lane, unnormalised.
template <int C>
__device__ __forceinline__ void warp_fwht(float (&x)[C], int lane) {
  fwht_reg<C>(x);
#pragma unroll
  for (int o = 1; o < 32; o <<= 1)
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const float y = __shfl_xor_sync(0xffffffffu, x[i], o);
      x[i] = (lane & o) ? y - x[i] : x[i] + y;
    }
}
__device__ __forceinline__ float all_sum(float v) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// This lane's C codes of a record, dequantized.
template <int C, int BITS>
__device__ __forceinline__ void read_record(const uint8_t* rec, const __half2* sz, int group, int lane, float (&y)[C]) {
  const int bit = lane * C * BITS;
  const float2 p = __half22float2(sz[lane * C / group]);
#pragma unroll
  for (int i = 0; i < C; ++i) {
    const int b = bit + i * BITS;
    uint32_t c = rec[b >> 3] >> (b & 7);
    if ((b & 7) + BITS > 8) c |= static_cast<uint32_t>(rec[(b >> 3) + 1]) << (8 - (b & 7));
    y[i] = fmaf(static_cast<float>(c & ((1u << BITS) - 1u)), p.x, p.y);
  }
}

// One warp per (row, query head).
template <int D, int BITS>
__global__ void __launch_bounds__(128) k_paged_rows(const PagedArgs a) {
  constexpr int C = D / 32, RB = D * BITS / 8;
  __shared__ float nat[4][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long wi = blockIdx.x * 4ll + warp;
  const int row = static_cast<int>(wi / a.Hq), qh = static_cast<int>(wi % a.Hq);
  if (row >= a.n_rows) return;
  int seq = -1, m = 0, i = 0;
  for (int s = 0; s < a.S; ++s) {
    const int b = __ldg(a.cu_rows + s), e = min(a.n_rows, __ldg(a.cu_rows + s + 1));
    if (row >= b && row < e && row - b < a.max_rows) seq = s, m = e - b, i = row - b;
  }
  if (seq < 0) return;
  const int h = qh / a.g, last = __ldg(a.kv_len + seq) - m + i;  // the last visible position
  const __half* qp = a.q + row * a.q_stride + qh * D;
  float q[C], qr[C], o[C], on[C], mx = -INFINITY, l = 0.0f;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    q[c] = __half2float(qp[lane * C + c]);
    qr[c] = a.kperm ? __half2float(qp[a.kperm[h * D + lane * C + c] & (D - 1)]) : q[c];
    o[c] = on[c] = 0.0f;
  }
  if (a.rot) {
    warp_fwht<C>(qr, lane);
#pragma unroll
    for (int c = 0; c < C; ++c) qr[c] *= a.rscale;
  }
  const int srow = a.n_sink ? (a.sink_slot ? __ldg(a.sink_slot + seq) : seq) : -1;
  for (int n = 0; n <= last; ++n) {
    float k[C], v[C], s = 0.0f;
    const bool sink = n < a.n_sink;
    const int pg = n / a.ps < a.max_pages ? __ldg(a.block_table + static_cast<size_t>(seq) * a.max_pages + n / a.ps) : -1;
    if (pg < 0 || pg >= a.n_pages) continue;
    if (sink) {
      if (srow < 0 || srow >= a.sink_rows || (a.rope && n >= a.rope_rows)) continue;
      const size_t at = ((static_cast<size_t>(srow) * a.H + h) * a.n_sink + n) * D;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int j = lane * C + c;
        float x = __half2float(a.ksink[at + j]);
        if (a.rope) {
          const int j2 = a.rope == 1 ? j ^ 1 : (j < D / 2 ? j + D / 2 : j - D / 2), pr = a.rope == 1 ? j / 2 : j % (D / 2);
          const float2 cs = reinterpret_cast<const float2*>(a.rope_cs)[static_cast<size_t>(n) * (D / 2) + pr];
          const bool up = a.rope == 1 ? (j & 1) : j >= D / 2;
          const float x2 = __half2float(a.ksink[at + j2]);
          x = up ? fmaf(x2, cs.y, x * cs.x) : fmaf(x, cs.x, -(x2 * cs.y));
        }
        s = fmaf(q[c], x, s);
        v[c] = __half2float(a.vsink[at + j]);
      }
    } else {
      const size_t rec = (static_cast<size_t>(pg) * a.H + h) * a.ps + n % a.ps;
      read_record<C, BITS>(a.kcodes + rec * RB, a.ksz + rec * (D / a.group), a.group, lane, k);
      read_record<C, BITS>(a.vcodes + rec * RB, a.vsz + rec * (D / a.group), a.group, lane, v);
#pragma unroll
      for (int c = 0; c < C; ++c) s = fmaf(qr[c], k[c], s);
    }
    s = all_sum(s) * a.scale;
    const float mn = fmaxf(mx, s), f = mx == mn ? 1.0f : __expf(mx - mn), p = __expf(s - mn);
    mx = mn;
    l = fmaf(l, f, p);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      o[c] = o[c] * f + (sink ? 0.0f : p * v[c]);
      on[c] = on[c] * f + (sink ? p * v[c] : 0.0f);
    }
  }
  if (a.rot) {
    warp_fwht<C>(o, lane);
#pragma unroll
    for (int c = 0; c < C; ++c) o[c] *= a.rscale;
  }
#pragma unroll
  for (int c = 0; c < C; ++c) nat[warp][a.vperm ? a.vperm[h * D + lane * C + c] & (D - 1) : lane * C + c] = o[c];
  __syncwarp();
  const float inv = l > 0.0f ? 1.0f / l : 0.0f;
#pragma unroll
  for (int c = 0; c < C; ++c)
    a.out[row * a.out_stride + qh * D + lane * C + c] = __float2half_rn((nat[warp][lane * C + c] + on[c]) * inv);
}

}  // namespace

size_t attend_paged_workspace_bytes(const kvq_desc&, int, const kvq_paged&, int, int) { return 256; }

kvq_status launch_attend_paged(const kvq_desc& dk, const kvq_desc&, const void* q, int64_t q_stride, int q_heads,
                               const kvq_packed& kc, const kvq_tables& tk, const kvq_packed& vc, const kvq_tables& tv,
                               const kvq_paged& pg, int max_rows, int, float scale, void* out, int64_t out_stride,
                               void*, cudaStream_t st, const LaunchCtx&) {
  PagedArgs a{};
  a.S = pg.n_seqs;
  a.n_rows = pg.n_rows;
  a.max_pages = pg.max_pages;
  a.sink_rows = pg.sink_rows;
  a.H = dk.heads;
  a.Hq = q_heads;
  a.g = q_heads / dk.heads;
  a.ps = dk.t_cap;
  a.n_pages = dk.batch;
  a.n_sink = dk.n_sink;
  a.rope = dk.rope;
  a.rope_rows = tk.rope_rows;
  a.rot = dk.rot == KVQ_ROT_FWHT_HEAD;
  a.group = dk.group;
  a.max_rows = max_rows;
  a.q_stride = q_stride;
  a.out_stride = out_stride;
  a.scale = scale;
  a.rscale = static_cast<float>(1.0 / sqrt(static_cast<double>(dk.head_dim)));
  a.q = static_cast<const __half*>(q);
  a.out = static_cast<__half*>(out);
  a.cu_rows = pg.cu_rows;
  a.kv_len = pg.kv_len;
  a.block_table = pg.block_table;
  a.sink_slot = pg.sink_slot;
  a.kperm = tk.perm;
  a.vperm = tv.perm;
  a.rope_cs = tk.rope_cs;
  a.kcodes = kc.codes;
  a.vcodes = vc.codes;
  a.ksz = static_cast<const __half2*>(kc.scale_zero);
  a.vsz = static_cast<const __half2*>(vc.scale_zero);
  a.ksink = static_cast<const __half*>(kc.sink);
  a.vsink = static_cast<const __half*>(vc.sink);
  const unsigned grid = static_cast<unsigned>((static_cast<long long>(pg.n_rows) * q_heads + 3) / 4);
#define KVQ_CASE(D_, B_) \
  if (dk.head_dim == D_ && dk.bits == B_) { k_paged_rows<D_, B_><<<grid, 128, 0, st>>>(a); return launch_status(); }
  KVQ_CASE(128, 2) KVQ_CASE(128, 3) KVQ_CASE(128, 4) KVQ_CASE(64, 2) KVQ_CASE(64, 3) KVQ_CASE(64, 4)
#undef KVQ_CASE
  return KVQ_ERR_UNSUPPORTED;
}

}  // namespace kvq
