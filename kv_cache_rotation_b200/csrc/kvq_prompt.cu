// Causal attention over whole packed prompts (kvq_attend_prompt):
//   out_i = sum_{n <= i} p_n v_n,  p = softmax_n(scale * q_i . k_n)
// in one pass over the keys with the running maximum and sum of the softmax.
//
// A CTA takes 128 or 2 x 128 query rows of one KV head: one or two slots of T =
// 128 / g tokens, the g query heads of the KV head side by side (row t * g + j of a
// slot is token t, head j), so a tile of keys serves every head that shares it
// and a short prompt still fills the rows. Keys and values come in tiles of
// 128 through one ring of TMA loads. Per tile and slot: scores = Q . K^T on
// the tensor cores into tensor memory, softmax by a warpgroup (a thread per
// row), the weights back into tensor memory in the scores' place, sums += P . V.
// Two slots alternate: while one's scores are in the softmax, the tensor
// cores work for the other.
//
// Warps: 0-3 and 4-7 softmax of slots 0 and 1; 8 loads; 9 issues the products;
// 10 and 11 clear what the mask hides in V (see below).
//
// Measured: 16384 tokens of 8 / 2 heads of 128, bf16, 531 us = 1036 TFLOP/s call after call, at the
// power limit (1.37 GHz); tensor pipe and exponentials 57 % of a launch's cycles each, in turn. Nine
// prompts, 6500 tokens, 32 / 8 heads, 118 us: set-up and epilogue of a CTA (about 4500 clocks) and a
// short grid's tail. One prompt of 77 tokens 8.8 us: a launch and one chain. The registers are full (20
// bytes a thread spilled with two slots, 48 to 56 with one).
//
// Masked keys get weight 0, but 0 * inf is not 0, so V must be finite wherever
// a weight is masked: only the last tiles of a CTA (from the diagonal on) hold
// masked keys, and two warps go over those: rows behind the sequence become
// zero, and a value that is not finite is taken out and its first row noted
// per channel, by kind; the rows that see it get it back at the end.
#include <math.h>

#include "kvq_flash.cuh"
#include "kvq_internal.h"

namespace kvq {
namespace {

// Threads: a warpgroup of softmax per slot, and one with the loads, the products and two warps of
// cleaning. Registers a thread has at launch (the launch bound's limit), and after the split by
// warpgroup; a sum above the launch's would wait for ever.
template <int SLOTS>
struct Split {
  static constexpr int kThreads = 128 * (SLOTS + 1);
  static constexpr int kLaunch = SLOTS == 2 ? 168 : 128, kSoftmax = SLOTS == 2 ? 208 : 200, kRest = SLOTS == 2 ? 80 : 56;
  static_assert(128 * SLOTS * kSoftmax + 128 * kRest <= kThreads * kLaunch, "register split");
};
constexpr int kEdges = 4;  // tiles of a CTA that can hold masked keys: 256 rows, not aligned to the tiles

template <int D, int SLOTS>
struct Cfg {
  static constexpr int kStages = (SLOTS == 2 ? 5 : 2) * (128 / D);
  static constexpr uint32_t kHead = D / 64 * kTileBytes;  // 128 rows of a head
  static constexpr uint32_t kRing = SLOTS * kHead;         // after the Q tiles
  static constexpr uint32_t kCols = 256 * SLOTS;           // tensor memory: scores of each slot, then the sums
  static constexpr uint32_t kMisc = kRing + kStages * kHead;
  static constexpr uint32_t kSmem = kMisc + 2048 + 1024;   // + alignment of the tiles
};

struct Misc {
  uint64_t q_full, full[10], empty[10], s_full[2], p_full[2], o_full[2], loaded[kEdges], clean[kEdges], drain;
  uint32_t tmem;
  int dirty;
  RowItem item;
  int first[3][128];  // first row with +inf, -inf, NaN in a channel of V, relative to the sequence
};
static_assert(sizeof(Misc) <= 2048, "fits behind the ring");

struct KernelArgs {
  PromptArgs p;
  int g, T;
  uint32_t* err;
  uint64_t wait_ns;
  float mul;  // scale * log2(e)
};

template <typename T, int D, int SLOTS>
__global__ void __launch_bounds__(Split<SLOTS>::kThreads, 3 - SLOTS)
    k_prompt_tiles(const KernelArgs a, const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                   const __grid_constant__ CUtensorMap mv) {
  using C = Cfg<D, SLOTS>;
  constexpr int ST = C::kStages;
  constexpr int LOAD = 4 * SLOTS, MMA = LOAD + 1, CLEAN = LOAD + 2;  // warps
  extern __shared__ uint8_t flash_smem[];
  const uint32_t base = (smem_u32(flash_smem) + 1023u) & ~1023u;
  uint8_t* const gbase = flash_smem + (base - smem_u32(flash_smem));
  Misc* const m = reinterpret_cast<Misc*>(gbase + C::kMisc);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int idx = static_cast<int>(blockIdx.x / static_cast<unsigned>(a.p.heads));
  const int h = static_cast<int>(blockIdx.x) - idx * a.p.heads;
  if (warp == LOAD) {
    find_item(a.p.cu_rows, a.p.n_seqs, a.p.n_rows, a.p.max_rows, SLOTS * a.T, idx, lane, &m->item);
  } else if (warp == MMA) {
    tmem_alloc(&m->tmem, C::kCols);
  } else if (tid == 0) {
    mbar_init(&m->q_full, 1);
    for (int i = 0; i < ST; ++i) mbar_init(&m->full[i], 1), mbar_init(&m->empty[i], 1);
    for (int t = 0; t < SLOTS; ++t) mbar_init(&m->s_full[t], 1), mbar_init(&m->p_full[t], 4), mbar_init(&m->o_full[t], 1);
    for (int i = 0; i < kEdges; ++i) mbar_init(&m->loaded[i], 1), mbar_init(&m->clean[i], 2);
    mbar_init(&m->drain, 1);
    m->dirty = 0;
    fence_mbar_init();
  } else if (warp == CLEAN) {
    for (int c = lane; c < 3 * 128; c += 32) m->first[c >> 7][c & 127] = 0x7fffffff;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = m->tmem;
  const int row0 = m->item.row0, len = m->item.len, q0 = m->item.q0;
  if (len == 0) {  // a tile that the bound of the grid allows for and no sequence has
    if (warp == MMA) tmem_dealloc(tmem, C::kCols);
    return;
  }
  const uint32_t ring = base + C::kRing;
  // tiles of keys that slot t sees
  int n_t[SLOTS];
#pragma unroll
  for (int t = 0; t < SLOTS; ++t) {
    const int b = q0 + t * a.T, e = min(len, b + a.T);
    n_t[t] = b < len ? (e + 127) >> 7 : 0;
  }
  const int n = max(n_t[0], n_t[SLOTS - 1]);
  const int edge = (q0 + 1) >> 7;  // tiles from here on hold keys that some row does not see

  if (warp < LOAD) {
    more_regs<Split<SLOTS>::kSoftmax>();
    const int t = warp >> 2;
    const int r = tid & 127, tok = q0 + t * a.T + r / a.g;
    const bool mine = r < a.T * a.g && tok < len;
    const int lim = mine ? tok + 1 : 0x7fffffff;  // a row of no token is computed unmasked and not stored
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(warp & 3) << 21);
    const uint32_t s_addr = lane_base + 128 * t, o_addr = lane_base + 128 * SLOTS + D * t;
    RowStat st;
    bool ok = true;
    const int nt = SLOTS == 2 && t ? n_t[SLOTS - 1] : n_t[0];
    for (int i = 0; i < nt; ++i) {
      ok = mbar_wait(&m->s_full[t], i & 1, a.wait_ns, a.err);
      if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
      tc_fence_after();
      const int left = lim - 128 * i;  // columns seen
      const uint32_t seen[4] = {first_bits(left, 0), first_bits(left, 32), first_bits(left, 64), first_bits(left, 96)};
      if (__any_sync(0xffffffffu, left < 128))
        softmax_tile<T, D, true>(s_addr, o_addr, i > 0, a.mul, st, seen);
      else
        softmax_tile<T, D, false>(s_addr, o_addr, i > 0, a.mul, st, seen);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&m->p_full[t]);
    }
    if (ok && nt > 0) ok = __all_sync(0xffffffffu, mbar_wait(&m->o_full[t], 0, a.wait_ns, a.err));
    if (ok && nt > 0) {
      tc_fence_after();
      const float inv = st.l > 0.0f || st.l != st.l ? 1.0f / st.l : 0.0f;
      const bool dirty = *reinterpret_cast<volatile int*>(&m->dirty) != 0;
      // Two slots (many CTAs): out over the slot's query rows, which nothing reads any more, so that a store writes
      // 128 bytes of each of four rows and not 16 of 32 (nine prompts 118 us against 122). One slot (a call that does
      // not fill the SMs): straight out, which is sooner done (77 tokens 8.5 us against 8.9 when this was chosen).
      uint8_t* const rows = gbase + t * C::kHead;
      T* const own = static_cast<T*>(a.p.out) + (static_cast<int64_t>(row0) + tok) * a.p.out_stride + (h * a.g + r % a.g) * D;
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        uint32_t o[32], w[16];
        tmem_ld32(o_addr + 32 * c, o);
        tmem_wait_ld32(o);
#pragma unroll
        for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * inv);
        if (dirty) {  // the values taken out of V that this row sees
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            float x = __uint_as_float(o[i]);
            if (m->first[0][32 * c + i] <= tok) x += INFINITY;
            if (m->first[1][32 * c + i] <= tok) x -= INFINITY;
            if (m->first[2][32 * c + i] <= tok) x = NAN;
            o[i] = __float_as_uint(x);
          }
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) w[i] = Elem<T>::pack(__uint_as_float(o[2 * i]), __uint_as_float(o[2 * i + 1]));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint4 four = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
          if constexpr (SLOTS == 2) *reinterpret_cast<uint4*>(rows + (c / 2) * kTileBytes + sw128(r, 4 * (c & 1) + i)) = four;
          else if (mine) reinterpret_cast<uint4*>(own + 32 * c)[i] = four;
        }
      }
      if constexpr (SLOTS == 2) {
        __syncwarp();
        int first = r & ~31;
        asm volatile("" : "+r"(first));  // nothing of this is worked out before the loop and kept in registers
#pragma unroll 2
        for (int i = 0; i < 8; ++i) {
          const int q = first + 4 * i + (lane >> 3), qt = q / a.g, at = q0 + t * a.T + qt;
          if (qt >= a.T || at >= len) continue;
          T* out = static_cast<T*>(a.p.out) + (static_cast<int64_t>(row0) + at) * a.p.out_stride +
                   (h * a.g + q - qt * a.g) * D + 8 * (lane & 7);
#pragma unroll
          for (int c = 0; c < D / 64; ++c)
            *reinterpret_cast<uint4*>(out + 64 * c) =
                *reinterpret_cast<const uint4*>(rows + c * kTileBytes + sw128(q, lane & 7));
        }
      }
    }
  } else {
    fewer_regs<Split<SLOTS>::kRest>();
  }
  if (warp == LOAD) {
    if (lane == 0) {  // tiles in the order K0 V0 K1 V1 ...
      const uint32_t qbytes = static_cast<uint32_t>(a.T * a.g) * 128u * (D / 64);
      mbar_arrive_expect_tx(&m->q_full, SLOTS * qbytes);
#pragma unroll
      for (int t = 0; t < SLOTS; ++t)
#pragma unroll
        for (int c = 0; c < D / 64; ++c)
          tma_load_3d(gbase + t * C::kHead + c * kTileBytes, &mq, 64 * c, h * a.g, row0 + q0 + t * a.T, &m->q_full);
      // V from the diagonal on lands on a barrier of its own, used once: its cleaners have not followed the ring's
      // phases. No other load follows on such a stage (two or four stages: only V, each on its own barrier;
      // five or ten: at most three such tiles, so the call's last load comes sooner).
      auto landed = [&](int i) {
        return (i & 1) && (i >> 1) >= edge ? &m->loaded[(i >> 1) - edge] : &m->full[i % ST];
      };
      int i = 0;
      for (; i < 2 * n; ++i) {
        const int s = i % ST;
        if (i >= ST && !mbar_wait(&m->empty[s], ((i / ST) & 1) ^ 1, a.wait_ns, a.err)) break;
        mbar_arrive_expect_tx(landed(i), C::kHead);
#pragma unroll
        for (int c = 0; c < D / 64; ++c)
          tma_load_3d(gbase + C::kRing + s * C::kHead + c * kTileBytes, (i & 1) ? &mv : &mk, 64 * c, h,
                      row0 + (i >> 1) * 128, landed(i));
      }
      // nothing leaves the CTA with a copy in flight, whatever the others met
      mbar_wait(&m->q_full, 0, a.wait_ns, a.err);
      for (int k = max(0, i - ST); k < i; ++k)
        mbar_wait(landed(k), landed(k) == &m->full[k % ST] ? (k / ST) & 1 : 0, a.wait_ns, a.err);
    }
  } else if (warp == MMA) {
    {
      bool ok = warp_wait(&m->q_full, 0, a.wait_ns, a.err);
      ok = ok && warp_wait(&m->full[0], 0, a.wait_ns, a.err);
      if (ok) {
        for (int t = 0; t < SLOTS; ++t)
          if (n_t[t] > 0) {
            issue_scores<T, D>(tmem + 128 * t, base + t * C::kHead, ring);
            tc_commit(&m->s_full[t]);
          }
        tc_commit(&m->empty[0]);
      }
      for (int j = 0; ok && j < n; ++j) {
        const int vi = 2 * j + 1, ki = 2 * j + 2;
        ok = j >= edge ? warp_wait(&m->clean[j - edge], 0, a.wait_ns, a.err)
                       : warp_wait(&m->full[vi % ST], (vi / ST) & 1, a.wait_ns, a.err);
        if (ok && j + 1 < n) ok = warp_wait(&m->full[ki % ST], (ki / ST) & 1, a.wait_ns, a.err);
        for (int t = 0; ok && t < SLOTS; ++t) {
          if (j >= n_t[t]) continue;
          ok = warp_wait(&m->p_full[t], j & 1, a.wait_ns, a.err);
          if (!ok) break;
          tc_fence_after();
          issue_values<T, D>(tmem + 128 * SLOTS + D * t, tmem + 128 * t, ring + (vi % ST) * C::kHead, j > 0);
          if (j + 1 < n_t[t]) {
            issue_scores<T, D>(tmem + 128 * t, base + t * C::kHead, ring + (ki % ST) * C::kHead);
            tc_commit(&m->s_full[t]);
          } else {
            tc_commit(&m->o_full[t]);
          }
        }
        if (ok) {
          tc_commit(&m->empty[vi % ST]);
          if (j + 1 < n) tc_commit(&m->empty[ki % ST]);
        }
      }
      if (!ok) {  // a wait ran out: the products in flight still end before the memory is given back
        tc_commit(&m->drain);
        warp_wait(&m->drain, 0, a.wait_ns, a.err);
      }
    }
  } else if (warp >= CLEAN) {
    for (int j = edge; j < n; ++j) {
      const int vi = 2 * j + 1;
      const bool ok = mbar_wait(&m->loaded[j - edge], 0, a.wait_ns, a.err);
      if (!__all_sync(0xffffffffu, ok)) break;
      // two warps, alternate rows; eight chunks of 16 bytes on their way at a time
      constexpr int CH = D / 8, PER = 32 / CH;  // chunks of a row, rows a warp reads at once
      const int c = lane % CH, keys = min(128, len - 128 * j), mine = (warp - CLEAN) * PER + lane / CH;
      uint8_t* const col = gbase + C::kRing + (vi % ST) * C::kHead + (c / 8) * kTileBytes;
      for (int r = mine; r < 128; r += 2 * PER)
        if (r >= keys) *reinterpret_cast<uint4*>(col + sw128(r, c % 8)) = make_uint4(0, 0, 0, 0);
      constexpr uint32_t A = 0x7fff7fffu, B = Elem<T>::kToTop, S = 0x80008000u;
      for (int r0 = mine; r0 < keys; r0 += 16 * PER) {
        uint4 v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = *reinterpret_cast<const uint4*>(col + sw128((r0 + 2 * PER * i) & 127, c % 8));
        uint32_t bad = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i)
          bad |= ((v[i].x & A) + B) | ((v[i].y & A) + B) | ((v[i].z & A) + B) | ((v[i].w & A) + B);
        if (!(bad & S)) continue;
        for (int i = 0; i < 8; ++i) {  // seldom: take them out one by one
          const int r = r0 + 2 * PER * i;
          if (r >= keys) break;
          uint16_t* e = reinterpret_cast<uint16_t*>(col + sw128(r, c % 8));
          for (int k = 0; k < 8; ++k) {
            const uint32_t x = e[k] & 0x7fffu;
            if (x < Elem<T>::kInf) continue;
            atomicMin(&m->first[x > Elem<T>::kInf ? 2 : e[k] >> 15][8 * c + k], 128 * j + r);
            e[k] = 0;
            *reinterpret_cast<volatile int*>(&m->dirty) = 1;
          }
        }
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&m->clean[j - edge]);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == MMA) tmem_dealloc(tmem, C::kCols);
}

// Row tiles of the call at most: the lengths are on the device.
long long max_tiles(const PromptArgs& p, int slots) {
  const long long tt = slots * (128 / (p.q_heads / p.heads));
  const long long by_rows = p.n_rows / tt + p.n_seqs, by_max = p.n_seqs * ((p.max_rows + tt - 1) / tt);
  return by_rows < by_max ? by_rows : by_max;
}

template <typename T, int D, int SLOTS>
kvq_status run(const PromptArgs& p, cudaStream_t st, const LaunchCtx& ctx) {
  using C = Cfg<D, SLOTS>;
  KernelArgs a{};
  a.p = p;
  a.g = p.q_heads / p.heads;
  a.T = 128 / a.g;
  a.err = ctx.err;
  a.wait_ns = ctx.wait_ns;
  a.mul = p.scale * 1.4426950408889634f;
  const CUtensorMapDataType type = p.bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  CUtensorMap mq, mk, mv;
  auto map = [&](CUtensorMap* m, const void* x, int heads, int64_t stride, uint32_t bh, uint32_t br) {
    const uint64_t dims[3] = {D, static_cast<uint64_t>(heads), static_cast<uint64_t>(p.n_rows)};
    const uint64_t str[2] = {2 * D, static_cast<uint64_t>(stride) * 2};
    const uint32_t box[3] = {64, bh, br};
    return make_map(m, type, 3, x, dims, str, box, CU_TENSOR_MAP_SWIZZLE_128B);
  };
  if (!map(&mq, p.q, p.q_heads, p.q_stride, static_cast<uint32_t>(a.g), static_cast<uint32_t>(a.T)) ||
      !map(&mk, p.k, p.heads, p.k_stride, 1, 128) || !map(&mv, p.v, p.heads, p.v_stride, 1, 128))
    return KVQ_ERR_CUDA;
  const long long grid = max_tiles(p, SLOTS) * p.heads;
  if (grid >= (1ll << 31)) return KVQ_ERR_UNSUPPORTED;
  const void* fn = reinterpret_cast<const void*>(k_prompt_tiles<T, D, SLOTS>);
  if (!set_smem_once(fn, C::kSmem) || !split_fits(fn, Split<SLOTS>::kLaunch)) return KVQ_ERR_CUDA;
  k_prompt_tiles<T, D, SLOTS><<<static_cast<unsigned>(grid), Split<SLOTS>::kThreads, C::kSmem, st>>>(a, mq, mk, mv);
  return launch_status();
}

template <typename T, int D>
kvq_status run_slots(const PromptArgs& p, cudaStream_t st, const LaunchCtx& ctx) {
  // Two slots keep the tensor cores busier (nine prompts, 6500 tokens: 118 us against 132; 16384 tokens:
  // 525 against 574); one slot is sooner done where the call does not fill the SMs (77 tokens: 8.5 us
  // against 10.3).
  return max_tiles(p, 2) * p.heads > ctx.num_sms ? run<T, D, 2>(p, st, ctx) : run<T, D, 1>(p, st, ctx);
}

}  // namespace

kvq_status launch_attend_prompt(const PromptArgs& p, cudaStream_t st, const LaunchCtx& ctx) {
  if (p.bf16)
    return p.head_dim == 128 ? run_slots<__nv_bfloat16, 128>(p, st, ctx) : run_slots<__nv_bfloat16, 64>(p, st, ctx);
  return p.head_dim == 128 ? run_slots<__half, 128>(p, st, ctx) : run_slots<__half, 64>(p, st, ctx);
}

}  // namespace kvq
