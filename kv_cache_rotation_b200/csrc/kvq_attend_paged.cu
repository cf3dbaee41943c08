// Attention of packed new rows over the pages of a compressed cache
// (kvq_attend_paged). With y the dequantized record and R = P^T H the rotation
// of a head (an orthonormal map), khat = R y and vhat = R y, so
//   q . khat = (R^T q) . y,   sum_n p_n vhat_n = R (sum_n p_n y_n):
// the query is rotated once, the output once, and the records are only
// dequantized. The sinks' fp16 rows enter in their own basis, in fp32.
//
// k_paged_tiles: a CTA takes a tile of query rows of one KV head (row t * g +
// j is token t, query head j of the group of g) and a stretch of its keys, in
// tiles of 128. A warpgroup turns records into fp16 tiles in shared memory (read
// through the block table, a thread per record), one thread issues the
// products, and a warpgroup per slot does the softmax (kvq_flash.cuh). The two
// slots are two tiles of 128 rows that share every tile of keys (a chunk of a
// prompt: SHARED), or the same rows with alternate tiles of keys (up to 128 rows,
// a decode step: the second slot is then half of the stretch). Each slot leaves
// its sums, reference and weight total per row in the workspace.
// k_paged_merge: a warp, or eight, per row and query head joins them with the sinks
// and turns the result back.
//
// Measured, 32 / 8 heads of 128: 512 rows on 16384 keys of 4 bits 212 to 216 us = 650 TFLOP/s
// (40 % of the products' rate): a slot's softmax of a tile, 2400 to 2800 clocks beside
// the record warps, and its products take turns, 4370 clocks for two slots' tile; a CTA's
// set-up, first tile and epilogue are 20000 more. Tensor pipe 40 %, exponentials 40 %.
// Twelve sequences of 1 to 131 rows on up to 8000 keys of 3 bits 175 us. The registers are
// full: the two-slot forms spill 156 to 226 bytes a thread, the one-slot forms 68 to 84, and
// part of it is in the loop (local loads and stores are 1.3 % of the chunk's instructions).
#include <math.h>

#include "kvq_flash.cuh"
#include "kvq_internal.h"

namespace kvq {
namespace {

constexpr int kProdWarps = 4;
constexpr int kThreads = 512;  // warps 0-7 softmax, 8-11 records, 12 products; 13-15 only help with the query rows
// Registers a thread has at launch (the launch bound's limit), and after the split by warpgroup. A sum
// above the launch's would wait for ever.
constexpr int kRegsLaunch = 128, kRegsSoftmax = 200, kRegsRecords = 88, kRegsIssue = 24;
static_assert(256 * kRegsSoftmax + 128 * kRegsRecords + 128 * kRegsIssue <= kThreads * kRegsLaunch, "register split");
constexpr int kMasks = 8;  // key masks kept: more tiles than are in flight

struct PagedArgs {
  int S, n_rows, max_pages, sink_rows, H, Hq, g, T, n_pages, n_sink, rope, rope_rows, rot, max_rows;
  int stretch, n_stretch, n_parts;  // keys of a CTA, CTAs along the keys, partial results per row
  int step_page, step_off;          // kFewStep keys in pages and a rest
  FastDiv div_ps, div_hq, div_g, div_stretch;  // page size, query heads, group, keys of a CTA
  int part_per;                                // partial results of a stretch
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
  float* part_o;   // [n_parts][n_rows * Hq][D], channels in tile order
  float2* part_s;  // [n_parts][n_rows * Hq] (reference in log2, weight total)
  uint32_t* err;
  uint64_t wait_ns;
};

// Channels sit in the tiles in the order that the codes unpack to: the two codes
// of a 32-bit register of halves come from the same bit of its two halves.
template <int BITS>
__host__ __device__ constexpr int tile_pos(int ch) {
  if (BITS == 2) return (ch & ~15) + 2 * (ch & 7) + ((ch >> 3) & 1);
  if (BITS == 4) return (ch & ~7) + 2 * (ch & 3) + ((ch >> 2) & 1);
  const int u = ch & 31;  // 3 bits: three runs of 10 codes, then two
  return u >= 30 ? ch : (ch & ~31) + 2 * (5 * (u / 10) + u % 5) + (u % 10) / 5;
}

// 2^-p as an fp16 pair, and -1024 * 2^-p.
__host__ __device__ constexpr uint32_t h2_exp(int p) { return static_cast<uint32_t>(15 - p) * 0x04000400u; }
__host__ __device__ constexpr uint32_t h2_bias(int p) { return 0x80008000u + static_cast<uint32_t>(25 - p) * 0x04000400u; }
__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
// The codes of BITS bits at bit `p` of both halves of x as y = c S + Z: 1024 + c 2^p is put together
// by masking, made c exactly by one fma, and rounded once to fp16 by the next.
template <int BITS, int P>
__device__ __forceinline__ uint32_t code_pair(uint32_t x, uint32_t S, uint32_t Z) {
  static_assert(P + BITS <= 10, "inside the mantissa");
  constexpr uint32_t M = ((1u << BITS) - 1u) << P;
  const uint32_t v = (x & (M | (M << 16))) | 0x64006400u;
  return hfma2(hfma2(v, h2_exp(P), h2_bias(P)), S, Z);
}

// One unit of codes (2 bits: a word, 16 channels; 4 bits: a word, 8; 3 bits: three words, 32) as
// fp16 pairs in tile order.
template <int BITS>
struct Unit;
template <>
struct Unit<2> {
  static constexpr int kWords = 1, kPairs = 8;
  static __device__ __forceinline__ void open(const uint32_t* w, uint32_t S, uint32_t Z, uint32_t* o) {
    const uint32_t a = w[0], b = w[0] >> 10;
    o[0] = code_pair<2, 0>(a, S, Z);
    o[1] = code_pair<2, 2>(a, S, Z);
    o[2] = code_pair<2, 4>(a, S, Z);
    o[3] = code_pair<2, 6>(a, S, Z);
    o[4] = code_pair<2, 8>(a, S, Z);
    o[5] = code_pair<2, 0>(b, S, Z);
    o[6] = code_pair<2, 2>(b, S, Z);
    o[7] = code_pair<2, 4>(b, S, Z);
  }
};
template <>
struct Unit<4> {
  static constexpr int kWords = 1, kPairs = 4;
  static __device__ __forceinline__ void open(const uint32_t* w, uint32_t S, uint32_t Z, uint32_t* o) {
    const uint32_t a = w[0], b = w[0] >> 8;
    o[0] = code_pair<4, 0>(a, S, Z);
    o[1] = code_pair<4, 4>(a, S, Z);
    o[2] = code_pair<4, 0>(b, S, Z);
    o[3] = code_pair<4, 4>(b, S, Z);
  }
};
template <>
struct Unit<3> {
  static constexpr int kWords = 3, kPairs = 16;
  static __device__ __forceinline__ void open(const uint32_t* w, uint32_t S, uint32_t Z, uint32_t* o) {
    const uint32_t run[3] = {w[0], __funnelshift_r(w[0], w[1], 30), __funnelshift_r(w[1], w[2], 28)};
#pragma unroll
    for (int k = 0; k < 3; ++k) {  // codes 0-4 in the low half, 5-9 in the high half
      const uint32_t a = (run[k] & 0x7fffu) | ((run[k] << 1) & 0x7fff0000u), b = a >> 9;
      o[5 * k] = code_pair<3, 0>(a, S, Z);
      o[5 * k + 1] = code_pair<3, 3>(a, S, Z);
      o[5 * k + 2] = code_pair<3, 6>(a, S, Z);
      o[5 * k + 3] = code_pair<3, 0>(b, S, Z);
      o[5 * k + 4] = code_pair<3, 3>(b, S, Z);
    }
    const uint32_t a = ((w[2] >> 26) & 7u) | ((w[2] >> 13) & 0x70000u);
    o[15] = code_pair<3, 0>(a, S, Z);
  }
};

// A record in registers.
template <int D, int BITS, int G>
struct Record {
  static constexpr int kWords = D * BITS / 32, kSz = D / G;
  uint32_t w[kWords], sz[kSz];
  __device__ __forceinline__ void load(const uint8_t* codes, const __half2* s, size_t rec, bool live) {
    if (!live) {
#pragma unroll
      for (int i = 0; i < kWords; ++i) w[i] = 0;
#pragma unroll
      for (int i = 0; i < kSz; ++i) sz[i] = 0;
      return;
    }
    const uint8_t* p = codes + rec * (4 * kWords);
    if constexpr (kWords % 4 == 0) {
#pragma unroll
      for (int i = 0; i < kWords / 4; ++i) {
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(p) + i);
        w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < kWords / 2; ++i) {
        const uint2 v = __ldg(reinterpret_cast<const uint2*>(p) + i);
        w[2 * i] = v.x, w[2 * i + 1] = v.y;
      }
    }
    const uint32_t* z = reinterpret_cast<const uint32_t*>(s) + rec * kSz;
#pragma unroll
    for (int i = 0; i < kSz; ++i) sz[i] = __ldg(z + i);
  }
  // Whether a channel can be infinite or NaN as fp16; the record becomes zero then.
  __device__ __forceinline__ bool clear_if_bad() {
    bool bad = false;
#pragma unroll
    for (int i = 0; i < kSz; ++i) {
      const float2 z = __half22float2(*reinterpret_cast<const __half2*>(&sz[i]));
      bad |= !(fabsf(z.y) < 65520.0f && fabsf(fmaf(static_cast<float>((1 << BITS) - 1), z.x, z.y)) < 65520.0f);
    }
    if (bad) {
#pragma unroll
      for (int i = 0; i < kSz; ++i) sz[i] = 0;
    }
    return bad;
  }
  // Row r of a tile as fp16: the eight lanes of a store phase have eight rows, so the swizzle sends
  // them to eight bank groups.
  __device__ __forceinline__ void store(uint32_t tile, int r) const {
    using U = Unit<BITS>;
    constexpr int UC = 2 * U::kPairs;  // channels of a unit
    const uint32_t row = tile + r * 128u, x = static_cast<uint32_t>(r & 7) << 4;
#pragma unroll
    for (int u = 0; u < D / UC; ++u) {
      const uint32_t s = sz[u * UC / G];
      uint32_t o[U::kPairs];
      U::open(w + u * U::kWords, __byte_perm(s, s, 0x1010), __byte_perm(s, s, 0x3232), o);
#pragma unroll
      for (int c = 0; c < UC / 8; ++c) {
        const uint32_t chunk = u * (UC / 8) + c;
        sts128(row + (chunk / 8) * kTileBytes + (((chunk % 8) << 4) ^ x), make_uint4(o[4 * c], o[4 * c + 1], o[4 * c + 2], o[4 * c + 3]));
      }
    }
  }
};

constexpr int kOutPitch = 20;  // words: eight rows' 16-byte pieces meet all banks
template <int D, bool SHARED>
struct Cfg {
  static constexpr uint32_t kHead = D / 64 * kTileBytes;
  static constexpr uint32_t kK = (SHARED ? 2 : 1) * kHead;  // two stages of keys behind the query rows
  static constexpr uint32_t kV = kK + 2 * kHead;
  static constexpr uint32_t kMisc = kV + 2 * kHead;
  // The sums on their way out, 32 rows x 16 channels of each softmax warp: over the slot's own query rows,
  // which nothing reads any more then, or (slots that share them) behind the rest. What shared memory does
  // not take is L1, where the records' lines wait for a thread's next 16 bytes: with 20 KB less of it a
  // tile took 4950 clocks, not 4370.
  static constexpr uint32_t kOutWarp = 32 * kOutPitch * 4;
  static constexpr uint32_t kOut = SHARED ? 0 : kMisc + 2048, kOutSlot = SHARED ? kHead : 4 * kOutWarp;
  static_assert(4 * kOutWarp <= kHead, "over the query rows");
  static constexpr uint32_t kSmem = kMisc + 2048 + (SHARED ? 0 : 8 * kOutWarp) + 1024;
  static constexpr int kAhead = SHARED ? 1 : 2;  // tiles of keys before the first tile of values
};

struct Misc {
  uint64_t first[2], full[2], empty[2], s_full[2], p_full[2], o_full[2], begun, drain;
  uint32_t tmem;
  int bad;  // first position of a value record that is not finite, among those that some row does not see
  RowItem item;
  alignas(16) uint32_t seen[kMasks][4];  // read 16 bytes at a time
  float mul[2][128];
};
static_assert(sizeof(Misc) <= 2048, "fits behind the rings");

// FWHT of D channels, C = D / 32 consecutive ones per lane, unnormalised.
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
__device__ __forceinline__ float all_max(float v) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// Positions that a block_table row covers, a few blocks below 2^31 so that steps past the end fit.
__device__ __forceinline__ int sat_pages(int pages, int ps) {
  const long long v = static_cast<long long>(pages) * ps;
  return v > 0x7ffffe00ll ? 0x7ffffe00 : static_cast<int>(v);
}

template <int D, int BITS, int G, bool SHARED>
__global__ void __launch_bounds__(kThreads, 1) k_paged_tiles(const PagedArgs a) {
  using C = Cfg<D, SHARED>;
  extern __shared__ uint8_t flash_smem[];
  const uint32_t base = (smem_u32(flash_smem) + 1023u) & ~1023u;
  uint8_t* const gbase = flash_smem + (base - smem_u32(flash_smem));
  Misc* const m = reinterpret_cast<Misc*>(gbase + C::kMisc);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // blocks in the order: key stretch, KV head, row tile (fastest to slowest)
  unsigned rest = blockIdx.x;
  const int z = static_cast<int>(rest % static_cast<unsigned>(a.n_stretch));
  rest /= static_cast<unsigned>(a.n_stretch);
  const int h = static_cast<int>(rest % static_cast<unsigned>(a.H));
  const int idx = static_cast<int>(rest / static_cast<unsigned>(a.H));
  constexpr int SLOTS = SHARED ? 2 : 1;  // tiles of query rows

  // the merge kernel may start once every CTA has: its prologue reads inputs alone
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (warp == 12) find_item(a.cu_rows, a.S, a.n_rows, a.max_rows, SLOTS * a.T, idx, lane, &m->item);
  __syncthreads();
  const RowItem it = m->item;
  if (it.len == 0) return;
  const int cached = max(__ldg(a.kv_len + it.seq), 0);
  const int kv = min(cached, sat_pages(a.max_pages, static_cast<int>(a.div_ps.d)));
  const int pos0 = cached - it.rows + it.q0;  // position of the tile's first token
  const int tokens = min(it.len - it.q0, SLOTS * a.T);
  // keys [k0, k1): this stretch, cut at what the last token sees; the last stretch has no end
  const long long kb = static_cast<long long>(z) * a.stretch;
  const long long ke = z + 1 == a.n_stretch ? 0x7fffffffll : kb + a.stretch;
  const int k0 = static_cast<int>(min(kb, 0x7fffffffll));
  const int k1 = static_cast<int>(min(ke, static_cast<long long>(min(kv, pos0 + tokens))));
  if (k1 <= k0) return;  // no row of the tile sees a key here: the merge does not look
  const int n = (k1 - k0 + 127) >> 7;

  if (warp == 12) tmem_alloc(&m->tmem, 512);
  const int live_warps = min(4, (min(tokens, a.T) * a.g + 31) >> 5);  // of a slot, with rows of a token
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&m->first[i], kProdWarps), mbar_init(&m->full[i], kProdWarps), mbar_init(&m->empty[i], 1);
      mbar_init(&m->s_full[i], 1), mbar_init(&m->o_full[i], 1);
      mbar_init(&m->p_full[i], SHARED ? 4 : live_warps);
    }
    mbar_init(&m->begun, 1), mbar_init(&m->drain, 1);
    m->bad = 0x7fffffff;
    fence_mbar_init();
  }
  // The query rows, rotated, scaled by a power of two into [1, 2) and rounded once to fp16: two lanes a
  // row, lane `half` with every other chunk of 8 channels, so all strides but 8 stay in registers. (With a
  // warp a row the shuffles alone took 13000 clocks for 256 rows, the set-up 21700 of a CTA's 320000.)
  {
    constexpr int NC = D / 16;  // chunks of a lane: 2k + half
    const int rr = tid >> 1, half = tid & 1, t = rr >> 7, tr = rr & 127;
    const int tk = tr / a.g, tok = t * a.T + tk, j = tr - tk * a.g;
    const bool mine = t < SLOTS && tk < a.T && tok < tokens;
    if (__any_sync(0xffffffffu, mine)) {
      const __half* qp = a.q + (static_cast<int64_t>(it.row0) + it.q0 + (mine ? tok : 0)) * a.q_stride + (h * a.g + (mine ? j : 0)) * D;
      uint4 raw[NC];
#pragma unroll
      for (int k = 0; k < NC; ++k) raw[k] = __ldg(reinterpret_cast<const uint4*>(qp) + 2 * k + half);
      if (a.kperm) {  // through a copy of the row where the keys will be
        uint32_t* const buf = reinterpret_cast<uint32_t*>(gbase + C::kK) + rr * (D / 2 + 1);
#pragma unroll
        for (int k = 0; k < NC; ++k) {
          uint32_t* b = buf + 4 * (2 * k + half);
          b[0] = raw[k].x, b[1] = raw[k].y, b[2] = raw[k].z, b[3] = raw[k].w;
        }
        __syncwarp();
        const uint16_t* row = reinterpret_cast<const uint16_t*>(buf);
#pragma unroll
        for (int k = 0; k < NC; ++k) {
          const uint4 pm = __ldg(reinterpret_cast<const uint4*>(a.kperm + h * D) + 2 * k + half);
          auto two = [&](uint32_t w) {
            return static_cast<uint32_t>(row[w & (D - 1)]) | (static_cast<uint32_t>(row[(w >> 16) & (D - 1)]) << 16);
          };
          raw[k] = make_uint4(two(pm.x), two(pm.y), two(pm.z), two(pm.w));
        }
        __syncwarp();
      }
      float x[NC][8];
#pragma unroll
      for (int k = 0; k < NC; ++k) h8_to_f32(raw[k], x[k]);
      // the partner's half of a chunk pair comes over, this lane's other half goes: then it has channels
      // 16 k + e and 16 k + 8 + e for four e, of the codes' order of channels
      constexpr bool kBy2 = BITS == 4;  // e = 2 half + {0, 1, 4, 5}; else 4 half + {0 .. 3}
      float top = 0.0f;
#pragma unroll
      for (int k = 0; k < NC; ++k) {
        if (a.rot) fwht_reg<8>(x[k]);
        float y[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int lo = kBy2 ? (i & 1) + 4 * (i >> 1) : i, hi = lo + (kBy2 ? 2 : 4);
          const float keep = half ? x[k][hi] : x[k][lo], give = half ? x[k][lo] : x[k][hi];
          const float got = __shfl_xor_sync(0xffffffffu, give, 1);
          const float a0 = half ? got : keep, a1 = half ? keep : got;  // channel 16 k + e, and 8 further
          y[i] = a.rot ? a0 + a1 : a0;
          y[4 + i] = a.rot ? a0 - a1 : a1;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) x[k][i] = y[i];
      }
      if (a.rot) {
#pragma unroll
        for (int o = 1; o < NC; o <<= 1)
#pragma unroll
          for (int k = 0; k < NC; ++k)
            if ((k & o) == 0)
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const float u = x[k][i], v = x[k + o][i];
                x[k][i] = u + v;
                x[k + o][i] = u - v;
              }
#pragma unroll
        for (int k = 0; k < NC; ++k)
#pragma unroll
          for (int i = 0; i < 8; ++i) x[k][i] *= a.rscale;
      }
#pragma unroll
      for (int k = 0; k < NC; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(x[k][i]));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      const int e = top > 0.0f && top < INFINITY ? static_cast<int>(__float_as_uint(top) >> 23) - 127 : 0;
      const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
      if (mine) {
        uint8_t* const tile = gbase + t * C::kHead;
        auto at = [&](int p) { return tile + (p / 64) * kTileBytes + sw128(tr, (p % 64) / 8) + 2 * (p % 8); };
        using E = Elem<__half>;
#pragma unroll
        for (int k = 0; k < NC; ++k) {
          float (&y)[8] = x[k];
#pragma unroll
          for (int i = 0; i < 8; ++i) y[i] *= down;
          if constexpr (BITS == 2) {  // 16 k + 2 e, + 1
            *reinterpret_cast<uint4*>(at(16 * k + 8 * half)) =
                make_uint4(E::pack(y[0], y[4]), E::pack(y[1], y[5]), E::pack(y[2], y[6]), E::pack(y[3], y[7]));
          } else if constexpr (BITS == 4) {  // 16 k + 2 (e & 3) + (e >> 2), and 8 further
            *reinterpret_cast<uint2*>(at(16 * k + 4 * half)) = make_uint2(E::pack(y[0], y[2]), E::pack(y[1], y[3]));
            *reinterpret_cast<uint2*>(at(16 * k + 8 + 4 * half)) = make_uint2(E::pack(y[4], y[6]), E::pack(y[5], y[7]));
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int ch = 16 * k + 8 * (i >> 2) + (i & 3), p = half ? tile_pos<BITS>(ch + 4) : tile_pos<BITS>(ch);
              *reinterpret_cast<__half*>(at(p)) = __float2half_rn(y[i]);
            }
          }
        }
        if (half == 0) m->mul[t][tr] = a.scale * 1.4426950408889634f * __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
      }
    }
    fence_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = m->tmem;
  // tiles of keys of each slot: all, or every other one
  int n_t[2];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int last = min(k1, pos0 + min(tokens, (t + 1) * a.T));
    n_t[t] = !SHARED ? (n + 1 - t) >> 1 : tokens > t * a.T && last > k0 ? (last - k0 + 127) >> 7 : 0;
  }

  if (warp < 8) {
    more_regs<kRegsSoftmax>();
    const int t = warp >> 2, tq = SHARED ? t : 0;
    const int r = tid & 127, tok = tq * a.T + r / a.g;
    const bool mine = r < a.T * a.g && tok < tokens;
    const int lim = mine ? pos0 + tok + 1 : 0x7fffffff;
    const float mul = mine ? m->mul[tq][r] : 0.0f;
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(warp & 3) << 21);
    const uint32_t s_addr = lane_base + 128 * t, o_addr = lane_base + 256 + D * t;
    RowStat st;
    if (!mine) st.m = 0.0f;  // whatever a row of no token holds, it asks for no rescaling below
    bool ok = true;
    const bool works = SHARED || (warp & 3) < live_warps;
    const int nt = works ? n_t[t] : 0;
    for (int i = 0; i < nt; ++i) {
      ok = warp_wait(&m->s_full[t], i & 1, a.wait_ns, a.err);
      if (!ok) break;
      tc_fence_after();
      const int tile = SHARED ? i : 2 * i + t;
      const uint4 bits = *reinterpret_cast<const uint4*>(m->seen[tile % kMasks]);
      const int left = lim - (k0 + 128 * tile);
      const uint32_t seen[4] = {bits.x & first_bits(left, 0), bits.y & first_bits(left, 32),
                                bits.z & first_bits(left, 64), bits.w & first_bits(left, 96)};
      if (__all_sync(0xffffffffu, (seen[0] & seen[1] & seen[2] & seen[3]) == 0xffffffffu))
        softmax_tile<__half, D, false>(s_addr, o_addr, i > 0, mul, st, seen);
      else
        softmax_tile<__half, D, true>(s_addr, o_addr, i > 0, mul, st, seen);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&m->p_full[t]);
    }
    if (ok && nt > 0) ok = warp_wait(&m->o_full[t], 0, a.wait_ns, a.err);
    if (ok && works) {
      // rows of a KV head in the order of the packed rows: row i of the warp's 32 is at first + i / g * Hq + i % g
      int rw = r & ~31;
      asm volatile("" : "+r"(rw));  // nothing of this is worked out before the loop and kept in registers
      const size_t part = static_cast<size_t>(SHARED ? z : 2 * z + t) * (static_cast<size_t>(a.n_rows) * a.Hq) + h * a.g;
      const int rt = (rw + lane) / a.g;
      const size_t at = part + (static_cast<size_t>(it.row0) + it.q0 + tq * a.T + rt) * a.Hq + (rw + lane - rt * a.g);
      if (nt > 0 && *reinterpret_cast<volatile int*>(&m->bad) < lim) st.l = NAN;
      if (mine) a.part_s[at] = make_float2(st.m, st.l);
      if (nt > 0) {
        // through shared memory, so that a store writes 64 bytes of each of eight rows, not 16 of 32
        tc_fence_after();
        float* const buf = reinterpret_cast<float*>(gbase + C::kOut + t * C::kOutSlot + (warp & 3) * C::kOutWarp);
        const uint32_t has = __ballot_sync(0xffffffffu, mine);
        const size_t base_row = part + (static_cast<size_t>(it.row0) + it.q0) * a.Hq;
        float* dst[4];  // of rows 8 i + lane / 4, this lane's four channels of sixteen
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int q = rw + 8 * i + (lane >> 2), qt = q / a.g;
          dst[i] = a.part_o + (base_row + static_cast<size_t>(tq * a.T + qt) * a.Hq + (q - qt * a.g)) * D + 4 * (lane & 3);
        }
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32];
          tmem_ld32(o_addr + 32 * c, o);
          tmem_wait_ld32(o);
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              *reinterpret_cast<uint4*>(buf + lane * kOutPitch + 4 * i) =
                  make_uint4(o[16 * hf + 4 * i], o[16 * hf + 4 * i + 1], o[16 * hf + 4 * i + 2], o[16 * hf + 4 * i + 3]);
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint4 v = *reinterpret_cast<const uint4*>(buf + (8 * i + (lane >> 2)) * kOutPitch + 4 * (lane & 3));
              if ((has >> (8 * i + (lane >> 2))) & 1u) *reinterpret_cast<uint4*>(dst[i] + 32 * c + 16 * hf) = v;
            }
            __syncwarp();
          }
        }
      }
    }
  } else if (warp < 12) {
    fewer_regs<kRegsRecords>();
    const int r = tid - 256;  // this thread's key of each tile
    using R = Record<D, BITS, G>;
    const int32_t* table = a.block_table + static_cast<size_t>(it.seq) * a.max_pages;
    // record of the key of tile i; live is false outside the stretch, among the sinks, without a page
    struct Place {
      size_t rec;
      bool live;
    };
    auto look_up = [&](int i) {
      Place p{0, false};
      if (i >= n) return p;
      const int pos = k0 + 128 * i + r;
      if (pos >= k1 || pos < a.n_sink) return p;
      const uint32_t e = a.div_ps.div(static_cast<uint32_t>(pos));
      const int pg = __ldg(table + e);
      p.live = pg >= 0 && pg < a.n_pages;
      if (p.live) p.rec = (static_cast<size_t>(pg) * a.H + h) * a.div_ps.d + a.div_ps.mod(static_cast<uint32_t>(pos), e);
      return p;
    };
    bool ok = true;
    const uint32_t ks = base + C::kK, vs = base + C::kV;  // two stages of each, by the tile's parity
    auto done = [&](uint64_t* bar) {
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    };
    auto note = [&](int i, const Place& p) {  // the keys that are there
      const uint32_t seen = __ballot_sync(0xffffffffu, p.live);
      if (lane == 0) m->seen[i % kMasks][warp - 8] = seen;
    };
    // K_0 .. K_(A-1) alone, then pairs (V_j, K_(j+A)); a record is asked for as soon as its registers are free
    constexpr int A = C::kAhead;
    R kr, vr;
    Place kp = look_up(0), vp = kp, kn = look_up(1);
    kr.load(a.kcodes, a.ksz, kp.rec, kp.live);
    vr.load(a.vcodes, a.vsz, vp.rec, vp.live);
    Place v2 = kn;  // the tile behind V's
#pragma unroll
    for (int i = 0; i < A; ++i) {
      if (i < n) {
        note(i, kp);
        kr.store(ks + (i & 1) * C::kHead, r);
        done(&m->first[i]);
      }
      kp = kn;
      kr.load(a.kcodes, a.ksz, kp.rec, kp.live);
      kn = look_up(i + 2);
    }
    for (int j = 0; j < n; ++j) {
      const int s = j & 1;
      if (j >= 2) ok = warp_wait(&m->empty[s], ((j >> 1) & 1) ^ 1, a.wait_ns, a.err);
      if (ok && j == 2 - A) ok = warp_wait(&m->begun, 0, a.wait_ns, a.err);  // K_2 takes the place of K_0
      if (!ok) break;
      // a weight of zero does not hide what is not finite: where some row does not see a key (behind the first
      // token's), such a record is taken out, and the rows that see it get a total of NaN
      if (k0 + 128 * j + 127 > pos0 && vr.clear_if_bad()) atomicMin(&m->bad, k0 + 128 * j + r);
      vr.store(vs + s * C::kHead, r);
      vp = v2;
      v2 = A == 1 ? kn : kp;
      vr.load(a.vcodes, a.vsz, vp.rec, vp.live);
      if (j + A < n) {
        note(j + A, kp);
        kr.store(ks + ((j + A) & 1) * C::kHead, r);
        kp = kn;
        kr.load(a.kcodes, a.ksz, kp.rec, kp.live);
        kn = look_up(j + A + 2);
      }
      done(&m->full[s]);
    }
  } else {
    fewer_regs<kRegsIssue>();
    if (warp == 12) {
      bool ok = true;
      auto wait = [&](uint64_t* bar, uint32_t parity) { ok = ok && warp_wait(bar, parity, a.wait_ns, a.err); };
      auto scores = [&](int t, int j) {
        issue_scores<__half, D>(tmem + 128 * t, base + (SHARED ? t : 0) * C::kHead, base + C::kK + (j & 1) * C::kHead);
        tc_commit(&m->s_full[t]);
      };
      // the weights of slot t for tile j, then the scores that replace them (products run in order)
      auto turn = [&](int t, int i, int j, int next) {
        wait(&m->p_full[t], i & 1);
        if (!ok) return;
        tc_fence_after();
        issue_values<__half, D>(tmem + 256 + D * t, tmem + 128 * t, base + C::kV + (j & 1) * C::kHead, i > 0);
        if (i + 1 < n_t[t]) scores(t, next);
        else tc_commit(&m->o_full[t]);
      };
      if (SHARED) {
        wait(&m->first[0], 0);
        for (int t = 0; ok && t < 2; ++t)
          if (n_t[t] > 0) scores(t, 0);
      } else {
        for (int j = 0; j < 2 && j < n; ++j) {
          wait(&m->first[j], 0);
          if (ok) scores(j, j);
        }
      }
      if (ok) tc_commit(&m->begun);
      for (int j = 0; ok && j < n; ++j) {
        wait(&m->full[j & 1], (j >> 1) & 1);
        if (SHARED) {
          for (int t = 0; ok && t < 2; ++t)
            if (j < n_t[t]) turn(t, j, j, j + 1);
        } else if (ok) {
          turn(j & 1, j >> 1, j, j + 2);
        }
        if (ok) tc_commit(&m->empty[j & 1]);
      }
      if (!ok) {  // a wait ran out: the products in flight still end before the memory is given back
        tc_commit(&m->drain);
        warp_wait(&m->drain, 0, a.wait_ns, a.err);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 12) tmem_dealloc(tmem, 512);
}

// C fp16 values as fp32, one load.
template <int C>
__device__ __forceinline__ void ld_halves(const __half* p, float (&x)[C]) {
  static_assert(C == 2 || C == 4, "D / 32");
  uint32_t w[C / 2];
  if constexpr (C == 4) {
    const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
    w[0] = v.x, w[1] = v.y;
  } else {
    w[0] = __ldg(reinterpret_cast<const uint32_t*>(p));
  }
#pragma unroll
  for (int i = 0; i < C / 2; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    x[2 * i] = f.x, x[2 * i + 1] = f.y;
  }
}

// Sink row n of K turned to its position: this lane's C channels, in the fma order of rope_fwd.
template <int D, int C>
__device__ __forceinline__ void sink_key(const PagedArgs& a, const __half* row, int n, int lane, float (&x)[C]) {
  ld_halves<C>(row + lane * C, x);
  if (a.rope == 0) return;
  const float2* cs = reinterpret_cast<const float2*>(a.rope_cs) + static_cast<size_t>(n) * (D / 2);
  if (a.rope == 1) {
#pragma unroll
    for (int c = 0; c < C; c += 2) {
      const float2 t = __ldg(cs + (lane * C + c) / 2);
      rope_fwd(x[c], x[c + 1], t.x, t.y);
    }
  } else {
    const bool up = lane >= 16;  // channels of the upper half
    float y[C];
    ld_halves<C>(row + (lane ^ 16) * C, y);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const float2 t = __ldg(cs + (lane & 15) * C + c);
      float lo = up ? y[c] : x[c], hi = up ? x[c] : y[c];
      rope_fwd(lo, hi, t.x, t.y);
      x[c] = up ? hi : lo;
    }
  }
}

// The last sequence whose first row is at or before `row`: 32 offsets at a time. One warp.
__device__ __forceinline__ int seq_of_row(const int32_t* cu_rows, int S, int row, int lane) {
  int lo = 0, hi = S;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) >> 5, at = lo + lane * step;
    const uint32_t before = __ballot_sync(0xffffffffu, at < hi && __ldg(cu_rows + at) <= row);
    lo += before ? (31 - __clz(before)) * step : 0;
    if (!before) break;
    hi = min(hi, lo + step);
  }
  return lo;
}

// W warps per row and query head (a CTA has 8), C = D / 32 channels a lane. TILE: the parts' channels
// are in tile order. The parts of a row are joined in a fixed order: warp w takes parts w, w + W, ...,
// and warp 0 the sinks before them. A row is a chain of dependent loads (its sequence, lengths, sinks,
// statistics, sums), which is what this kernel's time is; each link is read for four sinks or parts at
// a time.
template <int D, int BITS, bool TILE, int W>
__global__ void __launch_bounds__(256) k_paged_merge(const PagedArgs a) {
  constexpr int C = D / 32;
  __shared__ float nat[8][D];
  __shared__ float wtop[8], wsum[8];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, w = warp % W;
  // below 2^31 rows and query heads in all, and at most seven warps behind them
  const uint32_t wi = W == 8 ? blockIdx.x : blockIdx.x * 8u + warp, wr = a.div_hq.div(wi);
  const int row = static_cast<int>(wr), qh = static_cast<int>(a.div_hq.mod(wi, wr));
  // Every path waits for the tiles' grid: a kernel behind this one counts on both being done.
  auto after_tiles = [] { asm volatile("griddepcontrol.wait;" ::: "memory"); };
  if (wr >= static_cast<uint32_t>(a.n_rows)) {  // the W warps of a row agree, here and below
    after_tiles();
    return;
  }
  const int lo = seq_of_row(a.cu_rows, a.S, row, lane);
  const int b = min(max(__ldg(a.cu_rows + lo), 0), a.n_rows), e = min(max(__ldg(a.cu_rows + lo + 1), b), a.n_rows);
  const int h = static_cast<int>(a.div_g.div(static_cast<uint32_t>(qh))), len = max(__ldg(a.kv_len + lo), 0);
  if (row < b || row >= e || row - b >= a.max_rows) {
    after_tiles();
    return;
  }
  // keys [0, lim)
  const int lim = min(len - (e - b) + (row - b) + 1, min(len, sat_pages(a.max_pages, static_cast<int>(a.div_ps.d))));
  const float unit = a.scale * 1.4426950408889634f;
  float top = -INFINITY, total = 0.0f, own[C];
#pragma unroll
  for (int c = 0; c < C; ++c) own[c] = 0.0f;
  if (a.n_sink > 0 && w == 0) {  // the sinks' running sums, in their own basis
    constexpr int B = 4;
    const int srow = a.sink_slot ? __ldg(a.sink_slot + lo) : lo;
    const int last = srow >= 0 && srow < a.sink_rows ? min(a.n_sink, lim) : 0;
    const size_t first = (static_cast<size_t>(max(srow, 0)) * a.H + h) * a.n_sink * D;
    float q[C];
    ld_halves<C>(a.q + row * a.q_stride + qh * D + lane * C, q);
    for (int n0 = 0; n0 < last; n0 += B) {
      float s[B], v[B][C];
#pragma unroll
      for (int i = 0; i < B; ++i) {
        const int n = n0 + i;
        s[i] = -INFINITY;
#pragma unroll
        for (int c = 0; c < C; ++c) v[i][c] = 0.0f;
        if (n >= last || (a.rope && n >= a.rope_rows)) continue;
        const int pg = __ldg(a.block_table + static_cast<size_t>(lo) * a.max_pages + a.div_ps.div(static_cast<uint32_t>(n)));
        float k[C];
        sink_key<D, C>(a, a.ksink + first + static_cast<size_t>(n) * D, n, lane, k);
        ld_halves<C>(a.vsink + first + static_cast<size_t>(n) * D + lane * C, v[i]);
        float dot = 0.0f;
#pragma unroll
        for (int c = 0; c < C; ++c) dot = fmaf(q[c], k[c], dot);
        dot = all_sum(dot) * unit;
        if (pg >= 0 && pg < a.n_pages) {
          s[i] = dot;
        } else {
#pragma unroll
          for (int c = 0; c < C; ++c) v[i][c] = 0.0f;
        }
      }
      const float mn = fmaxf(fmaxf(fmaxf(s[0], s[1]), fmaxf(s[2], s[3])), top), ref = mn == -INFINITY ? 0.0f : mn;
      const float f = exp2f(top - ref);
      top = mn;
      total *= f;
#pragma unroll
      for (int c = 0; c < C; ++c) own[c] *= f;
#pragma unroll
      for (int i = 0; i < B; ++i) {
        const float p = exp2f(s[i] - ref);
        total += p;
#pragma unroll
        for (int c = 0; c < C; ++c) own[c] = fmaf(p, v[i][c], own[c]);
      }
    }
  }
  after_tiles();
  // the stretches that hold keys of this row, an empty part (weight total 0) left out
  const size_t rows = static_cast<size_t>(a.n_rows) * a.Hq, me = static_cast<size_t>(row) * a.Hq + qh;
  const int reach = static_cast<int>(a.div_stretch.div(static_cast<uint32_t>(max(lim, 1) - 1)));  // the stretch of the last key
  const int parts = lim > 0 ? min(a.n_stretch, reach + 1) * a.part_per : 0;
  auto part = [&](int p) { return p < parts ? a.part_s[p * rows + me] : make_float2(-INFINITY, 0.0f); };
  float all_top = top;
  if constexpr (W == 1) {  // at most kNarrow parts: every lane reads the statistics
#pragma unroll 2
    for (int p = 0; p < parts; ++p) {
      const float2 s = part(p);
      all_top = fmaxf(all_top, s.y != 0.0f ? s.x : -INFINITY);
    }
  } else {
    for (int p0 = w; p0 < parts; p0 += 32 * W) {
      const float2 s = part(p0 + lane * W);
      all_top = fmaxf(all_top, all_max(s.y != 0.0f ? s.x : -INFINITY));
    }
  }
  if constexpr (W > 1) {
    if (lane == 0) wtop[warp] = all_top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < W; ++i) all_top = fmaxf(all_top, wtop[i]);
  }
  const float ref = all_top == -INFINITY ? 0.0f : all_top;
  float o[C];
  const float fs = exp2f(top - ref);
#pragma unroll
  for (int c = 0; c < C; ++c) o[c] = 0.0f, own[c] *= fs;
  total *= fs;
  if constexpr (W == 1) {
#pragma unroll 2
    for (int p = 0; p < parts; ++p) {
      const float2 s = part(p);
      if (s.y == 0.0f) continue;  // what an empty part's sums hold is not read
      const float f = exp2f(s.x - ref);
      const float* src = a.part_o + (p * rows + me) * D;
      total = fmaf(s.y, f, total);
#pragma unroll
      for (int c = 0; c < C; ++c) o[c] = fmaf(src[TILE ? tile_pos<BITS>(lane * C + c) : lane * C + c], f, o[c]);
    }
  } else for (int p0 = w; p0 < parts; p0 += 32 * W) {
    const float2 s = part(p0 + lane * W);
    const bool live = s.y != 0.0f;
    const float f = live ? exp2f(s.x - ref) : 0.0f;
    total += all_sum(live ? s.y * f : 0.0f);
    const uint32_t has = __ballot_sync(0xffffffffu, live);
    const int n = min(32, (parts - p0 + W - 1) / W);
    for (int i0 = 0; i0 < n; i0 += 4) {
      float x[4][C];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int c = 0; c < C; ++c) x[i][c] = 0.0f;
        if (i0 + i < 32 && (has >> (i0 + i)) & 1u) {  // what an empty part's sums hold is not read
          const float* src = a.part_o + (static_cast<size_t>(p0 + (i0 + i) * W) * rows + me) * D;
#pragma unroll
          for (int c = 0; c < C; ++c) x[i][c] = src[TILE ? tile_pos<BITS>(lane * C + c) : lane * C + c];
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float fi = __shfl_sync(0xffffffffu, f, (i0 + i) & 31);
#pragma unroll
        for (int c = 0; c < C; ++c) o[c] = fmaf(x[i][c], i0 + i < n ? fi : 0.0f, o[c]);
      }
    }
  }
  if constexpr (W > 1) {
#pragma unroll
    for (int c = 0; c < C; ++c) nat[warp][lane * C + c] = o[c];
    if (lane == 0) wsum[warp] = total;
    __syncthreads();
    if (w > 0) return;
#pragma unroll
    for (int i = 1; i < W; ++i) {
      total += wsum[i];
#pragma unroll
      for (int c = 0; c < C; ++c) o[c] += nat[i][lane * C + c];
    }
    __syncwarp();
  }
  if (a.rot) {
    warp_fwht<C>(o, lane);
#pragma unroll
    for (int c = 0; c < C; ++c) o[c] *= a.rscale;
  }
#pragma unroll
  for (int c = 0; c < C; ++c) nat[warp][a.vperm ? a.vperm[h * D + lane * C + c] & (D - 1) : lane * C + c] = o[c];
  __syncwarp();
  const float inv = total != 0.0f ? 1.0f / total : 0.0f;
  __half* out = a.out + row * a.out_stride + qh * D + lane * C;
#pragma unroll
  for (int c = 0; c < C; c += 2)
    *reinterpret_cast<__half2*>(out + c) = __floats2half2_rn((nat[warp][lane * C + c] + own[c]) * inv,
                                                             (nat[warp][lane * C + c + 1] + own[c + 1]) * inv);
}

// ---------------------------------------------------------------- few rows
// A decode step (max_rows * g <= 8 rows a KV head, head_dim 128, 2 or 4 bits)
// is bound by instructions, not by the tensor cores, so it keeps the codes out
// of shared-memory tiles: a warp takes blocks of 16 keys through its own ring of
// cp.async stages, masks the codes in registers and multiplies them as they
// are (mma.sync m16n8k16, fp16 in, fp32 out).
//
// A code field left at its bit of a 16-bit half is the fp16 subnormal c 2^p
// 2^-24: one mask makes an operand register (two codes). 2^-p goes into the
// query (scores) or is undone on the sums (values), both exactly; the other
// operand is kept large (queries at 2^13, weights up to 2^15) so that its terms
// stay normal. Every query value and every weight enters as two fp16 terms, hi
// and lo, one column each (about 22 bits); fp32 statistics and sums.
//
//   scores: s = S_g sum_j q'_j c_j + Z_g sum_j q'_j per quantization group
//           (A = 16 keys x 16 channels of codes, B = queries, N = 8: 4 rows x hi, lo)
//   values: sum_n p_n y_n = sum_n (p_n S_n) c_n + sum_n p_n Z_n
//           (A = 16 channels x 16 keys of codes, B = weights)
// A weight p S is at most 2^15: the reference m follows s + log2 S (S >= 2^-30)
// and is raised when that exceeds it by 2^8; p = 2^(s - m + 7).
//
// Measured, 2 bits, one group, 32 / 8 heads: 64 sequences of up to 8191 keys 87 us (159
// MB, 1.8 TB/s), four of 32768 keys 45 us, each with its merge. 253 warp instructions per
// 16 keys, 16 of them products, and 3500 a CTA: ALU pipe 52 to 55 %, issue 56 to 57 %,
// DRAM 25 %; 118 registers, nothing spilled.
constexpr int kFewWarps = 4;
constexpr int kFewThreads = 32 * kFewWarps;
constexpr int kBlock = 16;
constexpr int kFewStep = kFewWarps * kBlock;  // keys between a warp's blocks
constexpr float kFewUp = 7.0f;
constexpr float kFewMinS = 9.3132257e-10f;  // 2^-30

// Which codes a lane masks. Keys (scores): lane quarter tig holds kWords words of a
// row, kPairs register pairs (code, code at +16 bits) each; pair p sits at bit
// `bit` of the word, or of the word shifted right by `down`; its channels are ch
// and ch + kFar. Values: lane group gr holds word(i) of two keys, merged to
// registers of 16-bit halves; m-tile mt takes a code for row gr and one for row gr + 8.
template <int BITS, int G>
struct Map;
template <int G>
struct Map<2, G> {
  static constexpr bool kFine = G == 32;  // two words a group
  static constexpr int kWords = kFine ? 4 : 2, kPairs = kFine ? 4 : 8, kFar = 8;
  static __device__ __forceinline__ int kword(int i, int tig) {
    return kFine ? 2 * i + (tig & 1) : G == 128 ? 2 * tig + i : tig + 4 * i;  // one group: adjacent words, one load
  }
  static __device__ __forceinline__ uint32_t kopen(uint32_t w, int tig) { return kFine ? w >> (8 * (tig >> 1)) : w; }
  static __device__ __forceinline__ int kch(int i, int p, int tig) {
    return 16 * kword(i, tig) + p + (kFine ? 4 * (tig >> 1) : 0);
  }
  static constexpr int kDown = 10;  // pairs 5 .. 7 are read after this shift
  static __host__ __device__ constexpr bool shifted(int p) { return p >= 5; }
  static __host__ __device__ constexpr int bit(int p) { return 2 * (p >= 5 ? p - 5 : p); }
  // a value's code c: from the register shifted by vshift (left if positive), at bit vbit
  static __device__ __forceinline__ uint32_t vshift(uint32_t y, int k) { return k == 0 ? y << 4 : k == 1 ? y : y >> 6; }
  static __host__ __device__ constexpr int vset(int c) { return c < 2 ? 0 : c < 5 ? 1 : 2; }
  static __host__ __device__ constexpr int vbit(int c) { return c < 2 ? 4 + 2 * c : c < 5 ? 2 * c : 2 * c - 6; }
  static __host__ __device__ constexpr int group(int i) { return kFine ? i : i * 64 / G; }
  // values
  static constexpr int kVWords = G == 128 ? 1 : G == 64 ? 2 : 4;
  static constexpr int kVRegs = G == 128 ? 2 : kVWords;
  static __device__ __forceinline__ int vword(int i, int gr) {
    return G == 128 ? gr : G == 64 ? 4 * i + (gr & 3) : 2 * i + (gr & 1);
  }
  // register r from the two keys' words
  static __device__ __forceinline__ uint32_t vopen(int r, uint32_t a, uint32_t b, int gr) {
    if (G == 128) return __byte_perm(a, b, r ? 0x7632 : 0x5410);
    const bool hi = G == 64 ? gr >> 2 : (gr >> 1) & 1;
    const uint32_t y = __byte_perm(a, b, hi ? 0x7632 : 0x5410);
    return G == 64 ? y : y >> (8 * (gr >> 2));
  }
  static __host__ __device__ constexpr int vwordof(int r) { return G == 128 ? 0 : r; }
  static __host__ __device__ constexpr int vreg(int mt, int row8) { return G == 128 ? row8 : G == 64 ? mt / 4 : mt / 2; }
  static __host__ __device__ constexpr int vcode(int mt, int row8) {
    return G == 128 ? mt : G == 64 ? mt % 4 + 4 * row8 : mt % 2 + 2 * row8;
  }
  static __device__ __forceinline__ int vch(int mt, int row8, int gr) {
    if (G == 128) return 16 * gr + 8 * row8 + mt;
    if (G == 64) return 16 * vword(mt / 4, gr) + 8 * (gr >> 2) + mt % 4 + 4 * row8;
    return 16 * vword(mt / 2, gr) + 8 * ((gr >> 1) & 1) + 4 * (gr >> 2) + mt % 2 + 2 * row8;
  }
  static __host__ __device__ constexpr int vgroup(int mt) { return G == 128 ? 0 : G == 64 ? mt / 4 : mt / 2; }
};
template <int G>
struct Map<4, G> {
  static constexpr bool kFine = G == 32;
  static constexpr int kWords = 4, kPairs = 4, kFar = 4, kDown = 8;
  static __device__ __forceinline__ int kword(int i, int tig) { return G == 128 ? 4 * tig + i : tig + 4 * i; }
  static __device__ __forceinline__ uint32_t kopen(uint32_t w, int) { return w; }
  static __device__ __forceinline__ int kch(int i, int p, int tig) { return 8 * kword(i, tig) + p; }
  static __host__ __device__ constexpr bool shifted(int p) { return p >= 2; }
  static __host__ __device__ constexpr int bit(int p) { return 4 * (p & 1); }
  static __device__ __forceinline__ uint32_t vshift(uint32_t y, int k) { return k == 0 ? y << 4 : k == 1 ? y : y >> (4 * k - 4); }
  static __host__ __device__ constexpr int vset(int c) { return c; }
  static __host__ __device__ constexpr int vbit(int) { return 4; }
  static __host__ __device__ constexpr int group(int i) { return 32 * i / G; }
  static constexpr int kVWords = kFine ? 4 : 2, kVRegs = 4;
  static __device__ __forceinline__ int vword(int i, int gr) { return kFine ? 4 * i + (gr & 3) : gr + 8 * i; }
  static __device__ __forceinline__ uint32_t vopen(int r, uint32_t a, uint32_t b, int gr) {
    const bool hi = kFine ? gr >> 2 : r & 1;
    return __byte_perm(a, b, hi ? 0x7632 : 0x5410);
  }
  static __host__ __device__ constexpr int vwordof(int r) { return kFine ? r : r / 2; }
  static __host__ __device__ constexpr int vreg(int mt, int row8) { return kFine ? mt / 2 : 2 * (mt / 4) + row8; }
  static __host__ __device__ constexpr int vcode(int mt, int row8) { return kFine ? mt % 2 + 2 * row8 : mt % 4; }
  static __device__ __forceinline__ int vch(int mt, int row8, int gr) {
    return kFine ? 8 * vword(mt / 2, gr) + 4 * (gr >> 2) + mt % 2 + 2 * row8 : 8 * vword(mt / 4, gr) + 4 * row8 + mt % 4;
  }
  static __host__ __device__ constexpr int vgroup(int mt) { return kFine ? mt / 2 : G == 64 ? mt / 4 : 0; }
};

template <int BITS, int G>
struct FewCfg {
  static constexpr int kRec = 128 * BITS / 8, kNG = 128 / G;
  static constexpr int kStage = 2 * kBlock * (kRec + 4 * kNG) + 16;  // key codes, value codes, their (S, Z), key mask
  static constexpr int kStages = BITS == 2 ? 6 : 4;
  static constexpr int kSmem = kFewWarps * kStages * kStage;
};

__device__ __forceinline__ void cp_async8(uint32_t dst, const void* src, uint32_t n) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void mma_h(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                      uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// x as fp16 hi + lo (hi in the low half).
__device__ __forceinline__ uint32_t hi_lo(float x) {
  const __half hi = __float2half_rn(x);
  const __half lo = __float2half_rn(x - __half2float(hi));
  return static_cast<uint32_t>(__half_as_ushort(hi)) | (static_cast<uint32_t>(__half_as_ushort(lo)) << 16);
}
__device__ __forceinline__ float2 h2f2(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2*>(&w)); }

// NT: column tiles, 4 rows each. One CTA per (stretch of keys, KV head, sequence).
template <int BITS, int G, int NT>
__global__ void __launch_bounds__(kFewThreads, NT == 1 ? 4 : 2) k_paged_few(const PagedArgs a) {
  using C = FewCfg<BITS, G>;
  using M = Map<BITS, G>;
  constexpr int D = 128, NG = C::kNG, RB = C::kRec, ST = C::kStages, R = 4 * NT;
  extern __shared__ __align__(128) uint8_t few_smem[];
  __shared__ float qrow[R][D];
  __shared__ float qmul[R], qsum[R][NG];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int gr = lane >> 2, tig = lane & 3;
  unsigned rest = blockIdx.x;
  const int z = static_cast<int>(rest % static_cast<unsigned>(a.n_stretch));
  rest /= static_cast<unsigned>(a.n_stretch);
  const int h = static_cast<int>(rest % static_cast<unsigned>(a.H));
  const int s = static_cast<int>(rest / static_cast<unsigned>(a.H));
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int row0 = min(max(__ldg(a.cu_rows + s), 0), a.n_rows);
  const int m_rows = min(max(__ldg(a.cu_rows + s + 1), row0), a.n_rows) - row0;
  const int tokens = min(m_rows, a.max_rows);
  const int cached = max(__ldg(a.kv_len + s), 0);
  const int kv = min(cached, sat_pages(a.max_pages, static_cast<int>(a.div_ps.d)));
  const int pos0 = cached - m_rows;
  const long long kb = static_cast<long long>(z) * a.stretch;
  const long long ke = z + 1 == a.n_stretch ? 0x7fffffffll : kb + a.stretch;
  const int k0 = static_cast<int>(min(kb, 0x7fffffffll));
  const int k1 = static_cast<int>(min(ke, static_cast<long long>(min(kv, pos0 + tokens))));
  if (tokens == 0 || k1 <= k0) return;  // no row sees a key here: the merge does not look
  const int n_rows = tokens * a.g;      // at most R
  const int blocks = (k1 - k0 + kBlock - 1) / kBlock;
  const int mine = blocks > warp ? (blocks - warp + kFewWarps - 1) / kFewWarps : 0;  // blocks warp + kFewWarps i

  // ---- the ring: lane copies half a record of key lane / 2, and its (S, Z) (even lanes keys, odd lanes values)
  const uint32_t wbase = smem_u32(few_smem) + warp * (ST * C::kStage);
  const uint8_t* const wgen = few_smem + warp * (ST * C::kStage);
  const int32_t* table = a.block_table + static_cast<size_t>(s) * a.max_pages;
  const int kt = lane >> 1, kh = lane & 1;
  // this lane's key of the next block to look up: position, entry of the table, offset in the page
  int pos = k0 + warp * kBlock + kt, entry = static_cast<int>(a.div_ps.div(static_cast<uint32_t>(pos)));
  int off = static_cast<int>(a.div_ps.mod(static_cast<uint32_t>(pos), entry));
  const int ps = static_cast<int>(a.div_ps.d);
  struct Key {
    int page, off;
  };
  auto look_up = [&](Key& k) {  // the page of a key that is not to be read is -1
    k.page = -1;
    k.off = off;
    if (pos < k1 && pos >= a.n_sink) {
      const int pg = __ldg(table + entry);
      k.page = pg < a.n_pages ? pg : -1;
    }
    pos = min(pos, k1) + kFewStep;
    entry += a.step_page;
    off += a.step_off;
    if (off >= ps) off -= ps, ++entry;
  };
  const uint32_t page_bytes = static_cast<uint32_t>(a.H * ps) * RB;  // below 2^31
  const size_t head_at = static_cast<size_t>(h) * ps * RB + kh * (RB / 2);
  const uint8_t* const kc0 = a.kcodes + head_at;
  const uint8_t* const vc0 = a.vcodes + head_at;
  const uint8_t* const z0 = reinterpret_cast<const uint8_t*>((kh ? a.vsz : a.ksz) + static_cast<size_t>(h) * ps * NG);
  auto issue = [&](uint32_t sb, const Key& k) {  // a block of this warp into the stage at sb
    const bool live = k.page >= 0;
    const uint32_t pg = live ? k.page : 0, o = live ? k.off : 0, n = live ? 16u : 0u;
    const size_t at = static_cast<uint64_t>(pg) * page_bytes + o * static_cast<uint32_t>(RB);
    const uint32_t to = sb + kt * RB + kh * (RB / 2);
#pragma unroll
    for (int c = 0; c < RB / 32; ++c) {
      cp_async16(to + 16 * c, kc0 + at + 16 * c, n);
      cp_async16(to + kBlock * RB + 16 * c, vc0 + at + 16 * c, n);
    }
    const uint8_t* sz = z0 + static_cast<uint64_t>(pg) * (page_bytes / (RB / (4 * NG))) + o * (4u * NG);
    const uint32_t zt = sb + 2 * kBlock * RB + (2 * kt + kh) * 4 * NG;
    if constexpr (NG == 1) cp_async4(zt, sz, live ? 4u : 0u);
    else if constexpr (NG == 2) cp_async8(zt, sz, live ? 8u : 0u);
    else cp_async16(zt, sz, n);
    const uint32_t seen = __ballot_sync(0xffffffffu, live);  // two bits a key
    if (lane == 0) asm volatile("st.shared.u32 [%0], %1;" ::"r"(sb + 2 * kBlock * (RB + 4 * NG)), "r"(seen) : "memory");
  };
  Key next;
#pragma unroll
  for (int i = 0; i < ST; ++i) {
    look_up(next);
    if (i < mine) issue(wbase + i * C::kStage, next);
    cp_async_commit();
  }
  look_up(next);

  // ---- query rows: rotated, scaled by a power of two to [2^13, 2^14)
  for (int r = warp; r < R; r += kFewWarps) {
    float x[4], top = 0.0f;
    const int tok = r / a.g, j = r - tok * a.g;
    const __half* qp = a.q + (static_cast<int64_t>(row0) + tok) * a.q_stride + (h * a.g + j) * D;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int ch = 4 * lane + c;
      x[c] = r < n_rows ? __half2float(qp[a.kperm ? a.kperm[h * D + ch] & (D - 1) : ch]) : 0.0f;
    }
    if (a.rot) {
      warp_fwht<4>(x, lane);
#pragma unroll
      for (int c = 0; c < 4; ++c) x[c] *= a.rscale;
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) top = fmaxf(top, fabsf(x[c]));
    top = all_max(top);
    const int e = top > 0.0f && top < INFINITY ? static_cast<int>(__float_as_uint(top) >> 23) - 127 : 0;
    const float up = __uint_as_float(static_cast<uint32_t>(127 + 13 - e) << 23);
    float sum = 0.0f;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      qrow[r][4 * lane + c] = x[c] * up;
      sum += x[c];
    }
    // lanes of a group: G / 4
#pragma unroll
    for (int o = 1; o < 32; o <<= 1)
      if (4 * o < G) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const float unit = a.scale * 1.4426950408889634f;
    if (lane % (G / 4) == 0) qsum[r][lane / (G / 4)] = sum * unit;
    if (lane == 0) qmul[r] = unit * __uint_as_float(static_cast<uint32_t>(127 - 13 + e) << 23) * 16777216.0f;
  }
  __syncthreads();
  // B fragments of the scores: column gr of tile t is row 4 t + gr / 2, term gr & 1. Each warp makes two k-steps.
  __shared__ uint2 frag[NT][8][32];
  {
    constexpr int PK = M::kPairs / 2;  // k-steps of a word
    uint32_t b2[NT][2];
#pragma unroll
    for (int ks = 0; ks < 8; ++ks) {
      if (ks % kFewWarps != warp) continue;
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const float* q = qrow[4 * t + (gr >> 1)];
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const int p = 2 * (ks % PK) + b, ch = M::kch(ks / PK, p, tig);
          const float down = 1.0f / static_cast<float>(1 << M::bit(p));
          b2[t][b] = __byte_perm(hi_lo(q[ch] * down), hi_lo(q[ch + M::kFar] * down), (gr & 1) ? 0x7632 : 0x5410);
        }
        frag[t][ks][lane] = make_uint2(b2[t][0], b2[t][1]);
      }
    }
  }
  __syncthreads();
  uint32_t bq[8][NT][2];
  float mul[NT], qz[NT][NG];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
#pragma unroll
    for (int ks = 0; ks < 8; ++ks) {
      const uint2 f = frag[t][ks][lane];
      bq[ks][t][0] = f.x;
      bq[ks][t][1] = f.y;
    }
    mul[t] = qmul[4 * t + tig];
#pragma unroll
    for (int k = 0; k < NG; ++k) qz[t][k] = qsum[4 * t + tig][k];
  }
  int lim[NT];  // keys [0, lim) are seen by this lane's row of each tile
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int r = 4 * t + tig;
    lim[t] = r < n_rows ? pos0 + r / a.g + 1 : 0x7fffffff;
  }

  // low: the lowest score of the keys that the row sees. A key whose scale or zero is not finite has channels of
  // both infinities, or NaN, and no score; S sum q'c + Z sum q' alone could be -infinity, which would hide the key.
  float acc[8][NT][4], mr[NT], lr[NT], zr[NT][NG], low[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    mr[t] = -INFINITY;
    low[t] = INFINITY;
    lr[t] = 0.0f;
#pragma unroll
    for (int k = 0; k < NG; ++k) zr[t][k] = 0.0f;
#pragma unroll
    for (int mt = 0; mt < 8; ++mt)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[mt][t][e] = 0.0f;
  }
  const int srcA = 8 * tig + (gr >> 1), srcB = srcA + 4;
  const uint32_t sel = (gr & 1) ? 0x7632u : 0x5410u;

  uint32_t stage = 0;
  int n0 = k0 + warp * kBlock, bad = 0x7fffffff;  // the first value record met that is not finite, see below
  for (int i = 0; i < mine; ++i, n0 += kFewStep) {
    cp_async_wait_group<ST - 1>();
    __syncwarp();
    const uint8_t* st = wgen + stage;
    const uint8_t* sz = st + 2 * kBlock * RB;  // [key][its groups' (S, Z) of the key, then of the value]
    const uint32_t seen = *reinterpret_cast<const uint32_t*>(st + 2 * kBlock * (RB + 4 * NG));
    // ---- scores of keys gr and gr + 8
    float sc[NG][NT][4];
#pragma unroll
    for (int k = 0; k < NG; ++k)
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[k][t][e] = 0.0f;
#pragma unroll
    for (int w = 0; w < M::kWords; ++w) {
      const uint32_t wa = M::kopen(*reinterpret_cast<const uint32_t*>(st + gr * RB + 4 * M::kword(w, tig)), tig);
      const uint32_t wb = M::kopen(*reinterpret_cast<const uint32_t*>(st + (gr + 8) * RB + 4 * M::kword(w, tig)), tig);
      const uint32_t da = wa >> M::kDown, db = wb >> M::kDown;
#pragma unroll
      for (int p = 0; p < M::kPairs; p += 2) {
        constexpr uint32_t F = (1u << BITS) - 1u;
        const uint32_t m0 = (F | F << 16) << M::bit(p), m1 = (F | F << 16) << M::bit(p + 1);
        const uint32_t a0 = (M::shifted(p) ? da : wa) & m0, a1 = (M::shifted(p) ? db : wb) & m0;
        const uint32_t a2 = (M::shifted(p + 1) ? da : wa) & m1, a3 = (M::shifted(p + 1) ? db : wb) & m1;
        const int ks = w * (M::kPairs / 2) + p / 2;
#pragma unroll
        for (int t = 0; t < NT; ++t) mma_h(sc[M::group(w)][t], a0, a1, a2, a3, bq[ks][t][0], bq[ks][t][1]);
      }
    }
    uint32_t ka[NG], kb2[NG], va[NG], vb[NG];
#pragma unroll
    for (int k = 0; k < NG; ++k) {
      ka[k] = *reinterpret_cast<const uint32_t*>(sz + (2 * gr * NG + k) * 4);
      kb2[k] = *reinterpret_cast<const uint32_t*>(sz + (2 * (gr + 8) * NG + k) * 4);
      va[k] = *reinterpret_cast<const uint32_t*>(sz + ((2 * gr + 1) * NG + k) * 4);
      vb[k] = *reinterpret_cast<const uint32_t*>(sz + ((2 * (gr + 8) + 1) * NG + k) * 4);
    }
    // A weight of zero does not hide what is not finite: in the blocks with keys that some row does not see,
    // such a record is taken out, and the rows that see it get a total of NaN.
    if (n0 + kBlock > pos0 + 1) {
      auto clear = [&](uint32_t (&z)[NG], int key) {
        bool out = false;
#pragma unroll
        for (int k = 0; k < NG; ++k) out |= (z[k] & 0x7c00u) == 0x7c00u || (z[k] & 0x7c000000u) == 0x7c000000u;
        if (!out) return;
#pragma unroll
        for (int k = 0; k < NG; ++k) z[k] = 0;
        bad = min(bad, key);
      };
      clear(va, n0 + gr);
      clear(vb, n0 + gr + 8);
    }
    // log2 of the largest value scale of each key, for the range of its weights
    float ta = kFewMinS, tb = kFewMinS;
    float2 va2[NG], vb2[NG];
#pragma unroll
    for (int k = 0; k < NG; ++k) {
      va2[k] = h2f2(va[k]);
      vb2[k] = h2f2(vb[k]);
      ta = fmaxf(ta, fabsf(va2[k].x));
      tb = fmaxf(tb, fabsf(vb2[k].x));
    }
    float lga, lgb;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(lga) : "f"(ta));
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(lgb) : "f"(tb));
    uint32_t wa2[NT][NG], wb2[NT][NG];
    float sa[NT], sb[NT];
    bool raise = false;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      sa[t] = sb[t] = 0.0f;
#pragma unroll
      for (int k = 0; k < NG; ++k) {
        const float2 za = h2f2(ka[k]), zb = h2f2(kb2[k]);
        sa[t] = fmaf(za.x * mul[t], sc[k][t][0] + sc[k][t][1], fmaf(za.y, qz[t][k], sa[t]));
        sb[t] = fmaf(zb.x * mul[t], sc[k][t][2] + sc[k][t][3], fmaf(zb.y, qz[t][k], sb[t]));
      }
      float la = sa[t], lb = sb[t];
      if (seen != 0xffffffffu || n0 + kBlock > lim[t]) {
        if (!((seen >> (2 * gr)) & 1u) || n0 + gr >= lim[t]) sa[t] = -INFINITY, la = INFINITY;
        if (!((seen >> (2 * gr + 16)) & 1u) || n0 + gr + 8 >= lim[t]) sb[t] = -INFINITY, lb = INFINITY;
      }
      low[t] = fminf(low[t], fminf(la, lb));
      raise |= fmaxf(sa[t] + lga, sb[t] + lgb) > mr[t] + kRaise;
    }
    if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        float top = fmaxf(sa[t] + lga, sb[t] + lgb);
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
        if (top > mr[t] + kRaise) {  // the same for the eight lanes of a row
          const float f = exp2_fast(mr[t] - top);
          mr[t] = top;
          lr[t] *= f;
#pragma unroll
          for (int k = 0; k < NG; ++k) zr[t][k] *= f;
#pragma unroll
          for (int mt = 0; mt < 8; ++mt)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[mt][t][e] *= f;
        }
      }
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const float ref = mr[t] == -INFINITY ? 0.0f : kFewUp - mr[t];
      const float pa = exp2_fast(sa[t] + ref), pb = exp2_fast(sb[t] + ref);
      lr[t] += pa + pb;
#pragma unroll
      for (int k = 0; k < NG; ++k) {
        zr[t][k] = fmaf(pa, va2[k].y, fmaf(pb, vb2[k].y, zr[t][k]));
        const uint32_t xa = hi_lo(pa * va2[k].x), xb = hi_lo(pb * vb2[k].x);
        // keys 2 tig, 2 tig + 1 (and + 8) of column gr
        wa2[t][k] = __byte_perm(__shfl_sync(0xffffffffu, xa, srcA), __shfl_sync(0xffffffffu, xa, srcB), sel);
        wb2[t][k] = __byte_perm(__shfl_sync(0xffffffffu, xb, srcA), __shfl_sync(0xffffffffu, xb, srcB), sel);
      }
    }
    // ---- values
    {
      const uint8_t* v0 = st + kBlock * RB + 2 * tig * RB;
      uint32_t y[2][M::kVRegs];
#pragma unroll
      for (int w = 0; w < M::kVWords; ++w) {
        const int at = 4 * M::vword(w, gr);
        const uint32_t u0 = *reinterpret_cast<const uint32_t*>(v0 + at), u1 = *reinterpret_cast<const uint32_t*>(v0 + RB + at);
        const uint32_t u8 = *reinterpret_cast<const uint32_t*>(v0 + 8 * RB + at), u9 = *reinterpret_cast<const uint32_t*>(v0 + 9 * RB + at);
#pragma unroll
        for (int r = 0; r < M::kVRegs; ++r)
          if (M::vwordof(r) == w) {
            y[0][r] = M::vopen(r, u0, u1, gr);
            y[1][r] = M::vopen(r, u8, u9, gr);
          }
      }
#pragma unroll
      for (int mt = 0; mt < 8; ++mt) {
        constexpr uint32_t F = (1u << BITS) - 1u;
        uint32_t x[2][2];  // [row gr / gr + 8][keys 2 tig / + 8]
#pragma unroll
        for (int r8 = 0; r8 < 2; ++r8)
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            const int c = M::vcode(mt, r8), r = M::vreg(mt, r8);
            x[r8][b] = M::vshift(y[b][r], M::vset(c)) & ((F | F << 16) << M::vbit(c));
          }
#pragma unroll
        for (int t = 0; t < NT; ++t)
          mma_h(acc[mt][t], x[0][0], x[1][0], x[0][1], x[1][1], wa2[t][M::vgroup(mt)], wb2[t][M::vgroup(mt)]);
      }
    }
    __syncwarp();
    if (i + ST < mine) issue(wbase + stage, next);  // the stage just read
    cp_async_commit();
    look_up(next);
    stage = stage == (ST - 1) * C::kStage ? 0u : stage + C::kStage;
  }
  cp_async_wait_all();

  // ---- every warp leaves a part of its own, channels in their natural order
  const size_t part = static_cast<size_t>(z * kFewWarps + warp) * (static_cast<size_t>(a.n_rows) * a.Hq);
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    // an infinite reference (a value scale that is infinite, on a key all rows see) leaves every weight zero, and
    // a part without weights would pass for an empty one
    if (bad < lim[t] || mr[t] == INFINITY || low[t] == -INFINITY) lr[t] = NAN;
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      lr[t] += __shfl_xor_sync(0xffffffffu, lr[t], o);
#pragma unroll
      for (int k = 0; k < NG; ++k) zr[t][k] += __shfl_xor_sync(0xffffffffu, zr[t][k], o);
    }
    const int r = 4 * t + tig;
    if (r >= n_rows) continue;
    const size_t at = part + (static_cast<size_t>(row0) + r / a.g) * a.Hq + h * a.g + r % a.g;
    if (gr == 0) a.part_s[at] = make_float2(mr[t] - kFewUp, lr[t]);
    if (lr[t] == 0.0f) continue;  // the merge does not read on
#pragma unroll
    for (int mt = 0; mt < 8; ++mt)
#pragma unroll
      for (int r8 = 0; r8 < 2; ++r8) {  // the zeros' part is the same for the channels of a group
        const float up = 16777216.0f / static_cast<float>(1 << M::vbit(M::vcode(mt, r8)));
        acc[mt][t][2 * r8] = fmaf(acc[mt][t][2 * r8] + acc[mt][t][2 * r8 + 1], up, zr[t][M::vgroup(mt)]);
      }
    float* dst = a.part_o + at * D;
    constexpr int RUN = G == 128 && BITS == 2 ? 8 : G == 32 ? 2 : 4;  // neighbouring channels in neighbouring m-tiles
#pragma unroll
    for (int mt = 0; mt < 8; mt += RUN)
#pragma unroll
      for (int r8 = 0; r8 < 2; ++r8) {
        float* p = dst + M::vch(mt, r8, gr);
        if constexpr (RUN == 2) {
          *reinterpret_cast<float2*>(p) = f2(acc[mt][t][2 * r8], acc[mt + 1][t][2 * r8]);
        } else {
#pragma unroll
          for (int i = 0; i < RUN; i += 4)
            reinterpret_cast<float4*>(p)[i / 4] = make_float4(acc[mt + i][t][2 * r8], acc[mt + i + 1][t][2 * r8],
                                                              acc[mt + i + 2][t][2 * r8], acc[mt + i + 3][t][2 * r8]);
        }
      }
  }
}

// The SMs that work is cut for. A constant, not the device's count: the workspace's size follows from the cut, and its
// query is a pure function that needs no device. On any other count every result is the same, only the cut is less apt.
constexpr int kPlanSms = 148;
// How a call's work is cut: row tiles, and stretches of keys per tile.
struct Plan {
  bool shared, few;
  int T, stretch, n_stretch, n_parts;
  long long tiles;
};
Plan make_plan(const kvq_desc& d, int q_heads, int n_seqs, int n_rows, int max_rows, int max_kv) {
  const int heads = d.heads;
  Plan p{};
  const int g = q_heads / heads;
  p.T = 128 / g;
  // The few-rows kernel where it has a form: its code maps are for 128 channels and codes that do not straddle words,
  // and more than eight rows would need a third column tile (the second takes 190 to 229 registers). At 2 bits 64
  // ragged sequences took 278 us through tiles and take 87 here. What it has no form for takes tiles of 128 rows for
  // its few: the same batch 323 us at 3 bits, 241 at 64 channels, 323 with 16 rows a head. The rule looks at the whole
  // call: one sequence with more rows sends all of them through tiles.
  p.few = d.head_dim == 128 && d.bits != 3 && static_cast<long long>(max_rows) * g <= 8 &&
          static_cast<long long>(d.heads) * d.t_cap * 64 < (1ll << 31);  // a page's codes in 32 bits
  p.shared = max_rows > p.T;
  const long long tt = p.shared ? 2 * p.T : p.T;
  const long long by_rows = n_rows / tt + n_seqs, by_max = n_seqs * ((max_rows + tt - 1) / tt);
  p.tiles = p.few ? n_seqs : by_rows < by_max ? by_rows : by_max;
  // Few rows: eight CTAs an SM (four at a time), so that ragged sequences even out; 64 sequences of up
  // to 8192 keys took 107 us with four an SM and 85 with eight, four of 32768 keys 43 and 45 (before the check of
  // infinite keys, which costs the first 1 us). Tiles, each
  // CTA with about 20000 clocks besides its keys: one CTA an SM at most where all sequences have the most
  // rows (512 rows on 16384 keys took 212 us so, 269, 227 and 234 with three, four and six stretches),
  // about two where they are ragged (twelve sequences of 1 to 131 rows on up to 8000 keys took 201 us with
  // one stretch, 178 with two or three, 193 with six).
  const long long all = p.tiles * heads, keys = max_kv > 0 ? max_kv : 1;
  long long n = all <= 0 ? 1 : p.few ? 8 * kPlanSms / all : by_rows < by_max ? (2 * kPlanSms + all - 1) / all : kPlanSms / all;
  const long long most = (keys + 511) / 512;  // of at least 512 keys
  n = n < 1 ? 1 : n > most ? most : n;
  if (n > 256) n = 256;
  long long len = (keys + n - 1) / n;
  len = (len + 255) / 256 * 256;
  p.stretch = static_cast<int>(len > 0x40000000ll ? 0x40000000ll : len);
  p.n_stretch = static_cast<int>((keys + p.stretch - 1) / p.stretch);
  if (p.n_stretch < 1) p.n_stretch = 1;
  p.n_parts = p.n_stretch * (p.few ? kFewWarps : p.shared ? 1 : 2);
  return p;
}

template <int D, int BITS, int G, bool SHARED>
kvq_status run_tiles(const PagedArgs& a, long long grid, cudaStream_t st) {
  constexpr uint32_t smem = Cfg<D, SHARED>::kSmem;
  const void* fn = reinterpret_cast<const void*>(k_paged_tiles<D, BITS, G, SHARED>);
  if (!set_smem_once(fn, smem) || !split_fits(fn, kRegsLaunch)) return KVQ_ERR_CUDA;
  k_paged_tiles<D, BITS, G, SHARED><<<static_cast<unsigned>(grid), kThreads, smem, st>>>(a);
  return launch_status();
}

template <int BITS, int G, int NT>
kvq_status run_few(const PagedArgs& a, long long grid, cudaStream_t st) {
  constexpr int smem = FewCfg<BITS, G>::kSmem;
  if (!set_smem_once(reinterpret_cast<const void*>(k_paged_few<BITS, G, NT>), smem)) return KVQ_ERR_CUDA;
  k_paged_few<BITS, G, NT><<<static_cast<unsigned>(grid), kFewThreads, smem, st>>>(a);
  return launch_status();
}

// Eight warps a row where there are more parts than a warp should read one after the other. With one warp and with
// eight, whole calls: 8 parts 13.7 and 14.4 us (16 sequences of 1000 keys, a token each), 32.3 and 49.1 (100 rows on
// 4000 keys); 12 parts 17.9 and 15.4, 16 parts 21.7 and 17.3 (1500 and 2000 keys).
constexpr int kNarrow = 8;
template <int D, int BITS, bool TILE>
kvq_status run_merge(const PagedArgs& a, cudaStream_t st) {
  const bool wide = a.n_parts > kNarrow;
  cudaLaunchConfig_t cfg{};
  const long long warps = static_cast<long long>(a.n_rows) * a.Hq * (wide ? 8 : 1);
  cfg.gridDim = dim3(static_cast<unsigned>((warps + 7) / 8));
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if ((wide ? cudaLaunchKernelEx(&cfg, k_paged_merge<D, BITS, TILE, 8>, a)
            : cudaLaunchKernelEx(&cfg, k_paged_merge<D, BITS, TILE, 1>, a)) != cudaSuccess)
    return KVQ_ERR_CUDA;
  return launch_status();
}

template <int D, int BITS, int G>
kvq_status run(const PagedArgs& a, const Plan& p, cudaStream_t st) {
  const long long grid = p.tiles * a.H * a.n_stretch;
  if (grid >= (1ll << 31)) return KVQ_ERR_UNSUPPORTED;
  kvq_status s;
  if constexpr (D == 128 && BITS != 3) {
    s = p.few ? (a.max_rows * a.g <= 4 ? run_few<BITS, G, 1>(a, grid, st) : run_few<BITS, G, 2>(a, grid, st))
              : p.shared ? run_tiles<D, BITS, G, true>(a, grid, st) : run_tiles<D, BITS, G, false>(a, grid, st);
  } else {
    s = p.shared ? run_tiles<D, BITS, G, true>(a, grid, st) : run_tiles<D, BITS, G, false>(a, grid, st);
  }
  if (s != KVQ_OK) return s;
  if constexpr (D == 128 && BITS != 3) {
    if (p.few) return run_merge<D, BITS, false>(a, st);
  }
  return run_merge<D, BITS, true>(a, st);
}

size_t align256(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }

}  // namespace

size_t attend_paged_workspace_bytes(const kvq_desc& dk, int q_heads, const kvq_paged& pg, int max_rows, int max_kv) {
  const Plan p = make_plan(dk, q_heads, pg.n_seqs, pg.n_rows, max_rows, max_kv);
  const size_t rows = static_cast<size_t>(pg.n_rows) * q_heads * p.n_parts;
  return align256(rows * dk.head_dim * 4) + align256(rows * 8) + 256;
}

kvq_status launch_attend_paged(const kvq_desc& dk, const kvq_desc&, const void* q, int64_t q_stride, int q_heads,
                               const kvq_packed& kc, const kvq_tables& tk, const kvq_packed& vc, const kvq_tables& tv,
                               const kvq_paged& pg, int max_rows, int max_kv, float scale, void* out,
                               int64_t out_stride, void* ws, cudaStream_t st, const LaunchCtx& ctx) {
  const Plan p = make_plan(dk, q_heads, pg.n_seqs, pg.n_rows, max_rows, max_kv);
  PagedArgs a{};
  a.S = pg.n_seqs;
  a.n_rows = pg.n_rows;
  a.max_pages = pg.max_pages;
  a.sink_rows = pg.sink_rows;
  a.H = dk.heads;
  a.Hq = q_heads;
  a.g = q_heads / dk.heads;
  a.T = p.T;
  a.n_pages = dk.batch;
  a.n_sink = dk.n_sink;
  a.rope = dk.rope;
  a.rope_rows = tk.rope_rows;
  a.rot = dk.rot == KVQ_ROT_FWHT_HEAD;
  a.max_rows = max_rows;
  a.stretch = p.stretch;
  a.n_stretch = p.n_stretch;
  a.n_parts = p.n_parts;
  a.div_ps = FastDiv(static_cast<uint32_t>(dk.t_cap));
  a.div_hq = FastDiv(static_cast<uint32_t>(q_heads));
  a.div_g = FastDiv(static_cast<uint32_t>(a.g));
  a.div_stretch = FastDiv(static_cast<uint32_t>(p.stretch));
  a.part_per = p.n_parts / p.n_stretch;
  a.step_page = kFewStep / dk.t_cap;
  a.step_off = kFewStep % dk.t_cap;
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
  const size_t rows = static_cast<size_t>(pg.n_rows) * q_heads * p.n_parts;
  a.part_o = static_cast<float*>(ws);
  a.part_s = reinterpret_cast<float2*>(static_cast<uint8_t*>(ws) + align256(rows * dk.head_dim * 4));
  a.err = ctx.err;
  a.wait_ns = ctx.wait_ns;
#define KVQ_CASE(D_, B_, G_) \
  if (dk.head_dim == D_ && dk.bits == B_ && dk.group == G_) return run<D_, B_, G_>(a, p, st);
#define KVQ_BITS(D_, G_) KVQ_CASE(D_, 2, G_) KVQ_CASE(D_, 3, G_) KVQ_CASE(D_, 4, G_)
  KVQ_BITS(128, 128) KVQ_BITS(128, 64) KVQ_BITS(128, 32) KVQ_BITS(64, 64) KVQ_BITS(64, 32)
#undef KVQ_BITS
#undef KVQ_CASE
  return KVQ_ERR_UNSUPPORTED;
}

}  // namespace kvq
