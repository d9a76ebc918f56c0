// qk_attn_paged.hip - attention of packed rows over the paged Q4_0 cache.
//
// One item is 16 (row, head of the group) pairs of one sequence that share a key / value
// head.  A workgroup of 4 wavefronts walks the item's positions in steps of 128, 32 to
// a wavefront, each with its own running softmax; the four are joined through LDS at the end.
//
// Both products run on mfma_16x16x32_f16 with q as the columns, so a lane's column (lane % 16)
// and with it the softmax state stay the same throughout:
//   scores  K codes (16 positions x 32 dims of one block) x q.  Codes are exact f16 integers; a
//           block's product is multiplied by its scale in f32, as the scale of a position
//           differs from block to block.
//   output  V codes (16 dims x 32 positions) x weights.  The scale of (position, block) goes into
//           the weight: w = p d, rounded once to f16.
// The score tile leaves positions 4 g + i (g = lane / 16) of two 16-position tiles in a lane,
// which are taken as the 8 k-slots of the second product: weights never change lanes.  Its
// other operand needs 8 positions of one dim: a lane takes byte m = (lane % 16) / 4 (two dims) of
// dword (lane % 4, block) of each position, one byte permute to a pair of positions.
//
// p = 2^(s - ref) with ref = m + E: m is a running maximum that moves only when a score passes it by
// more than 8 (so no cross-lane maximum in most tiles).  E is 0 but for f16, where it is the power of two
// that keeps w inside f16 for the value scales met so far, so that small value scales lose no bits.
//
// The score product is the same for every type: q is normalised to a power of two (bf16 then fits
// f16) and f32 split into two f16 pieces, 22 bits.  The output product is of the type: weights are
// rounded to f16 or bf16 (codes are exact in both), or stay f32 on mfma_16x16x4_f32.  A rounding to f16
// would lose the weights of a bf16 or f32 row that are 2^-30 and less of the largest, which is all
// that is left of a dim whose other values are 0.
//
// Work is split over the positions when the table allows more than kDirectSteps steps: all
// items' steps laid end to end are cut into equal ranges, one a workgroup, however uneven
// the sequences; ranges that hold a part of an item write (ref, sum, output) to the workspace and a
// second kernel joins them.
#include <cfloat>
#include <type_traits>

#include "qk_internal.h"
#include "qk_kv.h"

namespace qk {
namespace {

constexpr int kWaves = 4, kTile = 32, kStep = kWaves * kTile, kCols = 16;
constexpr int kDirectSteps = 8;  // 1024 positions
constexpr int kMinUnits = 3;     // least steps (the item's fixed cost counted as one) of a range

struct PagedArgs {
  KvBatch b;
  const uint8_t* pages;
  const void* q;
  void* out;
  float* part;  // workspace of the split, null: every workgroup takes one whole item
  int64_t q_stride, window;
  int n_heads, group, n_wg;
  float scale;
};

// Per-sequence work, the same for every item of the sequence.
struct SeqWork {
  int64_t row0, pos0;  // first packed row, its position
  int64_t tiles;       // items per key / value head
  int rows, lo, hi;    // positions lo (a multiple of kTile) .. hi - 1 are visited
  int units;           // steps + 1
};

__device__ __forceinline__ SeqWork seq_work(const PagedArgs& a, int64_t i) {
  const KvBatch& b = a.b;
  int64_t c0 = b.cu[i], c1 = b.cu[i + 1];
  SeqWork s;
  s.pos0 = b.start[i];
  if (c0 < 0) s.pos0 -= c0, c0 = 0;
  if (c1 > b.n_rows) c1 = b.n_rows;
  s.row0 = c0;
  s.rows = static_cast<int>(c1 > c0 ? c1 - c0 : 0);
  s.tiles = (static_cast<int64_t>(s.rows) * a.group + kCols - 1) / kCols;
  const int64_t cap = b.n_pages > 0 ? b.max_pages << b.page_shift : 0;
  int64_t hi = s.pos0 + s.rows, lo = a.window > 0 ? s.pos0 - a.window + 1 : 0;
  hi = hi < cap ? hi : cap;
  lo = lo > 0 ? lo : 0;
  if (hi <= lo) hi = lo = 0;
  s.lo = static_cast<int>(lo) & -kTile;
  s.hi = static_cast<int>(hi);
  s.units = (s.hi - s.lo + kStep - 1) / kStep + 1;
  return s;
}

__device__ __forceinline__ int64_t wave_scan(int64_t v) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int64_t o = __shfl_up(v, d);
    if (lane >= d) v += o;
  }
  return v;
}

__device__ __forceinline__ int64_t first_lane(int64_t v) {
  const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v));
  const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v >> 32));
  return static_cast<int64_t>((static_cast<uint64_t>(hi) << 32) | lo);
}

// Units of all items.
__device__ __forceinline__ int64_t total_units(const PagedArgs& a) {
  const int lane = threadIdx.x & 63;
  int64_t sum = 0;
  for (int i = 0; i < a.b.n_seq; i += 64) {
    int64_t w = 0;
    if (i + lane < a.b.n_seq) {
      const SeqWork s = seq_work(a, i + lane);
      w = s.tiles * s.units;
    }
    sum += __shfl(wave_scan(w), 63);
  }
  return first_lane(sum) * a.b.n_kv;
}

// The sequence whose share of the items (by_item) or of the units holds `at`; `items0` and `units0`
// are what comes before it.  n_seq when there is none.
__device__ __forceinline__ int find_seq(const PagedArgs& a, bool by_item, int64_t at, int64_t* items0, int64_t* units0) {
  const int lane = threadIdx.x & 63;
  int64_t items = 0, units = 0;
  for (int i = 0; i < a.b.n_seq; i += 64) {
    int64_t n = 0, w = 0;
    if (i + lane < a.b.n_seq) {
      const SeqWork s = seq_work(a, i + lane);
      n = s.tiles * a.b.n_kv;
      w = n * s.units;
    }
    const int64_t ni = wave_scan(n), wi = wave_scan(w);
    const uint64_t hit = __ballot((by_item ? items + ni : units + wi) > at);
    if (hit != 0) {
      const int l = __builtin_ctzll(hit);
      *items0 = first_lane(items + __shfl(ni - n, l));
      *units0 = first_lane(units + __shfl(wi - w, l));
      return __builtin_amdgcn_readfirstlane(i + l);
    }
    items += __shfl(ni, 63);
    units += __shfl(wi, 63);
  }
  return a.b.n_seq;
}

// How many workgroups share `total` units, and where the range of workgroup w begins.
__device__ __forceinline__ int64_t ranges(int64_t total, int n_wg) {
  const int64_t n = total / kMinUnits;
  return n < 1 ? 1 : (n < n_wg ? n : n_wg);
}
__device__ __forceinline__ int64_t range_begin(int64_t total, int64_t n, int64_t w) { return w * total / n; }

// N consecutive dwords at a lane's offset from a wave-uniform one.  Buffer loads, because they take both
// (and a page as their bound) without a 64-bit address in vector registers.
template <int N>
__device__ __forceinline__ void load_dwords(__amdgpu_buffer_rsrc_t page, uint32_t lane, uint32_t at, uint32_t* o) {
  if constexpr (N >= 4) {
    const auto v = __builtin_amdgcn_raw_buffer_load_b128(page, lane, at, 0);
#pragma unroll
    for (int k = 0; k < 4; ++k) o[k] = v[k];
    if constexpr (N > 4) load_dwords<N - 4>(page, lane + 16, at, o + 4);
  } else if constexpr (N == 3) {
    const auto v = __builtin_amdgcn_raw_buffer_load_b96(page, lane, at, 0);
#pragma unroll
    for (int k = 0; k < 3; ++k) o[k] = v[k];
  } else if constexpr (N == 2) {
    const auto v = __builtin_amdgcn_raw_buffer_load_b64(page, lane, at, 0);
    o[0] = v[0], o[1] = v[1];
  } else {
    o[0] = __builtin_amdgcn_raw_buffer_load_b32(page, lane, at, 0);
  }
}

// Keeps what is computed from loaded registers behind this point, so that it is not moved up to
// where the loads are still on the way.
template <int M, int N>
__device__ __forceinline__ void pin(uint32_t (&r)[M][N]) {
#pragma unroll
  for (int i = 0; i < M; ++i) {
#pragma unroll
    for (int k = 0; k < N; ++k) asm volatile("" : "+v"(r[i][k]));
  }
}

__device__ __forceinline__ float half_at(const uint32_t* w, int i) {
  const half2v h = __builtin_bit_cast(half2v, w[i >> 1]);
  return static_cast<float>(h[i & 1]);
}

// The larger of d and the magnitudes (as bits) of the two f16 of w.
__device__ __forceinline__ uint32_t largest_half(uint32_t w, uint32_t d) {
  const uint32_t u = w & 0x7FFF7FFFu;
  return max(d, max(u & 0xFFFFu, u >> 16));
}

// Two f16 that are exact in bf16, as bf16: the high halves of their f32.
__device__ __forceinline__ uint32_t half_pair_to_bf16(uint32_t w) {
  return __builtin_amdgcn_perm(__float_as_uint(half_at(&w, 1)), __float_as_uint(half_at(&w, 0)), 0x07060302u);
}

template <typename V>
__device__ __forceinline__ V operand(const uint32_t* w) {
  return __builtin_bit_cast(V, uint4v{w[0], w[1], w[2], w[3]});
}

__device__ __forceinline__ half8 pack8(const float* v) {
  half8 h;
#pragma unroll
  for (int i = 0; i < 8; ++i) h[i] = static_cast<_Float16>(v[i]);
  return h;
}

// The running softmax of one wavefront: lane's column is lane % 16.
template <int NB>
struct State {
  float m, lim, ref, l;    // l: this lane's positions only
  uint32_t e16, dlim;      // exponent field of the largest value scale met, first |scale| too large for it
  float4v o[NB][2];
};

// Dim of the output that element i of o[b][e] is, in lane group g.
__device__ __forceinline__ int out_dim(int b, int e, int i, int g) {
  const int n = 2 * g + e;
  return 32 * b + 8 * i + (n < 4 ? 2 * n : 2 * n - 7);
}

// Column values of `a` (row and head), written where the item's column is one.
template <typename T, int D>
__device__ __forceinline__ void store_out(const PagedArgs& a, const SeqWork& s, int64_t tile, int kv, int b, int e,
                                          const float4v& v, float inv) {
  const int lane = threadIdx.x & 63, g = lane / 16;
  const int64_t at = tile * kCols + lane % 16;
  if (at >= static_cast<int64_t>(s.rows) * a.group) return;
  T* p = static_cast<T*>(a.out) + ((s.row0 + at / a.group) * a.n_heads + kv * a.group + at % a.group) * D;
#pragma unroll
  for (int i = 0; i < 4; ++i) p[out_dim(b, e, i, g)] = static_cast<T>(v[i] * inv);
}

template <typename T, int D>
__global__ __launch_bounds__(256, D <= 128 ? 2 : 1) void attn_paged_kernel(PagedArgs a) {
  constexpr int NB = D / 32, kRegs = NB * 2;  // float4 registers of the output
  constexpr bool kF32T = std::is_same_v<T, float>, kF16T = std::is_same_v<T, _Float16>;
  constexpr int P = kF32T ? 2 : 1;  // f16 pieces of a query
  __shared__ float4v so[kWaves][kRegs][64];
  __shared__ float sref[kWaves][64], sl[kWaves][64];
  const KvBatch& b = a.b;
  const int lane = threadIdx.x & 63, wave = wave_id(), col = lane % 16, g = lane / 16;
  const int64_t tokens = int64_t(1) << b.page_shift, half = kv_half_bytes(tokens, D);
  const bool split = a.part != nullptr;

  int64_t at, end, items0, units0, total = 0;
  int seq;
  if (split) {
    total = total_units(a);
    const int64_t n = ranges(total, a.n_wg);
    if (blockIdx.x >= n) return;
    at = range_begin(total, n, blockIdx.x), end = range_begin(total, n, blockIdx.x + 1);
    seq = find_seq(a, false, at, &items0, &units0);
  } else {
    seq = find_seq(a, true, blockIdx.x, &items0, &units0);
    if (seq < b.n_seq) {
      const SeqWork s = seq_work(a, seq);
      at = units0 + (blockIdx.x - items0) * s.units, end = at + s.units;
    }
  }
  if (seq >= b.n_seq) return;
  const int64_t begin = at;
  while (at < end) {
    SeqWork s = seq_work(a, seq);
    const int64_t mine = s.tiles * b.n_kv * s.units;
    if (at >= units0 + mine) {  // the next sequence (empty ones have no units)
      units0 += mine;
      if (++seq >= b.n_seq) return;
      continue;
    }
    const int64_t item = first_lane((at - units0) / s.units);
    const int u0 = __builtin_amdgcn_readfirstlane(static_cast<int>((at - units0) % s.units));
    const int u1 = static_cast<int>(end - at < s.units - u0 ? u0 + (end - at) : s.units);
    const int kv = __builtin_amdgcn_readfirstlane(static_cast<int>(item / s.tiles));
    const int64_t tile = first_lane(item % s.tiles);
    const int k0 = u0 > 0 ? u0 - 1 : 0, k1 = u1 - 1;  // steps

    // the lane's column: its row's visible positions, its query normalised to 2^14 <= max < 2^15
    const int64_t cat = tile * kCols + col;
    const int64_t n_cols = static_cast<int64_t>(s.rows) * a.group;
    const bool real = cat < n_cols;
    const int64_t row = real ? cat / a.group : 0;
    const int64_t pos = s.pos0 + row;
    const int hi_q = static_cast<int>(pos < s.hi ? pos : s.hi - 1);
    const int lo_q = a.window > 0 && pos - a.window + 1 > 0 ? static_cast<int>(pos - a.window + 1) : 0;
    half8 qf[P][NB];
    float fac;
    {
      const T* p = static_cast<const T*>(a.q) + (s.row0 + row) * a.q_stride +
                   (static_cast<int64_t>(kv) * a.group + (real ? cat % a.group : 0)) * D + 8 * g;
      float x[NB][8], top = 0.0f;
#pragma unroll
      for (int blk = 0; blk < NB; ++blk) {
        load8(p + 32 * blk, x[blk]);
#pragma unroll
        for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(x[blk][i]));
      }
      top = rows_max(top);
      const int ex = __builtin_amdgcn_frexp_expf(top);
      fac = __builtin_ldexpf(a.scale * 1.4426950408889634f, ex - 15);
#pragma unroll
      for (int blk = 0; blk < NB; ++blk) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[blk][i] = __builtin_ldexpf(x[blk][i], 15 - ex);
        qf[0][blk] = pack8(x[blk]);
        if constexpr (P == 2) {
#pragma unroll
          for (int i = 0; i < 8; ++i) x[blk][i] -= static_cast<float>(qf[0][blk][i]);
          qf[1][blk] = pack8(x[blk]);
        }
      }
    }
    // tiles in lo_max .. hi_min + 1 - kTile need no mask
    const int64_t first = tile * kCols / a.group;
    const int64_t last = ((tile + 1) * kCols < n_cols ? (tile + 1) * kCols - 1 : n_cols - 1) / a.group;
    const int64_t hi_min = s.pos0 + first < s.hi ? s.pos0 + first : s.hi - 1;
    const int64_t lo_max = a.window > 0 ? s.pos0 + last - a.window + 1 : 0;

    State<NB> st;
    st.m = st.lim = st.ref = -FLT_MAX, st.l = 0.0f;
    st.e16 = 0, st.dlim = 0;
#pragma unroll
    for (int i = 0; i < NB; ++i) st.o[i][0] = st.o[i][1] = float4v{0, 0, 0, 0};

    // this wavefront's tiles: t0 + n * kStep
    const int t0 = s.lo + k0 * kStep + wave * kTile;
    const int t_end = s.lo + k1 * kStep < s.hi ? s.lo + k1 * kStep : s.hi;
    const int n_tiles = t0 < t_end ? (t_end - t0 + kStep - 1) / kStep : 0;
    int page_vec = -1;  // pages of the 16-position halves of tiles n & ~31 ..
    const int32_t* table = b.table + static_cast<int64_t>(seq) * b.max_pages;
    auto refill = [&](int n) {
      const int64_t p = t0 + static_cast<int64_t>((n & ~31) + lane / 2) * kStep + (lane & 1) * 16;
      page_vec = -1;
      if (p < s.hi) {
        const int32_t page = table[p >> b.page_shift];
        if (page >= 0 && page < b.n_pages) page_vec = page;
      }
    };
    constexpr int kHalf = 16;  // a tile is two halves of 16 positions, each inside one page
    const int mask = static_cast<int>(tokens) - 1;
    const uint32_t v_at = static_cast<uint32_t>(half), scales_at = static_cast<uint32_t>(tokens) * (D / 2);
    // lane offsets from a half's first code or scale: its row of K codes, its 4 positions' scales, its dwords
    // of the first of its 4 V rows, one dword of all the half's scales
    const uint32_t k_lane = col * (D / 2) + g * NB * 4, d_lane = 4 * g * NB * 2, v_lane = 4 * g * (D / 2) + (col % 4) * NB * 4,
                   top_lane = lane % (8 * NB) * 4;
    uint32_t kc[2][NB], dk[2][2 * NB], vc[2][4][NB], dv[2][2 * NB], dt[2];
    const uint32_t sel = (col / 4) | 0x0C000C00u | (4 + col / 4) << 16;  // byte m of two dwords, each in a 16-bit half
    for (int n = 0; n < n_tiles; ++n) {
      const int t = t0 + n * kStep;
      if ((n & 31) == 0) refill(n);
      bool bad[2];
      __amdgpu_buffer_rsrc_t rsrc[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int page = __builtin_amdgcn_readlane(page_vec, 2 * (n & 31) + h);
        bad[h] = page < 0;  // page 0 is read in its place, and masked
        const uint8_t* p = a.pages + (static_cast<int64_t>(page < 0 ? 0 : page) * b.n_kv + kv) * 2 * half;
        rsrc[h] = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(p), 0, static_cast<int>(2 * half), 0x00027000);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t slot = (t + kHalf * h) & mask;
        load_dwords<NB>(rsrc[h], k_lane, slot * (D / 2), kc[h]);
        load_dwords<2 * NB>(rsrc[h], d_lane, scales_at + slot * (NB * 2), dk[h]);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t slot = (t + kHalf * h) & mask;
        if constexpr (kF16T) load_dwords<1>(rsrc[h], top_lane, v_at + scales_at + slot * (NB * 2), &dt[h]);
        load_dwords<2 * NB>(rsrc[h], d_lane, v_at + scales_at + slot * (NB * 2), dv[h]);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t slot = (t + kHalf * h) & mask;
#pragma unroll
        for (int i = 0; i < 4; ++i) load_dwords<NB>(rsrc[h], v_lane + i * (D / 2), v_at + slot * (D / 2), vc[h][i]);
      }
      float sc[2][4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int i = 0; i < 4; ++i) sc[h][i] = 0.0f;
#pragma unroll
        for (int blk = 0; blk < NB; ++blk) {
          const half8 kf = nibbles_to_f16(kc[h][blk]);
          float4v c = {0, 0, 0, 0};
          if constexpr (P == 2) c = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf, qf[1][blk], c, 0, 0, 0);
          c = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf, qf[0][blk], c, 0, 0, 0);
#pragma unroll
          for (int i = 0; i < 4; ++i) sc[h][i] = fmaf(c[i], half_at(dk[h], i * NB + blk), sc[h][i]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) sc[h][i] *= fac;
        __builtin_amdgcn_sched_barrier(0);  // one half's products at a time in registers
      }
      pin(dv);
      uint32_t dtop = 0;
      if (t < lo_max || t + kTile > hi_min + 1 || bad[0] || bad[1]) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          bool see[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int p = t + 16 * h + 4 * g + i;
            see[i] = p <= hi_q && p >= lo_q && !bad[h];
            if (!see[i]) sc[h][i] = -INFINITY;
          }
          // what a masked slot holds is not to be multiplied even by 0
#pragma unroll
          for (int k = 0; k < 2 * NB; ++k) {
            dv[h][k] &= (see[2 * k / NB] ? 0xFFFFu : 0u) | (see[(2 * k + 1) / NB] ? 0xFFFF0000u : 0u);
            if constexpr (kF16T) dtop = largest_half(dv[h][k], dtop);
          }
        }
      } else if constexpr (kF16T) {
#pragma unroll
        for (int h = 0; h < 2; ++h) dtop = largest_half(dt[h], dtop);
      }
      float top = sc[0][0];
#pragma unroll
      for (int i = 1; i < 8; ++i) top = fmaxf(top, sc[i / 4][i % 4]);
      if (__any(top > st.lim || (kF16T && dtop > st.dlim))) {
        top = rows_max(top);
        st.m = fmaxf(st.m, top);
        st.lim = st.m + 8.0f;
        float ref = st.m;
        if constexpr (kF16T) {
          const uint32_t dm = static_cast<uint32_t>(wave_max(static_cast<float>(dtop)));
          st.e16 = max(st.e16, dm >> 10);
          st.dlim = (st.e16 + 2) << 10;
          // scales below 2^(e16 - 14), weights below 2^6 now and 2^15 until either limit is passed
          ref += static_cast<float>(static_cast<int>(st.e16)) - 20.0f;
        }
        const float keep = __builtin_amdgcn_exp2f(st.ref - ref);
        st.ref = ref;
        st.l *= keep;
#pragma unroll
        for (int i = 0; i < NB; ++i) st.o[i][0] *= keep, st.o[i][1] *= keep;
      }
      float p[2][4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          p[h][i] = __builtin_amdgcn_exp2f(sc[h][i] - st.ref);
          st.l += p[h][i];
        }
      }
#pragma unroll
      for (int blk = 0; blk < NB; ++blk) {
        float w[8];  // + 0: a multiply-add takes the f16 as it is (v_fma_mix_f32)
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = fmaf(p[i / 4][i % 4], half_at(dv[i / 4], i % 4 * NB + blk), 0.0f);
        uint32_t v0[4], v1[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t x = __builtin_amdgcn_perm(vc[k / 2][k % 2 * 2 + 1][blk], vc[k / 2][k % 2 * 2][blk], sel);
          v0[k] = low_nibbles(x);
          v1[k] = high_nibbles(x);
        }
        if constexpr (kF32T) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            st.o[blk][0] = __builtin_amdgcn_mfma_f32_16x16x4f32(half_at(v0, i), w[i], st.o[blk][0], 0, 0, 0);
            st.o[blk][1] = __builtin_amdgcn_mfma_f32_16x16x4f32(half_at(v1, i), w[i], st.o[blk][1], 0, 0, 0);
          }
        } else if constexpr (kF16T) {
          const half8 wf = pack8(w);
          st.o[blk][0] = __builtin_amdgcn_mfma_f32_16x16x32_f16(operand<half8>(v0), wf, st.o[blk][0], 0, 0, 0);
          st.o[blk][1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(operand<half8>(v1), wf, st.o[blk][1], 0, 0, 0);
        } else {
          bf16x8 wf;
#pragma unroll
          for (int i = 0; i < 8; ++i) wf[i] = static_cast<bf16>(w[i]);
#pragma unroll
          for (int k = 0; k < 4; ++k) v0[k] = half_pair_to_bf16(v0[k]), v1[k] = half_pair_to_bf16(v1[k]);
          st.o[blk][0] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(operand<bf16x8>(v0), wf, st.o[blk][0], 0, 0, 0);
          st.o[blk][1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(operand<bf16x8>(v1), wf, st.o[blk][1], 0, 0, 0);
        }
      }
    }

    // the four wavefronts' states into one: each takes a quarter of the output registers
    st.l = rows_sum(st.l);
    sref[wave][lane] = st.ref, sl[wave][lane] = st.l;
#pragma unroll
    for (int i = 0; i < kRegs; ++i) so[wave][i][lane] = st.o[i / 2][i % 2];
    __syncthreads();
    float ref = sref[0][lane], l = 0.0f, f[kWaves];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) ref = fmaxf(ref, sref[w][lane]);
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      f[w] = __builtin_amdgcn_exp2f(sref[w][lane] - ref);
      l += sl[w][lane] * f[w];
    }
    const bool whole = u0 == 0 && u1 == s.units;
    const float inv = l != 0.0f ? 1.0f / l : 0.0f;
    float* part = nullptr;
    if (!whole) {
      const int slot = units0 + item * s.units <= begin ? 0 : 1;
      part = a.part + (static_cast<int64_t>(blockIdx.x) * 2 + slot) * (kRegs * 256 + 128);
      if (wave == 0) part[lane] = ref, part[64 + lane] = l;
    }
    for (int i = wave; i < kRegs; i += kWaves) {
      float4v v = {0, 0, 0, 0};
#pragma unroll
      for (int w = 0; w < kWaves; ++w) v += so[w][i][lane] * f[w];
      if (whole) {
        store_out<T, D>(a, s, tile, kv, i / 2, i % 2, v, inv);
      } else if (real) {
        reinterpret_cast<float4v*>(part + 128)[i * 64 + lane] = v;
      }
    }
    __syncthreads();
    at += u1 - u0;
  }
}

// Workgroup (x, y): output register y of item x, joined from the ranges that hold parts of it.
template <typename T, int D>
__global__ __launch_bounds__(64) void attn_join_kernel(PagedArgs a) {
  constexpr int kRegs = D / 16;
  int64_t items0, units0;
  const int lane = threadIdx.x;
  const int64_t total = total_units(a);
  const int64_t n = ranges(total, a.n_wg);
  const int seq = find_seq(a, true, blockIdx.x, &items0, &units0);
  if (seq >= a.b.n_seq) return;
  const SeqWork s = seq_work(a, seq);
  const int64_t item = blockIdx.x - items0;
  const int64_t u0 = units0 + item * s.units, u1 = u0 + s.units;
  int64_t w0 = u0 * n / total;
  while (range_begin(total, n, w0 + 1) <= u0) ++w0;
  if (range_begin(total, n, w0 + 1) >= u1) return;  // one range holds all of it
  int64_t w1 = w0 + 1;
  while (w1 < n && range_begin(total, n, w1) < u1) ++w1;
  const int64_t tile = item % s.tiles;
  auto part = [&](int64_t w) {
    const int slot = u0 <= range_begin(total, n, w) ? 0 : 1;
    return a.part + (w * 2 + slot) * (kRegs * 256 + 128);
  };
  float ref = -FLT_MAX, l = 0.0f;
  for (int64_t w = w0; w < w1; ++w) ref = fmaxf(ref, part(w)[lane]);
  float4v v = {0, 0, 0, 0};
  if (tile * kCols + lane % 16 < static_cast<int64_t>(s.rows) * a.group) {
    for (int64_t w = w0; w < w1; ++w) {
      const float* p = part(w);
      const float f = __builtin_amdgcn_exp2f(p[lane] - ref);
      l += p[64 + lane] * f;
      v += reinterpret_cast<const float4v*>(p + 128)[blockIdx.y * 64 + lane] * f;
    }
  }
  store_out<T, D>(a, s, tile, static_cast<int>(item / s.tiles), blockIdx.y / 2, blockIdx.y % 2, v, l != 0.0f ? 1.0f / l : 0.0f);
}

// Workgroups that share the card in the split form: as many as run at once.
int split_groups(int dim) { return 256 * (dim <= 128 ? 2 : 1); }

// Most items a batch can have: every row with its group's heads, and a part-filled item to a sequence.
int64_t max_items(const KvBatch& b, int n_heads) {
  const int64_t seqs = b.n_seq < b.n_rows ? b.n_seq : b.n_rows;
  return (b.n_rows * (n_heads / b.n_kv) / kCols + seqs) * b.n_kv;
}

bool is_split(const KvBatch& b) { return (b.max_pages << b.page_shift) > kDirectSteps * kStep; }

template <typename T, int D>
hipError_t run(const PagedArgs& a, hipStream_t s) {
  unsigned gx = 0;
  const int64_t items = max_items(a.b, a.n_heads);
  if (a.part == nullptr) {
    if (!launch_grid(items, 256, &gx)) return hipErrorInvalidConfiguration;
    attn_paged_kernel<T, D><<<gx, 256, 0, s>>>(a);
    return hipGetLastError();
  }
  if (!launch_grid(items * (D / 16), 64, &gx)) return hipErrorInvalidConfiguration;
  attn_paged_kernel<T, D><<<a.n_wg, 256, 0, s>>>(a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  attn_join_kernel<T, D><<<dim3(static_cast<unsigned>(items), D / 16), 64, 0, s>>>(a);
  return hipGetLastError();
}

template <typename T>
hipError_t paged_t(const PagedArgs& a, int dim, hipStream_t s) {
  switch (dim) {
    case 64: return run<T, 64>(a, s);
    case 96: return run<T, 96>(a, s);
    case 128: return run<T, 128>(a, s);
    default: return run<T, 256>(a, s);
  }
}

}  // namespace

int64_t attn_paged_ws_bytes(const KvBatch& b, int dim, int) {
  return is_split(b) ? static_cast<int64_t>(split_groups(dim)) * 2 * (dim / 16 * 256 + 128) * 4 : 0;
}

hipError_t launch_attn_paged(const KvBatch& b, int dim, int dtype, const uint8_t* pages, const void* q, int64_t q_stride,
                             int n_heads, float scale, int64_t window, void* out, void* ws, hipStream_t s) {
  const PagedArgs a{b, pages, q, out, is_split(b) ? static_cast<float*>(ws) : nullptr, q_stride, window, n_heads,
                    n_heads / b.n_kv, split_groups(dim), scale};
  switch (dtype) {
    case kF32: return paged_t<float>(a, dim, s);
    case kF16: return paged_t<_Float16>(a, dim, s);
    default: return paged_t<bf16>(a, dim, s);
  }
}

}  // namespace qk
