// qk_kv.hip - writing rows to the paged Q4_0 cache (position rotation and quantization
// on the way) and reading them back.
#include <climits>
#include <type_traits>

#include "qk_internal.h"
#include "qk_kv.h"

namespace qk {
namespace {

// One lane holds 8 consecutive dims (one code dword); the 4 lanes of a quad hold one
// 32-element block.

// Rotates 8 dims of one head, x, by their (cos, sin): with halves, o holds the partners and cs a pair of 2
// dims each, sin negated in the low half (x cos - y sin is x cos + y (-sin) to the bit); else neighbours
// are pairs and cs[0], cs[1] hold 2 pairs each.  Every product and sum is rounded on its own: the
// stored codes are a function of these bits.
template <bool kHalves>
__device__ __forceinline__ void turn8(float (&x)[8], const float (&o)[8], const float4v (&cs)[4]) {
#pragma clang fp contract(off)
  if constexpr (kHalves) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = x[i] * cs[i / 2][i % 2 * 2] + o[i] * cs[i / 2][i % 2 * 2 + 1];
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float co = cs[i / 2][i % 2 * 2], si = cs[i / 2][i % 2 * 2 + 1];
      const float a = x[2 * i], b = x[2 * i + 1];
      x[2 * i] = a * co - b * si;
      x[2 * i + 1] = a * si + b * co;
    }
  }
}

// The first element of largest magnitude of the quad's 32, 0 when all are 0.
__device__ __forceinline__ float first_largest(const float (&v)[8]) {
  float key = 0.0f, val = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (key < fabsf(v[i])) key = fabsf(v[i]), val = v[i];
  }
  // quad swaps [1,0,3,2] and [2,3,0,1]; on equal magnitudes the lower lane's element came first
  const int lane = threadIdx.x & 3;
  float ok = dpp_f<0xB1>(key), ov = dpp_f<0xB1>(val);
  if (ok > key || (ok == key && (lane & 1))) key = ok, val = ov;
  ok = dpp_f<0x4E>(key), ov = dpp_f<0x4E>(val);
  if (ok > key || (ok == key && (lane & 2))) key = ok, val = ov;
  return val;
}

// The Q4_0 rule over the quad's 32 elements: the first element of largest magnitude over -8 is the scale.
// Returns the lane's code dword; scale is the quad's.  The largest magnitude is that of the maximum or the
// minimum; where they are equal (a block of zeros, or +-x) the search for the first decides.
// The code is trunc(v / d + 8.5) kept in 0 .. 15; the median also sends NaN (0 x inf, d subnormal) to 0.
__device__ __forceinline__ uint32_t q4_0_piece(const float (&v)[8], float* scale) {
#pragma clang fp contract(off)
  float up = v[0], down = v[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) up = fmaxf(up, v[i]), down = fminf(down, v[i]);
  up = fmaxf(up, dpp_f<0xB1>(up)), down = fminf(down, dpp_f<0xB1>(down));
  up = fmaxf(up, dpp_f<0x4E>(up)), down = fminf(down, dpp_f<0x4E>(down));
  float val = up > -down ? up : down;
  if (__any(up == -down)) val = first_largest(v);
  const float d = val / -8.0f;
  const float id = d != 0.0f ? 1.0f / d : 0.0f;
  uint32_t w = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t c = static_cast<uint32_t>(__builtin_amdgcn_fmed3f(v[j] * id + 8.5f, 0.0f, 15.0f));
    w |= c << (4 * ((j >> 1) + 4 * (j & 1)));
  }
  *scale = d;
  return w;
}

// A workgroup takes kRows rows, a thread 8 dims of one row (a piece) in several heads.  Consecutive positions
// of a head lie next to each other in a page, 16 of them as 1 KB of codes and 128 bytes of scales at
// D = 128, so a workgroup writes and reads whole lines there although the tensors' rows are one
// position each.  A row's place and a piece's angles are found once for all heads; the heads' loads are on
// their way together.
template <int D>
struct Shape {
  static constexpr int kPieces = D / 8, kRows = D == 64 ? 32 : 16, kThreads = kRows * kPieces;
};
// Heads of a thread.  Append: each turned by the same angles, read once; 2, 4, 8 measured 130, 122 and 106 us (with
// the read back, 7380 rows of 32 + 2 x 32 heads of 128 f16).  Read: 2, 4, 8 measured 34.4, 28.8, 29.9 us (28 K rows of
// 2 x 8 heads of 128 bf16, 6.0 TB/s).  Where that leaves most of the card without work, one head of a thread
// ends sooner (append of 64 rows of 32 + 2 x 8 heads: 4.4 us against 8.2).
constexpr int kAppendJobs = 8, kReadJobs = 4;
constexpr int64_t kManyGroups = 512;  // workgroups

struct Place {
  int64_t row, pos, page;  // page -1: none
  bool listed;             // the row belongs to a sequence
};

// The place of this thread's row.
template <int D>
__device__ __forceinline__ Place place_of(const KvBatch& b) {
  using S = Shape<D>;
  __shared__ int seqs[S::kRows];
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * S::kRows;
  for (int r = 4 * wave_id(); r < S::kRows; r += S::kThreads / 16) {
    int seq[4];
    row_seq4(b.cu, b.n_seq, row0 + r, seq);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if ((threadIdx.x & 63) == 0) seqs[r + i] = seq[i];
    }
  }
  __syncthreads();
  Place p;
  p.row = row0 + threadIdx.x / S::kPieces;
  const int seq = seqs[threadIdx.x / S::kPieces];
  p.listed = p.row < b.n_rows && seq < b.n_seq;
  p.pos = -1, p.page = -1;
  if (p.listed) {
    const int64_t at = p.row - b.cu[seq];
    p.listed = at >= 0;
    p.pos = static_cast<int64_t>(b.start[seq]) + at;
    if (p.listed) p.page = page_of(b, seq, p.pos);
  }
  return p;
}

// Memory bound: k, v and q are read once from HBM (a rotated half's partner comes from the same lines), 9/16
// byte per key and value dim is written.  Measured: 7380 rows of 32 + 2 x 32 heads of 128 f16, 272 MB: 67 us, 4.1 TB/s.
template <typename T, int D, bool kHalves, int kJobs>
__global__ __launch_bounds__(Shape<D>::kThreads) void kv_append_kernel(KvBatch b, uint8_t* pages, const T* k, int64_t k_stride,
                                                                       const T* v, int64_t v_stride, const T* q, int64_t q_stride,
                                                                       int n_heads, const float* rope, int64_t rope_rows, int n_rot,
                                                                       T* q_out) {
  constexpr int NB = D / 32;
  const Place at = place_of<D>(b);
  if (!at.listed || (n_rot > 0 && (at.pos < 0 || at.pos >= rope_rows))) return;
  const int e0 = threadIdx.x % Shape<D>::kPieces * 8;
  // heads in the order K, V, q
  const int head0 = blockIdx.y * kJobs, heads = 2 * b.n_kv + n_heads;
  const bool turns = e0 < n_rot, low = e0 < n_rot / 2;
  const int partner = kHalves && turns ? (low ? n_rot / 2 : -(n_rot / 2)) : 0;
  float4v cs[4] = {};
  if (turns) {
    const float4v* c = reinterpret_cast<const float4v*>(rope + at.pos * n_rot + (kHalves ? 2 * (low ? e0 : e0 - n_rot / 2) : e0));
#pragma unroll
    for (int i = 0; i < (kHalves ? 4 : 2); ++i) {
      cs[i] = c[i];
      if (kHalves && low) cs[i][1] = -cs[i][1], cs[i][3] = -cs[i][3];
    }
  }
  float x[kJobs][8], o[kJobs][8];
#pragma unroll
  for (int j = 0; j < kJobs; ++j) {
    const int h = head0 + j;
    if (h >= heads) break;
    const T* p = h < b.n_kv ? k + at.row * k_stride + h * D
                            : (h < 2 * b.n_kv ? v + at.row * v_stride + (h - b.n_kv) * D
                                              : q + at.row * q_stride + (h - 2 * b.n_kv) * D);
    load8(p + e0, x[j]);
    if constexpr (kHalves) load8(p + e0 + partner, o[j]);
  }
  const int64_t tokens = int64_t(1) << b.page_shift, slot = at.pos & (tokens - 1), half = kv_half_bytes(tokens, D);
#pragma unroll
  for (int j = 0; j < kJobs; ++j) {
    const int h = head0 + j;
    if (h >= heads) break;
    const bool is_v = h >= b.n_kv && h < 2 * b.n_kv;
    if (turns && !is_v) turn8<kHalves>(x[j], o[j], cs);
    if (h >= 2 * b.n_kv) {
      store8(q_out + (at.row * n_heads + h - 2 * b.n_kv) * D + e0, x[j]);
      continue;
    }
    float d;
    const uint32_t w = q4_0_piece(x[j], &d);
    if (at.page < 0) continue;
    uint8_t* base = pages + (at.page * b.n_kv + (is_v ? h - b.n_kv : h)) * 2 * half + (is_v ? half : 0);
    const int blk = e0 / 32, g = (e0 % 32) / 8;
    *reinterpret_cast<uint32_t*>(base + slot * (D / 2) + (g * NB + blk) * 4) = w;
    if (g == 0) *reinterpret_cast<uint16_t*>(base + tokens * (D / 2) + (slot * NB + blk) * 2) = f32_to_f16_bits(d);
  }
}

// Code dwords of the rows' K, then V heads; value = d * (code - 8), exact in f32, rounded once to T.
template <typename T, int D, int kJobs>
__global__ __launch_bounds__(Shape<D>::kThreads) void kv_read_kernel(KvBatch b, const uint8_t* pages, T* k_out, T* v_out) {
  constexpr int NB = D / 32;
  const Place at = place_of<D>(b);
  if (!at.listed) return;
  const int e = threadIdx.x % Shape<D>::kPieces, head0 = blockIdx.y * kJobs;
  const int64_t tokens = int64_t(1) << b.page_shift, slot = at.pos & (tokens - 1), half = kv_half_bytes(tokens, D);
  uint32_t code[kJobs] = {}, scale[kJobs] = {};
#pragma unroll
  for (int j = 0; j < kJobs; ++j) {
    const int h = head0 + j, is_v = h >= b.n_kv;
    if (h >= 2 * b.n_kv || at.page < 0) break;
    const uint8_t* base = pages + (at.page * b.n_kv + h - is_v * b.n_kv) * 2 * half + is_v * half;
    code[j] = *reinterpret_cast<const uint32_t*>(base + slot * (D / 2) + e * 4);
    scale[j] = *reinterpret_cast<const uint16_t*>(base + tokens * (D / 2) + (slot * NB + e % NB) * 2);
  }
#pragma unroll
  for (int j = 0; j < kJobs; ++j) {
    const int h = head0 + j, is_v = h >= b.n_kv;
    if (h >= 2 * b.n_kv) break;
    const half8 c = nibbles_to_f16(code[j]);
    const float d = f16_to_f32(scale[j]);
    float x[8];
#pragma unroll
    for (int n = 0; n < 8; ++n) x[n] = at.page >= 0 ? d * static_cast<float>(c[n]) : 0.0f;
    store8((is_v ? v_out : k_out) + (at.row * b.n_kv + h - is_v * b.n_kv) * D + e % NB * 32 + e / NB * 8, x);
  }
}

// Launches over the rows (x) and over `heads` heads of each, kJobs a workgroup (y).
template <int D, int kJobs, typename Kernel, typename... Args>
hipError_t launch(Kernel kernel, const KvBatch& b, int64_t heads, hipStream_t s, Args... args) {
  using S = Shape<D>;
  unsigned all = 0;
  const int64_t gx = (b.n_rows + S::kRows - 1) / S::kRows, gy = (heads + kJobs - 1) / kJobs;
  if (gy > 65535 || !launch_grid(gx * gy, S::kThreads, &all)) return hipErrorInvalidConfiguration;
  kernel<<<dim3(static_cast<unsigned>(gx), static_cast<unsigned>(gy)), S::kThreads, 0, s>>>(b, args...);
  return hipGetLastError();
}
template <int D>
bool many_groups(const KvBatch& b, int64_t heads, int jobs) {
  return (b.n_rows + Shape<D>::kRows - 1) / Shape<D>::kRows * ((heads + jobs - 1) / jobs) >= kManyGroups;
}

template <typename T, int D>
hipError_t append_d(const KvBatch& b, uint8_t* pages, const void* k, int64_t ks, const void* v, int64_t vs, const void* q,
                    int64_t qs, int n_heads, const float* rope, int64_t rope_rows, int n_rot, int halves, void* q_out,
                    hipStream_t s) {
  const int64_t heads = 2 * int64_t(b.n_kv) + n_heads;
  auto run = [&](auto jobs) {
    constexpr int kJobs = decltype(jobs)::value;
    return launch<D, kJobs>(halves ? kv_append_kernel<T, D, true, kJobs> : kv_append_kernel<T, D, false, kJobs>, b, heads, s, pages,
                            static_cast<const T*>(k), ks, static_cast<const T*>(v), vs, static_cast<const T*>(q), qs, n_heads,
                            rope, rope_rows, n_rot, static_cast<T*>(q_out));
  };
  return many_groups<D>(b, heads, kAppendJobs) ? run(std::integral_constant<int, kAppendJobs>{})
                                               : run(std::integral_constant<int, 1>{});
}

template <typename T, int D>
hipError_t read_d(const KvBatch& b, const uint8_t* pages, T* ko, T* vo, hipStream_t s) {
  const int64_t heads = 2 * int64_t(b.n_kv);
  return many_groups<D>(b, heads, kReadJobs) ? launch<D, kReadJobs>(kv_read_kernel<T, D, kReadJobs>, b, heads, s, pages, ko, vo)
                                             : launch<D, 1>(kv_read_kernel<T, D, 1>, b, heads, s, pages, ko, vo);
}

template <typename T>
hipError_t append_t(const KvBatch& b, int dim, uint8_t* pages, const void* k, int64_t ks, const void* v, int64_t vs,
                    const void* q, int64_t qs, int n_heads, const float* rope, int64_t rope_rows, int n_rot, int halves,
                    void* q_out, hipStream_t s) {
  auto run = [&](auto append) {
    return append(b, pages, k, ks, v, vs, q, qs, n_heads, rope, rope_rows, n_rot, halves, q_out, s);
  };
  switch (dim) {
    case 64: return run(append_d<T, 64>);
    case 96: return run(append_d<T, 96>);
    case 128: return run(append_d<T, 128>);
    default: return run(append_d<T, 256>);
  }
}

template <typename T>
hipError_t read_t(const KvBatch& b, int dim, const uint8_t* pages, void* k_out, void* v_out, hipStream_t s) {
  T *ko = static_cast<T*>(k_out), *vo = static_cast<T*>(v_out);
  switch (dim) {
    case 64: return read_d<T, 64>(b, pages, ko, vo, s);
    case 96: return read_d<T, 96>(b, pages, ko, vo, s);
    case 128: return read_d<T, 128>(b, pages, ko, vo, s);
    default: return read_d<T, 256>(b, pages, ko, vo, s);
  }
}

}  // namespace

hipError_t launch_kv_append(const KvBatch& b, int dim, int dtype, uint8_t* pages, const void* k, int64_t k_stride,
                            const void* v, int64_t v_stride, const void* q, int64_t q_stride, int n_heads,
                            const float* rope, int64_t rope_rows, int n_rot, int halves, void* q_out, hipStream_t s) {
  switch (dtype) {
    case kF32:
      return append_t<float>(b, dim, pages, k, k_stride, v, v_stride, q, q_stride, n_heads, rope, rope_rows, n_rot, halves,
                             q_out, s);
    case kF16:
      return append_t<_Float16>(b, dim, pages, k, k_stride, v, v_stride, q, q_stride, n_heads, rope, rope_rows, n_rot,
                                halves, q_out, s);
    default:
      return append_t<bf16>(b, dim, pages, k, k_stride, v, v_stride, q, q_stride, n_heads, rope, rope_rows, n_rot, halves,
                            q_out, s);
  }
}

hipError_t launch_kv_read(const KvBatch& b, int dim, int dtype, const uint8_t* pages, void* k_out, void* v_out,
                          hipStream_t s) {
  switch (dtype) {
    case kF32: return read_t<float>(b, dim, pages, k_out, v_out, s);
    case kF16: return read_t<_Float16>(b, dim, pages, k_out, v_out, s);
    default: return read_t<bf16>(b, dim, pages, k_out, v_out, s);
  }
}

}  // namespace qk
