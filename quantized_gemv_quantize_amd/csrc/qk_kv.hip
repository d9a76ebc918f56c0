// qk_kv.hip - writing rows to the paged Q4_0 cache (position rotation and quantization
// on the way) and reading them back.
#include <climits>

#include "qk_internal.h"
#include "qk_kv.h"

namespace qk {
namespace {

// One lane holds 8 consecutive dims (one code dword); the 4 lanes of a quad hold one
// 32-element block.

// Rotates v (dims e0 .. e0 + 7 of one head, at p) by the table row cs (n_rot / 2 pairs of
// cos, sin).  Every product and sum is rounded on its own: the stored codes are a function
// of these bits.
template <typename T>
__device__ __forceinline__ void rotate8(const T* p, int e0, int n_rot, bool halves, const float* cs, float* v) {
#pragma clang fp contract(off)
  if (e0 >= n_rot) return;
  if (halves) {
    const int half = n_rot / 2;
    const bool low = e0 < half;
    float o[8];
    load8(p + (low ? half : -half), o);
    const float4v* t = reinterpret_cast<const float4v*>(cs + 2 * (low ? e0 : e0 - half));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4v c = t[i];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float co = c[2 * k], si = c[2 * k + 1];
        const float x = v[2 * i + k], y = o[2 * i + k];
        // low half: x cos - y sin; high half: (the low element) sin + x cos
        v[2 * i + k] = low ? x * co - y * si : y * si + x * co;
      }
    }
  } else {
    const float4v* t = reinterpret_cast<const float4v*>(cs + e0);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float4v c = t[i];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float co = c[2 * k], si = c[2 * k + 1];
        const float x = v[4 * i + 2 * k], y = v[4 * i + 2 * k + 1];
        v[4 * i + 2 * k] = x * co - y * si;
        v[4 * i + 2 * k + 1] = x * si + y * co;
      }
    }
  }
}

__device__ __forceinline__ int trunc_code(float f) {
  if (f != f) return 0;
  return static_cast<int>(fminf(fmaxf(f, -2147483648.0f), 15.0f));
}

// The Q4_0 rule over the quad's 32 elements: the first element of largest magnitude over
// -8 is the scale.  Returns the lane's code dword; d is the quad's scale.
__device__ __forceinline__ uint32_t q4_0_piece(const float* v, float* scale) {
#pragma clang fp contract(off)
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
  const float d = val / -8.0f;
  const float id = d != 0.0f ? 1.0f / d : 0.0f;
  uint32_t w = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t c = static_cast<uint32_t>(min(trunc_code(v[j] * id + 8.5f), 15)) & 15u;
    w |= c << (4 * ((j >> 1) + 4 * (j & 1)));
  }
  *scale = d;
  return w;
}

// Workgroup (x, y): row x, pieces of 8 dims y * blockDim + thread, in the order K, V, q.
// Memory bound: k, v and q are read once from HBM (a rotated half's partner comes from the
// same wavefront's lines), 9/16 byte per key and value dim is written.
template <typename T, int D>
__global__ __launch_bounds__(256) void kv_append_kernel(KvBatch b, uint8_t* pages, const T* k, int64_t k_stride, const T* v,
                                                        int64_t v_stride, const T* q, int64_t q_stride, int n_heads,
                                                        const float* rope, int64_t rope_rows, int n_rot, int halves,
                                                        T* q_out) {
  constexpr int kPieces = D / 8, NB = D / 32;
  const int64_t row = blockIdx.x;
  const int seq = row_seq(b.cu, b.n_seq, row);
  if (seq >= b.n_seq || row < b.cu[seq]) return;
  const int64_t pos = static_cast<int64_t>(b.start[seq]) + (row - b.cu[seq]);
  if (n_rot > 0 && (pos < 0 || pos >= rope_rows)) return;
  const float* cs = rope + pos * n_rot;
  int piece = blockIdx.y * blockDim.x + threadIdx.x;
  const int kv_pieces = b.n_kv * kPieces;
  if (piece >= 2 * kv_pieces) {
    piece -= 2 * kv_pieces;
    if (piece >= n_heads * kPieces) return;
    const int e0 = piece % kPieces * 8;
    const T* p = q + row * q_stride + static_cast<int64_t>(piece) * 8;
    float x[8];
    load8(p, x);
    rotate8(p, e0, n_rot, halves != 0, cs, x);
    // in place (q_out == q) a partner half must be read before it is overwritten: both
    // halves of a head lie in one wavefront's pieces, see the launch
    store8(q_out + row * n_heads * D + static_cast<int64_t>(piece) * 8, x);
    return;
  }
  const int64_t page = page_of(b, seq, pos);
  if (page < 0) return;
  const bool is_v = piece >= kv_pieces;
  if (is_v) piece -= kv_pieces;
  const int head = piece / kPieces, e0 = piece % kPieces * 8;
  const T* p = (is_v ? v + row * v_stride : k + row * k_stride) + static_cast<int64_t>(piece) * 8;
  float x[8];
  load8(p, x);
  if (!is_v) rotate8(p, e0, n_rot, halves != 0, cs, x);
  float d;
  const uint32_t w = q4_0_piece(x, &d);
  const int64_t tokens = int64_t(1) << b.page_shift, slot = pos & (tokens - 1);
  const int64_t half = kv_half_bytes(tokens, D);
  uint8_t* base = pages + (page * b.n_kv + head) * 2 * half + (is_v ? half : 0);
  const int blk = e0 / 32, g = (e0 % 32) / 8;
  *reinterpret_cast<uint32_t*>(base + slot * (D / 2) + (g * NB + blk) * 4) = w;
  if (g == 0) *reinterpret_cast<uint16_t*>(base + tokens * (D / 2) + (slot * NB + blk) * 2) = f32_to_f16_bits(d);
}

// Workgroup (x, y): row x, code dwords y * blockDim + thread of the row's K, then V.
// value = d * (code - 8), exact in f32, rounded once to T.
template <typename T, int D>
__global__ __launch_bounds__(256) void kv_read_kernel(KvBatch b, const uint8_t* pages, T* k_out, T* v_out) {
  constexpr int kPieces = D / 8, NB = D / 32;
  const int64_t row = blockIdx.x;
  int piece = blockIdx.y * blockDim.x + threadIdx.x;
  const int kv_pieces = b.n_kv * kPieces;
  const int seq = row_seq(b.cu, b.n_seq, row);
  if (seq >= b.n_seq || row < b.cu[seq] || piece >= 2 * kv_pieces) return;
  const int64_t pos = static_cast<int64_t>(b.start[seq]) + (row - b.cu[seq]);
  const int64_t page = page_of(b, seq, pos);
  const bool is_v = piece >= kv_pieces;
  if (is_v) piece -= kv_pieces;
  const int head = piece / kPieces, at = piece % kPieces, g = at / NB, blk = at % NB;
  float x[8] = {};
  if (page >= 0) {
    const int64_t tokens = int64_t(1) << b.page_shift, slot = pos & (tokens - 1);
    const int64_t half = kv_half_bytes(tokens, D);
    const uint8_t* base = pages + (page * b.n_kv + head) * 2 * half + (is_v ? half : 0);
    const half8 c = nibbles_to_f16(*reinterpret_cast<const uint32_t*>(base + slot * (D / 2) + at * 4));
    const float d = f16_to_f32(*reinterpret_cast<const uint16_t*>(base + tokens * (D / 2) + (slot * NB + blk) * 2));
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = d * static_cast<float>(c[i]);
  }
  store8((is_v ? v_out : k_out) + (row * b.n_kv + head) * D + blk * 32 + g * 8, x);
}

template <typename T>
hipError_t append_t(const KvBatch& b, int dim, uint8_t* pages, const void* k, int64_t ks, const void* v, int64_t vs,
                    const void* q, int64_t qs, int n_heads, const float* rope, int64_t rope_rows, int n_rot, int halves,
                    void* q_out, hipStream_t s) {
  const int pieces = (2 * b.n_kv + n_heads) * (dim / 8);
  const int threads = pieces >= 256 ? 256 : (pieces + 63) / 64 * 64;
  unsigned gx = 0;
  const int64_t gy = (pieces + threads - 1) / threads;
  if (!launch_grid(b.n_rows * gy, threads, &gx) || gy > 65535) return hipErrorInvalidConfiguration;
  auto run = [&](auto kernel) {
    kernel<<<dim3(static_cast<unsigned>(b.n_rows), static_cast<unsigned>(gy)), threads, 0, s>>>(
        b, pages, static_cast<const T*>(k), ks, static_cast<const T*>(v), vs, static_cast<const T*>(q), qs, n_heads, rope,
        rope_rows, n_rot, halves, static_cast<T*>(q_out));
    return hipGetLastError();
  };
  switch (dim) {
    case 64: return run(kv_append_kernel<T, 64>);
    case 96: return run(kv_append_kernel<T, 96>);
    case 128: return run(kv_append_kernel<T, 128>);
    default: return run(kv_append_kernel<T, 256>);
  }
}

template <typename T>
hipError_t read_t(const KvBatch& b, int dim, const uint8_t* pages, void* k_out, void* v_out, hipStream_t s) {
  const int pieces = 2 * b.n_kv * (dim / 8);
  const int threads = pieces >= 256 ? 256 : (pieces + 63) / 64 * 64;
  unsigned gx = 0;
  const int64_t gy = (pieces + threads - 1) / threads;
  if (!launch_grid(b.n_rows * gy, threads, &gx) || gy > 65535) return hipErrorInvalidConfiguration;
  auto run = [&](auto kernel) {
    kernel<<<dim3(static_cast<unsigned>(b.n_rows), static_cast<unsigned>(gy)), threads, 0, s>>>(
        b, pages, static_cast<T*>(k_out), static_cast<T*>(v_out));
    return hipGetLastError();
  };
  switch (dim) {
    case 64: return run(kv_read_kernel<T, 64>);
    case 96: return run(kv_read_kernel<T, 96>);
    case 128: return run(kv_read_kernel<T, 128>);
    default: return run(kv_read_kernel<T, 256>);
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
