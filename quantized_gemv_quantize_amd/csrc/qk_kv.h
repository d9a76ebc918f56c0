// qk_kv.h - the paged Q4_0 KV cache: its layout and the device helpers that the
// append, read and attention kernels share.
//
// pages: uint8 [n_pages][n_kv_heads][page bytes].  One page of one head, T = tokens per
// page, D = head dim, NB = D / 32 blocks per row:
//   K codes  T rows of D / 2 bytes     K scales  T rows of NB f16
//   V codes  T rows of D / 2 bytes     V scales  T rows of NB f16
// The Q4_0 block's 18 bytes are split into a code plane and a scale plane, so that every
// code row is 16-byte aligned at any NB (18-byte blocks are 2-byte aligned) and four
// tokens' scales are one aligned load.  T is a multiple of 16, which makes every plane a
// multiple of 16 bytes.
//
// A code row is 4 groups g of NB dwords b; dword (g, b) holds dims 32 b + 8 g + j,
// j = 0..7.  A matrix-instruction operand takes from lane group g the 8 dims 8 g + j of
// one block, so a lane's operands of all NB blocks are NB consecutive dwords, one load.
// Nibble n of a dword holds j = 2 n (n < 4) or 2 (n - 4) + 1: masking a dword with
// 0x000F000F << 4 n leaves dims 2 n and 2 n + 1 in the two halves, which one OR turns
// into a pair of f16 (see nibbles_to_f16).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "qk_device.h"

namespace qk {

typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef _Float16 half2v __attribute__((ext_vector_type(2)));
typedef uint32_t uint4v __attribute__((ext_vector_type(4)));
typedef float float4v __attribute__((ext_vector_type(4)));
typedef __bf16 bf16;
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// The packed rows of a batch and where each lies in the cache (qk_kv_batch, checked).
struct KvBatch {
  const int32_t* table;  // [n_seq][max_pages]
  const int32_t* cu;     // [n_seq + 1] first packed row of each sequence
  const int32_t* start;  // [n_seq] cache position of that row
  int64_t max_pages, n_pages;
  int64_t n_rows;
  int n_seq, n_kv, page_shift;
};

// The packed rows of whole prompts: sequence i holds q rows cu_q[i] .. cu_q[i + 1] and keys
// cu_k[i] .. cu_k[i + 1], the last rows aligned.
struct PromptBatch {
  const int32_t *cu_q, *cu_k;  // [n_seq + 1]
  int64_t q_stride, k_stride, v_stride;
  int64_t n_q, n_k, window;
  int n_seq, n_heads, n_kv, causal;
};

__host__ __device__ constexpr int64_t kv_half_bytes(int64_t page_tokens, int64_t dim) {
  return page_tokens * (dim / 2 + dim / 16);
}

// Sequences of packed rows row0 .. row0 + 3: for each the number of cu[1..n_seq] that are <= row, n_seq when it
// lies behind the last sequence.  All 64 lanes of the wavefront call it with the same row; each tests
// one entry of 64, so the lookup is one load and four ballots up to 64 sequences (a binary search is a chain
// of 6 loads).
__device__ __forceinline__ void row_seq4(const int32_t* cu, int n_seq, int64_t row0, int* seq) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int r = 0; r < 4; ++r) seq[r] = 0;
  for (int i = 0; i < n_seq; i += 64) {
    const int64_t end = i + lane < n_seq ? cu[i + lane + 1] : INT64_MAX;
#pragma unroll
    for (int r = 0; r < 4; ++r) seq[r] += __popcll(__ballot(end <= row0 + r));
  }
}

// Page of `pos` in sequence `seq`, -1 when the position or the table's entry is out of
// range (such a page is never followed).
__device__ __forceinline__ int64_t page_of(const KvBatch& b, int seq, int64_t pos) {
  if (pos < 0) return -1;
  const int64_t at = pos >> b.page_shift;
  if (at >= b.max_pages) return -1;
  const int32_t page = b.table[seq * b.max_pages + at];
  return (page >= 0 && page < b.n_pages) ? page : -1;
}

// Codes as f16 integers -8..7 from bits 0..3 (low) or 4..7 (high) of both halves of x: 0x6400 | n is
// 1024 + n and 0x6400 | n << 4 is 1024 + 16 n, both exact; the subtraction and the multiply-add that
// bring them to n - 8 are exact too.  The constants are kept in registers (a scalar and a
// vector one) so that mask and OR are one v_and_or_b32, which takes no literals.
__device__ __forceinline__ uint32_t and_or(uint32_t x, uint32_t mask) {
  uint32_t magic = 0x64006400u;
  asm("" : "+v"(magic));
  asm("" : "+s"(mask));
  return (x & mask) | magic;
}
__device__ __forceinline__ uint32_t low_nibbles(uint32_t x) {
  const half2v off = {static_cast<_Float16>(-1032.0f), static_cast<_Float16>(-1032.0f)};
  return __builtin_bit_cast(uint32_t, __builtin_bit_cast(half2v, and_or(x, 0x000F000Fu)) + off);
}
__device__ __forceinline__ uint32_t high_nibbles(uint32_t x) {
  const half2v sixteenth = {static_cast<_Float16>(0.0625f), static_cast<_Float16>(0.0625f)};
  const half2v off = {static_cast<_Float16>(-72.0f), static_cast<_Float16>(-72.0f)};
  return __builtin_bit_cast(uint32_t,
                            __builtin_elementwise_fma(__builtin_bit_cast(half2v, and_or(x, 0x00F000F0u)), sixteenth, off));
}
// The 8 codes of a dword, in dim order.
__device__ __forceinline__ half8 nibbles_to_f16(uint32_t w) {
  const uint32_t w8 = w >> 8;
  return __builtin_bit_cast(half8, uint4v{low_nibbles(w), high_nibbles(w), low_nibbles(w8), high_nibbles(w8)});
}

// Largest value and sum over the four lanes of equal lane % 16, returned in all of them.
__device__ __forceinline__ float rows_max(float x) {
  auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  a = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
}
__device__ __forceinline__ float rows_sum(float x) {
  auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  a = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(a[0]) + __uint_as_float(a[1]);
}

// Starts a load of 16 bytes a lane from `rsrc` (offset `lane_at` a lane, `at` for all; zeros beyond its end)
// to LDS, lane i's at `to` + 16 i.  Nothing but wait_loads waits for it: the compiler orders no LDS read behind it.
__device__ __forceinline__ void load_to_lds(__amdgpu_buffer_rsrc_t rsrc, void* to, int lane_at, int at) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (__attribute__((address_space(3))) void*)to, 16, lane_at, at, 0, 0);
}
// Waits until at most N of the wavefront's loads are on the way; loads end in order.
template <int N>
__device__ __forceinline__ void wait_loads() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// 8 consecutive elements (16-byte aligned) as f32, and back with one rounding each.
__device__ __forceinline__ void load8(const float* p, float* v) {
  const float4v a = reinterpret_cast<const float4v*>(p)[0], b = reinterpret_cast<const float4v*>(p)[1];
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = a[i], v[4 + i] = b[i];
}
__device__ __forceinline__ void load8(const _Float16* p, float* v) {
  const half8 a = *reinterpret_cast<const half8*>(p);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = static_cast<float>(a[i]);
}
__device__ __forceinline__ void load8(const bf16* p, float* v) {
  const bf16x8 a = *reinterpret_cast<const bf16x8*>(p);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = static_cast<float>(a[i]);
}
__device__ __forceinline__ void store8(float* p, const float* v) {
  reinterpret_cast<float4v*>(p)[0] = float4v{v[0], v[1], v[2], v[3]};
  reinterpret_cast<float4v*>(p)[1] = float4v{v[4], v[5], v[6], v[7]};
}
__device__ __forceinline__ void store8(_Float16* p, const float* v) {
  half8 a;
#pragma unroll
  for (int i = 0; i < 8; ++i) a[i] = static_cast<_Float16>(v[i]);
  *reinterpret_cast<half8*>(p) = a;
}
__device__ __forceinline__ void store8(bf16* p, const float* v) {
  bf16x8 a;
#pragma unroll
  for (int i = 0; i < 8; ++i) a[i] = static_cast<bf16>(v[i]);
  *reinterpret_cast<bf16x8*>(p) = a;
}

}  // namespace qk
