// qk_attn_paged.hip - attention of packed rows over the paged Q4_0 cache.
#include "qk_internal.h"
#include "qk_kv.h"

namespace qk {
namespace {

// One wavefront per (row, head): 64 positions at a time, a lane's score each, then one
// dim per lane over the 64 weights, with the running maximum and sum of the softmax.
template <typename T, int D>
__global__ __launch_bounds__(64) void attn_paged_kernel(KvBatch b, const uint8_t* pages, const T* q, int64_t q_stride,
                                                        int n_heads, float scale, int64_t window, T* out) {
  constexpr int NB = D / 32;
  __shared__ float sq[D], sp[64];
  __shared__ int64_t sbase[64];
  const int64_t row = blockIdx.x;
  const int head = blockIdx.y, kv = head / (n_heads / b.n_kv), lane = threadIdx.x;
  const int seq = row_seq(b.cu, b.n_seq, row);
  if (seq >= b.n_seq || row < b.cu[seq]) return;
  const int64_t pos = static_cast<int64_t>(b.start[seq]) + (row - b.cu[seq]);
  const int64_t lo = (window > 0 && pos - window + 1 > 0) ? pos - window + 1 : 0;
  for (int e = lane; e < D; e += 64) sq[e] = static_cast<float>(q[row * q_stride + head * D + e]) * scale;
  const int64_t tokens = int64_t(1) << b.page_shift, half = kv_half_bytes(tokens, D);
  float m = -INFINITY, l = 0.0f, o[(D + 63) / 64] = {};
  for (int64_t t0 = lo; t0 <= pos; t0 += 64) {
    const int64_t t = t0 + lane;
    const int64_t page = t <= pos ? page_of(b, seq, t) : -1;
    const int64_t slot = t & (tokens - 1);
    const int64_t base = (page * b.n_kv + kv) * 2 * half;
    float s = -INFINITY;
    __syncthreads();
    if (page >= 0) {
      s = 0.0f;
      for (int blk = 0; blk < NB; ++blk) {
        float a = 0.0f;
        for (int g = 0; g < 4; ++g) {
          const half8 c = nibbles_to_f16(
              *reinterpret_cast<const uint32_t*>(pages + base + slot * (D / 2) + (g * NB + blk) * 4));
#pragma unroll
          for (int j = 0; j < 8; ++j) a += sq[blk * 32 + g * 8 + j] * static_cast<float>(c[j]);
        }
        s += a * f16_to_f32(*reinterpret_cast<const uint16_t*>(pages + base + tokens * (D / 2) + (slot * NB + blk) * 2));
      }
    }
    const float mt = fmaxf(m, wave_max(s));
    const float p = s == -INFINITY ? 0.0f : expf(s - mt);
    const float keep = m == -INFINITY ? 0.0f : expf(m - mt);
    l = l * keep + wave_sum(p);
    m = mt;
    sp[lane] = p;
    sbase[lane] = page >= 0 ? base + half : -1;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < (D + 63) / 64; ++i) {
      const int e = lane + 64 * i;
      if (e >= D) break;
      const int blk = e / 32, g = e % 32 / 8, j = e % 8, n = (j >> 1) + 4 * (j & 1);
      float a = o[i] * keep;
      for (int u = 0; u < 64; ++u) {
        const int64_t vb = sbase[u], vs = (t0 + u) & (tokens - 1);
        if (vb < 0) continue;
        const uint32_t w = *reinterpret_cast<const uint32_t*>(pages + vb + vs * (D / 2) + (g * NB + blk) * 4);
        const float d = f16_to_f32(*reinterpret_cast<const uint16_t*>(pages + vb + tokens * (D / 2) + (vs * NB + blk) * 2));
        a += sp[u] * d * static_cast<float>(static_cast<int>((w >> (4 * n)) & 15) - 8);
      }
      o[i] = a;
    }
  }
  for (int i = 0; i < (D + 63) / 64; ++i) {
    const int e = lane + 64 * i;
    if (e < D) out[(row * n_heads + head) * D + e] = static_cast<T>(l != 0.0f ? o[i] / l : 0.0f);
  }
}

template <typename T>
hipError_t paged_t(const KvBatch& b, int dim, const uint8_t* pages, const void* q, int64_t q_stride, int n_heads,
                   float scale, int64_t window, void* out, hipStream_t s) {
  unsigned gx = 0;
  if (!launch_grid(b.n_rows * n_heads, 64, &gx) || n_heads > 65535) return hipErrorInvalidConfiguration;
  auto run = [&](auto kernel) {
    kernel<<<dim3(static_cast<unsigned>(b.n_rows), n_heads), 64, 0, s>>>(b, pages, static_cast<const T*>(q), q_stride,
                                                                         n_heads, scale, window, static_cast<T*>(out));
    return hipGetLastError();
  };
  switch (dim) {
    case 64: return run(attn_paged_kernel<T, 64>);
    case 96: return run(attn_paged_kernel<T, 96>);
    case 128: return run(attn_paged_kernel<T, 128>);
    default: return run(attn_paged_kernel<T, 256>);
  }
}

}  // namespace

int64_t attn_paged_ws_bytes(const KvBatch&, int, int) { return 0; }

hipError_t launch_attn_paged(const KvBatch& b, int dim, int dtype, const uint8_t* pages, const void* q, int64_t q_stride,
                             int n_heads, float scale, int64_t window, void* out, void*, hipStream_t s) {
  switch (dtype) {
    case kF32: return paged_t<float>(b, dim, pages, q, q_stride, n_heads, scale, window, out, s);
    case kF16: return paged_t<_Float16>(b, dim, pages, q, q_stride, n_heads, scale, window, out, s);
    default: return paged_t<bf16>(b, dim, pages, q, q_stride, n_heads, scale, window, out, s);
  }
}

}  // namespace qk
