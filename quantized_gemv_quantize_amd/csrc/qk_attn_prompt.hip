// qk_attn_prompt.hip - attention over whole packed prompts held as float q, k, v.
#include "qk_internal.h"
#include "qk_kv.h"

namespace qk {
namespace {

// One wavefront per (row, head): 64 keys at a time, a lane's score each, then one dim per
// lane over the 64 weights, with the running maximum and sum of the softmax.
template <typename T, int D>
__global__ __launch_bounds__(64) void attn_prompt_kernel(PromptBatch b, const T* q, const T* k, const T* v, float scale,
                                                         T* out) {
  __shared__ float sq[D], sp[64];
  const int64_t row = blockIdx.x;
  const int head = blockIdx.y, kv = head / (b.n_heads / b.n_kv), lane = threadIdx.x;
  const int seq = row_seq(b.cu_q, b.n_seq, row);
  if (seq >= b.n_seq || row < b.cu_q[seq]) return;
  const int64_t q0 = b.cu_q[seq], q1 = b.cu_q[seq + 1];
  int64_t k0 = b.cu_k[seq], k1 = b.cu_k[seq + 1];
  k0 = k0 < 0 ? 0 : k0, k1 = k1 > b.n_k ? b.n_k : k1;
  const int64_t len = k1 - k0, at = row - q0 + len - (q1 - q0);
  const int64_t hi = b.causal ? (at + 1 < len ? at + 1 : len) : len;
  const int64_t lo = (b.window > 0 && at - b.window + 1 > 0) ? at - b.window + 1 : 0;
  for (int e = lane; e < D; e += 64) sq[e] = static_cast<float>(q[row * b.q_stride + head * D + e]) * scale;
  float m = -INFINITY, l = 0.0f, o[(D + 63) / 64] = {};
  for (int64_t t0 = lo; t0 < hi; t0 += 64) {
    const int64_t t = t0 + lane;
    float s = -INFINITY;
    __syncthreads();
    if (t < hi) {
      s = 0.0f;
      for (int e = 0; e < D; e += 8) {
        float x[8];
        load8(k + (k0 + t) * b.k_stride + kv * D + e, x);
#pragma unroll
        for (int j = 0; j < 8; ++j) s += sq[e + j] * x[j];
      }
    }
    const float mt = fmaxf(m, wave_max(s));
    const float p = t < hi ? expf(s - mt) : 0.0f;
    const float keep = m == -INFINITY ? 0.0f : expf(m - mt);
    l = l * keep + wave_sum(p);
    m = mt;
    sp[lane] = p;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < (D + 63) / 64; ++i) {
      const int e = lane + 64 * i;
      if (e >= D) break;
      float a = o[i] * keep;
      for (int u = 0; u < 64 && t0 + u < hi; ++u)
        a += sp[u] * static_cast<float>(v[(k0 + t0 + u) * b.v_stride + kv * D + e]);
      o[i] = a;
    }
  }
  for (int i = 0; i < (D + 63) / 64; ++i) {
    const int e = lane + 64 * i;
    if (e < D) out[(row * b.n_heads + head) * D + e] = static_cast<T>(l != 0.0f ? o[i] / l : 0.0f);
  }
}

template <typename T>
hipError_t prompt_t(const PromptBatch& b, int dim, const void* q, const void* k, const void* v, float scale, void* out,
                    hipStream_t s) {
  unsigned gx = 0;
  if (!launch_grid(b.n_q * b.n_heads, 64, &gx) || b.n_heads > 65535) return hipErrorInvalidConfiguration;
  auto run = [&](auto kernel) {
    kernel<<<dim3(static_cast<unsigned>(b.n_q), b.n_heads), 64, 0, s>>>(
        b, static_cast<const T*>(q), static_cast<const T*>(k), static_cast<const T*>(v), scale, static_cast<T*>(out));
    return hipGetLastError();
  };
  switch (dim) {
    case 64: return run(attn_prompt_kernel<T, 64>);
    case 96: return run(attn_prompt_kernel<T, 96>);
    case 128: return run(attn_prompt_kernel<T, 128>);
    default: return run(attn_prompt_kernel<T, 256>);
  }
}

}  // namespace

hipError_t launch_attn_prompt(const PromptBatch& b, int dim, int dtype, const void* q, const void* k, const void* v,
                              float scale, void* out, hipStream_t s) {
  switch (dtype) {
    case kF32: return prompt_t<float>(b, dim, q, k, v, scale, out, s);
    case kF16: return prompt_t<_Float16>(b, dim, q, k, v, scale, out, s);
    default: return prompt_t<bf16>(b, dim, q, k, v, scale, out, s);
  }
}

}  // namespace qk
