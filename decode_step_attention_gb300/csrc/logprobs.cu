// Log probabilities of given tokens, the entropy of the distribution and its best
// alternatives, for every row of a batch of logits (the scoring side of the sampler's
// softmax, sampler.cu):
//
//   z = logits / T,  M = max z,  S = sum e^(z - M),  lse = M + ln S
//   logprob(id) = z_id - lse
//   entropy     = ln S - (sum e^(z - M) (z - M)) / S      (nats)
//   top K       : the K largest logits, equal ones by the lower id
//
// One CTA per row: a pass for the maximum, one for the sums, one per alternative.
#include <math.h>

#include "dec_device.cuh"
#include "dec_launch.h"

namespace decattn {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;

__device__ __forceinline__ float logit(const LogprobArgs &a, size_t i) {
  return a.bf16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(a.logits)[i])
                : static_cast<const float *>(a.logits)[i];
}

// Orders by value, then by the lower id: larger is better. NaN orders by its bits.
__device__ __forceinline__ unsigned long long rank_key(float v, int id) {
  if (v == 0.f) v = 0.f;  // -0 and 0 are equal values
  unsigned u = __float_as_uint(v);
  u = (u & 0x80000000u) ? ~u : u | 0x80000000u;
  return ((unsigned long long)u << 32) | (unsigned)~id;
}

template <typename T, typename F>
__device__ T block_reduce(T v, T *s, F f) {
  for (int o = 16; o > 0; o >>= 1) v = f(v, __shfl_xor_sync(0xffffffffu, v, o));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
  __syncthreads();
  T r = s[0];
  for (int w = 1; w < kWarps; ++w) r = f(r, s[w]);
  return r;
}

__global__ void __launch_bounds__(kThreads) logprobs_kernel(const LogprobArgs a) {
  __shared__ float s_f[kWarps];
  __shared__ unsigned long long s_k[kWarps];
  pdl_launch_dependents();
  pdl_wait_prior_grid();
  const size_t row = blockIdx.x, base = row * (size_t)a.ld;
  const int tid = threadIdx.x;
  const float inv_t = 1.f / a.temperature;
  float m = -INFINITY;
  bool bad = false;
  for (int i = tid; i < a.V; i += kThreads) {
    const float v = logit(a, base + i);
    bad |= isnan(v);
    m = fmaxf(m, v);
  }
  bad = __syncthreads_or(bad);
  m = block_reduce(m, s_f, [](float x, float y) { return fmaxf(x, y); });
  float s = 0.f, c = 0.f;
  for (int i = tid; i < a.V; i += kThreads) {
    const float d = (logit(a, base + i) - m) * inv_t, e = expf(d);
    s += e;
    if (e > 0.f) c = fmaf(e, d, c);
  }
  auto add = [](float x, float y) { return x + y; };
  s = block_reduce(s, s_f, add);
  c = block_reduce(c, s_f, add);
  const float ln_s = (bad || isinf(m)) ? NAN : logf(s);
  if (tid == 0 && a.entropy != nullptr) a.entropy[row] = ln_s - c / s;
  for (int i = tid; i < a.C; i += kThreads) {
    const int id = a.ids[row * a.C + i];
    const float v = id >= 0 && id < a.V ? logit(a, base + id) : -INFINITY;
    a.logprobs[row * a.C + i] = (v - m) * inv_t - ln_s;
  }
  unsigned long long last = ~0ull;
  for (int k = 0; k < a.K; ++k) {
    unsigned long long best = 0;
    for (int i = tid; i < a.V; i += kThreads) {
      const unsigned long long key = rank_key(logit(a, base + i), i);
      if (key < last && key > best) best = key;
    }
    best = block_reduce(best, s_k, [](unsigned long long x, unsigned long long y) {
      return x > y ? x : y;
    });
    last = best;
    if (tid == 0) {
      const int id = (int)~(unsigned)best;
      a.top_ids[row * a.K + k] = id;
      a.top_logprobs[row * a.K + k] = (logit(a, base + id) - m) * inv_t - ln_s;
    }
  }
}

}  // namespace

cudaError_t launch_logprobs(const LogprobArgs &a, int B, cudaStream_t stream) {
  const cudaError_t e = launch_pdl(logprobs_kernel, dim3(B), kThreads, 0, stream, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace decattn
