// Single-query GQA attention over a paged cache of bf16 values or e4m3 codes with a scale per
// (page, KV head): out[b, h] = sum_t softmax_t(scale q[b, h] . K_t) V_t over the last `window` tokens
// (all of them without one).
//
// One block per (sequence, KV head): each of 8 warps takes every eighth token, a query group's heads
// in registers, with a running maximum and sum; the warps' states are joined at the end.
#include <cuda_fp8.h>

#include "dec_device.cuh"
#include "dec_launch.h"

namespace decattn {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kG = kSplitMaxG;

template <int D, bool kE4m3>
__device__ __forceinline__ void load_row(const void *pages, size_t row, int lane,
                                         float (&x)[D / 32]) {
  constexpr int E = D / 32;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const size_t i = row * D + lane * E + e;
    if (kE4m3) {
      __nv_fp8_e4m3 c;
      c.__x = static_cast<const uint8_t *>(pages)[i];
      x[e] = (float)c;
    } else {
      x[e] = __bfloat162float(static_cast<const __nv_bfloat16 *>(pages)[i]);
    }
  }
}

template <int D, bool kE4m3>
__global__ void __launch_bounds__(kThreads)
    paged_attn_kernel(const PagedCache c, const PagedAttnArgs a, int page_log2) {
  constexpr int E = D / 32;
  __shared__ float s_o[kWarps][kG][D], s_m[kWarps][kG], s_l[kWarps][kG];
  pdl_launch_dependents();
  pdl_wait_prior_grid();
  const int b = blockIdx.y, g = blockIdx.x, G = a.Hq / c.Hkv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int len = a.lens[b];
  const int L = min(max(len, 0), a.max_len);
  if (L != len && g == 0 && threadIdx.x == 0) atomicOr(a.error_word, kErrLenClamped);
  const int first = a.window > 0 ? max(0, L - a.window) : 0;
  float q[kG][E], o[kG][E] = {}, m[kG], l[kG] = {};
#pragma unroll
  for (int h = 0; h < kG; ++h) {
    m[h] = -INFINITY;
#pragma unroll
    for (int e = 0; e < E; ++e)
      q[h][e] = h < G ? __bfloat162float(a.q[((size_t)b * a.Hq + g * G + h) * D + lane * E + e]) *
                            a.scale_log2
                      : 0.f;
  }
  for (int t = first + warp; t < L; t += kWarps) {
    const int page = c.table[(size_t)b * c.max_pages + (t >> page_log2)];
    if (page < 0 || page >= c.num_pages) {
      if (g == 0 && lane == 0) atomicOr(a.error_word, kErrPageSkipped);
      continue;
    }
    const size_t head = (size_t)page * c.Hkv + g;
    const size_t row = (head << page_log2) + (t & ((1 << page_log2) - 1));
    const float ks = kE4m3 ? c.k_scale[head] : 1.f, vs = kE4m3 ? c.v_scale[head] : 1.f;
    float k[E], v[E];
    load_row<D, kE4m3>(c.k_pages, row, lane, k);
    load_row<D, kE4m3>(c.v_pages, row, lane, v);
#pragma unroll
    for (int h = 0; h < kG; ++h) {
      if (h >= G) break;
      float z = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) z = fmaf(q[h][e], k[e], z);
      z = warp_sum(z) * ks;
      const float to = fmaxf(m[h], z), base = to == -INFINITY ? 0.f : to;
      const float alpha = exp2f(m[h] - base), p = exp2f(z - base);
      m[h] = to;
      l[h] = l[h] * alpha + p;
#pragma unroll
      for (int e = 0; e < E; ++e) o[h][e] = o[h][e] * alpha + p * vs * v[e];
    }
  }
#pragma unroll
  for (int h = 0; h < kG; ++h) {
#pragma unroll
    for (int e = 0; e < E; ++e) s_o[warp][h][lane * E + e] = o[h][e];
    if (lane == 0) s_m[warp][h] = m[h], s_l[warp][h] = l[h];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < G * D; i += kThreads) {
    const int h = i / D, d = i - h * D;
    float M = -INFINITY, sum = 0.f, x = 0.f;
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_m[w][h]);
    const float base = M == -INFINITY ? 0.f : M;
    for (int w = 0; w < kWarps; ++w) {
      const float f = exp2f(s_m[w][h] - base);
      sum += f * s_l[w][h];
      x += f * s_o[w][h][d];
    }
    a.out[((size_t)b * a.Hq + g * G + h) * D + d] = __float2bfloat16(sum == 0.f ? 0.f : x / sum);
  }
}

}  // namespace

int paged_attn_parts(int, int, int, int, int) { return 1; }
size_t paged_attn_ws_bytes(int, int, int, int, int) { return 256; }

cudaError_t launch_paged_attn(const PagedCache &c, const PagedAttnArgs &a, int, void *,
                              cudaStream_t stream) {
  int log2 = 4;
  while ((1 << log2) < c.page) ++log2;
  auto *kernel = c.D == 128 ? (c.e4m3 ? paged_attn_kernel<128, true> : paged_attn_kernel<128, false>)
                            : (c.e4m3 ? paged_attn_kernel<64, true> : paged_attn_kernel<64, false>);
  const cudaError_t e = launch_pdl(kernel, dim3(c.Hkv, a.B), kThreads, 0, stream, c, a, log2);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace decattn
