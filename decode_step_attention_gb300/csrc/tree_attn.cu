// Attention of a draft tree's nodes over the cached prefix and their ancestors
// (the single-query attention of gqa_decode.cu for N queries per sequence).
//
//   z[n, h, t]   = scale q[b,n,h] . K_t          t over the cache rows [0, lens[b])
//                                                and the tree's nodes
//   z           <- cap tanh(z / cap)             (softcap > 0)
//   z           <- z - slope_h (pos_n - kpos_t)  (slopes given; kpos = slot or pos of node)
//   out[b,n,h]   = sum_t softmax_t(z) V_t        over the rows node n sees
//
// One CTA per (query head, node, sequence): 128 threads score 128 rows at a time, then add
// their weighted values with one thread per dimension.
#include <math.h>

#include "dec_device.cuh"
#include "dec_launch.h"

namespace decattn {
namespace {

constexpr int kThreads = 128;

template <int D>
__global__ void __launch_bounds__(kThreads) tree_attn_kernel(const TreeAttnArgs a) {
  __shared__ float s_q[D], s_p[kThreads], s_red[4];
  pdl_launch_dependents();
  pdl_wait_prior_grid();
  const int h = blockIdx.x, n = blockIdx.y, b = blockIdx.z, g = h / (a.Hq / a.Hkv);
  const int tid = threadIdx.x;
  int L = a.lens[b], live = a.n_nodes != nullptr ? a.n_nodes[b] : a.N;
  if (tid == 0 && h == 0 && n == 0) {
    if (L < 0 || L > a.T_cap) atomicOr(a.error_word, kErrLenClamped);
    if (live < 0 || live > a.N) atomicOr(a.error_word, kErrTreeClamped);
  }
  L = min(max(L, 0), a.T_cap);
  live = min(max(live, 0), a.N);
  if (n >= live) return;
  const size_t row = (size_t)b * a.N + n, pair = (size_t)b * a.Hkv + g;
  const uint64_t seen = a.mask[row];
  const int qpos = a.pos != nullptr ? max(a.pos[row], L) : 0;
  const float slope = a.slopes != nullptr ? a.slopes[h] : 0.f;
  const size_t q_at = (row * a.Hq + h) * D;
  for (int d = tid; d < D; d += kThreads) s_q[d] = __bfloat162float(a.q[q_at + d]);
  __syncthreads();
  float m = -INFINITY, l = 0.f, o = 0.f;
  for (int t0 = 0; t0 < L + live; t0 += kThreads) {
    const int t = t0 + tid, j = t - L;
    bool ok = t < L + live;
    int kpos = t;
    if (ok && j >= 0) {
      ok = (seen >> j) & 1;
      if (a.pos != nullptr) kpos = max(a.pos[(size_t)b * a.N + j], L);
    }
    if (a.window > 0) ok = ok && qpos - kpos < a.window;
    float z = -INFINITY;
    if (ok) {
      const __nv_bfloat16 *k = j >= 0 ? a.k_tree + (pair * a.N + j) * D
                                      : a.k_cache + (pair * a.T_cap + t) * D;
      float s = 0.f;
      for (int d = 0; d < D; ++d) s = fmaf(s_q[d], __bfloat162float(k[d]), s);
      s *= a.scale;
      if (a.softcap > 0.f) s = a.softcap * tanhf(s / a.softcap);
      z = s - slope * (float)(qpos - kpos);
    }
    float mx = z;
    for (int i = 16; i > 0; i >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, i));
    if ((tid & 31) == 0) s_red[tid >> 5] = mx;
    __syncthreads();
    mx = fmaxf(fmaxf(s_red[0], s_red[1]), fmaxf(s_red[2], s_red[3]));
    const float mn = fmaxf(m, mx), base = mn == -INFINITY ? 0.f : mn;
    const float corr = expf(m - base);
    m = mn;
    s_p[tid] = ok ? expf(z - base) : 0.f;
    // which rows are seen: a masked row's value may be anything and is not read
    const bool use = ok;
    const unsigned bits = __ballot_sync(0xffffffffu, use);
    __shared__ unsigned s_use[4];
    if ((tid & 31) == 0) s_use[tid >> 5] = bits;
    __syncthreads();
    l *= corr;
    o *= corr;
    for (int i = 0; i < kThreads; ++i) {
      if (!((s_use[i >> 5] >> (i & 31)) & 1)) continue;
      l += s_p[i];
      if (tid < D) {
        const int ti = t0 + i, ji = ti - L;
        const __nv_bfloat16 *v = ji >= 0 ? a.v_tree + (pair * a.N + ji) * D
                                         : a.v_cache + (pair * a.T_cap + ti) * D;
        o = fmaf(s_p[i], __bfloat162float(v[tid]), o);
      }
    }
    __syncthreads();
  }
  if (tid < D) a.out[q_at + tid] = __float2bfloat16(l == 0.f ? 0.f : o / l);
}

}  // namespace

int tree_parts(int, int, int, int, int, int num_parts, int) { return num_parts > 0 ? num_parts : 1; }

size_t tree_ws_bytes(int, int, int, int, int, int) { return kWsHeaderBytes; }

cudaError_t launch_tree_attn(const TreeAttnArgs &a, int B, int D, cudaStream_t stream) {
  const dim3 grid(a.Hq, a.N, B);
  const cudaError_t e = D == 128
                            ? launch_pdl(tree_attn_kernel<128>, grid, kThreads, 0, stream, a)
                            : launch_pdl(tree_attn_kernel<64>, grid, kThreads, 0, stream, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace decattn
