// The rotation of a draft tree's nodes and the commit of its accepted path.
//
// Rotation: per node n of sequence b, at position p = pos[b, n], the step of
// qknorm_rope_append.cu (per-head QK-RMSNorm, RoPE, fusedtok README "Operators";
// cutileGPT README "The current runtime includes") with the rotated key and the value
// written to the tree's own buffers [B, Hkv, N, D] instead of a cache slot: a node's slot
// is its index, not its position, and rejected nodes never touch the cache.
//
// Commit: the accepted path's keys and values from the tree's buffers into the cache
// slots behind the sequence's tokens, a bit copy.
#include "dec_device.cuh"
#include "dec_launch.h"
#include "rope_angles.cuh"
#include "rotate_head.cuh"

namespace decattn {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

struct TreeRopeArgs {
  const __nv_bfloat16 *q_in, *k_new, *v_new, *q_norm_w, *k_norm_w;
  __nv_bfloat16 *q_out, *k_tree, *v_tree;
  const int32_t *pos, *n_nodes;
  uint32_t *error_word;
  int N, Hq, Hkv, interleaved;
  float eps;
};

// One CTA per (node, block of heads): the node's D/2 angles once in shared memory, then a
// warp per head.
template <int D>
__global__ void __launch_bounds__(kThreads) tree_rope_kernel(const TreeRopeArgs a,
                                                             const InvFreq inv,
                                                             const RopeTurns turns) {
  using L = Lanes<D>;
  constexpr int E = L::kE;
  __shared__ float s_cos[D / 2];
  __shared__ float s_sin[D / 2];
  pdl_launch_dependents();
  pdl_wait_prior_grid();
  const int row = blockIdx.x, b = row / a.N, n = row - b * a.N;
  const int warp = threadIdx.x >> 5, e0 = (threadIdx.x & 31) * E;
  if (a.n_nodes != nullptr) {
    const int live = a.n_nodes[b];
    if ((live < 0 || live > a.N) && threadIdx.x == 0 && n == 0 && blockIdx.y == 0 &&
        a.error_word != nullptr)
      atomicOr(a.error_word, kErrTreeClamped);
    if (n >= live) return;
  }
  const int p = a.pos[row];
  if (p < 0) {
    if (threadIdx.x == 0 && blockIdx.y == 0 && a.error_word != nullptr)
      atomicOr(a.error_word, kErrPosSkipped);
    return;
  }
  for (int i = threadIdx.x; i < D / 2; i += kThreads)
    rope_sincos_turns(p, turns.v[i], s_sin[i], s_cos[i]);
  __syncthreads();
  const int task = blockIdx.y * kWarps + warp;
  if (task >= a.Hq + a.Hkv) return;
  const bool is_q = task < a.Hq;
  const int g = task - a.Hq;
  const __nv_bfloat16 *nw = is_q ? a.q_norm_w : a.k_norm_w;
  const size_t q_at = ((size_t)row * a.Hq + task) * D + e0;
  const size_t kv_at = ((size_t)row * a.Hkv + g) * D + e0;
  float x[E], w[E] = {}, y[E];
  L::load(is_q ? a.q_in + q_at : a.k_new + kv_at, x);
  if (nw != nullptr) L::load(nw + e0, w);
  LaneAngles<D> ang;
  ang.from_table(s_cos, s_sin, a.interleaved);
  double fr[E] = {};
  if (!is_q) lane_freqs<D>(inv, a.interleaved, fr);  // for the exact path of a cancelling K
  rotate_values<D>(x, w, nw != nullptr, !is_q, ang, p, fr, a.interleaved, a.eps, y);
  if (is_q) {
    L::store(a.q_out + q_at, y);
  } else {
    const size_t slot = (((size_t)b * a.Hkv + g) * a.N + n) * D + e0;
    L::store(a.k_tree + slot, y);
    L::copy(a.v_tree + slot, a.v_new + kv_at);
  }
}

struct TreeCommitArgs {
  const uint4 *k_tree, *v_tree;
  uint4 *k_cache, *v_cache;
  const int32_t *path, *n_path, *lens;
  uint32_t *error_word;
  int N, Hkv, T_cap, vec;  // vec: 16-byte words per row
};

// One CTA per (sequence, KV head): the path's rows of K and V, 16 bytes per thread.
__global__ void __launch_bounds__(kThreads) tree_commit_kernel(const TreeCommitArgs a) {
  pdl_launch_dependents();
  pdl_wait_prior_grid();
  const int b = blockIdx.y, g = blockIdx.x;
  int count = a.n_path[b];
  const int at = a.lens[b];
  const bool report = g == 0 && threadIdx.x == 0 && a.error_word != nullptr;
  if (count < 0 || count > a.N) {
    if (report) atomicOr(a.error_word, kErrTreeClamped);
    count = count < 0 ? 0 : a.N;
  }
  const size_t pair = (size_t)b * a.Hkv + g;
  for (int i = threadIdx.x; i < count * a.vec; i += kThreads) {
    const int r = i / a.vec, c = i - r * a.vec;
    const int node = a.path[(size_t)b * a.N + r];
    const long long slot = (long long)at + r;
    if (node < 0 || node >= a.N || slot < 0 || slot >= a.T_cap) {
      if (g == 0 && c == 0 && a.error_word != nullptr) atomicOr(a.error_word, kErrPosSkipped);
      continue;
    }
    const size_t src = (pair * a.N + node) * a.vec + c, dst = (pair * a.T_cap + slot) * a.vec + c;
    a.k_cache[dst] = a.k_tree[src];
    a.v_cache[dst] = a.v_tree[src];
  }
}

}  // namespace

cudaError_t launch_tree_rope(const void *q_in, void *q_out, const void *k_new, const void *v_new,
                             const void *q_norm_w, const void *k_norm_w, void *k_tree,
                             void *v_tree, const int32_t *pos, const int32_t *n_nodes, int B,
                             int N, int Hq, int Hkv, int D, const InvFreq &inv, int interleaved,
                             float eps, uint32_t *error_word, cudaStream_t stream) {
  auto in = [](const void *p) { return static_cast<const __nv_bfloat16 *>(p); };
  auto io = [](void *p) { return static_cast<__nv_bfloat16 *>(p); };
  const TreeRopeArgs a{in(q_in), in(k_new), in(v_new), in(q_norm_w), in(k_norm_w),
                       io(q_out), io(k_tree), io(v_tree), pos, n_nodes, error_word,
                       N, Hq, Hkv, interleaved, eps};
  const dim3 grid(B * N, (Hq + Hkv + kWarps - 1) / kWarps);
  const RopeTurns turns = make_rope_turns(D, inv);
  const cudaError_t e =
      D == 128 ? launch_pdl(tree_rope_kernel<128>, grid, kThreads, 0, stream, a, inv, turns)
               : launch_pdl(tree_rope_kernel<64>, grid, kThreads, 0, stream, a, inv, turns);
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_tree_commit(const void *k_tree, const void *v_tree, const int32_t *path,
                               const int32_t *n_path, void *k_cache, void *v_cache,
                               const int32_t *lens, int B, int N, int Hkv, int D, int T_cap,
                               uint32_t *error_word, cudaStream_t stream) {
  const TreeCommitArgs a{static_cast<const uint4 *>(k_tree), static_cast<const uint4 *>(v_tree),
                         static_cast<uint4 *>(k_cache), static_cast<uint4 *>(v_cache), path,
                         n_path, lens, error_word, N, Hkv, T_cap, D / 8};
  const cudaError_t e =
      launch_pdl(tree_commit_kernel, dim3(Hkv, B), kThreads, 0, stream, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace decattn
