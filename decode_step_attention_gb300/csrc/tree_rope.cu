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
#include <type_traits>

#include "dec_device.cuh"
#include "dec_launch.h"
#include "rope_angles.cuh"

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

// Elements of a rotated key whose fp32 rotation cancels (bits of this lane's 8), formed again
// in fp64 from the stored input and written over. Rare: one lane in some 300.
__device__ __noinline__ void exact_elements(const __nv_bfloat16 *k, const __nv_bfloat16 *w,
                                            __nv_bfloat16 *dst,
                                            const unsigned long long *turns, int half,
                                            int interleaved, int e0, int p, float rstd,
                                            unsigned bits) {
  for (; bits != 0; bits &= bits - 1) {
    const int j = e0 + __ffs(bits) - 1;
    const int other = interleaved ? j ^ 1 : j ^ half;  // the head's D is 2 half, a power of 2
    const int pair = interleaved ? j >> 1 : j & (half - 1);
    const bool second = interleaved ? (j & 1) != 0 : j >= half;
    const float wj = w != nullptr ? __bfloat162float(w[j]) : 1.f;
    const float wo = w != nullptr ? __bfloat162float(w[other]) : 1.f;
    dst[j] = __float2bfloat16(rope_exact_turns(p, turns[pair], __bfloat162float(k[j]) * wj,
                                               __bfloat162float(k[other]) * wo, rstd, second));
  }
}

// One CTA per (node, block of heads). A head is D / 8 lanes of 16 bytes, so a warp turns 2 (D =
// 128) or 4 (64) heads at a time, P times over: q heads, then k heads, then v heads (copied).
// Every load is in flight while the node's D/2 angles are formed in shared memory. The
// arithmetic is that of rotate_head.cuh in another lane layout: the same sums in the same
// order, the rotated pair with the same roundings, so both give the same bits.
//
// A node's chain (position, angles, barrier, rotation, stores) is hidden by the other CTAs of
// the SM, and the instructions, some 130 per 8 elements of a head and lane, take 80% of the
// issue slots: 6144 nodes of 32 query and 8 KV heads of 128 (interleaved, normed), 114 MB,
// in 27.2 us, 4.2 TB/s. With 8-byte lanes 105 us. Six CTAs per SM, at 40 registers, against
// five at 48: 26.8 and 27.6 us, 16 query heads 20.7 and 22.0; one pass (a few nodes) and
// four lose by it: 8 nodes 3.19 and 3.05 us, 64 query heads in four passes 47.7 and 46.9 (in
// two CTAs of three 44.2). (The
// packed products or a branch around the check for cancelling keys cost more in registers
// than they save: 28.3 and 29.9 us.)
//
// kMoreValues: there are more value heads than one pass of the CTA holds, so that a warp whose
// heads are all values in one pass may hold more in the next. Without it the warp is done there:
// the same 6144 nodes in 27.2 us, with it 28.9; 32 KV heads, which need it, 64 (interleaved).
template <int D, int P, bool kMoreValues>
__global__ void __launch_bounds__(kThreads, P == 2 || P == 3 ? 6 : 5)
    tree_rope_kernel(const TreeRopeArgs a, const __grid_constant__ RopeTurns turns) {
  constexpr int kLanes = D / 8;           // lanes per head
  constexpr int kHeads = 32 / kLanes;     // heads per warp and pass
  constexpr int kStep = kWarps * kHeads;  // heads per pass of the CTA
  constexpr int kOld = D / 32;            // elements summed in one chain
  constexpr int kChains = 8 / kOld;
  __shared__ __align__(16) float s_cos[D / 2];
  __shared__ __align__(16) float s_sin[D / 2];
  pdl_launch_dependents();
  pdl_wait_prior_grid();
  const int n = blockIdx.x, b = blockIdx.z;
  const size_t row = (size_t)b * a.N + n;
  const int live = a.n_nodes != nullptr ? a.n_nodes[b] : a.N;
  const int p = a.pos[row];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int hl = lane & (kLanes - 1), e0 = hl * 8;
  const int rotated = a.Hq + a.Hkv, heads = rotated + a.Hkv;
  const int task0 = (blockIdx.y * P * kWarps + warp) * kHeads + lane / kLanes;
  if (threadIdx.x == 0 && blockIdx.y == 0 && a.error_word != nullptr) {
    if (n == 0 && (live < 0 || live > a.N)) atomicOr(a.error_word, kErrTreeClamped);
    if (n < live && p < 0) atomicOr(a.error_word, kErrPosSkipped);
  }
  if (n >= live || p < 0) return;
  const __nv_bfloat16 *q_src = a.q_in + row * a.Hq * D + e0;
  const __nv_bfloat16 *k_src = a.k_new + row * a.Hkv * D + e0 - a.Hq * D;
  const __nv_bfloat16 *v_src = a.v_new + row * a.Hkv * D + e0 - rotated * D;
  uint4 raw[P], wq = {}, wk = {};
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int task = task0 + i * kStep;
    raw[i] = make_uint4(0u, 0u, 0u, 0u);
    if (task < heads)
      raw[i] = *reinterpret_cast<const uint4 *>(
          (task < a.Hq ? q_src : task < rotated ? k_src : v_src) + task * D);
  }
  const bool norm = a.q_norm_w != nullptr;
  if (norm) {
    wq = *reinterpret_cast<const uint4 *>(a.q_norm_w + e0);
    wk = *reinterpret_cast<const uint4 *>(a.k_norm_w + e0);
  }
  for (int i = threadIdx.x; i < D / 2; i += kThreads)
    rope_sincos_turns(p, turns.v[i], s_sin[i], s_cos[i]);
  __syncthreads();
  const bool first = hl < kLanes / 2;
  const size_t kv_at = ((size_t)b * a.Hkv * a.N + n) * D + e0;  // KV head 0 in the tree's buffers
  const int kv_step = a.N * D;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int task = task0 + i * kStep;
    if (task >= rotated && task < heads)
      *reinterpret_cast<uint4 *>(a.v_tree + kv_at + (size_t)(task - rotated) * kv_step) = raw[i];
    if (__all_sync(0xffffffffu, task >= rotated)) {
      if (!kMoreValues) return;
      continue;
    }
    const bool is_k = task >= a.Hq;
    auto unpack = [](uint4 v, float (&f)[8]) {
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        f[2 * j] = bf16_lo(w[j]);
        f[2 * j + 1] = bf16_hi(w[j]);
      }
    };
    float x[8], y[8];
    unpack(raw[i], x);
    float rstd = 1.f;
    if (norm) {
      float ss[kChains];
#pragma unroll
      for (int g = 0; g < kChains; ++g) {
        ss[g] = 0.f;
#pragma unroll
        for (int e = 0; e < kOld; ++e) ss[g] = fmaf(x[g * kOld + e], x[g * kOld + e], ss[g]);
      }
#pragma unroll
      for (int o = kLanes / 2; o > 0; o >>= 1)
#pragma unroll
        for (int g = 0; g < kChains; ++g) ss[g] += __shfl_xor_sync(0xffffffffu, ss[g], o);
#pragma unroll
      for (int o = kChains / 2; o > 0; o >>= 1)
#pragma unroll
        for (int g = 0; g < o; ++g) ss[g] += ss[g + o];
      rstd = rsqrtf(ss[0] * (1.0f / (float)D) + a.eps);
      float w[8];
      unpack(is_k ? wk : wq, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = x[e] * rstd * w[e];
    }
    unsigned cancels = 0;
    if (!a.interleaved) {
      const float4 *cp = reinterpret_cast<const float4 *>(s_cos) + (hl & (kLanes / 2 - 1)) * 2;
      const float4 *sp = reinterpret_cast<const float4 *>(s_sin) + (hl & (kLanes / 2 - 1)) * 2;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float4 c4 = cp[h], s4 = sp[h];
        const float cs[4] = {c4.x, c4.y, c4.z, c4.w}, sn[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int e = 4 * h + k;
          const float other = __shfl_xor_sync(0xffffffffu, x[e], kLanes / 2);
          y[e] = first ? rope_first(x[e], other, cs[k], sn[k])
                       : rope_second<false>(other, x[e], cs[k], sn[k]);
          if (is_k && rope_cancels(y[e], x[e], other)) cancels |= 1u << e;
        }
      }
    } else {
      const float4 c4 = reinterpret_cast<const float4 *>(s_cos)[hl];
      const float4 s4 = reinterpret_cast<const float4 *>(s_sin)[hl];
      const float cs[4] = {c4.x, c4.y, c4.z, c4.w}, sn[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        y[e] = rope_first(x[e], x[e + 1], cs[e / 2], sn[e / 2]);
        y[e + 1] = rope_second<D == 64>(x[e], x[e + 1], cs[e / 2], sn[e / 2]);
        if (is_k && rope_cancels(y[e], x[e], x[e + 1])) cancels |= 1u << e;
        if (is_k && rope_cancels(y[e + 1], x[e], x[e + 1])) cancels |= 2u << e;
      }
    }
    const uint4 out = make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]),
                                 pack_bf16x2(y[4], y[5]), pack_bf16x2(y[6], y[7]));
    if (task < a.Hq) {
      *reinterpret_cast<uint4 *>(a.q_out + (row * a.Hq + task) * D + e0) = out;
    } else if (task < rotated) {
      __nv_bfloat16 *dst = a.k_tree + kv_at + (size_t)(task - a.Hq) * kv_step;
      *reinterpret_cast<uint4 *>(dst) = out;
      if (cancels != 0)
        exact_elements(k_src - e0 + task * D, a.k_norm_w, dst - e0, turns.v, D / 2,
                       a.interleaved, e0, p, rstd, cancels);
    }
  }
}

struct TreeCommitArgs {
  const uint4 *k_tree, *v_tree;
  uint4 *k_cache, *v_cache;
  const int32_t *path, *n_path, *lens;
  uint32_t *error_word;
  int N, Hkv, T_cap;
};

// One CTA per (sequence, KV head): the path's rows of K and V, 16 bytes per thread, a thread's
// next kAtOnce rows of each loaded before the first is stored. Bound by latency: the
// count, the path's nodes and their rows follow one another. 256 sequences x 4 heads x 8 to 64
// rows of 128, 34 MB: 7.2 us; one row at a time 9.0, four 8.9.
constexpr int kAtOnce = 2;
template <int D>
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
  constexpr int kVec = D / 8;  // 16-byte words per row
  const int words = count * kVec;
  for (int first = threadIdx.x; first < words; first += kAtOnce * kThreads) {
    size_t dst[kAtOnce];
    uint4 k[kAtOnce], v[kAtOnce];
    bool good[kAtOnce];
    int node[kAtOnce];
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      const int i = first + u * kThreads;
      node[u] = i < words ? a.path[(size_t)b * a.N + i / kVec] : -1;
    }
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      const int i = first + u * kThreads, r = i / kVec, c = i - r * kVec;
      const long long slot = (long long)at + r;
      good[u] = node[u] >= 0 && node[u] < a.N && slot >= 0 && slot < a.T_cap;
      if (good[u]) {
        const size_t src = (pair * a.N + node[u]) * kVec + c;
        dst[u] = (pair * a.T_cap + slot) * kVec + c;
        k[u] = a.k_tree[src];
        v[u] = a.v_tree[src];
      } else if (i < words && g == 0 && c == 0 && a.error_word != nullptr) {
        atomicOr(a.error_word, kErrPosSkipped);
      }
    }
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u)
      if (good[u]) {
        a.k_cache[dst[u]] = k[u];
        a.v_cache[dst[u]] = v[u];
      }
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
  // Passes per warp: one while that leaves SMs without two CTAs, else as many as it takes (up
  // to 4) to hold a node's heads in one CTA.
  int sms = 152, dev = 0;
  if (cudaGetDevice(&dev) == cudaSuccess)
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  const int heads = Hq + 2 * Hkv, per = kWarps * (256 / D);
  int passes = 1;
  while (passes < 4 && per * passes < heads &&
         (long long)B * N * ((heads + per * passes - 1) / (per * passes)) > 2ll * sms)
    ++passes;
  const int blocks = (heads + per * passes - 1) / (per * passes);
  passes = (heads + per * blocks - 1) / (per * blocks);  // the same for each block
  const dim3 grid(N, blocks, B);
  const RopeTurns turns = make_rope_turns(D, inv);
  auto go = [&](auto kernel) {
    return launch_pdl(kernel, grid, kThreads, 0, stream, a, turns);
  };
  auto by_passes = [&](auto dim) {
    constexpr int kD = decltype(dim)::value;
    const bool more = Hkv > per;  // (a pass of the CTA is `per` heads)
    switch (passes) {
      case 1: return go(tree_rope_kernel<kD, 1, false>);
      case 2: return more ? go(tree_rope_kernel<kD, 2, true>) : go(tree_rope_kernel<kD, 2, false>);
      case 3: return more ? go(tree_rope_kernel<kD, 3, true>) : go(tree_rope_kernel<kD, 3, false>);
      default: return more ? go(tree_rope_kernel<kD, 4, true>) : go(tree_rope_kernel<kD, 4, false>);
    }
  };
  const cudaError_t e = D == 128 ? by_passes(std::integral_constant<int, 128>{})
                                 : by_passes(std::integral_constant<int, 64>{});
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_tree_commit(const void *k_tree, const void *v_tree, const int32_t *path,
                               const int32_t *n_path, void *k_cache, void *v_cache,
                               const int32_t *lens, int B, int N, int Hkv, int D, int T_cap,
                               uint32_t *error_word, cudaStream_t stream) {
  const TreeCommitArgs a{static_cast<const uint4 *>(k_tree), static_cast<const uint4 *>(v_tree),
                         static_cast<uint4 *>(k_cache), static_cast<uint4 *>(v_cache), path,
                         n_path, lens, error_word, N, Hkv, T_cap};
  const cudaError_t e = launch_pdl(D == 128 ? tree_commit_kernel<128> : tree_commit_kernel<64>,
                                   dim3(Hkv, B), kThreads, 0, stream, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace decattn
