// Log probabilities of given tokens, the entropy of the distribution and its best
// alternatives, for every row of a batch of logits (the scoring side of the sampler's
// softmax, sampler.cu):
//
//   z = logits / T,  M = max z,  S = sum e^(z - M),  lse = M + ln S
//   logprob(id) = z_id - lse
//   entropy     = ln S - (sum e^(z - M) (z - M)) / S      (nats)
//   top K       : the K largest logits, equal ones by the lower id
//
// One read of the logits. A row is cut over a cluster of CTAs; every thread streams groups of
// four 16-byte vectors (the next group in flight while it works on the last), keeping its
// largest logit with its id and both sums relative to it, moved only when a group exceeds
// it. The threads' sums meet in shared memory, the CTAs' in distributed shared memory.
//
// The instructions per logit bound it, so the exponents' arguments and both sums run as
// packed pairs, and a logit of -inf (0 times -inf in the entropy's sum) is not guarded against
// but found by the group's sum being NaN, and that group done again.
//
// Alternatives without a sort of the row: a value and its id form one 64-bit key, all
// different. The K-th largest of the threads' own maxima bounds the K-th largest key of the
// slice from below, and only the K threads whose maximum reaches it can hold a larger one. So
// K threads' vectors are read again (from L2), a warp each, into a list of the 32 largest
// keys held across its lanes; the lists are merged pairwise, then the CTAs' lists. The cost
// does not depend on the order of the values.
#include <math.h>

#include <atomic>

#include "dec_device.cuh"
#include "dec_launch.h"

namespace decattn {
namespace {

using u64 = unsigned long long;
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kCtasPerSm = 4;
constexpr int kUnroll = 4;       // vectors a thread works on at a time
constexpr int kMaxCluster = 16;
constexpr unsigned kAll = 0xffffffffu;
constexpr float kLn2 = 0.6931471805599453f;

// Orders by value, then by the lower id: larger is better. NaN orders by its bits.
__device__ __forceinline__ u64 rank_key(float v, int id) {
  unsigned u = __float_as_uint(v + 0.f);  // -0 and 0 are equal values
  u = (u & 0x80000000u) ? ~u : u | 0x80000000u;
  return ((u64)u << 32) | (unsigned)~id;
}
__device__ __forceinline__ int key_id(u64 k) { return (int)~(unsigned)k; }
__device__ __forceinline__ float key_value(u64 k) {
  const unsigned u = (unsigned)(k >> 32);
  return __uint_as_float((u & 0x80000000u) ? u ^ 0x80000000u : ~u);
}

__device__ __forceinline__ u64 umax(u64 a, u64 b) { return a > b ? a : b; }
__device__ __forceinline__ u64 umin(u64 a, u64 b) { return a < b ? a : b; }

// One key per lane, sorted downwards (bitonic).
__device__ __forceinline__ u64 warp_sort(u64 k) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
    for (int step = size >> 1; step > 0; step >>= 1) {
      const u64 o = __shfl_xor_sync(kAll, k, step);
      const bool first = (lane & step) == 0, down = (lane & size) == 0 || size == 32;
      k = first == down ? umax(k, o) : umin(k, o);
    }
  return k;
}
// The 32 largest of two lists sorted downwards; `b` is lane 31 - i's of the second.
__device__ __forceinline__ u64 warp_merge(u64 a, u64 b) {
  const int lane = threadIdx.x & 31;
  u64 k = umax(a, b);
#pragma unroll
  for (int step = 16; step > 0; step >>= 1) {
    const u64 o = __shfl_xor_sync(kAll, k, step);
    k = (lane & step) == 0 ? umax(k, o) : umin(k, o);
  }
  return k;
}
// A key into a list sorted downwards; the smallest falls off.
__device__ __forceinline__ u64 warp_insert(u64 list, u64 key) {
  const int lane = threadIdx.x & 31;
  const int at = __popc(__ballot_sync(kAll, list > key));
  const u64 up = __shfl_up_sync(kAll, list, 1);
  return lane < at ? list : lane == at ? key : up;
}
// The 32 largest of every warp's list, in warp 0 (all warps call; the others get what
// their part of the tree left). s: kWarps x 32.
__device__ __forceinline__ u64 block_merge(u64 list, u64 (*s)[32]) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int half = kWarps / 2; half > 0; half >>= 1) {
    if (warp >= half && warp < 2 * half) s[warp][lane] = list;
    __syncthreads();
    if (warp < half) list = warp_merge(list, s[warp + half][31 - lane]);
  }
  return list;
}

template <bool kBf16>
struct Vec {
  static constexpr int kN = kBf16 ? 8 : 4;
  // the largest of n vectors' values (a NaN is passed over)
  template <int n>
  __device__ static float largest(const uint4 (&x)[n]) {
    if constexpr (kBf16) {
      __nv_bfloat162 m[4];
#pragma unroll
      for (int u = 0; u < n; ++u) {
        const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const __nv_bfloat162 b = *reinterpret_cast<const __nv_bfloat162 *>(&w[i]);
          m[i] = u == 0 ? b : __hmax2(m[i], b);
        }
      }
      const __nv_bfloat162 a = __hmax2(__hmax2(m[0], m[1]), __hmax2(m[2], m[3]));
      return fmaxf(__low2float(a), __high2float(a));
    } else {
      float m[4];
#pragma unroll
      for (int u = 0; u < n; ++u) {
        const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
          m[i] = u == 0 ? __uint_as_float(w[i]) : fmaxf(m[i], __uint_as_float(w[i]));
      }
      return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
    }
  }
  __device__ static void unpack(uint4 x, float (&v)[kN]) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (kBf16) {
        v[2 * i] = bf16_lo(w[i]);
        v[2 * i + 1] = bf16_hi(w[i]);
      } else {
        v[i] = __uint_as_float(w[i]);
      }
    }
  }
  __device__ static float one(const void *row, int i) {
    return kBf16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(row)[i])
                 : static_cast<const float *>(row)[i];
  }
};

__device__ __forceinline__ uint4 ld_stream(const uint4 *p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max_nan(float a, float b) {  // NaN if either is
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}

// A running softmax state: the maximum logit m and, relative to the exponent r = m k with k =
// log2(e) / T, s = sum 2^(k v - r) and c = sum 2^(k v - r) (k v - r). (r is one rounded number
// that every exponent is taken against, in one rounding: never contracted.) Nothing seen: m = -inf.
struct State {
  float m, s, c;
  // the factors that move sums from this maximum to a larger one
  __device__ __forceinline__ void raise(float to, float k) {
    if (m != -INFINITY) {
      const float d = __fmul_rn(m, k) - __fmul_rn(to, k), f = ex2(d);
      c = f > 0.f ? f * fmaf(d, s, c) : 0.f * c;  // keeps a NaN
      s *= f;
    }
    m = to;
  }
  __device__ __forceinline__ void join(State o, float k) {
    const float to = fmaxf(m, o.m);
    raise(to, k);
    o.raise(to, k);
    s += o.s;
    c += o.c;
  }
};

// Two fp32 operations per instruction.
__device__ __forceinline__ u64 pair_of(float a, float b) {
  u64 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpair(u64 v, float &a, float &b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ u64 fma2(u64 a, u64 b, u64 c) {
  u64 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ u64 add2(u64 a, u64 b) {
  u64 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

struct Slice {  // what a CTA keeps for the others of its cluster
  State st;
  u64 list[32];
};

__device__ __forceinline__ uint32_t cluster_map(uint32_t saddr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\t"
               "barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ u64 ld_cluster_u64(uint32_t addr) {
  u64 v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

// grid (C, B), cluster (C, 1): CTA r of row b takes vectors [v0, v1) of the row; CTA 0 also
// the elements before the first aligned vector, the last CTA those behind the last.
template <bool kBf16>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) logprobs_kernel(const LogprobArgs a) {
  using V = Vec<kBf16>;
  constexpr int E = V::kN;
  __shared__ u64 s_list[kWarps][32];
  __shared__ Slice s_slice;
  __shared__ State s_state[kWarps];
  __shared__ float s_out[2];
  pdl_launch_dependents();
  pdl_wait_prior_grid();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int C = gridDim.x, rank = blockIdx.x;
  const size_t row = blockIdx.y;
  const char *base = static_cast<const char *>(a.logits) + row * (size_t)a.ld * (kBf16 ? 2 : 4);
  const float k = 1.4426950408889634f / a.temperature;
  // the row as [head elements][nvec vectors][tail elements]
  const int off = (int)((16u - (unsigned)(reinterpret_cast<uintptr_t>(base) & 15u)) & 15u);
  const int head = min(a.V, off / (kBf16 ? 2 : 4));
  const int nvec = (a.V - head) / E, tail0 = head + nvec * E;
  const uint4 *vec = reinterpret_cast<const uint4 *>(base + (size_t)head * (kBf16 ? 2 : 4));
  const int v0 = (int)((long long)nvec * rank / C), v1 = (int)((long long)nvec * (rank + 1) / C);

  // the given ids' logits, on their way while the row streams
  const bool has_id = rank == 0 && tid < a.C;
  float id_value = -INFINITY;
  if (has_id) {
    const int id = a.ids[row * a.C + tid];
    if (id >= 0 && id < a.V) id_value = V::one(base, id);
  }

  State st{-INFINITY, 0.f, 0.f};  // st.m is also this thread's largest logit
  int best_id = -1;               // and this its id; -1: nothing seen yet
  // n vectors' worth of logits, the first element of vector u being first + u * stride
  auto group = [&](auto &x, int first, int stride) {
    constexpr int n = sizeof(x) / sizeof(uint4);
    const float mx = V::template largest<n>(x);
    if (mx > st.m || best_id < 0) {  // strictly: of equal values the lower id stays
      st.raise(mx, k);
      bool found = false;
#pragma unroll
      for (int u = n - 1; u >= 0; --u) {
        float v[E];
        V::unpack(x[u], v);
#pragma unroll
        for (int i = E - 1; i >= 0; --i)
          if (v[i] == mx || !found) best_id = first + u * stride + i, found = true;
      }
    }
    const float r = st.m == -INFINITY ? 0.f : __fmul_rn(st.m, k);
    const u64 k2 = pair_of(k, k), r2 = pair_of(-r, -r);
    u64 s2[2] = {}, c2[2] = {};
#pragma unroll
    for (int u = 0; u < n; ++u) {
      float v[E];
      V::unpack(x[u], v);
#pragma unroll
      for (int i = 0; i < E; i += 2) {
        const u64 d = fma2(pair_of(v[i], v[i + 1]), k2, r2);
        float d0, d1;
        unpair(d, d0, d1);
        const u64 e = pair_of(ex2(d0), ex2(d1));
        s2[(i / 2) & 1] = add2(s2[(i / 2) & 1], e);
        c2[(i / 2) & 1] = fma2(e, d, c2[(i / 2) & 1]);
      }
    }
    float s0, s1, c0, c1;
    unpair(add2(s2[0], s2[1]), s0, s1);
    unpair(add2(c2[0], c2[1]), c0, c1);
    float c = c0 + c1;
    if (isnan(c)) {
      // -inf has weight 0 and adds nothing (a real NaN comes out again)
      c = 0.f;
#pragma unroll
      for (int u = 0; u < n; ++u) {
        float v[E];
        V::unpack(x[u], v);
#pragma unroll
        for (int i = 0; i < E; ++i) {
          const float d = max_nan(fmaf(v[i], k, -r), -400.f);
          c = fmaf(ex2(d), d, c);
        }
      }
    }
    st.s += s0 + s1;
    st.c += c;
  };
  // single elements (a row's ends) as a vector of one and -infs
  auto single = [&](int id) {
    const float v = V::one(base, id);
    uint4 x[1];
    if constexpr (kBf16)
      x[0] = make_uint4(0xff800000u | (__float_as_uint(v) >> 16), 0xff80ff80u, 0xff80ff80u,
                        0xff80ff80u);
    else
      x[0] = make_uint4(__float_as_uint(v), 0xff800000u, 0xff800000u, 0xff800000u);
    group(x, id, 0);
  };
  if (rank == 0 && tid < head) single(tid);
  {
    constexpr int kStep = kUnroll * kThreads;
    const int full = (v1 - v0) / kStep;  // groups that every thread has whole
    const uint4 *p = vec + v0 + tid;
    uint4 x[kUnroll], next[kUnroll];
    if (full > 0) {
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) next[u] = ld_stream(p + u * kThreads);
    }
    int first = head + (v0 + tid) * E;
    for (int i = 0; i < full; ++i) {
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) x[u] = next[u];
      p += kStep;
      if (i + 1 < full) {
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) next[u] = ld_stream(p + u * kThreads);
      }
      group(x, first, kThreads * E);
      first += kStep * E;
    }
    for (int at = v0 + full * kStep + tid; at < v1; at += kThreads) {
      uint4 y[1] = {ld_stream(vec + at)};
      group(y, head + at * E, 0);
    }
  }
  if (rank == C - 1 && tail0 + tid < a.V) single(tail0 + tid);

  const float st_max = st.m;
  // ---- the slice's sums
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    State x;
    x.m = __shfl_xor_sync(kAll, st.m, o);
    x.s = __shfl_xor_sync(kAll, st.s, o);
    x.c = __shfl_xor_sync(kAll, st.c, o);
    st.join(x, k);
  }
  if (lane == 0) s_state[warp] = st;

  // ---- the slice's 32 best
  if (a.K > 0) {
    const u64 mine = best_id < 0 ? 0ull : rank_key(st_max, best_id);
    u64 list = block_merge(warp_sort(mine), s_list);
    if (a.K > 1) {
      if (warp == 0) s_slice.list[lane] = list;
      __syncthreads();
      const u64 bar = s_slice.list[a.K - 1];  // 0: fewer than K threads hold anything
      list = 0;
      for (int i = warp; i < a.K; i += kWarps) {
        const u64 top = s_slice.list[i];
        if (top == 0) break;
        const int id = key_id(top);
        // its owner's elements: one of the head or tail, and every kThreads-th vector
        const int owner = id < head ? id : id >= tail0 ? id - tail0 : ((id - head) / E - v0) % kThreads;
        auto offer = [&](u64 key) {
          unsigned todo = __ballot_sync(kAll, key >= bar && key > 0);
          while (todo) {
            const int from = __ffs(todo) - 1;
            todo &= todo - 1;
            list = warp_insert(list, __shfl_sync(kAll, key, from));
          }
        };
        for (int j0 = v0 + owner; j0 < v1; j0 += 32 * kThreads) {
          const int j = j0 + lane * kThreads;
          uint4 x = make_uint4(0u, 0u, 0u, 0u);
          if (j < v1) x = ld_stream(vec + j);
          float v[E];
          V::unpack(x, v);
#pragma unroll
          for (int e = 0; e < E; ++e) offer(j < v1 ? rank_key(v[e], head + j * E + e) : 0ull);
        }
        u64 extra = 0;
        if (lane == 0 && rank == 0 && owner < head) extra = rank_key(V::one(base, owner), owner);
        if (lane == 1 && rank == C - 1 && tail0 + owner < a.V)
          extra = rank_key(V::one(base, tail0 + owner), tail0 + owner);
        offer(extra);
      }
      __syncthreads();  // the bound has been read by all
      list = block_merge(list, s_list);
    }
    if (warp == 0) s_slice.list[lane] = list;
  } else {
    __syncthreads();
  }
  if (tid == 0) {
    State t = s_state[0];
    for (int w = 1; w < kWarps; ++w) t.join(s_state[w], k);
    s_slice.st = t;
  }
  // ---- the row, in CTA 0
  cluster_sync();
  if (rank == 0) {
    const uint32_t here = smem_addr(&s_slice);
    if (warp == 0) {
      State t{-INFINITY, 0.f, 0.f};
      if (lane < C) {
        const uint32_t p = cluster_map(here, lane);
        t.m = ld_cluster_f32(p);
        t.s = ld_cluster_f32(p + 4);
        t.c = ld_cluster_f32(p + 8);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        State x;
        x.m = __shfl_xor_sync(kAll, t.m, o);
        x.s = __shfl_xor_sync(kAll, t.s, o);
        x.c = __shfl_xor_sync(kAll, t.c, o);
        t.join(x, k);
      }
      if (lane == 0) {
        const float log2_s = isinf(t.m) ? NAN : log2f(t.s);
        s_out[0] = __fmul_rn(t.m, k);
        s_out[1] = log2_s;
        if (a.entropy != nullptr) a.entropy[row] = (log2_s - t.c / t.s) * kLn2;
      }
    }
    u64 list = 0;
    if (a.K > 0) {
      for (int r = warp; r < C; r += kWarps) {
        const uint32_t p = cluster_map(here + (uint32_t)offsetof(Slice, list), r);
        list = warp_merge(list, ld_cluster_u64(p + 8 * (31 - lane)));
      }
    }
    __syncthreads();
    const float r = s_out[0], log2_s = s_out[1];
    auto logprob = [&](float v) { return (fmaf(v, k, -r) - log2_s) * kLn2; };
    if (has_id) a.logprobs[row * a.C + tid] = logprob(id_value);
    for (int i = tid + kThreads; i < a.C; i += kThreads) {
      const int id = a.ids[row * a.C + i];
      const float v = id >= 0 && id < a.V ? V::one(base, id) : -INFINITY;
      a.logprobs[row * a.C + i] = logprob(v);
    }
    if (a.K > 0) {
      list = block_merge(list, s_list);
      if (warp == 0 && lane < a.K) {
        // in a row with NaN fewer than K keys may have been found: any id in range then
        a.top_ids[row * a.K + lane] = list == 0 ? lane : key_id(list);
        a.top_logprobs[row * a.K + lane] = logprob(key_value(list));
      }
    }
  }
  if (C > 1) cluster_sync();  // no CTA leaves while another still reads its shared memory
}

// CTAs per row: the fewest that give every SM its CTAs and a few waves to even out, as long
// as each thread keeps at least two vectors.
int row_ctas(int B, int V, bool bf16, int sms) {
  const long long nvec = V / (bf16 ? 8 : 4);
  int c = 1;
  while (c < kMaxCluster && (long long)B * c < 2ll * kCtasPerSm * sms &&
         nvec >= 2ll * kThreads * (2 * c))
    c *= 2;
  return c;
}

template <bool kBf16>
cudaError_t launch(const LogprobArgs &a, int B, cudaStream_t stream) {
  static std::atomic<bool> ready[64];
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess)
    return e;
  if (dev >= 64 || !ready[dev].load(std::memory_order_relaxed)) {
    e = cudaFuncSetAttribute(logprobs_kernel<kBf16>,
                             cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    if (dev < 64) ready[dev].store(true, std::memory_order_relaxed);
  }
  const int c = row_ctas(B, a.V, kBf16, sms);
  constexpr int kMaxGridY = 65535;
  for (int b0 = 0; b0 < B; b0 += kMaxGridY) {
    LogprobArgs x = a;
    x.logits = static_cast<const char *>(a.logits) + (size_t)b0 * a.ld * (kBf16 ? 2 : 4);
    if (a.C > 0) {
      x.ids += (size_t)b0 * a.C;
      x.logprobs += (size_t)b0 * a.C;
    }
    if (a.entropy != nullptr) x.entropy += b0;
    if (a.K > 0) {
      x.top_ids += (size_t)b0 * a.K;
      x.top_logprobs += (size_t)b0 * a.K;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(c, B - b0 < kMaxGridY ? B - b0 : kMaxGridY);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)c;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    if ((e = cudaLaunchKernelEx(&cfg, logprobs_kernel<kBf16>, x)) != cudaSuccess) return e;
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_logprobs(const LogprobArgs &a, int B, cudaStream_t stream) {
  return a.bf16 ? launch<true>(a, B, stream) : launch<false>(a, B, stream);
}

}  // namespace decattn
