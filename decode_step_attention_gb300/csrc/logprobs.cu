// Log probabilities of given tokens, the entropy of the distribution and its best
// alternatives, for every row of a batch of logits (the scoring side of the sampler's
// softmax, sampler.cu):
//
//   z = logits / T,  M = max z,  S = sum e^(z - M),  lse = M + ln S
//   logprob(id) = z_id - lse
//   entropy     = ln S - (sum e^(z - M) (z - M)) / S      (nats)
//   top K       : the K largest logits, equal ones by the lower id
//
// One read of the logits. Resident clusters of CTAs take the rows in turn, each CTA a slice.
// Three kinds of warps, each running on into the next row without the others: one copies the
// slices into a ring of shared memory (bulk copies); twelve take groups of four 16-byte vectors
// per thread, keeping the thread's largest logit with its id and both sums relative to it
// (moved only when a group exceeds it), and leave these in shared memory; four put a row
// together from them, across the cluster through distributed shared memory. (The last part is
// a long chain of short steps, which among streaming warps took 6000 cycles a row and held
// them all up.)
//
// The instructions per logit bound it, so the exponents' arguments and both sums run as
// packed pairs, and a logit of -inf (0 times -inf in the entropy's sum) is not guarded against
// but found by the group's sum being NaN, and that group done again.
//
// Alternatives without a sort of the row: a value and its id form one 64-bit key, all
// different. The K-th largest of the maxima of 32 groups of threads bounds the K-th largest key
// of the slice from below (for K = 8 about 9 keys of the threads' reach it), and only threads
// whose own maximum reaches it can hold a larger one. Those threads' vectors are read again
// (from L2), a warp each; what reaches the bound goes into a list of the warp's 32 largest, and
// a key's place among all the lists' is the number of larger ones. No more than 32 keys per
// warp come through whatever the order of the values.
#include <math.h>

#include <atomic>

#include "dec_device.cuh"
#include "dec_launch.h"

namespace decattn {
namespace {

using u64 = unsigned long long;
constexpr int kThreads = 384;    // that stream the logits
constexpr int kWarps = kThreads / 32;
constexpr int kPost = 128;       // that put rows together
constexpr int kPostWarps = kPost / 32;
constexpr int kEach = kThreads / kPost;  // streaming threads to a post thread
constexpr int kBlock = kThreads + 32 + kPost;
constexpr int kCtasPerSm = 2;
constexpr int kUnroll = 4;       // vectors a thread works on at a time
constexpr int kStageVecs = kThreads * kUnroll;
constexpr int kStages = 3;
constexpr size_t kSmem = (size_t)kStages * kStageVecs * 16;
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

// A barrier of the post warps.
__device__ __forceinline__ void post_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(kPost) : "memory");
}
// A key into a warp's list sorted downwards; the smallest falls off.
__device__ __forceinline__ u64 warp_insert(u64 list, u64 key) {
  const int lane = threadIdx.x & 31;
  const int at = __popc(__ballot_sync(kAll, list > key));
  const u64 up = __shfl_up_sync(kAll, list, 1);
  return lane < at ? list : lane == at ? key : up;
}
// How many of n keys in shared memory are larger than `key`.
__device__ __forceinline__ int larger(const u64 *keys, int n, u64 key) {
  int r = 0;
#pragma unroll 8
  for (int i = 0; i < n; ++i) r += keys[i] > key ? 1 : 0;
  return r;
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
  __device__ static bool any_nan(uint4 x) {
    float v[kN];
    unpack(x, v);
    bool nan = false;
#pragma unroll
    for (int i = 0; i < kN; ++i) nan |= isnan(v[i]);
    return nan;
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
__device__ __forceinline__ uint4 ld_shared(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr));
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

// The lanes' states as one, in every lane.
__device__ __forceinline__ void warp_join(State &st, float k) {
  float to = st.m;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) to = fmaxf(to, __shfl_xor_sync(kAll, to, o));
  st.raise(to, k);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    st.s += __shfl_xor_sync(kAll, st.s, o);
    st.c += __shfl_xor_sync(kAll, st.c, o);
  }
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
// Arrive on a barrier of any CTA of the cluster; what this thread knows of is then visible to
// who waits there.
__device__ __forceinline__ void arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar)
               : "memory");
}
__device__ __forceinline__ bool try_wait_cluster(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(bar), "r"(parity)
      : "memory");
  return done != 0;
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

// A row as [head elements][nvec aligned vectors][tail elements], and a CTA's vectors of it.
template <bool kBf16>
struct Row {
  const char *base;
  const uint4 *vec;
  int head, tail0, v0, v1;
  __device__ __forceinline__ Row(const LogprobArgs &a, size_t row, int rank, int C) {
    constexpr int kSize = kBf16 ? 2 : 4, E = 16 / kSize;
    base = static_cast<const char *>(a.logits) + row * (size_t)a.ld * kSize;
    const int off = (int)((16u - (unsigned)(reinterpret_cast<uintptr_t>(base) & 15u)) & 15u);
    head = min(a.V, off / kSize);
    const int nvec = (a.V - head) / E;
    tail0 = head + nvec * E;
    vec = reinterpret_cast<const uint4 *>(base + (size_t)head * kSize);
    v0 = (int)((unsigned)nvec * (unsigned)rank / (unsigned)C);  // nvec <= 2^16
    v1 = (int)((unsigned)nvec * (unsigned)(rank + 1) / (unsigned)C);
  }
};

// One of a row's alternatives. (In a row with NaN fewer than K keys may have been found: any
// id in range then.)
__device__ __forceinline__ void emit(const LogprobArgs &a, size_t row, int place, u64 key, float k,
                                     const float *out) {
  a.top_ids[row * a.K + place] = key == 0 ? place : key_id(key);
  a.top_logprobs[row * a.K + place] =
      (fmaf(key == 0 ? NAN : key_value(key), k, -out[0]) - out[1]) * kLn2;
}

// grid (C, clusters), cluster (C, 1): cluster y takes rows y, y + clusters, ...; its CTA r
// takes vectors [v0, v1) of the row, CTA 0 also the elements before the first aligned vector,
// the last CTA those behind the last. Streaming thread t has the slice's vectors t, t +
// kThreads, ...
template <bool kBf16>
__global__ void __launch_bounds__(kBlock, kCtasPerSm) logprobs_kernel(const LogprobArgs a,
                                                                      int rows) {
  using V = Vec<kBf16>;
  constexpr int E = V::kN;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ uint64_t s_bar[2 * kStages + 8];
  __shared__ float4 s_sums[2][kThreads];  // (m, s, c) of a row's streaming threads
  __shared__ u64 s_keys[2][kThreads];     // and their largest keys (0: nothing seen)
  __shared__ Slice s_slices[2];
  __shared__ State s_states[kPostWarps];
  __shared__ u64 s_group[32];             // the largest key of every 12 streaming threads
  __shared__ u64 s_cand[kMaxCluster * 32];
  __shared__ float s_out[2];
  __shared__ int s_count[2];              // owners and candidates
  __shared__ short s_owner[kThreads];
  __shared__ volatile int s_abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int C = gridDim.x, rank = blockIdx.x;
  const uint32_t ring = smem_addr(smem), bar_full = smem_addr(s_bar);
  const uint32_t bar_empty = bar_full + 8 * kStages;
  // a row's sums are left; they have been taken; CTA 0's: a row's slices are there; every
  // CTA's: its slice has been read
  const uint32_t bar_left = bar_empty + 8 * kStages, bar_taken = bar_left + 16;
  const uint32_t bar_ready = bar_taken + 16, bar_free = bar_ready + 16;
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(bar_full + 8 * i, 1);
      mbar_init(bar_empty + 8 * i, kWarps);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar_left + 8 * i, kWarps);
      mbar_init(bar_taken + 8 * i, kPostWarps);
      mbar_init(bar_ready + 8 * i, C);
      mbar_init(bar_free + 8 * i, 1);
    }
    s_abort = 0;
    s_count[0] = s_count[1] = 0;
    fence_barrier_init();
  }
  cluster_sync();  // (also of the CTA) every barrier is ready for the others
  pdl_launch_dependents();
  pdl_wait_prior_grid();
  const float k = 1.4426950408889634f / a.temperature;
  // A bounded wait; one that gave up makes this and the later rows NaN.
  auto await = [&](uint32_t bar, uint32_t parity) {
    if (try_wait_cluster(bar, parity)) return true;
    const unsigned long long t0 = global_ns();
    while (!try_wait_cluster(bar, parity)) {
      if (s_abort) return false;
      if (global_ns() - t0 > kWaitLimitNs) {
        s_abort = 1;
        return false;
      }
    }
    return true;
  };
  int turn = 0;

  if (warp == kWarps) {
    // ---------------------------------------------------------------- copies
    if (lane == 0) {
      int n = 0;
      for (size_t row = blockIdx.y; row < rows && !s_abort; row += gridDim.y) {
        const Row<kBf16> r(a, row, rank, C);
        for (int at = r.v0; at < r.v1; at += kStageVecs, ++n) {
          const int slot = n % kStages;
          if (n >= kStages && !await(bar_empty + 8 * slot, (n / kStages - 1) & 1)) break;
          const uint32_t bytes = (uint32_t)min(kStageVecs, r.v1 - at) * 16u;
          mbar_arrive_expect_tx(bar_full + 8 * slot, bytes);
          bulk_load(ring + slot * (kStageVecs * 16), r.vec + at, bytes, bar_full + 8 * slot);
        }
      }
      if (s_abort)  // no copy into this CTA's shared memory may outlive it
        for (int j = max(0, n - kStages); j < n; ++j)
          mbar_wait_bounded(bar_full + 8 * (j % kStages), (j / kStages) & 1);
    }
    __syncwarp();
  } else if (warp < kWarps) {
    // ---------------------------------------------------------------- stream
    int n = 0;
    for (size_t row = blockIdx.y; row < rows; row += gridDim.y, ++turn) {
      const Row<kBf16> r_(a, row, rank, C);
      const int head = r_.head, v0 = r_.v0, v1 = r_.v1, par = turn & 1;
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
      for (int at = v0; at < v1; at += kStageVecs, ++n) {
        const int slot = n % kStages, here = min(kStageVecs, v1 - at);
        if (!__all_sync(kAll, await(bar_full + 8 * slot, (n / kStages) & 1) ? 1 : 0)) {
          st.s = NAN;  // a copy that never came
          break;
        }
        const uint32_t src = ring + slot * (kStageVecs * 16) + tid * 16;
        const int first = head + (at + tid) * E;
        if (here == kStageVecs) {
          uint4 x[kUnroll];
#pragma unroll
          for (int u = 0; u < kUnroll; ++u) x[u] = ld_shared(src + u * (kThreads * 16));
          group(x, first, kThreads * E);
        } else {
          for (int u = 0; tid + u * kThreads < here; ++u) {
            uint4 y[1] = {ld_shared(src + u * (kThreads * 16))};
            group(y, first + u * kThreads * E, 0);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_empty + 8 * slot);
      }
      if (turn >= 2) __all_sync(kAll, await(bar_taken + 8 * par, ((turn >> 1) + 1) & 1) ? 1 : 0);
      s_sums[par][tid] = make_float4(st.m, st.s, st.c, 0.f);
      s_keys[par][tid] = best_id < 0 ? 0ull : rank_key(st.m, best_id);
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_left + 8 * par);
    }
  } else {
    // ---------------------------------------------------------------- put rows together
    const int p = tid - kThreads - 32, pw = p >> 5;
    for (size_t row = blockIdx.y; row < rows; row += gridDim.y, ++turn) {
      const int par = turn & 1, phase = (turn >> 1) & 1;
      const int leader = turn % C;  // the CTA that puts this row together
      Slice &s_slice = s_slices[par];
      const Row<kBf16> r(a, row, rank, C);
      // a given id's logit and one element of each of the row's ends, while the row streams
      float given = -INFINITY;
      if (rank == leader && p < a.C) {
        const int id = a.ids[row * a.C + p];
        if (id >= 0 && id < a.V) given = V::one(r.base, id);
      }
      State st{-INFINITY, 0.f, 0.f};
      u64 ends[2] = {};
      auto single = [&](int id) {
        const float v = V::one(r.base, id);
        if (v > st.m) st.raise(v, k);
        const float x = st.m == -INFINITY ? 0.f : __fmul_rn(st.m, k);
        const float d = max_nan(fmaf(v, k, -x), -400.f), e = ex2(d);
        st.s += e;
        st.c = fmaf(e, d, st.c);
        return rank_key(v, id);
      };
      if (rank == 0 && p < r.head) ends[0] = single(p);
      if (rank == C - 1 && r.tail0 + p < a.V) ends[1] = single(r.tail0 + p);

      const bool left = await(bar_left + 8 * par, phase);
      u64 mine[kEach], most = umax(ends[0], ends[1]);
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        const float4 x = s_sums[par][p * kEach + i];
        mine[i] = s_keys[par][p * kEach + i];
        most = umax(most, mine[i]);
        st.join(State{x.x, x.y, x.z}, k);
      }
      if (!left) st.s = NAN;
#pragma unroll
      for (int o = 2; o > 0; o >>= 1) most = umax(most, __shfl_xor_sync(kAll, most, o));
      if ((lane & 3) == 0) s_group[p >> 2] = most;
      warp_join(st, k);
      if (lane == 0) s_states[pw] = st;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_taken + 8 * par);
      if (C > 1 && turn >= 2) await(bar_free + 8 * par, phase ^ 1);
      post_sync();
      auto finish = [&](const State &q) {  // one thread: the row's numbers
        const float log2_s = isinf(q.m) || s_abort ? NAN : log2f(q.s);
        s_out[0] = __fmul_rn(q.m, k);
        s_out[1] = log2_s;
        if (a.entropy != nullptr) a.entropy[row] = (log2_s - q.c / q.s) * kLn2;
      };
      if (p < 32) {
        State q{-INFINITY, 0.f, 0.f};
        if (lane < kPostWarps) q = s_states[lane];
        warp_join(q, k);
        if (lane == 0) {
          if (C == 1) finish(q);
          else s_slice.st = q;
        }
        __syncwarp();
      }
      int place = -1;  // this thread's key's place among the row's (or the slice's) best
      u64 key = 0;
      if (a.K > 0) {
        // the K-th largest of the 32, in every warp
        const u64 g = s_group[lane];
        const unsigned at = __ballot_sync(kAll, larger(s_group, 32, g) == a.K - 1 && g > 0);
        const u64 bound = at != 0 ? __shfl_sync(kAll, g, __ffs(at) - 1) : 1ull;  // 1: fewer
        if (a.K == 1) {
          if (p == 0) place = 0, key = bound > 1 ? bound : 0;
        } else {
#pragma unroll
          for (int i = 0; i < kEach; ++i)
            if (mine[i] >= bound) s_owner[atomicAdd(&s_count[0], 1)] = (short)(p * kEach + i);
          post_sync();
          const int owners = s_count[0];
          u64 list = 0;
          auto offer = [&](u64 key) {
            unsigned todo = __ballot_sync(kAll, key >= bound);
            while (todo) {
              const int from = __ffs(todo) - 1;
              todo &= todo - 1;
              list = warp_insert(list, __shfl_sync(kAll, key, from));
            }
          };
          offer(ends[0]);
          offer(ends[1]);
          // Items of 32 of an owner's vectors, four at a time so that their loads overlap. Most
          // hold nothing: one comparison of the largest value tells.
          const int chunks = (r.v1 - r.v0 + 32 * kThreads - 1) / (32 * kThreads);
          const float least = bound > 1 ? key_value(bound) : -INFINITY;
          for (int i0 = pw; i0 < owners * chunks; i0 += 4 * kPostWarps) {
            uint4 x[4];
            int j[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const int i = i0 + q * kPostWarps, o = i / chunks;
              j[q] = r.v1;
              if (i < owners * chunks)
                j[q] = r.v0 + s_owner[o] + ((i - o * chunks) * 32 + lane) * kThreads;
              if (j[q] < r.v1) x[q] = ld_stream(r.vec + j[q]);
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const uint4 one[1] = {x[q]};
              const bool in = j[q] < r.v1;
              // (not `<`: a NaN may be the largest key)
              if (!__any_sync(kAll, in && (!(V::template largest<1>(one) < least) || V::any_nan(x[q]))))
                continue;
              float v[E];
              V::unpack(x[q], v);
#pragma unroll
              for (int e = 0; e < E; ++e)
                offer(in ? rank_key(v[e], r.head + j[q] * E + e) : 0ull);
            }
          }
          const int found = min(a.K, __popc(__ballot_sync(kAll, list > 0)));
          int base_at = 0;
          if (lane == 0 && found > 0) base_at = atomicAdd(&s_count[1], found);
          base_at = __shfl_sync(kAll, base_at, 0);
          if (lane < found) s_cand[base_at + lane] = list;
          post_sync();
          const int cands = s_count[1];  // at most kPostWarps x 32 = kPost
          key = p < cands ? s_cand[p] : 0;
          place = p < cands ? larger(s_cand, cands, key) : p;  // (behind them: nothing there)
          if (place >= a.K) place = -1;
        }
      }
      if (C > 1) {
        // ---- the row, in CTA 0, from the CTAs' slices
        if (place >= 0) s_slice.list[place] = key;
        post_sync();
        if (p == 0) {
          s_count[0] = s_count[1] = 0;
          arrive_cluster(cluster_map(bar_ready + 8 * par, leader));
        }
        if (rank != leader) continue;
        // (C is even: a CTA always leads with the same `par`, every C-th row)
        await(bar_ready + 8 * par, (turn / C) & 1);
        const uint32_t here = smem_addr(&s_slice);
        if (p < 32) {
          State q{-INFINITY, 0.f, 0.f};
          if (lane < C) {
            const uint32_t at = cluster_map(here, lane);
            q.m = ld_cluster_f32(at);
            q.s = ld_cluster_f32(at + 4);
            q.c = ld_cluster_f32(at + 8);
          }
          warp_join(q, k);
          if (lane == 0) finish(q);
        }
        // Only keys that reach the largest of the slices' K-th ones can be among the K best (and
        // K of them do): these alone are ranked.
        u64 floor_key = 0;
        if (a.K > 0 && lane < C)
          floor_key = ld_cluster_u64(
              cluster_map(here + (uint32_t)offsetof(Slice, list), lane) + 8 * (a.K - 1));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
          floor_key = umax(floor_key, __shfl_xor_sync(kAll, floor_key, o));
        for (int i = p; i < C * a.K; i += kPost) {
          const u64 c = ld_cluster_u64(
              cluster_map(here + (uint32_t)offsetof(Slice, list), i / a.K) + 8 * (i % a.K));
          if (c > 0 && c >= floor_key) s_cand[atomicAdd(&s_count[1], 1)] = c;
        }
        post_sync();
        if (p < C) arrive_cluster(cluster_map(bar_free + 8 * par, p));
        place = -1;
        const int cands = s_count[1];  // at most 16 x 32
        for (int i = p; i < max(cands, a.K); i += kPost) {
          const u64 c = i < cands ? s_cand[i] : 0;
          const int at = i < cands ? larger(s_cand, cands, c) : i;  // (past them: a row with NaN)
          if (at < a.K) emit(a, row, at, c, k, s_out);
        }
        post_sync();
        if (p == 0) s_count[1] = 0;
      } else {
        post_sync();
        if (p == 0) s_count[0] = s_count[1] = 0;
      }
      if (place >= 0) emit(a, row, place, key, k, s_out);
      auto logprob = [&](float v) { return (fmaf(v, k, -s_out[0]) - s_out[1]) * kLn2; };
      if (p < a.C) a.logprobs[row * a.C + p] = logprob(given);
      for (int i = p + kPost; i < a.C; i += kPost) {
        const int id = a.ids[row * a.C + i];
        a.logprobs[row * a.C + i] =
            logprob(id >= 0 && id < a.V ? V::one(r.base, id) : -INFINITY);
      }
    }
  }
  cluster_sync();  // no CTA leaves while another may still reach its shared memory
}

// Clusters of c CTAs resident at once (cached per device).
template <bool kBf16>
int resident(int dev, int sms, int c) {
  static std::atomic<int> cache[64][kMaxCluster + 1];
  if (dev < 64) {
    const int n = cache[dev][c].load(std::memory_order_relaxed);
    if (n > 0) return n;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(c, 1);
  cfg.blockDim = dim3(kBlock);
  cfg.dynamicSmemBytes = kSmem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)c;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, logprobs_kernel<kBf16>, &cfg) != cudaSuccess) {
    (void)cudaGetLastError();
    n = 0;
  }
  if (n <= 0) n = c == 1 ? sms * kCtasPerSm : 0;
  if (dev < 64) cache[dev][c].store(n, std::memory_order_relaxed);
  return n;
}

// CTAs per row: the number that gets through the rows soonest, by rounds of resident clusters
// times a round's time. A slice costs 0.72 ns per vector (a CTA's share of HBM) and a fixed
// part, more of it across a cluster.
template <bool kBf16>
int row_ctas(int B, int V, int dev, int sms) {
  const double nvec = V / (kBf16 ? 8 : 4);
  int best = 1;
  double best_ns = 1e300;
  for (int c = 1; c <= kMaxCluster; c *= 2) {
    const int n = resident<kBf16>(dev, sms, c);
    if (n <= 0) continue;
    const double ns = ((B + n - 1) / n) * (nvec / c * 0.72 + (c > 1 ? 4000.0 : 2500.0));
    if (ns < best_ns) best_ns = ns, best = c;
  }
  return best;
}

template <bool kBf16>
cudaError_t launch(const LogprobArgs &a, int B, cudaStream_t stream) {
  static std::atomic<bool> ready[64];
  static std::atomic<int> sm_count[64];
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !ready[dev].load(std::memory_order_acquire)) {
    if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess ||
        (e = cudaFuncSetAttribute(logprobs_kernel<kBf16>,
                                  cudaFuncAttributeNonPortableClusterSizeAllowed, 1)) !=
            cudaSuccess ||
        (e = cudaFuncSetAttribute(logprobs_kernel<kBf16>,
                                  cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem)) !=
            cudaSuccess)
      return e;
    if (dev < 64) {
      sm_count[dev].store(sms, std::memory_order_relaxed);
      ready[dev].store(true, std::memory_order_release);
    }
  } else {
    sms = sm_count[dev].load(std::memory_order_relaxed);
  }
  const int c = row_ctas<kBf16>(B, a.V, dev, sms);
  const int n = resident<kBf16>(dev, sms, c);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(c, B < n ? B : n);
  cfg.blockDim = dim3(kBlock);
  cfg.dynamicSmemBytes = kSmem;
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
  if ((e = cudaLaunchKernelEx(&cfg, logprobs_kernel<kBf16>, a, B)) != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_logprobs(const LogprobArgs &a, int B, cudaStream_t stream) {
  return a.bf16 ? launch<true>(a, B, stream) : launch<false>(a, B, stream);
}

}  // namespace decattn
