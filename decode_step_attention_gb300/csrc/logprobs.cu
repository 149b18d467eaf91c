// Log probabilities of given tokens, the entropy of the distribution and its best
// alternatives, for every row of a batch of logits (the scoring side of the sampler's
// softmax, sampler.cu):
//
//   z = logits / T,  M = max z,  S = sum e^(z - M),  lse = M + ln S
//   logprob(id) = z_id - lse
//   entropy     = ln S - (sum e^(z - M) (z - M)) / S      (nats)
//   top K       : the K largest logits, equal ones by the lower id
//
// One read of the logits, each thread keeping its largest logit with its id and both sums
// relative to it, moved only when a group of vectors exceeds it. Two kernels:
//   many rows   a CTA takes whole rows in turn (two CTAs per SM). Three kinds of warps, each
//               running on into the next row without the others: one copies rows into a ring of
//               shared memory (bulk copies, up to 144 KB in flight per SM); twelve stream groups
//               of four 16-byte vectors per thread and leave their results in shared memory;
//               four put a row together from them. (That last part is a long chain of short
//               steps; among streaming warps it took 6000 cycles a row and held them all up.)
//               512 rows of 131072 fp32 logits: 50 us, 5.3 TB/s; 2047 rows of 50257 bf16: 48 us.
//   few rows    a row over a cluster of up to 16 CTAs, the slices' results joined through
//               distributed shared memory. One row of 151936 fp32 logits: 8 us.
//
// The instructions per logit bound the streaming, so the exponents' arguments and both sums run
// as packed pairs, and a logit of -inf (0 times -inf in the entropy's sum) is not guarded
// against but found by the group's sum being NaN, and that group done again.
//
// Alternatives without a sort of the row: a value and its id form one 64-bit key, all
// different. The K-th largest of the maxima of 32 or 128 groups of threads bounds the K-th
// largest key of the row from below (K = 8: about 9 of a CTA's threads reach it), and only
// threads whose own maximum reaches it can hold a larger one. Those threads' vectors are read
// again (from L2), a warp each; what reaches the bound goes into a list of the warp's 32
// largest, and a key's place is the number of larger ones among all the lists'. No more than
// 32 keys per warp come through whatever the order of the values.
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
__device__ __forceinline__ float max_nan(float a, float b) {  // NaN if either is
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}

// The exponent that a maximum's logits are taken against: m k with k = log2(e) / T, or -2^24 where
// that is less. A part of a row masked with -1e30 or the type's lowest value then has sums of 0 (its
// own m k may be -inf, and the rounding of m k alone would move exponents by thousands).
constexpr float kLowest = -0x1p24f;
__device__ __forceinline__ float base_of(float m, float k) { return fmaxf(__fmul_rn(m, k), kLowest); }

// A running softmax state: the base r of the largest logit and, relative to it, s = sum 2^(k v - r)
// and c = sum 2^(k v - r) (k v - r). (r is one rounded number that every exponent is taken
// against, in one rounding: never contracted.) Nothing seen: r = kLowest and no sums.
struct State {
  float r = kLowest, s = 0.f, c = 0.f;
  // moves the sums from this base to a larger one
  __device__ __forceinline__ void raise(float to) {
    const float d = r - to, f = ex2(d);
    c = f > 0.f ? f * fmaf(d, s, c) : 0.f * c;  // keeps a NaN
    s *= f;
    r = to;
  }
  __device__ __forceinline__ void join(State o) {
    const float to = fmaxf(r, o.r);
    raise(to);
    o.raise(to);
    s += o.s;
    c += o.c;
  }
};

// The lanes' states as one, in every lane.
__device__ __forceinline__ void warp_join(State &st) {
  float to = st.r;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) to = fmaxf(to, __shfl_xor_sync(kAll, to, o));
  st.raise(to);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    st.s += __shfl_xor_sync(kAll, st.s, o);
    st.c += __shfl_xor_sync(kAll, st.c, o);
  }
}

__device__ __forceinline__ u64 ld_cluster_u64(uint32_t addr) {
  u64 v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ int ld_cluster_s32(uint32_t addr) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
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

// A row's numbers from its sums (one thread): out[0] the exponent its logits are taken against,
// out[1] log2 of their sum, and the entropy. A far row, whose largest logit is beyond 2^24 / k on
// either side (1e7; a whole row masked with -1e9 or the type's lowest value, or nothing but -inf),
// gets an infinite out[0]: the rounding of m k moves exponents by 1 and more there.
__device__ __forceinline__ void finish_row(const LogprobArgs &a, size_t row, const State &q,
                                           float *out) {
  const float log2_s = log2f(q.s);
  out[0] = q.r > kLowest && q.r <= -kLowest ? q.r : INFINITY;
  out[1] = log2_s;
  out[2] = 0.f;
  if (a.entropy != nullptr) a.entropy[row] = (log2_s - q.c / q.s) * kLn2;
}
// A far row again, by `warps` warps: summed with exponents (v - m) k, m = out[2] the value of the
// largest of the groups' keys. `sync` is their barrier; one stands before the call. Rare, and slow:
// 512 rows of 131072 equal logits (K = 8) take 110 us at 0 and 235 at -1e30, one row of 151936
// (K = 20) 102 and 116.
template <bool kBf16, typename Sync>
__device__ __noinline__ void finish_far(const LogprobArgs &a, size_t row, const void *base, float k,
                                        int t, int warps, const u64 *group, int groups,
                                        State *states, float *out, Sync sync) {
  u64 top = 0;
  for (int i = 0; i < groups; ++i) top = umax(top, group[i]);
  const float m = top == 0 ? NAN : key_value(top);
  const bool some = fabsf(m) < INFINITY;  // else the row has no distribution
  const int V = some ? a.V : 0;
  State q[4];
  for (int i0 = t; i0 < V; i0 += 128 * warps)
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int i = i0 + u * 32 * warps;
      const float v = i < V ? Vec<kBf16>::one(base, i) : -INFINITY;
      const float d = max_nan((v - m) * k, -400.f), e = ex2(d);
      q[u].s += e;
      q[u].c = fmaf(e, d, q[u].c);
    }
  float s = (q[0].s + q[1].s) + (q[2].s + q[3].s), c = (q[0].c + q[1].c) + (q[2].c + q[3].c);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    s += __shfl_xor_sync(kAll, s, o);
    c += __shfl_xor_sync(kAll, c, o);
  }
  if ((t & 31) == 0) states[t >> 5].s = s, states[t >> 5].c = c;
  sync();
  if (t == 0) {
    for (int i = 1; i < warps; ++i) s += states[i].s, c += states[i].c;
    const float log2_s = some ? log2f(s) : NAN;
    out[1] = log2_s;
    out[2] = m;
    if (a.entropy != nullptr) a.entropy[row] = (log2_s - c / s) * kLn2;
  }
  sync();
}
__device__ __forceinline__ float logprob_of(const LogprobArgs &a, float v, float k, const float *out) {
  const float d = fmaf(v, k, -out[0]);
  if (!(fabsf(d) < INFINITY))  // a far row, or k v past the range, where z may not be (and lse is nothing)
    return fmaf(-kLn2, out[1], (v - out[2]) / a.temperature);
  return (d - out[1]) * kLn2;
}
// One of a row's alternatives. (In a row with NaN fewer than K keys may have been found: any
// id in range then.)
__device__ __forceinline__ void emit(const LogprobArgs &a, size_t row, int place, u64 key, float k,
                                     const float *out) {
  a.top_ids[row * a.K + place] = key == 0 ? place : key_id(key);
  a.top_logprobs[row * a.K + place] =
      logprob_of(a, key == 0 ? NAN : key_value(key), k, out);
}

// A thread's part of a row: its sums, and its largest logit with its id.
template <bool kBf16>
struct Running {
  using V = Vec<kBf16>;
  static constexpr int E = V::kN;
  State sums;
  float m = -INFINITY;
  int best_id = -1;  // nothing seen yet

  __device__ __forceinline__ u64 key() const {
    return best_id < 0 ? 0ull : rank_key(m, best_id);
  }
  // n vectors' worth of logits, the first element of vector u being first + u * stride
  template <int n>
  __device__ __forceinline__ void group(const uint4 (&x)[n], int first, int stride, float k) {
    const float mx = V::template largest<n>(x);
    if (mx > m || best_id < 0) {  // strictly: of equal values the lower id stays
      sums.raise(base_of(mx, k));
      m = mx;
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
    const float r = sums.r;
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
    sums.s += s0 + s1;
    sums.c += c;
  }
  __device__ __forceinline__ void single(float v, int id, float k) {
    if (v > m || best_id < 0) {
      sums.raise(base_of(v, k));
      m = v;
      best_id = id;
    }
    const float d = max_nan(fmaf(v, k, -sums.r), -400.f), e = ex2(d);
    sums.s += e;
    sums.c = fmaf(e, d, sums.c);
  }
};

// A warp's 32 largest keys that reach `bound`, sorted downwards across its lanes.
struct Best {
  u64 list = 0, bound;
  __device__ explicit Best(u64 bound) : bound(bound) {}
  __device__ __forceinline__ void offer(u64 key) {  // a key per lane
    unsigned todo = __ballot_sync(kAll, key >= bound);
    while (todo) {
      const int from = __ffs(todo) - 1;
      todo &= todo - 1;
      list = warp_insert(list, __shfl_sync(kAll, key, from));
    }
  }
  // a vector per lane (those with in = true), its first element's id; most hold nothing: one
  // comparison of the largest value tells
  template <bool kBf16>
  __device__ __forceinline__ void offer_vector(uint4 x, bool in, int id, float least) {
    using V = Vec<kBf16>;
    const uint4 one[1] = {x};
    // (not `<`: a NaN may be the largest key)
    if (!__any_sync(kAll, in && (!(V::template largest<1>(one) < least) || V::any_nan(x)))) return;
    float v[V::kN];
    V::unpack(x, v);
#pragma unroll
    for (int e = 0; e < V::kN; ++e) offer(in ? rank_key(v[e], id + e) : 0ull);
  }
};
__device__ __forceinline__ float least_of(u64 bound) {
  return bound > 1 ? key_value(bound) : -INFINITY;
}

// ------------------------------------------------------------------ few rows
// grid (C, rows), cluster (C, 1): CTA r takes vectors [v0, v1) of its row, CTA 0 also the
// elements before the first aligned vector, the last CTA those behind the last; thread t has
// vectors t, t + kFew, ... of the slice.
constexpr int kFew = 256;
constexpr int kFewWarps = kFew / 32;
constexpr int kMaxGroups = 128;  // of a row

struct Slice {  // what a CTA keeps for the others of its cluster
  State sums[kFewWarps];
  int n;          // keys of `list`
  u64 group[kMaxGroups];  // the largest keys of its groups of threads
  u64 list[32];   // its keys that reach the row's bound, at most K of them
};

template <bool kBf16>
__global__ void __launch_bounds__(kFew, 4) logprobs_few_kernel(const LogprobArgs a) {
  using V = Vec<kBf16>;
  constexpr int E = V::kN;
  __shared__ Slice s_slice;
  __shared__ u64 s_all[kMaxGroups], s_bound, s_cand[kMaxCluster * 32];
  __shared__ State s_states[kFewWarps];
  __shared__ float s_out[3];
  __shared__ int s_count;
  pdl_launch_dependents();
  pdl_wait_prior_grid();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int C = gridDim.x, rank = blockIdx.x;
  const size_t row = blockIdx.y;
  const float k = 1.4426950408889634f / a.temperature;
  const Row<kBf16> r(a, row, rank, C);
  Running<kBf16> run;
  if (tid == 0) {
    s_count = 0;
    s_bound = 1;  // for fewer than K keys
  }
  // the given ids' logits and the row's ends, on their way while the row streams
  const int my_id = rank == 0 && tid < a.C ? a.ids[row * a.C + tid] : -1;
  const int end_id = rank == 0 && tid < r.head ? tid
                     : rank == C - 1 && tid >= 32 && r.tail0 + tid - 32 < a.V ? r.tail0 + tid - 32
                                                                              : -1;
  const float end_value = end_id >= 0 ? V::one(r.base, end_id) : 0.f;
  {
    constexpr int kStep = kUnroll * kFew;
    const int full = (r.v1 - r.v0) / kStep;  // groups that every thread has whole
    const uint4 *p = r.vec + r.v0 + tid;
    uint4 x[kUnroll], next[kUnroll];
    if (full > 0) {
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) next[u] = ld_stream(p + u * kFew);
    }
    int first = r.head + (r.v0 + tid) * E;
    for (int i = 0; i < full; ++i) {
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) x[u] = next[u];
      p += kStep;
      if (i + 1 < full) {
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) next[u] = ld_stream(p + u * kFew);
      }
      run.group(x, first, kFew * E, k);
      first += kStep * E;
    }
    for (int at = r.v0 + full * kStep + tid; at < r.v1; at += kFew) {
      const uint4 y[1] = {ld_stream(r.vec + at)};
      run.group(y, r.head + at * E, 0, k);
    }
  }
  // (an end's id need not be in order here: keys of equal values are compared by id)
  const float given = my_id >= 0 && my_id < a.V ? V::one(r.base, my_id) : -INFINITY;
  const u64 vec_key = run.key(), end_key = end_id >= 0 ? rank_key(end_value, end_id) : 0ull;
  if (end_id >= 0) run.single(end_value, end_id, k);

  // ---- the slice: every warp's sums, the largest keys of its groups of threads
  const int per = kMaxGroups / C, groups = kMaxGroups;  // groups to a CTA, of the row
  State st = run.sums;
  warp_join(st);
  if (lane == 0) s_slice.sums[warp] = st;
  u64 g = umax(vec_key, end_key);
  for (int o = 1; o < kFew / per; o *= 2) g = umax(g, __shfl_xor_sync(kAll, g, o));
  if (tid % (kFew / per) == 0) s_slice.group[tid / (kFew / per)] = g;
  cluster_sync();
  const uint32_t here = smem_addr(&s_slice);
  if (tid < groups)
    s_all[tid] = ld_cluster_u64(
        cluster_map(here + (uint32_t)offsetof(Slice, group), tid / per) + 8 * (tid % per));
  if (rank == 0) {  // the row's sums: a state per (CTA, warp)
    State q;
    if (tid < C * kFewWarps) {
      const uint32_t at = cluster_map(here, tid / kFewWarps) +
                          (uint32_t)sizeof(State) * (tid % kFewWarps);
      q.r = ld_cluster_f32(at);
      q.s = ld_cluster_f32(at + 4);
      q.c = ld_cluster_f32(at + 8);
    }
    warp_join(q);
    if (lane == 0) s_states[warp] = q;
  }
  __syncthreads();
  if (rank == 0 && warp == kFewWarps - 1) {
    State q;
    if (lane < kFewWarps) q = s_states[lane];
    warp_join(q);
    if (lane == 0) finish_row(a, row, q, s_out);
  }
  auto far_row = [&] {  // (a barrier stands between s_out's writing and this)
    if (rank == 0 && isinf(s_out[0]))
      finish_far<kBf16>(a, row, r.base, k, tid, kFewWarps, s_all, groups, s_states, s_out,
                        [] { __syncthreads(); });
  };
  if (a.K > 0) {
    // the K-th largest of the groups' keys
    if (tid < groups && s_all[tid] > 0 && larger(s_all, groups, s_all[tid]) == a.K - 1)
      s_bound = s_all[tid];
    __syncthreads();
    const u64 bound = s_bound;
    Best best(bound);
    // who can hold more than its largest: its vectors again, a warp each
    unsigned owners = __ballot_sync(kAll, vec_key >= bound);
    const float least = least_of(bound);
    if (__any_sync(kAll, end_key >= bound)) best.offer(end_key);
    for (; owners != 0; owners &= owners - 1) {
      const int owner = warp * 32 + __ffs(owners) - 1;
      for (int j0 = r.v0 + owner; j0 < r.v1; j0 += 32 * kFew) {
        const int j = j0 + lane * kFew;
        uint4 x = make_uint4(0u, 0u, 0u, 0u);
        if (j < r.v1) x = ld_stream(r.vec + j);
        best.offer_vector<kBf16>(x, j < r.v1, r.head + j * E, least);
      }
    }
    const int found = min(a.K, __popc(__ballot_sync(kAll, best.list > 0)));
    if (found > 0) {
      int at = 0;
      if (lane == 0) at = atomicAdd(&s_count, found);
      at = __shfl_sync(kAll, at, 0);
      if (lane < found) s_cand[at + lane] = best.list;  // at most kFewWarps x 32
    }
    __syncthreads();
    const int cands = s_count;
    if (tid < cands) {
      const u64 key = s_cand[tid];
      const int place = larger(s_cand, cands, key);
      if (place < a.K) s_slice.list[place] = key;
    }
    if (tid == 0) s_slice.n = min(cands, a.K);
    cluster_sync();
    far_row();
    if (rank == 0) {
      if (tid == 0) s_count = 0;
      __syncthreads();
      int n = 0;
      if (lane < C) n = ld_cluster_s32(cluster_map(here + (uint32_t)offsetof(Slice, n), lane));
      for (int i0 = 0; i0 < C * a.K; i0 += kFew) {
        const int i = i0 + tid, c = min(i / a.K, C - 1), j = i - c * a.K;
        const int have = __shfl_sync(kAll, n, c);
        if (j < have && j < a.K)
          s_cand[atomicAdd(&s_count, 1)] = ld_cluster_u64(
              cluster_map(here + (uint32_t)offsetof(Slice, list), c) + 8 * j);
      }
      __syncthreads();
      const int all = s_count;  // at most 16 x 32
      for (int i = tid; i < max(all, a.K); i += kFew) {
        const u64 key = i < all ? s_cand[i] : 0;
        const int place = i < all ? larger(s_cand, all, key) : i;  // (past them: a row with NaN)
        if (place < a.K) emit(a, row, place, key, k, s_out);
      }
    }
  } else {
    __syncthreads();
    far_row();
  }
  if (rank == 0) {
    if (tid < a.C) a.logprobs[row * a.C + tid] = logprob_of(a, given, k, s_out);
    for (int i = tid + kFew; i < a.C; i += kFew) {
      const int id = a.ids[row * a.C + i];
      a.logprobs[row * a.C + i] =
          logprob_of(a, id >= 0 && id < a.V ? V::one(r.base, id) : -INFINITY, k, s_out);
    }
  }
  if (C > 1) cluster_exit_sync();  // no CTA leaves while another still reads its shared memory
}

// ----------------------------------------------------------------- many rows
// A barrier of the post warps.
__device__ __forceinline__ void post_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(kPost) : "memory");
}

// CTA x takes rows x, x + grid, ... Streaming thread t has a row's vectors t, t + kThreads, ...
template <bool kBf16>
__global__ void __launch_bounds__(kBlock, kCtasPerSm) logprobs_many_kernel(const LogprobArgs a,
                                                                           int rows) {
  using V = Vec<kBf16>;
  constexpr int E = V::kN;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ uint64_t s_bar[2 * kStages + 4];
  __shared__ float4 s_sums[2][kThreads];  // (r, s, c) of a row's streaming threads
  __shared__ u64 s_keys[2][kThreads];     // and their largest keys (0: nothing seen)
  __shared__ State s_states[kPostWarps];
  __shared__ u64 s_group[kPost], s_bound;  // the largest key of every 3 or 12 streaming threads
  __shared__ u64 s_cand[kPost];
  __shared__ float s_out[3];
  __shared__ int s_count[2];              // owners and candidates
  __shared__ short s_owner[kThreads];
  __shared__ volatile int s_abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t ring = smem_addr(smem), bar_full = smem_addr(s_bar);
  const uint32_t bar_empty = bar_full + 8 * kStages;
  // a row's sums are left; they have been taken
  const uint32_t bar_left = bar_empty + 8 * kStages, bar_taken = bar_left + 16;
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(bar_full + 8 * i, 1);
      mbar_init(bar_empty + 8 * i, kWarps);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar_left + 8 * i, kWarps);
      mbar_init(bar_taken + 8 * i, kPostWarps);
    }
    s_abort = 0;
    s_count[0] = s_count[1] = 0;
    fence_barrier_init();
  }
  __syncthreads();
  pdl_launch_dependents();
  pdl_wait_prior_grid();
  const float k = 1.4426950408889634f / a.temperature;
  // A bounded wait; one that gave up makes this and the later rows NaN.
  auto await = [&](uint32_t bar, uint32_t parity) {
    if (mbar_try_wait(bar, parity)) return true;
    const unsigned long long t0 = global_ns();
    while (!mbar_try_wait(bar, parity)) {
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
      for (size_t row = blockIdx.x; row < rows && !s_abort; row += gridDim.x) {
        const Row<kBf16> r(a, row, 0, 1);
        for (int at = 0; at < r.v1; at += kStageVecs, ++n) {
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
  } else if (warp < kWarps) {
    // ---------------------------------------------------------------- stream
    int n = 0;
    for (size_t row = blockIdx.x; row < rows; row += gridDim.x, ++turn) {
      const Row<kBf16> r(a, row, 0, 1);
      const int par = turn & 1;
      Running<kBf16> run;
      for (int at = 0; at < r.v1; at += kStageVecs, ++n) {
        const int slot = n % kStages, here = min(kStageVecs, r.v1 - at);
        if (!__all_sync(kAll, await(bar_full + 8 * slot, (n / kStages) & 1) ? 1 : 0)) {
          run.sums.s = NAN;  // a copy that never came
          break;
        }
        const uint32_t src = ring + slot * (kStageVecs * 16) + tid * 16;
        const int first = r.head + (at + tid) * E;
        if (here == kStageVecs) {
          uint4 x[kUnroll];
#pragma unroll
          for (int u = 0; u < kUnroll; ++u) x[u] = ld_shared(src + u * (kThreads * 16));
          run.group(x, first, kThreads * E, k);
        } else {
          for (int u = 0; tid + u * kThreads < here; ++u) {
            const uint4 y[1] = {ld_shared(src + u * (kThreads * 16))};
            run.group(y, first + u * kThreads * E, 0, k);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_empty + 8 * slot);
      }
      if (turn >= 2) __all_sync(kAll, await(bar_taken + 8 * par, ((turn >> 1) + 1) & 1) ? 1 : 0);
      s_sums[par][tid] = make_float4(run.sums.r, run.sums.s, run.sums.c, 0.f);
      s_keys[par][tid] = run.key();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_left + 8 * par);
    }
  } else {
    // ---------------------------------------------------------------- put rows together
    const int p = tid - kThreads - 32, pw = p >> 5;
    for (size_t row = blockIdx.x; row < rows; row += gridDim.x, ++turn) {
      const int par = turn & 1, phase = (turn >> 1) & 1;
      const Row<kBf16> r(a, row, 0, 1);
      // a given id's logit and one element of each of the row's ends, while the row streams
      float given = -INFINITY;
      if (p < a.C) {
        const int id = a.ids[row * a.C + p];
        if (id >= 0 && id < a.V) given = V::one(r.base, id);
      }
      Running<kBf16> run;
      u64 ends = 0;
      const int end_id = p < r.head ? p : p >= 32 && r.tail0 + p - 32 < a.V ? r.tail0 + p - 32 : -1;
      if (end_id >= 0) {
        const float v = V::one(r.base, end_id);
        run.single(v, end_id, k);
        ends = rank_key(v, end_id);
      }
      const bool left = await(bar_left + 8 * par, phase);
      State st = run.sums;
      u64 mine[kEach], most = ends;
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        const float4 x = s_sums[par][p * kEach + i];
        mine[i] = s_keys[par][p * kEach + i];
        most = umax(most, mine[i]);
        st.join(State{x.x, x.y, x.z});
      }
      if (!left) st.s = NAN;
      // 32 groups, or 128 where K of 32 would be too low a bound (K = 32, 64000 fp32 logits: 130
      // threads reach it against 37, 300 rows 55 us against 20)
      const int groups = a.K <= 8 ? 32 : kPost;
      if (a.K <= 8) {
#pragma unroll
        for (int o = 2; o > 0; o >>= 1) most = umax(most, __shfl_xor_sync(kAll, most, o));
        if ((lane & 3) == 0) s_group[p >> 2] = most;
      } else {
        s_group[p] = most;
      }
      warp_join(st);
      if (lane == 0) s_states[pw] = st;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_taken + 8 * par);
      if (p == 0) s_bound = 1;  // for fewer than K keys
      post_sync();
      if (pw == kPostWarps - 1) {
        State q;
        if (lane < kPostWarps) q = s_states[lane];
        warp_join(q);
        if (s_abort) q = State{0.f, NAN, NAN};
        if (lane == 0) finish_row(a, row, q, s_out);
      }
      int place = -1;  // this thread's key's place among the row's best
      u64 key = 0;
      if (a.K > 0) {
        if (p < groups && s_group[p] > 0 && larger(s_group, groups, s_group[p]) == a.K - 1)
          s_bound = s_group[p];  // the K-th largest of the groups' keys
        post_sync();
        const u64 bound = s_bound;
        if (a.K == 1) {
          if (p == 0) place = 0, key = bound > 1 ? bound : 0;
        } else {
#pragma unroll
          for (int i = 0; i < kEach; ++i)
            if (mine[i] >= bound) s_owner[atomicAdd(&s_count[0], 1)] = (short)(p * kEach + i);
          post_sync();
          Best best(bound);
          best.offer(ends);
          // Items of 32 vectors, of one owner or, in short rows, of several; four at a time so that
          // their loads overlap. (1416 rows of 6988 fp32, K = 32: 35 us, with an item per owner 47;
          // 512 rows of 131072, K = 8: 50.3 and 49.3.)
          const int owners = s_count[0], each = (r.v1 + kThreads - 1) / kThreads;
          const int wide = each > 16 ? 5 : each > 8 ? 4 : each > 4 ? 3 : 2;  // log2, lanes an owner
          const int chunks = (each + (1 << wide) - 1) >> wide;
          const int items = ((owners << wide) + 31) / 32 * chunks;
          const float least = least_of(bound);
          for (int i0 = pw; i0 < items; i0 += 4 * kPostWarps) {
            uint4 x[4];
            int j[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const int i = i0 + q * kPostWarps, of = i / chunks;
              const int o = ((of << 5) + lane) >> wide;
              j[q] = r.v1;
              x[q] = make_uint4(0u, 0u, 0u, 0u);
              if (i < items && o < owners)
                j[q] = s_owner[o] +
                       (((i - of * chunks) << wide) + (lane & ((1 << wide) - 1))) * kThreads;
              if (j[q] < r.v1) x[q] = ld_stream(r.vec + j[q]);
            }
#pragma unroll
            for (int q = 0; q < 4; ++q)
              best.offer_vector<kBf16>(x[q], j[q] < r.v1, r.head + j[q] * E, least);
          }
          const int found = min(a.K, __popc(__ballot_sync(kAll, best.list > 0)));
          int at = 0;
          if (lane == 0 && found > 0) at = atomicAdd(&s_count[1], found);
          at = __shfl_sync(kAll, at, 0);
          if (lane < found) s_cand[at + lane] = best.list;  // at most kPostWarps x 32
          post_sync();
          const int cands = s_count[1];
          key = p < cands ? s_cand[p] : 0;
          place = p < cands ? larger(s_cand, cands, key) : p;  // (past them: a row with NaN)
          if (place >= a.K) place = -1;
        }
      }
      post_sync();
      if (isinf(s_out[0]))
        finish_far<kBf16>(a, row, r.base, k, p, kPostWarps, s_group, groups, s_states, s_out,
                          [] { post_sync(); });
      if (p == 0) s_count[0] = s_count[1] = 0;
      if (place >= 0) emit(a, row, place, key, k, s_out);
      if (p < a.C) a.logprobs[row * a.C + p] = logprob_of(a, given, k, s_out);
      for (int i = p + kPost; i < a.C; i += kPost) {
        const int id = a.ids[row * a.C + i];
        a.logprobs[row * a.C + i] =
            logprob_of(a, id >= 0 && id < a.V ? V::one(r.base, id) : -INFINITY, k, s_out);
      }
    }
  }
}

// CTAs per row of the kernel for few rows: as many as keep at least two vectors per thread and
// one round of CTAs, at most 16 (a cluster).
int few_ctas(int B, int V, bool bf16, int sms) {
  const long long nvec = V / (bf16 ? 8 : 4);
  int c = 1;
  while (c < kMaxCluster && (long long)B * 2 * c <= 4ll * sms && nvec >= 2ll * kFew * (2 * c)) c *= 2;
  return c;
}

template <bool kBf16>
cudaError_t launch(const LogprobArgs &a, int B, cudaStream_t stream) {
  static std::atomic<int> sm_count[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  int sms = dev < 64 ? sm_count[dev].load(std::memory_order_acquire) : 0;
  if (sms == 0) {
    if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess ||
        (e = cudaFuncSetAttribute(logprobs_few_kernel<kBf16>,
                                  cudaFuncAttributeNonPortableClusterSizeAllowed, 1)) !=
            cudaSuccess ||
        (e = cudaFuncSetAttribute(logprobs_many_kernel<kBf16>,
                                  cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem)) !=
            cudaSuccess)
      return e;
    if (dev < 64) sm_count[dev].store(sms, std::memory_order_release);
  }
  // A row of up to 160 KB, or more rows than SMs: a CTA a row. K = 8 fp32, us of this kernel and of
  // the one for few rows: 32000 logits 7.9 and 7.0 (1 row), 7.8 and 8.6 (32); 131072 logits 16
  // and 7 (1), 21 and 18 (128), 24 and 25 (192), 95 and 108 (1024).
  if ((long long)a.V * (kBf16 ? 2 : 4) <= (160 << 10) || B > sms) {
    const int grid = B < kCtasPerSm * sms ? B : kCtasPerSm * sms;
    e = launch_pdl(logprobs_many_kernel<kBf16>, dim3(grid), kBlock, kSmem, stream, a, B);
    return e != cudaSuccess ? e : cudaGetLastError();
  }
  const int c = few_ctas(B, a.V, kBf16, sms);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(c, B);
  cfg.blockDim = dim3(kFew);
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
  if ((e = cudaLaunchKernelEx(&cfg, logprobs_few_kernel<kBf16>, a)) != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_logprobs(const LogprobArgs &a, int B, cudaStream_t stream) {
  return a.bf16 ? launch<true>(a, B, stream) : launch<false>(a, B, stream);
}

}  // namespace decattn
