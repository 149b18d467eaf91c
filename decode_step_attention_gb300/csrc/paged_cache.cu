// The paged key/value cache: the append of new tokens with the rotation on the way, and the
// gather of a range of tokens into a contiguous cache.
//
// Pages [num_pages, Hkv, page, D] in bf16, or in e4m3 codes with a scale per (page, KV head), found
// through table[b, p / page]. A stored value is code * scale; the append's scales are powers of two, so
// that a code's relative rounding (half a step, 2^-4) does not depend on them, scaling an input is
// exact, and a page whose scale has to grow keeps its codes' values but for those that fall into
// e4m3's steps of 2^-9 (a second rounding there, of half such a step).
//
// Append: per token i of sequence b at position p = start[b] + i the step of
// qknorm_rope_append.cu (fusedtok README, "Operators": RoPE with a kv-cache position offset;
// cutileGPT README, "The current runtime includes": fused QK-Norm + RoPE + KV-cache writes), the
// first rot_dim elements of a head rotated. Two kinds of work:
//   rows   a (token, head) by D / 16 lanes, 16 elements each: queries, and keys and values wherever a
//          page's scale needs no other token (bf16 pages; one token per sequence)
//   runs   the tokens of a call that share an e4m3 page, which one scale has to hold: read once, the
//          largest magnitude over all of them, then coded from registers
// A key's code is the nearest to the exact rotated key. The fp32 value settles it but where it lies
// within fp32's error of the border between two codes: those elements (one in some 50,000; 20,000
// with a norm) are formed again in fp64. The same for bf16 keys whose rotation cancels.
//
// What bounds it, and what it measured (us on the GPU; TB/s of what is read and written):
//   12.3 k tokens of 8 prompts, 32 + 8 heads of 128, e4m3 pages of 64  51  5.4  the rows alone 35 (memory),
//       the runs alone 38: the keys' instructions, a quarter of them for the borders of codes
//   9.2 k tokens in 3 chunks, bf16 pages, norm, 32 of 128 elements turned  39  5.8  memory
//   256 single tokens, 16 + 4 heads, e4m3  8.3  the chain of look-up, scale, rotation, exact elements
//   one token  3.7  the launch
// One warp per run and general sines measured 218 and 84 for the first two; short series 124, the
// exact elements off the common path 95, a run's angles once for several heads 81, rows and runs side
// by side 71, tokens that fill a block 66 and 47, heads on their way in shared memory 57 and 40, no
// branches where nothing is normed and all is turned 55, blocks of keys before those of values 51.
#include <cuda_fp8.h>

#include <algorithm>
#include <type_traits>

#include "dec_device.cuh"
#include "dec_launch.h"
#include "rope_angles.cuh"

namespace decattn {
namespace {

constexpr int kThreads = 256;  // of a block; 512 where a page takes as many
// Heads are spread over more blocks until there are so many (of 256 threads) per SM. (The prompts and
// chunks above, us with 2, 4, 6 and 8: 52.7 and 41.8, 51.3 and 38.8, 56.4 and 38.9, 56.4 and 38.8.)
constexpr int kBlocksPerSm = 4;
constexpr int kMostWarps = 16;
constexpr int kMinScaleExp = -64;  // the scale of a page of zeros, and the smallest

// A row (token, head) is D / 16 lanes; a lane has two groups of 8 elements, u and v, of which u[j]
// turns with v[j] when the lane's elements are rotated. NeoX: 8 elements of the first half of the
// rotated part and their partners of the second; the groups behind the rotated part two by two.
// Interleaved: 16 neighbours, the even ones in u. Pair j of lane l has frequency 8 l + j either way.
template <int D, bool kInterleaved>
struct Row {
  static constexpr int kLanes = D / 16;
  // elements where the lane's two loads of 8 begin
  __device__ static void places(int l, int rot, int &a, int &b) {
    const int pairs = rot >> 4;  // lanes with rotated elements
    if (kInterleaved) {
      a = 16 * l;
      b = a + 8;
    } else if (l < pairs) {
      a = 8 * l;
      b = 8 * (l + pairs);
    } else {
      a = 16 * l;  // (2 pairs + 2 (l - pairs)) * 8
      b = a + 8;
    }
  }
  __device__ static void unpack(uint4 x, uint4 y, float (&u)[8], float (&v)[8]) {
    const uint32_t a[4] = {x.x, x.y, x.z, x.w}, b[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (kInterleaved) {
        u[j] = bf16_lo(a[j]), v[j] = bf16_hi(a[j]);
        u[4 + j] = bf16_lo(b[j]), v[4 + j] = bf16_hi(b[j]);
      } else {
        u[2 * j] = bf16_lo(a[j]), u[2 * j + 1] = bf16_hi(a[j]);
        v[2 * j] = bf16_lo(b[j]), v[2 * j + 1] = bf16_hi(b[j]);
      }
    }
  }
  // back to the order of memory: f of elements a .. a + 7, then b .. b + 7
  __device__ static void order(const float (&u)[8], const float (&v)[8], float (&f)[16]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (kInterleaved) {
        f[2 * j] = u[j], f[2 * j + 1] = v[j];
      } else {
        f[j] = u[j], f[8 + j] = v[j];
      }
    }
  }
};

// sin and cos of position p's angle: p * turns modulo 2^64 is its fraction of a turn, the nearest quarter
// turn goes off in integers, and the Taylor series run to x^9 and x^8 at |x| <= pi / 4 (the next terms are
// below 2e-9 and 3e-8). Half the instructions of a general sincosf, whose reduction is not needed.
__device__ __forceinline__ void quick_sincos(int p, unsigned long long turns, float &s, float &c) {
  const unsigned hi = (unsigned)(((unsigned long long)(unsigned)p * turns) >> 32);
  const unsigned quarter = (hi + (1u << 29)) >> 30;
  const float x = (float)(int)(hi - (quarter << 30)) * 1.4629180792671596e-09f;  // 2 pi / 2^32
  const float z = x * x;
  float a = fmaf(z, 1.f / 362880.f, -1.f / 5040.f), b = fmaf(z, 1.f / 40320.f, -1.f / 720.f);
  a = fmaf(a, z, 1.f / 120.f);
  b = fmaf(b, z, 1.f / 24.f);
  a = fmaf(a, z, -1.f / 6.f);
  b = fmaf(b, z, -0.5f);
  a = fmaf(a * z, x, x);
  b = fmaf(b, z, 1.f);
  const float sn = quarter & 1 ? b : a, cs = quarter & 1 ? a : b;
  s = quarter & 2 ? -sn : sn;
  c = (quarter + 1) & 2 ? -cs : cs;
}

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ float2 from_e4m3x2(uint32_t codes) {
  const __half2_raw h =
      __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)codes, __NV_E4M3);
  return __half22float2(__half2(h));
}

// The smallest power of two s with amax <= 448 s (448 is e4m3's largest value, 1.75 * 2^8).
__device__ __forceinline__ float scale_for(float amax) {
  const uint32_t bits = __float_as_uint(amax);
  const int e = (int)(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
  return __uint_as_float((uint32_t)(max(e, kMinScaleExp) + 127) << 23);
}
// The magnitude of a finite value, 0 of any other: an infinity or a NaN must not set a page's scale.
__device__ __forceinline__ float finite_abs(float x) {
  const float a = fabsf(x);
  return a < INFINITY ? a : 0.f;
}
// x / s; a product when s is a power of two, exact then too.
__device__ __forceinline__ void unscale(const float (&u)[8], const float (&v)[8], float s,
                                        float (&a)[8], float (&b)[8]) {
  if ((__float_as_uint(s) & 0x7fffffu) == 0) {
    const float inv = 1.f / s;
#pragma unroll
    for (int j = 0; j < 8; ++j) a[j] = u[j] * inv, b[j] = v[j] * inv;
  } else {
#pragma unroll 1
    for (int j = 0; j < 16; ++j) {  // (a scale that the caller wrote: rare, and kept small)
      float x = 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k) x = j == k ? u[k] : j == 8 + k ? v[k] : x;
      x /= s;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        a[k] = j == k ? x : a[k];
        b[k] = j == 8 + k ? x : b[k];
      }
    }
  }
}

// Sixteen codes of a page by the ratio of its old scale to its new one.
__device__ __forceinline__ uint4 rescale16(uint4 w, float ratio) {
  uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 a = from_e4m3x2(x[i] & 0xffffu), b = from_e4m3x2(x[i] >> 16);
    x[i] = e4m3x2(a.x * ratio, a.y * ratio) | e4m3x2(b.x * ratio, b.y * ratio) << 16;
  }
  return make_uint4(x[0], x[1], x[2], x[3]);
}

struct AppendArgs {
  const __nv_bfloat16 *q_in, *k_new, *v_new, *q_norm_w, *k_norm_w;
  __nv_bfloat16 *q_out;
  void *k_pages, *v_pages;
  float *k_scale, *v_scale;  // e4m3 pages only
  const int32_t *table, *start, *cu_new;  // cu_new: may be null (one token per sequence)
  uint32_t *error_word;
  long long q_ld, qo_ld, k_ld, v_ld;
  int n, B, num_pages, page_log2, max_pages, Hq, Hkv, rot;
  float eps;
  // tokens and heads of a block of rows, and the blocks of them
  int tok_par, heads_per, row_blocks, head_blocks;
  int run_heads, run_blocks;  // KV heads (keys, then values) of a block of runs; blocks for them all
};

// Where token i goes: its sequence, its position, and the page's number (-1: nowhere). The whole warp
// calls it, with any i.
struct Place {
  int b, pos, page;
  long long end;  // the first token behind the sequence's
};
__device__ __forceinline__ Place place_of(const AppendArgs &a, int i) {
  Place p;
  long long first = i;
  p.end = i + 1;
  if (a.cu_new == nullptr) {
    p.b = i < a.n ? i : -1;
  } else {
    // the last sequence that begins at or before i: up to 32 at once, a lane each, more by halving
    int lo = 0, hi = a.B;
    if (a.B <= 32) {
      const int lane = threadIdx.x & 31, mine = a.cu_new[min(lane, a.B - 1)];
      for (int b = 1; b < a.B; ++b)
        if (__shfl_sync(0xffffffffu, mine, b) <= i) lo = b;
      first = __shfl_sync(0xffffffffu, mine, lo);
    } else {
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a.cu_new[mid] <= i) lo = mid; else hi = mid;
      }
      first = a.cu_new[lo];
    }
    p.b = lo;
    p.end = min(a.cu_new[lo + 1], a.n);
    if (first > i || p.end <= i) p.b = -1;  // a token of no sequence, or none
  }
  p.pos = p.page = -1;
  if (p.b < 0) return p;
  const long long pos = (long long)a.start[p.b] + (i - first);
  if (pos < 0 || pos > 0x7fffffffll || a.start[p.b] < 0) {
    if (a.error_word != nullptr) atomicOr(a.error_word, kErrPosSkipped);
    return p;
  }
  p.pos = (int)pos;
  const int slot = p.pos >> a.page_log2;
  if (slot >= a.max_pages) {
    if (a.error_word != nullptr) atomicOr(a.error_word, kErrPosSkipped);
    return p;
  }
  const int page = a.table[(size_t)p.b * a.max_pages + slot];
  if (page < 0 || page >= a.num_pages) {
    if (a.error_word != nullptr) atomicOr(a.error_word, kErrPageSkipped);
    return p;
  }
  p.page = page;
  return p;
}

// A lane's part of a row, normed and rotated.
struct Turned {
  float u[8], v[8];
};

// From the elements as loaded (x, y; wa, wb: the norm's weights). kPlain: no norm, and all are turned.
// kBits: the elements whose rotation cancels so far that fp32 leaves them more than half a bf16 step off
// (u, then v).
template <int D, bool kInterleaved, bool kPlain, bool kBits>
__device__ __forceinline__ unsigned turn(Turned &t, uint4 x, uint4 y, bool norm, uint4 wa, uint4 wb,
                                         float eps, bool rotated, const float (&cs)[8],
                                         const float (&sn)[8], bool key, float &rstd) {
  using R = Row<D, kInterleaved>;
  R::unpack(x, y, t.u, t.v);
  uint64_t u[4], v[4];  // two elements at a time
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    u[j] = pair_of(t.u[2 * j], t.u[2 * j + 1]);
    v[j] = pair_of(t.v[2 * j], t.v[2 * j + 1]);
  }
  if (!kPlain && norm) {
    uint64_t su = mul2(u[0], u[0]), sv = mul2(v[0], v[0]);
#pragma unroll
    for (int j = 1; j < 4; ++j) {
      su = fma2(u[j], u[j], su);
      sv = fma2(v[j], v[j], sv);
    }
    float s0, s1;
    unpair(add2(su, sv), s0, s1);
    s0 += s1;
#pragma unroll
    for (int o = R::kLanes / 2; o > 0; o >>= 1) s0 += __shfl_xor_sync(0xffffffffu, s0, o);
    rstd = rsqrtf(s0 * (1.0f / (float)D) + eps);
    const uint64_t r = pair_of(rstd, rstd);
    float p[8], q[8];
    R::unpack(wa, wb, p, q);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      u[j] = mul2(mul2(u[j], r), pair_of(p[2 * j], p[2 * j + 1]));
      v[j] = mul2(mul2(v[j], r), pair_of(q[2 * j], q[2 * j + 1]));
    }
  }
  unsigned bits = 0;
  if (kPlain || rotated) {
    // (the roundings are those of rope_first and rope_second: a product, then a fused sum)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint64_t c = pair_of(cs[2 * j], cs[2 * j + 1]), n = pair_of(sn[2 * j], sn[2 * j + 1]);
      const uint64_t a = fma2(u[j], c, mul2(v[j], pair_of(-sn[2 * j], -sn[2 * j + 1])));
      v[j] = fma2(u[j], n, mul2(v[j], c));
      u[j] = a;
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    unpair(u[j], t.u[2 * j], t.u[2 * j + 1]);
    unpair(v[j], t.v[2 * j], t.v[2 * j + 1]);
  }
  if (kPlain || rotated) {
    if (kBits && key)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        // fp32 is off by 7.5 2^-24 of |p| + |q| at most, half a bf16 step is 2^-9 of the value, |p| + |q|
        // at most 2^0.5 of the turned pair's length
        const float r = 0x1.7p-12f * (fabsf(t.u[j]) + fabsf(t.v[j]));
        bits |= (fabsf(t.u[j]) < r ? 1u << j : 0u) | (fabsf(t.v[j]) < r ? 0x100u << j : 0u);
      }
  }
  return bits;
}

// A double as the float that e4m3's rounding takes the same way: what is cut off leaves its mark in
// the last bit.
__device__ __forceinline__ float sticky(double x) {
  const float f = __double2float_rz(x);
  return (double)f == x ? f : __uint_as_float(__float_as_uint(f) | 1u);
}

// Elements of a key whose fp32 value does not settle the stored one (bits of this lane's 16: u, then
// v; l: its place in the row), again in fp64 from the inputs, and written over. The whole warp calls it;
// rare. A bf16 value takes the row's fp32 norm (1 without it), a code the exact one, whose sum of squares
// the warp forms together (by one lane, 8 us of a small call).
template <int D, bool kInterleaved, bool kE4m3>
__device__ __noinline__ void exact_elements(const __nv_bfloat16 *src, const __nv_bfloat16 *w,
                                            void *dst, float scale_or_rstd, float eps, int pos, int rot,
                                            int l, const unsigned long long *turns, unsigned bits) {
  const int lane = threadIdx.x & 31;
  double factor;  // the norm, and the scale's inverse
  if (kE4m3) {
    const double s = (double)scale_or_rstd, inv = (double)(1.f / scale_or_rstd);
    factor = inv * fma(-s, inv, 2.0);  // (a power of two's is exact before)
    if (w != nullptr) {
      for (unsigned who = __ballot_sync(0xffffffffu, bits != 0); who != 0; who &= who - 1) {
        const int from = __ffs(who) - 1;
        const __nv_bfloat16 *row = reinterpret_cast<const __nv_bfloat16 *>(
            __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(src), from));
        double ss = 0.0;
#pragma unroll
        for (int j = 0; j < D / 32; ++j) {
          const double x = (double)__bfloat162float(row[lane + 32 * j]);
          ss = fma(x, x, ss);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const double mean = fma(ss, 1.0 / D, (double)eps);
        const double r = (double)rsqrtf((float)mean);  // (one step from 2^-22 to 2^-43)
        if (lane == from) factor *= r * fma(-0.5 * mean * r, r, 1.5);
      }
    }
  } else {
    factor = (double)scale_or_rstd;
  }
  int ea, eb;
  Row<D, kInterleaved>::places(l, rot, ea, eb);
  const bool rotated = l < (rot >> 4);
  for (; bits != 0; bits &= bits - 1) {
    const int i = __ffs(bits) - 1, j = i & 7;
    const bool second = i >= 8;
    const int first_at = kInterleaved ? ea + 2 * j : ea + j;
    const int second_at = kInterleaved ? ea + 2 * j + 1 : eb + j;
    const int own_at = second ? second_at : first_at, other_at = second ? first_at : second_at;
    float own = __bfloat162float(src[own_at]), other = __bfloat162float(src[other_at]);
    if (w != nullptr) {  // (exact products of two bf16)
      own *= __bfloat162float(w[own_at]);
      other *= __bfloat162float(w[other_at]);
    }
    const double value =
        (rotated ? rope_element_turns(pos, turns[8 * l + j], own, other, second) : (double)own) *
        factor;
    if (kE4m3)
      static_cast<uint8_t *>(dst)[own_at] = (uint8_t)e4m3x2(sticky(value), 0.f);
    else
      static_cast<__nv_bfloat16 *>(dst)[own_at] = __float2bfloat16((float)value);
  }
}

// How far fp32 may have moved a value, of its pair's magnitudes: the angle's and the series' roundings 3.5
// 2^-24 and the rotation's 2 2^-24; with the norm 9.5 2^-24 more (its sum of 128 squares at most 11
// halved, rsqrt 4 halved, two products).
__device__ __forceinline__ float slack(bool norm) { return norm ? 15 * 0x1p-24f : 5.5f * 0x1p-24f; }

// The codes of a lane's 16 values, and with slack > 0 the values so near a border between two codes that
// the fp32 arithmetic before could have moved them across.
template <int D, bool kInterleaved>
__device__ __forceinline__ unsigned encode(const Turned &t, float scale, float slack, uint2 &a,
                                           uint2 &b) {
  using R = Row<D, kInterleaved>;
  float u[8] = {}, v[8] = {};
  unscale(t.u, t.v, scale, u, v);
  unsigned bits = 0;
  if (slack > 0.f) {
    uint32_t any = 0;
    auto off = [&](int j) {
      const float d = slack * (fabsf(u[j]) + fabsf(v[j]));
      return e4m3x2(u[j] - d, v[j] - d) ^ e4m3x2(u[j] + d, v[j] + d);
    };
#pragma unroll
    for (int j = 0; j < 8; ++j) any |= off(j);
    if (any != 0) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t x = off(j);
        bits |= (x & 0xffu ? 1u << j : 0u) | (x & 0xff00u ? 0x100u << j : 0u);
      }
    }
  }
  float f[16];
  R::order(u, v, f);
  a = make_uint2(e4m3x2(f[0], f[1]) | e4m3x2(f[2], f[3]) << 16,
                 e4m3x2(f[4], f[5]) | e4m3x2(f[6], f[7]) << 16);
  b = make_uint2(e4m3x2(f[8], f[9]) | e4m3x2(f[10], f[11]) << 16,
                 e4m3x2(f[12], f[13]) | e4m3x2(f[14], f[15]) << 16);
  return bits;
}

// The largest magnitude of a lane's values; the finite ones', once there is one that is not.
__device__ __forceinline__ float amax_of(const Turned &t) {
  float m = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) m = fmaxf(m, fmaxf(fabsf(t.u[j]), fabsf(t.v[j])));
  if (m == INFINITY) {
    m = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = fmaxf(m, fmaxf(finite_abs(t.u[j]), finite_abs(t.v[j])));
  }
  return m;
}

// An element of a key to be formed again when a block or a group of threads is done with the others.
struct Fix {
  const __nv_bfloat16 *src;
  void *dst;
  int pos, place;  // place: the row's lane, and the element's bit
  float scale_or_rstd;
};
constexpr int kFixes = 64;
// This lane's elements into a list; what it has no room for is left in `bits`.
__device__ __forceinline__ void put_off(Fix *fixes, int *count, const __nv_bfloat16 *src, void *dst,
                                        int pos, int l, float scale_or_rstd, unsigned &bits) {
  for (; bits != 0; bits &= bits - 1) {
    const int k = atomicAdd(count, 1);
    if (k >= kFixes) break;
    fixes[k] = Fix{src, dst, pos, l * 16 + __ffs(bits) - 1, scale_or_rstd};
  }
}
// The list, a lane each, by threads `of` them (whole warps).
template <int D, bool kInterleaved, bool kE4m3>
__device__ __forceinline__ void work_off(const AppendArgs &a, const RopeTurns &turns, const Fix *fixes,
                                         int count, int thread, int of) {
  count = min(count, kFixes);
  for (int k = thread; (k & ~31) < count; k += of) {
    const Fix f = fixes[k < count ? k : 0];
    exact_elements<D, kInterleaved, kE4m3>(f.src, a.k_norm_w, f.dst, f.scale_or_rstd, a.eps, f.pos,
                                           a.rot, f.place >> 4, turns.v,
                                           k < count ? 1u << (f.place & 15) : 0u);
  }
}

// ---- rows: (token, head) pairs that need nothing of each other ------------------------------
// Heads are counted q, k, v. A block has tok_par tokens side by side, times as many heads as fit,
// and goes through its heads_per heads with them: a lane keeps its token's angles.
template <int D, bool kInterleaved, bool kE4m3, int kBlock>
__device__ __forceinline__ void do_rows(const AppendArgs &a, const RopeTurns &turns, int heads,
                                        int which) {
  using R = Row<D, kInterleaved>;
  constexpr int kRows = kBlock / R::kLanes;
  const int lane = threadIdx.x & 31, l = lane % R::kLanes, row = threadIdx.x / R::kLanes;
  const int block = which % a.head_blocks, tile = which / a.head_blocks;
  const int i = tile * a.tok_par + (row & (a.tok_par - 1));
  const int step = kRows / a.tok_par;
  const int h0 = block * a.heads_per, h1 = min(heads, h0 + a.heads_per);
  const bool rotated = l < (a.rot >> 4), norm = a.q_norm_w != nullptr;
  int ea, eb;
  R::places(l, a.rot, ea, eb);
  // a head's two groups of this lane, on their way while the one before is turned (the first while the
  // token's place is looked up)
  const __nv_bfloat16 *q_src = a.q_in + i * a.q_ld;
  const __nv_bfloat16 *k_src = a.k_new + i * a.k_ld - (ptrdiff_t)a.Hq * D;
  const __nv_bfloat16 *v_src = a.v_new + i * a.v_ld - (ptrdiff_t)(a.Hq + a.Hkv) * D;
  __nv_bfloat16 *q_dst = a.q_out + i * a.qo_ld;
  auto load = [&](int h, uint4 &x, uint4 &y) {
    x = y = make_uint4(0u, 0u, 0u, 0u);
    if (i < a.n && h < h1) {
      const __nv_bfloat16 *src = (h < a.Hq ? q_src : h < a.Hq + a.Hkv ? k_src : v_src) + h * D;
      x = *reinterpret_cast<const uint4 *>(src + ea);
      y = *reinterpret_cast<const uint4 *>(src + eb);
    }
  };
  uint4 next_x, next_y;
  load(h0 + row / a.tok_par, next_x, next_y);
  const Place at = place_of(a, i);
  const bool some = at.pos >= 0;
  float cs[8], sn[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    cs[j] = 1.f;
    sn[j] = 0.f;
    if (rotated && some) quick_sincos(at.pos, turns.v[8 * l + j], sn[j], cs[j]);
  }
  const int in_page = at.pos & ((1 << a.page_log2) - 1);
  // keys of bf16 pages: within one step where the rotation cancels, worked off at the end
  constexpr bool kList = !kE4m3;
  __shared__ Fix s_fixes[kList ? kFixes : 1];
  __shared__ int s_fix_total;
  if (kList) {
    if (threadIdx.x == 0) s_fix_total = 0;
    __syncthreads();
  }
  for (int hh = h0; hh < h1; hh += step) {  // (the same number of times in every lane)
    const int h = hh + row / a.tok_par;
    const bool is_q = h < a.Hq, is_k = !is_q && h < a.Hq + a.Hkv;
    const int g = is_q ? h : is_k ? h - a.Hq : h - a.Hq - a.Hkv;
    const bool live = some && h < h1 && (is_q || at.page >= 0);
    Turned t;
    const uint4 x = next_x, y = next_y;
    if (hh + step < h1) load(h + step, next_x, next_y);
    const bool turns_here = is_q || is_k;
    uint4 wa{}, wb{};
    if (norm) {
      const __nv_bfloat16 *w = is_q ? a.q_norm_w : a.k_norm_w;
      wa = *reinterpret_cast<const uint4 *>(w + ea);
      wb = *reinterpret_cast<const uint4 *>(w + eb);
    }
    unsigned bits = 0;
    float rstd = 1.f;
    // (a warp may hold values beside keys: the norm's shuffles)
    if (norm ? __any_sync(0xffffffffu, turns_here) : turns_here)
      bits = turn<D, kInterleaved, false, !kE4m3>(t, x, y, norm, wa, wb, a.eps, rotated, cs, sn, is_k,
                                                  rstd);
    if (!turns_here) R::unpack(x, y, t.u, t.v);
    const size_t slot =
        live && !is_q
            ? ((((size_t)at.page * a.Hkv + g) << a.page_log2) + (size_t)in_page) * D
            : 0;
    float scale = 1.f;
    if (kE4m3) {
      float m = amax_of(t);
#pragma unroll
      for (int o = R::kLanes / 2; o > 0; o >>= 1)
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      scale = scale_for(m);
      float old = scale;
      float *sp = (is_k ? a.k_scale : a.v_scale) + (live && !is_q ? (size_t)at.page * a.Hkv + g : 0);
      bool grows = false;
      if (live && !is_q && in_page > 0) {
        old = *sp;
        grows = scale > old;
        scale = fmaxf(scale, old);
      }
      __syncwarp();  // every lane of the row has read the scale
      if (live && !is_q && l == 0 && (grows || in_page == 0)) *sp = scale;
      // codes that the page had before, under the grown scale: the warp's rows one after the other
      unsigned who = __ballot_sync(0xffffffffu, grows && l == 0);
      uint8_t *base = static_cast<uint8_t *>(is_k ? a.k_pages : a.v_pages) + slot -
                      (live && !is_q ? (size_t)in_page * D : 0);
      for (; who != 0; who &= who - 1) {
        const int from = __ffs(who) - 1;
        const float ratio = __shfl_sync(0xffffffffu, old / scale, from);
        uint4 *w = reinterpret_cast<uint4 *>(
            __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(base), from));
        const int words = __shfl_sync(0xffffffffu, in_page, from) * (D / 16);
#pragma unroll 4
        for (int k = lane; k < words; k += 32) w[k] = rescale16(w[k], ratio);
      }
    }
    void *dst = nullptr;
    if (live && (is_q || !kE4m3)) {
      float f[16];
      R::order(t.u, t.v, f);
      uint4 oa = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                            pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
      uint4 ob = make_uint4(pack_bf16x2(f[8], f[9]), pack_bf16x2(f[10], f[11]),
                            pack_bf16x2(f[12], f[13]), pack_bf16x2(f[14], f[15]));
      if (!turns_here) oa = x, ob = y;  // a copy, bit for bit
      __nv_bfloat16 *to = is_q ? q_dst + h * D
                               : static_cast<__nv_bfloat16 *>(is_k ? a.k_pages : a.v_pages) + slot;
      *reinterpret_cast<uint4 *>(to + ea) = oa;
      *reinterpret_cast<uint4 *>(to + eb) = ob;
      dst = to;
    } else if (live) {
      uint2 ca, cb;
      bits = encode<D, kInterleaved>(t, scale, is_k && (norm || rotated) ? slack(norm) : 0.f, ca, cb);
      uint8_t *to = static_cast<uint8_t *>(is_k ? a.k_pages : a.v_pages) + slot;
      *reinterpret_cast<uint2 *>(to + ea) = ca;
      *reinterpret_cast<uint2 *>(to + eb) = cb;
      dst = to;
    }
    const __nv_bfloat16 *key = k_src + h * D;
    if (!live || !is_k) bits = 0;
    if (kList) put_off(s_fixes, &s_fix_total, key, dst, at.pos, l, rstd, bits);
    if (__any_sync(0xffffffffu, bits != 0))  // (e4m3: the codes are the exact key's)
      exact_elements<D, kInterleaved, kE4m3>(key, a.k_norm_w, dst, kE4m3 ? scale : rstd, a.eps, at.pos,
                                             a.rot, l, turns.v, bits);
  }
  if (kList) {
    __syncthreads();
    work_off<D, kInterleaved, false>(a, turns, s_fixes, s_fix_total, threadIdx.x, kBlock);
  }
}

// Copies of 16 bytes into shared memory, to be read by the warp: loads on their way without registers.
// `bytes` of 0 leaves zeros.
__device__ __forceinline__ void copy16(uint32_t to, const void *from, int bytes = 16) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All but the last N groups of copies have arrived.
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 shared16(uint32_t at) {
  uint4 x;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
               : "r"(at)
               : "memory");
  return x;
}

// Where the rows of a block's lanes lie in shared memory while they are on their way: row after row in
// chunks of 16 bytes, every second 128 bytes with neighbours swapped, so that eight lanes that read
// every second chunk meet 32 banks. A lane copies chunks l and l + kLanes of its row, whole sectors side
// by side, and reads those that it turns, after the warp has met.
template <int D, bool kInterleaved, int kBlock>
struct RowsAhead {
  using R = Row<D, kInterleaved>;
  static constexpr int kBytes = 32 * kBlock;
  uint32_t to_a, to_b, from_a, from_b;
  int l;
  __device__ __forceinline__ RowsAhead(uint32_t base, int l_, int ea, int eb) : l(l_) {
    const int row = (int)threadIdx.x / R::kLanes * (D / 8);
    auto at = [&](int chunk) {
      const int i = row + chunk;
      return base + ((i ^ ((i >> 3) & 1)) << 4);
    };
    to_a = at(l);
    to_b = at(l + R::kLanes);
    from_a = at(ea >> 3);
    from_b = at(eb >> 3);
  }
  // (at: 0, kBytes, 2 kBytes ..; row: of the lane's own element 8 l)
  __device__ __forceinline__ void copy(int at, const __nv_bfloat16 *row, int bytes = 16) const {
    copy16(to_a + at, row, bytes);
    copy16(to_b + at, row + 8 * R::kLanes, bytes);
  }
};

// The same for batches that fill a block with tokens: a token per row, so that every row of the block is
// at the same head, and the heads go by in loops of their own. kAll: keys and values (bf16 pages) too.
// kHeadsAhead heads are on their way while one is turned, in dynamic shared memory, 8 KB a block for each
// (the prompts and chunks above, us with 1, 2, 3, 4, 5 and 7: 54.8 and 41.5, 52.0 and 39.7, 51.3 and 38.8,
// 50.7 and 38.2, 50.2 and 37.8, 51.6 and 37.9; one in registers, some steps before, 6 and 5 more than 3).
constexpr int kHeadsAhead = 3;
template <int D, bool kInterleaved, bool kPlain, bool kAll, int kBlock>
__device__ __forceinline__ void do_token_rows(const AppendArgs &a, const RopeTurns &turns, int heads,
                                              int which) {
  using R = Row<D, kInterleaved>;
  constexpr int kRows = kBlock / R::kLanes;
  extern __shared__ __align__(128) float s_table[];
  __shared__ Fix s_fixes[kAll ? kFixes : 1];
  __shared__ int s_fix_total;
  const int l = threadIdx.x % R::kLanes, row = threadIdx.x / R::kLanes;
  // kAll: one block of heads after the other for all tokens, keys and values last, the likelier in L2 when
  // they are read (the chunks above, appended and read back, 51.4 and 49.2 us; with a norm and all turned
  // the append alone 55.4 and 51.3). Queries alone: a token's heads side by side (51.4 us of the prompts, else
  // 52.2).
  const int tiles = a.row_blocks / a.head_blocks;
  const int block = kAll ? which / tiles : which % a.head_blocks;
  const int tile = kAll ? which % tiles : which / a.head_blocks;
  const int i = tile * kRows + row, from = min(i, a.n - 1);  // (rows behind the last token read its)
  const int h0 = block * a.heads_per, h1 = min(heads, h0 + a.heads_per);
  const bool rotated = l < (a.rot >> 4), norm = a.q_norm_w != nullptr;
  int ea, eb;
  R::places(l, a.rot, ea, eb);
  const RowsAhead<D, kInterleaved, kBlock> ahead(smem_addr(s_table), l, ea, eb);
  // the next head's row, and its place
  const __nv_bfloat16 *const k_row = a.k_new + from * a.k_ld + 8 * l, *const v_row =
      a.v_new + from * a.v_ld + 8 * l;
  const __nv_bfloat16 *next = !kAll || h0 < a.Hq ? a.q_in + from * a.q_ld + (ptrdiff_t)h0 * D + 8 * l
                              : h0 < a.Hq + a.Hkv ? k_row + (ptrdiff_t)(h0 - a.Hq) * D
                                                  : v_row + (ptrdiff_t)(h0 - a.Hq - a.Hkv) * D;
  int next_h = h0, next_at = 0, head_at = 0;
  auto after = [&](int at) { return at == kHeadsAhead * ahead.kBytes ? 0 : at + ahead.kBytes; };
  auto fetch = [&]() {
    if (next_h < h1) {
      ahead.copy(next_at, next);
      next += D;
      ++next_h;
      if (kAll && next_h == a.Hq) next = k_row;
      if (kAll && next_h == a.Hq + a.Hkv) next = v_row;
    }
    next_at = after(next_at);
    copies_end();
  };
  uint4 x, y;
  auto take = [&](uint32_t at_a, uint32_t at_b) {  // this lane's part of the next head
    __syncwarp();  // (the head before has been read, its place is the next one's)
    fetch();
    copies_wait<kHeadsAhead>();
    __syncwarp();
    x = shared16(at_a + head_at);
    y = shared16(at_b + head_at);
    head_at = after(head_at);
  };
#pragma unroll
  for (int k = 0; k < kHeadsAhead; ++k) fetch();  // (under way while the place is looked up)
  if (kAll) {
    if (threadIdx.x == 0) s_fix_total = 0;
    __syncthreads();
  }
  const Place at = place_of(a, i);
  const bool some = at.pos >= 0;
  float cs[8], sn[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    cs[j] = 1.f;
    sn[j] = 0.f;
    if (rotated && some) quick_sincos(at.pos, turns.v[8 * l + j], sn[j], cs[j]);
  }
  auto pack = [&](const Turned &t, __nv_bfloat16 *to) {
    float f[16];
    R::order(t.u, t.v, f);
    *reinterpret_cast<uint4 *>(to + ea) =
        make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                   pack_bf16x2(f[6], f[7]));
    *reinterpret_cast<uint4 *>(to + eb) =
        make_uint4(pack_bf16x2(f[8], f[9]), pack_bf16x2(f[10], f[11]), pack_bf16x2(f[12], f[13]),
                   pack_bf16x2(f[14], f[15]));
  };
  uint4 wa{}, wb{};
  auto weights = [&](const __nv_bfloat16 *w) {
    if (norm) {
      wa = *reinterpret_cast<const uint4 *>(w + ea);
      wb = *reinterpret_cast<const uint4 *>(w + eb);
    }
  };
  weights(a.q_norm_w);
  int h = h0;
  __nv_bfloat16 *q_dst = a.q_out + from * a.qo_ld + (ptrdiff_t)h0 * D;
  for (const int q1 = min(h1, a.Hq); h < q1; ++h, q_dst += D) {
    take(ahead.from_a, ahead.from_b);
    Turned t;
    float rstd;
    turn<D, kInterleaved, kPlain, false>(t, x, y, norm, wa, wb, a.eps, rotated, cs, sn, false, rstd);
    if (some) pack(t, q_dst);
  }
  if constexpr (kAll) {
    const bool kept = some && at.page >= 0;
    const int in_page = at.pos & ((1 << a.page_log2) - 1);
    const size_t head = (size_t)D << a.page_log2;  // elements of a page's head
    const size_t slot = kept ? (size_t)at.page * a.Hkv * head + (size_t)in_page * D : 0;
    if (h < h1) weights(a.k_norm_w);
    for (const int k1 = min(h1, a.Hq + a.Hkv); h < k1; ++h) {
      take(ahead.from_a, ahead.from_b);
      const int g = h - a.Hq;
      Turned t;
      float rstd = 1.f;
      unsigned bits = turn<D, kInterleaved, kPlain, true>(t, x, y, norm, wa, wb, a.eps, rotated, cs, sn,
                                                          true, rstd);
      __nv_bfloat16 *to = static_cast<__nv_bfloat16 *>(a.k_pages) + slot + g * head;
      if (kept) pack(t, to);
      else bits = 0;
      // within one step where the rotation cancels: worked off at the end
      const __nv_bfloat16 *key = a.k_new + from * a.k_ld + (ptrdiff_t)g * D;
      put_off(s_fixes, &s_fix_total, key, to, at.pos, l, rstd, bits);
      if (__any_sync(0xffffffffu, bits != 0))
        exact_elements<D, kInterleaved, false>(key, a.k_norm_w, to, rstd, a.eps, at.pos, a.rot, l,
                                               turns.v, bits);
    }
    for (; h < h1; ++h) {
      take(ahead.to_a, ahead.to_b);
      __nv_bfloat16 *to =
          static_cast<__nv_bfloat16 *>(a.v_pages) + slot + (h - a.Hq - a.Hkv) * head + 8 * l;
      if (kept) {
        *reinterpret_cast<uint4 *>(to) = x;
        *reinterpret_cast<uint4 *>(to + 8 * R::kLanes) = y;
      }
    }
    __syncthreads();
    work_off<D, kInterleaved, false>(a, turns, s_fixes, s_fix_total, threadIdx.x, kBlock);
  }
}

// ---- runs: the new tokens of one page under one scale ------------------------------------------
struct Run {
  int token, pos, page, count;
};

// One run of up to kPasses * kRows tokens, for the KV heads h0 .. h1 (keys first, then values) one after
// the other, by kGroup threads: a warp, or as many as a page's tokens take. These meet at the named
// barrier `meet` and have the run's angles in `table`: [token][4 pairs of each lane, then the others]
// cosines, then the sines.
// Rows of 128 dims, and pages of 128 tokens, go two tokens to a row's lanes: half the threads to meet.
// (The prompts above, us with one token and with two; 128 dims, pages of 16 and 32: 55.3, 51.4 and 56.1,
// 50.9; 64 dims, pages of 16, 32 and 64: 32.1, 40.7; 32.3, 35.8 and 32.3, 35.5. Larger pages with one would
// need blocks of 512 threads.)
__host__ __device__ constexpr int passes_of(int D, int page) { return D == 128 || page == 128 ? 2 : 1; }
template <int D, bool kInterleaved, bool kPlain, int kGroup, int kBlock, int kPasses>
__device__ __forceinline__ void do_run(const AppendArgs &a, const RopeTurns &turns, const Run &r,
                                       int h0, int h1, uint32_t slots, float *s_max, float *table,
                                       Fix *fixes, int *fix_count, int meet) {
  using R = Row<D, kInterleaved>;
  constexpr bool kWarp = kGroup == 32;
  constexpr int kRows = kGroup / R::kLanes;   // tokens side by side
  constexpr int kToken = D / 2;               // floats of a token's cosines
  constexpr int kSines = kPasses * kRows * kToken;
  const int in_group = threadIdx.x & (kGroup - 1);
  const int lane = threadIdx.x & 31, l = lane % R::kLanes, row = in_group / R::kLanes;
  const bool turned = l < (a.rot >> 4), norm = a.k_norm_w != nullptr;
  auto together = [&]() {
    if (kWarp) __syncwarp();
    else asm volatile("bar.sync %0, %1;" ::"r"(meet), "n"(kGroup) : "memory");
  };
  int ea, eb;
  R::places(l, a.rot, ea, eb);
  const int in_page = r.pos & ((1 << a.page_log2) - 1);
  if (!kWarp && h0 < a.Hkv) {
    for (int i = in_group; i < r.count * R::kLanes; i += kGroup) {
      const int j = i / R::kLanes, of = i % R::kLanes;
      if (of < (a.rot >> 4)) {
        float c[8], s[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) quick_sincos(r.pos + j, turns.v[8 * of + k], s[k], c[k]);
        float4 *to = reinterpret_cast<float4 *>(table + j * kToken) + of;
        to[0] = make_float4(c[0], c[1], c[2], c[3]);
        to[R::kLanes] = make_float4(c[4], c[5], c[6], c[7]);
        to += kSines / 4;
        to[0] = make_float4(s[0], s[1], s[2], s[3]);
        to[R::kLanes] = make_float4(s[4], s[5], s[6], s[7]);
      }
    }
    together();
  }
  // a head's rows, on their way while the one before is coded
  const RowsAhead<D, kInterleaved, kBlock> ahead(slots, l, ea, eb);
  auto fetch = [&](int head) {
    if (head < h1) {
      const bool is_k = head < a.Hkv;
      const __nv_bfloat16 *src =
          (is_k ? a.k_new : a.v_new) + (size_t)(is_k ? head : head - a.Hkv) * D + 8 * l;
      const long long ld = is_k ? a.k_ld : a.v_ld;
#pragma unroll
      for (int p = 0; p < kPasses; ++p) {
        const int j = p * kRows + row;  // (rows behind the run's last token: zeros)
        ahead.copy(p * ahead.kBytes, src + (r.token + min(j, r.count - 1)) * ld, j < r.count ? 16 : 0);
      }
    }
    copies_end();
  };
  fetch(h0);
  for (int head = h0; head < h1; ++head) {
    const bool is_k = head < a.Hkv;
    const int g = is_k ? head : head - a.Hkv;
    float *sp = (is_k ? a.k_scale : a.v_scale) + (size_t)r.page * a.Hkv + g;
    uint8_t *base = static_cast<uint8_t *>(is_k ? a.k_pages : a.v_pages) +
                    (((size_t)r.page * a.Hkv + g) << a.page_log2) * D;
    uint4 x[kPasses], y[kPasses], wa{}, wb{};
    float m = 0.f, old = 0.f;
    if (in_page > 0) old = *sp;
    if (is_k && norm) {
      wa = *reinterpret_cast<const uint4 *>(a.k_norm_w + ea);
      wb = *reinterpret_cast<const uint4 *>(a.k_norm_w + eb);
    }
    copies_wait<0>();
    __syncwarp();
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
      x[p] = shared16(ahead.from_a + p * ahead.kBytes);
      y[p] = shared16(ahead.from_b + p * ahead.kBytes);
    }
    Turned t[kPasses];
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
      if (is_k) {
        const int j = p * kRows + row;
        float cs[8], sn[8], rstd;
        if (kWarp) {
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            cs[k] = 1.f;
            sn[k] = 0.f;
            if (turned) quick_sincos(r.pos + j, turns.v[8 * l + k], sn[k], cs[k]);
          }
        } else {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float4 *at = reinterpret_cast<const float4 *>(table + j * kToken) + l + h * R::kLanes;
            const float4 c = at[0], s = at[kSines / 4];
            cs[4 * h] = c.x, cs[4 * h + 1] = c.y, cs[4 * h + 2] = c.z, cs[4 * h + 3] = c.w;
            sn[4 * h] = s.x, sn[4 * h + 1] = s.y, sn[4 * h + 2] = s.z, sn[4 * h + 3] = s.w;
          }
        }
        // (rows behind the run's last token turn zeros by what the table holds: they are masked)
        turn<D, kInterleaved, kPlain, false>(t[p], x[p], y[p], norm, wa, wb, a.eps, turned, cs, sn, true,
                                             rstd);
        if (j < r.count) m = fmaxf(m, amax_of(t[p]));
      } else {
        R::unpack(x[p], y[p], t[p].u, t[p].v);
        m = fmaxf(m, amax_of(t[p]));
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    fetch(head + 1);  // (its place has been read by the whole warp)
    if (!kWarp) {
      // (two sets of maxima in turn: a warp may be a head ahead of the group's others)
      float *mine = s_max + ((head & 1) ? kMostWarps : 0) + (threadIdx.x / kGroup) * (kGroup / 32);
      if (lane == 0) mine[in_group >> 5] = m;
      together();  // (and everyone has read the scale)
      m = mine[0];
#pragma unroll
      for (int w = 1; w < kGroup / 32; ++w) m = fmaxf(m, mine[w]);
    } else {
      together();
    }
    const float need = scale_for(m), scale = in_page > 0 ? fmaxf(need, old) : need;
    if (in_group == 0 && (scale > old || in_page == 0)) *sp = scale;
    if (in_page > 0 && scale > old) {
      const float ratio = old / scale;
      uint4 *w = reinterpret_cast<uint4 *>(base);
#pragma unroll 4
      for (int k = in_group; k < in_page * (D / 16); k += kGroup) w[k] = rescale16(w[k], ratio);
    }
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
      const int j = p * kRows + row;
      if (p * kRows >= r.count) break;  // (the same for the whole group)
      uint8_t *dst = base + (size_t)(in_page + j) * D;
      unsigned bits = 0;
      if (j < r.count) {
        uint2 ca, cb;
        bits = encode<D, kInterleaved>(t[p], scale, is_k && (norm || turned) ? slack(norm) : 0.f, ca,
                                       cb);
        if (kInterleaved) {  // (16 neighbours)
          *reinterpret_cast<uint4 *>(dst + ea) = make_uint4(ca.x, ca.y, cb.x, cb.y);
        } else {
          *reinterpret_cast<uint2 *>(dst + ea) = ca;
          *reinterpret_cast<uint2 *>(dst + eb) = cb;
        }
      }
      // The codes are the exact key's: a group's elements go into a list, which its threads work off when
      // the heads are done (on the way each would hold up the whole group).
      const __nv_bfloat16 *key = a.k_new + (size_t)g * D + (r.token + j) * a.k_ld;
      if (!kWarp) put_off(fixes, fix_count, key, dst, r.pos + j, l, scale, bits);
      if (__any_sync(0xffffffffu, bits != 0))
        exact_elements<D, kInterleaved, true>(key, a.k_norm_w, dst, scale, a.eps, r.pos + j, a.rot, l,
                                              turns.v, bits);
    }
  }
  if (!kWarp) {
    together();
    work_off<D, kInterleaved, true>(a, turns, fixes, *fix_count, in_group, kGroup);
    together();
    if (in_group == 0) *fix_count = 0;
  }
}

// The runs that begin among a block's `chunk` tokens, for some of the KV heads' keys and values: short
// ones by a warp each, the others by a group of as many threads as a page takes.
template <int D, bool kInterleaved, bool kPlain, int kBlock, int kPage>
__device__ __forceinline__ void do_runs(const AppendArgs &a, const RopeTurns &turns, int block) {
  using R = Row<D, kInterleaved>;
  constexpr int kPasses = passes_of(D, kPage);
  constexpr int kGroup = kPage * R::kLanes / kPasses;  // 64 (16 tokens of 64 dims) .. 512
  constexpr int kChunk = kPage > 64 ? kPage : 64, kWarpRun = kPasses * 32 / R::kLanes;
  extern __shared__ __align__(128) float s_table[];  // of each group: kPage * D
  __shared__ Run s_run[kChunk];
  __shared__ int s_short, s_long, s_fix_count[kBlock / kGroup];
  __shared__ float s_max[2 * kMostWarps];
  __shared__ Fix s_fix[kBlock / kGroup][kFixes];
  // (the heavier blocks, those of keys, first: what is left for the end is short)
  const int chunks = (a.n + kChunk - 1) / kChunk;
  const int c0 = block % chunks * kChunk, h0 = block / chunks * a.run_heads;
  const int h1 = min(2 * a.Hkv, h0 + a.run_heads);
  if (threadIdx.x == 0) s_short = s_long = 0;
  if (threadIdx.x < kBlock / kGroup) s_fix_count[threadIdx.x] = 0;
  __syncthreads();
  const int i = c0 + threadIdx.x;
  if ((int)threadIdx.x < kChunk) {  // (whole warps)
    const Place p = place_of(a, i);
    const bool begins = p.b >= 0 && (i == a.cu_new[p.b] || (p.pos & (kPage - 1)) == 0);
    if (begins && p.page >= 0) {
      const int count = (int)min(p.end - i, (long long)(kPage - (p.pos & (kPage - 1))));
      // short ones from the front of the list, long ones from its back
      const int k = count <= kWarpRun ? atomicAdd(&s_short, 1) : kChunk - 1 - atomicAdd(&s_long, 1);
      s_run[k] = Run{i, p.pos, p.page, count};
    }
  }
  __syncthreads();
  const int shorts = s_short, longs = s_long;
  const uint32_t slots = smem_addr(s_table) + kBlock / kGroup * kPage * D * 4;  // (behind the tables)
  for (int k = threadIdx.x >> 5; k < shorts; k += kBlock / 32)
    do_run<D, kInterleaved, kPlain, 32, kBlock, kPasses>(a, turns, s_run[k], h0, h1, slots, nullptr,
                                                         nullptr, nullptr, nullptr, 0);
  const int group = threadIdx.x / kGroup;
  for (int k = group; k < longs; k += kBlock / kGroup) {
    do_run<D, kInterleaved, kPlain, kGroup, kBlock, kPasses>(
        a, turns, s_run[kChunk - 1 - k], h0, h1, slots, s_max, s_table + group * kPage * D,
        s_fix[group], &s_fix_count[group], 1 + group);
    // (the next run's angles and maxima take this one's place)
    asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "n"(kGroup) : "memory");
  }
}

// kPage = 0: every block takes rows, of queries, keys and values. Else row_blocks of the blocks take the
// queries' rows, the others the runs of e4m3 pages of kPage tokens. kTokens: rows go a token to each, heads
// in loops (with kPage > 0 always). kPlain: no norm, all elements turned (the two branches cost a tenth of
// the instructions, most of them moves: the prompts above 57 and 55 us).
// Blocks of 256 threads go three to an SM, 80 registers a thread; four, with 64, spill: the prompts above
// then 59 and 86 us. Pages of 128 tokens of 128 dims in blocks of 512, one to an SM then 82 us (now 64),
// two 94.
template <int D, bool kInterleaved, bool kE4m3, bool kPlain, bool kTokens, int kPage, int kBlock>
__global__ void __launch_bounds__(kBlock, kBlock == 256 ? 3 : 1)
    paged_append_kernel(const AppendArgs a, const __grid_constant__ RopeTurns turns) {
  pdl_launch_dependents();
  pdl_wait_prior_grid();
  int block = blockIdx.x;
  if constexpr (kPage > 0) {
    // blocks of rows, which memory bounds, and of runs, which instructions do, side by side
    const unsigned all = gridDim.x, rows = a.row_blocks, i = blockIdx.x;
    const unsigned before = (unsigned)((unsigned long long)i * rows / all);
    const bool is_row = (unsigned)((unsigned long long)(i + 1) * rows / all) != before;
    block = is_row ? before : i - before;
    if (!is_row)
      do_runs<D, kInterleaved, kPlain, kBlock, kPage>(a, turns, block);
    else
      do_token_rows<D, kInterleaved, kPlain, false, kBlock>(a, turns, a.Hq, block);
  } else if constexpr (kTokens) {
    do_token_rows<D, kInterleaved, kPlain, true, kBlock>(a, turns, a.Hq + 2 * a.Hkv, block);
  } else {
    do_rows<D, kInterleaved, kE4m3, kBlock>(a, turns, a.Hq + 2 * a.Hkv, block);
  }
}

// ---- gather ---------------------------------------------------------------------------------------
struct GatherArgs {
  const void *k_pages, *v_pages;
  const float *k_scale, *v_scale;
  const int32_t *table, *start, *lens;  // start: may be null (0)
  __nv_bfloat16 *k_out, *v_out;
  uint32_t *error_word;
  int num_pages, page_log2, max_pages, Hkv, rows, rows_per;
};

// One block per (rows_per rows, KV head, sequence): 8 elements a thread at a time, K and V, so that each
// store fills whole sectors (16 elements, two stores of half sectors: 137 us below). A copy that memory
// bounds: 130 us for 32 sequences of 512 .. 8192 tokens in e4m3 (856 MB, 6.6 TB/s), 14.4 for 12.3 k tokens
// of prompts, 2.1 for 512 tokens. Rows of a block, us of the three with 16, 32 and 64: 172, 136, 130; 14.8,
// 14.4, 15.1; 2.1, 2.3, 2.8. Hence as few as kGatherBlocks blocks per SM allow.
constexpr int kGatherBlocks = 32;
template <int D, bool kE4m3>
__global__ void __launch_bounds__(kThreads) paged_gather_kernel(const GatherArgs a) {
  pdl_launch_dependents();
  pdl_wait_prior_grid();
  const int g = blockIdx.x % a.Hkv, r0 = blockIdx.x / a.Hkv * a.rows_per, b = blockIdx.y;
  const long long cap = (long long)a.max_pages << a.page_log2;
  const int len = a.lens[b], from = a.start != nullptr ? a.start[b] : 0;
  const int L = (int)min((long long)max(len, 0), cap), S = max(from, 0);
  if (r0 == 0 && g == 0 && threadIdx.x == 0 && a.error_word != nullptr) {
    if (L != len || (long long)L - S > a.rows) atomicOr(a.error_word, kErrLenClamped);
    if (S != from) atomicOr(a.error_word, kErrPosSkipped);
  }
  const int rows = min(min(L - min(S, L), a.rows) - r0, a.rows_per);
  constexpr int kWords = D / 8;
  const size_t out0 = (((size_t)b * a.Hkv + g) * a.rows + r0) * D;
  for (int k = threadIdx.x; k < rows * kWords; k += kThreads) {
    const int r = k / kWords, c = (k - r * kWords) * 8, t = S + r0 + r;
    const int page = a.table[(size_t)b * a.max_pages + (t >> a.page_log2)];
    if (page < 0 || page >= a.num_pages) {
      if (g == 0 && c == 0 && a.error_word != nullptr) atomicOr(a.error_word, kErrPageSkipped);
      continue;
    }
    const size_t head = (size_t)page * a.Hkv + g;
    const size_t src = ((head << a.page_log2) + (t & ((1 << a.page_log2) - 1))) * D + c;
    uint4 out[2];
    if (kE4m3) {
      const uint2 w[2] = {
          *reinterpret_cast<const uint2 *>(static_cast<const uint8_t *>(a.k_pages) + src),
          *reinterpret_cast<const uint2 *>(static_cast<const uint8_t *>(a.v_pages) + src)};
      const float s[2] = {a.k_scale[head], a.v_scale[head]};
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t x[2] = {w[i].x, w[i].y};
        uint32_t y[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 f = from_e4m3x2(j & 1 ? x[j >> 1] >> 16 : x[j >> 1] & 0xffffu);
          y[j] = pack_bf16x2(f.x * s[i], f.y * s[i]);
        }
        out[i] = make_uint4(y[0], y[1], y[2], y[3]);
      }
    } else {
      out[0] = *reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(a.k_pages) + src);
      out[1] = *reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(a.v_pages) + src);
    }
    *reinterpret_cast<uint4 *>(a.k_out + out0 + (size_t)k * 8) = out[0];
    *reinterpret_cast<uint4 *>(a.v_out + out0 + (size_t)k * 8) = out[1];
  }
}

int log2_of(int x) {
  int l = 0;
  while ((1 << l) < x) ++l;
  return l;
}

}  // namespace

cudaError_t launch_paged_append(const PagedCache &c, const PagedAppend &p, const InvFreq &inv,
                                int sms, cudaStream_t stream) {
  AppendArgs a{};
  a.q_in = static_cast<const __nv_bfloat16 *>(p.q_in);
  a.q_out = static_cast<__nv_bfloat16 *>(p.q_out);
  a.k_new = static_cast<const __nv_bfloat16 *>(p.k_new);
  a.v_new = static_cast<const __nv_bfloat16 *>(p.v_new);
  a.q_norm_w = static_cast<const __nv_bfloat16 *>(p.q_norm_w);
  a.k_norm_w = static_cast<const __nv_bfloat16 *>(p.k_norm_w);
  a.q_ld = p.q_ld, a.qo_ld = p.qo_ld, a.k_ld = p.k_ld, a.v_ld = p.v_ld;
  a.k_pages = c.k_pages, a.v_pages = c.v_pages;
  a.k_scale = c.k_scale, a.v_scale = c.v_scale;
  a.table = c.table, a.start = p.start, a.cu_new = p.cu_new;
  a.error_word = p.error_word;
  a.n = p.n, a.B = p.B;
  a.num_pages = c.num_pages, a.page_log2 = log2_of(c.page), a.max_pages = c.max_pages;
  a.Hq = p.Hq, a.Hkv = c.Hkv, a.rot = p.rot_dim, a.eps = p.eps;
  const bool runs = c.e4m3 && p.cu_new != nullptr;
  // (a page of 128 tokens of 128 dims is 512 threads' work)
  const int block = runs && c.page * (c.D / 16) > 512 ? 512 : 256;
  const int heads = runs ? p.Hq : p.Hq + 2 * c.Hkv, rows = block / (c.D / 16);
  const int enough = kBlocksPerSm * sms * 256 / block;
  // Tokens side by side: as many as there are, up to a block's rows. Heads one after the other: the
  // more, the fewer angles are formed twice; as few as it takes for enough blocks.
  a.tok_par = 1;
  while (a.tok_par < rows && (runs || a.tok_par < p.n)) a.tok_par *= 2;
  const long long tiles = ((long long)p.n + a.tok_par - 1) / a.tok_par;
  const int side = rows / a.tok_par;
  a.heads_per = side;
  while (a.heads_per < heads &&
         tiles * ((heads + 2 * a.heads_per - 1) / (2 * a.heads_per)) >= enough)
    a.heads_per *= 2;
  a.head_blocks = (heads + a.heads_per - 1) / a.heads_per;
  a.row_blocks = (int)(tiles * a.head_blocks);
  const int chunk = c.page > 64 ? c.page : 64;
  const long long chunks = ((long long)p.n + chunk - 1) / chunk;
  a.run_heads = 1;
  while (a.run_heads < c.Hkv &&
         chunks * ((2 * c.Hkv + 2 * a.run_heads - 1) / (2 * a.run_heads)) >= enough)
    a.run_heads *= 2;
  a.run_blocks = (2 * c.Hkv + a.run_heads - 1) / a.run_heads;
  const long long blocks = a.row_blocks + (runs ? chunks * a.run_blocks : 0);
  // the rows on their way; of runs also the angles of the pages that a block has under way at a time
  const size_t ahead = (size_t)block * 32;
  const int passes = passes_of(c.D, c.page);
  const size_t tables = (size_t)block * passes / (c.D / 16) * c.D * 4;
  const size_t smem = runs ? std::max(tables + passes * ahead, (kHeadsAhead + 1) * ahead)
                      : !c.e4m3 && side == 1 ? (kHeadsAhead + 1) * ahead : 0;
  const RopeTurns turns = make_rope_turns(p.rot_dim, inv);
  auto go = [&](auto dim, auto layout, auto all_turned) {
    constexpr int kD = decltype(dim)::value;
    constexpr bool kI = decltype(layout)::value, kP = decltype(all_turned)::value;
    constexpr int kLarge = kD == 128 ? 512 : 256;
    auto *kernel = runs ? (c.page == 16   ? paged_append_kernel<kD, kI, true, kP, true, 16, 256>
                           : c.page == 32 ? paged_append_kernel<kD, kI, true, kP, true, 32, 256>
                           : c.page == 64 ? paged_append_kernel<kD, kI, true, kP, true, 64, 256>
                                          : paged_append_kernel<kD, kI, true, kP, true, 128, kLarge>)
                   : c.e4m3 ? paged_append_kernel<kD, kI, true, false, false, 0, 256>
                   : side == 1 ? paged_append_kernel<kD, kI, false, kP, true, 0, 256>
                               : paged_append_kernel<kD, kI, false, false, false, 0, 256>;
    if (smem > 32 * 1024) {  // (48 KB with what the kernels declare needs no leave)
      const cudaError_t e =
          cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
      if (e != cudaSuccess) return e;
    }
    return launch_pdl(kernel, dim3((unsigned)blocks), block, smem, stream, a, turns);
  };
  using I64 = std::integral_constant<int, 64>;
  using I128 = std::integral_constant<int, 128>;
  const bool plain = p.k_norm_w == nullptr && p.rot_dim == c.D;
  auto with = [&](auto dim, auto layout) {
    return plain ? go(dim, layout, std::true_type{}) : go(dim, layout, std::false_type{});
  };
  const cudaError_t e = c.D == 128 ? (p.interleaved ? with(I128{}, std::true_type{})
                                                    : with(I128{}, std::false_type{}))
                                   : (p.interleaved ? with(I64{}, std::true_type{})
                                                    : with(I64{}, std::false_type{}));
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_paged_gather(const PagedCache &c, const int32_t *start, const int32_t *lens,
                                void *k_out, void *v_out, int B, int rows, uint32_t *error_word,
                                int sms, cudaStream_t stream) {
  int per = 16;
  auto blocks = [&]() { return ((long long)(rows - 1) / per + 1) * c.Hkv; };
  while (per < 64 && blocks() * B > (long long)kGatherBlocks * sms) per *= 2;
  const GatherArgs a{c.k_pages, c.v_pages, c.k_scale, c.v_scale, c.table, start, lens,
                     static_cast<__nv_bfloat16 *>(k_out), static_cast<__nv_bfloat16 *>(v_out),
                     error_word, c.num_pages, log2_of(c.page), c.max_pages, c.Hkv, rows, per};
  const dim3 grid((unsigned)blocks(), B);
  auto *kernel = c.D == 128 ? (c.e4m3 ? paged_gather_kernel<128, true> : paged_gather_kernel<128, false>)
                            : (c.e4m3 ? paged_gather_kernel<64, true> : paged_gather_kernel<64, false>);
  const cudaError_t e = launch_pdl(kernel, grid, kThreads, 0, stream, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace decattn
