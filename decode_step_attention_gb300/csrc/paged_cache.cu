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
// first rot_dim elements of a head rotated.
#include <cuda_fp8.h>

#include <type_traits>

#include "dec_device.cuh"
#include "dec_launch.h"
#include "rope_angles.cuh"

namespace decattn {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
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
// x / s, exact when s is a power of two.
struct Unscale {
  float s, inv;
  bool pow2;
  __device__ explicit Unscale(float scale) {
    s = scale;
    inv = 1.f / scale;
    pow2 = (__float_as_uint(scale) & 0x7fffffu) == 0;
  }
  __device__ float operator()(float x) const { return pow2 ? x * inv : x / s; }
};

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
  // tokens and heads of a block of rows; the blocks of them, and the tokens of a block of runs
  int tok_par, heads_per, row_blocks, head_blocks, chunk;
};

// Where token i goes: its sequence, its position, and the page's number (-1: nowhere).
struct Place {
  int b, pos, page;
  long long end;  // the first token behind the sequence's
};
__device__ __forceinline__ Place place_of(const AppendArgs &a, int i) {
  Place p;
  long long first = i;
  p.end = i + 1;
  if (a.cu_new == nullptr) {
    p.b = i;
  } else {
    int lo = 0, hi = a.B;  // cu_new[lo] <= i < cu_new[hi] where cu_new is in order
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (a.cu_new[mid] <= i) lo = mid; else hi = mid;
    }
    p.b = lo;
    first = a.cu_new[lo];
    p.end = min(a.cu_new[lo + 1], a.n);
    if (first > i || p.end <= i) p.b = -1;  // a token of no sequence
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

// One row of q or k in a lane's registers: normed and rotated.
template <int D, bool kInterleaved>
struct Turned {
  float u[8], v[8];    // the result
  float rstd;
  uint4 x, y;          // as loaded
};

template <int D, bool kInterleaved>
__device__ __forceinline__ void turn(Turned<D, kInterleaved> &t, bool norm, uint4 wa, uint4 wb,
                                     float eps, bool rotated, const float (&cs)[8],
                                     const float (&sn)[8]) {
  using R = Row<D, kInterleaved>;
  R::unpack(t.x, t.y, t.u, t.v);
  t.rstd = 1.f;
  if (norm) {
    float su = 0.f, sv = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      su = fmaf(t.u[j], t.u[j], su);
      sv = fmaf(t.v[j], t.v[j], sv);
    }
    su += sv;
#pragma unroll
    for (int o = R::kLanes / 2; o > 0; o >>= 1) su += __shfl_xor_sync(0xffffffffu, su, o);
    t.rstd = rsqrtf(su * (1.0f / (float)D) + eps);
    float p[8], q[8];
    R::unpack(wa, wb, p, q);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      t.u[j] = t.u[j] * t.rstd * p[j];
      t.v[j] = t.v[j] * t.rstd * q[j];
    }
  }
  if (rotated) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float p = t.u[j], q = t.v[j];
      t.u[j] = rope_first(p, q, cs[j], sn[j]);
      t.v[j] = rope_second<false>(p, q, cs[j], sn[j]);
    }
  }
}

// One element of a rotated pair (or one that is not rotated), before the norm's scale, in fp64.
__device__ __noinline__ double exact_element(int pos, unsigned long long turns, float own,
                                             float other, bool second, bool rotated) {
  return rotated ? rope_element_turns(pos, turns, own, other, second) : (double)own;
}

// Elements of a key whose fp32 value does not settle the stored one (bits of this lane's 16: u, then
// v), again in fp64 from the stored inputs: u and v get convert(value). The warp comes together; rare.
template <int D, bool kInterleaved, typename Convert>
__device__ __forceinline__ void exact_elements(const Turned<D, kInterleaved> &t, uint4 wa, uint4 wb,
                                               bool norm, float eps, bool rotated, int pos, int l,
                                               const unsigned long long *turns, unsigned bits,
                                               float (&u)[8], float (&v)[8], Convert convert) {
  using R = Row<D, kInterleaved>;
  if (!__any_sync(0xffffffffu, bits != 0)) return;
  float x[8], y[8];
  R::unpack(t.x, t.y, x, y);
  double rstd = 1.0;
  if (norm) {  // (the same for the whole warp)
    double ss = 0.0;
#pragma unroll
    for (int j = 0; j < 8; ++j) ss = fma((double)x[j], (double)x[j], fma((double)y[j], (double)y[j], ss));
#pragma unroll
    for (int o = R::kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    rstd = 1.0 / sqrt(ss / D + (double)eps);
    float p[8], q[8];
    R::unpack(wa, wb, p, q);
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] *= p[j], y[j] *= q[j];  // (exact products of two bf16)
  }
  do {
    if (bits != 0) {
      const int i = __ffs(bits) - 1;
      bits &= bits - 1;
      float first = 0.f, other = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if ((i & 7) == j) first = x[j], other = y[j];
      const bool second = i >= 8;
      const float z = convert(exact_element(pos, turns[8 * l + (i & 7)], second ? other : first,
                                            second ? first : other, second, rotated) *
                              rstd);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (i == j) u[j] = z;
        if (i == 8 + j) v[j] = z;
      }
    }
  } while (__any_sync(0xffffffffu, bits != 0));
}

// A double as the float that e4m3's rounding takes the same way: what is cut off leaves its mark in
// the last bit.
__device__ __forceinline__ float sticky(double x) {
  const float f = __double2float_rz(x);
  return (double)f == x ? f : __uint_as_float(__float_as_uint(f) | 1u);
}

// How far fp32 may have moved a value of a row that was normed or rotated: a few 2^-24 of its terms.
constexpr float kSlack = 0x1p-20f;

// The codes of a lane's 16 values. Where a warp has keys that were normed or rotated (inexact, norm:
// the same for the whole warp), a value of one (key) so near a border between two codes that the fp32
// arithmetic before it could have moved it across is formed again in fp64: the codes are the
// exact key's.
template <int D, bool kInterleaved>
__device__ __forceinline__ void encode(const Turned<D, kInterleaved> &t, const Unscale &un,
                                       uint4 wa, uint4 wb, bool inexact, bool norm, float eps,
                                       bool rotated, int pos, int l,
                                       const unsigned long long *turns, bool key, uint2 &a,
                                       uint2 &b) {
  using R = Row<D, kInterleaved>;
  float u[8], v[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) u[j] = un(t.u[j]), v[j] = un(t.v[j]);
  if (inexact) {
    unsigned bits = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float d = kSlack * (fabsf(u[j]) + fabsf(v[j]));
      const uint32_t off = e4m3x2(u[j] - d, v[j] - d) ^ e4m3x2(u[j] + d, v[j] + d);
      // (-0 and +0 are no border, but counting them as one costs nothing)
      bits |= (off & 0xffu ? 1u << j : 0u) | (off & 0xff00u ? 0x100u << j : 0u);
    }
    exact_elements<D, kInterleaved>(
        t, wa, wb, norm, eps, rotated, pos, l, turns, key ? bits : 0u, u, v,
        [&](double value) { return sticky(value / (double)un.s); });
  }
  float f[16];
  R::order(u, v, f);
  a = make_uint2(e4m3x2(f[0], f[1]) | e4m3x2(f[2], f[3]) << 16,
                 e4m3x2(f[4], f[5]) | e4m3x2(f[6], f[7]) << 16);
  b = make_uint2(e4m3x2(f[8], f[9]) | e4m3x2(f[10], f[11]) << 16,
                 e4m3x2(f[12], f[13]) | e4m3x2(f[14], f[15]) << 16);
}

template <int D, bool kInterleaved>
__device__ __forceinline__ float amax_of(const Turned<D, kInterleaved> &t) {
  float m = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) m = fmaxf(m, fmaxf(finite_abs(t.u[j]), finite_abs(t.v[j])));
  return m;
}

// ---- rows: (token, head) pairs that need nothing of each other ------------------------------
// Heads are counted q, k, v. A block has tok_par tokens side by side, times as many heads as fit,
// and goes through its heads_per heads with them: a lane keeps its token's angles.
template <int D, bool kInterleaved, bool kE4m3>
__device__ void do_rows(const AppendArgs &a, const RopeTurns &turns, int heads) {
  using R = Row<D, kInterleaved>;
  constexpr int kRows = kThreads / R::kLanes;
  const int lane = threadIdx.x & 31, l = lane % R::kLanes, row = threadIdx.x / R::kLanes;
  const int block = blockIdx.x % a.head_blocks, tile = blockIdx.x / a.head_blocks;
  const int i = tile * a.tok_par + (row & (a.tok_par - 1));
  const int step = kRows / a.tok_par;
  const int h0 = block * a.heads_per, h1 = min(heads, h0 + a.heads_per);
  Place at{};
  at.b = at.pos = at.page = -1;
  if (i < a.n) at = place_of(a, i);
  const bool some = at.pos >= 0;
  const bool rotated = l < (a.rot >> 4), norm = a.q_norm_w != nullptr;
  int ea, eb;
  R::places(l, a.rot, ea, eb);
  float cs[8], sn[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    cs[j] = 1.f;
    sn[j] = 0.f;
    if (rotated && some) rope_sincos_turns(at.pos, turns.v[8 * l + j], sn[j], cs[j]);
  }
  uint4 wqa{}, wqb{}, wka{}, wkb{};
  if (norm) {
    wqa = *reinterpret_cast<const uint4 *>(a.q_norm_w + ea);
    wqb = *reinterpret_cast<const uint4 *>(a.q_norm_w + eb);
    wka = *reinterpret_cast<const uint4 *>(a.k_norm_w + ea);
    wkb = *reinterpret_cast<const uint4 *>(a.k_norm_w + eb);
  }
  const int in_page = at.pos & ((1 << a.page_log2) - 1);
  for (int hh = h0; hh < h1; hh += step) {  // (the same number of times in every lane)
    const int h = hh + row / a.tok_par;
    const bool is_q = h < a.Hq, is_k = !is_q && h < a.Hq + a.Hkv;
    const int g = is_q ? h : is_k ? h - a.Hq : h - a.Hq - a.Hkv;
    const bool live = some && h < h1 && (is_q || at.page >= 0);
    Turned<D, kInterleaved> t;
    t.x = t.y = make_uint4(0u, 0u, 0u, 0u);
    if (live) {
      const __nv_bfloat16 *src = is_q   ? a.q_in + i * a.q_ld
                                 : is_k ? a.k_new + i * a.k_ld
                                        : a.v_new + i * a.v_ld;
      src += (size_t)g * D;
      t.x = *reinterpret_cast<const uint4 *>(src + ea);
      t.y = *reinterpret_cast<const uint4 *>(src + eb);
    }
    const bool turns_here = is_q || is_k;
    const uint4 wa = is_q ? wqa : wka, wb = is_q ? wqb : wkb;
    if (turns_here || norm) {  // (a warp may hold values beside keys: the norm's shuffles)
      turn(t, norm, wa, wb, a.eps, rotated, cs, sn);
    }
    if (!turns_here) R::unpack(t.x, t.y, t.u, t.v);
    const size_t slot =
        live && !is_q
            ? ((((size_t)at.page * a.Hkv + g) << a.page_log2) + (size_t)in_page) * D
            : 0;
    if (kE4m3) {
      float m = amax_of(t);
#pragma unroll
      for (int o = R::kLanes / 2; o > 0; o >>= 1)
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      float scale = scale_for(m), old = scale;
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
      uint2 ca, cb;
      encode<D, kInterleaved>(t, Unscale(scale), wka, wkb, norm || a.rot > 0, norm, a.eps, rotated,
                              at.pos, l, turns.v, live && is_k, ca, cb);
      if (live && !is_q) {
        uint8_t *dst = static_cast<uint8_t *>(is_k ? a.k_pages : a.v_pages) + slot;
        *reinterpret_cast<uint2 *>(dst + ea) = ca;
        *reinterpret_cast<uint2 *>(dst + eb) = cb;
      }
    } else if (__any_sync(0xffffffffu, live && is_k)) {
      // keys within one bf16 step where the rotation cancels
      float u[8], v[8];
      R::unpack(t.x, t.y, u, v);
      unsigned bits = 0;
      if (live && is_k && rotated) {
        float p[8], q[8];
        R::unpack(wka, wkb, p, q);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float x = norm ? u[j] * t.rstd * p[j] : u[j];
          const float y = norm ? v[j] * t.rstd * q[j] : v[j];
          bits |= (rope_cancels(t.u[j], x, y) ? 1u << j : 0u) |
                  (rope_cancels(t.v[j], x, y) ? 0x100u << j : 0u);
        }
      }
      exact_elements<D, kInterleaved>(t, wka, wkb, norm, a.eps, rotated, at.pos, l, turns.v, bits,
                                      t.u, t.v, [](double value) { return (float)value; });
    }
    if (live && (is_q || !kE4m3)) {
      float f[16];
      R::order(t.u, t.v, f);
      uint4 oa = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                            pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
      uint4 ob = make_uint4(pack_bf16x2(f[8], f[9]), pack_bf16x2(f[10], f[11]),
                            pack_bf16x2(f[12], f[13]), pack_bf16x2(f[14], f[15]));
      if (!turns_here) oa = t.x, ob = t.y;  // a copy, bit for bit
      __nv_bfloat16 *dst = is_q ? a.q_out + i * a.qo_ld + (size_t)g * D
                                : static_cast<__nv_bfloat16 *>(is_k ? a.k_pages : a.v_pages) + slot;
      *reinterpret_cast<uint4 *>(dst + ea) = oa;
      *reinterpret_cast<uint4 *>(dst + eb) = ob;
    }
  }
}

// ---- runs: the new tokens of one page under one scale ------------------------------------------
struct Run {
  int token, pos, page, count;
};

// One run of one KV head, by a warp (kGroup = 32, up to 4 * kRows tokens) or the block.
template <int D, bool kInterleaved, int kGroup>
__device__ __forceinline__ void do_run(const AppendArgs &a, const RopeTurns &turns, const Run &r,
                                       bool is_k, int g, uint4 wa, uint4 wb, float *s_max) {
  using R = Row<D, kInterleaved>;
  constexpr int kRows = kGroup / R::kLanes;   // tokens side by side
  constexpr int kPasses = kGroup == 32 ? 4 : 128 / kRows;
  const int in_group = threadIdx.x & (kGroup - 1);
  const int lane = threadIdx.x & 31, l = lane % R::kLanes, row = in_group / R::kLanes;
  const bool rotated = is_k && l < (a.rot >> 4), norm = is_k && a.k_norm_w != nullptr;
  int ea, eb;
  R::places(l, a.rot, ea, eb);
  const __nv_bfloat16 *src = (is_k ? a.k_new : a.v_new) + (size_t)g * D;
  const long long ld = is_k ? a.k_ld : a.v_ld;
  Turned<D, kInterleaved> t[kPasses];
  float m = 0.f;
#pragma unroll
  for (int p = 0; p < kPasses; ++p) {
    const int j = p * kRows + row;
    t[p].x = t[p].y = make_uint4(0u, 0u, 0u, 0u);
    if (j < r.count) {
      t[p].x = *reinterpret_cast<const uint4 *>(src + (r.token + j) * ld + ea);
      t[p].y = *reinterpret_cast<const uint4 *>(src + (r.token + j) * ld + eb);
    }
  }
#pragma unroll
  for (int p = 0; p < kPasses; ++p) {
    if (p * kRows >= r.count) break;  // (the same for the whole group)
    float cs[8], sn[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      cs[j] = 1.f;
      sn[j] = 0.f;
      if (rotated) rope_sincos_turns(r.pos + p * kRows + row, turns.v[8 * l + j], sn[j], cs[j]);
    }
    turn(t[p], norm, wa, wb, a.eps, rotated, cs, sn);
    m = fmaxf(m, amax_of(t[p]));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (kGroup > 32) {
    __syncthreads();  // the last run's maxima have been read
    if (lane == 0) s_max[threadIdx.x >> 5] = m;
    __syncthreads();
    m = s_max[0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) m = fmaxf(m, s_max[w]);
  }
  const int in_page = r.pos & ((1 << a.page_log2) - 1);
  float *sp = (is_k ? a.k_scale : a.v_scale) + (size_t)r.page * a.Hkv + g;
  uint8_t *base = static_cast<uint8_t *>(is_k ? a.k_pages : a.v_pages) +
                  (((size_t)r.page * a.Hkv + g) << a.page_log2) * D;
  float scale = scale_for(m), old = scale;
  if (in_page > 0) {
    old = *sp;
    scale = fmaxf(scale, old);
  }
  if (kGroup > 32) __syncthreads(); else __syncwarp();  // everyone has read the scale
  if (in_group == 0 && (scale > old || in_page == 0)) *sp = scale;
  if (scale > old) {
    const float ratio = old / scale;
    uint4 *w = reinterpret_cast<uint4 *>(base);
#pragma unroll 4
    for (int k = in_group; k < in_page * (D / 16); k += kGroup) w[k] = rescale16(w[k], ratio);
  }
  const Unscale un(scale);
#pragma unroll
  for (int p = 0; p < kPasses; ++p) {
    const int j = p * kRows + row;
    if (p * kRows >= r.count) break;
    uint2 ca, cb;
    encode<D, kInterleaved>(t[p], un, wa, wb, is_k && (norm || a.rot > 0), norm, a.eps, rotated,
                            r.pos + j, l, turns.v, is_k && j < r.count, ca, cb);
    if (j < r.count) {
      uint8_t *dst = base + (size_t)(in_page + j) * D;
      *reinterpret_cast<uint2 *>(dst + ea) = ca;
      *reinterpret_cast<uint2 *>(dst + eb) = cb;
    }
  }
}

// The runs that begin among a block's `chunk` tokens, for one KV head's keys or values.
template <int D, bool kInterleaved>
__device__ void do_runs(const AppendArgs &a, const RopeTurns &turns, int block) {
  using R = Row<D, kInterleaved>;
  __shared__ Run s_run[128];
  __shared__ int s_short, s_long;
  __shared__ float s_max[kWarps];
  constexpr int kWarpRun = 4 * 32 / R::kLanes;  // tokens that a warp takes at once
  const int head = block % (2 * a.Hkv), c0 = block / (2 * a.Hkv) * a.chunk;
  const bool is_k = head < a.Hkv;
  const int g = is_k ? head : head - a.Hkv;
  if (threadIdx.x == 0) s_short = s_long = 0;
  __syncthreads();
  const int i = c0 + threadIdx.x;
  if ((int)threadIdx.x < a.chunk && i < a.n) {
    const Place p = place_of(a, i);
    const int page = 1 << a.page_log2;
    const bool begins = p.b >= 0 && (i == a.cu_new[p.b] || (p.pos & (page - 1)) == 0);
    if (begins && p.page >= 0) {
      const int count = (int)min(p.end - i, (long long)(page - (p.pos & (page - 1))));
      // short ones from the front of the list, long ones from its back
      const int k = count <= kWarpRun ? atomicAdd(&s_short, 1) : 127 - atomicAdd(&s_long, 1);
      s_run[k] = Run{i, p.pos, p.page, count};
    }
  }
  __syncthreads();
  uint4 wa{}, wb{};
  if (is_k && a.k_norm_w != nullptr) {
    int ea, eb;
    R::places((threadIdx.x & 31) % R::kLanes, a.rot, ea, eb);
    wa = *reinterpret_cast<const uint4 *>(a.k_norm_w + ea);
    wb = *reinterpret_cast<const uint4 *>(a.k_norm_w + eb);
  }
  const int shorts = s_short, longs = s_long;
  for (int k = threadIdx.x >> 5; k < shorts; k += kWarps)
    do_run<D, kInterleaved, 32>(a, turns, s_run[k], is_k, g, wa, wb, s_max);
  for (int k = 0; k < longs; ++k)
    do_run<D, kInterleaved, kThreads>(a, turns, s_run[127 - k], is_k, g, wa, wb, s_max);
}

// The first row_blocks blocks take rows: the queries, and keys and values too unless kRuns.
template <int D, bool kInterleaved, bool kE4m3, bool kRuns>
__global__ void __launch_bounds__(kThreads)
    paged_append_kernel(const AppendArgs a, const __grid_constant__ RopeTurns turns) {
  pdl_launch_dependents();
  pdl_wait_prior_grid();
  if constexpr (kRuns) {
    if ((int)blockIdx.x >= a.row_blocks) {
      do_runs<D, kInterleaved>(a, turns, blockIdx.x - a.row_blocks);
      return;
    }
    do_rows<D, kInterleaved, false>(a, turns, a.Hq);
  } else {
    do_rows<D, kInterleaved, kE4m3>(a, turns, a.Hq + 2 * a.Hkv);
  }
}

// ---- gather ---------------------------------------------------------------------------------------
struct GatherArgs {
  const void *k_pages, *v_pages;
  const float *k_scale, *v_scale;
  const int32_t *table, *start, *lens;  // start: may be null (0)
  __nv_bfloat16 *k_out, *v_out;
  uint32_t *error_word;
  int num_pages, page_log2, max_pages, Hkv, rows;
};

constexpr int kGatherRows = 64;

// One block per (64 rows, KV head, sequence): 16 elements a thread at a time, K and V.
template <int D, bool kE4m3>
__global__ void __launch_bounds__(kThreads) paged_gather_kernel(const GatherArgs a) {
  pdl_launch_dependents();
  pdl_wait_prior_grid();
  const int g = blockIdx.x % a.Hkv, r0 = blockIdx.x / a.Hkv * kGatherRows, b = blockIdx.y;
  const long long cap = (long long)a.max_pages << a.page_log2;
  const int len = a.lens[b], from = a.start != nullptr ? a.start[b] : 0;
  const int L = (int)min((long long)max(len, 0), cap), S = max(from, 0);
  if (r0 == 0 && g == 0 && threadIdx.x == 0 && a.error_word != nullptr) {
    if (L != len || (long long)L - S > a.rows) atomicOr(a.error_word, kErrLenClamped);
    if (S != from) atomicOr(a.error_word, kErrPosSkipped);
  }
  const int rows = min(min(L - min(S, L), a.rows) - r0, kGatherRows);
  constexpr int kWords = D / 16;
  const size_t out0 = (((size_t)b * a.Hkv + g) * a.rows + r0) * D;
  for (int k = threadIdx.x; k < rows * kWords; k += kThreads) {
    const int r = k / kWords, c = (k - r * kWords) * 16, t = S + r0 + r;
    const int page = a.table[(size_t)b * a.max_pages + (t >> a.page_log2)];
    if (page < 0 || page >= a.num_pages) {
      if (g == 0 && c == 0 && a.error_word != nullptr) atomicOr(a.error_word, kErrPageSkipped);
      continue;
    }
    const size_t head = (size_t)page * a.Hkv + g;
    const size_t src = ((head << a.page_log2) + (t & ((1 << a.page_log2) - 1))) * D + c;
    uint4 out[2][2];
    if (kE4m3) {
      const uint4 w[2] = {
          *reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(a.k_pages) + src),
          *reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(a.v_pages) + src)};
      const float s[2] = {a.k_scale[head], a.v_scale[head]};
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t x[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
        uint32_t y[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float2 f = from_e4m3x2(j & 1 ? x[j >> 1] >> 16 : x[j >> 1] & 0xffffu);
          y[j] = pack_bf16x2(f.x * s[i], f.y * s[i]);
        }
        out[i][0] = make_uint4(y[0], y[1], y[2], y[3]);
        out[i][1] = make_uint4(y[4], y[5], y[6], y[7]);
      }
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        out[0][h] =
            reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(a.k_pages) + src)[h];
        out[1][h] =
            reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(a.v_pages) + src)[h];
      }
    }
    uint4 *ko = reinterpret_cast<uint4 *>(a.k_out + out0 + (size_t)r * D + c);
    uint4 *vo = reinterpret_cast<uint4 *>(a.v_out + out0 + (size_t)r * D + c);
    ko[0] = out[0][0], ko[1] = out[0][1];
    vo[0] = out[1][0], vo[1] = out[1][1];
  }
}

int log2_of(int x) {
  int l = 0;
  while ((1 << l) < x) ++l;
  return l;
}

}  // namespace

cudaError_t launch_paged_append(const PagedCache &c, const PagedAppend &p, const InvFreq &inv,
                                cudaStream_t stream) {
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
  const int heads = runs ? p.Hq : p.Hq + 2 * c.Hkv, rows = kThreads / (c.D / 16);
  int sms = 152, dev = 0;
  if (cudaGetDevice(&dev) == cudaSuccess)
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  // Tokens side by side: as many as there are, up to a block's rows. Heads one after the other: the
  // more, the fewer angles are formed twice; as few as it takes for two blocks per SM.
  a.tok_par = 1;
  while (a.tok_par < rows && a.tok_par < p.n) a.tok_par *= 2;
  const long long tiles = ((long long)p.n + a.tok_par - 1) / a.tok_par;
  const int side = rows / a.tok_par;
  a.heads_per = side;
  while (a.heads_per < heads && tiles * ((heads + 2 * a.heads_per - 1) / (2 * a.heads_per)) >= 2 * sms)
    a.heads_per *= 2;
  a.head_blocks = (heads + a.heads_per - 1) / a.heads_per;
  a.row_blocks = (int)(tiles * a.head_blocks);
  a.chunk = c.page > 64 ? c.page : 64;
  const long long blocks =
      a.row_blocks +
      (runs ? ((long long)p.n + a.chunk - 1) / a.chunk * 2 * c.Hkv : 0);
  const RopeTurns turns = make_rope_turns(p.rot_dim, inv);
  auto go = [&](auto dim, auto layout) {
    constexpr int kD = decltype(dim)::value;
    constexpr bool kI = decltype(layout)::value;
    auto *kernel = runs     ? paged_append_kernel<kD, kI, true, true>
                   : c.e4m3 ? paged_append_kernel<kD, kI, true, false>
                            : paged_append_kernel<kD, kI, false, false>;
    return launch_pdl(kernel, dim3((unsigned)blocks), kThreads, 0, stream, a, turns);
  };
  using I64 = std::integral_constant<int, 64>;
  using I128 = std::integral_constant<int, 128>;
  const cudaError_t e = c.D == 128 ? (p.interleaved ? go(I128{}, std::true_type{})
                                                    : go(I128{}, std::false_type{}))
                                   : (p.interleaved ? go(I64{}, std::true_type{})
                                                    : go(I64{}, std::false_type{}));
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_paged_gather(const PagedCache &c, const int32_t *start, const int32_t *lens,
                                void *k_out, void *v_out, int B, int rows, uint32_t *error_word,
                                cudaStream_t stream) {
  const GatherArgs a{c.k_pages, c.v_pages, c.k_scale, c.v_scale, c.table, start, lens,
                     static_cast<__nv_bfloat16 *>(k_out), static_cast<__nv_bfloat16 *>(v_out),
                     error_word, c.num_pages, log2_of(c.page), c.max_pages, c.Hkv, rows};
  const dim3 grid((unsigned)((rows + kGatherRows - 1) / kGatherRows * c.Hkv), B);
  auto *kernel = c.D == 128 ? (c.e4m3 ? paged_gather_kernel<128, true> : paged_gather_kernel<128, false>)
                            : (c.e4m3 ? paged_gather_kernel<64, true> : paged_gather_kernel<64, false>);
  const cudaError_t e = launch_pdl(kernel, grid, kThreads, 0, stream, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace decattn
