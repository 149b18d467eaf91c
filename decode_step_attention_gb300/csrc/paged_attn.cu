// Single-query GQA attention over a paged cache of bf16 values or e4m3 codes with a scale per
// (page, KV head), on the 5th-generation tensor cores:
//
//   z[h, t]   = scale q[b,h] . K_t = (scale s_q s_k) (q' . c_t)      c: codes, q = s_q q'
//   out[b,h]  = sum_t softmax_t(z) V_t over the last `window` tokens (all without one)
//
// Tokens are the M of the instructions, query heads the N: S^T[128 tokens, heads] = K Q^T takes a tile
// of keys as it lies in shared memory, codes included, and O^T[D, heads] = V^T P^T the values likewise
// (tokens x dims: the MN-major operand). No code is ever converted. N is 16, twice the 8 heads
// of a group, which gives each query and each weight two terms:
//   e4m3   q' = hi + lo / 16, both e4m3. bf16 has 8 significant bits and e4m3 4 (and a sign), so
//          the sum is exact but for elements below 2^-14 of their head's largest. A weight
//          p = hi + lo / 16 is within 2^-8 of itself.
//   bf16   p = hi + lo, both bf16 (the second half of Q's rows is zero).
// The weights' size is what e4m3 has little room for (2^-9 .. 448): each of four warps takes those of its
// tokens (32 of a tile of 128, 64 of one of 256) relative to a base of its own, which is 2^8 and stays
// from tile to tile while the largest weight lies within 2^2 .. 2^8.5, and has columns of its own in the
// product, which are joined in fp32 with the running maximum. A value's scale is part of its weight: with
// t = z + log2(s_v), the weight is 2^(8 + t - base) and its share of the softmax sum that over s_v.
// (Scores beyond 2^10, where fp32 no longer holds such sums closely, are taken apart from log2(s_v): see
// the warps of weights.)
//
// The tiles (128 tokens; 256 of 64 dims in e4m3) of all (sequence, KV head) pairs form one stream, cut
// into equal pieces, one per CTA (two CTAs per SM; one for bf16 rows of 128 dims, whose ring takes
// the shared memory). A pair that lies in several pieces leaves a partial in each (O, maximum, sum,
// fp32); the CTA that delivers a pair's last partial joins them when its own piece is done, in the
// order of the pieces, so that results do not depend on who that is. Counters are indexed by the piece
// in which a pair begins (one at most goes on from a piece), not by the pair, so that they lie in the
// same place for every shape and a workspace may serve several.
//
// Inside a CTA a tile goes through, each a step behind the other:
//   warp 8       page numbers (a batch ahead), the pages' K and V boxes by TMA into a ring of shared
//                memory, their scales beside them (cp.async), a descriptor per tile
//   warp 9       each segment's queries as the B operand, a segment ahead
//   warp 10      S^T into one of two buffers of tensor memory
//   warps 0-3    a token per thread: scores, weights, their sums
//   warp 11      the value product of the 32 tokens of each of these warps
//   warps 4-7    a dimension per thread: the running O, and a segment's end
//
// Pages that end inside a tile, windows and lengths cost nothing but the rows they leave unused: only
// pages with a token that is seen are copied, and rows of V that are not seen are cleared.
//
// What bounds it, and what it measured (us as a user's call with a workspace of its own; GB/s of K and V
// read; a plain copy moves 6687 GB/s):
//   256 ragged sequences (539 MB), 4 KV heads of 128, e4m3         88   6.1 TB/s   memory, and that
//                                                    equal pieces take the SMs 10-15% unequal times
//   32 sequences of 512 .. 8192 tokens, 8 KV heads of 128, bf16    91   6.3 TB/s   the same
//   131072 tokens of one sequence, 8 KV heads of 128, e4m3         48   5.5 TB/s   start and joining
//   192 windows of 4095 tokens, 2 KV heads of 64, e4m3             38   4.5 TB/s   start (a third),
//                                                    then the instructions of the weights
//   512 tokens, 8 KV heads of 128, e4m3                            11              the call (8 on the GPU)
// The steps that led here (the serving mix): one CTA per SM 168, two 124, weights relative to a base
// that stays while it is near 92, partials joined from bulk copies 90, a segment as one tile 87, bases
// of two terms for far scores 88. A kernel of plain loads and fp32 sums took 2126.
#include <cuda_fp8.h>
#include <limits.h>
#include <math.h>

#include <algorithm>
#include <atomic>
#include <type_traits>
#include <utility>

#include "dec_device.cuh"
#include "dec_launch.h"
#include "tcgen05.cuh"

namespace decattn {
namespace {

constexpr int kG = kSplitMaxG;
constexpr int kN = 16;       // columns of the products: two terms of each of up to 8 heads
constexpr int kThreads = 384;
constexpr int kTma = 8, kQuery = 9, kScore = 10, kValue = 11;  // warps
constexpr uint32_t kTmemCols = 256;
constexpr uint32_t kOCols = 4 * kN;       // an O buffer: 16 columns for each warp of tokens
// What beginning and ending a segment costs, in tiles: the stream is cut by tiles plus this, unless
// there are fewer than kFew tiles per piece. (256 ragged sequences, us on the GPU with 0, 1, 2, 3 and 5:
// 88.4, 88.0, 90.6, 92.7, 97.8; 192 windows of 64 dims 38.8, 38.3, 38.5, 39.2, 40.1; 32 sequences in bf16
// 90.8, 91.1, 90.3, 90.1, 91.2. kFew of 0, 1, 2, 4, 8 and 16: 8 sequences of 2048 tokens, 8 KV heads, 12.8,
// 12.9, 12.9, 12.6, 12.6, 12.6; 8 of 8192 27.0, 27.0, 27.0, 27.0, 27.1, 27.6.)
constexpr int kSegment = 1, kFew = 4;
// Weights are taken relative to a base. Up to this size of it (in powers of two) fp32 holds the base, the
// scores and log2 of a value's scale to 2^-14; beyond it, see the warps of weights.
constexpr float kFar = 1024.f;
constexpr int kCounters = 4096;           // a counter per piece
static_assert(kCounters == kPagedMaxParts, "one counter per piece");

// NH: heads of a group that the kernel computes, 4 or 8 (more than there are cost as much as others).
template <int D, bool kE4m3>
struct Geo {
  static constexpr int kRow = D * (kE4m3 ? 1 : 2);             // bytes of a row
  static constexpr int kWide = kRow < 128 ? kRow : 128;        // of it in a slab: the swizzle's width
  static constexpr int kSlabs = kRow / kWide;
  // Tokens per tile: a token, or two 128 apart, for each thread of the warps of weights. Two where the
  // products of a tile take less time than what surrounds them.
  static constexpr int kHalves = kRow == 64 ? 2 : 1;
  static constexpr int kTile = 128 * kHalves;
  static constexpr int kSlab = kTile * kWide;
  static constexpr int kTensor = kSlabs * kSlab;               // a K or a V tile
  static constexpr int kQ = kN * kRow;
  static constexpr int kP = kTile * (kE4m3 ? 16 : 32);
  static constexpr int kCtas = kTensor > 16384 ? 1 : 2;        // per SM
  static constexpr int kSlots = (192 / kCtas) * 1024 / kTensor;  // of the ring, half of them K's
  static constexpr int kTiles = kSlots / 2;
  static constexpr int kDescs = kTiles + 4;  // tile descriptors: none is overwritten while in use
  // barriers: where each kind begins, in this order
  static constexpr int kFullAt = 0, kEmptyAt = kFullAt + kSlots, kDescAt = kEmptyAt + kSlots,
                       kSAt = kDescAt + kDescs, kPAt = kSAt + 2, kOAt = kPAt + 2, kFreeAt = kOAt + 2,
                       kQAt = kFreeAt + 2, kQFreeAt = kQAt + 4, kEndAt = kQFreeAt + 2,
                       kSumAt = kEndAt + 2, kSegAt = kSumAt + 4, kSegFreeAt = kSegAt + 4,
                       kJoinAt = kSegFreeAt + 4, kBars = kJoinAt + 1;
  static_assert(kBars <= kThreads, "a barrier per thread");
  static constexpr uint32_t kOCol = 2 * kHalves * kN;  // of tensor memory: O's columns behind two S's
  static constexpr size_t kSmem = 1024 + (size_t)kSlots * kTensor + 2 * kQ + 2 * kP;
  // high words of the matrix descriptors: 8 rows to the next 8, the version bit, the swizzle mode
  static constexpr uint32_t kHi =
      (uint32_t)(8 * kWide >> 4) | (1u << 14) | ((kWide == 128 ? 2u : 4u) << 29);
  // of the weights' operand, not swizzled: bytes from 8 heads to the next 8 (bf16)
  static constexpr uint32_t kPHi = (uint32_t)(kTile * 16 >> 4) | (1u << 14);
  static constexpr uint32_t kType = kE4m3 ? 0u : 1u;
  static constexpr uint32_t idesc(int m, bool mn_major) {
    return (1u << 4) | (kType << 7) | (kType << 10) | ((mn_major ? 3u : 0u) << 15) |
           ((uint32_t)(kN >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
  }
};

// Workspace: the header, a counter per piece, then two partials per piece.
__host__ __device__ inline size_t slot_bytes(int G, int D) {
  return (size_t)G * (D * 4 + 16);  // O, then the maximum (two terms) and the sum
}
constexpr size_t kSlotsOffset = kWsHeaderBytes + kCounters * 4;

struct alignas(16) Tile {
  int lo, hi;      // rows of tokens that are seen
  int flags;
  int b, g;
  int slot;        // partial of this segment, -1: it is the whole pair
  int unit, tiles; // the pair's first tile in the stream, and how many there are
};
constexpr int kFirst = 1, kLast = 2, kEnd = 4;  // of a segment; of the piece (not a tile)

// A base, or a maximum of bases: hi + lo. lo is 0 but where scores are far from zero (is_far): there hi is
// the largest score, and lo what log2 of the values' scales add to it, which hi's steps would swallow.
__device__ __forceinline__ bool is_far(float hi) { return !(fabsf(hi) <= kFar) && hi != -INFINITY; }
struct Base {
  float hi, lo;
  // (hi first: equal ones cancel exactly; NaN for two that are -inf)
  __device__ __forceinline__ float above(const Base &o) const { return (hi - o.hi) + (lo - o.lo); }
  __device__ __forceinline__ Base max(const Base &o) const {
    return above(o) > 0.f || o.hi == -INFINITY ? *this : o;
  }
  // what is subtracted: 0 while there is none
  __device__ __forceinline__ Base or_zero() const { return Base{hi == -INFINITY ? 0.f : hi, lo}; }
};

struct PagedMaps {
  CUtensorMap k, v;
};

struct Waiter {
  volatile int *abort;
  uint32_t *error_word;
  __device__ __forceinline__ bool operator()(uint32_t bar, uint32_t parity) const {
    if (mbar_try_wait(bar, parity)) return true;
    if (*abort) return false;
    if (mbar_wait_bounded(bar, parity)) return true;
    *abort = 1;
    atomicOr(error_word, kErrWaitTimeout);
    return false;
  }
  // the same answer in every lane, and the warp together behind it
  __device__ __forceinline__ bool all(uint32_t bar, uint32_t parity) const {
    return __all_sync(0xffffffffu, (*this)(bar, parity) ? 1 : 0) != 0;
  }
  // three barriers, looked at side by side: all of them have completed more often than not
  __device__ __forceinline__ bool all(uint32_t b0, uint32_t p0, uint32_t b1, uint32_t p1,
                                      uint32_t b2, uint32_t p2) const {
    const bool t0 = mbar_try_wait(b0, p0), t1 = mbar_try_wait(b1, p1), t2 = mbar_try_wait(b2, p2);
    bool ok = t0 && t1 && t2;
    if (!ok) ok = (t0 || (*this)(b0, p0)) && (t1 || (*this)(b1, p1)) && (t2 || (*this)(b2, p2));
    return __all_sync(0xffffffffu, ok ? 1 : 0) != 0;
  }
};

__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

template <bool kE4m3>
__device__ __forceinline__ void umma(uint32_t d, uint32_t a_lo, uint32_t a_hi, uint32_t b_lo,
                                     uint32_t b_hi, uint32_t idesc, uint32_t accumulate) {
  if constexpr (kE4m3)
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "mov.b64 a, {%1, %2};\n\tmov.b64 b, {%3, %4};\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %5, p;\n\t}" ::"r"(d),
        "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "mov.b64 a, {%1, %2};\n\tmov.b64 b, {%3, %4};\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, p;\n\t}" ::"r"(d),
        "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lead) {
  return ((saddr >> 4) & 0x3FFFu) | ((lead >> 4) << 16);
}

__device__ __forceinline__ float warp_max(float x) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Values of at most 448, each as hi + lo / 16, both e4m3: the second term's own factor keeps it clear of
// e4m3's smallest steps. Four codes to a word.
constexpr float kLow = 1.f / 16;
template <int N>
__device__ __forceinline__ void two_terms_e4m3(const float (&x)[N], uint32_t (&hi)[N / 4],
                                               uint32_t (&lo)[N / 4]) {
#pragma unroll
  for (int i = 0; i < N / 2; ++i) {
    // (fp16 has 11 significant bits: the rounding to it is a 2^-12 beside the 2^-8 of what follows,
    // and none for x of 8 bits; hi, x - hi and the factor are then exact in it)
    const __half2 v = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
    const __half2_raw vr = v;
    const uint32_t h = __nv_cvt_halfraw2_to_fp8x2(vr, __NV_SATFINITE, __NV_E4M3);
    const __half2 f = __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)h, __NV_E4M3));
    const __half2_raw r = __hmul2(__hsub2(v, f), __float2half2_rn(16.f));
    const uint32_t l = __nv_cvt_halfraw2_to_fp8x2(r, __NV_SATFINITE, __NV_E4M3);
    if (i & 1) {
      hi[i / 2] |= h << 16;
      lo[i / 2] |= l << 16;
    } else {
      hi[i / 2] = h;
      lo[i / 2] = l;
    }
  }
}
template <int N>
__device__ __forceinline__ void two_terms_bf16(const float (&x)[N], uint32_t (&hi)[N / 2],
                                               uint32_t (&lo)[N / 2]) {
#pragma unroll
  for (int i = 0; i < N / 2; ++i) {
    hi[i] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
    lo[i] = pack_bf16x2(x[2 * i] - bf16_lo(hi[i]), x[2 * i + 1] - bf16_hi(hi[i]));
  }
}
// 8 or 16 fp32 columns of this thread's lane of tensor memory; wait with tmem_wait().
template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t addr, float (&v)[N]) {
  if constexpr (N == 16)
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
        "%11, %12, %13, %14, %15}, [%16];"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]),
          "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]),
          "=f"(v[14]), "=f"(v[15])
        : "r"(addr));
  else
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]),
          "=f"(v[7])
        : "r"(addr));
}
// The loads before it have arrived: v may be used (and its values depend on the wait).
template <int N>
__device__ __forceinline__ void tmem_wait(float (&v)[N]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+f"(v[i]));
}

__device__ __forceinline__ void fence_proxy_async_global() {
  asm volatile("fence.proxy.async.global;" ::: "memory");
}
__device__ __forceinline__ void st_shared16(uint32_t at, uint4 x) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(x.x), "r"(x.y), "r"(x.z),
               "r"(x.w)
               : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void *src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
// An arrival on `bar` once this thread's copies so far are there.
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" ::"r"(bar) : "memory");
}

struct Seq {
  int L, start, tile0, tiles;  // tokens start .. L are seen, in tiles tile0 .. tile0 + tiles
};
template <int kTile>
__device__ __forceinline__ Seq seq_of(const PagedAttnArgs &a, int b) {
  Seq s;
  s.L = min(max(a.lens[b], 0), a.max_len);
  s.start = a.window > 0 ? max(0, s.L - a.window) : 0;
  s.tile0 = s.start / kTile;
  s.tiles = s.L > s.start ? (s.L - 1) / kTile + 1 - s.tile0 : 0;  // (L: up to 2^31 - 1)
  return s;
}

// A token's weights into the operand of the value product.
template <int kTile, bool kE4m3, int NH>
__device__ __forceinline__ void put_weights(const float (&w)[NH], uint32_t at) {
  if constexpr (kE4m3) {
    uint32_t hi[NH / 4], lo[NH / 4];
    two_terms_e4m3<NH>(w, hi, lo);
    if constexpr (NH == 8)
      st_shared16(at, make_uint4(hi[0], hi[1], lo[0], lo[1]));
    else
      asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(at), "r"(hi[0]), "r"(lo[0]) : "memory");
  } else {
    uint32_t hi[NH / 2], lo[NH / 2];
    two_terms_bf16<NH>(w, hi, lo);
    if constexpr (NH == 8) {
      st_shared16(at, make_uint4(hi[0], hi[1], hi[2], hi[3]));
      st_shared16(at + kTile * 16, make_uint4(lo[0], lo[1], lo[2], lo[3]));
    } else {
      st_shared16(at, make_uint4(hi[0], hi[1], lo[0], lo[1]));
    }
  }
}

// A warp of weights: a token per thread (two of 256). A warp's weights are 2^(8 + t - base) with a base per
// head that stays while the largest t of a tile lies within 2^-6 .. 2^0.5 of it: then a tile's weights,
// sums and part of O need no factor of their own.
// Where a base lies beyond kFar, the steps of fp32 are no longer small beside a weight's exponent: the
// largest score is then subtracted from the scores before anything is added, which is exact for equal ones,
// every tile has bases of its own, and they have two terms (kAnyBase). From the first such tile on, a warp
// goes through what is left of the piece in any_base_tiles, a function so that its code lies apart from the
// common tiles': in line behind them it cost the windows above 9%, called tile by tile 4%, so 2% (37.0 to
// 37.7 us).
enum Step { kGo, kStop, kTooFar };
template <int D, bool kE4m3, int NH>
struct Weights {
  using Ge = Geo<D, kE4m3>;
  static constexpr int kHalves = Ge::kHalves, kTile = Ge::kTile;
  Waiter wait;
  const Tile *tile;
  const float (*scale)[2][8 * kHalves];
  const float (*qs)[kG];
  float (*top)[2][4][kG];
  float *base;  // the warp's: bases, 2^(base - maximum), the maximum of the bases so far (hi; its lo last),
                // which the sums are relative to, and what the sums are to be multiplied with
  float (*sums)[4][3][kG];
  uint32_t bars, s, p, ring;  // (s: S^T in this warp's lanes of tensor memory)
  int page_log2;
  int seg;
  float sum[NH];

  __device__ __forceinline__ uint32_t bar(int at, int i) const { return bars + 8 * (at + i); }
  __device__ __forceinline__ static void load4(float (&to)[NH], const float *from) {
#pragma unroll
    for (int h = 0; h < NH; h += 4) {
      const float4 x = *reinterpret_cast<const float4 *>(from + h);
      to[h] = x.x, to[h + 1] = x.y, to[h + 2] = x.z, to[h + 3] = x.w;
    }
  }
  template <bool kAnyBase>
  __device__ __forceinline__ Step step(int n) {
    constexpr int S = Ge::kSlots, ND = Ge::kDescs;
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int d = n % ND, buf = n & 1;
    // its descriptor, its S^T (or the end), and tile n - 2's weights and bases consumed
    const uint32_t phase = (n >> 1) & 1;
    if (!wait.all(bar(Ge::kDescAt, d), (n / ND) & 1, bar(Ge::kSAt, buf), phase, bar(Ge::kFreeAt, buf),
                  phase ^ 1))
      return kStop;
    if (tile[d].flags & kEnd) {
      mbar_arrive(bar(Ge::kPAt, buf));
      return kStop;
    }
    tc_fence_after();
    constexpr int kCols = kE4m3 ? 2 * NH : 8;
    float z[kHalves][kCols];
#pragma unroll
    for (int half = 0; half < kHalves; ++half) tmem_ld(s + (buf * kHalves + half) * kN, z[half]);
    const Tile t = tile[d];
    bool inside[kHalves];
    float ks[kHalves], lvs[kHalves], ivs[kHalves];
#pragma unroll
    for (int half = 0; half < kHalves; ++half) {
      const int row = tid + 128 * half;
      ks[half] = scale[d][0][row >> page_log2];
      const float vs = scale[d][1][row >> page_log2];
      inside[half] = row >= t.lo && row < t.hi;
      if (!inside[half]) ks[half] = -1.f;
      lvs[half] = kE4m3 ? lg2(vs) : 0.f;
      ivs[half] = ks[half] > 0.f ? (kE4m3 ? rcp(vs) : 1.f) : 0.f;
    }
    if (t.flags & kFirst) {
      ++seg;
      if (lane < kG) {
        base[lane] = base[2 * kG + lane] = -INFINITY;
        base[4 * kG + lane] = 0.f;
      }
#pragma unroll
      for (int h = 0; h < NH; ++h) sum[h] = 0.f;
      __syncwarp();
    }
    float q[NH], w[kHalves][NH];
    load4(q, qs[seg & 3]);
    if constexpr (kAnyBase) {
#pragma unroll
      for (int half = 0; half < kHalves; ++half) tmem_wait(z[half]);
      Base b{-INFINITY, 0.f};  // of the head lane & 7
#pragma unroll
      for (int h = 0; h < NH; ++h) {
        float m = -INFINITY, r = -INFINITY;
#pragma unroll
        for (int half = 0; half < kHalves; ++half) {
          const float *x = z[half];
          if constexpr (kE4m3)
            w[half][h] = fmaf(x[NH + h], kLow, x[h]) * (q[h] * ks[half]);
          else
            w[half][h] = x[h] * q[h];
          if (!(ks[half] > 0.f)) w[half][h] = -INFINITY;  // (not seen)
          m = fmaxf(m, w[half][h]);
        }
        m = warp_max(m);
        const float from = m == -INFINITY ? 0.f : m;
#pragma unroll
        for (int half = 0; half < kHalves; ++half) {
          w[half][h] -= from;
          if (ks[half] > 0.f) w[half][h] += lvs[half];
          r = fmaxf(r, w[half][h]);
        }
        r = m == -INFINITY ? 0.f : warp_max(r);
#pragma unroll
        for (int half = 0; half < kHalves; ++half) w[half][h] = ex2((w[half][h] - r) + 8.f);
        if ((lane & (kG - 1)) == h) b = is_far(m) ? Base{m, r} : Base{m + r, 0.f};
      }
      const Base old{base[2 * kG + (lane & (kG - 1))], base[4 * kG + (lane & (kG - 1))]};
      const Base to = b.max(old), by = to.or_zero();
      __syncwarp();
      if (lane < NH) {
        base[kG + lane] = ex2(b.above(by));
        base[2 * kG + lane] = to.hi;
        base[3 * kG + lane] = ex2(old.above(by));
        base[4 * kG + lane] = to.lo;
        top[buf][0][warp][lane] = b.hi;
        top[buf][1][warp][lane] = b.lo;
      }
      __syncwarp();
#pragma unroll
      for (int h = 0; h < NH; ++h) {
        float add = 0.f;
#pragma unroll
        for (int half = 0; half < kHalves; ++half) add = fmaf(w[half][h], ivs[half], add);
        sum[h] = fmaf(add, base[kG + h], sum[h] * base[3 * kG + h]);
      }
    } else {
      float at[NH], beta[NH], most[NH];  // (at: the bases)
      load4(at, base);
      load4(beta, base + kG);
      bool near = true;
#pragma unroll
      for (int half = 0; half < kHalves; ++half) tmem_wait(z[half]);
#pragma unroll
      for (int h = 0; h < NH; ++h) {
        float m = -INFINITY;
#pragma unroll
        for (int half = 0; half < kHalves; ++half) {
          const float *x = z[half];
          if constexpr (kE4m3)
            w[half][h] = fmaf(fmaf(x[NH + h], kLow, x[h]), q[h] * ks[half], lvs[half]);
          else
            w[half][h] = x[h] * q[h];
          if (!(ks[half] > 0.f)) w[half][h] = -INFINITY;  // (not seen)
          m = fmaxf(m, w[half][h]);
        }
        most[h] = warp_max(m);
        near = near && most[h] - at[h] <= 0.5f && most[h] - at[h] >= -6.f;
      }
      if (!near) {  // (the same for the whole warp) a head per lane
        float m = most[0];
#pragma unroll
        for (int h = 1; h < NH; ++h)
          if ((lane & (kG - 1)) == h) m = most[h];
        if (__any_sync(0xffffffffu, is_far(m))) {
          if (t.flags & kFirst) --seg;  // (the tile is gone through again)
          return kTooFar;
        }
        float b = base[lane & (kG - 1)];
        const float old = base[2 * kG + (lane & (kG - 1))], x = m - b;
        if (!(x <= 0.5f && x >= -6.f) && m != -INFINITY) b = m;
        const float to = fmaxf(old, b), by = to == -INFINITY ? 0.f : to;
        __syncwarp();
        if (lane < NH) {
          base[lane] = b;
          base[kG + lane] = ex2(b - by);
          base[2 * kG + lane] = to;
          base[3 * kG + lane] = ex2(old - by);
        }
        __syncwarp();
        load4(at, base);
        load4(beta, base + kG);
        float alpha[NH];
        load4(alpha, base + 3 * kG);
#pragma unroll
        for (int h = 0; h < NH; ++h) sum[h] *= alpha[h];
      }
#pragma unroll
      for (int h = 0; h < NH; ++h) {
        const float by = (at[h] == -INFINITY ? 0.f : at[h]) - 8.f;
        float add = 0.f;
#pragma unroll
        for (int half = 0; half < kHalves; ++half) {
          w[half][h] = ex2(w[half][h] - by);
          add = fmaf(w[half][h], ivs[half], add);
        }
        sum[h] = fmaf(add, beta[h], sum[h]);
      }
      if (lane == 0) {
#pragma unroll
        for (int h = 0; h < NH; h += 4)
          *reinterpret_cast<float4 *>(&top[buf][0][warp][h]) =
              make_float4(at[h], at[h + 1], at[h + 2], at[h + 3]);
      }
    }
#pragma unroll
    for (int half = 0; half < kHalves; ++half)
      put_weights<kTile, kE4m3, NH>(w[half], p + buf * Ge::kP + (tid + 128 * half) * 16);
    // Rows of V that are not seen can hold anything, and 0 times NaN is NaN: they are cleared. (A
    // page that does not exist was left zeros.)
    if (t.lo > 0 || t.hi < kTile) {
      const int slot = (2 * n + 1) % S;
      if (!wait.all(bar(Ge::kFullAt, slot), ((2 * n + 1) / S) & 1)) return kStop;
#pragma unroll
      for (int half = 0; half < kHalves; ++half)
        if (!inside[half])
#pragma unroll
          for (int i = 0; i < Ge::kRow / 16; ++i)
            st_shared16(ring + slot * Ge::kTensor + (i * 16 / Ge::kWide) * Ge::kSlab +
                            (tid + 128 * half) * Ge::kWide + (i * 16) % Ge::kWide,
                        make_uint4(0u, 0u, 0u, 0u));
    }
    if (t.flags & kLast) {
#pragma unroll
      for (int h = 0; h < NH; ++h) {
        const float x = warp_sum(sum[h]);
        if (lane == 0) {
          sums[seg & 3][warp][0][h] = x;
          sums[seg & 3][warp][1][h] = base[2 * kG + h];
          sums[seg & 3][warp][2][h] = base[4 * kG + h];
        }
      }
      if (lane == 0) mbar_arrive(bar(Ge::kSumAt, seg & 3));
    }
    fence_proxy_async_smem();
    tc_fence_before();
    mbar_arrive(bar(Ge::kPAt, buf));
    return kGo;
  }
};
template <int D, bool kE4m3, int NH>
__device__ __noinline__ void any_base_tiles(Weights<D, kE4m3, NH> role, int n) {
  while (role.template step<true>(n) == kGo) ++n;
}

template <int D, bool kE4m3, int NH>
__global__ void __launch_bounds__(kThreads, Geo<D, kE4m3>::kCtas)
    paged_attn_kernel(const __grid_constant__ PagedMaps maps, const PagedCache c,
                      const PagedAttnArgs a, int page_log2, uint8_t *workspace) {
  using Ge = Geo<D, kE4m3>;
  constexpr int S = Ge::kSlots, ND = Ge::kDescs, kTile = Ge::kTile, kHalves = Ge::kHalves;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t s_bar[Ge::kBars];
  __shared__ Tile s_tile[ND];
  __shared__ float s_scale[ND][2][8 * kHalves];  // of a tile's pages, K and V; < 0: no page
  __shared__ __align__(16) float s_qs[4][kG];  // a segment's score scales
  __shared__ __align__(16) float s_top[2][2][4][kG];    // a tile's bases (hi, lo), per warp of tokens
  __shared__ __align__(16) float s_base[4][5][kG];      // see the warps of weights
  __shared__ __align__(16) float s_sum[4][4][3][kG];    // a segment's sums and their maxima (hi, lo)
  __shared__ __align__(16) float s_f[4][5 * kG];        // factors, per warp of dimensions
  __shared__ int2 s_seg[4];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort, s_blk, s_parts, s_joins[2];
  __shared__ int4 s_part[2];                   // pairs that the piece leaves a partial of

  uint8_t *smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  const uint32_t ring = smem_addr(smem), q_s = ring + S * Ge::kTensor, p_s = q_s + 2 * Ge::kQ;
  const uint32_t bars = smem_addr(s_bar), bar_full = bars + 8 * Ge::kFullAt;
  const uint32_t bar_empty = bars + 8 * Ge::kEmptyAt;
  const uint32_t bar_desc = bars + 8 * Ge::kDescAt, bar_s = bars + 8 * Ge::kSAt, bar_p = bars + 8 * Ge::kPAt;
  const uint32_t bar_o = bars + 8 * Ge::kOAt, bar_free = bars + 8 * Ge::kFreeAt, bar_q = bars + 8 * Ge::kQAt;
  const uint32_t bar_qfree = bars + 8 * Ge::kQFreeAt, bar_end = bars + 8 * Ge::kEndAt;
  const uint32_t bar_sum = bars + 8 * Ge::kSumAt, bar_seg = bars + 8 * Ge::kSegAt;
  const uint32_t bar_segfree = bars + 8 * Ge::kSegFreeAt, bar_join = bars + 8 * Ge::kJoinAt;
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int G = a.Hq / c.Hkv;

  // A barrier per thread. (A barrier completes its next phase only when all that wait for the one
  // before have seen that: each role's waits say so, those for the end of the piece included.)
  if (tid < Ge::kBars) {
    const bool many = (tid >= Ge::kPAt && tid < Ge::kOAt) || (tid >= Ge::kFreeAt && tid < Ge::kQAt);
    mbar_init(bars + 8 * tid, tid >= Ge::kDescAt && tid < Ge::kSAt ? (kE4m3 ? 33 : 1)
                              : many                       ? 128
                              : tid >= Ge::kSumAt && tid < Ge::kSegAt ? 4
                                                              : 1);
    fence_barrier_init();
  }
  if (tid == 0) s_abort = s_parts = 0;
  if (warp == kTma) {
    if (lane == 0) {
      tma_prefetch_desc(&maps.k);
      tma_prefetch_desc(&maps.v);
    }
    tmem_alloc(smem_addr(&s_tmem), kTmemCols);
  }
  // rows of Q that no head fills stay zero, and so do the weights' unused columns
  for (int i = tid; i < 2 * (Ge::kQ + Ge::kP) / 16; i += kThreads)
    st_shared16(q_s + 16 * i, make_uint4(0u, 0u, 0u, 0u));
  fence_proxy_async_smem();  // (the zeros)
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_wait_prior_grid();
  pdl_launch_dependents();
  const int P = gridDim.x, piece = blockIdx.x;
  const uint32_t tmem = __shfl_sync(0xffffffffu, s_tmem, 0);
  const Waiter wait{&s_abort, a.error_word};

  if (warp == kTma) {
    // ---------------------------------------------------------------- loads
    const int page = 1 << page_log2, ppt = kTile >> page_log2;
    const int ppt_log2 = (kHalves == 2 ? 8 : 7) - page_log2;
    const int batch = 32 >> ppt_log2;  // tiles whose page numbers the lanes hold
    const uint64_t policy = l2_policy_evict_first();
    // Where this piece begins: a scan over the sequences, a run of them per lane.
    const int per = (a.B + 31) >> 5, b_first = min(a.B, lane * per), b_last = min(a.B, b_first + per);
    int2 mine = make_int2(0, 0);  // tiles, pairs
#pragma unroll 4
    for (int i = b_first; i < b_last; ++i) {
      const int tiles = seq_of<kTile>(a, i).tiles;
      mine.x += tiles;
      mine.y += tiles > 0;
    }
    mine.x *= c.Hkv, mine.y *= c.Hkv;
    int2 incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, incl.x, o), y = __shfl_up_sync(0xffffffffu, incl.y, o);
      if (lane >= o) incl.x += x, incl.y += y;
    }
    const int all = __shfl_sync(0xffffffffu, incl.x, 31), pairs = __shfl_sync(0xffffffffu, incl.y, 31);
    const int segment = all >= kFew * P ? kSegment : 0, total = all + segment * pairs;
    const int blk = max(1u, ((unsigned)total + P - 1) / (unsigned)P);
    const long long r0 = (long long)piece * blk;
    if (lane == 0) s_blk = blk;  // (for the end of a segment that is not a whole pair)
    // the walk: (b, g), its tiles t0 .. t1 of this piece (from the sequence's first seen one), and
    // those of them that the lanes have looked up
    int b = -1, g = 0, left = 0, t0 = 0, t1 = 0, off = 0, within = 0;
    Seq s{};
    {
      const int count = mine.x + segment * mine.y;
      int at = incl.x + segment * incl.y - count;
      if (at <= r0 && r0 < at + count) {
        for (b = b_first;; ++b) {
          const Seq x = seq_of<kTile>(a, b);
          const int u = x.tiles > 0 ? (x.tiles + segment) * c.Hkv : 0;
          if (r0 < at + u) break;
          at += u;
        }
        within = (int)r0 - at;
      }
      const unsigned who = __ballot_sync(0xffffffffu, b >= 0);
      const int from = who != 0 ? __ffs(who) - 1 : 0;
      b = __shfl_sync(0xffffffffu, b, from);
      within = __shfl_sync(0xffffffffu, within, from);
    }
    auto take = [&](int from) {  // from: units of this pair that lie before the piece
      t0 = max(0, from - segment);
      t1 = max(t0, min(s.tiles, from + left - segment));
      left -= min(left, t1 + segment - from);
    };
    bool more = b >= 0;
    if (more) {
      s = seq_of<kTile>(a, b);
      const int u = s.tiles + segment;
      g = (unsigned)within / (unsigned)u;
      const int from = within - g * u;
      off = (int)r0 - from;
      left = (int)min((long long)blk, total - r0);
      take(from);
    }
    // the next pair; false: none in this piece
    auto next_pair = [&]() {
      if (left <= 0) return false;
      off += s.tiles + segment;
      if (++g == c.Hkv) {
        g = 0;
        do {
          if (++b >= a.B) return false;
          s = seq_of<kTile>(a, b);
        } while (s.tiles == 0);
      }
      take(0);
      return true;
    };
    struct Batch {
      Seq s;
      int b, g, from, to, t0, t1, off, page;
    };
    Tile t{};
    int at_tile = t0;
    auto next_batch = [&](Batch &x) {
      while (more && at_tile >= t1) {
        more = next_pair();
        at_tile = t0;
      }
      if (!more) return false;
      x.s = s, x.b = b, x.g = g, x.t0 = t0, x.t1 = t1, x.off = off;
      x.from = at_tile;
      x.to = min(t1, at_tile + batch);
      at_tile = x.to;
      // this lane's page: tile from + lane / ppt, page lane % ppt of it; only where a token is seen
      const int slot = ((s.tile0 + x.from) << ppt_log2) + lane;
      const long long row = (long long)slot << page_log2;
      x.page = -1;
      if (row < s.L && row + page - 1 >= s.start && lane < (x.to - x.from) << ppt_log2)
        x.page = c.table[(size_t)b * c.max_pages + slot];
      return true;
    };
    int n = 0, seg = 0;
    bool ok = true;
    auto push_segment = [&](int b_, int g_) {
      if (seg >= 4 && !wait.all(bar_segfree + 8 * (seg & 3), ((seg >> 2) - 1) & 1)) return false;
      if (lane == 0) {
        s_seg[seg & 3] = make_int2(b_, g_);
        mbar_arrive(bar_seg + 8 * (seg & 3));
      }
      ++seg;
      return true;
    };
    Batch cur, nxt;
    bool have = next_batch(cur);
    while (have && ok) {
      const bool have_next = next_batch(nxt);
      for (int i = cur.from; i < cur.to && ok; ++i, ++n) {
        const int row0 = (cur.s.tile0 + i) * kTile;
        const int lo = max(0, cur.s.start - row0), hi = min(kTile, cur.s.L - row0);
        const int d = n % ND, ks = (2 * n) % S, vs = (2 * n + 1) % S;
        // pages p0 .. p1 of the tile hold tokens that are seen; a lane each
        const int p0 = lo >> page_log2, p1 = (hi + page - 1) >> page_log2;
        const int number =
            __shfl_sync(0xffffffffu, cur.page, ((i - cur.from) << ppt_log2) + (lane & (ppt - 1)));
        const bool here = lane >= p0 && lane < p1;
        const bool good = number >= 0 && number < c.num_pages;
        const int head = good ? number * c.Hkv + cur.g : -1;  // (-1: the copy leaves zeros)
        const int bytes = (p1 - p0) * page * Ge::kRow;
        if (2 * n >= S && !(ok = wait.all(bar_empty + 8 * ks, ((2 * n / S) - 1) & 1))) break;
        if (i == cur.t0) {
          if (!(ok = push_segment(cur.b, cur.g))) break;
          t.b = cur.b;
          t.g = cur.g;
          t.slot = cur.t0 == 0 && cur.t1 == cur.s.tiles ? -1 : 2 * piece + (cur.t0 == 0);
          t.unit = cur.off + segment;
          t.tiles = cur.s.tiles;
        }
        if (here) {
          if (!good) {
            s_scale[d][0][lane] = s_scale[d][1][lane] = -1.f;
            if (cur.g == 0) atomicOr(a.error_word, kErrPageSkipped);
          } else if (kE4m3) {
            cp_async4(smem_addr(&s_scale[d][0][lane]), c.k_scale + head);
            cp_async4(smem_addr(&s_scale[d][1][lane]), c.v_scale + head);
          } else {
            s_scale[d][0][lane] = s_scale[d][1][lane] = 1.f;
          }
        }
        if (lane == 0) {
          t.lo = lo;
          t.hi = hi;
          t.flags = (i == cur.t0 ? kFirst : 0) | (i == cur.t1 - 1 ? kLast : 0);
          s_tile[d] = t;
          mbar_arrive_expect_tx(bar_full + 8 * ks, bytes);
        }
        __syncwarp();
        if (here)
#pragma unroll
          for (int sl = 0; sl < Ge::kSlabs; ++sl)
            tma_load_3d(ring + ks * Ge::kTensor + sl * Ge::kSlab + (lane << page_log2) * Ge::kWide,
                        &maps.k, sl * (Ge::kWide / (kE4m3 ? 1 : 2)), 0, head, bar_full + 8 * ks,
                        policy);
        if (kE4m3) cp_async_arrive(bar_desc + 8 * d);
        if (lane == 0) mbar_arrive(bar_desc + 8 * d);
        if (2 * n + 1 >= S && !(ok = wait.all(bar_empty + 8 * vs, (((2 * n + 1) / S) - 1) & 1))) {
          ++n;  // (its keys are on their way)
          break;
        }
        if (lane == 0) mbar_arrive_expect_tx(bar_full + 8 * vs, bytes);
        __syncwarp();
        if (here)
#pragma unroll
          for (int sl = 0; sl < Ge::kSlabs; ++sl)
            tma_load_3d(ring + vs * Ge::kTensor + sl * Ge::kSlab + (lane << page_log2) * Ge::kWide,
                        &maps.v, sl * (Ge::kWide / (kE4m3 ? 1 : 2)), 0, head, bar_full + 8 * vs,
                        policy);
      }
      cur = nxt;
      have = have_next;
    }
    // the end of the piece, where the next tile would be
    const int d = n % ND;
    if (ok && (2 * n < S || wait.all(bar_empty + 8 * ((2 * n) % S), ((2 * n / S) - 1) & 1)) &&
        push_segment(-1, 0)) {
      if (lane == 0) s_tile[d].flags = kEnd;
      __syncwarp();
      if (kE4m3) cp_async_arrive(bar_desc + 8 * d);
      if (lane == 0) mbar_arrive(bar_desc + 8 * d);
    }
    // no copy into this CTA's shared memory may outlive it (all have landed unless a wait gave up)
    for (int j = max(0, n - (S + 1) / 2); j < n; ++j) {
      mbar_wait_bounded(bar_full + 8 * ((2 * j) % S), (2 * j / S) & 1);
      mbar_wait_bounded(bar_full + 8 * ((2 * j + 1) % S), ((2 * j + 1) / S) & 1);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if (warp == kQuery) {
    // ---------------------------------------------------------------- queries
    // 8 elements a lane: a head is D / 8 lanes.
    constexpr int kLanes = D / 8, kHeads = 32 / kLanes;
    for (int seg = 0;; ++seg) {
      const int r = seg & 3;
      if (!wait.all(bar_seg + 8 * r, (seg >> 2) & 1)) break;
      const int2 at_pair = s_seg[r];
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_segfree + 8 * r);
      if (at_pair.x < 0) break;
      const __nv_bfloat16 *q = a.q + ((size_t)at_pair.x * a.Hq + (size_t)at_pair.y * G) * D;
      constexpr int kLoads = kG / kHeads;
      uint4 w[kLoads];
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        w[i] = make_uint4(0u, 0u, 0u, 0u);
        if (i * kHeads + lane / kLanes < G)
          w[i] = *reinterpret_cast<const uint4 *>(q + (i * 32 + lane) * 8);
      }
      if (seg >= 2 && !wait.all(bar_qfree + 8 * (seg & 1), ((seg >> 1) - 1) & 1)) break;
      const uint32_t base = q_s + (seg & 1) * Ge::kQ;
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int h = i * kHeads + lane / kLanes, ch = lane % kLanes;
        float x[8] = {bf16_lo(w[i].x), bf16_hi(w[i].x), bf16_lo(w[i].y), bf16_hi(w[i].y),
                      bf16_lo(w[i].z), bf16_hi(w[i].z), bf16_lo(w[i].w), bf16_hi(w[i].w)};
        if (kE4m3) {
          float m = 0.f;
#pragma unroll
          for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(x[j]));
#pragma unroll
          for (int o = kLanes / 2; o > 0; o >>= 1)
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
          // 2^e with the largest below 2^8 times it (any finite one, down to 2^-119); an infinity makes
          // every score a NaN
          const int e = min(max((int)(__float_as_uint(m) >> 23) - 127 - 7, -126), 120);
          const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
          for (int j = 0; j < 8; ++j) x[j] *= inv;
          uint32_t hi[2], lo[2];
          two_terms_e4m3<8>(x, hi, lo);
          if (h < G) {
            if (ch == 0)
              s_qs[r][h] = m < INFINITY ? a.scale_log2 * __uint_as_float((uint32_t)(127 + e) << 23)
                                        : __uint_as_float(0x7fc00000u);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              const int row = h + t * NH, c16 = ch >> 1;
              const int sw = Ge::kWide == 128 ? row & 7 : (row >> 1) & 3;
              const uint32_t (&v)[2] = t ? lo : hi;
              asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(
                               base + row * Ge::kWide + ((c16 ^ sw) << 4) + ((ch & 1) << 3)),
                           "r"(v[0]), "r"(v[1])
                           : "memory");
            }
          }
        } else if (h < G) {
          if (ch == 0) s_qs[r][h] = a.scale_log2;
          st_shared16(base + (ch >> 3) * (kN * 128) + h * 128 + (((ch & 7) ^ (h & 7)) << 4), w[i]);
        }
      }
      if (lane < kG && lane >= G) s_qs[r][lane] = 0.f;
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_q + 8 * r);
    }
  } else if (warp == kScore) {
    // ---------------------------------------------------------------- S^T = K Q^T
    // (the warp stays together and an elected lane issues: the operands are then the same across
    // the warp as far as the compiler can tell)
    constexpr uint32_t idesc = Ge::idesc(128, false);
    int seg = -1;
    for (int n = 0;; ++n) {
      const int d = n % ND, slot = (2 * n) % S;
      if (!wait.all(bar_desc + 8 * d, (n / ND) & 1)) break;
      const int flags = s_tile[d].flags;
      // The buffer's last tile has been read: a barrier completes its next phase only when all that wait
      // for the one before have seen that.
      if (n >= 2 && !wait.all(bar_p + 8 * (n & 1), ((n - 2) >> 1) & 1)) break;
      if (flags & kEnd) {
        if (elect_one()) umma_commit(bar_s + 8 * (n & 1));  // (the warps of weights wait for both)
        break;
      }
      if (flags & kFirst) {
        ++seg;
        if (!wait.all(bar_q + 8 * (seg & 3), (seg >> 2) & 1)) break;
      }
      if (!wait.all(bar_full + 8 * slot, (2 * n / S) & 1)) break;
      tc_fence_after();
      const uint32_t k_lo = desc_lo(ring + slot * Ge::kTensor, 16);
      const uint32_t q_lo = desc_lo(q_s + (seg & 1) * Ge::kQ, 16);
      if (elect_one()) {
#pragma unroll
        for (int half = 0; half < kHalves; ++half)
#pragma unroll
          for (int k = 0; k < Ge::kRow / 32; ++k) {
            constexpr int kPer = Ge::kWide / 32;
            umma<kE4m3>(tmem + ((n & 1) * kHalves + half) * kN,
                        k_lo + (k / kPer) * (Ge::kSlab >> 4) + 2 * (k % kPer) +
                            half * (128 * Ge::kWide >> 4),
                        Ge::kHi, q_lo + (k / kPer) * (kN * Ge::kWide >> 4) + 2 * (k % kPer),
                        Ge::kHi, idesc, k > 0);
          }
        umma_commit(bar_empty + 8 * slot);
        umma_commit(bar_s + 8 * (n & 1));
        if (flags & kLast) umma_commit(bar_qfree + 8 * (seg & 1));
      }
      __syncwarp();
    }
    // what was issued finishes before tensor memory is given back
    __syncwarp();
    if (elect_one()) umma_commit(bar_end);
    __syncwarp();
    mbar_wait_bounded(bar_end, 0);
  } else if (warp == kValue) {
    // ---------------------------------------------------------------- O^T = V^T P^T, 32 tokens each
    constexpr uint32_t idesc = Ge::idesc(D, true);
    constexpr int kStep = kE4m3 ? 32 : 16;  // tokens of an instruction
    for (int n = 0;; ++n) {
      const int d = n % ND, slot = (2 * n + 1) % S;
      if (!wait.all(bar_desc + 8 * d, (n / ND) & 1)) break;
      if (n >= 2 && !wait.all(bar_free + 8 * (n & 1), ((n - 2) >> 1) & 1)) break;
      if (s_tile[d].flags & kEnd) {
        if (elect_one()) umma_commit(bar_o + 8 * (n & 1));
        break;
      }
      if (!wait.all(bar_full + 8 * slot, ((2 * n + 1) / S) & 1)) break;
      if (!wait.all(bar_p + 8 * (n & 1), (n >> 1) & 1)) break;
      tc_fence_after();
      const uint32_t v_lo = desc_lo(ring + slot * Ge::kTensor, Ge::kSlab);
      const uint32_t p_lo = desc_lo(p_s + (n & 1) * Ge::kP, 128);
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < kTile / kStep; ++k)
          umma<kE4m3>(tmem + Ge::kOCol + (n & 1) * kOCols + (k * kStep / 32 % 4) * kN,
                      v_lo + k * (kStep * Ge::kWide >> 4), Ge::kHi, p_lo + k * kStep, Ge::kPHi, idesc,
                      (k * kStep) % 32 != 0 || k * kStep >= 128);
        umma_commit(bar_empty + 8 * slot);
        umma_commit(bar_o + 8 * (n & 1));
      }
      __syncwarp();
    }
    __syncwarp();
    if (elect_one()) umma_commit(bar_end + 8);
    __syncwarp();
    mbar_wait_bounded(bar_end + 8, 0);
  } else if (warp < 4) {
    // ---------------------------------------------------------------- weights
    Weights<D, kE4m3, NH> role{wait, s_tile, s_scale, s_qs, s_top, s_base[warp][0], s_sum, bars,
                               tmem + ((uint32_t)(32 * warp) << 16), p_s, ring, page_log2, -1, {}};
    int n = 0;
    Step last;
    while ((last = role.template step<false>(n)) == kGo) ++n;
    if (last == kTooFar) any_base_tiles(role, n);
  } else {
    // ---------------------------------------------------------------- the running O
    // D = 64: an M of 64 puts row 16 w + i into lane i < 16 of warp w's quarter.
    const int w4 = warp - 4, dim = D == 128 ? 32 * w4 + lane : 16 * w4 + lane;
    const bool mine_too = D == 128 || lane < 16;
    const uint32_t my_o = tmem + ((uint32_t)(32 * w4) << 16) + Ge::kOCol;
    float acc[NH];
    Base top{-INFINITY, 0.f};  // the running maximum of the bases of head lane & 7
    int seg = -1;
    // sequences without tokens are nobody's tiles: their zeros
    for (int b = piece; b < a.B; b += P) {
      const Seq x = seq_of<kTile>(a, b);
      if (tid == 128 && x.L != a.lens[b]) atomicOr(a.error_word, kErrLenClamped);
      if (x.tiles == 0)
        for (int i = tid - 128; i < a.Hq * D / 8; i += 128)
          reinterpret_cast<uint4 *>(a.out + (size_t)b * a.Hq * D)[i] = make_uint4(0u, 0u, 0u, 0u);
    }
    for (int n = 0;; ++n) {
      const int d = n % ND, buf = n & 1;
      const uint32_t phase = (n >> 1) & 1;
      // the descriptor, the bases, and the product (or the end)
      if (!wait.all(bar_desc + 8 * d, (n / ND) & 1, bar_p + 8 * buf, phase, bar_o + 8 * buf, phase))
        break;
      const Tile t = s_tile[d];
      if (t.flags & kEnd) break;
      tc_fence_after();
      float o[2][2 * NH];
      tmem_ld(my_o + buf * kOCols, o[0]);
      tmem_ld(my_o + buf * kOCols + kN, o[1]);
      if (t.flags & kFirst) {
        ++seg;
        top = Base{-INFINITY, 0.f};
#pragma unroll
        for (int h = 0; h < NH; ++h) acc[h] = 0.f;
      }
      {
        Base x{s_top[buf][0][lane >> 3][lane & 7], 0.f}, to;
        if (__any_sync(0xffffffffu, (lane & 7) < NH && (is_far(x.hi) || is_far(top.hi)))) {
          if (is_far(x.hi)) x.lo = s_top[buf][1][lane >> 3][lane & 7];
          to = x;
#pragma unroll
          for (int o = 8; o < 32; o *= 2)
            to = to.max(Base{__shfl_xor_sync(0xffffffffu, to.hi, o),
                             __shfl_xor_sync(0xffffffffu, to.lo, o)});
          to = to.max(top);
          const Base base = to.or_zero();
          s_f[w4][lane] = ex2(x.above(base) - 8.f);
          if (lane < kG) s_f[w4][32 + lane] = ex2(top.above(base));
        } else {
          float m = fmaxf(x.hi, __shfl_xor_sync(0xffffffffu, x.hi, 8));
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
          to = Base{fmaxf(top.hi, m), 0.f};
          const float base = to.hi == -INFINITY ? 0.f : to.hi;
          s_f[w4][lane] = ex2(x.hi - base - 8.f);  // (0 where a warp saw nothing)
          if (lane < kG) s_f[w4][32 + lane] = ex2(top.hi - base);
        }
        top = to;
      }
      __syncwarp();
      const float4 *f4 = reinterpret_cast<const float4 *>(s_f[w4]);
#pragma unroll
      for (int h = 0; h < NH; h += 4) {
        const float4 x = f4[8 + h / 4];
        acc[h] *= x.x, acc[h + 1] *= x.y, acc[h + 2] *= x.z, acc[h + 3] *= x.w;
      }
#pragma unroll
      for (int w = 0; w < 4; w += 2) {
        tmem_wait(o[0]);
        tmem_wait(o[1]);
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int h = 0; h < NH; h += 4) {
            const float4 x = f4[2 * (w + u) + h / 4];
            const float f[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int j = 0; j < 4; ++j)
              acc[h + j] = fmaf(fmaf(o[u][NH + h + j], kE4m3 ? kLow : 1.f, o[u][h + j]), f[j],
                                acc[h + j]);
          }
        if (w == 0) {
          tmem_ld(my_o + buf * kOCols + 2 * kN, o[0]);
          tmem_ld(my_o + buf * kOCols + 3 * kN, o[1]);
        }
      }
      __syncwarp();
      if (!(t.flags & kLast)) {
        tc_fence_before();
        mbar_arrive(bar_free + 8 * buf);
        continue;
      }
      // a segment's end: the four warps' sums under one maximum
      if (!wait.all(bar_sum + 8 * (seg & 3), (seg >> 2) & 1)) break;
      float l = 0.f;
      const Base base = top.or_zero();
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const Base of{s_sum[seg & 3][w][1][lane & 7], s_sum[seg & 3][w][2][lane & 7]};
        l += s_sum[seg & 3][w][0][lane & 7] * ex2(of.above(base) - 8.f);
      }
      __syncwarp();
      tc_fence_before();
      mbar_arrive(bar_free + 8 * buf);  // (after the last read of what the tile and segment left)
      if (t.slot < 0) {
        const float inv = l == 0.f ? 0.f : 1.f / l;
        __nv_bfloat16 *out = a.out + ((size_t)t.b * a.Hq + (size_t)t.g * G) * D + dim;
#pragma unroll
        for (int h = 0; h < NH; ++h) {
          const float x = __shfl_sync(0xffffffffu, inv, h);
          if (h < G && mine_too) out[h * D] = __float2bfloat16(acc[h] * x);
        }
        continue;
      }
      uint8_t *part = workspace + kSlotsOffset + (size_t)t.slot * slot_bytes(G, D);
#pragma unroll
      for (int h = 0; h < NH; ++h)
        if (h < G && mine_too) reinterpret_cast<float *>(part)[h * D + dim] = acc[h];
      if (w4 == 0 && lane < G)
        reinterpret_cast<float4 *>(part + (size_t)G * D * 4)[lane] =
            make_float4(top.hi, top.lo, l, 0.f);
      fence_proxy_async_global();  // (they are read by bulk copies)
      if (tid == 128) s_part[s_parts++] = make_int4(t.unit, t.tiles, t.b, t.g);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kTma) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
  // ---- a pair whose last partial this piece delivers is joined here
  const int parts = s_parts;
  if (parts == 0 || s_abort) return;
  if (tid < parts) {
    const int4 x = s_part[tid];
    const int first = (unsigned)x.x / (unsigned)s_blk, last = (unsigned)(x.x + x.y - 1) / (unsigned)s_blk;
    int *counter = reinterpret_cast<int *>(workspace + kWsHeaderBytes) + first;
    __threadfence();  // the CTA's stores, which the barrier has gathered
    const bool all_there = atomicAdd(counter, 1) == last - first;
    if (all_there) *counter = 0;  // as the next call wants it
    __threadfence();
    fence_proxy_async_global();
    s_joins[tid] = all_there;
  }
  __syncthreads();
  // out = sum_c 2^(m_c - M) O_c / sum_c 2^(m_c - M) l_c in the order of the pieces: the partials come by
  // bulk copies into the ring, as many at a time as it holds, 4 neighbouring dims of a head a thread.
  const uint32_t slot = (uint32_t)slot_bytes(G, D);
  const int room = min(32, (int)(S * Ge::kTensor / slot));
  const int h = tid / (D / 4), dim4 = tid - h * (D / 4);
  uint32_t phase = 0;
  for (int i = 0; i < parts; ++i) {
    if (!s_joins[i]) continue;
    const int4 x = s_part[i];
    const int first = (unsigned)x.x / (unsigned)s_blk, last = (unsigned)(x.x + x.y - 1) / (unsigned)s_blk;
    Base M{-INFINITY, 0.f};
    float sum = 0.f, o[4] = {};
    for (int c0 = first; c0 <= last; c0 += room) {
      const int n = min(room, last + 1 - c0);
      if (warp == 0) {
        if (lane == 0) mbar_arrive_expect_tx(bar_join, n * slot);
        __syncwarp();
        if (lane < n)
          bulk_load(ring + lane * slot,
                    workspace + kSlotsOffset + (size_t)(2 * (c0 + lane) + (c0 + lane == first)) * slot,
                    slot, bar_join);
      }
      if (!mbar_wait_bounded(bar_join, phase)) atomicOr(a.error_word, kErrWaitTimeout);
      phase ^= 1;
      if (h < G) {
        const uint8_t *p = smem;
#pragma unroll 4
        for (int k = 0; k < n; ++k, p += slot) {
          const float4 y = reinterpret_cast<const float4 *>(p)[tid];
          const float4 ml = reinterpret_cast<const float4 *>(p + (size_t)G * D * 4)[h];
          const Base of{ml.x, ml.y}, to = of.max(M), base = to.or_zero();
          const float f = ex2(M.above(base)), w = ex2(of.above(base));
          M = to;
          sum = fmaf(sum, f, ml.z * w);
          o[0] = fmaf(o[0], f, y.x * w);
          o[1] = fmaf(o[1], f, y.y * w);
          o[2] = fmaf(o[2], f, y.z * w);
          o[3] = fmaf(o[3], f, y.w * w);
        }
      }
      __syncthreads();
    }
    if (h < G) {
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      __nv_bfloat16 *out = a.out + ((size_t)x.z * a.Hq + (size_t)x.w * G + h) * D + 4 * dim4;
      *reinterpret_cast<uint2 *>(out) =
          make_uint2(pack_bf16x2(o[0] * inv, o[1] * inv), pack_bf16x2(o[2] * inv, o[3] * inv));
    }
  }
}

template <int D, bool kE4m3, int NH>
cudaError_t launch(const PagedMaps &m, const PagedCache &c, const PagedAttnArgs &a, int parts,
                   uint8_t *ws, cudaStream_t stream) {
  // per device: the kernel's shared memory (set before its first launch there)
  static std::atomic<uint64_t> ready{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (!(ready.load(std::memory_order_relaxed) & bit)) {
    e = cudaFuncSetAttribute(paged_attn_kernel<D, kE4m3, NH>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)Geo<D, kE4m3>::kSmem);
    if (e != cudaSuccess) return e;
    ready.fetch_or(bit, std::memory_order_relaxed);
  }
  int log2 = 4;
  while ((1 << log2) < c.page) ++log2;
  return launch_pdl(paged_attn_kernel<D, kE4m3, NH>, dim3(parts), kThreads, Geo<D, kE4m3>::kSmem,
                    stream, m, c, a, log2, ws);
}

}  // namespace

// As many CTAs as the SMs hold, or fewer when there are not as many tiles.
int paged_attn_parts(int B, int Hkv, int D, int e4m3, int max_len, int num_parts, int sms) {
  auto of = [](auto geo) { return std::pair<int, int>(decltype(geo)::kCtas, decltype(geo)::kTile); };
  const auto [per, tile] = D == 128 ? (e4m3 ? of(Geo<128, true>{}) : of(Geo<128, false>{}))
                                    : (e4m3 ? of(Geo<64, true>{}) : of(Geo<64, false>{}));
  const long long tiles = (long long)B * Hkv * (((long long)max_len + tile - 1) / tile + 1);
  // (a piece's ring goes by 32-bit numbers, two to a tile)
  if (num_parts > 0) return std::max(num_parts, (int)((tiles + (1 << 28) - 1) >> 28));
  const long long most = per * sms < kPagedMaxParts ? per * sms : kPagedMaxParts;
  return (int)(tiles < 1 ? 1 : tiles < most ? tiles : most);
}

size_t paged_attn_ws_bytes(int Hq, int Hkv, int D, int parts) {
  return kSlotsOffset + (size_t)2 * parts * slot_bytes(Hq / Hkv, D);
}

cudaError_t launch_paged_attn(const CUtensorMap &k, const CUtensorMap &v, const PagedCache &c,
                              const PagedAttnArgs &a, int parts, void *workspace,
                              cudaStream_t stream) {
  const PagedMaps m{k, v};
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  auto go = [&](auto dim, auto e4m3) {
    constexpr int kD = decltype(dim)::value;
    constexpr bool kE = decltype(e4m3)::value;
    return a.Hq / c.Hkv <= 4 ? launch<kD, kE, 4>(m, c, a, parts, ws, stream)
                             : launch<kD, kE, 8>(m, c, a, parts, ws, stream);
  };
  using I64 = std::integral_constant<int, 64>;
  using I128 = std::integral_constant<int, 128>;
  const cudaError_t e =
      c.D == 128 ? (c.e4m3 ? go(I128{}, std::true_type{}) : go(I128{}, std::false_type{}))
                 : (c.e4m3 ? go(I64{}, std::true_type{}) : go(I64{}, std::false_type{}));
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace decattn
