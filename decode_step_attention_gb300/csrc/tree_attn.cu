// Attention of a draft tree's nodes over the cached prefix and their ancestors: the
// single-query attention of gqa_decode.cu for up to 64 queries per sequence, on the
// 5th-generation tensor cores.
//
//   z[n, h, t]   = scale q[b,n,h] . K_t          t over the cache rows [0, lens[b])
//                                                and the tree's nodes
//   z           <- cap tanh(z / cap)             (softcap > 0)
//   z           <- z - slope_h (pos_n - kpos_t)  (slopes given; kpos = slot or pos of node)
//   out[b,n,h]   = sum_t softmax_t(z) V_t        over the rows node n sees
//
// The rows of a (sequence, KV head) pair, node n and head-in-group i as row n G + i, are cut
// into tiles of 128, the M of one tensor-core instruction: every row of the tile shares one
// read of the K and V tiles. The keys are cut into tiles of 64 tokens, the tree's nodes being
// the last one. All (pair, row tile, key tile) units form one stream, cut into equal pieces,
// one per CTA (two CTAs per SM); a (pair, row tile) that crosses pieces leaves a partial
// (unnormalised O, running maximum and sum) per piece, which tree_merge_kernel joins.
//
// Short contexts take one launch instead: a (pair, row tile) is a CTA's, or a cluster's, which joins
// its partials through distributed shared memory (kJoin).
//
// Inside a CTA, per key tile:
//   warp 4   loads the K and V tiles (TMA, 128-byte swizzle) into a ring of shared memory;
//   warp 5   issues S = Q K^T (both operands in shared memory) into one of two tensor-memory
//            buffers, one tile ahead, and O += P V with P in tensor memory, V as it lies
//            (tokens x dims: the MN-major operand);
//   warps 0-3 take a row per thread: masks, online softmax in base 2, P as bf16 over S's
//            own columns. The running maximum only moves when a tile exceeds it by more than
//            2^8: O is then rescaled in tensor memory, otherwise left alone; the weights
//            stay below 2^8, where bf16 rounds them as well as below 1.
// Warps whose 32 rows are all past the tile's last row only keep the barriers company.
//
// Measured, a call among others with the merge (floor: bytes at the measured copy bandwidth, or
// operations at the measured bf16 rate; the sweeps below and the figures at the constants are the
// GPU's share alone, 3 to 6 us less, both sides measured alike):
//   131072 tokens, 26 nodes, 32 / 8 heads of 128       101 us (79); HBM, 6.0 TB/s in this kernel
//   32 sequences to 8192, 16 nodes, cap                103 us (85); HBM
//   192 sequences to 32768, one node, 16 / 4 of 64     74 us (59); S with 16 of 128 rows in use
//   16 sequences, window 4095, 64 nodes, 64 / 8 of 128 131 us (62); the tensor cores: an S with 64
//       keys takes as long as one with 128, because Q is read from shared memory for each
// Tried for the last: S for two key tiles at once. It needs both S buffers, so S, softmax and the
// value products of a CTA take turns, and two CTAs do not fill the gaps (144 us). Eight softmax
// warps of half a row's keys each, which agree on the maximum tile by tile: 171 us.
//
// The weights are one bf16 each (a rounding of at most 2^-8 of each); sums, maxima and O are fp32.
// Against 64 bits the result is off by 1.9e-3 to 2.4e-3 (relative, root mean square), of which the
// output's own rounding is 1.7e-3. The single-token kernel of gqa_decode.cu gives the value
// product a second bf16 per weight, what the first rounding left; here that makes the error 1.7e-3,
// and memory does not hide it: the GPU's share of four cases like those above goes from 97.0 to
// 100.4 us, 97.2 to 101, 76 to 88 and 125 to 147, that of 8 nodes over 512 tokens from 8.9 to 9.3.
#include <limits.h>
#include <math.h>

#include <atomic>
#include <type_traits>

#include "dec_device.cuh"
#include "dec_launch.h"
#include "tcgen05.cuh"

namespace decattn {
namespace {

constexpr int kTile = 64;      // keys per tile
constexpr int kRows = 128;     // query rows per tile (the MMA's M)
constexpr int kThreads = 192;  // 4 softmax warps, the TMA warp, the MMA warp
constexpr int kSoftmax = 128;
constexpr float kLargeCap = 256.f;
constexpr float kFar = 0x1p24f;   // maxima past this are subtracted before the scale is applied
constexpr float kRescale = 8.f;  // log2 of the growth of the maximum that moves it
constexpr int kMaxRowTiles = kTreeMaxNodes * kSplitMaxG / kRows;
// What beginning and ending a (pair, row tile) costs, in key tiles: the stream is cut by tiles
// plus this, so that CTAs with many short sequences finish with the others. (Short single-token
// sequences of 64 dims: 3 78.6 us, 4 74.7, 6 73.7; wide trees 128.1, 124.9, 123.9; one long
// sequence, cut evenly by any, 94.9, 95.4, 97.1.)
constexpr int kSegment = 6;
constexpr uint32_t kTmemCols = 256;
constexpr uint32_t kOCol = 2 * kTile;  // S/P buffers in columns [0, 128), O behind them

template <int D>
struct Geo {
  static constexpr int kSlabs = D / 64;                 // 128-byte swizzle slabs per row
  static constexpr int kSlab = kTile * 128;             // one slab of a key tile
  static constexpr int kTensor = kSlabs * kSlab;        // a K or a V tile
  static constexpr int kQ = kSlabs * kRows * 128;
  static constexpr int kStages = D == 128 ? 4 : 8;
  static constexpr size_t kSmem = 1024 + kQ + (size_t)kStages * kTensor;
};

// Partial slots: piece c leaves at most two, its first segment (slot 2c, when that began in
// an earlier piece) and its last (slot 2c + 1, when it goes on in a later one). A slot holds
// O [D / 8][128 rows][8] fp32 and (maximum, sum) [128 rows]. Records, one per (pair, row
// tile), written by the CTA that begins it: the pieces it lies in.
struct alignas(16) Record {
  int first, last;  // the same: nothing to merge
  int pad[2];
};

__host__ __device__ inline size_t slot_bytes(int D) { return (size_t)kRows * (D * 4 + 8); }
__host__ __device__ inline size_t records_offset() { return kWsHeaderBytes; }
__host__ __device__ inline size_t slots_offset(int records) {
  return (records_offset() + (size_t)records * sizeof(Record) + 255) & ~(size_t)255;
}

// A sequence's share of the stream.
struct Seq {
  int L, live, start, tiles, mt;
};

__device__ __forceinline__ Seq seq_of(const TreeAttnArgs &a, int b, bool report) {
  Seq s;
  const int L = a.lens[b], n = a.n_nodes != nullptr ? a.n_nodes[b] : a.N;
  s.L = min(max(L, 0), a.T_cap);
  s.live = min(max(n, 0), a.N);
  if (report) {
    if (s.L != L) atomicOr(a.error_word, kErrLenClamped);
    if (s.live != n) atomicOr(a.error_word, kErrTreeClamped);
  }
  // every node's position is at least L, so with a window no node sees below this slot
  s.start = a.window > 0 ? min(s.L, max(0, s.L - a.window + 1)) : 0;
  s.tiles = s.live > 0 ? (s.L - s.start + kTile - 1) / kTile + 1 : 0;
  s.mt = (s.live * (a.Hq / a.Hkv) + kRows - 1) / kRows;
  return s;
}

// The segments of a piece: runs of key tiles [t0, t1) of one (sequence, KV head) and row tile
// m. The stream of row tile m has kSegment + tiles units per (sequence, KV head), in order; the
// first kSegment stand for work that is not a tile. All pieces of a row tile come one after
// the other: the CTAs of different row tiles then walk the same keys at the same time and
// share them through L2.
struct Walk {
  Seq s;
  int b, g, m, t0, t1, left, off;  // off: first unit of this (sequence, KV head)
  __device__ __forceinline__ void take(int from) {  // from: units of this pair already behind
    t0 = max(0, from - kSegment);
    t1 = max(t0, min(s.tiles, from + left - kSegment));
    left -= t1 + kSegment - from;
  }
  // the piece of `units` from unit r0 on, `within` units into sequence b_; empty when t0 = t1
  __device__ __forceinline__ void begin(const TreeAttnArgs &a, int b_, int within, int units,
                                        int m_, int r0) {
    b = b_;
    m = m_;
    s = seq_of(a, b, false);
    const int per = s.tiles + kSegment;
    g = within / per;
    const int from = within - g * per;
    off = r0 - from;
    left = units;
    take(from);
  }
  __device__ __forceinline__ bool next(const TreeAttnArgs &a) {
    if (left <= kSegment) return false;
    off += s.tiles + kSegment;
    if (++g == a.Hkv) {
      g = 0;
      do s = seq_of(a, ++b, false);
      while (s.mt <= m);
    }
    take(0);
    return true;
  }
  __device__ __forceinline__ int rows(int G) const { return min(kRows, s.live * G - m * kRows); }
  // Key tile t: the cache's tiles from the newest tokens back (with a distance bias the maximum
  // then comes first and seldom moves), the tree's nodes last.
  __device__ __forceinline__ bool is_tree(int t) const { return t == s.tiles - 1; }
  __device__ __forceinline__ int token(int t) const { return s.start + (s.tiles - 2 - t) * kTile; }
};
// Lanes that share a row of the tile (see the kernel).
__device__ __forceinline__ int copies_of(int rows) { return rows <= 32 ? 4 : rows <= 64 ? 2 : 1; }

__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The smaller one; NaN if either is.
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// ---- tensor memory ---------------------------------------------------------------------
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t *r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, "
      "%30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t *r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, "
      "%29, %30, %31, %32};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]),
      "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
      "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_ld16_raw(uint32_t addr, uint32_t *r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(addr));
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t *r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t addr, const uint32_t *r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
      : "memory");
}
__device__ __forceinline__ void tmem_ld8(uint32_t addr, uint32_t *r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7])
      : "r"(addr));
}
// NC fp32 columns of this thread's lane; NC / 2 packed ones back, zeros over the other
// slices' part of the 32 packed columns.
template <int NC>
__device__ __forceinline__ void tmem_ld_cols(uint32_t addr, uint32_t *r) {
  if constexpr (NC == 64) {
    tmem_ld32(addr, r);
    tmem_ld32(addr + 32, r + 32);
  } else if constexpr (NC == 32) {
    tmem_ld32(addr, r);
  } else {
    tmem_ld16_raw(addr, r);
  }
}
template <int NC>
__device__ __forceinline__ void tmem_st_cols(uint32_t addr, const uint32_t *r) {
  if constexpr (NC == 32) {
    tmem_st32(addr, r);
  } else if constexpr (NC == 16) {
    tmem_st16(addr, r);
  } else {
    tmem_st8(addr, r);
  }
}
template <int NC>
__device__ __forceinline__ void tmem_st_weights(uint32_t addr, int slice, const uint32_t *pk) {
  if constexpr (NC == 64) {
    tmem_st32(addr, pk);
  } else if constexpr (NC == 32) {
    const uint32_t z[16] = {};
    tmem_st16(addr + (slice ^ 1) * 16, z);
    tmem_st16(addr + slice * 16, pk);
  } else {
    const uint32_t z[8] = {};
#pragma unroll
    for (int s = 1; s < 4; ++s) tmem_st8(addr + ((slice + s) & 3) * 8, z);
    tmem_st8(addr + slice * 8, pk);
  }
}
__device__ __forceinline__ uint32_t tmem_ld1(uint32_t addr) {
  uint32_t r;
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(r) : "r"(addr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
  return r;
}
__device__ __forceinline__ void tmem_wait_ld() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// One lane of a converged warp, the same one every time.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

// The MMAs with a descriptor in two halves: the low word (address and leading offset) is all
// that changes from one to the next, by an addition.
__device__ __forceinline__ void umma_bf16_ss(uint32_t tmem_d, uint32_t a_lo, uint32_t b_lo,
                                             uint32_t hi, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
      "mov.b64 a, {%1, %3};\n\tmov.b64 b, {%2, %3};\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n\t}" ::"r"(tmem_d),
      "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "r"(accumulate)
      : "memory");
}
// D[128 x N] (+)= A[128 x 16, tensor memory] B[16 x N]
__device__ __forceinline__ void umma_bf16_ts(uint32_t tmem_d, uint32_t tmem_a, uint32_t b_lo,
                                             uint32_t hi, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\t"
      "mov.b64 b, {%2, %3};\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}" ::"r"(tmem_d),
      "r"(tmem_a), "r"(b_lo), "r"(hi), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Descriptor halves of operands in 128-byte swizzle atoms (8 rows of 128 bytes). The high word:
// 1024 bytes from 8 rows to the next 8, the version bit, the swizzle mode. The low word: the
// address, and for an MN-major operand (V: tokens x dims) the leading offset, the step to the
// next 64 elements of MN (a K-major operand does not use it).
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lead) {
  return ((saddr >> 4) & 0x3FFFu) | ((lead >> 4) << 16);
}
constexpr uint32_t kBIsMnMajor = 1u << 16;  // instruction descriptor

// Bits [lo, hi) of a 64-bit word, for any lo and hi.
__device__ __forceinline__ uint64_t bit_range(int lo, int hi) {
  const uint64_t below_hi = hi >= 64 ? ~0ull : hi <= 0 ? 0ull : (1ull << hi) - 1;
  const uint64_t below_lo = lo >= 64 ? ~0ull : lo <= 0 ? 0ull : (1ull << lo) - 1;
  return below_hi & ~below_lo;
}

// A store of 8 consecutive floats.
__device__ __forceinline__ void st_v8(float *p, const float *r) {
  asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(r[0]),
               "f"(r[1]), "f"(r[2]), "f"(r[3]), "f"(r[4]), "f"(r[5]), "f"(r[6]), "f"(r[7])
               : "memory");
}

// ---- clusters ----------------------------------------------------------------------------
constexpr int kJoinCtas = 8;  // CTAs of a cluster at most
__device__ __forceinline__ void ld_cluster_f32x2(uint32_t addr, float &x, float &y) {
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(x), "=f"(y) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ld_cluster_f32x4(uint32_t addr, float (&x)[4]) {
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3])
               : "r"(addr)
               : "memory");
}
// Where 4 columns of a row of a CTA's partial lie: a row's chunks in an order of its own, so that
// neither rows nor columns meet in a bank.
template <int D>
__device__ __forceinline__ uint32_t part_at(int row, int chunk) {
  return (uint32_t)((row * (D / 4) + (chunk ^ (row & (D / 4 - 1)))) * 16);
}

struct TreeMaps {
  CUtensorMap k, v, kt, vt;
};

// What a waiting thread needs to give up: the shared abort flag and the error word.
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
};

// What the scores go through: nothing, a distance bias, or a cap (and a bias where slopes are
// given). Kernels of their own, for the registers and for the code that a tile runs through: what
// does not stay in the instruction caches costs more than it computes. (171 sequences of 56 to
// 226 tokens, 47 nodes, cap and bias: 106 us with everything in one kernel, 80 now.)
enum Scores { kPlain, kBias, kCap };

// kJoin: short contexts in one launch. A cluster of CTAs has a (pair, row tile) to itself, its tiles
// dealt out evenly, and joins its partials through distributed shared memory.
template <int D, Scores kScores, bool kJoin>
__global__ void __launch_bounds__(kThreads, 2)
    tree_attn_kernel(const __grid_constant__ TreeMaps maps, const TreeAttnArgs a, int B,
                     int mts_or_ctas, uint8_t *workspace) {
  using G = Geo<D>;
  constexpr int S = G::kStages;
  constexpr bool kMod = kScores != kPlain;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t s_bar[2 * S + 10];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  __shared__ int s_sum[kThreads / 32][kMaxRowTiles], s_begin[5];
  __shared__ float2 s_ml[kSoftmax];
  __shared__ unsigned long long s_odd;  // nodes with values that are not finite

  uint8_t *smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  const uint32_t q_s = smem_addr(smem), ring = q_s + G::kQ;
  const uint32_t bar_full = smem_addr(s_bar), bar_empty = bar_full + 8 * S;
  const uint32_t bar_s = bar_empty + 8 * S, bar_p = bar_s + 16, bar_pv = bar_p + 16;
  const uint32_t bar_q = bar_pv + 16, bar_end = bar_q + 8, bar_x = bar_end + 8, bar_v = bar_x + 8;
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int P = gridDim.x, piece = blockIdx.x, mts = kJoin ? mts_or_ctas & 255 : mts_or_ctas;

  if (tid == 5 * 32) {  // (the warps begin with different things)
    for (int i = 0; i < 2 * S; ++i) mbar_init(bar_full + 8 * i, 1);
    mbar_init(bar_s, 1);
    mbar_init(bar_s + 8, 1);
    mbar_init(bar_p, kSoftmax);
    mbar_init(bar_p + 8, kSoftmax);
    mbar_init(bar_pv, 1);
    mbar_init(bar_pv + 8, 1);
    mbar_init(bar_q, kSoftmax);
    mbar_init(bar_end, 1);
    mbar_init(bar_x, kSoftmax);
    mbar_init(bar_v, 1);
    s_abort = 0;
    fence_barrier_init();
  }
  if (warp == 4 && lane == 0) {
    tma_prefetch_desc(&maps.k);
    tma_prefetch_desc(&maps.v);
    tma_prefetch_desc(&maps.kt);
    tma_prefetch_desc(&maps.vt);
  }
  if (warp == 4) tmem_alloc(smem_addr(&s_tmem), kTmemCols);
  // the lengths and node counts, 32 to a line, on their way into L2
  if (tid * 32 < B) {
    asm volatile("prefetch.global.L2 [%0];" ::"l"(a.lens + tid * 32));
    if (a.n_nodes != nullptr) asm volatile("prefetch.global.L2 [%0];" ::"l"(a.n_nodes + tid * 32));
  }
  pdl_wait_prior_grid();
  pdl_launch_dependents();

  int p0 = 0, blk = 1;
  if constexpr (!kJoin) {
    // ---- where this CTA's piece begins: the units of every row tile m, the CTAs each m gets in
    // proportion, and a scan over the sequences for this CTA's m. Up to 32 sequences every warp
    // scans for itself, a lane each.
    const bool few = B <= 32;
    const int per = few ? 1 : (B + kThreads - 1) / kThreads;
    const int b_first = few ? lane : tid * per;
    int mine[kMaxRowTiles] = {}, m_total[kMaxRowTiles], m_before[kMaxRowTiles] = {};
    for (int b = b_first; b < min(B, b_first + per); ++b) {
      const Seq s = seq_of(a, b, piece == 0 && (!few || warp == 0));
#pragma unroll
      for (int m = 0; m < kMaxRowTiles; ++m)
        if (m < s.mt) mine[m] += (s.tiles + kSegment) * a.Hkv;
    }
#pragma unroll
    for (int m = 0; m < kMaxRowTiles; ++m)
      m_total[m] = m < mts ? __reduce_add_sync(0xffffffffu, mine[m]) : 0;
    if (!few) {
#pragma unroll
      for (int m = 0; m < kMaxRowTiles; ++m)
        if (lane == 0) s_sum[warp][m] = m_total[m];
      __syncthreads();
#pragma unroll
      for (int m = 0; m < kMaxRowTiles; ++m) {
        m_total[m] = 0;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) {
          if (w < warp) m_before[m] += s_sum[w][m];
          m_total[m] += s_sum[w][m];
        }
      }
    }
    int my_m = -1, total = 0, pieces = P, before = 0, count = 0;
    if (mts == 1) {
      my_m = 0;
      total = m_total[0];
      before = m_before[0];
      count = mine[0];
    } else {
      long long all = 0;
#pragma unroll
      for (int m = 0; m < kMaxRowTiles; ++m) all += m_total[m];
      int at = 0;
#pragma unroll
      for (int m = 0; m < kMaxRowTiles; ++m)
        if (m < mts) {
          const int n = 1 + (all > 0 ? (int)((long long)(P - mts) * m_total[m] / all) : 0);
          if (piece >= at && piece < at + n) {
            my_m = m;
            p0 = at;
            pieces = n;
            total = m_total[m];
            before = m_before[m];
            count = mine[m];
          }
          at += n;
        }
    }
    blk = max(1, (total + pieces - 1) / pieces);
    const int r0 = (int)min((long long)total, (long long)(piece - p0) * blk);
    const int units = min(blk, total - r0);
    const bool none = my_m < 0 || units <= 0;  // past the end of the stream
    int incl = count;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    const int excl = before + incl - count;
    const bool here = !none && excl <= r0 && r0 < excl + count;
    if (few) {
      const unsigned who = __ballot_sync(0xffffffffu, here);
      const int b = who != 0 ? __ffs(who) - 1 : 0;
      const int at = __shfl_sync(0xffffffffu, excl, b);
      if (tid == 0) {
        s_begin[0] = b;
        s_begin[1] = r0 - at;
      }
    } else if (here) {
      int at = excl, b = b_first;
      for (;; ++b) {
        const Seq s = seq_of(a, b, false);
        const int u = my_m < s.mt ? (s.tiles + kSegment) * a.Hkv : 0;
        if (r0 < at + u) break;
        at += u;
      }
      s_begin[0] = b;
      s_begin[1] = r0 - at;
    }
    // through shared memory, so that the compiler knows them to be the same in every lane (an
    // MMA issued with operands that might differ costs several times as much)
    if (tid == 0) {
      s_begin[2] = units;
      s_begin[3] = my_m;
      s_begin[4] = r0;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, s_tmem, 0);
  Walk w;
  bool idle, empty = false;  // empty: no tiles, but a cluster to join
  int rank = 0, ctas = 1;
  if constexpr (kJoin) {
    ctas = mts_or_ctas >> 8;
    rank = piece % ctas;
    const int pair = piece / ctas / mts;
    w.m = piece / ctas % mts;
    w.b = pair / a.Hkv;
    w.g = pair - w.b * a.Hkv;
    w.s = seq_of(a, w.b, tid == 0 && rank == 0 && w.m == 0 && w.g == 0);
    w.t0 = w.s.tiles * rank / ctas;
    w.t1 = w.s.tiles * (rank + 1) / ctas;
    w.left = w.off = 0;
    idle = w.m >= w.s.mt;  // all of the cluster
    empty = w.t0 == w.t1;
  } else {
    idle = s_begin[3] < 0 || s_begin[2] <= 0;
    if (!idle) {
      w.begin(a, s_begin[0], s_begin[1], s_begin[2], s_begin[3], s_begin[4]);
      // a piece of nothing but the units before a first tile; the next one begins it
      if (w.t0 == w.t1) idle = true;
    }
  }
  if (idle) {
    if (warp == 4) tmem_dealloc(tmem, kTmemCols);
    return;
  }
  const int Gq = a.Hq / a.Hkv;
  const int records = B * a.Hkv * mts;
  const Waiter wait{&s_abort, a.error_word};
  const bool split = kJoin && ctas > 1;  // this (pair, row tile) over a cluster

  if (empty) {
    if (tid < kRows) s_ml[tid] = make_float2(-INFINITY, 0.f);
  } else if (warp == 4) {
    // ---------------------------------------------------------------- loads
    if (lane == 0) {
      int it = 0;
      bool ok = true;
      do {
        // a pair with one row tile is read once; with more, the others find it in L2
        const uint64_t policy = w.s.mt == 1 ? l2_policy_evict_first() : l2_policy_evict_normal();
        const int pair = w.b * a.Hkv + w.g;
        for (int t = w.t0; t < w.t1 && ok; ++t) {
          const bool tree = w.is_tree(t);
          const int row = tree ? 0 : w.token(t);
#pragma unroll
          for (int kv = 0; kv < 2; ++kv, ++it) {
            const int slot = it % S;
            if (it >= S && !wait(bar_empty + 8 * slot, (it / S - 1) & 1)) {
              ok = false;
              break;
            }
            const CUtensorMap *map = tree ? (kv ? &maps.vt : &maps.kt) : (kv ? &maps.v : &maps.k);
            const uint32_t full = bar_full + 8 * slot, dst = ring + slot * G::kTensor;
            mbar_arrive_expect_tx(full, G::kTensor);
#pragma unroll
            for (int sl = 0; sl < G::kSlabs; ++sl)
              tma_load_3d(dst + sl * G::kSlab, map, sl * 64, row, pair, full, policy);
          }
        }
      } while (ok && w.next(a));
      if (!ok)  // no copy into this CTA's shared memory may outlive it
        for (int j = max(0, it - S); j < it; ++j)
          mbar_wait_bounded(bar_full + 8 * (j % S), (j / S) & 1);
    }
  } else if (warp == 5) {
    // ---------------------------------------------------------------- MMAs
    // The warp stays together and one elected lane issues: every operand is then the same across
    // the warp as far as the compiler can tell (under `lane == 0` an MMA took 65 cycles to
    // issue).
    constexpr uint32_t idesc_s = idesc_bf16_f32(kRows, kTile);
    constexpr uint32_t idesc_o = idesc_bf16_f32(kRows, D) | kBIsMnMajor;
    const uint32_t q_lo = desc_lo(q_s, 16), k_lo = desc_lo(ring, 16), v_lo = desc_lo(ring, G::kSlab);
    int n = 0, seg = 0;
    bool ok = true;
    auto wait_all = [&](uint32_t bar, uint32_t parity) {
      return __all_sync(0xffffffffu, wait(bar, parity) ? 1 : 0) != 0;
    };
    auto issue_s = [&](int i) {
      const int it = 2 * i, slot = it % S;
      // the buffer's last P, that of tile i - 2, is consumed
      if (i >= 2 && !wait_all(bar_pv + 8 * (i & 1), ((i - 2) >> 1) & 1)) return false;
      if (!wait_all(bar_full + 8 * slot, (it / S) & 1)) return false;
      tc_fence_after();
      const uint32_t k_at = k_lo + slot * (G::kTensor >> 4), d = tmem + (i & 1) * kTile;
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          umma_bf16_ss(d, q_lo + (k >> 2) * (kRows * 128 >> 4) + 2 * (k & 3),
                       k_at + (k >> 2) * (G::kSlab >> 4) + 2 * (k & 3), kDescHi, idesc_s, k > 0);
        umma_commit(bar_empty + 8 * slot);
        umma_commit(bar_s + 8 * (i & 1));
      }
      __syncwarp();
      return true;
    };
    // Rows of V that nobody may read can hold anything, and 0 times NaN is NaN: they are
    // cleared in shared memory.
    auto clear_rows = [&](uint32_t v_s, int from, int to) {
      for (int i = lane; i < (to - from) * (D / 8); i += 32) {
        const int r = from + i / (D / 8), ch = i % (D / 8);
        asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(
                         v_s + (ch >> 3) * G::kSlab + r * 128 + ((ch & 7) << 4)),
                     "r"(0u)
                     : "memory");
      }
    };
    // In the tree's tile, besides the rows behind the last node, the nodes that no row sees, and
    // single values that are not finite: the rows that do see those get them back at the end.
    // Returns their nodes.
    auto clear_tree = [&](uint32_t v_s, uint64_t used, int live) {
      clear_rows(v_s, live, a.N);  // (behind a.N the copy left zeros)
      uint64_t odd = 0;
      if (used == bit_range(0, live)) {  // and most often all there is to do: 0 x is 0, or NaN
        __nv_bfloat162 sum = __float2bfloat162_rn(0.f);
#pragma unroll 8
        for (int i = lane; i < live * (D / 8); i += 32) {
          const int r = i / (D / 8), ch = i % (D / 8);
          uint32_t x[4];
          asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
                       : "r"(v_s + (ch >> 3) * G::kSlab + r * 128 + ((ch & 7) << 4)));
#pragma unroll
          for (int k = 0; k < 4; ++k)
            sum = __hfma2(reinterpret_cast<const __nv_bfloat162 &>(x[k]),
                          __float2bfloat162_rn(0.f), sum);
        }
        if (!__any_sync(0xffffffffu, __hisnan(sum.x) || __hisnan(sum.y))) return odd;
      }
#pragma unroll 4
      for (int i = lane; i < live * (D / 8); i += 32) {
        const int r = i / (D / 8), ch = i % (D / 8);  // (any order within a row serves)
        const uint32_t at = v_s + (ch >> 3) * G::kSlab + r * 128 + ((ch & 7) << 4);
        uint32_t x[4];
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
                     : "r"(at));
        const bool clear = !((used >> r) & 1);
        bool bad = false;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if ((x[k] & 0x7f80u) == 0x7f80u) x[k] &= 0xffff0000u, bad = true;
          if ((x[k] & 0x7f800000u) == 0x7f800000u) x[k] &= 0xffffu, bad = true;
          if (clear) x[k] = 0;
        }
        if (bad && !clear) odd |= 1ull << r;
        if (bad || clear)
          asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(x[0]),
                       "r"(x[1]), "r"(x[2]), "r"(x[3])
                       : "memory");
      }
      return (uint64_t)__reduce_or_sync(0xffffffffu, (uint32_t)(odd >> 32)) << 32 |
             __reduce_or_sync(0xffffffffu, (uint32_t)odd);
    };
    do {
      const int cnt = w.t1 - w.t0;
      uint64_t used = 0;  // nodes that some row sees
      if (w.t1 == w.s.tiles) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (lane + 32 * h < w.s.live) used |= a.mask[(size_t)w.b * a.N + lane + 32 * h];
        used = ((uint64_t)__reduce_or_sync(0xffffffffu, (uint32_t)(used >> 32)) << 32 |
                __reduce_or_sync(0xffffffffu, (uint32_t)used)) &
               bit_range(0, w.s.live);
      }
      // With a window, the first cached row that some node sees: later than the segment's first
      // when every node lies past the sequence's length.
      int least = INT_MAX;
      if (a.window > 0) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (lane + 32 * h < w.s.live) least = min(least, a.pos[(size_t)w.b * a.N + lane + 32 * h]);
      }
      ok = ok && wait_all(bar_q, seg & 1) && issue_s(n);
      const int first_seen =
          a.window > 0 ? max(0, max(__reduce_min_sync(0xffffffffu, least), w.s.L) - a.window + 1) : 0;
      for (int i = 0; i < cnt && ok; ++i) {
        const int it = 2 * (n + i) + 1, slot = it % S, t = w.t0 + i;
        if (i + 1 < cnt) ok = issue_s(n + i + 1);
        ok = ok && wait_all(bar_full + 8 * slot, (it / S) & 1);
        if (!ok) break;
        const bool tree = w.is_tree(t);
        const int valid = w.s.L - w.token(t), unseen = first_seen - w.token(t);
        if (tree || valid < kTile || unseen > 0) {
          const uint32_t v_s = ring + slot * G::kTensor;
          if (tree) {
            const uint64_t odd = clear_tree(v_s, used, w.s.live);
            if (lane == 0) s_odd = odd;
          } else {
            clear_rows(v_s, 0, min(unseen, kTile));
            clear_rows(v_s, valid, kTile);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (tree && lane == 0) mbar_arrive(bar_v);
          __syncwarp();
        }
        ok = wait_all(bar_p + 8 * ((n + i) & 1), ((n + i) >> 1) & 1);
        if (!ok) break;
        tc_fence_after();
        const uint32_t v_at = v_lo + slot * (G::kTensor >> 4), p = tmem + ((n + i) & 1) * kTile;
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < kTile / 16; ++k)
            umma_bf16_ts(tmem + kOCol, p + 8 * k, v_at + k * (2048 >> 4), kDescHi, idesc_o,
                         i > 0 || k > 0);
          umma_commit(bar_empty + 8 * slot);
          umma_commit(bar_pv + 8 * ((n + i) & 1));
        }
        __syncwarp();
      }
      n += cnt;
      ++seg;
    } while (ok && w.next(a));
    if (!ok) {  // let what was issued finish before tensor memory is given back
      __syncwarp();
      if (elect_one()) umma_commit(bar_end);
      __syncwarp();
      mbar_wait_bounded(bar_end, 0);
    }
  } else {
    // ---------------------------------------------------------------- softmax
    const uint32_t my_tmem = tmem + ((uint32_t)(32 * warp) << 16);
    const float log2e = 1.4426950408889634f;
    const float sc = kMod ? 1.f : a.scale * log2e;
    int n = 0, seg = 0, x_phase = 0, trees = 0;
    bool ok = true;
    // the same answer in every lane, and the warp together behind it
    auto wait_all = [&](uint32_t bar, uint32_t parity) {
      return __all_sync(0xffffffffu, wait(bar, parity) ? 1 : 0) != 0;
    };
    auto q_row = [&](const Walk &v, int row) {
      const int node = row / Gq;
      return a.q + (((size_t)v.b * a.N + node) * a.Hq + (size_t)v.g * Gq + (row - node * Gq)) * D;
    };
    // this thread's row of Q into shared memory, K-major with the 128-byte swizzle
    auto load_q = [&](const Walk &v) {
      const int row = v.m * kRows + (tid & (kRows / copies_of(v.rows(Gq)) - 1)), node = row / Gq;
      const bool real = node < v.s.live;
      const uint4 *src = reinterpret_cast<const uint4 *>(q_row(v, row));
#pragma unroll
      for (int h = 0; h < D / 64; ++h) {
        uint4 x[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) x[c] = real ? src[h * 8 + c] : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int c = 0; c < 8; ++c)
          asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(
                           q_s + h * (kRows * 128) + tid * 128 + ((c ^ (tid & 7)) << 4)),
                       "r"(x[c].x), "r"(x[c].y), "r"(x[c].z), "r"(x[c].w)
                       : "memory");
      }
      fence_proxy_async_smem();
      mbar_arrive(bar_q);
    };
    // the same in two steps, the copies in flight between them
    auto start_q = [&](const Walk &v) {
      const int row = v.m * kRows + (tid & (kRows / copies_of(v.rows(Gq)) - 1)), node = row / Gq;
      const bool real = node < v.s.live;
      const __nv_bfloat16 *src = real ? q_row(v, row) : a.q;  // (16 bytes or none are read)
      const int bytes = real ? 16 : 0;
#pragma unroll
      for (int c = 0; c < D / 8; ++c)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                         q_s + (c >> 3) * (kRows * 128) + tid * 128 + (((c ^ tid) & 7) << 4)),
                     "l"(src + c * 8), "r"(bytes)
                     : "memory");
    };
    auto finish_q = [&] {
      asm volatile("cp.async.wait_all;" ::: "memory");
      fence_proxy_async_smem();
      mbar_arrive(bar_q);
    };
    load_q(w);
    bool more = true;
    while (more) {
      const int rows = w.rows(Gq), copies = copies_of(rows);
      const int my_row = tid & (kRows / copies - 1);      // within the row tile
      const int slice = tid / (kRows / copies);
      const int row = w.m * kRows + my_row, node = row / Gq, hi = row - node * Gq;
      const bool real = my_row < rows, active = copies > 1 || 32 * warp < rows;
      const size_t brow = (size_t)w.b * a.N;
      const bool has_tree = w.t1 == w.s.tiles;
      // what the tree's tile needs, on its way early: this row's ancestors, and two nodes'
      // positions per lane
      const uint64_t my_mask =
          has_tree && real ? a.mask[brow + node] & bit_range(0, w.s.live) : 0;
      const bool by_distance = a.window > 0 || (kMod && a.slopes != nullptr);
      int npos[2] = {};
      if (has_tree && by_distance) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (lane + 32 * h < w.s.live) npos[h] = max(a.pos[brow + lane + 32 * h], w.s.L);
      }
      const int qpos = real && by_distance ? max(a.pos[brow + node], w.s.L) : 0;
      const int low = real && a.window > 0 ? qpos - a.window + 1 : 0;  // first slot in the window
      const int low_max = __reduce_max_sync(0xffffffffu, low);
      float slope = 0.f;
      if constexpr (kMod)
        if (real && a.slopes != nullptr) slope = a.slopes[w.g * Gq + hi] * log2e;
      // what the common transformation adds to keys 0 to 7 of any 8: the cap, and the bias from
      // one to the next
      uint64_t off2[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float cap = kScores == kCap ? a.softcap * log2e : 0.f;
        off2[k] = pair_of(fmaf(slope, 2.f * k, cap), fmaf(slope, 2.f * k + 1.f, cap));
      }
      float m = -INFINITY, l = 0.f;
      // Plain scores are scaled within the exponent, z sc - m. Where |m| is past 2^24 the rounding of
      // m = z_max sc moves exponents by 1 and more (past 2^31 out of range): z_max, for those rows.
      float far = 0.f;
      bool any_far = false;
      // the segment after this one, and its Q on the way into L2
      Walk after = w;
      more = after.next(a);
      if (more) {
        const int r = after.m * kRows + (tid & (kRows / copies_of(after.rows(Gq)) - 1));
        if (r / Gq < after.s.live) {
          const __nv_bfloat16 *src = q_row(after, r);
          asm volatile("prefetch.global.L2 [%0];" ::"l"(src));
          if (D == 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(src + 64));
        }
      }
      for (int t = w.t0; t < w.t1; ++t, ++n) {
        const bool tree = w.is_tree(t);
        const int t_abs = w.token(t);
        const uint32_t p_addr = my_tmem + (n & 1) * kTile;
        // the keys of the tile this row sees: all of them, in most tiles
        const bool all = !tree && t_abs + kTile <= w.s.L && low_max <= t_abs;
        uint64_t see = ~0ull;
        if (tree) {
          see = my_mask;
          if (a.window > 0)
            for (int j = 0; j < w.s.live; ++j) {
              const int at = __shfl_sync(0xffffffffu, j < 32 ? npos[0] : npos[1], j & 31);
              if (qpos - at >= a.window) see &= ~(1ull << j);
            }
        } else if (!all) {
          see = bit_range(low - t_abs, w.s.L - t_abs);
        }
        if (!wait_all(bar_s + 8 * (n & 1), (n >> 1) & 1)) {
          ok = false;
          break;
        }
        tc_fence_after();
        // kMod: a tile whose keys need more than the common transformation gets its scores bent
        // in tensor memory first, 8 keys at a time. Unrolled with the rest for every key, that
        // code would not stay in the instruction caches (it cost the common tiles half their
        // time).
        const bool bent = (kScores == kCap && (a.softcap > kLargeCap || !all)) ||
                          (kMod && tree && a.slopes != nullptr);
        auto bend = [&](int from, int count) {
          const int keys = tree ? w.s.live : w.s.L - t_abs;
          const float inv = a.scale / a.softcap;
#pragma unroll 1
          for (int c = from; c < min(from + count, keys); c += 8) {  // (the others are masked)
            uint32_t raw[8];
            tmem_ld8(p_addr + c, raw);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              float z = __uint_as_float(raw[i]);
              if (kScores == kCap) {
                // tanh by its series below 0.3 (next term 9e-3 x^11): 1 - 2 / (1 + e^(2 x)) is off
                // by about 2^-22 of 1, too much of a small x under a large cap
                const float x = z * inv, x2 = x * x;
                const float near =
                    x * fmaf(x2, fmaf(x2, fmaf(x2, fmaf(x2, 62.f / 2835.f, -17.f / 315.f),
                                               2.f / 15.f),
                                      -1.f / 3.f),
                             1.f);
                const float far = fmaf(-2.f, rcp(1.f + ex2(x * (2.f * log2e))), 1.f);
                z = a.softcap * log2e * (fabsf(x) < 0.3f ? near : far);
              } else {
                z *= a.scale * log2e;
              }
              if (a.slopes != nullptr) {
                const int j = c + i;  // the same in every lane of the warp
                const int at = tree ? __shfl_sync(0xffffffffu, j < 32 ? npos[0] : npos[1], j & 31)
                                    : t_abs + j;
                if (!tree || j < w.s.live) z = fmaf(-slope, (float)(qpos - at), z);
              }
              raw[i] = __float_as_uint(z);
            }
            tmem_st8(p_addr + c, raw);
          }
          tmem_wait_st();
        };
        // the last S of the segment is there: Q's space is free, unless a join needs it first
        if (__builtin_expect(t + 1 == w.t1 && more && copies == 1, 0)) start_q(after);
        // this thread's scores of the keys from c0 on, as the softmax takes them
        auto scores = [&](auto &z, int c0) {
          constexpr int NC = sizeof(z) / 4;
          uint32_t raw[NC];
          tmem_ld_cols<NC>(p_addr + c0, raw);
          tmem_wait_ld();
#pragma unroll
          for (int c = 0; c < NC; ++c) z[c] = __uint_as_float(raw[c]);
          if constexpr (kMod) {
            if (!bent) {
              if constexpr (kScores == kCap) {
                // cap tanh(x / cap) = cap - 2 cap / (1 + e^(2 x / cap)), off by about 2^-20 cap
                // Four keys share a reciprocal, 1 / a = c (b d / (a c b d)). Past 2^30 the result
                // is the cap, and the product of four stays finite. (The row sees every
                // key here: one that is NaN may reach the other three.)
                const float in = 2.f * log2e * a.scale / a.softcap, cap = a.softcap * log2e;
                const uint64_t in2 = pair_of(in, in), one2 = pair_of(1.f, 1.f);
                const uint64_t minus2 = pair_of(-2.f * cap, -2.f * cap);
#pragma unroll
                for (int c = 0; c < NC; c += 4) {
                  uint64_t d[2];
#pragma unroll
                  for (int i = 0; i < 2; ++i) {
                    float x0, x1;
                    unpair(mul2(pair_of(z[c + 2 * i], z[c + 2 * i + 1]), in2), x0, x1);
                    d[i] = add2(pair_of(ex2(min_nan(x0, 30.f)), ex2(min_nan(x1, 30.f))), one2);
                  }
                  float ac, bd;
                  unpair(mul2(d[0], d[1]), ac, bd);
                  const float r = rcp(ac * bd);
                  const uint64_t part = pair_of(r * bd, r * ac);
                  unpair(fma2(minus2, mul2(part, d[1]), off2[(c / 2) & 3]), z[c], z[c + 1]);
                  unpair(fma2(minus2, mul2(part, d[0]), off2[(c / 2 + 1) & 3]), z[c + 2], z[c + 3]);
                }
              } else {
                const uint64_t by2 = pair_of(a.scale * log2e, a.scale * log2e);
#pragma unroll
                for (int c = 0; c < NC; c += 2)
                  unpair(fma2(pair_of(z[c], z[c + 1]), by2, off2[(c / 2) & 3]), z[c], z[c + 1]);
              }
              if (kScores == kBias || a.slopes != nullptr) {
                // (slope times the key's place among 8 is in off2)
                const float far = (float)(qpos - t_abs - c0);
                const uint64_t slope2 = pair_of(-slope, -slope);
#pragma unroll
                for (int c = 0; c < NC; c += 2)
                  unpair(fma2(slope2, pair_of(far - (float)(c & ~7), far - (float)(c & ~7)),
                              pair_of(z[c], z[c + 1])),
                         z[c], z[c + 1]);
              }
            }
          }
          if (!all) {
            const uint64_t mine = see >> c0;
            const uint32_t s0 = (uint32_t)mine, s1 = (uint32_t)(mine >> 32);
#pragma unroll
            for (int c = 0; c < NC; ++c)
              if (!(((c < 32 ? s0 : s1) >> (c & 31)) & 1u)) z[c] = -INFINITY;
          }
        };
        auto largest = [&](const auto &z) {
          constexpr int NC = sizeof(z) / 4;
          float m4[4] = {z[0], z[1], z[2], z[3]};  // four chains, for the latency
#pragma unroll
          for (int c = 4; c < NC; c += 8)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              m4[i] = c + 4 + i < NC ? fmaxf(m4[i], fmaxf(z[c + i], z[c + 4 + i]))
                                        : fmaxf(m4[i], z[c + i]);
          return fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
        };
        // the running maximum for a tile whose largest score is z_max
        auto settle = [&](float z_max) {
          const float mx = z_max * sc;
          const bool grow = mx > m + kRescale || (m == -INFINITY && mx > m);
          if (__any_sync(0xffffffffu, grow)) {
            const float mn = grow ? mx : m;
            if constexpr (!kMod) {
              if (grow) far = fabsf(mx) > kFar ? z_max : 0.f;
              any_far = __any_sync(0xffffffffu, far != 0.f);
            }
            const float corr = mn == -INFINITY ? 1.f : ex2(m - mn);
            m = mn;
            l *= corr;
            if (t > w.t0) {  // O holds the tiles before this one
              if (!wait_all(bar_pv + 8 * ((n - 1) & 1), ((n - 1) >> 1) & 1)) ok = false;
              tc_fence_after();
#pragma unroll 1
              for (int c = 0; c < D; c += 32) {
                uint32_t o[32];
                tmem_ld32(my_tmem + kOCol + c, o);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * corr);
                tmem_st32(my_tmem + kOCol + c, o);
              }
            }
          }
        };
        // the weights as bf16, their sum to l
        auto weights = [&](auto &z, auto &pk) {
          constexpr int NC = sizeof(z) / 4;
          float base = m == -INFINITY ? 0.f : m;
          if (!kMod && __builtin_expect(any_far, 0)) {
            if (far != 0.f) base = 0.f;
#pragma unroll
            for (int c = 0; c < NC; ++c) z[c] -= far;
          }
          const uint64_t sc2 = pair_of(sc, sc), base2 = pair_of(-base, -base);
          uint64_t l4[4] = {};
#pragma unroll
          for (int c = 0; c < NC; c += 2) {
            float x0, x1;
            unpair(fma2(pair_of(z[c], z[c + 1]), sc2, base2), x0, x1);
            const float p0 = ex2(x0), p1 = ex2(x1);
            l4[(c / 2) & 3] = add2(l4[(c / 2) & 3], pair_of(p0, p1));
            pk[c / 2] = pack_bf16x2(p0, p1);
          }
          float l0, l1;
          unpair(add2(add2(l4[0], l4[1]), add2(l4[2], l4[3])), l0, l1);
          l += l0 + l1;
        };
        auto at_once = [&](auto cols) {
          constexpr int NC = decltype(cols)::value;
          float z[NC];
          uint32_t pk[NC / 2];
          if (kMod && bent) bend(slice * NC, NC);
          scores(z, slice * NC);
          settle(largest(z));
          weights(z, pk);
          tmem_st_weights<NC>(p_addr, slice, pk);
          tmem_wait_st();
        };
        // With a cap a thread's keys go NC at a time, for the registers and the code's size: all but
        // the first chunk wait in tensor memory for the maximum, and come back in order, since
        // P lies over the first ones. NC divides the thread's kTile / copies keys.
        auto in_chunks = [&](auto cols) {
          constexpr int NC = decltype(cols)::value;
          const int span = kTile / copies, first = slice * span;
          float z[NC], mx = -INFINITY;
          uint32_t raw[NC];
          if (bent) bend(first, span);
#pragma unroll 1
          for (int c0 = span - NC;; c0 -= NC) {
            scores(z, first + c0);
            mx = fmaxf(mx, largest(z));
            if (c0 <= 0) break;
#pragma unroll
            for (int c = 0; c < NC; ++c) raw[c] = __float_as_uint(z[c]);
            tmem_st_cols<NC>(p_addr + first + c0, raw);
          }
          settle(mx);
          tmem_wait_st();
#pragma unroll 1
          for (int c0 = 0;; c0 += NC) {
            uint32_t pk[NC / 2];
            weights(z, pk);
            const bool last = c0 + NC >= span;
            if (!last) {
              tmem_ld_cols<NC>(p_addr + first + c0 + NC, raw);
              tmem_wait_ld();
#pragma unroll
              for (int c = 0; c < NC; ++c) z[c] = __uint_as_float(raw[c]);
            }
            tmem_st_cols<NC / 2>(p_addr + (first + c0) / 2, pk);
            if (last) break;
          }
          const uint32_t zero[8] = {};
#pragma unroll 1
          for (int c = 0; copies > 1 && c < kTile / 2; c += 8)  // the other slices' part
            if (2 * c / span != slice) tmem_st8(p_addr + c, zero);
          tmem_wait_st();
        };
        if constexpr (kScores == kCap) {
          if (copies == 4)
            in_chunks(std::integral_constant<int, 16>{});
          else if (active)
            in_chunks(std::integral_constant<int, 32>{});
        } else if (copies == 4) {
          at_once(std::integral_constant<int, 16>{});
        } else if (copies == 2) {
          at_once(std::integral_constant<int, 32>{});
        } else if (active) {
          at_once(std::integral_constant<int, 64>{});
        }
        tc_fence_before();
        mbar_arrive(bar_p + 8 * (n & 1));
      }
      if (!ok) break;
      // ---- the segment's end
      const Walk done = w;
      w = after;
      uint64_t odd = 0;
      if (has_tree) {
        if (!wait_all(bar_v, trees & 1)) break;
        ++trees;
        odd = *reinterpret_cast<volatile unsigned long long *>(&s_odd);
      }
      // the next segment's S may follow; P of the last tile must stay for the values to be given
      // back
      const bool early_q = more && odd == 0 && copies == 1;
      if (early_q) finish_q();
      if (!wait_all(bar_pv + 8 * ((n - 1) & 1), ((n - 1) >> 1) & 1)) break;
      tc_fence_after();
      const bool whole = kJoin ? !split : done.t0 == 0 && done.t1 == done.s.tiles;
      const int slot = 2 * piece + (done.t0 > 0 ? 0 : 1);
      float *part =
          reinterpret_cast<float *>(workspace + slots_offset(records) + (size_t)slot * slot_bytes(D));
      __nv_bfloat16 *dst = a.out + ((brow + node) * a.Hq + (size_t)done.g * Gq + hi) * D;
      // the values of nodes that are not finite, to the rows that see them
      auto give_back = [&](uint32_t (&o)[32], int c) {
        for (uint64_t left = odd; left != 0; left &= left - 1) {
          const int j = __ffsll((long long)left) - 1;
          const uint32_t pw = tmem_ld1(my_tmem + ((n - 1) & 1) * kTile + (j >> 1));
          const float p = (j & 1) ? bf16_hi(pw) : bf16_lo(pw);
          const bool sees = real && j / (kTile / copies) == slice && ((my_mask >> j) & 1) &&
                            !(a.window > 0 && qpos - max(a.pos[brow + j], done.s.L) >= a.window);
          const __nv_bfloat16 *v =
              a.v_tree + (((size_t)done.b * a.Hkv + done.g) * a.N + j) * D + c;
          if (sees)
            for (int i = 0; i < 32; ++i) {
              const float x = __bfloat162float(v[i]);
              if (!isfinite(x)) {
#pragma unroll
                for (int k = 0; k < 32; ++k)
                  if (k == i) o[k] = __float_as_uint(__uint_as_float(o[k]) + p * x);
              }
            }
          __syncwarp();
        }
      };
      auto store8 = [&](int col, const float *v) {  // 8 columns of this thread's row
        if (whole) {
          *reinterpret_cast<uint4 *>(dst + col) =
              make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                         pack_bf16x2(v[6], v[7]));
        } else if constexpr (kJoin) {  // the ring is free
#pragma unroll
          for (int i = 0; i < 2; ++i)
            asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(
                             ring + part_at<D>(my_row, col / 4 + i)),
                         "f"(v[4 * i]), "f"(v[4 * i + 1]), "f"(v[4 * i + 2]), "f"(v[4 * i + 3])
                         : "memory");
        } else {
          st_v8(part + ((size_t)(col / 8) * kRows + my_row) * 8, v);
        }
      };
      const bool aligned32 = (reinterpret_cast<uintptr_t>(a.out) & 31) == 0;
      auto store16 = [&](int col, const float *v) {
        if (whole && aligned32) {  // a sector at a time
          uint32_t x[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
          asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst + col),
                       "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]),
                       "r"(x[7])
                       : "memory");
        } else {
          store8(col, v);
          store8(col + 8, v + 8);
        }
      };
      if (copies == 1) {
        if (active) {
          const float scale = whole ? (l == 0.f ? 0.f : 1.f / l) : 1.f;
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            uint32_t o[32];
            tmem_ld32(my_tmem + kOCol + c, o);
            tmem_wait_ld();
            if (odd != 0) give_back(o, c);
            float v[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(o[i]) * scale;
            if (real) {
#pragma unroll
              for (int i = 0; i < 32; i += 16) store16(c + i, v + i);
            }
            __syncwarp();
          }
          if (!kJoin && !whole && real)
            reinterpret_cast<float2 *>(part + (size_t)kRows * D)[my_row] = make_float2(m, l);
          if (kJoin) s_ml[tid] = make_float2(m, l);
        }
      } else {
        // A row's keys were dealt to `copies` lanes, each with a maximum, sum and O of its
        // own: joined through Q's space (every S of the segment has been read), 32 columns
        // at a time, a lane taking 32 / copies of them.
        auto meet = [&] {
          mbar_arrive(bar_x);
          const bool here = wait_all(bar_x, x_phase & 1);
          ++x_phase;
          return here;
        };
        const int span = kRows / copies;
        constexpr int kCols = G::kQ / (kSoftmax * 4) < 64 ? G::kQ / (kSoftmax * 4) : 64;
        float weight[4] = {}, M = -INFINITY, L = 0.f;
        s_ml[tid] = make_float2(m, l);
        bool joined = true;
#pragma unroll 1
        for (int c = 0; c < D; c += kCols) {
          if (c > 0) joined = joined && meet();  // the space is free again
#pragma unroll
          for (int h = 0; h < kCols; h += 32) {
            uint32_t o[32];
            tmem_ld32(my_tmem + kOCol + c + h, o);
            tmem_wait_ld();
            if (odd != 0) give_back(o, c + h);
#pragma unroll
            for (int i = 0; i < 32; i += 4)
              asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                               q_s + (uint32_t)((h + i) / 4 * kSoftmax + tid) * 16),
                           "r"(o[i]), "r"(o[i + 1]), "r"(o[i + 2]), "r"(o[i + 3])
                           : "memory");
          }
          joined = joined && meet();
          if (!joined) break;
          if (c == 0) {
            float2 x[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
              x[k] = k < copies ? s_ml[my_row + k * span] : make_float2(-INFINITY, 0.f);
            M = fmaxf(fmaxf(x[0].x, x[1].x), fmaxf(x[2].x, x[3].x));
            const float base = M == -INFINITY ? 0.f : M;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              weight[k] = ex2(x[k].x - base);
              L += x[k].y * weight[k];
            }
            const float inv = whole ? (L == 0.f ? 0.f : 1.f / L) : 1.f;
#pragma unroll
            for (int k = 0; k < 4; ++k) weight[k] *= inv;
          }
          const int cols = kCols / copies;
          for (int i = slice * cols; i < (slice + 1) * cols; i += 8) {
            float4 x[4][2];
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (k < copies)
#pragma unroll
                for (int q = 0; q < 2; ++q)
                  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                               : "=f"(x[k][q].x), "=f"(x[k][q].y), "=f"(x[k][q].z),
                                 "=f"(x[k][q].w)
                               : "r"(q_s +
                                     (uint32_t)((i / 4 + q) * kSoftmax + my_row + k * span) * 16)
                               : "memory");
            float v[8] = {};
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (k < copies)
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                  v[4 * q] = fmaf(x[k][q].x, weight[k], v[4 * q]);
                  v[4 * q + 1] = fmaf(x[k][q].y, weight[k], v[4 * q + 1]);
                  v[4 * q + 2] = fmaf(x[k][q].z, weight[k], v[4 * q + 2]);
                  v[4 * q + 3] = fmaf(x[k][q].w, weight[k], v[4 * q + 3]);
                }
            if (real) store8(c + i, v);
          }
        }
        joined = joined && (!more || meet());
        if (!joined) break;
        if (!kJoin && !whole && real && slice == 0)
          reinterpret_cast<float2 *>(part + (size_t)kRows * D)[my_row] = make_float2(M, L);
        // (every lane has read its row's s_ml: there was a meeting since)
        if (kJoin && slice == 0) s_ml[my_row] = make_float2(M, L);
      }
      if (!kJoin && done.t0 == 0 && tid == 0) {
        Record r;
        r.first = piece;
        r.last = p0 + (done.off + kSegment + done.s.tiles - 1) / blk;
        r.pad[0] = r.pad[1] = 0;
        reinterpret_cast<Record *>(workspace +
                                   records_offset())[((size_t)done.b * a.Hkv + done.g) * mts + done.m] = r;
      }
      tc_fence_before();
      if (more && !early_q) {
        if (copies == 1)
          finish_q();
        else
          load_q(w);
      }
      ++seg;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");  // (after a wait that gave up)
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 4) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
  if constexpr (kJoin) {
    if (!split) return;
    // out = sum_c 2^(m_c - M) O_c / sum_c 2^(m_c - M) l_c over the cluster's CTAs: a thread's items
    // are 8 dims of a row, neighbouring threads in one row.
    cluster_sync();
    constexpr int kD8 = D / 8;
    const int rows = w.rows(Gq);
    const uint32_t ml = smem_addr(s_ml);
    for (int i = rank * kThreads + tid; i < rows * kD8; i += ctas * kThreads) {
      const int rr = i / kD8, d8 = i - rr * kD8, row = w.m * kRows + rr, node = row / Gq;
      float cm[kJoinCtas], cl[kJoinCtas], M = -INFINITY, L = 0.f, o[8] = {};
#pragma unroll
      for (int c = 0; c < kJoinCtas; ++c) {
        cm[c] = -INFINITY;
        cl[c] = 0.f;
        if (c < ctas) ld_cluster_f32x2(cluster_map(ml + rr * 8, c), cm[c], cl[c]);
        M = fmaxf(M, cm[c]);
      }
      const float base = M == -INFINITY ? 0.f : M;
#pragma unroll
      for (int c = 0; c < kJoinCtas; ++c)
        if (c < ctas && !(cl[c] == 0.f)) {  // (nothing was seen there: no O was left)
          const float f = ex2(cm[c] - base);
          L = fmaf(cl[c], f, L);
          const uint32_t at = cluster_map(ring, c);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float x[4];
            ld_cluster_f32x4(at + part_at<D>(rr, 2 * d8 + h), x);
#pragma unroll
            for (int k = 0; k < 4; ++k) o[4 * h + k] = fmaf(x[k], f, o[4 * h + k]);
          }
        }
      const float inv = L == 0.f ? 0.f : 1.f / L;
      *reinterpret_cast<uint4 *>(
          a.out + (((size_t)w.b * a.N + node) * a.Hq + (size_t)w.g * Gq + (row - node * Gq)) * D +
          d8 * 8) = make_uint4(pack_bf16x2(o[0] * inv, o[1] * inv), pack_bf16x2(o[2] * inv, o[3] * inv),
                               pack_bf16x2(o[4] * inv, o[5] * inv), pack_bf16x2(o[6] * inv, o[7] * inv));
    }
    cluster_sync();  // no CTA leaves while another reads its partial
  }
}

// Joins the partials of the (pair, row tile)s that cross pieces: out = sum_c 2^(m_c - M) O_c /
// sum_c 2^(m_c - M) l_c. CTA (x, y) takes kRowsPer rows of row tile x, a thread per (row, 8
// dims, every kGroups-th piece): 8 rows where a few long row tiles are cut into many pieces,
// 32 where many are cut in two. Attention and merge, us with 8 and with 32 rows, by pieces per
// row tile: 38 97 and 120; 13 71 and 81; 7.6 59 and 64; 4.2 54 and 57, 60.0 and 60.4; 2.1
// 109 and 108, 92 and 88; 0.6 141 and 124.
template <int D, int kRowsPer>
__global__ void __launch_bounds__(512) tree_merge_kernel(const uint8_t *workspace, int mts,
                                                         int records, int parts,
                                                         const TreeAttnArgs a) {
  constexpr int kD8 = D / 8, kGroups = 512 / (kRowsPer * kD8);
  static_assert(kGroups >= 1, "threads");
  __shared__ float s_o[kGroups > 1 ? kGroups : 1][kGroups > 1 ? kRowsPer : 1][D + 4];
  __shared__ float s_ml[kGroups][kRowsPer][2];
  pdl_launch_dependents();
  pdl_wait_prior_grid();
  const int m = blockIdx.x % mts, pair = blockIdx.x / mts, b = pair / a.Hkv, g = pair - b * a.Hkv;
  const Seq s = seq_of(a, b, false);
  if (m >= s.mt) return;  // no such row tile in this call, its record is an earlier one's
  const Record r = reinterpret_cast<const Record *>(workspace + records_offset())[blockIdx.x];
  const int row0 = blockIdx.y * kRowsPer;
  const int rows = min(kRows, s.live * (a.Hq / a.Hkv) - m * kRows);
  // (a record left by a launch that gave up is not trusted with addresses)
  if (r.first < 0 || r.first >= r.last || r.last >= parts || row0 >= rows) return;
  const int rr = threadIdx.x % kRowsPer, d8 = (threadIdx.x / kRowsPer) % kD8;
  const int grp = threadIdx.x / (kRowsPer * kD8), row = row0 + rr;
  const uint8_t *slots = workspace + slots_offset(records);
  float M = -INFINITY, l = 0.f, o[8] = {};
#pragma unroll 4
  for (int c = r.first + grp; c <= r.last; c += kGroups) {
    const float *p = reinterpret_cast<const float *>(
        slots + (size_t)(2 * c + (c == r.first ? 1 : 0)) * slot_bytes(D));
    const float2 ml = __ldcg(reinterpret_cast<const float2 *>(p + (size_t)kRows * D) + row);
    const float4 *src = reinterpret_cast<const float4 *>(p + ((size_t)d8 * kRows + row) * 8);
    const float4 x = __ldcg(src), y = __ldcg(src + 1);
    const float mn = fmaxf(M, ml.x);
    const float base = mn == -INFINITY ? 0.f : mn, f = ex2(M - base), e = ex2(ml.x - base);
    M = mn;
    l = l * f + ml.y * e;
    const float v[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = o[i] * f + v[i] * e;
  }
  if constexpr (kGroups > 1) {
#pragma unroll
    for (int i = 0; i < 8; ++i) s_o[grp][rr][d8 * 8 + i] = o[i];
    if (d8 == 0) {
      s_ml[grp][rr][0] = M;
      s_ml[grp][rr][1] = l;
    }
    __syncthreads();
    if (grp != 0) return;
    M = -INFINITY;
#pragma unroll
    for (int k = 0; k < kGroups; ++k) M = fmaxf(M, s_ml[k][rr][0]);
    const float base = M == -INFINITY ? 0.f : M;
    l = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = 0.f;
#pragma unroll
    for (int k = 0; k < kGroups; ++k) {
      const float e = ex2(s_ml[k][rr][0] - base);
      l += s_ml[k][rr][1] * e;
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] += s_o[k][rr][d8 * 8 + i] * e;
    }
  }
  if (row >= rows) return;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const int Gq = a.Hq / a.Hkv, q = m * kRows + row, node = q / Gq;
  __nv_bfloat16 *dst =
      a.out + (((size_t)b * a.N + node) * a.Hq + (size_t)g * Gq + (q - node * Gq)) * D + d8 * 8;
  *reinterpret_cast<uint4 *>(dst) =
      make_uint4(pack_bf16x2(o[0] * inv, o[1] * inv), pack_bf16x2(o[2] * inv, o[3] * inv),
                 pack_bf16x2(o[4] * inv, o[5] * inv), pack_bf16x2(o[6] * inv, o[7] * inv));
}

inline int row_tiles(int N, int G) { return (N * G + kRows - 1) / kRows; }

template <int D, Scores kScores, bool kJoin>
cudaError_t make_ready() {
  static std::atomic<bool> ready[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !ready[dev].load(std::memory_order_relaxed)) {
    e = cudaFuncSetAttribute(tree_attn_kernel<D, kScores, kJoin>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Geo<D>::kSmem);
    if (e != cudaSuccess) return e;
    if (dev < 64) ready[dev].store(true, std::memory_order_relaxed);
  }
  return cudaSuccess;
}

template <int D, Scores kScores>
cudaError_t launch(const TreeMaps &maps, const TreeAttnArgs &a, int B, int parts, int ctas,
                   cudaStream_t stream) {
  uint8_t *ws = reinterpret_cast<uint8_t *>(a.error_word);
  const int mts = row_tiles(a.N, a.Hq / a.Hkv), records = B * a.Hkv * mts;
  cudaError_t e;
  if (ctas > 0) {
    if ((e = make_ready<D, kScores, true>()) != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(records * ctas);
    cfg.blockDim = kThreads;
    cfg.dynamicSmemBytes = Geo<D>::kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)ctas;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, tree_attn_kernel<D, kScores, true>, maps, a, B,
                              mts | ctas << 8, ws);
  }
  if ((e = make_ready<D, kScores, false>()) != cudaSuccess) return e;
  e = launch_pdl(tree_attn_kernel<D, kScores, false>, dim3(parts), kThreads, Geo<D>::kSmem, stream,
                 maps, a, B, mts, ws);
  if (e != cudaSuccess || parts == 1) return e;
  const int rows = a.N * (a.Hq / a.Hkv) < kRows ? a.N * (a.Hq / a.Hkv) : kRows;
  if (parts >= 4 * records)
    return launch_pdl(tree_merge_kernel<D, 8>, dim3(records, (rows + 7) / 8), 512, 0, stream,
                      (const uint8_t *)ws, mts, records, parts, a);
  return launch_pdl(tree_merge_kernel<D, 32>, dim3(records, (rows + 31) / 32), 512, 0, stream,
                    (const uint8_t *)ws, mts, records, parts, a);
}

}  // namespace

// Two CTAs per SM, or fewer when the stream is shorter than that many key tiles; at least
// one for every row tile.
int tree_parts(int B, int N, int Hq, int Hkv, int max_len, int num_parts, int sms) {
  const int mt = row_tiles(N, Hq / Hkv);
  if (num_parts > 0) return num_parts < mt ? mt : num_parts;
  const long long units =
      (long long)B * Hkv * mt * ((max_len + kTile - 1) / kTile + 1 + kSegment);
  const long long most = units < mt ? mt : units;
  return (int)(most < 2 * sms ? most : 2 * sms < mt ? mt : 2 * sms);
}

// CTAs per (pair, row tile) of the one-launch form, 0 for the stream. The form has no merge and no
// scan, a CTA that ends makes room for the next, but it does not even out the lengths. us of the
// stream and of this form:
//   1 sequence, 8 nodes, 16 / 8 heads, 64 tokens 9.3 and 6.4; 512 10.9 and 9.0; 2000 15.8 and 11.3;
//     8000 21 and 19
//   93 sequences, 51 nodes, 32 / 8 heads, 64 tokens 51 and 45; 512 95 and 78; 1000 139 and 118
//   32 sequences, 4 nodes, 32 / 8 heads, 1 to 1000 tokens 25 and 22; 1 to 2000 34 and 35; 1 to 4000
//     52 and 64
//   107 sequences, 42 nodes, 32 / 4 heads of 64, 114 to 1827 tokens 91 and 78
// hence up to 17 tiles per CTA, or 32 where four rounds of CTAs even them out.
// A cluster where there are few tiles to share costs its join (8 nodes, 512 tokens, 1 and 4 CTAs:
// 11.1 and 9.0; 64 nodes: 11.8 and 12.7; 1000 tokens 17 and 14), and with more than four CTAs to three
// SMs the CTAs of one SM share its bandwidth (64 (pair, row tile)s, 1000 tokens, 2 and 4 CTAs:
// 15.9 and 17.5). Eight CTAs only pay for a few (8 of them, 2000 tokens, 4 and 8: 13.1 and 11.3;
// 16: 16.7 and 21.3).
int tree_join_ctas(int B, int N, int Hq, int Hkv, int max_len, int window, int num_parts, int sms) {
  if (num_parts > 0) return 0;
  const int G = Hq / Hkv;
  const long long records = (long long)B * Hkv * row_tiles(N, G);
  const int seen = window > 0 && window < max_len ? window : max_len;
  const int tiles = (seen + kTile - 1) / kTile + 1;
  int c = tiles <= (N * G <= 32 ? 5 : 9) ? 1 : tiles <= 20 || records > 8 ? 4 : kJoinCtas;
  while (c > 1 && 3 * records * c > 4 * sms) c /= 2;
  return (tiles + c - 1) / c <= (records >= 4 * sms ? 32 : 17) ? c : 0;
}

size_t tree_ws_bytes(int B, int N, int Hq, int Hkv, int D, int parts) {
  return slots_offset(B * Hkv * row_tiles(N, Hq / Hkv)) + (size_t)2 * parts * slot_bytes(D);
}

cudaError_t launch_tree_attn(const CUtensorMap *maps, const TreeAttnArgs &a, int B, int D,
                             int parts, int ctas, cudaStream_t stream) {
  const TreeMaps m{maps[0], maps[1], maps[2], maps[3]};
  auto go = [&](auto fn) { return fn(m, a, B, parts, ctas, stream); };
  const cudaError_t e =
      a.softcap > 0.f ? (D == 128 ? go(launch<128, kCap>) : go(launch<64, kCap>))
      : a.slopes != nullptr ? (D == 128 ? go(launch<128, kBias>) : go(launch<64, kBias>))
                            : (D == 128 ? go(launch<128, kPlain>) : go(launch<64, kPlain>));
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace decattn
