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
// The weights are rounded to bf16 (one rounding, at most 2^-8 of each, as large as the
// output's own rounding) because the value product wants both operands alike; sums, maxima
// and O are fp32.
#include <math.h>

#include <atomic>

#include "dec_device.cuh"
#include "dec_launch.h"
#include "tcgen05.cuh"

namespace decattn {
namespace {

constexpr int kTile = 64;      // keys per tile
constexpr int kRows = 128;     // query rows per tile (the MMA's M)
constexpr int kThreads = 192;  // 4 softmax warps, the TMA warp, the MMA warp
constexpr int kSoftmax = 128;
constexpr float kRescale = 8.f;  // log2 of the growth of the maximum that moves it
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
// O [D / 8][128 rows][8] fp32 and (maximum, sum) [128 rows]. Records, one per piece: the
// (pair, row tile) whose first piece boundary is this piece's start, for the merge.
struct Record {
  int b, g, m, first, last;  // pieces first .. last; first < 0: nothing to merge here
  int rows, pad0, pad1;
};

__host__ __device__ inline size_t slot_bytes(int D) { return (size_t)kRows * (D * 4 + 8); }
__host__ __device__ inline size_t records_offset() { return kWsHeaderBytes; }
__host__ __device__ inline size_t slots_offset(int parts) {
  return (records_offset() + (size_t)parts * sizeof(Record) + 255) & ~(size_t)255;
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

// The segments of a piece: runs of key tiles [t0, t1) of one (sequence, KV head, row tile).
struct Walk {
  Seq s;
  int b, g, m, t0, t1, left;
  __device__ __forceinline__ void begin(const TreeAttnArgs &a, int b_, int within, int units) {
    b = b_;
    s = seq_of(a, b, false);
    const int per_head = s.tiles * s.mt;
    g = within / per_head;
    const int r = within - g * per_head;
    m = r / s.tiles;
    t0 = r - m * s.tiles;
    left = units;
    t1 = min(s.tiles, t0 + left);
  }
  __device__ __forceinline__ bool next(const TreeAttnArgs &a) {
    left -= t1 - t0;
    if (left <= 0) return false;
    if (++m == s.mt) {
      m = 0;
      if (++g == a.Hkv) {
        g = 0;
        do s = seq_of(a, ++b, false);
        while (s.live == 0);
      }
    }
    t0 = 0;
    t1 = min(s.tiles, left);
    return true;
  }
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
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

// D[128 x N] (+)= A[128 x 16, tensor memory] B[16 x N]
__device__ __forceinline__ void umma_bf16_ts(uint32_t tmem_d, uint32_t tmem_a, uint64_t bdesc,
                                             uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(tmem_d),
      "r"(tmem_a), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Descriptor of an MN-major operand in 128-byte swizzle atoms (8 K rows of 64 MN elements):
// the leading offset steps to the next 64 elements of MN (`slab` bytes on), the stride
// offset to the next 8 rows of K.
__device__ __forceinline__ uint64_t smem_desc_mn_sw128(uint32_t saddr, uint32_t slab) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr >> 4) & 0x3FFF);
  d |= (uint64_t)(slab >> 4) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}
constexpr uint32_t kBIsMnMajor = 1u << 16;  // instruction descriptor

// Bits [lo, hi) of a 64-bit word, for any lo and hi.
__device__ __forceinline__ uint64_t bit_range(int lo, int hi) {
  const uint64_t below_hi = hi >= 64 ? ~0ull : hi <= 0 ? 0ull : (1ull << hi) - 1;
  const uint64_t below_lo = lo >= 64 ? ~0ull : lo <= 0 ? 0ull : (1ull << lo) - 1;
  return below_hi & ~below_lo;
}

// A store of 8 consecutive floats.
__device__ __forceinline__ void st_v8(float *p, const uint32_t *r) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
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

// kMod: a score cap or a distance bias.
template <int D, bool kMod>
__global__ void __launch_bounds__(kThreads, 2)
    tree_attn_kernel(const __grid_constant__ TreeMaps maps, const TreeAttnArgs a, int B,
                     uint8_t *workspace) {
  using G = Geo<D>;
  constexpr int S = G::kStages;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t s_bar[2 * S + 8];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  __shared__ int s_sum[kThreads / 32], s_begin[2];
  __shared__ unsigned long long s_odd[2];  // tree values that are not finite, by node

  uint8_t *smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  const uint32_t q_s = smem_addr(smem), ring = q_s + G::kQ;
  const uint32_t bar_full = smem_addr(s_bar), bar_empty = bar_full + 8 * S;
  const uint32_t bar_s = bar_empty + 8 * S, bar_p = bar_s + 16, bar_pv = bar_p + 16;
  const uint32_t bar_q = bar_pv + 16, bar_end = bar_q + 8;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int P = gridDim.x, piece = blockIdx.x;

  if (tid == 0) {
    for (int i = 0; i < 2 * S; ++i) mbar_init(bar_full + 8 * i, 1);
    mbar_init(bar_s, 1);
    mbar_init(bar_s + 8, 1);
    mbar_init(bar_p, kSoftmax);
    mbar_init(bar_p + 8, kSoftmax);
    mbar_init(bar_pv, 1);
    mbar_init(bar_pv + 8, 1);
    mbar_init(bar_q, kSoftmax);
    mbar_init(bar_end, 1);
    s_abort = 0;
    s_odd[0] = s_odd[1] = 0;
    fence_barrier_init();
  }
  if (warp == 4 && lane == 0) {
    tma_prefetch_desc(&maps.k);
    tma_prefetch_desc(&maps.v);
    tma_prefetch_desc(&maps.kt);
    tma_prefetch_desc(&maps.vt);
  }
  pdl_launch_dependents();
  pdl_wait_prior_grid();

  // ---- where this CTA's piece begins: a scan over the sequences' unit counts
  const int per = (B + kThreads - 1) / kThreads;
  int mine = 0;
  for (int b = tid * per; b < min(B, (tid + 1) * per); ++b) {
    const Seq s = seq_of(a, b, piece == 0);
    mine += s.tiles * s.mt * a.Hkv;
  }
  int incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) s_sum[warp] = incl;
  __syncthreads();
  int total = 0, before = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += s_sum[w];
    total += s_sum[w];
  }
  const int blk = max(1, (total + P - 1) / P);
  const long long r0l = (long long)piece * blk;
  const int r0 = (int)min((long long)total, r0l);
  const int units = min(blk, total - r0);
  Record *rec = reinterpret_cast<Record *>(workspace + records_offset()) + piece;
  if (units <= 0) {  // past the end of the stream: nothing to do, nothing to merge
    if (tid == 0) rec->first = -1;
    return;
  }
  const int excl = before + incl - mine;
  if (excl <= r0 && r0 < excl + mine) {
    int at = excl, b = tid * per;
    for (;; ++b) {
      const Seq s = seq_of(a, b, false);
      const int u = s.tiles * s.mt * a.Hkv;
      if (r0 < at + u) break;
      at += u;
    }
    s_begin[0] = b;
    s_begin[1] = r0 - at;
  }
  if (warp == 0) tmem_alloc(smem_addr(&s_tmem), kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  const int Gq = a.Hq / a.Hkv;
  const Waiter wait{&s_abort, a.error_word};
  Walk w;
  w.begin(a, s_begin[0], s_begin[1], units);
  if (tid == 0) {
    // does a (pair, row tile) meet its first piece boundary at this piece's start?
    Record r{};
    r.first = -1;
    const int off = r0 - w.t0;  // its first unit
    if (w.t0 > 0 && off / blk == piece - 1) {
      r.b = w.b;
      r.g = w.g;
      r.m = w.m;
      r.first = piece - 1;
      r.last = (off + w.s.tiles - 1) / blk;
      r.rows = min(kRows, w.s.live * Gq - w.m * kRows);
    }
    *rec = r;
  }

  if (warp == 4) {
    // ---------------------------------------------------------------- loads
    if (lane == 0) {
      int it = 0;
      bool ok = true;
      do {
        // a pair with one row tile is read once; with more, the others find it in L2
        const uint64_t policy = w.s.mt == 1 ? l2_policy_evict_first() : l2_policy_evict_normal();
        const int pair = w.b * a.Hkv + w.g;
        for (int t = w.t0; t < w.t1 && ok; ++t) {
          const bool tree = t == w.s.tiles - 1;
          const int row = tree ? 0 : w.s.start + t * kTile;
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
    if (lane == 0) {
      constexpr uint32_t idesc_s = idesc_bf16_f32(kRows, kTile);
      constexpr uint32_t idesc_o = idesc_bf16_f32(kRows, D) | kBIsMnMajor;
      int n = 0, seg = 0;
      bool ok = true;
      auto issue_s = [&](int i) {
        const int it = 2 * i, slot = it % S;
        // the buffer's last P, that of tile i - 2, is consumed
        if (i >= 2 && !wait(bar_pv + 8 * (i & 1), ((i - 2) >> 1) & 1)) return false;
        if (!wait(bar_full + 8 * slot, (it / S) & 1)) return false;
        tc_fence_after();
        const uint32_t k_s = ring + slot * G::kTensor;
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          umma_bf16(tmem + (i & 1) * kTile,
                    smem_desc_sw128(q_s + (k >> 2) * (kRows * 128) + 32 * (k & 3)),
                    smem_desc_sw128(k_s + (k >> 2) * G::kSlab + 32 * (k & 3)), idesc_s, k > 0);
        umma_commit(bar_empty + 8 * slot);
        umma_commit(bar_s + 8 * (i & 1));
        return true;
      };
      do {
        const int cnt = w.t1 - w.t0;
        ok = wait(bar_q, seg & 1) && issue_s(n);
        for (int i = 0; i < cnt && ok; ++i) {
          if (i + 1 < cnt) ok = issue_s(n + i + 1);
          const int it = 2 * (n + i) + 1, slot = it % S;
          ok = ok && wait(bar_p + 8 * ((n + i) & 1), ((n + i) >> 1) & 1) &&
               wait(bar_full + 8 * slot, (it / S) & 1);
          if (!ok) break;
          tc_fence_after();
          const uint32_t v_s = ring + slot * G::kTensor;
#pragma unroll
          for (int k = 0; k < kTile / 16; ++k)
            umma_bf16_ts(tmem + kOCol, tmem + ((n + i) & 1) * kTile + 8 * k,
                         smem_desc_mn_sw128(v_s + k * 2048, G::kSlab), idesc_o, i > 0 || k > 0);
          umma_commit(bar_empty + 8 * slot);
          umma_commit(bar_pv + 8 * ((n + i) & 1));
        }
        n += cnt;
        ++seg;
      } while (ok && w.next(a));
      if (!ok) {  // let what was issued finish before tensor memory is given back
        umma_commit(bar_end);
        mbar_wait_bounded(bar_end, 0);
      }
    }
  } else {
    // ---------------------------------------------------------------- softmax
    const uint32_t my_tmem = tmem + ((uint32_t)(32 * warp) << 16);
    const float log2e = 1.4426950408889634f;
    const float sc = kMod ? 1.f : a.scale * log2e;
    int n = 0, seg = 0;
    bool ok = true;
    // the same answer in every lane, and the warp together behind it
    auto wait_all = [&](uint32_t bar, uint32_t parity) {
      return __all_sync(0xffffffffu, wait(bar, parity) ? 1 : 0) != 0;
    };
    // this thread's row of Q into shared memory, K-major with the 128-byte swizzle
    auto load_q = [&](const Walk &v) {
      const int row = v.m * kRows + tid, node = row / Gq;
      const bool real = node < v.s.live;
      const size_t at =
          (((size_t)v.b * a.N + node) * a.Hq + (size_t)v.g * Gq + (row - node * Gq)) * D;
      const uint4 *src = reinterpret_cast<const uint4 *>(a.q + at);
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
    load_q(w);
    bool more = true;
    while (more) {
      const int row = w.m * kRows + tid, node = row / Gq, hi = row - node * Gq;
      const int rows = min(kRows, w.s.live * Gq - w.m * kRows);
      const bool real = tid < rows, active = 32 * warp < rows;
      const size_t brow = (size_t)w.b * a.N;
      const int qpos = real && a.pos != nullptr ? max(a.pos[brow + node], w.s.L) : 0;
      const int low = real && a.window > 0 ? qpos - a.window + 1 : 0;  // first slot in the window
      float slope = 0.f;
      if constexpr (kMod)
        if (real && a.slopes != nullptr) slope = a.slopes[w.g * Gq + hi] * log2e;
      float m = -INFINITY, l = 0.f;
      for (int t = w.t0; t < w.t1; ++t, ++n) {
        const bool tree = t == w.s.tiles - 1;
        const int t_abs = w.s.start + t * kTile;
        const uint32_t p_addr = my_tmem + (n & 1) * kTile;
        uint64_t see;
        if (tree) {
          see = real ? a.mask[brow + node] & bit_range(0, w.s.live) : 0;
          if (a.window > 0)
            for (int j = 0; j < w.s.live; ++j)
              if (qpos - max(a.pos[brow + j], w.s.L) >= a.window) see &= ~(1ull << j);
        } else {
          see = real ? bit_range(low - t_abs, w.s.L - t_abs) : 0;
        }
        if (!wait_all(bar_s + 8 * (n & 1), (n >> 1) & 1)) {
          ok = false;
          break;
        }
        tc_fence_after();
        // every thread has left the segment before this one, whose marks are now free
        if (t == w.t0 && tid == 0) s_odd[(seg + 1) & 1] = 0;
        if (active) {
          uint32_t raw[kTile];
          tmem_ld32(p_addr, raw);
          tmem_ld32(p_addr + 32, raw + 32);
          tmem_wait_ld();
          float z[kTile];
#pragma unroll
          for (int c = 0; c < kTile; ++c) z[c] = __uint_as_float(raw[c]);
          if constexpr (kMod) {
            if (a.softcap > 0.f) {
              // cap tanh(x / cap) = cap - 2 cap / (1 + e^(2 x / cap))
              const float in = 2.f * log2e * a.scale / a.softcap, cap = a.softcap * log2e;
#pragma unroll
              for (int c = 0; c < kTile; ++c)
                z[c] = fmaf(-2.f * cap, rcp(1.f + ex2(z[c] * in)), cap);
            } else {
#pragma unroll
              for (int c = 0; c < kTile; ++c) z[c] *= a.scale * log2e;
            }
            if (a.slopes != nullptr) {
              if (!tree) {
#pragma unroll
                for (int c = 0; c < kTile; ++c)
                  z[c] = fmaf(-slope, (float)(qpos - t_abs - c), z[c]);
              } else {
#pragma unroll
                for (int c = 0; c < kTile; ++c)
                  if (c < w.s.live)
                    z[c] = fmaf(-slope, (float)(qpos - max(a.pos[brow + c], w.s.L)), z[c]);
              }
            }
          }
          if (!__all_sync(0xffffffffu, see == ~0ull)) {
            const uint32_t s0 = (uint32_t)see, s1 = (uint32_t)(see >> 32);
#pragma unroll
            for (int c = 0; c < kTile; ++c)
              if (!(((c < 32 ? s0 : s1) >> (c & 31)) & 1u)) z[c] = -INFINITY;
          }
          float mx = z[0];
#pragma unroll
          for (int c = 1; c < kTile; ++c) mx = fmaxf(mx, z[c]);
          mx *= sc;
          const bool grow = mx > m + kRescale || (m == -INFINITY && mx > m);
          if (__any_sync(0xffffffffu, grow)) {
            const float mn = grow ? mx : m;
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
          const float base = m == -INFINITY ? 0.f : m;
          uint32_t pk[kTile / 2];
          float l0 = 0.f, l1 = 0.f;
#pragma unroll
          for (int c = 0; c < kTile; c += 2) {
            const float p0 = ex2(fmaf(z[c], sc, -base)), p1 = ex2(fmaf(z[c + 1], sc, -base));
            l0 += p0;
            l1 += p1;
            pk[c / 2] = pack_bf16x2(p0, p1);
          }
          l += l0 + l1;
          tmem_st32(p_addr, pk);
          tmem_wait_st();
        }
        // rows of V that nobody may read can hold anything, and 0 times NaN is NaN: they
        // are cleared in shared memory. In the tree's tile so are values that are not finite
        // (the nodes that do see them get them back at the end).
        const int valid = tree ? w.s.live : w.s.L - t_abs;
        if (tree || valid < kTile) {
          const int it = 2 * n + 1, slot = it % S;
          if (!wait_all(bar_full + 8 * slot, (it / S) & 1)) {
            ok = false;
            break;
          }
          const int r = tid >> 1;
          bool clear = r >= valid;
          if (tree && !clear) {
            uint64_t used = 0;
            for (int j = 0; j < w.s.live; ++j) used |= a.mask[brow + j];
            clear = !((used >> r) & 1);
          }
          bool odd = false;
#pragma unroll
          for (int c = 0; c < D / 16; ++c) {  // half a row per thread
            const int ch = (tid & 1) * (D / 16) + c;
            const uint32_t at = ring + slot * G::kTensor + (ch >> 3) * G::kSlab + r * 128 +
                                ((ch & 7) << 4);  // any order within the row serves
            uint32_t x[4];
            if (!clear && tree) {
              asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                           : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
                           : "r"(at));
              bool bad = false;
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                if ((x[i] & 0x7f80u) == 0x7f80u) x[i] &= 0xffff0000u, bad = true;
                if ((x[i] & 0x7f800000u) == 0x7f800000u) x[i] &= 0xffffu, bad = true;
              }
              odd |= bad;
              if (!bad) continue;
            } else if (clear) {
              x[0] = x[1] = x[2] = x[3] = 0;
            } else {
              continue;
            }
            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(x[0]),
                         "r"(x[1]), "r"(x[2]), "r"(x[3])
                         : "memory");
          }
          if (odd) atomicOr(&s_odd[seg & 1], 1ull << r);
          fence_proxy_async_smem();
        }
        tc_fence_before();
        mbar_arrive(bar_p + 8 * (n & 1));
      }
      if (!ok) break;
      // ---- the segment's end
      const Walk done = w;
      uint64_t odd = 0;
      if (done.t1 == done.s.tiles) {
        // every thread's mark is visible once the tile's last arrival is
        if (!wait_all(bar_p + 8 * ((n - 1) & 1), ((n - 1) >> 1) & 1)) break;
        odd = *reinterpret_cast<volatile unsigned long long *>(&s_odd[seg & 1]);
      }
      more = w.next(a);
      // every S of this segment has been read, so Q's space is free; P of the last tile must
      // stay for the values to be given back
      if (more && odd == 0) load_q(w);
      if (!wait_all(bar_pv + 8 * ((n - 1) & 1), ((n - 1) >> 1) & 1)) break;
      tc_fence_after();
      if (active) {
        const bool whole = done.t0 == 0 && done.t1 == done.s.tiles;
        const float scale = whole ? (l == 0.f ? 0.f : 1.f / l) : 1.f;
        const int slot = 2 * piece + (done.t0 > 0 ? 0 : 1);
        float *part = reinterpret_cast<float *>(workspace + slots_offset(P) +
                                                (size_t)slot * slot_bytes(D));
        __nv_bfloat16 *dst =
            a.out + ((brow + node) * a.Hq + (size_t)done.g * Gq + hi) * D;
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          uint32_t o[32];
          tmem_ld32(my_tmem + kOCol + c, o);
          tmem_wait_ld();
          for (uint64_t left = odd; left != 0; left &= left - 1) {
            const int j = __ffsll((long long)left) - 1;
            const uint32_t pw = tmem_ld1(my_tmem + ((n - 1) & 1) * kTile + (j >> 1));
            const float p = (j & 1) ? bf16_hi(pw) : bf16_lo(pw);
            const bool sees = real && ((a.mask[brow + node] >> j) & 1) &&
                              !(a.window > 0 &&
                                qpos - max(a.pos[brow + j], done.s.L) >= a.window);
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
          if (real && whole) {
#pragma unroll
            for (int i = 0; i < 32; i += 8) {
              uint32_t x[4];
#pragma unroll
              for (int k = 0; k < 4; ++k)
                x[k] = pack_bf16x2(__uint_as_float(o[i + 2 * k]) * scale,
                                   __uint_as_float(o[i + 2 * k + 1]) * scale);
              *reinterpret_cast<uint4 *>(dst + c + i) = make_uint4(x[0], x[1], x[2], x[3]);
            }
          } else if (real) {
#pragma unroll
            for (int i = 0; i < 32; i += 8)
              st_v8(part + ((size_t)((c + i) / 8) * kRows + tid) * 8, o + i);
          }
          __syncwarp();
        }
        if (!whole && real)
          reinterpret_cast<float2 *>(part + (size_t)kRows * D)[tid] = make_float2(m, l);
      }
      tc_fence_before();
      if (more && odd != 0) load_q(w);
      ++seg;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// Joins the partials of the (pair, row tile)s that cross pieces: out = sum_c 2^(m_c - M) O_c /
// sum_c 2^(m_c - M) l_c. CTA (c, y) takes 8 rows of the one whose first boundary is piece
// c's start, a thread per (row, 8 dims, every kGroups-th piece).
template <int D>
__global__ void __launch_bounds__(512) tree_merge_kernel(const uint8_t *workspace, int parts,
                                                         TreeAttnArgs a) {
  constexpr int kD8 = D / 8, kGroups = 512 / (8 * kD8);
  __shared__ float s_o[kGroups][8][D + 4];
  __shared__ float s_ml[kGroups][8][2];
  pdl_launch_dependents();
  pdl_wait_prior_grid();
  const Record r = reinterpret_cast<const Record *>(workspace + records_offset())[blockIdx.x];
  const int row0 = blockIdx.y * 8;
  if (r.first < 0 || row0 >= r.rows) return;
  const int rr = threadIdx.x & 7, d8 = (threadIdx.x >> 3) % kD8, grp = threadIdx.x / (8 * kD8);
  const int row = row0 + rr;
  const uint8_t *slots = workspace + slots_offset(parts);
  float M = -INFINITY, l = 0.f, o[8] = {};
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
#pragma unroll
  for (int i = 0; i < 8; ++i) s_o[grp][rr][d8 * 8 + i] = o[i];
  if (d8 == 0) {
    s_ml[grp][rr][0] = M;
    s_ml[grp][rr][1] = l;
  }
  __syncthreads();
  if (grp != 0 || row >= r.rows) return;
  float Mx = -INFINITY;
#pragma unroll
  for (int k = 0; k < kGroups; ++k) Mx = fmaxf(Mx, s_ml[k][rr][0]);
  const float base = Mx == -INFINITY ? 0.f : Mx;
  float lt = 0.f, t[8] = {};
#pragma unroll
  for (int k = 0; k < kGroups; ++k) {
    const float e = ex2(s_ml[k][rr][0] - base);
    lt += s_ml[k][rr][1] * e;
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] += s_o[k][rr][d8 * 8 + i] * e;
  }
  const float inv = lt == 0.f ? 0.f : 1.f / lt;
  const int Gq = a.Hq / a.Hkv, q = r.m * kRows + row, node = q / Gq;
  __nv_bfloat16 *dst =
      a.out + (((size_t)r.b * a.N + node) * a.Hq + (size_t)r.g * Gq + (q - node * Gq)) * D + d8 * 8;
  *reinterpret_cast<uint4 *>(dst) =
      make_uint4(pack_bf16x2(t[0] * inv, t[1] * inv), pack_bf16x2(t[2] * inv, t[3] * inv),
                 pack_bf16x2(t[4] * inv, t[5] * inv), pack_bf16x2(t[6] * inv, t[7] * inv));
}

template <int D, bool kMod>
cudaError_t launch(const TreeMaps &maps, const TreeAttnArgs &a, int B, int parts,
                   cudaStream_t stream) {
  static std::atomic<bool> ready[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !ready[dev].load(std::memory_order_relaxed)) {
    e = cudaFuncSetAttribute(tree_attn_kernel<D, kMod>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)Geo<D>::kSmem);
    if (e != cudaSuccess) return e;
    if (dev < 64) ready[dev].store(true, std::memory_order_relaxed);
  }
  uint8_t *ws = reinterpret_cast<uint8_t *>(a.error_word);
  e = launch_pdl(tree_attn_kernel<D, kMod>, dim3(parts), kThreads, Geo<D>::kSmem, stream, maps, a,
                 B, ws);
  if (e != cudaSuccess || parts == 1) return e;
  const int rows = a.N * (a.Hq / a.Hkv) < kRows ? a.N * (a.Hq / a.Hkv) : kRows;
  return launch_pdl(tree_merge_kernel<D>, dim3(parts, (rows + 7) / 8), 512, 0, stream,
                    (const uint8_t *)ws, parts, a);
}

}  // namespace

// Two CTAs per SM, or fewer when the stream is shorter than that many key tiles.
int tree_parts(int B, int N, int Hq, int Hkv, int max_len, int num_parts, int sms) {
  if (num_parts > 0) return num_parts;
  const long long mt = ((long long)N * (Hq / Hkv) + kRows - 1) / kRows;
  const long long units = (long long)B * Hkv * mt * ((max_len + kTile - 1) / kTile + 1);
  const long long most = units < 1 ? 1 : units;
  return (int)(most < 2 * sms ? most : 2 * sms);
}

size_t tree_ws_bytes(int D, int parts) {
  return slots_offset(parts) + (size_t)2 * parts * slot_bytes(D);
}

cudaError_t launch_tree_attn(const CUtensorMap *maps, const TreeAttnArgs &a, int B, int D,
                             int parts, cudaStream_t stream) {
  const TreeMaps m{maps[0], maps[1], maps[2], maps[3]};
  const bool mod = a.softcap > 0.f || a.slopes != nullptr;
  const cudaError_t e =
      D == 128 ? (mod ? launch<128, true>(m, a, B, parts, stream)
                      : launch<128, false>(m, a, B, parts, stream))
               : (mod ? launch<64, true>(m, a, B, parts, stream)
                      : launch<64, false>(m, a, B, parts, stream));
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace decattn
