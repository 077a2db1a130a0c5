// Attention of a drafted tree over the paged cache: the up to 64 rows of each sequence share its
// context and see, of one another, the nodes of their masks.
//
//   o[t][h] = sum_i e^(x_i - m) v_i / sum_i e^(x_i - m),  x_i = q[t][h].k_i / sqrt(D),  m = max x_i
//
// over the context keys 1..base (with a window: those above p - W) and the tree's keys base + 1 + j
// with bit j in the row's mask.
//
// The n G rows (node-major, then the G query heads of a KV head) are cut into tiles of 128, the lanes of
// a tcgen05 accumulator. An item is one or two tiles of one (sequence, KV head); its keys stream through
// shared memory once, in blocks of 64. Two streams of a CTA work on an item, so that one's softmax covers
// the other's matrix products: with two tiles each has a tile of its own and every block serves both;
// with one tile they take its blocks in turn, each with its own (m, sum, O), and are joined at the end.
// TMEM columns of stream s, from 256 s: S, then P over it, [0, 64); Q [64, 128); O [128, 128 + D).
//   S = Q . K^T      A = Q (TMEM), B = K block (shared memory, K-major)
//   O += P . V       A = P (TMEM), B = V block (MN-major)
// P is split into a high and a low bf16 half, so that the products keep FP32's accuracy.
//
// The blocks of all items, laid end to end and weighed by their tiles, are cut into equal ranges, one for
// each CTA; partials of an item that several ranges share go to the workspace and a second kernel joins
// them. Ranges are planned on the device from the sequences' own lengths.
//
// Warps: 0 loads (page table and TMA), 1 issues the matrix products, 4-7 and 8-11 the streams' softmax
// (a thread per row); over FP8 and NVFP4 pages 12-19 turn codes into bf16 tiles, exactly.
//
// A key that only some rows see may hold infinities or NaN, which 0 . V would carry into the others. Blocks
// that not all rows see in full are looked through before their product: rows of V outside the item's keys
// become zero, and so do elements that are no numbers; the rows that see them get them added at the end.
//
// The tensor pipe's FP32 accumulation drops about 2^-24 of the running sum per MMA, so after kFlush blocks
// O is added into FP32 scratch and begins afresh.
//
// Every mbarrier wait is bounded: on expiry the CTA records BEAM_DEV_TIMEOUT, lets its issued copies land,
// frees TMEM and returns.
#include <cuda.h>
#include <math.h>

#include <atomic>

#include "mma.cuh"
#include "paged.cuh"
#include "tcgen05.cuh"

namespace beam {
namespace paged {
namespace {

using namespace beam::tc;

constexpr int BK = 64;            // keys of a block
constexpr int ROWS = 128;         // rows of a tile
constexpr int kNodes = 64;        // tree rows of a sequence at most
constexpr int kMaxSeqs = 1024;    // sequences of one launch
constexpr int kGrid = 152;        // CTAs at most (the workspace is sized for this many)
constexpr int kFlush = 128;       // blocks of a stream between flushes of O: 1024 MMAs
constexpr float kNegInf = -INFINITY;
constexpr float kRescale = 8.f;   // log2 units by which the running max may lag

template <int FMT, int D_>
struct Cfg {
  static constexpr int D = D_, ROWB = row_bytes(FMT, D);
  static constexpr bool QUANT = FMT != kFmtBF16;
  static constexpr int THREADS = QUANT ? 640 : 384;
  static constexpr int NH = D / 64;                 // 64-wide halves of a tile's rows
  static constexpr int TILE = BK * D * 2;           // K or V block in bf16
  static constexpr int NST = QUANT ? 3 : (D == 128 ? 6 : 8);
  static constexpr int RAWK = QUANT ? BK * ROWB : 0;
  static constexpr int RBS = FMT == kFmtNVFP4 ? BK * (D / 16) : 0;   // block scales of K or V
  // a raw stage: K codes, V codes, K's and V's block scales, K's and V's row scales
  static constexpr int RAW = QUANT ? 2 * RAWK + 2 * RBS + 2 * BK : 0;
  static constexpr int NRAW = QUANT ? 6 : 0;
  static constexpr int K0 = 0, V0 = NST * TILE, R0 = 2 * NST * TILE;
  static constexpr int CUM = (R0 + NRAW * RAW + 15) / 16 * 16;       // [kMaxSeqs + 1] cost prefix
  static constexpr int XCH = CUM + (kMaxSeqs + 4) * 4;               // [2][128] (m, sum) of stream 1
  static constexpr int MASK = XCH + 2 * ROWS * 8;                    // [16] slices of a block that have a page
  static constexpr int BAR = MASK + 16 * 4;
  static constexpr int NBAR = 4 * NST + 2 * NRAW + 13;
  static constexpr int MISC = BAR + NBAR * 8;
  static constexpr int BYTES = MISC + 32 + 1024;
  static_assert(BYTES <= 227 * 1024, "shared memory");
};

struct Params {
  const uint16_t* q;
  const uint16_t* g;
  const uint16_t* gate_bias;
  const int32_t* seq_id;
  const int32_t* row_start;
  const int32_t* base;
  const uint64_t* mask;
  uint16_t* og;
  float* part_acc;   // [kGrid][2][2][ROWS][D]: partials of a range's first and last item, by tile
  float2* part_ml;   // [kGrid][2][2][ROWS]
  float* flush;      // [kGrid][2][ROWS][D]
  int4* join;        // [kGrid]: item that begins in the range and runs on: (sequence, head | item << 16, parts, -)
  beam_paged_kv c;
  int N, T, n_q, n_kv, G, max_pos, shift, least;
  int head_rows, tail_rows;   // whether rows before the first and behind the last sequence are this launch's
  float sl2;
};

struct Seq {
  int row0, n, sid, base, lo, blk0, nb, tiles;
  unsigned bad;
};
__device__ __forceinline__ Seq seq_of(const Params& P, int i) {
  Seq s;
  s.row0 = P.row_start[i];
  s.n = P.row_start[i + 1] - s.row0;
  s.sid = P.seq_id[i];
  s.base = P.base[i];
  s.bad = 0;
  if (s.n < 0 || s.n > kNodes || s.row0 < 0 || s.row0 > P.T - max(0, s.n)) s.bad = BEAM_DEV_BAD_SEQ;
  else if (s.n > 0 && (s.sid < 0 || s.sid >= P.c.num_seqs)) s.bad = BEAM_DEV_BAD_SEQ;
  else if (s.n > 0 && (s.base < 0 || s.base > P.max_pos - s.n ||
                       ((s.base + s.n - 1) >> P.shift) >= P.c.table_stride))
    s.bad = BEAM_DEV_BAD_POSITION;
  const bool none = s.bad || s.n == 0;
  s.lo = P.c.window > 0 ? max(1, s.base + 2 - P.c.window) : 1;
  s.blk0 = none ? 0 : (s.lo - 1) / BK;
  s.nb = none ? 0 : (s.base + s.n - 1) / BK - s.blk0 + 1;
  s.tiles = none ? 0 : (s.n * P.G + ROWS - 1) / ROWS;
  return s;
}

// A CTA's share [j0, j1) of the blocks of item m (tiles 2m, 2m + 1) of one (sequence, KV head).
struct Item {
  Seq s;
  int i, h, m, w, j0, j1, f, next;   // w: its tiles; f: cost at its first block
  bool split;
};

// Smallest cost of range r; the range of cost c.
__device__ __forceinline__ int range_lo(int r, int total, int R) { return int(int64_t(r) * total / R); }
__device__ __forceinline__ int range_of(int c, int total, int R) {
  return int((int64_t(c + 1) * R - 1) / total);
}

// The item at cost c of the range that ends at c1.
__device__ __forceinline__ Item item_at(const Params& P, const int* cum, int c, int c1) {
  int a = 0, b = P.N;   // cum[a] <= c < cum[b]
  while (b - a > 1) {
    const int mid = (a + b) >> 1;
    if (cum[mid] <= c) a = mid;
    else b = mid;
  }
  Item it;
  it.i = a;
  it.s = seq_of(P, a);
  const int per = it.s.nb * it.s.tiles, off = c - cum[a];
  it.h = off / per;
  const int rest = off - it.h * per;
  it.m = rest / (2 * it.s.nb);
  it.w = 2 * it.m + 1 < it.s.tiles ? 2 : 1;
  it.f = c - rest + it.m * 2 * it.s.nb;
  it.j0 = (c - it.f + it.w - 1) / it.w;
  it.next = it.f + it.w * it.s.nb;
  it.j1 = it.next <= c1 ? it.s.nb : (c1 - it.f + it.w - 1) / it.w;
  it.split = it.j0 > 0 || it.j1 < it.s.nb;
  return it;
}
// The next item of a range that has blocks in it, from cost c on.
__device__ __forceinline__ bool next_item(const Params& P, const int* cum, int& c, int c1, Item& it) {
  while (c < c1) {
    it = item_at(P, cum, c, c1);
    c = it.next;
    if (it.j0 < it.j1) return true;
  }
  return false;
}
// Blocks that stream s takes of an item.
__device__ __forceinline__ int units_of(const Item& it, int s) {
  const int n = it.j1 - it.j0;
  return it.w == 2 ? n : (n + 1 - s) / 2;
}

// Whether all rows of the item see all keys of block j (its pages aside).
__device__ __forceinline__ bool whole_block(const Params& P, const Seq& s, int j) {
  const int kb = (s.blk0 + j) * BK + 1;
  const int hi = P.c.window > 0 ? max(1, s.base + s.n + 1 - P.c.window) : 1;   // the deepest row's first key
  return kb >= hi && kb + BK - 1 <= s.base;
}

// Slices of 16 keys of block j that lie in a page; lanes 0..3 look them up.
__device__ __forceinline__ int page_of_slice(const Params& P, const Seq& s, int j, int e) {
  const int k0 = (s.blk0 + j) * BK + 16 * e;   // 0-based
  if (k0 + 16 < s.lo || k0 >= s.base + s.n) return -2;   // no key of the item
  const int pg = P.c.page_table[size_t(s.sid) * P.c.table_stride + (k0 >> P.shift)];
  return pg >= 0 && pg < P.c.num_pages ? pg : -1;
}
__device__ __forceinline__ unsigned slices_of(const Params& P, const Seq& s, int j) {
  const int lane = threadIdx.x & 31;
  const int pg = lane < 4 ? page_of_slice(P, s, j, lane) : -2;
  return __ballot_sync(0xffffffffu, pg >= 0) & 15u;
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t mbar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
          "r"(dst), "l"(src), "r"(bytes), "r"(mbar)
      : "memory");
}
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
__device__ __forceinline__ uint64_t f2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void f2_split(uint64_t r, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(r));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t sub2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Four neighbouring outputs, gated, rounded once.
__device__ __forceinline__ uint2 finish4(const Params& P, float4 o, size_t at, float bias) {
  if (P.g != nullptr) {
    const uint2 g = *reinterpret_cast<const uint2*>(P.g + at);
    o.x *= rcp(1.f + __expf(-(bf_lo(g.x) + bias)));
    o.y *= rcp(1.f + __expf(-(bf_hi(g.x) + bias)));
    o.z *= rcp(1.f + __expf(-(bf_lo(g.y) + bias)));
    o.w *= rcp(1.f + __expf(-(bf_hi(g.y) + bias)));
  }
  return make_uint2(pack_bf16x2(o.x, o.y), pack_bf16x2(o.z, o.w));
}

__device__ __forceinline__ bool no_number(uint32_t w) {   // either bf16 of a pair
  return (w & 0x7F80u) == 0x7F80u || (w & 0x7F800000u) == 0x7F800000u;
}

// What a row of an item sees.
struct RowView {
  uint64_t tree;   // nodes
  int lo, base;    // context keys lo..base
};
__device__ __forceinline__ RowView view_of(const Params& P, const Seq& s, int node) {
  RowView v;
  v.tree = node < s.n ? P.mask[s.row0 + node] : 0;
  if (s.n < 64) v.tree &= (uint64_t(1) << s.n) - 1;
  v.base = v.tree != 0 ? s.base : 0;
  v.lo = 1;
  if (P.c.window > 0) {
    const int depth = __popcll(v.tree);
    v.lo = max(1, s.base + depth + 1 - P.c.window);
    for (int d = depth; d > P.c.window; --d) v.tree &= v.tree - 1;   // ancestors before the window
  }
  return v;
}
// Its keys among the 64 from position kb on, whose 16-key slices `slices` lie in pages.
__device__ __forceinline__ uint64_t seen(const RowView& v, const Seq& s, int kb, unsigned slices) {
  uint64_t bits = 0;
  const int a = max(v.lo, kb) - kb, b = min(v.base, kb + BK - 1) - kb;   // context columns a..b
  if (a <= b) bits = (~uint64_t(0) >> (63 - (b - a))) << a;
  const int to = s.base + 1 - kb;   // column of node 0
  if (to < 64) bits |= to >= 0 ? v.tree << to : (to > -64 ? v.tree >> -to : 0);
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (!((slices >> e) & 1u)) bits &= ~(uint64_t(0xFFFF) << (16 * e));
  return bits;
}

// Elements of V that are no numbers, in keys that a row sees in blocks that not all rows do: added to
// 32 of its outputs.
template <int FMT, int D>
__device__ __noinline__ void add_no_numbers(const Params& P, const Item& it, const RowView& v, int c0, float* o) {
  const Seq& s = it.s;
  for (int j = it.j0; j < it.j1; ++j) {
    unsigned slices = 0;
    for (int e = 0; e < 4; ++e)
      if (page_of_slice(P, s, j, e) >= 0) slices |= 1u << e;
    if (whole_block(P, s, j) && slices == 15u) continue;
    const int kb = (s.blk0 + j) * BK + 1;
    uint64_t bits = seen(v, s, kb, slices);
    while (bits != 0) {
      const int c = __ffsll(static_cast<long long>(bits)) - 1;
      bits &= bits - 1;
      const int k0 = kb - 1 + c;
      const size_t pg = P.c.page_table[size_t(s.sid) * P.c.table_stride + (k0 >> P.shift)];
      const size_t head = pg * P.c.n_kv + it.h;
      const int off = k0 & (P.c.page_size - 1);
      if (FMT != kFmtBF16) {
        if (P.c.row_scale[(head * 2 + 1) * P.c.page_size + off] == 255)
          for (int x = 0; x < 32; ++x) o[x] = __uint_as_float(0x7FFFFFFFu);
        continue;
      }
      const uint16_t* src = static_cast<const uint16_t*>(P.c.v) + (head * P.c.page_size + off) * D + c0;
      for (int x = 0; x < 32; ++x) {
        const uint32_t b = src[x];
        if ((b & 0x7F80u) == 0x7F80u) o[x] += bf2f(uint16_t(b));
      }
    }
  }
}

template <int FMT, int D>
__global__ void __launch_bounds__(Cfg<FMT, D>::THREADS, 1)
paged_tree_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv, const Params P) {
  using C = Cfg<FMT, D>;
  constexpr int NST = C::NST, NRAW = C::NRAW;
  constexpr uint32_t IDESC_QK = idesc_bf16(ROWS, BK, false), IDESC_PV = idesc_bf16(ROWS, D, true);
  pdl_wait();
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = smem_u32(sm);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int* cum = reinterpret_cast<int*>(sm + C::CUM);
  uint32_t* masks = reinterpret_cast<uint32_t*>(sm + C::MASK);
  volatile int* misc = reinterpret_cast<volatile int*>(sm + C::MISC);   // TMEM address, abort, special, -
  const uint32_t k_full = sb + C::BAR, k_empty = k_full + 8 * NST, v_full = k_empty + 8 * NST,
                 v_empty = v_full + 8 * NST, r_full = v_empty + 8 * NST, r_empty = r_full + 8 * NRAW;
  const uint32_t q_full = r_empty + 8 * NRAW, s_full = q_full + 16, p_full = s_full + 16, pv_done = p_full + 16,
                 o_full = pv_done + 16, o_empty = o_full + 16, x_full = o_empty + 16;
  if (threadIdx.x == 0) {
    for (int i = 0; i < NST; ++i) {
      mbar_init(k_full + 8 * i, C::QUANT ? 8 : 1);
      mbar_init(k_empty + 8 * i, 1);
      mbar_init(v_full + 8 * i, C::QUANT ? 8 : 1);
      mbar_init(v_empty + 8 * i, 1);
    }
    for (int i = 0; i < NRAW; ++i) {
      mbar_init(r_full + 8 * i, 1);
      mbar_init(r_empty + 8 * i, 8);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(q_full + 8 * s, ROWS);
      mbar_init(s_full + 8 * s, 1);
      mbar_init(p_full + 8 * s, ROWS);
      mbar_init(pv_done + 8 * s, 1);
      mbar_init(o_full + 8 * s, 2);
      mbar_init(o_empty + 8 * s, ROWS);
    }
    mbar_init(x_full, ROWS);
    misc[1] = 0;
    misc[2] = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(sb + C::MISC), "r"(512) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  // ---- plan: prefix sums of the sequences' costs
  if (warp == 0) {
    int carry = 0;
    if (lane == 0) cum[0] = 0;
    for (int i0 = 0; i0 < P.N; i0 += 32) {
      int c = 0;
      if (i0 + lane < P.N) {
        const Seq s = seq_of(P, i0 + lane);
        c = s.nb * s.tiles * P.n_kv;
        if (s.bad && blockIdx.x == 0) flag(s.bad);
      }
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, c, o);
        if (lane >= o) c += y;
      }
      if (i0 + lane < P.N) cum[i0 + lane + 1] = carry + c;
      carry += __shfl_sync(0xffffffffu, c, 31);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = uint32_t(misc[0]);
  const int total = cum[P.N];
  const int R = max(1, min(int(gridDim.x), total / P.least));
  const int r = blockIdx.x;
  const int c0 = r < R ? range_lo(r, total, R) : 0, c1 = r < R ? range_lo(r + 1, total, R) : 0;

  if (warp == 0) {
    // ------------------------------------------------------------------ loads
    uint32_t nb = 0;   // blocks issued
    bool ok = true;
    Item it;
    for (int c = c0; ok && next_item(P, cum, c, c1, it);) {
      for (int j = it.j0; j < it.j1 && ok; ++j, ++nb) {
        const int pg = lane < 4 ? page_of_slice(P, it.s, j, lane) : -2;
        if (pg == -1 && it.h == 0 && it.m == 0) flag(BEAM_DEV_BAD_PAGE);
        const unsigned live = __ballot_sync(0xffffffffu, pg >= 0) & 15u;
        const int k0 = (it.s.blk0 + j) * BK;
        // a copy covers the slices of one page: `run` of them
        const int run = P.c.page_size >= BK ? 4 : P.c.page_size / 16;
        const int e0 = lane < 4 ? lane / run * run : 0;
        // pages of 64 keys and more: any slice that has keys names the page
        const int first = __ffs((live >> e0) & ((1u << run) - 1u));
        const int page = __shfl_sync(0xffffffffu, pg, first ? e0 + first - 1 : 0);
        const bool mine = lane < 4 && lane == e0 && first != 0;
        const int copies = __popc(__ballot_sync(0xffffffffu, mine));
        const int off = (k0 + 16 * e0) & (P.c.page_size - 1);
        const size_t head = size_t(mine ? page : 0) * P.c.n_kv + it.h;
        if constexpr (!C::QUANT) {
          const int st = int(nb % NST);
          const uint32_t ph = ((nb / NST) & 1) ^ 1;
          if (!__all_sync(0xffffffffu, mbar_wait(k_empty + 8 * st, ph)) ||
              !__all_sync(0xffffffffu, mbar_wait(v_empty + 8 * st, ph))) { ok = false; break; }
          const uint32_t bytes = uint32_t(copies * run * 16 * D * 2);
          if (lane == 0) {
            masks[st] = live;
            mbar_expect_tx(k_full + 8 * st, bytes);
            mbar_expect_tx(v_full + 8 * st, bytes);
          }
          __syncwarp();
          if (mine) {
#pragma unroll
            for (int x = 0; x < C::NH; ++x) {
              const uint32_t at = st * C::TILE + x * BK * 128 + e0 * 16 * 128;
              tma_load_3d(sb + C::K0 + at, &tk, 128 * x, off, int(head), k_full + 8 * st);
              tma_load_3d(sb + C::V0 + at, &tv, 128 * x, off, int(head), v_full + 8 * st);
            }
          }
        } else {
          const int st = int(nb % NRAW);
          if (!__all_sync(0xffffffffu, mbar_wait(r_empty + 8 * st, ((nb / NRAW) & 1) ^ 1))) { ok = false; break; }
          const uint32_t keys = uint32_t(run * 16);
          if (lane == 0) {
            masks[st] = live;
            mbar_expect_tx(r_full + 8 * st, uint32_t(copies) * keys * (2 * C::ROWB + 2 + (FMT == kFmtNVFP4 ? 2 * (D / 16) : 0)));
          }
          __syncwarp();
          if (mine) {
            const uint32_t at = sb + C::R0 + st * C::RAW, bar = r_full + 8 * st;
            const size_t row = head * P.c.page_size + off;
#pragma unroll
            for (int kv = 0; kv < 2; ++kv) {
              bulk_load(at + kv * C::RAWK + e0 * 16 * C::ROWB, static_cast<const uint8_t*>(kv ? P.c.v : P.c.k) + row * C::ROWB,
                        keys * C::ROWB, bar);
              const size_t sc = (head * 2 + kv) * P.c.page_size + off;
              if constexpr (FMT == kFmtNVFP4)
                bulk_load(at + 2 * C::RAWK + kv * C::RBS + e0 * 16 * (D / 16), P.c.block_scale + sc * (D / 16), keys * (D / 16), bar);
              bulk_load(at + 2 * C::RAWK + 2 * C::RBS + kv * BK + e0 * 16, P.c.row_scale + sc, keys, bar);
            }
          }
        }
      }
    }
    if (!ok && lane == 0) {
      misc[1] = 1;
      // copies in flight land before the CTA's shared memory goes away
      const uint32_t depth = C::QUANT ? NRAW : NST;
      for (uint32_t b = nb > depth ? nb - depth : 0; b < nb; ++b) {
        if constexpr (C::QUANT) {
          mbar_wait(r_full + 8 * (b % (NRAW ? NRAW : 1)), (b / (NRAW ? NRAW : 1)) & 1);
        } else {
          mbar_wait(k_full + 8 * (b % NST), (b / NST) & 1);
          mbar_wait(v_full + 8 * (b % NST), (b / NST) & 1);
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------ matrix products
    // Units of an item go to the streams in turn; after unit u's P.V the stream's next S is issued (operations
    // of one thread run in order, so it overwrites P only after P.V has read it).
    uint32_t nb = 0;                        // blocks of earlier items
    uint32_t un[2] = {0, 0}, ost[2] = {0, 0}, qn[2] = {0, 0};
    bool ok = true;
    auto all = [&](bool v) { return __all_sync(0xffffffffu, v); };
    const uint64_t dk = smem_desc(sb + C::K0), dv = smem_desc_mn(sb + C::V0, BK * 128, 1024);
    const uint32_t dk_hi = uint32_t(dk >> 32), dv_hi = uint32_t(dv >> 32);
    auto qk = [&](int s, int st) {
      const uint32_t lo = uint32_t(dk) + uint32_t((st * C::TILE) >> 4);
      const uint32_t ts = tmem + 256 * s;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk)
        umma_ts_e(ts, ts + 64 + 8 * kk, lo + uint32_t(((kk >> 2) * BK * 128 + (kk & 3) * 32) >> 4), dk_hi, IDESC_QK, kk > 0 ? 1u : 0u);
      umma_commit_e(s_full + 8 * s);
    };
    auto pv = [&](int s, int st, bool first) {
      const uint32_t lo = uint32_t(dv) + uint32_t((st * C::TILE) >> 4);
      const uint32_t ts = tmem + 256 * s, to = ts + 128;
#pragma unroll
      for (int kk = 0; kk < BK / 16; ++kk) {
        const uint32_t b = lo + uint32_t((kk * 16 * 128) >> 4), a = ts + 32 * (kk >> 1) + 8 * (kk & 1);
        umma_ts_e(to, a, b, dv_hi, IDESC_PV, first && kk == 0 ? 0u : 1u);
        umma_ts_e(to, a + 16, b, dv_hi, IDESC_PV, 1u);
      }
      umma_commit_e(pv_done + 8 * s);
    };
    Item it;
    for (int c = c0; ok && next_item(P, cum, c, c1, it);) {
      const int cnt = it.j1 - it.j0, units = it.w * cnt, step = it.w == 2 ? 1 : 0;
      for (int s = 0; s < 2; ++s)
        if (units_of(it, s) > 0) {
          ok = ok && all(mbar_wait(q_full + 8 * s, qn[s] & 1));
          ++qn[s];
        }
      if (!ok) break;
      tc_fence_after();
      auto first_qk = [&](int u) {
        const uint32_t b = nb + uint32_t(u >> step);
        const int st = int(b % NST);
        if (!all(mbar_wait(k_full + 8 * st, (b / NST) & 1))) return false;
        tc_fence_after();
        qk(u & 1, st);
        if (step == 0 || (u & 1)) umma_commit_e(k_empty + 8 * st);
        return true;
      };
      for (int u = 0; u < 2 && u < units && ok; ++u) ok = first_qk(u);
      for (int u = 0; u < units && ok; ++u) {
        const int s = u & 1, j = u >> step;
        const uint32_t b = nb + uint32_t(j);
        const int st = int(b % NST);
        const int k = u >> 1;                        // the stream's unit
        const bool fresh = k % kFlush == 0;
        if (!all(mbar_wait(v_full + 8 * st, (b / NST) & 1) && mbar_wait(p_full + 8 * s, un[s] & 1) &&
                 (!fresh || mbar_wait(o_empty + 8 * s, (ost[s] & 1) ^ 1)))) {
          ok = false;
          break;
        }
        if constexpr (!C::QUANT) {
          const unsigned live = masks[st];
          if ((step == 0 || s == 0) && (live != 15u || !whole_block(P, it.s, it.j0 + j))) {
            // rows of V outside the item's keys, and elements that are no numbers
            const int kb = (it.s.blk0 + it.j0 + j) * BK + 1;
            bool odd = false;
            for (int x = lane; x < C::TILE / 16; x += 32) {
              const int row = (x >> 3) & (BK - 1), key = kb + row;
              uint4* at = reinterpret_cast<uint4*>(sm + C::V0 + st * C::TILE) + x;
              if (key < it.s.lo || key > it.s.base + it.s.n || !((live >> (row >> 4)) & 1u)) {
                *at = make_uint4(0, 0, 0, 0);
                continue;
              }
              uint4 w = *at;
              if (no_number(w.x) || no_number(w.y) || no_number(w.z) || no_number(w.w)) {
                odd = true;
                uint32_t* y = reinterpret_cast<uint32_t*>(&w);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  if ((y[e] & 0x7F80u) == 0x7F80u) y[e] &= 0xFFFF0000u;
                  if ((y[e] & 0x7F800000u) == 0x7F800000u) y[e] &= 0x0000FFFFu;
                }
                *at = w;
              }
            }
            if (odd) misc[2] = 1;
            fence_proxy_async_smem();
            __syncwarp();
          }
        }
        tc_fence_after();
        if (fresh) ++ost[s];
        ++un[s];
        pv(s, st, fresh);
        if (step == 0 || s == 1) umma_commit_e(v_empty + 8 * st);
        if (u + 2 < units) ok = first_qk(u + 2);
      }
      if (!ok) break;
      nb += uint32_t(cnt);
      for (int s = 0; s < 2; ++s) {
        umma_commit_e(o_full + 8 * s);
        if (lane == 0) mbar_arrive(o_full + 8 * s);   // orders `special` before the streams' reads
      }
    }
    if (!ok) misc[1] = 1;
  } else if (warp >= 4 && warp < 12) {
    // ------------------------------------------------------------------ softmax
    const int s = (warp - 4) >> 2, q4 = warp & 3, lr = q4 * 32 + lane;
    const uint32_t ts = tmem + 256 * s + (uint32_t(q4 * 32) << 16), tq = ts + 64, to = ts + 128;
    float2* xch = reinterpret_cast<float2*>(sm + C::XCH);
    float* fl = P.flush + (size_t(blockIdx.x) * 2 * ROWS + lr) * D;   // stream 0's; 1's ROWS * D on
    uint32_t un = 0, items = 0, turns = 0;
    bool ok = true;
    auto all = [&](bool v) { return __all_sync(0xffffffffu, v); };
    int4 join = make_int4(0, 0, 0, 0);
    Item it;
    for (int c = c0; ok && next_item(P, cum, c, c1, it); ++items) {
      const int units = units_of(it, s);
      const int tile = 2 * it.m + (it.w == 2 ? s : 0);
      const int row = tile * ROWS + lr, node = row / P.G, hq = it.h * P.G + (row - node * P.G);
      const bool real = node < it.s.n;
      const RowView v = view_of(P, it.s, node);
      const size_t at = (size_t(it.s.row0 + (real ? node : 0)) * P.n_q + hq) * D;
      const bool work = __any_sync(0xffffffffu, v.tree != 0);   // any row that sees keys
      const bool none = __any_sync(0xffffffffu, real && v.tree == 0);   // a row among them that sees nothing
      if (units > 0) {
#pragma unroll 1
        for (int x = 0; x < D / 64; ++x) {
          uint32_t w[32];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const uint4 y = real ? reinterpret_cast<const uint4*>(P.q + at + 64 * x)[e] : make_uint4(0, 0, 0, 0);
            w[4 * e] = y.x; w[4 * e + 1] = y.y; w[4 * e + 2] = y.z; w[4 * e + 3] = y.w;
          }
          tmem_st32(tq + 32 * x, w);
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(q_full + 8 * s);
      }
      float m = kNegInf, l = 0.f;   // reference (log2 units; lags by up to kRescale) and sum
      bool flushed = false;
      for (int k = 0; k < units; ++k, ++un) {
        const int j = it.j0 + (it.w == 2 ? k : 2 * k + s);
        const unsigned slices = slices_of(P, it.s, j);
        const bool full = !none && slices == 15u && whole_block(P, it.s, j);
        if (!all(mbar_wait(s_full + 8 * s, un & 1))) { ok = false; break; }
        tc_fence_after();
        if (work) {
          const uint64_t bits = full ? ~uint64_t(0) : seen(v, it.s, (it.s.blk0 + j) * BK + 1, slices);
          float mx[4] = {kNegInf, kNegInf, kNegInf, kNegInf};
#pragma unroll 1
          for (int x = 0; x < 2; ++x) {
            uint32_t sv[32];
            tmem_ld32_nowait(ts + 32 * x, sv);
            tmem_wait_ld();
            if (!full) {
              const uint32_t b32 = uint32_t(bits >> (32 * x));
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (!((b32 >> e) & 1u)) sv[e] = __float_as_uint(kNegInf);
              tmem_st32(ts + 32 * x, sv);
              tmem_wait_st();
            }
#pragma unroll
            for (int e = 0; e < 32; ++e) mx[e & 3] = fmaxf(mx[e & 3], __uint_as_float(sv[e]));
          }
          const float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * P.sl2;
          const bool need = m != kNegInf && mt > m + kRescale;
          if (__any_sync(0xffffffffu, need)) {
            // O holds the stream's earlier products: the last one has to be done
            if (!all(mbar_wait(pv_done + 8 * s, (un - 1) & 1))) { ok = false; break; }
            tc_fence_after();
            const float f = need ? ex2(m - mt) : 1.f;
            if (k % kFlush != 0) {   // after a flush O is not read again
#pragma unroll 1
              for (int x = 0; x < D / 32; ++x) {
                uint32_t o[32];
                tmem_ld32_nowait(to + 32 * x, o);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                tmem_st32(to + 32 * x, o);
              }
              tmem_wait_st();
            }
            if (flushed && need)
              for (int x = 0; x < D; ++x) fl[s * ROWS * D + x] *= f;
            if (need) {
              l *= f;
              m = mt;
            }
          }
          if (m == kNegInf) m = mt;   // the row's first keys
          const float nm = m == kNegInf ? 0.f : -m;
          const uint64_t c2 = f2(P.sl2, P.sl2), nm2 = f2(nm, nm);
          uint64_t ls[4] = {0, 0, 0, 0};
#pragma unroll 1
          for (int x = 0; x < 2; ++x) {
            uint32_t sv[32], pk[32];
            tmem_ld32_nowait(ts + 32 * x, sv);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              float x0, x1;
              f2_split(fma2(f2(__uint_as_float(sv[2 * e]), __uint_as_float(sv[2 * e + 1])), c2, nm2), x0, x1);
              const float p0 = ex2(x0), p1 = ex2(x1);
              const uint64_t pp = f2(p0, p1);
              ls[e & 3] = add2(ls[e & 3], pp);
              const uint32_t hi = pack_bf16x2(p0, p1);
              float d0, d1;
              f2_split(sub2(pp, f2(bf_lo(hi), bf_hi(hi))), d0, d1);
              pk[e] = hi;
              pk[16 + e] = pack_bf16x2(d0, d1);
            }
            tmem_st32(ts + 32 * x, pk);
          }
          float a0, a1, b0, b1;
          f2_split(add2(ls[0], ls[1]), a0, a1);
          f2_split(add2(ls[2], ls[3]), b0, b1);
          l += (a0 + b0) + (a1 + b1);
          tmem_wait_st();
        }
        tc_fence_before();
        mbar_arrive(p_full + 8 * s);
        if ((k + 1) % kFlush == 0 && k + 1 < units) {
          if (!all(mbar_wait(pv_done + 8 * s, un & 1))) { ok = false; ++un; break; }
          tc_fence_after();
#pragma unroll 1
          for (int x = 0; x < D / 32; ++x) {
            uint32_t o[32];
            tmem_ld32_nowait(to + 32 * x, o);
            tmem_wait_ld();
            float4* y = reinterpret_cast<float4*>(fl + s * ROWS * D + 32 * x);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              float4 a = make_float4(__uint_as_float(o[4 * e]), __uint_as_float(o[4 * e + 1]), __uint_as_float(o[4 * e + 2]), __uint_as_float(o[4 * e + 3]));
              if (flushed) {
                const float4 z = y[e];
                a.x += z.x; a.y += z.y; a.z += z.z; a.w += z.w;
              }
              y[e] = a;
            }
          }
          flushed = true;
          tc_fence_before();
          mbar_arrive(o_empty + 8 * s);
        }
      }
      if (!ok) break;
      // ---- the item's end
      if (!all(mbar_wait(o_full + 8 * s, items & 1))) { ok = false; break; }
      tc_fence_after();
      float f0 = 1.f, f1 = 0.f;
      bool other = false;   // stream 1's share is added here
      if (it.w == 1) {
        if (s == 1) {
          // stream 0 writes for both
          xch[(turns & 1) * ROWS + lr] = make_float2(m, l);
          mbar_arrive(x_full);
          ++turns;
          continue;
        }
        if (!all(mbar_wait(x_full, turns & 1))) { ok = false; break; }
        const float2 y = xch[(turns & 1) * ROWS + lr];
        ++turns;
        other = units_of(it, 1) > 0;
        const float top = fmaxf(m, y.x);
        if (top != kNegInf) {
          f0 = m == kNegInf ? 0.f : ex2(m - top);
          f1 = y.x == kNegInf ? 0.f : ex2(y.x - top);
        }
        if (top != top) f0 = f1 = top;
        l = f0 * l + f1 * y.y;
        m = top;
      }
      const bool other_flushed = other && units_of(it, 1) > kFlush;
      const bool odd = misc[2] != 0;
      const float inv = l == 0.f ? 0.f : 1.f / l;
      const int slot = it.j0 > 0 ? 0 : 1;
      const size_t part = ((size_t(r) * 2 + slot) * 2 + (tile & 1)) * ROWS + lr;
      const float bias = P.g != nullptr && real ? bf2f(P.gate_bias[hq]) : 0.f;
#pragma unroll 1
      for (int x = 0; x < D / 32; ++x) {
        uint32_t o[32];
        tmem_ld32_nowait(to + 32 * x, o);
        tmem_wait_ld();
        float a[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) a[e] = f0 == 0.f ? 0.f : __uint_as_float(o[e]) * f0;
        if (flushed)
#pragma unroll
          for (int e = 0; e < 32; ++e) a[e] += fl[s * ROWS * D + 32 * x + e] * f0;
        if (other) {
          tmem_ld32_nowait(to + 256 + 32 * x, o);
          tmem_wait_ld();
          if (f1 != 0.f)
#pragma unroll
            for (int e = 0; e < 32; ++e) a[e] += __uint_as_float(o[e]) * f1;
          if (other_flushed && f1 != 0.f)
#pragma unroll
            for (int e = 0; e < 32; ++e) a[e] += fl[ROWS * D + 32 * x + e] * f1;
        }
        if (!real) continue;
        if (l == 0.f)
#pragma unroll
          for (int e = 0; e < 32; ++e) a[e] = 0.f;
        if (odd) add_no_numbers<FMT, D>(P, it, v, 32 * x, a);
        if (it.split) {
          float4* y = reinterpret_cast<float4*>(P.part_acc + part * D + 32 * x);
#pragma unroll
          for (int e = 0; e < 8; ++e) y[e] = make_float4(a[4 * e], a[4 * e + 1], a[4 * e + 2], a[4 * e + 3]);
        } else {
#pragma unroll
          for (int e = 0; e < 8; e += 2) {
            const uint2 u0 = finish4(P, make_float4(a[4 * e] * inv, a[4 * e + 1] * inv, a[4 * e + 2] * inv, a[4 * e + 3] * inv), at + 32 * x + 4 * e, bias);
            const uint2 u1 = finish4(P, make_float4(a[4 * e + 4] * inv, a[4 * e + 5] * inv, a[4 * e + 6] * inv, a[4 * e + 7] * inv), at + 32 * x + 4 * e + 4, bias);
            *reinterpret_cast<uint4*>(P.og + at + 32 * x + 4 * e) = make_uint4(u0.x, u0.y, u1.x, u1.y);
          }
        }
      }
      if (it.split && real) P.part_ml[part] = make_float2(m, l);
      tc_fence_before();
      if (units > 0) mbar_arrive(o_empty + 8 * s);
      if (other) mbar_arrive(o_empty + 8);
      if (it.split && it.j0 == 0)   // the item begins here and runs on
        join = make_int4(it.i, it.h | it.m << 16, range_of(it.f + it.w * (it.s.nb - 1), total, R) - r + 1, it.w);
    }
    if (!ok) misc[1] = 1;
    if (threadIdx.x == 4 * 32) P.join[r] = join;
  } else if (warp >= 12) {
    // ------------------------------------------------------------------ codes to bf16 tiles
    if constexpr (C::QUANT) {
      const int tid = threadIdx.x - 12 * 32;
      uint32_t nb = 0;
      bool ok = true, odd = false;
      auto all = [&](bool v) { return __all_sync(0xffffffffu, v); };
      Item it;
      for (int c = c0; ok && next_item(P, cum, c, c1, it);) {
        for (int j = it.j0; j < it.j1; ++j, ++nb) {
          const int rs = int(nb % NRAW), st = int(nb % NST);
          const uint32_t ph = ((nb / NST) & 1) ^ 1;
          if (!all(mbar_wait(r_full + 8 * rs, (nb / NRAW) & 1))) { ok = false; break; }
          const unsigned live = masks[rs];
          const bool whole = live == 15u && whole_block(P, it.s, j);
          const int kb = (it.s.blk0 + j) * BK + 1;
          const uint8_t* raw = sm + C::R0 + rs * C::RAW;
#pragma unroll
          for (int kv = 0; kv < 2; ++kv) {
            if (!all(mbar_wait((kv ? v_empty : k_empty) + 8 * st, ph))) { ok = false; break; }
            uint8_t* tile = sm + (kv ? C::V0 : C::K0) + st * C::TILE;
#pragma unroll
            for (int x = tid; x < BK * (D / 16); x += 256) {
              const int row = x / (D / 16), gr = x % (D / 16), key = kb + row;
              const unsigned b = raw[2 * C::RAWK + 2 * C::RBS + kv * BK + row];
              const float f = pow2_of(b);
              uint32_t w[8];
              if constexpr (FMT == kFmtFP8) {
                const uint4 y = *reinterpret_cast<const uint4*>(raw + kv * C::RAWK + row * C::ROWB + gr * 16);
                const uint32_t code[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  uint32_t h[2];
                  e4m3x4_f16(code[e], h[0], h[1]);
#pragma unroll
                  for (int z = 0; z < 2; ++z) {
                    float a0, a1;
                    unpack_f16(h[z], a0, a1);
                    w[2 * e + z] = pack_bf16x2(a0 * f, a1 * f);
                  }
                }
              } else {
                const uint2 y = *reinterpret_cast<const uint2*>(raw + kv * C::RAWK + row * C::ROWB + gr * 8);
                float sf, unused;
                unpack_f16(e4m3x2_f16x2(raw[2 * C::RAWK + kv * C::RBS + x]), sf, unused);
                const float unit = sf * f;
                uint32_t h[8];
                e2m1x8_f16(y.x, h);
                e2m1x8_f16(y.y, h + 4);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                  float a0, a1;
                  unpack_f16(h[e], a0, a1);
                  w[e] = pack_bf16x2(a0 * unit, a1 * unit);
                }
              }
              if (kv == 1 && !whole) {   // rows outside the item's keys, and rows that are no numbers
                const bool in = key >= it.s.lo && key <= it.s.base + it.s.n && ((live >> (row >> 4)) & 1u);
                if (in && b == 255) odd = true;
                if (!in || b == 255)
#pragma unroll
                  for (int e = 0; e < 8; ++e) w[e] = 0;
              }
              uint8_t* to = tile + (gr >> 2) * BK * 128 + row * 128;
              const int ch = (2 * gr) & 7;
              *reinterpret_cast<uint4*>(to + ((ch ^ (row & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
              *reinterpret_cast<uint4*>(to + (((ch + 1) ^ (row & 7)) << 4)) = make_uint4(w[4], w[5], w[6], w[7]);
            }
            if (odd) misc[2] = 1;
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive((kv ? v_full : k_full) + 8 * st);
          }
          if (!ok) break;
          if (lane == 0) mbar_arrive(r_empty + 8 * rs);
        }
      }
      if (!ok) misc[1] = 1;
    }
  } else {
    // ------------------------------------------------------------------ warps 2, 3: rows that attend to nothing
    const int tid = threadIdx.x - 64, wide = P.n_q * (D / 8);
    auto zero = [&](int a, int b) {   // rows a..b-1, this CTA's of them
      for (int t = max(a, 0) + r; t < min(b, P.T); t += int(gridDim.x))
        for (int x = tid; x < wide; x += 64)
          reinterpret_cast<uint4*>(P.og + size_t(t) * P.n_q * D)[x] = make_uint4(0, 0, 0, 0);
    };
    if (P.head_rows) zero(0, P.row_start[0]);
    if (P.tail_rows) zero(P.row_start[P.N], P.T);
    for (int i = 0; i < P.N; ++i)
      if (cum[i + 1] == cum[i]) zero(P.row_start[i], P.row_start[i + 1]);
  }
  tc_fence_before();
  __syncthreads();
  pdl_trigger();   // not earlier: the join and what follows would run beside the key stream
  if (threadIdx.x == 0 && misc[1]) flag(BEAM_DEV_TIMEOUT);
  if (warp == 1)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
}

// Join of the item that begins in range blockIdx.x and runs on past it: tile blockIdx.y, 16 rows a CTA, 16 threads a
// row.
template <int D>
__global__ void __launch_bounds__(256) paged_tree_join_kernel(const Params P) {
  pdl_trigger();
  pdl_wait();
  const int4 jn = P.join[blockIdx.x];
  if (jn.z == 0 || int(blockIdx.y) >= jn.w) return;
  const int lr = blockIdx.z * 16 + threadIdx.x / 16, d = (threadIdx.x % 16) * (D / 16);
  const int h = jn.y & 0xFFFF, tile = 2 * (jn.y >> 16) + blockIdx.y;
  const int row0 = P.row_start[jn.x], n = P.row_start[jn.x + 1] - row0;
  const int row = tile * ROWS + lr, node = row / P.G, hq = h * P.G + (row - node * P.G);
  if (node >= n) return;
  auto at = [&](int s) { return ((size_t(blockIdx.x + s) * 2 + (s == 0 ? 1 : 0)) * 2 + blockIdx.y) * ROWS + lr; };
  float M = kNegInf;
  for (int s = 0; s < jn.z; ++s) M = fmaxf(M, __ldcg(&P.part_ml[at(s)]).x);
  float L = 0.f, O[D / 16];
#pragma unroll
  for (int e = 0; e < D / 16; ++e) O[e] = 0.f;
  for (int s = 0; s < jn.z; ++s) {
    const float2 ml = __ldcg(&P.part_ml[at(s)]);
    const float f = ml.y == 0.f ? 0.f : ex2(ml.x - M);
    if (ml.y == 0.f) continue;   // no key of this part
    L += f * ml.y;
#pragma unroll
    for (int e = 0; e < D / 16; e += 4) {
      const float4 v = __ldcg(reinterpret_cast<const float4*>(P.part_acc + at(s) * D + d + e));
      O[e] += f * v.x; O[e + 1] += f * v.y; O[e + 2] += f * v.z; O[e + 3] += f * v.w;
    }
  }
  const float inv = L == 0.f ? 0.f : 1.f / L;
  const float bias = P.g != nullptr ? bf2f(P.gate_bias[hq]) : 0.f;
  const size_t o = (size_t(row0 + node) * P.n_q + hq) * D + d;
#pragma unroll
  for (int e = 0; e < D / 16; e += 4)
    *reinterpret_cast<uint2*>(P.og + o + e) = finish4(P, make_float4(O[e] * inv, O[e + 1] * inv, O[e + 2] * inv, O[e + 3] * inv), o + e, bias);
}

template <int FMT, int D>
cudaError_t allow_smem() {
  static std::atomic<bool> done[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 64 && done[dev].load(std::memory_order_relaxed)) return cudaSuccess;
  e = cudaFuncSetAttribute(paged_tree_kernel<FMT, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<FMT, D>::BYTES);
  if (e == cudaSuccess && dev < 64) done[dev].store(true, std::memory_order_relaxed);
  return e;
}

int max_grid() {
  const int sms = num_sms_cached();
  return sms < kGrid ? sms : kGrid;
}

template <int FMT, int D>
cudaError_t launch(const Params& p, cudaStream_t st) {
  using C = Cfg<FMT, D>;
  const beam_paged_kv& c = p.c;
  CUtensorMap mk{}, mv{};
  if (!C::QUANT) {
    const uint64_t dims[3] = {uint64_t(2 * D), uint64_t(c.page_size), uint64_t(c.num_pages) * c.n_kv};
    const uint64_t str[2] = {uint64_t(2 * D), uint64_t(c.page_size) * 2 * D};
    const uint32_t box[3] = {128, uint32_t(c.page_size < BK ? c.page_size : BK), 1};
    if (!encode_tiled(&mk, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, c.k, dims, str, box, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_tiled(&mv, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, c.v, dims, str, box, CU_TENSOR_MAP_SWIZZLE_128B))
      return cudaErrorInvalidValue;
  }
  cudaError_t e = allow_smem<FMT, D>();
  if (e != cudaSuccess) return e;
  const int grid = max_grid();
  e = launch_pdl(paged_tree_kernel<FMT, D>, dim3(grid), dim3(C::THREADS), C::BYTES, st, mk, mv, p);
  if (e != cudaSuccess) return e;
  const int tiles = p.G * kNodes > ROWS ? 2 : 1;
  return launch_pdl(paged_tree_join_kernel<D>, dim3(grid, tiles, ROWS / 16), dim3(256), 0, st, p);
}

constexpr size_t kParts = size_t(kGrid) * 2 * 2 * ROWS;   // rows of partial results

}  // namespace
}  // namespace paged
}  // namespace beam

extern "C" size_t beam_paged_tree_workspace_bytes(const beam_layer_cfg* cfg, int T) {
  using namespace beam;
  using namespace beam::paged;
  if (cfg == nullptr || T <= 0 || cfg->n_q <= 0 || cfg->head_dim <= 0) return 256;
  const size_t D = cfg->head_dim;
  return align_up(kParts * D * 4, 256) + align_up(kParts * 8, 256) + align_up(kGrid * sizeof(int4), 256) +
         align_up(size_t(kGrid) * 2 * ROWS * D * 4, 256) + align_up(size_t(T) * cfg->n_q * D * 2, 256);
}

extern "C" beam_status beam_paged_tree_attn(const beam_layer_cfg* cfg, const beam_bf16* q, const beam_bf16* g,
                                            const beam_bf16* gate_bias, const beam_paged_kv* cache,
                                            const int32_t* seq_id, const int32_t* row_start,
                                            const int32_t* base, const uint64_t* mask, int N, int T,
                                            int max_pos, const beam_bf16* w_o, beam_bf16* out, void* ws,
                                            size_t ws_bytes, beam_stream_t stream) {
  using namespace beam;
  using namespace beam::paged;
  beam_status stt = check_cfg_attn(cfg);
  if (stt != BEAM_OK) return stt;
  if ((stt = check(cache)) != BEAM_OK) return stt;
  if (cache->n_kv != cfg->n_kv || cache->head_dim != cfg->head_dim || N < 0 || T < 0 || max_pos < 0)
    return BEAM_ERR_INVALID_ARG;
  if (T == 0) return BEAM_OK;
  if (N == 0 || !q || !seq_id || !row_start || !base || !mask || !out || !ws || (g == nullptr) != (gate_bias == nullptr))
    return BEAM_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16_or_null(g) || !aligned16_or_null(w_o) || !aligned16(out) ||
      (reinterpret_cast<uintptr_t>(ws) & 255u) || (reinterpret_cast<uintptr_t>(mask) & 7u))
    return BEAM_ERR_INVALID_ARG;
  const int D = cfg->head_dim, HD = cfg->n_q * D, G = cfg->n_q / cfg->n_kv;
  // most blocks of a sequence: costs are 32-bit
  const int64_t table = int64_t(cache->table_stride) * cache->page_size;
  int64_t keys = max_pos < table ? max_pos : table;
  if (cache->window > 0 && int64_t(cache->window) + kNodes < keys) keys = int64_t(cache->window) + kNodes;
  const int64_t nb = keys / BK + 2;
  const int slice = N < kMaxSeqs ? N : kMaxSeqs;
  if (nb * ((kNodes * G + ROWS - 1) / ROWS) * slice * cfg->n_kv > 1 << 30 || cfg->n_kv > 65535) return BEAM_ERR_UNSUPPORTED;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  Carver cv{static_cast<char*>(ws), ws_bytes};
  Params p{};
  p.part_acc = cv.take<float>(kParts * D);
  p.part_ml = cv.take<float2>(kParts);
  p.join = cv.take<int4>(kGrid);
  p.flush = cv.take<float>(size_t(kGrid) * 2 * ROWS * D);
  uint16_t* og = w_o ? cv.take<uint16_t>(size_t(T) * HD) : out;
  if (!cv.ok) return BEAM_ERR_INVALID_ARG;
  if (!tc::tensor_map_encoder_ready()) return BEAM_ERR_UNSUPPORTED;
  p.q = q;
  p.g = g;
  p.gate_bias = gate_bias;
  p.mask = mask;
  p.og = og;
  p.c = *cache;
  p.T = T;
  p.n_q = cfg->n_q;
  p.n_kv = cfg->n_kv;
  p.G = G;
  p.max_pos = max_pos;
  p.shift = log2i(cache->page_size);
  p.least = 4;
  p.sl2 = float(1.4426950408889634 / sqrt(double(D)));
  for (int i0 = 0; i0 < N; i0 += kMaxSeqs) {   // slices in stream order share the workspace
    p.N = N - i0 < kMaxSeqs ? N - i0 : kMaxSeqs;
    p.seq_id = seq_id + i0;
    p.row_start = row_start + i0;
    p.base = base + i0;
    p.head_rows = i0 == 0;
    p.tail_rows = i0 + p.N == N;
    const bool wide = D == 128;
    cudaError_t e;
    if (cache->dtype == kFmtBF16) e = wide ? launch<kFmtBF16, 128>(p, st) : launch<kFmtBF16, 64>(p, st);
    else if (cache->dtype == kFmtFP8) e = wide ? launch<kFmtFP8, 128>(p, st) : launch<kFmtFP8, 64>(p, st);
    else e = wide ? launch<kFmtNVFP4, 128>(p, st) : launch<kFmtNVFP4, 64>(p, st);
    if (e != cudaSuccess) return cuda_status(e);
  }
  if (w_o != nullptr) {
    const cudaError_t ge = o_proj(og, T, HD, w_o, cfg->hidden, out, st);
    if (ge != cudaSuccess) return cuda_status(ge);
  }
  return BEAM_OK;
}
