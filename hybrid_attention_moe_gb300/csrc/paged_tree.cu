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
// TMEM columns of stream s, from 256 s: two buffers of S, then P over it, [0, 64) and [64, 128); O [128, 128 + D).
//   S = Q . K^T      A = Q, B = K block (shared memory, both K-major)
//   O += P . V       A = P (TMEM), B = V block (MN-major)
// A stream's next S is made while its softmax works on this one. BF16 pages: P is split into a high and a low bf16 half, so
// that the products keep FP32's accuracy. FP8 and NVFP4 pages: codes become f16 exactly, q becomes f16 by a power of two
// for each row (exact down to 2^-31 of the row's largest magnitude), the rows' own powers of two go to the
// logits (K) and to P (V), and P is rounded to f16 once (2^-11); its reference z follows the weights times their value
// rows' powers, so that a large value row of small weight keeps its bits, and what it takes from others is below 2^-32 of it (a
// block's first half goes to a new reference through FP32).
//
// The blocks of all items, laid end to end and weighed by their tiles, with a cost for each item besides, are cut into
// equal ranges, one for each CTA; partials of an item that several ranges share go to the workspace and a second kernel
// joins them. Ranges are planned on the device from the sequences' own lengths.
//
// Warps: 0 loads keys and 2 values (page table and TMA); 1 and 3 issue the streams' matrix products (the tensor pipe
// queues only a few, so what one spends on waits the other's products cover); 4-7 and 8-11 are the streams' softmax (a
// thread per row); over FP8 and NVFP4 pages 12-15 turn keys' codes and 16-19 values' codes into f16 tiles; over
// BF16 pages 12-15 clean blocks (below). From 12 on they first write the rows that attend to nothing.
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
//
// Measured with the join, 48 query and 8 KV heads of 128, pages of 64 (us; in brackets the floor of bytes or products):
//   1 sequence, 100K keys, BF16:   16 nodes 86 (60.5: keys at 4.8 TB/s)   64 nodes 186 (81; three tiles, the third read apart)
//                          FP8:    16 nodes 114 (30.5)                    64 nodes 289 (81)
//   32 sequences of 1 to 16 nodes over up to 16K keys:   BF16 219 (157)   FP8 259 (80)   NVFP4 270 (45)
//   1 sequence, 200 keys, 5 nodes: 17.3 (launch, plan 1, queries 3, four blocks 3, output 6, join)
// BF16 of one tile is bound by the key stream and the 10 us around it, of more by the streams' softmax beside the tensor pipe (a unit
// of 64 keys by 128 rows takes a stream 2.8K cycles, 1.5K of them arithmetic; the products 0.9K). Quantised pages are bound by
// issue slots: 1100 of them each block and SM sub-partition, of 2200 cycles, a third in the conversion, 40 % in the softmax.
// What paid, at 32 sequences over FP8 (us): first kernel 568; f16 and P by z 543; ranges that count an item's own cost 286 (the
// last CTA had 24 short items); conversions by turns of whole rows 276; output by sectors 263; P up to all of f16's range before its
// reference moves 259. Not kept: 32-wide output columns shared by the streams and queries
// and output out of line (registers of the loop over blocks: 16 nodes over FP8 119 -> 131 and 138), halves of an item of one tile
// for each stream (the keys of 64 nodes read once: 193 -> 197, not what bounds it).
// Without relocatable device code the status word's declaration is a variable of this unit's own, which nothing here
// uses: the kernel's bits go through the join.
#pragma nv_diag_suppress 20044
#include <cuda.h>

#include <atomic>

#include "paged_tree.cuh"
#include "tcgen05.cuh"

namespace beam {
namespace paged {
namespace tree {
namespace {

using namespace beam::tc;

// What the codes of a block's 64 keys leave to the softmax: K's powers of two relative to the largest, 2^top, and the
// exponents of V's.
struct Factors {
  float k[BK], v[BK], top, pad[3];
};
// Blocks that may be in use at once, from the loads of keys to the softmax: a stream at block c has S of c + 2 at most
// (items of one tile), c + 4 holds a stage, and up to eight stages (three, and three of codes) go on from there.
constexpr int kFac = 16;

template <int FMT, int D_>
struct Cfg {
  static constexpr int D = D_, ROWB = row_bytes(FMT, D);
  static constexpr bool QUANT = FMT != kFmtBF16;
  static constexpr int THREADS = QUANT ? 640 : 512;
  // registers of a thread: at launch (a fifth or a quarter of the SM's for each four warps), then of the softmax and of
  // the other warps; the shares add up to no more than the launch's
  static constexpr int REG = QUANT ? 96 : 128, REG_S = QUANT ? 144 : 200, REG_L = QUANT ? 64 : 56, REG_C = QUANT ? 64 : 56;
  static_assert(2 * REG_S + REG_L + (QUANT ? 2 : 1) * REG_C <= THREADS / 128 * REG, "register split");
  static constexpr int NH = D / 64;                 // 64-wide halves of a row
  static constexpr int TILE = BK * D * 2;           // K or V block in bf16
  static constexpr int NST = QUANT ? 3 : (D == 128 ? 4 : 8);
  static_assert(QUANT || NST % 2 == 0, "stages that keys' copies fill in any order: of items of one tile each is one stream's");
  static constexpr int RAWB = QUANT ? BK * ROWB : 0;
  static constexpr int RBS = FMT == kFmtNVFP4 ? BK * (D / 16) : 0;
  static constexpr int RAW = QUANT ? RAWB + RBS + 2 * BK : 0;   // a raw stage: codes, block scales, row scales (with K's: both)
  static constexpr int NRAW = QUANT ? 3 : 0;
  static constexpr int Q0 = 0, QB = ROWS * D * 2;           // each stream's query tile
  static constexpr int K0 = 2 * QB, V0 = K0 + NST * TILE;
  static constexpr int R0 = V0 + NST * TILE;                // raw stages of K, then of V
  static constexpr int SEQ = (R0 + 2 * NRAW * RAW + 15) / 16 * 16;   // [kMaxSeqs] (row0, n, sid, base)
  static constexpr int CUM = SEQ + kMaxSeqs * 16;                    // [kMaxSeqs + 1] cost prefix
  static constexpr int FAC = CUM + (kMaxSeqs + 4) * 4;               // [kFac] factors of a block's keys (Factors)
  static constexpr int XCH = FAC + (QUANT ? kFac * int(sizeof(Factors)) : 0);   // [128] (m, z, sum) of stream 1
  static constexpr int MASK = XCH + ROWS * 16;                    // [2][8] slices of a K or V stage that have a page
  static constexpr int LIVE = MASK + 16 * 4;                      // [kFac] the same of the blocks that may be in use at once
  static constexpr int BAR = LIVE + kFac * 4;
  static constexpr int NBAR = 5 * NST + 4 * NRAW + 22;
  static constexpr int MISC = BAR + NBAR * 8;
  static constexpr int BYTES = MISC + 32 + 1024;
  static_assert(BYTES <= 227 * 1024, "shared memory");
};

// A sequence as the plan found it; one that is out of range has no rows. What the kernel does hangs on these words alone,
// which every CTA keeps, so inputs that change under it cannot take it out of bounds.
__device__ __forceinline__ int4 read_seq(const Params& P, int i, unsigned& bad) {
  int4 s = make_int4(P.row_start[i], P.row_start[i + 1], P.seq_id[i], P.base[i]);
  s.y -= s.x;
  bad = 0;
  if (s.y < 0 || s.y > kNodes || s.x < 0 || s.x > P.T - max(0, s.y)) bad = BEAM_DEV_BAD_SEQ;
  else if (s.y > 0 && (s.z < 0 || s.z >= P.c.num_seqs)) bad = BEAM_DEV_BAD_SEQ;
  else if (s.y > 0 && (s.w < 0 || s.w > P.max_pos - s.y || ((s.w + s.y - 1) >> P.shift) >= P.c.table_stride))
    bad = BEAM_DEV_BAD_POSITION;
  if (bad) s.y = 0;
  return s;
}
struct Seq {
  int row0, n, sid, base, lo, blk0, nb, tiles;
};
__device__ __forceinline__ Seq seq_of(const Params& P, const int4& w) {
  Seq s;
  s.row0 = w.x;
  s.n = w.y;
  s.sid = w.z;
  s.base = w.w;
  s.lo = P.c.window > 0 ? max(1, s.base + 2 - P.c.window) : 1;
  s.blk0 = s.n == 0 ? 0 : (s.lo - 1) / BK;
  s.nb = s.n == 0 ? 0 : (s.base + s.n - 1) / BK - s.blk0 + 1;
  s.tiles = (s.n * P.G + ROWS - 1) / ROWS;
  return s;
}

// Cost of a sequence's items of one head: their blocks by their tiles, and P.item for each, before its blocks: what an
// item costs beside them.
__device__ __forceinline__ int cost_of(const Params& P, const Seq& s) { return s.nb * s.tiles + P.item * ((s.tiles + 1) / 2); }

// A CTA's share [j0, j1) of the blocks of item m (tiles 2m, 2m + 1) of one (sequence, KV head).
struct Item {
  Seq s;
  int h, m, w, j0, j1, f, next;   // w: its tiles; f: cost at its first block
  int wa, wb;                     // all rows see all keys of blocks wa..wb-1 (their pages aside)
  bool split;
  __device__ __forceinline__ bool whole(int j) const { return j >= wa && j < wb; }
};

// Smallest cost of range r; the range of cost c.
__device__ __forceinline__ int range_lo(int r, int total, int R) { return int(int64_t(r) * total / R); }
__device__ __forceinline__ int range_of(int c, int total, int R) {
  return int((int64_t(c + 1) * R - 1) / total);
}

// The item at cost c of the range that ends at c1.
struct Plan {
  const int* cum;
  const int4* seq;
};
__device__ __forceinline__ Item item_at(const Params& P, const Plan& L, int c, int c1) {
  const int* cum = L.cum;
  int a = 0, b = P.N;   // cum[a] <= c < cum[b]
  while (b - a > 1) {
    const int mid = (a + b) >> 1;
    if (cum[mid] <= c) a = mid;
    else b = mid;
  }
  Item it;
  it.s = seq_of(P, L.seq[a]);
  const int per = cost_of(P, it.s), pair = 2 * it.s.nb + P.item, off = c - cum[a];
  it.h = off / per;
  const int rest = off - it.h * per;
  it.m = rest / pair;
  it.w = 2 * it.m + 1 < it.s.tiles ? 2 : 1;
  it.f = c - rest + it.m * pair + P.item;
  it.j0 = max(0, c - it.f + it.w - 1) / it.w;
  it.next = it.f + it.w * it.s.nb;
  it.j1 = it.next <= c1 ? it.s.nb : max(0, c1 - it.f + it.w - 1) / it.w;
  it.split = it.j0 > 0 || it.j1 < it.s.nb;
  const int hi = P.c.window > 0 ? max(0, it.s.base + it.s.n - P.c.window) : 0;   // before the deepest row's first key
  it.wa = (hi + BK - 1) / BK - it.s.blk0;
  it.wb = it.s.base / BK - it.s.blk0;
  return it;
}
// The next item of a range that has blocks in it, from cost c on.
__device__ __forceinline__ bool next_item(const Params& P, const Plan& L, int& c, int c1, Item& it) {
  while (c < c1) {
    it = item_at(P, L, c, c1);
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

// Page table entry of the e-th 16 keys of block j, compared with the pages' number where it is used (a load ahead of that
// waits for nothing); -2: no key of the item among them.
__device__ __forceinline__ int entry_of_slice(const Params& P, const Seq& s, int j, int e) {
  const int k0 = (s.blk0 + j) * BK + 16 * e;   // 0-based
  if (k0 + 16 < s.lo || k0 >= s.base + s.n) return -2;
  return P.c.page_table[size_t(s.sid) * P.c.table_stride + (k0 >> P.shift)];
}
// The page, -1: none, -2: no key.
__device__ __forceinline__ int page_of_entry(const Params& P, const Seq& s, int j, int e, int entry) {
  const int k0 = (s.blk0 + j) * BK + 16 * e;
  if (k0 + 16 < s.lo || k0 >= s.base + s.n) return -2;
  return entry >= 0 && entry < P.c.num_pages ? entry : -1;
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t mbar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
          "r"(dst), "l"(src), "r"(bytes), "r"(mbar)
      : "memory");
}
// mbar_wait whose polls may suspend the thread for some microseconds: the many waiting warps of a CTA would otherwise poll
// away a quarter of its issue slots. False after about two seconds.
__device__ __forceinline__ bool wait(uint32_t a, uint32_t parity) {
  for (uint32_t i = 0; i < 1u << 18; ++i) {
    uint32_t ok;
    asm volatile(
        "{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3; selp.u32 %0, 1, 0, p; }"
        : "=r"(ok)
        : "r"(a), "r"(parity), "r"(8000u)
        : "memory");
    if (ok) return true;
  }
  return false;
}
// Arrival of a whole warp, once.
__device__ __forceinline__ void arrive(uint32_t a) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(a);
}
template <int N, bool MORE>
__device__ __forceinline__ void set_regs() {
  if (MORE) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
  else asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
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
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
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

__device__ __forceinline__ void l1_prefetch(const void* p) { asm volatile("prefetch.global.L1 [%0];" ::"l"(p)); }

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
      if (page_of_entry(P, s, j, e, entry_of_slice(P, s, j, e)) >= 0) slices |= 1u << e;
    if (it.whole(j) && slices == 15u) continue;
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
__global__ void __launch_bounds__(FMT == kFmtBF16 ? 512 : 640, 1)
paged_tree_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv, const Params P) {
  using C = Cfg<FMT, D>;
  constexpr int NST = C::NST, NRAW = C::NRAW;
  // bf16, or f16 over quantised pages: there the two format fields are zero
  constexpr uint32_t KIND = C::QUANT ? ~((1u << 7) | (1u << 10)) : ~0u;
  constexpr uint32_t IDESC_QK = idesc_bf16(ROWS, BK, false) & KIND, IDESC_PV = idesc_bf16(ROWS, D, true) & KIND;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = smem_u32(sm);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int* cum = reinterpret_cast<int*>(sm + C::CUM);
  uint32_t* masks = reinterpret_cast<uint32_t*>(sm + C::MASK);
  uint32_t* lives = reinterpret_cast<uint32_t*>(sm + C::LIVE);
  volatile int* misc = reinterpret_cast<volatile int*>(sm + C::MISC);   // TMEM address, abort, no numbers, status
  unsigned* status = reinterpret_cast<unsigned*>(sm + C::MISC) + 3;
  int4* seqs = reinterpret_cast<int4*>(sm + C::SEQ);
  const Plan plan{cum, seqs};
  // barriers; those of a stream's S buffers and of raw stages come in pairs [stream][buffer], [K | V][stage]
  const uint32_t k_full = sb + C::BAR, k_empty = k_full + 8 * NST, v_full = k_empty + 8 * NST,
                 v_empty = v_full + 8 * NST, r_full = v_empty + 8 * NST, r_empty = r_full + 16 * NRAW;
  const uint32_t q_full = r_empty + 16 * NRAW, s_full = q_full + 16, p_full = s_full + 32, pv_done = p_full + 32,
                 o_full = pv_done + 16, o_empty = o_full + 16, x_full = o_empty + 16, x_empty = x_full + 8, v_clean = x_empty + 8,
                 meet = v_clean + 8 * NST;   // [item's parity][stream]
  if (threadIdx.x == 0) {
    for (int i = 0; i < NST; ++i) {
      mbar_init(k_full + 8 * i, C::QUANT ? 4 : 1);
      mbar_init(k_empty + 8 * i, 2);   // both streams
      mbar_init(v_full + 8 * i, C::QUANT ? 4 : 1);
      mbar_init(v_empty + 8 * i, 2);
      mbar_init(v_clean + 8 * i, 4);   // of BF16 values, in place of v_full: looked through, and cleaned if need be
    }
    for (int i = 0; i < 2 * NRAW; ++i) {
      mbar_init(r_full + 8 * i, 1);
      mbar_init(r_empty + 8 * i, 4);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(q_full + 8 * s, 4);
      mbar_init(meet + 8 * s, 1);
      mbar_init(meet + 16 + 8 * s, 1);
      for (int i = 0; i < 2; ++i) {
        mbar_init(s_full + 16 * s + 8 * i, 1);
        mbar_init(p_full + 16 * s + 8 * i, 4);
      }
      mbar_init(pv_done + 8 * s, 1);
      mbar_init(o_full + 8 * s, 2);
      mbar_init(o_empty + 8 * s, 4);
    }
    mbar_init(x_full, 4);
    mbar_init(x_empty, 4);
    misc[1] = 0;
    misc[2] = 0;
    *status = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(sb + C::MISC), "r"(512) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  pdl_wait();
  // ---- plan: prefix sums of the sequences' costs
  if (warp == 0) {
    int carry = 0;
    if (lane == 0) cum[0] = 0;
    for (int i0 = 0; i0 < P.N; i0 += 32) {
      int c = 0;
      if (i0 + lane < P.N) {
        unsigned bad;
        const int4 w = read_seq(P, i0 + lane, bad);
        seqs[i0 + lane] = w;
        const Seq s = seq_of(P, w);
        c = s.n == 0 ? 0 : cost_of(P, s) * P.n_kv;
        if (bad && blockIdx.x == 0) atomicOr(status, bad);
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

  if (warp < 4) {
  set_regs<C::REG_L, false>();
  if (warp == 0 || warp == 2) {
    // ------------------------------------------------------------------ loads: keys, or values
    const int kv = warp >> 1, first_lane = lane < 4 ? lane : 0;
    const uint8_t* pool = static_cast<const uint8_t*>(kv ? P.c.v : P.c.k);
    const uint32_t full = C::QUANT ? r_full + 8 * kv * NRAW : (kv ? v_full : k_full);
    const uint32_t empty = C::QUANT ? r_empty + 8 * kv * NRAW : (kv ? v_empty : k_empty);
    constexpr uint32_t DEPTH = C::QUANT ? NRAW : NST;
    const int run = P.c.page_size >= BK ? 4 : P.c.page_size / 16;   // slices that one copy covers
    const int e0 = first_lane / run * run;
    uint32_t nb = 0;   // blocks issued
    bool ok = true;
    Item it;
    for (int c = c0; ok && next_item(P, plan, c, c1, it);) {
      int entry = lane < 4 ? entry_of_slice(P, it.s, it.j0, lane) : -2;
      for (int j = it.j0; j < it.j1; ++j, ++nb) {
        const int pg = lane < 4 ? page_of_entry(P, it.s, j, lane, entry) : -2;
        if (pg == -1 && kv == 0 && it.h == 0 && it.m == 0) atomicOr(status, BEAM_DEV_BAD_PAGE);
        const unsigned live = __ballot_sync(0xffffffffu, pg >= 0) & 15u;
        const int k0 = (it.s.blk0 + j) * BK;
        // any slice of a copy's that has keys names its page
        const int first = __ffs((live >> e0) & ((1u << run) - 1u));
        const int page = __shfl_sync(0xffffffffu, pg, first ? e0 + first - 1 : 0);
        const bool mine = lane < 4 && lane == e0 && first != 0;
        const int copies = __popc(__ballot_sync(0xffffffffu, mine));
        const int off = (k0 + 16 * e0) & (P.c.page_size - 1);
        const size_t head = size_t(mine ? page : 0) * P.c.n_kv + it.h;
        entry = lane < 4 && j + 1 < it.j1 ? entry_of_slice(P, it.s, j + 1, lane) : -2;   // the next block's, meanwhile
        const int st = int(nb % DEPTH);
        if (!__all_sync(0xffffffffu, wait(empty + 8 * st, ((nb / DEPTH) & 1) ^ 1))) { ok = false; break; }
        const uint32_t keys = uint32_t(run * 16), bar = full + 8 * st;
        if (lane == 0) {
          masks[8 * kv + st] = live;
          if (kv == 0) lives[nb % kFac] = live;
          mbar_expect_tx(bar, uint32_t(copies) * keys * (C::QUANT ? C::ROWB + 2 - kv + (FMT == kFmtNVFP4 ? D / 16 : 0) : 2 * D));
        }
        __syncwarp();
        if (!mine) continue;
        if constexpr (!C::QUANT) {
#pragma unroll
          for (int x = 0; x < C::NH; ++x)
            tma_load_3d(sb + (kv ? C::V0 : C::K0) + st * C::TILE + x * BK * 128 + e0 * 16 * 128, kv ? &tv : &tk, 128 * x, off,
                        int(head), bar);
        } else {
          const uint32_t at = sb + C::R0 + (kv * NRAW + st) * C::RAW;
          const size_t sc = (head * 2 + kv) * P.c.page_size + off;
          bulk_load(at + e0 * 16 * C::ROWB, pool + (head * P.c.page_size + off) * C::ROWB, keys * C::ROWB, bar);
          if constexpr (FMT == kFmtNVFP4)
            bulk_load(at + C::RAWB + e0 * 16 * (D / 16), P.c.block_scale + sc * (D / 16), keys * (D / 16), bar);
          bulk_load(at + C::RAWB + C::RBS + e0 * 16, P.c.row_scale + sc, keys, bar);
          if (kv == 0) bulk_load(at + C::RAWB + C::RBS + BK + e0 * 16, P.c.row_scale + sc + P.c.page_size, keys, bar);   // V's
        }
      }
    }
    if (!ok) {
      misc[1] = 1;
      // copies in flight land before the CTA's shared memory goes away
      for (uint32_t b = nb > DEPTH ? nb - DEPTH : 0; b < nb; ++b) wait(full + 8 * (b % DEPTH), (b / DEPTH) & 1);
    }
  } else {
    // ------------------------------------------------------------------ matrix products of stream s
    // A step is one block that both streams take (items of two tiles) or every other block, which the stream alone takes
    // and releases. S of step x + 2 is issued behind P.V of step x, whose buffer it takes (operations of one thread run
    // in order). A stream may wait for a stage's phase only where the one before is known to be over: the stage's block
    // before was its own, or was filled before one that it has seen (the quantised pages' three stages are filled in
    // order), or is of an earlier item, all of which are over for both where the streams meet.
    const int s = warp >> 1;
    const uint32_t v_ready = C::QUANT ? v_full : v_clean;
    uint32_t nb = 0;                            // blocks of earlier items
    uint32_t sn = 0, un = 0, ost = 0, qn = 0;   // S issued, P.V issued, fresh O, Q
    bool ok = true;
    auto all = [&](bool v) { return __all_sync(0xffffffffu, v); };
    const uint64_t dq = smem_desc(sb + C::Q0 + s * C::QB), dk = smem_desc(sb + C::K0), dv = smem_desc_mn(sb + C::V0, BK * 128, 1024);
    const uint32_t dq_lo = uint32_t(dq), dq_hi = uint32_t(dq >> 32), dk_hi = uint32_t(dk >> 32), dv_hi = uint32_t(dv >> 32);
    const uint32_t t0 = tmem + 256 * s;
    auto qk = [&](int st) {
      const uint32_t klo = uint32_t(dk) + uint32_t((st * C::TILE) >> 4), buf = sn & 1;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk)
        umma_ss_e(t0 + 64 * buf, dq_lo + uint32_t(((kk >> 2) * ROWS * 128 + (kk & 3) * 32) >> 4), dq_hi,
                  klo + uint32_t(((kk >> 2) * BK * 128 + (kk & 3) * 32) >> 4), dk_hi, IDESC_QK, kk > 0 ? 1u : 0u);
      umma_commit_e(s_full + 16 * s + 8 * buf);
      ++sn;
    };
    auto pv = [&](int st, bool first) {
      const uint32_t lo = uint32_t(dv) + uint32_t((st * C::TILE) >> 4);
      const uint32_t ts = t0 + 64 * (un & 1), to = t0 + 128;
#pragma unroll
      for (int kk = 0; kk < BK / 16; ++kk) {
        const uint32_t b = lo + uint32_t((kk * 16 * 128) >> 4), a = ts + 32 * (kk >> 1) + 8 * (kk & 1);
        if constexpr (C::QUANT) {
          umma_ts_e(to, ts + 8 * kk, b, dv_hi, IDESC_PV, first && kk == 0 ? 0u : 1u);
        } else {
          umma_ts_e(to, a, b, dv_hi, IDESC_PV, first && kk == 0 ? 0u : 1u);
          umma_ts_e(to, a + 16, b, dv_hi, IDESC_PV, 1u);
        }
      }
      umma_commit_e(pv_done + 8 * s);
      ++un;
    };
    Item it;
    for (int c = c0; ok && next_item(P, plan, c, c1, it);) {
      const int cnt = it.j1 - it.j0, per = it.w == 2 ? 1 : 2, off = it.w == 2 ? 0 : s, steps = units_of(it, s);
      ok = all(wait(q_full + 8 * s, qn & 1));
      if (!ok) break;
      tc_fence_after();
      if (lane == 0) mbar_arrive(meet + 16 * (qn & 1) + 8 * (s ^ 1));
      ok = all(wait(meet + 16 * (qn & 1) + 8 * s, (qn >> 1) & 1));
      ++qn;
      if (!ok) break;
#pragma unroll 1
      for (int x = -2; x < steps; ++x) {
        const uint32_t b = nb + uint32_t(per * x + off), bk = b + uint32_t(2 * per);   // blocks of V and of K that are due
        const int st = int(b % NST), sk = int(bk % NST);
        const bool values = x >= 0, more = x + 2 < steps, fresh = values && x % kFlush == 0;
        const uint32_t pb = p_full + 16 * s + 8 * (un & 1);
        // polled together, so that their latencies overlap, then waited for one by one
        const bool r0 = !values || mbar_test(v_ready + 8 * st, (b / NST) & 1);
        const bool r1 = !values || mbar_test(pb, (un >> 1) & 1);
        const bool r2 = !more || mbar_test(k_full + 8 * sk, (bk / NST) & 1);
        if (values) {
          if (!all(r0 && r1 && !fresh) &&
              !all((r0 || wait(v_ready + 8 * st, (b / NST) & 1)) && (!fresh || wait(o_empty + 8 * s, (ost & 1) ^ 1)) &&
                   (r1 || wait(pb, (un >> 1) & 1)))) {
            ok = false;
            break;
          }
          tc_fence_after();
          if (fresh) ++ost;
          pv(st, fresh);
          umma_commit_e(v_empty + 8 * st);
          if (per == 2) umma_commit_e(v_empty + 8 * st);
        }
        if (more) {
          if (!all(r2) && !all(wait(k_full + 8 * sk, (bk / NST) & 1))) {
            ok = false;
            break;
          }
          tc_fence_after();
          qk(sk);
          umma_commit_e(k_empty + 8 * sk);
          if (per == 2) umma_commit_e(k_empty + 8 * sk);
        }
      }
      if (!ok) break;
      nb += uint32_t(cnt);
      umma_commit_e(o_full + 8 * s);
      if (lane == 0) mbar_arrive(o_full + 8 * s);   // orders the cleaners' findings before the stream's reads
    }
    if (!ok) misc[1] = 1;
  }
  } else if (warp < 12) {
    set_regs<C::REG_S, true>();
    // ------------------------------------------------------------------ softmax
    const int s = (warp - 4) >> 2, q4 = warp & 3, lr = q4 * 32 + lane;
    const uint32_t t0 = tmem + 256 * s + (uint32_t(q4 * 32) << 16), to = t0 + 128;
    float* fl = P.flush + (size_t(blockIdx.x) * 2 * ROWS + lr) * D;   // stream 0's; 1's ROWS * D on
    uint32_t un = 0, items = 0, turns = 0, nb = 0;   // units, items, exchanges; blocks of earlier items
    bool ok = true;
    auto all = [&](bool v) { return __all_sync(0xffffffffu, v); };
    if (threadIdx.x == 4 * 32) P.join[2 * r] = make_int4(0, 0, 0, 0);   // no item begins here and runs on
    // The thread's row of an item, and its queries on their way to the products: for every item, so that these are never
    // more than one ahead.
    struct Row {
      RowView v;
      size_t at;
      int hq;
      float qe;   // log2 of the factor of q's f16 values
      bool real;
    };
    auto row_of = [&](const Item& i) {
      const int row = (2 * i.m + (i.w == 2 ? s : 0)) * ROWS + lr, node = row / P.G;
      Row x;
      x.real = node < i.s.n;
      x.qe = 0.f;
      x.hq = i.h * P.G + (row - node * P.G);
      x.v = view_of(P, i.s, node);
      x.at = (size_t(i.s.row0 + (x.real ? node : 0)) * P.n_q + x.hq) * D;
      if (x.real && P.g != nullptr) {   // the gate's row, for the item's end
        l1_prefetch(P.g + x.at);
        if (D == 128) l1_prefetch(P.g + x.at + 64);
      }
      if (units_of(i, s) > 0) {
        uint8_t* qt = sm + C::Q0 + s * C::QB + lr * 128;
        auto put = [&](int e, const uint4& y) {
          *reinterpret_cast<uint4*>(qt + (e >> 3) * ROWS * 128 + (((e & 7) ^ (lr & 7)) << 4)) = y;
        };
        const uint16_t* src = P.q + x.at;
        if constexpr (!C::QUANT) {
#pragma unroll
          for (int e = 0; e < D / 8; ++e) put(e, x.real ? ld_stream(src + 8 * e) : make_uint4(0, 0, 0, 0));
        } else {
          // to f16 by a power of two that takes the largest magnitude to 2^15 .. 2^16
          auto get = [&](int e) { return x.real ? __ldg(reinterpret_cast<const uint4*>(src) + e) : make_uint4(0, 0, 0, 0); };
          unsigned mx = 0;
#pragma unroll 8
          for (int e = 0; e < D / 8; ++e) mx = __vmaxu2(mx, abs_max(get(e)));
          const unsigned top = max(mx & 0xFFFFu, mx >> 16);
          // by 2^up in two steps; rows with an infinity or a NaN as they are
          const int ex = top >= 0x7F80u ? 142 : max(1, int(top >> 7)), up = 142 - ex;
          const float u0 = __uint_as_float(unsigned(127 + up / 2) << 23), u1 = __uint_as_float(unsigned(127 + up - up / 2) << 23);
          x.qe = float(-up);
#pragma unroll 4
          for (int e = 0; e < D / 8; ++e) {
            float f[8];
            unpack8(get(e), f);
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = f[i] * u0 * u1;
            put(e, make_uint4(pack_f16x2(f[0], f[1]), pack_f16x2(f[2], f[3]), pack_f16x2(f[4], f[5]), pack_f16x2(f[6], f[7])));
          }
        }
        fence_proxy_async_smem();
      }
      arrive(q_full + 8 * s);
      return x;
    };
    Item it, nx;
    int c = c0;
    bool more = next_item(P, plan, c, c1, it);
    Row w;
    if (more) w = row_of(it);
    for (; ok && more; ++items) {
      const int units = units_of(it, s), tile = 2 * it.m + (it.w == 2 ? s : 0);
      const Row cur = w;
      const RowView& v = cur.v;
      const bool real = cur.real;
      const bool work = __any_sync(0xffffffffu, v.tree != 0);   // any row that sees keys
      const bool none = __any_sync(0xffffffffu, real && v.tree == 0);   // a row among them that sees nothing
      // Reference and sum of the weights (log2 units; it lags by up to kRescale); z: that of O, which over quantised pages
      // follows the weights times their value rows' powers of two
      float m = kNegInf, l = 0.f, z = kNegInf;
      bool flushed = false;
      const int stride = it.w == 2 ? 1 : 2, j_first = it.j0 + (it.w == 2 ? 0 : s);
      for (int k = 0; k < units; ++k, ++un) {
        const int j = j_first + k * stride;
        const uint32_t ts = t0 + 64 * (un & 1), bar = 16 * s + 8 * (un & 1);
        if (!all(wait(s_full + bar, (un >> 1) & 1))) { ok = false; break; }
        tc_fence_after();
        if (work) {
          const uint32_t ring = (nb + uint32_t(j - it.j0)) % kFac;
          [[maybe_unused]] const Factors* fa = reinterpret_cast<const Factors*>(sm + C::FAC) + ring;
          const unsigned slices = lives[ring];   // of keys that have a page
          const bool full = !none && slices == 15u && it.whole(j);
          const uint64_t bits = full ? ~uint64_t(0) : seen(v, it.s, (it.s.blk0 + j) * BK + 1, slices);
          float rf = P.sl2;   // factor of S (over quantised pages, of S times its key's) in log2 units of the weight
          if constexpr (C::QUANT) rf *= ex2(fmaxf(fminf(fa->top + cur.qe, 120.f), -120.f));
          constexpr int HALF = C::QUANT ? 16 : 32;   // words of P of 32 keys
          // 32 keys at a time, in a loop: the code of all roles has to stay in the instruction cache
#pragma unroll 1
          for (int x = 0; x < 2; ++x) {
            const uint32_t b32 = uint32_t(bits >> (32 * x));
            uint32_t sv[32], pk[HALF];
            tmem_ld32_nowait(ts + 32 * x, sv);
            tmem_wait_ld();
            float sum = 0.f;
            bool lag = m == kNegInf;
#pragma unroll 1
            for (int turn = 0; turn < 2; ++turn) {
              if (!full) {   // keys that the row does not see
#pragma unroll
                for (int e = 0; e < 32; ++e)
                  if (!((b32 >> e) & 1u)) sv[e] = __float_as_uint(kNegInf);
              }
              if (turn == 1 || __any_sync(0xffffffffu, lag)) {
                // The references are taken anew: O, the sum and the P of this block's first half are brought to them by whole
                // powers of two.
                float mt = kNegInf, zt = kNegInf;
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                  if constexpr (C::QUANT) {
                    const float y = __uint_as_float(sv[e]) * fa->k[32 * x + e] * rf;
                    mt = fmaxf(mt, y);
                    zt = fmaxf(zt, y + fa->v[32 * x + e]);
                  } else {
                    mt = fmaxf(mt, __uint_as_float(sv[e]));
                  }
                }
                if constexpr (C::QUANT) zt -= float(kBias);
                else zt = mt = mt * rf;
                // a row that another's first keys brought here is held to the same bound
                const float by = lag ? 0.f : float(kRescale), byz = lag ? 0.f : float(C::QUANT ? kRise : kRescale);
                const bool need = m != kNegInf && (mt > m + by || zt > z + byz);
                if (__any_sync(0xffffffffu, need)) {
                  // O holds the stream's earlier products: the last one has to be done
                  if (!all(k == 0 || wait(pv_done + 8 * s, (un - 1) & 1))) { ok = false; break; }
                  tc_fence_after();
                  // (z down to a whole power: the largest product is at least 2^kBias then, as at a row's first keys)
                  const float dm = need ? fmaxf(0.f, ceilf(mt - m)) : 0.f;
                  const float dz = need ? fmaxf(0.f, C::QUANT ? floorf(zt - z) : ceilf(zt - z)) : 0.f;
                  const float f = ex2(-dz);
                  if (k % kFlush != 0) {   // else O is not read again
#pragma unroll 1
                    for (int y = 0; y < D / 16; ++y) {
                      uint32_t o[16];
                      tmem_ld16(to + 16 * y, o);
#pragma unroll
                      for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                      tmem_st16(to + 16 * y, o);
                    }
                  }
                  if (x == 1) {
                    // in FP32 for f16, which has no 2^-25, while a P of up to 2^16 times it is still a number there
                    const uint32_t fb = pack_bf16x2(f, f);
#pragma unroll 1
                    for (int y = 0; y < HALF / 16; ++y) {
                      uint32_t o[16];
                      tmem_ld16(ts + 16 * y, o);
#pragma unroll
                      for (int e = 0; e < 16; ++e) {
                        if constexpr (C::QUANT) {
                          float p0, p1;
                          unpack_f16(o[e], p0, p1);
                          o[e] = pack_f16x2(p0 * f, p1 * f);
                        } else {
                          o[e] = mul_bf16x2(o[e], fb);
                        }
                      }
                      tmem_st16(ts + 16 * y, o);
                    }
                  }
                  tmem_wait_st();
                  if (flushed && dz > 0.f)
                    for (int y = 0; y < D; ++y) fl[s * ROWS * D + y] *= f;
                  l *= ex2(-dm);
                  m += dm;
                  z += dz;
                }
                if (m == kNegInf) {   // the row's first keys
                  m = mt;
                  z = zt;
                }
                turn = 1;
              }
              // P, and the sum of the weights. BF16: 2^(S c - m), its high parts and low parts. Quantised:
              // 2^(S c k - m + e - (z - m)) in f16, with the keys' factors k and e.
              const float nm = m == kNegInf ? 0.f : -m;
              const uint64_t c2 = f2(rf, rf), nm2 = f2(nm, nm);
              uint64_t ls[4] = {0, 0, 0, 0};
              unsigned most = 0;   // the largest of P in f16
              if constexpr (!C::QUANT) {
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
              } else {
                const float nz = z == kNegInf ? 0.f : -z;
                const uint64_t nz2 = f2(nz, nz);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                  const float4 kf = reinterpret_cast<const float4*>(fa->k + 32 * x)[e], ve = reinterpret_cast<const float4*>(fa->v + 32 * x)[e];
#pragma unroll
                  for (int i = 0; i < 2; ++i) {
                    const uint64_t sk = mul2(f2(__uint_as_float(sv[4 * e + 2 * i]), __uint_as_float(sv[4 * e + 2 * i + 1])),
                                             i ? f2(kf.z, kf.w) : f2(kf.x, kf.y));
                    float y0, y1, z0, z1;
                    f2_split(fma2(sk, c2, nm2), y0, y1);
                    f2_split(fma2(sk, c2, add2(i ? f2(ve.z, ve.w) : f2(ve.x, ve.y), nz2)), z0, z1);
                    ls[2 * (e & 1) + i] = add2(ls[2 * (e & 1) + i], f2(ex2(y0), ex2(y1)));
                    const uint32_t w = pack_f16x2(ex2(z0), ex2(z1));
                    pk[2 * e + i] = w;
                    most = __vmaxu2(most, w);
                  }
                }
              }
              float a0, a1, b0, b1;
              f2_split(add2(ls[0], ls[1]), a0, a1);
              f2_split(add2(ls[2], ls[3]), b0, b1);
              sum = (a0 + b0) + (a1 + b1);
              // The references stay while the weights sum to no more than 2^kRescale (quantised pages: while FP32 holds them
              // and P is no more than kMostP).
              lag = C::QUANT ? !(sum <= 0x1p60f) || max(most & 0xFFFFu, most >> 16) > kMostP : !(sum <= float(1 << kRescale));
              if (turn == 0) {
                if (!__any_sync(0xffffffffu, lag)) break;
                tmem_ld32_nowait(ts + 32 * x, sv);   // P may have taken its registers
                tmem_wait_ld();
              }
            }
            if (!ok) break;
            l += sum;
            if constexpr (C::QUANT) tmem_st16(ts + 16 * x, pk);
            else tmem_st32(ts + 32 * x, pk);
          }
          if (!ok) break;
          tmem_wait_st();
        }
        tc_fence_before();
        arrive(p_full + bar);
        if ((k + 1) % kFlush == 0 && k + 1 < units) {
          if (!all(wait(pv_done + 8 * s, un & 1))) { ok = false; ++un; break; }
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
          arrive(o_empty + 8 * s);
        }
      }
      if (!ok) break;
      // ---- the item's end. The next one's queries first, if the stream has blocks of both: only then has the warp of its
      // products taken this item's and will wait for P of the next, so that neither q_full nor o_full is lapped
      more = next_item(P, plan, c, c1, nx);
      const bool ahead = more && units > 0 && units_of(nx, s) > 0;
      if (ahead) w = row_of(nx);
      if (!all(wait(o_full + 8 * s, items & 1))) { ok = false; break; }
      tc_fence_after();
      // O's factors h^2 (in two steps, which alone may leave FP32's range) to the reference m of what is written
      float h0 = 1.f, h1 = 0.f;
      bool other = false;   // stream 1's share is added here
      // O is the row's if it sees anything: a row that sees nothing has the others' P . V, or no P at all. Neither a factor nor a sum
      // of zero says that: a stream that the other outweighs, or whose logits all are -inf, may hold a NaN or an infinity of a
      // value that the row reads, which reaches it all the same.
      const bool sees = v.tree != 0;
      auto half = [](float zs, float top) { return zs == kNegInf ? 0.f : ex2(0.5f * (zs - top)); };
      if (it.w == 1) {
        float4* xch = reinterpret_cast<float4*>(sm + C::XCH);
        if (s == 1) {
          // stream 0 writes for both
          if (!all(wait(x_empty, (turns & 1) ^ 1))) { ok = false; break; }
          xch[lr] = make_float4(m, z, l, 0.f);
          arrive(x_full);
          ++turns;
          if (more && !ahead) w = row_of(nx);
          nb += uint32_t(it.j1 - it.j0);
          it = nx;
          continue;
        }
        if (!all(wait(x_full, turns & 1))) { ok = false; break; }
        const float4 y = xch[lr];
        arrive(x_empty);
        ++turns;
        other = units_of(it, 1) > 0;
        const float top = fmaxf(m, y.x);
        if (l != l || y.z != y.z || top == INFINITY) {   // a logit that is NaN (its stream's m may be -inf) or +inf
          l = h0 = h1 = __uint_as_float(0x7FFFFFFFu);
        } else if (top != kNegInf) {
          h0 = half(z, top);
          h1 = half(y.y, top);
          l = (l == 0.f ? 0.f : ex2(m - top) * l) + (y.z == 0.f ? 0.f : ex2(y.x - top) * y.z);
        }
        m = top;
      } else if (C::QUANT && m != kNegInf) {
        h0 = half(z, m);
      }
      const bool other_flushed = other && units_of(it, 1) > kFlush;
      const bool odd = misc[2] != 0;
      const float inv = l == 0.f ? 0.f : 1.f / l;
      const int slot = it.j0 > 0 ? 0 : 1;
      const size_t part = ((size_t(r) * 2 + slot) * 2 + (tile & 1)) * ROWS + lr;
      const bool gated = P.g != nullptr && !it.split;
      const bool gates = gated && real && l != 0.f;   // a row that sees nothing is zero, whatever its gate holds
      const float bias = gates ? bf2f(P.gate_bias[cur.hq]) : 0.f;
#pragma unroll 1
      for (int x = 0; x < D / 32; ++x) {
        uint4 g[4];
        if (gated)
#pragma unroll
          for (int e = 0; e < 4; ++e) g[e] = gates ? reinterpret_cast<const uint4*>(P.g + cur.at + 32 * x)[e] : make_uint4(0, 0, 0, 0);
        __syncwarp();
        uint32_t o[32];
        tmem_ld32_nowait(to + 32 * x, o);
        tmem_wait_ld();
        float a[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) a[e] = sees ? __uint_as_float(o[e]) * h0 * h0 : 0.f;
        if (flushed && sees)
#pragma unroll
          for (int e = 0; e < 32; ++e) a[e] += fl[s * ROWS * D + 32 * x + e] * h0 * h0;
        if (other) {
          tmem_ld32_nowait(to + 256 + 32 * x, o);
          tmem_wait_ld();
          if (sees)
#pragma unroll
            for (int e = 0; e < 32; ++e) a[e] += __uint_as_float(o[e]) * h1 * h1;
          if (other_flushed && sees)
#pragma unroll
            for (int e = 0; e < 32; ++e) a[e] += fl[ROWS * D + 32 * x + e] * h1 * h1;
        }
        if (real) {
          if (odd) {   // in an array of its own: the call takes its address
            float y[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) y[e] = a[e];
            add_no_numbers<FMT, D>(P, it, v, 32 * x, y);
#pragma unroll
            for (int e = 0; e < 32; ++e) a[e] = y[e];
          }
          if (it.split) {
            float4* y = reinterpret_cast<float4*>(P.part_acc + part * D + 32 * x);
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = make_float4(a[4 * e], a[4 * e + 1], a[4 * e + 2], a[4 * e + 3]);
          } else {
            [[maybe_unused]] uint4* y = reinterpret_cast<uint4*>(P.og + cur.at + 32 * x);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float* z = a + 8 * e;
              const uint2 u0 = finish4(gated, make_float4(z[0] * inv, z[1] * inv, z[2] * inv, z[3] * inv), make_uint2(g[e].x, g[e].y), bias);
              const uint2 u1 = finish4(gated, make_float4(z[4] * inv, z[5] * inv, z[6] * inv, z[7] * inv), make_uint2(g[e].z, g[e].w), bias);
              g[e] = make_uint4(u0.x, u0.y, u1.x, u1.y);
              if constexpr (!C::QUANT) y[e] = g[e];
            }
          }
        }
        if (C::QUANT && !it.split) {
          // Two lanes write one row's 32 bytes at a time, then the other's: whole sectors, half the lines of a store (32
          // sequences over FP8 274 -> 261 us; over BF16, whose warps wait for keys at the end, 217 -> 219)
          const bool odd_lane = lane & 1;
          auto swap = [](const uint4& v) {
            return make_uint4(__shfl_xor_sync(0xffffffffu, v.x, 1), __shfl_xor_sync(0xffffffffu, v.y, 1),
                              __shfl_xor_sync(0xffffffffu, v.z, 1), __shfl_xor_sync(0xffffffffu, v.w, 1));
          };
          const uint4 s0 = swap(odd_lane ? g[0] : g[1]), s1 = swap(odd_lane ? g[2] : g[3]);
          const size_t mate = __shfl_xor_sync(0xffffffffu, static_cast<unsigned long long>(cur.at), 1);
          const bool mate_real = __shfl_xor_sync(0xffffffffu, int(real), 1) != 0;
          uint4* own = reinterpret_cast<uint4*>(P.og + cur.at + 32 * x) + (odd_lane ? 1 : 0);
          uint4* its = reinterpret_cast<uint4*>(P.og + mate + 32 * x) + (odd_lane ? 1 : 0);
          uint4 *even = odd_lane ? its : own, *odd_row = odd_lane ? own : its;
          if (odd_lane ? mate_real : real) {
            even[0] = odd_lane ? s0 : g[0];
            even[2] = odd_lane ? s1 : g[2];
          }
          if (odd_lane ? real : mate_real) {
            odd_row[0] = odd_lane ? g[1] : s0;
            odd_row[2] = odd_lane ? g[3] : s1;
          }
        }
        __syncwarp();
      }
      if (it.split && real) P.part_ml[part] = make_float2(m, l);
      tc_fence_before();
      if (units > 0) arrive(o_empty + 8 * s);
      if (other) arrive(o_empty + 8);
      if (it.split && it.j0 == 0 && threadIdx.x == 4 * 32) {   // one does
        P.join[2 * r] = make_int4(it.h, it.m, range_of(it.f + it.w * (it.s.nb - 1), total, R) - r + 1, it.w);
        *reinterpret_cast<int2*>(P.join + 2 * r + 1) = make_int2(it.s.row0, it.s.n);
      }
      if (more && !ahead) w = row_of(nx);
      nb += uint32_t(it.j1 - it.j0);
      it = nx;
    }
    if (!ok) misc[1] = 1;
  } else {
    set_regs<C::REG_C, false>();
    // ------------------------------------------------------------------ rows that attend to nothing
    auto zero = [&](int a, int b) {   // rows a..b-1, this CTA's of them
      for (int t = max(a, 0) + r; t < min(b, P.T); t += int(gridDim.x))
        for (int x = threadIdx.x - 12 * 32; x < P.n_q * (D / 8); x += C::THREADS - 12 * 32)
          reinterpret_cast<uint4*>(P.og + size_t(t) * P.n_q * D)[x] = make_uint4(0, 0, 0, 0);
    };
    if (P.head_rows) zero(0, P.row_start[0]);
    if (P.tail_rows) zero(P.row_start[P.N], P.T);
    for (int i = 0; i < P.N; ++i)
      if (cum[i + 1] == cum[i]) zero(P.row_start[i], P.row_start[i + 1]);
    if constexpr (C::QUANT) {
      // ---------------------------------------------------------------- codes to f16 tiles
      const int kv = (warp - 12) >> 2, tid = threadIdx.x - (12 + 4 * kv) * 32;   // four warps for K, four for V
      const uint32_t full = kv ? v_full : k_full, empty = kv ? v_empty : k_empty;
      uint32_t nb = 0;
      bool ok = true, odd = false;
      auto all = [&](bool v) { return __all_sync(0xffffffffu, v); };
      Item it;
      for (int c = c0; ok && next_item(P, plan, c, c1, it);) {
        for (int j = it.j0; j < it.j1; ++j, ++nb) {
          const int rs = int(nb % (NRAW ? NRAW : 1)), st = int(nb % NST);
          if (!all(wait(r_full + 8 * (kv * NRAW + rs), (nb / (NRAW ? NRAW : 1)) & 1) &&
                   wait(empty + 8 * st, ((nb / NST) & 1) ^ 1))) {
            ok = false;
            break;
          }
          const unsigned live = masks[8 * kv + rs];
          const bool whole = live == 15u && it.whole(j);
          const int kb = (it.s.blk0 + j) * BK + 1;
          const uint8_t* raw = sm + C::R0 + (kv * NRAW + rs) * C::RAW;
          uint8_t* tile = sm + (kv ? C::V0 : C::K0) + st * C::TILE;
          const uint8_t* rows = raw + C::RAWB + C::RBS;
          auto inside = [&](int row) {   // one of the item's keys, in a page
            return kb + row >= it.s.lo && kb + row <= it.s.base + it.s.n && ((live >> (row >> 4)) & 1u);
          };
          const unsigned b0 = rows[lane], b1 = rows[lane + 32];
          if (kv == 0) {
            // the keys' factors: their powers of two relative to the largest, and those of their values
            unsigned top = b0 != 255 && (whole || inside(lane)) ? b0 : 0;
            if (b1 != 255 && (whole || inside(lane + 32))) top = max(top, b1);
            top = __reduce_max_sync(0xffffffffu, top);
            Factors* fa = reinterpret_cast<Factors*>(sm + C::FAC) + nb % kFac;
            const int row = 16 * (warp - 12) + (lane & 15);
            if (lane < 16) {
              // never zero: hidden keys' logits are -inf (a row that is no numbers brings its NaN in its codes)
              fa->k[row] = __uint_as_float(unsigned(min(127, max(1, int(rows[row]) - int(top) + 127))) << 23);
            } else {
              const unsigned bv = rows[BK + row];
              fa->v[row] = bv == 255 ? 0.f : float(int(bv) - 127);
            }
            if (row == 0 && lane == 0) fa->top = float(int(top) - 127);
          }
          // no row that needs a look: no NaN, and of values none that is not the item's
          const bool plain = (kv == 0 || whole) && !__any_sync(0xffffffffu, b0 == 255 || b1 == 255);
          // sixteen elements at a time; of the upper half's rows in pairs the other way round: eight lanes then store to all banks
          constexpr int STEP = 128 / (D / 16);   // rows of a turn, a multiple of 8
          const int gr = tid % (D / 16), row0 = (tid / (D / 16)) ^ (gr >> 2), ch = (2 * gr) & 7;
          const uint8_t* from = raw + row0 * C::ROWB + gr * (C::ROWB / (D / 16));
          uint8_t* to = tile + (gr >> 2) * BK * 128 + row0 * 128;
          uint8_t *to0 = to + ((ch ^ (row0 & 7)) << 4), *to1 = to + (((ch + 1) ^ (row0 & 7)) << 4);
#pragma unroll
          for (int i = 0; i < BK / STEP; ++i) {
            const int row = row0 + i * STEP;
            uint32_t w[8];
            if constexpr (FMT == kFmtFP8) {
              const uint4 y = *reinterpret_cast<const uint4*>(from + i * STEP * C::ROWB);
              e4m3x4_f16(y.x, w[0], w[1]);
              e4m3x4_f16(y.y, w[2], w[3]);
              e4m3x4_f16(y.z, w[4], w[5]);
              e4m3x4_f16(y.w, w[6], w[7]);
            } else {
              const uint2 y = *reinterpret_cast<const uint2*>(from + i * STEP * C::ROWB);
              const uint32_t unit = e4m3x2_f16x2(raw[C::RAWB + row * (D / 16) + gr] * 0x101u);
              e2m1x8_f16(y.x, w);
              e2m1x8_f16(y.y, w + 4);
#pragma unroll
              for (int e = 0; e < 8; ++e) w[e] = mul_f16x2(w[e], unit);
            }
            if (!plain) {
              // no numbers: NaN, but for values of blocks that not all rows see: zero, as for keys that are not the item's
              const bool none = rows[row] == 255, out = kv == 1 && !whole && !inside(row);
              if (none || out) {
                const bool zero = kv == 1 && !whole;
                if (zero && !out) odd = true;
#pragma unroll
                for (int e = 0; e < 8; ++e) w[e] = zero ? 0u : 0x7FFF7FFFu;
              }
            }
            *reinterpret_cast<uint4*>(to0 + i * STEP * 128) = make_uint4(w[0], w[1], w[2], w[3]);
            *reinterpret_cast<uint4*>(to1 + i * STEP * 128) = make_uint4(w[4], w[5], w[6], w[7]);
          }
          if (odd) misc[2] = 1;
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(full + 8 * st);
            mbar_arrive(r_empty + 8 * (kv * NRAW + rs));
          }
        }
      }
      if (!ok) misc[1] = 1;
    }
    // ---- blocks that not all rows see in full: rows of V outside the item's keys, elements that are no numbers
    if constexpr (!C::QUANT) {
      uint32_t nb = 0;
      bool ok = true;
      Item it;
      for (int c = c0; ok && next_item(P, plan, c, c1, it);) {
        for (int j = it.j0; j < it.j1; ++j, ++nb) {
          const int st = int(nb % NST), kb = (it.s.blk0 + j) * BK + 1;
          if (!__all_sync(0xffffffffu, wait(v_full + 8 * st, (nb / NST) & 1))) { ok = false; break; }
          const unsigned live = masks[8 + st];
          if (live == 15u && it.whole(j)) {
            __syncwarp();
            if (lane == 0) mbar_arrive(v_clean + 8 * st);
            continue;
          }
          bool odd = false;
          uint4* tile = reinterpret_cast<uint4*>(sm + C::V0 + st * C::TILE);
#pragma unroll 4
          for (int x = threadIdx.x - 12 * 32; x < C::TILE / 16; x += 128) {
            const int row = (x >> 3) & (BK - 1), key = kb + row;
            uint4 w = tile[x];
            const bool in = key >= it.s.lo && key <= it.s.base + it.s.n && ((live >> (row >> 4)) & 1u);
            const bool no = no_number(w.x) || no_number(w.y) || no_number(w.z) || no_number(w.w);
            if (!in) tile[x] = make_uint4(0, 0, 0, 0);
            else if (no) {
              odd = true;
              uint32_t* y = reinterpret_cast<uint32_t*>(&w);
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                if ((y[e] & 0x7F80u) == 0x7F80u) y[e] &= 0xFFFF0000u;
                if ((y[e] & 0x7F800000u) == 0x7F800000u) y[e] &= 0x0000FFFFu;
              }
              tile[x] = w;
            }
          }
          if (odd) misc[2] = 1;
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(v_clean + 8 * st);
        }
      }
      if (!ok) misc[1] = 1;
    }
  }
  tc_fence_before();
  __syncthreads();
  pdl_trigger();   // not earlier: the join and what follows would run beside the key stream
  if (threadIdx.x == 0) P.join[2 * r + 1].z = int(*status | (misc[1] ? BEAM_DEV_TIMEOUT : 0u));
  if (warp == 1)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
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
  return e != cudaSuccess ? e : join(p, grid, st);
}

constexpr size_t kParts = size_t(kGrid) * 2 * 2 * ROWS;   // rows of partial results

}  // namespace
}  // namespace tree
}  // namespace paged
}  // namespace beam

extern "C" size_t beam_paged_tree_workspace_bytes(const beam_layer_cfg* cfg, int T) {
  using namespace beam;
  using namespace beam::paged;
  using namespace beam::paged::tree;
  if (cfg == nullptr || T <= 0 || cfg->n_q <= 0 || cfg->head_dim <= 0) return 256;
  const size_t D = cfg->head_dim;
  return align_up(kParts * D * 4, 256) + align_up(kParts * 8, 256) + align_up(2 * kGrid * sizeof(int4), 256) +
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
  using namespace beam::paged::tree;
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
  if ((nb + kItemBF16) * ((kNodes * G + ROWS - 1) / ROWS) * slice * cfg->n_kv > 1 << 30 || cfg->n_kv > 65535) return BEAM_ERR_UNSUPPORTED;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  Carver cv{static_cast<char*>(ws), ws_bytes};
  Params p{};
  p.part_acc = cv.take<float>(kParts * D);
  p.part_ml = cv.take<float2>(kParts);
  p.join = cv.take<int4>(2 * kGrid);
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
  p.item = cache->dtype == kFmtBF16 ? kItemBF16 : kItemQuant;
  p.least = p.item + 4;
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
