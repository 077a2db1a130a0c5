// Decode attention over the paged cache: one new token per row, the row's keys split over the
// SMs and joined.
//
//   o[h] = sum_i e^(x_i - m) v_i / sum_i e^(x_i - m),  x_i = q[h].k_i / sqrt(D),  m = max x_i
//
// over the row's keys i, computed in one pass with the running (m, sum, O) of a softmax, which
// partial results of disjoint key ranges join by.
//
// What bounds it (device time in a graph; HBM 6784.5 GB/s as a copy): the bytes of the keys and
// values over long contexts: 128 sequences of 17 to 16,385 tokens in FP8 321 to 326 us, 98% of the
// copy rate; one of 100,001 in BF16 66.2 us, 91%, the rest being the start (1.6 us of plan, 0.9 us
// of page lookups) and the join (3 us). Over an NVFP4 cache the arithmetic: 4 sequences of 60,000 to
// 100,001 tokens 82.3 us, 67%: about 360 warp instructions for 16 keys of one KV head, 128 of them
// the conversions and the scaling of the codes, which keep the issue slots 66% and the integer
// pipe 58% busy.
//
// Split. A (row, KV head) pair's keys are cut into blocks of BK; the blocks of all pairs, laid
// end to end, are cut into equal ranges, two or three per CTA (one CTA per SM). The ranges are
// computed on the device from the rows' own lengths, so a batch of very unequal sequences still
// gives every SM the same bytes. A pair that one range holds whole is finished there; the partials
// of a split pair go to the workspace and a second small kernel joins them. Where pairs are short
// (the rule and its measurements stand at the launch) a CTA takes whole pairs, its groups share
// them, and it joins them itself.
//
// A CTA has two or three groups, each with its own range and ring of stages:
//  - a producer warp reads the page table (one lane per page of a block, a block ahead) and issues
//    a TMA load per page for K and V, bulk copies of the rows' scales and, with a pair's first
//    block, of its q rows;
//  - four consumer warps take one or two slices of 16 keys of every block. More warps with fewer
//    registers were slower (16 of 96 registers: FP8 370 us against 333, with spills);
//  - with two groups a finisher warp joins the consumers' partials of a pair while they go on
//    (330 -> 323 us; windows of 512 keys 37.3 -> 35.2). It takes four or eight heads at a time, without
//    a branch or a division between them: 106 sequences of 3 tokens, 8 KV heads of 16 heads each,
//    27.6 -> 17.1 us, of 5 each 12.4 -> 11.0. NVFP4, bound by arithmetic, has
//    a third group instead (4 sequences of 60,000 to 100,001 tokens 88.5 -> 82.4 us; head dim 64, 39
//    of 20,236, 160 -> 136), but for 9 to 16 heads at head dim 64 (199 -> 207).
//
// Tiles are transposed, so that the query heads of a KV group are the 8-wide N side of mma.sync
// m16n8k16 (two N tiles for 9 to 16 heads):
//   S^T[16 keys x 8 heads] = K[16 x D] . Q^T,   O^T[D x 8 heads] += V^T[D x 16 keys] . P^T
// The running max lags by up to 2^8: a vote decides whether it moves at all, so the common block
// has no shuffle (439 -> 393 us with the two points below).
//
// Roundings. Logits, sums and O are FP32. Over a BF16 cache P is split into a high and a low bf16
// half (16 bits). Over FP8 and NVFP4 the codes become f16 in registers, exactly (e2m1 times its
// e4m3 block scale has 6 significant bits), and P is rounded once to f16: its half step, 2^-11 of a
// weight, is far below the cache's own (2^-4 and 2^-2), and the low half cost a third of the
// arithmetic. The rows' powers of two never enter an f16 value: K's multiplies the FP32 logits x;
// V's (2^e) goes into P = 2^(x + e - Z + 7), where Z is a second running max, that of x + e. So P's
// largest values lie near the top of f16 whatever the scales are, a row of large values that
// weighs nothing takes no bits from the others, and what P loses below f16's smallest step is at
// most 2^-32 of the largest weighted scale for each key. (Z costs NVFP4 2 to 5%, 4 sequences of
// 60,000 to 100,001 tokens 80.4 -> 82.3 us; over FP8 the stream hides it, but for 16 heads, 39 of
// 20,236 276 -> 290.) Against 64 bits the outputs over quantised caches are 0.6% further off than
// with FP32 weights, the rest being their rounding to bf16. q is scaled by a power of two per head
// to the top of f16: its bf16 values stay exact down to 2^-31 of the head's largest magnitude, and
// smaller ones are off by at most 2^-39 of it. The d axis is permuted the same way in q
// and K, and undone on the output for V, so that a thread's codes are contiguous bytes.
//
// Every mbarrier wait is bounded: on expiry the CTA records BEAM_DEV_TIMEOUT, stops issuing, lets
// its issued copies land and finishes without valid results.
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

constexpr float kNegInf = -INFINITY;
constexpr float kLowest = -3e38f;   // a running max that has seen nothing: finite, so differences are
constexpr float kRescale = 8.f;     // log2 units by which the running max may lag
constexpr int kMaxGrid = 152;       // CTAs at most
constexpr int kMaxGroups = 3;      // groups of a CTA at most
constexpr int kMaxParts = kMaxGroups * kMaxGrid;   // ranges, and so parts of one pair, at most
constexpr int kMaxT = 1024;         // rows of one launch
constexpr int kBias = 7;            // P <= 2^kRescale, times 2^7: below 65504

template <int FMT, int D_, int NT_>
struct Cfg {
  static constexpr int D = D_, NT = NT_, HEADS = 8 * NT;
  static constexpr int ROWB = row_bytes(FMT, D);
  static constexpr int PLANES = ROWB > 128 ? 2 : 1;   // 128-byte columns of a row
  // A group is WPG consumer warps, SPW slices of 16 keys of a block each, with its own range of
  // blocks and ring of stages: what one group spends on waits and on a pair's end, the other's
  // arithmetic covers
  static constexpr bool HEAVY = FMT == kFmtBF16 ? D == 128 : NT == 2 && D == 128;   // one slice fills it
  static constexpr int GROUPS = FMT == kFmtNVFP4 && (D == 128 || NT == 1) ? 3 : 2;
  // over quantised caches q's fragments lie in shared memory, not in 8 to 32 registers: 39 sequences
  // of 20,236 tokens, 8 KV heads of 16 heads: FP8 313 -> 276 us, NVFP4 346 (with two groups) -> 292;
  // of 8 heads, NVFP4 184 -> 180, 64-wide 136 -> 132 (before the second running max: now 290, 294, 185, 135)
  static constexpr bool QSM = FMT != kFmtBF16;
  static constexpr int WPG = 4, SPW = HEAVY ? 1 : 2;
  // log2 units by which a reference may lag: P <= 2^(kRescale + kBias) in f16, below 65504
  static constexpr float LAG = FMT == kFmtBF16 ? kRescale : kRescale + kBias;
  static constexpr int NCW = WPG * GROUPS, NCT = WPG * 32;   // consumer warps, threads of a group
  // four more warps: a producer for each group, and with two groups a finisher for each, which
  // joins the consumer warps' partials of a pair while they take the next one
  static constexpr bool FIN = GROUPS == 2;
  static constexpr int THREADS = (NCW + 4) * 32;
  static constexpr int SLICES = WPG * SPW, BK = 16 * SLICES;
  static constexpr int KB = BK * ROWB;
  static constexpr int BSB = FMT == kFmtNVFP4 ? 2 * BK * (D / 16) : 0;
  static constexpr int RSB = FMT != kFmtBF16 ? 2 * BK : 0;
  static constexpr int QB = HEADS * D * 2;
  static constexpr int OBS = 2 * KB, ORS = OBS + BSB, OQ = ORS + RSB;   // offsets in a stage
  static constexpr int STAGE = (OQ + QB + 1023) / 1024 * 1024;
  static constexpr int OLD = D + 4;   // row stride of the combine buffer (floats)
  static constexpr int OWB = WPG * HEADS * OLD * 4, MLB = WPG * HEADS * 2 * 4;   // of one group
  // with a finisher no barrier lies between a pair's last read of them and the next pair's write
  static constexpr int QBUFS = FIN ? 2 : 1, QFB = QSM ? GROUPS * QBUFS * QB : 0;
  static constexpr int NOW = GROUPS < 3 && 4 * STAGE + 2 * GROUPS * (OWB + MLB) <= 216 * 1024 ? 2 : 1;
  static constexpr int FIT = (216 * 1024 - NOW * GROUPS * (OWB + MLB) - QFB) / STAGE;
  static constexpr int NSTG = FIT / GROUPS > 4 ? 4 : FIT / GROUPS, NST = NSTG * GROUPS;   // stages of a group
  static constexpr int OW = NST * STAGE;                  // [GROUPS][NOW][WPG][HEADS][OLD]: O partials
  static constexpr int MLW = OW + GROUPS * NOW * OWB;     // [GROUPS][NOW][WPG][HEADS][2]: (m, l)
  static constexpr int QF = MLW + GROUPS * NOW * MLB;     // [GROUPS][QBUFS][NT][D / 16][32 lanes] 8 bytes
  static constexpr int CUM = QF + QFB;    // [kMaxT + 1] block prefix
  static constexpr int POS = CUM + (kMaxT + 1) * 4;       // [kMaxT] positions
  static constexpr int MISC = (POS + kMaxT * 4 + 15) / 16 * 16;   // -, abort, -, -; masks
  static constexpr int JOIN = MISC + 16 + 12 * 4;         // [GROUPS] pairs that begin in a group's range
  static constexpr int BAR = JOIN + 3 * 16;
  static constexpr int BYTES = BAR + 2 * NST * 8 + 1024;  // + alignment slack
  static constexpr int ITEMS = (HEADS * (D / 4) + NCT - 1) / NCT;   // 4 outputs that a thread finishes
  static_assert(GROUPS <= kMaxGroups, "the workspace is sized for kMaxGroups ranges a CTA");
  static_assert(BYTES <= 227 * 1024, "stage ring exceeds shared memory");
  static_assert(NSTG >= 2 && NST <= 12, "one mask word per stage");
};

struct Params {
  const uint16_t* q;
  const uint16_t* g;
  const uint16_t* gate_bias;
  const int32_t* seq_id;
  const int32_t* pos;
  uint16_t* og;
  float* part_acc;   // [ranges][2][HEADS][D]: a range's partials of its first and its last pair
  float* part_ml;    // [ranges][2][HEADS][2]
  int4* join;        // [ranges]: (row, KV head, parts, slot of the first part); parts 0: nothing
  beam_paged_kv c;
  int T, n_q, n_kv, G, max_pos, shift, whole, ranges;
  float sl2;
};

// Row t's keys are positions [lo, p], in blocks blk0 .. blk0 + nb - 1 (block b: BK * b + 1 ..).
struct Row {
  int p, s, lo, blk0, nb;
  unsigned bad;
};
template <int BK>
__device__ __forceinline__ Row row_of(const Params& P, int t) {
  Row r;
  r.p = P.pos[t];
  r.s = P.seq_id[t];
  r.bad = 0;
  if (r.p < 0 || r.p > P.max_pos || (r.p > 0 && ((r.p - 1) >> P.shift) >= P.c.table_stride))
    r.bad = BEAM_DEV_BAD_POSITION;
  else if (r.p > 0 && (r.s < 0 || r.s >= P.c.num_seqs))
    r.bad = BEAM_DEV_BAD_SEQ;
  r.lo = P.c.window > 0 ? max(1, r.p - P.c.window + 1) : 1;
  r.blk0 = (r.lo - 1) / BK;
  r.nb = r.bad || r.p == 0 ? 0 : (r.p - 1) / BK - r.blk0 + 1;
  return r;
}

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t movtrans(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t r;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(sel));
  return r;
}
template <int W>
__device__ __forceinline__ void lds(uint32_t a, uint32_t* v) {
  if constexpr (W == 4)
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(a));
  else if constexpr (W == 2)
    asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(v[0]), "=r"(v[1]) : "r"(a));
  else
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v[0]) : "r"(a));
}
__device__ __forceinline__ uint32_t lds_u8(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds_u16(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Loads that stay where they are written, ahead of their use.
__device__ __forceinline__ uint2 ld_ahead(const uint16_t* p) {
  uint2 v;
  asm volatile("ld.global.v2.b32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}
__device__ __forceinline__ uint16_t ld_ahead16(const uint16_t* p) {
  uint16_t v;
  asm volatile("ld.global.u16 %0, [%1];" : "=h"(v) : "l"(p));
  return v;
}
template <int NTHREADS>
__device__ __forceinline__ void consumer_bar(int group) {
  asm volatile("bar.sync %0, %1;" ::"r"(1 + group * 5), "n"(NTHREADS) : "memory");
}
// Hand-over of combine buffer `buf` between a group's consumers and its finisher: full (which = 0)
// or empty (1). WAIT: the side that waits; the other only arrives.
template <int NTHREADS, bool WAIT>
__device__ __forceinline__ void pair_bar(int group, int which, int buf) {
  const int id = 2 + group * 5 + which * 2 + buf;
  __syncwarp();
  if (WAIT) asm volatile("bar.sync %0, %1;" ::"r"(id), "n"(NTHREADS) : "memory");
  else asm volatile("bar.arrive %0, %1;" ::"r"(id), "n"(NTHREADS) : "memory");
}
// Untiled bulk copy (16-byte aligned, a multiple of 16 bytes).
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes,
                                          uint32_t mbar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
          "r"(dst), "l"(src), "r"(bytes), "r"(mbar)
      : "memory");
}
// Byte o of a region of 128-byte rows under the 128-byte TMA swizzle.
__device__ __forceinline__ uint32_t sw(uint32_t o) { return o ^ (((o >> 7) & 7u) << 4); }

// Place of element d in a row of the combine buffer. Over a quantised cache lane g writes
// neighbours of the range [g D/8, (g + 1) D/8): exchanging groups of four spreads the eight lanes
// over all banks.
template <int FMT, int D>
__device__ __forceinline__ int spread(int d) {
  if (FMT == kFmtBF16) return d;
  return D == 128 ? d ^ (((d >> 4) & 7) << 2) : d ^ (((d >> 5) & 1) << 2);
}

// Reciprocals to one unit in FP32's last place, 2^-16 of the rounding to BF16 that follows; a
// division's slow path would end the overlap of a thread's outputs.
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Factor of a row's outputs whose weights sum to L (0 or at least a half).
__device__ __forceinline__ float inverse(float L) { return L == 0.f ? 0.f : rcp(L); }
__device__ __forceinline__ void gate4(float4& o, uint2 g, float bias) {
  o.x *= rcp(1.f + __expf(-(bf_lo(g.x) + bias)));
  o.y *= rcp(1.f + __expf(-(bf_hi(g.x) + bias)));
  o.z *= rcp(1.f + __expf(-(bf_lo(g.y) + bias)));
  o.w *= rcp(1.f + __expf(-(bf_hi(g.y) + bias)));
}
__device__ __forceinline__ uint2 pack4(float4 o) {
  return make_uint2(pack_bf16x2(o.x, o.y), pack_bf16x2(o.z, o.w));
}
// Four neighbouring outputs: normalised, gated, rounded once.
__device__ __forceinline__ void finish4(bool gated, float4 O, float L, uint2 g, float bias,
                                        uint16_t* out) {
  const float inv = inverse(L);
  float4 o = make_float4(O.x * inv, O.y * inv, O.z * inv, O.w * inv);
  if (gated) gate4(o, g, bias);
  *reinterpret_cast<uint2*>(out) = pack4(o);
}

// The state of one warp over its keys of a pair.
template <class C>
struct WarpState {
  float m[C::NT][2], l[C::NT][2];   // running max (lags by up to kRescale) and sum, heads 2c, 2c+1
  // quantised caches: acc holds sums of 2^x v relative to 2^z, z = the running max (lagging in the
  // same manner) of x + e, e the value rows' exponents, less kBias
  float z[C::NT][2];
  float acc[C::NT][C::D / 16][4];
};

// Offsets in a stage that a lane uses for every block.
template <int FMT, class C>
struct Lane {
  uint32_t k[2], v[4];   // codes of its keys: K rows g, g + 8; V rows 2c, 2c + 1, 2c + 8, 2c + 9
  int rs, pse;           // scale index of the slice's first key, and from K's scales to V's
};
template <int FMT, class C>
__device__ __forceinline__ Lane<FMT, C> lane_of(int slice, int pse) {
  const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  Lane<FMT, C> r;
  if constexpr (FMT == kFmtBF16) {
    // ldmatrix rows; the k step (or m tile) e XORs e << 5 into the chunk, 128-byte swizzle
    const int rk = 16 * slice + ((lane >> 3) & 1) * 8 + (lane & 7), ck = (lane >> 4) & 1;
    const int rv = 16 * slice + ((lane >> 4) & 1) * 8 + (lane & 7), cv = (lane >> 3) & 1;
    r.k[0] = uint32_t(rk * 128 + ((ck ^ (lane & 7)) << 4));
    r.v[0] = uint32_t(rv * 128 + ((cv ^ (lane & 7)) << 4)) + C::KB;
  } else {
#pragma unroll
    for (int e = 0; e < 2; ++e)
      r.k[e] = sw((16 * slice + g + 8 * e) * C::ROWB + c * (C::ROWB / 4));
#pragma unroll
    for (int e = 0; e < 4; ++e)
      r.v[e] = C::KB + sw((16 * slice + 2 * c + (e & 1) + 8 * (e >> 1)) * C::ROWB + g * (C::ROWB / 8));
  }
  // scales lie as [page][K | V][key of the page]; a slice lies in one page
  const int key = 16 * slice;
  r.rs = (key / pse) * 2 * pse + (key & (pse - 1));
  r.pse = pse;
  return r;
}

// One warp's slices (SPW of 16 keys, WPG slices apart) of a staged block. kb: the stage; kbase:
// position of the first slice's first key; live: bit i, slice i has keys; the row's keys are
// positions [lo, p]. q: fragments qb (BF16) or at qf. qs: FP32 factor of the logits per accumulator column.
template <int FMT, class C>
__device__ __forceinline__ void warp_block(uint32_t kb, const Lane<FMT, C> (&ln)[C::SPW],
                                           const uint32_t (&qb)[C::NT][C::D / 16][2], uint32_t qf,
                                           const float (&qs)[C::NT][2], int kbase, unsigned live,
                                           int lo, int p, WarpState<C>& S) {
  constexpr int D = C::D, NT = C::NT, KK = D / 16, SPW = C::SPW, GAP = 16 * C::WPG;
  const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const bool full = live == (1u << SPW) - 1 && kbase >= lo && kbase + (SPW - 1) * GAP + 15 <= p;
  auto valid = [&](int i, int key) {
    const int pos = kbase + i * GAP + key;
    return ((live >> i) & 1u) && pos >= lo && pos <= p;
  };
  float sx[SPW][NT][4];
  // ---- S^T = K . Q^T. Fragment: [0] (key g, head 2c), [1] (g, 2c+1), [2], [3] key g + 8
#pragma unroll
  for (int i = 0; i < SPW; ++i) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) sx[i][n][e] = 0.f;
    if constexpr (FMT == kFmtBF16) {
#pragma unroll
      for (int kk = 0; kk < KK; ++kk) {
        uint32_t a[4];
        ldsm_x4(kb + (kk >> 2) * (C::KB / C::PLANES) + (ln[i].k[0] ^ uint32_t((kk & 3) << 5)), a[0], a[1], a[2], a[3]);
#pragma unroll
        for (int n = 0; n < NT; ++n) mma_bf16(sx[i][n], a, qb[n][kk][0], qb[n][kk][1]);
      }
    } else {
      // a thread's codes of keys g and g + 8: the d range [c D/4, (c + 1) D/4), four of a k step
      constexpr int KW = C::ROWB / 16;   // words of a key in one thread
      auto mma_q = [&](int n, int kk, const uint32_t (&a)[4]) {
        uint32_t b[2];
        lds<2>(qf + (n * KK + kk) * 256, b);
        mma_f16(sx[i][n], a, b[0], b[1]);
      };
      uint32_t w0[KW], w1[KW];
      if constexpr (KW == 8) {
        lds<4>(kb + ln[i].k[0], w0);
        lds<4>(kb + (ln[i].k[0] ^ 16u), w0 + 4);
        lds<4>(kb + ln[i].k[1], w1);
        lds<4>(kb + (ln[i].k[1] ^ 16u), w1 + 4);
      } else {
        lds<KW>(kb + ln[i].k[0], w0);
        lds<KW>(kb + ln[i].k[1], w1);
      }
      if constexpr (FMT == kFmtFP8) {
#pragma unroll
        for (int kk = 0; kk < KK; ++kk) {
          uint32_t a[4];
          e4m3x4_f16(w0[kk], a[0], a[2]);
          e4m3x4_f16(w1[kk], a[1], a[3]);
#pragma unroll
          for (int n = 0; n < NT; ++n) mma_q(n, kk, a);
        }
      } else {
        // block scales of the thread's d range: two blocks (D 128) or one (D 64)
        const uint32_t s0 = kb + C::OBS + (ln[i].rs + g) * (D / 16);
        uint32_t f0, f1;
        if constexpr (D == 128) {
          f0 = e4m3x2_f16x2(lds_u16(s0 + 2 * c));
          f1 = e4m3x2_f16x2(lds_u16(s0 + 8 * (D / 16) + 2 * c));
        } else {
          f0 = e4m3x2_f16x2(lds_u8(s0 + c) * 0x101u);
          f1 = e4m3x2_f16x2(lds_u8(s0 + 8 * (D / 16) + c) * 0x101u);
        }
        uint32_t b0 = 0, b1 = 0;
#pragma unroll
        for (int j = 0; j < KW; ++j) {   // a word: the codes of two k steps
          uint32_t h0[4], h1[4];
          e2m1x8_f16(w0[j], h0);
          e2m1x8_f16(w1[j], h1);
          if (j % (KW / (D / 64)) == 0) {   // the next block's scale, in both halves
            const uint32_t sel = j == 0 ? 0x1010u : 0x3232u;
            b0 = prmt(f0, f0, sel);
            b1 = prmt(f1, f1, sel);
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint32_t a[4] = {mul_f16x2(h0[2 * e], b0), mul_f16x2(h1[2 * e], b1),
                                   mul_f16x2(h0[2 * e + 1], b0), mul_f16x2(h1[2 * e + 1], b1)};
#pragma unroll
            for (int n = 0; n < NT; ++n) mma_q(n, 2 * j + e, a);
          }
        }
      }
    }
  }
  // ---- y = x - m: log2 of a key's weight, x its logit in log2 units. Over a quantised cache also
  // z = x + e - Z: log2 of its weight times its value row's scale 2^e. Whether any exceeds its
  // reference is one vote; the references themselves are taken across the warp only then.
  int ev[SPW][2];        // scale bytes of the value rows (quantised caches)
  float fk[SPW][2];      // scales of the key rows
  float y[SPW][NT][4], z[SPW][NT][4];
  int top = 0;
#pragma unroll
  for (int i = 0; i < SPW; ++i) {
    if constexpr (FMT != kFmtBF16) {
      const uint32_t rs = kb + C::ORS + ln[i].rs + g;
      const uint32_t k2 = lds_u8(rs) | (lds_u8(rs + 8) << 8);
      ev[i][0] = int(lds_u8(rs + ln[i].pse));
      ev[i][1] = int(lds_u8(rs + ln[i].pse + 8));
      uint32_t f2;   // 2^(b - 127) of both rows as bf16 (NaN for 255)
      asm("{.reg .b16 b; cvt.u16.u32 b, %1; cvt.rn.bf16x2.ue8m0x2 %0, b;}" : "=r"(f2) : "r"(k2));
      fk[i][0] = bf_lo(f2);
      fk[i][1] = bf_hi(f2);
      // q's factor here, the key's below: their product alone may leave FP32's range
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) sx[i][n][e] *= qs[n][e & 1];
    }
  }
  if (!full) {   // keys that are not the row's weigh nothing, whatever their slots hold
#pragma unroll
    for (int i = 0; i < SPW; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (valid(i, g + 8 * h)) continue;
        ev[i][h] = 0;
        fk[i][h] = 1.f;
#pragma unroll
        for (int n = 0; n < NT; ++n) sx[i][n][2 * h] = sx[i][n][2 * h + 1] = kNegInf;
      }
  }
  auto factor = [&](int i, int n, int e) { return FMT == kFmtBF16 ? qs[n][e & 1] : fk[i][e >> 1]; };   // from sx to x
  auto weigh = [&] {
#pragma unroll
    for (int i = 0; i < SPW; ++i)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float f = factor(i, n, e);
          y[i][n][e] = fmaf(sx[i][n][e], f, -S.m[n][e & 1]);
          if constexpr (FMT != kFmtBF16)
            z[i][n][e] = fmaf(sx[i][n][e], f, float(ev[i][e >> 1] - 127) - S.z[n][e & 1]);
        }
  };
  weigh();
  float most = kNegInf;
#pragma unroll
  for (int i = 0; i < SPW; ++i) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        most = fmaxf(most, y[i][n][e]);
        if constexpr (FMT != kFmtBF16) most = fmaxf(most, z[i][n][e]);
      }
    if constexpr (FMT != kFmtBF16) top = max(top, max(ev[i][0], ev[i][1]));
  }
  bool over = most > C::LAG;
  if constexpr (FMT != kFmtBF16) over |= top == 255;
  if (__any_sync(0xffffffffu, over)) {
    if constexpr (FMT != kFmtBF16) {
#pragma unroll
      for (int i = 0; i < SPW; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (ev[i][h] != 255) continue;   // else a row that holds no numbers: neither does what reads it
#pragma unroll
          for (int n = 0; n < NT; ++n) sx[i][n][2 * h] = sx[i][n][2 * h + 1] = __uint_as_float(0x7FFFFFFFu);
        }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float cr[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float m = S.m[n][h], zz = FMT == kFmtBF16 ? 0.f : S.z[n][h] + kBias;
#pragma unroll
        for (int i = 0; i < SPW; ++i)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float x = sx[i][n][2 * r + h] * factor(i, n, 2 * r + h);
            m = fmaxf(m, x);
            if constexpr (FMT != kFmtBF16) zz = fmaxf(zz, x + float(ev[i][r] - 127));
          }
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
          if constexpr (FMT != kFmtBF16) zz = fmaxf(zz, __shfl_xor_sync(0xffffffffu, zz, o));
        }
        const float cm = ex2(S.m[n][h] - m);   // 0 at the first numbers seen
        S.m[n][h] = m;
        S.l[n][h] *= cm;
        cr[h] = cm;
        if constexpr (FMT != kFmtBF16) {
          zz -= kBias;
          cr[h] = ex2(S.z[n][h] - zz);
          S.z[n][h] = zz;
        }
      }
#pragma unroll
      for (int mt = 0; mt < KK; ++mt) {
        S.acc[n][mt][0] *= cr[0];
        S.acc[n][mt][1] *= cr[1];
        S.acc[n][mt][2] *= cr[0];
        S.acc[n][mt][3] *= cr[1];
      }
    }
    weigh();
  }
  // ---- P, then its transpose as the B fragments of P^T: b[0] = (keys 2c, 2c+1; head g),
  // b[1] = (keys 2c+8, 2c+9; head g). BF16: P in a high and a low half.
  constexpr int PH = FMT == kFmtBF16 ? 2 : 1;
  uint32_t pb[SPW][NT][PH][2];
#pragma unroll
  for (int i = 0; i < SPW; ++i) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] = ex2(y[i][n][e]);
      S.l[n][0] += w[0] + w[2];
      S.l[n][1] += w[1] + w[3];
      if constexpr (FMT == kFmtBF16) {
        const uint32_t h01 = pack_bf16x2(w[0], w[1]), h23 = pack_bf16x2(w[2], w[3]);
        pb[i][n][0][0] = movtrans(h01);
        pb[i][n][0][1] = movtrans(h23);
        pb[i][n][PH - 1][0] = movtrans(pack_bf16x2(w[0] - bf_lo(h01), w[1] - bf_hi(h01)));
        pb[i][n][PH - 1][1] = movtrans(pack_bf16x2(w[2] - bf_lo(h23), w[3] - bf_hi(h23)));
      } else {
        pb[i][n][0][0] = movtrans(pack_f16x2(ex2(z[i][n][0]), ex2(z[i][n][1])));
        pb[i][n][0][1] = movtrans(pack_f16x2(ex2(z[i][n][2]), ex2(z[i][n][3])));
      }
    }
  }
  // ---- O^T += V^T . P^T. Keys that are not the row's have their values replaced by zeros, so
  // that P = 0 there contributes exactly nothing (their slots may hold anything, NaN included).
#pragma unroll
  for (int i = 0; i < SPW; ++i) {
    if constexpr (FMT == kFmtBF16) {
      uint32_t m01 = 0xFFFFFFFFu, m89 = 0xFFFFFFFFu;
      if (!full) {
        m01 = (valid(i, 2 * c) ? 0x0000FFFFu : 0u) | (valid(i, 2 * c + 1) ? 0xFFFF0000u : 0u);
        m89 = (valid(i, 2 * c + 8) ? 0x0000FFFFu : 0u) | (valid(i, 2 * c + 9) ? 0xFFFF0000u : 0u);
      }
#pragma unroll
      for (int mt = 0; mt < KK; ++mt) {
        uint32_t a[4];
        ldsm_x4_t(kb + (mt >> 2) * (C::KB / C::PLANES) + (ln[i].v[0] ^ uint32_t((mt & 3) << 5)), a[0], a[1], a[2], a[3]);
        a[0] &= m01;
        a[1] &= m01;
        a[2] &= m89;
        a[3] &= m89;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          mma_bf16(S.acc[n][mt], a, pb[i][n][0][0], pb[i][n][0][1]);
          mma_bf16(S.acc[n][mt], a, pb[i][n][PH - 1][0], pb[i][n][PH - 1][1]);
        }
      }
    } else {
      // keys {2c, 2c+1, 2c+8, 2c+9}, d range [g D/8, (g + 1) D/8): logical row g of m tile mt is
      // d = g D/8 + 2 mt, row g + 8 the next one
      constexpr int VW = C::ROWB / 32;
      uint32_t r[4][VW], bs[4] = {0, 0, 0, 0};
#pragma unroll
      for (int k = 0; k < 4; ++k) lds<VW>(kb + ln[i].v[k], r[k]);
      if constexpr (FMT == kFmtNVFP4) {   // the d range lies in one block of 16: one scale per key
        const uint32_t sa = kb + C::OBS + (ln[i].rs + ln[i].pse + 2 * c) * (D / 16) + (D == 128 ? g : g >> 1);
#pragma unroll
        for (int k = 0; k < 4; ++k) bs[k] = lds_u8(sa + ((k & 1) + 8 * (k >> 1)) * (D / 16));
      }
      if (!full) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (valid(i, 2 * c + (k & 1) + 8 * (k >> 1))) continue;
          bs[k] = 0;
#pragma unroll
          for (int j = 0; j < VW; ++j) r[k][j] = 0;
        }
      }
      if constexpr (FMT == kFmtFP8) {
#pragma unroll
        for (int mt = 0; mt < KK; ++mt) {
          const uint32_t sel = (mt & 1) ? 0x7362u : 0x5140u;
          uint32_t a[4];
          e4m3x4_f16(prmt(r[0][mt >> 1], r[1][mt >> 1], sel), a[0], a[1]);
          e4m3x4_f16(prmt(r[2][mt >> 1], r[3][mt >> 1], sel), a[2], a[3]);
#pragma unroll
          for (int n = 0; n < NT; ++n) mma_f16(S.acc[n][mt], a, pb[i][n][0][0], pb[i][n][0][1]);
        }
      } else {
        const uint32_t f01 = e4m3x2_f16x2(bs[0] | (bs[1] << 8)), f89 = e4m3x2_f16x2(bs[2] | (bs[3] << 8));
        constexpr uint32_t kLow = 0x0F0F0F0Fu;
#pragma unroll
        for (int j = 0; j < VW; ++j) {
          // bytes of (key 2c, key 2c+1) code pairs: even elements of four m tiles, then odd ones
          uint32_t ae[4], ao[4], be[4], bo[4];
          e2m1x8_f16((r[0][j] & kLow) | ((r[1][j] << 4) & ~kLow), ae);
          e2m1x8_f16(((r[0][j] >> 4) & kLow) | (r[1][j] & ~kLow), ao);
          e2m1x8_f16((r[2][j] & kLow) | ((r[3][j] << 4) & ~kLow), be);
          e2m1x8_f16(((r[2][j] >> 4) & kLow) | (r[3][j] & ~kLow), bo);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const uint32_t a[4] = {mul_f16x2(ae[q], f01), mul_f16x2(ao[q], f01), mul_f16x2(be[q], f89),
                                   mul_f16x2(bo[q], f89)};
#pragma unroll
            for (int n = 0; n < NT; ++n) mma_f16(S.acc[n][4 * j + q], a, pb[i][n][0][0], pb[i][n][0][1]);
          }
        }
      }
    }
  }
}

// The consumer warps' partials of a pair (combine buffer b of the CTA), joined: the four outputs
// from element idx of the pair's [G][D / 4]. A pair that other ranges share goes to the workspace
// (rows pb ..), another is finished.
template <int FMT, class C>
__device__ __forceinline__ void join_warps(const Params& P, uint8_t* sm, int b, int idx, bool split,
                                           size_t pb, size_t o_pair, uint2 gv, float gb) {
  constexpr int D = C::D;
  const float* Ow = reinterpret_cast<const float*>(sm + C::OW + b * C::OWB);
  const float2* MLw = reinterpret_cast<const float2*>(sm + C::MLW + b * C::MLB);
  const int h = idx / (D / 4), d = 4 * (idx - h * (D / 4));
  float M = kLowest, L = 0.f;
  float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int ww = 0; ww < C::WPG; ++ww) M = fmaxf(M, MLw[ww * C::HEADS + h].x);
#pragma unroll
  for (int ww = 0; ww < C::WPG; ++ww) {
    const float2 ml = MLw[ww * C::HEADS + h];
    const float fw = ex2(ml.x - M);
    L += fw * ml.y;
    const float4 v = *reinterpret_cast<const float4*>(Ow + (ww * C::HEADS + h) * C::OLD + spread<FMT, D>(d));
    O.x += fw * v.x;
    O.y += fw * v.y;
    O.z += fw * v.z;
    O.w += fw * v.w;
  }
  if (split) {
    *reinterpret_cast<float4*>(P.part_acc + (pb + h) * D + d) = O;
    if (d == 0) *reinterpret_cast<float2*>(P.part_ml + (pb + h) * 2) = make_float2(M, L);
  } else {
    finish4(P.g != nullptr, O, L, gv, gb, P.og + o_pair + 4 * idx);
  }
}

// Row of the partial results of part s of a joined pair and its query head h: the first part's slot
// is jn.w, and in the ranges after it the pair is the first.
template <int HEADS>
__device__ __forceinline__ size_t part_row(const int4& jn, int range, int s, int h) {
  return (size_t(2 * (range + s)) + (s == 0 ? jn.w : 0)) * HEADS + h;
}

template <int FMT, int D, int NT>
__global__ void __launch_bounds__(Cfg<FMT, D, NT>::THREADS, 1) paged_decode_kernel(
    const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
    const Params P) {
  using C = Cfg<FMT, D, NT>;
  constexpr int NCT = C::NCT, BK = C::BK;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                           ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(sm);
  const uint32_t bar_full = sbase + C::BAR, bar_empty = bar_full + 8 * C::NST;
  volatile int* misc = reinterpret_cast<volatile int*>(sm + C::MISC);   // -, abort, -, -
  volatile unsigned* masks = reinterpret_cast<volatile unsigned*>(sm + C::MISC + 16);
  int4* joins = reinterpret_cast<int4*>(sm + C::JOIN);
  int* cum = reinterpret_cast<int*>(sm + C::CUM);
  int* rpos = reinterpret_cast<int*>(sm + C::POS);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::NST; ++s) {
      mbar_init(bar_full + 8 * s, 1);
      mbar_init(bar_empty + 8 * s, C::WPG);
    }
    misc[1] = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
  pdl_wait();
  // ---- plan: cum[t] = blocks of one KV head in rows 0 .. t - 1
  const int T = P.T;
  if (T <= 32) {   // every warp works it out, and writes the same
    const Row r = row_of<BK>(P, min(lane, T - 1));
    if (r.bad && lane < T && blockIdx.x == 0 && warp == 0) flag(r.bad);
    int run = lane < T ? r.nb : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, run, o);
      if (lane >= o) run += u;
    }
    if (lane < T) {
      cum[lane + 1] = run;
      rpos[lane] = r.p;
    }
    if (lane == 0) cum[0] = 0;
    __syncwarp();
  } else {
    for (int t = threadIdx.x; t < T; t += C::THREADS) {
      const Row r = row_of<BK>(P, t);
      cum[t + 1] = r.nb;
      rpos[t] = r.p;
      if (r.bad && blockIdx.x == 0) flag(r.bad);
    }
    __syncthreads();
    if (warp == 0) {
      const int per = (T + 31) / 32, a = min(T, lane * per), b = min(T, a + per);
      int sum = 0;
      for (int t = a; t < b; ++t) sum += cum[t + 1];
      int run = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, run, o);
        if (lane >= o) run += u;
      }
      run -= sum;
      for (int t = a; t < b; ++t) {
        run += cum[t + 1];
        cum[t + 1] = run;
      }
      if (lane == 0) cum[0] = 0;
    }
    __syncthreads();
  }
  const int total = cum[T] * P.n_kv;
  // row of flat block f: the last t with cum[t] * n_kv <= f
  auto row_at = [&](int f) {
    int a = 0, b = T;   // cum[a] * n_kv <= f < cum[b] * n_kv
    while (b - a > 1) {
      const int mid = (a + b) >> 1;
      if (cum[mid] * P.n_kv <= f) a = mid;
      else b = mid;
    }
    return a;
  };
  // the warp's group and its range of the flat blocks
  const int grp = warp < C::NCW ? warp / C::WPG : (warp - C::NCW) % C::GROUPS;
  const int range = P.whole ? int(blockIdx.x) * C::GROUPS + grp : grp * int(gridDim.x) + int(blockIdx.x);
  int f0 = 0, R, f_lo, f_hi;   // ranges of R blocks from f0
  if (P.whole) {
    // the CTA's equal share, both ends moved up to the next pair's first block, is cut for the groups
    const int share = max(1, (total + int(gridDim.x) - 1) / int(gridDim.x));
    auto up = [&](int64_t x) {
      if (x >= total) return total;
      const int f = int(x), t = row_at(f), nb = cum[t + 1] - cum[t], r = (f - cum[t] * P.n_kv) % nb;
      return r ? f + nb - r : f;
    };
    f0 = up(int64_t(blockIdx.x) * share);
    const int end = up(int64_t(blockIdx.x + 1) * share);
    R = max(1, (end - f0 + C::GROUPS - 1) / C::GROUPS);
    f_lo = min(end, f0 + grp * R);
    f_hi = min(end, f_lo + R);
  } else {
    R = max(1, (total + P.ranges - 1) / P.ranges);
    f_lo = int(min(int64_t(total), int64_t(range) * R));
    f_hi = min(total, f_lo + R);
  }
  const int t_lo = f_lo < f_hi ? row_at(f_lo) : 0;
  // the range's pairs in order: flat block f is block j0 of the pair whose blocks begin at f_pair;
  // the range holds its blocks j0 .. j1 - 1 of nb
  struct PairAt {
    int f, t, hk, nb, f_pair, j0, j1;
  };
  auto pair_at = [&](int f) {
    PairAt a{f, t_lo, 0, 1, f, 0, 0};
    if (f >= f_hi) return a;   // an empty range: no blocks from f on
    a.nb = cum[t_lo + 1] - cum[t_lo];
    const int r = f - cum[t_lo] * P.n_kv;
    a.hk = r / a.nb;
    a.j0 = r - a.hk * a.nb;
    a.f_pair = f - a.j0;
    a.j1 = min(a.nb, f_hi - a.f_pair);
    return a;
  };
  auto next_pair = [&](PairAt a) {
    a.f = a.f_pair + a.j1;
    if (a.f >= f_hi) return a;
    if (++a.hk == P.n_kv) {
      a.hk = 0;
      do ++a.t;
      while (cum[a.t + 1] == cum[a.t]);
      a.nb = cum[a.t + 1] - cum[a.t];
    }
    a.f_pair = a.f;
    a.j0 = 0;
    a.j1 = min(a.nb, f_hi - a.f);
    return a;
  };

  if (warp >= C::NCW && warp < C::NCW + C::GROUPS) {
    // ---------------- producers
    const int pse = min(P.c.page_size, BK), npg = BK / pse;   // keys of a page in a block, pages
    struct At {
      int t, hk, j, nb, blk0, lo, p, s;
    };
    auto load_row = [&](At& a) {
      const Row r = row_of<BK>(P, a.t);
      a.nb = r.nb;
      a.blk0 = r.blk0;
      a.lo = r.lo;
      a.p = r.p;
      a.s = r.s;
    };
    auto advance = [&](At& a) {   // there is a next block
      if (++a.j < a.nb) return;
      a.j = 0;
      if (++a.hk < P.n_kv) return;
      a.hk = 0;
      do ++a.t;
      while (cum[a.t + 1] == cum[a.t]);
      load_row(a);
    };
    // lane i's page of the block: its number, or -2 where the block has no key in it
    auto fetch = [&](const At& a) -> int {
      if (lane >= npg) return -2;
      const int k0 = (a.blk0 + a.j) * BK + lane * pse;   // keys k0 + 1 .. k0 + pse
      if (k0 + pse < a.lo || k0 + 1 > a.p) return -2;
      return P.c.page_table[size_t(a.s) * P.c.table_stride + (k0 >> P.shift)];
    };
    At at{t_lo, 0, 0, 1, 0, 1, 0, 0};
    int id = -2;
    if (f_lo < f_hi) {
      load_row(at);
      const int r = f_lo - cum[at.t] * P.n_kv;
      at.hk = r / at.nb;
      at.j = r - at.hk * at.nb;
      id = fetch(at);
    }
    int i = 0;
    for (int f = f_lo; f < f_hi; ++f, ++i) {
      const At a = at;
      const int page = id;
      if (f + 1 < f_hi) {
        advance(at);
        id = fetch(at);   // the pages of the next block, while this one waits
      }
      const int st = grp * C::NSTG + i % C::NSTG;
      bool go = misc[1] == 0;
      if (go && i >= C::NSTG) go = mbar_wait(bar_empty + 8 * st, ((i / C::NSTG) - 1) & 1);
      if (!__all_sync(0xffffffffu, go)) {
        if (lane == 0) misc[1] = 1;
        break;
      }
      const bool ok = page >= 0 && page < P.c.num_pages;
      if (page != -2 && !ok) flag(BEAM_DEV_BAD_PAGE);
      const unsigned okm = __ballot_sync(0xffffffffu, ok);
      const uint32_t base = sbase + st * C::STAGE, fb = bar_full + 8 * st;
      const int z = page * P.n_kv + a.hk;
      const int off = ((a.blk0 + a.j) * BK + lane * pse) & (P.c.page_size - 1);   // first key in the page
      const int y = C::PLANES == 2 ? off : off * C::ROWB / 128;
      const bool part = pse < P.c.page_size;   // part of a page: K's and V's scales lie apart
      const bool with_q = f == f_lo || a.j == 0;   // a pair's first block here
      const unsigned slices = __ballot_sync(0xffffffffu, lane < C::SLICES && ((okm >> (lane * 16 / pse)) & 1u));
      if (lane == 0) {
        masks[st] = slices;
        constexpr int row = C::ROWB + (FMT != kFmtBF16 ? 1 : 0) + (FMT == kFmtNVFP4 ? D / 16 : 0);
        mbar_expect_tx(fb, __popc(okm) * pse * 2 * row + (with_q ? P.G * D * 2 : 0));
      }
      __syncwarp();
      if (ok) {
        const uint32_t dk = base + lane * pse * (C::ROWB / C::PLANES), dv = dk + C::KB;
        tma_load_3d(dk, &tk, 0, y, z, fb);
        if constexpr (C::PLANES == 2) tma_load_3d(dk + C::KB / 2, &tk, 128, y, z, fb);
        tma_load_3d(dv, &tv, 0, y, z, fb);
        if constexpr (C::PLANES == 2) tma_load_3d(dv + C::KB / 2, &tv, 128, y, z, fb);
        if constexpr (FMT != kFmtBF16) {
          const size_t sr = size_t(z) * 2 * P.c.page_size + off;
          const uint32_t dr = base + C::ORS + lane * 2 * pse;
          bulk_load(dr, P.c.row_scale + sr, part ? pse : 2 * pse, fb);
          if (part) bulk_load(dr + pse, P.c.row_scale + sr + P.c.page_size, pse, fb);
          if constexpr (FMT == kFmtNVFP4) {
            const uint8_t* src = P.c.block_scale + sr * (D / 16);
            const uint32_t db = base + C::OBS + lane * 2 * pse * (D / 16);
            bulk_load(db, src, (part ? 1 : 2) * pse * (D / 16), fb);
            if (part) bulk_load(db + pse * (D / 16), src + P.c.page_size * (D / 16), pse * (D / 16), fb);
          }
        }
      }
      if (with_q && lane == 31)
        bulk_load(base + C::OQ, P.q + (size_t(a.t) * P.n_q + a.hk * P.G) * D, P.G * D * 2, fb);
      __syncwarp();
    }
    // normally done at once, with the last blocks: after an expired wait elsewhere, let the copies
    // in flight land before the CTA's shared memory is released
    if (lane == 0)
      for (int k = i - 1; k >= 0 && k >= i - C::NSTG; --k)
        mbar_wait(bar_full + 8 * (grp * C::NSTG + k % C::NSTG), (k / C::NSTG) & 1);
  } else if (warp >= C::NCW) {
    if constexpr (C::FIN) {
      // ---------------- finishers: all pairs but the range's last, which nothing follows
      int buf = 0;
      for (PairAt a = pair_at(f_lo); a.f_pair + a.j1 < f_hi; a = next_pair(a)) {
        const bool split = a.j0 > 0 || a.j1 < a.nb;
        const size_t o_pair = (size_t(a.t) * P.n_q + a.hk * P.G) * D;
        const size_t pb = size_t(2 * range) * C::HEADS;   // split: the range's first pair
        // A step finishes PER heads, four outputs a lane; lane h holds head h's weights. U steps at a
        // time without a branch between them, so that one's latencies cover another's.
        constexpr int PER = 128 / D, N = C::HEADS / PER, U = 4;
        const int hl = lane % C::HEADS, sub = lane / (D / 4), d = 4 * (lane % (D / 4));
        const bool gated = P.g != nullptr && !split;
        uint2 gv[N];   // the gates, ahead of the wait
        float bias = 0.f;
#pragma unroll
        for (int u = 0; u < N; ++u) gv[u] = make_uint2(0u, 0u);
        if (gated) {
          if (hl < P.G) bias = bf2f(ld_ahead16(P.gate_bias + a.hk * P.G + hl));
#pragma unroll
          for (int u = 0; u < N; ++u)
            if (u * PER + sub < P.G) gv[u] = ld_ahead(P.g + o_pair + (u * PER + sub) * D + d);
        }
        pair_bar<NCT + 32, true>(grp, 0, buf);
        const float* Ow = reinterpret_cast<const float*>(sm + C::OW + (grp * C::NOW + buf) * C::OWB);
        const float2* MLw = reinterpret_cast<const float2*>(sm + C::MLW + (grp * C::NOW + buf) * C::MLB);
        float M = kLowest, L = 0.f, fw[C::WPG];
#pragma unroll
        for (int ww = 0; ww < C::WPG; ++ww) M = fmaxf(M, MLw[ww * C::HEADS + hl].x);
#pragma unroll
        for (int ww = 0; ww < C::WPG; ++ww) {
          const float2 ml = MLw[ww * C::HEADS + hl];
          fw[ww] = ex2(ml.x - M);
          L += fw[ww] * ml.y;
        }
        const float inv = inverse(L);
        if (split && lane < P.G) *reinterpret_cast<float2*>(P.part_ml + (pb + lane) * 2) = make_float2(M, L);
#pragma unroll
        for (int u0 = 0; u0 < N; u0 += U) {
          if (u0 * PER >= P.G) break;
          float4 O[U];
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const int h = (u0 + u) * PER + sub;
            O[u] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int ww = 0; ww < C::WPG; ++ww) {
              const float f = __shfl_sync(0xffffffffu, fw[ww], h);
              const float4 v = *reinterpret_cast<const float4*>(Ow + (ww * C::HEADS + h) * C::OLD + spread<FMT, D>(d));
              O[u].x += f * v.x;
              O[u].y += f * v.y;
              O[u].z += f * v.z;
              O[u].w += f * v.w;
            }
          }
          if (split) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
              const int h = (u0 + u) * PER + sub;
              if (h < P.G) *reinterpret_cast<float4*>(P.part_acc + (pb + h) * D + d) = O[u];
            }
            continue;
          }
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const float f = __shfl_sync(0xffffffffu, inv, (u0 + u) * PER + sub);
            O[u] = make_float4(O[u].x * f, O[u].y * f, O[u].z * f, O[u].w * f);
          }
          if (gated) {
#pragma unroll
            for (int u = 0; u < U; ++u)
              gate4(O[u], gv[u0 + u], __shfl_sync(0xffffffffu, bias, (u0 + u) * PER + sub));
          }
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const int h = (u0 + u) * PER + sub;
            if (h < P.G) *reinterpret_cast<uint2*>(P.og + o_pair + h * D + d) = pack4(O[u]);
          }
        }
        pair_bar<NCT + 32, false>(grp, 1, buf);
        buf = C::NOW - 1 - buf;
      }
    }
  } else {
    // ---------------- consumers
    const int w = warp % C::WPG, g = lane >> 2, c = lane & 3, ct = threadIdx.x % NCT;
    Lane<FMT, C> ln[C::SPW];
#pragma unroll
    for (int e = 0; e < C::SPW; ++e) ln[e] = lane_of<FMT, C>(w + e * C::WPG, min(P.c.page_size, BK));
    const uint32_t qf = sbase + C::QF + grp * C::QBUFS * C::QB + lane * 8;
    bool dead = false;   // a wait has expired: the rest of the range passes without results
    const int G = P.G;
    int i = 0, buf = 0, pairs = 0;
    int4 join = make_int4(0, 0, 0, 0);
    for (PairAt at = pair_at(f_lo); at.f < f_hi; at = next_pair(at)) {
      const int p = rpos[at.t], lo = P.c.window > 0 ? max(1, p - P.c.window + 1) : 1;
      const int blk0 = (lo - 1) / BK, j0 = at.j0, j1 = at.j1;
      const bool split = j0 > 0 || j1 < at.nb;
      // the gate of the outputs that this thread finishes: fetched ahead
      uint2 gv[C::ITEMS];
      float gb[C::ITEMS];
      const size_t o_pair = (size_t(at.t) * P.n_q + at.hk * G) * D;
      auto fetch_gate = [&] {
        if (P.g == nullptr || split) return;
#pragma unroll
        for (int it = 0; it < C::ITEMS; ++it) {
          const int idx = ct + it * NCT;
          if (idx < G * (D / 4)) {
            gv[it] = ld_ahead(P.g + o_pair + 4 * idx);
            gb[it] = bf2f(ld_ahead16(P.gate_bias + at.hk * G + idx / (D / 4)));
          }
        }
      };
      const bool mine = !C::FIN || at.f_pair + j1 >= f_hi;   // no finisher, or the range's last pair
      const int q_buf = C::QBUFS == 2 ? pairs & 1 : 0;
      uint32_t qb[NT][D / 16][2];
      float qs[NT][2];
      WarpState<C> S;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        S.m[n][0] = S.m[n][1] = S.z[n][0] = S.z[n][1] = kLowest;
        S.l[n][0] = S.l[n][1] = 0.f;
#pragma unroll
        for (int mt = 0; mt < D / 16; ++mt) S.acc[n][mt][0] = S.acc[n][mt][1] = S.acc[n][mt][2] = S.acc[n][mt][3] = 0.f;
      }
      for (int j = j0; j < j1; ++j, ++i) {
        const int st = grp * C::NSTG + i % C::NSTG;
        const uint32_t kb = sbase + st * C::STAGE;
        if (!dead) dead = !__all_sync(0xffffffffu, mbar_wait(bar_full + 8 * st, (i / C::NSTG) & 1));
        if (!dead) {
          if (j == j0) {
            // q fragments (B operand, column = head g of the tile)
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              const int h = 8 * n + g;
              const bool rok = h < G;
              const uint32_t qa = kb + C::OQ + (rok ? h : 0) * D * 2;
              if constexpr (FMT == kFmtBF16) {
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                  lds<1>(qa + (8 * kk + c) * 4, &qb[n][kk][0]);
                  lds<1>(qa + (8 * kk + c + 4) * 4, &qb[n][kk][1]);
                  if (!rok) qb[n][kk][0] = qb[n][kk][1] = 0u;
                }
                qs[n][0] = qs[n][1] = P.sl2;
              } else {
                unsigned mx = 0;   // the head's largest magnitude, as a bf16 pattern (at first two)
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                  lds<2>(qa + (D / 8) * c * 4 + kk * 8, qb[n][kk]);
#pragma unroll
                  for (int e = 0; e < 2; ++e) {
                    if (!rok) qb[n][kk][e] = 0u;
                    mx = __vmaxu2(mx, qb[n][kk][e] & 0x7FFF7FFFu);
                  }
                }
                mx = max(mx & 0xFFFFu, mx >> 16);
                mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                // q * 2^(me - 127): the largest magnitude lies in [2^14, 2^15)
                const int me = min(254, 268 - int(mx >> 7));
                const float up = __uint_as_float(unsigned(me) << 23);
                // each warp writes its part of what all read
                uint8_t* dst = sm + C::QF + (grp * C::QBUFS + q_buf) * C::QB + n * D * 16 + lane * 8;
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                  if (kk % C::WPG != w) continue;
#pragma unroll
                  for (int e = 0; e < 2; ++e)
                    qb[n][kk][e] = pack_f16x2(bf_lo(qb[n][kk][e]) * up, bf_hi(qb[n][kk][e]) * up);
                  *reinterpret_cast<uint2*>(dst + kk * 256) = make_uint2(qb[n][kk][0], qb[n][kk][1]);
                }
                const float back = P.sl2 * pow2_of(unsigned(254 - me));
                qs[n][0] = __shfl_sync(0xffffffffu, back, 8 * c);
                qs[n][1] = __shfl_sync(0xffffffffu, back, 8 * c + 4);
              }
            }
            if constexpr (C::QSM) consumer_bar<NCT>(grp);   // once a pair and warp, live or dead
          }
          const int kbase = BK * (blk0 + j) + 16 * w + 1;
          unsigned live = 0;
#pragma unroll
          for (int e = 0; e < C::SPW; ++e) {
            const int k0 = kbase + 16 * C::WPG * e;
            if (((masks[st] >> (w + e * C::WPG)) & 1u) && k0 <= p && k0 + 15 >= lo) live |= 1u << e;
          }
          if (live) warp_block<FMT, C>(kb, ln, qb, qf + q_buf * C::QB, qs, kbase, live, lo, p, S);
        } else {
          if constexpr (C::QSM) {
            if (j == j0) consumer_bar<NCT>(grp);
          }
          if (lane == 0) misc[1] = 1;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_empty + 8 * st);
      }
      // ---- the warp's partial of the pair, into a buffer that its last reader has left
      if (mine) fetch_gate();
      if constexpr (C::FIN) {
        if (pairs >= C::NOW) pair_bar<NCT + 32, true>(grp, 1, buf);
      } else if constexpr (C::NOW == 1) {
        consumer_bar<NCT>(grp);
      }
      float* Ow = reinterpret_cast<float*>(sm + C::OW + (grp * C::NOW + buf) * C::OWB);
      float2* MLw = reinterpret_cast<float2*>(sm + C::MLW + (grp * C::NOW + buf) * C::MLB);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
          S.l[n][0] += __shfl_xor_sync(0xffffffffu, S.l[n][0], o);
          S.l[n][1] += __shfl_xor_sync(0xffffffffu, S.l[n][1], o);
        }
        const int h0 = w * C::HEADS + 8 * n + 2 * c;
        float* ow = Ow + h0 * C::OLD;
        // acc relative to 2^m, as l is: 2^(z - m) in two steps, which alone may leave FP32's range
        const float u0 = ex2(0.5f * (S.z[n][0] - S.m[n][0])), u1 = ex2(0.5f * (S.z[n][1] - S.m[n][1]));
#pragma unroll
        for (int mt = 0; mt < D / 16; ++mt) {
          const float(&a)[4] = S.acc[n][mt];
          if constexpr (FMT == kFmtBF16) {   // rows g, g + 8 of m tile mt
            ow[16 * mt + g] = a[0];
            ow[C::OLD + 16 * mt + g] = a[1];
            ow[16 * mt + g + 8] = a[2];
            ow[C::OLD + 16 * mt + g + 8] = a[3];
          } else {   // neighbours
            const int d = spread<FMT, D>(D / 8 * g + 2 * mt);
            *reinterpret_cast<float2*>(ow + d) = make_float2(a[0] * u0 * u0, a[2] * u0 * u0);
            *reinterpret_cast<float2*>(ow + C::OLD + d) = make_float2(a[1] * u1 * u1, a[3] * u1 * u1);
          }
        }
        if (g == 0) {
          MLw[h0] = make_float2(S.m[n][0], S.l[n][0]);
          MLw[h0 + 1] = make_float2(S.m[n][1], S.l[n][1]);
        }
      }
      if (!mine) {
        pair_bar<NCT + 32, false>(grp, 0, buf);
      } else {
        // without a finisher two buffers in turn: who writes one has passed the barrier of the pair
        // between, which its last readers came to later
        consumer_bar<NCT>(grp);
        const int slot = at.f == f_lo ? 0 : 1;   // the range's first pair, or its last
        const size_t pb = (size_t(2 * range) + slot) * C::HEADS;
#pragma unroll
        for (int it = 0; it < C::ITEMS; ++it) {
          const int idx = ct + it * NCT;
          if (idx < G * (D / 4)) join_warps<FMT, C>(P, sm, grp * C::NOW + buf, idx, split, pb, o_pair, gv[it], gb[it]);
        }
        if (j0 == 0 && j1 < at.nb)   // the pair begins here and runs on
          join = make_int4(at.t, at.hk, (at.f_pair + at.nb - 1 - f0) / R - (f_lo - f0) / R + 1, slot);
      }
      buf = C::NOW - 1 - buf;
      ++pairs;
    }
    // every release of a buffer is waited for: that of the last pair but one is left
    if (C::FIN && C::NOW == 2 && pairs >= 2) pair_bar<NCT + 32, true>(grp, 1, buf);
    if (ct == 0) {
      if (P.whole) joins[grp] = join;
      else if (range < P.ranges) P.join[range] = join;
    }
    // ---- rows that attend to nothing
    for (int r = blockIdx.x; r < T; r += gridDim.x)
      if (cum[r + 1] == cum[r])
        for (int x = threadIdx.x; x < P.n_q * (D / 8); x += C::GROUPS * NCT)
          reinterpret_cast<uint4*>(P.og + size_t(r) * P.n_q * D)[x] = make_uint4(0, 0, 0, 0);
  }
  __syncthreads();
  pdl_trigger();   // not earlier: the join and what follows would run beside the key stream
  if (P.whole) {
    // pairs that the CTA's groups share, joined here: at most GROUPS parts each
    for (int x = threadIdx.x; x < C::GROUPS * P.G * (D / 4); x += C::THREADS) {
      const int gr = x / (P.G * (D / 4)), y = x - gr * P.G * (D / 4), h = y / (D / 4), d = 4 * (y - h * (D / 4));
      const int4 jn = joins[gr];
      if (jn.z == 0) continue;
      const int first = int(blockIdx.x) * C::GROUPS + gr;
      float2 ml[C::GROUPS];
      float4 v[C::GROUPS];
      float M = kLowest, L = 0.f;
#pragma unroll
      for (int s = 0; s < C::GROUPS; ++s) {
        ml[s] = make_float2(kLowest, 0.f);
        v[s] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (s >= jn.z) continue;
        const size_t r = part_row<C::HEADS>(jn, first, s, h);
        ml[s] = __ldcg(reinterpret_cast<const float2*>(P.part_ml + 2 * r));
        v[s] = __ldcg(reinterpret_cast<const float4*>(P.part_acc + r * D + d));
        M = fmaxf(M, ml[s].x);
      }
      float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int s = 0; s < C::GROUPS; ++s) {
        const float fw = ex2(ml[s].x - M);
        L += fw * ml[s].y;
        O.x += fw * v[s].x;
        O.y += fw * v[s].y;
        O.z += fw * v[s].z;
        O.w += fw * v[s].w;
      }
      const int hq = jn.y * P.G + h;
      const size_t oi = (size_t(jn.x) * P.n_q + hq) * D + d;
      uint2 gv = make_uint2(0, 0);
      float gb = 0.f;
      if (P.g != nullptr) {
        gv = *reinterpret_cast<const uint2*>(P.g + oi);
        gb = bf2f(P.gate_bias[hq]);
      }
      finish4(P.g != nullptr, O, L, gv, gb, P.og + oi);
    }
  }
  if (threadIdx.x == 0 && misc[1]) flag(BEAM_DEV_TIMEOUT);
}

// Join of the pair that begins in range blockIdx.x and runs on past it: four neighbouring outputs
// a thread, WAYS threads to share their parts; the parts' weights are found as they come.
constexpr int kJoinThreads = 256;
template <int D, int HEADS, int WAYS>
__global__ void __launch_bounds__(kJoinThreads * WAYS) paged_join_kernel(const Params P) {
  pdl_trigger();
  __shared__ float4 acc[WAYS][kJoinThreads];
  __shared__ float2 part[WAYS][kJoinThreads];
  pdl_wait();
  const int4 jn = P.join[blockIdx.x];
  const int n = jn.z, lane = threadIdx.x % kJoinThreads, way = threadIdx.x / kJoinThreads;
  if (n == 0) return;
#pragma unroll
  for (int x0 = 0; x0 < HEADS * (D / 4); x0 += kJoinThreads) {
    const int x = x0 + lane, h = x / (D / 4), d = 4 * (x - h * (D / 4));
    const bool live = h < P.G;
    const int hq = jn.y * P.G + h;
    const size_t oi = (size_t(jn.x) * P.n_q + hq) * D + d;
    uint2 gv = make_uint2(0, 0);
    float gb = 0.f, M = kLowest, L = 0.f;
    float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
    if (live && way == 0 && P.g != nullptr) {
      gv = ld_ahead(P.g + oi);
      gb = bf2f(ld_ahead16(P.gate_bias + hq));
    }
    constexpr int U = WAYS == 1 ? 8 : 5;   // parts in flight
    for (int s0 = way; s0 < n && live; s0 += U * WAYS) {
      float2 ml[U];
      float4 v[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int s = s0 + u * WAYS;
        ml[u] = make_float2(kLowest, 0.f);
        v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (s >= n) continue;
        const size_t r = part_row<HEADS>(jn, blockIdx.x, s, h);
        ml[u] = __ldcg(reinterpret_cast<const float2*>(P.part_ml + 2 * r));
        v[u] = __ldcg(reinterpret_cast<const float4*>(P.part_acc + r * D + d));
      }
      float top = M;
#pragma unroll
      for (int u = 0; u < U; ++u) top = fmaxf(top, ml[u].x);
      const float f = ex2(M - top);
      M = top;
      L *= f;
      O.x *= f;
      O.y *= f;
      O.z *= f;
      O.w *= f;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const float fw = ex2(ml[u].x - M);
        L += fw * ml[u].y;
        O.x += fw * v[u].x;
        O.y += fw * v[u].y;
        O.z += fw * v[u].z;
        O.w += fw * v[u].w;
      }
    }
    if (WAYS > 1) {
      acc[way][lane] = O;
      part[way][lane] = make_float2(M, L);
      __syncthreads();
      if (way == 0) {
        float top = M;
#pragma unroll
        for (int u = 1; u < WAYS; ++u) top = fmaxf(top, part[u][lane].x);
        L = 0.f;
        O = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int u = 0; u < WAYS; ++u) {
          const float fw = ex2(part[u][lane].x - top);
          const float4 v = acc[u][lane];
          L += fw * part[u][lane].y;
          O.x += fw * v.x;
          O.y += fw * v.y;
          O.z += fw * v.z;
          O.w += fw * v.w;
        }
      }
      __syncthreads();
    }
    if (live && way == 0) finish4(P.g != nullptr, O, L, gv, gb, P.og + oi);
  }
}

template <int FMT>
int block_keys_of(int D, int nt) {
  if (D == 128) return nt == 1 ? Cfg<FMT, 128, 1>::BK : Cfg<FMT, 128, 2>::BK;
  return nt == 1 ? Cfg<FMT, 64, 1>::BK : Cfg<FMT, 64, 2>::BK;
}
int block_keys(int fmt, int D, int nt) {
  return fmt == kFmtBF16 ? block_keys_of<kFmtBF16>(D, nt)
         : fmt == kFmtFP8 ? block_keys_of<kFmtFP8>(D, nt) : block_keys_of<kFmtNVFP4>(D, nt);
}

// Rows of partial results: two pairs a range, 8 nt heads each.
size_t part_rows(int nt) { return size_t(kMaxParts) * 2 * 8 * nt; }

int max_grid() {
  const int sms = num_sms_cached();
  return sms < kMaxGrid ? sms : kMaxGrid;
}

// The paged_decode_kernel's shared memory, asked for once per device (0.2 us of the ~3.5 of a call).
// The attribute does not change again, so two threads that ask at once do no harm.
template <int FMT, int D, int NT>
cudaError_t allow_smem() {
  static std::atomic<bool> done[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 64 && done[dev].load(std::memory_order_relaxed)) return cudaSuccess;
  e = cudaFuncSetAttribute(paged_decode_kernel<FMT, D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           Cfg<FMT, D, NT>::BYTES);
  if (e == cudaSuccess && dev < 64) done[dev].store(true, std::memory_order_relaxed);
  return e;
}

// pairs: (row, KV head) pairs; blocks: an upper bound of their blocks
template <int FMT, int D, int NT>
cudaError_t launch(Params p, int64_t pairs, int64_t blocks, cudaStream_t st) {
  using C = Cfg<FMT, D, NT>;
  // no range smaller than a block, no CTA with less than a pair where CTAs do not share pairs
  const int sms = max_grid(), most = C::GROUPS * sms;
  p.ranges = int(blocks < most ? blocks : most);
  const int units = p.whole ? int(pairs < sms ? pairs : sms) : p.ranges;
  const int grid = units < sms ? units : sms;
  const beam_paged_kv& c = p.c;
  CUtensorMap mk, mv;
  const int rows = C::PLANES == 2 ? c.page_size : c.page_size * C::ROWB / 128;
  const int pse = c.page_size < C::BK ? c.page_size : C::BK;
  const uint64_t inner = C::PLANES == 2 ? 256 : 128;
  const uint64_t dims[3] = {inner, uint64_t(rows), uint64_t(c.num_pages) * c.n_kv};
  const uint64_t str[2] = {inner, uint64_t(c.page_size) * C::ROWB};
  const uint32_t box[3] = {128, uint32_t(C::PLANES == 2 ? pse : pse * C::ROWB / 128), 1};
  if (!encode_tiled(&mk, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, c.k, dims, str, box, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !encode_tiled(&mv, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, c.v, dims, str, box, CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  auto kern = paged_decode_kernel<FMT, D, NT>;
  cudaError_t e = allow_smem<FMT, D, NT>();
  if (e != cudaSuccess) return e;
  e = launch_pdl(kern, dim3(grid), dim3(C::THREADS), C::BYTES, st, mk, mv, p);
  if (e != cudaSuccess || p.whole) return e;
  // many parts to a pair: more threads fetch them at once
  if (p.ranges >= 8 * pairs)
    return launch_pdl(paged_join_kernel<D, C::HEADS, 4>, dim3(p.ranges), dim3(4 * kJoinThreads), 0, st, p);
  return launch_pdl(paged_join_kernel<D, C::HEADS, 1>, dim3(p.ranges), dim3(kJoinThreads), 0, st, p);
}

template <int FMT>
cudaError_t launch_fmt(const Params& p, int64_t pairs, int64_t blocks, cudaStream_t st) {
  const bool one = p.G <= 8;
  if (p.c.head_dim == 128)
    return one ? launch<FMT, 128, 1>(p, pairs, blocks, st) : launch<FMT, 128, 2>(p, pairs, blocks, st);
  return one ? launch<FMT, 64, 1>(p, pairs, blocks, st) : launch<FMT, 64, 2>(p, pairs, blocks, st);
}

}  // namespace
}  // namespace paged
}  // namespace beam

extern "C" size_t beam_paged_workspace_bytes(const beam_layer_cfg* cfg, int T, int max_pos) {
  using namespace beam;
  using namespace beam::paged;
  (void)max_pos;
  if (cfg == nullptr || T <= 0 || cfg->n_q <= 0 || cfg->head_dim <= 0) return 256;
  const size_t parts = part_rows(2);
  return align_up(parts * cfg->head_dim * 4, 256) + align_up(parts * 2 * 4, 256) +
         align_up(kMaxParts * sizeof(int4), 256) +
         align_up(size_t(T) * cfg->n_q * cfg->head_dim * 2, 256);
}

extern "C" beam_status beam_paged_attn(const beam_layer_cfg* cfg, const beam_bf16* q,
                                       const beam_bf16* g, const beam_bf16* gate_bias,
                                       const beam_paged_kv* cache, const int32_t* seq_id,
                                       const int32_t* pos, int T, int max_pos,
                                       const beam_bf16* w_o, beam_bf16* out, void* ws,
                                       size_t ws_bytes, beam_stream_t stream) {
  using namespace beam;
  using namespace beam::paged;
  beam_status stt = check_cfg_attn(cfg);
  if (stt != BEAM_OK) return stt;
  if ((stt = check(cache)) != BEAM_OK) return stt;
  if (cache->n_kv != cfg->n_kv || cache->head_dim != cfg->head_dim || T < 0 || max_pos < 0)
    return BEAM_ERR_INVALID_ARG;
  if (T == 0) return BEAM_OK;
  if (!q || !seq_id || !pos || !out || !ws || (g == nullptr) != (gate_bias == nullptr))
    return BEAM_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16_or_null(g) || !aligned16_or_null(w_o) || !aligned16(out) ||
      (reinterpret_cast<uintptr_t>(ws) & 255u))
    return BEAM_ERR_INVALID_ARG;
  if (!tc::tensor_map_encoder_ready()) return BEAM_ERR_UNSUPPORTED;
  const int D = cfg->head_dim, HD = cfg->n_q * D, G = cfg->n_q / cfg->n_kv, nt = G > 8 ? 2 : 1;
  const int BK = block_keys(cache->dtype, D, nt);
  const int64_t table = int64_t(cache->table_stride) * cache->page_size;
  const int64_t reach = max_pos < table ? max_pos : table;
  int64_t keys = reach;
  if (cache->window > 0 && cache->window < keys) keys = cache->window;
  // most blocks of a pair: a window may begin anywhere in its first block
  const int64_t nb = (keys + BK - 1) / BK + (keys < reach ? 1 : 0);
  const int slice = T < kMaxT ? T : kMaxT;
  if (nb * slice * cfg->n_kv > 1 << 30) return BEAM_ERR_UNSUPPORTED;   // flat block numbers are 32-bit
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  Carver cv{static_cast<char*>(ws), ws_bytes};
  const size_t parts = part_rows(nt);
  Params p{};
  p.part_acc = cv.take<float>(parts * D);
  p.part_ml = cv.take<float>(parts * 2);
  p.join = cv.take<int4>(kMaxParts);
  uint16_t* og = w_o ? cv.take<uint16_t>(size_t(T) * HD) : out;
  if (!cv.ok) return BEAM_ERR_INVALID_ARG;
  p.gate_bias = gate_bias;
  p.c = *cache;
  p.n_q = cfg->n_q;
  p.n_kv = cfg->n_kv;
  p.G = G;
  p.max_pos = max_pos;
  p.shift = log2i(cache->page_size);
  p.sl2 = float(1.4426950408889634 / sqrt(double(D)));
  for (int t0 = 0; t0 < T; t0 += kMaxT) {   // slices in stream order share the workspace
    p.T = T - t0 < kMaxT ? T - t0 : kMaxT;
    p.q = q + size_t(t0) * HD;
    p.g = g ? g + size_t(t0) * HD : nullptr;
    p.og = og + size_t(t0) * HD;
    p.seq_id = seq_id + t0;
    p.pos = pos + t0;
    const int64_t pairs = int64_t(p.T) * cfg->n_kv, blocks = nb * pairs;
    // Pairs stay in one CTA, whose groups share them out, where they have at most four blocks, or
    // eight with enough pairs for every SM: it saves the join's launch, 1.7 us of the host's time.
    // Device time measured, whole against split: BF16, 16 sequences of 256 keys (4 blocks) 8.3
    // against 9.1 us, 64 of 500 (8) 22.2 against 24.2, 1 of 200 (4) 6.7 against 6.4, 4 of 256 7.8 against
    // 6.7 (a call from the host: 7.8 against 9.4); but 4 of 500 12.1 against 8.4, FP8, 16 of 1000 (8)
    // 13.9 against 11.5.
    p.whole = nb <= 4 || (nb <= 8 && 5 * pairs >= nb * max_grid());
    cudaError_t e;
    if (cache->dtype == kFmtBF16) e = launch_fmt<kFmtBF16>(p, pairs, blocks, st);
    else if (cache->dtype == kFmtFP8) e = launch_fmt<kFmtFP8>(p, pairs, blocks, st);
    else e = launch_fmt<kFmtNVFP4>(p, pairs, blocks, st);
    if (e != cudaSuccess) return cuda_status(e);
  }
  if (w_o != nullptr) {
    const cudaError_t ge = o_proj(og, T, HD, w_o, cfg->hidden, out, st);
    if (ge != cudaSuccess) return cuda_status(ge);
  }
  return BEAM_OK;
}
