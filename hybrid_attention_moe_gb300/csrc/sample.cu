// Sampling from logits: temperature, top-k, top-p, min-p and one given uniform number per row.
//
//   w_i = e^((z_i - max z) / t);  tokens in order of z (equal ones by index): the first k; of these the fewest that
//   hold p of their weight; of these the ones with w_i >= min_p;  the first token, by index, at which the kept
//   weights' running sum passes u times their sum
//
// The kept tokens are those in front of a cut (key, index) in that order, so a row needs its maximum, its cuts
// and a running sum. A cluster of CTAs holds a row in shared memory: HBM is read once. Which token a sum
// that meets a border chooses hangs on its last bits, so weights are fixed-point numbers of 64 bits (w = 1 is
// 2^44; relative error near 2^-29): their sums are exact, and the same in every order.
//
// A cut is found from counts: the logits are counted into kBins bins of equal width, and a bin's count bounds its weight
// (that of its two edges times the count). The bins in which the bounds pass the target bracket the cut. A second pass adds
// the exact weights in front of the bracket, lists the logits in it and counts them in finer bins; up to kList are cut
// exactly in shared memory, brackets of more go on with the finer bins, equal logits are counted by index. Top-k starts from a
// bracket of the threads' largest logits instead of a count of all, and where the kept ones fit the list the row ends there.
//
// Measured, us: one row of 201,088 logits 14 (top-k 50), 22 to 69 (top-p, by how flat the row is and where the cut falls), 33 rows
// of 32,003 with top-k 18; 128 rows of 201,088: 45 (greedy: the row's load finds the largest, a pass over shared memory its
// index), 69 (min-p), 93 (top-k), 106 (no rule), 159 to 420 (top-p); 103 MB are 15.2 us of HBM. What bounds it is arithmetic (issue
// 55 %; a greedy row, by reading, its two passes of latency): a weight is 40 instructions, a comparison pass 10 a logit, and a
// row alone has 16 SMs (a cluster) and six exchanges of 2K cycles. The first kernel halved a range of keys 32 times, a pass each:
// one row with top-p took 147 us, 33 with top-k 193, 128 of mixed rules 811 (139 to 150 now). Clusters: 128 rows over 4 / 8 / 16
// CTAs 347 / 314 / 436 us, one row 49 / 31 / 25, 33 rows of 32,003 over 1 / 2 / 4 / 8 / 16: 24 / 20 / 18 / 19 / 33. Bins: 2048 cost
// the exchange 10K cycles, 512 2K.
#include <math.h>

#include "common.cuh"

namespace beam {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kMaxCluster = 16;
constexpr int kMaxChunk = 53248;   // logits of a CTA at most: 208 KB
constexpr int kBins = 512;         // one of a thread
constexpr int kList = 512;         // one of a thread
constexpr int kRounds = 3;         // of counting; what is left then is halved key by key
constexpr float kLeastT = 1e-30f;  // a temperature below it counts as 0
static_assert(kWarps == kMaxCluster && kBins == kThreads && kList == kThreads, "by thread");

struct Params {
  const float* logits;
  const float* u;
  const float* temperature;
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  int32_t* token;
  float* logprob;
  int64_t stride;
  int V, chunk, seg;   // chunk: logits of a CTA; seg: of a warp, a multiple of 128
  // 2^(j/16) * 2^30, rounded. (A parameter: __constant__ memory is the whole library's, and cost every kernel of it 0.1 to 0.2 us a
  // launch; paged writes of 32 tokens took 2.21 us for 2.00.)
  uint32_t table[16] = {1073741824u, 1121280436u, 1170923762u, 1222764986u, 1276901417u, 1333434672u, 1392470869u, 1454120821u,
                        1518500250u, 1585730000u, 1655936265u, 1729250827u, 1805811301u, 1885761398u, 1969251188u, 2056437387u};
};

using u64 = unsigned long long;

__device__ __forceinline__ uint32_t key_of(float z) {
  const uint32_t b = __float_as_uint(z);
  return b ^ (uint32_t(int32_t(b) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float of_key(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k); }

// What is joined over a row: a sum, a count, the smallest and the largest key.
struct Red {
  u64 a;
  uint32_t n, lo, hi, pad;
};
struct Given {
  float t;
  int k;
  float p, mp, u;
  u64 least;   // t log(min_p) in FP64: one lane's work (11K cycles of all threads), while the row is on its way
};
struct Shared {
  Red red[2][kMaxCluster];   // by CTA; two in turn
  Red warp[kWarps];
  u64 seg[kWarps];           // equal logits of each warp's
  u64 more[2][kMaxCluster];  // weights to add to those that reduce left: by CTA, and by the CTA's warps
  u64 total, before;
  u64 scan[2][kWarps];
  uint32_t table[16];        // 2^(j/16) in 2^-30
  Given given;
  int bracket[2], count, tie;
  uint32_t cut_key;
  int cut_index;
};

__device__ __forceinline__ uint32_t ctarank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t remote(const void* p, uint32_t rank) {
  uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(p)), r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
  return r;
}
__device__ __forceinline__ void remote_store(const void* p, uint32_t rank, u64 v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(remote(p, rank)), "l"(v) : "memory");
}
__device__ __forceinline__ void remote_store(const void* p, uint32_t rank, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(remote(p, rank)), "r"(v) : "memory");
}
__device__ __forceinline__ u64 remote_load(const u64* p, uint32_t rank) {
  u64 v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(remote(p, rank)) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t remote_load(const uint32_t* p, uint32_t rank) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(remote(p, rank)) : "memory");
  return v;
}

// The Reds of a warp's lanes joined; every lane has it.
__device__ __forceinline__ Red join(Red v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v.a += __shfl_xor_sync(0xffffffffu, v.a, o);
  v.n = __reduce_add_sync(0xffffffffu, v.n);
  v.lo = __reduce_min_sync(0xffffffffu, v.lo);
  v.hi = __reduce_max_sync(0xffffffffu, v.hi);
  return v;
}
__device__ __forceinline__ Red nothing() { return Red{0, 0, 0xFFFFFFFFu, 0, 0}; }

// One Red of each thread joined over the CTA and, by turns in two buffers, over the cluster (whose CTAs' own stay
// there, and the CTA's warps' in sh->warp): `publish`, a barrier of the cluster (of the CTA, if it is alone), `collect`.
// Every remote access is in front of a barrier of the cluster, so a CTA may leave after any of them.
__device__ __forceinline__ void publish(Shared* sh, int ctas, int& turn, Red v) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  v = join(v);
  __syncthreads();
  if (lane == 0) sh->warp[w] = v;
  __syncthreads();
  turn ^= 1;
  if (w != 0) return;
  v = join(lane < kWarps ? sh->warp[lane] : nothing());
  if (ctas > 1) {
    if (lane < ctas) {
      const Red* to = &sh->red[turn][ctarank()];
      remote_store(&to->a, lane, v.a);
      remote_store(&to->n, lane, v.n);
      remote_store(&to->lo, lane, v.lo);
      remote_store(&to->hi, lane, v.hi);
    }
  } else if (lane == 0) {
    sh->red[turn][0] = v;
  }
}
__device__ __forceinline__ void barrier(int ctas) {
  if (ctas > 1) cluster_sync();
  else __syncthreads();
}
__device__ __forceinline__ Red collect(const Shared* sh, int ctas, int turn) {
  const int lane = threadIdx.x & 31;
  return join(lane < ctas ? sh->red[turn][lane] : nothing());
}
__device__ Red reduce(Shared* sh, int ctas, int& turn, Red v) {
  publish(sh, ctas, turn, v);
  barrier(ctas);
  return collect(sh, ctas, turn);
}

struct Weights {
  float top, ch, cl;   // the largest logit; log2(e) / t in two parts
  const uint32_t* table;
  // e^((z - top) / t) = m 2^-(30 + shift), before what is below 2^-44 is cut off
  __device__ __forceinline__ uint32_t parts(float z, int& shift) const {
    const float dh = z - top, b = dh - z, dl = (z - (dh - b)) - (top + b);   // dh + dl = z - top
    float y = dh * ch;
    float lo = fmaf(dh, ch, -y);   // y + lo = (z - top) log2(e) / t
    lo = fmaf(dh, cl, lo);
    lo = fmaf(dl, ch, lo);
    y = fmaxf(y, -60.f);   // what is below shifts out, whatever lo is; no branch, so that several are under way
    // y = k / 16 + r, 2^r = 1 + r ln 2 + ... (|r| <= 1/32: the fifth term is below 2^-34)
    constexpr float kRound = 12582912.f;
    const float t = fmaf(y, 16.f, kRound);
    const int k = int(__float_as_uint(t)) - int(0x4B400000);
    const float r = fmaf(t - kRound, -0.0625f, y) + lo;
    const float p = r * fmaf(r, fmaf(r, fmaf(r, 0.00961812910762848f, 0.0555041086648216f), 0.240226506959101f), 0.693147180559945f);
    const uint32_t e = table[k & 15];
    shift = -(k >> 4);
    return e + uint32_t(__float2int_rn(p * float(e)));
  }
  // 2^44 e^((z - top) / t)
  __device__ __forceinline__ u64 operator()(float z) const {
    int shift;
    const uint32_t m = parts(z, shift);
    return (static_cast<u64>(m) << 14) >> shift;
  }
};

// s f of f < 1, rounded up or down; 0 of f <= 0 and of NaN.
__device__ __forceinline__ u64 times(u64 s, float f, bool up) {
  if (!(f > 0.f)) return 0;
  const uint32_t b = __float_as_uint(f), e = b >> 23;
  const u64 m = (b & 0x7FFFFFu) | (e != 0 ? 0x800000u : 0u);
  const int shift = 150 - int(max(e, 1u));   // f = m 2^-shift, shift >= 24
  const u64 lo = s * m, hi = __umul64hi(s, m);   // of 88 bits
  u64 x, rest;
  if (shift >= 88) {
    x = 0;
    rest = lo | hi;
  } else if (shift >= 64) {
    x = hi >> (shift - 64);
    rest = lo | (hi & ((u64(1) << (shift - 64)) - 1));
  } else {
    x = hi << (64 - shift) | lo >> shift;
    rest = lo & ((u64(1) << shift) - 1);
  }
  return x + (up && rest != 0);
}

// Tokens in front of a cut: larger keys, and equal ones up to an index.
struct Cut {
  uint32_t key;
  int index;
  __device__ __forceinline__ bool keeps(uint32_t k, int i) const { return k > key || (k == key && i <= index); }
};

__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const __grid_constant__ Params P) {
  extern __shared__ __align__(16) float row[];
  __shared__ Shared sh;
  __shared__ __align__(8) uint32_t hists[2][kBins];   // by turns; later the list's sums in kBins / 2 bins
  __shared__ u64 list[kList], q[kList];           // (key, ~index), of which larger ones are in front: the CTA's, the row's
  pdl_trigger();
  const int ctas = gridDim.x, rank = blockIdx.x, r = blockIdx.y;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int i0 = rank * P.chunk, n = max(0, min(P.chunk, P.V - i0));
  int turn = 0;
  if (threadIdx.x < 16) sh.table[threadIdx.x] = P.table[threadIdx.x];
  if (ctas > 1) cluster_sync();   // the others run
  pdl_wait();
  // ---- the row, its largest logit, and whether it has a distribution; what is given for the row, read once
  if (rank == 0 && w == 0) {
    Given g;
    g.t = P.temperature ? P.temperature[r] : 1.f;
    g.k = P.top_k ? P.top_k[r] : 0;
    g.p = P.top_p ? P.top_p[r] : 1.f;
    g.mp = P.min_p ? P.min_p[r] : 0.f;
    g.u = P.u[r];
    // one lane's, so that all CTAs have the same
    g.t = __shfl_sync(0xffffffffu, g.t, 0);
    g.k = __shfl_sync(0xffffffffu, g.k, 0);
    g.p = __shfl_sync(0xffffffffu, g.p, 0);
    g.mp = __shfl_sync(0xffffffffu, g.mp, 0);
    g.u = __shfl_sync(0xffffffffu, g.u, 0);
    g.least = 0;
    if (g.mp > 0.f) g.least = u64(__double_as_longlong(lane == 0 ? double(g.t) * log(double(g.mp)) : 0.0));
    g.least = __shfl_sync(0xffffffffu, g.least, 0);
    if (ctas == 1) {
      if (lane == 0) sh.given = g;
    } else if (lane < ctas) {
      remote_store(&sh.given.t, lane, __float_as_uint(g.t));
      remote_store(&sh.given.k, lane, uint32_t(g.k));
      remote_store(&sh.given.p, lane, __float_as_uint(g.p));
      remote_store(&sh.given.mp, lane, __float_as_uint(g.mp));
      remote_store(&sh.given.u, lane, __float_as_uint(g.u));
      remote_store(&sh.given.least, lane, g.least);
    }
  }
  const float* src = P.logits + int64_t(r) * P.stride + i0;
  const int n4 = (n + 3) & ~3;
  if (n + int(threadIdx.x) < n4) row[n + threadIdx.x] = -INFINITY;
  Red all = nothing();
  auto take = [&](float x) {
    const float z = x + 0.f;   // -0 is 0
    all.hi = max(all.hi, z != z ? 0xFFFFFFFFu : key_of(z));
    all.n += z > -INFINITY;
    all.lo = min(all.lo, z > -INFINITY ? key_of(z) : 0xFFFFFFFFu);
    return z;
  };
  const bool wide = (reinterpret_cast<uintptr_t>(src) & 15) == 0;   // rows of an odd stride begin anywhere
  const int n16 = wide ? n & ~3 : 0;
#pragma unroll 8
  for (int i = 4 * threadIdx.x; i < n16; i += 4 * kThreads) {
    const float4 z = __ldcs(reinterpret_cast<const float4*>(src + i));
    *reinterpret_cast<float4*>(row + i) = make_float4(take(z.x), take(z.y), take(z.z), take(z.w));
  }
#pragma unroll 16
  for (int i = n16 + threadIdx.x; i < n; i += kThreads) row[i] = take(__ldcs(src + i));
  const uint32_t best_of_mine = all.hi;
  all = reduce(&sh, ctas, turn, all);   // of the logits above -inf
  const uint32_t ktop = all.hi;
  const float ztop = of_key(ktop);
  if (!(ztop > -INFINITY && ztop < INFINITY)) {
    if (rank == 0 && threadIdx.x == 0) {
      flag(BEAM_DEV_BAD_LOGITS);
      P.token[r] = -1;
      if (P.logprob) P.logprob[r] = __uint_as_float(0x7FFFFFFFu);
    }
    return;
  }
  const Given given = sh.given;
  // segments: warp w holds logits [w seg, (w + 1) seg) of the CTA
  const int a = min(n4, w * P.seg), b = min(n4, a + P.seg);
  // f(four logits, the first's index in the CTA) for the warp's, and -inf behind them: by whole warps. Not unrolled: of few
  // logits a cold instruction cache takes most of a pass.
  auto fours = [&](auto f) {
#pragma unroll 1
    for (int i = a + 4 * lane; i - 4 * lane < b; i += 128) {
      float4 z = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
      if (i < b) z = *reinterpret_cast<const float4*>(row + i);
      const float y[4] = {z.x, z.y, z.z, z.w};
      f(y, i);
    }
  };
  if (!(given.t >= kLeastT) || given.k == 1) {
    Red best = nothing();
    fours([&](const float (&z)[4], int i) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (z[e] == ztop) best.lo = min(best.lo, uint32_t(i0 + i + e));
    });
    best = reduce(&sh, ctas, turn, best);
    if (rank == 0 && threadIdx.x == 0) {
      P.token[r] = int(best.lo);
      if (P.logprob) P.logprob[r] = 0.f;
    }
    return;
  }
  // log2(e) / t as a sum of two: the quotient's remainder is exact (FP64 divisions of all threads took 3 us)
  constexpr float kL = 1.44269502162933349609375f, kLrest = 1.92596299112661746887e-8f;
  const float ch = kL / given.t;
  const Weights weight{ztop, ch, (fmaf(-ch, given.t, kL) + kLrest) / given.t, sh.table};

  auto scale_of = [](float width, int bins) { return fminf(float(bins - 1) / width, 1e30f); };
  // The bins, one of each thread, in which the running sums of `most` and of `least` first reach the target (the last if they
  // do not); sh.before: what is in front of the first.
  auto find = [&](u64 most, u64 least, u64 target) {
    const u64 own[2] = {most, least};
    u64 before[2];
    if (threadIdx.x < 2) sh.bracket[threadIdx.x] = kBins - 1;
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      u64 s = own[y];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const u64 z = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += z;
      }
      if (lane == 31) sh.scan[y][w] = s;
      before[y] = s - own[y];
    }
    __syncthreads();
#pragma unroll
    for (int y = 0; y < 2; ++y) {
#pragma unroll
      for (int x = 0; x < kWarps; ++x) before[y] += x < w ? sh.scan[y][x] : 0;
      if (before[y] < target && before[y] + own[y] >= target) {
        sh.bracket[y] = threadIdx.x;
        if (y == 0) sh.before = before[0];
      }
    }
    __syncthreads();
    return make_int2(sh.bracket[0], sh.bracket[1]);
  };
  // What `gather` found of the row, one each of the first threads.
  auto fetch = [&](int m) {
    u64 v = 0;
    if (int(threadIdx.x) < m) {   // the CTAs' lists, end to end
      int at = threadIdx.x, x = 0;
      while (at >= int(sh.red[turn][x].n)) at -= int(sh.red[turn][x++].n);
      v = ctas > 1 ? remote_load(list + at, x) : list[at];
    }
    return v;
  };

  // Key that min-p's kept ones are above.
  auto least_key = [&] {
    const double least = fmin(double(ztop), double(ztop) + __longlong_as_double(static_cast<long long>(given.least)));
    float f = float(least);   // the smallest logit that is not below it
    if (double(f) < least) f = nextafterf(f, INFINITY);
    return key_of(f + 0.f) - 1;
  };
  auto wanted = [&](u64 sum) { return max(u64(1), times(sum, given.p, true)); };
  auto target_of = [&](u64 total) { return given.u >= 1.f ? total - 1 : times(total, given.u, false); };
  auto put = [&](int i, float z, u64 v, u64 total) {
    P.token[r] = i;
    if (!P.logprob) return;
    // near 1 by what is missing, which FP32 then holds to its last bits; else by the weight before it was cut to steps, of which a
    // small one has few
    int shift;
    const double whole = double(weight.parts(z, shift)) * __longlong_as_double((1023ll + 14 - shift) << 52);
    P.logprob[r] = float(v > total / 2 ? log1p(-double(total - v) / double(total)) : log(whole / double(total)));
  };
  Cut cut{0, P.V};   // all
  float zlow = of_key(all.lo);
  // Whether the sums that `reduce` left, with sh.more, are the weights in front of the cut, each CTA's and each warp's.
  bool known = false;
  auto keep_only = [&] {   // the row, from here on
    for (int i = a + lane; i < b; i += 32)
      if (!cut.keeps(key_of(row[i]), i0 + i)) row[i] = -INFINITY;
    zlow = of_key(cut.key);
    cut = Cut{0, P.V};
    __syncthreads();
  };
  // Two cuts: top-k's, by counting, and top-p's, by weight. A cut is the place behind which the sum of f (1, or the weight) over the
  // tokens in front of it, one by one, first reaches a target, which the sum over all does.
#pragma unroll 1
  for (int by_weight = 0; by_weight < 2; ++by_weight) {
    if (by_weight ? given.p >= 1.f : !(given.k > 0 && uint32_t(given.k) < all.n)) continue;   // (-inf weighs nothing)
    auto f = [&](float z) { return by_weight ? weight(z) : u64(1); };
    u64 target = u64(given.k);
    // The bracket: logits zl..zh, counted in bins of y = d s + o, d the distance from the largest; the last has no end. (In one
    // rounding, so that y is monotone and the same in every place.) Below the largest by 32 t a weight is less than
    // 2^-46 and so nothing.
    float zl = by_weight ? fmaxf(zlow, ztop - 32.f * given.t) : zlow, zh = ztop;
    float s = fmaxf(scale_of(ztop - zl, kBins), 1e-37f), o = 0.f;
    auto place = [&](float z, float s, float o) { return fmaf(__fsub_rn(ztop, z), s, o); };
    auto bin = [&](float y) { return int(fmaxf(fminf(y, float(kBins - 1)), 0.f)); };
    uint32_t* hist = hists[0];
    hist[threadIdx.x] = 0;
    __syncthreads();
    if (!by_weight) {
      // The k-th of the threads' largest logits is not above the row's k-th: the logits that are not below its bin hold
      // the kept ones, and are few more
      const float best = of_key(best_of_mine);
      if (best_of_mine != 0 && best > -INFINITY) atomicAdd(hist + bin(place(best, s, o)), 1u);
    } else {
      Red v = nothing();
      fours([&](const float (&z)[4], int) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (z[e] >= zl) atomicAdd(hist + bin(place(z[e], s, o)), 1u);
          v.a += weight(z[e]);
        }
      });
      publish(&sh, ctas, turn, v);   // collected behind the barrier of the counts
    }
    Red own = nothing(), g = own;   // own.a: the thread's in front of the bracket
#pragma unroll 1
    for (int round = 0;; ++round) {
      // ---- the bins in which the cut may lie
      uint32_t h = 0;
      barrier(ctas);
      if (ctas > 1) {
#pragma unroll 8
        for (int x = 0; x < ctas; ++x) h += remote_load(hist + threadIdx.x, x);
      } else {
        h = hist[threadIdx.x];
      }
      if (by_weight && round == 0) target = wanted(collect(&sh, ctas, turn).a);
      hist = hists[(round + 1) & 1];
      hist[threadIdx.x] = 0;
      u64 most = h, least = h;
      if (by_weight && h != 0) {
        // 2^-y at the bin's edges; the errors of y and of the function are below 2^-14 of it, that of a weight is one step
        const float by = ch / s, d0 = (float(threadIdx.x) - o) * by, d1 = threadIdx.x == kBins - 1 ? INFINITY : (float(threadIdx.x + 1) - o) * by;
        most = (u64(fminf(exp2f(-d0) * (1.f + 0x1p-13f), 1.f) * 0x1p44f) + 1) * h;
        least = u64(fmaxf(exp2f(-d1) * (1.f - 0x1p-13f) * 0x1p44f - 1.f, 0.f)) * h;
      }
      if (threadIdx.x == 0) sh.count = 0;
      int2 br = find(most, least, target - g.a);
      if (!by_weight && round == 0) br.x = 0;
      // ---- the sum in front of them; the number, the keys and the list of what lies in them, and its counts in finer bins
      const float first = br.x == 0 ? -INFINITY : float(br.x), end = br.y == kBins - 1 ? NAN : float(br.y + 1);
      const float finer = float(kBins) / float(br.y + 1 - br.x), s1 = s * finer, o1 = (o - float(br.x)) * finer;
      own.n = 0;
      own.lo = 0xFFFFFFFFu;
      own.hi = 0;
      fours([&](const float (&z)[4], int i) {
        bool front[4], any_front = false, any_inside = false, inside[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const bool in = z[e] >= zl && z[e] <= zh;
          const float y = place(z[e], s, o);
          front[e] = in && y < first;
          inside[e] = in && !(y < first) && !(y >= end);
          any_front |= front[e];
          any_inside |= inside[e];
        }
        if (__any_sync(0xffffffffu, any_front)) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const u64 x = f(z[e]);
            own.a += front[e] ? x : 0;
          }
        }
        if (__any_sync(0xffffffffu, any_inside)) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if (!inside[e]) continue;
            const uint32_t key = key_of(z[e]);
            ++own.n;
            own.lo = min(own.lo, key);
            own.hi = max(own.hi, key);
            atomicAdd(hist + bin(place(z[e], s1, o1)), 1u);
          }
          if (*static_cast<volatile int*>(&sh.count) <= kList) {   // a list that is full already is of no use
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const unsigned vote = __ballot_sync(0xffffffffu, inside[e]);
              if (vote == 0) continue;
              int at = 0;
              if (lane == 0) at = atomicAdd(&sh.count, __popc(vote));
              at = __shfl_sync(0xffffffffu, at, 0) + __popc(vote & ((1u << lane) - 1u));
              if (inside[e] && at < kList) list[at] = u64(key_of(z[e])) << 32 | uint32_t(~(i0 + i + e));
            }
          }
        }
      });
      g = reduce(&sh, ctas, turn, own);
      if (g.n <= uint32_t(kList) || g.lo >= g.hi || round == kRounds) break;
      zl = of_key(g.lo);
      zh = of_key(g.hi);
      s = s1;
      o = o1;
    }
    const int m = int(min(g.n, uint32_t(kList) + 1)), at = threadIdx.x;
    if (!by_weight && m <= kList && uint32_t(given.k) <= g.n && g.a == 0) {
      // All that can be kept is in the list: the row's first CTA does the rest there.
      u64 mine = 0;
      if (rank == 0) mine = fetch(m);
      if (ctas > 1) cluster_sync();   // the others' lists were read
      if (rank != 0) return;
      u64* wt = list;
      __syncthreads();
      const u64 v = at < m ? weight(of_key(uint32_t(mine >> 32))) : 0;
      q[at] = mine;
      wt[at] = v;
      __syncthreads();
      u64 before = 0;
      int place = 0;
      if (at < m) {
#pragma unroll 4
        for (int x = 0; x < m; ++x)
          if (q[x] > mine) {
            before += wt[x];
            ++place;
          }
        if (place == given.k - 1) sh.total = before + v;
      }
      __syncthreads();
      bool keep = at < m && place < given.k;
      if (!(given.p >= 1.f)) keep = keep && before < wanted(sh.total);
      if (given.mp > 0.f) keep = keep && uint32_t(mine >> 32) > least_key();
      wt[at] = keep ? v : 0;
      __syncthreads();
      if (keep) {
        u64 total = 0, run = 0;   // of all, and of those of lower indices: the list holds their complements
#pragma unroll 4
        for (int x = 0; x < m; ++x) {
          total += wt[x];
          if (uint32_t(q[x]) > uint32_t(mine)) run += wt[x];
        }
        const u64 goal = target_of(total);
        if (run <= goal && goal < run + v) put(int(~uint32_t(mine)), of_key(uint32_t(mine >> 32)), v, total);
      }
      return;
    }
    if (m <= kList) {
      // The list's sums in finer bins name one; those in it are ordered by comparing all with all.
      const u64 mine = fetch(m);
      const float z = of_key(uint32_t(mine >> 32)), zhi = of_key(g.hi), by_list = scale_of(zhi - of_key(g.lo), kBins / 2);
      const u64 v = at < m ? f(z) : 0;
      const int its = at < m ? int(fminf((zhi - z) * by_list, float(kBins / 2 - 1))) : kBins;
      u64* sums = reinterpret_cast<u64*>(hists[0]);   // the CTAs have read their counts
      hists[0][at] = 0;
      if (at < 2 * kMaxCluster) sh.more[at / kMaxCluster][at % kMaxCluster] = 0;
      if (at == 0) sh.count = 0;
      __syncthreads();
      if (at < m) atomicAdd(sums + its, v);
      __syncthreads();
      const u64 sum = at < kBins / 2 ? sums[at] : 0;
      const int it = find(sum, sum, target - g.a).x;
      if (its == it) q[atomicAdd(&sh.count, 1)] = mine;
      __syncthreads();
      bool keep = its < it;
      if (its == it) {
        const int n2 = sh.count;
        u64 before = g.a + sh.before;
        for (int x = 0; x < n2; ++x)
          if (q[x] > mine) before += (q[x] ^ mine) >> 32 ? f(of_key(uint32_t(q[x] >> 32))) : v;
        keep = before < target;
        if (keep && before + v >= target) {   // one
          sh.cut_key = uint32_t(mine >> 32);
          sh.cut_index = int(~uint32_t(mine));
        }
      }
      if (keep) {
        const int i = int(~uint32_t(mine)), x = i / P.chunk;
        atomicAdd(&sh.more[0][x], v);
        if (x == rank) atomicAdd(&sh.more[1][(i - i0) / P.seg], v);
      }
      __syncthreads();
      cut = Cut{sh.cut_key, sh.cut_index};
      known = by_weight;
      if (!by_weight) keep_only();
      continue;
    }
    // the key, by halves of what is left: the sum of keys >= klo reaches the target, that of keys >= khi does not
    uint32_t klo = g.lo, khi = g.hi + 1;
    u64 above = g.a;
    while (khi - klo > 1) {
      const uint32_t half = klo + (khi - klo) / 2;
      Red v = nothing();
      for (int i = a + lane; i < b; i += 32) {
        const uint32_t key = key_of(row[i]);
        if (key >= half) v.a += f(row[i]);
      }
      v = reduce(&sh, ctas, turn, v);
      if (v.a >= target) {
        klo = half;
      } else {
        khi = half;
        above = v.a;
      }
    }
    // as many of the equal ones as are needed, by index
    const u64 one = f(of_key(klo)), need = one == 0 ? ~0ull : (target - above + one - 1) / one;
    auto equal = [&](int i) { return i < b && key_of(row[i]) == klo; };
    Red count = nothing();
    for (int i = a + lane; i < b; i += 32) count.n += equal(i);
    const uint32_t warps = __reduce_add_sync(0xffffffffu, count.n);
    reduce(&sh, ctas, turn, count);
    if (lane == 0) sh.seg[w] = warps;
    u64 before = __reduce_add_sync(0xffffffffu, lane < rank ? sh.red[turn][lane].n : 0u);   // in CTAs before this one
    __syncthreads();
    for (int x = 0; x < w; ++x) before += sh.seg[x];
    Red last = nothing();
    if (before < need && before + warps >= need)
      for (int i = a + lane; i - lane < b; i += 32) {
        const unsigned vote = __ballot_sync(0xffffffffu, equal(i));
        if (equal(i) && before + __popc(vote & ((2u << lane) - 1u)) == need) last.hi = uint32_t(i0 + i) + 1;
        before += __popc(vote);
      }
    last = reduce(&sh, ctas, turn, last);
    cut = Cut{klo, last.hi == 0 ? P.V : int(last.hi) - 1};
    known = false;
    if (!by_weight) keep_only();
  }
  if (given.mp > 0.f) {
    const uint32_t key = least_key();
    if (key >= cut.key) {
      cut = Cut{key, -1};
      known = false;
    }
  }
  // ---- the kept weights' sums, and the token at which they pass u times their total
  if (!known) {
    if (threadIdx.x < 2 * kMaxCluster) sh.more[threadIdx.x / kMaxCluster][threadIdx.x % kMaxCluster] = 0;
    Red mine = nothing();
    fours([&](const float (&z)[4], int i) {
      bool keep[4], any = false;
#pragma unroll
      for (int e = 0; e < 4; ++e) any |= keep[e] = cut.keeps(key_of(z[e]), i0 + i + e);
      if (__any_sync(0xffffffffu, any)) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const u64 x = weight(z[e]);
          mine.a += keep[e] ? x : 0;
        }
      }
    });
    reduce(&sh, ctas, turn, mine);
  } else if (ctas > 1) {
    cluster_sync();   // the others have read this CTA's list
  }
  u64 before = 0, total = 0;
  for (int x = 0; x < ctas; ++x) {
    if (x == rank) before = total;
    total += sh.red[turn][x].a + sh.more[0][x];
  }
  const u64 cta = sh.red[turn][rank].a + sh.more[0][rank];
  u64 target = target_of(total);
  if (target < before || target >= before + cta) return;
  target -= before;
  auto seg = [&](int x) { return sh.warp[x].a + sh.more[1][x]; };
  int x = 0;
  while (target >= seg(x)) target -= seg(x++);
  // the CTA's warps share the segment
  const int s0 = min(n, x * P.seg), s1 = min(n, s0 + P.seg);
  for (int base = s0; base < s1; base += kThreads) {
    const int i = base + threadIdx.x;
    const u64 v = i < s1 && cut.keeps(key_of(row[i]), i0 + i) ? weight(row[i]) : 0;
    u64 run = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const u64 y = __shfl_up_sync(0xffffffffu, run, o);
      if (lane >= o) run += y;
    }
    __syncthreads();
    if (lane == 31) sh.scan[0][w] = run;
    __syncthreads();
    u64 sums = 0;
    for (int y = 0; y < kWarps; ++y) {
      if (y < w) run += sh.scan[0][y];
      sums += sh.scan[0][y];
    }
    if (run > target && run - v <= target) put(i0 + i, row[i], v, total);
    if (target < sums) break;
    target -= sums;
  }
}

}  // namespace
}  // namespace beam

extern "C" beam_status beam_sample(const float* logits, int64_t row_stride, int T, int V, const float* u,
                                   const float* temperature, const int32_t* top_k, const float* top_p,
                                   const float* min_p, int32_t* token, float* logprob, beam_stream_t stream) {
  using namespace beam;
  if (T < 0 || V <= 0 || row_stride < V) return BEAM_ERR_INVALID_ARG;
  if (T == 0) return BEAM_OK;
  if (!logits || !u || !token) return BEAM_ERR_INVALID_ARG;
  if (V > kMaxCluster * kMaxChunk || T > 65535) return BEAM_ERR_UNSUPPORTED;
  int ctas = 1;
  while (ctas < kMaxCluster && (V + ctas - 1) / ctas > kMaxChunk / 2) ctas *= 2;
  while (ctas < kMaxCluster && int64_t(T) * ctas * 2 <= num_sms_cached() && V / ctas > 4096) ctas *= 2;
  Params p{logits, u, temperature, top_k, top_p, min_p, token, logprob, row_stride, V, 0, 0};
  p.chunk = ((V + ctas - 1) / ctas + 3) / 4 * 4;
  p.seg = ((p.chunk + kWarps - 1) / kWarps + 127) / 128 * 128;
  const size_t smem = size_t(p.chunk) * 4;
  cudaError_t e = cudaFuncSetAttribute(sample_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxChunk * 4);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(sample_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return cuda_status(e);
  return cuda_status(launch_pdl_cluster(sample_kernel, dim3(ctas, T), dim3(kThreads), smem,
                                        reinterpret_cast<cudaStream_t>(stream), ctas, p));
}
