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
// (that of its two edges times the count). The bins in which the bounds pass the target bracket the cut (top-k: one bin; top-p: about
// 1 % of the weight). One pass adds the exact weights in front of the bracket and lists the logits in it; up to kList are
// ordered by comparing all with all. Brackets of more are counted again, over their keys; equal logits are counted by index.
#include <math.h>

#include "common.cuh"

namespace beam {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kMaxCluster = 16;
constexpr int kMaxChunk = 53248;   // logits of a CTA at most: 208 KB
constexpr int kBins = 512;         // one of a thread
constexpr int kList = 256;
constexpr int kRounds = 3;         // of counting; what is left then is halved key by key
constexpr float kLeastT = 1e-30f;  // a temperature below it counts as 0
static_assert(kWarps == kMaxCluster && kBins == kThreads, "by thread");

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
};
struct Shared {
  Red red[2][kMaxCluster];   // by CTA; two in turn
  Red warp[kWarps];
  u64 seg[kWarps];           // equal logits of each warp's
  u64 more[2][kMaxCluster];  // weights to add to those that reduce left: by CTA, and by the CTA's warps
  u64 total;
  u64 scan[2][kWarps];
  uint32_t table[16];        // 2^(j/16) in 2^-30
  Given given;
  int bracket[2], count, tie;
  uint32_t cut_key;
  int cut_index;
};
// 2^(j/16) * 2^30, rounded
__constant__ uint32_t kTable[16] = {1073741824u, 1121280436u, 1170923762u, 1222764986u, 1276901417u, 1333434672u,
                                    1392470869u, 1454120821u, 1518500250u, 1585730000u, 1655936265u, 1729250827u,
                                    1805811301u, 1885761398u, 1969251188u, 2056437387u};

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
// there, and the CTA's warps' in sh->warp). Every remote access is in front of a barrier of the cluster, so a CTA may leave after any of them.
__device__ Red reduce(Shared* sh, int ctas, int& turn, Red v) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  v = join(v);
  __syncthreads();
  if (lane == 0) sh->warp[w] = v;
  __syncthreads();
  v = join(lane < kWarps ? sh->warp[lane] : nothing());
  turn ^= 1;
  if (ctas > 1) {
    if (int(threadIdx.x) < ctas) {
      const Red* to = &sh->red[turn][ctarank()];
      remote_store(&to->a, threadIdx.x, v.a);
      remote_store(&to->n, threadIdx.x, v.n);
      remote_store(&to->lo, threadIdx.x, v.lo);
      remote_store(&to->hi, threadIdx.x, v.hi);
    }
    cluster_sync();
    v = join(lane < ctas ? sh->red[turn][lane] : nothing());
  } else {
    if (threadIdx.x == 0) sh->red[turn][0] = v;
    __syncthreads();
  }
  return v;
}

struct Weights {
  float top, ch, cl;   // the largest logit; log2(e) / t in two parts
  const uint32_t* table;
  // 2^44 e^((z - top) / t)
  __device__ __forceinline__ u64 operator()(float z) const {
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
    const uint32_t m = e + uint32_t(__float2int_rn(p * float(e)));
    return (static_cast<u64>(m) << 14) >> (-(k >> 4));
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

__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const Params P) {
  extern __shared__ __align__(16) float row[];
  __shared__ Shared sh;
  __shared__ uint32_t hist[kBins];
  __shared__ u64 list[kList];             // the CTA's (key, ~index): larger ones are in front
  __shared__ u64 q[kList], wt[kList];     // the row's, and f of them
  pdl_trigger();
  const int ctas = gridDim.x, rank = blockIdx.x, r = blockIdx.y;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int i0 = rank * P.chunk, n = max(0, min(P.chunk, P.V - i0));
  int turn = 0;
  if (threadIdx.x < 16) sh.table[threadIdx.x] = kTable[threadIdx.x];
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
    if (ctas == 1) {
      if (lane == 0) sh.given = g;
    } else if (lane < ctas) {
      remote_store(&sh.given.t, lane, __float_as_uint(g.t));
      remote_store(&sh.given.k, lane, uint32_t(g.k));
      remote_store(&sh.given.p, lane, __float_as_uint(g.p));
      remote_store(&sh.given.mp, lane, __float_as_uint(g.mp));
      remote_store(&sh.given.u, lane, __float_as_uint(g.u));
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
  auto fours = [&](auto f) {   // f(four logits, first index in the CTA) for the warp's, and -inf behind them: by whole warps
#pragma unroll 2
    for (int i = a + 4 * lane; i - 4 * lane < b; i += 128) {
      float4 z = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
      if (i < b) z = *reinterpret_cast<const float4*>(row + i);
      const float y[4] = {z.x, z.y, z.z, z.w};
      f(y, i);
    }
  };
  auto each = [&](auto f) {   // f(logit, index in the CTA)
    fours([&](const float (&z)[4], int i) {
#pragma unroll
      for (int e = 0; e < 4; ++e) f(z[e], i + e);
    });
  };
  if (!(given.t >= kLeastT) || given.k == 1) {
    Red best = nothing();
    each([&](float z, int i) {
      if (z == ztop) best.lo = min(best.lo, uint32_t(i0 + i));
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

  // Logits counted by bin: f(logit, index) is the bin, or kBins: none.
  auto count = [&](auto f) {
    hist[threadIdx.x] = 0;
    __syncthreads();
    each([&](float z, int i) {
      const int x = f(z, i);
      if (x < kBins) atomicAdd(hist + x, 1u);
    });
  };
  // The first and the last bin in which the cut may lie, `target` beyond what is in front of bin 0; edges(bin, most, least): bounds of a
  // logit's weight there.
  auto bracket = [&](auto edges, u64 target) {
    if (threadIdx.x < 2) sh.bracket[threadIdx.x] = kBins - 1;
    uint32_t h = 0;
    if (ctas > 1) {
      cluster_sync();
#pragma unroll 8
      for (int x = 0; x < ctas; ++x) h += remote_load(hist + threadIdx.x, x);
    } else {
      __syncthreads();
      h = hist[threadIdx.x];
    }
    u64 run[2] = {0, 0};
    if (h != 0) {
      edges(int(threadIdx.x), run[0], run[1]);
      run[0] *= h;
      run[1] *= h;
    }
    u64 before[2];
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      u64 s = run[y];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const u64 z = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += z;
      }
      if (lane == 31) sh.scan[y][w] = s;
      before[y] = s - run[y];
    }
    __syncthreads();
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      for (int x = 0; x < w; ++x) before[y] += sh.scan[y][x];
      if (before[y] < target && before[y] + run[y] >= target) sh.bracket[y] = threadIdx.x;
    }
    __syncthreads();
    return make_int2(sh.bracket[0], sh.bracket[1]);
  };
  // Joined over the row: the sum of f in front of a bracket, and the number and keys of what lies in it, the first kList of
  // which the CTA lists. where(logit, key): -1 in front, 0 inside, 1 behind.
  auto gather = [&](auto f, const Cut& in, auto where) {
    if (threadIdx.x == 0) sh.count = 0;
    __syncthreads();
    Red v = nothing();
    fours([&](const float (&z)[4], int i) {
      bool front[4], any_front = false, in_any = false, inside[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t key = key_of(z[e]);
        const bool valid = z[e] > -INFINITY && in.keeps(key, i0 + i + e);
        const int x = where(z[e], key);
        front[e] = valid && x < 0;
        inside[e] = valid && x == 0;
        any_front |= front[e];
        in_any |= inside[e];
      }
      if (__any_sync(0xffffffffu, any_front)) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const u64 y = f(z[e]);
          v.a += front[e] ? y : 0;
        }
      }
      if (__any_sync(0xffffffffu, in_any)) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t key = key_of(z[e]);
          const unsigned vote = __ballot_sync(0xffffffffu, inside[e]);
          if (vote == 0) continue;
          int at = 0;
          if (lane == 0) at = atomicAdd(&sh.count, __popc(vote));
          at = __shfl_sync(0xffffffffu, at, 0) + __popc(vote & ((1u << lane) - 1u));
          if (inside[e]) {
            ++v.n;
            v.lo = min(v.lo, key);
            v.hi = max(v.hi, key);
            if (at < kList) list[at] = u64(key) << 32 | uint32_t(~(i0 + i + e));
          }
        }
      }
    });
    return reduce(&sh, ctas, turn, v);
  };
  // What `reduce` left of the CTAs before this one: their counts.
  auto counted_before = [&] {
    const uint32_t x = lane < rank ? sh.red[turn][lane].n : 0u;
    return __reduce_add_sync(0xffffffffu, x);
  };

  // Bins of equal width from a logit down; the last has no end.
  auto bin_of = [&](float from, float z, float scale) { return int(fminf((from - z) * scale, float(kBins - 1))); };
  // -1, 0 or 1: in front of bins x.x..x.y, in them, behind them; without the bin
  auto against = [&](float from, float z, float scale, int2 x) {
    const float y = (from - z) * scale;   // a NaN (0 times infinity) is of the last bin, as in bin_of
    return y < float(x.x) ? -1 : int(x.y < kBins - 1 && !(y < float(x.y + 1)));
  };
  auto scale_of = [](float width) { return fminf(float(kBins - 1) / width, 1e30f); };
  // What `gather` found of the row, in q, with f of it in wt.
  auto fetch = [&](auto f, int m) {
    if (int(threadIdx.x) < m) {   // the CTAs' lists, end to end
      int at = threadIdx.x, x = 0;
      while (at >= int(sh.red[turn][x].n)) at -= int(sh.red[turn][x++].n);
      const u64 v = ctas > 1 ? remote_load(list + at, x) : list[at];
      q[threadIdx.x] = v;
      wt[threadIdx.x] = f(of_key(uint32_t(v >> 32)));
    }
  };
  // The cut behind which the sum of f over the tokens in front of it, one by one, first reaches `target`, which the sum
  // over all does. f is a function of the logit; only tokens in front of `in` count. g: what `gather` found of a
  // bracket. edges(d0, d1, most, least): bounds of f from distance d0 below the largest to d1. `known`: whether the sums
  // of f that `reduce` left, with sh.more, are those of the tokens in front of the cut, each CTA's and each warp's.
  bool known = false;
  auto bins = [&](auto edges, float off, float scale, u64 target) {
    return bracket(
        [&](int x, u64& most, u64& least) {
          edges(off + float(x) / scale, x == kBins - 1 ? INFINITY : off + float(x + 1) / scale, most, least);
        },
        target);
  };
  auto cut_at = [&](auto f, const Cut& in, u64 target, Red g, auto edges) {
    for (int round = 0; round < kRounds && g.n > uint32_t(kList) && g.lo < g.hi; ++round) {
      const uint32_t lo = g.lo, hi = g.hi;
      const float from = of_key(hi), scale = scale_of(from - of_key(lo));
      auto inside = [&](uint32_t key, int i) { return key >= lo && key <= hi && in.keeps(key, i0 + i); };
      count([&](float z, int i) { return inside(key_of(z), i) ? bin_of(from, z, scale) : kBins; });
      const int2 br = bins(edges, ztop - from, scale, target - g.a);
      g = gather(f, in, [&](float z, uint32_t key) {
        return key > hi ? -1 : key < lo ? 1 : against(from, z, scale, br);
      });
    }
    if (g.n <= uint32_t(kList)) {
      const int m = int(g.n);
      fetch(f, m);
      if (threadIdx.x < 2 * kMaxCluster) sh.more[threadIdx.x / kMaxCluster][threadIdx.x % kMaxCluster] = 0;
      __syncthreads();
      if (int(threadIdx.x) < m) {
        const u64 mine = q[threadIdx.x];
        u64 before = g.a;
#pragma unroll 4
        for (int x = 0; x < m; ++x)
          if (q[x] > mine) before += wt[x];
        if (before < target) {
          const int i = int(~uint32_t(mine)), x = i / P.chunk;
          atomicAdd(&sh.more[0][x], wt[threadIdx.x]);
          if (x == rank) atomicAdd(&sh.more[1][(i - i0) / P.seg], wt[threadIdx.x]);
          if (before + wt[threadIdx.x] >= target) {   // one
            sh.cut_key = uint32_t(mine >> 32);
            sh.cut_index = i;
          }
        }
      }
      __syncthreads();
      known = true;
      return Cut{sh.cut_key, sh.cut_index};
    }
    // the key, by halves of what is left
    uint32_t lo = g.lo, hi = g.hi + 1;   // the sum of keys >= lo reaches it, that of keys >= hi does not
    u64 above = g.a;
    while (hi - lo > 1) {
      const uint32_t half = lo + (hi - lo) / 2;
      Red s = nothing();
      each([&](float z, int i) {
        const uint32_t key = key_of(z);
        if (key >= half && in.keeps(key, i0 + i)) s.a += f(z);
      });
      s = reduce(&sh, ctas, turn, s);
      if (s.a >= target) {
        lo = half;
      } else {
        hi = half;
        above = s.a;
      }
    }
    // as many of the equal ones as are needed, by index
    const u64 one = f(of_key(lo)), need = one == 0 ? ~0ull : (target - above + one - 1) / one;
    auto equal = [&](float z, int i) { return key_of(z) == lo && in.keeps(lo, i0 + i); };
    Red s = nothing();
    each([&](float z, int i) { s.n += equal(z, i); });
    const uint32_t warps = __reduce_add_sync(0xffffffffu, s.n);
    s = reduce(&sh, ctas, turn, s);
    if (lane == 0) sh.seg[w] = warps;
    u64 before = counted_before();
    __syncthreads();
    for (int x = 0; x < w; ++x) before += sh.seg[x];
    Red at = nothing();
    if (before < need && before + warps >= need)
      for (int i = a + lane; i - lane < b; i += 32) {
        const bool hit = i < b && equal(row[i], i);
        const unsigned vote = __ballot_sync(0xffffffffu, hit);
        if (hit && before + __popc(vote & ((2u << lane) - 1u)) == need) at.hi = uint32_t(i0 + i) + 1;
        before += __popc(vote);
      }
    at = reduce(&sh, ctas, turn, at);
    return Cut{lo, at.hi == 0 ? P.V : int(at.hi) - 1};
  };

  // Key that min-p's kept ones are above.
  auto least_key = [&] {
    const double least = fmin(double(ztop), double(ztop) + double(given.t) * log(double(given.mp)));
    float f = float(least);   // the smallest logit that is not below it
    if (double(f) < least) f = nextafterf(f, INFINITY);
    return key_of(f + 0.f) - 1;
  };
  auto wanted = [&](u64 sum) { return max(u64(1), times(sum, given.p, true)); };
  auto target_of = [&](u64 total) { return given.u >= 1.f ? total - 1 : times(total, given.u, false); };
  auto put = [&](int i, u64 v, u64 total) {
    P.token[r] = i;
    // near 1 by what is missing, which FP32 then holds to its last bits
    if (P.logprob)
      P.logprob[r] = float(v > total / 2 ? log1p(-double(total - v) / double(total)) : log(double(v) / double(total)));
  };
  Cut cut{0, P.V};   // all
  const float zlow = of_key(all.lo);
  if (given.k > 0 && uint32_t(given.k) < all.n) {   // logits of -inf weigh nothing
    // The k-th of the threads' largest logits is not above the row's k-th: those that are not below its bin hold the
    // kept ones, and are few more
    const float scale = scale_of(ztop - zlow), best = of_key(best_of_mine);
    hist[threadIdx.x] = 0;
    __syncthreads();
    if (best_of_mine != 0 && best > -INFINITY) atomicAdd(hist + bin_of(ztop, best, scale), 1u);
    auto one = [](float) { return u64(1); };
    auto ones = [](float, float, u64& most, u64& least) { most = least = 1; };
    const int last = bins(ones, 0.f, scale, u64(given.k)).y;
    const Red g = gather(one, cut, [&](float z, uint32_t) { return against(ztop, z, scale, make_int2(0, last)); });
    if (g.n <= uint32_t(kList)) {
      // All that can be kept is in the list: the row's first CTA does the rest there.
      const int m = int(g.n), at = threadIdx.x;
      if (rank == 0) fetch(weight, m);
      if (ctas > 1) cluster_sync();   // the others' lists were read
      if (rank != 0) return;
      __syncthreads();
      const u64 mine = at < m ? q[at] : 0, v = at < m ? wt[at] : 0;
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
      if (at < m) wt[at] = keep ? v : 0;
      __syncthreads();
      if (keep) {
        u64 total = 0, run = 0;   // of all, and of those of lower indices: the list holds their complements
#pragma unroll 4
        for (int x = 0; x < m; ++x) {
          total += wt[x];
          if (uint32_t(q[x]) > uint32_t(mine)) run += wt[x];
        }
        const u64 target = target_of(total);
        if (run <= target && target < run + v) put(int(~uint32_t(mine)), v, total);
      }
      return;
    }
    cut = cut_at(one, cut, u64(given.k), g, ones);
    known = false;
  }
  if (!(given.p >= 1.f)) {
    // below the largest by 32 t a weight is less than 2^-46 and so nothing
    const float far = 32.f * given.t;
    const float scale = scale_of(fminf(ztop - (cut.key == 0 ? zlow : of_key(cut.key)), far));
    Red v = nothing();
    count([&](float z, int i) {
      const u64 x = cut.keeps(key_of(z), i0 + i) ? weight(z) : 0;
      v.a += x;
      return x != 0 ? bin_of(ztop, z, scale) : kBins;
    });
    const u64 want = wanted(reduce(&sh, ctas, turn, v).a);
    auto edges = [&](float d0, float d1, u64& most, u64& least) {
      // the errors of y and of the function are below 2^-14 of the weight, that of its fixed point is one step
      most = u64(fminf(exp2f(-d0 * ch) * (1.f + 0x1p-13f), 1.f) * 0x1p44f) + 1;
      least = u64(fmaxf(exp2f(-d1 * ch) * (1.f - 0x1p-13f) * 0x1p44f - 1.f, 0.f));
    };
    const int2 br = bins(edges, 0.f, scale, want);
    const Red g = gather(weight, cut, [&](float z, uint32_t) {
      const int x = against(ztop, z, scale, br);
      return x == 0 && ztop - z >= far ? 1 : x;
    });
    cut = cut_at(weight, cut, want, g, edges);
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
    each([&](float z, int i) {
      if (cut.keeps(key_of(z), i0 + i)) mine.a += weight(z);
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
    if (run > target && run - v <= target) put(i0 + i, v, total);
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
