// Sampling from logits: temperature, top-k, top-p, min-p and one given uniform number per row.
//
//   w_i = e^((z_i - max z) / t);  tokens in order of z (equal ones by index): the first k; of these the fewest that
//   hold p of their weight; of these the ones with w_i >= min_p;  the first token, by index, at which the kept
//   weights' running sum passes u times their sum
//
// The kept tokens are those in front of a cut (key, index) in that order, so a row needs its maximum, the cut
// and a running sum. A cluster of CTAs holds a row in shared memory: HBM is read once. Which token a sum
// that meets a border chooses hangs on its last bits, so weights are fixed-point numbers of 64 bits (w = 1 is
// 2^44; relative error near 2^-29): their sums are exact, and the same in every order.
#include <math.h>

#include "common.cuh"

namespace beam {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kMaxCluster = 16;
constexpr int kMaxChunk = 53248;   // logits of a CTA at most: 208 KB
constexpr float kLeastT = 1e-30f;  // a temperature below it counts as 0

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
  int V, chunk, seg;   // chunk: logits of a CTA; seg: of a warp, a multiple of 32
};

__device__ __forceinline__ uint32_t key_of(float z) {
  const uint32_t b = __float_as_uint(z);
  return b ^ (uint32_t(int32_t(b) >> 31) | 0x80000000u);
}

struct Shared {
  unsigned long long sums[2][kMaxCluster];     // a reduction's partials, by CTA; two in turn
  unsigned long long warp[kWarps];
  unsigned long long seg[kWarps];              // kept weight of each warp's logits
  unsigned long long result;
  uint32_t table[16];                          // 2^(j/16) in 2^-30
};

__device__ __forceinline__ uint32_t ctarank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void remote_store(const void* p, uint32_t rank, unsigned long long v) {
  uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(p)), r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(r), "l"(v) : "memory");
}

struct Add {
  __device__ unsigned long long operator()(unsigned long long a, unsigned long long b) const { return a + b; }
};
struct Max {
  __device__ unsigned long long operator()(unsigned long long a, unsigned long long b) const { return a > b ? a : b; }
};
struct Min {
  __device__ unsigned long long operator()(unsigned long long a, unsigned long long b) const { return a < b ? a : b; }
};

// One number of each thread joined over the CTA and, by turns in two buffers, over the cluster. Every remote
// store is in front of a barrier of the cluster, so a CTA may leave after any of them.
template <class Op>
__device__ unsigned long long reduce(Shared* sh, int ctas, int& turn, unsigned long long v, Op op) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, o));
  __syncthreads();
  if (lane == 0) sh->warp[w] = v;
  __syncthreads();
  v = sh->warp[lane % kWarps];
#pragma unroll
  for (int o = kWarps / 2; o > 0; o >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, o));
  if (ctas > 1) {
    if (int(threadIdx.x) < ctas) remote_store(&sh->sums[turn][ctarank()], threadIdx.x, v);
    cluster_sync();
    v = sh->sums[turn][0];
    for (int c = 1; c < ctas; ++c) v = op(v, sh->sums[turn][c]);
    turn ^= 1;
  }
  return v;
}

struct Weights {
  float top, ch, cl;   // the largest logit; log2(e) / t in two parts
  const uint32_t* table;
  // 2^44 e^((z - top) / t)
  __device__ __forceinline__ unsigned long long operator()(float z) const {
    const float dh = z - top, b = dh - z, dl = (z - (dh - b)) - (top + b);   // dh + dl = z - top
    const float y = dh * ch;
    if (!(y > -64.f)) return 0;
    float lo = fmaf(dh, ch, -y);   // y + lo = (z - top) log2(e) / t
    lo = fmaf(dh, cl, lo);
    lo = fmaf(dl, ch, lo);
    // y = k / 16 + r, 2^r = 1 + r ln 2 + ... (|r| <= 1/32: the fifth term is below 2^-34)
    constexpr float kRound = 12582912.f;
    const float t = fmaf(y, 16.f, kRound);
    const int k = int(__float_as_uint(t)) - int(0x4B400000);
    const float r = fmaf(t - kRound, -0.0625f, y) + lo;
    const float p = r * fmaf(r, fmaf(r, fmaf(r, 0.00961812910762848f, 0.0555041086648216f), 0.240226506959101f), 0.693147180559945f);
    const uint32_t e = table[k & 15];
    const uint32_t m = e + uint32_t(__float2int_rn(p * float(e)));
    return (static_cast<unsigned long long>(m) << 14) >> (-(k >> 4));
  }
};

// Tokens in front of a cut: larger keys, and equal ones up to an index.
struct Cut {
  uint32_t key;
  int index;
  __device__ __forceinline__ bool keeps(uint32_t k, int i) const { return k > key || (k == key && i <= index); }
};

__global__ void __launch_bounds__(kThreads) sample_kernel(const Params P) {
  pdl_trigger();
  pdl_wait();
  extern __shared__ __align__(16) float row[];
  __shared__ Shared sh;
  const int ctas = gridDim.x, rank = blockIdx.x, r = blockIdx.y;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int i0 = rank * P.chunk, n = max(0, min(P.chunk, P.V - i0));
  int turn = 0;
  if (threadIdx.x < 16) {
    const double x = exp2(double(threadIdx.x) / 16.0);
    sh.table[threadIdx.x] = uint32_t(x * 1073741824.0 + 0.5);
  }
  if (ctas > 1) cluster_sync();   // the others run
  // ---- the row, its maximum, and whether it has a distribution
  const float* src = P.logits + int64_t(r) * P.stride + i0;
  unsigned long long top = 0;
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const float z = src[i] + 0.f;   // -0 is 0
    row[i] = z;
    const unsigned long long k = z != z ? 0xFFFFFFFFu : key_of(z);
    top = max(top, k);
  }
  top = reduce(&sh, ctas, turn, top, Max());
  const float t = P.temperature ? P.temperature[r] : 1.f;
  const int k = P.top_k ? P.top_k[r] : 0;
  const uint32_t ktop = uint32_t(top);
  const float ztop = __uint_as_float(ktop & 0x80000000u ? ktop ^ 0x80000000u : ~ktop);
  if (!(ztop > -INFINITY && ztop < INFINITY)) {
    if (rank == 0 && threadIdx.x == 0) {
      flag(BEAM_DEV_BAD_LOGITS);
      P.token[r] = -1;
      if (P.logprob) P.logprob[r] = __uint_as_float(0x7FFFFFFFu);
    }
    return;
  }
  // segments: warp w holds logits [w seg, (w + 1) seg) of the CTA
  const int a = min(n, w * P.seg), b = min(n, a + P.seg);
  auto sum = [&](auto f) {   // over the row, of f(logit, index)
    unsigned long long s = 0;
    for (int i = a + lane; i < b; i += 32) s += f(row[i], i0 + i);
    return reduce(&sh, ctas, turn, s, Add());
  };
  if (!(t >= kLeastT) || k == 1) {
    unsigned long long best = ~0ull;
    for (int i = a + lane; i < b; i += 32)
      if (row[i] == ztop) best = min(best, static_cast<unsigned long long>(i0 + i));
    best = reduce(&sh, ctas, turn, best, Min());
    if (rank == 0 && threadIdx.x == 0) {
      P.token[r] = int(best);
      if (P.logprob) P.logprob[r] = 0.f;
    }
    return;
  }
  const double c = 1.4426950408889634 / double(t);
  const Weights weight{ztop, float(c), float(c - double(float(c))), sh.table};

  // The cut behind which the sum of f over the tokens in front of it, one by one, first reaches `target`; f
  // is a function of the logit, and only tokens in front of `in` count.
  auto cut_at = [&](auto f, const Cut& in, unsigned long long target) {
    uint32_t lo = in.key, hi = ktop + 1;   // the sum of keys >= lo reaches it, that of keys >= hi does not
    while (hi - lo > 1) {
      const uint32_t mid = lo + (hi - lo) / 2;
      const unsigned long long s = sum([&](float z, int i) {
        const uint32_t key = key_of(z);
        return key >= mid && in.keeps(key, i) ? f(z) : 0ull;
      });
      if (s >= target) lo = mid;
      else hi = mid;
    }
    const unsigned long long above = sum([&](float z, int i) {
      const uint32_t key = key_of(z);
      return key > lo && in.keeps(key, i) ? f(z) : 0ull;
    });
    const float z = __uint_as_float(lo & 0x80000000u ? lo ^ 0x80000000u : ~lo);
    const unsigned long long each = f(z), need = above >= target || each == 0 ? 0 : (target - above + each - 1) / each;
    int first = -1, last = in.key == lo ? in.index : P.V - 1;   // as many of the equal ones as are needed
    while (last - first > 1) {
      const int mid = first + (last - first) / 2;
      const unsigned long long s = sum([&](float z, int i) { return key_of(z) == lo && i <= mid ? 1ull : 0ull; });
      if (s >= need) last = mid;
      else first = mid;
    }
    return Cut{lo, last};
  };

  Cut cut{0, P.V};   // all
  if (k > 0 && k < P.V) cut = cut_at([](float) { return 1ull; }, cut, k);
  const float p = P.top_p ? P.top_p[r] : 1.f;
  if (!(p >= 1.f)) {
    const unsigned long long all = sum([&](float z, int i) { return cut.keeps(key_of(z), i) ? weight(z) : 0ull; });
    const double want = ceil(double(all) * double(fmaxf(p, 0.f)));
    cut = cut_at(weight, cut, max(1ull, static_cast<unsigned long long>(want)));
  }
  const float mp = P.min_p ? P.min_p[r] : 0.f;
  if (mp > 0.f) {
    const double least = fmin(double(ztop), double(ztop) + double(t) * log(double(mp)));
    float f = float(least);   // the smallest logit that is not below it
    if (double(f) < least) f = nextafterf(f, INFINITY);
    const uint32_t key = key_of(f + 0.f) - 1;
    if (key >= cut.key) cut = Cut{key, -1};
  }
  // ---- the kept weights' sums, and the token at which they pass u times their total
  unsigned long long mine = 0;
  for (int i = a + lane; i < b; i += 32)
    if (cut.keeps(key_of(row[i]), i0 + i)) mine += weight(row[i]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
  if (lane == 0) sh.seg[w] = mine;
  __syncthreads();
  unsigned long long cta = 0;
  for (int x = 0; x < kWarps; ++x) cta += sh.seg[x];
  unsigned long long before = 0, total = cta;
  if (ctas > 1) {
    if (int(threadIdx.x) < ctas) remote_store(&sh.sums[turn][rank], threadIdx.x, cta);
    cluster_sync();
    total = 0;
    for (int x = 0; x < ctas; ++x) {
      if (x < rank) before += sh.sums[turn][x];
      total += sh.sums[turn][x];
    }
  }
  const float uu = P.u[r];
  unsigned long long target = uu > 0.f ? static_cast<unsigned long long>(double(uu) * double(total)) : 0;
  target = min(target, total - 1);
  if (target < before || target >= before + cta) return;
  target -= before;
  int x = 0;
  while (target >= sh.seg[x]) target -= sh.seg[x++];
  // the CTA's warps share the segment
  const int s0 = min(n, x * P.seg), s1 = min(n, s0 + P.seg);
  for (int base = s0; base < s1; base += kThreads) {
    const int i = base + threadIdx.x;
    const unsigned long long v = i < s1 && cut.keeps(key_of(row[i]), i0 + i) ? weight(row[i]) : 0;
    unsigned long long run = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned long long y = __shfl_up_sync(0xffffffffu, run, o);
      if (lane >= o) run += y;
    }
    __syncthreads();
    if (lane == 31) sh.warp[w] = run;
    __syncthreads();
    unsigned long long all = 0;
    for (int y = 0; y < kWarps; ++y) {
      if (y < w) run += sh.warp[y];
      all += sh.warp[y];
    }
    if (run > target && run - v <= target) {
      P.token[r] = i0 + i;
      // near 1 by what is missing, which FP32 then holds to its last bits
      if (P.logprob)
        P.logprob[r] = float(v > total / 2 ? log1p(-double(total - v) / double(total)) : log(double(v) / double(total)));
    }
    if (target < all) break;
    target -= all;
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
  p.seg = ((p.chunk + kWarps - 1) / kWarps + 31) / 32 * 32;
  const size_t smem = size_t(p.chunk) * 4;
  cudaError_t e = cudaFuncSetAttribute(sample_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxChunk * 4);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(sample_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return cuda_status(e);
  return cuda_status(launch_pdl_cluster(sample_kernel, dim3(ctas, T), dim3(kThreads), smem,
                                        reinterpret_cast<cudaStream_t>(stream), ctas, p));
}
