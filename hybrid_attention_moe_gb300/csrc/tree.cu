// Bookkeeping of a drafted tree: masks and positions from the parents, the walk along the sampled tokens,
// and the move of the accepted rows to the front of the tree's slots.
//
// All are bound by a launch and a few dependent loads. A warp takes a sequence's up to 64 nodes, two a lane.
// Measured in a graph: plan, accept and keep of one tree of 16 nodes 5.4 us together; plan, accept and six layers' keep of
// 64 trees of up to 64 nodes over FP8 pages 20.2 us (from the host 72: eight calls of 9 us, as keep takes one layer's cache).
#include "paged.cuh"

namespace beam {
namespace paged {
namespace {

constexpr int kNodes = 64;

// The rows of sequence i, or an empty range and the bit to set.
struct Rows {
  int r0, n;
};
__device__ __forceinline__ Rows rows_of(const int32_t* start, int i, int T, unsigned& bad) {
  Rows x;
  x.r0 = start[i];
  x.n = start[i + 1] - x.r0;
  bad = 0;
  if (x.n < 0 || x.n > kNodes || x.r0 < 0 || x.r0 > T - max(0, x.n)) {
    bad = BEAM_DEV_BAD_SEQ;
    x.n = 0;
  }
  return x;
}

struct PlanParams {
  const int32_t* parent;
  const int32_t* row_start;
  const int32_t* seq_id;
  const int32_t* base;
  uint64_t* mask;
  int32_t* pos;
  int32_t* slot;
  int32_t* seq_out;
  int N, T;
};

// Masks by doubling: after round k a node's mask holds its nearest 2^k ancestors and itself, and its link
// points 2^k nodes up, so six rounds cover 64 nodes.
constexpr int kPlanWarps = 4;
__global__ void __launch_bounds__(32 * kPlanWarps) tree_plan_kernel(const PlanParams P) {
  pdl_trigger();
  pdl_wait();
  __shared__ uint64_t mask[kPlanWarps][kNodes];
  __shared__ int link[kPlanWarps][kNodes];   // -1: none; -2: of a node without a place in the tree
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31, i = blockIdx.x * kPlanWarps + w;
  if (i >= P.N) return;
  auto pad = [&](int a, int b) {
    for (int t = max(a, 0) + lane; t < min(b, P.T); t += 32) {
      P.mask[t] = 0;
      P.pos[t] = P.slot[t] = P.seq_out[t] = 0;
    }
  };
  unsigned bad;
  const Rows x = rows_of(P.row_start, i, P.T, bad);
  if (i == 0) pad(0, P.row_start[0]);
  if (i == P.N - 1) pad(P.row_start[P.N], P.T);
  if (bad) {
    if (lane == 0) flag(bad);
    pad(P.row_start[i], P.row_start[i + 1]);
    return;
  }
  const int base = P.base[i], s = P.seq_id[i];
  // behind no length, later nodes would take the slots of real tokens: all of them are lost
  bool lost = x.n > 0 && (base < 0 || base > INT32_MAX - kNodes);
  const bool none = lost;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int j = lane + 32 * e;
    int up = j < x.n ? P.parent[x.r0 + j] : -1;
    if (none || up < -1 || up >= j) {
      up = -2;
      lost = true;
    }
    mask[w][j] = uint64_t(1) << j;
    link[w][j] = up;
  }
  if (lost) flag(BEAM_DEV_BAD_POSITION);
  __syncwarp();
#pragma unroll
  for (int round = 0; round < 6; ++round) {
    uint64_t m[2];
    int up[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int j = lane + 32 * e, l = link[w][j];
      m[e] = mask[w][j] | (l >= 0 ? mask[w][l] : 0);
      up[e] = l >= 0 ? link[w][l] : l;
    }
    __syncwarp();
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      mask[w][lane + 32 * e] = m[e];
      link[w][lane + 32 * e] = up[e];
    }
    __syncwarp();
  }
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int j = lane + 32 * e;
    if (j >= x.n) continue;
    const bool in = link[w][j] == -1;
    const uint64_t m = in ? mask[w][j] : 0;
    P.mask[x.r0 + j] = m;
    P.pos[x.r0 + j] = in ? base + __popcll(m) : 0;
    P.slot[x.r0 + j] = in ? base + 1 + j : 0;
    P.seq_out[x.r0 + j] = s;
  }
}

struct AcceptParams {
  const int32_t* parent;
  const int32_t* token;
  const int32_t* sampled;
  const int32_t* row_start;
  int32_t* count;
  int32_t* path;
  int32_t* next;
  int N, T, stride;
};

// Each node that its parent's sampled token names offers itself as that parent's successor (the lowest
// index wins); the path follows the successors from the root. -1, the token of a row that could not be sampled, names none,
// and a node 0 with a parent is none that the plan has given a place.
__global__ void __launch_bounds__(32 * kPlanWarps) tree_accept_kernel(const AcceptParams P) {
  pdl_trigger();
  pdl_wait();
  __shared__ int to[kPlanWarps][kNodes], sam[kPlanWarps][kNodes], way[kPlanWarps][kNodes];
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31, i = blockIdx.x * kPlanWarps + w;
  if (i >= P.N) return;
  unsigned bad;
  const Rows x = rows_of(P.row_start, i, P.T, bad);
  if (bad && lane == 0) flag(bad);
  int up[2], tok[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int j = lane + 32 * e;
    const bool in = j < x.n;
    up[e] = in ? P.parent[x.r0 + j] : -1;
    tok[e] = in ? P.token[x.r0 + j] : 0;
    sam[w][j] = in ? P.sampled[x.r0 + j] : -1;
    to[w][j] = kNodes;
  }
  __syncwarp();
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int j = lane + 32 * e;
    if (up[e] >= 0 && up[e] < j && tok[e] >= 0 && tok[e] == sam[w][up[e]]) atomicMin(&to[w][up[e]], j);
  }
  __syncwarp();
  int n = 0, last = 0;
  const bool root = x.n > 0 && __shfl_sync(0xffffffffu, up[0], 0) == -1;
  for (int j = root ? 0 : kNodes; j < kNodes; j = to[w][j]) {   // successors come later: at most 64 steps
    if (lane == 0) way[w][n] = j;
    last = j;
    ++n;
  }
  __syncwarp();
  if (lane == 0) {
    P.count[i] = n;
    P.next[i] = n > 0 ? sam[w][last] : -1;
  }
  for (int k = lane; k < P.stride; k += 32) P.path[size_t(i) * P.stride + k] = k < n ? way[w][k] : -1;
}

struct KeepParams {
  beam_paged_kv c;
  const int32_t* seq_id;
  const int32_t* base;
  const int32_t* count;
  const int32_t* path;
  int N, stride, shift;
};

// A CTA takes one (sequence, KV head): it loads all rows that move, K and V, before it stores any, since one
// row's new place may be another's old one.
template <int FMT, int D>
__global__ void __launch_bounds__(256) paged_keep_kernel(const KeepParams P) {
  pdl_trigger();
  pdl_wait();
  constexpr int ROWB = row_bytes(FMT, D), CPR = ROWB / 16;    // 16-byte chunks of a row
  constexpr int ITEMS = kNodes * 2 * CPR / 256;               // chunks of a thread
  __shared__ int64_t from[kNodes], into[kNodes];              // rows of codes, or -1
  const int i = blockIdx.x, h = blockIdx.y, size = P.c.page_size;
  const int n = P.count[i];
  if (n < 0 || n > kNodes || n > P.stride) {
    if (threadIdx.x == 0 && h == 0) flag(BEAM_DEV_BAD_POSITION);
    return;
  }
  if (threadIdx.x < kNodes) {
    const int k = threadIdx.x;
    int64_t a = -1, b = -1;
    const int src = k < n ? P.path[size_t(i) * P.stride + k] : k;
    if (src != k) {
      const int s = P.seq_id[i], base = P.base[i];
      unsigned bad = 0;
      if (src < 0 || src >= kNodes || base < 0 || base > INT32_MAX - 2 * kNodes) bad = BEAM_DEV_BAD_POSITION;
      else {
        const int p0 = page_of(P.c, s, base + 1 + src, P.shift, bad);
        unsigned bad1 = 0;
        const int p1 = page_of(P.c, s, base + 1 + k, P.shift, bad1);
        bad |= bad1;
        if (!bad) {
          a = (int64_t(p0) * P.c.n_kv + h) * size + ((base + src) & (size - 1));
          b = (int64_t(p1) * P.c.n_kv + h) * size + ((base + k) & (size - 1));
        }
      }
      if (bad && h == 0) flag(bad);
    }
    from[k] = a;
    into[k] = b;
  }
  __syncthreads();
  uint4 x[ITEMS];
#pragma unroll
  for (int e = 0; e < ITEMS; ++e) {
    const int c = threadIdx.x + 256 * e, k = c / (2 * CPR), kv = (c / CPR) & 1;
    if (from[k] >= 0)
      x[e] = *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(kv ? P.c.v : P.c.k) + from[k] * ROWB + (c % CPR) * 16);
  }
  // scales: [page][head][K | V][key], thread (row, K or V)
  const int k = threadIdx.x >> 1, kv = threadIdx.x & 1;
  const bool scaled = FMT != kFmtBF16 && k < kNodes && from[k < kNodes ? k : 0] >= 0;
  auto scale_row = [&](int64_t r) { return 2 * r - (r & (size - 1)) + kv * size; };
  uint8_t rs = 0;
  uint2 bs = make_uint2(0, 0);
  if (scaled) {
    rs = P.c.row_scale[scale_row(from[k])];
    if (FMT == kFmtNVFP4) {
      const uint8_t* b = P.c.block_scale + scale_row(from[k]) * (D / 16);
      if (D == 128) bs = *reinterpret_cast<const uint2*>(b);
      else bs.x = *reinterpret_cast<const uint32_t*>(b);
    }
  }
  __syncthreads();
#pragma unroll
  for (int e = 0; e < ITEMS; ++e) {
    const int c = threadIdx.x + 256 * e, r = c / (2 * CPR), v = (c / CPR) & 1;
    if (from[r] >= 0)
      *reinterpret_cast<uint4*>(static_cast<uint8_t*>(v ? P.c.v : P.c.k) + into[r] * ROWB + (c % CPR) * 16) = x[e];
  }
  if (scaled) {
    P.c.row_scale[scale_row(into[k])] = rs;
    if (FMT == kFmtNVFP4) {
      uint8_t* b = P.c.block_scale + scale_row(into[k]) * (D / 16);
      if (D == 128) *reinterpret_cast<uint2*>(b) = bs;
      else *reinterpret_cast<uint32_t*>(b) = bs.x;
    }
  }
}

}  // namespace
}  // namespace paged
}  // namespace beam

extern "C" beam_status beam_tree_plan(const int32_t* parent, const int32_t* row_start, const int32_t* seq_id,
                                      const int32_t* base, int N, int T, uint64_t* mask, int32_t* pos,
                                      int32_t* slot, int32_t* row_seq, beam_stream_t stream) {
  using namespace beam;
  using namespace beam::paged;
  if (N < 0 || T < 0) return BEAM_ERR_INVALID_ARG;
  if (T == 0) return BEAM_OK;
  if (N == 0 || !parent || !row_start || !seq_id || !base || !mask || !pos || !slot || !row_seq ||
      (reinterpret_cast<uintptr_t>(mask) & 7u))
    return BEAM_ERR_INVALID_ARG;
  const PlanParams p{parent, row_start, seq_id, base, mask, pos, slot, row_seq, N, T};
  return cuda_status(launch_pdl(tree_plan_kernel, dim3((N + kPlanWarps - 1) / kPlanWarps), dim3(32 * kPlanWarps), 0,
                                reinterpret_cast<cudaStream_t>(stream), p));
}

extern "C" beam_status beam_tree_accept(const int32_t* parent, const int32_t* token, const int32_t* sampled,
                                        const int32_t* row_start, int N, int T, int32_t* count, int32_t* path,
                                        int path_stride, int32_t* next, beam_stream_t stream) {
  using namespace beam;
  using namespace beam::paged;
  if (N < 0 || T < 0 || path_stride < 1) return BEAM_ERR_INVALID_ARG;
  if (N == 0) return BEAM_OK;
  if (!row_start || !count || !path || !next || (T > 0 && (!parent || !token || !sampled))) return BEAM_ERR_INVALID_ARG;
  const AcceptParams p{parent, token, sampled, row_start, count, path, next, N, T, path_stride};
  return cuda_status(launch_pdl(tree_accept_kernel, dim3((N + kPlanWarps - 1) / kPlanWarps), dim3(32 * kPlanWarps), 0,
                                reinterpret_cast<cudaStream_t>(stream), p));
}

extern "C" beam_status beam_paged_kv_keep(const beam_paged_kv* cache, const int32_t* seq_id, const int32_t* base,
                                          const int32_t* count, const int32_t* path, int path_stride, int N,
                                          beam_stream_t stream) {
  using namespace beam;
  using namespace beam::paged;
  const beam_status st = check(cache);
  if (st != BEAM_OK) return st;
  if (N < 0 || path_stride < 1) return BEAM_ERR_INVALID_ARG;
  if (N == 0) return BEAM_OK;
  if (!seq_id || !base || !count || !path) return BEAM_ERR_INVALID_ARG;
  if (cache->n_kv > 65535) return BEAM_ERR_UNSUPPORTED;   // grid limit
  const KeepParams p{*cache, seq_id, base, count, path, N, path_stride, log2i(cache->page_size)};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool wide = cache->head_dim == 128;
  auto go = [&](auto kern) { return launch_pdl(kern, dim3(N, cache->n_kv), dim3(256), 0, s, p); };
  cudaError_t e;
  if (cache->dtype == kFmtBF16) e = wide ? go(paged_keep_kernel<kFmtBF16, 128>) : go(paged_keep_kernel<kFmtBF16, 64>);
  else if (cache->dtype == kFmtFP8) e = wide ? go(paged_keep_kernel<kFmtFP8, 128>) : go(paged_keep_kernel<kFmtFP8, 64>);
  else e = wide ? go(paged_keep_kernel<kFmtNVFP4, 128>) : go(paged_keep_kernel<kFmtNVFP4, 64>);
  return cuda_status(e);
}
