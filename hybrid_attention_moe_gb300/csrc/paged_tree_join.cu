// Joins the partials of the tree attention over pages (paged_tree.cu): o = sum_s 2^(m_s - m) O_s / sum_s 2^(m_s - m) l_s
// over an item's parts, m = max m_s, gated and rounded once. It also hands the kernel's status bits on. A few us behind the main kernel: partials are in L2.
#include "paged_tree.cuh"

namespace beam {
namespace paged {
namespace tree {
namespace {

// Join of the item that begins in range blockIdx.x and runs on past it: tile blockIdx.y, 32 rows a CTA, eight threads a
// row.
constexpr int kJoinRows = 32;
template <int D>
__global__ void __launch_bounds__(8 * kJoinRows) paged_tree_join_kernel(const Params P) {
  pdl_trigger();
  pdl_wait();
  const int4 jn = P.join[2 * blockIdx.x], rows = P.join[2 * blockIdx.x + 1];
  if (rows.z != 0 && blockIdx.y == 0 && blockIdx.z == 0 && threadIdx.x == 0) flag(unsigned(rows.z));
  if (jn.z == 0 || int(blockIdx.y) >= jn.w) return;
  const int lr = blockIdx.z * kJoinRows + threadIdx.x / 8, d = (threadIdx.x % 8) * 4;   // columns d + 32 e
  const int row = (2 * jn.y + blockIdx.y) * ROWS + lr, node = row / P.G, hq = jn.x * P.G + (row - node * P.G);
  if (node >= rows.y) return;
  auto at = [&](int s) { return ((size_t(blockIdx.x + s) * 2 + (s == 0 ? 1 : 0)) * 2 + blockIdx.y) * ROWS + lr; };
  float M = kNegInf, L = 0.f;
  float4 O[D / 32];
#pragma unroll
  for (int e = 0; e < D / 32; ++e) O[e] = make_float4(0.f, 0.f, 0.f, 0.f);
  const float bias = P.g != nullptr ? bf2f(P.gate_bias[hq]) : 0.f;
  const size_t o = (size_t(rows.x + node) * P.n_q + hq) * D + d;
  uint2 gv[D / 32];
#pragma unroll
  for (int e = 0; e < D / 32; ++e) gv[e] = P.g != nullptr ? *reinterpret_cast<const uint2*>(P.g + o + 32 * e) : make_uint2(0, 0);
  for (int s = 0; s < jn.z; ++s) M = fmaxf(M, __ldcg(&P.part_ml[at(s)]).x);
#pragma unroll 2
  for (int s = 0; s < jn.z; ++s) {
    const float2 ml = __ldcg(&P.part_ml[at(s)]);
    const float f = ml.y == 0.f ? 0.f : ex2(ml.x - M);
    L += f * ml.y;
#pragma unroll
    for (int e = 0; e < D / 32; ++e) {
      const float4 v = __ldcg(reinterpret_cast<const float4*>(P.part_acc + at(s) * D + d + 32 * e));
      O[e].x += f * v.x;
      O[e].y += f * v.y;
      O[e].z += f * v.z;
      O[e].w += f * v.w;
    }
  }
  const float inv = L == 0.f ? 0.f : 1.f / L;
  const bool gated = P.g != nullptr && L != 0.f;   // a row that sees nothing is zero, whatever its gate holds
#pragma unroll
  for (int e = 0; e < D / 32; ++e)
    *reinterpret_cast<uint2*>(P.og + o + 32 * e) =
        finish4(gated, make_float4(O[e].x * inv, O[e].y * inv, O[e].z * inv, O[e].w * inv), gv[e], bias);
}

}  // namespace

cudaError_t join(const Params& p, int grid, cudaStream_t st) {
  const dim3 dims(grid, p.G * kNodes > ROWS ? 2 : 1, ROWS / kJoinRows), block(8 * kJoinRows);
  return p.c.head_dim == 128 ? launch_pdl(paged_tree_join_kernel<128>, dims, block, 0, st, p)
                             : launch_pdl(paged_tree_join_kernel<64>, dims, block, 0, st, p);
}

}  // namespace tree
}  // namespace paged
}  // namespace beam
