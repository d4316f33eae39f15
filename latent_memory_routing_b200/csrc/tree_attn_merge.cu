// The merge of the bf16 tree attention's partials (tree_attn_few.cu,
// tree_attn_tc.cu): an item's parts, each with its own reference maximum m_i,
// sum l_i and unnormalised O_i, become
//   O = sum_i 2^(m_i - m) O_i / sum_i 2^(m_i - m) l_i,  m = max_i m_i,
// in a fixed order.  It reads each partial once and is bound by the latency of
// those loads (a few hundred KB in all), so many are in flight at a time: a
// block takes up to 16 of an item's rows, and where there are fewer (a decode
// step, whose items may have a hundred short parts) several warps share a
// row's parts.  Blocks of workers that cut no item end at once.
#include "tree_attn.cuh"

namespace msa {
namespace {

constexpr int kMergeWarps = 16;  // and rows of a block at most
constexpr int kBatch = 8;  // parts a warp has in flight

__device__ __forceinline__ uint32_t pack2(float a, float b) {
  __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&h);
}

// blockIdx.x: the worker whose range start cuts the item; blockIdx.y: rows
// kMergeWarps y .. of it.
template <int D>
__global__ void __launch_bounds__(32 * kMergeWarps)
tree_merge_kernel(const __grid_constant__ TreeArgs a, int part_rows,
                  const float* __restrict__ part_o, const float2* __restrict__ part_ml,
                  const TreeCut* __restrict__ cuts) {
  constexpr int VEC = D / 32;
  __shared__ float so[kMergeWarps][D];
  __shared__ float2 sml[kMergeWarps];
  pdl_trigger();
  pdl_wait();
  const TreeCut cut = cuts[blockIdx.x];
  const int rows = cut.rows - (int)blockIdx.y * kMergeWarps;  // of this block
  if (cut.last < 0 || rows <= 0) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int rp = 1;  // the rows, rounded up to a power of two
  while (rp < min(rows, kMergeWarps)) rp <<= 1;
  const int step = kMergeWarps / rp, sub = warp / rp;  // warps of a row, this one's turn
  const int rr = blockIdx.y * kMergeWarps + warp % rp;
  const bool live = rr < cut.rows;
  const int n_parts = live ? cut.last - (int)blockIdx.x + 2 : 0;
  float m = -INFINITY, l = 0.f, o[VEC];
#pragma unroll
  for (int x = 0; x < VEC; ++x) o[x] = 0.f;
  auto prow = [&](int i) {
    const int64_t w = (int64_t)blockIdx.x - 1 + i;
    return (w * 2 + (i == 0 ? 1 : 0)) * part_rows + rr;
  };
  auto join = [&](float2 ml, const float* v) {
    if (ml.y == 0.f) return;  // no weight (a NaN sum joins)
    const float mn = fmaxf(m, ml.x);
    const float ref = mn == -INFINITY ? 0.f : mn;
    const float c0 = exp2f(m - ref), c1 = ml.x == -INFINITY ? 1.f : exp2f(ml.x - ref);
    l = (l == 0.f ? 0.f : l * c0) + ml.y * c1;
#pragma unroll
    for (int x = 0; x < VEC; ++x) o[x] = o[x] * c0 + v[x] * c1;
    m = mn;
  };
  for (int i = sub; i < n_parts; i += kBatch * step) {
    float2 ml[kBatch];
    float v[kBatch][VEC];
#pragma unroll
    for (int x = 0; x < kBatch; ++x) {
      const int p = i + x * step;
      ml[x] = make_float2(-INFINITY, 0.f);
      if (p < n_parts) {
        const int64_t pr = prow(p);
        ml[x] = part_ml[pr];
        const float* src = part_o + pr * D + lane * VEC;
        if constexpr (VEC == 4) {
          const float4 f = *reinterpret_cast<const float4*>(src);
          v[x][0] = f.x, v[x][1] = f.y, v[x][2] = f.z, v[x][3] = f.w;
        } else {
          const float2 f = *reinterpret_cast<const float2*>(src);
          v[x][0] = f.x, v[x][1] = f.y;
        }
      }
    }
#pragma unroll
    for (int x = 0; x < kBatch; ++x) join(ml[x], v[x]);
  }
  if (step > 1) {
    if (lane == 0) sml[warp] = make_float2(m, l);
#pragma unroll
    for (int x = 0; x < VEC; ++x) so[warp][lane * VEC + x] = o[x];
    __syncthreads();
    if (sub > 0) return;
#pragma unroll 1
    for (int i = 1; i < min(n_parts, step); ++i)
      join(sml[warp + i * rp], &so[warp + i * rp][lane * VEC]);
  }
  if (!live) return;
  const int row = cut.row0 + rr;
  __nv_bfloat16* op = static_cast<__nv_bfloat16*>(a.out) +
                      ((cut.t0 + row / a.G) * a.Hq + cut.g * a.G + row % a.G) * D + lane * VEC;
  const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int x = 0; x < VEC; x += 2)
    *reinterpret_cast<uint32_t*>(op + x) = l == 0.f ? 0u : pack2(o[x] * inv, o[x + 1] * inv);
}

template <int D>
int launch(const TreeArgs& a, int workers, int part_rows, const float* part_o,
           const float2* part_ml, const TreeCut* cuts, cudaStream_t s) {
  return launch_pdl(tree_merge_kernel<D>,
                    dim3(workers, (part_rows + kMergeWarps - 1) / kMergeWarps),
                    dim3(32 * kMergeWarps), 0, s, a, part_rows, part_o, part_ml, cuts);
}

}  // namespace

int tree_merge_launch(const TreeArgs& a, int D, int workers, int part_rows, const float* part_o,
                      const float2* part_ml, const TreeCut* cuts, cudaStream_t s) {
  return D == 64 ? launch<64>(a, workers, part_rows, part_o, part_ml, cuts, s)
                 : launch<128>(a, workers, part_rows, part_o, part_ml, cuts, s);
}

}  // namespace msa
