// The merge of the tree attention's partials (tree_attn_few.cu,
// tree_attn_tc.cu): an item's parts, each with its own reference maximum m_i,
// sum l_i and unnormalised O_i, become
//   O = sum_i 2^(m_i - m) O_i / sum_i 2^(m_i - m) l_i,  m = max_i m_i,
// in a fixed order.  It reads each partial once and is bound by the latency of
// those loads (a few hundred KB to 40 MB), so many are in flight at a time: a
// block looks at the cuts of 32 workers and takes up to 16 of their rows, a
// warp each, and where there are fewer (one sequence's decode step, whose items
// have dozens of short parts) several warps share a row's parts.
#include <algorithm>

#include "tree_attn.cuh"

namespace msa {
namespace {

constexpr int kChunk = 32;       // workers whose cut rows a block looks at
constexpr int kMergeWarps = 16;  // and rows of a block at most

__device__ __forceinline__ uint32_t pack2(float a, float b) {
  __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&h);
}

// Of workers [kChunk x, kChunk x + kChunk), x = blockIdx.x, the rows that a
// border at their range starts cuts, at most `most` at a time (a power of
// two).  kCtas blocks an SM.
template <typename T, int D, int kCtas>
__global__ void __launch_bounds__(32 * kMergeWarps, kCtas)
tree_merge_kernel(const __grid_constant__ TreeArgs a, int workers, int most, int part_rows,
                  const float* __restrict__ part_o, const float2* __restrict__ part_ml,
                  const TreeCut* __restrict__ cuts) {
  constexpr int VEC = D / 32;
  constexpr int kBatch = kCtas == 1 ? 8 : 3;  // partial rows a warp has in flight
  __shared__ __align__(16) float so[kMergeWarps][D];
  __shared__ float2 sml[kMergeWarps];
  pdl_trigger();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  TreeCut cut{0, 0, 0, 0, -1};  // a lane a worker
  if ((int)blockIdx.x * kChunk + lane < workers) cut = cuts[blockIdx.x * kChunk + lane];
  int end = cut.last < 0 ? 0 : cut.rows;
#pragma unroll
  for (int s = 1; s < 32; s <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, end, s);
    if (lane >= s) end += v;
  }
  const int total = __shfl_sync(0xffffffffu, end, 31);
  for (int at0 = blockIdx.y * most; at0 < total; at0 += gridDim.y * most) {
    int rp = 1;  // the rows at hand, rounded up to a power of two
    while (rp < min(total - at0, most)) rp <<= 1;
    const int step = kMergeWarps / rp, sub = warp / rp;  // warps of a row, this one's turn
    const int at = at0 + warp % rp;
    const bool live = warp % rp < min(total - at0, most);
    const int src = live ? __popc(__ballot_sync(0xffffffffu, end <= at)) : 0;  // its worker
    TreeCut c;
    c.last = __shfl_sync(0xffffffffu, cut.last, src);
    c.t0 = __shfl_sync(0xffffffffu, cut.t0, src);
    c.g = __shfl_sync(0xffffffffu, cut.g, src);
    c.row0 = __shfl_sync(0xffffffffu, cut.row0, src);
    c.rows = __shfl_sync(0xffffffffu, cut.rows, src);
    const int rr = at - (__shfl_sync(0xffffffffu, end, src) - c.rows);
    const int worker = blockIdx.x * kChunk + src;
    const int n_parts = live ? c.last - worker + 2 : 0;
    const int mine = (n_parts - sub + step - 1) / step;  // parts sub, sub + step, ..
    // part 0 is (worker - 1, slot 1), part i (worker + i - 1, slot 0)
    auto prow = [&](int i) {
      const int p = sub + i * step;
      return ((int64_t)(worker - 1 + p) * 2 + (p == 0 ? 1 : 0)) * part_rows + rr;
    };
    float m = -INFINITY, l = 0.f, o[VEC];
#pragma unroll
    for (int x = 0; x < VEC; ++x) o[x] = 0.f;
    for (int i0 = 0; i0 < mine; i0 += 32) {
      // a lane a part: the weights 2^(m_i - m) of up to 32 parts
      const int n = min(32, mine - i0);
      float2 ml = make_float2(-INFINITY, 0.f);
      if (lane < n) ml = part_ml[prow(i0 + lane)];
      float v[kBatch][VEC];
      auto load = [&](int i) {
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
          const float* src = part_o + prow(i0 + min(i + b, n - 1)) * D + lane * VEC;
          if constexpr (VEC == 4) {
            const float4 f = *reinterpret_cast<const float4*>(src);
            v[b][0] = f.x, v[b][1] = f.y, v[b][2] = f.z, v[b][3] = f.w;
          } else {
            const float2 f = *reinterpret_cast<const float2*>(src);
            v[b][0] = f.x, v[b][1] = f.y;
          }
        }
      };
      load(0);  // in flight with the sums
      float mx = ml.y == 0.f ? -INFINITY : ml.x;  // no weight (a NaN sum has one)
#pragma unroll
      for (int s = 16; s; s >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, s));
      const float mn = fmaxf(m, mx), ref = mn == -INFINITY ? 0.f : mn;
      const float c = m == -INFINITY ? (l == 0.f ? 0.f : 1.f) : exp2f(m - ref);
      const float w = ml.y == 0.f ? 0.f : ml.x == -INFINITY ? 1.f : exp2f(ml.x - ref);
      float ls = ml.y == 0.f ? 0.f : w * ml.y;
#pragma unroll
      for (int s = 16; s; s >>= 1) ls += __shfl_xor_sync(0xffffffffu, ls, s);
      l = (l == 0.f ? 0.f : l * c) + ls;
#pragma unroll
      for (int x = 0; x < VEC; ++x) o[x] *= c;
      m = mn;
      for (int i = 0;;) {
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
          const float wb = __shfl_sync(0xffffffffu, w, min(i + b, 31));
#pragma unroll
          for (int x = 0; x < VEC; ++x)
            if (i + b < n && wb != 0.f) o[x] = fmaf(v[b][x], wb, o[x]);
        }
        if ((i += kBatch) >= n) break;
        load(i);
      }
    }
    if (step > 1) {
      if (lane == 0) sml[warp] = make_float2(m, l);
#pragma unroll
      for (int x = 0; x < VEC; ++x) so[warp][lane * VEC + x] = o[x];
      __syncthreads();
#pragma unroll 1
      for (int i = 1; sub == 0 && i < min(n_parts, step); ++i) {
        const float2 ml = sml[warp + i * rp];
        if (ml.y == 0.f) continue;
        const float mn = fmaxf(m, ml.x), ref = mn == -INFINITY ? 0.f : mn;
        const float c = m == -INFINITY ? (l == 0.f ? 0.f : 1.f) : exp2f(m - ref);
        const float w = ml.x == -INFINITY ? 1.f : exp2f(ml.x - ref);
        l = (l == 0.f ? 0.f : l * c) + w * ml.y;
#pragma unroll
        for (int x = 0; x < VEC; ++x)
          o[x] = fmaf(so[warp + i * rp][lane * VEC + x], w, o[x] * c);
        m = mn;
      }
    }
    if (live && sub == 0) {
      const int row = c.row0 + rr;
      T* op = static_cast<T*>(a.out) +
              ((c.t0 + row / a.G) * a.Hq + c.g * a.G + row % a.G) * D + lane * VEC;
      const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
      for (int x = 0; x < VEC; x += 2) {
        const float2 v = l == 0.f ? make_float2(0.f, 0.f) : make_float2(o[x] * inv, o[x + 1] * inv);
        if constexpr (sizeof(T) == 4)
          *reinterpret_cast<float2*>(op + x) = v;
        else
          *reinterpret_cast<uint32_t*>(op + x) = pack2(v.x, v.y);
      }
    }
    __syncthreads();  // so and sml have been read
  }
}

template <typename T, int D>
int launch(const TreeArgs& a, int ctas, int per, int part_rows, const float* part_o,
           const float2* part_ml, const TreeCut* cuts, cudaStream_t s) {
  const int workers = ctas * per, chunks = (workers + kChunk - 1) / kChunk;
  const int64_t items = std::min<int64_t>(
      workers, (int64_t)a.B * a.H * ((a.n_max * a.G + part_rows - 1) / part_rows));
  // Few items may have many parts each: eight warps then share a row's (two
  // items of 1,250 slices and 16 rows: 50 us with a warp a row, 20).
  const bool long_items = items * 32 <= workers;
  const int most = long_items ? 2 : kMergeWarps;
  const int y = (2 * num_sms() + chunks - 1) / chunks * (long_items ? 3 : 1);
  auto go = [&](auto kern) {
    return launch_pdl(kern, dim3(chunks, y), dim3(32 * kMergeWarps), 0, s, a, workers, most,
                      part_rows, part_o, part_ml, cuts);
  };
  // Few rows: one block an SM, with more loads in flight (one sequence of 4,316
  // keys: 13.8 us, 14.8 with two); many: two blocks (16 trees of up to 48 tokens:
  // 103, with one 110).
  return items * part_rows <= 2LL * kMergeWarps * num_sms() ? go(tree_merge_kernel<T, D, 1>)
                                                            : go(tree_merge_kernel<T, D, 2>);
}

}  // namespace

int tree_merge_launch(const TreeArgs& a, bool f32, int D, int ctas, int per, int part_rows,
                      const float* part_o, const float2* part_ml, const TreeCut* cuts,
                      cudaStream_t s) {
  auto go = [&](auto f) { return f(a, ctas, per, part_rows, part_o, part_ml, cuts, s); };
  if (f32) return D == 64 ? go(launch<float, 64>) : go(launch<float, 128>);
  return D == 64 ? go(launch<__nv_bfloat16, 64>) : go(launch<__nv_bfloat16, 128>);
}

}  // namespace msa
