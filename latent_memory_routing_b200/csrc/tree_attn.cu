// Attention for trees of drafted tokens over [memory rows ; paged cache ;
// drafted tokens], GQA: the serving form of the sparse attention once the
// local context lives in a paged cache (one token a sequence is plain
// decode, a chain is a causal block, a tree is what a drafter proposes).
//
// Method: "EverMind-AI/MSA: routing top-k compressed documents inside
// attention ..." (hysenlabs.com), §"Routing happens inside attention ..."
// (the selected documents' compressed K/V joined with the query's local K/V
// for autoregressive decoding).  Token i of a sequence sees every memory row,
// every cached row and, of the drafted tokens, itself and its ancestors:
//   o_i = sum_j softmax_j(scale q_i . k_j) v_j   over the keys it sees.
// Queries and cached keys are already rotated (msa_paged_append); memory
// rows keep their document-wise rotation.
//
// This file holds the CUDA-core kernel -- one CTA per (split of a
// sequence's keys, 16 query rows = tokens x heads of a KV group, KV head),
// 32-key tiles in shared memory in fp32, one pass with a running maximum and
// sum -- the kernel that joins the splits, and the entry point.
#include <algorithm>
#include <cmath>

#include "tree_attn.cuh"

namespace msa {
namespace {

constexpr int kThreads = 128;
constexpr int kRows = 16;   // query rows of a CTA
constexpr int kTile = 32;   // keys of a tile
constexpr float kLog2e = 1.4426950408889634f;

struct TreePlan {
  int n_blk, n_split;
  size_t po_bytes, ml_bytes, total;
};

// Splits: enough CTAs to cover the SMs twice, each of at least 64 keys of
// the longest sequence the buffers can hold, at most 64.
TreePlan tree_plan(int B, int n_max, int Hq, int H, int D, int m_cap, int max_pages,
                   int page_size) {
  TreePlan p{};
  p.n_blk = (n_max * (Hq / H) + kRows - 1) / kRows;
  const int64_t base = (int64_t)B * H * p.n_blk;
  const int64_t keys = (int64_t)m_cap + (int64_t)max_pages * page_size;
  const int64_t want = 2LL * num_sms();
  int64_t ns = (want + base - 1) / base;
  ns = std::min<int64_t>({ns, (keys + 63) / 64, 64});
  p.n_split = (int)std::max<int64_t>(1, ns);
  const size_t rows = (size_t)B * n_max * Hq;
  if (p.n_split > 1) {
    p.po_bytes = round_up(rows * p.n_split * D * sizeof(float), 256);
    p.ml_bytes = round_up(rows * p.n_split * sizeof(float2), 256);
  }
  p.total = p.po_bytes + p.ml_bytes;
  return p;
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
tree_simt_kernel(const __grid_constant__ TreeArgs a, int n_split, float* __restrict__ part_o,
                 float2* __restrict__ part_ml) {
  constexpr int PER = D / 32;
  constexpr int MAXR = kRows / (kThreads / 32);  // query rows a warp
  __shared__ float qs[kRows][D];
  __shared__ float ks[kTile][D + 1];
  __shared__ float vs[kTile][D];
  __shared__ TreeMask mask;
  pdl_trigger();
  pdl_wait();
  const int split = blockIdx.x, blk = blockIdx.y;
  const int b = blockIdx.z / a.H, g = blockIdx.z % a.H;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const TreeSeq s = tree_seq(a, b);
  if (s.error && tid == 0) record_error(a.status, s.error);
  const int G = a.G;
  const int row0 = blk * kRows;
  const int rows = min(kRows, s.n * G - row0);
  if (rows <= 0) return;
  tree_mask(a, s, mask, tid, [] { __syncthreads(); });

  for (int e = tid; e < rows * D; e += kThreads) {
    const int r = row0 + e / D, d = e % D;
    const int64_t off = ((s.t0 + r / G) * a.Hq + g * G + r % G) * D + d;
    qs[e / D][d] = Elem<T>::to_f(static_cast<const T*>(a.q)[off]) * a.qscale;
  }
  const int keys = s.M + s.cache;
  const int tiles = (keys + kTile - 1) / kTile;
  const int k_lo = (int)((int64_t)split * tiles / n_split) * kTile;
  const int k_hi = min(keys, (int)((int64_t)(split + 1) * tiles / n_split) * kTile);

  float m_run[MAXR], l_run[MAXR], o[MAXR][PER];
  uint4 anc[MAXR];
  bool alive[MAXR];
#pragma unroll
  for (int rr = 0; rr < MAXR; ++rr) {
    m_run[rr] = -INFINITY;
    l_run[rr] = 0.f;
#pragma unroll
    for (int x = 0; x < PER; ++x) o[rr][x] = 0.f;
    const int r = warp + 4 * rr;
    const int tok = r < rows ? (row0 + r) / G : 0;
    anc[rr] = mask.anc[tok];
    alive[rr] = r < rows && mask.up[tok] != kTreeDead;
  }

  for (int t0 = k_lo; t0 < k_hi; t0 += kTile) {
    __syncthreads();
    for (int e = tid; e < kTile * D; e += kThreads) {
      const int j = e / D, d = e % D;
      const int kk = t0 + j;
      float kv = 0.f, vv = 0.f;
      if (kk < k_hi) {
        if (kk < s.M) {
          const int64_t off = (((int64_t)b * a.m_cap + kk) * a.H + g) * D + d;
          kv = Elem<T>::to_f(static_cast<const T*>(a.k_mem)[off]);
          vv = Elem<T>::to_f(static_cast<const T*>(a.v_mem)[off]);
        } else {
          const int slot = kk - s.M;
          const int pg = a.block_table[(int64_t)b * a.max_pages + slot / a.page_size];
          if (pg >= 0 && pg < a.n_pages) {
            const int64_t off =
                (((int64_t)pg * a.H + g) * a.page_size + slot % a.page_size) * D + d;
            kv = Elem<T>::to_f(static_cast<const T*>(a.k_pages)[off]);
            vv = Elem<T>::to_f(static_cast<const T*>(a.v_pages)[off]);
          } else if (d == 0) {
            record_error(a.status, MSA_ERR_INVALID_ARG);
          }
        }
      }
      ks[j][d] = kv;
      vs[j][d] = vv;
    }
    __syncthreads();
    const int kk = t0 + lane;
#pragma unroll
    for (int rr = 0; rr < MAXR; ++rr) {
      const int r = warp + 4 * rr;
      if (r >= rows) break;  // warp-uniform
      float sc = 0.f;
#pragma unroll 8
      for (int d = 0; d < D; ++d) sc = fmaf(qs[r][d], ks[lane][d], sc);
      const int j = kk - s.M - s.L;  // drafted token, if >= 0
      const bool ok = alive[rr] && kk < k_hi && (j < 0 || tree_bit(anc[rr], j));
      sc = ok ? sc : -INFINITY;
      float mt = sc;
#pragma unroll
      for (int off = 16; off; off >>= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, off));
      // (a NaN score is no maximum: it makes its own weight NaN; a score of
      // -inf weighs nothing even while no other was seen)
      const float m_new = fmaxf(m_run[rr], mt);
      const float ref = m_new == -INFINITY ? 0.f : m_new;
      const float p = exp2f(sc - ref);
      const float corr = exp2f(m_run[rr] - ref);
      float ps = p;
#pragma unroll
      for (int off = 16; off; off >>= 1) ps += __shfl_xor_sync(0xffffffffu, ps, off);
      l_run[rr] = l_run[rr] * corr + ps;
      m_run[rr] = m_new;
#pragma unroll
      for (int x = 0; x < PER; ++x) o[rr][x] *= corr;
      // seen keys only: a masked value, NaN included, adds nothing
      for (uint32_t seen = __ballot_sync(0xffffffffu, ok); seen; seen &= seen - 1) {
        const int i = __ffs(seen) - 1;
        const float pi = __shfl_sync(0xffffffffu, p, i);
#pragma unroll
        for (int x = 0; x < PER; ++x) o[rr][x] = fmaf(pi, vs[i][lane + 32 * x], o[rr][x]);
      }
    }
  }

#pragma unroll
  for (int rr = 0; rr < MAXR; ++rr) {
    const int r = warp + 4 * rr;
    if (r >= rows) break;
    const int tok = (row0 + r) / G, hq = g * G + (row0 + r) % G;
    if (n_split == 1) {
      // no weight at all: zero; a NaN sum stays NaN
      const float inv = l_run[rr] == 0.f ? 0.f : 1.f / l_run[rr];
      T* op = static_cast<T*>(a.out) + ((s.t0 + tok) * a.Hq + hq) * D;
#pragma unroll
      for (int x = 0; x < PER; ++x)
        op[lane + 32 * x] = Elem<T>::from_f(l_run[rr] == 0.f ? 0.f : o[rr][x] * inv);
    } else {
      const int64_t row = ((int64_t)b * a.n_max + tok) * a.Hq + hq;
      float* po = part_o + (row * n_split + split) * D;
#pragma unroll
      for (int x = 0; x < PER; ++x) po[lane + 32 * x] = o[rr][x];
      if (lane == 0) part_ml[row * n_split + split] = make_float2(m_run[rr], l_run[rr]);
    }
  }
}

// Joins the key splits of one (token, head) row.
template <typename T, int D>
__global__ void __launch_bounds__(D)
tree_combine_kernel(const __grid_constant__ TreeArgs a, int n_split,
                    const float* __restrict__ part_o, const float2* __restrict__ part_ml) {
  pdl_trigger();
  pdl_wait();
  const int hq = blockIdx.x % a.Hq;
  const int i = blockIdx.x / a.Hq % a.n_max, b = blockIdx.x / a.Hq / a.n_max;
  const TreeSeq s = tree_seq(a, b);
  if (i >= s.n) return;
  const int64_t row = ((int64_t)b * a.n_max + i) * a.Hq + hq;
  const float2* ml = part_ml + row * n_split;
  float m = -INFINITY;
  for (int sp = 0; sp < n_split; ++sp) m = fmaxf(m, ml[sp].x);
  float l = 0.f, acc = 0.f;
  for (int sp = 0; sp < n_split; ++sp) {
    if (ml[sp].y == 0.f) continue;
    const float w = m == -INFINITY ? 1.f : exp2f(ml[sp].x - m);
    l += w * ml[sp].y;
    acc += w * part_o[(row * n_split + sp) * D + threadIdx.x];
  }
  static_cast<T*>(a.out)[((s.t0 + i) * a.Hq + hq) * D + threadIdx.x] =
      Elem<T>::from_f(l == 0.f ? 0.f : acc / l);
}

template <typename T, int D>
int launch_simt(const TreeArgs& a, const TreePlan& p, void* ws, cudaStream_t s) {
  float* part_o = static_cast<float*>(ws);
  float2* part_ml =
      reinterpret_cast<float2*>(static_cast<unsigned char*>(ws) + p.po_bytes);
  const dim3 grid((unsigned)p.n_split, (unsigned)p.n_blk, (unsigned)(a.B * a.H));
  if (int rc = launch_pdl(tree_simt_kernel<T, D>, grid, dim3(kThreads), 0, s, a, p.n_split,
                          part_o, part_ml))
    return rc;
  if (p.n_split == 1) return MSA_OK;
  return launch_pdl(tree_combine_kernel<T, D>, dim3((unsigned)((int64_t)a.B * a.n_max * a.Hq)),
                    dim3(D), 0, s, a, p.n_split, static_cast<const float*>(part_o),
                    static_cast<const float2*>(part_ml));
}

// Shape checks shared by the call and its workspace size; a MSA status.
int tree_shape(msa_dtype dt, int B, int n_max, int Hq, int H, int D, int m_cap, int max_pages,
               int page_size) {
  if ((dt != MSA_F32 && dt != MSA_BF16) || B <= 0 || n_max <= 0 || Hq <= 0 || H <= 0 ||
      m_cap < 0 || max_pages <= 0)
    return MSA_ERR_INVALID_ARG;
  if (Hq % H || Hq / H > 16 || (D != 64 && D != 128) || n_max > kTreeMax)
    return MSA_ERR_UNSUPPORTED;
  if (page_size != 16 && page_size != 32 && page_size != 64 && page_size != 128)
    return MSA_ERR_UNSUPPORTED;
  if ((int64_t)B * H > 65535 || (int64_t)m_cap + (int64_t)max_pages * page_size > (1LL << 30) ||
      (int64_t)B * m_cap > INT32_MAX || (int64_t)B * n_max * Hq > INT32_MAX)
    return MSA_ERR_UNSUPPORTED;
  return MSA_OK;
}

int tree_body(msa_dtype dt, int B, int64_t n_tok, int n_max, int Hq, int H, int D, const void* q,
              const int64_t* tok_offsets, const int32_t* parents, const void* k_mem,
              const void* v_mem, const int32_t* mem_len, int m_cap, const void* k_pages,
              const void* v_pages, int n_pages, int page_size, const int32_t* block_table,
              int max_pages, const int32_t* cache_len, float scale, void* out, void* ws,
              size_t ws_bytes, cudaStream_t s) {
  if (int rc = tree_shape(dt, B, n_max, Hq, H, D, m_cap, max_pages, page_size)) return rc;
  if (n_tok < 0 || n_pages <= 0 || !std::isfinite(scale)) return MSA_ERR_INVALID_ARG;
  if ((int64_t)n_pages * H * page_size > INT32_MAX || n_tok > INT32_MAX)
    return MSA_ERR_UNSUPPORTED;
  if (!tok_offsets || !block_table || !cache_len || !k_pages || !v_pages)
    return MSA_ERR_INVALID_ARG;
  if (m_cap > 0 && (!k_mem || !v_mem || !mem_len)) return MSA_ERR_INVALID_ARG;
  if (!aligned16(k_pages) || !aligned16(v_pages)) return MSA_ERR_INVALID_ARG;
  if (m_cap > 0 && (!aligned16(k_mem) || !aligned16(v_mem))) return MSA_ERR_INVALID_ARG;
  if (n_tok == 0) return MSA_OK;
  if (!q || !out || !aligned16(q) || !aligned16(out)) return MSA_ERR_INVALID_ARG;
  if (int rc = debug_check_offsets(tok_offsets, B, n_tok, s)) return rc;
  if (m_cap > 0)
    if (int rc = debug_check_mem_len(mem_len, B, m_cap, s)) return rc;
  if (int rc = debug_check_mem_len(cache_len, B, max_pages * page_size, s)) return rc;
  TreeArgs a{};
  a.B = B;
  a.n_max = n_max;
  a.Hq = Hq;
  a.H = H;
  a.G = Hq / H;
  a.n_tok = n_tok;
  a.q = q;
  a.tok_offsets = tok_offsets;
  a.parents = parents;
  a.k_mem = k_mem;
  a.v_mem = v_mem;
  a.mem_len = mem_len;
  a.m_cap = m_cap;
  a.k_pages = k_pages;
  a.v_pages = v_pages;
  a.n_pages = n_pages;
  a.page_size = page_size;
  a.max_pages = max_pages;
  a.block_table = block_table;
  a.cache_len = cache_len;
  a.qscale = (scale > 0.f ? scale : 1.0f / sqrtf((float)D)) * kLog2e;
  a.out = out;
  a.status = device_status_ptr();
  const TreePlan p = tree_plan(B, n_max, Hq, H, D, m_cap, max_pages, page_size);
  const bool few = tree_few_takes(n_max, a.G);
  const size_t need = dt == MSA_F32 ? p.total
                      : few         ? tree_few_workspace_size(n_max, a.G, D)
                                    : tree_tc_workspace_size(n_max, a.G, D);
  if (need && (!ws || ws_bytes < need || !aligned16(ws))) return MSA_ERR_WORKSPACE;
  if (dt == MSA_BF16)
    return few ? tree_few_launch(a, D, ws, s) : tree_tc_launch(a, D, ws, s);
  return D == 64 ? launch_simt<float, 64>(a, p, ws, s) : launch_simt<float, 128>(a, p, ws, s);
}

}  // namespace
}  // namespace msa

extern "C" size_t msa_tree_attn_workspace_size(msa_dtype dt, int B, int n_max, int Hq, int H,
                                               int D, int m_cap, int max_pages, int page_size) {
  using namespace msa;
  if (tree_shape(dt, B, n_max, Hq, H, D, m_cap, max_pages, page_size)) return 0;
  if (dt == MSA_BF16)
    return tree_few_takes(n_max, Hq / H) ? tree_few_workspace_size(n_max, Hq / H, D)
                                         : tree_tc_workspace_size(n_max, Hq / H, D);
  return tree_plan(B, n_max, Hq, H, D, m_cap, max_pages, page_size).total;
}

extern "C" int msa_tree_attn(msa_dtype dt, int B, int64_t n_tok, int n_max, int Hq, int H, int D,
                             const void* q, const int64_t* tok_offsets, const int32_t* parents,
                             const void* k_mem, const void* v_mem, const int32_t* mem_len,
                             int m_cap, const void* k_pages, const void* v_pages, int n_pages,
                             int page_size, const int32_t* block_table, int max_pages,
                             const int32_t* cache_len, float scale, void* out, void* ws,
                             size_t ws_bytes, msa_stream_t stream) {
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return msa::debug_finish(
      msa::tree_body(dt, B, n_tok, n_max, Hq, H, D, q, tok_offsets, parents, k_mem, v_mem,
                     mem_len, m_cap, k_pages, v_pages, n_pages, page_size, block_table, max_pages,
                     cache_len, scale, out, ws, ws_bytes, s),
      s);
}
