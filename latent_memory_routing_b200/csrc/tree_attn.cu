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
// This file holds the entry point and the kernel of small fp32 calls, on the
// CUDA cores; bf16 goes to tree_attn_few.cu and tree_attn_tc.cu, the other fp32
// calls to the first (in split tf32).  4 D operations a row and key: bound by the
// fp32 pipe for many rows and by latency for the small calls.  One CTA per
// (split of a sequence's keys, block of query rows = tokens x heads of a KV
// group, KV head), tiles of keys copied ahead by cp.async, one pass with a
// running maximum and sum; a second launch joins the splits.
// 4 RW rows a CTA, a key a lane, RW rows a warp: 2 sequences of up to 16
// tokens over 322 keys, 9 us (42 with scalar loads of one tile at a time and 64
// keys a split).
#include <algorithm>
#include <cmath>

#include "tree_attn.cuh"

namespace msa {
namespace {

constexpr int kThreads = 128;
constexpr int kTile = 32;   // keys of a tile
constexpr float kLog2e = 1.4426950408889634f;

struct TreePlan {
  int rw;  // rows of a warp
  int n_blk, n_split;
  size_t po_bytes, ml_bytes, total;
};

// Splits: enough CTAs to cover the SMs twice, each of at least one tile of
// the longest sequence the buffers can hold, at most 64.  Rows of a warp: the
// fewest that cover a sequence's rows, 8 at most (a key read from shared
// memory then serves 8), and fewer while even the most splits leave SMs empty.
TreePlan tree_plan(int B, int n_max, int Hq, int H, int D, int m_cap, int max_pages,
                   int page_size) {
  TreePlan p{};
  const int rows_kv = n_max * (Hq / H);
  const int64_t keys = (int64_t)m_cap + (int64_t)max_pages * page_size;
  const int64_t want = 2LL * num_sms();
  const int64_t most = std::min<int64_t>((keys + kTile - 1) / kTile, 64);
  p.rw = rows_kv <= 4 ? 1 : rows_kv <= 8 ? 2 : rows_kv <= 16 ? 4 : 8;
  for (;; p.rw /= 2) {
    p.n_blk = (rows_kv + 4 * p.rw - 1) / (4 * p.rw);
    const int64_t base = (int64_t)B * H * p.n_blk;
    p.n_split = (int)std::max<int64_t>(1, std::min((want + base - 1) / base, most));
    if (p.rw <= 1 || base * p.n_split >= num_sms()) break;
  }
  const size_t rows = (size_t)B * n_max * Hq;
  if (p.n_split > 1) {
    p.po_bytes = round_up(rows * p.n_split * D * sizeof(float), 256);
    p.ml_bytes = round_up(rows * p.n_split * sizeof(float2), 256);
  }
  p.total = p.po_bytes + p.ml_bytes;
  return p;
}

template <int D, int RW> struct SimtSmem {
  float ks[2][kTile][D + 4];  // padded: a quarter warp's 16-byte reads of 8 rows
  float vs[2][kTile][D];
  float qs[4 * RW][D];
  float ps[4 * RW][kTile];
  TreeMask mask;
};

// 16 bytes into shared memory, zeros where `live` is false.
__device__ __forceinline__ void cp16_or_zero(float* dst, const float* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                   (uint32_t)__cvta_generic_to_shared(dst)),
               "l"(src), "r"(live ? 16 : 0)
               : "memory");
}

template <int D, int RW>
__global__ void __launch_bounds__(kThreads)
tree_simt_kernel(const __grid_constant__ TreeArgs a, int n_split, float* __restrict__ part_o,
                 float2* __restrict__ part_ml) {
  constexpr int PER = D / 32;
  extern __shared__ __align__(16) unsigned char simt_raw[];
  SimtSmem<D, RW>& sm = *reinterpret_cast<SimtSmem<D, RW>*>(simt_raw);
  pdl_trigger();
  pdl_wait();
  const int split = blockIdx.x, blk = blockIdx.y;
  const int b = blockIdx.z / a.H, g = blockIdx.z % a.H;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const TreeSeq s = tree_seq(a, b);
  if (s.error && tid == 0) record_error(a.status, s.error);
  const int G = a.G;
  const int row0 = blk * 4 * RW;
  const int rows = min(4 * RW, s.n * G - row0);
  if (rows <= 0) return;

  const int keys = s.M + s.cache;
  const int tiles = (keys + kTile - 1) / kTile;
  const int t_lo = (int)((int64_t)split * tiles / n_split);
  const int t_hi = (int)((int64_t)(split + 1) * tiles / n_split);
  // Copies tile t into buffer t & 1: four threads a key; keys past the end
  // and on pages that are not there read as zeros.
  auto copy = [&](int t) {
    if (t < t_hi) {
      const int j = tid >> 2, kk = t * kTile + j, d0 = (tid & 3) * 4;
      const float *kp = static_cast<const float*>(a.k_pages),
                  *vp = static_cast<const float*>(a.v_pages);
      bool live = kk < keys;
      if (live) {
        int64_t off;
        if (kk < s.M) {
          kp = static_cast<const float*>(a.k_mem);
          vp = static_cast<const float*>(a.v_mem);
          off = (((int64_t)b * a.m_cap + kk) * a.H + g) * D;
        } else {
          const int slot = kk - s.M;
          const int pg = a.block_table[(int64_t)b * a.max_pages + slot / a.page_size];
          live = pg >= 0 && pg < a.n_pages;
          if (!live && (tid & 3) == 0) record_error(a.status, MSA_ERR_INVALID_ARG);
          off = live ? (((int64_t)pg * a.H + g) * a.page_size + slot % a.page_size) * D : 0;
        }
        kp += off;
        vp += off;
      }
#pragma unroll
      for (int d = 0; d < D; d += 16) {
        cp16_or_zero(&sm.ks[t & 1][j][d + d0], kp + d + d0, live);
        cp16_or_zero(&sm.vs[t & 1][j][d + d0], vp + d + d0, live);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  copy(t_lo);
  for (int e = tid; e < 4 * RW * (D / 4); e += kThreads) {
    const int i = e / (D / 4), d = e % (D / 4) * 4, r = row0 + i;
    float4 q = make_float4(0.f, 0.f, 0.f, 0.f);
    if (i < rows)
      q = *reinterpret_cast<const float4*>(static_cast<const float*>(a.q) +
                                           ((s.t0 + r / G) * a.Hq + g * G + r % G) * D + d);
    *reinterpret_cast<float4*>(&sm.qs[i][d]) =
        make_float4(q.x * a.qscale, q.y * a.qscale, q.z * a.qscale, q.w * a.qscale);
  }
  tree_mask(a, s, sm.mask, tid, [] { __syncthreads(); });

  float m_run[RW], l_part[RW], o[RW][PER];
  int tok[RW];
  bool alive[RW];
#pragma unroll
  for (int i = 0; i < RW; ++i) {
    m_run[i] = -INFINITY;
    l_part[i] = 0.f;
#pragma unroll
    for (int x = 0; x < PER; ++x) o[i][x] = 0.f;
    const int r = warp * RW + i;
    tok[i] = r < rows ? (row0 + r) / G : 0;
    alive[i] = r < rows && sm.mask.up[tok[i]] != kTreeDead;
  }

  for (int t = t_lo; t < t_hi; ++t) {
    copy(t + 1);
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    __syncthreads();
    const float (*ks)[D + 4] = sm.ks[t & 1];
    const float (*vs)[D] = sm.vs[t & 1];
    float sc[RW];
#pragma unroll
    for (int i = 0; i < RW; ++i) sc[i] = 0.f;
#pragma unroll 4
    for (int d = 0; d < D; d += 4) {
      const float4 k = *reinterpret_cast<const float4*>(&ks[lane][d]);
#pragma unroll
      for (int i = 0; i < RW; ++i) {
        const float4 q = *reinterpret_cast<const float4*>(&sm.qs[warp * RW + i][d]);
        sc[i] = fmaf(q.x, k.x, fmaf(q.y, k.y, fmaf(q.z, k.z, fmaf(q.w, k.w, sc[i]))));
      }
    }
    const int kk = t * kTile + lane, j = kk - s.M - s.L;  // j >= 0: drafted token
    // every alive row sees every key
    const bool all = (t + 1) * kTile <= s.M + s.L;
    uint32_t seen[RW];
#pragma unroll
    for (int i = 0; i < RW; ++i) {
      const bool ok =
          all || (kk < keys && (j < 0 || tree_bit(sm.mask.anc[tok[i]], j)));
      seen[i] = all ? 0xffffffffu : __ballot_sync(0xffffffffu, ok);
      sc[i] = ok ? sc[i] : -INFINITY;
      float mt = sc[i];
#pragma unroll
      for (int x = 16; x; x >>= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, x));
      // (a NaN score is no maximum: it makes its own weight NaN; a score of
      // -inf weighs nothing even while no other was seen)
      const float m_new = fmaxf(m_run[i], mt);
      const float ref = m_new == -INFINITY ? 0.f : m_new;
      const float p = exp2f(sc[i] - ref);
      const float corr = exp2f(m_run[i] - ref);
      l_part[i] = l_part[i] * corr + p;
      m_run[i] = m_new;
#pragma unroll
      for (int x = 0; x < PER; ++x) o[i][x] *= corr;
      sm.ps[warp * RW + i][lane] = p;
    }
    __syncwarp();
    // (seen keys only: a masked value, NaN included, adds nothing)
#pragma unroll 2
    for (int k = 0; k < kTile; k += 4) {
      float v[4][PER];
#pragma unroll
      for (int y = 0; y < 4; ++y)
#pragma unroll
        for (int x = 0; x < PER; ++x) v[y][x] = vs[k + y][lane + 32 * x];
#pragma unroll
      for (int i = 0; i < RW; ++i) {
        const float4 p4 = *reinterpret_cast<const float4*>(&sm.ps[warp * RW + i][k]);
        const float p[4] = {p4.x, p4.y, p4.z, p4.w};
        const uint32_t bits = seen[i] >> k;
#pragma unroll
        for (int y = 0; y < 4; ++y)
          if (bits & (1u << y)) {
#pragma unroll
            for (int x = 0; x < PER; ++x) o[i][x] = fmaf(p[y], v[y][x], o[i][x]);
          }
      }
    }
    __syncthreads();  // the buffer may be copied into again
  }

#pragma unroll
  for (int i = 0; i < RW; ++i) {
    const int r = warp * RW + i;
    if (r >= rows) break;
    float l = l_part[i];
#pragma unroll
    for (int x = 16; x; x >>= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
    if (!alive[i]) l = 0.f;  // pruned: weighs nothing
    const int hq = g * G + (row0 + r) % G;
    if (n_split == 1) {
      // no weight at all: zero; a NaN sum stays NaN
      const float inv = l == 0.f ? 0.f : 1.f / l;
      float* op = static_cast<float*>(a.out) + ((s.t0 + tok[i]) * a.Hq + hq) * D;
#pragma unroll
      for (int x = 0; x < PER; ++x) op[lane + 32 * x] = l == 0.f ? 0.f : o[i][x] * inv;
    } else {
      const int64_t row = ((int64_t)b * a.n_max + tok[i]) * a.Hq + hq;
      float* po = part_o + (row * n_split + split) * D;
#pragma unroll
      for (int x = 0; x < PER; ++x) po[lane + 32 * x] = o[i][x];
      if (lane == 0) part_ml[row * n_split + split] = make_float2(m_run[i], l);
    }
  }
}

// Joins the key splits of one (token, head) row.
template <int D>
__global__ void __launch_bounds__(D)
tree_combine_kernel(const __grid_constant__ TreeArgs a, int n_split,
                    const float* __restrict__ part_o, const float2* __restrict__ part_ml) {
  __shared__ float w[64];
  pdl_trigger();
  pdl_wait();
  const int hq = blockIdx.x % a.Hq;
  const int i = blockIdx.x / a.Hq % a.n_max, b = blockIdx.x / a.Hq / a.n_max;
  const int64_t row = ((int64_t)b * a.n_max + i) * a.Hq + hq;
  const int tid = threadIdx.x, lane = tid & 31;
  const TreeSeq s = tree_seq(a, b);
  if (i >= s.n) return;
  // every warp finds the weights of all splits, two a lane (n_split <= 64)
  float2 ml[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    ml[h] = make_float2(-INFINITY, 0.f);
    if (lane + 32 * h < n_split) ml[h] = part_ml[row * n_split + lane + 32 * h];
  }
  float m = fmaxf(ml[0].y == 0.f ? -INFINITY : ml[0].x, ml[1].y == 0.f ? -INFINITY : ml[1].x);
#pragma unroll
  for (int x = 16; x; x >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
  float l = 0.f;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    // (a split without weight is left out: its O may hold NaN)
    const float wt =
        ml[h].y == 0.f ? 0.f : m == -INFINITY ? 1.f : exp2f(ml[h].x - m);
    if (ml[h].y != 0.f) l += wt * ml[h].y;
    if (tid < 32) w[lane + 32 * h] = wt;
  }
#pragma unroll
  for (int x = 16; x; x >>= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
  __syncthreads();
  float acc = 0.f;
#pragma unroll 8
  for (int sp = 0; sp < n_split; ++sp) {
    const float v = part_o[(row * n_split + sp) * D + tid];
    if (w[sp] != 0.f) acc = fmaf(w[sp], v, acc);
  }
  static_cast<float*>(a.out)[((s.t0 + i) * a.Hq + hq) * D + tid] = l == 0.f ? 0.f : acc / l;
}

template <int D>
int dispatch_simt(const TreeArgs& a, const TreePlan& p, void* ws, cudaStream_t s) {
  float* part_o = static_cast<float*>(ws);
  float2* part_ml =
      reinterpret_cast<float2*>(static_cast<unsigned char*>(ws) + p.po_bytes);
  const dim3 grid((unsigned)p.n_split, (unsigned)p.n_blk, (unsigned)(a.B * a.H));
  auto go = [&](auto kern, size_t smem) -> int {
    if (int rc = ensure_smem_attr(reinterpret_cast<const void*>(kern), (int)smem)) return rc;
    return launch_pdl(kern, grid, dim3(kThreads), smem, s, a, p.n_split, part_o, part_ml);
  };
  int rc = p.rw == 1   ? go(tree_simt_kernel<D, 1>, sizeof(SimtSmem<D, 1>))
           : p.rw == 2 ? go(tree_simt_kernel<D, 2>, sizeof(SimtSmem<D, 2>))
           : p.rw == 4 ? go(tree_simt_kernel<D, 4>, sizeof(SimtSmem<D, 4>))
                       : go(tree_simt_kernel<D, 8>, sizeof(SimtSmem<D, 8>));
  if (rc || p.n_split == 1) return rc;
  return launch_pdl(tree_combine_kernel<D>, dim3((unsigned)((int64_t)a.B * a.n_max * a.Hq)),
                    dim3(D), 0, s, a, p.n_split, static_cast<const float*>(part_o),
                    static_cast<const float2*>(part_ml));
}

// Whether tree_attn_few.cu takes a call, by the rows R of a KV head.  bf16: one
// row tile of 16 (with two, 17 to 32 rows, a slice took a warp so long that
// loads waited: 16 sequences x 8,220 keys, 32 rows, 125 us against
// tree_attn_tc.cu's 103 for 36; 64 sequences x 100 keys 46 us against 24).
// fp32: once there are 2e7 products of a row and a key's element in the lengths
// that the buffers allow: its slices and merge take 11 to 14 us at the least,
// where tree_simt_kernel takes 6 to 9 (2 sequences of 16 tokens over 322 keys,
// 2.7e6 products: 12.5 against 8.9; 4 sequences x 4,104 keys, 4 / 16 / 32 rows,
// 1.7e7 to 1.3e8: 22 / 26 / 34 against 23 / 29 / 42; 8 x 32,104 keys: 147 / 150 /
// 282 against 218 / 444 / 718).  The lengths themselves are on the device: with
// a block table 16 times as wide as its sequences need, that first call takes
// 12.7 us.
bool takes_few(msa_dtype dt, int B, int n_max, int Hq, int H, int D, int m_cap, int max_pages,
               int page_size) {
  const int rows = n_max * (Hq / H);
  if (dt == MSA_BF16) return rows <= 16;
  const double keys = (double)m_cap + (double)max_pages * page_size;
  return (double)rows * B * H * keys * D > 2e7;
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
  const bool few = takes_few(dt, B, n_max, Hq, H, D, m_cap, max_pages, page_size);
  const int64_t keys = (int64_t)m_cap + (int64_t)max_pages * page_size;
  const size_t need = few               ? tree_few_workspace_size(n_max, a.G, D)
                      : dt == MSA_F32 ? p.total
                                      : tree_tc_workspace_size(B, n_max, a.G, H, D, keys);
  if (need && (!ws || ws_bytes < need || !aligned16(ws))) return MSA_ERR_WORKSPACE;
  if (few) return tree_few_launch(dt, a, D, ws, s);
  if (dt == MSA_BF16) return tree_tc_launch(a, D, ws, s);
  return D == 64 ? dispatch_simt<64>(a, p, ws, s) : dispatch_simt<128>(a, p, ws, s);
}

}  // namespace
}  // namespace msa

extern "C" size_t msa_tree_attn_workspace_size(msa_dtype dt, int B, int n_max, int Hq, int H,
                                               int D, int m_cap, int max_pages, int page_size) {
  using namespace msa;
  if (tree_shape(dt, B, n_max, Hq, H, D, m_cap, max_pages, page_size)) return 0;
  if (takes_few(dt, B, n_max, Hq, H, D, m_cap, max_pages, page_size))
    return tree_few_workspace_size(n_max, Hq / H, D);
  if (dt == MSA_BF16)
    return tree_tc_workspace_size(B, n_max, Hq / H, H, D,
                                  (int64_t)m_cap + (int64_t)max_pages * page_size);
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
