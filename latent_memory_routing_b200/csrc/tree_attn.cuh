// Attention for drafted token trees over [memory ; paged cache ; tree]:
// shared by the fp32 kernel and the entry point (tree_attn.cu) and the
// tensor-core kernel (tree_attn_tc.cu).
#pragma once

#include "msa_common.cuh"

namespace msa {

constexpr int kTreeMax = 128;  // drafted tokens of a sequence at most

struct TreeArgs {
  int B, n_max, Hq, H, G;
  int64_t n_tok;
  const void* q;
  const int64_t* tok_offsets;
  const int32_t* parents;  // NULL: a chain
  const void *k_mem, *v_mem;
  const int32_t* mem_len;
  int m_cap;
  const void *k_pages, *v_pages;
  int n_pages, page_size, max_pages;
  const int32_t *block_table, *cache_len;
  float qscale;  // softmax scale times log2 e
  void* out;
  int* status;
};

// One sequence of a call, its lengths brought into range.  Keys are
// numbered memory rows [0, M), cached rows [M, M + L), drafted [M + L, keys).
struct TreeSeq {
  int64_t t0;  // first token
  int n;       // drafted tokens
  int M, L;    // memory rows, cached rows
  int cache;   // cached and drafted rows: L + n, or the block table's capacity
  int error;   // what was out of range (a status code), 0 if nothing
};

__device__ __forceinline__ TreeSeq tree_seq(const TreeArgs& a, int b) {
  TreeSeq s;
  s.error = 0;
  s.t0 = a.tok_offsets[b];
  const int64_t t1 = a.tok_offsets[b + 1];
  if (s.t0 < 0 || t1 < s.t0 || t1 > a.n_tok) {
    s.error = MSA_ERR_INVALID_ARG;
    s.t0 = 0;
    s.n = 0;
  } else if (t1 - s.t0 > a.n_max) {
    s.error = MSA_ERR_INVALID_ARG;
    s.n = a.n_max;
  } else {
    s.n = (int)(t1 - s.t0);
  }
  s.M = a.m_cap > 0 ? a.mem_len[b] : 0;
  if (s.M < 0 || s.M > a.m_cap) {
    s.error = MSA_ERR_INVALID_ARG;
    s.M = min(max(s.M, 0), a.m_cap);
  }
  const int cap = a.max_pages * a.page_size;
  s.L = a.cache_len[b];
  if (s.L < 0) {
    s.error = MSA_ERR_INVALID_ARG;
    s.L = 0;
  }
  if (s.L > cap - s.n) {  // cap - n cannot overflow
    s.error = MSA_ERR_CAPACITY;
    s.L = min(s.L, cap);
    s.cache = cap;
  } else {
    s.cache = s.L + s.n;
  }
  return s;
}

// What each drafted token sees of its tree: anc[i] has bit j set when token j
// is token i or one of its ancestors; a pruned token (or one below a pruned
// token) sees nothing and gets alive[i] = 0.  Ancestor sets double in reach
// each round (7 rounds cover a depth of 128).  Called by a whole CTA of at
// least kTreeMax threads; ends with a barrier.
struct TreeMask {
  uint4 anc[kTreeMax];
  int up[kTreeMax];
};

__device__ __forceinline__ uint4 or4(uint4 a, uint4 b) {
  return make_uint4(a.x | b.x, a.y | b.y, a.z | b.z, a.w | b.w);
}

// up[i] of a finished mask: kTreeDead for a token that sees nothing.
constexpr int kTreeDead = -2;

// `bar` is a barrier over the calling threads, of index i (0 .. >= n - 1).
template <typename Bar>
__device__ __forceinline__ void tree_mask(const TreeArgs& a, const TreeSeq& s, TreeMask& m,
                                          int i, Bar bar) {
  uint4 anc = make_uint4(0, 0, 0, 0);
  int up = kTreeDead;
  if (i < s.n) {
    const int p = a.parents ? a.parents[s.t0 + i] : i - 1;
    if (p >= -1 && p < i) {
      up = p;
      const uint32_t bit = 1u << (i & 31);
      anc = make_uint4(i < 32 ? bit : 0, (i >> 5) == 1 ? bit : 0, (i >> 5) == 2 ? bit : 0,
                       (i >> 5) == 3 ? bit : 0);
    } else if (p >= i) {
      record_error(a.status, MSA_ERR_INVALID_ARG);  // a parent comes before its child
    }
    m.anc[i] = anc;
    m.up[i] = up;
  }
  bar();
  for (int reach = 1; reach < s.n; reach <<= 1) {
    uint4 pa = anc;
    int pu = up;
    if (up >= 0) {
      pa = or4(anc, m.anc[up]);
      pu = m.up[up];
    }
    bar();
    if (i < s.n) {
      anc = pa;
      up = pu;
      m.anc[i] = anc;
      m.up[i] = up;
    }
    bar();
  }
}

__device__ __forceinline__ bool tree_bit(const uint4& m, int j) {
  const uint32_t w = j < 64 ? (j < 32 ? m.x : m.y) : (j < 96 ? m.z : m.w);
  return (w >> (j & 31)) & 1;
}

// A bf16 pair with its non-finite halves (exponent all ones) replaced by 0.
__device__ __forceinline__ uint32_t finite_bf16x2(uint32_t w) {
  if ((w & 0x7f80u) == 0x7f80u) w &= 0xffff0000u;
  if ((w & 0x7f800000u) == 0x7f800000u) w &= 0xffffu;
  return w;
}

// What the merge of partials needs of an item whose first border between two
// workers' ranges lies at this worker's start: the parts are (worker - 1,
// slot 1) and (worker .. last, slot 0), rows [row0, row0 + rows) of the item.
struct TreeCut {
  int64_t t0;               // the sequence's first token
  int g, row0, rows, last;  // last < 0: nothing to merge here
};

// Merges the partials of ctas x per workers in a fixed order, into outputs in
// fp32 or bf16 (tree_attn_merge.cu): part (worker, slot) holds part_rows rows
// of fp32 O and (max, sum) in the base-2 domain.
int tree_merge_launch(const TreeArgs& a, bool f32, int D, int ctas, int per, int part_rows,
                      const float* part_o, const float2* part_ml, const TreeCut* cuts,
                      cudaStream_t s);

// A warp a worker (tree_attn_few.cu): up to 16 rows a KV head in bf16, any
// number in fp32.
size_t tree_few_workspace_size(int n_max, int G, int D);
int tree_few_launch(msa_dtype dt, const TreeArgs& a, int D, void* ws, cudaStream_t s);

// bf16 on tcgen05 (tree_attn_tc.cu): any shape the entry point takes.
// (keys: the most that the buffers allow a sequence.)
size_t tree_tc_workspace_size(int B, int n_max, int G, int H, int D, int64_t keys);
int tree_tc_launch(const TreeArgs& a, int D, void* ws, cudaStream_t s);

}  // namespace msa
