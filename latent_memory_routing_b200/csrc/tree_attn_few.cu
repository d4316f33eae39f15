// bf16 attention for drafted token trees over [memory ; paged cache ; drafted
// tokens] when a KV head has few query rows (method and semantics:
// tree_attn.cu): plain decode and small trees, R = n G <= 16 rows.
//
// Mathematics.  As tree_attn_tc.cu: S = Q K^T, p = 2^(scale log2(e) s - m),
// O += bf16(p) V, l += p, one pass over the keys.
//
// What bounds it.  4 D bytes a key and KV head against 4 R D operations: HBM,
// by far, so all that matters is bytes in flight and what happens at the ends
// of short sequences.  A 128-row tensor-core tile would spend most of its
// latency on handshakes for rows that do not exist (64 sequences x 2,268 keys,
// one token each: 114 us in tree_attn_tc.cu, 103 here with the merge, 5.8
// TB/s); here every warp is a worker of its own:
//   * The 16-key slices of all (sequence, KV head) items stand in one line,
//     cut into one contiguous range a worker (neighbours on different SMs).  An item inside one range is
//     written directly, one cut by a border as fp32 partials (at most two a
//     warp) that a second launch merges in a fixed order.
//   * A warp's lane 0 copies slices of K and V by TMA into the warp's own ring
//     (a slice never crosses a page: pages hold a multiple of 16 rows), waits
//     on its own barriers, and no warp waits for another.
//   * A slice is 16 x 16 of S and 16 x D of O on the warp-level
//     tensor instructions (m16n8k16): the accumulators stay in registers and
//     P's fragment is S's.  Their rate is no limit: a slice's 64 instructions
//     against the 8 KB that its SM receives in 350 cycles.
//   * In a slice that reaches past the sequence's rows or into its drafted
//     rows, unseen scores become -inf, V rows past the end zero, and
//     non-finite drafted values are taken out of V (0 times them would reach
//     every row) and added at the end for the rows that see them.
#include <algorithm>
#include <cmath>

#include "attn_tc.cuh"
#include "tc_ptx.cuh"
#include "tree_attn.cuh"

namespace msa {
namespace {

constexpr int kSlice = 16;                // keys of a slice
constexpr int kWarps = 8;                 // workers of a CTA, one CTA an SM
constexpr int kFewThreads = 32 * kWarps;
constexpr float kWholeItem = 8.f, kSqRange = 128.f;  // slices of an item
constexpr float kRescaleLog2 = 8.f;

template <int D> struct FC {
  static constexpr int KB = D / 64;                 // 64-dim blocks of a slice
  static constexpr int BLK = kSlice * 128;          // 2 KB
  static constexpr int SLICE = 2 * KB * BLK;        // K and V of a slice
  static constexpr int DEPTH = 24576 / SLICE;       // slices in flight: 24 KB a warp
  static constexpr size_t SMEM = 1024 + (size_t)kWarps * DEPTH * SLICE;
};

struct FewAux {
  int64_t pre[kFewThreads + 1];          // slices before each thread's sequences
  TreeSeq seq[kFewThreads];              // the sequences, where a thread has one at most
  uint64_t full[kWarps][6];              // ring slots (DEPTH <= 6)
  uint32_t anc[kWarps][16];           // what each row's token sees of its tree
  signed char par[kWarps][128];
};

__device__ __forceinline__ float ex2a(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&h);
}
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// c (16 x 8, fp32) += a (16 x 16) b (16 x 8).
__device__ __forceinline__ void mma16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                      uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ int slices(int rows) { return (rows + kSlice - 1) / kSlice; }
__device__ __forceinline__ int seq_slices(const TreeSeq& s) {
  return s.n == 0 ? 0 : slices(s.M) + slices(s.cache);
}

// A worker's place in its range: slice j of item (b, g); `left` slices of the
// range from here on.
struct Cursor {
  TreeSeq s;
  int b, g, j, nt;
  int64_t left;
  __device__ __forceinline__ void size() { nt = seq_slices(s); }
  // To slice 0 of the next item that has any (only while left > 0).
  template <typename Seq>
  __device__ __forceinline__ void next_item(int H, Seq seq) {
    j = 0;
    if (++g < H) return;
    g = 0;
    do {
      s = seq(++b);
      size();
    } while (nt == 0);
  }
};

template <int D>
__global__ void __launch_bounds__(kFewThreads, 1)
tree_few_kernel(const __grid_constant__ CUtensorMap tm_km,
                const __grid_constant__ CUtensorMap tm_vm,
                const __grid_constant__ CUtensorMap tm_kp,
                const __grid_constant__ CUtensorMap tm_vp, const __grid_constant__ TreeArgs a,
                int part_rows, float* __restrict__ part_o, float2* __restrict__ part_ml,
                TreeCut* __restrict__ cuts) {
  using C = FC<D>;
  pdl_trigger();  // the merge: its blocks come as this grid's leave
  pdl_wait();
  extern __shared__ __align__(1024) unsigned char dsm[];
  __shared__ FewAux aux;
  unsigned char* base = tc::smem_align<1024>(dsm);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  unsigned char* ring = base + warp * C::DEPTH * C::SLICE;
  uint64_t* full = aux.full[warp];
  if (lane == 0) {
    for (int i = 0; i < C::DEPTH; ++i) tc::mbar_init(&full[i], 1);
    tc::fence_mbar_init();
  }
  if (tid == 0) {
    tc::tma_prefetch_desc(&tm_kp);
    tc::tma_prefetch_desc(&tm_vp);
  }

  // The slices of all sequences, a run of sequences a thread, scanned over
  // the CTA's threads.
  const int per = (a.B + kFewThreads - 1) / kFewThreads;
  int64_t items;
  {
    int64_t mine = 0;
    for (int b = min(a.B, tid * per); b < min(a.B, (tid + 1) * per); ++b) {
      const TreeSeq s = tree_seq(a, b);
      if (s.error && blockIdx.x == 0) record_error(a.status, s.error);
      aux.seq[tid] = s;
      mine += (int64_t)seq_slices(s) * a.H;
    }
    items = (int64_t)(per == 1 ? __syncthreads_count(mine > 0) : a.B) * a.H;
    int64_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) aux.pre[warp] = incl;
    __syncthreads();
    int64_t before = 0, total = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
      if (i < warp) before += aux.pre[i];
      total += aux.pre[i];
    }
    __syncthreads();
    aux.pre[tid] = before + incl - mine;
    if (tid == 0) aux.pre[kFewThreads] = total;
    __syncthreads();
  }
  const int64_t total = aux.pre[kFewThreads];
  const int64_t worker = (int64_t)warp * gridDim.x + blockIdx.x;  // few: on as many SMs
  // Short items stay whole, a worker each.  Of a long one a range costs its
  // length and the merge their number, so the least length goes with the root
  // of the item's; one slice is too little where that would fill every worker.
  // (33 sequences of 9 keys: 33 us with ranges of 6 slices at least, 10; one
  // item of 125 slices: 14 with 6, 10.5; of 1,000: 18 with ranges of one, 14.)
  const int64_t all = (int64_t)gridDim.x * kWarps;
  const float mean = (float)total / (float)max(items, (int64_t)1);
  const int64_t least =
      max((int64_t)(total <= all ? 1 : 3), (int64_t)ceilf(sqrtf(mean / kSqRange)));
  const int64_t n_work = min(
      all, mean <= kWholeItem ? min(items, total) : (total + least - 1) / least);
  auto range_lo = [&](int64_t i) { return i * total / n_work; };
  const int64_t lo = worker < n_work ? range_lo(worker) : 0;
  const int64_t hi = worker < n_work ? range_lo(worker + 1) : 0;
  TreeCut cut{0, 0, 0, 0, -1};
  if (lo >= hi) {
    if (lane == 0) cuts[worker] = cut;
    return;
  }

  // sequence b (shared memory: a read at an item's start is on the way of its
  // loads)
  auto seq = [&](int b) -> TreeSeq {
    if (per == 1) return aux.seq[b];
    return tree_seq(a, b);
  };
  Cursor ld;  // the slice to load next
  {
    // the last thread whose sequences begin at or before slice lo
    int t = 0;
    for (int i = 0; i < kFewThreads; i += 32) {
      const uint32_t m = __ballot_sync(0xffffffffu, aux.pre[i + lane] <= lo);
      if (m) t = i + 31 - __clz(m);
    }
    int64_t at = aux.pre[t];
    ld.b = t * per;
    for (;;) {  // (its run holds lo, so this ends)
      ld.s = seq(ld.b);
      ld.size();
      const int64_t n = (int64_t)ld.nt * a.H;
      if (lo < at + n || ld.b + 1 >= a.B) break;
      at += n;
      ++ld.b;
    }
    const int64_t off = lo - at;
    ld.g = (int)(off / ld.nt);
    ld.j = (int)(off - (int64_t)ld.g * ld.nt);
    ld.left = hi - lo;
  }
  Cursor cu = ld;  // the slice to compute next
  if (ld.j > 0 && range_lo(worker - 1) <= lo - ld.j) {
    // the first border inside this item: its last part holds slice `end`
    const int64_t end = lo - ld.j + ld.nt - 1;
    int64_t c = min(n_work - 1, end * n_work / total);
    while (c + 1 < n_work && range_lo(c + 1) <= end) ++c;
    while (range_lo(c) > end) --c;
    cut.last = (int)c;
    cut.t0 = ld.s.t0;
    cut.g = ld.g;
    cut.rows = ld.s.n * a.G;
  }
  if (lane == 0) cuts[worker] = cut;

  // ------------------------------------------------------------------ loads
  // lane i holds the first tensor-map row of slice ids0 + i of the item
  int ids = -1, ids0 = 0;
  bool ids_fresh = true;
  auto issue = [&](int slot) {
    if (ld.left == 0) return;
    const int n_ms = slices(ld.s.M);
    if (ids_fresh || ld.j >= ids0 + 32) {
      ids0 = ld.j;
      ids = -1;
      const int j = ids0 + lane;
      if (j < n_ms) {
        ids = ld.b * a.m_cap + j * kSlice;
      } else if (j < ld.nt) {
        const int r0 = (j - n_ms) * kSlice;
        const int pg = a.block_table[(int64_t)ld.b * a.max_pages + r0 / a.page_size];
        if (pg >= 0 && pg < a.n_pages)
          ids = (pg * a.H + ld.g) * a.page_size + r0 % a.page_size;
        else
          record_error(a.status, MSA_ERR_INVALID_ARG);
      }
      ids_fresh = false;
    }
    const int row = __shfl_sync(0xffffffffu, ids, ld.j - ids0);
    if (lane == 0) {
      tc::mbar_arrive_expect_tx(&full[slot], row >= 0 ? C::SLICE : 0);
      if (row >= 0) {
        const bool mem = ld.j < n_ms;
        unsigned char* d = ring + slot * C::SLICE;
#pragma unroll
        for (int kb = 0; kb < C::KB; ++kb) {
          tc::tma_load_3d(d + kb * C::BLK, mem ? &tm_km : &tm_kp, &full[slot], kb * 64,
                          mem ? ld.g : 0, row);
          tc::tma_load_3d(d + (C::KB + kb) * C::BLK, mem ? &tm_vm : &tm_vp, &full[slot], kb * 64,
                          mem ? ld.g : 0, row);
        }
      }
    }
    --ld.left;
    if (++ld.j == ld.nt && ld.left > 0) {
      ld.next_item(a.H, seq);
      ids_fresh = true;
    }
  };
#pragma unroll 1
  for (int i = 0; i < C::DEPTH; ++i) issue(i);

  // ---------------------------------------------------------------- compute
  const int c2 = 2 * (lane & 3);  // this thread's columns of an 8-column tile
  const int r4 = lane >> 2;       // its rows of a 16-row tile: r4, r4 + 8
  // ldmatrix: this lane's row and 16-byte piece of a 16 x 16 block
  const int kr = ((lane >> 4) << 3) + (lane & 7), kc = (lane >> 3) & 1;
  const int vr = (((lane >> 3) & 1) << 3) + (lane & 7), vc = lane >> 4;
  const uint32_t ring_u = tc::smem_u32(ring);
  bool ok = true;
  int slot = 0;
  uint32_t ph = 0;
  while (cu.left > 0 && ok) {
    // an item's share: its queries, trees, and slices
    const TreeSeq s = cu.s;
    const int rows = s.n * a.G, n_ms = slices(s.M);
    const int cnt = (int)min((int64_t)(cu.nt - cu.j), cu.left), j_lo = cu.j;
    const int part = j_lo > 0 ? 0 : cnt < cu.nt ? 1 : -1;
    uint32_t qf[D / 16][4];
    int64_t out_row[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = r4 + 8 * h;
      out_row[h] = r < rows ? (s.t0 + r / a.G) * a.Hq + cu.g * a.G + r % a.G : (int64_t)-1;
      const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + out_row[h] * D + c2;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        qf[kk][h] = r < rows ? *reinterpret_cast<const uint32_t*>(q + kk * 16) : 0u;
        qf[kk][2 + h] = r < rows ? *reinterpret_cast<const uint32_t*>(q + kk * 16 + 8) : 0u;
      }
    }
    // ancestor sets, a lane a row
    __syncwarp();
    if (a.parents) {
      for (int i = lane; i < s.n; i += 32) {
        int p = a.parents[s.t0 + i];
        if (p >= i) {  // a parent comes before its child
          record_error(a.status, MSA_ERR_INVALID_ARG);
          p = -2;
        }
        aux.par[warp][i] = (signed char)max(p, -2);
      }
      __syncwarp();
    }
    if (lane < rows) {  // at most 16 rows, so at most 16 tokens
      uint32_t m = 0;
      int x = lane / a.G;
      if (a.parents) {
        do {
          m |= 1u << x;
          x = aux.par[warp][x];
        } while (x >= 0);
        if (x != -1) m = 0;  // pruned: sees nothing
      } else {
        m = (2u << x) - 1;
      }
      aux.anc[warp][lane] = m;
    }
    __syncwarp();

    float o[D / 8][4], m_ref[2], l[2];
    m_ref[0] = m_ref[1] = -INFINITY;
    l[0] = l[1] = 0.f;
#pragma unroll
    for (int d = 0; d < D / 8; ++d)
#pragma unroll
      for (int x = 0; x < 4; ++x) o[d][x] = 0.f;
    bool any_bad = false;

#pragma unroll 1
    for (int i = 0; i < cnt; ++i) {
      const int j = j_lo + i;
      const bool mem = j < n_ms;
      const int key0 = (mem ? j : j - n_ms) * kSlice;
      const int n_rows = (mem ? s.M : s.cache) - key0;
      const bool all = key0 + kSlice <= (mem ? s.M : s.L);  // every row sees every key
      ok = tc::mbar_wait(&full[slot], ph);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      const uint32_t kb_u = ring_u + slot * C::SLICE, vb_u = kb_u + C::KB * C::BLK;

      float sc[2][4];
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int x = 0; x < 4; ++x) sc[t][x] = 0.f;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        uint32_t b[4];
        ldsm4(kb_u + (kk >> 2) * C::BLK + kr * 128 + (((2 * (kk & 3) + kc) ^ (kr & 7)) << 4), b);
        mma16(sc[0], qf[kk], b[0], b[1]);
        mma16(sc[1], qf[kk], b[2], b[3]);
      }
      if (!all) {
        const int off = s.L - key0;  // column of the first drafted key
        const uint32_t in = n_rows >= 16 ? 0xffffu : (1u << n_rows) - 1;  // n_rows >= 1
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t vis = in;
          if (!mem) {
            const uint32_t anc = aux.anc[warp][r4 + 8 * h];
            vis &= off >= 16   ? 0xffffu
                   : off >= 0  ? (((1u << off) - 1) | (anc << off))
                   : off > -32 ? anc >> -off
                               : 0u;
          }
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int x = 0; x < 2; ++x)
              if (!((vis >> (8 * t + c2 + x)) & 1)) sc[t][2 * h + x] = -INFINITY;
        }
        // clean V: rows past the end, non-finite drafted values
        unsigned char* v = ring + slot * C::SLICE + C::KB * C::BLK;
        bool bad = false;
        for (int c = lane; c < kSlice * D / 8; c += 32) {
          const int r = (c & 127) >> 3;  // 128 pieces of 16 bytes a block
          uint4* p = reinterpret_cast<uint4*>(v + (c >> 7) * C::BLK + (c & 127) * 16);
          if (r >= n_rows) {
            *p = make_uint4(0, 0, 0, 0);
          } else if (!mem && key0 + r >= s.L && s.n > 1) {
            const uint4 x = *p;
            const uint4 y =
                make_uint4(finite_bf16x2(x.x), finite_bf16x2(x.y), finite_bf16x2(x.z),
                           finite_bf16x2(x.w));
            if (x.x != y.x || x.y != y.y || x.z != y.z || x.w != y.w) {
              *p = y;
              bad = true;
            }
          }
        }
        any_bad |= __any_sync(0xffffffffu, bad) != 0;
        tc::fence_proxy_async_smem();  // before the slot's next load
        __syncwarp();
      }
      float mx[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        mx[h] = fmaxf(fmaxf(sc[0][2 * h], sc[0][2 * h + 1]),
                      fmaxf(sc[1][2 * h], sc[1][2 * h + 1]));
        mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 1));
        mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 2));
        mx[h] *= a.qscale;
      }
      // the reference maximum moves only when a slice exceeds it by 2^8
      const bool g0 = mx[0] > m_ref[0] + kRescaleLog2, g1 = mx[1] > m_ref[1] + kRescaleLog2;
      if (__any_sync(0xffffffffu, g0 || g1)) {
        const float al0 = !g0 ? 1.f : m_ref[0] == -INFINITY ? 0.f : ex2a(m_ref[0] - mx[0]);
        const float al1 = !g1 ? 1.f : m_ref[1] == -INFINITY ? 0.f : ex2a(m_ref[1] - mx[1]);
        if (g0) m_ref[0] = mx[0];
        if (g1) m_ref[1] = mx[1];
        l[0] *= al0;
        l[1] *= al1;
#pragma unroll
        for (int d = 0; d < D / 8; ++d) {
          o[d][0] *= al0;
          o[d][1] *= al0;
          o[d][2] *= al1;
          o[d][3] *= al1;
        }
      }
      uint32_t pf[4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float nm = m_ref[h] == -INFINITY ? 0.f : -m_ref[h];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const float p0 = ex2a(fmaf(sc[t][2 * h], a.qscale, nm));
          const float p1 = ex2a(fmaf(sc[t][2 * h + 1], a.qscale, nm));
          l[h] += p0 + p1;
          pf[2 * t + h] = pack2(p0, p1);
        }
      }
#pragma unroll
      for (int d = 0; d < D / 16; ++d) {
        uint32_t b[4];
        ldsm4t(vb_u + (d >> 2) * C::BLK + vr * 128 + (((2 * (d & 3) + vc) ^ (vr & 7)) << 4), b);
        mma16(o[2 * d], pf, b[0], b[1]);
        mma16(o[2 * d + 1], pf, b[2], b[3]);
      }
      __syncwarp();  // every lane has read the slot
      issue(slot);
      if (++slot == C::DEPTH) {
        slot = 0;
        ph ^= 1;
      }
    }
    if (!ok) break;

    // write the item's share
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = r4 + 8 * h;
      float lr = l[h];
      lr += __shfl_xor_sync(0xffffffffu, lr, 1);
      lr += __shfl_xor_sync(0xffffffffu, lr, 2);
      if (r >= rows) continue;
      const uint32_t anc = aux.anc[warp][r];
      if (anc == 0) lr = 0.f;  // pruned
      const int64_t prow = (worker * 2 + max(part, 0)) * part_rows + r;
      const float inv = lr == 0.f ? 0.f : part >= 0 ? 1.f : 1.f / lr;
#pragma unroll
      for (int d = 0; d < D / 8; ++d) {
        // (a row without weight: its O may hold 0 times NaN)
        const float x = inv == 0.f ? 0.f : o[d][2 * h] * inv;
        const float y = inv == 0.f ? 0.f : o[d][2 * h + 1] * inv;
        if (part < 0)
          *reinterpret_cast<uint32_t*>(out + out_row[h] * D + d * 8 + c2) = pack2(x, y);
        else
          *reinterpret_cast<float2*>(part_o + prow * D + d * 8 + c2) = make_float2(x, y);
      }
      if (part >= 0 && c2 == 0) part_ml[prow] = make_float2(m_ref[h], lr);
      if (!any_bad) continue;
      // drafted values taken out of V, added for the rows that see them
#pragma unroll 1
      for (int t = 0; t < s.n; ++t) {
        const int kr2 = s.L + t, j = n_ms + kr2 / kSlice;
        if (!((anc >> t) & 1) || j < j_lo || j >= j_lo + cnt || kr2 >= s.cache) continue;
        const int pg = a.block_table[(int64_t)cu.b * a.max_pages + kr2 / a.page_size];
        if (pg < 0 || pg >= a.n_pages) continue;
        const __nv_bfloat16* v =
            static_cast<const __nv_bfloat16*>(a.v_pages) +
            (((int64_t)pg * a.H + cu.g) * a.page_size + kr2 % a.page_size) * D;
#pragma unroll 1
        for (int d = 0; d < D / 4; ++d) {  // this thread's columns
          const int col = 8 * (d >> 1) + c2 + (d & 1);
          const float f = __bfloat162float(v[col]);
          if (isfinite(f)) continue;
          if (part < 0) {
            __nv_bfloat16* p = out + out_row[h] * D + col;
            *p = __float2bfloat16(__bfloat162float(*p) + f);
          } else {
            part_o[prow * D + col] += f;
          }
        }
      }
    }
    cu.left -= cnt;
    cu.j += cnt;
    if (cu.left > 0) cu.next_item(a.H, seq);
  }
  if (!ok) {
    if (lane == 0) record_error(a.status, MSA_ERR_TIMEOUT);
    // loads still in flight land before the CTA exits
    for (int i = 0; i < C::DEPTH; ++i) {
      tc::mbar_wait(&full[slot], ph);
      if (++slot == C::DEPTH) {
        slot = 0;
        ph ^= 1;
      }
    }
  }
}

struct FewPlan {
  int part_rows;
  size_t po_bytes, ml_bytes, total;
};
FewPlan few_plan(int n_max, int G, int D) {
  FewPlan p{};
  p.part_rows = n_max * G;
  const size_t parts = 2 * (size_t)num_sms() * kWarps * p.part_rows;
  p.po_bytes = round_up(parts * D * sizeof(float), 256);
  p.ml_bytes = round_up(parts * sizeof(float2), 256);
  p.total = p.po_bytes + p.ml_bytes + round_up((size_t)num_sms() * kWarps * sizeof(TreeCut), 256);
  return p;
}

template <int D>
int launch_few(const TreeArgs& a, void* ws, cudaStream_t s) {
  using C = FC<D>;
  const FewPlan p = few_plan(a.n_max, a.G, D);
  unsigned char* w = static_cast<unsigned char*>(ws);
  float* part_o = reinterpret_cast<float*>(w);
  float2* part_ml = reinterpret_cast<float2*>(w + p.po_bytes);
  TreeCut* cuts = reinterpret_cast<TreeCut*>(w + p.po_bytes + p.ml_bytes);
  CUtensorMap km, vm, kp, vp;
  const int64_t page_rows = (int64_t)a.n_pages * a.H * a.page_size;
  bool ok = tma_map_sw128_bf16(&kp, a.k_pages, D, 1, page_rows, 1, kSlice) &&
            tma_map_sw128_bf16(&vp, a.v_pages, D, 1, page_rows, 1, kSlice);
  if (a.m_cap > 0)
    ok = ok && tma_map_sw128_bf16(&km, a.k_mem, D, a.H, (int64_t)a.B * a.m_cap, 1, kSlice) &&
         tma_map_sw128_bf16(&vm, a.v_mem, D, a.H, (int64_t)a.B * a.m_cap, 1, kSlice);
  else
    km = kp, vm = vp;  // never loaded from
  if (!ok) return note_cuda(cudaErrorInvalidValue);
  auto kern = tree_few_kernel<D>;
  if (int rc = ensure_smem_attr(reinterpret_cast<const void*>(kern), (int)C::SMEM)) return rc;
  const unsigned grid = (unsigned)num_sms();
  if (int rc = launch_pdl(kern, dim3(grid), dim3(kFewThreads), C::SMEM, s, km, vm, kp, vp, a,
                          p.part_rows, part_o, part_ml, cuts))
    return rc;
  return tree_merge_launch(a, D, (int)grid, kWarps, p.part_rows, part_o, part_ml, cuts, s);
}

}  // namespace

// One row tile of the warp's instructions.  (With two, 17 to 32 rows, a slice
// took a warp so long that loads waited: 16 sequences x 8,220 keys, 32 rows,
// 125 us against tree_attn_tc.cu's 103 for 36; 64 sequences x 100 keys 46 us
// against 24.)
bool tree_few_takes(int n_max, int G) { return n_max * G <= 16; }
size_t tree_few_workspace_size(int n_max, int G, int D) { return few_plan(n_max, G, D).total; }

int tree_few_launch(const TreeArgs& a, int D, void* ws, cudaStream_t s) {
  return D == 64 ? launch_few<64>(a, ws, s) : launch_few<128>(a, ws, s);
}

}  // namespace msa
