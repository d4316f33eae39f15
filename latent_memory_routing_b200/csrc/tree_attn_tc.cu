// bf16 attention for drafted token trees over [memory ; paged cache ; drafted
// tokens] on the tcgen05 tensor cores (method and semantics: tree_attn.cu).
//
// Mathematics.  The query rows of a KV head are (token, head of the group)
// pairs, R = n G of them; every row sees the same memory and cached keys, and
// of the drafted keys the bits of its ancestor set.  One pass over the keys
// with a running maximum and sum:
//   S = Q K^T (fp32), p = 2^(scale log2(e) s - m), O += bf16(p) V, l += p.
// The one rounding on the way is p's, to the MMA's operand type: it moves an
// output by at most 2^-8 of sum p |v| (the sums l take p unrounded; relative
// error over an output 0.0023, of which its own rounding is 0.0017).  A second
// bf16 term of p, as tree_attn_few.cu has, takes that away and half as many MMAs
// again, in the chain that sets the pace: 16 sequences, trees of up to 48 tokens
// over up to 8,220 keys, 103 -> 131 us; 2 x 150,065 keys, 64 tokens, 321 -> 424.
//
// What bounds it.  K and V are read once, 4 D bytes a key and KV head, for
// 4 R D operations: HBM up to about R = 256 rows, beyond that the tensor
// cores and the exponentials.  So the same tile shape serves all R: rows
// padded to the MMA's M = 128 cost tensor time that the stream hides.
// Measured (32 / 8 heads x 128): 16 sequences x 8,220 keys, 9 to 32 tokens
// each, 102 to 111 us (5.3 to 4.9 TB/s); 2 x 150,065 keys, 64 tokens, 312 us at
// 1,965 MHz and 378 under the power cap at 1,460 (1.01 to 0.83 PFLOP/s: the chain
// softmax -> P V -> S of each stream, 3,650 cycles a tile of which the tensor pipe
// works 2,048).
//
// Design.
//   * Even work: the 128-key tiles of all (sequence, KV head, row block)
//     items in one line, each item's behind kItemCost units that stand for its
//     start and end (without them a CTA of short items ended at 248,000
//     cycles, the others at 145,000; 16 sequences of unlike lengths up to 8,220
//     keys, up to 48 tokens: 128 us with 1, 108 with 3, 103 with 5, 104 with 8;
//     64 sequences x 164 keys, 64 tokens: 81, 78, 78, 74), cut into one contiguous
//     range a CTA (one CTA an SM).
//     An item inside one range is written directly; an item cut by a range
//     border is written as fp32 partials (at most two a CTA) that a second
//     launch merges in a fixed order.  The lengths stay on the device: every
//     CTA finds its range by a scan over the sequences.
//   * Two streams, each with its S tile (128 TMEM columns, overwritten by P
//     in bf16), its O accumulator (D columns) and its softmax warpgroup (a
//     thread a row).  Up to 128 rows (kQT = 1) the streams take the key tiles
//     in turn and join their (m, l, O) at an item's end, so a stream has the
//     time of two tiles; with kQT = 2 each holds 128 of an item's 256 rows and
//     both read the same tile.  129 to 192 rows, and more where the L2 holds
//     what two of them share (see tc_plan), are items of their own over the same
//     keys: 16 sequences of unlike lengths up to 8,253 keys, 33 tokens (304 MB),
//     76 us against 91 with kQT = 2, whose longest items end late.  (Of equal
//     lengths it is the other way round: 16 x 8,220 keys, 33 / 48 tokens, 187 / 192
//     us against 146 / 157.)
//   * Warp 0 loads K tiles, warp 3 V tiles (rings of their own: a K slot is
//     free after S, a V slot after P V), one lane a page (or 32 memory rows):
//     only pages that hold rows are read.  Warp 2 walks the range, publishes
//     the items with their trees and loads their queries.  Warp 1 issues the
//     MMAs.
//   * In a tile that reaches past the sequence's rows or into its drafted
//     rows, scores outside a row's 128-bit visibility mask become -inf, V
//     rows past the end are zeroed and non-finite drafted values taken out of
//     V (0 times them would reach every row); the rows that do see such a
//     token get it added at the end.
//   * Every wait is bounded; after a timeout all roles leave their loops.
#include <algorithm>
#include <cmath>

#include "attn_tc.cuh"
#include "tc_ptx.cuh"
#include "tree_attn.cuh"

namespace msa {
namespace {

constexpr int kKeys = 128;      // keys of a tile
constexpr int kMemRows = 32;    // memory rows of one load
constexpr int kTcThreads = 384; // 4 single warps, 2 softmax warpgroups
constexpr int kRing = 64 * 1024; // the K ring, and the V ring
constexpr int kStage = 4096;    // an output buffer of each softmax warp
constexpr int kSched = 3;       // published items
// Items whose `bad` is kept: one more than are published.  With items of one
// tile (kQT = 1) a stream may clean V for item k + 3, whose slot is free once
// everyone has read item k, while a warp of the other stream has yet to look at
// bad of item k; item k + 4 is that stream's own.
constexpr int kBad = kSched + 1;
constexpr int kReaders = 11;    // K warp, V warp, MMA, 8 softmax warps
constexpr int kItemCost = 5;    // what an item's start and end cost, in tiles
constexpr float kRescaleLog2 = 8.f;

template <int D> struct TC {
  static constexpr int KB = D / 64;
  static constexpr int TILE = KB * kKeys * 128;  // a K or V tile
  static constexpr int ST = kRing / TILE;        // ring slots
  static constexpr uint32_t IDESC_S = tc::idesc_bf16_f32(128, kKeys);
  static constexpr uint32_t IDESC_O = tc::idesc_bf16_f32(128, D) | (1u << 16);  // V MN-major
  // registers: 128 x LOW + 256 x HIGH = 384 x 168, the launch's allocation
  static constexpr int REG_LOW = 88, REG_HIGH = 208;
  static_assert(128 * REG_LOW + 256 * REG_HIGH == 384 * 168, "register split");
};

// A CTA's share of one item: key tiles [j_lo, j_lo + cnt) of a row block.
struct ItemE {
  int64_t t0;             // the sequence's first token
  int n, M, L, cache;     // as TreeSeq
  int b, g, row0, rows;   // row block: rows [row0, row0 + rows) of the n * G
  int j_lo, cnt;          // cnt < 0: no more items
  int part;               // partial slot, -1: the whole item, written directly
};

struct Aux {
  uint64_t kfull[4], kfree[4], vfull[4], vfree[4];  // ring slots, 4 at most
  uint64_t q_full[2], q_free[2], s_full[2], p_full[2], o_full[2], o_empty[2], ml_full;
  uint64_t sched_full[kSched], par_full[kSched], sched_empty[kSched];
  ItemE item[kSched];
  int bad[kBad];               // item ordinal + 1 where V held non-finite drafted values
  float2 ml[128];              // (m, l) of the stream that does not finish the item
  signed char par[kSched][128];  // the published items' parents: -1 root, -2 pruned
  int64_t start;               // first tile of the range within its sequence
  TreeSeq start_seq;
  int start_b;
  uint32_t tmem_base;
  int abort_flag;
};
// two Q buffers of 128 rows, the rings and the output buffers leave it this much
static_assert(1024 + 2 * 128 * 256 + 2 * kRing + 8 * kStage + sizeof(Aux) <= 227 * 1024,
              "shared memory");

__device__ __forceinline__ float ex2a(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float fmax3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&h);
}
__device__ __forceinline__ unsigned long long f2(float lo, float hi) {
  return (unsigned long long)__float_as_uint(lo) | ((unsigned long long)__float_as_uint(hi) << 32);
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
      "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]),
      "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]), "r"(v[21]),
      "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]),
      "r"(v[29]), "r"(v[30]), "r"(v[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
using u128 = unsigned __int128;
__device__ __forceinline__ u128 low_bits(int n) {  // bits 0 .. n-1
  return n <= 0 ? (u128)0 : n >= 128 ? ~(u128)0 : (((u128)1 << n) - 1);
}

// Tiles of one row block of a sequence, and its row blocks.
__device__ __forceinline__ int seq_tiles(const TreeSeq& s) {
  return s.n == 0 ? 0 : (s.M + kKeys - 1) / kKeys + (s.cache + kKeys - 1) / kKeys;
}

template <int D, int kQT>
__global__ void __launch_bounds__(kTcThreads, 1)
tree_tc_kernel(const __grid_constant__ CUtensorMap tm_q,
               const __grid_constant__ CUtensorMap tm_km, const __grid_constant__ CUtensorMap tm_vm,
               const __grid_constant__ CUtensorMap tm_kp, const __grid_constant__ CUtensorMap tm_vp,
               const __grid_constant__ TreeArgs a, int part_rows, int tile_rows,
               int q_rows, float* __restrict__ part_o, float2* __restrict__ part_ml,
               TreeCut* __restrict__ cuts) {
  using C = TC<D>;
  constexpr int KB = C::KB;
  const int blk_rows = tile_rows * kQT;  // rows of an item: whole tokens
  pdl_trigger();  // the merge: its blocks come as this grid's leave
  pdl_wait();
  extern __shared__ __align__(1024) unsigned char dsm[];
  unsigned char* base = tc::smem_align<1024>(dsm);
  // Q: two buffers of q_rows rows by item (kQT = 1), or two tiles of 128
  const int q_tile = KB * q_rows * 128;
  unsigned char* sQ = base;
  unsigned char* sK = sQ + 2 * q_tile;
  unsigned char* sV = sK + kRing;
  unsigned char* sOut = sV + kRing;
  Aux& aux = *reinterpret_cast<Aux*>(sOut + 8 * kStage);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = a.G;

  if (tid == 0) {
    for (int i = 0; i < C::ST; ++i) {
      tc::mbar_init(&aux.kfull[i], 1);
      tc::mbar_init(&aux.kfree[i], 1);
      tc::mbar_init(&aux.vfull[i], 1);
      tc::mbar_init(&aux.vfree[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&aux.q_full[i], 1);
      tc::mbar_init(&aux.q_free[i], 1);
      tc::mbar_init(&aux.s_full[i], 1);
      tc::mbar_init(&aux.p_full[i], 4);
      tc::mbar_init(&aux.o_full[i], 1);
      tc::mbar_init(&aux.o_empty[i], 4);
    }
    tc::mbar_init(&aux.ml_full, 4);
    for (int i = 0; i < kSched; ++i) {
      tc::mbar_init(&aux.sched_full[i], 1);
      tc::mbar_init(&aux.par_full[i], 1);
      tc::mbar_init(&aux.sched_empty[i], kReaders);
    }
    for (int i = 0; i < kBad; ++i) aux.bad[i] = 0;
    aux.abort_flag = 0;
    tc::fence_mbar_init();
    tc::tma_prefetch_desc(&tm_kp);
    tc::tma_prefetch_desc(&tm_vp);
    tc::tma_prefetch_desc(&tm_km);
    tc::tma_prefetch_desc(&tm_vm);
  }
  if (warp == 1) {
    tc::tmem_alloc(&aux.tmem_base, 512);
    tc::tmem_relinquish();
  }

  // This CTA's range: thread t sums the tiles of its run of sequences, a scan
  // over the threads places them, and the thread that holds the range's first
  // tile finds its sequence.
  auto units_of = [&](const TreeSeq& s) -> int64_t {
    const int nt = seq_tiles(s);
    if (nt == 0) return 0;
    return (int64_t)(nt + kItemCost) * ((s.n * G + blk_rows - 1) / blk_rows) * a.H;
  };
  int64_t* wsum = reinterpret_cast<int64_t*>(sK);  // [12], before any tile lands there
  const int per = (a.B + kTcThreads - 1) / kTcThreads;
  const int b_lo = min(a.B, tid * per), b_hi = min(a.B, b_lo + per);
  int64_t mine = 0;
  for (int b = b_lo; b < b_hi; ++b) {
    const TreeSeq s = tree_seq(a, b);
    if (s.error && blockIdx.x == 0) record_error(a.status, s.error);
    mine += units_of(s);
  }
  int64_t incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) wsum[warp] = incl;
  __syncthreads();
  int64_t before = 0, total = 0;
#pragma unroll
  for (int i = 0; i < kTcThreads / 32; ++i) {
    if (i < warp) before += wsum[i];
    total += wsum[i];
  }
  const int64_t ge = min((int64_t)gridDim.x, total);  // ranges that hold tiles
  auto range_lo = [&](int64_t c) { return c * total / ge; };
  const int64_t lo = blockIdx.x < ge ? range_lo(blockIdx.x) : 0;
  const int64_t hi = blockIdx.x < ge ? range_lo(blockIdx.x + 1) : 0;
  int64_t at = before + incl - mine;
  if (lo < hi && lo >= at && lo < at + mine) {
    for (int b = b_lo; b < b_hi; ++b) {
      const TreeSeq s = tree_seq(a, b);
      const int64_t t = units_of(s);
      if (lo < at + t) {
        aux.start_b = b;
        aux.start_seq = s;
        aux.start = lo - at;
        break;
      }
      at += t;
    }
  }
  tc::fence_proxy_async_smem();  // wsum's reads and writes before the tile loads
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = aux.tmem_base;
  // TMEM columns: S of stream s at 128 s, O at 256 + D s
  volatile int* abort_flag = &aux.abort_flag;
  auto fail = [&]() {
    record_error(a.status, MSA_ERR_TIMEOUT);
    *abort_flag = 1;
  };
  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    if (*abort_flag) return false;
    if (tc::mbar_wait(bar, parity)) return true;
    fail();
    return false;
  };

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(C::REG_LOW));
    if (warp == 2) {
      // --------------------------------------------- the range and the queries
      int64_t left = hi - lo;
      int b = 0, item = 0;
      TreeSeq s{};
      int nt = 0, nblk = 0;
      auto size_seq = [&]() {
        nt = seq_tiles(s);
        nblk = (s.n * G + blk_rows - 1) / blk_rows;
      };
      TreeCut cut{0, 0, 0, 0, -1};
      int pos = 0;  // units of the item at hand that lie before the range
      if (left > 0) {
        b = aux.start_b;
        s = aux.start_seq;
        size_seq();
        item = (int)(aux.start / (nt + kItemCost));
        pos = (int)(aux.start % (nt + kItemCost));
        if (pos > kItemCost && range_lo(blockIdx.x - 1) <= lo - pos + kItemCost) {
          // the first border inside this item's tiles: its last part holds the
          // item's last unit, `end`
          const int64_t end = lo - pos + kItemCost + nt - 1;
          int64_t c = min(ge - 1, end * ge / total);
          while (c + 1 < ge && range_lo(c + 1) <= end) ++c;
          while (range_lo(c) > end) --c;
          cut.last = (int)c;
          cut.t0 = s.t0;
          cut.g = item / nblk;
          cut.row0 = item % nblk * blk_rows;
          cut.rows = min(blk_rows, s.n * G - cut.row0);
        }
      }
      if (lane == 0) cuts[blockIdx.x] = cut;
      uint32_t q_loads = 0;
      for (uint32_t k = 0;; ++k) {
        const int slot = k % kSched;
        if (!wait(&aux.sched_empty[slot], ((k / kSched) & 1) ^ 1)) break;
        ItemE e{};
        e.cnt = -1;
        while (left > 0) {
          while (item == a.H * nblk || nt == 0) {  // the next sequence with tiles
            s = tree_seq(a, ++b);
            size_seq();
            item = 0;
          }
          const int take = (int)min((int64_t)(nt + kItemCost - pos), left);
          const int j_lo = max(pos - kItemCost, 0), j_hi = max(pos + take - kItemCost, 0);
          const int at = item++;
          left -= take;
          pos = 0;
          if (j_lo == j_hi) continue;  // the border lies before its first tile
          e.t0 = s.t0;
          e.n = s.n;
          e.M = s.M;
          e.L = s.L;
          e.cache = s.cache;
          e.b = b;
          e.g = at / nblk;
          e.row0 = at % nblk * blk_rows;
          e.rows = min(blk_rows, s.n * G - e.row0);
          e.j_lo = j_lo;
          e.cnt = j_hi - j_lo;
          e.part = j_lo > 0 ? 0 : j_hi < nt ? 1 : -1;
          break;
        }
        if (lane == 0) {
          aux.item[slot] = e;
          tc::mbar_arrive(&aux.sched_full[slot]);
        }
        if (e.cnt < 0) break;
        if (a.parents) {
          for (int i = lane; i < e.n; i += 32) {
            int p = a.parents[e.t0 + i];
            if (p >= i) {  // a parent comes before its child
              record_error(a.status, MSA_ERR_INVALID_ARG);
              p = -2;
            }
            aux.par[slot][i] = (signed char)max(p, -2);
          }
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&aux.par_full[slot]);
        }
        // its query rows, into buffer k & 1 (kQT = 1) or the two tiles (rows of
        // tokens behind the sequence's come along: nobody reads their S)
        const int qb = kQT == 1 ? k & 1 : 0;
        const uint32_t use = kQT == 1 ? k >> 1 : k;
        if (use > 0 && !wait(&aux.q_free[qb], (use - 1) & 1)) break;
        if (lane == 0) {
          const int tiles = kQT == 1 ? 1 : 2;
          tc::mbar_arrive_expect_tx(&aux.q_full[qb], (uint32_t)(tiles * KB * tile_rows * 128));
          for (int t = 0; t < tiles; ++t)
#pragma unroll
            for (int kb = 0; kb < KB; ++kb)
              tc::tma_load_3d(sQ + (kQT == 1 ? qb : t) * q_tile + kb * (q_rows * 128), &tm_q,
                              &aux.q_full[qb], kb * 64, e.g * G,
                              (int)(e.t0 + (e.row0 + t * tile_rows) / G));
        }
        ++q_loads;
        __syncwarp();
      }
      // the last loads of both buffers land before the CTA exits
      constexpr uint32_t kBufs = kQT == 1 ? 2 : 1;
      for (uint32_t v = q_loads > kBufs ? q_loads - kBufs : 0; v < q_loads; ++v)
        tc::mbar_wait(&aux.q_full[v % kBufs], (v / kBufs) & 1);
    } else if (warp == 0 || warp == 3) {
      // ----------------------------------------------------------- K, V loads
      const bool isv = warp == 3;
      unsigned char* ring = isv ? sV : sK;
      uint64_t* full = isv ? aux.vfull : aux.kfull;
      uint64_t* fre = isv ? aux.vfree : aux.kfree;
      const int n_st = C::ST;
      const CUtensorMap* mm = isv ? &tm_vm : &tm_km;
      const CUtensorMap* mp = isv ? &tm_vp : &tm_kp;
      const int page = a.page_size;
      int st = 0;
      uint32_t ph = 0, loads = 0;
      bool ok = true;
      for (uint32_t k = 0; ok; ++k) {
        const int slot = k % kSched;
        if (!wait(&aux.sched_full[slot], (k / kSched) & 1)) break;
        const ItemE e = aux.item[slot];
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&aux.sched_empty[slot]);
        if (e.cnt < 0) break;
        const int n_mt = (e.M + kKeys - 1) / kKeys;
        const int32_t* table = a.block_table + (int64_t)e.b * a.max_pages;
        // the first tensor-map row of this lane's piece of tile j, -1: none
        auto piece = [&](int j) -> int {
          if (j < n_mt) {
            const int r0 = j * kKeys + lane * kMemRows;
            return lane < kKeys / kMemRows && r0 < e.M ? e.b * a.m_cap + r0 : -1;
          }
          const int r0 = (j - n_mt) * kKeys + lane * page;
          if (lane * page >= kKeys || r0 >= e.cache) return -1;
          const int pg = table[r0 / page];
          if (pg < 0 || pg >= a.n_pages) {
            record_error(a.status, MSA_ERR_INVALID_ARG);
            return -1;
          }
          return (pg * a.H + e.g) * page;
        };
        int next = piece(e.j_lo);
        for (int i = 0; i < e.cnt; ++i) {
          const int j = e.j_lo + i, row = next;
          if (i + 1 < e.cnt) next = piece(j + 1);  // in flight while the slot drains
          const bool mem = j < n_mt;
          const int rows = mem ? kMemRows : page;
          ok = wait(&fre[st], ph ^ 1);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          const uint32_t live = __ballot_sync(0xffffffffu, row >= 0);
          if (lane == 0)
            tc::mbar_arrive_expect_tx(&full[st], (uint32_t)__popc(live) * rows * 128 * KB);
          __syncwarp();
          if (row >= 0) {
            unsigned char* d = ring + st * C::TILE + lane * rows * 128;
#pragma unroll
            for (int kb = 0; kb < KB; ++kb)
              tc::tma_load_3d(d + kb * kKeys * 128, mem ? mm : mp, &full[st], kb * 64,
                              mem ? e.g : 0, row);
          }
          ++loads;
          if (++st == n_st) {
            st = 0;
            ph ^= 1;
          }
        }
      }
      // every load issued lands before the CTA exits
      for (uint32_t v = loads > (uint32_t)n_st ? loads - n_st : 0; v < loads; ++v)
        tc::mbar_wait(&full[v % n_st], (v / n_st) & 1);
    } else if (lane == 0) {
      // ----------------------------------------------------------------- MMA
      // Virtual tile v belongs to stream v & 1: key tile v (kQT = 1) or
      // v >> 1 (kQT = 2) of the range.  S(v) may follow once P V(v - 2),
      // which reads the same TMEM columns, has been issued (one thread's
      // MMAs run in issue order), so S(v)'s commit also says that P V(v - 2)
      // is done.
      auto issue_s = [&](int s, int q_at, int st) {
        tc::tc_fence_after();
        const uint64_t qd = tc::sdesc_kmajor_sw128(tc::smem_u32(sQ + q_at * q_tile));
        const uint64_t kd = tc::sdesc_kmajor_sw128(tc::smem_u32(sK + st * C::TILE));
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          tc::mma_bf16_ss(tmem + s * 128,
                          tc::desc_add(qd, (kk >> 2) * (q_rows * 128) + (kk & 3) * 32),
                          tc::desc_add(kd, (kk >> 2) * (kKeys * 128) + (kk & 3) * 32),
                          C::IDESC_S, kk > 0 ? 1u : 0u);
        tc::mma_commit(&aux.s_full[s]);
      };
      auto issue_pv = [&](int s, int st, uint32_t acc) {
        tc::tc_fence_after();
        const uint64_t vd = tc::sdesc_mnmajor_sw128(tc::smem_u32(sV + st * C::TILE), kKeys * 128);
#pragma unroll
        for (int kk = 0; kk < kKeys / 16; ++kk)
          tc::mma_bf16_ts(tmem + 256 + s * D, tmem + s * 128 + kk * 8,
                          tc::desc_add(vd, kk * 16 * 128), C::IDESC_O, kk > 0 ? 1u : acc);
      };
     if constexpr (kQT == 2) {
      // Both streams on every tile, in a fixed order: P V_0 S_0 P V_1 S_1 of
      // consecutive tiles (what this thread does between two MMAs is time that
      // the tensor pipe idles: as one loop that polls for whichever is ready a
      // tile took 4,000 cycles, so 3,650); at an item's end both P V
      // first, since the next item's queries are still on their way.
      uint32_t tiles = 0;         // key tiles whose P V are issued
      int kst = 0, vst = 0;
      uint32_t kph = 0, vph = 0;
      auto next_k = [&]() {
        tc::mma_commit(&aux.kfree[kst]);
        if (++kst == C::ST) {
          kst = 0;
          kph ^= 1;
        }
      };
      for (uint32_t k = 0;; ++k) {
        const int slot = k % kSched;
        if (!wait(&aux.sched_full[slot], (k / kSched) & 1)) break;
        const int cnt = aux.item[slot].cnt;
        tc::mbar_arrive(&aux.sched_empty[slot]);
        if (cnt < 0) break;
        if (!wait(&aux.q_full[0], k & 1) || !wait(&aux.kfull[kst], kph)) break;
        issue_s(0, 0, kst);
        issue_s(1, 1, kst);
        next_k();
        if (cnt == 1) tc::mma_commit(&aux.q_free[0]);
        bool ok = true;
        for (int j = 0; ok && j < cnt; ++j, ++tiles) {
          const bool more = j + 1 < cnt;
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            if (s == 0) ok = ok && wait(&aux.vfull[vst], vph);
            if (j == 0 && k > 0) ok = ok && wait(&aux.o_empty[s], (k - 1) & 1);
            ok = ok && wait(&aux.p_full[s], tiles & 1);
            if (!ok) break;
            issue_pv(s, vst, j > 0 ? 1u : 0u);
            if (!more) {
              tc::mma_commit(&aux.o_full[s]);
            } else {
              if (s == 0 && !(ok = wait(&aux.kfull[kst], kph))) break;
              issue_s(s, s, kst);
            }
          }
          if (!ok) break;
          if (more) {
            next_k();
            if (j + 2 == cnt) tc::mma_commit(&aux.q_free[0]);
          }
          tc::mma_commit(&aux.vfree[vst]);
          if (++vst == C::ST) {
            vst = 0;
            vph ^= 1;
          }
        }
        if (!ok) break;
      }
     } else {
      // One key tile a stream in turn; P V and S are issued as they become
      // ready (the loads set the pace, and neither waits for the other's).
      uint32_t ks = 0, kp = 0;   // items taken by S, by P V
      int i_s = 0, n_s = 0;      // key tile within the item's share, tiles of it
      int i_p = 0, n_p = 0;
      uint32_t vs = 0, vp = 0;   // S and P V issued
      uint32_t ne[2] = {0, 0};   // items whose O a stream has begun
      int kst = 0, vst = 0;      // ring slots of the next S and P V
      uint32_t kph = 0, vph = 0;
      bool done = false, q_seen = false;
      uint64_t t_last = 0;
      uint32_t polls = 0;
      while (!(done && vp == vs)) {
        bool moved = false;
        if (vp < vs && tc::mbar_test(&aux.p_full[vp & 1], (vp >> 1) & 1)) {
          const int s = vp & 1;
          if (i_p == n_p) {  // published: S has read it
            const int slot = kp % kSched;
            n_p = aux.item[slot].cnt;
            i_p = 0;
            ++kp;
            tc::mbar_arrive(&aux.sched_empty[slot]);
          }
          const bool first = i_p < 2;
          if ((!first || ne[s] == 0 || tc::mbar_test(&aux.o_empty[s], (ne[s] - 1) & 1)) &&
              tc::mbar_test(&aux.vfull[vst], vph)) {
            if (first) ++ne[s];
            issue_pv(s, vst, first ? 0u : 1u);
            if (i_p + 2 >= n_p) tc::mma_commit(&aux.o_full[s]);
            tc::mma_commit(&aux.vfree[vst]);
            if (++vst == C::ST) {
              vst = 0;
              vph ^= 1;
            }
            ++i_p;
            ++vp;
            moved = true;
          }
        }
        if (vs < vp + 2 && !done) {
          if (i_s == n_s && tc::mbar_test(&aux.sched_full[ks % kSched], (ks / kSched) & 1)) {
            n_s = aux.item[ks % kSched].cnt;
            i_s = 0;
            done = n_s < 0;
            if (done) n_s = 0;
            ++ks;
            q_seen = false;
          }
          if (i_s < n_s) {
            const int s = vs & 1;
            const int qb = (ks - 1) & 1;
            if (!q_seen) q_seen = tc::mbar_test(&aux.q_full[qb], ((ks - 1) >> 1) & 1);
            if (q_seen && tc::mbar_test(&aux.kfull[kst], kph)) {
              issue_s(s, qb, kst);
              tc::mma_commit(&aux.kfree[kst]);
              if (++kst == C::ST) {
                kst = 0;
                kph ^= 1;
              }
              if (++i_s == n_s) tc::mma_commit(&aux.q_free[qb]);
              ++vs;
              moved = true;
            }
          }
        }
        if (moved) {
          polls = 0;
        } else {
          if (polls == 0) t_last = tc::globaltimer_ns();
          if ((++polls & 255u) == 0) {
            if (*abort_flag) break;
            if (tc::globaltimer_ns() - t_last > 2000000000ull) {
              fail();
              break;
            }
          }
        }
      }
     }
    }
  } else {
    // --------------------------------------------------------------- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(C::REG_HIGH));
    const int grp = (warp - 4) >> 2;   // stream
    const int quad = warp & 3;         // TMEM lane quarter
    const int r = quad * 32 + lane;    // row of the stream's tile; V row to clean
    const uint32_t lane_addr = (uint32_t)(quad * 32) << 16;
    const uint32_t tSP = tmem + grp * 128 + lane_addr;
    const float qscale = a.qscale;
    uint32_t w = 0;           // tiles of this stream so far
    uint32_t u = 0;           // key tiles of the CTA so far
    uint32_t ne[2] = {0, 0};  // items whose O a stream has held
    uint32_t n_pub = 0;
    for (uint32_t k = 0;; ++k) {
      const int slot = k % kSched;
      if (!wait(&aux.sched_full[slot], (k / kSched) & 1)) break;
      const ItemE e = aux.item[slot];
      if (e.cnt < 0) break;
      const int i0 = kQT == 1 ? (u ^ grp) & 1 : 0;
      const int step = kQT == 1 ? 2 : 1;
      const bool both = kQT == 1 && e.cnt >= 2;     // both streams hold a part of O
      const int owner = kQT == 1 ? (u + e.cnt - 1) & 1 : grp;
      const int rb = (kQT == 2 ? grp * tile_rows : 0) + r;  // row within the block
      const bool row_ok = r < tile_rows && rb < e.rows;
      const bool warp_on = (kQT == 2 ? grp * tile_rows : 0) + quad * 32 < e.rows;
      const int row = e.row0 + rb;
      const int tok = row / G;
      u128 anc = 0;
      if (i0 < e.cnt) {
        // what the row's token sees of its tree
        if (!a.parents) {
          anc = low_bits(tok + 1);
        } else {
          if (!wait(&aux.par_full[slot], (k / kSched) & 1)) break;
          if (row_ok) {
            const signed char* par = aux.par[slot];
            int x = tok;
            do {
              anc |= (u128)1 << x;
              x = par[x];
            } while (x >= 0);
            if (x != -1) anc = 0;  // pruned: sees nothing
          }
        }
      }
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&aux.sched_empty[slot]);
      if (i0 < e.cnt) {
        const bool dead = anc == 0;
        const int n_mt = (e.M + kKeys - 1) / kKeys;
        float m_run = -INFINITY, l_run = 0.f;
        for (int i = i0, t = 0; i < e.cnt; i += step, ++t, ++w) {
          const int j = e.j_lo + i;
          const bool mem = j < n_mt;
          const int key0 = (mem ? j : j - n_mt) * kKeys;
          const int n_rows = mem ? e.M - key0 : e.cache - key0;  // rows of the tile that exist
          const bool full = key0 + kKeys <= (mem ? e.M : e.L);   // every row sees every key
          if (!wait(&aux.s_full[grp], w & 1)) break;
          tc::tc_fence_after();
          if (!full && (kQT == 1 || grp == 0) && (n_rows < kKeys || e.n > 1)) {
            // V(u + i) has landed at most once since P V of the slot's last
            // tile, so the parity names this tile; P V waits for this
            // group's p_full below
            const uint32_t vi = u + i;
            if (!wait(&aux.vfull[vi % C::ST], (vi / C::ST) & 1)) break;
            // rows to look at: past the end, and drafted ones another row may
            // not see; 16-byte pieces, consecutive ones by consecutive threads
            unsigned char* vt = sV + (vi % C::ST) * C::TILE;
            const int first = mem || e.n == 1 ? n_rows : max(min(n_rows, e.L - key0), 0);
            bool bad = false;
#pragma unroll 4
            for (int p = first * (D / 8) + r; p < kKeys * (D / 8); p += 128) {
              const int vrow = p / (D / 8), c = p % (D / 8);
              uint4* v = reinterpret_cast<uint4*>(vt + (c >> 3) * (kKeys * 128) + vrow * 128 +
                                                  (c & 7) * 16);
              uint4 x = make_uint4(0, 0, 0, 0);
              if (vrow < n_rows) {
                const uint4 y = *v;
                x = make_uint4(finite_bf16x2(y.x), finite_bf16x2(y.y), finite_bf16x2(y.z),
                               finite_bf16x2(y.w));
                if (x.x == y.x && x.y == y.y && x.z == y.z && x.w == y.w) continue;
                bad = true;
              }
              *v = x;
            }
            if (bad) *(volatile int*)&aux.bad[k % kBad] = (int)k + 1;
            tc::fence_proxy_async_smem();
          }
          if (warp_on) {
            uint32_t sv[kKeys];
#pragma unroll
            for (int c = 0; c < kKeys / 32; ++c)
              tc::tmem_ld32(tSP + c * 32, *reinterpret_cast<uint32_t(*)[32]>(sv + c * 32));
            tc::tmem_ld_wait();
            if (!full) {
              u128 vis;
              if (mem) {
                vis = low_bits(n_rows);
              } else {
                const int off = e.L - key0;  // column of the first drafted key
                vis = low_bits(off) | (off >= 0 ? (off < 128 ? anc << off : (u128)0)
                                                : (off > -128 ? anc >> -off : (u128)0));
                vis &= low_bits(n_rows);
              }
#pragma unroll
              for (int q4 = 0; q4 < 4; ++q4) {
                const uint32_t bits = (uint32_t)(vis >> (32 * q4));
#pragma unroll
                for (int c = 0; c < 32; ++c)
                  if (!((bits >> c) & 1)) sv[32 * q4 + c] = 0xff800000u;
              }
            }
            // row maximum: 8 chains of 3-input max
            float mx[8];
#pragma unroll
            for (int c = 0; c < 8; ++c) mx[c] = __uint_as_float(sv[c]);
#pragma unroll
            for (int c = 8; c + 16 <= kKeys; c += 16)
#pragma unroll
              for (int x = 0; x < 8; ++x)
                mx[x] = fmax3(mx[x], __uint_as_float(sv[c + x]), __uint_as_float(sv[c + 8 + x]));
#pragma unroll
            for (int x = 0; x < 8; ++x) mx[x] = fmaxf(mx[x], __uint_as_float(sv[kKeys - 8 + x]));
            const float mt = qscale * fmax3(fmax3(mx[0], mx[1], mx[2]),
                                            fmax3(mx[3], mx[4], mx[5]), fmaxf(mx[6], mx[7]));
            // the reference maximum moves only when a tile exceeds it by 2^8
            const bool grow = row_ok && mt > m_run + kRescaleLog2;
            const bool held = m_run != -INFINITY;  // O holds weights, to be scaled
            float alpha = 1.f;                     // even where alpha underflows to 0
            if (grow) {
              alpha = m_run == -INFINITY ? 0.f : ex2a(m_run - mt);
              m_run = mt;
            }
            if (t > 0 && __any_sync(0xffffffffu, grow && held)) {
              const uint32_t tO = tmem + 256 + grp * D + lane_addr;
#pragma unroll 1
              for (int c = 0; c < D / 32; ++c) {
                uint32_t o[32];
                tc::tmem_ld32(tO + c * 32, o);
                tc::tmem_ld_wait();
#pragma unroll
                for (int x = 0; x < 32; ++x)
                  o[x] = __float_as_uint(__uint_as_float(o[x]) * alpha);
                tmem_st32(tO + c * 32, o);
              }
            }
            l_run *= alpha;
            const float neg_m = m_run == -INFINITY ? 0.f : -m_run;
            const unsigned long long sc2 = f2(qscale, qscale), nm2 = f2(neg_m, neg_m);
            unsigned long long ls2[2] = {0ull, 0ull};
#pragma unroll
            for (int c = 0; c < kKeys / 64; ++c) {
              uint32_t pw[32];
#pragma unroll
              for (int x = 0; x < 32; ++x) {
                const int k0 = c * 64 + 2 * x;
                unsigned long long x2 =
                    (unsigned long long)sv[k0] | ((unsigned long long)sv[k0 + 1] << 32);
                asm("fma.rn.f32x2 %0, %0, %1, %2;" : "+l"(x2) : "l"(sc2), "l"(nm2));
                const float p0 = ex2a(__uint_as_float((uint32_t)x2));
                const float p1 = ex2a(__uint_as_float((uint32_t)(x2 >> 32)));
                const unsigned long long p2 = f2(p0, p1);
                asm("add.rn.f32x2 %0, %0, %1;" : "+l"(ls2[x & 1]) : "l"(p2));
                pw[x] = pack2(p0, p1);
              }
              tmem_st32(tSP + c * 32, pw);
            }
            asm("add.rn.f32x2 %0, %0, %1;" : "+l"(ls2[0]) : "l"(ls2[1]));
            l_run += __uint_as_float((uint32_t)ls2[0]) + __uint_as_float((uint32_t)(ls2[0] >> 32));
            tmem_st_wait();
          }
          tc::tc_fence_before();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&aux.p_full[grp]);
        }
        if (dead) {
          m_run = -INFINITY;
          l_run = 0.f;
        }
        if (owner != grp) {
          // hand (m, l) to the other group, which reads this stream's O too
          if (ne[grp] > 0 && !wait(&aux.o_empty[grp], (ne[grp] - 1) & 1)) break;
          aux.ml[r] = make_float2(m_run, l_run);
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&aux.ml_full);
        } else {
          if (!wait(&aux.o_full[grp], ne[grp] & 1)) break;
          // O = c0 O_grp + c1 O_other; a part without weight is left out (its O
          // may hold 0 times NaN): c = 0
          float c0 = l_run == 0.f ? 0.f : 1.f, c1 = 0.f;
          if (both) {
            if (!wait(&aux.o_full[grp ^ 1], ne[grp ^ 1] & 1)) break;
            if (!wait(&aux.ml_full, n_pub & 1)) break;
            const float2 x = aux.ml[r];
            const float m = fmaxf(m_run, x.x);
            c0 = l_run == 0.f ? 0.f : m == -INFINITY ? 1.f : ex2a(m_run - m);
            c1 = x.y == 0.f ? 0.f : m == -INFINITY ? 1.f : ex2a(x.x - m);
            l_run = (l_run == 0.f ? 0.f : c0 * l_run) + (x.y == 0.f ? 0.f : c1 * x.y);
            m_run = m;
          }
          tc::tc_fence_after();
          const bool bad = *(volatile int*)&aux.bad[k % kBad] == (int)k + 1;
          if (e.part < 0) {
            const float inv = l_run == 0.f ? 0.f : 1.f / l_run;
            c0 *= inv;
            c1 *= inv;
          }
          // (a small loop: this code runs once an item, and what it costs first
          // is its way into the instruction cache; and by way of shared memory:
          // a thread holds a row, and a warp's stores of 16 bytes of each of 32
          // rows took an item of 256 rows 13,000 cycles)
          const int64_t prow = ((int64_t)blockIdx.x * 2 + e.part) * part_rows + rb;
          if (warp_on) {
            const uint32_t tO = tmem + 256 + grp * D + lane_addr;
            const uint32_t tO2 = tmem + 256 + (both ? grp ^ 1 : grp) * D + lane_addr;
            __nv_bfloat16* op = static_cast<__nv_bfloat16*>(a.out) +
                                ((e.t0 + tok) * a.Hq + e.g * G + row % G) * D;
            float* po = part_o + prow * D;
            const uint64_t mine = e.part < 0 ? reinterpret_cast<uint64_t>(op)
                                             : reinterpret_cast<uint64_t>(po);
            const uint32_t live = __ballot_sync(0xffffffffu, row_ok);
            unsigned char* stg = sOut + (warp - 4) * kStage;  // 32 rows of 128 bytes
#pragma unroll 1
            for (int c = 0; c < D; c += 16) {
              uint32_t x0[16], x1[16];
              float o[16];
              tc::tmem_ld16(tO + c, x0);
              if (kQT == 1) tc::tmem_ld16(tO2 + c, x1);
              tc::tmem_ld_wait();
#pragma unroll
              for (int x = 0; x < 16; ++x) {
                o[x] = c0 == 0.f ? 0.f : c0 * __uint_as_float(x0[x]);
                if (kQT == 1) o[x] += c1 == 0.f ? 0.f : c1 * __uint_as_float(x1[x]);
              }
              // 16-byte pieces of a row: columns c .. of 64 bf16, or of 32 fp32
              int p0;
              auto put = [&](int p, const uint4& v) {
                *reinterpret_cast<uint4*>(stg + lane * 128 + ((p ^ (lane & 7)) << 4)) = v;
              };
              if (e.part < 0) {
                p0 = (c & 63) >> 3;
#pragma unroll
                for (int x = 0; x < 16; x += 8)
                  put(p0 + (x >> 3),
                      make_uint4(pack2(o[x], o[x + 1]), pack2(o[x + 2], o[x + 3]),
                                 pack2(o[x + 4], o[x + 5]), pack2(o[x + 6], o[x + 7])));
                p0 += 2;
              } else {
                p0 = (c & 31) >> 2;
#pragma unroll
                for (int x = 0; x < 16; x += 4)
                  put(p0 + (x >> 2),
                      make_uint4(__float_as_uint(o[x]), __float_as_uint(o[x + 1]),
                                 __float_as_uint(o[x + 2]), __float_as_uint(o[x + 3])));
                p0 += 4;
              }
              __syncwarp();
              if (p0 == 8) {  // eight lanes a row, four rows a store
                const uint64_t at =
                    (uint64_t)(e.part < 0 ? (c & ~63) * 2 : (c & ~31) * 4) + (lane & 7) * 16;
#pragma unroll
                for (int x = 0; x < 8; ++x) {
                  const int rw = x * 4 + (lane >> 3);
                  const uint64_t dst = __shfl_sync(0xffffffffu, mine, rw) + at;
                  if ((live >> rw) & 1)
                    st16(reinterpret_cast<void*>(dst),
                         *reinterpret_cast<const uint4*>(stg + rw * 128 +
                                                         (((lane & 7) ^ (rw & 7)) << 4)));
                }
                __syncwarp();
              }
            }
            if (row_ok && e.part >= 0) part_ml[prow] = make_float2(m_run, l_run);
            if (row_ok && bad) {
              // drafted values taken out of V, added for the rows that see them
#pragma unroll 1
              for (int d = 0; d < e.n; ++d) {
                const int kr = e.L + d, j = n_mt + kr / kKeys;
                if (!((anc >> d) & 1) || j < e.j_lo || j >= e.j_lo + e.cnt || kr >= e.cache)
                  continue;
                const int pg = a.block_table[(int64_t)e.b * a.max_pages + kr / a.page_size];
                if (pg < 0 || pg >= a.n_pages) continue;
                const __nv_bfloat16* v =
                    static_cast<const __nv_bfloat16*>(a.v_pages) +
                    (((int64_t)pg * a.H + e.g) * a.page_size + kr % a.page_size) * D;
#pragma unroll 1
                for (int x = 0; x < D; ++x) {
                  const float f = __bfloat162float(v[x]);
                  if (isfinite(f)) continue;
                  if (e.part < 0) op[x] = __float2bfloat16(__bfloat162float(op[x]) + f);
                  else po[x] += f;
                }
              }
            }
          }
          tc::tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            tc::mbar_arrive(&aux.o_empty[grp]);
            if (both) tc::mbar_arrive(&aux.o_empty[grp ^ 1]);
          }
        }
      }
      if (kQT == 1) {
        ++ne[u & 1];
        if (both) {
          ++ne[(u & 1) ^ 1];
          ++n_pub;
        }
      } else {
        ++ne[grp];
      }
      u += e.cnt;
    }
  }

  tc::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, 512);
  }
}

struct TcPlan {
  int qt;          // Q tiles of an item
  int part_rows;   // rows of a partial
  int tile_tok;    // tokens of a tile: whole tokens, at most 128 rows
  int q_rows;
  size_t smem, po_bytes, ml_bytes, cut_bytes, total;
};

// kQT = 2 where two tiles have to share one pass over K and V: more than 192
// rows (fewer leave much of the second tile empty, and its time is spent all
// the same) of 128 dims (at 64 the chain of a tile, not HBM, is the bound), and
// more keys and values in the lengths that the buffers allow than the L2 keeps:
// 64 tokens, 2 sequences x 20,064 keys (164 MB) 61 us against 72 with kQT = 1,
// x 150,065 311 against 383; 4 x 564 (9 MB) 26.7 against 24.3.  In between the two
// are even (16 x 1,064 and 16 x 2,064, 70 and 135 MB: 60 to 66 and 76 to 88 us
// either way, as the GPU goes).  The lengths themselves are on the device: with a
// block table 16 times as wide as its sequences need, 4 x 564 keys take 26.5 us.
// The Q buffers hold no more rows than a tile can have (the MMA reads on into
// the ring: rows of S that nobody reads).
TcPlan tc_plan(int B, int n_max, int G, int H, int D, int64_t keys) {
  TcPlan p{};
  const int rows = n_max * G;
  p.qt = rows > 192 && D == 128 && (double)B * H * keys * D * 4 > 150e6 ? 2 : 1;
  p.tile_tok = std::min(n_max, 128 / G);
  p.part_rows = std::min(rows, p.tile_tok * G * p.qt);
  p.q_rows = (p.tile_tok * G + 7) / 8 * 8;
  p.smem = 1024 + 2 * (size_t)(D / 64) * p.q_rows * 128 + 2 * kRing + 8 * kStage + sizeof(Aux);
  const size_t parts = 2 * (size_t)num_sms() * p.part_rows;
  p.po_bytes = round_up(parts * D * sizeof(float), 256);
  p.ml_bytes = round_up(parts * sizeof(float2), 256);
  p.cut_bytes = round_up((size_t)num_sms() * sizeof(TreeCut), 256);
  p.total = p.po_bytes + p.ml_bytes + p.cut_bytes;
  return p;
}

template <int D, int kQT>
int launch_tc(const TreeArgs& a, const TcPlan& p, void* ws, cudaStream_t s) {
  unsigned char* w = static_cast<unsigned char*>(ws);
  float* part_o = reinterpret_cast<float*>(w);
  float2* part_ml = reinterpret_cast<float2*>(w + p.po_bytes);
  TreeCut* cuts = reinterpret_cast<TreeCut*>(w + p.po_bytes + p.ml_bytes);
  CUtensorMap qm, km, vm, kp, vp;
  const int64_t page_rows = (int64_t)a.n_pages * a.H * a.page_size;
  bool ok = tma_map_sw128_bf16(&qm, a.q, D, a.Hq, a.n_tok, a.G, p.tile_tok) &&
            tma_map_sw128_bf16(&kp, a.k_pages, D, 1, page_rows, 1, a.page_size) &&
            tma_map_sw128_bf16(&vp, a.v_pages, D, 1, page_rows, 1, a.page_size);
  if (a.m_cap > 0)
    ok = ok && tma_map_sw128_bf16(&km, a.k_mem, D, a.H, (int64_t)a.B * a.m_cap, 1, kMemRows) &&
         tma_map_sw128_bf16(&vm, a.v_mem, D, a.H, (int64_t)a.B * a.m_cap, 1, kMemRows);
  else
    km = kp, vm = vp;  // never loaded from
  if (!ok) return note_cuda(cudaErrorInvalidValue);
  auto kern = tree_tc_kernel<D, kQT>;
  if (int rc = ensure_smem_attr(reinterpret_cast<const void*>(kern), (int)p.smem)) return rc;
  const unsigned grid = (unsigned)num_sms();
  if (int rc = launch_pdl(kern, dim3(grid), dim3(kTcThreads), p.smem, s, qm, km, vm, kp, vp, a,
                          p.part_rows, p.tile_tok * a.G, p.q_rows, part_o, part_ml, cuts))
    return rc;
  return tree_merge_launch(a, false, D, (int)grid, 1, p.part_rows, part_o, part_ml, cuts, s);
}

}  // namespace

size_t tree_tc_workspace_size(int B, int n_max, int G, int H, int D, int64_t keys) {
  return tc_plan(B, n_max, G, H, D, keys).total;
}

int tree_tc_launch(const TreeArgs& a, int D, void* ws, cudaStream_t s) {
  const TcPlan p = tc_plan(a.B, a.n_max, a.G, a.H, D,
                           (int64_t)a.m_cap + (int64_t)a.max_pages * a.page_size);
  if (D == 64) return launch_tc<64, 1>(a, p, ws, s);
  return p.qt == 1 ? launch_tc<128, 1>(a, p, ws, s) : launch_tc<128, 2>(a, p, ws, s);
}

}  // namespace msa
