// Attention for drafted token trees over [memory ; paged cache ; drafted
// tokens] when a KV head has few query rows (method and semantics:
// tree_attn.cu): plain decode and small trees, R = n G <= 16 rows, in bf16; in
// fp32 any number, 16 an item.
//
// Mathematics.  As tree_attn_tc.cu: S = Q K^T, p = 2^(scale log2(e) s - m),
// O += p V, l += p, one pass over the keys.  With bf16 values p is two bf16
// terms, p = hi + lo to 2^-15 of it: one term alone moved an output by up to
// 2^-8 of sum p |v|, more than its own rounding (relative error over an output
// 0.0023, with two 0.0017), and the second costs 2% (64 sequences x 2,268 keys:
// 103 us with one, 105 with two).
//
// What bounds it.  4 D bytes a key and KV head against 4 R D operations: HBM,
// by far, so all that matters is bytes in flight and what happens at the ends
// of short sequences.  A 128-row tensor-core tile would spend most of its
// latency on handshakes for rows that do not exist (64 sequences x 2,268 keys,
// one token each: 114 us in tree_attn_tc.cu, 105 here with the merge, 5.7
// TB/s); here every warp is a worker of its own:
//   * The 16-key slices of all (sequence, KV head) items stand in one line,
//     cut into one contiguous range a worker (neighbours on different SMs).
//     An item inside one range is written directly, one cut by a border as
//     fp32 partials (at most two a warp) that a second launch merges in a
//     fixed order.
//   * A warp's lane 0 copies slices of K and V by TMA into the warp's own ring
//     (a slice never crosses a page: pages hold a multiple of 16 rows), waits
//     on its own barriers, and no warp waits for another.
//   * A slice is 16 x 16 of S and 16 x D of O on the warp-level
//     tensor instructions (m16n8k16): the accumulators stay in registers and
//     P's fragment is S's.  Their rate is hardly a limit: a slice's 48
//     instructions against the 8 KB that its SM receives in 350 cycles.
//   * In a slice that reaches past the sequence's rows or into its drafted
//     rows, unseen scores become -inf, V rows past the end zero, and
//     non-finite drafted values are taken out of V (0 times them would reach
//     every row) and added at the end for the rows that see them.
//   * fp32 takes slices of 8 keys on m16n8k8, operands split into two tf32
//     terms: 96 instructions a slice of 8 KB, which bound it (8 sequences x
//     32,104 keys: 147 us, 3.6 TB/s; with a third of the products 91 us, 5.8).
//     More rows are more items over the same keys, side by side and out of the
//     L2: 64 tokens, 4 sequences x 4,164 keys, 8 / 2 heads, 164 us (27 TFLOP/s;
//     fp32 register tiles of 64 x 64 one CTA a split took 169, and 2.4 times as
//     long over caches of unlike lengths up to 25,550 rows).
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "attn_tc.cuh"
#include "tc_ptx.cuh"
#include "tree_attn.cuh"

namespace msa {
namespace {

constexpr int kWarps = 8;                 // workers of a CTA, one CTA an SM
constexpr int kFewThreads = 32 * kWarps;
constexpr float kWholeItem = 8.f, kSqRange = 128.f;  // slices of an item
constexpr float kRescaleLog2 = 8.f;

template <typename T, int D> struct FC {
  static constexpr bool F32 = sizeof(T) == 4;
  static constexpr int SL = F32 ? 8 : 16;           // keys of a slice
  static constexpr int NT = SL / 8;                 // 8-key tiles of S
  static constexpr int KB = D * sizeof(T) / 128;    // 128-byte blocks of a row
  static constexpr int BLK = SL * 128;
  static constexpr int SLICE = 2 * KB * BLK;        // K and V of a slice
  static constexpr int DEPTH = 24576 / SLICE;       // slices in flight: 24 KB a warp
  static constexpr size_t SMEM = 1024 + (size_t)kWarps * DEPTH * SLICE;
};

// The drafted tokens that a row's token sees: bit t for token t, of 16 in
// bf16, 128 in fp32.
struct Seen16 {
  uint32_t m;
  __device__ __forceinline__ void clear() { m = 0; }
  __device__ __forceinline__ void set(int t) { m |= 1u << t; }
  __device__ __forceinline__ void upto(int t) { m = (2u << t) - 1; }
  __device__ __forceinline__ bool any() const { return m != 0; }
  __device__ __forceinline__ bool has(int t) const { return (m >> t) & 1; }
  // tokens t, t + 1, .. (t may be negative: those before 0 count as seen)
  __device__ __forceinline__ uint32_t from(int t) const {
    return t <= -16 ? 0xffffu : t <= 0 ? (((1u << -t) - 1) | (m << -t)) : t < 32 ? m >> t : 0u;
  }
};
struct Seen128 {
  uint4 m;
  __device__ __forceinline__ void clear() { m = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void set(int t) {
    const uint32_t bit = 1u << (t & 31);
    m.x |= t < 32 ? bit : 0;
    m.y |= (t >> 5) == 1 ? bit : 0;
    m.z |= (t >> 5) == 2 ? bit : 0;
    m.w |= (t >> 5) == 3 ? bit : 0;
  }
  __device__ __forceinline__ static uint32_t word_upto(int t) {  // t within or past a word
    return t < 0 ? 0u : t >= 31 ? 0xffffffffu : (2u << t) - 1;
  }
  __device__ __forceinline__ void upto(int t) {
    m = make_uint4(word_upto(t), word_upto(t - 32), word_upto(t - 64), word_upto(t - 96));
  }
  __device__ __forceinline__ bool any() const { return (m.x | m.y | m.z | m.w) != 0; }
  __device__ __forceinline__ bool has(int t) const { return tree_bit(m, t); }
  __device__ __forceinline__ uint32_t from(int t) const {  // 16 of them at least
    if (t <= -16) return 0xffffu;
    if (t <= 0) return ((1u << -t) - 1) | (m.x << -t);
    const int w = t >> 5;
    const uint32_t lo = w == 0 ? m.x : w == 1 ? m.y : w == 2 ? m.z : w == 3 ? m.w : 0u;
    const uint32_t hi = w == 0 ? m.y : w == 1 ? m.z : w == 2 ? m.w : 0u;
    return __funnelshift_r(lo, hi, t & 31);
  }
};

template <typename T> struct FewAux {
  using Seen = std::conditional_t<sizeof(T) == 4, Seen128, Seen16>;
  int64_t pre[kFewThreads + 1];          // slices before each thread's sequences
  TreeSeq seq[kFewThreads];              // the sequences, where a thread has one at most
  uint64_t full[kWarps][6];              // ring slots (DEPTH <= 6)
  Seen seen[kWarps][16];
  int tiles[kWarps];
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
// Two weights as bf16 terms, hi cut off and the rest rounded.  The rest gets
// 2^-20 of the weight on top, so that it is 0 only where the weight is: times an
// infinite value both terms are then that infinity.
__device__ __forceinline__ uint32_t hi2(float a, float b) {
  return __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
}
__device__ __forceinline__ float rest(float a) {
  return fmaf(a, 1.f + 0x1p-20f, -__uint_as_float(__float_as_uint(a) & 0xffff0000u));
}
__device__ __forceinline__ uint32_t rest2(float a, float b) { return pack2(rest(a), rest(b)); }
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

// The same of tf32 operands (16 x 8, 8 x 8).
__device__ __forceinline__ void mma8(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                     uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// x = hi + lo in tf32 (11 bits each): hi cut off, lo rounded, which leaves
// 2^-21 of x.  Integer instructions: the conversion's rate is a quarter of
// theirs (8 x 32,100 keys, 8 / 2 heads, a token: 167 us with it, 143).  An
// infinity becomes inf + (-0); a NaN stays one in hi, but for one whose payload
// lies in the low 13 bits, which becomes an infinity (arithmetic makes no such
// NaN, and keeping it costs 5%).
__device__ __forceinline__ uint32_t low32(float x, uint32_t hi) {
  return (__float_as_uint(x - __uint_as_float(hi)) + 0x1000u) & 0xffffe000u;
}
__device__ __forceinline__ void split32(float x, uint32_t& hi, uint32_t& lo) {
  hi = __float_as_uint(x) & 0xffffe000u;
  lo = low32(x, hi);
}
// The same of a query's element or a weight, with 2^-23 of it more in lo, about
// what the product of the rests that is left out amounts to on the average: lo is
// then 0 only where x is, and both terms times an infinity are that infinity.
__device__ __forceinline__ uint32_t low32_up(float x, uint32_t hi) {
  return (__float_as_uint(fmaf(x, 1.f + 0x1p-23f, -__uint_as_float(hi))) + 0x1000u) & 0xffffe000u;
}
__device__ __forceinline__ void split32_up(float x, uint32_t& hi, uint32_t& lo) {
  hi = __float_as_uint(x) & 0xffffe000u;
  lo = low32_up(x, hi);
}
// In its place: not taken out of the loop over slices (where 128 dims of 16
// rows would fill the registers).
__device__ __forceinline__ void split32_up_here(float x, uint32_t& hi, uint32_t& lo) {
  asm volatile("and.b32 %0, %1, 0xffffe000;" : "=r"(hi) : "r"(__float_as_uint(x)));
  lo = low32_up(x, hi);
}
__device__ __forceinline__ float4 lds128(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// The products of a slice with the 16 rows of a warp.  Lane (g, t) = (lane /
// 4, lane % 4) holds S and p of rows g and g + 8 at keys 8 n + 2 t, + 1 (the
// instruction's layout), and of O the columns col(d, x) below.
template <typename T, int D> struct Rows;

template <int D> struct Rows<__nv_bfloat16, D> {
  using C = FC<__nv_bfloat16, D>;
  uint32_t q[D / 16][4];
  __device__ __forceinline__ void load(const void* base, int64_t row, int h, bool on, int lane) {
    const __nv_bfloat16* p = static_cast<const __nv_bfloat16*>(base) + row * D + 2 * (lane & 3);
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
      q[kk][h] = on ? *reinterpret_cast<const uint32_t*>(p + kk * 16) : 0u;
      q[kk][2 + h] = on ? *reinterpret_cast<const uint32_t*>(p + kk * 16 + 8) : 0u;
    }
  }
  __device__ __forceinline__ void scores(uint32_t kb_u, int lane, float (&sc)[C::NT][4]) const {
    // ldmatrix: this lane's row and 16-byte piece of a 16 x 16 block
    const int kr = ((lane >> 4) << 3) + (lane & 7), kc = (lane >> 3) & 1;
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int x = 0; x < 4; ++x) sc[t][x] = 0.f;
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
      uint32_t b[4];
      ldsm4(kb_u + (kk >> 2) * C::BLK + kr * 128 + (((2 * (kk & 3) + kc) ^ (kr & 7)) << 4), b);
      mma16(sc[0], q[kk], b[0], b[1]);
      mma16(sc[1], q[kk], b[2], b[3]);
    }
  }
  __device__ __forceinline__ static void add(uint32_t vb_u, int lane, const float (&p)[C::NT][4],
                                             float (&o)[D / 8][4]) {
    const int vr = (((lane >> 3) & 1) << 3) + (lane & 7), vc = lane >> 4;
    const uint32_t pf[4] = {hi2(p[0][0], p[0][1]), hi2(p[0][2], p[0][3]),
                            hi2(p[1][0], p[1][1]), hi2(p[1][2], p[1][3])};
    const uint32_t pr[4] = {rest2(p[0][0], p[0][1]), rest2(p[0][2], p[0][3]),
                            rest2(p[1][0], p[1][1]), rest2(p[1][2], p[1][3])};
#pragma unroll
    for (int d = 0; d < D / 16; ++d) {
      uint32_t b[4];
      ldsm4t(vb_u + (d >> 2) * C::BLK + vr * 128 + (((2 * (d & 3) + vc) ^ (vr & 7)) << 4), b);
      mma16(o[2 * d], pf, b[0], b[1]);
      mma16(o[2 * d + 1], pf, b[2], b[3]);
      mma16(o[2 * d], pr, b[0], b[1]);
      mma16(o[2 * d + 1], pr, b[2], b[3]);
    }
  }
  __device__ __forceinline__ static int col(int d, int x, int lane) {
    return 8 * d + 2 * (lane & 3) + x;
  }
};

// fp32: every operand as two tf32 terms, three of the four products: each
// factor's rest is 2^-21 of it at most, lo lo 2^-20 of the product (a few 2^-24
// on the average), and sums are in fp32.  The instruction cuts its sum off
// instead of rounding it, so a slice's P V is summed by itself and added to O by
// an addition that rounds: O carried through the instructions lost 3e-6 of itself
// over ranges of 54 slices, more over longer ones (relative error over an output
// 3.6e-6, so 3.5e-7; 8 sequences x 32,104 keys 141 -> 147 us).  The order of dims
// and columns is free, and chosen so that a lane reads 16 bytes at a time without
// bank conflicts: its dims of a 32-dim block are 8 t .. 8 t + 7, its columns of V
// 4 g .. 4 g + 3.
template <int D> struct Rows<float, D> {
  using C = FC<float, D>;
  float4 q[D / 16][2];
  __device__ __forceinline__ void load(const void* base, int64_t row, int h, bool on, int lane) {
    const float* p = static_cast<const float*>(base) + row * D + 8 * (lane & 3);
#pragma unroll
    for (int c = 0; c < D / 16; ++c)
      q[c][h] = on ? *reinterpret_cast<const float4*>(p + 32 * (c >> 1) + 4 * (c & 1))
                   : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  __device__ __forceinline__ void scores(uint32_t kb_u, int lane, float (&sc)[C::NT][4]) const {
    const int g = lane >> 2, t = lane & 3;
    float s3[3][2][4];  // six chains of sums
#pragma unroll
    for (int i = 0; i < 3; ++i)
#pragma unroll
      for (int y = 0; y < 2; ++y)
#pragma unroll
        for (int x = 0; x < 4; ++x) s3[i][y][x] = 0.f;
#pragma unroll
    for (int c = 0; c < D / 16; ++c) {
      const float4 k = lds128(kb_u + (c >> 1) * C::BLK + g * 128 + (((2 * t + (c & 1)) ^ g) << 4));
      const float kf[4] = {k.x, k.y, k.z, k.w};
      const float q0[4] = {q[c][0].x, q[c][0].y, q[c][0].z, q[c][0].w};
      const float q1[4] = {q[c][1].x, q[c][1].y, q[c][1].z, q[c][1].w};
      uint32_t kh[4], kl[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) split32(kf[x], kh[x], kl[x]);
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        uint32_t ah[4], al[4];
        const float f[4] = {q0[2 * y], q1[2 * y], q0[2 * y + 1], q1[2 * y + 1]};
#pragma unroll
        for (int x = 0; x < 4; ++x)
          if constexpr (D == 128)
            split32_up_here(f[x], ah[x], al[x]);
          else
            split32_up(f[x], ah[x], al[x]);
        mma8(s3[0][y], ah, kh[2 * y], kh[2 * y + 1]);
        mma8(s3[1][y], ah, kl[2 * y], kl[2 * y + 1]);
        mma8(s3[2][y], al, kh[2 * y], kh[2 * y + 1]);
      }
    }
#pragma unroll
    for (int x = 0; x < 4; ++x)
      sc[0][x] = (s3[0][0][x] + s3[0][1][x]) +
                 ((s3[1][0][x] + s3[1][1][x]) + (s3[2][0][x] + s3[2][1][x]));
  }
  __device__ __forceinline__ static void add(uint32_t vb_u, int lane, const float (&p)[C::NT][4],
                                             float (&o)[D / 8][4]) {
    const int g = lane >> 2, t = lane & 3;
    uint32_t ph[4], pl[4];  // its keys 2 t and 2 t + 1 stand for t and t + 4
    split32_up(p[0][0], ph[0], pl[0]);
    split32_up(p[0][2], ph[1], pl[1]);
    split32_up(p[0][1], ph[2], pl[2]);
    split32_up(p[0][3], ph[3], pl[3]);
#pragma unroll
    for (int m = 0; m < D / 32; ++m) {
      const uint32_t at = vb_u + m * C::BLK + 2 * t * 128;
      const float4 v0 = lds128(at + ((g ^ (2 * t)) << 4));
      const float4 v1 = lds128(at + 128 + ((g ^ (2 * t + 1)) << 4));
      const float f0[4] = {v0.x, v0.y, v0.z, v0.w}, f1[4] = {v1.x, v1.y, v1.z, v1.w};
      uint32_t h0[4], l0[4], h1[4], l1[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        split32(f0[x], h0[x], l0[x]);
        split32(f1[x], h1[x], l1[x]);
      }
      float r[4][4];
#pragma unroll
      for (int x = 0; x < 4; ++x)
#pragma unroll
        for (int y = 0; y < 4; ++y) r[x][y] = 0.f;
#pragma unroll
      for (int x = 0; x < 4; ++x) mma8(r[x], ph, l0[x], l1[x]);
#pragma unroll
      for (int x = 0; x < 4; ++x) mma8(r[x], pl, h0[x], h1[x]);
#pragma unroll
      for (int x = 0; x < 4; ++x) mma8(r[x], ph, h0[x], h1[x]);
#pragma unroll
      for (int x = 0; x < 4; ++x)
#pragma unroll
        for (int y = 0; y < 4; ++y) o[4 * m + x][y] += r[x][y];
    }
  }
  __device__ __forceinline__ static int col(int d, int x, int lane) {
    return 32 * (d >> 2) + 8 * (lane & 3) + 4 * x + (d & 3);
  }
};

// 32 bits of V with non-finite values replaced by 0.
template <typename T> __device__ __forceinline__ uint32_t finite(uint32_t w) {
  if constexpr (sizeof(T) == 4)
    return (w & 0x7f800000u) == 0x7f800000u ? 0u : w;
  else
    return finite_bf16x2(w);
}

template <typename T> __device__ __forceinline__ float ex2(float x) {
  if constexpr (sizeof(T) == 4)
    return exp2f(x);
  else
    return ex2a(x);
}

// Slices of a sequence's item; its items are its KV heads' rows, 16 at a time.
template <typename T> __device__ __forceinline__ int slices(int rows) {
  constexpr int SL = FC<T, 64>::SL;
  return (rows + SL - 1) / SL;
}
template <typename T> __device__ __forceinline__ int seq_slices(const TreeSeq& s) {
  return s.n == 0 ? 0 : slices<T>(s.M) + slices<T>(s.cache);
}
template <typename T>
__device__ __forceinline__ int row_tiles(const TreeArgs& a, const TreeSeq& s) {
  return FC<T, 64>::F32 ? (s.n * a.G + 15) / 16 : 1;
}

// A worker's place in its range: slice j of item i of sequence b; `left`
// slices of the range from here on.
template <typename T> struct Cursor {
  TreeSeq s;
  int b, i, j, nt;
  int64_t left;
  __device__ __forceinline__ void size() { nt = seq_slices<T>(s); }
  // The KV head and the first row of item i.
  __device__ __forceinline__ int g(const TreeArgs& a) const { return i / row_tiles<T>(a, s); }
  __device__ __forceinline__ int row0(const TreeArgs& a) const {
    return i % row_tiles<T>(a, s) * 16;
  }
  // To slice 0 of the next item that has any (only while left > 0).
  template <typename Seq>
  __device__ __forceinline__ void next_item(const TreeArgs& a, Seq seq) {
    j = 0;
    if (++i < a.H * row_tiles<T>(a, s)) return;
    i = 0;
    do {
      s = seq(++b);
      size();
    } while (nt == 0);
  }
};

template <typename T, int D>
__global__ void __launch_bounds__(kFewThreads, 1)
tree_few_kernel(const __grid_constant__ CUtensorMap tm_km,
                const __grid_constant__ CUtensorMap tm_vm,
                const __grid_constant__ CUtensorMap tm_kp,
                const __grid_constant__ CUtensorMap tm_vp, const __grid_constant__ TreeArgs a,
                int part_rows, float* __restrict__ part_o, float2* __restrict__ part_ml,
                TreeCut* __restrict__ cuts) {
  using C = FC<T, D>;
  pdl_trigger();  // the merge: its blocks come as this grid's leave
  pdl_wait();
  extern __shared__ __align__(1024) unsigned char dsm[];
  __shared__ FewAux<T> aux;
  using Seen = typename FewAux<T>::Seen;
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
  int64_t items = 0;
  {
    int64_t mine = 0;
    int tiles = 0;
    for (int b = min(a.B, tid * per); b < min(a.B, (tid + 1) * per); ++b) {
      const TreeSeq s = tree_seq(a, b);
      if (s.error && blockIdx.x == 0) record_error(a.status, s.error);
      aux.seq[tid] = s;
      if (seq_slices<T>(s) > 0) tiles += row_tiles<T>(a, s);
      mine += (int64_t)seq_slices<T>(s) * a.H * row_tiles<T>(a, s);
    }
    const int w_tiles = __reduce_add_sync(0xffffffffu, tiles);
    if (lane == 0) aux.tiles[warp] = w_tiles;
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
      items += (int64_t)aux.tiles[i] * a.H;
    }
    __syncthreads();
    aux.pre[tid] = before + incl - mine;
    if (tid == 0) aux.pre[kFewThreads] = total;
    __syncthreads();
  }
  const int64_t total = aux.pre[kFewThreads];
  const int64_t worker = (int64_t)warp * gridDim.x + blockIdx.x;  // few: on as many SMs
  // Short items get a range each, which is an item where their lengths are equal;
  // of unlike ones the even borders cut most.  Of a long item a range costs its
  // length and the merge their number, so the least length goes with the root
  // of the item's; one slice is too little where that would fill every worker.
  // (33 sequences of 9 keys: 33 us with ranges of 6 slices at least, 8; 34 of
  // unlike lengths up to 175 keys 22; one item of 125 slices: 14 with 6, 12; of
  // 1,000: 18 with ranges of one, 17.)
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
  Cursor<T> ld;  // the slice to load next
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
      const int64_t n = (int64_t)ld.nt * a.H * row_tiles<T>(a, ld.s);
      if (lo < at + n || ld.b + 1 >= a.B) break;
      at += n;
      ++ld.b;
    }
    const int64_t off = lo - at;
    ld.i = (int)(off / ld.nt);
    ld.j = (int)(off - (int64_t)ld.i * ld.nt);
    ld.left = hi - lo;
  }
  Cursor<T> cu = ld;  // the slice to compute next
  if (ld.j > 0 && range_lo(worker - 1) <= lo - ld.j) {
    // the first border inside this item: its last part holds slice `end`
    const int64_t end = lo - ld.j + ld.nt - 1;
    int64_t c = min(n_work - 1, end * n_work / total);
    while (c + 1 < n_work && range_lo(c + 1) <= end) ++c;
    while (range_lo(c) > end) --c;
    cut.last = (int)c;
    cut.t0 = ld.s.t0;
    cut.g = ld.g(a);
    cut.row0 = ld.row0(a);
    cut.rows = min(ld.s.n * a.G - cut.row0, 16);
  }
  if (lane == 0) cuts[worker] = cut;

  // ------------------------------------------------------------------ loads
  // lane i holds the first tensor-map row of slice ids0 + i of the item
  int ids = -1, ids0 = 0;
  bool ids_fresh = true;
  auto issue = [&](int slot) {
    if (ld.left == 0) return;
    const int n_ms = slices<T>(ld.s.M);
    if (ids_fresh || ld.j >= ids0 + 32) {
      ids0 = ld.j;
      ids = -1;
      const int j = ids0 + lane;
      if (j < n_ms) {
        ids = ld.b * a.m_cap + j * C::SL;
      } else if (j < ld.nt) {
        const int r0 = (j - n_ms) * C::SL;
        const int pg = a.block_table[(int64_t)ld.b * a.max_pages + r0 / a.page_size];
        if (pg >= 0 && pg < a.n_pages)
          ids = (pg * a.H + ld.g(a)) * a.page_size + r0 % a.page_size;
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
                          mem ? ld.g(a) : 0, row);
          tc::tma_load_3d(d + (C::KB + kb) * C::BLK, mem ? &tm_vm : &tm_vp, &full[slot], kb * 64,
                          mem ? ld.g(a) : 0, row);
        }
      }
    }
    --ld.left;
    if (++ld.j == ld.nt && ld.left > 0) {
      ld.next_item(a, seq);
      ids_fresh = true;
    }
  };
#pragma unroll 1
  for (int i = 0; i < C::DEPTH; ++i) issue(i);

  // ---------------------------------------------------------------- compute
  const int c2 = 2 * (lane & 3);  // this thread's columns of an 8-column tile
  const int r4 = lane >> 2;       // its rows of a 16-row tile: r4, r4 + 8
  const uint32_t ring_u = tc::smem_u32(ring);
  bool ok = true;
  int slot = 0;
  uint32_t ph = 0;
  while (cu.left > 0 && ok) {
    // an item's share: its queries, trees, and slices
    const TreeSeq s = cu.s;
    const int g = cu.g(a), row0 = cu.row0(a);
    const int rows = min(s.n * a.G - row0, 16), n_ms = slices<T>(s.M);
    const int cnt = (int)min((int64_t)(cu.nt - cu.j), cu.left), j_lo = cu.j;
    const int part = j_lo > 0 ? 0 : cnt < cu.nt ? 1 : -1;
    Rows<T, D> q;
    int64_t out_row[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = row0 + r4 + 8 * h;
      out_row[h] = r4 + 8 * h < rows ? (s.t0 + r / a.G) * a.Hq + g * a.G + r % a.G : (int64_t)0;
      q.load(a.q, out_row[h], h, r4 + 8 * h < rows, lane);
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
    if (lane < rows) {
      Seen m;
      m.clear();
      int x = (row0 + lane) / a.G;
      if (a.parents) {
        do {
          m.set(x);
          x = aux.par[warp][x];
        } while (x >= 0);
        if (x != -1) m.clear();  // pruned: sees nothing
      } else {
        m.upto(x);
      }
      aux.seen[warp][lane] = m;
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
      const int key0 = (mem ? j : j - n_ms) * C::SL;
      const int n_rows = (mem ? s.M : s.cache) - key0;
      const bool all = key0 + C::SL <= (mem ? s.M : s.L);  // every row sees every key
      ok = tc::mbar_wait(&full[slot], ph);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      const uint32_t kb_u = ring_u + slot * C::SLICE, vb_u = kb_u + C::KB * C::BLK;

      float sc[C::NT][4];
      q.scores(kb_u, lane, sc);
      if (!all) {
        const uint32_t in = n_rows >= C::SL ? 0xffffu : (1u << n_rows) - 1;  // n_rows >= 1
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t vis = in;
          if (!mem) vis &= aux.seen[warp][r4 + 8 * h].from(key0 - s.L);
#pragma unroll
          for (int t = 0; t < C::NT; ++t)
#pragma unroll
            for (int x = 0; x < 2; ++x)
              if (!((vis >> (8 * t + c2 + x)) & 1)) sc[t][2 * h + x] = -INFINITY;
        }
        // clean V: rows past the end, non-finite drafted values
        unsigned char* v = ring + slot * C::SLICE + C::KB * C::BLK;
        bool bad = false;
        for (int c = lane; c < C::KB * C::SL * 8; c += 32) {
          const int r = (c / 8) % C::SL;  // 8 pieces of 16 bytes a row of a block
          uint4* p = reinterpret_cast<uint4*>(v + c * 16);
          if (r >= n_rows) {
            *p = make_uint4(0, 0, 0, 0);
          } else if (!mem && key0 + r >= s.L && s.n > 1) {
            const uint4 x = *p;
            const uint4 y =
                make_uint4(finite<T>(x.x), finite<T>(x.y), finite<T>(x.z), finite<T>(x.w));
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
        mx[h] = fmaxf(sc[0][2 * h], sc[0][2 * h + 1]);
        if constexpr (C::NT == 2) mx[h] = fmaxf(mx[h], fmaxf(sc[1][2 * h], sc[1][2 * h + 1]));
        mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 1));
        mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 2));
        mx[h] *= a.qscale;
      }
      // the reference maximum moves only when a slice exceeds it by 2^8
      const bool g0 = mx[0] > m_ref[0] + kRescaleLog2, g1 = mx[1] > m_ref[1] + kRescaleLog2;
      if (__any_sync(0xffffffffu, g0 || g1)) {
        const float al0 = !g0 ? 1.f : m_ref[0] == -INFINITY ? 0.f : ex2<T>(m_ref[0] - mx[0]);
        const float al1 = !g1 ? 1.f : m_ref[1] == -INFINITY ? 0.f : ex2<T>(m_ref[1] - mx[1]);
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
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float nm = m_ref[h] == -INFINITY ? 0.f : -m_ref[h];
#pragma unroll
        for (int t = 0; t < C::NT; ++t) {
          const float p0 = ex2<T>(fmaf(sc[t][2 * h], a.qscale, nm));
          const float p1 = ex2<T>(fmaf(sc[t][2 * h + 1], a.qscale, nm));
          l[h] += p0 + p1;
          sc[t][2 * h] = p0;
          sc[t][2 * h + 1] = p1;
        }
      }
      Rows<T, D>::add(vb_u, lane, sc, o);
      __syncwarp();  // every lane has read the slot
      issue(slot);
      if (++slot == C::DEPTH) {
        slot = 0;
        ph ^= 1;
      }
    }
    if (!ok) break;

    // write the item's share
    T* out = static_cast<T*>(a.out);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = r4 + 8 * h;
      float lr = l[h];
      lr += __shfl_xor_sync(0xffffffffu, lr, 1);
      lr += __shfl_xor_sync(0xffffffffu, lr, 2);
      if (r >= rows) continue;
      const Seen seen = aux.seen[warp][r];
      if (!seen.any()) lr = 0.f;  // pruned
      const int64_t prow = (worker * 2 + max(part, 0)) * part_rows + r;
      const float inv = lr == 0.f ? 0.f : part >= 0 ? 1.f : 1.f / lr;
      // (a row without weight: its O may hold 0 times NaN)
      auto at = [&](int d, int x) { return inv == 0.f ? 0.f : o[d][2 * h + x] * inv; };
      if constexpr (C::F32) {
        float* dst = part < 0 ? out + out_row[h] * D : part_o + prow * D;
#pragma unroll
        for (int d = 0; d < D / 8; d += 4)
#pragma unroll
          for (int x = 0; x < 2; ++x)
            *reinterpret_cast<float4*>(dst + Rows<T, D>::col(d, x, lane)) =
                make_float4(at(d, x), at(d + 1, x), at(d + 2, x), at(d + 3, x));
      } else {
#pragma unroll
        for (int d = 0; d < D / 8; ++d) {
          const int col = Rows<T, D>::col(d, 0, lane);
          if (part < 0)
            *reinterpret_cast<uint32_t*>(out + out_row[h] * D + col) = pack2(at(d, 0), at(d, 1));
          else
            *reinterpret_cast<float2*>(part_o + prow * D + col) = make_float2(at(d, 0), at(d, 1));
        }
      }
      if (part >= 0 && c2 == 0) part_ml[prow] = make_float2(m_ref[h], lr);
      if (!any_bad) continue;
      // drafted values taken out of V, added for the rows that see them
#pragma unroll 1
      for (int t = 0; t < s.n; ++t) {
        const int kr2 = s.L + t, j = n_ms + kr2 / C::SL;
        if (!seen.has(t) || j < j_lo || j >= j_lo + cnt || kr2 >= s.cache) continue;
        const int pg = a.block_table[(int64_t)cu.b * a.max_pages + kr2 / a.page_size];
        if (pg < 0 || pg >= a.n_pages) continue;
        const T* v = static_cast<const T*>(a.v_pages) +
                     (((int64_t)pg * a.H + g) * a.page_size + kr2 % a.page_size) * D;
#pragma unroll 1
        for (int d = 0; d < D / 4; ++d) {  // this thread's columns
          const int col = Rows<T, D>::col(d >> 1, d & 1, lane);
          const float f = Elem<T>::to_f(v[col]);
          if (isfinite(f)) continue;
          if (part < 0) {
            T* p = out + out_row[h] * D + col;
            *p = Elem<T>::from_f(Elem<T>::to_f(*p) + f);
          } else {
            part_o[prow * D + col] += f;
          }
        }
      }
    }
    cu.left -= cnt;
    cu.j += cnt;
    if (cu.left > 0) cu.next_item(a, seq);
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
  p.part_rows = std::min(n_max * G, 16);
  const size_t parts = 2 * (size_t)num_sms() * kWarps * p.part_rows;
  p.po_bytes = round_up(parts * D * sizeof(float), 256);
  p.ml_bytes = round_up(parts * sizeof(float2), 256);
  p.total = p.po_bytes + p.ml_bytes + round_up((size_t)num_sms() * kWarps * sizeof(TreeCut), 256);
  return p;
}

template <typename T, int D>
int launch_few(const TreeArgs& a, void* ws, cudaStream_t s) {
  using C = FC<T, D>;
  constexpr int W = D * sizeof(T) / 2;  // a row in the maps' 16-bit units
  const FewPlan p = few_plan(a.n_max, a.G, D);
  unsigned char* w = static_cast<unsigned char*>(ws);
  float* part_o = reinterpret_cast<float*>(w);
  float2* part_ml = reinterpret_cast<float2*>(w + p.po_bytes);
  TreeCut* cuts = reinterpret_cast<TreeCut*>(w + p.po_bytes + p.ml_bytes);
  CUtensorMap km, vm, kp, vp;
  const int64_t page_rows = (int64_t)a.n_pages * a.H * a.page_size;
  bool ok = tma_map_sw128_bf16(&kp, a.k_pages, W, 1, page_rows, 1, C::SL) &&
            tma_map_sw128_bf16(&vp, a.v_pages, W, 1, page_rows, 1, C::SL);
  if (a.m_cap > 0)
    ok = ok && tma_map_sw128_bf16(&km, a.k_mem, W, a.H, (int64_t)a.B * a.m_cap, 1, C::SL) &&
         tma_map_sw128_bf16(&vm, a.v_mem, W, a.H, (int64_t)a.B * a.m_cap, 1, C::SL);
  else
    km = kp, vm = vp;  // never loaded from
  if (!ok) return note_cuda(cudaErrorInvalidValue);
  auto kern = tree_few_kernel<T, D>;
  if (int rc = ensure_smem_attr(reinterpret_cast<const void*>(kern), (int)C::SMEM)) return rc;
  const unsigned grid = (unsigned)num_sms();
  if (int rc = launch_pdl(kern, dim3(grid), dim3(kFewThreads), C::SMEM, s, km, vm, kp, vp, a,
                          p.part_rows, part_o, part_ml, cuts))
    return rc;
  return tree_merge_launch(a, C::F32, D, (int)grid, kWarps, p.part_rows, part_o, part_ml, cuts,
                           s);
}

}  // namespace

size_t tree_few_workspace_size(int n_max, int G, int D) { return few_plan(n_max, G, D).total; }

int tree_few_launch(msa_dtype dt, const TreeArgs& a, int D, void* ws, cudaStream_t s) {
  if (dt == MSA_F32)
    return D == 64 ? launch_few<float, 64>(a, ws, s) : launch_few<float, 128>(a, ws, s);
  return D == 64 ? launch_few<__nv_bfloat16, 64>(a, ws, s)
                 : launch_few<__nv_bfloat16, 128>(a, ws, s);
}

}  // namespace msa
