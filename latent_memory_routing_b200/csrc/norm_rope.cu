// Per-head RMS norm of queries and keys with the position rotation in the
// same pass (forward and backward), and the append of a step's keys and
// values to a paged cache with both applied on the way.
//
// Mathematics, for one head row x of D elements at position p:
//   r = (mean_d x_d^2 + eps)^(-1/2),  z = x r w,  y = R(p) z,
// R(p) turning the pairs (i, i + D/2) by the angle p base^(-2i/D); a tensor
// without weight is rotated only (z = x).  Backward, from dy:
//   dz = R(-p) dy,  g = dz w,  dx = r (g - x r mean_d(g x r)),
//   dw = sum over rows of dz x r.
//
// Every row is read once and written once and nothing else is, so HBM
// bounds all three kernels.  A row's halves are 16-byte vectors of D / 2 /
// VEC neighbouring lanes (a thread holds VEC pairs: both partners of each), so
// the mean is a shuffle over those lanes and one pass of a warp takes
// 32 / lanes rows.  What feeds HBM is bytes in flight: a warp walks a
// contiguous run of tokens and each lane copies its own vectors of the passes
// to come into its own slots of shared memory (cp.async), kDepth passes
// ahead, with no barrier between lanes and no registers held (loads straight
// into registers reached 4.1 TB/s with one pass a warp in flight and 5.1 with
// five; this 6.2, the gradient 5.8, a plain copy 6.6).  A token's D / 2
// (cos, sin) are built once, two or fewer a lane, for all its rows.  Tokens
// of few rows leave lanes of a pass empty, and the instructions of a pass
// bound them instead: 123,000 tokens of 8 + 1 heads of 64, 2.6 TB/s.
//
// The angle needs no double arithmetic on the device: the host gives each
// pair's frequency in turns as a 64-bit binary fraction f, and p * f modulo
// 2^64 is the exact fraction of a turn (error p 2^-64), rounded once to
// 2^-32 of a turn and its rest of a quarter to fp32 -- about 1e-7 rad at any
// 32-bit position, also a negative one.
#include <algorithm>
#include <cmath>

#include "msa_common.cuh"

namespace msa {
namespace {

constexpr int kNRWarps = 8;
constexpr int kNRThreads = 32 * kNRWarps;
constexpr int kMaxHalf = 64;  // D / 2 at most

// Rotation frequencies of a call in turns: f[i] = base^(-2i/D) / (2 pi)
// modulo 1, times 2^64.
struct TurnTab {
  uint64_t f[kMaxHalf];
};

// One power a call (64 of them cost the host 15 us): the rest are products,
// whose relative error grows to i 2^-64, 2^-30 turns at the farthest position.
TurnTab turn_tab(float base, int D) {
  TurnTab t{};
  const long double ratio = powl((long double)base, -2.0L / D);
  long double turns = 1.0L / 6.283185307179586476925286766559L;
  for (int i = 0; i < D / 2; ++i, turns *= ratio) {
    const long double frac = turns - floorl(turns);
    t.f[i] = (uint64_t)(frac * 18446744073709551616.0L);  // frac < 1 exactly: no overflow
  }
  return t;
}

// 16 bytes into this lane's slot of shared memory.  (Global reads of the L2:
// an output may alias its input exactly.)
__device__ __forceinline__ void cp16(uint4* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                   (uint32_t)__cvta_generic_to_shared(dst)),
               "l"(src)
               : "memory");
}
__device__ __forceinline__ void cp_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
// This lane's copies are done but for those of the last N groups.
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Two floats in one 64-bit register: the arithmetic below runs on pairs
// (f32x2 instructions), two elements of a row each.
using f2 = unsigned long long;
__device__ __forceinline__ f2 mk2(float a, float b) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 un2(f2 v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
  f2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// 16 bytes of type E as Vec16<E>::N / 2 pairs, and back.
template <typename E>
__device__ __forceinline__ void pairs(const uint4& v, f2* p) {
  float f[Vec16<E>::N];
  Vec16<E>::unpack(v, f);
#pragma unroll
  for (int i = 0; i < Vec16<E>::N / 2; ++i) p[i] = mk2(f[2 * i], f[2 * i + 1]);
}
template <typename E>
__device__ __forceinline__ uint4 from_pairs(const f2* p) {
  float f[Vec16<E>::N];
#pragma unroll
  for (int i = 0; i < Vec16<E>::N / 2; ++i) {
    const float2 x = un2(p[i]);
    f[2 * i] = x.x;
    f[2 * i + 1] = x.y;
  }
  return Vec16<E>::pack(f);
}

// How a warp's lanes lie over head rows of D elements of type T.
template <typename T, int D> struct RowMap {
  static constexpr int HALF = D / 2;
  static constexpr int VEC = Vec16<T>::N;       // pairs a thread holds
  static constexpr int LPR = HALF / VEC;        // lanes a row
  static constexpr int RPW = 32 / LPR;          // rows a warp
};

// (cos, sin) of position p at N frequencies f.  The fraction of a turn, as a
// 32-bit integer, is cut into the nearest quarter turn and a rest of at most
// pi / 4, exactly; the rest's Taylor series (sine to x^9, cosine to x^10,
// errors below 3e-9) run on pairs, and the quarter turns swap and negate.
template <int N>
__device__ __forceinline__ void turn_cs(int32_t p, const uint64_t (&f)[N], float (&co)[N],
                                        float (&si)[N]) {
  int32_t quarter[2];
  float x[2] = {0.f, 0.f};
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const uint64_t u = (uint64_t)(int64_t)p * f[i];
    const int32_t h = (int32_t)((u + 0x80000000ull) >> 32);  // 2^-32 turns, nearest
    quarter[i] = (int32_t)((uint32_t)h + 0x20000000u) >> 30;
    const int32_t rest = (int32_t)((uint32_t)h - ((uint32_t)quarter[i] << 30));
    x[i] = (float)rest * 1.4629180792671596e-9f;  // 2 pi 2^-32
  }
  const f2 y = mk2(x[0], x[1]), z = mul2(y, y);
  auto k = [](float v) { return mk2(v, v); };
  f2 a = fma2(z, k(1.f / 362880), k(-1.f / 5040));
  a = fma2(z, a, k(1.f / 120));
  a = fma2(z, a, k(-1.f / 6));
  a = fma2(mul2(y, z), a, y);
  f2 b = fma2(z, k(-1.f / 3628800), k(1.f / 40320));
  b = fma2(z, b, k(-1.f / 720));
  b = fma2(z, b, k(1.f / 24));
  b = fma2(z, b, k(-.5f));
  b = fma2(z, b, k(1.f));
  const float sn[2] = {un2(a).x, un2(a).y}, cn[2] = {un2(b).x, un2(b).y};
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const bool odd = quarter[i] & 1;
    const uint32_t s_neg = (uint32_t)(quarter[i] & 2) << 30;
    const uint32_t c_neg = (uint32_t)((quarter[i] + 1) & 2) << 30;
    si[i] = __uint_as_float(__float_as_uint(odd ? cn[i] : sn[i]) ^ s_neg);
    co[i] = __uint_as_float(__float_as_uint(odd ? sn[i] : cn[i]) ^ c_neg);
  }
}

// The token's angles into cs[0 .. HALF) (cosines) and cs[HALF .. D) (sines),
// by one warp; f holds the lane's frequencies (read once: the constant bank
// serves one address at a time).
template <int HALF>
__device__ __forceinline__ void token_cs(const uint64_t (&f)[HALF / 32], int32_t p, float* cs,
                                         int lane) {
  float co[HALF / 32], si[HALF / 32];
  turn_cs(p, f, co, si);
  __syncwarp();  // earlier readers of cs are done
#pragma unroll
  for (int i = 0; i < HALF / 32; ++i) {
    cs[i * 32 + lane] = co[i];
    cs[HALF + i * 32 + lane] = si[i];
  }
  __syncwarp();
}

// The passes of a warp, in order: (token, part) work items w, w + step, ..,
// each a range of the token's row groups.
struct Passes {
  int64_t w, w_hi, step, t;
  int gi, g_hi;
  __device__ __forceinline__ bool more() const { return w < w_hi; }
  __device__ __forceinline__ void start(int splits, int groups) {
    if (splits == 1) {
      t = w;
      gi = 0;
      g_hi = groups;
    } else {
      t = w / splits;
      const int part = (int)(w - t * splits);
      gi = part * groups / splits;
      g_hi = (part + 1) * groups / splits;
    }
  }
  // Moves on; true when the next pass begins another work item.
  __device__ __forceinline__ bool next(int splits, int groups) {
    if (++gi < g_hi) return false;
    if ((w += step) < w_hi) start(splits, groups);
    return true;
  }
};

// What warp i of n takes of n_work items: a contiguous share (a long append:
// its tokens then mostly share a sequence; the backward pass: 87 us against
// 89), or every n-th item, so that the warps running together read and write
// neighbouring tokens (the norms: 114 us against 130).
__device__ __forceinline__ Passes warp_share(int64_t n_work, int64_t i, int64_t n, int splits,
                                             int groups, bool contiguous) {
  Passes p;
  p.w = contiguous ? n_work * i / n : i;
  p.w_hi = contiguous ? n_work * (i + 1) / n : n_work;
  p.step = contiguous ? 1 : n;
  p.t = 0;
  p.gi = p.g_hi = 0;
  if (p.more()) p.start(splits, groups);
  return p;
}

// A weight into shared memory in fp32 (ones without), by the whole CTA.
template <typename T, int D>
__device__ __forceinline__ void stage_weight(const void* w, float* out) {
  for (int d = threadIdx.x; d < D; d += kNRThreads)
    out[d] = w ? Elem<T>::to_f(static_cast<const T*>(w)[d]) : 1.f;
}
// N pairs from shared memory (16-byte aligned).
template <int N>
__device__ __forceinline__ void lds_pairs(const float* p, f2* out) {
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(p + 2 * i);
    out[i] = v.x;
    out[i + 1] = v.y;
  }
}

struct NRArgs {
  int64_t n_tok;
  int Hq, H, splits;
  const void *q, *k, *v;
  int64_t q_stride, k_stride, v_stride;  // elements from token to token
  const void *wq, *wk;
  const int32_t* positions;
  float eps;
  void *q_out, *k_out;
  // paged append only
  int B, max_pages, page_size, n_pages;
  const int64_t* tok_offsets;
  const int32_t *block_table, *cache_len;
  void *k_pages, *v_pages;
  int* status;
  TurnTab tab;
};

// Forward: rows a lane holds in a pass and passes in flight (6 KB a warp
// either way).  Two rows, two independent chains of arithmetic, serve the
// append, whose tokens are short and dear to place (22,000 tokens of 16 rows:
// 52 us with one row, 38 with two); one row serves the norms, which stream
// better in smaller steps (32,799 tokens of 40 rows: 114 us against 121).
template <bool kAppend> struct FwdCfg {
  static constexpr int ROWS = kAppend ? 2 : 1;
  static constexpr int DEPTH = 6 / ROWS;
};

template <typename T, int D, bool kAppend>
__global__ void __launch_bounds__(kNRThreads, 2)
norm_rope_kernel(const __grid_constant__ NRArgs a) {
  using M = RowMap<T, D>;
  constexpr int HALF = M::HALF, VEC = M::VEC, NP2 = VEC / 2;
  constexpr int U = FwdCfg<kAppend>::ROWS, kDepth = FwdCfg<kAppend>::DEPTH;
  constexpr int GR = M::RPW * U;                     // rows of a pass
  extern __shared__ __align__(16) uint4 ring_all[];  // [warp][kDepth][U][2][lane]
  __shared__ __align__(16) float cs_all[kNRWarps][D];
  __shared__ __align__(16) float wts[2][D];
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int l = lane % M::LPR, sub = lane / M::LPR;
  float* cs = cs_all[warp];
  uint4* ring = ring_all + warp * kDepth * U * 64 + lane;
  const int gq = (a.Hq + GR - 1) / GR, gk = (a.H + GR - 1) / GR;
  const int groups = gq + gk + (kAppend ? gk : 0);
  const bool rot = a.positions != nullptr;

  Passes at = warp_share(a.n_tok * a.splits, (int64_t)blockIdx.x * kNRWarps + warp,
                         (int64_t)gridDim.x * kNRWarps, a.splits, groups,
                         kAppend && a.splits == 1);
  Passes ahead = at;
  auto issue = [&](int slot) {
    if (ahead.more()) {
      const T* src;
      int r = ahead.gi, heads = a.H;
      if (r < gq) {
        heads = a.Hq;
        src = static_cast<const T*>(a.q) + ahead.t * a.q_stride;
      } else if (!kAppend || r < gq + gk) {
        r -= gq;
        src = static_cast<const T*>(a.k) + ahead.t * a.k_stride;
      } else {
        r -= gq + gk;
        src = static_cast<const T*>(a.v) + ahead.t * a.v_stride;
      }
      r = r * GR + sub;
      src += r * D + l * VEC;
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (r + u * M::RPW < heads) {
          uint4* d = ring + (slot * U + u) * 64;
          cp16(d, src + u * M::RPW * D);
          cp16(d + 32, src + u * M::RPW * D + HALF);
        }
      ahead.next(a.splits, groups);
    }
    cp_commit();
  };
#pragma unroll
  for (int i = 0; i < kDepth; ++i) issue(i);

  stage_weight<T, D>(a.wq, wts[0]);
  stage_weight<T, D>(a.wk, wts[1]);
  if (!rot)  // (the sines are not used)
    for (int i = lane; i < D; i += 32) cs[i] = i < HALF ? 1.f : 0.f;
  __syncthreads();
  uint64_t freq[HALF / 32];
#pragma unroll
  for (int i = 0; i < HALF / 32; ++i) freq[i] = a.tab.f[i * 32 + lane];

  // append: the sequence of the last token, and where this token's rows go:
  // row 0 of head 0 in the pages, -1: nowhere, -2: padding, nothing is written
  int64_t seq = -1, seq_lo = 0, seq_hi = -1, cache_row = -1;
  int seq_len = 0;
  const int64_t tok_lo = kAppend ? a.tok_offsets[0] : 0;
  const int64_t tok_hi = kAppend ? a.tok_offsets[a.B] : 0;
  // y1 = x1 ca + x2 cb, y2 = x2 cc + x1 cd, of x scaled by r: the weight and
  // the rotation of the token and tensor at hand
  f2 ca[NP2], cb[NP2], cc[NP2], cd[NP2];
  bool fresh = true;
  for (int slot = 0; at.more(); slot = slot + 1 == kDepth ? 0 : slot + 1) {
    const int64_t t = at.t;
    const int gi = at.gi;
    if (fresh) {
      if (kAppend) {
        cache_row = -2;
        if (t >= tok_lo && t < tok_hi) {
          cache_row = -1;
          if (t < seq_lo || t >= seq_hi) {
            seq = warp_find_segment(a.tok_offsets, a.B, t);
            seq_lo = a.tok_offsets[seq];
            seq_hi = a.tok_offsets[seq + 1];
            seq_len = a.cache_len[seq];
          }
          const int64_t row = (int64_t)seq_len + (t - seq_lo);
          if (row < 0) {
            if (lane == 0) record_error(a.status, MSA_ERR_INVALID_ARG);
          } else if (row >= (int64_t)a.max_pages * a.page_size) {
            if (lane == 0) record_error(a.status, MSA_ERR_CAPACITY);
          } else {
            const int pi = (int)row / a.page_size;  // row < 2^31: checked by the host
            const int pg = a.block_table[seq * a.max_pages + pi];
            if (pg < 0 || pg >= a.n_pages) {
              if (lane == 0) record_error(a.status, MSA_ERR_INVALID_ARG);
            } else {
              cache_row = (int64_t)pg * a.H * a.page_size + ((int)row - pi * a.page_size);
            }
          }
        }
      }
      if (rot) token_cs<HALF>(freq, a.positions[t], cs, lane);
    }
    const bool isq = gi < gq, isv = kAppend && gi >= gq + gk;
    const bool weighted = isq ? a.wq != nullptr : a.wk != nullptr;
    const bool copied = isv || !(weighted || rot);
    if ((fresh || gi == gq) && !copied) {
      f2 w1[NP2], w2[NP2], c[NP2], s[NP2];
      lds_pairs<NP2>(wts[!isq] + l * VEC, w1);
      lds_pairs<NP2>(wts[!isq] + HALF + l * VEC, w2);
      lds_pairs<NP2>(cs + l * VEC, c);
      lds_pairs<NP2>(cs + HALF + l * VEC, s);
#pragma unroll
      for (int e = 0; e < NP2; ++e) {
        ca[e] = mul2(w1[e], c[e]);
        cb[e] = mul2(w2[e], s[e]) ^ 0x8000000080000000ull;
        cc[e] = mul2(w2[e], c[e]);
        cd[e] = mul2(w1[e], s[e]);
      }
    }
    // this lane's first row: where it is written, the next U - 1 rows dst_step on
    const int r = (isq ? gi : isv ? gi - gq - gk : gi - gq) * GR + sub;
    int heads = isq ? a.Hq : a.H;
    T* dst;
    int64_t dst_step = M::RPW * D;
    if (isq) {
      dst = static_cast<T*>(a.q_out) + (t * a.Hq + r) * D;
      if (kAppend && cache_row == -2) heads = 0;
    } else if (!kAppend) {
      dst = static_cast<T*>(a.k_out) + (t * a.H + r) * D;
    } else {
      if (cache_row < 0) heads = 0;
      dst = static_cast<T*>(isv ? a.v_pages : a.k_pages) +
            (cache_row + (int64_t)r * a.page_size) * D;
      dst_step *= a.page_size;
    }
    dst += l * VEC;
    cp_wait<kDepth - 1>();
    uint4 r1[U], r2[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      r1[u] = ring[(slot * U + u) * 64];
      r2[u] = ring[(slot * U + u) * 64 + 32];
    }
    if (!copied) {
      f2 x1[U][NP2], x2[U][NP2];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        pairs<T>(r1[u], x1[u]);
        pairs<T>(r2[u], x2[u]);
      }
      if (weighted) {
        // (lanes without a row sum garbage among themselves)
        float ss[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          f2 s1 = mul2(x1[u][0], x1[u][0]), s2 = mul2(x2[u][0], x2[u][0]);
#pragma unroll
          for (int e = 1; e < NP2; ++e) {
            s1 = fma2(x1[u][e], x1[u][e], s1);
            s2 = fma2(x2[u][e], x2[u][e], s2);
          }
          ss[u] = (un2(s1).x + un2(s1).y) + (un2(s2).x + un2(s2).y);
        }
#pragma unroll
        for (int o = M::LPR / 2; o; o >>= 1)
#pragma unroll
          for (int u = 0; u < U; ++u) ss[u] += __shfl_xor_sync(0xffffffffu, ss[u], o);
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const float rs = rsqrtf(fmaf(ss[u], 1.f / D, a.eps));
          const f2 rr = mk2(rs, rs);
#pragma unroll
          for (int e = 0; e < NP2; ++e) {
            x1[u][e] = mul2(x1[u][e], rr);
            x2[u][e] = mul2(x2[u][e], rr);
          }
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (kAppend || rot) {
#pragma unroll
          for (int e = 0; e < NP2; ++e) {
            const f2 y1 = fma2(x1[u][e], ca[e], mul2(x2[u][e], cb[e]));
            x2[u][e] = fma2(x2[u][e], cc[e], mul2(x1[u][e], cd[e]));
            x1[u][e] = y1;
          }
        } else {  // (0 times an infinite partner would be NaN)
#pragma unroll
          for (int e = 0; e < NP2; ++e) {
            x1[u][e] = mul2(x1[u][e], ca[e]);
            x2[u][e] = mul2(x2[u][e], cc[e]);
          }
        }
        r1[u] = from_pairs<T>(x1[u]);
        r2[u] = from_pairs<T>(x2[u]);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (r + u * M::RPW < heads) {
        st16(dst + u * dst_step, r1[u]);
        st16(dst + u * dst_step + HALF, r2[u]);
      }
    issue(slot);  // this lane's reads of the slot have been used
    fresh = at.next(a.splits, groups);
  }
  cp_wait<0>();
}

struct NRBArgs {
  int64_t n_tok;
  int Hq, H;
  const void *q, *k;
  int64_t q_stride, k_stride;
  const void *wq, *wk;
  const int32_t* positions;
  float eps;
  const void *dq_out, *dk_out;
  void *dq, *dk;
  int64_t dq_stride, dk_stride;
  float* part;  // [grid][2][D] partial weight gradients
  TurnTab tab;
};

constexpr int kDepthBack = 2;  // backward: passes in flight, 2 or 3 KB each a warp

// Backward: the same walk over x and dy, first of q, then of k; the weight
// gradient of a lane's dims stays in registers over all its rows, each CTA
// writes one partial per weight, in a fixed order.
template <typename T, typename E, int D>
__global__ void __launch_bounds__(kNRThreads, 2)
norm_rope_backward_kernel(const __grid_constant__ NRBArgs a) {
  using M = RowMap<T, D>;
  constexpr int HALF = M::HALF, VEC = M::VEC, EV = VEC / Vec16<E>::N;
  constexpr int NP2 = VEC / 2, EP = Vec16<E>::N / 2;
  constexpr int NP = 2 + 2 * EV;                     // 16-byte pieces of a lane and pass
  extern __shared__ __align__(16) uint4 ring_all[];  // [warp][kDepthBack][NP][lane]
  __shared__ __align__(16) float cs_all[kNRWarps][D];
  __shared__ __align__(16) float wts[2][D];
  __shared__ float red[kNRWarps][D];
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int l = lane % M::LPR, sub = lane / M::LPR;
  float* cs = cs_all[warp];
  uint4* ring = ring_all + warp * kDepthBack * NP * 32 + lane;
  const bool rot = a.positions != nullptr;
  stage_weight<T, D>(a.wq, wts[0]);
  stage_weight<T, D>(a.wk, wts[1]);
  __syncthreads();
  uint64_t freq[HALF / 32];
#pragma unroll
  for (int i = 0; i < HALF / 32; ++i) freq[i] = a.tab.f[i * 32 + lane];

  for (int side = 0; side < 2; ++side) {
    const int heads = side ? a.H : a.Hq;
    if (heads == 0) continue;
    const T* x = static_cast<const T*>(side ? a.k : a.q);
    const int64_t xs = side ? a.k_stride : a.q_stride;
    const E* dy = static_cast<const E*>(side ? a.dk_out : a.dq_out);
    E* dx = static_cast<E*>(side ? a.dk : a.dq);
    const int64_t ds = side ? a.dk_stride : a.dq_stride;
    const bool weighted = side ? a.wk != nullptr : a.wq != nullptr;
    const int groups = (heads + M::RPW - 1) / M::RPW;
    Passes at = warp_share(a.n_tok, (int64_t)blockIdx.x * kNRWarps + warp,
                           (int64_t)gridDim.x * kNRWarps, 1, groups, true);
    Passes ahead = at;
    auto issue = [&](int slot) {
      if (ahead.more()) {
        const int r = ahead.gi * M::RPW + sub;
        if (r < heads) {
          uint4* d = ring + slot * NP * 32;
          const E* gp = dy + (ahead.t * heads + r) * D + l * VEC;
#pragma unroll
          for (int v = 0; v < EV; ++v) {
            cp16(d + 32 * (2 + v), gp + v * Vec16<E>::N);
            cp16(d + 32 * (2 + EV + v), gp + HALF + v * Vec16<E>::N);
          }
          if (weighted) {
            const T* xp = x + ahead.t * xs + r * D + l * VEC;
            cp16(d, xp);
            cp16(d + 32, xp + HALF);
          }
        }
        ahead.next(1, groups);
      }
      cp_commit();
    };
#pragma unroll
    for (int i = 0; i < kDepthBack; ++i) issue(i);

    f2 a1[NP2], a2[NP2];  // the weight's gradient
#pragma unroll
    for (int e = 0; e < NP2; ++e) a1[e] = a2[e] = 0;
    bool fresh = true;
    for (int slot = 0; at.more(); slot = slot + 1 == kDepthBack ? 0 : slot + 1) {
      const int64_t t = at.t;
      if (fresh && rot) token_cs<HALF>(freq, a.positions[t], cs, lane);
      const int r = at.gi * M::RPW + sub;
      const bool ok = r < heads;
      cp_wait<kDepthBack - 1>();
      const uint4* d = ring + slot * NP * 32;
      f2 x1[NP2], x2[NP2], g1[NP2], g2[NP2];
#pragma unroll
      for (int v = 0; v < EV; ++v) {
        pairs<E>(d[32 * (2 + v)], g1 + v * EP);
        pairs<E>(d[32 * (2 + EV + v)], g2 + v * EP);
      }
      pairs<T>(d[0], x1);
      pairs<T>(d[32], x2);
      if (!ok) {  // lanes without a row add zeros to the weight's gradient
#pragma unroll
        for (int e = 0; e < NP2; ++e) {
          x1[e] = x2[e] = mk2(1.f, 1.f);
          g1[e] = g2[e] = 0;
        }
      }
      if (rot) {  // dz = R(-p) dy
        f2 c[NP2], s[NP2];
        lds_pairs<NP2>(cs + l * VEC, c);
        lds_pairs<NP2>(cs + HALF + l * VEC, s);
#pragma unroll
        for (int e = 0; e < NP2; ++e) {
          const f2 z1 = fma2(g1[e], c[e], mul2(g2[e], s[e]));
          g2[e] = fma2(g2[e], c[e], mul2(g1[e], s[e]) ^ 0x8000000080000000ull);
          g1[e] = z1;
        }
      }
      if (weighted) {
        f2 w1[NP2], w2[NP2];
        lds_pairs<NP2>(wts[side] + l * VEC, w1);
        lds_pairs<NP2>(wts[side] + HALF + l * VEC, w2);
        f2 s1 = 0, s2 = 0, h1 = 0, h2 = 0;
#pragma unroll
        for (int e = 0; e < NP2; ++e) {
          s1 = fma2(x1[e], x1[e], s1);
          s2 = fma2(x2[e], x2[e], s2);
          w1[e] = mul2(g1[e], w1[e]);
          w2[e] = mul2(g2[e], w2[e]);
          h1 = fma2(w1[e], x1[e], h1);
          h2 = fma2(w2[e], x2[e], h2);
        }
        float ss = (un2(s1).x + un2(s1).y) + (un2(s2).x + un2(s2).y);
        float gx = (un2(h1).x + un2(h1).y) + (un2(h2).x + un2(h2).y);
#pragma unroll
        for (int o = M::LPR / 2; o; o >>= 1) {
          ss += __shfl_xor_sync(0xffffffffu, ss, o);
          gx += __shfl_xor_sync(0xffffffffu, gx, o);
        }
        const float rs = rsqrtf(fmaf(ss, 1.f / D, a.eps));
        const float m = -rs * rs * (gx * (1.f / D));  // - r mean(g x r)
        const f2 rr = mk2(rs, rs), mm = mk2(m, m);
#pragma unroll
        for (int e = 0; e < NP2; ++e) {
          a1[e] = fma2(g1[e], mul2(x1[e], rr), a1[e]);
          a2[e] = fma2(g2[e], mul2(x2[e], rr), a2[e]);
          g1[e] = mul2(rr, fma2(x1[e], mm, w1[e]));
          g2[e] = mul2(rr, fma2(x2[e], mm, w2[e]));
        }
      }
      if (ok) {
        E* op = dx + t * ds + r * D + l * VEC;
#pragma unroll
        for (int v = 0; v < EV; ++v) {
          st16(op + v * Vec16<E>::N, from_pairs<E>(g1 + v * EP));
          st16(op + HALF + v * Vec16<E>::N, from_pairs<E>(g2 + v * EP));
        }
      }
      issue(slot);  // this lane's reads of the slot have been used
      fresh = at.next(1, groups);
    }
    cp_wait<0>();
    if (!weighted) continue;

    // the warp's rows, then the CTA's warps
    __syncthreads();  // earlier readers of red are done
#pragma unroll
    for (int e = 0; e < NP2; ++e) {
      float v[4] = {un2(a1[e]).x, un2(a1[e]).y, un2(a2[e]).x, un2(a2[e]).y};
#pragma unroll
      for (int o = M::LPR; o < 32; o <<= 1)
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
      if (sub == 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) red[warp][(i >> 1) * HALF + l * VEC + 2 * e + (i & 1)] = v[i];
      }
    }
    __syncthreads();
    for (int d = threadIdx.x; d < D; d += kNRThreads) {
      float v = 0.f;
#pragma unroll
      for (int i = 0; i < kNRWarps; ++i) v += red[i][d];
      a.part[((int64_t)blockIdx.x * 2 + side) * D + d] = v;
    }
  }
}

// Sums the CTAs' partials: block (x, y) 32 dims from 32 x of the weight of q
// (y = 0) or k, thread (i, d) every 32nd partial; in double, in a fixed order,
// rounded once.
template <int D>
__global__ void __launch_bounds__(1024)
weight_grad_kernel(int n_part, const float* __restrict__ part, float* __restrict__ dwq,
                   float* __restrict__ dwk) {
  __shared__ double red[32][33];
  pdl_trigger();
  pdl_wait();
  float* dw = blockIdx.y ? dwk : dwq;
  if (!dw) return;
  const int d = threadIdx.x & 31, i0 = threadIdx.x >> 5;
  double v = 0.0;
#pragma unroll 4
  for (int i = i0; i < n_part; i += 32)
    v += (double)part[((int64_t)i * 2 + blockIdx.y) * D + blockIdx.x * 32 + d];
  red[i0][d] = v;
  __syncthreads();
  // warp i0 joins dim i0's 32 sums
  v = red[d][i0];
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (d == 0) dw[blockIdx.x * 32 + i0] = (float)v;
}

// Parts a token's row groups are cut into: whole tokens once a resident warp
// has four or more of them, else so many parts that there are about four a
// warp (the shares are then even, and a short call reaches every SM).
int head_splits(int64_t n_tok, int groups, int64_t warps) {
  const int64_t s = (4 * warps + n_tok - 1) / n_tok;
  return (int)std::max<int64_t>(1, std::min<int64_t>(s, groups));
}

constexpr int kCtasFwd = 2, kCtasBack = 2;  // resident on an SM

template <typename T, int D, bool kAppend>
int launch_forward(NRArgs a, cudaStream_t s) {
  using M = RowMap<T, D>;
  using F = FwdCfg<kAppend>;
  constexpr int GR = M::RPW * F::ROWS;
  const int gq = (a.Hq + GR - 1) / GR, gk = (a.H + GR - 1) / GR;
  const int64_t ctas = (int64_t)kCtasFwd * num_sms();
  a.splits = head_splits(a.n_tok, gq + gk * (kAppend ? 2 : 1), ctas * kNRWarps);
  const int64_t need = (a.n_tok * a.splits + kNRWarps - 1) / kNRWarps;
  constexpr int kSmem = kNRWarps * F::DEPTH * F::ROWS * 64 * 16;
  auto kern = norm_rope_kernel<T, D, kAppend>;
  if (int rc = ensure_smem_attr(reinterpret_cast<const void*>(kern), kSmem)) return rc;
  return launch_pdl(kern, dim3((unsigned)std::min(ctas, need)), dim3(kNRThreads), kSmem, s, a);
}

template <bool kAppend>
int dispatch_forward(msa_dtype dt, int D, const NRArgs& a, cudaStream_t s) {
  if (dt == MSA_F32)
    return D == 64 ? launch_forward<float, 64, kAppend>(a, s)
                   : launch_forward<float, 128, kAppend>(a, s);
  return D == 64 ? launch_forward<__nv_bfloat16, 64, kAppend>(a, s)
                 : launch_forward<__nv_bfloat16, 128, kAppend>(a, s);
}

int backward_grid(int64_t n_tok) {
  const int64_t ctas = (n_tok + kNRWarps - 1) / kNRWarps;
  return (int)std::max<int64_t>(1, std::min<int64_t>(ctas, (int64_t)kCtasBack * num_sms()));
}

template <typename T, typename E, int D>
int launch_backward(const NRBArgs& a, float* dwq, float* dwk, cudaStream_t s) {
  const int grid = backward_grid(a.n_tok);
  constexpr int kSmem = kNRWarps * kDepthBack * (2 + 2 * (RowMap<T, D>::VEC / Vec16<E>::N)) * 512;
  auto kern = norm_rope_backward_kernel<T, E, D>;
  if (int rc = ensure_smem_attr(reinterpret_cast<const void*>(kern), kSmem)) return rc;
  if (int rc = launch_pdl(kern, dim3(grid), dim3(kNRThreads), kSmem, s, a)) return rc;
  if (!dwq && !dwk) return MSA_OK;
  return launch_pdl(weight_grad_kernel<D>, dim3(D / 32, 2), dim3(1024), 0, s, grid,
                    static_cast<const float*>(a.part), dwq, dwk);
}

size_t esize(msa_dtype dt) { return dt == MSA_F32 ? 4 : 2; }
bool dtype_ok(msa_dtype dt) { return dt == MSA_F32 || dt == MSA_BF16; }

// A strided operand [n_tok][heads][D]: rows start on 16-byte boundaries and
// do not overlap.
bool rows_ok(const void* p, int64_t stride, int heads, int D, size_t es) {
  return p && aligned16(p) && stride >= (int64_t)heads * D && (stride * es) % 16 == 0;
}

// The checks shared by every call of this file; a MSA status.
int common_checks(msa_dtype dt, int64_t n_tok, int Hq, int H, int D, float eps, float rope_base) {
  if (!dtype_ok(dt) || n_tok < 0 || Hq < 0 || H < 0 || (int64_t)Hq + H == 0)
    return MSA_ERR_INVALID_ARG;
  if (!(eps >= 0.f) || !std::isfinite(eps) || !(rope_base > 0.f) || !std::isfinite(rope_base))
    return MSA_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return MSA_ERR_UNSUPPORTED;
  if (n_tok > INT32_MAX || Hq > 65536 || H > 65536) return MSA_ERR_UNSUPPORTED;
  return MSA_OK;
}

int forward_body(msa_dtype dt, int64_t n_tok, int Hq, int H, int D, const void* q,
                 int64_t q_stride, const void* k, int64_t k_stride, const void* q_weight,
                 const void* k_weight, const int32_t* positions, float eps, float rope_base,
                 void* q_out, void* k_out, cudaStream_t s) {
  if (int rc = common_checks(dt, n_tok, Hq, H, D, eps, rope_base)) return rc;
  if (n_tok == 0) return MSA_OK;
  const size_t es = esize(dt);
  if (Hq && (!rows_ok(q, q_stride, Hq, D, es) || !q_out || !aligned16(q_out)))
    return MSA_ERR_INVALID_ARG;
  if (H && (!rows_ok(k, k_stride, H, D, es) || !k_out || !aligned16(k_out)))
    return MSA_ERR_INVALID_ARG;
  if (!aligned16(q_weight) || !aligned16(k_weight)) return MSA_ERR_INVALID_ARG;
  NRArgs a{};
  a.n_tok = n_tok;
  a.Hq = Hq;
  a.H = H;
  a.q = q;
  a.k = k;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.wq = q_weight;
  a.wk = k_weight;
  a.positions = positions;
  a.eps = eps;
  a.q_out = q_out;
  a.k_out = k_out;
  a.tab = turn_tab(rope_base, D);
  return dispatch_forward<false>(dt, D, a, s);
}

int append_body(msa_dtype dt, int B, int64_t n_tok, int Hq, int H, int D, const void* q,
                int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                int64_t v_stride, const void* q_weight, const void* k_weight,
                const int64_t* tok_offsets, const int32_t* positions, float eps,
                float rope_base, const int32_t* block_table, int max_pages,
                const int32_t* cache_len, int page_size, int n_pages, void* k_pages,
                void* v_pages, void* q_out, cudaStream_t s) {
  if (int rc = common_checks(dt, n_tok, Hq, H, D, eps, rope_base)) return rc;
  if (B <= 0 || H <= 0 || max_pages <= 0 || n_pages <= 0) return MSA_ERR_INVALID_ARG;
  if (page_size != 16 && page_size != 32 && page_size != 64 && page_size != 128)
    return MSA_ERR_UNSUPPORTED;
  if ((int64_t)n_pages * H * page_size > INT32_MAX || (int64_t)max_pages * page_size > INT32_MAX)
    return MSA_ERR_UNSUPPORTED;
  if (!tok_offsets || !block_table || !cache_len) return MSA_ERR_INVALID_ARG;
  if (!k_pages || !v_pages || !aligned16(k_pages) || !aligned16(v_pages))
    return MSA_ERR_INVALID_ARG;
  if (n_tok == 0) return MSA_OK;
  if (!positions) return MSA_ERR_INVALID_ARG;
  const size_t es = esize(dt);
  if (!rows_ok(k, k_stride, H, D, es) || !rows_ok(v, v_stride, H, D, es))
    return MSA_ERR_INVALID_ARG;
  if (Hq && (!rows_ok(q, q_stride, Hq, D, es) || !q_out || !aligned16(q_out)))
    return MSA_ERR_INVALID_ARG;
  if (!aligned16(q_weight) || !aligned16(k_weight)) return MSA_ERR_INVALID_ARG;
  if (int rc = debug_check_offsets(tok_offsets, B, n_tok, s)) return rc;
  if (int rc = debug_check_mem_len(cache_len, B, max_pages * page_size, s)) return rc;
  NRArgs a{};
  a.n_tok = n_tok;
  a.Hq = Hq;
  a.H = H;
  a.q = q;
  a.k = k;
  a.v = v;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.wq = q_weight;
  a.wk = k_weight;
  a.positions = positions;
  a.eps = eps;
  a.q_out = q_out;
  a.B = B;
  a.max_pages = max_pages;
  a.page_size = page_size;
  a.n_pages = n_pages;
  a.tok_offsets = tok_offsets;
  a.block_table = block_table;
  a.cache_len = cache_len;
  a.k_pages = k_pages;
  a.v_pages = v_pages;
  a.status = device_status_ptr();
  a.tab = turn_tab(rope_base, D);
  return dispatch_forward<true>(dt, D, a, s);
}

int backward_body(msa_dtype dt, msa_dtype grad_dt, int64_t n_tok, int Hq, int H, int D,
                  const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                  const void* q_weight, const void* k_weight, const int32_t* positions,
                  float eps, float rope_base, const void* dq_out, const void* dk_out, void* dq,
                  int64_t dq_stride, void* dk, int64_t dk_stride, float* dq_weight,
                  float* dk_weight, void* ws, size_t ws_bytes, cudaStream_t s) {
  if (int rc = common_checks(dt, n_tok, Hq, H, D, eps, rope_base)) return rc;
  if (!dtype_ok(grad_dt)) return MSA_ERR_INVALID_ARG;
  if (dt == MSA_F32 && grad_dt != MSA_F32) return MSA_ERR_UNSUPPORTED;
  const bool wq = Hq && q_weight, wk = H && k_weight;
  // a weight's gradient is asked for exactly where the weight is given
  if (wq != (dq_weight != nullptr) || wk != (dk_weight != nullptr)) return MSA_ERR_INVALID_ARG;
  if (n_tok == 0) {  // empty sums
    if (wq)
      if (int rc = note_cuda(cudaMemsetAsync(dq_weight, 0, D * sizeof(float), s))) return rc;
    if (wk)
      if (int rc = note_cuda(cudaMemsetAsync(dk_weight, 0, D * sizeof(float), s))) return rc;
    return MSA_OK;
  }
  const size_t es = esize(dt), gs = esize(grad_dt);
  if (Hq && (!rows_ok(q, q_stride, Hq, D, es) || !rows_ok(dq, dq_stride, Hq, D, gs) || !dq_out ||
             !aligned16(dq_out)))
    return MSA_ERR_INVALID_ARG;
  if (H && (!rows_ok(k, k_stride, H, D, es) || !rows_ok(dk, dk_stride, H, D, gs) || !dk_out ||
            !aligned16(dk_out)))
    return MSA_ERR_INVALID_ARG;
  if (!aligned16(q_weight) || !aligned16(k_weight)) return MSA_ERR_INVALID_ARG;
  const size_t need = (size_t)backward_grid(n_tok) * 2 * D * sizeof(float);
  if ((wq || wk) && (!ws || ws_bytes < need || !aligned16(ws))) return MSA_ERR_WORKSPACE;
  NRBArgs a{};
  a.n_tok = n_tok;
  a.Hq = Hq;
  a.H = H;
  a.q = q;
  a.k = k;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.wq = q_weight;
  a.wk = k_weight;
  a.positions = positions;
  a.eps = eps;
  a.dq_out = dq_out;
  a.dk_out = dk_out;
  a.dq = dq;
  a.dk = dk;
  a.dq_stride = dq_stride;
  a.dk_stride = dk_stride;
  a.part = static_cast<float*>(ws);
  a.tab = turn_tab(rope_base, D);
  if (dt == MSA_F32)
    return D == 64 ? launch_backward<float, float, 64>(a, dq_weight, dk_weight, s)
                   : launch_backward<float, float, 128>(a, dq_weight, dk_weight, s);
  if (grad_dt == MSA_F32)
    return D == 64 ? launch_backward<__nv_bfloat16, float, 64>(a, dq_weight, dk_weight, s)
                   : launch_backward<__nv_bfloat16, float, 128>(a, dq_weight, dk_weight, s);
  return D == 64 ? launch_backward<__nv_bfloat16, __nv_bfloat16, 64>(a, dq_weight, dk_weight, s)
                 : launch_backward<__nv_bfloat16, __nv_bfloat16, 128>(a, dq_weight, dk_weight, s);
}

}  // namespace
}  // namespace msa

extern "C" int msa_qk_norm_rope(msa_dtype dt, int64_t n_tok, int Hq, int H, int D, const void* q,
                                int64_t q_stride, const void* k, int64_t k_stride,
                                const void* q_weight, const void* k_weight,
                                const int32_t* positions, float eps, float rope_base,
                                void* q_out, void* k_out, msa_stream_t stream) {
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return msa::debug_finish(
      msa::forward_body(dt, n_tok, Hq, H, D, q, q_stride, k, k_stride, q_weight, k_weight,
                        positions, eps, rope_base, q_out, k_out, s),
      s);
}

extern "C" size_t msa_qk_norm_rope_backward_workspace_size(int64_t n_tok, int D) {
  if (n_tok <= 0 || D <= 0) return 0;
  return (size_t)msa::backward_grid(n_tok) * 2 * D * sizeof(float);
}

extern "C" int msa_qk_norm_rope_backward(
    msa_dtype dt, msa_dtype grad_dt, int64_t n_tok, int Hq, int H, int D, const void* q,
    int64_t q_stride, const void* k, int64_t k_stride, const void* q_weight,
    const void* k_weight, const int32_t* positions, float eps, float rope_base,
    const void* dq_out, const void* dk_out, void* dq, int64_t dq_stride, void* dk,
    int64_t dk_stride, float* dq_weight, float* dk_weight, void* ws, size_t ws_bytes,
    msa_stream_t stream) {
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return msa::debug_finish(
      msa::backward_body(dt, grad_dt, n_tok, Hq, H, D, q, q_stride, k, k_stride, q_weight,
                         k_weight, positions, eps, rope_base, dq_out, dk_out, dq, dq_stride, dk,
                         dk_stride, dq_weight, dk_weight, ws, ws_bytes, s),
      s);
}

extern "C" int msa_paged_append(msa_dtype dt, int B, int64_t n_tok, int Hq, int H, int D,
                                const void* q, int64_t q_stride, const void* k,
                                int64_t k_stride, const void* v, int64_t v_stride,
                                const void* q_weight, const void* k_weight,
                                const int64_t* tok_offsets, const int32_t* positions, float eps,
                                float rope_base, const int32_t* block_table, int max_pages,
                                const int32_t* cache_len, int page_size, int n_pages,
                                void* k_pages, void* v_pages, void* q_out,
                                msa_stream_t stream) {
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return msa::debug_finish(
      msa::append_body(dt, B, n_tok, Hq, H, D, q, q_stride, k, k_stride, v, v_stride, q_weight,
                       k_weight, tok_offsets, positions, eps, rope_base, block_table, max_pages,
                       cache_len, page_size, n_pages, k_pages, v_pages, q_out, s),
      s);
}
