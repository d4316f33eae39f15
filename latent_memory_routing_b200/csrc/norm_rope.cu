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
// bounds all three kernels.  A row's halves are loaded as 16-byte vectors by
// D / 2 / VEC neighbouring lanes (a thread holds VEC pairs: both partners of
// each), the mean is a shuffle over those lanes, and a warp works through
// the heads of one token so that the token's D/2 (cos, sin) are built once
// (two or fewer a lane, shared through shared memory) for all of them.
//
// The angle needs no double arithmetic on the device: the host gives each
// pair's frequency in turns as a 64-bit binary fraction f, and p * f modulo
// 2^64 is the exact fraction of a turn (error p 2^-64), rounded once to fp32
// for sincospif -- about 1e-7 rad at any 32-bit position, also a negative
// one.
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

TurnTab turn_tab(float base, int D) {
  TurnTab t{};
  const long double two_pi = 6.283185307179586476925286766559L;
  for (int i = 0; i < D / 2; ++i) {
    const long double turns = powl((long double)base, -2.0L * i / D) / two_pi;
    const long double frac = turns - floorl(turns);
    // 2^64 * frac, in two 32-bit steps (frac < 1)
    const long double hi = floorl(frac * 4294967296.0L);
    const long double lo = floorl((frac * 4294967296.0L - hi) * 4294967296.0L);
    t.f[i] = ((uint64_t)hi << 32) | (uint64_t)lo;
  }
  return t;
}

// (cos, sin) of position p at frequency f.
__device__ __forceinline__ float2 turn_cs(int32_t p, uint64_t f) {
  const uint64_t u = (uint64_t)(int64_t)p * f;
  const int32_t h = (int32_t)((u + 0x80000000ull) >> 32);  // 2^-32 turns, nearest
  float s, c;
  sincospif((float)h * 4.656612873077393e-10f, &s, &c);  // h 2^-31 half turns
  return make_float2(c, s);
}

// Plain (coherent) load that is not kept in L1: an output may alias its
// input exactly, so the read-only path is not used.
__device__ __forceinline__ uint4 ld16(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// N consecutive elements of type E as floats (16-byte aligned).
template <typename E, int N>
__device__ __forceinline__ void load_f(const E* p, float* f) {
#pragma unroll
  for (int i = 0; i < N; i += Vec16<E>::N) Vec16<E>::unpack(ld16(p + i), f + i);
}
template <typename E, int N>
__device__ __forceinline__ void store_f(E* p, const float* f) {
#pragma unroll
  for (int i = 0; i < N; i += Vec16<E>::N) st16(p + i, Vec16<E>::pack(f + i));
}

// How a warp's lanes lie over head rows of D elements of type T.
template <typename T, int D> struct RowMap {
  static constexpr int HALF = D / 2;
  static constexpr int VEC = Vec16<T>::N;       // pairs a thread holds
  static constexpr int LPR = HALF / VEC;        // lanes a row
  static constexpr int RPW = 32 / LPR;          // rows a warp
};

// Sum over the LPR lanes of a row.
template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = LPR / 2; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The token's (cos, sin) into cs[0 .. D/2), by one warp.
template <int HALF>
__device__ __forceinline__ void token_cs(const TurnTab& tab, int32_t p, float2* cs, int lane) {
  __syncwarp();  // earlier readers of cs are done
#pragma unroll
  for (int i = lane; i < HALF; i += 32) cs[i] = turn_cs(p, tab.f[i]);
  __syncwarp();
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

// Forward.  A warp takes one token and one of `splits` equal parts of its
// head rows: q heads, then k heads, then (append) v heads.
template <typename T, int D, bool kAppend>
__global__ void __launch_bounds__(kNRThreads)
norm_rope_kernel(const __grid_constant__ NRArgs a) {
  using M = RowMap<T, D>;
  constexpr int HALF = M::HALF, VEC = M::VEC;
  __shared__ float2 cs_all[kNRWarps][HALF];
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int l = lane % M::LPR, sub = lane / M::LPR;
  float2* cs = cs_all[warp];
  const int rows = a.Hq + a.H + (kAppend ? a.H : 0);
  const int groups = (rows + M::RPW - 1) / M::RPW;
  const int64_t n_work = a.n_tok * a.splits;
  for (int64_t w = (int64_t)blockIdx.x * kNRWarps + warp; w < n_work;
       w += (int64_t)gridDim.x * kNRWarps) {
    const int64_t t = w / a.splits;
    const int part = (int)(w % a.splits);
    const int h_lo = (int)((int64_t)part * groups / a.splits) * M::RPW;
    const int h_hi = min(rows, (int)((int64_t)(part + 1) * groups / a.splits) * M::RPW);
    int64_t cache_row = -1;  // row 0 of this token's head 0 in the pages, or none
    if (kAppend) {
      if (t < a.tok_offsets[0] || t >= a.tok_offsets[a.B]) continue;  // padding token
      const int64_t b = warp_find_segment(a.tok_offsets, a.B, t);
      const int64_t slot = (int64_t)a.cache_len[b] + (t - a.tok_offsets[b]);
      if (slot < 0) {
        if (lane == 0) record_error(a.status, MSA_ERR_INVALID_ARG);
      } else if (slot >= (int64_t)a.max_pages * a.page_size) {
        if (lane == 0) record_error(a.status, MSA_ERR_CAPACITY);
      } else {
        const int pg = a.block_table[b * a.max_pages + slot / a.page_size];
        if (pg < 0 || pg >= a.n_pages) {
          if (lane == 0) record_error(a.status, MSA_ERR_INVALID_ARG);
        } else {
          cache_row = (int64_t)pg * a.H * a.page_size + slot % a.page_size;
        }
      }
    }
    const bool rot = a.positions != nullptr;
    float c[VEC], s[VEC];
    if (rot) {
      token_cs<HALF>(a.tab, a.positions[t], cs, lane);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        c[e] = cs[l * VEC + e].x;
        s[e] = cs[l * VEC + e].y;
      }
    }
    for (int h0 = h_lo; h0 < h_hi; h0 += M::RPW) {
      const int h = h0 + sub;
      const bool ok = h < h_hi;
      const bool isq = h < a.Hq, isv = kAppend && h >= a.Hq + a.H;
      const T* src = nullptr;
      T* dst = nullptr;
      const T* wt = nullptr;
      if (ok && isq) {
        src = static_cast<const T*>(a.q) + t * a.q_stride + (int64_t)h * D;
        dst = static_cast<T*>(a.q_out) + (t * a.Hq + h) * D;
        wt = static_cast<const T*>(a.wq);
      } else if (ok) {
        const int g = isv ? h - a.Hq - a.H : h - a.Hq;
        src = isv ? static_cast<const T*>(a.v) + t * a.v_stride + (int64_t)g * D
                  : static_cast<const T*>(a.k) + t * a.k_stride + (int64_t)g * D;
        wt = isv ? nullptr : static_cast<const T*>(a.wk);
        if (kAppend) {
          if (cache_row >= 0)
            dst = static_cast<T*>(isv ? a.v_pages : a.k_pages) +
                  (cache_row + (int64_t)g * a.page_size) * D;
        } else {
          dst = static_cast<T*>(a.k_out) + (t * a.H + g) * D;
        }
      }
      float x1[VEC], x2[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) x1[e] = x2[e] = 0.f;
      if (dst) {
        load_f<T, VEC>(src + l * VEC, x1);
        load_f<T, VEC>(src + HALF + l * VEC, x2);
      }
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < VEC; ++e) ss = fmaf(x1[e], x1[e], fmaf(x2[e], x2[e], ss));
      ss = row_sum<M::LPR>(ss);
      if (!dst) continue;
      if (wt) {
        const float r = rsqrtf(ss * (1.f / D) + a.eps);
        float w1[VEC], w2[VEC];
        load_f<T, VEC>(wt + l * VEC, w1);
        load_f<T, VEC>(wt + HALF + l * VEC, w2);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          x1[e] *= r * w1[e];
          x2[e] *= r * w2[e];
        }
      }
      if (rot && !isv) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const float y1 = x1[e] * c[e] - x2[e] * s[e];
          x2[e] = x2[e] * c[e] + x1[e] * s[e];
          x1[e] = y1;
        }
      }
      store_f<T, VEC>(dst + l * VEC, x1);
      store_f<T, VEC>(dst + HALF + l * VEC, x2);
    }
  }
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

// Backward: warps walk the tokens, first over the q heads, then over the k
// heads, keeping the weight gradient of their lanes' dims in registers; each
// CTA writes one partial per weight, in fixed order.
template <typename T, typename E, int D>
__global__ void __launch_bounds__(kNRThreads)
norm_rope_backward_kernel(const __grid_constant__ NRBArgs a) {
  using M = RowMap<T, D>;
  constexpr int HALF = M::HALF, VEC = M::VEC;
  __shared__ float2 cs_all[kNRWarps][HALF];
  __shared__ float red[kNRWarps][D];
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int l = lane % M::LPR, sub = lane / M::LPR;
  float2* cs = cs_all[warp];
  const bool rot = a.positions != nullptr;
  for (int side = 0; side < 2; ++side) {
    const int heads = side ? a.H : a.Hq;
    if (heads == 0) continue;
    const T* x = static_cast<const T*>(side ? a.k : a.q);
    const int64_t xs = side ? a.k_stride : a.q_stride;
    const T* wt = static_cast<const T*>(side ? a.wk : a.wq);
    const E* dy = static_cast<const E*>(side ? a.dk_out : a.dq_out);
    E* dx = static_cast<E*>(side ? a.dk : a.dq);
    const int64_t ds = side ? a.dk_stride : a.dq_stride;
    float w1[VEC], w2[VEC], a1[VEC], a2[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) a1[e] = a2[e] = 0.f;
    if (wt) {
      load_f<T, VEC>(wt + l * VEC, w1);
      load_f<T, VEC>(wt + HALF + l * VEC, w2);
    }
    for (int64_t t = (int64_t)blockIdx.x * kNRWarps + warp; t < a.n_tok;
         t += (int64_t)gridDim.x * kNRWarps) {
      float c[VEC], s[VEC];
      if (rot) {
        token_cs<HALF>(a.tab, a.positions[t], cs, lane);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          c[e] = cs[l * VEC + e].x;
          s[e] = cs[l * VEC + e].y;
        }
      }
      for (int h0 = 0; h0 < heads; h0 += M::RPW) {
        const int h = h0 + sub;
        const bool ok = h < heads;
        float x1[VEC], x2[VEC], g1[VEC], g2[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) x1[e] = x2[e] = g1[e] = g2[e] = 0.f;
        if (ok) {
          const E* gp = dy + (t * heads + h) * D;
          load_f<E, VEC>(gp + l * VEC, g1);
          load_f<E, VEC>(gp + HALF + l * VEC, g2);
          if (wt) {
            const T* xp = x + t * xs + (int64_t)h * D;
            load_f<T, VEC>(xp + l * VEC, x1);
            load_f<T, VEC>(xp + HALF + l * VEC, x2);
          }
        }
        if (rot) {  // dz = R(-p) dy
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            const float z1 = g1[e] * c[e] + g2[e] * s[e];
            g2[e] = g2[e] * c[e] - g1[e] * s[e];
            g1[e] = z1;
          }
        }
        if (wt) {
          float ss = 0.f, gx = 0.f;
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            ss = fmaf(x1[e], x1[e], fmaf(x2[e], x2[e], ss));
            gx = fmaf(g1[e] * w1[e], x1[e], fmaf(g2[e] * w2[e], x2[e], gx));
          }
          ss = row_sum<M::LPR>(ss);
          gx = row_sum<M::LPR>(gx);
          const float r = ok ? rsqrtf(ss * (1.f / D) + a.eps) : 0.f;
          const float m = r * r * (gx * (1.f / D));  // r mean(g x r)
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            a1[e] = fmaf(g1[e], x1[e] * r, a1[e]);
            a2[e] = fmaf(g2[e], x2[e] * r, a2[e]);
            g1[e] = r * (g1[e] * w1[e] - x1[e] * m);
            g2[e] = r * (g2[e] * w2[e] - x2[e] * m);
          }
        }
        if (ok) {
          E* op = dx + t * ds + (int64_t)h * D;
          store_f<E, VEC>(op + l * VEC, g1);
          store_f<E, VEC>(op + HALF + l * VEC, g2);
        }
      }
    }
    if (!wt) continue;
    // the warp's rows, then the CTA's warps
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
#pragma unroll
      for (int o = M::LPR; o < 32; o <<= 1) {
        a1[e] += __shfl_xor_sync(0xffffffffu, a1[e], o);
        a2[e] += __shfl_xor_sync(0xffffffffu, a2[e], o);
      }
    }
    __syncthreads();  // earlier readers of red are done
    if (sub == 0) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        red[warp][l * VEC + e] = a1[e];
        red[warp][HALF + l * VEC + e] = a2[e];
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

// Sums the CTAs' partials of one weight (blockIdx.x: 0 = q, 1 = k): 1024 / D
// threads a dim, each a fixed stride of the CTAs, in double (a few hundred
// values; the sum is rounded once).
template <int D>
__global__ void __launch_bounds__(1024)
weight_grad_kernel(int n_part, const float* __restrict__ part, float* __restrict__ dwq,
                   float* __restrict__ dwk) {
  __shared__ double red[1024];
  pdl_trigger();
  pdl_wait();
  float* dw = blockIdx.x ? dwk : dwq;
  if (!dw) return;
  const int d = threadIdx.x % D, i0 = threadIdx.x / D;
  double v = 0.0;
  for (int i = i0; i < n_part; i += 1024 / D)
    v += (double)part[((int64_t)i * 2 + blockIdx.x) * D + d];
  red[threadIdx.x] = v;
  __syncthreads();
  if (i0 == 0) {
    for (int i = 1; i < 1024 / D; ++i) v += red[i * D + d];
    dw[d] = (float)v;
  }
}

// Parts a token's head rows are cut into: one warp a token once there are
// about 16 warps an SM, else parts of at least one warp-load of rows, so a
// short call still reaches every SM.
int head_splits(int64_t n_tok, int rows, int rpw) {
  const int64_t want = 16LL * num_sms();
  const int64_t s = (want + n_tok - 1) / n_tok;
  return (int)std::max<int64_t>(1, std::min<int64_t>(s, (rows + rpw - 1) / rpw));
}

template <typename T, int D, bool kAppend>
int launch_forward(NRArgs a, cudaStream_t s) {
  const int rows = a.Hq + a.H + (kAppend ? a.H : 0);
  a.splits = head_splits(a.n_tok, rows, RowMap<T, D>::RPW);
  const int64_t ctas = (a.n_tok * a.splits + kNRWarps - 1) / kNRWarps;
  const unsigned grid = (unsigned)std::min<int64_t>(ctas, 1 << 20);
  return launch_pdl(norm_rope_kernel<T, D, kAppend>, dim3(grid), dim3(kNRThreads), 0, s, a);
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
  return (int)std::max<int64_t>(1, std::min<int64_t>(ctas, 2LL * num_sms()));
}

template <typename T, typename E, int D>
int launch_backward(const NRBArgs& a, float* dwq, float* dwk, cudaStream_t s) {
  const int grid = backward_grid(a.n_tok);
  if (int rc = launch_pdl(norm_rope_backward_kernel<T, E, D>, dim3(grid), dim3(kNRThreads), 0, s,
                          a))
    return rc;
  if (!dwq && !dwk) return MSA_OK;
  return launch_pdl(weight_grad_kernel<D>, dim3(2), dim3(1024), 0, s, grid,
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
