// RMS norm of each query and key head, with the rotary position in the same
// pass, and its gradient.
//
//     h = x r,  r = 1 / sqrt(mean(x^2) + eps),     y = R (w h)
//
// over the d dims of one head's row; R turns the pairs of the first `rot` dims
// by the row's position and scales them by mscale (rotary.cu).  R's transpose
// turns back with the same factor, so with g = R^T dy and c = w g
//
//     dx = r (c - h mean(c h)),     dw = sum over the rows of g h.
//
// Everything is fp32 and rounded once, at the store.  A pass moves every row in
// and out once; both kernels are bound by memory.
//
// The lanes of a row: each holds two runs of V dims of 16 bytes, the runs that
// the rotation pairs (rotary.cuh), so that the mean is log2(d / 2V) shuffles
// and the rotation needs no exchange.  Rows that do not fit this (d / 2V no
// power of two up to 32, strides, alignment, rot no multiple of 2V) go to a
// warp a row through shared memory.
#include <cuda_bf16.h>

#include <cmath>
#include <cstdint>

#include "kernels.h"
#include "paged.h"
#include "rotary.cuh"

namespace blkattn {
namespace {

constexpr int kThreads = 256;
constexpr int kMostHeads = 8;  // heads of one thread and token

// The query heads (set 0) or the key heads (set 1).
struct NormSet {
  const void* x;
  int64_t x_b, x_h, x_t, x_d;
  const void* w;  // nullptr: rows are not normed
  int64_t w_s;
  void* y;  // forward: the result; backward: dx
  int64_t y_b, y_h, y_t, y_d;
  const void* g;  // backward: dy
  int64_t g_b, g_h, g_t, g_d;
  float* dw;  // backward
  int64_t dw_s;
  int heads;
};

struct NormParams {
  NormSet set[2];
  int n_sets;
  const int32_t* pos;
  int64_t p_b, p_t;
  const int64_t* phases;
  int64_t ph_s;
  bool w_f32;
  bool skip_negative;  // rows at a negative position are left out
  float mscale, eps, inv_d;
  int rot, d, B, T;
  int hg;         // heads of a thread (fast kernels)
  int groups[2];  // ceil(heads / hg) of each set
  int blocks;     // backward: blocks along the tokens
  float* ws;      // backward: partial dw [block of the grid][d]
};

__device__ __forceinline__ float weight_at(const NormSet& s, bool f32, int i) {
  if (s.w == nullptr) return 1.f;
  return f32 ? static_cast<const float*>(s.w)[i * s.w_s]
             : __bfloat162float(static_cast<const __nv_bfloat16*>(s.w)[i * s.w_s]);
}

// What a lane of the fast kernels holds of every row: item `it` of d / 2V, the
// two runs at a0 and a1.
struct Item {
  int it, a0, a1;
  bool turn;
};
template <int V>
__device__ __forceinline__ Item item_of(int it, int rot, int d) {
  Item m;
  m.it = it;
  m.turn = it < rot / (2 * V);
  const int part0 = m.turn ? 0 : rot, part = m.turn ? rot : d - rot;
  m.a0 = part0 + V * (it - part0 / (2 * V));
  m.a1 = m.a0 + part / 2;
  return m;
}

// Arithmetic on pairs of neighbouring dims (.f32x2): half the instructions.
__device__ __forceinline__ uint64_t fmul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ float sum2(uint64_t a) {
  float lo, hi;
  f2_split(a, lo, hi);
  return lo + hi;
}

// The angles of an item's V pairs, for two runs of V dims as V pairs of
// neighbours: x[0 .. V/2) the first run, x[V/2 .. V) the second.
template <int V, bool INTER>
struct Angles {
  float sn[INTER ? V : 1], cs[INTER ? V : 1];
  uint64_t c[INTER ? 1 : V / 2], s[INTER ? 1 : V / 2], ns[INTER ? 1 : V / 2];
  __device__ void take(const NormParams& p, const Item& m, int pos, float sign) {
    if (!m.turn) return;
    float a[V], b[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int pair = !INTER ? V * m.it + j : (j < V / 2 ? m.a0 / 2 + j : m.a1 / 2 + j - V / 2);
      turn_of(pos, p.phases[pair * p.ph_s], b[j], a[j]);
      b[j] *= sign * p.mscale;
      a[j] *= p.mscale;
      if constexpr (INTER) {
        sn[j] = b[j];
        cs[j] = a[j];
      }
    }
    if constexpr (!INTER) {
#pragma unroll
      for (int j = 0; j < V / 2; ++j) {
        c[j] = f2(a[2 * j], a[2 * j + 1]);
        s[j] = f2(b[2 * j], b[2 * j + 1]);
        ns[j] = f2(-b[2 * j], -b[2 * j + 1]);
      }
    }
  }
  __device__ __forceinline__ void turn(const Item& m, uint64_t (&x)[V]) const {
    if (!m.turn) return;
#pragma unroll
    for (int j = 0; j < (INTER ? V : V / 2); ++j) {
      if constexpr (INTER) {
        float u, v;
        f2_split(x[j], u, v);
        x[j] = f2(u * cs[j] - v * sn[j], u * sn[j] + v * cs[j]);
      } else {
        const uint64_t u = x[j], v = x[V / 2 + j];
        x[j] = ffma2(u, c[j], fmul2(v, ns[j]));
        x[V / 2 + j] = ffma2(v, c[j], fmul2(u, s[j]));
      }
    }
  }
};
// 16 bytes as pairs: 4 of bf16, 2 of f32.
template <typename T>
__device__ __forceinline__ void pairs_of(const uint4& w, uint64_t* x) {
  const uint32_t* v = &w.x;
  if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = f2(bf16lo(v[j]), bf16hi(v[j]));
  } else {
#pragma unroll
    for (int j = 0; j < 2; ++j) x[j] = f2(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1]));
  }
}
template <typename TO, int V>
__device__ __forceinline__ void store_pairs(TO* dst, const Item& m, const uint64_t (&x)[V]) {
  float y[2 * V];
#pragma unroll
  for (int j = 0; j < V; ++j) f2_split(x[j], y[2 * j], y[2 * j + 1]);
  Vec<TO, V> y0, y1;
  pack_runs<TO, V>(y, y0, y1);
  store(dst + m.a0, y0);
  store(dst + m.a1, y1);
}
template <int V>
__device__ __forceinline__ void weights_of(const NormParams& p, const NormSet& s, const Item& m, uint64_t (&w)[V]) {
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int i = j < V / 2 ? m.a0 + 2 * j : m.a1 + 2 * j - V;
    w[j] = f2(weight_at(s, p.w_f32, i), weight_at(s, p.w_f32, i + 1));
  }
}

// The lanes of a thread's row, n (a power of two) neighbours.
__device__ __forceinline__ unsigned lanes_of_row(int n) {
  const int lane = threadIdx.x & 31;
  return (n == 32 ? 0xffffffffu : (1u << n) - 1) << (lane & ~(n - 1));
}

// Pairs of rows (two heads of a token) in a thread's slots (its own, in shared
// memory): one at work, the others on their way.
constexpr int kRing = 4;
constexpr int kResident = 2;  // blocks of either kernel on an SM (three spill; the gradient of f32 rows and f32
                              // gradients has 128 KB of slots, and its blocks run in two waves)

// V elements (16 or 8 bytes) of a row to the thread's slot, and from there.
template <typename T, int V>
struct Slot {
  static constexpr int kBytes = V * (int)sizeof(T);
  static_assert(kBytes == 16 || kBytes == 8, "one copy");
  static __device__ __forceinline__ void copy(unsigned char* block, const T* src) {
    const uint32_t at = smem_u32(block + threadIdx.x * kBytes);
    if constexpr (kBytes == 16) cp_async_16(at, src, 16);
    else asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(at), "l"(src) : "memory");
  }
  static __device__ __forceinline__ void pairs(const unsigned char* block, uint64_t* x) {
    if constexpr (kBytes == 16) {
      pairs_of<T>(reinterpret_cast<const uint4*>(block)[threadIdx.x], x);
    } else {
      const uint2 w = reinterpret_cast<const uint2*>(block)[threadIdx.x];
      x[0] = f2(bf16lo(w.x), bf16hi(w.x));
      x[1] = f2(bf16lo(w.y), bf16hi(w.y));
    }
  }
};

// The rows that a thread takes: hg heads of one token, then those of the token
// `step` further, with its item of each.
struct Walk {
  int64_t tok;
  int k, b, t, pos;
  // the walk's first token from `token` on that is not left out
  __device__ void at(const NormParams& p, int64_t token, int64_t step) {
    k = 0;
    for (tok = token;; tok += step) {
      b = (int)tok / p.T;  // B T < 2^31
      t = (int)tok - b * p.T;
      if (p.pos == nullptr || tok >= (int64_t)p.B * p.T) return;
      pos = p.pos[b * p.p_b + t * p.p_t];
      if (!p.skip_negative || pos >= 0) return;
    }
  }
};

// Forward: persistent blocks; a thread walks over its tokens with its item of
// the rows, two heads at a time (one alone leaves the chain of its sum and
// shuffles with nothing beside it), the next ones on their way to shared memory
// (asynchronous copies: no register holds them).  2 x 8192 tokens of 32 and 8
// heads: 59 us; a block for each 32 tokens, all heads copied and then
// computed as in the rotary kernel, 62.
template <typename TI, typename TO, int V, bool INTER>
__global__ void __launch_bounds__(kThreads, kResident) norm_kernel(const __grid_constant__ NormParams p) {
  using SX = Slot<TI, V>;
  constexpr int kRow = 2 * SX::kBytes * kThreads;
  const int si = blockIdx.y >= p.groups[0] ? 1 : 0;
  const NormSet& s = p.set[si];
  const int h0 = ((int)blockIdx.y - (si ? p.groups[0] : 0)) * p.hg, nh = min(p.hg, s.heads - h0);
  const int items = p.d / (2 * V);  // (a power of two)
  const int per_block = kThreads / items;
  const Item m = item_of<V>(threadIdx.x & (items - 1), p.rot, p.d);
  const unsigned lanes = lanes_of_row(items);
  const int64_t n_tok = (int64_t)p.B * p.T, step = (int64_t)gridDim.x * per_block;
  Walk cur, next;
  next.at(p, (int64_t)blockIdx.x * per_block + threadIdx.x / items, step);
  cur = next;
  auto row_x = [&](const Walk& a) { return static_cast<const TI*>(s.x) + (a.b * s.x_b + a.t * s.x_t + h0 * s.x_h); };
  auto row_y = [&](const Walk& a) { return static_cast<TO*>(s.y) + (a.b * s.y_b + a.t * s.y_t + h0 * s.y_h); };
  const TI* x_in = row_x(next);
  TO* y_out = row_y(cur);
  extern __shared__ __align__(16) unsigned char slots[];
  int put = 0, get = 0;
  auto issue = [&]() {
    if (next.tok < n_tok) {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        if (next.k + r < nh) {
          unsigned char* at = slots + (2 * put + r) * kRow;
          SX::copy(at, x_in + m.a0);
          SX::copy(at + SX::kBytes * kThreads, x_in + m.a1);
          x_in += s.x_h;
        }
      }
      if ((next.k += 2) >= nh) {
        next.at(p, next.tok + step, step);
        x_in = row_x(next);
      }
    }
    put = (put + 1) & (kRing - 1);
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int i = 0; i < kRing - 1; ++i) issue();
  uint64_t w[V];
  weights_of<V>(p, s, m, w);
  Angles<V, INTER> angles;
  if (p.rot && cur.tok < n_tok) angles.take(p, m, cur.pos, 1.f);
  while (cur.tok < n_tok) {  // (whole rows leave)
    issue();
    asm volatile("cp.async.wait_group %0;" ::"n"(kRing - 1) : "memory");
    const bool two = cur.k + 1 < nh;
    uint64_t x[2][V];
#pragma unroll
    for (int r = 0; r < 2; ++r) {  // (what an absent row's slots hold is not used)
      const unsigned char* at = slots + (2 * get + r) * kRow;
      SX::pairs(at, x[r]);
      SX::pairs(at + SX::kBytes * kThreads, x[r] + V / 2);
    }
    get = (get + 1) & (kRing - 1);
    if (s.w != nullptr) {
      float ss[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        uint64_t a = fmul2(x[r][0], x[r][0]);
#pragma unroll
        for (int j = 1; j < V; ++j) a = ffma2(x[r][j], x[r][j], a);
        ss[r] = sum2(a);
      }
      for (int off = items >> 1; off >= 1; off >>= 1) {
#pragma unroll
        for (int r = 0; r < 2; ++r) ss[r] += __shfl_xor_sync(lanes, ss[r], off);
      }
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float rs = rsqrtf(fmaf(ss[r], p.inv_d, p.eps));
        const uint64_t rr = f2(rs, rs);
#pragma unroll
        for (int j = 0; j < V; ++j) x[r][j] = fmul2(fmul2(x[r][j], rr), w[j]);
      }
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      if (r == 1 && !two) break;
      angles.turn(m, x[r]);
      store_pairs<TO, V>(y_out, m, x[r]);
      y_out += s.y_h;
    }
    if ((cur.k += 2) >= nh) {
      cur.at(p, cur.tok + step, step);
      y_out = row_y(cur);
      if (p.rot && cur.tok < n_tok) angles.take(p, m, cur.pos, 1.f);
    }
  }
}

// Backward: persistent blocks; a thread walks with its item, so its 2V sums of
// dw stay in registers, and joins the block's in shared memory at the end; the
// rows ahead of the one at work are on their way to shared memory (straight to
// registers, one row at a time: 191 us for the call above).  Each block leaves
// its sums in the workspace, and sum_dw_kernel adds those in a fixed order: no
// atomics, the same bits every time.
//
// Runs of 4 dims: with runs of 8 f32 a warp's 16-byte copies of dy touch every
// second half of a sector.  Two rows at a time: one alone leaves the chain of
// its sums and shuffles with nothing beside it.
constexpr int kBackV = 4;

template <typename TX, typename TG, typename TO, bool INTER>
__global__ void __launch_bounds__(kThreads, kResident) norm_bwd_kernel(const __grid_constant__ NormParams p) {
  constexpr int V = kBackV;
  using SX = Slot<TX, V>;
  using SG = Slot<TG, V>;
  constexpr int kRow = 2 * (SX::kBytes + SG::kBytes) * kThreads;  // a row's slots of all threads
  const int si = blockIdx.y >= p.groups[0] ? 1 : 0;
  const NormSet& s = p.set[si];
  const int h0 = ((int)blockIdx.y - (si ? p.groups[0] : 0)) * p.hg, nh = min(p.hg, s.heads - h0);
  const int items = p.d / (2 * V);
  const int per_block = kThreads / items;
  const Item m = item_of<V>(threadIdx.x & (items - 1), p.rot, p.d);
  const unsigned lanes = lanes_of_row(items);
  const int64_t n_tok = (int64_t)p.B * p.T, step = (int64_t)gridDim.x * per_block;
  Walk cur, next;
  next.at(p, (int64_t)blockIdx.x * per_block + threadIdx.x / items, step);
  cur = next;
  auto row_x = [&](const Walk& a) { return static_cast<const TX*>(s.x) + (a.b * s.x_b + a.t * s.x_t + h0 * s.x_h); };
  auto row_g = [&](const Walk& a) { return static_cast<const TG*>(s.g) + (a.b * s.g_b + a.t * s.g_t + h0 * s.g_h); };
  auto row_y = [&](const Walk& a) { return static_cast<TO*>(s.y) + (a.b * s.y_b + a.t * s.y_t + h0 * s.y_h); };
  const TX* x_in = row_x(next);
  const TG* g_in = row_g(next);
  TO* y_out = row_y(cur);
  extern __shared__ __align__(16) unsigned char slots[];
  int put = 0, get = 0;
  auto issue = [&]() {
    if (next.tok < n_tok) {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        if (next.k + r < nh) {
          unsigned char* at = slots + (2 * put + r) * kRow;
          SX::copy(at, x_in + m.a0);
          SX::copy(at + SX::kBytes * kThreads, x_in + m.a1);
          at += 2 * SX::kBytes * kThreads;
          SG::copy(at, g_in + m.a0);
          SG::copy(at + SG::kBytes * kThreads, g_in + m.a1);
          x_in += s.x_h;
          g_in += s.g_h;
        }
      }
      if ((next.k += 2) >= nh) {
        next.at(p, next.tok + step, step);
        x_in = row_x(next);
        g_in = row_g(next);
      }
    }
    put = (put + 1) & (kRing - 1);
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  uint64_t w[V], dw[V];
  weights_of<V>(p, s, m, w);
#pragma unroll
  for (int j = 0; j < V; ++j) dw[j] = 0;
  Angles<V, INTER> angles;
  if (p.rot && cur.tok < n_tok) angles.take(p, m, cur.pos, -1.f);
#pragma unroll
  for (int i = 0; i < kRing - 1; ++i) issue();
  while (cur.tok < n_tok) {  // (whole rows leave)
    issue();
    asm volatile("cp.async.wait_group %0;" ::"n"(kRing - 1) : "memory");
    const bool two = cur.k + 1 < nh;
    uint64_t x[2][V], g[2][V];
    float ss[2], ch[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const unsigned char* at = slots + (2 * get + r) * kRow;
      SX::pairs(at, x[r]);
      SX::pairs(at + SX::kBytes * kThreads, x[r] + V / 2);
      at += 2 * SX::kBytes * kThreads;
      SG::pairs(at, g[r]);
      SG::pairs(at + SG::kBytes * kThreads, g[r] + V / 2);
      if (r == 1 && !two) {  // (what an absent row's slots hold is not used)
#pragma unroll
        for (int j = 0; j < V; ++j) x[r][j] = g[r][j] = 0;
      }
      angles.turn(m, g[r]);
      uint64_t ss2 = 0, ch2 = 0;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        ss2 = ffma2(x[r][j], x[r][j], ss2);
        ch2 = ffma2(fmul2(g[r][j], w[j]), x[r][j], ch2);
      }
      ss[r] = sum2(ss2);
      ch[r] = sum2(ch2);
    }
    get = (get + 1) & (kRing - 1);
    for (int off = items >> 1; off >= 1; off >>= 1) {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        ss[r] += __shfl_xor_sync(lanes, ss[r], off);
        ch[r] += __shfl_xor_sync(lanes, ch[r], off);
      }
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      if (r == 1 && !two) break;
      const float rs = rsqrtf(fmaf(ss[r], p.inv_d, p.eps));
      const float mean = -ch[r] * rs * p.inv_d;  // of c h, negative
      const uint64_t rr = f2(rs, rs), mm = f2(mean, mean);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const uint64_t h = fmul2(x[r][j], rr);
        dw[j] = ffma2(g[r][j], h, dw[j]);
        x[r][j] = fmul2(rr, ffma2(h, mm, fmul2(g[r][j], w[j])));
      }
      store_pairs<TO, V>(y_out, m, x[r]);
      y_out += s.y_h;
    }
    if ((cur.k += 2) >= nh) {
      cur.at(p, cur.tok + step, step);
      y_out = row_y(cur);
      if (p.rot && cur.tok < n_tok) angles.take(p, m, cur.pos, -1.f);
    }
  }
  // the sums of the threads with the same item: a column each (over the slots: all copies have landed)
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  __syncthreads();
  float* red = reinterpret_cast<float*>(slots);  // [kThreads][2 V + 1]
#pragma unroll
  for (int j = 0; j < V; ++j)
    f2_split(dw[j], red[threadIdx.x * (2 * V + 1) + 2 * j], red[threadIdx.x * (2 * V + 1) + 2 * j + 1]);
  __syncthreads();
  float* out = p.ws + ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * p.d;
  for (int c = threadIdx.x; c < p.d; c += kThreads) {
    const int it = c / (2 * V), j = c % (2 * V);
    float sum = 0.f;
    for (int i = it; i < kThreads; i += items) sum += red[i * (2 * V + 1) + j];
    const Item q = item_of<V>(it, p.rot, p.d);
    out[j < V ? q.a0 + j : q.a1 + j - V] = sum;
  }
}

// Rows of any d, strides and rot: a warp a row, the row in shared memory.
constexpr int kWarps = kThreads / 32;

// Row u of both sets in order (set, b, head, t); false past the last.
__device__ __forceinline__ bool row_of(const NormParams& p, int64_t u, int& si, int& b, int& h, int& t) {
  si = 0;
  const int64_t n0 = (int64_t)p.B * p.set[0].heads * p.T;
  if (u >= n0) {
    u -= n0;
    si = 1;
    if (p.n_sets < 2) return false;
  }
  const int heads = p.set[si].heads;
  if (u >= (int64_t)p.B * heads * p.T) return false;
  t = (int)(u % p.T);
  const int64_t bh = u / p.T;
  h = (int)(bh % heads);
  b = (int)(bh / heads);
  return true;
}
__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
  return x;
}
// Dim j of R row (or, back, of R^T row), the row in shared memory.
template <bool INTER>
__device__ __forceinline__ float turned_at(const NormParams& p, const float* row, int j, int pos, bool back) {
  if (j >= p.rot) return row[j];
  const int half = p.rot / 2;
  const int pair = INTER ? j >> 1 : (j < half ? j : j - half);
  const bool second = INTER ? (j & 1) : j >= half;
  const float u = row[INTER ? 2 * pair : pair], v = row[INTER ? 2 * pair + 1 : pair + half];
  float sn, cs;
  turn_of(pos, p.phases[pair * p.ph_s], sn, cs);
  sn *= back ? -p.mscale : p.mscale;
  cs *= p.mscale;
  return second ? u * sn + v * cs : u * cs - v * sn;
}

template <typename TI, typename TO, bool INTER>
__global__ void __launch_bounds__(kThreads) norm_rows_kernel(const __grid_constant__ NormParams p) {
  extern __shared__ float rows[];
  float* row = rows + (threadIdx.x >> 5) * p.d;
  const int lane = threadIdx.x & 31;
  int si, b, h, t;
  if (!row_of(p, (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5), si, b, h, t)) return;
  if (p.skip_negative && p.pos[b * p.p_b + t * p.p_t] < 0) return;
  const NormSet& s = p.set[si];
  const TI* x = static_cast<const TI*>(s.x) + (b * s.x_b + h * s.x_h + t * s.x_t);
  float ss = 0.f;
  for (int j = lane; j < p.d; j += 32) {
    const float v = to_f32(x[j * s.x_d]);
    ss = fmaf(v, v, ss);
    row[j] = v;
  }
  if (s.w != nullptr) {
    const float r = rsqrtf(fmaf(warp_sum(ss), p.inv_d, p.eps));
    for (int j = lane; j < p.d; j += 32) row[j] = row[j] * r * weight_at(s, p.w_f32, j);
  }
  __syncwarp();
  TO* y = static_cast<TO*>(s.y) + (b * s.y_b + h * s.y_h + t * s.y_t);
  const int pos = p.rot ? p.pos[b * p.p_b + t * p.p_t] : 0;
  for (int j = lane; j < p.d; j += 32) y[j * s.y_d] = from_f32<TO>(turned_at<INTER>(p, row, j, pos, false));
}

// blockIdx.y: the set; a block walks every gridDim.x-th group of kWarps rows of
// it.  Shared memory: a row of g and one of dw a warp.
template <typename TX, typename TG, typename TO, bool INTER>
__global__ void __launch_bounds__(kThreads) norm_bwd_rows_kernel(const __grid_constant__ NormParams p) {
  extern __shared__ float rows[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float* gr = rows + warp * p.d;
  float* dw = rows + (kWarps + warp) * p.d;
  const int si = blockIdx.y;
  const NormSet& s = p.set[si];
  for (int j = lane; j < p.d; j += 32) dw[j] = 0.f;
  const int64_t n = (int64_t)p.B * s.heads * p.T;
  for (int64_t u = (int64_t)blockIdx.x * kWarps + warp; u < n; u += (int64_t)gridDim.x * kWarps) {
    const int t = (int)(u % p.T);
    const int64_t bh = u / p.T;
    const int h = (int)(bh % s.heads), b = (int)(bh / s.heads);
    const TX* x = static_cast<const TX*>(s.x) + (b * s.x_b + h * s.x_h + t * s.x_t);
    const TG* g = static_cast<const TG*>(s.g) + (b * s.g_b + h * s.g_h + t * s.g_t);
    __syncwarp();
    for (int j = lane; j < p.d; j += 32) gr[j] = to_f32(g[j * s.g_d]);
    __syncwarp();
    const int pos = p.rot ? p.pos[b * p.p_b + t * p.p_t] : 0;
    float ss = 0.f, ch = 0.f;
    for (int j = lane; j < p.d; j += 32) {
      const float v = to_f32(x[j * s.x_d]);
      ss = fmaf(v, v, ss);
      ch = fmaf(turned_at<INTER>(p, gr, j, pos, true) * weight_at(s, p.w_f32, j), v, ch);
    }
    ss = warp_sum(ss);
    ch = warp_sum(ch);
    const float r = rsqrtf(fmaf(ss, p.inv_d, p.eps)), mean = ch * r * p.inv_d;
    TO* y = static_cast<TO*>(s.y) + (b * s.y_b + h * s.y_h + t * s.y_t);
    for (int j = lane; j < p.d; j += 32) {
      const float gj = turned_at<INTER>(p, gr, j, pos, true), hj = to_f32(x[j * s.x_d]) * r;
      dw[j] = fmaf(gj, hj, dw[j]);
      y[j * s.y_d] = from_f32<TO>(r * (gj * weight_at(s, p.w_f32, j) - hj * mean));
    }
  }
  __syncthreads();
  float* out = p.ws + ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * p.d;
  for (int c = threadIdx.x; c < p.d; c += kThreads) {
    float sum = 0.f;
    for (int k = 0; k < kWarps; ++k) sum += rows[(kWarps + k) * p.d + c];
    out[c] = sum;
  }
}

// dw: the blocks' sums of each set, 32 dims a block, eight strided sums a dim
// and then those, in order.
__global__ void __launch_bounds__(kThreads) sum_dw_kernel(const __grid_constant__ NormParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");  // (the blocks' sums)
  const NormSet& s = p.set[blockIdx.y];
  const int lane = threadIdx.x & 31, part = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  const int n = p.groups[blockIdx.y] * p.blocks;
  const float* in = p.ws + (int64_t)(blockIdx.y ? p.groups[0] : 0) * p.blocks * p.d;
  float sum = 0.f;
  if (c < p.d)
    for (int i = part; i < n; i += kWarps) sum += in[(int64_t)i * p.d + c];
  __shared__ float red[kWarps][32];
  red[part][lane] = sum;
  __syncthreads();
  if (part == 0 && c < p.d) {
#pragma unroll
    for (int k = 1; k < kWarps; ++k) sum += red[k][lane];
    s.dw[c * s.dw_s] = sum;
  }
}

// ------------------------------------------------------------- launches
bool run_fits(const void* base, int bytes, int V, bool used_b, int64_t sb, bool used_h, int64_t sh, bool used_t,
              int64_t st, int64_t sd) {
  const int access = V * bytes;
  return sd == 1 && reinterpret_cast<uintptr_t>(base) % 16 == 0 && (!used_b || sb * bytes % access == 0) &&
         (!used_h || sh * bytes % access == 0) && (!used_t || st * bytes % access == 0);
}
// Whether the fast kernels take these rows (a stride of a dim of size 1 is not used).
bool fast_ok(const NormParams& p, int in_bytes, int out_bytes, int g_bytes) {
  const int V = g_bytes ? kBackV : 16 / in_bytes, items = p.d / (2 * V);
  if (p.d % (2 * V) != 0 || p.rot % (2 * V) != 0 || items > 32 || (items & (items - 1)) != 0) return false;
  for (int i = 0; i < p.n_sets; ++i) {
    const NormSet& s = p.set[i];
    const bool ub = p.B > 1, uh = s.heads > 1, ut = p.T > 1;
    if (!run_fits(s.x, in_bytes, V, ub, s.x_b, uh, s.x_h, ut, s.x_t, s.x_d) ||
        !run_fits(s.y, out_bytes, V, ub, s.y_b, uh, s.y_h, ut, s.y_t, s.y_d) ||
        (g_bytes && !run_fits(s.g, g_bytes, V, ub, s.g_b, uh, s.g_h, ut, s.g_t, s.g_d)))
      return false;
    // (stores of 8 floats are one access of 32 bytes)
    if (V * out_bytes == 32 && reinterpret_cast<uintptr_t>(s.y) % 32 != 0) return false;
  }
  return true;
}

int set_groups(NormParams* p, int hg) {
  p->hg = hg < 1 ? 1 : (hg > kMostHeads ? kMostHeads : hg);
  int n = 0;
  for (int i = 0; i < p->n_sets; ++i) n += p->groups[i] = (p->set[i].heads + p->hg - 1) / p->hg;
  return n;
}
int most_heads(const NormParams& p) {
  return p.n_sets > 1 && p.set[1].heads > p.set[0].heads ? p.set[1].heads : p.set[0].heads;
}

template <typename TI, typename TO, bool INTER>
cudaError_t launch_forward(NormParams p, cudaStream_t stream) {
  constexpr int V = 16 / sizeof(TI);
  if (fast_ok(p, sizeof(TI), sizeof(TO), 0)) {
    const int per_block = kThreads / (p.d / (2 * V));
    int64_t blocks = ((int64_t)p.B * p.T + per_block - 1) / per_block;
    int dev = 0, sms = 0;
    if (cudaError_t e = cudaGetDevice(&dev); e != cudaSuccess) return e;
    if (cudaError_t e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev); e != cudaSuccess) return e;
    const int fill = kResident * sms;  // blocks resident at once
    // heads of a group: as many as leave enough groups to fill the machine (at most
    // 2 x 32767 groups: in a grid's range)
    const int64_t want = (fill + blocks - 1) / blocks;
    const int groups = set_groups(&p, (int)((most_heads(p) + want - 1) / want));
    // one wave of blocks and no block more
    const int64_t most = groups < fill ? fill / groups : 1;
    if (blocks > most) blocks = most;
    constexpr int smem = 2 * kRing * 2 * V * (int)sizeof(TI) * kThreads;
    static DeviceOnce once;
    if (cudaError_t e = once.set_smem(reinterpret_cast<const void*>(&norm_kernel<TI, TO, V, INTER>), smem);
        e != cudaSuccess)
      return e;
    norm_kernel<TI, TO, V, INTER><<<dim3((unsigned)blocks, (unsigned)groups), kThreads, smem, stream>>>(p);
    return cudaGetLastError();
  }
  const int64_t rows = (int64_t)p.B * p.T * (p.set[0].heads + (p.n_sets > 1 ? p.set[1].heads : 0));
  const int64_t blocks = (rows + kWarps - 1) / kWarps;  // (kMostRows: in a grid's range)
  norm_rows_kernel<TI, TO, INTER><<<(unsigned)blocks, kThreads, kWarps * p.d * sizeof(float), stream>>>(p);
  return cudaGetLastError();
}

// The grid of the backward kernel, the same for every type: set_groups and
// `blocks` in *p.  Blocks along the tokens so that the machine is full once
// (two resident blocks an SM; every block costs a row of partial sums).
bool plan_backward(NormParams* p, int in_bytes, int out_bytes, int g_bytes, int sms) {
  const bool fast = fast_ok(*p, in_bytes, out_bytes, g_bytes);
  int groups = p->n_sets;
  int64_t most;
  if (fast) {
    const int per_block = kThreads / (p->d / (2 * kBackV));
    groups = set_groups(p, kMostHeads);
    most = ((int64_t)p->B * p->T + per_block - 1) / per_block;
  } else {
    p->groups[0] = p->groups[1] = 1;
    most = ((int64_t)p->B * p->T * most_heads(*p) + kWarps - 1) / kWarps;
  }
  // (one wave and no block more: one more than fits took 200 us in place of 151)
  int64_t blocks = kResident * sms / (groups < 1 ? 1 : groups);
  if (blocks > most) blocks = most;
  p->blocks = (int)(blocks < 1 ? 1 : blocks);
  return fast;
}

template <typename TX, typename TG, typename TO, bool INTER>
cudaError_t launch_backward_t(const NormParams& p, bool fast, cudaStream_t stream) {
  constexpr int V = kBackV;
  const int groups = p.groups[0] + (p.n_sets > 1 ? p.groups[1] : 0);
  const dim3 grid((unsigned)p.blocks, (unsigned)groups);
  if (groups == 0) {  // no heads at all: dw is zeros
  } else if (fast) {
    constexpr int ring = 2 * kRing * 2 * V * (int)(sizeof(TX) + sizeof(TG)) * kThreads, red = kThreads * (2 * V + 1) * 4;
    constexpr int smem = ring > red ? ring : red;
    static DeviceOnce once;
    if (cudaError_t e = once.set_smem(reinterpret_cast<const void*>(&norm_bwd_kernel<TX, TG, TO, INTER>), smem);
        e != cudaSuccess)
      return e;
    norm_bwd_kernel<TX, TG, TO, INTER><<<grid, kThreads, smem, stream>>>(p);
  } else {
    const int smem = 2 * kWarps * p.d * (int)sizeof(float);
    if (smem > 48 * 1024) {
      static DeviceOnce once;
      if (cudaError_t e = once.set_smem(reinterpret_cast<const void*>(&norm_bwd_rows_kernel<TX, TG, TO, INTER>),
                                        2 * kWarps * (int)kMaxDim * (int)sizeof(float));
          e != cudaSuccess)
        return e;
    }
    norm_bwd_rows_kernel<TX, TG, TO, INTER><<<grid, kThreads, smem, stream>>>(p);
  }
  if (cudaError_t e = cudaGetLastError(); e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((p.d + 31) / 32), (unsigned)p.n_sets);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr;  // scheduled while the backward kernel drains
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, sum_dw_kernel, p);
}
template <typename TX, typename TG, typename TO>
cudaError_t launch_backward_l(const NormParams& p, bool fast, bool inter, cudaStream_t stream) {
  return inter ? launch_backward_t<TX, TG, TO, true>(p, fast, stream)
               : launch_backward_t<TX, TG, TO, false>(p, fast, stream);
}
template <typename TX>
cudaError_t launch_backward_x(const NormParams& p, bool fast, int32_t g, int32_t out, bool inter, cudaStream_t stream) {
  if (g == BLKATTN_F32)
    return out == BLKATTN_F32 ? launch_backward_l<TX, float, float>(p, fast, inter, stream)
                              : launch_backward_l<TX, float, __nv_bfloat16>(p, fast, inter, stream);
  return out == BLKATTN_F32 ? launch_backward_l<TX, __nv_bfloat16, float>(p, fast, inter, stream)
                            : launch_backward_l<TX, __nv_bfloat16, __nv_bfloat16>(p, fast, inter, stream);
}

template <typename TI, typename TO>
cudaError_t launch_forward_l(const NormParams& p, bool inter, cudaStream_t stream) {
  return inter ? launch_forward<TI, TO, true>(p, stream) : launch_forward<TI, TO, false>(p, stream);
}

// ------------------------------------------------------------- arguments
int bytes_of(int32_t t) { return t == BLKATTN_BF16 ? 2 : 4; }

// x, y (and g) of one shape; y writable.
int check_set(const blkattn_tensor* x, const blkattn_tensor* w, const blkattn_tensor* y, const blkattn_tensor* g,
              const blkattn_tensor* dw) {
  if (!tensor_dims_ok(x, 4) || !tensor_dims_ok(w, 1) || !tensor_dims_ok(y, 4)) return BLKATTN_ERR_INVALID_ARG;
  if (!floats(x) || !floats(w) || !floats(y) || w->sizes[0] != x->sizes[3]) return BLKATTN_ERR_INVALID_ARG;
  for (int i = 0; i < 4; ++i)
    if (x->sizes[i] != y->sizes[i]) return BLKATTN_ERR_INVALID_ARG;
  if (!writable(y) || !in_place_ok(g ? g : x, y)) return BLKATTN_ERR_INVALID_ARG;
  if (!g) return BLKATTN_OK;
  if (!tensor_dims_ok(g, 4) || !floats(g) || !tensor_dims_ok(dw, 1) || dw->dtype != BLKATTN_F32 ||
      dw->sizes[0] != x->sizes[3] || !writable(dw))
    return BLKATTN_ERR_INVALID_ARG;
  for (int i = 0; i < 4; ++i)
    if (g->sizes[i] != x->sizes[i]) return BLKATTN_ERR_INVALID_ARG;
  return BLKATTN_OK;
}

struct Call {
  const blkattn_tensor *x[2], *w[2], *y[2], *g[2], *dw[2];
  const blkattn_tensor *pos, *ph;
  int32_t layout;
  float mscale, eps;
};

void fill_set(NormSet* s, const Call& c, int i) {
  auto four = [](const blkattn_tensor* t, int64_t& b, int64_t& h, int64_t& n, int64_t& d) {
    b = t->strides[0]; h = t->strides[1]; n = t->strides[2]; d = t->strides[3];
  };
  s->x = c.x[i]->data;
  four(c.x[i], s->x_b, s->x_h, s->x_t, s->x_d);
  if (c.w[i]) {
    s->w = c.w[i]->data;
    s->w_s = c.w[i]->strides[0];
  }
  s->y = c.y[i]->data;
  four(c.y[i], s->y_b, s->y_h, s->y_t, s->y_d);
  s->heads = (int)c.x[i]->sizes[1];
  if (!c.g[i]) return;
  s->g = c.g[i]->data;
  four(c.g[i], s->g_b, s->g_h, s->g_t, s->g_d);
  s->dw = static_cast<float*>(c.dw[i]->data);
  s->dw_s = c.dw[i]->strides[0];
}

NormParams fill_params(const Call& c, int n_sets) {
  NormParams p{};
  p.n_sets = n_sets;
  for (int i = 0; i < n_sets; ++i) fill_set(&p.set[i], c, i);
  p.p_b = c.pos->strides[0]; p.p_t = c.pos->strides[1];
  if (c.ph) {
    p.pos = static_cast<const int32_t*>(c.pos->data);
    p.phases = static_cast<const int64_t*>(c.ph->data);
    p.ph_s = c.ph->strides[0];
    p.rot = (int)(2 * c.ph->sizes[0]);
  }
  p.w_f32 = c.w[0] && c.w[0]->dtype == BLKATTN_F32;
  p.mscale = c.mscale;
  p.eps = c.eps;
  p.B = (int)c.x[0]->sizes[0]; p.T = (int)c.x[0]->sizes[2]; p.d = (int)c.x[0]->sizes[3];
  p.inv_d = 1.f / (float)p.d;
  return p;
}

cudaError_t launch_forward_types(const NormParams& p, int32_t in, int32_t out, bool inter, cudaStream_t stream) {
  if (in == BLKATTN_BF16)
    return out == BLKATTN_BF16 ? launch_forward_l<__nv_bfloat16, __nv_bfloat16>(p, inter, stream)
                               : launch_forward_l<__nv_bfloat16, float>(p, inter, stream);
  return out == BLKATTN_BF16 ? launch_forward_l<float, __nv_bfloat16>(p, inter, stream)
                             : launch_forward_l<float, float>(p, inter, stream);
}

int norm(const Call& c, bool back, blkattn_stream_t stream_) {
  // the second set: all of it or none
  const bool two = c.x[1] != nullptr;
  if (two != (c.w[1] != nullptr) || two != (c.y[1] != nullptr) ||
      (back && (two != (c.g[1] != nullptr) || two != (c.dw[1] != nullptr))))
    return BLKATTN_ERR_INVALID_ARG;
  if (back && c.g[0] == nullptr) return BLKATTN_ERR_INVALID_ARG;
  const int n_sets = two ? 2 : 1;
  for (int i = 0; i < n_sets; ++i)
    if (int st = check_set(c.x[i], c.w[i], c.y[i], c.g[i], c.dw[i]); st != BLKATTN_OK) return st;
  const int64_t B = c.x[0]->sizes[0], T = c.x[0]->sizes[2], d = c.x[0]->sizes[3];
  if (!tensor_dims_ok(c.pos, 2) || c.pos->dtype != BLKATTN_I32 || c.pos->sizes[0] != B || c.pos->sizes[1] != T || d < 1)
    return BLKATTN_ERR_INVALID_ARG;
  if (two) {
    // one type and one shape but for the heads
    for (int i : {0, 2, 3})
      if (c.x[1]->sizes[i] != c.x[0]->sizes[i]) return BLKATTN_ERR_INVALID_ARG;
    if (c.x[1]->dtype != c.x[0]->dtype || c.w[1]->dtype != c.w[0]->dtype || c.y[1]->dtype != c.y[0]->dtype ||
        (back && c.g[1]->dtype != c.g[0]->dtype))
      return BLKATTN_ERR_INVALID_ARG;
    if (c.y[0]->data == c.y[1]->data && c.y[0]->data != nullptr) return BLKATTN_ERR_INVALID_ARG;
    if (back && c.dw[0]->data == c.dw[1]->data && c.dw[0]->data != nullptr) return BLKATTN_ERR_INVALID_ARG;
  }
  if (c.ph) {
    if (int st = check_phases(c.ph, c.layout, d); st != BLKATTN_OK) return st;
    if (!finite(c.mscale)) return BLKATTN_ERR_INVALID_ARG;
  }
  if (!finite(c.eps) || c.eps < 0.f) return BLKATTN_ERR_INVALID_ARG;
  if (!tensors_on_one_device(c.x[0], {c.x[1], c.w[0], c.w[1], c.y[0], c.y[1], c.g[0], c.g[1], c.dw[0], c.dw[1], c.pos, c.ph}))
    return BLKATTN_ERR_INVALID_ARG;
  int64_t heads = 0;
  for (int i = 0; i < n_sets; ++i) {
    if (c.x[i]->sizes[1] > 0x7fff) return BLKATTN_ERR_UNSUPPORTED;
    heads += c.x[i]->sizes[1];
  }
  if (d > kMaxDim || B > 0x7fffffff || T > 0x7fffffff || (B > 0 && T > 0x7fffffff / B) || B * T * heads > kMostRows)
    return BLKATTN_ERR_UNSUPPORTED;
  const bool rows = B > 0 && T > 0 && heads > 0;
  if (!rows && !back) return BLKATTN_OK;
  for (int i = 0; i < n_sets; ++i) {
    if (c.w[i]->data == nullptr || (back && c.dw[i]->data == nullptr)) return BLKATTN_ERR_INVALID_ARG;
    if (B > 0 && T > 0 && c.x[i]->sizes[1] > 0 &&
        (c.x[i]->data == nullptr || c.y[i]->data == nullptr || (back && c.g[i]->data == nullptr)))
      return BLKATTN_ERR_INVALID_ARG;
  }
  if (rows && ((c.pos->data == nullptr && c.ph) || (c.ph && c.ph->data == nullptr))) return BLKATTN_ERR_INVALID_ARG;
  if (int st = require_current_device(c.x[0]->device); st != BLKATTN_OK) return st;
  NormParams p = fill_params(c, n_sets);
  const bool inter = c.ph && c.layout == BLKATTN_ROPE_INTERLEAVED;
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  const int32_t ti = c.x[0]->dtype, to = c.y[0]->dtype;
  if (!back) {
    // (a set without heads takes no place)
    if (p.set[0].heads == 0) p.set[0] = p.set[1];
    if (p.n_sets == 2 && (p.set[1].heads == 0 || c.x[0]->sizes[1] == 0)) p.n_sets = 1;
    const cudaError_t e = launch_forward_types(p, ti, to, inter, stream);
    return e == cudaSuccess ? BLKATTN_OK : report_cuda_failure(e);
  }
  const int32_t tg = c.g[0]->dtype;
  const Library lib;
  int sms = 0;
  if (int st = lib.sms(&sms); st != BLKATTN_OK) return st;
  const bool fast = plan_backward(&p, bytes_of(ti), bytes_of(to), bytes_of(tg), sms);
  void* ws = nullptr;
  const int64_t groups = p.groups[0] + (p.n_sets > 1 ? p.groups[1] : 0);
  if (int st = lib.workspace((size_t)(groups * p.blocks * d) * sizeof(float), stream, &ws); st != BLKATTN_OK) return st;
  p.ws = static_cast<float*>(ws);
  const cudaError_t e = ti == BLKATTN_BF16 ? launch_backward_x<__nv_bfloat16>(p, fast, tg, to, inter, stream)
                                           : launch_backward_x<float>(p, fast, tg, to, inter, stream);
  return e == cudaSuccess ? BLKATTN_OK : report_cuda_failure(e);
}

}  // namespace

cudaError_t launch_query_rows(const blkattn_tensor* q, const blkattn_tensor* q_weight, const blkattn_tensor* pos,
                              const blkattn_tensor* phases, int32_t layout, float mscale, float eps,
                              const blkattn_tensor* q_out, cudaStream_t stream) {
  const Call c{{q, nullptr}, {q_weight, nullptr}, {q_out, nullptr}, {}, {}, pos, phases, layout, mscale, eps};
  NormParams p = fill_params(c, 1);
  p.skip_negative = true;
  p.pos = static_cast<const int32_t*>(pos->data);
  return launch_forward_types(p, q->dtype, q_out->dtype, phases && layout == BLKATTN_ROPE_INTERLEAVED, stream);
}

}  // namespace blkattn

extern "C" {

int blkattn_qk_norm_rope(const blkattn_tensor* q, const blkattn_tensor* q_weight, const blkattn_tensor* k,
                         const blkattn_tensor* k_weight, const blkattn_tensor* pos, const blkattn_tensor* phases,
                         int32_t layout, float mscale, float eps, const blkattn_tensor* q_out,
                         const blkattn_tensor* k_out, blkattn_stream_t stream) {
  const blkattn::Call c{{q, k}, {q_weight, k_weight}, {q_out, k_out}, {}, {}, pos, phases, layout, mscale, eps};
  return blkattn::norm(c, false, stream);
}

int blkattn_qk_norm_rope_bwd(const blkattn_tensor* dq_out, const blkattn_tensor* dk_out, const blkattn_tensor* q,
                             const blkattn_tensor* q_weight, const blkattn_tensor* k, const blkattn_tensor* k_weight,
                             const blkattn_tensor* pos, const blkattn_tensor* phases, int32_t layout, float mscale,
                             float eps, const blkattn_tensor* dq, const blkattn_tensor* dk,
                             const blkattn_tensor* dq_weight, const blkattn_tensor* dk_weight,
                             blkattn_stream_t stream) {
  const blkattn::Call c{{q, k},     {q_weight, k_weight},   {dq, dk}, {dq_out, dk_out}, {dq_weight, dk_weight},
                        pos,        phases,                 layout,   mscale,           eps};
  return blkattn::norm(c, true, stream);
}

}  // extern "C"
