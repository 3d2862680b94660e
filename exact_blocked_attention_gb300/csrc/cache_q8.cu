// The 8-bit paged cache written and read back (q8.cuh has its numbers).
//
// Append.  K rows are normed (with a weight), turned (with phases) and
// quantised, V rows quantised; q rows normed and turned on the way.  A block of
// S cache rows of one head shares a scale, so its rows are one unit of work:
//
//     e_new = e(max |x| over the new rows)                      if row 0 is new
//           = max(that, e_old), rows that stay rounded again    otherwise
//
// A call that writes a block's row 0 begins the block anew, so what a page held
// for another sequence does not decide its scales.  Infinities and NaN have no
// 8-bit form: they are stored as NaN and do not take part in the maximum.
//
// A sequence's rows come in ascending positions, so the new rows of a block are
// one run of t (with padding between, perhaps).  A CTA takes a window of t and
// the blocks whose run begins in it, panels of max(S, 16) cache rows at a time:
// the panel's angles go to shared memory once, then a warp takes 2048 numbers of
// a head of K or V (16 dims a lane), in registers from the load to the store;
// where a panel has more, warps share it and its maxima through shared memory.
// (A warp for the whole panel, which computes its rows for the maximum and again
// for the store: 55 us for a prompt of 5120 rows and 8 KV heads in blocks of 32,
// 38 so.)
//
// Latency bounds a decode step's append: one launch, the query rows in CTAs of
// their own.  Memory bounds a prompt's, most of it the query rows': from
// kOwnKernelRows on they go to the norm kernel, which keeps more rows in flight.
#include <cuda_bf16.h>

#include <cstdint>

#include "kernels.h"
#include "paged.h"
#include "q8.cuh"
#include "rotary.cuh"

namespace blkattn {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kQHeads = 32;   // query heads of a CTA
constexpr int kScan = 8;      // positions of a lane in flight where padding is passed over (one: 17 us past 1500 rows)
// query rows from which on they have a kernel of their own
constexpr int64_t kOwnKernelRows = 16384;

struct Rows {
  const void* p;
  int64_t s_b, s_h, s_t, s_d;
};
struct Pool {
  unsigned char* p;
  int64_t s_n, s_h, s_r;  // page, head, row (bytes)
  unsigned char* scales;
  int64_t e_n, e_h, e_i;  // page, head, block
};
struct AppendParams {
  Rows src[2];   // k, v
  Pool pool[2];
  Rows q;
  void* q_out;
  int64_t o_b, o_h, o_t, o_d;
  const void* wq;
  const void* wk;
  int64_t wq_s, wk_s;
  bool w_f32;
  float eps, mscale;
  const int32_t* pos;
  int64_t p_b, p_t;
  const int64_t* phases;
  int64_t ph_s;
  int rot, B, T, Hkv, Hq;
  int shift;    // log2 S
  int panel;    // max(S, 16) rows
  int kv_groups;
  PageTable pages;
};

// The dims of a lane: two runs of 8 (rotary.cuh).  RUNS: rot is a multiple of
// 16 and the runs are those that the rotation pairs; otherwise the row goes
// through shared memory.
template <int D>
struct Lane {
  static constexpr int kLanes = D / 16;        // of a row
  static constexpr int kRows = 32 / kLanes;    // of a pass
  int it, slot, a0, a1;
  bool turn;
  unsigned lanes;
  __device__ Lane(int lane, int rot, bool runs) {
    it = lane % kLanes;
    slot = lane / kLanes;
    const int r = runs ? rot : 0;
    turn = it < r / 16;
    const int part0 = turn ? 0 : r, part = turn ? r : D - r;
    a0 = part0 + 8 * (it - part0 / 16);
    a1 = a0 + part / 2;
    lanes = ((1u << kLanes) - 1) << (lane & ~(kLanes - 1));
  }
};

template <typename T, bool VEC>
__device__ __forceinline__ void load8(const T* p, int64_t s_d, float* x) {
  if constexpr (VEC) {
    constexpr int N = 16 / sizeof(T);
#pragma unroll
    for (int c = 0; c < 8; c += N) {
      const uint4 w = __ldg(reinterpret_cast<const uint4*>(p + c));
      const T* e = reinterpret_cast<const T*>(&w);
#pragma unroll
      for (int j = 0; j < N; ++j) x[c + j] = to_f32(e[j]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = to_f32(p[j * s_d]);
  }
}

__device__ __forceinline__ float weight_of(const void* w, int64_t s, bool f32, int i) {
  return f32 ? static_cast<const float*>(w)[i * s] : __bfloat162float(static_cast<const __nv_bfloat16*>(w)[i * s]);
}

// One row of k or q: normed (w not NULL), then turned by the angles `cs` (its
// pairs' (cos, sin) mscale; not read when rot = 0).  stage: RUNS = false, D floats of the
// row's own.
template <typename T, int D, bool RUNS, bool INTER>
__device__ __forceinline__ void row_values(const AppendParams& p, const Lane<D>& l, const float* w, bool norm,
                                           bool rotate, const float2* cs, float* stage, float (&x)[16]) {
  if (norm) {
    uint64_t s2 = 0;  // (pairs: half the instructions)
#pragma unroll
    for (int j = 0; j < 16; j += 2) {
      const uint64_t v = f2(x[j], x[j + 1]);
      s2 = ffma2(v, v, s2);
    }
    float ss, odd;
    f2_split(s2, ss, odd);
    ss += odd;
#pragma unroll
    for (int off = Lane<D>::kLanes / 2; off >= 1; off >>= 1) ss += __shfl_xor_sync(l.lanes, ss, off);
    const float r = rsqrt_fine(fmaf(ss, 1.f / D, p.eps));
#pragma unroll
    for (int j = 0; j < 16; ++j) x[j] = x[j] * r * w[j];
  }
  if (!rotate) return;
  if constexpr (RUNS) {
    if (l.turn) {
      float sn[8], c[8], y[16];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int pair = !INTER ? 8 * l.it + j : (j < 4 ? l.a0 / 2 + j : l.a1 / 2 + j - 4);
        const float2 v = cs[pair];
        c[j] = v.x;
        sn[j] = v.y;
      }
      turn_pairs<8, INTER>(x, true, sn, c, y);
#pragma unroll
      for (int j = 0; j < 16; ++j) x[j] = y[j];
    }
  } else {
    __syncwarp(l.lanes);
#pragma unroll
    for (int j = 0; j < 16; ++j) stage[j < 8 ? l.a0 + j : l.a1 + j - 8] = x[j];
    __syncwarp(l.lanes);
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const int i = j < 8 ? l.a0 + j : l.a1 + j - 8;
      if (i < p.rot) {
        const int half = p.rot / 2;
        const int pair = INTER ? i >> 1 : (i < half ? i : i - half);
        const bool second = INTER ? (i & 1) : i >= half;
        const float u = stage[INTER ? 2 * pair : pair], v = stage[INTER ? 2 * pair + 1 : pair + half];
        const float2 a = cs[pair];
        x[j] = second ? u * a.y + v * a.x : u * a.x - v * a.y;
      }
    }
  }
}

// The angles of `n` rows: (cos, sin) mscale of every pair; pos_of(i) gives row
// i's position, or a negative one (left out).  A thread keeps its pair, whose
// phase it loads at the kernel's start (phase_of).
__device__ __forceinline__ int64_t phase_of(const AppendParams& p) {
  return p.rot > 0 ? p.phases[threadIdx.x % (p.rot / 2) * p.ph_s] : 0;
}
template <typename F>
__device__ __forceinline__ void fill_angles(const AppendParams& p, int64_t phase, float2* cs, int n, F&& pos_of) {
  const int pairs = p.rot / 2, step = kThreads / pairs;  // (at most 64 pairs)
  const int pair = threadIdx.x % pairs;
  int i = threadIdx.x / pairs;
  if (i >= step) return;
#pragma unroll 2
  for (; i < n; i += step) {
    const int t = pos_of(i);
    if (t < 0) continue;
    float sn, c;
    turn_of_fine(t, phase, sn, c);
    cs[i * pairs + pair] = make_float2(c * p.mscale, sn * p.mscale);
  }
}

template <int D, bool RUNS>
constexpr int kStage = RUNS ? 0 : kWarps * Lane<D>::kRows * D;  // floats

template <typename T, int D, bool RUNS, bool INTER, bool VEC>
__global__ void __launch_bounds__(kThreads, 2) append_q8_kernel(const __grid_constant__ AppendParams p) {
  extern __shared__ __align__(16) float smem[];
  float* stage_all = smem;
  float2* cs = reinterpret_cast<float2*>(smem + kStage<D, RUNS>);  // [panel rows][rot / 2]
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const Lane<D> l(lane, p.rot, RUNS);
  float* stage = stage_all + (warp * Lane<D>::kRows + l.slot) * D;
  const int windows = (p.T + p.panel - 1) / p.panel;
  const int b = blockIdx.x / windows, t0 = (blockIdx.x - b * windows) * p.panel;
  const int n = min(p.panel, p.T - t0);
  const int32_t* pos = p.pos + b * p.p_b;
  const int64_t phase = phase_of(p);

  if ((int)blockIdx.y >= p.kv_groups) {  // ---- query rows of the window
    const int h0 = ((int)blockIdx.y - p.kv_groups) * kQHeads, nh = min(kQHeads, p.Hq - h0);
    if (p.rot) fill_angles(p, phase, cs, n, [&](int i) { return pos[(t0 + i) * p.p_t]; });
    float w[16];
    const bool norm = p.wq != nullptr;
#pragma unroll
    for (int j = 0; j < 16; ++j)
      w[j] = norm ? weight_of(p.wq, p.wq_s, p.w_f32, j < 8 ? l.a0 + j : l.a1 + j - 8) : 1.f;
    __syncthreads();
    for (int u = warp * Lane<D>::kRows + l.slot; u < n * nh; u += kWarps * Lane<D>::kRows) {
      const int i = u / nh, h = h0 + u - i * nh, t = t0 + i;
      if (pos[t * p.p_t] < 0) continue;
      float x[16];
      const T* in = static_cast<const T*>(p.q.p) + (b * p.q.s_b + h * p.q.s_h + t * p.q.s_t);
      load8<T, VEC>(in + l.a0 * p.q.s_d, p.q.s_d, x);
      load8<T, VEC>(in + l.a1 * p.q.s_d, p.q.s_d, x + 8);
      row_values<T, D, RUNS, INTER>(p, l, w, norm, p.rot > 0, cs + i * (p.rot / 2), stage, x);
      T* o = static_cast<T*>(p.q_out) + (b * p.o_b + h * p.o_h + t * p.o_t);
      if constexpr (VEC) {
        Vec<T, 8> y0, y1;
        pack_runs<T, 8>(x, y0, y1);
        if constexpr (sizeof(T) == 2) {
          store(o + l.a0, y0);
          store(o + l.a1, y1);
        } else {  // (16-byte alignment)
          const float4* f0 = reinterpret_cast<const float4*>(&y0);
          const float4* f1 = reinterpret_cast<const float4*>(&y1);
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            reinterpret_cast<float4*>(o + l.a0)[c] = f0[c];
            reinterpret_cast<float4*>(o + l.a1)[c] = f1[c];
          }
        }
      } else {
#pragma unroll
        for (int j = 0; j < 16; ++j) o[(j < 8 ? l.a0 + j : l.a1 + j - 8) * p.o_d] = from_f32<T>(x[j]);
      }
    }
    return;
  }

  // ---- the blocks of cache rows whose run of new rows begins in the window
  __shared__ int lead[kMaxScaleRows];       // the runs' first t
  __shared__ int n_lead;
  __shared__ int src[kMaxScaleRows];        // t of the panel's rows, -1: not new
  __shared__ int page[16], first_row[16];   // of the panel's blocks: page (-1: none), row in page,
  __shared__ int first_pos[16];             // position of their first row
  __shared__ float amax[kWarps][kMaxScaleRows];  // of each pair's rows
  const int S = 1 << p.shift;
  // `parts` warps share a pair's rows, kPasses passes each
  constexpr int kPasses = 4;
  const int parts = max(1, p.panel / (kPasses * Lane<D>::kRows)), part = warp % parts;
  // pairs: K's heads, then V's (whose CTAs need no angles)
  const int pair = blockIdx.y * (kWarps / parts) + warp / parts, which = pair >= p.Hkv ? 1 : 0;
  const int h = pair - which * p.Hkv;
  const bool turns = p.rot > 0 && (int)blockIdx.y * (kWarps / parts) < p.Hkv;
  const int row0 = part * kPasses * Lane<D>::kRows;
  // the first rows, on their way while the runs are found
  if (part == 0 && h < p.Hkv && lane < 2 * n) {
    const Rows& rows = p.src[which];
    const T* r = static_cast<const T*>(rows.p) + (b * rows.s_b + h * rows.s_h + (t0 + (lane >> 1)) * rows.s_t +
                                                  (lane & 1) * (D / 2) * rows.s_d);
    asm volatile("prefetch.global.L1 [%0];" ::"l"(r));
  }
  if (warp == 0) {
    int found = 0;
    // (a window of padding has nothing to look for)
    bool any = false;
#pragma unroll 4
    for (int i = lane; i < n; i += 32) any |= pos[(t0 + i) * p.p_t] >= 0;
    any = __any_sync(0xffffffffu, any);
    // the last row before the window that is not padding
    int prev = -1;
    for (int u = t0; any && u > 0 && prev < 0; u -= 32 * kScan) {
      int v[kScan];
#pragma unroll
      for (int i = 0; i < kScan; ++i) {
        const int t = u - 32 * (i + 1) + lane;
        v[i] = t >= 0 ? pos[t * p.p_t] : -1;
      }
#pragma unroll
      for (int i = 0; i < kScan; ++i) {
        const unsigned m = __ballot_sync(0xffffffffu, v[i] >= 0);
        if (m && prev < 0) prev = __shfl_sync(0xffffffffu, v[i], 31 - __clz(m));
      }
    }
    for (int i0 = 0; any && i0 < n; i0 += 32) {
      const int c = i0 + lane < n ? pos[(t0 + i0 + lane) * p.p_t] : -1;
      const unsigned rows = __ballot_sync(0xffffffffu, c >= 0), below = rows & ((1u << lane) - 1);
      const int near = __shfl_sync(0xffffffffu, c, below ? 31 - __clz(below) : 0);
      const int from = below ? near : prev;
      const bool leads = c >= 0 && page_of(p.pages, b, c) >= 0 && (from < 0 || (from >> p.shift) != (c >> p.shift));
      const unsigned m = __ballot_sync(0xffffffffu, leads);
      if (leads) lead[found + __popc(m & ((1u << lane) - 1))] = t0 + i0 + lane;
      if (rows) prev = __shfl_sync(0xffffffffu, c, 31 - __clz(rows));
      found += __popc(m);
    }
    if (lane == 0) n_lead = found;
  }
  float w[16];
#pragma unroll
  for (int j = 0; j < 16; ++j)
    w[j] = p.wk ? weight_of(p.wk, p.wk_s, p.w_f32, j < 8 ? l.a0 + j : l.a1 + j - 8) : 1.f;
  const int per_panel = p.panel >> p.shift;
  __syncthreads();
  const int runs = n_lead;
  for (int r0 = 0; r0 < runs; r0 += per_panel) {
    for (int k = warp; k < per_panel; k += kWarps) {  // the runs' rows, a warp a run
      int pg = -1, row = 0, first = 0;
      for (int i = lane; i < S; i += 32) src[k * S + i] = -1;
      __syncwarp();
      if (r0 + k < runs) {
        const int t = lead[r0 + k], c = pos[t * p.p_t];
        pg = page_of(p.pages, b, c);
        row = (c & (p.pages.rows - 1)) & ~(S - 1);
        first = c & ~(S - 1);
        bool more = true;
        for (int u = t; more && u < p.T; u += 32 * kScan) {
          int v[kScan];
#pragma unroll
          for (int i = 0; i < kScan; ++i) v[i] = u + 32 * i + lane < p.T ? pos[(u + 32 * i + lane) * p.p_t] : -1;
#pragma unroll
          for (int i = 0; i < kScan; ++i) {
            const unsigned other = __ballot_sync(0xffffffffu, v[i] >= 0 && (v[i] >> p.shift) != (c >> p.shift));
            const int end = other ? __ffs(other) - 1 : 32;
            if (more && lane < end && v[i] >= 0)
              atomicMax(&src[k * S + (v[i] & (S - 1))], u + 32 * i + lane);  // (the later row stays)
            more = more && other == 0;
          }
        }
      }
      if (lane == 0) {
        page[k] = pg;
        first_row[k] = row;
        first_pos[k] = first;
      }
    }
    __syncthreads();
    // the warp's pair (head, K or V) and its rows of the panel: kPasses passes of them, in registers
    const bool works = pair < 2 * p.Hkv;
    const Pool& pool = p.pool[which];
    const Rows& rows = p.src[which];
    float x[kPasses][16];
    bool is_new[kPasses];
    if (works) {
      const T* in = static_cast<const T*>(rows.p) + (b * rows.s_b + h * rows.s_h);
#pragma unroll
      for (int k = 0; k < kPasses; ++k) {
        const int r = row0 + k * Lane<D>::kRows + l.slot;
        const int t = r < p.panel ? src[r] : -1;
        is_new[k] = t >= 0;  // (the lanes of a row together)
        if (is_new[k]) {
          load8<T, VEC>(in + t * rows.s_t + l.a0 * rows.s_d, rows.s_d, x[k]);
          load8<T, VEC>(in + t * rows.s_t + l.a1 * rows.s_d, rows.s_d, x[k] + 8);
        }
      }
    }
    // the scales as they are, one lane a block (before any warp writes them)
    unsigned char* scale = nullptr;
    int old = 0;
    if (works && lane < per_panel && page[lane] >= 0) {
      scale = pool.scales + (page[lane] * pool.e_n + h * pool.e_h + (first_row[lane] >> p.shift) * pool.e_i);
      old = (int)*scale - 127;
    }
    if (turns) {  // (while the rows arrive)
      fill_angles(p, phase, cs, p.panel, [&](int i) { return src[i] < 0 ? -1 : first_pos[i >> p.shift] + (i & (S - 1)); });
      __syncthreads();
    }
    if (works) {
#pragma unroll
      for (int k = 0; k < kPasses; ++k) {
        const int r = row0 + k * Lane<D>::kRows + l.slot;
        uint32_t a = 0;
        if (is_new[k]) {
          row_values<T, D, RUNS, INTER>(p, l, w, which == 0 && p.wk != nullptr, which == 0 && p.rot > 0,
                                        cs + r * (p.rot / 2), stage, x[k]);
          // sizes as bit patterns: those of infinities and NaN are the largest, and rare
#pragma unroll
          for (int j = 0; j < 16; ++j) a = max(a, __float_as_uint(x[k][j]) & 0x7fffffffu);
          if (a >= 0x7f800000u) {
            a = 0;
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const uint32_t v = __float_as_uint(x[k][j]) & 0x7fffffffu;
              if (v >= 0x7f800000u) x[k][j] = __uint_as_float(0x7fc00000u);  // they have no 8-bit form
              else a = max(a, v);
            }
          }
#pragma unroll
          for (int off = Lane<D>::kLanes / 2; off >= 1; off >>= 1) a = max(a, __shfl_xor_sync(l.lanes, a, off));
        }
        if (l.it == 0 && r < p.panel) amax[warp / parts][r] = __uint_as_float(a);
      }
    }
    __syncthreads();
    if (works) {
      // the blocks' maxima: rows lane, lane + 32, .., then over the lanes of a block
      float a = 0.f;
      for (int i = lane; i < p.panel; i += 32) a = fmaxf(a, amax[warp / parts][i]);
      for (int off = min(S, 32) >> 1; off >= 1; off >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, off));
      a = __shfl_sync(0xffffffffu, a, (lane << p.shift) & 31);  // lane i: of block i
      int now = 0;
      if (scale != nullptr) {
        const bool fresh = src[lane << p.shift] >= 0;
        const int e = scale_exp(a);
        now = fresh ? e : max(e, old);
        if (part == 0 && (fresh || now != old)) *scale = (unsigned char)(now + 127);
        if (fresh) old = now;  // (rows that stay are not touched)
      }
#pragma unroll
      for (int k = 0; k < kPasses; ++k) {
        const int r = row0 + k * Lane<D>::kRows + l.slot, blk = (r >> p.shift) & 15;
        const int e_new = __shfl_sync(0xffffffffu, now, blk), e_old = __shfl_sync(0xffffffffu, old, blk);
        if (r >= p.panel || page[blk] < 0 || (!is_new[k] && e_new == e_old)) continue;
        unsigned char* o = pool.p + (page[blk] * pool.s_n + h * pool.s_h + (first_row[blk] + (r & (S - 1))) * pool.s_r);
        uint2 y0, y1;
        if (is_new[k]) {
          const float f = e_new < 128 ? pow2(-e_new) : __uint_as_float(0x7fc00000u);
          float v[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) v[j] = x[k][j] * f;
          y0.x = to_e4m3x2(v[0], v[1]) | to_e4m3x2(v[2], v[3]) << 16;
          y0.y = to_e4m3x2(v[4], v[5]) | to_e4m3x2(v[6], v[7]) << 16;
          y1.x = to_e4m3x2(v[8], v[9]) | to_e4m3x2(v[10], v[11]) << 16;
          y1.y = to_e4m3x2(v[12], v[13]) | to_e4m3x2(v[14], v[15]) << 16;
        } else {  // the scale rose: rounded again
          const float f = pow2(e_old - e_new);
          auto again = [f](uint32_t z) {
            const float2 u = e4m3x2_to_f2(z & 0xffffu), c = e4m3x2_to_f2(z >> 16);
            return to_e4m3x2(u.x * f, u.y * f) | to_e4m3x2(c.x * f, c.y * f) << 16;
          };
          y0 = *reinterpret_cast<const uint2*>(o + l.a0);
          y1 = *reinterpret_cast<const uint2*>(o + l.a1);
          y0 = make_uint2(again(y0.x), again(y0.y));
          y1 = make_uint2(again(y1.x), again(y1.y));
        }
        *reinterpret_cast<uint2*>(o + l.a0) = y0;
        *reinterpret_cast<uint2*>(o + l.a1) = y1;
      }
    }
    __syncthreads();
  }
}

// ---- reading back: 16 numbers a thread (8 looked up pages and scales twice as
// often: 163 us in place of 135 for a cache of 131072 rows and 8 heads), stored
// by whole sectors, kRead rows in flight
constexpr int kRead = 4;
struct ReadParams {
  Pool pool[2];
  void* out[2];
  int64_t o_b[2], o_h[2], o_t[2], o_d[2];
  const int32_t* pos;
  int64_t p_b, p_t;
  int T, H, shift;
  bool vec;  // 32-byte stores
  PageTable pages;
};

// 16 numbers times their scale, as TO.
template <typename TO>
__device__ __forceinline__ void put16(TO* o, int64_t s_d, bool vec, const uint4& w, float f) {
  float x[16];
  const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 a = e4m3x2_to_f2(v[j] & 0xffffu), c = e4m3x2_to_f2(v[j] >> 16);
    x[4 * j] = a.x * f;
    x[4 * j + 1] = a.y * f;
    x[4 * j + 2] = c.x * f;
    x[4 * j + 3] = c.y * f;
  }
  if (!vec) {
#pragma unroll
    for (int j = 0; j < 16; ++j) o[j * s_d] = from_f32<TO>(x[j]);
  } else if constexpr (sizeof(TO) == 2) {
    Vec<float, 8> y;
#pragma unroll
    for (int j = 0; j < 8; ++j) y.x[j] = __uint_as_float(pack_bf16(x[2 * j], x[2 * j + 1]));
    store(reinterpret_cast<float*>(o), y);
  } else {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      Vec<float, 8> y;
#pragma unroll
      for (int i = 0; i < 8; ++i) y.x[i] = x[8 * j + i];
      store(o + 8 * j, y);
    }
  }
}

// grid: x row chunks, y KV head x {K, V}, z sequence
template <typename TO, int D>
__global__ void __launch_bounds__(kThreads) read_q8_kernel(const __grid_constant__ ReadParams p) {
  constexpr int kLanes = D / 16, kRows = kThreads / kLanes;
  const int which = blockIdx.y & 1, h = blockIdx.y >> 1, b = blockIdx.z;
  const Pool& pool = p.pool[which];
  const int c0 = (threadIdx.x % kLanes) * 16;
  const int t0 = blockIdx.x * (kRows * kRead) + threadIdx.x / kLanes;
  int pg[kRead], r[kRead];
#pragma unroll
  for (int k = 0; k < kRead; ++k) {
    const int t = t0 + k * kRows;
    const int c = t < p.T ? p.pos[b * p.p_b + t * p.p_t] : -1;
    pg[k] = c < 0 ? -1 : page_of(p.pages, b, c);
    r[k] = c & (p.pages.rows - 1);
  }
  uint4 w[kRead];
  int e[kRead];
#pragma unroll
  for (int k = 0; k < kRead; ++k) {
    w[k] = make_uint4(0, 0, 0, 0);
    e[k] = 127;
    if (pg[k] >= 0) {
      w[k] = *reinterpret_cast<const uint4*>(pool.p + (pg[k] * pool.s_n + h * pool.s_h + r[k] * pool.s_r) + c0);
      e[k] = pool.scales[pg[k] * pool.e_n + h * pool.e_h + (r[k] >> p.shift) * pool.e_i];
    }
  }
  TO* out = static_cast<TO*>(p.out[which]) + (b * p.o_b[which] + h * p.o_h[which] + c0 * p.o_d[which]);
#pragma unroll
  for (int k = 0; k < kRead; ++k) {
    const int t = t0 + k * kRows;
    if (t < p.T) put16(out + t * p.o_t[which], p.o_d[which], p.vec, w[k], scale_of(e[k]));
  }
}

// ---- the cache as bf16 for the prompt kernel (kernels.h: ExpandParams)
// grid: x row chunks, y KV head x {K, V}, z sequence
template <int D>
__global__ void __launch_bounds__(kThreads) expand_q8_kernel(const __grid_constant__ ExpandParams p) {
  constexpr int kLanes = D / 16, kRows = kThreads / kLanes;
  const int which = blockIdx.y & 1, h = blockIdx.y >> 1, b = blockIdx.z;
  const int t_max = p.pages.entries * p.pages.rows;
  const int chunk0 = blockIdx.x * (kRows * kRead), chunk1 = chunk0 + kRows * kRead;
  if (blockIdx.y == 0) {  // the table's entries that begin in the chunk
    for (int i = (chunk0 + p.pages.rows - 1) / p.pages.rows + threadIdx.x; i < p.pages.entries && i * p.pages.rows < chunk1;
         i += kThreads)
      p.table[(int64_t)b * p.pages.entries + i] = page_of(p.pages, b, i * p.pages.rows) < 0 ? -1 : b * p.pages.entries + i;
  }
  int len = p.seqlens[b * p.sl_s];
  len = len > t_max ? t_max : len;
  if (chunk0 >= len) return;
  if (p.window > 0) {  // nothing before the earliest key that a row sees
    int first = 0x7fffffff;
    for (int i = threadIdx.x; i < p.Tq; i += kThreads) {
      const int pos = p.qpos[b * p.qp_sb + i * p.qp_si];
      if (pos >= 0) first = min(first, pos >= p.window ? pos - p.window + 1 : 0);
    }
    if (!__syncthreads_or(first < chunk1)) return;
  }
  const int c0 = (threadIdx.x % kLanes) * 16;
  uint4 w[kRead];
  int e[kRead], t[kRead];
#pragma unroll
  for (int k = 0; k < kRead; ++k) {
    t[k] = chunk0 + threadIdx.x / kLanes + k * kRows;
    const int pg = t[k] < len ? page_of(p.pages, b, t[k]) : -1;
    const int r = t[k] & (p.pages.rows - 1);
    w[k] = make_uint4(0, 0, 0, 0);
    e[k] = 127;
    if (pg < 0) {
      t[k] = -1;
    } else {
      w[k] = *reinterpret_cast<const uint4*>(p.pool[which] + (pg * p.s_n[which] + h * p.s_h[which] + r * p.s_r[which]) + c0);
      e[k] = p.scales[which][pg * p.e_n[which] + h * p.e_h[which] + (r >> p.scale_shift) * p.e_i[which]];
    }
  }
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out[which]);
#pragma unroll
  for (int k = 0; k < kRead; ++k) {
    if (t[k] < 0) continue;
    const int64_t page = (int64_t)b * p.pages.entries + (t[k] >> p.pages.shift);
    put16(out + ((page * p.Hkv + h) * p.pages.rows + (t[k] & (p.pages.rows - 1))) * D + c0, 1, true, w[k], scale_of(e[k]));
  }
}

// ------------------------------------------------------------- launches
template <typename T, int D, bool RUNS, bool INTER>
cudaError_t launch_append_v(const AppendParams& p, bool vec, dim3 grid, cudaStream_t stream) {
  const int smem = kStage<D, RUNS> * 4 + p.panel * (p.rot / 2) * 8;
  auto go = [&](auto kernel, DeviceOnce& once) {
    if (smem > 32 * 1024) {  // (with what the kernel has besides)
      const int most = kStage<D, RUNS> * 4 + (int)kMaxScaleRows * (D / 2) * 8;
      if (cudaError_t e = once.set_smem(reinterpret_cast<const void*>(kernel), most, false); e != cudaSuccess) return e;
    }
    kernel<<<grid, kThreads, smem, stream>>>(p);
    return cudaGetLastError();
  };
  if constexpr (RUNS) {
    if (vec) {
      static DeviceOnce once;
      return go(append_q8_kernel<T, D, RUNS, INTER, true>, once);
    }
  }
  static DeviceOnce once;
  return go(append_q8_kernel<T, D, RUNS, INTER, false>, once);
}
template <typename T, int D>
cudaError_t launch_append(const AppendParams& p, bool inter, bool vec, dim3 grid, cudaStream_t stream) {
  if (p.rot % 16 == 0)
    return inter && p.rot ? launch_append_v<T, D, true, true>(p, vec, grid, stream)
                          : launch_append_v<T, D, true, false>(p, vec, grid, stream);
  return inter ? launch_append_v<T, D, false, true>(p, vec, grid, stream)
               : launch_append_v<T, D, false, false>(p, vec, grid, stream);
}

// ------------------------------------------------------------- arguments
Rows rows_of(const blkattn_tensor* t) { return {t->data, t->strides[0], t->strides[1], t->strides[2], t->strides[3]}; }
Pool pool_of(const blkattn_tensor& t, const blkattn_tensor* e) {
  return {static_cast<unsigned char*>(t.data), t.strides[0], t.strides[1], t.strides[2],
          static_cast<unsigned char*>(e->data), e->strides[0], e->strides[1], e->strides[2]};
}
// Rows that the kernels move by 16 (or 32) bytes (a stride of a dim of size 1 is not used).
bool vec_rows(const blkattn_tensor* t, int access = 16) {
  const int64_t bytes = t->dtype == BLKATTN_BF16 ? 2 : 4;
  if (t->strides[3] != 1 || reinterpret_cast<uintptr_t>(t->data) % access != 0) return false;
  for (int i = 0; i < 3; ++i)
    if (t->sizes[i] > 1 && t->strides[i] * bytes % access != 0) return false;
  return true;
}

}  // namespace

cudaError_t launch_expand_q8(const ExpandParams& p, int d, cudaStream_t stream) {
  const int rows = kThreads / (d / 16) * kRead;
  const int64_t t_max = (int64_t)p.pages.entries * p.pages.rows;
  const dim3 grid((unsigned)((t_max + rows - 1) / rows), (unsigned)(2 * p.Hkv), (unsigned)p.B);
  if (d == 128) expand_q8_kernel<128><<<grid, kThreads, 0, stream>>>(p);
  else expand_q8_kernel<64><<<grid, kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

int check_pages_q8(const blkattn_tensor* k_pages, const blkattn_tensor* v_pages, const blkattn_tensor* k_scales,
                   const blkattn_tensor* v_scales, const blkattn_tensor* table, int64_t B, int64_t H, int64_t d,
                   blkattn_tensor* kn, blkattn_tensor* vn, PageTable* out, int* shift) {
  if (int st = check_pages(k_pages, v_pages, table, BLKATTN_E4M3, B, H, d, out); st != BLKATTN_OK) return st;
  if (!tensor_dims_ok(k_scales, 3) || !tensor_dims_ok(v_scales, 3)) return BLKATTN_ERR_INVALID_ARG;
  if (k_scales->dtype != BLKATTN_E8M0 || v_scales->dtype != BLKATTN_E8M0) return BLKATTN_ERR_INVALID_ARG;
  const int64_t P = out->rows, n = k_scales->sizes[2];
  if (n < 1 || n > P || P % n != 0 || (n & (n - 1)) != 0) return BLKATTN_ERR_INVALID_ARG;
  for (const blkattn_tensor* e : {k_scales, v_scales}) {
    if (e->sizes[0] != k_pages->sizes[0] || e->sizes[1] != H || e->sizes[2] != n) return BLKATTN_ERR_INVALID_ARG;
    if (!writable(e)) return BLKATTN_ERR_INVALID_ARG;
  }
  if (P / n > kMaxScaleRows || (d != 64 && d != 128)) return BLKATTN_ERR_UNSUPPORTED;
  *shift = 0;
  while ((n << *shift) < P) ++*shift;
  *kn = *k_pages;
  *vn = *v_pages;
  for (blkattn_tensor* t : {kn, vn}) {
    for (int i = 0; i < 3; ++i) {
      if (t->sizes[i] == 1) t->strides[i] = d;
      if (t->strides[i] == 0 || t->strides[i] % 16 != 0) return BLKATTN_ERR_INVALID_ARG;
    }
    if (t->strides[3] != 1 || reinterpret_cast<uintptr_t>(t->data) % 16 != 0) return BLKATTN_ERR_INVALID_ARG;
  }
  return BLKATTN_OK;
}

}  // namespace blkattn

extern "C" {

int blkattn_paged_append_q8(const blkattn_tensor* k, const blkattn_tensor* v, const blkattn_tensor* pos,
                            const blkattn_tensor* page_table, const blkattn_tensor* k_pages,
                            const blkattn_tensor* v_pages, const blkattn_tensor* k_scales,
                            const blkattn_tensor* v_scales, const blkattn_tensor* k_weight_opt, float eps,
                            const blkattn_tensor* phases_opt, int32_t layout, float mscale,
                            const blkattn_tensor* q_opt, const blkattn_tensor* q_weight_opt,
                            const blkattn_tensor* q_out_opt, blkattn_stream_t stream_) {
  using namespace blkattn;
  if (!tensor_dims_ok(k, 4) || !tensor_dims_ok(v, 4) || !tensor_dims_ok(pos, 2)) return BLKATTN_ERR_INVALID_ARG;
  if (!floats(k) || v->dtype != k->dtype || pos->dtype != BLKATTN_I32) return BLKATTN_ERR_INVALID_ARG;
  const int64_t B = k->sizes[0], H = k->sizes[1], T = k->sizes[2], d = k->sizes[3];
  for (int i = 0; i < 4; ++i)
    if (v->sizes[i] != k->sizes[i]) return BLKATTN_ERR_INVALID_ARG;
  if (pos->sizes[0] != B || pos->sizes[1] != T || d < 1) return BLKATTN_ERR_INVALID_ARG;
  PageTable pt;
  blkattn_tensor kn, vn;
  int shift = 0;
  if (int st = check_pages_q8(k_pages, v_pages, k_scales, v_scales, page_table, B, H, d, &kn, &vn, &pt, &shift);
      st != BLKATTN_OK)
    return st;
  if ((k_pages->data == v_pages->data && k_pages->data != nullptr) ||
      (k_scales->data == v_scales->data && k_scales->data != nullptr))
    return BLKATTN_ERR_INVALID_ARG;
  if (phases_opt) {
    if (int st = check_phases(phases_opt, layout, d); st != BLKATTN_OK) return st;
    if (!finite(mscale)) return BLKATTN_ERR_INVALID_ARG;
  }
  if ((q_opt == nullptr) != (q_out_opt == nullptr) || (q_weight_opt && !q_opt)) return BLKATTN_ERR_INVALID_ARG;
  for (const blkattn_tensor* w : {k_weight_opt, q_weight_opt})
    if (w && (!tensor_dims_ok(w, 1) || !floats(w) || w->sizes[0] != d)) return BLKATTN_ERR_INVALID_ARG;
  if (k_weight_opt && q_weight_opt && k_weight_opt->dtype != q_weight_opt->dtype) return BLKATTN_ERR_INVALID_ARG;
  if ((k_weight_opt || q_weight_opt) && (!finite(eps) || eps < 0.f)) return BLKATTN_ERR_INVALID_ARG;
  int64_t Hq = 0;
  if (q_opt) {
    if (!tensor_dims_ok(q_opt, 4) || !tensor_dims_ok(q_out_opt, 4)) return BLKATTN_ERR_INVALID_ARG;
    if (q_opt->dtype != k->dtype || q_out_opt->dtype != k->dtype) return BLKATTN_ERR_INVALID_ARG;
    Hq = q_opt->sizes[1];
    if (q_opt->sizes[0] != B || q_opt->sizes[2] != T || q_opt->sizes[3] != d) return BLKATTN_ERR_INVALID_ARG;
    for (int i = 0; i < 4; ++i)
      if (q_out_opt->sizes[i] != q_opt->sizes[i]) return BLKATTN_ERR_INVALID_ARG;
    if (!writable(q_out_opt) || !in_place_ok(q_opt, q_out_opt)) return BLKATTN_ERR_INVALID_ARG;
  }
  if (!tensors_on_one_device(k, {v, pos, page_table, k_pages, v_pages, k_scales, v_scales, k_weight_opt, phases_opt,
                                 q_opt, q_weight_opt, q_out_opt}))
    return BLKATTN_ERR_INVALID_ARG;
  if (H > 0x7fff || Hq > 0x7fff || B > 0x7fffffff || T > 0x7fffffff - 0xffff || (B > 0 && T > 0x7fffffff / B) ||
      B * T * Hq > kMostRows)
    return BLKATTN_ERR_UNSUPPORTED;
  if (B == 0 || T == 0) return BLKATTN_OK;
  for (const blkattn_tensor* t : {k, v, pos, page_table, k_pages, v_pages, k_scales, v_scales})
    if (t->data == nullptr) return BLKATTN_ERR_INVALID_ARG;
  for (const blkattn_tensor* t : {phases_opt, k_weight_opt, q_weight_opt})
    if (t && t->data == nullptr) return BLKATTN_ERR_INVALID_ARG;
  if (q_opt && Hq > 0 && (q_opt->data == nullptr || q_out_opt->data == nullptr)) return BLKATTN_ERR_INVALID_ARG;
  if (int st = require_current_device(k->device); st != BLKATTN_OK) return st;
  AppendParams p{};
  p.src[0] = rows_of(k);
  p.src[1] = rows_of(v);
  p.pool[0] = pool_of(kn, k_scales);
  p.pool[1] = pool_of(vn, v_scales);
  bool vec = vec_rows(k) && vec_rows(v);
  if (q_opt && Hq > 0) {
    p.q = rows_of(q_opt);
    p.q_out = q_out_opt->data;
    p.o_b = q_out_opt->strides[0]; p.o_h = q_out_opt->strides[1];
    p.o_t = q_out_opt->strides[2]; p.o_d = q_out_opt->strides[3];
  }
  if (q_weight_opt) { p.wq = q_weight_opt->data; p.wq_s = q_weight_opt->strides[0]; }
  if (k_weight_opt) { p.wk = k_weight_opt->data; p.wk_s = k_weight_opt->strides[0]; }
  const blkattn_tensor* w = k_weight_opt ? k_weight_opt : q_weight_opt;
  p.w_f32 = w && w->dtype == BLKATTN_F32;
  p.eps = eps;
  p.mscale = mscale;
  p.pos = static_cast<const int32_t*>(pos->data);
  p.p_b = pos->strides[0]; p.p_t = pos->strides[1];
  if (phases_opt) {
    p.phases = static_cast<const int64_t*>(phases_opt->data);
    p.ph_s = phases_opt->strides[0];
    p.rot = (int)(2 * phases_opt->sizes[0]);
  }
  p.B = (int)B; p.T = (int)T; p.Hkv = (int)H; p.Hq = (int)Hq;
  p.shift = shift;
  p.panel = (1 << shift) < 16 ? 16 : 1 << shift;
  const int parts = p.panel * (int)d / 2048 < 1 ? 1 : p.panel * (int)d / 2048;  // (as in the kernel)
  p.kv_groups = (int)((2 * H * parts + kWarps - 1) / kWarps);
  p.pages = pt;
  const int64_t q_groups = (Hq + kQHeads - 1) / kQHeads;
  // (many KV heads in blocks of many rows leave the grid no room for the query rows)
  const bool own = B * T * Hq >= kOwnKernelRows || (Hq > 0 && p.kv_groups + q_groups > 65535);
  if (Hq > 0 && !own) vec = vec && vec_rows(q_opt) && vec_rows(q_out_opt);
  const dim3 grid((unsigned)(B * ((T + p.panel - 1) / p.panel)), (unsigned)(p.kv_groups + (own ? 0 : q_groups)));
  const bool inter = layout == BLKATTN_ROPE_INTERLEAVED;
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  cudaError_t e;
  if (k->dtype == BLKATTN_BF16)
    e = d == 128 ? launch_append<__nv_bfloat16, 128>(p, inter, vec, grid, stream)
                 : launch_append<__nv_bfloat16, 64>(p, inter, vec, grid, stream);
  else
    e = d == 128 ? launch_append<float, 128>(p, inter, vec, grid, stream)
                 : launch_append<float, 64>(p, inter, vec, grid, stream);
  if (e == cudaSuccess && own)
    e = launch_query_rows(q_opt, q_weight_opt, pos, phases_opt, layout, mscale, eps, q_out_opt, stream);
  return e == cudaSuccess ? BLKATTN_OK : report_cuda_failure(e);
}

int blkattn_paged_read_q8(const blkattn_tensor* pos, const blkattn_tensor* page_table, const blkattn_tensor* k_pages,
                          const blkattn_tensor* v_pages, const blkattn_tensor* k_scales,
                          const blkattn_tensor* v_scales, const blkattn_tensor* k_out, const blkattn_tensor* v_out,
                          blkattn_stream_t stream_) {
  using namespace blkattn;
  if (!tensor_dims_ok(pos, 2) || !tensor_dims_ok(k_out, 4) || !tensor_dims_ok(v_out, 4)) return BLKATTN_ERR_INVALID_ARG;
  if (pos->dtype != BLKATTN_I32 || !floats(k_out) || v_out->dtype != k_out->dtype) return BLKATTN_ERR_INVALID_ARG;
  const int64_t B = k_out->sizes[0], H = k_out->sizes[1], T = k_out->sizes[2], d = k_out->sizes[3];
  for (int i = 0; i < 4; ++i)
    if (v_out->sizes[i] != k_out->sizes[i]) return BLKATTN_ERR_INVALID_ARG;
  if (pos->sizes[0] != B || pos->sizes[1] != T) return BLKATTN_ERR_INVALID_ARG;
  PageTable pt;
  blkattn_tensor kn, vn;
  int shift = 0;
  if (int st = check_pages_q8(k_pages, v_pages, k_scales, v_scales, page_table, B, H, d, &kn, &vn, &pt, &shift);
      st != BLKATTN_OK)
    return st;
  if (!writable(k_out) || !writable(v_out) || (k_out->data == v_out->data && k_out->data != nullptr))
    return BLKATTN_ERR_INVALID_ARG;
  if (!tensors_on_one_device(pos, {page_table, k_pages, v_pages, k_scales, v_scales, k_out, v_out}))
    return BLKATTN_ERR_INVALID_ARG;
  if (H > 0x7fff || B > 0xffff || T > 0x7fffffff - 0xffff) return BLKATTN_ERR_UNSUPPORTED;
  if (B == 0 || T == 0) return BLKATTN_OK;
  for (const blkattn_tensor* t : {pos, page_table, k_pages, v_pages, k_scales, v_scales, k_out, v_out})
    if (t->data == nullptr) return BLKATTN_ERR_INVALID_ARG;
  if (int st = require_current_device(pos->device); st != BLKATTN_OK) return st;
  ReadParams p{};
  p.pool[0] = pool_of(kn, k_scales);
  p.pool[1] = pool_of(vn, v_scales);
  const blkattn_tensor* outs[2] = {k_out, v_out};
  for (int i = 0; i < 2; ++i) {
    p.out[i] = outs[i]->data;
    p.o_b[i] = outs[i]->strides[0]; p.o_h[i] = outs[i]->strides[1];
    p.o_t[i] = outs[i]->strides[2]; p.o_d[i] = outs[i]->strides[3];
  }
  p.pos = static_cast<const int32_t*>(pos->data);
  p.p_b = pos->strides[0]; p.p_t = pos->strides[1];
  p.T = (int)T; p.H = (int)H; p.shift = shift;
  p.vec = vec_rows(k_out, 32) && vec_rows(v_out, 32);
  p.pages = pt;
  const int rows = kThreads / (int)(d / 16) * kRead;
  const dim3 grid((unsigned)((T + rows - 1) / rows), (unsigned)(2 * H), (unsigned)B);
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  if (k_out->dtype == BLKATTN_BF16) {
    if (d == 128) read_q8_kernel<__nv_bfloat16, 128><<<grid, kThreads, 0, stream>>>(p);
    else read_q8_kernel<__nv_bfloat16, 64><<<grid, kThreads, 0, stream>>>(p);
  } else {
    if (d == 128) read_q8_kernel<float, 128><<<grid, kThreads, 0, stream>>>(p);
    else read_q8_kernel<float, 64><<<grid, kThreads, 0, stream>>>(p);
  }
  if (cudaError_t e = cudaGetLastError(); e != cudaSuccess) return report_cuda_failure(e);
  return BLKATTN_OK;
}

}  // extern "C"
