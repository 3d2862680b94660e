// Attention of few query rows over the 8-bit paged cache (q8.cuh has its
// numbers): decode and verify rows, token trees, windows.
//
// With k = 2^ek k8 and v = 2^ev v8, e a block's exponent,
//
//     z_j = scale 2^ek_j (q . k8_j),   out = sum e^z_j 2^ev_j v8_j / sum e^z_j.
//
// e4m3 is exact in f16 and so is a bf16 row after a power of two of its own, so
// the products run on f16 with the rows' and blocks' powers of two outside:
// 2^ek goes into the score, 2^ev into the weight.  A row has two running
// references (base 2): M >= max z - 8 for the sum l of e^z, and, relative to it,
// R >= max (z - M + ev) - 4 for the weights of the value product, so that weights
// use f16's range whatever the blocks' exponents are.  (R is kept as a difference:
// z + ev would lose ev beside a large z.)
//
// The path of a byte.  What bounds these calls is memory, and with 8-bit keys
// an SM has half of a bf16 cache's time for a key: 4 KB of K and V must be
// taken in every 95 ns.  Rows go by 16-byte asynchronous copies into slots of
// the copying thread's own in shared memory and from there, by that thread,
// straight into mma fragments: the contraction's order is free, so a lane takes
// neighbouring bytes and q is laid out to match.  No thread reads another's
// slot, so there is no barrier in the stream, and a byte crosses shared memory
// twice (through a converted tile for tcgen05 it would cross it six times, more
// than shared memory's rate allows at the card's: K and V written, read,
// written as f16, read by the product).
//
//   S [16 keys x 8 rows]  = K8 Q^T      A = K8 (m = keys), B = Q (n = rows)
//   U^T [d x 8 rows]     += V8^T P^T    A = V8^T (m = dims; two keys' bytes
//                                       interleaved), B = P^T (S transposed in
//                                       registers)
//
// Work split: tiles of 128 keys (16 a warp) of all (sequence, KV head, row
// group) units in order, cut into equal ranges, one a CTA; a warp keeps its own
// statistics, joined when a unit ends.  A unit that lies in several CTAs leaves
// partial states, and the CTA that arrives last joins them in order.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kernels.h"
#include "ptx.cuh"
#include "q8.cuh"

namespace blkattn {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kNegInf = -__builtin_huge_valf();
constexpr float kLazyM = 8.f, kLazyR = 4.f;
constexpr float kLift = 11.f;  // weights reach 2^(kLift + kLazyR) = 2^15 in f16
constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kStep = 16;                // keys of a warp in a tile
constexpr int kTile = kStep * kWarps;

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transposed(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// Copies of 16 and 8 bytes to the thread's own slot; n = 0: zeros.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, int n) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void copy8(uint32_t dst, const void* src, int n) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}

template <int D, int NT>
struct Q8Layout {
  // (tiles in flight: 8 or, with two resident CTAs of 8 rows, 16 warps of 4 KB each)
  static constexpr int kStages = NT == 1 ? 2 : 3;
  static constexpr int kRows = 8 * NT;
  static constexpr int kStageBytes = kStep * D * 2;  // a warp's keys, K and V
  static constexpr int kRing = kWarps * kStages * kStageBytes;
  static constexpr int kPad = D + 4;
  static constexpr int kOffU = kRing;                             // float [kWarps][kRows][kPad]
  static constexpr int kOffStat = kOffU + kWarps * kRows * kPad * 4;  // float [3][kWarps][kRows]
  static constexpr int kOffRow = kOffStat + 3 * kWarps * kRows * 4;   // float [3][kRows]
  static constexpr int kOffTab = (kOffRow + 3 * kRows * 4 + 7) / 8 * 8;  // uint64 [B], then int [5 B + 1]
  static constexpr int bytes(int B) { return kOffTab + B * 8 + (5 * B + 1) * 4; }
  static_assert(kOffU % 16 == 0 && kPad % 4 == 0, "alignment");
  static_assert(kRows * kDecodeQ8MaxCtas <= kWarps * kRows * kPad, "the factors of a unit's parts");
};

// Where a tile lies: unit (b, kvh, rg), tile j of its nt.
struct Place {
  int b, kvh, rg, j, nt;
};

template <int D, int NT, bool FINE>
__global__ void __launch_bounds__(kThreads, NT == 1 ? 2 : 1) decode_q8_kernel(const __grid_constant__ Q8Params p) {
  using L = Q8Layout<D, NT>;
  constexpr int kRows = L::kRows;
  constexpr int KL = D / 64;  // 16-byte runs of a K row in a lane
  constexpr int VB = D / 8;   // bytes of a V row in a lane
  constexpr int MT = D / 16;  // m-tiles of the value product
  extern __shared__ __align__(16) unsigned char sm[];
  float* s_u = reinterpret_cast<float*>(sm + L::kOffU);
  float* s_stat = reinterpret_cast<float*>(sm + L::kOffStat);
  float* s_row = reinterpret_cast<float*>(sm + L::kOffRow);
  uint64_t* s_seen = reinterpret_cast<uint64_t*>(sm + L::kOffTab);  // [B] tree nodes that some row lists
  int* s_end = reinterpret_cast<int*>(s_seen + p.B);  // [B] keys that some row sees are [start, end)
  int* s_start = s_end + p.B;                            // (a multiple of kStep)
  int* s_nt = s_start + p.B;
  int* s_tree = s_nt + p.B;  // [B] key of the tree's first node
  int* s_pre = s_tree + p.B;  // [B + 1] tiles before the sequence
  __shared__ int s_last;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t4 = lane & 3;
  const int units_b = p.Hkv * p.row_groups;  // units of a sequence

  // ---- the sequences' key ranges and the order of all tiles
  for (int b = threadIdx.x; b < p.B; b += kThreads) {
    int len = p.seqlens[b * p.sl_s];
    len = len < 0 ? 0 : (len > p.Tmax ? p.Tmax : len);
    int end = 0, start = 0x7fffffff;
    uint64_t seen = 0;
#pragma unroll 4
    for (int i = 0; i < p.Tq; ++i) {
      if (p.tree) seen |= (uint64_t)p.tree[b * p.tr_sb + i * p.tr_si];
      const int pos = p.qpos[b * p.qp_sb + i * p.qp_si];
      const int e = pos < 0 ? 0 : (pos >= len ? len : pos + 1);
      const int f = p.window > 0 && pos >= p.window ? pos - p.window + 1 : 0;
      if (e > f) {
        end = max(end, e);
        start = min(start, f);
      }
    }
    start = end > 0 ? start & ~(kStep - 1) : 0;
    s_seen[b] = seen;
    s_tree[b] = p.tree ? len - p.Tq : 0x7fffffff;
    s_end[b] = end;
    s_start[b] = start;
    s_nt[b] = (end - start + kTile - 1) / kTile;
  }
  __syncthreads();
  if (warp == 0) {
    int before = 0;
    for (int b0 = 0; b0 < p.B; b0 += 32) {
      const int n = b0 + lane < p.B ? s_nt[b0 + lane] * units_b : 0;
      int x = n;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, off);
        if (lane >= off) x += y;
      }
      if (b0 + lane < p.B) s_pre[b0 + lane] = before + x - n;
      before += __shfl_sync(0xffffffffu, x, 31);
    }
    if (lane == 0) s_pre[p.B] = before;
  }
  __syncthreads();
  const int64_t W = s_pre[p.B];

  auto out_row = [&](int b, int kvh, int row, int& h, int& i) {  // row of the KV head's G Tq
    const int hg = row / p.Tq;
    i = row - hg * p.Tq;
    h = kvh * p.G + hg;
  };
  auto store_out = [&](int b, int h, int i, int d, float o) {
    const int64_t at = b * p.o_sb + h * p.o_sh + i * p.o_si + d * p.o_sd;
    if (p.out_bf16)
      static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(o);
    else
      static_cast<float*>(p.out)[at] = o;
  };
  // sequences that see nothing: zeros, -inf
  for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
    if (s_nt[b] > 0) continue;
    for (int64_t u = threadIdx.x; u < (int64_t)p.Hq * p.Tq * D; u += kThreads) {
      const int d = (int)(u % D);
      const int64_t r = u / D;
      const int i = (int)(r % p.Tq), h = (int)(r / p.Tq);
      store_out(b, h, i, d, 0.f);
      if (d == 0) p.lse[b * p.l_sb + h * p.l_sh + i * p.l_si] = kNegInf;
    }
  }
  const int64_t P = W < (int64_t)gridDim.x ? W : (int64_t)gridDim.x;
  if ((int64_t)blockIdx.x >= P) return;
  const int t0 = (int)(blockIdx.x * W / P), t1 = (int)((blockIdx.x + 1) * W / P);
  auto cta_of = [&](int64_t t) { return (int)(((t + 1) * P + W - 1) / W) - 1; };

  auto place_of = [&](int t) {
    int lo = 0, hi = p.B - 1;  // the last sequence with s_pre <= t (and tiles)
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (s_pre[mid] <= t) lo = mid;
      else hi = mid - 1;
    }
    Place a;
    a.b = lo;
    a.nt = s_nt[lo];
    const int off = t - s_pre[lo], u = off / a.nt;
    a.j = off - u * a.nt;
    a.kvh = u / p.row_groups;
    a.rg = u - a.kvh * p.row_groups;
    return a;
  };
  auto next = [&](Place& a) {
    if (++a.j < a.nt) return;
    a.j = 0;
    if (++a.rg < p.row_groups) return;
    a.rg = 0;
    if (++a.kvh < p.Hkv) return;
    a.kvh = 0;
    do {
      ++a.b;
      a.nt = a.b < p.B ? s_nt[a.b] : 1;
    } while (a.nt == 0);
  };

  // ---- the stream: a tile's page numbers, then its rows and scales, ahead of its use
  unsigned char* ring = sm + warp * (L::kStages * L::kStageBytes);
  auto key0_of = [&](const Place& a) { return s_start[a.b] + a.j * kTile + warp * kStep; };
  // page of key (lane mod 16) of the warp's, -1: none, or no row sees the key
  // (past the end, a tree node that no row lists: its row may hold anything)
  auto look_up = [&](const Place& a) {
    const int key = key0_of(a) + (lane & 15), node = key - s_tree[a.b];
    if (key >= s_end[a.b] || (node >= 0 && !((s_seen[a.b] >> node) & 1))) return -1;
    return page_of(p.pages, a.b, key);
  };
  auto issue = [&](const Place& a, int pg, int stage) {  // returns the lane's scale byte
    const int key0 = key0_of(a), mask = p.pages.rows - 1;
    const uint32_t dst = smem_u32(ring + stage * L::kStageBytes);
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int pr = __shfl_sync(0xffffffffu, pg, g + 8 * r);
      const char* src = p.k + (int64_t)max(pr, 0) * p.k_sn + a.kvh * p.k_sh + ((key0 + g + 8 * r) & mask) * p.k_sr + 16 * t4;
#pragma unroll
      for (int h = 0; h < KL; ++h) copy16(dst + (r * KL + h) * 512 + lane * 16, src + 64 * h, pr < 0 ? 0 : 16);
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int kk = 2 * t4 + (r & 1) + 8 * (r >> 1);
      const int pr = __shfl_sync(0xffffffffu, pg, kk);
      const char* src = p.v + (int64_t)max(pr, 0) * p.v_sn + a.kvh * p.v_sh + ((key0 + kk) & mask) * p.v_sr + VB * g;
      const uint32_t at = dst + 2 * KL * 512 + r * (32 * VB) + lane * VB;
      if constexpr (VB == 16) copy16(at, src, pr < 0 ? 0 : 16);
      else copy8(at, src, pr < 0 ? 0 : 8);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    // lanes 0-15: the scale of K of key `lane`; 16-31: of V
    int e = 127;
    if (pg >= 0) {
      const int blk = ((key0 + (lane & 15)) & mask) >> p.scale_shift;
      e = lane < 16 ? p.k_sc[(int64_t)pg * p.ke_sn + a.kvh * p.ke_sh + blk * p.ke_si]
                    : p.v_sc[(int64_t)pg * p.ve_sn + a.kvh * p.ve_sh + blk * p.ve_si];
    }
    return e;
  };

  Place ahead = place_of(t0), cur = ahead;
  const int n = t1 - t0;
  int pg_next = look_up(ahead);
  int pg[L::kStages], sc[L::kStages];  // of the tiles in flight, the oldest first
  int issued = 0;
  auto issue_next = [&](int slot) {
    pg[slot] = -1;
    sc[slot] = 127;
    if (issued < n) {
      pg[slot] = pg_next;
      sc[slot] = issue(ahead, pg_next, issued % L::kStages);
      if (issued + 1 < n) {
        next(ahead);
        pg_next = look_up(ahead);
      }
    } else {
      asm volatile("cp.async.commit_group;" ::: "memory");
    }
    ++issued;
  };
#pragma unroll
  for (int i = 0; i < L::kStages - 1; ++i) issue_next(i);

  // ---- one unit's state in this warp
  float U[NT][MT][4];
  float M[NT][2], R[NT][2], ls[NT][2], fac[NT][2];
  int r_end[NT][2], r_first[NT][2];
  uint32_t Q[NT][KL * 4][2];
  int min_end = 0, max_first = 0, tree_base = 0x7fffffff, rows = 0, row0 = 0;

  auto begin_unit = [&]() {
    row0 = cur.rg * p.rows_cta;
    rows = min(p.rows_cta, p.G * p.Tq - row0);
    int len = p.seqlens[cur.b * p.sl_s];
    len = len < 0 ? 0 : (len > p.Tmax ? p.Tmax : len);
    tree_base = s_tree[cur.b];
    min_end = 0x7fffffff;
    max_first = 0;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      // the fragments of row 8 nt + g, scaled by a power of two into f16's upper range
      const int r = 8 * nt + g;
      float x[KL][16];
      float amax = 0.f;
      int h, i;
      out_row(cur.b, cur.kvh, row0 + min(r, rows - 1), h, i);
      const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.q) + (cur.b * p.q_sb + h * p.q_sh + i * p.q_si);
#pragma unroll
      for (int c = 0; c < KL; ++c) {
        if (p.q_vec) {
          const uint4* v = reinterpret_cast<const uint4*>(q + 64 * c + 16 * t4);
          const uint4 a = __ldg(v), b = __ldg(v + 1);
          const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            x[c][2 * k] = bf16lo(w[k]);
            x[c][2 * k + 1] = bf16hi(w[k]);
          }
        } else {
#pragma unroll
          for (int k = 0; k < 16; ++k) x[c][k] = __bfloat162float(q[(64 * c + 16 * t4 + k) * p.q_sd]);
        }
#pragma unroll
        for (int k = 0; k < 16; ++k) amax = fmaxf(amax, fabsf(x[c][k]));
      }
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      const int e = amax > 0.f ? (int)(__float_as_uint(amax) >> 23) - 127 : 14;
      // (two factors: 14 - e may pass 127; inf and NaN pass through)
      const float f1 = pow2((14 - e) / 2), f2 = pow2((14 - e) - (14 - e) / 2);
#pragma unroll
      for (int c = 0; c < KL; ++c)
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          Q[nt][4 * c + s][0] = pack_h2(x[c][4 * s] * f1 * f2, x[c][4 * s + 1] * f1 * f2);
          Q[nt][4 * c + s][1] = pack_h2(x[c][4 * s + 2] * f1 * f2, x[c][4 * s + 3] * f1 * f2);
        }
      const float back = p.scale_log2 * pow2(e - 14);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int rr = 8 * nt + 2 * t4 + c;
        fac[nt][c] = __shfl_sync(0xffffffffu, back, (2 * t4 + c) * 4);
        int end = 0, first = 0;
        if (rr < rows) {
          out_row(cur.b, cur.kvh, row0 + rr, h, i);
          const int pos = p.qpos[cur.b * p.qp_sb + i * p.qp_si];
          end = pos < 0 ? 0 : (pos >= len ? len : pos + 1);
          first = p.window > 0 && pos >= p.window ? pos - p.window + 1 : 0;
          min_end = min(min_end, end);
          max_first = max(max_first, first);
        }
        r_end[nt][c] = end;
        r_first[nt][c] = first;
        M[nt][c] = R[nt][c] = kNegInf;
        ls[nt][c] = 0.f;
      }
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int c = 0; c < 4; ++c) U[nt][m][c] = 0.f;
    }
#pragma unroll
    for (int off = 1; off <= 2; off <<= 1) {
      min_end = min(min_end, __shfl_xor_sync(0xffffffffu, min_end, off));
      max_first = max(max_first, __shfl_xor_sync(0xffffffffu, max_first, off));
    }
  };

  // the unit's rows from u, l and the references, in this CTA's shared memory
  // or joined from parts
  // R of a state at M as it is at a common M
  auto moved = [](float r, float m, float common) { return m == common ? r : r + (m - common); };
  auto finish_row = [&](float u, float l, float m, float r, int row, int d) {
    int h, i;
    out_row(cur.b, cur.kvh, row0 + row, h, i);
    const bool none = l == 0.f;
    const float f = none ? 0.f : fast_exp2(0.5f * (r - kLift));  // (the whole factor may pass fp32's range)
    store_out(cur.b, h, i, d, none ? 0.f : u * f / l * f);
    if (d == 0) p.lse[cur.b * p.l_sb + h * p.l_sh + i * p.l_si] = none ? kNegInf : (m + __log2f(l)) * kLn2;
  };

  auto end_unit = [&](int first_tile) {
    // the warps' states in shared memory, on common references
    float* sM = s_stat + warp * kRows;
    float* sR = sM + kWarps * kRows;
    float* sL = sR + kWarps * kRows;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float l = ls[nt][c];
#pragma unroll
        for (int off = 4; off <= 16; off <<= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
        if (g == 0) {
          const int r = 8 * nt + 2 * t4 + c;
          sM[r] = M[nt][c];
          sR[r] = R[nt][c];
          sL[r] = l;
        }
      }
    __syncthreads();
    if (threadIdx.x < kRows) {
      float m = kNegInf, r = kNegInf, l = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) m = fmaxf(m, s_stat[w * kRows + threadIdx.x]);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float mw = s_stat[w * kRows + threadIdx.x];
        r = fmaxf(r, moved(s_stat[(kWarps + w) * kRows + threadIdx.x], mw, m));
        l += s_stat[(2 * kWarps + w) * kRows + threadIdx.x] * (mw == m ? 1.f : fast_exp2(mw - m));
      }
      s_row[threadIdx.x] = m;
      s_row[kRows + threadIdx.x] = r;
      s_row[2 * kRows + threadIdx.x] = l;
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int row = 8 * nt + 2 * t4 + c;
        float m = kNegInf, r = kNegInf;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) m = fmaxf(m, s_stat[w * kRows + row]);
#pragma unroll
        for (int w = 0; w < kWarps; ++w)
          r = fmaxf(r, moved(s_stat[(kWarps + w) * kRows + row], s_stat[w * kRows + row], m));
        const float own = moved(R[nt][c], M[nt][c], m), f = own == r ? 1.f : fast_exp2(own - r);
        float* o = s_u + (warp * kRows + row) * L::kPad + VB * g;
#pragma unroll
        for (int m = 0; m < MT; ++m)
          *reinterpret_cast<float2*>(o + 2 * m) = make_float2(U[nt][m][c] * f, U[nt][m][2 + c] * f);
      }
    __syncthreads();
    const int u = (cur.b * p.Hkv + cur.kvh) * p.row_groups + cur.rg;
    const int64_t su = (int64_t)s_pre[cur.b] + (int64_t)(cur.kvh * p.row_groups + cur.rg) * cur.nt;  // its first tile
    const int c0 = cta_of(su), c1 = cta_of(su + cur.nt - 1);
    float* ws_m = p.ws;
    const int64_t slots = (int64_t)gridDim.x + (int64_t)p.B * units_b;
    float* ws_u = p.ws + slots * 3 * kRows;
    for (int x = threadIdx.x; x < rows * D; x += kThreads) {
      const int row = x / D, d = x % D;
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) v += s_u[(w * kRows + row) * L::kPad + d];
      if (c0 == c1)
        finish_row(v, s_row[2 * kRows + row], s_row[row], s_row[kRows + row], row, d);
      else
        ws_u[((int64_t)(blockIdx.x + u) * kRows + row) * D + d] = v;
    }
    if (c0 != c1) {
      if (threadIdx.x < 3 * kRows) ws_m[(int64_t)(blockIdx.x + u) * 3 * kRows + threadIdx.x] = s_row[threadIdx.x];
      __threadfence();
      __syncthreads();
      if (threadIdx.x == 0) {
        const unsigned arrived = atomicAdd(p.cnt + u, 1u) + 1;
        s_last = arrived == (unsigned)(c1 - c0 + 1);
        if (s_last) p.cnt[u] = 0;
      }
      __syncthreads();
      if (s_last) {
        __threadfence();
        const float* wm = ws_m + (int64_t)(c0 + u) * 3 * kRows;
        const float* wu = ws_u + (int64_t)(c0 + u) * kRows * D;
        const int parts = c1 - c0 + 1;
        float* s_f = s_u;  // [part][row] factors of the parts' u
        for (int row = warp; row < rows; row += kWarps) {
          float m = kNegInf, r = kNegInf, l = 0.f;
          for (int c = lane; c < parts; c += 32) m = fmaxf(m, __ldcg(wm + c * 3 * kRows + row));
#pragma unroll
          for (int off = 16; off >= 1; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
          for (int c = lane; c < parts; c += 32) {
            const float mc = __ldcg(wm + c * 3 * kRows + row);
            const float rc = moved(__ldcg(wm + c * 3 * kRows + kRows + row), mc, m);
            l += __ldcg(wm + c * 3 * kRows + 2 * kRows + row) * (mc == m ? 1.f : fast_exp2(mc - m));
            r = fmaxf(r, rc);
            s_f[c * kRows + row] = rc;
          }
#pragma unroll
          for (int off = 16; off >= 1; off >>= 1) r = fmaxf(r, __shfl_xor_sync(0xffffffffu, r, off));
          for (int c = lane; c < parts; c += 32) {
            const float rc = s_f[c * kRows + row];
            s_f[c * kRows + row] = rc == r ? 1.f : fast_exp2(rc - r);
          }
#pragma unroll
          for (int off = 16; off >= 1; off >>= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
          if (lane == 0) {
            s_row[row] = m;
            s_row[kRows + row] = r;
            s_row[2 * kRows + row] = l;
          }
        }
        __syncthreads();
        for (int x = threadIdx.x; x < rows * D; x += kThreads) {
          const int row = x / D;
          float v = 0.f;
#pragma unroll 8
          for (int c = 0; c < parts; ++c) v = fmaf(__ldcg(wu + (int64_t)c * kRows * D + x), s_f[c * kRows + row], v);
          finish_row(v, s_row[2 * kRows + row], s_row[row], s_row[kRows + row], row, x % D);
        }
      }
    }
    __syncthreads();  // (the next unit writes the same shared memory)
  };

  bool fresh = true;
  for (int s = 0; s < n; ++s) {
    issue_next(L::kStages - 1);
    if (fresh) begin_unit();
    asm volatile("cp.async.wait_group %0;" ::"n"(L::kStages - 1) : "memory");
    const unsigned char* st = ring + (s % L::kStages) * L::kStageBytes;
    const int key0 = key0_of(cur);
    if (key0 < s_end[cur.b]) {
      // ---- scores of 16 keys
      float S[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) S[nt][0] = S[nt][1] = S[nt][2] = S[nt][3] = 0.f;
#pragma unroll
      for (int c = 0; c < KL; ++c) {
        const uint4 x0 = *reinterpret_cast<const uint4*>(st + c * 512 + lane * 16);
        const uint4 x1 = *reinterpret_cast<const uint4*>(st + (KL + c) * 512 + lane * 16);
        const uint32_t w0[4] = {x0.x, x0.y, x0.z, x0.w}, w1[4] = {x1.x, x1.y, x1.z, x1.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t a0 = e4m3x2_to_h2(w0[k] & 0xffffu), a2 = e4m3x2_to_h2(w0[k] >> 16);
          const uint32_t a1 = e4m3x2_to_h2(w1[k] & 0xffffu), a3 = e4m3x2_to_h2(w1[k] >> 16);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma_f16(S[nt], a0, a1, a2, a3, Q[nt][4 * c + k][0], Q[nt][4 * c + k][1]);
        }
      }
      float ks[2], ev[2];
      int page_r[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        ks[r] = scale_of(__shfl_sync(0xffffffffu, sc[0], g + 8 * r));
        const int e = __shfl_sync(0xffffffffu, sc[0], 16 + g + 8 * r);
        ev[r] = e == 255 ? __uint_as_float(0x7fc00000u) : (float)(e - 127);
        page_r[r] = __shfl_sync(0xffffffffu, pg[0], g + 8 * r);
      }
      const bool whole = __all_sync(0xffffffffu, pg[0] >= 0) && key0 + kStep <= min_end && key0 >= max_first &&
                         key0 + kStep <= tree_base;
      bool raise = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int r = k >> 1, c = k & 1;
          float z = S[nt][k] * (ks[r] * fac[nt][c]);
          if (!whole) {
            const int key = key0 + g + 8 * r;
            bool see = page_r[r] >= 0 && key < r_end[nt][c] && key >= r_first[nt][c];
            if (see && key >= tree_base) {
              int h, i;
              out_row(cur.b, cur.kvh, row0 + 8 * nt + 2 * t4 + c, h, i);
              see = (p.tree[cur.b * p.tr_sb + i * p.tr_si] >> (key - tree_base)) & 1;
            }
            z = see ? z : kNegInf;
          }
          S[nt][k] = z;
        }
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          // (no key seen yet: M is -inf, and any score raises it)
          const float m = M[nt][c] == kNegInf ? 0.f : M[nt][c];
          const float z0 = S[nt][c] - m, z1 = S[nt][2 + c] - m;
          raise |= fmaxf(z0, z1) > (M[nt][c] == kNegInf ? kNegInf : kLazyM);
          raise |= fmaxf(z0 + ev[0], z1 + ev[1]) > R[nt][c] + kLazyR;
        }
      }
      if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float zm = fmaxf(S[nt][c], S[nt][2 + c]);
#pragma unroll
            for (int off = 4; off <= 16; off <<= 1) zm = fmaxf(zm, __shfl_xor_sync(0xffffffffu, zm, off));
            const float m = fmaxf(M[nt][c], zm), m0 = m == kNegInf ? 0.f : m;
            ls[nt][c] *= M[nt][c] == m ? 1.f : fast_exp2(M[nt][c] - m);
            float ym = fmaxf(S[nt][c] - m0 + ev[0], S[nt][2 + c] - m0 + ev[1]);
#pragma unroll
            for (int off = 4; off <= 16; off <<= 1) ym = fmaxf(ym, __shfl_xor_sync(0xffffffffu, ym, off));
            const float old = moved(R[nt][c], M[nt][c], m), r = fmaxf(old, ym);
            const float f = old == r ? 1.f : fast_exp2(old - r);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              U[nt][mt][c] *= f;
              U[nt][mt][2 + c] *= f;
            }
            M[nt][c] = m;
            R[nt][c] = r;
          }
      }
      // ---- weights, as the value product's B fragments
      uint32_t hi[NT][2], lo[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int c = k & 1;
          const float z = S[nt][k] - (M[nt][c] == kNegInf ? 0.f : M[nt][c]);
          ls[nt][c] += fast_exp2(z);
          w[k] = fast_exp2(z + (ev[k >> 1] - (R[nt][c] == kNegInf ? 0.f : R[nt][c]) + kLift));
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const uint32_t h2 = pack_h2(w[2 * r], w[2 * r + 1]);
          hi[nt][r] = transposed(h2);
          if constexpr (FINE) {
            const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&h2));
            lo[nt][r] = transposed(pack_h2(w[2 * r] - b.x, w[2 * r + 1] - b.y));
          }
        }
      }
      // ---- values: bytes of two keys side by side, then as f16
      uint32_t v[4][VB / 4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const unsigned char* at = st + 2 * KL * 512 + r * (32 * VB) + lane * VB;
        if constexpr (VB == 16) {
          const uint4 x = *reinterpret_cast<const uint4*>(at);
          v[r][0] = x.x; v[r][1] = x.y; v[r][2] = x.z; v[r][3] = x.w;
        } else {
          const uint2 x = *reinterpret_cast<const uint2*>(at);
          v[r][0] = x.x; v[r][1] = x.y;
        }
      }
#pragma unroll
      for (int q4 = 0; q4 < VB / 4; ++q4) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const uint32_t sel = half ? 0x7362 : 0x5140;
          const uint32_t x = __byte_perm(v[0][q4], v[1][q4], sel), z = __byte_perm(v[2][q4], v[3][q4], sel);
          const uint32_t a0 = e4m3x2_to_h2(x & 0xffffu), a1 = e4m3x2_to_h2(x >> 16);
          const uint32_t a2 = e4m3x2_to_h2(z & 0xffffu), a3 = e4m3x2_to_h2(z >> 16);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma_f16(U[nt][2 * q4 + half], a0, a1, a2, a3, hi[nt][0], hi[nt][1]);
            if constexpr (FINE) mma_f16(U[nt][2 * q4 + half], a0, a1, a2, a3, lo[nt][0], lo[nt][1]);
          }
        }
      }
    }
#pragma unroll
    for (int i = 0; i + 1 < L::kStages; ++i) {
      pg[i] = pg[i + 1];
      sc[i] = sc[i + 1];
    }
    fresh = cur.j + 1 == cur.nt || s + 1 == n;
    if (fresh) end_unit(s);
    next(cur);
  }
}

template <int D, int NT, bool FINE>
cudaError_t launch(const Q8Params& p, int ctas, cudaStream_t stream) {
  using L = Q8Layout<D, NT>;
  static DeviceOnce once;
  if (cudaError_t e = once.set_smem(reinterpret_cast<const void*>(&decode_q8_kernel<D, NT, FINE>),
                                    L::bytes(kDecodeQ8MaxBatch));
      e != cudaSuccess)
    return e;
  decode_q8_kernel<D, NT, FINE><<<ctas, kThreads, L::bytes(p.B), stream>>>(p);
  return cudaGetLastError();
}
template <int D>
cudaError_t launch_d(const Q8Params& p, int ctas, cudaStream_t stream) {
  if (p.rows_cta <= 8) return p.out_bf16 ? launch<D, 1, false>(p, ctas, stream) : launch<D, 1, true>(p, ctas, stream);
  return p.out_bf16 ? launch<D, 2, false>(p, ctas, stream) : launch<D, 2, true>(p, ctas, stream);
}

}  // namespace

Q8Plan plan_decode_q8(int64_t B, int64_t Hkv, int64_t rows, int64_t Tmax, int d, int sms) {
  Q8Plan pl;
  pl.row_groups = (rows + 15) / 16;
  pl.rows_cta = (int)((rows + pl.row_groups - 1) / pl.row_groups);
  const int k = pl.rows_cta <= 8 ? 8 : 16;
  pl.ctas = sms * (k == 8 ? 2 : 1);
  if (pl.ctas > kDecodeQ8MaxCtas) pl.ctas = kDecodeQ8MaxCtas;
  pl.units = B * Hkv * pl.row_groups;
  pl.tiles = pl.units * ((Tmax + kTile - 1) / kTile + 1);
  pl.ws_bytes = (size_t)(pl.ctas + pl.units) * k * (3 + d) * sizeof(float);
  return pl;
}

cudaError_t launch_decode_q8(const Q8Params& p, int d, int ctas, cudaStream_t stream) {
  return d == 128 ? launch_d<128>(p, ctas, stream) : launch_d<64>(p, ctas, stream);
}

}  // namespace blkattn
