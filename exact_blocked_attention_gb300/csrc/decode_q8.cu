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
// Work split: tiles of 256 keys (32 a warp) of all (sequence, KV head, row
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
constexpr int kMostUp = 110;
constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kOwn = 32;               // keys of a warp in a tile: two products of 16, side by side
constexpr int kTile = kOwn * kWarps;

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
  static constexpr int kRows = 8 * NT;
  static constexpr int kHalf = kOwn * D;             // K, then V, of a warp's keys in a tile
  static constexpr int kRing = kWarps * 2 * kHalf;
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
  int* s_start = s_end + p.B;
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
    start = end > 0 ? start : 0;
    s_seen[b] = seen;
    s_tree[b] = p.tree ? len - p.Tq : 0x7fffffff;
    s_end[b] = end;
    s_start[b] = start;
    s_nt[b] = (end - (start & ~(kOwn - 1)) + kTile - 1) / kTile;
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

  // ---- the stream: a tile's page numbers and scales ahead of its rows, those ahead of their use
  unsigned char* ring = sm + warp * (2 * L::kHalf);
  const uint32_t ring_k = smem_u32(ring) + lane * 16, ring_v = smem_u32(ring) + L::kHalf + lane * VB;
  auto key0_of = [&](const Place& a) { return (s_start[a.b] & ~(kOwn - 1)) + a.j * kTile + warp * kOwn; };
  // What lane i knows of the warp's key i in a tile.
  struct Keys {
    int key0;        // of the warp
    uint32_t any;    // lanes whose key some row sees and has a page; the others' rows may hold anything
    uint32_t ko, vo; // offsets of the key's rows in the pools, in 16 bytes
    int ek, ev;      // scale bytes, on their way
  };
  auto look_up = [&](const Place& a, Keys& k) {
    k.key0 = key0_of(a);
    const int key = k.key0 + lane, node = key - s_tree[a.b];
    // (past the end, before the windows, or a tree node that no row lists: not seen)
    const bool seen = key < s_end[a.b] && key >= s_start[a.b] && (node < 0 || ((s_seen[a.b] >> node) & 1));
    const int page = seen ? page_of(p.pages, a.b, key) : -1;
    const int row = key & (p.pages.rows - 1);
    k.ek = k.ev = 127;
    k.ko = k.vo = 0;
    if (page >= 0) {
      const int blk = row >> p.scale_shift;
      k.ek = p.k_sc[(int64_t)page * p.ke_sn + a.kvh * p.ke_sh + blk * p.ke_si];
      k.ev = p.v_sc[(int64_t)page * p.ve_sn + a.kvh * p.ve_sh + blk * p.ve_si];
      k.ko = (uint32_t)page * p.k_sn16 + (uint32_t)row * p.k_sr16;
      k.vo = (uint32_t)page * p.v_sn16 + (uint32_t)row * p.v_sr16;
    }
    k.any = __ballot_sync(0xffffffffu, page >= 0);
  };
  // K rows g + 8 r, 16 t4 bytes in; V rows 8 r + 2 t4 and the next, VB g bytes in
  auto issue_k = [&](const Place& a, const Keys& k) {
    const char* base = p.k + a.kvh * p.k_sh + 16 * t4;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const char* src = base + (uint64_t)__shfl_sync(0xffffffffu, k.ko, g + 8 * r) * 16;
      const int n = k.any == 0xffffffffu || ((k.any >> (g + 8 * r)) & 1) ? 16 : 0;
#pragma unroll
      for (int c = 0; c < KL; ++c) copy16(ring_k + (r * KL + c) * 512, src + 64 * c, n);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  auto issue_v = [&](const Place& a, const Keys& k) {
    const char* base = p.v + a.kvh * p.v_sh + VB * g;
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int key = 8 * r + 2 * t4 + c;
        const char* src = base + (uint64_t)__shfl_sync(0xffffffffu, k.vo, key) * 16;
        const int n = k.any == 0xffffffffu || ((k.any >> key) & 1) ? VB : 0;
        const uint32_t dst = ring_v + (2 * r + c) * (32 * VB);
        if constexpr (VB == 16) copy16(dst, src, n);
        else copy8(dst, src, n);
      }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };

  Place ahead = place_of(t0), cur = ahead;
  const int n = t1 - t0;
  Keys nxt;
  look_up(ahead, nxt);
  issue_k(ahead, nxt);
  issue_v(ahead, nxt);

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
      // the fragments of row 8 nt + g, scaled by a power of two into f16's upper range,
      // but by 2^kMostUp at most: what every bf16 needs to be a number of f16 (2^-133 is
      // 2^-23 then, f16's step 2^-24), and 2^-kMostUp times a scale is a normal float
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
      const int up = min(14 - e, kMostUp);  // (inf and NaN pass through)
      const float f = pow2(up);
#pragma unroll
      for (int c = 0; c < KL; ++c)
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          Q[nt][4 * c + s][0] = pack_h2(x[c][4 * s] * f, x[c][4 * s + 1] * f);
          Q[nt][4 * c + s][1] = pack_h2(x[c][4 * s + 2] * f, x[c][4 * s + 3] * f);
        }
      const float back = p.scale_log2 * pow2(-up);
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
          // (a row that sees nothing takes part in tiles without a mask; what comes of
          // it is dropped)
          if (end > 0) {
            min_end = min(min_end, end);
            max_first = max(max_first, first);
          }
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
          sL[r] = r_end[nt][c] > 0 ? l : 0.f;
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
    if (fresh) begin_unit();
    const Keys now = nxt;
    const bool more = s + 1 < n;
    if (more) {
      next(ahead);
      look_up(ahead, nxt);
    }
    if (now.any == 0) {  // (nothing to see for this warp)
      asm volatile("cp.async.wait_group 0;" ::: "memory");  // (its zeros, before the slots' next rows)
      if (more) {
        issue_k(ahead, nxt);
        issue_v(ahead, nxt);
      }
    } else {
      // ---- scores of two times 16 keys
      float S[2][NT][4];
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) S[x][nt][0] = S[x][nt][1] = S[x][nt][2] = S[x][nt][3] = 0.f;
      asm volatile("cp.async.wait_group 1;" ::: "memory");
#pragma unroll
      for (int c = 0; c < KL; ++c) {
        uint4 w[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) w[r] = *reinterpret_cast<const uint4*>(ring + (r * KL + c) * 512 + lane * 16);
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            uint32_t a0, a1, a2, a3;
            e4m3x4_to_h2((&w[2 * x].x)[k], a0, a2);
            e4m3x4_to_h2((&w[2 * x + 1].x)[k], a1, a3);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma_f16(S[x][nt], a0, a1, a2, a3, Q[nt][4 * c + k][0], Q[nt][4 * c + k][1]);
          }
      }
      // (K's rows are in the products: the next ones may land)
      if (more) issue_k(ahead, nxt);
      else asm volatile("cp.async.commit_group;" ::: "memory");
      const float my_ks = scale_of(now.ek);
      const float my_ev = now.ev == 255 ? __uint_as_float(0x7fc00000u) : (float)(now.ev - 127);
      // (every key seen by every row: no mask)
      const bool whole = now.any == 0xffffffffu && now.key0 + kOwn <= min_end && now.key0 >= max_first &&
                         now.key0 + kOwn <= tree_base;
      float ev[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float ks = __shfl_sync(0xffffffffu, my_ks, 8 * r + g);
        ev[r] = __shfl_sync(0xffffffffu, my_ev, 8 * r + g);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) S[r >> 1][nt][2 * (r & 1) + c] *= ks * fac[nt][c];
      }
      if (!whole) {
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const int key = now.key0 + g + 8 * r;
              bool see = ((now.any >> (8 * r + g)) & 1) && key < r_end[nt][c] && key >= r_first[nt][c];
              if (see && key >= tree_base) {
                int h, i;
                out_row(cur.b, cur.kvh, row0 + 8 * nt + 2 * t4 + c, h, i);
                see = (p.tree[cur.b * p.tr_sb + i * p.tr_si] >> (key - tree_base)) & 1;
              }
              if (!see) S[r >> 1][nt][2 * (r & 1) + c] = kNegInf;
            }
      }
      bool raise = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          // (no key seen yet: M is -inf, and any score raises it)
          const float m = M[nt][c] == kNegInf ? 0.f : M[nt][c];
          const float z0 = S[0][nt][c] - m, z1 = S[0][nt][2 + c] - m, z2 = S[1][nt][c] - m, z3 = S[1][nt][2 + c] - m;
          raise |= fmaxf(fmaxf(z0, z1), fmaxf(z2, z3)) > (M[nt][c] == kNegInf ? kNegInf : kLazyM);
          raise |= fmaxf(fmaxf(z0 + ev[0], z1 + ev[1]), fmaxf(z2 + ev[2], z3 + ev[3])) > R[nt][c] + kLazyR;
        }
      if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float zm = fmaxf(fmaxf(S[0][nt][c], S[0][nt][2 + c]), fmaxf(S[1][nt][c], S[1][nt][2 + c]));
#pragma unroll
            for (int off = 4; off <= 16; off <<= 1) zm = fmaxf(zm, __shfl_xor_sync(0xffffffffu, zm, off));
            const float m = fmaxf(M[nt][c], zm), m0 = m == kNegInf ? 0.f : m;
            ls[nt][c] *= M[nt][c] == m ? 1.f : fast_exp2(M[nt][c] - m);
            float ym = fmaxf(fmaxf(S[0][nt][c] - m0 + ev[0], S[0][nt][2 + c] - m0 + ev[1]),
                             fmaxf(S[1][nt][c] - m0 + ev[2], S[1][nt][2 + c] - m0 + ev[3]));
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
      uint32_t hi[2][NT][2], lo[2][NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float m[2], lift[2];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          m[c] = M[nt][c] == kNegInf ? 0.f : M[nt][c];
          lift[c] = kLift - (R[nt][c] == kNegInf ? 0.f : R[nt][c]);
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          float w[2];
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const float z = S[r >> 1][nt][2 * (r & 1) + c] - m[c];
            ls[nt][c] += fast_exp2(z);
            w[c] = fast_exp2(z + (ev[r] + lift[c]));
          }
          const uint32_t h2 = pack_h2(w[0], w[1]);
          hi[r >> 1][nt][r & 1] = transposed(h2);
          if constexpr (FINE) {
            const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&h2));
            lo[r >> 1][nt][r & 1] = transposed(pack_h2(w[0] - b.x, w[1] - b.y));
          }
        }
      }
      // ---- values: bytes of two keys side by side, then as f16
      asm volatile("cp.async.wait_group 1;" ::: "memory");
      constexpr int kWords = VB / 4;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        uint32_t v[4][kWords];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const unsigned char* at = ring + L::kHalf + (4 * x + r) * (32 * VB) + lane * VB;
          if constexpr (VB == 16) {
            const uint4 y = *reinterpret_cast<const uint4*>(at);
            v[r][0] = y.x; v[r][1] = y.y; v[r][2] = y.z; v[r][3] = y.w;
          } else {
            const uint2 y = *reinterpret_cast<const uint2*>(at);
            v[r][0] = y.x; v[r][1] = y.y;
          }
        }
#pragma unroll
        for (int q4 = 0; q4 < kWords; ++q4)
#pragma unroll
          for (int odd = 0; odd < 2; ++odd) {
            const uint32_t sel = odd ? 0x7362 : 0x5140;
            uint32_t a0, a1, a2, a3;
            e4m3x4_to_h2(__byte_perm(v[0][q4], v[1][q4], sel), a0, a1);
            e4m3x4_to_h2(__byte_perm(v[2][q4], v[3][q4], sel), a2, a3);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              mma_f16(U[nt][2 * q4 + odd], a0, a1, a2, a3, hi[x][nt][0], hi[x][nt][1]);
              if constexpr (FINE) mma_f16(U[nt][2 * q4 + odd], a0, a1, a2, a3, lo[x][nt][0], lo[x][nt][1]);
            }
          }
      }
      if (more) issue_v(ahead, nxt);
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
