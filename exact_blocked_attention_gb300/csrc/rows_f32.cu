// Paged attention of many fp32 query rows per KV head, on the CUDA cores.
//
// Exact blocked attention (Algorithm 33.1, the statistics of eq. 33.3) over a
// cache in pages, for verify and prompt rows in fp32: fp32 products have no
// tensor-core form that keeps their accuracy, so what bounds it is the FMA
// rate, and what it is built for is FMAs from registers.  A CTA (128 threads)
// owns up to 64 query rows that read one KV head and one split of the keys, 32
// at a time:
//
//   S = Q K^T   thread (ty, tx) of 8 x 16: RT rows x 8 keys x D / 4 dims,
//               summed over four threads,
//   U += P V    the same rows x D / 16 dims,
//
// with Q, two stages of K and V (16-byte asynchronous copies a tile ahead) and
// P in shared memory.  A 16-byte read of a warp takes four cycles of the SM's
// one path to registers, whether or not lanes share addresses, so what counts
// is FMAs a read: 32 RT for RT + 8 of them in a step of S (RT rows x 2 keys
// over all dims: 8 RT for RT + 2), RT D / 4 for RT + D / 16 in a step of U.
//
// decode_split.cu, with 8 rows a CTA at most and a key to a lane, re-read K and
// V once per 8 rows and spent its time on the loads.  Measured (there, here;
// the FMAs alone): 7 sequences x 32 heads x 17 rows at 1000 keys 221, 102 us
// (26); 12 x 64 x 8 at 560 keys 151, 75 (24); 512 rows x 32 heads at 2048 keys
// 995, 572 (203); 16 x 7 x 17 at 800 keys 106, 42 (10); d = 64: 122, 84; 83,
// 57; 518, 331; 62, 29.  The busiest SMs issue 72 % of the time, FMAs 57 %; two
// blocks an SM (three to five at d = 64) are what the registers and Q allow.
//
// A row's maximum is taken over the 16 threads that share it, its sum is kept
// per thread until the end.  Splits and partial states are those of
// decode_split.cu (row * n_splits + split, joined by split_merge_kernel).
#include <cuda_bf16.h>

#include "kernels.h"
#include "ptx.cuh"

namespace blkattn {
namespace {

constexpr float kLn2 = 0.6931471805599453f;
constexpr float kNegInf = -__builtin_huge_valf();
constexpr int kThreads = 128;
constexpr int BN = 32;      // keys a tile: one lane looks each one's page up
constexpr int kPRow = BN + 4;

template <int D, int RT>
struct RowsLayout {
  static constexpr int kQRow = D + 4, kKRow = D + 16, kVRow = D;  // floats (the skews spread the banks)
  static constexpr int BM = 8 * RT;
  static constexpr int kStage = BN * (kKRow + kVRow);
  static constexpr int kOffKV = BM * kQRow;          // [stage] K [BN][kKRow], V [BN][kVRow]
  static constexpr int kOffP = kOffKV + 2 * kStage;  // [BM][kPRow]
  static constexpr int kOffInt = kOffP + BM * kPRow;    // end[BM], lo[BM], alive[2]
  static constexpr int kOffTree = (kOffInt + 2 * BM + 2 + 1) / 2 * 2;
  static constexpr int kBytes = (kOffTree + 2 * BM) * 4;
  // blocks an SM that shared memory and registers allow
  static constexpr int kBlocks = D == 128 ? 2 : (RT <= 2 ? 5 : (RT <= 4 ? 4 : 3));
};

template <int D, int RT>
__global__ void __launch_bounds__(kThreads, RowsLayout<D, RT>::kBlocks) rows_f32_kernel(const FwdParams p) {
  using L = RowsLayout<D, RT>;
  constexpr int BM = L::BM, kQRow = L::kQRow, kKRow = L::kKRow, kVRow = L::kVRow, C = D / 4, NV = D / 64;
  extern __shared__ __align__(16) float smem[];
  float* q_s = smem;
  float* p_s = smem + L::kOffP;
  int* end_s = reinterpret_cast<int*>(smem + L::kOffInt);
  int* lo_s = end_s + BM;
  unsigned* alive_s = reinterpret_cast<unsigned*>(lo_s + BM);
  uint64_t* tree_s = reinterpret_cast<uint64_t*>(smem + L::kOffTree);

  const int split = blockIdx.x;
  const int hk = blockIdx.y;
  const int b = blockIdx.z / p.row_groups;
  const int rg = blockIdx.z % p.row_groups;
  const int tid = threadIdx.x, lane = tid & 31;
  const int ty = tid >> 4, tx = tid & 15;
  const int kx = tx >> 2, dq = tx & 3;  // of the scores: keys kx + 4 j, dims 16 c + 4 dq
  const int j0 = kx + 8 * dq;           // the thread's two keys after the sums: j0, j0 + 4
  const int R = p.rows_cta;
  const int pk0 = rg * R;
  const int rows = min(R, p.rows_per_head - pk0);  // real rows of the CTA

  // ---- visibility of the rows ----
  int len = p.seqlens[b * p.sl_s];
  len = len < 0 ? 0 : (len > p.Tmax ? p.Tmax : len);
  const int tbase = p.tree != nullptr ? len - p.Tq : 0x7fffffff;
  if (tid < BM) {
    int e = 0, lo = 0;
    uint64_t tr = ~0ull;
    if (tid < rows) {
      const int i = (pk0 + tid) % p.Tq;
      const int pos = p.qpos[b * p.qp_sb + i * p.qp_si];
      e = pos < 0 ? 0 : (pos >= len ? len : pos + 1);
      if (p.window > 0 && pos >= 0) lo = max(0, pos - p.window + 1);
      if (p.tree != nullptr) tr = (uint64_t)p.tree[(int64_t)b * p.tr_sb + (int64_t)i * p.tr_si];
    }
    end_s[tid] = e;
    lo_s[tid] = lo;
    tree_s[tid] = tr;
  }
  if (tid < 2) alive_s[tid] = 0u;
  auto q_row = [&](int r) {
    const int pk = pk0 + r, g = pk / p.Tq, i = pk - g * p.Tq;
    return static_cast<const float*>(p.q) + ((int64_t)b * p.q_sb + (int64_t)(hk * p.G + g) * p.q_sh + (int64_t)i * p.q_si);
  };
  if (p.q_sd == 1 && (reinterpret_cast<uintptr_t>(p.q) & 15) == 0 && ((p.q_sb | p.q_sh | p.q_si) & 3) == 0) {
    // 16-byte copies, awaited with the first tile's
    for (int idx = tid; idx < BM * C; idx += kThreads) {
      const int r = idx / C, c = idx % C;
      cp_async_16(smem_u32(q_s + r * kQRow + 4 * c), r < rows ? q_row(r) + 4 * c : p.q, r < rows ? 16u : 0u);
    }
  } else {
    for (int idx = tid; idx < BM * D; idx += kThreads) {
      const int r = idx / D, d = idx % D;
      q_s[r * kQRow + d] = r < rows ? q_row(r)[d * p.q_sd] : 0.f;
    }
  }
  __syncthreads();
  int cta_end = 0, min_end = 0x7fffffff, cta_start = 0x7fffffff, max_lo = 0;
  for (int r = lane; r < rows; r += 32) {
    const int e = end_s[r], lo = lo_s[r];
    cta_end = max(cta_end, e);
    min_end = min(min_end, e);
    if (lo < e) cta_start = min(cta_start, lo);
    max_lo = max(max_lo, lo);
  }
  cta_end = __reduce_max_sync(0xffffffffu, cta_end);
  min_end = __reduce_min_sync(0xffffffffu, min_end);
  cta_start = __reduce_min_sync(0xffffffffu, cta_start);
  max_lo = __reduce_max_sync(0xffffffffu, max_lo);

  const int k0 = split * p.chunk;
  // Split 0 always runs: it writes the rows that no split sees.
  if (split > 0 && k0 >= cta_end) return;
  const int k1 = min(k0 + p.chunk, cta_end);
  // first key that is copied: the split's, or the tile of the rows' earliest
  // visible key
  const int f0 = cta_start > k0 ? min(k0 + (cta_start - k0) / BN * BN, k1) : k0;
  const int n_tiles = k1 > f0 ? (k1 - f0 + BN - 1) / BN : 0;

  float m[RT], l[RT], u[RT][4 * NV];
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    m[r] = kNegInf;
    l[r] = 0.f;
#pragma unroll
    for (int e = 0; e < 4 * NV; ++e) u[r][e] = 0.f;
  }

  // copies of tile t, by all threads; page: of the lane's key, looked up a
  // tile before (a key without a page reads zeros and is masked)
  auto look_up = [&](int t) {
    const int key = f0 + t * BN + lane;
    return t < n_tiles && key < k1 ? page_of(p.pages, b, key) : -1;
  };
  const uint32_t kv0 = smem_u32(smem + L::kOffKV);
  auto copy = [&](int t, int page) {
    if (t < n_tiles) {
      const int row = (f0 + t * BN + lane) & (p.pages.rows - 1);
      const char* kr = page < 0 ? nullptr : p.k + (page * p.k_sb + hk * p.k_sh + row * p.k_st);
      const char* vr = page < 0 ? nullptr : p.v + (page * p.v_sb + hk * p.v_sh + row * p.v_st);
      const uint32_t dst = kv0 + (t & 1) * (L::kStage * 4);
#pragma unroll 4
      for (int i = 0; i < BN * C / kThreads; ++i) {
        const int r = (i * kThreads + tid) / C, c = (i * kThreads + tid) % C;  // key and 16-byte chunk
        const char* ks = reinterpret_cast<const char*>(__shfl_sync(0xffffffffu, reinterpret_cast<uintptr_t>(kr), r));
        const char* vs = reinterpret_cast<const char*>(__shfl_sync(0xffffffffu, reinterpret_cast<uintptr_t>(vr), r));
        const uint32_t n = ks != nullptr ? 16u : 0u;  // 0: zeros (the address is not read)
        cp_async_16(dst + (r * kKRow + 4 * c) * 4, n ? ks + c * 16 : p.k, n);
        cp_async_16(dst + (BN * kKRow + r * kVRow + 4 * c) * 4, n ? vs + c * 16 : p.k, n);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    return __ballot_sync(0xffffffffu, page >= 0);
  };
  int page = look_up(0);
  unsigned have_next = copy(0, page);
  page = look_up(1);

  for (int t = 0; t < n_tiles; ++t) {
    const unsigned have = have_next;  // bit j: key j of the tile has a page
    have_next = copy(t + 1, page);    // (its stage was last read before the barrier that ended tile t - 1)
    page = look_up(t + 2);
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    __syncthreads();  // every thread's copies of tile t are in
    const int key0 = f0 + t * BN;
    const float* k_s = smem + L::kOffKV + (t & 1) * L::kStage;
    const float* v_s = k_s + BN * kKRow;

    // ---- scores: a quarter of the dims of 8 keys, then the sums over the four
    // threads that share them, each left with two keys ----
    float s[RT][2];
    {
      float a[RT][8];
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int j = 0; j < 8; ++j) a[r][j] = 0.f;
#pragma unroll 2
      for (int c = 4 * dq; c < D; c += 16) {
        float4 k[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) k[j] = *reinterpret_cast<const float4*>(k_s + (kx + 4 * j) * kKRow + c);
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          const float4 q = *reinterpret_cast<const float4*>(q_s + (ty * RT + r) * kQRow + c);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            a[r][j] = fmaf(q.x, k[j].x, a[r][j]);
            a[r][j] = fmaf(q.y, k[j].y, a[r][j]);
            a[r][j] = fmaf(q.z, k[j].z, a[r][j]);
            a[r][j] = fmaf(q.w, k[j].w, a[r][j]);
          }
        }
      }
      const bool up2 = (dq & 2) != 0, up1 = (dq & 1) != 0;
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        float h[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float send = up2 ? a[r][j] : a[r][j + 4];
          h[j] = (up2 ? a[r][j + 4] : a[r][j]) + __shfl_xor_sync(0xffffffffu, send, 2);
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float send = up1 ? h[j] : h[j + 2];
          s[r][j] = (up1 ? h[j + 2] : h[j]) + __shfl_xor_sync(0xffffffffu, send, 1);
        }
      }
    }

    // ---- mask (by select), block maximum, online statistics ----
    const bool masked = have != 0xffffffffu || key0 + BN > min_end || key0 < max_lo || key0 + BN > tbase ||
                        key0 + BN > k1;
    if (masked) {
      unsigned seen = 0;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int j = j0 + 4 * x, key = key0 + j;
        const bool there = ((have >> j) & 1u) && key < k1;
        bool any = false;
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          const int row = ty * RT + r;
          bool vis = there && key < end_s[row] && key >= lo_s[row];
          if (key >= tbase) {
            const int node = key - tbase;
            vis = vis && node < 64 && ((tree_s[row] >> (node & 63)) & 1ull);
          }
          s[r][x] = vis ? s[r][x] : kNegInf;
          any = any || vis;
        }
        seen |= any ? 1u << j : 0u;
      }
      seen = __reduce_or_sync(0xffffffffu, seen);
      if (lane == 0) atomicOr(&alive_s[t & 1], seen);
    }
    if (tid == 0) alive_s[(t + 1) & 1] = 0u;  // (last read before the barrier that ended tile t - 1)
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      float x0 = s[r][0] == kNegInf ? kNegInf : s[r][0] * p.scale_log2;
      float x1 = s[r][1] == kNegInf ? kNegInf : s[r][1] * p.scale_log2;
      float mt = fmaxf(x0, x1);
#pragma unroll
      for (int off = 8; off >= 1; off >>= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, off));
      // (a NaN score, which no maximum shows beside masked keys, is a weight of
      // NaN: the row is not an empty one)
      float p0 = x0 != x0 ? x0 : 0.f, p1 = x1 != x1 ? x1 : 0.f;
      if (mt != kNegInf) {  // this block has a valid key for the row
        const float m_new = fmaxf(m[r], mt);
        if (m_new != m[r]) {
          const float alpha = m[r] == kNegInf ? 0.f : fast_exp2(m[r] - m_new);
          m[r] = m_new;
          l[r] *= alpha;
#pragma unroll
          for (int e = 0; e < 4 * NV; ++e) u[r][e] *= alpha;
        }
        p0 = fast_exp2(x0 - m_new);  // (masked: 2^-inf = 0)
        p1 = fast_exp2(x1 - m_new);
      }
      l[r] += p0 + p1;
      p_s[(ty * RT + r) * kPRow + j0] = p0;
      p_s[(ty * RT + r) * kPRow + j0 + 4] = p1;
    }
    __syncthreads();

    // ---- U += P V, dims 4 tx + 64 j; keys that no row sees are skipped (rows
    // that were never written may hold anything) ----
    const unsigned alive = masked ? alive_s[t & 1] : 0xffffffffu;
#pragma unroll 2
    for (int c = 0; c < BN; c += 4) {
      float4 w[RT];
#pragma unroll
      for (int r = 0; r < RT; ++r) w[r] = *reinterpret_cast<const float4*>(p_s + (ty * RT + r) * kPRow + c);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (!((alive >> (c + k)) & 1u)) continue;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          const float4 v = *reinterpret_cast<const float4*>(v_s + (c + k) * kVRow + 4 * tx + 64 * j);
#pragma unroll
          for (int r = 0; r < RT; ++r) {
            const float pw = k == 0 ? w[r].x : (k == 1 ? w[r].y : (k == 2 ? w[r].z : w[r].w));
            u[r][4 * j] = fmaf(pw, v.x, u[r][4 * j]);
            u[r][4 * j + 1] = fmaf(pw, v.y, u[r][4 * j + 1]);
            u[r][4 * j + 2] = fmaf(pw, v.z, u[r][4 * j + 2]);
            u[r][4 * j + 3] = fmaf(pw, v.w, u[r][4 * j + 3]);
          }
        }
      }
    }
    __syncthreads();  // P and the stage are free
  }

  // ---- final rows, or this split's partial states ----
#pragma unroll
  for (int r = 0; r < RT; ++r) {
#pragma unroll
    for (int off = 8; off >= 1; off >>= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], off);
    if (l[r] != l[r]) m[r] = l[r];
    const int row = ty * RT + r;
    if (row >= rows) continue;
    const int pk = pk0 + row, g = pk / p.Tq, i = pk - g * p.Tq, h = hk * p.G + g;
    const int n_active = (end_s[row] + p.chunk - 1) / p.chunk;
    if (n_active <= 1) {
      if (split > 0) continue;
      const float inv = m[r] == kNegInf ? 0.f : 1.f / l[r];
      const int64_t o = (int64_t)b * p.o_sb + (int64_t)h * p.o_sh + (int64_t)i * p.o_si;
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int64_t oi = o + (int64_t)(4 * tx + 64 * j + e) * p.o_sd;
          const float y = u[r][4 * j + e] * inv;
          if (p.out_bf16)
            static_cast<__nv_bfloat16*>(p.out)[oi] = __float2bfloat16_rn(y);
          else
            static_cast<float*>(p.out)[oi] = y;
        }
      if (tx == 0)
        p.lse[(int64_t)b * p.l_sb + (int64_t)h * p.l_sh + (int64_t)i * p.l_si] =
            m[r] == kNegInf ? kNegInf : (m[r] + __log2f(l[r])) * kLn2;
    } else if (split < n_active) {
      const int64_t idx = (((int64_t)b * p.Hq + h) * p.Tq + i) * p.n_splits + split;
#pragma unroll
      for (int j = 0; j < NV; ++j)
        *reinterpret_cast<float4*>(p.ws_u + idx * D + 4 * tx + 64 * j) =
            make_float4(u[r][4 * j], u[r][4 * j + 1], u[r][4 * j + 2], u[r][4 * j + 3]);
      if (tx == 0) {
        p.ws_m[idx] = m[r];
        p.ws_l[idx] = l[r];
      }
    }
  }
}

template <int D, int RT>
cudaError_t launch_rt(const FwdParams& p, int n_splits, cudaStream_t stream) {
  constexpr int bytes = RowsLayout<D, RT>::kBytes;
  static DeviceOnce once;
  if (cudaError_t e = once.set_smem(reinterpret_cast<const void*>(&rows_f32_kernel<D, RT>), bytes); e != cudaSuccess)
    return e;
  const dim3 grid((unsigned)n_splits, (unsigned)p.Hkv, (unsigned)(p.B * p.row_groups));
  rows_f32_kernel<D, RT><<<grid, kThreads, bytes, stream>>>(p);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_d(const FwdParams& p, int n_splits, cudaStream_t stream) {
  switch ((p.rows_cta + 7) / 8) {
    case 1: case 2: return launch_rt<D, 2>(p, n_splits, stream);
    case 3: return launch_rt<D, 3>(p, n_splits, stream);
    case 4: return launch_rt<D, 4>(p, n_splits, stream);
    case 5: return launch_rt<D, 5>(p, n_splits, stream);
    case 6: return launch_rt<D, 6>(p, n_splits, stream);
    case 7: case 8: return launch_rt<D, 8>(p, n_splits, stream);
    default: return cudaErrorInvalidValue;
  }
}

template <int D>
size_t smem_d(int rows) {
  switch ((rows + 7) / 8) {
    case 1: case 2: return RowsLayout<D, 2>::kBytes;
    case 3: return RowsLayout<D, 3>::kBytes;
    case 4: return RowsLayout<D, 4>::kBytes;
    case 5: return RowsLayout<D, 5>::kBytes;
    case 6: return RowsLayout<D, 6>::kBytes;
    default: return RowsLayout<D, 8>::kBytes;
  }
}

}  // namespace

size_t rows_f32_smem_bytes(int d, int rows) { return d == 128 ? smem_d<128>(rows) : smem_d<64>(rows); }

cudaError_t launch_rows_f32(const FwdParams& p, int d, int n_splits, cudaStream_t stream) {
  if (d == 128) return launch_d<128>(p, n_splits, stream);
  if (d == 64) return launch_d<64>(p, n_splits, stream);
  return cudaErrorInvalidValue;
}

}  // namespace blkattn
