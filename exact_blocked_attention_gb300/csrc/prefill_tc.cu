// Causal prefill kernel on the 5th-generation tensor cores (tcgen05 + TMEM).
//
// Exact blocked attention ("Chapter 33: inference compute optimisation"
// §33.2, Algorithm 33.1; §33.3 for the on-chip tiling and the skipping of
// fully invisible blocks): a CTA owns TWO query tiles of 128 consecutive rows
// of one head (rows [i0, i0 + 256)) and walks the key tiles of 128 keys that
// hold any key visible to them, keeping per row the statistics (m, l, u) of
// eq. 33.3 with u in tensor memory.  Both query tiles share every K/V tile
// the CTA loads; key tiles beyond the CTA's last visible key are never loaded.
//
//   S_j  = Q K_j^T     tcgen05.mma M=128 N=128 K=16 x 8      (smem x smem -> TMEM)
//   U   += P_j V_j     tcgen05.mma M=128 N=128 K=16 x 8 (x 2 on split tiles; P from TMEM, V smem)
//
// Roles (320 threads): warps 0-3 and 4-7 = one thread per query row of the
// first / second query tile (a TMEM lane each): scores, mask by select,
// online statistics, P; warp 8 = TMA producer (both Q tiles once, K and V
// tiles into 2-stage rings released separately; over pages warps 8 and 10, see
// the kernel); warp 9 = TMEM allocation
// and the single thread that issues every MMA.  Each query tile has one S
// buffer in TMEM and P_j is written over it.  On a key tile that some row of
// the query tile does not see in full (the diagonal, a window's leading
// edge: where the rows with few keys get most of their weight) P_j goes in
// as bf16 P_hi and P_lo (P = P_hi + P_lo to ~16 bits, two PV products, ~2^-17
// relative accuracy although P is not an input); on the other tiles as one
// bf16 P rounded to nearest, with l summing the rounded values so that u / l
// stays a convex combination of the values (rows that see those tiles see
// at least 128 keys in each, and the rounding errors average out: measured
// well inside the output bar).  The MMA thread tells the two kinds of tile
// apart by the same rule as the rows.  S_{j+1} is issued right after U +=
// P_j V_j (products execute in issue order).  The two query tiles ping-pong: while
// one tile's rows compute P, the tensor core runs the other tile's products.
// Each tile's chain S_j -> P_j -> products -> S_{j+1} passes through the
// MMA thread, so its issue path is kept short: shared-memory descriptors are
// formed once per operand buffer and only their address word moves.
// The epilogue (o = u / l) stages fp32 rows in the freed K / V ring and
// stores them with tiled TMA when the output layout allows it.
//
// Online rescaling is lazy: a row keeps its reference maximum m until a tile
// raises the row maximum by more than 8 (base-2 units); only then is its U
// row rescaled in TMEM.  S_j ready implies U += P_{j-1} V_{j-1} completed, so
// the rescale needs no extra wait.  With any reference m >= (true max - 8)
// the state (m, l, u) still represents the same set (eqs. 33.4-33.5 hold for
// any common reference), and P <= 2^8.
//
// With a sliding window ("Chapter 33" §33.7, the paragraph of eq. 33.16;
// the WIN instantiation) a row at position pos sees keys pos - W < j <= pos:
// each query tile gets a first key tile (its rows' earliest visible key), the
// CTA loads from the smaller of the two, and the leading tiles are masked per
// row.  The unwindowed instantiation is unchanged by this.
//
// Rows with no visible key keep the empty state and get out = 0,
// lse = -inf.  V rows of the last tile past the CTA's last visible key (cache
// padding, possibly NaN) are zero-filled in shared memory before the PV
// product so that 0 * garbage never reaches U.
#include <cuda_bf16.h>

#include "kernels.h"
#include "paged_tma.cuh"
#include "ptx.cuh"
#include "tc.cuh"

namespace blkattn {
namespace {

constexpr float kLn2 = 0.6931471805599453f;
constexpr float kNegInf = -__builtin_huge_valf();
constexpr float kLazyRescale = 8.f;  // base-2 units: rescale only when max grows by > 2^8

constexpr int BM = 128;  // query rows per query tile (TMEM lanes)
constexpr int QT = 2;    // query tiles per CTA
constexpr int BN = 128;  // keys per tile
constexpr int kBox = 128 * 128;       // one 64-dim (128-byte) box of 128 rows: 16 KB
// Head dims 128 and (over pages) 64: with 64 the tiles are half the size and
// the ring has twice the stages.
template <int D>
struct Layout {
  static constexpr int kBoxes = D / 64;
  static constexpr int kTileBytes = kBoxes * kBox;  // one Q, K or V tile of 128 rows
  static constexpr int kStages = 2 * (2 / kBoxes);
  static constexpr int kOffQ = 0;
  static constexpr int kOffK = kOffQ + QT * kTileBytes;
  static constexpr int kOffV = kOffK + kStages * kTileBytes;
  static constexpr int kOffBar = kOffV + kStages * kTileBytes;
  // q_full, k_full[S], v_full[S], k_empty[S], v_empty[S], s_full[QT], p_full[QT], drain
  static constexpr int kNumBars = 1 + 4 * kStages + QT + QT + 1;
  static constexpr int kOffMisc = kOffBar + kNumBars * 8;
  static constexpr int kSmemBytes = kOffMisc + 64 + 1024;  // + slack to align to 1024
};
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kTileCols = 256;  // per query tile: S / P at [0, 128), U at [128, 256)
constexpr uint32_t kColS = 0;
constexpr uint32_t kColPlo = 64;     // P_hi at [0, 64), P_lo at [64, 128) (bf16 pairs)
constexpr uint32_t kColO = 128;
constexpr int kTmaWarp = 8;
constexpr int kMmaWarp = 9;
constexpr int kPageVWarp = 10;  // PAGED: V tiles (kTmaWarp: K tiles)
template <bool PAGED>
constexpr int kThreads = 32 * (PAGED ? 11 : 10);
constexpr uint32_t kIdescQK = tc::idesc_bf16(BM, BN, 0, 0);  // Q, K both K-major
template <int D>
constexpr uint32_t kIdescPV = tc::idesc_bf16(BM, D, 0, 1);   // P (TMEM), V MN-major

__device__ __forceinline__ uint64_t policy_evict_last() {
  uint64_t pol;
  asm volatile("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(pol));
  return pol;
}

// a += the two bf16 of w (low half first), exactly widened by the addition.
__device__ __forceinline__ void add_bf16x2(float2& a, uint32_t w) {
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "mov.b32 {lo, hi}, %2;\n\t"
      "add.f32.bf16 %0, lo, %0;\n\t"
      "add.f32.bf16 %1, hi, %1;\n\t}"
      : "+f"(a.x), "+f"(a.y)
      : "r"(w));
}

// The first key tile of a CTA whose first row is at position q0 under a
// sliding window (rows at their own index, the prefill layout).
__device__ __forceinline__ int spec_first_tile(int q0, int window) {
  const int64_t s0 = (int64_t)q0 - (int64_t)window + 1;
  return s0 > 0 ? (int)(s0 / BN) : 0;
}

// Query-tile pair and (sequence, head) of item r of the dispatch order: groups
// of head_group (sequence, head) pairs whose K/V fit in L2 together; within a
// group every head's longest (latest) query-tile pair goes before any shorter
// one.  The next group's long pairs start while the previous group's short
// ones finish.  (Over pages the last group is as small as it is; over a
// contiguous cache it is padded.)
template <bool PAGED>
__device__ __forceinline__ void item_of(const FwdParams& p, int r, int n_pairs, int& pair, int& bh) {
  const int hg = p.head_group;
  const int per_group = n_pairs * hg;
  const int group = r / per_group;
  const int r_in = r % per_group;
  const int heads = PAGED ? min(hg, p.Hq * p.B - group * hg) : hg;
  pair = n_pairs - 1 - r_in / heads;
  bh = group * hg + r_in % heads;
}

// PAGED: the cache lies in pages (paged.h).  A key tile is one box of a page of
// at least 128 rows or the boxes of 128 / P pages: the lanes of two producer
// warps (K, V) look their pages up a tile ahead and issue the copies, with
// packed rows of 128 dims both halves in one box (WIDE), as in the decode
// kernel: a copy takes its warp some 50 ns to issue, and one warp with a box a
// half took 576 us for the case below in pages of 8, 398 in pages of 16, 355
// in pages of 128; two 359 in any (with one sum of the weights; 371 to 377 with
// both, below).  A page number outside the pool goes to the
// copy as -1 (zeros) and the rows mask its keys, in tensor memory (a mask in
// registers spilled 576 bytes).  The chain of a key tile bounds it as over a
// contiguous cache: 2 x 2048 rows of 32 heads at 8192 keys 371 us on the device
// (1300 TFLOP/s, 66 % of the bf16 burst rate; 384 a call among others),
// contiguous 385.
// At d = 64 the chain's products are half as long: 1.1 us a key tile for one
// query tile, 1.36 for two (d = 128: 1.4 and 1.6); 1024 rows of 32 heads at
// 2048 keys 35 us, 102 with the decode kernel.
template <int D, bool WIN, bool PAGED, bool WIDE>
__global__ void __launch_bounds__(kThreads<PAGED>, 1)
    prefill_tc_kernel(const FwdParams p, const __grid_constant__ CUtensorMap tmq,
                      const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv,
                      const __grid_constant__ CUtensorMap tmo) {
  using L = Layout<D>;
  constexpr int STAGES = L::kStages, kTileBytes = L::kTileBytes, kBoxes = L::kBoxes;
  constexpr int kOffQ = L::kOffQ, kOffK = L::kOffK, kOffV = L::kOffV, kOffBar = L::kOffBar, kOffMisc = L::kOffMisc;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* sm = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + kOffBar);
  uint64_t* q_full = bars;
  uint64_t* k_full = q_full + 1;
  uint64_t* v_full = k_full + STAGES;
  uint64_t* k_empty = v_full + STAGES;
  uint64_t* v_empty = k_empty + STAGES;
  uint64_t* s_full = v_empty + STAGES;  // [QT]
  uint64_t* p_full = s_full + QT;       // [QT]
  uint64_t* drain = p_full + QT;
  // misc: [0] tmem base, [1 + 2x] end of query tile x, [2 + 2x] min end of x, [5] timeout,
  // (sliding window) [6 + 2x] smallest and [7 + 2x] largest first visible key of x's rows
  int* misc = reinterpret_cast<int*>(sm + kOffMisc);

  // Linear grid in dispatch order; over pages the items from split_from on
  // have `parts` CTAs each
  const int n_pairs = (p.Tq + 2 * BM - 1) / (2 * BM);
  int item = blockIdx.x, part = 0, parts = 1;
  if (PAGED && item >= p.split_from) {
    const int e = item - p.split_from;
    parts = p.n_splits;
    item = p.split_from + e / parts;
    part = e % parts;
  }
  // (the joining kernel's blocks may take their places as soon as every CTA
  // runs; they wait for this kernel's end)
  if (PAGED && p.n_splits > 1) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  int pair, bh;
  item_of<PAGED>(p, item, n_pairs, pair, bh);
  if (!PAGED && bh >= p.Hq * p.B) return;  // padding of the last group
  const int h = bh % p.Hq;
  const int b = bh / p.Hq;
  const int hk = h / p.G;
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int x = warp >> 2;  // query tile of a row warp (0 or 1)
  const int i0 = (2 * pair + (warp < 8 ? x : 0)) * BM;

  const uint64_t pol_q = policy_evict_first();
  const uint64_t pol_kv = policy_evict_last();  // K/V tiles are re-read by the other query tiles
  // Barriers and tensor memory first: the producer then starts both Q tiles
  // and the first K/V tile (always inside the cache, T_max >= 1) while the
  // rows read their positions.
  if (threadIdx.x == 0) {
    misc[1] = 0; misc[2] = 0x7fffffff;
    misc[3] = 0; misc[4] = 0x7fffffff;
    misc[5] = 0;
    misc[6] = 0x7fffffff; misc[7] = 0;
    misc[8] = 0x7fffffff; misc[9] = 0;
    mbar_init(q_full, 1);
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&k_full[s], 1);
      mbar_init(&v_full[s], 1);
      mbar_init(&k_empty[s], 1);
      mbar_init(&v_empty[s], 1);
    }
    for (int t = 0; t < QT; ++t) {
      mbar_init(&s_full[t], 1);
      mbar_init(&p_full[t], 4);  // one arrival per row warp of the query tile
    }
    mbar_init(drain, 1);
    fence_barrier_init();
  }
  if (warp == kMmaWarp) {
    tc::alloc(reinterpret_cast<uint32_t*>(&misc[0]), kTmemCols);
    tc::relinquish();
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (warp == kTmaWarp && lane == 0) {
    const int q0 = 2 * pair * BM;
    mbar_arrive_expect_tx(q_full, QT * kTileBytes);
    for (int t = 0; t < QT; ++t) {
      tma_load_4d(sm + kOffQ + t * kTileBytes, &tmq, 0, q0 + t * BM, h, b, q_full, pol_q);
      if (kBoxes == 2) tma_load_4d(sm + kOffQ + t * kTileBytes + kBox, &tmq, 64, q0 + t * BM, h, b, q_full, pol_q);
    }
    if (!PAGED) {
    // K/V tile 0 of the CTA's range right away; with a window the range
    // starts at the key tile of the CTA's earliest visible key, known only
    // from the positions, so the copy goes to the tile that rows at positions
    // q0 + r would start at (ring position 0; if the positions say otherwise,
    // the CTA's tiles start at ring position 1 and this copy is dropped)
    const int key_first = WIN ? spec_first_tile(2 * pair * BM, p.window) * BN : 0;
    mbar_arrive_expect_tx(&k_full[0], kTileBytes);
    tma_load_4d(sm + kOffK, &tmk, 0, key_first, hk, b, &k_full[0], pol_kv);
    tma_load_4d(sm + kOffK + kBox, &tmk, 64, key_first, hk, b, &k_full[0], pol_kv);
    mbar_arrive_expect_tx(&v_full[0], kTileBytes);
    tma_load_4d(sm + kOffV, &tmv, 0, key_first, hk, b, &v_full[0], pol_kv);
    tma_load_4d(sm + kOffV + kBox, &tmv, 64, key_first, hk, b, &v_full[0], pol_kv);
    }
  }

  // ---- visibility of the rows (integers) ----
  int len = p.seqlens[b * p.sl_s];
  len = len < 0 ? 0 : (len > p.Tmax ? p.Tmax : len);
  int my_end = 0, my_start = 0;
  bool my_row = false;
  const int row_i = i0 + (int)(threadIdx.x & 127);
  if (warp < 8 && row_i < p.Tq) {
    const int pos = p.qpos[b * p.qp_sb + row_i * p.qp_si];
    my_end = pos < 0 ? 0 : (pos >= len ? len : pos + 1);
    my_row = true;
    if constexpr (WIN) {
      // sliding window: keys pos - W < j <= pos (pos >= 0 first: no overflow)
      my_start = pos < 0 ? 0 : max(0, pos - p.window + 1);
      if (my_end > my_start) {
        atomicMin(&misc[6 + 2 * x], my_start);
        atomicMax(&misc[7 + 2 * x], my_start);
      } else {
        // a window that starts at or past the cache length holds no key: the
        // row is masked by its end on every tile, like a row at pos < 0
        my_end = 0;
      }
    }
    atomicMax(&misc[1 + 2 * x], my_end);
    // (over pages rows without keys are masked by their own warp, below, and
    // do not make every key tile a partly visible one: a chunk of 2 x 1335
    // rows, three of them padding, x 7 heads at 2908 keys 73 us, 48 with this; 51 with both sums of the
    // weights)
    if (!PAGED || my_end > 0) atomicMin(&misc[2 + 2 * x], my_end);
  }
  __syncthreads();
  // key tiles [f_x, e_x) of query tile x (f_x = 0 without a window), and the
  // CTA's range [j_lo, j_hi) over the query tiles that see any key; ring
  // slots and phases count from j_lo
  int e_t0 = (misc[1] + BN - 1) / BN;
  int e_t1 = (misc[3] + BN - 1) / BN;
  int f_t0 = 0, f_t1 = 0;
  if constexpr (WIN) {
    f_t0 = misc[6] == 0x7fffffff ? e_t0 : misc[6] / BN;
    f_t1 = misc[8] == 0x7fffffff ? e_t1 : misc[8] / BN;
    if (f_t0 >= e_t0) f_t0 = e_t0 = 0;  // no row of the tile sees a key
    if (f_t1 >= e_t1) f_t1 = e_t1 = 0;
  }
  if (PAGED && parts > 1) {
    // this CTA's share of the key tiles
    const int lo0 = !WIN ? 0 : (e_t0 == f_t0 ? f_t1 : (e_t1 == f_t1 ? f_t0 : min(f_t0, f_t1)));
    const int n = max(e_t0, e_t1) - lo0;
    const int lo = lo0 + n * part / parts, hi = lo0 + n * (part + 1) / parts;
    f_t0 = max(f_t0, lo);
    f_t1 = max(f_t1, lo);
    e_t0 = min(e_t0, hi);
    e_t1 = min(e_t1, hi);
    if (f_t0 >= e_t0) f_t0 = e_t0 = 0;
    if (f_t1 >= e_t1) f_t1 = e_t1 = 0;
  }
  const int n_t0 = e_t0 - f_t0;  // key tiles per query tile
  const int n_t1 = e_t1 - f_t1;
  const int j_lo = !WIN && !PAGED ? 0 : (n_t0 == 0 ? f_t1 : (n_t1 == 0 ? f_t0 : min(f_t0, f_t1)));
  const int j_hi = max(e_t0, e_t1);
  const int n_max = j_hi - j_lo;  // key tiles the CTA loads
  // ring position of the CTA's key tile j: j + ro (ro = 1 when the copy made
  // before the positions were read holds another tile)
  const int ro = (WIN && !PAGED && j_lo != spec_first_tile(2 * pair * BM, p.window)) ? 1 : 0;
  // paged cache: the CTA's earliest visible key (V rows before it are zeroed)
  const int cta_start = WIN && PAGED ? min(n_t0 > 0 ? misc[6] : 0x7fffffff, n_t1 > 0 ? misc[8] : 0x7fffffff) : 0;
  const int cta_end = max(n_t0 > 0 ? misc[1] : 0, n_t1 > 0 ? misc[3] : 0);
  const int64_t out_row = (int64_t)b * p.o_sb + (int64_t)h * p.o_sh + (int64_t)row_i * p.o_si;
  const int64_t lse_idx = (int64_t)b * p.l_sb + (int64_t)h * p.l_sh + (int64_t)row_i * p.l_si;

  // partial states of a split item: row of the slot in ws_m, ws_l, ws_u
  const int64_t ws_row = PAGED ? ((int64_t)(item - p.split_from) * parts + part) * (QT * BM) : 0;

  auto write_empty_row = [&]() {  // the defined output of a row with no visible key
    if (PAGED && parts > 1) {
      p.ws_m[ws_row + threadIdx.x] = kNegInf;
      return;
    }
    for (int d = 0; d < D; ++d) {
      if (p.out_bf16)
        static_cast<__nv_bfloat16*>(p.out)[out_row + (int64_t)d * p.o_sd] = __float2bfloat16_rn(0.f);
      else
        static_cast<float*>(p.out)[out_row + (int64_t)d * p.o_sd] = 0.f;
    }
    p.lse[lse_idx] = kNegInf;
  };
  const uint32_t tb = static_cast<uint32_t>(misc[0]);
  const uint32_t sQ = smem_u32(sm + kOffQ);
  const uint32_t sK = smem_u32(sm + kOffK);
  const uint32_t sV = smem_u32(sm + kOffV);

  if (n_max == 0) {
    // no row of the CTA sees a key: the defined empty output; the first
    // copies must still land before the CTA exits
    if (my_row) write_empty_row();
    if (warp == kTmaWarp && lane == 0) {
      bool landed = mbar_wait(q_full, 0);
      if (!PAGED) {
        landed = mbar_wait(&k_full[0], 0) && landed;
        landed = mbar_wait(&v_full[0], 0) && landed;
      }
      if (!landed) record_error(p.err, kErrTimeout);
    }
  } else if (PAGED && (warp == kTmaWarp || warp == kPageVWarp)) {
    // ---------------- TMA producers, pages (whole warps, one for K, one for V) ----------------
    const bool kv = warp == kPageVWarp;
    const void* map = kv ? static_cast<const void*>(&tmv) : static_cast<const void*>(&tmk);
    uint64_t* full = kv ? v_full : k_full;
    uint64_t* empty = kv ? v_empty : k_empty;
    const int box_shift = min(p.pages.shift, 7);
    const int n_pieces = BN >> box_shift;
    const int piece = lane & (n_pieces - 1);  // of the tile's keys
    const int half = lane >> (7 - box_shift);  // 64-dim box
    const bool copies = half < (WIDE ? 1 : kBoxes);
    const uint32_t dst_off = (kv ? kOffV : kOffK) + (WIDE ? (uint32_t)((piece << box_shift) * 256)
                                                          : (uint32_t)(half * kBox + (piece << box_shift) * 128));
    auto look_up = [&](int j) {  // this lane's page of key tile j: -1 (zeros) past the rows' ends
      const int key = (j_lo + j) * BN + (piece << box_shift);
      return j < n_max && key < cta_end ? page_of(p.pages, b, key) : -1;
    };
    int issued = 0;  // ring positions
    bool ok = true;
    int page = look_up(0);
    for (int j = 0; j < n_max && ok; ++j) {
      const int s = j % STAGES;
      const int row = ((j_lo + j) * BN + (piece << box_shift)) & (p.pages.rows - 1);
      const int page_next = look_up(j + 1);  // (the load is in flight meanwhile)
      bool w = true;
      if (lane == 0) {
        if (j >= STAGES) w = mbar_wait(&empty[s], ((j / STAGES) - 1) & 1);
        if (w) mbar_arrive_expect_tx(&full[s], kTileBytes);
      }
      ok = __shfl_sync(0xffffffffu, w, 0);  // (also orders the expected bytes before the copies)
      if (!ok) break;
      __syncwarp();
      if (copies) {
        unsigned char* dst = sm + s * kTileBytes + dst_off;
        if (WIDE)
          tma_load_5d(dst, map, 0, 0, hk * p.pages.wide_h2, (row >> 3) + hk * p.pages.wide_h3, page, &full[s], pol_kv);
        else
          tma_load_4d(dst, map, 64 * half, row, hk, page, &full[s], pol_kv);
      }
      issued = j + 1;
      page = page_next;
    }
    __syncwarp();
    if (lane == 0) {
      // every issued copy must land before the CTA can exit
      if (!kv && !mbar_wait(q_full, 0)) ok = false;
      for (int j = issued - STAGES < 0 ? 0 : issued - STAGES; j < issued; ++j)
        if (!mbar_wait(&full[j % STAGES], (j / STAGES) & 1)) ok = false;
      if (!ok) {
        record_error(p.err, kErrTimeout);
        misc[5] = 1;
      }
    }
  } else if (warp == kTmaWarp) {
    // ---------------- TMA producer ----------------
    if (lane == 0) {
      // Q and ring position 0 are in flight already; positions issued so far
      int k_issued = 1, v_issued = 1;
      bool ok = true;
      if (ro == 1) {
        // position 0 holds another tile: it lands, then its slot is released
        ok = mbar_wait(&k_full[0], 0) && mbar_wait(&v_full[0], 0);
        mbar_arrive(&k_empty[0]);
        mbar_arrive(&v_empty[0]);
      }
      for (int j = 1 - ro; j < n_max && ok; ++j) {
        const int u = j + ro;
        const int s = u % STAGES;
        const int key0 = (j_lo + j) * BN;
        if (u >= STAGES && !mbar_wait(&k_empty[s], ((u / STAGES) - 1) & 1)) { ok = false; break; }
        unsigned char* kd = sm + kOffK + s * kTileBytes;
        mbar_arrive_expect_tx(&k_full[s], kTileBytes);
        tma_load_4d(kd, &tmk, 0, key0, hk, b, &k_full[s], pol_kv);
        tma_load_4d(kd + kBox, &tmk, 64, key0, hk, b, &k_full[s], pol_kv);
        k_issued = u + 1;
        if (u >= STAGES && !mbar_wait(&v_empty[s], ((u / STAGES) - 1) & 1)) { ok = false; break; }
        unsigned char* vd = sm + kOffV + s * kTileBytes;
        mbar_arrive_expect_tx(&v_full[s], kTileBytes);
        tma_load_4d(vd, &tmv, 0, key0, hk, b, &v_full[s], pol_kv);
        tma_load_4d(vd + kBox, &tmv, 64, key0, hk, b, &v_full[s], pol_kv);
        v_issued = u + 1;
      }
      // every issued copy must land before the CTA can exit
      if (!mbar_wait(q_full, 0)) ok = false;
      for (int j = k_issued - STAGES < 0 ? 0 : k_issued - STAGES; j < k_issued; ++j)
        if (!mbar_wait(&k_full[j % STAGES], (j / STAGES) & 1)) ok = false;
      for (int j = v_issued - STAGES < 0 ? 0 : v_issued - STAGES; j < v_issued; ++j)
        if (!mbar_wait(&v_full[j % STAGES], (j / STAGES) & 1)) ok = false;
      if (!ok) {
        record_error(p.err, kErrTimeout);
        misc[5] = 1;
      }
    }
  } else if (warp == kMmaWarp) {
    // ---------------- MMA issue (one thread) ----------------
    if (lane == 0) {
      bool ok = mbar_wait(q_full, 0);
      // K and V tiles: 64-dim boxes 16 KB apart, rows 128 bytes apart; a page's
      // wide box instead has the two halves of 8 rows side by side (8-row
      // groups 2 KB apart, the second half 1 KB behind the first)
      constexpr uint32_t kHi = tc::desc_hi(1024);
      constexpr uint32_t kHiKV = WIDE ? tc::desc_hi(2048) : kHi;
      constexpr uint32_t kHalf = WIDE ? 1024u : (uint32_t)kBox;
      // S_jj = Q_t K_jj^T into query tile t's S buffer
      auto issue_qk = [&](int t, int jj) {
        // descriptors: only the start address moves (split-word form)
        const uint32_t klo = tc::desc_lo(sK + ((jj + ro) % STAGES) * kTileBytes, 16);
        const uint32_t qlo = tc::desc_lo(sQ + t * kTileBytes, 16);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const uint64_t adesc = tc::desc_join(qlo + (uint32_t)(((ks >> 2) * kBox + (ks & 3) * 32) >> 4), kHi);
          const uint64_t bdesc = tc::desc_join(klo + (((uint32_t)(ks >> 2) * kHalf + (ks & 3) * 32) >> 4), kHiKV);
          tc::mma_ss(tb + t * kTileCols + kColS, adesc, bdesc, kIdescQK, ks > 0 ? 1u : 0u);
        }
        tc::commit(&s_full[t]);
      };
      // U_t += P_jj V_jj (P_hi, then P_lo on the tiles that split P);
      // `more`: U_t already holds a tile
      const int min_end[QT] = {misc[2], misc[4]};
      const int win_max[QT] = {WIN ? misc[7] : 0, WIN ? misc[9] : 0};
      auto issue_pv = [&](int t, int jj, bool more) {
        const uint32_t vlo = tc::desc_lo(sV + ((jj + ro) % STAGES) * kTileBytes, kHalf);
        const uint32_t tcol = tb + t * kTileCols;
        const int k0 = (j_lo + jj) * BN;
        const bool split = k0 + BN > min_end[t] || (WIN && k0 < win_max[t]);
#pragma unroll
        for (int part = 0; part < 2; ++part) {
          if (part == 1 && !split) break;
#pragma unroll
          for (int ks = 0; ks < BN / 16; ++ks) {
            // B = V rows [16ks, 16ks+16) (keys, K) x 128 dims (N, two 64-dim boxes 16 KB apart)
            const uint64_t bdesc = tc::desc_join(vlo + (uint32_t)(ks * (WIDE ? 4096 : 2048) >> 4), kHiKV);
            const uint32_t acol = tcol + kColS + part * kColPlo + 8 * ks;
            tc::mma_ts(tcol + kColO, acol, bdesc, kIdescPV<D>, (more || part > 0 || ks > 0) ? 1u : 0u);
          }
        }
      };
      // (j counts the CTA's key tiles from j_lo; query tile t covers
      // [a_t, a_t + n_t) of them, a_t = 0 without a window)
      const int a_t0 = f_t0 - j_lo, a_t1 = f_t1 - j_lo;
      // prologue: the first scores of the query tiles that start at j_lo
      if (ok && !mbar_wait(&k_full[ro], 0)) ok = false;  // ring position ro < STAGES: phase 0
      if (ok) {
        tc::fence_after();
        if (n_t0 > 0 && a_t0 == 0) issue_qk(0, 0);
        if (n_t1 > 0 && a_t1 == 0) issue_qk(1, 0);
        tc::commit(&k_empty[ro]);
      }
      for (int j = 0; ok && j < n_max; ++j) {
        const int u = j + ro;  // ring position
        const int s = u % STAGES;
        const bool next = j + 1 < n_max;
        if (!mbar_wait(&v_full[s], (u / STAGES) & 1)) { ok = false; break; }
        if (next && !mbar_wait(&k_full[(u + 1) % STAGES], ((u + 1) / STAGES) & 1)) { ok = false; break; }
        for (int t = 0; t < QT && ok; ++t) {
          const int nt = t == 0 ? n_t0 : n_t1;
          const int at = t == 0 ? a_t0 : a_t1;
          if (j < at || j >= at + nt) {
            // a query tile whose range starts at the next key tile: its first scores
            if (WIN && nt > 0 && j + 1 == at) issue_qk(t, j + 1);
            continue;
          }
          // U += P_j V_j as soon as this query tile's P_j is ready, then
          // S_{j+1} into the same TMEM columns (issue order = execution order)
          if (!mbar_wait(&p_full[t], (j - at) & 1)) { ok = false; break; }
          tc::fence_after();
          issue_pv(t, j, j > at);
          if (j + 1 < at + nt) issue_qk(t, j + 1);
        }
        if (!ok) break;
        tc::commit(&v_empty[s]);                           // V_j free once these products complete
        if (next) tc::commit(&k_empty[(u + 1) % STAGES]);  // K_{j+1} likewise
      }
      if (!ok) {
        record_error(p.err, kErrTimeout);
        misc[5] = 1;
      }
      // every MMA issued must complete before TMEM is released
      tc::commit(drain);
      if (!mbar_wait(drain, 0)) {
        record_error(p.err, kErrTimeout);
        misc[5] = 1;
      }
    }
  } else {
    // ---------------- rows: online softmax statistics (query tile x) ----------------
    const int n_mine = x == 0 ? n_t0 : n_t1;
    const int my_min = misc[2 + 2 * x];
    // key tiles that reach past this are masked by select
    const int mask_min = PAGED ? (int)__reduce_min_sync(0xffffffffu, my_row ? my_end : 0x7fffffff) : my_min;
    const int f_mine = x == 0 ? f_t0 : f_t1;            // first key tile (0 without a window)
    const int win_max = WIN ? misc[7 + 2 * x] : 0;     // keys below it are masked for some row
    // a key tile some row of the query tile does not see in full (the
    // diagonal, a window's leading edge): P goes to the product as P_hi +
    // P_lo (the few-key rows live here); elsewhere as one bf16 P
    auto split_tile = [&](int k0) { return k0 + BN > my_min || (WIN && k0 < win_max); };
    if (n_mine == 0) {
      if (my_row) write_empty_row();
    } else {
      const uint32_t tl = tb + x * kTileCols + ((uint32_t)(32 * (warp & 3)) << 16);  // lane quarter
      float m_ref = kNegInf;  // reference maximum (base-2 units), -inf = no valid key yet
      float l = 0.f;
      float lx = 0.f;  // PAGED: the sum of the weights before any rounding, for lse
      bool ok = true;
      // waits are made warp-uniform: the tensor-memory accesses that follow
      // are warp-collective
      auto wait_all = [&](uint64_t* bar, uint32_t parity) -> bool {
        return __all_sync(0xffffffffu, mbar_wait(bar, parity));
      };
      for (int j = 0; j < n_mine; ++j) {
        // paged cache: bit i: piece i of this key tile has no page (looked up
        // before the wait: the load is in flight meanwhile)
        unsigned gone = 0;
        if (PAGED) {
          const int box_shift = min(p.pages.shift, 7);
          const int key = (f_mine + j) * BN + (lane << box_shift);
          const bool none = lane < (BN >> box_shift) && key < cta_end && page_of(p.pages, b, key) < 0;
          gone = __ballot_sync(0xffffffffu, none);
        }
        if (!wait_all(&s_full[x], j & 1)) { ok = false; break; }
        tc::fence_after();
        if (PAGED && gone != 0) {
          // their scores become -inf in tensor memory, 8 keys at a time (no
          // register of the ordinary tiles is spent on it)
          const int box_shift = min(p.pages.shift, 7);
          uint32_t neg[8];
#pragma unroll
          for (int c = 0; c < 8; ++c) neg[c] = __float_as_uint(kNegInf);
#pragma unroll 1
          for (int c8 = 0; c8 < BN / 8; ++c8)
            if ((gone >> ((8 * c8) >> box_shift)) & 1u) tc::st8(tl + kColS + 8 * c8, neg);
          tc::wait_st();
        }
        float xs[128];
        {
          // all four 32-column loads in flight, one wait
          uint32_t r0[32], r1[32], r2[32], r3[32];
          tc::ld32(tl + kColS, r0);
          tc::ld32(tl + kColS + 32, r1);
          tc::ld32(tl + kColS + 64, r2);
          tc::ld32(tl + kColS + 96, r3);
          tc::wait_ld();
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            xs[c] = __uint_as_float(r0[c]);
            xs[32 + c] = __uint_as_float(r1[c]);
            xs[64 + c] = __uint_as_float(r2[c]);
            xs[96 + c] = __uint_as_float(r3[c]);
          }
        }
        const int key0 = (f_mine + j) * BN;
        // the mask (select, diagonal tiles only) before any arithmetic
        if (key0 + BN > mask_min) {
#pragma unroll
          for (int c = 0; c < 128; ++c) xs[c] = (key0 + c < my_end) ? xs[c] : kNegInf;
        }
        if constexpr (WIN) {
          // sliding window: keys before the row's first visible key
          if (key0 < win_max) {
#pragma unroll
            for (int c = 0; c < 128; ++c) xs[c] = (key0 + c >= my_start) ? xs[c] : kNegInf;
          }
        }
        // block maximum on the raw scores (scale > 0), a tree of short chains
        // (three-input max: 8 chains of 8 steps over 16 values each)
        float mx8[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) mx8[c] = xs[c];
#pragma unroll
        for (int c = 8; c < 128; c += 2) mx8[(c >> 1) & 7] = fmax3(mx8[(c >> 1) & 7], xs[c], xs[c + 1]);
        const float mraw = fmaxf(fmax3(mx8[0], mx8[1], mx8[2]), fmax3(fmax3(mx8[3], mx8[4], mx8[5]), mx8[6], mx8[7]));
        const float mt = (mraw == kNegInf) ? kNegInf : mraw * p.scale_log2;
        float alpha = 1.f;
        bool resc = false;
        if (mt != kNegInf) {
          if (m_ref == kNegInf) {
            m_ref = mt;  // first block with a valid key initialises the state
          } else if (mt > m_ref + kLazyRescale) {
            alpha = fast_exp2(m_ref - mt);
            m_ref = mt;
            l *= alpha;
            if (PAGED) lx *= alpha;
            resc = true;
          }
        }
        if (__any_sync(0xffffffffu, resc)) {
          // U rows change reference (U += P_{j-1} V_{j-1} has completed: S_j
          // was issued after it)
#pragma unroll 1
          for (int q4 = 0; q4 < D / 32; ++q4) {
            uint32_t r[32];
            tc::ld32(tl + kColO + 32 * q4, r);
            tc::wait_ld();
#pragma unroll
            for (int c = 0; c < 32; ++c) r[c] = __float_as_uint(__uint_as_float(r[c]) * alpha);
            tc::st32(tl + kColO + 32 * q4, r);
          }
        }
        // p = 2^(s * scale_log2 - m): masked entries are -inf and give exactly 0;
        // a row with no valid key yet has only masked entries in this tile.
        // Pairs of keys in float2 registers (packed fp32 arithmetic).
        const float m_use = (m_ref == kNegInf) ? 0.f : m_ref;
        const float2 sc2 = make_float2(p.scale_log2, p.scale_log2);
        const float2 nm2 = make_float2(-m_use, -m_use);
        const float2 neg1 = make_float2(-1.f, -1.f);
        // sums of the weights; over pages, where l and lx differ, the first three
        // for l and the last for lx
        float2 ls[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f),
                        make_float2(0.f, 0.f)};
        const bool split = split_tile(key0);
        if (split) {
#pragma unroll
          for (int q4 = 0; q4 < 4; ++q4) {  // 32 keys -> 16 columns of P_hi and of P_lo
            uint32_t hi[16], lo[16];
#pragma unroll
            for (int c = 0; c < 16; ++c) {
              const int k2 = 32 * q4 + 2 * c;
              const float2 e = __ffma2_rn(make_float2(xs[k2], xs[k2 + 1]), sc2, nm2);
              const float2 pp = make_float2(fast_exp2(e.x), fast_exp2(e.y));
              ls[c & 3] = __fadd2_rn(ls[c & 3], pp);
              // P = P_hi + P_lo: P_hi = the upper halves (truncation, exact),
              // P_lo = bf16(P - P_hi) (P - P_hi exact in fp32, below 2^-7 P)
              asm("prmt.b32 %0, %1, %2, 0x7632;" : "=r"(hi[c]) : "r"(__float_as_uint(pp.x)), "r"(__float_as_uint(pp.y)));
              const float2 th = make_float2(__uint_as_float(__float_as_uint(pp.x) & 0xffff0000u),
                                            __uint_as_float(__float_as_uint(pp.y) & 0xffff0000u));
              const float2 rem = __ffma2_rn(th, neg1, pp);
              lo[c] = pack_bf16(rem.x, rem.y);
            }
            tc::st16(tl + kColS + 16 * q4, hi);
            tc::st16(tl + kColPlo + 16 * q4, lo);
          }
        } else {
          // every row sees every key of the tile: P rounded to bf16 (to
          // nearest) is the product's operand, and l sums the rounded values,
          // so u / l stays a convex combination of the values: one key that
          // holds all the weight gives its value back, whatever its rounding.
          // Over pages lse takes the sum before the rounding, which keeps it
          // fp32 accurate (one sum, the unrounded, 361 us for the case above;
          // both 377, 381 with two accumulators each, 390 with more registers for
          // them, 403 with the halves unpacked by shift and mask)
#pragma unroll
          for (int q4 = 0; q4 < 4; ++q4) {  // 32 keys -> 16 columns of P
            uint32_t pb[16];
#pragma unroll
            for (int c = 0; c < 16; ++c) {
              const int k2 = 32 * q4 + 2 * c;
              const float2 e = __ffma2_rn(make_float2(xs[k2], xs[k2 + 1]), sc2, nm2);
              const float2 pp = make_float2(fast_exp2(e.x), fast_exp2(e.y));
              pb[c] = pack_bf16(pp.x, pp.y);
              if (PAGED) {
                add_bf16x2(ls[c % 3], pb[c]);
                ls[3] = __fadd2_rn(ls[3], pp);
              } else {
                ls[c & 3] = __fadd2_rn(ls[c & 3], make_float2(__uint_as_float(pb[c] << 16),
                                                              __uint_as_float(pb[c] & 0xffff0000u)));
              }
            }
            tc::st16(tl + kColS + 16 * q4, pb);
          }
        }
        {
          const float2 a = __fadd2_rn(ls[0], ls[1]);
          if (PAGED && !split) {
            const float2 t2 = __fadd2_rn(a, ls[2]);
            l += t2.x + t2.y;
            lx += ls[3].x + ls[3].y;
          } else {
            const float2 t2 = __fadd2_rn(a, __fadd2_rn(ls[2], ls[3]));
            const float t = t2.x + t2.y;
            l += t;
            if (PAGED) lx += t;
          }
        }
        if (key0 + BN > cta_end || (WIN && PAGED && key0 < cta_start)) {
          // last tile of the CTA: zero the V rows past every visible key of
          // both query tiles (both may do it; the values are the same); in
          // pages also those before every row's window
          const int u = f_mine - j_lo + j + ro;  // ring position of this key tile
          const int s = u % STAGES;
          if (!wait_all(&v_full[s], (u / STAGES) & 1)) { ok = false; break; }
          unsigned char* vt = sm + kOffV + s * kTileBytes;
          const int z0 = WIN && PAGED ? min(max(cta_end - key0, 0), BN) : cta_end - key0;
          const int z1 = WIN && PAGED ? min(max(cta_start - key0, 0), BN) : 0;
          const int nz = BN - z0 + z1;  // rows [z0, BN), then [0, z1)
          for (int idx = (int)(threadIdx.x & 127); idx < nz * (D / 8); idx += 128) {
            int r = z0 + idx / (D / 8);
            if (WIN && PAGED && r >= BN) r -= BN;
            const int c = idx % (D / 8);  // 16-byte chunk over the dims (64 a box)
            const int at = WIDE ? (r >> 3) * 2048 + (c >> 3) * 1024 + (r & 7) * 128 : (c >> 3) * kBox + r * 128;
            *reinterpret_cast<uint4*>(vt + at + (((c & 7) ^ (r & 7)) << 4)) =
                make_uint4(0, 0, 0, 0);
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        }
        tc::wait_st();
        tc::fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[x]);
      }
      // ---- epilogue: o = u / l, lse = m + ln l ----
      // `drain` completes once every MMA of the CTA has (single phase)
      if (ok && !wait_all(drain, 0)) ok = false;
      if (!ok) {
        if (lane == 0) {
          record_error(p.err, kErrTimeout);
          misc[5] = 1;
        }
      } else {
        tc::fence_after();
        // (over pages a NaN score, which no maximum shows where the tile's other
        // keys are masked, makes the row NaN instead of empty)
        if (PAGED && l != l) m_ref = l;
        const float inv = PAGED && parts > 1 ? 1.f : ((m_ref == kNegInf) ? 0.f : 1.f / l);
        if ((p.o_tma && !WIN) || (PAGED && parts > 1)) {
          // (fp32 rows of the output, or of a split item's partial U)
          // Every MMA has completed (drain), so the K (query tile 0) or V
          // (query tile 1) ring is free.  Each warp stages its 32 rows, 64
          // dims at a time (rows padded to 68 floats: conflict-free both
          // ways), and stores them back 16 lanes to a row (256 contiguous
          // bytes per row per store instruction).  (Measured against the
          // tiled-TMA form below: faster for full causal tiles, slower for
          // the short windowed CTAs, which keep TMA.)
          constexpr int kRow = 68;
          float* stg = reinterpret_cast<float*>(sm + (x == 0 ? kOffK : kOffV) + (warp & 3) * 32 * kRow * 4);
          const int r0 = (2 * pair + x) * BM + 32 * (warp & 3);
          const int rows = min(32, p.Tq - r0);
          const int64_t dst_si = PAGED && parts > 1 ? D : p.o_si;
          float* dst0 = PAGED && parts > 1
                            ? p.ws_u + (ws_row + x * BM + 32 * (warp & 3)) * D
                            : static_cast<float*>(p.out) + (int64_t)b * p.o_sb + (int64_t)h * p.o_sh + (int64_t)r0 * p.o_si;
#pragma unroll 1
          for (int half = 0; half < kBoxes; ++half) {
#pragma unroll 1
            for (int q2 = 0; q2 < 2; ++q2) {
              uint32_t r[32];
              tc::ld32(tl + kColO + 64 * half + 32 * q2, r);
              tc::wait_ld();
#pragma unroll
              for (int c = 0; c < 32; c += 4)
                *reinterpret_cast<float4*>(stg + lane * kRow + 32 * q2 + c) =
                    make_float4(__uint_as_float(r[c]) * inv, __uint_as_float(r[c + 1]) * inv,
                                __uint_as_float(r[c + 2]) * inv, __uint_as_float(r[c + 3]) * inv);
            }
            __syncwarp();
#pragma unroll 4
            for (int it = 0; it < 16; ++it) {
              const int rr = 2 * it + (lane >> 4);
              if (rr < rows)
                *reinterpret_cast<float4*>(dst0 + rr * dst_si + 64 * half + 4 * (lane & 15)) =
                    *reinterpret_cast<const float4*>(stg + rr * kRow + 4 * (lane & 15));
            }
            __syncwarp();
          }
        } else if (p.o_tma) {
          // Every MMA has completed (drain), so the K (query tile 0) or V
          // (query tile 1) ring is free.  Each warp stages its 32 rows x 128
          // dims there as four 4 KB boxes of 32 dims in the 128-byte swizzled
          // layout of the output map (16-byte chunk c of row r at c ^ (r mod
          // 8): conflict-free) and one lane stores them with tiled TMA.
          // One 32-dim box at a time (a short loop body for code that runs
          // once per CTA).
          unsigned char* stage = sm + (x == 0 ? kOffK : kOffV) + (warp & 3) * 4 * 4096;
#pragma unroll 1
          for (int q4 = 0; q4 < D / 32; ++q4) {
            uint32_t r[32];
            tc::ld32(tl + kColO + 32 * q4, r);
            tc::wait_ld();
            float4* box = reinterpret_cast<float4*>(stage + q4 * 4096);
#pragma unroll
            for (int c = 0; c < 8; ++c)
              box[lane * 8 + (c ^ (lane & 7))] =
                  make_float4(__uint_as_float(r[4 * c]) * inv, __uint_as_float(r[4 * c + 1]) * inv,
                              __uint_as_float(r[4 * c + 2]) * inv, __uint_as_float(r[4 * c + 3]) * inv);
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // staged rows -> TMA
          __syncwarp();
          const int row_w = (2 * pair + x) * BM + 32 * (warp & 3);
          if (lane == 0 && row_w < p.Tq) {
            // rows past Tq are clipped by the map
#pragma unroll
            for (int q4 = 0; q4 < D / 32; ++q4) tma_store_4d(&tmo, stage + q4 * 4096, 32 * q4, row_w, h, b);
            bulk_commit();
          }
        } else if (p.o_vec16) {
          // bf16 rows, staged like the fp32 ones: 64 dims at a time, rows
          // padded to 144 bytes, stored back 8 lanes to a row (128 contiguous
          // bytes per row per store instruction)
          constexpr int kRow = 36;  // words
          uint32_t* stg = reinterpret_cast<uint32_t*>(sm + (x == 0 ? kOffK : kOffV) + (warp & 3) * 32 * kRow * 4);
          const int r0 = (2 * pair + x) * BM + 32 * (warp & 3);
          const int rows = min(32, p.Tq - r0);
          __nv_bfloat16* dst0 =
              static_cast<__nv_bfloat16*>(p.out) + (int64_t)b * p.o_sb + (int64_t)h * p.o_sh + (int64_t)r0 * p.o_si;
#pragma unroll 1
          for (int half = 0; half < kBoxes; ++half) {
#pragma unroll 1
            for (int q2 = 0; q2 < 2; ++q2) {
              uint32_t r[32];
              tc::ld32(tl + kColO + 64 * half + 32 * q2, r);
              tc::wait_ld();
#pragma unroll
              for (int c = 0; c < 32; c += 8) {
                uint32_t w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  w[e] = pack_bf16(__uint_as_float(r[c + 2 * e]) * inv, __uint_as_float(r[c + 2 * e + 1]) * inv);
                *reinterpret_cast<uint4*>(stg + lane * kRow + 16 * q2 + c / 2) = make_uint4(w[0], w[1], w[2], w[3]);
              }
            }
            __syncwarp();
#pragma unroll
            for (int it = 0; it < 8; ++it) {
              const int rr = 4 * it + (lane >> 3);
              if (rr < rows)
                *reinterpret_cast<uint4*>(dst0 + rr * p.o_si + 64 * half + 8 * (lane & 7)) =
                    *reinterpret_cast<const uint4*>(stg + rr * kRow + 4 * (lane & 7));
            }
            __syncwarp();
          }
        } else {
          // the tensor-memory loads are warp-collective: every lane takes
          // part, rows past Tq store nothing
#pragma unroll 1
          for (int q4 = 0; q4 < D / 32; ++q4) {
            uint32_t r[32];
            tc::ld32(tl + kColO + 32 * q4, r);
            tc::wait_ld();
            if (my_row) {
#pragma unroll
              for (int c = 0; c < 32; ++c) {
                const float o = __uint_as_float(r[c]) * inv;
                const int64_t oi = out_row + (int64_t)(32 * q4 + c) * p.o_sd;
                if (p.out_bf16)
                  static_cast<__nv_bfloat16*>(p.out)[oi] = __float2bfloat16_rn(o);
                else
                  static_cast<float*>(p.out)[oi] = o;
              }
            }
          }
        }
        if (PAGED && parts > 1) {
          if (my_row) {
            p.ws_m[ws_row + threadIdx.x] = m_ref;
            reinterpret_cast<float2*>(p.ws_l)[ws_row + threadIdx.x] = make_float2(l, lx);
          }
        } else if (my_row) {
          p.lse[lse_idx] = (m_ref == kNegInf) ? kNegInf : (m_ref + __log2f(PAGED ? lx : l)) * kLn2;
        }
        // the staging buffer is released with the CTA: the stores must have
        // read it (no-op for a lane without stores)
        if (WIN && p.o_tma && lane == 0) bulk_wait_read();
      }
    }
  }

  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (warp == kMmaWarp) tc::dealloc(tb, kTmemCols);
}

// Joins the parts of the split items (eqs. 33.4-33.5), a warp a row; the parts
// in their order, so the result does not depend on which finished first.
constexpr int kJoinWarps = 8;
template <int D>
__global__ void __launch_bounds__(32 * kJoinWarps) prompt_join_kernel(const FwdParams p) {
  // launched as a programmatic dependent of the prompt kernel
  asm volatile("griddepcontrol.wait;" ::: "memory");
  constexpr int DPL = D / 32;  // dims a lane
  const int lane = threadIdx.x & 31;
  const int idx = blockIdx.x * kJoinWarps + (threadIdx.x >> 5);  // of the split items' rows
  const int n_pairs = (p.Tq + 2 * BM - 1) / (2 * BM);
  const int e = idx / (QT * BM), r = idx % (QT * BM);
  int pair, bh;
  item_of<true>(p, p.split_from + e, n_pairs, pair, bh);
  const int i = pair * (QT * BM) + r;
  if (i >= p.Tq) return;
  const int parts = p.n_splits;  // <= 32
  const int64_t row0 = (int64_t)e * parts * (QT * BM) + r;
  const float m = lane < parts ? p.ws_m[row0 + lane * (QT * BM)] : kNegInf;
  const float2 lp = lane < parts ? reinterpret_cast<const float2*>(p.ws_l)[row0 + lane * (QT * BM)]
                                 : make_float2(0.f, 0.f);  // l, lx
  float M = m;
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
  // a part without a visible key of this row wrote no l and no U: whatever
  // lies there is dropped by select
  const float w = m == kNegInf ? 0.f : fast_exp2(m - M);
  float l = m == kNegInf ? 0.f : w * lp.x, lx = m == kNegInf ? 0.f : w * lp.y;
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) {
    l += __shfl_xor_sync(0xffffffffu, l, off);
    lx += __shfl_xor_sync(0xffffffffu, lx, off);
  }
  float u[DPL];
#pragma unroll
  for (int c = 0; c < DPL; ++c) u[c] = 0.f;
  constexpr int kBatch = 4;  // parts whose loads are in flight together
  for (int s0 = 0; s0 < parts; s0 += kBatch) {
    float v[kBatch][DPL];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const float* us = p.ws_u + (row0 + min(s0 + k, parts - 1) * (QT * BM)) * D + lane * DPL;
      if constexpr (DPL == 4) {
        const float4 x = *reinterpret_cast<const float4*>(us);
        v[k][0] = x.x; v[k][1] = x.y; v[k][2] = x.z; v[k][3] = x.w;
      } else {
        const float2 x = *reinterpret_cast<const float2*>(us);
        v[k][0] = x.x; v[k][1] = x.y;
      }
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const float ws = __shfl_sync(0xffffffffu, w, min(s0 + k, 31));  // (0 past the last part)
#pragma unroll
      for (int c = 0; c < DPL; ++c) u[c] = ws == 0.f ? u[c] : fmaf(ws, v[k][c], u[c]);
    }
  }
  // (l = 0: no part saw a key; a maximum would hide a part's NaN)
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const int b = bh / p.Hq, h = bh % p.Hq;
  const int64_t o = (int64_t)b * p.o_sb + (int64_t)h * p.o_sh + (int64_t)i * p.o_si;
  const int d0 = lane * DPL;
  if (p.o_tma) {  // aligned fp32 rows
    float* dst = static_cast<float*>(p.out) + o + d0;
    if constexpr (DPL == 4)
      *reinterpret_cast<float4*>(dst) = make_float4(u[0] * inv, u[1] * inv, u[2] * inv, u[3] * inv);
    else
      *reinterpret_cast<float2*>(dst) = make_float2(u[0] * inv, u[1] * inv);
  } else if (p.o_vec16) {  // aligned bf16 rows
    uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(p.out) + o + d0);
    if constexpr (DPL == 4)
      *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16(u[0] * inv, u[1] * inv), pack_bf16(u[2] * inv, u[3] * inv));
    else
      *dst = pack_bf16(u[0] * inv, u[1] * inv);
  } else {
#pragma unroll
    for (int c = 0; c < DPL; ++c) {
      const int64_t oi = o + (int64_t)(d0 + c) * p.o_sd;
      if (p.out_bf16)
        static_cast<__nv_bfloat16*>(p.out)[oi] = __float2bfloat16_rn(u[c] * inv);
      else
        static_cast<float*>(p.out)[oi] = u[c] * inv;
    }
  }
  if (lane == 0)
    p.lse[(int64_t)b * p.l_sb + (int64_t)h * p.l_sh + (int64_t)i * p.l_si] =
        l == 0.f ? kNegInf : (M + __log2f(lx)) * kLn2;
}

}  // namespace

int prefill_tc_smem_bytes() { return Layout<128>::kSmemBytes; }

namespace {

template <int D, bool WIN, bool PAGED, bool WIDE>
cudaError_t launch_kernel(const FwdParams& p, unsigned blocks, const CUtensorMap& tmq, const CUtensorMap& tmk,
                          const CUtensorMap& tmv, const CUtensorMap& tmo, cudaStream_t stream) {
  static DeviceOnce once;
  constexpr int kSmemBytes = Layout<D>::kSmemBytes;
  if (cudaError_t e = once.set_smem(reinterpret_cast<const void*>(&prefill_tc_kernel<D, WIN, PAGED, WIDE>), kSmemBytes);
      e != cudaSuccess)
    return e;
  prefill_tc_kernel<D, WIN, PAGED, WIDE><<<blocks, kThreads<PAGED>, kSmemBytes, stream>>>(p, tmq, tmk, tmv, tmo);
  return cudaGetLastError();
}

template <int D, bool PAGED, bool WIDE>
cudaError_t launch_form(const FwdParams& p, int n_pairs, const CUtensorMap& tmq, const CUtensorMap& tmk,
                        const CUtensorMap& tmv, const CUtensorMap& tmo, cudaStream_t stream) {
  const int64_t heads = (int64_t)p.Hq * p.B;
  if (p.head_group < 1) return cudaErrorInvalidValue;
  const int64_t groups = (heads + p.head_group - 1) / p.head_group;
  int64_t blocks = groups * p.head_group * n_pairs;
  if (PAGED) blocks = p.split_from + (heads * n_pairs - p.split_from) * p.n_splits;
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  if (p.window > 0) return launch_kernel<D, true, PAGED, WIDE>(p, (unsigned)blocks, tmq, tmk, tmv, tmo, stream);
  return launch_kernel<D, false, PAGED, WIDE>(p, (unsigned)blocks, tmq, tmk, tmv, tmo, stream);
}

}  // namespace

cudaError_t launch_prefill_tc(const FwdParams& p, int n_pairs, const CUtensorMap& tmq, const CUtensorMap& tmk,
                              const CUtensorMap& tmv, const CUtensorMap& tmo, cudaStream_t stream) {
  return launch_form<128, false, false>(p, n_pairs, tmq, tmk, tmv, tmo, stream);
}

cudaError_t launch_prefill_tc_paged(const FwdParams& p, int d, int n_pairs, const CUtensorMap& tmq,
                                    const CUtensorMap& tmk, const CUtensorMap& tmv, const CUtensorMap& tmo,
                                    cudaStream_t stream) {
  if (d != 128 && d != 64) return cudaErrorInvalidValue;
  if (cudaError_t e = d == 64        ? launch_form<64, true, false>(p, n_pairs, tmq, tmk, tmv, tmo, stream)
                      : p.pages.wide ? launch_form<128, true, true>(p, n_pairs, tmq, tmk, tmv, tmo, stream)
                                     : launch_form<128, true, false>(p, n_pairs, tmq, tmk, tmv, tmo, stream);
      e != cudaSuccess || p.n_splits == 1)
    return e;
  const int64_t rows = ((int64_t)p.Hq * p.B * n_pairs - p.split_from) * (QT * BM);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(rows / kJoinWarps));
  cfg.blockDim = dim3(32 * kJoinWarps);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return d == 128 ? cudaLaunchKernelEx(&cfg, prompt_join_kernel<128>, p)
                  : cudaLaunchKernelEx(&cfg, prompt_join_kernel<64>, p);
}

}  // namespace blkattn
