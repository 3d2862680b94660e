// Decode and verify rows over the 8-bit paged cache on the 5th-generation tensor
// cores (tcgen05, kind::f8f6f4), heads of 128.
//
// The cache's bytes are the products' operands: 128 keys at a time go by TMA into
// shared memory and are read there by the tensor core, nothing converts them.
// The other operands are split into pieces of 8 bits side by side along N, so that
// a tile is read once:
//
//   S^T_j  = K_j [q_hi | q_lo]^T      M = 128 keys, N = 2 NR rows, K = 32 x 4
//   U^T   += V_j^T [p_1 | p_2 | ..]^T  M = 128 dims, N = pieces x NR, K = 32 x 4
//
// q: a row scaled by a power of two to 2^7 <= max |q| < 2^8; q_hi its nearest
// e4m3 (4 bits) and q_lo = 32 (q - q_hi) the rest of a bf16's 8 bits, exact but
// for dims below 2^-14 of the row's largest (off by at most 2^-22 of it).
// p: a weight as f16, taken apart exactly into 4 pieces of e5m2: an f16's upper
// byte is the first (its value cut to 3 bits), the rest times 2^4 has 8 bits, its
// upper byte is the second, the rest of that times 2^2 the third's, and so on: e5m2's
// least step, 2^-16, reaches f16's, 2^-24, at the last.  U = U_1 + (U_2 + (U_3 + U_4 /
// 4) / 4) / 16.  An f16's step is 2^-27 of the row's largest weight or finer: a weight
// below 2^-16 of it is off by as much as 2^-28, which a long tail of equal keys beside
// one strong key adds up (n keys of a CTA's range: n 2^-28; a million, what rounding
// to bf16 does).  (One factor 2^8 for the last three pieces leaves room for weights to
// 2^11 only and steps of 2^-23; the rests of the fp32 weights instead of f16's, 12
// bits and steps of 2^-29, took five-row chains of 64 heads 124 us where these took
// 117; pieces of e4m3, two conversions each, 129.)
// With k = 2^ek k8 and v = 2^ev v8: x = (S_hi + S_lo / 32) 2^ek fac_row, and the
// weight is 2^(x - m + ev - r), of two references a row: m >= max x for the
// sum of fp32 weights, and r >= max (x - m + ev) - 7 for the product's (r relative
// to m: beside a large x, ev would be lost).
//
// Otherwise the kernel is the one of decode_tc.cu over pages: the same cut of
// all units' tiles into equal ranges, one a CTA, the same roles, order of
// products, ring and waits; the unit loader also brings each key's scales.
//
// What bounds it: memory for up to 16 rows once the stream runs (5.8 TB/s; 11 us of
// cold latency before).  For more, the chain of a tile, which all key threads pass
// together: wait for the scores, load them from tensor memory, weights, a vote over
// all of them, P^T, arrival, some 1.5 us a tile of 128 keys in which no pipe is over
// a third busy (40 rows: 117 us where the bytes take 42), and raises of a reference,
// 2.5 us each.
//
// Every wait is bounded (%globaltimer); on a timeout the CTA records the error
// word, stops issuing work, lets its own copies and products drain and frees
// its tensor memory.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kernels.h"
#include "ptx.cuh"
#include "q8.cuh"
#include "tc.cuh"

namespace blkattn {
namespace {

constexpr float kLn2 = 0.6931471805599453f;
constexpr float kNegInf = -__builtin_huge_valf();
// m is set 2^24 above the largest score so far (the sum of fp32 weights loses
// nothing by it) and rises when one passes it.
constexpr float kMarginM = 24.f;
// In place of m where a row has none yet: any score is above, a masked one's weight 0.
constexpr float kNoM = -3e38f;
// r stays above: 2^(kLift - r) is a float.  (Values all below 2^-100 448 lose bits.)
constexpr float kLeastR = -118.f;
// And below kMostR, so that 2^(kLift - r) stays a float, not a subnormal one: a
// product's largest is 2^127 (x <= m, ev <= 127), 2^(kLift + 127 - kMostR) = 2 then.
constexpr float kMostR = 134.f;
// A weight at the reference is 2^kLift, and the reference is set 2^kMargin above
// the largest weight so far: there is room for a maximum 2^12 above that before the
// reference has to rise, which costs a tile 2.5 us (with room for 2^6 ten tiles of
// 57 raised one of 40 rows', with this four; for 2^11 and 2^10 five-row chains of 64
// heads 120 us, for this 117).  kMostW: the largest f16 whose rest times 2^4 is one.
constexpr float kLift = 8.f, kMargin = 5.f;
constexpr float kMostW = 32752.f;
static_assert(kMostR == kLift + 126.f, "2^(kLift - kMostR) is the least normal float");

constexpr int D = 128;
constexpr int BK = 128;               // keys of a product (TMEM lanes of S^T)
constexpr int kSlotBytes = BK * D;    // a ring slot, K or V: 128 rows of 128 bytes
constexpr int kBarRows = 1;           // named barrier of the key threads
constexpr int kBarFirst = 2;          // of the key threads and the unit loader: the first unit's query rows
constexpr uint32_t kTmemCols = 512;

// Instruction descriptor for kind::f8f6f4: e4m3 A, e4m3 (0) or e5m2 (1) B, fp32
// accumulator.
constexpr uint32_t idesc_f8(int b_type, int M, int N, int a_mn, int b_mn) {
  return (1u << 4) | ((uint32_t)b_type << 10) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) | ((uint32_t)(N >> 3) << 17) |
         ((uint32_t)(M >> 4) << 24);
}
__device__ __forceinline__ void mma_f8(uint32_t d_taddr, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_taddr),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ uint32_t h2_to_e4m3x2(uint32_t h) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(h));
  return r;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Integer facts of the rows of one unit (written by the unit loader).
template <int NR>
struct RowFacts {
  int64_t ooff[NR];  // output row offsets
  int64_t loff[NR];  // lse offsets
  uint64_t tree[NR]; // token tree: bit k = the row sees key tree_base + k (all ones without a tree);
                     // with a sliding window instead: the row's first visible key
  int end[NR];       // visible keys are [0, end): min(len, pos + 1), 0 for padding rows
  float fac[NR];     // scale log2(e) times the power of two that the row was divided by
  int unit_end;      // max over the rows
  int unit_start;    // the earliest key that a row sees (INT_MAX: none)
  uint64_t tree_seen;  // bit k = some row sees tree node k
  int min_end;       // min over the rows that see keys
  int tree_base;     // first key of the token tree (len - T_q); INT_MAX without a tree
  int win_max;       // sliding window: the largest first visible key of the rows (0 without)
};

template <int NR>
struct TcLayout {
  // Up to 16 rows a tile is 256 keys, two subtiles, each with key threads of its
  // own: what a tile takes is a chain of waits, loads and a vote, some 1.5 us
  // whatever its size.  More rows: 128 keys.
  // (12 key warps of 16 rows each for 48, not 8 of 24: 157 us in place of 190
  // for five-row chains of 64 heads when it was tried)
  static constexpr int kSub = NR <= 16 ? 2 : 1;
  static constexpr int kParts = NR == 8 ? 1 : (NR == 16 ? 2 : (NR == 32 ? 2 : 3));
  static constexpr int kKeyWarps = 4 * kSub * kParts;        // a warp a TMEM lane quarter, subtile and part of the rows
  static constexpr int kThreads = 32 * (kKeyWarps + 4);
  static constexpr int kTileKeys = kSub * BK;
  static constexpr int kPieces = 4;
  static constexpr int kPN = kPieces * NR;                   // N of the value product
  static constexpr int kPSub = (kPN > 128 ? 2 : 1) * BK * 128;  // P^T of a subtile: atoms of 128 columns
  static constexpr int kPBytes = kSub * kPSub;               // one P^T buffer
  static constexpr int kQBytes = 2 * NR * 128;               // q_hi rows, then q_lo rows
  static constexpr int kSlots = NR > 32 ? 7 : (NR > 16 ? 10 : 8);
  static constexpr int kScaleRing = 8 * kSub;                // subtiles whose scales lie in shared memory
  static constexpr uint32_t kColS = 0;                       // S^T: tiles of even / odd index, their subtiles
  static constexpr uint32_t kSubS = 2 * NR;
  static constexpr uint32_t kStepS = kSub * kSubS;
  // U^T of units of even / odd index; more than 32 rows: one, read out before the
  // next unit's first P is written
  static constexpr int kBufU = NR > 32 ? 1 : 2;
  static constexpr uint32_t kColU = 2 * kStepS;
  static constexpr uint32_t kStepU = kBufU == 2 ? kPN : 0;
  static constexpr int kOffQ = kSlots * kSlotBytes;              // two query buffers
  static constexpr int kOffP = kOffQ + 2 * kQBytes;              // two P^T buffers
  static constexpr int kOffRows = kOffP + 2 * kPBytes;           // RowFacts[2]
  static constexpr int kRowsBytes = (int)((sizeof(RowFacts<NR>) + 15) / 16 * 16);
  static constexpr int kOffNTab = kOffRows + 2 * kRowsBytes;     // uint16 tiles, first tile per (sequence, row group)
  static constexpr int kOffRed = kOffNTab + 2 * kDecodeTcMaxEntries * 2;  // float [8][NR]
  // float [NR] each: m, m_use, r, 2^(lift - r), factor of l, factor of U of the
  // current unit; m, l, r, 1 / l of the finished unit whose U readout is pending
  static constexpr int kOffStat = kOffRed + 8 * NR * 4;
  static constexpr int kOffScale = kOffStat + 10 * NR * 4;       // uint32 [kScaleRing][BK]: each key's scale bytes
  static constexpr int kOffBar = kOffScale + kScaleRing * BK * 4;
  // full[kSlots], empty[kSlots], q_full[2], q_empty[2], p_full[2], u_full[2], drain, sc_full[kScaleRing], sc_empty[kScaleRing]
  static constexpr int kNumBars = 2 * kSlots + 2 + 2 + 2 + 2 + 1 + 2 * kScaleRing;
  static constexpr int kOffMisc = kOffBar + kNumBars * 8;
  static constexpr int kBytes = kOffMisc + 128 + 1024;  // + slack to align to 1024
  static_assert(kOffQ % 1024 == 0 && kOffP % 1024 == 0 && kQBytes % 1024 == 0, "swizzle atoms");
  static_assert(kOffBar % 8 == 0 && kOffStat % 16 == 0 && kOffScale % 16 == 0, "alignment");
  static_assert(kColU + kBufU * kPN <= kTmemCols, "tensor memory");
  static_assert(kBytes <= 232448, "shared memory per block");
};

// The CTA's start in the tile order (written once by warp 0).
struct Start {
  int t0, t1, W, P, su;  // (the host keeps the tile count below 2^24)
  int b, kvh, rg, j;
};

// Position in the tile order: global tile t of unit (b, kvh, rg), local tile
// j of n, the unit's first global tile su.  Each unit spans n real tiles and
// `extra` weight-only tiles after them (the partition charges a unit for its
// set-up and readout, so CTAs holding many short units get fewer tiles).
struct Cursor {
  int t, su;
  int b, kvh, rg, j, n;
  int extra;
  int s0;               // the unit's first tile (sliding window; 0 otherwise)
  const uint16_t* st;   // per-unit first tiles, or nullptr
  int tk;               // keys of a tile
  __device__ __forceinline__ int key0() const { return (s0 + j) * tk; }
  // to the first tile of the next unit
  __device__ __forceinline__ void step_unit(const uint16_t* ntab, int RG, int Hkv, int B) {
    su += n + extra;
    t = su;
    j = 0;
    if (++rg == RG) {
      rg = 0;
      if (++kvh == Hkv) {
        kvh = 0;
        ++b;
      }
    }
    n = (b < B) ? (int)ntab[b * RG + rg] : 1;
    s0 = (b < B && st != nullptr) ? (int)st[b * RG + rg] : 0;
  }
  __device__ __forceinline__ void next(const uint16_t* ntab, int RG, int Hkv, int B) {
    if (j + 1 == n) {
      step_unit(ntab, RG, Hkv, B);
    } else {
      ++t;
      ++j;
    }
  }
};

// CTA whose range [c W / P, (c + 1) W / P) holds global tile t.
// (32-bit arithmetic: the host keeps the tile count below 2^24 and
// P <= 255, so (t + 1) P < 2^32.)
__device__ __forceinline__ int cta_of(int t, int W, int P) {
  return (int)((((uint32_t)t + 1u) * (uint32_t)P + (uint32_t)W - 1u) / (uint32_t)W) - 1;
}

// N consecutive TMEM columns of this thread's lane (N = 8, 16 or 24; the
// column offset is a multiple of 8, of 16 for N = 16) -> floats.
template <int N>
__device__ __forceinline__ void ld_cols(uint32_t taddr, float (&x)[N]) {
  uint32_t r[N];
  if constexpr (N == 16) {
    tc::ld16(taddr, &r[0]);
  } else {
#pragma unroll
    for (int c = 0; c < N; c += 8) tc::ld8(taddr + c, &r[c]);
  }
  tc::wait_ld();
#pragma unroll
  for (int c = 0; c < N; ++c) x[c] = __uint_as_float(r[c]);
}

template <int N>
__device__ __forceinline__ void st_cols(uint32_t taddr, const float (&x)[N]) {
  uint32_t r[N];
#pragma unroll
  for (int c = 0; c < N; ++c) r[c] = __float_as_uint(x[c]);
  if constexpr (N == 16) {
    tc::st16(taddr, &r[0]);
  } else {
#pragma unroll
    for (int c = 0; c < N; c += 8) tc::st8(taddr + c, &r[c]);
  }
}

// Reduce NH values per lane across the 32 lanes of a warp (NH = 8, 16, 24):
// three reduce-scatter steps (xor 16, 8, 4) halve the values a lane keeps,
// two full steps (xor 2, 1) finish them.  Afterwards lane l holds the
// results for rows base + i, i < NH / 8, base = (l >> 4 & 1) NH / 2 +
// (l >> 3 & 1) NH / 4 + (l >> 2 & 1) NH / 8, in v[0 .. NH / 8).  The
// shuffles of one step are independent (27 in all for NH = 24).
template <int NH, bool kMax>
__device__ __forceinline__ void warp_reduce_scatter(float (&v)[NH], int lane) {
  auto op = [](float a, float b) { return kMax ? fmaxf(a, b) : a + b; };
#pragma unroll
  for (int step = 0; step < 3; ++step) {
    const int off = 16 >> step;
    const int half = NH >> (step + 1);  // values kept after this step
    const bool upper = (lane & off) != 0;
#pragma unroll
    for (int i = 0; i < half; ++i) {
      const float send = upper ? v[i] : v[i + half];
      const float keep = upper ? v[i + half] : v[i];
      v[i] = op(keep, __shfl_xor_sync(0xffffffffu, send, off));
    }
  }
#pragma unroll
  for (int off = 2; off >= 1; off >>= 1)
#pragma unroll
    for (int i = 0; i < NH / 8; ++i) v[i] = op(v[i], __shfl_xor_sync(0xffffffffu, v[i], off));
}

template <int NH>
__device__ __forceinline__ int scatter_base(int lane) {
  return ((lane >> 4) & 1) * (NH / 2) + ((lane >> 3) & 1) * (NH / 4) + ((lane >> 2) & 1) * (NH / 8);
}

template <int NR>
__global__ void __launch_bounds__(TcLayout<NR>::kThreads, 1)
    decode_tc_q8_kernel(const __grid_constant__ Q8Params p, const __grid_constant__ CUtensorMap tmk,
                        const __grid_constant__ CUtensorMap tmv) {
  using L = TcLayout<NR>;
  constexpr uint32_t kIdescQK = idesc_f8(0, 128, 2 * NR, 0, 0);   // K, Q both K-major
  constexpr uint32_t kIdescPV = idesc_f8(1, 128, L::kPN, 1, 1);   // V^T, P^T both MN-major
  constexpr int kSlots = L::kSlots, kSub = L::kSub, TK = L::kTileKeys, kScaleRing = L::kScaleRing;
  constexpr int kPieces = L::kPieces;
  constexpr int kKeyWarps = L::kKeyWarps, kKeyThreads = 32 * kKeyWarps, kThreads = L::kThreads;
  constexpr int kPageKWarp = kKeyWarps, kMmaWarp = kKeyWarps + 1, kLoadWarp = kKeyWarps + 2, kPageVWarp = kKeyWarps + 3;
  // weight-only tiles per unit in the partition (its set-up and readout)
  constexpr int kUnitExtra = NR >= 48 ? 2 : 0;

  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* sm = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  RowFacts<NR>* facts0 = reinterpret_cast<RowFacts<NR>*>(sm + L::kOffRows);
  uint16_t* ntab = reinterpret_cast<uint16_t*>(sm + L::kOffNTab);
  uint16_t* stab = ntab + kDecodeTcMaxEntries;  // the units' first tiles (sliding window)
  float* red = reinterpret_cast<float*>(sm + L::kOffRed);
  float* s_m = reinterpret_cast<float*>(sm + L::kOffStat);  // reference maximum, -inf = none yet
  float* s_muse = s_m + NR;                                  // m, or kNoM when none yet
  float* s_r = s_m + 2 * NR;                                 // reference of the weights, -inf = none yet
  float* s_h = s_m + 3 * NR;                                 // 2^(lift - r), 1 when none yet
  float* s_alpha = s_m + 4 * NR;
  float* s_beta = s_m + 5 * NR;
  float* s_mfin = s_m + 6 * NR;
  float* s_lfin = s_m + 7 * NR;
  float* s_rfin = s_m + 8 * NR;
  float* s_inv = s_m + 9 * NR;
  uint32_t* s_sc = reinterpret_cast<uint32_t*>(sm + L::kOffScale);
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + L::kOffBar);
  uint64_t* full = bars;
  uint64_t* empty = full + kSlots;
  uint64_t* q_full = empty + kSlots;  // [2]
  uint64_t* q_empty = q_full + 2;     // [2]
  uint64_t* p_full = q_empty + 2;     // [2] by tile parity
  uint64_t* u_full = p_full + 2;      // [2] by unit parity
  uint64_t* drain = u_full + 2;
  uint64_t* sc_full = drain + 1;            // [kScaleRing]
  uint64_t* sc_empty = sc_full + kScaleRing;
  // misc: [0] tmem base, [1] error seen by the producer / MMA thread,
  // [2] abort of the key threads, [3] "this CTA folds the unit", [4], [5] "a
  // row's m rises in this tile", by parity (written before a barrier of the key
  // threads, read after it)
  int* misc = reinterpret_cast<int*>(sm + L::kOffMisc);
  Start* start = reinterpret_cast<Start*>(sm + L::kOffMisc + 64);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int RG = p.row_groups;
  const int R = p.rows_cta;
  const int rows_per_head = p.G * p.Tq;
  const int B = p.B;
  const int Hkv = p.Hkv;

  // ---------------- schedule: tiles per (sequence, row group) ----------------
  {
    int* nb = reinterpret_cast<int*>(sm + L::kOffP);  // per-sequence totals (P^T area, start-up only)
    const int E = B * RG;
    for (int e = threadIdx.x; e < E; e += kThreads) {
      const int b = e / RG;
      const int rg = e - b * RG;
      // the row end min(len, pos + 1) (0 for pos < 0) grows with pos, so the
      // unit's end follows from the largest position of its rows; all loads
      // are independent (one round trip)
      const int len_raw = p.seqlens[b * p.sl_s];
      const int pk0 = rg * R;
      const int pk1 = min(pk0 + R, rows_per_head);
      int maxpos = -1, minpos = 0x7fffffff;  // minpos over the rows that see keys
      if (pk1 - pk0 >= p.Tq) {
#pragma unroll 4
        for (int i = 0; i < p.Tq; ++i) {
          const int ps = p.qpos[b * p.qp_sb + i * p.qp_si];
          maxpos = max(maxpos, ps);
          if (ps >= 0) minpos = min(minpos, ps);
        }
      } else {
#pragma unroll 4
        for (int pk = pk0; pk < pk1; ++pk) {
          const int ps = p.qpos[b * p.qp_sb + (pk % p.Tq) * p.qp_si];
          maxpos = max(maxpos, ps);
          if (ps >= 0) minpos = min(minpos, ps);
        }
      }
      const int len = len_raw < 0 ? 0 : (len_raw > p.Tmax ? p.Tmax : len_raw);
      const int uend = maxpos < 0 ? 0 : min(maxpos, len - 1) + 1;  // (a position may be INT_MAX)
      // sliding window: the unit starts at the tile of its earliest visible key
      const int s0 = (p.window > 0 && minpos != 0x7fffffff) ? max(0, minpos - p.window + 1) / TK : 0;
      const int n = (uend + TK - 1) / TK - s0;
      ntab[e] = (uint16_t)(n < 1 ? 1 : n);  // an all-empty unit still takes one (masked) tile
      if (p.window > 0) stab[e] = (uint16_t)s0;
    }
    if (threadIdx.x == 0) {
      misc[1] = 0;
      misc[2] = misc[4] = misc[5] = 0;
      for (int s = 0; s < kSlots; ++s) {
        mbar_init(&full[s], 1);
        mbar_init(&empty[s], 1);
      }
      for (int x = 0; x < 2; ++x) {
        mbar_init(&q_full[x], 1);
        // query buffer x is free once the unit's last S product completed
        // (MMA commit) and its row facts are no longer read (key threads)
        mbar_init(&q_empty[x], 2);
        mbar_init(&u_full[x], 1);
      }
      for (int x = 0; x < 2; ++x) mbar_init(&p_full[x], kKeyWarps);  // one arrival per key warp
      for (int x = 0; x < kScaleRing; ++x) {
        mbar_init(&sc_full[x], 1);
        mbar_init(&sc_empty[x], kKeyWarps / kSub);
      }
      mbar_init(drain, 1);
      fence_barrier_init();
    }
    if (threadIdx.x < NR) {
      s_m[threadIdx.x] = kNegInf;
      s_muse[threadIdx.x] = kNoM;
      s_r[threadIdx.x] = kNegInf;
      s_h[threadIdx.x] = 1.f;
    }
    if (warp == kMmaWarp) {
      tc::alloc(reinterpret_cast<uint32_t*>(&misc[0]), kTmemCols);
      tc::relinquish();
    }
    __syncthreads();
    for (int b = threadIdx.x; b < B; b += kThreads) {
      int s = 0;
      for (int rg = 0; rg < RG; ++rg) s += ntab[b * RG + rg] + kUnitExtra;
      nb[b] = s;
    }
    __syncthreads();
    if (warp == 0) {
      // tiles of sequence b: Hkv * nb[b]; lane l sums a contiguous run of sequences
      const int per = (B + 31) / 32;
      const int b0 = min(lane * per, B);
      const int b1 = min(b0 + per, B);
      long long s = 0;
      for (int b = b0; b < b1; ++b) s += (long long)nb[b] * Hkv;
      long long incl = s;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += v;
      }
      const long long W = __shfl_sync(0xffffffffu, incl, 31);
      // with fewer tiles than CTAs the last CTAs stay idle, so that every
      // working CTA has a tile and the CTAs holding one unit are consecutive
      long long P = W < (long long)gridDim.x ? W : (long long)gridDim.x;
      if (P > 0) {
        // Short units spread over every CTA make many parts, and one CTA
        // folds a unit's, 512 items (4 dims of a row) at a time, four parts a
        // round trip: t tiles a CTA cost about 1.5 t us, and units of n tiles
        // 0.17 n / t us a fold pass.  At least the t of the minimum (with
        // twice the fold's cost, which fits best).  4 x 8 units of 1000 keys
        // 17.6 us without, 13.2 with it.
        const float n = (float)W / (float)(B * Hkv * RG);
        const int t_min = (int)ceilf(sqrtf(0.233f * n * (float)((R * D + 2047) / 2048)) - 0.01f);
        if (t_min > 1) P = min(P, max(1ll, W / t_min));
      }
      const bool works = (long long)blockIdx.x < P;
      // c W / P in 32 bits: W = q P + r, c W / P = c q + c r / P (c r < 2^16)
      const uint32_t q = (uint32_t)W / (uint32_t)(P > 0 ? P : 1), r = (uint32_t)W - q * (uint32_t)P;
      const uint32_t c = blockIdx.x;
      const long long t0 = works ? (long long)(c * q + c * r / (uint32_t)P) : W;
      const long long t1 = works ? (long long)((c + 1) * q + (c + 1) * r / (uint32_t)P) : W;
      const long long excl = incl - s;
      const unsigned own = __ballot_sync(0xffffffffu, t0 < t1 && excl <= t0 && t0 < incl);
      if (lane == 0) {
        start->t0 = (int)t0;
        start->t1 = (int)t1;
        start->W = (int)W;
        start->P = (int)P;
      }
      if (own != 0 && lane == __ffs(own) - 1) {
        long long pre = excl;
        int b = b0;
        while (pre + (long long)nb[b] * Hkv <= t0) {
          pre += (long long)nb[b] * Hkv;
          ++b;
        }
        const long long o = t0 - pre;
        const int kvh = (int)((uint32_t)o / (uint32_t)nb[b]);
        long long o2 = o - (long long)kvh * nb[b];
        long long su = pre + (long long)kvh * nb[b];
        int rg = 0;
        while (o2 >= ntab[b * RG + rg] + kUnitExtra) {
          o2 -= ntab[b * RG + rg] + kUnitExtra;
          su += ntab[b * RG + rg] + kUnitExtra;
          ++rg;
        }
        start->b = b;
        start->kvh = kvh;
        start->rg = rg;
        start->j = (int)o2;
        start->su = (int)su;
      }
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
  }
  const int t0 = start->t0;
  const int t1 = start->t1;
  const int W = start->W;
  const int P_work = start->P;  // CTAs that hold tiles: [0, P_work)
  const uint32_t tb = static_cast<uint32_t>(misc[0]);
  const uint32_t sRing = smem_u32(sm);
  const uint32_t sQ = smem_u32(sm + L::kOffQ);
  const uint32_t sP = smem_u32(sm + L::kOffP);
  Cursor cur;
  cur.t = t0;
  cur.su = start->su;
  cur.b = start->b;
  cur.kvh = start->kvh;
  cur.rg = start->rg;
  cur.j = start->j;
  cur.n = (t0 < t1) ? (int)ntab[cur.b * RG + cur.rg] : 1;
  cur.extra = kUnitExtra;
  cur.tk = TK;
  cur.st = p.window > 0 ? stab : nullptr;
  cur.s0 = (t0 < t1 && cur.st != nullptr) ? (int)stab[cur.b * RG + cur.rg] : 0;
  // a range may start among a unit's weight-only tiles: begin at the next unit
  if (t0 < t1 && cur.j >= cur.n) cur.step_unit(ntab, RG, Hkv, B);

  // Query row r (4 dims a lane) scaled by a power of two, taken apart into q_hi and
  // q_lo and written in the 128-byte swizzled K-major layout; returns the row's
  // factor.
  auto put_row = [&](unsigned char* qs, int r, const uint2& w) -> float {
    // (the largest of bit patterns: a NaN is the largest)
    const uint32_t a0 = w.x & 0x7fff7fffu, a1 = w.y & 0x7fff7fffu;
    const uint32_t top = __reduce_max_sync(
        0xffffffffu, max(max(a0 & 0xffffu, a0 >> 16), max(a1 & 0xffffu, a1 >> 16)));
    const int e = top == 0 ? 0 : min(7 + 127 - (int)(top >> 7), 127);  // rows times 2^e
    // (infinities and NaN make the whole row NaN)
    const float f = top >= 0x7f80u ? __uint_as_float(0x7fc00000u) : pow2(e);
    uint32_t hi[2], lo[2];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const uint32_t x = c ? w.y : w.x;
      const __half2 h = __floats2half2_rn(bf16lo(x) * f, bf16hi(x) * f);
      hi[c] = h2_to_e4m3x2(*reinterpret_cast<const uint32_t*>(&h));
      const uint32_t back = e4m3x2_to_h2(hi[c]);
      const __half2 rest = __hmul2(__hsub2(h, *reinterpret_cast<const __half2*>(&back)), __float2half2_rn(32.f));
      lo[c] = h2_to_e4m3x2(*reinterpret_cast<const uint32_t*>(&rest));
    }
    const int at = r * 128 + (((lane >> 2) ^ (r & 7)) << 4) + (lane & 3) * 4;
    *reinterpret_cast<uint32_t*>(qs + at) = hi[0] | hi[1] << 16;
    *reinterpret_cast<uint32_t*>(qs + NR * 128 + at) = lo[0] | lo[1] << 16;
    return p.scale_log2 * pow2(-e);
  };

  if (warp == kPageKWarp || warp == kPageVWarp) {
    // ---------------- producers: K tiles, V tiles from pages (whole warps) ----------------
    // Each takes every second ring entry, so with the even number of slots here a
    // slot's entries are of one of them (with an odd one they alternate; the wait
    // by parity holds for both: see decode_tc.cu).
    const int kv = warp == kPageVWarp ? 1 : 0;
    const void* map = kv ? static_cast<const void*>(&tmv) : static_cast<const void*>(&tmk);
    const uint64_t pol = policy_evict_first();
    if (lane == 0) asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
    // lane: piece `lane` of a tile, a page or the tile's part of one
    const int box_shift = min(p.pages.shift, 7);
    const int n_pieces = BK >> box_shift;
    const bool copies = lane < n_pieces;
    const int piece = lane & (n_pieces - 1);
    // What the lane looks up for a tile, one tile ahead: its piece's table entry
    // and the sequence's length.
    int nx_key = 0, nx_entry = -1, nx_len = 0;
    auto look_up = [&](const Cursor& c, int sub) {
      nx_key = c.key0() + sub * BK + (piece << box_shift);
      nx_entry = entry_of(p.pages, c.b, nx_key);
      nx_len = p.seqlens[c.b * p.sl_s];
    };
    int issued = 0;  // entries
    bool ok = true;
    int sub = 0;
    if (cur.t < t1) look_up(cur, 0);
    for (int g = 0; ok && cur.t < t1; ++g) {
      const int row = nx_key & (p.pages.rows - 1);
      const int kvh = cur.kvh;
      // past the length, or no page: -1 (zeros)
      const int page = nx_key < nx_len && (unsigned)nx_entry < (unsigned)p.pages.n_pages ? nx_entry : -1;
      if (++sub == kSub) {
        sub = 0;
        cur.next(ntab, RG, Hkv, B);
      }
      if (cur.t < t1) look_up(cur, sub);
      const int seq = 2 * g + kv;  // (g counts subtiles)
      const int s = seq % kSlots;
      bool w = true;
      if (lane == 0) {
        if (seq >= kSlots) w = mbar_wait(&empty[s], (uint32_t)(((seq / kSlots) - 1) & 1));
        if (w) mbar_arrive_expect_tx(&full[s], kSlotBytes);
      }
      ok = __shfl_sync(0xffffffffu, w, 0);  // (also orders the expected bytes before the copies)
      if (!ok) break;
      __syncwarp();
      if (copies)
        tma_load_4d(sm + s * kSlotBytes + ((piece << box_shift) * 128), map, 0, row, kvh, page, &full[s], pol);
      issued = seq + 1;
      // after the first tile, let the first unit's query rows land before the
      // stream fills the memory queues (they gate the first product)
      if (g == 0) {
        if (lane == 0) w = mbar_wait(&q_full[0], 0);
        ok = __shfl_sync(0xffffffffu, w, 0);
      }
    }
    __syncwarp();
    if (lane == 0) {
      // every issued copy must land before the CTA exits (an entry that has a
      // successor in its slot has: the successor waited for its consumption)
      const bool clean = ok;
      const int all = (issued + 1) / 2 * 2;  // entries of both producers
      for (int seq = issued - 1; seq >= 0 && seq >= all - kSlots - (clean ? 0 : kSlots); seq -= 2)
        if (!mbar_wait(&full[seq % kSlots], (uint32_t)((seq / kSlots) & 1))) ok = false;
      if (!ok) {
        record_error(p.err, kErrTimeout);
        misc[1] = 1;
      }
    }
  } else if (warp == kLoadWarp) {
    // ---------------- loader: query rows and row facts of each unit, scales of each tile ----------------
    int uidx = 0;
    bool ok = true;
    // The scales of lane l's keys 4 l .. 4 l + 3 (of one page), as bytes: a word a
    // key, ek | ev << 8 | 1 << 16 (0: no key).  The table entry of a subtile is on
    // its way three subtiles before the bytes are handed over, the bytes two.
    struct Ask {
      int entry, key, kvh, len;
      bool live;
    };
    struct Bytes {  // (apart, so that nothing waits for them before they are stored)
      int k[4], v[4];
      int n;  // keys that exist
    };
    Cursor at = cur;
    int at_sub = 0;
    bool more = at.t < t1;
    const bool fine = p.scale_shift < 2;  // else one scale for the four
    auto ask = [&]() {
      Ask a{-1, 0, 0, 0, more};
      if (more) {
        a.key = at.key0() + at_sub * BK + 4 * lane;
        a.entry = entry_of(p.pages, at.b, a.key);
        a.len = p.seqlens[at.b * p.sl_s];
        a.kvh = at.kvh;
        if (++at_sub == kSub) {
          at_sub = 0;
          at.next(ntab, RG, Hkv, B);
          more = at.t < t1;
        }
      }
      return a;
    };
    auto fetch = [&](const Ask& a) {
      Bytes y{{}, {}, 0};
      if (a.live && (unsigned)a.entry < (unsigned)p.pages.n_pages) {
        const int row = a.key & (p.pages.rows - 1);
        const unsigned char* ks = p.k_sc + (int64_t)a.entry * p.ke_sn + a.kvh * p.ke_sh;
        const unsigned char* vs = p.v_sc + (int64_t)a.entry * p.ve_sn + a.kvh * p.ve_sh;
        y.n = a.len - a.key;
        y.k[0] = ks[(row >> p.scale_shift) * p.ke_si];
        y.v[0] = vs[(row >> p.scale_shift) * p.ve_si];
        if (fine) {
#pragma unroll
          for (int i = 1; i < 4; ++i) {
            const int blk = (row + i) >> p.scale_shift;
            y.k[i] = ks[blk * p.ke_si];
            y.v[i] = vs[blk * p.ve_si];
          }
        }
      }
      return y;
    };
    Ask a1 = ask(), a2 = ask();
    Bytes y0, y1;
    int gs = 0;  // subtiles handed over
    auto hand_over = [&]() -> bool {
      const int sr = gs % kScaleRing;
      bool w = true;
      if (lane == 0 && gs >= kScaleRing) w = mbar_wait(&sc_empty[sr], (uint32_t)((gs / kScaleRing - 1) & 1));
      if (!__shfl_sync(0xffffffffu, w, 0)) return false;
      uint32_t word[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int ek = fine ? y0.k[i] : y0.k[0], ev = fine ? y0.v[i] : y0.v[0];
        word[i] = i < y0.n ? (uint32_t)(ek | ev << 8 | 1 << 16) : 0u;
      }
      reinterpret_cast<uint4*>(s_sc + sr * BK)[lane] = make_uint4(word[0], word[1], word[2], word[3]);
      __syncwarp();
      if (lane == 0) mbar_arrive(&sc_full[sr]);
      // (only now: what is moved on has arrived)
      y0 = y1;
      y1 = fetch(a2);
      a2 = ask();
      ++gs;
      return true;
    };
    for (; t0 < t1 && cur.su < t1; cur.step_unit(ntab, RG, Hkv, B), ++uidx) {
      const int qb = uidx & 1;
      if (uidx >= 2) {
        bool w = true;
        if (lane == 0) w = mbar_wait(&q_empty[qb], (uint32_t)(((uidx >> 1) - 1) & 1));
        if (!__shfl_sync(0xffffffffu, w, 0)) { ok = false; break; }
      }
      // lane l describes rows l and l + 32 (one division each), then every
      // global load of the unit is issued before any is used (one round
      // trip): cache length, positions, query rows
      unsigned char* qs = sm + L::kOffQ + qb * L::kQBytes;
      const int b = cur.b;
      const int len_raw = p.seqlens[b * p.sl_s];
      bool real[2];
      int hrow[2], irow[2], pos[2] = {-1, -1};
      const __nv_bfloat16* qrow[2];
#pragma unroll
      for (int h2 = 0; h2 < 2; ++h2) {
        const int r = lane + 32 * h2;
        const int pk = cur.rg * R + r;
        real[h2] = r < NR && r < R && pk < rows_per_head;
        const int g = real[h2] ? pk / p.Tq : 0;
        irow[h2] = real[h2] ? pk - g * p.Tq : 0;
        hrow[h2] = cur.kvh * p.G + g;
        qrow[h2] = static_cast<const __nv_bfloat16*>(p.q) + (int64_t)b * p.q_sb + (int64_t)hrow[h2] * p.q_sh +
                   (int64_t)irow[h2] * p.q_si;
        if (real[h2]) pos[h2] = p.qpos[b * p.qp_sb + irow[h2] * p.qp_si];
      }
      // query rows, 8 in flight (the first unit's are the key threads' work, which
      // have nothing else to do yet: 13 us of the loader's for 48 rows of a cold
      // cache), rows past the unit's end as zeros
      // (a loop: unrolled over 48 rows its code alone took 50 us of the first unit)
      float fac[2] = {0.f, 0.f};
      if (uidx == 0) {
        y0 = fetch(a1);
        y1 = fetch(a2);
        a2 = ask();
      }
#pragma unroll 1
      for (int r0 = uidx == 0 ? NR : 0; r0 < NR; r0 += 8) {
        uint2 w[8];
        const bool high = r0 >= 32;
        const uintptr_t base = reinterpret_cast<uintptr_t>(high ? qrow[1] : qrow[0]);
        const unsigned live = __ballot_sync(0xffffffffu, high ? real[1] : real[0]);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint2* src = reinterpret_cast<const uint2*>(__shfl_sync(0xffffffffu, base, (r0 + i) & 31));
          w[i] = (live >> ((r0 + i) & 31)) & 1 ? __ldg(src + lane) : make_uint2(0, 0);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int r = r0 + i;
          const float f = put_row(qs, r, w[i]);
          if (lane == (r & 31)) {
            if (high) fac[1] = f;
            else fac[0] = f;
          }
        }
      }
      if (uidx == 0) bar_sync(kBarFirst, kKeyThreads + 32);
      // integer facts of the rows
      const int len = len_raw < 0 ? 0 : (len_raw > p.Tmax ? p.Tmax : len_raw);
      RowFacts<NR>& rf = facts0[qb];
      int umax = 0, umin = 0x7fffffff, wmax = 0, ustart = 0x7fffffff;
      uint64_t nodes = 0;
#pragma unroll
      for (int h2 = 0; h2 < 2; ++h2) {
        const int r = lane + 32 * h2;
        if (r >= NR) break;
        int e = 0;
        int64_t oo = 0, lo = 0;
        uint64_t tr = ~0ull;
        if (real[h2]) {
          const int h = hrow[h2], i = irow[h2];
          e = pos[h2] < 0 ? 0 : min(pos[h2], len - 1) + 1;
          if (p.tree != nullptr) tr = (uint64_t)p.tree[(int64_t)b * p.tr_sb + (int64_t)i * p.tr_si];
          if (p.window > 0) {  // the row's first visible key (no overflow: pos >= 0 first)
            tr = (uint64_t)(pos[h2] < 0 ? 0 : max(0, pos[h2] - p.window + 1));
            wmax = max(wmax, (int)tr);
          }
          const int from = p.window > 0 ? (int)tr : 0;
          if (from < e) ustart = min(ustart, from);
          const int within = e - (len - p.Tq);  // nodes before the row's end
          if (p.tree != nullptr && within > 0) nodes |= within < 64 ? tr & ((1ull << within) - 1) : tr;
          oo = (int64_t)b * p.o_sb + (int64_t)h * p.o_sh + (int64_t)i * p.o_si;
          lo = (int64_t)b * p.l_sb + (int64_t)h * p.l_sh + (int64_t)i * p.l_si;
          // (a row that sees nothing takes part in tiles without a mask, with scores of
          // 0, and what comes of it is dropped: the tiles of its unit stay fast)
          if (e > 0) umin = min(umin, e);
          else fac[h2] = 0.f;
        }
        umax = max(umax, e);
        rf.end[r] = e;
        rf.tree[r] = tr;
        if (uidx > 0 || e == 0) rf.fac[r] = fac[h2];
        rf.ooff[r] = oo;
        rf.loff[r] = lo;
      }
      umax = __reduce_max_sync(0xffffffffu, umax);
      umin = __reduce_min_sync(0xffffffffu, umin);
      if (p.window > 0) wmax = __reduce_max_sync(0xffffffffu, wmax);
      ustart = __reduce_min_sync(0xffffffffu, ustart);
      if (p.tree != nullptr)
        nodes = (uint64_t)__reduce_or_sync(0xffffffffu, (unsigned)nodes) |
                (uint64_t)__reduce_or_sync(0xffffffffu, (unsigned)(nodes >> 32)) << 32;
      if (lane == 0) {
        rf.unit_end = umax;
        rf.unit_start = ustart;
        rf.tree_seen = nodes;
        rf.min_end = umin;
        rf.tree_base = p.tree != nullptr ? len - p.Tq : 0x7fffffff;
        rf.win_max = wmax;
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // Q rows -> tensor core
      __syncwarp();
      if (lane == 0) mbar_arrive(&q_full[qb]);
      const int here = min(cur.n - cur.j, t1 - cur.t) * kSub;  // the unit's subtiles of this CTA
      for (int i = 0; ok && i < here; ++i) ok = hand_over();
      if (!ok) break;
    }
    if (!ok && lane == 0) {
      record_error(p.err, kErrTimeout);
      misc[1] = 1;
    }
  } else if (warp == kMmaWarp) {
    // ---------------- MMA issue (one thread) ----------------
    // Order S_0, S_1, U += P_0 V_0, S_2, U += P_1 V_1, ...: the products of
    // the next tile's scores run while the key threads work on this tile.
    if (lane == 0) {
      // The S side runs one tile ahead of the U side.  Per tile only `left`
      // (the unit's tiles of this CTA still to come) counts down; the cursors
      // move from unit to unit.
      auto tiles_here = [&](const Cursor& c) { return c.t < t1 ? min(c.n - c.j, t1 - c.t) : 0; };
      Cursor cq = cur;  // unit of the next S product
      int left_q = tiles_here(cq), left = left_q;
      bool first_q = true, first = true;
      int uq = 0, up = 0;  // unit counters of the S and the U sides
      // Ring positions of the next K (even entries) and V (odd entries)
      // tiles: slot and phase advance by two entries per tile, without
      // divisions on this thread's path.
      struct RingPos {
        uint32_t slot, phase;
        __device__ void adv2() {
          slot += 2;
          if (slot >= (uint32_t)kSlots) {
            slot -= (uint32_t)kSlots;
            phase ^= 1u;
          }
        }
      };
      RingPos kpos{0u, 0u}, vpos{1u, 0u};
      constexpr uint32_t kHi = tc::desc_hi(1024);
      // shared-memory descriptors: only the address word moves per MMA
      const uint32_t qlo0 = tc::desc_lo(sQ, 16);
      auto issue_qk = [&](uint32_t buf) -> bool {
        const int qb = uq & 1;
        if (first_q && !mbar_wait(&q_full[qb], (uint32_t)((uq >> 1) & 1))) return false;
        const uint32_t qlo = qlo0 + (uint32_t)(qb * L::kQBytes >> 4);
#pragma unroll
        for (int x = 0; x < kSub; ++x) {
          const uint32_t ks_slot = kpos.slot;
          if (!mbar_wait(&full[ks_slot], kpos.phase)) return false;
          kpos.adv2();
          tc::fence_after();
          // S^T = K_j Q^T into the S buffer of the tile's parity
          const uint32_t klo = tc::desc_lo(sRing + ks_slot * kSlotBytes, 16);
#pragma unroll
          for (int ks = 0; ks < D / 32; ++ks)
            mma_f8(tb + L::kColS + L::kStepS * buf + L::kSubS * x, tc::desc_join(klo + (uint32_t)(ks * 32 >> 4), kHi),
                   tc::desc_join(qlo + (uint32_t)(ks * 32 >> 4), kHi), kIdescQK, ks > 0 ? 1u : 0u);
          tc::commit(&empty[ks_slot]);  // K_j is free and S_j is ready
        }
        first_q = false;
        if (--left_q == 0) {
          tc::commit(&q_empty[qb]);
          ++uq;
          cq.step_unit(ntab, RG, Hkv, B);
          left_q = tiles_here(cq);
          first_q = true;
        }
        return true;
      };
      bool ok = left_q == 0 || issue_qk(0);
      uint32_t buf = 0, p_phase = 0;  // tile parity, phase of its P^T buffer
      while (ok && left > 0) {
        if (left_q > 0 && !issue_qk(buf ^ 1u)) { ok = false; break; }
        // U^T += V_j^T [p_1 | p_2 | ..]^T once the key threads wrote P^T
        if (!mbar_wait(&p_full[buf], p_phase)) { ok = false; break; }
        const uint32_t ucol = tb + L::kColU + L::kStepU * (uint32_t)(up & 1);
#pragma unroll
        for (int x = 0; x < kSub; ++x) {
          const uint32_t vs_slot = vpos.slot;
          if (!mbar_wait(&full[vs_slot], vpos.phase)) { ok = false; break; }
          vpos.adv2();
          tc::fence_after();
          const uint32_t vlo = tc::desc_lo(sRing + vs_slot * kSlotBytes, 16);
          const uint32_t plo = tc::desc_lo(sP + buf * L::kPBytes + x * L::kPSub, BK * 128);  // (atoms of 128 columns 16 KB apart)
#pragma unroll
          for (int ks = 0; ks < BK / 32; ++ks)
            // A = V^T: 128 dims x keys [32 ks, +32); B = P^T: the same keys x the pieces
            mma_f8(ucol, tc::desc_join(vlo + (uint32_t)(ks * 4096 >> 4), kHi),
                   tc::desc_join(plo + (uint32_t)(ks * 4096 >> 4), kHi), kIdescPV,
                   (!first || x > 0 || ks > 0) ? 1u : 0u);
          tc::commit(&empty[vs_slot]);
        }
        if (!ok) break;
        first = false;
        p_phase ^= buf;
        buf ^= 1u;
        if (--left == 0) {
          tc::commit(&u_full[up & 1]);
          ++up;
          cur.step_unit(ntab, RG, Hkv, B);
          left = tiles_here(cur);
          first = true;
        }
      }
      if (!ok) {
        record_error(p.err, kErrTimeout);
        misc[1] = 1;
      }
      // every MMA issued must complete before TMEM is released
      tc::commit(drain);
      if (!mbar_wait(drain, 0)) {
        record_error(p.err, kErrTimeout);
        misc[1] = 1;
      }
    }
  } else {
    // ---------------- key threads ----------------
    // warp w: TMEM lane quarter (w mod 4) and group w / 4: thread = key k of the
    // group's subtile with the group's part of the rows, [c0, c0 + NH); value dim k in
    // the epilogue, with the same rows (the first subtile's groups)
    constexpr int NH = NR / L::kParts;
    constexpr int kRed = 4 * kSub;  // warps that share a row's maximum
    const int quarter = warp & 3;
    const int group = warp >> 2;
    const int k = 32 * quarter + lane;
    const int sub = group % kSub, part = group / kSub;
    const int c0 = part * NH;
    const bool has_u = sub == 0;
    const int red_row = quarter + 4 * sub;
    const uint32_t tl = tb + ((uint32_t)(32 * quarter) << 16);
    auto wait_all = [&](uint64_t* bar, uint32_t parity) -> bool {
      return __all_sync(0xffffffffu, mbar_wait(bar, parity));
    };
    if (cur.t < t1) {  // the first unit's query rows, a warp a row
      constexpr int kOwn = NR / kKeyWarps;
      static_assert(NR % kKeyWarps == 0, "rows of a warp");
      uint2 w[kOwn];
#pragma unroll
      for (int i = 0; i < kOwn; ++i) {
        const int r = warp + kKeyWarps * i, pk = cur.rg * R + r, g = pk / p.Tq;
        w[i] = make_uint2(0, 0);
        if (r < R && pk < rows_per_head)
          w[i] = __ldg(reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p.q) + (int64_t)cur.b * p.q_sb +
                                                      (int64_t)(cur.kvh * p.G + g) * p.q_sh + (int64_t)(pk - g * p.Tq) * p.q_si) +
                       lane);
      }
#pragma unroll
      for (int i = 0; i < kOwn; ++i) {
        const int r = warp + kKeyWarps * i;
        const float f = put_row(sm + L::kOffQ, r, w[i]);
        if (lane == 0) facts0[0].fac[r] = f;
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // Q rows -> tensor core
      asm volatile("bar.arrive %0, %1;" ::"n"(kBarFirst), "n"(kKeyThreads + 32) : "memory");
    }
    // R of a state at m as it is at a common m
    auto moved = [](float r, float m, float common) { return m == common ? r : r + (m - common); };
    float lp[NH];  // this thread's partial sums of P over its keys
#pragma unroll
    for (int r = 0; r < NH; ++r) lp[r] = 0.f;
    int uidx = 0;
    bool ok = true;
    auto put_out = [&](int64_t at, float o) { static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(o); };
    // A finished unit's U is read one tile later, after the next tile's P: by then
    // its last product has completed and the readout does not stall the pipeline.
    // Its statistics wait in s_mfin, .., its row facts stay in their buffer until
    // the readout releases them.
    bool pend = false;
    int pend_uidx = 0, pend_b = 0, pend_kvh = 0, pend_rg = 0, pend_n = 1;
    int pend_su = 0;
    auto flush = [&]() -> bool {
      const int pb = pend_uidx & 1;
      const RowFacts<NR>& pf = facts0[pb];
      if (!bar_and(kBarRows, kKeyThreads, wait_all(&u_full[pb], (uint32_t)((pend_uidx >> 1) & 1)))) return false;
      tc::fence_after();
      float u[NH];
      if (has_u) {
        const uint32_t ua = tl + L::kColU + L::kStepU * (uint32_t)pb + c0;
        ld_cols<NH>(ua + (kPieces - 1) * NR, u);
#pragma unroll
        for (int c = kPieces - 2; c >= 0; --c) {  // U = U_1 + (U_2 + ..) / 2^8
          float hi[NH];
          ld_cols<NH>(ua + c * NR, hi);
#pragma unroll
          for (int r = 0; r < NH; ++r) u[r] = fmaf(u[r], c > 0 ? 0x1p-2f : 0x1p-4f, hi[r]);
        }
      }
      const int64_t unit = ((int64_t)pend_b * Hkv + pend_kvh) * RG + pend_rg;
      const int cf = cta_of(pend_su, W, P_work);
      const int nparts = cta_of(pend_su + pend_n - 1, W, P_work) - cf + 1;
      const int64_t slots = (int64_t)gridDim.x + (int64_t)B * Hkv * RG;
      float* ws_m = p.ws;
      float* ws_l = ws_m + slots * R;
      float* ws_r = ws_l + slots * R;
      float* ws_u = ws_m + (3 * slots * R + 3) / 4 * 4;
      const int rr = min(R, rows_per_head - pend_rg * R);  // real rows of the unit
      if (nparts == 1) {
#pragma unroll
        for (int r = 0; r < NH; ++r) {
          const int row = c0 + r;
          if (row >= rr || !has_u) break;
          // (two factors: the power of two may pass fp32's range)
          const float f = s_lfin[row] == 0.f ? 0.f : fast_exp2(0.5f * s_rfin[row]);
          put_out(pf.ooff[row] + (int64_t)k * p.o_sd, s_lfin[row] == 0.f ? 0.f : u[r] * f * s_inv[row] * f);
        }
        if (group == 0 && k < rr)
          p.lse[pf.loff[k]] = s_lfin[k] == 0.f ? kNegInf : (s_mfin[k] + __log2f(s_lfin[k])) * kLn2;
      } else {
        // (kept in L2 until the fold reads it: the key stream passing through
        // meanwhile is marked evict-first)
        const uint64_t keep = policy_evict_last();
        // this CTA's partial state of the unit, then the last of the unit's CTAs to
        // get here folds all of them, in CTA order
        const int64_t slot = (int64_t)blockIdx.x + unit;
#pragma unroll
        for (int r = 0; r < NH; ++r) {
          const int row = c0 + r;
          if (row >= rr || !has_u) break;
          st_global_hint(ws_u + ((slot * R + row) * D) + k, u[r], keep);
        }
        if (group == 0 && k < rr) {
          st_global_hint(ws_m + slot * R + k, s_mfin[k], keep);
          st_global_hint(ws_l + slot * R + k, s_lfin[k], keep);
          st_global_hint(ws_r + slot * R + k, s_rfin[k], keep);
        }
        bar_sync(kBarRows, kKeyThreads);
        if (threadIdx.x == 0) {
          // one thread's fences order all: the barriers before and after it carry
          // the other threads' stores and loads
          __threadfence();  // the partial state is visible before the count says so
          misc[3] = (atomicAdd(&p.cnt[unit], 1u) == (unsigned)(nparts - 1)) ? 1 : 0;
          __threadfence();  // the other parts are read after the count
        }
        bar_sync(kBarRows, kKeyThreads);
        if (misc[3] != 0) {
          if (threadIdx.x == 0) p.cnt[unit] = 0u;  // ready for the next launch
          const int64_t fs = cf + unit;  // the unit's first slot; its parts are consecutive
          // items (row, 4 value dims) over the key threads, the parts in batches of
          // 4: all loads of a batch in flight
          constexpr int kBatch = 4;
          for (int item = threadIdx.x; item < rr * (D / 4); item += kKeyThreads) {
            const int row = item / (D / 4), d4 = item % (D / 4);
            float M = kNegInf, Ls = 0.f, Rs = kNegInf;
            float4 Us = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int s0 = 0; s0 < nparts; s0 += kBatch) {
              float ms[kBatch], ls[kBatch], rs[kBatch];
              float4 us[kBatch];
#pragma unroll
              for (int e = 0; e < kBatch; ++e) {
                ms[e] = rs[e] = kNegInf;
                ls[e] = 0.f;
                us[e] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (s0 + e < nparts) {
                  const int64_t idx = (fs + s0 + e) * R + row;
                  ms[e] = __ldcg(ws_m + idx);
                  ls[e] = __ldcg(ws_l + idx);
                  rs[e] = __ldcg(ws_r + idx);
                  us[e] = __ldcg(reinterpret_cast<const float4*>(ws_u + idx * D) + d4);
                }
              }
#pragma unroll
              for (int e = 0; e < kBatch; ++e) {
                const float m = fmaxf(M, ms[e]);
                const float ra = moved(Rs, M, m), rb = moved(rs[e], ms[e], m);
                Ls = Ls * (M == m ? 1.f : fast_exp2(M - m)) + ls[e] * (ms[e] == m ? 1.f : fast_exp2(ms[e] - m));
                M = m;
                Rs = fmaxf(ra, rb);
                const float ca = ra == Rs ? 1.f : fast_exp2(ra - Rs), cb = rb == Rs ? 1.f : fast_exp2(rb - Rs);
                Us.x = fmaf(Us.x, ca, cb * us[e].x);
                Us.y = fmaf(Us.y, ca, cb * us[e].y);
                Us.z = fmaf(Us.z, ca, cb * us[e].z);
                Us.w = fmaf(Us.w, ca, cb * us[e].w);
              }
            }
            const bool none = Ls == 0.f;  // (a part of NaN leaves its trace in the sum)
            const float f = none ? 0.f : fast_exp2(0.5f * Rs), inv = none ? 0.f : 1.f / Ls;
            const float o4[4] = {Us.x * f * inv * f, Us.y * f * inv * f, Us.z * f * inv * f, Us.w * f * inv * f};
#pragma unroll
            for (int e = 0; e < 4; ++e)
              put_out(pf.ooff[row] + (int64_t)(4 * d4 + e) * p.o_sd, none ? 0.f : o4[e]);
            if (d4 == 0) p.lse[pf.loff[row]] = none ? kNegInf : (M + __log2f(Ls)) * kLn2;
          }
        }
      }
      bar_sync(kBarRows, kKeyThreads);  // the finished unit's statistics and row facts are read
      if (threadIdx.x == 0) mbar_arrive(&q_empty[pb]);
      return true;
    };
    // A key that no row of the unit sees, past every end, before the windows or a
    // tree node that no row lists: its rows and scales may hold anything.
    auto unseen = [](const RowFacts<NR>& rf, int key) {
      const int node = key - rf.tree_base;
      return key >= rf.unit_end || key < rf.unit_start ||
             (rf.tree_base != 0x7fffffff && node >= 0 && node < 64 && !((rf.tree_seen >> node) & 1ull));
    };
    // rows' maxima of v over the tile's keys: red[..][row]
    auto tile_max = [&](const float (&v)[NH]) {
      float t[NH];
#pragma unroll
      for (int r = 0; r < NH; ++r) t[r] = v[r];
      warp_reduce_scatter<NH, true>(t, lane);
      if ((lane & 3) == 0) {
        const int base = scatter_base<NH>(lane);
#pragma unroll
        for (int i = 0; i < NH / 8; ++i) red[red_row * NR + c0 + base + i] = t[i];
      }
    };
    auto red_max = [&](int row) {
      float m = red[row];
#pragma unroll
      for (int w = 1; w < kRed; ++w) m = fmaxf(m, red[w * NR + row]);
      return m;
    };
    uint32_t kslot = 2 * sub, kphase = 0;  // ring slot of the current K subtile and its phase
    for (int g = 0; cur.t < t1; cur.next(ntab, RG, Hkv, B), ++g) {
      const bool first = cur.t == t0 || cur.j == 0;
      const bool last = cur.t == t1 - 1 || cur.j == cur.n - 1;
      const int ub = uidx & 1;
      const RowFacts<NR>& rf = facts0[ub];
      if (L::kBufU == 1 && pend) {
        if (!flush()) { ok = false; break; }
        pend = false;
      }
      if (first) {
        // the row facts come with the query rows
        const bool w = bar_and(kBarRows, kKeyThreads, wait_all(&q_full[ub], (uint32_t)((uidx >> 1) & 1)));
        if (!w) { ok = false; break; }
      }
      const int key0 = cur.key0();
      const int sub0 = key0 + sub * BK, key = sub0 + k;
      const int gs = kSub * g + sub;  // the subtile, of this CTA's
      float x[NH];
      float ks = 0.f, ev = kNegInf;  // the key's scales: 2^ks', 2^ev
      bool sok = wait_all(&sc_full[gs % kScaleRing], (uint32_t)((gs / kScaleRing) & 1));
      if (sok) {
        const uint32_t sc = s_sc[(gs % kScaleRing) * BK + k];
        if (sc != 0) {
          const int e = (sc >> 8) & 255;
          ks = scale_of(sc & 255);
          ev = e < 255 ? (float)(e - 127) : (unseen(rf, key) ? 0.f : __uint_as_float(0x7fc00000u));
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sc_empty[gs % kScaleRing]);
        sok = wait_all(&empty[kslot], kphase);
      }
      bool trig = !sok;
      // 2^ev in two factors, around the row's 2^(lift - r): whatever the exponents are,
      // the weights between stay in fp32's range (five-row chains of 64 heads 110 us with
      // one factor, 117 so)
      const float half = floorf(0.5f * ev);
      const float f1 = ev == kNegInf ? 0.f : fast_exp2(half), f2 = ev == kNegInf ? 0.f : fast_exp2(ev - half);
      float pr[NH];         // the weights e^z at m's reference
      uint32_t w2[NH / 2];  // with the values' scales, at r's, pairs of rows as f16
      float z_max = kNegInf;  // above 0: some m has to rise
      auto weigh = [&]() {
        const float2 fa = make_float2(f1, f1), fb = make_float2(f2, f2), neg = make_float2(-1.f, -1.f);
#pragma unroll
        for (int r4 = 0; r4 < NH / 4; ++r4) {
          const float4 m4 = reinterpret_cast<const float4*>(s_muse + c0)[r4];
          const float4 h4 = reinterpret_cast<const float4*>(s_h + c0)[r4];
          const float2 mu[2] = {make_float2(m4.x, m4.y), make_float2(m4.z, m4.w)};
          const float2 h[2] = {make_float2(h4.x, h4.y), make_float2(h4.z, h4.w)};
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int r = 4 * r4 + 2 * e;
            const float2 z = __ffma2_rn(mu[e], neg, make_float2(x[r], x[r + 1]));
            z_max = max3(z_max, z.x, z.y);
            const float2 pp = make_float2(fast_exp2(z.x), fast_exp2(z.y));  // masked: 2^-inf = 0
            pr[r] = pp.x;
            pr[r + 1] = pp.y;
            const float2 w = __fmul2_rn(__fmul2_rn(__fmul2_rn(pp, fa), h[e]), fb);
            const __half2 h2 = __floats2half2_rn(w.x, w.y);
            w2[r / 2] = *reinterpret_cast<const uint32_t*>(&h2);
          }
        }
      };
      if (sok) {
        tc::fence_after();
        float lo[NH];
        const uint32_t sa = tl + L::kColS + L::kStepS * (uint32_t)(g & 1) + L::kSubS * sub + c0;
        ld_cols<NH>(sa, x);
        ld_cols<NH>(sa + NR, lo);
        const float2 low = make_float2(0.03125f, 0.03125f), ks2 = make_float2(ks, ks);
#pragma unroll
        for (int r4 = 0; r4 < NH / 4; ++r4) {
          const float4 f4 = reinterpret_cast<const float4*>(rf.fac + c0)[r4];
          const float2 fc[2] = {make_float2(f4.x, f4.y), make_float2(f4.z, f4.w)};
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int r = 4 * r4 + 2 * e;
            const float2 v = __ffma2_rn(make_float2(lo[r], lo[r + 1]), low, make_float2(x[r], x[r + 1]));
            const float2 xx = __fmul2_rn(v, __fmul2_rn(ks2, fc[e]));
            x[r] = xx.x;
            x[r + 1] = xx.y;
          }
        }
        // (every row sees every key of the subtile: no mask)
        if (sub0 + BK > rf.min_end || sub0 < rf.win_max || sub0 + BK > rf.tree_base || ev == kNegInf) {
          // row ends, windows, trees, keys without a page
          const int node = key - rf.tree_base;
          const bool in_tree = rf.tree_base != 0x7fffffff && node >= 0 && node < 64;
          const bool window = p.window > 0;
          const int last_key = ev == kNegInf ? 0x7fffffff : key;
#pragma unroll
          for (int r = 0; r < NH; ++r) {
            const uint64_t t = rf.tree[c0 + r];
            if (last_key >= rf.end[c0 + r] || (window && key < (int)t) || (in_tree && !((t >> node) & 1ull))) x[r] = kNegInf;
          }
        }
      } else if (lane == 0) {
        misc[2] = 1;
      }
      bool resc = false;
      for (bool again = false;; again = true) {
        weigh();
        if (again) break;
        trig |= z_max > 0.f;
        if (trig) misc[4 + (int)(g & 1)] = 1;  // m has to rise (read after the vote's barrier)
        __half2 top = *reinterpret_cast<const __half2*>(&w2[0]);
#pragma unroll
        for (int i = 1; i < NH / 2; ++i) top = __hmax2(top, *reinterpret_cast<const __half2*>(&w2[i]));
        trig |= __high2float(top) > kMostW || __low2float(top) > kMostW;
        if (!bar_or(kBarRows, kKeyThreads, trig)) break;
        if (misc[2] != 0) { ok = false; break; }  // read after the barrier: same answer everywhere (both loops end)
        // ---- raise the references: m, then r at the new m ----
        const bool raise_m = misc[4 + (int)(g & 1)] != 0;
        if (raise_m) {
          tile_max(x);
          bar_sync(kBarRows, kKeyThreads);
          if (group == 0 && k < NR) {
            const float tmax = red_max(k);
            const float mo = s_m[k];
            float a = 1.f;
            if (tmax > mo) {
              const float mn = tmax + kMarginM;
              a = mo == kNegInf ? 1.f : fast_exp2(mo - mn);  // a row with no key yet has l = u = 0
              s_r[k] = mo == kNegInf ? kNegInf : s_r[k] + (mo - mn);
              s_m[k] = mn;
              s_muse[k] = mn;
            }
            s_alpha[k] = a;
          }
          if (threadIdx.x == 0) misc[4 + (int)(g & 1)] = 0;  // (its next use is two tiles on)
          bar_sync(kBarRows, kKeyThreads);
        }
        {
          float y[NH];
#pragma unroll
          for (int r = 0; r < NH; ++r) y[r] = x[r] == kNegInf ? kNegInf : x[r] - s_muse[c0 + r] + ev;
          tile_max(y);
        }
        bar_sync(kBarRows, kKeyThreads);
        if (group == 0 && k < NR) {
          const float ymax = red_max(k), ro = s_r[k];
          float bt = 1.f, rn = ro;
          // (r fell with m: what it may rise to is measured from there)
          if (ymax > ro) rn = ymax + kMargin;
          if (rn != kNegInf) rn = fminf(fmaxf(rn, kLeastR), kMostR);
          if (rn != ro) bt = ro == kNegInf ? 1.f : fast_exp2(ro - rn);
          // U's reference in absolute terms moved by bt, and not by m's step
          s_r[k] = rn;
          s_h[k] = rn == kNegInf ? 1.f : fast_exp2(kLift - rn);
          s_beta[k] = bt;
        }
        bar_sync(kBarRows, kKeyThreads);
        if (raise_m) {
#pragma unroll
          for (int r4 = 0; r4 < NH / 4; ++r4) {
            const float4 a4 = reinterpret_cast<const float4*>(s_alpha + c0)[r4];
            lp[4 * r4] *= a4.x;
            lp[4 * r4 + 1] *= a4.y;
            lp[4 * r4 + 2] *= a4.z;
            lp[4 * r4 + 3] *= a4.w;
          }
        }
        if (!first) {
          // U^T lane k = value dim k, the group's columns of all pieces; the product
          // with P_{j-1} must have completed (U += P_j V_j waits for this tile's P)
          const int pv_seq = 2 * kSub * g - 1;  // V_{j-1}, its last subtile
          const bool done = wait_all(&empty[pv_seq % kSlots], (uint32_t)((pv_seq / kSlots) & 1));
          const bool pv = bar_and(kBarRows, kKeyThreads, done);
          if (!pv) { ok = false; break; }  // (both loops)
          tc::fence_after();
          const uint32_t ua = tl + L::kColU + L::kStepU * (uint32_t)ub + c0;
#pragma unroll 1
          for (int c = 0; has_u && c < kPieces; ++c) {
            float u[NH];
            ld_cols<NH>(ua + NR * c, u);
#pragma unroll
            for (int r = 0; r < NH; ++r) u[r] *= s_beta[c0 + r];
            st_cols<NH>(ua + NR * c, u);
          }
          resc = has_u;
        }
      }
      if (!ok) break;
      // ---- P^T row of key k, the group's rows: the weights' pieces, exact ----
      {
        unsigned char* ph = sm + L::kOffP + (int)(g & 1) * L::kPBytes + sub * L::kPSub + k * 128;
#pragma unroll
        for (int r = 0; r < NH; ++r) lp[r] += pr[r];
#pragma unroll
        for (int c = 0; c < kPieces; ++c) {
          uint32_t by[NH / 4];  // the upper bytes, four rows a word
#pragma unroll
          for (int i = 0; i < NH / 4; ++i) by[i] = __byte_perm(w2[2 * i], w2[2 * i + 1], 0x7531);
          if (c < kPieces - 1) {
#pragma unroll
            for (int i = 0; i < NH / 2; ++i) {  // the rest
              const uint32_t top = w2[i] & 0xff00ff00u;
              __half2 rest = __hsub2(*reinterpret_cast<const __half2*>(&w2[i]), *reinterpret_cast<const __half2*>(&top));
              rest = __hmul2(rest, __float2half2_rn(c == 0 ? 16.f : 4.f));
              w2[i] = *reinterpret_cast<const uint32_t*>(&rest);
            }
          }
          const int n0 = c * NR + c0;  // column of the first row
          if constexpr (NH == 16) {
            unsigned char* at = ph + (n0 >= 128 ? BK * 128 : 0) + ((((n0 & 127) >> 4) ^ (k & 7)) << 4);
            *reinterpret_cast<uint4*>(at) = make_uint4(by[0], by[1], by[2], by[3]);
          } else {
#pragma unroll
            for (int i = 0; i < NH / 8; ++i) {
              const int n = n0 + 8 * i;
              unsigned char* at = ph + (n >= 128 ? BK * 128 : 0) + ((((n & 127) >> 4) ^ (k & 7)) << 4) + (n & 8);
              *reinterpret_cast<uint2*>(at) = make_uint2(by[2 * i], by[2 * i + 1]);
            }
          }
        }
      }
      if ((cur.j == cur.n - 1 && key0 + TK > rf.unit_end) || key0 < rf.unit_start || key0 + TK > rf.tree_base) {
        // zero the V rows that no row sees (one group of each subtile)
        const int sv = 2 * gs + 1;
        const bool vok = bar_and(kBarRows, kKeyThreads, wait_all(&full[sv % kSlots], (uint32_t)((sv / kSlots) & 1)));
        if (!vok) { ok = false; break; }
        if (unseen(rf, key) && part == 0) {
          unsigned char* vr = sm + (int)(sv % kSlots) * kSlotBytes + k * 128;
#pragma unroll
          for (int c = 0; c < 8; ++c) *reinterpret_cast<uint4*>(vr + (c << 4)) = make_uint4(0, 0, 0, 0);
        }
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // P^T, V rows -> tensor core
      if (resc) tc::wait_st();
      tc::fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_full[g & 1]);
      kslot += 2 * kSub;
      if (kslot >= (uint32_t)kSlots) {
        kslot -= (uint32_t)kSlots;
        kphase ^= 1u;
      }

      // the U readout of the previous unit (its last product has long
      // completed by now)
      if (pend) {
        if (!flush()) { ok = false; break; }
        pend = false;
      }
      if (last) {
        // ---- close the unit (or this CTA's part of it): l over the keys ----
        warp_reduce_scatter<NH, false>(lp, lane);
        if ((lane & 3) == 0) {
          const int base = scatter_base<NH>(lane);
#pragma unroll
          for (int i = 0; i < NH / 8; ++i) red[red_row * NR + c0 + base + i] = lp[i];
        }
#pragma unroll
        for (int r = 0; r < NH; ++r) lp[r] = 0.f;
        bar_sync(kBarRows, kKeyThreads);
        if (group == 0 && k < NR) {
          float l = red[k];
#pragma unroll
          for (int w = 1; w < kRed; ++w) l += red[w * NR + k];
          if (rf.end[k] == 0) l = 0.f;  // (sees nothing)
          // (a NaN among a row's scores, which no maximum shows, is in the sum)
          s_mfin[k] = s_m[k];
          s_lfin[k] = l;
          s_rfin[k] = s_r[k] - kLift;
          s_inv[k] = l == 0.f ? 0.f : 1.f / l;
          // fresh statistics for the next unit
          s_m[k] = kNegInf;
          s_muse[k] = kNoM;
          s_r[k] = kNegInf;
          s_h[k] = 1.f;
        }
        bar_sync(kBarRows, kKeyThreads);
        pend = true;
        pend_uidx = uidx;
        pend_su = cur.su;
        pend_b = cur.b;
        pend_kvh = cur.kvh;
        pend_rg = cur.rg;
        pend_n = cur.n;
        ++uidx;
      }
    }
    if (ok && pend && !flush()) ok = false;
    if (!ok && lane == 0) record_error(p.err, kErrTimeout);
  }

  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (warp == kMmaWarp) tc::dealloc(tb, kTmemCols);
}

template <int NR>
cudaError_t launch(const Q8Params& p, int ctas, const CUtensorMap& tmk, const CUtensorMap& tmv, cudaStream_t stream) {
  using L = TcLayout<NR>;
  static DeviceOnce once;
  if (cudaError_t e = once.set_smem(reinterpret_cast<const void*>(&decode_tc_q8_kernel<NR>), L::kBytes);
      e != cudaSuccess)
    return e;
  decode_tc_q8_kernel<NR><<<ctas, L::kThreads, L::kBytes, stream>>>(p, tmk, tmv);
  return cudaGetLastError();
}

}  // namespace

Q8Plan plan_decode_tc_q8(int64_t B, int64_t Hkv, int64_t rows, int64_t Tmax, int sms) {
  Q8Plan pl;
  pl.row_groups = (rows + 47) / 48;
  pl.rows_cta = (int)((rows + pl.row_groups - 1) / pl.row_groups);
  pl.ctas = sms < 255 ? sms : 255;
  pl.units = B * Hkv * pl.row_groups;
  pl.tiles = pl.units * ((Tmax + 127) / 128 + 2);  // + the per-unit weight; at most
  pl.ws_bytes = (size_t)((pl.ctas + pl.units) * pl.rows_cta * (3 + D) + 4) * sizeof(float);
  return pl;
}

bool decode_tc_q8_takes(const Q8Plan& pl, int64_t B, int64_t Tmax) {
  // (16-bit tile counts, 32-bit arithmetic of the cut)
  return B * pl.row_groups <= kDecodeTcMaxEntries && Tmax <= 65535LL * 128 && pl.tiles < (1LL << 24);
}

cudaError_t launch_decode_tc_q8(const Q8Params& p, int ctas, const CUtensorMap& tmk, const CUtensorMap& tmv,
                                cudaStream_t stream) {
  if (p.rows_cta <= 8) return launch<8>(p, ctas, tmk, tmv, stream);
  if (p.rows_cta <= 16) return launch<16>(p, ctas, tmk, tmv, stream);
  if (p.rows_cta <= 32) return launch<32>(p, ctas, tmk, tmv, stream);
  return launch<48>(p, ctas, tmk, tmv, stream);
}

}  // namespace blkattn
