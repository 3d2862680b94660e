// Rotary positions: rows rotated by their logical position, forward and
// backward, and appended to a paged KV cache with the rotation on the way.
//
// Pair i of a row's rotated dims turns by t w_i at position t:
//
//     (y_a, y_b) = mscale (x_a cos - x_b sin, x_a sin + x_b cos)
//
// and the gradient turns back by the same angle (the map is mscale times a
// rotation, so its transpose is mscale times the inverse rotation).  The
// angles come as phases F_i = round(2^64 w_i / 2 pi): the product t F_i mod
// 2^64 is t w_i in units of 2^-64 turns with whole turns dropped, exactly, so
// a position near 2^31 loses no more than one near 0 (the table's rounding
// grows to |t| 2^-65 turns).  Its top 32 bits as a float go to sincospif: the
// bits dropped are less than 2^-32 turns, and the float is off by at most
// 2^-24 of the angle (|angle| <= pi).
// All arithmetic is fp32; the only rounding to fewer bits is the store.
//
// One kernel serves every operator: up to three row sets (append: k, v, q)
// with their own source, destination, heads and whether they turn.
#include <cuda_bf16.h>

#include <cmath>
#include <cstdint>

#include "kernels.h"
#include "paged.h"
#include "ptx.cuh"
#include "rotary.cuh"

namespace blkattn {
namespace {

struct RowSet {
  const void* src;
  int64_t s_b, s_h, s_t, s_d;  // element strides
  void* dst;
  int64_t d_b, d_h, d_t, d_d;  // dense: batch, head, row, dim; paged: page, head, row in page, dim
  int heads;
  bool turn;   // false: rows are copied
  bool paged;  // destination rows follow the page table
};

struct RotaryParams {
  RowSet set[3];
  int n_sets;
  const int32_t* pos;
  int64_t p_b, p_t;
  const int64_t* phases;
  int64_t ph_s;
  bool back;           // turn by the negative angle
  bool skip_negative;  // append: rows at a negative position are padding
  float mscale;
  int rot, d;
  int B, T;
  int hg;         // heads of a thread
  int groups[3];  // ceil(heads / hg) of each set
  PageTable pages;
};

constexpr int kThreads = 256;
constexpr int kRegHeads = 4;  // V < 8: heads whose loads a thread has in flight
// Blocks below which a thread takes fewer heads, so that every SM has its
// threads: 152 SMs of four blocks (the kernels' registers; the slots of up to
// six heads; eight heads' 64 KB allow three)
constexpr int kFillBlocks = 152 * 4;

// Runs of 16 bytes go through slots in shared memory, shorter ones through
// registers.
template <typename TI, int V>
constexpr bool kSlots = sizeof(TI) * V == 16;
constexpr int kMostHeads = 8;  // heads of one thread: 64 KB of slots a block

// One thread turns one item of a token's rows, in `hg` heads: two runs of V
// dims, one from each half of the rotated part (HALF: V pairs across them;
// INTERLEAVED: V / 2 pairs within each), or copies two runs of the dims past
// it.  Runs from the two halves, not 2 V neighbours: with these a warp's
// 16-byte accesses would touch every second half of a sector (measured on
// bf16 rows of 128, INTERLEAVED: 36.5 us with neighbours against 32.4).
// Angles depend on the token and the pair alone,
// so a thread takes its V sines and cosines once and walks its heads with
// them in registers.  Consecutive threads hold consecutive items, then the
// next token: a warp moves whole 128-byte lines.
//
// What bounds it is memory: an SM needs some 50 KB in flight to stream at the
// card's rate.  Runs of 16 bytes (8 bf16, 4 f32) are copied to slots of the
// thread's own in shared memory, all its heads' at once (asynchronous copies:
// no register holds them, no other thread reads them), and the sines are
// taken while they land.  Measured, bf16 rows of 2 x 8192 tokens x 32 heads:
// 45 us, 90 % of the copy bandwidth; with the runs in registers instead 63 us
// (four heads in flight take over 128 registers and leave one block an SM,
// two leave too few bytes in flight); the f32 to bf16 gradient 60.5 us, 99 %,
// against 64 us in registers.
template <typename TI, typename TO, int V, bool INTER>
__global__ void __launch_bounds__(kThreads, kSlots<TI, V> ? 4 : 1) rotary_kernel(const __grid_constant__ RotaryParams p) {
  // blockIdx.y: the row set and its group of heads
  int grp = blockIdx.y, si = 0;
  while (grp >= p.groups[si]) grp -= p.groups[si++];
  const RowSet& s = p.set[si];
  const int h0 = grp * p.hg, nh = min(p.hg, s.heads - h0);
  const int rot = s.turn ? p.rot : 0;
  const int items = (p.d + 2 * V - 1) / (2 * V);  // (an odd d only with V = 1)
  const int64_t n = (int64_t)p.B * p.T * items;
  const int64_t u = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (u >= n) return;
  int tok, it;  // B T < 2^31
  if (n <= 0x7fffffff) {  // (a 64-bit division is a long sequence)
    tok = (int)((unsigned)u / (unsigned)items);
    it = (int)u - tok * items;
  } else {
    tok = (int)(u / items);
    it = (int)(u - (int64_t)tok * items);
  }
  const int b = tok / p.T;
  const int t = tok - b * p.T;
  const bool turn = it < rot / (2 * V);
  // the item's two runs of V dims (single dims of an INTERLEAVED pair are
  // neighbours)
  const int part0 = turn ? 0 : rot, part = turn ? rot : p.d - rot;  // of the row
  const int i = it - part0 / (2 * V);                               // item within the part
  const int a0 = part0 + (V > 1 || (turn && !INTER) ? V * i : 2 * i);
  const int a1 = V > 1 || (turn && !INTER) ? a0 + part / 2 : a0 + 1;
  const bool second = V > 1 || a1 < p.d;
  const TI* src = static_cast<const TI*>(s.src) + (b * s.s_b + t * s.s_t + h0 * s.s_h);
  TO* dst = static_cast<TO*>(s.dst) + h0 * s.d_h;
  if (!turn && !s.paged && s.src == s.dst) return;  // in place: nothing to copy
  const int pos = p.pos[b * p.p_b + t * p.p_t];
  if (p.skip_negative && pos < 0) return;  // (before the rows' loads: padding costs no traffic)
  if (s.paged) {
    const int page = page_of(p.pages, b, pos);
    if (page < 0) return;
    dst += page * s.d_b + (pos & (p.pages.rows - 1)) * s.d_t;
  } else {
    dst += b * s.d_b + t * s.d_t;
  }
  float sn[V], cs[V];
  auto angles = [&]() {
    if (!turn) return;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      // pair j of the item
      const int pair = !INTER || V == 1 ? V * it + j : (j < V / 2 ? a0 / 2 + j : a1 / 2 + j - V / 2);
      turn_of(pos, p.phases[pair * p.ph_s], sn[j], cs[j]);
      sn[j] *= p.back ? -p.mscale : p.mscale;
      cs[j] *= p.mscale;
    }
  };
  if constexpr (kSlots<TI, V>) {
    extern __shared__ __align__(16) unsigned char slots[];
    // run r of head k: slot (2 k + r) kThreads + thread (conflict-free)
    uint4* mine = reinterpret_cast<uint4*>(slots) + threadIdx.x;
#pragma unroll
    for (int k = 0; k < kMostHeads; ++k) {
      if (k < nh) {
        const TI* r = src + k * s.s_h;
        cp_async_16(smem_u32(mine + 2 * k * kThreads), r + a0, 16);
        cp_async_16(smem_u32(mine + (2 * k + 1) * kThreads), r + a1, 16);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    }
    angles();
#pragma unroll
    for (int k = 0; k < kMostHeads; ++k) {
      wait_copies(kMostHeads - 1 - k);
      if (k < nh) {
        Vec<TI, V> x0, x1;
        reinterpret_cast<uint4&>(x0) = mine[2 * k * kThreads];
        reinterpret_cast<uint4&>(x1) = mine[(2 * k + 1) * kThreads];
        Vec<TO, V> y0, y1;
        turn_run<TI, TO, V, INTER>(x0, x1, turn, sn, cs, y0, y1);
        TO* r = dst + k * s.d_h;
        store(r + a0, y0);
        store(r + a1, y1);
      }
    }
  } else {
    Vec<TI, V> x0[kRegHeads], x1[kRegHeads];
    auto load_heads = [&](int h) {
#pragma unroll
      for (int k = 0; k < kRegHeads; ++k)
        if (h + k < nh) {
          const TI* r = src + (h + k) * s.s_h;
          x0[k] = *reinterpret_cast<const Vec<TI, V>*>(r + a0 * s.s_d);
          if (second) x1[k] = *reinterpret_cast<const Vec<TI, V>*>(r + a1 * s.s_d);
        }
    };
    load_heads(0);
    angles();
    for (int h = 0; h < nh; h += kRegHeads) {
      if (h > 0) load_heads(h);
#pragma unroll
      for (int k = 0; k < kRegHeads; ++k)
        if (h + k < nh) {
          Vec<TO, V> y0, y1;
          turn_run<TI, TO, V, INTER>(x0[k], x1[k], turn, sn, cs, y0, y1);
          TO* r = dst + (h + k) * s.d_h;
          store(r + a0 * s.d_d, y0);
          if (second) store(r + a1 * s.d_d, y1);
        }
    }
  }
}

template <typename TI, typename TO, int V, bool INTER>
cudaError_t launch_v(RotaryParams p, cudaStream_t stream) {
  const int64_t n = (int64_t)p.B * p.T * ((p.d + 2 * V - 1) / (2 * V));
  const int64_t blocks = (n + kThreads - 1) / kThreads;
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;  // (more elements than the card holds)
  // Heads of a thread: enough that the sines cost little, few enough that
  // every SM has its threads
  int most = 0;
  for (int i = 0; i < p.n_sets; ++i) most = p.set[i].heads > most ? p.set[i].heads : most;
  const int64_t want = (kFillBlocks + blocks - 1) / blocks;  // groups that fill the machine
  int64_t hg = (most + want - 1) / want;
  p.hg = (int)(hg < 1 ? 1 : (hg > kMostHeads ? kMostHeads : hg));
  auto count_groups = [&]() {
    int n = 0;
    for (int i = 0; i < p.n_sets; ++i) n += p.groups[i] = (p.set[i].heads + p.hg - 1) / p.hg;
    return n;
  };
  int groups = count_groups();
  if (groups > 65535) {  // (grid y; at most 98301 heads)
    p.hg = kMostHeads;
    groups = count_groups();
  }
  const int smem = kSlots<TI, V> ? p.hg * 32 * kThreads : 0;
  if (smem > 48 * 1024) {
    static DeviceOnce once;
    if (cudaError_t e = once.set_smem(reinterpret_cast<const void*>(&rotary_kernel<TI, TO, V, INTER>), kMostHeads * 32 * kThreads);
        e != cudaSuccess)
      return e;
  }
  rotary_kernel<TI, TO, V, INTER><<<dim3((unsigned)blocks, (unsigned)groups), kThreads, smem, stream>>>(p);
  return cudaGetLastError();
}

// Whether every row set can move runs of V elements as vectors: whole runs on
// both sides of the rotated part's end, neighbouring dims, and base addresses
// and strides that are multiples of the access (a stride of a dim of size 1
// is never used).
template <typename TI, typename TO>
bool runs_of(const RotaryParams& p, int V) {
  if (p.rot % (2 * V) != 0 || p.d % (2 * V) != 0) return false;
  auto fits = [V](const void* base, int bytes, int64_t sb, int64_t sh, int64_t st, int64_t sd) {
    const int access = V * bytes;
    return sd == 1 && reinterpret_cast<uintptr_t>(base) % access == 0 && sb * bytes % access == 0 &&
           sh * bytes % access == 0 && st * bytes % access == 0;
  };
  for (int i = 0; i < p.n_sets; ++i) {
    const RowSet& s = p.set[i];
    const int64_t B = s.paged ? p.pages.n_pages : p.B, T = s.paged ? p.pages.rows : p.T;
    if (!fits(s.src, sizeof(TI), p.B > 1 ? s.s_b : 0, s.heads > 1 ? s.s_h : 0, p.T > 1 ? s.s_t : 0, s.s_d) ||
        !fits(s.dst, sizeof(TO), B > 1 ? s.d_b : 0, s.heads > 1 ? s.d_h : 0, T > 1 ? s.d_t : 0, s.d_d))
      return false;
  }
  return true;
}

template <typename TI, typename TO, int V>
cudaError_t launch_layout(const RotaryParams& p, bool inter, cudaStream_t stream) {
  return inter ? launch_v<TI, TO, V, true>(p, stream) : launch_v<TI, TO, V, false>(p, stream);
}

template <typename TI, typename TO>
cudaError_t launch_types(const RotaryParams& p, bool inter, cudaStream_t stream) {
  if constexpr (sizeof(TI) == 2)
    if (runs_of<TI, TO>(p, 8)) return launch_layout<TI, TO, 8>(p, inter, stream);
  if (runs_of<TI, TO>(p, 4)) return launch_layout<TI, TO, 4>(p, inter, stream);
  if (runs_of<TI, TO>(p, 2)) return launch_layout<TI, TO, 2>(p, inter, stream);
  return launch_layout<TI, TO, 1>(p, inter, stream);
}

cudaError_t launch_rotary(const RotaryParams& p, int32_t in, int32_t out, bool inter, cudaStream_t stream) {
  if (in == BLKATTN_BF16 && out == BLKATTN_BF16) return launch_types<__nv_bfloat16, __nv_bfloat16>(p, inter, stream);
  if (in == BLKATTN_BF16) return launch_types<__nv_bfloat16, float>(p, inter, stream);
  if (out == BLKATTN_BF16) return launch_types<float, __nv_bfloat16>(p, inter, stream);
  return launch_types<float, float>(p, inter, stream);
}

// ------------------------------------------------------------- validation
void set_src(RowSet* s, const blkattn_tensor* t) {
  s->src = t->data;
  s->s_b = t->strides[0]; s->s_h = t->strides[1]; s->s_t = t->strides[2]; s->s_d = t->strides[3];
  s->heads = (int)t->sizes[1];
}
void set_dst(RowSet* s, const blkattn_tensor* t) {
  s->dst = t->data;
  s->d_b = t->strides[0]; s->d_h = t->strides[1]; s->d_t = t->strides[2]; s->d_d = t->strides[3];
}

int rope(const blkattn_tensor* x, const blkattn_tensor* pos, const blkattn_tensor* ph, int32_t layout, float mscale,
         const blkattn_tensor* y, bool back, blkattn_stream_t stream) {
  if (!tensor_dims_ok(x, 4) || !tensor_dims_ok(pos, 2) || !tensor_dims_ok(y, 4)) return BLKATTN_ERR_INVALID_ARG;
  if (!floats(x) || !floats(y) || pos->dtype != BLKATTN_I32) return BLKATTN_ERR_INVALID_ARG;
  for (int i = 0; i < 4; ++i)
    if (x->sizes[i] != y->sizes[i]) return BLKATTN_ERR_INVALID_ARG;
  const int64_t B = x->sizes[0], H = x->sizes[1], T = x->sizes[2], d = x->sizes[3];
  if (pos->sizes[0] != B || pos->sizes[1] != T) return BLKATTN_ERR_INVALID_ARG;
  if (int st = check_phases(ph, layout, d); st != BLKATTN_OK) return st;
  if (!finite(mscale) || !writable(y) || !in_place_ok(x, y)) return BLKATTN_ERR_INVALID_ARG;
  if (!tensors_on_one_device(x, {pos, ph, y})) return BLKATTN_ERR_INVALID_ARG;
  if (d > kMaxDim || H > 0xffff || B > 0x7fffffff || T > 0x7fffffff || (B > 0 && T > 0x7fffffff / B))
    return BLKATTN_ERR_UNSUPPORTED;
  if (B == 0 || H == 0 || T == 0) return BLKATTN_OK;
  for (const blkattn_tensor* t : {x, pos, ph, y})
    if (t->data == nullptr) return BLKATTN_ERR_INVALID_ARG;
  if (int st = require_current_device(x->device); st != BLKATTN_OK) return st;
  RotaryParams p{};
  set_src(&p.set[0], x);
  set_dst(&p.set[0], y);
  p.set[0].turn = true;
  p.n_sets = 1;
  p.pos = static_cast<const int32_t*>(pos->data);
  p.p_b = pos->strides[0]; p.p_t = pos->strides[1];
  p.phases = static_cast<const int64_t*>(ph->data);
  p.ph_s = ph->strides[0];
  p.rot = (int)(2 * ph->sizes[0]);
  p.back = back;
  p.mscale = mscale;
  p.d = (int)d; p.B = (int)B; p.T = (int)T;
  if (cudaError_t e = launch_rotary(p, x->dtype, y->dtype, layout == BLKATTN_ROPE_INTERLEAVED,
                                    reinterpret_cast<cudaStream_t>(stream));
      e != cudaSuccess)
    return report_cuda_failure(e);
  return BLKATTN_OK;
}

}  // namespace
}  // namespace blkattn

extern "C" {

int blkattn_rope_angles(const blkattn_rope_spec* spec, double* angles, float* mscale) {
  if (spec == nullptr || angles == nullptr) return BLKATTN_ERR_INVALID_ARG;
  const int r = spec->rot;
  if (r < 2 || r % 2 != 0 || r > blkattn::kMaxDim || !(spec->base > 1.0) || std::isinf(spec->base))
    return BLKATTN_ERR_INVALID_ARG;
  const bool scaled = spec->scaling != BLKATTN_ROPE_PLAIN;
  if (scaled && (!(spec->factor >= 1.0) || std::isinf(spec->factor))) return BLKATTN_ERR_INVALID_ARG;
  double base = spec->base;
  switch (spec->scaling) {
    case BLKATTN_ROPE_PLAIN:
    case BLKATTN_ROPE_LINEAR: break;
    case BLKATTN_ROPE_BASE:
      if (r < 4) return BLKATTN_ERR_INVALID_ARG;
      base *= std::pow(spec->factor, (double)r / (r - 2));
      break;
    case BLKATTN_ROPE_RAMP:
      if (!(spec->trained > 0.0) || !(spec->low >= 0.0) || !(spec->high > spec->low) || std::isinf(spec->high) ||
          std::isinf(spec->trained))
        return BLKATTN_ERR_INVALID_ARG;
      break;
    default: return BLKATTN_ERR_INVALID_ARG;
  }
  const double two_pi = 6.283185307179586476925286766559;
  for (int i = 0; i < r / 2; ++i) {
    double w = std::pow(base, -2.0 * i / r);
    if (spec->scaling == BLKATTN_ROPE_LINEAR) w /= spec->factor;
    if (spec->scaling == BLKATTN_ROPE_RAMP) {
      double keep = (spec->trained * w / two_pi - spec->low) / (spec->high - spec->low);
      keep = keep < 0.0 ? 0.0 : (keep > 1.0 ? 1.0 : keep);
      w = w * keep + w / spec->factor * (1.0 - keep);
    }
    angles[i] = w;
  }
  if (mscale) *mscale = spec->scaling == BLKATTN_ROPE_RAMP ? (float)(0.1 * std::log(spec->factor) + 1.0) : 1.f;
  return BLKATTN_OK;
}

int blkattn_rope_phases(const double* angles, int64_t n, int64_t* phases) {
  if (n < 0 || (n > 0 && (angles == nullptr || phases == nullptr))) return BLKATTN_ERR_INVALID_ARG;
  for (int64_t i = 0; i < n; ++i)
    if (!(std::fabs(angles[i]) <= 8.0)) return BLKATTN_ERR_INVALID_ARG;
  // 2^66 / (2 pi) = 2^64 * 2 / pi rounded down: 64 bits and 64 below the point
  constexpr uint64_t kTurnHi = 0xA2F9836E4E441529ull, kTurnLo = 0xFC2757D1F534DDC0ull;
  for (int64_t i = 0; i < n; ++i) {
    int e = 0;
    const double m = std::frexp(std::fabs(angles[i]), &e);  // angle = m 2^e, m in [1/2, 1)
    const uint64_t M = (uint64_t)std::ldexp(m, 53);         // exact: 53 bits
    // angle 2^64 / (2 pi) = M 2^(e - 53) * 2^64 * (kTurnHi + kTurnLo 2^-64) 2^-66;
    // the product's whole part decides the rounding
    const unsigned __int128 prod =
        (unsigned __int128)M * kTurnHi + (((unsigned __int128)M * kTurnLo) >> 64);  // below 2^117
    const int sh = 55 - e;  // phase = prod 2^-sh, rounded; at least 51 for the angles allowed
    const uint64_t f = sh > 118 ? 0 : (uint64_t)((prod + ((unsigned __int128)1 << (sh - 1))) >> sh);
    phases[i] = (int64_t)(angles[i] < 0.0 ? 0 - f : f);
  }
  return BLKATTN_OK;
}

int blkattn_rope(const blkattn_tensor* x, const blkattn_tensor* pos, const blkattn_tensor* phases, int32_t layout,
                 float mscale, const blkattn_tensor* y, blkattn_stream_t stream) {
  return blkattn::rope(x, pos, phases, layout, mscale, y, false, stream);
}

int blkattn_rope_bwd(const blkattn_tensor* dy, const blkattn_tensor* pos, const blkattn_tensor* phases,
                     int32_t layout, float mscale, const blkattn_tensor* dx, blkattn_stream_t stream) {
  return blkattn::rope(dy, pos, phases, layout, mscale, dx, true, stream);
}

int blkattn_paged_append(const blkattn_tensor* k, const blkattn_tensor* v, const blkattn_tensor* pos,
                         const blkattn_tensor* page_table, const blkattn_tensor* k_pages,
                         const blkattn_tensor* v_pages, const blkattn_tensor* phases_opt, int32_t layout,
                         float mscale, const blkattn_tensor* q_opt, const blkattn_tensor* q_out_opt,
                         blkattn_stream_t stream) {
  using namespace blkattn;
  if (!tensor_dims_ok(k, 4) || !tensor_dims_ok(v, 4) || !tensor_dims_ok(pos, 2)) return BLKATTN_ERR_INVALID_ARG;
  if (!floats(k) || v->dtype != k->dtype || pos->dtype != BLKATTN_I32) return BLKATTN_ERR_INVALID_ARG;
  const int64_t B = k->sizes[0], H = k->sizes[1], T = k->sizes[2], d = k->sizes[3];
  for (int i = 0; i < 4; ++i)
    if (v->sizes[i] != k->sizes[i]) return BLKATTN_ERR_INVALID_ARG;
  if (pos->sizes[0] != B || pos->sizes[1] != T || d < 1) return BLKATTN_ERR_INVALID_ARG;
  PageTable pt;
  if (int st = check_pages(k_pages, v_pages, page_table, k->dtype, B, H, d, &pt); st != BLKATTN_OK) return st;
  if (!writable(k_pages) || !writable(v_pages) || (k_pages->data == v_pages->data && k_pages->data != nullptr))
    return BLKATTN_ERR_INVALID_ARG;
  if (phases_opt) {
    if (int st = check_phases(phases_opt, layout, d); st != BLKATTN_OK) return st;
    if (!finite(mscale)) return BLKATTN_ERR_INVALID_ARG;
  }
  if ((q_opt == nullptr) != (q_out_opt == nullptr)) return BLKATTN_ERR_INVALID_ARG;
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
  if (!tensors_on_one_device(k, {v, pos, page_table, k_pages, v_pages, phases_opt, q_opt, q_out_opt}))
    return BLKATTN_ERR_INVALID_ARG;
  if (d > kMaxDim || H > 0x7fff || Hq > 0x7fff || B > 0x7fffffff || T > 0x7fffffff ||
      (B > 0 && T > 0x7fffffff / B))
    return BLKATTN_ERR_UNSUPPORTED;
  if (B == 0 || T == 0) return BLKATTN_OK;
  for (const blkattn_tensor* t : {k, v, pos, page_table, k_pages, v_pages})
    if (t->data == nullptr) return BLKATTN_ERR_INVALID_ARG;
  if (phases_opt && phases_opt->data == nullptr) return BLKATTN_ERR_INVALID_ARG;
  if (q_opt && Hq > 0 && (q_opt->data == nullptr || q_out_opt->data == nullptr)) return BLKATTN_ERR_INVALID_ARG;
  if (int st = require_current_device(k->device); st != BLKATTN_OK) return st;
  RotaryParams p{};
  set_src(&p.set[0], k);
  set_dst(&p.set[0], k_pages);
  p.set[0].turn = phases_opt != nullptr;
  p.set[0].paged = true;
  set_src(&p.set[1], v);
  set_dst(&p.set[1], v_pages);
  p.set[1].paged = true;
  p.n_sets = 2;
  if (q_opt && Hq > 0) {
    set_src(&p.set[2], q_opt);
    set_dst(&p.set[2], q_out_opt);
    p.set[2].turn = phases_opt != nullptr;
    p.n_sets = 3;
  }
  p.pos = static_cast<const int32_t*>(pos->data);
  p.p_b = pos->strides[0]; p.p_t = pos->strides[1];
  if (phases_opt) {
    p.phases = static_cast<const int64_t*>(phases_opt->data);
    p.ph_s = phases_opt->strides[0];
    p.rot = (int)(2 * phases_opt->sizes[0]);
  }
  p.skip_negative = true;
  p.mscale = mscale;
  p.d = (int)d; p.B = (int)B; p.T = (int)T;
  p.pages = pt;
  if (cudaError_t e = launch_rotary(p, k->dtype, k->dtype, phases_opt && layout == BLKATTN_ROPE_INTERLEAVED,
                                    reinterpret_cast<cudaStream_t>(stream));
      e != cudaSuccess)
    return report_cuda_failure(e);
  return BLKATTN_OK;
}

}  // extern "C"
