// Rows turned by their logical position: what the rotary kernels, the head
// norms and the 8-bit append share (rotary.cu has the mathematics), and the
// checks of their arguments.
#pragma once
#include <cuda_bf16.h>

#include <cstdint>

#include "paged.h"
#include "ptx.cuh"

namespace blkattn {

template <typename T>
__device__ __forceinline__ float to_f32(T x) { return static_cast<float>(x); }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_f32(float x) { return static_cast<T>(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// sin and cos of position t at phase F.
__device__ __forceinline__ void turn_of(int t, int64_t F, float& sn, float& cs) {
  const uint64_t a = (uint64_t)(int64_t)t * (uint64_t)F;
  // the top 32 bits: a signed fraction of half a turn in [-1, 1)
  sincospif((float)(int32_t)(a >> 32) * 0x1p-31f, &sn, &cs);
}
// The same with what the float cannot hold of those 32 bits, to first order: for
// rows that are rounded to few bits next, where an angle's last bit moves a
// value over a step now and then.
__device__ __forceinline__ void turn_of_fine(int t, int64_t F, float& sn, float& cs) {
  const uint64_t a = (uint64_t)(int64_t)t * (uint64_t)F;
  const int32_t h = (int32_t)(a >> 32);
  const int32_t most = h & ~0xff;  // 24 bits
  float s, c;
  sincospif((float)most * 0x1p-31f, &s, &c);
  const float r = (float)(h - most) * (0x1p-31f * 3.14159265f);
  sn = fmaf(c, r, s);
  cs = fmaf(-s, r, c);
}
// 1 / sqrt(x), with a step of Newton's after the approximation.
__device__ __forceinline__ float rsqrt_fine(float x) {
  const float r = rsqrtf(x);
  const float f = fmaf(0.5f * r, fmaf(-x * r, r, 1.f), r);
  return f - f == 0.f ? f : r;  // (zeros and infinities)
}

// V elements of a row in registers, moved as one access.
template <typename T, int V>
struct alignas(sizeof(T) * V > 16 ? 16 : sizeof(T) * V) Vec {
  T x[V];
};
template <typename T, int V>
__device__ __forceinline__ void store(T* p, const Vec<T, V>& y) {
  if constexpr (sizeof(T) * V == 32) {
    // 8 floats in one 32-byte store (whole sectors)
    asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(y.x[0]), "f"(y.x[1]),
                 "f"(y.x[2]), "f"(y.x[3]), "f"(y.x[4]), "f"(y.x[5]), "f"(y.x[6]), "f"(y.x[7])
                 : "memory");
  } else {
    *reinterpret_cast<Vec<T, V>*>(p) = y;
  }
}

// Waits until at most n (0..7, a constant after unrolling) of the thread's
// groups of asynchronous copies are pending.
__device__ __forceinline__ void wait_copies(int n) {
  switch (n) {
    case 0: asm volatile("cp.async.wait_group 0;" ::: "memory"); break;
    case 1: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
    case 2: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
    case 3: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;
    case 4: asm volatile("cp.async.wait_group 4;" ::: "memory"); break;
    case 5: asm volatile("cp.async.wait_group 5;" ::: "memory"); break;
    case 6: asm volatile("cp.async.wait_group 6;" ::: "memory"); break;
    default: asm volatile("cp.async.wait_group 7;" ::: "memory"); break;
  }
}

// The rotation of 2 V dims u in fp32, two runs of V: pair j is (j, V + j), or the
// neighbours (2j, 2j + 1).
template <int V, bool INTER>
__device__ __forceinline__ void turn_pairs(const float (&u)[2 * V], bool turn, const float (&sn)[V],
                                           const float (&cs)[V], float (&w)[2 * V]) {
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int a = INTER ? 2 * j : j, b = INTER ? 2 * j + 1 : V + j;
    w[a] = turn ? u[a] * cs[j] - u[b] * sn[j] : u[a];
    w[b] = turn ? u[a] * sn[j] + u[b] * cs[j] : u[b];
  }
}
template <typename TI, int V>
__device__ __forceinline__ void unpack_runs(const Vec<TI, V>& x0, const Vec<TI, V>& x1, float (&u)[2 * V]) {
#pragma unroll
  for (int j = 0; j < V; ++j) {
    u[j] = to_f32(x0.x[j]);
    u[V + j] = to_f32(x1.x[j]);
  }
}
template <typename TO, int V>
__device__ __forceinline__ void pack_runs(const float (&w)[2 * V], Vec<TO, V>& y0, Vec<TO, V>& y1) {
  if constexpr (sizeof(TO) == 2 && V > 1) {
    uint32_t* q0 = reinterpret_cast<uint32_t*>(&y0);
    uint32_t* q1 = reinterpret_cast<uint32_t*>(&y1);
#pragma unroll
    for (int j = 0; j < V / 2; ++j) {
      q0[j] = pack_bf16(w[2 * j], w[2 * j + 1]);
      q1[j] = pack_bf16(w[V + 2 * j], w[V + 2 * j + 1]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      y0.x[j] = from_f32<TO>(w[j]);
      y1.x[j] = from_f32<TO>(w[V + j]);
    }
  }
}
template <typename TI, typename TO, int V, bool INTER>
__device__ __forceinline__ void turn_run(const Vec<TI, V>& x0, const Vec<TI, V>& x1, bool turn, const float (&sn)[V],
                                         const float (&cs)[V], Vec<TO, V>& y0, Vec<TO, V>& y1) {
  float u[2 * V], w[2 * V];
  unpack_runs<TI, V>(x0, x1, u);
  turn_pairs<V, INTER>(u, turn, sn, cs, w);
  pack_runs<TO, V>(w, y0, y1);
}

// ------------------------------------------------------------- validation
constexpr int64_t kMaxDim = 1024;
constexpr int64_t kMostRows = 1LL << 33;  // of one call of the head norms

inline bool floats(const blkattn_tensor* t) { return t->dtype == BLKATTN_BF16 || t->dtype == BLKATTN_F32; }

// No two elements of a tensor that is written share an address through a
// broadcast dim.
inline bool writable(const blkattn_tensor* t) {
  bool ok = true, empty = false;
  for (int i = 0; i < t->ndim; ++i) {
    empty = empty || t->sizes[i] == 0;
    ok = ok && !(t->sizes[i] > 1 && t->strides[i] == 0);
  }
  return ok || empty;
}

// Rows of the same shape at one address: the call may work in place only on
// the very same view.
inline bool in_place_ok(const blkattn_tensor* a, const blkattn_tensor* b) {
  if (a->data != b->data || a->data == nullptr) return true;  // (no rows: nothing overlaps)
  if (a->dtype != b->dtype) return false;
  for (int i = 0; i < a->ndim; ++i)
    if (a->sizes[i] > 1 && a->strides[i] != b->strides[i]) return false;
  return true;
}

inline bool finite(float x) { return x - x == 0.f; }

// Phases [rot / 2] int64, rot <= d; and the layout.
inline int check_phases(const blkattn_tensor* ph, int32_t layout, int64_t d) {
  if (layout != BLKATTN_ROPE_HALF && layout != BLKATTN_ROPE_INTERLEAVED) return BLKATTN_ERR_INVALID_ARG;
  if (!tensor_dims_ok(ph, 1) || ph->dtype != BLKATTN_I64 || ph->sizes[0] < 1 || 2 * ph->sizes[0] > d)
    return BLKATTN_ERR_INVALID_ARG;
  return BLKATTN_OK;
}

}  // namespace blkattn
