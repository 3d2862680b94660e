// The paged KV cache: pools of pages [N, H_kv, rows, d] and a table of page
// numbers per sequence.  Cache row t of sequence b is row t mod `rows` of page
// table[b, t / rows]; an entry outside [0, N) holds no page.
#pragma once
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>
#include <initializer_list>

#include "blkattn.h"

namespace blkattn {

struct PageTable {
  const int32_t* table;
  int64_t sb, sp;  // strides of the sequence and the entry
  int entries;     // per sequence
  int shift;       // log2 of the rows of a page
  int rows;
  int n_pages;     // pages in the pool
  // rows of 128 bf16 dims whose heads or rows lie packed: one copy brings both
  // 64-dim halves of a piece (5-D map: 64 dims, 8 rows, halves, 8-row groups,
  // pages; the head moves the halves' or the groups' coordinate)
  int wide;
  int wide_h2, wide_h3;
};

// Table entry of cache row t of sequence b, -1 for a t outside the table (or
// negative); any value may stand there.
__device__ __forceinline__ int entry_of(const PageTable& pt, int b, int t) {
  const int i = t >> pt.shift;  // (negative t: negative i)
  return (unsigned)i < (unsigned)pt.entries ? __ldg(pt.table + b * pt.sb + i * pt.sp) : -1;
}

// Page of cache row t of sequence b, or -1: no page there.
__device__ __forceinline__ int page_of(const PageTable& pt, int b, int t) {
  const int page = entry_of(pt, b, t);
  return (unsigned)page < (unsigned)pt.n_pages ? page : -1;
}

constexpr int64_t kMinPageRows = 8, kMaxPageRows = 65536;
constexpr int64_t kMaxCacheRows = (1 << 30) - 1;  // of a sequence: 32-bit sums of a key and a chunk do not overflow

// A kernel's shared-memory limit, raised once on each device that launches it
// (the attribute belongs to the device's copy of the kernel).
struct DeviceOnce {
  std::atomic<uint64_t> done{0};  // bit d: device d
  // carveout: also prefer all of the unified storage as shared memory
  cudaError_t set_smem(const void* kernel, int bytes, bool carveout = true) {
    int dev = 0;
    if (cudaError_t e = cudaGetDevice(&dev); e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (dev < 64 && (done.load(std::memory_order_acquire) & bit)) return cudaSuccess;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && carveout)
      e = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
    return e;
  }
};

// Host checks shared by the operators of the paged cache (no CUDA call).
bool tensor_dims_ok(const blkattn_tensor* t, int ndim);
// Every tensor given (NULL skipped) names the device of `first`, a real one.
bool tensors_on_one_device(const blkattn_tensor* first, std::initializer_list<const blkattn_tensor*> ts);
int require_current_device(int32_t device);
// k_pages, v_pages [N, H, rows, d] of one dtype, and table int32 [B, entries].
int check_pages(const blkattn_tensor* k_pages, const blkattn_tensor* v_pages, const blkattn_tensor* table,
                int32_t dtype, int64_t B, int64_t H, int64_t d, PageTable* out);

}  // namespace blkattn
