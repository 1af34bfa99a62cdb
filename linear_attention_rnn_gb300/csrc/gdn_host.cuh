// gdn_host.cuh -- what the operators' extern "C" entry points share on the host.
#pragma once
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "gdn.h"
#include "gdn_common.cuh"
#include "gdn_kernels.cuh"

namespace gdn {

constexpr size_t ALIGN = 256;
inline size_t up(size_t x) { return (x + ALIGN - 1) / ALIGN * ALIGN; }
inline bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline int cuda_status(cudaError_t e) { return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA; }

template <typename T>
T* at(void* ws, size_t off) {
  return reinterpret_cast<T*>(static_cast<char*>(ws) + off);
}

inline int sm_count() {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms <= 0)
    sms = 152;
  return sms;
}

// rows of H heads, `stride` elements apart: whole 16-byte pieces that do not overlap
inline bool row_stride_ok(long long stride, int H) { return stride >= (long long)H * HD && stride % 8 == 0; }

// A workspace that would hold the status word alone may be left out.
constexpr size_t STATUS_BYTES = ALIGN;
inline bool workspace_ok(const void* ws, size_t ws_bytes, size_t need) {
  return ws ? ws_bytes >= need : need <= STATUS_BYTES;
}

// Pages of a cache: whole 16-row pieces, as the attention kernels load them.
constexpr int PAGE_PIECE = 16;
inline int pages_check(int n_pages, int page_size) {
  if (n_pages < 0 || page_size <= 0) return GDN_ERR_ARG;
  if (page_size % PAGE_PIECE != 0) return GDN_ERR_SHAPE;
  return (long long)n_pages * page_size <= INT32_MAX ? GDN_OK : GDN_ERR_ARG;  // (rows are counted in 32 bits)
}
// Pages whose rows are loaded in boxes of at most `tile` rows (a power of two).
inline PageArgs page_args(int n_pages, int page_size, int max_pages, long long table_stride, int tile) {
  PageArgs p;
  p.page = page_size;
  p.n_pages = n_pages;
  p.box = tile;
  while (page_size % p.box != 0) p.box /= 2;  // (16 divides it)
  p.capacity = n_pages > 0 ? max_pages * page_size : 0;
  p.table_stride = table_stride;
  // division by multiplication with 2^32 (2^shift - page) / page + 1 (Granlund and Montgomery,
  // "Division by invariant integers using multiplication", 1994)
  p.shift = 0;
  while ((1LL << p.shift) < page_size) ++p.shift;
  p.mul = (uint32_t)((((1ULL << p.shift) - (uint64_t)page_size) << 32) / (uint64_t)page_size + 1);
  return p;
}
// Strides in elements: whole 16-byte pieces, at least a row apart, within what a tensor map holds.
inline bool page_strides_ok(const gdn_page_strides* s) {
  if (!s) return false;
  const long long v[] = {s->page, s->row, s->head};
  for (long long x : v)
    if (x < HD || x % 8 != 0 || x >= (1LL << 38)) return false;
  return true;
}

}  // namespace gdn
