// gdn_attn.cuh -- what the attention kernels share: sequence ranges, the rows of a
// query tile, loads and row stores.
//
// A query tile has 128 rows: as many whole tokens as fit, each with the G query
// heads of one key head (row = token * G + head in the group).  Every K and V
// tile is thus read once for the group, a group's gradients of k and v are sums
// over rows of one product, and a few tokens (or one) still fill G rows each.
// Rows past 128 / G tokens, and of tokens past the sequence's end, are masked.
#pragma once
#include "gdn_kernels.cuh"
#include "gdn_tc05.cuh"

namespace gdn {
namespace attn {

constexpr uint32_t TILE = CH * HD * 2;  // a [128 x 128] bf16 tile
constexpr float LOG2E = 1.4426950408889634f;

struct Seq {
  int q0, ql, k0, kl;  // first row and rows of q, first row and used rows of k
};
// (held inside the tensors whatever the arrays say)
__device__ __forceinline__ Seq seq_of(const AttnArgs& a, int s) {
  Seq r;
  if (a.cu_q) {
    r.q0 = min(max(a.cu_q[s], 0), a.total_q);
    r.ql = min(max(a.cu_q[s + 1], r.q0), a.total_q) - r.q0;
  } else {
    r.ql = a.total_q / a.n_seqs;
    r.q0 = s * r.ql;
  }
  if (a.cu_k) {
    r.k0 = min(max(a.cu_k[s], 0), a.total_k);
    r.kl = min(max(a.cu_k[s + 1], r.k0), a.total_k) - r.k0;
  } else {
    r.kl = a.total_k / a.n_seqs;
    r.k0 = s * r.kl;
  }
  if (a.k_len) r.kl = min(max(a.k_len[s], 0), r.kl);
  return r;
}

// Tile slots: sequence s has the slots first_slot(s) .. first_slot(s + 1) - 1, at
// least as many as it has tiles of K rows and at most one more than total / K
// over all sequences together.
__device__ __forceinline__ int first_slot(const int* cu, int s, int each, int total, int K) {
  return (cu ? min(max(cu[s], 0), total) : s * each) / K + s;
}
// Sequence and tile of a slot, by all threads of the block together (sequence
// -1: none).
__device__ __forceinline__ int2 find_tile(const int* cu, int n_seqs, int total, int K, int slot) {
  __shared__ int2 found;
  if (threadIdx.x == 0) found = make_int2(-1, 0);
  __syncthreads();
  const int each = total / n_seqs;
  for (int s = threadIdx.x; s < n_seqs; s += blockDim.x) {
    const int a = first_slot(cu, s, each, total, K);
    if (slot >= a && slot < first_slot(cu, s + 1, each, total, K)) found = make_int2(s, slot - a);
  }
  __syncthreads();
  return found;
}

// 128 rows of one head
__device__ __forceinline__ void load_rows(unsigned char* dst, const CUtensorMap* m, int head, int row, uint64_t* bar) {
  tc::arrive_expect_tx(bar, TILE);
  tc::tma_load_3d(dst, m, 0, head, row, bar);
  tc::tma_load_3d(dst + TILE / 2, m, 64, head, row, bar);
}
// a query tile: the map's box holds the group's G heads of 128 / G tokens
__device__ __forceinline__ void load_group(unsigned char* dst, const CUtensorMap* m, int kh, int G, int tok,
                                           uint64_t* bar) {
  tc::arrive_expect_tx(bar, 2u * 128u * (uint32_t)(CH / G * G));
  tc::tma_load_3d(dst, m, 0, kh * G, tok, bar);
  tc::tma_load_3d(dst + TILE / 2, m, 64, kh * G, tok, bar);
}

// Zeros in rows [from, 128) of an SW128 tile, by `nthreads` threads.
__device__ __forceinline__ void zero_rows(unsigned char* tile, int from, int t, int nthreads) {
  for (int i = from * 16 + t; i < CH * 16; i += nthreads)
    *reinterpret_cast<uint4*>(tile + tc::sw128_chunk(i >> 4, i & 15, CH)) = make_uint4(0u, 0u, 0u, 0u);
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void store32(bf16* dst, const float (&v)[32], float f) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint4 o;
    o.x = pack_bf16(f * v[8 * i], f * v[8 * i + 1]);
    o.y = pack_bf16(f * v[8 * i + 2], f * v[8 * i + 3]);
    o.z = pack_bf16(f * v[8 * i + 4], f * v[8 * i + 5]);
    o.w = pack_bf16(f * v[8 * i + 6], f * v[8 * i + 7]);
    *reinterpret_cast<uint4*>(dst + 8 * i) = o;
  }
}

}  // namespace attn
}  // namespace gdn
