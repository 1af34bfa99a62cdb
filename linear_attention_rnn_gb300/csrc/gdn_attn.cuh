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
// Sequence s of n_seqs over `total` rows (cu null: equal lengths), as (first row,
// rows), held inside the tensor whatever the array says.
__device__ __forceinline__ int2 rows_of(const int* cu, int s, int n_seqs, int total) {
  if (!cu) return make_int2(s * (total / n_seqs), total / n_seqs);
  const int a = min(max(cu[s], 0), total);
  return make_int2(a, min(max(cu[s + 1], a), total) - a);
}
// Both sides of the first 32 sequences, one to a lane, read at the kernel's start,
// where one trip to memory fetches them all.
struct Lanes {
  int2 q, k;
  int used;
};
__device__ __forceinline__ Lanes read_lanes(const AttnArgs& a) {
  const int s = min((int)(threadIdx.x & 31), a.n_seqs - 1);
  Lanes l;
  l.q = rows_of(a.cu_q, s, a.n_seqs, a.total_q);
  l.k = rows_of(a.cu_k, s, a.n_seqs, a.total_k);
  l.used = a.k_len ? min(max(a.k_len[s], 0), l.k.y) : l.k.y;
  return l;
}
__device__ __forceinline__ Seq seq_of(const AttnArgs& a, const Lanes& l, int s) {
  int2 q, k;
  int used;
  if (s < 32) {
    q = make_int2(__shfl_sync(0xffffffffu, l.q.x, s), __shfl_sync(0xffffffffu, l.q.y, s));
    k = make_int2(__shfl_sync(0xffffffffu, l.k.x, s), 0);
    used = __shfl_sync(0xffffffffu, l.used, s);
  } else {
    q = rows_of(a.cu_q, s, a.n_seqs, a.total_q);
    k = rows_of(a.cu_k, s, a.n_seqs, a.total_k);
    used = a.k_len ? min(max(a.k_len[s], 0), k.y) : k.y;
  }
  Seq r;
  r.q0 = q.x;
  r.ql = q.y;
  r.k0 = k.x;
  r.kl = used;
  return r;
}

// The rank-th of all sequences' tiles, those with the highest index in their sequence first
// (the work of a tile grows with it, and CTAs start in order of rank); sequence -1: there
// are fewer.  tiles(s): those of sequence s, n0: of the lane's own, the first 32.  Every warp
// finds it for itself: a lane counts for every 32nd sequence, and the index of rank's
// tile is found by bisection.
template <typename F>
__device__ __forceinline__ int2 find_nth(F tiles, int n0, int n_seqs, int rank) {
  const int lane = threadIdx.x & 31;
  auto count_above = [&](int t) {                  // tiles of index t or more
    int c = max(n0 - t, 0);
    for (int s = lane + 32; s < n_seqs; s += 32) c += max(tiles(s) - t, 0);
    return __reduce_add_sync(0xffffffffu, c);
  };
  int most = n0;
  for (int s = lane + 32; s < n_seqs; s += 32) most = max(most, tiles(s));
  most = __reduce_max_sync(0xffffffffu, most);
  if (rank >= count_above(0)) return make_int2(-1, 0);
  int lo = 0, hi = most;  // count_above(lo) > rank >= count_above(hi)
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (count_above(mid) > rank)
      lo = mid;
    else
      hi = mid;
  }
  int k = rank - count_above(lo + 1);  // the k-th sequence that has a tile lo
  for (int s0 = 0; s0 < n_seqs; s0 += 32) {
    const bool has = s0 + lane < n_seqs && (s0 ? tiles(s0 + lane) : n0) > lo;
    unsigned m = __ballot_sync(0xffffffffu, has);
    const int c = __popc(m);
    if (k < c) {
      for (; k > 0; --k) m &= m - 1;
      return make_int2(s0 + __ffs((int)m) - 1, lo);
    }
    k -= c;
  }
  return make_int2(-1, 0);
}
// The same for tiles of K rows (lane_rows: the rows of the lane's own sequence).
__device__ __forceinline__ int2 find_tile(const int* cu, int lane_rows, int n_seqs, int total, int K, int rank) {
  return find_nth([&](int s) { return (rows_of(cu, s, n_seqs, total).y + K - 1) / K; },
                  (int)(threadIdx.x & 31) < n_seqs ? (lane_rows + K - 1) / K : 0, n_seqs, rank);
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

// ---- keys in pages ----------------------------------------------------------------
// A tile of KEYS rows of a sequence is loaded piece by piece: `box` rows, the largest
// power of two that divides the page size (at most KEYS), lie in one page.  Pieces are
// shared out to the lanes of the loading warp, which reads a tile's table entries ahead
// of its slot.  An entry that names no page, and a piece behind the keys, reads as zeros
// (the map's fill for page -1).
template <int KEYS>
struct Paged {
  const int* row;  // the sequence's part of the table
  int kl;
  __device__ __forceinline__ Paged(const AttnArgs& a, int seq, int keys)
      : row(a.table + (long)seq * a.pages.table_stride), kl(keys) {}
  // the page of this lane's piece of the tile from key0 on (-1: none)
  __device__ __forceinline__ int entry(const PageArgs& p, int key0) const {
    const int lane = threadIdx.x & 31, key = key0 + lane * p.box;
    if (lane >= KEYS / p.box || key >= kl) return -1;
    const int e = row[p.page_of(key)];
    return (unsigned)e < (unsigned)p.n_pages ? e : -1;
  }
  // by a whole warp
  __device__ __forceinline__ void load(const PageArgs& p, unsigned char* dst, const CUtensorMap* m, int head, int key0,
                                       int entry, uint64_t* bar) const {
    const int lane = threadIdx.x & 31;
    if (lane == 0) tc::arrive_expect_tx(bar, KEYS * HD * 2);
    __syncwarp();
    if (lane < KEYS / p.box) {
      const int key = key0 + lane * p.box, y = key - p.page_of(key) * p.page;
      unsigned char* d = dst + lane * p.box * 128;
      tc::tma_load_4d(d, m, 0, head, y, entry, bar);
      tc::tma_load_4d(d + KEYS * 128, m, 64, head, y, entry, bar);
    }
  }
  // one bit for every 16 keys of the tile from key0 on whose page is absent, the same in all
  // lanes; ask() reads the table, absent() a tile later so that nobody waits for it
  __device__ __forceinline__ int ask(const PageArgs& p, int key0) const {
    const int lane = threadIdx.x & 31, key = key0 + lane * 16;
    return lane < KEYS / 16 && key < kl ? row[p.page_of(key)] : 0;
  }
  __device__ __forceinline__ uint32_t absent(const PageArgs& p, int asked) const {
    return __ballot_sync(0xffffffffu, (unsigned)asked >= (unsigned)p.n_pages);
  }
};

// Zeros in rows [from, 128) of an SW128 tile, by `nthreads` threads.
__device__ __forceinline__ void zero_rows(unsigned char* tile, int from, int t, int nthreads) {
  for (int i = from * 16 + t; i < CH * 16; i += nthreads)
    *reinterpret_cast<uint4*>(tile + tc::sw128_chunk(i >> 4, i & 15, CH)) = make_uint4(0u, 0u, 0u, 0u);
}

// 32 columns (c0 ..) of row r, times f, into an SW128 tile that a tensor map stores
__device__ __forceinline__ void stage32(unsigned char* tile, int r, int c0, const float (&v)[32], float f) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint4 o;
    o.x = pack_bf16(f * v[8 * i], f * v[8 * i + 1]);
    o.y = pack_bf16(f * v[8 * i + 2], f * v[8 * i + 3]);
    o.z = pack_bf16(f * v[8 * i + 4], f * v[8 * i + 5]);
    o.w = pack_bf16(f * v[8 * i + 6], f * v[8 * i + 7]);
    *reinterpret_cast<uint4*>(tile + tc::sw128_chunk(r, (c0 >> 3) + i, CH)) = o;
  }
}
// The staged tile's two halves to (head, row) of a map, by one thread, which waits
// until they have been read.
__device__ __forceinline__ void store_tile(const CUtensorMap* m, int head, int row, const unsigned char* tile) {
  tc::tma_store_3d(m, 0, head, row, tile);
  tc::tma_store_3d(m, 64, head, row, tile + TILE / 2);
  tc::bulk_commit();
  tc::bulk_wait_read();
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
