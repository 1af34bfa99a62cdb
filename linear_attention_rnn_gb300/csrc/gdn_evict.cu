// gdn_evict.cu -- eviction of the lightest keys from a cache in pages.
//
// Per sequence and key head: the last `recent` keys stay, and of the others the
// heaviest, `budget` in all; equal weights stay from the lowest index on.  What stays
// moves, in its order, to the first rows of the target pages (keys, values and weights).
// Keys on absent pages are gone already and never stay.
//
// k_evict_select, one block to a sequence and head, finds the smallest weight that stays
// by its digits: weights are mapped to unsigned numbers of the same order, the digits
// that all share are passed over, and each further digit of 8 bits takes one count over
// the candidates.  The weights are held in shared memory where they fit.  A last pass in
// index order writes the list of rows that stay: a warp counts over its own range of
// keys, a scan over the warps gives each its place.
//
// k_evict_move copies the rows of the lists, 16 lanes to a row.  Into other pages any
// block may take any part of a list.  In place (the target pages are the sequence's
// own) one block walks a list in its order: a row's target never lies behind it, so
// what a round writes are rows that this round and the earlier ones have read.
//
// Bound: HBM, 4 bytes a key and head and 1,024 a row that stays.
#include <stdint.h>

#include "gdn_kernels.cuh"

namespace gdn {

namespace {

constexpr int SELECT_THREADS = 1024, SELECT_WARPS = SELECT_THREADS / 32;
constexpr int SELECT_HELD = 49152;  // weights that shared memory holds
constexpr int MOVE_THREADS = 256, MOVE_ROWS = 64;  // rows of a list to a block (16 side by side)
constexpr int WALK_THREADS = 1024, WALK_ROWS = 128;

// The sequence's keys, and where the ones that always stay begin.
struct Cut {
  int kl, old, recent;
};
__device__ __forceinline__ Cut cut_of(const EvictArgs& a, int seq) {
  Cut c;
  c.kl = min(max(a.k_len[seq], 0), a.pages.capacity);
  c.recent = min(min(a.recent, a.budget), c.kl);
  c.old = c.kl - c.recent;
  return c;
}

// Order of weights as unsigned numbers, 1 and up: -0 is 0, NaN is below all others.
__device__ __forceinline__ uint32_t rank_of(float w) {
  if (isnan(w)) return 1u;
  const uint32_t u = __float_as_uint(w + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__global__ void __launch_bounds__(SELECT_THREADS, 1) k_evict_select(const __grid_constant__ EvictArgs a) {
  extern __shared__ uint32_t held[];
  __shared__ uint32_t hist[256];
  __shared__ uint32_t least, most;
  __shared__ int present[2];          // of the candidates, of the last ones
  __shared__ int digit, above;
  __shared__ int warps[SELECT_WARPS][2];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int kh = blockIdx.x % a.Hk, seq = blockIdx.x / a.Hk;
  pdl_wait();
  pdl_release();
  const Cut c = cut_of(a, seq);
  const int* table = a.table + (long)seq * a.pages.table_stride;
  const bool fits = c.old <= SELECT_HELD;
  // rank of key j (0: on an absent page)
  auto fetch = [&](int j) -> uint32_t {
    const int e = table[j / a.pages.page];
    if ((unsigned)e >= (unsigned)a.pages.n_pages) return 0u;
    return rank_of(a.weights[((long)e * a.Hk + kh) * a.pages.page + j % a.pages.page]);
  };
  auto rank = [&](int j) { return fits ? held[j] : fetch(j); };

  if (tid == 0) {
    least = 0xffffffffu;
    most = 0u;
    present[0] = present[1] = 0;
  }
  __syncthreads();
  uint32_t lo = 0xffffffffu, hi = 0u;
  int n0 = 0, n1 = 0;
  for (int j = tid; j < c.old; j += SELECT_THREADS) {
    const uint32_t r = fetch(j);
    if (fits) held[j] = r;
    if (r) {
      lo = min(lo, r);
      hi = max(hi, r);
      ++n0;
    }
  }
  for (int j = c.old + tid; j < c.kl; j += SELECT_THREADS)
    n1 += (unsigned)table[j / a.pages.page] < (unsigned)a.pages.n_pages;
  lo = __reduce_min_sync(0xffffffffu, lo);
  hi = __reduce_max_sync(0xffffffffu, hi);
  n0 = __reduce_add_sync(0xffffffffu, n0);
  n1 = __reduce_add_sync(0xffffffffu, n1);
  if (lane == 0) {
    atomicMin(&least, lo);
    atomicMax(&most, hi);
    atomicAdd(&present[0], n0);
    atomicAdd(&present[1], n1);
  }
  __syncthreads();
  const int take = min(present[0], a.budget - present[1]);  // of the candidates (recent <= budget)
  if (kh == 0 && tid == 0) a.new_len[seq] = take + present[1];
  // The candidates that stay: ranks above `edge`, and the first `ties` of rank `edge`.
  uint32_t edge = 0u;
  int ties = 0;
  if (take > 0 && take < present[0]) {
    // the digits below the highest one in which candidates differ
    int shift = 32 - __clz(least ^ most);       // bits that differ
    edge = shift < 32 ? most >> shift << shift : 0u;
    ties = take;
    while (shift > 0) {
      const int bits = min(shift, 8), low = shift - bits;
      for (int i = tid; i < 256; i += SELECT_THREADS) hist[i] = 0u;
      __syncthreads();
      const uint32_t mask = shift < 32 ? ~0u << shift : 0u;
      for (int j = tid; j < c.old; j += SELECT_THREADS) {
        const uint32_t r = rank(j);
        if (r && (r & mask) == edge) atomicAdd(&hist[r >> low & ((1u << bits) - 1u)], 1u);
      }
      __syncthreads();
      // the digit at which the count from the top reaches what is still to take
      if (warp == 0) {
        int mine = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) mine += hist[8 * lane + i];
        int from = mine;  // in this lane's digits and above
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_down_sync(0xffffffffu, from, o);
          if (lane + o < 32) from += y;
        }
        int over = from - mine;  // above this lane's digits
        if (over < ties && from >= ties) {
          int d = 8 * lane + 7;
          while (over + (int)hist[d] < ties) over += hist[d--];
          digit = d;
          above = over;
        }
      }
      __syncthreads();
      edge |= (uint32_t)digit << low;
      ties -= above;
      shift = low;
    }
  } else if (take > 0) {
    edge = 0u;  // all of them
  } else {
    edge = 0xffffffffu;  // none (no rank is above it)
  }

  // the list, in index order: warp w's range of keys, counted first
  const int per = ((c.kl + SELECT_WARPS - 1) / SELECT_WARPS + 31) & ~31;
  const int j0 = min(warp * per, c.kl), j1 = min(j0 + per, c.kl);
  auto kind = [&](int j) -> int {  // 1: stays, 2: stays if it is among the first ties
    if (j >= j1) return 0;
    if (j >= c.old) return (unsigned)table[j / a.pages.page] < (unsigned)a.pages.n_pages ? 1 : 0;
    const uint32_t r = rank(j);
    return r > edge ? 1 : r == edge && r ? 2 : 0;
  };
  int stay = 0, tied = 0;
  for (int j = j0; j < j1; j += 32) {
    const int k = kind(j + lane);
    stay += __popc(__ballot_sync(0xffffffffu, k == 1));
    tied += __popc(__ballot_sync(0xffffffffu, k == 2));
  }
  if (lane == 0) {
    warps[warp][0] = stay;
    warps[warp][1] = tied;
  }
  __syncthreads();
  int out = 0, seen = 0;
  for (int i = 0; i < warp; ++i) {
    out += warps[i][0];
    seen += warps[i][1];
  }
  out += min(seen, ties);
  int* list = a.list + ((long)seq * a.Hk + kh) * a.keep;
  for (int j = j0; j < j1; j += 32) {
    const int k = kind(j + lane);
    const uint32_t below = (1u << lane) - 1u, tie = __ballot_sync(0xffffffffu, k == 2);
    const bool keep = k == 1 || (k == 2 && seen + __popc(tie & below) < ties);
    const uint32_t kept = __ballot_sync(0xffffffffu, keep);
    if (keep) list[out + __popc(kept & below)] = j + lane;
    out += __popc(kept);
    seen += __popc(tie);
  }
}

// A row's halves of 16 lanes: the places of key j among keys, values and weights.
struct Place {
  long k, v, w;
};
__device__ __forceinline__ bool place_of(const EvictArgs& a, const int* table, int kh, int j, Place& p) {
  const int t = j / a.pages.page, row = j - t * a.pages.page, e = table[t];
  if ((unsigned)e >= (unsigned)a.pages.n_pages) return false;
  p.k = e * a.sk_page + row * a.sk_row + kh * a.sk_head;
  p.v = e * a.sv_page + row * a.sv_row + kh * a.sv_head;
  p.w = ((long)e * a.Hk + kh) * a.pages.page + row;
  return true;
}

__global__ void __launch_bounds__(MOVE_THREADS) k_evict_move(const __grid_constant__ EvictArgs a) {
  const int kh = blockIdx.x % a.Hk, seq = blockIdx.x / a.Hk;
  const int l = threadIdx.x & 15;
  pdl_wait();
  pdl_release();
  const int n = a.new_len[seq];
  const int* from = a.table + (long)seq * a.pages.table_stride;
  const int* to = a.to + (long)seq * a.to_stride;
  const int* list = a.list + ((long)seq * a.Hk + kh) * a.keep;
  constexpr int R = MOVE_ROWS / (MOVE_THREADS / 16);
  for (long base = (long)blockIdx.y * MOVE_ROWS; base < n; base += (long)gridDim.y * MOVE_ROWS) {
    uint4 k[R], v[R];
    float w[R];
    Place d[R];
    bool ok[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int i = (int)base + (threadIdx.x >> 4) + r * (MOVE_THREADS / 16);
      Place s;
      ok[r] = i < n && place_of(a, from, kh, list[i], s) && place_of(a, to, kh, i, d[r]);
      if (ok[r]) {
        k[r] = *reinterpret_cast<const uint4*>(a.k + s.k + 8 * l);
        v[r] = *reinterpret_cast<const uint4*>(a.v + s.v + 8 * l);
        w[r] = a.weights[s.w];
      }
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (ok[r]) {
        *reinterpret_cast<uint4*>(a.k + d[r].k + 8 * l) = k[r];
        *reinterpret_cast<uint4*>(a.v + d[r].v + 8 * l) = v[r];
        if (l == 0) a.weights[d[r].w] = w[r];
      }
  }
}

__global__ void __launch_bounds__(WALK_THREADS) k_evict_walk(const __grid_constant__ EvictArgs a) {
  const int kh = blockIdx.x % a.Hk, seq = blockIdx.x / a.Hk;
  const int l = threadIdx.x & 15;
  pdl_wait();
  pdl_release();
  const int n = a.new_len[seq];
  const int* table = a.table + (long)seq * a.pages.table_stride;
  const int* list = a.list + ((long)seq * a.Hk + kh) * a.keep;
  constexpr int R = WALK_ROWS / (WALK_THREADS / 16);
  for (int base = 0; base < n; base += WALK_ROWS) {
    uint4 k[R], v[R];
    float w[R];
    Place d[R];
    bool ok[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int i = base + (threadIdx.x >> 4) + r * (WALK_THREADS / 16);
      const int j = i < n ? list[i] : 0;
      Place s;
      // (a row that stays where it is needs no copy)
      ok[r] = i < n && j != i && place_of(a, table, kh, j, s) && place_of(a, table, kh, i, d[r]);
      if (ok[r]) {
        k[r] = *reinterpret_cast<const uint4*>(a.k + s.k + 8 * l);
        v[r] = *reinterpret_cast<const uint4*>(a.v + s.v + 8 * l);
        w[r] = a.weights[s.w];
      }
    }
    __syncthreads();  // the round's rows have been read
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (ok[r]) {
        *reinterpret_cast<uint4*>(a.k + d[r].k + 8 * l) = k[r];
        *reinterpret_cast<uint4*>(a.v + d[r].v + 8 * l) = v[r];
        if (l == 0) a.weights[d[r].w] = w[r];
      }
  }
}

}  // namespace

cudaError_t launch_evict(const EvictArgs& a, cudaStream_t s) {
  const unsigned rows = (unsigned)a.n_seqs * (unsigned)a.Hk;
  const size_t smem = sizeof(uint32_t) * (size_t)(a.pages.capacity < SELECT_HELD ? a.pages.capacity : SELECT_HELD);
  cudaError_t e = cudaFuncSetAttribute(k_evict_select, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)(SELECT_HELD * sizeof(uint32_t)));
  if (e != cudaSuccess) return e;
  if ((e = launch_pdl(k_evict_select, dim3(rows), dim3(SELECT_THREADS), smem, s, a)) != cudaSuccess) return e;
  if (a.keep == 0) return cudaSuccess;
  if (!a.to) return launch_pdl(k_evict_walk, dim3(rows), dim3(WALK_THREADS), 0, s, a);
  const long parts = ((long)a.keep + MOVE_ROWS - 1) / MOVE_ROWS;
  return launch_pdl(k_evict_move, dim3(rows, (unsigned)(parts < 65535 ? parts : 65535)), dim3(MOVE_THREADS), 0, s, a);
}

}  // namespace gdn
