// gdn_evict.cu -- eviction of the lightest keys from a cache in pages.
//
// Per sequence and key head: the last `recent` keys stay, and of the others the
// heaviest, `budget` in all; equal weights stay from the lowest index on.  What stays
// moves, in its order, to the first rows of the target pages (keys, values and weights).
// Keys on absent pages are gone already and never stay.
//
// k_evict_select, a block or a cluster of them to a sequence and head, finds the smallest
// weight that stays by its digits: weights are mapped to unsigned numbers of the same
// order, the digits that all share are passed over, and each further digit of 11 bits takes
// one count over the candidates, until all that have the digits so far stay.  The weights
// are held in shared memory where they fit.  A last pass in index order writes the list of
// rows that stay (as places in the cache): a warp counts over its own range of keys, scans
// over blocks, warps and lanes give each its place.
//
// k_evict_move copies the rows of the lists, 16 lanes to a row.  Into other pages any
// block may take any part of a list.  In place (the target pages are the sequence's
// own) a block or a cluster walks a list in its order: a row's target never lies behind it, so
// what a round writes are rows that this round and the earlier ones have read, and the next
// round's rows are on their way meanwhile.
//
// Bound: HBM, 4 bytes a key and head and 1,024 a row that stays.  32 caches of 1 to 16214 keys,
// 4096 kept of 4 heads: 89 us in a row of calls, the copies some 70 (424 MB of traffic, 6.0 TB/s; a plain copy with as
// much 65), the lists some 20, by the longest cache's block.  1024 keys, 512 kept: 9 us,
// latencies.  In place the walk's rounds bound: the 32 caches, with a block to a list, 100 us,
// one of 65536 keys, half of them kept, by clusters of eight 113 (into other pages 43).
#include <stdint.h>

#include "gdn_kernels.cuh"
#include "gdn_tc05.cuh"

namespace gdn {

namespace {

constexpr int SELECT_THREADS = 1024, SELECT_WARPS = SELECT_THREADS / 32;
constexpr int SELECT_HELD = 49152;  // weights that shared memory holds
// Bits of a digit.  With eight, weights of few binades meet in a few dozen places, and a warp's
// additions there wait for one another (the 32 caches 2 us more).
constexpr int DIGIT = 11;
constexpr int PASSES = (32 + DIGIT - 1) / DIGIT;
static_assert(1 << DIGIT == 2 * SELECT_THREADS, "two digits to a thread");
// Rows of a list to a block, 16 side by side: the 32 caches into other pages 89 us, with 64 rows 101,
// with 128 124 (fewer blocks to an SM; with six of 32 rows instead of eight 94).
constexpr int MOVE_THREADS = 256, MOVE_ROWS = 32;
// Rows to a round of a block in place: 65536 keys, half kept, 113 us, the 32 caches 100; with 64 rows 147 and
// 109, with 256, which spill, 176 and 276.
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

// A value of CTA `rank` of the cluster, where p points in this one's shared memory.
__device__ __forceinline__ uint2 ld_cluster(const uint32_t* p, int rank) {
  uint32_t at;
  uint2 v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at) : "memory");
  return v;
}

__global__ void __launch_bounds__(SELECT_THREADS, 1) k_evict_select(const __grid_constant__ EvictArgs a) {
  extern __shared__ __align__(16) uint32_t held[];
  __shared__ __align__(16) uint32_t hist[PASSES][1 << DIGIT];
  __shared__ __align__(8) uint32_t range[2];    // complement of the least rank, the highest one
  __shared__ __align__(8) uint32_t present[2];  // of the candidates, of the last ones
  __shared__ __align__(8) uint32_t total[2];    // that stay, tied
  __shared__ int digit, above, same;
  __shared__ int warps[SELECT_WARPS][2];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int C = a.split, rank = blockIdx.x % C, kh = blockIdx.x / C % a.Hk, seq = blockIdx.x / C / a.Hk;
  auto meet = [&] {  // the threads of all CTAs of the list
    if (C > 1) {
      tc::cluster_arrive();
      tc::cluster_wait();
    } else {
      __syncthreads();
    }
  };
  pdl_wait();
  pdl_release();
  const Cut c = cut_of(a, seq);
  const int* table = a.table + (long)seq * a.pages.table_stride;
  // this CTA's keys, and the candidates among them
  const int span = ((c.kl + C - 1) / C + 127) & ~127;
  const int b0 = min(rank * span, c.kl), b1 = min(b0 + span, c.kl), old1 = min(b1, c.old);
  const bool fits = span <= SELECT_HELD;
  // ranks of the candidates j .. j + 3 (j a multiple of 4: one page); 0: none, or on an absent page
  auto fetch = [&](int j) -> uint4 {
    const int t = a.pages.page_of(j), e = table[t];
    if ((unsigned)e >= (unsigned)a.pages.n_pages) return make_uint4(0u, 0u, 0u, 0u);
    const float* at = a.weights + ((long)e * a.Hk + kh) * a.pages.page + (j - t * a.pages.page);
    const float4 w = *reinterpret_cast<const float4*>(at);
    return make_uint4(rank_of(w.x), j + 1 < c.old ? rank_of(w.y) : 0u, j + 2 < c.old ? rank_of(w.z) : 0u,
                      j + 3 < c.old ? rank_of(w.w) : 0u);
  };
  auto ranks = [&](int j) { return fits ? *reinterpret_cast<const uint4*>(held + (j - b0)) : fetch(j); };

#pragma unroll
  for (int p = 0; p < PASSES; ++p) hist[p][tid] = hist[p][tid + SELECT_THREADS] = 0u;
  if (tid < 2) range[tid] = present[tid] = 0u;
  __syncthreads();
  uint32_t lo = 0xffffffffu, hi = 0u;
  int n0 = 0, n1 = 0;
#pragma unroll 4
  for (int j = b0 + 4 * tid; j < old1; j += 4 * SELECT_THREADS) {
    const uint4 r = fetch(j);
    if (fits) *reinterpret_cast<uint4*>(held + (j - b0)) = r;
    const uint32_t x[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (x[i]) {
        lo = min(lo, x[i]);
        hi = max(hi, x[i]);
        ++n0;
      }
  }
  for (int j = max(b0, c.old) + tid; j < b1; j += SELECT_THREADS)
    n1 += (unsigned)table[a.pages.page_of(j)] < (unsigned)a.pages.n_pages;
  lo = __reduce_min_sync(0xffffffffu, lo);
  hi = __reduce_max_sync(0xffffffffu, hi);
  n0 = __reduce_add_sync(0xffffffffu, n0);
  n1 = __reduce_add_sync(0xffffffffu, n1);
  if (lane == 0) {
    atomicMax(&range[0], ~lo);
    atomicMax(&range[1], hi);
    atomicAdd(&present[0], (uint32_t)n0);
    atomicAdd(&present[1], (uint32_t)n1);
  }
  meet();
  const uint2 ends = lane < C ? ld_cluster(range, lane) : make_uint2(0u, 0u);
  const uint2 counts = lane < C ? ld_cluster(present, lane) : make_uint2(0u, 0u);
  const uint32_t least = ~__reduce_max_sync(0xffffffffu, ends.x), most = __reduce_max_sync(0xffffffffu, ends.y);
  const int candidates = __reduce_add_sync(0xffffffffu, counts.x), recent = __reduce_add_sync(0xffffffffu, counts.y);
  const int take = min(candidates, a.budget - recent);  // of the candidates (recent <= budget)
  if (kh == 0 && rank == 0 && tid == 0) a.new_len[seq] = take + recent;
  // The candidates that stay: ranks above `edge`, and the first `ties` of rank `edge`.
  uint32_t edge = 0u;  // (all of them)
  int ties = 0;
  if (take == 0) {
    edge = 0xffffffffu;  // none: no rank is above it, and no number has it
  } else if (take < candidates) {
    // the digits below the highest bit in which candidates differ
    int shift = 32 - __clz(least ^ most);
    edge = shift < 32 ? most >> shift << shift : 0u;
    ties = take;
    for (int p = 0; shift > 0; ++p) {
      const int bits = min(shift, DIGIT), low = shift - bits;
      const uint32_t mask = shift < 32 ? ~0u << shift : 0u;
      for (int j = b0 + 4 * tid; j < old1; j += 4 * SELECT_THREADS) {
        const uint4 r = ranks(j);
        const uint32_t x[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (x[i] && (x[i] & mask) == edge) atomicAdd(&hist[p][x[i] >> low & ((1u << bits) - 1u)], 1u);
      }
      meet();
      // the digit at which the count from the top reaches what is still to take: a warp has 64 of them
      int d0 = 0, d1 = 0;
      for (int r = 0; r < C; ++r) {
        const uint2 n = ld_cluster(&hist[p][2 * tid], r);
        d0 += (int)n.x;
        d1 += (int)n.y;
      }
      int from = d0 + d1;  // in this lane's digits and those above in the warp
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_down_sync(0xffffffffu, from, o);
        if (lane + o < 32) from += y;
      }
      if (lane == 0) warps[warp][0] = from;
      __syncthreads();
      const int over = __reduce_add_sync(0xffffffffu, lane > warp ? warps[lane][0] : 0) + from - d0 - d1;  // above them
      if (over < ties && over + d0 + d1 >= ties) {
        const bool upper = over + d1 >= ties;
        digit = 2 * tid + upper;
        above = upper ? over : over + d1;
        same = upper ? d1 : d0;
      }
      __syncthreads();
      edge |= (uint32_t)digit << low;
      ties -= above;
      shift = low;
      if (ties == same) {  // all that have these digits: no need to tell them apart
        edge = edge ? edge - 1u : 0u;
        ties = 0;
        break;
      }
    }
  }

  // the list, in index order: warp w's range of keys, counted first; a lane has four at a time
  const int per = ((b1 - b0 + SELECT_WARPS - 1) / SELECT_WARPS + 127) & ~127;
  const int j0 = min(b0 + warp * per, b1), j1 = min(j0 + per, b1);
  // of the keys j .. j + 3 on page e: bits 0 to 3, those that stay, 4 to 7, those that stay if they are
  // among the first ties
  auto kinds = [&](int j, int e) -> uint32_t {
    if (j >= j1 || (unsigned)e >= (unsigned)a.pages.n_pages) return 0u;
    uint32_t y = 0u;
    if (j < c.old) {
      const uint4 r = ranks(j);
      const uint32_t x[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) y |= (x[i] > edge ? 1u : x[i] == edge ? 16u : 0u) << i;
      if (edge == 0u) y &= 15u;  // (a rank of zero is no key)
    }
    if (j + 4 > c.old) {  // (the last ones begin here, or earlier)
      const uint32_t last = 0xfu << max(c.old - j, 0) & 0xfu >> max(j + 4 - c.kl, 0);
      y = (y & ~(last * 17u)) | last;
    }
    return y;
  };
  auto page_at = [&](int j) { return j < j1 ? table[a.pages.page_of(j)] : -1; };
  int stay = 0, tied = 0;
#pragma unroll 2
  for (int j = j0 + 4 * lane; j < j1; j += 128) {
    const uint32_t y = kinds(j, page_at(j));
    stay += __popc(y & 15u);
    tied += __popc(y >> 4);
  }
  stay = __reduce_add_sync(0xffffffffu, stay);
  tied = __reduce_add_sync(0xffffffffu, tied);
  if (lane == 0) {
    warps[warp][0] = stay;
    warps[warp][1] = tied;
  }
  __syncthreads();
  int out = 0, seen = 0;  // ahead of the warp's keys: those that stay, the tied ones
  if (C > 1) {
    if (warp == 0) {
      const int x = __reduce_add_sync(0xffffffffu, warps[lane][0]), y = __reduce_add_sync(0xffffffffu, warps[lane][1]);
      if (lane == 0) {
        total[0] = (uint32_t)x;
        total[1] = (uint32_t)y;
      }
    }
    meet();
    const uint2 ahead = lane < rank ? ld_cluster(total, lane) : make_uint2(0u, 0u);
    out = __reduce_add_sync(0xffffffffu, ahead.x);
    seen = __reduce_add_sync(0xffffffffu, ahead.y);
  }
  for (int i = 0; i < warp; ++i) {
    out += warps[i][0];
    seen += warps[i][1];
  }
  int* list = a.list + ((long)seq * a.Hk + kh) * a.keep;
  for (int j = j0; j < j1; j += 128) {
    const int key = j + 4 * lane, e = page_at(key);
    const uint32_t y = kinds(key, e), mine = __popc(y & 15u) | __popc(y >> 4) << 16;
    uint32_t upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t z = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += z;
    }
    int s = out + (int)((upto - mine) & 0xffffu), t = seen + (int)((upto - mine) >> 16);
    const int row = e * a.pages.page + key - a.pages.page_of(key) * a.pages.page;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool stays = y >> i & 1u, tie = y >> (4 + i) & 1u;
      if (stays || (tie && t < ties)) list[s + min(t, ties)] = row + i;
      s += stays;
      t += tie;
    }
    const uint32_t all = __shfl_sync(0xffffffffu, upto, 31);
    out += (int)(all & 0xffffu);
    seen += (int)(all >> 16);
  }
  if (C > 1) meet();  // no CTA ends while another reads its counts
}

// Keys, values and weight of row `row` (page * page size + row in it), one lane's share of 16.
struct Row {
  uint4 k, v;
  float w;
  __device__ __forceinline__ void read(const EvictArgs& a, int kh, int l, int row) {
    const int e = a.pages.page_of(row), i = row - e * a.pages.page;
    k = *reinterpret_cast<const uint4*>(a.k + e * a.sk_page + i * a.sk_row + kh * a.sk_head + 8 * l);
    v = *reinterpret_cast<const uint4*>(a.v + e * a.sv_page + i * a.sv_row + kh * a.sv_head + 8 * l);
    w = a.weights[((long)e * a.Hk + kh) * a.pages.page + i];
  }
  __device__ __forceinline__ void write(const EvictArgs& a, int kh, int l, int row) const {
    const int e = a.pages.page_of(row), i = row - e * a.pages.page;
    *reinterpret_cast<uint4*>(a.k + e * a.sk_page + i * a.sk_row + kh * a.sk_head + 8 * l) = k;
    *reinterpret_cast<uint4*>(a.v + e * a.sv_page + i * a.sv_row + kh * a.sv_head + 8 * l) = v;
    if (l == 0) a.weights[((long)e * a.Hk + kh) * a.pages.page + i] = w;
  }
};
// Row i of the pages that `table` lists (-1: on an absent page).
__device__ __forceinline__ int row_at(const EvictArgs& a, const int* table, int i) {
  const int t = a.pages.page_of(i), e = table[t];
  return (unsigned)e < (unsigned)a.pages.n_pages ? e * a.pages.page + (i - t * a.pages.page) : -1;
}

__global__ void __launch_bounds__(MOVE_THREADS, 8) k_evict_move(const __grid_constant__ EvictArgs a) {
  const int kh = blockIdx.x % a.Hk, seq = blockIdx.x / a.Hk;
  const int l = threadIdx.x & 15, i0 = threadIdx.x >> 4;
  pdl_wait();
  pdl_release();
  const int n = a.new_len[seq];
  const int* to = a.to + (long)seq * a.to_stride;
  const int* list = a.list + ((long)seq * a.Hk + kh) * a.keep;
  constexpr int R = MOVE_ROWS / (MOVE_THREADS / 16);
  for (long base = (long)blockIdx.y * MOVE_ROWS; base < a.keep; base += (long)gridDim.y * MOVE_ROWS) {
    int from[R], dst[R];
    Row x[R];
    // (the list, the target's page and the length are asked for at once: what lies behind the length is not used)
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int i = min((int)base + i0 + r * (MOVE_THREADS / 16), a.keep - 1);
      from[r] = list[i];
      dst[r] = row_at(a, to, i);
    }
    if (base >= n) return;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if ((int)base + i0 + r * (MOVE_THREADS / 16) >= n) dst[r] = -1;
      if (dst[r] >= 0) x[r].read(a, kh, l, from[r]);
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (dst[r] >= 0) x[r].write(a, kh, l, dst[r]);
  }
}

__global__ void __launch_bounds__(WALK_THREADS) k_evict_walk(const __grid_constant__ EvictArgs a) {
  const int C = a.walks, rank = blockIdx.x % C, kh = blockIdx.x / C % a.Hk, seq = blockIdx.x / C / a.Hk;
  const int l = threadIdx.x & 15, i0 = rank * WALK_ROWS + (threadIdx.x >> 4);
  pdl_wait();
  pdl_release();
  const int n = a.new_len[seq], step = C * WALK_ROWS;
  const int* table = a.table + (long)seq * a.pages.table_stride;
  const int* list = a.list + ((long)seq * a.Hk + kh) * a.keep;
  constexpr int R = WALK_ROWS / (WALK_THREADS / 16);
  struct Round {
    int dst[R];
    Row x[R];
  };
  int from[R], to[R];  // the places of the round whose rows are read next
  auto ask = [&](int base) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int i = i0 + r * (WALK_THREADS / 16);
      from[r] = to[r] = -1;
      if (base < n && i < n - base) {
        from[r] = list[base + i];
        to[r] = row_at(a, table, base + i);
      }
    }
  };
  auto read = [&](Round& t) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      t.dst[r] = to[r] == from[r] ? -1 : to[r];  // (it stays where it is)
      if (t.dst[r] >= 0) t.x[r].read(a, kh, l, from[r]);
    }
  };
  auto round = [&](int base, const Round& now, Round& next) {
    read(next);  // (rows behind all that this round writes)
    ask(base + 2 * step);
    if (C > 1) {  // the round's rows have been read
      tc::cluster_arrive();
      tc::cluster_wait();
    } else {
      __syncthreads();
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (now.dst[r] >= 0) now.x[r].write(a, kh, l, now.dst[r]);
  };
  Round even, odd;
  ask(0);
  read(even);
  ask(step);
  for (int base = 0; base < n; base += 2 * step) {
    round(base, even, odd);
    if (n - base <= step) break;
    round(base + step, odd, even);
  }
}

}  // namespace

cudaError_t launch_evict(const EvictArgs& a, cudaStream_t s) {
  const unsigned rows = (unsigned)a.n_seqs * (unsigned)a.Hk;
  const long span = (((long)a.pages.capacity + a.split - 1) / a.split + 127) & ~127L;  // as in the kernel, at most
  const size_t smem = sizeof(uint32_t) * (size_t)(span < SELECT_HELD ? span : SELECT_HELD);
  cudaError_t e = cudaFuncSetAttribute(k_evict_select, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)(SELECT_HELD * sizeof(uint32_t)));
  if (e != cudaSuccess) return e;
  auto launch = [&](auto kernel, int ctas, int threads, size_t bytes) {  // `ctas` to a list
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(rows * (unsigned)ctas);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)ctas;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, a);
  };
  if ((e = launch(k_evict_select, a.split, SELECT_THREADS, smem)) != cudaSuccess) return e;
  if (a.keep == 0) return cudaSuccess;
  if (!a.to) return launch(k_evict_walk, a.walks, WALK_THREADS, 0);
  const long parts = ((long)a.keep + MOVE_ROWS - 1) / MOVE_ROWS;
  return launch_pdl(k_evict_move, dim3(rows, (unsigned)(parts < 65535 ? parts : 65535)), dim3(MOVE_THREADS), 0, s, a);
}

}  // namespace gdn
