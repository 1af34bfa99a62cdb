// gdn_weigh.cu -- the attention weight that each cached key receives:
//   weight_j += sum over the sequence's queries i that see key j, and the heads h of
//               key head kh's group, of  e^{scale q_ih . k_j - lse_ih}
// with lse the attention's log-sums.  The scores are formed transposed, S^T = K Q^T by
// tcgen05 with fp32 accumulators in tensor memory: a key is a TMEM lane and so a thread,
// the sum over queries runs along the thread's own columns, and no value crosses
// threads.  Keys that a tile's queries do not all see take a masked sum, 32 columns at a
// time; the other columns take one fma, one exponential and one addition each, in pairs.
//
// Many queries (prompts): a CTA keeps one tile of 128 keys and streams the query tiles
// that see it through a ring; two groups of four warps take them in turn.
// Few queries (tokens over caches): a CTA keeps the query tile and streams key tiles;
// only as many columns are formed as there are rows, two CTAs to an SM.
//
// A key's sum is formed by one thread in a fixed order and added once to its place
// (by an atomic addition: sequences that share a page each add theirs).
#include <math.h>

#include "gdn_attn.cuh"

namespace gdn {

namespace {

using namespace attn;

// What a query tile's columns need: the negative log-sum in base 2, and the last key that
// the row sees (-1: none, or no row).
struct Columns {
  float nl[CH];
  int lim[CH];
};

// Column r of the query tile from token tok0 on.
__device__ __forceinline__ void column(const WeighArgs& a, const Seq& sq, int kh, int G, int TT, int tok0, int r,
                                       float& nl, int& lim) {
  const int tok = tok0 + r / G;
  float l = -INFINITY;
  if (r < TT * G && tok < sq.ql) l = a.lse[((long)sq.q0 + tok) * a.at.Hq + kh * G + r % G];
  const bool sees = l != -INFINITY;  // (a log-sum of NaN makes the keys' weights NaN)
  nl = sees ? -l * LOG2E : 0.f;
  lim = sees ? tok + sq.kl - sq.ql : -1;
}

// Sum of the key's exponentials over 32 columns.  All rows see every key up to `clean`.
__device__ __forceinline__ float sum32(uint32_t S, const Columns& c, int c0, int key, int tile_end, int clean, float sc) {
  float v[32];
  tc::ld32(S + c0, v);
  float sum[4] = {0.f, 0.f, 0.f, 0.f};
  if (tile_end <= clean) {
#pragma unroll
    for (int j = 0; j < 32; j += 4) {
      const float4 n = *reinterpret_cast<const float4*>(&c.nl[c0 + j]);
      float p[4] = {v[j], v[j + 1], v[j + 2], v[j + 3]};
      tc::axpy2(p[0], p[1], sc, n.x, n.y);
      tc::axpy2(p[2], p[3], sc, n.z, n.w);
#pragma unroll
      for (int i = 0; i < 4; ++i) p[i] = ex2(p[i]);
      tc::add2(sum[0], sum[1], p[0], p[1]);
      tc::add2(sum[2], sum[3], p[2], p[3]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      const float p = ex2(fmaf(v[j], sc, c.nl[c0 + j]));
      if (key <= c.lim[c0 + j]) sum[j & 3] += p;
    }
  }
  return (sum[0] + sum[1]) + (sum[2] + sum[3]);
}

// The key's place among the weights, or null: behind the keys, or on no page.
__device__ __forceinline__ float* place(const WeighArgs& a, const Paged<CH>& pg, int kh, int key) {
  if (key >= pg.kl) return nullptr;
  const int e = pg.row[key / a.at.pages.page];
  if ((unsigned)e >= (unsigned)a.at.pages.n_pages) return nullptr;
  return a.weights + ((long)e * a.at.Hk + kh) * a.at.pages.page + key % a.at.pages.page;
}

// ---- many queries ----------------------------------------------------------------------
constexpr int MANY_THREADS = 320, MANY_SLOTS = 5;

struct ManySmem {
  unsigned char k[TILE];
  unsigned char slot[MANY_SLOTS][TILE];
  Columns cols[2];
  int clean[2][4];  // of 32 columns: the last key that all of their rows see
  float sums[CH];
  uint64_t full[MANY_SLOTS], empty[MANY_SLOTS];
  uint64_t barK, barS[4], barE[4];
  uint32_t tmem;
};

__global__ void __launch_bounds__(MANY_THREADS, 1) k_weigh_many(const __grid_constant__ WeighArgs a) {
  extern __shared__ unsigned char raw[];
  ManySmem& sm = *reinterpret_cast<ManySmem*>(raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u));
  const int tid = threadIdx.x, lane = tid & 31, warp = tc::warp_index();
  pdl_wait();
  pdl_release();
  clear_status(a.at.status);
  const int G = a.at.Hq / a.at.Hk, TT = CH / G;
  // heads run fastest, then sequences, then key tiles: the first ones see the most queries
  const int kh = blockIdx.x % a.at.Hk, seq = blockIdx.x / a.at.Hk % a.at.n_seqs;
  const int tile0 = blockIdx.x / a.at.Hk / a.at.n_seqs;
  Seq sq;
  {
    const int2 q = rows_of(a.at.cu_q, seq, a.at.n_seqs, a.at.total_q);
    sq.q0 = q.x;
    sq.ql = q.y;
    sq.k0 = 0;
    sq.kl = min(max(a.at.k_len[seq], 0), a.at.pages.capacity);
  }
  const int off = sq.kl - sq.ql, nq = (sq.ql + TT - 1) / TT;
  // the last CTA of a sequence takes the key tiles that are left, where there are more than foreseen
  const int tiles = (sq.kl + CH - 1) / CH, tile1 = tile0 == a.key_tiles - 1 ? tiles : min(tile0 + 1, tiles);
  if (tile0 >= tile1 || nq == 0) return;

  if (warp == 9 && lane == 0) {
    for (int k = 0; k < MANY_SLOTS; ++k) {
      tc::mbar_init(&sm.full[k], 1);
      tc::mbar_init(&sm.empty[k], 1);
    }
    tc::mbar_init(&sm.barK, 1);
    for (int k = 0; k < 4; ++k) {
      tc::mbar_init(&sm.barS[k], 1);
      tc::mbar_init(&sm.barE[k], 128);
    }
    tc::mbar_fence_init();
  }
  if (warp == 0) tc::alloc(&sm.tmem, 512);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  tc::Wait w;
  const Paged<CH> pg(a.at, seq, sq.kl);
  // the first query tile that sees the key tile
  auto first = [&](int tile) { return max(0, tile * CH - off) / TT; };

  // `t` counts query tiles over all of the CTA's key tiles
  int t = 0, done = 0;
  for (int tile = tile0; tile < tile1; ++tile, ++done) {
    const int q0 = first(tile);
    if (warp == 9) {
      // (the sums' barrier at a tile's end orders this load behind the last product of the tile before)
      pg.load(a.at.pages, sm.k, &a.at.k, kh, tile * CH, pg.entry(a.at.pages, tile * CH), &sm.barK);
      if (lane == 0) {
        for (int i = q0; i < nq && w.ok; ++i, ++t) {
          if (t >= MANY_SLOTS) w.on(&sm.empty[t % MANY_SLOTS], t / MANY_SLOTS - 1);
          if (w.ok) load_group(sm.slot[t % MANY_SLOTS], &a.at.q, kh, G, sq.q0 + i * TT, &sm.full[t % MANY_SLOTS]);
        }
        // no copy is in flight when the CTA ends
        if (w.ok) {
          w.on(&sm.barK, done);
          for (int u = max(0, t - MANY_SLOTS); u < t; ++u) w.on(&sm.full[u % MANY_SLOTS], u / MANY_SLOTS);
        }
        if (!w.ok) {
          tc::mbar_wait_sleep(&sm.barK, done & 1, 4000000LL);
          for (int k = 0; k < MANY_SLOTS; ++k) tc::mbar_wait_sleep(&sm.full[k], 0, 4000000LL);
        }
      }
      __syncwarp();
    } else if (warp == 8) {
      const uint32_t lead = tc::elect_leader();
      w.warp_on(&sm.barK, done);
      for (int i = q0; i < nq; ++i, ++t) {
        w.warp_on(&sm.full[t % MANY_SLOTS], t / MANY_SLOTS);
        if (t >= 4) w.warp_on(&sm.barE[t & 3], t / 4 - 1);
        tc::fence_after();
        tc::gemm128_by<false>(lead, sm.tmem + 128 * (t & 3), smem_u32(sm.k), smem_u32(sm.slot[t % MANY_SLOTS]), false);
        tc::commit_by(lead, &sm.barS[t & 3]);
        if (tile + 1 < tile1 || i + MANY_SLOTS < nq) tc::commit_by(lead, &sm.empty[t % MANY_SLOTS]);
      }
    } else {
      const int x = warp >> 2, r = tid & 127, key = tile * CH + r;
      const uint32_t lane_base = (uint32_t)(32 * (warp & 3)) << 16;
      const float sc = a.at.scale * LOG2E;
      float* at = x == 0 ? place(a, pg, kh, key) : nullptr;
      float sum = 0.f, nl = 0.f;
      int lim = -1;
      // the group's tiles: those of its parity, counted over the whole CTA
      int i = q0 + ((t ^ x) & 1);
      if (i < nq) column(a, sq, kh, G, TT, i * TT, r, nl, lim);
      for (; i < nq; i += 2) {
        const int u = t + i - q0;
        // the group's columns: all of its threads have read the ones before
        asm volatile("bar.sync %0, 128;" ::"r"(1 + x) : "memory");
        sm.cols[x].nl[r] = nl;
        sm.cols[x].lim[r] = lim;
        const int least = __reduce_min_sync(0xffffffffu, lim);
        if (lane == 0) sm.clean[x][warp & 3] = least;
        asm volatile("bar.sync %0, 128;" ::"r"(1 + x) : "memory");
        if (i + 2 < nq) column(a, sq, kh, G, TT, (i + 2) * TT, r, nl, lim);
        w.warp_on(&sm.barS[u & 3], u / 4);
        tc::fence_after();
        const uint32_t S = sm.tmem + 128 * (u & 3) + lane_base;
        float part[4];
#pragma unroll
        for (int g = 0; g < 4; ++g) part[g] = sum32(S, sm.cols[x], 32 * g, key, tile * CH + CH - 1, sm.clean[x][g], sc);
        tc::fence_before();
        tc::mbar_arrive(&sm.barE[u & 3]);
        sum += (part[0] + part[1]) + (part[2] + part[3]);
      }
      t += nq - q0;
      if (x == 1) sm.sums[r] = sum;
      asm volatile("bar.sync 3, 256;" ::: "memory");
      sum += x == 0 ? sm.sums[r] : 0.f;
      if (at && sum != 0.f) atomicAdd(at, sum);
    }
    if (tile + 1 < tile1) __syncthreads();
  }
  if (!w.ok && a.at.status) atomicOr(a.at.status, 1);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (warp == 0) tc::dealloc(sm.tmem, 512);
}

// ---- few queries -------------------------------------------------------------------------
constexpr int FEW_THREADS = 192, FEW_SLOTS = 2;

struct FewSmem {
  unsigned char q[TILE];
  unsigned char slot[FEW_SLOTS][TILE];
  Columns cols;
  int clean[4];
  uint64_t full[FEW_SLOTS], empty[FEW_SLOTS];
  uint64_t barQ, barS[2], barE[2];
  uint32_t tmem;
};

__global__ void __launch_bounds__(FEW_THREADS, 2) k_weigh_few(const __grid_constant__ WeighArgs a) {
  extern __shared__ unsigned char raw[];
  FewSmem& sm = *reinterpret_cast<FewSmem*>(raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u));
  const int tid = threadIdx.x, lane = tid & 31, warp = tc::warp_index();
  pdl_wait();
  pdl_release();
  if (blockIdx.y == 0) clear_status(a.at.status);
  const int G = a.at.Hq / a.at.Hk, TT = CH / G;
  const int kh = blockIdx.x % a.at.Hk, seq = blockIdx.x / a.at.Hk;
  Seq sq;
  {
    const int2 q = rows_of(a.at.cu_q, seq, a.at.n_seqs, a.at.total_q);
    sq.q0 = q.x;
    sq.ql = q.y;
    sq.k0 = 0;
    sq.kl = min(max(a.at.k_len[seq], 0), a.at.pages.capacity);
  }
  const int nq = (sq.ql + TT - 1) / TT, tiles = (sq.kl + CH - 1) / CH;
  const int tile0 = min((int)blockIdx.y * a.key_tiles, tiles);
  const int n = (blockIdx.y == gridDim.y - 1 ? tiles : min(tile0 + a.key_tiles, tiles)) - tile0;
  if (n == 0 || nq == 0) return;
  const Paged<CH> pg(a.at, seq, sq.kl);

  int entry = -1;
  if (warp == 5) entry = pg.entry(a.at.pages, tile0 * CH);
  if (warp == 5 && lane == 0) {
    for (int k = 0; k < FEW_SLOTS; ++k) {
      tc::mbar_init(&sm.full[k], 1);
      tc::mbar_init(&sm.empty[k], 1);
    }
    tc::mbar_init(&sm.barQ, 1);
    for (int k = 0; k < 2; ++k) {
      tc::mbar_init(&sm.barS[k], 1);
      tc::mbar_init(&sm.barE[k], 128);
    }
    tc::mbar_fence_init();
  }
  if (warp == 0) tc::alloc(&sm.tmem, 256);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  tc::Wait w;

  // `t` counts key tiles over all query tiles (mostly one)
  int t = 0;
  for (int i = 0; i < nq; ++i) {
    const int tok0 = i * TT, rows = min(TT, sq.ql - tok0) * G, N = (rows + 15) & ~15;
    if (warp == 5) {
      if (lane == 0) load_group(sm.q, &a.at.q, kh, G, sq.q0 + tok0, &sm.barQ);
      __syncwarp();
      const int t0 = t;
      for (; t < t0 + n && w.ok; ++t) {
        const int key0 = (tile0 + t - t0) * CH;
        if (t >= FEW_SLOTS) w.on(&sm.empty[t % FEW_SLOTS], t / FEW_SLOTS - 1);
        w.ok = __all_sync(0xffffffffu, w.ok);
        if (w.ok) pg.load(a.at.pages, sm.slot[t % FEW_SLOTS], &a.at.k, kh, key0, entry, &sm.full[t % FEW_SLOTS]);
        // (behind the last tile the next query tile begins with the first)
        entry = pg.entry(a.at.pages, t + 1 < t0 + n ? key0 + CH : tile0 * CH);
      }
      if (lane == 0) {  // no copy is in flight when the CTA ends
        if (w.ok) {
          w.on(&sm.barQ, i);
          for (int u = max(0, t - FEW_SLOTS); u < t; ++u) w.on(&sm.full[u % FEW_SLOTS], u / FEW_SLOTS);
        }
        if (!w.ok) {
          tc::mbar_wait_sleep(&sm.barQ, i & 1, 4000000LL);
          for (int k = 0; k < FEW_SLOTS; ++k) tc::mbar_wait_sleep(&sm.full[k], 0, 4000000LL);
        }
      }
      __syncwarp();
    } else if (warp == 4) {
      const uint32_t lead = tc::elect_leader();
      w.warp_on(&sm.barQ, i);
      for (int u = t + n; t < u; ++t) {
        w.warp_on(&sm.full[t % FEW_SLOTS], t / FEW_SLOTS);
        if (t >= 2) w.warp_on(&sm.barE[t & 1], t / 2 - 1);
        tc::fence_after();
        tc::gemm128xN_by(lead, sm.tmem + 128 * (t & 1), smem_u32(sm.slot[t % FEW_SLOTS]), smem_u32(sm.q), N);
        tc::commit_by(lead, &sm.barS[t & 1]);
        if (i + 1 < nq || t + FEW_SLOTS < u) tc::commit_by(lead, &sm.empty[t % FEW_SLOTS]);
      }
    } else {
      const int r = tid;
      const uint32_t lane_base = (uint32_t)(32 * warp) << 16;
      const float sc = a.at.scale * LOG2E;
      float nl;
      int lim;
      column(a, sq, kh, G, TT, tok0, r, nl, lim);
      sm.cols.nl[r] = nl;
      sm.cols.lim[r] = lim;
      const int least = __reduce_min_sync(0xffffffffu, lim);
      if (lane == 0) sm.clean[warp] = least;
      asm volatile("bar.sync 1, 128;" ::: "memory");
      for (int u = t + n, tile = tile0; t < u; ++t, ++tile) {
        const int key = tile * CH + r;
        float* at = place(a, pg, kh, key);
        w.warp_on(&sm.barS[t & 1], t / 2);
        tc::fence_after();
        const uint32_t S = sm.tmem + 128 * (t & 1) + lane_base;
        float sum = 0.f;
        // (columns past N hold what earlier products left; no row there sees a key)
        for (int g = 0; 32 * g < N; ++g) sum += sum32(S, sm.cols, 32 * g, key, tile * CH + CH - 1, sm.clean[g], sc);
        tc::fence_before();
        tc::mbar_arrive(&sm.barE[t & 1]);
        if (at && sum != 0.f) atomicAdd(at, sum);
      }
    }
    if (i + 1 < nq) __syncthreads();  // the query tile and its columns have been read
  }
  if (!w.ok && a.at.status) atomicOr(a.at.status, 1);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (warp == 0) tc::dealloc(sm.tmem, 256);
}

}  // namespace

cudaError_t launch_weigh(const WeighArgs& a, cudaStream_t s) {
  const auto kernel = a.few ? k_weigh_few : k_weigh_many;
  const size_t smem = (a.few ? sizeof(FewSmem) : sizeof(ManySmem)) + 1024;
  static_assert(sizeof(ManySmem) + 1024 <= 227 * 1024 && 2 * (sizeof(FewSmem) + 2048) <= 228 * 1024, "shared memory");
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  const unsigned rows = (unsigned)a.at.Hk * (unsigned)a.at.n_seqs;
  const dim3 grid = a.few ? dim3(rows, (unsigned)a.n_splits) : dim3(rows * (unsigned)a.key_tiles);
  return launch_pdl(kernel, grid, dim3(a.few ? FEW_THREADS : MANY_THREADS), smem, s, a);
}

}  // namespace gdn
