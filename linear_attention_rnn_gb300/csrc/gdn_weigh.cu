// gdn_weigh.cu -- the attention weight that each cached key receives:
//   weight_j += sum over the sequence's queries i that see key j, and the heads h of
//               key head kh's group, of  e^{scale q_ih . k_j - lse_ih}
// with lse the attention's log-sums.  The scores are formed transposed, S^T = K Q^T by
// tcgen05 with fp32 accumulators in tensor memory: a key is a TMEM lane and so a thread,
// the sum over queries runs along the thread's own columns, and no value crosses
// threads.  Keys that a tile's queries do not all see take a masked sum, 32 columns at a
// time; the other columns take one fma, one exponential and one addition each, in pairs.
//
// Many queries (prompts): a CTA, or a pair of them, takes one tile of 128 keys after another and
// streams the query tiles that see it through a ring; four groups of four warps take them in
// turn.  One warp plans the key tiles and loads them, one loads the queries; the loads and
// products of a key tile begin while the one before is summed up.
// Few queries (tokens over caches): a CTA keeps the query tile and streams key tiles;
// only as many columns are formed as there are rows, two CTAs to an SM, each with an
// equal run of all sequences' key tiles.
//
// Where lengths may differ both are started, and each takes the sequences that suit it.
//
// A key's sum is formed by one thread in a fixed order (a query tile's terms in four chains, then
// tile by tile, so that no chain is longer than some 64 additions and one to 128 terms) and added once to
// its place (by an atomic addition: sequences that share a page each add theirs).
//
// Bounds.  Prompts: shared memory, where a tile's product of 128 x 128 reads 64 KB beside the 32
// that the load writes, 768 clocks; a tile takes 0.41 us (its product alone 0.33, its
// exponentials 0.27).  8192 + 640 + 77 tokens with 16/4 heads: 105 us (138 GFLOP, 1.3 PFLOP/s; 115
// where a key tile began behind the last one's end).  With the keys in tensor memory there is
// room for three S buffers only, whose way round is then longer: 120 us, handed back by halves
// 114.  Chunks over caches: the same (2048 over 32768 keys 192 us), short ones the latency of a key
// tile's start, some 2.5 us (16 x 128 tokens over 4096 keys 41 us).  Tokens: HBM, 32 over 1 to
// 16214 keys 47 us for 274 MB, 5.8 TB/s.
#include <math.h>

#include "gdn_attn.cuh"

namespace gdn {

namespace {

using namespace attn;

// What a query tile's columns need: the negative log-sum in base 2, and the last key that
// the row sees (-1: none, or no row).
template <int N>
struct Columns {
  float nl[N];
  int lim[N];
};

// Whether all 128 threads of named barrier `id` say so.
__device__ __forceinline__ bool all128(int id, bool ok) {
  uint32_t y;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\tbar.red.and.pred q, %2, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}\n"
      : "=r"(y)
      : "r"((uint32_t)ok), "r"(id)
      : "memory");
  return y != 0;
}

// Inclusive sums over the lanes of a warp, and one lane's value.
__device__ __forceinline__ long sums(long v) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long y = (long)__shfl_up_sync(0xffffffffu, (unsigned long long)v, o);
    if ((threadIdx.x & 31) >= o) v += y;
  }
  return v;
}
__device__ __forceinline__ long from(long v, int lane) {
  return (long)__shfl_sync(0xffffffffu, (unsigned long long)v, lane);
}

// Column r of the query tile of TT tokens from token tok0 on.
__device__ __forceinline__ void column(const WeighArgs& a, const Seq& sq, int kh, int G, int TT, int tok0, int r,
                                       float& nl, int& lim) {
  const int tok = tok0 + r / G;
  float l = -INFINITY;
  if (r < TT * G && tok < sq.ql) l = a.lse[((long)sq.q0 + tok) * a.at.Hq + kh * G + r % G];
  const bool sees = l != -INFINITY;  // (a log-sum of NaN makes the keys' weights NaN)
  nl = sees ? -l * LOG2E : 0.f;
  lim = sees ? tok + sq.kl - sq.ql : -1;
}

// Adds the key's exponentials over the 32 columns v from column c0 on to sum.  All rows see
// every key up to `clean`.
template <int N>
__device__ __forceinline__ void add32(const float (&v)[32], const Columns<N>& c, int c0, int key, int tile_end, int clean,
                                      float sc, float (&sum)[4]) {
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
}

// The key's place among the weights, or null: behind the keys, or on no page.
__device__ __forceinline__ float* place(const WeighArgs& a, const Paged<CH>& pg, int kh, int key) {
  if (key >= pg.kl) return nullptr;
  const int t = a.at.pages.page_of(key), e = pg.row[t];
  if ((unsigned)e >= (unsigned)a.at.pages.n_pages) return nullptr;
  return a.weights + ((long)e * a.at.Hk + kh) * a.at.pages.page + (key - t * a.at.pages.page);
}

// ---- many queries ----------------------------------------------------------------------
// Two warps issue in turn: a product holds its issuer for the time that it takes, and the two
// waits before the next one would come on top of that (a prompt of 8192 tokens: 131 us with
// one, 114 with two).  An even number of slots and of S buffers, so that a barrier's phases
// are one issuer's, in their order.
constexpr int MANY_GROUPS = 4, MANY_THREADS = 128 * MANY_GROUPS + 128, MANY_SLOTS = 4, MANY_S = 4;
static_assert(MANY_SLOTS % 2 == 0 && MANY_S % 2 == 0, "each issuer's own");
static_assert(MANY_GROUPS == MANY_S, "a group's scores lie in one buffer");

// A unit of work: a key tile and head, and the CTA's share of the query tiles that see it.
struct Unit {
  int kh, tile, kl, off;  // off: keys ahead of the first query
  int row, ql;            // the sequence's rows of q
  int q0, mine;           // the first of the CTA's query tiles, and how many
  const int* table;
};

struct ManySmem {
  unsigned char k[2][TILE];
  unsigned char slot[MANY_SLOTS][TILE];
  Columns<CH> cols[MANY_GROUPS][2];
  int clean[MANY_GROUPS][2][4];  // of 32 columns: the last key that all of their rows see
  float sums[2][MANY_GROUPS - 1][CH];
  float other[2][CH];  // the other CTA's sums
  Unit unit[2];
  uint64_t full[MANY_SLOTS], empty[MANY_SLOTS];
  // the unit there, its keys there, both free again
  uint64_t barU[2], barK[2], barF[2], barS[MANY_S], barE[MANY_S];
  uint32_t tmem;
};

__global__ void __launch_bounds__(MANY_THREADS, 1) k_weigh_many(const __grid_constant__ WeighArgs a) {
  extern __shared__ unsigned char raw[];
  ManySmem& sm = *reinterpret_cast<ManySmem*>(raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u));
  const int tid = threadIdx.x, lane = tid & 31, warp = tc::warp_index();
  constexpr int ISSUES = 4 * MANY_GROUPS, LOADS = ISSUES + 2, PLANS = ISSUES + 3, NG = MANY_GROUPS, NS = MANY_S;
  pdl_wait();
  pdl_release();
  if (!a.rule.few) clear_status(a.at.status);  // (the kernel ahead has)
  const int G = a.at.Hq / a.at.Hk, TT = CH / G;
  const int split = a.rule.split, rank = blockIdx.x % split, team = blockIdx.x / split, teams = gridDim.x / split;
  // the lengths of a sequence, and its key tiles (none without queries, or where it is not this kernel's)
  auto rows = [&](int s) { return rows_of(a.at.cu_q, s, a.at.n_seqs, a.at.total_q); };
  auto keys = [&](int s) { return min(max(a.at.k_len[s], 0), a.at.pages.capacity); };
  auto count = [&](int ql, int kl) {
    return ql > 0 && (a.rule.many == WeighRule::ALL || !WeighRule::small(ql, G)) ? (kl + CH - 1) / CH : 0;
  };
  auto tiles = [&](int s) { return count(rows(s).y, keys(s)); };
  int2 lane_q = make_int2(0, 0);  // of the first 32 sequences
  int lane_kl = 0;
  if (lane < a.at.n_seqs) {
    lane_q = rows(lane);
    lane_kl = keys(lane);
  }
  const int own = count(lane_q.y, lane_kl);

  if (warp == LOADS && lane == 0) {
    for (int k = 0; k < MANY_SLOTS; ++k) {
      tc::mbar_init(&sm.full[k], 1);
      tc::mbar_init(&sm.empty[k], 1);
    }
    for (int k = 0; k < 2; ++k) {
      tc::mbar_init(&sm.barU[k], 1);
      tc::mbar_init(&sm.barK[k], 1);
      tc::mbar_init(&sm.barF[k], 4 * NG + 3);
    }
    for (int k = 0; k < NS; ++k) {
      tc::mbar_init(&sm.barS[k], 1);
      tc::mbar_init(&sm.barE[k], 128);
    }
    tc::mbar_fence_init();
  }
  if (warp == 0) tc::alloc(&sm.tmem, 512);
  // Units, of up to 32 sequences those with the most queries first, to the teams there and back again.
  // Every warp knows how many are the team's, whatever its waits come to.
  int n_units;
  {
    // (summed over the lanes at the end instead, this loop has the compiler order the groups' in
    // another way, which takes 5% longer)
    long all = __reduce_add_sync(0xffffffffu, own);
    for (int s = 32; s < a.at.n_seqs; s += 32)
      all += __reduce_add_sync(0xffffffffu, s + lane < a.at.n_seqs ? tiles(s + lane) : 0);
    all *= a.at.Hk;
    const long rounds = all / teams, rest = all - rounds * teams;
    n_units = (int)rounds + ((rounds & 1 ? teams - 1 - team : team) < rest ? 1 : 0);
  }
  tc::fence_before();
  if (split > 1) {  // (the other CTA's shared memory is there from here on)
    tc::cluster_arrive();
    tc::cluster_wait();
  } else {
    __syncthreads();
  }
  tc::fence_after();
  tc::Wait w;

  // t counts query tiles over all of the CTA's units.
  int t = 0;
  if (warp == PLANS) {
    // of more sequences than lanes a lane adds up a 32nd, one behind another
    const int block = (a.at.n_seqs + 31) / 32;
    long mine = 0, upto = 0;
    if (block > 1) {
#pragma unroll 4
      for (int i = 0; i < block; ++i) {
        const int s = lane * block + i, k = tiles(min(s, a.at.n_seqs - 1));
        if (s < a.at.n_seqs) mine += k;
      }
      upto = sums(mine);
    }
    for (int n = 0; n < n_units; ++n) {
      const int b = n & 1;
      const long unit = (long)n * teams + (n & 1 ? teams - 1 - team : team), rank_of = unit / a.at.Hk;
      int seq, from_end = 0, from_start = 0;
      if (block == 1) {  // (a tile's index from its sequence's end)
        const int2 at = find_nth(tiles, own, a.at.n_seqs, (int)rank_of);
        seq = max(at.x, 0);
        from_end = at.y;
      } else {  // one sequence behind another: enough of them to even out (sorted, by a search over all
                // sequences for each unit, 1000 prompts of 100 tokens took 509 us for 117)
        int l = __ffs((int)__ballot_sync(0xffffffffu, upto > rank_of)) - 1;
        long before = from(upto - mine, l);
        for (int s = l * block;; s += 32) {
          const long k = s + lane < a.at.n_seqs ? tiles(s + lane) : 0, in = before + sums(k);
          const unsigned past = __ballot_sync(0xffffffffu, in > rank_of);
          if (past) {
            l = __ffs((int)past) - 1;
            seq = s + l;
            from_start = (int)(rank_of - from(in - k, l));
            break;
          }
          before = from(in, 31);
        }
      }
      int2 q;
      Unit u;
      if (seq < 32) {
        q = make_int2(__shfl_sync(0xffffffffu, lane_q.x, seq), __shfl_sync(0xffffffffu, lane_q.y, seq));
        u.kl = __shfl_sync(0xffffffffu, lane_kl, seq);
      } else {
        q = rows(seq);
        u.kl = keys(seq);
      }
      u.kh = (int)(unit % a.at.Hk);
      u.off = u.kl - q.y;
      u.tile = block == 1 ? (u.kl + CH - 1) / CH - 1 - from_end : from_start;
      u.row = q.x;
      u.ql = q.y;
      u.table = a.at.table + (long)seq * a.at.pages.table_stride;
      // the CTA's query tiles, of those that see the key tile: q0 + split j
      u.q0 = max(0, u.tile * CH - u.off) / TT + rank;
      u.mine = max(0, (q.y + TT - 1) / TT - u.q0 + split - 1) / split;
      const Paged<CH> pg(a.at, seq, u.kl);
      const int entry = pg.entry(a.at.pages, u.tile * CH);
      if (n >= 2) w.on(&sm.barF[b], n / 2 - 1);
      w.ok = __all_sync(0xffffffffu, w.ok);
      if (w.ok) {
        if (lane == 0) {
          sm.unit[b] = u;
          tc::mbar_arrive(&sm.barU[b]);
        }
        pg.load(a.at.pages, sm.k[b], &a.at.k, u.kh, u.tile * CH, entry, &sm.barK[b]);
      }
      if (split > 1) {  // (in step with the groups, a unit later)
        if (n > 0) tc::cluster_wait();
        tc::cluster_arrive();
      }
    }
    if (lane == 0) {  // no copy is in flight when the CTA ends
      if (w.ok)
        for (int n = max(0, n_units - 2); n < n_units; ++n) w.on(&sm.barK[n & 1], n / 2);
      if (!w.ok)
        for (int k = 0; k < 2; ++k) tc::mbar_wait_sleep(&sm.barK[k], 0, 4000000LL);
    }
    __syncwarp();
    if (split > 1 && n_units > 0) tc::cluster_wait();
  } else if (warp == LOADS) {
    for (int n = 0; n < n_units; ++n) {
      if (lane == 0) {
        w.on(&sm.barU[n & 1], n / 2);
        const Unit u = sm.unit[n & 1];
        tc::mbar_arrive(&sm.barF[n & 1]);
        for (int j = 0; w.ok && j < u.mine; ++j, ++t) {
          if (t >= MANY_SLOTS) w.on(&sm.empty[t % MANY_SLOTS], t / MANY_SLOTS - 1);
          if (w.ok)
            load_group(sm.slot[t % MANY_SLOTS], &a.at.q, u.kh, G, u.row + (u.q0 + split * j) * TT,
                       &sm.full[t % MANY_SLOTS]);
        }
      }
      __syncwarp();
      if (split > 1) {
        if (n > 0) tc::cluster_wait();
        tc::cluster_arrive();
      }
    }
    if (lane == 0) {  // no copy is in flight when the CTA ends
      if (w.ok)
        for (int u = max(0, t - MANY_SLOTS); u < t; ++u) w.on(&sm.full[u % MANY_SLOTS], u / MANY_SLOTS);
      if (!w.ok)
        for (int k = 0; k < MANY_SLOTS; ++k) tc::mbar_wait_sleep(&sm.full[k], 0, 4000000LL);
    }
    __syncwarp();
    if (split > 1 && n_units > 0) tc::cluster_wait();
  } else if (warp >= ISSUES) {
    const uint32_t lead = tc::elect_leader();
    for (int n = 0; n < n_units; ++n) {
      const int b = n & 1;
      w.warp_on(&sm.barU[b], n / 2);
      w.ok = __all_sync(0xffffffffu, w.ok);
      const int mine = w.ok ? sm.unit[b].mine : 0;
      w.warp_on(&sm.barK[b], n / 2);
      for (int j = 0; j < mine; ++j, ++t) {
        if ((t ^ warp) & 1) continue;  // the other issuer's
        w.warp_on(&sm.full[t % MANY_SLOTS], t / MANY_SLOTS);
        if (t >= NS) w.warp_on(&sm.barE[t % NS], t / NS - 1);
        tc::fence_after();
        tc::gemm128_by<false>(lead, sm.tmem + 128 * (t % NS), smem_u32(sm.k[b]), smem_u32(sm.slot[t % MANY_SLOTS]), false);
        tc::commit_by(lead, &sm.barS[t % NS]);
        tc::commit_by(lead, &sm.empty[t % MANY_SLOTS]);
      }
      tc::commit_by(lead, &sm.barF[b]);  // (at once where the unit had no product of this warp's)
      if (split > 1) {
        if (n > 0) tc::cluster_wait();
        tc::cluster_arrive();
      }
    }
    // every commit has arrived before the CTA ends
    for (int u = max(0, t - MANY_SLOTS); u < t; ++u)
      if (((u ^ warp) & 1) == 0) w.warp_on(&sm.empty[u % MANY_SLOTS], u / MANY_SLOTS);
    for (int n = max(0, n_units - 2); n < n_units; ++n) w.warp_on(&sm.barF[n & 1], n / 2);
    if (split > 1 && n_units > 0) tc::cluster_wait();
  } else {
    const int x = warp >> 2, r = tid & 127, tok = r / G;  // column r of a query tile: its token there
    const bool row_ok = r < TT * G, adds = x == 0 && rank == 0;
    const uint32_t S = sm.tmem + 128 * x + ((uint32_t)(32 * (warp & 3)) << 16);
    const float sc = a.at.scale * LOG2E;
    int buf = 0;
    // the unit, the table's entry for the thread's key, and the first log-sum, which are asked for
    // while the unit before is summed up
    Unit u;
    int entry, j;
    float l;
    auto read = [&](int i) {  // of the CTA's i-th query tile
      const int at = (u.q0 + split * i) * TT + tok;
      l = row_ok && at < u.ql ? a.lse[((long)u.row + at) * a.at.Hq + u.kh * G + r - tok * G] : -INFINITY;
    };
    auto take = [&](int n) {
      w.warp_on(&sm.barU[n & 1], n / 2);
      w.ok = all128(1 + x, w.ok);  // (the group takes as many steps in all of its threads)
      u = sm.unit[n & 1];
      if (!w.ok) u.mine = u.kl = 0;
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&sm.barF[n & 1]);
      const int key = u.tile * CH + r;
      entry = adds && key < u.kl ? u.table[a.at.pages.page_of(key)] : -1;
      j = (x + NG - t % NG) % NG;  // the group's: every fourth one, counted over all units
      if (j < u.mine) read(j);
    };
    if (n_units > 0) take(0);
    for (int n = 0; n < n_units; ++n) {
      const int key = u.tile * CH + r, kh = u.kh, page = entry, end = u.tile * CH + CH - 1;
      float all = 0.f;  // (tile by tile: a chain over all of a long prompt's terms rounds them all)
      for (; j < u.mine; j += NG) {
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
        Columns<CH>& cols = sm.cols[x][buf];
        const bool sees = l != -INFINITY;  // (a log-sum of NaN makes the keys' weights NaN)
        const int lim = sees ? (u.q0 + split * j) * TT + tok + u.off : -1;
        cols.nl[r] = sees ? -l * LOG2E : 0.f;
        cols.lim[r] = lim;
        const int least = __reduce_min_sync(0xffffffffu, lim);
        if (lane == 0) sm.clean[x][buf][warp & 3] = least;
        // (two sets of columns in turn: whoever writes one again has met the others here since)
        asm volatile("bar.sync %0, 128;" ::"r"(1 + x) : "memory");
        if (j + NG < u.mine) read(j + NG);
        const int* clean = sm.clean[x][buf];
        buf ^= 1;
        w.warp_on(&sm.barS[x], (t + j) / NS);
        tc::fence_after();
        float v[32];
        tc::ld32(S, v);
        add32(v, cols, 0, key, end, clean[0], sc, sum);
        tc::ld32(S + 32, v);
        add32(v, cols, 32, key, end, clean[1], sc, sum);
        tc::ld32(S + 64, v);
        add32(v, cols, 64, key, end, clean[2], sc, sum);
        tc::ld32(S + 96, v);
        tc::fence_before();
        tc::mbar_arrive(&sm.barE[x]);
        add32(v, cols, 96, key, end, clean[3], sc, sum);
        all += (sum[0] + sum[1]) + (sum[2] + sum[3]);
      }
      t += u.mine;
      if (n + 1 < n_units) take(n + 1);
      // (two sets of sums in turn: whoever writes one again has met the reader here since)
      if (x > 0) sm.sums[n & 1][x - 1][r] = all;
      asm volatile("bar.sync %0, %1;" ::"n"(1 + NG), "n"(128 * NG) : "memory");
      if (x == 0) {
#pragma unroll
        for (int g = 0; g < NG - 1; ++g) all += sm.sums[n & 1][g][r];
        if (rank == 1) tc::st_cluster(&sm.other[n & 1][r], 0, all);
      }
      if (split > 1) {
        tc::cluster_arrive();
        tc::cluster_wait();
        if (adds) all += sm.other[n & 1][r];
      }
      if ((unsigned)page < (unsigned)a.at.pages.n_pages && all != 0.f)
        atomicAdd(a.weights + ((long)page * a.at.Hk + kh) * a.at.pages.page + (key - a.at.pages.page_of(key) * a.at.pages.page), all);
    }
  }
  if (!w.ok && a.at.status) atomicOr(a.at.status, 1);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (warp == 0) tc::dealloc(sm.tmem, 512);
}

// ---- few queries -------------------------------------------------------------------------
// A query tile has 64 rows here.  The key tiles of all sequences and heads, one behind
// another, are cut into equal runs, one to a CTA.
constexpr int FEW_THREADS = 192, FEW_SLOTS = 2, FEW_ROWS = WEIGH_FEW_ROWS, FEW_S = 4;
constexpr uint32_t QTILE = FEW_ROWS * HD * 2;

struct FewSmem {
  unsigned char q[2][QTILE];
  unsigned char slot[FEW_SLOTS][TILE];
  Columns<FEW_ROWS> cols;
  int clean[FEW_ROWS / 32];
  uint64_t full[FEW_SLOTS], empty[FEW_SLOTS];
  uint64_t qfull[2], qempty[2], barS[FEW_S], barE[FEW_S];
  uint32_t tmem;
};

// A CTA's run over (sequence, head, key tile), which every warp walks by itself: the
// lengths of 32 sequences lie in its lanes.
struct Run {
  const WeighArgs& a;
  int left;           // units of the run that are left, this one included
  int s0, lane_ql, lane_q0, lane_kl;
  int seq, kh, tile, tiles;
  Seq sq;

  __device__ __forceinline__ int count(int ql, int kl) const {
    const bool mine = a.rule.few == WeighRule::ALL || WeighRule::small(ql, a.at.Hq / a.at.Hk);
    return ql > 0 && mine ? (kl + CH - 1) / CH : 0;
  }
  __device__ __forceinline__ void read(int from) {
    s0 = from;
    const int s = s0 + (threadIdx.x & 31);
    lane_ql = lane_q0 = lane_kl = 0;
    if (s < a.at.n_seqs) {
      const int2 q = rows_of(a.at.cu_q, s, a.at.n_seqs, a.at.total_q);
      lane_q0 = q.x;
      lane_ql = q.y;
      lane_kl = min(max(a.at.k_len[s], 0), a.at.pages.capacity);
    }
  }
  __device__ __forceinline__ void take() {  // the numbers of sequence `seq`, which lies in the lanes
    sq.q0 = __shfl_sync(0xffffffffu, lane_q0, seq - s0);
    sq.ql = __shfl_sync(0xffffffffu, lane_ql, seq - s0);
    sq.kl = __shfl_sync(0xffffffffu, lane_kl, seq - s0);
    sq.k0 = 0;
    tiles = count(sq.ql, sq.kl);
  }
  // A lane counts for a 32nd of the sequences, one behind another, so that their lengths are asked for
  // at once.
  __device__ __forceinline__ explicit Run(const WeighArgs& args) : a(args), left(0) {
    const int lane = threadIdx.x & 31, block = (a.at.n_seqs + 31) / 32;
    int mine = 0;
    if (block == 1) {
      read(0);
      mine = count(lane_ql, lane_kl);
    } else {
#pragma unroll 4
      for (int i = 0; i < block; ++i) {
        const int s = min(lane * block + i, a.at.n_seqs - 1);
        const int ql = rows_of(a.at.cu_q, s, a.at.n_seqs, a.at.total_q).y;
        const int kl = min(max(a.at.k_len[s], 0), a.at.pages.capacity);
        if (lane * block + i < a.at.n_seqs) mine += count(ql, kl);
      }
    }
    long upto = sums(mine);
    const long total = from(upto, 31) * a.at.Hk;
    const long lo = total * blockIdx.x / gridDim.x, hi = total * (blockIdx.x + 1) / gridDim.x;
    left = (int)(hi - lo);
    if (left == 0) return;
    // the lane, or behind it the sequence of its block, in which the run begins
    int l = __ffs((int)__ballot_sync(0xffffffffu, upto * a.at.Hk > lo)) - 1;
    long before = from(upto - mine, l);  // key tiles ahead of it
    seq = l;
    if (block > 1) {
      for (int s = l * block;; s += 32) {
        read(s);
        mine = count(lane_ql, lane_kl);
        upto = before + sums(mine);
        const unsigned past = __ballot_sync(0xffffffffu, upto * a.at.Hk > lo);
        if (past) {
          l = __ffs((int)past) - 1;
          before = from(upto - mine, l);
          seq = s + l;
          break;
        }
        before = from(upto, 31);
      }
    }
    take();
    const long in = lo - before * a.at.Hk;
    kh = (int)(in / tiles);
    tile = (int)(in - (long)kh * tiles);
  }
  __device__ __forceinline__ bool last_of_head() const { return left == 1 || tile + 1 == tiles; }
  __device__ __forceinline__ void next() {
    if (--left == 0) return;
    if (++tile < tiles) return;
    tile = 0;
    if (++kh < a.at.Hk) return;
    kh = 0;
    do {  // (a later sequence has units, since some are left)
      if (++seq == s0 + 32) read(seq);
      take();
    } while (tiles == 0);
  }
};

__global__ void __launch_bounds__(FEW_THREADS, 2) k_weigh_few(const __grid_constant__ WeighArgs a) {
  extern __shared__ unsigned char raw[];
  FewSmem& sm = *reinterpret_cast<FewSmem*>(raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u));
  const int tid = threadIdx.x, lane = tid & 31, warp = tc::warp_index();
  pdl_wait();
  pdl_release();
  clear_status(a.at.status);
  const int G = a.at.Hq / a.at.Hk, TT = FEW_ROWS / G;
  Run run(a);
  if (run.left == 0) return;

  if (warp == 5 && lane == 0) {
    for (int k = 0; k < FEW_SLOTS; ++k) {
      tc::mbar_init(&sm.full[k], 1);
      tc::mbar_init(&sm.empty[k], 1);
    }
    for (int k = 0; k < 2; ++k) {
      tc::mbar_init(&sm.qfull[k], 1);
      tc::mbar_init(&sm.qempty[k], 1);
    }
    for (int k = 0; k < FEW_S; ++k) {
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

  // A query tile stays for all key tiles of a head where the sequence has one; else each key
  // tile goes through all of them.  t counts key tiles, i query tiles, u products.
  int t = 0, i = 0, u = 0;
  if (warp == 5) {
    bool fresh = true;  // the query tile of the head is not there yet
    for (; run.left > 0 && w.ok; run.next(), ++t) {
      const int nq = (run.sq.ql + TT - 1) / TT;
      const Paged<CH> pg(a.at, run.seq, run.sq.kl);
      const int entry = pg.entry(a.at.pages, run.tile * CH);
      for (int qt = 0; qt < nq && w.ok; ++qt) {
        if (nq > 1 || fresh) {
          if (i >= 2) w.on(&sm.qempty[i & 1], i / 2 - 1);
          w.ok = __all_sync(0xffffffffu, w.ok);
          if (w.ok && lane == 0) {
            tc::arrive_expect_tx(&sm.qfull[i & 1], 2u * 128u * (uint32_t)(TT * G));
            tc::tma_load_3d(sm.q[i & 1], &a.q, 0, run.kh * G, run.sq.q0 + qt * TT, &sm.qfull[i & 1]);
            tc::tma_load_3d(sm.q[i & 1] + QTILE / 2, &a.q, 64, run.kh * G, run.sq.q0 + qt * TT, &sm.qfull[i & 1]);
          }
          ++i;
        }
        if (qt == 0) {
          if (t >= FEW_SLOTS) w.on(&sm.empty[t % FEW_SLOTS], t / FEW_SLOTS - 1);
          w.ok = __all_sync(0xffffffffu, w.ok);
          if (w.ok) pg.load(a.at.pages, sm.slot[t % FEW_SLOTS], &a.at.k, run.kh, run.tile * CH, entry, &sm.full[t % FEW_SLOTS]);
        }
      }
      fresh = run.last_of_head();
    }
    if (lane == 0) {  // no copy is in flight when the CTA ends
      if (w.ok) {
        for (int k = max(0, i - 2); k < i; ++k) w.on(&sm.qfull[k & 1], k / 2);
        for (int k = max(0, t - FEW_SLOTS); k < t; ++k) w.on(&sm.full[k % FEW_SLOTS], k / FEW_SLOTS);
      }
      if (!w.ok) {
        for (int k = 0; k < 2; ++k) tc::mbar_wait_sleep(&sm.qfull[k], 0, 4000000LL);
        for (int k = 0; k < FEW_SLOTS; ++k) tc::mbar_wait_sleep(&sm.full[k], 0, 4000000LL);
      }
    }
    __syncwarp();
  } else if (warp == 4) {
    const uint32_t lead = tc::elect_leader();
    bool fresh = true;
    for (; run.left > 0; run.next(), ++t) {
      const int nq = (run.sq.ql + TT - 1) / TT;
      const bool last = run.last_of_head();
      for (int qt = 0; qt < nq; ++qt, ++u) {
        if (nq > 1 || fresh) {
          w.warp_on(&sm.qfull[i & 1], i / 2);
          ++i;
        }
        if (qt == 0) w.warp_on(&sm.full[t % FEW_SLOTS], t / FEW_SLOTS);
        if (u >= FEW_S) w.warp_on(&sm.barE[u % FEW_S], u / FEW_S - 1);
        tc::fence_after();
        const int N = (min(TT, run.sq.ql - qt * TT) * G + 15) & ~15;
        tc::gemm128xN_by<FEW_ROWS>(lead, sm.tmem + FEW_ROWS * (u % FEW_S), smem_u32(sm.slot[t % FEW_SLOTS]),
                                   smem_u32(sm.q[(i - 1) & 1]), N);
        tc::commit_by(lead, &sm.barS[u % FEW_S]);
        if (nq > 1 || last) tc::commit_by(lead, &sm.qempty[(i - 1) & 1]);
        if (qt + 1 == nq) tc::commit_by(lead, &sm.empty[t % FEW_SLOTS]);
      }
      fresh = last;
    }
    // every commit has arrived before the CTA ends
    for (int k = max(0, i - 2); k < i; ++k) w.warp_on(&sm.qempty[k & 1], k / 2);
    for (int k = max(0, t - FEW_SLOTS); k < t; ++k) w.warp_on(&sm.empty[k % FEW_SLOTS], k / FEW_SLOTS);
  } else {
    const int r = tid;
    const uint32_t lane_base = (uint32_t)(32 * warp) << 16;
    const float sc = a.at.scale * LOG2E;
    bool fresh = true;
    for (; run.left > 0; run.next(), ++t) {
      const int nq = (run.sq.ql + TT - 1) / TT;
      const Paged<CH> pg(a.at, run.seq, run.sq.kl);
      const int key = run.tile * CH + r;
      float* at = place(a, pg, run.kh, key);
      float even = 0.f, odd = 0.f;  // of the query tiles
      for (int qt = 0; qt < nq; ++qt, ++u) {
        const int rows = min(TT, run.sq.ql - qt * TT) * G;
        if (nq > 1 || fresh) {
          float nl = 0.f;
          int lim = -1;
          if (r < FEW_ROWS) column(a, run.sq, run.kh, G, TT, qt * TT, r, nl, lim);
          asm volatile("bar.sync 1, 128;" ::: "memory");  // the columns before have been read
          if (r < FEW_ROWS) {
            sm.cols.nl[r] = nl;
            sm.cols.lim[r] = lim;
            const int least = __reduce_min_sync(0xffffffffu, lim);
            if (lane == 0) sm.clean[warp] = least;
          }
          asm volatile("bar.sync 1, 128;" ::: "memory");
        }
        w.warp_on(&sm.barS[u % FEW_S], u / FEW_S);
        tc::fence_after();
        const uint32_t S = sm.tmem + FEW_ROWS * (u % FEW_S) + lane_base;
        float part[4] = {0.f, 0.f, 0.f, 0.f};
        // (columns past the product's hold what earlier ones left; no row there sees a key)
        for (int g = 0; 32 * g < rows; ++g) {
          float v[32];
          tc::ld32(S + 32 * g, v);
          add32(v, sm.cols, 32 * g, key, run.tile * CH + CH - 1, sm.clean[g], sc, part);
        }
        tc::fence_before();
        tc::mbar_arrive(&sm.barE[u % FEW_S]);
        const float tile = (part[0] + part[1]) + (part[2] + part[3]);
        if (qt & 1)
          odd += tile;
        else
          even += tile;
      }
      const float sum = even + odd;
      if (at && sum != 0.f) atomicAdd(at, sum);
      fresh = run.last_of_head();
    }
  }
  if (!w.ok && a.at.status) atomicOr(a.at.status, 1);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (warp == 0) tc::dealloc(sm.tmem, 256);
}

}  // namespace

cudaError_t launch_weigh(const WeighArgs& a, cudaStream_t s) {
  static_assert(sizeof(ManySmem) + 1024 <= 227 * 1024 && 2 * (sizeof(FewSmem) + 2048) <= 228 * 1024, "shared memory");
  cudaError_t e = cudaSuccess;
  if (a.rule.few) {
    const size_t smem = sizeof(FewSmem) + 1024;
    e = cudaFuncSetAttribute(k_weigh_few, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e == cudaSuccess) e = launch_pdl(k_weigh_few, dim3((unsigned)a.rule.few_ctas), dim3(FEW_THREADS), smem, s, a);
  }
  if (e != cudaSuccess || !a.rule.many) return e;
  const size_t smem = sizeof(ManySmem) + 1024;
  e = cudaFuncSetAttribute(k_weigh_many, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.rule.split * a.rule.ctas));
  cfg.blockDim = dim3(MANY_THREADS);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)a.rule.split;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, k_weigh_many, a);
}

}  // namespace gdn
