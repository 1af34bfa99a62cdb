// gdn_attn_paged.cu -- attention of new tokens over a cache in pages.
//
// The mathematics and the roles of the warps are those of gdn_attn_fwd.cu and
// gdn_attn_split.cu; keys are loaded page by page (gdn_attn.cuh).  What differs is who does
// what: a serving step mixes parts of prompts with single tokens over caches of any length,
// and the host knows none of the lengths.  The keys of all items are cut into equal runs, one
// to a CTA (gdn_attn_runs.cuh), which walks its run without a pause: the ring of K and V
// tiles goes on into the next item while the last one's output leaves.  A part of an item
// that is cut goes to a slot of its own, normalised and with its log-sum, in fp32, and
// k_paged_join puts the parts together in their order.
//
// k_paged_many holds two query tiles against tiles of 128 keys, or one query tile whose key
// tiles its two groups of warps take in turn; k_paged_few (for calls whose sequences are
// known to fit one query tile) holds one against tiles of 64 keys, two CTAs to an SM.
//
// P meets V rounded once to bf16, the only type that the product takes beside V's; scores, maxima, sums (of
// the p as they were), O and parts are fp32.  The rounding is as large as that of the result: o is off by
// 2.3e-3 in the 2-norm, where the exact result in bf16 is by 1.7e-3.
//
// Bounds.  Chunks of prompts: the tensor rate, 2048 tokens over 32768 keys with 16/4 heads take
// 308 us, 1.73 PFLOP/s (tensor pipe 77% busy; CTAs that each took one item 367).  Tokens: HBM,
// 32 of them over 1 to 16214 keys take 92 us for 532 MB, 5.8 TB/s (an equal number of key tiles
// of each item to a CTA: 98).  A mixed step (512 + 300 + 129 tokens and 20 single ones, 16/2
// heads): 55 us (82 before), of which some 20 are the start, the plan and the join, and single
// tokens fill 8 of a tile's 128 rows.  One token over 777 keys: 16.5 us, latencies alone.
//
#include <math.h>

#include "gdn_attn_runs.cuh"

namespace gdn {

namespace {

using namespace attn;

constexpr float RAISE = 8.f;  // base-2 headroom before the running maximum is raised
constexpr int BATCH = 16;     // items that are planned at a time

// The N threads that have a role: they meet around a new plan, twice.  (Not at the block's barrier, where
// warps without a role may be already, which go straight to the kernel's end.)
template <int N>
__device__ __forceinline__ void roles_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(N) : "memory");
}

// two warps that have the same rows
__device__ __forceinline__ void pair_sync(int id) { asm volatile("bar.sync %0, 64;" ::"r"(id) : "memory"); }

// Output of 32 columns of a row, or of a part of it.
__device__ __forceinline__ void leave(const Item& it, bf16* o, float* part, float (&y)[32], bool none, float inv) {
  if (none) {
#pragma unroll
    for (int j = 0; j < 32; ++j) y[j] = 0.f;
  }
  if (it.whole) {
    store32(o, y, inv);
  } else if (!none) {  // (the join reads no part whose lse is minus infinity)
#pragma unroll
    for (int j = 0; j < 32; j += 4)  // (16 bytes: a workspace need not lie at a multiple of more)
      *reinterpret_cast<float4*>(part + j) = make_float4(inv * y[j], inv * y[j + 1], inv * y[j + 2], inv * y[j + 3]);
  }
}

// 32 columns of a warp's 32 rows, through shared memory, so that whole lines leave: a store of
// every lane's own row touches 32 lines at a time, and a part of 256 rows took some 8 us.
// `rows`: those that are written; `part`: the warp's first row, `o`: the tile's first, `at`: elements
// from there to the row that is the lane's in step k (its four lanes have 64 bytes).
struct alignas(16) Stage {
  float4 v[32][8];
};
__device__ __forceinline__ void leave_part(Stage& st, float* part, const float (&y)[32], float inv, uint32_t rows) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int c = 0; c < 8; ++c)
    st.v[lane][c ^ (lane & 7)] = make_float4(inv * y[4 * c], inv * y[4 * c + 1], inv * y[4 * c + 2], inv * y[4 * c + 3]);
  __syncwarp();
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int r = 4 * k + (lane >> 3), c = lane & 7;
    if (rows >> r & 1u) *reinterpret_cast<float4*>(part + (long)r * HD + 4 * c) = st.v[r][c ^ (r & 7)];
  }
  __syncwarp();
}
__device__ __forceinline__ void leave_whole(Stage& st, bf16* o, const int (&at)[4], const float (&y)[32], float inv,
                                            uint32_t rows) {
  const int lane = threadIdx.x & 31;
  uint4(&s)[32][4] = *reinterpret_cast<uint4(*)[32][4]>(&st);
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const float* v = y + 8 * c;
    s[lane][c ^ (lane >> 1 & 3)] = make_uint4(pack_bf16(inv * v[0], inv * v[1]), pack_bf16(inv * v[2], inv * v[3]),
                                              pack_bf16(inv * v[4], inv * v[5]), pack_bf16(inv * v[6], inv * v[7]));
  }
  __syncwarp();
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int r = 8 * k + (lane >> 2), c = lane & 3;
    if (rows >> r & 1u) *reinterpret_cast<uint4*>(o + at[k] + 8 * c) = s[r][c ^ (r >> 1 & 3)];
  }
  __syncwarp();
}

// ---- sequences of more than one query tile ---------------------------------------------------
constexpr int NSLOT = 4;
constexpr int MANY_THREADS = 384, MANY_ROLES = 320;  // (two groups of softmax, one warp that issues, one that plans and loads)
// Keys that an item's start and end take the time of, and a run's width, at least.  Measured in us
// for a mixed step, 2048 tokens over 32768 keys, 40 over 16384: 55, 308, 28; without extra and 128
// at least 90, 309, 29; 1024 and 1536 61, 315, 35.
constexpr int MANY_EXTRA = 256, MANY_RUN = 512;
constexpr int REGS_LAUNCH = 168, REGS_SOFTMAX = 208, REGS_ISSUE = 88;  // (as in gdn_attn_fwd.cu)
static_assert(2 * REGS_SOFTMAX + REGS_ISSUE <= 3 * REGS_LAUNCH, "the groups' registers come from the block's");

struct ManySmem {
  unsigned char q[2][TILE];
  unsigned char slot[NSLOT][TILE];
  Stage stage[8];
  RunsSmem<BATCH> runs;
  uint64_t full[NSLOT], empty[NSLOT];
  // Q there and free again, S, the halves of P, O there and free again
  uint64_t barQ[2], barQF[2], barS[2], barP[2][2], barO[2], barF[2];
  uint32_t tmem;
};

__global__ void __launch_bounds__(MANY_THREADS, 1) k_paged_many(const __grid_constant__ PagedArgs pa) {
  extern __shared__ unsigned char raw[];
  const AttnArgs& a = pa.at;
  ManySmem& sm = *reinterpret_cast<ManySmem*>(raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u));
  const int tid = threadIdx.x, lane = tid & 31, warp = tc::warp_index();
  pdl_wait();
  pdl_release();
  clear_status(a.status);
  const int G = a.Hq / a.Hk, TT = CH / G;  // tokens to a tile
  Planner<MANY_EXTRA> plan(a, 2 * TT);
  // key tiles of the two groups in an item's part; returns those that are loaded.  A single
  // query tile is held by both groups, each with every second key tile.
  auto tiles = [&](const Item& it, int (&n)[2]) {
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const int keys = w * TT < it.toks ? min(it.kl, it.lim + min((w + 1) * TT, it.toks)) : 0;
      n[w] = max(0, min((max(keys, 0) + CH - 1) / CH, it.ke) - it.kb);
    }
    const int all = max(n[0], n[1]);
    if (it.toks <= TT) {
      n[1] = all / 2;
      n[0] = all - n[1];
    }
    return all;
  };

  if (warp == 9 && lane == 0) {
    for (int k = 0; k < NSLOT; ++k) {
      tc::mbar_init(&sm.full[k], 1);
      tc::mbar_init(&sm.empty[k], 1);
    }
    for (int w = 0; w < 2; ++w) {
      tc::mbar_init(&sm.barQ[w], 1);
      tc::mbar_init(&sm.barQF[w], 1);
      tc::mbar_init(&sm.barS[w], 1);
      tc::mbar_init(&sm.barO[w], 1);
      tc::mbar_init(&sm.barP[w][0], 128);
      tc::mbar_init(&sm.barP[w][1], 128);
      tc::mbar_init(&sm.barF[w], 128);
    }
    tc::mbar_fence_init();
  }
  if (warp == 9) {
    if (lane == 0) pa.joins[blockIdx.x].last = -1;
    __syncwarp();
    plan.start((int)blockIdx.x, (int)gridDim.x, MANY_RUN);
    plan.fill(sm.runs, pa.joins, (int)blockIdx.x);
  }
  if (warp == 0) tc::alloc(&sm.tmem, 512);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tS = sm.tmem, tO = sm.tmem + 256;
  tc::Wait w;

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_ISSUE));
    if (warp == 9) {
      int t = 0, qc[2] = {0, 0};  // ring tiles, query tiles so far
      for (;;) {
        for (int e = 0; e < sm.runs.count && w.ok; ++e) {
          const Item& it = sm.runs.item[e];
          int n[2];
          const int nmax = tiles(it, n), kb = it.kb, kh = it.kh, row = it.row;
          const bool dual = it.toks <= TT;
          if (nmax == 0) continue;
          const Paged<CH> pg(a, it.seq, it.kl);
          int entry = pg.entry(a.pages, kb * CH);
          for (int i = 0; i < nmax && w.ok; ++i) {
            const int key0 = (kb + i) * CH, now = entry;
            if (i + 1 < nmax) entry = pg.entry(a.pages, key0 + CH);
#pragma unroll
            for (int v = 0; v < 2; ++v, ++t) {
              if (t >= NSLOT) w.on(&sm.empty[t % NSLOT], t / NSLOT - 1);
              w.ok = __all_sync(0xffffffffu, w.ok);
              if (w.ok) pg.load(a.pages, sm.slot[t % NSLOT], v ? &a.v : &a.k, kh, key0, now, &sm.full[t % NSLOT]);
            }
            if (i > 0) continue;
            // (behind the first key tile, which needs no free query buffer)
#pragma unroll
            for (int x = 0; x < 2; ++x)
              if (n[x] > 0 && !(dual && x)) {
                if (qc[x] > 0) w.on(&sm.barQF[x], qc[x] - 1);
                w.ok = __all_sync(0xffffffffu, w.ok);
                if (w.ok && lane == 0)
                  load_group(sm.q[x], &a.q, kh, G, row + x * TT, &sm.barQ[x]);
                ++qc[x];
              }
          }
        }
        if (!sm.runs.more) break;
        roles_sync<MANY_ROLES>();  // the items have been read
        plan.fill(sm.runs, pa.joins, (int)blockIdx.x);
        roles_sync<MANY_ROLES>();
      }
      if (lane == 0) {  // no copy is in flight when the CTA ends
        if (w.ok) {
          for (int x = 0; x < 2; ++x)
            if (qc[x] > 0) w.on(&sm.barQ[x], qc[x] - 1);
          for (int u = max(0, t - NSLOT); u < t; ++u) w.on(&sm.full[u % NSLOT], u / NSLOT);
        }
        if (!w.ok) {
          for (int x = 0; x < 2; ++x) tc::mbar_wait_sleep(&sm.barQ[x], 0, 4000000LL);
          for (int k = 0; k < NSLOT; ++k) tc::mbar_wait_sleep(&sm.full[k], 0, 4000000LL);
        }
      }
      __syncwarp();
    } else if (warp == 8) {
      const uint32_t lead = tc::elect_leader();
      // ring tiles, query tiles, a group's items and key tiles so far
      int t0 = 0, qc[2] = {0, 0}, oc[2] = {0, 0}, sc[2] = {0, 0};
      for (;;) {
        for (int e = 0; e < sm.runs.count; ++e) {
          const Item& it = sm.runs.item[e];
          int n[2];
          const int nmax = tiles(it, n);
          const bool dual = it.toks <= TT;
          if (nmax == 0) continue;
          auto slot = [&](int t) { return smem_u32(sm.slot[(t0 + t) % NSLOT]); };
          auto arrived = [&](int t) { w.warp_on(&sm.full[(t0 + t) % NSLOT], (t0 + t) / NSLOT); };
          auto release = [&](int t) { tc::commit_by(lead, &sm.empty[(t0 + t) % NSLOT]); };
          // S of group x = Q K^T of key tile i; `last`: of this query tile
          auto scores = [&](int x, int q, int i, bool last) {
            tc::gemm128_by<false>(lead, tS + 128 * x, smem_u32(sm.q[q]), slot(2 * i), false);
            tc::commit_by(lead, &sm.barS[x]);
            if (last) tc::commit_by(lead, &sm.barQF[q]);
          };
          // O of group x += P V of key tile i, the group's j-th; P arrives by halves
          auto values = [&](int x, int i, int j) {
            if (j == 0 && oc[x] > 0) w.warp_on(&sm.barF[x], oc[x] - 1);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              w.warp_on(&sm.barP[x][h], sc[x] + j);
              tc::fence_after();
              tc::gemm_ts64_by(lead, tO + 128 * x, tS + 128 * x + 32 * h, slot(2 * i + 1) + 8192 * h, j > 0 || h > 0);
            }
            if (j + 1 == n[x]) tc::commit_by(lead, &sm.barO[x]);
          };
          arrived(0);
          if (n[0] > 0) w.warp_on(&sm.barQ[0], qc[0]);
          if (dual) {
            scores(0, 0, 0, nmax == 1);
            release(0);
            if (nmax > 1) {
              arrived(2);
              scores(1, 0, 1, nmax == 2);
              release(2);
            }
            for (int i = 0; i < nmax; ++i) {
              arrived(2 * i + 1);
              values(i & 1, i, i >> 1);
              release(2 * i + 1);
              if (i + 2 < nmax) {
                arrived(2 * i + 4);
                scores(i & 1, 0, i + 2, i + 3 == nmax);
                release(2 * i + 4);
              }
            }
            ++qc[0];
          } else {
            if (n[0] > 0) scores(0, 0, 0, n[0] == 1);
            if (n[1] > 0) {
              w.warp_on(&sm.barQ[1], qc[1]);
              scores(1, 1, 0, n[1] == 1);
            }
            release(0);
            for (int i = 0; i < nmax; ++i) {
              arrived(2 * i + 1);
              if (i + 1 < nmax) arrived(2 * i + 2);
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                if (i < n[x]) values(x, i, i);
                if (x == 1) release(2 * i + 1);
                if (i + 1 < n[x]) scores(x, x, i + 1, i + 2 == n[x]);
              }
              if (i + 1 < nmax) release(2 * i + 2);
            }
            qc[0] += n[0] > 0;
            qc[1] += n[1] > 0;
          }
          t0 += 2 * nmax;
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            oc[x] += n[x] > 0;
            sc[x] += n[x];
          }
        }
        if (!sm.runs.more) break;
        roles_sync<MANY_ROLES>();
        roles_sync<MANY_ROLES>();
      }
      // every commit has arrived before the CTA ends
      for (int u = max(0, t0 - NSLOT); u < t0; ++u) w.warp_on(&sm.empty[u % NSLOT], u / NSLOT);
#pragma unroll
      for (int x = 0; x < 2; ++x)
        if (qc[x] > 0) w.warp_on(&sm.barQF[x], qc[x] - 1);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS_SOFTMAX));
    const int x = warp >> 2, r = 32 * (warp & 3) + lane;
    const uint32_t lane_base = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t S = tS + 128 * x + lane_base, O = tO + 128 * x + lane_base;
    const float sc = a.scale * LOG2E;
    int t0 = 0, s0 = 0, items = 0;  // ring tiles, the group's key tiles and items so far
    for (;;) {
      for (int e = 0; e < sm.runs.count; ++e) {
        const Item& it = sm.runs.item[e];
        int n[2];
        const int nmax = tiles(it, n);
        const bool dual = it.toks <= TT;
        const int mine = n[x], kb = it.kb, kl = it.kl, step = dual ? 2 : 1, at0 = dual ? x : 0;  // the group's key tiles
        const int tok = (dual ? 0 : x * TT) + r / G;
        const bool valid = r < TT * G && tok < it.toks;
        const int lim = valid ? it.lim + tok : -1;  // the last key that the row sees
        const bool any = __any_sync(0xffffffffu, valid);
        const Paged<CH> pg(a, it.seq, kl);
        float m = -INFINITY, l = 0.f;
        int asked = 0;
        if (mine > 0) asked = pg.ask(a.pages, (kb + at0) * CH);
        for (int i = 0; i < mine; ++i) {
          const int tile = at0 + step * i, key0 = (kb + tile) * CH;
          const uint32_t absent = pg.absent(a.pages, asked);  // 16 keys to a bit
          asked = pg.ask(a.pages, key0 + step * CH);
          w.warp_on(&sm.barS[x], s0 + i);
          if (key0 + CH > kl) {  // rows past the keys: whatever they hold, they count as zero
            // (behind S, which says that the issuer is at this item: a group whose part of the last one
            // was short may be whole rounds of the ring ahead of it, where a phase's parity says nothing)
            const int t = t0 + 2 * tile + 1;
            w.warp_on(&sm.full[t % NSLOT], t / NSLOT);
            zero_rows(sm.slot[t % NSLOT], kl - key0, tid & 127, 128);
            tc::fence_proxy_async();
          }
          tc::fence_after();
          if (any) {
            float v[128];
            tc::ld64(S, *reinterpret_cast<float(*)[64]>(v));
            tc::ld64(S + 64, *reinterpret_cast<float(*)[64]>(v + 64));
            if (key0 + CH - 1 > lim) {
#pragma unroll
              for (int j = 0; j < 128; ++j) v[j] = key0 + j <= lim ? v[j] : -INFINITY;
            }
            if (absent) {
#pragma unroll
              for (int j = 0; j < 128; ++j) v[j] = absent >> (j / 16) & 1u ? -INFINITY : v[j];
            }
            float mt[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
            for (int j = 4; j < 124; j += 8) {
#pragma unroll
              for (int c = 0; c < 4; ++c) mt[c] = tc::max3(mt[c], v[j + c], v[j + 4 + c]);
            }
            const float mn =
                fmaxf(tc::max3(mt[0], mt[1], fmaxf(v[124], v[125])), tc::max3(mt[2], mt[3], fmaxf(v[126], v[127])));
            // raise the maximum (a first one counts); O is idle: this S was issued after the last P V
            if (__any_sync(0xffffffffu, mn > m && (mn - m) * sc > RAISE)) {
              const float to = fmaxf(m, mn);
              const float f = m == to ? 1.f : ex2((m - to) * sc);  // 0 for a first maximum
              m = to;
              l *= f;
              if (i > 0) {
#pragma unroll 1
                for (int g = 0; g < 4; ++g) {
                  float y[32];
                  tc::ld32(O + 32 * g, y);
#pragma unroll
                  for (int j = 0; j < 32; ++j) y[j] *= f;
                  tc::st32(O + 32 * g, y);
                }
                tc::wait_st();
              }
            }
            const float ms = m == -INFINITY ? 0.f : -m * sc;
            float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
              for (int g = 0; g < 2; ++g) {
                float(&p)[32] = *reinterpret_cast<float(*)[32]>(v + 64 * h + 32 * g);
#pragma unroll
                for (int j = 0; j < 32; j += 2) {
                  tc::fma2(p[j], p[j + 1], sc, sc, ms);
                  p[j] = ex2(p[j]);
                  p[j + 1] = ex2(p[j + 1]);
                  tc::add2(sum[j & 2], sum[(j & 2) + 1], p[j], p[j + 1]);
                }
                tc::st16_bf16(S + 32 * h + 16 * g, p);
              }
              tc::wait_st();
              tc::fence_before();
              tc::mbar_arrive(&sm.barP[x][h]);
            }
            l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
          } else {
            tc::fence_before();
            tc::mbar_arrive(&sm.barP[x][0]);
            tc::mbar_arrive(&sm.barP[x][1]);
          }
        }
        t0 += 2 * nmax;
        s0 += mine;
        if (mine > 0) {
          w.warp_on(&sm.barO[x], items);
          tc::fence_after();
          ++items;
        }
        const int w4 = warp & 3;
        float f = 1.f;  // what the group's own O counts for
        if (dual) {
          // the two groups' maxima and sums; group 1's part of O goes through its stage, 32 columns at a
          // time, to the warp of group 0 that has the same rows
          *reinterpret_cast<float2*>(&sm.stage[warp].v[lane][0]) = make_float2(m, l);
          pair_sync(3 + w4);
          const float2 other = *reinterpret_cast<const float2*>(&sm.stage[warp ^ 4].v[lane][0]);
          pair_sync(3 + w4);
          const float top = fmaxf(m, other.x);
          f = m == top ? 1.f : ex2((m - top) * sc);
          l = f * l + (other.x == top ? 1.f : ex2((other.x - top) * sc)) * other.y;  // (0 and 0: neither sees a key)
          m = top;
        }
        if (any) {
          // (a sum of zero: the row sees no key; one of NaN is neither greater nor equal, and goes on)
          const bool none = nmax == 0 || l == 0.f;
          const float inv = none ? 0.f : 1.f / l;
          const float lse = none ? -INFINITY : m * a.scale + logf(l);
          // (the join reads no part whose lse is minus infinity)
          const uint32_t rows = __ballot_sync(0xffffffffu, valid && (it.whole || !none));
          const long first = ((long)it.row + (dual ? 0 : x * TT)) * a.Hq + it.kh * G;  // row of the tile's first
          const long part = (long)it.slot * 256 + (dual ? 0 : 128 * x) + 32 * w4;
          int at[4];  // of the rows that are this lane's in the output
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int rr = 32 * w4 + 8 * k + (lane >> 2), t = rr / G;
            at[k] = (t * a.Hq + rr - t * G) * HD;
          }
#pragma unroll 1
          for (int g = 0; g < 4; ++g) {
            float y[32];
            if (mine > 0) tc::ld32(O + 32 * g, y);
            if (none || mine == 0) {
#pragma unroll
              for (int j = 0; j < 32; ++j) y[j] = 0.f;
            }
            if (dual) {
#pragma unroll
              for (int j = 0; j < 32; ++j) y[j] *= f;
              Stage& st = sm.stage[4 + w4];
              if (x == 1) {
#pragma unroll
                for (int c = 0; c < 8; ++c)
                  st.v[lane][c ^ (lane & 7)] = make_float4(y[4 * c], y[4 * c + 1], y[4 * c + 2], y[4 * c + 3]);
              }
              pair_sync(3 + w4);
              if (x == 0) {
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                  const float4 o = st.v[lane][c ^ (lane & 7)];
                  y[4 * c] += o.x, y[4 * c + 1] += o.y, y[4 * c + 2] += o.z, y[4 * c + 3] += o.w;
                }
              }
              pair_sync(3 + w4);
              if (x == 1) continue;
            }
            if (it.whole)
              leave_whole(sm.stage[warp], a.o + first * HD + 32 * g, at, y, inv, rows);
            else
              leave_part(sm.stage[warp], a.part + part * HD + 32 * g, y, inv, rows);
          }
          if (valid && !(dual && x)) {
            if (it.whole) {
              if (a.lse) a.lse[first + r / G * a.Hq + r % G] = lse;
            } else {
              a.part_lse[part + lane] = lse;
            }
          }
        }
        if (mine > 0) {
          tc::fence_before();
          tc::mbar_arrive(&sm.barF[x]);
        }
      }
      if (!sm.runs.more) break;
      roles_sync<MANY_ROLES>();
      roles_sync<MANY_ROLES>();
    }
  }
  if (!w.ok && a.status) atomicOr(a.status, 1);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (warp == 0) tc::dealloc(sm.tmem, 512);
}

// ---- sequences of one query tile ---------------------------------------------------------------
constexpr int KEYS = 64, FEW_SLOTS = 4;
// As above: one token over 777 keys, 32 over 1 to 16214, in us: 16.5, 94; without extra and 128 at
// least 15.6, 102; 128 and 1024 29, 94; 512 and 1024 23, 95.
constexpr int FEW_EXTRA = 128, FEW_RUN = 256;
constexpr int FEW_THREADS = 192;  // four warps of softmax, one that issues, one that plans and loads

struct FewSmem {
  unsigned char q[TILE];
  unsigned char slot[FEW_SLOTS][KEYS * HD * 2];
  RunsSmem<BATCH> runs;
  uint64_t full[FEW_SLOTS], empty[FEW_SLOTS];
  uint64_t barQ, barQF, barS, barP, barO, barF;
  uint32_t tmem;
};

__global__ void __launch_bounds__(FEW_THREADS, 2) k_paged_few(const __grid_constant__ PagedArgs pa) {
  extern __shared__ unsigned char raw[];
  const AttnArgs& a = pa.at;
  FewSmem& sm = *reinterpret_cast<FewSmem*>(raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u));
  const int tid = threadIdx.x, lane = tid & 31, warp = tc::warp_index();
  pdl_wait();
  pdl_release();
  clear_status(a.status);
  const int G = a.Hq / a.Hk, TT = CH / G;  // tokens to a tile
  Planner<FEW_EXTRA> plan(a, TT);
  // key tiles of an item's part
  auto tiles = [&](const Item& it) {
    const int keys = min(it.kl, it.lim + it.toks);
    return max(0, min((max(keys, 0) + KEYS - 1) / KEYS, it.ke * (CH / KEYS)) - it.kb * (CH / KEYS));
  };
  if (warp == 5) {
    if (lane == 0) {
      for (int k = 0; k < FEW_SLOTS; ++k) {
        tc::mbar_init(&sm.full[k], 1);
        tc::mbar_init(&sm.empty[k], 1);
      }
      tc::mbar_init(&sm.barQ, 1);
      tc::mbar_init(&sm.barQF, 1);
      tc::mbar_init(&sm.barS, 1);
      tc::mbar_init(&sm.barO, 1);
      tc::mbar_init(&sm.barP, 128);
      tc::mbar_init(&sm.barF, 128);
      tc::mbar_fence_init();
      pa.joins[blockIdx.x].last = -1;
    }
    __syncwarp();
    plan.start((int)blockIdx.x, (int)gridDim.x, FEW_RUN);
    plan.fill(sm.runs, pa.joins, (int)blockIdx.x);
  }
  if (warp == 0) tc::alloc(&sm.tmem, 256);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tS = sm.tmem, tO = sm.tmem + 128;
  tc::Wait w;

  if (warp == 5) {
    int t = 0, qc = 0;  // ring tiles, query tiles so far
    for (;;) {
      for (int e = 0; e < sm.runs.count && w.ok; ++e) {
        const Item& it = sm.runs.item[e];
        const int n = tiles(it), key_b = it.kb * CH, kh = it.kh, row = it.row;
        if (n == 0) continue;
        const Paged<KEYS> pg(a, it.seq, it.kl);
        int entry = pg.entry(a.pages, key_b);
        for (int i = 0; i < n && w.ok; ++i) {
          const int key0 = key_b + i * KEYS, now = entry;
          if (i + 1 < n) entry = pg.entry(a.pages, key0 + KEYS);
#pragma unroll
          for (int v = 0; v < 2; ++v, ++t) {
            if (t >= FEW_SLOTS) w.on(&sm.empty[t % FEW_SLOTS], t / FEW_SLOTS - 1);
            w.ok = __all_sync(0xffffffffu, w.ok);
            if (w.ok) pg.load(a.pages, sm.slot[t % FEW_SLOTS], v ? &a.v : &a.k, kh, key0, now, &sm.full[t % FEW_SLOTS]);
          }
          if (i > 0) continue;
          // (behind the first key tile, which needs no free query buffer)
          if (qc > 0) w.on(&sm.barQF, qc - 1);
          w.ok = __all_sync(0xffffffffu, w.ok);
          if (w.ok && lane == 0) load_group(sm.q, &a.q, kh, G, row, &sm.barQ);
          ++qc;
        }
      }
      if (!sm.runs.more) break;
      roles_sync<FEW_THREADS>();  // the items have been read
      plan.fill(sm.runs, pa.joins, (int)blockIdx.x);
      roles_sync<FEW_THREADS>();
    }
    if (lane == 0) {  // no copy is in flight when the CTA ends
      if (w.ok) {
        if (qc > 0) w.on(&sm.barQ, qc - 1);
        for (int u = max(0, t - FEW_SLOTS); u < t; ++u) w.on(&sm.full[u % FEW_SLOTS], u / FEW_SLOTS);
      }
      if (!w.ok) {
        tc::mbar_wait_sleep(&sm.barQ, 0, 4000000LL);
        for (int k = 0; k < FEW_SLOTS; ++k) tc::mbar_wait_sleep(&sm.full[k], 0, 4000000LL);
      }
    }
    __syncwarp();
  } else if (warp == 4) {
    const uint32_t lead = tc::elect_leader();
    int t0 = 0, qc = 0, sc = 0;  // ring tiles, items, key tiles so far
    for (;;) {
      for (int e = 0; e < sm.runs.count; ++e) {
        const int n = tiles(sm.runs.item[e]);
        if (n == 0) continue;
        auto slot = [&](int t) { return smem_u32(sm.slot[(t0 + t) % FEW_SLOTS]); };
        auto arrived = [&](int t) { w.warp_on(&sm.full[(t0 + t) % FEW_SLOTS], (t0 + t) / FEW_SLOTS); };
        auto release = [&](int t) { tc::commit_by(lead, &sm.empty[(t0 + t) % FEW_SLOTS]); };
        auto scores = [&](int i) {
          arrived(2 * i);
          tc::gemm128x64_by(lead, tS, smem_u32(sm.q), slot(2 * i));
          tc::commit_by(lead, &sm.barS);
          release(2 * i);
          if (i + 1 == n) tc::commit_by(lead, &sm.barQF);
        };
        w.warp_on(&sm.barQ, qc);
        scores(0);
        for (int i = 0; i < n; ++i) {
          arrived(2 * i + 1);
          if (i == 0 && qc > 0) w.warp_on(&sm.barF, qc - 1);
          w.warp_on(&sm.barP, sc + i);
          tc::fence_after();
          tc::gemm_ts64_by<KEYS>(lead, tO, tS, slot(2 * i + 1), i > 0);
          release(2 * i + 1);
          if (i + 1 < n) scores(i + 1);
        }
        tc::commit_by(lead, &sm.barO);
        t0 += 2 * n;
        sc += n;
        ++qc;
      }
      if (!sm.runs.more) break;
      roles_sync<FEW_THREADS>();
      roles_sync<FEW_THREADS>();
    }
    // every commit has arrived before the CTA ends
    for (int u = max(0, t0 - FEW_SLOTS); u < t0; ++u) w.warp_on(&sm.empty[u % FEW_SLOTS], u / FEW_SLOTS);
    if (qc > 0) w.warp_on(&sm.barQF, qc - 1);
  } else {
    const int r = 32 * warp + lane;
    const uint32_t lane_base = (uint32_t)(32 * warp) << 16;
    const uint32_t S = tS + lane_base, O = tO + lane_base;
    const float sc = a.scale * LOG2E;
    int t0 = 0, s0 = 0, items = 0;  // ring tiles, key tiles, items so far
    for (;;) {
      for (int e = 0; e < sm.runs.count; ++e) {
        const Item& it = sm.runs.item[e];
        const int n = tiles(it), key_b = it.kb * CH, kl = it.kl;
        const bool valid = r < TT * G && r / G < it.toks;
        const int lim = valid ? it.lim + r / G : -1;  // the last key that the row sees
        const bool any = __any_sync(0xffffffffu, valid);
        const Paged<KEYS> pg(a, it.seq, kl);
        float m = -INFINITY, l = 0.f;
        int asked = 0;
        if (n > 0) asked = pg.ask(a.pages, key_b);
        for (int i = 0; i < n; ++i) {
          const int key0 = key_b + i * KEYS;
          const uint32_t absent = pg.absent(a.pages, asked);  // 16 keys to a bit
          asked = pg.ask(a.pages, key0 + KEYS);
          if (key0 + KEYS > kl) {  // rows past the keys: whatever they hold, they count as zero
            const int t = t0 + 2 * i + 1;
            w.warp_on(&sm.full[t % FEW_SLOTS], t / FEW_SLOTS);
            for (int c = (kl - key0) * 16 + tid; c < KEYS * 16; c += 128)
              *reinterpret_cast<uint4*>(sm.slot[t % FEW_SLOTS] + tc::sw128_chunk(c >> 4, c & 15, KEYS)) =
                  make_uint4(0u, 0u, 0u, 0u);
            tc::fence_proxy_async();
          }
          w.warp_on(&sm.barS, s0 + i);
          tc::fence_after();
          if (any) {
            float v[64];
            tc::ld64(S, v);
            if (key0 + KEYS - 1 > lim) {
#pragma unroll
              for (int j = 0; j < 64; ++j) v[j] = key0 + j <= lim ? v[j] : -INFINITY;
            }
            if (absent) {
#pragma unroll
              for (int j = 0; j < 64; ++j) v[j] = absent >> (j / 16) & 1u ? -INFINITY : v[j];
            }
            float mt[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
            for (int j = 4; j < 60; j += 8) {
#pragma unroll
              for (int c = 0; c < 4; ++c) mt[c] = tc::max3(mt[c], v[j + c], v[j + 4 + c]);
            }
            const float mn = fmaxf(tc::max3(mt[0], mt[1], fmaxf(v[60], v[61])), tc::max3(mt[2], mt[3], fmaxf(v[62], v[63])));
            // raise the maximum (a first one counts); O is idle: this S was issued after the last P V
            if (__any_sync(0xffffffffu, mn > m && (mn - m) * sc > RAISE)) {
              const float to = fmaxf(m, mn);
              const float f = m == to ? 1.f : ex2((m - to) * sc);  // 0 for a first maximum
              m = to;
              l *= f;
              if (i > 0) {
#pragma unroll 1
                for (int g = 0; g < 4; ++g) {
                  float y[32];
                  tc::ld32(O + 32 * g, y);
#pragma unroll
                  for (int j = 0; j < 32; ++j) y[j] *= f;
                  tc::st32(O + 32 * g, y);
                }
              }
            }
            const float ms = m == -INFINITY ? 0.f : -m * sc;
            float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int g = 0; g < 2; ++g) {
              float(&p)[32] = *reinterpret_cast<float(*)[32]>(v + 32 * g);
#pragma unroll
              for (int j = 0; j < 32; j += 2) {
                tc::fma2(p[j], p[j + 1], sc, sc, ms);
                p[j] = ex2(p[j]);
                p[j + 1] = ex2(p[j + 1]);
                tc::add2(sum[j & 2], sum[(j & 2) + 1], p[j], p[j + 1]);
              }
              tc::st16_bf16(S + 16 * g, p);
            }
            tc::wait_st();
            l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
          }
          tc::fence_before();
          tc::mbar_arrive(&sm.barP);
        }
        t0 += 2 * n;
        s0 += n;
        if (n > 0) {
          w.warp_on(&sm.barO, items);
          tc::fence_after();
          ++items;
        }
        if (any) {
          const long row = ((long)it.row + r / G) * a.Hq + it.kh * G + r % G, at = (long)it.slot * CH + r;
          // (a sum of zero: the row sees no key; one of NaN is neither greater nor equal, and goes on)
          const float inv = l != 0.f ? 1.f / l : 0.f;
          const float lse = l != 0.f ? m * a.scale + logf(l) : -INFINITY;
#pragma unroll 1
          for (int g = 0; g < 4; ++g) {
            float y[32];
            if (n > 0) tc::ld32(O + 32 * g, y);
            if (valid) leave(it, a.o + row * HD + 32 * g, a.part + at * HD + 32 * g, y, n == 0 || l == 0.f, inv);
            __syncwarp();
          }
          if (valid && !it.whole) a.part_lse[at] = lse;
          if (valid && it.whole && a.lse) a.lse[row] = lse;
        }
        if (n > 0) {
          tc::fence_before();
          tc::mbar_arrive(&sm.barF);
        }
      }
      if (!sm.runs.more) break;
      roles_sync<FEW_THREADS>();
      roles_sync<FEW_THREADS>();
    }
  }
  if (!w.ok && a.status) atomicOr(a.status, 1);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (warp == 0) tc::dealloc(sm.tmem, 256);
}

// ---- the items that were cut ------------------------------------------------------------------
// o = sum_s e^{lse_s - lse} o_s over the parts, in a fixed order.  Blocks (c, y): 32 / P rows of
// the item that begins in run c and is cut, 8 P lanes to a row: eight have 16 columns each of
// every P-th part.  A part of NaN makes the row NaN, as it would be in one piece.  Bound by the
// latency of its loads: 9 us for 32 tokens' parts, 14 for the 36 MB of a chunk's.
template <int P>
__global__ void __launch_bounds__(256) k_paged_join(const __grid_constant__ PagedArgs pa) {
  pdl_wait();
  pdl_release();
  const AttnArgs& a = pa.at;
  const int cta = blockIdx.x, rows = pa.few ? CH : 2 * CH;
  const Join j = pa.joins[cta];
  if (j.last < 0) return;
  const int l = threadIdx.x & 7, g = (threadIdx.x >> 3) & (P - 1), G = a.Hq / a.Hk, TT = CH / G, n = j.last - cta + 1;
  const int rr = (blockIdx.y * 256 + threadIdx.x) / (8 * P), r = rr & (CH - 1), tok = (rr / CH) * TT + r / G;
  if (r >= TT * G || tok >= j.toks) return;  // (the lanes of a row together)
  const unsigned mask = P == 4 ? 0xffffffffu : 0xffu << (threadIdx.x & 24);
  // part s: the last slot of the run in which the item begins, then the first ones of the others
  auto at = [&](int s) { return (long)(s == 0 ? 2 * cta + 1 : 2 * (cta + s)) * rows + rr; };
  float top = -INFINITY;
  bool nan = false;  // (which fmaxf passes over)
  for (int s = 8 * g + l; s < n; s += 8 * P) {
    const float x = a.part_lse[at(s)];
    nan |= isnan(x);
    top = fmaxf(top, x);
  }
#pragma unroll
  for (int o = 4 * P; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(mask, top, o));
  if (__any_sync(mask, nan)) top = NAN;
  float total = 0.f, y[16];
#pragma unroll
  for (int k = 0; k < 16; ++k) y[k] = 0.f;
  if (top != -INFINITY) {
    for (int s0 = g; s0 < n; s0 += 2 * P) {  // two parts at a time
      float f[2];
      float4 v[2][4];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int s = s0 + u * P;
        f[u] = s < n ? a.part_lse[at(s)] : -INFINITY;
        const float* p = a.part + at(s < n ? s : s0) * HD + 4 * l;
#pragma unroll
        for (int k = 0; k < 4; ++k) v[u][k] = *reinterpret_cast<const float4*>(p + 32 * k);
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        if (f[u] == -INFINITY) continue;  // (a part without keys for the row has not been written)
        const float e = expf(f[u] - top);
        total += e;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          y[4 * k] += e * v[u][k].x;
          y[4 * k + 1] += e * v[u][k].y;
          y[4 * k + 2] += e * v[u][k].z;
          y[4 * k + 3] += e * v[u][k].w;
        }
      }
    }
  }
#pragma unroll
  for (int o = 8; o < 8 * P; o <<= 1) {
    total += __shfl_xor_sync(mask, total, o);
#pragma unroll
    for (int k = 0; k < 16; ++k) y[k] += __shfl_xor_sync(mask, y[k], o);
  }
  const float inv = total != 0.f ? 1.f / total : 0.f;
  const long row = ((long)j.row + tok) * a.Hq + j.kh * G + r % G;
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (k % P == g)
      *reinterpret_cast<uint2*>(a.o + row * HD + 32 * k + 4 * l) =
          make_uint2(pack_bf16(inv * y[4 * k], inv * y[4 * k + 1]), pack_bf16(inv * y[4 * k + 2], inv * y[4 * k + 3]));
  if (a.lse && l == 0 && g == 0) a.lse[row] = total != 0.f ? top + logf(total) : -INFINITY;
}

}  // namespace

size_t paged_join_bytes() { return sizeof(Join); }

cudaError_t launch_attn_paged(const PagedArgs& a, cudaStream_t s) {
  const auto kernel = a.few ? k_paged_few : k_paged_many;
  const size_t smem = (a.few ? sizeof(FewSmem) : sizeof(ManySmem)) + 1024;
  static_assert(2 * (sizeof(FewSmem) + 2048) <= 228 * 1024, "shared memory of two CTAs");
  static_assert(sizeof(ManySmem) + 1024 <= 227 * 1024, "shared memory");
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  if (!a.few) {  // (the register hand-over waits for ever where the block was launched with fewer)
    cudaFuncAttributes fa;
    if ((e = cudaFuncGetAttributes(&fa, k_paged_many)) != cudaSuccess) return e;
    if (fa.numRegs < REGS_LAUNCH) return cudaErrorInvalidConfiguration;
  }
  e = launch_pdl(kernel, dim3((unsigned)a.ctas), dim3(a.few ? FEW_THREADS : MANY_THREADS), smem, s, a);
  if (e != cudaSuccess || a.ctas <= 1) return e;
  const unsigned rows = (a.few ? 1 : 2) * CH;
  return a.many_parts ? launch_pdl(k_paged_join<4>, dim3((unsigned)a.ctas, rows / 8), dim3(256), 0, s, a)
                      : launch_pdl(k_paged_join<1>, dim3((unsigned)a.ctas, rows / 32), dim3(256), 0, s, a);
}

}  // namespace gdn
