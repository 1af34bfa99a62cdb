// gdn_attn_fwd.cu -- causal softmax attention over packed sequences, grouped heads.
//
//   o_i = sum_j p_ij v_j / sum_j p_ij,  p_ij = e^{scale q_i . k_j - max},  j <= i + keys - queries
//
// One pass over the keys with a running maximum and sum per row.  A CTA holds
// two query tiles of 128 rows (gdn_attn.cuh) and streams K and V tiles of 128
// keys through a ring of five 32 KiB slots.  S = Q K^T and O += P V are tcgen05
// products with fp32 accumulators in tensor memory (S and O of both tiles: 4 x
// 128 columns); P goes back to tensor memory as a bf16 A operand over the half
// of S that its row has already been read from.  Four warps own a tile, one
// thread a row, so the row's maximum and sum need no exchange.  The two tiles
// alternate: while one's softmax runs, the other's products do.
//
// The running maximum is only raised when a row's new one is larger by more than
// 8 in base 2 (p then stays below 2^8, exact in scale for bf16 and fp32), which
// after the first tiles is rare: O is rescaled in tensor memory by the row's own
// thread, between the product that wrote it and the next one.
//
// Few rows over many keys (a prompt's part over a cache): the keys are split over
// CTAs, each writes its own normalised output and log-sum in fp32, and a second
// kernel joins them.
//
// Bound: the two products, 1024 cycles per 128 x 128 tile pair at the tensor rate, for
// long prompts: 16384 tokens, 16 query and 2 key heads, in 658 us on a GB300, 1.67
// PFLOP/s, 0.88 of a large library product's rate (beside the products a pair takes 128
// x 128 exponentials, 1024 cycles of the SM's four units, which the other tile's
// products have to hide).  Packed prompts of 0 to 3000 tokens (4 key heads): 64 us,
// 1.05 PFLOP/s; the starts and ends of CTAs (some 5 us each, 3.5 CTAs to an SM), diagonal
// tiles and the last round are the rest.
// (Calls with few rows to a sequence: gdn_attn_split.cu.)
#include <limits.h>
#include <math.h>

#include "gdn_attn.cuh"

namespace gdn {

namespace {

using namespace attn;

constexpr int NSLOT = 5;
// Three groups of four warps: two of softmax, one whose first two warps issue and
// load.  At 384 threads a block may have 168 registers a thread; the third group
// hands most of its own over (2 x 208 + 88 = 3 x 168), and a softmax row's 128
// values stay in registers.
constexpr int FWD_THREADS = 384;
constexpr int REGS_LAUNCH = 168, REGS_SOFTMAX = 208, REGS_ISSUE = 88;
static_assert(2 * REGS_SOFTMAX + REGS_ISSUE <= 3 * REGS_LAUNCH, "the groups' registers come from the block's");
constexpr float RAISE = 8.f;  // base-2 headroom before the running maximum is raised

struct FwdSmem {
  unsigned char q[2][TILE];
  unsigned char slot[NSLOT][TILE];
  uint64_t full[NSLOT], empty[NSLOT];
  uint64_t barQ[2], barS[2], barP[2][2], barO[2];  // barP: the halves of P
  uint32_t tmem;
};

__global__ void __launch_bounds__(FWD_THREADS, 1) k_attn_fwd(const __grid_constant__ AttnArgs a) {
  extern __shared__ unsigned char raw[];
  FwdSmem& sm = *reinterpret_cast<FwdSmem*>(raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u));
  const int tid = threadIdx.x, lane = tid & 31, warp = tc::warp_index();
  pdl_wait();
  pdl_release();
  if (blockIdx.y == 0) clear_status(a.status);
  const int G = a.Hq / a.Hk, TT = CH / G;  // tokens to a tile
  const int kh = blockIdx.x % a.Hk, split = blockIdx.y;
  const Lanes lanes = read_lanes(a);
  const int2 at = find_tile(a.cu_q, lanes.q.y, a.n_seqs, a.total_q, 2 * TT, (int)(blockIdx.x / a.Hk));
  if (at.x < 0) return;
  const Seq sq = seq_of(a, lanes, at.x);
  const int off = sq.kl - sq.ql;
  const int tok0 = at.y * 2 * TT;
  if (tok0 >= sq.ql) return;
  // Key tiles from kb on: n[0] and n[1] of the two query tiles.  A single query
  // tile of a split call is held by both groups of warps, each with every second
  // key tile (`dual`).
  int n[2];
  const int kb = split * a.split_tiles, most = split == a.n_splits - 1 ? INT_MAX : a.split_tiles;
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const int first = tok0 + w * TT, last = min(first + TT, sq.ql) - 1;
    const int keys = last >= first ? min(sq.kl, last + off + 1) : 0;
    n[w] = max(0, min((max(keys, 0) + CH - 1) / CH - kb, most));
  }
  const bool dual = a.n_splits > 1 && tok0 + TT >= sq.ql;
  const int nmax = max(n[0], n[1]);  // key tiles that are loaded
  if (dual) {
    n[1] = nmax / 2;
    n[0] = nmax - n[1];
  }
  const float sc = a.scale * LOG2E;

  const int nt = 2 * nmax;  // ring tiles: K, V of every key tile
  auto load = [&](int t) {
    load_rows(sm.slot[t % NSLOT], (t & 1) ? &a.v : &a.k, kh, sq.k0 + (kb + t / 2) * CH, &sm.full[t % NSLOT]);
  };
  if (warp == 9 && lane == 0) {
    for (int k = 0; k < NSLOT; ++k) {
      tc::mbar_init(&sm.full[k], 1);
      tc::mbar_init(&sm.empty[k], 1);
    }
    for (int w = 0; w < 2; ++w) {
      tc::mbar_init(&sm.barQ[w], 1);
      tc::mbar_init(&sm.barS[w], 1);
      tc::mbar_init(&sm.barO[w], 1);
      tc::mbar_init(&sm.barP[w][0], 128);
      tc::mbar_init(&sm.barP[w][1], 128);
    }
    tc::mbar_fence_init();
    for (int x = 0; x < (dual ? 1 : 2); ++x)  // the first loads at once
      if (n[x] > 0) load_group(sm.q[x], &a.q, kh, G, sq.q0 + tok0 + x * TT, &sm.barQ[x]);
    for (int t = 0; t < min(nt, NSLOT); ++t) load(t);
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
    if (lane == 0 && nmax > 0) {
      for (int t = NSLOT; t < nt && w.ok; ++t) {
        w.on(&sm.empty[t % NSLOT], t / NSLOT - 1);
        if (w.ok) load(t);
      }
      if (w.ok)  // no copy is in flight when the CTA ends
        for (int t = max(0, nt - NSLOT); t < nt; ++t) w.on(&sm.full[t % NSLOT], t / NSLOT);
      else
        for (int k = 0; k < NSLOT; ++k) tc::mbar_wait_sleep(&sm.full[k], 0, 4000000LL);
    }
  } else if (warp == 8) {
    const uint32_t lead = tc::elect_leader();
    if (nmax > 0) {
      auto slot = [&](int t) { return smem_u32(sm.slot[t % NSLOT]); };
      auto arrived = [&](int t) { w.warp_on(&sm.full[t % NSLOT], t / NSLOT); };
      auto release = [&](int t) {
        if (t + NSLOT < nt) tc::commit_by(lead, &sm.empty[t % NSLOT]);
      };
      auto scores = [&](int x, int q, int i) {  // S of group x = Q K^T of key tile i
        tc::gemm128_by<false>(lead, tS + 128 * x, smem_u32(sm.q[q]), slot(2 * i), false);
        tc::commit_by(lead, &sm.barS[x]);
      };
      // O of group x += P V of key tile i, the group's j-th; P arrives by halves
      auto values = [&](int x, int i, int j) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          w.warp_on(&sm.barP[x][h], j);
          tc::fence_after();
          tc::gemm_ts64_by(lead, tO + 128 * x, tS + 128 * x + 32 * h, slot(2 * i + 1) + 8192 * h, j > 0 || h > 0);
        }
        if (j + 1 == n[x]) tc::commit_by(lead, &sm.barO[x]);
      };
      if (n[0] > 0) w.warp_on(&sm.barQ[0], 0);  // (early rows may see no key)
      arrived(0);
      if (dual) {
        scores(0, 0, 0);
        release(0);
        if (nmax > 1) {
          arrived(2);
          scores(1, 0, 1);
          release(2);
        }
        for (int i = 0; i < nmax; ++i) {
          arrived(2 * i + 1);
          values(i & 1, i, i >> 1);
          release(2 * i + 1);
          if (i + 2 < nmax) {
            arrived(2 * i + 4);
            scores(i & 1, 0, i + 2);
            release(2 * i + 4);
          }
        }
      } else {
        if (n[0] > 0) scores(0, 0, 0);
        if (n[1] > 0) {
          w.warp_on(&sm.barQ[1], 0);
          scores(1, 1, 0);
        }
        release(0);
        for (int i = 0; i < nmax; ++i) {
          arrived(2 * i + 1);
          if (i + 1 < nmax) arrived(2 * i + 2);
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            if (i < n[x]) values(x, i, i);
            if (x == 1) release(2 * i + 1);
            if (i + 1 < n[x]) scores(x, x, i + 1);
          }
          if (i + 1 < nmax) release(2 * i + 2);
        }
      }
    }
  }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS_SOFTMAX));
    const int x = warp >> 2, r = 32 * (warp & 3) + lane;
    const uint32_t lane_base = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t S = tS + 128 * x + lane_base, O = tO + 128 * x + lane_base;
    const int tok = tok0 + (dual ? 0 : x * TT) + r / G;
    const bool valid = r < TT * G && tok < sq.ql;
    const int lim = valid ? tok + off : -1;  // the last key that the row sees
    const bool any = __any_sync(0xffffffffu, valid);
    float m = -INFINITY, l = 0.f;
    for (int i = 0; i < n[x]; ++i) {
      const int tile = dual ? 2 * i + x : i;  // of the CTA's key tiles
      const int key0 = (kb + tile) * CH;
      if (key0 + CH > sq.kl) {  // rows past the keys: whatever they hold, they count as zero
        const int t = 2 * tile + 1;
        w.warp_on(&sm.full[t % NSLOT], t / NSLOT);
        zero_rows(sm.slot[t % NSLOT], sq.kl - key0, tid & 127, 128);
        tc::fence_proxy_async();
      }
      w.warp_on(&sm.barS[x], i);
      tc::fence_after();
      if (any) {
        float v[128];
        tc::ld64(S, *reinterpret_cast<float(*)[64]>(v));
        tc::ld64(S + 64, *reinterpret_cast<float(*)[64]>(v + 64));
        if (key0 + CH - 1 > lim) {
#pragma unroll
          for (int j = 0; j < 128; ++j) v[j] = key0 + j <= lim ? v[j] : -INFINITY;
        }
        float mt[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
        for (int j = 4; j < 124; j += 8) {
#pragma unroll
          for (int c = 0; c < 4; ++c) mt[c] = tc::max3(mt[c], v[j + c], v[j + 4 + c]);
        }
        const float mn = fmaxf(tc::max3(mt[0], mt[1], fmaxf(v[124], v[125])), tc::max3(mt[2], mt[3], fmaxf(v[126], v[127])));
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
    if (n[x] > 0) w.warp_on(&sm.barO[x], 0);
    tc::fence_after();
    // a whole tile leaves through shared memory (the Q tile, which the last scores have
    // read) and one TMA store, rows of a part of one from their own threads
    const int first = tok0 + (dual ? 0 : x * TT);
    const bool tile = a.n_splits == 1 && first + TT <= sq.ql;
    if (any) {
      const long row = ((long)sq.q0 + tok) * a.Hq + kh * G + r % G;
      // (a sum of zero: the row sees no key; one of NaN is neither greater nor equal, and goes on)
      const float inv = l != 0.f ? 1.f / l : 0.f;
      const float lse = l != 0.f ? m * a.scale + logf(l) : -INFINITY;
#pragma unroll 1
      for (int g = 0; g < 4; ++g) {
        float y[32];
        if (n[x] > 0) {
          tc::ld32(O + 32 * g, y);
        }
        if (valid) {
          if (n[x] == 0 || l == 0.f) {
#pragma unroll
            for (int j = 0; j < 32; ++j) y[j] = 0.f;
          }
          if (tile) {
            stage32(sm.q[x], r, 32 * g, y, inv);
          } else if (a.n_splits == 1) {
            store32(a.o + row * HD + 32 * g, y, inv);
          } else if (l != 0.f) {  // (the join reads no part whose lse is minus infinity)
            float* d = a.part + ((long)(2 * split + x) * a.total_q * a.Hq + row) * HD + 32 * g;
#pragma unroll
            for (int j = 0; j < 8; ++j)
              *reinterpret_cast<float4*>(d + 4 * j) =
                  make_float4(inv * y[4 * j], inv * y[4 * j + 1], inv * y[4 * j + 2], inv * y[4 * j + 3]);
          }
        }
        __syncwarp();
      }
      if (valid) {
        if (a.n_splits > 1) {
          // (two parts to a split; a query tile that one group holds alone leaves the other empty)
          if (!dual) a.part_lse[(long)(2 * split + 1 - x) * a.total_q * a.Hq + row] = -INFINITY;
          a.part_lse[(long)(2 * split + x) * a.total_q * a.Hq + row] = lse;
        } else if (a.lse) {
          a.lse[row] = lse;
        }
      }
    }
    if (tile) {
      tc::fence_proxy_async();
      asm volatile("bar.sync %0, 128;" ::"r"(1 + x) : "memory");
      if ((tid & 127) == 0) store_tile(&a.mo, kh * G, sq.q0 + first, sm.q[x]);
    }
    tc::fence_before();
  }
  if (!w.ok && a.status) atomicOr(a.status, 1);
  __syncthreads();
  tc::fence_after();
  if (warp == 0) tc::dealloc(sm.tmem, 512);
}

// Joins the splits of a row: o = sum_s e^{lse_s - lse} o_s.  One warp per row.  A part of
// NaN makes the row NaN, as it would be in one piece.
__global__ void __launch_bounds__(256) k_attn_join(const __grid_constant__ AttnArgs a) {
  pdl_wait();
  pdl_release();
  const long rows = (long)a.total_q * a.Hq, row = (long)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (row >= rows) return;
  float top = -INFINITY;
  bool nan = false;  // (which fmaxf passes over)
  for (int s = lane; s < a.n_parts; s += 32) {
    const float l = a.part_lse[s * rows + row];
    nan |= isnan(l);
    top = fmaxf(top, l);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if (__any_sync(0xffffffffu, nan)) top = NAN;
  float total = 0.f, y[4] = {0.f, 0.f, 0.f, 0.f};
  if (top != -INFINITY)
    for (int s = 0; s < a.n_parts; ++s) {
      const float l = a.part_lse[s * rows + row];
      if (l == -INFINITY) continue;
      const float f = expf(l - top);
      const float4 p = *reinterpret_cast<const float4*>(a.part + (s * rows + row) * HD + 4 * lane);
      total += f;
      y[0] += f * p.x;
      y[1] += f * p.y;
      y[2] += f * p.z;
      y[3] += f * p.w;
    }
  const float inv = total != 0.f ? 1.f / total : 0.f;
  *reinterpret_cast<uint2*>(a.o + row * HD + 4 * lane) =
      make_uint2(pack_bf16(inv * y[0], inv * y[1]), pack_bf16(inv * y[2], inv * y[3]));
  if (a.lse && lane == 0) a.lse[row] = total != 0.f ? top + logf(total) : -INFINITY;
}

}  // namespace

cudaError_t launch_attn_fwd(const AttnArgs& a, cudaStream_t s) {
  constexpr size_t smem = sizeof(FwdSmem) + 1024;
  static_assert(smem <= 227 * 1024, "shared memory");
  cudaError_t e = cudaFuncSetAttribute(k_attn_fwd, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  // (the register hand-over waits for ever where the block was launched with fewer)
  cudaFuncAttributes fa;
  if ((e = cudaFuncGetAttributes(&fa, k_attn_fwd)) != cudaSuccess) return e;
  if (fa.numRegs < REGS_LAUNCH) return cudaErrorInvalidConfiguration;
  const int K = 2 * (CH / (a.Hq / a.Hk));
  const dim3 grid((unsigned)a.Hk * (unsigned)(a.total_q / K + a.n_seqs), (unsigned)a.n_splits);
  e = launch_pdl(k_attn_fwd, grid, dim3(FWD_THREADS), smem, s, a);
  return e != cudaSuccess || a.n_splits == 1 ? e : launch_attn_join(a, s);
}

cudaError_t launch_attn_join(const AttnArgs& a, cudaStream_t s) {
  const long rows = (long)a.total_q * a.Hq;
  return launch_pdl(k_attn_join, dim3((unsigned)((rows + 7) / 8)), dim3(256), 0, s, a);
}

}  // namespace gdn
