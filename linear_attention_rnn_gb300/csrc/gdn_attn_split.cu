// gdn_attn_split.cu -- attention of a few query rows to a sequence: single tokens (or a
// few new ones) over a cache, short prompts.
//
// The mathematics of gdn_attn_fwd.cu for one query tile (128 rows: 128 / G tokens of a
// sequence, each with the G query heads of one key head; most of them are empty for
// single tokens) against tiles of 64 keys.  The keys of long sequences are split over
// CTAs, each of which writes its own normalised output and log-sum in fp32; k_attn_join
// puts them together.
//
// Bound: HBM (k and v once).  What a CTA's start and end take, some 6 us in which it
// reads nothing, is hidden by a second CTA on the same SM: half the keys to a tile and
// one query tile leave room for two (96 KiB of shared memory, 256 TMEM columns each),
// with 2 x 64 KiB of K and V on their way.  S is issued behind the P V before it, so one
// S buffer is enough: softmax, P V and the next S take some 1500 cycles a tile, and two
// CTAs need one each in 2100 to take in what memory gives an SM.  Measured on a GB300, one
// token each: 32 caches of 4096 rows, 16 heads without groups, 166 us, 6.5 TB/s, 0.96 of a
// copy's rate; 32 caches of 1 to 16214 rows, 4 key heads, 95 us, 0.82 of it (unequal CTAs).
#include "gdn_attn.cuh"

namespace gdn {

namespace {

using namespace attn;

constexpr int KEYS = 64, NSLOT = 4;
constexpr uint32_t KTILE = KEYS * HD * 2;
constexpr int SPLIT_THREADS = 192;  // four warps of softmax, one that issues, one that loads
constexpr float RAISE = 8.f;        // base-2 headroom before the running maximum is raised

struct SplitSmem {
  unsigned char q[TILE];
  unsigned char slot[NSLOT][KTILE];
  uint64_t full[NSLOT], empty[NSLOT];
  uint64_t barQ, barS, barP, barO;
  uint32_t tmem;
};

__global__ void __launch_bounds__(SPLIT_THREADS, 2) k_attn_split(const __grid_constant__ AttnArgs a) {
  extern __shared__ unsigned char raw[];
  SplitSmem& sm = *reinterpret_cast<SplitSmem*>(raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u));
  const int tid = threadIdx.x, lane = tid & 31, warp = tc::warp_index();
  pdl_wait();
  pdl_release();
  if (blockIdx.y == 0) clear_status(a.status);
  const int G = a.Hq / a.Hk, TT = CH / G;  // tokens to a tile
  const int kh = blockIdx.x % a.Hk, split = blockIdx.y;
  const Lanes lanes = read_lanes(a);
  const int2 at = find_tile(a.cu_q, lanes.q.y, a.n_seqs, a.total_q, TT, (int)(blockIdx.x / a.Hk));
  if (at.x < 0) return;
  const Seq sq = seq_of(a, lanes, at.x);
  const int off = sq.kl - sq.ql, tok0 = at.y * TT;
  if (tok0 >= sq.ql) return;
  // keys [kb, ke) of this CTA
  const int keys = max(0, min(sq.kl, min(tok0 + TT, sq.ql) + off));
  const long run = (long)a.split_tiles * CH;
  const int kb = (int)min(split * run, (long)keys);
  const int ke = split == a.n_splits - 1 ? keys : (int)min((split + 1) * run, (long)keys);
  const int n = (ke - kb + KEYS - 1) / KEYS;

  const int nt = 2 * n;
  auto load = [&](int t) {
    uint64_t* bar = &sm.full[t % NSLOT];
    const CUtensorMap* m = (t & 1) ? &a.v : &a.k;
    unsigned char* dst = sm.slot[t % NSLOT];
    const int row = sq.k0 + kb + (t / 2) * KEYS;
    tc::arrive_expect_tx(bar, KTILE);
    tc::tma_load_3d(dst, m, 0, kh, row, bar);
    tc::tma_load_3d(dst + KTILE / 2, m, 64, kh, row, bar);
  };
  if (warp == 5 && lane == 0) {
    for (int k = 0; k < NSLOT; ++k) {
      tc::mbar_init(&sm.full[k], 1);
      tc::mbar_init(&sm.empty[k], 1);
    }
    tc::mbar_init(&sm.barQ, 1);
    tc::mbar_init(&sm.barS, 1);
    tc::mbar_init(&sm.barO, 1);
    tc::mbar_init(&sm.barP, 128);
    tc::mbar_fence_init();
    if (n > 0) load_group(sm.q, &a.q, kh, G, sq.q0 + tok0, &sm.barQ);  // the first loads at once
    for (int t = 0; t < min(nt, NSLOT); ++t) load(t);
  }
  if (warp == 0) tc::alloc(&sm.tmem, 256);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tS = sm.tmem, tO = sm.tmem + 128;
  tc::Wait w;

  if (warp == 5) {
    if (lane == 0 && n > 0) {
      for (int t = NSLOT; t < nt && w.ok; ++t) {
        w.on(&sm.empty[t % NSLOT], t / NSLOT - 1);
        if (w.ok) load(t);
      }
      if (w.ok)  // no copy is in flight when the CTA ends
        for (int t = max(0, nt - NSLOT); t < nt; ++t) w.on(&sm.full[t % NSLOT], t / NSLOT);
      else
        for (int k = 0; k < NSLOT; ++k) tc::mbar_wait_sleep(&sm.full[k], 0, 4000000LL);
    }
  } else if (warp == 4) {
    const uint32_t lead = tc::elect_leader();
    if (n > 0) {
      auto slot = [&](int t) { return smem_u32(sm.slot[t % NSLOT]); };
      auto arrived = [&](int t) { w.warp_on(&sm.full[t % NSLOT], t / NSLOT); };
      auto release = [&](int t) {
        if (t + NSLOT < nt) tc::commit_by(lead, &sm.empty[t % NSLOT]);
      };
      auto scores = [&](int i) {
        arrived(2 * i);
        tc::gemm128x64_by(lead, tS, smem_u32(sm.q), slot(2 * i));
        tc::commit_by(lead, &sm.barS);
        release(2 * i);
      };
      w.warp_on(&sm.barQ, 0);
      scores(0);
      for (int i = 0; i < n; ++i) {
        arrived(2 * i + 1);
        w.warp_on(&sm.barP, i);
        tc::fence_after();
        tc::gemm_ts64_by<KEYS>(lead, tO, tS, slot(2 * i + 1), i > 0);
        release(2 * i + 1);
        if (i + 1 < n) scores(i + 1);
      }
      tc::commit_by(lead, &sm.barO);
    }
  } else {
    const int r = 32 * warp + lane;
    const uint32_t lane_base = (uint32_t)(32 * warp) << 16;
    const uint32_t S = tS + lane_base, O = tO + lane_base;
    const int tok = tok0 + r / G;
    const bool valid = r < TT * G && tok < sq.ql;
    const int lim = valid ? tok + off : -1;  // the last key that the row sees
    const bool any = __any_sync(0xffffffffu, valid);
    const float sc = a.scale * LOG2E;
    float m = -INFINITY, l = 0.f;
    for (int i = 0; i < n; ++i) {
      const int key0 = kb + i * KEYS;
      if (key0 + KEYS > sq.kl) {  // rows past the keys: whatever they hold, they count as zero
        const int t = 2 * i + 1;
        w.warp_on(&sm.full[t % NSLOT], t / NSLOT);
        for (int c = (sq.kl - key0) * 16 + tid; c < KEYS * 16; c += 128)
          *reinterpret_cast<uint4*>(sm.slot[t % NSLOT] + tc::sw128_chunk(c >> 4, c & 15, KEYS)) = make_uint4(0u, 0u, 0u, 0u);
        tc::fence_proxy_async();
      }
      w.warp_on(&sm.barS, i);
      tc::fence_after();
      if (any) {
        float v[64];
        tc::ld64(S, v);
        if (key0 + KEYS - 1 > lim) {
#pragma unroll
          for (int j = 0; j < 64; ++j) v[j] = key0 + j <= lim ? v[j] : -INFINITY;
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
    if (n > 0) w.warp_on(&sm.barO, 0);
    tc::fence_after();
    if (any) {
      const long row = ((long)sq.q0 + tok) * a.Hq + kh * G + r % G, part = (long)split * a.total_q * a.Hq + row;
      // (a sum of zero: the row sees no key; one of NaN is neither greater nor equal, and goes on)
      const float inv = l != 0.f ? 1.f / l : 0.f;
#pragma unroll 1
      for (int g = 0; g < 4; ++g) {
        float y[32];
        if (n > 0) {
          tc::ld32(O + 32 * g, y);
        }
        if (valid && a.n_splits == 1) {
          if (l == 0.f) {
#pragma unroll
            for (int j = 0; j < 32; ++j) y[j] = 0.f;
          }
          store32(a.o + row * HD + 32 * g, y, inv);
        } else if (valid && l != 0.f) {  // (the join reads no part whose lse is minus infinity)
          float* d = a.part + part * HD + 32 * g;
#pragma unroll
          for (int j = 0; j < 8; ++j)
            *reinterpret_cast<float4*>(d + 4 * j) =
                make_float4(inv * y[4 * j], inv * y[4 * j + 1], inv * y[4 * j + 2], inv * y[4 * j + 3]);
        }
        __syncwarp();
      }
      const float lse = l != 0.f ? m * a.scale + logf(l) : -INFINITY;
      if (valid && a.n_splits > 1) a.part_lse[part] = lse;
      if (valid && a.n_splits == 1 && a.lse) a.lse[row] = lse;
    }
    tc::fence_before();
  }
  if (!w.ok && a.status) atomicOr(a.status, 1);
  __syncthreads();
  tc::fence_after();
  if (warp == 0) tc::dealloc(sm.tmem, 256);
}

}  // namespace

cudaError_t launch_attn_split(const AttnArgs& a, cudaStream_t s) {
  constexpr size_t smem = sizeof(SplitSmem) + 1024;
  static_assert(2 * (smem + 1024) <= 228 * 1024, "shared memory of two CTAs");
  cudaError_t e = cudaFuncSetAttribute(k_attn_split, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)a.Hk * (unsigned)(a.total_q / (CH / (a.Hq / a.Hk)) + a.n_seqs), (unsigned)a.n_splits);
  e = launch_pdl(k_attn_split, grid, dim3(SPLIT_THREADS), smem, s, a);
  return e != cudaSuccess || a.n_splits == 1 ? e : launch_attn_join(a, s);
}

}  // namespace gdn
