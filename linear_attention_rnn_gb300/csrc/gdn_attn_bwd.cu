// gdn_attn_bwd.cu -- backward of causal softmax attention over packed sequences.
//
// With p_ij = e^{scale q_i . k_j - lse_i} (recomputed), dp_ij = dO_i . v_j and
// delta_i = dO_i . o_i:
//     ds_ij = p_ij (dp_ij - delta_i),
//     dv_j = sum_i p_ij dO_i,   dk_j = scale sum_i ds_ij q_i,   dq_i = scale sum_j ds_ij k_j.
//
// Two kinds of CTAs, so that every gradient is summed in one CTA, in a fixed order,
// without atomics (seven products per tile pair instead of five):
//   dkv   one CTA per 128 keys and key head, over the query tiles that see
//               them: S^T = K Q^T, dP^T = V dO^T, dV += P^T dO, dK += dS^T Q.  A query
//               tile holds all heads of the group, so the sum over them is part
//               of the product.
//   dq    one CTA per query tile, over the key tiles: S = Q K^T, dP = dO V^T,
//               dQ += dS K.
// Accumulators in tensor memory, P and dS as bf16 A operands there too (each
// half over the fp32 half that its own four warps have read).  Eight compute
// warps hold a tile, 64 columns to a thread.  While they form dS, the tensor
// cores run the next S; while they form P, the last gradient product.
//
// Roundings: P and dS become bf16 once, as operands, and so does every result; delta
// takes the forward's rounded o, as the caller has it, where a row sees more than EARLY
// keys.  A gradient's error against 64 bits is then 2.3e-3 to 2.5e-3 in the 2-norm
// (rounding the result alone: 1.7e-3); scores, lse, delta and all sums are fp32.
//
// Bound: the tensor rate (7 x 512 cycles per pair of 128 x 128 tiles).  Measured on a
// GB300, 4096 + 2048 + 1000 + 977 + 71 packed tokens, 16 query and 4 key heads: 236 us,
// the tensor pipe busy for 0.62 of it; delta 15 us; with the forward 334 us.  Two CTAs
// for the heaviest key tiles were slower (by 15 us): the SMs are busy to the end as it is.
#include "gdn_attn.cuh"

namespace gdn {

namespace {

using namespace attn;

constexpr int BWD_THREADS = 256 + 64;
constexpr int KV_SLOTS = 4;  // Q, dO of two query tiles
constexpr int Q_SLOTS = 5;   // K, V of two key tiles and a half

// ---- delta_i = dO_i . o_i: half a warp to a row, four rows in flight ------------------
// The caller's o is rounded to bf16, which shows in the gradients of rows that see few
// keys (their dP - delta is largest, and cancels most).  For rows with up to EARLY keys
// delta is therefore formed as sum_j p_ij dp_ij: one pass over a sequence's first keys, by
// blocks of their own, first in the grid.  It brings the error of dq and dk against 64
// bits from 2.5e-3 to 2.4e-3 in the 2-norm, of sequences of two or three tokens from 7e-3
// to 2.5e-3, and costs 2 us of 323 (16 keys: 2.38e-3, and 3 to 6 us).
constexpr int DELTA_ROWS = 64;  // rows per block of 256 threads
constexpr int EARLY = 8;
constexpr int EARLY_BLOCKS = 65536;  // at most

__device__ __forceinline__ float dot8(const uint4& x, const uint4& y) {
  const uint32_t u[4] = {x.x, x.y, x.z, x.w}, v[4] = {y.x, y.y, y.z, y.w};
  float d = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = unpack_bf16(u[i]), q = unpack_bf16(v[i]);
    d += p.x * q.x + p.y * q.y;
  }
  return d;
}
__device__ __forceinline__ float sum16(float d, unsigned mask) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) d += __shfl_xor_sync(mask, d, o);
  return d;
}

// Rows (sequence, keys seen - 1, head), half a warp to each
__device__ __forceinline__ void early_delta(const AttnArgs& a, int early_blocks) {
  const int G = a.Hq / a.Hk, c = 8 * (threadIdx.x & 15);
  const unsigned half = 0xffffu << (threadIdx.x & 16);
  const long all = (long)a.n_seqs * EARLY * a.Hq;
  for (long i = (long)blockIdx.x * 16 + (threadIdx.x >> 4); i < all; i += 16L * early_blocks) {
    const int head = (int)(i % a.Hq), vis = (int)(i / a.Hq % EARLY), s = (int)(i / a.Hq / EARLY);
    const int2 q = rows_of(a.cu_q, s, a.n_seqs, a.total_q), k = rows_of(a.cu_k, s, a.n_seqs, a.total_k);
    const int t = vis - (k.y - q.y);
    if (t < 0 || t >= q.y || vis >= k.y) continue;
    const long row = ((long)q.x + t) * a.Hq + head;
    const uint4 x = *reinterpret_cast<const uint4*>(a.pq + ((long)q.x + t) * a.sq + head * HD + c);
    const uint4 y = *reinterpret_cast<const uint4*>(a.dOp + row * HD + c);
    const bf16* kp = a.pk + (long)k.x * a.sk + head / G * HD + c;
    const bf16* vp = a.pv + (long)k.x * a.sv + head / G * HD + c;
    const float lse = a.lse[row] * LOG2E, sc = a.scale * LOG2E;
    float d = 0.f;
#pragma unroll 4
    for (int j = 0; j <= vis; ++j) {
      const float z = sum16(dot8(x, *reinterpret_cast<const uint4*>(kp + j * a.sk)), half);
      const float dp = sum16(dot8(y, *reinterpret_cast<const uint4*>(vp + j * a.sv)), half);
      d += ex2(z * sc - lse) * dp;
    }
    if ((threadIdx.x & 15) == 0) a.delta[row] = d;
  }
}

__global__ void __launch_bounds__(256, 4) k_attn_delta(const __grid_constant__ AttnArgs a, int early_blocks) {
  pdl_wait();  // (before it lets the next kernel start, which reads its inputs without a wait)
  pdl_release();
  clear_status(a.status);
  if ((int)blockIdx.x < early_blocks) {
    early_delta(a, early_blocks);
    return;
  }
  const long rows = (long)a.total_q * a.Hq;
  const long row0 = (long)((int)blockIdx.x - early_blocks) * DELTA_ROWS + (threadIdx.x >> 4);
  const int c = 8 * (threadIdx.x & 15);
  uint4 x[4], y[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const long row = min(row0 + 16 * k, rows - 1);
    x[k] = *reinterpret_cast<const uint4*>(a.dOp + row * HD + c);
    y[k] = *reinterpret_cast<const uint4*>(a.op + row * HD + c);
  }
  // whether the four rows are early_delta's, a row to a lane, while they are on their way
  const int tok = (int)(min(row0 + 16 * (threadIdx.x & 3), rows - 1) / a.Hq);
  int s = a.cu_q ? 0 : tok / (a.total_q / a.n_seqs);
  if (a.cu_q)
    for (int hi = a.n_seqs; hi - s > 1;) {  // the last sequence that begins at tok or before
      const int mid = (s + hi) >> 1;
      if (a.cu_q[mid] <= tok)
        s = mid;
      else
        hi = mid;
    }
  const int2 q = rows_of(a.cu_q, s, a.n_seqs, a.total_q), kk = rows_of(a.cu_k, s, a.n_seqs, a.total_k);
  const int vis = tok - q.x + kk.y - q.y;
  const unsigned skip = __ballot_sync(0xffffffffu, vis >= 0 && vis < EARLY) >> (threadIdx.x & 16);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float d = sum16(dot8(x[k], y[k]), 0xffffffffu);
    if ((threadIdx.x & 15) == 0 && row0 + 16 * k < rows && !(skip >> k & 1)) a.delta[row0 + 16 * k] = d;
  }
}

// ---- dK, dV -------------------------------------------------------------------------
struct KvSmem {
  unsigned char k[TILE], v[TILE];
  unsigned char slot[KV_SLOTS][TILE];
  alignas(16) float lse[2][CH];  // of the query rows: -lse in base 2, delta, the last key seen
  alignas(16) float delta[2][CH];
  alignas(16) int lim[2][CH];
  uint64_t full[KV_SLOTS], empty[KV_SLOTS];
  uint64_t barKV, barS, barD, barP, barDs, barEnd;
  uint32_t tmem;
};

__device__ __forceinline__ void dkv(const AttnArgs& a, unsigned char* raw, int block) {
  KvSmem& sm = *reinterpret_cast<KvSmem*>(raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u));
  const int tid = threadIdx.x, lane = tid & 31, warp = tc::warp_index();
  const int G = a.Hq / a.Hk, TT = CH / G;
  const int kh = block % a.Hk;
  const Lanes lanes = read_lanes(a);
  const int2 at = find_tile(a.cu_k, lanes.k.y, a.n_seqs, a.total_k, CH, block / a.Hk);
  if (at.x < 0) return;
  const Seq sq = seq_of(a, lanes, at.x);
  // (a sequence's first keys are seen by the most queries: index 0 is its last tile)
  const int key0 = ((sq.kl + CH - 1) / CH - 1 - at.y) * CH, off = sq.kl - sq.ql;
  const int first = max(0, key0 - off) / TT;                 // first query tile that sees key0
  const int n = max(0, (sq.ql + TT - 1) / TT - first);

  const int nt = 2 * n;
  auto load = [&](int t) {
    load_group(sm.slot[t % KV_SLOTS], (t & 1) ? &a.dO : &a.q, kh, G, sq.q0 + (first + t / 2) * TT,
               &sm.full[t % KV_SLOTS]);
  };
  if (warp == 9 && lane == 0) {
    for (int k = 0; k < KV_SLOTS; ++k) {
      tc::mbar_init(&sm.full[k], 1);
      tc::mbar_init(&sm.empty[k], 1);
    }
    tc::mbar_init(&sm.barKV, 1);
    tc::mbar_init(&sm.barS, 1);
    tc::mbar_init(&sm.barD, 1);
    tc::mbar_init(&sm.barEnd, 1);
    tc::mbar_init(&sm.barP, 256);
    tc::mbar_init(&sm.barDs, 256);
    tc::mbar_fence_init();
    if (n > 0) {  // the first loads at once
      tc::arrive_expect_tx(&sm.barKV, 2 * TILE);
      for (int h = 0; h < 2; ++h) {
        tc::tma_load_3d(sm.k + h * (TILE / 2), &a.k, 64 * h, kh, sq.k0 + key0, &sm.barKV);
        tc::tma_load_3d(sm.v + h * (TILE / 2), &a.v, 64 * h, kh, sq.k0 + key0, &sm.barKV);
      }
      for (int t = 0; t < min(nt, KV_SLOTS); ++t) load(t);
    }
  }
  if (warp == 0) tc::alloc(&sm.tmem, 512);
  if (TT * G < CH)  // rows that no load writes, but the products over rows read
    for (int k = 0; k < KV_SLOTS; ++k) zero_rows(sm.slot[k], TT * G, tid, BWD_THREADS);
  tc::fence_proxy_async();
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tS = sm.tmem, tP = tS + 128, tV = tS + 256, tK = tS + 384;
  tc::Wait w;

  if (warp == 9) {
    if (lane == 0 && n > 0) {
      for (int t = KV_SLOTS; t < nt && w.ok; ++t) {
        w.on(&sm.empty[t % KV_SLOTS], t / KV_SLOTS - 1);
        if (w.ok) load(t);
      }
      if (w.ok) {
        w.on(&sm.barKV, 0);
        for (int t = max(0, nt - KV_SLOTS); t < nt; ++t) w.on(&sm.full[t % KV_SLOTS], t / KV_SLOTS);
      } else {
        for (int k = 0; k < KV_SLOTS; ++k) tc::mbar_wait_sleep(&sm.full[k], 0, 4000000LL);
      }
    }
  } else if (warp == 8) {
    const uint32_t lead = tc::elect_leader();
    if (n > 0) {
      auto slot = [&](int t) { return smem_u32(sm.slot[t % KV_SLOTS]); };
      auto arrived = [&](int t) { w.warp_on(&sm.full[t % KV_SLOTS], t / KV_SLOTS); };
      auto release = [&](int t) {
        if (t + KV_SLOTS < nt) tc::commit_by(lead, &sm.empty[t % KV_SLOTS]);
      };
      auto scores = [&](int i) {
        arrived(2 * i);
        tc::gemm128_by<false>(lead, tS, smem_u32(sm.k), slot(2 * i), false);
        tc::commit_by(lead, &sm.barS);
      };
      auto dscores = [&](int i) {
        arrived(2 * i + 1);
        tc::gemm128_by<false>(lead, tP, smem_u32(sm.v), slot(2 * i + 1), false);
        tc::commit_by(lead, &sm.barD);
      };
      w.warp_on(&sm.barKV, 0);
      scores(0);
      dscores(0);
      for (int i = 0; i < n; ++i) {
        w.warp_on(&sm.barP, i);
        tc::fence_after();
        tc::gemm_ts_by(lead, tV, tS, slot(2 * i + 1), i > 0);  // dV += P^T dO
        if (i + 1 < n) scores(i + 1);
        w.warp_on(&sm.barDs, i);
        tc::fence_after();
        tc::gemm_ts_by(lead, tK, tP, slot(2 * i), i > 0);      // dK += dS^T Q
        release(2 * i);
        release(2 * i + 1);
        if (i + 1 < n) dscores(i + 1);
      }
      tc::commit_by(lead, &sm.barEnd);
    }
  } else {
    const int g0 = warp >> 2, r = 32 * (warp & 3) + lane;  // key row r, columns 64 g0 .. 64 g0 + 63
    const uint32_t lane_base = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t S = tS + lane_base + 64 * g0, P = tP + lane_base + 64 * g0;
    const int key = key0 + r;
    const float sc = a.scale * LOG2E;
    // Per query row (a column here): lse (base 2), delta and the last key that it
    // sees, read from global memory two tiles ahead, written to shared memory one ahead.
    float c_lse = 0.f, c_delta = 0.f;
    int c_lim = -1;
    auto fetch_cols = [&](int i) {
      const int tok = (first + i) * TT + tid / G;
      const bool ok = tid < TT * G && tok < sq.ql;
      const long row = ((long)sq.q0 + tok) * a.Hq + kh * G + tid % G;
      c_lim = ok ? tok + off : -1;
      c_lse = ok ? a.lse[row] : 0.f;
      c_delta = ok ? a.delta[row] : 0.f;
    };
    auto put_cols = [&](int i) {
      sm.lim[i & 1][tid] = c_lim;
      sm.lse[i & 1][tid] = -c_lse * LOG2E;
      sm.delta[i & 1][tid] = c_delta;
    };
    pdl_wait();  // (delta, from the kernel before; everything else was complete when it began)
    pdl_release();
    if (n > 0 && tid < CH) {
      fetch_cols(0);
      put_cols(0);
      fetch_cols(1);
    }
    asm volatile("bar.sync 1, 256;" ::: "memory");
    for (int i = 0; i < n; ++i) {
      const int b = i & 1;
      const int tok0 = (first + i) * TT, live = min(sq.ql - tok0, TT) * G;  // rows of tokens that exist
      const bool whole = live == CH && key0 + CH - 1 <= tok0 + off;         // every row sees every key
      const float4* c_l = reinterpret_cast<const float4*>(sm.lse[b] + 64 * g0);
      const float4* c_d = reinterpret_cast<const float4*>(sm.delta[b] + 64 * g0);
      const int4* c_m = reinterpret_cast<const int4*>(sm.lim[b] + 64 * g0);
      float p[64];
      w.warp_on(&sm.barS, i);
      tc::fence_after();
      tc::ld64(S, p);
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const float4 l = c_l[j];
        p[4 * j] = ex2(p[4 * j] * sc + l.x);
        p[4 * j + 1] = ex2(p[4 * j + 1] * sc + l.y);
        p[4 * j + 2] = ex2(p[4 * j + 2] * sc + l.z);
        p[4 * j + 3] = ex2(p[4 * j + 3] * sc + l.w);
      }
      if (!whole) {
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const int4 m = c_m[j];
          p[4 * j] = key <= m.x ? p[4 * j] : 0.f;
          p[4 * j + 1] = key <= m.y ? p[4 * j + 1] : 0.f;
          p[4 * j + 2] = key <= m.z ? p[4 * j + 2] : 0.f;
          p[4 * j + 3] = key <= m.w ? p[4 * j + 3] : 0.f;
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) tc::st16_bf16(S + 16 * h, *reinterpret_cast<float(*)[32]>(p + 32 * h));
      if (live < TT * G) {  // rows past the sequence's end: whatever they hold, they count as zero
        const int t = 2 * i;
        w.warp_on(&sm.full[t % KV_SLOTS], t / KV_SLOTS);
        w.warp_on(&sm.full[(t + 1) % KV_SLOTS], (t + 1) / KV_SLOTS);
        w.warp_on(&sm.barD, i);  // (dO's product with V has read it)
        zero_rows(sm.slot[t % KV_SLOTS], live, tid, 256);
        zero_rows(sm.slot[(t + 1) % KV_SLOTS], live, tid, 256);
        tc::fence_proxy_async();
      }
      tc::wait_st();
      tc::fence_before();
      tc::mbar_arrive(&sm.barP);
      if (tid < CH && i + 1 < n) {
        put_cols(i + 1);
        fetch_cols(i + 2);
      }
      w.warp_on(&sm.barD, i);
      tc::fence_after();
      float v[64];
      tc::ld64(P, v);
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const float4 d = c_d[j];
        v[4 * j] = p[4 * j] * (v[4 * j] - d.x);
        v[4 * j + 1] = p[4 * j + 1] * (v[4 * j + 1] - d.y);
        v[4 * j + 2] = p[4 * j + 2] * (v[4 * j + 2] - d.z);
        v[4 * j + 3] = p[4 * j + 3] * (v[4 * j + 3] - d.w);
      }
      if (!whole) {  // (a masked dP may be anything, NaN too)
#pragma unroll
        for (int j = 0; j < 64; ++j) v[j] = p[j] == 0.f ? 0.f : v[j];
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) tc::st16_bf16(P + 16 * h, *reinterpret_cast<float(*)[32]>(v + 32 * h));
      tc::wait_st();
      tc::fence_before();
      tc::mbar_arrive(&sm.barDs);
      asm volatile("bar.sync 1, 256;" ::: "memory");  // the next tile's columns are in shared memory
    }
    if (n > 0) w.warp_on(&sm.barEnd, 0);
    tc::fence_after();
    // warps 0-3 write dV, 4-7 dK: a whole tile through V's or K's place in shared memory
    // (the last products have read them) and one TMA store, else row by row
    const long row = ((long)sq.k0 + key) * a.Hk + kh;
    const bool tile = key0 + CH <= sq.kl;
    unsigned char* staged = g0 ? sm.k : sm.v;
#pragma unroll 1
    for (int h = 0; h < 4; ++h) {
      float v[32];
      if (n > 0) {
        tc::ld32((g0 ? tK : tV) + lane_base + 32 * h, v);
      } else {
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = 0.f;
      }
      if (tile)
        stage32(staged, r, 32 * h, v, g0 ? a.scale : 1.f);
      else if (key < sq.kl)
        store32((g0 ? a.dk : a.dv) + row * HD + 32 * h, v, g0 ? a.scale : 1.f);
      __syncwarp();
    }
    if (tile) {
      tc::fence_proxy_async();
      asm volatile("bar.sync %0, 128;" ::"r"(2 + g0) : "memory");
      if ((tid & 127) == 0) store_tile(g0 ? &a.mdk : &a.mdv, kh, sq.k0 + key0, staged);
    }
    tc::fence_before();
  }
  if (!w.ok && a.status) atomicOr(a.status, 1);
  __syncthreads();
  tc::fence_after();
  if (warp == 0) tc::dealloc(sm.tmem, 512);
}

// ---- dQ ---------------------------------------------------------------------------------
struct QSmem {
  unsigned char q[TILE], dO[TILE];
  unsigned char slot[Q_SLOTS][TILE];
  uint64_t full[Q_SLOTS], empty[Q_SLOTS];
  // barS: of even and odd key tiles.  S runs one tile ahead of its readers, so a
  // barrier for both could complete two phases before a late one has seen the first.
  uint64_t barQ, barS[2], barD, barDs, barEnd;
  uint32_t tmem;
};

__device__ __forceinline__ void dq(const AttnArgs& a, unsigned char* raw, int block) {
  QSmem& sm = *reinterpret_cast<QSmem*>(raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u));
  const int tid = threadIdx.x, lane = tid & 31, warp = tc::warp_index();
  const int G = a.Hq / a.Hk, TT = CH / G;
  const int kh = block % a.Hk;
  const Lanes lanes = read_lanes(a);
  const int2 at = find_tile(a.cu_q, lanes.q.y, a.n_seqs, a.total_q, TT, block / a.Hk);
  if (at.x < 0) return;
  const Seq sq = seq_of(a, lanes, at.x);
  const int tok0 = at.y * TT, off = sq.kl - sq.ql;
  if (tok0 >= sq.ql) return;
  const int keys = max(0, min(sq.kl, min(tok0 + TT, sq.ql) + off));
  const int n = (keys + CH - 1) / CH;

  const int nt = 2 * n;
  auto load = [&](int t) {
    load_rows(sm.slot[t % Q_SLOTS], (t & 1) ? &a.v : &a.k, kh, sq.k0 + (t / 2) * CH, &sm.full[t % Q_SLOTS]);
  };
  if (warp == 9 && lane == 0) {
    for (int k = 0; k < Q_SLOTS; ++k) {
      tc::mbar_init(&sm.full[k], 1);
      tc::mbar_init(&sm.empty[k], 1);
    }
    tc::mbar_init(&sm.barQ, 1);
    tc::mbar_init(&sm.barS[0], 1);
    tc::mbar_init(&sm.barS[1], 1);
    tc::mbar_init(&sm.barD, 1);
    tc::mbar_init(&sm.barEnd, 1);
    tc::mbar_init(&sm.barDs, 256);
    tc::mbar_fence_init();
    if (n > 0) {  // the first loads at once
      tc::arrive_expect_tx(&sm.barQ, 2u * 2u * 128u * (uint32_t)(TT * G));
      for (int h = 0; h < 2; ++h) {
        tc::tma_load_3d(sm.q + h * (TILE / 2), &a.q, 64 * h, kh * G, sq.q0 + tok0, &sm.barQ);
        tc::tma_load_3d(sm.dO + h * (TILE / 2), &a.dO, 64 * h, kh * G, sq.q0 + tok0, &sm.barQ);
      }
      for (int t = 0; t < min(nt, Q_SLOTS); ++t) load(t);
    }
  }
  if (warp == 0) tc::alloc(&sm.tmem, 512);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tS = sm.tmem, tP = tS + 256, tQ = tS + 384;  // S of even and odd key tiles at 0 and 128
  tc::Wait w;

  if (warp == 9) {
    if (lane == 0 && n > 0) {
      for (int t = Q_SLOTS; t < nt && w.ok; ++t) {
        w.on(&sm.empty[t % Q_SLOTS], t / Q_SLOTS - 1);
        if (w.ok) load(t);
      }
      if (w.ok) {
        w.on(&sm.barQ, 0);
        for (int t = max(0, nt - Q_SLOTS); t < nt; ++t) w.on(&sm.full[t % Q_SLOTS], t / Q_SLOTS);
      } else {
        for (int k = 0; k < Q_SLOTS; ++k) tc::mbar_wait_sleep(&sm.full[k], 0, 4000000LL);
      }
    }
  } else if (warp == 8) {
    const uint32_t lead = tc::elect_leader();
    if (n > 0) {
      auto slot = [&](int t) { return smem_u32(sm.slot[t % Q_SLOTS]); };
      auto arrived = [&](int t) { w.warp_on(&sm.full[t % Q_SLOTS], t / Q_SLOTS); };
      auto release = [&](int t) {
        if (t + Q_SLOTS < nt) tc::commit_by(lead, &sm.empty[t % Q_SLOTS]);
      };
      auto scores = [&](int i) {
        arrived(2 * i);
        tc::gemm128_by<false>(lead, tS + 128 * (i & 1), smem_u32(sm.q), slot(2 * i), false);
        tc::commit_by(lead, &sm.barS[i & 1]);
      };
      auto dscores = [&](int i) {
        arrived(2 * i + 1);
        tc::gemm128_by<false>(lead, tP, smem_u32(sm.dO), slot(2 * i + 1), false);
        release(2 * i + 1);
        tc::commit_by(lead, &sm.barD);
      };
      w.warp_on(&sm.barQ, 0);
      scores(0);
      dscores(0);
      for (int i = 0; i < n; ++i) {
        if (i + 1 < n) scores(i + 1);  // (its buffer's last S was read before dS i - 1 was signalled)
        w.warp_on(&sm.barDs, i);
        tc::fence_after();
        tc::gemm_ts_by(lead, tQ, tP, slot(2 * i), i > 0);  // dQ += dS K
        release(2 * i);
        if (i + 1 < n) dscores(i + 1);
      }
      tc::commit_by(lead, &sm.barEnd);
    }
  } else {
    const int g0 = warp >> 2, r = 32 * (warp & 3) + lane;  // query row r, columns 64 g0 .. 64 g0 + 63
    const uint32_t lane_base = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t P = tP + lane_base + 64 * g0;
    const int tok = tok0 + r / G;
    const bool valid = r < TT * G && tok < sq.ql;
    const long row = ((long)sq.q0 + tok) * a.Hq + kh * G + r % G;
    const int lim = valid ? tok + off : -1;
    const float sc = a.scale * LOG2E;
    pdl_wait();  // (as dkv)
    pdl_release();
    const float lse = valid ? a.lse[row] * LOG2E : 0.f, delta = valid ? a.delta[row] : 0.f;
    for (int i = 0; i < n; ++i) {
      const int key0 = i * CH;
      const bool whole = key0 + CH - 1 <= lim;
      const uint32_t S = tS + 128 * (i & 1) + lane_base + 64 * g0;
      float p[64];
      w.warp_on(&sm.barS[i & 1], i >> 1);
      tc::fence_after();
      tc::ld64(S, p);
#pragma unroll
      for (int j = 0; j < 64; ++j) p[j] = ex2(p[j] * sc - lse);
      if (key0 + CH > sq.kl) {  // rows past the keys: whatever they hold, they count as zero
        const int t = 2 * i;
        w.warp_on(&sm.full[t % Q_SLOTS], t / Q_SLOTS);
        zero_rows(sm.slot[t % Q_SLOTS], sq.kl - key0, tid, 256);
        tc::fence_proxy_async();
      }
      w.warp_on(&sm.barD, i);
      tc::fence_after();
      float v[64];
      tc::ld64(P, v);
#pragma unroll
      for (int j = 0; j < 64; ++j) v[j] = p[j] * (v[j] - delta);
      if (!whole) {
#pragma unroll
        for (int j = 0; j < 64; ++j) v[j] = key0 + 64 * g0 + j <= lim ? v[j] : 0.f;
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) tc::st16_bf16(P + 16 * h, *reinterpret_cast<float(*)[32]>(v + 32 * h));
      tc::wait_st();
      tc::fence_before();
      tc::mbar_arrive(&sm.barDs);
    }
    if (n > 0) w.warp_on(&sm.barEnd, 0);
    tc::fence_after();
    const bool tile = tok0 + TT <= sq.ql;  // (as dkv: through Q's place)
#pragma unroll 1
    for (int h = 0; h < 2; ++h) {
      float v[32];
      if (n > 0) {
        tc::ld32(tQ + lane_base + 64 * g0 + 32 * h, v);
      } else {
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = 0.f;
      }
      if (tile)
        stage32(sm.q, r, 64 * g0 + 32 * h, v, a.scale);
      else if (valid)
        store32(a.dq + row * HD + 64 * g0 + 32 * h, v, a.scale);
      __syncwarp();
    }
    if (tile) {
      tc::fence_proxy_async();
      asm volatile("bar.sync 1, 256;" ::: "memory");
      if (tid == 0) store_tile(&a.mo, kh * G, sq.q0 + tok0, sm.q);
    }
    tc::fence_before();
  }
  if (!w.ok && a.status) atomicOr(a.status, 1);
  __syncthreads();
  tc::fence_after();
  if (warp == 0) tc::dealloc(sm.tmem, 512);
}

// Both in one launch: the dkv CTAs, whose longest ones are few and long, start
// first, and the dq CTAs fill the SMs beside and after them.
__global__ void __launch_bounds__(BWD_THREADS, 1) k_attn_bwd(const __grid_constant__ AttnArgs a, int kv_blocks) {
  extern __shared__ unsigned char raw[];
  if ((int)blockIdx.x < kv_blocks)
    dkv(a, raw, (int)blockIdx.x);
  else
    dq(a, raw, (int)blockIdx.x - kv_blocks);
  if (blockIdx.x == 0) pdl_wait();  // the grid ends after the one before it, whatever its CTAs had to do
}

}  // namespace

cudaError_t launch_attn_bwd(const AttnArgs& a, cudaStream_t s) {
  constexpr size_t smem = (sizeof(KvSmem) > sizeof(QSmem) ? sizeof(KvSmem) : sizeof(QSmem)) + 1024;
  static_assert(smem <= 227 * 1024, "shared memory");
  cudaError_t e = cudaFuncSetAttribute(k_attn_bwd, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  const int TT = CH / (a.Hq / a.Hk);
  const long rows = (long)a.total_q * a.Hq;
  const long early_rows = (long)a.n_seqs * EARLY * a.Hq;
  const int early = (int)((early_rows + 15) / 16 < EARLY_BLOCKS ? (early_rows + 15) / 16 : EARLY_BLOCKS);
  e = launch_pdl(k_attn_delta, dim3((unsigned)((rows + DELTA_ROWS - 1) / DELTA_ROWS + early)), dim3(256), 0, s, a, early);
  if (e != cudaSuccess) return e;
  const int kv = a.Hk * (a.total_k / CH + a.n_seqs), q = a.Hk * (a.total_q / TT + a.n_seqs);
  return launch_pdl(k_attn_bwd, dim3((unsigned)(kv + q)), dim3(BWD_THREADS), smem, s, a, kv);
}

}  // namespace gdn
