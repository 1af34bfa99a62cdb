// gdn_attn_bwd.cu -- backward of causal softmax attention over packed sequences.
//
// With p_ij = e^{scale q_i . k_j - lse_i} (recomputed), dp_ij = dO_i . v_j and
// delta_i = dO_i . o_i:
//     ds_ij = scale p_ij (dp_ij - delta_i),
//     dv_j = sum_i p_ij dO_i,   dk_j = sum_i ds_ij q_i,   dq_i = sum_j ds_ij k_j.
//
// Two kernels, so that every gradient is summed in one CTA, in a fixed order,
// without atomics (seven products per tile pair instead of five):
//   k_attn_dkv  one CTA per 128 keys and key head, over the query tiles that see
//               them: S^T = K Q^T, dP^T = V dO^T, dV += P^T dO, dK += dS^T Q.  A query
//               tile holds all heads of the group, so the sum over them is part
//               of the product.
//   k_attn_dq   one CTA per query tile, over the key tiles: S = Q K^T, dP = dO V^T,
//               dQ += dS K.
// Accumulators in tensor memory, P and dS as bf16 A operands there too (each
// half over the fp32 half that its own four warps have read).  Eight compute
// warps hold a tile, 64 columns to a thread.  While they form dS, the tensor
// cores run the next S; while they form P, the last gradient product.
//
// Bound: the tensor rate (7 x 512 cycles per pair of 128 x 128 tiles).
#include "gdn_attn.cuh"

namespace gdn {

namespace {

using namespace attn;

constexpr int BWD_THREADS = 256 + 64;
constexpr int KV_SLOTS = 4;  // Q, dO of two query tiles
constexpr int Q_SLOTS = 5;   // K, V of two key tiles and a half

// ---- delta_i = dO_i . o_i, one warp per row ----------------------------------------------
__global__ void __launch_bounds__(256) k_attn_delta(const __grid_constant__ AttnArgs a) {
  pdl_wait();
  pdl_release();
  const long rows = (long)a.total_q * a.Hq, row = (long)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (row >= rows) return;
  const uint2 x = *reinterpret_cast<const uint2*>(a.dOp + row * HD + 4 * lane);
  const uint2 y = *reinterpret_cast<const uint2*>(a.op + row * HD + 4 * lane);
  const float2 x0 = unpack_bf16(x.x), x1 = unpack_bf16(x.y), y0 = unpack_bf16(y.x), y1 = unpack_bf16(y.y);
  float d = x0.x * y0.x + x0.y * y0.y + x1.x * y1.x + x1.y * y1.y;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
  if (lane == 0) a.delta[row] = d;
}

// ---- dK, dV -------------------------------------------------------------------------
struct KvSmem {
  unsigned char k[TILE], v[TILE];
  unsigned char slot[KV_SLOTS][TILE];
  float lse[2][CH], delta[2][CH];
  int lim[2][CH];
  uint64_t full[KV_SLOTS], empty[KV_SLOTS];
  uint64_t barKV, barS, barD, barP, barDs, barEnd;
  uint32_t tmem;
};

__global__ void __launch_bounds__(BWD_THREADS, 1) k_attn_dkv(const __grid_constant__ AttnArgs a) {
  extern __shared__ unsigned char raw[];
  KvSmem& sm = *reinterpret_cast<KvSmem*>(raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u));
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_wait();
  pdl_release();
  const int G = a.Hq / a.Hk, TT = CH / G;
  const int kh = blockIdx.x % a.Hk;
  const int2 at = find_tile(a.cu_k, a.n_seqs, a.total_k, CH, (int)(blockIdx.x / a.Hk));
  if (at.x < 0) return;
  const Seq sq = seq_of(a, at.x);
  const int key0 = at.y * CH, off = sq.kl - sq.ql;
  if (key0 >= sq.kl) return;
  const int first = max(0, key0 - off) / TT;                 // first query tile that sees key0
  const int n = max(0, (sq.ql + TT - 1) / TT - first);

  if (tid == 0) {
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
  const int nt = 2 * n;

  if (warp == 9) {
    if (lane == 0 && n > 0) {
      tc::arrive_expect_tx(&sm.barKV, 2 * TILE);
      for (int h = 0; h < 2; ++h) {
        tc::tma_load_3d(sm.k + h * (TILE / 2), &a.k, 64 * h, kh, sq.k0 + key0, &sm.barKV);
        tc::tma_load_3d(sm.v + h * (TILE / 2), &a.v, 64 * h, kh, sq.k0 + key0, &sm.barKV);
      }
      for (int t = 0; t < nt && w.ok; ++t) {
        const int k = t % KV_SLOTS;
        if (t >= KV_SLOTS) w.on(&sm.empty[k], t / KV_SLOTS - 1);
        if (!w.ok) break;
        load_group(sm.slot[k], (t & 1) ? &a.dO : &a.q, kh, G, sq.q0 + (first + t / 2) * TT, &sm.full[k]);
      }
      if (w.ok) {
        w.on(&sm.barKV, 0);
        for (int t = max(0, nt - KV_SLOTS); t < nt; ++t) w.on(&sm.full[t % KV_SLOTS], t / KV_SLOTS);
      } else {
        for (int k = 0; k < KV_SLOTS; ++k) tc::mbar_wait_sleep(&sm.full[k], 0, 4000000LL);
      }
    }
  } else if (warp == 8) {
    if (lane == 0 && n > 0) {
      auto slot = [&](int t) { return smem_u32(sm.slot[t % KV_SLOTS]); };
      auto arrived = [&](int t) { w.on(&sm.full[t % KV_SLOTS], t / KV_SLOTS); };
      auto release = [&](int t) {
        if (t + KV_SLOTS < nt) tc::commit(&sm.empty[t % KV_SLOTS]);
      };
      auto scores = [&](int i) {
        arrived(2 * i);
        tc::gemm128(tS, smem_u32(sm.k), false, slot(2 * i), false, false);
        tc::commit(&sm.barS);
      };
      auto dscores = [&](int i) {
        arrived(2 * i + 1);
        tc::gemm128(tP, smem_u32(sm.v), false, slot(2 * i + 1), false, false);
        tc::commit(&sm.barD);
      };
      w.on(&sm.barKV, 0);
      scores(0);
      dscores(0);
      for (int i = 0; i < n; ++i) {
        w.on(&sm.barP, i);
        tc::fence_after();
        gemm_ts_halves(tV, tS, slot(2 * i + 1), i > 0);  // dV += P^T dO
        if (i + 1 < n) scores(i + 1);
        w.on(&sm.barDs, i);
        tc::fence_after();
        gemm_ts_halves(tK, tP, slot(2 * i), i > 0);      // dK += dS^T Q
        release(2 * i);
        release(2 * i + 1);
        if (i + 1 < n) dscores(i + 1);
      }
      tc::commit(&sm.barEnd);
    }
  } else {
    const int g0 = warp >> 2, r = 32 * (warp & 3) + lane;  // key row r, columns 64 g0 .. 64 g0 + 63
    const uint32_t lane_base = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t S = tS + lane_base + 64 * g0, P = tP + lane_base + 64 * g0;
    const int key = key0 + r;
    const float sc = a.scale * LOG2E;
    // what a query row needs: the last key that it sees, lse (base 2), delta
    auto load_cols = [&](int i) {
      if (tid < CH) {
        const int tok = (first + i) * TT + tid / G;
        const bool ok = tid < TT * G && tok < sq.ql;
        const long row = ((long)sq.q0 + tok) * a.Hq + kh * G + tid % G;
        sm.lim[i & 1][tid] = ok ? tok + off : -1;
        sm.lse[i & 1][tid] = ok ? a.lse[row] * LOG2E : 0.f;
        sm.delta[i & 1][tid] = ok ? a.delta[row] : 0.f;
      }
    };
    if (n > 0) load_cols(0);
    asm volatile("bar.sync 1, 256;" ::: "memory");
    for (int i = 0; i < n; ++i) {
      if (i + 1 < n) load_cols(i + 1);
      const int b = i & 1;
      const int tok0 = (first + i) * TT, live = min(sq.ql - tok0, TT) * G;  // rows of tokens that exist
      const bool whole = live == CH && key0 + CH - 1 <= tok0 + off;         // every row sees every key
      float p[64];
      w.warp_on(&sm.barS, i);
      tc::fence_after();
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float(&v)[32] = *reinterpret_cast<float(*)[32]>(p + 32 * h);
        tc::ld32(S + 32 * h, v);
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          const int c = 64 * g0 + 32 * h + j;
          const float e = ex2(v[j] * sc - sm.lse[b][c]);
          v[j] = whole || key <= sm.lim[b][c] ? e : 0.f;
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
      w.warp_on(&sm.barD, i);
      tc::fence_after();
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float v[32];
        tc::ld32(P + 32 * h, v);
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          const int c = 64 * g0 + 32 * h + j;
          const float q = p[32 * h + j];
          v[j] = whole || key <= sm.lim[b][c] ? q * (v[j] - sm.delta[b][c]) * a.scale : 0.f;
        }
        tc::st16_bf16(P + 16 * h, v);
      }
      tc::wait_st();
      tc::fence_before();
      tc::mbar_arrive(&sm.barDs);
      asm volatile("bar.sync 1, 256;" ::: "memory");  // the next tile's columns are in shared memory
    }
    if (n > 0) w.warp_on(&sm.barEnd, 0);
    tc::fence_after();
    const long row = ((long)sq.k0 + key) * a.Hk + kh;
#pragma unroll 1
    for (int h = 0; h < 4; ++h) {  // warps 0-3 write dV, 4-7 dK
      float v[32];
      if (n > 0) {
        tc::ld32((g0 ? tK : tV) + lane_base + 32 * h, v);
      } else {
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = 0.f;
      }
      if (key < sq.kl) store32((g0 ? a.dk : a.dv) + row * HD + 32 * h, v, 1.f);
      __syncwarp();
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
  uint64_t barQ, barS, barD, barDs, barEnd;
  uint32_t tmem;
};

__global__ void __launch_bounds__(BWD_THREADS, 1) k_attn_dq(const __grid_constant__ AttnArgs a) {
  extern __shared__ unsigned char raw[];
  QSmem& sm = *reinterpret_cast<QSmem*>(raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u));
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_wait();
  pdl_release();
  const int G = a.Hq / a.Hk, TT = CH / G;
  // a sequence's last tiles, which see the most keys, start first
  const int kh = blockIdx.x % a.Hk;
  const int2 at = find_tile(a.cu_q, a.n_seqs, a.total_q, TT, (int)((gridDim.x - 1 - blockIdx.x) / a.Hk));
  if (at.x < 0) return;
  const Seq sq = seq_of(a, at.x);
  const int tok0 = at.y * TT, off = sq.kl - sq.ql;
  if (tok0 >= sq.ql) return;
  const int keys = max(0, min(sq.kl, min(tok0 + TT, sq.ql) + off));
  const int n = (keys + CH - 1) / CH;

  if (tid == 0) {
    for (int k = 0; k < Q_SLOTS; ++k) {
      tc::mbar_init(&sm.full[k], 1);
      tc::mbar_init(&sm.empty[k], 1);
    }
    tc::mbar_init(&sm.barQ, 1);
    tc::mbar_init(&sm.barS, 1);
    tc::mbar_init(&sm.barD, 1);
    tc::mbar_init(&sm.barEnd, 1);
    tc::mbar_init(&sm.barDs, 256);
    tc::mbar_fence_init();
  }
  if (warp == 0) tc::alloc(&sm.tmem, 512);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tS = sm.tmem, tP = tS + 256, tQ = tS + 384;  // S of even and odd key tiles at 0 and 128
  tc::Wait w;
  const int nt = 2 * n;

  if (warp == 9) {
    if (lane == 0 && n > 0) {
      tc::arrive_expect_tx(&sm.barQ, 2u * 2u * 128u * (uint32_t)(TT * G));
      for (int h = 0; h < 2; ++h) {
        tc::tma_load_3d(sm.q + h * (TILE / 2), &a.q, 64 * h, kh * G, sq.q0 + tok0, &sm.barQ);
        tc::tma_load_3d(sm.dO + h * (TILE / 2), &a.dO, 64 * h, kh * G, sq.q0 + tok0, &sm.barQ);
      }
      for (int t = 0; t < nt && w.ok; ++t) {
        const int k = t % Q_SLOTS;
        if (t >= Q_SLOTS) w.on(&sm.empty[k], t / Q_SLOTS - 1);
        if (!w.ok) break;
        load_rows(sm.slot[k], (t & 1) ? &a.v : &a.k, kh, sq.k0 + (t / 2) * CH, &sm.full[k]);
      }
      if (w.ok) {
        w.on(&sm.barQ, 0);
        for (int t = max(0, nt - Q_SLOTS); t < nt; ++t) w.on(&sm.full[t % Q_SLOTS], t / Q_SLOTS);
      } else {
        for (int k = 0; k < Q_SLOTS; ++k) tc::mbar_wait_sleep(&sm.full[k], 0, 4000000LL);
      }
    }
  } else if (warp == 8) {
    if (lane == 0 && n > 0) {
      auto slot = [&](int t) { return smem_u32(sm.slot[t % Q_SLOTS]); };
      auto arrived = [&](int t) { w.on(&sm.full[t % Q_SLOTS], t / Q_SLOTS); };
      auto release = [&](int t) {
        if (t + Q_SLOTS < nt) tc::commit(&sm.empty[t % Q_SLOTS]);
      };
      auto scores = [&](int i) {
        arrived(2 * i);
        tc::gemm128(tS + 128 * (i & 1), smem_u32(sm.q), false, slot(2 * i), false, false);
        tc::commit(&sm.barS);
      };
      auto dscores = [&](int i) {
        arrived(2 * i + 1);
        tc::gemm128(tP, smem_u32(sm.dO), false, slot(2 * i + 1), false, false);
        release(2 * i + 1);
        tc::commit(&sm.barD);
      };
      w.on(&sm.barQ, 0);
      scores(0);
      dscores(0);
      for (int i = 0; i < n; ++i) {
        if (i + 1 < n) scores(i + 1);  // (its buffer's last S was read before dS i - 1 was signalled)
        w.on(&sm.barDs, i);
        tc::fence_after();
        gemm_ts_halves(tQ, tP, slot(2 * i), i > 0);  // dQ += dS K
        release(2 * i);
        if (i + 1 < n) dscores(i + 1);
      }
      tc::commit(&sm.barEnd);
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
    const float lse = valid ? a.lse[row] * LOG2E : 0.f, delta = valid ? a.delta[row] : 0.f;
    for (int i = 0; i < n; ++i) {
      const int key0 = i * CH;
      const bool whole = key0 + CH - 1 <= lim;
      const uint32_t S = tS + 128 * (i & 1) + lane_base + 64 * g0;
      float p[64];
      w.warp_on(&sm.barS, i);
      tc::fence_after();
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float(&v)[32] = *reinterpret_cast<float(*)[32]>(p + 32 * h);
        tc::ld32(S + 32 * h, v);
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = ex2(v[j] * sc - lse);
      }
      if (key0 + CH > sq.kl) {  // rows past the keys: whatever they hold, they count as zero
        const int t = 2 * i;
        w.warp_on(&sm.full[t % Q_SLOTS], t / Q_SLOTS);
        zero_rows(sm.slot[t % Q_SLOTS], sq.kl - key0, tid, 256);
        tc::fence_proxy_async();
      }
      w.warp_on(&sm.barD, i);
      tc::fence_after();
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float v[32];
        tc::ld32(P + 32 * h, v);
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          const float d = p[32 * h + j] * (v[j] - delta) * a.scale;
          v[j] = whole || key0 + 64 * g0 + 32 * h + j <= lim ? d : 0.f;
        }
        tc::st16_bf16(P + 16 * h, v);
      }
      tc::wait_st();
      tc::fence_before();
      tc::mbar_arrive(&sm.barDs);
    }
    if (n > 0) w.warp_on(&sm.barEnd, 0);
    tc::fence_after();
#pragma unroll 1
    for (int h = 0; h < 2; ++h) {
      float v[32];
      if (n > 0) {
        tc::ld32(tQ + lane_base + 64 * g0 + 32 * h, v);
      } else {
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = 0.f;
      }
      if (valid) store32(a.dq + row * HD + 64 * g0 + 32 * h, v, 1.f);
      __syncwarp();
    }
    tc::fence_before();
  }
  if (!w.ok && a.status) atomicOr(a.status, 1);
  __syncthreads();
  tc::fence_after();
  if (warp == 0) tc::dealloc(sm.tmem, 512);
}

template <typename K>
cudaError_t set_smem(K k, size_t bytes) {
  return cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

}  // namespace

cudaError_t launch_attn_bwd(const AttnArgs& a, cudaStream_t s) {
  constexpr size_t kv = sizeof(KvSmem) + 1024, qs = sizeof(QSmem) + 1024;
  static_assert(kv <= 227 * 1024 && qs <= 227 * 1024, "shared memory");
  cudaError_t e = set_smem(k_attn_dkv, kv);
  if (e == cudaSuccess) e = set_smem(k_attn_dq, qs);
  if (e != cudaSuccess) return e;
  const int TT = CH / (a.Hq / a.Hk);
  const long rows = (long)a.total_q * a.Hq;
  e = launch_pdl(k_attn_delta, dim3((unsigned)((rows + 7) / 8)), dim3(256), 0, s, a);
  if (e != cudaSuccess) return e;
  e = launch_pdl(k_attn_dkv, dim3((unsigned)a.Hk * (unsigned)(a.total_k / CH + a.n_seqs)), dim3(BWD_THREADS), kv, s, a);
  if (e != cudaSuccess) return e;
  return launch_pdl(k_attn_dq, dim3((unsigned)a.Hk * (unsigned)(a.total_q / TT + a.n_seqs)), dim3(BWD_THREADS), qs, s, a);
}

}  // namespace gdn
