// gdn_decay.cu -- linear attention with a decay for each head, over packed
// sequences: S_t = e^w S_{t-1} + k_t v_t^T, o_t = S_t^T q_t, forward and backward.
//
// One operation does all of it.  With rows a, b, c of 128 values and a state X,
//     out_t = sum_{s <= t} e^{w (t - s)} (a_t . b_s) c_s + (decayed X0)^T a_t,
// the forward is (a, b, c) = (q, k, v) with X0 = h0, and the gradients are
//     dq:  (dO, v, k),  X0 = h0^T,   forwards in time,
//     dv:  (k, q, dO),  X0 = dhT,    backwards in time (s >= t),
//     dk:  (v, dO, q),  X0 = dhT^T,  backwards in time;
// the state that the dv pass ends with is dh0.  dq and dk of a key head are sums
// over its value heads.
//
// Chunks of 128 tokens (n valid in a sequence's last one), rows i and columns j
// of a chunk, per chunk:
//     out = diag(f) A X + ((A B^T) o M) C,    X <- e^{w n} X + B^T diag(e) C
//   forwards:  M_ij = e^{w (i - j)}, j <= i;  f_i = e^{w (i + 1)};  e_j = e^{w (n - 1 - j)}
//   backwards: M_ij = e^{w (j - i)}, j >= i;  f_i = e^{w (n - 1 - i)};  e_j = e^{w (j + 1)}
// (every exponent that is used is <= 0, so nothing overflows for any w <= 0).
//
// k_decay, one CTA per (pass, sequence, head, segment): five tcgen05 products of
// 128^3 per chunk (P = A B^T, O1 = A X, O2 = P C, and two for X), accumulators in
// tensor memory (P, O1, O2, X: 4 x 128 columns).  X stays there in fp32 for the whole
// segment; it is scaled there once a chunk and rounded to bf16 only as the operand of
// A X.  B^T diag(e) C has to keep the state's fp32: the rows of B are scaled in fp32
// and split into two bf16 terms, a product each.  The masked P goes back to tensor
// memory as a bf16 A operand.  Warps 0-7 mask P and write the output, 8-15 carry the
// state and scale B, one warp issues the products, one the loads (a ring of five
// 32 KiB tiles, three to a chunk), one the stores.  So an output element has three
// roundings to bf16: of P or X as an operand, twice, and its own (its error against 64
// bits is 2.3e-3 in the 2-norm, where rounding alone gives 1.7e-3).
//
// With few sequences and heads the SMs are filled by segments: k_decay_fold
// forms each segment's own X (rows weighted to the segment's end, so that its
// chunks accumulate in tensor memory without a rescale), k_decay_prefix turns
// them into entering states, and k_decay starts every segment from its own.  With
// one segment to a sequence the fold forms the final states, beside the walk (in a
// launch of its own, or, in short calls, in the walk's: k_decay_small).
//
// Bound: shared memory.  A product whose operands both lie there reads 64 KiB in the
// 512 cycles that it takes, all of an SM's 128 bytes per cycle; with the loads, the
// scaled rows, X's image and the staged output a chunk of the walk moves 576 KiB,
// 4600 cycles, and takes 4800 to 5800 (2.4 to 2.9 us); the fold's 2300 (two terms) take
// 2600, its 3100 where a final state needs three about 3050.  Measured on a GB300, 16 key and
// 32 value heads: 65536 tokens in 504 to 520 us (fold 177, prefix 10, walk 316; the bytes
// alone 238), 4096 tokens in 50 us (21, 7, 35, partly overlapped; 15); forward and backward of
// 4096 + 2500 + 1000 + 595 + 1 packed tokens in 280 us (walks 94 and 159, the longest
// sequence's 32 chunks deciding the first one; the bytes alone 87).
#include "gdn_kernels.cuh"
#include "gdn_tc05.cuh"

namespace gdn {

namespace {

constexpr uint32_t TILE = CH * HD * 2;  // a [128 x 128] bf16 tile
constexpr int WALK_THREADS = 16 * 32 + 96;
constexpr int FOLD_SLOTS = 5;
constexpr int FOLD_TERMS = 3;
constexpr int FOLD_THREADS = 256 + 64;

struct Range {
  int start, len;
};
// sequence s of the packed rows (cu null: equal lengths), held inside [0, total]
__device__ __forceinline__ Range seq_range(const int* cu, int s, int T, int total) {
  Range r;
  if (cu) {
    const int a = min(max(cu[s], 0), total), b = min(max(cu[s + 1], a), total);
    r.start = a;
    r.len = b - a;
  } else {
    r.start = s * T;
    r.len = T;
  }
  return r;
}

// A head's log-decay: minus infinity (nothing is kept) as a number, so that it times a
// distance of zero is zero.
__device__ __forceinline__ float log_decay(const float* decay, int j) {
  const float w = decay[j];
  return w == -INFINITY ? -1e30f : w;
}

// Segment slots.  Sequence s has the slots first_slot(s) .. first_slot(s + 1) - 1,
// at least as many as it has segments of K = 128 seg_chunks tokens and at most
// one more than total / K over all sequences together, so that neither grids
// nor states grow with sequences x longest sequence.
__device__ __forceinline__ int first_slot(const int* cu, int s, int T, int total, int K) {
  return (cu ? min(max(cu[s], 0), total) : s * T) / K + s;
}
// Sequence and segment of a slot, found by every warp for itself (sequence -1:
// none).  With one segment to a sequence a slot is a sequence, the longest first
// (of 32 at most: CTAs start in order of slots, and the long ones decide when a
// call ends).
__device__ __forceinline__ int2 find_segment(const int* cu, int n_seqs, int T, int total, int seg_chunks, int nseg,
                                             int slot) {
  const int K = seg_chunks * CH, lane = threadIdx.x & 31;
  if (nseg == 1) {
    if (n_seqs == 1 || n_seqs > 32 || !cu) return make_int2(slot, 0);
    const int len = seq_range(cu, min(lane, n_seqs - 1), T, total).len;
    int longer = 0;
    for (int k = 0; k < n_seqs; ++k) {
      const int l = __shfl_sync(0xffffffffu, len, k);
      longer += l > len || (l == len && k < lane);
    }
    return make_int2(__ffs((int)__ballot_sync(0xffffffffu, lane < n_seqs && longer == slot)) - 1, 0);
  }
  for (int s0 = 0; s0 < n_seqs; s0 += 32) {
    const int s = min(s0 + lane, n_seqs - 1), a = first_slot(cu, s, T, total, K);
    const unsigned m = __ballot_sync(0xffffffffu, slot >= a && slot < first_slot(cu, s + 1, T, total, K));
    if (m) {
      const int l = __ffs((int)m) - 1;
      return make_int2(min(s0 + l, n_seqs - 1), slot - __shfl_sync(0xffffffffu, a, l));
    }
  }
  return make_int2(-1, 0);
}

// The states of segments lie in the workspace so that lanes with consecutive rows
// touch consecutive addresses: float4 (row r, columns 4 g .. 4 g + 3) at g * 128 + r.
__device__ __forceinline__ int seg_index(int r, int c) { return ((c >> 2) * HD + r) * 4 + (c & 3); }

// Row r of an SW128 tile scaled by f and split into TERMS bf16 terms, 16-byte chunks
// j .. j + 3: term 0 in place, the others to the same place of the tiles at `rest`.
// The leading terms are the value's upper 16 bits as they stand (the
// remainder is then exact), the last one is rounded: 8 bits more of the fp32
// product per term, at a permute, two ands and half a multiply-add per pair.  A
// row that is not `valid` (past the sequence's end) becomes zero, whatever it holds.
template <int TERMS>
__device__ __forceinline__ void scale_row(unsigned char* tile, unsigned char* rest, int r, int j, float f, bool valid) {
  uint4 u[4];  // all loads in flight at once
#pragma unroll
  for (int c = 0; c < 4; ++c) u[c] = *reinterpret_cast<const uint4*>(tile + tc::sw128_chunk(r, j + c, CH));
  if (!valid) {
#pragma unroll
    for (int c = 0; c < 4; ++c) u[c] = make_uint4(0u, 0u, 0u, 0u);
  }
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const uint32_t up[4] = {u[c].x, u[c].y, u[c].z, u[c].w};
    uint32_t o[TERMS][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float x = __uint_as_float(up[i] << 16), y = __uint_as_float(up[i] & 0xffff0000u);
      tc::mul2(x, y, f, f);
#pragma unroll
      for (int t = 0; t < TERMS - 1; ++t) {
        o[t][i] = __byte_perm(__float_as_uint(x), __float_as_uint(y), 0x7632);
        float hx = __uint_as_float(__float_as_uint(x) & 0xffff0000u);
        float hy = __uint_as_float(__float_as_uint(y) & 0xffff0000u);
        tc::axpy2(hx, hy, -1.f, x, y);
        x = hx;
        y = hy;
      }
      o[TERMS - 1][i] = pack_bf16(x, y);
    }
    const uint32_t at = tc::sw128_chunk(r, j + c, CH);
#pragma unroll
    for (int t = 0; t < TERMS; ++t)
      *reinterpret_cast<uint4*>((t == 0 ? tile : rest + (t - 1) * TILE) + at) =
          make_uint4(o[t][0], o[t][1], o[t][2], o[t][3]);
  }
}
__device__ __forceinline__ void zero_row(unsigned char* tile, int r, int j0, int nj) {
  for (int j = j0; j < j0 + nj; ++j)
    *reinterpret_cast<uint4*>(tile + tc::sw128_chunk(r, j, CH)) = make_uint4(0u, 0u, 0u, 0u);
}

__device__ __forceinline__ void load_tile(unsigned char* dst, const CUtensorMap* m, int head, int row, uint64_t* bar) {
  tc::arrive_expect_tx(bar, TILE);
  tc::tma_load_3d(dst, m, 0, head, row, bar);
  tc::tma_load_3d(dst + TILE / 2, m, 64, head, row, bar);
}

// ---- the chunk walk ----------------------------------------------------------------
// B' = diag(e) B enters X += B'^T C in two bf16 terms, which leave an error of some
// 1e-5 in the state, far below the rounding of the output's operands (a final
// state that is returned in fp32 comes from k_decay_fold, in three).
constexpr int NSLOT = 5;
struct WalkSmem {
  unsigned char slot[NSLOT][TILE];
  unsigned char lo[TILE];               // second term of the scaled B rows (the first one in place)
  unsigned char X[TILE];                // the entering state in bf16, [128 (b) rows x 128 (c)]
  alignas(16) float tab[CH];            // e^{w d}
  alignas(16) float col[2][32];         // e^{w (31 - d)}, e^{-w d}
  uint64_t full[NSLOT], empty[NSLOT];
  // barSt: of even and odd chunks.  The storing thread may be a chunk behind the
  // writers; the slot that it frees keeps them from getting two ahead.
  uint64_t barP, barPm, barK[2], barS, barX, barO, barOf, barSt[2];
  uint32_t tmem;
};

// Row r, columns c0 .. c0 + 31 of the state that the walk begins with, by the state's
// 256 threads together (c0 of a thread: its half's 0 or 32).  Rows of a caller's
// state go through shared memory (`stage`, 32 KiB), so that a warp reads whole
// lines of it.
__device__ __forceinline__ void first_state(const DecayRole& R, unsigned char* stage, const float* x0, int r, int c0,
                                            float (&v)[32]) {
  if (!x0) {
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = 0.f;
  } else if (R.xseg && !R.xt) {
#pragma unroll
    for (int i = 0; i < 32; i += 4) {
      const float4 f = *reinterpret_cast<const float4*>(x0 + seg_index(r, c0 + i));
      v[i] = f.x;
      v[i + 1] = f.y;
      v[i + 2] = f.z;
      v[i + 3] = f.w;
    }
  } else if (R.xt) {
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = x0[R.xseg ? seg_index(c0 + i, r) : (c0 + i) * HD + r];
  } else {
    // columns c, c + 64 of the pass (c = 0 .. 31, or 32 .. 63): 128 rows x 2 x 128 bytes
    const int t = threadIdx.x & 255, cc = c0 & 63;
    asm volatile("bar.sync 2, 256;" ::: "memory");  // (the pass before has been read)
    float4 f[8];
#pragma unroll
    for (int l = 0; l < 8; ++l) {
      const int i = t + 256 * l, row = i >> 4, p = i & 15;  // 16-byte piece p of the row's two
      f[l] = *reinterpret_cast<const float4*>(x0 + row * HD + (p >> 3) * 64 + cc + 4 * (p & 7));
    }
#pragma unroll
    for (int l = 0; l < 8; ++l) {
      const int i = t + 256 * l, row = i >> 4, p = i & 15;
      *reinterpret_cast<float4*>(stage + row * 256 + ((p ^ (row & 7)) << 4)) = f[l];
    }
    asm volatile("bar.sync 2, 256;" ::: "memory");
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int p = 8 * (c0 >> 6) + k;
      const float4 x = *reinterpret_cast<const float4*>(stage + r * 256 + ((p ^ (r & 7)) << 4));
      v[4 * k] = x.x;
      v[4 * k + 1] = x.y;
      v[4 * k + 2] = x.z;
      v[4 * k + 3] = x.w;
    }
  }
}

// Waits (bounded, by a whole warp) until the flag is `value` or more and what was
// written before it can be read.  Where a wait of the warp has given up before (lane 0's
// `ok` says so), at once, so that a walk without its flags ends within one limit, not one to a chunk.
__device__ __forceinline__ bool wait_flag(const int* flag, int value, bool ok) {
  if (ok && (threadIdx.x & 31) == 0) {
    const long long t0 = clock64();
    for (int v = 0;;) {
      asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(flag) : "memory");
      if (v >= value) break;
      if (clock64() - t0 > tc::WAIT_LIMIT_CYCLES) {
        ok = false;
        break;
      }
      __nanosleep(100);
    }
  }
  __syncwarp();  // (lane 0's acquire holds for the other lanes' reads; a shuffle orders none)
  return __shfl_sync(0xffffffffu, (int)ok, 0) != 0;
}

// One CTA's walk over the chunks [cb, ce) of head hd in sequence s (rows q); REV: backwards.
template <bool SUM, bool REV>
__device__ __forceinline__ void walk(const DecayArgs& a, const DecayRole& R, WalkSmem& sm, const Range q, int s,
                                     int slot_id, int hd, int cb, int ce) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tc::warp_index();
  const int n_it = ce - cb, G = a.Hv / a.Hk, kh = hd / G;
  const int g = hd - kh * G, ho = R.shared ? kh : hd;  // place in the group, output head
  auto chunk_of = [&](int it) { return REV ? ce - 1 - it : cb + it; };
  auto rows_of = [&](int c) { return min(CH, q.len - c * CH); };

  auto load = [&](int t) {  // tile t (a, b, c of every chunk) into its slot
    const int kind = t % 3, row = q.start + chunk_of(t / 3) * CH;
    const CUtensorMap* m = kind == 0 ? &R.a : kind == 1 ? &R.b : &R.c;
    const int per_v = kind == 0 ? R.ha : kind == 1 ? R.hb : R.hc;
    load_tile(sm.slot[t % NSLOT], m, per_v ? hd : kh, row, &sm.full[t % NSLOT]);
  };
  const int nt = 3 * n_it;
  const float* x0 = R.xseg ? R.xseg + ((long)slot_id * a.Hv + hd) * HD * HD
                           : (R.x0 ? R.x0 + ((long)s * a.Hv + hd) * HD * HD : nullptr);
  if (!R.xseg && x0 && tid < HD * HD / 32)  // on its way to L2 while the CTA sets up
    asm volatile("prefetch.global.L2 [%0];" ::"l"(x0 + 32 * tid));
  if (warp == 17 && lane == 0) {
    for (int k = 0; k < NSLOT; ++k) {
      tc::mbar_init(&sm.full[k], 1);
      tc::mbar_init(&sm.empty[k], 1);
    }
    tc::mbar_init(&sm.barP, 1);
    tc::mbar_init(&sm.barX, 1);
    tc::mbar_init(&sm.barO, 1);
    tc::mbar_init(&sm.barPm, 256);
    tc::mbar_init(&sm.barK[0], 256);
    tc::mbar_init(&sm.barK[1], 256);
    tc::mbar_init(&sm.barS, 256);
    tc::mbar_init(&sm.barOf, 256);
    tc::mbar_init(&sm.barSt[0], 256);
    tc::mbar_init(&sm.barSt[1], 256);
    tc::mbar_fence_init();
    // The first tiles are requested at once.  After the prefix kernel q, k, v and dO
    // are complete already: it starts no dependent before its own wait is over,
    // and that is for the fold, which read them.
    for (int t = 0; t < min(nt, NSLOT); ++t) load(t);
  }
  if (warp == 0) tc::alloc(&sm.tmem, 512);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tP = sm.tmem, tO1 = tP + 128, tO2 = tP + 256, tX = tP + 384;
  tc::Wait w;

  // whether chunk `it`'s output rows are stored as a tile: a whole chunk, of the last head summed
  auto flag_of = [&](int c) {
    return R.flags + (long)kh * (a.total / CH + a.n_seqs) + first_slot(a.cu, s, a.T, a.total, CH) + c;
  };
  const bool adds = SUM && R.shared && g > 0, last = !SUM || !R.shared || g == G - 1;
  auto whole = [&](int it) { return last && rows_of(chunk_of(it)) == CH; };

  if (warp == 18) {  // ---- output tiles: staged in the slot of the chunk's C, which O has consumed
    if (lane == 0) {
      for (int it = 0; it < n_it && w.ok; ++it) {
        const int t = 3 * it + 2;
        w.on(&sm.barSt[it & 1], it >> 1);
        if (!w.ok) break;
        if (whole(it)) {
          const unsigned char* tile = sm.slot[t % NSLOT];
          const int row = q.start + chunk_of(it) * CH;
          tc::tma_store_3d(&R.o, 0, ho, row, tile);
          tc::tma_store_3d(&R.o, 64, ho, row, tile + TILE / 2);
          tc::bulk_commit();
          tc::bulk_wait_read();
        }
        if (t + NSLOT < 3 * n_it) tc::mbar_arrive(&sm.empty[t % NSLOT]);
        // the chunk's sums are in memory: the flag says so to the next head's CTA (from
        // here, where the wait for the writes holds up nobody else)
        if (!last)
          asm volatile("st.release.gpu.global.s32 [%0], %1;" ::"l"(flag_of(chunk_of(it))), "r"(g + 1) : "memory");
      }
      tc::bulk_wait();
    }
  } else if (warp == 17) {  // ---- TMA: tiles a, b, c of every chunk, in the order consumed
    if (lane == 0) {
      for (int t = NSLOT; t < nt && w.ok; ++t) {
        w.on(&sm.empty[t % NSLOT], t / NSLOT - 1);
        if (w.ok) load(t);
      }
      // no copy is in flight when the CTA ends
      if (w.ok)
        for (int t = max(0, nt - NSLOT); t < nt; ++t) w.on(&sm.full[t % NSLOT], t / NSLOT);
      else
        for (int k = 0; k < NSLOT; ++k) tc::mbar_wait_sleep(&sm.full[k], 0, 4000000LL);
    }
  } else if (warp == 16) {  // ---- products
    const uint32_t lead = tc::elect_leader();
    auto slot = [&](int t) { return smem_u32(sm.slot[t % NSLOT]); };
    auto arrived = [&](int t) { w.warp_on(&sm.full[t % NSLOT], t / NSLOT); };
    auto release = [&](int t) {
      if (t + NSLOT < nt) tc::commit_by(lead, &sm.empty[t % NSLOT]);
    };
    auto scores = [&](int it) {  // P = A B^T
      arrived(3 * it);
      arrived(3 * it + 1);
      tc::gemm128_by<false>(lead, tP, slot(3 * it), slot(3 * it + 1), false);
      tc::commit_by(lead, &sm.barP);
    };
    scores(0);
    for (int it = 0; it < n_it; ++it) {
      const int ta = 3 * it, tb = ta + 1, tcc = ta + 2;
      w.warp_on(&sm.barS, it);
      if (it > 0) w.warp_on(&sm.barOf, it - 1);
      tc::fence_after();
      tc::gemm128_by<true>(lead, tO1, slot(ta), smem_u32(sm.X), false);  // A X
      release(ta);
      arrived(tcc);
#pragma unroll
      for (int h = 0; h < 2; ++h) {  // X += B'^T C, 64 tokens at a time
        w.warp_on(&sm.barK[h], it);
        tc::fence_after();
        const uint32_t c = slot(tcc) + 8192 * h;
        tc::gemm_rows_by<64>(lead, tX, slot(tb) + 8192 * h, c, true);
        tc::gemm_rows_by<64>(lead, tX, smem_u32(sm.lo) + 8192 * h, c, true);
      }
      tc::commit_by(lead, &sm.barX);
      release(tb);
      w.warp_on(&sm.barPm, it);
      tc::fence_after();
      tc::gemm_ts_by(lead, tO2, tP, slot(tcc), false);  // P C
      tc::commit_by(lead, &sm.barO);
      if (it + 1 < n_it) scores(it + 1);
    }
  } else {
    // Eight warps for the scores and the output, eight for the state and the scaled
    // rows: thread (r, half) has row r = TMEM lane r and 64 of its 128 columns.
    const int half = (warp >> 2) & 1, r = 32 * (warp & 3) + lane;
    const uint32_t lane_base = (uint32_t)(32 * (warp & 3)) << 16, cols = lane_base + 64 * half;
    const float wd = log_decay(a.decay, hd);
    if (warp < 8) {
      const int own = warp & 3, Ho = R.shared ? a.Hk : a.Hv;
      // O of chunk `it`, whose products have been issued
      auto output = [&](int it) {
        const int c = chunk_of(it), n = rows_of(c);
        const float f = expf(wd * (float)(REV ? max(n - 1 - r, 0) : r + 1));
        const bool tile = whole(it);
        const long row = (long)q.start + (long)c * CH + r;
        bf16* dst = R.out + (row * Ho + ho) * HD + 64 * half;
        unsigned char* staged = sm.slot[(3 * it + 2) % NSLOT];
        auto put = [&](int j, const float* x) {  // columns 8 j .. 8 j + 7 of the half
          const uint4 o = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]),
                                     pack_bf16(x[6], x[7]));
          if (tile)
            *reinterpret_cast<uint4*>(staged + tc::sw128_chunk(r, 8 * half + j, CH)) = o;
          else if (r < n)
            *reinterpret_cast<uint4*>(dst + 8 * j) = o;
        };
        if constexpr (!SUM) {
          w.warp_on(&sm.barO, it);
          tc::fence_after();
#pragma unroll 1
          for (int g = 0; g < 2; ++g) {
            float x[32], y[32];
            tc::ld32(tO1 + cols + 32 * g, x);
            tc::ld32(tO2 + cols + 32 * g, y);
            if (g == 1) {
              tc::fence_before();
              tc::mbar_arrive(&sm.barOf);
            }
#pragma unroll
            for (int i = 0; i < 32; i += 2) tc::axpy2(x[i], x[i + 1], f, y[i], y[i + 1]);
#pragma unroll
            for (int i = 0; i < 4; ++i) put(4 * g + i, x + 8 * i);
            __syncwarp();
          }
        } else {
          // The sum over the value heads runs from CTA to CTA, [head][4-column group][row]
          // in the workspace; a flag per chunk says how many heads are in it.
          const bool add = adds && r < n;
          float4* acc = reinterpret_cast<float4*>(R.acc) + ((long)kh * 32 + 16 * half) * a.total + row;
          if (adds) w.ok = wait_flag(flag_of(c), g, w.ok) && w.ok;
          float4 p[2][4];  // 32 columns of it are on their way at any time
          auto request = [&](int k) {
            if (add) {
#pragma unroll
              for (int i = 0; i < 4; ++i) p[k & 1][i] = acc[(long)(4 * k + i) * a.total];
            }
          };
          request(0);
          request(1);
          w.warp_on(&sm.barO, it);
          tc::fence_after();
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            float x[16], y[16];
            tc::ld16(tO1 + cols + 16 * k, x);
            tc::ld16(tO2 + cols + 16 * k, y);
            if (k == 3) {
              tc::fence_before();
              tc::mbar_arrive(&sm.barOf);
            }
#pragma unroll
            for (int i = 0; i < 16; i += 2) tc::axpy2(x[i], x[i + 1], f, y[i], y[i + 1]);
            if (add) {
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                x[4 * i] += p[k & 1][i].x;
                x[4 * i + 1] += p[k & 1][i].y;
                x[4 * i + 2] += p[k & 1][i].z;
                x[4 * i + 3] += p[k & 1][i].w;
              }
            }
            if (k < 2) request(k + 2);
            if (last) {
              put(2 * k, x);
              put(2 * k + 1, x + 8);
            } else if (r < n) {
#pragma unroll
              for (int i = 0; i < 4; ++i)
                acc[(long)(4 * k + i) * a.total] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
            }
            __syncwarp();
          }
        }
        tc::fence_proxy_async();
        tc::mbar_arrive(&sm.barSt[it & 1]);
      };
      if (half == 0) {
        sm.tab[r] = expf(wd * (float)r);
        if (r < 32) {
          sm.col[0][r] = expf(wd * (float)(31 - r));
          sm.col[1][r] = expf(-wd * (float)r);
        }
      }
      const bool mild = wd > -2.5f;  // (e^{-31 w} and e^{31 w} are normal fp32 numbers)
      asm volatile("bar.sync 1, 256;" ::: "memory");
      for (int it = 0; it < n_it; ++it) {
        if (it > 0) output(it - 1);
        const int n = rows_of(chunk_of(it));
        w.warp_on(&sm.barP, it);
        tc::fence_after();
        // Of the four 32 x 32 blocks of a warp's rows, those on the far side of the
        // diagonal are zero, those on the near side have the factor e^{w |i - j|} = (to
        // the block's edge) * (from the edge), both <= 1.  On the diagonal block it is
        // e^{w i} * e^{-w j} from the block's corner, unless one of them could leave fp32's
        // range.  The scores meet the finished factor only: they may be of any size.
#pragma unroll 1
        for (int h = 4 * half; h < 4 * half + 4; ++h) {  // 16 columns at a time
          const int g = h >> 1, j0 = 16 * h;
          float v[16];
          if (REV ? g < own : g > own) {
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = 0.f;
          } else {
            tc::ld16(tP + lane_base + j0, v);
            if (g != own || mild) {
              const float edge = REV ? (g == own ? sm.col[1][lane] : sm.tab[32 * g - r])
                                     : sm.tab[g == own ? lane : r - 32 * g - 31];
              const float* col = (REV ? sm.tab : sm.col[g == own]) + (j0 & 16);
#pragma unroll
              for (int i = 0; i < 16; i += 4) {
                float4 f = *reinterpret_cast<const float4*>(col + i);
                tc::mul2(f.x, f.y, edge, edge);  // (the factor first: it is at most 1, its parts may not be)
                tc::mul2(f.z, f.w, edge, edge);
                tc::mul2(v[i], v[i + 1], f.x, f.y);
                tc::mul2(v[i + 2], v[i + 3], f.z, f.w);
              }
            } else {
#pragma unroll
              for (int i = 0; i < 16; ++i) v[i] *= sm.tab[max(REV ? j0 + i - r : r - j0 - i, 0)];
            }
            if (g == own) {
              const int d0 = r - j0;  // column of the diagonal
#pragma unroll
              for (int i = 0; i < 16; ++i) v[i] = (REV ? i >= d0 : i <= d0) ? v[i] : 0.f;
            }
            if (REV && j0 + 16 > n) {  // (forwards, rows of tokens see tokens only)
#pragma unroll
              for (int i = 0; i < 16; ++i) v[i] = j0 + i < n ? v[i] : 0.f;
            }
          }
          tc::st8_bf16(tP + cols + 8 * (h & 3), v);  // (columns of this half that were read already)
        }
        tc::wait_st();
        tc::fence_before();
        tc::mbar_arrive(&sm.barPm);
      }
      output(n_it - 1);
    } else {
      if (a.nseg > 1) {  // the entering states come from the kernel before
        pdl_wait();
        pdl_release();
      }
#pragma unroll 1
      for (int k = 0; k < 2; ++k) {
        float v[32];
        first_state(R, sm.lo, x0, r, 64 * half + 32 * k, v);
        tc::st32(tX + cols + 32 * k, v);
      }
      tc::wait_st();
      asm volatile("bar.sync 2, 256;" ::: "memory");  // (the staged state has been read)
      for (int it = 0; it < n_it; ++it) {
        const int n = rows_of(chunk_of(it));
        const float keep = expf(wd * (float)n);
        // ---- the state: bf16 image of X, X <- e^{w n} X
        if (it > 0) {
          w.warp_on(&sm.barX, it - 1);
          tc::fence_after();
        }
#pragma unroll 1
        for (int g = 0; g < 2; ++g) {
          float v[32];
          tc::ld32(tX + cols + 32 * g, v);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint4 o;
            o.x = pack_bf16(v[8 * c], v[8 * c + 1]);
            o.y = pack_bf16(v[8 * c + 2], v[8 * c + 3]);
            o.z = pack_bf16(v[8 * c + 4], v[8 * c + 5]);
            o.w = pack_bf16(v[8 * c + 6], v[8 * c + 7]);
            *reinterpret_cast<uint4*>(sm.X + tc::sw128_chunk(r, 8 * half + 4 * g + c, CH)) = o;
          }
#pragma unroll
          for (int i = 0; i < 32; i += 2) tc::mul2(v[i], v[i + 1], keep, keep);
          tc::st32(tX + cols + 32 * g, v);
        }
        tc::wait_st();
        tc::fence_before();
        tc::fence_proxy_async();
        tc::mbar_arrive(&sm.barS);
        // ---- B' = diag(e) B in bf16 terms; rows past the sequence's end are cleared
        const int tb = 3 * it + 1, tcc = tb + 1;
        w.warp_on(&sm.full[tb % NSLOT], tb / NSLOT);
        if (n < CH) w.warp_on(&sm.full[tcc % NSLOT], tcc / NSLOT);
        w.warp_on(&sm.barP, it);  // (A B^T, which reads the raw tile, has completed)
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {  // 64 rows at a time, four threads to a row
          const int i = 64 * h + (tid & 63), j = 4 * ((tid >> 6) & 3);
          const float e = expf(wd * (float)(REV ? i + 1 : max(n - 1 - i, 0)));
          scale_row<2>(sm.slot[tb % NSLOT], sm.lo, i, j, e, i < n);
          if (i >= n) zero_row(sm.slot[tcc % NSLOT], i, j, 4);
          tc::fence_proxy_async();
          tc::mbar_arrive(&sm.barK[h]);
        }
      }
    }
  }
  if (!w.ok && a.status) atomicOr(a.status, 1);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (warp == 0) tc::dealloc(sm.tmem, 512);
}

// ---- segments and final states ----------------------------------------------------------------------
struct FoldSmem {
  unsigned char slot[FOLD_SLOTS][TILE];
  unsigned char rest[FOLD_TERMS - 1][TILE];  // further terms of the scaled B rows
  uint64_t full[FOLD_SLOTS], empty[FOLD_SLOTS];
  uint64_t barK[2], barM[2];
  uint32_t tmem;
};

// The first ten warps of a block: 0-7 scale, 8 issues the products, 9 loads.
__device__ __forceinline__ void fold_block(const DecayFoldArgs& a, const DecayFoldRole& R, FoldSmem& sm, int slot, int j) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tc::warp_index();
  const int G = a.Hv / a.Hk;
  const int2 at = find_segment(a.cu, a.n_seqs, a.T, a.total, a.seg_chunks, a.nseg, slot);
  const int s = at.x, seg = at.y;
  if (s < 0) return;
  const Range q = seq_range(a.cu, s, a.T, a.total);
  const int nch = (q.len + CH - 1) / CH;
  const int cb = seg * a.seg_chunks, ce = a.nseg == 1 ? nch : min(nch, cb + a.seg_chunks), nc = ce - cb;
  const long sh = (long)s * a.Hv + j;
  if (nc <= 0) {
    if (a.nseg == 1)  // an empty sequence ends in the state that it began with
#pragma unroll 4
      for (int i = 4 * tid; i < HD * HD; i += 4 * (int)blockDim.x)
        *reinterpret_cast<float4*>(R.last + sh * HD * HD + i) =
            R.x0 ? *reinterpret_cast<const float4*>(R.x0 + sh * HD * HD + i) : make_float4(0.f, 0.f, 0.f, 0.f);
    return;
  }
  // the segment that the walk ends with matters only for the final state
  if (!R.last && (R.rev ? cb == 0 : ce == nch)) return;
  const int end = min(q.len, ce * CH);  // one past the segment's last token

  // in the order of growing weights: the fp32 sums of the tensor cores lose a little of
  // whatever is added to a larger sum
  auto chunk_of = [&](int i) { return R.rev ? ce - 1 - i : cb + i; };
  auto load = [&](int t) {
    load_tile(sm.slot[t % FOLD_SLOTS], (t & 1) ? &R.c : &R.b, (t & 1) ? j : j / G, q.start + chunk_of(t / 2) * CH,
              &sm.full[t % FOLD_SLOTS]);
  };
  const int nt = 2 * nc;
  if (a.nseg == 1 && R.x0 && tid < HD * HD / 64) {  // on its way to L2 meanwhile
    asm volatile("prefetch.global.L2 [%0];" ::"l"(R.x0 + sh * HD * HD + 64 * tid));
    asm volatile("prefetch.global.L2 [%0];" ::"l"(R.x0 + sh * HD * HD + 64 * tid + 32));
  }
  if (warp == 9 && lane == 0) {
    for (int k = 0; k < FOLD_SLOTS; ++k) {
      tc::mbar_init(&sm.full[k], 1);
      tc::mbar_init(&sm.empty[k], 1);
    }
    for (int h = 0; h < 2; ++h) {
      tc::mbar_init(&sm.barK[h], 256);
      tc::mbar_init(&sm.barM[h], 1);
    }
    tc::mbar_fence_init();
    for (int t = 0; t < min(nt, FOLD_SLOTS); ++t) load(t);
  }
  if (warp == 0) tc::alloc(&sm.tmem, 512);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tX = sm.tmem;
  tc::Wait w;
  const float wd = log_decay(a.decay, j);
  // The rows' third terms (2^-17 of their size) are for the final state alone.  All of its
  // chunks have them: an old one's may be all that is left in it, where newer rows are zero.
  const bool third = R.last;
  if (warp == 9) {
    if (lane == 0) {
      for (int t = FOLD_SLOTS; t < nt && w.ok; ++t) {
        w.on(&sm.empty[t % FOLD_SLOTS], t / FOLD_SLOTS - 1);
        if (w.ok) load(t);
      }
      if (w.ok)
        for (int t = max(0, nt - FOLD_SLOTS); t < nt; ++t) w.on(&sm.full[t % FOLD_SLOTS], t / FOLD_SLOTS);
      else
        for (int k = 0; k < FOLD_SLOTS; ++k) tc::mbar_wait_sleep(&sm.full[k], 0, 4000000LL);
    }
  } else if (warp == 8) {
    const uint32_t lead = tc::elect_leader();
    for (int i = 0; i < nc; ++i) {
      const int tb = 2 * i, tcc = tb + 1;
      w.warp_on(&sm.full[tcc % FOLD_SLOTS], tcc / FOLD_SLOTS);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        w.warp_on(&sm.barK[h], i);
        tc::fence_after();
        const uint32_t c = smem_u32(sm.slot[tcc % FOLD_SLOTS]) + 8192 * h;
        // The tensor cores' fp32 sums lose a little at every step: the first terms of
        // even and odd chunks and the small further terms have sums of their own.
        const uint32_t t0 = tX + 128 * (i & 1), t1 = tX + 256 + 128 * (i & 1);
        tc::gemm_rows_by<64>(lead, t0, smem_u32(sm.slot[tb % FOLD_SLOTS]) + 8192 * h, c, i > 1 || h > 0);
        tc::gemm_rows_by<64>(lead, t1, smem_u32(sm.rest[0]) + 8192 * h, c, i > 1 || h > 0);
        if (third) tc::gemm_rows_by<64>(lead, t1, smem_u32(sm.rest[1]) + 8192 * h, c, true);
        if (h == 1) {
          if (tb + FOLD_SLOTS < 2 * nc) tc::commit_by(lead, &sm.empty[tb % FOLD_SLOTS]);
          if (tcc + FOLD_SLOTS < 2 * nc) tc::commit_by(lead, &sm.empty[tcc % FOLD_SLOTS]);
        }
        tc::commit_by(lead, &sm.barM[h]);
      }
    }
  } else if (warp < 8) {
    const int j0 = 4 * (tid >> 6);  // 64 rows at a time, four threads to a row
    for (int i = 0; i < nc; ++i) {
      const int n = min(CH, q.len - chunk_of(i) * CH), tb = 2 * i, tcc = tb + 1;
      w.warp_on(&sm.full[tb % FOLD_SLOTS], tb / FOLD_SLOTS);
      if (n < CH) w.warp_on(&sm.full[tcc % FOLD_SLOTS], tcc / FOLD_SLOTS);
#pragma unroll 1
      for (int h = 0; h < 2; ++h) {
        const int r = 64 * h + (tid & 63), t0 = chunk_of(i) * CH + r;
        // weight to the segment's end (forwards) or to its start (backwards)
        const float e = expf(wd * (float)(R.rev ? t0 - cb * CH + 1 : max(end - 1 - t0, 0)));
        if (i > 0) w.warp_on(&sm.barM[h], i - 1);  // (these rows' further terms have been read)
        unsigned char* b = sm.slot[tb % FOLD_SLOTS];
        if (third)
          scale_row<3>(b, sm.rest[0], r, j0, e, r < n);
        else
          scale_row<2>(b, sm.rest[0], r, j0, e, r < n);
        if (r >= n) zero_row(sm.slot[tcc % FOLD_SLOTS], r, j0, 4);
        tc::fence_proxy_async();
        tc::mbar_arrive(&sm.barK[h]);
      }
    }
    w.warp_on(&sm.barM[1], nc - 1);
    tc::fence_after();
    const int row = 32 * (warp & 3) + lane, g0 = 2 * (warp >> 2);
    const uint32_t lane_base = (uint32_t)(32 * (warp & 3)) << 16;
    // With one segment this is the final state but for the initial one's share: through
    // shared memory (the tiles are done with), so that a warp touches whole rows.
    float* dst = R.x + ((long)slot * a.Hv + j) * HD * HD;
    unsigned char* staged = sm.slot[0];
    auto place = [&](int r, int c4) { return reinterpret_cast<float4*>(staged + r * 512 + ((c4 ^ (r & 7)) << 4)); };
#pragma unroll 1
    for (int g = g0; g < g0 + 2; ++g) {
      float v[32];
      tc::ld32(tX + 256 + lane_base + 32 * g, v);
#pragma unroll 1
      for (int k = 384; k >= 0; k -= 128) {  // the small sums first; odd chunks' where there were any
        if (k == 256 || (k & 128 && nc == 1)) continue;
        float y[32];
        tc::ld32(tX + k + lane_base + 32 * g, y);
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] += y[i];
      }
#pragma unroll
      for (int i = 0; i < 32; i += 4) {
        const int c = 32 * g + i;
        *(a.nseg == 1 ? place(row, c >> 2) : reinterpret_cast<float4*>(dst + seg_index(row, c))) =
            make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
      }
    }
    if (a.nseg == 1) {
      asm volatile("bar.sync 1, 256;" ::: "memory");
      const float keep = expf(wd * (float)q.len);
      // (both may be one state: an element is read and written by the same thread)
      const float* x0 = R.x0 ? R.x0 + sh * HD * HD + 4 * lane : nullptr;
      float* out = R.last + sh * HD * HD + 4 * lane;
#pragma unroll 1
      for (int r0 = warp; r0 < HD; r0 += 64) {
        float4 x[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
          x[k] = x0 ? *reinterpret_cast<const float4*>(x0 + (r0 + 8 * k) * HD) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float4 o = *place(r0 + 8 * k, lane);
          *reinterpret_cast<float4*>(out + (r0 + 8 * k) * HD) =
              make_float4(o.x + keep * x[k].x, o.y + keep * x[k].y, o.z + keep * x[k].z, o.w + keep * x[k].w);
        }
      }
    }
    tc::fence_before();
  }
  if (!w.ok && a.status) atomicOr(a.status, 1);
  __syncthreads();
  tc::fence_after();
  if (warp == 0) tc::dealloc(sm.tmem, 512);
}

// The segments' own states; with one segment to a sequence the final states, beside the
// walk (in three bf16 terms: an error of 1e-7 of the sums' sizes).
__global__ void __launch_bounds__(FOLD_THREADS, 1) k_decay_fold(const __grid_constant__ DecayFoldArgs a) {
  extern __shared__ unsigned char raw[];
  if (!a.beside) {
    pdl_wait();
    pdl_release();
    if (blockIdx.y == 0 && !a.behind) clear_status(a.status);  // (its call's first kernel)
  }
  fold_block(a, a.role[blockIdx.y], *reinterpret_cast<FoldSmem*>(raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u)),
             blockIdx.x / a.Hv, blockIdx.x % a.Hv);
  if (blockIdx.x == 0 && blockIdx.y == 0) pdl_wait();  // the grid ends after the one before it
}

// The walks of all passes.  SUM: an output head is the sum over a group's value heads,
// whose CTAs run side by side, each one a chunk or so behind the one before it.  FOLD:
// and the final states, from CTAs beside them (f.n_roles of them a sequence and head).
template <bool SUM, bool FOLD>
__device__ __forceinline__ void decay_block(const DecayArgs& a, const DecayFoldArgs* f) {
  extern __shared__ unsigned char raw[];
  unsigned char* smem = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
  if (a.nseg == 1 && !a.beside) {  // (with segments, only the entering states wait for the kernel before)
    pdl_wait();
    pdl_release();
    clear_status(a.status);
  }
  // This CTA's sequence (or segment), pass and head: the longest sequences' CTAs of all
  // passes come first, a group's heads side by side in the order of their sum.  Where a CTA
  // waits for the head before its own, places are handed out in the order of starts: that
  // head's CTA is then running or done, whatever order the CTAs of a grid start in.
  int place = (int)blockIdx.x;
  if constexpr (SUM) {
    __shared__ int started;
    if (threadIdx.x == 0) started = atomicAdd(a.ticket, 1);
    __syncthreads();
    place = started;
  }
  const int hd = place % a.Hv, u = place / a.Hv, kinds = a.n_roles + (FOLD ? f->n_roles : 0);
  const int ri = u % kinds, slot = u / kinds;
  if constexpr (FOLD) {
    if (ri >= a.n_roles) {
      fold_block(*f, f->role[ri - a.n_roles], *reinterpret_cast<FoldSmem*>(smem), slot, hd);
      return;
    }
  }
  const DecayRole& R = a.role[ri];
  WalkSmem& sm = *reinterpret_cast<WalkSmem*>(smem);
  const int2 at = find_segment(a.cu, a.n_seqs, a.T, a.total, a.seg_chunks, a.nseg, slot);
  if (at.x < 0) return;
  const Range q = seq_range(a.cu, at.x, a.T, a.total);
  const int nch = (q.len + CH - 1) / CH, cb = at.y * a.seg_chunks, ce = a.nseg == 1 ? nch : min(nch, cb + a.seg_chunks);
  if (cb >= ce) return;
  if (R.rev)
    walk<SUM, true>(a, R, sm, q, at.x, slot, hd, cb, ce);
  else
    walk<SUM, false>(a, R, sm, q, at.x, slot, hd, cb, ce);
}
template <bool SUM>
__global__ void __launch_bounds__(WALK_THREADS, 1) k_decay(const __grid_constant__ DecayArgs a) {
  decay_block<SUM, false>(a, nullptr);
  if (blockIdx.x == 0) pdl_wait();  // the grid ends after the one before it, whatever its CTAs had to do
}
template <bool SUM>
__global__ void __launch_bounds__(WALK_THREADS, 1) k_decay_small(const __grid_constant__ DecayArgs a,
                                                                 const __grid_constant__ DecayFoldArgs f) {
  decay_block<SUM, true>(a, &f);
}

// Entering states from the segments' own ones, in place, and the final state:
// run <- X0;  per segment in the pass's order: x <- run, run <- e^{w len} run + x.
__global__ void __launch_bounds__(256) k_decay_prefix(const __grid_constant__ DecayFoldArgs a) {
  pdl_wait();
  pdl_release();
  const int j = blockIdx.x % a.Hv, s = blockIdx.x / a.Hv;
  const DecayFoldRole& R = a.role[blockIdx.z];
  const Range q = seq_range(a.cu, s, a.T, a.total);
  const int nch = (q.len + CH - 1) / CH, nseg = (nch + a.seg_chunks - 1) / a.seg_chunks;
  const long sh = (long)s * a.Hv + j;
  const int e = 4 * (blockIdx.y * 256 + threadIdx.x);  // 16 blocks cover the state, in the segments' order
  const int e0 = ((e >> 2) & (HD - 1)) * HD + 4 * (e >> 9);  // the same place in a caller's state
  const float wd = log_decay(a.decay, j);
  const int slot0 = first_slot(a.cu, s, a.T, a.total, a.seg_chunks * CH);
  float4 run = R.x0 ? *reinterpret_cast<const float4*>(R.x0 + sh * HD * HD + e0) : make_float4(0.f, 0.f, 0.f, 0.f);
  constexpr int AHEAD = 4;  // loads in flight
  for (int i0 = 0; i0 < nseg; i0 += AHEAD) {
    float4 x[AHEAD];
    float4* p[AHEAD];
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      const int i = i0 + k, seg = R.rev ? nseg - 1 - i : i;
      p[k] = reinterpret_cast<float4*>(R.x + ((long)(slot0 + seg) * a.Hv + j) * HD * HD + e);
      x[k] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i < nseg && (R.last || i + 1 < nseg)) x[k] = *p[k];  // (the last one's own is not formed otherwise)
    }
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      const int i = i0 + k, seg = R.rev ? nseg - 1 - i : i;
      if (i >= nseg) break;
      *p[k] = run;
      const int len = min(q.len, (seg + 1) * a.seg_chunks * CH) - seg * a.seg_chunks * CH;
      const float keep = expf(wd * (float)len);
      run = make_float4(keep * run.x + x[k].x, keep * run.y + x[k].y, keep * run.z + x[k].z, keep * run.w + x[k].w);
    }
  }
  if (R.last) *reinterpret_cast<float4*>(R.last + sh * HD * HD + e0) = run;
}

template <typename K>
cudaError_t set_smem(K k, size_t bytes) {
  return cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

}  // namespace

template <bool SUM>
static cudaError_t launch_walk(const DecayArgs& a, const DecayFoldArgs& f, cudaStream_t s) {
  constexpr size_t smem = (sizeof(WalkSmem) > sizeof(FoldSmem) ? sizeof(WalkSmem) : sizeof(FoldSmem)) + 1024;
  static_assert(smem <= 227 * 1024, "shared memory");
  const cudaError_t e = f.n_roles ? set_smem(k_decay_small<SUM>, smem) : set_smem(k_decay<SUM>, smem);
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)((long)(a.n_roles + f.n_roles) * a.slots * a.Hv)), block(WALK_THREADS);
  return f.n_roles ? launch_pdl(k_decay_small<SUM>, grid, block, smem, s, a, f)
                   : launch_pdl(k_decay<SUM>, grid, block, smem, s, a);
}

cudaError_t launch_decay(const DecayArgs& a, const DecayFoldArgs& f, cudaStream_t s) {
  return a.Hv > a.Hk && a.role[0].shared ? launch_walk<true>(a, f, s) : launch_walk<false>(a, f, s);
}

cudaError_t launch_decay_fold(const DecayFoldArgs& a, cudaStream_t s) {
  constexpr size_t smem = sizeof(FoldSmem) + 1024;
  static_assert(smem <= 227 * 1024, "shared memory");
  cudaError_t e = set_smem(k_decay_fold, smem);
  if (e != cudaSuccess) return e;
  const unsigned sh = (unsigned)((long)a.n_seqs * a.Hv);
  e = launch_pdl(k_decay_fold, dim3((unsigned)a.slots * (unsigned)a.Hv, (unsigned)a.n_roles), dim3(FOLD_THREADS), smem, s, a);
  if (e != cudaSuccess || a.nseg == 1) return e;
  return launch_pdl(k_decay_prefix, dim3(sh, HD * HD / 1024, (unsigned)a.n_roles), dim3(256), 0, s, a);
}

}  // namespace gdn
