// gdn_rope.cu -- norms of query and key heads with the position rotation in the same
// pass, its gradients, and the form that writes keys and values into a cache's pages.
//
// Per token and head, x [128] in bf16, everything between in fp32:
//   n = x r w,  r = 1 / sqrt(mean(x^2) + eps)         (no weight w: n = x)
//   y = n with each of its first P pairs (a, b) turned: a cos - b sin, b cos + a sin,
//       by the angle  position on the pair's axis x frequency of the pair
// and back, for a cotangent dy, with u = x r:
//   dn = dy turned by the opposite angles,   dw = sum over tokens and heads of dn u,
//   g = dn w,   dx = r (g - u mean(g u))               (no weight: dx = dn)
//
// Angles.  Only the angle's fraction of a turn counts, and a position times a frequency
// in fp32 has lost it at some 10^5 (an error of 2^-24 of the angle itself).  The
// frequency is taken as a 64-bit fraction of a turn instead; the product with the
// position modulo 2^64 is one integer multiplication and keeps every bit: the angle is
// right to 4e-7 at any position.  sincospi of its upper 32 bits follows.
//
// Layout.  Eight lanes hold a head, 16 values each in two 16-byte pieces that hold
// whole pairs in either order of pairs, so that only the norm's sum crosses lanes.  A
// warp takes four heads at a time, first those of q, then those of k (then those of v),
// token by token, forms a token's cosines and sines once, and has three steps' rows on
// their way.  The warps that stay resident share all steps equally: blocks that start one after
// another for their tokens took 55 us forward and backward of 8192 tokens, these 45.
//
// Bound: HBM, and on the way there the issue of instructions (the two are near each other: no
// warp waits for memory first).  14040 tokens of 16/16 heads: forward 39 us (230 MB, 5.9 TB/s),
// backward 55 us (345 MB, 6.2 TB/s).  8192 tokens of 16/4: 19 and 26 us (84 and 126 MB), a
// third of it starts and ends.  77 tokens: 6 us.
#include "gdn_kernels.cuh"

namespace gdn {

namespace {

constexpr int LANES = 8, SIDE = 32 / LANES;  // to a head; heads side by side in a warp
constexpr int ROPE_THREADS = 256, WARPS = ROPE_THREADS / 32;
constexpr int PAIRS = HD / 2;                // at most
constexpr int AHEAD = 3;                     // steps (of four heads) whose rows are on their way (1: 46 us for 45)

// Cosines and sines of a warp's token, in the order in which the lanes of a head read them:
// four values of each lane (pairs 8 l ..), then the next four (no two lanes on one bank).
struct Turns {
  float cos[PAIRS], sin[PAIRS];
  static __device__ __forceinline__ int at(int j) { return (j >> 2 & 1) * (PAIRS / 2) + (j >> 3) * 4 + (j & 3); }
};
// Rows on their way: each lane fetches its own pieces and alone reads them, so that no
// barrier comes between a load and its use.
template <bool BACK>
struct RopeSmem {
  float w[2][4][LANES][4];  // the weights of q and k, in the lanes' order likewise
  Turns turns[WARPS];
  uint4 row[WARPS][AHEAD + 1][BACK ? 2 : 1][2][32];
};

__device__ __forceinline__ void fetch16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void fetch_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void fetch_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A frequency as the fraction of a turn that a position adds, in 2^-64 of a turn: the 24
// bits of its significand times 2^64 / (2 pi), shifted by its exponent.
__device__ __forceinline__ unsigned long long turn_step(float f) {
  constexpr unsigned long long PER_RADIAN = 0x28BE60DB9391054Aull;  // 2^64 / (2 pi)
  const uint32_t u = __float_as_uint(f), e = u >> 23 & 255u;
  const unsigned long long m = e ? (u & 0x7fffffu) | 0x800000u : (u & 0x7fffffu);
  const unsigned long long lo = m * PER_RADIAN, hi = __umul64hi(m, PER_RADIAN);
  const int right = 150 - (int)(e ? e : 1u);  // the value is m 2^-right
  unsigned long long r;
  if (right <= 0)
    r = right > -64 ? lo << -right : 0ull;
  else if (right < 64)
    r = lo >> right | hi << (64 - right);
  else
    r = right < 128 ? hi >> (right - 64) : 0ull;
  return u >> 31 ? 0ull - r : r;
}

// A lane's two pairs of its warp's token: lane and lane + 32.
struct Angles {
  unsigned long long step[2];
  const int* pos[2];
  int at[2];  // their positions for the next token
  __device__ __forceinline__ explicit Angles(const RopeArgs& a) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int j = (threadIdx.x & 31) + 32 * i;
      pos[i] = j < a.P ? a.pos + (a.axes > 1 ? (long)a.axis[j] * a.n : 0) : nullptr;
      step[i] = j < a.P ? turn_step(a.freq[j]) : 0ull;
      at[i] = 0;
    }
  }
  __device__ __forceinline__ void read(int t) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (pos[i]) at[i] = pos[i][t];
  }
  __device__ __forceinline__ void form(Turns& to) const {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int j = (threadIdx.x & 31) + 32 * i;
      const unsigned long long turn = step[i] * (unsigned long long)(long long)at[i];
      sincospif((float)(int)(turn >> 32) * 0x1p-31f, &to.sin[Turns::at(j)], &to.cos[Turns::at(j)]);
    }
  }
};

// Two fp32 values, for the instructions that work on pairs.
struct F2 {
  unsigned long long v;
};
__device__ __forceinline__ F2 pair(float x, float y) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ float2 parts(F2 a) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
  return r;
}
__device__ __forceinline__ F2 operator*(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 fma(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}

// a head's 16 values of a lane, piece by piece
__device__ __forceinline__ void unpack16(const uint4 (&u)[2], F2 (&x)[8]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t w[4] = {u[h].x, u[h].y, u[h].z, u[h].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[4 * h + i] = pair(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
  }
}
__device__ __forceinline__ uint4 pack8(const F2* x) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = parts(x[i]);
    w[i] = pack_bf16(f.x, f.y);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ float dot(const F2 (&x)[8], const F2 (&y)[8]) {
  F2 s = x[0] * y[0], t = x[1] * y[1];
#pragma unroll
  for (int i = 2; i < 8; i += 2) {
    s = fma(x[i], y[i], s);
    t = fma(x[i + 1], y[i + 1], t);
  }
  const float2 a = parts(s), b = parts(t);
  return (a.x + a.y) + (b.x + b.y);
}

// Where lane `l` of a head's eight finds its two pieces: pairs 8 l .. 8 l + 7, or
// two pieces of what is not turned.
__device__ __forceinline__ void pieces(const RopeArgs& a, int l, int& p0, int& p1) {
  if (a.interleaved || 8 * l >= a.P) {
    p0 = 16 * l;  // (behind the pairs of the other order, too: 2 P + 16 (l - P / 8))
    p1 = p0 + 8;
  } else {
    p0 = 8 * l;
    p1 = a.P + 8 * l;
  }
}

// The lane's pairs turned by the token's angles (back: by the opposite ones).
template <bool BACK, bool INTER>
__device__ __forceinline__ void turn(const RopeArgs& a, const Turns& s, int l, F2 (&x)[8]) {
  if (8 * l >= a.P) return;
  F2 c[4], d[4];  // of two pairs each
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const ulonglong2 u = *reinterpret_cast<const ulonglong2*>(&s.cos[4 * l + (PAIRS / 2) * i]);
    const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(&s.sin[4 * l + (PAIRS / 2) * i]);
    c[2 * i].v = u.x, c[2 * i + 1].v = u.y;
    d[2 * i].v = v.x, d[2 * i + 1].v = v.y;
  }
  const F2 minus = pair(-1.f, -1.f);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (INTER) {
      const float2 cc = parts(c[i]), ss = parts(d[i]);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float cs = k ? cc.y : cc.x, sn = BACK ? -(k ? ss.y : ss.x) : (k ? ss.y : ss.x);
        const float2 v = parts(x[2 * i + k]);
        x[2 * i + k] = fma(pair(v.y, v.x), pair(-sn, sn), x[2 * i + k] * pair(cs, cs));
      }
    } else {
      const F2 p = x[i], q = x[4 + i];
      x[i] = fma(BACK ? q : q * minus, d[i], p * c[i]);
      x[4 + i] = fma(BACK ? p * minus : p, d[i], q * c[i]);
    }
  }
}

// Sum over the eight lanes of a head.
__device__ __forceinline__ float head_sum(float v) {
#pragma unroll
  for (int o = 1; o < LANES; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// A step is four heads of a token, side by side: those of q, then those of k (then those
// of v).  Every warp walks an equal run of all tokens' steps.
template <bool BACK, bool INTER, bool PAGED>
__global__ void __launch_bounds__(ROPE_THREADS, BACK ? 2 : 3) k_rope(const __grid_constant__ RopeArgs a) {
  extern __shared__ __align__(16) unsigned char raw[];
  RopeSmem<BACK>& sm = *reinterpret_cast<RopeSmem<BACK>*>(raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, l = lane & (LANES - 1), side = lane / LANES;
  pdl_wait();
  pdl_release();
  const RopePart &q = a.part[0], &k = a.part[1], &v = a.part[2];
  const int Hqk = q.H + k.H, H = PAGED ? Hqk + v.H : Hqk, steps = (H + SIDE - 1) / SIDE;
  const int me = (int)blockIdx.x * WARPS + warp, count = a.run + (me < a.longer ? 1 : 0);
  const unsigned first = (unsigned)me * (unsigned)a.run + (unsigned)min(me, a.longer);
  int c0, c1;
  pieces(a, l, c0, c1);
  const int hop = c1 - c0;
  const int t0 = (int)(first / (unsigned)steps), i0 = (int)(first - (unsigned)t0 * (unsigned)steps);

  // the rows ahead: the lane's place in the token's rows of q and of k (and of v), as if
  // each had all heads
  const int at = side * HD + c0;
  const bf16* qx = q.x + (t0 * q.sx + at);
  const bf16* kx = k.x + (t0 * k.sx + at - q.H * HD);
  const bf16* vx = PAGED ? v.x + (t0 * v.sx + at - Hqk * HD) : nullptr;
  const bf16* qg = BACK ? q.g + (t0 * q.sg + at) : nullptr;
  const bf16* kg = BACK ? k.g + (t0 * k.sg + at - q.H * HD) : nullptr;
  const bool normed = q.w || k.w;
  int fi = i0, fleft = count, fslot = 0;
  auto fetch = [&] {
    if (fleft > 0) {
      const int h = SIDE * fi + side, off = fi * (SIDE * HD);
      if (h < H) {
        if (!BACK || (h < q.H ? q.w : k.w)) {
          const bf16* x = (h < q.H ? qx : !PAGED || h < Hqk ? kx : vx) + off;
          fetch16(&sm.row[warp][fslot][0][0][lane], x);
          fetch16(&sm.row[warp][fslot][0][1][lane], x + hop);
        }
        if (BACK) {
          const bf16* g = (h < q.H ? qg : kg) + off;
          fetch16(&sm.row[warp][fslot][BACK][0][lane], g);
          fetch16(&sm.row[warp][fslot][BACK][1][lane], g + hop);
        }
      }
      --fleft;
      if (++fi == steps) {
        fi = 0;
        qx += q.sx;
        kx += k.sx;
        if (PAGED) vx += v.sx;
        if (BACK) {
          qg += q.sg;
          kg += k.sg;
        }
      }
      fslot = (fslot + 1) & AHEAD;
    }
    fetch_commit();
  };
  static_assert((AHEAD & (AHEAD + 1)) == 0, "slots in turn");
#pragma unroll
  for (int u = 0; u < AHEAD; ++u) fetch();

  for (int e = warp; e < 32; e += WARPS) {  // four of a lane's values at a time
    const float* w = a.part[e / 16].w;
    const int piece = e / 4 % 4, from = (piece < 2 ? c0 : c1) + 4 * (piece & 1) + (e & 3);
    if (lane < LANES) sm.w[e / 16][piece][lane][e & 3] = w ? w[from] : 1.f;
  }
  Angles angles(a);
  int row = 0;  // of the next token in the cache
  if (count > 0) {
    angles.read(t0);
    if (PAGED) row = a.slots[t0];
  }
  F2 dq[8], dk[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) dq[j] = dk[j] = pair(0.f, 0.f);
  __syncthreads();

  int t = t0, slot = 0, i = i0;
  bf16* qy = q.y + (t0 * q.sy + at);
  bf16* ky = PAGED ? nullptr : k.y + (t0 * k.sy + at - q.H * HD);
  bf16* vy = nullptr;
  bool placed = !PAGED;  // (paged: the token has a row)
  Turns& turns = sm.turns[warp];
  for (int u = 0; u < count; ++u) {
    fetch();
    if (u == 0 || i == steps) {  // a new token
      if (u > 0) {
        i = 0;
        ++t;
        qy += q.sy;
        if (!PAGED) ky += k.sy;
      }
      __syncwarp();  // (the last one's turns have been read)
      if (a.P > 0) angles.form(turns);
      if (PAGED) {
        placed = row >= 0 && row < a.cache_rows;  // (else a padded token of the batch)
        const int page = placed ? a.pages.page_of(row) : 0;
        const long in = row - page * a.pages.page;
        ky = k.y + (page * k.sy + in * k.sy_row + side * k.sy_head + c0);
        vy = v.y + (page * v.sy + in * v.sy_row + side * v.sy_head + c0);
      }
      if (t + 1 < a.n) {
        angles.read(t + 1);
        if (PAGED) row = a.slots[t + 1];
      }
      __syncwarp();
    }
    fetch_wait<AHEAD>();
    const int h = SIDE * i + side;
    const bool own = h < H, is_k = h >= q.H;
    const uint4* from = &sm.row[warp][slot][0][0][lane];
    uint4 o[2] = {from[0], from[32]};
    F2 x[8], y[8];
    if (!BACK) {
      unpack16(o, x);
      // (the sums cross heads of keys and of values, which a step may have side by side: the whole warp forms
      // them where one of its heads has a norm, and those of values are not used)
      float r = 1.f;
      if (normed && (!PAGED || SIDE * i < Hqk)) r = rsqrtf(head_sum(dot(x, x)) * (1.f / HD) + a.eps);
      if (!PAGED || h < Hqk) {
        if (normed) {
          if (!(is_k ? k.w : q.w)) r = 1.f;
          const F2 rr = pair(r, r);
#pragma unroll
          for (int j = 0; j < 8; j += 2) {
            const ulonglong2 ww = *reinterpret_cast<const ulonglong2*>(sm.w[is_k][j / 2][l]);
            x[j] = x[j] * (rr * F2{ww.x});
            x[j + 1] = x[j + 1] * (rr * F2{ww.y});
          }
        }
        turn<false, INTER>(a, turns, l, x);
        o[0] = pack8(x);
        o[1] = pack8(x + 4);
      }
    } else {
      const uint4 g[2] = {from[64], from[96]};
      unpack16(g, y);
      turn<true, INTER>(a, turns, l, y);
      if (normed) {
        unpack16(o, x);
        const float r = rsqrtf(head_sum(dot(x, x)) * (1.f / HD) + a.eps);
        const F2 rr = pair(r, r);
        F2 gx[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = x[j] * rr;
        if (own && !is_k) {
#pragma unroll
          for (int j = 0; j < 8; ++j) dq[j] = fma(y[j], x[j], dq[j]);
        } else if (own) {
#pragma unroll
          for (int j = 0; j < 8; ++j) dk[j] = fma(y[j], x[j], dk[j]);
        }
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
          const ulonglong2 ww = *reinterpret_cast<const ulonglong2*>(sm.w[is_k][j / 2][l]);
          gx[j] = y[j] * F2{ww.x};
          gx[j + 1] = y[j + 1] * F2{ww.y};
        }
        // r (g - u mean(g u))
        const float gu = -r * (head_sum(dot(gx, x)) * (1.f / HD));
        const F2 mean = pair(gu, gu);
        if (is_k ? k.w : q.w) {
#pragma unroll
          for (int j = 0; j < 8; ++j) y[j] = fma(x[j], mean, gx[j] * rr);
        }
      }
      o[0] = pack8(y);
      o[1] = pack8(y + 4);
    }
    bf16* dst;
    if (!PAGED || !is_k)
      dst = (is_k ? ky : qy) + i * (SIDE * HD);
    else if (h < Hqk)
      dst = ky + (SIDE * i - q.H) * k.sy_head;
    else
      dst = vy + (SIDE * i - Hqk) * v.sy_head;
    if (own && (placed || !is_k)) {
      *reinterpret_cast<uint4*>(dst) = o[0];
      *reinterpret_cast<uint4*>(dst + hop) = o[1];
    }
    slot = (slot + 1) & AHEAD;
    ++i;
  }
  if constexpr (BACK) {
    if (!q.dw && !k.dw) return;
    // the block's sums: over the warp's four heads, then over the warps
    __syncthreads();
    float* red = reinterpret_cast<float*>(&sm.row[0][0][0][0][0]);  // [warps][2][HD]
    static_assert(sizeof(sm.row) >= WARPS * 2 * HD * sizeof(float), "room for the sums");
#pragma unroll
    for (int w = 0; w < 2; ++w) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float2 d = parts(w ? dk[j] : dq[j]);
#pragma unroll
        for (int o = LANES; o < 32; o <<= 1) {
          d.x += __shfl_xor_sync(0xffffffffu, d.x, o);
          d.y += __shfl_xor_sync(0xffffffffu, d.y, o);
        }
        if (lane < LANES) *reinterpret_cast<float2*>(red + (2 * warp + w) * HD + (j < 4 ? c0 + 2 * j : c1 + 2 * j - 8)) = d;
      }
    }
    __syncthreads();
    float sum = 0.f;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) sum += red[2 * w * HD + tid];
    a.partial[(long)blockIdx.x * 2 * HD + tid] = sum;
  }
}

// The gradients of the two weights: the blocks' sums, in a fixed order.  Bound by the latency of
// its loads, 0.3 MB of partial sums in 6 us; a thread to a column that adds row by row took 37.
constexpr int DW_THREADS = 1024, DW_ROWS = DW_THREADS * 4 / HD;
__global__ void __launch_bounds__(DW_THREADS) k_rope_dw(const __grid_constant__ RopeArgs a) {
  __shared__ float red[DW_ROWS][HD];
  pdl_wait();
  pdl_release();
  const RopePart& p = a.part[blockIdx.x];
  if (!p.dw) return;
  const int c = 4 * (threadIdx.x % (HD / 4)), s = threadIdx.x / (HD / 4);
  const float* from = a.partial + blockIdx.x * HD + c;
  float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
  for (int i = s; i < a.blocks; i += DW_ROWS) {
    const float4 v = *reinterpret_cast<const float4*>(from + (long)i * 2 * HD);
    sum.x += v.x;
    sum.y += v.y;
    sum.z += v.z;
    sum.w += v.w;
  }
  *reinterpret_cast<float4*>(&red[s][c]) = sum;
  __syncthreads();
  if (threadIdx.x < HD) {
    float total = 0.f;
#pragma unroll
    for (int i = 0; i < DW_ROWS; ++i) total += red[i][threadIdx.x];
    p.dw[threadIdx.x] = total;
  }
}

template <bool BACK, bool PAGED>
cudaError_t launch(RopeArgs a, cudaStream_t s) {
  const int H = a.part[0].H + a.part[1].H + a.part[2].H;
  const long steps = a.n * ((H + SIDE - 1) / SIDE), warps = (long)a.blocks * WARPS;
  a.run = (int)(steps / warps);
  a.longer = (int)(steps % warps);
  const auto kernel = a.interleaved ? k_rope<BACK, true, PAGED> : k_rope<BACK, false, PAGED>;
  constexpr size_t smem = sizeof(RopeSmem<BACK>);
  if (smem > 48 * 1024) {  // (what a block may have without being asked)
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(kernel, dim3((unsigned)a.blocks), dim3(ROPE_THREADS), smem, s, a);
}

}  // namespace

int rope_blocks(int backward, long n, int H, int (*sms)()) {
  const long steps = n * ((H + SIDE - 1) / SIDE), need = (steps + WARPS - 1) / WARPS;
  if (need <= 64) return (int)need;  // (fewer than any device has SMs for: not worth the question)
  const long most = (long)(backward ? 2 : 3) * sms();
  return (int)(need < most ? need : most);
}

cudaError_t launch_rope_fwd(const RopeArgs& a, cudaStream_t s) {
  return a.part[2].H > 0 ? launch<false, true>(a, s) : launch<false, false>(a, s);
}

cudaError_t launch_rope_bwd(const RopeArgs& a, cudaStream_t s) {
  cudaError_t e = launch<true, false>(a, s);
  if (e != cudaSuccess || (!a.part[0].dw && !a.part[1].dw)) return e;
  return launch_pdl(k_rope_dw, dim3(2), dim3(DW_THREADS), 0, s, a);
}

}  // namespace gdn
