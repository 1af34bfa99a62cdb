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
// block takes the heads of q, of k or of v for some tokens and forms the tokens' cosines
// and sines once.
//
// Bound: HBM.
#include "gdn_kernels.cuh"

namespace gdn {

namespace {

constexpr int LANES = 8;                          // to a head
constexpr int ROPE_THREADS = 256;
constexpr int GROUPS = ROPE_THREADS / LANES;      // heads side by side
constexpr int PAIRS = HD / 2;                     // at most
constexpr int TOKENS = 32;                        // of a block, at most

struct Turns {
  float cos[TOKENS][PAIRS], sin[TOKENS][PAIRS];
};

// Cosines and sines of `count` tokens from t0 on.
__device__ __forceinline__ void form_turns(const RopeArgs& a, Turns& s, long t0, int count) {
  const int j = threadIdx.x & (PAIRS - 1);
  if (j >= a.P) return;
  double turns = (double)a.freq[j] * 0.15915494309189535;  // a position's step, 1 / (2 pi) to a radian
  turns -= floor(turns);
  const unsigned long long step = (unsigned long long)(turns * 18446744073709551616.0);
  const int* pos = a.pos + (long)a.axis[j] * a.n + t0;
  for (int t = threadIdx.x / PAIRS; t < count; t += ROPE_THREADS / PAIRS) {
    const unsigned long long at = step * (unsigned long long)(long long)pos[t];
    sincospif((float)(int)(at >> 32) * 0x1p-31f, &s.sin[t][j], &s.cos[t][j]);
  }
}

__device__ __forceinline__ void unpack16(const uint4 (&u)[2], float (&x)[16]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t w[4] = {u[h].x, u[h].y, u[h].z, u[h].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = unpack_bf16(w[i]);
      x[8 * h + 2 * i] = f.x;
      x[8 * h + 2 * i + 1] = f.y;
    }
  }
}
__device__ __forceinline__ uint4 pack8(const float* x) {
  return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
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
template <bool BACK>
__device__ __forceinline__ void turn(const RopeArgs& a, const Turns& s, int t, int l, float (&x)[16]) {
  if (8 * l >= a.P) return;
  float c[8], d[8];
#pragma unroll
  for (int i = 0; i < 8; i += 4) {
    *reinterpret_cast<float4*>(c + i) = *reinterpret_cast<const float4*>(&s.cos[t][8 * l + i]);
    *reinterpret_cast<float4*>(d + i) = *reinterpret_cast<const float4*>(&s.sin[t][8 * l + i]);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float sn = BACK ? -d[i] : d[i];
    if (a.interleaved) {
      const float p = x[2 * i], q = x[2 * i + 1];
      x[2 * i] = p * c[i] - q * sn;
      x[2 * i + 1] = q * c[i] + p * sn;
    } else {
      const float p = x[i], q = x[8 + i];
      x[i] = p * c[i] - q * sn;
      x[8 + i] = q * c[i] + p * sn;
    }
  }
}

// Sum over the eight lanes of a head.
__device__ __forceinline__ float head_sum(float v) {
#pragma unroll
  for (int o = 1; o < LANES; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The block's part: its rows (q, k or v) and its place among the blocks of that part.
__device__ __forceinline__ int part_of(const RopeArgs& a, int& block) {
  block = blockIdx.x;
  int r = 0;
#pragma unroll
  for (int i = 0; i < 2; ++i)
    if (r == i && block >= a.part[i].blocks) {
      block -= a.part[i].blocks;
      r = i + 1;
    }
  return r;
}

__global__ void __launch_bounds__(ROPE_THREADS) k_rope_fwd(const __grid_constant__ RopeArgs a) {
  __shared__ Turns s;
  int block;
  const RopePart& p = a.part[part_of(a, block)];
  const int l = threadIdx.x & (LANES - 1), group = threadIdx.x / LANES;
  pdl_wait();
  pdl_release();
  const long t0 = (long)block * p.tokens;
  const int count = (int)min((long)p.tokens, a.n - t0), rows = count * p.H;
  int c0, c1;
  pieces(a, l, c0, c1);
  if (p.turned) form_turns(a, s, t0, count);
  float w[16];
  if (p.w) {
#pragma unroll
    for (int i = 0; i < 8; i += 4) {
      *reinterpret_cast<float4*>(w + i) = *reinterpret_cast<const float4*>(p.w + c0 + i);
      *reinterpret_cast<float4*>(w + 8 + i) = *reinterpret_cast<const float4*>(p.w + c1 + i);
    }
  }
  __syncthreads();
  for (int i0 = 0; i0 < rows; i0 += GROUPS) {
    const int i = min(i0 + group, rows - 1);  // (past the end: the last row once more, not written)
    const int t = i / p.H, h = i - t * p.H;
    const bf16* src = p.x + (t0 + t) * p.sx + h * HD;
    uint4 u[2] = {*reinterpret_cast<const uint4*>(src + c0), *reinterpret_cast<const uint4*>(src + c1)};
    if (p.turned || p.w) {
      float x[16];
      unpack16(u, x);
      if (p.w) {
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < 16; ++j) ss += x[j] * x[j];
        const float r = rsqrtf(head_sum(ss) * (1.f / HD) + a.eps);
#pragma unroll
        for (int j = 0; j < 16; ++j) x[j] *= r * w[j];
      }
      if (p.turned) turn<false>(a, s, t, l, x);
      u[0] = pack8(x);
      u[1] = pack8(x + 8);
    }
    if (i0 + group >= rows) break;
    bf16* dst;
    if (p.paged) {
      const long slot = a.slots[t0 + t];
      if (slot < 0 || slot >= a.cache_rows) continue;  // a padded row of the batch
      const long page = slot / a.page;
      dst = p.y + page * p.sy + (slot - page * a.page) * p.sy_row + h * p.sy_head;
    } else {
      dst = p.y + (t0 + t) * p.sy + h * HD;
    }
    *reinterpret_cast<uint4*>(dst + c0) = u[0];
    *reinterpret_cast<uint4*>(dst + c1) = u[1];
  }
}

__global__ void __launch_bounds__(ROPE_THREADS) k_rope_bwd(const __grid_constant__ RopeArgs a) {
  __shared__ Turns s;
  __shared__ float red[ROPE_THREADS / 32][HD];
  int block;
  const int which = part_of(a, block);
  const RopePart& p = a.part[which];
  const int l = threadIdx.x & (LANES - 1), group = threadIdx.x / LANES;
  pdl_wait();
  pdl_release();
  int c0, c1;
  pieces(a, l, c0, c1);
  float w[16], dw[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) dw[i] = 0.f;
  if (p.w) {
#pragma unroll
    for (int i = 0; i < 8; i += 4) {
      *reinterpret_cast<float4*>(w + i) = *reinterpret_cast<const float4*>(p.w + c0 + i);
      *reinterpret_cast<float4*>(w + 8 + i) = *reinterpret_cast<const float4*>(p.w + c1 + i);
    }
  }
  for (long t0 = (long)block * p.tokens; t0 < a.n; t0 += (long)p.blocks * p.tokens) {
    const int count = (int)min((long)p.tokens, a.n - t0), rows = count * p.H;
    if (p.turned) form_turns(a, s, t0, count);
    __syncthreads();
    for (int i0 = 0; i0 < rows; i0 += GROUPS) {
      const int i = min(i0 + group, rows - 1);  // (past the end: the last row once more, neither written nor summed)
      const bool own = i0 + group < rows;
      const int t = i / p.H, h = i - t * p.H;
      const bf16* gs = p.g + (t0 + t) * p.sg + h * HD;
      const uint4 ug[2] = {*reinterpret_cast<const uint4*>(gs + c0), *reinterpret_cast<const uint4*>(gs + c1)};
      float g[16];
      if (p.w) {
        const bf16* xs = p.x + (t0 + t) * p.sx + h * HD;
        const uint4 ux[2] = {*reinterpret_cast<const uint4*>(xs + c0), *reinterpret_cast<const uint4*>(xs + c1)};
        float x[16];
        unpack16(ux, x);
        unpack16(ug, g);
        if (p.turned) turn<true>(a, s, t, l, g);
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < 16; ++j) ss += x[j] * x[j];
        const float r = rsqrtf(head_sum(ss) * (1.f / HD) + a.eps);
        float gu = 0.f;
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          x[j] *= r;
          if (own) dw[j] += g[j] * x[j];
          g[j] *= w[j];
          gu += g[j] * x[j];
        }
        gu = head_sum(gu) * (1.f / HD);
#pragma unroll
        for (int j = 0; j < 16; ++j) g[j] = r * (g[j] - x[j] * gu);
      } else {
        unpack16(ug, g);
        if (p.turned) turn<true>(a, s, t, l, g);
      }
      if (own) {
        bf16* dst = p.y + (t0 + t) * p.sy + h * HD;
        *reinterpret_cast<uint4*>(dst + c0) = pack8(g);
        *reinterpret_cast<uint4*>(dst + c1) = pack8(g + 8);
      }
    }
    __syncthreads();
  }
  if (!p.dw) return;
  // the block's sum of dw: over the warp's four heads, then over the warps
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    dw[j] += __shfl_xor_sync(0xffffffffu, dw[j], 8);
    dw[j] += __shfl_xor_sync(0xffffffffu, dw[j], 16);
  }
  const int warp = threadIdx.x >> 5;
  if ((threadIdx.x & 31) < LANES) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      red[warp][c0 + j] = dw[j];
      red[warp][c1 + j] = dw[8 + j];
    }
  }
  __syncthreads();
  if (threadIdx.x < HD) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < ROPE_THREADS / 32; ++i) sum += red[i][threadIdx.x];
    a.partial[(long)blockIdx.x * HD + threadIdx.x] = sum;
  }
}

// The gradients of the two weights: the blocks' sums in their order.
__global__ void __launch_bounds__(1024) k_rope_dw(const __grid_constant__ RopeArgs a) {
  __shared__ double red[8][HD];
  pdl_wait();
  pdl_release();
  const RopePart& p = a.part[blockIdx.x];
  if (!p.dw) return;
  const int c = threadIdx.x & (HD - 1), s = threadIdx.x / HD;
  const float* from = a.partial + (blockIdx.x ? (long)a.part[0].blocks * HD : 0) + c;
  double sum = 0.0;
  for (int i = s; i < p.blocks; i += 8) sum += from[(long)i * HD];
  red[s][c] = sum;
  __syncthreads();
  if (s == 0) {
#pragma unroll
    for (int i = 1; i < 8; ++i) sum += red[i][c];
    p.dw[c] = (float)sum;
  }
}

}  // namespace

int rope_tokens(int H) { return H >= 64 ? 1 : H > 64 / TOKENS ? 64 / H : TOKENS; }

cudaError_t launch_rope_fwd(const RopeArgs& a, cudaStream_t s) {
  return launch_pdl(k_rope_fwd, dim3((unsigned)(a.part[0].blocks + a.part[1].blocks + a.part[2].blocks)), dim3(ROPE_THREADS),
                    0, s, a);
}

cudaError_t launch_rope_bwd(const RopeArgs& a, cudaStream_t s) {
  cudaError_t e =
      launch_pdl(k_rope_bwd, dim3((unsigned)(a.part[0].blocks + a.part[1].blocks)), dim3(ROPE_THREADS), 0, s, a);
  if (e != cudaSuccess || (!a.part[0].dw && !a.part[1].dw)) return e;
  return launch_pdl(k_rope_dw, dim3(2), dim3(1024), 0, s, a);
}

}  // namespace gdn
