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
// and sines once, a token block ahead; as many blocks as stay resident walk over the
// tokens.
//
// Bound: HBM.
#include "gdn_kernels.cuh"

namespace gdn {

namespace {

constexpr int LANES = 8;                          // to a head
constexpr int ROPE_THREADS = 256;
constexpr int GROUPS = ROPE_THREADS / LANES;      // heads side by side
constexpr int PAIRS = HD / 2;                     // at most
constexpr int TOKENS = 16;                        // of a block, at most
constexpr int PER = 2;                            // heads of a group in one round
constexpr int ROUND = PER * GROUPS;

// Rows on their way: each thread fetches its own pieces rounds ahead and alone reads them,
// so that no barrier comes between a load and its use.
template <bool BACK>
struct Ring {
  static constexpr int ROUNDS = BACK ? 3 : 3, SRC = BACK ? 2 : 1;
  uint4 row[ROUNDS][SRC][PER][2][ROPE_THREADS];
};
struct Turns {
  float cos[PAIRS], sin[PAIRS];
};

__device__ __forceinline__ void fetch16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void fetch_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void fetch_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A thread's share of a block's angles: pair tid % 64 of every fourth token.  The
// positions are read a block ahead.
struct Angles {
  static constexpr int N = TOKENS * PAIRS / ROPE_THREADS;
  unsigned long long step;  // a position's step, in 2^-64 of a turn
  const int* pos;
  int at[N];
  __device__ __forceinline__ Angles(const RopeArgs& a) {
    const int j = threadIdx.x & (PAIRS - 1);
    pos = nullptr;
    step = 0;
    if (j >= a.P) return;
    double turns = (double)a.freq[j] * 0.15915494309189535;  // 1 / (2 pi)
    turns -= floor(turns);
    step = (unsigned long long)(turns * 18446744073709551616.0);
    pos = a.pos + (long)a.axis[j] * a.n;
  }
  __device__ __forceinline__ void read(const RopeArgs& a, long t0, int tokens) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int t = threadIdx.x / PAIRS + i * (ROPE_THREADS / PAIRS);
      at[i] = pos && t < tokens && t0 + t < a.n ? pos[t0 + t] : 0;
    }
  }
  __device__ __forceinline__ void form(Turns* to, int tokens) const {
    if (!pos) return;
    const int j = threadIdx.x & (PAIRS - 1);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int t = threadIdx.x / PAIRS + i * (ROPE_THREADS / PAIRS);
      if (t >= tokens) break;
      const unsigned long long turn = step * (unsigned long long)(long long)at[i];
      sincospif((float)(int)(turn >> 32) * 0x1p-31f, &to[t].sin[j], &to[t].cos[j]);
    }
  }
};

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
__device__ __forceinline__ void turn(const RopeArgs& a, const Turns& s, int l, float (&x)[16]) {
  if (8 * l >= a.P) return;
  float c[8], d[8];
#pragma unroll
  for (int i = 0; i < 8; i += 4) {
    *reinterpret_cast<float4*>(c + i) = *reinterpret_cast<const float4*>(&s.cos[8 * l + i]);
    *reinterpret_cast<float4*>(d + i) = *reinterpret_cast<const float4*>(&s.sin[8 * l + i]);
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

// A block walks token blocks t0 = tokens * (block, block + blocks, ..) of its part, each
// in rounds of 64 heads, eight lanes to a head and two heads to a group of lanes.
template <bool BACK>
__global__ void __launch_bounds__(ROPE_THREADS, BACK ? 2 : 3) k_rope(const __grid_constant__ RopeArgs a) {
  extern __shared__ __align__(16) unsigned char raw[];
  Ring<BACK>& ring = *reinterpret_cast<Ring<BACK>*>(raw);
  Turns* turns = reinterpret_cast<Turns*>(raw + sizeof(Ring<BACK>));  // [2][tokens]
  constexpr int ROUNDS = Ring<BACK>::ROUNDS;
  int block;
  const RopePart& p = a.part[part_of(a, block)];
  const int tid = threadIdx.x, l = tid & (LANES - 1), group = tid / LANES;
  pdl_wait();
  pdl_release();
  int c0, c1;
  pieces(a, l, c0, c1);
  const long step = (long)p.blocks * p.tokens;
  const int H = p.H, most = p.tokens * H;

  // the rounds ahead: token block f0, its round from head f_i on
  long f0 = (long)block * p.tokens;
  int fi = 0, fslot = 0;
  auto fetch = [&] {
    if (f0 < a.n) {
      const int rows = (int)min((long)p.tokens, a.n - f0) * H;
#pragma unroll
      for (int u = 0; u < PER; ++u) {
        const int i = fi + group + u * GROUPS;
        if (i < rows) {
          const int t = i / H, h = i - t * H;
          if (!BACK || p.w) {
            const bf16* x = p.x + (f0 + t) * p.sx + h * HD;
            fetch16(&ring.row[fslot][0][u][0][tid], x + c0);
            fetch16(&ring.row[fslot][0][u][1][tid], x + c1);
          }
          if (BACK) {
            const bf16* g = p.g + (f0 + t) * p.sg + h * HD;
            fetch16(&ring.row[fslot][Ring<BACK>::SRC - 1][u][0][tid], g + c0);
            fetch16(&ring.row[fslot][Ring<BACK>::SRC - 1][u][1][tid], g + c1);
          }
        }
      }
      fi += ROUND;
      if (fi >= most) {
        fi = 0;
        f0 += step;
      }
      fslot = fslot + 1 == ROUNDS ? 0 : fslot + 1;
    }
    fetch_commit();
  };
#pragma unroll
  for (int k = 0; k < ROUNDS - 1; ++k) fetch();

  float w[16], dw[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) w[i] = 1.f, dw[i] = 0.f;
  if (p.w) {
#pragma unroll
    for (int i = 0; i < 8; i += 4) {
      *reinterpret_cast<float4*>(w + i) = *reinterpret_cast<const float4*>(p.w + c0 + i);
      *reinterpret_cast<float4*>(w + 8 + i) = *reinterpret_cast<const float4*>(p.w + c1 + i);
    }
  }
  Angles angles(a);
  const long first = (long)block * p.tokens;
  int buf = 0, slot = 0;
  if (p.turned) {
    angles.read(a, first, p.tokens);
    angles.form(turns, p.tokens);
    angles.read(a, first + step, p.tokens);
  }
  for (long t0 = first; t0 < a.n; t0 += step) {
    const int rows = (int)min((long)p.tokens, a.n - t0) * H;
    if (p.turned) {
      __syncthreads();  // this block's turns are there, the last block's have been read
      if (t0 + step < a.n) angles.form(turns + (buf ^ 1) * p.tokens, p.tokens);
      angles.read(a, t0 + 2 * step, p.tokens);
    }
    for (int i0 = 0; i0 < most; i0 += ROUND) {
      fetch();
      fetch_wait<ROUNDS - 1>();
#pragma unroll
      for (int u = 0; u < PER; ++u) {
        const int i = i0 + group + u * GROUPS, t = i / H, h = i - t * H;
        const bool own = i < rows;  // (the lanes of a head agree; others go along for the sums)
        if (!__any_sync(0xffffffffu, own)) break;
        const Turns& turn_of = turns[buf * p.tokens + (own ? t : 0)];
        uint4 v[2] = {ring.row[slot][0][u][0][tid], ring.row[slot][0][u][1][tid]};
        float x[16], y[16];
        if (!BACK) {
          if (p.turned || p.w) {
            unpack16(v, x);
            if (p.w) {
              float ss = 0.f;
#pragma unroll
              for (int j = 0; j < 16; ++j) ss += x[j] * x[j];
              const float r = rsqrtf(head_sum(ss) * (1.f / HD) + a.eps);
#pragma unroll
              for (int j = 0; j < 16; ++j) x[j] *= r * w[j];
            }
            if (p.turned) turn<false>(a, turn_of, l, x);
            v[0] = pack8(x);
            v[1] = pack8(x + 8);
          }
        } else {
          const uint4 g[2] = {ring.row[slot][Ring<BACK>::SRC - 1][u][0][tid], ring.row[slot][Ring<BACK>::SRC - 1][u][1][tid]};
          unpack16(g, y);
          if (p.turned) turn<true>(a, turn_of, l, y);
          if (p.w) {
            unpack16(v, x);
            float ss = 0.f;
#pragma unroll
            for (int j = 0; j < 16; ++j) ss += x[j] * x[j];
            const float r = rsqrtf(head_sum(ss) * (1.f / HD) + a.eps);
            float gu = 0.f;
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              x[j] *= r;
              if (own) dw[j] += y[j] * x[j];
              y[j] *= w[j];
              gu += y[j] * x[j];
            }
            gu = head_sum(gu) * (1.f / HD);
#pragma unroll
            for (int j = 0; j < 16; ++j) y[j] = r * (y[j] - x[j] * gu);
          }
          v[0] = pack8(y);
          v[1] = pack8(y + 8);
        }
        if (!own) continue;
        bf16* dst;
        if (!BACK && p.paged) {
          const long row = a.slots[t0 + t];
          if (row < 0 || row >= a.cache_rows) continue;  // a padded token of the batch
          const long page = row / a.page;
          dst = p.y + page * p.sy + (row - page * a.page) * p.sy_row + h * p.sy_head;
        } else {
          dst = p.y + (t0 + t) * p.sy + h * HD;
        }
        *reinterpret_cast<uint4*>(dst + c0) = v[0];
        *reinterpret_cast<uint4*>(dst + c1) = v[1];
      }
      slot = slot + 1 == ROUNDS ? 0 : slot + 1;
    }
    buf ^= 1;
  }
  if constexpr (BACK) {
  if (!p.dw) return;
  // the block's sum of dw: over the warp's four heads, then over the warps
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    dw[j] += __shfl_xor_sync(0xffffffffu, dw[j], 8);
    dw[j] += __shfl_xor_sync(0xffffffffu, dw[j], 16);
  }
  __syncthreads();
  float* red = reinterpret_cast<float*>(raw);  // [warps][HD]
  if ((tid & 31) < LANES) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      red[(tid >> 5) * HD + c0 + j] = dw[j];
      red[(tid >> 5) * HD + c1 + j] = dw[8 + j];
    }
  }
  __syncthreads();
  if (tid < HD) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < ROPE_THREADS / 32; ++i) sum += red[i * HD + tid];
    a.partial[(long)blockIdx.x * HD + tid] = sum;
  }
  }
}

// The gradients of the two weights: the blocks' sums, in a fixed order.
constexpr int DW_THREADS = 1024, DW_ROWS = DW_THREADS * 4 / HD;
__global__ void __launch_bounds__(DW_THREADS) k_rope_dw(const __grid_constant__ RopeArgs a) {
  __shared__ float red[DW_ROWS][HD];
  pdl_wait();
  pdl_release();
  const RopePart& p = a.part[blockIdx.x];
  if (!p.dw) return;
  const int c = 4 * (threadIdx.x % (HD / 4)), s = threadIdx.x / (HD / 4);
  const float* from = a.partial + (blockIdx.x ? (long)a.part[0].blocks * HD : 0) + c;
  float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
  for (int i = s; i < p.blocks; i += DW_ROWS) {
    const float4 v = *reinterpret_cast<const float4*>(from + (long)i * HD);
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

template <bool BACK>
cudaError_t launch(const RopeArgs& a, int parts, cudaStream_t s) {
  int tokens = 0;
  unsigned blocks = 0;
  for (int i = 0; i < parts; ++i) {
    blocks += (unsigned)a.part[i].blocks;
    if (a.part[i].turned && a.part[i].tokens > tokens) tokens = a.part[i].tokens;
  }
  const size_t smem = sizeof(Ring<BACK>) + 2 * sizeof(Turns) * (size_t)tokens;
  static_assert(sizeof(Ring<true>) + 2 * TOKENS * sizeof(Turns) <= 113 * 1024, "two blocks to an SM");
  cudaError_t e = cudaFuncSetAttribute(k_rope<BACK>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)(sizeof(Ring<BACK>) + 2 * TOKENS * sizeof(Turns)));
  return e != cudaSuccess ? e : launch_pdl(k_rope<BACK>, dim3(blocks), dim3(ROPE_THREADS), smem, s, a);
}

}  // namespace

int rope_tokens(int H) { return H >= ROUND ? 1 : H * TOKENS > ROUND ? ROUND / H : TOKENS; }
int rope_resident(int backward) { return backward ? 2 : 3; }

cudaError_t launch_rope_fwd(const RopeArgs& a, cudaStream_t s) { return launch<false>(a, 3, s); }

cudaError_t launch_rope_bwd(const RopeArgs& a, cudaStream_t s) {
  cudaError_t e = launch<true>(a, 2, s);
  if (e != cudaSuccess || (!a.part[0].dw && !a.part[1].dw)) return e;
  return launch_pdl(k_rope_dw, dim3(2), dim3(DW_THREADS), 0, s, a);
}

}  // namespace gdn
