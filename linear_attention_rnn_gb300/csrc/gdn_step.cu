// gdn_step.cu -- single-token forms: one token per row, the row's state updated in
// place, for the gated delta rule and for linear attention with a decay for
// each head.  Per row r, value head j (key head kh = j / (Hv / Hk)) and its
// state h [128 (d_k)][128 (d_v)] in fp32:
//   delta:  h <- e^g (h - beta k (k^T h)) + beta k v^T,     o = h^T q
//   decay:  h <- e^w h + k v^T,                             o = h^T q
// Every column of h evolves by itself, so the new column and its output need
// only two dot products with the old column, x = k^T h and y = q^T h:
//   n = beta (v - e^g x)  (decay: n = v),   h <- e^g h + k n,   o = e^g y + (q . k) n
// which one pass over the state forms: it is read once into registers, reduced
// across the block once, and written once.
//
// Bound: HBM.  A state is 64 KiB read and 64 KiB written against 1.3 KiB of
// everything else and 5 to 9 operations per element.  Measured on a GB300, 32 heads:
// 256 rows 156 us (decay) and 512 rows 310 us (delta), 6.9 TB/s, 1.02 of the rate of
// a plain copy; one row 4 us, a launch's and a memory round trip's latency.  A block of 128 threads
// holds 32 columns (one 128-byte line of each of the 128 rows), 32 values to a
// thread, all of its loads in flight at once; four blocks share a state.  Small
// blocks make the loads of a single row spread over 4 Hv SMs (128 at 32 heads)
// and keep enough of them resident to cover the memory latency in large calls.
#include "gdn_kernels.cuh"

namespace gdn {

namespace {

constexpr int STEP_COLS = 32;                   // state columns per block
constexpr int STEP_SPLIT = HD / STEP_COLS;      // blocks per state
constexpr int STEP_THREADS = 128;               // 8 column groups (float4) x 16 row groups of 8 rows

__device__ __forceinline__ void load8(const bf16* p, float (&x)[8]) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = unpack_bf16(w[i]);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}

template <bool DELTA>
__global__ void __launch_bounds__(STEP_THREADS) k_step(const __grid_constant__ StepArgs a) {
  __shared__ float red[4][2][STEP_COLS];  // per warp: k^T h and q^T h of the block's columns
  __shared__ float redqk[4];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int cg = lane & 7, rg = tid >> 3;  // columns 4 cg .. 4 cg + 3, rows 8 rg .. 8 rg + 7
  const long unit = (long)blockIdx.x / STEP_SPLIT;
  const int c0 = (int)(blockIdx.x % STEP_SPLIT) * STEP_COLS + 4 * cg;
  const long r = unit / a.Hv;
  const int j = (int)(unit % a.Hv), kh = j / (a.Hv / a.Hk);
  pdl_wait();
  pdl_release();
  const long slot = a.slots ? (long)a.slots[r] : r;
  bf16* orow = a.o + (r * a.Hv + j) * HD;
  if (slot < 0 || slot >= a.n_slots) {  // a row without a state: zero output, nothing else touched
    if (rg == 0) *reinterpret_cast<uint2*>(orow + c0) = make_uint2(0u, 0u);
    return;
  }
  float* st = a.state + ((slot * a.Hv + j) * HD + 8 * rg) * (long)HD + c0;
  float4 h[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) h[i] = *reinterpret_cast<const float4*>(st + (long)i * HD);
  float k[8], q[8];
  load8(a.k + r * a.sk + kh * HD + 8 * rg, k);
  load8(a.q + r * a.sq + kh * HD + 8 * rg, q);
  const float2 v01 = unpack_bf16(*reinterpret_cast<const uint32_t*>(a.v + r * a.sv + j * HD + c0));
  const float2 v23 = unpack_bf16(*reinterpret_cast<const uint32_t*>(a.v + r * a.sv + j * HD + c0 + 2));
  const float eg = expf(DELTA ? a.g[r * a.Hv + j] : a.g[j]);
  const float beta = DELTA ? a.beta[r * a.Hv + j] : 1.f;

  float x[4] = {0.f, 0.f, 0.f, 0.f}, y[4] = {0.f, 0.f, 0.f, 0.f}, qk = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float hv[4] = {h[i].x, h[i].y, h[i].z, h[i].w};
    qk += q[i] * k[i];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      if (DELTA) x[c] += k[i] * hv[c];
      y[c] += q[i] * hv[c];
    }
  }
#pragma unroll
  for (int off = 8; off <= 16; off <<= 1) {  // over the warp's four row groups
    qk += __shfl_xor_sync(0xffffffffu, qk, off);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      if (DELTA) x[c] += __shfl_xor_sync(0xffffffffu, x[c], off);
      y[c] += __shfl_xor_sync(0xffffffffu, y[c], off);
    }
  }
  if (lane < 8) {
    if (DELTA) *reinterpret_cast<float4*>(&red[warp][0][4 * cg]) = make_float4(x[0], x[1], x[2], x[3]);
    *reinterpret_cast<float4*>(&red[warp][1][4 * cg]) = make_float4(y[0], y[1], y[2], y[3]);
  }
  if (lane == 0) redqk[warp] = qk;
  __syncthreads();
  qk = redqk[0] + redqk[1] + redqk[2] + redqk[3];
  const float v[4] = {v01.x, v01.y, v23.x, v23.y};
  float n[4], o[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const float ys = red[0][1][4 * cg + c] + red[1][1][4 * cg + c] + red[2][1][4 * cg + c] + red[3][1][4 * cg + c];
    n[c] = v[c];
    if (DELTA) {
      const float xs =
          red[0][0][4 * cg + c] + red[1][0][4 * cg + c] + red[2][0][4 * cg + c] + red[3][0][4 * cg + c];
      n[c] = beta * (v[c] - eg * xs);
    }
    o[c] = eg * ys + qk * n[c];
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    *reinterpret_cast<float4*>(st + (long)i * HD) =
        make_float4(eg * h[i].x + k[i] * n[0], eg * h[i].y + k[i] * n[1], eg * h[i].z + k[i] * n[2],
                    eg * h[i].w + k[i] * n[3]);
  if (rg == 0) *reinterpret_cast<uint2*>(orow + c0) = make_uint2(pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3]));
}

}  // namespace

cudaError_t launch_step(const StepArgs& a, cudaStream_t s) {
  const dim3 grid((unsigned)(a.R * a.Hv * STEP_SPLIT));
  return a.beta ? launch_pdl(k_step<true>, grid, dim3(STEP_THREADS), 0, s, a)
                : launch_pdl(k_step<false>, grid, dim3(STEP_THREADS), 0, s, a);
}

}  // namespace gdn
