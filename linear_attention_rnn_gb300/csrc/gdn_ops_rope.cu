// gdn_ops_rope.cu -- the extern "C" boundary of the head norms with rotation
// (include/gdn.h).  Arguments are checked on the host before anything is enqueued.
#include <math.h>
#include <string.h>

#include "gdn_host.cuh"
#include "gdn_kernels.cuh"

using namespace gdn;

namespace {

int rope_check(int n, int Hq, int Hk, int d, int n_axes, int n_pairs, const unsigned char* pair_axis, const float* qw,
               const float* kw, const int* pos, const float* freq, float eps) {
  if (n < 0 || Hq <= 0 || Hk <= 0 || n_axes < 1) return GDN_ERR_ARG;
  if (d != HD || n_pairs < 0 || n_pairs > HD / 2 || n_pairs % 8 != 0) return GDN_ERR_SHAPE;
  if (!(eps >= 0.f) || isinf(eps)) return GDN_ERR_ARG;
  if ((long long)n * ((long long)Hq + 2LL * Hk + 3) > (1LL << 32)) return GDN_ERR_ARG;  // (steps of four heads in 32 bits)
  if (n_axes > 1 && n_pairs > 0 && !pair_axis) return GDN_ERR_ARG;
  if (pair_axis)
    for (int j = 0; j < n_pairs; ++j)
      if (pair_axis[j] >= n_axes) return GDN_ERR_ARG;
  if (!aligned(qw, 16) || !aligned(kw, 16) || !aligned(pos, 4) || !aligned(freq, 4)) return GDN_ERR_ARG;
  if (n > 0 && n_pairs > 0 && (!pos || !freq)) return GDN_ERR_ARG;
  return GDN_OK;
}

RopeArgs rope_args(int n, int n_axes, int n_pairs, const unsigned char* pair_axis, const int* pos, const float* freq,
                   int interleaved, float eps) {
  RopeArgs a;
  memset(&a, 0, sizeof a);
  a.n = n;
  a.P = n_pairs;
  a.axes = n_axes;
  a.pos = pos;
  a.freq = freq;
  a.interleaved = interleaved != 0;
  a.eps = eps;
  if (pair_axis) memcpy(a.axis, pair_axis, (size_t)n_pairs);
  return a;
}

RopePart part(const void* x, void* y, const float* w, long long sx, long long sy, int H) {
  RopePart p;
  memset(&p, 0, sizeof p);
  p.x = static_cast<const bf16*>(x);
  p.y = static_cast<bf16*>(y);
  p.w = w;
  p.sx = sx;
  p.sy = sy;
  p.H = H;
  return p;
}

}  // namespace

extern "C" {

int gdn_rope_fwd(const void* q, const void* k, const float* q_weight, const float* k_weight, const int* positions,
                 const float* inv_freq, const unsigned char* pair_axis, void* q_out, void* k_out, int n, int Hq, int Hk,
                 int d, int n_axes, int n_pairs, int interleaved, float eps, long long q_stride, long long k_stride,
                 long long qo_stride, long long ko_stride, void* stream) {
  int rc = rope_check(n, Hq, Hk, d, n_axes, n_pairs, pair_axis, q_weight, k_weight, positions, inv_freq, eps);
  if (rc) return rc;
  if (!row_stride_ok(q_stride, Hq) || !row_stride_ok(k_stride, Hk) || !row_stride_ok(qo_stride, Hq) ||
      !row_stride_ok(ko_stride, Hk))
    return GDN_ERR_ARG;
  const void* ptrs[] = {q, k, q_out, k_out};
  for (const void* p : ptrs)
    if (!aligned(p, 16) || (n > 0 && !p)) return GDN_ERR_ARG;
  if (n == 0) return GDN_OK;
  RopeArgs a = rope_args(n, n_axes, n_pairs, pair_axis, positions, inv_freq, interleaved, eps);
  a.part[0] = part(q, q_out, q_weight, q_stride, qo_stride, Hq);
  a.part[1] = part(k, k_out, k_weight, k_stride, ko_stride, Hk);
  a.blocks = rope_blocks(0, n, Hq + Hk, sm_count);
  return cuda_status(launch_rope_fwd(a, static_cast<cudaStream_t>(stream)));
}

size_t gdn_rope_workspace_bytes(int n, int Hq, int Hk, int d) {
  if (rope_check(n, Hq, Hk, d, 1, 0, nullptr, nullptr, nullptr, nullptr, nullptr, 0.f) != GDN_OK) return 0;
  return up((size_t)rope_blocks(1, n, Hq + Hk, sm_count) * 2 * HD * sizeof(float));
}

int gdn_rope_bwd(const void* q, const void* k, const float* q_weight, const float* k_weight, const int* positions,
                 const float* inv_freq, const unsigned char* pair_axis, const void* dq_out, const void* dk_out, void* dq,
                 void* dk, float* dq_weight, float* dk_weight, int n, int Hq, int Hk, int d, int n_axes, int n_pairs,
                 int interleaved, float eps, long long q_stride, long long k_stride, long long dqo_stride,
                 long long dko_stride, long long dq_stride, long long dk_stride, void* ws, size_t ws_bytes,
                 void* stream) {
  int rc = rope_check(n, Hq, Hk, d, n_axes, n_pairs, pair_axis, q_weight, k_weight, positions, inv_freq, eps);
  if (rc) return rc;
  if (!row_stride_ok(q_stride, Hq) || !row_stride_ok(k_stride, Hk) || !row_stride_ok(dqo_stride, Hq) ||
      !row_stride_ok(dko_stride, Hk) || !row_stride_ok(dq_stride, Hq) || !row_stride_ok(dk_stride, Hk))
    return GDN_ERR_ARG;
  if ((dq_weight && !q_weight) || (dk_weight && !k_weight)) return GDN_ERR_ARG;
  if (!aligned(dq_weight, 4) || !aligned(dk_weight, 4) || !aligned(ws, 16)) return GDN_ERR_ARG;
  const void* ptrs[] = {dq_out, dk_out, dq, dk};
  for (const void* p : ptrs)
    if (!aligned(p, 16) || (n > 0 && !p)) return GDN_ERR_ARG;
  // (the rows themselves are read for the norms alone)
  if (!aligned(q, 16) || !aligned(k, 16) || (n > 0 && ((q_weight && !q) || (k_weight && !k)))) return GDN_ERR_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (n == 0) {
    if (dq_weight && (rc = cuda_status(cudaMemsetAsync(dq_weight, 0, HD * sizeof(float), s)))) return rc;
    return dk_weight ? cuda_status(cudaMemsetAsync(dk_weight, 0, HD * sizeof(float), s)) : GDN_OK;
  }
  RopeArgs a = rope_args(n, n_axes, n_pairs, pair_axis, positions, inv_freq, interleaved, eps);
  a.part[0] = part(q, dq, q_weight, q_stride, dq_stride, Hq);
  a.part[1] = part(k, dk, k_weight, k_stride, dk_stride, Hk);
  a.part[0].g = static_cast<const bf16*>(dq_out);
  a.part[1].g = static_cast<const bf16*>(dk_out);
  a.part[0].sg = dqo_stride;
  a.part[1].sg = dko_stride;
  a.part[0].dw = dq_weight;
  a.part[1].dw = dk_weight;
  a.blocks = rope_blocks(1, n, Hq + Hk, sm_count);
  if (dq_weight || dk_weight) {
    if (!ws || ws_bytes < gdn_rope_workspace_bytes(n, Hq, Hk, d)) return GDN_ERR_WORKSPACE;
    a.partial = static_cast<float*>(ws);
  }
  return cuda_status(launch_rope_bwd(a, s));
}

int gdn_rope_append(const void* q, const void* k, const void* v, const float* q_weight, const float* k_weight,
                    const int* positions, const float* inv_freq, const unsigned char* pair_axis, void* q_out,
                    void* k_pages, void* v_pages, const int* slots, int n, int n_pages, int page_size, int Hq, int Hk,
                    int d, int n_axes, int n_pairs, int interleaved, float eps, long long q_stride, long long k_stride,
                    long long v_stride, long long qo_stride, const gdn_page_strides* k_strides,
                    const gdn_page_strides* v_strides, void* stream) {
  int rc = rope_check(n, Hq, Hk, d, n_axes, n_pairs, pair_axis, q_weight, k_weight, positions, inv_freq, eps);
  if (rc) return rc;
  if (!row_stride_ok(q_stride, Hq) || !row_stride_ok(k_stride, Hk) || !row_stride_ok(v_stride, Hk) ||
      !row_stride_ok(qo_stride, Hq))
    return GDN_ERR_ARG;
  if ((rc = pages_check(n_pages, page_size)) || !page_strides_ok(k_strides) || !page_strides_ok(v_strides))
    return rc ? rc : GDN_ERR_ARG;
  const void* ptrs[] = {q, k, v, q_out};
  for (const void* p : ptrs)
    if (!aligned(p, 16) || (n > 0 && !p)) return GDN_ERR_ARG;
  if (!aligned(k_pages, 16) || !aligned(v_pages, 16) || (n_pages > 0 && n > 0 && (!k_pages || !v_pages)))
    return GDN_ERR_ARG;
  if (!aligned(slots, 4) || (n > 0 && !slots)) return GDN_ERR_ARG;
  if (n == 0) return GDN_OK;
  RopeArgs a = rope_args(n, n_axes, n_pairs, pair_axis, positions, inv_freq, interleaved, eps);
  a.slots = slots;
  a.pages = page_args(n_pages, page_size, 0, 0, PAGE_PIECE);
  a.cache_rows = n_pages * page_size;
  a.part[0] = part(q, q_out, q_weight, q_stride, qo_stride, Hq);
  a.part[1] = part(k, k_pages, k_weight, k_stride, k_strides->page, Hk);
  a.part[2] = part(v, v_pages, nullptr, v_stride, v_strides->page, Hk);
  a.part[1].sy_row = k_strides->row;
  a.part[1].sy_head = k_strides->head;
  a.part[2].sy_row = v_strides->row;
  a.part[2].sy_head = v_strides->head;
  a.blocks = rope_blocks(0, n, Hq + 2 * Hk, sm_count);
  return cuda_status(launch_rope_fwd(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
