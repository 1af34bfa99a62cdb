// gdn_ops.cu -- the extern "C" boundary of the operators around the chunked rule
// (include/gdn.h): the single-token forms, linear attention with a decay for
// each head, and causal softmax attention.  Arguments are checked on the host before anything is enqueued.
#include <stdint.h>
#include <string.h>

#include "gdn.h"
#include "gdn_kernels.cuh"
#include "gdn_tmap.cuh"

using namespace gdn;

namespace {

constexpr size_t ALIGN = 256;
inline size_t up(size_t x) { return (x + ALIGN - 1) / ALIGN * ALIGN; }
inline bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
int cuda_status(cudaError_t e) { return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA; }

template <typename T>
T* at(void* ws, size_t off) {
  return reinterpret_cast<T*>(static_cast<char*>(ws) + off);
}

int sm_count() {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms <= 0)
    sms = 152;
  return sms;
}

// rows of H heads, `stride` elements apart: whole 16-byte pieces that do not overlap
inline bool row_stride_ok(long long stride, int H) { return stride >= (long long)H * HD && stride % 8 == 0; }

// A workspace that would hold the status word alone may be left out.
constexpr size_t STATUS_BYTES = ALIGN;
inline bool workspace_ok(const void* ws, size_t ws_bytes, size_t need) {
  return ws ? ws_bytes >= need : need <= STATUS_BYTES;
}

// ---- linear attention with a decay for each head -----------------------------------
struct DecayPlan {
  int nseg, seg_chunks, slots;
  size_t status, xf, xr, accq, acck, flags, flag_bytes, total;
};

// Segments.  One CTA walks a segment of a head (three of them in the backward, for
// dq, dk and dv); without segments a call takes as long as its longest
// sequence however few CTAs there are.  With segments k and v (q and dO) are read
// twice, and two more kernels start.  The estimate, in chunks of the walk (2.7 us
// measured): equal CTAs run in rounds over the SMs, CTAs of mixed lengths take
// their average and a part of the longest one's; a CTA starts in 1.5, the fold
// takes half a chunk's time (0.57 with the third terms of a final state, which the
// estimate leaves out), the two launches together 4.
double decay_rounds(double ctas, double longest, double sms, bool mixed) {
  if (ctas <= sms) return longest;
  if (mixed) return ctas * longest / sms + 0.3 * longest;
  return (double)(long)((ctas + sms - 1.0) / sms) * longest;
}

DecayPlan decay_plan(int backward, int n_seqs, int total, int max_seqlen, int Hk, int Hv) {
  DecayPlan p;
  memset(&p, 0, sizeof p);
  const long longest = max_seqlen < total ? max_seqlen : total;
  const long nch = (longest + CH - 1) / CH;
  p.nseg = 1;
  p.seg_chunks = nch > 0 ? (int)nch : 1;
  const double sms = sm_count();
  const double all = (double)total / CH + 0.5 * n_seqs;  // chunks of all sequences
  double best = 1e300;
  for (long k = 1; k <= nch && k <= 128; ++k) {
    const double L = (double)((nch + k - 1) / k);
    const long segs = (nch + (long)L - 1) / (long)L;
    // segments that are as long as L
    const double parts = n_seqs == 1 ? (double)segs : k == 1 ? all / L : all / L + 0.25 * (n_seqs - 1);
    const bool mixed = n_seqs > 1 || backward;
    double t = decay_rounds(parts * Hv * (backward ? 3.0 : 1.0), L + 1.5, sms, mixed);
    if (segs > 1) t += decay_rounds(parts * Hv * (backward ? 2.0 : 1.0), 0.5 * L + 1.5, sms, mixed) + 4.0;
    if (t < best * 0.97) {
      best = t;
      p.nseg = (int)segs;
      p.seg_chunks = (int)L;
    }
  }
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off += up(bytes);
    return o;
  };
  p.status = take(sizeof(int));
  p.slots = n_seqs + (p.nseg > 1 ? total / (p.seg_chunks * CH) : 0);
  const size_t states = p.nseg > 1 ? (size_t)p.slots * Hv * HD * HD * sizeof(float) : 0;
  p.xf = take(states);
  if (backward) {
    p.xr = take(states);
    const size_t acc = Hv > Hk ? (size_t)total * Hk * HD * sizeof(float) : 0;
    p.accq = take(acc);
    p.acck = take(acc);
    p.flag_bytes = Hv > Hk ? (size_t)Hk * (total / CH + n_seqs) * sizeof(int) : 0;  // of dq or dk
    p.flags = take(2 * p.flag_bytes + (p.flag_bytes ? sizeof(int) : 0));  // and the count of started CTAs
  }
  p.total = off;
  return p;
}

// Final states without segments.  Where every CTA of the call finds an SM at once and
// sequences are short, they are formed in the walk's own launch: the two codes in one
// kernel cost the walk up to a tenth of its time, a launch costs the host some 4 us
// (forwards, 2 to 4 sequences of 2 to 6 chunks: 19-23 us against 24-26; of 8 and 16
// chunks: 28 and 51 us against 27 and 47).
bool one_launch(const DecayArgs& a) {
  return a.seg_chunks <= 6 && (long)(a.n_roles + 1) * a.slots * a.Hv <= sm_count();
}

// Whether two states' buffers of `bytes` share any of them.
inline bool overlap(const void* a, const void* b, size_t bytes) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a && b && (x < y ? y - x : x - y) < bytes;
}
inline size_t state_bytes(int n_seqs, int Hv) { return (size_t)n_seqs * Hv * HD * HD * sizeof(float); }

DecayFoldArgs fold_args(const DecayArgs& a) {
  DecayFoldArgs f;
  memset(&f, 0, sizeof f);
  f.decay = a.decay;
  f.cu = a.cu;
  f.status = a.status;
  f.n_seqs = a.n_seqs;
  f.total = a.total;
  f.T = a.T;
  f.Hk = a.Hk;
  f.Hv = a.Hv;
  f.nseg = a.nseg;
  f.seg_chunks = a.seg_chunks;
  f.slots = a.slots;
  return f;
}

int decay_check(int n_seqs, int total, int max_seqlen, int Hk, int Hv, int d_k, int d_v, const int* cu, long long sq,
                long long sk, long long sv) {
  if (n_seqs < 0 || total < 0 || max_seqlen < 0 || Hk <= 0 || Hv <= 0 || Hv % Hk != 0) return GDN_ERR_ARG;
  if (d_k != HD || d_v != HD) return GDN_ERR_SHAPE;
  if (!cu && n_seqs > 0 && total % n_seqs != 0) return GDN_ERR_ARG;
  // (blocks of the three passes and the final state in one grid dimension)
  if (((long long)n_seqs + total / CH) * Hv >= (1LL << 29)) return GDN_ERR_ARG;
  if (!row_stride_ok(sq, Hk) || !row_stride_ok(sk, Hk) || !row_stride_ok(sv, Hv)) return GDN_ERR_ARG;
  return GDN_OK;
}

// ---- causal softmax attention ---------------------------------------------------------
struct AttnPlan {
  int few, split_tiles, n_splits, n_parts;
  size_t status, part, part_lse, delta, total;
};

// The forward's kernel and its key splits.
//
// Calls with one query tile to a sequence on average (tokens over caches) or at most five
// key tiles (short prompts) take k_attn_split, two CTAs to an SM: 32 caches of up to
// 16214 rows 94 us against 103 in k_attn_fwd, 256 of 1024 102 against 136, 64 prompts of
// 100 tokens 22 against 32, 8 of 600 25 against 28, but 8 of 1000 52 against 47.  (The
// average is all that is known here: a long prompt among many single tokens goes the same way.)
// Its estimate, in us: memory's time for all keys (64 KiB per key tile and head, contexts
// being 0.8 of the longest one on average), or what one CTA takes by itself (1.6 a key
// tile, measured), 10 for each round of CTAs, 9 and 0.2 a split for the join and its launch.
//
// Else a CTA of k_attn_fwd holds 256 / G tokens of one key head.  The estimate, in key
// tiles of a CTA (0.8 us measured): the work of all CTAs over the SMs, contexts being
// 0.6 of the longest one on average, most of the longest CTA's behind it, 6 for a CTA's
// start and end, 4 for the join.
AttnPlan attn_plan(int backward, int n_seqs, int total_q, int max_k, int Hq, int Hk) {
  AttnPlan p;
  memset(&p, 0, sizeof p);
  const long tiles = ((long)max_k + CH - 1) / CH;
  const double ctas = (double)((long)total_q / (2 * (CH / (Hq / Hk))) + n_seqs) * Hk, sms = sm_count();
  p.split_tiles = tiles > 0 ? (int)tiles : 1;
  p.n_splits = 1;
  double best = 1e300;
  p.few = !backward && tiles > 0 && (total_q <= (long)n_seqs * (CH / (Hq / Hk)) || tiles <= 5);
  if (p.few) {
    const double heads = (double)Hk * n_seqs, all = 0.0097 * 0.8 * heads * tiles;
    for (long k = 1; k <= 64 && k <= tiles; ++k) {
      const long per = (tiles + k - 1) / k, splits = (tiles + per - 1) / per;
      const double rounds = (double)(long)(heads * splits / (2.0 * sms) + 0.999);
      const double t = (all + 0.4 * per > 1.6 * per ? all + 0.4 * per : 1.6 * per) + 10.0 * (rounds > 1.0 ? rounds : 1.0) +
                       (splits > 1 ? 9.0 + 0.2 * splits : 0.0);
      if (t < best) {
        best = t;
        p.split_tiles = (int)per;
        p.n_splits = (int)splits;
      }
    }
  }
  for (long k = 1; !backward && !p.few && k <= 64 && 4 * k <= tiles + 3; ++k) {
    const long per = (tiles + k - 1) / k, splits = (tiles + per - 1) / per;
    const double t = ctas * (0.6 * tiles + 6.0 * splits) / sms + 0.8 * (per + 6.0) + (splits > 1 ? 4.0 : 0.0);
    if (t < best * 0.97) {
      best = t;
      p.split_tiles = (int)per;
      p.n_splits = (int)splits;
    }
  }
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off += up(bytes);
    return o;
  };
  p.status = take(sizeof(int));
  const size_t rows = (size_t)total_q * Hq;
  if (backward) {
    p.delta = take(rows * sizeof(float));
  } else if (p.n_splits > 1) {
    p.n_parts = p.few ? p.n_splits : 2 * p.n_splits;
    p.part = take(rows * p.n_parts * HD * sizeof(float));
    p.part_lse = take(rows * p.n_parts * sizeof(float));
  }
  p.total = off;
  return p;
}

int attn_check(int n_seqs, int total_q, int total_k, int max_k, int Hq, int Hk, int d, const int* cu_q,
               const int* cu_k, float scale, long long sq, long long sk, long long sv) {
  if (n_seqs < 0 || total_q < 0 || total_k < 0 || max_k < 0 || Hq <= 0 || Hk <= 0 || Hq % Hk != 0) return GDN_ERR_ARG;
  if (d != HD || Hq / Hk > CH) return GDN_ERR_SHAPE;
  if (!(scale > 0.f) || scale > 1e30f) return GDN_ERR_ARG;
  if (n_seqs > 0 && ((!cu_q && total_q % n_seqs != 0) || (!cu_k && total_k % n_seqs != 0))) return GDN_ERR_ARG;
  if (!row_stride_ok(sq, Hq) || !row_stride_ok(sk, Hk) || !row_stride_ok(sv, Hk)) return GDN_ERR_ARG;
  // (blocks of one launch in one grid dimension)
  const long long tiles = (long long)total_q / (CH / (Hq / Hk)) + total_k / CH + n_seqs;
  if (tiles * Hk > (1LL << 30) || (long long)total_q * Hq > (1LL << 33)) return GDN_ERR_ARG;
  return GDN_OK;
}

// Tensor maps and the arguments that both directions share.
int attn_args(AttnArgs& a, const void* q, const void* k, const void* v, const int* cu_q, const int* cu_k, int n_seqs,
              int total_q, int total_k, int Hq, int Hk, float scale, long long sq, long long sk, long long sv,
              int key_rows = CH) {
  memset(&a, 0, sizeof a);
  a.cu_q = cu_q;
  a.cu_k = cu_k;
  a.scale = scale;
  a.n_seqs = n_seqs;
  a.total_q = total_q;
  a.total_k = total_k;
  a.Hq = Hq;
  a.Hk = Hk;
  const int G = Hq / Hk;
  if (!tmap_rows(&a.q, q, total_q, Hq, HD, (uint64_t)sq * 2, G, CH / G)) return GDN_ERR_CUDA;
  if (total_k == 0) return GDN_OK;  // (no key tile is ever loaded)
  if (!tmap_rows(&a.k, k, total_k, Hk, HD, (uint64_t)sk * 2, 1, key_rows) ||
      !tmap_rows(&a.v, v, total_k, Hk, HD, (uint64_t)sv * 2, 1, key_rows))
    return GDN_ERR_CUDA;
  return GDN_OK;
}

}  // namespace

extern "C" {

static int step(const void* q, const void* k, const void* v, const float* g, const float* beta, float* state,
                const int* slots, void* o, int R, int n_slots, int Hk, int Hv, int d_k, int d_v, long long sq,
                long long sk, long long sv, void* stream) {
  if (R < 0 || n_slots < 0 || Hk <= 0 || Hv <= 0 || Hv % Hk != 0) return GDN_ERR_ARG;
  if (d_k != HD || d_v != HD) return GDN_ERR_SHAPE;
  if ((long long)R * Hv > (1LL << 28)) return GDN_ERR_ARG;  // four blocks to a state, one grid dimension
  if (R == 0) return GDN_OK;
  if (!q || !k || !v || !g || !state || !o) return GDN_ERR_ARG;
  if (!row_stride_ok(sq, Hk) || !row_stride_ok(sk, Hk) || !row_stride_ok(sv, Hv)) return GDN_ERR_ARG;
  const void* ptrs[] = {q, k, v, g, beta, state, o};
  for (const void* p : ptrs)
    if (p && !aligned(p, 16)) return GDN_ERR_ARG;
  if (!aligned(slots, 4)) return GDN_ERR_ARG;
  StepArgs a;
  a.q = static_cast<const bf16*>(q);
  a.k = static_cast<const bf16*>(k);
  a.v = static_cast<const bf16*>(v);
  a.g = g;
  a.beta = beta;
  a.state = state;
  a.slots = slots;
  a.o = static_cast<bf16*>(o);
  a.R = R;
  a.n_slots = n_slots;
  a.sq = sq;
  a.sk = sk;
  a.sv = sv;
  a.Hk = Hk;
  a.Hv = Hv;
  return cuda_status(launch_step(a, static_cast<cudaStream_t>(stream)));
}

int gdn_delta_step(const void* q, const void* k, const void* v, const float* g, const float* beta, float* state,
                   const int* slots, void* o, int R, int n_slots, int Hk, int Hv, int d_k, int d_v,
                   long long q_stride, long long k_stride, long long v_stride, void* stream) {
  if (R > 0 && !beta) return GDN_ERR_ARG;
  return step(q, k, v, g, beta, state, slots, o, R, n_slots, Hk, Hv, d_k, d_v, q_stride, k_stride, v_stride, stream);
}

int gdn_decay_step(const void* q, const void* k, const void* v, const float* decay, float* state, const int* slots,
                   void* o, int R, int n_slots, int Hk, int Hv, int d_k, int d_v, long long q_stride,
                   long long k_stride, long long v_stride, void* stream) {
  return step(q, k, v, decay, nullptr, state, slots, o, R, n_slots, Hk, Hv, d_k, d_v, q_stride, k_stride, v_stride,
              stream);
}

size_t gdn_decay_workspace_bytes(int backward, int n_seqs, int total, int max_seqlen, int Hk, int Hv, int d_k,
                                 int d_v) {
  if (decay_check(n_seqs, total, max_seqlen, Hk, Hv, d_k, d_v, reinterpret_cast<const int*>(4), (long long)Hk * HD,
                  (long long)Hk * HD, (long long)Hv * HD) != GDN_OK)
    return 0;
  return decay_plan(backward != 0, n_seqs, total, max_seqlen, Hk, Hv).total;
}

// No rows at all: every sequence ends in the state that it began with.
static int pass_state(const float* x0, float* xT, int n_seqs, int Hv, cudaStream_t s) {
  if (!xT || xT == x0) return GDN_OK;
  const size_t bytes = state_bytes(n_seqs, Hv);
  return cuda_status(x0 ? cudaMemcpyAsync(xT, x0, bytes, cudaMemcpyDeviceToDevice, s)
                        : cudaMemsetAsync(xT, 0, bytes, s));
}

int gdn_decay_fwd(const void* q, const void* k, const void* v, const float* decay, const float* h0,
                  const int* cu_seqlens, void* o, float* hT, int n_seqs, int total, int max_seqlen, int Hk, int Hv,
                  int d_k, int d_v, long long q_stride, long long k_stride, long long v_stride, void* ws,
                  size_t ws_bytes, void* stream) {
  int rc = decay_check(n_seqs, total, max_seqlen, Hk, Hv, d_k, d_v, cu_seqlens, q_stride, k_stride, v_stride);
  if (rc) return rc;
  const void* ptrs[] = {q, k, v, h0, o, hT, ws};
  for (const void* p : ptrs)
    if (p && !aligned(p, 16)) return GDN_ERR_ARG;
  if (!aligned(decay, 4) || !aligned(cu_seqlens, 4)) return GDN_ERR_ARG;
  if (hT != h0 && overlap(hT, h0, state_bytes(n_seqs, Hv))) return GDN_ERR_ARG;
  if (n_seqs == 0) return GDN_OK;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (total == 0) return pass_state(h0, hT, n_seqs, Hv, s);
  if (!q || !k || !v || !decay || !o) return GDN_ERR_ARG;
  const DecayPlan p = decay_plan(0, n_seqs, total, max_seqlen, Hk, Hv);
  if (!workspace_ok(ws, ws_bytes, p.total)) return GDN_ERR_WORKSPACE;
  DecayArgs a;
  memset(&a, 0, sizeof a);
  a.decay = decay;
  a.cu = cu_seqlens;
  a.status = ws ? at<int>(ws, p.status) : nullptr;
  a.n_seqs = n_seqs;
  a.total = total;
  a.T = total / n_seqs;
  a.Hk = Hk;
  a.Hv = Hv;
  a.nseg = p.nseg;
  a.seg_chunks = p.seg_chunks;
  a.slots = p.slots;
  a.n_roles = 1;
  DecayRole& r = a.role[0];
  if (!tmap_rows(&r.a, q, total, Hk, HD, (uint64_t)q_stride * 2, 1, CH) ||
      !tmap_rows(&r.b, k, total, Hk, HD, (uint64_t)k_stride * 2, 1, CH) ||
      !tmap_rows(&r.c, v, total, Hv, HD, (uint64_t)v_stride * 2, 1, CH) ||
      !tmap_rows(&r.o, o, total, Hv, HD, (uint64_t)Hv * HD * 2, 1, CH))
    return GDN_ERR_CUDA;
  r.hc = 1;
  r.x0 = h0;
  r.out = static_cast<bf16*>(o);
  DecayFoldArgs f = fold_args(a);
  f.n_roles = 1;
  f.role[0].b = r.b;
  f.role[0].c = r.c;
  f.role[0].x0 = h0;
  f.role[0].last = hT;
  if (p.nseg > 1) {
    f.role[0].x = at<float>(ws, p.xf);
    if ((rc = cuda_status(launch_decay_fold(f, s)))) return rc;
    r.xseg = f.role[0].x;
  }
  // The final states, with one segment.  Written over the entering ones they come behind
  // the walk, which reads those; else beside it.  (With segments the prefix kernel reads
  // each value before it writes it, and the walk reads the workspace.)
  const bool last = p.nseg == 1 && hT, in_place = hT && hT == h0;
  f.n_roles = last && !in_place && one_launch(a);
  if ((rc = cuda_status(launch_decay(a, f, s))) || !last || f.n_roles) return rc;
  f.n_roles = 1;
  f.beside = !in_place;
  f.behind = in_place;
  return cuda_status(launch_decay_fold(f, s));
}

int gdn_decay_bwd(const void* q, const void* k, const void* v, const float* decay, const float* h0, const void* dO,
                  const float* dhT, const int* cu_seqlens, void* dq, void* dk, void* dv, float* dh0, int n_seqs,
                  int total, int max_seqlen, int Hk, int Hv, int d_k, int d_v, long long q_stride,
                  long long k_stride, long long v_stride, void* ws, size_t ws_bytes, void* stream) {
  int rc = decay_check(n_seqs, total, max_seqlen, Hk, Hv, d_k, d_v, cu_seqlens, q_stride, k_stride, v_stride);
  if (rc) return rc;
  const void* ptrs[] = {q, k, v, h0, dO, dhT, dq, dk, dv, dh0, ws};
  for (const void* p : ptrs)
    if (p && !aligned(p, 16)) return GDN_ERR_ARG;
  if (!aligned(decay, 4) || !aligned(cu_seqlens, 4)) return GDN_ERR_ARG;
  if (dh0 != dhT && overlap(dh0, dhT, state_bytes(n_seqs, Hv))) return GDN_ERR_ARG;
  if (overlap(dh0, h0, state_bytes(n_seqs, Hv))) return GDN_ERR_ARG;
  if (n_seqs == 0) return GDN_OK;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (total == 0) return pass_state(dhT, dh0, n_seqs, Hv, s);
  if (!q || !k || !v || !decay || !dO || !dq || !dk || !dv) return GDN_ERR_ARG;
  const DecayPlan p = decay_plan(1, n_seqs, total, max_seqlen, Hk, Hv);
  if (!workspace_ok(ws, ws_bytes, p.total)) return GDN_ERR_WORKSPACE;
  DecayArgs a;
  memset(&a, 0, sizeof a);
  a.decay = decay;
  a.cu = cu_seqlens;
  a.status = ws ? at<int>(ws, p.status) : nullptr;
  a.n_seqs = n_seqs;
  a.total = total;
  a.T = total / n_seqs;
  a.Hk = Hk;
  a.Hv = Hv;
  a.nseg = p.nseg;
  a.seg_chunks = p.seg_chunks;
  a.slots = p.slots;
  a.n_roles = 3;
  CUtensorMap mq, mk, mv, md;
  if (!tmap_rows(&mq, q, total, Hk, HD, (uint64_t)q_stride * 2, 1, CH) ||
      !tmap_rows(&mk, k, total, Hk, HD, (uint64_t)k_stride * 2, 1, CH) ||
      !tmap_rows(&mv, v, total, Hv, HD, (uint64_t)v_stride * 2, 1, CH) ||
      !tmap_rows(&md, dO, total, Hv, HD, (uint64_t)Hv * HD * 2, 1, CH))
    return GDN_ERR_CUDA;
  DecayRole &rq = a.role[0], &rk = a.role[1], &rv = a.role[2];
  rq.a = md, rq.b = mv, rq.c = mk;
  rq.ha = rq.hb = 1;
  rq.xt = 1;
  rq.shared = 1;
  rq.x0 = h0;
  if (Hv > Hk) {
    rq.acc = at<float>(ws, p.accq);
    rq.flags = at<int>(ws, p.flags);
    a.ticket = rq.flags + 2 * p.flag_bytes / sizeof(int);
    if ((rc = cuda_status(cudaMemsetAsync(rq.flags, 0, 2 * p.flag_bytes + sizeof(int), s)))) return rc;
  }
  rq.out = static_cast<bf16*>(dq);
  rk.a = mv, rk.b = md, rk.c = mq;
  rk.ha = rk.hb = 1;
  rk.rev = 1;
  rk.xt = 1;
  rk.shared = 1;
  rk.x0 = dhT;
  if (Hv > Hk) {
    rk.acc = at<float>(ws, p.acck);
    rk.flags = rq.flags + p.flag_bytes / sizeof(int);
  }
  rk.out = static_cast<bf16*>(dk);
  rv.a = mk, rv.b = mq, rv.c = md;
  rv.hc = 1;
  rv.rev = 1;
  rv.x0 = dhT;
  rv.out = static_cast<bf16*>(dv);
  if (!tmap_rows(&rq.o, dq, total, Hk, HD, (uint64_t)Hk * HD * 2, 1, CH) ||
      !tmap_rows(&rk.o, dk, total, Hk, HD, (uint64_t)Hk * HD * 2, 1, CH) ||
      !tmap_rows(&rv.o, dv, total, Hv, HD, (uint64_t)Hv * HD * 2, 1, CH))
    return GDN_ERR_CUDA;
  DecayFoldArgs f = fold_args(a);
  DecayFoldRole &ff = f.role[0], &fr = f.role[1];
  ff.b = mk;
  ff.c = mv;
  ff.x0 = h0;
  fr.b = mq;
  fr.c = md;
  fr.rev = 1;
  fr.x0 = dhT;
  fr.last = dh0;
  if (p.nseg > 1) {
    f.n_roles = 2;
    ff.x = at<float>(ws, p.xf);
    fr.x = at<float>(ws, p.xr);
    if ((rc = cuda_status(launch_decay_fold(f, s)))) return rc;
    rq.xseg = ff.x;
    rk.xseg = rv.xseg = fr.x;
  }
  const bool last = p.nseg == 1 && dh0, in_place = dh0 && dh0 == dhT;  // (as in the forward)
  f.role[0] = fr;
  f.n_roles = last && !in_place;
  if (f.n_roles && !one_launch(a)) {
    // ahead of the walk: its CTAs are short, and behind the walk's they would start
    // only when the last of those has
    if ((rc = cuda_status(launch_decay_fold(f, s)))) return rc;
    a.beside = 1;
    f.n_roles = 0;
  }
  if ((rc = cuda_status(launch_decay(a, f, s))) || !last || !in_place) return rc;
  f.n_roles = 1;
  f.behind = 1;
  return cuda_status(launch_decay_fold(f, s));
}

size_t gdn_attn_workspace_bytes(int backward, int n_seqs, int total_q, int total_k, int max_k, int Hq, int Hk,
                                int d) {
  const int* some = reinterpret_cast<const int*>(4);
  if (attn_check(n_seqs, total_q, total_k, max_k, Hq, Hk, d, some, some, 1.f, (long long)Hq * HD, (long long)Hk * HD,
                 (long long)Hk * HD) != GDN_OK)
    return 0;
  return attn_plan(backward != 0, n_seqs, total_q, max_k < total_k ? max_k : total_k, Hq, Hk).total;
}

int gdn_attn_fwd(const void* q, const void* k, const void* v, const int* cu_q, const int* cu_k, const int* k_len,
                 void* o, float* lse, int n_seqs, int total_q, int total_k, int max_k, int Hq, int Hk, int d,
                 float scale, long long q_stride, long long k_stride, long long v_stride, void* ws, size_t ws_bytes,
                 void* stream) {
  int rc = attn_check(n_seqs, total_q, total_k, max_k, Hq, Hk, d, cu_q, cu_k, scale, q_stride, k_stride, v_stride);
  if (rc) return rc;
  const void* ptrs[] = {q, k, v, o, ws};
  for (const void* p : ptrs)
    if (p && !aligned(p, 16)) return GDN_ERR_ARG;
  if (!aligned(cu_q, 4) || !aligned(cu_k, 4) || !aligned(k_len, 4) || !aligned(lse, 4)) return GDN_ERR_ARG;
  if (n_seqs == 0 || total_q == 0) return GDN_OK;
  if (!q || !o || (total_k > 0 && (!k || !v))) return GDN_ERR_ARG;
  const AttnPlan p = attn_plan(0, n_seqs, total_q, max_k < total_k ? max_k : total_k, Hq, Hk);
  if (!workspace_ok(ws, ws_bytes, p.total)) return GDN_ERR_WORKSPACE;
  AttnArgs a;
  if ((rc = attn_args(a, q, k, v, cu_q, cu_k, n_seqs, total_q, total_k, Hq, Hk, scale, q_stride, k_stride, v_stride,
                      p.few ? CH / 2 : CH)))
    return rc;
  if (!tmap_rows(&a.mo, o, total_q, Hq, HD, (uint64_t)Hq * HD * 2, Hq / Hk, CH / (Hq / Hk))) return GDN_ERR_CUDA;
  a.k_len = k_len;
  a.o = static_cast<bf16*>(o);
  a.lse = lse;
  a.status = ws ? at<int>(ws, p.status) : nullptr;
  a.split_tiles = p.split_tiles;
  a.n_splits = p.n_splits;
  a.n_parts = p.n_parts;
  a.part = at<float>(ws, p.part);
  a.part_lse = at<float>(ws, p.part_lse);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return cuda_status(p.few ? launch_attn_split(a, s) : launch_attn_fwd(a, s));
}

int gdn_attn_bwd(const void* q, const void* k, const void* v, const void* o, const float* lse, const void* dO,
                 const int* cu_q, const int* cu_k, void* dq, void* dk, void* dv, int n_seqs, int total_q, int total_k,
                 int Hq, int Hk, int d, float scale, long long q_stride, long long k_stride, long long v_stride,
                 void* ws, size_t ws_bytes, void* stream) {
  int rc = attn_check(n_seqs, total_q, total_k, 0, Hq, Hk, d, cu_q, cu_k, scale, q_stride, k_stride, v_stride);
  if (rc) return rc;
  const void* ptrs[] = {q, k, v, o, dO, dq, dk, dv, ws};
  for (const void* p : ptrs)
    if (p && !aligned(p, 16)) return GDN_ERR_ARG;
  if (!aligned(cu_q, 4) || !aligned(cu_k, 4) || !aligned(lse, 4)) return GDN_ERR_ARG;
  if (n_seqs == 0) return GDN_OK;
  if (total_q > 0 && (!q || !o || !lse || !dO || !dq)) return GDN_ERR_ARG;
  if (total_k > 0 && (!k || !v || !dk || !dv)) return GDN_ERR_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (total_q == 0 || total_k == 0) {  // no pair of a query and a key: zero gradients
    const size_t nq = (size_t)total_q * Hq * HD * sizeof(bf16), nk = (size_t)total_k * Hk * HD * sizeof(bf16);
    if (nq && (rc = cuda_status(cudaMemsetAsync(dq, 0, nq, s)))) return rc;
    if (nk && (rc = cuda_status(cudaMemsetAsync(dk, 0, nk, s)))) return rc;
    return nk ? cuda_status(cudaMemsetAsync(dv, 0, nk, s)) : GDN_OK;
  }
  const AttnPlan p = attn_plan(1, n_seqs, total_q, total_k, Hq, Hk);
  if (!workspace_ok(ws, ws_bytes, p.total)) return GDN_ERR_WORKSPACE;
  AttnArgs a;
  if ((rc = attn_args(a, q, k, v, cu_q, cu_k, n_seqs, total_q, total_k, Hq, Hk, scale, q_stride, k_stride, v_stride)))
    return rc;
  if (!tmap_rows(&a.dO, dO, total_q, Hq, HD, (uint64_t)Hq * HD * 2, Hq / Hk, CH / (Hq / Hk)) ||
      !tmap_rows(&a.mo, dq, total_q, Hq, HD, (uint64_t)Hq * HD * 2, Hq / Hk, CH / (Hq / Hk)) ||
      !tmap_rows(&a.mdk, dk, total_k, Hk, HD, (uint64_t)Hk * HD * 2, 1, CH) ||
      !tmap_rows(&a.mdv, dv, total_k, Hk, HD, (uint64_t)Hk * HD * 2, 1, CH))
    return GDN_ERR_CUDA;
  a.lse = const_cast<float*>(lse);
  a.dOp = static_cast<const bf16*>(dO);
  a.op = static_cast<const bf16*>(o);
  a.pq = static_cast<const bf16*>(q);
  a.pk = static_cast<const bf16*>(k);
  a.pv = static_cast<const bf16*>(v);
  a.sq = q_stride;
  a.sk = k_stride;
  a.sv = v_stride;
  a.delta = at<float>(ws, p.delta);
  a.dq = static_cast<bf16*>(dq);
  a.dk = static_cast<bf16*>(dk);
  a.dv = static_cast<bf16*>(dv);
  a.status = ws ? at<int>(ws, p.status) : nullptr;
  return cuda_status(launch_attn_bwd(a, s));
}

}  // extern "C"
