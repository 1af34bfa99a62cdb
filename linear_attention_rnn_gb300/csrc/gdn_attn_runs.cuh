// gdn_attn_runs.cuh -- who computes what in attention over pages.
//
// An item is a stretch of S tokens of a sequence, for one key head, against the keys that
// they see.  The keys of all items, laid one behind another (by sequence, key head and
// stretch), are cut into equal runs, one to each CTA, whatever the lengths are.  An item
// that lies in one run is that CTA's alone; of one that is cut every CTA computes a part,
// its key tiles, and the parts are joined in their order.
//
// Runs are measured in keys, with EXTRA of them for an item's start and end, and cut at
// multiples of 128 keys, so that sums in closed form say where a run begins.  One warp plans:
// it writes the items of its CTA's run to shared memory, some at a time.
#pragma once
#include "gdn_attn.cuh"

namespace gdn {
namespace attn {

struct Item {
  int seq, kh;
  int row, toks;   // its first token's row of q, its tokens
  int kl, lim;     // the sequence's keys; the last key that the first token sees
  int kb, ke;      // key tiles of the CTA's part
  int whole;       // the part is the item
  int slot;        // where a part's output goes: 2 CTA, or 2 CTA + 1 if the item begins in this run
};
// What the join of an item needs, written by the CTA in whose run it begins (parts: none, or
// one in this CTA and one in every CTA up to `last`).
struct Join {
  int row, toks, kh, last;
};

// A sequence's items.
template <int EXTRA>
struct Stretches {
  int off, kl, n, S, flat;  // flat: items ahead of the first that sees a key (but not the last item)
  __device__ __forceinline__ Stretches(int ql, int keys, int s) : off(keys - ql), kl(keys), n((ql + s - 1) / s), S(s) {
    flat = off >= 0 ? 0 : min(n - 1, (int)((unsigned)-off / (unsigned)S));
  }
  __device__ __forceinline__ int keys(int i) const { return i + 1 >= n ? kl : max(0, off + (i + 1) * S); }
  __device__ __forceinline__ int width(int i) const { return EXTRA + keys(i); }
  // widths of the first i items, i < n
  __device__ __forceinline__ long before(int i) const {
    const long w = (long)i * EXTRA;
    return i <= flat ? w : w + (long)(i - flat) * off + S * ((long)(flat + 1 + i) * (i - flat) / 2);
  }
  __device__ __forceinline__ long total() const { return n > 0 ? before(n - 1) + width(n - 1) : 0; }
  // key tiles ahead of place x of an item that is `wide`
  __device__ __forceinline__ int tiles(int x, int wide) const {
    return x >= wide ? (wide - EXTRA + CH - 1) / CH : max(0, x - EXTRA) / CH;
  }
};

template <int N>
struct RunsSmem {
  Item item[N];
  int count, more;
};

// The plan of one CTA's run, walked by one warp; the lengths of 32 sequences lie in its lanes.
template <int EXTRA>
struct Planner {
  typedef Stretches<EXTRA> Seqs;
  const AttnArgs& a;
  const int S;
  int s0, lane_q0, lane_ql, lane_kl;
  long each, longer;     // width of a run; runs that are wider by one
  long left;             // width of what is left of this one
  int ctas;              // that have a run
  int seq, kh, i, x0;    // the next item, where the run begins in it
  int q0, ql, kl;        // its sequence

  __device__ __forceinline__ Planner(const AttnArgs& args, int s) : a(args), S(s), s0(-32) {}
  __device__ __forceinline__ long begin(int c) const { return each * c + min((long)c, longer); }
  __device__ __forceinline__ int keys(int s) const { return min(max(a.k_len[s], 0), a.pages.capacity); }
  __device__ __forceinline__ void read(int from) {
    s0 = from;
    const int s = s0 + (threadIdx.x & 31);
    lane_q0 = lane_ql = lane_kl = 0;
    if (s < a.n_seqs) {
      const int2 q = rows_of(a.cu_q, s, a.n_seqs, a.total_q);
      lane_q0 = q.x;
      lane_ql = q.y;
      lane_kl = keys(s);
    }
  }
  __device__ __forceinline__ void take() {
    q0 = __shfl_sync(0xffffffffu, lane_q0, seq - s0);
    ql = __shfl_sync(0xffffffffu, lane_ql, seq - s0);
    kl = __shfl_sync(0xffffffffu, lane_kl, seq - s0);
  }
  // inclusive sums over the lanes
  static __device__ __forceinline__ long sums(long v) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long y = (long)__shfl_up_sync(0xffffffffu, (unsigned long long)v, o);
      if ((threadIdx.x & 31) >= o) v += y;
    }
    return v;
  }
  static __device__ __forceinline__ long from(long v, int lane) {
    return (long)__shfl_sync(0xffffffffu, (unsigned long long)v, lane);
  }
  // The run of CTA `cta` of `most`; fewer have one where it would be narrower than `narrow`.  A lane
  // adds up a 32nd of the sequences, one behind another, so that their lengths are asked for at
  // once (32 at a time, one after another, 256 tokens over 1024 keys each took 104 us for 98, 1000
  // over 300 153 for 129).
  __device__ __forceinline__ void start(int cta, int most_ctas, int narrow) {
    const int lane = threadIdx.x & 31, block = (a.n_seqs + 31) / 32;
    long mine = 0;
    if (block == 1) {
      read(0);
      mine = Seqs(lane_ql, lane_kl, S).total();
    } else {
#pragma unroll 4
      for (int i = 0; i < block; ++i) {
        const int s = min(lane * block + i, a.n_seqs - 1);
        const int ql = rows_of(a.cu_q, s, a.n_seqs, a.total_q).y, kl = keys(s);
        if (lane * block + i < a.n_seqs) mine += Seqs(ql, kl, S).total();
      }
    }
    long upto = sums(mine * a.Hk);
    const long all = from(upto, 31);
    ctas = all >= (long)narrow * most_ctas ? most_ctas : max(1, (int)((unsigned)all / (unsigned)narrow));
    each = all >> 32 ? all / ctas : (long)((unsigned)all / (unsigned)ctas);  // (the short division where it does)
    longer = all - each * ctas;
    const long lo = begin(cta);
    left = cta < ctas ? begin(cta + 1) - lo : 0;
    if (left <= 0) return;
    // the lane, or behind it the sequence of its block, in which the run begins
    int l = __ffs((int)__ballot_sync(0xffffffffu, upto > lo)) - 1;
    long ahead = from(upto - mine * a.Hk, l);
    seq = l;
    if (block > 1) {
      for (int s = l * block;; s += 32) {
        read(s);
        mine = s + lane < a.n_seqs ? Seqs(lane_ql, lane_kl, S).total() : 0;
        upto = ahead + sums(mine * a.Hk);
        const unsigned past = __ballot_sync(0xffffffffu, upto > lo);
        if (past) {
          l = __ffs((int)past) - 1;
          ahead = from(upto - mine * a.Hk, l);
          seq = s + l;
          break;
        }
        ahead = from(upto, 31);
      }
    }
    take();
    const Seqs it(ql, kl, S);
    const long one = it.total();
    long in = lo - ahead;
    kh = 0;
    while (in >= one) {  // (a few heads)
      in -= one;
      ++kh;
    }
    int b = 0, e = it.n;  // before(b) <= in < before(e)
    while (e - b > 1) {
      const int m = (b + e) >> 1;
      if (it.before(m) <= in)
        b = m;
      else
        e = m;
    }
    i = b;
    x0 = (int)(in - it.before(b));
  }
  // The next N items of the run (or those that are left); those without work for this CTA are
  // left out.
  template <int N>
  __device__ __forceinline__ void fill(RunsSmem<N>& sm, Join* joins, int cta) {
    const int lane = threadIdx.x & 31;
    int count = 0;
    while (left > 0 && count < N) {
      const Seqs it(ql, kl, S);
      const int wide = it.width(i), x1 = (int)min((long)wide, x0 + left);
      Item o;
      o.seq = seq;
      o.kh = kh;
      o.row = q0 + i * S;
      o.toks = min(S, ql - i * S);
      o.kl = kl;
      o.lim = i * S + kl - ql;
      o.kb = it.tiles(x0, wide);
      o.ke = it.tiles(x1, wide);
      o.whole = 1;
      o.slot = 2 * cta + (x0 > 0 ? 0 : 1);
      bool mine = true;
      if (x0 > 0 || x1 < wide) {
        // the last run that the item lies in: where that has all key tiles, the item is its alone
        const long begins = (x0 > 0 ? begin(cta) : begin(cta + 1) - x1 + x0) - x0;
        int last = cta;
        while (last + 1 < ctas && begin(last + 1) < begins + wide) ++last;
        const bool alone = it.tiles((int)max(0L, begin(last) - begins), wide) == 0;
        o.whole = alone;
        mine = !alone || last == cta;
        if (mine && !alone && x0 == 0 && lane == 0) joins[cta] = Join{o.row, o.toks, kh, last};
      }
      if (mine) {
        if (lane == 0) sm.item[count] = o;
        ++count;
      }
      left -= x1 - x0;
      x0 = 0;
      if (left <= 0) break;
      if (++i < it.n) continue;
      i = 0;
      if (++kh < a.Hk) continue;
      kh = 0;
      do {  // (a later sequence has items, since something is left)
        if (++seq == s0 + 32) read(seq);
        take();
      } while (ql == 0);
    }
    if (lane == 0) {
      sm.count = count;
      sm.more = left > 0;
    }
  }
};

}  // namespace attn
}  // namespace gdn
