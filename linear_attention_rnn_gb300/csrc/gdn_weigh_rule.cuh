// gdn_weigh_rule.cuh -- which kernels form the weights of keys in pages, and of how many CTAs: a rule of
// sizes alone, without CUDA, so that it can be compiled and run by itself.
#pragma once

#ifdef __CUDACC__
#define GDN_BOTH __host__ __device__ __forceinline__
#else
#define GDN_BOTH inline
#endif

namespace gdn {

constexpr int WEIGH_FEW_ROWS = 64;  // rows of a query tile in the kernel for few of them
constexpr int WEIGH_FEW_TILES = 4;  // to a sequence, at most

struct WeighRule {
  // Which sequences k_weigh_few takes, and which k_weigh_many: all, none, or (BY_SIZE, both) those of up
  // to WEIGH_FEW_TILES query tiles of the former and the others.
  enum { NONE, ALL, BY_SIZE };
  int few, many;
  int few_ctas;
  int ctas;   // many: teams of `split` CTAs
  int split;  // CTAs that share the queries of a key tile, 1 or 2
  GDN_BOTH static bool small(int ql, int G) {
    return G <= WEIGH_FEW_ROWS && ql <= WEIGH_FEW_TILES * WEIGH_FEW_ROWS / G;
  }
};

// total_q rows of n_seqs sequences (both above zero; alike: of one length), each of at most max_q (0: not
// known) and at most `longest` keys; key tiles and query tiles of `tile` rows.
inline WeighRule weigh_rule(int n_seqs, int total_q, int max_q, long long longest, bool alike, int Hq, int Hk, int tile,
                            long long sms) {
  WeighRule w;
  const int G = Hq / Hk;
  const long long tiles = longest > tile ? (longest + tile - 1) / tile : 1, TT = tile / G;
  const long long most_q = max_q > 0 && max_q < total_q ? max_q : total_q;
  // Sequences of up to four of its query tiles suit the kernel for few rows (16 caches of 4096 rows,
  // 16/4 heads: 64 new tokens 31 us against 37 in the other, 128 53 against 41; one of 32768 rows:
  // 22 against 25 and 33 against 27).  Where lengths may differ both are started, and each takes its
  // own (a prompt of 2048 tokens and 64 single tokens over 3000 keys: 67 us; in the kernel for few rows
  // alone 2039, in the other 474), unless so few can be short that the other kernel's start
  // takes longer (3 to 4 us; a key tile in the kernel for many rows 2.5 an SM).
  const long long few_q = G <= WEIGH_FEW_ROWS ? WEIGH_FEW_TILES * WEIGH_FEW_ROWS / G : 0;
  const bool small = WeighRule::small((int)(alike ? total_q / n_seqs : most_q), G);
  bool none = alike || few_q == 0;  // that are short
  if (!none && !small) {            // (the longest are above few_q then, as far as known)
    long long shorts = n_seqs;      // at most: the others have no more than most_q
    if (total_q > n_seqs * few_q) shorts -= (total_q - n_seqs * few_q + most_q - few_q - 1) / (most_q - few_q);
    none = shorts * tiles * Hk <= 2 * sms;
  }
  w.few = small ? WeighRule::ALL : none ? WeighRule::NONE : WeighRule::BY_SIZE;
  w.many = small ? WeighRule::NONE : none ? WeighRule::ALL : WeighRule::BY_SIZE;
  // Pairs share a key tile where one CTA would still be at the first, which sees all queries of
  // its sequence, when the others are done (in query tiles; a causal prompt has half of all): a
  // prompt of 2500 tokens, 16/4 heads, 25 us against 39, four of 1024 18 against 21, of 2500
  // 54 against 47.  With long units the smaller pieces alone win something (8192 + 640 + 77
  // tokens: 105 against 109, 16384 with 16/2 heads: 382 against 412), with short ones the pair's
  // meeting at each costs more (768 tokens, 16/16: 12.5 against 10.4).
  const long long first = most_q / TT, each = total_q / TT * tiles * Hk / 2 / sms;
  w.split = first >= 8 && (first > 2 * each || (first >= 64 && first > each)) ? 2 : 1;
  const long long units = tiles * Hk;
  // two CTAs to an SM (few), or one, but no more than there can be key tiles
  auto ctas = [&](long long most) { return (int)(units < most && units * n_seqs < most ? units * n_seqs : most); };
  w.few_ctas = ctas(2 * sms);
  w.ctas = ctas(sms / w.split);
  return w;
}

}  // namespace gdn
