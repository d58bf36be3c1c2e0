// Which of the two attention kernels a prefix call takes.  Plain C++, so that the
// rule is also checked on the host.
#pragma once

#include <algorithm>

namespace sv {

struct PrefixKernels {
  bool rows;   // the row kernel: entries of `unit` rows per KV head at most, where it is in the call
  bool tiles;  // the tile kernel: all others
};

// One of them at least, as max_tokens is: without the first, an entry of a token or
// more may have more than `unit` rows, so the second is in the call.  The row kernel
// stays out where every sequence has more: where the shortest does, the others being at
// their longest.  Token rows may lie behind the last sequence, so what is left of
// `total_tokens` for the shortest says no more than max_tokens: a padded step of single
// tokens stays in the row kernel.  (Padded chunks may leave it, with the short
// sequences among them.)
inline PrefixKernels prefix_kernels(long long total_tokens, long long batch, long long max_tokens,
                                    long long group_tokens, long long heads_per_kv, long long unit) {
  const long long shortest = std::min(max_tokens, total_tokens - (batch - 1) * max_tokens);
  const long long most = std::max(group_tokens, max_tokens) * heads_per_kv;
  return {heads_per_kv <= unit && shortest * heads_per_kv <= unit, most > unit};
}

}  // namespace sv
