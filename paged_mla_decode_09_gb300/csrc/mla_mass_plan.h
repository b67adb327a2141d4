// How many CTAs of mla_attn_mass share a key tile (host arithmetic only).
#pragma once

#include <cstdint>

namespace mla {
namespace mass {

// 1, 2, 4 or 8 CTAs for each of at most `tiles` key tiles, for `rows` query
// rows per request on a device of `sms` multiprocessors.  The grid has
// sms / cluster clusters, and a cluster that shares a key tile may own no
// second one, so cluster * tiles never exceeds sms; nor 128, as that many CTAs
// in clusters of 8 fit a GB300's groups of multiprocessors at once.  Every CTA
// gets a row tile of 64 or more.
inline int cluster_of(int64_t tiles, int64_t rows, int sms) {
  const int64_t most = sms < 128 ? sms : 128;
  int cluster = 1;
  while (cluster < 8 && 2 * cluster * tiles <= most && 2 * cluster * 64 <= rows) cluster *= 2;
  return cluster;
}

}  // namespace mass
}  // namespace mla
