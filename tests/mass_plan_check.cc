// Prints every (multiprocessors, key tiles, rows) for which a cluster of
// mla_attn_mass could own more than one key tile, or a CTA no row tile.
#include <cstdio>
#include <initializer_list>

#include "mla_mass_plan.h"

int main() {
  int bad = 0;
  for (int sms = 1; sms <= 200; ++sms)
    for (int tiles = 1; tiles <= 200; ++tiles)
      for (int rows : {129, 192, 255, 256, 511, 512, 1000, 100000}) {
        const int c = mla::mass::cluster_of(tiles, rows, sms);
        if (c != 1 && c != 2 && c != 4 && c != 8) ++bad;
        if (c == 1) continue;
        if (sms / c < tiles || (rows + 63) / 64 < c) {
          if (bad++ < 5) std::printf("sms %d tiles %d rows %d: clusters of %d\n", sms, tiles, rows, c);
        }
      }
  // a GB300's choices
  std::printf("%d %d %d %d\n", mla::mass::cluster_of(16, 512, 152), mla::mass::cluster_of(17, 512, 152),
              mla::mass::cluster_of(16, 511, 152), mla::mass::cluster_of(65, 512, 152));
  return bad != 0;
}
