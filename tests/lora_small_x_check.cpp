// Host check of k_lora_small's look-ahead loads (lora_small_x.h): no lane reads behind its token's row
// (the last row ends where the caller's X may end), and every piece that is multiplied is the right one.
// Built and run by test_lora_small_x_cpu.py.
#define __host__
#define __device__
#include <cstdio>
#include <initializer_list>
#include "lora_small_x.h"

int main() {
  long outside = 0, wrong = 0;
  for (int d = 8; d <= 1536; d += 8) {
    const int steps = (d + 127) / 128, ragged = d % 128 ? steps - 1 : -1;
    for (int s0 = 0; s0 < steps; ++s0)
      for (int s1 = s0 + 1; s1 <= steps; ++s1)
        for (int xa : {1, 3})        // pieces ahead, with more and with up to 8 tokens
          for (int t4 = 0; t4 < 4; ++t4) {
            int held[4];             // columns of the pieces that a lane holds, -2: zeros
            auto load = [&](int s, int q) {
              const int at = gptq::small_x_piece(d, s, q, s1, ragged, t4);
              const int column = s * 128 + t4 * 32 + 8 * at;
              if (at >= 0 && column + 8 > d) ++outside;
              held[q % (xa + 1)] = at < 0 ? -2 : column;
            };
            for (int q = 0; q < xa; ++q) load(s0, q);
            for (int s = s0; s < s1; ++s)
              for (int q = 0; q < 4; ++q) {
                load(s, q + xa);
                const int want = s * 128 + t4 * 32 + 8 * q;
                if (held[q % (xa + 1)] != (want < d ? want : -2)) ++wrong;
              }
          }
  }
  printf("outside=%ld wrong=%ld\n", outside, wrong);
  return outside != 0 || wrong != 0;
}
