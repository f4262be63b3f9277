// Host program for tests/test_rotary_turn_host.py: the fraction of a turn of positions and frequencies, against the
// product in 128 bits.  Built with the sanitizer of signed overflow, which ends the program.
#include <cstdio>

#include "spa_rotary_turn.h"

int main() {
  const int32_t positions[] = {0, 1, -1, 5, -5, 4097, 1 << 20, -(1 << 20), 1 << 30, 0x7fffffff, -0x7fffffff - 1};
  uint64_t x = 0x9e3779b97f4a7c15ull;
  long long checked = 0;
  for (int k = 0; k < 200000; ++k) {
    x ^= x << 13, x ^= x >> 7, x ^= x << 17;
    const int64_t turns = k < 4 ? (int64_t[]){0, -1, INT64_MIN, INT64_MAX}[k] : (int64_t)(x >> (k % 40)) * (k % 2 ? 1 : -1);
    for (const int32_t p : positions) {
      const __int128 full = (__int128)p * turns;                      // (at most 2^94)
      const int64_t low = (int64_t)(uint64_t)(unsigned __int128)full; // modulo 2^64, in turns of 2^64 parts
      if (spa::turn_of(p, turns) != (int32_t)(low >> 32)) {
        std::printf("differs at %d %lld\n", p, (long long)turns);
        return 1;
      }
      ++checked;
    }
  }
  std::printf("ok %lld\n", checked);
  return 0;
}
