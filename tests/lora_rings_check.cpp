// Host model of the code units' pipeline in k_lora_tc (lora_rings.h): a producer fills slots in order,
// copies land in any order, two groups take the units in turn and wait by parity, the consumer frees
// operand stages in order.  Counts the waits that return before the unit's own copy has landed, and the
// runs that come to a stop.  Built and run by test_lora_rings_cpu.py.
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>
#include "lora_rings.h"

struct Result { long early, stuck; };

// slots, barriers, and how many units the operand ring holds
Result model(int slots, int barriers, int ahead, int units, unsigned seed) {
  std::mt19937 rng(seed);
  std::vector<int> full(barriers), freed(slots);      // completed phases
  std::vector<char> landed(units), written(units);
  int issued = 0, consumed = 0, next[2] = {0, 1};
  Result r{0, 0};
  auto passes = [](int phases, int parity) { return (phases & 1) != parity; };   // an mbarrier's parity wait
  while (next[0] < units || next[1] < units) {
    std::vector<int> moves;
    if (issued < units && passes(freed[issued % slots], ((issued / slots) & 1) ^ 1)) moves.push_back(0);
    for (int u = 0; u < issued; ++u)
      if (!landed[u]) moves.push_back(10 + u);
    for (int g = 0; g < 2; ++g) {
      const int u = next[g];
      // (the operand ring's own waits are exact: its barriers complete in order)
      if (u < units && passes(full[u % barriers], (u / barriers) & 1) && u < consumed + ahead)
        moves.push_back(1 + g);
    }
    if (consumed < units && written[consumed]) moves.push_back(3);
    if (moves.empty()) { ++r.stuck; break; }
    const int m = moves[rng() % moves.size()];
    if (m == 0) ++issued;
    else if (m == 3) ++consumed;
    else if (m >= 10) { landed[m - 10] = 1; ++full[(m - 10) % barriers]; }
    else {
      const int u = next[m - 1];
      if (!landed[u]) { ++r.early; break; }
      written[u] = 1;
      ++freed[u % slots];
      next[m - 1] += 2;
    }
  }
  return r;
}

int main() {
  long bad = 0, odd = 0;
  for (int slots : {gptq::kLoraCodeSlotsForward, gptq::kLoraCodeSlotsBackward})
    for (int ahead : {3, 4})          // 6 stages (256 tokens) and 8 (128), two a unit
      for (unsigned seed = 0; seed < 20000; ++seed) {
        const Result r = model(slots, gptq::lora_code_barriers(slots), ahead, 24, seed);
        bad += r.early + r.stuck;
      }
  // the model finds the fault that the rule avoids: three slots with a barrier each
  for (unsigned seed = 0; seed < 20000; ++seed) odd += model(3, 3, 4, 24, seed).early;
  printf("bad=%ld odd_found=%d\n", bad, odd > 0);
  return bad != 0 || odd == 0;
}
