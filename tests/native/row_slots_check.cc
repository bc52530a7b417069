// Rows through RowSlots<kSlots> with a barrier for each slot as the hardware has them, for every number of rows and every
// row whose arrival is given up. Fails where a slot is asked for before its last row arrived or was read, where a wait is
// for another row than the one on its way, and where a group ends with a copy in flight that it has not waited for.
#include <cstdio>
#include <initializer_list>
#include <set>
#include <string>

#include "row_slots.cuh"

static int failures = 0, runs = 0;
static void check(bool ok, const char* what, long long rows, long long step, long long fails) {
  static std::set<std::string> seen;
  if (!ok) ++failures;
  if (!ok && seen.insert(what).second) std::printf("%s: %lld rows, step %lld, row %lld gives up\n", what, rows, step, fails);
}

template <int kSlots>
static void run(long long first, long long step, long long rows, long long fails) {
  struct {
    long long row = -1;  // asked for, not known to have arrived
    uint32_t phase = 0;
    bool read = true;
  } bars[kSlots];
  ++runs;
  auto bring = [&](int slot, long long row) {
    check(row < rows, "a row past the last one", rows, step, fails);
    check(bars[slot].row < 0 && bars[slot].read, "a slot that is in use", rows, step, fails);
    bars[slot].row = row;
    bars[slot].read = false;
  };
  long long waits = 0;
  auto arrived = [&](int slot, uint32_t parity, long long row) {
    check(bars[slot].row == row && bars[slot].phase == parity, "a wait for another row", rows, step, fails);
    bars[slot].row = -1;
    bars[slot].phase ^= 1u;
    ++waits;
  };
  moe::RowSlots<kSlots> s(step, rows);
  s.start(first, bring);
  for (long long row = first; row < rows; row += step) {
    if (row == fails) {
      long long next = row;
#ifndef WITHOUT_LEAVING
      s.leave(row, [&](int slot, uint32_t parity) {
        arrived(slot, parity, next);
        next += step;
      });
      break;
#endif
    } else {
      arrived(s.slot, s.parity, row);
    }
    bars[s.slot].read = true;
    s.again(row, bring);
    s.next();
  }
  for (auto& b : bars) check(b.row < 0, "a copy in flight at the end", rows, step, fails);
  if (fails < 0) check(waits == (rows > first ? (rows - first + step - 1) / step : 0), "a row left out", rows, step, fails);
}

int main() {
  for (long long rows = 0; rows < 40; ++rows)
    for (long long step : {1, 3, 7})
      for (long long first = 0; first < step; ++first) {
        run<2>(first, step, rows, -1);
        run<3>(first, step, rows, -1);
        for (long long fails = first; fails < rows; fails += step) {
          run<2>(first, step, rows, fails);
          run<3>(first, step, rows, fails);
        }
      }
  std::printf("%d runs, %d failures\n", runs, failures);
  return failures != 0;
}
