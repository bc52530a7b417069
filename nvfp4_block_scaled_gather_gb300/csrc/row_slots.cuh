// The slots of shared memory that a group's rows come to in turn, and what may be on its way to them. (Plain arithmetic:
// it compiles for the host too.)
#pragma once
#include <cstdint>

#ifdef __CUDACC__
#define MOE_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define MOE_HOST_DEVICE inline
#endif

namespace moe {

// Of the rows first, first + step, ... below `rows`. A row is asked for kSlots rows ahead, into the slot that is free then;
// `bring(slot, row)` asks for one.
template <int kSlots>
struct RowSlots {
  long long step, rows;
  int slot = 0;         // of the present row
  uint32_t parity = 0;  // of its arrival

  MOE_HOST_DEVICE RowSlots(long long step, long long rows) : step(step), rows(rows) {}

  template <typename Bring>
  MOE_HOST_DEVICE void start(long long first, Bring bring) const {
    for (int i = 0; i < kSlots; ++i)
      if (first + i * step < rows) bring(i, first + i * step);
  }
  // The present row's slot has been read.
  template <typename Bring>
  MOE_HOST_DEVICE void again(long long row, Bring bring) const {
    if (row + kSlots * step < rows) bring(slot, row + kSlots * step);
  }
  MOE_HOST_DEVICE void next() {
    if (++slot == kSlots) {
      slot = 0;
      parity ^= 1u;
    }
  }
  // For a group that ends at `row`, whose arrival it gave up: `wait(slot, parity)` for every row that has been asked for
  // and not arrived.
  template <typename Wait>
  MOE_HOST_DEVICE void leave(long long row, Wait wait) {
    for (int i = 0; i < kSlots; ++i, next())
      if (row + i * step < rows) wait(slot, parity);
  }
};

}  // namespace moe
