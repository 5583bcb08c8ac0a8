// qcast_stages.h -- how rows of x that do not fit LDS at once come in stages of
// it (matvec.hip). Plain C++, the same on the host, which sizes the launch, and
// in the kernel, whose loop over the stages ends only where one holds something.
//
// x is counted in units of k; a row of a stage takes `unit_bytes` a unit (its
// values and their scales) and 16 bytes more. The waves that share a column tile
// go through a stage in rounds: every wave's turns in flight.
#pragma once

#include <stdint.h>

namespace qcast {

// Units of a stage for `rows` rows in `lds` bytes: all of them, or as many whole
// rounds as fit. 0 where not one does.
constexpr uint32_t stage_units(uint32_t lds, uint32_t rows, uint32_t unit_bytes, uint32_t round,
                               uint32_t units) {
  const uint32_t of_row = lds / rows;
  const uint32_t most = of_row < 16 ? 0 : (of_row - 16) / unit_bytes;
  return most < units ? most / round * round : units;
}

// `waves` halved until a round of theirs, `units_of_wave` units each, fits a stage;
// one wave at least, whether its own fits or not.
constexpr uint32_t stage_waves(uint32_t lds, uint32_t rows, uint32_t unit_bytes,
                               uint32_t units_of_wave, uint32_t waves) {
  while (waves > 1 && stage_units(lds, rows, unit_bytes, waves * units_of_wave, ~0u) == 0)
    waves /= 2;
  return waves;
}

}  // namespace qcast
