// ring.h -- what a CTA that walks rows through a ring of shared-memory stages
// has to wait for before it leaves, at whatever row it does.  Plain C++: the
// host tests walk it.
#pragma once

#include <cstdint>

#include "hb_internal.h"

namespace hb {

// Row i goes to stage i % stages and completes that stage's phase i / stages.
// `stages` rows are asked for at first, and one more each time a row has been
// read, as long as there are any.
struct RowRing {
  int stages;
  int issued;    // rows asked for

  // a walk of `rows` rows that was left while row k was read (k = rows: at its end)
  HB_HD RowRing(int stages_, int rows, int k)
      : stages(stages_), issued(rows < k + stages_ ? rows : k + stages_) {}
  // stages that have had a row, and the parity of the phase that stage s's last one completes
  HB_HD int used() const { return issued < stages ? issued : stages; }
  HB_HD uint32_t last_parity(int s) const { return (uint32_t)((issued - 1 - s) / stages) & 1u; }
};

}  // namespace hb
