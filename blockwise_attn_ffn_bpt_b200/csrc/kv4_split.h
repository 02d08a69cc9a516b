// The even split of the 4-bit attention's work over the warps of the device
// (host and device code: the kernels and a host program of the tests use it).
//
// Segments are (sequence, row) in that order, a row being a key/value head and a
// block of columns. A segment of nb > 0 blocks of 64 tokens counts nb +
// KVA_SWITCH units: the first ones stand for the start of a segment (its
// queries, and the sums of the one before), which takes a warp about as long as
// that many blocks. The `total` units of all segments (below 2^31) are cut into
// one run a warp; the first total % warps runs have one unit more than the
// others. The result of warp w for segment s goes to slot s + w (both grow along
// the runs, so no two share one).
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define KVA_HD __host__ __device__ __forceinline__
#else
#define KVA_HD inline
#endif

namespace bpt {

// Measured at 16 contexts of 4096 tokens, 32 heads of 128: 62.1 us with 0, 61.3
// with 1, 61.9 with 2; at 8 of 32768 tokens 200.7, 198.8 and 199.9.
constexpr int KVA_SWITCH = 1;

// Units of a segment of nb blocks.
KVA_HD uint32_t kva_units(uint32_t nb) { return nb ? nb + KVA_SWITCH : 0; }

struct KvaSplit {
  uint32_t total, warps, each, rest;
  KVA_HD KvaSplit(uint32_t t, uint32_t max_warps) : total(t) {
    warps = t < max_warps ? t : max_warps;
    if (warps < 1) warps = 1;
    each = t / warps;
    rest = t - each * warps;
  }
  // First unit of warp w's run, and the warp of a unit.
  KVA_HD uint32_t first(uint32_t w) const { return each * w + (w < rest ? w : rest); }
  KVA_HD uint32_t warp_of(uint32_t unit) const {
    const uint32_t longer = (each + 1) * rest;
    return unit < longer ? unit / (each + 1) : rest + (unit - longer) / each;
  }
};

// Unit, counted from its sequence's first one, of a row's first block.
KVA_HD uint32_t kva_first_block(uint32_t row, uint32_t nb) { return row * (nb + KVA_SWITCH) + KVA_SWITCH; }

// A place in a run: block `blk` of row `row` of sequence beta, which has nb
// blocks; `left` units of the run from there on (none: the run is done).
struct KvaPlace {
  int beta, row, blk, nb, left;

  // The place of unit r of sequence beta (nb blocks), in a run of n units from there.
  static KVA_HD KvaPlace in_sequence(int beta, uint32_t nb, uint32_t r, int n) {
    const uint32_t row = r / (nb + KVA_SWITCH);
    const int unit = (int)(r - row * (nb + KVA_SWITCH)), start = unit < KVA_SWITCH ? KVA_SWITCH - unit : 0;
    return KvaPlace{beta, (int)row, unit + start - KVA_SWITCH, (int)nb, n - start};
  }

  // Takes n blocks of the row; at its end, on to the next segment that has any.
  // blocks(beta): the blocks of a sequence, of b sequences of `rows` rows.
  template <class Blocks>
  KVA_HD void advance(Blocks&& blocks, int b, int rows, int n) {
    blk += n;
    left -= n;
    if (blk < nb || left <= 0) return;
    blk = 0;
    if (++row == rows) {
      row = 0;
      do ++beta;
      while (beta < b && (nb = blocks(beta)) == 0);
      if (beta == b) left = 0;
    }
    left -= KVA_SWITCH;
  }
};

}  // namespace bpt
