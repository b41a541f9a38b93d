// pkv_latent_schedule.h - how the decode over shared latents cuts a batch's key tiles: into whole
// items, equal parts of items, or equal ranges of all tiles. Plain C++, for the kernel and for the
// host.
#pragma once

#ifdef __CUDACC__
#define PKV_SCHED_FN __host__ __device__ __forceinline__
#else
#define PKV_SCHED_FN inline
#endif

namespace pkv {
namespace latent {

// The schedule, from the sequences' tiles alone, so that it needs no other kernel's work.
//
// Up to as many items as workers: an item of nt tiles is cut into ceil(nt / S) equal parts, for the
// smallest S (in steps of 1/32) at which all parts find a worker; every worker has one part, loads Q
// once and has nothing to wait for between items. Where the longest item has at most kWholeSlack
// tiles more than S nothing is cut at all: partial results are 256 KB each for 128 rows, written,
// read and joined by a kernel that is otherwise done at once (a cut costs about two tiles' time).
//
// More items than workers, or parts that are longer than an equal share by more than a quarter and
// kRangeCost tiles (equal ranges cost the workers a second item, with its queries' loads and another
// partial: 16 x ~20000 keys, parts of 37 tiles against ranges of 32: 77.7 us against 85.1): the tiles
// of all items stand in a row (at most 2^30, which the host sees to), sequence by sequence, its row blocks one
// after another; worker w's range begins at tile w * each + min(w, more). A cut inside an item moves
// to one of its ends if that is at most kCutReach tiles away (one tile where ranges are long), and to
// the closer one.
//
// Both sides of the borders, measured with pages of 64 (us; 76 workers; n x k: n items of k tiles):
// - whole against parts, 16 query rows: 8 x 2 10.5 / 11.0, 8 x 3 12.0 / 11.4, 8 x 4 13.6 / 11.3; 38 x 3
//   14.3 / 16.1, 38 x 4 16.0 / 16.4, 38 x 8 21.1 / 20.5. 128 rows, whose partials are eight times as
//   large: 8 x 2 11.1 / 13.2, 8 x 3 12.8 / 13.4, 8 x 5 15.9 / 14.6; 25 x 3 14.6 / 20.0, 25 x 8 21.6 /
//   24.7, 25 x 12 27.3 / 26.5; 38 x 4 17.4 / 22.4, 38 x 12 28.8 / 30.1. So one tile is right up to a few
//   dozen parts of few rows; many parts of 128 rows are worth having from six or so tiles on, which
//   the rule does not know.
// - parts against ranges. Parts by the rule (S / equal share): 16 x U[8, 32] (5 / 4) 21.9 / 25.6 with 16
//   rows, 26.3 / 28.9 with 128; 16 x U[16, 64] (10 / 8) 30.8 / 33.5, 36.8 / 44.3; 40 x U[16, 64] (28 / 21
//   and 31 / 23) 56.6 / 54.1, 69.1 / 75.4. Ranges by the rule: 40 x U[64, 125] (66 / 50) 124.5 / 104.7,
//   138.8 / 123.8; 70 x U[1, 63] (44 / 32 and 37 / 27) 103.5 / 78.0, 103.1 / 96.1; but 64 x U[8, 32] (24 / 16)
//   56.1 / 49.2, 60.4 / 66.8 and 70 x U[1, 16] (12 / 7 and 14 / 8) 37.0 / 35.5, 40.1 / 47.9.
// - a reach of 1 / 3 / 5 tiles, 16 and 128 rows: ranges of 8 tiles 34.7 / 33.4 / 33.3 and 49.6 / 43.9 /
//   42.2; of 18 tiles 49.3 / 49.9 / 53.2 and 74.2 / 66.7 / 64.6; of 40 86.1 / 86.2 / 90.6 and 111.3 / 108.9 /
//   106.2; of 82 161 / 170 / 174 and 194 / 192 / 190.
constexpr int kWholeSlack = 1;
constexpr int kCutReach = 3;
constexpr int kRangeCost = 3;

struct PartRule {
  bool parts;  // parts (or whole items), else ranges
  int len;     // tiles of a part at most
};
// items: with keys; most: the longest one's tiles; each, more: an equal share of all tiles, and how
// many workers have one tile more; parts_of(len): the parts of all items at that length. The search
// ends at the longest part that is worth having (after at most about a dozen lengths, each of which
// asks for a pass over the batch).
template <class PartsOf>
PKV_SCHED_FN PartRule part_rule(int items, int most, int workers, int each, int more,
                                PartsOf parts_of) {
  const int longest = each + each / 4 + kRangeCost;
  int len = each + (more > 0 ? 1 : 0);
  if (len < 1) len = 1;
  if (items > workers) return {false, len};
  for (;; len += len >= 64 ? len >> 5 : 1) {
    if (most <= len + kWholeSlack) {
      len = most > 1 ? most : 1;
      break;
    }
    if (len > longest || parts_of(len) <= workers) break;
  }
  return {len <= longest, len};
}

PKV_SCHED_FN int move_cut(int x, int i0, int i1, int reach) {
  if (x - i0 <= reach && x - i0 <= i1 - x) return i0;
  if (i1 - x <= reach) return i1;
  return x;
}

}  // namespace latent
}  // namespace pkv
