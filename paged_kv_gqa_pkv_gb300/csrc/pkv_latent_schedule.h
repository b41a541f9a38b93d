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
