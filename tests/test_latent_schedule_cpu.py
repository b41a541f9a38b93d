"""The decode's rule of how a batch's key tiles are cut, compiled for the host, against the search
that it stands for."""

import ctypes
import os
import random
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "paged_kv_gqa_pkv_gb300", "csrc")

SOURCE = """
#include "pkv_latent_schedule.h"
extern "C" int rule(const int* tiles, int n, int row_blocks, int workers, int* len) {
  int items = 0, most = 0, total = 0, passes = 0;
  for (int b = 0; b < n; ++b) {
    items += tiles[b] > 0 ? row_blocks : 0;
    most = tiles[b] > most ? tiles[b] : most;
    total += tiles[b] * row_blocks;
  }
  const int each = total / workers, more = total % workers;
  const pkv::latent::PartRule r = pkv::latent::part_rule(items, most, workers, each, more, [&](int l) {
    int k = 0;
    for (int b = 0; b < n; ++b) k += (tiles[b] + l - 1) / l;
    ++passes;
    return k * row_blocks;
  });
  *len = r.len;
  return r.parts ? passes : -1 - passes;
}
"""


@pytest.fixture(scope="module")
def rule(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("no host compiler")
    d = tmp_path_factory.mktemp("schedule")
    (d / "rule.cpp").write_text(SOURCE)
    subprocess.run(["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-I", CSRC, "-o", str(d / "rule.so"),
                    str(d / "rule.cpp")], check=True)
    lib = ctypes.CDLL(str(d / "rule.so"))

    def call(tiles, row_blocks, workers):
        n = ctypes.c_int()
        r = lib.rule((ctypes.c_int * len(tiles))(*tiles), len(tiles), row_blocks, workers, ctypes.byref(n))
        return (True, n.value, r) if r >= 0 else (False, None, -1 - r)
    return call


def whole_search(tiles, row_blocks, workers):
    """The shortest parts that find a worker each (or whole items that are about as short), if they are
    worth having beside equal ranges: every length tried until one fits."""
    items, most = sum(t > 0 for t in tiles) * row_blocks, max(tiles)
    each, more = divmod(sum(tiles) * row_blocks, workers)
    if items > workers:
        return False, None
    n = max(each + (more > 0), 1)
    while True:
        if most <= n + 1:
            n = max(most, 1)
            break
        if sum(-(-t // n) for t in tiles) * row_blocks <= workers:
            break
        n += max(1, n >> 5)
    return (True, n) if n <= each + each // 4 + 3 else (False, None)


def test_skewed_batches_are_searched_no_longer_than_parts_are_worth(rule):
    """One long sequence among short ones that just fill the workers."""
    for tiles, blocks, workers in (([1] * 75 + [256], 1, 76), ([1] * 60 + [4000], 1, 76), ([1] * 37 + [1 << 20], 2, 76),
                                   ([5] * 74 + [3000, 2900], 1, 76)):
        parts, n, passes = rule(tiles, blocks, workers)
        assert (parts, n) == whole_search(tiles, blocks, workers)
        assert passes <= 15, (tiles[-1], passes)


def test_same_rule_as_the_whole_search(rule):
    rng = random.Random(3)
    for _ in range(4000):
        workers = rng.choice([1, 2, 5, 66, 76])
        blocks = rng.choice([1, 1, 1, 2, 3])
        top = int(2 ** rng.uniform(0, 12))
        tiles = [rng.randint(0, top) for _ in range(rng.randint(1, 80))]
        for _ in range(rng.randint(0, 2)):
            tiles[rng.randrange(len(tiles))] = int(2 ** rng.uniform(0, 16))
        if max(tiles) == 0:
            tiles[0] = 1
        parts, n, passes = rule(tiles, blocks, workers)
        assert (parts, n) == whole_search(tiles, blocks, workers), (tiles, blocks, workers)
        assert passes <= 15
