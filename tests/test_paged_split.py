"""The share-out of a ragged batch (fa_paged_split.cuh), compiled for the host: an item's key
range against brute force over the mask; and over random batches, every key tile of every
item in exactly one CTA's stretch, no part empty, at most one part begun and one gone on
with per CTA, stretches even."""

import os
import random
import subprocess

import pytest

from exact_io_aware_69_b200 import build

PROGRAM = r'''
#include <cstdio>
#define __host__
#define __device__
#define __align__(n) alignas(n)
#include "fa_paged_split.cuh"
int main() {
  char what;
  while (std::scanf(" %c", &what) == 1) {
    if (what == 'k') {  // p tpi n nk wl wr
      int p, tpi, n, nk, wl, wr;
      std::scanf("%d %d %d %d %d %d", &p, &tpi, &n, &nk, &wl, &wr);
      const fa::KeyRange r = fa::item_keys(p, tpi, n, nk, wl, wr);
      std::printf("%d %d %d %d\n", r.lo, r.hi, r.first, r.count);
    } else if (what == 's') {  // W c least
      unsigned W, c, least;
      std::scanf("%u %u %u", &W, &c, &least);
      std::printf("%u\n", fa::split_start(W, c, least));
    } else {  // r start
      unsigned r;
      int start;
      std::scanf("%u %d", &r, &start);
      std::printf("%d\n", fa::split_tile(r, start));
    }
  }
  std::printf("%d %d %d\n", fa::kSplitGrid, fa::kStepItemCost, fa::kChunkItemCost);
  return 0;
}
'''


@pytest.fixture(scope="module")
def ask(tmp_path_factory):
    d = tmp_path_factory.mktemp("split")
    (d / "split.cpp").write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", build.CSRC_PAGED, str(d / "split.cpp"), "-o",
                    str(d / "split")], check=True)

    def run(lines):
        out = subprocess.run([str(d / "split")], input="\n".join(lines), capture_output=True,
                             text=True, check=True).stdout.split("\n")
        return [tuple(int(x) for x in line.split()) for line in out if line]
    return run


FAR = 1 << 30


def test_item_keys_against_brute_force(ask):
    rng = random.Random(1)
    asked = []
    for _ in range(2000):
        n, nk = rng.randint(1, 40), rng.choice([0, 1, 5, 100, 127, 128, 129, 700])
        tpi = rng.choice([1, 2, 5, 16, 64])
        p = rng.randrange(-(-n // tpi))
        asked.append((p, tpi, n, nk, rng.choice([FAR, 0, 1, 30, 500]), rng.choice([FAR, 0, 3, 200])))
    got = ask("k " + " ".join(map(str, a)) for a in asked)
    for (p, tpi, n, nk, wl, wr), (lo, hi, first, count) in zip(asked, got):
        seen = [j for i in range(p * tpi, min(n, (p + 1) * tpi))
                for j in range(max(0, i + nk - n - wl), min(nk - 1, i + nk - n + wr) + 1)]
        if not seen:
            assert lo > hi and count == 0
        else:
            assert (lo, hi) == (min(seen), max(seen))
            assert first == lo // 128 and first + count - 1 == hi // 128


@pytest.mark.parametrize("seed", range(30))
def test_every_tile_in_one_stretch(ask, seed):
    rng = random.Random(seed)
    grid, *starts_cost = ask([])[-1]
    overhead = starts_cost[seed % 2]
    counts = [rng.choice([0, 0, 1, 2, 3, rng.randint(1, 40), rng.randint(1, 600)])
              for _ in range(rng.choice([1, 2, 8, 60, 400]))]
    least = rng.choice([1, 2, 4, 9])
    W = sum(c + overhead for c in counts)
    starts = [s for s, in ask([f"s {W} {c} {least}" for c in range(grid + 1)])[:-1]]
    assert starts[0] == 0 and starts[-1] == W and starts == sorted(starts)
    lengths = [b - a for a, b in zip(starts, starts[1:])]
    full = [x for x in lengths if x]
    assert max(full) <= max(least, -(-W // grid))
    assert all(x >= min(full[:-1] or full) for x in full[:-1]) and \
        (len(full) == 1 or min(full[:-1]) >= least)
    # where a boundary r units into an item cuts it
    cuts = [t for t, in ask([f"t {r} {overhead}" for r in range(max(counts) + overhead + 1)])[:-1]]
    at, tiles = 0, [[0] * c for c in counts]
    parts = [[] for _ in range(grid)]
    for i, c in enumerate(counts):
        cost, owners = c + overhead, 0
        for cta, (x0, x1) in enumerate(zip(starts, starts[1:])):
            if x0 >= x1 or x1 <= at or x0 >= at + cost:
                continue
            j0 = cuts[x0 - at] if at < x0 else 0
            j1 = c if at + cost <= x1 else cuts[x1 - at]
            if j1 > j0 or (c == 0 and at + cost <= x1):
                owners += 1
                for j in range(j0, j1):
                    tiles[i][j] += 1
                if j0 > 0 or j1 < c:
                    parts[cta].append((j0 > 0, j1 < c))
        assert owners >= 1, "an item that nobody writes"
        at += cost
    assert all(n == 1 for item in tiles for n in item)
    for p in parts:  # one part that went on from another CTA, one that a later CTA goes on with
        assert sum(1 for went_on, _ in p if went_on) <= 1
        assert sum(1 for went_on, goes_on in p if not went_on and goes_on) <= 1
