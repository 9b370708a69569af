"""The scheduler of the attention kernels (fa_paged_split.cuh) on the host: a warp is 32
threads that meet in every exchange, and each of the 148 CTAs hands its items to a list.
Every key tile of every item goes to one CTA, whatever the batch; lengths that no batch can
have give out nothing that the caller's buffers do not hold."""

import os
import random
import re
import subprocess

import pytest

from exact_io_aware_69_b200 import build

COMMON = r'''
#pragma once
#include <algorithm>
#include <barrier>
#include <cstdint>
#include <cstdio>
#include <thread>
#include <vector>
#define __host__
#define __device__
#define __forceinline__ inline
#define __align__(n) alignas(n)
using std::min;
struct Index { unsigned x; };
inline thread_local Index threadIdx;
inline Index blockIdx;
inline std::barrier<> meet(32);
inline unsigned box[32];
inline int __ffs(unsigned v) { return __builtin_ffs(static_cast<int>(v)); }
template <class T> T exchange(T v, int from) {
  box[threadIdx.x] = static_cast<unsigned>(v);
  meet.arrive_and_wait();
  const T got = static_cast<T>(box[from]);
  meet.arrive_and_wait();
  return got;
}
template <class T> T __shfl_sync(unsigned, T v, int from) { return exchange(v, from & 31); }
template <class T> T __shfl_up_sync(unsigned, T v, int d) {
  const int me = threadIdx.x;
  return exchange(v, me >= d ? me - d : me);
}
template <class Op> unsigned all_of(unsigned v, Op op) {
  box[threadIdx.x] = v;
  meet.arrive_and_wait();
  unsigned r = 0;
  for (int i = 0; i < 32; ++i) r = op(r, i, box[i]);
  meet.arrive_and_wait();
  return r;
}
inline unsigned __reduce_add_sync(unsigned, unsigned v) {
  return all_of(v, [](unsigned r, int, unsigned x) { return r + x; });
}
inline unsigned __ballot_sync(unsigned, bool v) {
  return all_of(v, [](unsigned r, int i, unsigned x) { return r | x << i; });
}
inline bool __any_sync(unsigned m, bool v) { return __ballot_sync(m, v) != 0; }
inline bool __all_sync(unsigned m, bool v) { return __ballot_sync(m, v) == 0xffffffffu; }
namespace fa {
inline int g_fa_status = 0;
constexpr int kStatusInvalid = -1;
inline void atomicExch(int* at, int v) { __atomic_store_n(at, v, __ATOMIC_RELAXED); }
@VIEW@
}
'''

RING = r'''
struct ItemRing {
  std::vector<Item> items;
  bool put(const Item& it, volatile int*) { items.push_back(it); return true; }
};
'''

PROGRAM = r'''
#include "fa_paged_split.cuh"
#include <cstdlib>
template <bool ONE>
void cta(const fa::PagedView& c, int tpi, int max_q, int wl, int wr, int least) {
  fa::ItemRing ring;
  std::vector<fa::PartInfo> parts(fa::kSplitGrid);
  std::vector<std::thread> warp;
  for (unsigned lane = 0; lane < 32; ++lane)
    warp.emplace_back([&, lane] {
      threadIdx.x = lane;
      fa::Scheduler<ONE> s(c, tpi, max_q, wl, wr);
      s.locate(least);
      s.run(ring, nullptr, parts.data());
    });
  for (auto& t : warp) t.join();
  for (const fa::Item& it : ring.items)
    if (it.begin >= 0)
      std::printf("item %u %d %d %d %d %d %d %d %d\n", blockIdx.x, it.b, it.h, it.p, it.begin,
                  it.keys.first, it.keys.count, it.j0, it.j1);
  const fa::PartInfo& p = parts[blockIdx.x];
  std::printf("part %u %d %d %d %d %d\n", blockIdx.x, p.begins, p.token0, p.tokens, p.head,
              p.goes_on);
}
int main() {
  fa::PagedView c{};
  int one, tpi, max_q, wl, wr, from, to;
  std::scanf("%d %d %d %d %d %d %d %d %d %d %d %d", &one, &tpi, &max_q, &wl, &wr, &c.table_width,
             &c.page_shift, &c.heads, &c.batch, &c.tokens, &from, &to);
  std::vector<int> cu(c.batch + 1), sk(c.batch);
  for (int& x : cu) std::scanf("%d", &x);
  for (int& x : sk) std::scanf("%d", &x);
  c.cu_q = cu.data();
  c.seq_k = sk.data();
  for (int i = from; i < to; ++i) {
    blockIdx.x = i;
    one ? cta<true>(c, tpi, max_q, wl, wr, 2) : cta<false>(c, tpi, max_q, wl, wr, 2);
  }
  std::printf("status %d\n", fa::g_fa_status);
}
'''


@pytest.fixture(scope="module")
def schedule(tmp_path_factory):
    d = tmp_path_factory.mktemp("scheduler")
    common = open(os.path.join(build.CSRC_PAGED, "fa_paged_common.cuh")).read()
    split = open(os.path.join(build.CSRC_PAGED, "fa_paged_split.cuh")).read()
    view = common[common.index("struct PagedView"):common.index("// max of three")]
    (d / "fa_paged_common.cuh").write_text(COMMON.replace("@VIEW@", view))
    split, rings = re.subn(r"// The ring: .*?(?=// The scheduler: one warp)", lambda m: RING, split,
                           flags=re.S)
    assert rings == 1
    (d / "fa_paged_split.cuh").write_text(split.replace("#ifdef __CUDACC__", "#if 1"))
    (d / "main.cpp").write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++20", "-O1", "-pthread", str(d / "main.cpp"), "-o",
                    str(d / "main")], check=True)

    def run(cu_q, seq_k, tpi, max_q, heads, width, one, wl=1 << 30, wr=0, shift=4, tokens=None,
            ctas=(0, 148)):
        """(items, parts by CTA, status): items as (cta, b, h, p, begin, first, count, j0, j1)."""
        values = [int(one), tpi, max_q, wl, wr, width, shift, heads, len(seq_k),
                  cu_q[-1] if tokens is None else tokens, *ctas, *cu_q, *seq_k]
        out = subprocess.run([str(d / "main")], input=" ".join(map(str, values)), text=True,
                             capture_output=True, check=True, timeout=120).stdout.split("\n")
        rows = [line.split() for line in out if line]
        items = [tuple(map(int, r[1:])) for r in rows if r[0] == "item"]
        parts = {int(r[1]): tuple(map(int, r[2:])) for r in rows if r[0] == "part"}
        return items, parts, int(rows[-1][1])
    return run


def running(lengths):
    cu = [0]
    for n in lengths:
        cu.append(cu[-1] + n)
    return cu


@pytest.mark.parametrize("seed", range(8))
def test_every_tile_goes_to_one_cta(schedule, seed):
    rng = random.Random(seed)
    one = seed % 2 == 0
    tpi = 4 if one else rng.choice([2, 32, 128])
    top = tpi if one else rng.choice([40, 700])
    batch = rng.choice([1, 5, 40, 70])
    n = [rng.choice([0, 1, rng.randint(1, top)]) for _ in range(batch)]
    nk = [rng.choice([0, k, k + rng.randint(0, 3000)]) for k in n]
    heads, wl = rng.choice([1, 3]), rng.choice([1 << 30, 200])
    items, parts, status = schedule(running(n), nk, tpi, top, heads, 400, one, wl=wl)
    assert status == 0
    want = {(b, h, p) for b in range(batch) for h in range(heads) for p in range(-(-n[b] // tpi))}
    seen = {}
    for cta, b, h, p, begin, first, count, j0, j1 in items:
        assert begin == sum(n[:b]) and 0 <= j0 <= j1 <= count
        seen.setdefault((b, h, p), []).append((j0, j1, count, cta))
    assert set(seen) == want
    for (b, h, p), pieces in seen.items():
        pieces.sort()
        assert pieces[0][0] == 0 and pieces[-1][1] == pieces[-1][2]
        for (_, j1, _, cta), (j0, _, _, after) in zip(pieces, pieces[1:]):
            assert j1 == j0 and after == cta + 1
        if len(pieces) > 1:  # what the merge kernel is told
            first = pieces[0][3]
            assert parts[first][:4] == (1, sum(n[:b]) + p * tpi, min(tpi, n[b] - p * tpi), h)
            assert [parts[c][4] for *_, c in pieces[1:]] == [1] * (len(pieces) - 2) + [0]


@pytest.mark.parametrize("one", [True, False])
@pytest.mark.parametrize("cu_q", [[0, 3, 2, 6, 9], [3, 0, 4, 8, 9], [0, 2, 5, 9, 8]])
def test_rows_given_to_two_sequences(schedule, one, cu_q):
    """Where cu_q decreases, rows may belong to two sequences: the batch is left out."""
    items, parts, status = schedule(cu_q, [50] * 4, 4, 4, 2, 10, one, tokens=9)
    assert not items and status == -1
    assert all(p == (0, 0, 0, 0, 0) for p in parts.values())


def test_more_rows_than_the_launch_allows_for(schedule):
    """Sequences that each claim all rows, between others that run backwards: 16 x 32 x 31
    items of 2^20 tiles, past 32 bits, where the launch counts on 64 x 31. The last CTA must
    not leave a part for a later one: the merge would look for the rest behind the workspace."""
    tokens, batch, keys = 32 * 64, 32, 1 << 27
    cu_q = [0 if i % 2 == 0 else tokens for i in range(batch + 1)]
    items, parts, status = schedule(cu_q, [keys] * batch, 64, tokens, 31, keys >> 10, False,
                                    wr=1 << 30, shift=10, tokens=tokens, ctas=(147, 148))
    assert not items and parts[147] == (0, 0, 0, 0, 0)
