"""Where the row tiles of the attention to the 8-bit cache lie (csrc/qz_attention.h), on the host: with starts that are in
order every row is in exactly one tile, and with any others no tile reaches past the call's rows."""
import itertools
import os
import subprocess

import numpy as np
import pytest

from conftest import ROOT

PROGRAM = r'''
#include <cstdio>
#include "qz_attention.h"
// as the kernels do: a start held to the rows, the sequences whose key is at most u counted a block at a time
static int start_of(const int* st, int s, int tokens) { return st[s] < 0 ? 0 : st[s] < tokens ? st[s] : tokens; }
int main() {
  int tokens, seqs, group, nq, block;
  while (scanf("%d %d %d %d %d", &tokens, &seqs, &group, &nq, &block) == 5) {
    static int st[4096];
    for (int s = 0; s <= seqs; ++s) if (scanf("%d", st + s) != 1) return 1;
    const int rows = 128 * nq;
    const long long slots = (long long)tokens * group / rows + seqs;
    printf("%lld", slots);
    for (long long slot = 0; slot < slots; ++slot) {
      int n = 0;
      for (int s0 = 0; s0 < seqs; s0 += block) {
        int got = 0;
        for (int s = s0; s < s0 + block && s < seqs; ++s) got += qz::tc_first_slot(start_of(st, s, tokens), s, group, rows) <= slot;
        n += got;
        if (got < block) break;
      }
      const int s = n - 1;
      if (s < 0) { printf(" -1 0 0 0"); continue; }
      const int a = start_of(st, s, tokens), b = start_of(st, s + 1, tokens), held = b > a ? b - a : 0;
      const long long all = (long long)held * group, row0 = qz::tc_tile_row(slot, qz::tc_first_slot(a, s, group, rows), all, rows);
      printf(" %d %d %lld %lld", s, a, row0, all);
    }
    printf("\n");
  }
  return 0;
}
'''


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    from precision_quantization_gb300 import _build
    d = tmp_path_factory.mktemp("rows")
    (d / "rows.cu").write_text(PROGRAM)
    subprocess.run([_build.nvcc(), "-std=c++17", "-I", os.path.join(ROOT, "include"), "-I", _build.CSRC, str(d / "rows.cu"), "-o", str(d / "rows")],
                   check=True)
    return str(d / "rows")


def tiles(program, cases):
    """For each (tokens, group, nq, block, starts): (sequence, its first row, the tile's first row or -1, the sequence's rows) of each slot."""
    text = "\n".join(f"{t} {len(st) - 1} {g} {nq} {b} " + " ".join(map(str, st)) for t, g, nq, b, st in cases)
    out = subprocess.run([program], input=text, capture_output=True, text=True, check=True).stdout.splitlines()
    assert len(out) == len(cases)
    for line in out:
        v = [int(x) for x in line.split()]
        assert len(v) == 1 + 4 * v[0]
        yield [v[1 + 4 * i:5 + 4 * i] for i in range(v[0])]


def inside(case, found):
    """How often each row (token, head of the group) is in a tile; no tile reaches past the call's rows."""
    tokens, group, nq, _, _ = case
    seen = np.zeros(tokens * group, int)
    for s, a, row0, rows in found:
        if s < 0 or row0 == -1:
            continue
        assert 0 <= row0 < rows and a >= 0 and a * group + rows <= tokens * group, (case, s, a, row0, rows)
        seen[a * group + row0:a * group + min(row0 + 128 * nq, rows)] += 1
    return seen


def test_rows_in_order_are_in_one_tile(program):
    rng, cases = np.random.default_rng(0), []
    for k in range(400):
        seqs, group, nq = int(rng.integers(1, 9)), int(rng.choice([1, 3, 4, 7, 16, 40])), int(rng.integers(1, 3))
        new = rng.integers(0, rng.choice([2, 5, 40, 400]), seqs)
        st = np.concatenate(([0], np.cumsum(new))) + int(rng.integers(0, 3))
        cases.append((int(st[-1]) + int(rng.integers(0, 4)), group, nq, int(rng.choice([2, 640])), [int(x) for x in st]))
    new = rng.integers(0, 3, 1500)   # more sequences than a CTA has threads
    cases.append((int(new.sum()), 48, 1, 640, [0] + [int(x) for x in np.cumsum(new)]))
    for case, found in zip(cases, tiles(program, cases)):
        tokens, group, _, _, st = case
        want = np.zeros(tokens * group, int)
        want[st[0] * group:st[-1] * group] = 1
        assert np.array_equal(inside(case, found), want), case


def test_starts_that_decrease_reach_no_other_rows(program):
    cases = [(t, g, nq, b, list(st)) for t, g, nq, b, st in
             [(128, 4, 2, 640, (128, 0, 2)), (200, 4, 2, 640, (0, 200, 100, 200)), (300, 4, 2, 640, (300, 0, 150, 300)),
              (400, 4, 1, 640, (400, 0, 0, 0)), (400, 4, 2, 640, (400, 0, 0, 0)), (128, 4, 2, 640, (0, 128, 0, 0, 0))]]
    some = (-(1 << 30), -1, 0, 1, 100, 299, 300, 1 << 30)
    cases += [(300, g, nq, 640, list(st)) for g, nq in ((4, 2), (3, 1)) for st in itertools.product(some, repeat=4)]
    rng = np.random.default_rng(1)
    for k in range(2000):
        tokens, seqs = int(rng.integers(1, 700)), int(rng.integers(1, 7))
        cases.append((tokens, int(rng.choice([1, 3, 4, 16, 40])), int(rng.integers(1, 3)), int(rng.choice([2, 640])),
                      [int(x) for x in rng.integers(-5, tokens + 5, seqs + 1)]))
    for case, found in zip(cases, tiles(program, cases)):
        inside(case, found)
