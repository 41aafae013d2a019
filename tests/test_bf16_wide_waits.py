"""The waits of the 256 x 256 bf16 kernel, checked on the CPU against the order
in which a wave issues its copies and stores and reads what was copied: every
read comes after a wait that covers its copies (and the barrier behind that
wait), and no region is filled before its readers are past it.

Copies and stores complete in the order they are issued, and a wait for N
leaves at most the N newest on their way."""
import os
import subprocess

import pytest

from bf16_plan import MODES
from conftest import ROOT

CSRC = os.path.join(ROOT, "fp8_block_scaled_bias_amd", "csrc")

PRINT = r"""
#include <cstdio>
#include "bf16_wide_waits.h"
using namespace moe::bf16;
int main() {
  for (int m = 0; m < 5; ++m)
    for (int f = 0; f < 2; ++f)
      for (int l = 0; l < 2; ++l)
        for (int p = 0; p < 4; ++p) std::printf("phase %d %d %d %d %d\n", m, f, l, p, waits::phase(m, f, l, p));
}
"""

# slots (of 16) of a half's epilogue -> stores issued in them
STORES = {
    "gemm": {4: 4, 8: 4, 12: 4, 15: 4},
    "dgrad": {4: 4, 8: 4, 12: 4, 15: 4},
    "glu": {8: 4, 15: 4},
    "glu kept": {2: 4, 4: 4, 8: 4, 10: 4, 12: 4, 15: 4},
    "dgrad_glu": {s: 4 for s in range(1, 16, 2)},
    "wgrad": {**{s: 4 for s in range(2, 16, 2)}, 15: 4},
}


@pytest.fixture(scope="module")
def waits(tmp_path_factory):
    d = tmp_path_factory.mktemp("waits")
    (d / "w.cpp").write_text(PRINT)
    subprocess.run(["g++", "-std=c++17", "-I", CSRC, str(d / "w.cpp"), "-o", str(d / "w")], check=True)
    out = subprocess.run([str(d / "w")], check=True, stdout=subprocess.PIPE, text=True).stdout
    return {tuple(map(int, f[1:-1])): int(f[-1]) for f in map(str.split, out.splitlines())}


class Wave:
    """One wave's operations; all waves issue the same."""

    def __init__(self, waits, mode, gather, blocks):
        self.w, self.mode, self.m = waits, mode, MODES.index(mode.split()[0])
        self.blocks = blocks      # K blocks of each tile
        self.rows = gather and mode != "wgrad"     # a tile's row indices, read by every wave
        self.index = gather and mode == "wgrad"    # a K block's, read by the wave that copied them
        self.issued = self.landed = self.step = 0
        self.newest, self.read_at, self.faults = {}, {}, []
        self.co = self.ck = self.cb = self.xb = 0

    def issue(self, what=None):
        self.issued += 1
        if what is not None:
            self.newest[what] = self.issued

    def wait_and_meet(self, n):
        self.landed = max(self.landed, self.issued - n)
        self.step += 1

    def need(self, what):
        if self.newest.get(what, self.issued + 1) > self.landed:
            self.faults.append((self.step, what))

    def length(self, o):
        return self.blocks[min(o, len(self.blocks) - 1)]

    def index_block(self):
        self.issue(("index", self.xb))
        self.xb += 1

    def aim_block(self):
        if self.index:
            self.need(("index", self.cb))

    def copy_tile(self):
        if self.rows:
            self.need(("rows", self.co))
            self.issue(("rows", self.co + 1))
        self.aim_block()

    def copy_next(self):
        self.cb += 1
        if self.index:
            if self.xb - self.cb > 3:
                self.faults.append("four slots of indices")
            self.index_block()
        self.ck += 1
        if self.ck == self.length(self.co):
            self.ck, self.co = 0, self.co + 1
            self.copy_tile()
        else:
            self.aim_block()

    def copy_one(self, region):
        if self.read_at.get((self.cb & 1, region), -1) >= self.step:
            self.faults.append((self.step, "filled too early", region, self.cb))
        self.issue((region, self.cb))

    def read(self, region, block):
        self.need((region, block))
        self.read_at[(block & 1, region)] = self.step

    def phase(self, reads, block, copies, part, wait):
        self.read(reads, block)
        for n in range(8):
            if n >= 4:
                self.copy_one(copies)
            if part is not None:
                for _ in range(STORES[self.mode].get(8 * part + n, 0)):
                    self.issue()
        self.wait_and_meet(wait)

    def run(self):
        if self.index:
            for _ in range(3):
                self.index_block()
        if self.rows:
            self.issue(("rows", 0))
        if self.index or self.rows:
            self.wait_and_meet(0)
        self.copy_tile()
        for s in range(2):
            for region in ("A0", "B0", "B1", "A1"):
                for _ in range(4):
                    self.copy_one(region)
            if s == 0:
                self.copy_next()
        self.wait_and_meet(24)
        self.read("A0", 0)
        self.read("B0", 0)
        self.wait_and_meet(0 if self.index else 24)
        self.copy_next()
        for _ in range(4):
            self.copy_one("A0")
        self.wait_and_meet(4)
        b = 0
        for nkb in self.blocks:
            for k in range(nkb):
                first, last = k == 0, k == nkb - 1
                w = [self.w[self.m, first, last, p] for p in range(4)]
                self.phase("B1", b, "B0", 0 if first else None, w[0])
                self.phase("A1", b, "B1", 1 if first else None, w[1])
                self.phase("A0", b + 1, "A1", 0 if last else None, w[2])
                self.copy_next()
                self.phase("B0", b + 1, "A0", 1 if last else None, w[3])
                b += 1
        return self.faults


@pytest.mark.parametrize("mode", sorted(STORES))
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("blocks", [[2] * 4, [3] * 4, [4, 4], [7] * 3, [112] * 2, [2, 14, 2, 2, 3, 30, 2]])
def test_every_read_is_covered(waits, mode, gather, blocks):
    assert Wave(waits, mode, gather, blocks).run() == []


def test_waits_fit_their_counter(waits):
    assert all(24 <= n < 64 for n in waits.values())


def test_the_check_finds_a_wait_that_is_too_long(waits):
    lax = {k: n + 4 for k, n in waits.items()}
    assert all(Wave(lax, mode, False, [3] * 4).run() for mode in ("gemm", "glu"))
