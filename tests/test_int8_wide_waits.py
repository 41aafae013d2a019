"""The waits of the 256 x 256 int8 kernel, checked on the CPU against the order
in which a wave issues its copies and stores and reads what was copied: every
read comes after a wait that covers its copies (and the barrier behind that
wait), and no region is filled before its readers are past it.

Copies and stores complete in the order they are issued, and a wait for N
leaves at most the N newest on their way."""
import os
import subprocess

import pytest

from conftest import ROOT

CSRC = os.path.join(ROOT, "fp8_block_scaled_bias_amd", "csrc")

PRINT = r"""
#include <cstdio>
#include "int8_wide_waits.h"
using namespace moe::int8;
int main() {
  for (int i = 0; i < 3; ++i) std::printf("prologue %d %d\n", i, waits::prologue(i));
  for (int s = 0; s < 2; ++s) {
    for (int p = 0; p < 2; ++p) std::printf("stores %d %d %d\n", s, p, waits::stores(s, p));
    for (int f = 0; f < 2; ++f)
      for (int l = 0; l < 2; ++l)
        for (int p = 0; p < 4; ++p) std::printf("phase %d %d %d %d %d\n", s, f, l, p, waits::phase(s, f, l, p));
  }
}
"""


@pytest.fixture(scope="module")
def waits(tmp_path_factory):
    d = tmp_path_factory.mktemp("waits")
    (d / "w.cpp").write_text(PRINT)
    subprocess.run(["g++", "-std=c++17", "-I", CSRC, str(d / "w.cpp"), "-o", str(d / "w")], check=True)
    out = subprocess.run([str(d / "w")], check=True, stdout=subprocess.PIPE, text=True).stdout
    return {tuple(f[0:1]) + tuple(map(int, f[1:-1])): int(f[-1]) for f in map(str.split, out.splitlines())}


class Wave:
    """One wave's operations; all waves issue the same."""

    def __init__(self, waits, swiglu, gather, nkb, tiles):
        self.w, self.swiglu, self.gather, self.nkb, self.tiles = waits, swiglu, gather, nkb, tiles
        self.issued = self.landed = 0
        self.newest = {}     # what was copied -> number of its newest operation
        self.step = 0        # barriers passed
        self.read_at = {}    # (stage, region) -> step of its last read
        self.faults = []
        self.co = self.ck = self.cb = 0   # the copies' tile, K block, blocks in all

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

    def copy_tile(self):
        if self.gather:
            self.need(("index", self.co))
            self.issue(("index", self.co + 1))

    def copy_next(self):
        self.ck, self.cb = self.ck + 1, self.cb + 1
        if self.ck == self.nkb:
            self.ck, self.co = 0, self.co + 1
            self.copy_tile()

    def copy_one(self, region):
        if self.read_at.get((self.cb & 1, region), -1) >= self.step:
            self.faults.append((self.step, "filled too early", region, self.cb))
        self.issue((region, self.cb))

    def read(self, region, block):
        self.need((region, block))
        self.read_at[(block & 1, region)] = self.step

    def phase(self, reads, block, copies, part, scales_of, wait):
        """part: of an epilogue, or None; scales_of: the tile it stores."""
        self.read(reads, block)
        per = 4 if self.swiglu else 2     # slots of an epilogue block
        stores = 0
        if part is not None and scales_of >= 0:
            self.need(("scales", scales_of))
        for n in range(8):
            if n >= 4:
                self.copy_one(copies)
            if part is not None:
                s = 8 * part + n
                for _ in range(2 * (s % per == 0 and s > 0) + 2 * (s == 15)):
                    self.issue()
                    stores += 1
        if part is not None:
            assert stores == self.w["stores", self.swiglu, part]
        self.wait_and_meet(wait)

    def run(self):
        if self.gather:
            self.issue(("index", 0))
            self.wait_and_meet(0)
        self.copy_tile()
        for s in range(2):
            for region in ("A0", "B0", "B1", "A1"):
                for _ in range(4):
                    self.copy_one(region)
            if s == 0:
                self.copy_next()
        self.wait_and_meet(self.w["prologue", 0])
        self.read("A0", 0)
        self.read("B0", 0)
        self.wait_and_meet(self.w["prologue", 1])
        self.copy_next()
        for _ in range(4):
            self.copy_one("A0")
        self.wait_and_meet(self.w["prologue", 2])
        b = 0
        for to in range(self.tiles):
            for k in range(self.nkb):
                first, last = k == 0, k == self.nkb - 1
                w = [self.w["phase", self.swiglu, first, last, p] for p in range(4)]
                if first:
                    if self.gather:
                        self.need(("index", to))
                    self.issue(("scales", to))
                    self.issue(("scales", to))
                before = 0 if first else None, 1 if first else None
                after = 0 if last else None, 1 if last else None
                self.phase("B1", b, "B0", before[0], to - 1, w[0])
                self.phase("A1", b, "B1", before[1], to - 1, w[1])
                self.phase("A0", b + 1, "A1", after[0], to, w[2])
                self.copy_next()
                self.phase("B0", b + 1, "A0", after[1], to, w[3])
                b += 1
        return self.faults


@pytest.mark.parametrize("swiglu", [0, 1])
@pytest.mark.parametrize("gather", [0, 1])
@pytest.mark.parametrize("nkb", [2, 3, 4, 7, 56])
def test_every_read_is_covered(waits, swiglu, gather, nkb):
    assert Wave(waits, swiglu, gather, nkb, 4).run() == []


@pytest.mark.parametrize("swiglu", [0, 1])
def test_waits_fit_their_counter(waits, swiglu):
    assert all(0 <= n < 64 for key, n in waits.items() if key[0] != "stores")
