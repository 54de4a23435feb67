"""The loop of a workgroup over its tiles (csrc/walk.h), as a program on the host: a
tile after the last one is not run, whatever the memory that would have held it has."""

import shutil
import subprocess

import pytest

from mixture_experts_ffn_route_amd import build

PROGRAM = r"""
#include <cstdio>
#include <vector>
#include "walk.h"

struct Item {
  int blocks = 0, id = 0;
};
static int bad = 0;

// Tiles of these heights; a body that finds no next tile leaves `rest` where one would
// stand, as memory may hold anything there.
template <int HIGH>
void walk(const std::vector<int> &heights, int rest) {
  std::vector<int> seen;
  size_t at = 0;
  moe::walk_tiles<HIGH>(Item{heights[0], 0}, [&](auto height, const Item &it, Item &nx) {
    if (it.blocks != decltype(height)::value || it.id != (int)seen.size()) ++bad;
    seen.push_back(decltype(height)::value);
    const bool more = ++at < heights.size();
    nx = more ? Item{heights[at], (int)at} : Item{rest, (int)at};
    return more && seen.size() <= heights.size();
  });
  if (seen != heights) {
    ++bad;
    std::printf("HIGH %d first %d of %zu, then %d: %zu bodies\n", HIGH, heights[0], heights.size(),
                rest, seen.size());
  }
}

template <int HIGH>
void all() {
  for (int rest = -1; rest <= 5; ++rest)
    for (int a = 1; a <= HIGH; ++a) {
      walk<HIGH>({a}, rest);
      for (int b = 1; b <= HIGH; ++b) {
        walk<HIGH>({a, b}, rest);
        for (int c = 1; c <= HIGH; ++c) walk<HIGH>({a, b, c}, rest);
      }
    }
}

int main() {
  all<1>();
  all<2>();
  all<4>();
  return bad ? 1 : 0;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs a host compiler")
def test_no_tile_after_the_last(tmp_path):
    source, program = tmp_path / "walk.cpp", tmp_path / "walk"
    source.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", build.CSRC, "-o", str(program), str(source)],
                   check=True)
    out = subprocess.run([str(program)], capture_output=True, text=True, timeout=60)
    assert out.returncode == 0, out.stdout
