"""Which tile a ticket is for, and the steps that lie in it: the arithmetic that the
gated linear recurrence's tiles take their addresses from, compiled for the host.
CPU only.

Tickets at and past the number of tiles are what two calls at once draw that have
been given the same workspace: such a block must have no tile at all, forward and
backward, however many the tickets are.
"""

import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "selective_state_space_87_amd", "csrc")

PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include <initializer_list>
#include "gated_linear_args.h"

static void need(bool ok, const char* what, long long a, long long b, long long c) {
  if (!ok) std::printf("%s: %lld %lld %lld\n", what, a, b, c), std::exit(1);
}

int main() {
  using namespace ssm;
  const int64_t lengths[] = {65, 128, 129, 777, 8192, 65536, (int64_t(1) << 27) - 64, (int64_t(1) << 30) - 1};
  for (const int size : {kGlrFwdSteps, kGlrBwdSteps}) {
    const bool back = size == kGlrBwdSteps;
    for (const int64_t L : lengths) {
      const uint32_t tiles = static_cast<uint32_t>((L + size - 1) / size);
      // tickets of the call's own blocks: every tile once, in the chain's order, its steps the sequence's
      int64_t steps = 0;
      const uint32_t stride = tiles > 5000 ? tiles / 997 : 1;
      for (uint32_t t = 0; t < tiles; t += stride) {
        const uint32_t k = glr_tile_of(t, tiles, back);
        need(k == (back ? tiles - 1 - t : t), "tile", t, tiles, k);
        const int64_t t0 = static_cast<int64_t>(k) * size;
        const int n = glr_steps_in(L, t0, size);
        need(n > 0 && n <= size && t0 + n <= L, "steps", L, t0, n);
        steps += n;
      }
      need(stride > 1 || steps == L, "sum", L, steps, size);
      // tickets past the last tile, up to any word
      const uint32_t past[] = {tiles, tiles + 1, 2 * tiles - 1, 2 * tiles, 8 * tiles, 1u << 24, 0x7fffffffu, 0x80000000u,
                               0xfffffffeu, 0xffffffffu};
      for (const uint32_t t : past) {
        if (t >= tiles) need(glr_tile_of(t, tiles, back) == kGlrNoTile, "past", t, tiles, L);
      }
      // a batch row's steps in every tile that a ticket can give: at most size, 0 or less behind the row's end
      for (uint32_t t = 0; t < tiles; t += stride) {
        const int64_t t0 = static_cast<int64_t>(glr_tile_of(t, tiles, back)) * size;
        for (const int64_t have : {int64_t(0), int64_t(1), L / 2, L - 1, L}) {
          const int64_t exact = have - t0 < size ? have - t0 : size;
          need(glr_steps_in(have, t0, size) == exact && exact > -(int64_t(1) << 30), "within", have, t0, exact);
        }
      }
    }
  }
  // Why there must be a check before a ticket is reversed: without one the first ticket past the end of 128 steps
  // in tiles of 64 is a tile whose first step is 2^38 - 64, and the difference to it in 32 bits is positive.
  const int64_t far = static_cast<int64_t>(uint32_t(2 - 1 - 2)) * 64;
  need(far == (int64_t(1) << 38) - 64 && static_cast<int32_t>(128 - far) > 0, "premise", far, 0, 0);
  static_assert(glr_tile_of(2, 2, true) == kGlrNoTile && glr_tile_of(2, 2, false) == kGlrNoTile);
  std::puts("ok");
}
"""


def test_tickets_past_the_last_tile_have_none(tmp_path):
    if shutil.which("g++") is None:
        pytest.skip("g++ not available")
    src, exe = tmp_path / "places.cpp", tmp_path / "places"
    src.write_text(PROGRAM)
    r = subprocess.run(["g++", "-O1", "-std=c++17", "-Wall", "-I", CSRC, str(src), "-o", str(exe)], capture_output=True,
                       text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout == "ok\n", r.stdout


def test_kernels_take_their_tile_before_anything_else():
    """No kernel makes a place of a ticket by itself."""
    for name in ("gated_linear_fwd.h", "gated_linear_bwd.h"):
        text = open(os.path.join(CSRC, name)).read()
        after = text.split("glr_ticket<", 1)[1].split(";", 2)
        assert after[1].split() == ["if", "(k", "==", "kGlrNoTile)", "return"], name
        assert "tiles - 1 - k" not in text, name
