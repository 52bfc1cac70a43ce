"""How the 64-row chunk attention shares its work list (csrc/tv_share.cuh), compiled for the host: every half
tile of every item goes to exactly one CTA, in order, and the join is told those CTAs, also where the list
has more than 2^31 and 2^32 places."""

import os
import shutil
import subprocess

import pytest

from tree_speculative_verify_gb300 import build as tvbuild

PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include <vector>

#include "tv_share.cuh"

using namespace tv::few;

// requests tokens heads before window ctas: items of 64 rows, token by token, as the kernel lists them
int main(int, char** arg) {
  const long long requests = atoll(arg[1]), tokens = atoll(arg[2]), H = atoll(arg[3]);
  const long long before = atoll(arg[4]), W = atoll(arg[5]);
  const int G = atoi(arg[6]);
  std::vector<int> units;
  for (long long b = 0; b < requests; ++b)
    for (long long row = 0; row < tokens * H; row += 64) {
      const long long last = row + 63 < tokens * H ? row + 63 : tokens * H - 1;
      const long long lo = before + row / H, hi = before + last / H, t0 = lo > W ? lo - W : 0;
      units.push_back((int)((hi / 4 + 63) / 64 + (hi / 128 + 63) / 64 + (hi + 1 - t0 + 63) / 64));
    }
  long long total = 0;
  int most = 0;
  std::vector<long long> front;
  for (int u : units) {
    front.push_back(total);
    total += places_of(u);
    if (places_of(u) > most) most = places_of(u);
  }
  const long long share = share_of(total, most, G);
  if (share < 1 || share * G < total) return printf("share %lld of %lld\n", share, total), 1;
  std::vector<int> done(units.size(), 0), first(units.size(), -1), ctas(units.size(), 0);
  size_t at = 0;   // the item in which the CTA's share starts
  for (int c = 0; c < G; ++c) {
    const long long start = c * share;
    if (start >= total) break;
    while (at + 1 < units.size() && front[at + 1] <= start) ++at;
    Cut cut;
    cut.first((int)(start - front[at]), share < total - start ? share : total - start);
    for (size_t i = at; cut.left > 0 && i < units.size(); ++i) {
      if (i > at) cut.next();
      if (!cut.take(units[i])) break;
      if (cut.ub != done[i]) return printf("item %zu: CTA %d from %d behind %d\n", i, c, cut.ub, done[i]), 1;
      done[i] = cut.ue;
      if (first[i] < 0) first[i] = c;
      if (c != first[i] + ctas[i]) return printf("item %zu: CTA %d after a gap\n", i, c), 1;
      ++ctas[i];
    }
  }
  for (size_t i = 0; i < units.size(); ++i) {
    const Piece p = piece_of(front[i], places_of(units[i]), share, G);
    if (done[i] != units[i] || p.first != first[i] || p.ctas != ctas[i] || p.first < 0 || p.first + p.ctas > G)
      return printf("item %zu: %d of %d half tiles, CTAs %d + %d, told %d + %d\n", i, done[i], units[i],
                    first[i], ctas[i], p.first, p.ctas), 1;
  }
  for (int k = 0; k < 48; ++k)
    for (long long n : {(1ll << k) - 1, 1ll << k, (1ll << k) * 4 / 3 + k})
      if (n + G <= 1ll << 48 && even_share(n, G) != (n + G - 1) / G) return printf("%lld / %d\n", n, G), 1;
  const Piece none = piece_of(5, places_of(0), share, G);
  if (none.ctas != 0) return 1;
  printf("%lld\n", total);
}
"""


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("g++ not installed")
    where = tmp_path_factory.mktemp("share")
    (where / "share.cpp").write_text(PROGRAM)
    r = subprocess.run([cxx, "-std=c++17", "-O1", "-Wall", "-Wextra", "-Werror", "-fsanitize=undefined",
                        "-fno-sanitize-recover", "-I", tvbuild.CSRC, str(where / "share.cpp"), "-o",
                        str(where / "share")], capture_output=True, text=True)
    if "ubsan" in r.stderr:       # (the sanitizer's library is not installed)
        r = subprocess.run([cxx, "-std=c++17", "-O1", "-I", tvbuild.CSRC, str(where / "share.cpp"), "-o",
                            str(where / "share")], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return str(where / "share")


def total_of(program, *args):
    r = subprocess.run([program, *map(str, args)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    return int(r.stdout)


@pytest.mark.parametrize("ctas", [1, 7, 148, 152])
@pytest.mark.parametrize("requests,tokens,H,before", [
    (1, 1, 1, 0), (1, 1, 64, 8192), (64, 1, 64, 3000), (3, 5, 24, 70000), (4, 1, 64, 16000), (500, 2, 3, 40),
    (1, 700, 16, 0), (1, 1, 64, 300000)])
def test_every_half_tile_has_one_cta(program, requests, tokens, H, before, ctas):
    for window in (0, 128, 1024):
        total_of(program, requests, tokens, H, before, window, ctas)


@pytest.mark.parametrize("requests,tokens,H,before,least", [
    (1, 1048576, 64, 0, 2 ** 31), (1, 262144, 128, 1048576, 2 ** 31), (1, 1048576, 128, 0, 2 ** 32),
    (1048576, 1, 1, 524287, 2 ** 31)])
def test_lists_of_more_places_than_32_bits_count(program, requests, tokens, H, before, least):
    assert total_of(program, requests, tokens, H, before, 128, 152) > least
