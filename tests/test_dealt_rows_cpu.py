"""The order in which the log-probability kernel's CTAs take rows that the
hardware deals out (csrc/dealt_rows.h), run on the host: whatever order the
numbers come in, every valid row is streamed once, every masked row is written
once, and no CTA asks again after it was told that none is left."""
import os
import shutil
import subprocess

import pytest

import ppo_policy_loss_gb300._build as build

PROGRAM = r"""
#include <algorithm>
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>
#include "dealt_rows.h"

int failures = 0;
#define CHECK(c) do { if (!(c)) { ++failures; std::printf("%s (R %lld, pattern %d, order %d)\n", #c, R, pattern, order); } } while (0)

// `resident` CTAs share the numbers of R not started; a number that nobody was
// given in time starts a CTA of its own.
void run(long long R, int resident, int pattern, int order, std::mt19937& g) {
  std::vector<char> valid(R);
  for (long long r = 0; r < R; ++r)
    valid[r] = pattern == 0 ? 1 : pattern == 1 ? 0 : pattern == 2 ? g() % 10 < 6 : pattern == 3 ? r < 3 : r >= R - 5;
  std::vector<long long> rows;
  for (long long r = 0; r < R; ++r) if (valid[r]) rows.push_back(r);
  std::vector<long long> pool;
  for (long long n = resident; n < R; ++n) pool.push_back(n);
  if (order == 1) std::reverse(pool.begin(), pool.end());
  if (order == 2) std::shuffle(pool.begin(), pool.end(), g);
  size_t next = 0;
  std::vector<int> streamed(R), written(R);
  for (long long cta = 0; cta < std::min<long long>(resident, R); ++cta) {
    // the CTAs run one after another: each takes a random share of the pool
    const size_t stop = cta + 1 == std::min<long long>(resident, R) ? pool.size() : std::min(pool.size(), next + g() % (2 * pool.size() / resident + 2));
    long long pending = -2;  // -2: nothing asked
    bool told = false, ended = false;
    rl::take_rows(cta, 0, true,
        [&]() { CHECK(pending == -2 && !told); pending = next < stop ? pool[next++] : -1; },
        [&]() { CHECK(pending != -2); const long long n = pending; pending = -2; told = told || n < 0; return n; },
        [&](long long n) { return n < static_cast<long long>(rows.size()) ? rows[n] : -1; },
        [&](long long row) { CHECK(!ended); if (row < 0) ended = true; else ++streamed[row]; return true; },
        [&](long long n) { if (!valid[n]) ++written[n]; });
    CHECK(ended && told && pending == -2);
  }
  for (long long r = 0; r < R; ++r) {
    CHECK(streamed[r] == (valid[r] ? 1 : 0));
    CHECK(written[r] == (valid[r] ? 0 : 1));
  }
}

// Fixed shares, and a wait that gives up.
void fixed(long long R, long long stride) {
  const int pattern = -1, order = -1;
  std::vector<int> streamed(R);
  for (long long first = 0; first < stride; ++first) {
    int ends = 0;
    rl::take_rows(first, stride, false, [] { std::abort(); }, []() -> long long { std::abort(); },
        [&](long long n) { return n < R ? n : -1; },
        [&](long long row) { if (row < 0) ++ends; else ++streamed[row]; return true; }, [](long long) { std::abort(); });
    CHECK(ends == 1);
  }
  for (int s : streamed) CHECK(s == 1);
  for (int dealt = 0; dealt < 2; ++dealt) {
    int rows = 0, asked = 0;
    rl::take_rows(0, 1, dealt != 0, [&] { ++asked; }, [&]() -> long long { return asked; }, [&](long long n) { return n; },
        [&](long long row) { CHECK(row >= 0); return ++rows < 3; }, [](long long) {});
    CHECK(rows == 3 && asked == (dealt ? 3 : 0));
  }
}

int main() {
  std::mt19937 g(7);
  for (int pattern = 0; pattern < 5; ++pattern)
    for (int order = 0; order < 3; ++order)
      for (long long R : {1, 5, 40, 1000}) for (int resident : {1, 3, 17}) run(R, resident, pattern, order, g);
  for (long long R : {0, 1, 7, 100}) for (long long stride : {1, 3, 8}) fixed(R, stride);
  return failures != 0;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="no C++ compiler")
def test_rows_are_dealt_out_in_any_order(tmp_path):
    src, exe = tmp_path / "t.cpp", tmp_path / "t"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-I", build.CSRC, str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout[:2000]
