"""What the token operators leave behind after a wait that gave up
(csrc/lost_rows.h), run on the host: NaN in every output of a row, wherever the
row lies, in any number of shares, and nothing beside it."""
import os
import shutil
import subprocess

import pytest

import ppo_policy_loss_gb300._build as build

PROGRAM = r"""
#include <cmath>
#include <vector>
#include "lost_rows.h"

struct Out {
  float* logp; float* entropy; float* lse; long long* topk_ids; float* topk_logp;
  int n_ids, k;
};

int main() {
  int bad = 0;
  const long long R = 5;
  for (int n : {0, 1, 3, 128}) for (int k : {0, 1, 70}) for (int parts : {1, 32}) for (int opt = 0; opt < 2; ++opt)
    for (long long row = 0; row < R; ++row) {
      std::vector<float> logp(R * n, 1.f), ent(R, 1.f), lse(R, 1.f), lp(R * k, 1.f);
      std::vector<long long> ids(R * k, 7);
      const Out o{logp.data(), opt ? ent.data() : nullptr, opt ? lse.data() : nullptr, ids.data(), lp.data(), n, k};
      for (int p = 0; p < parts; ++p) rl::lose_logprobs(o, row, p, parts);
      for (long long r = 0; r < R; ++r) {
        const bool lost = r == row;
        for (int q = 0; q < n; ++q) bad += std::isnan(logp[r * n + q]) != lost;
        for (int q = 0; q < k; ++q) bad += std::isnan(lp[r * k + q]) != lost || (ids[r * k + q] == -1) != lost;
        bad += std::isnan(ent[r]) != (lost && opt) || std::isnan(lse[r]) != (lost && opt);
      }
    }
  rl_distill_stats s = {1, 2, 3, 4, 5, 6, 7, 8};
  rl::lose_record(s);
  bad += !(std::isnan(s.loss) && std::isnan(s.forward_kl) && std::isnan(s.reverse_kl) && std::isnan(s.teacher_tail) &&
           std::isnan(s.student_tail)) || s.n_rows != 6 || s.device_error != 7;
  return bad != 0;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="no C++ compiler")
def test_a_lost_row_is_nan(tmp_path):
    src, exe = tmp_path / "t.cpp", tmp_path / "t"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-I", build.CSRC, "-I", build.INCLUDE, str(src), "-o", str(exe)],
                   check=True)
    assert subprocess.run([str(exe)]).returncode == 0


def test_both_kernels_call_it_after_a_timeout():
    """The last step of each kernel that waits."""
    for name, call in (("token_logprobs.cu", "lose_logprobs(a, row"), ("topk_distill.cu", "lose_record(o)")):
        with open(os.path.join(build.CSRC, name), encoding="utf-8") as f:
            assert call in f.read(), name
