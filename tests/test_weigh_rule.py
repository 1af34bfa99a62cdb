"""The rule that chooses the kernels for key weights, compiled by itself with checks of divisions and
overflows, over bounds of every kind: too small, too large, not known (CPU)."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "linear_attention_rnn_gb300", "csrc")

PROGRAM = r"""
#include <cstdio>
#include <initializer_list>
#include "gdn_weigh_rule.cuh"
using namespace gdn;
int main() {
  long cases = 0, bad = 0;
  for (int sms : {2, 148, 152})
    for (int Hk : {1, 2, 4, 16})
      for (int G : {1, 2, 3, 4, 16, 64, 100, 128})
        for (int n : {1, 2, 3, 64, 1000})
          for (int total : {1, 2, 64, 65, 77, 256, 257, 1000, 2048, 2112, 1 << 20, 0x7fffffff})
            for (int max_q : {0, 1, 2, 3, 4, 16, 63, 64, 65, 85, 128, 255, 256, 257, 2048, 1 << 20, 0x7fffffff})
              for (long long longest : {0LL, 1LL, 128LL, 129LL, 3000LL, 1LL << 30})
                for (int alike : {0, 1}) {
                  if ((n == 1 && !alike) || (n > 1 && alike && total % n)) continue;
                  const WeighRule w = weigh_rule(n, total, max_q, longest, alike, G * Hk, Hk, 128, sms);
                  ++cases;
                  const bool each_once = (w.few == WeighRule::ALL && w.many == WeighRule::NONE) ||
                                         (w.few == WeighRule::NONE && w.many == WeighRule::ALL) ||
                                         (w.few == WeighRule::BY_SIZE && w.many == WeighRule::BY_SIZE && !alike);
                  // (groups wider than its query tile are not the kernel's for few rows)
                  const bool fits = w.few == WeighRule::NONE || G <= WEIGH_FEW_ROWS;
                  const bool sized = w.few_ctas >= 1 && w.few_ctas <= 2 * sms && w.ctas >= 1 &&
                                     w.split >= 1 && w.split <= 2 && w.ctas * w.split <= sms;
                  if (!each_once || !fits || !sized) ++bad;
                }
  printf("%ld %ld\n", cases, bad);
  return 0;
}
"""


@pytest.mark.parametrize("level", ["-O0", "-O2"])
def test_rule_over_all_bounds(tmp_path, level):
    cc = shutil.which("g++")
    if cc is None:
        pytest.skip("no C++ compiler")
    (tmp_path / "rule.cpp").write_text(PROGRAM)
    subprocess.run([cc, "-std=c++17", level, "-fsanitize=integer-divide-by-zero,signed-integer-overflow",
                    "-fsanitize-undefined-trap-on-error", "-I", CSRC, str(tmp_path / "rule.cpp"), "-o", str(tmp_path / "rule")],
                   check=True)
    run = subprocess.run([str(tmp_path / "rule")], capture_output=True, text=True)
    assert run.returncode == 0, f"ended with {run.returncode} (a division by zero, or an overflow)"
    cases, bad = map(int, run.stdout.split())
    assert cases > 100000 and bad == 0
