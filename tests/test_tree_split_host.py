"""How windowed cached attention cuts its work, on devices of any size (no GPU:
the rule is host code, built here by itself)."""
import os
import subprocess

from io_aware_exact_15_gb300 import build

MAIN = r"""
#include <stdio.h>
#include <initializer_list>
#include "fa_tree_host.h"
using namespace fa;
int main() {
  int bad = 0, shared = 0;
  for (int sms = 1; sms <= 700; sms += sms < 160 ? 1 : 27)
    for (int format = 0; format < 3; ++format)
      for (int d = 64; d <= 128; d += 64)
        for (int rows : {1, 4, 8, 9, 16, 24, 25, 128, 256, 300})
          for (int B : {1, 2, 3, 7, 16, 31, 48, 95, 96, 190, 400})
            for (int Hkv : {1, 4})
              for (int window : {1, 512, 4096}) {
                TreeParams p = {};
                p.B = B, p.Hkv = Hkv, p.T = 1, p.rows = rows;
                p.pair = rows > kTile;
                p.groups = (rows + 2 * kTile - 1) / (2 * kTile);
                p.log_page = 6, p.max_pages = 500, p.window = window, p.sinks = 4;
                split_window(&p, format, d, sms);
                const bool few = tree_few_rows(rows, format);
                const int grid = tree_grid(p, sms * (few ? few_ctas(rows, format, d) : 1));
                shared += p.cluster > 0;
                // (CTA c of a cluster uses places 2 c and 2 c + 1 of 2 * most_ctas)
                if (grid < 1 || grid > most_ctas(rows) || (p.cluster && p.whole)) {
                  if (!bad++) printf("sms %d format %d d %d rows %d B %d: %d\n", sms, format, d, rows, B, grid);
                }
              }
  printf("%d bad, %d shared\n", bad, shared);
  return bad || !shared;
}
"""


def test_no_more_ctas_than_the_workspace_has_parts_for(tmp_path):
    (tmp_path / "main.cpp").write_text(MAIN)
    exe = tmp_path / "main"
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-I", build.CSRC, "-I",
                        os.path.join(build.CUDA_HOME, "include"), "-o", str(exe),
                        str(tmp_path / "main.cpp")],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
