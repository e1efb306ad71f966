"""Host proof that the adapters' first product reads nothing past the factors: the
rule that ends its unconditional loads, compiled for the host from the kernels'
own header and walked over ranks, widths and batches."""
import os
import subprocess

from bit_quantized_lora_quantize_amd import build_lib

PROGRAM = r"""
#include <cstdio>
#include "qlora_kernels.h"
using namespace qlora;

int main() {
  const int step = 64;   // k_shrink's
  long long ranges = 0, whole_steps = 0;
  for (int64_t M : {1, 4096, 16384, 40000, 65536, 200000})
    for (int r = 1; r <= 256; r = r < 40 ? r + 1 : r + 7)
      for (int64_t K = 1; K <= 2200; K = K < 600 ? K + 1 : K + 37) {
        int64_t kper;
        const int splits = shrink_splits(M, K, &kper);
        for (int s = 0; s < splits; ++s) {
          const int64_t kb = s * kper, ke = kb + kper < K ? kb + kper : K;
          const int64_t piece = (r + 7) / 8 * 8;   // elements from a row's start to its last piece's end
          const int64_t we = shrink_whole_end(kb, ke, K, r, true, step);
          ++ranges;
          whole_steps += (we - kb) / step;
          if (we < kb || we > ke || (we - kb) % step) {
            std::printf("r=%d K=%lld range %lld..%lld: whole steps end at %lld\n", r, (long long)K, (long long)kb,
                        (long long)ke, (long long)we);
            return 1;
          }
          if (we > kb && (we - 1) * r + piece > K * r) {
            std::printf("r=%d K=%lld range %lld..%lld: row %lld is read %lld elements past the factor\n", r,
                        (long long)K, (long long)kb, (long long)ke, (long long)(we - 1),
                        (long long)((we - 1) * r + piece - K * r));
            return 1;
          }
          // and no step is kept out of them without need
          if (we + step <= ke && (we + step - 1) * r + piece <= K * r) {
            std::printf("r=%d K=%lld range %lld..%lld: a step too few\n", r, (long long)K, (long long)kb, (long long)ke);
            return 1;
          }
          // stored [r][K], or in rows of whole pieces: every whole step
          const int64_t all = kb + (ke - kb) / step * step;
          if (shrink_whole_end(kb, ke, K, r, false, step) != all || (r % 8 == 0 && we != all)) return 2;
        }
      }
  std::printf("%lld ranges, %lld steps\n", ranges, whole_steps);
  return 0;
}
"""


def test_unconditional_loads_of_a_factor_end_inside_it(tmp_path):
    src, exe = tmp_path / "walk.cpp", tmp_path / "walk"
    src.write_text(PROGRAM)
    env = {k: v for k, v in os.environ.items() if k != "LD_PRELOAD"}   # (a sanitizer's runtime is not the compiler's)
    subprocess.run([build_lib.HIPCC, "-x", "hip", "--offload-host-only", "-O1", "-std=c++17", "-I", build_lib.INCLUDE, "-I", build_lib.CSRC,
                    str(src), "-o", str(exe)], check=True, env=env, capture_output=True, text=True)
    res = subprocess.run([str(exe)], env=env, capture_output=True, text=True, timeout=60)
    assert res.returncode == 0, res.stdout + res.stderr
    assert "ranges" in res.stdout
