"""The embedding kernels' index arithmetic, checked on the host: the header's
carry() and locate(), which turn a place in the count of all rows' units into a
row and a unit, are compiled for the CPU (hipcc, host pass only) and compared
with the plain division, at row widths up to the widest, at places below and
beyond 2^32 units.
"""
import os
import shutil
import subprocess
import textwrap

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = textwrap.dedent(r"""
    #include <cstdio>
    #include "row_units.hpp"
    using namespace forge;

    static Rows rows_of(uint64_t units) {        // as the launches form it
      Rows r;
      r.units = uint32_t(units);
      r.magic = uint32_t(((int64_t(1) << 20) + units - 1) / units);
      return r;
    }

    static bool same(const Rows& r, uint64_t first, uint32_t tid) {
      uint32_t row, unit;
      locate(r, first, tid, row, unit);
      const uint64_t at = first + tid;
      if (row == at / r.units && unit == at % r.units) return true;
      printf("units %u first %llu tid %u: row %u unit %u\n", r.units, (unsigned long long)first,
             tid, row, unit);
      return false;
    }

    int main() {
      // Every place that carry() can be asked for, at every width below 256.
      for (uint32_t units = 1; units < 256; ++units)
        for (uint32_t q = 0; q < units + 256; ++q) {
          const Rows r = rows_of(units);
          uint32_t row = 7, unit;
          carry(r, q, row, unit);
          if (row != 7 + q / units || unit != q % units) {
            printf("carry: units %u q %u: row %u unit %u\n", units, q, row, unit);
            return 1;
          }
        }
      // Widths up to 2^20 units of 4 columns and 2^22 rows: pieces of 256 units around the
      // beginning, row borders, 2^32 units, and the end.
      const uint64_t max_rows = uint64_t(1) << 22, widest = uint64_t(1) << 20;
      for (uint64_t units = 1; units <= widest; units += units < 1100 ? 1 : units / 97) {
        const Rows r = rows_of(units);
        const uint64_t all = units * max_rows;
        const uint64_t around[] = {0, units, 255 * units, all / 3, uint64_t(1) << 31,
                                   uint64_t(1) << 32, 3 * (uint64_t(1) << 32), all - 256};
        for (uint64_t a : around)
          for (int64_t k = -3; k <= 3; ++k) {
            const int64_t first = int64_t(a / 256) * 256 + 256 * k;
            if (first < 0 || uint64_t(first) >= all) continue;
            for (uint32_t tid : {0u, 1u, 63u, 64u, 128u, 200u, 254u, 255u})
              if (!same(r, uint64_t(first), tid)) return 1;
          }
      }
      printf("OK\n");
      return 0;
    }
""")


def _hipcc():
    for c in (shutil.which("hipcc"), "/opt/rocm/bin/hipcc"):
        if c and os.path.exists(c):
            return c
    return None


def test_rows_and_units_equal_a_division(tmp_path):
    hipcc = _hipcc()
    if hipcc is None:
        pytest.skip("hipcc not available")
    src, exe = tmp_path / "index.hip", tmp_path / "index"
    src.write_text(PROGRAM)
    csrc = os.path.join(ROOT, "weight_gradient_gemm_amd", "csrc")
    subprocess.run([hipcc, "--offload-arch=gfx950", "--cuda-host-only", "-O1", "-std=c++17",
                    "-I", os.path.join(ROOT, "include"), "-I", csrc, str(src), "-o", str(exe)],
                   check=True, capture_output=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert out.returncode == 0 and out.stdout.strip() == "OK", out.stdout + out.stderr
