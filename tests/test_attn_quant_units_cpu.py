"""The numbering of the 8-bit cache's writing and reading kernels, at sizes that no test could run."""
import os
import subprocess

from gated_deltanet_cpr_gb300 import build

HERE = os.path.dirname(os.path.abspath(__file__))


def test_units_stay_in_range(tmp_path):
    exe = str(tmp_path / "quant_units_test")
    subprocess.check_call([build.nvcc(), *build.ARCH, "-O1", "-std=c++17", "-I", os.path.join(build.ROOT, "include"), "-o", exe,
                           os.path.join(HERE, "cpp", "quant_units_test.cu")])
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0 and " 0 bad" in r.stdout, r.stdout[:2000]
    assert int(r.stdout.split()[0]) > 1000
