"""Launch plans of the block-scaled FP8 products over sizes from one token to the largest: abi.cpp linked with launchers that check
every buffer, range, form and grid (tests/plan/fp8_plan_driver.cpp)."""
import os
import subprocess

from rank_error_compensation_amd import build as B

DRIVER = os.path.join(os.path.dirname(os.path.abspath(__file__)), "plan", "fp8_plan_driver.cpp")


def _run(cmd):
    p = subprocess.run(cmd, capture_output=True, text=True)
    assert p.returncode == 0, f"{' '.join(cmd)}\n{p.stdout[-4000:]}\n{p.stderr[-4000:]}"
    return p.stdout


def test_plans(tmp_path):
    objs = [os.path.join(B.BUILD, s + ".o") for s in B.SOURCES if s != "fp8.hip"]
    if not all(os.path.exists(o) for o in objs):
        B.build()
    drv, exe = str(tmp_path / "driver.o"), str(tmp_path / "driver")
    _run([B.hipcc(), "-x", "hip", "-c", DRIVER, "-o", drv] + B.common_flags())
    _run([B.hipcc(), f"--offload-arch={B.ARCH}", "-o", exe, drv] + objs)
    print(_run([exe]))
