"""What the plan over a 4-bit pool deals out, on the CPU: see plan_i4_check.cpp."""
import os
import re
import subprocess


def test_plan_covers_every_key_and_result_once(padoc_lib, tmp_path):
    from tree_structured_shared_gb300 import build
    src = os.path.join(os.path.dirname(os.path.abspath(__file__)), "plan_i4_check.cpp")
    exe = str(tmp_path / "plan_i4_check")
    objs = [os.path.join(build.BUILD, x + ".o") for x in build.SOURCES if x != "host.cpp"]
    r = subprocess.run([build._nvcc(), *build.ARCH, "-O1", "-std=c++17", "-I", build.CSRC, src, *objs, "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    r = subprocess.run([exe, "3000"], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    # every kind of unit was among them
    assert all(int(n) > 1000 for n in re.findall(r" (\d+)", r.stdout)), r.stdout
