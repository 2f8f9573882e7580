"""What a tree descriptor uploads, on the CPU: see tree_desc_check.cpp."""
import os
import re
import subprocess


def test_one_copy_that_holds_every_query_once(padoc_lib, tmp_path):
    from tree_structured_shared_gb300 import build
    src = os.path.join(os.path.dirname(os.path.abspath(__file__)), "tree_desc_check.cpp")
    exe = str(tmp_path / "tree_desc_check")
    objs = [os.path.join(build.BUILD, x + ".o") for x in build.SOURCES if x != "host.cpp"]
    r = subprocess.run([build._nvcc(), *build.ARCH, "-O1", "-std=c++17", "-I", build.CSRC, src, *objs, "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    r = subprocess.run([exe, "1500"], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    # descriptors with parts and without were among them
    assert all(int(n) > 50 for n in re.findall(r" (\d+)", r.stdout)), r.stdout
