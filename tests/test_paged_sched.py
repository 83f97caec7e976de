"""The work split of the attention over a paged cache, checked on the host by
counting (tests/paged_sched_check.cu, compiled here)."""
import os
import subprocess

from attention_core_gb300 import build as lib_build

HERE = os.path.dirname(os.path.abspath(__file__))


def test_every_block_is_visited_once(tmp_path):
    exe = str(tmp_path / "check")
    res = subprocess.run([lib_build._nvcc(), *lib_build.ARCH, "-O2", "-std=c++17", "-o", exe,
                          os.path.join(HERE, "paged_sched_check.cu")], capture_output=True, text=True)
    assert res.returncode == 0, res.stderr
    res = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert res.returncode == 0, res.stdout
