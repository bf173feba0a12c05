"""What the attention launchers keep (resident CTAs, with the kernel's shared-memory
limit raised) is kept for each device: a second GPU of a process must not be
launched on with the first one's.  No second GPU is needed: the helper that keeps
it runs on the host, and no launcher keeps such a number without it."""

import os
import re
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "decode_attention_paged_kv_gb300", "csrc")


def test_once_a_device(tmp_path):
    exe = str(tmp_path / "check")
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-I", CSRC, "-o", exe,
                    os.path.join(HERE, "native", "per_device_check.cpp")], check=True)
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout


def test_no_number_kept_for_the_process():
    for f in sorted(os.listdir(CSRC)):
        if f.endswith((".cu", ".cuh", ".h", ".cpp")):
            with open(os.path.join(CSRC, f)) as src:
                assert not re.search(r"^\s*static (int|bool|size_t) \w+ = ", src.read(), re.M), f
