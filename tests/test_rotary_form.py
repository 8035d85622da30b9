"""How rotary positions share out a head's elements and a token's heads, on the
host (no GPU): nothing outside is touched at the largest sizes that are taken."""
import os
import shutil
import subprocess

from pseudo_grad_sync_gb300 import _build

HERE = os.path.dirname(os.path.abspath(__file__))


def test_every_element_and_head_once():
    work = os.path.join(HERE, "_cabi", f"form{os.getpid()}")
    os.makedirs(work, exist_ok=True)
    try:
        exe = os.path.join(work, "rotary_form_check")
        r = subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Wextra", "-Werror", "-I", _build.CSRC,
                            os.path.join(HERE, "rotary_form_check.cpp"), "-o", exe],
                           capture_output=True, text=True)
        assert r.returncode == 0, r.stderr
        r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
        assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout
    finally:
        shutil.rmtree(work, ignore_errors=True)
        try:
            os.rmdir(os.path.dirname(work))
        except OSError:
            pass
