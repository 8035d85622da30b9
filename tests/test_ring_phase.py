"""The bookkeeping of the norms' rings of copies, on the host (no GPU): after a
wait that runs out, a block waits for exactly the copies that it has in flight."""
import os
import shutil
import subprocess

from pseudo_grad_sync_gb300 import _build

HERE = os.path.dirname(os.path.abspath(__file__))


def test_a_failed_wait_leaves_no_copy_in_flight():
    work = os.path.join(HERE, "_cabi", f"ring{os.getpid()}")
    os.makedirs(work, exist_ok=True)
    try:
        exe = os.path.join(work, "ring_phase_check")
        r = subprocess.run(["g++", "-std=c++17", "-Wall", "-Wextra", "-Werror", "-I", _build.CSRC,
                            os.path.join(HERE, "ring_phase_check.cpp"), "-o", exe],
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
