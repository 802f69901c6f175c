"""The packed kernels (recurrence, convolution) and group norm under host
emulation: every CUDA thread a std::thread, under AddressSanitizer against the
FP64 oracle and under ThreadSanitizer.  Bad bounds, slots out of the pool and
repeated slots are run here, before any device sees them."""
import os
import shutil
import subprocess
import sys

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
sys.path.insert(0, os.path.join(HERE, "host_emu"))
pytestmark = pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")


def _run(sanitizer, *args):
    import emu_build  # noqa: E402  (tests/host_emu on sys.path)
    env = dict(os.environ, LD_PRELOAD=emu_build.sanitizer_runtime(sanitizer), ASAN_OPTIONS="detect_leaks=0",
               TSAN_OPTIONS="halt_on_error=0", OMP_NUM_THREADS="1")
    return subprocess.run([sys.executable, os.path.join(HERE, "host_emu", "run_packed.py"), *args], env=env,
                          capture_output=True, text=True, timeout=900)


def test_packed_kernels_under_host_emulation():
    import emu_packed  # noqa: E402
    import run_packed  # noqa: E402
    emu_packed.build()
    r = _run("address")
    assert r.returncode == 0, r.stdout[-4000:] + r.stderr[-4000:]
    assert "MISMATCH" not in r.stdout and r.stdout.count(" ok ") == len(run_packed.CASES), r.stdout


def test_packed_kernels_have_no_data_race():
    import emu_packed  # noqa: E402
    lib = emu_packed.build(sanitizer="thread")
    r = _run("thread", "--races", lib)
    assert r.returncode == 0 and "data race" not in r.stderr, r.stderr[-4000:]
    assert "race run done" in r.stdout
