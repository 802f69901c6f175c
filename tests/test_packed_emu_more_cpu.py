"""Further host-emulated runs of the packed kernels: what the cases of
test_packed_emu_cpu.py do not reach."""
import os
import shutil
import subprocess
import sys

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
sys.path.insert(0, os.path.join(HERE, "host_emu"))
pytestmark = pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")


def _run(name, sanitizer="address"):
    import emu_build  # noqa: E402  (tests/host_emu on sys.path)
    import emu_packed  # noqa: E402
    lib = emu_packed.build(sanitizer=sanitizer)
    env = dict(os.environ, LD_PRELOAD=emu_build.sanitizer_runtime(sanitizer), ASAN_OPTIONS="detect_leaks=0",
               TSAN_OPTIONS="halt_on_error=0", OMP_NUM_THREADS="1")
    r = subprocess.run([sys.executable, os.path.join(HERE, "host_emu", "run_packed_more.py"), name, lib], env=env,
                       capture_output=True, text=True, timeout=900)
    assert r.returncode == 0 and "done" in r.stdout, r.stdout[-4000:] + r.stderr[-4000:]
    return r


def test_chunk_form_is_as_exact_as_a_recurrence_in_32_bits():
    _run("precision")


def test_chunk_form_comes_round():
    _run("chunk_rounds")


def test_chunk_form_comes_round_without_data_races():
    """Every wait that guards a buffer used again: stages of K and Q, B and the row
    factors, T, V, the products for the prep warps, the state from chunk to chunk."""
    r = _run("chunk_rounds_races", "thread")
    assert "data race" not in r.stderr, r.stderr[-4000:]


def test_empty_sequences_may_name_anothers_slot():
    _run("empty_sequences")


def test_convolution_skips_bad_bounds_only():
    _run("conv_bounds")
