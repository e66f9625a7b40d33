"""The gated, INT8, clipping and FP8 kernels run on the host, lane by lane, under
AddressSanitizer (tests/host): the GPU tests of sizes that take a second or two that
way, and a few of the largest tiles.  Shows indexing, waits and arithmetic; not the hardware's rounding inside a
matrix instruction, the order of memory beyond barriers, streams or time."""
import os
import re
import subprocess
import sys

import pytest

from tests.host import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FILES = ("test_gpu_clip_grads.py", "test_gpu_feed_forward_layer.py", "test_gpu_fp8_gated.py", "test_gpu_int8.py")
# what fills a GPU, and tests whose inputs alone take long; of the largest tiles one case each
LARGEST = ("bf16-128-4100-2048-272", "4100-8200-400", "many_tiles and bf16-264")
LONG = ("far_rows", "past_31_bits", "many_tiles", "largest_sums and not 3-40", "1000-264-2064", "70-4160-1040",
        "600-1000", "1000-520-8192", "70-8300-2064", "512-4104", "90-16400")
# of the second run, which has no new case
SECOND = ("16-8200", "130-2100", "200-333", "3-256-6144", "1048576", "f32-silu", "bf16-gelu", "training")


@pytest.fixture(scope="module")
def library():
    if not build.available():
        pytest.skip("needs clang and its sanitizer runtime on x86-64")
    return build.build()


def run(library, report, *args, **env):
    """Runs tests over the host library; how many passed."""
    options = "detect_leaks=0:detect_stack_use_after_return=0:halt_on_error=1:allocator_may_return_null=1:" \
              f"handle_abort=1:log_path={report}/report"
    res = subprocess.run(
        [sys.executable, "-m", "pytest", "-q", "-x", "-n", str(min(8, os.cpu_count() or 1)), "-p", "tests.host.on_host",
         "-p", "no:cacheprovider", "-m", "gpu", *args],
        cwd=ROOT, capture_output=True, text=True, timeout=1500,
        env=dict(os.environ, HOST_LIB=library, LD_PRELOAD=build.sanitizer(), ASAN_OPTIONS=options, OMP_NUM_THREADS="1",
                 PYTHONPATH=ROOT, **env))
    out = res.stdout + res.stderr
    passed = re.search(r"(\d+) passed", out)
    reports = [p.read_text(errors="replace")[:3000] for p in sorted(report.iterdir())]
    assert res.returncode == 0 and passed, "\n".join([out[-6000:], *reports[:2]])
    return int(passed[1])


def all_but(words, also=()):
    which = " and ".join(f"not ({w})" for w in words)
    return ["-k", " or ".join([f"({which})", *also]), *(os.path.join("tests", f) for f in FILES)]


def test_with_loads_that_land_late(library, tmp_path):
    assert run(library, tmp_path, *all_but(LONG, LARGEST), HOST_LATE="1", HOST_SEED="2") > 400


def test_with_loads_that_land_at_once(library, tmp_path):
    assert run(library, tmp_path, *all_but(LONG + SECOND), HOST_LATE="0", HOST_SEED="3") > 200
