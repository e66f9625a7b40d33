"""pytest plugin: runs GPU tests on CPU tensors over the host build of the kernels
(build.py).  HOST_LIB is its path; HOST_LATE=0 lets direct loads land at once instead
of when a wait asks for them; HOST_SEED draws the order of waves."""
import ctypes
import os

import pytest

import nvfp4_block_scaled_gemm_amd as nv
import nvfp4_block_scaled_gemm_amd._lib as binding
import tests.gpu_util

binding.LIB_PATH = os.environ["HOST_LIB"]
nv.load()
ctypes.CDLL(binding.LIB_PATH).lanes_mode(int(os.environ.get("HOST_LATE", "1")), int(os.environ.get("HOST_SEED", "1")))
tests.gpu_util.need_gpu = lambda: None

# what tests of streams, graphs and of the refusal of CPU tensors are called
NEEDS_GPU = ("captured", "graph", "two_streams", "_refusals")
_need = binding._need


def _need_but_a_gpu(cond, msg):
    if not cond and "GPU" in msg:
        return
    _need(cond, msg)


binding._need = _need_but_a_gpu
binding._here = lambda stream, dev: True
binding._stream = lambda stream=None, dev=None: 0


def pytest_collection_modifyitems(items):
    for item in items:
        module = item.module
        if hasattr(module, "DEV"):
            module.DEV = "cpu"
        if hasattr(module, "need_gpu"):
            module.need_gpu = tests.gpu_util.need_gpu
        if any(word in item.name for word in NEEDS_GPU):
            item.add_marker(pytest.mark.skip(reason="needs a GPU"))
