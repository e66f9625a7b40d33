"""Compiles the FP8, INT8 and gradient kernels and the C ABI for the host, over
hip/hip_runtime.h and lanes.cpp, with AddressSanitizer.

The sources are taken as they are but for what only a GPU compiler reads: launches
(``kernel<<<grid, threads, lds, stream>>>(..)``), the dynamic LDS, its address
space and the barrier instruction.  Lanes do not run in step here, so where a wave
reads from the LDS what its other lanes wrote without a barrier between (the
staging of a tile's outputs) the lanes are made to meet.
"""
from __future__ import annotations

import concurrent.futures
import glob
import hashlib
import os
import platform
import re
import subprocess
import tempfile

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(os.path.dirname(HERE))
CSRC = os.path.join(ROOT, "nvfp4_block_scaled_gemm_amd", "csrc")
OUT = os.path.join(ROOT, "_build", "host")
CLANG = "/opt/rocm/llvm/bin/clang++"
SOURCES = ("api.cpp", "fp8_gated.hip", "fp8_gated_backward.hip", "fp8_gemm.hip", "fp8_quantize.hip", "fp8_stream.hip",
           "grad_clip.hip", "int8_gemm.hip", "int8_quantize.hip")
FLAGS = ["-std=c++17", "-O1", "-g1", "-fPIC", "-w", "-fno-strict-aliasing", "-mfma", "-mf16c",
         "-ffp-contract=fast-honor-pragmas", "-Xarch_host", "-fsanitize=address", "-mllvm", "-asan-stack=0"]


def sanitizer():
    """The sanitizer's runtime library, or None."""
    found = glob.glob("/opt/rocm/llvm/lib/clang/*/lib/*/libclang_rt.asan-x86_64.so")
    return found[0] if found else None


def available() -> bool:
    if platform.machine() != "x86_64" or not os.path.exists(CLANG) or sanitizer() is None:
        return False
    with open("/proc/cpuinfo") as fh:
        return {"fma", "f16c"} <= set(fh.read().split())


def _launches(text: str) -> str:
    """kernel<..><<<a>>>(b) -> lanes::launch(kernel<..>, a)(b)."""
    while "<<<" in text:
        i = text.index("<<<")
        end = len(text[:i].rstrip())
        k = end
        if text[k - 1] == ">":
            depth = 0
            while True:
                k -= 1
                depth += {">": 1, "<": -1}.get(text[k], 0)
                if depth == 0:
                    break
        while re.match(r"[\w:]", text[k - 1]):
            k -= 1
        close = text.index(">>>", i)
        text = f"{text[:k]}lanes::launch({text[k:end]}, {text[i + 3:close]}){text[close + 3:]}"
    return text


def _meet(text: str, before: str, count: int) -> str:
    """Lanes of a wave meet before each of the `count` places that match."""
    text, n = re.subn(before, lambda m: "lanes::wave_sync();\n" + m[0], text)
    if n != count:
        raise RuntimeError(f"{n} places match {before!r}, not {count}: say again where a wave's lanes meet")
    return text


def _for_host(name: str, text: str) -> str:
    text = text.replace('asm volatile("s_barrier" ::: "memory")', "lanes::barrier()")
    text = text.replace("extern __shared__ __attribute__((aligned(16))) uint8_t smem[];",
                        "uint8_t* smem = lanes::dynamic_lds();")
    text = text.replace("__attribute__((address_space(3))) void*", "void*")
    if name == "fp8_tile.h":
        # a pass's writes after the last pass's reads: the gated epilogue and the plain one
        text = _meet(text, r"#pragma unroll\n +for \(int h = 0; h < 2; \+\+h\)\n#pragma unroll\n"
                           r" +for \(int i = 0; i < FN; \+\+i\)\n +\*reinterpret_cast<", 2)
        # its reads after its writes
        text = _meet(text, r"#pragma unroll\n +for \(int p = 0; p < 2; \+\+p\) \{\n +const int r = p \* 16", 1)
        text = _meet(text, r"if constexpr \(INT8\) \{\n +// eight outputs a lane", 1)
    return _launches(text)


def _compile(src: str) -> str:
    obj = src + ".o"
    res = subprocess.run([CLANG, *FLAGS, "-I", HERE, "-I", os.path.join(ROOT, "include"), "-I", os.path.dirname(src),
                          "-c", src, "-o", obj], capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"{os.path.basename(src)} does not compile for the host:\n{res.stderr[:6000]}")
    return obj


def _symbols(kind: str, objs) -> set:
    res = subprocess.run(["nm", kind, *objs], capture_output=True, text=True, check=True)
    return {line.split()[-1] for line in res.stdout.splitlines() if "_ZN5nvfp4" in line}


def build() -> str:
    """The library's path; built only where a source changed since the last time."""
    inputs = {}
    for d, names in ((CSRC, sorted(os.listdir(CSRC))), (os.path.join(ROOT, "include"), ("nvfp4.h",)),
                     (HERE, ("build.py", "lanes.cpp", os.path.join("hip", "hip_runtime.h")))):
        for f in names:
            if f.endswith(".h") or f in SOURCES or d == HERE:
                with open(os.path.join(d, f)) as fh:
                    inputs[f] = fh.read()
    key = hashlib.sha256("\0".join(f"{k}\0{v}" for k, v in sorted(inputs.items())).encode()).hexdigest()[:16]
    lib = os.path.join(OUT, f"libnvfp4_host_{key}.so")
    if os.path.exists(lib):
        return lib
    os.makedirs(OUT, exist_ok=True)
    with tempfile.TemporaryDirectory(dir=OUT) as work:
        os.replace(_link(work, inputs), lib)
    for other in glob.glob(os.path.join(OUT, "libnvfp4_host_*.so")):  # of older sources
        if other != lib:
            os.remove(other)
    return lib


def _link(work: str, inputs: dict) -> str:
    srcs = []
    for name, text in inputs.items():
        if os.path.exists(os.path.join(CSRC, name)) or name == "lanes.cpp":
            path = os.path.join(work, name.replace(".hip", ".cpp"))
            with open(path, "w") as fh:
                fh.write(_for_host(name, text))
            if path.endswith(".cpp"):
                srcs.append(path)
    with concurrent.futures.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        objs = list(ex.map(_compile, srcs))
    # the C ABI's other kernels are not built: whoever calls one ends the program
    missing = sorted(_symbols("-u", objs) - _symbols("--defined-only", objs))
    rest = os.path.join(work, "rest.cpp")
    with open(rest, "w") as fh:
        fh.write("#include <stdlib.h>\n" + "".join(f'extern "C" void {s}() {{ abort(); }}\n' for s in missing))
    objs.append(_compile(rest))
    lib = os.path.join(work, "linked.so")
    res = subprocess.run([CLANG, "-shared", "-Xarch_host", "-fsanitize=address", "-shared-libasan", *objs, "-o", lib],
                         capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"the host library does not link:\n{res.stderr[:6000]}")
    return lib


if __name__ == "__main__":
    print(build())
