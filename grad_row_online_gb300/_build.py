"""Builds libgrpo_gb300.so in-tree with nvcc for sm_103a, and _native.so (the
native Python calls of some entry points, csrc/binding.cpp) against PyTorch."""
from __future__ import annotations

import importlib.util
import os
import subprocess
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libgrpo_gb300.so")
NATIVE = os.path.join(HERE, "_native.so")
SOURCES = ["grpo_api.cu", "grpo_prep.cu", "grpo_rows.cu", "grpo_reduce.cu",
           "grpo_logps.cu", "grpo_static.cu", "grpo_vocab.cu", "grpo_token.cu", "grpo_clip.cu"]
ARCH = "-gencode=arch=compute_103a,code=sm_103a"
FLAGS = [ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xptxas", "-v"]


def compile_commands() -> list[list[str]]:
    return [["nvcc", *FLAGS, "-c", os.path.join(CSRC, s),
             "-o", os.path.join(BUILD, s.replace(".cu", ".o"))] for s in SOURCES]


def link_command() -> list[str]:
    return ["nvcc", ARCH, "-shared", *[os.path.join(BUILD, s.replace(".cu", ".o")) for s in SOURCES],
            "-o", LIB, "-lcudart"]


def _torch_dir() -> str:
    return importlib.util.find_spec("torch").submodule_search_locations[0]


def native_compile_command() -> list[str]:
    inc = os.path.join(_torch_dir(), "include")
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-I" + inc,
            "-I" + os.path.join(inc, "torch", "csrc", "api", "include"),
            "-I" + sysconfig.get_paths()["include"], "-I" + os.path.join(cuda, "include"),
            "-c", os.path.join(CSRC, "binding.cpp"), "-o", os.path.join(BUILD, "binding.o")]


def native_link_command() -> list[str]:
    """(after link_command: it is linked against libgrpo_gb300.so)"""
    lib = os.path.join(_torch_dir(), "lib")
    return ["g++", "-shared", os.path.join(BUILD, "binding.o"), "-o", NATIVE, "-L" + HERE,
            "-l:libgrpo_gb300.so", "-L" + lib, "-ltorch_python", "-ltorch_cpu", "-lc10_cuda",
            "-lc10", "-Wl,-rpath,$ORIGIN", "-Wl,-rpath," + lib]


def build(verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    procs = []
    for c in compile_commands() + [native_compile_command()]:
        log = open(c[-1] + ".log", "w")
        procs.append((subprocess.Popen(c, stdout=log, stderr=subprocess.STDOUT), c, log))
    for p, c, log in procs:
        rc = p.wait()
        log.close()
        if rc != 0 or verbose:
            print(open(c[-1] + ".log").read())
        if rc != 0:
            raise RuntimeError("nvcc failed: " + " ".join(c))
    subprocess.run(link_command(), check=True)
    subprocess.run(native_link_command(), check=True)
    return LIB


if __name__ == "__main__":
    build(verbose=True)
