"""Build libfp4q.so (HIP, gfx950) in-tree with hipcc, and beside it the Python
binding _calls.so (host C++ against torch's headers).

    python -m block_scaled_fp4_reduce_amd.build [--asm]

Flags: gfx950 only; no fp contraction (every fused multiply-add in the
kernels is an explicit fmaf, so results are reproducible bit for bit);
packed fp32 instructions disabled; fp32 division stays correctly rounded
(the HIP default).
"""
from __future__ import annotations

import importlib.util
import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libfp4q.so")
BINDING = os.path.join(HERE, "_calls.so")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC", "-shared",
    "-ffp-contract=off",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-function", "-Wno-unused-command-line-argument",
]


def sources():
    return [os.path.join(CSRC, f) for f in ("fp4q.hip", "attention.hip")]


def deps():
    out = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    out.append(os.path.join(os.path.dirname(HERE), "include", "fp4q.h"))
    return out


def binding_command(out):
    """g++ command of the binding, linked to the libfp4q.so beside it; None
    without torch, which the C library does not need."""
    torch = importlib.util.find_spec("torch")
    if torch is None:
        return None
    root = torch.submodule_search_locations[0]
    inc = [os.path.join(root, "include"), os.path.join(root, "include/torch/csrc/api/include"),
           "/opt/rocm/include", sysconfig.get_paths()["include"]]
    return [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall",
            "-D__HIP_PLATFORM_AMD__=1", "-DUSE_ROCM", *["-isystem" + i for i in inc],
            os.path.join(CSRC, "binding.cpp"), "-o", out, "-L" + HERE, "-lfp4q",
            "-Wl,-rpath,$ORIGIN", "-L" + os.path.join(root, "lib"), "-lc10", "-lc10_hip",
            "-ltorch_cpu", "-ltorch_python"]


def build(verbose: bool = False) -> str:
    tmp = LIB + ".tmp%d" % os.getpid()
    objs = ["%s.%s.o" % (tmp, os.path.basename(src)) for src in sources()]
    cflags = [f for f in FLAGS if f != "-shared"]
    jobs = [[HIPCC, *cflags, "-c", src, "-o", obj] for src, obj in zip(sources(), objs)]
    link = [HIPCC, *FLAGS, *objs, "-o", tmp]
    try:
        running = []
        for cmd in jobs:                 # the sources compile side by side
            if verbose:
                print(" ".join(cmd), flush=True)
            running.append(subprocess.Popen(cmd))
        failed = [cmd for cmd, p in zip(jobs, running) if p.wait() != 0]
        if failed:
            raise subprocess.CalledProcessError(1, failed[0])
        if verbose:
            print(" ".join(link), flush=True)
        subprocess.check_call(link)
        os.replace(tmp, LIB)
        cmd = binding_command(tmp)       # links to the library, so it comes after
        if cmd is None:
            print("torch is not installed: libfp4q.so is built without the Python binding _calls.so",
                  flush=True)
            return LIB
        if verbose:
            print(" ".join(cmd), flush=True)
        subprocess.check_call(cmd)
        os.replace(tmp, BINDING)
    finally:
        for f in [*objs, tmp]:
            if os.path.exists(f):
                os.remove(f)
    return LIB


def up_to_date() -> bool:
    if not (os.path.exists(LIB) and os.path.exists(BINDING)):
        return False
    t = min(os.path.getmtime(LIB), os.path.getmtime(BINDING))
    return all(os.path.getmtime(d) <= t for d in deps())


def dump_asm(out_dir: str) -> str:
    """Device assembly of the kernels, for inspection."""
    os.makedirs(out_dir, exist_ok=True)
    for src in sources():
        name = os.path.splitext(os.path.basename(src))[0]
        cmd = [HIPCC, *[f for f in FLAGS if f not in ("-shared", "-fPIC")],
               "--cuda-device-only", "-S", src, "-o", os.path.join(out_dir, name + "-gfx950.s")]
        subprocess.check_call(cmd)
    return os.path.join(out_dir, "fp4q-gfx950.s")


if __name__ == "__main__":
    if "--asm" in sys.argv:
        print(dump_asm(os.path.join(os.path.dirname(HERE), "_build", "asm")))
    else:
        print(build(verbose=True))
