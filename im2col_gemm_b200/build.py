"""Build step of libmqc: compiles the CUDA sources in ``csrc/`` for sm_100a
into ``libmqc.so`` next to this file (in-tree, so the library travels with the
source tree)."""
from __future__ import annotations

import glob
import os
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))
LIB = os.path.join(HERE, "libmqc.so")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-lineinfo", "-std=c++17",
         "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden"]
OBJ = os.path.join(HERE, "build")


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(HERE, "csrc", "*.cu")) + glob.glob(os.path.join(HERE, "csrc", "*.cuh"))
                  + glob.glob(os.path.join(HERE, "csrc", "*.h"))
                  + [os.path.join(os.path.dirname(HERE), "include", "mqc.h")])


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(s) <= t for s in sources())


def object_up_to_date(obj: str) -> bool:
    """Newer than every file of its dependency list (written by nvcc -MD; one
    that was cut short names none, or is not there)."""
    if not os.path.exists(obj) or not os.path.exists(obj + ".d"):
        return False
    with open(obj + ".d") as f:
        files = f.read().replace("\\\n", " ").partition(":")[2].split()
    t = os.path.getmtime(obj)
    return bool(files) and all(os.path.exists(x) and os.path.getmtime(x) <= t for x in files)


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date():
        return LIB
    # one object per translation unit, compiled side by side; an object is
    # kept when nothing it includes has changed
    os.makedirs(OBJ, exist_ok=True)
    units = sorted(glob.glob(os.path.join(HERE, "csrc", "*.cu")))
    objects, running = [], []
    for unit in units:
        obj = os.path.join(OBJ, os.path.basename(unit)[:-3] + ".o")
        objects.append(obj)
        if not force and object_up_to_date(obj):
            continue
        tmp = obj + f".tmp{os.getpid()}"
        cmd = [NVCC, *FLAGS, "-MD", "-MF", tmp + ".d", "-c", "-o", tmp, unit]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        running.append((subprocess.Popen(cmd), cmd, tmp, obj))
    failed = []
    for proc, cmd, tmp, obj in running:
        if proc.wait() == 0:
            # the list first: beside the old object it names what made that old
            os.replace(tmp + ".d", obj + ".d")
            os.replace(tmp, obj)
            continue
        failed.append(cmd)
        for left in (tmp, tmp + ".d"):
            if os.path.exists(left):
                os.remove(left)
    if failed:
        raise subprocess.CalledProcessError(1, failed[0])
    tmp = LIB + f".tmp{os.getpid()}"
    subprocess.check_call([NVCC, *FLAGS, "-shared", "-o", tmp, *objects])
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose=True))
