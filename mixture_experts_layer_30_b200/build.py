"""Builds libmoe_b200.so (sm_100a) in-tree with nvcc.

    python -m mixture_experts_layer_30_b200.build

One object per translation unit, compiled in parallel; an object is compiled
again when a file that it includes is newer.
"""
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
OBJ = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libmoe_b200.so")
SOURCES = [os.path.join(CSRC, "moe_api.cu"), os.path.join(CSRC, "block_api.cu")]


def nvcc_path() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _newest_input_mtime() -> float:
    paths = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    paths.append(os.path.join(ROOT, "include", "moe.h"))
    paths.append(os.path.abspath(__file__))
    return max(os.path.getmtime(p) for p in paths)


def _object_of(src: str) -> str:
    return os.path.join(OBJ, os.path.splitext(os.path.basename(src))[0] + ".o")


def _stale(obj: str) -> bool:
    """Whether an object is missing or older than a file its last compile read."""
    deps = obj + ".d"
    if not (os.path.exists(obj) and os.path.exists(deps)):
        return True
    with open(deps) as f:
        names = f.read().replace("\\\n", " ").split(":", 1)[-1].split()
    t = os.path.getmtime(obj)
    return any(not os.path.exists(n) or os.path.getmtime(n) > t
               for n in names + [os.path.abspath(__file__)])


def build(force: bool = False, verbose: bool = False, ptxas_verbose: bool = False) -> str:
    if not force and os.path.exists(LIB) and os.path.getmtime(LIB) >= _newest_input_mtime():
        return LIB
    os.makedirs(OBJ, exist_ok=True)
    base = [nvcc_path(), "-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-lineinfo",
            "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O3",
            "-I", os.path.join(ROOT, "include"), "-I", CSRC]
    if ptxas_verbose:
        base[1:1] = ["-Xptxas", "-v"]
    runs = []
    for src in SOURCES:
        obj = _object_of(src)
        if force or _stale(obj):
            cmd = base + ["-MD", "-MF", obj + ".d", "-c", src, "-o", obj + ".tmp"]
            runs.append((obj, subprocess.Popen(cmd, stdout=subprocess.PIPE,
                                               stderr=subprocess.STDOUT, text=True)))
    failed = ""
    for obj, proc in runs:
        out, _ = proc.communicate()
        if verbose or ptxas_verbose:
            sys.stdout.write(out)
        if proc.returncode != 0:
            failed += out[-4000:]
        else:
            os.replace(obj + ".tmp", obj)
    if failed:
        raise RuntimeError("nvcc failed:\n" + failed)
    tmp = LIB + ".tmp"
    res = subprocess.run(base + ["-shared", "-o", tmp] + [_object_of(s) for s in SOURCES],
                         capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("link failed:\n" + (res.stdout + res.stderr)[-4000:])
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True,
                ptxas_verbose="--ptxas-v" in sys.argv))
