"""Builds libmoe_b200.so (sm_100a) and the binding's native module _calls.so in-tree.

    python -m mixture_experts_layer_30_b200.build

One object per translation unit, compiled in parallel; an object is compiled
again when a file that it includes is newer, the native module also when torch or
Python is another one.
"""
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
OBJ = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libmoe_b200.so")
CALLS = os.path.join(PKG, "_calls.so")
CALLS_SRC = os.path.join(CSRC, "calls.cpp")
CALLS_FOR = os.path.join(OBJ, "_calls.for")  # the torch and Python that CALLS was built for
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


def _calls_tag() -> str:
    import torch
    return (f"torch {torch.__version__}, C++11 ABI {int(torch._C._GLIBCXX_USE_CXX11_ABI)}, "
            f"{sysconfig.get_config_var('SOABI')}")


def _calls_match() -> bool:
    """Whether _calls.so was built for this torch and Python."""
    if not os.path.exists(CALLS_FOR):
        return False
    with open(CALLS_FOR) as f:
        return f.read() == _calls_tag()


def _calls_commands():
    """Compile and link commands of _calls.so: a CPython module on torch's tensors that
    calls libmoe_b200.so beside it."""
    import torch
    home = os.path.dirname(torch.__file__)
    obj = _object_of(CALLS_SRC)
    compile_cmd = [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-DNDEBUG",
                   f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
                   "-I", os.path.join(ROOT, "include"),
                   "-isystem", sysconfig.get_paths()["include"],
                   "-isystem", os.path.join(home, "include"),
                   "-isystem", os.path.join(home, "include", "torch", "csrc", "api", "include"),
                   "-isystem", os.path.join(os.path.dirname(os.path.dirname(nvcc_path())),
                                            "include"),
                   "-MD", "-MF", obj + ".d", "-c", CALLS_SRC, "-o", obj + ".tmp"]
    link_cmd = [compile_cmd[0], "-shared", "-o", CALLS + ".tmp", obj, LIB,
                "-L", os.path.join(home, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10_cuda",
                "-lc10", "-Wl,-rpath,$ORIGIN"]
    return obj, compile_cmd, link_cmd


def build(force: bool = False, verbose: bool = False, ptxas_verbose: bool = False) -> str:
    newest = _newest_input_mtime()
    lib_fresh, calls_fresh = (not force and os.path.exists(f) and os.path.getmtime(f) >= newest
                              for f in (LIB, CALLS))
    same_torch = _calls_match()
    if lib_fresh and calls_fresh and same_torch:
        return LIB
    os.makedirs(OBJ, exist_ok=True)
    base = [nvcc_path(), "-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-lineinfo",
            "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O3",
            "-I", os.path.join(ROOT, "include"), "-I", CSRC]
    if ptxas_verbose:
        base[1:1] = ["-Xptxas", "-v"]
    runs = []
    for src in [] if lib_fresh else SOURCES:
        obj = _object_of(src)
        if force or _stale(obj):
            cmd = base + ["-MD", "-MF", obj + ".d", "-c", src, "-o", obj + ".tmp"]
            runs.append((obj, subprocess.Popen(cmd, stdout=subprocess.PIPE,
                                               stderr=subprocess.STDOUT, text=True)))
    calls_obj, calls_compile, calls_link = _calls_commands()
    if force or not same_torch or _stale(calls_obj):
        runs.append((calls_obj, subprocess.Popen(calls_compile, stdout=subprocess.PIPE,
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
        raise RuntimeError("compilation failed:\n" + failed)
    soname = ["-Xlinker", "-soname=" + os.path.basename(LIB)]
    links = [(LIB, base + ["-shared", "-o", LIB + ".tmp"] + soname
              + [_object_of(s) for s in SOURCES]), (CALLS, calls_link)]
    for out, cmd in links[1:] if lib_fresh else links:
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError("link failed:\n" + (res.stdout + res.stderr)[-4000:])
        os.replace(out + ".tmp", out)
    with open(CALLS_FOR, "w") as f:
        f.write(_calls_tag())
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True,
                ptxas_verbose="--ptxas-v" in sys.argv))
