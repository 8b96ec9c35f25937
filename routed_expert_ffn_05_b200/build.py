"""Build libmoe.so in-tree with nvcc for sm_100a (no GPU needed to compile)."""
from __future__ import annotations

import concurrent.futures
import glob
import importlib.util
import os
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libmoe.so")
MARSHAL = os.path.join(PKG, "_marshal" + sysconfig.get_config_var("EXT_SUFFIX"))  # the binding's C part

NVCC = os.environ.get("NVCC", "nvcc")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
         "-I", INCLUDE, "-I", CSRC, "--expt-relaxed-constexpr"]


def _torch_include():
    """torch's include folder, which holds the DLPack header, or None (found, not imported)."""
    spec = importlib.util.find_spec("torch")
    return os.path.join(list(spec.submodule_search_locations)[0], "include") if spec else None


def build_marshal(target: str = MARSHAL, torch_include: str | None = None) -> bool:
    """The binding's C part. It only makes calls shorter (the package works without it, through ctypes), so what
    hinders it is said and not raised; without a DLPack header it looks at tensors through their methods."""
    cmd = ["gcc", "-O2", "-std=c11", "-Wall", "-fPIC", "-shared", "-I", sysconfig.get_paths()["include"], "-I", INCLUDE]
    if torch_include:
        cmd += ["-I", torch_include]
    tmp = target + f".tmp{os.getpid()}"
    try:
        r = subprocess.run([*cmd, os.path.join(PKG, "marshal.c"), "-o", tmp], capture_output=True, text=True)
        why = f"{r.stdout}\n{r.stderr}" if r.returncode else None
    except OSError as e:
        why = str(e)
    if why is None:
        os.replace(tmp, target)
        return True
    for f in (tmp, target):  # no older one stays beside a newer library
        if os.path.exists(f):
            os.remove(f)
    sys.stderr.write(f"marshal.c was not built, calls go through ctypes: {why}\n")
    return False


def _headers():
    return glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        glob.glob(os.path.join(INCLUDE, "*.h"))


def _stale(target, deps):
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _compile(src, verbose_ptxas=False):
    obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
    if _stale(obj, [src] + _headers()) or verbose_ptxas:
        cmd = [NVCC, *ARCH, *FLAGS, "-c", src, "-o", obj]
        if verbose_ptxas:
            cmd.insert(1, "-Xptxas=-v")
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose_ptxas:
            sys.stderr.write(r.stderr)
    return obj


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    if force:
        for o in glob.glob(os.path.join(BUILD, "*.o")):
            os.remove(o)
    with concurrent.futures.ThreadPoolExecutor(max_workers=os.cpu_count() or 4) as ex:
        objs = list(ex.map(lambda s: _compile(s, verbose_ptxas), srcs))
    if force or _stale(LIB, objs):
        tmp = LIB + f".tmp{os.getpid()}"
        r = subprocess.run([NVCC, *ARCH, "-shared", "-o", tmp, *objs], capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, LIB)
    if force or _stale(MARSHAL, [os.path.join(PKG, "marshal.c"), os.path.join(INCLUDE, "moe.h")]):
        build_marshal(torch_include=_torch_include())
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose_ptxas="--ptxas-v" in sys.argv))
