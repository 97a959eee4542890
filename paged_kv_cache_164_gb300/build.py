"""Builds the pkv CUDA library (``_build/libpkv.so``) for sm_103a with nvcc.

Each ``csrc/*.cu`` file is compiled to an object in parallel, then linked into
one shared object with the CUDA runtime linked statically, so the library
depends on nothing but the driver at run time.

``csrc/pkv_binding.cpp`` becomes ``_build/pkv_binding.so``, the quick form of
some Python calls, which needs the headers of Python and torch.  Where they are
missing it is left out with a warning: those calls are then checked and passed
on in Python.
"""
from __future__ import annotations

import concurrent.futures
import contextlib
import glob
import hashlib
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT_DIR = os.path.join(HERE, "_build")
LIB = os.path.join(OUT_DIR, "libpkv.so")
BINDING_SOURCE = os.path.join(CSRC, "pkv_binding.cpp")
BINDING = os.path.join(OUT_DIR, "pkv_binding.so")
# The NaN-sentinel debug build (-DPKV_DEBUG), kept apart from the normal one.
DEBUG_DIR = os.path.join(HERE, "_build_debug")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE,
              "-I", CSRC, "--expt-relaxed-constexpr"]


def _nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found")
    return cand


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _inputs_digest(flags) -> str:
    h = hashlib.sha256()
    h.update(" ".join(flags).encode())
    files = _sources() + sorted(glob.glob(os.path.join(CSRC, "*.cuh"))) + \
        [os.path.join(INCLUDE, "pkv.h"), os.path.abspath(__file__)]
    for f in files:
        h.update(f.encode())
        with open(f, "rb") as fh:
            h.update(fh.read())
    return h.hexdigest()


def _binding_command():
    import torch
    from torch.utils.cpp_extension import include_paths, library_paths
    flags = ["-O2", "-std=c++17", "-fPIC", "-shared", "-I", INCLUDE,
             "-I", sysconfig.get_paths()["include"],
             "-I", os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include"),
             f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
             f'-DPKV_TORCH_VERSION="{torch.__version__}"']
    for d in include_paths():
        flags += ["-isystem", d]
    for d in library_paths():
        flags += ["-L", d]
    libs = ["-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    return ["g++", *flags, BINDING_SOURCE, *libs]


def build_binding(force: bool = False) -> bool:
    """Compiles the binding module unless an up-to-date build exists; False: it
    cannot be built here."""
    tmp = BINDING + f".tmp{os.getpid()}"
    try:
        cmd = _binding_command()
        h = hashlib.sha256(" ".join([sys.version, *cmd]).encode())
        for f in (BINDING_SOURCE, os.path.join(INCLUDE, "pkv.h"), os.path.abspath(__file__)):
            with open(f, "rb") as fh:
                h.update(fh.read())
        stamp = BINDING + ".stamp"
        if not force and os.path.exists(BINDING) and os.path.exists(stamp):
            with open(stamp) as f:
                if f.read().strip() == h.hexdigest():
                    return True
        os.makedirs(OUT_DIR, exist_ok=True)
        r = subprocess.run([*cmd, "-o", tmp], capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(r.stderr[-2000:])
        # (another process may be building too: each step holds whatever that one has done)
        _remove(stamp)
        os.replace(tmp, BINDING)
        with open(tmp, "w") as f:
            f.write(h.hexdigest())
        os.replace(tmp, stamp)
        return True
    except (ImportError, AttributeError, OSError, RuntimeError) as e:
        print(f"pkv: the quick binding is left out: {e}", file=sys.stderr)
        for f in (tmp, BINDING):  # never one of other headers than these
            _remove(f)
        return False


def _remove(path: str) -> None:
    with contextlib.suppress(OSError):
        os.remove(path)


def build(force: bool = False, verbose: bool = False, debug: bool = False) -> str:
    """Compiles and links the library, and the binding module, unless up-to-date
    builds exist.

    ``debug``: the -DPKV_DEBUG build (NaN-filled ring slots), in its own
    directory.  PKV_NVCC_EXTRA adds flags to either build.
    """
    extra = os.environ.get("PKV_NVCC_EXTRA", "").split() + (["-DPKV_DEBUG"] if debug else [])
    out_dir = DEBUG_DIR if debug else OUT_DIR
    lib = os.path.join(out_dir, "libpkv.so")
    digest = _inputs_digest(extra)
    stamp = os.path.join(out_dir, "stamp")
    if not force and os.path.exists(lib) and os.path.exists(stamp):
        with open(stamp) as f:
            if f.read().strip() == digest:
                build_binding()
                return lib
    os.makedirs(out_dir, exist_ok=True)
    nvcc = _nvcc()

    def compile_one(src):
        obj = os.path.join(out_dir, os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc, *ARCH, *NVCC_FLAGS, *extra, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr, file=sys.stderr)
        return obj

    with concurrent.futures.ThreadPoolExecutor(max_workers=os.cpu_count() or 4) as ex:
        binding = ex.submit(build_binding, force)
        objs = list(ex.map(compile_one, _sources()))
        binding.result()
    tmp = lib + f".tmp{os.getpid()}"
    cmd = [nvcc, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, lib)
    with open(stamp, "w") as f:
        f.write(digest)
    return lib


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv,
                debug="--debug" in sys.argv))
