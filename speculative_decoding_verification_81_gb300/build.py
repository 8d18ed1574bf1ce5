"""Build libspecverify.so in place (nvcc, sm_103a only, one -gencode), and
the extension that marshals the paged-cache calls (g++, against torch).

The translation units compile in parallel into ``_build/`` beside the
package and link into ``libspecverify.so`` next to this file.  A rebuild
happens only when a source or header is newer than the library.  The
extension's file name carries the Python and torch that it was built for, so
another one's is not found.  Where it cannot be built, a warning says why and
the library is used without it: the binding's own marshalling takes every call.
"""
from __future__ import annotations

import glob
import os
import re
import subprocess
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(ROOT, "_build")
LIB_PATH = os.path.join(HERE, "libspecverify.so")
BIND_SOURCE = os.path.join(CSRC, "sv_bind.cpp")

SOURCES = ["sv_api.cu", "sv_attention.cu", "sv_attention_tc.cu", "sv_vocab.cu", "sv_compact.cu",
           "sv_noalloc.cu", "sv_step.cu", "sv_pages.cu",
           "sv_chunk.cu", "sv_chunk_tc.cu", "sv_chunk_few.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", f"-I{INCLUDE}"]


def _nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _inputs():
    return ([os.path.join(CSRC, s) for s in SOURCES] + glob.glob(os.path.join(CSRC, "*.cuh"))
            + glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(INCLUDE, "*.h")))


def up_to_date(lib_path: str = LIB_PATH) -> bool:
    if not os.path.exists(lib_path):
        return False
    t = os.path.getmtime(lib_path)
    return all(os.path.getmtime(p) <= t for p in _inputs())


def bind_path() -> str:
    """The extension's file for the running interpreter and its torch."""
    import sysconfig

    import torch
    tag = f"{sysconfig.get_config_var('SOABI')}-torch-{torch.__version__}"
    return os.path.join(HERE, f"_sv_bind.{re.sub('[^A-Za-z0-9-]', '_', tag)}.so")


def _start_bind(path):
    """g++ at work on the extension (torch's and Python's headers): the process
    and the file it writes."""
    import sysconfig

    import torch
    troot = os.path.join(os.path.dirname(torch.__file__))
    inc = [os.path.join(troot, "include"), os.path.join(troot, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"],
           os.path.join(os.path.dirname(os.path.dirname(_nvcc())) or "/usr/local/cuda", "include")]
    tmp = path + f".tmp{os.getpid()}"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", *[f"-isystem{i}" for i in inc], BIND_SOURCE, "-o", tmp,
           f"-L{os.path.join(troot, 'lib')}", "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10_cuda", "-lc10"]
    return subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT), tmp


def bind_up_to_date(path: str) -> bool:
    if not os.path.exists(path):
        return False
    t = os.path.getmtime(path)
    return all(os.path.getmtime(p) <= t for p in [BIND_SOURCE, *glob.glob(os.path.join(INCLUDE, "*.h"))])


def _finish_bind(path, proc, tmp) -> None:
    out, _ = proc.communicate()
    if proc.returncode == 0:
        os.replace(tmp, path)
        return
    if os.path.exists(path):  # an older source's: it may call another interface
        os.remove(path)
    warnings.warn(f"the extension is left out, g++ failed for {BIND_SOURCE}:\n{out.decode(errors='replace')}")


def build(force: bool = False, verbose: bool = False, defines=(), lib_path: str = LIB_PATH,
          build_dir: str = BUILD_DIR) -> str:
    """Compile the library; `defines` (e.g. SV_PHASE_STAMPS) go to every
    translation unit, for a diagnostic build at another `lib_path`."""
    bind = None
    if lib_path == LIB_PATH:
        try:
            path = bind_path()
            if force or not bind_up_to_date(path):
                bind = path, *_start_bind(path)
        except (ImportError, OSError) as e:  # no torch, no g++
            warnings.warn(f"the extension is left out: {e}")
    try:
        return _build_lib(force, verbose, defines, lib_path, build_dir)
    finally:
        if bind is not None:
            _finish_bind(*bind)


def _build_lib(force, verbose, defines, lib_path, build_dir) -> str:
    if not force and up_to_date(lib_path):
        return lib_path
    os.makedirs(build_dir, exist_ok=True)
    nvcc = _nvcc()
    procs = []
    objs = []
    for src in SOURCES:
        obj = os.path.join(build_dir, src.replace(".cu", ".o"))
        objs.append(obj)
        cmd = [nvcc, *ARCH, *NVCC_FLAGS, *[f"-D{d}" for d in defines], "-c",
               os.path.join(CSRC, src), "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
    failed = []
    for src, p in procs:
        out, _ = p.communicate()
        if verbose or p.returncode != 0:
            print(out.decode(errors="replace"))
        if p.returncode != 0:
            failed.append(src)
    if failed:
        raise RuntimeError(f"nvcc failed for {failed}")
    tmp = lib_path + f".tmp{os.getpid()}"
    subprocess.check_call([nvcc, "-shared", *ARCH, *objs, "-o", tmp])
    os.replace(tmp, lib_path)
    return lib_path


if __name__ == "__main__":
    import sys
    build(force="--force" in sys.argv, verbose="-v" in sys.argv)
    print(LIB_PATH)
