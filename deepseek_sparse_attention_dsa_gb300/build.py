"""Build the CUDA library (libdsa_gb300.so) in-tree for sm_103a.

    python -m deepseek_sparse_attention_dsa_gb300.build

Each translation unit under csrc/ is compiled by nvcc in parallel, then linked
into deepseek_sparse_attention_dsa_gb300/_build/libdsa_gb300.so (git-ignored).
csrc/binding.cpp, the tensors' way into the calls whose host time counts, becomes
the extension module _build/_dsa_binding.so beside it.  The library needs nvcc
alone and is there before the module is linked; where the module cannot be built
(no torch, or one without CUDA or headers) a note says why, and only the calls
that go through it are missing.
"""
from __future__ import annotations

import concurrent.futures as cf
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT_DIR = os.path.join(PKG, "_build")
LIB = os.path.join(OUT_DIR, "libdsa_gb300.so")
BINDING = os.path.join(OUT_DIR, "_dsa_binding.so")
BINDING_SOURCE = "binding.cpp"
SOURCES = ["api.cu", "plan_device.cu", "store_keys.cu", "quantize.cu", "indexer.cu", "indexer_f8q.cu", "topk.cu",
           "attend.cu", "msa.cu", "rmsnorm.cu", "quantize_rows.cu", "project.cu",
           "rotary.cu", "append.cu", "prefix.cu", "prefix_tc.cu", "static_scratch.cu", "selftest.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libdsa_gb300.so")
    return cand


def _newest(files) -> float:
    return max(os.path.getmtime(f) for f in files)


def _library_deps():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f != BINDING_SOURCE]
    return _newest(files + [os.path.join(INCLUDE, "dsa.h"), __file__])


def _binding_deps():
    return _newest([os.path.join(CSRC, BINDING_SOURCE), os.path.join(INCLUDE, "dsa.h"), __file__])


def _binding_key() -> str:
    """What the module was compiled against: the interpreter's ABI and the
    installed torch (its version file, read without importing it)."""
    spec = importlib.util.find_spec("torch")
    version = os.path.join(os.path.dirname(spec.origin), "version.py") if spec and spec.origin else ""
    text = open(version).read() if os.path.exists(version) else "no torch"
    return "%s\n%s\n%s" % (sysconfig.get_config_var("SOABI"), version, text)


def library_up_to_date() -> bool:
    return os.path.exists(LIB) and os.path.getmtime(LIB) >= _library_deps()


def binding_matches(path: str) -> bool:
    """Whether the module at this path was built for this interpreter and torch."""
    key = path + ".key"
    return os.path.exists(key) and open(key).read() == _binding_key()


def binding_up_to_date() -> bool:
    return os.path.exists(BINDING) and os.path.getmtime(BINDING) >= _binding_deps() and binding_matches(BINDING)


def up_to_date() -> bool:
    return library_up_to_date() and binding_up_to_date()


def _compile_binding() -> str:
    """binding.cpp -> an object (the module is linked once the library is there)."""
    import torch
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(_nvcc()))), "include")
    obj = os.path.join(OUT_DIR, "binding.o")
    cmd = [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-I", INCLUDE, "-isystem", inc,
           "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"), "-isystem", cuda,
           "-isystem", sysconfig.get_paths()["include"], "-c", os.path.join(CSRC, BINDING_SOURCE), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("g++ failed for binding.cpp:\n%s%s" % (r.stdout, r.stderr))
    return obj


def _link_binding(obj: str):
    import torch
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = BINDING + ".%d.tmp" % os.getpid()
    cmd = [shutil.which("g++") or "g++", "-shared", "-o", tmp, obj, "-L", OUT_DIR, "-l:libdsa_gb300.so", "-L", lib,
           "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link of the binding failed:\n%s%s" % (r.stdout, r.stderr))
    os.replace(tmp, BINDING)
    with open(BINDING + ".key", "w") as f:
        f.write(_binding_key())


def build(force: bool = False, verbose: bool = False, ptxas_verbose: bool = False) -> str:
    """Builds what is out of date; returns the library's path.  Raises where the library does not build."""
    library, binding = force or not library_up_to_date(), force or not binding_up_to_date()
    if not library and not binding:
        return LIB
    os.makedirs(OUT_DIR, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        obj = ex.submit(_compile_binding) if binding else None
        if library:
            _build_library(ex, verbose, ptxas_verbose)
        if obj is not None:
            try:
                _link_binding(obj.result())
            except Exception as e:
                sys.stderr.write("_dsa_binding.so is not built; the 8-bit rows and projections cannot be called from Python "
                                 "(%s: %s)\n" % (type(e).__name__, e))
                # a module of other sources, or of another torch, is none
                for f in (BINDING, BINDING + ".key"):
                    if os.path.exists(f):
                        os.remove(f)
    return LIB


def _build_library(ex: cf.Executor, verbose: bool, ptxas_verbose: bool):
    nvcc = _nvcc()
    common = [nvcc, *ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE,
              "--expt-relaxed-constexpr"]
    if ptxas_verbose:
        common += ["-Xptxas", "-v"]

    def compile_one(src):
        obj = os.path.join(OUT_DIR, os.path.splitext(src)[0] + ".o")
        cmd = common + ["-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed for %s:\n%s%s" % (src, r.stdout, r.stderr))
        if verbose or ptxas_verbose:
            sys.stderr.write(r.stdout + r.stderr)
        return obj

    objs = list(ex.map(compile_one, SOURCES))
    tmp = LIB + ".%d.tmp" % os.getpid()
    cuda_lib = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "lib64")
    cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs, "-Xlinker", "-soname", "-Xlinker", "libdsa_gb300.so", "-lcudart", "-Xlinker", "-rpath", "-Xlinker", cuda_lib]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n%s%s" % (r.stdout, r.stderr))
    os.replace(tmp, LIB)


if __name__ == "__main__":
    print(build(force=True, verbose=True, ptxas_verbose="-v" in sys.argv))
