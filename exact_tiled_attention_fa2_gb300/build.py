"""Build the in-tree CUDA library ``libfa2_gb300.so`` for sm_103a.

Each translation unit under ``csrc/`` is compiled in parallel with nvcc
(``-gencode arch=compute_103a,code=sm_103a -lineinfo``) and linked into one
shared library with the CUDA runtime linked statically, so loading it needs no
driver until the first CUDA call.  The driver API entry point for TMA tensor
maps is fetched at run time.

The binding of the paged-cache calls to torch (``_paged_binding``, a Python
extension module with its ABI in its name) is compiled beside it with g++
against torch's headers and linked to the library; again when torch changes.
The library needs neither: without torch only it is built, and it is linked
before a binding that does not compile is reported.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD_DIR = os.path.join(HERE, "_build")
LIB_NAME = "libfa2_gb300.so"
LIB_PATH = os.path.join(HERE, LIB_NAME)
BINDING_SOURCE = "paged_binding.cpp"
BINDING_PATH = os.path.join(HERE, "_paged_binding" + (sysconfig.get_config_var("EXT_SUFFIX") or ".so"))
PUBLIC_HEADER = os.path.join(os.path.dirname(HERE), "include", "fa2.h")
SOURCES = ["fa2_abi.cu", "fa2_fwd_d64.cu", "fa2_fwd_d128.cu", "fa2_fwd_d256.cu", "fa2_bwd_d64.cu", "fa2_bwd_d128.cu",
           "fa2_bwd_d256.cu", "fa2_decode_d64.cu", "fa2_decode_d128.cu", "fa2_decode_d256.cu",
           "fa2_paged_abi.cu", "fa2_paged_cache.cu", "fa2_paged_d64.cu", "fa2_paged_d128.cu", "fa2_paged_d256.cu"]
HEADERS = ["fa2_common.cuh", "fa2_tile.cuh", "fa2_fwd_dbuf.cuh", "fa2_bwd.cuh", "fa2_bwd64.cuh", "fa2_bwd256.cuh",
           "fa2_decode.cuh", "fa2_decode_tc.cuh", "fa2_paged.cuh", "fa2_paged.h",
           "fa2_internal.h",
           "sm103_ptx.cuh"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
                     "--expt-relaxed-constexpr"]


def _nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found; the CUDA toolkit is required to build " + LIB_NAME)
    return cand


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _binding_commands(obj: str, out: str):
    """Compile and link commands of the binding."""
    import torch

    base = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    compile_cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-Wall", "-D_GLIBCXX_USE_CXX11_ABI=%d"
                   % int(torch._C._GLIBCXX_USE_CXX11_ABI), "-I", os.path.join(base, "include"),
                   "-I", os.path.join(base, "include", "torch", "csrc", "api", "include"),
                   "-I", sysconfig.get_paths()["include"], "-I", os.path.join(cuda, "include"),
                   "-c", os.path.join(CSRC, BINDING_SOURCE), "-o", obj]
    link_cmd = ["g++", "-shared", "-o", out, obj, "-L", HERE, "-l:" + LIB_NAME, "-L", os.path.join(base, "lib"),
                "-ltorch", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python", "-lc10", "-lc10_cuda", "-L", os.path.join(cuda, "lib64"),
                "-lcudart", "-Wl,-rpath,$ORIGIN"]
    return compile_cmd, link_cmd


class _Binding:
    """The binding's compilation, beside the library's: start(), then link() once the library is there."""

    def __init__(self, force: bool, verbose: bool):
        self.obj, self.stamp = (os.path.join(BUILD_DIR, "paged_binding" + x) for x in (".o", ".stamp"))
        self.tmp, self.verbose, self.proc = BINDING_PATH + ".tmp%d" % os.getpid(), verbose, None
        try:
            import torch
        except ImportError:   # nothing could call it
            self.compile_cmd = None
            return
        self.compile_cmd, self.link_cmd = _binding_commands(self.obj, self.tmp)
        self.made_for = "\n".join([torch.__version__, sys.version] + self.compile_cmd)
        self.force = force or not self._made_for_this()

    def _made_for_this(self) -> bool:
        try:
            with open(self.stamp) as f:
                return f.read() == self.made_for
        except OSError:
            return False

    def start(self) -> None:
        if self.compile_cmd and (self.force or _stale(self.obj, [os.path.join(CSRC, BINDING_SOURCE), PUBLIC_HEADER])):
            if self.verbose:
                print(" ".join(self.compile_cmd), flush=True)
            if os.path.exists(self.stamp):
                os.remove(self.stamp)
            self.proc = subprocess.Popen(self.compile_cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)

    def link(self) -> None:
        if not self.compile_cmd:
            return
        if self.proc:
            out, _ = self.proc.communicate()
            if self.verbose or self.proc.returncode:
                sys.stdout.write(out)
            if self.proc.returncode:
                raise RuntimeError("compilation failed for %s (%s is built)" % (BINDING_SOURCE, LIB_NAME))
        if self.proc or _stale(BINDING_PATH, [self.obj]):
            subprocess.run(self.link_cmd, check=True)
            os.replace(self.tmp, BINDING_PATH)
        if self.proc:
            with open(self.stamp, "w") as f:
                f.write(self.made_for)


def build(force: bool = False, verbose: bool = False, ptxas_verbose: bool = False) -> str:
    """Compile (if stale) and return the path of the shared library."""
    os.makedirs(BUILD_DIR, exist_ok=True)
    nvcc = _nvcc()
    hdrs = [os.path.join(CSRC, h) for h in HEADERS] + [PUBLIC_HEADER]
    objs, procs = [], []
    for src in SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(BUILD_DIR, src.replace(".cu", ".o"))
        objs.append(o)
        if force or _stale(o, [s] + hdrs):
            cmd = [nvcc] + NVCC_FLAGS + (["-Xptxas", "-v"] if ptxas_verbose else []) + ["-c", s, "-o", o]
            if verbose:
                print(" ".join(cmd), flush=True)
            procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)))
    binding = _Binding(force, verbose)
    binding.start()
    failed = []
    for src, p in procs:
        out, _ = p.communicate()
        if verbose or ptxas_verbose or p.returncode:
            sys.stdout.write(out)
        if p.returncode:
            failed.append(src)
    if failed:
        raise RuntimeError("nvcc failed for " + ", ".join(failed))
    if force or procs or _stale(LIB_PATH, objs):
        tmp = LIB_PATH + ".tmp%d" % os.getpid()
        cmd = [nvcc] + ARCH + ["-shared", "-o", tmp] + objs
        subprocess.run(cmd, check=True)
        os.replace(tmp, LIB_PATH)
    binding.link()
    return LIB_PATH


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, ptxas_verbose="-v" in sys.argv))
