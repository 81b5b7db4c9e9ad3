"""Build the CUDA libraries in-tree: io_aware_exact_fa2_gb300/libfa2_gb300.so (the
dense passes, include/fa2.h), libfa2_cache_gb300.so (the 8-bit cache, include/fa2_cache.h)
and libfa2_paged_gb300.so (the 16-bit cache and the position rotation, include/fa2_paged.h),
then, where there is a torch with CUDA, the Python module that hands tensors to the last.

nvcc compiles each translation unit in csrc/ for sm_103a (in parallel), then
links the shared libraries with the CUDA runtime linked statically and only the
``fa2_*`` C symbols exported (a linker version script), so a library never
interposes on, or binds to, another copy of the CUDA runtime in the process.

    python -m io_aware_exact_fa2_gb300.build [--force] [--verbose]
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import hashlib
import importlib.metadata
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
BUILD = os.path.join(PKG, "_build")
LIB_NAME = "libfa2_gb300.so"
LIB_PATH = os.path.join(PKG, LIB_NAME)
SOURCES = ["fa2_api.cu", "fa2_noalloc.cu", "fa2_fwd_d64.cu", "fa2_fwd_d128.cu", "fa2_fwd_d256.cu",
           "fa2_fwd_fp8_d128.cu", "fa2_bwd.cu"]
# the 8-bit cache is a library of its own, so that the dense one's boundary stays what fa2.h declares
CACHE_LIB_NAME = "libfa2_cache_gb300.so"
CACHE_LIB_PATH = os.path.join(PKG, CACHE_LIB_NAME)
CACHE_SOURCES = ["fa2_cache_api.cu", "fa2_cache_move.cu", "fa2_cache_attn_d64.cu", "fa2_cache_attn_d128.cu",
                 "fa2_cache_attn_d256.cu"]
# the 16-bit cache and the rotation, likewise
PAGED_LIB_NAME = "libfa2_paged_gb300.so"
PAGED_LIB_PATH = os.path.join(PKG, PAGED_LIB_NAME)
PAGED_SOURCES = ["fa2_paged_api.cu", "fa2_paged_move.cu", "fa2_paged_attn_d64.cu", "fa2_paged_attn_d128.cu",
                 "fa2_paged_attn_d256.cu"]
# the 16-bit library's Python side: a module that takes torch tensors apart
PY_SOURCE = "fa2_paged_py.cpp"
PY_MODULE = "_fa2_paged_py"
PY_MODULE_PATH = os.path.join(PKG, PY_MODULE + ".so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "--expt-relaxed-constexpr",
              "-Xcompiler", "-fPIC,-fvisibility=hidden", "-Xptxas", "-v",
              "-I" + INCLUDE, "-I" + CSRC]


def nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found; the CUDA toolkit is required to build the library")
    return path


def source_digest() -> str:
    """Hash of the libraries' sources and the public headers (for staleness checks)."""
    h = hashlib.sha256()
    files = sorted(f for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh", ".h")))
    for f in files:
        with open(os.path.join(CSRC, f), "rb") as fh:
            h.update(f.encode() + b"\0" + fh.read())
    for f in ("fa2.h", "fa2_cache.h", "fa2_paged.h"):
        with open(os.path.join(INCLUDE, f), "rb") as fh:
            h.update(fh.read())
    return h.hexdigest()[:16]


def torch_with_cuda() -> str | None:
    """The folder of this Python's torch (found, not imported: that takes seconds); None if there is
    none, or one without CUDA."""
    spec = importlib.util.find_spec("torch")
    path = os.path.dirname(spec.origin) if spec and spec.origin else None
    return path if path and os.path.exists(os.path.join(path, "lib", "libc10_cuda.so")) else None


def module_digest() -> str:
    """Hash of the module's source and headers, and of what it is built against."""
    h = hashlib.sha256(f"{sys.version} torch {importlib.metadata.version('torch')}".encode())
    for f in (os.path.join(CSRC, PY_SOURCE), os.path.join(INCLUDE, "fa2.h"), os.path.join(INCLUDE, "fa2_paged.h")):
        with open(f, "rb") as fh:
            h.update(fh.read())
    return h.hexdigest()[:16]


def kernel_digest() -> str:
    """Hash of the sources that decide what the forward kernel does on the device: the
    kernel template, its PTX wrappers, the launch logic and the per-D instantiations (not
    the C ABI wrapper or the header), so that recorded profiler counters stay valid
    across host-only changes.  Whole-line comments and blank lines are left out, so a
    change to them alone keeps the recorded counters."""
    h = hashlib.sha256()
    files = sorted(f for f in os.listdir(CSRC)
                   if f in ("fa2_fwd_kernel.cuh", "sm103_ptx.cuh", "fa2_launch.cuh", "fa2_split_ranges.h")
                   or (f.startswith("fa2_fwd_") and f.endswith(".cu")))
    for f in files:
        with open(os.path.join(CSRC, f), "rb") as fh:
            code = [ln.rstrip() for ln in fh.read().split(b"\n")]
        code = [ln for ln in code if ln.strip() and not ln.lstrip().startswith(b"//")]
        h.update(f.encode() + b"\0" + b"\n".join(code))
    return h.hexdigest()[:16]


def _stamp_path() -> str:
    return os.path.join(BUILD, "digest.txt")


def _module_stamp_path() -> str:
    return os.path.join(BUILD, PY_MODULE + ".digest.txt")


def _stamped(stamp: str, digest: str) -> bool:
    if not os.path.exists(stamp):
        return False
    with open(stamp) as fh:
        return fh.read().strip() == digest


def _libraries_fresh() -> bool:
    return all(os.path.exists(p) for p in (LIB_PATH, CACHE_LIB_PATH, PAGED_LIB_PATH)) and \
        _stamped(_stamp_path(), source_digest())


def _module_fresh() -> bool:
    """True also where no module can be built."""
    return torch_with_cuda() is None or (os.path.exists(PY_MODULE_PATH) and _stamped(_module_stamp_path(), module_digest()))


def is_fresh() -> bool:
    return _libraries_fresh() and _module_fresh()


def _compile(src: str, verbose: bool, build_dir: str, extra_flags) -> str:
    obj = os.path.join(build_dir, os.path.splitext(src)[0] + ".o")
    cmd = [nvcc(), *ARCH, *NVCC_FLAGS, *extra_flags, "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    log = os.path.join(build_dir, os.path.splitext(src)[0] + ".ptxas.txt")
    with open(log, "w") as fh:
        fh.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
    if verbose:
        sys.stdout.write(r.stderr)
    return obj


def _build_module(bdir: str) -> None:
    """PY_SOURCE against this Python and its torch."""
    torch = torch_with_cuda()
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    tmp = PY_MODULE_PATH + f".tmp{os.getpid()}"
    cmd = [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden", "-I" + INCLUDE,
           "-I" + sysconfig.get_paths()["include"], "-I" + os.path.join(torch, "include"),
           "-I" + os.path.join(torch, "include", "torch", "csrc", "api", "include"), "-I" + os.path.join(cuda, "include"),
           os.path.join(CSRC, PY_SOURCE), "-o", tmp, "-L" + os.path.join(torch, "lib"),
           "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    with open(os.path.join(bdir, PY_MODULE + ".txt"), "w") as fh:
        fh.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on {PY_SOURCE}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, PY_MODULE_PATH)
    with open(_module_stamp_path(), "w") as fh:
        fh.write(module_digest())


def _link(objs, out: str, bdir: str) -> None:
    vscript = os.path.join(bdir, "exports.map")
    tmp = out + f".tmp{os.getpid()}"
    cmd = [nvcc(), *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs,
           "-Xlinker", f"--version-script={vscript}", "-Xlinker", "-Bsymbolic"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, out)


def build(force: bool = False, verbose: bool = False, extra_flags=(), lib_path: str | None = None,
          build_dir: str | None = None) -> str:
    """Compile and link the libraries unless they are already up to date, and the Python module.
    Returns the path of the dense library.

    extra_flags / lib_path / build_dir build a separate copy of the dense library (e.g.
    with -D tile overrides for tuning) without touching the in-tree ones.
    """
    default = lib_path is None and not extra_flags
    libraries = force or not default or not _libraries_fresh()
    module = default and torch_with_cuda() is not None and (force or not _module_fresh())
    out = LIB_PATH if lib_path is None else lib_path
    bdir = BUILD if build_dir is None else build_dir
    if not libraries and not module:
        return out
    os.makedirs(bdir, exist_ok=True)
    sources = SOURCES + (CACHE_SOURCES + PAGED_SOURCES if default else [])
    with cf.ThreadPoolExecutor(max_workers=len(sources) + 1) as ex:
        # (beside the libraries, which do not wait for it nor fail with it)
        done = ex.submit(_build_module, bdir) if module else None
        if libraries:
            objs = list(ex.map(lambda s: _compile(s, verbose, bdir, tuple(extra_flags)), sources))
            with open(os.path.join(bdir, "exports.map"), "w") as fh:
                fh.write("{\n  global: fa2_*;\n  local: *;\n};\n")
            _link(objs[:len(SOURCES)], out, bdir)
            if default:
                rest = objs[len(SOURCES):]
                _link(rest[:len(CACHE_SOURCES)], CACHE_LIB_PATH, bdir)
                _link(rest[len(CACHE_SOURCES):], PAGED_LIB_PATH, bdir)
                with open(_stamp_path(), "w") as fh:
                    fh.write(source_digest())
        if done:
            done.result()
    if default and torch_with_cuda() is None:
        print(f"{PY_MODULE} is not built: there is no torch with CUDA (the C libraries need none)", file=sys.stderr)
    return out


def main() -> None:
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    args = ap.parse_args()
    print(build(force=args.force, verbose=args.verbose))


if __name__ == "__main__":
    main()
