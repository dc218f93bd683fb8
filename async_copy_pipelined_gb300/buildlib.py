"""Build the CUDA library in-tree: nvcc, sm_103a only, translation units in parallel.

    python -m async_copy_pipelined_gb300.buildlib [--force] [--verbose]

Produces ``async_copy_pipelined_gb300/_build/libpipelined_gemm.so`` and, by g++
against the installed torch, the feed-forward operators' native binding
``_build/_feedforward.so`` (both git-ignored).  The library needs no torch and is
put in place first; where torch is without CUDA the binding is left out, and where
it does not compile a warning says so (the compiler's words are in
``_build/binding.log``): the operators' calls then go through ctypes.
``-Xptxas -v`` resource lines (registers, spills, shared memory per kernel)
are written next to it in ``ptxas.log``.
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import contextlib
import fcntl
import glob
import importlib.util
import os
import re
import shutil
import subprocess
import sys
import sysconfig
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
OUT_DIR = os.path.join(HERE, "_build")
LIB_NAME = "libpipelined_gemm.so"
LIB_PATH = os.path.join(OUT_DIR, LIB_NAME)
INCLUDE = os.path.join(ROOT, "include")
BINDING_SOURCE = os.path.join(CSRC, "feedforward_binding.cpp")
BINDING_PATH = os.path.join(OUT_DIR, "_feedforward.so")
BINDING_LOG = os.path.join(OUT_DIR, "binding.log")

GENCODE = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-std=c++17", "-O3", "-lineinfo", *GENCODE, "-Xcompiler", "-fPIC,-O2",
              "-Xptxas", "-v", "--expt-relaxed-constexpr", f"-I{INCLUDE}", f"-I{CSRC}"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: set NVCC or put the CUDA toolkit on PATH")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _headers():
    return glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)]


def _deps():
    return (_sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + _headers())


def _torch_dir():
    """Where torch is (None: not installed, which the library does not need; the
    binding, used with torch's tensors, is then left out)."""
    spec = importlib.util.find_spec("torch")
    return list(spec.submodule_search_locations)[0] if spec else None


def _binding_wanted() -> bool:
    """Whether torch has the CUDA streams that the binding asks for."""
    torch_dir = _torch_dir()
    return bool(torch_dir) and os.path.exists(os.path.join(torch_dir, "lib", "libc10_cuda.so"))


def _torch_version() -> str:
    """The installed torch's, all of it, without importing torch."""
    try:
        with open(os.path.join(_torch_dir(), "version.py")) as f:
            return re.search(r"^__version__ = ['\"]([^'\"]+)['\"]", f.read(), flags=re.M).group(1)
    except (OSError, AttributeError):
        return "unknown"


def _newer(path: str, deps) -> bool:
    return os.path.exists(path) and all(os.path.getmtime(d) <= os.path.getmtime(path) for d in deps)


def _library_up_to_date() -> bool:
    return _newer(LIB_PATH, _deps())


def _binding_up_to_date() -> bool:
    """Built, or found not to compile, from what is there now and for the torch
    that is installed; or not wanted."""
    if not _binding_wanted():
        return True
    if not _newer(BINDING_LOG, [BINDING_SOURCE] + _headers()):
        return False
    with open(BINDING_LOG) as f:
        said = f.readline().strip()
    return said == _binding_line("failed") or (said == _binding_line("built") and os.path.exists(BINDING_PATH))


def _binding_line(outcome: str) -> str:
    """First line of the binding's log."""
    return f"torch {_torch_version()}: {outcome}"


def up_to_date() -> bool:
    return _library_up_to_date() and _binding_up_to_date()


def _compile(src: str) -> tuple[str, str]:
    obj = os.path.join(OUT_DIR, os.path.basename(src).replace(".cu", ".o"))
    cmd = [nvcc(), *NVCC_FLAGS, "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
    return obj, r.stderr


def _compile_binding() -> str:
    """The binding as a shared object, beside its place."""
    torch_dir = _torch_dir()
    headers = os.path.join(torch_dir, "include")
    lib = os.path.join(torch_dir, "lib")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
    tmp = BINDING_PATH + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX") or "g++", "-std=c++17", "-O2", "-fPIC", "-shared", "-fvisibility=hidden",
           f'-DBINDING_TORCH="{_torch_version()}"', f"-I{INCLUDE}", f"-I{sysconfig.get_paths()['include']}", f"-I{headers}",
           f"-I{os.path.join(headers, 'torch', 'csrc', 'api', 'include')}", f"-I{cuda}", BINDING_SOURCE, "-o", tmp,
           f"-L{lib}", "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for {os.path.basename(BINDING_SOURCE)}:\n{r.stdout}\n{r.stderr}")
    return tmp


@contextlib.contextmanager
def _build_lock():
    """One build at a time per tree (several ranks of one job may call build())."""
    os.makedirs(OUT_DIR, exist_ok=True)
    with open(os.path.join(OUT_DIR, ".build.lock"), "w") as f:
        fcntl.flock(f, fcntl.LOCK_EX)
        try:
            yield
        finally:
            fcntl.flock(f, fcntl.LOCK_UN)


def build(force: bool = False, verbose: bool = False) -> str:
    if force or not up_to_date():
        with _build_lock():
            _build_locked(force, verbose)  # what another process built while we waited is not built again
    if _binding_wanted() and not os.path.exists(BINDING_PATH):
        warnings.warn("the feed-forward operators' native binding does not build here, so that their calls take the "
                      f"host longer: see {BINDING_LOG}, and build again with --force", RuntimeWarning, stacklevel=2)
    return LIB_PATH


def _build_locked(force: bool, verbose: bool) -> None:
    library = force or not _library_up_to_date()
    wanted = _binding_wanted() and (force or not _binding_up_to_date())
    srcs = _sources() if library else []
    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(srcs) + 1, os.cpu_count() or 4))) as ex:
        binding = ex.submit(_compile_binding) if wanted else None
        results = list(ex.map(_compile, srcs))
    if library:
        _link(results, verbose)
    if binding:
        try:
            os.replace(binding.result(), BINDING_PATH)
            said = _binding_line("built")
        except Exception as e:  # the library does not need it
            said = f"{_binding_line('failed')}\n{e}"
            if os.path.exists(BINDING_PATH):  # of other sources
                os.remove(BINDING_PATH)
        with open(BINDING_LOG, "w") as f:
            f.write(said + "\n")


def _link(results, verbose: bool) -> None:
    logs = "\n".join(f"== {os.path.basename(o)}\n{err}" for o, err in results)
    with open(os.path.join(OUT_DIR, "ptxas.log"), "w") as f:
        f.write(logs)
    if verbose:
        print(logs)
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    cmd = [nvcc(), "-shared", *GENCODE, "-o", tmp, *[o for o, _ in results], "-cudart", "static"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB_PATH)


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__)
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    args = ap.parse_args(argv)
    path = build(force=args.force, verbose=args.verbose)
    print(path)


if __name__ == "__main__":
    sys.exit(main())
