"""Builds libflint_moe.so (the C-ABI library) in-tree for sm_103a with nvcc.

    python -m moe_decode_router_gb300.build [--force] [-v]

Each .cu file under csrc/ compiles to its own object in parallel; the objects
link into moe_decode_router_gb300/_lib/libflint_moe.so.  csrc/binding.cpp, the
compiled marshalling of the short Python calls, becomes an extension module beside
it, whose name holds what it was built against: the interpreter and the installed
torch.  A rebuild happens only when a source or header is newer than what was
built.  Every build works in a folder of its own and moves what it made into place,
so that several processes may build at once.  Without the module (no host compiler,
no torch headers) every call is marshalled by Python: a warning, not an error.
"""

from __future__ import annotations

import argparse
import concurrent.futures as cf
import importlib.util
import os
import re
import shutil
import subprocess
import sys
import sysconfig
import tempfile
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT_DIR = os.path.join(PKG, "_lib")
LIB = os.path.join(OUT_DIR, "libflint_moe.so")
BINDING_SRC = os.path.join(CSRC, "binding.cpp")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc_path() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libflint_moe.so")


def _sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _deps():
    files = _sources() + [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    files += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE) if f.endswith(".h")]
    files.append(os.path.abspath(__file__))
    return files


def _torch_dir() -> str:
    return importlib.util.find_spec("torch").submodule_search_locations[0]


def _torch_version() -> str:
    with open(os.path.join(_torch_dir(), "version.py")) as f:
        found = re.search(r"""^__version__ = ['"]([^'"]+)""", f.read(), re.M)
    return found.group(1) if found else "unknown"


def binding_path() -> str:
    """The compiled marshalling for this interpreter and this torch; one built for others is another file."""
    return os.path.join(OUT_DIR, f"_flint_binding-torch{_torch_version()}{sysconfig.get_config_var('EXT_SUFFIX')}")


def _newer(out, deps) -> bool:
    return os.path.exists(out) and all(os.path.getmtime(f) <= os.path.getmtime(out) for f in deps)


def library_up_to_date() -> bool:
    return _newer(LIB, _deps())


def binding_up_to_date() -> bool:
    header = os.path.join(INCLUDE, "flint_moe.h")
    return _newer(binding_path(), [BINDING_SRC, header, os.path.join(_torch_dir(), "version.py")])


def up_to_date() -> bool:
    return library_up_to_date() and binding_up_to_date()


def _run(cmd, what):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")
    return r


def _build_binding(work: str) -> None:
    torch_dir = _torch_dir()
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc_path())))
    tmp = os.path.join(work, "binding.so")
    _run([os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", BINDING_SRC, "-o", tmp,
          "-I", INCLUDE, "-I", sysconfig.get_paths()["include"], "-I", os.path.join(torch_dir, "include"),
          "-I", os.path.join(cuda, "include"), "-L", os.path.join(torch_dir, "lib"),
          "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"], f"g++ on {BINDING_SRC}")
    os.replace(tmp, binding_path())


def _build_library(work: str, verbose: bool) -> None:
    nvcc = nvcc_path()
    common = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC]
    if verbose:
        common += ["-Xptxas", "-v"]

    def compile_one(src):
        obj = os.path.join(work, os.path.basename(src)[:-3] + ".o")
        return obj, _run([nvcc, *common, "-c", src, "-o", obj], f"nvcc on {src}").stderr

    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        results = list(ex.map(compile_one, _sources()))
    if verbose:
        for _, log in results:
            sys.stderr.write(log)
    tmp = os.path.join(work, "lib.so")
    _run([nvcc, *ARCH, "-shared", "-o", tmp, *(o for o, _ in results)], "the link")
    os.replace(tmp, LIB)


def build(force: bool = False, verbose: bool = False) -> str:
    library, binding = force or not library_up_to_date(), force or not binding_up_to_date()
    if not library and not binding:
        return LIB
    os.makedirs(OUT_DIR, exist_ok=True)
    with tempfile.TemporaryDirectory(prefix="build-", dir=OUT_DIR) as work, cf.ThreadPoolExecutor(1) as ex:
        made = ex.submit(_build_binding, work) if binding else None
        if library:
            _build_library(work, verbose)
        try:
            if made:
                made.result()
        except Exception as e:
            warnings.warn(f"the compiled marshalling could not be built; Python marshals every call instead: {e}",
                          RuntimeWarning)
    return LIB


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("-v", "--verbose", action="store_true")
    a = ap.parse_args()
    print(build(force=a.force, verbose=a.verbose))


if __name__ == "__main__":
    main()
