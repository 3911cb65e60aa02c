"""Build libgdr.so in-tree: every csrc/*.cu compiled for sm_103a only, in parallel, then linked; and
gdr_binding.so, the torch binding of the block operators (csrc/gdr_binding.cpp, g++).

    python -m chunked_gated_delta_04_gb300.build [--force] [--delay]

--delay builds the delay-injection variant libgdr_delay.so instead (-DGDR_DEBUG_DELAY: one role
at each cross-role hand-off sleeps a short bounded time; see csrc/gdr_instrument.cuh), which the
tests compare bit for bit with libgdr.so.

nvcc flags: -gencode arch=compute_103a,code=sm_103a -O3 -std=c++17 -lineinfo, no fast-math.
Each device pass checks __CUDA_ARCH_FEAT_SM103_ALL and fails if the gencode was lost.
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import glob
import os
import shutil
import subprocess

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libgdr.so")
BUILD_DIR = os.path.join(PKG, "_build")
DELAY_LIB = os.path.join(PKG, "libgdr_delay.so")
DELAY_BUILD_DIR = os.path.join(PKG, "_build_delay")
BINDING = os.path.join(PKG, "gdr_binding.so")
BINDING_SRC = os.path.join(CSRC, "gdr_binding.cpp")
INCLUDE = os.path.join(os.path.dirname(PKG), "include")
GENCODE = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc_path() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libgdr.so")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + sorted(glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh"))) + [
        os.path.join(INCLUDE, "gdr.h"), os.path.join(INCLUDE, "gdr_block.h")]


def _target(delay: bool):
    """(library path, object directory, flags stamp) of the normal or the delay-injection build."""
    lib = DELAY_LIB if delay else LIB
    return lib, (DELAY_BUILD_DIR if delay else BUILD_DIR), lib + ".flags"


def _flags(delay: bool = False) -> list:
    flags = GENCODE + ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-I", INCLUDE,
                       "--expt-relaxed-constexpr", "-Xptxas", "-warn-spills"]
    if delay:
        flags += ["-DGDR_DEBUG_DELAY=1"]
    return flags + os.environ.get("GDR_NVCC_EXTRA", "").split()


def up_to_date(delay: bool = False) -> bool:
    lib, _, stamp = _target(delay)
    if not os.path.exists(lib) or not os.path.exists(stamp):
        return False
    with open(stamp) as f:
        if f.read() != " ".join(_flags(delay)):
            return False
    t = os.path.getmtime(lib)
    return all(os.path.getmtime(p) <= t for p in _deps())


def _binding_flags() -> list:
    import sysconfig

    import torch

    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc_path())))
    inc = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
           os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    return (["-O2", "-std=c++17", "-fPIC", "-shared", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}"]
            + [f for i in inc for f in ("-isystem", i)]
            + ["-L" + os.path.join(root, "lib"), "-Wl,-rpath," + os.path.join(root, "lib")])


def build_binding(force: bool = False) -> str:
    """Builds gdr_binding.so for the torch that is installed unless it is up to date; returns its path."""
    import torch

    flags = _binding_flags()
    stamp, stamp_path = " ".join([torch.__version__] + flags), BINDING + ".flags"
    deps = [BINDING_SRC, os.path.join(INCLUDE, "gdr.h"), os.path.join(INCLUDE, "gdr_block.h")]
    if not force and os.path.exists(BINDING) and os.path.exists(stamp_path):
        with open(stamp_path) as f:
            if f.read() == stamp and all(os.path.getmtime(p) <= os.path.getmtime(BINDING) for p in deps):
                return BINDING
    tmp = BINDING + f".tmp{os.getpid()}"
    r = subprocess.run(["g++"] + flags + [BINDING_SRC, "-o", tmp, "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python"],
                       capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on {BINDING_SRC}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING)
    with open(stamp_path, "w") as f:
        f.write(stamp)
    return BINDING


def build(force: bool = False, delay: bool = False, verbose: bool = False) -> str:
    """Builds libgdr.so and gdr_binding.so (or, with delay, libgdr_delay.so) unless they are up to date;
    returns the library's path."""
    lib, build_dir, stamp_path = _target(delay)
    if not force and up_to_date(delay):
        if not delay:
            build_binding()
        return lib
    nvcc = nvcc_path()
    os.makedirs(build_dir, exist_ok=True)
    flags = _flags(delay)
    stamp = " ".join(flags)
    if verbose:
        flags = flags + ["-Xptxas", "-v"]

    def compile_one(src):
        obj = os.path.join(build_dir, os.path.basename(src) + ".o")
        cmd = [nvcc] + flags + ["-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        return obj, r.stderr

    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        binding = None if delay else ex.submit(build_binding, force)
        results = list(ex.map(compile_one, _sources()))
        if binding is not None:
            binding.result()
    if verbose:
        for _, err in results:
            print(err)
    objs = [o for o, _ in results]
    tmp = lib + f".tmp{os.getpid()}"
    cmd = [nvcc] + GENCODE + ["-shared", "-o", tmp] + objs + ["-lcudart_static", "-ldl",
                                                                "-lrt", "-lpthread"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, lib)
    with open(stamp_path, "w") as f:
        f.write(stamp)
    return lib


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--delay", action="store_true", help="build the delay-injection variant libgdr_delay.so")
    ap.add_argument("-v", "--verbose", action="store_true")
    args = ap.parse_args()
    print(build(force=args.force, delay=args.delay, verbose=args.verbose))
