"""Build the KDA prefill C-ABI library (``libkda.so``) in-tree for sm_103a.

Each ``csrc/*.cu`` translation unit is compiled in parallel with nvcc, then
the objects are linked into ``kimi_delta_attention_kda_gb300/libkda.so``
(CUDA runtime linked statically, so the library needs only the driver).
``csrc/kda_torch.cpp``, the operators' calls on PyTorch tensors, becomes the
module ``_kda_torch.so`` beside it, built against the installed PyTorch.  The
library does not need it: without a PyTorch for CUDA it is left out.  A note
beside the module says which PyTorch and Python it was built for: it is built
again for others, and not loaded with them.
"""

from __future__ import annotations

import concurrent.futures
import contextlib
import glob
import importlib.util
import json
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD_DIR = os.path.join(HERE, "_build")
LIB_PATH = os.path.join(HERE, "libkda.so")
TORCH_PATH = os.path.join(HERE, "_kda_torch.so")
TORCH_NOTE = os.path.join(BUILD_DIR, "kda_torch.json")
ARCH_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
              "--expt-relaxed-constexpr"]


def nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found")
    return cand


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _headers():
    return sorted(glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) +
                  glob.glob(os.path.join(HERE, "..", "include", "*.h")))


def _stale(target, deps):
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _torch_dir():
    """The installed PyTorch's folder, or None without one that has CUDA."""
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.submodule_search_locations:
        return None
    path = spec.submodule_search_locations[0]
    return path if os.path.exists(os.path.join(path, "lib", "libc10_cuda.so")) else None


def _torch_command(torch_dir, target):
    """The compiler's command for ``csrc/kda_torch.cpp``."""
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    include = [os.path.join(torch_dir, "include"), os.path.join(torch_dir, "include/torch/csrc/api/include"),
               sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    return (["g++", "-O2", "-std=c++17", "-fPIC", "-shared"] + ["-I" + d for d in include] +
            ["-L" + os.path.join(torch_dir, "lib"), os.path.join(CSRC, "kda_torch.cpp"),
             "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda", "-o", target])


def torch_abi():
    """What ``_kda_torch.so`` is built against: the installed PyTorch's version
    file as it is (the version, the commit, CUDA's version) and Python's ABI."""
    torch_dir = _torch_dir()
    if torch_dir is None:
        return None
    with open(os.path.join(torch_dir, "version.py")) as fh:
        return {"torch": fh.read(), "python": sysconfig.get_config_var("SOABI")}


def torch_note():
    """The note of the module that is there: ``torch_abi()`` and the compiler's
    command, or None."""
    try:
        with open(TORCH_NOTE) as fh:
            return json.load(fh)
    except (OSError, ValueError):
        return None


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    """Compile and link ``libkda.so`` and ``_kda_torch.so``; returns the former's path.
    A module that does not compile is an error only once the library is linked."""
    os.makedirs(BUILD_DIR, exist_ok=True)
    srcs = _sources()
    hdrs = _headers()
    objs = []
    jobs = []
    for src in srcs:
        obj = os.path.join(BUILD_DIR, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        if force or ptxas_info or _stale(obj, [src] + hdrs):
            cmd = [nvcc()] + NVCC_FLAGS + ARCH_FLAGS + ["-c", src, "-o", obj]
            if ptxas_info:
                cmd += ["-Xptxas", "-v"]
            jobs.append(cmd)

    torch_tmp = TORCH_PATH + ".tmp.%d" % os.getpid()
    torch_src = os.path.join(CSRC, "kda_torch.cpp")
    torch_dir = _torch_dir()
    if torch_dir is None:
        sys.stderr.write("no PyTorch for CUDA: _kda_torch.so is not built, libkda.so does without\n")
    torch_job = None
    if torch_dir is not None:
        # (The package's own path is left out: it may be reached by several.)
        note = {"abi": torch_abi(), "command": [x.replace(HERE, "") for x in _torch_command(torch_dir, TORCH_PATH)]}
        if force or _stale(TORCH_PATH, [torch_src] + hdrs) or torch_note() != note:
            torch_job = _torch_command(torch_dir, torch_tmp)

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        return cmd, r

    failed = []
    torch_failed = False
    with concurrent.futures.ThreadPoolExecutor(max_workers=len(jobs) + 1) as ex:
        for cmd, r in ex.map(run, jobs + ([torch_job] if torch_job else [])):
            if verbose or ptxas_info or r.returncode != 0:
                sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
            if r.returncode != 0 and cmd is torch_job:
                torch_failed = True
            elif r.returncode != 0:
                failed.append(cmd[cmd.index("-c") + 1])
    if failed:
        raise RuntimeError("the compiler failed for: " + ", ".join(failed))
    if force or jobs or _stale(LIB_PATH, objs):
        tmp = LIB_PATH + ".tmp.%d" % os.getpid()
        cmd = [nvcc()] + ARCH_FLAGS + ["-shared", "-o", tmp] + objs
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("link failed:\n" + r.stdout + r.stderr)
        os.replace(tmp, LIB_PATH)
    if torch_failed:
        raise RuntimeError("libkda.so is built, but the compiler failed for: " + torch_src)
    if torch_job:
        # (Between the two there is a module without its note: it is not loaded.)
        with contextlib.suppress(FileNotFoundError):
            os.remove(TORCH_NOTE)
        os.replace(torch_tmp, TORCH_PATH)
        tmp = TORCH_NOTE + ".tmp.%d" % os.getpid()
        with open(tmp, "w") as fh:
            json.dump(note, fh)
        os.replace(tmp, TORCH_NOTE)
    return LIB_PATH


TEST_HOOKS_LIB = os.path.join(HERE, "libkda_testhooks.so")
TEST_WAIT_BOUND_CYCLES = 100000


def build_test_hooks(force: bool = False) -> str:
    """Compile the test-only library ``libkda_testhooks.so``: the hooks of
    ``csrc/kda_test_hooks.cu`` with the library's wait bound cut to 10^5
    cycles, so that a test can make a bounded wait run out.  Never linked
    into ``libkda.so``."""
    src = os.path.join(CSRC, "kda_test_hooks.cu")
    if force or _stale(TEST_HOOKS_LIB, [src] + _headers()):
        tmp = TEST_HOOKS_LIB + ".tmp.%d" % os.getpid()
        cmd = ([nvcc()] + NVCC_FLAGS + ARCH_FLAGS +
               ["-DKDA_TEST_HOOKS", "-DKDA_WAIT_BOUND_CYCLES=%dLL" % TEST_WAIT_BOUND_CYCLES,
                "-shared", "-o", tmp, src])
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed for the test hooks:\n" + r.stdout + r.stderr)
        os.replace(tmp, TEST_HOOKS_LIB)
    return TEST_HOOKS_LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas-info" in sys.argv)
    print(LIB_PATH)
