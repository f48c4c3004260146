"""Builds libnts.so in-tree (normalization_token_split_gb300/_build/) with
nvcc for sm_103a, and the Python extension beside it (marshal_nts.*.so, from
binding/) with g++.  Translation units compile in parallel; a unit is rebuilt
only when it or a header is newer than its object, and a library is linked anew
when it is older than one of its objects: what an earlier run compiled and did
not come to link is linked by the next.  libnts.so needs neither torch nor
Python: without their headers it is built alone, with a warning, and the
operators that need the extension raise.

    python -m normalization_token_split_gb300.build [--force] [--verbose]
"""
from __future__ import annotations

import argparse
import glob
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

from ._abi import marshal_name, torch_dir

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(BUILD, "libnts.so")
BINDING = os.path.join(PKG, "binding", "marshal.cpp")
MARSHAL = os.path.join(BUILD, marshal_name())

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _cuda_home() -> str:
    env = os.environ.get("CUDA_HOME") or os.environ.get("CUDA_PATH")
    if env:
        return env
    nvcc = shutil.which("nvcc")
    if nvcc:
        return os.path.dirname(os.path.dirname(os.path.realpath(nvcc)))
    return "/usr/local/cuda"


def _newest_header() -> float:
    hdrs = glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        glob.glob(os.path.join(INCLUDE, "*.h"))
    return max((os.path.getmtime(h) for h in hdrs), default=0.0)


def _compile_cmd(src: str, obj: str, nvcc: str, cuda: str, verbose: bool):
    inc = ["-I", INCLUDE, "-I", CSRC]
    if src.endswith(".cu"):
        cmd = [nvcc, *ARCH, "-lineinfo", "-O3", "-std=c++17", "-Xcompiler", "-fPIC",
               "-Xcompiler", "-fvisibility=hidden", *inc, "-c", src, "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
    else:
        cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
               "-I", os.path.join(cuda, "include"), *inc, "-c", src, "-o", obj]
    return cmd


def _missing_for_binding():
    """What the extension needs and this machine lacks, or None."""
    torch = torch_dir()
    if torch is None:
        return "torch"
    for path in (os.path.join(sysconfig.get_paths()["include"], "Python.h"),
                 os.path.join(torch, "include", "ATen", "ATen.h"),
                 os.path.join(torch, "lib", "libc10_cuda.so")):
        if not os.path.exists(path):
            return path
    return None


def _binding_cmds(obj: str, cuda: str):
    """Compile and link commands of the Python extension (torch's headers and
    libraries, this interpreter, libnts.so beside it)."""
    torch = torch_dir()
    inc = [os.path.join(torch, "include"), os.path.join(torch, "include/torch/csrc/api/include"),
           sysconfig.get_paths()["include"], os.path.join(cuda, "include"), INCLUDE]
    compile_ = ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
                *[a for i in inc for a in ("-I", i)], "-c", BINDING, "-o", obj]
    tmp = MARSHAL + f".{os.getpid()}.tmp"
    link = ["g++", "-shared", "-o", tmp, obj, "-L", BUILD, "-l:libnts.so", "-Wl,-rpath,$ORIGIN",
            "-L", os.path.join(torch, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10"]
    return compile_, link, tmp


def _stale(target: str, *inputs: str) -> bool:
    """Whether target is missing or older than one of its inputs."""
    return not os.path.exists(target) or \
        os.path.getmtime(target) < max(map(os.path.getmtime, inputs))


def build(force: bool = False, verbose: bool = False) -> str:
    cuda = _cuda_home()
    nvcc = os.path.join(cuda, "bin", "nvcc")
    if not os.path.exists(nvcc):
        nvcc = shutil.which("nvcc") or nvcc
    os.makedirs(BUILD, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cpp")))
    hdr_time = _newest_header()
    jobs = []
    objs = []
    for src in srcs:
        obj = os.path.join(BUILD, os.path.basename(src) + ".o")
        objs.append(obj)
        stale = (force or not os.path.exists(obj)
                 or os.path.getmtime(obj) < max(os.path.getmtime(src), hdr_time))
        if stale:
            jobs.append(_compile_cmd(src, obj, nvcc, cuda, verbose))

    # the binding: its object compiles along with the others, and links after libnts.so
    obj = MARSHAL[:-len("so")] + "o"
    missing = _missing_for_binding()
    if missing is not None:
        print(f"the extension is not built ({missing} is missing): the operators around a "
              "projection will raise", file=sys.stderr)
    else:
        bind, bind_link, bind_tmp = _binding_cmds(obj, cuda)
        if force or _stale(obj, BINDING, os.path.join(INCLUDE, "nts.h")):
            jobs.append(bind)

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        return cmd, r

    failed = []
    if jobs:
        with ThreadPoolExecutor(max_workers=min(len(jobs), os.cpu_count() or 4)) as ex:
            for cmd, r in ex.map(run, jobs):
                out = (r.stdout + r.stderr).strip()
                if verbose and out:
                    print(out)
                if r.returncode != 0:
                    failed.append((cmd, out))
    if failed:
        msg = "\n\n".join(" ".join(c) + "\n" + o for c, o in failed)
        raise RuntimeError("libnts compilation failed:\n" + msg)

    if force or _stale(LIB, *objs):
        tmp = LIB + f".{os.getpid()}.tmp"
        link = [nvcc, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs,
                "-lpthread", "-ldl", "-lrt"]
        r = subprocess.run(link, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("libnts link failed:\n" + " ".join(link) + "\n" + r.stdout + r.stderr)
        os.replace(tmp, LIB)
    if missing is None and (force or _stale(MARSHAL, obj)):
        r = subprocess.run(bind_link, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("binding link failed:\n" + " ".join(bind_link) + "\n" + r.stdout +
                               r.stderr)
        os.replace(bind_tmp, MARSHAL)
    return LIB


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true", help="print ptxas resource usage")
    a = ap.parse_args(argv)
    print(build(force=a.force, verbose=a.verbose))


if __name__ == "__main__":
    sys.exit(main())
