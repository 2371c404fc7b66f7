"""Build libdvl.so in place: nvcc for the CUDA sources (sm_103a only), g++
for the host-only ranks builder, one shared library with the CUDA runtime
linked statically; and _step.so, the Python module of the drafting step's
operators (g++ against PyTorch's headers), which calls libdvl.so.  Object
files go to _build/ next to this file."""
from __future__ import annotations

import concurrent.futures as cf
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libdvl.so")
STEP = os.path.join(HERE, "_step.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                     "-Xptxas", "-v", "-I", INCLUDE, "-I", CSRC]
CXX_FLAGS = ["-O2", "-std=c++17", "-fPIC", "-I", INCLUDE]


def _nvcc() -> str:
    for c in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("nvcc not found")


def _torch_dir() -> str:
    spec = importlib.util.find_spec("torch")
    if spec is None or spec.origin is None:
        raise RuntimeError("PyTorch not found")
    return os.path.dirname(spec.origin)


def _step_compile(obj: str):
    """The command that compiles the Python module's source."""
    torch = _torch_dir()
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    inc = [INCLUDE, sysconfig.get_paths()["include"], os.path.join(torch, "include"),
           os.path.join(torch, "include", "torch", "csrc", "api", "include"), os.path.join(cuda, "include")]
    flags = [x for d in inc for x in ("-isystem" if d != INCLUDE else "-I", d)]
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-D_GLIBCXX_USE_CXX11_ABI=1",
            *flags, "-c", os.path.join(CSRC, "step_binding.cc"), "-o", obj]


def _step_link(obj: str, out: str):
    libs = os.path.join(_torch_dir(), "lib")
    return ["g++", "-shared", "-o", out, obj, f"-L{HERE}", "-l:libdvl.so", f"-L{libs}", "-ltorch_python", "-ltorch", "-ltorch_cpu",
            "-lc10_cuda", "-lc10", "-Wl,-rpath,$ORIGIN"]


def sources():
    cu = sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))
    cpp = sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cpp"))
    return cu, cpp


def _deps():
    cu, cpp = sources()
    hdr = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".h", ".cuh"))]
    hdr.append(os.path.join(INCLUDE, "dvl.h"))
    hdr.append(os.path.join(CSRC, "step_binding.cc"))
    return cu + cpp + hdr + [os.path.abspath(__file__)]


def up_to_date() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(STEP):
        return False
    t = min(os.path.getmtime(LIB), os.path.getmtime(STEP))
    return all(os.path.getmtime(p) <= t for p in _deps())


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile and link libdvl.so and _step.so if any source is newer."""
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()
    cu, cpp = sources()
    jobs = []
    for src in cu:
        obj = os.path.join(BUILD, os.path.basename(src) + ".o")
        jobs.append(([nvcc, *NVCC_FLAGS, "-c", src, "-o", obj], obj, src))
    for src in cpp:
        obj = os.path.join(BUILD, os.path.basename(src) + ".o")
        jobs.append((["g++", *CXX_FLAGS, "-c", src, "-o", obj], obj, src))

    step_obj = os.path.join(BUILD, "step_binding.o")
    # the longest compile first
    jobs.insert(0, (_step_compile(step_obj), step_obj, "step_binding.cc"))

    def run(job):
        cmd, obj, src = job
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"compile failed: {src}\n{r.stdout}\n{r.stderr}")
        with open(obj + ".log", "w") as f:
            f.write(r.stdout + r.stderr)
        return obj

    with cf.ThreadPoolExecutor(max(1, min(len(jobs), os.cpu_count() or 1))) as ex:
        objs = list(ex.map(run, jobs))[1:]
    tmp = LIB + f".tmp{os.getpid()}"
    r = subprocess.run([nvcc, *ARCH, "-shared", "-o", tmp, *objs], capture_output=True,
                       text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    tmp = STEP + f".tmp{os.getpid()}"
    r = subprocess.run(_step_link(step_obj, tmp), capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed: _step.so\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, STEP)
    if verbose:
        for o in objs:
            if os.path.exists(o + ".log"):
                sys.stdout.write(open(o + ".log").read())
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
