"""Build libdvl.so in place: nvcc for the CUDA sources (sm_103a only), g++
for the host-only ranks builder, one shared library with the CUDA runtime
linked statically; and _step.so, the Python module of the drafting step's
operators (g++ against PyTorch's headers), which calls libdvl.so and is left
out where there is no PyTorch with CUDA.  Object files go to _build/ next to
this file."""
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
STEP_FOR = os.path.join(BUILD, "step_binding.for")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                     "-Xptxas", "-v", "-I", INCLUDE, "-I", CSRC]
CXX_FLAGS = ["-O2", "-std=c++17", "-fPIC", "-I", INCLUDE]


def _nvcc() -> str:
    for c in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("nvcc not found")


def _torch_dir() -> str | None:
    """Where a PyTorch with CUDA is installed, or None: libdvl.so needs none."""
    spec = importlib.util.find_spec("torch")
    if spec is None or spec.origin is None:
        return None
    torch = os.path.dirname(spec.origin)
    return torch if os.path.exists(os.path.join(torch, "lib", "libc10_cuda.so")) else None


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
    return cu + cpp + hdr + [os.path.abspath(__file__)]


def _newer(out: str, deps) -> bool:
    return os.path.exists(out) and all(os.path.getmtime(p) <= os.path.getmtime(out) for p in deps)


def _step_made_for() -> str:
    """The Python and the PyTorch that _step.so is compiled for: neither runs another's."""
    torch = _torch_dir()
    with open(os.path.join(torch, "version.py")) as f:
        return f"{sysconfig.get_config_var('SOABI')}\n{torch}\n{f.read()}"


def _step_up_to_date() -> bool:
    if _torch_dir() is None:
        return True
    if not os.path.exists(STEP_FOR) or open(STEP_FOR).read() != _step_made_for():
        return False
    return _newer(
        STEP, [os.path.join(CSRC, "step_binding.cc"), os.path.join(INCLUDE, "dvl.h"), os.path.abspath(__file__)])


def up_to_date() -> bool:
    return _newer(LIB, _deps()) and _step_up_to_date()


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile and link libdvl.so and _step.so, each where a source is newer."""
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    with_lib = force or not _newer(LIB, _deps())
    with_step = _torch_dir() is not None and (force or not _step_up_to_date())
    jobs = []
    step_obj = os.path.join(BUILD, "step_binding.o")
    if with_step:  # the longest compile first
        jobs.append((_step_compile(step_obj), step_obj, "step_binding.cc"))
    if with_lib:
        nvcc = _nvcc()
        cu, cpp = sources()
        for src in cu:
            obj = os.path.join(BUILD, os.path.basename(src) + ".o")
            jobs.append(([nvcc, *NVCC_FLAGS, "-c", src, "-o", obj], obj, src))
        for src in cpp:
            obj = os.path.join(BUILD, os.path.basename(src) + ".o")
            jobs.append((["g++", *CXX_FLAGS, "-c", src, "-o", obj], obj, src))

    def run(job):
        cmd, obj, src = job
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"compile failed: {src}\n{r.stdout}\n{r.stderr}")
        with open(obj + ".log", "w") as f:
            f.write(r.stdout + r.stderr)
        return obj

    def link(cmd, out):
        tmp = out + f".tmp{os.getpid()}"
        r = subprocess.run(cmd(tmp), capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed: {os.path.basename(out)}\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, out)

    with cf.ThreadPoolExecutor(max(1, min(len(jobs), os.cpu_count() or 1))) as ex:
        objs = [o for o in ex.map(run, jobs) if o != step_obj]
    if with_lib:
        link(lambda tmp: [nvcc, *ARCH, "-shared", "-o", tmp, *objs], LIB)
    if with_step:
        link(lambda tmp: _step_link(step_obj, tmp), STEP)
        with open(STEP_FOR, "w") as f:
            f.write(_step_made_for())
    if verbose:
        for o in objs:
            if os.path.exists(o + ".log"):
                sys.stdout.write(open(o + ".log").read())
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
