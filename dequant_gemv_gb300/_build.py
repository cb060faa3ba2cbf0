"""In-tree build of libq4nx.so for sm_103a (nvcc, one -gencode, parallel TUs).

``python dequant_gemv_gb300/_build.py`` or ``build()`` compiles every
``csrc/*.cu`` into ``_objs/`` and links ``libq4nx.so`` next to this file, and
the native binding of the decode-step operators (``csrc/serving_binding.cpp``,
g++ against the installed torch's headers) into ``_serving.so``.  The library comes
first and needs neither: where the binding cannot be built, build() raises with the
library in place, and without torch (C callers) there is no binding to build.
Objects are rebuilt only when a source or header is newer.  No cmake.
"""
from __future__ import annotations

import glob
import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
OBJS = os.path.join(PKG, "_objs")
LIB = os.path.join(PKG, "libq4nx.so")
BINDING = os.path.join(PKG, "_serving.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-fno-strict-aliasing"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libq4nx.so")


def _headers() -> list[str]:
    return glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(ROOT, "include", "*.h"))


def _stale(target: str, deps: list[str]) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _other_link(target: str, record: str, cmd: list[str]) -> bool:
    """Whether target was linked by another command than cmd, as record tells: going back to an
    earlier torch finds that one's object older than the binding of the later one."""
    try:
        with open(record) as f:
            return f.read() != "\n".join(cmd)
    except OSError:
        return os.path.exists(target)


def _binding_jobs(nvcc: str) -> tuple[list[str], list[str]] | None:
    """Commands that compile and link the native binding against the installed torch (None: there is none)."""
    spec = importlib.util.find_spec("torch")
    if spec is None:
        return None
    torch = list(spec.submodule_search_locations)[0]
    inc = [os.path.join(torch, "include"), os.path.join(torch, "include", "torch", "csrc", "api", "include"),
           os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include"),
           "/usr/local/cuda/include", sysconfig.get_paths()["include"]]
    gxx = os.environ.get("CXX") or shutil.which("g++") or "g++"
    # the object's name holds torch's version: another torch is another build
    obj = os.path.join(OBJS, f"serving_binding-torch{importlib.metadata.version('torch')}.o")
    compile_ = [gxx, "-O2", "-std=c++17", "-fPIC", "-fno-strict-aliasing", *[f"-I{d}" for d in inc], "-c",
                os.path.join(CSRC, "serving_binding.cpp"), "-o", obj]
    link = [gxx, "-shared", obj, f"-L{os.path.join(torch, 'lib')}", "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10_cuda",
            "-lc10", f"-L{PKG}", "-lq4nx", "-Wl,-rpath,$ORIGIN", "-o"]
    return compile_, link


def build(verbose: bool = False, ptxas_info: bool = False) -> str:
    nvcc = _nvcc()
    os.makedirs(OBJS, exist_ok=True)
    sources = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    headers = _headers()
    jobs = []
    for src in sources:
        obj = os.path.join(OBJS, os.path.basename(src)[:-3] + ".o")
        if _stale(obj, [src] + headers) or ptxas_info:
            cmd = [nvcc, *ARCH, *FLAGS, "-c", src, "-o", obj]
            if ptxas_info:
                cmd.insert(1, "-Xptxas=-v")
            jobs.append((src, cmd))

    binding, link = _binding_jobs(nvcc) or (None, None)
    source = os.path.join(CSRC, "serving_binding.cpp")
    if binding and _stale(binding[-1], [source, os.path.join(ROOT, "include", "q4nx.h")]):
        jobs.append((source, binding))

    def run(job):
        src, cmd = job
        try:
            p = subprocess.run(cmd, capture_output=True, text=True)
        except OSError as e:                               # no such compiler
            return src, 127, f"{e}\n"
        return src, p.returncode, p.stdout + p.stderr

    if jobs:
        with ThreadPoolExecutor(max_workers=max(1, min(len(jobs), os.cpu_count() or 4))) as ex:
            results = list(ex.map(run, jobs))
        failed = [s for s, rc, out in results if rc != 0]
        for s, rc, out in results:
            if verbose or ptxas_info or rc != 0:
                sys.stderr.write(f"== {os.path.basename(s)} (rc={rc})\n{out}")
        if any(s != source for s in failed):
            raise RuntimeError("compilation failed on: " + ", ".join(os.path.basename(s) for s in failed))
    else:
        failed = []
    objs = [os.path.join(OBJS, os.path.basename(s)[:-3] + ".o") for s in sources]
    if _stale(LIB, objs) or jobs:
        tmp = LIB + f".tmp{os.getpid()}"
        cmd = [nvcc, *ARCH, "-shared", "-cudart", "shared", "-o", tmp, *objs]
        p = subprocess.run(cmd, capture_output=True, text=True)
        if p.returncode != 0:
            raise RuntimeError("link of libq4nx.so failed:\n" + p.stdout + p.stderr)
        os.replace(tmp, LIB)
    if failed:
        raise RuntimeError("compilation failed on: serving_binding.cpp (libq4nx.so is built; without the binding the "
                           "package's products work and the operators around them refuse)")
    record = os.path.join(OBJS, "serving_binding.link")
    if binding and (_stale(BINDING, [binding[-1]]) or _other_link(BINDING, record, link)):
        tmp = BINDING + f".tmp{os.getpid()}"
        _, rc, out = run((source, [*link, tmp]))
        if rc != 0:
            raise RuntimeError("link of _serving.so failed:\n" + out)
        os.replace(tmp, BINDING)
        with open(record, "w") as f:
            f.write("\n".join(link))
    return LIB


if __name__ == "__main__":
    print(build(verbose=True, ptxas_info="--ptxas" in sys.argv))
