"""Build libsq.so (the CUDA kernels + C ABI) and libsq_peak.so (the tensor-core
peak measurement used as the GEMM roofline denominator) in-tree with nvcc for
sm_100a, and _sqbind.so (libsq's calls for PyTorch tensors) with the host
compiler against the installed torch."""
from __future__ import annotations

import importlib.metadata
import importlib.util
import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
SO = os.path.join(HERE, "libsq.so")
# translation units of libsq.so and the headers each includes
UNITS = {
    "libsq.cu": ["common.cuh", "host.cuh", "ptx_sm100.cuh", "calib.cuh", "robust.cuh", "quant.cuh", "gemm.cuh"],
    "libsq_fp4.cu": ["common.cuh", "host.cuh", "ptx_sm100.cuh", "gemm.cuh", "fp4.cuh", "gemm_fp4.cuh", "kvcache.cuh"],
}
OBJ = os.path.join(HERE, "_build")
PEAK_SO = os.path.join(HERE, "libsq_peak.so")
PEAK_SOURCES = ["peak.cu"]
PEAK_HEADERS = ["common.cuh", "ptx_sm100.cuh"]
BIND_SO = os.path.join(HERE, "_sqbind.so")
BIND_SOURCES = ["bind.cpp"]
BIND_STAMP = os.path.join(OBJ, "_sqbind.versions")

NVCC_FLAGS = [
    "-O3", "-std=c++17", "-lineinfo",
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-Xcompiler", "-fPIC",
    "--expt-relaxed-constexpr",
]


def nvcc() -> str:
    for c in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc"):
        if c and os.path.exists(c):
            return c
    return "nvcc"


def _stale(so: str, sources, headers) -> bool:
    if not os.path.exists(so):
        return True
    t = os.path.getmtime(so)
    deps = [os.path.join(CSRC, f) for f in list(sources) + list(headers)] + [os.path.join(ROOT, "include", "sq.h")]
    return any(os.path.getmtime(d) > t for d in deps)


def _nvcc_cmd(out: str, args, extra) -> list[str]:
    return [nvcc(), *NVCC_FLAGS, *(extra or []), "-I", os.path.join(ROOT, "include"), "-I", CSRC, "-o", out, *args]


def _bind_cmd(out: str) -> list[str]:
    torch_dir = importlib.util.find_spec("torch").submodule_search_locations[0]
    cuda = os.path.dirname(os.path.dirname(nvcc())) or "/usr/local/cuda"
    includes = [os.path.join(ROOT, "include"), sysconfig.get_paths()["include"], os.path.join(torch_dir, "include"),
                os.path.join(cuda, "include")]
    return [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", *[f"-I{d}" for d in includes], "-o", out,
            *[os.path.join(CSRC, f) for f in BIND_SOURCES], "-L" + os.path.join(torch_dir, "lib"), "-lc10", "-lc10_cuda",
            "-ltorch_cpu", "-ltorch_python", "-L" + HERE, "-l:libsq.so", "-Wl,-rpath,$ORIGIN"]


def _bind_versions() -> str:
    """What _sqbind.so is compiled against besides its sources: another Python or torch makes it stale."""
    return f"python {sys.version} {sysconfig.get_config_var('SOABI')}\ntorch {importlib.metadata.version('torch')}\n"


def _bind_stale(so: str, stamp: str) -> bool:
    if _stale(so, BIND_SOURCES, []) or not os.path.exists(stamp):
        return True
    with open(stamp) as f:
        return f.read() != _bind_versions()


def _run(jobs, verbose: bool) -> None:
    """Runs compilers side by side.  A job is (temporary, final, command): what a command has made takes its final
    name; the first failure is raised after all have ended."""
    procs = []
    for _, _, cmd in jobs:
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        procs.append(subprocess.Popen(cmd))
    failed = None
    for (tmp, final, cmd), p in zip(jobs, procs):
        if p.wait() == 0:
            os.replace(tmp, final)
        else:
            failed = failed or subprocess.CalledProcessError(p.returncode, cmd)
    if failed:
        raise failed


def build(force: bool = False, verbose: bool = False, extra: list[str] | None = None) -> str:
    os.makedirs(OBJ, exist_ok=True)
    tag = f".tmp{os.getpid()}"

    def job(final, args, flags=extra):
        return final + tag, final, _nvcc_cmd(final + tag, args, flags)

    jobs = []
    for unit, headers in UNITS.items():
        obj = os.path.join(OBJ, unit[:-3] + ".o")
        if force or _stale(obj, [unit], headers):
            jobs.append(job(obj, ["-c", os.path.join(CSRC, unit)]))
    if force or _stale(PEAK_SO, PEAK_SOURCES, PEAK_HEADERS):
        jobs.append(job(PEAK_SO, ["-shared", *[os.path.join(CSRC, f) for f in PEAK_SOURCES]]))
    _run(jobs, verbose)
    objs = [os.path.join(OBJ, unit[:-3] + ".o") for unit in UNITS]
    if force or not os.path.exists(SO) or any(os.path.getmtime(o) > os.path.getmtime(SO) for o in objs):
        _run([job(SO, ["-shared", *objs], None)], verbose)
    if force or _bind_stale(BIND_SO, BIND_STAMP):
        _run([(BIND_SO + tag, BIND_SO, _bind_cmd(BIND_SO + tag))], verbose)
        with open(BIND_STAMP, "w") as f:
            f.write(_bind_versions())
    return SO


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True,
          extra=["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else None)
