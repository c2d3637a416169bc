"""Build the libraries in-tree for sm_103a (GB300).

Produces device_logits_sampling_gb300/_lib/libarcsample.so (the sampler and
the decode-loop commit) from csrc/ and libarcserve.so (the paged 8-bit cache
and the 4-bit products of the step before it) from csrc/serve/: one nvcc
process per translation unit, all at once (the six kernel sets dominate the
build), then one link each.  Runs on any host with nvcc (no GPU needed).
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIBDIR = os.path.join(PKG, "_lib")
LIB = os.path.join(LIBDIR, "libarcsample.so")
SOURCES = [os.path.join(CSRC, f) for f in ("kernels_bf16.cu", "kernels_bf16_hist.cu", "kernels_f32.cu",
                                            "kernels_f32_hist.cu", "kernels_f16.cu", "kernels_f16_hist.cu",
                                            "arc_sample.cu", "arc_decode.cu")]
SERVE_LIB = os.path.join(LIBDIR, "libarcserve.so")
SERVE_SOURCES = [os.path.join(CSRC, "serve", f) for f in ("kv_append.cu", "kv_attend.cu", "w4_matvec.cu",
                                                           "w4_many.cu",
                                                           "arc_serve.cu")]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc_path() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libarcsample.so")


def _start(sources: list[str], target: str, verbose: bool, extra: list[str] | None):
    """Start one nvcc per source; the jobs' (command, object, process)."""
    objdir = target + ".obj"
    os.makedirs(objdir, exist_ok=True)
    nvcc = nvcc_path()
    common = [*ARCH, "-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC,
              "-Xptxas", "-v" if verbose else "-O3", *(extra or [])]
    jobs = []
    for src in sources:
        obj = os.path.join(objdir, os.path.basename(src) + ".o")
        cmd = [nvcc, *common, "-c", "-o", obj, src]
        jobs.append((cmd, obj, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.PIPE, text=True)))
    return jobs


def _finish(jobs, target: str, verbose: bool) -> str:
    """Wait for the jobs and link their objects into `target`."""
    failed = None
    for cmd, _, proc in jobs:
        so, se = proc.communicate()
        if proc.returncode != 0 and failed is None:
            failed = (proc.returncode, cmd, so + se)
        elif verbose:
            sys.stderr.write(se)
    if failed is not None:
        sys.stderr.write(failed[2])
        raise RuntimeError(f"nvcc failed ({failed[0]}): {' '.join(failed[1])}")
    link = [nvcc_path(), *ARCH, "-shared", "-o", target + ".tmp", *[obj for _, obj, _ in jobs]]
    res = subprocess.run(link, capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError(f"nvcc link failed ({res.returncode}): {' '.join(link)}")
    os.replace(target + ".tmp", target)
    shutil.rmtree(target + ".obj", ignore_errors=True)
    return target


def build(verbose: bool = False, extra: list[str] | None = None, out: str | None = None) -> str:
    """Both libraries (libarcsample.so into `out` where given, and then alone)."""
    os.makedirs(LIBDIR, exist_ok=True)
    target = out or LIB
    jobs = _start(SOURCES, target, verbose, extra)
    serve = None if out else _start(SERVE_SOURCES, SERVE_LIB, verbose, extra)
    if serve is not None:
        _finish(serve, SERVE_LIB, verbose)
    return _finish(jobs, target, verbose)


def build_serve(verbose: bool = False, extra: list[str] | None = None, out: str | None = None) -> str:
    """libarcserve.so alone."""
    os.makedirs(LIBDIR, exist_ok=True)
    target = out or SERVE_LIB
    return _finish(_start(SERVE_SOURCES, target, verbose, extra), target, verbose)


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
