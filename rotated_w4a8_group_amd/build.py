"""Builds the package's HIP library ``libpq.so`` in-tree for gfx950 with hipcc, and the compiled part of the
Python binding, ``_binding.so``, against the interpreter's and torch's headers.

Usage: ``python -m rotated_w4a8_group_amd.build`` (also called by ``__graft_entry__.build``).
Every call recompiles. Objects go to ``_build/`` under the repository root.
"""
import os
import shutil
import signal
import subprocess
import sys
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT = os.path.join(PKG, "libpq.so")
BINDING = os.path.join(PKG, "_binding.so")
BUILD_DIR = os.path.join(ROOT, "_build")
ARCH = "gfx950"

# hipcc flags for every HIP translation unit. Packed fp32 instructions are disabled.
HIP_FLAGS = ["-O3", "-std=c++17", "-fPIC", f"--offload-arch={ARCH}",
             "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
             "-Wall", "-Wno-unused-result", "-Wno-unused-command-line-argument"]

SOURCES = [
    # (source, extra flags)
    ("pq_host.cpp", []),
    # the prologue's results are defined by binary32 ops that each round: no contraction
    ("pq_prologue.hip", ["-ffp-contract=off"]),
    ("pq_norms.hip", []),
    ("pq_kv.hip", []),
    ("pq_attn_decode.hip", ["-mllvm", "-amdgpu-mfma-vgpr-form"]),
    ("pq_attn_prefill.hip", ["-mllvm", "-amdgpu-mfma-vgpr-form"]),
    # matrix-core results land in VGPRs (the fold reads them there; no AGPR copies)
    ("pq_matvec.hip", ["-mllvm", "-amdgpu-mfma-vgpr-form"]),
    ("pq_glu.hip", ["-mllvm", "-amdgpu-mfma-vgpr-form"]),
    ("pq_gemm.hip", ["-mllvm", "-amdgpu-mfma-vgpr-form"]),
]


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found (ROCm is required to build the library)")


def binding_command(out: str) -> list:
    """Host code only: the device is reached through libpq.so's entry points."""
    import sysconfig

    import torch
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    dirs = [INCLUDE, inc, os.path.join(inc, "torch", "csrc", "api", "include"), sysconfig.get_paths()["include"],
            os.path.join(os.path.dirname(os.path.dirname(hipcc())), "include")]
    cmd = [os.environ.get("CXX") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", "-D__HIP_PLATFORM_AMD__=1", "-DUSE_ROCM=1"]
    for d in dirs:
        cmd += ["-isystem" if d.startswith(inc) else "-I", d]
    return cmd + [os.path.join(CSRC, "pq_binding.cpp"), "-L", os.path.join(os.path.dirname(inc), "lib"),
                  "-lc10", "-lc10_hip", "-ltorch_cpu", "-ltorch_python", "-o", out]


def _start_binding(verbose: bool):
    """(command, process, None), or (None, None, why it cannot be started)."""
    try:
        cmd = binding_command(BINDING + ".tmp")
        if verbose:
            print(" ".join(cmd), flush=True)
        return cmd, subprocess.Popen(cmd, start_new_session=True), None
    except (ImportError, OSError, RuntimeError) as e:
        return None, None, f"{type(e).__name__}: {e}"


def build(verbose: bool = False) -> str:
    """The library needs hipcc alone. Without torch, g++ or their headers there is no ``_binding.so``: a warning says why, an
    older one is taken away, and every call goes through Python and ctypes."""
    cc = hipcc()
    os.makedirs(BUILD_DIR, exist_ok=True)
    objs, jobs = [], []
    binding, why = None, None
    try:
        for src, extra in SOURCES:
            obj = os.path.join(BUILD_DIR, os.path.splitext(src)[0] + ".o")
            lang = ["-x", "hip"]
            cmd = [cc, "-c"] + lang + HIP_FLAGS + extra + ["-I", INCLUDE, "-I", CSRC,
                                                           os.path.join(CSRC, src), "-o", obj]
            if verbose:
                print(" ".join(cmd), flush=True)
            jobs.append((cmd, subprocess.Popen(cmd, start_new_session=True)))
            objs.append(obj)
        bcmd, binding, why = _start_binding(verbose)
        failed = [(job.returncode, cmd) for cmd, job in jobs if job.wait() != 0]   # waits for every one
        if failed:
            raise subprocess.CalledProcessError(*failed[0])
        tmp = OUT + ".tmp"
        cmd = [cc, "-shared", "-fPIC", f"--offload-arch={ARCH}"] + objs + ["-o", tmp]
        if verbose:
            print(" ".join(cmd), flush=True)
        subprocess.run(cmd, check=True)
        os.replace(tmp, OUT)
        if binding is not None and binding.wait() != 0:
            why = f"exit status {binding.returncode} of {' '.join(bcmd)}"
        if why is None:
            os.replace(BINDING + ".tmp", BINDING)
        else:
            if os.path.exists(BINDING):
                os.remove(BINDING)
            warnings.warn(f"_binding.so is not built, calls go through Python: {why}")
    finally:   # whatever was raised, no compiler runs on
        for _, job in jobs + [(None, binding)]:
            if job is not None and job.poll() is None:
                os.killpg(job.pid, signal.SIGKILL)   # with what it started
                job.wait()
    return OUT


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
