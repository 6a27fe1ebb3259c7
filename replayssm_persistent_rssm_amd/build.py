"""Build librssm_materialize.so (the operation) and librssm_pool.so (the
contiguous-pool placement helper, a separate library so that the operation's
library exports nothing that allocates) for gfx950 with hipcc, and the
binding's marshalling extension with the host compiler, in-tree, no JIT.  The
extension is left out where torch is not installed: the libraries are plain C ABI
and need neither torch nor the binding.

Each state dtype's kernel instances live in their own translation unit and
compile in parallel; the host launcher is one more.  Flags: -O3, C++17,
packed-fp32 instructions disabled (plain fp32 VALU code only), correctly
rounded fp32 division and square root (hipcc's default, never relaxed: the
one-byte encode divides).
"""
from __future__ import annotations

import concurrent.futures
import os
import re
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB_PATH = os.path.join(PKG, "librssm_materialize.so")
POOL_LIB_PATH = os.path.join(PKG, "librssm_pool.so")
BUILD_DIR = os.path.join(PKG, "_build")

SOURCES = ["rssm_inst_f32.hip", "rssm_inst_bf16.hip", "rssm_inst_f16.hip", "rssm_inst_i8.hip",
           "rssm_inst_f8.hip", "rssm_inst_gdn.hip", "rssm_inst_ssu.hip", "rssm_materialize.hip",
           "rssm_inst_linattn_f32.hip", "rssm_inst_linattn_bf16.hip", "rssm_inst_linattn_f16.hip",
           "rssm_inst_paged_f32.hip", "rssm_inst_paged_bf16.hip", "rssm_inst_paged_f16.hip",
           "rssm_inst_norm_f32.hip", "rssm_inst_norm_bf16.hip", "rssm_inst_norm_f16.hip",
           "rssm_inst_scan_f32.hip", "rssm_inst_scan_bf16.hip", "rssm_inst_scan_f16.hip",
           "rssm_linear_attention.hip", "rssm_paged_attention.hip", "rssm_block_norm.hip", "rssm_causal_conv.hip",
           "rssm_selective_scan.hip", "rssm_rotary.hip", "rssm_pages.hip"]
POOL_SOURCES = ["rssm_pool.hip"]
# Kernels that hold their states in registers: the build fails where the compiler spills one of them to scratch.
NO_SCRATCH = ["rssm_inst_scan_f32.hip", "rssm_inst_scan_bf16.hip", "rssm_inst_scan_f16.hip"]
# the binding's marshalling extension (host code against torch's headers)
FAST_SOURCE = "fast_calls.cpp"
FAST_PATH = os.path.join(PKG, "_fast_calls.so")
ARCH = os.environ.get("RSSM_OFFLOAD_ARCH", "gfx950")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

CFLAGS = ["--offload-arch=" + ARCH, "-O3", "-std=c++17", "-fPIC", "-Wall",
          "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
          "-I" + INCLUDE, "-I" + CSRC]


def _compile(src: str, verbose: bool) -> str:
    obj = os.path.join(BUILD_DIR, os.path.splitext(src)[0] + ".o")
    report = ["-Rpass-analysis=kernel-resource-usage"] if src in NO_SCRATCH else []
    cmd = [HIPCC] + CFLAGS + report + ["-c", os.path.join(CSRC, src), "-o", obj]
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    # hipcc's host pass does not know the device feature flag: drop that warning only
    noise = [ln for ln in res.stderr.splitlines() if "packed-fp32-ops" not in ln and ln.strip()]
    if res.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n" + "\n".join(noise))
    if report:
        _check_scratch(src, res.stderr)
        noise = [ln for ln in noise if "warning" in ln]
    if noise and verbose:
        print("\n".join(noise), file=sys.stderr)
    return obj


def _check_scratch(src: str, report: str) -> None:
    """Raise where the compiler's resource report of `src` has a kernel with scratch memory, or no kernel."""
    kernels = re.findall(r"Function Name: (\S+)|ScratchSize \[bytes/lane\]: (\d+)", report)
    names, sizes = [n for n, _ in kernels if n], [int(s) for _, s in kernels if s]
    if not names or len(names) != len(sizes):
        raise RuntimeError(f"no resource report of the kernels in {src}")
    spilled = [f"{n} ({s} bytes a lane)" for n, s in zip(names, sizes) if s > 0]
    if spilled:
        raise RuntimeError(f"kernels of {src} use scratch memory: " + ", ".join(spilled))


def _link(objs, path: str, verbose: bool) -> None:
    tmp = path + ".tmp"
    cmd = [HIPCC, "--offload-arch=" + ARCH, "-shared", "-fPIC", "-Wl,-soname," + os.path.basename(path), "-o", tmp] + objs
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link of {os.path.basename(path)} failed:\n" + res.stderr)
    os.replace(tmp, path)


def _cxx() -> str:
    """Host compiler: $CXX, g++, or the compiler that comes with hipcc."""
    return os.environ.get("CXX") or shutil.which("g++") or os.path.join(os.path.dirname(HIPCC), "amdclang++")


def _build_fast(verbose: bool) -> bool:
    """The marshalling extension, linked to the operation library beside it; False without torch, whose
    tensors are all it handles."""
    import sysconfig
    try:
        import torch
    except ImportError:
        print(f"torch is not installed: {os.path.basename(FAST_PATH)}, the torch binding's extension, is left out",
              file=sys.stderr)
        return False
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = FAST_PATH + ".tmp"
    cmd = [_cxx(), "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           "-D_GLIBCXX_USE_CXX11_ABI=%d" % int(torch._C._GLIBCXX_USE_CXX11_ABI), "-I" + INCLUDE,
           "-I" + sysconfig.get_paths()["include"], "-I" + inc,
           "-I" + os.path.join(inc, "torch", "csrc", "api", "include"), os.path.join(CSRC, FAST_SOURCE), "-o", tmp,
           "-L" + lib, "-ltorch_python", "-ltorch_cpu", "-lc10", LIB_PATH, "-Wl,-rpath,$ORIGIN"]
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"build of {os.path.basename(FAST_PATH)} failed:\n" + res.stderr)
    os.replace(tmp, FAST_PATH)
    return True


def build(verbose: bool = False, jobs: int = 8) -> str:
    """Compile and link both libraries and the binding's extension; returns the operation library's path."""
    os.makedirs(BUILD_DIR, exist_ok=True)
    srcs = SOURCES + POOL_SOURCES
    with concurrent.futures.ThreadPoolExecutor(max_workers=min(jobs, len(srcs))) as ex:
        objs = list(ex.map(lambda s: _compile(s, verbose), srcs))
    _link(objs[:len(SOURCES)], LIB_PATH, verbose)
    _link(objs[len(SOURCES):], POOL_LIB_PATH, verbose)
    _build_fast(verbose)
    return LIB_PATH


if __name__ == "__main__":
    print(build(verbose=True))
