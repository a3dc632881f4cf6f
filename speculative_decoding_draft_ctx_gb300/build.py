"""In-tree build of libdspark_ctx_kv.so for sm_103a (no cmake, no torch
extension machinery): the kernel TU is compiled by nvcc and the host TU by
g++ in parallel, then linked by nvcc against the static CUDA runtime."""

from __future__ import annotations

import os
import shutil
import subprocess
import sys
import threading
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(PKG, "_build")
LIB_NAME = "libdspark_ctx_kv.so"
LIB_PATH = os.path.join(PKG, LIB_NAME)

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
KERNEL_SRC = os.path.join(CSRC, "ctx_kv_kernel.cu")
TMA_SRC = os.path.join(CSRC, "ctx_kv_tma.cu")
QK_SRC = os.path.join(CSRC, "qk_insert_kernel.cu")
PROJ_SRC = os.path.join(CSRC, "proj_gemm.cu")
NORM_SRC = os.path.join(CSRC, "hidden_norm.cu")
GENERAL_SRC = os.path.join(CSRC, "ctx_kv_general.cu")
WARP_SRC = os.path.join(CSRC, "ctx_kv_warp.cu")
NOALLOC_SRC = os.path.join(CSRC, "ctx_kv_noalloc.cu")
ROPE_SRC = os.path.join(CSRC, "rope.cu")
EVICT_SRC = os.path.join(CSRC, "kv_evict.cu")
ATTN_SRCS = tuple(os.path.join(CSRC, f) for f in ("tree_attn.cu", "attn_weight.cu", "tree_attn_d64.cu", "tree_attn_d128.cu", "tree_attn_d256.cu",
                                                     "tree_attn_tc_d64.cu", "tree_attn_tc_d128.cu", "tree_attn_scaled_d64.cu",
                                                     "tree_attn_scaled_d128.cu", "tree_attn_scaled_d256.cu",
                                                     "tree_attn_tc_scaled_d64.cu", "tree_attn_tc_scaled_d128.cu"))
STEP_SRCS = tuple(os.path.join(CSRC, f) for f in ("verify.cu", "kv_pages.cu", "kv_insert_scaled.cu"))
CU_SRCS = (KERNEL_SRC, TMA_SRC, QK_SRC, PROJ_SRC, NORM_SRC, GENERAL_SRC, WARP_SRC, NOALLOC_SRC, ROPE_SRC, EVICT_SRC,
           *ATTN_SRCS, *STEP_SRCS)
API_SRC = os.path.join(CSRC, "ctx_kv_api.cpp")
DRAFT_API_SRC = os.path.join(CSRC, "draft_attn_api.cpp")
STEP_API_SRC = os.path.join(CSRC, "draft_step_api.cpp")
API_SRCS = (API_SRC, DRAFT_API_SRC, STEP_API_SRC)
HEADERS = [os.path.join(CSRC, "ctx_kv_internal.h"), os.path.join(CSRC, "ctx_kv_device.cuh"),
           os.path.join(CSRC, "ctx_kv_pipe.cuh"), os.path.join(CSRC, "draft_attn_internal.h"),
           os.path.join(CSRC, "tree_attn_mma.cuh"), os.path.join(CSRC, "tree_attn_split.cuh"),
           os.path.join(CSRC, "tree_attn_tc.cuh"),
           os.path.join(CSRC, "tc_ptx.cuh"), os.path.join(CSRC, "attn_weight.cuh"),
           os.path.join(CSRC, "draft_api_checks.h"), os.path.join(CSRC, "draft_step_internal.h"),
           os.path.join(CSRC, "page_scale.cuh"), os.path.join(INCLUDE, "dspark_ctx_kv.h"),
           os.path.join(INCLUDE, "dspark_draft_attn.h"), os.path.join(INCLUDE, "dspark_draft_step.h")]

_lock = threading.Lock()


def cuda_home() -> str:
    home = os.environ.get("CUDA_HOME") or os.environ.get("CUDA_PATH")
    if home:
        return home
    nvcc = shutil.which("nvcc")
    if nvcc:
        return os.path.dirname(os.path.dirname(os.path.realpath(nvcc)))
    return "/usr/local/cuda"


def _stale() -> bool:
    if not os.path.exists(LIB_PATH):
        return True
    t = os.path.getmtime(LIB_PATH)
    return any(os.path.getmtime(s) > t for s in [*CU_SRCS, *API_SRCS, *HEADERS])


def _run(cmd):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"build step failed ({' '.join(cmd)}):\n{r.stdout}\n{r.stderr}")
    return r.stdout + r.stderr


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile the library if a source is newer than it; returns its path."""
    with _lock:
        if not force and not _stale():
            return LIB_PATH
        os.makedirs(BUILD_DIR, exist_ok=True)
        home = cuda_home()
        nvcc = os.path.join(home, "bin", "nvcc")
        objs, cmds = [], []
        for src in CU_SRCS:
            obj = os.path.join(BUILD_DIR, os.path.basename(src)[:-3] + ".o")
            cmd = [nvcc, *ARCH, "-lineinfo", "-O3", "-std=c++17", "-Xcompiler", "-fPIC",
                   "-I", INCLUDE, "-c", src, "-o", obj]
            if verbose:
                cmd.insert(1, "-Xptxas=-v")
            objs.append(obj)
            cmds.append(cmd)
        for src in API_SRCS:
            aobj = os.path.join(BUILD_DIR, os.path.basename(src)[:-4] + ".o")
            cmds.append(["g++", "-O2", "-std=c++17", "-fPIC", "-Wall", "-I", os.path.join(home, "include"),
                         "-I", INCLUDE, "-c", src, "-o", aobj])
            objs.append(aobj)
        with ThreadPoolExecutor(len(cmds)) as ex:
            outs = list(ex.map(_run, cmds))
        if verbose:
            sys.stderr.write("".join(outs[:len(CU_SRCS)]))
        tmp = LIB_PATH + f".tmp{os.getpid()}"
        _run([nvcc, *ARCH, "-shared", "-o", tmp, *objs, "-lpthread", "-ldl", "-lrt"])
        os.replace(tmp, LIB_PATH)
        return LIB_PATH


if __name__ == "__main__":
    build(force=True, verbose="-v" in sys.argv)
    print(LIB_PATH)
