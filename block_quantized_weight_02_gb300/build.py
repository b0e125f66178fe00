"""Builds libcq.so (sm_103a) in-tree with nvcc: one object per .cu file,
compiled in parallel, linked with the static CUDA runtime so the library
has no link-time dependency on the driver library."""
from __future__ import annotations

import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
OUT_DIR = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libcq.so")
SOURCES = ["cq_api.cu", "k_aux.cu", "k_skinny.cu", "k_tc.cu", "k_tc_ffn.cu", "k_tc_q4a.cu", "k_tc_q8b.cu", "k_rows.cu", "cq_noalloc.cu",
           "kv8/kv8_api.cu", "kv8/kv8_store.cu", "kv8/kv8_attn.cu", "kv8/kv8_decode.cu", "kv8/kv8_tiles.cu", "kv8/kv8_narrow.cu",
           "kv8/kv8_decode_tree.cu", "kv8/kv8_tiles_tree.cu", "kv8/kv8_narrow_tree.cu", "draft/draft_api.cu", "draft/rope.cu", "draft/verify.cu"]
HEADERS = ["cq_internal.h", "cq_ptx.cuh", "k_tc.cuh", "kv8/kv8.cuh", "kv8/attn_common.cuh",
           "kv8/tiles_common.cuh", "kv8/f32x2.cuh", "kv8/store_common.cuh", "kv8/kv8_checks.h", "kv8/kv8_decode.cuh", "kv8/kv8_tiles.cuh", "kv8/kv8_narrow.cuh",
           "draft/draft.cuh"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-I", os.path.join(HERE, "..", "include")]


def nvcc() -> str:
    for c in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if c and (os.path.isabs(c) and os.path.exists(c) or not os.path.isabs(c)):
            return c
    return "nvcc"


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    os.makedirs(OUT_DIR, exist_ok=True)
    hdrs = [os.path.join(CSRC, h) for h in HEADERS] + [os.path.join(HERE, "..", "include", h) for h in ("cq.h", "cq_kv8.h", "cq_draft.h")]
    procs = []
    objs = []
    for src in SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(OUT_DIR, os.path.basename(src).replace(".cu", ".o"))
        objs.append(o)
        if force or _stale(o, [s] + hdrs):
            cmd = [nvcc(), *ARCH, *FLAGS, *extra, "-c", s, "-o", o]
            if verbose:
                print(" ".join(cmd), file=sys.stderr)
            procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
    errs = []
    for src, p in procs:
        out, _ = p.communicate()
        if p.returncode != 0:
            errs.append(f"--- {src}\n{out.decode(errors='replace')}")
        elif verbose and out:
            print(out.decode(errors="replace"), file=sys.stderr)
    if errs:
        raise RuntimeError("nvcc failed:\n" + "\n".join(errs))
    if force or procs or _stale(LIB, objs):
        tmp = LIB + f".tmp{os.getpid()}"
        cmd = [nvcc(), *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs, "-lrt", "-ldl", "-lpthread"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("link failed:\n" + r.stdout + r.stderr)
        os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    v = "-v" in sys.argv
    extra = ["-Xptxas", "-v"] if "--ptxas" in sys.argv else []
    print(build(force="-f" in sys.argv, verbose=v or bool(extra), extra=extra))
