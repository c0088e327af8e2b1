"""Builds libpath_attn.so in-tree for sm_103a with nvcc.

Each .cu translation unit compiles in its own nvcc process (in parallel), then
one nvcc link step produces the shared library in
dependent_position_encoded_gb300/_build/. The CUDA runtime is linked
statically, so the library needs only the driver at run time.
"""
import concurrent.futures
import os
import shutil
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT_DIR = os.path.join(HERE, "_build")
LIB = os.path.join(OUT_DIR, "libpath_attn.so")

SOURCES = ["path_api.cu", "ut_prepare.cu", "ut_prepare_tc.cu", "pair_combine.cu",
           "fox_exit.cu", "scan_tc.cu", "scan_tc_fox.cu", "scan_tc128.cu", "scan_f32.cu", "decode.cu", "producer.cu", "backward.cu", "backward_tc.cu",
           "backward_block_mm.cu", "backward_d128.cu", "backward_tc128.cu",
           "fwd_d128.cu", "paged_api.cu", "paged_decode.cu", "paged_f32.cu", "paged_pages.cu",
           "paged_prep_tc.cu", "paged_prep_more_tc.cu", "paged_attn_tc.cu", "paged_attn_more_tc.cu",
           "paged_window_tc.cu", "paged_single_tc.cu", "paged_prefix_tc.cu", "paged_prefix_f32.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC]


def nvcc():
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libpath_attn.so")
    return path


def _inputs():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files.append(os.path.join(INCLUDE, "path_attn.h"))
    return files


def up_to_date():
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(f) <= t for f in _inputs())


def build(force=False, verbose=False, extra_flags=()):
    """Compiles every kernel for sm_103a and links libpath_attn.so; returns its path."""
    if not force and up_to_date():
        return LIB
    os.makedirs(OUT_DIR, exist_ok=True)
    cc = nvcc()

    def compile_one(src):
        obj = os.path.join(OUT_DIR, os.path.splitext(src)[0] + ".o")
        cmd = [cc, *ARCH, *FLAGS, *extra_flags, "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed on %s:\n%s%s" % (src, r.stdout, r.stderr))
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr)
        return obj

    with concurrent.futures.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(compile_one, SOURCES))
    tmp = LIB + ".tmp.%d" % os.getpid()
    cmd = [cc, *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("nvcc link failed:\n%s%s" % (r.stdout, r.stderr))
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    import sys
    print(build(force=True, verbose="-v" in sys.argv,
                extra_flags=("-Xptxas", "-v") if "-v" in sys.argv else ()))
