"""Build libnq.so (the CUDA library behind include/nq.h) in-tree for sm_103a.

Each translation unit is compiled by its own nvcc process, in parallel, then
linked into e8_lattice_vector_gb300/_build/libnq.so.  No cmake, no torch
extension machinery: the library is plain C ABI over the CUDA runtime.
"""
import concurrent.futures as cf
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
CSRC_PAGED = os.path.join(HERE, "csrc_paged")
OUT_DIR = os.path.join(HERE, "_build")
LIB = os.path.join(OUT_DIR, "libnq.so")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")

SOURCES = ["nq_api.cu", "nq_compress.cu", "nq_compress_delta.cu", "nq_decompress.cu", "nq_decompress_delta.cu", "nq_roundtrip.cu", "nq_stats.cu", "nq_layers.cu", "nq_noalloc.cu"]
# the paged-cache operators, in a folder of their own: the codec's traffic record names a hash of csrc
PAGED_SOURCES = ["nq_page_map.cu", "nq_paged_append.cu", "nq_paged_attention.cu", "nq_paged_small.cu",
                 "nq_paged_chunk.cu"]


def _headers(folder):
    return [os.path.join(folder, f) for f in sorted(os.listdir(folder)) if f.endswith((".cuh", ".h"))]


ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + [
    "-O3", "-lineinfo", "-std=c++17", "--fmad=false", "-Xcompiler", "-fPIC",
    "-Xcompiler", "-ffp-contract=off", "-I", INCLUDE,
]


def _nvcc():
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _stale(target, deps):
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    os.makedirs(OUT_DIR, exist_ok=True)
    nvcc = _nvcc()
    common_deps = _headers(CSRC) + _headers(CSRC_PAGED) + [os.path.join(INCLUDE, "nq.h"), __file__]
    sources = [os.path.join(CSRC, f) for f in SOURCES] + [os.path.join(CSRC_PAGED, f) for f in PAGED_SOURCES]
    objs, jobs = [], []
    for s in sources:
        o = os.path.join(OUT_DIR, os.path.basename(s).replace(".cu", ".o"))
        objs.append(o)
        if force or _stale(o, [s] + common_deps):
            cmd = [nvcc] + NVCC_FLAGS + (["-Xptxas", "-v"] if verbose_ptxas else []) + ["-c", s, "-o", o]
            jobs.append(cmd)
    if jobs:
        with cf.ThreadPoolExecutor(max_workers=len(jobs)) as ex:
            results = list(ex.map(lambda c: subprocess.run(c, capture_output=True, text=True), jobs))
        for cmd, r in zip(jobs, results):
            if verbose_ptxas or r.returncode != 0:
                sys.stderr.write(r.stdout + r.stderr)
            if r.returncode != 0:
                raise RuntimeError("nvcc failed: " + " ".join(cmd))
    if force or jobs or _stale(LIB, objs):
        tmp = LIB + ".tmp.%d" % os.getpid()
        subprocess.run([nvcc] + ARCH + ["-shared", "-o", tmp] + objs, check=True)
        os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose_ptxas="-v" in sys.argv))
