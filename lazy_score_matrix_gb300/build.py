"""Build libtp.so in-tree: every csrc/*.cu and csrc_logits/*.cu compiled for sm_103a in parallel, then linked; and
_tp_logits.so, the PyTorch binding of include/tp_logits.h (csrc_logits/tp_logits_torch.cpp), against it.

Usage: ``python -m lazy_score_matrix_gb300.build`` (or ``__graft_entry__.build()``).
Objects go to ``lazy_score_matrix_gb300/_build/``; the library to ``lazy_score_matrix_gb300/libtp.so``.
A translation unit is recompiled when it or any header in csrc/, csrc_logits/ or include/ is newer than its object; the
binding also when its object was made for another PyTorch or Python.

csrc/ holds the consumers of lazy scores (include/tp.h), csrc_logits/ those of stored score rows
(include/tp_logits.h). They are apart because the recorded traffic and instruction counts of the lazy
consumers' benchmark are keyed to a hash of csrc/ and tp.h (bench.py, source_hash).
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
CSRC_LOGITS = os.path.join(PKG, "csrc_logits")
INCLUDE = os.path.join(ROOT, "include")
OBJ_DIR = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libtp.so")
BINDING_SRC = os.path.join(CSRC_LOGITS, "tp_logits_torch.cpp")
BINDING = os.path.join(PKG, "_tp_logits.so")
# calibration library of the benchmark (measured fp32 / fp64 FMA and exp2 rates), not part of libtp
PEAKS_SRC = os.path.join(PKG, "peaks", "tp_peaks.cu")
PEAKS_LIB = os.path.join(PKG, "libtp_peaks.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-std=c++17", "-O3", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
              "-I" + INCLUDE, "-I" + CSRC, "-I" + CSRC_LOGITS]


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA 13 toolkit is required to build libtp")


def _headers_mtime() -> float:
    hs = [h for d in (CSRC, CSRC_LOGITS, INCLUDE) for h in glob.glob(os.path.join(d, "*.h")) + glob.glob(os.path.join(d, "*.cuh"))]
    return max(os.path.getmtime(h) for h in hs)


def _compile(src: str, extra: list[str]) -> tuple[str, int, str]:
    obj = os.path.join(OBJ_DIR, os.path.basename(src)[:-3] + ".o")
    cmd = [nvcc(), *ARCH, *NVCC_FLAGS, *extra, "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    return obj, r.returncode, (r.stdout + r.stderr)


def _torch_dirs() -> tuple[list[str], str]:
    """PyTorch's include directories (with Python's and CUDA's) and its library directory, without importing it."""
    import importlib.util
    import sysconfig
    torch = os.path.dirname(importlib.util.find_spec("torch").origin)
    inc = os.path.join(torch, "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")
    return [inc, os.path.join(inc, "torch", "csrc", "api", "include"), sysconfig.get_paths()["include"], cuda], os.path.join(torch, "lib")


def _binding_key() -> str:
    """What the binding was compiled against: an object for another PyTorch or Python is not reused."""
    import importlib.util
    spec = os.path.dirname(importlib.util.find_spec("torch").origin)
    return f"{sys.version}\n{spec}\n{open(os.path.join(spec, 'version.py')).read()}"


def _binding_due() -> bool:
    obj, key = os.path.join(OBJ_DIR, "tp_logits_torch.o"), os.path.join(OBJ_DIR, "tp_logits_torch.key")
    if not os.path.exists(obj) or not os.path.exists(key) or open(key).read() != _binding_key():
        return True
    return os.path.getmtime(obj) < max(os.path.getmtime(f) for f in [BINDING_SRC, *glob.glob(os.path.join(INCLUDE, "*.h"))])


def _compile_binding() -> tuple[str, int, str]:
    obj = os.path.join(OBJ_DIR, "tp_logits_torch.o")
    incs, _ = _torch_dirs()
    cmd = ["g++", "-std=c++17", "-O2", "-fPIC", "-fvisibility=hidden", "-DTORCH_API_INCLUDE_EXTENSION_H",
           "-I" + INCLUDE, *[a for d in incs for a in ("-isystem", d)], "-c", BINDING_SRC, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode == 0:
        with open(os.path.join(OBJ_DIR, "tp_logits_torch.key"), "w") as f:
            f.write(_binding_key())
    return obj, r.returncode, (r.stdout + r.stderr)


def _link_binding() -> None:
    tmp = BINDING + f".tmp{os.getpid()}"
    lib = _torch_dirs()[1]
    r = subprocess.run(["g++", "-shared", "-o", tmp, os.path.join(OBJ_DIR, "tp_logits_torch.o"), "-L" + PKG, "-l:libtp.so",
                        "-Wl,-rpath,$ORIGIN", "-L" + lib, "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10_cuda", "-lc10"], capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError("_tp_logits link failed")
    os.replace(tmp, BINDING)


def build(force: bool = False, jobs: int | None = None, verbose: bool = False, extra: list[str] | None = None) -> str:
    os.makedirs(OBJ_DIR, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu"))) + sorted(glob.glob(os.path.join(CSRC_LOGITS, "*.cu")))
    hdr = _headers_mtime()
    todo = []
    for s in srcs:
        obj = os.path.join(OBJ_DIR, os.path.basename(s)[:-3] + ".o")
        if force or not os.path.exists(obj) or os.path.getmtime(obj) < max(os.path.getmtime(s), hdr):
            todo.append(s)
    bound = os.path.join(OBJ_DIR, "tp_logits_torch.o")
    bind = force or _binding_due()
    jobs = jobs or max(1, min(len(todo) + bind or 1, os.cpu_count() or 4))
    errors = []
    if todo or bind:
        with cf.ThreadPoolExecutor(jobs) as ex:
            work = ([_compile_binding] if bind else []) + [lambda s=s: _compile(s, extra or []) for s in todo]
            for obj, rc, out in ex.map(lambda f: f(), work):
                if rc != 0:
                    errors.append((obj, out))
                elif verbose and out.strip():
                    print(out)
    if errors:
        for obj, out in errors:
            sys.stderr.write(f"--- {os.path.basename(obj)} ---\n{out[-4000:]}\n")
        raise RuntimeError(f"libtp build failed in {len(errors)} translation unit(s)")
    if force or not os.path.exists(PEAKS_LIB) or os.path.getmtime(PEAKS_LIB) < os.path.getmtime(PEAKS_SRC):
        tmp = PEAKS_LIB + f".tmp{os.getpid()}"
        r = subprocess.run([nvcc(), *ARCH, "-O3", "-Xcompiler", "-fPIC", "-shared", "-o", tmp, PEAKS_SRC],
                           capture_output=True, text=True)
        if r.returncode != 0:
            sys.stderr.write(r.stdout + r.stderr)
            raise RuntimeError("libtp_peaks build failed")
        os.replace(tmp, PEAKS_LIB)
    objs = [os.path.join(OBJ_DIR, os.path.basename(s)[:-3] + ".o") for s in srcs]
    if todo or not os.path.exists(LIB) or os.path.getmtime(LIB) < max(os.path.getmtime(o) for o in objs):
        tmp = LIB + f".tmp{os.getpid()}"
        r = subprocess.run([nvcc(), *ARCH, "-shared", "-o", tmp, *objs], capture_output=True, text=True)
        if r.returncode != 0:
            sys.stderr.write(r.stdout + r.stderr)
            raise RuntimeError("libtp link failed")
        os.replace(tmp, LIB)
    if bind or not os.path.exists(BINDING) or os.path.getmtime(BINDING) < os.path.getmtime(bound):
        _link_binding()
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
