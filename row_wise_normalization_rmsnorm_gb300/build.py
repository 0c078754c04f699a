"""Build librmsnorm_gb300.so in-tree with nvcc for sm_103a, and the native
Python module _heads_ext.so beside it with the host compiler.

The translation units compile in parallel (one nvcc per file) into
``_build/`` and link into ``librmsnorm_gb300.so`` next to this file. The
CUDA runtime is linked statically so the library loads without a matching
libcudart on the library path; it shares the device's primary context with
any other CUDA user in the process (device pointers and streams from
PyTorch are valid in it).

Usage:  python -m row_wise_normalization_rmsnorm_gb300.build [--force]
"""
from __future__ import annotations

import concurrent.futures as cf
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "librmsnorm_gb300.so")
HEADER = os.path.join(ROOT, "include", "rmsnorm.h")
EXT = os.path.join(HERE, "_heads_ext.so")
EXT_SOURCES = [os.path.join(CSRC, f) for f in ("heads_ext.cpp", "rows_ext.cpp")]
EXT_HEADERS = [os.path.join(CSRC, "ext_args.h")]
EXT_STAMP = os.path.join(BUILD, "heads_ext.stamp")  # the Python and PyTorch that EXT was built against

SOURCES = ["api.cu", "fwd_bf16.cu", "fwd_f32.cu", "fwd_f16.cu", "fwd_bf16w32.cu", "fwd_f16w32.cu",
           "fwd8_bf16.cu", "fwd8_f16.cu", "fwd8_f32.cu", "fwd8_bf16w32.cu", "fwd8_f16w32.cu", "ln_bf16.cu", "ln_f16.cu", "ln_f32.cu", "ln_bf16w32.cu", "ln_f16w32.cu",
           "bwd_bf16.cu", "bwd_f32.cu", "bwd_f16.cu", "bwd_bf16w32.cu", "bwd_f16w32.cu",
           "fwd_peel_f32.cu", "fwd_peel_bf16.cu", "fwd_peel_f16.cu", "bwd_peel_f32.cu", "bwd_peel_bf16.cu",
           "bwd_peel_f16.cu", "noalloc.cu", "rope.cu", "paged_attn.cu",
           "groupnorm.cu", "groupnorm_f32.cu", "groupnorm_bf16.cu", "groupnorm_f16.cu",
           "ckpt8.cu", "rows_f32.cu", "rows_bf16.cu", "rows_f16.cu", "embed.cu"]
HEADERS = ["common.cuh", "plans.h", "fwd_kernels.cuh", "bwd_kernels.cuh", "head_rows.h", "tcgen05.cuh",
           "rows8.cuh", "groupnorm_kernels.cuh", "groupnorm_held.cuh", "groupnorm_flow.cuh", "rows_kernels.cuh", "embed.cuh", "train_rows.h"]

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
              "--expt-relaxed-constexpr"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build librmsnorm_gb300.so")


def _mtime(p):
    return os.path.getmtime(p) if os.path.exists(p) else 0.0


def _cuda_home() -> str:
    return os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))


def _torch_dir() -> str:
    spec = importlib.util.find_spec("torch")  # found, not imported
    if spec is None or not spec.origin:
        raise RuntimeError("PyTorch is required to build the Python module")
    return os.path.dirname(spec.origin)


def _python_include() -> str:
    return sysconfig.get_paths()["include"]


def _ext_missing() -> str | None:
    """What the Python module's build lacks here (None: nothing). The C
    library needs none of it."""
    try:
        torch = _torch_dir()
    except RuntimeError as e:
        return str(e)
    if not os.path.exists(os.path.join(torch, "include", "ATen", "core", "Tensor.h")):
        return "PyTorch's headers are missing"
    if not os.path.exists(os.path.join(_python_include(), "Python.h")):
        return "Python.h is missing"
    return None if shutil.which("g++") else "g++ is missing"


def _ext_for() -> str:
    """The Python and PyTorch that a module built now is for ("": none)."""
    try:
        torch = _torch_dir()
    except RuntimeError:
        return ""
    return "\n".join([str(sysconfig.get_config_var("SOABI")), torch, _text(os.path.join(torch, "version.py"))])


def _text(p: str) -> str:
    try:
        with open(p, encoding="utf-8") as f:
            return f.read()
    except OSError:
        return ""


def _ext_stale(force: bool) -> bool:
    deps = EXT_SOURCES + EXT_HEADERS + [HEADER, os.path.abspath(__file__)]
    return (force or not os.path.exists(EXT) or max(_mtime(p) for p in deps) > _mtime(EXT)
            or _text(EXT_STAMP) != _ext_for())


def _compile_ext(source: str) -> str:
    t = _torch_dir()
    obj = os.path.join(BUILD, os.path.splitext(os.path.basename(source))[0] + ".o")
    inc = [os.path.join(t, "include"), os.path.join(t, "include", "torch", "csrc", "api", "include"),
           os.path.join(_cuda_home(), "include"), _python_include()]
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", *(a for d in inc for a in ("-isystem", d)),
           "-c", source, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for {os.path.basename(source)}:\n{r.stdout}\n{r.stderr}")
    return obj


def _link_ext(objs: list[str]) -> None:
    """The module finds the library beside itself; PyTorch's libraries are in
    the process that imports it."""
    t = os.path.join(_torch_dir(), "lib")
    tmp = EXT + f".tmp{os.getpid()}"
    cmd = ["g++", "-shared", "-o", tmp, *objs, "-L" + HERE, "-l:" + os.path.basename(LIB), "-Wl,-rpath,$ORIGIN", "-L" + t,
           "-Wl,-rpath," + t, "-ltorch_python", "-ltorch_cuda", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link of heads_ext failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, EXT)
    with open(EXT_STAMP, "w", encoding="utf-8") as f:
        f.write(_ext_for())


def _stale(force: bool) -> bool:
    if force or not os.path.exists(LIB):
        return True
    deps = [os.path.join(CSRC, f) for f in SOURCES + HEADERS] + [HEADER, os.path.abspath(__file__)]
    return max(_mtime(p) for p in deps) > _mtime(LIB)


def _compile(src: str, extra: list[str]) -> str:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    cmd = [nvcc(), *ARCH, *NVCC_FLAGS, *extra, "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    return obj


def build(force: bool = False, verbose: bool = False, extra: list[str] | None = None) -> str:
    """Compile (if any source changed) and return the library path.

    The C library needs nvcc alone. Where the Python module cannot be built,
    the library still is, and the calls on head rows say that their module is
    not built."""
    lib_stale, ext_stale = _stale(force), _ext_stale(force)
    missing = _ext_missing() if ext_stale else None
    if missing:
        print(f"_heads_ext is not built: {missing}", file=sys.stderr)
        if os.path.exists(EXT):  # of an older source, Python or PyTorch
            os.remove(EXT)
        ext_stale = False
    if not lib_stale and not ext_stale:
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    extra = list(extra or [])
    if verbose:
        extra += ["-Xptxas", "-v"]
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + len(EXT_SOURCES)) as ex:
        ext_objs = [ex.submit(_compile_ext, s) for s in EXT_SOURCES] if ext_stale else []
        if lib_stale:
            _link(list(ex.map(lambda s: _compile(s, extra), SOURCES)))
        if ext_objs:
            _link_ext([o.result() for o in ext_objs])
    return LIB


def _link(objs: list[str]) -> None:
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc(), *ARCH, "-shared", "--cudart", "static", "-o", tmp, *objs, "-lpthread", "-ldl", "-lrt"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
