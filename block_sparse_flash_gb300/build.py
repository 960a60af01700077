"""Builds libsplash.so in-tree (block_sparse_flash_gb300/_build/) with nvcc for
sm_103a, and the compiled part of the Python binding with g++.  Translation
units are compiled in parallel and linked into one shared library; nothing is
installed outside the repository."""
import contextlib
import os
import subprocess
import sys
import sysconfig
import warnings
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT_DIR = os.path.join(HERE, "_build")
LIB = os.path.join(OUT_DIR, "libsplash.so")
# (source, object, defines): attention_fwd.cu is compiled once per pattern
# mode and paged_decode.cu once per cache type, so that their kernel
# instantiations build in parallel
SOURCES = [("api.cu", "api", []), ("mask_info.cu", "mask_info", []),
           ("attention_fwd.cu", "attention_fwd", ["-DSPLASH_FWD_PM=0"]),
           ("attention_fwd.cu", "attention_fwd_band", ["-DSPLASH_FWD_PM=1"]),
           ("attention_fwd.cu", "attention_fwd_band_seg", ["-DSPLASH_FWD_PM=2"]),
           ("attention_bwd.cu", "attention_bwd", []), ("host_pipeline.cu", "host_pipeline", []),
           ("rope.cu", "rope", []), ("paged_decode.cu", "paged_decode_bf16", ["-DSPLASH_DECODE_E4M3=0"]),
           ("paged_decode.cu", "paged_decode_e4m3", ["-DSPLASH_DECODE_E4M3=1"])]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
# the compiled part of the Python binding, for this Python and this torch
BINDING_SOURCE = "binding.cpp"


def binding_path() -> str:
    import torch
    return os.path.join(OUT_DIR, f"_binding.{sysconfig.get_config_var('SOABI')}.torch-{torch.__version__}.so")


FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC]


def _nvcc():
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _stale(output, sources):
    """Whether output is older than one of its sources, the interface or this file."""
    files = [os.path.join(CSRC, f) for f in sources] + [os.path.join(INCLUDE, "splash.h"), os.path.abspath(__file__)]
    return not os.path.exists(output) or os.path.getmtime(output) < max(os.path.getmtime(f) for f in files)


def _torch_root():
    import torch
    return os.path.dirname(torch.__file__)


def _run(cmd, what):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what}:\n{r.stdout}\n{r.stderr}")


def _compile_binding() -> str:
    import torch
    root, obj = _torch_root(), os.path.join(OUT_DIR, "binding.o")
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    _run(["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
          f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", INCLUDE,
          "-I", os.path.join(root, "include"), "-I", os.path.join(root, "include", "torch", "csrc", "api", "include"),
          "-I", sysconfig.get_paths()["include"], "-I", os.path.join(cuda, "include"),
          "-c", os.path.join(CSRC, BINDING_SOURCE), "-o", obj], f"g++ failed for {BINDING_SOURCE}")
    return obj


def _link_binding(obj: str, path: str) -> None:
    libs, tmp = os.path.join(_torch_root(), "lib"), path + f".tmp{os.getpid()}"
    _run(["g++", "-shared", "-o", tmp, obj, "-L", OUT_DIR, "-lsplash", "-L", libs, "-ltorch_python", "-ltorch",
          "-ltorch_cpu", "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{libs}"], "link of the binding failed")
    os.replace(tmp, path)


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    """Compiles what is stale and returns the path of libsplash.so.

    The library needs nvcc and its host compiler.  The binding also needs the
    headers of Python and torch: where it cannot be built, that is a warning,
    and only the serving calls are missing (they raise SplashLibraryMissing)."""
    os.makedirs(OUT_DIR, exist_ok=True)
    with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        binding = ex.submit(_binding_object, force)  # (while nvcc compiles)
        if force or _stale(LIB, [f for f in os.listdir(CSRC) if f != BINDING_SOURCE]):
            _build_library(ex, verbose, extra)
    try:
        path, obj = binding.result()
        if obj is not None:
            _link_binding(obj, path)
    except Exception as e:
        warnings.warn(f"the serving calls are not available: {e}", RuntimeWarning, stacklevel=2)
    return LIB


def _binding_object(force):
    """(path of the binding, its new object or None where it is up to date)."""
    path = binding_path()
    if not force and not _stale(path, [BINDING_SOURCE]):
        return path, None
    with contextlib.suppress(FileNotFoundError):
        os.remove(path)  # (not left behind if it no longer builds)
    return path, _compile_binding()


def _build_library(ex, verbose, extra):
    nvcc = _nvcc()

    def compile_one(entry):
        src, name, defines = entry
        obj = os.path.join(OUT_DIR, name + ".o")
        cmd = [nvcc, *ARCH, *FLAGS, *defines, *extra, "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr, file=sys.stderr)
        return obj

    objs = list(ex.map(compile_one, SOURCES))
    tmp = LIB + f".tmp{os.getpid()}"
    _run([nvcc, *ARCH, "-shared", "-o", tmp, *objs], "link failed")
    os.replace(tmp, LIB)


if __name__ == "__main__":
    v = "-v" in sys.argv
    print(build(force="--force" in sys.argv, verbose=v, extra=["-Xptxas", "-v"] if v else []))
