"""Build the CUDA library libw4a8.so (sm_103a) in-tree, under _build/.

Each .cu under csrc/ is compiled by its own nvcc process (in parallel) and
the objects are linked into one shared library with the CUDA runtime linked
statically, so loading it needs no CUDA shared libraries.  Beside it comes
_w4a8.so, the Python entry points of binding.cpp, which links the library and
the torch of this interpreter.  The library needs neither Python nor torch and is
built whatever becomes of the module; where that does not build, the calls that
need it say why.  Rebuilds only when a source or header is newer than what was
built, and the module also for another torch.
"""
import contextlib
import glob
import json
import os
import subprocess
import sys
import sysconfig
import tempfile
import warnings
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
OUT_DIR = os.path.join(HERE, "_build")
LIB = os.path.join(OUT_DIR, "libw4a8.so")
EXT = os.path.join(OUT_DIR, "_w4a8.so")
STAMP = os.path.join(OUT_DIR, "_w4a8.json")      # the torch that the module was built for, and why it was not
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-ftz=false", "-prec-div=true", "-prec-sqrt=true", "-I", os.path.join(ROOT, "include")]


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return (_sources() + glob.glob(os.path.join(CSRC, "*.cpp")) + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))
            + glob.glob(os.path.join(ROOT, "include", "*.h")) + [__file__])


def _compile(src, extra):
    obj = os.path.join(OUT_DIR, os.path.basename(src) + ".o")
    cmd = [NVCC, *ARCH, *FLAGS, *extra, "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
    return obj, r.stderr


def _link(results, verbose):
    if verbose:
        for _, log in results:
            print(log)
    fd, tmp = tempfile.mkstemp(suffix=".so", dir=OUT_DIR)
    os.close(fd)
    cmd = [NVCC, *ARCH, "-shared", "-cudart", "static", "-Xlinker", "-soname=libw4a8.so", "-o", tmp, *[o for o, _ in results]]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)


def _compile_binding():
    import torch
    top = os.path.join(os.path.dirname(torch.__file__), "include")
    obj = os.path.join(OUT_DIR, "binding.cpp.o")
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I", os.path.join(ROOT, "include"), "-isystem", top, "-isystem", os.path.join(top, "torch", "csrc", "api", "include"),
           "-isystem", sysconfig.get_paths()["include"], "-isystem", os.path.join(os.path.dirname(os.path.dirname(NVCC)), "include"),
           "-c", os.path.join(CSRC, "binding.cpp"), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on binding.cpp:\n{r.stdout}\n{r.stderr}")
    return obj


def _link_binding(obj):
    import torch
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    fd, tmp = tempfile.mkstemp(suffix=".so", dir=OUT_DIR)
    os.close(fd)
    cmd = ["g++", "-shared", "-o", tmp, obj, "-L", OUT_DIR, "-lw4a8", "-L", libs, "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda",
           "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{libs}"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, EXT)


def _torch_id():
    """What the module is bound to beside its sources."""
    try:
        import torch
    except ImportError:
        return "none"
    return f"{torch.__version__} in {os.path.dirname(torch.__file__)}, {sys.implementation.cache_tag}, C++11 ABI {int(torch._C._GLIBCXX_USE_CXX11_ABI)}"


def _stamp():
    try:
        with open(STAMP) as f:
            return json.load(f)
    except (OSError, ValueError):
        return {}


def binding_error():
    """Why the last build made no module ("" where it did)."""
    return _stamp().get("error", "")


def _built(path):
    return os.path.exists(path) and os.path.getmtime(path) >= max(os.path.getmtime(p) for p in _deps())


def _finish_binding(compiled):
    """Links the module from what its compilation (a future) gave, and notes how that went."""
    error = ""
    try:
        _link_binding(compiled.result())
    except Exception as e:                       # whatever it is, the library is there
        error = str(e) or repr(e)
        with contextlib.suppress(FileNotFoundError):     # of older sources, or of another torch
            os.remove(EXT)
        warnings.warn("the Python module of prompt attention and the 8-bit cache was not built: " + error)
    fd, tmp = tempfile.mkstemp(suffix=".json", dir=OUT_DIR)
    with os.fdopen(fd, "w") as f:
        json.dump({"torch": _torch_id(), "error": error}, f)
    os.replace(tmp, STAMP)


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Compile csrc/*.cu for sm_103a and link _build/libw4a8.so (and _w4a8.so); returns the library's path."""
    os.makedirs(OUT_DIR, exist_ok=True)
    stamp = _stamp()
    have_lib = not force and _built(LIB)
    have_ext = not force and _built(STAMP) and stamp.get("torch") == _torch_id() and (stamp.get("error") or _built(EXT))
    if have_lib and have_ext:
        return LIB
    extra = list(extra_flags) + (["-Xptxas", "-v"] if verbose else [])
    with ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        binding = None if have_ext else ex.submit(_compile_binding)
        if not have_lib:
            _link(list(ex.map(lambda s: _compile(s, extra), _sources())), verbose)
    if binding:
        _finish_binding(binding)
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose="-v" in sys.argv))
