"""In-tree build of libqsa.so (nvcc, sm_103a only)."""
from __future__ import annotations

import glob
import os
import subprocess
import tempfile

_HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(_HERE, "csrc")
LIB_PATH = os.path.join(_HERE, "libqsa.so")
INCLUDE = os.path.join(os.path.dirname(_HERE), "include")

NVCC_FLAGS = [
    "-O3", "-std=c++17", "-gencode", "arch=compute_103a,code=sm_103a", "-lineinfo",
    "-Xptxas", "-v", "-Xcompiler", "-fPIC", "-I", INCLUDE,
]


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + [os.path.join(INCLUDE, "qsa.h")]


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile every .cu under csrc/ into libqsa.so next to this file, then
    the CPython entry points of the per-step calls (build_fastcall); beside
    both the checks of their tensors (build_tensors)."""
    tensors = _start_tensors(force)
    _build_lib(force, verbose)
    build_fastcall(force)
    _finish_tensors(tensors)
    return LIB_PATH


def _build_lib(force: bool, verbose: bool) -> str:
    newest = max(os.path.getmtime(p) for p in _deps())
    if not force and os.path.exists(LIB_PATH) and os.path.getmtime(LIB_PATH) >= newest:
        return LIB_PATH
    nvcc = os.environ.get("NVCC", "nvcc")
    if not os.path.exists(nvcc) and os.path.exists("/usr/local/cuda/bin/nvcc"):
        nvcc = "/usr/local/cuda/bin/nvcc"
    tmp = LIB_PATH + f".{os.getpid()}.tmp"
    with tempfile.TemporaryDirectory() as obj_dir:
        # one object per source, compiled side by side, then linked
        objs, runs = [], []
        for src in _sources():
            objs.append(os.path.join(obj_dir, os.path.basename(src) + ".o"))
            runs.append(subprocess.Popen([nvcc, *NVCC_FLAGS, "-c", "-o", objs[-1], src], stdout=subprocess.PIPE,
                                         stderr=subprocess.PIPE, text=True))
        said = [r.communicate() for r in runs]
        for r, (out, err) in zip(runs, said):
            if r.returncode != 0:
                raise RuntimeError(f"nvcc failed ({r.returncode}):\n{out}\n{err}")
        r = subprocess.run([nvcc, "-shared", "-o", tmp, *objs], capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed ({r.returncode}):\n{r.stdout}\n{r.stderr}")
    if verbose:
        print("\n".join(err for _, err in said))
    os.replace(tmp, LIB_PATH)
    return LIB_PATH


FASTCALL_SRC = os.path.join(_HERE, "_fastcall.c")


def fastcall_path() -> str:
    import sysconfig
    return os.path.join(_HERE, "_fastcall" + (sysconfig.get_config_var("EXT_SUFFIX") or ".so"))


def build_fastcall(force: bool = False) -> str | None:
    """Compile the CPython entry points of the per-step calls (_fastcall.c)
    against libqsa.so; None where the Python headers or a C compiler are
    missing (the ctypes path is used then)."""
    import shutil
    import sysconfig
    out = fastcall_path()
    inc = sysconfig.get_paths().get("include", "")
    cc = os.environ.get("CC", "gcc")
    if not inc or not os.path.exists(os.path.join(inc, "Python.h")) or shutil.which(cc) is None:
        return None
    deps = [FASTCALL_SRC, os.path.join(INCLUDE, "qsa.h"), LIB_PATH]
    if not force and os.path.exists(out) and os.path.getmtime(out) >= max(os.path.getmtime(p) for p in deps):
        return out
    tmp = out + f".{os.getpid()}.tmp"
    cmd = [cc, "-O2", "-shared", "-fPIC", "-I", inc, "-I", INCLUDE, FASTCALL_SRC, "-o", tmp, "-L", _HERE,
           "-l:libqsa.so", "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        return None
    os.replace(tmp, out)
    return out


TENSORS_SRC = os.path.join(_HERE, "_tensors.cpp")


def tensors_path() -> str:
    import sysconfig
    return os.path.join(_HERE, "_tensors" + (sysconfig.get_config_var("EXT_SUFFIX") or ".so"))


def _tensors_stamp() -> str:
    """The file that says for which torch tensors_path() was built.  The
    extension has torch's tensor layout compiled in, and another torch's files
    may be older than it."""
    return tensors_path() + ".torch"


def _torch_version(torch_dir: str) -> str | None:
    """The version that torch.__version__ gives, without importing torch."""
    import re
    try:
        with open(os.path.join(torch_dir, "version.py")) as f:
            m = re.search(r"^__version__\s*=\s*['\"]([^'\"]+)['\"]", f.read(), re.M)
    except OSError:
        return None
    return m.group(1) if m else None


def _read(path: str) -> str | None:
    try:
        with open(path) as f:
            return f.read()
    except OSError:
        return None


def _start_tensors(force: bool):
    """Starts the compiler on _tensors.cpp: (process, its output), or None
    where there is nothing to do or no way (the Python form is used then)."""
    import importlib.util
    import shutil
    import sysconfig
    out = tensors_path()
    inc = sysconfig.get_paths().get("include", "")
    cxx = os.environ.get("CXX", "g++")
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.submodule_search_locations or shutil.which(cxx) is None:
        return None
    torch_dir = spec.submodule_search_locations[0]
    headers = os.path.join(torch_dir, "include")
    if not inc or not os.path.exists(os.path.join(inc, "Python.h")) or not os.path.isdir(headers):
        return None
    version = _torch_version(torch_dir)
    if version is None:
        return None
    if (not force and os.path.exists(out) and os.path.getmtime(out) >= os.path.getmtime(TENSORS_SRC)
            and _read(_tensors_stamp()) == version):
        return None
    tmp = out + f".{os.getpid()}.tmp"
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    cmd = [cxx, "-O2", "-std=c++17", "-shared", "-fPIC", f'-DQSA_TORCH_VERSION="{version}"', "-I", inc, "-isystem", headers, "-isystem",
           os.path.join(headers, "torch", "csrc", "api", "include"), "-isystem", os.path.join(cuda, "include"),
           TENSORS_SRC, "-o", tmp, "-L", os.path.join(torch_dir, "lib"), "-lc10", "-ltorch_cpu", "-ltorch_python"]
    return subprocess.Popen(cmd, stdout=subprocess.DEVNULL, stderr=subprocess.PIPE, text=True), tmp, version


def _finish_tensors(started) -> str | None:
    if started is None:
        return None
    run, tmp, version = started
    run.communicate()
    if run.returncode != 0:
        return None
    os.replace(tmp, tensors_path())
    with open(tmp, "w") as f:
        f.write(version)
    os.replace(tmp, _tensors_stamp())
    return tensors_path()


def build_tensors(force: bool = False) -> str | None:
    """Compile the checks of a call's tensors (_tensors.cpp) against the
    installed torch; None where its headers or a compiler are missing."""
    return _finish_tensors(_start_tensors(force))
