"""Build libzero (the CUDA library behind include/zero.h) in-tree for sm_103a.

    python -m zero_partitioned_mixed_flat_gb300.build [--force]

Compiles csrc/*.cu and csrc/*.cpp with nvcc in parallel and links
zero_partitioned_mixed_flat_gb300/_lib/libzero.so (CUDA runtime linked
statically, so the library loads without a GPU; device calls need one), and, where
torch is installed, the Python module _lib/_tensors.so (csrc/tensors.cc, g++)
that calls it on torch tensors.  The library does not depend on the module: where
the module's compiler, Python's headers or torch's are missing, the build says so
and leaves _lib/_tensors.error, which the calls that need the module raise.
"""
import hashlib
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT_DIR = os.path.join(PKG, "_lib")
LIB = os.path.join(OUT_DIR, "libzero.so")
TENSORS = os.path.join(OUT_DIR, "_tensors.so")
TENSORS_ERROR = os.path.join(OUT_DIR, "_tensors.error")   # why there is no module
TENSORS_SRC = os.path.join(CSRC, "tensors.cc")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", shutil.which("nvcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA 13 toolkit is required to build libzero")


COMMON = ["-std=c++17", "-O3", "-Xcompiler", "-fPIC,-ffp-contract=off,-Wall",
          "-I", INCLUDE, "-I", CSRC]
DEVICE = ARCH + ["-lineinfo", "--fmad=false", "-Xptxas", "-warn-spills"]


def _sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC)
                  if f.endswith((".cu", ".cpp")))


def _torch_dir():
    """Where torch is installed, without importing it; None: nowhere."""
    spec = importlib.util.find_spec("torch")
    return os.path.dirname(spec.origin) if spec and spec.origin else None


def _tensors_commands(torch_dir, out):
    """The compiler's and the linker's commands of the Python module."""
    obj = TENSORS + ".o"
    include = [sysconfig.get_paths()["include"], os.path.join(torch_dir, "include"),
               os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"), INCLUDE]
    compile_it = ["g++", "-std=c++17", "-O2", "-fPIC", *("-I" + d for d in include), "-c", TENSORS_SRC, "-o", obj]
    link = ["g++", "-shared", obj, "-o", out, "-L" + OUT_DIR, "-l:libzero.so", "-Wl,-rpath,$ORIGIN",
            "-L" + os.path.join(torch_dir, "lib"), "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10"]
    return compile_it, link


def _digest(files, *texts) -> str:
    h = hashlib.sha256()
    for f in files:
        h.update(f.encode())
        with open(f, "rb") as fh:
            h.update(fh.read())
    for text in texts:
        h.update(text.encode())
    return h.hexdigest()


def _fingerprint(srcs) -> str:
    headers = sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".h", ".cuh")))
    return _digest(srcs + headers + [os.path.join(INCLUDE, "zero.h"), os.path.abspath(__file__)], " ".join(COMMON + DEVICE))


def _tensors_fingerprint(torch_dir) -> str:
    return _digest([TENSORS_SRC, os.path.join(INCLUDE, "zero.h"), os.path.abspath(__file__), os.path.join(torch_dir, "version.py")],
                   sys.version)


def _stamp(target):
    return os.path.splitext(target)[0] + ".stamp"


def _current(target, fp) -> bool:
    """Whether the target was built from what fp stands for."""
    if not os.path.exists(target) or not os.path.exists(_stamp(target)):
        return False
    with open(_stamp(target)) as f:
        return f.read().strip() == fp


def _done(target, fp):
    with open(_stamp(target), "w") as f:
        f.write(fp)


def _run(cmd, what):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("%s:\n%s%s" % (what, r.stdout, r.stderr))
    return r.stdout + r.stderr


def _build_library(srcs, verbose):
    tool = nvcc()

    def compile_one(src):
        obj = os.path.join(OUT_DIR, os.path.basename(src) + ".o")
        cmd = [tool, *COMMON, "-c", src, "-o", obj]
        if src.endswith(".cu"):
            cmd[1:1] = DEVICE
        said = _run(cmd, "nvcc failed on %s" % src)
        if verbose and said:
            print(said)
        return obj

    with ThreadPoolExecutor(max_workers=len(srcs)) as ex:
        objs = list(ex.map(compile_one, srcs))
    tmp = LIB + ".tmp.%d" % os.getpid()
    _run([tool, "-shared", *ARCH, "-o", tmp, *objs, "-cudart", "static", "-lrt", "-ldl", "-lpthread"], "link failed")
    os.replace(tmp, LIB)


def build(force: bool = False, verbose: bool = False) -> str:
    srcs = _sources()
    torch_dir = _torch_dir()
    fp, tensors_fp = _fingerprint(srcs), _tensors_fingerprint(torch_dir) if torch_dir else None
    library = force or not _current(LIB, fp)
    module = torch_dir and (force or not _current(TENSORS, tensors_fp))
    if not library and not module:
        return LIB
    os.makedirs(OUT_DIR, exist_ok=True)
    with ThreadPoolExecutor(max_workers=1) as ex:
        if module:
            tmp = TENSORS + ".tmp.%d" % os.getpid()
            compile_it, link = _tensors_commands(torch_dir, tmp)
            compiled = ex.submit(_run, compile_it, "g++ failed on %s" % TENSORS_SRC)
        if library:
            _build_library(srcs, verbose)
            _done(LIB, fp)
        if module:
            try:
                compiled.result()
                _run(link, "link of _tensors.so failed")
                os.replace(tmp, TENSORS)
            except (RuntimeError, OSError) as e:   # OSError: no such compiler
                for stale in (TENSORS, _stamp(TENSORS)):    # of an earlier source: not to be loaded
                    if os.path.exists(stale):
                        os.remove(stale)
                with open(TENSORS_ERROR, "w") as f:
                    f.write(str(e))
                warnings.warn("libzero is built, its module for torch tensors is not (gated_linear, adamw_step): %s" % e,
                              RuntimeWarning, stacklevel=2)
            else:
                if os.path.exists(TENSORS_ERROR):
                    os.remove(TENSORS_ERROR)
                _done(TENSORS, tensors_fp)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
