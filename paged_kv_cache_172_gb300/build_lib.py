"""Build ``libpagedkv.so`` (the C-ABI CUDA library) in-tree for sm_103a.

Each ``csrc/*.cu`` is compiled in parallel with nvcc for
``-gencode arch=compute_103a,code=sm_103a`` and linked with a static CUDA
runtime into ``paged_kv_cache_172_gb300/libpagedkv.so``, and ``csrc/py_grouped.cpp``
with g++ into ``_grouped.so`` beside it.  Objects go to
``paged_kv_cache_172_gb300/_build/``.  Rebuilds only what changed.
"""
import glob
import hashlib
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OBJ_DIR = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libpagedkv.so")
BINDING = os.path.join(PKG, "_grouped.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "--expt-relaxed-constexpr",
              "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall", "-I", INCLUDE, "-I", CSRC]


def nvcc():
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libpagedkv")
    return path


def _headers_mtime():
    hs = glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(INCLUDE, "*.h"))
    return max(os.path.getmtime(h) for h in hs)


def _compile(src, extra, obj_dir):
    obj = os.path.join(obj_dir, os.path.basename(src) + ".o")
    if (os.path.exists(obj) and os.path.getmtime(obj) >= os.path.getmtime(src)
            and os.path.getmtime(obj) >= _headers_mtime()):
        return obj, None
    cmd = [nvcc(), *ARCH, *NVCC_FLAGS, *extra, "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        return obj, f"$ {' '.join(cmd)}\n{r.stdout}\n{r.stderr}"
    return obj, r.stderr if "warning" in r.stderr.lower() else None


def _torch_dir():
    """Where torch is installed, None where it is not."""
    spec = importlib.util.find_spec("torch")
    return None if spec is None else os.path.dirname(spec.origin)


def _compile_binding(obj_dir):
    """The Python binding of the grouped-head calls: host C++ against torch's and
    Python's headers.  Kept while its source, the headers, the command, torch and
    Python are those it was compiled with."""
    src = os.path.join(CSRC, "py_grouped.cpp")
    obj = os.path.join(obj_dir, "py_grouped.o")
    torch_dir = _torch_dir()
    tdir = os.path.join(torch_dir, "include")
    system = [tdir, os.path.join(tdir, "torch", "csrc", "api", "include"),
              sysconfig.get_paths()["include"],
              os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")]
    cmd = [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-Wall", "-I", INCLUDE,
           *(x for d in system for x in ("-isystem", d)), "-c", src, "-o", obj]
    with open(os.path.join(torch_dir, "version.py")) as f:
        made_with = "\n".join([sys.version, " ".join(cmd), f.read()])
    stamp = obj + ".made_with"
    if (os.path.exists(obj) and os.path.getmtime(obj) >= os.path.getmtime(src)
            and os.path.getmtime(obj) >= _headers_mtime() and _read(stamp) == made_with):
        return obj
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed:\n$ {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    with open(stamp, "w") as f:
        f.write(made_with)
    return obj


def _read(path):
    """A file's text, None where there is none."""
    if not os.path.exists(path):
        return None
    with open(path) as f:
        return f.read()


def _link_binding(obj, lib):
    if os.path.exists(BINDING) and os.path.getmtime(BINDING) >= max(os.path.getmtime(obj),
                                                                    os.path.getmtime(lib)):
        return
    tmp = BINDING + f".tmp{os.getpid()}"
    cmd = [shutil.which("g++") or "g++", "-shared", obj, "-o", tmp, "-L",
           os.path.join(_torch_dir(), "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10",
           "-lc10_cuda", "-L", PKG, "-l:" + os.path.basename(lib), "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n$ {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING)


def build(verbose: bool = False, extra_flags=(), out=None, sources=None) -> str:
    """Compile and link the library, then the binding of its grouped-head calls (left
    out where torch is not installed; an error of its own, with the library in place).
    ``extra_flags`` (e.g. -D tuning macros) build a variant with its own object
    directory; ``out`` names its library path; ``sources`` (file names in csrc/)
    limits a variant to those files; a variant has no binding."""
    extra_flags = tuple(extra_flags)
    product = not extra_flags and out is None and sources is None
    lib = out or LIB
    obj_dir = OBJ_DIR
    if extra_flags:
        tag = hashlib.sha256(" ".join(extra_flags).encode()).hexdigest()[:10]
        obj_dir = os.path.join(OBJ_DIR, "variant_" + tag)
    os.makedirs(obj_dir, exist_ok=True)
    if sources is None:
        srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    else:
        srcs = [os.path.join(CSRC, s) for s in sources]
    with_binding = product and _torch_dir() is not None
    if product and not with_binding:
        print("torch is not installed: the library is built without the Python binding of its "
              "grouped-head calls", file=sys.stderr)
    with ThreadPoolExecutor(max_workers=min(os.cpu_count() or 8, len(srcs) + 1)) as ex:
        binding = ex.submit(_compile_binding, obj_dir) if with_binding else None
        results = list(ex.map(lambda s: _compile(s, list(extra_flags), obj_dir), srcs))
    errors = [msg for _, msg in results if msg and "error" in msg.lower()]
    if errors:
        raise RuntimeError("nvcc failed:\n" + "\n".join(errors))
    if verbose:
        for _, msg in results:
            if msg:
                print(msg, file=sys.stderr)
    objs = [o for o, _ in results]
    if not (os.path.exists(lib)
            and all(os.path.getmtime(lib) >= os.path.getmtime(o) for o in objs)):
        tmp = lib + f".tmp{os.getpid()}"
        cmd = [nvcc(), *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n$ {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, lib)
    if binding is not None:  # the library stands whatever becomes of it
        try:
            _link_binding(binding.result(), lib)
        except RuntimeError:
            if os.path.exists(BINDING):  # of other sources
                os.remove(BINDING)
            raise
    return lib


if __name__ == "__main__":
    print(build(verbose=True, extra_flags=tuple(sys.argv[1:])))
