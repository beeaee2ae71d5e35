"""Build libindexcache.so (CUDA for sm_100a) in-tree with nvcc.

Each csrc/*.cu is compiled to an object file under _build/ (in parallel) and
linked into cross_layer_top_b200/libindexcache.so with the static CUDA
runtime.  The measurement and test aids in csrc/probe/ become a separate
library, libindexcache_probe.so, linked against libindexcache.so.  The
binding's own helper, csrc/bind/tensors.cpp, becomes the Python module _tensors
(host code, g++ with torch's headers).
``python -m cross_layer_top_b200.build`` or ``build()``.
"""
import concurrent.futures
import importlib.util
import os
import re
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
OBJ = os.path.join(ROOT, "_build")
LIB = os.path.join(HERE, "libindexcache.so")
PROBE_DIR = os.path.join(CSRC, "probe")
PROBE_LIB = os.path.join(HERE, "libindexcache_probe.so")
INCLUDE = os.path.join(ROOT, "include")
BIND_SRC = os.path.join(CSRC, "bind", "tensors.cpp")
BIND_LIB = os.path.join(HERE, "_tensors" + sysconfig.get_config_var("EXT_SUFFIX"))
BIND_STAMP = os.path.join(OBJ, "_tensors.built_for")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    exe = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(exe):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libindexcache")
    return exe


def sources(folder=CSRC):
    return sorted(os.path.join(folder, f) for f in os.listdir(folder) if f.endswith(".cu"))


def headers():
    hs = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".h", ".cuh"))]
    return hs + [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE) if f.endswith(".h")]


def _obj(src: str) -> str:
    sub = "probe_" if os.path.dirname(src) == PROBE_DIR else ""
    return os.path.join(OBJ, sub + os.path.basename(src)[:-3] + ".o")


def _compile(src: str, verbose_ptxas: bool) -> str:
    obj = _obj(src)
    newest_dep = max(os.path.getmtime(p) for p in headers() + [src])
    if os.path.exists(obj) and os.path.getmtime(obj) >= newest_dep and not verbose_ptxas:
        return obj
    cmd = [nvcc()] + ARCH + FLAGS + (["-Xptxas", "-v"] if verbose_ptxas else []) + \
        ["-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("nvcc failed for %s:\n%s%s" % (src, r.stdout, r.stderr))
    if verbose_ptxas:
        sys.stderr.write(r.stderr)
    return obj


def _link(lib: str, objs, extra=()) -> None:
    deps = list(objs) + [p for p in extra if p.endswith(".so")]
    if os.path.exists(lib) and max(os.path.getmtime(o) for o in deps) <= os.path.getmtime(lib):
        return
    tmp = lib + ".tmp%d" % os.getpid()
    cmd = [nvcc()] + ARCH + ["-shared", "-cudart", "static", "-o", tmp] + list(objs)
    if extra:
        cmd += ["-L", HERE, "-lindexcache", "-Xlinker", "-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n%s%s" % (r.stdout, r.stderr))
    os.replace(tmp, lib)


def _torch_version(torch_dir: str) -> str:
    """torch.__version__, without importing torch."""
    with open(os.path.join(torch_dir, "version.py")) as f:
        return re.search(r"^__version__ *= *['\"]([^'\"]+)", f.read(), re.M).group(1)


def _build_bind() -> None:
    """The Python module _tensors.  It needs torch's libraries, which are loaded (torch imported)
    before it is, and is built anew when its sources, torch or Python's ABI change: BIND_STAMP says
    what the present one was built for, and the module itself which torch."""
    torch_dir = importlib.util.find_spec("torch").submodule_search_locations[0]
    version = _torch_version(torch_dir)
    with open(os.path.join(torch_dir, "version.py")) as f:
        stamp = "%s\n%s\n%s" % (torch_dir, os.path.basename(BIND_LIB), f.read())
    newest_dep = max(os.path.getmtime(p) for p in headers() + [BIND_SRC])
    if os.path.exists(BIND_LIB) and os.path.getmtime(BIND_LIB) >= newest_dep and os.path.exists(BIND_STAMP):
        with open(BIND_STAMP) as f:
            if f.read() == stamp:
                return
    tmp = BIND_LIB + ".tmp%d" % os.getpid()
    cmd = [shutil.which("g++") or "c++", "-O2", "-std=c++17", "-Wall", "-shared", "-fPIC", "-I", INCLUDE,
           '-DIC_TORCH_VERSION="%s"' % version,
           "-isystem", sysconfig.get_paths()["include"], "-isystem", os.path.join(torch_dir, "include"),
           "-isystem", os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
           BIND_SRC, "-o", tmp, "-L", os.path.join(torch_dir, "lib"), "-ltorch_python", "-ltorch_cpu",
           "-lc10"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("g++ failed for %s:\n%s%s" % (BIND_SRC, r.stdout, r.stderr))
    os.replace(tmp, BIND_LIB)
    with open(BIND_STAMP, "w") as f:
        f.write(stamp)


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    os.makedirs(OBJ, exist_ok=True)
    srcs = sources()
    probe_srcs = sources(PROBE_DIR)
    if force:
        for s in srcs + probe_srcs:
            if os.path.exists(_obj(s)):
                os.remove(_obj(s))
        if os.path.exists(BIND_LIB):
            os.remove(BIND_LIB)
    with concurrent.futures.ThreadPoolExecutor(max_workers=min(8, len(srcs))) as ex:
        bind = ex.submit(_build_bind)
        objs = list(ex.map(lambda s: _compile(s, verbose_ptxas), srcs + probe_srcs))
        bind.result()
    _link(LIB, objs[:len(srcs)])
    _link(PROBE_LIB, objs[len(srcs):], extra=[LIB])
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose_ptxas="-v" in sys.argv))
