"""Build ``libew.so`` (the C ABI of include/ew.h) in-tree with nvcc for sm_103a,
and beside it the row operators' torch binding.

The translation units are compiled in parallel, then linked into
``memory_bound_elementwise_gb300/_lib/libew.so`` with the CUDA runtime linked
statically.  Floating-point flags keep IEEE behaviour: no flush-to-zero, no
contraction of separate multiplies and adds, IEEE division and square root
(the kernels spell out their rounding in PTX anyway).
"""
import concurrent.futures as cf
import hashlib
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT_DIR = os.path.join(PKG, "_lib")
LIB = os.path.join(OUT_DIR, "libew.so")
OBJ_DIR = os.path.join(OUT_DIR, "obj")
BINDING_SOURCE = os.path.join(CSRC, "ew_torch.cpp")
BINDING = os.path.join(OUT_DIR, "_ew_torch.so")  # CPython extension over torch's C++ headers

SOURCES = ["ew_api.cu", "ew_kernels_f32.cu", "ew_kernels_f16.cu", "ew_kernels_bf16.cu", "ew_tma.cu",
           "ew_gather_fixed.cu", "ew_gather_fixed_wide.cu", "ew_rows_api.cu", "ew_rows.cu", "ew_embed.cu",
           "ew_norm_f32.cu", "ew_norm_f16.cu", "ew_norm_bf16.cu",
           "ew_logits_f32.cu", "ew_logits_f16.cu", "ew_logits_bf16.cu",
           "ew_distill_f32.cu", "ew_distill_f16.cu", "ew_distill_bf16.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC,-fvisibility=hidden",
              "-ftz=false", "-prec-div=true", "-prec-sqrt=true", "-fmad=false",
              "-I", INCLUDE, "-I", CSRC]


def nvcc():
    exe = shutil.which("nvcc")
    if exe:
        return exe
    cand = "/usr/local/cuda/bin/nvcc"
    if os.path.exists(cand):
        return cand
    raise RuntimeError("nvcc not found")


ROW_OPERATORS = ("ew_rows", "ew_embed", "ew_norm", "ew_logits", "ew_distill")  # what their sources' names begin with


def _kernel_digest(skip=()):
    """SHA-256 over the CUDA sources (kernels and dispatch) but for those whose
    names begin with one of `skip`, and the compiler flags, independent of where
    the repository sits on disk."""
    h = hashlib.sha256()
    files = [os.path.join(CSRC, name) for name in sorted(os.listdir(CSRC))
             if name.endswith((".cu", ".cuh", ".h")) and not name.startswith(skip)]
    for path in files:
        h.update(os.path.relpath(path, ROOT).encode())
        with open(path, "rb") as f:
            h.update(f.read())
    flags = [f for f in ARCH + NVCC_FLAGS if f not in (INCLUDE, CSRC)]
    h.update(" ".join(flags).encode())
    return h.hexdigest()


def source_digest():
    """SHA-256 over the sources and flags of the elementwise kernels: what the
    profiler's figures that bench.py reports were taken on."""
    return _kernel_digest(ROW_OPERATORS)


def _torch_dir():
    """The installed torch's folder, found without importing it; None where there is none."""
    try:
        spec = importlib.util.find_spec("torch")
    except (ImportError, ValueError):
        spec = None
    return list(spec.submodule_search_locations)[0] if spec is not None and spec.submodule_search_locations else None


def _digest_of(start, paths):
    h = hashlib.sha256(start.encode())
    for path in paths:
        with open(path, "rb") as f:
            h.update(f.read())
    return h.hexdigest()


def _inputs_digest():
    """Build stamp of the library: the kernel sources and flags, and the public header."""
    return _digest_of(_kernel_digest(), [os.path.join(INCLUDE, "ew.h")])


def _binding_digest(torch_dir):
    """Build stamp of the binding: its source, the header, and what it is built for."""
    return _digest_of(sys.version, [os.path.join(INCLUDE, "ew.h"), BINDING_SOURCE, os.path.join(torch_dir, "version.py")])


def _build_binding(torch_dir):
    """Compiles the torch binding; it is linked against libew.so and the installed torch."""
    include, lib = os.path.join(torch_dir, "include"), os.path.join(torch_dir, "lib")
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    cuda_include = [d for d in [os.path.join(cuda, "include")] +
                    [os.path.join(cuda, "targets", t, "include") for t in ("x86_64-linux", "sbsa-linux")]
                    if os.path.exists(os.path.join(d, "cuda_runtime_api.h"))][:1]
    obj = os.path.join(OBJ_DIR, "ew_torch.o")
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-I", INCLUDE, "-isystem", include, "-isystem",
           os.path.join(include, "torch", "csrc", "api", "include"), "-isystem", sysconfig.get_paths()["include"],
           "-D_GLIBCXX_USE_CXX11_ABI=1", "-c", BINDING_SOURCE, "-o", obj]
    for d in cuda_include:
        cmd += ["-isystem", d]
    r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    if r.returncode != 0:
        raise RuntimeError("g++ failed for ew_torch.cpp:\n%s" % r.stdout)
    return obj, lib


def _link_binding(obj, torch_lib):
    tmp = BINDING + ".tmp.%d" % os.getpid()
    # by name: the library has no soname, and by path its place would be written down
    cmd = ["g++", "-shared", "-o", tmp, obj, "-L", OUT_DIR, "-l:" + os.path.basename(LIB), "-L", torch_lib, "-lc10",
           "-lc10_cuda", "-ltorch_cpu", "-ltorch_python", "-Wl,-rpath,$ORIGIN", "-Wl,-rpath," + torch_lib]
    r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    if r.returncode != 0:
        raise RuntimeError("link of the torch binding failed:\n%s" % r.stdout)
    os.replace(tmp, BINDING)


def _up_to_date(product, stamp, digest):
    return os.path.exists(product) and os.path.exists(stamp) and open(stamp).read().strip() == digest


def _write(path, text):
    with open(path, "w") as f:
        f.write(text)


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Compile and link libew.so and the torch binding unless up-to-date builds exist.

    The library needs nvcc alone.  Without torch there is no binding."""
    stamp, binding_stamp = os.path.join(OUT_DIR, "build.sha256"), os.path.join(OUT_DIR, "binding.sha256")
    digest = _inputs_digest() + ("|" + " ".join(extra_flags) if extra_flags else "")
    torch_dir = _torch_dir()
    with_lib = force or not _up_to_date(LIB, stamp, digest)
    with_binding = torch_dir is not None and (force or not _up_to_date(BINDING, binding_stamp, _binding_digest(torch_dir)))
    if torch_dir is None:
        sys.stderr.write("torch not found: the row operators' torch binding is not built\n")
    if not with_lib and not with_binding:
        return LIB
    os.makedirs(OBJ_DIR, exist_ok=True)
    exe = nvcc() if with_lib else None

    def compile_one(src):
        obj = os.path.join(OBJ_DIR, src.replace(".cu", ".o"))
        cmd = [exe, *ARCH, *NVCC_FLAGS, *extra_flags, "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed for %s:\n%s" % (src, r.stdout))
        return obj, r.stdout

    with cf.ThreadPoolExecutor(max_workers=min(len(SOURCES) + 1, os.cpu_count() or 4)) as ex:
        binding = ex.submit(_build_binding, torch_dir) if with_binding else None  # the longest: first
        if with_lib:
            results = list(ex.map(compile_one, SOURCES))
            if verbose:
                for _, log in results:
                    sys.stdout.write(log)
            tmp = LIB + ".tmp.%d" % os.getpid()
            cmd = [exe, *ARCH, "-shared", "-o", tmp, *[o for o, _ in results], "-cudart", "static"]
            r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
            if r.returncode != 0:
                raise RuntimeError("link failed:\n%s" % r.stdout)
            os.replace(tmp, LIB)
            _write(stamp, digest)
        if with_binding:
            _link_binding(*binding.result())
            _write(binding_stamp, _binding_digest(torch_dir))
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
