"""Compile the CUDA sources into the in-tree shared library ``libfa_gb300.so``,
and the native torch binding of the serving-cache conveniences (``_fa_torch.so``).

One nvcc process per translation unit, run in parallel, then one link step.
Only ``-gencode arch=compute_103a,code=sm_103a`` is emitted: the library runs
on GB300 (sm_103a) and nowhere else.  The CUDA runtime is linked statically so
the library depends on no particular libcudart being on the loader path.
"""
import concurrent.futures as cf
import os
import shutil
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
ROOT = os.path.dirname(HERE)
LIB = os.path.join(HERE, "libfa_gb300.so")
TORCH_LIB = os.path.join(HERE, "_fa_torch.so")  # the native binding of the serving-cache conveniences
BUILD = os.path.join(ROOT, "_build")
SOURCES = ["fa_api.cu", "fa_fwd.cu", "fa_fwd_fp8.cu", "fa_bwd.cu", "fa_decode.cu", "fa_decode_mma.cu",
           "fa_rope.cu", "fa_cache.cu", "fa_decode_fp8.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-I" + os.path.join(ROOT, "include")]


def nvcc():
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libfa_gb300.so")
    return cand


def _stale(srcs, out):
    if not os.path.exists(out):
        return True
    t = os.path.getmtime(out)
    return any(os.path.getmtime(s) > t for s in srcs)


TORCH_OBJ = os.path.join(BUILD, "fa_torch.o")


def _torch_stamp():
    """The file that names the torch which TORCH_LIB was compiled and linked against."""
    return os.path.join(BUILD, "fa_torch.version")


def _cxx():
    return shutil.which("g++") or "g++"


def _build_torch(run, force):
    """Compiles the native binding against the torch that is installed here, if the source, the C ABI or that torch is
    another one."""
    import sysconfig
    import torch
    src, stamp = os.path.join(CSRC, "fa_torch.cpp"), _torch_stamp()
    if not force and not _stale([src, os.path.join(ROOT, "include", "fa.h")], TORCH_OBJ):
        if os.path.exists(stamp) and open(stamp).read() == torch.__version__:
            return
    if os.path.exists(stamp):
        os.remove(stamp)  # until the binding is linked
    root = os.path.dirname(torch.__file__)
    inc = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_path("include"), os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")]
    run([_cxx(), "-O2", "-std=c++20", "-fPIC", "-fvisibility=hidden",
         "-D_GLIBCXX_USE_CXX11_ABI=%d" % int(torch._C._GLIBCXX_USE_CXX11_ABI)] + ["-isystem" + i for i in inc]
        + ["-c", src, "-o", TORCH_OBJ])


def _torch_link(out):
    import torch
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    return [_cxx(), "-shared", "-o", out, TORCH_OBJ, "-L" + libs, "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python",
            "-L" + HERE, "-l:libfa_gb300.so", "-Wl,-rpath,$ORIGIN", "-Wl,-rpath," + libs]


def build(force=False, verbose=False, ptxas_info=False):
    """Build libfa_gb300.so and the native binding if any source or header is newer; return the library's path."""
    os.makedirs(BUILD, exist_ok=True)
    headers = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    headers.append(os.path.join(ROOT, "include", "fa.h"))
    cc = nvcc()
    objs, jobs = [], []
    for src in SOURCES:
        path = os.path.join(CSRC, src)
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        objs.append(obj)
        if force or _stale([path] + headers, obj):
            cmd = [cc] + ARCH + FLAGS + (["-Xptxas", "-v"] if ptxas_info else []) + ["-c", path, "-o", obj]
            jobs.append(cmd)
    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed:\n%s\n%s%s" % (" ".join(cmd), r.stdout, r.stderr))
        return r.stdout + r.stderr
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        binding = ex.submit(_build_torch, run, force)
        for out in ex.map(run, jobs):
            if verbose and out.strip():
                print(out)
        binding.result()
    if force or jobs or _stale(objs, LIB):
        tmp = LIB + ".tmp%d" % os.getpid()
        run([cc] + ARCH + ["-shared", "-cudart", "static", "-o", tmp] + objs)
        os.replace(tmp, LIB)
    if force or not os.path.exists(_torch_stamp()) or _stale([TORCH_OBJ], TORCH_LIB):
        import torch
        tmp = TORCH_LIB + ".tmp%d" % os.getpid()
        run(_torch_link(tmp))
        os.replace(tmp, TORCH_LIB)
        with open(_torch_stamp(), "w") as f:
            f.write(torch.__version__)
    return LIB


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose=True, ptxas_info="-v" in sys.argv))
