"""Build ``libpagedkv.so`` in-tree with nvcc for sm_103a.

Each CUDA translation unit under ``csrc/`` is compiled in its own process
(they are independent), then linked into one shared library next to this
file. The CUDA runtime is linked statically, so loading the library needs no
driver until the first CUDA call. ``_binding.so``, the Python module over some of
its entry points (csrc/binding.cpp), is compiled with them against this Python's
and torch's headers.
"""
import concurrent.futures
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
LIBRARY = os.path.join(HERE, "libpagedkv.so")
BINDING = os.path.join(HERE, "_binding.so")
BUILD_DIR = os.path.join(HERE, "_build")
SOURCES = ["api.cu", "api_packed.cu", "append.cu", "cache_q4.cu", "cache_q8.cu", "tables.cu", "pages.cu", "swap.cu",
           "merge.cu", "prefill.cu", "prefill_tc.cu", "decode_f32.cu", "decode_f16.cu",
           "decode_bf16.cu", "decode_q4_f16.cu", "decode_q4_bf16.cu", "decode_q8_f16.cu", "decode_q8_bf16.cu",
           "decode_noalloc.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr"]


def _nvcc():
    exe = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(exe):
        raise RuntimeError("nvcc not found; the CUDA toolkit is required to build libpagedkv")
    return exe


def _inputs():
    deps = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    deps.append(os.path.join(INCLUDE, "pagedkv.h"))
    return deps


def _stale():
    if not os.path.exists(LIBRARY) or not os.path.exists(BINDING):
        return True
    built = min(os.path.getmtime(LIBRARY), os.path.getmtime(BINDING))
    return any(os.path.getmtime(p) > built for p in _inputs())


def _binding_commands(obj):
    """The compile and link commands of the Python module."""
    import torch
    cxx = shutil.which("g++") or "g++"
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    compile_cmd = [cxx, "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
                   f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
                   "-I", os.path.join(root, "include"),
                   "-I", os.path.join(root, "include", "torch", "csrc", "api", "include"),
                   "-I", sysconfig.get_paths()["include"], "-I", os.path.join(cuda, "include"),
                   "-c", os.path.join(CSRC, "binding.cpp"), "-o", obj]
    link_cmd = [cxx, "-shared", obj, "-o", BINDING + ".tmp", "-L", HERE, "-l:libpagedkv.so",
                "-Wl,-rpath,$ORIGIN", "-L", os.path.join(root, "lib"), "-ltorch_python", "-ltorch_cpu",
                "-lc10", "-lc10_cuda"]
    return compile_cmd, link_cmd


def build(force=False, verbose=False, ptxas_info=False):
    """Compile and link; returns the library path. Skips work when up to date."""
    if not force and not _stale():
        return LIBRARY
    nvcc = _nvcc()
    os.makedirs(BUILD_DIR, exist_ok=True)
    extra = ["-Xptxas", "-v"] if ptxas_info else []

    bind_obj = os.path.join(BUILD_DIR, "binding.o")
    bind_compile, bind_link = _binding_commands(bind_obj)

    def compile_one(src):
        if src == "binding.cpp":
            res = subprocess.run(bind_compile, capture_output=True, text=True)
            return src, None, bind_compile, res
        obj = os.path.join(BUILD_DIR, os.path.splitext(src)[0] + ".o")
        cmd = [nvcc, *ARCH, *FLAGS, *extra, "-I", INCLUDE, "-c", os.path.join(CSRC, src), "-o", obj]
        res = subprocess.run(cmd, capture_output=True, text=True)
        return src, obj, cmd, res

    objs = []
    failures = []
    sources = [*SOURCES, "binding.cpp"]
    workers = min(len(sources), os.cpu_count() or 1)
    with concurrent.futures.ThreadPoolExecutor(max_workers=workers) as pool:
        for src, obj, cmd, res in pool.map(compile_one, sources):
            if verbose or ptxas_info:
                sys.stderr.write(res.stderr)
            if res.returncode != 0:
                failures.append(f"{' '.join(cmd)}\n{res.stdout}{res.stderr}")
            if obj:
                objs.append(obj)
    if failures:
        raise RuntimeError("libpagedkv build failed:\n" + "\n".join(failures))
    tmp = LIBRARY + ".tmp"
    cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("libpagedkv link failed:\n" + " ".join(cmd) + "\n" + res.stderr)
    os.replace(tmp, LIBRARY)
    res = subprocess.run(bind_link, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("binding link failed:\n" + " ".join(bind_link) + "\n" + res.stderr)
    os.replace(BINDING + ".tmp", BINDING)
    return LIBRARY


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas" in sys.argv))
