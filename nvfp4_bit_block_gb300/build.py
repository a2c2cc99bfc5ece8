"""Build the CUDA libraries in-tree with plain nvcc (one -gencode, sm_103a):

* nvfp4_bit_block_gb300/_build/libnvfp4.so -- the quantizer and its GEMM (the
  C ABI of include/nvfp4.h and its kernels);
* nvfp4_bit_block_gb300/_build/libnvfp4_layer.so -- the operators around the
  linear layer (the C ABI of include/nvfp4_layer.h and its kernels), a library
  of its own because the quantizer's arithmetic is compiled without fused
  multiply-adds and theirs with them; _build/_nvfp4_layer.so is its Python
  binding (a CPython extension against torch's C++ interface);
* tests/selftest/_build/libnvfp4_selftest.so and libnvfp4_layer_selftest.so --
  device self-checks used only by the tests (build_selftest,
  build_layer_selftest); they hold no product entry point.

Translation units compile in parallel; the CUDA runtime is linked statically.
"""
from __future__ import annotations

import os
import subprocess
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(BUILD, "libnvfp4.so")
LAYER_BUILD = os.path.join(BUILD, "layer")
LAYER_LIB = os.path.join(BUILD, "libnvfp4_layer.so")
LAYER_EXT = os.path.join(BUILD, "_nvfp4_layer.so")
INCLUDE = os.path.join(ROOT, "include")
SELFTEST_DIR = os.path.join(ROOT, "tests", "selftest")
SELFTEST_BUILD = os.path.join(SELFTEST_DIR, "_build")
SELFTEST_LIB = os.path.join(SELFTEST_BUILD, "libnvfp4_selftest.so")
LAYER_SELFTEST_LIB = os.path.join(SELFTEST_BUILD, "libnvfp4_layer_selftest.so")

SOURCES = ["api.cu", "tmap.cu", "amax.cu", "quant1d.cu", "quant1d_sr.cu", "quant1d_46mae.cu", "quant1d_46mse.cu", "quant1d_46max.cu",
           "quant2d.cu", "dequant.cu", "analysis.cu", "gemm.cu"]
LAYER_SOURCES = ["layer_api.cu", "layernorm.cu", "layernorm_backward.cu", "act_backward.cu", "linear.cu", "linear_split.cu", "linear_many.cu", "out_tmap.cu",
                 "tmap.cu"]
NVCC_FLAGS = [
    "-gencode", "arch=compute_103a,code=sm_103a",
    "-O3", "-lineinfo", "-std=c++17",
    "-fmad=false", "-ftz=false", "-prec-div=true", "-prec-sqrt=true",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
    "--expt-relaxed-constexpr",
]
LAYER_NVCC_FLAGS = ["-fmad=true" if f == "-fmad=false" else f for f in NVCC_FLAGS]


def _nvcc() -> str:
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    cand = os.path.join(cuda, "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _headers():
    hs = [os.path.join(CSRC, h) for h in os.listdir(CSRC) if h.endswith((".cuh", ".h"))]
    hs += [os.path.join(INCLUDE, h) for h in ("nvfp4.h", "nvfp4_layer.h")]
    return hs


def _run(cmd, verbose=False):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    if verbose:
        print(r.stdout, r.stderr)


def _build_lib(sources, build_dir, lib, force, verbose, flags=NVCC_FLAGS):
    """Compile `sources` (absolute paths) to objects in build_dir and link `lib`."""
    os.makedirs(build_dir, exist_ok=True)
    headers = _headers()
    nvcc = _nvcc()
    objs, jobs = [], []
    for s in sources:
        o = os.path.join(build_dir, os.path.basename(s).replace(".cu", ".o"))
        objs.append(o)
        if force or _stale(o, [s] + headers):
            jobs.append([nvcc, *flags, "-I", INCLUDE, "-I", CSRC, "-c", s, "-o", o])
    if jobs:
        with ThreadPoolExecutor(max_workers=min(len(jobs), os.cpu_count() or 4)) as ex:
            list(ex.map(lambda c: _run(c, verbose), jobs))
    if force or jobs or _stale(lib, objs):
        tmp = lib + f".tmp{os.getpid()}"
        _run([nvcc, "-shared", "-gencode", "arch=compute_103a,code=sm_103a", "-cudart", "static", "-o", tmp, *objs],
             verbose)
        os.replace(tmp, lib)
    return lib


EXT_STAMP = os.path.join(LAYER_BUILD, "layer_binding.txt")


def _ext_tag() -> str:
    """What the binding's object and its library paths depend on beside the sources."""
    import sys

    import torch
    return f"python {sys.version}\ntorch {torch.__version__} {torch.__file__}\n"


def _ext_stale() -> bool:
    """Whether the binding was built against another Python or torch (or never)."""
    if not os.path.exists(EXT_STAMP):
        return True
    with open(EXT_STAMP) as f:
        return f.read() != _ext_tag()


def _build_ext(force: bool, verbose: bool) -> tuple:
    """Compile the layer's binding; returns (object, whether it is new)."""
    import sysconfig

    from torch.utils.cpp_extension import include_paths
    os.makedirs(LAYER_BUILD, exist_ok=True)
    src, o = os.path.join(CSRC, "layer_binding.cpp"), os.path.join(LAYER_BUILD, "layer_binding.o")
    stale = force or _ext_stale() or _stale(o, [src] + [h for h in _headers() if h.startswith(INCLUDE)])
    if stale:
        cuda = os.path.dirname(os.path.dirname(_nvcc()))
        inc = [*include_paths(), sysconfig.get_paths()["include"], os.path.join(cuda, "include"), INCLUDE]
        _run([os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-w",
              *[x for i in inc for x in ("-I", i)], "-c", src, "-o", o], verbose)
    return o, stale


def _link_ext(o: str, force: bool, verbose: bool) -> None:
    from torch.utils.cpp_extension import library_paths
    if not force and not _stale(LAYER_EXT, [o]):
        return
    libs = library_paths()
    tmp = LAYER_EXT + f".tmp{os.getpid()}"
    # the library by its name, not its path: the binding loads the one beside it ($ORIGIN), wherever the tree is
    _run([os.environ.get("CXX", "g++"), "-shared", "-o", tmp, o, *[f"-L{p}" for p in [BUILD, *libs]],
          "-l:" + os.path.basename(LAYER_LIB), *[f"-Wl,-rpath,{p}" for p in ["$ORIGIN", *libs]], "-lc10", "-lc10_cuda",
          "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python"], verbose)
    os.replace(tmp, LAYER_EXT)
    with open(EXT_STAMP, "w") as f:
        f.write(_ext_tag())


def build(force: bool = False, verbose: bool = False) -> str:
    """The product libraries and the layer's binding, side by side; returns the path of libnvfp4.so."""
    with ThreadPoolExecutor(max_workers=3) as ex:
        ext = ex.submit(_build_ext, force, verbose)
        main = ex.submit(_build_lib, [os.path.join(CSRC, s) for s in SOURCES], BUILD, LIB, force, verbose)
        layer = ex.submit(_build_lib, [os.path.join(CSRC, s) for s in LAYER_SOURCES], LAYER_BUILD, LAYER_LIB, force,
                          verbose, LAYER_NVCC_FLAGS)
        layer.result()
        o, fresh = ext.result()
        _link_ext(o, fresh, verbose)
        return main.result()


def build_layer_selftest(force: bool = False, verbose: bool = False) -> str:
    """The test-only build of nvfp4_linear whose copies are never issued; returns its path."""
    srcs = [os.path.join(SELFTEST_DIR, "nvfp4_layer_selftest.cu")]
    srcs += [os.path.join(CSRC, s) for s in ("linear.cu", "linear_split.cu", "linear_many.cu", "out_tmap.cu", "tmap.cu")]
    return _build_lib(srcs, os.path.join(SELFTEST_BUILD, "layer"), LAYER_SELFTEST_LIB, force, verbose,
                      [*LAYER_NVCC_FLAGS, "-DNVFP4_TEST_NO_COPIES"])


def build_selftest(force: bool = False, verbose: bool = False) -> str:
    """The test-only self-check library (its own copy of the tensor-map
    helper); returns its path."""
    srcs = [os.path.join(SELFTEST_DIR, "nvfp4_selftest.cu"), os.path.join(CSRC, "tmap.cu")]
    return _build_lib(srcs, SELFTEST_BUILD, SELFTEST_LIB, force, verbose)


if __name__ == "__main__":
    print(build(verbose=True))
    print(build_selftest(verbose=True))
    print(build_layer_selftest(verbose=True))
