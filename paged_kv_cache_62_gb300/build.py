"""Build ``libpkv.so`` (the CUDA library behind include/pkv.h) in-tree with nvcc.

Every translation unit is compiled for sm_103a only, in parallel, then linked
into one shared library next to this file.  The CUDA runtime is linked
statically, so the library needs nothing beyond the NVIDIA driver at run time.
``_pkv_torch.so``, the native argument checks of the int8 and rotary bindings,
is compiled beside it against the installed torch.  Where that fails (no torch
or Python headers, say), the library and the other bindings are built all the
same; the int8 and rotary bindings then raise.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
ROOT = os.path.dirname(HERE)
BUILD_DIR = os.path.join(ROOT, "_build")
LIB_PATH = os.path.join(HERE, "libpkv.so")
TORCH_PATH = os.path.join(HERE, "_pkv_torch.so")
TORCH_OBJ, TORCH_KEY = os.path.join(BUILD_DIR, "pkv_torch.o"), os.path.join(BUILD_DIR, "pkv_torch.key")
SOURCES = ["pkv_api.cu", "pkv_store.cu", "pkv_decode.cu", "pkv_decode_fp8.cu", "pkv_decode_qs.cu", "pkv_decode_wide.cu",
           "pkv_decode_tc5.cu", "pkv_decode_i8.cu", "pkv_decode_i8_wide.cu", "pkv_decode_i8_tc5.cu", "pkv_store_i8.cu",
           "pkv_rope.cu", "pkv_noalloc.cu", "pkv_alloc.cpp"]
HEADERS = ["pkv_device.cuh", "pkv_host.h", "pkv_decode_kernel.cuh", "pkv_i8_tile.cuh", "pkv_i8_codes.cuh",
           "pkv_i8_tc5.cuh"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
# Hidden visibility: only the PKV_API (extern "C") entry points are exported, so
# internal statics never merge with those of another copy of the library.
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
         "--expt-relaxed-constexpr", "-Xcompiler", "-Wall"]


def nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libpkv.so")
    return cand


def _stale(target: str, deps: list[str]) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def torch_commands(tmp: str) -> tuple[list[str], list[str]]:
    """Compile and link commands of _pkv_torch.so (found at run time: torch's own libraries, already loaded, and
    libpkv.so beside it)."""
    import torch
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    inc = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    compile_ = ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-Wall",
                f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
                f'-DPKV_TORCH_VERSION="{torch.__version__}"',
                *(x for i in inc for x in ("-isystem", i)), "-c", os.path.join(CSRC, "pkv_torch.cpp"), "-o", TORCH_OBJ]
    libs = os.path.join(root, "lib")
    link = ["g++", "-shared", "-o", tmp, TORCH_OBJ, "-L", HERE, "-lpkv", "-L", libs, "-ltorch_python", "-ltorch_cpu",
            "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{libs}"]
    return compile_, link


def torch_key() -> str:
    """What _pkv_torch.so is bound to besides its sources: the installed torch and the Python ABI."""
    import torch
    return f"{torch.__version__} {sysconfig.get_config_var('SOABI')}"


def _torch_part(lib_built: "cf.Future", force: bool) -> str | None:
    """Build _pkv_torch.so if it is missing, stale or bound to another torch or Python; the library's link is waited
    for before its own.  Returns why it could not be built (it is then not there, not an old one), or None."""
    tmp = TORCH_PATH + f".tmp{os.getpid()}"
    try:
        key = torch_key()
        other = not os.path.exists(TORCH_KEY) or open(TORCH_KEY).read() != key
        deps = [os.path.join(CSRC, "pkv_torch.cpp"), os.path.join(ROOT, "include", "pkv.h")]
        if force or other or _stale(TORCH_OBJ, deps):
            _run(torch_commands(tmp)[0])
        lib_built.result()
        if force or other or _stale(TORCH_PATH, [TORCH_OBJ, LIB_PATH]):
            _run(torch_commands(tmp)[1])
            os.replace(tmp, TORCH_PATH)
            with open(TORCH_KEY, "w") as f:
                f.write(key)
        return None
    except (RuntimeError, OSError, ImportError) as e:
        if not lib_built.done() or lib_built.exception() is None:
            for path in (TORCH_PATH, TORCH_OBJ):
                if os.path.exists(path):
                    os.remove(path)
        return str(e) or type(e).__name__


def _run(cmd: list[str], echo: bool = False) -> None:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if echo or r.returncode:
        sys.stderr.write(r.stdout + r.stderr)
    if r.returncode:
        raise RuntimeError("failed: " + " ".join(cmd))


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    os.makedirs(BUILD_DIR, exist_ok=True)
    include = os.path.join(ROOT, "include")
    hdrs = [os.path.join(CSRC, h) for h in HEADERS] + [os.path.join(include, "pkv.h")]
    objs, jobs = [], []
    for src in SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(BUILD_DIR, os.path.splitext(src)[0] + ".o")
        objs.append(o)
        if force or ptxas_info or _stale(o, [s] + hdrs):
            cmd = [nvcc(), *ARCH, *FLAGS, "-I", include, "-c", s, "-o", o]
            if ptxas_info:
                cmd.insert(1, "-Xptxas=-v")
            jobs.append(cmd)

    lib_built = cf.Future()
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        torch_part = ex.submit(_torch_part, lib_built, force)
        try:
            for _ in ex.map(lambda cmd: _run(cmd, verbose or ptxas_info), jobs):
                pass
            if force or jobs or _stale(LIB_PATH, objs):
                tmp = LIB_PATH + f".tmp{os.getpid()}"
                _run([nvcc(), *ARCH, "-shared", "-o", tmp, *objs, "-cudart", "static"])
                os.replace(tmp, LIB_PATH)
            lib_built.set_result(None)
        except BaseException as e:
            lib_built.set_exception(RuntimeError("the library was not built"))
            raise e
    if (why := torch_part.result()) is not None:
        sys.stderr.write(f"_pkv_torch.so was not built, the int8 and rotary bindings are not available: {why}\n")
    return LIB_PATH


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas-info" in sys.argv)
    print(LIB_PATH)
