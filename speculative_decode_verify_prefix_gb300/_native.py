"""Build and load the in-tree CUDA library (libverify_splitkv.so, sm_103a).

The library is compiled from ``csrc/*.cu`` with nvcc into ``_build/`` next to
this file: every translation unit (the host side, and the kernels of each
head_dim) in parallel, then linked into one shared library.  ``csrc/views.cpp``
becomes the extension module that packs the views of a call's tensors.  Loading the
library never falls back to anything: if it is missing or fails to load, callers get
an exception.  The module only saves host time: where it cannot be built (no Python
headers), build() warns and the calls pack their views in Python.
"""
from __future__ import annotations

import ctypes
import os
import platform
import subprocess
import sysconfig
import threading
import warnings

_HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(_HERE, "csrc")
SRCS = sorted(os.path.join(CSRC, n) for n in os.listdir(CSRC) if n.endswith(".cu"))
HEADER = os.path.join(os.path.dirname(_HERE), "include", "verify_splitkv.h")
BUILD_DIR = os.path.join(_HERE, "_build")
OBJ_DIR = os.path.join(BUILD_DIR, f"obj_{platform.machine()}")
LIB_PATH = os.path.join(BUILD_DIR, f"libverify_splitkv_{platform.machine()}.so")
VIEWS_SRC = os.path.join(CSRC, "views.cpp")
VIEWS_PATH = os.path.join(BUILD_DIR, "vsk_views" + sysconfig.get_config_var("EXT_SUFFIX"))  # (names the Python and the machine)
NVCC_ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = [*NVCC_ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC"]


def nvcc_path() -> str:
    for cand in (os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc"), "nvcc"):
        if os.path.sep not in cand or os.path.exists(cand):
            return cand
    return "nvcc"


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile the CUDA library for sm_103a (no-op when up to date): each
    translation unit in parallel, then one link.  ``verbose`` passes
    ``-Xptxas=-v`` (registers, spills, shared memory per kernel)."""
    from concurrent.futures import ThreadPoolExecutor

    os.makedirs(OBJ_DIR, exist_ok=True)
    with ThreadPoolExecutor(1) as ex:
        views = ex.submit(_build_views, force)
        path = _build_lib(force, verbose)
        try:
            views.result()
        except (RuntimeError, OSError) as e:
            warnings.warn(f"the views module was not built, calls will take longer on the host: {e}", RuntimeWarning, stacklevel=2)
    return path


def _views_stamp() -> str:
    """The torch that runs: what a views module built against another one is told by."""
    import torch

    return f"{torch.__version__}\n{os.path.dirname(torch.__file__)}\n"


def _views_match() -> bool:
    """Whether the views module is there and was built against this torch."""
    try:
        with open(VIEWS_PATH + ".torch") as f:
            return f.read() == _views_stamp() and os.path.exists(VIEWS_PATH)
    except OSError:
        return False


def _build_views(force: bool) -> None:
    """The views module, with the host compiler, against the torch that runs it."""
    import torch

    if not force and _views_match() and os.path.getmtime(VIEWS_PATH) >= max(os.path.getmtime(VIEWS_SRC), os.path.getmtime(HEADER)):
        return
    if os.path.exists(VIEWS_PATH + ".torch"):  # a module that is not made anew is none
        os.remove(VIEWS_PATH + ".torch")
    root = os.path.dirname(torch.__file__)
    inc = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")]
    lib = os.path.join(root, "lib")
    tmp = VIEWS_PATH + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *[f"-I{p}" for p in inc], VIEWS_SRC, "-o", tmp,
           f"-L{lib}", "-ltorch_python", "-ltorch_cpu", "-lc10", f"-Wl,-rpath,{lib}"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on views.cpp:\n{r.stderr}")
    os.replace(tmp, VIEWS_PATH)
    with open(VIEWS_PATH + ".torch", "w") as f:
        f.write(_views_stamp())


def _build_lib(force: bool, verbose: bool) -> str:
    from concurrent.futures import ThreadPoolExecutor

    headers = [HEADER] + [os.path.join(CSRC, n) for n in os.listdir(CSRC) if n.endswith(".cuh")]
    newest_header = max(os.path.getmtime(h) for h in headers)
    if not force and os.path.exists(LIB_PATH):
        if os.path.getmtime(LIB_PATH) >= max(newest_header, *(os.path.getmtime(s) for s in SRCS)):
            return LIB_PATH
    nvcc = nvcc_path()

    def compile_one(src):
        obj = os.path.join(OBJ_DIR, os.path.basename(src)[:-3] + ".o")
        if not force and os.path.exists(obj) and os.path.getmtime(obj) >= max(newest_header, os.path.getmtime(src)):
            return obj, ""
        tmp = obj + f".tmp{os.getpid()}"
        cmd = [nvcc, *NVCC_FLAGS, *(["-Xptxas=-v"] if verbose else []), "-c", src, "-o", tmp]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stderr}")
        os.replace(tmp, obj)
        return obj, r.stderr

    with ThreadPoolExecutor(len(SRCS)) as ex:
        results = list(ex.map(compile_one, SRCS))
    if verbose:
        for _, log in results:
            print(log, end="")
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    subprocess.run([nvcc, *NVCC_ARCH, "-shared", *[o for o, _ in results], "-o", tmp], check=True)
    os.replace(tmp, LIB_PATH)
    return LIB_PATH


class VskTensor(ctypes.Structure):
    _fields_ = [
        ("data", ctypes.c_void_p),
        ("dtype", ctypes.c_int32),
        ("ndim", ctypes.c_int32),
        ("shape", ctypes.c_int64 * 3),
        ("stride", ctypes.c_int64 * 3),
    ]


DTYPE_BF16, DTYPE_FP8E4M3, DTYPE_I32, DTYPE_I64, DTYPE_U8, DTYPE_F32 = 0, 1, 2, 3, 4, 5

_lib = None
_lock = threading.Lock()

_P = ctypes.POINTER(VskTensor)
_V = ctypes.c_void_p  # a VskTensor by address


def _bind(lib):
    lib.vsk_can_handle.restype = ctypes.c_int
    lib.vsk_can_handle.argtypes = [_P] * 8 + [ctypes.c_int, ctypes.c_int64, ctypes.c_int64, ctypes.c_int,
                                              ctypes.c_float, ctypes.c_int64]
    lib.verify_splitkv_fwd.restype = ctypes.c_int
    lib.verify_splitkv_fwd.argtypes = [_P] * 9 + [ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_float,
                                                  ctypes.c_float, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]
    lib.verify_splitkv_tree_fwd.restype = ctypes.c_int
    lib.verify_splitkv_tree_fwd.argtypes = [_P] * 11 + [ctypes.c_int64, ctypes.c_float, ctypes.c_float, ctypes.c_float,
                                                        ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]
    lib.verify_splitkv_paged_fwd.restype = ctypes.c_int
    lib.verify_splitkv_paged_fwd.argtypes = [_P] * 6 + [ctypes.c_int64, ctypes.c_int64, ctypes.c_float, ctypes.c_float,
                                                        ctypes.c_float, ctypes.c_void_p, ctypes.c_size_t,
                                                        ctypes.c_void_p]
    lib.verify_splitkv_write_fwd.restype = ctypes.c_int
    lib.verify_splitkv_write_fwd.argtypes = [_P] * 10 + [ctypes.c_int64, ctypes.c_float, ctypes.c_float, ctypes.c_float,
                                                         ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]
    lib.verify_splitkv_paged_write_fwd.restype = ctypes.c_int
    lib.verify_splitkv_paged_write_fwd.argtypes = [_P] * 8 + [ctypes.c_int64, ctypes.c_int64, ctypes.c_float,
                                                              ctypes.c_float, ctypes.c_float, ctypes.c_void_p,
                                                              ctypes.c_size_t, ctypes.c_void_p]
    lib.prompt_attn_fwd.restype = ctypes.c_int
    lib.prompt_attn_fwd.argtypes = [_V] * 5 + [ctypes.c_float, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]
    lib.verify_splitkv_shared_fwd.restype = ctypes.c_int
    lib.verify_splitkv_shared_fwd.argtypes = [_V] * 10 + [ctypes.c_int64, ctypes.c_float, ctypes.c_float,
                                                          ctypes.c_float, ctypes.c_void_p, ctypes.c_size_t,
                                                          ctypes.c_void_p]
    lib.verify_splitkv_mass.restype = ctypes.c_int
    lib.verify_splitkv_mass.argtypes = [_V] * 8 + [ctypes.c_int64, ctypes.c_float, ctypes.c_float, ctypes.c_void_p,
                                                   ctypes.c_size_t, ctypes.c_void_p]
    lib.kv_evict.restype = ctypes.c_int
    lib.kv_evict.argtypes = [_V] * 3 + [ctypes.c_int64, ctypes.c_int64] + [_V] * 4 + [
        ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]
    lib.rope_fwd.restype = ctypes.c_int
    lib.rope_fwd.argtypes = [_V] * 6 + [ctypes.c_int, ctypes.c_float, ctypes.c_void_p]
    lib.rope_append_fwd.restype = ctypes.c_int
    lib.rope_append_fwd.argtypes = [_V] * 10 + [ctypes.c_int, ctypes.c_float, ctypes.c_float, ctypes.c_float,
                                                ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]
    lib.rope_append_block_fwd.restype = ctypes.c_int
    lib.rope_append_block_fwd.argtypes = [_V] * 14 + [ctypes.c_int64, ctypes.c_int, ctypes.c_float, ctypes.c_void_p,
                                                      ctypes.c_size_t, ctypes.c_void_p]
    lib.verify_splitkv_block_fwd.restype = ctypes.c_int
    lib.verify_splitkv_block_fwd.argtypes = [_V] * 13 + [ctypes.c_int64, ctypes.c_int64, ctypes.c_float, ctypes.c_void_p,
                                                         ctypes.c_size_t, ctypes.c_void_p]
    lib.vsk_rope_frequencies.restype = ctypes.c_float
    lib.vsk_rope_frequencies.argtypes = [ctypes.c_void_p, ctypes.c_int64, ctypes.c_double, ctypes.c_int] + [
        ctypes.c_double] * 4
    lib.vsk_block_workspace_size.restype = ctypes.c_size_t
    lib.vsk_block_workspace_size.argtypes = [ctypes.c_int64] * 5
    lib.vsk_shared_workspace_size.restype = ctypes.c_size_t
    lib.vsk_shared_workspace_size.argtypes = [ctypes.c_int64] * 5
    lib.vsk_workspace_size.restype = ctypes.c_size_t
    lib.vsk_workspace_size.argtypes = [ctypes.c_int64] * 6
    lib.vsk_workspace_size_for_sms.restype = ctypes.c_size_t
    lib.vsk_workspace_size_for_sms.argtypes = [ctypes.c_int] + [ctypes.c_int64] * 6
    lib.vsk_workspace_init.restype = ctypes.c_int
    lib.vsk_workspace_init.argtypes = [ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]
    lib.vsk_read_error_flags.restype = ctypes.c_int
    lib.vsk_read_error_flags.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.POINTER(ctypes.c_uint32)]
    lib.vsk_set_tuning.restype = None
    lib.vsk_set_tuning.argtypes = [ctypes.c_int, ctypes.c_int]
    lib.vsk_set_tuning_tiles.restype = None
    lib.vsk_set_tuning_tiles.argtypes = [ctypes.c_int]
    lib.vsk_set_tuning_tc.restype = None
    lib.vsk_set_tuning_tc.argtypes = [ctypes.c_int]
    lib.vsk_set_tuning_colsplit.restype = None
    lib.vsk_set_tuning_colsplit.argtypes = [ctypes.c_int]
    lib.vsk_set_tuning_split_launch.restype = None
    lib.vsk_set_tuning_split_launch.argtypes = [ctypes.c_int]
    lib.vsk_set_tuning_cluster.restype = None
    lib.vsk_set_tuning_cluster.argtypes = [ctypes.c_int]
    lib.vsk_set_tuning_pdl.restype = None
    lib.vsk_set_tuning_pdl.argtypes = [ctypes.c_int]
    lib.vsk_set_tuning_pipe.restype = None
    lib.vsk_set_tuning_pipe.argtypes = [ctypes.c_int]
    lib.vsk_set_tuning_colsplit2.restype = None
    lib.vsk_set_tuning_colsplit2.argtypes = [ctypes.c_int]
    lib.vsk_launches_per_call.restype = ctypes.c_int
    lib.vsk_launches_per_call.argtypes = [ctypes.c_int64] * 6
    lib.vsk_call_form.restype = ctypes.c_char_p
    lib.vsk_call_form.argtypes = [ctypes.c_int64] * 7 + [ctypes.c_int]
    lib.vsk_set_tuning_shape.restype = None
    lib.vsk_set_tuning_shape.argtypes = [ctypes.c_int, ctypes.c_int]
    lib.vsk_last_error.restype = ctypes.c_char_p
    lib.vsk_last_error.argtypes = []
    lib.vsk_version.restype = ctypes.c_char_p
    lib.vsk_version.argtypes = []
    return lib


def lib():
    """The loaded CUDA library; raises if it was not built."""
    global _lib
    if _lib is None:
        with _lock:
            if _lib is None:
                if not os.path.exists(LIB_PATH):
                    raise RuntimeError(
                        f"CUDA library {LIB_PATH} is missing: run __graft_entry__.build() "
                        "(there is no CPU fallback)")
                _lib = _bind(ctypes.CDLL(LIB_PATH))
    return _lib


_views = None


def views():
    """The function of the views module; raises if it was not built, or not for the
    Python and torch that run."""
    global _views
    if _views is None:
        with _lock:
            if _views is None:
                if not _views_match():
                    state = "was built against another torch" if os.path.exists(VIEWS_PATH) else "is missing"
                    raise RuntimeError(f"module {VIEWS_PATH} {state}: run build()")
                import torch  # noqa: F401  (its libraries, before the module that needs them)
                from importlib.machinery import ExtensionFileLoader
                from importlib.util import module_from_spec, spec_from_loader

                spec = spec_from_loader("vsk_views", ExtensionFileLoader("vsk_views", VIEWS_PATH))
                module = module_from_spec(spec)
                spec.loader.exec_module(module)
                _views = module.views
    return _views


def last_error() -> str:
    return lib().vsk_last_error().decode()
