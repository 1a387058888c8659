"""Build and load libmlp_chain.so (the CUDA library behind include/mlp_chain.h and mlp_block.h), and
_marshal (the argument checks of block.py, compiled against torch's headers).

The library is compiled in-tree with nvcc for sm_103a only. Loading it never falls back to
anything else: if the shared object is missing, ``load()`` raises.  _marshal needs torch to be
compiled and to be used, the library does not.
"""
from __future__ import annotations

import ctypes
import glob
import importlib.util
import os
import runpy
import shutil
import subprocess
import sys
import sysconfig
import tempfile
import threading

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB_PATH = os.path.join(PKG, "libmlp_chain.so")
MARSHAL_SOURCE = os.path.join(CSRC, "marshal.cpp")
SOURCES = [os.path.join(CSRC, f) for f in ("mlp_chain.cu", "host_protocol.cpp", "linear.cu", "layer_norm.cu")]
DEPENDS = SOURCES + [os.path.join(CSRC, f) for f in ("chain_kernel.cuh", "ptx.cuh", "protocol.h", "dep_groups.h",
                                                     "linear_kernel.cuh", "cuda_call.h", "row_blocks.h")] + [
    os.path.join(INCLUDE, f) for f in ("mlp_chain.h", "mlp_block.h")]

NVCC_FLAGS = [
    "-std=c++17", "-O3", "-gencode", "arch=compute_103a,code=sm_103a", "-lineinfo",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-pthread",
]

_lock = threading.Lock()
_lib = None
_marshal = None


def _older(path: str, sources) -> bool:
    return not os.path.exists(path) or any(os.path.getmtime(f) > os.path.getmtime(path) for f in sources)


def _torch_dir():
    spec = importlib.util.find_spec("torch")
    return spec.submodule_search_locations[0] if spec else None


def marshal_path(torch_dir: str) -> str:
    """Where _marshal is for this Python and this torch: compiled against another one's headers it is another module."""
    version = runpy.run_path(os.path.join(torch_dir, "version.py"))["__version__"]
    return os.path.join(PKG, f"_marshal.{sys.implementation.cache_tag}-torch-{version}.so")


def _marshal_flags(torch_dir: str):
    return (["-I", os.path.join(torch_dir, "include"), "-I", sysconfig.get_paths()["include"]],
            ["-L", os.path.join(torch_dir, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10"])


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile what is older than its sources, with nvcc (cross-compiles without a GPU): the library, and _marshal where torch
    is installed. Returns the library's path."""
    nvcc = os.environ.get("NVCC", "nvcc")
    torch_dir = _torch_dir()
    marshal = torch_dir and marshal_path(torch_dir)
    work = tempfile.mkdtemp(prefix="mlp_chain_build")
    tmp = f".tmp{os.getpid()}"
    procs = []

    def start(cmd):
        if verbose:
            print(" ".join(cmd))
        procs.append(subprocess.Popen(cmd))
        return procs[-1]

    def finish(proc):
        if proc.wait():
            raise subprocess.CalledProcessError(proc.returncode, proc.args)

    try:   # one compiler per source, side by side
        checks, objs, parts = None, [], []
        if marshal and (force or _older(marshal, [MARSHAL_SOURCE, os.path.join(INCLUDE, "mlp_block.h")])):
            compile_flags, link_flags = _marshal_flags(torch_dir)
            checks = start([nvcc, *NVCC_FLAGS, *compile_flags, "-shared", "-o", marshal + tmp, MARSHAL_SOURCE, *link_flags])
        if force or _older(LIB_PATH, DEPENDS):
            objs = [os.path.join(work, os.path.basename(f) + ".o") for f in SOURCES]
            parts = [start([nvcc, *NVCC_FLAGS, "-I", INCLUDE, "-c", "-o", o, f]) for f, o in zip(SOURCES, objs)]
        for p in parts:
            finish(p)
        if parts:
            finish(start([nvcc, *NVCC_FLAGS, "-shared", "-o", LIB_PATH + tmp, *objs]))
            os.replace(LIB_PATH + tmp, LIB_PATH)
        if checks:   # (after the library, which does not need it)
            finish(checks)
            for f in glob.glob(os.path.join(glob.escape(PKG), "_marshal*.so")):   # for other versions
                os.remove(f)
            os.replace(marshal + tmp, marshal)
    finally:
        for p in procs:
            p.wait()
        for f in (LIB_PATH + tmp, (marshal or "") + tmp):
            if os.path.exists(f):
                os.remove(f)
        shutil.rmtree(work, ignore_errors=True)
    return LIB_PATH


i32, i64, u32, u64 = ctypes.c_int32, ctypes.c_int64, ctypes.c_uint32, ctypes.c_uint64
vp, szt = ctypes.c_void_p, ctypes.c_size_t
MAX_GEMMS = 4


class ChainDesc(ctypes.Structure):
    _fields_ = [
        ("M", i64), ("num_gemms", i32), ("dims", i64 * (MAX_GEMMS + 1)),
        ("in_dtype", ctypes.c_int), ("acc_dtype", ctypes.c_int), ("h_dtype", ctypes.c_int),
        ("out_dtype", ctypes.c_int), ("tile_m", i32), ("tile_n", i32 * MAX_GEMMS), ("tile_k", i32),
        ("epilogue", ctypes.c_int), ("residual", i32), ("mode", ctypes.c_int),
        ("microbatch_rows", i32), ("device", i32), ("debug_flags", u32), ("drop_tile", i32),
        ("timeout_us", u32), ("grid_ctas", i32), ("raster_group", i32), ("pipe_stages", i32),
        ("weight_layout", i32), ("k_split", i32 * MAX_GEMMS), ("acc_split", i32), ("gated", i32), ("cta_pair", i32),
        ("splitk_exchange", i32), ("split_clusters", i32),
    ]


class Event(ctypes.Structure):
    _fields_ = [("stage", i32), ("tile", i32), ("smid", i32), ("cta", i32), ("t_start", u64),
                ("t_end", u64), ("seq_start", u32), ("seq_end", u32), ("t_acc", u64)]


class ChainInfo(ctypes.Structure):
    _fields_ = [
        ("num_gemms", i32), ("tile_m", i32), ("tile_k", i32), ("tile_n", i32 * MAX_GEMMS),
        ("tiles_m", i32 * MAX_GEMMS), ("tiles_n", i32 * MAX_GEMMS), ("grid_ctas", i32),
        ("num_sms", i32), ("pipe_stages", i32), ("smem_bytes", i32), ("tmem_cols", i32),
        ("launches_per_run", i32), ("cluster_size", i32), ("k_split", i32 * MAX_GEMMS), ("cta_pair", i32),
        ("raster_group", i32), ("fill_k", i32 * MAX_GEMMS),
        ("split_across", i32 * MAX_GEMMS), ("queue_free", i32 * MAX_GEMMS),
    ]


class LinearDesc(ctypes.Structure):
    _fields_ = [("K", i64), ("N", i64), ("experts", i32), ("weight_layout", i32), ("activation", ctypes.c_int),
                ("bias_dtype", ctypes.c_int), ("dw_dtype", ctypes.c_int), ("device", i32), ("timeout_us", u32)]


class LinearPlan(ctypes.Structure):
    _fields_ = [("form", i32), ("cta_pair", i32), ("tile_cols", i32), ("k_split", i32), ("pipe_stages", i32)]


class Scoreboard(ctypes.Structure):
    _fields_ = [("producers", i32), ("consumers", i32), ("groups", i32), ("edges", i32),
                ("releases_per_producer", i32), ("pg_off", vp), ("pg_tgt", vp), ("grp_off", vp),
                ("grp_mem", vp), ("grp_target", vp), ("cons_grp", vp)]


# every symbol include/mlp_chain.h and include/mlp_block.h declare: name -> (restype, argtypes)
SIGNATURES = {
    "mlp_chain_create": (ctypes.c_int, [ctypes.POINTER(ChainDesc), ctypes.POINTER(vp)]),
    "mlp_chain_workspace_size": (ctypes.c_int, [vp, ctypes.POINTER(szt)]),
    "mlp_chain_run": (ctypes.c_int, [vp, vp, vp, vp, vp, vp]),
    "mlp_chain_run_host": (ctypes.c_int, [vp, vp, vp, vp, vp, vp, vp, vp]),
    "mlp_chain_check": (ctypes.c_int, [vp, vp]),
    "mlp_chain_get_deps": (ctypes.c_int, [vp, i32, ctypes.POINTER(vp), ctypes.POINTER(vp),
                                          ctypes.POINTER(vp), ctypes.POINTER(i32), ctypes.POINTER(i32)]),
    "mlp_scoreboard_build": (ctypes.c_int, [i64, i64, i64, i32, i32, i32, i32, i32, ctypes.POINTER(Scoreboard)]),
    "mlp_chain_get_scoreboard": (ctypes.c_int, [vp, i32, ctypes.POINTER(Scoreboard)]),
    "mlp_chain_get_event_log": (ctypes.c_int, [vp, vp, szt, ctypes.POINTER(szt)]),
    "mlp_chain_get_info": (ctypes.c_int, [vp, ctypes.POINTER(ChainInfo)]),
    "mlp_chain_destroy": (ctypes.c_int, [vp]),
    "mlp_deps_build": (i64, [i64, i64, i64, i32, i32, i32, i32, vp, vp, i64, vp]),
    "mlp_protocol_model": (ctypes.c_int, [i32, i32, vp, i32, i32, i32, u64, i32, u32, vp]),
    "mlp_protocol_model_slices": (ctypes.c_int, [i32, i32, vp, vp, i32, i32, i32, u64, i32, i32, u32, vp]),
    "mlp_chain_run_noalloc": (ctypes.c_int, [i64, i64, i64, i64, vp, vp, vp, vp, i32, vp]),
    "mlp_status_str": (ctypes.c_char_p, [ctypes.c_int]),
    "mlp_layernorm_forward": (ctypes.c_int, [i64, i64, vp, i64, ctypes.c_int, vp, vp, ctypes.c_int, ctypes.c_float, vp,
                                             i64, vp, vp, vp]),
    "mlp_layernorm_backward": (ctypes.c_int, [i64, i64, vp, i64, vp, i64, ctypes.c_int, vp, ctypes.c_int, vp, vp, vp,
                                              i64, vp, i64, vp, vp, vp, vp]),
    "mlp_layernorm_workspace_size": (ctypes.c_int, [i64, i64, ctypes.POINTER(szt)]),
    "mlp_linear_create": (ctypes.c_int, [ctypes.POINTER(LinearDesc), ctypes.POINTER(vp)]),
    "mlp_linear_destroy": (ctypes.c_int, [vp]),
    "mlp_linear_workspace_size": (ctypes.c_int, [vp, i64, ctypes.POINTER(szt)]),
    "mlp_linear_forward": (ctypes.c_int, [vp, i64, vp, i64, vp, vp, vp, i64, vp, vp, i64, vp, i64, vp]),
    "mlp_linear_backward": (ctypes.c_int, [vp, i64, vp, i64, vp, i64, vp, vp, i64, vp, vp, i64, vp, vp, vp, vp]),
    "mlp_linear_check": (ctypes.c_int, [vp, vp]),
    "mlp_linear_get_plan": (ctypes.c_int, [vp, i64, i32, ctypes.POINTER(LinearPlan)]),
}


def load():
    """The loaded library. Raises if it has not been built (there is no fallback path)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(f"CUDA library {LIB_PATH} is missing: call "
                                   "mlp_latency_gb300.build() (needs nvcc) first")
            lib = ctypes.CDLL(LIB_PATH)
            for name, (res, args) in SIGNATURES.items():
                fn = getattr(lib, name)
                fn.restype = res
                fn.argtypes = args
            _lib = lib
    return _lib


def load_marshal():
    """The argument checks of block.py, bound to the loaded library."""
    global _marshal
    lib = load()
    with _lock:
        if _marshal is None:
            import torch  # noqa: F401  (the module's symbols are torch's)
            path = marshal_path(os.path.dirname(torch.__file__))
            if not os.path.exists(path):
                raise RuntimeError(f"{path} is missing: call mlp_latency_gb300.build() first")
            spec = importlib.util.spec_from_file_location("mlp_latency_gb300._marshal", path)
            module = importlib.util.module_from_spec(spec)
            spec.loader.exec_module(module)
            module.bind(*(ctypes.cast(getattr(lib, f), ctypes.c_void_p).value for f in (
                "mlp_layernorm_forward", "mlp_layernorm_backward", "mlp_layernorm_workspace_size", "mlp_linear_workspace_size",
                "mlp_linear_forward", "mlp_linear_backward")))
            _marshal = module
    return _marshal
