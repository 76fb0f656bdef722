"""The grouped products' choice of kernel, from the library's own rule compiled
for the host: by these names a test says which kernel its shape is meant for."""
import ctypes
import functools
import os
import subprocess
import tempfile

HERE = os.path.dirname(os.path.abspath(__file__))

FEW, SWIGLU_PAIRS, NARROW, WIDE_F8, WIDE_16 = 32, 96, 128, 192, 256


@functools.lru_cache(None)
def host():
    so = os.path.join(tempfile.mkdtemp(prefix="gmm_plan_"), "libgmm_plan.so")
    subprocess.run(["g++", "-std=c++17", "-O1", "-fPIC", "-shared", "-x", "c++", "-o", so,
                    os.path.join(HERE, "host", "gmm_plan.cpp")], check=True)
    lib = ctypes.CDLL(so)
    lib.token_tile_host.argtypes = [ctypes.c_longlong] + [ctypes.c_int] * 6
    lib.max_tiles_host.argtypes = [ctypes.c_longlong] + [ctypes.c_int] * 3
    lib.max_tiles_host.restype = ctypes.c_longlong
    return lib


def kernel(kind, m, n, groups=None, swiglu=False, sms=152):
    """Token columns of the tiles that m rows by n weight rows take; groups: None
    for one matrix without offsets."""
    nb = -(-n // 128)
    return host().token_tile_host(m, groups or 1, groups is not None, nb, kind == "f8", swiglu,
                                  sms)


def pair_tiles(nt, sizes, n):
    """Tiles that the pair kernel makes of groups of these sizes."""
    return sum(-(-s // nt) for s in sizes) * -(-(-(-n // 128)) // 2)


def device_sms():
    import torch
    return torch.cuda.get_device_properties(0).multi_processor_count
