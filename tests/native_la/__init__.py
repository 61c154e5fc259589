"""Test-only CUDA library ``libla_testing.so``: the linear-attention kernels compiled with GDN_WAIT_LIMIT=0, so that
every pipeline wait gives up on its first poll (the waits that drain copies and products in flight keep their own
limits). ``short_waits.cu`` exposes the forward and the backward."""
import ctypes
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "_build", "libla_testing.so")


def load():
    from fp8_state_qat_gb300 import build as pb
    short = ["GDN_WAIT_LIMIT=0u"]
    srcs = [os.path.join(HERE, "short_waits.cu")] + [(os.path.join(pb.CSRC, f), short) for f in
                                                    ("la_chunk.cu", "la_state.cu", "la_out.cu", "tma_maps.cu")]
    deps = [s if isinstance(s, str) else s[0] for s in srcs] + pb.headers() + [__file__]
    if not pb.newer_than(LIB_PATH, deps):
        pb.compile_library(srcs, LIB_PATH, os.path.join(HERE, "_build", "obj"))
    return ctypes.CDLL(LIB_PATH)
