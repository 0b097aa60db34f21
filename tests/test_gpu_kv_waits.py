"""What an attention call leaves behind when one of its CTAs gave up on a wait:
a build of the kernels for tests (kv_giveup.cu) lets a chosen CTA run as after
an expired wait."""

import ctypes
import os
import subprocess

import numpy as np
import pytest

from page_scoring_top_b200 import build as b200_build
from test_gpu_kv import attn_case, upload

torch = pytest.importorskip("torch")

HERE = os.path.dirname(os.path.abspath(__file__))
SOURCE = os.path.join(HERE, "kv_giveup.cu")
LIB = os.path.join(HERE, "libkv_giveup.so")


def build_giveup():
    deps = [SOURCE] + [f for f in b200_build._deps() if os.path.basename(f) in
                       ("kv_attn.cuh", "kv_attn.cu", "kv_attn_tc.cu", "kv.cuh", "tc.cuh", "common.cuh", "kernels.h")]
    if not os.path.exists(LIB) or any(os.path.getmtime(f) > os.path.getmtime(LIB) for f in deps):
        tmp = LIB + ".tmp%d" % os.getpid()
        subprocess.check_call([os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc"), "-shared", "-O3", "-std=c++17",
                               *b200_build.ARCH, "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler",
                               "-fvisibility=hidden", "--expt-relaxed-constexpr", "-I",
                               os.path.join(b200_build.ROOT, "include"), "-I",
                               os.path.join(b200_build.HERE, "csrc"), SOURCE, "-o", tmp])
        os.replace(tmp, LIB)
    lib = ctypes.CDLL(LIB)
    p, i = ctypes.c_void_p, ctypes.c_int
    lib.giveup_ws_floats.restype = ctypes.c_int64
    lib.giveup_attention.argtypes = [p, p, p, p, p, i, p, i, p, i, i, i, i, i, i, ctypes.c_float, p, p, p, p, p, i, i]
    return lib


def test_the_test_build_compiles():
    assert build_giveup().giveup_ws_floats(148) > 0


@pytest.fixture(scope="module")
def giveup():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    lib = build_giveup()
    sms = torch.cuda.get_device_properties(0).multi_processor_count

    class Launcher:
        """Workspace, counters and status word of a context; run() one call on them."""
        num_sms = sms

        def __init__(self):
            self.ws = torch.zeros(lib.giveup_ws_floats(sms), device="cuda")
            self.arrive = torch.zeros(sms, dtype=torch.int32, device="cuda")
            self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

        def run(self, c, t, cta=-1):
            B, T, Q, D = c["q64"].shape
            n, H, P, _ = c["kc"].shape
            out = torch.full((B, T, Q, D), float("nan"), dtype=torch.bfloat16, device="cuda")
            lse = torch.full((B, T, Q), float("nan"), device="cuda")
            torch.cuda.synchronize()
            at = [x.data_ptr() for x in t[:6]]
            assert lib.giveup_attention(c["q"].data_ptr(), *at[:4], n, at[4], c["table"].shape[1], at[5], B, T, Q,
                                        H, D, P, c["scale"], out.data_ptr(), lse.data_ptr(), self.ws.data_ptr(),
                                        self.arrive.data_ptr(), self.status.data_ptr(), sms, cta) == 0
            bits = int(self.status.item())
            self.status.zero_()
            return out, lse, bits

    return Launcher


# streamed kernel with large and small pages, prompt kernel with large and small
# pages: one long row cut over all SMs, then rows that end inside an SM's share
SHAPES = [(1, 1, 4, 64, 64, [[19190]]), (5, 1, 8, 64, 64, [[19200], [3], [9000], [0], [12345]]),
          (6, 1, 4, 48, 16, [[9600], [1], [0], [31], [5000], [33]]),
          (3, 16, 8, 64, 64, None), (2, 40, 4, 64, 16, None)]


def case(i):
    B, T, Q, D, P, counts = SHAPES[i]
    if counts is None:
        counts = np.array([19000, 700, 8000][:B])[:, None] + np.arange(T)
    return attn_case(40 + i, B, T, Q, 1, D, P, -(-int(np.max(counts)) // P), "e4m3", counts)


@pytest.mark.gpu
@pytest.mark.parametrize("i", range(len(SHAPES)))
def test_a_cta_that_gives_up_is_reported_and_leaves_the_gpu_usable(giveup, i):
    c = case(i)
    t = upload(c)
    want, wl, bits = giveup().run(c, t)
    assert bits == 0 and not torch.isnan(want).any()
    for cta in (0, 1, giveup.num_sms // 2, giveup.num_sms - 1):
        assert giveup().run(c, t, cta)[2] == 2
        again, al, bits = giveup().run(c, t)
        assert bits == 0 and torch.equal(again, want) and torch.equal(al, wl)


@pytest.mark.gpu
@pytest.mark.parametrize("i", range(len(SHAPES)))
def test_later_calls_on_the_same_workspace_are_right(giveup, i):
    # the counters of the items that the CTA shares are back at zero, and the
    # next call joins its parts when all of them are there
    c = case(i)
    t = upload(c)
    ctx = giveup()
    want, wl, bits = ctx.run(c, t)
    assert bits == 0 and not ctx.arrive.any()
    for cta in range(0, giveup.num_sms, 3):
        assert ctx.run(c, t, cta)[2] == 2
        assert not ctx.arrive.any(), "counters left by CTA %d" % cta
        ctx.ws.fill_(float("nan"))  # a part joined before it is written shows
        out, lse, bits = ctx.run(c, t)
        assert bits == 0 and torch.equal(out, want) and torch.equal(lse, wl)
