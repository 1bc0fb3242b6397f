"""Packed-document calls at their edges, without a GPU: what is refused before a launch."""
import ctypes

import pytest

pytest.importorskip("torch")

SHAPE = -2
P = 1 << 20  # a 16-byte aligned fake device address; nothing is read before a launch


@pytest.fixture(scope="module")
def wan():
    from video_diffusion_transformer_wan_b200 import build
    build.build()
    import video_diffusion_transformer_wan_b200 as w
    return w


@pytest.fixture(autouse=True)
def no_launch(wan):
    n = wan.launch_count()
    yield
    assert wan.launch_count() == n


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("scale,cap", [
    (0.0, 1e-40),    # scale / cap is no fp32 number: a score of 0 became NaN
    (0.0, 3e38),     # cap log2(e) is none
    (3e38, 0.0), (-3e38, 0.0), (1e30, 1e-30),
    (1e-30, 1e30),   # scale / cap loses its digits
])
def test_factors_that_are_no_numbers(wan, dtype, scale, cap):
    cfg = wan.make_config(1536, 12, 64, dtype=dtype)
    docs = wan.Documents(2, P, P, None, 0, scale, cap, None)
    r = ctypes.byref(wan.packed.Rows(P, 1536))
    args = (ctypes.byref(cfg), ctypes.byref(docs), 8, 8, 12, r, r, r, r)
    assert wan.lib.wan_attention_packed_fwd(*args, None, None, 0, None) == SHAPE
    assert wan.lib.wan_attention_packed_bwd(*args, P, r, r, r, r, P, 1 << 30, None) == SHAPE
