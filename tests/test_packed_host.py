"""Packed-document calls: refusals and workspace sizes (no GPU), and the 64-bit forms
against small hand-made cases."""
import ctypes
import math

import pytest

import packed_ref as R

torch = pytest.importorskip("torch")

NULL, SHAPE, ALIGN, WORKSPACE, UNSUPPORTED = -1, -2, -4, -5, -8
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


def _rows(wan, ptr=P, stride=1536):
    return ctypes.byref(wan.packed.Rows(ptr, stride))


def _rope_call(wan, spec=None, cfg=None, rows=4, kv=12, norm=0, q=None, k="same", w=P, out=None):
    cfg = cfg or wan.make_config(1536, 12, 64)
    spec = spec or wan.rope([44, 42, 42])
    q = q or _rows(wan)
    k = q if k == "same" else k
    return wan.lib.wan_qk_norm_rope_fwd(ctypes.byref(cfg), ctypes.byref(spec), P, rows, kv, norm, q, k, w, w, out or q, k,
                                        None)


@pytest.mark.parametrize("change,status", [
    (dict(axis=[64, 62, 4]), SHAPE),          # more dims than the head has
    (dict(axis=[43, 42, 42]), SHAPE),         # odd
    (dict(theta=1.0), SHAPE), (dict(theta=math.nan), SHAPE), (dict(amplitude=0.0), SHAPE),
    (dict(amplitude=math.inf), SHAPE), (dict(scaling=9), SHAPE), (dict(layout=2), SHAPE), (dict(n_axes=4), SHAPE),
    (dict(scaling=1, factor=0.0), SHAPE), (dict(scaling=1, factor=math.nan), SHAPE),
    (dict(scaling=2, axis=[2, 42, 42], factor=2.0), SHAPE),
    (dict(scaling=3, factor=2.0), SHAPE),     # no original length
    (dict(scaling=3, factor=2.0, orig=8, fast=1.0, slow=1.0), SHAPE),
])
def test_rope_refuses_specs(wan, change, status):
    spec = wan.rope([44, 42, 42])
    for a, n in enumerate(change.pop("axis", [])):
        spec.axis_dim[a] = n
    f, o = change.pop("factor", None), change.pop("orig", None)
    for a in range(3):
        if f is not None:
            spec.factor[a] = f
        if o is not None:
            spec.orig_len[a] = o
    for name, v in change.items():
        setattr(spec, name, v)
    assert _rope_call(wan, spec) == status


def test_rope_refuses_arguments(wan):
    assert _rope_call(wan, rows=-1) == SHAPE
    assert _rope_call(wan, kv=0) == SHAPE
    assert _rope_call(wan, norm=3) == SHAPE
    assert _rope_call(wan, q=_rows(wan, 0)) == NULL
    assert _rope_call(wan, q=_rows(wan, P + 8)) == ALIGN
    assert _rope_call(wan, q=_rows(wan, P, 1535)) == SHAPE
    assert _rope_call(wan, norm=1, w=None) == NULL
    assert _rope_call(wan, cfg=wan.make_config(6400, 50, 64), q=_rows(wan, P, 6400), kv=50) == UNSUPPORTED
    assert _rope_call(wan, cfg=wan.make_config(1536, 6, 64)) == SHAPE  # head_dim 256
    cfg = wan.make_config(1536, 12, 64)
    n = wan.qk_norm_rope_workspace_bytes(cfg, 1000, 12, "width")
    assert n > 0 and wan.qk_norm_rope_workspace_bytes(cfg, 1000, 12, "none") == 0
    r = _rows(wan)
    args = (ctypes.byref(cfg), ctypes.byref(wan.rope([128])), P, 1000, 12, 2, r, r, r, r, P, P, r, r, P, P)
    assert wan.lib.wan_qk_norm_rope_bwd(*args, None, n, None) == NULL
    assert wan.lib.wan_qk_norm_rope_bwd(*args, P, n - 1, None) == WORKSPACE
    with pytest.raises(ValueError):
        wan.rope([64], layout="other")
    with pytest.raises(ValueError):
        wan.rope([64], scaling="linear")


def _residual_call(wan, cfg=None, x=P, y=P, e=P, cu=P, n=2, rows=8, w_post=None, **opt):
    cfg = cfg or wan.make_config(1536, 12, 64)
    spec = wan.residual_norm()
    spec.w_post = w_post
    for k, v in opt.items():
        setattr(spec, k, v)
    return wan.lib.wan_gated_residual_norm_fwd(ctypes.byref(cfg), ctypes.byref(spec), x, y, e, None, cu, n, rows, P, P, None)


def test_residual_norm_refuses(wan):
    for bad in (dict(pre=0), dict(pre=3), dict(post=3), dict(gate=6), dict(gate=-2), dict(chunk=2),
                dict(residual_scale=math.inf), dict(gate=3, chunk=1), dict(gate=1, chunk=0), dict(w_post=P),
                dict(rows=-1), dict(n=-1)):
        assert _residual_call(wan, **bad) == SHAPE, bad
    assert _residual_call(wan, gate=2, e=None) == NULL
    assert _residual_call(wan, x=None) == NULL
    assert _residual_call(wan, y=P + 4) == ALIGN
    assert _residual_call(wan, cu=None) == NULL
    assert _residual_call(wan, cfg=wan.make_config(8256, 129, 64)) == UNSUPPORTED
    cfg, g = wan.make_config(1536, 12, 64), wan.packed.ResidualNormGrads(P)
    n = wan.gated_residual_norm_workspace_bytes(cfg, 8, 2)
    args = (ctypes.byref(cfg), ctypes.byref(wan.residual_norm(gate=2)), P, P, P, None, P, 2, 8, P, None, P, P, ctypes.byref(g))
    assert wan.lib.wan_gated_residual_norm_bwd(*args, None, n, None) == NULL
    assert wan.lib.wan_gated_residual_norm_bwd(*args, P, n - 1, None) == WORKSPACE


def _attn_call(wan, cfg=None, docs=None, nq=8, nk=8, kv=12, q=None, v=None, lse=None, **opt):
    cfg = cfg or wan.make_config(1536, 12, 64)
    if docs is None:
        docs = wan.Documents(2, P, P, None, 0, 0.0, 0.0, None)
    for k, val in opt.items():
        setattr(docs, k, val)
    q = q or _rows(wan)
    return wan.lib.wan_attention_packed_fwd(ctypes.byref(cfg), ctypes.byref(docs), nq, nk, kv, q, _rows(wan), v or _rows(wan),
                                            _rows(wan), lse, None, 0, None)


def test_attention_refuses(wan):
    for bad in (dict(nq=-1), dict(nk=-1), dict(kv=5), dict(kv=0), dict(n_docs=-1), dict(causal_block=-1), dict(cap=-1.0),
                dict(cap=math.nan), dict(scale=math.inf), dict(q=_rows(wan, P, 1528))):
        assert _attn_call(wan, **bad) == SHAPE, bad
    assert _attn_call(wan, q=_rows(wan, 0)) == NULL
    assert _attn_call(wan, cu_q=None) == NULL
    assert _attn_call(wan, q=_rows(wan, P + 2)) == ALIGN
    assert _attn_call(wan, v=_rows(wan, P, 1540)) == ALIGN
    assert _attn_call(wan, prefix=P + 4) == ALIGN
    assert _attn_call(wan, lse=P + 4) == ALIGN
    assert _attn_call(wan, cfg=wan.make_config(768, 12, 64), q=_rows(wan, P, 768)) == UNSUPPORTED  # bf16, head_dim 64
    cfg, r = wan.make_config(1536, 12, 64), _rows(wan)
    n = wan.attention_packed_workspace_bytes(cfg, 8, 8, 2, 12, True)
    args = (ctypes.byref(cfg), ctypes.byref(wan.Documents(2, P, P)), 8, 8, 12, r, r, r, r, P, r, r, r, r)
    assert n > 0
    assert wan.lib.wan_attention_packed_bwd(*args, None, n, None) == NULL
    assert wan.lib.wan_attention_packed_bwd(*args, P, n - 1, None) == WORKSPACE
    assert wan.attention_packed_workspace_bytes(cfg, -1, 8, 2, 12) == 0
    assert wan.attention_packed_workspace_bytes(cfg, 8, 8, 2, 5, True) == 0


def test_binding_refuses_tensors(wan):
    cfg = wan.make_config(256, 2, 64)
    cpu = torch.zeros(4, 256, dtype=torch.bfloat16)
    cu = torch.tensor([0, 4], dtype=torch.int32)
    for call in (lambda: wan.attention_packed_fwd(cfg, wan.documents(cu), cpu, cpu, cpu, cpu),
                 lambda: wan.qk_norm_rope_fwd(cfg, wan.rope([128]), torch.zeros(4, 1, dtype=torch.int32), cpu, cpu, cpu, cpu),
                 lambda: wan.gated_residual_norm_fwd(cfg, wan.residual_norm(), cpu.float(), cpu, None, None, cu, cpu.float(), cpu)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


# ------------------------------------------------------------------ the 64-bit forms themselves
def test_reference_masks():
    see = R.visible(4, 4, 1, 0, "cpu")
    assert torch.equal(see, torch.ones(4, 4).tril().bool())
    assert torch.equal(R.visible(2, 5, 1, 0, "cpu").sum(1), torch.tensor([4, 5]))   # aligned at the ends
    assert torch.equal(R.visible(5, 2, 1, 0, "cpu").sum(1), torch.tensor([0, 0, 0, 1, 2]))
    assert torch.equal(R.visible(6, 6, 4, 0, "cpu").sum(1), torch.tensor([4, 4, 4, 4, 6, 6]))
    assert torch.equal(R.visible(3, 3, 1, 2, "cpu").sum(1), torch.tensor([2, 2, 3]))
    assert R.visible(3, 7, 0, 0, "cpu").all()


def test_reference_attention_gradient():
    """The written-out gradient against automatic differentiation of the forward."""
    torch.manual_seed(0)
    q, k, v = (torch.randn(7, w, dtype=torch.float64, requires_grad=True) for w in (16, 8, 8))
    do = torch.randn(7, 16, dtype=torch.float64)
    opt = dict(block=2, prefix=[1, 0], cap=3.0, slopes=[0.5, 0.25])
    out = R.attention(q, k, v, 2, 1, [0, 4, 7], [0, 4, 7], torch.float32, do=do, **opt)
    auto = torch.autograd.grad(out["o"][0], (q, k, v), do)
    for n, g in zip(("dq", "dk", "dv"), auto):
        assert torch.allclose(out[n][0], g, atol=1e-12)


def test_reference_rope_turns_by_relative_positions():
    """A score of two rotated vectors depends on the difference of their positions only."""
    torch.manual_seed(0)
    q, k = torch.randn(1, 8, dtype=torch.float64), torch.randn(1, 8, dtype=torch.float64)
    for layout in ("interleaved", "half"):
        s = []
        for base in (3, 1000):
            a, b = (R.rope_angles(torch.tensor([[base + x, 2 * base]]), [4, 4]) for x in (5, 0))
            s.append((R.rope_forward(q, None, 1, a, layout, "none", 1.0) * R.rope_forward(k, None, 1, b, layout, "none", 1.0)).sum())
        assert abs(s[0] - s[1]) < 1e-10
