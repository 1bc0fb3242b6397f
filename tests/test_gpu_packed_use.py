"""Packed-document operators as they are used: one after another with their gradients, on side
streams, captured and replayed, over tensors of more than 2^31 elements, with offsets that do
not fit, and the calls that the binding refuses."""
import pytest

import packed_ref as R
from gpu_util import rms_err

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ACT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def wan():
    import video_diffusion_transformer_wan_b200 as w
    return w


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Step:
    """The part of a block between the q/k/v projection and the FFN, over packed documents:
    rotary q and k with the width norm, attention in documents, gated residual and norms;
    then its gradient. Buffers are made once, so that a step can be captured."""

    def __init__(self, wan, dtype, lens, H, Hk, d, seed=0, causal=0):
        self.wan, self.H, self.Hk, self.d, self.lens, act = wan, H, Hk, d, lens, ACT[dtype]
        g = torch.Generator(device="cuda").manual_seed(seed)
        rnd = lambda *s, k=1.0, t=act: (torch.randn(*s, generator=g, device="cuda") * k).to(t)  # noqa: E731
        D, n, self.act, self.causal = H * d, sum(lens), act, causal
        self.cfg = wan.make_config(D, H, 64, dtype=dtype)
        self.cu = _i32(R.cu_of(lens))
        self.pos = torch.randint(0, 500, (n, 3), generator=g, device="cuda", dtype=torch.int32)
        self.qkv, self.x = rnd(n, (H + 2 * Hk) * d), rnd(n, D, t=torch.float32)
        self.wq, self.wk = rnd(D, k=0.1) + 1, rnd(Hk * d, k=0.1) + 1
        self.e, self.mb = rnd(len(lens), 6, D, k=0.2, t=torch.float32), rnd(6, D, k=0.1, t=torch.float32)
        self.dh, self.up = rnd(n, D), rnd(n, D, t=torch.float32)
        self.axes = [d // 2, d // 4, d // 4]
        self.rope, self.op = wan.rope(self.axes), wan.residual_norm(pre="layer", post="rms", gate=2, chunk=1)
        self.docs = wan.documents(self.cu, causal_block=causal)
        new = lambda *s, t=act: torch.empty(*s, dtype=t, device="cuda")  # noqa: E731
        W = Hk * d
        self.q, self.k, self.o, self.lse = new(n, D), new(n, W), new(n, D), new(H, n, t=torch.float32)
        self.x2, self.h = new(n, D, t=torch.float32), new(n, D)
        self.dx, self.dy, self.dqr, self.dkr = new(n, D, t=torch.float32), new(n, D), new(n, D), new(n, W)
        self.dqkv = new(n, D + 2 * W)
        self.dwq, self.dwk, self.de = new(D, t=torch.float32), new(W, t=torch.float32), torch.zeros_like(self.e)
        size = max(wan.attention_packed_workspace_bytes(self.cfg, n, n, len(lens), Hk, True),
                   wan.gated_residual_norm_workspace_bytes(self.cfg, n, len(lens)),
                   wan.qk_norm_rope_workspace_bytes(self.cfg, n, Hk, "width"))
        self.ws = new(size, t=torch.uint8)

    def parts(self, t):
        D, W = self.H * self.d, self.Hk * self.d
        return t[:, :D], t[:, D:D + W], t[:, D + W:]

    def run(self):
        w, kw = self.wan, dict(kv_heads=self.Hk)
        q, k, v = self.parts(self.qkv)
        norm = dict(norm="width", w_q=self.wq, w_k=self.wk)
        w.qk_norm_rope_fwd(self.cfg, self.rope, self.pos, q, k, self.q, self.k, **kw, **norm)
        w.attention_packed_fwd(self.cfg, self.docs, self.q, self.k, v, self.o, self.lse, ws=self.ws, **kw)
        args = (self.e, self.mb, self.cu)
        w.gated_residual_norm_fwd(self.cfg, self.op, self.x, self.o, *args, self.x2, self.h)
        w.gated_residual_norm_bwd(self.cfg, self.op, self.x2, self.o, *args, self.dh, self.up, self.dx, self.dy, self.ws,
                                  de=self.de)
        dq, dk, dv = self.parts(self.dqkv)
        w.attention_packed_bwd(self.cfg, self.docs, self.q, self.k, v, self.o, self.lse, self.dy, self.dqr, self.dkr, dv,
                               ws=self.ws, **kw)
        w.qk_norm_rope_bwd(self.cfg, self.rope, self.pos, self.dqr, self.dkr, q, k, dq, dk, dw_q=self.dwq, dw_k=self.dwk,
                           ws=self.ws, **kw, **norm)

    def results(self):
        return [t.clone() for t in (self.x2, self.h, self.dx, self.dqkv, self.dwq, self.dwk, self.de)]

    def reference(self):
        leaf = lambda t: t.double().requires_grad_(True)  # noqa: E731
        qkv, x, wq, wk, e = leaf(self.qkv), leaf(self.x), leaf(self.wq), leaf(self.wk), leaf(self.e)
        q, k, v = self.parts(qkv)
        ang = R.rope_angles(self.pos, self.axes)
        q = R.rope_forward(q, wq, self.H, ang, "interleaved", "width", 1.0)
        k = R.rope_forward(k, wk, self.Hk, ang, "interleaved", "width", 1.0)
        cu = R.cu_of(self.lens)
        o = R.attention(q, k, v, self.H, self.Hk, cu, cu, self.act, block=self.causal)["o"][0]
        m, xs, hs = e + self.mb.double(), [], []
        for i in range(len(self.lens)):
            s = slice(cu[i], cu[i + 1])
            if s.stop > s.start:
                xs.append(x[s] + R.residual_branch(o[s], m[i], 2, "rms", None))
                hs.append(R.residual_norm_out(xs[-1], m[i], 1, "layer", None, None))
        x2, h = torch.cat(xs), torch.cat(hs)
        loss = (h * self.dh.double()).sum() + (x2 * self.up.double()).sum()
        dx, dqkv, dwq, dwk, de = torch.autograd.grad(loss, (x, qkv, wq, wk, e))
        return [t.detach() for t in (x2, h, dx, dqkv, dwq, dwk, de)]


@pytest.mark.parametrize("dtype,lens,H,Hk,causal", [("bf16", [300, 0, 77, 1], 4, 2, 0), ("bf16", [260, 130], 3, 1, 32),
                                                    ("f32", [100, 41], 4, 2, 0), ("f32", [64, 1, 30], 2, 2, 8)])
def test_step_and_its_gradient(wan, dtype, lens, H, Hk, causal):
    s = Step(wan, dtype, lens, H, Hk, 128 if dtype == "bf16" else 64, causal=causal)
    s.run()
    assert wan.device_status() == 0
    # The longest way (a gradient of q or k) passes 7 bf16 tensors (q, o, h's input, dy, dqr and
    # the operands p and ds): each rounds to within 2^-9 RMS (half a step is 2^-8 at most, 2^-9
    # RMS or less), and the norm of a softmax's difference, ds = p (dp - delta), loses at most a
    # factor 2 of relative accuracy: 2 sqrt(7) 2^-9 = 1.04e-2. fp32: the same with 2^-24 and sums
    # of a few hundred terms, well under 2e-6.
    bar = 1.04e-2 if dtype == "bf16" else 2e-6
    for name, got, ref in zip(("x", "h", "dx", "dqkv", "dw_q", "dw_k", "de"), s.results(), s.reference()):
        if name == "de":
            got, ref = got[:, 2:5], ref[:, 2:5]
        assert rms_err(got.double().cpu().numpy(), ref.cpu().numpy()) <= bar, name


def test_side_stream_capture_and_replay(wan):
    """A step captured on a side stream; replays follow inputs copied into its buffers. Two
    graphs share one workspace and are replayed in turn."""
    steps = [Step(wan, "bf16", lens, 4, 2, 128, seed=i, causal=c) for i, (lens, c) in enumerate([([500, 33], 0), ([256, 700], 64)])]
    steps[0].ws = steps[1].ws = max((s.ws for s in steps), key=lambda t: t.numel())
    want = []
    for s in steps:
        s.run()
        want.append(s.results())
    torch.cuda.synchronize()
    side, graphs = torch.cuda.Stream(), []
    with torch.cuda.stream(side):
        for s in steps:
            s.run()
        side.synchronize()
        for s in steps:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                s.run()
            graphs.append(g)
    for s in steps:
        for t in (s.x2, s.h, s.dx, s.dqkv, s.dwq, s.dwk):
            t.zero_()
    torch.cuda.synchronize()
    for _ in range(2):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for s, w in zip(steps, want):
        assert all(torch.equal(a, b) for a, b in zip(s.results(), w))
    s, other = steps[0], Step(wan, "bf16", [500, 33], 4, 2, 128, seed=9)
    other.run()
    for name in ("qkv", "x", "dh", "up", "e", "mb", "wq", "wk", "pos"):
        getattr(s, name).copy_(getattr(other, name))
    graphs[0].replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(s.results(), other.results()))
    assert wan.device_status() == 0


def test_two_streams_at_once(wan):
    steps = [Step(wan, "bf16", [900, 40], 4, 2, 128, seed=i) for i in range(2)]
    want = []
    for s in steps:
        s.run()
        want.append(s.results())
        for t in (s.x2, s.h, s.dx, s.dqkv, s.dwq, s.dwk):
            t.zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in steps]
    for _ in range(5):
        for s, st in zip(steps, streams):
            with torch.cuda.stream(st):
                s.run()
    torch.cuda.synchronize()
    for s, w in zip(steps, want):
        assert all(torch.equal(a, b) for a, b in zip(s.results(), w))


@pytest.mark.parametrize("H,Hk", [(132, 1), (200, 2)])
def test_more_query_heads_than_a_tile_has_rows(wan, H, Hk):
    """Groups of 132 and 100 heads: packs of 66 and 100, and of 44 and 50 in the keys' gradient."""
    d, n = 128, 70
    g = torch.Generator(device="cuda").manual_seed(1)
    q, do = (torch.randn(n, H * d, generator=g, device="cuda").bfloat16() for _ in range(2))
    k, v = (torch.randn(n, Hk * d, generator=g, device="cuda").bfloat16() for _ in range(2))
    cfg, docs = wan.make_config(H * d, H, 64), wan.documents(_i32([0, 3, n]), causal_block=1)
    o, lse = torch.empty_like(q), torch.empty(H, n, device="cuda")
    ws = torch.empty(wan.attention_packed_workspace_bytes(cfg, n, n, 2, Hk, True), dtype=torch.uint8, device="cuda")
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    wan.attention_packed_fwd(cfg, docs, q, k, v, o, lse, kv_heads=Hk, ws=ws)
    wan.attention_packed_bwd(cfg, docs, q, k, v, o, lse, do, dq, dk, dv, kv_heads=Hk, ws=ws)
    assert wan.device_status() == 0
    want = R.attention(q.double(), k.double(), v.double(), H, Hk, [0, 3, n], [0, 3, n], torch.bfloat16, do=do.double(), block=1)
    for name, t in (("o", o), ("lse", lse), ("dq", dq), ("dk", dk), ("dv", dv)):
        R.assert_close(t, *want[name], name)


@pytest.mark.parametrize("lens,H,Hk,causal", [([520] * 40 + [3, 0, 700], 64, 64, 0),   # more long documents than are walked in waves
                                              ([1, 3, 0, 2] * 175, 2, 1, 1)])         # hundreds of short ones
def test_many_documents(wan, lens, H, Hk, causal):
    d, n = 128, sum(lens)
    g = torch.Generator(device="cuda").manual_seed(5)
    q, k, v, do = (torch.randn(n, h * d, generator=g, device="cuda").bfloat16() for h in (H, Hk, Hk, H))
    cfg, docs, cu = wan.make_config(H * d, H, 64), wan.documents(_i32(R.cu_of(lens)), causal_block=causal), R.cu_of(lens)
    ws = torch.empty(wan.attention_packed_workspace_bytes(cfg, n, n, len(lens), Hk, True), dtype=torch.uint8, device="cuda")
    o, lse = torch.empty_like(q), torch.empty(H, n, device="cuda")
    want = R.attention(q.double(), k.double(), v.double(), H, Hk, cu, cu, torch.bfloat16,
                       do=do.double() if causal else None, block=causal)
    for w in (ws, None):
        o.fill_(7.0)
        wan.attention_packed_fwd(cfg, docs, q, k, v, o, lse, kv_heads=Hk, ws=w)
        assert wan.device_status() == 0
        R.assert_close(o, *want["o"], "o")
        R.assert_close(lse, *want["lse"], "lse")
    if causal:
        dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
        wan.attention_packed_bwd(cfg, docs, q, k, v, o, lse, do, dq, dk, dv, kv_heads=Hk, ws=ws)
        assert wan.device_status() == 0
        for name, t in (("dq", dq), ("dk", dk), ("dv", dv)):
            R.assert_close(t, *want[name], name)


def test_offsets_past_32_bits(wan):
    """A qkv tensor of more than 2^31 elements whose documents lie at its end."""
    H, d, n = 12, 128, 480000
    D = H * d
    qkv = torch.zeros(n, 3 * D, dtype=torch.bfloat16, device="cuda")
    assert qkv.numel() > 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(2)
    lens, first = [150, 90], n - 250
    tail = slice(first, first + sum(lens))
    qkv[tail] = torch.randn(sum(lens), 3 * D, generator=g, device="cuda").bfloat16()
    q, k, v = qkv[:, :D], qkv[:, D:2 * D], qkv[:, 2 * D:]
    cfg, cu = wan.make_config(D, H, 64), R.cu_of(lens, first)
    docs = wan.documents(_i32(cu))
    out = torch.zeros(n, 3 * D, dtype=torch.bfloat16, device="cuda")
    o, dq, dk = out[:, :D], out[:, D:2 * D], out[:, 2 * D:]
    lse, dv = torch.zeros(H, n, device="cuda"), torch.zeros(n, D, dtype=torch.bfloat16, device="cuda")
    do = torch.zeros(n, D, dtype=torch.bfloat16, device="cuda")
    do[tail] = torch.randn(sum(lens), D, generator=g, device="cuda").bfloat16()
    ws = torch.empty(wan.attention_packed_workspace_bytes(cfg, n, n, 2, H, True), dtype=torch.uint8, device="cuda")
    wan.attention_packed_fwd(cfg, docs, q, k, v, o, lse, ws=ws)
    wan.attention_packed_bwd(cfg, docs, q, k, v, o, lse, do, dq, dk, dv, ws=ws)
    assert wan.device_status() == 0
    small = R.cu_of(lens)
    want = R.attention(*(t[tail].double() for t in (q, k, v)), H, H, small, small, torch.bfloat16, do=do[tail].double())
    for name, t in (("o", o), ("dq", dq), ("dk", dk), ("dv", dv)):
        R.assert_close(t[tail], *want[name], name)
        assert not t[:first].any() and not t[first + sum(lens):].any()
    R.assert_close(lse[:, tail], *want["lse"], "lse")
    # the rotation in place, the last rows against those alone
    pos = torch.randint(0, 1000, (n, 1), generator=g, device="cuda", dtype=torch.int32)
    spec, w = wan.rope([d]), torch.ones(D, dtype=torch.bfloat16, device="cuda")
    alone = [t[tail].contiguous() for t in (q, k)]
    wan.qk_norm_rope_fwd(cfg, spec, pos[tail].contiguous(), *alone, *alone, norm="width", w_q=w, w_k=w)
    wan.qk_norm_rope_fwd(cfg, spec, pos, q, k, q, k, norm="width", w_q=w, w_k=w)
    assert torch.equal(q[tail], alone[0]) and torch.equal(k[tail], alone[1])


@pytest.mark.parametrize("bad", [[0, 90, 20, 60], [-7, 10, 30, 64], [0, 10, 30, 2 ** 31 - 1], [70, 80, 90, 100], [64, 0, 64, 0]])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_offsets_out_of_order_stay_inside(wan, bad, dtype):
    """Offsets are clamped into the tensor and into order: guard rows behind it stay as they
    were, and nothing faults."""
    n, H, d, act = 64, 2, 128 if dtype == "bf16" else 64, ACT[dtype]
    D, guard = H * d, 64
    cfg, cu = wan.make_config(D, H, 64, dtype=dtype), _i32(bad)
    full = lambda *s, t=act: torch.full(s, 7.0, dtype=t, device="cuda")  # noqa: E731
    g = torch.Generator(device="cuda").manual_seed(3)
    q, k, v, do = (torch.randn(n, D, generator=g, device="cuda").to(act) for _ in range(4))
    outs = [full(n + guard, D) for _ in range(4)]
    o, dq, dk, dv = (t[:n] for t in outs)
    lse = torch.zeros(H, n, device="cuda")
    ws = torch.empty(max(16, wan.attention_packed_workspace_bytes(cfg, n, n, 3, H, True)), dtype=torch.uint8, device="cuda")
    docs = wan.documents(cu, causal_block=4)
    wan.attention_packed_fwd(cfg, docs, q, k, v, o, lse, ws=ws)
    wan.attention_packed_bwd(cfg, docs, q, k, v, o, lse, do, dq, dk, dv, ws=ws)
    op = wan.residual_norm(pre="rms", gate=0)
    x, e = torch.randn(n, D, generator=g, device="cuda"), torch.randn(3, 6, D, generator=g, device="cuda")
    xs, hs = full(n + guard, D, t=torch.float32), full(n + guard, D)
    wan.gated_residual_norm_fwd(cfg, op, x, q, e, None, cu, xs[:n], hs[:n])
    dxs, dys, de = full(n + guard, D, t=torch.float32), full(n + guard, D), torch.zeros_like(e)
    ws2 = torch.empty(wan.gated_residual_norm_workspace_bytes(cfg, n, 3), dtype=torch.uint8, device="cuda")
    wan.gated_residual_norm_bwd(cfg, op, x, q, e, None, cu, do, None, dxs[:n], dys[:n], ws2, de=de)
    assert wan.device_status() == 0
    assert all((t[n:] == 7).all() for t in outs + [xs, hs, dxs, dys])


def test_binding_refuses(wan):
    cfg = wan.make_config(256, 2, 64)
    t = torch.zeros(8, 256, dtype=torch.bfloat16, device="cuda")
    cu, x = _i32([0, 8]), torch.zeros(8, 256, device="cuda")
    docs, spec, pos = wan.documents(cu), wan.rope([128]), torch.zeros(8, 1, dtype=torch.int32, device="cuda")
    n = wan.launch_count()
    for call in (
            lambda: wan.attention_packed_fwd(cfg, docs, t, t.float(), t, t),                       # type
            lambda: wan.attention_packed_fwd(cfg, docs, t, t[:, :128], t, t),                      # width
            lambda: wan.attention_packed_fwd(cfg, docs, t, t.t().contiguous().t()[:, :256], t, t),  # dense rows
            lambda: wan.attention_packed_fwd(cfg, wan.documents(cu.long()), t, t, t, t),
            lambda: wan.attention_packed_fwd(cfg, wan.documents(cu, _i32([0, 4, 8])), t, t, t, t),
            lambda: wan.attention_packed_fwd(cfg, wan.documents(cu, prefix=_i32([0, 0])), t, t, t, t),
            lambda: wan.attention_packed_fwd(cfg, docs, t, t, t, t, lse=x),
            lambda: wan.attention_packed_bwd(cfg, docs, t, t, t, t, None, t, t, t, t),
            lambda: wan.qk_norm_rope_fwd(cfg, spec, pos[:4], t, t, t, t),
            lambda: wan.qk_norm_rope_fwd(cfg, spec, pos, t, None, t, t),
            lambda: wan.qk_norm_rope_fwd(cfg, spec, pos, t, t, t, t, norm="head"),
            lambda: wan.qk_norm_rope_bwd(cfg, spec, pos, t, t, None, None, t, t, dw_q=x[0]),
            lambda: wan.gated_residual_norm_fwd(cfg, wan.residual_norm(gate=1), x, t, None, None, cu, x, t),
            lambda: wan.gated_residual_norm_fwd(cfg, wan.residual_norm(), x, t, None, None, cu, x[:4], t),
            lambda: wan.gated_residual_norm_fwd(cfg, wan.residual_norm(w_pre=x[0]), x, t, None, None, cu, x, t),
            lambda: wan.gated_residual_norm_bwd(cfg, wan.residual_norm(), x, t, None, None, cu, t, x, x, t, dw_post=x[0])):
        with pytest.raises(ValueError):
            call()
    for status, call in (
            (-4, lambda: wan.attention_packed_fwd(cfg, docs, torch.zeros(8, 260, dtype=torch.bfloat16, device="cuda")[:, :256], t, t, t)),
            (-5, lambda: wan.attention_packed_fwd(cfg, docs, t, t, t, t, ws=torch.zeros(64, dtype=torch.uint8, device="cuda"))),
            (-1, lambda: wan.attention_packed_bwd(cfg, docs, t, t, t, t, torch.zeros(2, 8, device="cuda"), t, t, t, t)),
            (-2, lambda: wan.attention_packed_fwd(cfg, docs, t, t.expand(8, 256)[:1].expand(8, 256), t, t))):
        with pytest.raises(wan.WanError) as err:
            call()
        assert err.value.status == status
    assert wan.launch_count() == n
