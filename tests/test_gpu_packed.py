"""Packed-document operators on the GPU against their 64-bit forms (packed_ref)."""
import math

import pytest

import packed_ref as R

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ACT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def wan():
    import video_diffusion_transformer_wan_b200 as w
    return w


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, *shape, scale=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _sevens(*shape, dtype):
    return torch.full(shape, 7.0, dtype=dtype, device="cuda")


# ------------------------------------------------------------------ rotary positions
ROPE = [
    # rows, heads, kv_heads, d, axes, options, layout, norm
    (1, 2, 2, 64, [64], {}, "interleaved", "none"),
    (5, 3, 1, 64, [20, 22, 22], {}, "half", "head"),
    (77, 12, 12, 128, [44, 42, 42], {}, "interleaved", "width"),
    (301, 12, 4, 128, [96], dict(scaling="ramp", factor=[8.0], orig_len=[131072]), "half", "head"),
    (2000, 6, 2, 128, [64, 32, 32], dict(scaling="linear", factor=[2.0, 4.0, 1.0]), "half", "width"),
    (33, 40, 40, 128, [128], dict(scaling="base", factor=[4.0], theta=1e6), "interleaved", "width"),
    (700, 1, 1, 64, [8, 8, 8], dict(theta=256.0), "half", "none"),
    (19, 4, 2, 32, [6, 10], {}, "half", "head"),       # quads do not divide the halves
    (40, 64, 32, 2, [2], {}, "interleaved", "width"),  # one pair a head
    (13, 7, 7, 64, [10], {}, "half", "width"),
    (50, 20, 20, 128, [128], {}, "half", "width"),     # 2560 columns a side
    (21, 48, 48, 128, [64, 64], {}, "interleaved", "width"),
]


def _rope_case(wan, case, dtype, seed=0):
    rows, H, Hk, d, axes, opt, layout, norm = case
    act = ACT[dtype]
    g = _gen(seed + rows + H)
    cfg = wan.make_config(H * d, H, 64, dtype=dtype)
    amp = 1.25 if opt else 1.0
    spec = wan.rope(axes, layout=layout, amplitude=amp, **opt)
    pos = torch.randint(-1000, 2000000, (rows, len(axes)), generator=g, device="cuda", dtype=torch.int32)
    qkv = _normal(g, rows, (H + 2 * Hk) * d + 4, dtype=act)  # 4 spare columns: rows of 8 bytes' alignment
    q, k = qkv[:, :H * d], qkv[:, H * d:(H + Hk) * d]
    w_q = w_k = None
    if norm != "none":
        w_q = _normal(g, d if norm == "head" else H * d, scale=0.2, dtype=act) + 1
        w_k = _normal(g, d if norm == "head" else Hk * d, scale=0.2, dtype=act) + 1
    angles = R.rope_angles(pos, axes, **opt)
    return cfg, spec, pos, q, k, w_q, w_k, angles, amp


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", ROPE, ids=lambda c: f"{c[0]}x{c[1]}_{c[2]}x{c[3]}_{c[6]}_{c[7]}")
@pytest.mark.parametrize("aligned", [True, False])
def test_rope_forward(wan, case, dtype, aligned):
    rows, H, Hk, d, axes, opt, layout, norm = case
    cfg, spec, pos, q, k, w_q, w_k, angles, amp = _rope_case(wan, case, dtype)
    act = ACT[dtype]
    if aligned:
        q, k = q.contiguous(), k.contiguous()
    elif H * d * q.element_size() % 16:
        pytest.skip("k would start off a 16-byte boundary: refused, see the host test")
    qo, ko = _sevens(rows, H * d, dtype=act), _sevens(rows, Hk * d, dtype=act)
    wan.qk_norm_rope_fwd(cfg, spec, pos, q, k, qo, ko, kv_heads=Hk, norm=norm, w_q=w_q, w_k=w_k)
    qi, ki = q.clone(), k.clone()  # in place; the clones' rows are dense, so the access widths may differ
    wan.qk_norm_rope_fwd(cfg, spec, pos, qi, ki, qi, ki, kv_heads=Hk, norm=norm, w_q=w_q, w_k=w_k)
    for x, w, heads, outs in ((q, w_q, H, (qo, qi)), (k, w_k, Hk, (ko, ki))):
        ref = R.rope_forward(x.double(), None if w is None else w.double(), heads, angles, layout, norm, amp)
        # one rounding of the output; fp32 before it: the sine and cosine (an angle reduced in 64
        # bits, 2^-22 absolute), the norm's mean (a sum of at most heads*d terms, relative
        # error (log2 + 4) 2^-24 of a positive sum) and four products, each 2^-24 of the parts
        size = R.rope_forward(x.double(), None if w is None else w.double().abs(), heads, torch.zeros_like(angles), layout, norm, abs(amp)).abs()
        pair = size.reshape(rows, -1).amax(1, keepdim=True)  # the larger of a pair's parts is at most this
        for out in outs:
            R.assert_close(out, ref, R.U[act] * ref.abs() + 2.0 ** -20 * pair, "out")
    if aligned:
        assert torch.equal(qi, qo) and torch.equal(ki, ko)
    only = _sevens(rows, H * d, dtype=act)
    wan.qk_norm_rope_fwd(cfg, spec, pos, q, None, only, None, norm=norm, w_q=w_q)
    assert torch.equal(only, qo)
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", ROPE, ids=lambda c: f"{c[0]}x{c[1]}_{c[2]}x{c[3]}_{c[6]}_{c[7]}")
def test_rope_gradient(wan, case, dtype):
    rows, H, Hk, d, axes, opt, layout, norm = case
    cfg, spec, pos, q, k, w_q, w_k, angles, amp = _rope_case(wan, case, dtype, seed=5)
    act, g = ACT[dtype], _gen(9)
    q, k = q.contiguous(), k.contiguous()
    gq, gk = _normal(g, rows, H * d, dtype=act), _normal(g, rows, Hk * d, dtype=act)
    dq, dk = _sevens(rows, H * d, dtype=act), _sevens(rows, Hk * d, dtype=act)
    dw = [None, None] if norm == "none" else [_sevens(*w.shape, dtype=torch.float32) for w in (w_q, w_k)]
    n = wan.qk_norm_rope_workspace_bytes(cfg, rows, Hk, norm)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda") if n else None
    wan.qk_norm_rope_bwd(cfg, spec, pos, gq, gk, q, k, dq, dk, kv_heads=Hk, norm=norm, w_q=w_q, w_k=w_k, dw_q=dw[0],
                         dw_k=dw[1], ws=ws)
    for x, w, heads, go, dx, dwx in ((q, w_q, H, gq, dq, dw[0]), (k, w_k, Hk, gk, dk, dw[1])):
        x64 = x.double().requires_grad_(True)
        w64 = None if w is None else w.double().requires_grad_(True)
        out = R.rope_forward(x64, w64, heads, angles, layout, norm, amp)
        grads = torch.autograd.grad(out, [t for t in (x64, w64) if t is not None], go.double())
        # every part of a row's gradient is bounded by the row's largest |g w| r (and the term
        # x r^2 mean(g w x) r, no larger by Cauchy-Schwarz than that times sqrt(width))
        row = go.double().abs().amax(1, keepdim=True) * abs(amp) * 2
        if norm != "none":
            ms = (x64.detach().reshape(rows, heads, d) ** 2).mean(2 if norm == "head" else (1, 2), keepdim=True)
            r = 1 / torch.sqrt(ms + 1e-6)
            r = r.expand(rows, heads, 1).amax(1)
            row = row * w64.detach().abs().max() * r * (1 + x64.detach().abs().amax(1, keepdim=True) * r)
        R.assert_close(dx, grads[0], R.U[act] * grads[0].abs() + 2.0 ** -19 * row, "dx")
        if w is not None:
            # a sum of `count` fp32 terms, in partial sums: relative error of the terms (2^-19 of
            # the row's size) and at most `count` 2^-24 of their absolute sum
            xh = x64.detach().abs() * r.reshape(rows, 1)
            terms = (go.double().abs().amax(1, keepdim=True) * abs(amp) * 2 * xh).reshape(rows, heads, d)
            size = terms.sum((0, 1)) if norm == "head" else terms.sum(0).reshape(-1)
            count = rows * (heads if norm == "head" else 1)
            R.assert_close(dwx, grads[1], size * (2.0 ** -19 + min(count, 4096) * R.F), "dw")
    # a difference of the 64-bit form along a random direction agrees with the gradient
    v = _normal(g, rows, H * d).double()
    step = 1e-5
    f = lambda s: (R.rope_forward(q.double() + s * v, None if w_q is None else w_q.double(), H, angles, layout, norm, amp)  # noqa: E731
                   * gq.double()).sum()
    slope, got = (f(step) - f(-step)) / (2 * step), (dq.double() * v).sum()
    err = (R.U[act] * dq.double().abs() + 2.0 ** -19 * dq.double().abs().max()) * v.abs()
    assert abs(slope - got) <= 4 * err.sum() + 1e-4
    first = (dq.clone(), dk.clone(), [None if t is None else t.clone() for t in dw])
    wan.qk_norm_rope_bwd(cfg, spec, pos, gq, gk, q, k, gq, gk, kv_heads=Hk, norm=norm, w_q=w_q, w_k=w_k, dw_q=dw[0],
                         dw_k=dw[1], ws=ws)  # in place, and the same from run to run
    assert torch.equal(gq, first[0]) and torch.equal(gk, first[1])
    for a, b in zip(dw, first[2]):
        assert a is None or torch.equal(a, b)


def test_rope_no_rows(wan):
    cfg = wan.make_config(128, 2, 64, dtype="bf16")
    spec = wan.rope([64])
    z = torch.empty(0, 128, dtype=torch.bfloat16, device="cuda")
    pos = torch.empty(0, 1, dtype=torch.int32, device="cuda")
    wan.qk_norm_rope_fwd(cfg, spec, pos, z, z, z, z)
    w = torch.ones(128, dtype=torch.bfloat16, device="cuda")
    dw = _sevens(128, dtype=torch.float32)
    wan.qk_norm_rope_bwd(cfg, spec, pos, z, z, z, z, z, z, norm="width", w_q=w, w_k=w, dw_q=dw)
    assert (dw == 0).all()


# ------------------------------------------------------------------ gated residual and norms
RESNORM = [
    # lens, D, first row, spare rows, options
    ([1], 64, 0, 0, dict(pre="rms")),
    ([5, 0, 1, 9], 128, 2, 3, dict(pre="layer", post="rms", gate=2, chunk=1, weights=True)),
    ([700, 33, 1], 1536, 0, 7, dict(pre="layer", post="none", gate=5, chunk=0, residual_scale=0.7)),
    ([64, 200], 5120, 0, 1, dict(pre="layer", post="rms", gate=2, chunk=1, weights=True)),
    ([3, 80], 8192, 0, 0, dict(pre="rms", post="layer", gate=-1, chunk=0, weights=True)),
    ([2000, 1500, 0], 320, 5, 5, dict(pre="rms", post="layer", gate=1, chunk=-1, weights=True, residual_scale=-0.5)),
    ([40] * 50 + [0] * 20, 512, 0, 0, dict(pre="layer", post="rms", gate=0, chunk=1)),
    ([0, 0], 64, 0, 4, dict(pre="layer", gate=2, chunk=1, weights=True)),
    ([17], 2048, 0, 0, dict(pre="layer", post="layer", gate=-1, chunk=-1, weights=True)),
]


def _resnorm_case(wan, case, dtype, seed=0):
    lens, D, first, spare, opt = case
    opt = dict(opt)
    weights = opt.pop("weights", False)
    g, act = _gen(seed + D), ACT[dtype]
    rows = first + sum(lens) + spare
    x, y = _normal(g, rows, D) + 0.3, _normal(g, rows, D, dtype=act)
    for t in (x, y):  # rows of no document are not used
        t[:first], t[first + sum(lens):] = math.nan, math.nan
    e, mb = _normal(g, len(lens), 6, D, scale=0.3), _normal(g, 6, D, scale=0.1)
    w = [None, None, None]
    if weights:
        w = [_normal(g, D, scale=0.1, dtype=act) + 1, _normal(g, D, scale=0.1, dtype=act),
             _normal(g, D, scale=0.1, dtype=act) + 1 if opt.get("post", "none") != "none" else None]
    cfg = wan.make_config(D, D // 64, 64, dtype=dtype)
    spec = wan.residual_norm(w_pre=w[0], b_pre=w[1], w_post=w[2], **opt)
    full = dict(pre="layer", post="none", gate=-1, chunk=-1, residual_scale=1.0)
    full.update(opt)
    return cfg, spec, full, rows, R.cu_of(lens, first), x, y, e, mb, w


def _resnorm_size(x, y, m, o, w):
    """Sizes that bound the parts of h and of the branch, row by row."""
    b = R._norm(y, o["post"]).abs().amax(1, keepdim=True)
    if w[2] is not None:
        b = b * w[2].double().abs().max()
    if o["gate"] >= 0:
        b = b * m[o["gate"]].abs().max()
    return b


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", RESNORM, ids=lambda c: f"{sum(c[0])}x{c[1]}")
def test_residual_norm_forward(wan, case, dtype):
    cfg, spec, o, rows, cu, x, y, e, mb, w = _resnorm_case(wan, case, dtype)
    act, D = ACT[dtype], x.shape[1]
    xo, ho = _sevens(rows, D, dtype=torch.float32), _sevens(rows, D, dtype=act)
    wan.gated_residual_norm_fwd(cfg, spec, x, y, e, mb, _i32(cu), xo, ho)
    new = lambda: torch.full((rows, D), math.nan, dtype=torch.float64, device="cuda")  # noqa: E731
    vx, tx, vh, th = new(), new(), new(), new()
    d64 = lambda t: None if t is None else t.double()  # noqa: E731
    for i in range(len(cu) - 1):
        s = slice(cu[i], cu[i + 1])
        if s.stop == s.start:
            continue
        m = e[i].double() + mb.double()
        branch = R.residual_branch(y[s].double(), m, o["gate"], o["post"], d64(w[2]))
        vx[s] = o["residual_scale"] * x[s].double() + branch
        # fp32: the norm's statistics (relative (log2 D + 8) 2^-24) and five products
        tx[s] = 2.0 ** -23 * vx[s].abs() + 2.0 ** -19 * _resnorm_size(x[s].double(), y[s].double(), m, o, w)
        vh[s] = R.residual_norm_out(vx[s], m, o["chunk"], o["pre"], d64(w[0]), d64(w[1]))
        # h from an x' off by tx: its norm moves by at most 2 max(tx) r, r = |h/x'|-like scale
        c = vx[s] - vx[s].mean(1, keepdim=True) if o["pre"] == "layer" else vx[s]
        r = 1 / torch.sqrt((c * c).mean(1, keepdim=True) + 1e-6)
        scale = (w[0].double().abs().max() if w[0] is not None else 1.0) * ((1 + m[3 * o["chunk"] + 1]).abs().max() if o["chunk"] >= 0 else 1.0)
        big = (c.abs().amax(1, keepdim=True) + vx[s].abs().amax(1, keepdim=True)) * r
        th[s] = R.U[act] * vh[s].abs() + scale * (3 * r * tx[s].amax(1, keepdim=True) * (1 + big) + 2.0 ** -20 * big) + 2.0 ** -22 * (1 + vh[s].abs())
    R.assert_close(xo, vx, tx, "x")
    R.assert_close(ho, vh, th, "h")
    x2, y2 = x.clone(), y.clone()
    wan.gated_residual_norm_fwd(cfg, spec, x2, y2, e, mb, _i32(cu), x2, y2)  # in place
    s = slice(cu[0], cu[-1])
    assert torch.equal(x2[s], xo[s]) and torch.equal(y2[s], ho[s])
    assert torch.isnan(x2[:cu[0]]).all() and torch.isnan(y2[cu[-1]:]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", RESNORM, ids=lambda c: f"{sum(c[0])}x{c[1]}")
@pytest.mark.parametrize("upstream", [True, False])
def test_residual_norm_gradient(wan, case, dtype, upstream):
    cfg, spec, o, rows, cu, xo, y, e, mb, w = _resnorm_case(wan, case, dtype, seed=3)
    act, D, g = ACT[dtype], xo.shape[1], _gen(17)
    dh = _normal(g, rows, D, dtype=act)
    up = _normal(g, rows, D) if upstream else None
    n = len(cu) - 1
    used = sorted({v for v in ([o["gate"]] if o["gate"] >= 0 else []) + ([3 * o["chunk"], 3 * o["chunk"] + 1] if o["chunk"] >= 0 else [])})
    out = dict(de=_sevens(n, 6, D, dtype=torch.float32), dmod_bias=_sevens(6, D, dtype=torch.float32),
               dw_pre=_sevens(D, dtype=torch.float32), db_pre=_sevens(D, dtype=torch.float32))
    if o["post"] != "none":
        out["dw_post"] = _sevens(D, dtype=torch.float32)
    dx, dy = _sevens(rows, D, dtype=torch.float32), _sevens(rows, D, dtype=act)
    ws = torch.empty(wan.gated_residual_norm_workspace_bytes(cfg, rows, n), dtype=torch.uint8, device="cuda")
    args = (cfg, spec, xo, y, e, mb, _i32(cu), dh, up)
    wan.gated_residual_norm_bwd(*args, dx, dy, ws, **out)
    ones = torch.ones(D, dtype=torch.float64, device="cuda")
    leaves = dict(e=e.double(), dmod_bias=mb.double(), dw_pre=ones if w[0] is None else w[0].double(),
                  db_pre=0 * ones if w[1] is None else w[1].double(), dw_post=ones if w[2] is None else w[2].double())
    leaves = {k: v.clone().requires_grad_(True) for k, v in leaves.items()}
    sums = {k: torch.zeros_like(v) for k, v in leaves.items()}
    size = {k: torch.zeros_like(v) for k, v in leaves.items()}
    new = lambda: torch.full((rows, D), math.nan, dtype=torch.float64, device="cuda")  # noqa: E731
    vx, tx, vy, ty = new(), new(), new(), new()
    for i in range(n):
        s = slice(cu[i], cu[i + 1])
        if s.stop == s.start:
            continue
        X, Y = xo[s].double().requires_grad_(True), y[s].double().requires_grad_(True)
        m = leaves["e"][i] + leaves["dmod_bias"]
        h = R.residual_norm_out(X, m, o["chunk"], o["pre"], leaves["dw_pre"], leaves["db_pre"])
        branch = R.residual_branch(Y, m, o["gate"], o["post"], leaves["dw_post"])
        G = torch.autograd.grad(h, X, dh[s].double(), retain_graph=True)[0]
        if up is not None:
            G = G + up[s].double()
        names = list(leaves)
        ga = torch.autograd.grad(h, [leaves[k] for k in names], dh[s].double(), allow_unused=True, retain_graph=True)
        gb = torch.autograd.grad(branch, [leaves[k] for k in names] + [Y], G, allow_unused=True, retain_graph=True)
        vx[s], vy[s] = o["residual_scale"] * G, gb[-1]
        # sizes: |dn| r and its projections; fp32 statistics and about ten products, 2^-19 of them
        c = X.detach() - X.detach().mean(1, keepdim=True) if o["pre"] == "layer" else X.detach()
        r = 1 / torch.sqrt((c * c).mean(1, keepdim=True) + 1e-6)
        nh = (c * r).abs().amax(1, keepdim=True)
        sc = leaves["dw_pre"].detach().abs().max() * ((1 + m[3 * o["chunk"] + 1]).abs().max().detach() if o["chunk"] >= 0 else 1.0)
        gsz = (0 if up is None else up[s].double().abs().amax(1, keepdim=True)) + r * sc * dh[s].double().abs().amax(1, keepdim=True) * (2 + nh)
        tx[s] = 2.0 ** -23 * vx[s].abs() + 2.0 ** -19 * gsz * abs(o["residual_scale"])
        yn = R._norm(Y.detach(), o["post"])
        ynm = yn.abs().amax(1, keepdim=True)
        gg = gsz * leaves["dw_post"].detach().abs().max() * (m[o["gate"]].abs().max().detach() if o["gate"] >= 0 else 1.0)
        ry = 1.0
        if o["post"] != "none":
            yc = Y.detach() - Y.detach().mean(1, keepdim=True) if o["post"] == "layer" else Y.detach()
            ry = 1 / torch.sqrt((yc * yc).mean(1, keepdim=True) + 1e-6) * (2 + ynm)
        ty[s] = R.U[act] * vy[s].abs() + 2.0 ** -18 * gg * ry
        for j, k in enumerate(names):
            for part in (ga[j], gb[j]):
                if part is not None:
                    sums[k] += part
        # every summand of these sums is at most one of these
        hb = (dh[s].double().abs() * (1 + nh) * (1 + sc)).sum(0)
        gb_ = (gsz * (1 + ynm) * (1 + leaves["dw_post"].detach().abs().max()) * (1 + (m[o["gate"]].abs().max().detach() if o["gate"] >= 0 else 0.0))).sum()
        both = hb + gb_
        for k in names:
            if k == "e":
                size[k][i] += both
            else:
                size[k] += both
    R.assert_close(dx, vx, tx, "dx")
    R.assert_close(dy, vy, ty, "dy")
    # fp32 sums: 2^-19 of the summands' sizes, and partial sums of at most 4096 terms
    rel = 2.0 ** -19 + min(max(sum(case[0]), 1), 4096) * R.F
    for k, t in (("dw_pre", out["dw_pre"]), ("db_pre", out["db_pre"]), ("dw_post", out.get("dw_post"))):
        if t is not None:
            R.assert_close(t, sums[k], rel * size[k], k)
    for row in range(6):
        if row in used:
            R.assert_close(out["de"][:, row], sums["e"][:, row], rel * size["e"][:, row], f"de[{row}]")
            R.assert_close(out["dmod_bias"][row], sums["dmod_bias"][row], rel * size["dmod_bias"][row], f"dmod_bias[{row}]")
        else:
            assert (out["de"][:, row] == 7).all() and (out["dmod_bias"][row] == 7).all()
    # without the sums, in place over its inputs, and the same from run to run
    up2, dh2 = (up.clone() if up is not None else torch.empty(rows, D, device="cuda")), dh.clone()
    wan.gated_residual_norm_bwd(*args[:-2], dh2, up2 if up is not None else None, up2, dh2)
    s = slice(cu[0], cu[-1])
    assert torch.equal(up2[s], dx[s]) and torch.equal(dh2[s], dy[s])
    again = {k: _sevens(*v.shape, dtype=v.dtype) for k, v in out.items()}
    wan.gated_residual_norm_bwd(*args, dx, dy, ws, **again)
    assert all(torch.equal(again[k], out[k]) for k in out)


# ------------------------------------------------------------------ attention in documents
ATTN = [
    # q_lens, k_lens, H, Hk, first row, spare rows, options
    ([1], [1], 1, 1, 0, 0, {}),
    ([3], [0], 2, 1, 0, 0, {}),
    ([128], [128], 2, 2, 0, 0, {}),
    ([129], [257], 2, 1, 0, 1, {}),
    ([256, 0, 1, 300], [256, 5, 128, 77], 3, 1, 4, 9, {}),
    ([500, 33], [500, 33], 4, 2, 0, 3, dict(block=1)),
    ([300, 45, 1], [300, 45, 1], 2, 1, 0, 0, dict(block=1, prefix=[20, 0, 0], cap=20.0)),
    ([600, 200], [600, 200], 6, 2, 1, 2, dict(block=150, prefix=[150, 70], cap=30.0, slopes=True)),
    ([40, 70], [20, 300], 5, 1, 0, 0, dict(block=16)),             # more queries than keys: rows that see nothing
    ([40], [20], 2, 2, 0, 0, dict(block=7, prefix=[3], slopes=True)),
    ([1] * 7, [700, 1, 128, 0, 1000, 64, 129], 12, 4, 0, 0, dict(block=1)),
    ([2, 1, 5], [3000, 2049, 513], 12, 1, 0, 5, dict(block=1, slopes=True)),
    ([1], [9000], 4, 4, 0, 0, dict(cap=5.0)),
    ([700], [40], 3, 3, 0, 0, dict(scale=1.0)),                    # sharp scores
    ([5] * 40, [9] * 40, 2, 1, 0, 0, dict(block=2, slopes=True)),  # more documents than a warp
    ([260], [260], 24, 1, 0, 0, dict(block=64)),                   # a large group
]


def _attn_case(wan, case, dtype, seed=0, big=1.0):
    q_lens, k_lens, H, Hk, first, spare, opt = case
    d, act, g = (128 if dtype == "bf16" else 64), ACT[dtype], _gen(seed + sum(q_lens) + H)
    nq, nk = first + sum(q_lens) + spare, first + sum(k_lens) + spare
    q = _normal(g, nq, H * d, dtype=act, scale=big)
    kv = _normal(g, nk, 2 * Hk * d, dtype=act)
    do = _normal(g, nq, H * d, dtype=act)
    for t, n in ((q, sum(q_lens)), (kv, sum(k_lens)), (do, sum(q_lens))):
        t[:first], t[first + n:] = math.nan, math.nan  # rows of no document are not used
    opt = dict(opt)
    slopes = torch.tensor([2.0 ** (-8.0 * (h + 1) / H) for h in range(H)], device="cuda") if opt.pop("slopes", False) else None
    prefix = opt.pop("prefix", None)
    cu_q, cu_k = R.cu_of(q_lens, first), R.cu_of(k_lens, first)
    docs = wan.documents(_i32(cu_q), _i32(cu_k), prefix=None if prefix is None else _i32(prefix),
                         causal_block=opt.get("block", 0), cap=opt.get("cap", 0.0), slopes=slopes,
                         scale=opt.get("scale", 0.0))
    cfg = wan.make_config(H * d, H, 64, dtype=dtype)
    ref = lambda grads: R.attention(q.double(), kv[:, :Hk * d].double(), kv[:, Hk * d:].double(), H, Hk, cu_q, cu_k, act,  # noqa: E731
                                    do=do.double() if grads else None, prefix=prefix,
                                    slopes=None if slopes is None else [float(s) for s in slopes], **opt)
    return cfg, docs, q, kv[:, :Hk * d], kv[:, Hk * d:], do, ref, H, Hk, d


def _attn_ws(wan, cfg, q, k, docs, Hk, backward):
    n = wan.attention_packed_workspace_bytes(cfg, q.shape[0], k.shape[0], docs.n_docs, Hk, backward)
    return torch.empty(n, dtype=torch.uint8, device="cuda") if n else None


def _status(wan):
    assert wan.device_status() == 0


_attn_id = lambda c: f"{sum(c[0])}x{sum(c[1])}x{len(c[0])}_{c[2]}_{c[3]}"  # noqa: E731


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", ATTN, ids=_attn_id)
def test_attention_forward(wan, case, dtype):
    cfg, docs, q, k, v, do, ref, H, Hk, d = _attn_case(wan, case, dtype)
    want = ref(False)
    for ws in (None, _attn_ws(wan, cfg, q, k, docs, Hk, False)):
        o, lse = _sevens(*q.shape, dtype=q.dtype), _sevens(H, q.shape[0], dtype=torch.float32)
        wan.attention_packed_fwd(cfg, docs, q, k, v, o, lse, kv_heads=Hk, ws=ws)
        _status(wan)
        R.assert_close(o, *want["o"], "o")
        R.assert_close(lse, *want["lse"], "lse")
        o2 = _sevens(*q.shape, dtype=q.dtype)
        wan.attention_packed_fwd(cfg, docs, q, k, v, o2, None, kv_heads=Hk, ws=ws)
        assert torch.equal(o2, o)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", ATTN, ids=_attn_id)
def test_attention_gradient(wan, case, dtype):
    cfg, docs, q, k, v, do, ref, H, Hk, d = _attn_case(wan, case, dtype, seed=1)
    want = ref(True)
    o, lse = _sevens(*q.shape, dtype=q.dtype), _sevens(H, q.shape[0], dtype=torch.float32)
    wan.attention_packed_fwd(cfg, docs, q, k, v, o, lse, kv_heads=Hk)
    ws = _attn_ws(wan, cfg, q, k, docs, Hk, True)
    got = None
    for _ in range(2):
        new = [_sevens(*t.shape, dtype=q.dtype) for t in (q, k, v)]
        wan.attention_packed_bwd(cfg, docs, q, k, v, o, lse, do, *new, kv_heads=Hk, ws=ws)
        _status(wan)
        assert got is None or all(torch.equal(a, b) for a, b in zip(got, new))  # the same from run to run
        got = new
    for name, t in zip(("dq", "dk", "dv"), got):
        R.assert_close(t, *want[name], name)


def test_attention_large_scores(wan):
    """Scores whose running maximum grows tile by tile: the rescaling path."""
    case = ([200], [2000], 2, 2, 0, 0, {})
    cfg, docs, q, k, v, do, ref, H, Hk, d = _attn_case(wan, case, "bf16", big=6.0)
    k.copy_((k.float() * torch.linspace(0.1, 4.0, 2000, device="cuda")[:, None]).to(k.dtype))
    o, lse = _sevens(*q.shape, dtype=q.dtype), _sevens(H, 200, dtype=torch.float32)
    wan.attention_packed_fwd(cfg, docs, q, k, v, o, lse, kv_heads=Hk)
    _status(wan)
    want = ref(False)
    R.assert_close(o, *want["o"], "o")
    R.assert_close(lse, *want["lse"], "lse")


def test_attention_gradient_differences(wan):
    """The fp32 gradient against differences of the 64-bit forward along random directions."""
    case = ([60, 9], [70, 9], 4, 2, 0, 0, dict(block=4, prefix=[5, 2], cap=8.0, slopes=True))
    cfg, docs, q, k, v, do, ref, H, Hk, d = _attn_case(wan, case, "f32")
    o, lse = torch.empty_like(q), torch.empty(H, q.shape[0], device="cuda")
    wan.attention_packed_fwd(cfg, docs, q, k, v, o, lse, kv_heads=Hk)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k, memory_format=torch.contiguous_format), torch.empty(k.shape, device="cuda")
    wan.attention_packed_bwd(cfg, docs, q, k, v, o, lse, do, dq, dk, dv, kv_heads=Hk, ws=_attn_ws(wan, cfg, q, k, docs, Hk, True))
    g = _gen(4)
    cu_q, cu_k = [int(x) for x in docs.tensors[0]], [int(x) for x in docs.tensors[1]]
    opt = dict(block=4, prefix=[5, 2], cap=8.0, slopes=[float(s) for s in docs.tensors[3]])
    base = [t.double() for t in (q, k, v)]
    for which, grad in enumerate((dq, dk, dv)):
        way = torch.randn(*grad.shape, generator=g, device="cuda").double()

        def f(step):
            x = list(base)
            x[which] = x[which] + step * way
            return (R.attention(*x, H, Hk, cu_q, cu_k, torch.float32, **opt)["o"][0] * do.double()).sum()

        slope = (f(1e-5) - f(-1e-5)) / 2e-5
        # the difference's own error is about step^2 and 1e-16 / step; the gradient's is fp32
        assert abs(float(slope - (grad.double() * way).sum())) <= 1e-5 * float((grad.double() * way).abs().sum()) + 1e-6
