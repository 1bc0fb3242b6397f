"""Packed-document operators at their edges: what neighbours and unused rows hold, empty
documents and batches, head dims and scales other than the usual ones, cut units of every kind."""
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


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _attention(wan, cfg, docs, q, k, v, Hk, do=None, split=True):
    """o, lse (and dq, dk, dv) of one call; rows that are not written hold 7."""
    H, n = cfg.heads, docs.n_docs
    size = wan.attention_packed_workspace_bytes(cfg, q.shape[0], k.shape[0], n, Hk, do is not None)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda") if size else None
    full = lambda t: torch.full(t.shape, 7.0, dtype=t.dtype, device="cuda")  # noqa: E731
    out = dict(o=full(q), lse=torch.full((H, q.shape[0]), 7.0, device="cuda"))
    wan.attention_packed_fwd(cfg, docs, q, k, v, out["o"], out["lse"], kv_heads=Hk, ws=ws if split else None)
    if do is not None:
        out.update(dq=full(q), dk=full(k), dv=full(v))
        wan.attention_packed_bwd(cfg, docs, q, k, v, out["o"], out["lse"], do, out["dq"], out["dk"], out["dv"],
                                 kv_heads=Hk, ws=ws)
    assert wan.device_status() == 0
    return out


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("block,slopes", [(0, False), (1, True)])
def test_neighbours_do_not_reach_a_document(wan, dtype, block, slopes):
    """The same document in front of neighbours of size 1 and of size 1e4 (and rows of no document
    alike): every bit of its results is the same, with capped scores too."""
    H, Hk, d, act, lens = 4, 2, 128 if dtype == "bf16" else 64, ACT[dtype], [70, 90]
    n = sum(lens) + 20
    cfg = wan.make_config(H * d, H, 64, dtype=dtype)
    docs = wan.documents(_i32(R.cu_of(lens)), causal_block=block, cap=15.0,
                         slopes=torch.tensor([0.5, 0.25, 0.125, 0.0625], device="cuda") if slopes else None)
    got = []
    for big in (1.0, 1e4):
        g = _gen(7)
        q, k, v, do = (torch.randn(n, h * d, generator=g, device="cuda") for h in (H, Hk, Hk, H))
        for t in (q, k, v, do):
            t[lens[0]:] *= big
        got.append(_attention(wan, cfg, docs, *(t.to(act) for t in (q, k, v)), Hk, do=do.to(act)))
    for name in got[0]:
        a, b = (t[name][:, :lens[0]] if name == "lse" else t[name][:lens[0]] for t in got)
        assert torch.equal(a, b), name


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_modulation_of_an_empty_document_is_not_used(wan, dtype, bad):
    """Unused slots of a batch of fixed size: whatever their modulation holds, no sum sees it."""
    lens, D, act = [3, 0, 5, 0], 128, ACT[dtype]
    n, g = sum(lens), _gen(2)
    rnd = lambda *s, t=torch.float32: torch.randn(*s, generator=g, device="cuda").to(t)  # noqa: E731
    cfg = wan.make_config(D, 2, 64, dtype=dtype)
    w = [rnd(D, t=act) for _ in range(3)]
    spec = wan.residual_norm(pre="layer", post="rms", gate=2, chunk=1, w_pre=w[0], b_pre=w[1], w_post=w[2])
    x, y, e, mb, dh, up = rnd(n, D), rnd(n, D, t=act), rnd(4, 6, D), rnd(6, D), rnd(n, D, t=act), rnd(n, D)
    ws = torch.empty(wan.gated_residual_norm_workspace_bytes(cfg, n, 4), dtype=torch.uint8, device="cuda")
    got = []
    for fill in (0.0, bad):
        e[1], e[3] = fill, fill
        sums = dict(de=torch.zeros(4, 6, D, device="cuda"), dmod_bias=torch.zeros(6, D, device="cuda"),
                    **{k: torch.empty(D, device="cuda") for k in ("dw_pre", "db_pre", "dw_post")})
        dx, dy = torch.empty(n, D, device="cuda"), torch.empty(n, D, dtype=act, device="cuda")
        wan.gated_residual_norm_bwd(cfg, spec, x, y, e, mb, _i32(R.cu_of(lens)), dh, up, dx, dy, ws, **sums)
        got.append(dict(dx=dx, dy=dy, **sums))
    for name in got[0]:
        assert torch.isfinite(got[1][name]).all() and torch.equal(got[0][name], got[1][name]), name
    assert not got[1]["de"][1].any() and not got[1]["de"][3].any()


def test_gradient_with_warps_of_uneven_pace(wan):
    """One query (one warp of scores has work, the others none) over many key tiles, scores on both
    sides of half the cap: the same bits from run to run, within the bounds."""
    H, d, nk = 4, 128, 9000
    g = _gen(3)
    q, k, v, do = (torch.randn(n, H * d, generator=g, device="cuda").bfloat16() for n in (1, nk, nk, 1))
    cfg, docs = wan.make_config(H * d, H, 64), wan.documents(_i32([0, 1]), _i32([0, nk]), cap=5.0)
    want = R.attention(*(t.double() for t in (q, k, v)), H, H, [0, 1], [0, nk], torch.bfloat16, do=do.double(), cap=5.0)
    first = _attention(wan, cfg, docs, q, k, v, H, do=do)
    for name in first:
        R.assert_close(first[name], *want[name], name)
    for _ in range(200):
        again = _attention(wan, cfg, docs, q, k, v, H, do=do)
        assert all(torch.equal(again[name], first[name]) for name in first)


@pytest.mark.parametrize("rows,n_docs", [(0, 0), (0, 2), (4, 0)])
def test_residual_norm_gradient_of_nothing(wan, rows, n_docs):
    """No rows, no documents, or neither, with the workspace that the sizing call asks for: the sums
    are zeros, rows of no document stay as they were, and only what ran is counted."""
    D = 128
    cfg, spec = wan.make_config(D, 2, 64, dtype="f32"), wan.residual_norm(pre="layer", post="rms", gate=2, chunk=1)
    full = lambda *s: torch.full(s, 7.0, device="cuda")  # noqa: E731
    x, y, dx, dy = (full(rows, D) for _ in range(4))
    e, mb, cu = full(n_docs, 6, D), full(6, D), _i32([0] * (n_docs + 1))
    ws = torch.empty(wan.gated_residual_norm_workspace_bytes(cfg, rows, n_docs), dtype=torch.uint8, device="cuda")
    assert (ws.numel() == 0) == (rows == 0 and n_docs == 0)
    sums = dict(de=full(n_docs, 6, D), dmod_bias=full(6, D), dw_pre=full(D), db_pre=full(D), dw_post=full(D))
    before = wan.launch_count()
    wan.gated_residual_norm_bwd(cfg, spec, x, y, e, mb, cu, x, None, dx, dy, ws, **sums)
    torch.cuda.synchronize()
    assert wan.launch_count() - before == (3 if n_docs else 1)
    assert (dx == 7).all() and (dy == 7).all()
    for name in ("dw_pre", "db_pre", "dw_post"):
        assert not sums[name].any(), name
    for name in ("de", "dmod_bias"):
        t = sums[name]
        assert not t[..., 2:5, :].any() and (t[..., :2, :] == 7).all() and (t[..., 5, :] == 7).all(), name
    before = wan.launch_count()
    wan.gated_residual_norm_bwd(cfg, spec, x, y, e, mb, cu, x, None, dx, dy, ws)
    assert wan.launch_count() == before


def test_extreme_caps(wan):
    """A cap far above all scores is none; one far below them leaves every key alike, and no
    gradient but the values'."""
    H, d, n = 2, 128, 150
    g = _gen(6)
    q, k, v, do = (torch.randn(n, H * d, generator=g, device="cuda").bfloat16() for _ in range(4))
    q[5] = 0  # scores of 0
    cfg, cu = wan.make_config(H * d, H, 64), _i32([0, n])
    want = R.attention(*(t.double() for t in (q, k, v)), H, H, [0, n], [0, n], torch.bfloat16, do=do.double())
    got = _attention(wan, cfg, wan.documents(cu, cap=1e30), q, k, v, H, do=do)
    for name in got:
        R.assert_close(got[name], *want[name], name)
    got = _attention(wan, cfg, wan.documents(cu, cap=1e-30), q, k, v, H, do=do)
    want = R.attention(*(t.double() for t in (q, k, v)), H, H, [0, n], [0, n], torch.bfloat16, do=do.double(), cap=1e-30)
    for name in ("o", "lse", "dv"):
        R.assert_close(got[name], *want[name], name)
    others = torch.arange(n, device="cuda") != 5
    assert not got["dq"][others].any() and torch.isfinite(got["dq"]).all() and torch.isfinite(got["dk"]).all()


def _against_reference(wan, dtype, d, H, Hk, q_lens, k_lens, seed, split=True, first=0, spare=0, grads=True, k_growth=None, **opt):
    """One call (and its gradient) against the 64-bit form; returns what the call wrote."""
    act, g, opt = ACT[dtype], _gen(seed), dict(opt)
    nq, nk = first + sum(q_lens) + spare, first + sum(k_lens) + spare
    q, do = (torch.randn(nq, H * d, generator=g, device="cuda") for _ in range(2))
    k, v = (torch.randn(nk, Hk * d, generator=g, device="cuda") for _ in range(2))
    if k_growth:
        k *= torch.linspace(*k_growth, nk, device="cuda")[:, None]
    q, k, v, do = (t.to(act) for t in (q, k, v, do))
    slopes = [2.0 ** (-8.0 * (h + 1) / H) for h in range(H)] if opt.pop("slopes", False) else None
    cu_q, cu_k = R.cu_of(q_lens, first), R.cu_of(k_lens, first)
    scale = opt.get("scale", 0.0)
    docs = wan.documents(_i32(cu_q), _i32(cu_k), prefix=_i32(opt["prefix"]) if opt.get("prefix") else None,
                         causal_block=opt.get("block", 0), cap=opt.get("cap", 0.0), scale=scale,
                         slopes=None if slopes is None else torch.tensor(slopes, device="cuda"))
    cfg = wan.make_config(H * d, H, 64, dtype=dtype)
    got = _attention(wan, cfg, docs, q, k, v, Hk, do=do if grads else None, split=split)
    # a negative scale is a positive one with -q, and -dq
    flip = -1.0 if scale < 0 else 1.0
    opt["scale"] = abs(scale)
    want = R.attention(flip * q.double(), k.double(), v.double(), H, Hk, cu_q, cu_k, act, do=do.double() if grads else None,
                       slopes=slopes, **opt)
    for name in got:
        R.assert_close(flip * got[name].double() if name == "dq" else got[name], *want[name], name,
                       untouched=flip * 7.0 if name == "dq" else 7.0)
    return got


@pytest.mark.parametrize("d,H,Hk", [(4, 16, 4), (32, 4, 2), (60, 16, 16), (68, 16, 8), (96, 2, 1), (128, 3, 1), (128, 2, 2)])
@pytest.mark.parametrize("case", [([60, 0, 33], [50, 7, 70], dict()), ([100, 1], [100, 1], dict(block=1, slopes=True)),
                                  ([37, 20], [37, 20], dict(block=8, prefix=[9, 0], cap=4.0)), ([3], [300], dict(block=1, cap=15.0, slopes=True))],
                         ids=["texts", "causal", "frames", "step"])
def test_float32_head_dims(wan, d, H, Hk, case):
    q_lens, k_lens, opt = case
    _against_reference(wan, "f32", d, H, Hk, q_lens, k_lens, seed=d + H, first=2, spare=3, **opt)


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f32", 64), ("f32", 128)])
@pytest.mark.parametrize("opt", [dict(), dict(cap=2.0), dict(slopes=True), dict(cap=2.0, slopes=True, block=1)],
                         ids=["plain", "cap", "slopes", "all"])
def test_negative_scale(wan, dtype, d, opt):
    _against_reference(wan, dtype, d, 4, 2, [70, 200], [70, 200], seed=3, scale=-0.11, **opt)


def _cut_pieces(H, Hk, lq, lk, block):
    """The forward's shares of one document in causal blocks (no waves): for every piece of a cut
    unit, the key tiles that its two query tiles have in it."""
    group = H // Hk
    pack = max(n for n in range(1, 129) if group % n == 0)
    per_tile, ctas = 128 // pack, torch.cuda.get_device_properties(0).multi_processor_count

    def tiles(first, rows):
        if first >= lq:
            return 0
        pos = min(first + rows, lq) - 1 + lk - lq
        return -(-max(0, min(lk, (pos // block + 1) * block if pos >= 0 else 0)) // 128)

    units = [max(1, tiles(u, 2 * per_tile)) for u in range(0, lq, 2 * per_tile)] * (H // pack)
    firsts = list(range(0, lq, 2 * per_tile)) * (H // pack)
    total = sum(n + 2 for n in units)
    share = max(1, min(ctas, total // 4))
    at, out = 0, []
    for n, f in zip(units, firsts):
        ends = {total * c // share for c in range(share + 1)}
        cuts = [0] + sorted(e - at for e in ends if 0 < e - at < n) + [n]
        if n > 8 and len(cuts) > 2:
            for a, b in zip(cuts, cuts[1:]):
                out.append([max(0, min(tiles(f + t * per_tile, per_tile), b) - a) for t in range(2)])
        at += n + 2
    return out


@pytest.mark.parametrize("H,Hk,lq,lk,block,opt", [
    (2, 2, 700, 2600, 128, dict()), (4, 2, 515, 3100, 1, dict(cap=15.0)), (6, 2, 900, 1800, 300, dict(slopes=True)),
    (3, 3, 1300, 1300, 64, dict(prefix=[40], cap=30.0, slopes=True)), (2, 1, 1500, 1200, 50, dict())])
def test_units_cut_under_an_order_mask(wan, H, Hk, lq, lk, block, opt):
    pieces = _cut_pieces(H, Hk, lq, lk, block)
    assert len(pieces) > 4
    if (H, lq) in ((2, 700), (4, 515)):
        assert any(a == 0 and b > 0 for a, b in pieces)  # keys that only the second query tile sees
    _against_reference(wan, "bf16", 128, H, Hk, [lq], [lk], seed=lq, block=block, grads=False, spare=3, **opt)


@pytest.mark.parametrize("growth", [(0.1, 8.0), (8.0, 0.1)])
@pytest.mark.parametrize("lq,H,Hk,opt", [(200, 2, 2, dict()), (300, 4, 2, dict(block=32)), (1, 6, 2, dict(block=1)),
                                         (2, 8, 1, dict(slopes=True))])
def test_scores_that_grow_through_cut_units(wan, growth, lq, H, Hk, opt):
    """The base of the exponentials moves inside the parts and differs between them."""
    cut = _against_reference(wan, "bf16", 128, H, Hk, [lq], [4000], seed=8, grads=False, k_growth=growth, **opt)
    whole = _against_reference(wan, "bf16", 128, H, Hk, [lq], [4000], seed=8, grads=False, k_growth=growth, split=False, **opt)
    assert any(not torch.equal(cut[name], whole[name]) for name in cut)  # other sums, of the same value


def test_capped_scores_and_their_gradient_on_both_sides_of_half_the_cap(wan):
    for cap in (1.0, 3.0, 400.0):
        _against_reference(wan, "bf16", 128, 4, 2, [300, 45], [300, 45], seed=5, block=1, cap=cap, scale=1.0)
