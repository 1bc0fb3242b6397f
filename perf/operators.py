"""Measured cases of the packed-document operators: rotary positions with the q/k norm,
the gated residual fused with the norms around a block, and attention over documents.

Each case is one pass through one operator on random inputs of a stated shape. ``run``
computes the plain form (elementary torch operations in float32, angles in float64) or,
with ``own`` set, calls the framework. ``exact`` is the definition in float64.
"""
import math

import torch

own = False

# A document is a clip, an image or a text of its own length; documents follow one
# another along the row axis of a packed tensor. Lengths are written "a,b,c", grids
# (frames x height x width in tokens) "FxHxW;FxHxW".


def _ints(text):
    return [int(v) for v in text.split(",")] if text else []


def _grids(text):
    return [tuple(int(v) for v in g.split("x")) for g in text.split(";")]


# ------------------------------------------------------------------------- the cases
def listed():
    rope = dict(op="rope", dtype="bf16", norm="width", layout="interleaved", axes="44,42,42", theta=10000.0,
                scaling="none", factor="1,1,1", orig="0,0,0", amplitude=1.0, head_dim=128)
    norm = dict(op="norm", dtype="bf16", residual_scale=1.0, pre="layer", post="none", gate=2, chunk=1,
                affine=False, pad=0)
    attn = dict(op="attn", dtype="bf16", head_dim=128, prefix="", causal_block=0, cap=0.0, slopes=False, pad=0)
    return [
        # q and k of one block over a whole 81-frame 480P clip: 21 x 30 x 52 tokens, 12 heads
        dict(rope, name="rope_480p_clip", dir="fwd", grids="21x30x52", heads=12, kv_heads=12),
        # one new token for each of 9 sequences at far positions: half layout on part of the head,
        # per-head norm, shared key heads, positions stretched by the ramped scaling
        dict(rope, name="rope_step_far", dir="fwd", grids="", rows=9, start=900000, heads=12, kv_heads=4, norm="head",
             layout="half", axes="96", scaling="ramp", factor="8", orig="131072", amplitude=1.2),
        # gradient of q, k and both norm weights over three clips of mixed size
        dict(rope, name="rope_grad_clips", dir="bwd", grids="13x30x52;1x45x80;7x17x31", heads=12, kv_heads=12),
        # between self-attention and FFN, a packed batch of four clips, 1.3B width
        dict(norm, name="norm_clips_1536", dir="fwd", lens="20280,1560,7801,3119", dim=1536, post="rms", affine=True),
        # the same step for a handful of rows, where the launch counts
        dict(norm, name="norm_few_rows", dir="fwd", lens="1,0,6,2", dim=1536),
        # gradient at the 14B width: a quarter of a 720P clip's 75600 rows and a still image
        dict(norm, name="norm_grad_5120", dir="bwd", lens="18900,3600,1", dim=5120, post="rms", affine=True, pad=7),
        # self-attention over four packed clips and images, 1.3B heads
        dict(attn, name="attn_clips", dir="fwd", q_lens="14040,1560,6273,1527", k_lens="", heads=12, kv_heads=12),
        # cross-attention of packed clips to ragged texts, one of them empty
        dict(attn, name="attn_ragged_text", dir="fwd", q_lens="7800,4680,1560,33", k_lens="512,77,301,0", heads=12,
             kv_heads=12, pad=15),
        # frame-by-frame causal clips (1560 tokens a frame) with a given first frame, shared
        # key heads, capped scores and a penalty on distance
        dict(attn, name="attn_frames_capped", dir="fwd", q_lens="6240,3120", k_lens="", heads=12, kv_heads=4,
             prefix="1560,700", causal_block=1560, cap=30.0, slopes=True),
        # one new token for each of 8 sequences over long kept keys
        dict(attn, name="attn_step_long_keys", dir="fwd", q_lens="1,1,1,1,1,1,1,1",
             k_lens="32760,20281,1560,9361,32760,4681,15600,977", heads=12, kv_heads=4, causal_block=1),
        # forward and gradient over packed clips, 1.3B heads
        dict(attn, name="attn_train_clips", dir="train", q_lens="4680,1560,3131", k_lens="", heads=12, kv_heads=12),
        # forward and gradient of a small float32 model, token-causal with a prefix
        dict(attn, name="attn_train_small_f32", dir="train", dtype="f32", q_lens="300,45,1", k_lens="", heads=2,
             kv_heads=1, head_dim=64, prefix="20,0,0", causal_block=1, cap=20.0),
    ]


def _spread(rng, lo, hi):
    """An integer of [lo, hi], spread over the logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def _cut(rng, total, parts):
    """`total` cut into `parts` lengths, some of them possibly 0 or 1."""
    at = sorted(rng.randint(0, total) for _ in range(parts - 1))
    return [b - a for a, b in zip([0] + at, at + [total])]


def draw(rng):
    op = rng.choice(["rope", "norm", "attn", "attn"])
    f32 = rng.random() < 0.3
    if op == "rope":
        heads = rng.choice([2, 4, 6, 12, 20, 40])
        kv = rng.choice([h for h in range(1, heads + 1) if heads % h == 0])
        hd = 64 if f32 else 128
        layout = rng.choice(["interleaved", "half"])
        if rng.random() < 0.6:
            axes = rng.choice(["20,22,22", "32,16,16", "8,8,8"]) if f32 else rng.choice(["44,42,42", "64,32,32", "16,24,24"])
            n = _spread(rng, 1, 4)
            grids = ";".join("%dx%dx%d" % (rng.randint(1, 21), rng.randint(1, 30), rng.randint(1, 45 // n + 1)) for _ in range(n))
            where = dict(grids=grids)
            n_axes = 3
        else:
            axes = rng.choice(["64", "32"]) if f32 else rng.choice(["128", "96", "64"])
            where = dict(grids="", rows=_spread(rng, 1, 9000), start=_spread(rng, 1, 1000000))
            n_axes = 1
        scaling = rng.choice(["none", "linear", "base", "ramp"])
        return dict(op="rope", dtype="f32" if f32 else "bf16", dir=rng.choice(["fwd", "bwd"]), head_dim=hd, heads=heads,
                    kv_heads=kv, norm=rng.choice(["none", "head", "width"]), layout=layout, axes=axes,
                    theta=rng.choice([10000.0, 256.0, 1e6]), scaling=scaling,
                    factor=",".join(str(rng.choice([1, 2, 4, 8])) for _ in range(n_axes)),
                    orig=",".join(str(rng.choice([16, 1024, 32768])) for _ in range(n_axes)),
                    amplitude=round(rng.uniform(0.9, 1.4), 3), **where)
    if op == "norm":
        dim = rng.choice([128, 320, 512, 1024, 1536, 2048, 5120])
        total = _spread(rng, 1, 16000)
        lens = ",".join(map(str, _cut(rng, total, _spread(rng, 1, 12))))
        return dict(op="norm", dtype="f32" if f32 else "bf16", dir=rng.choice(["fwd", "bwd"]), lens=lens, dim=dim,
                    residual_scale=rng.choice([1.0, 0.7]), pre=rng.choice(["layer", "rms"]),
                    post=rng.choice(["none", "rms", "layer"]), gate=rng.choice([-1, 2, 5]),
                    chunk=rng.choice([-1, 0, 1]), affine=rng.random() < 0.5, pad=rng.choice([0, 0, 5]))
    parts = _spread(rng, 1, 9)
    heads = rng.choice([2, 4, 6, 12])
    kv = rng.choice([h for h in range(1, heads + 1) if heads % h == 0])
    direction = rng.choice(["fwd", "fwd", "train"])
    most = 1200 if f32 else 9000 if direction == "fwd" else 6000
    q = _cut(rng, _spread(rng, 1, most), parts)
    k = []
    kind = rng.random()
    if kind < 0.25 and direction == "fwd" and not f32:
        # single new tokens over kept keys
        q = [1] * parts
        k = [_spread(rng, 1, 16000) for _ in range(parts)]
    elif kind < 0.5:
        # keys of their own: ragged texts
        k = _cut(rng, _spread(rng, 1, 1200), parts)
    block = rng.choice([0, 0, 1, 30, 256])
    prefix = ",".join(str(rng.randint(0, n)) for n in (k or q)) if block and rng.random() < 0.5 else ""
    return dict(op="attn", dtype="f32" if f32 else "bf16", dir=direction, heads=heads, kv_heads=kv,
                head_dim=64 if f32 else 128, q_lens=",".join(map(str, q)), k_lens=",".join(map(str, k)), prefix=prefix,
                causal_block=block, cap=rng.choice([0.0, 0.0, 15.0, 50.0]), slopes=rng.random() < 0.3,
                pad=rng.choice([0, 0, 9]))


# ---------------------------------------------------------------------------- inputs
_ACT = {"bf16": torch.bfloat16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f32": 4}
EPS = 1e-6


def _cu(lens):
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    return torch.tensor(at, dtype=torch.int32, device="cuda")


def _rope_rows(case):
    return sum(f * h * w for f, h, w in _grids(case["grids"])) if case["grids"] else case["rows"]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    act = _ACT[case["dtype"]]

    def normal(*shape, scale=1.0, dtype=None):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype or act)

    s = dict(case=case)
    if case["op"] == "rope":
        rows, H, Hk, d = _rope_rows(case), case["heads"], case["kv_heads"], case["head_dim"]
        if case["grids"]:
            parts = []
            for f, h, w in _grids(case["grids"]):
                parts.append(torch.cartesian_prod(torch.arange(f), torch.arange(h), torch.arange(w)).reshape(-1, 3))
            s["pos"] = torch.cat(parts).to(device="cuda", dtype=torch.int32)
        else:
            s["pos"] = (case["start"] + torch.randint(0, 1000, (rows, 1), generator=g, device="cuda")).to(torch.int32)
        # q | k | v side by side, as the projection writes them; q and k are columns of it
        qkv = normal(rows, (H + 2 * Hk) * d)
        s["q"], s["k"] = qkv[:, :H * d], qkv[:, H * d:(H + Hk) * d]
        if case["norm"] != "none":
            width = case["norm"] == "width"
            s["w_q"] = normal(H * d if width else d, scale=0.2) + 1
            s["w_k"] = normal(Hk * d if width else d, scale=0.2) + 1
        if case["dir"] == "bwd":
            s["dq_out"], s["dk_out"] = normal(rows, H * d), normal(rows, Hk * d)
        s["q_res"], s["k_res"] = torch.empty(rows, H * d, dtype=act, device="cuda"), torch.empty(rows, Hk * d, dtype=act, device="cuda")
    elif case["op"] == "norm":
        lens, D = _ints(case["lens"]), case["dim"]
        rows = sum(lens) + case["pad"]
        s["cu"] = _cu(lens)
        s["e"], s["mod_bias"] = normal(len(lens), 6, D, scale=0.2, dtype=torch.float32), normal(6, D, scale=0.02, dtype=torch.float32)
        s["x"], s["y"] = normal(rows, D, dtype=torch.float32), normal(rows, D)
        if case["affine"]:
            s["w_pre"], s["b_pre"] = normal(D, scale=0.1) + 1, normal(D, scale=0.1)
            if case["post"] != "none":
                s["w_post"] = normal(D, scale=0.1) + 1
        s["x_res"] = torch.zeros(rows, D, dtype=torch.float32, device="cuda")
        s["h_res"] = torch.zeros(rows, D, dtype=act, device="cuda")
        if case["dir"] == "bwd":
            s["dh"], s["dx_out"] = normal(rows, D), normal(rows, D, dtype=torch.float32)
    else:
        q_lens = _ints(case["q_lens"])
        k_lens = _ints(case["k_lens"]) or q_lens
        H, Hk, d = case["heads"], case["kv_heads"], case["head_dim"]
        Tq, Tk = sum(q_lens) + case["pad"], sum(k_lens) + case["pad"]
        s["cu_q"], s["cu_k"] = _cu(q_lens), _cu(k_lens)
        s["prefix"] = torch.tensor(_ints(case["prefix"]), dtype=torch.int32, device="cuda") if case["prefix"] else None
        s["slopes"] = torch.tensor([2.0 ** (-8.0 * (h + 1) / H) for h in range(H)], device="cuda") if case["slopes"] else None
        s["q"] = normal(Tq, H * d)
        kv = normal(Tk, 2 * Hk * d)
        s["k"], s["v"] = kv[:, :Hk * d], kv[:, Hk * d:]
        s["o"] = torch.zeros(Tq, H * d, dtype=act, device="cuda")
        s["lse"] = torch.zeros(H, Tq, dtype=torch.float32, device="cuda")
        if case["dir"] == "train":
            s["do"] = normal(Tq, H * d)
            s["dq"] = torch.zeros_like(s["o"])
            s["dk"], s["dv"] = torch.zeros(Tk, Hk * d, dtype=act, device="cuda"), torch.zeros(Tk, Hk * d, dtype=act, device="cuda")
    return s


# ------------------------------------------------------------------------ plain forms
def _frequencies(case):
    """Frequency of every rotated pair, its axis, in float64."""
    f, axis = [], []
    factors, origs = [float(v) for v in case["factor"].split(",")], _ints(case["orig"])
    for a, n in enumerate(_ints(case["axes"])):
        i = torch.arange(n // 2, dtype=torch.float64)
        theta, k = case["theta"], factors[a]
        if case["scaling"] == "base":
            theta = theta * k ** (n / (n - 2))
        w = theta ** (-2 * i / n)
        if case["scaling"] == "linear":
            w = w / k
        elif case["scaling"] == "ramp":
            # whole turns over the original length: pairs above 32 keep their frequency,
            # pairs below 1 are stretched by the factor, a ramp between
            keep = ((origs[a] * w / (2 * math.pi) - 1) / (32 - 1)).clamp(0, 1)
            w = w * (keep + (1 - keep) / k)
        f.append(w)
        axis += [a] * (n // 2)
    return torch.cat(f).cuda(), torch.tensor(axis, device="cuda")


def _cos_sin(s, dtype):
    case = s["case"]
    f, axis = _frequencies(case)
    angle = s["pos"].double()[:, axis] * f
    a = case["amplitude"]
    return (angle.cos() * a).to(dtype)[:, None], (angle.sin() * a).to(dtype)[:, None]


def _rotate(x, cos, sin, layout):
    """x [rows, heads, d], cos and sin [rows, 1, pairs]."""
    n = 2 * cos.shape[-1]
    y = x.clone()
    if layout == "interleaved":
        a, b = x[..., 0:n:2], x[..., 1:n:2]
        y[..., 0:n:2], y[..., 1:n:2] = a * cos - b * sin, a * sin + b * cos
    else:
        a, b = x[..., :n // 2], x[..., n // 2:n]
        y[..., :n // 2], y[..., n // 2:n] = a * cos - b * sin, a * sin + b * cos
    return y


def _rope_one(x, w, heads, case, cos, sin, act):
    rows, d = x.shape[0], case["head_dim"]
    x = x.to(cos.dtype).reshape(rows, heads, d)
    if case["norm"] == "head":
        x = x * (x.square().mean(-1, keepdim=True) + EPS).rsqrt() * w.to(x.dtype)
    elif case["norm"] == "width":
        x = x * (x.square().mean((1, 2), keepdim=True) + EPS).rsqrt() * w.to(x.dtype).reshape(heads, d)
    return _rotate(x, cos, sin, case["layout"]).reshape(rows, heads * d).to(act)


def _rope_one_bwd(dout, x, w, heads, case, cos, sin, act):
    rows, d = x.shape[0], case["head_dim"]
    g = _rotate(dout.to(cos.dtype).reshape(rows, heads, d), cos, -sin, case["layout"])
    if case["norm"] == "none":
        return g.reshape(rows, heads * d).to(act), None
    x, over = x.to(cos.dtype).reshape(rows, heads, d), -1 if case["norm"] == "head" else (1, 2)
    r = (x.square().mean(over, keepdim=True) + EPS).rsqrt()
    xh = x * r
    w = w.to(x.dtype) if case["norm"] == "head" else w.to(x.dtype).reshape(heads, d)
    gw = g * w
    dx = r * (gw - xh * (gw * xh).mean(over, keepdim=True))
    dw = (g * xh).sum((0, 1)) if case["norm"] == "head" else (g * xh).sum(0).reshape(-1)
    return dx.reshape(rows, heads * d).to(act), dw


def _rope(s, dtype, act):
    case = s["case"]
    cos, sin = _cos_sin(s, dtype)
    H, Hk = case["heads"], case["kv_heads"]
    if case["dir"] == "fwd":
        return dict(q=_rope_one(s["q"], s.get("w_q"), H, case, cos, sin, act),
                    k=_rope_one(s["k"], s.get("w_k"), Hk, case, cos, sin, act))
    dq, dwq = _rope_one_bwd(s["dq_out"], s["q"], s.get("w_q"), H, case, cos, sin, act)
    dk, dwk = _rope_one_bwd(s["dk_out"], s["k"], s.get("w_k"), Hk, case, cos, sin, act)
    return dict(dq=dq, dk=dk) if dwq is None else dict(dq=dq, dk=dk, dw_q=dwq, dw_k=dwk)


def _doc_of(cu, rows):
    """Document of each row, -1 for a row behind the last document."""
    r = torch.arange(rows, device=cu.device)
    d = torch.searchsorted(cu[1:].long(), r, right=True)
    return torch.where(d < cu.numel() - 1, d, -1)


def _normalise(x, kind):
    if kind == "layer":
        x = x - x.mean(-1, keepdim=True)
    r = (x.square().mean(-1, keepdim=True) + EPS).rsqrt()
    return x * r, r


def _normalise_bwd(g, n, r, kind):
    """Gradient of n = normalise(x) with respect to x."""
    g = g - n * (g * n).mean(-1, keepdim=True)
    if kind == "layer":
        g = g - g.mean(-1, keepdim=True)
    return g * r


def _modulation(s, dtype):
    """Per document: gate, shift and 1 + scale, [documents, D] each (None where absent)."""
    case = s["case"]
    m = s["e"].to(dtype) + s["mod_bias"].to(dtype)
    c = case["chunk"]
    return (m[:, case["gate"]] if case["gate"] >= 0 else None, m[:, 3 * c] if c >= 0 else None,
            1 + m[:, 3 * c + 1] if c >= 0 else None)


def _norm_fwd(s, dtype, act, x_type):
    case = s["case"]
    rows = s["x"].shape[0] - case["pad"]
    doc = _doc_of(s["cu"], s["x"].shape[0])[:rows]
    gate, shift, scale = _modulation(s, dtype)
    y = s["y"][:rows].to(dtype)
    if case["post"] != "none":
        y = _normalise(y, case["post"])[0]
        if "w_post" in s:
            y = y * s["w_post"].to(dtype)
    if gate is not None:
        y = y * gate[doc]
    x = s["x"][:rows].to(dtype) * case["residual_scale"] + y
    h = _normalise(x, case["pre"])[0]
    if case["affine"]:
        h = h * s["w_pre"].to(dtype) + s["b_pre"].to(dtype)
    if shift is not None:
        h = h * scale[doc] + shift[doc]
    behind = (0, 0, 0, case["pad"])
    return dict(x=torch.nn.functional.pad(x.to(x_type), behind), h=torch.nn.functional.pad(h.to(act), behind))


def _per_document(v, doc, n):
    return torch.zeros(n, v.shape[1], dtype=v.dtype, device=v.device).index_add_(0, doc, v)


def _norm_bwd(s, dtype, act, x_type):
    """Here s["x"] is the forward's x output and s["y"] its branch input."""
    case = s["case"]
    rows = s["x"].shape[0] - case["pad"]
    n_docs, D = s["e"].shape[0], case["dim"]
    doc = _doc_of(s["cu"], s["x"].shape[0])[:rows]
    gate, shift, scale = _modulation(s, dtype)
    dh = s["dh"][:rows].to(dtype)
    n, r = _normalise(s["x"][:rows].to(dtype), case["pre"])
    a = n
    w, b = torch.ones(D, dtype=dtype, device="cuda"), torch.zeros(D, dtype=dtype, device="cuda")
    if case["affine"]:
        w, b = s["w_pre"].to(dtype), s["b_pre"].to(dtype)
        a = n * w + b
    out = {}
    de = torch.zeros(n_docs, 6, D, dtype=dtype, device="cuda")
    da = dh
    if shift is not None:
        de[:, 3 * case["chunk"]] = _per_document(dh, doc, n_docs)
        de[:, 3 * case["chunk"] + 1] = _per_document(dh * a, doc, n_docs)
        da = dh * scale[doc]
    if case["affine"]:
        out["dw_pre"], out["db_pre"] = (da * n).sum(0).to(x_type), da.sum(0).to(x_type)
    dx = s["dx_out"][:rows].to(dtype) + _normalise_bwd(da * w, n, r, case["pre"])
    y = s["y"][:rows].to(dtype)
    yn, ry = _normalise(y, case["post"]) if case["post"] != "none" else (y, None)
    yw = yn * s["w_post"].to(dtype) if "w_post" in s else yn
    dyw = dx
    if gate is not None:
        de[:, case["gate"]] = _per_document(dx * yw, doc, n_docs)
        dyw = dx * gate[doc]
    if "w_post" in s:
        out["dw_post"] = (dyw * yn).sum(0).to(x_type)
        dyw = dyw * s["w_post"].to(dtype)
    dy = _normalise_bwd(dyw, yn, ry, case["post"]) if ry is not None else dyw
    behind = (0, 0, 0, case["pad"])
    out["dx"] = torch.nn.functional.pad((dx * case["residual_scale"]).to(x_type), behind)
    out["dy"] = torch.nn.functional.pad(dy.to(act), behind)
    if gate is not None or shift is not None:
        out["de"] = de.to(x_type)
    return out


def _attn(s):
    """Scores of every query against every key, with the document and order mask."""
    case = s["case"]
    H, Hk, d, act = case["heads"], case["kv_heads"], case["head_dim"], s["q"].dtype
    Tq, Tk = s["q"].shape[0], s["k"].shape[0]
    q_doc, k_doc = _doc_of(s["cu_q"], Tq), _doc_of(s["cu_k"], Tk)
    cu_q, cu_k = s["cu_q"].long(), s["cu_k"].long()
    n_k = (cu_k[1:] - cu_k[:-1])[q_doc]
    i = torch.arange(Tq, device="cuda") - cu_q[q_doc] + n_k - (cu_q[1:] - cu_q[:-1])[q_doc]
    j = torch.arange(Tk, device="cuda") - cu_k[k_doc]
    seen = n_k
    if case["causal_block"]:
        g = case["causal_block"]
        seen = torch.minimum((torch.div(i, g, rounding_mode="floor") + 1) * g, n_k).clamp(min=0)
        if s["prefix"] is not None:
            seen = torch.maximum(seen, torch.minimum(s["prefix"].long()[q_doc], n_k))
    hide = (q_doc[:, None] != k_doc) | (q_doc[:, None] < 0) | (j >= seen[:, None])
    split = lambda t, h: t.float().reshape(-1, h, d).transpose(0, 1)  # noqa: E731
    group = lambda t: split(t, Hk).repeat_interleave(H // Hk, 0)  # noqa: E731
    scale = d ** -0.5
    q, k, v = split(s["q"], H), group(s["k"]), group(s["v"])
    a = (q * scale) @ k.transpose(1, 2)
    slope_t = None
    if case["cap"]:
        a.div_(case["cap"]).tanh_()
        slope_t = 1 - a.square() if case["dir"] == "train" else None
        a.mul_(case["cap"])
    if s["slopes"] is not None:
        a.sub_(s["slopes"][:, None, None] * (i[:, None] - j).abs().float())
    a.masked_fill_(hide, -math.inf)
    m = a.amax(-1, keepdim=True)
    a.sub_(torch.where(m.isinf(), 0.0, m)).exp_()
    total = a.sum(-1, keepdim=True)
    one = torch.where(total > 0, total, 1.0)
    join = lambda t: t.transpose(0, 1).reshape(-1, t.shape[0] * d).to(act)  # noqa: E731
    of_doc = q_doc >= 0
    lse = torch.where(of_doc, (m + total.log())[..., 0], 0.0)
    o = a @ v / one
    out = dict(o=join(o), lse=lse)
    if case["dir"] == "train":
        do = split(s["do"], H)
        a.div_(one)
        shared = lambda t: t.reshape(Hk, H // Hk, Tk, d).sum(1)  # noqa: E731
        out["dv"] = join(shared(a.transpose(1, 2) @ do))
        ds = do @ v.transpose(1, 2)
        ds.sub_((do * o).sum(-1, keepdim=True)).mul_(a)
        if slope_t is not None:
            ds.mul_(slope_t)
        out["dq"], out["dk"] = join(ds @ k * scale), join(shared(ds.transpose(1, 2) @ (q * scale)))
    return out


# ------------------------------------------------------------------------------- run
def _run_own(s):
    import video_diffusion_transformer_wan_b200 as wan
    case = s["case"]
    if case["op"] == "norm":
        D = case["dim"]
        cfg = wan.make_config(D, D // 64, 64, dtype=case["dtype"])
        spec = wan.residual_norm(pre=case["pre"], post=case["post"], gate=case["gate"], chunk=case["chunk"],
                                 residual_scale=case["residual_scale"], w_pre=s.get("w_pre"), b_pre=s.get("b_pre"),
                                 w_post=s.get("w_post"))
        if case["dir"] == "fwd":
            wan.gated_residual_norm_fwd(cfg, spec, s["x"], s["y"], s["e"], s["mod_bias"], s["cu"], s["x_res"], s["h_res"])
            return dict(x=s["x_res"], h=s["h_res"])
        ws = torch.empty(wan.gated_residual_norm_workspace_bytes(cfg, s["x"].shape[0], s["e"].shape[0]), dtype=torch.uint8, device="cuda")
        out = dict(dx=s["x_res"], dy=s["h_res"])
        new = lambda: torch.empty(D, device="cuda")  # noqa: E731
        if case["gate"] >= 0 or case["chunk"] >= 0:
            out["de"] = torch.zeros_like(s["e"])
        if "w_pre" in s:
            out["dw_pre"], out["db_pre"] = new(), new()
        if "w_post" in s:
            out["dw_post"] = new()
        wan.gated_residual_norm_bwd(cfg, spec, s["x"], s["y"], s["e"], s["mod_bias"], s["cu"], s["dh"], s["dx_out"],
                                    s["x_res"], s["h_res"], ws, de=out.get("de"), dw_pre=out.get("dw_pre"),
                                    db_pre=out.get("db_pre"), dw_post=out.get("dw_post"))
        return out
    H, Hk, d = case["heads"], case["kv_heads"], case["head_dim"]
    cfg = wan.make_config(H * d, H, 64, dtype=case["dtype"])
    if case["op"] == "rope":
        rope = wan.rope(_ints(case["axes"]), layout=case["layout"], theta=case["theta"], scaling=case["scaling"],
                        factor=[float(v) for v in case["factor"].split(",")], orig_len=_ints(case["orig"]),
                        amplitude=case["amplitude"])
        if case["dir"] == "fwd":
            wan.qk_norm_rope_fwd(cfg, rope, s["pos"], s["q"], s["k"], s["q_res"], s["k_res"], kv_heads=Hk,
                                 norm=case["norm"], w_q=s.get("w_q"), w_k=s.get("w_k"))
            return dict(q=s["q_res"], k=s["k_res"])
        out = dict(dq=s["q_res"], dk=s["k_res"])
        ws = None
        if case["norm"] != "none":
            out["dw_q"], out["dw_k"] = torch.empty(s["w_q"].shape, device="cuda"), torch.empty(s["w_k"].shape, device="cuda")
            ws = torch.empty(wan.qk_norm_rope_workspace_bytes(cfg, s["q"].shape[0], Hk, case["norm"]), dtype=torch.uint8, device="cuda")
        wan.qk_norm_rope_bwd(cfg, rope, s["pos"], s["dq_out"], s["dk_out"], s["q"], s["k"], s["q_res"], s["k_res"],
                             kv_heads=Hk, norm=case["norm"], w_q=s.get("w_q"), w_k=s.get("w_k"), dw_q=out.get("dw_q"),
                             dw_k=out.get("dw_k"), ws=ws)
        return out
    docs = wan.documents(s["cu_q"], s["cu_k"], prefix=s["prefix"], causal_block=case["causal_block"], cap=case["cap"],
                         slopes=s["slopes"])
    Tq, Tk, n = s["q"].shape[0], s["k"].shape[0], s["cu_q"].numel() - 1
    train = case["dir"] == "train"
    size = wan.attention_packed_workspace_bytes(cfg, Tq, Tk, n, Hk, backward=train)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda") if size else None
    wan.attention_packed_fwd(cfg, docs, s["q"], s["k"], s["v"], s["o"], s["lse"], kv_heads=Hk, ws=ws)
    out = dict(o=s["o"], lse=s["lse"])
    if train:
        wan.attention_packed_bwd(cfg, docs, s["q"], s["k"], s["v"], s["o"], s["lse"], s["do"], s["dq"], s["dk"],
                                 s["dv"], kv_heads=Hk, ws=ws)
        out.update(dq=s["dq"], dk=s["dk"], dv=s["dv"])
    return out


def run(state):
    if own:
        return _run_own(state)
    case = state["case"]
    act = _ACT[case["dtype"]]
    if case["op"] == "rope":
        return _rope(state, torch.float32, act)
    if case["op"] == "norm":
        return (_norm_fwd if case["dir"] == "fwd" else _norm_bwd)(state, torch.float32, act, torch.float32)
    return _attn(state)


# ------------------------------------------------------------------------------ work
def _seen_keys(case):
    """Per document: rows, keys, and the pairs of a query with a key that it sees."""
    q_lens = _ints(case["q_lens"])
    k_lens = _ints(case["k_lens"]) or q_lens
    prefix = _ints(case["prefix"]) or [0] * len(q_lens)
    g, out = case["causal_block"], []
    for lq, lk, p in zip(q_lens, k_lens, prefix):
        if not g:
            out.append((lq, lk, lq * lk))
        else:
            out.append((lq, lk, sum(max(min(p, lk), min(lk, max(0, ((i + lk - lq) // g + 1) * g))) for i in range(lq))))
    return out


def _n_axes(case):
    return len(_ints(case["axes"]))


def work(case):
    es = _SIZE[case["dtype"]]
    if case["op"] == "rope":
        rows, w = _rope_rows(case), (case["heads"] + case["kv_heads"]) * case["head_dim"]
        reads = 1 if case["dir"] == "fwd" else 1 if case["norm"] == "none" else 2
        return {"bytes": rows * (w * es * (reads + 1) + _n_axes(case) * 4), "flops": rows * w * (8 if reads == 1 else 20)}
    if case["op"] == "norm":
        lens, D = _ints(case["lens"]), case["dim"]
        el = sum(lens) * D
        bwd = case["dir"] == "bwd"
        vectors = len(lens) * D * 4 * (3 if not bwd else 6)
        return {"bytes": el * ((4 + es) * 2 + (4 + es if bwd else 0)) + vectors, "flops": el * (30 if bwd else 15)}
    H, Hk, d = case["heads"], case["kv_heads"], case["head_dim"]
    seen = _seen_keys(case)
    pairs = sum(p for _, _, p in seen)
    rows, keys = sum(a for a, _, p in seen), sum(b for _, b, p in seen if p)
    train = case["dir"] == "train"
    return {"bytes": es * d * (rows * H * (4 if train else 2) + keys * Hk * (4 if train else 2)) + rows * H * 4,
            "flops": pairs * H * d * (14 if train else 4)}


# ----------------------------------------------------------------------------- exact
def _exact_rope(s):
    """From complex numbers: a pair (a, b) is a + ib, a rotation a product with amplitude e^(i angle)."""
    case = s["case"]
    f, axis = [], []
    factor, orig = [float(v) for v in case["factor"].split(",")], _ints(case["orig"])
    for a, n in enumerate(_ints(case["axes"])):
        for i in range(n // 2):
            base = case["theta"] * (factor[a] ** (n / (n - 2)) if case["scaling"] == "base" else 1.0)
            w = base ** (-2.0 * i / n)
            if case["scaling"] == "linear":
                w /= factor[a]
            if case["scaling"] == "ramp":
                turns = orig[a] * w / (2 * math.pi)
                keep = min(1.0, max(0.0, (turns - 1.0) / 31.0))
                w = keep * w + (1 - keep) * w / factor[a]
            f.append(w)
            axis.append(a)
    angle = s["pos"].double()[:, axis] * torch.tensor(f, dtype=torch.float64, device="cuda")
    turn = torch.polar(torch.full_like(angle, case["amplitude"]), angle)[:, None]
    n, d = len(f), case["head_dim"]
    out = {}
    for name, heads in (("q", case["heads"]), ("k", case["kv_heads"])):
        x = s[name].double().reshape(-1, heads, d)

        def pairs(t):
            p = t[..., :2 * n].reshape(-1, heads, n, 2) if case["layout"] == "interleaved" else t[..., :2 * n].reshape(-1, heads, 2, n).transpose(2, 3)
            return torch.view_as_complex(p.contiguous())

        def back(z, t):
            p = torch.view_as_real(z)
            p = p.reshape(-1, heads, 2 * n) if case["layout"] == "interleaved" else p.transpose(2, 3).reshape(-1, heads, 2 * n)
            return torch.cat([p, t[..., 2 * n:]], -1)

        if case["dir"] == "fwd":
            if case["norm"] != "none":
                w = s["w_" + name].double()
                ms = x.pow(2).mean(2, keepdim=True) if case["norm"] == "head" else x.pow(2).mean((1, 2), keepdim=True)
                x = x / (ms + EPS).sqrt() * (w if case["norm"] == "head" else w.reshape(heads, d))
            out[name] = back(pairs(x) * turn, x).reshape(-1, heads * d)
        else:
            g = s["d%s_out" % name].double().reshape(-1, heads, d)
            g = back(pairs(g) * turn.conj(), g)
            if case["norm"] == "none":
                out["d" + name] = g.reshape(-1, heads * d)
                continue
            w = s["w_" + name].double()
            w = w.expand(heads, d) if case["norm"] == "head" else w.reshape(heads, d)
            dims = (2,) if case["norm"] == "head" else (1, 2)
            ms = x.pow(2).mean(dims, keepdim=True) + EPS
            # d/dx of x w ms^(-1/2), term by term
            dx = g * w * ms.pow(-0.5) - x * ms.pow(-1.5) * (g * w * x).mean(dims, keepdim=True)
            dw = g * x * ms.pow(-0.5)
            out["d" + name] = dx.reshape(-1, heads * d)
            out["dw_" + name] = dw.sum((0, 1)) if case["norm"] == "head" else dw.sum(0).reshape(-1)
    return out


def _exact_norm(s):
    """Document by document; the gradient by automatic differentiation of the definition."""
    case = s["case"]
    D, lens, bwd = case["dim"], _ints(case["lens"]), case["dir"] == "bwd"
    rows = s["x"].shape[0]
    leaf = lambda t: t.double().requires_grad_(bwd)  # noqa: E731
    e = leaf(s["e"])
    w_pre, b_pre, w_post = (leaf(s[k]) if k in s else None for k in ("w_pre", "b_pre", "w_post"))
    m = e + s["mod_bias"].double()
    first = torch.zeros(rows, D, dtype=torch.float64, device="cuda")
    second = torch.zeros_like(first)

    def norm(t, kind):
        if kind == "layer":
            return torch.nn.functional.layer_norm(t, (D,), eps=EPS)
        return t / (t.pow(2).mean(1, keepdim=True) + EPS).sqrt()

    at, grads = 0, {}
    for doc, n in enumerate(lens):
        if not n:
            continue
        x, y = leaf(s["x"][at:at + n]), leaf(s["y"][at:at + n])
        branch = y if case["post"] == "none" else norm(y, case["post"])
        if w_post is not None:
            branch = branch * w_post
        if case["gate"] >= 0:
            branch = branch * m[doc, case["gate"]]
        out = x if bwd else case["residual_scale"] * x + branch
        h = norm(out, case["pre"])
        if w_pre is not None:
            h = h * w_pre + b_pre
        if case["chunk"] >= 0:
            h = h * (1 + m[doc, 3 * case["chunk"] + 1]) + m[doc, 3 * case["chunk"]]
        if not bwd:
            first[at:at + n], second[at:at + n] = out, h
        else:
            # x holds the forward's x output: first through h, then through the sum
            total = torch.autograd.grad(h, x, s["dh"][at:at + n].double(), retain_graph=True)[0] + s["dx_out"][at:at + n].double()
            leaves = [t for t in (e, w_pre, b_pre, w_post, y) if t is not None]
            g1 = torch.autograd.grad(h, leaves, s["dh"][at:at + n].double(), retain_graph=True, allow_unused=True)
            g2 = torch.autograd.grad(branch, leaves, total, retain_graph=True, allow_unused=True)
            both = [(0 if a is None else a) + (0 if b is None else b) for a, b in zip(g1, g2)]
            names = [k for k, t in (("de", e), ("dw_pre", w_pre), ("db_pre", b_pre), ("dw_post", w_post)) if t is not None]
            for k, v in zip(names, both):
                grads[k] = grads.get(k, 0) + v
            first[at:at + n], second[at:at + n] = case["residual_scale"] * total, both[-1]
        at += n
    if not bwd:
        return dict(x=first, h=second)
    if case["gate"] < 0 and case["chunk"] < 0:
        grads.pop("de")
    return dict(dx=first, dy=second, **grads)


def _exact_attn(s):
    """Document by document and head by head, from the definition of the softmax."""
    case = s["case"]
    H, Hk, d = case["heads"], case["kv_heads"], case["head_dim"]
    q_lens = _ints(case["q_lens"])
    k_lens = _ints(case["k_lens"]) or q_lens
    prefix = _ints(case["prefix"]) or [0] * len(q_lens)
    Tq, Tk, train = s["q"].shape[0], s["k"].shape[0], case["dir"] == "train"
    new = lambda t, w: torch.zeros(t, w, dtype=torch.float64, device="cuda")  # noqa: E731
    o, lse = new(Tq, H * d), new(H, Tq)
    dq, dk, dv = new(Tq, H * d), new(Tk, Hk * d), new(Tk, Hk * d)
    q0 = k0 = 0
    for lq, lk, pre in zip(q_lens, k_lens, prefix):
        qs, ks = slice(q0, q0 + lq), slice(k0, k0 + lk)
        q0, k0 = q0 + lq, k0 + lk
        if lk == 0:
            lse[:, qs] = -math.inf
        if lq == 0 or lk == 0:
            continue
        i, j = torch.arange(lq, device="cuda")[:, None] + lk - lq, torch.arange(lk, device="cuda")
        visible = torch.ones(lq, lk, dtype=torch.bool, device="cuda")
        if case["causal_block"]:
            g = case["causal_block"]
            visible = (torch.div(j, g, rounding_mode="floor") <= torch.div(i, g, rounding_mode="floor")) | (j < pre)
        for h in range(H):
            cols, kcols = slice(h * d, h * d + d), slice(h // (H // Hk) * d, h // (H // Hk) * d + d)
            q, k, v = s["q"][qs, cols].double(), s["k"][ks, kcols].double(), s["v"][ks, kcols].double()
            z = q @ k.T / math.sqrt(d)
            t = None
            if case["cap"]:
                t = torch.tanh(z / case["cap"])
                z = case["cap"] * t
            if s["slopes"] is not None:
                z = z - s["slopes"][h].double() * (i - j).abs()
            z = z.masked_fill(~visible, -math.inf)
            lse[h, qs] = torch.logsumexp(z, 1)
            p = torch.exp(z - lse[h, qs][:, None]).masked_fill(~visible, 0.0)
            o[qs, cols] = p @ v
            if train:
                go = s["do"][qs, cols].double()
                gp = go @ v.T
                gz = p * (gp - (p * gp).sum(1, keepdim=True))
                if t is not None:
                    gz = gz * (1 - t * t)
                gz = gz / math.sqrt(d)
                dq[qs, cols] = gz @ k
                dk[ks, kcols] += gz.T @ q
                dv[ks, kcols] += p.T @ go
    return dict(o=o, lse=lse, dq=dq, dk=dk, dv=dv) if train else dict(o=o, lse=lse)


def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "norm": _exact_norm, "attn": _exact_attn}[case["op"]](s)
