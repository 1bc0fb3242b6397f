"""Plain 64-bit forms of the packed-document operators, with bounds on how far a kernel
that works in the stated types may be off. Every function takes and returns torch float64
tensors (any device); documents are handled one by one.

Bounds: u is half a step of the activation type (bf16 2^-8, fp32 2^-24), f = 2^-24.
They add up, term by term, the roundings that the operators allow: one rounding of each
output, of the probabilities and of the scores' gradients to the activation type (the
tensor-core operands), and fp32 arithmetic elsewhere.
"""
import math

import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
F = 2.0 ** -24


def cu_of(lens, first=0):
    at = [first]
    for n in lens:
        at.append(at[-1] + n)
    return at


# ------------------------------------------------------------------------ rotary positions
def rope_angles(pos, axes, theta=10000.0, scaling="none", factor=(), orig_len=(), fast=32.0, slow=1.0):
    cols = []
    for a, n in enumerate(axes):
        for i in range(n // 2):
            base = theta * factor[a] ** (n / (n - 2)) if scaling == "base" else theta
            f = base ** (-2.0 * i / n)
            if scaling == "linear":
                f /= factor[a]
            if scaling == "ramp":
                keep = min(1.0, max(0.0, (orig_len[a] * f / (2 * math.pi) - slow) / (fast - slow)))
                f = f * keep + f / factor[a] * (1 - keep)
            cols.append(pos[:, a].double() * f)
    return torch.stack(cols, 1)


def rope_forward(x, w, heads, angles, layout, norm, amplitude, eps=1e-6):
    """x [rows, heads*d] float64 (may require grad), w float64 or None."""
    rows, d = x.shape[0], x.shape[1] // heads
    x = x.reshape(rows, heads, d)
    if norm == "head":
        x = x / torch.sqrt((x * x).mean(2, keepdim=True) + eps) * w
    elif norm == "width":
        x = x / torch.sqrt((x * x).mean((1, 2), keepdim=True) + eps) * w.reshape(heads, d)
    n = angles.shape[1]
    c, s = (angles.cos() * amplitude)[:, None], (angles.sin() * amplitude)[:, None]
    if layout == "interleaved":
        a, b = x[..., 0:2 * n:2], x[..., 1:2 * n:2]
        turned = torch.stack((a * c - b * s, a * s + b * c), -1).reshape(rows, heads, 2 * n)
    else:
        a, b = x[..., :n], x[..., n:2 * n]
        turned = torch.cat((a * c - b * s, a * s + b * c), -1)
    return torch.cat((turned, x[..., 2 * n:]), -1).reshape(rows, heads * d)


# ------------------------------------------------------------------------ residual and norms
def _norm(t, kind, eps=1e-6):
    if kind == "none":
        return t
    if kind == "layer":
        t = t - t.mean(1, keepdim=True)
    return t / torch.sqrt((t * t).mean(1, keepdim=True) + eps)


def residual_branch(y, m, gate, post, w_post):
    b = _norm(y, post)
    if w_post is not None:
        b = b * w_post
    return b * m[gate] if gate >= 0 else b


def residual_norm_out(x, m, chunk, pre, w_pre, b_pre):
    h = _norm(x, pre)
    if w_pre is not None:
        h = h * w_pre
    if b_pre is not None:
        h = h + b_pre
    return h * (1 + m[3 * chunk + 1]) + m[3 * chunk] if chunk >= 0 else h


# ------------------------------------------------------------------------ attention
def visible(lq, lk, block, prefix, device):
    """[lq, lk]: query i sees key j."""
    i = torch.arange(lq, device=device)[:, None] + lk - lq
    j = torch.arange(lk, device=device)[None, :]
    if block == 0:
        return torch.ones(lq, lk, dtype=torch.bool, device=device)
    return ((j // block) <= torch.div(i, block, rounding_mode="floor")) | (j < prefix)


def attention(q, k, v, heads, kv_heads, cu_q, cu_k, act, do=None, block=0, prefix=None, cap=0.0, slopes=None,
              scale=0.0):
    """Outputs and bounds: dict name -> (value, bound); rows of no document hold NaN in
    both. q, k, v, do float64 (the values that the kernel was given)."""
    u, dev = U[act], q.device
    d = q.shape[1] // heads
    scale = scale or d ** -0.5
    new = lambda r, w: torch.full((r, w), math.nan, dtype=torch.float64, device=dev)  # noqa: E731
    names = ["o"] + (["dq", "dk", "dv"] if do is not None else [])
    shape = {"o": q.shape, "dq": q.shape, "dk": k.shape, "dv": k.shape}
    val, tol = {n: new(*shape[n]) for n in names}, {n: new(*shape[n]) for n in names}
    val["lse"], tol["lse"] = new(heads, q.shape[0]), new(heads, q.shape[0])
    group = heads // kv_heads
    for doc in range(len(cu_q) - 1):
        qs, ks = slice(cu_q[doc], cu_q[doc + 1]), slice(cu_k[doc], cu_k[doc + 1])
        lq, lk = qs.stop - qs.start, ks.stop - ks.start
        if do is not None:
            for n in ("dk", "dv"):
                val[n][ks], tol[n][ks] = 0.0, 0.0
        see = visible(lq, lk, block, prefix[doc] if prefix is not None else 0, dev)
        empty = ~see.any(1) if lk else torch.ones(lq, dtype=torch.bool, device=dev)
        far = (torch.arange(lq, device=dev)[:, None] + lk - lq - torch.arange(lk, device=dev)[None]).abs().double()
        for h in range(heads):
            c, kc = slice(h * d, h * d + d), slice(h // group * d, h // group * d + d)
            Q, K, V = q[qs, c], k[ks, kc], v[ks, kc]
            z = Q @ K.T * scale
            # fp32 dot product of d terms, its scaling and what follows; a tanh within 2^-20 of
            # the cap (its exponential and division are within a few units of fp32)
            dz = (d + 8) * F * scale * (Q.abs() @ K.abs().T)
            turn = torch.ones_like(z)
            if cap:
                t = torch.tanh(z / cap)
                z, turn = cap * t, 1 - t * t
                dz = dz + cap * 2.0 ** -20
            if slopes is not None:
                z = z - slopes[h] * far
                dz = dz + 4 * F * slopes[h] * far
            dz = dz + 4 * F * z.abs()
            z = z.masked_fill(~see, -math.inf)
            lse = torch.logsumexp(z, 1) if lk else torch.full((lq,), -math.inf, dtype=torch.float64, device=dev)
            safe = torch.where(empty, torch.zeros_like(lse), lse)
            p = torch.exp(z - safe[:, None]).masked_fill(~see, 0.0)
            dz = dz.masked_fill(~see, 0.0)
            # relative error of a probability: its score's, the row sum's (a mean of the scores'
            # errors) and the exponentials'; `u` more once it is rounded to an operand
            rel = dz + (p * dz).sum(1, keepdim=True) + 2.0 ** -20
            O = p @ V
            tol_o = u * O.abs() + (p * (rel + (u if u > F else 0.0))) @ V.abs() + (lk + 4) * F * (p @ V.abs())
            val["o"][qs, c], tol["o"][qs, c] = O, tol_o
            val["lse"][h, qs] = lse
            tol["lse"][h, qs] = torch.where(empty, 0.0, (p * dz).sum(1) + 2.0 ** -19 + 4 * F * safe.abs())
            if do is None:
                continue
            G = do[qs, c]
            dp = G @ V.T
            delta = (p * dp).sum(1, keepdim=True)
            ds = p * (dp - delta) * turn
            mag = G.abs() @ V.abs().T
            # the kernel's delta is the sum of do times the o that it was given
            tol_delta = (G.abs() * tol_o).sum(1, keepdim=True) + (d + 4) * F * (G.abs() * O.abs()).sum(1, keepdim=True)
            lse_rel = dz + tol["lse"][h, qs][:, None] + 2.0 ** -20
            e_ds = (p * turn * ((d + 4) * F * mag + tol_delta) + lse_rel * ds.abs() + (u if u > F else 4 * F) * ds.abs())
            if cap:  # 1 - t^2 from a t within 2^-20
                e_ds = e_ds + p * (dp - delta).abs() * 2.0 ** -18
            val["dq"][qs, c] = ds @ K * scale
            tol["dq"][qs, c] = scale * (e_ds @ K.abs() + (lk + 4) * F * (ds.abs() @ K.abs()))
            val["dk"][ks, kc] += ds.T @ Q * scale
            tol["dk"][ks, kc] += scale * (e_ds.T @ Q.abs() + (lq * group + 4) * F * (ds.abs().T @ Q.abs()))
            val["dv"][ks, kc] += p.T @ G
            tol["dv"][ks, kc] += (p * (lse_rel + (u if u > F else 0.0))).T @ G.abs() + (lq * group + 4) * F * (p.T @ G.abs())
    for n in names[1:]:
        tol[n] += u * val[n].abs()  # the output's rounding
    return {n: (val[n], tol[n]) for n in val}


def assert_close(got, value, bound, name, untouched=7.0):
    """Entries with a value lie within the bound; entries of no document still hold
    `untouched`; -inf has to be met exactly."""
    got, none = got.double(), torch.isnan(value)
    assert (got[none] == untouched).all(), f"{name}: rows of no document were written"
    inf = torch.isinf(value)
    assert (got[inf] == value[inf]).all(), f"{name}: infinities differ"
    rest = ~none & ~inf
    err = (got[rest] - value[rest]).abs()
    bad = ~(err <= bound[rest] + 1e-30)
    assert not bad.any(), (f"{name}: {int(bad.sum())} of {bad.numel()} values off, worst {float((err / (bound[rest] + 1e-30)).max()):.2f} "
                           f"bounds, error {float(err.max()):.3e}")
