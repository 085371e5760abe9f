"""The operators of a training step around PACK3D attention, as they are measured: layer norm,
cross attention to states of another length, and the global gradient norm with clipping.

A case is one pass through one operator: a plain dict with its name under "op" ("norm", "norm_train",
"cross", "cross_train", "clip") and its sizes. `run` computes it with elementary torch operations in
32 bits, or, when `own` is true, with the calls of geometry_aware_local_pack3d_b200.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4}
EPS = 1e-5


def listed():
    return [
        # the norm of every head's q rows before the field's rotation (65,536 tokens, 2 x 8 heads)
        dict(name="norm q rows of 96", op="norm", rows=1048576, cols=96, dtype="bf16", wtype="f32"),
        # the norm of a tiny field's tokens (8 x 8 x 8): the smallest call
        dict(name="norm 512 tokens f32", op="norm", rows=512, cols=384, dtype="f32", wtype="f32"),
        # the pre-norm of a 65,536-token field of 8 heads of 96, batch of 2, in a training step
        dict(name="norm train field 65k", op="norm_train", rows=131072, cols=768, dtype="bf16", wtype="f32"),
        # a ragged set of rows of an odd width
        dict(name="norm train odd f32", op="norm_train", rows=4099, cols=1001, dtype="f32", wtype="f32"),
        # a field's tokens attend to a coarser field's 1,024 states
        dict(name="cross field to 1024 states", op="cross", batch=2, heads=8, kv_heads=8, n=65536, l=1024,
             d=96, dtype="bf16", mask="none"),
        # a field conditioned on a short padded sequence
        dict(name="cross field to 77 padded", op="cross", batch=2, heads=8, kv_heads=4, n=32768, l=77,
             d=96, dtype="bf16", mask="pad"),
        # a single token of each of 8 sequences reads a long encoder output
        dict(name="cross one token", op="cross", batch=8, heads=8, kv_heads=2, n=1, l=16384, d=96,
             dtype="bf16", mask="pad"),
        # a training step over a field of 32^3 and an encoder's ragged states
        dict(name="cross train 32k to 500", op="cross_train", batch=2, heads=8, kv_heads=8, n=32768, l=500,
             d=96, dtype="bf16", mask="pad"),
        # the same over a short padded sequence, shared heads
        dict(name="cross train 65k to 77", op="cross_train", batch=1, heads=8, kv_heads=4, n=65536, l=77,
             d=48, dtype="bf16", mask="pad"),
        # the 32-bit path, odd lengths, states left out at random
        dict(name="cross train f32", op="cross_train", batch=1, heads=4, kv_heads=2, n=1000, l=333, d=48,
             dtype="f32", mask="random"),
        # the gradients of a large model, 16-bit and 32-bit buckets
        dict(name="clip 300 tensors", op="clip", tensors=300, numel=150000000, dtype="mixed", factor=0.1),
        # the gradients of one small layer
        dict(name="clip 12 tensors", op="clip", tensors=12, numel=1200000, dtype="f32", factor=0.5),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case: rows 1 to 10^6 and widths 1 to 8,192; fields of 1 to 65,536 tokens against 1 to
    16,384 states; 1 to 300 gradients of up to 150 million numbers in all."""
    op = rng.choice(["norm", "norm_train", "cross", "cross", "cross_train", "cross_train", "clip"])
    if op in ("norm", "norm_train"):
        cols = rng.choice([48, 64, 96, 128, 384, 768, _log(rng, 1, 8192), _log(rng, 1, 8192)])
        rows = _log(rng, 1, max(1, min(1000000, 100000000 // cols)))
        return dict(op=op, rows=rows, cols=cols, dtype=rng.choice(["bf16", "f32"]), wtype=rng.choice(["bf16", "f32"]))
    if op == "clip":
        return dict(op=op, tensors=_log(rng, 1, 300), numel=_log(rng, 1000, 150000000),
                    dtype=rng.choice(["bf16", "f32", "mixed"]), factor=rng.choice([0.1, 0.5, 2.0]))
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    d = rng.choice([48, 96, 64, 128])
    kv_heads = rng.choice([1, 2, 4, 8])
    heads = kv_heads * rng.choice([1, 1, 2, 4])
    batch = rng.choice([1, 2, 3, 8])
    n, l = rng.choice([1, _log(rng, 1, 65536), _log(rng, 64, 65536)]), _log(rng, 1, 16384)
    # no more than the listed cases' work, and less of it in 32 bits
    most = 4.0 * 8 * 65536 * 77 * 96 if dtype == "f32" else 4.0 * 16 * 65536 * 512 * 96
    most /= 3.5 if op == "cross_train" else 1.0
    while 4.0 * batch * heads * n * l * d > most:
        if batch > 1:
            batch = 1
        elif n > l:
            n = max(1, n // 2 + rng.choice([0, 1]))
        else:
            l = max(1, l // 2 + rng.choice([0, 1]))
    return dict(op=op, batch=batch, heads=heads, kv_heads=kv_heads, n=n, l=l, d=d, dtype=dtype,
                mask=rng.choice(["none", "pad", "random"]))


def _sizes(case):
    """The lengths of the gradients: a few large ones, many small ones, odd ones among them."""
    n, total = case["tensors"], case["numel"]
    w = [1.0 / (1 + (7 * i) % n) for i in range(n)]
    s = sum(w)
    return [max(1, int(total * x / s) | (i & 1)) for i, x in enumerate(w)]


def _normal(gen, *shape, dtype, std=1.0):
    return (torch.randn(*shape, generator=gen, device="cuda") * std).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, s = case["op"], dict(case=case)
    if op in ("norm", "norm_train"):
        dt, wt = TYPES[case["dtype"]], TYPES[case["wtype"]]
        r, c = case["rows"], case["cols"]
        # activations with an offset and rows of different size, as residual streams have
        size = 0.5 + 3.0 * torch.rand(r, 1, generator=gen, device="cuda")
        s["x"] = (torch.randn(r, c, generator=gen, device="cuda") * size + 0.3).to(dt)
        s["w"] = (1.0 + _normal(gen, c, dtype=torch.float32, std=0.2)).to(wt)
        s["b"] = _normal(gen, c, dtype=wt, std=0.2)
        if op == "norm_train":
            s["dy"] = _normal(gen, r, c, dtype=dt)
    elif op in ("cross", "cross_train"):
        dt = TYPES[case["dtype"]]
        b, h, hk, n, l, d = (case[k] for k in ("batch", "heads", "kv_heads", "n", "l", "d"))
        s["q"] = _normal(gen, b, h, n, d, dtype=dt)
        s["k"] = _normal(gen, b, hk, l, d, dtype=dt)
        s["v"] = _normal(gen, b, hk, l, d, dtype=dt)
        at = torch.arange(l, device="cuda")
        if case["mask"] == "pad":  # every sequence has a length of its own, from one half up
            lens = torch.randint((l + 1) // 2, l + 1, (b, 1), generator=gen, device="cuda")
            s["mask"] = at < lens
        elif case["mask"] == "random":
            s["mask"] = torch.rand(b, l, generator=gen, device="cuda") < 0.7
        else:
            s["mask"] = None
        if op == "cross_train":
            s["dO"] = _normal(gen, b, h, n, d, dtype=dt)
    else:
        # gradient buckets: one per type, the gradients views of it at 16-byte boundaries
        sizes, kind = _sizes(case), case["dtype"]
        types = ["bf16", "f32"] if kind == "mixed" else [kind]
        s["flat"], s["out"], s["grads"], s["outs"] = [], [], [], []
        for t, name in enumerate(types):
            mine = sizes[t::len(types)]
            starts, at = [], 0
            for m in mine:
                starts.append(at)
                at += -(-m // 8) * 8
            flat = torch.randn(max(at, 8), generator=gen, device="cuda").mul_(0.01).to(TYPES[name])
            keep = torch.zeros(max(at, 8), dtype=torch.bool, device="cuda")
            for a, m in zip(starts, mine):
                keep[a:a + m] = True
            flat = torch.where(keep, flat, torch.zeros((), dtype=flat.dtype, device="cuda"))
            out = torch.zeros_like(flat)
            s["flat"].append(flat)
            s["out"].append(out)
            s["grads"] += [flat[a:a + m] for a, m in zip(starts, mine)]
            s["outs"] += [out[a:a + m] for a, m in zip(starts, mine)]
        s["max_norm"] = case["factor"] * 0.01 * math.sqrt(sum(sizes))
    return s


def run(s):
    op = s["case"]["op"]
    if own:
        return _own(op, s)
    if op == "norm":
        return _norm(s["x"], s["w"], s["b"])[0]
    if op == "norm_train":
        return _norm_train(s["x"], s["w"], s["b"], s["dy"])
    if op == "cross":
        o, lse = _cross(s["q"], s["k"], s["v"], s["mask"])[:2]
        return dict(o=o.to(s["q"].dtype), lse=lse)
    if op == "cross_train":
        return _cross_train(s["q"], s["k"], s["v"], s["mask"], s["dO"])
    return _clip(s["flat"], s["max_norm"])


def _own(op, s):
    import geometry_aware_local_pack3d_b200 as p3d
    if op == "norm":
        return p3d.pack3d_layer_norm_fwd(s["x"], s["w"], s["b"], eps=EPS)["y"]
    if op == "norm_train":
        f = p3d.pack3d_layer_norm_fwd(s["x"], s["w"], s["b"], eps=EPS, save_for_backward=True)
        g = p3d.pack3d_layer_norm_bwd(s["dy"], s["x"], s["w"], f)
        return dict(y=f["y"], dx=g["dx"], dw=g["dweight"], db=g["dbias"])
    if op == "cross":
        f = p3d.pack3d_cross_attn_fwd(s["q"], s["k"], s["v"], mask=s["mask"], save_for_backward=True)
        return dict(o=f["o"], lse=f["lse"])
    if op == "cross_train":
        f = p3d.pack3d_cross_attn_fwd(s["q"], s["k"], s["v"], mask=s["mask"], save_for_backward=True)
        g = p3d.pack3d_cross_attn_bwd(s["q"], s["k"], s["v"], f, s["dO"], mask=s["mask"])
        return dict(o=f["o"], dq=g["dq"], dk=g["dk"], dv=g["dv"])
    norm = p3d.pack3d_clip_grad_norm(s["grads"], s["max_norm"], outs=s["outs"])
    return dict(norm=norm, out=s["out"])


# ------------------------------------------------------------------------------ plain forms
def _norm(x, w, b):
    xf = x.float()
    mean = xf.mean(1, keepdim=True)
    xc = xf - mean
    rstd = 1.0 / torch.sqrt((xc * xc).mean(1, keepdim=True) + EPS)
    xh = xc * rstd
    return (xh * w.float() + b.float()).to(x.dtype), xh, rstd


def _norm_train(x, w, b, dy):
    y, xh, rstd = _norm(x, w, b)
    dyf = dy.float()
    g = dyf * w.float()
    dx = rstd * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    # a column's sum runs over up to a million rows
    dw = (dyf * xh).sum(0, dtype=torch.float64)
    db = dyf.sum(0, dtype=torch.float64)
    return dict(y=y, dx=dx.to(x.dtype), dw=dw.to(w.dtype), db=db.to(w.dtype))


def _cross(q, k, v, mask):
    """o and lse in 32 bits, the probabilities and the operands. The query heads of one KV head are
    rows of one product."""
    b, h, n, d = q.shape
    hk, l = k.shape[1], k.shape[2]
    qf = q.float().reshape(b, hk, -1, d)
    kf, vf = k.float(), v.float()
    x = torch.matmul(qf, kf.transpose(2, 3)) * (1.0 / math.sqrt(d))
    if mask is not None:
        x = x.masked_fill(~mask[:, None, None, :], float("-inf"))
    m = x.max(3, keepdim=True).values
    m = torch.where(m == float("-inf"), torch.zeros_like(m), m)  # a row with no state
    e = torch.exp(x - m)
    t = e.sum(3, keepdim=True)
    lse = (torch.log(t) + m).reshape(b, h, n)
    p = e / torch.where(t == 0, torch.ones_like(t), t)
    o = torch.matmul(p, vf)
    return o.reshape(b, h, n, d), lse, p, qf, kf, vf


def _cross_train(q, k, v, mask, dO):
    o, _, p, qf, kf, vf = _cross(q, k, v, mask)
    scale = 1.0 / math.sqrt(q.shape[3])
    g = dO.float().reshape(qf.shape)
    dv = torch.matmul(p.transpose(2, 3), g)
    dp = torch.matmul(g, vf.transpose(2, 3))
    ds = p * (dp - (g * o.reshape(qf.shape)).sum(3, keepdim=True)) * scale
    dq = torch.matmul(ds, kf).reshape(q.shape)
    dk = torch.matmul(ds.transpose(2, 3), qf)
    return dict(o=o.to(q.dtype), dq=dq.to(q.dtype), dk=dk.to(k.dtype), dv=dv.to(v.dtype))


def _clip(flat, max_norm):
    parts = torch.stack([f.float().square().sum(dtype=torch.float64) for f in flat])
    norm = parts.sum().sqrt().float()
    coef = torch.clamp(max_norm / (norm + 1e-6), max=1.0)
    return dict(norm=norm.reshape(1), out=[(f.float() * coef).to(f.dtype) for f in flat])


# ------------------------------------------------------------------------------- definitions
def exact(case, seed):
    """The outputs from the definitions in 64 bits."""
    s, op = prepare(case, seed), case["op"]
    if op in ("norm", "norm_train"):
        x, w, b = s["x"].double(), s["w"].double(), s["b"].double()
        c = x.shape[1]
        mu = torch.einsum("rc->r", x) / c
        var = torch.einsum("rc,rc->r", x, x) / c - mu ** 2 if c > 1 else torch.zeros_like(mu)
        sd = (var + EPS).sqrt()
        z = (x - mu[:, None]) / sd[:, None]
        y = torch.addcmul(b.expand_as(z), z, w.expand_as(z))
        if op == "norm":
            return y
        dy = s["dy"].double()
        # the Jacobian of z: dz_i/dx_j = (delta_ij - 1/c - z_i z_j / c) / sd
        gz = dy * w
        proj = torch.einsum("rc,rc->r", gz, z) / c
        dx = (gz - (torch.einsum("rc->r", gz) / c)[:, None] - z * proj[:, None]) / sd[:, None]
        return dict(y=y, dx=dx, dw=torch.einsum("rc,rc->c", dy, z), db=torch.einsum("rc->c", dy))
    if op in ("cross", "cross_train"):
        return _exact_cross(s, op)
    sq = sum(float((f.double() ** 2).sum()) for f in s["flat"])
    norm = math.sqrt(sq)
    by = min(1.0, s["max_norm"] / (norm + 1e-6))
    return dict(norm=torch.tensor([norm], dtype=torch.float64), out=[f.double() * by for f in s["flat"]])


def _exact_cross(s, op):
    """One batch and head at a time, over its unmasked states alone."""
    q, k, v = (s[n].double() for n in "qkv")
    b, h, n, d = q.shape
    group, tau = h // k.shape[1], d ** -0.5
    o, lse = torch.zeros_like(q), torch.full((b, h, n), -math.inf, dtype=q.dtype, device=q.device)
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    for i in range(b):
        at = torch.arange(k.shape[2], device=q.device)
        if s["mask"] is not None:
            at = at[s["mask"][i]]
        if at.numel() == 0:
            continue
        for j in range(h):
            kj, vj = k[i, j // group, at], v[i, j // group, at]
            logits = tau * (q[i, j] @ kj.T)
            lse[i, j] = torch.logsumexp(logits, 1)
            p = torch.exp(logits - lse[i, j][:, None])
            o[i, j] = p @ vj
            if op == "cross_train":
                g = s["dO"][i, j].double()
                dp = g @ vj.T
                ds = p * (dp - (p * dp).sum(1, keepdim=True))
                dq[i, j] = tau * (ds @ kj)
                dk[i, j // group, at] += tau * (ds.T @ q[i, j])
                dv[i, j // group, at] += p.T @ g
    if op == "cross":
        return dict(o=o, lse=lse)
    return dict(o=o, dq=dq, dk=dk, dv=dv)


def work(case):
    op = case["op"]
    if op in ("norm", "norm_train"):
        n, e, w = case["rows"] * case["cols"], BYTES[case["dtype"]], BYTES[case["wtype"]] * case["cols"]
        if op == "norm":
            return dict(bytes=2 * n * e + 2 * w, flops=8 * n)
        return dict(bytes=4 * n * e + 4 * w, flops=22 * n)
    if op in ("cross", "cross_train"):
        e = BYTES[case["dtype"]]
        nq = case["batch"] * case["heads"] * case["n"]
        nk = case["batch"] * case["kv_heads"] * case["l"]
        keep = {"none": 1.0, "pad": 0.75, "random": 0.7}[case["mask"]]  # states that take part
        d = case["d"]
        prod = 2.0 * nq * case["l"] * keep * d
        if op == "cross":
            return dict(bytes=2 * nq * d * e + 4 * nq + 2 * nk * keep * d * e, flops=2 * prod)
        return dict(bytes=4 * nq * d * e + 2 * nk * (1 + keep) * d * e, flops=7 * prod)
    sizes, kind = _sizes(case), case["dtype"]
    bytes_ = sum(m * (2 if kind == "bf16" or (kind == "mixed" and i % 2 == 0) else 4) for i, m in enumerate(sizes))
    return dict(bytes=2 * bytes_, flops=3 * sum(sizes))
