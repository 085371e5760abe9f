"""The operators as a training step of a conditioned block runs them: norms of the heads' q and k
rows, PACK3D attention, a norm of its output, cross attention to states of another length, the
backward of all of it and the clipping of every gradient; against a dense float64 formulation
through torch.autograd."""
import math

import pytest
import torch

import inputs
from . import dense_reference as dr

pytestmark = pytest.mark.gpu

EPS = 1e-5
# the bars that hold for the PACK3D layer alone (tests/test_gpu_parity.py): float32 1e-4 absolute
# and bfloat16 5e-3 in relative L2; three more operators in the chain each add a rounding of their
# own (2^-9 rms of a bfloat16 value), so four times the square root: sqrt(4) times the layer's bar
F32_TOL, BF16_REL = 2e-4, 1e-2


def leaves(w, dtype, L, hkv):
    gen = torch.Generator().manual_seed(21)
    d, B, H = w["d"], w["batch"], w["heads"]
    rnd = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    t = dict(q=w["q"], k=w["k"], v=w["v"], a=w["a"], kc=rnd(B, hkv, L, d), vc=rnd(B, hkv, L, d))
    t = {n: x.to(dtype) for n, x in t.items()}
    for n in ("wq", "wk", "wo"):
        t[n] = 1 + 0.2 * rnd(d)
    for n in ("bq", "bk", "bo"):
        t[n] = 0.2 * rnd(d)
    mask = torch.arange(L)[None] < torch.tensor([[L], [L // 3], [1]])[:B]
    dO = rnd(B, H, w["q"].shape[2], d).to(dtype)
    return t, mask, dO


def dense(t, mask, dO, w, max_norm):
    x = {n: y.double().requires_grad_() for n, y in t.items()}
    d = w["d"]
    normed = {}

    def norm(y, a, b):
        normed[a] = torch.nn.functional.layer_norm(y, (d,), x[a], x[b], EPS)
        normed[a].retain_grad()
        return normed[a]

    o = dr.pack3d_dense(norm(x["q"], "wq", "bq"), norm(x["k"], "wk", "bk"), x["v"], x["a"], w["coords"],
                        w["grid"], w["block"])["o"]
    h = norm(o, "wo", "bo")
    G = h.shape[1] // t["kc"].shape[1]
    kc, vc = x["kc"].repeat_interleave(G, 1), x["vc"].repeat_interleave(G, 1)
    s = (h @ kc.transpose(2, 3)) / math.sqrt(d)
    y = torch.softmax(s.masked_fill(~mask[:, None, None, :], -math.inf), 3) @ vc
    (y * dO.double()).sum().backward()
    g = {n: z.grad for n, z in x.items()}
    total = math.sqrt(sum(float((z ** 2).sum()) for z in g.values()))
    c = min(1.0, max_norm / (total + 1e-6))
    # the rows that a weight's or bias's gradient sums
    rows = {p + n[1]: float(z.grad.norm()) * c for n, z in normed.items() for p in "wb"}
    return y.detach(), {n: z * c for n, z in g.items()}, total, rows


def on_gpu(t, mask, dO, w, max_norm):
    import geometry_aware_local_pack3d_b200 as p3d
    x = {n: y.cuda().contiguous() for n, y in t.items()}
    mask, dO = mask.cuda(), dO.cuda()
    ix = p3d.pack3d_build_index(p3d.make_geom(w["grid"], w["block"], w["d"]),
                                coords=torch.from_numpy(w["coords"]).cuda())
    fq = p3d.pack3d_layer_norm_fwd(x["q"], x["wq"], x["bq"], eps=EPS, save_for_backward=True)
    fk = p3d.pack3d_layer_norm_fwd(x["k"], x["wk"], x["bk"], eps=EPS, save_for_backward=True)
    ksum, vsum = p3d.pack3d_summarize(ix, fk["y"], x["v"])
    fa = p3d.pack3d_attn_fwd(ix, fq["y"], fk["y"], x["v"], x["a"], ksum, vsum, save_for_backward=True)
    fo = p3d.pack3d_layer_norm_fwd(fa["o"], x["wo"], x["bo"], eps=EPS, save_for_backward=True)
    fc = p3d.pack3d_cross_attn_fwd(fo["y"], x["kc"], x["vc"], mask=mask, save_for_backward=True, status=ix)
    gc = p3d.pack3d_cross_attn_bwd(fo["y"], x["kc"], x["vc"], fc, dO, mask=mask, status=ix)
    go = p3d.pack3d_layer_norm_bwd(gc["dq"], fa["o"], x["wo"], fo)
    ga = p3d.pack3d_attn_bwd(ix, fq["y"], fk["y"], x["v"], x["a"], ksum, vsum, fa, go["dx"])
    gq = p3d.pack3d_layer_norm_bwd(ga["dq"], x["q"], x["wq"], fq)
    gk = p3d.pack3d_layer_norm_bwd(ga["dk"], x["k"], x["wk"], fk)
    g = dict(q=gq["dx"], k=gk["dx"], v=ga["dv"], a=ga["dgate"], kc=gc["dk"], vc=gc["dv"],
             wq=gq["dweight"], bq=gq["dbias"], wk=gk["dweight"], bk=gk["dbias"], wo=go["dweight"],
             bo=go["dbias"])
    total = p3d.pack3d_clip_grad_norm(list(g.values()), max_norm)
    assert p3d.pack3d_device_status(ix) == 0
    return fc["o"], g, total


@pytest.mark.parametrize("dtype,d,grid,hkv", [("fp32", 48, (4, 4, 8), 2), ("bf16", 96, (8, 8, 8), 1)])
def test_block_step_forward_backward_and_clip(dtype, d, grid, hkv):
    cfg = dict(grid=grid, block=(2, 2, 4), batch=3, heads=2, d=d, dtype=dtype, packing="random", qkv_std=1.0,
               exclude_near=False)
    w = inputs.make_workload(cfg)
    tt = torch.float32 if dtype == "fp32" else torch.bfloat16
    t, mask, dO = leaves(w, tt, 75, hkv)
    _, _, total0, _ = dense(t, mask, dO, w, math.inf)
    y, g, total, rows = dense(t, mask, dO, w, 0.5 * total0)  # clipping halves everything
    y1, g1, total1 = on_gpu(t, mask, dO, w, 0.5 * total0)
    torch.cuda.synchronize()
    assert abs(float(total1) - total) <= (1e-5 if dtype == "fp32" else BF16_REL) * total
    for n, want, got in [("y", y, y1)] + [(n, g[n], g1[n]) for n in g]:
        got = got.double().cpu()
        if dtype == "fp32":
            # weights' gradients sum thousands of rows: the bar is relative to their size there
            err = float((got - want).abs().max()) / max(1.0, float(want.abs().max()))
            assert err <= F32_TOL, (n, err)
        else:
            # A weight's or bias's gradient is a sum over rows y_r that nearly cancel (a shift of
            # every key hardly moves a softmax). Rows that are off by e_r, |e| <= BF16_REL |y|, put
            # it off by |sum e_r|; roundings of different rows are independent, so that is
            # sqrt(sum |e_r|^2) = |e| <= BF16_REL |y|: relative to the rows, not to what is left.
            rel = float((got - want).norm()) / max(float(want.norm()), rows.get(n, 0.0))
            assert rel <= BF16_REL, (n, rel)
