"""The global gradient norm and clipping on the GPU against float64."""
import math

import pytest
import torch

from . import ops_bounds as ob

pytestmark = pytest.mark.gpu


def p3d():
    import geometry_aware_local_pack3d_b200 as m
    return m


def make(sizes, seed=0, std=1.0, types=(torch.bfloat16, torch.float32)):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return [(std * torch.randn(n, generator=gen, device="cuda")).to(types[i % len(types)])
            for i, n in enumerate(sizes)]


def run_and_check(grads, max_norm):
    before = [g.clone() for g in grads]
    norm, bound, outs = ob.clip(grads, max_norm)
    n0 = p3d().pack3d_grad_norm(grads)
    assert abs(float(n0) - norm) <= bound
    to = [torch.full_like(g, 9.0) for g in grads]
    n1 = p3d().pack3d_clip_grad_norm(grads, max_norm, outs=to)
    assert torch.equal(n0, n1)
    for i, (g, want) in enumerate(zip(to, outs)):
        ob.check(g, want, f"out {i}")
    assert all(torch.equal(a, b) for a, b in zip(before, grads))
    n2 = p3d().pack3d_clip_grad_norm(grads, max_norm)  # in place
    assert torch.equal(n0, n2)
    assert all(torch.equal(a, b) for a, b in zip(to, grads))


@pytest.mark.parametrize("sizes", [[1], [7, 0, 3], [16384], [100000, 1, 5, 4097, 33333], [10] * 700,
                                   [2000000, 77, 500001]])
@pytest.mark.parametrize("factor", [0.3, 5.0])
def test_sizes(sizes, factor):
    run_and_check(make(sizes), factor * math.sqrt(sum(sizes)))


@pytest.mark.parametrize("shift_g,shift_o", [(1, 1), (3, 3), (1, 2), (0, 5)])
def test_views_at_any_element(shift_g, shift_o):
    for dt in (torch.bfloat16, torch.float32):
        flat, out = make([50000 + 16], types=(dt,))[0], torch.full((50000 + 16,), 4.0, dtype=dt, device="cuda")
        g, o = flat[shift_g:shift_g + 50000], out[shift_o:shift_o + 50000]
        norm, bound, want = ob.clip([g], 10.0)
        n = p3d().pack3d_clip_grad_norm([g], 10.0, outs=[o])
        assert abs(float(n) - norm) <= bound
        ob.check(o, want[0], "out")
        assert bool((out[:shift_o] == 4.0).all()) and bool((out[shift_o + 50000:] == 4.0).all())


@pytest.mark.parametrize("std", [1e-30, 1e-18, 1e18, 3e36])
def test_squares_outside_the_range_of_fp32(std):
    g = make([5000, 3000], std=std)
    norm, bound, _ = ob.clip(g, 1.0)
    assert abs(float(p3d().pack3d_grad_norm(g)) - norm) <= bound


def test_infinite_and_nan_norms_scale_as_the_formula_says():
    g = make([100], types=(torch.float32,))
    g[0][5] = float("inf")
    n = p3d().pack3d_clip_grad_norm(g, 1.0)
    assert float(n) == math.inf and bool(g[0][5].isnan())
    assert bool((torch.cat([g[0][:5], g[0][6:]]) == 0).all())
    g = make([100], types=(torch.float32,))
    g[0][5] = float("nan")
    n = p3d().pack3d_clip_grad_norm(g, 1.0)
    assert math.isnan(float(n)) and bool(g[0].isnan().all())


def test_no_tensors_zero_gradients_and_a_zero_bound():
    assert float(p3d().pack3d_grad_norm([], device="cuda")) == 0.0
    assert float(p3d().pack3d_clip_grad_norm([], 1.0, device="cuda")) == 0.0
    z = [torch.zeros(1000, device="cuda")]
    assert float(p3d().pack3d_clip_grad_norm(z, 1.0)) == 0.0 and not bool(z[0].any())
    g = make([1000])
    p3d().pack3d_clip_grad_norm(g, 0.0)
    assert not bool(g[0].any())


def test_overlapping_tensors_are_refused():
    m = p3d()
    g = make([1000], types=(torch.float32,))[0]
    before = g.clone()
    for grads, outs in (([g, g], None), ([g[:600], g[500:]], None), ([g[:500]], [g[100:600]]),
                        ([g[:100], g[500:600]], [g[100:200], g[550:650]])):
        with pytest.raises(m.Pack3DError) as e:
            m.pack3d_clip_grad_norm(grads, 1.0, outs=outs)
        assert e.value.status == 1
    torch.cuda.synchronize()
    assert torch.equal(g, before)
    # reading a tensor twice is no conflict: it counts twice
    assert abs(float(m.pack3d_grad_norm([g, g])) - float(before.double().norm()) * math.sqrt(2)) < 1e-3


def test_capture_replays_with_new_gradients():
    g = make([40000, 777, 123456])
    out = [torch.empty_like(x) for x in g]
    p3d().pack3d_clip_grad_norm(g, 1.0, outs=out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        n = p3d().pack3d_clip_grad_norm(g, 1.0, outs=out)
    for a, b in zip(g, make([40000, 777, 123456], seed=6)):
        a.copy_(b)
    graph.replay()
    torch.cuda.synchronize()
    norm, bound, want = ob.clip(g, 1.0)
    assert abs(float(n) - norm) <= bound
    for a, w in zip(out, want):
        ob.check(a, w, "out")
