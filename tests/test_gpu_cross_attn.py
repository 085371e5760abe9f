"""Cross attention on the GPU, forward and backward, against float64 with elementwise bounds
(tests/ops_bounds.py derives them from the roundings)."""
import math

import pytest
import torch

from . import ops_bounds as ob

pytestmark = pytest.mark.gpu


def p3d():
    import geometry_aware_local_pack3d_b200 as m
    return m


def make(B, H, HK, N, L, d, dtype, mask="none", seed=0, garbage=False, spread=1.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    q, dO = (spread * rnd(B, H, N, d)).to(dtype), rnd(B, H, N, d).to(dtype)
    k, v = rnd(B, HK, L, d).to(dtype), rnd(B, HK, L, d).to(dtype)
    at = torch.arange(L, device="cuda")
    if mask == "none":
        m = None
    elif mask == "pad":
        m = at < torch.randint(0, L + 1, (B, 1), generator=gen, device="cuda")
    elif mask == "left":
        m = at >= torch.randint(0, L + 1, (B, 1), generator=gen, device="cuda")
    elif mask == "random":
        m = torch.rand(B, L, generator=gen, device="cuda") < 0.6
    elif mask == "sparse":  # whole tiles of 128 states without one that takes part
        m = (torch.rand(B, L, generator=gen, device="cuda") < 0.02) & ((at // 128) % 3 != 1)
    elif mask == "empty":   # the first entry has no state, the last has one
        m = torch.zeros(B, L, dtype=torch.bool, device="cuda")
        m[-1, L // 2] = True
    if garbage and m is not None:
        off = ~m[:, None, :, None]
        bad = torch.tensor([float("nan"), float("inf"), -float("inf"), 3e38], device="cuda").to(dtype)
        fill = bad[torch.arange(L * d, device="cuda").reshape(1, 1, L, d) % 4]
        k, v = torch.where(off, fill, k), torch.where(off, fill, v)
    return q.contiguous(), k.contiguous(), v.contiguous(), m, dO.contiguous()


def run_and_check(q, k, v, m, dO, backward=True, scale=None):
    f = p3d().pack3d_cross_attn_fwd(q, k, v, mask=m, scale=scale, save_for_backward=True)
    want = ob.cross(q, k, v, m, scale, dO if backward else None)
    ob.check(f["o"], want["o"], "o")
    ob.check(f["lse"], want["lse"], "lse")
    if backward:
        g = p3d().pack3d_cross_attn_bwd(q, k, v, f, dO, mask=m, scale=scale)
        for n in ("dq", "dk", "dv"):
            ob.check(g[n], want[n], n)
        return f, g
    return f, None


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d", [48, 64, 96, 128])
@pytest.mark.parametrize("N,L", [(1, 1), (128, 128), (257, 129), (63, 300)])
def test_head_dims_and_tile_edges(dtype, d, N, L):
    run_and_check(*make(2, 2, 2, N, L, d, dtype))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("mask", ["pad", "left", "random", "sparse", "empty"])
@pytest.mark.parametrize("L", [77, 500])
def test_masks_and_what_masked_states_hold(dtype, mask, L):
    run_and_check(*make(3, 4, 2, 130, L, 96 if L == 77 else 48, dtype, mask, garbage=True))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("H,HK", [(8, 8), (8, 2), (6, 1), (3, 3)])
def test_shared_heads(dtype, H, HK):
    run_and_check(*make(2, H, HK, 75, 200, 48, dtype, "random", seed=3))


@pytest.mark.parametrize("B,H,HK,N,L,mask", [
    (1, 8, 2, 1, 5000, "none"), (2, 4, 4, 1, 4097, "pad"), (1, 2, 1, 3, 16384, "sparse"),
    (3, 1, 1, 200, 2049, "random"), (1, 1, 1, 1, 256, "empty")])
def test_few_rows_over_a_long_context(B, H, HK, N, L, mask):
    # the states are split over CTAs and the splits joined
    q, k, v, m, dO = make(B, H, HK, N, L, 96, torch.bfloat16, mask, seed=5, garbage=True)
    f, g = run_and_check(q, k, v, m, dO)
    again = p3d().pack3d_cross_attn_fwd(q, k, v, mask=m, save_for_backward=True)
    assert torch.equal(f["o"], again["o"]) and torch.equal(f["lse"], again["lse"])


@pytest.mark.parametrize("d", [48, 64, 96, 128])
@pytest.mark.parametrize("B,H,HK,N,L,mask", [
    (2, 6, 3, 8, 129, "random"),     # 16 rows, the largest count with a kernel of its own
    (1, 17, 1, 1, 300, "pad"),       # 17 rows: the general one
    (3, 5, 1, 1, 4099, "left"), (2, 2, 2, 2, 1024, "empty"),
    (40, 8, 8, 1, 4500, "random")])  # more states than a warp lists at once, one block per problem
def test_rows_of_single_tokens(d, B, H, HK, N, L, mask):
    run_and_check(*make(B, H, HK, N, L, d, torch.bfloat16, mask, garbage=True), backward=False)


def test_many_units_per_cta_and_split_row_ranges():
    # more 256-row units than SMs, a last unit of one tile, key gradients over several ranges
    run_and_check(*make(2, 4, 4, 8192 + 100, 260, 96, torch.bfloat16, "pad", seed=7))


@pytest.mark.parametrize("L,d,mask", [(77, 96, "pad"), (64, 48, "none"), (128, 64, "random"), (33, 128, "empty"),
                                      (1, 96, "none")])
def test_short_contexts_stay_in_shared_memory_over_many_units(L, d, mask):
    # every CTA takes a run of row tiles that crosses from problem to problem
    run_and_check(*make(3, 4, 2, 20000, L, d, torch.bfloat16, mask, seed=13, garbage=True))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("spread,scale", [(30.0, None), (1.0, 3.0), (0.01, 0.5)])
def test_peaked_and_flat_rows(dtype, spread, scale):
    # the running reference moves by large steps; nearly one-hot and nearly uniform rows
    run_and_check(*make(1, 2, 2, 200, 700, 64, dtype, spread=spread), scale=scale)


def test_growing_logits_move_the_reference_every_tile():
    q, k, v, m, dO = make(1, 1, 1, 128, 1024, 64, torch.bfloat16)
    q = torch.ones_like(q)
    k = (torch.arange(1024, device="cuda").reshape(1, 1, -1, 1) * 0.02).expand_as(k).to(q.dtype).contiguous()
    run_and_check(q, k, v, m, dO)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_no_rows_and_no_states(dtype):
    q, k, v, _, dO = make(2, 2, 2, 5, 7, 48, dtype)
    e = torch.empty(2, 2, 0, 48, device="cuda", dtype=dtype)
    f = p3d().pack3d_cross_attn_fwd(q, e, e, save_for_backward=True)
    assert torch.equal(f["o"], torch.zeros_like(q)) and bool((f["lse"] == -math.inf).all())
    g = p3d().pack3d_cross_attn_bwd(q, e, e, f, dO)
    assert torch.equal(g["dq"], torch.zeros_like(q)) and g["dk"].numel() == 0
    f = p3d().pack3d_cross_attn_fwd(e, k, v, save_for_backward=True)
    assert f["o"].numel() == 0
    g = p3d().pack3d_cross_attn_bwd(e, k, v, f, e)
    assert torch.equal(g["dk"], torch.zeros_like(k)) and torch.equal(g["dv"], torch.zeros_like(v))


def test_gradient_against_differences():
    # the forward's own output differenced along a random direction (bfloat16 is too coarse to)
    q, k, v, m, dO = make(1, 2, 1, 9, 40, 48, torch.float32, "random", seed=11)
    f = p3d().pack3d_cross_attn_fwd(q, k, v, mask=m, save_for_backward=True)
    g = p3d().pack3d_cross_attn_bwd(q, k, v, f, dO, mask=m)
    gen = torch.Generator(device="cuda").manual_seed(1)
    for name, x in (("dq", q), ("dk", k), ("dv", v)):
        t = torch.randn(x.shape, generator=gen, device="cuda")
        h = 2.0 ** -6
        vals = []
        for s in (h, -h):
            a = {"dq": q, "dk": k, "dv": v, name: x + s * t}
            o = p3d().pack3d_cross_attn_fwd(a["dq"], a["dk"], a["dv"], mask=m)["o"]
            vals.append(float((o.double() * dO.double()).sum()))
        got = (vals[0] - vals[1]) / (2 * h)
        want = float((g[name].double() * t.double()).sum())
        # third-order term h^2 |t|^3 / 6 of a smooth function of unit scale, and fp32 noise / h
        assert abs(got - want) <= 2e-3 * (1 + abs(want)), name


def test_repeated_calls_are_bit_identical_and_leave_inputs_alone():
    q, k, v, m, dO = make(2, 4, 2, 300, 333, 96, torch.bfloat16, "random")
    before = [t.clone() for t in (q, k, v, m, dO)]
    f, g = run_and_check(q, k, v, m, dO)
    f2 = p3d().pack3d_cross_attn_fwd(q, k, v, mask=m, save_for_backward=True)
    g2 = p3d().pack3d_cross_attn_bwd(q, k, v, f2, dO, mask=m)
    for n in ("dq", "dk", "dv"):
        assert torch.equal(g[n], g2[n]), n
    assert torch.equal(f["o"], f2["o"])
    assert all(torch.equal(a, b) for a, b in zip(before, (q, k, v, m, dO)))


@pytest.mark.parametrize("N,L", [(300, 77), (2, 3000)])
def test_capture_and_replay_with_new_inputs(N, L):
    q, k, v, m, dO = make(2, 2, 2, N, L, 96, torch.bfloat16, "random")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        f = p3d().pack3d_cross_attn_fwd(q, k, v, mask=m, save_for_backward=True)
        p3d().pack3d_cross_attn_bwd(q, k, v, f, dO, mask=m)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f = p3d().pack3d_cross_attn_fwd(q, k, v, mask=m, save_for_backward=True)
        g = p3d().pack3d_cross_attn_bwd(q, k, v, f, dO, mask=m)
    q2, k2, v2, m2, dO2 = make(2, 2, 2, N, L, 96, torch.bfloat16, "pad", seed=9)
    for a, b in zip((q, k, v, m, dO), (q2, k2, v2, m2, dO2)):
        a.copy_(b)
    graph.replay()
    torch.cuda.synchronize()
    want = ob.cross(q, k, v, m, None, dO)
    for n, t in (("o", f["o"]), ("lse", f["lse"]), ("dq", g["dq"]), ("dk", g["dk"]), ("dv", g["dv"])):
        ob.check(t, want[n], n)


def test_two_streams_at_once():
    a = make(2, 4, 4, 1000, 300, 96, torch.bfloat16, "random", seed=1)
    b = make(1, 8, 2, 1, 6000, 96, torch.bfloat16, "pad", seed=2)
    refs = [run_and_check(*x) for x in (a, b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [[], []]
    for _ in range(5):
        for i, (x, s) in enumerate(zip((a, b), streams)):
            q, k, v, m, dO = x
            f = p3d().pack3d_cross_attn_fwd(q, k, v, mask=m, save_for_backward=True, stream=s)
            g = p3d().pack3d_cross_attn_bwd(q, k, v, f, dO, mask=m, stream=s)
            outs[i].append((f, g))
    torch.cuda.synchronize()
    for i, (f, g) in enumerate(refs):
        for f2, g2 in outs[i]:
            assert torch.equal(f["o"], f2["o"]) and torch.equal(g["dk"], g2["dk"])
            assert torch.equal(g["dq"], g2["dq"]) and torch.equal(g["dv"], g2["dv"])


def test_given_buffers_are_used_and_a_longer_workspace_is_accepted():
    m3 = p3d()
    q, k, v, m, _ = make(1, 2, 2, 5, 2000, 64, torch.bfloat16, "random")
    need = m3.pack3d_cross_attn_workspace_bytes(1, 1, 2, 2, 5, 2000, 64, True, False)
    ws = torch.full((need + 256,), 255, dtype=torch.uint8, device="cuda")
    o, lse = torch.full_like(q, 7.0), torch.zeros(1, 2, 5, device="cuda")
    f = m3.pack3d_cross_attn_fwd(q, k, v, mask=m, o=o, lse=lse, workspace=ws)
    assert f["o"] is o and f["lse"] is lse
    want = ob.cross(q, k, v, m)
    ob.check(o, want["o"], "o")
    ob.check(lse, want["lse"], "lse")
    assert bool((ws[need:] == 255).all())


def test_rows_behind_the_last_are_left_as_they_were():
    # outputs inside a longer buffer: the copies clip at the last row of each problem
    m3 = p3d()
    q, k, v, m, dO = make(1, 2, 2, 130, 77, 96, torch.bfloat16, "random")
    buf = torch.full((q.numel() + 128 * 96,), 5.0, dtype=q.dtype, device="cuda")
    o = buf[:q.numel()].view_as(q)
    m3.pack3d_cross_attn_fwd(q, k, v, mask=m, o=o)
    torch.cuda.synchronize()
    assert bool((buf[q.numel():] == 5.0).all())
    ob.check(o, ob.cross(q, k, v, m)["o"], "o")


def test_wait_timeout_is_reported_and_the_next_call_is_right():
    m3 = p3d()
    q, k, v, m, dO = make(2, 2, 2, 300, 500, 96, torch.bfloat16, "random")
    f, g = run_and_check(q, k, v, m, dO)
    torch.cuda.synchronize()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for call in ("fwd", "bwd"):
        prev = m3.pack3d_testing_set_wait_budget(1)
        try:
            if call == "fwd":
                m3.pack3d_cross_attn_fwd(q, k, v, mask=m, status=status)
            else:
                m3.pack3d_cross_attn_bwd(q, k, v, f, dO, mask=m, status=status)
            torch.cuda.synchronize()
        finally:
            m3.pack3d_testing_set_wait_budget(prev)
        assert m3.pack3d_read_status(status) == 6, call  # PACK3D_ERR_TIMEOUT, read and cleared
        assert m3.pack3d_read_status(status) == 0
    f2, g2 = run_and_check(q, k, v, m, dO)
    assert torch.equal(f["o"], f2["o"]) and torch.equal(g["dk"], g2["dk"])


@pytest.mark.parametrize("d", [48, 64, 96, 128])
@pytest.mark.parametrize("B,H,HK,N,L,mask", [
    (1, 8, 2, 1, 5000, "none"), (2, 4, 4, 1, 4097, "pad"), (1, 2, 1, 3, 16384, "sparse"),
    (3, 1, 1, 200, 2049, "random"), (2, 1, 1, 1, 300, "empty")])
def test_few_rows_over_a_long_context_f32(d, B, H, HK, N, L, mask):
    # ranges of states in blocks of their own: o and lse joined, dq summed
    q, k, v, m, dO = make(B, H, HK, N, L, d, torch.float32, mask, seed=5, garbage=True)
    f, g = run_and_check(q, k, v, m, dO)
    again = p3d().pack3d_cross_attn_fwd(q, k, v, mask=m, save_for_backward=True)
    assert torch.equal(f["o"], again["o"]) and torch.equal(f["lse"], again["lse"])
    g2 = p3d().pack3d_cross_attn_bwd(q, k, v, f, dO, mask=m)
    assert all(torch.equal(g[n], g2[n]) for n in ("dq", "dk", "dv"))
    # without lse
    o = p3d().pack3d_cross_attn_fwd(q, k, v, mask=m)["o"]
    assert torch.equal(o, f["o"])


@pytest.mark.parametrize("d", [48, 64, 96, 128])
@pytest.mark.parametrize("B,H,HK,N,L,mask", [
    (1, 2, 2, 1, 6000, "none"), (3, 4, 2, 130, 4099, "pad"), (2, 2, 1, 200, 2049, "empty"),
    (2, 3, 3, 1, 8192, "sparse"), (1, 2, 2, 300, 1100, "left")])
def test_gradients_of_few_rows_over_a_long_context(d, B, H, HK, N, L, mask):
    # the rows' gradients summed over ranges of states, some of them without a step
    q, k, v, m, dO = make(B, H, HK, N, L, d, torch.bfloat16, mask, seed=17, garbage=True)
    f, g = run_and_check(q, k, v, m, dO)
    g2 = p3d().pack3d_cross_attn_bwd(q, k, v, f, dO, mask=m)
    assert all(torch.equal(g[n], g2[n]) for n in ("dq", "dk", "dv"))


@pytest.mark.parametrize("N,L", [(300, 77), (3000, 20), (20, 5000)])
def test_wait_timeouts_of_short_contexts_and_split_states(N, L):
    m3 = p3d()
    q, k, v, m, dO = make(3, 4, 2, N, L, 96, torch.bfloat16, "random", seed=23)
    f, g = run_and_check(q, k, v, m, dO)
    torch.cuda.synchronize()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for call in ("fwd", "bwd"):
        prev = m3.pack3d_testing_set_wait_budget(1)
        try:
            if call == "fwd":
                m3.pack3d_cross_attn_fwd(q, k, v, mask=m, status=status)
            else:
                m3.pack3d_cross_attn_bwd(q, k, v, f, dO, mask=m, status=status)
            torch.cuda.synchronize()
        finally:
            m3.pack3d_testing_set_wait_budget(prev)
        assert m3.pack3d_read_status(status) == 6, call
    f2, g2 = run_and_check(q, k, v, m, dO)
    assert torch.equal(f["o"], f2["o"]) and all(torch.equal(g[n], g2[n]) for n in ("dq", "dk", "dv"))


@pytest.mark.parametrize("dtype,N,L", [(torch.float32, 2, 3000), (torch.bfloat16, 40, 5000),
                                       (torch.bfloat16, 1, 1), (torch.float32, 300, 77)])
def test_two_captured_graphs_replayed_in_turn(dtype, N, L):
    # each graph has a workspace of its own, and replays see the inputs of the moment
    m3 = p3d()
    cases = [make(2, 4, 2, N, L, 64, dtype, "random", seed=s) for s in (31, 32)]
    graphs, outs = [], []
    for q, k, v, m, dO in cases:
        run_and_check(q, k, v, m, dO)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            f = m3.pack3d_cross_attn_fwd(q, k, v, mask=m, save_for_backward=True)
            g = m3.pack3d_cross_attn_bwd(q, k, v, f, dO, mask=m)
        graphs.append(graph)
        outs.append(dict(f, **g))
    for i in (0, 1, 0):
        graphs[i].replay()
    for i in (0, 1):
        q, k, v, m, dO = cases[i]
        q.mul_(0.5)
        graphs[i].replay()
        torch.cuda.synchronize()
        want = ob.cross(q, k, v, m, None, dO)
        for n in ("o", "lse", "dq", "dk", "dv"):
            ob.check(outs[i][n], want[n], n)


@pytest.mark.parametrize("budget", [10_000, 2_000_000, 200_000_000])
def test_a_wait_gives_up_after_its_budget(budget):
    # a barrier on which nothing arrives: the wait ends after the budget (0.1 s at most here) and at most
    # 0.2 ms later, ten times its longest nap of 20 us, at 2 GHz
    m3 = p3d()
    prev = m3.pack3d_testing_set_wait_budget(budget)
    try:
        gave_up, cycles = m3.pack3d_testing_wait()
    finally:
        m3.pack3d_testing_set_wait_budget(prev)
    assert gave_up and budget < cycles <= budget + 400_000


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("mask", ["random", "empty"])
@pytest.mark.parametrize("N,L,d", [(300, 77, 96), (130, 20, 48), (200, 128, 64), (40, 100, 128), (150, 300, 96),
                                   (2, 500, 48), (1000, 2000, 64)])
def test_rows_that_are_not_finite_keep_to_their_own_gradients(dtype, mask, N, L, d):
    # an infinity in dO and a NaN in q: gradients of states left out stay 0, as do those of rows
    # without any state, and every row and batch entry without one is as it was
    q, k, v, m, dO = make(3, 4, 2, N, L, d, dtype, mask, seed=41, garbage=True)
    if mask == "random":
        m[1] = False  # the entry in the middle has no state
    f = p3d().pack3d_cross_attn_fwd(q, k, v, mask=m, save_for_backward=True)
    g = p3d().pack3d_cross_attn_bwd(q, k, v, f, dO, mask=m)
    bad = torch.zeros(3, 4, N, dtype=torch.bool, device="cuda")  # rows touched
    bad[0, 1, N // 2] = bad[1, 2, N - 1] = bad[1, 0, 0] = True
    q2, dO2 = q.clone(), dO.clone()
    dO2[0, 1, N // 2, 5] = math.inf
    dO2[1, 2, N - 1, d - 1] = -math.inf
    q2[1, 0, 0, 3] = math.nan
    f2 = p3d().pack3d_cross_attn_fwd(q2, k, v, mask=m, save_for_backward=True)
    g2 = p3d().pack3d_cross_attn_bwd(q2, k, v, f2, dO2, mask=m)
    off = ~m[:, None, :, None].expand_as(k)
    for n in ("dk", "dv"):
        assert bool((g2[n][off] == 0).all()), n
        assert torch.equal(g2[n][2], g[n][2]), n
        assert torch.equal(g2[n][0, 1], g[n][0, 1]), n  # the other KV head of the entry
    none = (~m.any(1))[:, None, None, None].expand_as(q)
    assert bool((g2["dq"][none] == 0).all()) and bool((f2["o"][none] == 0).all())
    assert torch.equal(g2["dq"][~bad], g["dq"][~bad])


@pytest.mark.parametrize("d", [48, 64, 96, 128])
@pytest.mark.parametrize("N,L,mask", [(1000, 700, "none"), (90, 1500, "random"), (3000, 100, "pad")])
def test_results_under_other_traffic(d, N, L, mask):
    # another stream copies without a pause, so that this one's copies land late and in other orders
    m3 = p3d()
    q, k, v, m, dO = make(2, 4, 2, N, L, d, torch.bfloat16, mask, seed=51, garbage=True)
    f, g = run_and_check(q, k, v, m, dO)
    a, b = (torch.empty(1 << 28, dtype=torch.uint8, device="cuda") for _ in range(2))
    torch.cuda.synchronize()
    noise, mine = torch.cuda.Stream(), torch.cuda.Stream()
    outs = []
    for _ in range(10):
        with torch.cuda.stream(noise):
            for _ in range(2):
                b.copy_(a)
        f2 = m3.pack3d_cross_attn_fwd(q, k, v, mask=m, save_for_backward=True, stream=mine)
        g2 = m3.pack3d_cross_attn_bwd(q, k, v, f2, dO, mask=m, stream=mine)
        outs.append((f2, g2))
    torch.cuda.synchronize()
    for f2, g2 in outs:
        assert torch.equal(f["o"], f2["o"]) and torch.equal(f["lse"], f2["lse"])
        assert all(torch.equal(g[n], g2[n]) for n in ("dq", "dk", "dv"))
