"""Cross attention, layer norm and gradient clipping: what their calls refuse, checked on the host
before any launch (no GPU), and the float64 references of the GPU tests against autograd."""
import ctypes
import math

import pytest
import torch

from geometry_aware_local_pack3d_b200 import binding as b

from . import ops_bounds as ob

FAKE, ODD = 0x100000, 0x100004


def cross_fwd(**kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, mask=None, dtype=1, batch=1, heads=2, kv_heads=2, n=20, l=200, d=96,
             scale=0.1, o=FAKE, lse=None, ws=None, bytes=0, status=None)
    a.update(kw)
    return b.lib().pack3d_cross_attn_fwd(a["q"], a["k"], a["v"], a["mask"], a["dtype"], a["batch"],
                                         a["heads"], a["kv_heads"], a["n"], a["l"], a["d"], a["scale"],
                                         a["o"], a["lse"], a["ws"], a["bytes"], a["status"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=2), 1), (dict(batch=0), 1), (dict(heads=0), 1), (dict(n=-1), 1), (dict(l=-1), 1),
    (dict(heads=6, kv_heads=4), 1), (dict(kv_heads=-1), 1), (dict(heads=2, kv_heads=4), 1),
    (dict(batch=40000), 2), (dict(d=32), 2), (dict(d=50), 2), (dict(l=(1 << 30) + 1), 2),
    (dict(n=1 << 30, heads=4, kv_heads=2), 2), (dict(scale=0.0), 1), (dict(scale=-1.0), 1),
    (dict(scale=math.nan), 1), (dict(scale=math.inf), 1), (dict(q=None), 1), (dict(k=None), 1),
    (dict(v=None), 1), (dict(o=None), 1), (dict(q=ODD), 5), (dict(k=ODD), 5), (dict(v=ODD), 5),
    (dict(o=ODD), 5), (dict(mask=FAKE), 1), (dict(mask=FAKE, ws=FAKE, bytes=8), 8),
    (dict(mask=FAKE, ws=FAKE + 16, bytes=1 << 20), 5)])
def test_cross_forward_refusals(kw, status):
    assert cross_fwd(**kw) == status
    assert b.lib().pack3d_last_launch_count() == 0


def cross_bwd(**kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, mask=None, o=FAKE, lse=FAKE, dO=FAKE, n=10, l=10, scale=0.1, dq=FAKE,
             dk=FAKE, dv=FAKE, ws=FAKE, bytes=1 << 30)
    a.update(kw)
    return b.lib().pack3d_cross_attn_bwd(a["q"], a["k"], a["v"], a["mask"], a["o"], a["lse"], a["dO"], 1, 1,
                                         2, 2, a["n"], a["l"], 96, a["scale"], a["dq"], a["dk"], a["dv"],
                                         a["ws"], a["bytes"], None, None)


@pytest.mark.parametrize("kw,status", [
    (dict(lse=None), 1), (dict(dO=None), 1), (dict(o=None), 1), (dict(dq=None), 1), (dict(dk=None), 1),
    (dict(dv=None), 1), (dict(dO=ODD), 5), (dict(dk=ODD), 5), (dict(ws=None), 1), (dict(bytes=16), 8),
    (dict(ws=FAKE + 128), 5), (dict(scale=0.0), 1), (dict(n=0, dk=None), 1), (dict(l=0, dq=None), 1)])
def test_cross_backward_refusals(kw, status):
    assert cross_bwd(**kw) == status
    assert b.lib().pack3d_last_launch_count() == 0


def test_the_wait_hook_refuses_a_null_pointer():
    assert b.lib().pack3d_testing_wait(None, None) == 1
    assert b.lib().pack3d_last_launch_count() == 0


def test_cross_workspace_sizes():
    f = b.pack3d_cross_attn_workspace_bytes
    assert f(1, 1, 2, 2, 10, 10, 50) == 0 and f(1, 1, 3, 2, 10, 10, 96) == 0
    assert f(1, 1, 2, 2, 0, 10, 96, True, True) == 0 and f(1, 1, 2, 2, 10, 0, 96, True, True) == 0
    assert f(1, 1, 2, 2, 300, 77, 96) == 0 and f(1, 1, 2, 2, 300, 77, 96, True) == 0  # short contexts
    assert f(1, 200, 2, 2, 300, 300, 96) == 0 and f(1, 200, 2, 2, 300, 300, 96, True) > 0
    assert f(1, 1, 2, 2, 1, 8192, 96) > 0                       # the states are split
    assert f(1, 1, 2, 2, 300, 300, 96, False, True) >= 2 * 384 * 8
    assert f(1, 1, 2, 2, 300, 77, 96, False, True) > 0
    # the sizes do not wrap: a long context's partial sums
    assert f(0, 1, 8, 8, 1 << 20, 1 << 20, 128, False, True) >= 8 * (1 << 20) * 4


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=3), 1), (dict(wdtype=-1), 1), (dict(rows=-1), 1), (dict(cols=0), 1), (dict(cols=-5), 1),
    (dict(rows=1 << 60, cols=1 << 20), 2), (dict(eps=-1.0), 1), (dict(eps=math.nan), 1),
    (dict(eps=math.inf), 1), (dict(x=None), 1), (dict(y=None), 1), (dict(x=ODD), 5), (dict(y=ODD), 5),
    (dict(y=FAKE), 1)])
def test_layer_norm_forward_refusals(kw, status):
    a = dict(x=FAKE, w=None, b=None, dtype=1, wdtype=0, rows=4, cols=8, eps=1e-5, y=2 * FAKE)
    a.update(kw)
    assert b.lib().pack3d_layer_norm_fwd(a["x"], a["w"], a["b"], a["dtype"], a["wdtype"], a["rows"],
                                         a["cols"], a["eps"], a["y"], None, None, None) == status
    assert b.lib().pack3d_last_launch_count() == 0


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=3), 1), (dict(dy=None), 1), (dict(mean=None), 1), (dict(rstd=None), 1), (dict(dx=None), 1),
    (dict(dx=ODD), 5), (dict(dx=FAKE), 1), (dict(ws=None), 1), (dict(bytes=16), 8), (dict(ws=ODD), 5)])
def test_layer_norm_backward_refusals(kw, status):
    a = dict(dy=FAKE, x=FAKE, mean=FAKE, rstd=FAKE, dtype=1, wdtype=0, rows=4, cols=8, dx=2 * FAKE, dw=FAKE,
             db=FAKE, ws=FAKE, bytes=1 << 20)
    a.update(kw)
    assert b.lib().pack3d_layer_norm_bwd(a["dy"], a["x"], None, a["mean"], a["rstd"], a["dtype"],
                                         a["wdtype"], a["rows"], a["cols"], a["dx"], a["dw"], a["db"],
                                         a["ws"], a["bytes"], None) == status
    assert b.lib().pack3d_last_launch_count() == 0


def clip(ptrs, counts, codes, outs=None, max_norm=1.0, norm=FAKE, ws=FAKE, size=1 << 20):
    n = len(ptrs)
    arr = lambda t, v: (t * max(n, 1))(*v)  # noqa: E731
    return b.lib().pack3d_clip_grad_norm(arr(ctypes.c_void_p, ptrs),
                                         arr(ctypes.c_void_p, ptrs if outs is None else outs),
                                         arr(ctypes.c_int64, counts), arr(ctypes.c_int, codes), n, max_norm,
                                         norm, ws, size, None)


@pytest.mark.parametrize("args,kw,status", [
    (([FAKE], [10], [2]), {}, 1), (([FAKE], [-1], [0]), {}, 1), (([None], [10], [0]), {}, 1),
    (([FAKE + 2], [10], [0]), {}, 5), (([FAKE + 1], [10], [1]), {}, 5),
    (([FAKE], [10], [0]), dict(outs=[FAKE + 2]), 5), (([FAKE], [10], [0]), dict(outs=[None]), 1),
    (([FAKE], [10], [0]), dict(max_norm=-1.0), 1), (([FAKE], [10], [0]), dict(max_norm=math.nan), 1),
    (([FAKE], [10], [0]), dict(norm=None), 1), (([FAKE], [10], [0]), dict(ws=None), 1),
    (([FAKE], [10], [0]), dict(size=64), 8), (([FAKE], [10], [0]), dict(ws=ODD), 5),
    (([FAKE, FAKE], [10, 10], [0, 0]), {}, 1), (([FAKE, FAKE + 36], [10, 10], [0, 0]), {}, 1),
    (([FAKE], [10], [0]), dict(outs=[FAKE + 4]), 1),
    (([FAKE, FAKE + 400], [10, 10], [0, 0]), dict(outs=[FAKE + 800, FAKE + 4]), 1)])
def test_clip_refusals(args, kw, status):
    assert clip(*args, **kw) == status
    assert b.lib().pack3d_last_launch_count() == 0


def test_binding_refuses_tensors_it_cannot_use():
    t = torch.zeros(1, 2, 4, 96)
    for call in (lambda: b.pack3d_cross_attn_fwd(t, t, t), lambda: b.pack3d_layer_norm_fwd(t),
                 lambda: b.pack3d_grad_norm([t])):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        b.pack3d_layer_norm_fwd(t.half())


# ------------------------------------------------- the references of the GPU tests, on the CPU
def test_cross_reference_matches_autograd():
    g = torch.Generator().manual_seed(0)
    B, H, HK, N, L, d = 2, 4, 2, 5, 9, 48
    q, dO = (torch.randn(B, H, N, d, generator=g, dtype=torch.float64) for _ in range(2))
    k, v = (torch.randn(B, HK, L, d, generator=g, dtype=torch.float64) for _ in range(2))
    mask = torch.rand(B, L, generator=g) < 0.6
    mask[0, 0] = mask[1, 1] = True
    qq, kk, vv = (x.clone().requires_grad_() for x in (q, k, v))
    o = torch.nn.functional.scaled_dot_product_attention(
        qq, kk.repeat_interleave(2, 1), vv.repeat_interleave(2, 1), attn_mask=mask[:, None, None, :])
    (o * dO).sum().backward()
    f32 = [x.to(torch.float64) for x in (q, k, v)]
    ob_half = ob.half_step
    try:
        ob.half_step = lambda dt: 0.0
        want = ob.cross(*f32, mask, None, dO)
    finally:
        ob.half_step = ob_half
    for n, x in (("o", o), ("dq", qq.grad), ("dk", kk.grad), ("dv", vv.grad)):
        assert torch.allclose(want[n][0], x, atol=1e-12), n


def test_layer_norm_reference_matches_autograd():
    g = torch.Generator().manual_seed(0)
    x, dy = (torch.randn(7, 20, generator=g, dtype=torch.float64) for _ in range(2))
    w, bb = (torch.randn(20, generator=g, dtype=torch.float64) for _ in range(2))
    xx, ww, b2 = (t.clone().requires_grad_() for t in (x, w, bb))
    y = torch.nn.functional.layer_norm(xx, (20,), ww, b2, 1e-5)
    (y * dy).sum().backward()
    want = ob.layer_norm(x, w, bb, 1e-5, dy)
    for n, t in (("y", y), ("dx", xx.grad), ("dweight", ww.grad), ("dbias", b2.grad)):
        assert torch.allclose(want[n][0], t, atol=1e-12), n


def test_an_oracle_with_a_mistake_is_noticed():
    # a mistake planted in the reference (a forgotten mask entry) lies far outside the bounds
    g = torch.Generator().manual_seed(1)
    q, k, v = (torch.randn(1, 1, 4, 48, generator=g).to(torch.bfloat16) for _ in range(3))
    mask = torch.tensor([[True, True, False, True]])
    good = ob.cross(q, k, v, mask)["o"]
    bad = ob.cross(q, k, v, torch.ones_like(mask))["o"][0]
    with pytest.raises(AssertionError):
        ob.check(bad, good, "o")


def test_f32_cross_workspace_of_split_states_and_rows():
    f = b.pack3d_cross_attn_workspace_bytes
    # few rows over a long context: partial o and lse, partial dq, in 32 bits
    assert f(0, 1, 2, 2, 1, 8192, 96) >= 2 * 2 * (96 + 1) * 4
    assert f(0, 1, 2, 2, 1, 8192, 96, False, True) >= 2 * 4 + 2 * 2 * 96 * 4
    # rows enough for every SM: none
    assert f(0, 8, 8, 8, 65536, 300, 96) == 0


def test_binding_refuses_a_stream_of_another_device():
    class Stream:
        device, cuda_stream = torch.device("cuda", 1), 7
    assert b._stream_of(1, Stream) == 7
    with pytest.raises(ValueError):
        b._stream_of(0, Stream)


def test_list_helper_refuses_what_is_no_dense_tensor_of_the_device():
    t = torch.zeros(4)
    for bad in ([t], [t.to_sparse()], [torch.zeros(4, device="meta")], [torch.zeros(4, 4).t()]):
        with pytest.raises(ValueError):
            b._tensor_list(bad, "grads", 0)
    with pytest.raises(TypeError):
        b._tensor_list([t, None][1:], "grads", 0)
    assert b._tensor_list([], "grads", 0) == (b"", b"", b"")


class Shaped:
    """A CUDA tensor of a shape, as far as the binding's checks look."""

    is_cuda, dtype = True, torch.bfloat16

    def __init__(self, *shape):
        self.shape = torch.Size(shape)

    def dim(self):
        return len(self.shape)

    def is_contiguous(self):
        return True

    def get_device(self):
        return 0


def test_binding_refuses_sizes_that_the_abi_would_wrap():
    # 2^32 + 96 would reach the library as 96
    big = (1 << 32) + 96
    x = Shaped(1, 2, 3, big)
    for call in (lambda: b.pack3d_cross_attn_fwd(x, x, x), lambda: b.pack3d_layer_norm_fwd(x),
                 lambda: b.pack3d_layer_norm_bwd(x, x, None, {}),
                 lambda: b._cross_shapes(Shaped(1, big, 0, 96), *[Shaped(1, 2, 3, 96)] * 2, None)):
        with pytest.raises(ValueError, match="less than 2\\^31"):
            call()
    assert b._cross_shapes(*[Shaped(1, 2, 3, 96)] * 3, None)[:6] == (1, 2, 2, 3, 3, 96)


@pytest.mark.parametrize("dtype,cols,at,status", [
    (1, 8, 2, 5), (1, 16384, 2, 5), (0, 4, 4, 5), (0, 8192, 4, 5),  # whole pieces: 16 bytes
    (1, 333, 1, 5), (1, 16392, 1, 5), (0, 333, 2, 5), (0, 8196, 2, 5)])  # otherwise: an element
def test_layer_norm_alignment_by_the_rows_length(dtype, cols, at, status):
    for off in ((at, 0, 0), (0, at, 0), (0, 0, at)):
        x, dy, y = FAKE + off[0], 2 * FAKE + off[1], 3 * FAKE + off[2]
        if off[1] == 0:
            assert b.lib().pack3d_layer_norm_fwd(x, None, None, dtype, 0, 1, cols, 1e-5, y, None, None,
                                                 None) == status
        assert b.lib().pack3d_layer_norm_bwd(dy, x, None, FAKE, FAKE, dtype, 0, 1, cols, y, None, None, None, 0,
                                             None) == status
        assert b.lib().pack3d_last_launch_count() == 0


def test_the_library_is_built_without_the_list_helper(monkeypatch, tmp_path):
    from geometry_aware_local_pack3d_b200 import build as bd
    steps = []

    def no_compiler(*a, **k):
        steps.append("helper")
        raise FileNotFoundError("g++")

    monkeypatch.setattr(bd, "build_library", lambda *a: steps.append("library") or bd.LIB)
    monkeypatch.setattr(bd, "tensor_list_path", lambda: str(tmp_path / "none.so"))
    monkeypatch.setattr(bd.subprocess, "run", no_compiler)
    with pytest.warns(UserWarning, match="lists of tensors"):
        assert bd.build() == bd.LIB
    assert steps == ["library", "helper"]
    # the calls over lists of tensors then say what is missing
    monkeypatch.setattr(b, "_list_module", None)
    with pytest.raises(RuntimeError, match="none.so not found"):
        b._tensor_list([], "grads", 0)


def test_the_list_helper_of_another_torch_or_python_is_not_taken(monkeypatch):
    from geometry_aware_local_pack3d_b200 import build as bd
    here = bd.tensor_list_path()
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    other_torch = bd.tensor_list_path()
    monkeypatch.setattr(bd.sysconfig, "get_config_var", lambda n: "cpython-1")
    assert len({here, other_torch, bd.tensor_list_path()}) == 3


FAKE_RUNTIME = """
#include "launch.h"
static int device = 0, looks = 0;
thread_local int p3d::g_launches = 0;
extern "C" {
cudaError_t cudaGetDevice(int* d) { *d = device; return cudaSuccess; }
cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr, int) { *v = 148; return cudaSuccess; }
cudaError_t cudaFuncSetAttribute(const void*, cudaFuncAttribute, int) { return cudaSuccess; }
int look_on(int d, int answer) {
  static p3d::PerDevice cache;
  device = d;
  return cache.get([&] { ++looks; return answer; });
}
int looks_so_far(void) { return looks; }
}
"""


def test_what_a_launch_keeps_is_kept_per_device(tmp_path):
    import shutil
    import subprocess

    from geometry_aware_local_pack3d_b200 import build as bd
    (tmp_path / "fake.cpp").write_text(FAKE_RUNTIME)
    cuda = bd.os.path.join(bd.os.path.dirname(bd.os.path.dirname(bd.os.path.realpath(bd.nvcc()))), "include")
    out = str(tmp_path / "fake.so")
    subprocess.run([shutil.which("g++") or "g++", "-std=c++17", "-shared", "-fPIC", "-Wl,-Bsymbolic", "-I", cuda,
                    "-I", bd.CSRC, str(tmp_path / "fake.cpp"), "-o", out], check=True)
    fake = ctypes.CDLL(out)
    assert [fake.look_on(0, 296), fake.look_on(1, 264), fake.look_on(0, 7), fake.look_on(1, 7)] == \
        [296, 264, 296, 264] and fake.looks_so_far() == 2
    # a failed look is asked again, and so is a device beyond the cache
    assert [fake.look_on(2, 0), fake.look_on(2, 5), fake.look_on(2, 6)] == [0, 5, 5]
    assert [fake.look_on(64, 8), fake.look_on(64, 9)] == [8, 9]


def test_no_launch_keeps_a_device_number_per_process():
    import re

    from geometry_aware_local_pack3d_b200 import build as bd
    for path in bd.sources():
        text = open(path).read()
        assert not re.search(r"static const (int|bool) \w+ = (grid_for|\[\])", text), path


def test_a_context_of_one_tile_is_never_the_general_forwards():
    # k_cross_fwd walks two state tiles or more: up to 64 states every head_dim has the kernel for short
    # contexts, which needs no workspace, where the general one builds tables of the mask
    for d in (48, 64, 96, 128):
        for l in (1, 33, 64):
            assert b.pack3d_cross_attn_workspace_bytes(1, 1, 2, 2, 300, l, d, True) == 0
        assert b.pack3d_cross_attn_workspace_bytes(1, 1, 2, 2, 300, 129, d, True) > 0
