"""The two ways of a call from Python to the library, the compiled host path and ctypes: a call that fails has changed
nothing, whichever way it went."""
import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(params=["host", "ctypes"])
def g(request, monkeypatch):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gated_deltanet_03_b200 as lib
    if request.param == "ctypes":
        monkeypatch.setattr(lib, "_host", None)
    elif lib._host is None:
        pytest.skip("the compiled host path is not built")
    return lib


class NoViews(TorchDispatchMode):
    """Refuses to make views, as a tracer or an allocation that fails would."""

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        if func.overloadpacket in (torch.ops.aten.view, torch.ops.aten.slice, torch.ops.aten.narrow, torch.ops.aten.reshape):
            raise RuntimeError("no views here")
        return func(*args, **(kwargs or {}))


@pytest.mark.parametrize("parts", [(64, 128, 64), None])
def test_a_call_that_fails_has_not_advanced_the_pool(g, parts):
    B, C = 3, 256
    x, w = torch.randn(B, C, device="cuda").to(BF), torch.randn(C, 4, device="cuda")
    pool, at = torch.randn(5, 3, C, device="cuda").to(BF), torch.tensor([4, 0, 2], dtype=torch.int32, device="cuda")
    before, y = pool.clone(), torch.zeros(B * C, dtype=BF, device="cuda")
    with pytest.raises(RuntimeError, match="no views here"), NoViews():
        g.gdn_short_conv1d_silu_decode_pooled(x, w, pool, at, parts=parts, y=y)
    assert torch.equal(pool, before) and (y == 0).all()
    out = g.gdn_short_conv1d_silu_decode_pooled(x, w, pool, at, parts=parts, y=y)
    once, y2 = before.clone(), torch.empty_like(y)
    g.gdn_short_conv1d_silu_decode_pooled(x, w, once, at, parts=parts, y=y2)
    assert torch.equal(pool, once) and torch.equal(y, y2) and torch.equal(pool[4, 2], x[0])
    assert (out.data_ptr() if parts is None else out[0].data_ptr()) == y.data_ptr()


@pytest.mark.parametrize("parts", [(64, 128, 72), (64, 128), (264, -8), (64,) * 5, (64, 64, 32, 32, 64)])
def test_widths_that_do_not_fit_are_refused(g, parts):
    x, w = torch.randn(3, 256, device="cuda").to(BF), torch.randn(256, 4, device="cuda")
    pool, at = torch.randn(5, 3, 256, device="cuda").to(BF), torch.tensor([4, 0, 2], dtype=torch.int32, device="cuda")
    before = pool.clone()
    with pytest.raises(g.GdnError):
        g.gdn_short_conv1d_silu_decode_pooled(x, w, pool, at, parts=parts)
    assert torch.equal(pool, before)


def calls():
    """Well-formed calls of every host function, in each of its forms: (function, arguments)."""
    import gated_deltanet_03_b200 as lib
    gen = torch.Generator("cuda").manual_seed(0)
    r = lambda *s, dt=BF: torch.randn(*s, device="cuda", generator=gen).to(dt)  # noqa: E731
    f32, f8 = torch.float32, torch.float8_e4m3fn
    B, Hk, Hv, D, C = 5, 2, 4, 128, 1024
    new = lambda *s, dt: torch.empty(*s, dtype=dt, device="cuda")  # noqa: E731
    x, w, big = r(B, 272), r(144, 272, dt=f32), r(B, 800)
    aq, as_ = lib._fp8_quantize(lib.LIB.fp8_quantize_act, x, None, None, True, None)
    bq, bs = lib._fp8_quantize(lib.LIB.fp8_quantize_weight, w, None, None, False, None)
    o, z, nw = r(B, Hv, D), r(B, Hv, D), r(D, dt=f32)
    at = torch.tensor([3, -1, 0, 6, 2], dtype=torch.int32, device="cuda")
    step = lambda gates: (r(B, Hk, D), r(B, Hk, D), r(B, Hv, D), r(B, Hv, dt=gates), r(B, Hv, dt=gates), r(Hv, dt=f32), r(Hv, dt=f32),  # noqa: E731
                          r(7, Hv, D, D, dt=f32), at)
    cw, pool = r(C, 4, dt=f32), r(7, 3, C)
    rows = r(B, C + 64)
    h = lib._host
    return [
        (h.fp8_gemm, (aq, as_, bq, bs, None, False)), (h.fp8_gemm, (aq, as_, bq, bs, None, True)),
        (h.fp8_gemm, (aq, as_, bq, bs, new(B, 144, dt=f32), False)), (h.fp8_gemm, (aq[:1], as_[:1], bq, bs, new(144, dt=BF), False)),
        (h.fp8_quantize, (x, None, None, False)), (h.fp8_quantize, (w, new(144, 272, dt=f8), new(6, dt=f32), True)),
        (h.fp8_quantize, (big[:, 16:288], None, None, False)), (h.fp8_quantize, (big[:1, 16:288], None, None, True)),
        (h.tail, (o, z, nw, 1e-6, None, None)), (h.tail, (o.float(), z.float(), nw, 0, new(B, 512, dt=f8), new(B, 4, dt=f32))),
        (h.decode, (*step(f32), 1.0, True, None, False)), (h.decode, (*step(BF), 0.5, False, None, True)),
        (h.decode, (*step(BF), 1, 1, new(B, Hv, D, dt=f32), False)),
        (h.decode, (*step(f32), 1.0, True, None, z, nw, 1e-6, None, None)),
        (h.decode, (*step(BF), 1.0, True, new(B, Hv, D, dt=BF), r(B, 600)[:, 8:520].unflatten(1, (Hv, D)), nw, 1e-6,
                    new(B, 512, dt=f8), new(B, Hv, dt=f32))),
        (h.conv, (rows[:, :C], cw, pool, at, None, None)), (h.conv, (rows[:, 64:], cw, pool, at, (256, 256, 512), None)),
        (h.conv, (rows[:, 64:], cw, pool, at, [1024], new(B * C, dt=BF))), (h.conv, (rows[:, 64:], cw, pool, at, None, new(B * C, dt=BF))),
        (h.conv, (rows[:1, 64:], cw, pool, at[:1], None, None)),
    ]


def test_the_host_path_takes_the_plain_calls():
    """The binding hides a host function that declines: its call goes through ctypes. So each is asked directly."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gated_deltanet_03_b200 as lib
    if lib._host is None:
        pytest.skip("the compiled host path is not built")
    for f, args in calls():
        assert f(*args) is not None, (f.__name__, [getattr(a, "shape", a) for a in args])
    # a call that is not one it takes
    x = torch.zeros(4, 64, device="cuda", dtype=BF)
    assert lib._host.fp8_quantize(x.half(), None, None, False) is None
    assert lib._host.fp8_quantize(x.t(), None, None, False) is None
    assert lib._host.fp8_quantize(x[:, :8], None, None, False) is None
    assert lib.gdn_get_device_status() == 0


def test_both_ways_give_the_same(monkeypatch):
    """A whole chain, by the host path where it is built and by ctypes: the same bytes."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gated_deltanet_03_b200 as lib

    def chain():
        gen = torch.Generator("cuda").manual_seed(1)
        r = lambda *s, dt=BF: torch.randn(*s, device="cuda", generator=gen).to(dt)  # noqa: E731
        f32 = torch.float32
        at = torch.tensor([3, -1, 0], dtype=torch.int32, device="cuda")
        win, hidden = lib.fp8_quantize_weight(r(1024 + 512 + 16, 384, dt=f32)), r(3, 384)
        p = lib.fp8_gemm(*lib.fp8_quantize_act(hidden), *win)
        conv_pool, pool = r(4, 3, 1024), r(4, 4, 128, 128, dt=f32)
        q, k, v = lib.gdn_short_conv1d_silu_decode_pooled(p[:, :1024], r(1024, 4, dt=f32), conv_pool, at, parts=(256, 256, 512))
        step = (q.view(3, 2, 128), k.view(3, 2, 128), v.view(3, 4, 128), p[:, 1536:1540], p[:, 1544:1548], r(4, dt=f32), r(4, dt=f32))
        nw, z = r(128, dt=f32), p[:, 1024:1536].unflatten(1, (4, 128))
        o = lib.gdn_decode_step_pooled(*step, pool.clone(), at, out_dtype=f32)
        xq, xs, _ = lib.gdn_decode_step_pooled_gated_fp8(*step, pool, at, z, nw)
        tq, ts = lib.gdn_gated_rmsnorm_silu_fp8(o, z.contiguous().float(), nw)
        return [t.contiguous().view(torch.uint8) for t in (p, q, k, v, o, xq, xs, tq, ts, conv_pool, pool)]

    first = chain()
    monkeypatch.setattr(lib, "_host", None)
    assert all(torch.equal(a, b) for a, b in zip(first, chain()))
    assert lib.gdn_get_device_status() == 0
