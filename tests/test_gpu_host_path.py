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
