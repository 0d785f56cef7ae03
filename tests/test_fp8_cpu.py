"""Refusals of the FP8 and pooled calls: by the binding before any CUDA call, by the library before any launch
(the addresses are aligned placeholders that nothing reads)."""
import pytest
import torch

import gated_deltanet_03_b200 as g

F8, BF, F32 = torch.float8_e4m3fn, torch.bfloat16, torch.float32
A = 1 << 20
BAD, UNSUPPORTED, OK = g.GDN_ERR_INVALID_ARG, g.GDN_ERR_UNSUPPORTED, g.GDN_OK
BF16, FP32 = g.GDN_BF16, g.GDN_F32


@pytest.mark.parametrize("fn", [g.LIB.fp8_quantize_act, g.LIB.fp8_quantize_weight])
def test_quantize_refusals(fn):
    assert fn(A, 64, BF16, 4, 72, A, A, None) == BAD                # rows shorter than K
    assert fn(A, 72, BF16, 4, 72, A, A, None) == UNSUPPORTED        # K % 16
    assert fn(A, 64, 7, 4, 64, A, A, None) == BAD                   # dtype
    assert fn(A, 68, BF16, 4, 64, A, A, None) == BAD                # rows not 16-byte aligned
    assert fn(A + 8, 64, BF16, 4, 64, A, A, None) == BAD
    assert fn(A, 64, BF16, 4, 64, A + 4, A, None) == BAD
    assert fn(None, 64, BF16, 4, 64, A, A, None) == BAD
    assert fn(A, 64, BF16, -1, 64, A, A, None) == BAD
    assert fn(A, 4096, FP32, 2 ** 31 - 1, 4096, A, A, None) == UNSUPPORTED
    assert fn(None, 64, BF16, 0, 64, None, None, None) == OK


def test_tail_refusals():
    fn = g.LIB.gdn_gated_rmsnorm_silu_fp8
    assert fn(A, A, A, 1e-6, 4, 2, 96, BF16, A, A, None) == UNSUPPORTED
    assert fn(A, A, A, -1.0, 4, 2, 128, BF16, A, A, None) == BAD
    assert fn(A, A, A, float("nan"), 4, 2, 128, BF16, A, A, None) == BAD
    assert fn(A, A, A, 1e-6, 4, 2, 128, BF16, None, A, None) == BAD
    assert fn(A, A, A, 1e-6, 4, 2, 128, BF16, A + 8, A, None) == BAD
    assert fn(A, A, A, 1e-6, 2 ** 30, 32, 128, BF16, A, A, None) == UNSUPPORTED
    assert fn(None, None, None, 1e-6, 0, 2, 128, BF16, None, None, None) == OK


def test_gemm_refusals():
    fn = g.LIB.fp8_gemm
    assert fn(A, A, A, A, 4, 24, 64, BF16, A, None) == UNSUPPORTED
    assert fn(A, A, A, A, 4, 32, 72, BF16, A, None) == UNSUPPORTED
    assert fn(A, A, A, A, 4, 32, 0, BF16, A, None) == UNSUPPORTED
    assert fn(A, A, A, A, 128 * 65535 + 1, 32, 64, BF16, A, None) == UNSUPPORTED
    assert fn(A, A, A, A, 4, 32, 64, 5, A, None) == BAD
    assert fn(A + 1, A, A, A, 4, 32, 64, BF16, A, None) == BAD
    assert fn(A, A, A, A, 4, 32, 64, BF16, A + 2, None) == BAD
    assert fn(A, None, A, A, 4, 32, 64, BF16, A, None) == BAD
    assert fn(A, A, A, A, -1, 32, 64, BF16, A, None) == BAD
    assert fn(None, None, None, None, 0, 32, 64, BF16, None, None) == OK


def pooled(fn=g.LIB.gdn_decode_step_pooled, **kw):
    d = dict(q=A, k=A, v=A, a=A, b=A, ldg=4, gate=FP32, A_log=A, dt=A, B=3, Hk=2, Hv=4, Dk=128, Dv=128, scale=1.0, l2=1, io=BF16,
             pool=A, slots=5, at=A, z=A, ldz=512, w=A, eps=1e-6, xq=A, xs=A, o=A, out=BF16)
    d.update(kw)
    head = [d[n] for n in ("q", "k", "v", "a", "b", "ldg", "gate", "A_log", "dt", "B", "Hk", "Hv", "Dk", "Dv", "scale", "l2", "io", "pool",
                           "slots", "at")]
    if fn is g.LIB.gdn_decode_step_pooled:
        return fn(*head, d["o"], d["out"], None)
    return fn(*head, d["z"], d["ldz"], d["w"], d["eps"], d["xq"], d["xs"], d["o"], None)


@pytest.mark.parametrize("fn", [g.LIB.gdn_decode_step_pooled, g.LIB.gdn_decode_step_pooled_gated_fp8])
def test_pooled_decode_refusals(fn):
    for bad in (dict(Hv=3, Hk=2), dict(ldg=3), dict(gate=3), dict(io=9), dict(slots=-1), dict(B=-1), dict(q=None), dict(q=A + 8),
                dict(at=None), dict(pool=None), dict(pool=A + 4), dict(A_log=None), dict(a=None), dict(o=A + 2)):
        assert pooled(fn, **bad) == BAD, bad
    for bad in (dict(Dk=64, Dv=64, ldz=4096), dict(io=FP32), dict(B=2 ** 30), dict(B=65536)):
        assert pooled(fn, **bad) == UNSUPPORTED, bad
    assert pooled(fn, B=0, q=None, at=None) == OK


def test_pooled_tail_refusals():
    fn = g.LIB.gdn_decode_step_pooled_gated_fp8
    for bad in (dict(z=None), dict(z=A + 2), dict(ldz=511), dict(ldz=516), dict(w=None), dict(xq=None), dict(xs=None), dict(xq=A + 8),
                dict(eps=-1.0)):
        assert pooled(fn, **bad) == BAD, bad
    assert pooled(o=None) == BAD


def test_pooled_conv_refusals():
    fn = g.LIB.gdn_short_conv1d_silu_decode_pooled
    X, W, S, Y, T = 1 << 24, 1 << 20, 1 << 26, 1 << 28, 1 << 30
    assert fn(X, 256, W, 4, 256, 5, S, 9, T, Y, None, 0, None) == UNSUPPORTED
    assert fn(X, 256, W, 4, 252, 4, S, 9, T, Y, None, 0, None) == UNSUPPORTED
    assert fn(X, 256, W, 4 * 65535 + 1, 256, 4, S, 9, T, Y, None, 0, None) == UNSUPPORTED
    assert fn(X, 256, W, 4, 256, 4, S, -1, T, Y, None, 0, None) == BAD
    assert fn(X, 256, W, 4, 256, 4, S, 9, None, Y, None, 0, None) == BAD
    assert fn(X, 256, W, 4, 256, 4, None, 9, T, Y, None, 0, None) == BAD
    assert fn(X, 248, W, 4, 256, 4, S, 9, T, Y, None, 0, None) == BAD
    assert fn(X, 256, W, 4, 256, 4, Y + 512, 9, T, Y, None, 0, None) == BAD        # pool over y
    assert fn(X, 256, W, 4, 256, 4, X - 512, 9, T, Y, None, 0, None) == BAD        # pool over x
    assert fn(None, 256, None, 0, 256, 4, None, 0, None, None, None, 0, None) == OK


def binding_args(B=3, Hk=1, Hv=2):
    z = lambda *s, dtype=BF: torch.zeros(*s, dtype=dtype)  # noqa: E731
    return dict(q=z(B, Hk, 128), k=z(B, Hk, 128), v=z(B, Hv, 128), a=z(B, Hv, dtype=F32), b=z(B, Hv, dtype=F32), A_log=z(Hv, dtype=F32),
                dt_bias=z(Hv, dtype=F32), state_pool=z(4, Hv, 128, 128, dtype=F32), slots=z(B, dtype=torch.int32))


@pytest.mark.parametrize("name,value,err,msg", [
    ("slots", torch.zeros(3, dtype=torch.int64), TypeError, "slots must be torch.int32"),
    ("slots", torch.zeros(2, dtype=torch.int32), ValueError, "slots holds 2"),
    ("slots", None, ValueError, "required"),
    ("state_pool", torch.zeros(4, 2, 128, 64), ValueError, "state_pool must be"),
    ("state_pool", torch.zeros(4, 2, 128, 128, dtype=BF), TypeError, "state_pool must be torch.float32"),
    ("state_pool", torch.zeros(4, 2, 128, 256)[..., ::2], ValueError, "contiguous|CUDA"),
    ("a", torch.zeros(3, 2, dtype=BF), TypeError, "b must be torch.bfloat16"),
    ("a", torch.zeros(3, 3), ValueError, "a, b must be"),
    ("v", torch.zeros(3, 2, 64, dtype=BF), ValueError, "v"),
    ("q", torch.zeros(3, 1, 128), TypeError, "q must be torch.bfloat16"),
    ("k", torch.zeros(2, 1, 128, dtype=BF), ValueError, "k as q"),
])
def test_pooled_binding_refusals(name, value, err, msg):
    args = binding_args()
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        g.gdn_decode_step_pooled(**args)
    args[name] = value
    with pytest.raises(err, match=msg):
        g.gdn_decode_step_pooled(**args)
    with pytest.raises(err, match=msg):
        g.gdn_decode_step_pooled_gated_fp8(**args, z=torch.zeros(3, 2, 128, dtype=BF), norm_weight=torch.zeros(128))


def test_fp8_binding_refusals():
    x, q = torch.zeros(4, 64, dtype=BF), torch.zeros(4, 64, dtype=F8)
    s = torch.zeros(4, 1)
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        g.fp8_quantize_act(x)
    with pytest.raises(TypeError, match="x must be"):
        g.fp8_quantize_weight(x.half())
    with pytest.raises(ValueError, match="unit column stride"):
        g.fp8_quantize_act(x.t())
    with pytest.raises(TypeError, match="xq must be torch.float8_e4m3fn"):
        g.fp8_quantize_act(x, xq=q.view(torch.uint8))
    with pytest.raises(ValueError, match="xs holds 3"):
        g.fp8_quantize_act(x, xs=s[:3])
    with pytest.raises(TypeError, match="bq must be torch.float8_e4m3fn"):
        g.fp8_gemm(q, s, x, s)
    with pytest.raises(ValueError, match="as_ holds 3"):
        g.fp8_gemm(q, s[:3], q, s)
    with pytest.raises(ValueError, match="bs holds 0"):
        g.fp8_gemm(q, s, q, s[:0])
    with pytest.raises(ValueError, match="y holds"):
        g.fp8_gemm(q, s, q, s, y=torch.zeros(3, 4))
    o = torch.zeros(4, 2, 128, dtype=BF)
    with pytest.raises(TypeError, match="z must be"):
        g.gdn_gated_rmsnorm_silu_fp8(o, o.float(), torch.zeros(128))
    with pytest.raises(ValueError, match="conv_pool must be"):
        g.gdn_short_conv1d_silu_decode_pooled(x, torch.zeros(64, 4), torch.zeros(5, 4, 64, dtype=BF), torch.zeros(4, dtype=torch.int32))
    with pytest.raises(ValueError, match="required"):
        g.gdn_short_conv1d_silu_decode_pooled(x, torch.zeros(64, 4), None, torch.zeros(4, dtype=torch.int32))


def test_host_path_is_built_and_declines_quietly():
    """The compiled host path is there; what it does not take it answers with None, whatever it is given."""
    assert g._host is not None
    x = torch.zeros(4, 64, dtype=BF)
    odd = [(), (1,), (None,) * 6, (x,) * 4, (x, None, None, False), ("a", 2.0, None, x, x, 1), (x,) * 6, (x,) * 13, (x,) * 17,
           (x, x, x, x, (64, "b"), None), (None,) * 17]
    for f in (g._host.fp8_gemm, g._host.fp8_quantize, g._host.tail, g._host.decode, g._host.conv):
        for args in odd:
            assert f(*args) is None
    with pytest.raises(TypeError):
        g._host.bind(1, 2)
