"""Decode on pools of states: the delta rule (plain and with the FP8 tail) and the convolution against the
calls on contiguous states bit for bit and against the oracle, rows without a slot left as they are, bad and
repeated slots reported and passed over, and a whole FP8 layer over several steps."""
import numpy as np
import pytest
import torch

import oracle
import workloads
from helpers import TOL_CONV_ATOL, TOL_CONV_RTOL, dev, to_np

pytestmark = pytest.mark.gpu
F8, BF, F32 = torch.float8_e4m3fn, torch.bfloat16, torch.float32


@pytest.fixture(scope="module", params=["host", "ctypes"])
def g(request):
    """The library with its calls made by the compiled host path, and through ctypes alone."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gated_deltanet_03_b200 as lib
    lib.gdn_get_device_status()
    host = lib._host
    assert host is not None
    lib._host = host if request.param == "host" else None
    yield lib
    lib._host = host
    assert lib.gdn_get_device_status() == 0


def batch(B, Hk, Hv, slots, dead=(), seed=0, gates=F32):
    gen = torch.Generator("cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, device="cuda", generator=gen)  # noqa: E731
    at = torch.randperm(slots, device="cuda", generator=gen)[:B].to(torch.int32)
    for i in dead:
        at[i] = -1 - i
    return dict(q=r(B, Hk, 128).to(BF), k=r(B, Hk, 128).to(BF), v=r(B, Hv, 128).to(BF), a=r(B, Hv).to(gates), b=r(B, Hv).to(gates),
                A_log=torch.rand(Hv, device="cuda", generator=gen) * 2.7, dt_bias=r(Hv) * 0.1, state_pool=r(slots, Hv, 128, 128) * 0.1,
                slots=at), dict(z=r(B, Hv, 128).to(BF), norm_weight=torch.rand(128, device="cuda", generator=gen) + 0.5)


def contiguous_step(g, x, **kw):
    """(live rows, o fp32, new states) by gdn_decode_step on the gathered states."""
    live = (x["slots"] >= 0).nonzero().squeeze(1)
    S = x["state_pool"][x["slots"][live].long()].clone()
    row = {n: x[n][live].contiguous() for n in ("q", "k", "v")}
    o = g.gdn_decode_step(**row, a=x["a"][live].float(), b=x["b"][live].float(), A_log=x["A_log"], dt_bias=x["dt_bias"], state=S,
                          out_dtype=F32, **kw)
    return live, o, S


CASES = [(1, 1, 1, 1, ()), (1, 16, 32, 3, ()), (4, 2, 4, 9, (1,)), (5, 1, 3, 5, (0, 4)), (7, 4, 4, 40, (0, 1, 2, 3, 4, 5, 6)),
         (40, 16, 16, 50, (3, 39)), (129, 2, 2, 129, ())]


@pytest.mark.parametrize("B,Hk,Hv,slots,dead", CASES)
@pytest.mark.parametrize("gates", [F32, BF])
def test_decode_equals_contiguous(g, B, Hk, Hv, slots, dead, gates):
    x, tail = batch(B, Hk, Hv, slots, dead, seed=B * 7 + Hv, gates=gates)
    live, o_ref, S_ref = contiguous_step(g, x, scale=0.25)
    want = x["state_pool"].clone()
    want[x["slots"][live].long()] = S_ref
    before = x["state_pool"].clone()
    for out in (F32, BF):
        x["state_pool"].copy_(before)
        o = torch.full((B, Hv, 128), 5.0, dtype=out, device="cuda")
        g.gdn_decode_step_pooled(**x, scale=0.25, o=o)
        assert torch.equal(x["state_pool"], want)
        expect = torch.full_like(o, 5.0)
        expect[live] = o_ref.to(out)
        assert torch.equal(o, expect)
    # the fused form: o's bytes, the same states, padded rows of every output left alone
    x["state_pool"].copy_(before)
    xq = torch.full((B, Hv * 128), 3.0, device="cuda").to(F8)
    xs = torch.full((B, Hv), 9.0, device="cuda")
    o = torch.full((B, Hv, 128), 5.0, dtype=BF, device="cuda")
    g.gdn_decode_step_pooled_gated_fp8(**x, **tail, scale=0.25, xq=xq, xs=xs, o=o)
    assert torch.equal(x["state_pool"], want)
    q2, s2 = torch.full_like(xq, 3.0), torch.full_like(xs, 9.0)
    if len(live):
        a, b = g.gdn_gated_rmsnorm_silu_fp8(o_ref, tail["z"][live].float(), tail["norm_weight"])
        q2.view(torch.uint8)[live], s2[live] = a.view(torch.uint8), b
    assert torch.equal(xs, s2) and torch.equal(xq.view(torch.uint8), q2.view(torch.uint8))
    expect = torch.full_like(o, 5.0)
    expect[live] = o_ref.to(BF)
    assert torch.equal(o, expect)


@pytest.mark.parametrize("l2norm", [True, False])
def test_decode_against_oracle(g, l2norm):
    B, Hk, Hv, slots = 6, 2, 4, 11
    x, _ = batch(B, Hk, Hv, slots, seed=3)
    if not l2norm:
        x["q"], x["k"] = x["q"] * 0.1, x["k"] * 0.1
    n = {k: to_np(v) for k, v in x.items()}
    at = n["slots"].astype(int)
    o_ref, S_ref = oracle.gdn_scan(n["q"], n["k"], n["v"], n["a"], n["b"], n["A_log"], n["dt_bias"],
                                   cu_seqlens=np.arange(B + 1, dtype=np.int32), initial_state=n["state_pool"][at], qk_l2norm=l2norm)
    o = g.gdn_decode_step_pooled(**x, qk_l2norm=l2norm, out_dtype=F32)
    # a dot of 128 terms is at most 128 roundings of 2^-24 (lanes and shuffles make it 12); two of them, the
    # norms and the gates (a decay's error is |g| alpha times its steps', and |g| alpha <= 1/e) are on the
    # way to o, on terms whose sizes the state's rows and the values bound
    head = np.repeat(np.arange(Hk), Hv // Hk)
    unit = lambda t: t / np.sqrt((t.astype(np.float64) ** 2).sum(-1, keepdims=True) + 1e-6) if l2norm else t  # noqa: E731
    q, k = (np.abs(unit(n[m]))[:, head] for m in ("q", "k"))
    S0 = np.abs(n["state_pool"][at]).astype(np.float64)
    u = np.abs(n["v"]) + np.einsum("bhij,bhj->bhi", S0, k)
    S_size = S0 + u[..., None] * k[:, :, None, :]
    o_size = np.einsum("bhij,bhj->bhi", S_size, q)
    c = (2 * 128 + 40) * 2.0 ** -24
    assert (np.abs(to_np(o) - o_ref) <= c * o_size).all()
    assert (np.abs(to_np(x["state_pool"])[at] - S_ref) <= c * S_size).all()


def test_decode_strided_projection_rows(g):
    """z, a and b as column slices of one projection output."""
    B, Hk, Hv = 9, 2, 4
    x, tail = batch(B, Hk, Hv, 12, (2,), seed=8, gates=BF)
    proj = torch.randn(B, 64 + Hv * 128 + 24, device="cuda").to(BF)
    z, a, b = proj[:, 64:64 + Hv * 128].unflatten(1, (Hv, 128)), proj[:, 64 + Hv * 128:][:, 1:1 + Hv], proj[:, -Hv:]
    pool = x["state_pool"].clone()
    got = g.gdn_decode_step_pooled_gated_fp8(**{**x, "a": a, "b": b, "state_pool": pool}, z=z, norm_weight=tail["norm_weight"])
    pool2 = x["state_pool"].clone()
    want = g.gdn_decode_step_pooled_gated_fp8(**{**x, "a": a.contiguous(), "b": b.contiguous(), "state_pool": pool2}, z=z.contiguous(),
                                              norm_weight=tail["norm_weight"])
    assert torch.equal(pool, pool2) and torch.equal(got[1], want[1])
    assert torch.equal(got[0].view(torch.uint8), want[0].view(torch.uint8))


@pytest.mark.parametrize("B", [3, 70])
def test_bad_slots_are_reported_and_passed_over(g, B):
    """A repeated slot goes to its first row; a slot past the pool goes to nobody."""
    import gated_deltanet_03_b200 as lib
    x, tail = batch(B, 2, 2, 80, seed=4)
    good = x["slots"].clone()
    x["slots"][B - 1] = x["slots"][0]
    x["slots"][1] = 80 if B == 3 else 2 ** 31 - 1
    before = x["state_pool"].clone()
    xq, xs, _ = g.gdn_decode_step_pooled_gated_fp8(**x, **tail)
    assert lib.gdn_get_device_status() == lib.GDN_ERR_INVALID_ARG
    assert lib.gdn_get_device_status() == 0
    got = x["state_pool"].clone()
    # the same with those rows marked as padding
    x["slots"][1], x["slots"][B - 1] = -1, -1
    x["state_pool"].copy_(before)
    q2, s2, _ = g.gdn_decode_step_pooled_gated_fp8(**x, **tail)
    assert lib.gdn_get_device_status() == 0
    assert torch.equal(got, x["state_pool"]) and torch.equal(xs, s2) and torch.equal(xq.view(torch.uint8), q2.view(torch.uint8))
    assert (xs[1] == 0).all() and (xs[B - 1] == 0).all() and (xs[0] > 0).all()

    C = 264
    c = torch.randn(B, C, device="cuda").to(BF)
    w, pool = torch.randn(C, 4, device="cuda"), torch.randn(80, 3, C, device="cuda").to(BF)
    at = good.clone()
    at[B - 1], at[1] = at[0], 80
    p1, p2 = pool.clone(), pool.clone()
    y1 = g.gdn_short_conv1d_silu_decode_pooled(c, w, p1, at)
    assert lib.gdn_get_device_status() == lib.GDN_ERR_INVALID_ARG
    at[B - 1], at[1] = -1, -2
    y2 = g.gdn_short_conv1d_silu_decode_pooled(c, w, p2, at)
    assert lib.gdn_get_device_status() == 0
    assert torch.equal(y1, y2) and torch.equal(p1, p2)


def test_no_slots_at_all(g):
    """An empty pool with padded rows only, and an empty batch."""
    x, tail = batch(2, 1, 2, 2, (0, 1), seed=5)
    x["state_pool"] = x["state_pool"][:0]
    xq, xs, _ = g.gdn_decode_step_pooled_gated_fp8(**x, **tail)
    assert (xs == 0).all() and (xq.float() == 0).all()
    x, tail = batch(0, 1, 2, 2, seed=5)
    assert g.gdn_decode_step_pooled(**x).shape == (0, 2, 128)


def test_large_pool_offsets(g):
    """Slots whose states lie past 2^31 elements."""
    Hv, n = 16, 8300                         # 8300 * 16 * 16384 = 2.18e9 elements
    x, _ = batch(2, 16, Hv, 4, seed=6)
    pool = torch.empty(n, Hv, 128, 128, device="cuda")
    assert pool.numel() > 2 ** 31
    at = torch.tensor([n - 1, n - 2], dtype=torch.int32, device="cuda")
    pool[at.long()] = x["state_pool"][:2]
    S = x["state_pool"][:2].clone()
    o = g.gdn_decode_step_pooled(**{**x, "state_pool": pool, "slots": at}, out_dtype=F32)
    o2 = g.gdn_decode_step(x["q"], x["k"], x["v"], x["a"], x["b"], x["A_log"], x["dt_bias"], S, out_dtype=F32)
    assert torch.equal(o, o2) and torch.equal(pool[at.long()], S)


@pytest.mark.parametrize("B,C,K,slots,dead", [(1, 8, 4, 1, ()), (3, 264, 4, 5, (1,)), (5, 1032, 3, 9, (0, 4)), (6, 2048, 2, 6, ()),
                                              (2, 128, 1, 2, ()), (70, 6144, 4, 90, (7, 69))])
def test_conv_equals_contiguous(g, B, C, K, slots, dead):
    gen = torch.Generator("cuda").manual_seed(C + K)
    row = torch.randn(B, C + 40, device="cuda", generator=gen).to(BF)
    x = row[:, 16:16 + C]
    w = torch.randn(C, K, device="cuda", generator=gen)
    pool = torch.randn(slots, K - 1, C, device="cuda", generator=gen).to(BF)
    at = torch.randperm(slots, device="cuda", generator=gen)[:B].to(torch.int32)
    for i in dead:
        at[i] = -5
    live = (at >= 0).nonzero().squeeze(1)
    st = pool[at[live].long()].clone()
    y_ref = g.gdn_short_conv1d_silu_decode(x[live], w, st)
    want = pool.clone()
    want[at[live].long()] = st
    n_pool, n_x = to_np(pool)[at.cpu().numpy()], to_np(x)
    y = torch.full((B, C), 4.0, dtype=BF, device="cuda")
    g.gdn_short_conv1d_silu_decode_pooled(x, w, pool, at, y=y)
    expect = torch.full_like(y, 4.0)
    expect[live] = y_ref
    assert torch.equal(y, expect) and torch.equal(pool, want)
    win = np.concatenate([n_pool, n_x[:, None]], 1).astype(np.float64)
    pre = np.einsum("bkc,ck->bc", win, to_np(w).astype(np.float64))
    ref = (pre / (1 + np.exp(-pre)))[live.cpu().numpy()]
    assert (np.abs(to_np(y_ref) - ref) <= TOL_CONV_RTOL * np.abs(ref) + TOL_CONV_ATOL).all()


def test_conv_planes(g):
    B, widths = 5, (128, 128, 256)
    C = sum(widths)
    x, w = torch.randn(B, C, device="cuda").to(BF), torch.randn(C, 4, device="cuda")
    pool = torch.randn(7, 3, C, device="cuda").to(BF)
    at = torch.tensor([6, 0, -1, 3, 2], dtype=torch.int32, device="cuda")
    whole = g.gdn_short_conv1d_silu_decode_pooled(x, w, pool.clone(), at)
    parts = g.gdn_short_conv1d_silu_decode_pooled(x, w, pool, at, parts=widths)
    assert torch.equal(torch.cat(parts, 1), whole) and (whole[2] == 0).all()


def test_two_batches_of_one_pool_at_once(g):
    """Two calls on two streams, their slots interleaved in one pool, equal the calls made one after the other."""
    gen = torch.Generator("cuda").manual_seed(5)
    r = lambda *s: torch.randn(*s, device="cuda", generator=gen)  # noqa: E731
    B, Hk, Hv, slots = 40, 4, 8, 80
    at = [torch.arange(i, slots, 2, dtype=torch.int32, device="cuda") for i in (0, 1)]
    rows = [[r(B, Hk, 128).to(BF), r(B, Hk, 128).to(BF), r(B, Hv, 128).to(BF), r(B, Hv), r(B, Hv)] for _ in at]
    A_log, dt_bias, pool = torch.rand(Hv, device="cuda"), torch.zeros(Hv, device="cuda"), r(slots, Hv, 128, 128)
    one = pool.clone()
    want = [g.gdn_decode_step_pooled(*x, A_log, dt_bias, one, s) for x, s in zip(rows, at)]
    streams, outs = [torch.cuda.Stream(), torch.cuda.Stream()], [torch.empty_like(w) for w in want]
    torch.cuda.synchronize()
    for x, s, o, st in zip(rows, at, outs, streams):
        g.gdn_decode_step_pooled(*x, A_log, dt_bias, pool, s, o=o, stream=st)
    torch.cuda.synchronize()
    assert torch.equal(pool, one) and all(torch.equal(a, b) for a, b in zip(outs, want))


class Layer:
    """One layer served in FP8: encode, fused input projection, convolution, delta rule + tail, output projection."""

    def __init__(self, g, slots, Hk=2, Hv=4, d_model=384, seed=0):
        self.g, self.Hk, self.Hv, self.slots = g, Hk, Hv, slots
        gen = torch.Generator("cuda").manual_seed(seed)
        r = lambda *s: torch.randn(*s, device="cuda", generator=gen)  # noqa: E731
        self.C = (2 * Hk + Hv) * 128
        self.N = self.C + Hv * 128 + 16
        self.w_in, self.w_out = r(self.N, d_model) * d_model ** -0.5, r(d_model, Hv * 128) * (Hv * 128) ** -0.5
        self.win_q, self.wout_q = g.fp8_quantize_weight(self.w_in), g.fp8_quantize_weight(self.w_out)
        self.conv_w = r(self.C, 4) * 0.5
        self.A_log, self.dt_bias = torch.rand(Hv, device="cuda", generator=gen) * 2.7, torch.zeros(Hv, device="cuda")
        self.norm_w = torch.rand(128, device="cuda", generator=gen) + 0.5
        self.conv_pool = torch.zeros(slots, 3, self.C, dtype=BF, device="cuda")
        self.pool = torch.zeros(slots, Hv, 128, 128, device="cuda")

    def step(self, x, at, seen=None):
        g, Hk, Hv, C = self.g, self.Hk, self.Hv, self.C
        B = x.shape[0]
        p = g.fp8_gemm(*g.fp8_quantize_act(x), *self.win_q)
        q, k, v = g.gdn_short_conv1d_silu_decode_pooled(p[:, :C], self.conv_w, self.conv_pool, at, parts=(Hk * 128, Hk * 128, Hv * 128))
        xq, xs, _ = g.gdn_decode_step_pooled_gated_fp8(
            q.view(B, Hk, 128), k.view(B, Hk, 128), v.view(B, Hv, 128), p[:, C + Hv * 128:][:, :Hv], p[:, C + Hv * 128 + 8:][:, :Hv],
            self.A_log, self.dt_bias, self.pool, at, p[:, C:C + Hv * 128].unflatten(1, (Hv, 128)), self.norm_w)
        if seen is not None:
            seen.update(p=p, xq=xq, xs=xs)
        return g.fp8_gemm(xq, xs, *self.wout_q)


def decoded(q, s, rows):
    return q.double() * s.double().repeat_interleave(rows, 0)[:q.shape[0]].repeat_interleave(128, 1)[:, :q.shape[1]]


def check_product(y, x, xs, w, ws):
    """As for the GEMM's own test: (128 + blocks + 3) 2^-23 sum |a b|, and half a step of bf16."""
    a, b = decoded(x, xs, 1), decoded(w, ws, 128)
    ref, size = a @ b.t(), a.abs() @ b.abs().t()
    assert ((y.double() - ref).abs() <= (131 + xs.shape[1]) * 2.0 ** -23 * size + 2.0 ** -8 * ref.abs()).all()


def test_layer_in_fp8_over_steps(g):
    """Requests join, pause and leave over eight steps. Link by link: the products against 64 bits on the codes
    they were given, the rest bit for bit against the calls on one request's own states (the convolution,
    the delta rule in fp32, the plain tail, the encoder)."""
    L = Layer(g, slots=6)
    Hk, Hv, C = L.Hk, L.Hv, L.C
    hist, S = {}, {}
    gen = torch.Generator("cuda").manual_seed(1)
    plan = [[0], [0, 3], [3, -1, 0, 5], [5, 0], [-1, -1], [1, 0, 2, 3, 4, 5], [4, 5, -1], [2, 1, 0]]
    for at in plan:
        x = torch.randn(len(at), 384, device="cuda", generator=gen).to(BF)
        seen = {}
        y = L.step(x, torch.tensor(at, dtype=torch.int32, device="cuda"), seen)
        check_product(seen["p"], *g.fp8_quantize_act(x), *L.win_q)
        check_product(y, seen["xq"], seen["xs"], *L.wout_q)
        for i, slot in enumerate(at):
            if slot < 0:
                assert (y[i] == 0).all() and (seen["xs"][i] == 0).all()
                continue
            p = seen["p"][i:i + 1]
            h = hist.setdefault(slot, torch.zeros(1, 3, C, dtype=BF, device="cuda"))
            q, k, v = g.gdn_short_conv1d_silu_decode(p[:, :C].contiguous(), L.conv_w, h, parts=(Hk * 128, Hk * 128, Hv * 128))
            st = S.setdefault(slot, torch.zeros(1, Hv, 128, 128, device="cuda"))
            z, a, b = (p[:, C + o:C + o + n].contiguous() for o, n in ((0, Hv * 128), (Hv * 128, Hv), (Hv * 128 + 8, Hv)))
            o = g.gdn_decode_step(q.view(1, Hk, 128), k.view(1, Hk, 128), v.view(1, Hv, 128), a.float(), b.float(), L.A_log,
                                  L.dt_bias, st, out_dtype=F32)
            xq, xs = g.fp8_quantize_act(g.gdn_gated_rmsnorm_silu(o, z.view(1, Hv, 128).float(), L.norm_w))
            assert torch.equal(seen["xs"][i], xs[0]) and torch.equal(seen["xq"][i].view(torch.uint8), xq[0].view(torch.uint8))
    for slot in range(6):
        assert torch.equal(L.pool[slot], S[slot][0]) and torch.equal(L.conv_pool[slot], hist[slot][0])


def test_layer_captured(g):
    """The five launches captured once and replayed equal the eager steps bit for bit."""
    A, Bq = Layer(g, 8, seed=2), Layer(g, 8, seed=2)
    x, at = torch.zeros(5, 384, dtype=BF, device="cuda"), torch.tensor([4, -1, 7, 0, 2], dtype=torch.int32, device="cuda")
    s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=s):
        y = A.step(x, at)
    for i in range(4):
        x.copy_(torch.randn(5, 384, device="cuda", generator=torch.Generator("cuda").manual_seed(i)).to(BF))
        if i == 2:
            at.copy_(torch.tensor([0, 1, -1, -1, 7], dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, Bq.step(x, at))
    assert torch.equal(A.pool, Bq.pool) and torch.equal(A.conv_pool, Bq.conv_pool)
