"""FP8 encoders, tail and GEMM on the GPU against plain implementations: the encoders bit for bit against the
stated fp32 operations (numpy) and within half an E4M3 step of the formula in 64 bits, the tail bit for bit
against the two-call path, the GEMM element by element against the fp64 product of the decoded operands."""
import numpy as np
import pytest
import torch

import oracle
import workloads
from helpers import TOL_TAIL, dev, to_np

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


def codes(t):
    return t.view(torch.uint8).cpu().numpy()


def values(t):
    """The values that E4M3 codes stand for."""
    return t.float().cpu().numpy()


def blocks_of(x, rows):
    """[ceil(M / rows), ceil(K / 128), rows * 128] blocks of x, zero past the edge."""
    M, K = x.shape
    p = np.zeros((-(-M // rows) * rows, -(-K // 128) * 128), x.dtype)
    p[:M, :K] = x
    b = p.reshape(p.shape[0] // rows, rows, p.shape[1] // 128, 128).transpose(0, 2, 1, 3)
    return b.reshape(b.shape[0], b.shape[1], -1)


def spread(s, rows, shape):
    return np.repeat(np.repeat(s, rows, 0), 128, 1)[:shape[0], :shape[1]]


def encode_fp32(x, rows):
    """The header's operations in numpy fp32: scales, and the codes by torch's E4M3 rounding on the CPU."""
    with np.errstate(all="ignore"):
        amax = np.fmax.reduce(np.abs(blocks_of(x, rows)), axis=2, initial=0.0)
        s = np.maximum(amax / np.float32(448), np.float32(2.0 ** -126))
        r = np.float32(1) / s
        p = x * spread(r, rows, x.shape)
    q = torch.from_numpy(p).clamp(-448, 448).to(F8)
    return q.view(torch.uint8).numpy(), s


def special_rows(x):
    """Rows at the edges of the format in front of random ones."""
    M, K = x.shape
    rows = [np.zeros(K), np.full(K, 1e-42), np.full(K, 3e38), np.where(np.arange(K) % 7 == 3, 448.0, 2.0 ** -9)]
    for i, r in enumerate(rows[:M]):
        x[i] = r.astype(np.float32)
    return x


@pytest.mark.parametrize("M,K", [(1, 16), (5, 128), (37, 144), (257, 4096), (1000, 80), (64, 2064)])
@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [1, 128])
def test_quantize(g, M, K, io, rows):
    x = special_rows(np.random.default_rng(M * 31 + K).standard_normal((M, K)).astype(np.float32) * 3)
    if io == "bf16":
        x = workloads.round_bf16(np.clip(x, -3e38, 3e38))
    f = g.fp8_quantize_act if rows == 1 else g.fp8_quantize_weight
    xq, xs = f(dev(x, BF if io == "bf16" else F32))
    q_ref, s_ref = encode_fp32(x, rows)
    np.testing.assert_array_equal(to_np(xs), s_ref)
    np.testing.assert_array_equal(codes(xq), q_ref)
    # against the formula in 64 bits: s one rounding; codes half a step (2^-4 relative, 2^-10 below the
    # normal range) and the roundings of 1 / s and of the product (2^-24 each, and s's own, relative)
    s64 = np.maximum(np.abs(blocks_of(x.astype(np.float64), rows)).max(2) / 448, 2.0 ** -126)
    assert (np.abs(to_np(xs) - s64) <= 2.0 ** -24 * s64).all()
    v = x / spread(s64, rows, x.shape)
    assert (np.abs(values(xq) - v) <= np.maximum(2.0 ** -4 * np.abs(v), 2.0 ** -10) + 3 * 2.0 ** -24 * np.abs(v)).all()


@pytest.mark.parametrize("rows", [1, 128])
def test_quantize_not_finite(g, rows):
    """NaN stays NaN and is passed over by the scale; an infinity makes the scale infinite, the block NaN."""
    x = np.random.default_rng(5).standard_normal((200, 384)).astype(np.float32)
    x[3, 5] = np.nan
    x[130, 300] = -np.inf
    x[140, 128:256] = np.nan
    f = g.fp8_quantize_act if rows == 1 else g.fp8_quantize_weight
    xq, xs = f(dev(x, F32))
    q_ref, s_ref = encode_fp32(x, rows)
    np.testing.assert_array_equal(to_np(xs), s_ref)
    got, want = codes(xq), q_ref
    nan = np.isnan(torch.from_numpy(want).view(F8).float().numpy())
    np.testing.assert_array_equal((got & 127) == 127, nan)
    np.testing.assert_array_equal(got[~nan], want[~nan])
    with np.errstate(invalid="ignore"):
        back = values(xq) * spread(to_np(xs), rows, x.shape)
    assert np.isnan(back[130, 256:]).all() and np.isnan(back[3, 5])
    assert np.isfinite(back[3, 6:128]).all()


def test_quantize_strided(g):
    big = torch.randn(70, 640, device="cuda").to(BF)
    for x in (big[:, 128:400], big[::3, 64:208], big[5:6, 8:24]):
        for f in (g.fp8_quantize_act, g.fp8_quantize_weight):
            for a, b in zip(f(x), f(x.contiguous())):
                assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("M,Hv,D", [(1, 1, 16), (3, 5, 16), (67, 3, 32), (33, 7, 64), (130, 1, 128), (257, 32, 128)])
@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_tail(g, M, Hv, D, io):
    rng = np.random.default_rng(M + Hv + D)
    o, z = (rng.standard_normal((M, Hv, D)).astype(np.float32) for _ in range(2))
    o[0] = 0
    z[-1] *= 40
    if io == "bf16":
        o, z = workloads.round_bf16(o), workloads.round_bf16(z)
    w = rng.uniform(0.5, 1.5, D).astype(np.float32)
    dt = BF if io == "bf16" else F32
    xq, xs = g.gdn_gated_rmsnorm_silu_fp8(dev(o, dt), dev(z, dt), dev(w, F32))
    # the same bytes as the plain tail in fp32 and then the encoder
    y = g.gdn_gated_rmsnorm_silu(dev(o, dt), dev(z, dt), dev(w, F32), out_dtype=F32)
    q2, s2 = g.fp8_quantize_act(y)
    assert torch.equal(xs, s2) and torch.equal(xq.view(torch.uint8), q2.view(torch.uint8))
    # against the formula in 64 bits: the tail's own tolerance relative to each value plus half a step
    ref = oracle.gated_rmsnorm_silu(o, z, w).reshape(M, Hv * D).astype(np.float64)
    s64 = np.maximum(np.abs(blocks_of(ref, 1)).max(2) / 448, 2.0 ** -126)
    assert (np.abs(to_np(xs) - s64) <= TOL_TAIL * s64).all()
    v = ref / spread(s64, 1, ref.shape)
    assert (np.abs(values(xq) - v) <= np.maximum(2.0 ** -4 * np.abs(v), 2.0 ** -10) + 2 * TOL_TAIL * np.abs(v)).all()


def gemm_operands(M, N, K, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    kb = -(-K // 128)
    aq = (torch.randn(M, K, device="cuda", generator=gen) * 60).clamp(-448, 448).to(F8)
    bq = (torch.randn(N, K, device="cuda", generator=gen) * 60).clamp(-448, 448).to(F8)
    as_ = torch.rand(M, kb, device="cuda", generator=gen) * 0.02 + 1e-3
    bs = torch.rand(-(-N // 128), kb, device="cuda", generator=gen) * 0.02 + 1e-3
    return aq, as_, bq, bs


def check_gemm(y, aq, as_, bq, bs):
    """|y - ref| <= (128 + blocks + 3) 2^-23 sum |a b| + half a step of y's type: at most 128 additions inside a
    block and one per block, each off by no more than one unit in the last place (2^-23, which also covers
    an accumulator that truncates), the factor's product and the final rounding."""
    M, K = aq.shape
    kcol, nrow = torch.arange(K, device="cuda") // 128, torch.arange(bq.shape[0], device="cuda") // 128
    a, b = aq.double() * as_.double()[:, kcol], bq.double() * bs.double()[nrow][:, kcol]
    ref, size = a @ b.t(), a.abs() @ b.abs().t()
    tol = (128 + as_.shape[1] + 3) * 2.0 ** -23 * size + torch.finfo(y.dtype).eps / 2 * ref.abs()
    assert ((y.double() - ref).abs() <= tol).all()


# token counts around every tile width, ragged N and K, split and unsplit K, more than one tile each way
@pytest.mark.parametrize("M,N,K", [(1, 16, 16), (1, 2048, 4096), (3, 144, 144), (16, 272, 2064), (17, 128, 128), (32, 2048, 512),
                                   (33, 16, 8192), (64, 1040, 1040), (65, 128, 256), (128, 12352, 2048), (129, 48, 400),
                                   (256, 4096, 128), (300, 1040, 2064), (511, 528, 5120), (1024, 2048, 640), (2100, 784, 1552),
                                   (4096, 1024, 2048), (5000, 2064, 272),
                                   # K split over two, four and eight CTAs at each tile width, uneven shares among them
                                   (5, 4096, 2064), (16, 6208, 8192), (8, 10240, 5136), (30, 2048, 4112), (64, 1024, 2320),
                                   (100, 1024, 4112), (128, 4096, 8208), (200, 1024, 8192), (75, 5280, 6048)])
@pytest.mark.parametrize("out", [BF, F32])
def test_gemm(g, M, N, K, out):
    ops = gemm_operands(M, N, K, M + N + K)
    y = torch.full((M + 1, N), 7.0, dtype=out, device="cuda")
    g.fp8_gemm(*ops, y=y[:M])
    check_gemm(y[:M], *ops)
    assert (y[M] == 7).all()          # nothing is written past the last row
    y2 = g.fp8_gemm(*ops, out_dtype=out)
    assert torch.equal(y2, y[:M])     # the order of the sums is fixed


@pytest.mark.parametrize("M", [1, 40, 200, 2048])
def test_gemm_nan_stays_in_its_row_and_column(g, M):
    """A NaN code reaches its own row (or column) of y only, a zero scale of a block drops the block."""
    N, K = 272, 400
    aq, as_, bq, bs = gemm_operands(M, N, K, 1)
    as_[0, 1] = 0
    clean = g.fp8_gemm(aq, as_, bq, bs, out_dtype=F32)
    check_gemm(clean, aq, as_, bq, bs)
    bad = bq.clone()
    bad.view(torch.uint8)[200, 390] = 0x7F
    y = g.fp8_gemm(aq, as_, bad, bs, out_dtype=F32)
    assert y[:, 200].isnan().all()
    keep = [n for n in range(N) if n != 200]
    assert torch.equal(y[:, keep], clean[:, keep])
    if M > 1:
        bad = aq.clone()
        bad.view(torch.uint8)[M - 2, 3] = 0xFF
        y = g.fp8_gemm(bad, as_, bq, bs, out_dtype=F32)
        assert y[M - 2].isnan().all()
        keep = [m for m in range(M) if m != M - 2]
        assert torch.equal(y[keep], clean[keep])


def test_gemm_large_output_offsets(g):
    """y of more than 2^31 elements: the last rows against the product of those rows alone."""
    M, N, K = 131200, 16400, 128
    aq, as_, bq, bs = gemm_operands(M, N, K, 2)
    y = g.fp8_gemm(aq, as_, bq, bs)
    assert y.numel() > 2 ** 31
    for sl in (slice(0, 200), slice(M - 200, M)):
        check_gemm(y[sl], aq[sl], as_[sl], bq, bs)


def test_gemm_many_rows(g):
    """More row tiles of 16 than a grid has rows."""
    ops = gemm_operands(1100000, 16, 16, 3)
    check_gemm(g.fp8_gemm(*ops, out_dtype=F32), *ops)


def test_two_graphs_at_once(g):
    """Two captured chains replayed side by side on two streams, nothing of one in the other's results."""
    chains, streams = [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for i, M in enumerate((9, 300)):
        x, ops = torch.randn(M, 2064, device="cuda").to(BF), gemm_operands(8, 1040, 2064, i)
        want = g.fp8_gemm(*g.fp8_quantize_act(x), *ops[2:])
        streams[i].wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=streams[i]):
            y = g.fp8_gemm(*g.fp8_quantize_act(x), *ops[2:])
        chains.append((graph, y, want, x, ops))
    for _ in range(30):
        for c, s in zip(chains, streams):
            with torch.cuda.stream(s):
                c[0].replay()
    torch.cuda.synchronize()
    for _, y, want, _, _ in chains:
        assert torch.equal(y, want)


def test_graph_and_streams(g):
    """Captured and replayed with new contents, and two products on two streams at once."""
    ops = [gemm_operands(M, 2048, 4096, M) for M in (4, 700)]
    want = [g.fp8_gemm(*o) for o in ops]
    outs = [torch.empty_like(w) for w in want]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        g.fp8_gemm(*ops[0], y=outs[0], stream=side)
        g.fp8_gemm(*ops[1], y=outs[1])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))

    x = torch.randn(7, 4096, device="cuda").to(BF)
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    xq, xs = torch.empty(7, 4096, dtype=F8, device="cuda"), torch.empty(7, 32, device="cuda")
    y = torch.empty(7, 2048, dtype=BF, device="cuda")
    with torch.cuda.graph(graph, stream=s):
        g.fp8_quantize_act(x, xq, xs)
        g.fp8_gemm(xq, xs, ops[0][2], ops[0][3], y=y)
    for seed in (1, 2):
        x.copy_(torch.randn(7, 4096, device="cuda", generator=torch.Generator("cuda").manual_seed(seed)).to(BF))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, g.fp8_gemm(*g.fp8_quantize_act(x), ops[0][2], ops[0][3]))


def test_empty(g):
    w, ws = g.fp8_quantize_weight(torch.randn(32, 64, device="cuda"))
    xq, xs = g.fp8_quantize_act(torch.empty(0, 64, device="cuda"))
    assert xq.shape == (0, 64) and xs.shape == (0, 1)
    assert g.fp8_gemm(xq, xs, w, ws).shape == (0, 32)
    e = torch.empty(0, 2, 128, device="cuda")
    assert g.gdn_gated_rmsnorm_silu_fp8(e, e, torch.ones(128, device="cuda"))[0].shape == (0, 256)
