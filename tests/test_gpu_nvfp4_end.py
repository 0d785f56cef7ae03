"""The end of the NVFP4 product, where a CTA pair's last signals are still on their way, and what runs on the same SMs next."""
import pytest
import torch

pytestmark = pytest.mark.gpu


# fewer K tiles than ring stages, and more; one output tile a pair, and several
@pytest.mark.parametrize("M,N,K", [(8192, 256, 64), (8192, 1024, 512), (4096, 2048, 2048), (6000, 4096, 1024)])
def test_what_follows_a_product(M, N, K):
    """Products on CTA pairs, each with a decode step on the same SMs right behind it: no late signal of a pair lands in
    what the next CTAs keep in shared memory."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gated_deltanet_03_b200 as g
    gen = torch.Generator("cuda").manual_seed(M + K)
    r = lambda *s: torch.randn(*s, device="cuda", generator=gen)  # noqa: E731
    bf = torch.bfloat16
    (aq, sa), (bq, sb) = g.nvfp4_quantize_act(r(M, K).to(bf), 1.0), g.nvfp4_quantize_act(r(N, K).to(bf), 1.0)
    y = torch.empty(M, N, dtype=bf, device="cuda")
    want = g.nvfp4_gemm(aq, sa, bq, sb, 1.0)
    # the codes decoded, in 64 bits: fp32 sums of K products, at most one unit in the last place off for each, and bf16's half step
    a, b = (g.nvfp4_dequantize_act(q, s, 1.0, out_dtype=torch.float32).double() for q, s in ((aq, sa), (bq, sb)))
    ref, size = a @ b.t(), a.abs() @ b.abs().t()
    assert ((want.double() - ref).abs() <= K * 2.0 ** -23 * size + 2.0 ** -8 * ref.abs()).all()
    q, k, v = r(64, 2, 128).to(bf), r(64, 2, 128).to(bf), r(64, 4, 128).to(bf)
    ga, gb, A_log, dt = r(64, 4), r(64, 4), torch.rand(4, device="cuda"), torch.zeros(4, device="cuda")
    pool, slots = r(64, 4, 128, 128), torch.arange(64, dtype=torch.int32, device="cuda")
    S, o = pool.clone(), torch.empty(64, 4, 128, dtype=bf, device="cuda")
    for _ in range(10):
        want_o = g.gdn_decode_step(q, k, v, ga, gb, A_log, dt, S)
        g.nvfp4_gemm(aq, sa, bq, sb, 1.0, y=y)
        g.gdn_decode_step_pooled(q, k, v, ga, gb, A_log, dt, pool, slots, o=o)
        assert torch.equal(y, want) and torch.equal(o, want_o) and torch.equal(pool, S)
    assert g.gdn_get_device_status() == 0
