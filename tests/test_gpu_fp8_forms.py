"""The FP8 GEMM's kernels one by one: their ends, where a CTA pair's last signals are still on their way, and what runs on
the same SMs next."""
import pytest
import torch

from test_gpu_fp8 import check_gemm, gemm_operands

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def g():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gated_deltanet_03_b200 as lib
    lib.gdn_get_device_status()
    yield lib
    assert lib.gdn_get_device_status() == 0


# fewer K blocks than accumulators, than ring stages, more than both; one tile a pair, and several
@pytest.mark.parametrize("M,N,K", [(8192, 256, 16), (8192, 1024, 144), (4096, 1536, 384), (20000, 1040, 640), (2048, 2048, 1152)])
def test_what_follows_a_wide_product(g, M, N, K):
    """Products on CTA pairs, each with a small product on the same SMs right behind it: no late signal of a pair lands
    in what the next CTAs keep in shared memory."""
    wide, small = gemm_operands(M, N, K, 1), gemm_operands(5, 2048, 2064, 2)
    y, s = torch.empty(M, N, dtype=BF, device="cuda"), torch.empty(5, 2048, dtype=F32, device="cuda")
    want_y, want_s = g.fp8_gemm(*wide), g.fp8_gemm(*small, out_dtype=F32)
    check_gemm(want_y, *wide)
    check_gemm(want_s, *small)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        for _ in range(20):
            g.fp8_gemm(*wide, y=y)
            g.fp8_gemm(*small, y=s)
    for _ in range(5):
        y.zero_()
        s.zero_()
        graph.replay()
        assert torch.equal(y, want_y) and torch.equal(s, want_s)
    torch.cuda.synchronize()
    assert g.gdn_get_device_status() == 0
