"""The FP8 GEMM's kernels one by one: every form and split at ragged sizes, whichever the call would pick, and their ends,
where a CTA pair's last signals are still on their way, and what runs on the same SMs next."""
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


@pytest.fixture(params=[BF, F32], ids=["bf16", "fp32"])
def out(request):
    return request.param


def in_form(g, form, split, M, N, K, out):
    ops = gemm_operands(M, N, K, M + N + K)
    y = torch.full((M + 1, N), 7.0, dtype=out, device="cuda")
    g.gdn_debug_fp8_gemm(*ops, form, split, y=y[:M])
    check_gemm(y[:M], *ops)
    assert (y[M] == 7).all()                    # nothing is written past the last row
    y2 = g.gdn_debug_fp8_gemm(*ops, form, split, out_dtype=out)
    assert torch.equal(y2, y[:M])               # the order of the sums is fixed


@pytest.mark.parametrize("split", [1, 2, 4, 8])
@pytest.mark.parametrize("form", [0, 1, 2, 3])
def test_narrow_forms(g, form, split, out):
    """Every tile of rows with every split of K: one row, ragged rows on several tiles, K blocks that do not divide
    evenly among the CTAs (one each at the least) and a last block of 16 values."""
    tile = g.FP8_GEMM_FORMS[form][1]
    blocks = 2 * split + split // 2 + 1         # (of 8 CTAs some have two, some three)
    for M, N, K in ((1, 16, 128 * split), (tile, 272, 128 * blocks + 16), (3 * tile - 5, 1040, 128 * (4 * split + 7))):
        in_form(g, form, split, M, N, K, out)


@pytest.mark.parametrize("form", [4, 5, 6])
@pytest.mark.parametrize("M,N,K", [(1, 16, 16), (300, 528, 2064)])
def test_wide_forms_on_a_few_tiles(g, form, M, N, K, out):
    in_form(g, form, 1, M, N, K, out)


@pytest.mark.parametrize("form", [4, 5, 6])
@pytest.mark.parametrize("K", [384, 1232])
def test_wide_forms_over_many_tiles(g, form, K, out):
    """Three tiles and more a pair: the ring, the factors' slots, the accumulators and the output pieces run on from one
    tile to the next, with fewer K blocks than ring stages and with more."""
    N = 2064
    M = 256 * -(-3 * 74 // -(-N // g.FP8_GEMM_FORMS[form][1])) + 37
    in_form(g, form, 1, M, N, K, out)


def test_forms_that_cannot_are_refused(g):
    ops = gemm_operands(5, 32, 272, 0)          # three K blocks
    for form, split in ((0, 4), (3, 8), (0, 3), (4, 2), (6, 0), (7, 1), (-1, 1)):
        with pytest.raises(g.GdnError):
            g.gdn_debug_fp8_gemm(*ops, form, split)
    M = 16 * 65535 + 1                          # more tiles of 16 rows than a grid has
    ops = gemm_operands(M, 16, 16, 1)
    with pytest.raises(g.GdnError):
        g.gdn_debug_fp8_gemm(*ops, 0)
    check_gemm(g.gdn_debug_fp8_gemm(*ops, 1, out_dtype=F32), *ops)
    assert g.gdn_debug_fp8_gemm_form(M, 16, 16) != (0, 1)


def test_a_call_takes_the_form_that_is_picked(g):
    """fp8_gemm equals its own pick's bytes, over sizes that reach the forms."""
    for M, N, K in ((1, 2048, 4096), (30, 2048, 4112), (64, 4032, 8080), (121, 14976, 4224), (107, 6656, 7296), (256, 12352, 2048),
                    (1037, 1040, 2064), (4096, 4096, 512)):
        ops = gemm_operands(M, N, K, 3)
        form, split = g.gdn_debug_fp8_gemm_form(M, N, K)
        assert torch.equal(g.fp8_gemm(*ops), g.gdn_debug_fp8_gemm(*ops, form, split))
