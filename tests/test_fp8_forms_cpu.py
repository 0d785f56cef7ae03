"""Which form of the FP8 GEMM a call takes, worked out on the host from a device's numbers."""
import math
import random

import pytest

import gated_deltanet_03_b200 as g

DEVICES = [(148, 74, 32, 15, 74), (148, 73, 36, 17, 74), (132, 64, 30, 14, 66)]
ALL = {(f, s) for f in range(4) for s in (1, 2, 4, 8)} | {(f, 1) for f in (4, 5, 6)}


def shapes(n, seed):
    rng = random.Random(seed)
    log = lambda lo, hi: int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))  # noqa: E731
    for _ in range(n):
        yield log(1, 32768), 16 * log(1, 1024), 16 * log(1, 2048)


@pytest.mark.parametrize("device", DEVICES)
def test_every_form_and_split_is_some_call_s(device):
    seen = {g.gdn_debug_fp8_gemm_form(*s, device) for s in shapes(60000, 1)}
    assert seen == ALL


@pytest.mark.parametrize("device", DEVICES)
def test_a_pick_can_do_its_call(device):
    sms, c2, c4, c8, _ = device
    for M, N, K in shapes(20000, 2):
        form, split = g.gdn_debug_fp8_gemm_form(M, N, K, device)
        kind, tile = g.FP8_GEMM_FORMS[form]
        if kind == "wide":
            assert split == 1 and M > 64
            continue
        assert -(-M // tile) <= 65535
        if split > 1:
            per_sm = 2 if tile <= 32 else 1
            ctas = -(-N // 128) * -(-M // tile)
            assert -(-K // 128) >= 2 * split and ctas * split <= per_sm * sms
            assert ctas <= per_sm * {2: c2, 4: c4, 8: c8}[split]


@pytest.mark.parametrize("M", [16 * 65535, 16 * 65535 + 1, 64 * 65535 + 1, 128 * 65535])
def test_row_tiles_stay_within_a_grid(M):
    """On a device whose numbers favour the narrow tiles, calls of more rows than a grid has for them."""
    form, split = g.gdn_debug_fp8_gemm_form(M, 16, 16, (1 << 20, 1, 1, 1, 1))
    kind, tile = g.FP8_GEMM_FORMS[form]
    assert kind == "narrow" and -(-M // tile) <= 65535
    if M <= 16 * 65535:
        assert tile == 16


def test_refusals():
    for bad in ((0, 16, 16), (1, 0, 16), (1, 16, 0)):
        with pytest.raises(g.GdnError):
            g.gdn_debug_fp8_gemm_form(*bad, DEVICES[0])
    with pytest.raises(g.GdnError):
        g.gdn_debug_fp8_gemm_form(1, 16, 16, (0, 0, 0, 0, 0))
    A = 1 << 20
    for form in (-1, 7):
        assert g.LIB.gdn_debug_fp8_gemm(A, A, A, A, 4, 32, 64, g.GDN_BF16, A, form, 1, None) == g.GDN_ERR_INVALID_ARG
