"""How the softmax weights of attention over pages are rounded for the value
product: a row's largest weight is exactly 1, as in attn_decode.

Each row has two keys that count, in two tiles one after the other, the second
2^peak times as heavy as the first, and all values are 1. O is then the sum of
the rounded weights over the sum of the unrounded ones. With the weights taken
relative to the row's largest score, the second one is 1 and only the first, a
share of 2^-peak, is rounded (by half a step, 2^-8 of it): with peak >= 6, O is
within 2^-14 of 1 before its own rounding, fp32 sums included, so it has to be 1
(its neighbours in bf16 are 2^-8 and 2^-7 away). With the weights relative to
the first key's score, the second one is 2^peak, rounded by up to 2^-8 of itself,
and some rows give another number.

LSE: the scores are products of two numbers, exact in fp32; scaling, exponential,
logarithm and their sum are off by 2^-22 each, of a number of at most 8 in log2
units, below 1e-5 together."""
import math

import pytest
import torch

PEAK = 6.25  # log2 of the weights' ratio for a query of 1

PAGED = [(74, 4, 1), (74, 8, 1), (74, 16, 1), (74, 8, 4), (37, 16, 4)]  # key/value heads, group, tokens
LATENT = [(16, 1), (32, 1), (64, 1), (128, 1), (16, 4)]                 # heads, tokens


@pytest.fixture(scope="module")
def attn():
    from exact_softmax_attention_04_b200 import build_lib
    build_lib.build()
    import exact_softmax_attention_04_b200 as pkg
    return pkg


@pytest.fixture
def gpu(attn):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return attn


def factors(rows):
    """A row's query: 1 to 1.25, in bf16's steps of 2^-7."""
    return 1 + (torch.arange(rows) % 33) / 128


def two_peaks(positions, first, second):
    """Keys (of one element): 0 and 1 at the two places, far below elsewhere."""
    x = torch.full((positions,), -100.0)
    x[first], x[second] = 0.0, 1.0
    return x


@pytest.mark.parametrize("rows", sorted({G * T for _, G, T in PAGED} | {H * T for H, T in LATENT}))
def test_the_rows_tell_a_lagging_reference(rows):
    """The arithmetic restated: weights relative to the first key's score give
    another number than 1 in some row, relative to the largest none."""
    s = (factors(rows).double() * PEAK)[:, None] * two_peaks(256, 5, 135).double()
    lag, exact = torch.exp2(s), torch.exp2(s - s.amax(1, keepdim=True))
    o = [(p.bfloat16().double().sum(1) / p.sum(1)).bfloat16() for p in (lag, exact)]
    assert (o[0] != 1).any() and (o[1] == 1).all()


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hkv,G,T", PAGED)
def test_paged_largest_weight_is_exact(gpu, d, Hkv, G, T):
    B, page, n = 8, 32, 256
    k = torch.zeros((B * n // page, Hkv, page, d), dtype=torch.bfloat16, device="cuda")
    k[..., 0] = two_peaks(n, 5, 135).view(-1, 1, page).repeat(B, 1, 1).cuda()
    v = torch.ones_like(k)
    table = torch.arange(B * n // page, dtype=torch.int32, device="cuda").view(B, -1)
    lens = torch.full((B,), n, dtype=torch.int32, device="cuda")
    q = torch.zeros((B, Hkv * G, T, d), dtype=torch.bfloat16, device="cuda")
    q[..., 0] = factors(G * T).view(1, 1, G, T).expand(B, Hkv, G, T).reshape(B, Hkv * G, T).cuda()
    o, lse = gpu.attn_decode_paged(q, k, v, table, lens, scale=PEAK * math.log(2))
    assert gpu.sync_status() == gpu.ATTN_OK
    assert (o == 1).all()
    want = torch.logaddexp(torch.zeros_like(q[..., 0]).double(), q[..., 0].double() * PEAK * math.log(2))
    assert (lse.double() - want).abs().max() < 1e-5


@pytest.mark.gpu
@pytest.mark.parametrize("rank", [256, 512])
@pytest.mark.parametrize("H,T", LATENT)
def test_latent_largest_weight_is_exact(gpu, rank, H, T):
    B, page, n = 296, 32, 128
    c = torch.ones((B * n // page, page, rank + 64), dtype=torch.bfloat16, device="cuda")
    c[..., rank:] = 0
    c[..., rank] = two_peaks(n, 5, 71).view(-1, page).repeat(B, 1).cuda()
    table = torch.arange(B * n // page, dtype=torch.int32, device="cuda").view(B, -1)
    lens = torch.full((B,), n, dtype=torch.int32, device="cuda")
    q = torch.zeros((B, H, T, rank + 64), dtype=torch.bfloat16, device="cuda")
    q[..., rank] = factors(H * T).view(1, H, T).cuda()
    o, lse = gpu.attn_decode_latent(q, c, table, lens, PEAK * math.log(2))
    assert gpu.sync_status() == gpu.ATTN_OK
    assert (o == 1).all()
    want = torch.logaddexp(torch.zeros_like(q[..., rank]).double(), q[..., rank].double() * PEAK * math.log(2))
    assert (lse.double() - want).abs().max() < 1e-5
