"""Paged caches in the parts of their ranges that change a kernel's path: more
rows than a plan keeps in shared memory, positions past 32 bits, windows with
every layout, group and batch size, chunks, and rows of many heads."""
import random

import pytest
import torch

from paged_reference import attention, check
from test_paged import make, paged_case, queries
from test_pages import Both, int32


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


@pytest.mark.gpu
@pytest.mark.parametrize("n", [20, 3000])
def test_more_rows_than_a_plan_keeps_in_shared_memory(gpu, n):
    """8192 of them it does; rows named twice and out of range among the requests."""
    R, P = 9001, 20000
    rng = random.Random(n)
    s = Both(R, 4, P, 1, 2, 8, "latent", 5)
    some = lambda: [rng.choice([rng.randrange(R), rng.randrange(8000, R), R - 1, -1, R]) for _ in range(n)]
    rows, want = some(), [rng.randrange(10) for _ in range(n)]
    ok = s.reserve(gpu, rows, want)
    lens = [0] * R
    for r, w, y in zip(rows, want, ok):
        if y:
            lens[r] = w
    s.set_lens(lens)
    s.fork(gpu, some(), some())
    s.free(gpu, some())
    s.reserve(gpu, some(), [8] * n)
    s.compact(gpu)


@pytest.mark.gpu
@pytest.mark.parametrize("pools", [1, 2])
def test_append_at_positions_past_32_bits(gpu, pools):
    """A table of 2^32 + 2^17 positions; tokens on both sides of 2^31."""
    page, width, d = 1 << 16, (1 << 16) + 2, 8
    k = torch.zeros((3, 1, page, d), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    table = torch.full((2, width), -1, dtype=torch.int32, device="cuda")
    at = 1 << 15  # position 2^31's entry
    table[0, at - 1], table[0, at], table[1, at - 1] = 2, 0, 1
    new = torch.randn((2, 1, 7, d), device="cuda").bfloat16()
    pos = int32([2 ** 31 - 3, 2 ** 31 - 2])  # the second row has no page behind 2^31
    if pools == 2:
        gpu.pages_append(new, -new, k, v, table, pos)
    else:
        gpu.pages_append(new, None, k, None, table, pos)
    want = torch.zeros_like(k)
    want[2, 0, -3:], want[0, 0, :4], want[1, 0, -2:] = new[0, 0, :3], new[0, 0, 3:], new[1, 0, :2]
    assert torch.equal(k, want) and torch.equal(v, -want if pools == 2 else torch.zeros_like(v))


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("layout", ["hnd", "nhd"])
@pytest.mark.parametrize("Hkv,G,T", [(2, 4, 1), (1, 8, 4), (2, 3, 9), (1, 4, 20)])
@pytest.mark.parametrize("window", [0, 100, 333])
def test_windows_with_every_layout_and_group(gpu, d, layout, Hkv, G, T, window):
    paged_case(gpu, Hkv, G, T, d, 16, [0, 3, 129, 700, 1500], window=window, layout=layout, seed=window + T)


@pytest.mark.gpu
@pytest.mark.parametrize("Hkv,G,T", [(1, 4, 1), (1, 10, 2)])
def test_windows_over_more_sequences_than_the_joining_kernel_sums(gpu, Hkv, G, T):
    paged_case(gpu, Hkv, G, T, 64, 8, [(i * 137) % 2500 for i in range(200)], window=400, layout="nhd", seed=G)


@pytest.mark.gpu
@pytest.mark.parametrize("window", [-1, 150])
def test_a_chunk_of_a_prompt(gpu, window):
    """64 tokens x 4 heads: 256 columns, the most there may be; the first tokens of
    a short sequence see nothing."""
    paged_case(gpu, 2, 4, 64, 128, 64, [40, 64, 1000, 2049], window=window, seed=3)


@pytest.mark.gpu
@pytest.mark.parametrize("rank", [256, 512])
@pytest.mark.parametrize("H,T", [(16, 2), (128, 1)])
def test_latent_rows_of_more_sequences_than_the_joining_kernel_sums(gpu, rank, H, T):
    lens = [(i * 137) % 900 for i in range(150)]
    c, _, table, ln, g = make(len(lens), 1, 8, rank + 64, lens, 4)
    q = queries(g, len(lens), H, T, rank + 64)
    o, lse = gpu.attn_decode_latent(q, c[:, 0], table, ln, 0.07)
    assert gpu.sync_status() == gpu.ATTN_OK
    check(o, lse, attention(q, c, c[..., :rank], table, ln, 0.07))
