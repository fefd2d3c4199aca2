"""Table entries that are no page: any number outside [0, num_pages), to every
operator alike. Expected values are written out."""
import pytest
import torch

TOP = 2 ** 31 - 1


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


def int32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.gpu
@pytest.mark.parametrize("others", [0, 40])  # (beyond 32 requests the plan takes three launches)
def test_reserve_fills_every_entry_that_is_no_page(gpu, others):
    P, page = 8, 4
    table = int32([[3, P, -1, TOP], [P, P + 1, 5, -9], [-1] * 4])
    refs = int32([0, 0, 0, 1, 0, 1, 0, 0])
    rows, want = [0, 1, 2] + [99] * others, [16, 16, 4] + [0] * others
    granted = gpu.pages_reserve(table, refs, int32(rows), int32(want), page)
    # free: 0 1 2 4 6 7; three for row 0, three for row 1, none left for row 2
    assert granted.tolist() == [1, 1, 0] + [0] * others
    assert table.tolist() == [[3, 0, 1, 2], [4, 6, 5, 7], [-1] * 4]
    assert refs.tolist() == [1] * P
    # what was granted holds tokens
    k = torch.zeros((P, page, 8), dtype=torch.bfloat16, device="cuda")
    new = torch.arange(1, 33, device="cuda").bfloat16().view(2, 1, 16, 1).expand(-1, -1, -1, 8).contiguous()
    gpu.pages_append(new, None, k, None, table[:2].contiguous(), int32([0, 0]))
    assert torch.equal(k[table[:2].long()].view(2, 16, 8), new[:, 0])


@pytest.mark.gpu
def test_reserve_leaves_a_row_that_it_refuses(gpu):
    table, refs = int32([[9, 4, -1, -1], [0, -1, -1, -1]]), int32([1, 0, 1, 0])
    granted = gpu.pages_reserve(table, refs, int32([0, 1]), int32([3, 2]), 1)  # three asked for, two free
    assert granted.tolist() == [0, 0]
    assert table.tolist() == [[9, 4, -1, -1], [0, -1, -1, -1]] and refs.tolist() == [1, 0, 1, 0]


@pytest.mark.gpu
def test_fork_takes_a_child_whose_first_entry_is_no_page(gpu):
    P, page = 8, 4
    k = torch.arange(P * page, device="cuda").bfloat16().view(P, page, 1).expand(-1, -1, 8).contiguous()
    table = int32([[3, 5, -1], [P, -1, -1], [TOP, 7, -1], [6, -1, -1]])
    lens, refs = int32([6, 0, 0, 0]), int32([0, 0, 0, 1, 0, 1, 0, 0])
    fresh, granted = gpu.pages_fork(k, None, table, lens, refs, int32([0, 0, 0]), int32([1, 2, 3]))
    # row 3 holds page 6 in its first entry: not empty
    assert granted.tolist() == [1, 1, 0] and fresh.tolist() == [0, 1, -1]
    assert table.tolist() == [[3, 5, -1], [3, 0, -1], [3, 1, -1], [6, -1, -1]]
    assert lens.tolist() == [6, 6, 6, 0] and refs.tolist() == [1, 1, 0, 3, 0, 1, 0, 0]
    for p in (0, 1):
        assert torch.equal(k[p, :2], k[5, :2])


@pytest.mark.gpu
def test_fork_takes_a_child_whose_length_is_negative(gpu):
    """A negative length counts as 0, a parent's and a child's."""
    P, page = 8, 4
    k = torch.zeros((P, page, 8), dtype=torch.bfloat16, device="cuda")
    table = int32([[3, 5], [-1, -1], [2, -1], [-1, -1]])
    lens, refs = int32([8, -3, -1, 0]), int32([0, 0, 1, 1, 0, 1, 0, 0])
    fresh, granted = gpu.pages_fork(k, None, table, lens, refs, int32([0, 2]), int32([1, 3]))
    assert granted.tolist() == [1, 1] and fresh.tolist() == [-1, -1]
    assert table.tolist() == [[3, 5], [3, 5], [2, -1], [-1, -1]]
    assert lens.tolist() == [8, 8, -1, 0] and refs.tolist() == [0, 0, 1, 2, 0, 2, 0, 0]
