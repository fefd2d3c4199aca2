"""What the paged kernels report when they cannot do their work, without a GPU
fault: a build with a test-only hook takes the latent kernel's shared memory for
unusable, so that every block returns at once."""
import pytest
import torch

from paged_reference import attention, check


@pytest.mark.gpu
@pytest.mark.parametrize("B", [3, 200])  # (beyond 128 sequences the joining kernel reads what the first one planned)
def test_unusable_shared_memory_is_reported_as_such(B, fault_lib):
    import exact_softmax_attention_04_b200 as pkg
    page, n, rank, H = 16, 100, 256, 8
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    c = torch.randn((B * 7, page, rank + 64), generator=g, device="cuda").bfloat16()
    q = torch.randn((B, H, 1, rank + 64), generator=g, device="cuda").bfloat16()
    table = torch.arange(B * 7, dtype=torch.int32, device="cuda").view(B, 7)
    lens = torch.full((B,), n, dtype=torch.int32, device="cuda")
    ws = torch.full((pkg.decode_latent_workspace_bytes(B, H, 1, 7, page, rank),), 255, dtype=torch.uint8, device="cuda")
    o, lse = torch.empty((B, H, 1, rank), dtype=torch.bfloat16, device="cuda"), torch.empty((B, H, 1), device="cuda")
    stream = torch.cuda.current_stream().cuda_stream
    assert fault_lib.attn_decode_latent(q.data_ptr(), c.data_ptr(), None, table.data_ptr(), lens.data_ptr(),
                                        o.data_ptr(), lse.data_ptr(), ws.data_ptr(), ws.numel(), B, H, 1, B * 7, page,
                                        7, rank, 0.05, stream) == pkg.ATTN_OK
    assert fault_lib.attn_sync_status(stream) == pkg.ATTN_ERR_CUDA
    assert fault_lib.attn_sync_status(stream) == pkg.ATTN_OK  # read and cleared
    # the context is intact
    o, lse = pkg.attn_decode_latent(q, c, table, lens, 0.05)
    assert pkg.sync_status() == pkg.ATTN_OK
    check(o, lse, attention(q, c[:, None], c[:, None, :, :rank], table, lens, 0.05))


@pytest.fixture(scope="module")
def fault_lib(tmp_path_factory):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import exact_softmax_attention_04_b200 as pkg
    from exact_softmax_attention_04_b200 import build_lib
    build_lib.build()
    path = tmp_path_factory.mktemp("fault") / "libattn_fault_latent.so"
    return pkg.load_library(build_lib.build_variant(path, ["ATTN_FAULT_LATENT_SMEM_BASE"]))
