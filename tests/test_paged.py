"""Attention over paged caches (attn_decode_paged, attn_decode_latent) against
plain 64-bit sums, with bounds derived in paged_reference.bounds, and their
refusals."""
import math

import pytest
import torch

from paged_reference import attention, check

FAKE = 0x10000  # 16-byte aligned, never dereferenced


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


# ---------------------------------------------------------------- refusals

PAGED = dict(q=FAKE, k=FAKE, v=FAKE, strides=None, table=FAKE, lens=FAKE, o=FAKE, lse=FAKE, workspace=FAKE,
             ws_bytes=1 << 40, B=2, H=8, Hkv=2, T=1, P=64, page=16, width=8, window=-1, d=128, scale=0.1)


def strides(*s):
    import ctypes
    return (ctypes.c_int64 * len(s))(*s)


@pytest.mark.parametrize("kw,code", [
    (dict(q=0), 1), (dict(k=0), 1), (dict(v=0), 1), (dict(table=0), 1), (dict(lens=0), 1), (dict(o=0), 1),
    (dict(lse=0), 1), (dict(workspace=0), 1), (dict(ws_bytes=0), 1), (dict(q=FAKE + 8), 1), (dict(v=FAKE + 8), 1),
    (dict(table=FAKE + 2), 1), (dict(B=0), 1), (dict(T=0), 1), (dict(P=0), 1), (dict(width=0), 1),
    (dict(page=0), 1), (dict(H=0), 1), (dict(Hkv=3), 1), (dict(scale=0.0), 1), (dict(scale=math.nan), 1),
    (dict(scale=math.inf), 1), (dict(strides=strides(4096, 2048, 127)), 1), (dict(strides=strides(4096, 2048, 132)), 1),
    (dict(strides=strides(4096, 0, 128)), 1),
    (dict(page=4), 2), (dict(page=24), 2), (dict(d=96), 2), (dict(d=256), 2), (dict(width=1 << 27), 2),
    (dict(H=514, Hkv=2), 2), (dict(B=1 << 20, H=1024, Hkv=512), 2), (dict(B=1 << 12, width=1 << 26), 2),
    (dict(H=8192, Hkv=8192), 2),
])
def test_decode_paged_refuses_before_any_cuda_call(attn, kw, code):
    a = PAGED | kw
    rc = attn.lib().attn_decode_paged(a["q"], a["k"], a["v"], a["strides"], a["table"], a["lens"], a["o"], a["lse"],
                                      a["workspace"], a["ws_bytes"], a["B"], a["H"], a["Hkv"], a["T"], a["P"],
                                      a["page"], a["width"], a["window"], a["d"], a["scale"], None)
    assert rc == code


@pytest.mark.parametrize("kw,code", [
    (dict(q=0), 1), (dict(k=0), 1), (dict(table=0), 1), (dict(lens=0), 1), (dict(o=0), 1), (dict(lse=0), 1),
    (dict(workspace=0), 1), (dict(ws_bytes=0), 1), (dict(k=FAKE + 8), 1), (dict(B=0), 1), (dict(T=0), 1),
    (dict(H=0), 1), (dict(P=-1), 1), (dict(scale=-1.0), 1), (dict(strides=strides(9216, 572)), 1),
    (dict(strides=strides(8, 576)), 1), (dict(rank=128), 2), (dict(rank=576), 2), (dict(page=20), 2),
    (dict(H=1025), 2), (dict(H=128, T=9), 2),
])
def test_decode_latent_refuses_before_any_cuda_call(attn, kw, code):
    a = PAGED | dict(rank=512, H=16) | kw
    rc = attn.lib().attn_decode_latent(a["q"], a["k"], a["strides"], a["table"], a["lens"], a["o"], a["lse"],
                                       a["workspace"], a["ws_bytes"], a["B"], a["H"], a["T"], a["P"], a["page"],
                                       a["width"], a["rank"], a["scale"], None)
    assert rc == code


def test_workspace_sizes(attn):
    assert attn.decode_paged_workspace_bytes(4, 32, 8, 1, 512, 16, 128) > 0
    assert attn.decode_latent_workspace_bytes(4, 128, 1, 512, 64, 512) > 0
    for bad in [(0, 8, 2, 1, 8, 16, 128), (2, 8, 2, 1, 8, 12, 128), (2, 8, 3, 1, 8, 16, 128), (2, 8, 2, 1, 8, 16, 80)]:
        with pytest.raises(ValueError):
            attn.decode_paged_workspace_bytes(*bad)
    for bad in [(0, 16, 1, 8, 64, 512), (1, 16, 1, 8, 64, 320), (1, 2000, 1, 8, 64, 512)]:
        with pytest.raises(ValueError):
            attn.decode_latent_workspace_bytes(*bad)


def test_binding_checks_tensors(attn):
    q = torch.zeros(1, 2, 64, dtype=torch.bfloat16)
    pages = torch.zeros(4, 2, 8, 64, dtype=torch.bfloat16)
    table, lens = torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        attn.attn_decode_paged(q, pages, pages, table, lens)  # host tensors
    with pytest.raises(ValueError):
        attn.attn_decode_latent(q, pages[:, 0], table, lens, 1.0)


# ------------------------------------------------------------------ helpers

def make(B, Hkv, page, D, lens, seed, layout="hnd", extra=3, width=None, nan=True):
    """Pools of shuffled pages, the table and the lengths; unwritten slots hold
    NaN."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    counts = [-(-max(n, 0) // page) for n in lens]
    width = width or max(counts) + 1
    P = sum(counts) + extra
    ids = torch.randperm(P, generator=g, device="cuda").int()
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    pools = []
    written = torch.zeros((P, page), dtype=torch.bool, device="cuda")
    at = 0
    for b, n in enumerate(counts):
        table[b, :n] = ids[at:at + n]
        if n:
            slots = written[ids[at:at + n].long()].view(-1)
            slots[:lens[b]] = True
            written[ids[at:at + n].long()] = slots.view(n, page)
        at += n
    for _ in range(2):
        x = torch.randn((P, page, Hkv, D), generator=g, device="cuda").bfloat16()
        if nan:
            x[~written] = float("nan")
        x = x.transpose(1, 2)
        pools.append(x if layout == "nhd" else x.contiguous())
    return pools[0], pools[1], table, torch.tensor(lens, dtype=torch.int32, device="cuda"), g


def queries(g, B, H, T, D, std=1.0):
    return (torch.randn((B, H, T, D), generator=g, device="cuda") * std).bfloat16()


def run_paged(attn, q, k, v, table, lens, window=-1, scale=None, **kw):
    o, lse = attn.attn_decode_paged(q, k, v, table, lens, window, scale, **kw)
    assert attn.sync_status() == attn.ATTN_OK
    return o, lse


def paged_case(attn, Hkv, G, T, d, page, lens, window=-1, layout="hnd", seed=1, std=2.0):
    B = len(lens)
    k, v, table, ln, g = make(B, Hkv, page, d, lens, seed, layout)
    q = queries(g, B, Hkv * G, T, d, std)
    o, lse = run_paged(attn, q, k, v, table, ln, window)
    check(o, lse, attention(q, k, v, table, ln, 1 / math.sqrt(d), window))


def latent_case(attn, H, T, rank, page, lens, seed=1, std=1.0, scale=0.07):
    B = len(lens)
    c, _, table, ln, g = make(B, 1, page, rank + 64, lens, seed)
    q = queries(g, B, H, T, rank + 64, std)
    o, lse = attn.attn_decode_latent(q, c[:, 0], table, ln, scale)
    assert attn.sync_status() == attn.ATTN_OK
    check(o, lse, attention(q, c, c[..., :rank], table, ln, scale))


# -------------------------------------------------------------------- paged

LENS = [0, 1, 7, 8, 63, 64, 65, 127, 128, 129, 300, 1025]


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [8, 16, 32, 64, 128, 256])
@pytest.mark.parametrize("layout", ["hnd", "nhd"])
def test_paged_pages_and_lengths(gpu, d, page, layout):
    paged_case(gpu, 2, 4, 1, d, page, LENS, layout=layout, seed=page + d)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hkv,G,T", [(1, 1, 1), (3, 1, 2), (2, 3, 1), (1, 5, 3), (4, 8, 1), (1, 16, 1), (2, 4, 4),
                                     (1, 17, 1), (2, 8, 4), (1, 64, 1), (1, 32, 8)])
def test_paged_heads_and_tokens(gpu, d, Hkv, G, T):
    paged_case(gpu, Hkv, G, T, d, 16, [0, 1, 2, 5, 130, 517], seed=G * 7 + T)


@pytest.mark.gpu
@pytest.mark.parametrize("window", [0, 1, 15, 128, 200, 5000])
@pytest.mark.parametrize("T", [1, 4])
def test_paged_window(gpu, window, T):
    paged_case(gpu, 2, 4, T, 128, 32, [1, 3, 129, 700, 1500], window=window, seed=window + T)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hkv,G,T,lens", [(1, 1, 1, [50001]), (2, 8, 2, [20000, 3, 0, 9999]), (1, 16, 1, [131071]),
                                          (8, 4, 1, [4000 + 37 * i for i in range(24)])])
def test_paged_split_over_the_length(gpu, d, Hkv, G, T, lens):
    paged_case(gpu, Hkv, G, T, d, 64, lens, seed=len(lens))


@pytest.mark.gpu
def test_paged_many_short_sequences(gpu):
    paged_case(gpu, 2, 4, 1, 64, 16, [(i * 37) % 90 for i in range(700)], seed=5)


@pytest.mark.gpu
def test_paged_more_sequences_than_one_block_sums(gpu):
    paged_case(gpu, 1, 4, 1, 64, 16, [(i * 83) % 600 for i in range(1500)], seed=6)


@pytest.mark.gpu
def test_paged_large_logits(gpu):
    paged_case(gpu, 2, 4, 1, 128, 16, [5, 400, 3000], seed=9, std=12.0)


@pytest.mark.gpu
def test_paged_entries_that_are_no_page(gpu):
    """Their positions are left out, wherever they lie; a row of none is empty."""
    for page in (8, 32, 256):
        lens = [1000, 1000, 1000, 1000]
        k, v, table, ln, g = make(4, 2, page, 64, lens, 3)
        k, v = (torch.nan_to_num(x, nan=1.0) for x in (k, v))
        P = k.shape[0]
        table[0, 1] = -1
        table[0, -2] = P
        table[1, 0] = 2 ** 31 - 1
        table[1, 2:4] = -2 ** 31
        table[2, :] = -7
        q = queries(g, 4, 8, 1, 64)
        o, lse = run_paged(gpu, q, k, v, table, ln)
        check(o, lse, attention(q, k, v, table, ln, 1 / 8))
        assert torch.isneginf(lse[2]).all()


@pytest.mark.gpu
def test_paged_lengths_out_of_range(gpu):
    """Below 0: empty. Beyond the table: the table's capacity."""
    k, v, table, ln, g = make(3, 2, 16, 64, [64, 64, 64], 4, width=4)
    ln = torch.tensor([-5, 64, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    q = queries(g, 3, 4, 1, 64)
    o, lse = run_paged(gpu, q, k, v, table, ln)
    check(o, lse, attention(q, k, v, table, ln, 1 / 8))


@pytest.mark.gpu
def test_paged_infinite_and_nan_values_stay_in_their_place(gpu):
    """A NaN or infinite value that is attended reaches its own columns only."""
    k, v, table, ln, g = make(2, 1, 16, 128, [200, 77], 6)
    q = queries(g, 2, 4, 1, 128)
    ref = run_paged(gpu, q, k, v, table, ln)[0]
    page = int(table[0, 3])
    v[page, 0, 2, 5] = float("inf")
    v[page, 0, 3, 9] = float("nan")
    o, _ = run_paged(gpu, q, k, v, table, ln)
    rest = torch.ones(128, dtype=torch.bool, device="cuda")
    rest[[5, 9]] = False
    assert torch.equal(o[..., rest], ref[..., rest]) and torch.equal(o[1], ref[1])
    assert torch.isnan(o[0, :, 0, 9]).all() and not torch.isfinite(o[0, :, 0, 5]).any()


@pytest.mark.gpu
def test_paged_strided_pools(gpu):
    """Keys and values interleaved in one tensor, rows padded."""
    g = torch.Generator(device="cuda")
    g.manual_seed(8)
    both = torch.randn((40, 2, 3, 16, 72), generator=g, device="cuda").bfloat16()
    k, v = both[:, 0, :, :, :64], both[:, 1, :, :, :64]
    table = torch.randperm(40, generator=g, device="cuda").int().view(4, 10)
    ln = torch.tensor([160, 1, 33, 100], dtype=torch.int32, device="cuda")
    q = queries(g, 4, 6, 1, 64)
    o, lse = run_paged(gpu, q, k, v, table, ln)
    check(o, lse, attention(q, k, v, table, ln, 1 / 8))


@pytest.mark.gpu
def test_paged_matches_the_rolling_cache(gpu):
    """The same keys in a full rolling cache and in pages, by both kernels."""
    B, Hkv, G, W, d = 3, 2, 4, 256, 128
    k, v, table, ln, g = make(B, Hkv, 64, d, [W] * B, 12, nan=False)
    q = queries(g, B, Hkv * G, 1, d)
    o, lse = run_paged(gpu, q, k, v, table, ln)
    kc, vc = (x[table[:, :4].long()].permute(0, 2, 1, 3, 4).reshape(B, Hkv, W, d).contiguous() for x in (k, v))
    pos = torch.full((B,), W - 1, dtype=torch.int32, device="cuda")
    o2, lse2 = gpu.attn_decode(q[:, :, 0].contiguous(), kc, vc, pos)
    ref = attention(q, k, v, table, ln, 1 / math.sqrt(d))
    check(o, lse, ref)
    check(o2.unsqueeze(2), lse2.unsqueeze(2), ref)


@pytest.mark.gpu
def test_paged_repeats_bit_for_bit_with_any_workspace(gpu):
    k, v, table, ln, g = make(3, 2, 16, 128, [9000, 11, 4321], 13)
    q = queries(g, 3, 16, 1, 128)
    need = gpu.decode_paged_workspace_bytes(3, 16, 2, 1, table.shape[1], 16, 128)
    outs = []
    for fill in (0, 255, 127):
        ws = torch.full((need,), fill, dtype=torch.uint8, device="cuda")
        outs.append(run_paged(gpu, q, k, v, table, ln, workspace=ws))
    for o, lse in outs[1:]:
        assert torch.equal(o, outs[0][0]) and torch.equal(lse, outs[0][1])


@pytest.mark.gpu
def test_paged_one_token_shape_and_given_outputs(gpu):
    k, v, table, ln, g = make(2, 2, 16, 64, [50, 900], 14)
    q = queries(g, 2, 4, 1, 64)
    o4, lse4 = run_paged(gpu, q, k, v, table, ln)
    out = torch.empty((2, 4, 64), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((2, 4), device="cuda")
    o3, lse3 = run_paged(gpu, q[:, :, 0].contiguous(), k, v, table, ln, out=out, lse=lse)
    assert o3 is out and lse3 is lse and torch.equal(o3, o4[:, :, 0]) and torch.equal(lse3, lse4[:, :, 0])
    with pytest.raises(ValueError):
        gpu.attn_decode_paged(q, k, v, table, ln, out=out)
    with pytest.raises(ValueError):
        gpu.attn_decode_paged(q, k, v, table.long(), ln)
    with pytest.raises(ValueError):
        gpu.attn_decode_paged(q, k, v[:1], table, ln)
    with pytest.raises(ValueError):
        gpu.attn_decode_paged(q, k, v.transpose(1, 2).contiguous().transpose(1, 2), table, ln)


@pytest.mark.gpu
def test_on_a_given_stream(gpu):
    """What a call allocates belongs to the stream it was given."""
    k, v, table, ln, g = make(4, 2, 16, 128, [900, 5, 64, 3000], 22, nan=False)
    q = queries(g, 4, 8, 1, 128)
    want = run_paged(gpu, q, k, v, table, ln)
    c = torch.cat([k[:, 0], v[:, 0], k[:, 0], v[:, 0], k[:, 0, :, :64]], -1).contiguous()
    ql = queries(g, 4, 8, 1, 576)
    want_l = gpu.attn_decode_latent(ql, c, table, ln, 0.05)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        got = gpu.attn_decode_paged(q, k, v, table, ln, stream=s)
        got_l = gpu.attn_decode_latent(ql, c, table, ln, 0.05, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    for a, b in zip(got + got_l, want + want_l):
        assert torch.equal(a, b)
    assert gpu.sync_status() == gpu.ATTN_OK


@pytest.mark.gpu
def test_binding_refuses_what_does_not_fit(gpu):
    k, v, table, ln, g = make(2, 2, 16, 64, [50, 900], 23)
    q = queries(g, 2, 4, 1, 64)
    ws = torch.empty(16, dtype=torch.uint8, device="cuda")
    bad = [dict(q=q.float()), dict(q=q.cpu()), dict(q=q[..., :32]), dict(q=q[0, 0]), dict(table=table[0]),
           dict(table=table.cpu()), dict(lens=ln[:1]), dict(k=k.float()), dict(v=k[..., :32]), dict(k=k[:, 0]),
           dict(out=torch.empty_like(q, dtype=torch.float32)), dict(lse=torch.empty(2, 4, device="cuda"))]
    for kw in bad:
        a = dict(q=q, k=k, v=v, table=table, lens=ln, out=None, lse=None) | kw
        with pytest.raises(ValueError):
            gpu.attn_decode_paged(a["q"], a["k"], a["v"], a["table"], a["lens"], out=a["out"], lse=a["lse"])
    with pytest.raises(TypeError):
        gpu.attn_decode_paged(q, k, None, table, ln)
    with pytest.raises(gpu.AttnError):
        gpu.attn_decode_paged(q, k, v, table, ln, workspace=ws)
    with pytest.raises(gpu.AttnError):
        gpu.attn_decode_paged(q, k, v, table, ln, scale=-1.0)
    with pytest.raises(ValueError):
        gpu.attn_decode_latent(queries(g, 2, 4, 1, 64), k[:, 0], table, ln, 0.1)
    # a window of any size is a window
    o, lse = gpu.attn_decode_paged(q, k, v, table, ln, window=1 << 40)
    o2, lse2 = gpu.attn_decode_paged(q, k, v, table, ln)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.gpu
@pytest.mark.parametrize("form", ["paged", "latent"])
def test_captured_and_replayed_on_another_stream(gpu, form):
    """A captured step reads lengths and tables at replay; two graphs with
    workspaces of their own run at the same time."""
    lens = [700, 90, 2500]
    if form == "paged":
        k, v, table, ln, g = make(3, 2, 16, 128, lens, 15, nan=False)
        q = queries(g, 3, 8, 1, 128)
        call = lambda n, **kw: gpu.attn_decode_paged(q, k, v, table, n, **kw)
        truth = lambda n: attention(q, k, v, table, n, 1 / math.sqrt(128))
    else:
        k, _, table, ln, g = make(3, 1, 16, 576, lens, 15, nan=False)
        q = queries(g, 3, 16, 1, 576)
        call = lambda n, **kw: gpu.attn_decode_latent(q, k[:, 0], table, n, 0.05, **kw)
        truth = lambda n: attention(q, k, k[..., :512], table, n, 0.05)
    call(ln)
    torch.cuda.synchronize()
    graphs = []
    for i in range(2):
        n = ln.clone()
        s = torch.cuda.Stream()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            out = call(n)
        graphs.append((graph, n, out, s))
    for step in range(3):
        for i, (graph, n, out, s) in enumerate(graphs):
            n.copy_(ln - 37 * step * (i + 1))
        torch.cuda.synchronize()
        for graph, n, out, s in graphs:
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        assert gpu.sync_status() == gpu.ATTN_OK
        for graph, n, out, s in graphs:
            check(*out, truth(n))


@pytest.mark.gpu
@pytest.mark.parametrize("form", ["paged", "latent"])
@pytest.mark.parametrize("captured", [False, True])
def test_steps_follow_on_what_the_kernel_before_wrote(gpu, form, captured):
    """Lengths, tables, queries and cache rows written by kernels right before
    each call, ten steps without a synchronisation, one workspace for all."""
    B, Hkv, G, page, steps = 5, 2, 4, 16, 10
    d = 128 if form == "paged" else 576
    Hkv = Hkv if form == "paged" else 1
    start = [3, 700, 64, 15, 2000]
    k, v, table, ln, g = make(B, Hkv, page, d, [n + steps for n in start], 21, nan=False)
    new = [(torch.randn((steps, B, Hkv, 1, d), generator=g, device="cuda")).bfloat16() for _ in range(2)]
    q = queries(g, steps * B, Hkv * G, 1, d).view(steps, B, Hkv * G, 1, d)
    first = torch.tensor(start, dtype=torch.int32, device="cuda")
    cur, pos, tb, qq = torch.empty_like(ln), torch.empty_like(ln), torch.empty_like(table), torch.empty_like(q[0])
    if form == "paged":
        need = gpu.decode_paged_workspace_bytes(B, Hkv * G, Hkv, 1, table.shape[1], page, d)
    else:
        need = gpu.decode_latent_workspace_bytes(B, G, 1, table.shape[1], page, 512)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    outs = []

    def step(i):
        tb.copy_(table)
        qq.copy_(q[i])
        torch.add(first, i, out=pos)
        torch.add(first, i + 1, out=cur)
        if form == "paged":
            gpu.pages_append(new[0][i], new[1][i], k, v, tb, pos)
            outs.append(gpu.attn_decode_paged(qq, k, v, tb, cur, workspace=ws))
        else:
            gpu.pages_append(new[0][i], None, k[:, 0], None, tb, pos)
            outs.append(gpu.attn_decode_latent(qq, k[:, 0], tb, cur, 0.05, workspace=ws))
        tb.fill_(-1)
        cur.fill_(1)

    if captured:
        kept = k.clone(), v.clone()
        step(0)
        outs.clear()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for i in range(steps):
                step(i)
        k.copy_(kept[0])
        v.copy_(kept[1])
        graph.replay()
    else:
        for i in range(steps):
            step(i)
    torch.cuda.synchronize()
    assert gpu.sync_status() == gpu.ATTN_OK
    for i, (o, lse) in enumerate(outs):
        n = first + i + 1
        if form == "paged":
            check(o, lse, attention(q[i], k, v, table, n, 1 / math.sqrt(d)))
        else:
            check(o, lse, attention(q[i], k, k[..., :512], table, n, 0.05))


@pytest.mark.gpu
def test_paged_offsets_past_32_bits(gpu):
    """A pool of more than 2^32 elements, used at both ends."""
    P, Hkv, page, d = 34000, 8, 128, 128
    k = torch.empty((P, Hkv, page, d), dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    ids = torch.tensor([[P - 1, 0, 33000, 17], [3, P - 2, 20000, P - 3]], dtype=torch.int32, device="cuda")
    used = ids.flatten().long()
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    for x in (k, v):
        x[used] = torch.randn((8, Hkv, page, d), generator=g, device="cuda").bfloat16()
    ln = torch.tensor([500, 512], dtype=torch.int32, device="cuda")
    q = queries(g, 2, 16, 1, d)
    o, lse = run_paged(gpu, q, k, v, ids, ln)
    check(o, lse, attention(q, k[used], v[used], torch.arange(8, device="cuda").int().view(2, 4), ln, 1 / math.sqrt(d)))


@pytest.mark.gpu
def test_paged_large_pages_and_a_wide_table(gpu):
    """Pages of 2^20 tokens, a table of 2^30 positions, 1.3 million tokens."""
    page, width = 1 << 20, 1 << 10
    g = torch.Generator(device="cuda")
    g.manual_seed(31)
    k, v = (torch.randn((3, 1, page, 64), generator=g, device="cuda").bfloat16() for _ in range(2))
    table = torch.full((2, width), -1, dtype=torch.int32, device="cuda")
    table[0, :2] = torch.tensor([2, 0])
    table[1, 0] = 1
    ln = torch.tensor([page + 300001, 77], dtype=torch.int32, device="cuda")
    q = queries(g, 2, 4, 1, 64)
    for window in (-1, 1000000):
        o, lse = run_paged(gpu, q, k, v, table, ln, window)
        check(o, lse, attention(q, k, v, table[:, :2], ln, 1 / 8, window))


@pytest.mark.gpu
@pytest.mark.parametrize("form", ["paged", "latent"])
def test_padded_rows_and_the_same_sequence_twice(gpu, form):
    """Rows without a sequence, whatever their queries hold; rows that share a
    table row give the same bits where their queries are the same (each tile is
    a run of its own in a call of this size)."""
    d = 128 if form == "paged" else 576
    k, v, table, ln, g = make(3, 1, 16, d, [300, 17, 1000], 32)
    table = torch.cat([table[[0, 2, 2]], torch.full_like(table[:2], -1), table[1:2]]).contiguous()
    ln = torch.tensor([300, 1000, 1000, 0, 0, 17], dtype=torch.int32, device="cuda")
    q = queries(g, 6, 5, 1, d)
    q[2] = q[1]
    q[3:5] = float("nan")
    if form == "paged":
        o, lse = run_paged(gpu, q, k, v, table, ln)
        ref = attention(q.nan_to_num(), k, v, table, ln, 1 / math.sqrt(d))
    else:
        o, lse = gpu.attn_decode_latent(q, k[:, 0], table, ln, 0.05)
        assert gpu.sync_status() == gpu.ATTN_OK
        ref = attention(q.nan_to_num(), k, k[..., :512], table, ln, 0.05)
    check(o, lse, ref)
    assert torch.equal(o[1], o[2]) and torch.equal(lse[1], lse[2])


# ------------------------------------------------------------------- latent

@pytest.mark.gpu
@pytest.mark.parametrize("rank", [256, 512])
@pytest.mark.parametrize("page", [8, 16, 64, 128])
def test_latent_pages_and_lengths(gpu, rank, page):
    latent_case(gpu, 16, 1, rank, page, LENS, seed=page)


@pytest.mark.gpu
@pytest.mark.parametrize("rank", [256, 512])
@pytest.mark.parametrize("H,T", [(1, 1), (8, 1), (20, 1), (16, 2), (32, 3), (64, 1), (65, 1), (128, 1), (64, 4),
                                 (128, 8)])
def test_latent_heads_and_tokens(gpu, rank, H, T):
    latent_case(gpu, H, T, rank, 64, [0, 1, 3, 65, 700], seed=H + T)


@pytest.mark.gpu
@pytest.mark.parametrize("H,lens", [(16, [50001]), (128, [30000, 5]), (64, [3000 + 61 * i for i in range(20)]),
                                    (16, [(i * 37) % 90 for i in range(300)])])
def test_latent_split_over_the_length(gpu, H, lens):
    latent_case(gpu, H, 1, 512, 32, lens, seed=H)


@pytest.mark.gpu
def test_latent_large_logits(gpu):
    latent_case(gpu, 32, 1, 512, 64, [5, 400, 3000], seed=9, std=6.0, scale=0.2)


@pytest.mark.gpu
def test_latent_entries_that_are_no_page(gpu):
    for page in (8, 32, 128):
        c, _, table, ln, g = make(4, 1, page, 576, [1000] * 4, 3)
        c = torch.nan_to_num(c, nan=1.0)
        table[0, 1] = -1
        table[0, -2] = c.shape[0]
        table[1, 0] = 2 ** 31 - 1
        table[1, 2:4] = -2 ** 31
        table[2, :] = -7
        q = queries(g, 4, 24, 1, 576)
        o, lse = gpu.attn_decode_latent(q, c[:, 0], table, ln, 0.05)
        assert gpu.sync_status() == gpu.ATTN_OK
        check(o, lse, attention(q, c, c[..., :512], table, ln, 0.05))
        assert torch.isneginf(lse[2]).all()


@pytest.mark.gpu
def test_latent_strided_and_large_pool(gpu):
    """Padded rows, and offsets past 32 bits."""
    P, page, D = 60000, 128, 576
    pool = torch.empty((P, page, D + 8), dtype=torch.bfloat16, device="cuda")
    c = pool[..., :D]
    ids = torch.tensor([[P - 1, 0, 31000, 17], [3, P - 2, 58000, P - 3]], dtype=torch.int32, device="cuda")
    used = ids.flatten().long()
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    c[used] = torch.randn((8, page, D), generator=g, device="cuda").bfloat16()
    ln = torch.tensor([500, 512], dtype=torch.int32, device="cuda")
    q = queries(g, 2, 16, 1, D)
    o, lse = gpu.attn_decode_latent(q, c, ids, ln, 0.05)
    assert gpu.sync_status() == gpu.ATTN_OK
    cc = c[used].unsqueeze(1)
    check(o, lse, attention(q, cc, cc[..., :512], torch.arange(8, device="cuda").int().view(2, 4), ln, 0.05))


@pytest.mark.gpu
def test_latent_repeats_bit_for_bit_with_any_workspace(gpu):
    c, _, table, ln, g = make(3, 1, 16, 576, [9000, 11, 4321], 13)
    q = queries(g, 3, 128, 1, 576)
    need = gpu.decode_latent_workspace_bytes(3, 128, 1, table.shape[1], 16, 512)
    outs = []
    for fill in (0, 255, 127):
        ws = torch.full((need,), fill, dtype=torch.uint8, device="cuda")
        outs.append(gpu.attn_decode_latent(q, c[:, 0], table, ln, 0.05, workspace=ws))
    assert gpu.sync_status() == gpu.ATTN_OK
    for o, lse in outs[1:]:
        assert torch.equal(o, outs[0][0]) and torch.equal(lse, outs[0][1])
