"""The paged cache in other forms: keys and values in one allocation, shared pages, offsets past 32 bits, many
rows, a part of the device, a thread's first call, tables of the smallest and largest pages; with the tolerances of
tests/test_gpu_paged.py, or the bits of a plain call on the same values."""
import threading

import numpy as np
import pytest
import torch

from tests import paged64 as P
from tests.test_gpu_paged import DT, Attn, Cache, _f, _i32, _turns

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _free():
    yield
    torch.cuda.empty_cache()


def _moved(c, pool, at, stride):
    """The cache's pages at places `at` of flat pools, `stride` values apart."""
    size = c.page * c.Hkv * c.D
    for i in range(2):
        pool[i].view(-1)  # flat
        for p, n in enumerate(at):
            pool[i][n * stride:n * stride + size] = c.pools[i].tensor[p, :size]


def _attend(kda, a, pages, k, v, decode, **kw):
    c = a.c
    p = c.params(kda, causal=a.causal, window=a.window, q_row_stride=a.p.q_row_stride, **kw)
    need = (kda.kda_paged_attn_decode_workspace_bytes(p, c.N) if decode else kda.kda_paged_attn_workspace_bytes(p, c.N, a.rows))
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
    rest = (c.kv_lens, pages, a.q, k, v, a.out.tensor, a.lse.tensor, ws, need, c.status)
    a.out.tensor.fill_(7.0)
    a.lse.tensor.fill_(7.0)
    if decode:
        kda.check(kda.kda_paged_attn_decode(p, c.N, *rest))
    else:
        kda.check(kda.kda_paged_attn_varlen(p, c.cu, c.N, a.rows, *rest))
    torch.cuda.synchronize()


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("decode", [False, True])
@pytest.mark.parametrize("major", ["token", "head"])
def test_keys_and_values_in_one_allocation(cuda_lib, major, decode, io):
    c = Cache([1, 1, 1] if decode else [20, 3, 150], [40, 100, 200], D=64, page=32, io=io, major=major)
    a = Attn(c, cuda_lib, decode=decode).run()
    want = a.out.tensor.clone()
    size = c.page * c.Hkv * c.D
    both = torch.full((c.num_pages, 2, size), float("nan"), dtype=DT[io], device="cuda")
    both[:, 0], both[:, 1] = c.pools[0].tensor[:, :size], c.pools[1].tensor[:, :size]
    _attend(cuda_lib, a, c.pages, both[:, 0], both[:, 1], decode, cache_page_stride=2 * size)
    assert torch.equal(a.out.tensor, want)
    a.check()


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("decode", [False, True])
@pytest.mark.parametrize("D,page", [(128, 64), (256, 16)])
def test_pages_past_32_bits(cuda_lib, D, page, decode, io):
    """Pages 2^28 values apart: the last ones lie past 2^31 values, and past 2^32 bytes."""
    c = Cache([1, 1] if decode else [5, 70], [page * 3 + 5, page * 4], D=D, page=page, io=io)
    a = Attn(c, cuda_lib, decode=decode).run()
    want = a.out.tensor.clone()
    stride = 1 << 28
    assert c.num_pages * stride > 1 << 31
    pool = [torch.zeros(c.num_pages * stride, dtype=DT[io], device="cuda") for _ in range(2)]
    _moved(c, pool, range(c.num_pages), stride)
    _attend(cuda_lib, a, c.pages, *pool, decode, cache_page_stride=stride)
    assert torch.equal(a.out.tensor, want)
    # the append writes there too
    q = torch.randn(a.rows, c.Hq, D, device="cuda").to(DT[io])
    k, v = (torch.randn(a.rows, c.Hkv, D, device="cuda").to(DT[io]) for _ in range(2))
    p = c.params(cuda_lib, cache_page_stride=stride)
    args = (c.kv_lens, c.pages, None, q, k, v, torch.empty_like(q), *pool, c.status)
    if decode:
        cuda_lib.check(cuda_lib.kda_paged_append_decode(p, c.N, *args))
    else:
        cuda_lib.check(cuda_lib.kda_paged_append_varlen(p, c.cu, c.N, a.rows, *args))
    torch.cuda.synchronize()
    for s in range(c.N):
        tok = c.kv[s] - 1
        at = int(c.table[s, tok // page]) * stride + tok % page * c.Hkv * D
        row = int(c.cu[s + 1]) - 1
        assert torch.equal(pool[0][at:at + c.Hkv * D], k[row].flatten()) and torch.equal(pool[1][at:at + c.Hkv * D], v[row].flatten())
    # rows before a sequence's first token (70 rows of 64 tokens) are flagged by the append, not by the attention
    early = any(n > L for n, L in zip(c.lens, c.kv))
    assert int(c.status.item()) == (cuda_lib.KDA_DEV_BAD_SEQLENS if early else 0)


@pytest.mark.parametrize("decode", [False, True])
def test_rows_past_32_bits(cuda_lib, decode):
    """More than 2^31 values of q and out: rows that see one token each give its value."""
    kda = cuda_lib
    Hq, Hkv, D, T, page = 256, 16, 256, 32768 + 9, 16
    g = torch.Generator(device="cuda").manual_seed(1)
    q = torch.empty(T, Hq, D, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    v = torch.empty(40, page, Hkv, D, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    out = torch.empty_like(q)
    pages = (torch.arange(T, device="cuda") % 40).to(torch.int32)[:, None].contiguous()
    kv, cu = torch.ones(T, dtype=torch.int32, device="cuda"), torch.arange(T + 1, dtype=torch.int32, device="cuda")
    p = kda.PagedParams(Hq, Hkv, D, page, 40, 1)
    status = _i32([0])
    if decode:
        need = kda.kda_paged_attn_decode_workspace_bytes(p, T)
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        kda.check(kda.kda_paged_attn_decode(p, T, kv, pages, q, v, v, out, None, ws, need, status))
    else:
        need = kda.kda_paged_attn_workspace_bytes(p, T, T)
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        kda.check(kda.kda_paged_attn_varlen(p, cu, T, T, kv, pages, q, v, v, out, None, ws, need, status))
    torch.cuda.synchronize()
    for r in (0, 1, T // 2, T - 2, T - 1):
        wrong = (out[r].view(Hkv, Hq // Hkv, D) != v[r % 40, 0][:, None]).sum().item()
        assert wrong == 0, (r, wrong)
    assert int(status.item()) == 0


def test_rope_of_rows_past_32_bits(cuda_lib):
    kda = cuda_lib
    H, D, rows = 128, 512, 32768 + 77
    x = torch.empty(rows, H, D, dtype=torch.bfloat16, device="cuda").normal_()
    pos = torch.arange(rows, dtype=torch.int32, device="cuda")
    p = kda.RopeParams(H, D, 256, _turns(kda, 256))
    y, small = torch.empty_like(x), torch.empty_like(x[:50])
    kda.check(kda.kda_rope(p, rows, pos, x, y))
    tail = pos[-50:].clone()
    kda.check(kda.kda_rope(p, 50, tail, x[-50:].contiguous(), small))
    torch.cuda.synchronize()
    assert torch.equal(y[-50:], small)


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_sequences_that_share_pages(cuda_lib, io):
    """A common prompt's pages in every table."""
    c = Cache([1] * 5, [200 + 30 * i for i in range(5)], D=128, page=64, io=io)
    shared = 3  # pages
    for s in range(1, 5):
        c.table[s, :shared] = c.table[0, :shared]
        for i in range(2):
            c.tok[s][i][:, :shared * 64] = c.tok[0][i][:, :shared * 64]
    c.pages = _i32(c.table)
    Attn(c, cuda_lib, decode=True).run().check()
    Attn(c, cuda_lib).run().check()


@pytest.mark.parametrize("decode", [False, True])
def test_on_a_part_of_the_device(cuda_lib, decode):
    from tests.green import stream_on_part

    c = Cache([1] * 9 if decode else [300, 1, 900], [3000 + 40 * i for i in range(9 if decode else 3)], D=128, page=64)
    a = Attn(c, cuda_lib, decode=decode).run()
    want = a.out.tensor.clone()
    a.out.tensor.fill_(7.0)
    torch.cuda.synchronize()
    with stream_on_part(32) as (cu, stream, sms):
        assert sms < torch.cuda.get_device_properties(0).multi_processor_count
        a.call(stream.value)
        assert cu.cuStreamSynchronize(stream) == 0
    assert torch.equal(a.out.tensor, want) and int(c.status.item()) == 0


@pytest.mark.parametrize("decode", [False, True])
def test_from_another_thread(cuda_lib, decode):
    """A thread whose first CUDA call this is: the same bits."""
    c = Cache([1, 1] if decode else [40, 7], [500, 70], D=128)
    a = Attn(c, cuda_lib, decode=decode).run()
    want = a.out.tensor.clone()
    a.out.tensor.fill_(7.0)
    stream = torch.cuda.current_stream().cuda_stream
    torch.cuda.synchronize()
    t = threading.Thread(target=lambda: a.call(stream))
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert torch.equal(a.out.tensor, want)


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_a_layer_captured_and_replayed(cuda_lib, io):
    """Append and attention of next tokens in one graph, lengths advanced between replays, against plain calls."""
    kda = cuda_lib
    B, Hkv, G, D, page, W = 3, 2, 4, 64, 16, 8
    Hq = Hkv * G
    k0, v0 = (torch.randn(B * W + 1, page, Hkv, D, device="cuda").to(DT[io]) for _ in range(2))
    table = _i32(np.random.default_rng(0).permutation(B * W).reshape(B, W))
    p = kda.PagedParams(Hq, Hkv, D, page, B * W + 1, W, io_dtype=kda.KDA_DTYPE_BF16 if io == "bf16" else kda.KDA_DTYPE_F32, scale=D ** -0.5,
                        rotary_dim=D, rope_turns=_turns(kda, D))
    need = kda.kda_paged_attn_decode_workspace_bytes(p, B)

    class State:
        def __init__(self):
            self.k, self.v, self.kv = k0.clone(), v0.clone(), _i32([5, 60, 31])
            self.x = torch.zeros(B, Hq + 2 * Hkv, D, dtype=DT[io], device="cuda")
            self.qr, self.out = (torch.zeros(B, Hq, D, dtype=DT[io], device="cuda") for _ in range(2))
            self.ws, self.status = torch.empty(need, dtype=torch.uint8, device="cuda"), _i32([0])

        def step(self, stream=None):
            q, k, v = self.x[:, :Hq].contiguous(), self.x[:, Hq:Hq + Hkv].contiguous(), self.x[:, Hq + Hkv:].contiguous()
            self.kv += 1
            kda.check(kda.kda_paged_append_decode(p, B, self.kv, table, None, q, k, v, self.qr, self.k, self.v, self.status, stream))
            kda.check(kda.kda_paged_attn_decode(p, B, self.kv, table, self.qr, self.k, self.v, self.out, None, self.ws, need, self.status, stream))

    plain, held = State(), State()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    State().step()  # the calls' one-time set-up
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        held.step(side)
    for i in range(6):
        x = torch.randn(B, Hq + 2 * Hkv, D, device="cuda").to(DT[io])
        plain.x.copy_(x)
        held.x.copy_(x)
        plain.step()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(plain.out, held.out) and torch.equal(plain.k, held.k) and torch.equal(plain.v, held.v), i
    assert int(held.status.item()) == int(plain.status.item()) == 0 and held.kv.tolist() == [11, 66, 37]


def test_random_calls(cuda_lib):
    """Lengths, heads, widths, pages, windows and holes at random, all kinds of calls."""
    r = np.random.default_rng(77)
    for i in range(60):
        D, io = int(r.choice([32, 64, 128, 256])), str(r.choice(["bf16", "bf16", "f32"]))
        N, decode = int(r.integers(1, 7)), bool(r.integers(0, 2))
        lens = [1] * N if decode else [int(x) for x in r.integers(0, 60, N)]
        kv = [int(max(-1, n + r.integers(-3, 260))) for n in lens]
        page = int(r.choice([16, 32, 64, 128, 256]))
        c = Cache(lens, kv, Hkv=int(r.integers(1, 4)), G=int(r.choice([1, 2, 3, 5, 8, 11, 17])), D=D, page=page, io=io,
                  major=str(r.choice(["token", "head"])), seed=i)
        status = 0
        causal = bool(r.integers(0, 4))
        window = int(r.choice([0, 0, r.integers(1, 100)])) if causal else 0
        if not window:
            for s in range(N):
                if lens[s] and kv[s] > page and r.integers(0, 3) == 0:
                    c.hide(s, 0)
                    # the first page is looked at if a row sees it
                    status = cuda_lib.KDA_DEV_BAD_PAGE
        Attn(c, cuda_lib, decode=decode, causal=causal, window=window, seed=i).run().check(status=status)


def test_rope_matches_the_append(cuda_lib):
    """The rotation by itself and on the way into the cache: the same bits."""
    kda = cuda_lib
    c = Cache([7, 30], [50, 31], D=128, page=16)
    T = 37
    x = torch.randn(T, c.Hq + 2 * c.Hkv, 128, device="cuda").to(torch.bfloat16)
    q, k, v = (x[:, a:b].contiguous() for a, b in ((0, c.Hq), (c.Hq, c.Hq + c.Hkv), (c.Hq + c.Hkv, c.Hq + 2 * c.Hkv)))
    turns = _turns(kda, 128)
    pos = _i32(list(range(43, 50)) + list(range(1, 31)))
    y = torch.empty(T, c.Hq + c.Hkv, 128, dtype=torch.bfloat16, device="cuda")
    kda.check(kda.kda_rope(kda.RopeParams(c.Hq + c.Hkv, 128, 128, turns, x_row_stride=x.shape[1] * 128), T, pos, x, y))
    qr = torch.empty_like(q)
    kda.check(kda.kda_paged_append_varlen(c.params(kda, rotary_dim=128, rope_turns=turns), c.cu, 2, T, c.kv_lens, c.pages, None, q, k, v, qr,
                                          *[g.tensor for g in c.pools], c.status))
    torch.cuda.synchronize()
    assert torch.equal(qr, y[:, :c.Hq])
    row = 0
    for s, (n, L) in enumerate(zip(c.lens, c.kv)):
        for t in range(L - n, L):
            assert torch.equal(c.views[0][int(c.table[s, t // 16]), t % 16], y[row, c.Hq:])
            row += 1
    assert np.allclose(P.radians(128)[0], 1.0) and _f(v).size


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("decode", [False, True])
def test_nan_in_a_query_or_in_many_keys_is_not_lost(cuda_lib, decode, io):
    # a short sequence is one unit within a stretch, a long one is cut into parts, some of which meet nothing but NaN
    n = [1, 1, 1] if decode else [30, 5, 20]
    c = Cache(n, [40, 9000, 60], D=64, page=64, io=io)
    a = Attn(c, cuda_lib, decode=decode).run()
    clean, lse = a.out.tensor.clone(), a.lse.tensor.clone()
    ends = np.cumsum(n)
    q = a.q.clone()
    rows = [0, int(ends[0])]  # of the short and of the long sequence
    for r in rows:
        a.q[r, 2 * 64:3 * 64] = float("nan")  # head 2
    a.run()
    hit = torch.zeros_like(clean, dtype=torch.bool)
    for r in rows:
        hit[r, 2] = True
    hit[c.T:] = False
    same = ~hit
    assert torch.isnan(a.out.tensor[hit]).all() and torch.isnan(a.lse.tensor[hit[..., 0]]).all()
    assert torch.equal(a.out.tensor[same], clean[same]) and torch.equal(a.lse.tensor[same[..., 0]], lse[same[..., 0]])
    a.q.copy_(q)
    pg = torch.from_numpy(c.table[1][10:70].astype(np.int64)).cuda()
    c.views[0][pg, :, 1] = float("nan")  # keys of tokens 640 to 4479, key head 1
    a.run()
    hit[:] = False
    hit[int(ends[0]):int(ends[1]), c.G:2 * c.G] = True
    same = ~hit
    assert torch.isnan(a.out.tensor[hit]).all() and torch.isnan(a.lse.tensor[hit[..., 0]]).all()
    assert torch.equal(a.out.tensor[same], clean[same]) and torch.equal(a.lse.tensor[same[..., 0]], lse[same[..., 0]])


@pytest.mark.parametrize("D", [64, 256])
def test_rows_without_tokens_between_rows_with_some(cuda_lib, D):
    """Far more units than CTAs, so that each takes rows that see nothing and rows that see something in turn: sequences
    without tokens, and with more rows than tokens, among ordinary ones."""
    r = np.random.default_rng(D)
    lens = [int(r.integers(1, 4)) for _ in range(2400)]
    kv = [0 if i % 2 else int(n + r.integers(0, 30)) for i, n in enumerate(lens)]
    lens += [200, 5] * 6
    kv += [9, 40] * 6
    for io in ("f32", "bf16"):
        Attn(Cache(lens, kv, Hkv=1, G=3, D=D, io=io, seed=D), cuda_lib).run().check()


@pytest.mark.parametrize("decode,io,D,G", [(False, "bf16", 64, 4), (False, "bf16", 128, 4), (False, "bf16", 128, 3), (False, "bf16", 256, 2),
                                           (True, "bf16", 128, 4), (True, "bf16", 256, 12), (True, "f32", 64, 3)])
def test_waits_that_run_out(cuda_lib, decode, io, D, G):
    """A CTA that loads nothing (made by the host: those who wait for its tiles give up after 2^16 polls): the status says so, a row of which any part
    is missing keeps what it held, every other one has its bits; and the next call is as ever."""
    kda = cuda_lib
    lens = [1] * 5 if decode else [300, 40, 500, 7, 1]
    c = Cache(lens, [6000, 100, 2500, 7, 20000], Hkv=2, G=G, D=D, page=64, io=io)
    a = Attn(c, kda, decode=decode).run()
    want, lse = a.out.tensor.clone(), a.lse.tensor.clone()
    kept_rows = 0
    for cta in (0, 70, 151):
        a.out.tensor.fill_(7.0)
        a.lse.tensor.fill_(7.0)
        a.ws.tensor.fill_(0xFF)
        kda.check(kda.kda_debug_paged_attn_stalled(a.p, None if decode else c.cu, c.N, a.rows, c.kv_lens, c.pages, a.q, *[g.tensor for g in c.pools],
                                                   a.out.tensor, a.lse.tensor, a.ws.tensor, a.need, c.status, 1 << 16, 1 << 16, cta))
        torch.cuda.synchronize()
        assert int(c.status.item()) == kda.KDA_DEV_TIMEOUT
        c.status.zero_()
        same, kept = (a.out.tensor == want).all(-1), (a.out.tensor == 7.0).all(-1)
        assert (same | kept)[:c.T].all() and kept[:c.T].any() and same[:c.T].any() and kept[c.T:].all()
        assert torch.equal(a.lse.tensor, torch.where(kept, 7.0, lse))
        kept_rows += int(kept[:c.T].sum())
        a.run()
        assert torch.equal(a.out.tensor, want) and torch.equal(a.lse.tensor, lse) and int(c.status.item()) == 0
    assert kept_rows < 2 * c.T * c.Hq  # a CTA has a part in a few units only
    for g in (a.out, a.lse, a.ws, *c.pools):
        assert g.intact()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("G,lens,kv", [(4, [20] * 8, [100] * 8), (3, [20] * 8, [100] * 8), (16, [20] * 40, [1500] * 40)], ids=["whole tokens", "cut tokens", "long units"])
def test_no_wait_runs_out_in_silence(cuda_lib, D, G, lens, kv):
    """The waits that last a unit (for its rows' place, for its outputs) limited to one poll, nothing else wrong: whatever did not come is flagged."""
    kda = cuda_lib
    c = Cache(lens, kv, Hkv=2, G=G, D=D, page=64)
    a = Attn(c, kda).run()
    want, lse = a.out.tensor.clone(), a.lse.tensor.clone()
    for _ in range(5):
        a.out.tensor.fill_(7.0)
        kda.check(kda.kda_debug_paged_attn_stalled(a.p, c.cu, c.N, a.rows, c.kv_lens, c.pages, a.q, *[g.tensor for g in c.pools], a.out.tensor,
                                                   a.lse.tensor, a.ws.tensor, a.need, c.status, 1 << 14, 1, -1))
        torch.cuda.synchronize()
        # outputs leave 128 channels at a time
        same, kept = ((a.out.tensor == x).view(-1, c.Hq, max(D // 128, 1), min(D, 128)).all(-1)[:c.T] for x in (want, 7.0))
        assert (same | kept).all()
        assert int(c.status.item()) in ((kda.KDA_DEV_TIMEOUT,) if kept.any() else (0, kda.KDA_DEV_TIMEOUT))
        c.status.zero_()
    a.run()
    assert torch.equal(a.out.tensor, want) and torch.equal(a.lse.tensor, lse) and int(c.status.item()) == 0


def test_waits_over_a_long_unit_are_as_long(cuda_lib):
    """Units of 2^24 tokens (two pages again and again), one a CTA, 170 ms: the waits that last a unit go by its length.  Their limit here, 2^15 polls (3.7 us each
    where nothing ends them, 121 ms), is shorter than the unit; by its length it is three times that."""
    kda = cuda_lib
    Hkv, G, D, page, T, pages = 152, 2, 64, 1024, 128, 1 << 14
    g = torch.Generator(device="cuda").manual_seed(5)
    k, v = (torch.randn(2, Hkv, page, D, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    q = torch.randn(T, Hkv * G, D, generator=g, device="cuda").to(torch.bfloat16)
    table = (torch.arange(pages, device="cuda") % 2).to(torch.int32)[None].contiguous()
    p = kda.PagedParams(Hkv * G, Hkv, D, page, 2, pages, causal=False, scale=D ** -0.5, cache_page_stride=Hkv * page * D, cache_token_stride=D,
                        cache_head_stride=page * D)
    outs = []
    for tokens in (2 * page, pages * page):
        need = kda.kda_paged_attn_workspace_bytes(p, 1, T)
        ws, out, status = torch.empty(need, dtype=torch.uint8, device="cuda"), torch.full_like(q, 7.0), _i32([0])
        start, end = torch.cuda.Event(True), torch.cuda.Event(True)
        start.record()
        kda.check(kda.kda_debug_paged_attn_stalled(p, _i32([0, T]), 1, T, _i32([tokens]), table, q, k, v, out, None, ws, need, status, 1 << 22, 1 << 15, -1))
        end.record()
        torch.cuda.synchronize()
        assert int(status.item()) == 0, (tokens, start.elapsed_time(end))
        outs.append(out.double())
    # the same tokens 2^13 times each: the same means, but for 2^17 sums of tiles in fp32 (2^-24 of each, 2^-23 where a product's sum is cut off),
    # over values of mean size below 1 (of either sign; the weights are positive), and the outputs' rounding
    assert (outs[0] - outs[1]).abs().max() <= 2 * 2.0 ** (17 - 23) + 2.0 ** -7


@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("G", [4, 3])
def test_units_of_two_tiles_and_of_one_in_turn(cuda_lib, D, G):
    """Thousands of short units, with the second tile of rows in use or not from one to the next."""
    r = np.random.default_rng(G)
    n = 256 // G
    lens = [int(x) for _ in range(300) for x in (r.integers(n // 2 + 1, n + 1), r.integers(1, n // 2 + 1))]
    kv = [int(x + r.integers(0, 300)) for x in lens]
    c = Cache(lens, kv, Hkv=8, G=G, D=D, page=64)
    a = Attn(c, cuda_lib).run()
    want = a.out.tensor.clone()
    for _ in range(20):
        a.run()
        assert torch.equal(a.out.tensor, want) and int(c.status.item()) == 0
    a.check(rows=sorted(r.choice(c.T, 40, replace=False).tolist()))


@pytest.mark.parametrize("D", [32, 64, 128, 256])
def test_short_units_through_the_ring(cuda_lib, D):
    """Thousands of units of one key tile, all of whole tokens: outputs of neighbouring units close behind one another."""
    c = Cache([64] * 500, [64 + i % 40 for i in range(500)], Hkv=8, G=4, D=D, page=64)
    a = Attn(c, cuda_lib).run()
    want = a.out.tensor.clone()
    for _ in range(20):
        a.run()
        assert torch.equal(a.out.tensor, want) and int(c.status.item()) == 0
    a.check(rows=[0, 63, 64, 16000, 31937, 31999])


@pytest.mark.parametrize("decode", [False, True])
@pytest.mark.parametrize("G", [2, 32, 64, 128])
@pytest.mark.parametrize("D", [32, 64, 128, 256])
def test_groups_whose_tokens_fill_a_tile(cuda_lib, D, G, decode):
    """Powers of two: rows and outputs in boxes of 128 / G tokens (single tokens of more than 16 heads as chunks of one)."""
    lens, kv = ([1] * 5, [300, 1, 64, 700, 129]) if decode else ([1, 9, 128 // G, 3], [200, 9, 90, 500])
    c = Cache(lens, kv, Hkv=2, G=G, D=D, page=32)
    Attn(c, cuda_lib, decode=decode, q_extra=32).run().check()


@pytest.mark.parametrize("io,G,decode", [("bf16", 4, True), ("bf16", 20, True), ("bf16", 32, True), ("f32", 3, True), ("f32", 9, True), ("bf16", 4, False), ("f32", 4, False)])
@pytest.mark.parametrize("D,page", [(64, 16), (128, 128), (256, 64)])
def test_values_before_the_window_have_no_effect(cuda_lib, D, page, io, G, decode):
    """NaN and infinities in values that no row of the call sees, in the page and the tile in which the window begins."""
    c = Cache([1, 1, 1] if decode else [3, 1, 2], [300, 1000, 130], Hkv=2, G=G, D=D, page=page, io=io)
    window = 77
    a = Attn(c, cuda_lib, decode=decode, window=window).run()
    want, lse = a.out.tensor.clone(), a.lse.tensor.clone()
    for s, (n, L) in enumerate(zip(c.lens, c.kv)):
        for t in range(0, L - n - window + 1):
            c.views[1][int(c.table[s, t // page]), t % page] = float("nan") if t % 3 else float("inf")
    a.run()
    assert torch.equal(a.out.tensor, want) and torch.equal(a.lse.tensor, lse)
    a.check()


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("window", [(1 << 31) - 1, (1 << 31) - 100])
def test_the_widest_window_and_rows_before_the_first_token(cuda_lib, window, io):
    """Positions below zero less the window pass 32 bits."""
    c = Cache([300, 5, 40], [20, 2, 90], io=io)
    Attn(c, cuda_lib, window=window).run().check()
    Attn(Cache([1] * 3, [0, 1, 90], io=io), cuda_lib, decode=True, window=window).run().check()
