"""Rotary positions, the append to a paged cache and the attention over it on the GPU, against their
definitions in 64 bits.

Tolerances.  Rotation: half a step of the output type, and of |x1| + |x2| the fp32 arithmetic: the angle (2^-25 of
half a turn is 2^-23.3), sine and cosine (2 ulp, 2^-22), amplitude, two products and a sum (2^-24 each): 2^-21 together;
angles of position p in 64 bits are off by p 2^-51 themselves.
Attention: half a step of the output type.  A score is a sum of D fp32 products, off by (D + 8) 2^-24 of the sum of
their magnitudes (the 8: scale, base-2 factor, difference from the maximum, exponential); a weight is off by that
factor, once in the sum of values and once in the weights' sum; bf16 rows of a chunk round each weight to bf16 (half a step,
2^-8), single tokens of up to 16 heads a key head to two bf16 (2^-16); those of more heads run as chunks do.  Both are relative to the weighted mean of |v|.
"""
import numpy as np
import pytest
import torch

from linear_attention_serving_kda_gb300.runtime import Guarded
from tests import paged64 as P

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF_STEP = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
LAYOUT = {"half": 0, "pairs": 1}
SCALING = {"none": 0, "linear": 1, "base": 2, "ramp": 3, "smooth": 4}


def _code(kda, io):
    return kda.KDA_DTYPE_BF16 if io == "bf16" else kda.KDA_DTYPE_F32


def _f(x):
    return x.double().cpu().numpy()


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def _within(got, want, tol, what):
    d = np.abs(got - want)
    bad = ~(d <= tol)
    assert not bad.any(), (what, int(bad.sum()), bad.size, float(np.nanmax(np.where(bad, d / np.maximum(tol, 1e-300), 0))))


def _turns(kda, rd, kind="none", **kw):
    t = torch.empty(rd // 2, dtype=torch.int64)
    kda.check(kda.kda_rope_turns(kda.RopeScaling(kind=SCALING[kind], **kw), rd, None, t))
    return t.cuda()


# ---------------------------------------------------------------- rotation

def _rope(kda, rows, H, D, rd, layout, io, far, transpose=False, amplitude=1.0, in_place=False, extra=0, kind="none", **kw):
    r = np.random.default_rng(rows + H + D + rd)
    stride = H * D + extra
    x = torch.from_numpy(r.standard_normal((rows, stride))).to(DT[io]).cuda()
    pos = r.integers(0, far, rows)
    if rows > 2:
        pos[1] = -1
        pos[2] = 0
    g = Guarded((rows, H * D), DT[io], "cuda")
    g.tensor.fill_(7.0)
    x0, y = _f(x)[:, :H * D].reshape(rows, H, D), x if in_place else g.tensor
    p = kda.RopeParams(num_heads=H, head_dim=D, rotary_dim=rd, rope_turns=_turns(kda, rd, kind, **kw), rope_layout=LAYOUT[layout],
                       rope_amplitude=amplitude, transpose=transpose, io_dtype=_code(kda, io), x_row_stride=stride,
                       y_row_stride=stride if in_place else 0)
    kda.check(kda.kda_rope(p, rows, _i32(pos), x, y))
    torch.cuda.synchronize()
    f = P.radians(rd, kind, **kw)
    want, size = P.rope(x0, pos, f, layout, np.float32(amplitude).astype(np.float64), transpose)
    got = _f(y)[:, :H * D].reshape(rows, H, D)
    on = pos >= 0
    tol = HALF_STEP[io] * np.abs(want) + (2.0 ** -21 + far * 2.0 ** -51) * size
    _within(got[on], want[on], tol[on], "rope")
    assert (got[~on] == (x0[~on] if in_place else 7.0)).all() and g.intact()


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("layout", ["half", "pairs"])
@pytest.mark.parametrize("D,rd", [(16, 2), (32, 32), (48, 24), (64, 16), (80, 80), (128, 128), (128, 126), (256, 64), (512, 512)])
def test_rope_widths(cuda_lib, D, rd, layout, io):
    _rope(cuda_lib, 37, 3, D, rd, layout, io, 5000)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("kw", [dict(transpose=True, amplitude=0.7), dict(in_place=True), dict(in_place=True, extra=64, transpose=True),
                                dict(extra=128)], ids=str)
@pytest.mark.parametrize("layout", ["half", "pairs"])
def test_rope_forms(cuda_lib, kw, layout, io):
    _rope(cuda_lib, 50, 5, 64, 32, layout, io, 100, **kw)


@pytest.mark.parametrize("rows,H", [(1, 1), (1, 200), (700, 40), (5000, 1), (3, 1000)])
def test_rope_counts(cuda_lib, rows, H):
    _rope(cuda_lib, rows, H, 32, 32, "half", "bf16", 9000)


@pytest.mark.parametrize("kind", sorted(SCALING))
def test_rope_scalings_and_far_positions(cuda_lib, kind):
    _rope(cuda_lib, 300, 2, 128, 128, "half", "f32", 1 << 22, kind=kind, factor=8.0, fast=32.0 if kind == "ramp" else 4.0)


def test_rope_last_position(cuda_lib):
    _rope(cuda_lib, 300, 2, 64, 64, "pairs", "f32", (1 << 31) - 1)


def test_rope_transpose_undoes_and_is_the_gradient(cuda_lib):
    """<g, R x> = <R^T g, x>, and differences of <g, R x> along each channel are R^T g."""
    kda = cuda_lib
    r = np.random.default_rng(3)
    x, g = (torch.from_numpy(r.standard_normal((4, 2, 32))).float().cuda() for _ in range(2))
    pos, turns = _i32([0, 5, 77, 4000]), _turns(kda, 16)

    def turn(v, transpose):
        y = torch.empty_like(v)
        kda.check(kda.kda_rope(kda.RopeParams(2, 32, 16, turns, rope_amplitude=1.25, transpose=transpose, io_dtype=kda.KDA_DTYPE_F32),
                               4, pos, v, y))
        return y

    grad, eps = turn(g, True), 2.0 ** -6
    for c in range(32):
        d = torch.zeros_like(x)
        d[..., c] = eps
        slope = ((turn(x + d, False).double() - turn(x - d, False).double()) * g.double()).sum(-1) / (2 * eps)
        # x + d, x - d and both rotations are off by at most 2^-20 of values below 8; over 2 eps = 2^-5, 32 of them
        assert (slope - grad[..., c].double()).abs().max() < 2.0 ** -7


def test_rope_graph_and_other_stream(cuda_lib):
    kda = cuda_lib
    x = torch.randn(40, 256, device="cuda")
    y, z = torch.empty_like(x), torch.empty_like(x)
    pos = torch.arange(40, dtype=torch.int32, device="cuda")
    p = kda.RopeParams(2, 128, 128, _turns(kda, 128), io_dtype=kda.KDA_DTYPE_F32)
    kda.check(kda.kda_rope(p, 40, pos, x, z))
    g, st = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=st):
        kda.check(kda.kda_rope(p, 40, pos, x, y, st))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, z)
    x.neg_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, -z)


# ---------------------------------------------------------------- a cache with its sequences

class Cache:
    """Sequences with `kv` tokens, the last `lens` of them new, in pages of any order; what no token lies in is NaN."""

    def __init__(self, lens, kv, Hkv=2, G=2, D=64, page=16, io="bf16", major="token", seed=0, width=None, fill=True, gap=0,
                 spread=1.0):
        r = self.r = np.random.default_rng(seed)
        self.lens, self.kv, self.Hkv, self.G, self.D, self.page, self.io, self.major = list(lens), list(kv), Hkv, G, D, page, io, major
        self.N, self.T, self.Hq = len(lens), int(sum(lens)), Hkv * G
        need = [(max(n, 0) + page - 1) // page for n in kv]
        self.width = width or max(need + [1]) + 1
        self.num_pages = sum(min(n, self.width) for n in need) + 2
        order = r.permutation(self.num_pages)
        self.table = np.full((self.N, self.width), 1 << 30)  # entries past the tokens: never read
        at = 0
        for s, n in enumerate(need):
            n = min(n, self.width)
            self.table[s, :n] = order[at:at + n]
            at += n
        inner = (page, Hkv, D) if major == "token" else (Hkv, page, D)
        self.stride = dict(cache_token_stride=Hkv * D, cache_head_stride=D) if major == "token" else dict(cache_token_stride=D, cache_head_stride=page * D)
        self.stride["cache_page_stride"] = page * Hkv * D + gap
        self.pools = []
        for _ in range(2):
            g = Guarded((self.num_pages, page * Hkv * D + gap), DT[io], "cuda")
            g.tensor.fill_(float("nan"))
            self.pools.append(g)
        self.inner = inner
        self.views = [g.tensor[:, :page * Hkv * D].view(self.num_pages, *inner) for g in self.pools]
        self.tok = [[None, None] for _ in kv]
        if fill:
            for s, n in enumerate(kv):
                n = min(n, self.width * page)
                if n <= 0:
                    continue
                pg, pl = torch.from_numpy(self.table[s][np.arange(n) // page]).cuda(), torch.arange(n, device="cuda") % page
                for i in range(2):
                    x = torch.from_numpy(r.standard_normal((n, Hkv, D)) * (spread if i == 0 else 1.0)).to(DT[io]).cuda()
                    if major == "token":
                        self.views[i][pg, pl] = x
                    else:
                        self.views[i][pg, :, pl] = x
                    self.tok[s][i] = _f(x).transpose(1, 0, 2)
        self.pages, self.kv_lens = _i32(self.table), _i32(self.kv)
        self.cu = _i32(np.concatenate([[0], np.cumsum(lens)]))
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.hidden = {}

    def params(self, kda, **kw):
        return kda.PagedParams(**{**dict(num_heads_q=self.Hq, num_heads_kv=self.Hkv, head_dim=self.D, page_size=self.page,
                                         num_pages=self.num_pages, pages_per_seq=self.width, io_dtype=_code(kda, self.io),
                                         scale=self.D ** -0.5), **self.stride, **kw})

    def hide(self, s, i, value=-1):
        """Page i of sequence s: no page at all."""
        self.table[s, i] = value
        self.pages[s, i] = value
        self.hidden.setdefault(s, []).append(i)

    def tokens(self, s):
        n = self.kv[s]
        visible = np.ones(n, bool)
        for i in self.hidden.get(s, []):
            visible[i * self.page:(i + 1) * self.page] = False
        z = np.zeros((self.Hkv, n, self.D))
        return [z if t is None else t for t in self.tok[s]] + [visible]


class Attn:
    def __init__(self, c, kda, decode=False, causal=True, window=0, q_extra=0, lse=True, seed=1, q_std=1.0):
        r = np.random.default_rng(seed)
        self.c, self.kda, self.decode, self.causal, self.window = c, kda, decode, causal, window
        rows = max(c.T, 1) + 2  # two rows behind the last sequence
        self.rows = c.N if decode else c.T + 2
        self.q = torch.from_numpy(r.standard_normal((rows, c.Hq * c.D + q_extra)) * q_std).to(DT[c.io]).cuda()
        self.q[c.T:] = float("nan")
        self.out, self.lse = Guarded((rows, c.Hq, c.D), DT[c.io], "cuda"), Guarded((rows, c.Hq), torch.float32, "cuda")
        self.with_lse = lse
        self.p = c.params(kda, causal=causal, window=window, q_row_stride=c.Hq * c.D + q_extra)
        need = kda.kda_paged_attn_decode_workspace_bytes(self.p, c.N) if decode else kda.kda_paged_attn_workspace_bytes(self.p, c.N, self.rows)
        self.ws, self.need = Guarded((max(need, 16),), torch.uint8, "cuda"), need
        self.ws.tensor.fill_(0xFF)  # NaN and -1: no need of any contents

    def call(self, stream=None):
        c, kda = self.c, self.kda
        rest = (c.kv_lens, c.pages, self.q, *[g.tensor for g in c.pools], self.out.tensor, self.lse.tensor if self.with_lse else None,
                self.ws.tensor, self.need, c.status, stream)
        if self.decode:
            kda.check(kda.kda_paged_attn_decode(self.p, c.N, *rest))
        else:
            kda.check(kda.kda_paged_attn_varlen(self.p, c.cu, c.N, self.rows, *rest))

    def run(self):
        self.out.tensor.fill_(7.0)
        self.lse.tensor.fill_(7.0)
        self.call()
        torch.cuda.synchronize()
        return self

    def check(self, status=0, lens=None, kv=None, rows=None):
        """rows: only these are compared (long calls)."""
        c = self.c
        q = _f(self.q)[:c.T, :c.Hq * c.D].reshape(c.T, c.Hq, c.D)
        if rows is None:
            out, lse, mean, size = P.attn(c.lens, kv or c.kv, q, c.tokens, c.D ** -0.5, self.causal, self.window)
        else:
            out, lse, mean, size = self.some(q, rows)
        got, glse = _f(self.out.tensor), _f(self.lse.tensor)
        assert (got[c.T:] == 7.0).all() and (glse[c.T:] == 7.0).all(), "rows behind the last sequence"
        off = (c.D + 8) * 2.0 ** -24 * size
        weight = 0.0 if c.io == "f32" else 2.0 ** -16 if self.decode and c.G <= 16 else 2.0 ** -8
        tol = HALF_STEP[c.io] * np.abs(out) + (2 * off[..., None] + weight) * mean * 1.01
        m = ~np.isnan(out)
        full = slice(None) if rows is None else rows
        _within(got[:c.T][full][m], out[m], tol[m], "out")
        if rows is None:
            assert (got[:c.T][~m] == 7.0).all()
        m = ~np.isnan(lse)
        if self.with_lse:
            g = glse[:c.T][full][m]
            inf = np.isinf(lse[m])
            assert (np.isneginf(g) == inf).all()
            _within(g[~inf], lse[m][~inf], (off + 2.0 ** -21 + 2.0 ** -22 * np.abs(lse))[m][~inf], "lse")
            if rows is None:
                assert (glse[:c.T][~m] == 7.0).all()
        else:
            assert (glse == 7.0).all()
        assert int(c.status.item()) == status
        for g in (self.out, self.lse, self.ws, *c.pools):
            assert g.intact()

    def some(self, q, rows):
        c, parts = self.c, []
        ends = np.cumsum(c.lens)
        for r in rows:
            s = int(np.searchsorted(ends, r, side="right"))
            p = c.kv[s] - (ends[s] - r)  # its token
            L = p + 1 if self.causal else c.kv[s]
            k, v, vis = c.tokens(s)
            parts.append(P.attn([1], [L], q[r:r + 1], lambda _: (k[:, :L], v[:, :L], vis[:L]), c.D ** -0.5, self.causal, self.window))
        return [np.concatenate([x[i] for x in parts]) for i in range(4)]


# ---------------------------------------------------------------- append

def _append(kda, c, rd, layout="half", decode=False, with_q=True, positions=False, fused=True, in_place=False, amplitude=1.0):
    r = np.random.default_rng(11)
    rows, D, Hq, Hkv = max(c.T, 1) + 1, c.D, c.Hq, c.Hkv
    width = (Hq + 2 * Hkv) * D
    qkv = torch.from_numpy(r.standard_normal((rows, width))).to(DT[c.io]).cuda()
    q, k, v = qkv[:, :Hq * D], qkv[:, Hq * D:(Hq + Hkv) * D], qkv[:, (Hq + Hkv) * D:]
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    st = width if fused else 0
    x = [_f(t).reshape(rows, -1, D) for t in (q, k, v)]
    qo = Guarded((rows, Hq, D), DT[c.io], "cuda")
    qo.tensor.fill_(7.0)
    turn = dict(rotary_dim=rd, rope_layout=LAYOUT[layout], rope_turns=_turns(kda, rd), rope_amplitude=amplitude) if rd else {}
    p = c.params(kda, q_in_row_stride=st, k_row_stride=st, v_row_stride=st, q_row_stride=st if in_place else 0, **turn)
    pos_h = r.integers(0, 5000, rows) if positions else None
    pos = _i32(pos_h) if positions else None
    before = [_f(t) for t in c.views]
    args = (c.kv_lens, c.pages, pos, q if with_q else None, k, v, (q if in_place else qo.tensor) if with_q else None,
            *[g.tensor for g in c.pools], c.status)
    if decode:
        kda.check(kda.kda_paged_append_decode(p, c.N, *args))
    else:
        kda.check(kda.kda_paged_append_varlen(p, c.cu, c.N, rows, *args))
    torch.cuda.synchronize()
    got_q = _f(q).reshape(rows, Hq, D) if in_place else _f(qo.tensor)
    got = [_f(t) for t in c.views]
    if c.major == "head":
        before, got = [b.transpose(0, 2, 1, 3) for b in before], [b.transpose(0, 2, 1, 3) for b in got]
    want, tol, want_q, tol_q = before, [np.zeros_like(b) for b in before], (x[0].copy() if in_place else np.full(x[0].shape, 7.0)), np.zeros(x[0].shape)
    f = P.radians(rd) if rd else np.zeros(0)
    t = 0
    for s, (n, L) in enumerate(zip(c.lens, c.kv)):
        for i in range(n):
            row, tok = t + i, L - n + i
            if L < 0 or L > c.width * c.page or tok < 0 or not 0 <= c.table[s, tok // c.page] < c.num_pages:
                continue
            at = np.array([tok if pos_h is None else pos_h[row]])
            pg, pl = c.table[s, tok // c.page], tok % c.page
            y, size = P.rope(x[1][row:row + 1], at, f, layout, amplitude)
            want[0][pg, pl], tol[0][pg, pl] = y[0], HALF_STEP[c.io] * np.abs(y[0]) + 2.0 ** -21 * size[0]
            want[1][pg, pl] = x[2][row]
            if with_q:
                y, size = P.rope(x[0][row:row + 1], at, f, layout, amplitude)
                want_q[row], tol_q[row] = y[0], HALF_STEP[c.io] * np.abs(y[0]) + 2.0 ** -21 * size[0]
        t += n
    for w, g, e in zip(want, got, tol):
        assert np.array_equal(np.isnan(w), np.isnan(g))
        m = ~np.isnan(w)
        _within(g[m], w[m], e[m], "cache")
    if with_q:
        _within(got_q, want_q, tol_q, "q")
    assert qo.intact() and all(g.intact() for g in c.pools)
    return int(c.status.item())


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("major", ["token", "head"])
@pytest.mark.parametrize("D,rd,layout,page", [(32, 32, "half", 16), (64, 16, "pairs", 32), (128, 128, "half", 64), (256, 64, "half", 16),
                                              (64, 0, "half", 128), (32, 10, "pairs", 1024)])
def test_append(cuda_lib, D, rd, layout, page, major, io):
    c = Cache([1, 40, 0, 17, 3], [1, 55, 9, 200, 30], D=D, page=page, io=io, major=major, gap=32)
    assert _append(cuda_lib, c, rd, layout) == 0


@pytest.mark.parametrize("kw", [dict(with_q=False), dict(positions=True), dict(fused=False), dict(in_place=True),
                                dict(in_place=True, fused=False, amplitude=1.5)], ids=str)
@pytest.mark.parametrize("decode", [False, True])
def test_append_forms(cuda_lib, decode, kw):
    lens = [1] * 9 if decode else [5, 1, 30]
    c = Cache(lens, [n + 13 * i for i, n in enumerate(lens)], Hkv=3, G=5)
    assert _append(cuda_lib, c, 64, decode=decode, **kw) == 0


def test_append_many_sequences_and_heads(cuda_lib):
    lens = [1 + i % 3 for i in range(700)]
    assert _append(cuda_lib, Cache(lens, [n + i % 90 for i, n in enumerate(lens)], Hkv=1, G=1, D=32), 32) == 0
    assert _append(cuda_lib, Cache([3, 9], [3, 40], Hkv=16, G=20, D=128), 128) == 0


def test_append_faults(cuda_lib):
    kda = cuda_lib
    # padding; more rows than tokens; a missing page, one past the pool; more tokens than the table names
    c = Cache([4, 6, 20, 20, 5], [-1, 4, 40, 40, 16 * 4 + 1], width=4)
    c.table[2, 1], c.table[3, 2] = -3, c.num_pages
    c.pages = _i32(c.table)
    assert _append(kda, c, 64) == kda.KDA_DEV_BAD_SEQLENS | kda.KDA_DEV_BAD_PAGE
    c = Cache([4, 6], [-1, 30])
    assert _append(kda, c, 64) == 0
    c = Cache([1, 1, 1], [0, -1, 5])
    assert _append(kda, c, 64, decode=True) == kda.KDA_DEV_BAD_SEQLENS


# ---------------------------------------------------------------- attention of chunks

@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("D", [32, 64, 128, 256])
@pytest.mark.parametrize("lens,kv", [([1], [1]), ([3, 1, 0, 7], [3, 90, 20, 7]), ([130], [130]), ([65, 200], [300, 201]), ([1, 2], [700, 513])], ids=str)
def test_attn_lengths(cuda_lib, lens, kv, D, io):
    c = Cache(lens, kv, D=D, io=io, seed=sum(lens) + D)
    Attn(c, cuda_lib).run().check()


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256, 512, 1024])
@pytest.mark.parametrize("major", ["token", "head"])
def test_attn_pages(cuda_lib, page, major, io):
    c = Cache([20, 33], [page + 20, 2 * page + 40], D=128, page=page, io=io, major=major, gap=64)
    Attn(c, cuda_lib, q_extra=64).run().check()


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("Hkv,G", [(1, 1), (1, 16), (3, 3), (2, 5), (8, 1), (4, 7), (1, 130)])
def test_attn_head_groups(cuda_lib, Hkv, G, io):
    c = Cache([9, 50], [30, 170], Hkv=Hkv, G=G, io=io)
    Attn(c, cuda_lib, lse=G % 2 == 0).run().check()


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 256])
@pytest.mark.parametrize("window", [1, 2, 17, 100, 128, 1 << 30])
def test_attn_window(cuda_lib, window, D, io):
    c = Cache([150, 40], [400, 290], D=D, io=io)
    Attn(c, cuda_lib, window=window).run().check()


@pytest.mark.parametrize("page", [16, 256])
@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_attn_pages_before_the_window_may_be_gone(cuda_lib, io, page):
    c = Cache([20, 3], [900, 1300], io=io, page=page)
    for s, n in enumerate(c.lens):
        gone = max(c.kv[s] - n - 100 + 1, 0) // page
        c.pages[s, :gone] = -1
    Attn(c, cuda_lib, window=100).run().check()


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_attn_without_causal(cuda_lib, io):
    c = Cache([7, 300, 2], [40, 310, 260], io=io)
    Attn(c, cuda_lib, causal=False).run().check()


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_attn_rows_that_see_nothing(cuda_lib, io):
    for lens, kv in (([5, 300, 3], [2, 20, 0]), ([4, 4], [0, 0]), ([600], [1])):
        Attn(Cache(lens, kv, io=io), cuda_lib).run().check()
    Attn(Cache([4, 4], [0, 7], io=io), cuda_lib, causal=False).run().check()


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("D,page", [(64, 16), (128, 64), (256, 16), (128, 256)])
def test_attn_pages_that_are_not_there(cuda_lib, io, D, page):
    c = Cache([30, 5, 40], [10 * page, 7 * page, 20 * page], io=io, D=D, page=page)
    c.hide(0, 0)
    c.hide(0, 9, c.num_pages)
    for i in range(7):
        c.hide(1, i)
    c.hide(2, 3, -(1 << 31))
    c.hide(2, 4, (1 << 31) - 1)
    Attn(c, cuda_lib).run().check(status=cuda_lib.KDA_DEV_BAD_PAGE)


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_attn_skipped_and_bad_sequences(cuda_lib, io):
    kda = cuda_lib
    c = Cache([20, 5, 40], [-1, 20, 100], io=io)
    Attn(c, kda).run().check()
    c = Cache([20, 5, 40], [30, 16 * 8 + 1, 100], io=io, width=8)
    Attn(c, kda).run().check(status=kda.KDA_DEV_BAD_SEQLENS, kv=[30, -1, 100])
    c = Cache([20, 5, 40], [30, 20, 100], io=io)
    c.cu[1] = 70  # past its successor and the rows: two sequences are bad
    Attn(c, kda).run().check(status=kda.KDA_DEV_BAD_SEQLENS, kv=[-1, -1, 100])


def test_attn_many_sequences(cuda_lib):
    r = np.random.default_rng(2)
    for N in (17, 33, 400):
        lens = r.integers(0, 4, N)
        c = Cache(lens, lens + r.integers(0, 60, N), Hkv=1, G=3, D=32)
        Attn(c, cuda_lib).run().check()


@pytest.mark.parametrize("io,D", [("bf16", 128), ("bf16", 64), ("bf16", 256), ("f32", 64)])
def test_attn_few_rows_over_many_tokens(cuda_lib, io, D):
    """Cut along the tokens, and joined."""
    c = Cache([2, 8], [20000, 7777], Hkv=1, G=4, D=D, io=io, page=64)
    Attn(c, cuda_lib).run().check()
    Attn(c, cuda_lib, window=3333).run().check()


@pytest.mark.parametrize("io,D", [("bf16", 128), ("bf16", 64), ("bf16", 256), ("f32", 128)])
def test_attn_long_chunk(cuda_lib, io, D):
    c = Cache([1500, 2300], [4000, 2300], Hkv=2, G=4, D=D, io=io, page=64, major="head")
    rows = sorted(np.random.default_rng(0).choice(3800, 60, replace=False).tolist() + [0, 1499, 1500, 3799])
    Attn(c, cuda_lib).run().check(rows=rows)
    Attn(c, cuda_lib, window=777).run().check(rows=rows)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("std", [8.0, 40.0])
def test_attn_large_scores(cuda_lib, io, std):
    """Maxima that keep growing along the tokens, by far more than a power of two's range."""
    c = Cache([40, 200], [500, 900], D=128, io=io, spread=std)
    for s in range(2):
        n = c.kv[s]
        ramp = torch.linspace(0.1, 1.5, n, device="cuda")
        pg, pl = torch.from_numpy(c.table[s][np.arange(n) // c.page]).cuda(), torch.arange(n, device="cuda") % c.page
        k = (c.views[0][pg, pl].float() * ramp[:, None, None]).to(DT[io])
        c.views[0][pg, pl] = k
        c.tok[s][0] = _f(k).transpose(1, 0, 2)
    Attn(c, cuda_lib).run().check()


def test_attn_nan_stays_in_its_sequence_and_head(cuda_lib):
    for io in ("bf16", "f32"):
        c = Cache([40, 40], [90, 90], io=io)
        a = Attn(c, cuda_lib).run()
        clean = a.out.tensor.clone()
        pg = int(c.table[0, 0])
        c.views[0][pg, 3, 1] = float("nan")  # a key of sequence 0, key head 1, seen by all its rows
        a.run()
        assert torch.isnan(a.out.tensor[:40, 2:]).all()
        assert torch.equal(a.out.tensor[:40, :2], clean[:40, :2]) and torch.equal(a.out.tensor[40:80], clean[40:80])


def test_attn_same_bits_again_and_in_a_graph(cuda_lib):
    c = Cache([3, 500, 2], [9000, 800, 4000], D=128, page=64)
    a = Attn(c, cuda_lib).run()
    first = a.out.tensor.clone()
    for _ in range(3):
        assert torch.equal(a.run().out.tensor, first)
    g, st = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=st):
        a.call(st)
    a.out.tensor.fill_(7.0)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(a.out.tensor, first)
    c.kv[:] = [8000, 700, -1]  # read at each replay
    c.kv_lens.copy_(_i32(c.kv))
    a.out.tensor.fill_(7.0)
    a.lse.tensor.fill_(7.0)
    g.replay()
    torch.cuda.synchronize()
    for s in range(2):
        c.tok[s] = [x[:, :c.kv[s]] for x in c.tok[s]]
    a.check(rows=list(range(3)) + [3, 100, 400, 502])
    assert (a.out.tensor[503:505] == 7.0).all()


def test_attn_two_calls_at_once(cuda_lib):
    cs = [Cache([300, 2], [900, 9000], D=128, seed=i) for i in range(2)]
    calls = [Attn(c, cuda_lib, seed=i) for i, c in enumerate(cs)]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    for _ in range(5):
        for a, st in zip(calls, streams):
            a.call(st)
    torch.cuda.synchronize()
    for a in calls:
        got = a.out.tensor[:302].clone()
        assert torch.equal(a.run().out.tensor[:302], got)


# ---------------------------------------------------------------- attention of single tokens

@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("D", [32, 64, 128, 256])
@pytest.mark.parametrize("kv", [[1], [5, 0, 64, 65], [300, -1, 1, 16], [1000]], ids=str)
def test_token_lengths(cuda_lib, kv, D, io):
    Attn(Cache([1] * len(kv), kv, D=D, io=io), cuda_lib, decode=True).run().check()


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("page", [16, 64, 256, 1024])
@pytest.mark.parametrize("major", ["token", "head"])
def test_token_pages(cuda_lib, page, major, io):
    c = Cache([1] * 3, [page, 3 * page + 5, 40], D=128, page=page, io=io, major=major, gap=64)
    Attn(c, cuda_lib, decode=True, q_extra=64).run().check()


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("Hkv,G", [(1, 1), (8, 1), (2, 3), (1, 8), (2, 16), (1, 17), (2, 40), (1, 130)])
def test_token_head_groups(cuda_lib, Hkv, G, io):
    c = Cache([1] * 5, [200, 3, 77, 130, 1], Hkv=Hkv, G=G, io=io)
    Attn(c, cuda_lib, decode=True, lse=G % 2 == 0).run().check()


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("D", [32, 64, 128, 256])
@pytest.mark.parametrize("G", [8, 9, 16])
def test_token_every_head_of_a_unit(cuda_lib, G, D, io):
    c = Cache([1] * 4, [200, 3, 500, 130], Hkv=2, G=G, D=D, io=io)
    Attn(c, cuda_lib, decode=True).run().check()


@pytest.mark.parametrize("io,D", [("bf16", 128), ("bf16", 256), ("bf16", 32), ("f32", 64)])
@pytest.mark.parametrize("window", [1, 15, 100, 1000])
def test_token_window(cuda_lib, window, io, D):
    c = Cache([1] * 4, [50, 3000, 1001, 1], io=io, D=D)
    for s, L in enumerate(c.kv):
        c.pages[s, :max(L - window, 0) // c.page] = -1  # gone
    Attn(c, cuda_lib, decode=True, window=window).run().check()


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_token_pages_that_are_not_there(cuda_lib, io):
    c = Cache([1] * 3, [300, 100, 5000], io=io, D=128)
    c.hide(0, 3)
    for i in range(7):
        c.hide(1, i, c.num_pages + i)
    c.hide(2, 200, -(1 << 31))
    Attn(c, cuda_lib, decode=True).run().check(status=cuda_lib.KDA_DEV_BAD_PAGE)
    c = Cache([1] * 3, [30, 16 * 8 + 1, 100], io=io, width=8)
    Attn(c, cuda_lib, decode=True).run().check(status=cuda_lib.KDA_DEV_BAD_SEQLENS, kv=[30, -1, 100])


@pytest.mark.parametrize("io,D,Hkv", [("bf16", 128, 1), ("bf16", 256, 2), ("bf16", 64, 3), ("f32", 128, 1)])
def test_token_long_and_short(cuda_lib, io, D, Hkv):
    c = Cache([1] * 6, [30000, 1, 900, 17000, 64, 12345], Hkv=Hkv, G=4, D=D, io=io, page=64)
    Attn(c, cuda_lib, decode=True).run().check()


@pytest.mark.parametrize("N", [1000, 5000])
def test_token_many_sequences(cuda_lib, N):
    kv = np.random.default_rng(N).integers(-1, 70, N)
    Attn(Cache([1] * N, kv, Hkv=1, G=2, D=32), cuda_lib, decode=True).run().check()


@pytest.mark.parametrize("D", [32, 64, 128, 256])
def test_token_every_row_of_a_long_batch(cuda_lib, D):
    """Rings of tiles that wrap many times, at every width: each batch position against the same sequence by itself."""
    c = Cache([1] * 40, [700 + 211 * i for i in range(40)], Hkv=2, G=3, D=D, page=32)
    a = Attn(c, cuda_lib, decode=True).run()
    first = a.out.tensor.clone()
    for _ in range(20):
        assert torch.equal(a.run().out.tensor, first)
    a.check()


def test_token_large_scores(cuda_lib):
    for io in ("bf16", "f32"):
        Attn(Cache([1] * 3, [700, 1500, 40], D=128, io=io, spread=30.0), cuda_lib, decode=True).run().check()


def test_token_same_bits_again_and_in_a_graph(cuda_lib):
    c = Cache([1] * 4, [9000, 30, 4000, 1], D=128, page=64)
    a = Attn(c, cuda_lib, decode=True).run()
    first = a.out.tensor.clone()
    g, st = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=st):
        a.call(st)
    for _ in range(3):
        a.out.tensor.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(a.out.tensor, first)


def test_token_is_a_chunk_of_one(cuda_lib):
    """The same rows through both entry points."""
    c = Cache([1] * 5, [500, 3, 64, 2000, 1], D=128)
    one, many = Attn(c, cuda_lib, decode=True).run(), Attn(c, cuda_lib).run()
    d = (one.out.tensor[:5].double() - many.out.tensor[:5].double()).abs()
    assert (d <= 2.0 ** -6 * (1 + many.out.tensor[:5].double().abs())).all()
    one.check()
    many.check()


# ---------------------------------------------------------------- together

@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_prompt_fork_and_next_tokens(cuda_lib, io):
    """Two prompts in two pieces, a copy of one's pages for a second continuation, then a token of each:
    rotated, appended, attended, as a serving loop calls them."""
    kda = cuda_lib
    r = np.random.default_rng(9)
    Hkv, G, D, page, rd, W = 2, 3, 64, 16, 32, 8
    Hq, pages_all = Hkv * G, 40
    k_cache, v_cache = (torch.full((pages_all, page, Hkv, D), float("nan"), dtype=DT[io], device="cuda") for _ in range(2))
    order = r.permutation(pages_all)
    table = np.stack([order[:W], order[W:2 * W], order[2 * W:3 * W]])
    turns, f = _turns(kda, rd), P.radians(rd)
    status = _i32([0])
    base = dict(num_heads_q=Hq, num_heads_kv=Hkv, head_dim=D, page_size=page, num_pages=pages_all, pages_per_seq=W,
                io_dtype=_code(kda, io), scale=D ** -0.5, rotary_dim=rd, rope_turns=turns)
    width = (Hq + 2 * Hkv) * D
    p_in = kda.PagedParams(**base, q_in_row_stride=width, k_row_stride=width, v_row_stride=width)
    p = kda.PagedParams(**base)
    keys, values = [[], [], []], [[], [], []]

    def step(lens, kv, tab, who, decode=False):
        T, N = sum(lens), len(lens)
        qkv = torch.from_numpy(r.standard_normal((T, width))).to(DT[io]).cuda()
        q, k, v = qkv[:, :Hq * D], qkv[:, Hq * D:(Hq + Hkv) * D], qkv[:, (Hq + Hkv) * D:]
        qr, out = torch.empty(T, Hq, D, dtype=DT[io], device="cuda"), torch.empty(T, Hq, D, dtype=DT[io], device="cuda")
        cu, kvl, tb = _i32(np.concatenate([[0], np.cumsum(lens)])), _i32(kv), _i32(tab)
        if decode:
            kda.check(kda.kda_paged_append_decode(p_in, N, kvl, tb, None, q, k, v, qr, k_cache, v_cache, status))
            need = kda.kda_paged_attn_decode_workspace_bytes(p, N)
            ws = torch.empty(need, dtype=torch.uint8, device="cuda")
            kda.check(kda.kda_paged_attn_decode(p, N, kvl, tb, qr, k_cache, v_cache, out, None, ws, need, status))
        else:
            kda.check(kda.kda_paged_append_varlen(p_in, cu, N, T, kvl, tb, None, q, k, v, qr, k_cache, v_cache, status))
            need = kda.kda_paged_attn_workspace_bytes(p, N, T)
            ws = torch.empty(need, dtype=torch.uint8, device="cuda")
            kda.check(kda.kda_paged_attn_varlen(p, cu, N, T, kvl, tb, qr, k_cache, v_cache, out, None, ws, need, status))
        torch.cuda.synchronize()
        want, t = [], 0
        for s, n, L in zip(who, lens, kv):
            x = _f(qkv[t:t + n]).reshape(n, -1, D)
            pos = np.arange(L - n, L)
            # what the cache holds is rounded: a reference row of it is taken from there, after it was checked
            kk, size = P.rope(x[:, Hq:Hq + Hkv], pos, f)
            held = _f(k_cache)[table[s][pos // page], pos % page]
            _within(held, kk, HALF_STEP[io] * np.abs(kk) + 2.0 ** -21 * size, "key")
            keys[s].append(held)
            values[s].append(x[:, Hq + Hkv:])
            K, V = np.concatenate(keys[s]).transpose(1, 0, 2), np.concatenate(values[s]).transpose(1, 0, 2)
            want.append(P.attn([n], [L], _f(qr[t:t + n]), lambda _: (K, V, np.ones(L, bool)), D ** -0.5))
            t += n
        w, _, mean, size = [np.concatenate(z) for z in zip(*want)]
        weight = 0.0 if io == "f32" else 2.0 ** -16 if decode else 2.0 ** -8
        _within(_f(out), w, HALF_STEP[io] * np.abs(w) + (2 * (D + 8) * 2.0 ** -24 * size[..., None] + weight) * mean * 1.01, "out")

    step([37, 20], [37, 20], table[:2], [0, 1])
    step([5, 30], [42, 50], table[:2], [0, 1])
    # sequence 1 goes on twice: its pages copied to those of sequence 2 (a page is a slot of the pools)
    used = 4
    size = page * Hkv * D * k_cache.element_size()
    for pool in (k_cache, v_cache):
        kda.check(kda.kda_slots_copy(kda.SlotPool(pool, 1, pages_all, size, pages_all * size), used, _i32(table[1][:used]), _i32(table[2][:used]), status))
    keys[2], values[2] = list(keys[1]), list(values[1])
    for i in range(3):
        step([1, 1, 1], [43 + i, 51 + i, 51 + i], table, [0, 1, 2], decode=True)
    assert int(status.item()) == 0
