"""The gated delta rule with one decay per head on the GPU, against its
definition in 64 bits.

Tolerances (2-norm, relative), from the roundings on the way:
  - fp32 results.  An operand split into two fp16 values is off by 2^-22 of
    the largest value of its 16-term tile column at most, a gate's exponential by
    2 ulp plus its argument's rounding (about 2^-22 for |G| up to 4), an fp32
    accumulation of n terms by about sqrt(n) 2^-24.  A handful of these in a row: STATE = 2^-18.
  - bf16 outputs: half a step is 2^-8 of the value, and the high fp16 parts
    (2^-11 of the operands) of S, U and P in front of it: OUT = 2^-8 + 2^-10.
  - fp32 rows and the single-token form run in fp32 throughout: 2^-20.
"""
import math

import numpy as np
import pytest
import torch

from linear_attention_serving_kda_gb300.runtime import Guarded
from tests import plain64 as P

pytestmark = pytest.mark.gpu

STATE, OUT, FP32 = 2.0 ** -18, 2.0 ** -8 + 2.0 ** -10, 2.0 ** -20
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


class Case:
    """Rows of q|k|v side by side, guarded outputs and states on the GPU, and the 64-bit arrays of the same values."""

    def __init__(self, lens, Hk=2, Hv=4, dk=128, dv=128, io="bf16", out="bf16", seed=0, slots=None, num_slots=None,
                 l2=True, scale=None, dense=False, gate=0.0, dt=None, beta=0.0, spread=1.0):
        r = np.random.default_rng(seed)
        self.lens, self.T, self.N = list(lens), int(sum(lens)), len(lens)
        self.Hk, self.Hv, self.dk, self.dv, self.io, self.out_t, self.l2 = Hk, Hv, dk, dv, io, out, l2
        self.scale = dk ** -0.5 if scale is None else scale
        T = max(self.T, 1)
        x = r.standard_normal((T, 2 * Hk * dk + Hv * dv))
        x = x / (1 + np.exp(-x)) * spread
        self.rows = torch.from_numpy(x).to(DT[io]).cuda()
        if not l2:  # unit keys, as a caller without the option passes them
            kq = self.rows[:, :2 * Hk * dk].float().reshape(T, 2 * Hk, dk)
            self.rows[:, :2 * Hk * dk] = (kq / kq.norm(dim=-1, keepdim=True)).reshape(T, -1).to(DT[io])
        w = [Hk * dk, Hk * dk, Hv * dv]
        parts = self.rows.split(w, 1)
        self.stride = 0 if dense else self.rows.shape[1]
        self.q, self.k, self.v = (p.contiguous() for p in parts) if dense else parts
        self.a = torch.from_numpy(r.standard_normal((T, Hv)) + gate).to(DT[io]).cuda()
        self.b = torch.from_numpy(r.standard_normal((T, Hv)) + beta).to(DT[io]).cuda()
        self.A_log = torch.from_numpy(np.log(r.uniform(1, 16, Hv))).float().cuda()
        step = np.exp(r.uniform(math.log(1e-3), math.log(1e-1), Hv))
        self.dt_bias = torch.from_numpy(np.log(np.expm1(step)) if dt is None else np.full(Hv, dt)).float().cuda()
        self.slots_h = list(range(self.N)) if slots is None else list(slots)
        self.slots = None if slots is None else torch.tensor(slots, dtype=torch.int32, device="cuda")
        self.num_slots = num_slots or max(self.N, 1)
        self.state0 = torch.from_numpy(r.standard_normal((self.num_slots, Hv, dk, dv)) * 0.1).float().cuda()
        self.g_state = Guarded(self.state0.shape, torch.float32, "cuda")
        self.g_out = Guarded((T, Hv, dv), DT[out], "cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
        self.reset()

    def reset(self):
        self.g_state.tensor.copy_(self.state0)
        self.g_out.tensor.fill_(7.0)

    def params(self, kda):
        code = {"bf16": kda.KDA_DTYPE_BF16, "f32": kda.KDA_DTYPE_F32}
        return kda.GdnParams(num_heads_k=self.Hk, num_heads_v=self.Hv, head_dim_k=self.dk, head_dim_v=self.dv,
                             A_log=self.A_log, dt_bias=self.dt_bias, l2_norm=self.l2, scale=self.scale,
                             io_dtype=code[self.io], out_dtype=code[self.out_t], num_slots=self.num_slots,
                             q_row_stride=self.stride, k_row_stride=self.stride, v_row_stride=self.stride)

    def prefill(self, kda, r0=0, lens=None, stream=None):
        """The call over sequences of `lens` starting at row r0 (default: all)."""
        lens = self.lens if lens is None else lens
        cu = self.cu if lens is self.lens else torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
        p, T = self.params(kda), int(sum(lens))
        need = kda.kda_gdn_prefill_workspace_bytes(p, len(lens), T)
        ws = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
        kda.check(kda.kda_gdn_prefill_varlen(p, cu, len(lens), T, self.q[r0:], self.k[r0:], self.v[r0:], self.a[r0:].clone(),
                                             self.b[r0:].clone(), self.slots, self.g_state.tensor,
                                             self.g_out.tensor[r0:], ws, need, self.status, stream))
        torch.cuda.synchronize()

    def decode(self, kda, stream=None):
        kda.check(kda.kda_gdn_decode(self.params(kda), self.N, self.q, self.k, self.v, self.a, self.b, self.slots,
                                     self.g_state.tensor, self.g_out.tensor, self.status, stream))
        torch.cuda.synchronize()

    def want(self):
        T = self.T
        f = lambda x, *s: x[:T].double().cpu().numpy().reshape(T, *s)  # noqa: E731
        return P.gdn(self.lens, f(self.q, self.Hk, self.dk), f(self.k, self.Hk, self.dk), f(self.v, self.Hv, self.dv),
                     f(self.a, self.Hv), f(self.b, self.Hv), self.A_log.double().cpu().numpy(),
                     self.dt_bias.double().cpu().numpy(), self.state0.double().cpu().numpy(), self.slots_h, self.scale, self.l2)

    def check(self, tol_out=None, tol_state=None, status=0):
        out, state = self.want()
        chunk = self.io == "bf16"
        tol_out = tol_out or (OUT if self.out_t == "bf16" else STATE if chunk else FP32)
        tol_state = tol_state or (STATE if chunk else FP32)
        got_o, got_s = self.g_out.tensor[:self.T].double().cpu().numpy(), self.g_state.tensor.double().cpu().numpy()
        assert np.isfinite(got_o).all() and np.isfinite(got_s).all()
        eo, es = P.rel(got_o, out), P.rel(got_s, state)
        assert es <= tol_state, f"state off by {es:.3g}"
        assert eo <= tol_out, f"out off by {eo:.3g}"
        assert (got_o[np.isnan(out)] == 7.0).all()  # rows that are nobody's stay as they were
        assert int(self.status.item()) == status
        assert self.g_state.intact() and self.g_out.intact()
        return eo, es


@pytest.mark.parametrize("lens", [[1], [2], [15], [16], [17], [63], [64], [65], [127], [128], [129], [193], [320],
                                  [1, 0, 130, 64, 0, 7], [0, 0, 5]])
def test_prefill_lengths(cuda_lib, lens):
    c = Case(lens, seed=sum(lens))
    c.prefill(cuda_lib)
    c.check()


@pytest.mark.parametrize("io,out", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("dk,dv", [(32, 32), (32, 128), (64, 64), (128, 32), (128, 64), (64, 128), (128, 128)])
def test_prefill_types_and_widths(cuda_lib, dk, dv, io, out):
    c = Case([70, 1, 150], dk=dk, dv=dv, io=io, out=out, seed=dk + dv)
    c.prefill(cuda_lib)
    c.check()


@pytest.mark.parametrize("Hk,Hv", [(1, 1), (1, 4), (3, 3), (3, 6), (5, 20)])
@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_prefill_head_groups(cuda_lib, Hk, Hv, io):
    c = Case([100, 30], Hk=Hk, Hv=Hv, dk=64, dv=64, io=io, out="f32", seed=Hv)
    c.prefill(cuda_lib)
    c.check()


@pytest.mark.parametrize("heads", [1, 40])
def test_prefill_one_head_as_among_many(cuda_lib, heads):
    """A head's results do not depend on how many others the call has: the same bits."""
    c = Case([200, 90], Hk=heads, Hv=heads, seed=3)
    c.prefill(cuda_lib)
    c.check()
    if heads == 1:
        return
    one = Case([200, 90], Hk=heads, Hv=heads, seed=3)
    one.q, one.k, one.v = (x[:, :128] for x in (one.q, one.k, one.v))
    one.a, one.b = one.a[:, :1].contiguous(), one.b[:, :1].contiguous()
    one.Hk = one.Hv = 1
    one.state0 = one.state0[:, :1].contiguous()
    one.g_state, one.g_out = Guarded(one.state0.shape, torch.float32, "cuda"), Guarded((290, 1, 128), torch.bfloat16, "cuda")
    one.reset()
    one.prefill(cuda_lib)
    assert torch.equal(one.g_out.tensor[:, 0], c.g_out.tensor[:, 0])
    assert torch.equal(one.g_state.tensor[:, 0], c.g_state.tensor[:, 0])


@pytest.mark.parametrize("dense", [False, True])
def test_prefill_strides(cuda_lib, dense):
    c = Case([90, 41], dense=dense, seed=8)
    c.prefill(cuda_lib)
    c.check()


@pytest.mark.parametrize("io,out", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
def test_prefill_without_l2_norm(cuda_lib, io, out):
    c = Case([130, 65], l2=False, io=io, out=out, seed=9)
    c.prefill(cuda_lib)
    c.check()


@pytest.mark.parametrize("kw", [
    dict(gate=-30.0),                  # no decay at all
    dict(gate=30.0, dt=5.0),           # every row forgets everything
    dict(gate=1e30, dt=0.0),           # an infinite log decay is a clean reset
    dict(gate=2.0, dt=1.0),            # strong decays: sums far below zero within a chunk
    dict(beta=12.0, gate=-30.0),       # beta near one: full corrections
    dict(beta=-25.0),                  # beta near zero: the state hardly takes anything
    dict(spread=1e-12), dict(spread=1e12),
], ids=str)
@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_prefill_gates_and_ranges(cuda_lib, kw, io):
    c = Case([150, 64], seed=11, io=io, out="f32", **kw)
    if kw.get("spread"):
        c.state0 *= kw["spread"]
        c.reset()
    c.prefill(cuda_lib)
    c.check(tol_out=2 * STATE)


def test_prefill_mixed_decays(cuda_lib):
    """Rows that reset the state between rows that keep it: a row's reset may
    not cost the digits of the small decays after it."""
    c = Case([200], Hk=2, Hv=2, seed=12, out="f32")
    c.a[::3] = 60.0
    c.a[1::3] = -4.0
    c.prefill(cuda_lib)
    c.check()


def test_prefill_correlated_keys(cuda_lib):
    """Nearly equal keys: I + A is far from the identity."""
    c = Case([256], Hk=2, Hv=2, seed=13, out="f32", beta=3.0, gate=-10.0)
    c.k[:] = c.k[:1] + 0.05 * c.k
    c.prefill(cuda_lib)
    c.check(tol_out=2.0 ** -16, tol_state=2.0 ** -16)  # products of the 64 corrections, each 2^-22 off


def test_prefill_slots(cuda_lib):
    """A pool larger than the batch, a padded sequence, a slot out of range:
    what is nobody's stays as it was."""
    c = Case([40, 70, 5, 130], slots=[5, -1, 0, 3], num_slots=7, seed=14)
    c.prefill(cuda_lib)
    c.check()
    bad = Case([40, 70], slots=[7, 2], num_slots=7, seed=15)
    bad.slots_h = [-1, 2]
    bad.prefill(cuda_lib)
    bad.check(status=cuda_lib.KDA_DEV_BAD_SLOT)


def test_prefill_bad_cu_seqlens(cuda_lib):
    c = Case([50, 60, 40], seed=16)
    c.cu[2] = 40       # sequence 1 would run backwards, sequence 2 from 40 to 150
    c.prefill(cuda_lib)
    assert int(c.status.item()) == cuda_lib.KDA_DEV_BAD_SEQLENS
    assert torch.equal(c.g_state.tensor[1], c.state0[1])
    c = Case([50, 60], seed=16)
    c.cu[2] = 111      # past the last row
    c.prefill(cuda_lib)
    assert int(c.status.item()) == cuda_lib.KDA_DEV_BAD_SEQLENS
    assert torch.equal(c.g_state.tensor[1], c.state0[1]) and (c.g_out.tensor[50:] == 7.0).all()


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("cuts", [(64, 128, 108), (1, 99, 200)])
def test_prefill_in_pieces(cuda_lib, out, cuts):
    c = Case([300], seed=17, out=out)
    r0 = 0
    for ln in cuts:
        c.prefill(cuda_lib, r0, [ln])
        r0 += ln
    c.check()


def test_prefill_nan_stays_in_its_sequence_and_head(cuda_lib):
    c = Case([70, 70], Hk=2, Hv=2, seed=18)
    clean = Case([70, 70], Hk=2, Hv=2, seed=18)
    clean.prefill(cuda_lib)
    c.v[80, 5] = float("nan")     # sequence 1, head 0, column 5
    c.q[10, 3] = float("inf")     # sequence 0, head 0: its row alone
    c.prefill(cuda_lib)
    a, b = c.g_out.tensor, clean.g_out.tensor
    keep = torch.ones_like(a, dtype=torch.bool)
    keep[10, 0] = False
    keep[70:, 0, 5] = False
    assert torch.equal(a[keep], b[keep])
    assert torch.equal(c.g_state.tensor[0], clean.g_state.tensor[0])
    assert a[10, 0].isnan().all() and a[80:, 0, 5].isnan().all()


def test_prefill_more_sequences_than_threads(cuda_lib):
    """More sequences than threads of a CTA: they keep their order."""
    r = np.random.default_rng(1)
    lens = r.integers(0, 6, 300).tolist()
    c = Case(lens, Hk=1, Hv=1, dk=32, dv=32, seed=19)
    c.prefill(cuda_lib)
    c.check()


@pytest.mark.parametrize("B", [1, 2, 7, 33])
@pytest.mark.parametrize("io,out", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("dk,dv", [(128, 128), (32, 64), (64, 32), (128, 32), (32, 128)])
def test_decode(cuda_lib, B, io, out, dk, dv):
    c = Case([1] * B, Hk=2, Hv=6, dk=dk, dv=dv, io=io, out=out, seed=B + dk)
    c.decode(cuda_lib)
    c.check(tol_out=2.0 ** -8 if out == "bf16" else FP32, tol_state=FP32)


def test_decode_large_batch_slots(cuda_lib):
    c = Case([1] * 40, Hk=4, Hv=8, slots=[-1] + list(range(41, 2, -1)), num_slots=42, seed=20)
    c.decode(cuda_lib)
    c.check(tol_out=2.0 ** -8, tol_state=FP32)
    bad = Case([1] * 3, slots=[1, 9, 0], num_slots=3, seed=21)
    bad.slots_h = [1, -1, 0]
    bad.decode(cuda_lib)
    bad.check(tol_out=2.0 ** -8, tol_state=FP32, status=cuda_lib.KDA_DEV_BAD_SLOT)


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_prefill_then_decode(cuda_lib, io):
    """A prompt's rows cut after any row: prefill, then single tokens, is one recurrence."""
    lens, tail = [70, 33], 3
    c = Case(lens, io=io, out="f32", seed=22)
    heads = [ln - tail for ln in lens]
    first = np.concatenate([[0], np.cumsum(lens)])[:-1]
    idx = np.concatenate([np.arange(f, f + h) for f, h in zip(first, heads)])
    p = c.params(cuda_lib)
    cu = torch.tensor([0, heads[0], sum(heads)], dtype=torch.int32, device="cuda")
    take = lambda x: x[idx].contiguous()  # noqa: E731
    stride = dict(q_row_stride=0, k_row_stride=0, v_row_stride=0)
    p.__dict__.update(stride)
    T = sum(heads)
    out = torch.empty(T, c.Hv, c.dv, device="cuda")
    need = cuda_lib.kda_gdn_prefill_workspace_bytes(p, 2, T)
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
    cuda_lib.check(cuda_lib.kda_gdn_prefill_varlen(p, cu, 2, T, take(c.q), take(c.k), take(c.v), take(c.a), take(c.b),
                                                   None, c.g_state.tensor, out, ws, need, c.status))
    c.g_out.tensor[idx] = out
    for i in range(tail):
        rows = [f + h + i for f, h in zip(first, heads)]
        one = lambda x: x[rows].contiguous()  # noqa: E731
        o = torch.empty(2, c.Hv, c.dv, device="cuda")
        cuda_lib.check(cuda_lib.kda_gdn_decode(p, 2, one(c.q), one(c.k), one(c.v), one(c.a), one(c.b), None,
                                               c.g_state.tensor, o, c.status))
        c.g_out.tensor[rows] = o
    torch.cuda.synchronize()
    c.check(tol_out=STATE, tol_state=STATE)


def test_graph_replay_and_other_stream(cuda_lib):
    """Captured on a stream of its own and replayed: the eager calls' bits,
    each replay on what the buffers hold by then."""
    c, d = Case([130, 20], seed=23), Case([1] * 5, seed=24)
    c.prefill(cuda_lib)
    d.decode(cuda_lib)
    want = [x.clone() for x in (c.g_out.tensor, c.g_state.tensor, d.g_out.tensor, d.g_state.tensor)]
    for x in (c, d):
        x.reset()
    p = c.params(cuda_lib)
    need = cuda_lib.kda_gdn_prefill_workspace_bytes(p, 2, 150)
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cuda_lib.check(cuda_lib.kda_gdn_prefill_varlen(p, c.cu, 2, 150, c.q, c.k, c.v, c.a, c.b, None, c.g_state.tensor,
                                                       c.g_out.tensor, ws, need, c.status))
        cuda_lib.check(cuda_lib.kda_gdn_decode(d.params(cuda_lib), 5, d.q, d.k, d.v, d.a, d.b, None, d.g_state.tensor,
                                               d.g_out.tensor, d.status))
    for _ in range(2):
        for x in (c, d):
            x.reset()
        graph.replay()
        torch.cuda.synchronize()
        for got, w in zip((c.g_out.tensor, c.g_state.tensor, d.g_out.tensor, d.g_state.tensor), want):
            assert torch.equal(got, w)


def test_two_calls_at_once(cuda_lib):
    """Two calls on two streams, a workspace each: each has its own result."""
    cs = [Case([257, 100], seed=25 + i) for i in range(2)]
    for c in cs:
        c.prefill(cuda_lib)
    want = [(c.g_out.tensor.clone(), c.g_state.tensor.clone()) for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    for c in cs:
        c.reset()
    torch.cuda.synchronize()
    keep = []
    for c, s in zip(cs, streams):
        p = c.params(cuda_lib)
        need = cuda_lib.kda_gdn_prefill_workspace_bytes(p, 2, 357)
        keep.append(torch.empty(max(need, 16), dtype=torch.uint8, device="cuda"))
        torch.cuda.synchronize()
    for c, s, ws in zip(cs, streams, keep):
        p = c.params(cuda_lib)
        need = cuda_lib.kda_gdn_prefill_workspace_bytes(p, 2, 357)
        cuda_lib.check(cuda_lib.kda_gdn_prefill_varlen(p, c.cu, 2, 357, c.q, c.k, c.v, c.a, c.b, None, c.g_state.tensor,
                                                       c.g_out.tensor, ws, need, c.status, s))
    torch.cuda.synchronize()
    for c, (o, st) in zip(cs, want):
        assert torch.equal(c.g_out.tensor, o) and torch.equal(c.g_state.tensor, st)


def test_long_prompt(cuda_lib):
    """Many chunks of one sequence: errors do not pile up."""
    c = Case([4000], Hk=1, Hv=2, out="f32", seed=30)
    c.prefill(cuda_lib)
    c.check()


def _beside(c):
    """Whether a call of this case runs its chains beside prep (up to 64 sequences, more slots than one wave of prep)."""
    slots = c.T // 64 + c.N
    return c.N <= 64 and slots * c.Hv > (3 if c.out_t == "bf16" else 2) * 152


@pytest.mark.parametrize("Hk,Hv,dk,dv,out,lens", [
    (1, 8, 32, 32, "bf16", [4100]),
    (2, 8, 32, 64, "f32", [0, 1500, 1, 700, 0, 130]),
    (8, 8, 64, 32, "f32", [1800, 900]),
    (3, 3, 32, 128, "bf16", [40, 9900]),
    (4, 16, 128, 128, "bf16", [1100, 64, 65, 700]),
])
def test_prefill_chains_beside_prep(cuda_lib, Hk, Hv, dk, dv, out, lens):
    slots = list(range(len(lens)))
    if len(lens) > 3:
        slots[3] = -1  # a padded sequence among them
    c = Case(lens, Hk=Hk, Hv=Hv, dk=dk, dv=dv, out=out, seed=40 + dk, slots=slots)
    assert _beside(c)
    c.prefill(cuda_lib)
    c.check()


def test_prefill_beside_gives_the_bits_of_one_after_the_other(cuda_lib):
    """The same rows as a call of their own (chains beside prep) and among
    so many others that prep runs first: the same bits; and again on a
    workspace full of ones."""
    lens = [1400, 1100]
    c = Case(lens, Hk=6, Hv=12, dk=64, dv=64, seed=50)
    assert _beside(c)
    c.prefill(cuda_lib)
    want = c.g_out.tensor.clone(), c.g_state.tensor.clone()
    c.reset()
    p = c.params(cuda_lib)
    need = cuda_lib.kda_gdn_prefill_workspace_bytes(p, 2, c.T)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    cuda_lib.check(cuda_lib.kda_gdn_prefill_varlen(p, c.cu, 2, c.T, c.q, c.k, c.v, c.a, c.b, None, c.g_state.tensor,
                                                   c.g_out.tensor, ws, need, c.status))
    torch.cuda.synchronize()
    assert torch.equal(c.g_out.tensor, want[0]) and torch.equal(c.g_state.tensor, want[1])
    many = Case(lens + [1] * 63, Hk=6, Hv=12, dk=64, dv=64, seed=51)
    assert not _beside(many)
    n = c.T
    many.rows[:n].copy_(c.rows)
    many.a[:n].copy_(c.a)
    many.b[:n].copy_(c.b)
    many.A_log, many.dt_bias = c.A_log, c.dt_bias
    many.state0[:2].copy_(c.state0)
    many.reset()
    many.prefill(cuda_lib)
    assert torch.equal(many.g_out.tensor[:n], want[0]) and torch.equal(many.g_state.tensor[:2], want[1])


def test_beside_in_a_graph_and_twice_at_once(cuda_lib):
    """Captured and replayed; and two such calls on two streams, a workspace each."""
    cs = [Case([2600, 500], Hk=4, Hv=16, dk=32, dv=32, seed=60 + i) for i in range(2)]
    assert _beside(cs[0])
    for c in cs:
        c.prefill(cuda_lib)
    want = [(c.g_out.tensor.clone(), c.g_state.tensor.clone()) for c in cs]
    p = cs[0].params(cuda_lib)
    need = cuda_lib.kda_gdn_prefill_workspace_bytes(p, 2, 3100)
    ws = [torch.empty(need, dtype=torch.uint8, device="cuda") for _ in cs]

    def call(i, stream=None):
        c = cs[i]
        cuda_lib.check(cuda_lib.kda_gdn_prefill_varlen(c.params(cuda_lib), c.cu, 2, 3100, c.q, c.k, c.v, c.a, c.b, None,
                                                       c.g_state.tensor, c.g_out.tensor, ws[i], need, c.status, stream))

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(0)
    for _ in range(2):
        cs[0].reset()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(cs[0].g_out.tensor, want[0][0]) and torch.equal(cs[0].g_state.tensor, want[0][1])
    for c in cs:
        c.reset()
    torch.cuda.synchronize()
    for i, s in enumerate([torch.cuda.Stream(), torch.cuda.Stream()]):
        call(i, s)
    torch.cuda.synchronize()
    for c, (o, st) in zip(cs, want):
        assert torch.equal(c.g_out.tensor, o) and torch.equal(c.g_state.tensor, st) and int(c.status.item()) == 0


def test_back_to_back_calls_keep_their_order(cuda_lib):
    """Calls right behind one another on a stream, each on the states and rows the one before left (their
    kernels may start early, their memory accesses may not)."""
    c = Case([1] * 4, Hk=2, Hv=4, seed=70)
    for _ in range(20):
        cuda_lib.check(cuda_lib.kda_gdn_decode(c.params(cuda_lib), 4, c.q, c.k, c.v, c.a, c.b, None, c.g_state.tensor,
                                               c.g_out.tensor, c.status))
    torch.cuda.synchronize()
    got = c.g_state.tensor.clone()
    c.reset()
    for _ in range(20):
        c.decode(cuda_lib)
    assert torch.equal(got, c.g_state.tensor)


@pytest.mark.parametrize("out,Hk,Hv,dk", [("f32", 8, 16, 32), ("bf16", 4, 16, 64), ("bf16", 5, 15, 32)])
@pytest.mark.parametrize("ones", [0, 60])
def test_prefill_many_heads_of_shared_keys(cuda_lib, out, Hk, Hv, dk, ones):
    """Enough chunk-heads that prep takes two heads of one key head together (an odd group: one); more chains
    than SMs, odd and even ones, taken one after the other beside prep, or (many sequences) after it."""
    lens = [200, 0, 65, 700, 1, 64, 333, 128, 500, 130, 90, 640]
    c = Case(lens + [1] * ones, Hk=Hk, Hv=Hv, dk=dk, dv=32, out=out, seed=80,
             slots=[3, 0, 7, -1, 5, 1, 2, 11, 4, 6, 8, 9] + list(range(12, 12 + ones)))
    assert _beside(c) == (ones == 0) and (c.T // 64 + c.N) * Hv > 3 * 152
    c.prefill(cuda_lib)
    c.check()


def test_prefill_many_chains_for_each_cta(cuda_lib):
    r = np.random.default_rng(5)
    c = Case(r.integers(0, 200, 64).tolist(), Hk=4, Hv=32, dk=32, dv=32, seed=81, num_slots=70,
             slots=[int(s) if i % 9 else -1 for i, s in enumerate(r.permutation(70)[:64])])
    assert _beside(c)
    c.prefill(cuda_lib)
    c.check()


def test_prefill_beside_flags_bad_sequences_and_slots(cuda_lib):
    c = Case([900, 60, 500, 1200], Hk=4, Hv=16, dk=32, dv=32, seed=82, slots=[2, 9, 1, 0], num_slots=4)
    c.slots_h[1] = -1
    assert _beside(c)
    c.prefill(cuda_lib)
    c.check(status=cuda_lib.KDA_DEV_BAD_SLOT)
    c = Case([900, 60, 500, 1200], Hk=4, Hv=16, dk=32, dv=32, seed=82)
    c.cu[4] = c.T + 1
    c.prefill(cuda_lib)
    assert int(c.status.item()) == cuda_lib.KDA_DEV_BAD_SEQLENS
    assert torch.equal(c.g_state.tensor[3], c.state0[3]) and (c.g_out.tensor[1460:] == 7.0).all()


@pytest.mark.parametrize("huge", [2.0 ** 30, float("inf"), float("nan")])
@pytest.mark.parametrize("l2", [False, True])
def test_prefill_keys_of_the_next_sequence_do_not_matter(cuda_lib, l2, huge):
    """A chunk's last rows come with the next sequence's first ones: whatever stands there changes no bit."""
    c, clean = (Case([70, 30], Hk=2, Hv=2, seed=90, out="f32", l2=l2) for _ in range(2))
    clean.prefill(cuda_lib)
    clean.check()
    c.k[70:90] *= huge
    c.prefill(cuda_lib)
    assert torch.equal(c.g_out.tensor[:70], clean.g_out.tensor[:70])
    assert torch.equal(c.g_state.tensor[0], clean.g_state.tensor[0])


@pytest.mark.parametrize("N", [33, 1100])
def test_prefill_many_sequences(cuda_lib, N):
    lens = np.random.default_rng(N).integers(0, 4, N)
    lens[N // 2] = 140
    c = Case(lens.tolist(), Hk=1, Hv=2, dk=32, dv=32, seed=91, slots=np.random.default_rng(1).permutation(N).tolist())
    c.prefill(cuda_lib)
    c.check()


@pytest.mark.parametrize("Hv,rows", [(2, 200), (16, 2600)])
def test_prefill_bad_gates_stay_in_their_sequence_and_head(cuda_lib, Hv, rows):
    """A NaN or infinite gate logit ends in its own sequence's rows and state, and leaves no wait behind."""
    bad, clean = (Case([rows, 70, 130], Hk=2, Hv=Hv, dk=32, dv=32, seed=95) for _ in range(2))
    assert _beside(bad) == (Hv == 16)
    clean.prefill(cuda_lib)
    bad.a[30, 1] = float("nan")
    bad.b[rows + 3, 0] = float("nan")
    bad.a[rows + 75, 1] = float("-inf")   # no decay at all: finite
    bad.prefill(cuda_lib)
    same = torch.ones(bad.T, Hv, dtype=torch.bool, device="cuda")
    same[:rows, 1] = same[rows:rows + 70, 0] = same[rows + 70:, 1] = False
    assert torch.equal(bad.g_out.tensor[same], clean.g_out.tensor[same])
    assert torch.equal(bad.g_state.tensor[0, 0], clean.g_state.tensor[0, 0])
    assert torch.equal(bad.g_state.tensor[1, 1:], clean.g_state.tensor[1, 1:])
    assert bad.g_state.tensor[0, 1].isnan().all() and bad.g_out.tensor[rows + 70:].isfinite().all()
    assert int(bad.status.item()) == 0


@pytest.mark.parametrize("lens,Hk,Hv,dk,dv,seed,kw", [
    ([436], 8, 16, 128, 64, 739419993, dict(gate=3.0)),
    ([300], 2, 4, 64, 128, 96, dict(beta=4.0)),
    ([521], 4, 8, 32, 128, 1023189493, dict(l2=False)),
    ([200, 130], 2, 2, 128, 128, 97, dict(l2=False, gate=2.0)),
])
@pytest.mark.parametrize("spread", [1e-6, 2.0 ** -40])
def test_prefill_rows_far_below_the_state_they_meet(cuda_lib, lens, Hk, Hv, dk, dv, seed, kw, spread):
    """Rows of another magnitude than the state decay it by many orders to theirs (and, normalised, are small
    next to the norm's eps): the small state that is left has all its digits.

    Tolerance: a row of T R is a sum of up to 64 terms, each off by 2^-22 of the largest.  Errors of either sign
    add up to 8 * 2^-22, half of STATE; but the 64 rows of a chunk on 32 dims are never independent, each is
    corrected along the ones before it, and errors of one sign add up to 64 * 2^-22 = 2^-16."""
    c = Case(lens, Hk=Hk, Hv=Hv, dk=dk, dv=dv, seed=seed, out="f32", spread=spread, **kw)
    c.prefill(cuda_lib)
    tol = 2.0 ** -16 if dk < 64 else STATE
    c.check(tol_out=tol, tol_state=tol)


@pytest.mark.parametrize("Hv,dk", [(2, 128), (4, 64)])
def test_prefill_keys_of_all_magnitudes(cuda_lib, Hv, dk):
    """Without the norm, keys from 2^-12 to 2^12 side by side, their beta |k|^2 up to one: T as it stands would
    have entries of 2^24 and more."""
    c = Case([200, 90], Hk=2, Hv=Hv, dk=dk, dv=64, seed=98, out="f32", l2=False)
    e = torch.from_numpy(np.random.default_rng(98).integers(-12, 13, (c.T, 1))).cuda()
    c.k.copy_(torch.ldexp(c.k.float(), e))
    c.b.copy_((-2 * math.log(2.0)) * e.clamp(min=0) + c.b.float().clamp(max=0))
    c.prefill(cuda_lib)
    c.check()


@pytest.mark.parametrize("lens,Hv,dk", [([64], 1, 128), ([200, 70], 2, 64), ([100, 3], 4, 32)])
@pytest.mark.parametrize("kind", ["zeros", "zeros after a reset", "one small row"])
@pytest.mark.parametrize("l2", [False, True])
def test_prefill_rows_of_zeros_on_a_large_state(cuda_lib, lens, Hv, dk, kind, l2):
    """Rows that give next to nothing (2^-120 of the keys, no values) on states near 2^58: what the rows' scale
    and the state's make together has to stay finite."""
    c = Case(lens, Hk=1, Hv=Hv, dk=dk, dv=32, seed=99, out="f32", l2=l2, gate=-30.0)
    c.state0 *= 2.0 ** 59
    c.rows.zero_()
    if kind == "zeros after a reset":
        c.a[65:66] = 1e30  # the state is all zeros from there on, its last scale still there
    if kind == "one small row":
        c.v[1:2] = 2.0 ** -60
        c.k[1:2, 3] = 1.0
    c.reset()
    c.prefill(cuda_lib)
    c.check()


def test_prefill_on_a_part_of_the_device(cuda_lib):
    """A long call on a stream that may use a part of the SMs only: no grid that needs them all, the same bits."""
    from tests.green import stream_on_part

    c = Case([1100, 64, 65, 700], Hk=4, Hv=16, seed=100)
    assert _beside(c)
    c.prefill(cuda_lib)
    c.check()
    want = c.g_out.tensor.clone(), c.g_state.tensor.clone()
    c.reset()
    torch.cuda.synchronize()
    with stream_on_part(32) as (cu, stream, sms):
        assert sms < torch.cuda.get_device_properties(0).multi_processor_count
        c.prefill(cuda_lib, stream=stream.value)
        assert cu.cuStreamSynchronize(stream) == 0
    assert torch.equal(c.g_out.tensor, want[0]) and torch.equal(c.g_state.tensor, want[1]) and int(c.status.item()) == 0


@pytest.mark.parametrize("fall", [16, 20])
@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 32), (32, 64)])
def test_prefill_state_far_below_the_one_a_chunk_met(cuda_lib, dk, dv, fall):
    """One chunk whose decays leave a state 2^fall below the one it met.

    Tolerance: T is kept with D on either side, D >= 2^-12 the rows' decay to the chunk's end, so that its entries
    are off by 2^-25 (fp16's smallest half step) at most; the chunk's first rows meet them with D R, 2^(fall - 12)
    times the new state, and up to 64 of them add up, of either sign: 2^(fall - 37) * 8 of the new state, beside STATE."""
    c = Case([64, 64], Hk=2, Hv=2, dk=dk, dv=dv, seed=110 + fall, out="f32")
    c.A_log.zero_()
    c.a.zero_()
    c.dt_bias.fill_(math.log(math.expm1(fall * math.log(2.0) / 64)))
    c.state0 *= 2.0 ** fall / 0.1
    c.reset()
    c.prefill(cuda_lib)
    tol = 2.0 ** (fall - 34) + STATE
    c.check(tol_out=tol, tol_state=tol)


@pytest.mark.parametrize("l2", [False, True])
@pytest.mark.parametrize("spread", [1.0, 2.0 ** -40])
def test_prefill_rows_of_zeros_among_strong_decays(cuda_lib, l2, spread):
    """Rows of zeros (whose scale is the largest there is) that the chunk's end has forgotten, between others."""
    c = Case([150, 64], Hk=2, Hv=2, dk=64, dv=64, seed=101, out="f32", l2=l2, gate=1.0, dt=0.0, spread=spread)
    c.state0 *= spread
    c.rows[::3] = 0
    c.rows[64:100] = 0
    c.reset()
    c.prefill(cuda_lib)
    c.check()


@pytest.mark.parametrize("lens", [[90, 41], [1100, 64, 65, 700]])
def test_calls_from_another_thread(cuda_lib, lens):
    """A thread whose first CUDA call this is: the same bits."""
    import threading

    c = Case(lens, Hk=4, Hv=16, seed=102)
    c.prefill(cuda_lib)
    want = c.g_out.tensor.clone(), c.g_state.tensor.clone()
    c.reset()
    p = c.params(cuda_lib)
    need = cuda_lib.kda_gdn_prefill_workspace_bytes(p, c.N, c.T)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream
    torch.cuda.synchronize()
    rc = []
    t = threading.Thread(target=lambda: rc.append(cuda_lib.kda_gdn_prefill_varlen(
        p, c.cu, c.N, c.T, c.q, c.k, c.v, c.a, c.b, None, c.g_state.tensor, c.g_out.tensor, ws, need, c.status, stream)))
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert rc == [cuda_lib.KDA_OK] and int(c.status.item()) == 0
    assert torch.equal(c.g_out.tensor, want[0]) and torch.equal(c.g_state.tensor, want[1])


@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 32), (32, 128)])
def test_prefill_nearly_equal_keys_of_the_largest_norm(cuda_lib, dk, dv):
    """Nearly equal keys of beta |k|^2 near 2, hardly any decay: every correction turns the last one around.

    Tolerance: T's entries alternate around +-2 along 64 rows, so the sums that make M and S' are of 64 terms of
    one size and either sign, each 2^-22 of 2 off: 2^-15."""
    c = Case([150, 64], Hk=1, Hv=2, dk=dk, dv=dv, seed=103, out="f32", l2=False, gate=-10.0, beta=9.0)
    c.k[:] = c.k[:1] + 0.05 * c.k
    k = c.k.float()
    c.k.copy_(k / k.norm(dim=-1, keepdim=True) * 1.4)
    c.prefill(cuda_lib)
    c.check(tol_out=2.0 ** -15, tol_state=2.0 ** -15)
