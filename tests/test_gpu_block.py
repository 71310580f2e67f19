"""The convolution with carried state, the norms around a block and the slot
operations on the GPU, against their definitions in 64 bits.

Tolerances: half a step of the output type (bf16 2^-8, fp32 2^-24 relative to
the value) plus the fp32 arithmetic in front of it: K products and the SiLU's two
special-function results (2 ulp each) for the convolution, a sum of up to
16384 squares (sqrt(n) 2^-24) and three products for the norms: 2^-20 covers
both.
"""
import numpy as np
import pytest
import torch

from linear_attention_serving_kda_gb300.runtime import Guarded
from tests import plain64 as P

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
TOL = {"bf16": 2.0 ** -8, "f32": 2.0 ** -20}


def _code(kda, io):
    return kda.KDA_DTYPE_BF16 if io == "bf16" else kda.KDA_DTYPE_F32


def _f(x):
    return x.double().cpu().numpy()


class Conv:
    def __init__(self, lens, C, K, io, seed, slots=None, num_slots=None):
        r = np.random.default_rng(seed)
        self.lens, self.T, self.N, self.C, self.K, self.io = lens, int(sum(lens)), len(lens), C, K, io
        t = lambda a: torch.from_numpy(a).to(DT[io]).cuda()  # noqa: E731
        self.x = t(r.standard_normal((max(self.T, 1), C)))
        self.w = torch.from_numpy(r.standard_normal((C, K))).float().cuda()
        self.num_slots = num_slots or self.N
        self.state0 = t(r.standard_normal((self.num_slots, K - 1, C)))
        self.slots_h = list(range(self.N)) if slots is None else slots
        self.slots = None if slots is None else torch.tensor(slots, dtype=torch.int32, device="cuda")
        self.state, self.y = Guarded(self.state0.shape, DT[io], "cuda"), Guarded(self.x.shape, DT[io], "cuda")
        self.state.tensor.copy_(self.state0)
        self.y.tensor.fill_(7.0)
        self.cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def params(self, kda):
        return kda.ConvParams(channels=self.C, conv_kernel=self.K, conv_weight=self.w, io_dtype=_code(kda, self.io),
                              num_slots=self.num_slots)

    def run(self, kda, decode=False):
        if decode:
            rc = kda.kda_conv_decode(self.params(kda), self.N, self.x, self.slots, self.state.tensor, self.y.tensor, self.status)
        else:
            rc = kda.kda_conv_varlen(self.params(kda), self.cu, self.N, self.T, self.x, self.slots, self.state.tensor,
                                     self.y.tensor, self.status)
        kda.check(rc)
        torch.cuda.synchronize()

    def check(self, status=0):
        y, st = P.conv(self.lens, _f(self.x), _f(self.w), _f(self.state0), self.slots_h)
        got = _f(self.y.tensor)
        assert P.rel(got, y) <= TOL[self.io]
        assert (got[np.isnan(y)] == 7.0).all()
        assert np.array_equal(_f(self.state.tensor), st)  # raw rows, copied
        assert int(self.status.item()) == status and self.y.intact() and self.state.intact()


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("K", [2, 3, 4])
@pytest.mark.parametrize("lens", [[1], [2, 1, 3], [31, 32, 33, 0, 64, 65], [200]], ids=str)
@pytest.mark.parametrize("C", [8, 136, 1032])
def test_conv_varlen(cuda_lib, lens, K, C, io):
    c = Conv(lens, C, K, io, sum(lens) + C)
    c.run(cuda_lib)
    c.check()


def test_conv_varlen_slots_and_faults(cuda_lib):
    c = Conv([40, 3, 70], 64, 4, "bf16", 3, slots=[4, -1, 0], num_slots=6)
    c.run(cuda_lib)
    c.check()
    c = Conv([40, 3, 70], 64, 4, "bf16", 3, slots=[6, 1, 0], num_slots=6)
    c.slots_h = [-1, 1, 0]
    c.run(cuda_lib)
    c.check(status=cuda_lib.KDA_DEV_BAD_SLOT)
    c = Conv([40, 30], 64, 4, "bf16", 4)
    c.cu[2] = 71
    c.run(cuda_lib)
    assert int(c.status.item()) == cuda_lib.KDA_DEV_BAD_SEQLENS and (c.y.tensor[40:] == 7.0).all()


def test_conv_many_sequences(cuda_lib):
    c = Conv(np.random.default_rng(0).integers(0, 5, 300).tolist(), 32, 4, "bf16", 5)
    c.run(cuda_lib)
    c.check()


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("K", [2, 3, 4])
@pytest.mark.parametrize("B,C", [(1, 8), (3, 1032), (17, 256)])
def test_conv_decode(cuda_lib, B, C, K, io):
    slots = list(range(B, 0, -1))
    slots[0] = -1 if B > 1 else 1
    c = Conv([1] * B, C, K, io, B + C, slots=slots, num_slots=B + 1)
    c.run(cuda_lib, decode=True)
    c.check()


def test_conv_prefill_then_decode(cuda_lib):
    """Rows one by one after a prompt: the same values and the same state as in one call."""
    whole = Conv([70], 64, 4, "bf16", 6)
    whole.run(cuda_lib)
    c = Conv([70], 64, 4, "bf16", 6)
    c.cu[1] = 66
    cuda_lib.check(cuda_lib.kda_conv_varlen(c.params(cuda_lib), c.cu, 1, 66, c.x, None, c.state.tensor, c.y.tensor, c.status))
    for t in range(66, 70):
        cuda_lib.check(cuda_lib.kda_conv_decode(c.params(cuda_lib), 1, c.x[t:], None, c.state.tensor, c.y.tensor[t:], c.status))
    torch.cuda.synchronize()
    assert torch.equal(c.y.tensor, whole.y.tensor) and torch.equal(c.state.tensor, whole.state.tensor)


@pytest.mark.parametrize("io,res", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("D", [8, 24, 128, 256, 264, 520, 1024, 1032, 4096, 8200, 16384])
@pytest.mark.parametrize("post,act,has_res,pre,weights", [
    (True, 2, False, False, True), (True, 1, True, True, True), (False, 0, True, True, False), (True, 0, False, True, True)])
def test_block_norm(cuda_lib, D, io, res, post, act, has_res, pre, weights):
    r = np.random.default_rng(D + act)
    rows = 5 if D > 1024 else 19
    t = lambda dt, s=1.0: torch.from_numpy(r.standard_normal((rows, D)) * s).to(DT[dt]).cuda()  # noqa: E731
    y, g, x0 = t(io, 0.5), t(io) if act else None, t(res, 2.0) if has_res else None
    w = [torch.from_numpy(1 + 0.1 * r.standard_normal(D)).float().cuda() if weights else None for _ in range(2)]
    h, x = Guarded((rows, D), DT[res], "cuda"), Guarded((rows, D), DT[io], "cuda") if pre else None
    p = cuda_lib.NormParams(dim=D, post_norm=post, gate_act=act, residual_scale=0.75, norm_eps=1e-6, post_weight=w[0],
                            pre_weight=w[1], io_dtype=_code(cuda_lib, io), res_dtype=_code(cuda_lib, res))
    cuda_lib.check(cuda_lib.kda_block_norm(p, rows, y, g, x0, h.tensor, None if x is None else x.tensor))
    torch.cuda.synchronize()
    ww = [_f(a) if a is not None else 1.0 for a in w]
    eh, ex = P.block_norm(_f(y), _f(g) if act else None, act, _f(x0) if has_res else None, 0.75, post, ww[0], ww[1], 1e-6)
    assert P.rel(_f(h.tensor), eh) <= TOL[res] and h.intact()
    if pre:
        assert P.rel(_f(x.tensor), ex) <= TOL[io] and x.intact()
        alone = torch.empty_like(x.tensor)  # without h: the same bits
        cuda_lib.check(cuda_lib.kda_block_norm(p, rows, y, g, x0, None, alone))
        torch.cuda.synchronize()
        assert torch.equal(alone, x.tensor)
    # in place: h in the residual's buffer, x in the block output's
    if has_res:
        cuda_lib.check(cuda_lib.kda_block_norm(p, rows, y, g, x0, x0, y if pre else None))
        torch.cuda.synchronize()
        assert torch.equal(x0, h.tensor)
        if pre:
            assert torch.equal(y, x.tensor)


def test_block_norm_zero_and_bad_rows(cuda_lib):
    D = 256
    y = torch.ones(4, D, device="cuda").to(torch.bfloat16)
    y[1] = 0
    y[2, 7] = float("inf")
    x, h = torch.empty_like(y), torch.empty_like(y)
    p = cuda_lib.NormParams(dim=D)
    cuda_lib.check(cuda_lib.kda_block_norm(p, 4, y, None, None, h, x))
    torch.cuda.synchronize()
    assert (x[0] == 1).all() and (x[3] == 1).all() and (x[1] == 0).all() and x[2].isnan().any()


def _pool(cuda_lib, L, S, n, dtype=torch.float32, gap=0, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = Guarded((L, S * n + gap), dtype, "cuda")
    t.tensor.copy_(torch.randn(L, S * n + gap, generator=g, device="cuda"))
    size = t.tensor.element_size()
    return t, cuda_lib.SlotPool(pool=t.tensor, num_layers=L, num_slots=S, slot_bytes=n * size,
                                layer_stride_bytes=(S * n + gap) * size)


def _i32(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _copied(before, S, n, pairs):
    want = before.clone()
    for s, d in pairs:
        want[:, d * n:(d + 1) * n] = before[:, s * n:(s + 1) * n]
    return want


@pytest.mark.parametrize("n", [4, 36, 4096, 4100, 20000])
@pytest.mark.parametrize("L,S,gap", [(1, 5, 0), (3, 9, 16)])
def test_slots_copy(cuda_lib, L, S, gap, n):
    t, pool = _pool(cuda_lib, L, S, n, gap=gap)
    before, status = t.tensor.clone(), _i32(0)
    # a fork, a padded pair, a copy to itself
    cuda_lib.check(cuda_lib.kda_slots_copy(pool, 5, _i32(2, 2, -1, 3, 1), _i32(0, 4, 1, 3, -1), status))
    torch.cuda.synchronize()
    assert torch.equal(t.tensor, _copied(before, S, n, [(2, 0), (2, 4)])) and t.intact() and int(status) == 0


def test_slots_copy_conflicts(cuda_lib):
    """Pairs whose order would matter are flagged and left out, the others run."""
    n, S = 100, 12
    for src, dst, good in [
        ((1, 2, 3), (5, 5, 6), [(3, 6)]),             # one target twice
        ((1, 5, 3), (5, 7, 6), [(5, 7), (3, 6)]),     # a target that is read
        ((1, 2, 3), (2, 1, 6), [(3, 6)]),             # an exchange
        ((1, 12, 3), (4, 5, 99), [(1, 4)]),           # out of range
        ((1, 1), (4, 4), []),                         # the same pair twice
    ]:
        t, pool = _pool(cuda_lib, 2, S, n)
        before, status = t.tensor.clone(), _i32(0)
        cuda_lib.check(cuda_lib.kda_slots_copy(pool, len(src), _i32(*src), _i32(*dst), status))
        torch.cuda.synchronize()
        assert torch.equal(t.tensor, _copied(before, S, n, good)), (src, dst)
        assert int(status) == cuda_lib.KDA_DEV_BAD_SLOT


def test_slots_copy_long_lists(cuda_lib):
    """More pairs than one pass keeps, most of them padding."""
    S, n = 6000, 4
    t, pool = _pool(cuda_lib, 2, S, n)
    before = t.tensor.clone()
    src, dst = torch.full((S,), -1, dtype=torch.int32), torch.full((S,), -1, dtype=torch.int32)
    src[::3], dst[::3] = torch.arange(0, 2000, dtype=torch.int32), torch.arange(4000, 6000, dtype=torch.int32)
    cuda_lib.check(cuda_lib.kda_slots_copy(pool, S, src.cuda(), dst.cuda(), None))
    torch.cuda.synchronize()
    assert torch.equal(t.tensor, _copied(before, S, n, [(i, 4000 + i) for i in range(2000)])) and t.intact()


def test_slots_zero(cuda_lib):
    n, S = 4104, 7
    t, pool = _pool(cuda_lib, 3, S, n, dtype=torch.bfloat16, gap=8)
    want, status = t.tensor.clone(), _i32(0)
    for s in (6, 2):
        want[:, s * n:(s + 1) * n] = 0
    cuda_lib.check(cuda_lib.kda_slots_zero(pool, 4, _i32(6, -1, 2, 6), status))
    torch.cuda.synchronize()
    assert torch.equal(t.tensor, want) and t.intact() and int(status) == 0
    cuda_lib.check(cuda_lib.kda_slots_zero(pool, 1, _i32(7), status))
    torch.cuda.synchronize()
    assert torch.equal(t.tensor, want) and int(status) == cuda_lib.KDA_DEV_BAD_SLOT


@pytest.mark.parametrize("S", [1, 2, 31, 257, 1024, 1025, 5000])
@pytest.mark.parametrize("share", [0.0, 0.1, 0.6, 1.0])
def test_compact(cuda_lib, S, share):
    """Plan and copy: the live slots end up below their count, each where remap says."""
    r = np.random.default_rng(S)
    live = r.random(S) < share
    t, pool = _pool(cuda_lib, 2, S, 4)
    before = t.tensor.clone()
    src, dst, remap = (Guarded((S,), torch.int32, "cuda") for _ in range(3))
    lv = torch.from_numpy(live.astype(np.int32) * 5).cuda()
    cuda_lib.check(cuda_lib.kda_slots_compact_plan(pool, lv, src.tensor, dst.tensor, remap.tensor))
    cuda_lib.check(cuda_lib.kda_slots_copy(pool, S, src.tensor, dst.tensor, None))
    torch.cuda.synchronize()
    moves, want = P.compact_plan(live)
    pad = [-1] * (S - len(moves))
    assert src.tensor.tolist() == [m[0] for m in moves] + pad and dst.tensor.tolist() == [m[1] for m in moves] + pad
    assert remap.tensor.tolist() == want
    assert torch.equal(t.tensor, _copied(before, S, 4, moves))
    assert all(x.intact() for x in (t, src, dst, remap))


def test_layer_as_served(cuda_lib):
    """The operators one after another as a layer runs them: norm, conv, rule, head norm with gate, residual;
    a prompt, a fork of its states, then a different next token on each branch."""
    r = np.random.default_rng(2)
    bf = torch.bfloat16
    Hk, Hv, d, D, T, K = 2, 4, 64, 256, 75, 4
    C = 2 * Hk * d + Hv * d
    t = lambda *s, sd=1.0: torch.from_numpy(r.standard_normal(s) * sd).cuda()  # noqa: E731
    W, Wo = t(C + Hv * d + 2 * Hv, D, sd=D ** -0.5).to(bf), t(D, Hv * d, sd=(Hv * d) ** -0.5).to(bf)
    conv_w, A_log, dt = t(C, K, sd=0.5).float(), t(Hv, sd=0.3).float(), t(Hv).float() - 3
    resid = t(T + 2, D).to(bf)   # the prompt's rows, then the two branches' next rows
    S = 3
    conv_state, rec = torch.zeros(S, K - 1, C, dtype=bf, device="cuda"), torch.zeros(S, Hv, d, d, device="cuda")
    kda = cuda_lib
    status = _i32(0)

    def layer(x, cu, slots):
        n = x.shape[0]
        p_in = kda.NormParams(dim=D, post_norm=False, res_dtype=kda.KDA_DTYPE_BF16)
        xin = torch.empty_like(x)
        kda.check(kda.kda_block_norm(p_in, n, x, None, None, None, xin))
        proj = xin @ W.t()
        qkv, z, a, b = (y.contiguous() for y in proj.split([C, Hv * d, Hv, Hv], 1))
        cp = kda.ConvParams(channels=C, conv_kernel=K, conv_weight=conv_w, num_slots=S)
        gp = kda.GdnParams(Hk, Hv, d, d, A_log, dt, scale=d ** -0.5, num_slots=S, q_row_stride=C, k_row_stride=C, v_row_stride=C)
        y, o = torch.empty_like(qkv), torch.empty(n, Hv, d, dtype=bf, device="cuda")
        q, k, v = y[:, :Hk * d], y[:, Hk * d:2 * Hk * d], y[:, 2 * Hk * d:]
        if cu is None:
            kda.check(kda.kda_conv_decode(cp, n, qkv, slots, conv_state, y, status))
            kda.check(kda.kda_gdn_decode(gp, n, q, k, v, a, b, slots, rec, o, status))
        else:
            kda.check(kda.kda_conv_varlen(cp, cu, 1, n, qkv, slots, conv_state, y, status))
            need = kda.kda_gdn_prefill_workspace_bytes(gp, 1, n)
            ws = torch.empty(max(16, need), dtype=torch.uint8, device="cuda")
            kda.check(kda.kda_gdn_prefill_varlen(gp, cu, 1, n, q, k, v, a, b, slots, rec, o, ws, need, status))
        hn = kda.NormParams(dim=d, gate_act=kda.KDA_NORM_GATE_SILU)
        kda.check(kda.kda_block_norm(hn, n * Hv, o, z, None, o))
        yo = o.reshape(n, -1) @ Wo.t()
        rp = kda.NormParams(dim=D, post_norm=True, residual_scale=0.5)
        h = torch.empty_like(x)
        kda.check(kda.kda_block_norm(rp, n, yo, None, x, h))
        torch.cuda.synchronize()
        return h

    first = layer(resid[:T].contiguous(), _i32(0, T), _i32(1))
    for tensor, per in ((conv_state, (K - 1) * C * 2), (rec, Hv * d * d * 4)):
        pool = kda.SlotPool(pool=tensor, num_layers=1, num_slots=S, slot_bytes=per, layer_stride_bytes=S * per)
        kda.check(kda.kda_slots_copy(pool, 1, _i32(1), _i32(2), status))
    branch = layer(resid[T:].contiguous(), None, _i32(1, 2))
    assert int(status) == 0

    # the same in 64 bits, all rows of a branch in one go
    f = lambda x: x.double().cpu().numpy()  # noqa: E731
    for i in range(2):
        x = np.concatenate([f(resid[:T]), f(resid[T + i:T + i + 1])])
        xin = x / np.sqrt((x * x).mean(-1, keepdims=True) + 1e-6)
        qkv, z, a, b = np.split(xin @ f(W).T, np.cumsum([C, Hv * d, Hv]), 1)
        y, _ = P.conv([T + 1], qkv, f(conv_w), np.zeros((1, K - 1, C)), [0])
        q, k, v = np.split(y, [Hk * d, 2 * Hk * d], 1)
        o, _ = P.gdn([T + 1], q.reshape(-1, Hk, d), k.reshape(-1, Hk, d), v.reshape(-1, Hv, d), a, b, f(A_log), f(dt),
                     np.zeros((1, Hv, d, d)), [0], d ** -0.5)
        on, _ = P.block_norm(o, z.reshape(-1, Hv, d), 2, None, 1.0, True, 1.0, 1.0, 1e-6)
        h, _ = P.block_norm(on.reshape(T + 1, -1) @ f(Wo).T, None, 0, x, 0.5, True, 1.0, 1.0, 1e-6)
        # seven bf16 roundings in a row on the way to h, of which the branch is about a third of h
        assert P.rel(f(first), h[:T]) <= 7 * 2.0 ** -8
        assert P.rel(f(branch[i]), h[T]) <= 7 * 2.0 ** -8


def test_conv_thousands_of_sequences(cuda_lib):
    lens = np.random.default_rng(2).integers(0, 40, 2500)
    c = Conv(lens.tolist(), 16, 3, "f32", 6, slots=np.random.default_rng(3).permutation(2500).tolist())
    c.run(cuda_lib)
    c.check()


def _conv64(c):
    """The definition in 64 bits on the GPU, for cases that take too long on the host."""
    x, w, state = c.x.double(), c.w.double(), c.state0.double()
    y, t = torch.full_like(x, float("nan")), 0
    for ln, s in zip(c.lens, c.slots_h):
        if s >= 0 and ln:
            full = torch.cat([state[s], x[t:t + ln]])
            acc = sum(full[j:j + ln] * w[:, j] for j in range(c.K))
            y[t:t + ln] = acc * torch.sigmoid(acc)
            state[s] = full[ln:]
        t += ln
    return y, state


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("K", [2, 3, 4])
def test_conv_long_tiles(cuda_lib, K, io):
    """Enough rows for tiles of 128: lengths around a tile's and around its batches of eight rows, every row by
    itself, and the bits of the same rows in calls that are too short for such tiles."""
    lens = [6000, 127, 128, 129, 0, 255, 257, 1, 130, 5000, 137, 12, 4999, 2900]
    slots = [3, 0, 7, 5, 1, 2, 4, 6, -1, 9, 8, 11, 10, 12]
    c = Conv(lens, 4104, K, io, 50 + K, slots=slots, num_slots=14)
    cols, sms = -(-c.C // 512), torch.cuda.get_device_properties(0).multi_processor_count
    assert c.T // 128 * cols >= 8 * sms
    c.run(cuda_lib)
    y, st = _conv64(c)
    got, real = c.y.tensor.double(), ~y[:, 0].isnan()
    # a row's values may all be small: half a step of its own, or of a hundredth of the RMS row
    err, ref = (got - y)[real].norm(dim=1), y[real].norm(dim=1)
    assert (err <= TOL[io] * ref.clamp(min=float(ref.square().mean().sqrt()) / 100)).all()
    assert (got[~real] == 7.0).all()
    assert torch.equal(c.state.tensor.double(), st)
    assert int(c.status) == 0 and c.y.intact() and c.state.intact()
    # the same in calls of a few sequences, long ones in two pieces
    want_y, want_state = c.y.tensor.clone(), c.state.tensor.clone()
    c.state.tensor.copy_(c.state0)
    c.y.tensor.fill_(7.0)
    t = 0
    for ln, s in zip(lens, slots):
        for n in ([ln // 2, ln - ln // 2] if ln > 3000 else [ln]):
            assert n // 128 * cols < 8 * sms
            cuda_lib.check(cuda_lib.kda_conv_varlen(c.params(cuda_lib), _i32(0, n), 1, n, c.x[t:], _i32(s), c.state.tensor,
                                                    c.y.tensor[t:], c.status))
            t += n
    torch.cuda.synchronize()
    assert torch.equal(c.y.tensor, want_y) and torch.equal(c.state.tensor, want_state)


def test_conv_rows_behind_the_last_sequence(cuda_lib):
    c = Conv([40, 3, 70], 64, 4, "bf16", 7)
    cuda_lib.check(cuda_lib.kda_conv_varlen(c.params(cuda_lib), c.cu, 2, c.T, c.x, None, c.state.tensor, c.y.tensor, c.status))
    torch.cuda.synchronize()
    y, _ = P.conv(c.lens, _f(c.x), _f(c.w), _f(c.state0), c.slots_h)
    assert P.rel(_f(c.y.tensor[:43]), y[:43]) <= TOL["bf16"] and (c.y.tensor[43:] == 7.0).all()
    assert torch.equal(c.state.tensor[2], c.state0[2]) and int(c.status) == 0


def test_largest_pool(cuda_lib):
    """As many slots as a pool may have: copy, zero, and the plan and moves of a compaction."""
    S, n = cuda_lib.KDA_MAX_POOL_SLOTS, 4
    t, pool = _pool(cuda_lib, 2, S, n)
    before, status = t.tensor.clone(), _i32(0)
    cuda_lib.check(cuda_lib.kda_slots_copy(pool, 5, _i32(S - 1, S - 1, S, 0, 7), _i32(S - 2, 1, 3, S - 3, S - 4), status))
    cuda_lib.check(cuda_lib.kda_slots_zero(pool, 2, _i32(S - 1, S - 5), status))
    torch.cuda.synchronize()
    want = _copied(before, S, n, [(S - 1, S - 2), (S - 1, 1), (0, S - 3), (7, S - 4)])
    for s in (S - 1, S - 5):
        want[:, s * n:(s + 1) * n] = 0
    assert torch.equal(t.tensor, want) and t.intact() and int(status) == cuda_lib.KDA_DEV_BAD_SLOT
    live = np.random.default_rng(9).random(S) < 0.4
    src, dst, remap = (Guarded((S,), torch.int32, "cuda") for _ in range(3))
    lv = torch.from_numpy(live.astype(np.int32)).cuda()
    cuda_lib.check(cuda_lib.kda_slots_compact_plan(pool, lv, src.tensor, dst.tensor, remap.tensor))
    cuda_lib.check(cuda_lib.kda_slots_copy(pool, S, src.tensor, dst.tensor, None))
    torch.cuda.synchronize()
    moves, where = P.compact_plan(live)
    assert remap.tensor.tolist() == where and src.tensor[:len(moves)].tolist() == [m[0] for m in moves]
    m = torch.tensor(moves, device="cuda")
    got = want.view(2, S, n).clone()
    got[:, m[:, 1]] = want.view(2, S, n)[:, m[:, 0]]
    assert torch.equal(t.tensor, got.view(2, S * n)) and all(x.intact() for x in (t, src, dst, remap))


def test_layer_captured(cuda_lib):
    """A layer's calls one behind the other in a captured graph (kernels that may start early, a memory set and a
    grid of all SMs between them): replayed twice, the eager calls' bits."""
    r = np.random.default_rng(12)
    bf = torch.bfloat16
    Hk, Hv, d, K, N = 4, 16, 64, 4, 2
    C, lens = (2 * Hk + Hv) * d, [1500, 700]
    T = sum(lens)
    t = lambda *s, sd=1.0: torch.from_numpy(r.standard_normal(s) * sd).cuda()  # noqa: E731
    x, z, a, b = t(T, C).to(bf), t(T, Hv * d).to(bf), t(T, Hv).to(bf), t(T, Hv).to(bf)
    conv_w, A_log, dt = t(C, K, sd=0.5).float(), t(Hv, sd=0.3).float(), t(Hv).float() - 3
    S = 4
    conv0, rec0 = t(S, K - 1, C).to(bf), t(S, Hv, d, d, sd=0.1).float()
    conv_state, rec, xn, y = conv0.clone(), rec0.clone(), torch.empty_like(x), torch.empty_like(x)
    o, on = (torch.empty(T, Hv, d, dtype=bf, device="cuda") for _ in range(2))
    cu, slots, status = _i32(0, lens[0], T), _i32(2, 0), _i32(0)
    kda = cuda_lib
    cp = kda.ConvParams(channels=C, conv_kernel=K, conv_weight=conv_w, num_slots=S)
    gp = kda.GdnParams(Hk, Hv, d, d, A_log, dt, scale=d ** -0.5, num_slots=S, q_row_stride=C, k_row_stride=C, v_row_stride=C)
    need = kda.kda_gdn_prefill_workspace_bytes(gp, N, T)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    pools = [kda.SlotPool(pool=p, num_layers=1, num_slots=S, slot_bytes=n, layer_stride_bytes=S * n)
             for p, n in ((conv_state, (K - 1) * C * 2), (rec, Hv * d * d * 4))]
    src, dst, gone, next_rows = _i32(2, 0), _i32(1, 3), _i32(2), _i32(1, 3)
    assert (T // 64 + N) * Hv > 3 * torch.cuda.get_device_properties(0).multi_processor_count

    def calls():
        kda.check(kda.kda_block_norm(kda.NormParams(dim=C, post_norm=False), T, x, None, None, None, xn))
        kda.check(kda.kda_conv_varlen(cp, cu, N, T, xn, slots, conv_state, y, status))
        q, k, v = y[:, :Hk * d], y[:, Hk * d:2 * Hk * d], y[:, 2 * Hk * d:]
        kda.check(kda.kda_gdn_prefill_varlen(gp, cu, N, T, q, k, v, a, b, slots, rec, o, ws, need, status))
        kda.check(kda.kda_block_norm(kda.NormParams(dim=d, gate_act=kda.KDA_NORM_GATE_SILU), T * Hv, o, z, None, None, on))
        for p in pools:  # fork both sequences, free one, then a token of the copies
            kda.check(kda.kda_slots_copy(p, 2, src, dst, status))
            kda.check(kda.kda_slots_zero(p, 1, gone, status))
        kda.check(kda.kda_conv_decode(cp, N, xn, next_rows, conv_state, y, status))
        kda.check(kda.kda_gdn_decode(gp, N, q, k, v, a, b, next_rows, rec, o, status))

    outs = (xn, y, o, on, conv_state, rec)

    def reset():
        conv_state.copy_(conv0)
        rec.copy_(rec0)
        for buf in (xn, y, o, on):
            buf.fill_(7.0)

    reset()
    calls()
    torch.cuda.synchronize()
    want = [buf.clone() for buf in outs]
    assert int(status) == 0 and all(w.isfinite().all() for w in want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    for _ in range(2):
        reset()
        graph.replay()
        torch.cuda.synchronize()
        for got, w in zip(outs, want):
            assert torch.equal(got, w)


@pytest.mark.parametrize("D", [24, 512, 16384])
@pytest.mark.parametrize("e", [56, -50])
def test_block_norm_ends_of_the_range(cuda_lib, D, e):
    """The largest and smallest values whose squares the sums hold, in every place and in one alone, without eps."""
    y = torch.zeros(3, D, device="cuda")
    y[0] = 2.0 ** e
    y[1, D - 1] = -2.0 ** e
    y[2] = torch.ldexp(torch.rand(D, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda") + 0.5, torch.tensor(e - 1))
    F32 = cuda_lib.KDA_DTYPE_F32
    h, x = torch.empty_like(y), torch.empty_like(y)
    p = cuda_lib.NormParams(dim=D, norm_eps=0.0, io_dtype=F32, res_dtype=F32)
    cuda_lib.check(cuda_lib.kda_block_norm(p, 3, y, None, None, h, x))
    torch.cuda.synchronize()
    eh, ex = P.block_norm(_f(y), None, 0, None, 1.0, True, 1.0, 1.0, 0.0)
    for r in range(3):
        assert P.rel(_f(h[r]), eh[r]) <= TOL["f32"] and P.rel(_f(x[r]), ex[r]) <= TOL["f32"]
