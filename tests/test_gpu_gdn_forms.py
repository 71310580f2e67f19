"""The chunked one-decay prefill's forms (chains beside prep in one grid, or one
after the other; one or two value heads a team; each width and output type), with
every row of every head held to a bound of its own.

Bounds of a (row, head): half a bf16 step (2^-8 of the row) where outputs are
bf16, plus 2^-14 of the RMS row: the 2^-18 of an average row (tests/test_gpu_gdn.py)
times 16 for the worst of up to a few hundred thousand rows, small ones among them.
"""
import numpy as np
import pytest
import torch

from tests import plain64 as P
from tests.test_gpu_gdn import Case

pytestmark = pytest.mark.gpu

PREP_CTAS, MERGED = 3, 64  # teams of prep an SM holds; the most sequences of one grid


def beside(c):
    """Whether a call of this case runs its chains beside prep: up to 64 sequences, more slots than one wave of prep."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    return c.N <= MERGED and (c.T // 64 + c.N) * c.Hv > PREP_CTAS * sms


def check_rows(c, status=0):
    """Case.check, and every (row, head) by itself."""
    c.check(status=status)
    out, _ = c.want()
    got = c.g_out.tensor[:c.T].double().cpu().numpy()
    err, ref = np.linalg.norm(got - out, axis=-1), np.linalg.norm(out, axis=-1)
    m = ~np.isnan(ref)
    rms = np.sqrt((ref[m] ** 2).mean())
    over = err[m] - (2.0 ** -8 if c.out_t == "bf16" else 0.0) * ref[m] - 2.0 ** -14 * rms
    assert (over <= 0).all(), f"{(over > 0).sum()} of {m.sum()} rows off, the worst by {err[m][over.argmax()] / rms:.3g} of the RMS row"


@pytest.mark.parametrize("Hk,Hv,dk,dv,out,lens", [
    (4, 16, 128, 128, "f32", [1100, 64, 65, 900]),
    (4, 16, 128, 128, "bf16", [1100, 64, 65, 900]),
    (8, 8, 128, 128, "f32", [2600, 1300]),
    (8, 8, 128, 128, "bf16", [2600, 1300]),
    (3, 9, 128, 64, "f32", [1700, 1, 2000]),
    (3, 9, 128, 64, "bf16", [1700, 1, 2000]),
    (8, 16, 128, 32, "f32", [1900, 130]),
    (5, 15, 128, 32, "bf16", [1000, 1200]),
    (2, 16, 64, 128, "f32", [700, 0, 1300, 130]),
    (4, 16, 64, 32, "bf16", [1000, 500, 600]),
    (8, 8, 64, 32, "f32", [3000, 900]),
    (2, 8, 32, 64, "f32", [0, 3500, 1, 700, 0, 130]),
    (6, 18, 32, 32, "f32", [1500, 400]),
])
def test_chains_beside_prep(cuda_lib, Hk, Hv, dk, dv, out, lens):
    slots = list(range(len(lens)))
    if len(lens) > 3:
        slots[3] = -1  # a padded sequence among them
    c = Case(lens, Hk=Hk, Hv=Hv, dk=dk, dv=dv, out=out, seed=140 + dk + dv, slots=slots)
    assert beside(c)
    c.prefill(cuda_lib)
    check_rows(c)


@pytest.mark.parametrize("Hk,Hv,dk,dv,out", [
    (4, 16, 128, 128, "f32"), (2, 8, 128, 128, "bf16"), (4, 4, 128, 64, "f32"), (3, 9, 64, 64, "f32"), (2, 8, 32, 128, "bf16")])
@pytest.mark.parametrize("ones", [3, 70])
def test_one_after_the_other(cuda_lib, Hk, Hv, dk, dv, out, ones):
    """Few slots, or more sequences than one grid takes; one and two heads a team."""
    c = Case([200, 0, 65, 333] + [1] * ones, Hk=Hk, Hv=Hv, dk=dk, dv=dv, out=out, seed=150 + dk,
             slots=[3, 0, -1, 1] + list(range(4, 4 + ones)))
    assert not beside(c)
    c.prefill(cuda_lib)
    check_rows(c)


@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_many_chains_for_each_cta(cuda_lib, out):
    r = np.random.default_rng(5)
    c = Case(r.integers(0, 200, 64).tolist(), Hk=4, Hv=32, dk=32, dv=32, out=out, seed=81, num_slots=70,
             slots=[int(s) if i % 9 else -1 for i, s in enumerate(r.permutation(70)[:64])])
    assert beside(c)
    c.prefill(cuda_lib)
    check_rows(c)


@pytest.mark.parametrize("N", [33, 300, 1100])
def test_rows_of_many_sequences(cuda_lib, N):
    lens = np.random.default_rng(N).integers(0, 6, N)
    lens[N // 2] = 140
    c = Case(lens.tolist(), Hk=1, Hv=2, dk=64, dv=32, seed=91, slots=np.random.default_rng(1).permutation(N).tolist())
    c.prefill(cuda_lib)
    check_rows(c)


def test_the_rows_bound_sees_one_wrong_row():
    """The bound on rows fails for one wrong row of one head in a case of this size, where the 2-norm passes."""
    r = np.random.default_rng(0)
    out = r.standard_normal((6400, 32, 32))
    got = out.copy()
    got[77, 3] = -got[77, 3]
    assert P.rel(got, out) < 2.0 ** -8 + 2.0 ** -10
    err, ref = np.linalg.norm(got - out, axis=-1), np.linalg.norm(out, axis=-1)
    assert (err > 2.0 ** -8 * ref + 2.0 ** -14 * np.sqrt((ref ** 2).mean())).sum() == 1


@pytest.mark.parametrize("N", [129, 300])
def test_fp32_rows_of_many_sequences(cuda_lib, N):
    """More sequences than are put in order by their lengths."""
    lens = np.random.default_rng(N).integers(0, 6, N)
    lens[N // 2] = 140
    c = Case(lens.tolist(), Hk=1, Hv=2, dk=64, dv=32, io="f32", out="f32", seed=92, slots=np.random.default_rng(2).permutation(N).tolist())
    c.prefill(cuda_lib)
    check_rows(c)


@pytest.mark.parametrize("io,Hv,first", [("bf16", 2, 70), ("bf16", 16, 2600), ("f32", 2, 70)])
def test_rows_behind_the_last_sequence(cuda_lib, io, Hv, first):
    """A call over more rows than its sequences have: the rows behind them, and everyone else's state, stay."""
    c = Case([first, 30, 41], Hk=2, Hv=Hv, dk=64, dv=32, io=io, out="f32", seed=160)
    c.N = 2
    assert beside(c) == (Hv == 16)
    p = c.params(cuda_lib)
    need = cuda_lib.kda_gdn_prefill_workspace_bytes(p, 2, c.T)
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
    cuda_lib.check(cuda_lib.kda_gdn_prefill_varlen(p, c.cu, 2, c.T, c.q, c.k, c.v, c.a, c.b, None, c.g_state.tensor,
                                                   c.g_out.tensor, ws, need, c.status))
    torch.cuda.synchronize()
    out, _ = c.want()
    n = first + 30
    assert (c.g_out.tensor[n:] == 7.0).all() and torch.equal(c.g_state.tensor[2], c.state0[2])
    assert P.rel(c.g_out.tensor[:n].double().cpu().numpy(), out[:n]) <= 2.0 ** -18 and int(c.status.item()) == 0
