"""Offsets past 32 bits: tensors of more than 2^31 values, whose far ends are held
to the bits of a small call on the same values (the arithmetic of a sequence does not
depend on where it lies)."""
import pytest
import torch

from tests.test_gpu_gdn import Case

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.fixture(autouse=True)
def _free():
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("call", ["prefill", "prefill_f32", "decode"])
def test_states_of_a_large_pool(cuda_lib, call):
    io = "f32" if call == "prefill_f32" else "bf16"
    lens = [1, 1] if call == "decode" else [130, 20]
    small = Case(lens, Hk=16, Hv=32, io=io, out="f32", seed=1)
    run = lambda c: c.decode(cuda_lib) if call == "decode" else c.prefill(cuda_lib)  # noqa: E731
    run(small)
    S = (1 << 31) // small.state0[0].numel() + 3
    far = Case(lens, Hk=16, Hv=32, io=io, out="f32", seed=1)
    pool = torch.zeros(S, *small.state0.shape[1:], device="cuda")
    at = [S - 1, S // 2]
    pool[at] = small.state0
    far.num_slots, far.slots = S, torch.tensor(at, dtype=torch.int32, device="cuda")
    far.g_state.tensor = pool
    run(far)
    assert torch.equal(far.g_out.tensor, small.g_out.tensor)
    assert torch.equal(pool[at], small.g_state.tensor)
    pool[at] = 0
    assert not pool.any() and int(far.status.item()) == 0


def test_prefill_of_many_rows(cuda_lib):
    """A prompt behind more than 2^31 values of others: its rows, its outputs and its chunks' places in the workspace."""
    Hk, Hv, d = 2, 32, 128
    tail = 333
    T = (1 << 31) // (Hv * d) + 64 * 40 + 17 + tail
    g = torch.Generator(device="cuda").manual_seed(2)
    rows = torch.empty(T, (2 * Hk + Hv) * d, dtype=BF, device="cuda").normal_(generator=g)
    a, b = (torch.empty(T, Hv, dtype=BF, device="cuda").normal_(generator=g) for _ in range(2))
    A_log, dt = torch.zeros(Hv, device="cuda"), torch.full((Hv,), -3.0, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def run(r0, lens):
        n, N = sum(lens), len(lens)
        x = rows[r0:r0 + n]
        q, k, v = x[:, :Hk * d], x[:, Hk * d:2 * Hk * d], x[:, 2 * Hk * d:]
        p = cuda_lib.GdnParams(Hk, Hv, d, d, A_log, dt, scale=d ** -0.5, num_slots=N, q_row_stride=x.shape[1],
                               k_row_stride=x.shape[1], v_row_stride=x.shape[1])
        state, out = torch.zeros(N, Hv, d, d, device="cuda"), torch.empty(n, Hv, d, dtype=BF, device="cuda")
        need = cuda_lib.kda_gdn_prefill_workspace_bytes(p, N, n)
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        cu = torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist(), dtype=torch.int32, device="cuda")
        cuda_lib.check(cuda_lib.kda_gdn_prefill_varlen(p, cu, N, n, q, k, v, a[r0:r0 + n].clone(), b[r0:r0 + n].clone(), None,
                                                       state, out, ws, need, status))
        torch.cuda.synchronize()
        return out, state

    cut = (T - tail) // 8
    lens = [cut] * 7 + [T - tail - 7 * cut, tail]
    out, state = run(0, lens)
    alone, last = run(T - tail, [tail])
    assert torch.equal(out[T - tail:], alone) and torch.equal(state[-1], last[0]) and int(status) == 0
    assert out.isfinite().all()


def test_conv_of_many_rows(cuda_lib):
    C, K, tail = 4608, 4, 333
    T = (1 << 31) // C + 1000 + tail
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.empty(T, C, dtype=BF, device="cuda").normal_(generator=g)
    w = torch.randn(C, K, generator=g, device="cuda")

    def run(r0, lens):
        st, y = torch.zeros(len(lens), K - 1, C, dtype=BF, device="cuda"), torch.empty(sum(lens), C, dtype=BF, device="cuda")
        cu = torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist(), dtype=torch.int32, device="cuda")
        p = cuda_lib.ConvParams(channels=C, conv_kernel=K, conv_weight=w, num_slots=len(lens))
        cuda_lib.check(cuda_lib.kda_conv_varlen(p, cu, len(lens), sum(lens), x[r0:], None, st, y, None))
        torch.cuda.synchronize()
        return y, st

    y, st = run(0, [T - tail, tail])
    alone, last = run(T - tail, [tail])
    assert torch.equal(y[T - tail:], alone) and torch.equal(st[1], last[0]) and torch.equal(st[0], x[T - tail - 3:T - tail])
    # a far slot of a large pool, one row
    S = (1 << 31) // ((K - 1) * C) + 5
    pool = torch.zeros(S, K - 1, C, dtype=BF, device="cuda")
    pool[S - 1] = last[0]
    p = cuda_lib.ConvParams(channels=C, conv_kernel=K, conv_weight=w, num_slots=S)
    one, far = torch.empty(1, C, dtype=BF, device="cuda"), torch.empty(1, C, dtype=BF, device="cuda")
    small = cuda_lib.ConvParams(channels=C, conv_kernel=K, conv_weight=w, num_slots=1)
    slot = torch.tensor([S - 1], dtype=torch.int32, device="cuda")
    cuda_lib.check(cuda_lib.kda_conv_decode(p, 1, x, slot, pool, far, None))
    cuda_lib.check(cuda_lib.kda_conv_decode(small, 1, x, None, last, one, None))
    torch.cuda.synchronize()
    assert torch.equal(far, one) and torch.equal(pool[S - 1], last[0]) and not pool[:S - 1].any()


@pytest.mark.parametrize("D", [128, 16384])
def test_norm_of_many_rows(cuda_lib, D):
    rows = (1 << 31) // D + 77
    g = torch.Generator(device="cuda").manual_seed(4)
    y, gate = (torch.empty(rows, D, dtype=BF, device="cuda").normal_(generator=g) for _ in range(2))
    p = cuda_lib.NormParams(dim=D, gate_act=cuda_lib.KDA_NORM_GATE_SILU)
    x, few = torch.empty_like(y), torch.empty(99, D, dtype=BF, device="cuda")
    cuda_lib.check(cuda_lib.kda_block_norm(p, rows, y, gate, None, None, x))
    cuda_lib.check(cuda_lib.kda_block_norm(p, 99, y[rows - 99:].clone(), gate[rows - 99:].clone(), None, None, few))
    torch.cuda.synchronize()
    assert torch.equal(x[rows - 99:], few)


def test_slots_far_apart(cuda_lib):
    """A pool of 9 GB over two layers: a fork and a zeroing at both its ends."""
    S, per, layers = 70, 1 << 26, 2  # bytes of a slot
    pool = torch.zeros(layers, S, per // 4, device="cuda")
    pool[:, 3] = torch.randn(layers, per // 4, generator=torch.Generator(device="cuda").manual_seed(5), device="cuda")
    pool[:, S - 1] = 5.0
    desc = cuda_lib.SlotPool(pool=pool, num_layers=layers, num_slots=S, slot_bytes=per, layer_stride_bytes=S * per)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    cuda_lib.check(cuda_lib.kda_slots_copy(desc, 2, i32(3, 3), i32(S - 2, 0), None))
    cuda_lib.check(cuda_lib.kda_slots_zero(desc, 1, i32(S - 1), None))
    torch.cuda.synchronize()
    for s in (0, S - 2):
        assert torch.equal(pool[:, s], pool[:, 3])
    pool[:, [0, 3, S - 2]] = 0
    assert not pool.any()
