"""The gated delta rule with one decay per head, and the operators around it: measured cases.

Each operator is there twice: in its plain form (elementary torch operations in 32 bits, 64 for the
decays' running sums) and, where ``own`` is true, as the calls a program makes of the library.

  gdn_prefill  the chunked rule over prompt rows of variable-length sequences
  gdn_decode   the rule's single-token form on slot-indexed states
  conv         the causal depthwise convolution with carried state and SiLU in front of the rule
  norm         the norms around a block: after it (with its gate), the scaled residual, before the next
  slots        forking, compacting and freeing the slots of state pools
"""
import math
import random

import torch

own = False

DEV = "cuda"
C = 64  # rows of a chunk in the plain form
L2_EPS = 1e-6
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one user's next token: launch and latency
        dict(name="decode_b1", op="gdn_decode", B=1, Hk=16, Hv=32, dk=128, dv=128, io="bf16", out="bf16", skip=0),
        # a full serving batch, two of its places padded: the states' bandwidth
        dict(name="decode_b250", op="gdn_decode", B=250, Hk=16, Hv=32, dk=128, dv=128, io="bf16", out="bf16", skip=2),
        # a few short prompts, one of a single token and one empty
        dict(name="prefill_short", op="gdn_prefill", N=4, T=333, cut=5, Hk=4, Hv=8, dk=128, dv=128, io="bf16", out="bf16", skip=0),
        # a batch of prompts of mixed lengths
        dict(name="prefill_n8", op="gdn_prefill", N=8, T=32768, cut=1, Hk=16, Hv=32, dk=128, dv=128, io="bf16", out="bf16", skip=0),
        # one long prompt: few chains, long ones
        dict(name="prefill_long", op="gdn_prefill", N=1, T=32768, cut=0, Hk=16, Hv=32, dk=128, dv=128, io="bf16", out="bf16", skip=0),
        # a smaller model: heads of 64, as many key heads as value heads, outputs in fp32
        dict(name="prefill_d64", op="gdn_prefill", N=5, T=7001, cut=3, Hk=12, Hv=12, dk=64, dv=64, io="bf16", out="f32", skip=1),
        # q|k|v channels of the batch of prompts
        dict(name="conv_n8", op="conv", N=8, T=32768, cut=1, C=8192, K=4, io="bf16", skip=0),
        # the same channels, one row for each sequence of a serving batch
        dict(name="conv_decode_b64", op="conv_decode", B=64, C=8192, K=4, io="bf16", skip=1),
        # per-head norm of a decode batch's outputs with its SiLU gate
        dict(name="norm_heads", op="norm", rows=64 * 32, D=128, post=True, act="silu", residual=False, pre=False, alpha=1.0, io="bf16", res="bf16"),
        # norm after a block, gate, scaled residual and the next block's norm, prompt rows, fp32 residual stream
        dict(name="norm_block", op="norm", rows=16384, D=4096, post=True, act="sigmoid", residual=True, pre=True, alpha=0.5, io="bf16", res="f32"),
        # one sequence's states in every layer forked to seven others
        dict(name="slots_fork", op="slots", kind="fork", layers=24, slots=40, slot=32 * 128 * 128, n=7, cut=2, io="f32"),
        # the conv states of a pool with holes closed up
        dict(name="slots_compact", op="slots", kind="compact", layers=24, slots=257, slot=3 * 8192, n=150, cut=4, io="bf16"),
    ]


def draw(rng):
    log = lambda a, b: int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))  # noqa: E731
    op = rng.choice(["gdn_prefill", "gdn_prefill", "gdn_decode", "conv", "conv_decode", "norm", "slots"])
    io = rng.choice(["bf16", "bf16", "bf16", "f32"])
    cut = rng.randrange(1, 1 << 20)
    if op in ("gdn_prefill", "gdn_decode"):
        Hk = rng.choice([1, 2, 3, 4, 8, 16])
        Hv = Hk * rng.choice([1, 2, 4] if Hk <= 8 else [1, 2])
        dims = dict(Hk=Hk, Hv=Hv, dk=rng.choice([32, 64, 128, 128]), dv=rng.choice([32, 64, 128, 128]), io=io, out=rng.choice(["bf16", "bf16", "f32"]) if io == "bf16" else "f32")
        if op == "gdn_decode":
            B = log(1, 250)
            return dict(op=op, B=B, skip=rng.randrange(0, 1 + B // 8), **dims)
        T = log(1, 32768 if io == "bf16" else 4096)
        N = rng.randrange(1, 17)
        return dict(op=op, N=N, T=T, cut=cut, skip=rng.randrange(0, 2) if N > 2 else 0, **dims)
    if op == "conv":
        N = rng.randrange(1, 17)
        return dict(op=op, N=N, T=log(1, 32768), cut=cut, C=8 * log(16, 1024 if io == "bf16" else 512), K=rng.choice([2, 3, 4]), io=io, skip=rng.randrange(0, 2) if N > 2 else 0)
    if op == "conv_decode":
        return dict(op=op, B=log(1, 512), C=8 * log(16, 1024), K=rng.choice([2, 3, 4]), io=io, skip=rng.randrange(0, 2))
    if op == "norm":
        D = 8 * log(4, 1024)
        act = rng.choice(["none", "sigmoid", "silu"])
        pre = rng.choice([True, False])
        return dict(op=op, rows=log(1, (1 << 26) // D), D=D, post=rng.choice([True, True, False]) or not pre, act=act, residual=rng.choice([True, False]), pre=pre, alpha=rng.choice([1.0, 0.25]), io=io, res=rng.choice([io, "f32"]))
    kind = rng.choice(["fork", "compact", "free"])
    slots = log(3, 300)
    layers = rng.choice([1, 4, 24])
    slot = 64 * log(4, min(8192, max(5, 700_000_000 // (64 * 4 * layers * slots))))
    return dict(op=op, kind=kind, layers=layers, slots=slots, slot=slot, n=rng.randrange(1, slots - 1), cut=cut, io=io)


def _lens(case):
    """Sequence lengths of a case: N random cuts of T rows (empty sequences happen); cut == 0: one sequence."""
    T, N = case["T"], case["N"]
    r = random.Random(case["cut"])
    ends = sorted(r.randrange(0, T + 1) for _ in range(N - 1)) + [T]
    if case.get("name") == "prefill_short":
        ends = [1, 1, 130, 333]
    return [b - a for a, b in zip([0] + ends, ends)]


# ---------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _randn(g, *shape, dtype=torch.float32, std=1.0):
    return (torch.randn(*shape, generator=g, device=DEV) * std).to(dtype)


def _silu_rows(g, rows, ch, dtype):
    """Rows as they leave a convolution with SiLU: mostly small, skewed to the positive side."""
    x = torch.randn(rows, ch, generator=g, device=DEV)
    return (x * torch.sigmoid(x)).to(dtype)


def _slots_of(g, n, skip):
    """A shuffled slot for each of n sequences out of n + 3, the first `skip` of them negative (padding)."""
    p = torch.randperm(n + 3, generator=g, device=DEV)[:n].to(torch.int32)
    if skip:
        p[:skip] = -1
    return p


def _inputs(case, seed):
    """The case's tensors, made on the GPU from the seed."""
    g = _gen(seed)
    s = {}
    op = case["op"]
    if op in ("gdn_prefill", "gdn_decode"):
        Hk, Hv, dk, dv = case["Hk"], case["Hv"], case["dk"], case["dv"]
        n = case["B"] if op == "gdn_decode" else case["N"]
        T = n if op == "gdn_decode" else case["T"]
        dt = DT[case["io"]]
        # one convolution output holds the q|k|v channels of a row
        rows = _silu_rows(g, T, 2 * Hk * dk + Hv * dv, dt)
        s["rows"] = rows
        s["q"], s["k"], s["v"] = rows[:, :Hk * dk], rows[:, Hk * dk:2 * Hk * dk], rows[:, 2 * Hk * dk:]
        s["gate"] = _randn(g, T, Hv, dtype=dt)
        s["beta"] = _randn(g, T, Hv, dtype=dt)
        # decay rates of 1 .. 16 and time steps of 0.001 .. 0.1, as such layers start out
        s["A_log"] = torch.log(1 + 15 * torch.rand(Hv, generator=g, device=DEV))
        step = torch.exp(math.log(1e-3) + math.log(100.0) * torch.rand(Hv, generator=g, device=DEV))
        s["dt_bias"] = torch.log(torch.expm1(step))
        s["slots"] = _slots_of(g, n, case["skip"])
        s["rec_state"] = _randn(g, n + 3, Hv, dk, dv, std=0.05)
        s["out"] = torch.zeros(T, Hv, dv, dtype=DT[case["out"]], device=DEV)
        if op == "gdn_prefill":
            s["cu_seqlens"] = torch.tensor([0] + _lens(case), device=DEV).cumsum(0).to(torch.int32)
    elif op in ("conv", "conv_decode"):
        n = case["B"] if op == "conv_decode" else case["N"]
        T = n if op == "conv_decode" else case["T"]
        ch, K, dt = case["C"], case["K"], DT[case["io"]]
        s["x"] = _randn(g, T, ch, dtype=dt)
        s["weight"] = _randn(g, ch, K, std=K ** -0.5)
        s["slots"] = _slots_of(g, n, case["skip"])
        s["conv_state"] = _randn(g, n + 3, K - 1, ch, dtype=dt)
        s["y"] = torch.zeros(T, ch, dtype=dt, device=DEV)
        if op == "conv":
            s["cu_seqlens"] = torch.tensor([0] + _lens(case), device=DEV).cumsum(0).to(torch.int32)
    elif op == "norm":
        rows, D, dt, rt = case["rows"], case["D"], DT[case["io"]], DT[case["res"]]
        s["y"] = _randn(g, rows, D, dtype=dt, std=0.5)
        s["gate"] = _randn(g, rows, D, dtype=dt) if case["act"] != "none" else None
        s["residual"] = _randn(g, rows, D, dtype=rt, std=2.0) if case["residual"] else None
        s["post_w"] = 1 + _randn(g, D, std=0.1)
        s["pre_w"] = 1 + _randn(g, D, std=0.1)
        s["h"] = torch.empty(rows, D, dtype=rt, device=DEV)
        s["x"] = torch.empty(rows, D, dtype=dt, device=DEV) if case["pre"] else None
    else:
        L, S, n = case["layers"], case["slots"], case["n"]
        s["pool"] = _randn(g, L, S, case["slot"], dtype=DT[case["io"]])
        r = random.Random(case["cut"])
        order = list(range(S))
        r.shuffle(order)
        if case["kind"] == "fork":  # the first slot's sequence goes to n others
            s["src"] = torch.tensor([order[0]] * n, dtype=torch.int32, device=DEV)
            s["dst"] = torch.tensor(order[1:1 + n], dtype=torch.int32, device=DEV)
        elif case["kind"] == "free":
            s["dst"] = torch.tensor(order[:n], dtype=torch.int32, device=DEV)
        else:  # n live slots, scattered
            s["live"] = torch.zeros(S, dtype=torch.int32, device=DEV)
            s["live"][torch.tensor(order[:n], device=DEV)] = 1
            s["src"] = torch.empty(S, dtype=torch.int32, device=DEV)
            s["dst"] = torch.empty(S, dtype=torch.int32, device=DEV)
            s["remap"] = torch.empty(S, dtype=torch.int32, device=DEV)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if own:
        s["calls"] = _calls(case, s)
    return s


# ---------------------------------------------------------------- the library's calls

def _calls(case, s):
    """The calls of one pass with their arguments marshalled, as a serving loop keeps them."""
    import linear_attention_serving_kda_gb300 as kda

    code = {"bf16": kda.KDA_DTYPE_BF16, "f32": kda.KDA_DTYPE_F32}
    op = case["op"]
    if op in ("gdn_prefill", "gdn_decode"):
        stride = s["rows"].shape[1]
        p = kda.GdnParams(num_heads_k=case["Hk"], num_heads_v=case["Hv"], head_dim_k=case["dk"], head_dim_v=case["dv"],
                          A_log=s["A_log"], dt_bias=s["dt_bias"], l2_norm=True, l2_eps=L2_EPS, scale=case["dk"] ** -0.5,
                          io_dtype=code[case["io"]], out_dtype=code[case["out"]], num_slots=s["rec_state"].shape[0],
                          q_row_stride=stride, k_row_stride=stride, v_row_stride=stride)
        if op == "gdn_decode":
            return [kda.Prepared("kda_gdn_decode", p, case["B"], s["q"], s["k"], s["v"], s["gate"], s["beta"], s["slots"],
                                 s["rec_state"], s["out"], None)]
        need = kda.kda_gdn_prefill_workspace_bytes(p, case["N"], case["T"])
        s["workspace"] = torch.empty(need, dtype=torch.uint8, device=DEV) if need else None
        return [kda.Prepared("kda_gdn_prefill_varlen", p, s["cu_seqlens"], case["N"], case["T"], s["q"], s["k"], s["v"],
                             s["gate"], s["beta"], s["slots"], s["rec_state"], s["out"], s["workspace"], need, None)]
    if op in ("conv", "conv_decode"):
        p = kda.ConvParams(channels=case["C"], conv_kernel=case["K"], conv_weight=s["weight"], io_dtype=code[case["io"]],
                           num_slots=s["conv_state"].shape[0])
        if op == "conv_decode":
            return [kda.Prepared("kda_conv_decode", p, case["B"], s["x"], s["slots"], s["conv_state"], s["y"], None)]
        return [kda.Prepared("kda_conv_varlen", p, s["cu_seqlens"], case["N"], case["T"], s["x"], s["slots"], s["conv_state"],
                             s["y"], None)]
    if op == "norm":
        act = {"none": kda.KDA_NORM_GATE_NONE, "sigmoid": kda.KDA_NORM_GATE_SIGMOID, "silu": kda.KDA_NORM_GATE_SILU}
        p = kda.NormParams(dim=case["D"], post_norm=case["post"], gate_act=act[case["act"]], residual_scale=case["alpha"],
                           norm_eps=1e-6, post_weight=s["post_w"], pre_weight=s["pre_w"], io_dtype=code[case["io"]],
                           res_dtype=code[case["res"]])
        return [kda.Prepared("kda_block_norm", p, case["rows"], s["y"], s["gate"], s["residual"], s["h"], s["x"])]
    size = s["pool"].element_size()
    pool = kda.SlotPool(pool=s["pool"], num_layers=case["layers"], num_slots=case["slots"], slot_bytes=case["slot"] * size,
                        layer_stride_bytes=case["slots"] * case["slot"] * size)
    if case["kind"] == "free":
        return [kda.Prepared("kda_slots_zero", pool, case["n"], s["dst"], None)]
    if case["kind"] == "fork":
        return [kda.Prepared("kda_slots_copy", pool, case["n"], s["src"], s["dst"], None)]
    return [kda.Prepared("kda_slots_compact_plan", pool, s["live"], s["src"], s["dst"], s["remap"]),
            kda.Prepared("kda_slots_copy", pool, case["slots"], s["src"], s["dst"], None)]


def run(s):
    case = s["case"]
    if own:
        for call in s["calls"]:
            if call() != 0:
                raise RuntimeError("the library refused %r" % (case,))
    else:
        PLAIN[case["op"]](case, s)
    return _outputs(case, s)


def _outputs(case, s):
    op = case["op"]
    if op in ("gdn_prefill", "gdn_decode"):
        return {"out": s["out"], "state": s["rec_state"]}
    if op in ("conv", "conv_decode"):
        return {"y": s["y"], "state": s["conv_state"]}
    if op == "norm":
        return {"h": s["h"], "x": s["x"]} if case["pre"] else {"h": s["h"]}
    if case["kind"] == "compact":
        return {"pool": s["pool"], "remap": s["remap"]}
    return {"pool": s["pool"]}


# ---------------------------------------------------------------- plain forms

def _gates(s, dtype):
    """(log decay, beta) of every row and value head."""
    a = s["gate"].to(dtype) + s["dt_bias"].to(dtype)
    soft = torch.clamp(a, min=0) + torch.log1p(torch.exp(-a.abs()))
    return -torch.exp(s["A_log"].to(dtype)) * soft, torch.sigmoid(s["beta"].to(dtype))


def _unit(x, dtype):
    x = x.to(dtype)
    return x * torch.rsqrt((x * x).sum(-1, keepdim=True) + L2_EPS)


def _heads(case, s, dtype):
    """Normalised q, k and plain v rows, a key head's rows repeated for its value heads: [T][Hv][d]."""
    T, Hk, Hv = s["q"].shape[0], case["Hk"], case["Hv"]
    q = _unit(s["q"].reshape(T, Hk, case["dk"]), dtype).repeat_interleave(Hv // Hk, 1)
    k = _unit(s["k"].reshape(T, Hk, case["dk"]), dtype).repeat_interleave(Hv // Hk, 1)
    return q, k, s["v"].reshape(T, Hv, case["dv"]).to(dtype)


def _plain_decode(case, s):
    q, k, v = _heads(case, s, torch.float32)
    g, beta = _gates(s, torch.float32)
    rows = torch.arange(case["skip"], case["B"], device=DEV)  # the padded places come first
    slot = s["slots"][rows].long()
    q, k, v, beta = q[rows], k[rows], v[rows], beta[rows]
    S = s["rec_state"][slot] * torch.exp(g[rows])[..., None, None]
    u = beta[..., None] * (v - (S * k[..., None]).sum(-2))
    S = S + k[..., None] * u[..., None, :]
    s["rec_state"][slot] = S
    s["out"][rows] = ((S * q[..., None]).sum(-2) * case["dk"] ** -0.5).to(s["out"].dtype)


def _unit_lower_inverse(A):
    """(I + A)^-1 for strictly lower A, by doubling the blocks that are already inverted."""
    n = A.shape[-1]
    T = torch.eye(n, device=A.device).expand(A.shape).clone()
    b = 1
    while b < n:  # log2(n) steps, each over all blocks at once
        Tb = T.unflatten(-2, (n // (2 * b), 2, b)).unflatten(-1, (n // (2 * b), 2, b))
        Ab = A.unflatten(-2, (n // (2 * b), 2, b)).unflatten(-1, (n // (2 * b), 2, b))
        i = torch.arange(n // (2 * b), device=A.device)
        top, low = Tb[..., i, 0, :, i, 0, :], Tb[..., i, 1, :, i, 1, :]
        Tb[..., i, 1, :, i, 0, :] = -(low @ (Ab[..., i, 1, :, i, 0, :] @ top))
        b *= 2
    return T


def _plain_prefill(case, s):
    """The rule in chunks of 64 rows: everything within a chunk at once over all chunks, and a loop over
    the chunks' order for the states, which follow one another."""
    lens = _lens(case)
    T, Hv, dk, dv = case["T"], case["Hv"], case["dk"], case["dv"]
    start, chunks, order = 0, [], []
    for n, ln in enumerate(lens):
        if n >= case["skip"]:  # the padded sequences come first
            for c in range(0, ln, C):
                order.append((c // C, n, len(chunks)))
                chunks.append((start + c, min(C, ln - c)))
        start += ln
    if not chunks:
        return
    at = torch.tensor(chunks, device=DEV)
    r = torch.arange(C, device=DEV)
    real = r < at[:, 1:2]                                     # [NC][C]
    idx = torch.where(real, at[:, :1] + r, 0)
    q, k, v = _heads(case, s, torch.float32)
    g, beta = _gates(s, torch.float64)
    pick = lambda x: (x[idx] * real.reshape(real.shape + (1,) * (x.dim() - 1))).transpose(1, 2)  # noqa: E731  [NC][Hv][C]...
    q, k, v, g, beta = pick(q), pick(k), pick(v), pick(g), pick(beta.float())
    G = g.cumsum(-1)
    low = r[:, None] >= r
    decay = torch.where(low, torch.exp(torch.where(low, G[..., :, None] - G[..., None, :], 0)), 0).float()
    A = (k @ k.transpose(-1, -2)) * decay * beta[..., None] * (r[:, None] > r)
    inv = _unit_lower_inverse(A)
    P = (q @ k.transpose(-1, -2)) * decay
    eG = torch.exp(G).float()
    U = inv @ (beta[..., None] * v)
    W = inv @ ((beta * eG)[..., None] * k)
    q = q * eG[..., None]
    k = k * torch.exp(G[..., -1:] - G).float()[..., None]
    last = eG[..., -1]
    O = torch.empty_like(v)
    slot = s["slots"].long()
    S = s["rec_state"]
    order.sort()
    steps = {}
    for c, n, j in order:
        steps.setdefault(c, ([], []))
        steps[c][0].append(n)
        steps[c][1].append(j)
    flat = torch.tensor([x for c in sorted(steps) for x in steps[c][0] + steps[c][1]], device=DEV)
    p = 0
    for c in sorted(steps):
        m = len(steps[c][0])
        sl, j = slot[flat[p:p + m]], flat[p + m:p + 2 * m]
        p += 2 * m
        Sc = S[sl]
        Uc = U[j] - W[j] @ Sc
        O[j] = q[j] @ Sc + P[j] @ Uc
        S[sl] = last[j][..., None, None] * Sc + k[j].transpose(-1, -2) @ Uc
    s["out"][idx[real]] = (O.transpose(1, 2)[real] * dk ** -0.5).to(s["out"].dtype)


def _rows_of(case, s):
    """(sequence, first row) of every row, on the GPU."""
    if case["op"] == "conv_decode":
        n = torch.arange(case["B"], device=DEV)
        return n, n
    cu = s["cu_seqlens"].long()
    n = torch.repeat_interleave(torch.arange(case["N"], device=DEV), cu[1:] - cu[:-1], output_size=case["T"])
    return n, cu[n]


def _conv(case, s, dtype):
    """(outputs, new states, kept rows) of the convolution; rows and states of padded sequences are not kept."""
    K = case["K"]
    n, first = _rows_of(case, s)
    t = torch.arange(n.shape[0], device=DEV)
    slot = s["slots"].long()
    at = slot.clamp(min=0)
    w = s["weight"].to(dtype)
    acc = torch.zeros(s["x"].shape, dtype=dtype, device=DEV)
    for j in range(K):
        back = t - (K - 1 - j)
        hist = s["conv_state"][at[n], (K - 1 + back - first).clamp(0, K - 2)] if K > 1 else None
        acc += w[:, j] * torch.where((back >= first)[:, None], s["x"][back.clamp(min=0)], hist).to(dtype)
    y = acc * torch.sigmoid(acc)
    if case["op"] == "conv_decode":
        lo, ln = t, torch.ones_like(t)
    else:
        cu = s["cu_seqlens"].long()
        lo, ln = cu[:-1], cu[1:] - cu[:-1]
    r = torch.arange(K - 1, device=DEV)
    src = ln[:, None] + r - (K - 1)                            # row of the sequence; negative: old state row
    old = s["conv_state"][at[:, None], (K - 1 + src).clamp(0, K - 2)]
    new = torch.where((src >= 0)[..., None], s["x"][(lo[:, None] + src).clamp(0, max(0, t.shape[0] - 1))], old)
    return y, new, slot, slot[n] >= 0


def _plain_conv(case, s):
    y, new, slot, kept = _conv(case, s, torch.float32)
    k = case["skip"]
    s["y"].copy_(torch.where(kept[:, None], y.to(s["y"].dtype), s["y"]))
    s["conv_state"][slot[k:]] = new[k:]


def _norm(case, s, dtype):
    t = s["y"].to(dtype)
    if case["post"]:
        t = t * torch.rsqrt((t * t).mean(-1, keepdim=True) + 1e-6) * s["post_w"].to(dtype)
    if case["act"] != "none":
        g = s["gate"].to(dtype)
        t = t * torch.sigmoid(g) * (g if case["act"] == "silu" else 1)
    t = t * case["alpha"]
    if case["residual"]:
        t = s["residual"].to(dtype) + t
    x = t * torch.rsqrt((t * t).mean(-1, keepdim=True) + 1e-6) * s["pre_w"].to(dtype) if case["pre"] else None
    return t, x


def _plain_norm(case, s):
    h, x = _norm(case, s, torch.float32)
    s["h"].copy_(h)
    if case["pre"]:
        s["x"].copy_(x)


def _plan(live):
    """Moves that close the holes below the number of live slots: (sources, targets, new place of each slot)."""
    S = live.shape[0]
    live = live != 0
    pos = torch.arange(S, device=live.device)
    n = live.sum()
    hole, mover = ~live & (pos < n), live & (pos >= n)
    put = lambda m: torch.full((S + 1,), -1, device=live.device).scatter_(0, torch.where(m, m.cumsum(0) - 1, S), torch.where(m, pos, -1))[:S]  # noqa: E731
    src, dst = put(mover), put(hole)
    return src, dst, torch.where(mover, dst[(mover.cumsum(0) - 1).clamp(min=0)], torch.where(live, pos, -1))


def _plain_slots(case, s):
    if case["kind"] == "free":
        s["pool"][:, s["dst"].long()] = 0
        return
    if case["kind"] == "compact":
        src, dst, remap = _plan(s["live"])
        s["remap"].copy_(remap)
        move = src >= 0
        src, dst = src[move], dst[move]
    else:
        src, dst = s["src"].long(), s["dst"].long()
    s["pool"][:, dst] = s["pool"][:, src]


PLAIN = {"gdn_prefill": _plain_prefill, "gdn_decode": _plain_decode, "conv": _plain_conv, "conv_decode": _plain_conv,
         "norm": _plain_norm, "slots": _plain_slots}


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    op = case["op"]
    size = {"bf16": 2, "f32": 4}
    io = size[case["io"]]
    if op in ("gdn_prefill", "gdn_decode"):
        Hk, Hv, dk, dv = case["Hk"], case["Hv"], case["dk"], case["dv"]
        if op == "gdn_decode":
            rows = seqs = case["B"] - case["skip"]
        else:
            lens = _lens(case)[case["skip"]:]
            rows, seqs = sum(lens), sum(1 for x in lens if x)
        row = io * (2 * Hk * dk + Hv * dv + 2 * Hv) + size[case["out"]] * Hv * dv
        # decayed read, correction, update and readout of a dk x dv state per row and head
        return {"bytes": rows * row + seqs * Hv * dk * dv * 8 + 8 * Hv, "flops": rows * Hv * 6 * dk * dv + 1}
    if op in ("conv", "conv_decode"):
        ch, K = case["C"], case["K"]
        if op == "conv_decode":
            rows = seqs = case["B"] - case["skip"]
        else:
            lens = _lens(case)[case["skip"]:]
            rows, seqs = sum(lens), sum(1 for x in lens if x)
        return {"bytes": 2 * rows * ch * io + 2 * seqs * (K - 1) * ch * io + ch * K * 4, "flops": rows * ch * (2 * K + 4)}
    if op == "norm":
        n, res = case["rows"] * case["D"], size[case["res"]]
        b = n * (io + (io if case["act"] != "none" else 0) + (res if case["residual"] else 0) + res + (io if case["pre"] else 0))
        return {"bytes": b, "flops": n * 10}
    one = case["layers"] * case["slot"] * io
    if case["kind"] == "fork":
        return {"bytes": one * (1 + case["n"]), "flops": 0}
    if case["kind"] == "free":
        return {"bytes": one * case["n"], "flops": 0}
    r = random.Random(case["cut"])
    order = list(range(case["slots"]))
    r.shuffle(order)
    moves = sum(1 for x in order[:case["n"]] if x >= case["n"])
    return {"bytes": 2 * one * moves + 16 * case["slots"], "flops": 0}


# ---------------------------------------------------------------- in 64 bits, from the definitions

def exact(case, seed):
    s = _inputs(case, seed)
    op = case["op"]
    f8 = torch.float64
    if op in ("gdn_prefill", "gdn_decode"):
        return _exact_rule(case, s)
    if op in ("conv", "conv_decode"):
        return _exact_conv(case, s)
    if op == "norm":
        y = s["y"].to(f8)
        if case["post"]:
            y = s["post_w"].to(f8) * y / ((y ** 2).sum(1, keepdim=True) / case["D"] + 1e-6).sqrt()
        if case["act"] != "none":
            g = s["gate"].to(f8)
            y = y / (1 + torch.exp(-g))
            y = y * g if case["act"] == "silu" else y
        h = case["alpha"] * y + (s["residual"].to(f8) if case["residual"] else 0)
        if not case["pre"]:
            return {"h": h}
        return {"h": h, "x": s["pre_w"].to(f8) * h / ((h ** 2).sum(1, keepdim=True) / case["D"] + 1e-6).sqrt()}
    pool = s["pool"]
    if case["kind"] == "free":
        for d in s["dst"].tolist():
            pool[:, d] = 0
        return {"pool": pool}
    pairs, remap = [], None
    if case["kind"] == "fork":
        pairs = list(zip(s["src"].tolist(), s["dst"].tolist()))
    else:
        live = s["live"].tolist()
        n = sum(live)
        holes = [i for i in range(n) if not live[i]]
        remap = [i if live[i] and i < n else -1 for i in range(len(live))]
        for i in range(n, len(live)):
            if live[i]:
                remap[i] = holes[len(pairs)]
                pairs.append((i, remap[i]))
    for a, b in pairs:
        pool[:, b] = pool[:, a]
    out = {"pool": pool}
    if case["kind"] == "compact":
        out["remap"] = torch.tensor(remap, dtype=torch.int32)
    return out


def _exact_rule(case, s):
    """Row by row, all sequences that still have one at once (longest first)."""
    f8 = torch.float64
    Hk, Hv, dk, dv = case["Hk"], case["Hv"], case["dk"], case["dv"]
    rep = Hv // Hk
    lens = [1] * case["B"] if case["op"] == "gdn_decode" else _lens(case)
    first = [sum(lens[:i]) for i in range(len(lens))]
    live = sorted((n for n in range(len(lens)) if n >= case["skip"] and lens[n]), key=lambda n: -lens[n])
    state = s["rec_state"].to(f8)
    out = s["out"].to(f8)
    if live:
        slot = s["slots"].long()[torch.tensor(live, device=DEV)]
        begin = torch.tensor([first[n] for n in live], device=DEV)
        S = state[slot]
        logdecay = -torch.exp(s["A_log"].to(f8)) * torch.nn.functional.softplus(s["gate"].to(f8) + s["dt_bias"].to(f8), threshold=40)
        alpha, beta = torch.exp(logdecay), 1 / (1 + torch.exp(-s["beta"].to(f8)))
        q = s["q"].reshape(-1, Hk, 1, dk).to(f8)
        k = s["k"].reshape(-1, Hk, 1, dk).to(f8)
        q = (q / (q.square().sum(-1, keepdim=True) + L2_EPS).sqrt() * dk ** -0.5).expand(-1, Hk, rep, dk).reshape(-1, Hv, dk)
        k = (k / (k.square().sum(-1, keepdim=True) + L2_EPS).sqrt()).expand(-1, Hk, rep, dk).reshape(-1, Hv, dk)
        v = s["v"].reshape(-1, Hv, dv)
        for t in range(lens[live[0]]):
            m = len(live)
            while m and lens[live[m - 1]] <= t:
                m -= 1
            if m < len(live):  # the shorter ones are done
                state[slot[m:]] = S[m:]
                live, slot, begin, S = live[:m], slot[:m], begin[:m], S[:m].clone()
            r = begin + t
            kt = k[r]
            S.mul_(alpha[r][..., None, None])
            u = beta[r][..., None] * (v[r].to(f8) - torch.einsum("nhkv,nhk->nhv", S, kt))
            S.add_(kt[..., :, None] * u[..., None, :])
            out[r] = torch.einsum("nhkv,nhk->nhv", S, q[r])
        state[slot] = S
    return {"out": out, "state": state}


def _exact_conv(case, s):
    """Sequence by sequence, as a convolution over the old state's rows and the sequence's own."""
    f8 = torch.float64
    K = case["K"]
    lens = [1] * case["B"] if case["op"] == "conv_decode" else _lens(case)
    y, state, w = s["y"].to(f8), s["conv_state"].to(f8), s["weight"].to(f8)
    if y.numel() > 1 << 29:
        return None
    lo = 0
    for n, ln in enumerate(lens):
        if n >= case["skip"] and ln:
            sl = int(s["slots"][n])
            x = torch.cat([state[sl], s["x"][lo:lo + ln].to(f8)])
            a = sum(x[j:j + ln] * w[:, j] for j in range(K))
            y[lo:lo + ln] = a / (1 + torch.exp(-a))
            state[sl] = x[ln:]
        lo += ln
    return {"y": y, "state": state}
