"""Softmax attention over a paged cache, and what stands in front of it: measured cases.

Each operator is there twice: in its plain form (elementary torch operations in 32 bits, 64 for the
angles of positions), and, where ``own`` is true, as the calls a program makes of the library.

  rope         rotary positions on the q and k heads of rows, or the gradient of that
  append       prompt rows' keys (rotated) and values into a paged cache, their queries rotated
  append_decode  the same for one row per sequence
  attn         attention of chunks of new rows over their sequences' pages
  attn_decode  the same for one row per sequence
"""
import math
import random

import torch

own = False

DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
BLOCK = 1 << 28  # scores that the plain form holds at a time


# ---------------------------------------------------------------- cases

def listed():
    return [
        # q and k heads of a decode batch's rows, the first half of each head turned, positions beyond the trained length
        dict(name="rope_decode_b64", op="rope", rows=64, H=40, D=128, rd=64, layout="half", scaling="ramp", transpose=False, far=1 << 20, io="bf16"),
        # q and k heads of a batch of prompts
        dict(name="rope_prompt", op="rope", rows=32768, H=40, D=128, rd=128, layout="half", scaling="none", transpose=False, far=32768, io="bf16"),
        # gradient of the rotation in a small fp32 model
        dict(name="rope_gradient", op="rope", rows=7001, H=12, D=64, rd=64, layout="pairs", scaling="linear", transpose=True, far=7001, io="f32"),
        # next tokens of a decode batch, two places padded
        dict(name="append_decode_b64", op="append_decode", B=64, L=8192, Hkv=8, G=4, D=128, rd=128, layout="half", scaling="none", page=64, major="token", io="bf16", skip=2, cut=3),
        # a batch of prompts of mixed lengths onto what they had before
        dict(name="append_prompt", op="append", N=8, T=32768, past=4096, Hkv=8, G=4, D=128, rd=128, layout="half", scaling="smooth", page=64, major="head", io="bf16", skip=0, cut=1),
        # a few ragged fp32 prompts on small pages
        dict(name="append_ragged", op="append", N=5, T=701, past=100, Hkv=3, G=4, D=64, rd=32, layout="pairs", scaling="base", page=16, major="token", io="f32", skip=1, cut=2),
        # one user's next token over a long cache: latency
        dict(name="attn_decode_b1", op="attn_decode", B=1, L=32768, Hkv=8, G=4, D=128, window=0, page=64, major="token", io="bf16", skip=0, cut=0),
        # a serving batch of mixed lengths: the cache's bandwidth
        dict(name="attn_decode_b64", op="attn_decode", B=64, L=32768, Hkv=8, G=4, D=128, window=0, page=64, major="head", io="bf16", skip=2, cut=3),
        # wide heads that share two key heads, within a window, on small pages
        dict(name="attn_decode_wide", op="attn_decode", B=250, L=8192, Hkv=2, G=8, D=256, window=2048, page=16, major="token", io="bf16", skip=0, cut=4),
        # a batch of prompts of mixed lengths, some onto what they had before
        dict(name="attn_prompt_n8", op="attn", N=8, T=32768, past=4096, Hkv=8, G=4, D=128, causal=True, window=0, page=64, major="head", io="bf16", skip=0, early=False, cut=1),
        # draft rows of 32 sequences on long caches
        dict(name="attn_verify_b32_w8", op="attn", N=32, T=256, past=8192, Hkv=8, G=4, D=128, causal=True, window=0, page=64, major="token", io="bf16", skip=0, early=False, cut=-1),
        # a few short fp32 prompts; the first one's first rows see nothing
        dict(name="attn_ragged", op="attn", N=5, T=333, past=500, Hkv=4, G=3, D=64, causal=True, window=0, page=16, major="token", io="f32", skip=1, early=True, cut=5),
    ]


def draw(rng):
    log = lambda a, b: int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))  # noqa: E731
    op = rng.choice(["rope", "append", "append_decode", "attn", "attn", "attn_decode", "attn_decode"])
    io = rng.choice(["bf16", "bf16", "bf16", "f32"])
    D = rng.choice([32, 64, 128, 128, 256])
    rd = rng.choice([D, D, D // 2, D // 4])
    turn = dict(rd=rd, layout=rng.choice(["half", "pairs"]), scaling=rng.choice(["none", "linear", "base", "ramp", "smooth"]))
    cut = rng.randrange(1, 1 << 20)
    if op == "rope":
        H = rng.randrange(1, 49)
        return dict(op=op, rows=log(1, min(32768, (1 << 27) // (H * D))), H=H, D=D, transpose=rng.choice([True, False]), far=log(1, 1 << 21), io=io, **turn)
    heads = dict(Hkv=rng.randrange(1, 9), G=rng.choice([1, 2, 3, 4, 5, 6, 7, 8]), D=D, page=rng.choice([16, 32, 64, 128, 256]), major=rng.choice(["token", "head"]), io=io, cut=cut)
    row = heads["Hkv"] * D
    if op == "append":
        N = rng.randrange(1, 17)
        return dict(op=op, N=N, T=log(1, 32768 if row * heads["G"] <= 4096 else 8192), past=log(1, 4096), skip=rng.randrange(0, 2) if N > 2 else 0, **heads, **turn)
    if op == "append_decode":
        B = log(1, 250)
        return dict(op=op, B=B, L=log(1, 8192), skip=rng.randrange(0, 1 + B // 8), **heads, **turn)
    if op == "attn_decode":
        B = log(1, 250)
        L = log(1, min(32768, (1 << 30) // (B * row)))
        return dict(op=op, B=B, L=L, window=rng.choice([0, 0, log(1, 8192)]), skip=rng.randrange(0, 1 + B // 8), **heads)
    N = rng.randrange(1, 17)
    T = log(1, 8192 if io == "bf16" else 1024)
    causal = rng.choice([True, True, True, False])
    return dict(op=op, N=N, T=T, past=log(1, 16384 if io == "bf16" else 2048), causal=causal, window=rng.choice([0, 0, log(1, 8192)]) if causal else 0,
                skip=rng.randrange(0, 2) if N > 2 else 0, early=rng.choice([True, False, False]), **heads)


def _lens(case):
    """(new rows, cached tokens with them; negative: padding) of each sequence."""
    r = random.Random(case["cut"])
    if "B" in case:
        lens = [1] * case["B"]
        kv = [case["L"] if case["cut"] == 0 else r.randrange(1, case["L"] + 1) for _ in lens]
    else:
        T, N = case["T"], case["N"]
        ends = [T * (n + 1) // N for n in range(N)] if case["cut"] < 0 else sorted(r.randrange(0, T + 1) for _ in range(N - 1)) + [T]
        lens = [b - a for a, b in zip([0] + ends, ends)]
        kv = [n + r.randrange(0, case["past"] + 1) for n in lens]
    for n in range(case["skip"]):  # the padded sequences come first
        kv[n] = -1
    if case.get("early"):  # more rows than tokens that are there: the first ones see nothing
        kv[case["skip"]] = (lens[case["skip"]] + 1) // 2
    return lens, kv


# ---------------------------------------------------------------- inputs

def _randn(g, *shape, dtype=torch.float32, std=1.0):
    return (torch.randn(*shape, generator=g, device=DEV) * std).to(dtype)


def _radians(case):
    """Angle of each pair per position, and the amplitude, of the case's scaling: for contexts 8 times 4096 long."""
    rd, kind, factor, length = case["rd"], case["scaling"], 8.0, 4096.0
    base = 10000.0
    if kind == "base" and rd > 2:
        base *= factor ** (rd / (rd - 2))
    f = [base ** (-2 * i / rd) for i in range(rd // 2)]
    if kind == "linear":
        f = [x / factor for x in f]
    if kind == "ramp":  # pairs that turn often keep their angle, slow ones turn factor times slower, a ramp over the pairs between
        dim = lambda turns: rd * math.log(length / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        lo, hi = max(math.floor(dim(32.0)), 0), min(math.ceil(dim(1.0)), rd - 1)
        ramp = [min(max((i - lo) / max(hi - lo, 1e-3), 0), 1) for i in range(rd // 2)]
        f = [x / factor * r + x * (1 - r) for x, r in zip(f, ramp)]
    if kind == "smooth":  # the same by the turns a pair makes over the length
        keep = [min(max((length * x / (2 * math.pi) - 1.0) / (4.0 - 1.0), 0), 1) for x in f]
        f = [x / factor * (1 - k) + x * k for x, k in zip(f, keep)]
    return f, 0.1 * math.log(factor) + 1 if kind == "ramp" else 1.0


def _inputs(case, seed):
    """The case's tensors, made on the GPU from the seed."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    dt, D, op = DT[case["io"]], case["D"], case["op"]
    s = {}
    if op == "rope":
        rows, H = case["rows"], case["H"]
        s["qkv"] = _randn(g, rows, (H + 8) * D, dtype=dt)  # the v heads of a row stay out
        s["x"] = s["qkv"][:, :H * D]
        s["y"] = torch.zeros(rows, H, D, dtype=dt, device=DEV)
        s["positions"] = torch.randint(0, case["far"], (rows,), generator=g, device=DEV, dtype=torch.int32)
        return s
    lens, kv = _lens(case)
    Hkv, Hq, P = case["Hkv"], case["Hkv"] * case["G"], case["page"]
    T, N = sum(lens), len(lens)
    per = [(max(n, 0) + P - 1) // P for n in kv]
    width, num = max(per) + 2, sum(per) + 3
    # a pool of pages in any order
    order = torch.randperm(num, generator=g, device=DEV).to(torch.int32)
    s["pages"] = torch.full((N, width), -1, dtype=torch.int32, device=DEV)
    at = torch.tensor([sum(per[:n]) for n in range(N)], device=DEV)
    i = torch.arange(width, device=DEV)
    real = i < torch.tensor(per, device=DEV)[:, None]
    s["pages"][real] = order[(at[:, None] + i)[real]]
    shape = (num, P, Hkv, D) if case["major"] == "token" else (num, Hkv, P, D)
    s["k_cache"], s["v_cache"] = _randn(g, *shape, dtype=dt), _randn(g, *shape, dtype=dt)
    s["kv_lens"] = torch.tensor(kv, dtype=torch.int32, device=DEV)
    s["cu_seqlens"] = torch.tensor([0] + lens, device=DEV).cumsum(0).to(torch.int32)
    if op in ("append", "append_decode"):
        s["qkv"] = _randn(g, T, (Hq + 2 * Hkv) * D, dtype=dt)
        s["q"], s["k"], s["v"] = s["qkv"][:, :Hq * D], s["qkv"][:, Hq * D:(Hq + Hkv) * D], s["qkv"][:, (Hq + Hkv) * D:]
        s["q_out"] = torch.zeros(T, Hq, D, dtype=dt, device=DEV)
    else:
        s["q"] = _randn(g, T, Hq, D, dtype=dt, std=1.5)
        s["out"] = torch.zeros(T, Hq, D, dtype=dt, device=DEV)
        s["lse"] = torch.zeros(T, Hq, device=DEV)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if "rd" in case:
        f, s["amplitude"] = _radians(case)
        s["radians"] = torch.tensor(f, dtype=torch.float64, device=DEV)
    if own:
        s["call"] = _call(case, s)
    return s


# ---------------------------------------------------------------- the library's calls

def _call(case, s):
    """The call of one pass with its arguments marshalled, as a serving loop keeps it."""
    import linear_attention_serving_kda_gb300 as kda

    code = {"bf16": kda.KDA_DTYPE_BF16, "f32": kda.KDA_DTYPE_F32}[case["io"]]
    op, D = case["op"], case["D"]
    turn = {}
    if "rd" in case:
        kind = {"none": kda.KDA_ROPE_SCALE_NONE, "linear": kda.KDA_ROPE_SCALE_LINEAR, "base": kda.KDA_ROPE_SCALE_BASE,
                "ramp": kda.KDA_ROPE_SCALE_RAMP, "smooth": kda.KDA_ROPE_SCALE_SMOOTH}[case["scaling"]]
        fast = 32.0 if case["scaling"] == "ramp" else 4.0
        scaling = kda.RopeScaling(kind=kind, base=10000.0, factor=8.0, length=4096.0, fast=fast, slow=1.0)
        turns = torch.empty(case["rd"] // 2, dtype=torch.int64)
        kda.check(kda.kda_rope_turns(scaling, case["rd"], None, turns))
        s["turns"] = turns.to(DEV)
        layout = {"half": kda.KDA_ROPE_HALF, "pairs": kda.KDA_ROPE_PAIRS}[case["layout"]]
        turn = dict(rotary_dim=case["rd"], rope_layout=layout, rope_amplitude=s["amplitude"], rope_turns=s["turns"])
    if op == "rope":
        p = kda.RopeParams(num_heads=case["H"], head_dim=D, io_dtype=code, transpose=case["transpose"], x_row_stride=s["qkv"].shape[1], **turn)
        return kda.Prepared("kda_rope", p, case["rows"], s["positions"], s["x"], s["y"])
    P, Hkv = case["page"], case["Hkv"]
    major = dict(cache_token_stride=Hkv * D, cache_head_stride=D) if case["major"] == "token" else dict(cache_token_stride=D, cache_head_stride=P * D)
    shape = dict(num_heads_q=Hkv * case["G"], num_heads_kv=Hkv, head_dim=D, io_dtype=code, page_size=P, num_pages=s["k_cache"].shape[0],
                 pages_per_seq=s["pages"].shape[1], cache_page_stride=P * Hkv * D, **major)
    N, T = s["pages"].shape[0], s["q"].shape[0]
    if op in ("append", "append_decode"):
        stride = s["qkv"].shape[1]
        p = kda.PagedParams(q_in_row_stride=stride, k_row_stride=stride, v_row_stride=stride, **shape, **turn)
        rest = (s["kv_lens"], s["pages"], None, s["q"], s["k"], s["v"], s["q_out"], s["k_cache"], s["v_cache"], None)
        if op == "append":
            return kda.Prepared("kda_paged_append_varlen", p, s["cu_seqlens"], N, T, *rest)
        return kda.Prepared("kda_paged_append_decode", p, N, *rest)
    p = kda.PagedParams(scale=D ** -0.5, causal=case.get("causal", True), window=case["window"], **shape)
    rest = (s["kv_lens"], s["pages"], s["q"], s["k_cache"], s["v_cache"], s["out"], s["lse"])
    if op == "attn":
        need = kda.kda_paged_attn_workspace_bytes(p, N, T)
    else:
        need = kda.kda_paged_attn_decode_workspace_bytes(p, N)
    s["workspace"] = torch.empty(need, dtype=torch.uint8, device=DEV) if need else None
    if op == "attn":
        return kda.Prepared("kda_paged_attn_varlen", p, s["cu_seqlens"], N, T, *rest, s["workspace"], need, None)
    return kda.Prepared("kda_paged_attn_decode", p, N, *rest, s["workspace"], need, None)


def run(s):
    case = s["case"]
    if own:
        if s["call"]() != 0:
            raise RuntimeError("the library refused %r" % (case,))
    else:
        PLAIN[case["op"]](case, s)
    if case["op"] == "rope":
        return {"y": s["y"]}
    if "q_out" in s:
        return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    return {"out": s["out"], "lse": s["lse"]}


# ---------------------------------------------------------------- plain forms

def _turned(case, s, x, positions):
    """x [rows][H][D] with each row turned to its position, in 32 bits."""
    rd = case["rd"]
    angle = positions.double()[:, None] * s["radians"]
    cos, sin = (torch.cos(angle) * s["amplitude"]).float()[:, None], (torch.sin(angle) * s["amplitude"]).float()[:, None]
    if case.get("transpose"):
        sin = -sin
    x = x.float()
    if case["layout"] == "half":
        a, b = x[..., :rd // 2], x[..., rd // 2:rd]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = x[..., 0:rd:2], x[..., 1:rd:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([turned, x[..., rd:]], -1)


def _plain_rope(case, s):
    s["y"].copy_(_turned(case, s, s["x"].unflatten(-1, (case["H"], case["D"])), s["positions"]))


def _plain_append(case, s):
    D, P = case["D"], case["page"]
    T, N = s["q"].shape[0], s["pages"].shape[0]
    cu, kv = s["cu_seqlens"].long(), s["kv_lens"].long()
    n = torch.repeat_interleave(torch.arange(N, device=DEV), cu[1:] - cu[:-1], output_size=T)
    rows = torch.arange(int(sum(_lens(case)[0][:case["skip"]])), T, device=DEV)  # the padded sequences come first
    n = n[rows]
    pos = kv[n] - (cu[n + 1] - rows)
    page, place = s["pages"][n, pos // P].long(), pos % P
    heads = lambda x: x[rows].unflatten(-1, (-1, D))  # noqa: E731
    s["q_out"][rows] = _turned(case, s, heads(s["q"]), pos).to(s["q_out"].dtype)
    k, v = _turned(case, s, heads(s["k"]), pos).to(s["k_cache"].dtype), heads(s["v"])
    if case["major"] == "token":
        s["k_cache"][page, place], s["v_cache"][page, place] = k, v
    else:
        s["k_cache"][page, :, place], s["v_cache"][page, :, place] = k, v


def _tokens(case, s, n, lo, hi):
    """Cached keys and values lo .. hi - 1 of sequence n: [Hkv][hi - lo][D], in 32 bits."""
    P = case["page"]
    pages = s["pages"][n, lo // P:(hi + P - 1) // P].long()
    out = []
    for c in (s["k_cache"], s["v_cache"]):
        x = c[pages]
        x = x.transpose(1, 2) if case["major"] == "token" else x
        out.append(x.transpose(0, 1).flatten(1, 2)[:, lo % P:lo % P + hi - lo].float())
    return out


def _plain_attn(case, s):
    lens, kv = _lens(case)
    G, Hkv, D, W = case["G"], case["Hkv"], case["D"], case["window"]
    causal = case.get("causal", True)
    begin = 0
    for n, (ln, L) in enumerate(zip(lens, kv)):
        rows, begin = range(begin, begin + ln), begin + ln
        if L < 0 or ln == 0:
            continue
        step = max(1, BLOCK // (Hkv * G * max(L, 1)))
        for r0 in range(rows[0], rows[-1] + 1, step):
            r1 = min(r0 + step, rows[-1] + 1)
            first = L - (rows[-1] + 1 - r0)  # position of row r0
            lo = max(0, first - W + 1) if W else 0
            hi = max(min(L, first + r1 - r0), lo) if causal else L
            if hi == lo:
                s["out"][r0:r1] = 0
                s["lse"][r0:r1] = -math.inf
                continue
            k, v = _tokens(case, s, n, lo, hi)
            q = s["q"][r0:r1].float().unflatten(1, (Hkv, G)).permute(1, 0, 2, 3).reshape(Hkv, -1, D)
            x = (q @ k.transpose(1, 2)) * D ** -0.5
            x = x.view(Hkv, r1 - r0, G, hi - lo)
            if causal:
                p, j = first + torch.arange(r1 - r0, device=DEV)[:, None], torch.arange(lo, hi, device=DEV)
                hide = (j > p) | (j <= p - W) if W else j > p
                x.masked_fill_(hide[None, :, None], -math.inf)
            m = x.amax(-1, keepdim=True)
            x = x.sub_(torch.where(m == -math.inf, 0, m)).exp_()
            l = x.sum(-1, keepdim=True)  # noqa: E741
            o = (x.view(Hkv, -1, hi - lo) @ v).view(Hkv, r1 - r0, G, D) / torch.where(l == 0, 1, l)
            s["out"][r0:r1] = o.permute(1, 0, 2, 3).reshape(r1 - r0, Hkv * G, D).to(s["out"].dtype)
            s["lse"][r0:r1] = (m + torch.log(l))[..., 0].permute(1, 0, 2).reshape(r1 - r0, -1)


PLAIN = {"rope": _plain_rope, "append": _plain_append, "append_decode": _plain_append, "attn": _plain_attn, "attn_decode": _plain_attn}


# ---------------------------------------------------------------- what a pass cannot do without

def _seen(case):
    """(pairs of a row and a token that it sees, tokens that any row of their sequence sees)."""
    W, pairs, tokens = case["window"], 0, 0
    for ln, L in zip(*_lens(case)):
        if L < 0 or ln == 0:
            continue
        if not case.get("causal", True):
            pairs += ln * L
            tokens += L
            continue
        first = max(L - ln, 0)               # position of the first row that sees something
        tokens += min(L, L - first + W - 1) if W else L
        for a, b in ((first, min(L, W)), (max(first, W), L)) if W else ((first, L),):
            if b > a:                        # rows at positions a .. b - 1
                pairs += (b - a) * W if W and a >= W else (a + 1 + b) * (b - a) // 2
    return pairs, tokens


def work(case):
    size, D = {"bf16": 2, "f32": 4}[case["io"]], case["D"]
    if case["op"] == "rope":
        n = case["rows"] * case["H"] * D
        return {"bytes": 2 * n * size + 4 * case["rows"], "flops": 3 * n}
    lens, kv = _lens(case)
    rows = sum(n for n, L in zip(lens, kv) if L >= 0)
    Hq, Hkv = case["Hkv"] * case["G"], case["Hkv"]
    if "rd" in case:
        return {"bytes": 2 * rows * (Hq + 2 * Hkv) * D * size + 8 * len(lens), "flops": 3 * rows * (Hq + Hkv) * case["rd"]}
    pairs, tokens = _seen(case)
    return {"bytes": rows * Hq * (2 * D * size + 4) + 2 * tokens * Hkv * D * size + 8 * len(lens), "flops": 4 * D * Hq * pairs + 1}


# ---------------------------------------------------------------- in 64 bits, from the definitions

def _exact_turn(case, x, pos):
    """As complex numbers: a pair times amplitude e^(i angle)."""
    rd = case["rd"]
    f, amplitude = _radians(case)
    angle = pos.to(torch.float64).unsqueeze(1) * torch.tensor(f, dtype=torch.float64, device=DEV)
    z = torch.polar(torch.full_like(angle, amplitude), -angle if case.get("transpose") else angle).unsqueeze(1)
    y = x.to(torch.float64).clone()
    i = torch.arange(rd // 2, device=DEV)
    one, two = (i, i + rd // 2) if case["layout"] == "half" else (2 * i, 2 * i + 1)
    w = torch.complex(y[..., one], y[..., two]) * z
    y[..., one], y[..., two] = w.real, w.imag
    return y


def exact(case, seed):
    s = _inputs(case, seed)
    f8, D = torch.float64, case["D"]
    if case["op"] == "rope":
        return {"y": _exact_turn(case, s["x"].reshape(case["rows"], case["H"], D), s["positions"])}
    lens, kv = _lens(case)
    P, G, Hkv = case["page"], case["G"], case["Hkv"]
    kc, vc = s["k_cache"], s["v_cache"]
    if case["major"] == "head":
        kc, vc = kc.transpose(1, 2), vc.transpose(1, 2)   # both as [page][place][head][D]
    if "q_out" in s:
        if kc.numel() > 1 << 29:
            return None
        q, kc, vc, begin = s["q_out"].to(f8), kc.to(f8), vc.to(f8), 0
        for n, ln in enumerate(lens):
            at = slice(begin, begin + ln)
            begin += ln
            if kv[n] < 0 or ln == 0:
                continue
            pos = torch.arange(kv[n] - ln, kv[n], device=DEV)
            page, place = s["pages"][n].long()[pos // P], pos % P
            q[at] = _exact_turn(case, s["q"][at].reshape(ln, -1, D), pos)
            kc[page, place] = _exact_turn(case, s["k"][at].reshape(ln, -1, D), pos)
            vc[page, place] = s["v"][at].reshape(ln, -1, D).to(f8)
        if case["major"] == "head":
            kc, vc = kc.transpose(1, 2), vc.transpose(1, 2)
        return {"q": q, "k_cache": kc, "v_cache": vc}
    if 4 * D * G * Hkv * sum(a * max(b, 0) for a, b in zip(lens, kv)) > 8e12:
        return None
    out, lse, begin = s["out"].to(f8), s["lse"].to(f8), 0
    for n, ln in enumerate(lens):
        r0, begin, L = begin, begin + ln, kv[n]
        if L < 0 or ln == 0:
            continue
        page = s["pages"][n, :(L + P - 1) // P].long()
        for h in range(Hkv):
            k, v = kc[page, :, h].reshape(-1, D)[:L].to(f8), vc[page, :, h].reshape(-1, D)[:L].to(f8)
            for a in range(0, ln, 2048):
                b = min(a + 2048, ln)
                at, heads = slice(r0 + a, r0 + b), slice(h * G, h * G + G)
                x = torch.einsum("tgd,jd->tgj", s["q"][at, heads].to(f8), k) / math.sqrt(D)
                if case.get("causal", True):
                    behind = torch.arange(L - ln + a, L - ln + b, device=DEV)[:, None, None] - torch.arange(L, device=DEV)
                    x = torch.where((behind >= 0) & (behind < (case["window"] or L + 1)), x, -math.inf)
                e = torch.logsumexp(x, -1) if L else torch.full(x.shape[:2], -math.inf, dtype=f8, device=DEV)
                lse[at, heads] = e
                weight = torch.exp(x - torch.where(e == -math.inf, 0, e)[..., None])
                out[at, heads] = torch.einsum("tgj,jd->tgd", weight, v)
    return {"out": out, "lse": lse}
