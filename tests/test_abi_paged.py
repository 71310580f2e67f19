"""Refusals of rotary positions, the append to a paged cache and the attention over it: every one of them
before any launch, without a GPU; and the angles that the host computes."""
import ctypes
import math

import pytest
import torch

import linear_attention_serving_kda_gb300 as kda
from linear_attention_serving_kda_gb300 import build as kbuild
from tests import paged64 as P

FAKE = 1 << 20  # 16-byte-aligned addresses far apart; never dereferenced
STEP = 1 << 34
INVALID, GEOMETRY, OK = kda.KDA_ERR_INVALID_ARGUMENT, kda.KDA_ERR_UNSUPPORTED_GEOMETRY, kda.KDA_OK
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module", autouse=True)
def lib():
    kbuild.build()
    return kda.load()


def addr(i):
    return FAKE + i * STEP


def _turns(rd=64, radians=None, turns=True, **kw):
    t = torch.empty(max(rd // 2, 1), dtype=torch.int64) if turns else None
    return kda.kda_rope_turns(kda.RopeScaling(**kw), rd, radians, t), t


@pytest.mark.parametrize("kind,kw", [("none", {}), ("linear", dict(factor=8.0)), ("base", dict(factor=8.0)), ("ramp", dict(factor=16.0)),
                                     ("smooth", dict(factor=8.0, fast=4.0)), ("none", dict(base=500000.0)), ("ramp", dict(factor=4.0, length=2.0))])
@pytest.mark.parametrize("rd", [4, 64, 126, 512])
def test_turns(rd, kind, kw):
    rc, t = _turns(rd, kind=dict(none=0, linear=1, base=2, ramp=3, smooth=4)[kind], **kw)
    assert rc == OK
    f = P.radians(rd, kind, **kw)
    for i in range(rd // 2):
        got = (int(t[i]) % (1 << 64)) / 2.0 ** 64
        # a handful of roundings of 64-bit values in either computation, the power's argument (up to 17 in size) among them,
        # and the fixed-point value's own step of 2^-64, cut off
        assert abs(got - f[i] / (2 * math.pi) % 1) <= 2.0 ** -47 * f[i] / (2 * math.pi) + 2.0 ** -64, i


def test_turns_of_given_angles():
    f = torch.tensor([2 * math.pi * 0.25, -2 * math.pi * 0.25, 0.0, 2 * math.pi * 3.5], dtype=torch.float64)
    rc, t = _turns(8, radians=f)
    assert rc == OK and [int(x) % (1 << 64) >> 48 for x in t] in ([0x4000, 0xC000, 0, 0x8000], [0x3FFF, 0xC000, 0, 0x8000])
    rc, t = _turns(8, radians=f, kind=1, factor=2.0)
    assert rc == OK and int(t[3]) % (1 << 64) >> 48 == 0xC000
    assert _turns(8, radians=f, kind=2, factor=2.0)[0] == INVALID
    assert _turns(8, radians=f, base=0.0)[0] == OK  # not read
    for bad in (INF, NAN):
        assert _turns(8, radians=torch.tensor([0.0, 1.0, bad, 1.0], dtype=torch.float64))[0] == INVALID


@pytest.mark.parametrize("kw,rc", [
    (dict(rd=0), GEOMETRY), (dict(rd=3), GEOMETRY), (dict(rd=514), GEOMETRY), (dict(rd=-2), GEOMETRY), (dict(turns=False), INVALID),
    (dict(kind=5), INVALID), (dict(kind=-1), INVALID), (dict(base=1.0), INVALID), (dict(base=NAN), INVALID), (dict(base=INF), INVALID),
    (dict(kind=1, factor=0.0), INVALID), (dict(kind=1, factor=NAN), INVALID), (dict(kind=2, rd=2), INVALID),
    (dict(kind=3, length=0.0), INVALID), (dict(kind=3, fast=1.0, slow=1.0), INVALID), (dict(kind=4, slow=0.0), INVALID),
    (dict(kind=4, fast=INF), INVALID), (dict(factor=0.0), OK), (dict(kind=1, length=NAN, factor=2.0), OK),
])
def test_turns_refusals(kw, rc):
    assert _turns(**kw)[0] == rc


def test_turns_without_a_finite_angle():
    big = torch.full((32,), 1e308, dtype=torch.float64)
    for kind in (1, 3, 4):
        assert _turns(kind=kind, factor=1e-320)[0] == INVALID, kind
        assert _turns(kind=kind, factor=1e-5, radians=big)[0] == INVALID, kind
    for factor in (1e-300, 1e300):
        assert _turns(4, kind=2, factor=factor)[0] == INVALID
    assert _turns(kind=2, factor=1e-4, base=10.0)[0] == OK


ROPE = dict(num_heads=4, head_dim=64, rotary_dim=32, rope_turns=addr(9))


def _rope(rows=5, pos=addr(1), x=addr(2), y=addr(3), **kw):
    return kda.kda_rope(kda.RopeParams(**{**ROPE, **kw}), rows, pos, x, y, 0)


@pytest.mark.parametrize("kw,rc", [
    (dict(num_heads=0), INVALID), (dict(head_dim=8), GEOMETRY), (dict(head_dim=40), GEOMETRY), (dict(head_dim=528), GEOMETRY),
    (dict(rotary_dim=0), GEOMETRY), (dict(rotary_dim=31), GEOMETRY), (dict(rotary_dim=66), GEOMETRY), (dict(rope_layout=2), INVALID),
    (dict(transpose=2), INVALID), (dict(rope_amplitude=NAN), INVALID), (dict(rope_turns=None), INVALID), (dict(rope_turns=addr(9) + 8), INVALID),
    (dict(io_dtype=2), INVALID), (dict(x_row_stride=248), INVALID), (dict(x_row_stride=260), INVALID), (dict(y_row_stride=-8), INVALID),
    (dict(y_row_stride=1 << 29), INVALID), (dict(num_heads=1 << 30), INVALID),
    (dict(rows=-1), INVALID), (dict(rows=1 << 31), INVALID), (dict(pos=None), INVALID), (dict(pos=addr(1) + 4), INVALID),
    (dict(x=None), INVALID), (dict(x=addr(2) + 8), INVALID), (dict(y=None), INVALID),
    (dict(y=addr(2), y_row_stride=264), INVALID), (dict(y=addr(2) + 256), INVALID), (dict(y=addr(1)), INVALID), (dict(y=addr(9)), INVALID),
    (dict(rows=0, x=None), OK),
])
def test_rope_refusals(kw, rc):
    assert _rope(**kw) == rc


PAGED = dict(num_heads_q=4, num_heads_kv=2, head_dim=64, page_size=16, num_pages=10, pages_per_seq=4)


def _params(**kw):
    return kda.PagedParams(**{**PAGED, **kw})


def _append(p, decode=False, N=2, T=6, cu=addr(1), kv=addr(2), pages=addr(3), pos=None, q=addr(4), k=addr(5), v=addr(6), qo=addr(7),
            kc=addr(8), vc=addr(10)):
    if decode:
        return kda.kda_paged_append_decode(p, N, kv, pages, pos, q, k, v, qo, kc, vc, None, 0)
    return kda.kda_paged_append_varlen(p, cu, N, T, kv, pages, pos, q, k, v, qo, kc, vc, None, 0)


def _attn(p, decode=False, N=2, T=6, cu=addr(1), kv=addr(2), pages=addr(3), q=addr(4), kc=addr(8), vc=addr(10), out=addr(11), lse=addr(12),
          ws=addr(13), nws=1 << 33):
    if decode:
        return kda.kda_paged_attn_decode(p, N, kv, pages, q, kc, vc, out, lse, ws, nws, None, 0)
    return kda.kda_paged_attn_varlen(p, cu, N, T, kv, pages, q, kc, vc, out, lse, ws, nws, None, 0)


@pytest.mark.parametrize("kw,rc", [
    (dict(num_heads_kv=0), INVALID), (dict(num_heads_q=0), INVALID), (dict(num_heads_q=5), INVALID), (dict(num_heads_q=1026), INVALID),
    (dict(head_dim=96), GEOMETRY), (dict(head_dim=512), GEOMETRY), (dict(io_dtype=7), INVALID),
    (dict(page_size=8), GEOMETRY), (dict(page_size=48), GEOMETRY), (dict(page_size=2048), GEOMETRY), (dict(page_size=0), GEOMETRY),
    (dict(num_pages=0), INVALID), (dict(pages_per_seq=0), INVALID), (dict(pages_per_seq=1 << 28), INVALID),
    (dict(cache_head_stride=68), INVALID), (dict(cache_head_stride=32), INVALID), (dict(cache_token_stride=120), INVALID),
    (dict(cache_token_stride=64, cache_head_stride=64 * 15), INVALID),   # the heads' tokens overlap
    (dict(cache_token_stride=120, cache_head_stride=64), INVALID),
    (dict(cache_page_stride=16 * 128 - 8), INVALID), (dict(cache_token_stride=-128), INVALID), (dict(cache_page_stride=1 << 37), INVALID),
    (dict(q_row_stride=248), INVALID), (dict(q_in_row_stride=260), INVALID), (dict(k_row_stride=64), INVALID), (dict(v_row_stride=1 << 29), INVALID),
])
def test_paged_params(kw, rc):
    p = _params(**kw)
    for d in (False, True):
        assert _append(p, d) == rc and _attn(p, d) == rc
    assert kda.kda_paged_attn_workspace_bytes(p, 2, 6) == 0 and kda.kda_paged_attn_decode_workspace_bytes(p, 2) == 0


@pytest.mark.parametrize("kw,rc", [
    (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID), (dict(scale=NAN), INVALID), (dict(scale=INF), INVALID), (dict(scale=3e38), INVALID), (dict(causal=2), INVALID),
    (dict(window=-1), INVALID), (dict(window=4, causal=False), INVALID),
])
def test_attn_params(kw, rc):
    for d in (False, True):
        assert _attn(_params(**kw), d) == rc
    assert kda.kda_paged_attn_workspace_bytes(_params(**kw), 2, 6) == 0


@pytest.mark.parametrize("kw,rc", [
    (dict(rotary_dim=66), GEOMETRY), (dict(rotary_dim=5), GEOMETRY), (dict(rotary_dim=-2), GEOMETRY), (dict(rope_turns=None), INVALID),
    (dict(rope_layout=3), INVALID), (dict(rope_amplitude=INF), INVALID), (dict(rope_turns=addr(9) + 8), INVALID),
])
def test_append_rotation(kw, rc):
    for d in (False, True):
        assert _append(_params(**{**dict(rotary_dim=64, rope_turns=addr(9)), **kw}), d) == rc


def test_caches_past_64_bits():
    """Pages and strides that are in their ranges, and a cache of 2^67 values, whose bytes no overlap could be told from."""
    for pages, stride in (((1 << 31) - 1, 1 << 36), (1 << 25, 1 << 36)):
        p = _params(num_pages=pages, cache_page_stride=stride)
        for d in (False, True):
            assert _attn(p, d, out=addr(8)) == INVALID and _attn(p, d) == INVALID and _append(p, d) == INVALID
        assert kda.kda_paged_attn_workspace_bytes(p, 2, 6) == 0


@pytest.mark.parametrize("io", [kda.KDA_DTYPE_BF16, kda.KDA_DTYPE_F32])
def test_keys_and_values_that_share_places(io):
    """Against all places of a small cache, counted one by one.  (A call that gets past this check stops at its rotation, whose width is odd.)"""
    size = 2 if io == kda.KDA_DTYPE_BF16 else 4
    D = 32
    # key heads, strides of pages, tokens and heads: dense, either order, with gaps, pools side by side in a page, one head
    for Hkv, ps, ts, hs, pages in [(*x, 3) for x in [(2, 16 * 64, 64, 32), (2, 16 * 64, 32, 16 * 32), (2, 2048, 64, 32), (2, 2048, 32, 512), (2, 4096, 128, 32), (2, 4096, 128, 64),
                            (3, 4992, 48, 1024), (1, 16 * 32, 32, 32), (1, 1024, 64, 8192), (1, 576, 32, 8192)]] + [
                                   (2, 64, 64, 32, 1), (2, 128, 32, 512, 1), (1, 32, 64, 32, 1)]:
        p = _params(num_heads_q=Hkv, num_heads_kv=Hkv, head_dim=D, num_pages=pages, io_dtype=io, cache_page_stride=ps, cache_token_stride=ts,
                    cache_head_stride=hs, rotary_dim=5)
        starts = {pg * ps + t * ts + h * hs for pg in range(pages) for t in range(16) for h in range(Hkv)}
        taken = {s + i for s in starts for i in range(0, D, 8)}
        seen = set()
        for delta in {8 * i for i in range(-40, 41)} | {x + 8 * i for x in (ps, 2 * ps, 3 * ps, -ps, 15 * ts, 16 * ts, hs, hs * Hkv, ps // 2) for i in range(-9, 10)}:
            meet = any(s + delta + i in taken for s in starts for i in range(0, D, 8))
            seen.add(meet)
            for d in (False, True):
                assert _append(p, d, kc=addr(8), vc=addr(8) + delta * size) == (INVALID if meet else GEOMETRY), (Hkv, ps, ts, hs, delta)
        assert seen == {True, False}


def test_append_pointers():
    p = _params()
    for d in (False, True):
        for name, i in dict(kv=2, pages=3, k=5, v=6, kc=8, vc=10).items():
            assert _append(p, d, **{name: None}) == INVALID and _append(p, d, **{name: addr(i) + 8}) == INVALID, name
        assert _append(p, d, q=None) == INVALID and _append(p, d, qo=None) == INVALID
        assert _append(p, d, qo=addr(7) + 8) == INVALID and _append(p, d, pos=addr(14) + 4) == INVALID
        # what is written apart from what is read
        for name in ("q", "k", "v", "kv", "pages"):
            assert _append(p, d, **{name: addr(8) + 10 * 16 * 128 * 2 - 16}) == INVALID, name
            assert _append(p, d, **{name: addr(10)}) == INVALID, name
        assert _append(p, d, k=addr(7)) == INVALID and _append(p, d, qo=addr(4) + 16) == INVALID
        assert _append(p, d, pos=addr(7)) == INVALID and _append(p, d, qo=addr(8)) == INVALID and _append(p, d, vc=addr(8)) == INVALID
        # q rotated in place while k or v shares its channels
        assert _append(_params(q_in_row_stride=512, q_row_stride=512, k_row_stride=512), d, qo=addr(4), k=addr(4) + 2 * 240) == INVALID
        assert _append(p, d, N=-1) == INVALID and _append(p, d, N=1 << 30) == INVALID and _append(p, d, N=0) == OK
    assert _append(p, cu=None) == INVALID and _append(p, cu=addr(8)) == INVALID and _append(p, T=-1) == INVALID and _append(p, T=0) == OK


def test_attn_pointers():
    p = _params()
    for d in (False, True):
        for name, i in dict(kv=2, pages=3, q=4, kc=8, vc=10, out=11).items():
            assert _attn(p, d, **{name: None}) == INVALID and _attn(p, d, **{name: addr(i) + 8}) == INVALID, name
        assert _attn(p, d, lse=addr(12) + 4) == INVALID
        for out in ("out", "lse", "ws"):
            for other in (2, 3, 4, 8, 10):
                assert _attn(p, d, **{out: addr(other)}) == INVALID, (out, other)
        assert _attn(p, d, lse=addr(11)) == INVALID and _attn(p, d, ws=addr(11)) == INVALID and _attn(p, d, ws=addr(12)) == INVALID
        assert _attn(p, d, out=addr(8) + 10 * 16 * 128 * 2 - 16) == INVALID
        assert _attn(p, d, N=-1) == INVALID and _attn(p, d, N=1 << 30) == INVALID and _attn(p, d, N=0) == OK
        need = kda.kda_paged_attn_decode_workspace_bytes(p, 2) if d else kda.kda_paged_attn_workspace_bytes(p, 2, 6)
        assert need > 0
        for bad in (dict(ws=None), dict(nws=need - 1), dict(ws=addr(13) + 8)):
            assert _attn(p, d, **bad) == kda.KDA_ERR_WORKSPACE, bad
    assert _attn(p, cu=None) == INVALID and _attn(p, T=-1) == INVALID and _attn(p, T=0) == OK


def test_stalled_refusals():
    def call(cu=addr(1), N=2, T=6, polls=1, unit=1, **kw):
        return kda.kda_debug_paged_attn_stalled(_params(**kw), cu, N, T, addr(2), addr(3), addr(4), addr(8), addr(10), addr(11), addr(12), None, 0, None,
                                                polls, unit, 0, 0)

    assert call(polls=0) == INVALID and call(unit=0) == INVALID and call(cu=None) == INVALID and call(scale=0.0) == INVALID
    assert call(head_dim=96) == GEOMETRY and call(N=-1) == INVALID and call(T=0) == OK
    assert call() == kda.KDA_ERR_WORKSPACE and call(cu=None, T=2) == kda.KDA_ERR_WORKSPACE


def test_workspaces():
    p = _params()
    assert kda.kda_paged_attn_workspace_bytes(p, -1, 6) == 0 and kda.kda_paged_attn_workspace_bytes(p, 2, 0) == 0
    for io in (kda.KDA_DTYPE_BF16, kda.KDA_DTYPE_F32):
        q = _params(io_dtype=io, num_heads_q=32, num_heads_kv=8, head_dim=128)
        assert 0 < kda.kda_paged_attn_workspace_bytes(q, 8, 32768) < 1 << 28
        assert 0 < kda.kda_paged_attn_decode_workspace_bytes(q, 256) < 1 << 28


def test_struct_layouts():
    k = kda.kda
    assert ctypes.sizeof(k.kda_rope_scaling) == 48 and ctypes.sizeof(k.kda_rope_params) == 56
    assert ctypes.sizeof(k.kda_paged_params) == 56 + 7 * 8 + 8


def test_struct_layouts_as_c_sees_them(tmp_path):
    import os
    import shutil
    import subprocess

    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    lines, want = [], []
    for s in (kda.kda.kda_rope_scaling, kda.kda.kda_rope_params, kda.kda.kda_paged_params):
        lines.append(f'printf("%zu\\n", sizeof({s.__name__}));')
        want.append(ctypes.sizeof(s))
        for f, _ in s._fields_:
            lines.append(f'printf("%zu\\n", offsetof({s.__name__}, {f}));')
            want.append(getattr(s, f).offset)
    src = tmp_path / "layout.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "kda.h"\nint main(void)\n{\n' + "\n".join(lines) + "\nreturn 0;\n}\n")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(kbuild._nvcc())))
    exe = tmp_path / "layout"
    subprocess.run([cc, "-std=c11", "-I", os.path.join(root, "include"), "-I", os.path.join(cuda, "include"), str(src), "-o", str(exe)], check=True)
    got = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()
    assert [int(x) for x in got] == want
