"""Refusals of the one-decay rule, the convolution, the block norms and the
slot operations: every one of them before any launch, without a GPU."""
import ctypes

import pytest

import linear_attention_serving_kda_gb300 as kda
from linear_attention_serving_kda_gb300 import build as kbuild

FAKE = 1 << 20  # 16-byte-aligned addresses far apart; never dereferenced
STEP = 1 << 34
INVALID, GEOMETRY = kda.KDA_ERR_INVALID_ARGUMENT, kda.KDA_ERR_UNSUPPORTED_GEOMETRY


@pytest.fixture(scope="module", autouse=True)
def lib():
    kbuild.build()
    return kda.load()


def addr(i):
    return FAKE + i * STEP


def _gdn(**kw):
    base = dict(num_heads_k=2, num_heads_v=4, head_dim_k=128, head_dim_v=128, A_log=addr(20), dt_bias=addr(21), num_slots=4)
    base.update(kw)
    return kda.GdnParams(**base)


ROWS = dict(q=addr(1), k=addr(2), v=addr(3), gate=addr(4), beta=addr(5), slots=None, rec_state=addr(6), out=addr(7))


def _decode(p, B=2, **over):
    a = {**ROWS, **over}
    return kda.kda_gdn_decode(p, B, *a.values(), None, 0)


def _prefill(p, N=2, T=8, cu=addr(8), ws=None, nws=0, **over):
    a = {**ROWS, **over}
    return kda.kda_gdn_prefill_varlen(p, cu, N, T, *a.values(), ws, nws, None, 0)


@pytest.mark.parametrize("kw,rc", [
    (dict(num_heads_k=0), INVALID), (dict(num_heads_v=5), INVALID), (dict(num_heads_v=0), INVALID),
    (dict(num_heads_k=1025, num_heads_v=1025), INVALID),
    (dict(head_dim_k=96), GEOMETRY), (dict(head_dim_v=256), GEOMETRY), (dict(head_dim_v=0), GEOMETRY),
    (dict(l2_norm=2), INVALID), (dict(l2_eps=-1.0), INVALID), (dict(l2_eps=float("nan")), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(io_dtype=3), INVALID), (dict(out_dtype=-1), INVALID),
    (dict(io_dtype=kda.KDA_DTYPE_F32, out_dtype=kda.KDA_DTYPE_BF16), INVALID), (dict(num_slots=0), INVALID),
    (dict(q_row_stride=248), INVALID), (dict(k_row_stride=260), INVALID), (dict(v_row_stride=-8), INVALID),
    (dict(v_row_stride=1 << 29), INVALID), (dict(A_log=None), INVALID), (dict(dt_bias=addr(21) + 4), INVALID),
])
def test_gdn_params(kw, rc):
    p = _gdn(**kw)
    assert _decode(p) == rc and _prefill(p) == rc
    assert kda.kda_gdn_prefill_workspace_bytes(p, 2, 8) == 0


def test_gdn_pointers():
    p = _gdn()
    for name in ("q", "k", "v", "gate", "beta", "rec_state", "out"):
        for bad in (None, ROWS[name] + 8):
            assert _decode(p, **{name: bad}) == INVALID and _prefill(p, **{name: bad}) == INVALID, name
    assert _decode(p, slots=addr(9) + 4) == INVALID
    assert _prefill(p, cu=None) == INVALID and _prefill(p, cu=addr(8) + 4) == INVALID
    assert _decode(p, B=-1) == INVALID and _prefill(p, N=-1) == INVALID and _prefill(p, T=-1) == INVALID
    assert _decode(p, B=1 << 29) == INVALID
    # nothing to do
    assert _decode(p, B=0) == kda.KDA_OK and _prefill(p, N=0) == kda.KDA_OK and _prefill(p, T=0) == kda.KDA_OK
    # outputs and states apart from the inputs, to the last byte
    rows = 2 * 4 * 128 * 2
    assert _decode(p, out=ROWS["v"] + rows - 16) == INVALID
    assert _decode(p, out=ROWS["rec_state"] + 4 * 4 * 128 * 128 * 4 - 16) == INVALID
    assert _decode(p, rec_state=ROWS["k"]) == INVALID
    wide = _gdn(q_row_stride=1024)
    assert _decode(wide, out=ROWS["q"] + 1024 * 2 + 256) == INVALID


def test_gdn_workspace():
    p = _gdn()
    need = kda.kda_gdn_prefill_workspace_bytes(p, 1, 4096)
    assert kda.kda_gdn_prefill_workspace_bytes(p, -1, 4096) == 0
    assert kda.kda_gdn_prefill_workspace_bytes(_gdn(io_dtype=kda.KDA_DTYPE_F32, out_dtype=kda.KDA_DTYPE_F32), 1, 4096) == 0
    if need:
        assert _prefill(p, N=1, T=4096) == kda.KDA_ERR_WORKSPACE
        assert _prefill(p, N=1, T=4096, ws=addr(10), nws=need - 1) == kda.KDA_ERR_WORKSPACE
        assert _prefill(p, N=1, T=4096, ws=addr(10) + 8, nws=need) == kda.KDA_ERR_WORKSPACE


def test_conv():
    def call(decode=False, n=2, T=8, cu=addr(1), x=addr(2), slots=None, st=addr(3), y=addr(4), **kw):
        p = kda.ConvParams(**{**dict(channels=64, conv_kernel=4, conv_weight=addr(9), num_slots=3), **kw})
        if decode:
            return kda.kda_conv_decode(p, n, x, slots, st, y, None, 0)
        return kda.kda_conv_varlen(p, cu, n, T, x, slots, st, y, None, 0)

    for d in (False, True):
        for kw, rc in ((dict(conv_kernel=5), GEOMETRY), (dict(conv_kernel=1), GEOMETRY), (dict(channels=0), INVALID),
                       (dict(channels=12), GEOMETRY), (dict(channels=(1 << 20) + 8), GEOMETRY), (dict(io_dtype=2), INVALID),
                       (dict(num_slots=0), INVALID), (dict(conv_weight=None), INVALID), (dict(x=None), INVALID),
                       (dict(st=addr(3) + 8), INVALID), (dict(y=None), INVALID), (dict(slots=addr(5) + 2), INVALID),
                       (dict(n=-1), INVALID), (dict(y=addr(2)), INVALID), (dict(y=addr(2) + 128), INVALID),
                       (dict(y=addr(3)), INVALID), (dict(st=addr(2)), INVALID)):
            assert call(d, **kw) == rc, (d, kw)
        assert call(d, n=0) == kda.KDA_OK
    assert call(cu=None) == INVALID and call(T=-1) == INVALID and call(T=0) == kda.KDA_OK


def test_block_norm():
    def call(rows=4, y=addr(1), gate=None, res=None, h=addr(4), x=addr(5), **kw):
        return kda.kda_block_norm(kda.NormParams(**{**dict(dim=256), **kw}), rows, y, gate, res, h, x, 0)

    F32 = kda.KDA_DTYPE_F32
    for kw, rc in ((dict(dim=0), INVALID), (dict(dim=12), GEOMETRY), (dict(dim=16392), GEOMETRY), (dict(gate_act=3), INVALID),
                   (dict(post_norm=2), INVALID), (dict(residual_scale=float("nan")), INVALID), (dict(norm_eps=-1.0), INVALID),
                   (dict(io_dtype=9), INVALID), (dict(res_dtype=9), INVALID), (dict(post_weight=addr(6) + 4), INVALID),
                   (dict(rows=-1), INVALID), (dict(rows=1 << 31), INVALID), (dict(y=None), INVALID), (dict(gate_act=1), INVALID),
                   (dict(res=addr(3) + 2), INVALID), (dict(h=None, x=None), INVALID), (dict(h=addr(4) + 8), INVALID),
                   (dict(x=addr(4)), INVALID),                                # both outputs in one buffer
                   (dict(h=addr(1) + 512), INVALID),                          # part of an input
                   (dict(h=addr(1), res_dtype=F32), INVALID),                 # an input of another type
                   (dict(res=addr(4), x=addr(4) + 16), INVALID),
                   (dict(pre_weight=addr(5)), INVALID)):
        assert call(**kw) == rc, kw
    assert call(rows=0) == kda.KDA_OK


def test_slots():
    def pool(**kw):
        return kda.SlotPool(**{**dict(pool=addr(1), num_layers=2, num_slots=8, slot_bytes=64, layer_stride_bytes=512), **kw})

    bad = [dict(pool=None), dict(pool=addr(1) + 8), dict(num_layers=0), dict(num_slots=0), dict(slot_bytes=0),
           dict(slot_bytes=40), dict(layer_stride_bytes=496), dict(layer_stride_bytes=520),
           dict(num_slots=kda.KDA_MAX_POOL_SLOTS + 1, layer_stride_bytes=1 << 40),
           dict(slot_bytes=1 << 62, layer_stride_bytes=1 << 62), dict(layer_stride_bytes=1 << 62, num_layers=1000)]
    for kw in bad:
        p = pool(**kw)
        assert kda.kda_slots_copy(p, 2, addr(2), addr(3), None, 0) == INVALID, kw
        assert kda.kda_slots_zero(p, 2, addr(2), None, 0) == INVALID, kw
        assert kda.kda_slots_compact_plan(p, addr(2), addr(3), addr(4), addr(5), 0) == INVALID, kw
    p = pool()
    assert kda.kda_slots_copy(p, -1, addr(2), addr(3), None, 0) == INVALID
    assert kda.kda_slots_copy(p, 0, None, None, None, 0) == kda.KDA_OK and kda.kda_slots_zero(p, 0, None, None, 0) == kda.KDA_OK
    assert kda.kda_slots_copy(p, 2, None, addr(3), None, 0) == INVALID
    assert kda.kda_slots_copy(p, 2, addr(1) + 960, addr(3), None, 0) == INVALID   # a list inside the pool
    assert kda.kda_slots_zero(p, 2, addr(2) + 4, None, 0) == INVALID
    assert kda.kda_slots_compact_plan(p, addr(2), addr(3), addr(3) + 16, addr(5), 0) == INVALID
    assert kda.kda_slots_compact_plan(p, addr(2), addr(3), addr(4), None, 0) == INVALID


def test_struct_sizes():
    """The binding's structures lay out as the header's (natural alignment, no holes but before pointers)."""
    k = kda.kda
    assert ctypes.sizeof(k.kda_gdn_params) == 40 + 24 + 16
    assert ctypes.sizeof(k.kda_conv_params) == 24
    assert ctypes.sizeof(k.kda_norm_params) == 32 + 16
    assert ctypes.sizeof(k.kda_slot_pool) == 32


def test_lists_and_workspace_apart_from_what_is_written():
    p = _gdn()
    need = kda.kda_gdn_prefill_workspace_bytes(p, 2, 8)
    assert _prefill(p, cu=ROWS["out"]) == INVALID and _prefill(p, slots=ROWS["rec_state"] + 64) == INVALID
    assert _decode(p, slots=ROWS["out"]) == INVALID and _decode(_gdn(A_log=ROWS["out"])) == INVALID
    for other in ("q", "gate", "out", "rec_state"):
        assert _prefill(p, ws=ROWS[other], nws=need) == INVALID, other
        assert _prefill(p, ws=ROWS[other] - need + 16, nws=need) == INVALID, other
    conv = kda.ConvParams(channels=64, conv_kernel=4, conv_weight=addr(9), num_slots=3)
    assert kda.kda_conv_varlen(conv, addr(4), 2, 8, addr(2), None, addr(3), addr(4), None, 0) == INVALID
    assert kda.kda_conv_decode(conv, 2, addr(2), addr(3), addr(3), addr(4), None, 0) == INVALID
    conv = kda.ConvParams(channels=64, conv_kernel=4, conv_weight=addr(4), num_slots=3)
    assert kda.kda_conv_varlen(conv, addr(1), 2, 8, addr(2), None, addr(3), addr(4), None, 0) == INVALID
    conv = kda.ConvParams(channels=64, conv_kernel=4, conv_weight=addr(9), num_slots=3)
    assert kda.kda_conv_varlen(conv, addr(1), (1 << 31) - 1, 1 << 20, addr(2), None, addr(3), addr(4), None, 0) == INVALID


def test_row_counts_past_the_index_range():
    rows = (1 << 31) - 1
    assert _prefill(_gdn(num_heads_k=1, num_heads_v=1, head_dim_k=32, head_dim_v=32), N=1, T=rows) == INVALID
    conv = kda.ConvParams(channels=8, conv_kernel=2, conv_weight=addr(9), num_slots=3)
    far = 1 << 50
    assert kda.kda_conv_varlen(conv, addr(1), 1, rows, far, None, addr(3), 2 * far, None, 0) == INVALID
    assert kda.kda_conv_decode(conv, rows, far, None, addr(3), 2 * far, None, 0) == INVALID


def test_sequence_counts_past_the_index_range():
    """The search for a row tile counts in blocks of 32 sequences: counts within 31 of the index range's end wrapped."""
    conv = kda.ConvParams(channels=8, conv_kernel=2, conv_weight=addr(9), num_slots=3)
    far = 1 << 50
    for N in ((1 << 31) - 1, (1 << 31) - 31, kda.KDA_MAX_ROWS + 1):
        assert kda.kda_conv_varlen(conv, far, N, 8, addr(2), None, addr(3), addr(4), None, 0) == INVALID
        assert _prefill(_gdn(num_heads_k=1, num_heads_v=1), N=N, T=8, cu=far) == INVALID
    assert kda.kda_conv_varlen(conv, far, kda.KDA_MAX_ROWS, 16, addr(2), None, addr(3), addr(4), None, 0) == INVALID


def test_struct_layouts_as_c_sees_them(tmp_path):
    """Sizes and offsets of every parameter structure from a C program built against the header."""
    import os
    import shutil
    import subprocess

    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    k = kda.kda
    structs = [k.kda_params, k.kda_gdn_params, k.kda_conv_params, k.kda_norm_params, k.kda_slot_pool]
    lines, want = [], []
    for s in structs:
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
    subprocess.run([cc, "-std=c11", "-I", os.path.join(root, "include"), "-I", os.path.join(cuda, "include"), str(src), "-o", str(exe)],
                   check=True)
    got = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()
    assert [int(x) for x in got] == want
