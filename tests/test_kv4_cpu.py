"""The 4-bit K/V cache without a GPU: sizes, refusals, and pins of its oracle."""
import ctypes

import numpy as np
import pytest

import ulysses_sequence_attention_repack_b200 as U
from oracle import kv4_oracle as orc
from ulysses_sequence_attention_repack_b200 import _lib


def _code(*args):
    try:
        U.ulysses_kv4_plan(*args)
        return 0
    except U.UlyssesError as e:
        return e.code


def test_plan_refusals():
    assert _code(1, 1, 128, 32) == 0
    assert _code(1024, 63, 128, 64) == 0
    assert _code(1, 8, 64, 32) == _lib.ULYSSES_ERR_UNSUPPORTED
    assert _code(0, 8, 128, 32) == _lib.ULYSSES_ERR_ARG
    assert _code(1, 0, 128, 32) == _lib.ULYSSES_ERR_ARG
    assert _code(1, 8, 128, 0) == _lib.ULYSSES_ERR_ARG
    assert _code(1, 8, 128, -32) == _lib.ULYSSES_ERR_ARG
    assert _code(1, 8, 128, 33) == _lib.ULYSSES_ERR_ALIGN
    assert _code(1025, 1, 128, 32) == _lib.ULYSSES_ERR_UNSUPPORTED
    assert _code(1, 1025, 128, 32) == _lib.ULYSSES_ERR_UNSUPPORTED
    assert _code(1024, 64, 128, 32) == _lib.ULYSSES_ERR_UNSUPPORTED
    assert _code(1, 1, 128, 1 << 31) == _lib.ULYSSES_ERR_UNSUPPORTED
    assert _code((1 << 32) + 1, 1, 128, 32) == _lib.ULYSSES_ERR_UNSUPPORTED      # no wrapping into an int32
    assert _code(1, -(1 << 32) + 1, 128, 32) == _lib.ULYSSES_ERR_ARG
    assert U.load().ulysses_kv4_plan(None, 1, 1, 128, 32) == _lib.ULYSSES_ERR_ARG


def test_a_capacity_does_not_wrap_into_64_bits():
    assert _code(1, 1, 128, (1 << 64) + 32) == _lib.ULYSSES_ERR_ALIGN   # held at 2^63 - 1
    assert _code(1, 1, 128, -(1 << 64) + 32) == _lib.ULYSSES_ERR_ARG


@pytest.mark.parametrize("B,H,cap", [(1, 1, 32), (3, 8, 1024), (1, 56, 104448), (24, 8, 8192)])
def test_sizes(B, H, cap):
    kv = U.ulysses_kv4_plan(B, H, 128, cap)
    n = B * H * cap
    assert kv.weight_offset == n * 144
    assert kv.position_offset == n * 148
    assert kv.cache_bytes == n * 152
    assert kv.workspace_bytes(H, 1) > 0
    extra = kv.workspace_bytes(2 * H, 3, True) - kv.workspace_bytes(2 * H, 3)
    assert 0 <= extra - 4 * B * H * 6 * cap < 8 * B * H * 6 + 256      # the logits, and a pair for each row
    assert kv.workspace_bytes(H + 1 if H > 1 else 0, 1) == 0
    assert kv.workspace_bytes(H, 0) == 0


ROWS = dict(cache=0x10000000, k=0x20000000, v=0x30000000, rows=16, ts=1024, hs=128, rs=0, hl=8, cu=0x40000000,
            start=0x40001000)


def _rows(name, **kw):
    a = dict(ROWS, **kw)
    kv = U.ulysses_kv4_plan(2, 8, 128, 64)
    args = [kv.handle if a.get("kv", 1) else None, a["cache"], a["k"], a["v"], a["rows"], a["ts"], a["hs"], a["rs"],
            a["hl"], a["cu"], a["start"]]
    if name == "append":
        return U.load().ulysses_kv4_append(*args, a.get("pos0"), None)
    return U.load().ulysses_kv4_load(*args, None)


@pytest.mark.parametrize("name", ["append", "load"])
def test_row_refusals(name):
    ok, arg, align = _lib.ULYSSES_ERR_CUDA, _lib.ULYSSES_ERR_ARG, _lib.ULYSSES_ERR_ALIGN
    cuda = _lib.load and __import__("torch").cuda.is_available()
    if not cuda:   # a good call is refused for the missing device alone
        assert _rows(name) == ok
        assert _rows(name, ts=3 * 1024, v=0x20000000 + 2048) == ok                 # planes of packed rows
        assert _rows(name, hl=4, ts=512, rs=16 * 512 * 3, v=0x20000000 + 16 * 512 * 2) == ok   # planes of a head slab
    for null in ("kv", "cache", "k", "v", "cu", "start"):
        assert _rows(name, **{null: None}) == arg, null
    assert _rows(name, rows=-1) == arg
    assert _rows(name, rows=1 << 31, ts=8) == _lib.ULYSSES_ERR_UNSUPPORTED
    assert _rows(name, hl=0) == _lib.ULYSSES_ERR_DIVISIBILITY
    assert _rows(name, hl=3) == _lib.ULYSSES_ERR_DIVISIBILITY
    assert _rows(name, ts=-1024) == arg
    assert _rows(name, ts=1 << 60) == arg
    assert _rows(name, ts=1028) == align
    assert _rows(name, hs=132) == align
    assert _rows(name, hl=4, rs=4) == align
    for p in ("cache", "k", "v"):
        assert _rows(name, **{p: ROWS[p] + 8}) == align
    for p in ("cu", "start"):
        assert _rows(name, **{p: ROWS[p] + 2}) == align
    kv = U.ulysses_kv4_plan(2, 8, 128, 64)
    assert _rows(name, k=ROWS["cache"] + kv.cache_bytes - 16) == arg               # rows inside the cache
    if name == "append":
        assert _rows(name, pos0=0x40002001) == align
        assert _rows(name, cu=ROWS["cache"]) == arg
        assert _rows(name, pos0=ROWS["cache"] + 64) == arg
    else:                                                                            # destination rows that share elements
        assert _rows(name, ts=0) == arg
        assert _rows(name, hs=0) == arg
        assert _rows(name, hs=64) == arg
        assert _rows(name, ts=512) == arg
        assert _rows(name, v=ROWS["k"]) == arg
        assert _rows(name, v=ROWS["k"] + 512) == arg
        assert _rows(name, cu=ROWS["k"] + 32) == arg
        assert _rows(name, start=ROWS["v"] + 32) == arg


ATTN = dict(cache=0x10000000, q=0x20000000, qh=16, ql=2, ts=2048, hs=128, out=0x30000000, lse=0x38000000,
            lengths=0x40000000, scale=0.1, flags=0, ws=0x50000000, wb=1 << 30)


def _attn(**kw):
    a = dict(ATTN, **kw)
    kv = U.ulysses_kv4_plan(2, 8, 128, 64)
    return U.load().ulysses_kv4_attn(kv.handle if a.get("kv", 1) else None, a["cache"], a["q"], a["qh"], a["ql"],
                                     a["ts"], a["hs"], a["out"], a["lse"], a["lengths"], a["scale"], a["flags"],
                                     a["ws"], a["wb"], None)


def test_attention_refusals():
    arg, align = _lib.ULYSSES_ERR_ARG, _lib.ULYSSES_ERR_ALIGN
    kv = U.ulysses_kv4_plan(2, 8, 128, 64)
    if not __import__("torch").cuda.is_available():
        assert _attn() == _lib.ULYSSES_ERR_CUDA
        assert _attn(lse=None) == _lib.ULYSSES_ERR_CUDA
        assert _attn(wb=kv.workspace_bytes(16, 2)) == _lib.ULYSSES_ERR_CUDA
        assert _attn(flags=3, wb=kv.workspace_bytes(16, 2, True)) == _lib.ULYSSES_ERR_CUDA
    for null in ("kv", "cache", "q", "out", "lengths"):
        assert _attn(**{null: None}) == arg, null
    assert _attn(flags=4) == arg
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        assert _attn(scale=scale) == arg
    assert _attn(qh=0) == arg
    assert _attn(ql=0) == arg
    assert _attn(qh=12) == _lib.ULYSSES_ERR_DIVISIBILITY
    assert _attn(ql=1 << 30) == _lib.ULYSSES_ERR_UNSUPPORTED
    assert _attn(ts=-8) == arg
    assert _attn(ts=1 << 60) == arg
    assert _attn(ts=2052) == align
    assert _attn(hs=4) == align
    for p in ("cache", "q", "out", "ws"):
        assert _attn(**{p: ATTN[p] + 8}) == align, p
    for p in ("lse", "lengths"):
        assert _attn(**{p: ATTN[p] + 2}) == align, p
    assert _attn(ws=None) == _lib.ULYSSES_ERR_WORKSPACE
    assert _attn(wb=kv.workspace_bytes(16, 2) - 1) == _lib.ULYSSES_ERR_WORKSPACE
    assert _attn(flags=2, wb=kv.workspace_bytes(16, 2, True) - 1) == _lib.ULYSSES_ERR_WORKSPACE
    assert _attn(out=ATTN["q"]) == arg
    assert _attn(out=ATTN["cache"] + 4096) == arg
    assert _attn(lse=ATTN["out"] + 256) == arg
    assert _attn(ws=ATTN["out"]) == arg
    assert _attn(lengths=ATTN["ws"] + 64) == arg


EVICT = dict(src=0x10000000, dst=0x20000000, lengths=0x40000000, new=0x40001000, keep=32, sink=4, recent=8)


def _evict(other=(2, 8, 128, 32), **kw):
    a = dict(EVICT, **kw)
    kv, to = U.ulysses_kv4_plan(2, 8, 128, 64), U.ulysses_kv4_plan(*other)
    return U.load().ulysses_kv4_evict(kv.handle if a.get("kv", 1) else None, a["src"],
                                      to.handle if a.get("to", 1) else None, a["dst"], a["lengths"], a["new"],
                                      a["keep"], a["sink"], a["recent"], None)


def test_eviction_refusals():
    arg, align = _lib.ULYSSES_ERR_ARG, _lib.ULYSSES_ERR_ALIGN
    if not __import__("torch").cuda.is_available():
        assert _evict() == _lib.ULYSSES_ERR_CUDA
        assert _evict(sink=16, recent=16) == _lib.ULYSSES_ERR_CUDA
    for null in ("kv", "to", "src", "dst", "lengths", "new"):
        assert _evict(**{null: None}) == arg, null
    assert _evict(other=(2, 4, 128, 32)) == arg
    assert _evict(other=(1, 8, 128, 32)) == arg
    assert _evict(keep=0) == arg
    assert _evict(keep=33) == arg                    # past the destination's capacity
    assert _evict(sink=-1) == arg
    assert _evict(recent=-1) == arg
    assert _evict(sink=25) == arg                    # more protected slots than kept ones
    assert _evict(sink=(1 << 31) - 1, recent=(1 << 31) - 1) == arg
    for p in ("src", "dst"):
        assert _evict(**{p: EVICT[p] + 8}) == align
    for p in ("lengths", "new"):
        assert _evict(**{p: EVICT[p] + 2}) == align
    assert _evict(dst=EVICT["src"]) == arg
    assert _evict(dst=EVICT["src"] + 1024) == arg
    assert _evict(new=EVICT["lengths"]) == arg
    assert _evict(new=EVICT["src"] + 64) == arg
    assert _evict(lengths=EVICT["dst"] + 64) == arg


def test_binding_refuses_what_is_no_cuda_tensor():
    import torch
    kv = U.ulysses_kv4_plan(1, 2, 128, 32)
    x = torch.zeros((4, 2, 128), dtype=torch.bfloat16)
    c, i = torch.zeros(kv.cache_bytes, dtype=torch.uint8), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(TypeError):
        U.ulysses_kv4_append(kv, c, x, x, i, i)
    with pytest.raises(TypeError):
        U.ulysses_kv4_load(kv, c, x, x, i, i)
    with pytest.raises(TypeError):
        U.ulysses_kv4_attn(kv, c, x[None], x[None], i, 0.1)
    with pytest.raises(TypeError):
        U.ulysses_kv4_evict(kv, c, kv, c, i, i, 4)


# ------------------------------------------------------------------------------------------ the oracle

def test_oracle_bf16_rounding():
    import torch
    g = torch.Generator().manual_seed(0)
    x = torch.cat([torch.randn(500, generator=g), torch.randn(200, generator=g) * 1e-39,
                   torch.tensor([0.0, -0.0, 1.0, 3.3895e38, 1.00390625, 1.01171875, 9.2e-41, float("inf")])])
    want = x.to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)
    assert np.array_equal(orc.f64_to_bf16(x.double().numpy()), want)


def test_oracle_row_by_hand():
    x = np.zeros(128)
    x[:16] = np.arange(16)            # group 0: m = 0, s = 1, codes 0..15 then 0
    x[64:] = -3.0                     # group 1: constant: s = 0, m = -3
    rows, meta = orc.quantise_row(x)
    assert meta.tolist() == [0x3F80, 0x0000, 0x0000, 0xC040]
    assert rows[:4].tolist() == [0x10, 0x32, 0x54, 0x76]      # chunk 0, group 0: dims 0..7
    assert rows[8:12].tolist() == [0x98, 0xBA, 0xDC, 0xFE]    # chunk 1, group 0: dims 8..15
    assert not rows[4:8].any() and not rows[12:].any()


def test_oracle_round_trip_is_within_half_a_step():
    rng = np.random.default_rng(1)
    for scale in (1e-30, 1.0, 1e30):
        x = orc.bf16_to_f64(orc.f64_to_bf16(rng.standard_normal(128) * scale))
        rows, meta = orc.quantise_row(x)
        raw = np.zeros(4608 + 8 * 32, dtype=np.uint8)
        c = orc.Cache(raw, 1, 1, 32)
        c.row(0, 0, 5, 1)[:] = rows
        c.meta(0, 0, 5, 1)[:] = meta
        got, steps = c.values(0, 0, 5, 6, 1)
        for w in (0, 1):
            # half a step, and at the top 15 steps of a scale rounded by 2^-8 of itself or less
            tol = steps[0, w] * (0.5 + 15 * 2.0 ** -8)
            assert np.abs(got[0, 64 * w:64 * w + 64] - x[64 * w:64 * w + 64]).max() <= tol


def test_oracle_refuses_what_is_not_finite():
    for bad in (np.inf, -np.inf, np.nan):
        x = np.ones(128)
        x[70] = bad
        rows, meta = orc.quantise_row(x)
        assert meta.tolist() == [0, 0x3F80, 0x7FC0, 0x7FC0] and not rows.any()
    x = np.ones(128) * 3.3895313892515355e38
    x[0] = -x[0]
    assert orc.quantise_row(x)[1].tolist()[:2] == [0x7FC0, 0x7FC0]


def test_oracle_kept_slots():
    w = np.array([5, 1, 3, 3, np.nan, 3, 0, 9, 2, 2], dtype=np.float32)
    assert orc.kept_slots(w, 10, 10, 0, 0).tolist() == list(range(10))
    assert orc.kept_slots(w, 10, 3, 0, 0).tolist() == [0, 2, 7]
    assert orc.kept_slots(w, 10, 4, 0, 0).tolist() == [0, 2, 3, 7]
    assert orc.kept_slots(w, 10, 5, 2, 2).tolist() == [0, 1, 7, 8, 9]
    assert orc.kept_slots(w, 10, 9, 0, 0).tolist() == [0, 1, 2, 3, 5, 6, 7, 8, 9]
    assert orc.kept_slots(w, 4, 4, 2, 2).tolist() == [0, 1, 2, 3]
