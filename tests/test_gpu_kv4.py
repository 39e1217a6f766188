"""The 4-bit K/V cache on the GPU against its fp64 oracle.

Quantised bytes, loaded rows, kept slots, positions and lengths are compared
exactly.  Attention is compared element by element with a bound derived from
the kernel's arithmetic (`bound`); no tolerance here was fitted to a run.
"""
import math

import numpy as np
import pytest
from oracle import kv4_oracle as orc

import ulysses_sequence_attention_repack_b200 as U

pytestmark = pytest.mark.gpu

D = 128
SCALE = 1.0 / math.sqrt(D)


def _bits(t):
    import torch
    return t.detach().contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def _f64(t):
    return orc.bf16_to_f64(_bits(t))


def _i32(v, dev):
    import torch
    return torch.tensor(v, dtype=torch.int32, device=dev)


def _host(kv, cache):
    return orc.Cache(cache.cpu().numpy().copy(), kv.batch, kv.heads, kv.capacity)


def _cu(lens):
    return [0, *np.cumsum(lens).tolist()]


def _make(dev, lens, heads, capacity, seed, spread=1.0):
    """A plan, a cache filled by append from random rows (behind every length: bytes that decode to
    NaN), and its host copy."""
    import torch
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    kv = U.ulysses_kv4_plan(len(lens), heads, D, capacity)
    cache = torch.full((kv.cache_bytes,), 0xFF, dtype=torch.uint8, device=dev)
    n = sum(lens)
    k = (torch.randn((n, heads, D), generator=g, device=dev) * spread).to(torch.bfloat16)
    v = (torch.randn((n, heads, D), generator=g, device=dev) + 0.5).to(torch.bfloat16)
    U.ulysses_kv4_append(kv, cache, k, v, _i32(_cu(lens), dev), _i32([0] * len(lens), dev))
    return kv, cache, k, v


# ------------------------------------------------------------------------------------------ append and load

def _check_append(kv, cache, k, v, lens, start, pos0=None):
    host = _host(kv, cache)
    kk, vv = _f64(k), _f64(v)
    at = 0
    for b, n in enumerate(lens):
        for i in range(n):
            slot = start[b] + i
            for h in range(kv.heads):
                for plane, x in ((0, kk), (1, vv)):
                    rows, meta = orc.quantise_row(x[at + i, h])
                    assert np.array_equal(host.row(b, h, slot, plane), rows), (b, h, slot, plane)
                    got = host.meta(b, h, slot, plane)
                    # -0 and +0 are one minimum
                    assert np.array_equal(got & np.where(got == 0x8000, 0, 0xFFFF),
                                          meta & np.where(meta == 0x8000, 0, 0xFFFF)), (b, h, slot, plane, got, meta)
                assert host.weight[b, h, slot] == 0
                assert host.pos[b, h, slot] == (slot if pos0 is None else pos0[b] + i)
        at += n
    return host


@pytest.mark.parametrize("lens,start,heads,capacity", [
    ([1], [0], 1, 32), ([1, 1, 1], [31, 32, 63], 3, 64), ([37, 0, 9, 64], [5, 0, 87, 0], 7, 96), ([33], [30], 56, 64)])
def test_append_writes_the_oracle_bytes(gpu, lens, start, heads, capacity):
    import torch
    g = torch.Generator(device=gpu)
    g.manual_seed(sum(lens))
    kv = U.ulysses_kv4_plan(len(lens), heads, D, capacity)
    cache = torch.full((kv.cache_bytes,), 0xA5, dtype=torch.uint8, device=gpu)
    packed = torch.randn((sum(lens) + 3, 3, heads, D), generator=g, device=gpu).to(torch.bfloat16)
    k, v = packed[:, 1], packed[:, 2]                 # planes of packed rows; the last three rows are no sequence's
    before = cache.clone()
    pos0 = [1000 * b + 7 for b in range(len(lens))]
    U.ulysses_kv4_append(kv, cache, k, v, _i32(_cu(lens), gpu), _i32(start, gpu), _i32(pos0, gpu))
    host = _check_append(kv, cache, k, v, lens, start, pos0)
    untouched = orc.Cache(before.cpu().numpy().copy(), kv.batch, heads, capacity)
    for b, n in enumerate(lens):
        for slot in set(range(capacity)) - set(range(start[b], start[b] + n)):
            assert np.array_equal(host.row(b, 0, slot, 0), untouched.row(b, 0, slot, 0))
            assert np.array_equal(host.meta(b, heads - 1, slot, 1), untouched.meta(b, heads - 1, slot, 1))
            assert host.pos[b, 0, slot] == untouched.pos[b, 0, slot]
    assert U.ulysses_kv4_last_device_error(kv) == 0


def test_append_of_special_rows(gpu):
    import torch
    rng = np.random.default_rng(3)
    x = rng.standard_normal((14, D))
    x[0] = 0.0
    x[1] = -0.0
    x[2] = 5.5
    x[3, 64:] = np.inf
    x[4, 0] = np.nan
    x[5, 127] = -np.inf
    x[6] *= 1e-38                        # steps below the normal numbers
    x[7] *= 1e37
    x[8, :2] = 3.3895e38, -3.3895e38     # a spread past the fp32 range
    x[9] = np.repeat(np.arange(16), 8)   # every code, no rounding
    x[10] = np.tile([0.0, 0.5, 1.0, 1.5, 2.5, 7.5, 14.5, 15.0], 16)   # on the borders: ties to even
    x[11] = 1.0
    x[11, ::2] = 1.0078125               # two neighbours of a binade
    x[12] *= 1e-41
    x[13] = np.tile([-0.0, 0.0, -1e-30, 1e-30], 32)
    k = torch.tensor(x, device=gpu).to(torch.bfloat16)[:, None]
    v = torch.flip(k, [0]).contiguous()
    kv = U.ulysses_kv4_plan(1, 1, D, 32)
    cache = torch.zeros(kv.cache_bytes, dtype=torch.uint8, device=gpu)
    U.ulysses_kv4_append(kv, cache, k, v, _i32([0, 14], gpu), _i32([0], gpu))
    _check_append(kv, cache, k, v, [14], [0])


@pytest.mark.parametrize("P", [1, 2, 4])
def test_append_and_load_take_planes_of_a_head_slab(gpu, P):
    """T [P, C, Np, Hl, D]: K and V are planes 1 and 2, heads split over ranks."""
    import torch
    g = torch.Generator(device=gpu)
    g.manual_seed(P)
    n, H = 45, 8
    T = torch.randn((P, 3, n, H // P, D), generator=g, device=gpu).to(torch.bfloat16)
    kv = U.ulysses_kv4_plan(1, H, D, 64)
    cache = torch.zeros(kv.cache_bytes, dtype=torch.uint8, device=gpu)
    cu, start = _i32([0, n], gpu), _i32([2], gpu)
    U.ulysses_kv4_append(kv, cache, T[:, 1], T[:, 2], cu, start)
    flat = T.permute(1, 2, 0, 3, 4).reshape(3, n, H, D)
    host = _check_append(kv, cache, flat[1], flat[2], [n], [2])
    back = torch.full_like(T, 7.0)
    U.ulysses_kv4_load(kv, cache, back[:, 1], back[:, 2], cu, start)
    got = back.permute(1, 2, 0, 3, 4).reshape(3, n, H, D)
    assert bool((back[:, 0] == 7).all())
    for h in range(H):
        for plane in (0, 1):
            want, _ = host.values(0, h, 2, 2 + n, plane)
            assert np.array_equal(_bits(got[1 + plane][:, h]), orc.f64_to_bf16(want))


@pytest.mark.parametrize("lens,start", [([1], [0]), ([40, 0, 7], [3, 96, 31]), ([96], [0])])
def test_load_brings_back_the_held_values(gpu, lens, start):
    import torch
    heads = 5
    kv, cache, _, _ = _make(gpu, [96] * len(lens), heads, 96, 5)
    host = _host(kv, cache)
    out = torch.full((sum(lens) + 2, 3, heads, D), 9.0, dtype=torch.bfloat16, device=gpu)
    U.ulysses_kv4_load(kv, cache, out[:, 1], out[:, 2], _i32(_cu(lens), gpu), _i32(start, gpu))
    at = 0
    for b, n in enumerate(lens):
        for h in range(heads):
            for plane in (0, 1):
                want, _ = host.values(b, h, start[b], start[b] + n, plane)
                # m + s n, rounded once
                assert np.array_equal(_bits(out[at:at + n, 1 + plane, h]), orc.f64_to_bf16(want))
        at += n
    assert bool((out[at:] == 9).all()) and bool((out[:, 0] == 9).all())      # rows of no sequence, the other plane


def test_rows_outside_the_cache_are_skipped_and_reported(gpu):
    import torch
    kv, cache, k, v = _make(gpu, [32, 32], 2, 32, 6)
    before = cache.clone()
    rows = k[:8].contiguous()
    for start in ([32, 0], [-8, 0], [1 << 30, 0]):
        U.ulysses_kv4_append(kv, cache, rows, rows, _i32([0, 8, 8], gpu), _i32(start, gpu))
        assert U.ulysses_kv4_last_device_error(kv) == 16
        assert torch.equal(cache, before)
    out = torch.full((8, 2, D), 3.0, dtype=torch.bfloat16, device=gpu)
    U.ulysses_kv4_load(kv, cache, out, torch.empty_like(out), _i32([0, 8, 8], gpu), _i32([28, 0], gpu))
    assert U.ulysses_kv4_last_device_error(kv) == 16
    assert bool((out[4:] == 3).all()) and not bool((out[:4] == 3).all())
    # prefix sums that are none: rows below the first and at or past the last are no sequence's
    U.ulysses_kv4_append(kv, cache, rows, rows, _i32([8, 8, 3], gpu), _i32([0, 0], gpu))
    assert torch.equal(cache, before)
    assert U.ulysses_kv4_last_device_error(kv) == 0


# ------------------------------------------------------------------------------------------ attention

def bound(q, k, v, vs, scale, o, p):
    """Largest |kernel - exact| of an output row, element by element.

    u16 = 2^-11 is half a step of fp16, u = 2^-24 of fp32, bf16 has 2^-8.
    * z: sums of at most 130 fp32 terms whose magnitudes sum to Z, in whatever order and, on the
      tensor core, possibly truncated (2 u a step): 260 u Z, times the slope of exp and twice,
      since the normaliser has it too;
    * p: exp2 (2^-22 of itself) and its fp32 argument (u |z| log2 e, inside the above);
    * w = p s rounded to fp16: u16 of itself, and at least half the smallest step: with
      w = p s 2^(5 - c), s >= 2^c somewhere, that is 2^-25 2^-5 of the largest step, per slot;
      it multiplies codes of at most 15;
    * sums over the slots in fp32, the tensor core's truncated: 2 u per term of magnitudes p |code s| and p |m|;
      a CTA sums up to n terms one after another;
    * the result's rounding to bf16.
    """
    n = k.shape[0]
    if n == 0:
        return np.zeros(D)
    u = 2.0 ** -24
    # a held value is m + s n with 0 <= n <= 15, so |m| and |s n| are at most |x| + 15 s
    mag = np.abs(v) + 15 * np.repeat(vs, 64, axis=1)
    zmax = np.max(scale * ((np.abs(k) + 2 * np.abs(k).max(1, keepdims=True)) @ np.abs(q)))
    rel = 2 * 260 * u * zmax + 2.0 ** -21
    w = (p[:, None] * 15 * np.repeat(vs, 64, axis=1)).sum(0) * 2.0 ** -11
    tiny = n * 15 * np.repeat(vs.max(0), 64) * 2.0 ** -30
    sums = 2 * u * n * (p[:, None] * mag).sum(0)
    core = rel * (p[:, None] * mag).sum(0) + w + tiny + sums
    return core + (np.abs(o) + core) * 2.0 ** -8


def _check_attn(kv, host, q, out, lse, lengths, causal, weights=None, before=None, scale=SCALE):
    B, q_len, q_heads, _ = q.shape
    G = q_heads // kv.heads
    qq, oo = _f64(q), _f64(out)
    ls = lse.cpu().numpy().astype(np.float64) if lse is not None else None
    for b in range(B):
        for h in range(kv.heads):
            n = lengths[b]
            k, ks = host.values(b, h, 0, n, 0)
            v, vs = host.values(b, h, 0, n, 1)
            total = np.zeros(n)
            slack = np.zeros(n)
            for i in range(q_len):
                m = max(0, n - q_len + i + 1) if causal else n
                for j in range(h * G, (h + 1) * G):
                    o, z, p = orc.attention(qq[b, i, j], k[:m], v[:m], scale)
                    tol = bound(qq[b, i, j], k[:m], v[:m], vs[:m], scale, o, p)
                    err = np.abs(oo[b, i, j] - o)
                    assert np.all(err <= tol), (b, i, j, float((err / np.maximum(tol, 1e-30)).max()))
                    if ls is not None and m == 0:
                        assert ls[b, j, i] == -np.inf
                    if m == 0:
                        continue
                    zabs = scale * np.max((np.abs(k[:m]) + 2 * np.abs(k[:m]).max(1, keepdims=True)) @
                                          np.abs(qq[b, i, j])) / np.log(2.0)
                    dz = 2 * 260 * 2.0 ** -24 * zabs + 2.0 ** -20 + 2.0 ** -23 * abs(z)
                    if ls is not None:
                        assert abs(ls[b, j, i] - z) <= dz, (b, i, j, ls[b, j, i], z)
                    total[:m] += p
                    slack[:m] += p * 2 * dz + 2.0 ** -126
            if weights is not None:
                got = weights[b, h].astype(np.float64) - before[b, h].astype(np.float64)
                room = slack + 2.0 ** -23 * (G * q_len + 1) * (total + np.abs(before[b, h][:n]) + np.abs(got[:n]))
                assert np.all(np.abs(got[:n] - total) <= room), (b, h, np.abs(got[:n] - total).max())
                assert np.array_equal(weights[b, h][n:].view(np.int32), before[b, h][n:].view(np.int32))


def _run_attn(dev, lens, heads, G, q_len, capacity, seed, causal=False, weights=False, want_lse=True, spread=1.0,
              qscale=1.0):
    import torch
    kv, cache, _, _ = _make(dev, lens, heads, capacity, seed, spread)
    g = torch.Generator(device=dev)
    g.manual_seed(seed + 1)
    wide = (torch.randn((len(lens), q_len, heads * G + 1, 2, D), generator=g, device=dev) * qscale).to(torch.bfloat16)
    q = wide[:, :, 1:, 1]                                # rows and heads with strides of their own
    host = _host(kv, cache)
    if weights:                                          # weights that are there already
        w = torch.rand(len(lens) * heads * capacity, generator=g, device=dev)
        at = kv.weight_offset
        cache[at:at + 4 * w.numel()].view(torch.float32).copy_(w)
        host = _host(kv, cache)
    before = host.weight.copy()
    out = torch.full((len(lens), q_len, heads * G, D), 5.0, dtype=torch.bfloat16, device=dev)
    lse = torch.full((len(lens), heads * G, q_len), 5.0, device=dev) if want_lse else None
    ws = torch.full((kv.workspace_bytes(heads * G, q_len, weights),), 0xFF, dtype=torch.uint8, device=dev)
    bytes_before = cache.clone()
    U.ulysses_kv4_attn(kv, cache, q, out, _i32(lens, dev), SCALE, lse=lse, causal=causal, weights=weights,
                       workspace=ws)
    torch.cuda.synchronize()
    assert U.ulysses_kv4_last_device_error(kv) == 0
    after = _host(kv, cache).weight if weights else None
    _check_attn(kv, host, q, out, lse, lens, causal, after, before)
    at = kv.weight_offset
    assert torch.equal(cache[:at], bytes_before[:at])
    if not weights:
        assert torch.equal(cache, bytes_before)
    return kv, cache, q, out, lse


@pytest.mark.parametrize("n", [0, 1, 2, 7, 8, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 1000])
def test_attention_at_every_edge_of_a_block(gpu, n):
    _run_attn(gpu, [n], 2, 1, 1, 1024, 10 + n)


@pytest.mark.parametrize("heads,G", [(1, 1), (3, 2), (8, 7), (2, 8), (1, 9), (2, 16), (1, 17), (1, 40)])
@pytest.mark.parametrize("weights", [False, True])
def test_attention_of_shared_heads(gpu, heads, G, weights):
    _run_attn(gpu, [300, 45], heads, G, 1, 320, 40 + G, weights=weights)


@pytest.mark.parametrize("q_len,G,lens", [(2, 1, [200, 1, 0]), (5, 3, [130, 4, 33]), (8, 2, [129, 8, 7]),
                                          (16, 1, [65, 15, 400]), (33, 1, [40, 33, 20])])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("weights", [False, True])
def test_attention_of_a_block_of_tokens(gpu, q_len, G, lens, causal, weights):
    _run_attn(gpu, lens, 2, G, q_len, 416, 60 + q_len, causal=causal, weights=weights)


def test_attention_of_a_ragged_batch(gpu):
    lens = [5, 0, 1500, 33, 700, 0, 0, 128, 1, 2047, 64, 32]
    _run_attn(gpu, lens, 2, 2, 1, 2048, 80, weights=True)


@pytest.mark.parametrize("B", [33, 70, 130])
def test_attention_of_many_sequences(gpu, B):
    """More sequences than a warp looks through at once, most of them short, some empty."""
    rng = np.random.default_rng(B)
    lens = [int(n) for n in rng.choice([0, 0, 1, 5, 31, 128, 129, 200], B)]
    _run_attn(gpu, lens, 1, 1, 1, 224, 82 + B, weights=True)
    _run_attn(gpu, lens, 1, 3, 1, 224, 83 + B)


def test_the_largest_batch(gpu):
    """1,024 sequences, three of them with tokens: append, attention and load find them."""
    import torch
    B = 1024
    lens = [0] * B
    lens[0], lens[511], lens[1023] = 3, 70, 33
    kv, cache, k, v = _make(gpu, lens, 1, 96, 84)
    host = _host(kv, cache)
    back_k, back_v = torch.zeros_like(k), torch.zeros_like(v)
    U.ulysses_kv4_load(kv, cache, back_k, back_v, _i32(_cu(lens), gpu), _i32([0] * B, gpu))
    g = torch.Generator(device=gpu)
    g.manual_seed(85)
    q = torch.randn((B, 1, 1, D), generator=g, device=gpu).to(torch.bfloat16)
    out = torch.full_like(q, 4.0)
    ws = torch.empty(kv.workspace_bytes(1, 1), dtype=torch.uint8, device=gpu)
    U.ulysses_kv4_attn(kv, cache, q, out, _i32(lens, gpu), SCALE, workspace=ws)
    at = 0
    for b in (0, 511, 1023):
        n = lens[b]
        want, _ = host.values(b, 0, 0, n, 0)
        assert np.array_equal(_bits(back_k[at:at + n, 0]), orc.f64_to_bf16(want))
        v64, vs = host.values(b, 0, 0, n, 1)
        o, _, p = orc.attention(_f64(q)[b, 0, 0], want, v64, SCALE)
        assert np.all(np.abs(_f64(out)[b, 0, 0] - o) <= bound(_f64(q)[b, 0, 0], want, v64, vs, SCALE, o, p))
        at += n
    rest = [b for b in range(B) if not lens[b]]
    assert not bool(out[rest].any())
    assert U.ulysses_kv4_last_device_error(kv) == 0


def test_attention_of_constant_rows(gpu):
    """Steps of 0: a slot's rows are their minima, and the codes do not count."""
    import torch
    n = 150
    kv = U.ulysses_kv4_plan(1, 2, D, 160)
    cache = torch.zeros(kv.cache_bytes, dtype=torch.uint8, device=gpu)
    g = torch.Generator(device=gpu)
    g.manual_seed(86)
    k = torch.randn((n, 2, 2, 1), generator=g, device=gpu).expand(n, 2, 2, 64).reshape(n, 2, D).to(torch.bfloat16)
    v = torch.randn((n, 2, 2, 1), generator=g, device=gpu).expand(n, 2, 2, 64).reshape(n, 2, D).to(torch.bfloat16)
    v[:, 1] = 0
    U.ulysses_kv4_append(kv, cache, k, v, _i32([0, n], gpu), _i32([0], gpu))
    q = torch.randn((1, 1, 2, D), generator=g, device=gpu).to(torch.bfloat16)
    out, lse = torch.empty_like(q), torch.empty((1, 2, 1), device=gpu)
    ws = torch.empty(kv.workspace_bytes(2, 1), dtype=torch.uint8, device=gpu)
    U.ulysses_kv4_attn(kv, cache, q, out, _i32([n], gpu), SCALE, lse=lse, workspace=ws)
    _check_attn(kv, _host(kv, cache), q, out, lse, [n], False)
    assert not bool(out[0, 0, 1].any())


@pytest.mark.parametrize("scale", [1e-30, 1e-3, 50.0])
def test_attention_scales(gpu, scale):
    import torch
    kv, cache, _, _ = _make(gpu, [300], 2, 320, 87)
    g = torch.Generator(device=gpu)
    g.manual_seed(88)
    q = torch.randn((1, 1, 10, D), generator=g, device=gpu).to(torch.bfloat16)
    out, lse = torch.empty_like(q), torch.empty((1, 10, 1), device=gpu)
    ws = torch.empty(kv.workspace_bytes(10, 1), dtype=torch.uint8, device=gpu)
    U.ulysses_kv4_attn(kv, cache, q, out, _i32([300], gpu), scale, lse=lse, workspace=ws)
    _check_attn(kv, _host(kv, cache), q, out, lse, [300], False, scale=scale)


def test_attention_split_over_every_cta(gpu):
    """One pair, more tiles than CTAs: every CTA leaves a part."""
    _run_attn(gpu, [80_001], 1, 1, 1, 80_032, 81, weights=True)


@pytest.mark.parametrize("qscale,spread", [(30.0, 1.0), (1e-20, 1.0), (1e10, 1e-10), (1.0, 1e-6), (0.0, 1.0)])
def test_attention_of_sharp_and_flat_rows(gpu, qscale, spread):
    _run_attn(gpu, [700], 2, 2, 2, 704, 90, weights=True, qscale=qscale, spread=spread, want_lse=False)


def test_attention_of_values_of_very_different_sizes(gpu):
    """Steps that grow 2^40-fold along the cache and between the groups, and keys whose logits rise with the
    slot, so that the running maximum and the power of two of the scales move again and again."""
    import torch
    n = 900
    g = torch.Generator(device=gpu)
    g.manual_seed(7)
    kv = U.ulysses_kv4_plan(1, 2, D, 928)
    cache = torch.zeros(kv.cache_bytes, dtype=torch.uint8, device=gpu)
    rise = torch.linspace(0, 1, n, device=gpu)[:, None, None]
    k = (torch.randn((n, 2, D), generator=g, device=gpu) * 0.1 + rise * 3).to(torch.bfloat16)
    v = torch.randn((n, 2, D), generator=g, device=gpu)
    v[..., :64] *= torch.exp2(40 * rise - 20)
    v[:, 1] *= 1e-9
    v = v.to(torch.bfloat16)
    U.ulysses_kv4_append(kv, cache, k, v, _i32([0, n], gpu), _i32([0], gpu))
    q = (torch.rand((1, 1, 2, D), generator=g, device=gpu) * 3).to(torch.bfloat16)
    out = torch.empty_like(q)
    lse = torch.empty((1, 2, 1), device=gpu)
    ws = torch.empty(kv.workspace_bytes(2, 1), dtype=torch.uint8, device=gpu)
    U.ulysses_kv4_attn(kv, cache, q, out, _i32([n], gpu), SCALE, lse=lse, workspace=ws)
    _check_attn(kv, _host(kv, cache), q, out, lse, [n], False)


@pytest.mark.parametrize("kscale,vscale,qscale", [(1.0, 1e36, 1.0), (1e30, 1e-30, 1e-30), (1e-30, 3e36, 1e30),
                                                  (1.0, 1e-36, 1.0), (1.0, 3e-37, 1.0), (1e36, 1.0, 1e-37)])
def test_attention_over_the_range_of_bf16(gpu, kscale, vscale, qscale):
    import torch
    n = 180
    g = torch.Generator(device=gpu)
    g.manual_seed(17)
    kv = U.ulysses_kv4_plan(1, 2, D, 192)
    cache = torch.zeros(kv.cache_bytes, dtype=torch.uint8, device=gpu)
    k = (torch.randn((n, 2, D), generator=g, device=gpu) * kscale).to(torch.bfloat16)
    v = (torch.randn((n, 2, D), generator=g, device=gpu) * vscale).to(torch.bfloat16)
    U.ulysses_kv4_append(kv, cache, k, v, _i32([0, n], gpu), _i32([0], gpu))
    for heads in (2, 10):                                # one query row a K/V head, and five
        q = (torch.randn((1, 1, heads, D), generator=g, device=gpu) * qscale).to(torch.bfloat16)
        out, lse = torch.empty_like(q), torch.empty((1, heads, 1), device=gpu)
        ws = torch.empty(kv.workspace_bytes(heads, 1), dtype=torch.uint8, device=gpu)
        U.ulysses_kv4_attn(kv, cache, q, out, _i32([n], gpu), SCALE, lse=lse, workspace=ws)
        _check_attn(kv, _host(kv, cache), q, out, lse, [n], False)


def test_attention_of_queries_past_the_range(gpu):
    """A query row that reaches 2^115 gives NaN, whatever the keys; the rows beside it keep their results."""
    import torch
    for heads in (2, 10):
        kv, cache, _, _ = _make(gpu, [100], 2, 128, 23)
        g = torch.Generator(device=gpu)
        g.manual_seed(24)
        q = torch.randn((1, 1, heads, D), generator=g, device=gpu).to(torch.bfloat16)
        out, lse = torch.empty_like(q), torch.empty((1, heads, 1), device=gpu)
        ws = torch.empty(kv.workspace_bytes(heads, 1), dtype=torch.uint8, device=gpu)
        U.ulysses_kv4_attn(kv, cache, q, out, _i32([100], gpu), SCALE, lse=lse, workspace=ws)
        want, want_lse = out.clone(), lse.clone()
        q[0, 0, 1] = 0
        q[0, 0, 1, 5] = -2.0 ** 115
        U.ulysses_kv4_attn(kv, cache, q, out, _i32([100], gpu), SCALE, lse=lse, workspace=ws)
        assert torch.isnan(out[0, 0, 1]).all() and torch.isnan(lse[0, 1]).all()
        rest = [h for h in range(heads) if h != 1]
        assert torch.equal(out[0, 0, rest], want[0, 0, rest]) and torch.equal(lse[0, rest], want_lse[0, rest])


def test_attention_keeps_nan_where_it_is_seen_only(gpu):
    """A NaN value row reaches the rows that see it, in its group alone; a row masked from it is untouched.
    A NaN key makes the rows that see it NaN."""
    import torch
    kv, cache, k, v = _make(gpu, [200, 200], 2, 224, 11)
    bad = v[:1].clone()
    bad[0, 0, 70] = float("inf")                 # sequence 0, head 0, group 1, slot 199
    U.ulysses_kv4_append(kv, cache, k[199:200].contiguous(), bad, _i32([0, 1, 1], gpu), _i32([199, 0], gpu))
    bad = k[:1].clone()
    bad[0, 1, 3] = float("nan")                  # sequence 1, head 1, slot 199
    U.ulysses_kv4_append(kv, cache, bad, v[399:400].contiguous(), _i32([0, 0, 1], gpu), _i32([0, 199], gpu))
    g = torch.Generator(device=gpu)
    g.manual_seed(12)
    q = torch.randn((2, 2, 2, D), generator=g, device=gpu).to(torch.bfloat16)
    out = torch.empty_like(q)
    ws = torch.empty(kv.workspace_bytes(2, 2), dtype=torch.uint8, device=gpu)
    U.ulysses_kv4_attn(kv, cache, q, out, _i32([200, 200], gpu), SCALE, causal=True, workspace=ws)
    nan = torch.isnan(out).cpu().numpy()
    want = np.zeros_like(nan)
    want[0, 1, 0, 64:] = True
    want[1, 1, 1] = True
    assert np.array_equal(nan, want)
    # a query that is not finite has no softmax
    q[0, 0, 1, 5] = float("inf")
    q[1, 0, 0, 5] = float("nan")
    U.ulysses_kv4_attn(kv, cache, q, out, _i32([200, 200], gpu), SCALE, causal=True, workspace=ws)
    nan = torch.isnan(out).cpu().numpy()
    want[0, 0, 1] = True
    want[1, 0, 0] = True
    assert np.array_equal(nan, want)


def test_lengths_outside_the_cache_are_held_inside_and_reported(gpu):
    import torch
    kv, cache, _, _ = _make(gpu, [64, 64], 2, 64, 13)
    g = torch.Generator(device=gpu)
    g.manual_seed(14)
    q = torch.randn((2, 1, 2, D), generator=g, device=gpu).to(torch.bfloat16)
    ws = torch.empty(kv.workspace_bytes(2, 1, True), dtype=torch.uint8, device=gpu)
    out, want = torch.empty_like(q), torch.empty_like(q)
    U.ulysses_kv4_attn(kv, cache, q, want, _i32([64, 0], gpu), SCALE, workspace=ws)
    assert U.ulysses_kv4_last_device_error(kv) == 0
    U.ulysses_kv4_attn(kv, cache, q, out, _i32([1 << 30, -5], gpu), SCALE, weights=True, workspace=ws)
    assert U.ulysses_kv4_last_device_error(kv) == 16
    assert torch.equal(out, want)


# ------------------------------------------------------------------------------------------ eviction

def _check_evict(kv, cache, dst_kv, dst, before, lens, new, keep, sink, recent):
    src, got, old = _host(kv, cache), _host(dst_kv, dst), _host(dst_kv, before)
    assert new.cpu().tolist() == [min(n, keep) for n in lens]
    for b, n in enumerate(lens):
        for h in range(kv.heads):
            slots = orc.kept_slots(src.weight[b, h], n, keep, sink, recent)
            assert got.pos[b, h, :len(slots)].tolist() == src.pos[b, h][slots].tolist(), (b, h)
            assert np.array_equal(got.weight[b, h, :len(slots)].view(np.int32), src.weight[b, h][slots].view(np.int32))
            for j, t in enumerate(slots):
                for plane in (0, 1):
                    assert np.array_equal(got.row(b, h, j, plane), src.row(b, h, t, plane))
                    assert np.array_equal(got.meta(b, h, j, plane), src.meta(b, h, t, plane))
            for j in range(len(slots), dst_kv.capacity):
                assert got.pos[b, h, j] == old.pos[b, h, j]
                assert np.array_equal(got.row(b, h, j, 0), old.row(b, h, j, 0))
                assert np.array_equal(got.meta(b, h, j, 1), old.meta(b, h, j, 1))
            assert np.array_equal(got.weight[b, h, len(slots):].view(np.int32), old.weight[b, h, len(slots):].view(np.int32))


def _weights(kind, shape, rng):
    if kind == "spread":
        return np.exp(rng.standard_normal(shape) * 3).astype(np.float32)
    if kind == "ties":
        return (rng.integers(0, 3, shape) * 0.25).astype(np.float32)
    if kind == "equal":
        return np.full(shape, 0.125, dtype=np.float32)
    if kind == "close":            # neighbours in fp32: every digit of the key counts
        return (np.float32(1.0).view(np.int32) + rng.integers(0, 4000, shape)).astype(np.int32).view(np.float32)
    special = np.array([np.nan, -np.nan, np.inf, -np.inf, -0.0, 0.0, -1.0, 1e-45, -1e-45, 3.0], dtype=np.float32)
    return special[rng.integers(0, len(special), shape)]


@pytest.mark.parametrize("kind", ["spread", "ties", "equal", "close", "special"])
@pytest.mark.parametrize("lens,keep,sink,recent", [
    ([200], 50, 0, 0), ([200, 50, 0, 51, 1], 50, 4, 10), ([130, 33], 32, 32, 0), ([130, 33], 32, 0, 32),
    ([100, 2], 1, 0, 0), ([100], 1, 1, 0), ([300, 299], 299, 3, 290), ([64], 64, 0, 0)])
def test_eviction_keeps_the_heaviest_slots(gpu, kind, lens, keep, sink, recent):
    import torch
    heads = 3
    rng = np.random.default_rng(len(kind) + keep)
    kv, cache, _, _ = _make(gpu, lens, heads, 320, 20)
    w = torch.from_numpy(_weights(kind, (len(lens), heads, 320), rng)).to(gpu)
    at = kv.weight_offset
    cache[at:at + 4 * w.numel()].view(torch.float32).copy_(w.view(-1))
    dst_kv = U.ulysses_kv4_plan(len(lens), heads, D, (keep + 31) // 32 * 32)
    dst = torch.full((dst_kv.cache_bytes,), 0x3C, dtype=torch.uint8, device=gpu)
    before = dst.clone()
    new = torch.full((len(lens),), -7, dtype=torch.int32, device=gpu)
    source = cache.clone()
    U.ulysses_kv4_evict(kv, cache, dst_kv, dst, _i32(lens, gpu), new, keep, sink, recent)
    assert U.ulysses_kv4_last_device_error(kv) == 0
    assert torch.equal(cache, source)
    _check_evict(kv, cache, dst_kv, dst, before, lens, new, keep, sink, recent)


@pytest.mark.parametrize("keep", [150, 160, 170, 199])
def test_eviction_whose_border_is_among_nan(gpu, keep):
    """A fifth of the weights are NaN, so the last kept slots are the lowest of those."""
    import torch
    rng = np.random.default_rng(keep)
    kv, cache, _, _ = _make(gpu, [200, 198], 3, 224, 21)
    w = rng.random((2, 3, 224), dtype=np.float32)
    w[rng.random(w.shape) < 0.2] = np.nan
    at = kv.weight_offset
    cache[at:at + 4 * w.size].view(torch.float32).copy_(torch.from_numpy(w).to(gpu).view(-1))
    dst_kv = U.ulysses_kv4_plan(2, 3, D, 256)
    dst = torch.zeros(dst_kv.cache_bytes, dtype=torch.uint8, device=gpu)
    before, new = dst.clone(), _i32([0, 0], gpu)
    U.ulysses_kv4_evict(kv, cache, dst_kv, dst, _i32([200, 198], gpu), new, keep)
    _check_evict(kv, cache, dst_kv, dst, before, [200, 198], new, keep, 0, 0)


def test_eviction_into_a_larger_cache_and_of_lengths_outside(gpu):
    import torch
    kv, cache, _, _ = _make(gpu, [60, 64, 10], 2, 64, 22)
    dst_kv = U.ulysses_kv4_plan(3, 2, D, 128)
    dst = torch.full((dst_kv.cache_bytes,), 0x11, dtype=torch.uint8, device=gpu)
    before, new = dst.clone(), _i32([0, 0, 0], gpu)
    U.ulysses_kv4_evict(kv, cache, dst_kv, dst, _i32([60, 64, 10], gpu), new, 100, 10, 10)
    _check_evict(kv, cache, dst_kv, dst, before, [60, 64, 10], new, 100, 10, 10)
    assert U.ulysses_kv4_last_device_error(kv) == 0
    dst.copy_(before)
    U.ulysses_kv4_evict(kv, cache, dst_kv, dst, _i32([-1, 1 << 30, 10], gpu), new, 20)
    assert U.ulysses_kv4_last_device_error(kv) == 16
    _check_evict(kv, cache, dst_kv, dst, before, [0, 64, 10], new, 20, 0, 0)


def test_eviction_of_more_keys_than_a_block_holds(gpu):
    """150 pairs, so that one block has a pair's 23,000 slots and makes the keys anew each time."""
    import torch
    B, n, keep, cap = 150, 23_000, 1_000, 23_008
    kv = U.ulysses_kv4_plan(B, 1, D, cap)
    cache = torch.zeros(kv.cache_bytes, dtype=torch.uint8, device=gpu)
    rng = np.random.default_rng(23)
    w = (rng.integers(0, 5000, (B, cap)) / 64).astype(np.float32)
    at = kv.weight_offset
    cache[at:at + 4 * w.size].view(torch.float32).copy_(torch.from_numpy(w).to(gpu).view(-1))
    at = kv.position_offset
    cache[at:].view(torch.int32).copy_(torch.arange(cap, dtype=torch.int32, device=gpu).repeat(B))
    dst_kv = U.ulysses_kv4_plan(B, 1, D, 1024)
    dst = torch.zeros(dst_kv.cache_bytes, dtype=torch.uint8, device=gpu)
    new = torch.zeros(B, dtype=torch.int32, device=gpu)
    lens = [n - b for b in range(B)]
    U.ulysses_kv4_evict(kv, cache, dst_kv, dst, _i32(lens, gpu), new, keep, 4, 100)
    got = _host(dst_kv, dst)
    for b in (0, 1, 2, 3, 77, 148, 149):
        assert np.array_equal(got.pos[b, 0, :keep], orc.kept_slots(w[b], lens[b], keep, 4, 100)), b


@pytest.mark.parametrize("kind", ["spread", "ties"])
def test_eviction_of_a_long_cache(gpu, kind):
    """The selection against a full sort, where a pair's slots need many passes of a block."""
    import torch
    n, heads, keep, sink, recent = 70_001, 2, 9_999, 4, 1_001
    cap = 70_016
    g = torch.Generator(device=gpu)
    g.manual_seed(30)
    kv = U.ulysses_kv4_plan(1, heads, D, cap)
    cache = torch.randint(0, 256, (kv.cache_bytes,), generator=g, device=gpu, dtype=torch.uint8)
    rng = np.random.default_rng(31)
    w = _weights(kind, (heads, cap), rng)
    at = kv.weight_offset
    cache[at:at + 4 * w.size].view(torch.float32).copy_(torch.from_numpy(w).to(gpu).view(-1))
    at = kv.position_offset
    cache[at:].view(torch.int32).copy_(torch.arange(cap, dtype=torch.int32, device=gpu).repeat(heads))
    dst_kv = U.ulysses_kv4_plan(1, heads, D, 10_016)
    dst = torch.zeros(dst_kv.cache_bytes, dtype=torch.uint8, device=gpu)
    new = torch.zeros(1, dtype=torch.int32, device=gpu)
    U.ulysses_kv4_evict(kv, cache, dst_kv, dst, _i32([n], gpu), new, keep, sink, recent)
    src, got = _host(kv, cache), _host(dst_kv, dst)
    for h in range(heads):
        slots = orc.kept_slots(w[h], n, keep, sink, recent)
        assert np.array_equal(got.pos[0, h, :keep], slots)
        for j in rng.integers(0, keep, 200):
            for plane in (0, 1):
                assert np.array_equal(got.row(0, h, j, plane), src.row(0, h, slots[j], plane))
                assert np.array_equal(got.meta(0, h, j, plane), src.meta(0, h, slots[j], plane))


# ------------------------------------------------------------------------------------------ together

def test_offsets_past_32_bits(gpu):
    """A cache of 6.7 GB whose last pairs hold the only tokens."""
    import torch
    B, heads, cap = 14, 32, 104_448
    kv = U.ulysses_kv4_plan(B, heads, D, cap)
    assert kv.weight_offset > 1 << 32
    cache = torch.zeros(kv.cache_bytes, dtype=torch.uint8, device=gpu)
    g = torch.Generator(device=gpu)
    g.manual_seed(50)
    n, start = 90, cap - 90
    k = torch.randn((n, heads, D), generator=g, device=gpu).to(torch.bfloat16)
    cu = _i32([0] * B + [n], gpu)
    st = _i32([0] * (B - 1) + [start], gpu)
    U.ulysses_kv4_append(kv, cache, k, k, cu, st)
    got, got_v = torch.empty_like(k), torch.empty_like(k)
    U.ulysses_kv4_load(kv, cache, got, got_v, cu, st)
    assert torch.equal(got, got_v)
    for h in (0, heads - 1):
        want = np.stack([_row_back(x) for x in _f64(k[:, h])])
        assert np.array_equal(_bits(got[:, h]), orc.f64_to_bf16(want))
    # the slots below `start` are zeros: keys of logit 0 and values of 0
    q = torch.randn((B, 1, heads, D), generator=g, device=gpu).to(torch.bfloat16)
    out = torch.empty_like(q)
    ws = torch.empty(kv.workspace_bytes(heads, 1), dtype=torch.uint8, device=gpu)
    U.ulysses_kv4_attn(kv, cache, q, out, _i32([0] * (B - 1) + [cap], gpu), SCALE, workspace=ws)
    assert not bool(out[:-1].any())
    z = torch.einsum("hd,nhd->hn", q[-1, 0].double(), got.double()) * SCALE
    e = torch.exp(z)
    o = torch.einsum("hn,nhd->hd", e / (e.sum(1, keepdim=True) + start), got.double())
    err = (out[-1, 0].double() - o).abs()
    # w rounded to fp16 (2^-11 of p s n, here below 2^-11 * sum p * 8), bf16 result
    tol = o.abs() * 2.0 ** -8 + (e.sum(1) / (e.sum(1) + start))[:, None] * 8 * 2.0 ** -10 + 2.0 ** -22
    assert bool((err <= tol).all())
    dst_kv = U.ulysses_kv4_plan(B, heads, D, 64)
    dst = torch.zeros(dst_kv.cache_bytes, dtype=torch.uint8, device=gpu)
    new = torch.zeros(B, dtype=torch.int32, device=gpu)
    U.ulysses_kv4_evict(kv, cache, dst_kv, dst, _i32([0] * (B - 1) + [cap], gpu), new, 64, 0, 64)
    assert new.tolist() == [0] * (B - 1) + [64]
    kk, vv = torch.empty_like(k[:64]), torch.empty_like(k[:64])
    U.ulysses_kv4_load(dst_kv, dst, kk, vv, _i32([0] * B + [64], gpu), _i32([0] * B, gpu))
    assert torch.equal(kk, got[-64:]) and torch.equal(vv, got[-64:])


def _row_back(x):
    rows, meta = orc.quantise_row(x)
    c = orc.Cache(np.zeros(4608 + 256, dtype=np.uint8), 1, 1, 32)
    c.row(0, 0, 0, 0)[:] = rows
    c.meta(0, 0, 0, 0)[:] = meta
    return c.values(0, 0, 0, 1, 0)[0][0]


def test_prompt_decode_evict_decode(gpu):
    """A causal prompt through the layer's attention, its K and V planes into the cache, decoding steps that
    keep the weights, an eviction into a budget, further steps, and the cached rows back for the layer's
    attention."""
    import torch
    N, H, P, steps, keep = 203, 4, 2, 5, 64
    g = torch.Generator(device=gpu)
    g.manual_seed(60)
    plan = U.ulysses_plan(N, H, D, P, 3, causal=True)
    Np = plan.padded_tokens
    S = torch.zeros((Np, 3, H, D), dtype=torch.bfloat16, device=gpu)
    S[:N] = torch.randn((N, 3, H, D), generator=g, device=gpu).to(torch.bfloat16)
    T = torch.empty((P, 3, Np, H // P, D), dtype=torch.bfloat16, device=gpu)
    O = torch.empty((P, Np, H // P, D), dtype=torch.bfloat16, device=gpu)
    U.ulysses_repack_fwd(plan, S, T)
    U.ulysses_attn_fwd(plan, T, O, SCALE)
    kv = U.ulysses_kv4_plan(1, H, D, 224)
    cache = torch.zeros(kv.cache_bytes, dtype=torch.uint8, device=gpu)
    zero, length = _i32([0], gpu), _i32([N], gpu)
    U.ulysses_kv4_append(kv, cache, T[:, 1, :N], T[:, 2, :N], _i32([0, N], gpu), zero)
    ws = torch.empty(kv.workspace_bytes(H, 1, True), dtype=torch.uint8, device=gpu)
    one = _i32([0, 1], gpu)
    n = N
    for _ in range(steps):
        new = torch.randn((1, 3, H, D), generator=g, device=gpu).to(torch.bfloat16)
        U.ulysses_kv4_append(kv, cache, new[:, 1], new[:, 2], one, length)
        length += 1
        n += 1
        before = _host(kv, cache).weight.copy()
        out = torch.empty((1, 1, H, D), dtype=torch.bfloat16, device=gpu)
        U.ulysses_kv4_attn(kv, cache, new[:, 0][:, None], out, length, SCALE, weights=True, workspace=ws)
        host = _host(kv, cache)
        _check_attn(kv, host, new[:, 0][:, None], out, None, [n], False, host.weight, before)
    small = U.ulysses_kv4_plan(1, H, D, 96)
    cut = torch.zeros(small.cache_bytes, dtype=torch.uint8, device=gpu)
    old = cut.clone()
    left = torch.zeros_like(length)
    U.ulysses_kv4_evict(kv, cache, small, cut, length, left, keep, 4, 16)
    _check_evict(kv, cache, small, cut, old, [n], left, keep, 4, 16)
    seen = length.clone()                              # positions go on where the sequence is
    n = keep
    for _ in range(2):
        new = torch.randn((1, 3, H, D), generator=g, device=gpu).to(torch.bfloat16)
        U.ulysses_kv4_append(small, cut, new[:, 1], new[:, 2], one, left, seen)
        left += 1
        seen += 1
        n += 1
        out = torch.empty((1, 1, H, D), dtype=torch.bfloat16, device=gpu)
        U.ulysses_kv4_attn(small, cut, new[:, 0][:, None], out, left, SCALE, workspace=ws)
        _check_attn(small, _host(small, cut), new[:, 0][:, None], out, None, [n], False)
    assert _host(small, cut).pos[0, 0, n - 1] == N + steps + 1
    # the kept rows back into a slab, and the last token's attention by the layer's kernel
    back = U.ulysses_plan(n, H, D, P, 3, causal=True)
    T2 = torch.zeros((P, 3, back.padded_tokens, H // P, D), dtype=torch.bfloat16, device=gpu)
    U.ulysses_kv4_load(small, cut, T2[:, 1, :n], T2[:, 2, :n], _i32([0, n], gpu), zero)
    T2[:, 0, n - 1] = new[0, 0].view(P, H // P, D)
    O2 = torch.empty((P, back.padded_tokens, H // P, D), dtype=torch.bfloat16, device=gpu)
    U.ulysses_attn_fwd(back, T2, O2, SCALE)
    a, b = O2[:, n - 1].reshape(H, D).double(), out[0, 0].double()
    assert float((a - b).norm() / b.norm()) <= 1e-2    # the layer's bound: K, V and P rounded to bf16
    assert U.ulysses_kv4_last_device_error(kv) == 0 and U.ulysses_kv4_last_device_error(small) == 0


def test_a_captured_decoding_loop(gpu):
    """append, attention and the advance of the lengths in one graph; replays equal direct calls."""
    import torch
    B, heads, G, cap = 3, 2, 2, 160
    kv, cache, _, _ = _make(gpu, [100, 31, 0], heads, cap, 70)
    direct = cache.clone()
    g = torch.Generator(device=gpu)
    g.manual_seed(71)
    steps = torch.randn((6, B, heads * G + 2 * heads, D), generator=g, device=gpu).to(torch.bfloat16)
    cur = steps[0].clone()
    cu = _i32(list(range(B + 1)), gpu)
    out = torch.empty((B, 1, heads * G, D), dtype=torch.bfloat16, device=gpu)
    ws = torch.empty(kv.workspace_bytes(heads * G, 1, True), dtype=torch.uint8, device=gpu)

    def step(c, lengths):
        U.ulysses_kv4_append(kv, c, cur[:, heads * G:heads * (G + 1)], cur[:, heads * (G + 1):], cu, lengths)
        lengths += 1
        U.ulysses_kv4_attn(kv, c, cur[:, None, :heads * G], out, lengths, SCALE, weights=True, workspace=ws)

    lengths = _i32([100, 31, 0], gpu)
    want = []
    for i in range(6):
        cur.copy_(steps[i])
        step(direct, lengths)
        want.append(out.clone())
    lengths = _i32([100, 31, 0], gpu)
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        step(cache, lengths)
    for i in range(6):
        cur.copy_(steps[i])
        graph.replay()
        assert torch.equal(out, want[i]), i
    assert torch.equal(cache, direct)
    assert U.ulysses_kv4_last_device_error(kv) == 0


def test_a_captured_eviction(gpu):
    """Eviction and load in a graph; a replay goes by the lengths and weights of its time."""
    import torch
    kv, cache, _, _ = _make(gpu, [90, 40], 2, 96, 72)
    g = torch.Generator(device=gpu)
    g.manual_seed(73)
    n = 2 * 2 * 96
    w = cache[kv.weight_offset:kv.weight_offset + 4 * n].view(torch.float32)
    dst_kv = U.ulysses_kv4_plan(2, 2, D, 64)
    dst = torch.zeros(dst_kv.cache_bytes, dtype=torch.uint8, device=gpu)
    lengths, new = _i32([90, 40], gpu), _i32([0, 0], gpu)
    cu, start = _i32([0, 50, 90], gpu), _i32([0, 0], gpu)
    k, v = (torch.zeros((90, 2, D), dtype=torch.bfloat16, device=gpu) for _ in range(2))
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        U.ulysses_kv4_evict(kv, cache, dst_kv, dst, lengths, new, 50, 2, 7)
        U.ulysses_kv4_load(dst_kv, dst, k, v, cu, start)
    for lens in ([90, 40], [60, 96], [3, 50]):
        w.copy_(torch.rand(n, generator=g, device=gpu))
        lengths.copy_(_i32(lens, gpu))
        before = dst.clone()
        graph.replay()
        _check_evict(kv, cache, dst_kv, dst, before, lens, new, 50, 2, 7)
        host = _host(dst_kv, dst)
        want, _ = host.values(0, 1, 0, 50, 0)
        assert np.array_equal(_bits(k[:50, 1]), orc.f64_to_bf16(want))


def test_strides_of_single_rows_and_heads_do_not_count(gpu):
    import torch
    kv, cache, k, v = _make(gpu, [40], 1, 64, 96)
    row = torch.randn(2, 1, 1, D, device=gpu).to(torch.bfloat16)
    odd = [torch.as_strided(row[i], (1, 1, D), (3, 5, 1), row[i].storage_offset()) for i in range(2)]
    U.ulysses_kv4_append(kv, cache, odd[0], torch.as_strided(odd[1], (1, 1, D), (7, 1, 1), odd[1].storage_offset()),
                         _i32([0, 1], gpu), _i32([40], gpu))
    _check_append(kv, cache, row[0], row[1], [1], [40])
    q = torch.as_strided(row, (1, 1, 1, D), (1, 3, 5, 1))
    out = torch.empty((1, 1, 1, D), dtype=torch.bfloat16, device=gpu)
    ws = torch.empty(kv.workspace_bytes(1, 1), dtype=torch.uint8, device=gpu)
    U.ulysses_kv4_attn(kv, cache, q, out, _i32([41], gpu), SCALE, workspace=ws)
    _check_attn(kv, _host(kv, cache), q, out, None, [41], False)


def test_append_repeats_a_row_that_heads_share(gpu):
    """A head stride of 0: one K/V row for all heads."""
    import torch
    kv = U.ulysses_kv4_plan(1, 6, D, 32)
    cache = torch.zeros(kv.cache_bytes, dtype=torch.uint8, device=gpu)
    k = torch.randn((9, 1, D), device=gpu).to(torch.bfloat16).expand(9, 6, D)
    v = torch.randn((9, 1, D), device=gpu).to(torch.bfloat16).expand(9, 6, D)
    U.ulysses_kv4_append(kv, cache, k, v, _i32([0, 9], gpu), _i32([3], gpu))
    _check_append(kv, cache, k, v, [9], [3])
    # a rank stride of 0: the same two heads for all three ranks
    two = torch.randn((2, 1, 9, 2, D), device=gpu).to(torch.bfloat16).expand(2, 3, 9, 2, D)
    U.ulysses_kv4_append(kv, cache, two[0], two[1], _i32([0, 9], gpu), _i32([12], gpu))
    flat = two.permute(0, 2, 1, 3, 4).reshape(2, 9, 6, D)
    _check_append(kv, cache, flat[0], flat[1], [9], [12])
    with pytest.raises(U.UlyssesError):
        U.ulysses_kv4_load(kv, cache, k, v, _i32([0, 9], gpu), _i32([3], gpu))


def test_two_calls_at_once_on_two_streams(gpu):
    import torch
    made = [_make(gpu, [3000 + 500 * i], 4, 4096, 90 + i) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in made]
    g = torch.Generator(device=gpu)
    g.manual_seed(92)
    q = torch.randn((1, 1, 8, D), generator=g, device=gpu).to(torch.bfloat16)
    ws = [torch.empty(m[0].workspace_bytes(8, 1), dtype=torch.uint8, device=gpu) for m in made]
    lens = [_i32([3000 + 500 * i], gpu) for i in range(2)]
    alone, outs = [torch.empty_like(q) for _ in made], [torch.empty_like(q) for _ in made]
    for i, (kv, cache, _, _) in enumerate(made):
        U.ulysses_kv4_attn(kv, cache, q, alone[i], lens[i], SCALE, workspace=ws[i])
    torch.cuda.synchronize()
    for _ in range(20):
        for i, (kv, cache, _, _) in enumerate(made):
            U.ulysses_kv4_attn(kv, cache, q, outs[i], lens[i], SCALE, workspace=ws[i], stream=streams[i])
    torch.cuda.synchronize()
    assert torch.equal(outs[0], alone[0]) and torch.equal(outs[1], alone[1])


def test_binding_checks_shapes(gpu):
    import torch
    kv, cache, k, v = _make(gpu, [8], 2, 32, 95)
    cu, st = _i32([0, 8], gpu), _i32([0], gpu)
    with pytest.raises(ValueError):
        U.ulysses_kv4_append(kv, cache[:-16], k, v, cu, st)
    with pytest.raises(ValueError):
        U.ulysses_kv4_append(kv, cache, k[:, :1], v[:, :1], cu, st)
    with pytest.raises(ValueError):
        U.ulysses_kv4_append(kv, cache, k, v[:4], cu, st)
    with pytest.raises(ValueError):
        U.ulysses_kv4_append(kv, cache, k, v, st, st)
    with pytest.raises(TypeError):
        U.ulysses_kv4_append(kv, cache, k, v, cu.long(), st)
    with pytest.raises(TypeError):
        U.ulysses_kv4_load(kv, cache, k.float(), v.float(), cu, st)
    q = torch.zeros((1, 3, 2, D), dtype=torch.bfloat16, device=gpu)
    ws = torch.empty(kv.workspace_bytes(2, 3), dtype=torch.uint8, device=gpu)
    ln = _i32([8], gpu)
    with pytest.raises(ValueError):
        U.ulysses_kv4_attn(kv, cache, q[:, :, :, :64], q, ln, SCALE, workspace=ws)
    with pytest.raises(ValueError):
        U.ulysses_kv4_attn(kv, cache, q, q[:, :2].clone(), ln, SCALE, workspace=ws)
    with pytest.raises(ValueError):
        U.ulysses_kv4_attn(kv, cache, q, torch.empty_like(q), ln, SCALE, lse=torch.zeros(5, device=gpu), workspace=ws)
    with pytest.raises(U.UlyssesError):
        U.ulysses_kv4_attn(kv, cache, q, torch.empty_like(q), ln, SCALE)
    with pytest.raises(U.UlyssesError):
        U.ulysses_kv4_evict(kv, cache, kv, cache, ln, _i32([0], gpu), 8)
    empty = k[:0]
    U.ulysses_kv4_append(kv, cache, empty, empty, _i32([0, 0], gpu), st)     # nothing to do
    U.ulysses_kv4_load(kv, cache, empty, empty, _i32([0, 0], gpu), st)


# ------------------------------------------------------------------------------------------ rows on their own

def row_bound(q, k, v, vs, scale, o, p):
    """As `bound`, element by element, with what one slot can cost another taken from p s instead of s:

    * a row's power of two for a group is that of the largest p s it has met (the maximum and its p of the time, which
      later maxima scale down for both), or 2^-114, so an operand below fp16's normal numbers is off by at most
      2^-25 2^-5 of that: 2^-30 max p s + 2^-144 a slot, times codes of at most 15;
    * the logits' terms are those of their own group (|m| and 15 s are at most twice the group's largest magnitude);
    * a maximum moves by 2^8 at least, each time with an exp2 (2^-22) in what was summed before: at most
      (range of z in powers of two) / 8 + 1 times.
    """
    n = k.shape[0]
    u = 2.0 ** -24
    mag = np.abs(v) + 15 * np.repeat(vs, 64, axis=1)
    top = np.repeat(np.abs(k).reshape(n, 2, 64).max(2), 64, axis=1)
    zmax = np.max(scale * ((np.abs(k) + 2 * top) @ np.abs(q)))
    rel = 2 * 260 * u * zmax + 2.0 ** -21 + (2 * zmax * 1.45 / 8 + 1) * 2.0 ** -22
    w = (p[:, None] * 15 * np.repeat(vs, 64, axis=1)).sum(0) * 2.0 ** -11
    tiny = n * 15 * (np.repeat((p[:, None] * vs).max(0), 64) * 2.0 ** -30 + 2.0 ** -144)
    sums = 2 * u * n * (p[:, None] * mag).sum(0)
    core = rel * (p[:, None] * mag).sum(0) + w + tiny + sums
    return core + (np.abs(o) + core) * 2.0 ** -8, 2 * 260 * u * zmax / np.log(2.0) + 2.0 ** -20


def _check_rows(kv, host, q, out, lse, lens, causal, scale=SCALE, weights=None, before=None):
    """Every row against the slots it sees and nothing else: a group of V that is not finite makes that group of the
    row NaN, a K or a query that is not makes the row, its log-sum and its share of the weights NaN, and a row that
    sees nothing gives zeros, -infinity and no weight, whatever its query is."""
    B, q_len, q_heads, _ = q.shape
    G = q_heads // kv.heads
    qq, oo, ls = _f64(q), _f64(out), lse.cpu().numpy().astype(np.float64)
    for b in range(B):
        for h in range(kv.heads):
            n = lens[b]
            k, _ = host.values(b, h, 0, n, 0)
            v, vs = host.values(b, h, 0, n, 1)
            total, slack = np.zeros(n), np.zeros(n)
            for i in range(q_len):
                m = max(0, n - q_len + i + 1) if causal else n
                for j in range(h * G, (h + 1) * G):
                    where = (b, i, j)
                    got = oo[b, i, j]
                    if m == 0:
                        assert not got.any() and ls[b, j, i] == -np.inf, where
                        continue
                    if not (np.isfinite(qq[b, i, j]).all() and np.isfinite(k[:m]).all()):
                        assert np.isnan(got).all() and np.isnan(ls[b, j, i]), where
                        total[:m] = np.nan
                        continue
                    seen = np.where(np.isfinite(vs[:m]), vs[:m], 0.0)
                    vv = np.where(np.isfinite(v[:m]), v[:m], 0.0)
                    o, z, p = orc.attention(qq[b, i, j], k[:m], vv, scale)
                    tol, dz = row_bound(qq[b, i, j], k[:m], vv, seen, scale, o, p)
                    nan = np.repeat(~np.isfinite(vs[:m]).all(0), 64)
                    assert np.array_equal(np.isnan(got), nan), where
                    err = np.abs(got - o)[~nan]
                    assert np.all(err <= tol[~nan]), (*where, float((err / tol[~nan]).max()))
                    dz += 2.0 ** -23 * abs(z)
                    assert abs(ls[b, j, i] - z) <= dz, (*where, ls[b, j, i], z)
                    total[:m] += p
                    slack[:m] += p * 2 * dz + 2.0 ** -126
            if weights is None:
                continue
            old, new = before[b, h].astype(np.float64), weights[b, h].astype(np.float64)
            assert np.array_equal(np.isnan(new[:n]), np.isnan(total)), (b, h)
            ok = ~np.isnan(total)
            room = slack + 2.0 ** -23 * (G * q_len + 1) * (total + np.abs(old[:n]) + np.abs(new[:n]))
            assert np.all(np.abs(new[:n] - old[:n] - total)[ok] <= room[ok]), (b, h)
            assert np.array_equal(weights[b, h][n:].view(np.int32), before[b, h][n:].view(np.int32))


# query tokens and heads that make 1 to 2, 3 to 8, 9 to 16 and more rows of a K/V head
SHAPES = [(1, 1), (2, 1), (3, 1), (2, 4), (3, 3), (2, 8), (20, 1)]


def _attend(dev, kv, cache, q, lens, causal, weights=False, scale=SCALE):
    import torch
    host = _host(kv, cache)
    B, q_len, q_heads, _ = q.shape
    out = torch.full((B, q_len, q_heads, D), 5.0, dtype=torch.bfloat16, device=dev)
    lse = torch.full((B, q_heads, q_len), 5.0, device=dev)
    ws = torch.full((kv.workspace_bytes(q_heads, q_len, weights),), 0xFF, dtype=torch.uint8, device=dev)
    U.ulysses_kv4_attn(kv, cache, q, out, _i32(lens, dev), scale, lse=lse, causal=causal, weights=weights,
                       workspace=ws)
    assert U.ulysses_kv4_last_device_error(kv) == 0
    _check_rows(kv, host, q, out, lse, lens, causal, scale, _host(kv, cache).weight if weights else None,
                host.weight)


def _queries(dev, B, q_len, heads, seed):
    import torch
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    return torch.randn((B, q_len, heads, D), generator=g, device=dev).to(torch.bfloat16)


@pytest.mark.parametrize("q_len,G", SHAPES)
@pytest.mark.parametrize("n", [8, 33, 200, 1000])
def test_values_that_are_not_finite_stay_with_the_rows_that_see_them(gpu, q_len, G, n):
    """The newest token's V holds an infinity in one group of one head (and another sequence's a NaN): the tokens
    before it, which do not see it, keep their values in that group too."""
    kv, cache, k, v = _make(gpu, [n, n], 2, 1024, 100 + n)
    bad = v[[n - 1, 2 * n - 1]].clone()
    bad[0, 0, 70] = float("inf")
    bad[1, 1, 3] = float("nan")
    U.ulysses_kv4_append(kv, cache, k[[n - 1, 2 * n - 1]].contiguous(), bad, _i32([0, 1, 2], gpu),
                         _i32([n - 1, n - 1], gpu))
    _attend(gpu, kv, cache, _queries(gpu, 2, q_len, 2 * G, 101), [n, n], True)


@pytest.mark.parametrize("q_len,G", SHAPES)
@pytest.mark.parametrize("kind", ["hidden", "light", "lighter", "none", "early"])
@pytest.mark.parametrize("n", [20, 300])
def test_a_large_step_rounds_nothing_else(gpu, q_len, G, kind, n):
    """Slots whose V steps are 2^30 times the others' and more, which some rows do not see or give hardly any weight:
    the other slots' share of a row keeps its precision."""
    import torch
    kv, cache, k, v = _make(gpu, [n], 2, 320, 110 + n)
    k, v = k.clone(), v.clone()
    q = _queries(gpu, 1, q_len, 2 * G, 111).abs()           # so that a negative key is a light slot
    if kind == "early":                                      # the first blocks of a warp, before its maximum rises
        k[:n // 2] = k[:n // 2] * 0.1 - 3
        v[:n // 2, :, :64] *= 2.0 ** 30
    else:
        at = n - 1 if kind == "hidden" else n // 2
        if kind != "hidden":
            k[at] = {"light": -1.5, "lighter": -4.0, "none": -20.0}[kind]
        v[at, :, :64] *= 2.0 ** 40
    U.ulysses_kv4_append(kv, cache, k, v, _i32([0, n], gpu), _i32([0], gpu))
    _attend(gpu, kv, cache, q, [n], True)


@pytest.mark.parametrize("q_len,G", SHAPES)
@pytest.mark.parametrize("weights", [False, True])
@pytest.mark.parametrize("n", [1, 2, 19])
def test_rows_that_see_nothing_give_zeros_whatever_their_query(gpu, q_len, G, weights, n):
    """Fewer slots than queries: the first ones see none, and what is in them (padding, say) does not count."""
    kv, cache, _, _ = _make(gpu, [n, n], 2, 32, 120)
    q = _queries(gpu, 2, q_len, 2 * G, 121)
    unseen = max(0, q_len - n)
    q[0, :unseen, 0] = float("nan")
    q[0, :unseen, -1, 7] = float("-inf")
    q[1, :unseen, 0, 100] = 2.0 ** 120
    _attend(gpu, kv, cache, q, [n, n], True, weights)


@pytest.mark.parametrize("q_len,G", SHAPES)
@pytest.mark.parametrize("weights", [False, True])
def test_a_zero_query_at_a_very_small_scale(gpu, q_len, G, weights):
    """All logits are 0 however small the scale: equal weights for the slots that are seen."""
    kv, cache, _, _ = _make(gpu, [45], 2, 64, 122)
    q = _queries(gpu, 1, q_len, 2 * G, 123)
    q[:, ::2] = 0
    _attend(gpu, kv, cache, q, [45], True, weights, scale=1e-30)


@pytest.mark.parametrize("q_len,G", SHAPES)
@pytest.mark.parametrize("n", [24, 150])
def test_a_row_without_a_softmax_adds_no_weight_to_slots_it_does_not_see(gpu, q_len, G, n):
    """A query that is not finite makes the weights of the slots it sees NaN, and of no others; nor does a key that is
    not finite reach the weights of rows before it."""
    import torch
    kv, cache, k, v = _make(gpu, [n, n], 2, 160, 130)
    at = kv.weight_offset
    w = torch.rand(2 * 2 * 160, device=gpu)
    cache[at:at + 4 * w.numel()].view(torch.float32).copy_(w)
    q = _queries(gpu, 2, q_len, 2 * G, 131)
    q[0, 0, 0, 5] = float("nan")
    bad = k[2 * n - 1:].clone()
    bad[0, 1, 9] = float("inf")
    U.ulysses_kv4_append(kv, cache, bad, v[2 * n - 1:].contiguous(), _i32([0, 0, 1], gpu), _i32([0, n - 1], gpu))
    _attend(gpu, kv, cache, q, [n, n], True, True)


@pytest.mark.parametrize("q_len,G", SHAPES)
@pytest.mark.parametrize("sign", [1, -1])
def test_logits_past_the_range_of_fp32_give_nan(gpu, q_len, G, sign):
    """Keys and queries of 1e30: no logit that is seen is a number, and the row says so instead of passing for one
    that sees nothing.  The head beside it keeps its results."""
    import torch
    n = 70
    kv, cache, k, v = _make(gpu, [n], 2, 96, 140)
    q = _queries(gpu, 1, q_len, 2 * G, 141)
    out, lse = torch.empty_like(q), torch.empty((1, 2 * G, q_len), device=gpu)
    ws = torch.empty(kv.workspace_bytes(2 * G, q_len, True), dtype=torch.uint8, device=gpu)
    U.ulysses_kv4_attn(kv, cache, q, out, _i32([n], gpu), SCALE, lse=lse, causal=True, workspace=ws)
    want, want_lse = out.clone(), lse.clone()
    k[:, 0] = k[:, 0].abs() * 1e30
    q[:, :, :G] = q[:, :, :G].abs() * (sign * 1e30)
    U.ulysses_kv4_append(kv, cache, k, v, _i32([0, n], gpu), _i32([0], gpu))
    U.ulysses_kv4_attn(kv, cache, q, out, _i32([n], gpu), SCALE, lse=lse, causal=True, weights=True, workspace=ws)
    assert torch.isnan(out[:, :, :G]).all() and torch.isnan(lse[:, :G]).all()
    assert torch.equal(out[:, :, G:], want[:, :, G:]) and torch.equal(lse[:, G:], want_lse[:, G:])
    w = torch.from_numpy(_host(kv, cache).weight)[0]
    assert torch.isnan(w[0, :n]).all() and not torch.isnan(w[1, :n]).any()
    U.ulysses_kv4_attn(kv, cache, q, out, _i32([0], gpu), SCALE, lse=lse, workspace=ws)
    assert not bool(out.any()) and bool((lse == float("-inf")).all())


@pytest.mark.parametrize("q_len,G", SHAPES)
def test_small_query_values_keep_their_bits(gpu, q_len, G):
    """Values down to 2^-28 of the power of two of their row's largest enter with all 8 bits: a query whose second
    group is that small against keys whose second group is as much larger (and whose first is 0)."""
    n = 90
    kv, cache, k, v = _make(gpu, [n], 2, 96, 150)
    q = _queries(gpu, 1, q_len, 2 * G, 151)
    small = q[..., 64:].abs().clamp(1, 1.9921875) * q[..., 64:].sign()
    q[..., :64] = 0
    q[..., 0] = 1.9921875
    q[..., 64:] = small * 2.0 ** -28
    k[..., :64] = 0
    k[..., 64:] *= 2.0 ** 28
    U.ulysses_kv4_append(kv, cache, k, v, _i32([0, n], gpu), _i32([0], gpu))
    _attend(gpu, kv, cache, q, [n], True)


def test_a_load_of_many_tokens_equals_loads_of_few(gpu):
    """Ragged sequences at odd slots in one call, which takes runs of tokens, against a call a sequence, which takes
    one at a time; two heads against the held values."""
    import torch
    heads, lens, start = 56, [40, 0, 7, 1, 5, 60, 3], [3, 0, 31, 95, 30, 33, 64]
    B = len(lens)
    kv, cache, _, _ = _make(gpu, [96] * B, heads, 96, 160)
    host = _host(kv, cache)
    n = sum(lens)
    k = torch.full((n + 2, heads, D), 9.0, dtype=torch.bfloat16, device=gpu)
    v = torch.full_like(k, 9.0)
    U.ulysses_kv4_load(kv, cache, k, v, _i32(_cu(lens), gpu), _i32(start, gpu))
    one_k, one_v = torch.full_like(k, 9.0), torch.full_like(k, 9.0)
    at = 0
    for b, m in enumerate(lens):
        cu = [0] * (b + 1) + [m] * (B - b)
        U.ulysses_kv4_load(kv, cache, one_k[at:at + m], one_v[at:at + m], _i32(cu, gpu), _i32(start, gpu))
        for h in (0, heads - 1):
            for plane, got in ((0, k), (1, v)):
                want, _ = host.values(b, h, start[b], start[b] + m, plane)
                assert np.array_equal(_bits(got[at:at + m, h]), orc.f64_to_bf16(want))
        at += m
    assert torch.equal(k, one_k) and torch.equal(v, one_v)
    assert bool((k[n:] == 9).all()) and U.ulysses_kv4_last_device_error(kv) == 0


@pytest.mark.parametrize("q_len,G", SHAPES)
@pytest.mark.parametrize("kind", ["within", "beyond", "zeros"])
def test_steps_of_one_block_that_differ(gpu, q_len, G, kind):
    """The first power of two by the block's least step (steps within 2^8 of each other) and by each row's largest
    p s (beyond that, and beside rows of one value, whose step is 0), for rows that look at different slots."""
    import torch
    n = 61
    kv, cache, k, v = _make(gpu, [n], 2, 64, 170)
    g = torch.Generator(device=gpu)
    g.manual_seed(171)
    wide = torch.rand((n, 2, 1), generator=g, device=gpu) * {"within": 7.0, "beyond": 24.0, "zeros": 3.0}[kind]
    v = (v * torch.exp2(wide)).to(torch.bfloat16)
    if kind == "zeros":
        v[::3, :, :64] = v[::3, :, :1]
        v[1::5, :, 64:] = 0
    q = _queries(gpu, 1, q_len, 2 * G, 172) * 4              # sharp: a row's weight sits on a few slots
    U.ulysses_kv4_append(kv, cache, k, v, _i32([0, n], gpu), _i32([0], gpu))
    _attend(gpu, kv, cache, q, [n], True, True)
