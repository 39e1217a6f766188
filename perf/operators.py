"""Cases that measure the 4-bit K/V cache operators: append, load, attention and eviction.

Each case builds its inputs with ``prepare``; ``run`` makes one pass, either through the plain PyTorch
form of the operators below (``own`` false) or through the library's entry points (``own`` true);
``exact`` gives the same outputs from the definition in 64 bits.

The cache.  A (sequence, head) pair has ``capacity`` slots in blocks of 32.  A block is 4608 bytes:
K codes (32 slots x 64 bytes), V codes (32 x 64 bytes), then 32 x 8 bf16 values
(ks0, km0, ks1, km1, vs0, vm0, vs1, vm1).  A row of 128 values is two groups of 64 (d < 64, d >= 64);
in each group  x ~ m + s * n  with  m = min(x),  s = bf16((max(x) - min(x)) / 15)  and the code
n = round((x - m) / s) in 0..15 (0 where s is 0; a group that is not finite is held as s = m = NaN).
Byte 8 g + 4 w + i of a row holds the codes of d = 64 w + 8 g + 2 i (low half) and of the next d (high
half).  After the blocks of all pairs come the accumulated attention weights (fp32) and the token
positions (int32), each [batch, heads, capacity].
"""
import math
import random

import torch

own = False

D = 128
BLOCK = 32
BLOCK_BYTES = 4608
LOG2E = 1.0 / math.log(2.0)


# ------------------------------------------------------------------------------------------ cases

def listed():
    return [
        # one decoding step of the tiny layer (8 heads, 1024 tokens): launch latency
        dict(name="attn_tiny", kind="attn", batch=1, heads=8, group=1, q_len=1, longest=1024, weights=False,
             causal=False, lens_seed=0),
        # one decoding step against a cached Video-DiT sequence, keeping the weights that eviction goes by
        dict(name="attn_dit19k", kind="attn", batch=1, heads=56, group=1, q_len=1, longest=19394, weights=True,
             causal=False, lens_seed=0),
        # one decoding step against the long clip: the largest cache of one sequence
        dict(name="attn_long104k", kind="attn", batch=1, heads=56, group=1, q_len=1, longest=104448, weights=False,
             causal=False, lens_seed=0),
        # a served batch of ragged lengths whose 7 query heads share a K/V head, keeping the weights
        dict(name="attn_batch", kind="attn", batch=24, heads=8, group=7, q_len=1, longest=8191, weights=True,
             causal=False, lens_seed=4),
        # a block of 8 new tokens at a time, causal among themselves, 2 query heads for each K/V head
        dict(name="attn_block", kind="attn", batch=5, heads=14, group=2, q_len=8, longest=19394, weights=False,
             causal=True, lens_seed=5),
        # a whole Video-DiT prompt quantised into an empty cache
        dict(name="append_dit19k", kind="append", batch=1, heads=56, new=19394, before=0, lens_seed=0),
        # the new token of every sequence of a decoding batch
        dict(name="append_token", kind="append", batch=48, heads=8, new=1, before=2047, lens_seed=7),
        # chunks of prompts of ragged lengths behind what is cached already
        dict(name="append_ragged", kind="append", batch=7, heads=14, new=1025, before=513, lens_seed=8),
        # the cached prefix of a long prompt brought back as bf16 rows for the attention of its next chunk
        dict(name="load_clip38k", kind="load", batch=1, heads=56, span=38912, before=0, lens_seed=0),
        # parts of several short sequences, from odd slots
        dict(name="load_ragged", kind="load", batch=6, heads=8, span=777, before=129, lens_seed=10),
        # the long clip's cache cut down to a budget after its prompt
        dict(name="evict_long104k", kind="evict", batch=1, heads=56, longest=104448, keep=8192, sink=4, recent=1024,
             lens_seed=0),
        # a decoding batch that has run past its budget, cut back to it
        dict(name="evict_budget", kind="evict", batch=24, heads=8, longest=2303, keep=2047, sink=4, recent=255,
             lens_seed=12),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["attn", "attn", "attn", "append", "load", "evict"])
    heads = rng.choice([1, 2, 3, 4, 7, 8, 14, 28, 56])
    batch = _log(rng, 1, 48)
    seed = rng.randrange(1 << 30)
    room = 56 * 104448 // (heads * batch)            # slots of a sequence at the largest listed cache
    if kind == "attn":
        group = rng.choice([1, 1, 2, 4, 5, 7, 8])
        q_len = rng.choice([1, 1, 1, 2, 3, 5, 8])
        rows = -(-group * q_len // 8)
        longest = _log(rng, 1, max(1, min(104448, room // rows)))
        return dict(kind=kind, batch=batch, heads=heads, group=group, q_len=q_len, longest=longest,
                    weights=rng.random() < 0.5, causal=q_len > 1 and rng.random() < 0.7, lens_seed=seed)
    if kind == "append":
        most = max(1, 56 * 19394 // (heads * batch))
        return dict(kind=kind, batch=batch, heads=heads, new=_log(rng, 1, min(38912, most)),
                    before=rng.choice([0, _log(rng, 1, 4096)]), lens_seed=seed)
    if kind == "load":
        most = max(1, 56 * 38912 // (heads * batch))
        return dict(kind=kind, batch=batch, heads=heads, span=_log(rng, 1, min(104448, most)),
                    before=rng.choice([0, _log(rng, 1, 4096)]), lens_seed=seed)
    longest = _log(rng, 2, max(2, min(104448, room)))
    keep = _log(rng, 1, max(1, min(longest, 56 * 8192 // (heads * batch))))
    sink = rng.randint(0, min(keep, 8))
    return dict(kind=kind, batch=batch, heads=heads, longest=longest, keep=keep, sink=sink,
                recent=rng.randint(0, keep - sink), lens_seed=seed)


def _spread(case, most):
    """The sequences' lengths: the longest, then ragged ones, an empty one among four or more."""
    r = random.Random(case["lens_seed"])
    lens = [most] + [r.randint((most + 3) // 4, most) for _ in range(case["batch"] - 1)]
    if case["batch"] >= 4 and case["kind"] != "append":
        lens[2] = 0
    return lens


def _lens(case):
    return _spread(case, case[{"attn": "longest", "evict": "longest", "append": "new", "load": "span"}[case["kind"]]])


def work(case):
    lens, heads = _lens(case), case["heads"]
    slots = sum(lens) * heads
    row = 2 * 64 + 16                                # K and V codes, scales and minima of one slot
    if case["kind"] == "attn":
        rows = case["batch"] * case["q_len"] * heads * case["group"]
        b = slots * (row + (8 if case["weights"] else 0)) + rows * (2 * 2 * D + 4)
        return {"bytes": b, "flops": 4 * D * slots * case["group"] * case["q_len"]}
    if case["kind"] == "append":                     # rows in, slots out with weight and position, read back, rows out
        return {"bytes": slots * (4 * D + row + 8 + row + 4 * D), "flops": slots * 2 * D * 4}
    if case["kind"] == "load":
        return {"bytes": slots * (row + 4 * D), "flops": slots * 4 * D}
    kept = sum(min(n, case["keep"]) for n in lens) * heads
    return {"bytes": slots * 4 + kept * (2 * row + 4 * 3 + row + 4 * D), "flops": kept * 4 * D}


# ------------------------------------------------------------------------------------------ inputs

def _sections(cache, batch, heads, capacity):
    """The blocks [batch, heads, capacity / 32, 4608], weights and positions of a cache's bytes."""
    n = batch * heads * capacity
    nb = n // BLOCK * BLOCK_BYTES
    blocks = cache[:nb].view(batch, heads, capacity // BLOCK, BLOCK_BYTES)
    weight = cache[nb:nb + 4 * n].view(torch.float32).view(batch, heads, capacity)
    pos = cache[nb + 4 * n:nb + 8 * n].view(torch.int32).view(batch, heads, capacity)
    return blocks, weight, pos


def _capacity(n):
    return max(BLOCK, (n + BLOCK - 1) // BLOCK * BLOCK)


def _int32(v, dev):
    return torch.tensor(v, dtype=torch.int32, device=dev)


def _filled(batch, heads, capacity, g, dev):
    """A cache as appends of normalised rows leave it: random codes, steps around 0.3 and minima around -2.3."""
    n = batch * heads * capacity
    cache = torch.randint(0, 256, (n // BLOCK * BLOCK_BYTES + 8 * n,), generator=g, device=dev, dtype=torch.uint8)
    blocks, weight, pos = _sections(cache, batch, heads, capacity)
    step = torch.rand((batch, heads, capacity, 4, 1), generator=g, device=dev) * 0.2 + 0.2
    low = -step * (6.5 + 2 * torch.rand(step.shape, generator=g, device=dev))
    meta = torch.cat([step, low], -1).to(torch.bfloat16).view(batch, heads, capacity // BLOCK, BLOCK * 8)
    blocks[..., 4096:] = meta.view(torch.uint8).view(batch, heads, capacity // BLOCK, BLOCK * 16)
    # attention mass is spread unevenly over the slots; slots that nothing has looked at yet tie at zero
    w = torch.exp(2.0 * torch.randn(weight.shape, generator=g, device=dev)) / capacity
    weight.copy_(torch.where(torch.rand(w.shape, generator=g, device=dev) < 0.1, torch.zeros_like(w), w))
    pos.copy_(torch.arange(capacity, device=dev, dtype=torch.int32).expand(pos.shape))
    return cache


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    kind, batch, heads = case["kind"], case["batch"], case["heads"]
    lens = _lens(case)
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    s = dict(kind=kind, batch=batch, heads=heads, lens=lens, case=case)
    s["before"] = case.get("before", 0)
    s["capacity"] = _capacity(max(lens) + s["before"])
    s["host"] = random.Random(case["lens_seed"] + 1)
    if kind in ("append", "load"):
        starts = [s["host"].randint(s["before"] // 2, s["before"]) for _ in range(batch)]
        s["starts"], s["start"], s["cu"] = starts, _int32(starts, dev), _int32(cu, dev)
        s["index"] = _index(lens, starts, dev)
        s["k_out"] = torch.zeros((cu[-1], heads, D), dtype=torch.bfloat16, device=dev)
        s["v_out"] = torch.zeros_like(s["k_out"])
    if kind == "append":
        s["cache"] = torch.zeros(batch * heads * s["capacity"] // BLOCK * (BLOCK_BYTES + 8 * BLOCK),
                                 dtype=torch.uint8, device=dev)
        # the K and V planes of packed rows [n, 3, heads, 128], as the layer takes them
        packed = torch.empty((cu[-1], 3, heads, D), dtype=torch.bfloat16, device=dev)
        for plane in range(3):
            packed[:, plane] = torch.randn((cu[-1], heads, D), generator=g, device=dev)
        s["packed"] = packed
    else:
        s["cache"] = _filled(batch, heads, s["capacity"], g, dev)
    if kind == "attn":
        hq = heads * case["group"]
        s["lengths"] = _int32(lens, dev)
        # a query looks for some keys more than for others: noise plus a part of one cached key
        q = torch.randn((batch, case["q_len"], hq, D), generator=g, device=dev)
        at = torch.randint(0, max(lens), (batch,), generator=g, device=dev)
        blocks, _, _ = _sections(s["cache"], batch, heads, s["capacity"])
        k, _ = _values(blocks[torch.arange(batch, device=dev), :, at // BLOCK].view(batch, heads, 1, BLOCK_BYTES))
        k = k[torch.arange(batch, device=dev), :, at % BLOCK]
        q += 0.5 * k.repeat_interleave(case["group"], 1)[:, None]
        s["q"] = q.to(torch.bfloat16)
        s["out"] = torch.zeros_like(s["q"])
        s["lse"] = torch.zeros((batch, hq, case["q_len"]), device=dev)
        s["scale"] = 1.0 / math.sqrt(D)
    if kind == "evict":
        kept = [min(n, case["keep"]) for n in lens]
        s["kept"], s["to"] = kept, _capacity(case["keep"])
        s["lengths"] = _int32(lens, dev)
        s["new_lengths"] = torch.zeros(batch, dtype=torch.int32, device=dev)
        s["dst"] = torch.zeros(batch * heads * s["to"] // BLOCK * (BLOCK_BYTES + 8 * BLOCK), dtype=torch.uint8,
                               device=dev)
        cu = [0]
        for n in kept:
            cu.append(cu[-1] + n)
        s["cu"], s["start"] = _int32(cu, dev), _int32([0] * batch, dev)
        s["index"] = _index(kept, [0] * batch, dev)
        s["k_out"] = torch.zeros((cu[-1], heads, D), dtype=torch.bfloat16, device=dev)
        s["v_out"] = torch.zeros_like(s["k_out"])
    if own:
        import ulysses_sequence_attention_repack_b200 as U
        s["U"] = U
        s["kv"] = U.ulysses_kv4_plan(batch, heads, D, s["capacity"])
        if kind == "evict":
            s["kv_dst"] = U.ulysses_kv4_plan(batch, heads, D, s["to"])
        if kind == "attn":
            n = s["kv"].workspace_bytes(heads * case["group"], case["q_len"], case["weights"])
            s["workspace"] = torch.empty(max(n, 1), dtype=torch.uint8, device=dev)
    return s


def _index(lens, starts, dev):
    """The sequence and the slot of every row of a packed batch."""
    n = torch.tensor(lens, device=dev)
    b = torch.repeat_interleave(torch.arange(len(lens), device=dev), n)
    first = torch.cumsum(n, 0) - n
    return b, torch.arange(b.numel(), device=dev) - first[b] + torch.tensor(starts, device=dev)[b]


# ------------------------------------------------------------------------------------------ the plain form

def _unpack(codes):
    """Codes 0..15 [..., 128] of rows of 64 bytes."""
    lead = codes.shape[:-1]
    n = torch.stack([codes & 15, codes >> 4], -1).view(*lead, 8, 2, 4, 2)
    return n.transpose(-4, -3).reshape(*lead, D)


def _values(blocks):
    """K and V in fp32, [batch, heads, slots, 128] each, of whole blocks."""
    b, h, nb, _ = blocks.shape
    meta = blocks[..., 4096:].reshape(b, h, nb * BLOCK, 16).view(torch.bfloat16).float()
    out = []
    for i in (0, 1):
        n = _unpack(blocks[..., 2048 * i:2048 * (i + 1)].reshape(b, h, nb * BLOCK, 64))
        m = meta[..., 4 * i:4 * i + 4].reshape(b, h, nb * BLOCK, 2, 2)
        n = n.float().view(b, h, nb * BLOCK, 2, 64)
        out.append((n * m[..., 0:1] + m[..., 1:2]).view(b, h, nb * BLOCK, D))
    return out


def _quantise(x):
    """The 64 code bytes and the (s, m) pairs of two groups, of rows [..., 128]."""
    lead = x.shape[:-1]
    g = x.float().view(*lead, 2, 64)
    m = g.amin(-1)
    s = ((g.amax(-1) - m) / 15.0).to(torch.bfloat16).float()
    bad = ~(torch.isfinite(s) & torch.isfinite(m))
    n = torch.round((g - m[..., None]) / s[..., None]).clamp(0, 15)
    n = torch.where(((s == 0) | bad)[..., None], torch.zeros_like(n), n).to(torch.uint8)
    nan = torch.full_like(s, math.nan)
    pairs = torch.stack([torch.where(bad, nan, s), torch.where(bad, nan, m)], -1)
    n = n.view(*lead, 2, 8, 4, 2).transpose(-4, -3)
    return (n[..., 0] | (n[..., 1] << 4)).reshape(*lead, 64), pairs.to(torch.bfloat16).view(*lead, 4)


def _part(blocks, first, wide):
    """The rows of `wide` bytes that begin at byte `first` of the blocks: [batch, heads, blocks, 32, wide]."""
    return blocks[..., first:first + BLOCK * wide].unflatten(-1, (BLOCK, wide))


def _plain_load(s, cache, capacity):
    blocks, _, _ = _sections(cache, s["batch"], s["heads"], capacity)
    b, slot = s["index"]
    block, at = slot // BLOCK, slot % BLOCK
    meta = _part(blocks, 4096, 16)[b, :, block, at].view(torch.bfloat16).float()      # [rows, heads, 8]
    for i, to in ((0, s["k_out"]), (1, s["v_out"])):
        n = _unpack(_part(blocks, 2048 * i, 64)[b, :, block, at]).float().unflatten(-1, (2, 64))
        m = meta[..., 4 * i:4 * i + 4].unflatten(-1, (2, 2))
        to.copy_((n * m[..., 0:1] + m[..., 1:2]).flatten(-2))


def _plain_append(s):
    blocks, weight, pos = _sections(s["cache"], s["batch"], s["heads"], s["capacity"])
    b, slot = s["index"]
    kc, km = _quantise(s["packed"][:, 1])
    vc, vm = _quantise(s["packed"][:, 2])
    meta = torch.cat([km, vm], -1).view(torch.uint8)                          # [rows, heads, 16]
    block, at = slot // BLOCK, slot % BLOCK
    for first, wide, data in ((0, 64, kc), (2048, 64, vc), (4096, 16, meta)):
        _part(blocks, first, wide)[b, :, block, at] = data
    weight[b, :, slot] = 0.0
    pos[b, :, slot] = slot.to(torch.int32)[:, None]
    return weight, pos


def _plain_attn(s):
    case, batch, heads, group = s["case"], s["batch"], s["heads"], s["case"]["group"]
    q_len = case["q_len"]
    blocks, weight, _ = _sections(s["cache"], batch, heads, s["capacity"])
    k, v = _values(blocks)
    rows = q_len * group
    q = s["q"].float().view(batch, q_len, heads, group, D).permute(0, 2, 1, 3, 4).reshape(batch, heads, rows, D)
    logits = torch.matmul(q, k.transpose(-1, -2)) * s["scale"]
    slot = torch.arange(s["capacity"], device=k.device)
    limit = s["lengths"].long()[:, None].expand(batch, q_len)
    if case["causal"]:
        limit = limit - (q_len - 1) + torch.arange(q_len, device=k.device)
    seen = slot < limit.repeat_interleave(group, 1)[:, None, :, None]          # [batch, 1, rows, slots]
    logits = torch.where(seen, logits, -math.inf)
    top = logits.amax(-1, keepdim=True)
    e = torch.exp(logits - torch.where(torch.isinf(top), torch.zeros_like(top), top))
    total = e.sum(-1, keepdim=True)
    p = torch.where(total > 0, e / total, torch.zeros_like(e))
    beyond = (slot >= s["lengths"].long()[:, None])[:, None, :, None]
    o = torch.matmul(p, torch.where(beyond, torch.zeros_like(v), v))
    if case["weights"]:
        weight += p.sum(2)
    lse = torch.where(total > 0, (top + torch.log(total)) * LOG2E, -math.inf)
    s["out"].copy_(o.view(batch, heads, q_len, group, D).permute(0, 2, 1, 3, 4).reshape(s["out"].shape))
    s["lse"].copy_(lse.view(batch, heads, q_len, group).permute(0, 1, 3, 2).reshape(s["lse"].shape))
    return (s["out"], s["lse"], weight) if case["weights"] else (s["out"], s["lse"])


def _plain_evict(s):
    case, batch, heads = s["case"], s["batch"], s["heads"]
    blocks, weight, pos = _sections(s["cache"], batch, heads, s["capacity"])
    to, to_weight, to_pos = _sections(s["dst"], batch, heads, s["to"])
    slot = torch.arange(s["capacity"], device=weight.device)
    n = s["lengths"].long()[:, None, None]
    # protected slots first, then by weight, the lower slot first among equals; no slot behind the length
    rank = torch.where((slot < case["sink"]) | (slot >= n - case["recent"]), math.inf, weight)
    rank = torch.where(slot < n, rank, -math.inf)
    order = torch.sort(rank, dim=-1, descending=True, stable=True).indices[..., :case["keep"]]
    order = torch.where(torch.arange(order.shape[-1], device=n.device) < n, order, s["capacity"])
    order = torch.sort(order, dim=-1).values                                   # slots in their order, the missing last
    kept = torch.clamp(s["lengths"], max=case["keep"])
    s["new_lengths"].copy_(kept)
    here = (order < s["capacity"]).nonzero(as_tuple=True)
    b, h, j = here
    src = order[here]
    to_weight[b, h, j] = weight[b, h, src]
    to_pos[b, h, j] = pos[b, h, src]
    for first, wide in ((0, 64), (2048, 64), (4096, 16)):
        rows = _part(blocks, first, wide)[b, h, src // BLOCK, src % BLOCK]
        _part(to, first, wide)[b, h, j // BLOCK, j % BLOCK] = rows
    return to_weight, to_pos


def run(state):
    """One pass.  What is held in 4 bits comes back as bf16 rows, by the load that a user would make."""
    s, kind = state, state["kind"]
    if kind == "append":
        if own:
            U = s["U"]
            k, v = s["packed"][:, 1], s["packed"][:, 2]
            U.ulysses_kv4_append(s["kv"], s["cache"], k, v, s["cu"], s["start"])
            U.ulysses_kv4_load(s["kv"], s["cache"], s["k_out"], s["v_out"], s["cu"], s["start"])
            _, weight, pos = _sections(s["cache"], s["batch"], s["heads"], s["capacity"])
        else:
            weight, pos = _plain_append(s)
            _plain_load(s, s["cache"], s["capacity"])
        return {"k": s["k_out"], "v": s["v_out"], "weight": weight, "pos": pos}
    if kind == "load":
        if own:
            s["U"].ulysses_kv4_load(s["kv"], s["cache"], s["k_out"], s["v_out"], s["cu"], s["start"])
        else:
            _plain_load(s, s["cache"], s["capacity"])
        return {"k": s["k_out"], "v": s["v_out"]}
    if kind == "evict":
        case = s["case"]
        if own:
            U = s["U"]
            U.ulysses_kv4_evict(s["kv"], s["cache"], s["kv_dst"], s["dst"], s["lengths"], s["new_lengths"],
                                case["keep"], case["sink"], case["recent"])
            U.ulysses_kv4_load(s["kv_dst"], s["dst"], s["k_out"], s["v_out"], s["cu"], s["start"])
            _, weight, pos = _sections(s["dst"], s["batch"], s["heads"], s["to"])
        else:
            weight, pos = _plain_evict(s)
            _plain_load(s, s["dst"], s["to"])
        return {"k": s["k_out"], "v": s["v_out"], "weight": weight, "pos": pos, "new_lengths": s["new_lengths"]}
    case = s["case"]
    if own:
        s["U"].ulysses_kv4_attn(s["kv"], s["cache"], s["q"], s["out"], s["lengths"], s["scale"], lse=s["lse"],
                                causal=case["causal"], weights=case["weights"], workspace=s["workspace"])
        got = [s["out"], s["lse"]]
        if case["weights"]:
            got.append(_sections(s["cache"], s["batch"], s["heads"], s["capacity"])[1])
    else:
        got = _plain_attn(s)
    return dict(zip(("out", "lse", "weight"), got))


# ------------------------------------------------------------------------------------------ 64 bits

def _nibbles64(rows):
    """float64 codes [n, 128] of rows [n, 64] of bytes, word by word."""
    words = rows.contiguous().view(torch.int32).long()                         # [n, 16]
    codes = torch.empty((rows.shape[0], D), dtype=torch.float64, device=rows.device)
    for w in range(16):
        first = 64 * (w % 2) + 8 * (w // 2)
        for j in range(8):
            codes[:, first + j] = ((words[:, w] >> (4 * j)) & 15).double()
    return codes


def _head64(blocks, b, h, lo, hi):
    """K and V in float64, [hi - lo, 128] each, of slots lo..hi of one sequence and head."""
    part = blocks[b, h, lo // BLOCK:(hi + BLOCK - 1) // BLOCK]
    cut = slice(lo % BLOCK, lo % BLOCK + hi - lo)
    scales = part[:, 4096:].reshape(-1, 16)[cut].contiguous().view(torch.bfloat16).double()
    out = []
    for i in (0, 1):
        x = _nibbles64(part[:, 2048 * i:2048 * i + 2048].reshape(-1, 64)[cut])
        for w in (0, 1):
            x[:, 64 * w:64 * w + 64] *= scales[:, 4 * i + 2 * w, None]
            x[:, 64 * w:64 * w + 64] += scales[:, 4 * i + 2 * w + 1, None]
        out.append(x)
    return out


def _exact_rows(s, blocks, lens, starts):
    k = torch.empty(s["k_out"].shape, dtype=torch.float64, device=s["k_out"].device)
    v = torch.empty_like(k)
    at = 0
    for b, n in enumerate(lens):
        for h in range(s["heads"]):
            if n:
                k[at:at + n, h], v[at:at + n, h] = _head64(blocks, b, h, starts[b], starts[b] + n)
        at += n
    return k, v


def _exact_group(x):
    """The value that each element of rows [n, 64] is held as."""
    x = x.double()
    low = x.min(1, keepdim=True).values
    step = ((x.max(1, keepdim=True).values - low) / 15).to(torch.bfloat16).double()
    n = torch.clamp(torch.round((x - low) / torch.where(step == 0, torch.ones_like(step), step)), 0, 15)
    return low + step * torch.where(step == 0, torch.zeros_like(n), n)


def exact(case, seed):
    s = prepare(case, seed)
    kind, batch, heads = s["kind"], s["batch"], s["heads"]
    if batch * heads > 1024:
        return None
    blocks, weight, pos = _sections(s["cache"], batch, heads, s["capacity"])
    if kind == "append":
        k = torch.empty(s["k_out"].shape, dtype=torch.float64, device=blocks.device)
        v = torch.empty_like(k)
        for h in range(heads):
            for plane, to in ((1, k), (2, v)):
                for w in (0, 1):
                    to[:, h, 64 * w:64 * w + 64] = _exact_group(s["packed"][:, plane, h, 64 * w:64 * w + 64])
        return {"k": k, "v": v, "weight": weight.double(), "pos": None}
    if kind == "load":
        k, v = _exact_rows(s, blocks, s["lens"], s["starts"])
        return {"k": k, "v": v}
    if kind == "evict":
        to_weight = torch.zeros((batch, heads, s["to"]), dtype=torch.float64, device=blocks.device)
        k = torch.empty(s["k_out"].shape, dtype=torch.float64, device=blocks.device)
        v = torch.empty_like(k)
        at = 0
        for b, (n, keep) in enumerate(zip(s["lens"], s["kept"])):
            for h in range(heads):
                if not n:
                    continue
                w = weight[b, h, :n].double()
                held = torch.zeros(n, dtype=torch.bool, device=w.device)
                if n <= keep:
                    held[:] = True
                else:
                    held[:case["sink"]] = True
                    held[n - case["recent"]:] = True
                    free = (~held).nonzero()[:, 0]
                    # the k-th largest, and as many of its equals as there is room for, from the front
                    room = keep - int(held.sum())
                    if room:
                        least = torch.topk(w[free], room).values[-1]
                        held[free[w[free] > least]] = True
                        held[free[w[free] == least][:keep - int(held.sum())]] = True
                at_slots = held.nonzero()[:, 0]
                to_weight[b, h, :keep] = w[at_slots]
                kk, vv = _head64(blocks, b, h, 0, n)
                k[at:at + keep, h], v[at:at + keep, h] = kk[at_slots], vv[at_slots]
            at += keep
        return {"k": k, "v": v, "weight": to_weight, "pos": None, "new_lengths": None}
    group, q_len = case["group"], case["q_len"]
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=blocks.device)
    lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device=blocks.device)
    total = weight.double()
    for b, n in enumerate(s["lens"]):
        for h in range(heads):
            if not n:
                continue
            k, v = _head64(blocks, b, h, 0, n)
            for i in range(q_len):
                m = n - (q_len - 1 - i) if case["causal"] else n
                if m <= 0:
                    continue
                for j in range(h * group, (h + 1) * group):
                    x = k[:m] @ s["q"][b, i, j].double() * s["scale"]
                    z = torch.logsumexp(x, 0)
                    p = torch.exp(x - z)
                    out[b, i, j] = p @ v[:m]
                    lse[b, j, i] = z / math.log(2.0)
                    total[b, h, :m] += p
    got = {"out": out, "lse": lse}
    return dict(got, weight=total) if case["weights"] else got
