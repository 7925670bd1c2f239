"""The attention-side operators of a decode layer, in plain torch and as the library's calls.

Operators (one case names one):
  rope    per-head RMS norm of queries and keys (optional) and rotary positions, one pass
  append  new keys and values quantised into the 8-bit cache, and read back as the values it holds
  attend  attention over the 8-bit cache, one token per sequence or a prompt's chunk; with "score"
          the softmax weights are also added up per block of tokens and kv head
  evict   blocks with the least accumulated weight leave the cache's table

The cache.  A block is 32 tokens of one kv head and is one page of two halves of 32*D unsigned
bytes (keys, values) with a scale each: the value is scale * (code - 128), where scale = amax / 127 in
32 bits, code = 128 + rint(127 * x / amax) and amax is the block's largest magnitude.  The last,
partly filled block's rows are also kept as they came ("open"), and its codes follow from them anew
with every append.  Byte orders inside a page:
  keys    [token / 16][d / 64][(d / 16) % 4][token % 16][d % 16]
  values  [d / 32][g][d % 16][(d / 16) % 2][j], token = 16 * (j / 4) + 4 * g + j % 4 (g < 4, j < 8)
table[sequence][kv head][block] names the page.  lens[sequence] counts the tokens held, those
of the call among them.
"""

import math

import numpy as np
import torch

own = False

BLOCK = 32
DTYPES = {"f16": torch.float16, "f32": torch.float32}


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one decode token of a Llama2-70B-shaped layer: latency is all of it
        dict(name="rope, one token", op="rope", dtype="f16", tokens=1, heads=64, kv_heads=8, head_dim=128,
             rot=128, layout="half", norm=False, scaling="none", first=4095),
        # a prompt of that shape with per-head norms, positions scaled for a long context
        dict(name="rope, prompt, norms, scaled", op="rope", dtype="f16", tokens=4096, heads=64, kv_heads=8,
             head_dim=128, rot=128, layout="half", norm=True, scaling="yarn", first=120000),
        # part of the head rotated in the interleaved layout, fp32, an odd token count
        dict(name="rope, part of the head, fp32", op="rope", dtype="f32", tokens=777, heads=56, kv_heads=56,
             head_dim=128, rot=32, layout="interleaved", norm=False, scaling="linear", first=5000),
        # a decode step of eight sequences
        dict(name="append, a token each", op="append", dtype="f16", seqs=8, new=1, before=4113, step=37,
             kv_heads=8, head_dim=128),
        # two prompts' chunks behind cached tokens, Falcon-40B-shaped heads (64 wide)
        dict(name="append, prompts", op="append", dtype="f16", seqs=2, new=2047, before=530, step=95,
             kv_heads=8, head_dim=64),
        # one decode token over a short chat turn
        dict(name="attend, short", op="attend", dtype="f16", seqs=1, new=1, length=131, step=0, heads=64,
             kv_heads=8, head_dim=128, score=False),
        # a serving batch of decode tokens, ragged lengths, weights accumulated for eviction
        dict(name="attend, batch, scores", op="attend", dtype="f16", seqs=32, new=1, length=16384, step=211,
             heads=64, kv_heads=8, head_dim=128, score=True),
        # one decode token over a long document
        dict(name="attend, long", op="attend", dtype="f16", seqs=1, new=1, length=131072, step=0, heads=64,
             kv_heads=8, head_dim=128, score=False),
        # fp32, every head with keys of its own (OPT-30B-shaped heads)
        dict(name="attend, fp32, own heads", op="attend", dtype="f32", seqs=4, new=1, length=4001, step=577,
             heads=56, kv_heads=56, head_dim=128, score=False),
        # a prompt's chunk over what is cached, Falcon-40B-shaped heads (16 queries' heads to a key's)
        dict(name="attend, prompt chunk", op="attend", dtype="f16", seqs=1, new=512, length=8200, step=0,
             heads=128, kv_heads=8, head_dim=64, score=False),
        # one sequence over its budget
        dict(name="evict, one sequence", op="evict", seqs=1, kv_heads=8, blocks=130, step=0, keep=96, recent=8),
        # a batch of long sequences
        dict(name="evict, batch, long", op="evict", seqs=32, kv_heads=8, blocks=4096, step=50, keep=2048,
             recent=32),
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "attend", "attend", "evict"])
    dtype = rng.choice(["f16", "f16", "f32"])
    head_dim = rng.choice([64, 128])
    kv_heads = rng.choice([1, 2, 7, 8])
    group = rng.choice([1, 3, 8, 16])
    if op == "rope":
        return dict(op=op, dtype=dtype, tokens=_log(rng, 1, 2048), heads=kv_heads * group // 2 + 1,
                    kv_heads=kv_heads, head_dim=head_dim, rot=rng.choice([head_dim, head_dim // 2, 20]),
                    layout=rng.choice(["half", "interleaved"]), norm=rng.random() < 0.5,
                    scaling=rng.choice(["none", "linear", "ntk", "yarn"]), first=_log(rng, 1, 1000000))
    if op == "append":
        return dict(op=op, dtype=dtype, seqs=rng.randint(1, 4), new=_log(rng, 1, 1500),
                    before=_log(rng, 1, 5000), step=rng.randint(0, 100), kv_heads=kv_heads, head_dim=head_dim)
    if op == "attend":
        new = rng.choice([1, 1, 1, _log(rng, 2, 200)])
        seqs = _log(rng, 1, 12) if new == 1 else rng.randint(1, 2)
        length = new + _log(rng, 1, 30000 if new == 1 else 6000)
        return dict(op=op, dtype=dtype, seqs=seqs, new=new, length=length, step=rng.randint(0, length // seqs),
                    heads=kv_heads * group, kv_heads=kv_heads, head_dim=head_dim, score=rng.random() < 0.4)
    blocks = _log(rng, 20, 4000)
    return dict(op=op, seqs=rng.randint(1, 16), kv_heads=kv_heads, blocks=blocks, step=rng.randint(0, 5),
                keep=max(9, int(blocks * rng.uniform(0.3, 0.95))), recent=rng.randint(1, 8))


def _lens(case):
    """Tokens held per sequence (the call's own among them); ragged by `step`."""
    if case["op"] == "append":
        return [max(0, case["before"] - s * case["step"]) + case["new"] for s in range(case["seqs"])]
    if case["op"] == "evict":
        return [max(1, (case["blocks"] - s * case["step"]) * BLOCK - 5 * (s + 1)) for s in range(case["seqs"])]
    return [max(case["new"], case["length"] - s * case["step"]) for s in range(case["seqs"])]


def _blocks(n):
    return (n + BLOCK - 1) // BLOCK


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _frequencies(rot, scaling, base=10000.0, factor=8.0, trained=4096):
    """Turns per position of each rotated pair (64 bits), and what cosine and sine are multiplied by."""
    i = np.arange(rot // 2, dtype=np.float64)
    if scaling == "ntk":
        base = base * factor ** (rot / (rot - 2))
    f = base ** (-2.0 * i / rot) / (2.0 * math.pi)
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "yarn":
        def pair(turns):
            return rot * math.log(trained / (turns * 2.0 * math.pi)) / (2.0 * math.log(base))
        lo, hi = max(math.floor(pair(32.0)), 0), min(math.ceil(pair(1.0)), rot - 1)
        keep = 1.0 - np.clip((i - lo) / max(hi - lo, 0.001), 0.0, 1.0)
        return f / factor * (1.0 - keep) + f * keep, 0.1 * math.log(factor) + 1.0
    return f, 1.0


def _cache(case, g, dev, blocks):
    """Pages of a used cache: codes as quantised keys and values have them, scales that vary from block to
    block, pages in no order."""
    n_pages, d = case["seqs"] * case["kv_heads"] * blocks, case["head_dim"]
    pages = torch.empty((n_pages, 2, BLOCK * d), dtype=torch.uint8, device=dev)
    for part in pages.split(16384):
        part.copy_((torch.randn(part.shape, generator=g, device=dev) * 32).round_().clamp_(-127, 127).add_(128))
    scales = torch.exp(torch.randn((n_pages, 2), generator=g, device=dev) * 0.3) / 32
    table = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32)
    return dict(pages=pages, scales=scales, table=table.view(case["seqs"], case["kv_heads"], blocks))


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    st = dict(case=case)
    if case["op"] == "evict":
        st["lens"] = torch.tensor(_lens(case), dtype=torch.int32, device=dev)
        shape = (case["seqs"], case["kv_heads"], case["blocks"] + 3)
        n = shape[0] * shape[1] * shape[2]
        st["table"] = torch.randperm(n, generator=g, device=dev).to(torch.int32).view(shape)
        # weights have a heavy tail, and blocks that nothing ever looked at tie at zero
        w = torch.exp(torch.randn(shape, generator=g, device=dev) * 2.0)
        st["score"] = torch.where(torch.rand(shape, generator=g, device=dev) < 0.05, torch.zeros_like(w), w)
        if own:
            import activation_sparse_rank_amd as pi
            st["out"] = (torch.empty_like(st["table"]), torch.empty_like(st["score"]), torch.empty_like(st["lens"]))
            st["evict"] = pi.kv_evict
        return st
    dt, d, hk = DTYPES[case["dtype"]], case["head_dim"], case["kv_heads"]
    if case["op"] == "rope":
        h, n = case["heads"], case["tokens"]
        # rows of a fused projection: queries, keys, values side by side
        qkv = torch.randn((n, (h + 2 * hk) * d), generator=g, device=dev).to(dt)
        st["q"] = qkv[:, :h * d].unflatten(1, (h, d))
        st["k"] = qkv[:, h * d:(h + hk) * d].unflatten(1, (hk, d))
        st["pos"] = torch.arange(case["first"], case["first"] + n, dtype=torch.int32, device=dev)
        f, st["mul"] = _frequencies(case["rot"], case["scaling"])
        st["freqs"] = torch.from_numpy(f).to(dev)
        st["wq"] = 1 + 0.1 * torch.randn(d, generator=g, device=dev) if case["norm"] else None
        st["wk"] = 1 + 0.1 * torch.randn(d, generator=g, device=dev) if case["norm"] else None
        if own:
            import activation_sparse_rank_amd as pi
            st["rope"] = pi.Rope(st["freqs"], d, layout=case["layout"], scale=st["mul"], q_norm=st["wq"],
                                 k_norm=st["wk"], eps=1e-6)
            st["out"] = tuple(torch.empty(t.shape, dtype=dt, device=dev) for t in (st["q"], st["k"]))
            st["qk_rope"] = pi.qk_rope
        return st
    lens = _lens(case)
    n = case["seqs"] * case["new"]
    blocks = _blocks(max(lens)) + 1
    st["lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    st.update(_cache(case, g, dev, blocks))
    st["start"] = torch.arange(case["seqs"] + 1, dtype=torch.int32, device=dev) * case["new"]
    if case["op"] == "append":
        st["open"] = torch.randn((case["seqs"], hk, 2, BLOCK, d), generator=g, device=dev).to(dt)
        kv = torch.randn((n, 2 * hk * d), generator=g, device=dev).to(dt)
        st["k"], st["v"] = (kv[:, i * hk * d:(i + 1) * hk * d].unflatten(1, (hk, d)) for i in (0, 1))
        if own:
            import activation_sparse_rank_amd as pi
            st["cache"] = pi.KVCache(st["pages"], st["scales"], st["open"], st["table"])
            st["out"] = tuple(torch.empty((n, hk, d), dtype=dt, device=dev) for _ in range(2))
            st["kv_append"], st["kv_read"] = pi.kv_append, pi.kv_read
        return st
    h = case["heads"]
    st["q"] = (torch.randn((n, h, d), generator=g, device=dev) * 2.0).to(dt)
    st["score"] = torch.rand((case["seqs"], hk, blocks), generator=g, device=dev) if case["score"] else None
    if own:
        import activation_sparse_rank_amd as pi
        st["open"] = torch.zeros((case["seqs"], hk, 2, BLOCK, d), dtype=dt, device=dev)
        st["cache"] = pi.KVCache(st["pages"], st["scales"], st["open"], st["table"], st["score"])
        st["out"] = torch.empty((n, h, d), dtype=dt, device=dev)
        # the length bound that a scheduler knows, and a workspace for it, kept from call to call
        st["max_len"] = max(lens)
        st["ws"] = pi.alloc_attend_workspace(st["cache"], h, case["new"], max_len=st["max_len"],
                                             add_score=case["score"])
        st["attend"] = pi.attend
    return st


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(st):
    case = st["case"]
    if case["op"] == "rope":
        return _rope_own(st) if own else _rope_plain(st)
    if case["op"] == "append":
        return _append_own(st) if own else _append_plain(st)
    if case["op"] == "attend":
        return _attend_own(st) if own else _attend_plain(st)
    return _evict_own(st) if own else _evict_plain(st)


def _rope_own(st):
    q, k = st["out"]
    st["qk_rope"](st["rope"], st["q"], st["k"], st["pos"], q_out=q, k_out=k)
    return {"q": q, "k": k}


def _append_own(st):
    k, v = st["out"]
    new = st["case"]["new"]
    st["kv_append"](st["cache"], st["k"], st["v"], st["lens"], q_start=st["start"], max_new=new)
    st["kv_read"](st["cache"], st["lens"], k, v, q_start=st["start"], max_new=new)
    return {"k": k, "v": v, "open": st["open"]}


def _attend_own(st):
    case = st["case"]
    st["attend"](st["cache"], st["q"], st["lens"], st["out"], q_start=st["start"], max_q=case["new"],
                 max_len=st["max_len"], add_score=case["score"], ws=st["ws"])
    return {"out": st["out"], "score": st["score"]}


def _evict_own(st):
    table, score, lens = st["out"]
    case = st["case"]
    st["evict"](st["table"], st["score"], st["lens"], case["keep"], case["recent"], lens, table_out=table,
                score_out=score)
    return {"table": table, "score": score, "lens": lens}


def _rotate(x, w, cos, sin, case):
    """RMS norm over the head where a weight is given, then the rotation of its first `rot` elements."""
    rot = case["rot"]
    y = x.float()
    if w is not None:
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6) * w
    r, rest = y[..., :rot], y[..., rot:]
    if case["layout"] == "half":
        a, b = r[..., :rot // 2], r[..., rot // 2:]
        r = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    else:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    return torch.cat((r, rest), -1).to(x.dtype)


def _rope_plain(st):
    # angles in 64 bits: far positions times the fastest frequency leave no fraction in 32
    angle = (st["pos"].double()[:, None] * st["freqs"]).frac() * (2.0 * math.pi)
    cos, sin = (st["mul"] * angle.cos()).float()[:, None], (st["mul"] * angle.sin()).float()[:, None]
    return {"q": _rotate(st["q"], st["wq"], cos, sin, st["case"]),
            "k": _rotate(st["k"], st["wk"], cos, sin, st["case"])}


def _to_pages(keys, values):
    """Codes [..., 32, D] of a block's keys and values in the page's byte order: [..., 2, 32 * D]."""
    d, lead = keys.shape[-1], keys.shape[:-2]
    n = len(lead)
    k = keys.reshape(*lead, 2, 16, d // 64, 4, 16).permute(*range(n), n, n + 2, n + 3, n + 1, n + 4)
    v = values.reshape(*lead, 2, 4, 4, d // 32, 2, 16).permute(*range(n), n + 3, n + 1, n + 5, n + 4, n, n + 2)
    return torch.stack((k.reshape(*lead, BLOCK * d), v.reshape(*lead, BLOCK * d)), -2)


def _from_pages(pages, d):
    """The inverse of _to_pages: codes of keys and values, each [..., 32, D]."""
    lead = pages.shape[:-2]
    n = len(lead)
    k = pages[..., 0, :].reshape(*lead, 2, d // 64, 4, 16, 16).permute(*range(n), n, n + 3, n + 1, n + 2, n + 4)
    v = pages[..., 1, :].reshape(*lead, d // 32, 4, 16, 2, 2, 4).permute(
        *range(n), n + 4, n + 1, n + 5, n, n + 3, n + 2)
    return k.reshape(*lead, BLOCK, d), v.reshape(*lead, BLOCK, d)


def _append_plain(st):
    case, dt = st["case"], DTYPES[st["case"]["dtype"]]
    new, seqs, hk, d = case["new"], case["seqs"], case["kv_heads"], case["head_dim"]
    dev = st["lens"].device
    before = st["lens"].long() - new
    first = before // BLOCK                                   # the first block that this call touches
    count = (new + 2 * BLOCK - 2) // BLOCK                    # the most blocks it can touch
    offset = before % BLOCK
    # raw rows of the touched blocks [seqs, hk, 2, count * 32, d]: what was open, then the new rows
    raw = torch.zeros((seqs, hk, 2, count * BLOCK, d), dtype=dt, device=dev)
    slot = torch.arange(BLOCK, device=dev)
    raw[:, :, :, :BLOCK] = torch.where((slot < offset[:, None])[:, None, None, :, None], st["open"], 0)
    at = (offset[:, None] + torch.arange(new, device=dev))[:, None, None, :, None].expand(seqs, hk, 2, new, d)
    rows = torch.stack((st["k"], st["v"])).view(2, seqs, new, hk, d).permute(1, 3, 0, 2, 4)
    raw.scatter_(3, at, rows)
    blocks = raw.view(seqs, hk, 2, count, BLOCK, d).transpose(2, 3)
    amax = blocks.abs().amax((-2, -1)).double()
    scale = (amax / 127).float()
    # in 64 bits: values next to the middle of two codes go the way that the definition says
    codes = (127 * blocks.double() / torch.where(amax > 0, amax, 1.0)[..., None, None]).round().to(torch.int16) + 128
    last = (st["lens"].long() + BLOCK - 1) // BLOCK
    block = first[:, None] + torch.arange(count, device=dev)                         # [seqs, count]
    touched = (block < last[:, None])[:, None].expand(seqs, hk, count)
    at = block.clamp(max=st["table"].shape[2] - 1)[:, None].expand(seqs, hk, count)
    page = st["table"].long().gather(2, at)
    st["pages"][page[touched]] = _to_pages(codes[:, :, :, 0], codes[:, :, :, 1])[touched].to(torch.uint8)
    st["scales"][page[touched]] = scale[touched]
    # the rows of the block that stays open: its first `filled` slots
    filled = st["lens"].long() % BLOCK
    base = (st["lens"].long() // BLOCK - first) * BLOCK
    at = (base[:, None] + slot).clamp(max=count * BLOCK - 1)[:, None, None, :, None].expand(seqs, hk, 2, BLOCK, d)
    keep = (slot < filled[:, None])[:, None, None, :, None]
    st["open"].copy_(torch.where(keep, raw.gather(3, at), st["open"]))
    # read back the new tokens' values
    k, v = _from_pages(st["pages"][page], d)                                        # [seqs, hk, count, 32, d]
    kv = torch.stack((k, v), 2).float() - 128
    kv = kv * st["scales"][page].transpose(2, 3)[..., None, None]
    at = (offset[:, None] + torch.arange(new, device=dev))[:, None, None, :, None].expand(seqs, hk, 2, new, d)
    kv = kv.reshape(seqs, hk, 2, count * BLOCK, d).gather(3, at).permute(2, 0, 3, 1, 4).reshape(2, seqs * new, hk, d)
    return {"k": kv[0].to(dt), "v": kv[1].to(dt), "open": st["open"]}


def _attend_plain(st):
    case, dt = st["case"], DTYPES[st["case"]["dtype"]]
    new, seqs, hk, d = case["new"], case["seqs"], case["kv_heads"], case["head_dim"]
    group = case["heads"] // hk
    table = st["table"].long()
    nb = table.shape[2]
    k, v = _from_pages(st["pages"][table], d)                                       # [seqs, hk, nb, 32, d]
    scales = st["scales"][table][..., None, None]
    k = ((k.float() - 128) * scales[..., 0, :, :]).view(seqs, hk, nb * BLOCK, d)
    v = ((v.float() - 128) * scales[..., 1, :, :]).view(seqs, hk, nb * BLOCK, d)
    q = st["q"].float().view(seqs, new, hk, group, d).permute(0, 2, 1, 3, 4).reshape(seqs, hk, new * group, d)
    s = (q @ k.transpose(2, 3).contiguous()) / math.sqrt(d)
    token = torch.arange(nb * BLOCK, device=q.device)
    sees = st["lens"].long()[:, None] - new + 1 + torch.arange(new, device=q.device)           # [seqs, new]
    hidden = token >= sees.repeat_interleave(group, 1)[..., None]                              # [seqs, rows, tokens]
    s.masked_fill_(hidden[:, None], float("-inf"))
    p = torch.exp(s - s.amax(-1, keepdim=True))
    p /= p.sum(-1, keepdim=True)
    out = (p @ v).view(seqs, hk, new, group, d).permute(0, 2, 1, 3, 4).reshape(seqs * new, hk * group, d)
    if case["score"]:
        st["score"] += p.sum(2).view(seqs, hk, nb, BLOCK).sum(-1)
    return {"out": out.to(dt), "score": st["score"]}


def _evict_plain(st):
    case, table, score, lens = st["case"], st["table"], st["score"], st["lens"].long()
    keep, recent, n = case["keep"], case["recent"], table.shape[2]
    nb = ((lens + BLOCK - 1) // BLOCK)[:, None, None]
    slot = torch.arange(n, device=table.device)
    over = nb > keep
    older = (slot < nb - recent).expand_as(table)
    # older blocks by weight, the largest first, ties by the lower slot
    order = torch.where(older, score, float("-inf")).sort(dim=-1, descending=True, stable=True).indices
    rank = torch.empty_like(order).scatter_(-1, order, slot.expand_as(order))
    out = older & (rank >= keep - recent) & over
    gone = (nb - keep).clamp(min=0)
    # kept blocks and recent ones in order, then those that leave, then the slots past the end
    to = torch.where(out, nb - gone + out.cumsum(-1) - 1, torch.where(slot < nb, slot - out.cumsum(-1), slot))
    left = torch.where((slot < nb) & out, torch.zeros_like(score), score)
    return {"table": torch.empty_like(table).scatter_(-1, to, table),
            "score": torch.empty_like(score).scatter_(-1, to, left),
            "lens": (lens - BLOCK * gone[:, 0, 0]).to(torch.int32)}


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    if case["op"] == "evict":
        n = case["seqs"] * case["kv_heads"] * (case["blocks"] + 3)
        return {"bytes": 16 * n + 8 * case["seqs"], "flops": 0}
    size, d, hk = {"f16": 2, "f32": 4}[case["dtype"]], case["head_dim"], case["kv_heads"]
    if case["op"] == "rope":
        n = case["tokens"] * (case["heads"] + hk) * d
        return {"bytes": 2 * n * size + 4 * case["tokens"] + 4 * case["rot"],
                "flops": 3 * case["tokens"] * (case["heads"] + hk) * case["rot"] + (4 * n if case["norm"] else 0)}
    lens = _lens(case)
    if case["op"] == "append":
        new = case["seqs"] * case["new"]
        held = sum((n - case["new"]) % BLOCK for n in lens)       # rows of the open blocks, read again
        left = sum(min(n % BLOCK, case["new"]) for n in lens)     # new rows that stay open
        row = 2 * hk * d
        codes = sum(n - (n - case["new"]) // BLOCK * BLOCK for n in lens)
        return {"bytes": row * ((new + held + left + new) * size + codes + new), "flops": 4 * row * codes}
    group, new = case["heads"] // hk, case["new"]
    pairs = sum(sum(n - new + 1 + t for t in range(new)) for n in lens)
    pages = sum(lens) * hk * 2 * d + sum(_blocks(n) for n in lens) * hk * 12
    return {"bytes": pages + 2 * case["seqs"] * new * case["heads"] * d * size
            + (8 * sum(_blocks(n) for n in lens) * hk if case["score"] else 0),
            "flops": 4 * pairs * group * hk * d}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "rope":
        return _rope_exact(st)
    if case["op"] == "append":
        return _append_exact(st)
    if case["op"] == "attend":
        return _attend_exact(st)
    return _evict_exact(st)


def _rope_exact(st):
    """Pairs as complex numbers, turned by exp(2 pi i f p)."""
    case = st["case"]
    half = case["rot"] // 2
    pairs = torch.arange(half, device=st["pos"].device)
    a, b = (pairs, pairs + half) if case["layout"] == "half" else (2 * pairs, 2 * pairs + 1)
    turns = torch.outer(st["pos"].double(), st["freqs"])
    turn = torch.polar(torch.full_like(turns, st["mul"]), 2.0 * math.pi * (turns - turns.floor()))
    res = {}
    for name, w in (("q", st["wq"]), ("k", st["wk"])):
        x = st[name].double()
        if w is not None:
            x = x / (x.pow(2).sum(-1, keepdim=True) / case["head_dim"] + 1e-6).sqrt() * w.double()
        z = torch.complex(x[..., a], x[..., b]) * turn[:, None]
        y = x.clone()
        y[..., a], y[..., b] = z.real, z.imag
        res[name] = y
    return res


def _append_exact(st):
    """Block after block from the rows themselves; nothing is stored in between."""
    case = st["case"]
    new, hk, d = case["new"], case["kv_heads"], case["head_dim"]
    parts, opens = {"k": [], "v": []}, st["open"].double()
    for s, n in enumerate(_lens(case)):
        before = n - new
        old = before % BLOCK
        for i, name in enumerate(("k", "v")):
            rows = torch.cat((st["open"][s, :, i, :old].double(),
                              st[name][s * new:(s + 1) * new].double().transpose(0, 1)), 1)    # [hk, old + new, d]
            vals = []
            for b in rows.split(BLOCK, 1):
                m = b.abs().flatten(1).amax(1)[:, None, None]
                vals.append(torch.where(m > 0, torch.round(b * 127 / m) * m / 127, 0.0))
            parts[name].append(torch.cat(vals, 1)[:, old:].transpose(0, 1))
            if n % BLOCK:
                opens[s, :, i, :n % BLOCK] = rows[:, -(-rows.shape[1] // BLOCK) * BLOCK - BLOCK:]
    return {"k": torch.cat(parts["k"]), "v": torch.cat(parts["v"]), "open": opens}


def _attend_exact(st):
    """A kv head of a sequence at a time, its codes picked out of the pages by their places."""
    case = st["case"]
    new, hk, d = case["new"], case["kv_heads"], case["head_dim"]
    group, dev = case["heads"] // hk, st["q"].device
    t, e = torch.arange(BLOCK, device=dev)[:, None], torch.arange(d, device=dev)
    k_at = ((t // 16 * (d // 64) + e // 64) * 4 + e // 16 % 4) * 256 + t % 16 * 16 + e % 16
    v_at = (e // 32 * 4 + t % 16 // 4) * 256 + e % 16 * 16 + e // 16 % 2 * 8 + t // 16 * 4 + t % 4
    out = torch.zeros((case["seqs"] * new, case["heads"], d), dtype=torch.float64, device=dev)
    score = st["score"].double() if case["score"] else None
    for s, n in enumerate(_lens(case)):
        nb = _blocks(n)
        limit = n - new + 1 + torch.arange(new, device=dev).repeat_interleave(group)
        for h in range(hk):
            page = st["table"][s, h, :nb].long()
            k = (st["pages"][page, 0][:, k_at].double() - 128) * st["scales"][page, 0].double()[:, None, None]
            v = (st["pages"][page, 1][:, v_at].double() - 128) * st["scales"][page, 1].double()[:, None, None]
            k, v = k.flatten(0, 1), v.flatten(0, 1)
            q = st["q"][s * new:(s + 1) * new, h * group:(h + 1) * group].double().flatten(0, 1)
            logit = torch.mm(q, k.t().contiguous()) * d ** -0.5
            logit[torch.arange(nb * BLOCK, device=dev) >= limit[:, None]] = float("-inf")
            p = torch.softmax(logit, -1)
            out[s * new:(s + 1) * new, h * group:(h + 1) * group] = torch.mm(p, v).view(new, group, d)
            if score is not None:
                score[s, h, :nb] += p.sum(0).view(nb, BLOCK).sum(1)
    return {"out": out, "score": score}


def _evict_exact(st):
    """A row of the table at a time, as lists."""
    case = st["case"]
    score, table = st["score"].double().cpu().numpy(), st["table"].cpu().numpy()
    lens, moved, pages = _lens(case), score.copy(), table.copy()
    for s, n in enumerate(_lens(case)):
        nb = _blocks(n)
        if nb <= case["keep"]:
            continue
        lens[s] = n - BLOCK * (nb - case["keep"])
        for h in range(case["kv_heads"]):
            older = sorted(range(nb - case["recent"]), key=lambda b: (-score[s, h, b], b))
            stay = sorted(older[:case["keep"] - case["recent"]]) + list(range(nb - case["recent"], nb))
            leave = sorted(older[case["keep"] - case["recent"]:])
            moved[s, h, :nb] = np.concatenate((score[s, h, stay], np.zeros(len(leave))))
            pages[s, h, :nb] = table[s, h, stay + leave]
    return {"table": torch.from_numpy(pages), "score": torch.from_numpy(moved),
            "lens": torch.tensor(lens, dtype=torch.int32)}
