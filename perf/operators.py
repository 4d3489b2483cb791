"""The attention half of a decoder layer around the INT8 linears: what is measured of it.

Four operators, as a serving program calls them one after another:

  norm_rope   queries and keys normalised per head and rotated by their position
  append      the same for the queries of a step, whose keys and values go to a paged INT8 cache
  read        tokens of that cache back as BF16 keys and values
  attn        attention of a step's queries over the cache: single tokens, short runs, whole prompts

The cache holds INT8 codes [pages, kv_heads, page, dim] and one FP32 scale for every 16 tokens of a page and
head.  Sequence b's tokens lie in the pages page_table[b] names; kv_len[b] counts them with this step's, which are
the last cu[b + 1] - cu[b] of them.  Here are the operators in plain torch (``own`` false) and through the
library (``own`` true), and their definition in 64 bits (``exact``).
"""
import math
import random

import torch

own = False

BLOCK = 16                 # cached tokens that share a scale
EPS = 1e-6
SHIFT_MOST = 2.0 ** 24     # beyond this growth nothing of a block's old codes is left


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the 12-token conditioning prompt of the benchmark's encoder: 64 query and 8 key heads of 128
        dict(name="norm_rope 12 tokens", op="norm_rope", tokens=12, q_heads=64, kv_heads=8, dim=128, rot=128, axes=1,
             pairs="half", norm=True),
        # a video model's joint sequence (5376 = 42 heads of 128), three position axes (time, height, width)
        dict(name="norm_rope 8191 x 42", op="norm_rope", tokens=8191, q_heads=42, kv_heads=42, dim=128, rot=128, axes=3,
             pairs="half", norm=True),
        # one decode step of a full serving batch
        dict(name="append 64 x 1", op="append", seqs=64, new=1, ctx=4100, q_heads=64, kv_heads=8, dim=128, page=64,
             rot=128, pairs="half", norm=True),
        # prompts of several users in one prefill step, some of them continued in the middle of a block
        dict(name="append 5 x 1700", op="append", seqs=5, new=1700, ctx=300, q_heads=64, kv_heads=8, dim=128, page=64,
             rot=128, pairs="half", norm=True),
        # the start of a conversation read back, an odd length
        dict(name="read 1 x 33", op="read", seqs=1, ctx=33, kv_heads=8, dim=128, page=16),
        # a batch's whole prefixes gathered for a consumer of BF16 keys and values
        dict(name="read 8 x 4096", op="read", seqs=8, ctx=4096, kv_heads=8, dim=128, page=64),
        # a single user's next token after a short prompt: latency
        dict(name="decode 1 x 577", op="attn", seqs=1, new=1, ctx=577, q_heads=64, kv_heads=8, dim=128, page=16,
             causal=True),
        # a full serving batch with contexts of many lengths
        dict(name="decode 64 x 8192", op="attn", seqs=64, new=1, ctx=8192, q_heads=64, kv_heads=8, dim=128, page=64,
             causal=True),
        # few users with very long contexts
        dict(name="decode 3 x 131071", op="attn", seqs=3, new=1, ctx=131071, q_heads=64, kv_heads=8, dim=128, page=128,
             causal=True),
        # the 12-token conditioning prompt again, now its attention
        dict(name="prompt 12", op="attn", seqs=1, new=12, ctx=12, q_heads=64, kv_heads=8, dim=128, page=64, causal=True),
        # chunks of prompts appended to longer contexts, one key head for each of 40 query heads of 64
        dict(name="chunks 3 x 517", op="attn", seqs=3, new=517, ctx=3001, q_heads=40, kv_heads=40, dim=64, page=32,
             causal=True),
        # one long prompt
        dict(name="prompt 8192", op="attn", seqs=1, new=8192, ctx=8192, q_heads=64, kv_heads=8, dim=128, page=64,
             causal=True),
    ]


def _spread(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    dim = rng.choice([64, 128, 128])
    kv_heads = rng.choice([1, 2, 4, 5, 8, 8])
    q_heads = kv_heads * rng.choice([1, 2, 4, 5, 7, 8, 8])
    page = rng.choice([16, 32, 64, 128, 256])
    op = rng.choice(["norm_rope", "append", "append", "read", "decode", "decode", "prompt", "prompt"])
    pairs, norm = rng.choice(["half", "half", "adjacent"]), rng.random() < 0.75
    rot = rng.choice([dim, dim, dim // 2])
    if op == "norm_rope":
        return dict(op=op, tokens=_spread(rng, 1, 8191), q_heads=q_heads, kv_heads=kv_heads, dim=dim, rot=rot,
                    axes=rng.choice([1, 1, 2, 3]), pairs=pairs, norm=norm)
    if op == "append":
        seqs = _spread(rng, 1, 96)
        new = 1 if rng.random() < 0.4 else _spread(rng, 1, max(1, 6000 // seqs))
        return dict(op=op, seqs=seqs, new=new, ctx=_spread(rng, 1, 4100), q_heads=q_heads, kv_heads=kv_heads, dim=dim,
                    page=page, rot=rot, pairs=pairs, norm=norm)
    if op == "read":
        seqs = _spread(rng, 1, 32)
        return dict(op=op, seqs=seqs, ctx=_spread(rng, 1, 32768 // seqs), kv_heads=kv_heads, dim=dim, page=page)
    if op == "decode":
        seqs = _spread(rng, 1, 96)
        ctx = _spread(rng, 1, min(131071, 400000 // seqs))
        new = rng.choice([1, 1, 1, 1, 2, 3, 5])
        return dict(op="attn", seqs=seqs, new=new, ctx=max(ctx, new), q_heads=q_heads, kv_heads=kv_heads, dim=dim,
                    page=page, causal=True)
    seqs = _spread(rng, 1, 8)
    new = _spread(rng, 6, 4096 // seqs)
    ctx = max(new, _spread(rng, new, min(8192, 16_000_000 // (new * seqs))))
    return dict(op="attn", seqs=seqs, new=new, ctx=ctx, q_heads=q_heads, kv_heads=kv_heads, dim=dim, page=page,
                causal=rng.random() < 0.75)


def _lengths(count, most, least=1):
    """Lengths of `count` sequences, the longest of them `most`: the same for every seed."""
    r = random.Random(1000003 * most + count)
    return [most] + [r.randint(min(most, max(least, most // 4)), most) for _ in range(count - 1)]


def _steps(case):
    """(new tokens, cached tokens with the new ones) of every sequence."""
    n = _lengths(case["seqs"], case["new"])
    if case["op"] == "append":
        old = _lengths(case["seqs"], case["ctx"], 0)
        return n, [a + b for a, b in zip(n, old)]
    return n, [max(a, b) for a, b in zip(n, _lengths(case["seqs"], case["ctx"]))]


def work(case):
    """Every input read once, every output written once."""
    op, dim, hk = case["op"], case["dim"], case["kv_heads"]
    token = 2 * hk * (dim + 4 / BLOCK)                       # a cached token: codes and its share of the scales
    if op == "norm_rope":
        rows = case["tokens"] * (case["q_heads"] + hk)
        return {"bytes": 4 * rows * dim + case["tokens"] * (4 * case["rot"] + 4 * case["axes"]), "flops": 7 * rows * dim}
    if op == "read":
        n = sum(_lengths(case["seqs"], case["ctx"]))
        return {"bytes": n * (token + 4 * hk * dim), "flops": 2 * n * hk * dim}
    hq = case["q_heads"]
    n, kv = _steps(case)
    if op == "append":
        opened = sum(min(BLOCK, b - (b - a) // BLOCK * BLOCK) for a, b in zip(n, kv))   # old tokens beside new ones
        t = sum(n)
        back = t + sum((b - a) % BLOCK for a, b in zip(n, kv))
        return {"bytes": t * (4 * hq * dim + 4 * hk * dim + token + 4 * case["rot"]) + opened * token + back * 4 * hk * dim,
                "flops": t * dim * (7 * hq + 9 * hk)}
    seen = sum(a * b - (a * (a - 1) // 2 if case["causal"] else 0) for a, b in zip(n, kv))
    return {"bytes": sum(kv) * token + sum(n) * hq * (4 * dim + 4), "flops": 4 * dim * hq * seen}


# ------------------------------------------------------------------ inputs
def _rope_table(positions, rot, device):
    angle = torch.arange(positions, device=device, dtype=torch.float64)[:, None] * \
        (1e6 ** (-torch.arange(0, rot, 2, device=device, dtype=torch.float64) / rot))
    return torch.stack([angle.cos(), angle.sin()], -1).float()


def _ints(v, device):
    return torch.tensor(v, dtype=torch.int32, device=device)


def _cumulated(n):
    return [sum(n[:i]) for i in range(len(n) + 1)]


def _projections(s, case, tokens, g, device):
    """A step's queries, keys and values as the layer's projections leave them, in one buffer; some channels of
    the keys are large, as trained models have them."""
    hq, hk, dim = case["q_heads"], case["kv_heads"], case["dim"]
    qkv = torch.randn(tokens, hq + 2 * hk, dim, generator=g, device=device)
    qkv[:, hq:hq + hk, 3::29] *= 8
    qkv = qkv.bfloat16()
    s.update(q=qkv[:, :hq], k=qkv[:, hq:hq + hk], v=qkv[:, hq + hk:], qw=None, kw=None)
    if case["norm"]:
        s["qw"], s["kw"] = (1 + 0.2 * torch.randn(2, dim, generator=g, device=device)).bfloat16()


def _paged(s, case, kv, g, device):
    """A cache with the sequences' tokens in pages in no order, and random contents."""
    hk, dim, page = case["kv_heads"], case["dim"], case["page"]
    need = [-(-x // page) for x in kv]
    pages, wide = sum(need) + 2, max(need)
    order = torch.randperm(pages, generator=g, device=device).int()
    at = _ints(_cumulated(need)[:-1], device)[:, None] + torch.arange(wide, device=device, dtype=torch.int32)
    s["table"] = order[at.clamp(max=pages - 1).long()].contiguous()
    for name in ("k", "v"):
        codes = torch.randn(pages, hk, page, dim, generator=g, device=device).mul_(36).round_().clamp_(-127, 127)
        s["c" + name] = codes.to(torch.int8)
        s["s" + name] = (0.5 + 1.5 * torch.rand(pages, hk, page // BLOCK, generator=g, device=device)) / 36
    s.update(kv_len=_ints(kv, device), page=page)


def prepare(case, seed):
    device = "cuda"
    g = torch.Generator(device).manual_seed(seed)
    op, dim = case["op"], case["dim"]
    s = {"op": op}
    if op == "norm_rope":
        t, axes = case["tokens"], case["axes"]
        _projections(s, case, t, g, device)
        s["table_cs"] = _rope_table(max(t, 64), case["rot"], device)
        s["adjacent"] = case["pairs"] == "adjacent"
        s["positions"] = torch.randint(0, max(t, 64), (axes, t), generator=g, device=device, dtype=torch.int32)
        s["axis"] = (torch.arange(case["rot"] // 2, device=device) % axes).to(torch.uint8) if axes > 1 else None
        s["q_out"], s["k_out"] = (torch.empty(t, x.shape[1], dim, dtype=torch.bfloat16, device=device) for x in (s["q"], s["k"]))
    elif op == "read":
        kv = _lengths(case["seqs"], case["ctx"])
        _paged(s, case, kv, g, device)
        s["cu"], s["total"] = _ints(_cumulated(kv), device), sum(kv)
    else:
        n, kv = _steps(case)
        _paged(s, case, kv, g, device)
        s.update(cu=None if max(n) == 1 else _ints(_cumulated(n), device), total=sum(n), new_most=max(n), hq=case["q_heads"])
        if op == "append":
            _projections(s, case, sum(n), g, device)
            s["table_cs"], s["adjacent"] = _rope_table(max(kv), case["rot"], device), case["pairs"] == "adjacent"
            s["q_out"] = torch.empty(sum(n), case["q_heads"], dim, dtype=torch.bfloat16, device=device)
            back = [a + (b - a) % BLOCK for a, b in zip(n, kv)]          # from the first touched block's start
            s["back_cu"], s["back"] = _ints(_cumulated(back), device), sum(back)
        else:
            s["q"] = (1.5 * torch.randn(sum(n), case["q_heads"], dim, generator=g, device=device)).bfloat16()
            s.update(causal=case["causal"], scale=dim ** -0.5, out=torch.empty_like(s["q"]),
                     lse=torch.empty(sum(n), case["q_heads"], device=device))
    if op in ("read", "append"):
        rows = s["total"] if op == "read" else s["back"]
        s["k_back"], s["v_back"] = (torch.empty(rows, case["kv_heads"], dim, dtype=torch.bfloat16, device=device) for _ in "kv")
    if own:
        s["calls"] = _calls(s)
    return s


# ------------------------------------------------------------------ the library's calls
def _calls(s):
    """The prepared calls that a serving program keeps for a step of these tensors."""
    import rotated_int8_quantized_b200 as cr

    op = s["op"]
    rope = cr.Rope(s["table_cs"], adjacent=s["adjacent"], axis=s.get("axis")) if "table_cs" in s else None
    if op == "norm_rope":
        return [cr.QKNormRope(s["q"], s["k"], s["q_out"], s["k_out"], q_weight=s["qw"], k_weight=s["kw"], eps=EPS, rope=rope,
                              positions=s["positions"])]
    cache = cr.KV8Cache(s["ck"], s["cv"], s["sk"], s["sv"])
    if op == "attn":
        return [cr.AttnKV8(s["q"], cache, s["table"], s["kv_len"], s["out"], cu=s["cu"], lse=s["lse"], scale=s["scale"],
                           causal=s["causal"])]
    if op == "read":
        return [cr.KV8Read(cache, s["table"], s["kv_len"], s["k_back"], s["v_back"], cu=s["cu"])]
    return [cr.KV8Append(s["q"], s["k"], s["v"], cache, s["table"], s["kv_len"], s["q_out"], cu=s["cu"], q_weight=s["qw"],
                         k_weight=s["kw"], eps=EPS, rope=rope),
            cr.KV8Read(cache, s["table"], s["kv_len"], s["k_back"], s["v_back"], cu=s["back_cu"])]


# ------------------------------------------------------------------ the plain form
def _norm_rotate(x, weight, table, positions, axis, adjacent):
    """x [t, heads, dim] normalised per head, the first table.shape[1] pairs of dims rotated; FP32."""
    y = x.float()
    if weight is not None:
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS) * weight.float()
    half = table.shape[1]
    if axis is None:
        cs = table[positions[0].long()]
    else:
        cs = table[positions[axis.long()].T.long(), torch.arange(half, device=x.device)]
    c, s = cs[:, None, :, 0], cs[:, None, :, 1]
    head, rest = y[..., :2 * half], y[..., 2 * half:]
    a, b = (head[..., 0::2], head[..., 1::2]) if adjacent else (head[..., :half], head[..., half:])
    u, v = a * c - b * s, b * c + a * s
    turned = torch.stack([u, v], -1).flatten(-2) if adjacent else torch.cat([u, v], -1)
    return torch.cat([turned, rest], -1)


def _places(s, cu, total):
    """Sequence, position, page and row within the page of a step's tokens."""
    kv = s["kv_len"].long()
    if cu is None:
        cu = torch.arange(kv.numel() + 1, device=kv.device)
    cu, t = cu.long(), torch.arange(total, device=kv.device)
    b = torch.searchsorted(cu, t, right=True) - 1
    at = kv[b] - cu[b + 1] + t
    return b, at, s["table"][b, at // s["page"]].long(), at % s["page"]


def _store(codes, scales, x, first, b, page, row, table, size):
    """x [t, heads, dim] FP32 into the cache: `first` [seqs] is the position of each sequence's first new token."""
    heads = x.shape[1]
    blocks = scales.shape[2]
    flat = scales.permute(0, 2, 1).reshape(-1, heads)                       # [pages * blocks, heads]
    block = page * blocks + row // BLOCK
    most = torch.zeros_like(flat).index_reduce_(0, block, x.abs().amax(-1), "amax")
    # blocks that hold older tokens keep their scale unless the new ones outgrow it, and then it doubles
    open_page = table[torch.arange(first.numel(), device=first.device), first // size].long()
    open_block = open_page * blocks + first % size // BLOCK
    kept = torch.zeros(flat.shape[0], dtype=torch.bool, device=x.device)
    kept[open_block] = first % BLOCK != 0
    ratio = most / (127.5 * flat)
    grown = torch.ldexp(flat, torch.where(ratio >= 1, torch.frexp(ratio)[1], 0))
    fits = kept[:, None] & (flat > 0) & (ratio < SHIFT_MOST)
    touched = torch.zeros_like(kept)
    touched[block] = True
    fresh = torch.where(kept[:, None] & (most == 0), flat, most / 127)
    new = torch.where(touched[:, None], torch.where(fits, grown, fresh), flat)
    # the older codes of those blocks on the new scale
    rows = (first % size // BLOCK * BLOCK)[:, None] + torch.arange(BLOCK, device=x.device)
    old = codes[open_page[:, None], :, rows].float()                        # [seqs, 16, heads, dim]
    shrink = torch.where(fits, flat / new, 0)[open_block][:, None, :, None]
    older = (torch.arange(BLOCK, device=x.device) < first[:, None] % BLOCK)[..., None, None]
    codes[open_page[:, None], :, rows] = torch.where(older & (new > 0)[open_block][:, None, :, None],
                                                     (old * shrink).round(), old).to(torch.int8)
    step = new[block][..., None]
    codes[page, :, row] = torch.where(step > 0, x / step, 0).round().clamp(-127, 127).to(torch.int8)
    scales.copy_(new.reshape(-1, blocks, heads).permute(0, 2, 1))


def _read_back(s, cu, total):
    _, _, page, row = _places(s, cu, total)
    return [(s["c" + n][page, :, row].float() * s["s" + n][page, :, row // BLOCK][..., None]).bfloat16() for n in "kv"]


def _whole(codes, scales, table):
    """[seqs, heads, tokens, dim] in FP32."""
    x = codes[table.long()].float()                                         # [seqs, pages, heads, page, dim]
    x = x * scales[table.long()].repeat_interleave(BLOCK, -1)[..., None]
    return x.permute(0, 2, 1, 3, 4).flatten(2, 3)


def _attention(s):
    k, v = _whole(s["ck"], s["sk"], s["table"]), _whole(s["cv"], s["sv"], s["table"])
    seqs, hk, length, dim = k.shape
    n, hq, dev = s["new_most"], s["hq"], k.device
    kv = s["kv_len"].long()
    cu = torch.arange(seqs + 1, device=dev) if s["cu"] is None else s["cu"].long()
    i = torch.arange(n, device=dev)
    q = s["q"][(cu[:-1, None] + i).clamp(max=s["total"] - 1)].float()       # [seqs, n, heads, dim]
    q = q.view(seqs, n, hk, hq // hk, dim).permute(0, 2, 3, 1, 4).flatten(2, 3)
    scores = torch.matmul(q, k.transpose(-1, -2)).mul_(s["scale"]).view(seqs, hk, hq // hk, n, length)
    at = torch.arange(length, device=dev)
    last = (kv - (cu[1:] - cu[:-1]))[:, None] + i if s["causal"] else (kv - 1)[:, None] + 0 * i
    hidden = (at > last[..., None]) | (at >= kv[:, None, None])
    scores.masked_fill_(hidden[:, None, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    scores.sub_(torch.where(top.isinf(), 0, top)).exp_()
    total = scores.sum(-1, keepdim=True)
    out = torch.matmul(scores.flatten(2, 3), v).view(seqs, hk, hq // hk, n, dim) / torch.where(total > 0, total, 1)
    lse = (top + total.log())[..., 0]
    b = torch.searchsorted(cu, torch.arange(s["total"], device=dev), right=True) - 1
    j = torch.arange(s["total"], device=dev) - cu[b]
    return [out[b, :, :, j].flatten(1, 2).bfloat16(), lse[b, :, :, j].flatten(1, 2)]


def run(s):
    op = s["op"]
    if own:
        for call in s["calls"]:
            call()
        if op == "attn":
            return [s["out"], s["lse"]]
        if op == "read":
            return [s["k_back"], s["v_back"]]
        return [s["q_out"], s["k_out"]] if op == "norm_rope" else [s["q_out"], s["k_back"], s["v_back"]]
    if op == "norm_rope":
        return [_norm_rotate(x, w, s["table_cs"], s["positions"], s["axis"], s["adjacent"]).bfloat16()
                for x, w in ((s["q"], s["qw"]), (s["k"], s["kw"]))]
    if op == "attn":
        return _attention(s)
    if op == "read":
        return _read_back(s, s["cu"], s["total"])
    b, at, page, row = _places(s, s["cu"], s["total"])
    q, k = (_norm_rotate(x, w, s["table_cs"], at[None], None, s["adjacent"]) for x, w in ((s["q"], s["qw"]), (s["k"], s["kw"])))
    news = s["kv_len"].new_ones(s["kv_len"].numel()) if s["cu"] is None else s["cu"][1:] - s["cu"][:-1]
    first = (s["kv_len"] - news).long()
    _store(s["ck"], s["sk"], k, first, b, page, row, s["table"], s["page"])
    _store(s["cv"], s["sv"], s["v"].float(), first, b, page, row, s["table"], s["page"])
    return [q.bfloat16()] + _read_back(s, s["back_cu"], s["back"])


# ------------------------------------------------------------------ the definition in 64 bits
def _turned(x, weight, angles, adjacent):
    """Normalised heads as complex numbers times unit numbers; angles complex [t, pairs]."""
    y = x.double()
    if weight is not None:
        y = y / (y.pow(2).sum(-1, keepdim=True) / y.shape[-1] + EPS).sqrt() * weight.double()
    pairs = angles.shape[1]
    parts = y[..., :2 * pairs].unflatten(-1, (pairs, 2) if adjacent else (2, pairs))
    z = torch.view_as_complex((parts if adjacent else parts.transpose(-1, -2)).contiguous()) * angles[:, None]
    out = torch.view_as_real(z)
    y = y.clone()
    y[..., :2 * pairs] = (out if adjacent else out.transpose(-1, -2)).flatten(-2)
    return y


def _block_values(x, offset, codes, scale):
    """A block's values after x [m, heads, dim] joins `offset` older tokens, codes [heads, 16, dim]."""
    most = x.abs().amax((0, 2))
    if offset == 0:
        scale, old = most / 127, codes[:, :0].double()
    else:
        old = codes[:, :offset].double()
        for _ in range(24):
            over = most / scale.clamp(min=1e-300) >= 127.5
            scale = torch.where(over, 2 * scale, scale)
            old = torch.where(over[:, None, None], old / 2, old)
    new = (x.transpose(0, 1) / scale.clamp(min=1e-300)[:, None, None]).round().clamp(-127, 127)
    return (torch.cat([old.round(), new], 1) * scale[:, None, None]).transpose(0, 1)


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op == "norm_rope":
        cs = torch.view_as_complex(s["table_cs"].double())
        pick = torch.zeros(cs.shape[1], dtype=torch.long, device=cs.device) if s["axis"] is None else s["axis"].long()
        angles = torch.stack([cs[s["positions"][int(a)].long(), i] for i, a in enumerate(pick.tolist())], 1)
        return [_turned(s["q"], s["qw"], angles, s["adjacent"]), _turned(s["k"], s["kw"], angles, s["adjacent"])]
    page = s["page"]
    kv = s["kv_len"].tolist()
    n = [1] * len(kv) if s["cu"] is None else (s["cu"][1:] - s["cu"][:-1]).tolist()
    starts = _cumulated(n)

    def stored(name, b, low, high):
        """[high - low, heads, dim] of sequence b's cached values."""
        at = torch.arange(low, high, device="cuda")
        pages, rows = s["table"][b].long()[at // page], at % page
        return s["c" + name][pages, :, rows].double() * s["s" + name][pages, :, rows // BLOCK].double()[..., None]

    if op == "read":
        return [torch.cat([stored(name, b, 0, kv[b]) for b in range(len(kv))]) for name in "kv"]
    if op == "append":
        at = torch.cat([torch.arange(kv[b] - n[b], kv[b], device="cuda") for b in range(len(kv))])
        angles = torch.view_as_complex(s["table_cs"].double())[at]
        q, k = _turned(s["q"], s["qw"], angles, s["adjacent"]), _turned(s["k"], s["kw"], angles, s["adjacent"])
        got = [q]
        for name, x in (("k", k), ("v", s["v"].double())):
            values = []
            for b in range(len(kv)):
                p, t = kv[b] - n[b], starts[b]
                while p < kv[b]:
                    offset = p % BLOCK
                    m = min(BLOCK - offset, kv[b] - p)
                    where, row = int(s["table"][b, p // page]), p % page // BLOCK
                    values.append(_block_values(x[t:t + m], offset, s["c" + name][where, :, row * BLOCK:(row + 1) * BLOCK],
                                                s["s" + name][where, :, row].double()))
                    p, t = p + m, t + m
            got.append(torch.cat(values))
        return got
    hq = s["hq"]
    outs, sums = [], []
    for b in range(len(kv)):
        k, v = stored("k", b, 0, kv[b]), stored("v", b, 0, kv[b])
        q = s["q"][starts[b]:starts[b + 1]].double() * s["scale"]
        o, z = torch.empty_like(q), q.new_empty(n[b], hq)
        last = torch.arange(kv[b] - n[b], kv[b], device="cuda") if case["causal"] else torch.full((n[b],), kv[b], device="cuda")
        seen = torch.arange(kv[b], device="cuda") <= last[:, None]
        for h in range(hq):
            w = torch.einsum("id,jd->ij", q[:, h], k[:, h * k.shape[1] // hq]).masked_fill(~seen, -math.inf)
            z[:, h] = torch.logsumexp(w, -1)
            o[:, h] = torch.einsum("ij,jd->id", (w - z[:, h, None]).exp(), v[:, h * k.shape[1] // hq])
        outs.append(o)
        sums.append(z)
    return [torch.cat(outs), torch.cat(sums)]
