"""The operators of the 4-bit K/V cache: what is measured, and their plain forms.

A cache with ``kv_bits = 4`` holds every row (the d values of one token and KV head) in groups
of 32 values: s = bf16(max|x| / 7) per group and one 4-bit code per value,
c = 8 + sign(x) floor(|x| / s + 1/2), so that a value reads back as (c - 8) s. A page holds one
block of one group (batch entry, KV head): [block][d/2] bytes of codes, then [block][d/32] bf16
scales. In a K row the word at byte c*(d/8) + 4g has the codes of values 32g + 8c + 0..7 (lowest
bits first); in a V row the 16-bit word at byte r*(d/16) + 2g has those of 32g + 4r + 0..3.

Three operators, by a case's "op":
  write   K and V of a run of tokens per sequence go into the cache's pages; the cache is read
          back, so that the outputs are the values that it holds
  read    tokens of the cache come back as bf16
  attend  decode attention of one query token per sequence over selected blocks of the cache
"""
import math

import torch

own = False

GROUP = 32


# ------------------------------------------------------------------------------- cases
def listed():
    return [
        # one decoded token for each sequence of a batch, in the middle of a block: latency
        dict(name="write one token", op="write", B=16, Hq=32, Hkv=8, d=128, block=64, T=1, ragged=False, start=32741),
        # a few prompts of unlike lengths, one after the other in one buffer, small heads and blocks
        dict(name="write ragged prompts", op="write", B=5, Hq=8, Hkv=2, d=64, block=32, T=4097, ragged=True, start=0),
        # the prompts of a batch on a Llama-shaped layer
        dict(name="write long prompts", op="write", B=4, Hq=32, Hkv=8, d=128, block=64, T=32768, ragged=False, start=0),
        # a prompt continued in chunks: the chunk before it comes back for its attention
        dict(name="read one chunk", op="read", B=1, Hq=32, Hkv=8, d=128, block=64, T=509, ragged=False, start=1024),
        # sequences of unlike lengths, large blocks
        dict(name="read ragged", op="read", B=7, Hq=16, Hkv=4, d=64, block=128, T=8191, ragged=True, start=0),
        # a whole layer's cache handed to a dense prompt attention
        dict(name="read long", op="read", B=4, Hq=32, Hkv=8, d=128, block=64, T=32768, ragged=False, start=0),
        # one short sequence, few heads: latency
        dict(name="attend tiny", op="attend", B=1, Hq=8, Hkv=2, d=64, block=64, T=4097, ragged=False, k=16),
        # a decode batch on a Llama-shaped layer, 64 of 513 blocks
        dict(name="attend decode batch", op="attend", B=16, Hq=32, Hkv=8, d=128, block=64, T=32769, ragged=False, k=64),
        # eight query heads to a KV head, large blocks, unlike lengths, the shortest below its budget
        dict(name="attend ragged wide groups", op="attend", B=6, Hq=64, Hkv=8, d=128, block=128, T=16384, ragged=True, k=24),
        # one query head to a KV head, small heads and blocks
        dict(name="attend single heads", op="attend", B=8, Hq=16, Hkv=16, d=64, block=32, T=8191, ragged=False, k=77),
        # one long sequence, every block: few rows over a long axis
        dict(name="attend one whole cache", op="attend", B=1, Hq=32, Hkv=8, d=128, block=64, T=131072, ragged=False, k=2048),
        # a batch of long sequences, every block
        dict(name="attend whole caches", op="attend", B=4, Hq=32, Hkv=8, d=128, block=64, T=131072, ragged=False, k=2048),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["write", "read", "attend", "attend"])
    d, block = rng.choice([64, 128]), rng.choice([32, 64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 4, 8])
    case = dict(op=op, B=_log(rng, 1, 32), Hq=Hkv * G, Hkv=Hkv, d=d, block=block, ragged=rng.random() < 0.5)
    # at most a quarter of the largest listed case's rows, and what the cache can hold
    rows = (4 * 32768 * 8) // (case["B"] * Hkv)
    case["T"] = _log(rng, 1, max(2, min(65536, rows)))
    if op == "attend":
        n = -(-case["T"] // block)
        case["k"] = min(n, _log(rng, 1, max(1, n)))
    else:
        case["start"] = rng.choice([0, rng.randrange(1, 4096)])
    return case


def _lengths(case):
    """Tokens of each sequence: all T, or (ragged) spread between 1 and T, the first one T."""
    B, T = case["B"], case["T"]
    return [T if not case["ragged"] or b == 0 else 1 + (b * 7919 * (T // 3 + 1)) % T for b in range(B)]


def work(case):
    lens, d, Hkv, G = _lengths(case), case["d"], case["Hkv"], case["Hq"] // case["Hkv"]
    packed = 2 * (d // 2 + d // 16)  # bytes of one token's K and V in the cache
    plain = 2 * 2 * d                # and in bf16
    if case["op"] == "attend":
        rows = Hkv * sum(min(L, case["k"] * case["block"]) for L in lens)
        return {"bytes": rows * packed + case["B"] * case["Hq"] * d * 6, "flops": 4 * G * d * rows}
    rows = Hkv * sum(lens)
    if case["op"] == "read":
        return {"bytes": rows * (packed + plain), "flops": 2 * 2 * d * rows}
    return {"bytes": rows * (2 * plain + packed), "flops": 2 * 8 * d * rows}


# ------------------------------------------------------------------------------- inputs
def _rows(gen, n, Hkv, d, keys):
    """K or V rows [n, Hkv, d]: normal values; keys with a few channels of larger spread."""
    x = torch.randn(n, Hkv, d, generator=gen, device="cuda", dtype=torch.bfloat16)
    if keys:
        x[..., 3::29] *= 4
    return x


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    B, Hkv, d, block = case["B"], case["Hkv"], case["d"], case["block"]
    lens = _lengths(case)
    start = case.get("start", 0)
    blocks = -(-(start + max(lens)) // block)
    cu = [0]
    for L in lens:
        cu.append(cu[-1] + L)
    s = dict(op=case["op"], B=B, Hq=case["Hq"], Hkv=Hkv, d=d, block=block, blocks=blocks, n=cu[-1], k=case.get("k", 1),
             lens=torch.tensor(lens, device="cuda", dtype=torch.int32), cu=torch.tensor(cu, device="cuda", dtype=torch.int32),
             start=torch.full((B,), start, device="cuda", dtype=torch.int32))
    if case["op"] == "write":
        s["k_in"], s["v_in"] = _rows(gen, s["n"], Hkv, d, True), _rows(gen, s["n"], Hkv, d, False)
    else:
        # a filled cache: pages of [B*Hkv][blocks], every token of them written
        pages = []
        for keys in (True, False):
            x = _rows(gen, B * Hkv, blocks * block, d, keys)
            pages.append(_pack(*_quantise(x.view(B * Hkv, blocks, block, d)), keys))
        s["k_pages"], s["v_pages"] = pages
    if case["op"] == "attend":
        s["q"] = torch.randn(B, case["Hq"], d, generator=gen, device="cuda", dtype=torch.bfloat16)
        # each group's blocks: k of its sequence's, ascending, -1 where it has fewer
        n = ((s["lens"] + block - 1) // block).repeat_interleave(Hkv)
        r = torch.rand(B * Hkv, blocks, generator=gen, device="cuda")
        r[torch.arange(blocks, device="cuda") >= n[:, None]] = 2.0
        sel = r.argsort(dim=1)[:, : case["k"]]
        sel = torch.where(torch.gather(r, 1, sel) < 1.5, sel, blocks).sort(dim=1).values
        s["sel"] = torch.where(sel < blocks, sel, -1).to(torch.int32)
        s["out"] = torch.empty(B, case["Hq"], d, device="cuda")
    else:
        s["k_out"] = torch.empty(s["n"], Hkv, d, device="cuda", dtype=torch.bfloat16)
        s["v_out"] = torch.empty_like(s["k_out"])
    if own:
        # the handle that a serving program keeps for each layer
        import kv_cache_offload_nosa_b200 as nosa
        cfg = nosa.make_config(B, case["Hq"], Hkv, d, block, 16, min(s["k"], blocks), 0, blocks, kv_bits=4)
        s["cache"] = nosa.NosaCache(cfg)
        if case["op"] != "write":
            s["cache"].pool_view("k_pool").copy_(s["k_pages"])
            s["cache"].pool_view("v_pool").copy_(s["v_pages"])
            s["cache"].init(s["lens"])
    return s


# ------------------------------------------------------------------------------- plain forms
def _quantise(x):
    """Codes (0..15, uint8) and scales (bf16) of rows x[..., d]."""
    g = x.float().view(*x.shape[:-1], -1, GROUP)
    s = (g.abs().amax(dim=-1, keepdim=True) / 7).to(torch.bfloat16).float()
    s = torch.where(s < 2.0**-126, torch.zeros_like(s), s)
    c = torch.sign(g) * torch.floor(g.abs() / torch.where(s == 0, torch.ones_like(s), s) + 0.5)
    c = torch.where(s == 0, torch.zeros_like(c), c)
    return (c + 8).to(torch.uint8), s.squeeze(-1).to(torch.bfloat16)


def _value(codes, scales):
    """float32 values (c - 8) s of codes[..., d/32, 32] and scales[..., d/32]."""
    return ((codes.float() - 8) * scales.float().unsqueeze(-1)).flatten(-2)


def _pack(codes, scales, keys):
    """Pages [ng, blocks, bytes] (uint8) of codes [ng, blocks, block, d/32, 32] and their scales."""
    ng, blocks, block, ngr = scales.shape
    i = 8 if keys else 4  # codes of a word, chunks of a row: 32 / i
    w = codes.view(ng, blocks, block, ngr, GROUP // i, i).transpose(3, 4).reshape(ng, blocks, block, -1, 2)
    w = (w[..., 0] | (w[..., 1] << 4)).reshape(ng, blocks, -1)
    return torch.cat([w, scales.contiguous().view(torch.uint8).reshape(ng, blocks, -1)], dim=2)


def _unpack(pages, block, d, keys):
    """float32 values [pages, block, d] of pages [n, bytes]."""
    n, ngr, i = pages.shape[0], d // GROUP, 8 if keys else 4
    w = pages[:, : block * d // 2].reshape(n, block, GROUP // i, ngr, i // 2)
    codes = torch.stack([w & 15, w >> 4], dim=-1).transpose(2, 3).reshape(n, block, ngr, GROUP)
    scales = pages[:, block * d // 2 :].contiguous().view(torch.bfloat16).reshape(n, block, ngr)
    return _value(codes, scales)


def _read(s):
    """K and V of the tokens of each sequence, [n, Hkv, d] in bf16."""
    t = torch.arange(s["n"], device="cuda")
    b = torch.searchsorted(s["cu"][1:].long(), t, right=True)
    pos = s["start"].long()[b] + t - s["cu"].long()[b]
    page = (b[:, None] * s["Hkv"] + torch.arange(s["Hkv"], device="cuda")) * s["blocks"] + (pos // s["block"])[:, None]
    at = page * s["block"] + (pos % s["block"])[:, None]
    out = {}
    for name, keys in (("k", True), ("v", False)):
        x = _unpack(s[name + "_pages"].flatten(0, 1), s["block"], s["d"], keys)
        out[name] = x.view(-1, s["d"])[at].to(torch.bfloat16)
    return out


def _attend(s):
    B, Hkv, G, d, block, k = s["B"], s["Hkv"], s["Hq"] // s["Hkv"], s["d"], s["block"], s["sel"].shape[1]
    ng = B * Hkv
    page = torch.arange(ng, device="cuda")[:, None] * s["blocks"] + s["sel"].long().clamp(min=0)
    K = _unpack(s["k_pages"].flatten(0, 1)[page.view(-1)], block, d, True).view(ng, k * block, d)
    V = _unpack(s["v_pages"].flatten(0, 1)[page.view(-1)], block, d, False).view(ng, k * block, d)
    tok = s["sel"].long()[:, :, None] * block + torch.arange(block, device="cuda")
    seen = (s["sel"][:, :, None] >= 0) & (tok < s["lens"].long().repeat_interleave(Hkv)[:, None, None])
    x = torch.matmul(s["q"].float().view(ng, G, d), K.transpose(1, 2)) / math.sqrt(d)
    x = x.masked_fill(~seen.view(ng, 1, k * block), float("-inf"))
    p = torch.exp(x - x.amax(dim=-1, keepdim=True))
    return (torch.matmul(p, V) / p.sum(dim=-1, keepdim=True)).view(B, s["Hq"], d)


def run(s):
    if own:
        if s["op"] == "attend":
            s["cache"].decode_attn(s["q"], s["sel"], s["out"])
            return {"out": s["out"]}
        if s["op"] == "write":
            s["cache"].write(s["k_in"], s["v_in"], s["cu"], s["start"])
        s["cache"].read(s["k_out"], s["v_out"], s["cu"], s["start"])
        return {"k": s["k_out"], "v": s["v_out"]}
    if s["op"] == "attend":
        return {"out": _attend(s)}
    if s["op"] == "read":
        return _read(s)
    return {"k": _value(*_quantise(s["k_in"])).to(torch.bfloat16), "v": _value(*_quantise(s["v_in"])).to(torch.bfloat16)}


# ------------------------------------------------------------------------------- 64 bits
def _held(x):
    """The values that the cache holds for rows x, in 64 bits, from the definition: the scale is
    the multiple of its last place (2^-7 of its power of two) nearest to max|x| / 7, a value the
    multiple of the scale nearest to x, halves away from zero."""
    y = x.double().unflatten(-1, (-1, GROUP))
    a = y.abs().max(dim=-1, keepdim=True).values / 7
    ulp = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0**-126))) - 7)
    step = torch.round(a / ulp) * ulp  # a / 7 is never half way between two multiples
    m = torch.trunc(2 * y / step.clamp(min=2.0**-126))
    m = torch.where(m < 0, -torch.div(1 - m, 2, rounding_mode="floor"), torch.div(m + 1, 2, rounding_mode="floor"))
    return torch.where(step >= 2.0**-126, m * step, 0.0).flatten(-2)


def _held_page(page, block, d, chunk):
    """64-bit values of pages [n, bytes], by each value's own place in its page (chunk: codes in a word)."""
    e = torch.arange(d, device="cuda")
    g, c, i = e // 32, e % 32 // chunk, e % chunk
    byte = c * (d * chunk // 64) + g * (chunk // 2) + i // 2
    row = torch.arange(block, device="cuda")[:, None]
    code = (page[:, row * (d // 2) + byte] >> (4 * (i % 2)).to(torch.uint8)) & 15
    at = block * d // 2 + row * (d // 16) + 2 * g
    bits = page[:, at].int() | (page[:, at + 1].int() << 8)
    return (code.double() - 8) * (bits << 16).view(torch.float32).double()


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "write":
        return {"k": _held(s["k_in"]), "v": _held(s["v_in"])}
    B, Hkv, d, block = s["B"], s["Hkv"], s["d"], s["block"]
    lens, start, G = s["lens"].tolist(), s["start"].tolist(), s["Hq"] // s["Hkv"]
    if s["op"] == "read":
        out = {}
        for name, chunk in (("k", 8), ("v", 4)):
            runs = []
            for b in range(B):
                heads = [_held_page(s[name + "_pages"][b * Hkv + h], block, d, chunk).flatten(0, 1) for h in range(Hkv)]
                runs.append(torch.stack([x[start[b] : start[b] + lens[b]] for x in heads], dim=1))
            out[name] = torch.cat(runs)
        return out
    out = torch.zeros(B, s["Hq"], d, dtype=torch.float64, device="cuda")
    for b in range(B):
        for h in range(Hkv):
            blocks = s["sel"][b * Hkv + h]
            blocks = blocks[blocks >= 0].long()
            at = (blocks[:, None] * block + torch.arange(block, device="cuda")).flatten()
            K = _held_page(s["k_pages"][b * Hkv + h][blocks], block, d, 8).flatten(0, 1)[at < lens[b]]
            V = _held_page(s["v_pages"][b * Hkv + h][blocks], block, d, 4).flatten(0, 1)[at < lens[b]]
            w = torch.softmax(s["q"][b, h * G : (h + 1) * G].double() @ K.T * d**-0.5, dim=-1)
            out[b, h * G : (h + 1) * G] = w @ V
    return {"out": out}
