"""Operators of grouped-query caches in 4 bits and of the unquantized latent cache: cases and plain forms.

Three operators of the library stand here next to a plain statement of what they compute:

  kv4_append   keys and values of new tokens enter a paged cache in 4 bits; keys (and the step's
               queries) are rotated to their positions on the way.
  kv4_attn     attention of ragged query rows over that cache: single tokens, a few drafted
               tokens, or chunks of a prompt; causal, optionally within a sliding window.
  append_bf16  latent rows enter the paged BF16 cache that the unquantized decode reads: RMS norm
               of the latent, rotation of the positional key and of the queries' positional part.

The cache in 4 bits holds, for each token, head and group of channels, an FP16 minimum m (rounded
down), an FP16 scale s (rounded up) and codes 0..15; a code n stands for m + n s. A page has one
region for each kv head: P rows of key codes, P rows of value codes (D/2 bytes each), then for
each token and group the four FP16 numbers (key scale, key minimum, value scale, value minimum).
The order of the channels inside a row of codes is given by _key_order and _value_order below.
"""
import math
import random

import torch

own = False


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one user's chat, one new token after 1K tokens: latency alone counts
        dict(name="attn_one_1k", op="attn", B=1, lens="same", T=1024, q_len=1, Hq=32, Hkv=8, D=128, group=128, P=64, dtype="bf16",
             window=0, lse=True, salt=1),
        # a served batch in its steady state
        dict(name="attn_batch_8k", op="attn", B=32, lens="same", T=8192, q_len=1, Hq=32, Hkv=8, D=128, group=128, P=128, dtype="bf16",
             window=0, lse=True, salt=2),
        # continuous batching: every length between 512 and 16K, pages scattered over the pool
        dict(name="attn_ragged_serve", op="attn", B=64, lens="ragged", T=16384, q_len=1, Hq=16, Hkv=2, D=128, group=64, P=64,
             dtype="fp16", window=0, lse=True, salt=3),
        # one long document
        dict(name="attn_long_128k", op="attn", B=1, lens="same", T=131072, q_len=1, Hq=64, Hkv=8, D=128, group=128, P=128, dtype="bf16",
             window=0, lse=True, salt=4),
        # five drafted tokens verified at once, lengths of no round number
        dict(name="attn_verify_5", op="attn", B=8, lens="ragged", T=32003, q_len=5, Hq=32, Hkv=4, D=128, group=64, P=128, dtype="bf16",
             window=0, lse=True, salt=5),
        # a small drafting model with a sliding window, seven query heads to a kv head
        dict(name="attn_window_d64", op="attn", B=16, lens="ragged", T=20011, q_len=1, Hq=14, Hkv=2, D=64, group=64, P=16, dtype="fp16",
             window=4096, lse=True, salt=6),
        # the second 4K chunk of two prompts
        dict(name="attn_prompt_4k_of_8k", op="attn", B=2, lens="same", T=8192, q_len=4096, Hq=32, Hkv=8, D=128, group=128, P=128,
             dtype="bf16", window=0, lse=False, salt=7),
        # short prompts of odd lengths in one call
        dict(name="attn_prompts_odd", op="attn", B=5, lens="ragged", T=3333, q_len=777, Hq=14, Hkv=2, D=64, group=32, P=16, dtype="fp16",
             window=0, lse=False, salt=8),
        # the append of one decode step
        dict(name="append_step_b32", op="append", B=32, lens="ragged", T=8192, q_len=1, Hq=32, Hkv=8, D=128, group=128, P=128,
             dtype="bf16", rot=128, interleaved=False, salt=9),
        # the append of four prompts
        dict(name="append_prompt_16k", op="append", B=4, lens="same", T=9001, q_len=4096, Hq=32, Hkv=8, D=128, group=64, P=64,
             dtype="bf16", rot=128, interleaved=False, salt=10),
        # the latent cache, one decode step of 16 heads
        dict(name="append_bf16_step_b32", op="append_bf16", B=32, lens="ragged", T=8192, q_len=1, Hq=16, P=64, interleaved=True, salt=11),
        # the latent cache, two prompts
        dict(name="append_bf16_prompt_16k", op="append_bf16", B=2, lens="ragged", T=8192, q_len=8192, Hq=16, P=128, interleaved=True,
             salt=12),
    ]


def _log(rng, lo, hi):
    """A whole number, spread over the logarithm of [lo, hi]."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "append", "append_bf16"])
    c = dict(op=op, lens=rng.choice(["same", "ragged"]), P=rng.choice([16, 32, 64, 128]), salt=rng.randrange(1 << 30))
    if op == "append_bf16":
        c.update(P=rng.choice([32, 64, 128]), Hq=rng.choice([16, 32, 64, 128]), interleaved=rng.random() < 0.5, B=_log(rng, 1, 64))
        c["q_len"] = _log(rng, 1, max(1, min(8192, 16384 * 16 // (c["Hq"] * c["B"]))))
        c["T"] = c["q_len"] + _log(rng, 1, 8192)
        return c
    D = rng.choice([64, 128, 128])
    Hkv, G = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 5, 7, 8, 12, 16])
    c.update(D=D, Hkv=Hkv, Hq=Hkv * G, group=rng.choice([g for g in (32, 64, 128) if g <= D]), dtype=rng.choice(["bf16", "fp16"]),
             B=_log(rng, 1, 64))
    if op == "append":
        c["rot"] = rng.choice([D, D, D // 2])
        c["interleaved"] = rng.random() < 0.5
        c["q_len"] = _log(rng, 1, max(1, min(8192, 12288 * 48 * 128 // ((c["Hq"] + 2 * Hkv) * D * c["B"]))))
        c["T"] = c["q_len"] + _log(rng, 1, 8192)
        return c
    kind = rng.choice(["one", "one", "few", "prompt"])
    tokens = 32 * 8192 * 8 * 128 // (Hkv * D * c["B"])  # cached tokens of one sequence, at most
    c["T"] = _log(rng, 1, min(131072, tokens))
    if kind == "prompt":
        pairs = 2 * 4096 * 8192 * 32 * 128 // (c["Hq"] * D * c["B"])  # query rows x cached tokens of one sequence, at most
        c["T"] = min(c["T"], 8192, max(1, int(math.sqrt(pairs * 2))))
        c["q_len"] = _log(rng, 1, max(1, min(c["T"], pairs // c["T"])))
    else:
        c["q_len"] = 1 if kind == "one" else min(c["T"], rng.randint(2, 8))
    c["window"] = rng.choice([0, 0, 0, _log(rng, 1, 8192)])
    c["lse"] = kind != "prompt"
    return c


def _lengths(case):
    """(cached tokens with the new ones, new rows) of each sequence: part of the case, not of the seed."""
    rng = random.Random(case["salt"])
    B, T, n = case["B"], case["T"], case["q_len"]
    if case["lens"] == "same":
        return [T] * B, [n] * B
    lens = [rng.randint(max(1, T // 32), T) for _ in range(B)]
    new = [min(t, n if n <= 8 else rng.randint(max(1, n // 8), n)) for t in lens]
    lens[0], new[0] = T, min(n, T)
    return lens, new


def _pairs(case):
    """Query rows x tokens that they see, of one head."""
    w = case.get("window", 0)
    total = 0
    for t, n in zip(*_lengths(case)):
        first = t - n + 1  # tokens that the first row sees without a window; the last one sees t
        rising = t if not w else max(first - 1, min(t, w))  # rows that see first, first + 1, ... rising tokens, then rows that see w
        total += (first + rising) * (rising - first + 1) // 2 + (t - rising) * min(t, w or t)
    return total


def _seen(case):
    """Cached tokens that some query row sees."""
    w = case.get("window", 0)
    return sum(min(t, n + w - 1) if w else t for t, n in zip(*_lengths(case)))


def work(case):
    lens, new = _lengths(case)
    rows = sum(new)
    if case["op"] == "append_bf16":
        H = case["Hq"]
        return {"bytes": rows * (2 * 576 * 2 + 2 * H * 64 * 2 + 64 * 4) + 512 * 2, "flops": rows * (512 * 4 + (H + 1) * 64 * 3)}
    D, Hq, Hkv, groups = case["D"], case["Hq"], case["Hkv"], case["D"] // case["group"]
    if case["op"] == "append":
        kv = 2 * Hkv * D
        return {"bytes": rows * (2 * kv * 2 + 2 * Hq * D * 2 + kv // 2 + Hkv * groups * 8 + case["rot"] * 4),
                "flops": rows * ((Hq + Hkv) * case["rot"] * 3 + kv * 4)}
    return {"bytes": _seen(case) * Hkv * (D + 8 * groups) + 2 * rows * Hq * D * 2 + (rows * Hq * 4 if case["lse"] else 0),
            "flops": 4 * D * Hq * _pairs(case)}


# ---------------------------------------------------------------- the cache in 4 bits, plainly
def _half_down(x):
    """The largest FP16 value that is no more than x (float64)."""
    h = x.to(torch.float32).to(torch.float16)
    bits = h.view(torch.int16).to(torch.int32) & 0xFFFF
    below = torch.where(bits == 0, 0x8001, torch.where(bits < 0x8000, bits - 1, bits + 1))
    bits = torch.where(h.double() > x, below, bits)
    bits = torch.where((bits & 0x7FFF) == 0, torch.zeros_like(bits), bits)  # zero is +0
    return bits.to(torch.int16).view(torch.float16)


def _half_up(x):
    return -_half_down(-x) + 0.0


def _quantize(x, group):
    """x [..., D] in 32 bits -> codes [..., D] (uint8), scale and minimum [..., D / group] (FP16)."""
    v = x.double().unflatten(-1, (-1, group))
    m = _half_down(v.amin(-1))
    s = _half_up((v.amax(-1) - m.double()) / 15.0)
    step = torch.where(s > 0, s.double(), torch.ones_like(s, dtype=torch.float64))
    codes = torch.round((v - m.double().unsqueeze(-1)) / step.unsqueeze(-1)).clamp(0, 15)
    codes = torch.where(s.unsqueeze(-1) > 0, codes, torch.zeros_like(codes))
    return codes.to(torch.uint8).flatten(-2), s, m


def _values(codes, s, m, group):
    v = codes.unflatten(-1, (-1, group)).float()
    return (v * s.float().unsqueeze(-1) + m.float().unsqueeze(-1)).flatten(-2)


def _key_order(D):
    """Channel of each nibble of a row of key codes (nibble i: byte i // 2, the low one first)."""
    return torch.arange(D).view(D // 32, 4, 8).permute(1, 0, 2).reshape(-1)


def _value_order(D):
    return torch.arange(D).view(D // 64, 4, 2, 8).permute(3, 0, 2, 1).reshape(-1)


def _pack(codes, order):
    n = codes[..., order]
    return n[..., 0::2] | (n[..., 1::2] << 4)


def _unpack(packed, order):
    n = torch.stack([packed & 15, packed >> 4], -1).flatten(-2)
    return n[..., torch.argsort(order)]


def _head_bytes(D, group, P):
    return P * (D + 8 * (D // group))


def _page_of(kc, ks, km, vc, vs, vm, D, P):
    """Codes and numbers of whole pages, [pages, Hkv, P, ...] -> [pages, bytes]."""
    dev = kc.device
    meta = torch.stack([ks, km, vs, vm], -1).contiguous()
    parts = [_pack(kc, _key_order(D).to(dev)).flatten(-2), _pack(vc, _value_order(D).to(dev)).flatten(-2),
             meta.view(torch.uint8).flatten(-3)]
    return torch.cat(parts, -1).flatten(1).contiguous()


# ---------------------------------------------------------------- inputs
def _type(case):
    return torch.float16 if case["dtype"] == "fp16" else torch.bfloat16


def _tables(n_pos, rot, dev):
    """cos, sin [n_pos, rot / 2] of the angles pos * 10000^(-2 i / rot), formed in 64 bits."""
    a = torch.arange(n_pos, device=dev, dtype=torch.float64)[:, None] * \
        10000.0 ** (-torch.arange(0, rot, 2, device=dev, dtype=torch.float64) / rot)[None]
    return a.cos().float(), a.sin().float()


def _ints(v, dev):
    return torch.tensor(v, dtype=torch.int32, device=dev)


def _offsets(new, dev):
    out = [0]
    for n in new:
        out.append(out[-1] + n)
    return _ints(out, dev)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed * 7919 + 17)
    lens, new = _lengths(case)
    B, P, rows = case["B"], case["P"], sum(new)
    max_pages = -(-max(lens) // P) + 1
    n_pages = B * max_pages
    table = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32).view(B, max_pages)
    randn = lambda *shape: torch.randn(shape, generator=g, device=dev)  # noqa: E731
    s = dict(case=case, page_table=table, cu=_offsets(new, dev), max_new=max(new), err=torch.zeros(1, dtype=torch.int32, device=dev))
    if case["op"] == "append_bf16":
        H = case["Hq"]
        s["lens"] = _ints([t - n for t, n in zip(lens, new)], dev)
        s["cos"], s["sin"] = _tables(max(lens), 64, dev)
        s["kv"] = (randn(rows, 576) * 2).bfloat16()
        s["weight"] = (1 + 0.1 * randn(512)).bfloat16()
        s["q"] = randn(rows, H, 192).bfloat16()  # a head's query: 128 channels without a position, then 64 with one
        s["pool"] = randn(n_pages, P, 576).bfloat16()
        s["q_out"] = torch.empty(rows, H, 64, dtype=torch.bfloat16, device=dev)
        s["next"] = torch.empty_like(s["lens"])
        return s
    D, Hq, Hkv, group, dtype = case["D"], case["Hq"], case["Hkv"], case["group"], _type(case)
    loud = 1 + 3 * (torch.rand(D, generator=g, device=dev) < 0.05).float()  # the few channels that stand out in keys
    if case["op"] == "append":
        s["lens"] = _ints([t - n for t, n in zip(lens, new)], dev)
        s["cos"], s["sin"] = _tables(max(lens), case["rot"], dev)
        qkv = randn(rows, Hq + 2 * Hkv, D)  # one projection's output: queries, keys and values are views of it
        qkv[:, Hq:Hq + Hkv] *= loud
        qkv = qkv.to(dtype)
        s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        s["pool"] = torch.randint(0, 256, (n_pages, Hkv * _head_bytes(D, group, P)), generator=g, device=dev, dtype=torch.uint8)
        s["q_out"] = torch.empty(rows, Hq, D, dtype=dtype, device=dev)
        s["k_deq"] = torch.empty(rows, Hkv, D, dtype=dtype, device=dev)
        s["v_deq"] = torch.empty(rows, Hkv, D, dtype=dtype, device=dev)
        s["next"] = torch.empty_like(s["lens"])
        return s
    s["lens"] = _ints(lens, dev)
    s["scale"] = 1.0 / math.sqrt(D)
    s["q"] = (randn(rows, Hq, D) * 1.5).to(dtype)
    k = (randn(n_pages, Hkv, P, D) * loud).to(dtype).float()
    kc, ks, km = _quantize(k, group)
    del k
    vc, vs, vm = _quantize(randn(n_pages, Hkv, P, D).to(dtype).float(), group)
    s["pool"] = _page_of(kc, ks, km, vc, vs, vm, D, P)
    s["out"] = torch.empty(rows, Hq, D, dtype=dtype, device=dev)
    s["lse"] = torch.empty(rows, Hq, device=dev) if case["lse"] else None
    return s


# ---------------------------------------------------------------- one pass
def run(state):
    case = state["case"]
    if own:
        return _own(state, case)
    if case["op"] == "attn":
        return _attn(state, case)
    if case["op"] == "append":
        return _append(state, case)
    return _append_bf16(state, case)


def _own(s, case):
    import bit_mla_kv_qcache_gb300 as fw
    if case["op"] == "append_bf16":
        fw.mla_qcache_append_bf16(s["kv"], s["cu"], s["lens"], s["max_new"], s["page_table"], s["pool"], s["err"],
                                  norm_weight=s["weight"], eps=1e-6, cos=s["cos"], sin=s["sin"], interleaved=case["interleaved"],
                                  q_rope=s["q"][..., 128:], q_out=s["q_out"], seq_lens_next=s["next"])
        return {"pool": s["pool"], "q": s["q_out"], "lens": s["next"]}
    if "cfg" not in s:
        s["cfg"] = fw.make_kv4_config(case["Hkv"], case["D"], group=case["group"], page_size=case["P"])
    if case["op"] == "append":
        fw.mla_qcache_kv4_append(s["cfg"], s["k"], s["v"], s["cu"], s["lens"], s["max_new"], s["page_table"], s["pool"], s["err"],
                                 cos=s["cos"], sin=s["sin"], interleaved=case["interleaved"], q=s["q"], q_out=s["q_out"],
                                 k_deq=s["k_deq"], v_deq=s["v_deq"], seq_lens_next=s["next"])
        return {"pool": s["pool"], "q": s["q_out"], "k": s["k_deq"], "v": s["v_deq"], "lens": s["next"]}
    if "ws" not in s:  # kept by the program, zeroed once
        need = fw.kv4_workspace_bytes(s["cfg"], case["B"], case["Hq"], s["max_new"], s["page_table"].shape[1])
        s["ws"] = torch.zeros(need, dtype=torch.uint8, device=s["q"].device)
    fw.mla_qcache_kv4_attn(s["cfg"], s["q"], s["page_table"], s["lens"], s["pool"], s["scale"], s["out"], s["ws"], s["err"],
                           cu_q=s["cu"], max_q=s["max_new"], lse=s["lse"], window=case["window"])
    return {"out": s["out"], "lse": s["lse"]}


def _rows(s):
    """Sequence and position of each new row."""
    cu, r = s["cu"].long(), torch.arange(int(s["q"].shape[0]), device=s["q"].device)
    b = torch.searchsorted(cu, r, right=True) - 1
    return b, r - cu[b]


def _rotate(x, cos, sin, interleaved):
    """x [rows, heads, D] in 32 bits; cos, sin [rows, rot / 2]: the first rot channels are turned in pairs."""
    half = cos.shape[-1]
    c, t = cos[:, None], sin[:, None]
    turned, rest = x[..., :2 * half], x[..., 2 * half:]
    if interleaved:
        a, b = turned[..., 0::2], turned[..., 1::2]
        turned = torch.stack([a * c - b * t, b * c + a * t], -1).flatten(-2)
    else:
        a, b = turned[..., :half], turned[..., half:]
        turned = torch.cat([a * c - b * t, b * c + a * t], -1)
    return torch.cat([turned, rest], -1)


def _append(s, case):
    D, P, group, dtype, dev = case["D"], case["P"], case["group"], _type(case), s["q"].device
    b, i = _rows(s)
    pos = s["lens"].long()[b] + i
    cos, sin = s["cos"][pos], s["sin"][pos]
    k = _rotate(s["k"].float(), cos, sin, case["interleaved"])
    q = _rotate(s["q"].float(), cos, sin, case["interleaved"]).to(dtype)
    kc, ks, km = _quantize(k, group)
    vc, vs, vm = _quantize(s["v"].float(), group)
    head = _head_bytes(D, group, P)
    pages = s["pool"].view(s["pool"].shape[0], -1, head)
    page, t = s["page_table"].long()[b, pos // P], pos % P
    groups = D // group
    pages[:, :, :P * D // 2].unflatten(-1, (P, D // 2))[page, :, t] = _pack(kc, _key_order(D).to(dev))
    pages[:, :, P * D // 2:P * D].unflatten(-1, (P, D // 2))[page, :, t] = _pack(vc, _value_order(D).to(dev))
    meta = torch.stack([ks, km, vs, vm], -1).contiguous().view(torch.uint8).flatten(-2)
    pages[:, :, P * D:].unflatten(-1, (P, 8 * groups))[page, :, t] = meta
    return {"pool": s["pool"], "q": q, "k": _values(kc, ks, km, group).to(dtype), "v": _values(vc, vs, vm, group).to(dtype),
            "lens": s["lens"] + (s["cu"][1:] - s["cu"][:-1])}


def _append_bf16(s, case):
    b, i = _rows(s)
    pos = s["lens"].long()[b] + i
    cos, sin = s["cos"][pos], s["sin"][pos]
    x = s["kv"][:, :512].float()
    x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * s["weight"].float()
    kr = _rotate(s["kv"][:, None, 512:].float(), cos, sin, case["interleaved"])[:, 0]
    q = _rotate(s["q"][..., 128:].float(), cos, sin, case["interleaved"])
    page = s["page_table"].long()[b, pos // case["P"]]
    s["pool"][page, pos % case["P"]] = torch.cat([x, kr], -1).bfloat16()
    return {"pool": s["pool"], "q": q.bfloat16(), "lens": s["lens"] + (s["cu"][1:] - s["cu"][:-1])}


def _attn(s, case):
    B, D, P, group, Hq, Hkv = (case[x] for x in ("B", "D", "P", "group", "Hq", "Hkv"))
    G, dev, head = Hq // Hkv, s["q"].device, _head_bytes(D, group, P)
    pages = s["pool"].view(-1, Hkv, head)[s["page_table"].long()]  # [B, pages, Hkv, bytes]
    tokens = lambda x: x.transpose(1, 2).flatten(2, 3)  # noqa: E731  [B, pages, Hkv, P, ...] -> [B, Hkv, T, ...]
    meta = tokens(pages[..., P * D:].contiguous().view(torch.float16).unflatten(-1, (P, D // group, 4)))
    k = _values(_unpack(tokens(pages[..., :P * D // 2].unflatten(-1, (P, D // 2))), _key_order(D).to(dev)),
                meta[..., 0], meta[..., 1], group)
    v = _values(_unpack(tokens(pages[..., P * D // 2:P * D].unflatten(-1, (P, D // 2))), _value_order(D).to(dev)),
                meta[..., 2], meta[..., 3], group)
    b, i = _rows(s)
    n = s["max_new"]
    q = torch.zeros(B, n, Hq, D, device=dev)
    q[b, i] = s["q"].float()
    q = q.view(B, n, Hkv, G, D).permute(0, 2, 3, 1, 4).flatten(2, 3)  # [B, Hkv, G n, D]
    new = (s["cu"][1:] - s["cu"][:-1]).long()
    at = (s["lens"].long() - new)[:, None] + torch.arange(n, device=dev)  # [B, n] position of each row
    t = torch.arange(k.shape[2], device=dev)
    seen = (t <= at[..., None]) & (t < s["lens"].long()[:, None, None])
    if case["window"]:
        seen &= t > at[..., None] - case["window"]
    score = (q @ k.transpose(-1, -2)).mul_(s["scale"]).view(B, Hkv, G, n, -1)
    score.masked_fill_(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top > -math.inf, top, torch.zeros_like(top))
    p = score.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p.flatten(2, 3) @ v).view(B, Hkv, G, n, D) / torch.where(total > 0, total, torch.ones_like(total))
    o = o.permute(0, 3, 1, 2, 4).reshape(B, n, Hq, D)[b, i].to(_type(case))
    if not case["lse"]:
        return {"out": o, "lse": None}
    return {"out": o, "lse": (top + total.log()).squeeze(-1).permute(0, 3, 1, 2).reshape(B, n, Hq)[b, i]}


# ---------------------------------------------------------------- in 64 bits, from the definitions
def exact(case, seed):
    s = prepare(case, seed)
    lens, new = _lengths(case)
    if case["op"] == "attn":
        return _exact_attn(s, case, lens, new)
    base = [t - n for t, n in zip(lens, new)]
    pos = torch.cat([torch.arange(a, a + n) for a, n in zip(base, new)]).to(s["q"].device)

    def turn(x, rot):
        """x [rows, heads, D] in 64 bits: channel pairs as complex numbers, times e^(i angle) as the tables round it."""
        half = rot // 2
        e = torch.complex(s["cos"].double(), s["sin"].double())[pos][:, None]
        y = x.clone()
        first, second = (slice(0, rot, 2), slice(1, rot, 2)) if case["interleaved"] else (slice(0, half), slice(half, rot))
        z = torch.complex(x[..., first].contiguous(), x[..., second].contiguous()) * e
        y[..., first], y[..., second] = z.real, z.imag
        return y

    if case["op"] == "append_bf16":
        x = s["kv"].double()
        y = x.clone()
        y[:, :512] = x[:, :512] / (x[:, :512].pow(2).sum(-1, keepdim=True) / 512 + 1e-6).sqrt() * s["weight"].double()
        y[:, 512:] = turn(x[:, None, 512:], 64)[:, 0]
        pool, r = s["pool"].double(), 0
        for b in range(case["B"]):
            t = base[b]
            while t < lens[b]:
                n = min(lens[b] - t, case["P"] - t % case["P"])  # the rows that this page takes
                pool[int(s["page_table"][b, t // case["P"]]), t % case["P"]:t % case["P"] + n] = y[r:r + n]
                t, r = t + n, r + n
        return {"pool": pool, "q": turn(s["q"][..., 128:].double(), 64), "lens": None}

    def held(x):
        """The values that a cache of 16 levels between a group's ends holds in place of x."""
        v = x.reshape(*x.shape[:-1], -1, case["group"])
        lo, hi = v.min(-1, keepdim=True).values, v.max(-1, keepdim=True).values
        m = _on_half_grid(lo, False)
        step = _on_half_grid((hi - m) / 15, True)
        n = torch.where(step > 0, ((v - m) / step.clamp_min(1e-30)).round(), torch.zeros_like(v))
        return (m + n.clamp(0, 15) * step).reshape(x.shape)

    return {"pool": None, "q": turn(s["q"].double(), case["rot"]), "k": held(turn(s["k"].double(), case["rot"])),
            "v": held(s["v"].double()), "lens": None}


def _on_half_grid(y, up):
    """y (64 bits) on the grid of FP16 values, rounded up or down: 11 significant bits, 2^-24 at the least."""
    unit = torch.exp2((torch.frexp(y.abs())[1].double() - 11).clamp_min(-24.0))
    return (torch.ceil(y / unit) if up else torch.floor(y / unit)) * unit


def _exact_attn(s, case, lens, new):
    D, P, group, G = case["D"], case["P"], case["group"], case["Hq"] // case["Hkv"]
    head, dev = _head_bytes(D, group, P), s["q"].device
    ch = torch.arange(D, device=dev)
    # nibble that holds channel c: keys in words (4 lanes x 32-channel blocks), values in words (8 lanes x 64-channel blocks)
    k_at = (ch % 32 // 8) * (D // 32) * 8 + ch // 32 * 8 + ch % 8
    v_at = (ch % 8) * (D // 64) * 8 + ch // 64 * 8 + ch // 8 % 2 * 4 + ch // 16 % 4
    out, lse, r = [], [], 0
    for b in range(case["B"]):
        T, n = lens[b], new[b]
        page = s["page_table"][b, :-(-T // P)].long()
        rows = torch.empty(n, case["Hq"], D, dtype=torch.float64, device=dev)
        l = torch.empty(n, case["Hq"], dtype=torch.float64, device=dev)
        at = torch.arange(T - n, T, device=dev)
        t = torch.arange(T, device=dev)
        hidden = t[None] > at[:, None]
        if case["window"]:
            hidden |= t[None] <= at[:, None] - case["window"]
        for h in range(case["Hkv"]):
            region = s["pool"][page, h * head:(h + 1) * head]
            num = region[:, P * D:].contiguous().view(torch.float16).double().view(-1, D // group, 4)[:T]
            num = num.repeat_interleave(group, 1)  # [T, D, 4]
            kb, vb = region[:, :P * D // 2].reshape(-1, D // 2)[:T], region[:, P * D // 2:P * D].reshape(-1, D // 2)[:T]
            k = (kb[:, k_at // 2] >> (k_at % 2 * 4).to(torch.uint8) & 15).double() * num[..., 0] + num[..., 1]
            v = (vb[:, v_at // 2] >> (v_at % 2 * 4).to(torch.uint8) & 15).double() * num[..., 2] + num[..., 3]
            q = s["q"][r:r + n, h * G:(h + 1) * G].double()
            for j in range(G):
                w = (q[:, j] @ k.T) / math.sqrt(D)
                w.masked_fill_(hidden, -math.inf)
                l[:, h * G + j] = torch.logsumexp(w, -1)
                rows[:, h * G + j] = torch.softmax(w, -1) @ v
        out.append(rows)
        lse.append(l)
        r += n
    return {"out": torch.cat(out), "lse": torch.cat(lse) if case["lse"] else None}
