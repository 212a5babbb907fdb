"""Operators of decoding with trees of drafted tokens over the grouped-query cache in 4 bits: cases and plain forms.

  attn_tree  attention of the nodes of a tree of drafted tokens over a paged cache in 4 bits: a node sees the tokens
             before the tree (within a sliding window, if any) and its own ancestors in the tree.
  verify     which drafted tokens the target model accepts, and the token that follows them: from the target's and the
             draft's probabilities and given random numbers, or greedily from the target's logits.
  keep       the accepted tokens of a tree move to the places behind the cache's older tokens; the others go.

A tree's nodes are rows 0, 1, .. of a sequence, a parent before its children; row 0 is the last token that was accepted
before. Its shape stands in one mask per row: bit j says that node j is an ancestor of the row's node or that node itself.

The cache holds, for each token, head and group of channels, an FP16 minimum m, an FP16 scale s and codes 0..15; a code n
stands for m + n s. A page has one region for each kv head: P rows of key codes, P rows of value codes (D/2 bytes each),
then for each token and group the four FP16 numbers (key scale, key minimum, value scale, value minimum).
"""
import math
import random

import torch

own = False


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one user's chat of 1K tokens, eight nodes: latency alone counts
        dict(name="attn_tree_one_1k", op="attn_tree", B=1, lens="same", T=1031, tree=8, rows=8, shape="tree", Hq=32, Hkv=8, D=128,
             group=128, P=64, dtype="bf16", window=0, lse=True, salt=1),
        # a served batch at odd lengths, the usual tree of a drafting head
        dict(name="attn_tree_26_b8", op="attn_tree", B=8, lens="ragged", T=32003, tree=26, rows=26, shape="tree", Hq=32, Hkv=4,
             D=128, group=64, P=128, dtype="bf16", window=0, lse=True, salt=2),
        # one long document, a wide tree
        dict(name="attn_tree_64_long", op="attn_tree", B=1, lens="same", T=65536, tree=64, rows=64, shape="tree", Hq=64, Hkv=8,
             D=128, group=128, P=128, dtype="bf16", window=0, lse=False, salt=3),
        # the drafting model itself as it grows its tree: the newest eight nodes of up to 40, behind a sliding window
        dict(name="attn_tree_level_d64", op="attn_tree", B=16, lens="ragged", T=20011, tree=40, rows=8, shape="tree", Hq=14, Hkv=2,
             D=64, group=64, P=16, dtype="fp16", window=4096, lse=True, salt=4),
        # continuous batching of many short contexts
        dict(name="attn_tree_16_b64", op="attn_tree", B=64, lens="ragged", T=8192, tree=16, rows=16, shape="tree", Hq=32, Hkv=8,
             D=128, group=32, P=64, dtype="fp16", window=0, lse=True, salt=5),
        # one user, four drafted tokens, a small vocabulary
        dict(name="verify_one", op="verify", how="drawn", B=1, rows=5, shape="chain", V=32000, salt=6),
        # a served batch of five drafted tokens each
        dict(name="verify_chain_b64", op="verify", how="drawn", B=64, rows=6, shape="chain", V=102400, salt=7),
        # trees of the draft's most likely tokens, an odd vocabulary
        dict(name="verify_tree_picked", op="verify", how="picked", B=16, rows=32, shape="tree", V=65537, salt=8),
        # greedy decoding of a batch; logits as the last product leaves them
        dict(name="verify_greedy_b32", op="verify", how="greedy", B=32, rows=6, shape="chain", V=150001, dtype="bf16", salt=9),
        # greedy decoding with large trees
        dict(name="verify_greedy_tree", op="verify", how="greedy", B=4, rows=64, shape="tree", V=102400, dtype="fp32", salt=10),
        # a step of a served batch: a few of 26 nodes were accepted
        dict(name="keep_step_b32", op="keep", B=32, T=500, tree=26, most=6, Hkv=8, D=128, group=128, P=64, salt=11),
        # long drafts that were mostly accepted
        dict(name="keep_deep_b64", op="keep", B=64, T=700, tree=250, most=240, Hkv=8, D=128, group=64, P=128, salt=12),
    ]


def _log(rng, lo, hi):
    """A whole number, spread over the logarithm of [lo, hi]."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attn_tree", "attn_tree", "verify", "verify", "keep"])
    c = dict(op=op, salt=rng.randrange(1 << 30))
    if op == "verify":
        c.update(how=rng.choice(["drawn", "picked", "greedy"]), shape=rng.choice(["chain", "tree"]), B=_log(rng, 1, 64))
        c["rows"] = rng.randint(2, 8) if c["shape"] == "chain" else _log(rng, 4, 100)
        c["V"] = min(_log(rng, 500, 200000), 64 * 6 * 102400 // (c["B"] * c["rows"]))
        if c["how"] == "greedy":
            c["dtype"] = rng.choice(["bf16", "fp16", "fp32"])
        return c
    D = rng.choice([64, 128, 128])
    c.update(P=rng.choice([16, 32, 64, 128]), D=D, Hkv=rng.choice([1, 2, 4, 8]), B=_log(rng, 1, 64),
             group=rng.choice([g for g in (32, 64, 128) if g <= D]))
    if op == "keep":
        c["tree"] = _log(rng, 2, 250)
        c["most"] = rng.randint(1, c["tree"])
        c["T"] = c["tree"] + _log(rng, 1, 600)
        return c
    G = rng.choice([1, 2, 4, 5, 7, 8, 12, 16])
    c.update(Hq=c["Hkv"] * G, dtype=rng.choice(["bf16", "fp16"]), lens=rng.choice(["same", "ragged"]), shape=rng.choice(["tree", "tree", "chain"]))
    c["tree"] = _log(rng, 2, 200)
    c["rows"] = rng.choice([c["tree"], c["tree"], rng.randint(1, c["tree"])])
    most = min(65536, 64 * 8192 * 8 * 128 // (c["Hkv"] * D * c["B"]), 64 * 8192 * 32 * 16 // (c["Hq"] * c["rows"] * c["B"]))
    c["T"] = c["tree"] + _log(rng, 1, max(1, most - c["tree"]))
    c["window"] = rng.choice([0, 0, 0, _log(rng, 1, 8192)])
    c["lse"] = rng.random() < 0.5
    return c


def _parents(case, rng, n):
    """Parent of each of a tree's nodes (-1: the root): no node has more than eight children, as a drafting model has its candidates."""
    if case.get("shape") == "chain":
        return [i - 1 for i in range(n)]
    out, count = [-1], [0] * n
    for i in range(1, n):
        p = rng.choice([j for j in range(max(0, i - 10), i) if count[j] < 8])
        count[p] += 1
        out.append(p)
    return out


def _trees(case):
    """Parents of each sequence's tree: part of the case, not of the seed."""
    rng = random.Random(case["salt"])
    n = case["tree"] if case["op"] == "attn_tree" else case["rows"]
    sizes = [n if b == 0 or case.get("lens") != "ragged" else rng.randint(max(1, n // 2), n) for b in range(case["B"])]
    return [_parents(case, rng, k) for k in sizes]


def _masks(parents):
    out = []
    for i, p in enumerate(parents):
        out.append((out[p] if p >= 0 else 0) | 1 << i)
    return out


def _lengths(case, trees):
    """(cached tokens with the tree, rows of queries) of each sequence; the rows are the tree's newest nodes."""
    rng = random.Random(case["salt"] + 1)
    T = case["T"]
    lens = [T if case["lens"] == "same" or b == 0 else rng.randint(max(len(t), T // 16), T) for b, t in enumerate(trees)]
    return lens, [min(case["rows"], len(t)) for t in trees]


def _matching(case, trees):
    """Greedy cases: which nodes carry the token that the target chooses at their parent (at most one child of each)."""
    rng = random.Random(case["salt"] + 2)
    out = []
    for parents in trees:
        taken, flags = set(), []
        for p in parents:
            flag = p >= 0 and p not in taken and rng.random() < 0.7
            if flag:
                taken.add(p)
            flags.append(flag)
        out.append(flags)
    return out


def _kept(case):
    """How many of each tree's nodes stay (the root among them)."""
    rng = random.Random(case["salt"] + 3)
    return [rng.randint(max(1, case["most"] // 2), case["most"]) for _ in range(case["B"])]


def work(case):
    if case["op"] == "verify":
        B, V, trees = case["B"], case["V"], _trees(case)
        rows = sum(len(t) for t in trees)
        if case["how"] == "greedy":  # a row of logits for each node that is reached
            reached = 0
            for parents, flags in zip(trees, _matching(case, trees)):
                on = [True]
                for i in range(1, len(parents)):
                    on.append(on[parents[i]] and flags[i])
                reached += sum(on)
            return {"bytes": reached * V * (4 if case["dtype"] == "fp32" else 2) + rows * 12 + B * case["rows"] * 8, "flops": reached * V}
        arrays = 2 if case["how"] == "drawn" else 1  # a row of each array for each sequence: the one that the new token comes from
        return {"bytes": B * V * 4 * arrays + rows * 16 + B * case["rows"] * 8, "flops": B * V * 4}
    D, Hkv, groups = case["D"], case["Hkv"], case["D"] // case["group"]
    if case["op"] == "keep":
        moved = sum(k - 1 for k in _kept(case))
        return {"bytes": moved * Hkv * (D + 8 * groups) * 2 + sum(_kept(case)) * 4 + case["B"] * 12, "flops": 0}
    trees = _trees(case)
    lens, rows = _lengths(case, trees)
    Hq, w = case["Hq"], case["window"]
    cells = pairs = 0
    for t, T, n in zip(trees, lens, rows):
        base, low = T - len(t), T
        for m in _masks(t)[len(t) - n:]:
            depth = bin(m).count("1")
            lo = max(0, base + depth - w) if w else 0
            low = min(low, lo)
            pairs += max(0, base - lo) + depth
        cells += T - min(low, base)
    return {"bytes": cells * Hkv * (D + 8 * groups) + sum(rows) * Hq * (4 * D + (4 if case["lse"] else 0)) + sum(rows) * 8 * _words(case["tree"]),
            "flops": 4 * D * Hq * pairs}


# ---------------------------------------------------------------- the cache in 4 bits, plainly
def _quantize(x, group):
    """x [..., D] in 32 bits -> codes [..., D] (uint8), scale and minimum [..., D / group] (FP16)."""
    v = x.unflatten(-1, (-1, group))
    m = v.amin(-1).half()
    s = ((v.amax(-1) - m.float()).clamp_min(0) / 15).half()
    step = s.float().unsqueeze(-1)
    codes = torch.where(step > 0, ((v - m.float().unsqueeze(-1)) / step.clamp_min(1e-30)).round().clamp(0, 15), torch.zeros_like(v))
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


def _regions(pool, D, group, P):
    """Views of whole pages [pages, bytes]: key codes, value codes and numbers, each [pages, Hkv, P, bytes of a token]."""
    pages = pool.view(pool.shape[0], -1, _head_bytes(D, group, P))
    return [pages[:, :, a:a + P * w].unflatten(-1, (P, w)) for a, w in ((0, D // 2), (P * D // 2, D // 2), (P * D, 8 * (D // group)))]


# ---------------------------------------------------------------- inputs
def _type(case):
    return {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}[case["dtype"]]


def _ints(v, dev):
    return torch.tensor(v, dtype=torch.int32, device=dev)


def _offsets(sizes, dev):
    out = [0]
    for n in sizes:
        out.append(out[-1] + n)
    return _ints(out, dev)


def _words(n):
    return -(-n // 64)


def _mask_words(masks, words, dev):
    """Masks as rows of 64-bit words, the lowest bits first."""
    signed = lambda x: x - (1 << 64) if x >> 63 else x  # noqa: E731
    return torch.tensor([[signed(m >> (64 * w) & (1 << 64) - 1) for w in range(words)] for m in masks], dtype=torch.int64, device=dev)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed * 7919 + 23)
    randn = lambda *shape: torch.randn(shape, generator=g, device=dev)  # noqa: E731
    s = dict(case=case, err=torch.zeros(1, dtype=torch.int32, device=dev))
    if case["op"] == "verify":
        return _prepare_verify(case, s, g, dev)
    D, Hkv, group, P, B = case["D"], case["Hkv"], case["group"], case["P"], case["B"]
    if case["op"] == "keep":
        rng = random.Random(seed * 31 + case["salt"])
        max_pages = -(-case["T"] // P) + 1
        n_pages = B * max_pages
        s["page_table"] = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32).view(B, max_pages)
        s["pool"] = torch.randint(0, 256, (n_pages, Hkv * _head_bytes(D, group, P)), generator=g, device=dev, dtype=torch.uint8)
        s["base"] = _ints([rng.randint(0, case["T"] - case["tree"]) for _ in range(B)], dev)
        s["lens"] = s["base"] + case["tree"]
        kept = _kept(case)
        rows = [[0] + sorted(rng.sample(range(1, case["tree"]), k - 1)) + [-1] * (case["tree"] - k) for k in kept]
        s["kept"], s["n_kept"] = _ints(rows, dev), _ints(kept, dev)
        return s
    trees = _trees(case)
    lens, rows = _lengths(case, trees)
    max_pages = -(-max(lens) // P) + 1
    n_pages, total, dtype = B * max_pages, sum(rows), _type(case)
    s["page_table"] = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32).view(B, max_pages)
    s["lens"], s["cu"], s["max_rows"] = _ints(lens, dev), _offsets(rows, dev), max(rows)
    s["base"] = _ints([T - len(t) for T, t in zip(lens, trees)], dev)
    s["mask"] = _mask_words([m for t, n in zip(trees, rows) for m in _masks(t)[len(t) - n:]], _words(case["tree"]), dev)
    s["scale"] = 1.0 / math.sqrt(D)
    loud = 1 + 3 * (torch.rand(D, generator=g, device=dev) < 0.05).float()  # the few channels that stand out in keys
    s["q"] = (randn(total, case["Hq"], D) * 1.5).to(dtype)
    s["pool"] = torch.empty(n_pages, Hkv * _head_bytes(D, group, P), dtype=torch.uint8, device=dev)
    at = _regions(s["pool"], D, group, P)
    for k in range(0, n_pages, 4096):
        n = min(4096, n_pages - k)
        kc, ks, km = _quantize(randn(n, Hkv, P, D) * loud, group)
        vc, vs, vm = _quantize(randn(n, Hkv, P, D), group)
        at[0][k:k + n] = _pack(kc, _key_order(D).to(dev))
        at[1][k:k + n] = _pack(vc, _value_order(D).to(dev))
        at[2][k:k + n] = torch.stack([ks, km, vs, vm], -1).contiguous().view(torch.uint8).flatten(-2)
    s["out"] = torch.empty(total, case["Hq"], D, dtype=dtype, device=dev)
    s["lse"] = torch.empty(total, case["Hq"], device=dev) if case["lse"] else None
    return s


def _prepare_verify(case, s, g, dev):
    B, V, trees = case["B"], case["V"], _trees(case)
    n = sum(len(t) for t in trees)
    s["cu"], s["max_rows"] = _offsets([len(t) for t in trees], dev), case["rows"]
    s["mask"] = None if case["shape"] == "chain" else _mask_words([m for t in trees for m in _masks(t)], _words(case["rows"]), dev)
    first, above, nth = 0, [], []  # of each node: the row of its parent (its own for a root), its place among its siblings
    for t in trees:
        seen = {}
        for i, p in enumerate(t):
            above.append(first + max(p, 0))
            nth.append(seen.get(p, 0))
            seen[p] = nth[-1] + 1
        first += len(t)
    above = torch.tensor(above, device=dev)
    logits = torch.randn(n, V, generator=g, device=dev) * 4.5
    out = lambda w: torch.empty(B, w, dtype=torch.int32, device=dev)  # noqa: E731
    s["kept"], s["new"], s["n_kept"] = out(case["rows"]), out(case["rows"]), torch.empty(B, dtype=torch.int32, device=dev)
    if case["how"] == "greedy":
        s["target"] = logits.to(_type(case))
        best = _first_best(s["target"].float())
        other = torch.randint(0, V, (n,), generator=g, device=dev)
        match = torch.tensor([f for t in _matching(case, trees) for f in t], device=dev)
        s["tokens"] = torch.where(match, best[above], torch.where(other == best[above], (other + 1) % V, other)).to(torch.int32)
        return s
    s["target"] = torch.softmax(logits, -1)
    logits += torch.randn(n, V, generator=g, device=dev) * 0.7
    if case["how"] == "drawn":
        s["draft"] = torch.softmax(logits, -1)
        race = torch.empty(V, device=dev)
        tokens = [(s["draft"][r] / race.exponential_(generator=g)).argmax() for r in above.tolist()]
        s["tokens"] = torch.stack(tokens).to(torch.int32)
    else:
        s["draft"] = None
        top = logits.topk(min(9, V), -1).indices
        s["tokens"] = top[above, torch.tensor(nth, device=dev)].to(torch.int32)
    s["u_accept"] = torch.rand(n, generator=g, device=dev)
    s["u_sample"] = torch.rand(B, generator=g, device=dev)
    return s


# ---------------------------------------------------------------- one pass
def run(state):
    case = state["case"]
    if own:
        return _own(state, case)
    if case["op"] == "attn_tree":
        return _attn_tree(state, case)
    if case["op"] == "keep":
        return _keep(state, case)
    return _greedy(state, case) if case["how"] == "greedy" else _sampled(state, case)


def _own(s, case):
    import bit_mla_kv_qcache_gb300 as fw
    if case["op"] == "verify":
        if case["how"] == "greedy":
            fw.mla_qcache_verify_greedy(s["target"], s["tokens"], s["cu"], s["max_rows"], s["kept"], s["new"], s["n_kept"], s["err"],
                                        tree_mask=s["mask"])
        else:
            fw.mla_qcache_verify_sampled(s["target"], s["tokens"], s["cu"], s["max_rows"], s["u_accept"], s["u_sample"], s["kept"],
                                         s["new"], s["n_kept"], s["err"], draft_probs=s["draft"], tree_mask=s["mask"])
        return {"kept": s["kept"], "new": s["new"], "n_kept": s["n_kept"]}
    if "cfg" not in s:
        s["cfg"] = fw.make_kv4_config(case["Hkv"], case["D"], group=case["group"], page_size=case["P"])
    if case["op"] == "keep":
        fw.mla_qcache_kv4_keep(s["cfg"], s["kept"], s["n_kept"], s["base"], s["page_table"], s["pool"], s["lens"], s["err"])
        return {"pool": s["pool"], "lens": s["lens"]}
    if "ws" not in s:  # kept by the program, zeroed once
        need = fw.kv4_workspace_bytes(s["cfg"], case["B"], case["Hq"], s["max_rows"], s["page_table"].shape[1])
        s["ws"] = torch.zeros(need, dtype=torch.uint8, device=s["q"].device)
    fw.mla_qcache_kv4_attn_tree(s["cfg"], s["q"], s["mask"], s["cu"], s["max_rows"], s["page_table"], s["lens"], s["pool"], s["scale"],
                                s["out"], s["ws"], s["err"], tree_base=s["base"], lse=s["lse"], window=case["window"])
    return {"out": s["out"], "lse": s["lse"]}


def _rows(s, n):
    """Sequence and place in it of each of n rows."""
    cu, r = s["cu"].long(), torch.arange(n, device=s["cu"].device)
    b = torch.searchsorted(cu, r, right=True) - 1
    return b, r - cu[b]


def _bits(mask):
    """[rows, words] -> [rows, 64 words] truth values."""
    at = torch.arange(64, device=mask.device)
    return ((mask.unsqueeze(-1) >> at) & 1).flatten(-2).bool()


def _attn_tree(s, case):
    B, D, P, group, Hq, Hkv = (case[x] for x in ("B", "D", "P", "group", "Hq", "Hkv"))
    G, dev, n = Hq // Hkv, s["q"].device, s["max_rows"]
    table = s["page_table"].long()
    kc, vc, num = (x[table].transpose(1, 2).flatten(2, 3) for x in _regions(s["pool"], D, group, P))  # [B, Hkv, T, bytes]
    num = num.contiguous().view(torch.float16).unflatten(-1, (D // group, 4))
    k = _values(_unpack(kc, _key_order(D).to(dev)), num[..., 0], num[..., 1], group)
    v = _values(_unpack(vc, _value_order(D).to(dev)), num[..., 2], num[..., 3], group)
    b, i = _rows(s, s["q"].shape[0])
    q = torch.zeros(B, n, Hq, D, device=dev)
    q[b, i] = s["q"].float()
    q = q.view(B, n, Hkv, G, D).permute(0, 2, 3, 1, 4).flatten(2, 3)  # [B, Hkv, G n, D]
    bits = torch.zeros(B, n, 64 * s["mask"].shape[1], dtype=torch.bool, device=dev)
    bits[b, i] = _bits(s["mask"])
    t, base, T = torch.arange(k.shape[2], device=dev), s["base"].long(), s["lens"].long()
    node = t - base[:, None]  # [B, tokens] the tree's node that a token is
    ancestor = bits.gather(2, node.clamp(0, bits.shape[2] - 1)[:, None].expand(B, n, -1))
    seen = torch.where((node < 0)[:, None], torch.ones_like(ancestor), ancestor & (t < T[:, None])[:, None] & (node < bits.shape[2])[:, None])
    if case["window"]:  # a node's position: as many tokens behind the base as it has ancestors
        pos = base[:, None] + bits.sum(-1) - 1
        seen &= (node >= 0)[:, None] | (t > pos[..., None] - case["window"])
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


def _keep(s, case):
    kept, count, base = s["kept"].long(), s["n_kept"].long(), s["base"].long()
    place = torch.arange(kept.shape[1], device=kept.device).expand_as(kept)
    stays = place < count[:, None]
    here = base[:, None] + torch.where(stays, kept, torch.zeros_like(kept))  # the root where there is nothing to move
    to = base[:, None] + torch.where(stays, place, torch.zeros_like(kept))
    table, P = s["page_table"].long(), case["P"]
    for x in _regions(s["pool"], case["D"], case["group"], P):
        x[table.gather(1, to // P), :, to % P] = x[table.gather(1, here // P), :, here % P]
    return {"pool": s["pool"], "lens": (base + count).to(torch.int32)}


def _walk(s):
    """Local parent [B, rows], tokens [B, rows] (-1 behind a sequence's last), row of each sequence's root, rows of each."""
    B, n, dev = s["n_kept"].shape[0], s["max_rows"], s["tokens"].device
    b, i = _rows(s, s["tokens"].shape[0])
    parent = torch.full((B, n), -2, device=dev)
    if s["mask"] is None:
        parent[b, i] = i - 1
    else:
        bits, j = _bits(s["mask"]), torch.arange(64 * s["mask"].shape[1], device=dev)
        parent[b, i] = torch.where(bits & (j < i[:, None]), j, torch.full_like(bits, -1, dtype=torch.int64)).amax(-1)
    tokens = torch.full((B, n), -1, device=dev)
    tokens[b, i] = s["tokens"].long()
    return parent, tokens, s["cu"][:-1].long()


def _answer(kept, new, count):
    return {"kept": kept.to(torch.int32), "new": new.to(torch.int32), "n_kept": count.to(torch.int32)}


def _first_best(x):
    """Lowest index of the largest value of each row."""
    at = torch.arange(x.shape[-1], device=x.device)
    return torch.where(x == x.amax(-1, keepdim=True), at, torch.full_like(at, x.shape[-1])).amin(-1)


def _greedy(s, case):
    parent, tokens, root = _walk(s)
    B, n = parent.shape
    every = torch.arange(B, device=root.device)
    best = _first_best(s["target"].float())
    at, count = torch.zeros_like(root), torch.ones_like(root)
    kept, new = torch.full_like(parent, -1), torch.full_like(parent, -1)
    kept[:, 0] = 0
    for i in range(1, n):  # a parent comes before its children
        on = (parent[:, i] == at) & (tokens[:, i] == best[root + at])
        kept[every, count.clamp_max(n - 1)] = torch.where(on, torch.full_like(at, i), kept[every, count.clamp_max(n - 1)])
        new[every, count - 1] = torch.where(on, tokens[:, i], new[every, count - 1])
        at = torch.where(on, torch.full_like(at, i), at)
        count = count + on
    new[every, count - 1] = best[root + at]
    return _answer(kept, new, count)


def _sampled(s, case):
    """In 64 bits: what is left of a node's probabilities after k rejections is max(p - c_k q, 0) with c_0 = 0, Z_0 = 1 and
    c_(k+1) = c_k + Z_k, Z_k the sum of what is left; a child x is accepted where u q(x) Z_k < max(p(x) - c_k q(x), 0). Drafts
    that were picked without chance have q(x) = 1 at their token alone: a rejected one's probability goes."""
    parent, tokens, root = _walk(s)
    B, n, V, drawn = *parent.shape, case["V"], s["draft"] is not None
    every = torch.arange(B, device=root.device)
    at, count = torch.zeros_like(root), torch.ones_like(root)
    kept, new = torch.full_like(parent, -1), torch.full_like(parent, -1)
    kept[:, 0] = 0
    zero = torch.zeros(B, dtype=torch.float64, device=root.device)
    c, Z = zero, zero + 1
    gone = None if drawn else torch.zeros(B, V, dtype=torch.bool, device=root.device)

    def left():
        p = s["target"][root + at].double()
        return (p - c[:, None] * s["draft"][root + at].double()).clamp_min(0) if drawn else p.masked_fill(gone, 0)

    for i in range(1, n):
        x = tokens[:, i]
        child = (parent[:, i] == at) & (x >= 0) & (x < V)
        xx = x.clamp(0, V - 1)
        px, u = s["target"][root + at, xx].double(), s["u_accept"][(root + i).clamp_max(s["u_accept"].shape[0] - 1)].double()
        if drawn:
            qx = s["draft"][root + at, xx].double()
            on = child & (u * qx * Z < (px - c * qx).clamp_min(0))
        else:
            px = torch.where(gone[every, xx], zero, px)
            on = child & (u * Z < px)
        off = child & ~on
        kept[every, count.clamp_max(n - 1)] = torch.where(on, torch.full_like(at, i), kept[every, count.clamp_max(n - 1)])
        new[every, count - 1] = torch.where(on, x, new[every, count - 1])
        if drawn:
            c = torch.where(off, c + Z, c)
            Z = torch.where(off, left().sum(-1), Z)
            c = torch.where(on, zero, c)
        else:
            Z = torch.where(off, Z - px, Z)
            gone[every, xx] |= off
            gone &= ~on[:, None]
        Z = torch.where(on, zero + 1, Z)
        at = torch.where(on, torch.full_like(at, i), at)
        count = count + on
    rest = left()
    rest = torch.where((rest.sum(-1, keepdim=True) > 0), rest, s["target"][root + at].double())
    upto = rest.cumsum(-1)
    token = (upto <= (s["u_sample"].double() * upto[:, -1])[:, None]).sum(-1)
    last = torch.where(rest > 0, torch.arange(V, device=root.device), torch.full_like(at[:1], -1)).amax(-1)
    new[every, count - 1] = torch.minimum(token, last)
    return _answer(kept, new, count)


# ---------------------------------------------------------------- in 64 bits, from the definitions
def exact(case, seed):
    if case["op"] != "attn_tree":  # whole numbers
        return None
    s = prepare(case, seed)
    trees = _trees(case)
    lens, rows = _lengths(case, trees)
    D, P, group, G = case["D"], case["P"], case["group"], case["Hq"] // case["Hkv"]
    head, dev = _head_bytes(D, group, P), s["q"].device
    ch = torch.arange(D, device=dev)
    # nibble that holds channel c: keys in words (4 lanes x 32-channel blocks), values in words (8 lanes x 64-channel blocks)
    k_at = (ch % 32 // 8) * (D // 32) * 8 + ch // 32 * 8 + ch % 8
    v_at = (ch % 8) * (D // 64) * 8 + ch // 64 * 8 + ch // 8 % 2 * 4 + ch // 16 % 4
    out, lse, r = [], [], 0
    for b, (parents, T, n) in enumerate(zip(trees, lens, rows)):
        base, first = T - len(parents), len(parents) - n
        hidden = torch.zeros(n, T, dtype=torch.bool)
        for i in range(n):
            hidden[i, base:] = True
            j, depth = first + i, 0
            while j >= 0:  # up to the root
                hidden[i, base + j] = False
                j, depth = parents[j], depth + 1
            if case["window"]:
                hidden[i, :max(0, min(base, base + depth - case["window"]))] = True
        hidden = hidden.to(dev).repeat_interleave(G, 0)
        page = s["page_table"][b, :-(-T // P)].long()
        o = torch.empty(n, case["Hq"], D, dtype=torch.float64, device=dev)
        l = torch.empty(n, case["Hq"], dtype=torch.float64, device=dev)
        for h in range(case["Hkv"]):
            region = s["pool"][page, h * head:(h + 1) * head]
            num = region[:, P * D:].contiguous().view(torch.float16).double().view(-1, D // group, 4)[:T].repeat_interleave(group, 1)
            kb, vb = region[:, :P * D // 2].reshape(-1, D // 2)[:T], region[:, P * D // 2:P * D].reshape(-1, D // 2)[:T]
            k = (kb[:, k_at // 2] >> (k_at % 2 * 4).to(torch.uint8) & 15).double() * num[..., 0] + num[..., 1]
            v = (vb[:, v_at // 2] >> (v_at % 2 * 4).to(torch.uint8) & 15).double() * num[..., 2] + num[..., 3]
            w = (s["q"][r:r + n, h * G:(h + 1) * G].double().reshape(n * G, D) @ k.T) / math.sqrt(D)
            w.masked_fill_(hidden, -math.inf)
            l[:, h * G:(h + 1) * G] = torch.logsumexp(w, -1).view(n, G)
            o[:, h * G:(h + 1) * G] = (torch.softmax(w, -1) @ v).view(n, G, D)
        out.append(o)
        lse.append(l)
        r += n
    return {"out": torch.cat(out), "lse": torch.cat(lse) if case["lse"] else None}
