"""One round of decoding by a tree of drafted tokens over the 8-bit key/value cache: the cases of its
operators, their plain forms and exact values.

A sequence has ``counts`` [B] nodes (none given: n): node 0 is the token already decided, the others
are drafts, each with a parent of a lower number (``parents`` [B, n], -1 for node 0).  The cache is
that of ``perf/operators.py``; its ``lengths`` count the nodes, which lie at its end.

    mask     words of the nodes that each node sees, itself and its ancestors (attn_tree_mask)
    attend   attention of grouped query heads over the cache: a node sees every token before the
             tree and the nodes of its words (attn_fwd_kv8_tree)
    verify   which nodes the target's probabilities accept, and the token after them, from given
             random numbers (attn_draft_verify)
    keep     moves the accepted nodes' keys and values next to the tokens before the tree, each
             block with a scale of its own again (attn_kv8_keep)
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
F8 = torch.float8_e4m3fn


def listed():
    return [
        # The smallest tree: one conversation's next few tokens.
        dict(name="mask_one", op="mask", B=1, n=16, width=2, ragged=False, salt=21),
        # Wide trees of a large batch, some smaller than others.
        dict(name="mask_batch", op="mask", B=128, n=256, width=40, ragged=True, salt=22),
        # The smallest call: one conversation just begun on a small model, a handful of drafts.
        dict(name="attend_first", op="attend", dtype="f16", B=1, G=1, Hk=8, d=64, block=32, n=8, width=2,
             lo=257, hi=257, cap=512, ragged=False, salt=23),
        # A batch whose drafts are few: a token and three guesses after it.
        dict(name="attend_guesses", op="attend", dtype="bf16", B=16, G=4, Hk=8, d=128, block=64, n=4, width=3,
             lo=2000, hi=8192, cap=8192, ragged=False, salt=24),
        # A batch of trees, each sequence with as many nodes as its draft gave.
        dict(name="attend_batch", op="attend", dtype="bf16", B=16, G=8, Hk=8, d=128, block=32, n=26, width=8,
             lo=4001, hi=8191, cap=8192, ragged=True, salt=25),
        # Two long documents being answered, 64 nodes each.
        dict(name="attend_long", op="attend", dtype="bf16", B=2, G=4, Hk=8, d=128, block=128, n=64, width=10,
             lo=120001, hi=131072, cap=131072, ragged=False, salt=26),
        # Wide trees on a small model.
        dict(name="attend_wide", op="attend", dtype="f16", B=4, G=4, Hk=8, d=64, block=64, n=256, width=60,
             lo=12000, hi=16384, cap=16384, ragged=True, salt=27),
        # A chain of five drafts of one conversation, over a small vocabulary.
        dict(name="verify_chain", op="verify", dtype="f32", B=1, n=6, width=0, V=32768, drawn=True,
             ragged=False, salt=28),
        # Trees of a batch, drawn from a draft's probabilities, over a large vocabulary.
        dict(name="verify_batch", op="verify", dtype="f32", B=32, n=32, width=6, V=131072, drawn=True,
             ragged=True, salt=29),
        # Drafts that were looked up, not drawn: they have no probabilities of their own.
        dict(name="verify_looked_up", op="verify", dtype="bf16", B=64, n=16, width=3, V=100003, drawn=False,
             ragged=True, salt=30),
        # The batch of trees above brought to what was accepted of it.
        dict(name="keep_batch", op="keep", B=16, Hk=8, d=128, block=32, n=26, width=8, lo=4001, hi=8191,
             cap=8192, ragged=True, salt=31),
        # Every head with a cache of its own, trees of 256 nodes.
        dict(name="keep_heads", op="keep", B=32, Hk=16, d=128, block=64, n=256, width=20, lo=2000, hi=4096,
             cap=4096, ragged=True, salt=32),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["mask", "attend", "attend", "attend", "verify", "verify", "keep"])
    c = dict(op=op, salt=rng.randrange(1 << 30))
    d, block = rng.choice([64, 128, 128]), rng.choice([16, 32, 64, 128])
    Hk, G = rng.choice([1, 2, 4, 8, 16]), rng.choice([1, 2, 3, 4, 5, 8, 12])
    c["n"] = rng.choice([1, 2, rng.randint(3, 9), _log(rng, 10, 64), _log(rng, 16, 256)])
    c["width"] = rng.choice([0, 1, 2, rng.randint(1, c["n"])])
    # No more than the largest listed cases have: probabilities, codes, and scores of the heads.
    if op == "mask":
        c.update(B=_log(rng, 1, 128), n=_log(rng, 10, 256), width=rng.randint(2, 60))
    elif op == "verify":
        c["dtype"], c["drawn"] = rng.choice(["f32", "f32", "bf16", "f16"]), rng.random() < 0.7
        c["n"], c["V"] = min(c["n"], 32), _log(rng, 1000, 160000)
        c["B"] = min((1 << 27) // (c["n"] * c["V"]), _log(rng, 1, 64))
    else:
        c.update(Hk=Hk, d=d, block=block)
        most = min(131072 if op == "attend" else 16384, (1 << 28) // (Hk * d))
        if op == "attend":
            c.update(dtype=rng.choice(["bf16", "bf16", "f16"]), G=G)
            most = min(most, (1 << 29) // (Hk * G * c["n"]))
        hi = _log(rng, max(c["n"], 64), most // block * block)
        c.update(lo=max(c["n"], int(hi * rng.choice([0.25, 0.6, 1.0]))), hi=hi, cap=-(-hi // block) * block)
        most = (1 << 28) // (Hk * c["cap"] * d)
        if op == "attend":
            most = min(most, (1 << 29) // (Hk * G * c["n"] * c["cap"]))
        c["B"] = min(most, _log(rng, 1, 64))
    c["ragged"] = c["n"] > 1 and rng.random() < 0.5
    return c


def _trees(case):
    """Lengths, counts, parents and one path for each sequence: whole numbers, by the case alone.  The
    path is a leaf's: the nodes down to it, as if they were accepted."""
    r, n = random.Random(case["salt"]), case["n"]
    lens = [r.randint(case.get("lo", n), case.get("hi", n)) for _ in range(case["B"])]
    counts = [r.randint(max(1, n // 2), n) if case.get("ragged") else n for _ in lens]
    parents = [[-1] + [max(0, i - 1 - r.randint(0, case["width"])) for i in range(1, n)] for _ in lens]
    paths = []
    for cnt, up in zip(counts, parents):
        path = [r.randrange(cnt)]
        while path[0] > 0:
            path.insert(0, up[path[0]])
        paths.append(path)
    return lens, counts, parents, paths


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _scale(amax):
    """Least power of two s with amax <= 448 s, between 2^-100 and 2^120."""
    m, e = torch.frexp(amax)
    e = torch.where(m > 0.875, e - 8, e - 9)
    e = torch.where(amax > 0, e, torch.full_like(e, -100)).clamp(-100, 120)
    return torch.ldexp(torch.ones_like(amax), e)


def _codes(x):
    """E4M3 codes of values already divided by their scale."""
    x = torch.where(x.isfinite(), x.clamp(-448.0, 448.0), torch.full_like(x, float("nan")))
    return x.to(F8)


def _cache(B, Hk, cap, d, block, gen):
    """Codes and scales of a cache whose channels differ in size, as keys' do."""
    chan = torch.exp(0.5 * torch.randn(1, Hk, 1, d, generator=gen, device="cuda"))
    x = torch.randn(B, Hk, cap, d, generator=gen, device="cuda", dtype=torch.float32)
    x = (x * chan).view(B, Hk, cap // block, block * d)
    s = _scale(x.abs().amax(-1))
    return _codes(x / s[..., None]).view(B, Hk, cap, d), s


def _words(parents, counts, n):
    """Words [B, n, ceil(n / 32)] of each node and its ancestors (rows from counts on: none)."""
    rows = []
    for up, cnt in zip(parents, counts):
        sees = []
        for i in range(n):
            sees.append((1 << i | (sees[up[i]] if up[i] >= 0 else 0)) if i < cnt else 0)
        rows.append([[(s >> 32 * w & 0xFFFFFFFF) - ((s >> 32 * w & 0x80000000) << 1)
                      for w in range(-(-n // 32))] for s in sees])
    return _ints(rows)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(1000003 * seed + case["salt"] % 1000003)
    op, B, n = case["op"], case["B"], case["n"]
    lens, counts, parents, paths = _trees(case)
    st = dict(case=case, counts=_ints(counts) if case.get("ragged") else None)
    if op == "mask":
        back = torch.randint(0, case["width"] + 1, (B, n), generator=gen, device="cuda")
        parents = (torch.arange(n, device="cuda") - 1 - back).clamp(min=0)
        parents[:, 0] = -1
        st["parents"] = parents.to(torch.int32)
        return st
    if op == "verify":
        dt, V = DTYPES[case["dtype"]], case["V"]
        st["parents"] = _ints(parents)
        # Logits whose largest few hold most of the mass; the draft's are near the target's.
        x = torch.randn(B, n, V, generator=gen, device="cuda")
        x.abs_().pow_(1.5).mul_(2.5)
        st["target"] = torch.softmax(x, -1).to(dt)
        x += 0.7 * torch.randn(B, n, V, generator=gen, device="cuda")
        x = torch.softmax(x, -1)
        up = st["parents"].long().clamp(min=0)
        # Node i's token, drawn from the draft's probabilities after its parent.
        cum = x.double().cumsum(-1)
        u = torch.rand(B, n, 1, generator=gen, device="cuda", dtype=torch.float64)
        rows = torch.arange(B, device="cuda")[:, None]
        st["tokens"] = torch.searchsorted(cum[rows, up], u).clamp(max=V - 1)[..., 0].to(torch.int32)
        st["draft"] = x.to(dt) if case["drawn"] else None
        st["uniforms"] = torch.rand(B, n, generator=gen, device="cuda")
        return st
    Hk, d, block, cap = (case[k] for k in ("Hk", "d", "block", "cap"))
    st.update(lengths=_ints(lens), block=block)
    st["k8"], st["ks"] = _cache(B, Hk, cap, d, block, gen)
    st["v8"], st["vs"] = _cache(B, Hk, cap, d, block, gen)
    if op == "attend":
        st["tree"] = _words(parents, counts, n)
        st["q"] = torch.randn(B, Hk * case["G"], n, d, generator=gen, device="cuda").to(DTYPES[case["dtype"]])
        st["c"] = d ** -0.5
        return st
    st["path"] = _ints([p + [-1] * (n - len(p)) for p in paths])
    st["accepted"] = _ints([len(p) for p in paths])
    st["w"] = torch.rand(B, Hk, cap, generator=gen, device="cuda")
    return st


def run(st):
    return _own(st) if own else _plain(st)


# ------------------------------------------------------------------ the framework's operators

def _own(st):
    import exact_io_aware_gb300 as ea

    op = st["case"]["op"]
    if op == "mask":
        return ea.attn_tree_mask(st["parents"], counts=st["counts"])
    if op == "attend":
        return ea.attn_fwd_kv8_tree(st["q"], st["k8"], st["v8"], st["ks"], st["vs"], st["lengths"],
                                    st["tree"], st["c"], counts=st["counts"])
    if op == "verify":
        return ea.attn_draft_verify(st["target"], st["draft"], st["tokens"], st["parents"], st["uniforms"],
                                    counts=st["counts"])
    lengths = ea.attn_kv8_keep(st["k8"], st["v8"], st["ks"], st["vs"], st["lengths"], st["path"],
                               st["accepted"], counts=st["counts"], weights=st["w"])
    return st["k8"], st["v8"], st["ks"], st["vs"], st["w"], lengths


# ------------------------------------------------------------------ the plain form

def _plain(st):
    return {"mask": _mask, "attend": _attend, "verify": _verify, "keep": _keep}[st["case"]["op"]](st)


def _mask(st):
    B, n = st["parents"].shape
    dev = st["parents"].device
    j = torch.arange(n, device=dev)
    sees = ((st["parents"][..., None] == j) | (j[:, None] == j)).float()
    # Steps to a parent, then to a grandparent, then four up: a product doubles the reach.
    reach = 1
    while reach < n:
        sees = ((sees @ sees) > 0).float()
        reach *= 2
    if st["counts"] is not None:
        sees = sees * (j < st["counts"][:, None])[..., None]
    words = -(-n // 32)
    bits = torch.zeros(B, n, 32 * words, dtype=torch.int64, device=dev)
    bits[..., :n] = sees.long()
    value = (bits.view(B, n, words, 32) << torch.arange(32, device=dev)).sum(-1)
    return torch.where(value >= 1 << 31, value - (1 << 32), value).to(torch.int32)


def _values(codes, scales, block):
    B, Hk, cap, d = codes.shape
    x = codes.float().view(B, Hk, cap // block, block * d) * scales[..., None]
    return x.view(B, Hk, cap, d)


def _seen(st):
    """[B, n, cap]: keys each node sees."""
    n, cap, dev = st["q"].shape[2], st["k8"].shape[2], st["q"].device
    lens = st["lengths"].long()
    cnt = torch.full_like(lens, n) if st["counts"] is None else st["counts"].long()
    i, j = torch.arange(n, device=dev), torch.arange(cap, device=dev)
    node = j - (lens - cnt)[:, None]                                      # [B, cap]
    at = node.clamp(0, n - 1)
    word = st["tree"].gather(2, (at // 32)[:, None].expand(-1, n, -1))
    bit = (word >> (at % 32)[:, None].to(torch.int32)) & 1
    inside = (j < lens[:, None])[:, None]
    return inside & (i < cnt[:, None])[..., None] & ((node < 0)[:, None] | (bit == 1))


def _attend(st):
    B, H, n, d = st["q"].shape
    Hk, cap = st["k8"].shape[1:3]
    q = st["q"].float().view(B, Hk, H // Hk, n, d)
    k = _values(st["k8"], st["ks"], st["block"])
    s = (q.reshape(B, Hk, -1, d) @ k.transpose(2, 3)).view(B, Hk, H // Hk, n, cap) * st["c"]
    s = s.masked_fill(~_seen(st)[:, None, None], float("-inf"))
    m = s.amax(-1, keepdim=True)
    m = torch.where(m.isfinite(), m, torch.zeros_like(m))
    p = (s - m).exp_()
    l = p.sum(-1, keepdim=True)
    v = _values(st["v8"], st["vs"], st["block"])
    o = (p.view(B, Hk, -1, cap) @ v).view(B, Hk, H // Hk, n, d) / torch.where(l > 0, l, 1.0)
    return o.reshape(B, H, n, d).to(st["q"].dtype), (m + l.log()).reshape(B, H, n)


def _verify(st):
    """At node a, with p and q the target's and the draft's probabilities after it, the residual that a
    refusal leaves is max(p - S q, 0) of mass W (S the sum of the masses before it, W = 1 at first): a
    child x is accepted if u q(x) W is below its residual.  Where the drafts were not drawn, q(x)
    is 1 and a refused token leaves the residual.  In 64 bits: decisions next to a border."""
    target, draft, tokens = st["target"], st["draft"], st["tokens"].long()
    B, n, V = target.shape
    dev = target.device
    cnt = torch.full((B,), n, device=dev) if st["counts"] is None else st["counts"].long()
    u, up, b = st["uniforms"].double(), st["parents"].long(), torch.arange(B, device=dev)
    node = torch.zeros(B, dtype=torch.long, device=dev)
    S, W = torch.zeros(B, dtype=torch.float64, device=dev), torch.ones(B, dtype=torch.float64, device=dev)
    gone = torch.zeros(B, V, dtype=torch.bool, device=dev)  # refused tokens of drafts that were not drawn
    accept = torch.zeros(B, n, dtype=torch.bool, device=dev)
    accept[:, 0] = cnt > 0

    def residual():
        r = target[b, node].double()
        if draft is None:
            return torch.where(gone, 0.0, r)
        return (r - S[:, None] * draft[b, node].double()).clamp(min=0.0)

    # Each node's fate hangs on those before it; children come after their parents.
    for i in range(1, n):
        x = tokens[:, i]
        asked = (up[:, i] == node) & (i < cnt)
        p = target[b, node, x].double()
        if draft is None:
            r = torch.where(gone[b, x], 0.0, p)
            yes = asked & (u[:, i] * W < r)
            no = asked & ~yes
            W = torch.where(no, W - r, W)
            gone[b, x] |= no
            gone &= ~yes[:, None]
        else:
            q = draft[b, node, x].double()
            yes = asked & (u[:, i] * q * W < (p - S * q).clamp(min=0.0))
            no = asked & ~yes
            before = S
            S = torch.where(no, S + W, S)
            mass = residual().sum(-1)
            left = mass > 0
            W = torch.where(no & left, mass, W)
            S = torch.where(no & ~left, before, S)
        node = torch.where(yes, i, node)
        S, W = torch.where(yes, 0.0, S), torch.where(yes, 1.0, W)
        accept[:, i] = yes
    cum = residual().cumsum(-1)
    above = cum > u[:, :1] * cum[:, -1:]
    token = torch.where(above.any(-1) & (cnt > 0), above.long().argmax(-1), -1)
    order = torch.where(accept, torch.arange(n, device=dev), n).sort(-1).values
    path = torch.where(order < n, order, -1)
    return path.to(torch.int32), accept.sum(-1).to(torch.int32), token.to(torch.int32)


def _keep(st):
    B, Hk, cap, d = st["k8"].shape
    block, dev = st["block"], st["k8"].device
    n = st["path"].shape[1]
    lens, acc = st["lengths"].long(), st["accepted"].long()
    cnt = torch.full_like(lens, n) if st["counts"] is None else st["counts"].long()
    first = lens - cnt
    # A window of whole blocks around the tree's places, inside the cache.
    size = min(cap, (n + block - 1) // block * block + block)
    w0 = torch.clamp(first // block * block, max=cap - size)
    pos = w0[:, None] + torch.arange(size, device=dev)                    # [B, size]
    new = (pos >= first[:, None]) & (pos < (first + acc)[:, None])
    held = pos < first[:, None]
    node = st["path"].long().gather(1, (pos - first[:, None]).clamp(0, n - 1))
    src = torch.where(new, first[:, None] + node, pos)
    b, h = torch.arange(B, device=dev)[:, None, None], torch.arange(Hk, device=dev)[None, :, None]
    at, come = (b, h, pos[:, None, :]), (b, h, src[:, None, :])
    st["w"][at] = st["w"][come]
    for codes, scales in ((st["k8"], st["ks"]), (st["v8"], st["vs"])):
        blk = (b, h, (pos[:, ::block] // block)[:, None, :])
        old = scales[blk]                                                 # [B, Hk, size / block]
        x = codes[come].float() * scales[b, h, (src // block)[:, None, :]][..., None]
        cut = lambda m: m.view(B, 1, size // block, block)
        fin = torch.where(x.isfinite(), x.abs(), torch.zeros_like(x)).amax(-1)
        amax = torch.where(cut(new), fin.view(B, Hk, size // block, block), torch.zeros((), device=dev))
        need = _scale(amax.amax(-1))
        holds, takes = cut(held).any(-1), cut(new).any(-1)
        s = torch.where(takes, torch.where(holds, torch.maximum(old, need), need), old)
        each = lambda t: t.repeat_interleave(block, -1)[..., None]
        was = codes[at].float()
        moved = torch.where(held[:, None, :, None] & (each(s) > each(old)), _codes(was * each(old / s)).float(), was)
        codes[at] = torch.where(new[:, None, :, None], _codes(x / each(s)).float(), moved).to(F8)
        scales[blk] = s
    return st["k8"], st["v8"], st["ks"], st["vs"], st["w"], (first + acc).to(torch.int32)


# ------------------------------------------------------------------ what a pass cannot do without

def _depths(up, cnt):
    deep = []
    for i in range(cnt):
        deep.append(1 + (deep[up[i]] if up[i] >= 0 else 0))
    return deep


def work(case):
    lens, counts, parents, paths = _trees(case)
    B, n = case["B"], case["n"]
    words = -(-n // 32)
    if case["op"] == "mask":
        return {"bytes": B * n * (4 + 4 * words), "flops": B * n}
    if case["op"] == "verify":
        # One row of the target's probabilities, where the last token comes from; of drawn drafts the
        # draft's too, as a refusal needs it.
        size = 4 if case["dtype"] == "f32" else 2
        rows = 2 if case["drawn"] else 1
        nodes = sum(counts)
        return {"bytes": B * case["V"] * size * rows + nodes * (12 + size * rows) + B * (4 * n + 8),
                "flops": 3 * rows * B * case["V"]}
    Hk, d, block = case["Hk"], case["d"], case["block"]
    blocks = lambda m: -(-m // block)
    if case["op"] == "keep":
        # Of the accepted nodes only those that change their place move.
        moved = Hk * sum(sum(i != node for i, node in enumerate(p)) for p in paths)
        scales = Hk * sum(blocks(len(p)) for p in paths)
        return {"bytes": moved * (4 * d + 8) + 16 * scales + 4 * sum(len(p) for p in paths) + 16 * B,
                "flops": 4 * moved * d}
    H = Hk * case["G"]
    pairs = H * sum(c * (m - c) + sum(_depths(up, c)) for m, c, up in zip(lens, counts, parents))
    rows = H * sum(counts)
    return {"bytes": 2 * Hk * d * sum(lens) + 8 * Hk * sum(blocks(m) for m in lens) + rows * (4 * d + 4)
            + 4 * words * sum(counts) + 8 * B, "flops": 4 * d * pairs}


# ------------------------------------------------------------------ exact values, in 64 bits

def exact(case, seed):
    if case["op"] in ("mask", "verify"):
        return None  # whole numbers
    lens, counts, parents, paths = _trees(case)
    B, Hk, d, block, n = (case[k] for k in ("B", "Hk", "d", "block", "n"))
    if case["op"] == "keep":
        if Hk * sum(len(p) for p in paths) > 16384:
            return None  # token by token this takes too long
        return _exact_keep(prepare(case, seed), lens, counts, paths, block)
    H = Hk * case["G"]
    if H * n * sum(lens) > 1 << 31:
        return None
    st = prepare(case, seed)
    o = torch.zeros(B, H, n, d, dtype=torch.float64, device="cuda")
    lse = torch.full((B, H, n), float("-inf"), dtype=torch.float64, device="cuda")
    per = lambda t, b, hk, m: t[b, hk].double().repeat_interleave(block)[:m, None]
    for b, (m, cnt, up) in enumerate(zip(lens, counts, parents)):
        sees = torch.zeros(cnt, m, dtype=torch.bool)
        sees[:, :m - cnt] = True
        for i in range(cnt):
            a = i
            while a >= 0:
                sees[i, m - cnt + a] = True
                a = up[a]
        sees = sees.cuda()
        for hk in range(Hk):
            heads = slice(hk * case["G"], (hk + 1) * case["G"])
            k = st["k8"][b, hk, :m].double() * per(st["ks"], b, hk, m)
            s = torch.einsum("gid,jd->gij", st["q"][b, heads, :cnt].double(), k) * d ** -0.5
            s = torch.where(sees, s, float("-inf"))
            v = st["v8"][b, hk, :m].double() * per(st["vs"], b, hk, m)
            lse[b, heads, :cnt] = torch.logsumexp(s, -1)
            o[b, heads, :cnt] = torch.softmax(s, -1) @ v
    return o, lse


def _round_e4m3(x):
    """Nearest E4M3 value of x (ties to even), |x| up to 448."""
    a = x.abs().clamp(max=448.0)
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))).clamp(min=-6.0) - 3.0)
    # log2 may land on the wrong side of a power of two: put the step right.
    step = torch.where(a < 8.0 * step, torch.clamp(step / 2, min=2.0 ** -9), step)
    step = torch.where(a >= 16.0 * step, step * 2, step)
    return torch.copysign(torch.round(a / step) * step, x)


def _least_scale(a):
    """Least power of two s in 2^-100 .. 2^120 with a <= 448 s."""
    if not a > 0:
        return 2.0 ** -100
    e = math.ceil(math.log2(a / 448.0))
    e = e + 1 if a > 448.0 * 2.0 ** e else e - 1 if a <= 448.0 * 2.0 ** (e - 1) else e
    return 2.0 ** max(-100, min(120, e))


def _exact_keep(st, lens, counts, paths, block):
    out = [st[x].float().double() for x in ("k8", "v8", "ks", "vs", "w")]
    was = [x.clone() for x in out]
    for b, (m, cnt, path) in enumerate(zip(lens, counts, paths)):
        base = m - cnt
        for h in range(out[0].shape[1]):
            for i, node in enumerate(path):
                out[4][b, h, base + i] = was[4][b, h, base + node]
            for c, s, c0, s0 in ((out[0], out[2], was[0], was[2]), (out[1], out[3], was[1], was[3])):
                for t in range(base // block, (base + len(path) - 1) // block + 1):
                    here = [i for i in range(len(path)) if (base + i) // block == t]
                    from_ = [base + path[i] for i in here]
                    x = torch.stack([c0[b, h, j] * s0[b, h, j // block] for j in from_])
                    sc = _least_scale(float(x.abs().max()))
                    if base > t * block:
                        old = float(s0[b, h, t])
                        if sc > old:
                            c[b, h, t * block:base] = _round_e4m3(c0[b, h, t * block:base] * (old / sc))
                        sc = max(sc, old)
                    s[b, h, t] = sc
                    c[b, h, base + here[0]:base + here[-1] + 1] = _round_e4m3(x / sc)
    lengths = torch.tensor([m - c + len(p) for m, c, p in zip(lens, counts, paths)])
    return (*out, lengths.cuda())
