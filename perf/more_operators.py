"""Operators of a serving step around the paged cache and the MoE block: the cases they are measured on, and their
plain form.

norm     y = scale * (x + gate * N(block; post)) and n = N(y; pre), with N(v; w) = v / rms(v) * (1 + w): the norms
         after one block and before the next, with the residual between them.
rotary   queries and keys turned by positions on one to three axes (time, height, width): pair i of a head turns
         by positions[axis[i], token] * freq[i].
tree     attention of a tree of drafted tokens per sequence over its paged cache: node i sees the context before
         the tree, its ancestors and itself, through an optional sliding window and first tokens that stay visible.
keep     the accepted path of each tree moves to the slots after the context, in all layers' caches.
select   the best candidates over beams and vocabulary, by score + logit - logsumexp(logits of the beam).
reorder  the caches and page tables of users' beams follow the beams' parents.
"""
import math

import torch

own = False

FMT_BYTES = {"bf16": 2, "e4m3": 1}
# (query heads, kv heads, head width): the model's sliding and global layers, and generic ones.
HEADS = ((16, 8, 256), (16, 2, 512), (32, 8, 128), (8, 8, 128), (12, 4, 128))
# The same for rotary positions alone, with widths of image encoders.
ROTARY_HEADS = HEADS + ((16, 16, 64), (16, 16, 72), (12, 12, 80))
HIDDEN = 2816
VOCAB = 262144


def listed():
    return [
        # The residual and the next norm of a decode step's tokens.
        {"name": "norm_decode", "op": "norm", "tokens": 64, "hidden": HIDDEN, "gate": "none"},
        # A prompt's tokens, with a gate per token as image blocks have it.
        {"name": "norm_prompt_gated", "op": "norm", "tokens": 8192, "hidden": HIDDEN, "gate": "token"},
        # A decode step of text: one axis, positions far into a long context.
        {"name": "rotary_decode", "op": "rotary", "tokens": 64, "hq": 16, "hkv": 8, "d": 256, "turned": 256, "axes": 1,
         "interleaved": False, "far": 1000000},
        # A prompt with images in a layer of the model: three axes, a part of the head turned.
        {"name": "rotary_images", "op": "rotary", "tokens": 9001, "hq": 16, "hkv": 2, "d": 512, "turned": 384, "axes": 3,
         "interleaved": False, "far": 20000},
        # One user's draft of a dozen tokens in a sliding layer.
        {"name": "tree_one_window", "op": "tree", "fmt": "bf16", "hq": 16, "hkv": 8, "d": 256, "page": 16, "seqs": 1,
         "new_lo": 12, "new_hi": 12, "old_lo": 2043, "old_hi": 2043, "window": 1024, "sinks": 4},
        # Many users' drafts in a global layer over an 8-bit cache, ragged contexts.
        {"name": "tree_users_e4m3", "op": "tree", "fmt": "e4m3", "hq": 16, "hkv": 2, "d": 512, "page": 64, "seqs": 32,
         "new_lo": 5, "new_hi": 32, "old_lo": 65, "old_hi": 16001, "window": 0, "sinks": 0},
        # The accepted tokens of one draft, one layer.
        {"name": "keep_one", "op": "keep", "fmt": "bf16", "hkv": 8, "d": 128, "page": 16, "seqs": 1, "new_lo": 12,
         "new_hi": 12, "old_lo": 37, "old_hi": 37, "layers": 1},
        # The accepted tokens of many users' drafts, in several layers.
        {"name": "keep_users_e4m3", "op": "keep", "fmt": "e4m3", "hkv": 2, "d": 512, "page": 64, "seqs": 64, "new_lo": 8,
         "new_hi": 60, "old_lo": 20, "old_hi": 200, "layers": 6},
        # One user's beams.
        {"name": "select_one", "op": "select", "dtype": "bf16", "users": 1, "beams": 4, "vocab": VOCAB, "count": 8,
         "done": False},
        # A batch of users' beams, some of which have ended.
        {"name": "select_users", "op": "select", "dtype": "bf16", "users": 32, "beams": 5, "vocab": VOCAB, "count": 10,
         "done": True},
        # One user's beams move in one layer.
        {"name": "reorder_one", "op": "reorder", "fmt": "e4m3", "hkv": 8, "d": 256, "page": 32, "users": 1, "beams": 4,
         "len_lo": 150, "len_hi": 150, "layers": 1},
        # A batch of users' beams move in several layers.
        {"name": "reorder_users", "op": "reorder", "fmt": "bf16", "hkv": 2, "d": 512, "page": 64, "users": 16, "beams": 5,
         "len_lo": 40, "len_hi": 300, "layers": 6},
    ]


def draw(rng):
    def log(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))

    op = rng.choice(("norm", "rotary", "tree", "tree", "keep", "select", "reorder"))
    if op == "norm":
        c = {"op": op, "tokens": log(1, 40000), "hidden": rng.choice((HIDDEN, 8 * log(8, 1024))),
             "gate": rng.choice(("none", "one", "token"))}
        shrink = ("tokens",)
    elif op == "rotary":
        hq, hkv, d = rng.choice(ROTARY_HEADS)
        c = {"op": op, "tokens": log(1, 20000), "hq": hq, "hkv": hkv, "d": d,
             "turned": rng.choice((d, d, 8 * rng.randint(1, d // 8))), "axes": rng.choice((1, 2, 3)),
             "interleaved": rng.random() < 0.4, "far": log(100, 4000000)}
        shrink = ("tokens",)
    elif op == "tree":
        hq, hkv, d = rng.choice(HEADS)
        new_hi, old_hi = log(2, 128), log(1, 60000)
        window = rng.choice((0, 0, log(1, 5000), 1024))
        c = {"op": op, "fmt": rng.choice(("bf16", "e4m3")), "hq": hq, "hkv": hkv, "d": d,
             "page": rng.choice((16, 32, 64, 128)), "seqs": log(1, 128), "new_lo": log(1, new_hi), "new_hi": new_hi,
             "old_lo": log(1, old_hi), "old_hi": old_hi, "window": window,
             "sinks": rng.choice((0, 4, log(1, 300))) if window else 0}
        shrink = ("seqs", "new_hi", "old_hi")
    elif op == "select":
        beams = rng.randint(1, 16)
        c = {"op": op, "dtype": rng.choice(("bf16", "fp32")), "users": log(1, 64), "beams": beams,
             "vocab": rng.choice((VOCAB, log(500, 300000))), "count": rng.choice((2 * beams, rng.randint(1, 32))),
             "done": rng.random() < 0.5}
        shrink = ("users", "vocab")
    else:
        hq, hkv, d = rng.choice(HEADS)
        hi = log(1, 400)
        c = {"op": op, "fmt": rng.choice(("bf16", "e4m3")), "hkv": hkv, "d": d, "page": rng.choice((16, 32, 64, 128)),
             "layers": rng.randint(1, 12)}
        if op == "keep":
            new_hi = log(2, 128)
            c.update(seqs=log(1, 100), new_lo=log(1, new_hi), new_hi=new_hi, old_lo=log(1, hi), old_hi=hi)
            shrink = ("seqs", "layers")
        else:
            c.update(users=log(1, 32), beams=rng.randint(2, 8), len_lo=log(1, hi), len_hi=hi)
            shrink = ("users", "layers")
    # Sizes shrink until the case costs no more than the largest listed ones and its plain form fits.
    while not _affordable(c):
        key = max(shrink, key=lambda k: c[k])
        c[key] = max(1, c[key] * 2 // 3)
        for lo, hi in (("new_lo", "new_hi"), ("old_lo", "old_hi")):
            if lo in c:
                c[lo] = min(c[lo], c[hi])
    return c


def _affordable(c):
    w = work(c)
    if c["op"] == "tree":
        new, kv = _lengths(c)
        padded, scores = c["seqs"] * max(kv) * c["hkv"] * c["d"], c["seqs"] * max(new) * max(kv) * c["hq"]
        return w["flops"] <= 2.8e11 and w["bytes"] <= 3.3e8 and padded <= 6e8 and scores <= 3e8
    if c["op"] in ("keep", "reorder"):
        return c["layers"] * _pages_of(c)[2] * c["page"] * c["hkv"] * c["d"] * 2 * FMT_BYTES[c["fmt"]] <= 3.6e8
    return w["bytes"] <= {"norm": 2.31e8, "rotary": 3.32e8, "select": 8.4e7}[c["op"]]


def _spread(lo, hi, n, step):
    """n lengths from lo to hi, evenly spaced on a log scale, in a mixed order."""
    if lo == hi or n == 1:
        return [hi] * n
    at = [int(round(math.exp(math.log(lo) + (math.log(hi) - math.log(lo)) * i / (n - 1)))) for i in range(n)]
    return [at[i * step % n] for i in range(n)] if math.gcd(step, n) == 1 else at


def _lengths(c):
    """Each sequence's drafted tokens, and all its cached tokens with them."""
    new = _spread(c["new_lo"], c["new_hi"], c["seqs"], 7)
    old = _spread(c["old_lo"], c["old_hi"], c["seqs"], 11)
    return new, [a + b for a, b in zip(new, old)]


def _pages_of(c):
    """What the page tables of a case hold: pages of each row that are its own, shared ones before them, and how many
    pages the cache has."""
    if c["op"] == "reorder":
        # A user's beams share the pages before the one under way; each has that one and the next for itself.
        shared = [n // c["page"] for n in _spread(c["len_lo"], c["len_hi"], c["users"], 7)]
        own_pages = [2] * (c["users"] * c["beams"])
        used = sum(shared) + sum(own_pages)
    else:
        shared, own_pages = None, [-(-n // c["page"]) for n in _lengths(c)[1]]
        used = sum(own_pages)
    return own_pages, shared, used + used // 8 + 3


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape, dtype=torch.bfloat16):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=dtype)

    s = {"case": c}
    if own:
        from mixture_experts_ffn_router_gb300 import binding as B
    if c["op"] == "norm":
        T, H = c["tokens"], c["hidden"]
        # A residual stream with a few channels of large magnitude, and a block's output.
        s["x"] = randn(T, H) * 4
        s["x"][:, ::97] *= 30
        s["block"] = randn(T, H)
        s["gate"] = None if c["gate"] == "none" else randn(T if c["gate"] == "token" else 1, H).expand(T, H)
        s["post"], s["pre"] = (0.1 * randn(H, dtype=torch.float32) for _ in range(2))
        s["scale"] = 0.8
    elif c["op"] == "rotary":
        T, P = c["tokens"], c["turned"] // 2
        # Queries and keys as they leave the projections: views of one fused row per token.
        fused = randn(T, (c["hq"] + 2 * c["hkv"]) * c["d"])
        s["q"], s["k"], _ = fused.view(T, -1, c["d"]).split((c["hq"], c["hkv"], c["hkv"]), 1)
        s["freqs"] = [1e4 ** (-i / P) for i in range(P)]
        s["axis"] = [i * c["axes"] // P for i in range(P)]  # the first pairs turn with time, the last with width
        # Text, then pictures whose rows and columns count on from where they stand.
        t = torch.arange(T, device="cuda", dtype=torch.int32)
        first = int(torch.randint(0, c["far"], (1,), generator=gen, device="cuda"))
        s["positions"] = torch.stack((t // 700 + first, t // 28 % 25 + first, t % 28 + first))[:c["axes"]].contiguous()
        if c["axes"] == 1:
            s["positions"] = t + first
        if own:
            s["rotary"] = B.Rotary(s["freqs"], s["axis"], interleaved=c["interleaved"])
        else:
            s["freqs"] = torch.tensor(s["freqs"], dtype=torch.float64, device="cuda")
            s["axis"] = torch.tensor(s["axis"], device="cuda")
    elif c["op"] == "select":
        rows = c["users"] * c["beams"]
        # Beams that are sure of the next token and beams that are not.
        sure = torch.rand(rows, 1, generator=gen, device="cuda") * 3 + 0.5
        dtype = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
        s["logits"] = (randn(rows, c["vocab"], dtype=torch.float32) * sure).to(dtype)
        s["scores"] = -8 * torch.rand(c["users"], c["beams"], generator=gen, device="cuda")
        s["finished"] = None
        if c["done"]:
            s["finished"] = torch.rand(c["users"], c["beams"], generator=gen, device="cuda") < 0.2
        s["end"] = 1
        if own:
            s["search"] = B.BeamSearch(c["users"], c["beams"], c["vocab"], c["count"])
    else:
        _prepare_cache(s, gen, randn)
        if own:
            _prepare_handles(s)
    return s


def _prepare_cache(s, gen, randn):
    c = s["case"]
    P, layers = c["page"], c.get("layers", 1)
    own_pages, shared, n_pages = _pages_of(c)
    order = torch.randperm(n_pages, generator=gen, device="cuda", dtype=torch.int64).to(torch.int32).tolist()
    rows = []
    if shared is not None:
        for n in shared:
            front = [order.pop() for _ in range(n)]
            rows += [front + [order.pop(), order.pop()] for _ in range(c["beams"])]
    else:
        rows = [[order.pop() for _ in range(n)] for n in own_pages]
    width = max(len(r) for r in rows)
    s["pages"] = torch.tensor([r + [-1] * (width - len(r)) for r in rows], dtype=torch.int32).cuda()
    s["n_pages"] = n_pages
    shape = (layers, n_pages, c["hkv"], P, c["d"])
    s["cache"] = {}
    for n in ("k", "v"):
        x = randn(*shape)
        if c["fmt"] == "bf16":
            s["cache"][n] = x
        else:
            x = x.float()
            scale = x.abs().amax(-1) / 448
            s["cache"][n], s["cache"][n + "_scale"] = (x / scale[..., None]).to(torch.float8_e4m3fn), scale
        del x
    if c["op"] == "reorder":
        s["lengths"] = torch.tensor(_spread(c["len_lo"], c["len_hi"], c["users"], 7), dtype=torch.int32).cuda()
        # Beams that go on keep their place; the others' places go to further children of those.
        stays = torch.rand(c["users"], c["beams"], generator=gen, device="cuda") < 0.5
        stays[:, 0] = True
        rank = torch.rand(c["users"], c["beams"], c["beams"], generator=gen, device="cuda")
        other = rank.masked_fill(~stays[:, None], -1).argmax(-1)
        s["parents"] = torch.where(stays, torch.arange(c["beams"], device="cuda"), other).to(torch.int32)
        return
    new, kv = _lengths(c)
    cu = torch.zeros(c["seqs"] + 1, dtype=torch.int32)
    cu[1:] = torch.tensor(new).cumsum(0)
    T = int(cu[-1])
    s.update(cu_q=cu.cuda(), kv_len=torch.tensor(kv, dtype=torch.int32).cuda(), tokens=T, max_new=max(new), max_kv=max(kv))
    node = torch.cat([torch.arange(n) for n in new]).cuda()
    u = torch.rand(T, generator=gen, device="cuda", dtype=torch.float64)
    if c["op"] == "tree":
        # Each node below an earlier one, or a root (-1); likelier below a late one.
        s["parents"] = ((node + 1) * u.sqrt()).long().minimum(node).to(torch.int32) - 1
        s["q"] = randn(T, c["hq"], c["d"]) * torch.linspace(1.0, 2.5, c["hq"], device="cuda").view(1, -1, 1).to(torch.bfloat16)
        return
    # Up to six accepted nodes: the first guesses of each depth come first in a draft, the others late in it.
    depth = min(6, max(new))
    count = (torch.rand(c["seqs"], generator=gen, device="cuda") * (depth + 1)).int().clamp(max=depth)
    s["counts"] = torch.minimum(count, torch.tensor(new, dtype=torch.int32, device="cuda"))
    n = torch.tensor(new, device="cuda").view(-1, 1)
    i = torch.arange(depth, device="cuda").view(1, -1)
    straight = (torch.rand(c["seqs"], 1, generator=gen, device="cuda") * (depth + 1)).int()
    late = torch.rand(c["seqs"], max(new), generator=gen, device="cuda")
    at = torch.arange(max(new), device="cuda").view(1, -1)
    late = late.masked_fill((at >= n) | (at < s["counts"].view(-1, 1)), 2.0).argsort(1)[:, :depth].sort(1).values
    fits = (n - s["counts"].view(-1, 1)) >= depth
    s["nodes"] = torch.where((i < straight) | ~fits, i, late).to(torch.int32).contiguous()


def _prepare_handles(s):
    from mixture_experts_ffn_router_gb300 import binding as B
    c = s["case"]
    seqs = c["users"] * c["beams"] if c["op"] == "reorder" else c["seqs"]
    s["kv"] = B.PagedKV(c.get("hq", c["hkv"]), c["hkv"], c["d"], c["page"], s["n_pages"], c["fmt"],
                        max_tokens=max(s.get("tokens", 1), 1), max_seqs=seqs)
    s["layers"] = [s["kv"].cache(**{n: t[i] for n, t in s["cache"].items()}) for i in range(c.get("layers", 1))]
    if c["op"] != "reorder":
        s["batch"] = B.KVBatch(s["cu_q"], s["kv_len"], s["pages"], max_new=s["max_new"])
    if c["op"] == "tree":
        s["tree"] = s["kv"].tree(s["batch"], s["parents"])


def run(state):
    s, c = state, state["case"]
    if not own:
        return {"norm": _norm, "rotary": _rotary, "tree": _tree, "keep": _keep, "select": _select,
                "reorder": _reorder}[c["op"]](s)
    if c["op"] == "norm":
        from mixture_experts_ffn_router_gb300 import binding as B
        y, n = B.block_norm(s["x"], s["block"], post=s["post"], gate=s["gate"], scale=s["scale"], pre=s["pre"])
        return {"y": y, "n": n}
    if c["op"] == "rotary":
        q, k = s["rotary"].apply(s["q"], s["k"], s["positions"])
        return {"q": q, "k": k}
    if c["op"] == "tree":
        out, lse = s["kv"].tree_attention(s["layers"][0], s["batch"], s["tree"], s["q"], window=c["window"], sinks=c["sinks"])
        return {"out": out, "lse": lse}
    if c["op"] == "keep":
        return {"kv_len": s["kv"].keep(s["layers"], s["batch"], s["nodes"], s["counts"]), **s["cache"]}
    if c["op"] == "select":
        scores, beams, tokens = s["search"].select(s["logits"], s["scores"], finished=s["finished"], end_token=s["end"])
        return {"scores": scores, "beams": beams, "tokens": tokens}
    s["kv"].reorder(s["layers"], s["pages"], s["lengths"], s["parents"])
    return {"pages": s["pages"], **s["cache"]}


# ------------------------------------------------------------------ the plain forms

def _norm(s):
    def normed(v, w):
        return v * (v.square().mean(-1, keepdim=True) + 1e-6).rsqrt() * (1 + w)

    b = normed(s["block"].float(), s["post"])
    if s["gate"] is not None:
        b = b * s["gate"].float()
    y = (s["x"].float() + b) * s["scale"]
    return {"y": y.to(torch.bfloat16), "n": normed(y, s["pre"]).to(torch.bfloat16)}


def _rotary(s):
    c = s["case"]
    T, P, R = c["tokens"], c["turned"] // 2, c["turned"]
    angle = s["positions"].view(-1, T)[s["axis"]].T.double() * s["freqs"]             # [T, P]
    cos, sin = angle.cos().float().view(T, 1, P), angle.sin().float().view(T, 1, P)

    def turn(x):
        x = x.float()
        y = x.clone()
        if c["interleaved"]:
            a, b = x[..., 0:R:2], x[..., 1:R:2]
            y[..., 0:R:2], y[..., 1:R:2] = a * cos - b * sin, b * cos + a * sin
        else:
            a, b = x[..., :P], x[..., P:R]
            y[..., :P], y[..., P:R] = a * cos - b * sin, b * cos + a * sin
        return y.to(torch.bfloat16)

    return {"q": turn(s["q"]), "k": turn(s["k"])}


def _values(s, n, at):
    """The first layer's values of K or V at the places `at`, in fp32."""
    if s["case"]["fmt"] == "bf16":
        return s["cache"][n][0][at].float()
    return s["cache"][n][0].view(torch.uint8)[at].view(torch.float8_e4m3fn).float() * s["cache"][n + "_scale"][0][at][..., None]


def _tree(s):
    c = s["case"]
    B, Q, L, P, hkv, d = c["seqs"], s["max_new"], s["max_kv"], c["page"], c["hkv"], c["d"]
    g = c["hq"] // hkv
    cu = s["cu_q"].long()
    count = (cu[1:] - cu[:-1]).view(B, 1)
    i = torch.arange(Q, device="cuda").view(1, Q)
    row = (cu[:-1].view(B, 1) + i).clamp(max=s["tokens"] - 1)                          # [B, Q]
    # Who is above whom: paths of up to 2^7 steps, doubled seven times.
    parent = torch.where(i < count, s["parents"][row].long(), -1)
    above = (parent.unsqueeze(-1) == i.view(1, 1, Q)).float() + torch.eye(Q, device="cuda")
    above = (above @ above > 0).float()
    above = (above @ above > 0).float()
    above = (above @ above > 0).float()
    above = (above @ above > 0).float()
    above = (above @ above > 0).float()
    above = (above @ above > 0).float()
    above = above @ above > 0                                                         # [B, Q, Q], itself among them
    depth = above.sum(-1) - 1                                                         # [B, Q]
    old = s["kv_len"].long().view(B, 1) - count                                       # the context's length
    j = torch.arange(L, device="cuda").view(1, L)
    page = s["pages"][:, j[0] // P].long().clamp(min=0)                               # [B, L]
    at = (page, slice(None), (j % P).expand(B, L))
    used = (j < s["kv_len"].view(B, 1)).view(B, 1, L, 1)
    k, v = (torch.where(used, _values(s, n, at).transpose(1, 2), 0.0) for n in ("k", "v"))  # [B, hkv, L, d]
    # Position and visibility of each cached token for each node: the slots behind the context hold the tree.
    node = (j - old).clamp(0, Q - 1)                                                  # [B, L]
    in_tree = (j >= old) & (j < old + count)
    kpos = torch.where(in_tree, old + depth.gather(1, node), j)                       # [B, L]
    pos = (old + depth).unsqueeze(-1)                                                 # [B, Q, 1]
    seen = torch.where(in_tree.unsqueeze(1), above.gather(2, node.unsqueeze(1).expand(B, Q, L)), (j < old).unsqueeze(1))
    if c["window"]:
        seen &= (kpos.unsqueeze(1) > pos - c["window"]) | (kpos < c["sinks"]).unsqueeze(1)
    q = s["q"][row].float().view(B, Q, hkv, g, d).permute(0, 2, 3, 1, 4).reshape(B, hkv, g * Q, d)
    x = (q @ k.transpose(2, 3)).mul_(d ** -0.5).view(B, hkv, g, Q, L)
    x.masked_fill_(~seen.view(B, 1, 1, Q, L), -math.inf)
    top = x.amax(-1, keepdim=True).clamp(min=-3e38)
    x = x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    out = (x.view(B, hkv, g * Q, L) @ v).view(B, hkv, g, Q, d) / total.clamp(min=1e-38)
    lse = (top + total.log())[..., 0]
    live = i < count
    out = out.permute(0, 3, 1, 2, 4).reshape(B, Q, c["hq"], d)[live].to(torch.bfloat16)
    return {"out": out, "lse": lse.permute(0, 3, 1, 2).reshape(B, Q, c["hq"])[live]}


def _bytes(t):
    """Codes as bytes, which can be indexed; other tensors as they are."""
    return t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t


def _keep(s):
    c = s["case"]
    P, cu = c["page"], s["cu_q"]
    old = (s["kv_len"] - (cu[1:] - cu[:-1])).long().view(-1, 1)
    i = torch.arange(s["nodes"].shape[1], device="cuda").view(1, -1)
    seq, to = torch.nonzero(i < s["counts"].view(-1, 1), as_tuple=True)
    a, b = old[seq, 0] + s["nodes"][seq, to].long(), old[seq, 0] + to
    src, dst = (s["pages"][seq, a // P].long(), a % P), (s["pages"][seq, b // P].long(), b % P)
    moved = [_move(_bytes(t), src, dst) for t in s["cache"].values()]
    assert len(moved) == len(s["cache"])
    return {"kv_len": (old[:, 0] + s["counts"]).to(torch.int32), **s["cache"]}


def _move(t, src, dst):
    """Rows [layers, page, head, slot, ...] at `src` to `dst`, all read before one is written."""
    t[:, dst[0], :, dst[1]] = t[:, src[0], :, src[1]]
    return t


def _select(s):
    c = s["case"]
    U, K, V = c["users"], c["beams"], c["vocab"]
    x = s["logits"].double().view(U, K, V)
    top = x.amax(-1, keepdim=True)
    x = x - (top + (x - top).exp().sum(-1, keepdim=True).log())                        # 64 bits: borders are near
    if s["finished"] is not None:
        ended = torch.where(torch.arange(V, device="cuda") == s["end"], 0.0, -math.inf).double()
        x = torch.where(s["finished"].unsqueeze(-1), ended, x)
    x = (x + s["scores"].double().unsqueeze(-1)).view(U, K * V)
    best, at = torch.sort(x, dim=1, descending=True, stable=True)
    best, at = best[:, :c["count"]], at[:, :c["count"]].to(torch.int32)
    none = ~(best > -math.inf)
    return {"scores": best.float(), "beams": (at // V).masked_fill(none, -1), "tokens": (at % V).masked_fill(none, -1)}


def _reorder(s):
    c = s["case"]
    U, K, P = c["users"], c["beams"], c["page"]
    table = s["pages"].view(U, K, -1)
    width = table.shape[-1]
    whole = (s["lengths"] // P).long().view(U, 1, 1)                                   # pages that are full
    rest = (s["lengths"] % P).view(U, 1, 1).expand(U, K, 1)
    parent = s["parents"].long().unsqueeze(-1)
    page = table.gather(2, whole.clamp(max=width - 1).expand(U, K, 1))                # each beam's page under way
    user, beam, slot = torch.nonzero((torch.arange(P, device="cuda") < rest) & (parent != torch.arange(K, device="cuda").view(K, 1)),
                                     as_tuple=True)
    dst = (page[user, beam, 0].long(), slot)
    src = (page[user, parent[user, beam, 0], 0].long(), slot)
    moved = [_move(_bytes(t), src, dst) for t in s["cache"].values()]
    assert len(moved) == len(s["cache"])
    full = torch.arange(width, device="cuda") < whole
    s["pages"].copy_(torch.where(full, table.gather(1, parent.expand(U, K, width)), table).view(U * K, width))
    return {"pages": s["pages"], **s["cache"]}


# ------------------------------------------------------------------ work and exact values

def work(case):
    c = case
    if c["op"] == "norm":
        values = c["tokens"] * c["hidden"]
        gate = {"none": 0, "one": 2 * c["hidden"], "token": 2 * values}[c["gate"]]
        return {"bytes": 8 * values + gate + 8 * c["hidden"], "flops": 12 * values}
    if c["op"] == "rotary":
        heads = c["tokens"] * (c["hq"] + c["hkv"])
        return {"bytes": 4 * heads * c["d"] + 4 * c["tokens"] * c["axes"], "flops": 3 * heads * c["turned"]}
    if c["op"] == "select":
        rows = c["users"] * c["beams"]
        return {"bytes": rows * c["vocab"] * (2 if c["dtype"] == "bf16" else 4) + 5 * rows + 12 * c["users"] * c["count"],
                "flops": 4 * rows * c["vocab"]}
    row = c["hkv"] * (2 * c["d"] * FMT_BYTES[c["fmt"]] + (8 if c["fmt"] == "e4m3" else 0))  # a token's keys and values
    if c["op"] == "keep":
        # Half of up to six accepted tokens, half of them already in place.
        new = _lengths(c)[0]
        return {"bytes": c["layers"] * sum(min(n, 6) for n in new) * 0.25 * 2 * row + 12 * c["seqs"], "flops": 0}
    if c["op"] == "reorder":
        # Half of the beams take another's page under way; the tables are read and written.
        lengths = _spread(c["len_lo"], c["len_hi"], c["users"], 7)
        rest = sum(n % c["page"] for n in lengths) * c["beams"] * 0.5
        table = 2 * 4 * sum(n // c["page"] for n in lengths) * c["beams"]
        return {"bytes": c["layers"] * rest * 2 * row + table + 4 * c["users"] * c["beams"], "flops": 0}
    new, kv = _lengths(c)
    keys = pairs = 0
    for n, L in zip(new, kv):
        old = L - n
        # A node sees its depth in the tree, about log2 of its number, beside the context's part.
        seen = min(old, c["window"] + c["sinks"]) if c["window"] else old
        keys += seen + n
        pairs += n * (seen + 1 + int(math.log2(n)))
    rows = sum(new) * c["hq"]
    return {"bytes": keys * row + rows * (4 * c["d"] + 4), "flops": 4 * c["d"] * pairs * c["hq"]}


def exact(case, seed):
    """The operators' definitions in 64 bits, token by token or user by user."""
    s = prepare(case, seed)
    c = s["case"]
    return {"norm": _exact_norm, "rotary": _exact_rotary, "tree": _exact_tree, "keep": _exact_keep, "select": _exact_select,
            "reorder": _exact_reorder}[c["op"]](s, c)


def _exact_norm(s, c):
    x, b = s["x"].double(), s["block"].double()
    g = 1.0 if s["gate"] is None else s["gate"].double()
    rms = torch.linalg.vector_norm(b, dim=-1, keepdim=True) ** 2 / c["hidden"] + 1e-6
    y = s["scale"] * (x + g * (b / rms.sqrt() * (1.0 + s["post"].double())))
    rms = torch.linalg.vector_norm(y, dim=-1, keepdim=True) ** 2 / c["hidden"] + 1e-6
    return {"y": y, "n": y / rms.sqrt() * (1.0 + s["pre"].double())}


def _exact_rotary(s, c):
    P = c["turned"] // 2
    freqs = torch.as_tensor(s["freqs"].tolist() if torch.is_tensor(s["freqs"]) else s["freqs"], dtype=torch.float64)
    axis = s["axis"].tolist() if torch.is_tensor(s["axis"]) else s["axis"]
    where = s["positions"].view(-1, c["tokens"]).cpu().double()
    turn = torch.polar(torch.ones((), dtype=torch.float64), torch.stack([where[axis[i]] * freqs[i] for i in range(P)], 1)).cuda()
    out = {}
    for n in ("q", "k"):
        y = s[n].double()
        if c["interleaved"]:
            z = torch.view_as_complex(y[..., :2 * P].unflatten(-1, (P, 2)).contiguous()) * turn[:, None]
            y[..., :2 * P] = torch.view_as_real(z).flatten(-2)
        else:
            z = torch.complex(y[..., :P], y[..., P:2 * P]) * turn[:, None]
            y[..., :2 * P] = torch.cat((z.real, z.imag), -1)
        out[n] = y
    return out


def _exact_tree(s, c):
    P, g = c["page"], c["hq"] // c["hkv"]
    cu, kv_len, table, parents = s["cu_q"].tolist(), s["kv_len"].tolist(), s["pages"].cpu(), s["parents"].tolist()
    out = torch.zeros(s["tokens"], c["hq"], c["d"], dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["tokens"], c["hq"], dtype=torch.float64, device="cuda")
    for b in range(c["seqs"]):
        n, L = cu[b + 1] - cu[b], kv_len[b]
        old = L - n
        mask, depths = torch.zeros(n, L, dtype=torch.bool), []
        for i in range(n):
            path = [i]
            while parents[cu[b] + path[-1]] >= 0:
                path.append(parents[cu[b] + path[-1]])
            here = old + len(path) - 1
            depths.append(here)
            positions = [depths[p] for p in path]
            low = here - c["window"] + 1 if c["window"] else 0
            mask[i, max(0, min(low, old)):old] = True
            mask[i, :min(c["sinks"], old)] = True
            for p, where in zip(path, positions):
                mask[i, old + p] = where >= low or where < c["sinks"]
        mask = mask.cuda()
        pos = torch.arange(L)
        page, slot = table[b][pos // P].long().cuda(), (pos % P).cuda()
        for h in range(c["hkv"]):
            kv = []
            for name in ("k", "v"):
                t = s["cache"][name][0][:, h]
                x = (t.view(torch.uint8) if c["fmt"] == "e4m3" else t)[page, slot]
                x = x.view(torch.float8_e4m3fn).double() if c["fmt"] == "e4m3" else x.double()
                if c["fmt"] == "e4m3":
                    x = x * s["cache"][name + "_scale"][0][page, h, slot].double()[:, None]
                kv.append(x)
            for hq in range(h * g, h * g + g):
                x = s["q"][cu[b]:cu[b + 1], hq].double() @ kv[0].T / math.sqrt(c["d"])
                x[~mask] = -math.inf
                lse[cu[b]:cu[b + 1], hq] = torch.logsumexp(x, -1)
                out[cu[b]:cu[b + 1], hq] = torch.softmax(x, -1) @ kv[1]
    return {"out": out, "lse": lse}


def _exact_keep(s, c):
    cu, kv_len, table = s["cu_q"].tolist(), s["kv_len"].tolist(), s["pages"].tolist()
    nodes, counts, P = s["nodes"].tolist(), s["counts"].tolist(), c["page"]
    before = {n: t.clone() for n, t in s["cache"].items()}
    got = {n: t.clone() for n, t in before.items()}
    for b in range(c["seqs"]):
        old = kv_len[b] - (cu[b + 1] - cu[b])
        for i in range(counts[b]):
            a, z = old + nodes[b][i], old + i
            for n in got:
                _bytes(got[n])[:, table[b][z // P], :, z % P] = _bytes(before[n])[:, table[b][a // P], :, a % P]
    return {"kv_len": torch.tensor([kv_len[b] - (cu[b + 1] - cu[b]) + counts[b] for b in range(c["seqs"])], dtype=torch.int32),
            **got}


def _exact_select(s, c):
    U, K, V, n = c["users"], c["beams"], c["vocab"], c["count"]
    out = {"scores": torch.full((U, n), -math.inf, dtype=torch.float64), "beams": torch.full((U, n), -1, dtype=torch.int32),
           "tokens": torch.full((U, n), -1, dtype=torch.int32)}
    for u in range(U):
        found = []
        for k in range(K):
            score = float(s["scores"][u, k].double())
            if s["finished"] is not None and bool(s["finished"][u, k]):
                found.append((-score, k, s["end"]))
                continue
            lp = torch.log_softmax(s["logits"][u * K + k].double(), -1) + score
            least = torch.topk(lp, min(n, V)).values[-1]
            at = torch.nonzero(lp >= least)[:, 0]
            found += [(-v, k, i) for v, i in zip(lp[at].tolist(), at.tolist())]
        for i, (v, k, t) in enumerate(sorted(found)[:n]):
            out["scores"][u, i], out["beams"][u, i], out["tokens"][u, i] = -v, k, t
    return out


def _exact_reorder(s, c):
    table, lengths, parents = s["pages"].tolist(), s["lengths"].tolist(), s["parents"].tolist()
    before = {n: t.clone() for n, t in s["cache"].items()}
    got, pages = {n: t.clone() for n, t in before.items()}, [list(r) for r in table]
    for u in range(c["users"]):
        whole, rest = divmod(lengths[u], c["page"])
        for k in range(c["beams"]):
            me, of = u * c["beams"] + k, u * c["beams"] + parents[u][k]
            pages[me][:whole] = table[of][:whole]
            if rest:
                for n in got:
                    _bytes(got[n])[:, table[me][whole], :, :rest] = _bytes(before[n])[:, table[of][whole], :, :rest]
    return {"pages": torch.tensor(pages, dtype=torch.int32), **got}
