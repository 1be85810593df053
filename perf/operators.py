"""The paged key/value cache and its attention: the cases they are measured on, and their plain form.

Three operators of a serving step: writing new keys and values into a paged cache (bf16, or e4m3
with one fp32 scale per token and head), reading cached tokens back as bf16, and attention of each
sequence's new tokens over its cached ones, causal, with an optional sliding window and first
tokens that stay visible. Sequence b brings n_b new tokens; its newest cached token is at position
kv_len[b] - 1, so new token i is at position kv_len[b] - n_b + i, slot (position % page) of page
pages[b, position // page].
"""
import math

import torch

own = False

E4M3_MAX = 448.0
FMT_BYTES = {"bf16": 2, "e4m3": 1}

# (query heads, kv heads, head width): the model's sliding and global layers, and generic ones of
# width 128 with groups of 4, 1 and 3.
HEADS = ((16, 8, 256), (16, 2, 512), (32, 8, 128), (8, 8, 128), (12, 4, 128))


def listed():
    return [
        # One token of a single short sequence: nothing but latency.
        _case("decode_one_short", "attend", "bf16", 32, 8, 128, 16, 1, (1, 1), (37, 37)),
        # A serving batch in a global layer's shape over an 8-bit cache, ragged lengths.
        _case("decode_64_global_e4m3", "attend", "e4m3", 16, 2, 512, 64, 64, (1, 1), (65, 16001)),
        # The same model's sliding layers: only the window and the sinks are read of long caches.
        _case("decode_256_window", "attend", "bf16", 16, 8, 256, 16, 256, (1, 1), (100, 7000), 1024, 4),
        # One user's long context, one token at a time: a few rows and a very long axis.
        _case("decode_long_bf16", "attend", "bf16", 16, 2, 512, 128, 1, (1, 1), (131071, 131071)),
        # A prompt's chunk in a sliding layer, after an earlier part of the prompt.
        _case("chunk_window", "attend", "bf16", 16, 8, 256, 64, 1, (4096, 4096), (4099, 4099), 1024, 4),
        # A prompt's chunk in a global layer over a long earlier part.
        _case("chunk_global", "attend", "bf16", 16, 2, 512, 128, 1, (2048, 2048), (16384, 16384)),
        # Prompts of several users from their first token, full attention, head width 256.
        _case("prompts_256", "attend", "bf16", 16, 8, 256, 32, 4, (1500, 4100), (0, 0)),
        # Chunks of many users beside single tokens in one call, over an 8-bit cache.
        _case("mixed_e4m3", "attend", "e4m3", 32, 8, 128, 32, 24, (1, 700), (5, 5000)),
        # A decode step's new tokens into the 8-bit cache.
        _case("write_decode_e4m3", "write", "e4m3", 16, 8, 256, 64, 64, (1, 1), (1, 900)),
        # Whole prompts into the 8-bit cache.
        _case("write_prompt_e4m3", "write", "e4m3", 16, 8, 256, 16, 8, (500, 9001), (0, 0)),
        # A few short contexts read back.
        _case("read_short_bf16", "read", "bf16", 16, 2, 512, 32, 3, (17, 201), (0, 0)),
        # Whole contexts out of the 8-bit cache, as for moving or sharing a prefix.
        _case("read_e4m3", "read", "e4m3", 16, 8, 256, 64, 32, (300, 5001), (0, 0)),
    ]


def _case(name, op, fmt, hq, hkv, d, page, seqs, new, old, window=0, sinks=0):
    return {"name": name, "op": op, "fmt": fmt, "hq": hq, "hkv": hkv, "d": d, "page": page, "seqs": seqs,
            "new_lo": new[0], "new_hi": new[1], "old_lo": old[0], "old_hi": old[1], "window": window, "sinks": sinks}


def draw(rng):
    def log(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))

    op = rng.choice(("attend", "attend", "attend", "write", "read"))
    fmt = rng.choice(("bf16", "e4m3"))
    hq, hkv, d = rng.choice(HEADS)
    page = rng.choice((16, 32, 64, 128))
    seqs = log(1, 256)
    # Sizes halve until the case costs no more than the largest listed ones and its plain form fits.
    window, sinks = (0, 0)
    if op == "attend":
        window = rng.choice((0, 0, log(1, 5000), 1024))
        sinks = rng.choice((0, 4, log(1, 300))) if window else 0
        new_hi = rng.choice((1, 1, log(2, 16), log(16, 4096)))
        old_hi = log(1, 131072)
        old_lo = log(1, old_hi)
        new_lo = log(1, new_hi)
    else:
        new_hi = log(1, 16384)
        new_lo = log(1, new_hi)
        old_hi = rng.choice((0, log(1, 4000)))
        old_lo = 0 if old_hi == 0 else log(1, old_hi)
    case = _case("", op, fmt, hq, hkv, d, page, seqs, (new_lo, new_hi), (old_lo, old_hi), window, sinks)
    del case["name"]
    while not _affordable(case):
        key = max(("seqs", "new_hi", "old_hi"), key=lambda k: case[k] if k != "seqs" else 64 * case[k])
        case[key] = max(1, case[key] * 2 // 3)
        case["new_lo"] = min(case["new_lo"], case["new_hi"])
        case["old_lo"] = min(case["old_lo"], case["old_hi"])
    return case


def _affordable(c):
    w = work(c)
    new, kv = _lengths(c)
    padded = c["seqs"] * max(kv) * c["hkv"] * c["d"]
    scores = c["seqs"] * max(new) * max(kv) * c["hq"] if c["op"] == "attend" else 0
    return w["flops"] <= 1.1e12 and w["bytes"] <= 1.1e9 and padded <= 1 << 31 and scores <= 1 << 30


def _spread(lo, hi, n, step):
    """n lengths from lo to hi, evenly spaced on a log scale (from 0: all equal), in a mixed order."""
    if lo == hi or n == 1:
        return [hi] * n
    at = [int(round(math.exp(math.log(max(lo, 1)) + (math.log(hi) - math.log(max(lo, 1))) * i / (n - 1))))
          for i in range(n)]
    return [at[i * step % n] for i in range(n)] if math.gcd(step, n) == 1 else at


def _lengths(c):
    """Each sequence's new tokens, and all its cached tokens with them."""
    new = _spread(c["new_lo"], c["new_hi"], c["seqs"], 7)
    old = _spread(c["old_lo"], c["old_hi"], c["seqs"], 11)
    return new, [a + b for a, b in zip(new, old)]


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    new, kv = _lengths(c)
    n_pages_of = [-(-n // c["page"]) for n in kv]
    used = sum(n_pages_of)
    n_pages = used + used // 8 + 3  # some pages belong to nobody
    order = torch.randperm(n_pages, generator=gen, device="cuda", dtype=torch.int64).to(torch.int32)
    width = max(n_pages_of)
    count = torch.tensor(n_pages_of, device="cuda").view(-1, 1)
    first = count.cumsum(0) - count
    col = torch.arange(width, device="cuda").view(1, -1)
    pages = torch.where(col < count, order[(first + col).clamp(max=n_pages - 1)], torch.full_like(order[:1], -1))
    cu = torch.zeros(c["seqs"] + 1, dtype=torch.int32)
    cu[1:] = torch.tensor(new).cumsum(0)
    T = int(cu[-1])
    s = {"case": c, "pages": pages.contiguous(), "cu_q": cu.cuda(), "kv_len": torch.tensor(kv, dtype=torch.int32).cuda(),
         "n_pages": n_pages, "max_new": max(new), "max_kv": max(kv), "tokens": T}
    shape = (n_pages, c["hkv"], c["page"], c["d"])
    if c["op"] == "write":
        # Keys and values as they leave the projections: a view of one fused row per token, with a
        # few channels of large magnitude.
        width = c["hkv"] * c["d"]
        fused = torch.randn(T, 2 * width, generator=gen, device="cuda", dtype=torch.bfloat16)
        fused[:, ::61] *= 8
        s["k"], s["v"] = (t.view(T, c["hkv"], c["d"]) for t in fused.split(width, 1))
        dtype = torch.bfloat16 if c["fmt"] == "bf16" else torch.float8_e4m3fn
        s["cache"] = {n: torch.zeros(shape, dtype=dtype, device="cuda") for n in ("k", "v")}
        if c["fmt"] == "e4m3":
            s["cache"].update({n: torch.zeros(shape[:3], device="cuda") for n in ("k_scale", "v_scale")})
    else:
        s["cache"] = {}
        for n in ("k", "v"):
            x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16)
            if c["fmt"] == "bf16":
                s["cache"][n] = x
            else:
                s["cache"][n], s["cache"][n + "_scale"] = _quantise(x)
            del x
        # Gains between 1 and 2.5 on the queries: heads that attend broadly and heads that pick out.
        gain = torch.linspace(1.0, 2.5, c["hq"], device="cuda").view(1, -1, 1)
        q = torch.randn(T, c["hq"], c["d"], generator=gen, device="cuda") * gain
        s["q"] = q.to(torch.bfloat16)
    if own:
        from mixture_experts_ffn_router_gb300 import binding as B
        s["kv"] = B.PagedKV(c["hq"], c["hkv"], c["d"], c["page"], n_pages, c["fmt"], max_tokens=T, max_seqs=c["seqs"])
        s["batch"] = B.KVBatch(s["cu_q"], s["kv_len"], s["pages"], max_new=s["max_new"])
        s["layer"] = s["kv"].cache(**s["cache"])
    return s


def run(state):
    c = state["case"]
    if own:
        kv, layer, batch = state["kv"], state["layer"], state["batch"]
        if c["op"] == "write":
            kv.write(layer, batch, state["k"], state["v"])
            return state["cache"]
        if c["op"] == "read":
            k, v = kv.read(layer, batch, state["tokens"])
            return {"k": k, "v": v}
        out, lse = kv.attention(layer, batch, state["q"], window=c["window"], sinks=c["sinks"])
        return {"out": out, "lse": lse}
    return {"write": _write, "read": _read, "attend": _attend}[c["op"]](state)


# ------------------------------------------------------------------ the plain form

def _quantise(x):
    """e4m3 codes and fp32 scales of rows: the largest magnitude becomes 448; a zero row keeps scale 0."""
    x = x.float()
    scale = x.abs().amax(-1) / E4M3_MAX
    codes = torch.where(scale[..., None] > 0, x / scale[..., None], torch.zeros_like(x))
    return codes.to(torch.float8_e4m3fn), scale


def _places(s):
    """(page, slot) of every new token, in the order of the rows."""
    row = torch.arange(s["tokens"], device="cuda", dtype=torch.int32)
    seq = torch.searchsorted(s["cu_q"], row, right=True) - 1
    pos = s["kv_len"][seq].long() - s["cu_q"][seq + 1].long() + row
    P = s["case"]["page"]
    return s["pages"][seq, pos // P].long(), pos % P


def _write(s):
    page, slot = _places(s)
    cache = s["cache"]
    for n in ("k", "v"):
        if s["case"]["fmt"] == "bf16":
            cache[n][page, :, slot] = s[n]
        else:
            codes, scale = _quantise(s[n])
            cache[n].view(torch.uint8)[page, :, slot] = codes.view(torch.uint8)
            cache[n + "_scale"][page, :, slot] = scale
    return cache


def _values(s, n, at):
    """The cached values of K or V at the places `at`, in fp32."""
    x = s["cache"][n].view(torch.uint8 if s["case"]["fmt"] == "e4m3" else torch.bfloat16)[at]
    if s["case"]["fmt"] == "bf16":
        return x.float()
    return x.view(torch.float8_e4m3fn).float() * s["cache"][n + "_scale"][at][..., None]


def _read(s):
    page, slot = _places(s)
    at = (page, slice(None), slot)
    return {n: _values(s, n, at).to(torch.bfloat16) for n in ("k", "v")}


def _attend(s):
    c = s["case"]
    B, Q, L, P, hkv, d = c["seqs"], s["max_new"], s["max_kv"], c["page"], c["hkv"], c["d"]
    g = c["hq"] // hkv
    j = torch.arange(L, device="cuda")
    page = s["pages"][:, j // P].long().clamp(min=0)                       # [B, L]
    at = (page, slice(None), (j % P).expand(B, L))
    used = (j < s["kv_len"].view(-1, 1)).view(B, 1, L, 1)
    k, v = (torch.where(used, _values(s, n, at).transpose(1, 2), 0.0) for n in ("k", "v"))  # [B, hkv, L, d]
    i = torch.arange(Q, device="cuda").view(1, -1)
    cu = s["cu_q"].long()
    count = (cu[1:] - cu[:-1]).view(-1, 1)
    row = (cu[:-1].view(-1, 1) + i).clamp(max=s["tokens"] - 1)             # [B, Q]
    q = s["q"][row].float().view(B, Q, hkv, g, d).permute(0, 2, 3, 1, 4).reshape(B, hkv, g * Q, d)
    x = (q @ k.transpose(2, 3)).mul_(d ** -0.5).view(B, hkv, g, Q, L)
    p = (s["kv_len"].view(-1, 1) - count + i).view(B, 1, 1, Q, 1)
    seen = (j <= p) & (p >= 0)
    if c["window"]:
        seen &= (j > p - c["window"]) | (j < c["sinks"])
    x.masked_fill_(~seen, -math.inf)
    top = x.amax(-1, keepdim=True).clamp(min=-3e38)
    x = x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    out = (x.view(B, hkv, g * Q, L) @ v).view(B, hkv, g, Q, d) / total.clamp(min=1e-38)
    lse = (top + total.log())[..., 0]
    live = i < count                                                        # [B, Q]
    out = out.permute(0, 3, 1, 2, 4).reshape(B, Q, c["hq"], d)[live].to(torch.bfloat16)
    return {"out": out, "lse": lse.permute(0, 3, 1, 2).reshape(B, Q, c["hq"])[live]}


# ------------------------------------------------------------------ work and exact values

def work(case):
    c = case
    new, kv = _lengths(c)
    T, row = sum(new), 2 * c["d"] * FMT_BYTES[c["fmt"]] + (8 if c["fmt"] == "e4m3" else 0)
    if c["op"] != "attend":
        return {"bytes": T * c["hkv"] * (row + 4 * c["d"]), "flops": 0}
    keys = pairs = 0
    W, S = c["window"], c["sinks"]
    for n, L in zip(new, kv):
        first = L - n
        if not W:
            keys += L
            pairs += n * first + n * (n + 1) // 2
            continue
        lo = max(0, first - W + 1)                       # the oldest key inside any window
        keys += L - lo + min(S, lo)
        full = min(n, max(0, W - 1 - first))             # rows whose window reaches back to key 0
        pairs += full * (first + 1) + full * (full - 1) // 2 + (n - full) * W
        # The sinks below the window's lower end p - W + 1, over the remaining rows.
        p0, p1 = first + full, L - 1
        a, b = p0 - W + 1, p1 - W + 1
        if n > full and S:
            ramp = max(0, min(b, S) - a + 1) if a <= S else 0
            pairs += sum(range(a, a + ramp)) + (b - a + 1 - ramp) * S
    rows = T * c["hq"]
    return {"bytes": keys * c["hkv"] * row + rows * (4 * c["d"] + 4), "flops": 4 * c["d"] * pairs * c["hq"]}


def exact(case, seed):
    """The operators' definitions in 64 bits, sequence by sequence and head by head."""
    if work(case)["flops"] > 1.3e12:
        return None
    s = prepare(case, seed)
    c, P = s["case"], case["page"]
    cu, kv_len, table = s["cu_q"].tolist(), s["kv_len"].tolist(), s["pages"].cpu()

    def stored(n, seq, lo, hi, head):
        pos = torch.arange(lo, hi)
        page, slot = table[seq][pos // P].long().cuda(), (pos % P).cuda()
        x = s["cache"][n][:, head].reshape(-1, c["d"]).view(torch.uint8 if c["fmt"] == "e4m3" else torch.bfloat16)
        x = x[page * P + slot]
        if c["fmt"] == "bf16":
            return x.double()
        return x.view(torch.float8_e4m3fn).double() * s["cache"][n + "_scale"][page, head, slot].double()[:, None]

    if c["op"] == "write":
        got = {n: t.double() for n, t in s["cache"].items()}
        for b in range(c["seqs"]):
            n = cu[b + 1] - cu[b]
            pos = torch.arange(kv_len[b] - n, kv_len[b])
            page, slot = table[b][pos // P].long().cuda(), (pos % P).cuda()
            for name in ("k", "v"):
                x = s[name][cu[b]:cu[b + 1]].double()
                if c["fmt"] == "e4m3":
                    scale = x.abs().amax(-1) / E4M3_MAX
                    got[name + "_scale"][page, :, slot] = scale
                    x = x / scale[..., None]
                got[name][page, :, slot] = x
        return got
    if c["op"] == "read":
        out = {n: torch.empty(s["tokens"], c["hkv"], c["d"], dtype=torch.float64, device="cuda") for n in ("k", "v")}
        for b in range(c["seqs"]):
            for h in range(c["hkv"]):
                for n in out:
                    out[n][cu[b]:cu[b + 1], h] = stored(n, b, kv_len[b] - (cu[b + 1] - cu[b]), kv_len[b], h)
        return out
    g = c["hq"] // c["hkv"]
    out = torch.zeros(s["tokens"], c["hq"], c["d"], dtype=torch.float64, device="cuda")
    lse = torch.full((s["tokens"], c["hq"]), -math.inf, dtype=torch.float64, device="cuda")
    for b in range(c["seqs"]):
        n, L = cu[b + 1] - cu[b], kv_len[b]
        key = torch.arange(L, device="cuda")
        pos = torch.arange(L - n, L, device="cuda")[:, None]
        hidden = key[None] > pos
        if c["window"]:
            hidden |= (pos - key[None] >= c["window"]) & (key[None] >= c["sinks"])
        for h in range(c["hkv"]):
            k, v = stored("k", b, 0, L, h), stored("v", b, 0, L, h)
            for hq in range(h * g, h * g + g):
                x = s["q"][cu[b]:cu[b + 1], hq].double() @ k.T / math.sqrt(c["d"])
                x[hidden] = -math.inf
                lse[cu[b]:cu[b + 1], hq] = torch.logsumexp(x, -1)
                out[cu[b]:cu[b + 1], hq] = torch.softmax(x, -1) @ v
    return {"out": out, "lse": lse}
