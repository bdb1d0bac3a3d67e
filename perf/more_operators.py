"""The token mixing of a layer, between its q|k|v projections and the output projection, as cases to
measure: rotating and appending keys and values to a paged cache, attention over that cache for a batch
that shares a prefix, and linear attention with a decay for each head.

`run` computes a case in plain torch operations (fp32, rounded once at the end), or, when `own` is
set, through the library's calls.  `exact` gives the same outputs from the definitions in float64.
"""
import math

import torch

own = False


# ----------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------
def listed():
    return [
        # one request in decode: the new token of a layer with 32 query and 8 key heads, from one fused projection
        {"name": "append 1 token", "op": "append", "M": 1, "q_heads": 32, "kv_heads": 8, "dim": 128, "rot": 128,
         "interleaved": False, "page": 64, "bf16": False, "prompt": False},
        # a decode batch, some rows padding; half of each head rotated, in neighbouring pairs
        {"name": "append 64 tokens", "op": "append", "M": 64, "q_heads": 16, "kv_heads": 2, "dim": 256, "rot": 128,
         "interleaved": True, "page": 16, "bf16": True, "prompt": False},
        # a long prompt, behind normalised heads (bf16)
        {"name": "append 4001 prompt tokens", "op": "append", "M": 4001, "q_heads": 32, "kv_heads": 8, "dim": 128,
         "rot": 128, "interleaved": False, "page": 64, "bf16": True, "prompt": True},
        # one request in decode, nothing shared
        {"name": "attention 1 token of 777", "op": "attention", "seqs": 1, "q": 1, "ragged_q": False, "own": 777,
         "prefix": 0, "q_heads": 32, "kv_heads": 8, "dim": 128, "page": 64, "int8": False},
        # a decode batch behind one system prompt, each request with a turn of its own
        {"name": "attention 64 tokens shared", "op": "attention", "seqs": 64, "q": 1, "ragged_q": False, "own": 2000,
         "prefix": 8192, "q_heads": 32, "kv_heads": 8, "dim": 128, "page": 64, "int8": False},
        # verify windows of up to four drafted tokens over an 8-bit cache, seven query heads a key head
        {"name": "attention 16 windows int8", "op": "attention", "seqs": 16, "q": 4, "ragged_q": True, "own": 9001,
         "prefix": 1000, "q_heads": 28, "kv_heads": 4, "dim": 128, "page": 16, "int8": True},
        # the prompts of five requests behind a shared prefix, narrow heads
        {"name": "attention 5 prompts shared", "op": "attention", "seqs": 5, "q": 700, "ragged_q": True, "own": 700,
         "prefix": 2500, "q_heads": 16, "kv_heads": 4, "dim": 64, "page": 64, "int8": False},
        # the last piece of a long prompt
        {"name": "attention 4096 prompt tokens", "op": "attention", "seqs": 1, "q": 4096, "ragged_q": False, "own": 12288,
         "prefix": 4096, "q_heads": 32, "kv_heads": 8, "dim": 128, "page": 64, "int8": False},
        # one request in decode: 32 states of 128 x 128, a decay from the token
        {"name": "linear 1 token", "op": "linear", "seqs": 1, "T": 1, "ragged": False, "k_heads": 16, "v_heads": 32,
         "dk": 128, "dv": 128, "by_token": True},
        # a decode batch
        {"name": "linear 64 tokens", "op": "linear", "seqs": 64, "T": 1, "ragged": False, "k_heads": 16, "v_heads": 32,
         "dk": 128, "dv": 128, "by_token": True},
        # three prompts, no whole number of chunks
        {"name": "linear 3 prompts", "op": "linear", "seqs": 3, "T": 333, "ragged": True, "k_heads": 8, "v_heads": 8,
         "dk": 64, "dv": 128, "by_token": False},
        # one long prompt
        {"name": "linear 4096 prompt tokens", "op": "linear", "seqs": 1, "T": 4096, "ragged": False, "k_heads": 16,
         "v_heads": 32, "dk": 128, "dv": 128, "by_token": True},
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attention", "attention", "attention", "linear", "linear"])
    if op == "append":
        kv_heads, dim = rng.choice([1, 2, 4, 5, 8]), rng.choice([64, 128, 256])
        heads = kv_heads * rng.choice([1, 2, 4, 7])
        M = _log_uniform(rng, 1, max(1, min(8192, 4001 * 48 * 128 // ((heads + 2 * kv_heads) * dim))))
        return {"op": "append", "M": M, "q_heads": heads, "kv_heads": kv_heads, "dim": dim,
                "rot": rng.choice([dim, dim, dim // 2, dim // 4]), "interleaved": rng.random() < 0.3,
                "page": rng.choice([16, 32, 64, 256]), "bf16": rng.random() < 0.5, "prompt": M > 16 and rng.random() < 0.6}
    if op == "attention":
        kv_heads, dim = rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 128, 256])
        heads = kv_heads * rng.choice([1, 2, 4, 5, 8])
        kind = rng.choice(["decode", "decode", "window", "prompt"])
        q = {"decode": 1, "window": rng.randint(2, 8), "prompt": _log_uniform(rng, 16, 4096)}[kind]
        most = 4096 * 32 * 8192 * 128 // (heads * dim)      # rows and keys of the largest case, with room to spare
        seqs = _log_uniform(rng, 1, max(1, min(256, 8192 // q)))
        mine = q + _log_uniform(rng, 1, max(2, min(16384, most // (seqs * q), (1 << 30) // (seqs * kv_heads * dim)) - q))
        prefix = rng.choice([0, 1, 1]) * _log_uniform(rng, 1, max(2, min(16384, most // (seqs * q))))
        return {"op": "attention", "seqs": seqs, "q": q, "ragged_q": q > 1 and rng.random() < 0.6, "own": mine,
                "prefix": prefix, "q_heads": heads, "kv_heads": kv_heads, "dim": dim,
                "page": rng.choice([16, 32, 64, 256]), "int8": rng.random() < 0.3}
    k_heads = rng.choice([1, 2, 4, 8, 16])
    v_heads = k_heads * rng.choice([1, 2])
    T = 1 if rng.random() < 0.4 else _log_uniform(rng, 2, 4096)
    return {"op": "linear", "seqs": _log_uniform(rng, 1, max(1, min(256, 4096 // T))), "T": T, "ragged": T > 1 and rng.random() < 0.6,
            "k_heads": k_heads, "v_heads": v_heads, "dk": rng.choice([64, 128]), "dv": rng.choice([64, 128]),
            "by_token": rng.random() < 0.7}


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------
# The cache's pages, in the order that its matrix products read: keys [page][head][token/16][dim/8][16][8],
# values [page][head][token/8][dim][8]; an 8-bit cache has a scale for each token and head beside its codes.
def _key_shape(pages, heads, page, dim):
    return pages, heads, page // 16, dim // 8, 16, 8


def _value_shape(pages, heads, page, dim):
    return pages, heads, page // 8, dim, 8


def _inputs(case, seed):
    """The case's input tensors from the seed alone."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device="cuda") * std

    def uniform(*shape):
        return torch.rand(*shape, generator=g, device="cuda")

    def integers(lo, hi, *shape):
        return torch.randint(lo, hi, shape, generator=g, device="cuda", dtype=torch.int32)

    def lengths(n, most, ragged):
        return integers(max(1, most // 4), most + 1, n) if ragged else torch.full((n,), most, device="cuda", dtype=torch.int32)

    def starts(lens):
        return torch.cat([torch.zeros(1, device="cuda", dtype=torch.int32), torch.cumsum(lens, 0).to(torch.int32)])

    if case["op"] == "append":
        M, H, KH, D, page = case["M"], case["q_heads"], case["kv_heads"], case["dim"], case["page"]
        pages = -(-M // page) + 3
        if case["prompt"]:      # one request's next tokens, in pages that lie anywhere
            first = integers(0, page, 1)
            at = first + torch.arange(M, device="cuda", dtype=torch.int32)
            table = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
            slots = table[at // page] * page + at % page
            pos = integers(0, 30000, 1) // page * page + at
        else:                   # a token of each request; one row in 16 is padding
            slots = torch.randperm(pages * page, generator=g, device="cuda")[:M].to(torch.int32)
            if M > 1:
                slots = torch.where(uniform(M) < 1 / 16, -1, slots)
            pos = integers(0, 40960, M)
        x = normal(M, (H + 2 * KH) * D)
        x[:, : H * D : 37] *= 8
        s = {"inv_freq": 1e6 ** (-torch.arange(case["rot"] // 2, device="cuda", dtype=torch.float32) * 2 / case["rot"]),
             "slots": slots, "pos": pos.to(torch.int32), "pages": pages,
             "key": normal(*_key_shape(pages, KH, page, D)).bfloat16(),
             "value": normal(*_value_shape(pages, KH, page, D)).bfloat16(),
             "q_out": torch.empty(M, H, D, device="cuda", dtype=torch.bfloat16)}
        s["q"], s["k"], s["v"] = x[:, : H * D], x[:, H * D : (H + KH) * D], x[:, (H + KH) * D :]
        if case["bf16"]:        # heads that were normalised on the way; values as the projection wrote them
            s["q"], s["k"] = s["q"].contiguous().bfloat16(), s["k"].contiguous().bfloat16()
        return s
    if case["op"] == "attention":
        n, H, KH, D, page, P = (case[k] for k in ("seqs", "q_heads", "kv_heads", "dim", "page", "prefix"))
        q_len = lengths(n, case["q"], case["ragged_q"])
        own_len = q_len + lengths(n, case["own"] - case["q"], n > 1) if case["own"] > case["q"] else q_len.clone()
        cols, shared = -(-case["own"] // page), -(-P // page)
        pages = n * cols + shared
        order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        M = n * case["q"]       # rows behind the last sequence are padding
        s = {"q": (normal(M, H, D) * 2).bfloat16(), "q_start": starts(q_len), "own_len": own_len,
             "table": order[: n * cols].view(n, cols).contiguous(), "shared": order[n * cols :].contiguous(),
             "pages": pages, "M": M, "out": torch.zeros(M, H, D, device="cuda", dtype=torch.bfloat16)}
        for name, shape in (("key", _key_shape), ("value", _value_shape)):
            x = normal(*shape(pages, KH, page, D))
            if case["int8"]:
                s[name] = (x * 42).round_().clamp_(-127, 127).to(torch.int8)
                s[name + "_scale"] = (0.5 + uniform(pages, KH, page)) / 42
            else:
                s[name] = x.bfloat16()
        return s
    n, KH, H, dk, dv = (case[k] for k in ("seqs", "k_heads", "v_heads", "dk", "dv"))
    M = n * case["T"]
    s = {"q": normal(M, KH, dk).bfloat16(), "k": normal(M, KH, dk, std=dk ** -0.5).bfloat16(), "v": normal(M, H, dv).bfloat16(),
         "q_start": starts(lengths(n, case["T"], case["ragged"])), "M": M,
         "slots": torch.randperm(n + 2, generator=g, device="cuda")[:n].to(torch.int32),
         # a decode step goes on, a prompt may begin a sequence
         "fresh": (uniform(n) < (0.3 if case["T"] > 1 else 0.0)).to(torch.int32), "state": normal(n + 2, H, dk, dv),
         "state_out": torch.zeros(n + 2, H, dk, dv, device="cuda"), "out": torch.zeros(M, H, dv, device="cuda")}
    slow = torch.exp(-1 - 6 * uniform(H))       # what a head forgets a token, from a third to a thousandth
    s["decay"] = -slow * torch.exp(normal(M, H, std=0.5)) if case["by_token"] else -slow
    return s


def _sequence_of(s):
    """Of each row its sequence and its place there; rows behind the last sequence get -1."""
    at, start = torch.arange(s["M"], device="cuda"), s["q_start"].long()
    seq = torch.searchsorted(start, at, right=True) - 1
    inside = at < start[-1]
    return torch.where(inside, seq, -1), at - start[seq.clamp(max=len(start) - 2)], inside


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if own:
        import gemm_q4nx_chunk_amd as q
        if case["op"] == "append":
            s["cache"] = q.kv_cache(case["kv_heads"], case["dim"], case["page"], s["pages"], s["key"], s["value"])
            s["rope"] = q.rope(s["inv_freq"], s["pos"], case["rot"], interleaved=case["interleaved"])
        elif case["op"] == "attention":
            s["cache"] = q.kv_cache(case["kv_heads"], case["dim"], case["page"], s["pages"], s["key"], s["value"],
                                    k_scale=s.get("key_scale"), v_scale=s.get("value_scale"))
            s["batch"] = q.attn_batch(s["q_start"], s["own_len"], s["table"], case["q"], prefix_len=case["prefix"],
                                      prefix_pages=s["shared"])
            s["ws"] = torch.empty(q.attention_ws(s["cache"], s["batch"], case["q_heads"], s["M"]), dtype=torch.uint8, device="cuda")
        else:
            s["args"] = q.linear_attn_seqs(s["q_start"], s["slots"], case["T"], fresh=s["fresh"])
            s["ws"] = torch.empty(q.linear_attn_ws(s["args"], case["k_heads"], case["v_heads"], case["dk"], case["dv"], s["M"]),
                                  dtype=torch.uint8, device="cuda")
    return s


# ----------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------
def run(state):
    op = state["case"]["op"]
    if own:
        return {"append": _own_append, "attention": _own_attention, "linear": _own_linear}[op](state)
    return {"append": _plain_append, "attention": _plain_attention, "linear": _plain_linear}[op](state)


def _own_append(s):
    import gemm_q4nx_chunk_amd as q
    c = s["case"]
    q.kv_append(s["cache"], s["k"], s["v"], s["slots"], c["M"], rope=s["rope"], q=s["q"], q_heads=c["q_heads"], q_out=s["q_out"])
    return {"q": s["q_out"], "key": s["key"], "value": s["value"]}


def _own_attention(s):
    import gemm_q4nx_chunk_amd as q
    c = s["case"]
    q.attention(s["cache"], s["batch"], s["q"], c["q_heads"], s["M"], c["dim"] ** -0.5, s["out"], s["ws"])
    return s["out"]


def _own_linear(s):
    import gemm_q4nx_chunk_amd as q
    c = s["case"]
    q.linear_attn(s["args"], s["q"], s["k"], s["v"], s["decay"], c["k_heads"], c["v_heads"], c["dk"], c["dv"], s["M"],
                  c["dk"] ** -0.5, s["state"], s["out"], s["ws"], state_out=s["state_out"])
    return {"out": s["out"], "state": s["state_out"]}


def _plain_append(s):
    c = s["case"]
    M, H, KH, D, R, page = c["M"], c["q_heads"], c["kv_heads"], c["dim"], c["rot"], c["page"]
    angle = s["pos"].double()[:, None] * s["inv_freq"].double()[None, :]
    cos, sin = torch.cos(angle).float()[:, None, :], torch.sin(angle).float()[:, None, :]

    def rotated(x, heads):
        x = x.float().reshape(M, heads, D)
        a, b = (x[..., 0:R:2], x[..., 1:R:2]) if c["interleaved"] else (x[..., : R // 2], x[..., R // 2 : R])
        a, b = a * cos - b * sin, b * cos + a * sin
        turned = torch.stack([a, b], -1).flatten(2) if c["interleaved"] else torch.cat([a, b], -1)
        return torch.cat([turned, x[..., R:]], -1).bfloat16()

    s["q_out"].copy_(rotated(s["q"], H))
    keep = (s["slots"] >= 0)[:, None, None]
    slot, head, d = s["slots"].long().clamp(min=0)[:, None, None], torch.arange(KH, device="cuda")[None, :, None], torch.arange(D, device="cuda")
    at = ((slot // page) * KH + head) * page * D
    tok = slot % page
    key_at = at + (tok // 16) * 16 * D + (d // 8) * 128 + (tok % 16) * 8 + d % 8
    value_at = at + (tok // 8) * 8 * D + d * 8 + tok % 8
    key, value = s["key"].view(-1), s["value"].view(-1)
    spare = torch.zeros((), dtype=torch.bfloat16, device="cuda")
    for_key, for_value = rotated(s["k"], KH), s["v"].reshape(M, KH, D).bfloat16()
    # what belongs to a padding row goes past the end
    more_key, more_value = torch.cat([key, spare[None]]), torch.cat([value, spare[None]])
    more_key[torch.where(keep, key_at, key.numel())] = for_key
    more_value[torch.where(keep, value_at, value.numel())] = for_value
    key.copy_(more_key[:-1])
    value.copy_(more_value[:-1])
    return {"q": s["q_out"], "key": s["key"], "value": s["value"]}


def _plain_keys_values(s, table):
    """The cached keys and values of a table of pages, fp32 [..., heads, tokens, dim]."""
    lead, t = table.shape[:-1], table.long()
    KH, D = s["case"]["kv_heads"], s["case"]["dim"]
    k, v = s["key"][t].float(), s["value"][t].float()
    if s["case"]["int8"]:
        k = k * s["key_scale"][t].unflatten(-1, (-1, 1, 16, 1))
        v = v * s["value_scale"][t].unflatten(-1, (-1, 1, 8))
    n = len(lead)
    k = k.permute(*range(n), n + 1, n, n + 2, n + 4, n + 3, n + 5).reshape(*lead, KH, -1, D)
    v = v.permute(*range(n), n + 1, n, n + 2, n + 4, n + 3).reshape(*lead, KH, -1, D)
    return k, v


def _plain_part(q, k, v, seen):
    """Maximum, sum and weighted values of the keys that are seen."""
    z = torch.where(seen, q @ k.transpose(-1, -2), float("-inf"))
    m = z.amax(-1, keepdim=True)
    e = torch.exp(z - torch.where(m > float("-inf"), m, 0.0))
    return m, e.sum(-1, keepdim=True), e @ v


def _plain_attention(s):
    """The shared prefix with all rows at once, each sequence's own keys with its rows, and the two joined."""
    c = s["case"]
    n, H, KH, D, M = c["seqs"], c["q_heads"], c["kv_heads"], c["dim"], s["M"]
    group = H // KH
    seq, place, inside = _sequence_of(s)
    rows = s["q"].float().view(M, KH, group, D) * D ** -0.5
    q_len, own_len = (s["q_start"][1:] - s["q_start"][:-1]).long(), s["own_len"].long()
    at = s["q_start"][:-1].long()[:, None] + torch.arange(c["q"], device="cuda")[None, :]     # [n, q]
    mine = rows[at.clamp(max=M - 1)].permute(0, 2, 1, 3, 4).reshape(n, KH, c["q"] * group, D)
    k, v = _plain_keys_values(s, s["table"])
    last = own_len[:, None] - q_len[:, None] + torch.arange(c["q"], device="cuda")[None, :]
    last = last[:, :, None].expand(n, c["q"], group).reshape(n, 1, -1, 1)
    place_k = torch.arange(k.shape[2], device="cuda")
    seen = (place_k <= last) & (place_k < own_len[:, None, None, None])
    pick = (seq.clamp(min=0), place.clamp(0, c["q"] - 1))
    m, l, o = (x.view(n, KH, c["q"], group, -1).permute(0, 2, 1, 3, 4)[pick] for x in _plain_part(mine, k, v, seen))
    if c["prefix"]:
        k, v = _plain_keys_values(s, s["shared"])
        seen = torch.arange(k.shape[1], device="cuda") < c["prefix"]
        m2, l2, o2 = (x.view(KH, M, group, -1).transpose(0, 1) for x in _plain_part(rows.transpose(0, 1).reshape(KH, M * group, D), k, v, seen))
        top = torch.maximum(m, m2)
        a, b = torch.exp(m - top), torch.exp(m2 - top)
        l, o = a * l + b * l2, a * o + b * o2
    s["out"].copy_(torch.where(inside[:, None, None], (o / l).reshape(M, H, D), 0.0))
    return s["out"]


def _plain_linear(s):
    """Every row with every row before it in its sequence, and with the state that the sequence began with."""
    c = s["case"]
    n, KH, H, dk, dv, M = c["seqs"], c["k_heads"], c["v_heads"], c["dk"], c["dv"], s["M"]
    seq, _, inside = _sequence_of(s)
    q, k = (s[x].float().repeat_interleave(H // KH, 1).transpose(0, 1) * f for x, f in (("q", dk ** -0.5), ("k", 1.0)))
    v = s["v"].float().transpose(0, 1)
    total = torch.cumsum(s["decay"].double().expand(M, H), 0).t().contiguous()       # [H, M]
    before = torch.cat([torch.zeros(H, 1, dtype=torch.float64, device="cuda"), total], 1)
    first, last = s["q_start"][:-1].long(), s["q_start"][1:].long()
    at = torch.arange(M, device="cuda")
    sees = (seq[:, None] == seq[None, :]) & (at[:, None] >= at[None, :]) & inside[:, None]
    weight = torch.exp(torch.where(sees, total[:, :, None] - total[:, None, :], float("-inf")).float())
    start = torch.where(s["fresh"].bool()[:, None, None, None], 0.0, s["state"][s["slots"].long()])   # [n, H, dk, dv]
    out = ((q @ k.transpose(1, 2)) * weight) @ v
    own_seq = seq.clamp(min=0)
    since = torch.exp((total - before[:, first][:, own_seq]).float())                # [H, M]
    # each row's product with its sequence's state, over a row's sequences padded to the longest
    to = first[:, None] + torch.arange(c["T"], device="cuda")[None, :]
    padded = q[:, to.clamp(max=M - 1)].transpose(0, 1) @ start                       # [n, H, T, dv]
    out += since[:, :, None] * padded[own_seq, :, (at - first[own_seq]).clamp(0, c["T"] - 1)].transpose(0, 1)
    s["out"].copy_(torch.where(inside[:, None, None], out.transpose(0, 1), 0.0))
    in_seq = to < last[:, None]                                                      # [n, T]
    left = before[:, last][:, :, None] - total[:, to.clamp(max=M - 1)]               # [H, n, T]
    left = torch.exp(torch.where(in_seq[None], left, float("-inf")).float()).transpose(0, 1)     # [n, H, T]
    ks, vs = (x[:, to.clamp(max=M - 1)].transpose(0, 1) for x in (k, v))
    kept = torch.exp((before[:, last] - before[:, first]).float()).t()[:, :, None, None]
    s["state_out"][s["slots"].long()] = kept * start + (ks * left[..., None]).transpose(2, 3) @ vs
    return {"out": s["out"], "state": s["state_out"]}


# ----------------------------------------------------------------------------
# the definitions in 64 bits
# ----------------------------------------------------------------------------
def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "append":
        M, D, R, page = case["M"], case["dim"], case["rot"], case["page"]
        turn = torch.polar(torch.ones(M, R // 2, dtype=torch.float64, device="cuda"), s["pos"].double()[:, None] * s["inv_freq"].double())
        first = torch.arange(R // 2, device="cuda") * (2 if case["interleaved"] else 1)
        second = first + (1 if case["interleaved"] else R // 2)

        def rotated(x, heads):
            x = x.double().reshape(M, heads, D)
            z = torch.complex(x[..., first], x[..., second]) * turn[:, None, :]
            y = x.clone()
            y[..., first], y[..., second] = z.real, z.imag
            return y
        key, value = s["key"].double(), s["value"].double()
        k, v = rotated(s["k"], case["kv_heads"]), s["v"].double().reshape(M, case["kv_heads"], D)
        kept = (s["slots"] >= 0).nonzero()[:, 0]
        where, tok = s["slots"][kept].long() // page, s["slots"][kept].long() % page
        key.permute(0, 2, 4, 1, 3, 5)[where, tok // 16, tok % 16] = k[kept].unflatten(-1, (-1, 8))
        value.permute(0, 2, 4, 1, 3)[where, tok // 8, tok % 8] = v[kept]
        return {"q": rotated(s["q"], case["q_heads"]), "key": key, "value": value}
    if case["op"] == "attention":
        P, KH, D = case["prefix"], case["kv_heads"], case["dim"]
        group, out = case["q_heads"] // KH, torch.zeros(s["M"], case["q_heads"], D, dtype=torch.float64, device="cuda")
        q_start, own_len = s["q_start"].tolist(), s["own_len"].tolist()
        pages = {}
        for name, order in (("key", (0, 2, 4, 3, 5)), ("value", (0, 1, 3, 2))):
            def head_of(table, h, name=name, order=order):
                x = s[name][table.long(), h].double()
                if case["int8"]:
                    d = s[name + "_scale"][table.long(), h].double()
                    x = x * (d.unflatten(1, (-1, 1, 16, 1)) if name == "key" else d.unflatten(1, (-1, 1, 8)))
                x = x.permute(0, 1, 3, 2, 4) if name == "key" else x.permute(0, 1, 3, 2)
                return x.reshape(-1, D)
            pages[name] = head_of
        for h in range(KH):
            shared = [pages[name](s["shared"], h)[:P] for name in ("key", "value")] if P else None
            for i, have in enumerate(own_len):
                r0, r1 = q_start[i], q_start[i + 1]
                k, v = (pages[name](s["table"][i], h)[:have] for name in ("key", "value"))
                if P:
                    k, v = torch.cat([shared[0], k]), torch.cat([shared[1], v])
                place = torch.arange(k.shape[0], device="cuda") - P
                see = place[None, :] <= (have - (r1 - r0) + torch.arange(r1 - r0, device="cuda"))[:, None]
                for j in range(h * group, (h + 1) * group):
                    z = s["q"][r0:r1, j].double() @ k.t() / math.sqrt(D)
                    out[r0:r1, j] = torch.softmax(z.masked_fill(~see, float("-inf")), 1) @ v
        return out
    # the recurrence itself is too long a loop: in blocks of rows, each from the state before it
    KH, H, M = case["k_heads"], case["v_heads"], s["M"]
    out, state = torch.zeros(M, H, case["dv"], dtype=torch.float64, device="cuda"), s["state_out"].double()
    decay, q_start = s["decay"].double().expand(M, H), s["q_start"].tolist()
    for i, slot in enumerate(s["slots"].tolist()):
        S = s["state"][slot].double() * (0 if s["fresh"][i] else 1)
        for r0 in range(q_start[i], q_start[i + 1], 128):
            r1 = min(r0 + 128, q_start[i + 1])
            C = torch.cumsum(decay[r0:r1], 0).t()                                    # [H, rows]
            q = s["q"][r0:r1].double().repeat_interleave(H // KH, 1).transpose(0, 1) / math.sqrt(case["dk"])
            k = s["k"][r0:r1].double().repeat_interleave(H // KH, 1).transpose(0, 1)
            v = s["v"][r0:r1].double().transpose(0, 1)
            A = torch.tril(torch.exp((C[:, :, None] - C[:, None, :]).clamp(max=0)) * (q @ k.transpose(1, 2)))
            out[r0:r1] = (A @ v + torch.exp(C)[..., None] * (q @ S)).transpose(0, 1)
            S = torch.exp(C[:, -1])[:, None, None] * S + (torch.exp(C[:, -1:] - C)[..., None] * k).transpose(1, 2) @ v
        state[slot] = S
    return {"out": out, "state": state}


# ----------------------------------------------------------------------------
# what a pass cannot do without
# ----------------------------------------------------------------------------
def work(case):
    if case["op"] == "append":
        M, H, KH, D = case["M"], case["q_heads"], case["kv_heads"], case["dim"]
        size = 2 if case["bf16"] else 4
        return {"bytes": M * D * (H * (size + 2) + KH * (size + 4 + 4)) + 8 * M, "flops": 3 * M * (H + KH) * case["rot"]}
    if case["op"] == "attention":
        n, H, KH, D, P = case["seqs"], case["q_heads"], case["kv_heads"], case["dim"], case["prefix"]
        rows = case["q"] * (0.625 if case["ragged_q"] else 1)
        mine = rows + (case["own"] - case["q"]) * (0.625 if n > 1 else 1)
        token = 2 * KH * (D + 4 if case["int8"] else 2 * D)
        return {"bytes": (P + n * mine) * token + 4 * n * rows * H * D, "flops": 4 * n * rows * H * D * (P + mine - (rows - 1) / 2)}
    n, KH, H, dk, dv = (case[k] for k in ("seqs", "k_heads", "v_heads", "dk", "dv"))
    rows = n * case["T"] * (0.625 if case["ragged"] else 1)
    states = n * (2 if case["T"] == 1 else 1.7) * H * dk * dv * 4
    return {"bytes": rows * (4 * KH * dk + 6 * H * dv + (4 * H if case["by_token"] else 0)) + states,
            "flops": 4 * rows * H * dk * dv}
