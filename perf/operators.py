"""The operators of the end of a step, as cases to measure: low-rank adapters beside a shared
projection, the residual addition with its RMS norm, and log probabilities over the head's logits.

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
        # one request in decode: the q, k and v projections of a 2560-wide layer share x
        {"name": "lora 1 row qkv", "op": "lora", "M": 1, "K": 2560, "rows": "4096,1024,1024", "rank": 16,
         "adapters": 8, "mixed": False, "prompt": False},
        # eight requests in decode, each its own adapter of its own rank: gate and up
        {"name": "lora 8 rows gate up", "op": "lora", "M": 8, "K": 2560, "rows": "9728,9728", "rank": 32,
         "adapters": 32, "mixed": True, "prompt": False},
        # a full decode batch over many adapters, some rows with none: the down projection
        {"name": "lora 64 rows down", "op": "lora", "M": 64, "K": 9728, "rows": "2560", "rank": 64,
         "adapters": 64, "mixed": True, "prompt": False},
        # the prompts of seven requests in one call, not a whole number of tiles
        {"name": "lora 1000 rows prompt", "op": "lora", "M": 1000, "K": 4096, "rows": "4096", "rank": 16,
         "adapters": 7, "mixed": False, "prompt": True},
        # the longest prompt call: a wide down projection at a large rank
        {"name": "lora 4096 rows prompt", "op": "lora", "M": 4096, "K": 14336, "rows": "4096", "rank": 64,
         "adapters": 4, "mixed": False, "prompt": True},
        # one decoded token and five alternatives, over a 151936-token vocabulary
        {"name": "logprobs 1 row top 5", "op": "logprobs", "M": 1, "n": 151936, "pad": 0, "tokens": 1, "k": 5,
         "masked": False},
        # a decode batch with twenty alternatives a row
        {"name": "logprobs 64 rows top 20", "op": "logprobs", "M": 64, "n": 151936, "pad": 0, "tokens": 1, "k": 20,
         "masked": False},
        # constrained decoding: most logits are -inf, one row has none left; odd vocabulary, padded rows
        {"name": "logprobs 16 rows masked", "op": "logprobs", "M": 16, "n": 50001, "pad": 6, "tokens": 4, "k": 8,
         "masked": True},
        # scoring prompts: the next token's log probability at every position
        {"name": "logprobs 1000 rows scoring", "op": "logprobs", "M": 1000, "n": 151936, "pad": 0, "tokens": 1,
         "k": 1, "masked": False},
        # between two projections of one decoded token
        {"name": "norm 1 row", "op": "norm", "M": 1, "D": 2560, "residual": True},
        # the q and k head norms of a 64-token prompt block: 40 heads of 128
        {"name": "norm heads", "op": "norm", "M": 2560, "D": 128, "residual": False},
        # a long prompt's residual stream
        {"name": "norm 4096 rows", "op": "norm", "M": 4096, "D": 4096, "residual": True},
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["lora", "lora", "logprobs", "logprobs", "norm"])
    if op == "lora":
        M = _log_uniform(rng, 1, 4096)
        K = 256 * _log_uniform(rng, 1, 56)
        jobs = rng.choice([1, 1, 2, 3])
        rows = [32 * _log_uniform(rng, 2, 128 // jobs if M > 512 else 300) for _ in range(jobs)]
        return {"op": "lora", "M": M, "K": K, "rows": ",".join(map(str, rows)),
                "rank": 8 * _log_uniform(rng, 1, 8 if M > 512 else 16), "adapters": _log_uniform(rng, 1, 8 if M > 512 else 100),
                "mixed": rng.random() < 0.5, "prompt": M > 64 and rng.random() < 0.8}
    if op == "logprobs":
        n = _log_uniform(rng, 1000, 160000)
        M = _log_uniform(rng, 1, max(1, min(4096, 150_000_000 // n)))
        return {"op": "logprobs", "M": M, "n": n, "pad": rng.choice([0, 0, 1, 6, 64]), "tokens": rng.choice([1, 1, 2, 5]),
                "k": rng.choice([0, 1, 3, 5, 10, 20, 32]), "masked": rng.random() < 0.3}
    D = _log_uniform(rng, 64, 8192)
    M = _log_uniform(rng, 1, max(1, min(8192, 4096 * 4096 // D)))
    return {"op": "norm", "M": M, "D": D, "residual": rng.random() < 0.7}


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------
def _inputs(case, seed):
    """The case's input tensors from the seed alone."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device="cuda") * std

    def uniform(*shape):
        return torch.rand(*shape, generator=g, device="cuda")

    if case["op"] == "lora":
        M, K, R, E = case["M"], case["K"], case["rank"], case["adapters"]
        if case["prompt"]:      # runs of rows, one request each
            order = torch.randperm(E, generator=g, device="cuda")
            cuts = torch.sort(torch.randint(0, M + 1, (E - 1,), generator=g, device="cuda")).values
            ids = order[torch.bucketize(torch.arange(M, device="cuda"), cuts, right=True)]
        else:                   # any request's row anywhere; one row in 16 has no adapter
            ids = torch.randint(0, E, (M,), generator=g, device="cuda")
            if M > 1:
                ids = torch.where(uniform(M) < 1 / 16, -1, ids)
        ranks = (torch.randint(1, R + 1, (E,), generator=g, device="cuda") if case["mixed"]
                 else torch.full((E,), R, device="cuda")).to(torch.int32)
        used = torch.arange(R, device="cuda")[None, :] < ranks[:, None]
        s = {"x": normal(M, K).bfloat16(), "ids": ids.to(torch.int32), "ranks": ranks,
             "scale": 0.5 + 1.5 * uniform(E), "jobs": []}
        for N in map(int, case["rows"].split(",")):
            a = torch.where(used[:, :, None], normal(E, R, K, std=K ** -0.5), 0).bfloat16()
            b = torch.where(used[:, None, :], normal(E, N, R, std=0.3 * R ** -0.5), 0).bfloat16()
            s["jobs"].append({"a": a, "b": b, "base": normal(M, N), "y": torch.empty(M, N, device="cuda")})
        return s
    if case["op"] == "logprobs":
        M, n, c, k = case["M"], case["n"], case["tokens"], case["k"]
        y = normal(M, n + case["pad"], std=2.0)
        # a few likely tokens a row, as a trained head has them
        y[:, :n].scatter_add_(1, torch.randint(0, n, (M, 6), generator=g, device="cuda"), 10 * uniform(M, 6))
        if case["masked"]:      # what a grammar allows: a run of tokens and a few apart; the last row has none left
            at = torch.arange(n + case["pad"], device="cuda")[None, :]
            first = torch.randint(0, n, (M, 1), generator=g, device="cuda")
            keep = ((at >= first) & (at < first + 40)) | (uniform(M, n + case["pad"]) < 0.001)
            if M > 1:
                keep[M - 1] = False
            y = torch.where(keep, y, float("-inf"))
        tokens = torch.randint(0, n, (M, c), generator=g, device="cuda")
        tokens[:, 0] = (y[:, :n] - torch.log(-torch.log(uniform(M, n).clamp(1e-9, 1 - 1e-7)))).argmax(1)
        s = {"y": y, "tokens": tokens.to(torch.int32), "logp": torch.empty(M, c, device="cuda"),
             "entropy": torch.empty(M, device="cuda")}
        if k:
            s["top_ids"] = torch.empty(M, k, dtype=torch.int32, device="cuda")
            s["top_logp"] = torch.empty(M, k, device="cuda")
        return s
    M, D = case["M"], case["D"]
    s = {"r": normal(M, D) * (1 + 20 * (uniform(D) < 0.01)), "w": (1 + normal(D, std=0.2)).bfloat16(),
         "x": torch.empty(M, D, dtype=torch.bfloat16, device="cuda")}
    if case["residual"]:
        s["y"] = normal(M, D)
        s["r_out"] = torch.empty(M, D, device="cuda")
    return s


EPS = 1e-6


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if own:
        import gemm_q4nx_chunk_amd as q
        if case["op"] == "lora":
            tables = [q.lora_table(case["adapters"], case["rank"], j["b"].shape[1], case["K"], j["a"], j["b"],
                                   s["scale"], ranks=s["ranks"] if case["mixed"] else None) for j in s["jobs"]]
            s["args"] = q.lora_jobs([(t, j["base"], j["y"]) for t, j in zip(tables, s["jobs"])])
            s["ws"] = torch.empty(q.lora_batched_ws(s["args"], case["M"]), dtype=torch.uint8, device="cuda")
        elif case["op"] == "logprobs":
            s["ws"] = torch.empty(q.token_logprobs_ws(case["n"], case["M"], case["k"]), dtype=torch.uint8, device="cuda")
    return s


# ----------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------
def run(state):
    op = state["case"]["op"]
    if own:
        return {"lora": _own_lora, "logprobs": _own_logprobs, "norm": _own_norm}[op](state)
    return {"lora": _plain_lora, "logprobs": _plain_logprobs, "norm": _plain_norm}[op](state)


def _own_lora(s):
    import gemm_q4nx_chunk_amd as q
    q.lora_add_batched(s["args"], s["x"], s["ids"], s["case"]["M"], s["ws"])
    return [j["y"] for j in s["jobs"]]


def _own_logprobs(s):
    import gemm_q4nx_chunk_amd as q
    c = s["case"]
    out = {"logp": s["logp"], "entropy": s["entropy"]}
    if c["k"]:
        out |= {"top_ids": s["top_ids"], "top_logp": s["top_logp"]}
    q.token_logprobs(s["y"], c["n"], c["M"], s["ws"], tokens=s["tokens"], n_tok=c["tokens"], k=c["k"],
                     ldy=c["n"] + c["pad"], **out)
    return out


def _own_norm(s):
    import gemm_q4nx_chunk_amd as q
    c = s["case"]
    q.add_rmsnorm(s["r"], s["w"], c["M"], c["D"], EPS, s["x"], y=s.get("y"), r_out=s.get("r_out"))
    return {"x": s["x"], "r": s["r_out"]} if c["residual"] else {"x": s["x"]}


def _plain_lora(s):
    """Every adapter's products for every row, of which each row keeps its own adapter's."""
    x, ids = s["x"].float(), s["ids"].long()
    M = x.shape[0]
    row, e = torch.arange(M, device="cuda"), ids.clamp(min=0)
    out = []

    def one(j):
        E, R, K = j["a"].shape
        u = (x @ j["a"].float().view(E * R, K).t()).view(M, E, R)[row, e]
        u = u * (s["scale"][e] * (ids >= 0))[:, None]
        mine = torch.zeros(M, E, R, device="cuda")
        mine[row, e] = u
        return j["base"] + mine.view(M, E * R) @ j["b"].float().transpose(1, 2).reshape(E * R, -1)

    out.extend(map(one, s["jobs"]))
    return out


def _plain_logprobs(s):
    """Sums over everything but one maximum, so that a likely token's log probability keeps its digits."""
    c = s["case"]
    n, k = c["n"], c["k"]
    y = s["y"][:, :n]
    at = torch.arange(n, device="cuda")[None, :]
    y = torch.where(y == y, y, float("-inf"))
    m = y.amax(1, keepdim=True)
    any_left = m > float("-inf")
    first = torch.where(y == m, at, n).amin(1, keepdim=True)
    d = torch.where(y == m, 0.0, y - m)
    e = torch.where(at == first, 0.0, torch.exp(d))
    rest = e.sum(1, keepdim=True)
    t = torch.where(e > 0, e * d, 0.0).sum(1, keepdim=True)
    lz = torch.log1p(rest)
    nan = float("nan")
    tok = s["tokens"].long()
    inside = (tok >= 0) & (tok < n)
    logp = torch.where(inside & any_left, d.gather(1, tok.clamp(0, n - 1)) - lz, nan)
    out = {"logp": logp, "entropy": torch.where(any_left, lz - t / (1 + rest), nan)[:, 0]}
    if k:
        bits = torch.where(y == 0, 0.0, y).contiguous().view(torch.int32).long()
        order = torch.where(bits < 0, -(bits & 0x7FFFFFFF), bits)       # larger value, larger number
        key, pick = torch.topk((order << 32) - at, k, 1)
        ids = torch.where(y.gather(1, pick) > float("-inf"), pick, -1)
        out["top_ids"] = ids.to(torch.int32)
        out["top_logp"] = torch.where(ids >= 0, d.gather(1, pick) - lz, nan)
    return out


def _plain_norm(s):
    v = s["r"] + s["y"] if "y" in s else s["r"]
    x = (v * torch.rsqrt((v * v).mean(1, keepdim=True) + EPS) * s["w"].float()).bfloat16()
    return {"x": x, "r": v} if "y" in s else {"x": x}


# ----------------------------------------------------------------------------
# the definitions in 64 bits
# ----------------------------------------------------------------------------
def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "lora":
        out = []
        for j in s["jobs"]:
            y = j["base"].double()
            for e in range(case["adapters"]):
                mine = (s["ids"] == e).nonzero()[:, 0]
                h = s["x"][mine].double() @ j["a"][e].double().t()
                y[mine] += s["scale"][e].double() * (h @ j["b"][e].double().t())
            out.append(y)
        return out
    if case["op"] == "logprobs":
        n, k = case["n"], case["k"]
        rows = {"logp": [], "entropy": [], "top_ids": [], "top_logp": []}
        for y32, tokens in zip(s["y"][:, :n].split(64), s["tokens"].long().split(64)):
            logp = torch.log_softmax(y32.double(), 1)
            p = torch.exp(logp)
            rows["logp"].append(logp.gather(1, tokens))
            rows["entropy"].append(-torch.special.xlogy(p, p).sum(1))
            top = torch.sort(y32, stable=True, dim=1, descending=True).indices[:, :k]
            none = torch.isinf(y32.gather(1, top))
            rows["top_ids"].append(torch.where(none, -1, top).to(torch.int32))
            rows["top_logp"].append(torch.where(none, float("nan"), logp.gather(1, top)))
        return {name: torch.cat(v) for name, v in rows.items() if k or not name.startswith("top")}
    v = s["r"].double() + (s["y"].double() if "y" in s else 0)
    x = v / torch.sqrt(v.square().mean(1, keepdim=True) + EPS) * s["w"].double()
    return {"x": x, "r": v} if "y" in s else {"x": x}


# ----------------------------------------------------------------------------
# what a pass cannot do without
# ----------------------------------------------------------------------------
def work(case):
    if case["op"] == "lora":
        M, K, E, R = case["M"], case["K"], case["adapters"], case["rank"]
        N = sum(map(int, case["rows"].split(",")))
        rank = (R + 1) / 2 if case["mixed"] else R
        with_one = M if case["prompt"] or M == 1 else M * 15 / 16
        used = min(E, M) if case["prompt"] else E * (1 - (1 - 1 / E) ** with_one) if E > 1 else 1
        jobs = len(case["rows"].split(","))
        return {"bytes": 2 * M * K + 4 * M + 8 * M * N + used * 2 * rank * (jobs * K + N),
                "flops": 2 * with_one * rank * (jobs * K + N)}
    if case["op"] == "logprobs":
        M, n = case["M"], case["n"]
        return {"bytes": 4 * M * n + M * (8 * case["tokens"] + 4 + 8 * case["k"]), "flops": 6 * M * n}
    M, D = case["M"], case["D"]
    return {"bytes": M * D * (14 if case["residual"] else 6) + 2 * D, "flops": 5 * M * D}
