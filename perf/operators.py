"""Performance cases of the 8-bit head and of sampling: `quantize`, `project` and `sample`.

Where ``own`` is false, ``run`` computes each operator in its plain form with elementary torch
operations; where it is true, it makes the calls of output_projection_kl_amd. The shapes are those
of the framework's workloads (d = 2880 with V = 201088, d = 4096 with V = 128256, top-100 teacher
lists) and generic ones around them.
"""

import math

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def _device():
    return torch.device("cuda", torch.cuda.current_device())


def listed():
    return [
        # hidden states of a 4096-token pass, quantised before a product
        {"name": "quantize_tokens", "op": "quantize", "rows": 4096, "cols": 2880, "type": "bf16"},
        # a whole head, quantised once when it is loaded
        {"name": "quantize_head", "op": "quantize", "rows": 128256, "cols": 4096, "type": "bf16"},
        # the smallest call: a few tokens through a narrow layer, latency only
        {"name": "project_small", "op": "project", "M": 5, "K": 1024, "N": 1024, "a": "i8", "out": "bf16",
         "bias": False},
        # one token of one sequence against the whole head
        {"name": "project_decode_1", "op": "project", "M": 1, "K": 2880, "N": 201088, "a": "bf16", "out": "f32",
         "bias": False},
        # one token of each of 48 sequences, hidden states as the model leaves them
        {"name": "project_decode_48", "op": "project", "M": 48, "K": 4096, "N": 128256, "a": "bf16", "out": "bf16",
         "bias": False},
        # a ragged batch of draft tokens, odd in every size, with a bias
        {"name": "project_odd", "op": "project", "M": 201, "K": 2887, "N": 32003, "a": "f16", "out": "f16",
         "bias": True},
        # a teacher scoring a packed batch of 8192 tokens
        {"name": "project_score", "op": "project", "M": 8192, "K": 4096, "N": 128256, "a": "i8", "out": "bf16",
         "bias": False},
        # one token of one sequence, the usual mixture of filters
        {"name": "sample_decode_1", "op": "sample", "N": 1, "V": 201088, "type": "f32", "T": 0.8, "k": 50, "p": 0.95,
         "q": 0.0, "rowwise": False, "masked": 0.0, "ids": False},
        # a decode batch under nucleus sampling: the mass of the whole row counts
        {"name": "sample_nucleus_64", "op": "sample", "N": 64, "V": 128256, "type": "bf16", "T": 1.0, "k": 0,
         "p": 0.9, "q": 0.0, "rowwise": False, "masked": 0.0, "ids": False},
        # a serving batch whose requests each bring their own settings, greedy ones among them
        {"name": "sample_mixed_512", "op": "sample", "N": 512, "V": 201088, "type": "f32", "T": 1.0, "k": 100,
         "p": 0.95, "q": 0.05, "rowwise": True, "masked": 0.0, "ids": False},
        # plain draws under a grammar that masks most tokens (all of them in some rows), odd vocabulary
        {"name": "sample_masked_130", "op": "sample", "N": 130, "V": 50257, "type": "f16", "T": 1.1, "k": 0,
         "p": 1.0, "q": 0.0, "rowwise": False, "masked": 0.97, "ids": False},
        # hard labels drawn from the cached top-100 lists of a packed batch
        {"name": "sample_lists", "op": "sample", "N": 16384, "V": 100, "type": "f32", "T": 1.0, "k": 0, "p": 0.98,
         "q": 0.0, "rowwise": False, "masked": 0.0, "ids": True},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quantize", "project", "project", "sample", "sample"])
    if op == "quantize":
        cols = _log_int(rng, 64, 16384)
        rows = _log_int(rng, 1, min(131072, (1 << 28) // cols))
        return {"op": op, "rows": rows, "cols": cols, "type": rng.choice(sorted(TYPES))}
    if op == "project":
        K = _log_int(rng, 64, 8192)
        N = _log_int(rng, 64, 201088)
        M = _log_int(rng, 1, max(1, min(8192, (1 << 28) // N)))
        if rng.random() < 0.6:  # sizes as layers have them; the others are odd ones
            K, N = -(-K // 64) * 64, -(-N // 64) * 64
        return {"op": op, "M": M, "K": K, "N": N, "a": rng.choice(["i8", "i8", "bf16", "f16", "f32"]),
                "out": rng.choice(["bf16", "f16", "f32"]), "bias": rng.random() < 0.3}
    V = _log_int(rng, 64, 262144)
    N = _log_int(rng, 1, max(1, min(16384, (1 << 26) // V)))
    if rng.random() < 0.5:
        V = -(-V // 8) * 8
    return {"op": op, "N": N, "V": V, "type": rng.choice(sorted(TYPES)), "T": rng.choice([0.6, 0.8, 1.0, 1.0, 1.3]),
            "k": rng.choice([0, 0, 1, 20, 50, 200]), "p": rng.choice([1.0, 0.8, 0.9, 0.95]),
            "q": rng.choice([0.0, 0.0, 0.02, 0.1]), "rowwise": rng.random() < 0.4,
            "masked": rng.choice([0.0, 0.0, 0.0, 0.9]), "ids": V <= 1024}


def _int8_rows(rows, cols, g, dev):
    """int8 rows laid out as a program keeps them: each padded to a multiple of 16 bytes."""
    x = torch.empty((rows, -(-cols // 16) * 16), dtype=torch.int8, device=dev)
    x.random_(-127, 128, generator=g)
    return x[:, :cols]


def _logits(N, V, g, dev):
    """Next-token logits: a broad bulk, and a few dozen likely tokens that stand out of it by more in some rows
    than in others."""
    x = torch.randn((N, V), generator=g, device=dev).mul_(2.0)
    n = min(64, V)
    top = 14.0 + 8.0 * torch.rand((N, 1), generator=g, device=dev)
    slope = 0.6 + 1.2 * torch.rand((N, 1), generator=g, device=dev)
    rank = torch.arange(n, device=dev, dtype=torch.float32)
    likely = top - slope * torch.log1p(rank) + 0.3 * torch.randn((N, n), generator=g, device=dev)
    at = torch.randint(0, V, (N, n), generator=g, device=dev)
    return x.scatter_(1, at, likely)


def prepare(case, seed):
    dev = _device()
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    st = {"op": case["op"]}
    if case["op"] == "quantize":
        # hidden states: a few channels are far larger than the rest
        x = torch.randn((case["rows"], case["cols"]), generator=g, device=dev, dtype=TYPES[case["type"]])
        big = torch.randint(0, case["cols"], (max(1, case["cols"] // 256),), generator=g, device=dev)
        x[:, big] *= 20
        st["x"] = x
        return st
    if case["op"] == "project":
        M, K, N = case["M"], case["K"], case["N"]
        st["b"] = _int8_rows(N, K, g, dev)
        st["b_scale"] = (0.5 + torch.rand(N, generator=g, device=dev)) / (127 * math.sqrt(K))
        if case["a"] == "i8":
            st["a"] = _int8_rows(M, K, g, dev)
            st["a_scale"] = (2.0 + 2.0 * torch.rand(M, generator=g, device=dev)) / 127
        else:
            st["a"] = torch.randn((M, K), generator=g, device=dev, dtype=TYPES[case["a"]])
            st["a_scale"] = None
        st["bias"] = torch.randn(N, generator=g, device=dev) if case["bias"] else None
        st["out"] = TYPES[case["out"]]
        return st
    N, V = case["N"], case["V"]
    x = _logits(N, V, g, dev)
    if case["masked"]:
        x.masked_fill_(torch.rand((N, V), generator=g, device=dev) < case["masked"], -math.inf)
        empty = torch.rand((N, 1), generator=g, device=dev) < 0.02
        empty[0] = N > 1
        x.masked_fill_(empty, -math.inf)
    st["ids"] = None
    if case["ids"]:  # a cached list: descending logits with the indices that they belong to
        x = x.sort(dim=1, descending=True).values
        st["ids"] = torch.rand((N, 201088 // 128), generator=g, device=dev).topk(V).indices.to(torch.int32) * 128
    st["x"] = x.to(TYPES[case["type"]])
    st["u"] = torch.rand(N, generator=g, device=dev)
    if case["rowwise"]:
        # each request's own settings: one in eight greedy, one in eight without top-k, top-p or min-p each
        def some(value, off, dtype, share=8):
            r = torch.randint(0, share, (N,), generator=g, device=dev)
            return torch.where(r == 0, off, value).to(dtype)
        st["T"] = some(case["T"] * (0.6 + 0.6 * torch.rand(N, generator=g, device=dev)), 0.0, torch.float32)
        st["k"] = some(torch.randint(1, 2 * max(1, case["k"]) + 1, (N,), generator=g, device=dev), 0, torch.int32)
        st["p"] = some(torch.full((N,), case["p"], device=dev), 1.0, torch.float32)
        st["q"] = some(torch.full((N,), case["q"], device=dev), 0.0, torch.float32)
    else:
        st["T"], st["k"], st["p"], st["q"] = case["T"], case["k"], case["p"], case["q"]
    return st


def _plain_quantize(x):
    # a row's border values are whole numbers and a half: 64 bits decide them
    x = x.double()
    a = x.abs().amax(dim=1, keepdim=True)
    q = torch.round(x * 127 / torch.where(a > 0, a, torch.ones_like(a)))
    return q.float(), (a / 127).float()


def _plain_project(a, a_scale, b, b_scale, bias, dtype):
    if a_scale is None:
        a, s = _plain_quantize(a)
    else:
        a, s = a.float(), a_scale[:, None]
    out = (a @ b.float().T).mul_(s).mul_(b_scale)
    return (out if bias is None else out.add_(bias)).to(dtype)


def _plain_sample(x, u, T, k, p, q, ids):
    N, V = x.shape
    dev = x.device

    def column(v, dtype):
        return (v.to(dtype) if isinstance(v, torch.Tensor) else torch.full((N,), v, device=dev, dtype=dtype))[:, None]

    # whether a token is drawn goes by sums over the whole row: 64 bits
    x = x.double()
    x = torch.where(torch.isnan(x), -math.inf, x)
    T, k = column(T, torch.float32).double(), column(k, torch.int64)
    p, q = column(p, torch.float32).double(), column(q, torch.float32).double()
    k = torch.where(T == 0, 1, torch.where((k <= 0) | (k > V), V, k))
    T = torch.where(T == 0, 1.0, T)
    x, order = x.sort(dim=1, descending=True, stable=True)
    top = x[:, :1]
    w = torch.where(x == -math.inf, 0.0, torch.where(x == top, 1.0, torch.exp((x - top) / T)))
    place = torch.arange(V, device=dev)
    w = torch.where(place < k, w, 0.0)
    before = torch.cumsum(w, dim=1) - w
    first = place == 0
    kept = first | ((p >= 1) | (before < p * w.sum(dim=1, keepdim=True))) & (w >= q)
    w = torch.zeros_like(w).scatter_(1, order, torch.where(kept, w, 0.0))
    below = torch.cumsum(w, dim=1)
    total = below[:, -1:]
    at = (below <= u.double()[:, None] * total).sum(dim=1, keepdim=True).clamp_(max=V - 1)
    none = total[:, 0] == 0
    logprob = torch.where(none, -math.inf, torch.log(w.gather(1, at) / total)[:, 0]).float()
    token = at[:, 0] if ids is None else ids.gather(1, at)[:, 0]
    return torch.where(none, -1, token).to(torch.int32), logprob


def run(state):
    if own:
        import output_projection_kl_amd as fkl
    st = state
    if st["op"] == "quantize":
        q, scale = fkl.quantize(st["x"]) if own else _plain_quantize(st["x"])
        return torch.mul(q, scale.reshape(-1, 1)), scale.reshape(-1)
    if st["op"] == "project":
        if own:
            return fkl.project(st["a"], st["b"], st["b_scale"], a_scale=st["a_scale"], bias=st["bias"],
                               out_dtype=st["out"])
        return _plain_project(st["a"], st["a_scale"], st["b"], st["b_scale"], st["bias"], st["out"])
    if own:
        return fkl.sample(st["x"], st["u"], temperature=st["T"], top_k=st["k"], top_p=st["p"], min_p=st["q"],
                          ids=st["ids"])
    return _plain_sample(st["x"], st["u"], st["T"], st["k"], st["p"], st["q"], st["ids"])


def work(case):
    if case["op"] == "quantize":
        n = case["rows"] * case["cols"]
        return {"bytes": n * (TYPES[case["type"]].itemsize + 1) + 4 * case["rows"], "flops": 8 * n}
    if case["op"] == "project":
        M, K, N = case["M"], case["K"], case["N"]
        size = 1 if case["a"] == "i8" else TYPES[case["a"]].itemsize
        read = M * K * size + N * K + 4 * N * (2 if case["bias"] else 1) + (4 * M if case["a"] == "i8" else 0)
        return {"bytes": read + M * N * TYPES[case["out"]].itemsize, "flops": 2 * M * N * K}
    n = case["N"] * case["V"]
    return {"bytes": n * TYPES[case["type"]].itemsize + 12 * case["N"], "flops": 4 * n}


def _exact_levels(x):
    """Each row's levels (whole numbers of at most 127) and its largest magnitude."""
    x = x.to(torch.float64)
    high = torch.maximum(x.max(dim=1).values, -x.min(dim=1).values)
    t = x.mul_((127 / high)[:, None])
    low = torch.floor(t)
    rest = t.sub_(low)
    up = (rest > 0.5 + 1e-12) | ((rest >= 0.5 - 1e-12) & (low % 2 != 0))
    return low.add_(up), high


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "quantize":
        parts = [_exact_levels(x) for x in st["x"].split(16384)]
        scale = torch.cat([h for _, h in parts]) / 127
        return torch.cat([v.mul_(h[:, None] / 127) for v, h in parts]), scale
    if case["op"] == "project":
        if st["a_scale"] is None:
            a, high = _exact_levels(st["a"])
            a = a * (high / 127)[:, None]
        else:
            a = st["a"].to(torch.float64) * st["a_scale"].to(torch.float64)[:, None]
        b = st["b"].to(torch.float64).mul_(st["b_scale"].to(torch.float64)[:, None])
        out = torch.mm(a, b.t())
        return out if st["bias"] is None else out.add_(st["bias"].to(torch.float64))
    # row by row, by searching the sorted row for each filter's border; a drawn token is no computed value
    N, V = st["x"].shape

    def of(value, r):
        return float(value[r]) if isinstance(value, torch.Tensor) else float(value)

    if V <= 4096:  # many short rows: quicker on the host
        st = {n: v.cpu() if isinstance(v, torch.Tensor) else v for n, v in st.items()}
    logprob = []
    for r in range(N):
        T, k, p, q = (of(st[n], r) for n in ("T", "k", "p", "q"))
        if not isinstance(st["T"], torch.Tensor):
            p, q, T = (float(torch.tensor(v, dtype=torch.float32)) for v in (p, q, T))
        x = st["x"][r].to(torch.float64)
        at = torch.nonzero(x > -math.inf)[:, 0]
        if at.numel() == 0:
            logprob.append(x.new_tensor(-math.inf))
            continue
        x = x[at]
        by = torch.sort(-x, stable=True).indices
        n = 1 if T == 0 else min(int(k), by.numel()) if k > 0 else by.numel()
        by = by[:n]
        weight = torch.exp((x[by] - x[by[0]]) / (T or 1.0))
        keep = torch.ones(n, dtype=torch.bool, device=x.device)
        if p < 1:
            run_up = torch.cumsum(weight, 0)
            reached = torch.searchsorted(run_up, p * run_up[-1:])
            keep &= torch.arange(n, device=x.device) <= reached
        keep &= weight >= min(q, 1.0)
        by, weight = by[keep], weight[keep]
        weight = weight[torch.argsort(by)]
        up = torch.cumsum(weight, 0)
        i = torch.searchsorted(up, st["u"][r].to(torch.float64) * up[-1:], right=True).clamp_(max=up.numel() - 1)
        logprob.append(torch.log(weight[i[0]] / up[-1]))
    return None, torch.stack(logprob).to(_device())
