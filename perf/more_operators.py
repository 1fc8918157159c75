"""Cases of the operators that stand round the framework's products: the router ahead of
the product grouped by expert (choice, counts, order, balance loss and its gradient), the
weighted sum of the experts' rows behind it with its gradient, and the low-rank adapters
of many requests beside a shared projection.

    listed()             the cases
    draw(rng)            one more case of the same ranges
    prepare(case, seed)  inputs on the GPU, made from the seed alone
    run(state)           one pass through one operator
    work(case)           bytes and operations the pass cannot do without
    exact(case, seed)    the same outputs from the definition in 64 bits

With ``own`` false, run() is the plain form in elementary torch operations; with ``own``
true it makes the calls a user of w4a16_dequant_gemm_amd makes.
"""
import torch

own = False

BLOCK = 128          # columns of K per fp8 scale
DTYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
E4M3 = torch.float8_e4m3fn


def listed():
    return [
        # 8 decoding requests, 8 of 64 experts each: launch latency
        dict(name="route_decode", op="route", T=8, E=64, top=8, renormalize=True, padded=0.0,
             skew=1.0, dtype="fp32"),
        # a long prompt over 128 experts
        dict(name="route_prefill", op="route", T=8192, E=128, top=8, renormalize=True, padded=0.0,
             skew=0.5, dtype="bf16"),
        # a training step of a short batch with padding behind its sequences
        dict(name="balance_ragged", op="balance", T=519, E=60, top=6, renormalize=False,
             padded=0.2, skew=1.0, dtype="bf16"),
        # a training step of a large batch over many experts
        dict(name="balance_train", op="balance", T=65536, E=256, top=8, renormalize=True,
             padded=0.0, skew=0.5, dtype="fp32"),
        # the sum of 8 experts' rows for 8 decoding requests
        dict(name="combine_decode", op="combine", T=8, top=8, E=64, N=4096, padded=0.0,
             residual=True, dtype="bf16"),
        # the sum of 2 experts' rows for a long prompt
        dict(name="combine_prefill", op="combine", T=8192, top=2, E=16, N=8192, padded=0.0,
             residual=True, dtype="bf16"),
        # its gradient: a chunk of prompts with padding, an odd width
        dict(name="combine_grad_ragged", op="combine_grad", T=519, top=6, E=64, N=2831, padded=0.1,
             residual=False, dtype="fp16"),
        # its gradient: a training batch, 8 experts a token
        dict(name="combine_grad_train", op="combine_grad", T=8192, top=8, E=64, N=4096, padded=0.0,
             residual=False, dtype="bf16"),
        # one decoding request with its adapter beside a square projection
        dict(name="lora_decode", op="lora", M=1, K=4096, N=4096, R=16, L=8, longest=1, without=0.0,
             rows="x16", dtype="fp16"),
        # 64 decoding requests with any of 32 adapters beside the widest layer
        dict(name="lora_batch", op="lora", M=64, K=8192, N=28672, R=16, L=32, longest=1,
             without=0.1, rows="x16", dtype="bf16"),
        # chunks of prompts behind the fp8 quantisers, some without an adapter, an odd N
        dict(name="lora_ragged", op="lora", M=1037, K=7184, N=10001, R=40, L=12, longest=200,
             without=0.2, rows="fp8", dtype="bf16"),
        # prompts of four adapters beside the widest layer
        dict(name="lora_prefill", op="lora", M=4096, K=8192, N=28672, R=64, L=4, longest=2048,
             without=0.0, rows="x16", dtype="bf16"),
    ]


def _log(rng, low, high):
    return low * (high / low) ** rng.random()


def _size(rng, low, high, step=1):
    """A size spread over the logarithm of low..high, a multiple of step."""
    return max(low, min(high, int(round(_log(rng, low, high) / step)) * step))


def draw(rng):
    op = rng.choice(["route", "balance", "combine", "combine_grad", "lora", "lora", "lora"])
    if op in ("route", "balance"):
        E = _size(rng, 4, 512)
        T = _size(rng, 1, min(65536, 65536 * 256 // E))
        top = rng.choice([k for k in (1, 2, 3, 4, 6, 8) if k <= E])
        return dict(op=op, T=T, E=E, top=top, renormalize=rng.random() < 0.5,
                    padded=rng.choice([0.0, 0.0, 0.3]), skew=rng.choice([0.25, 0.5, 1.0]),
                    dtype=rng.choice(["fp32", "bf16", "fp16"]))
    if op in ("combine", "combine_grad"):
        top, E = rng.choice([1, 2, 4, 6, 8]), _size(rng, 8, 128)
        N = _size(rng, 256, 8192, rng.choice([1, 8, 128]))
        T = _size(rng, 1, min(16384, 8192 * 8 * 4096 // (top * N)))
        return dict(op=op, T=T, top=top, E=E, N=N, padded=rng.choice([0.0, 0.0, 0.3]),
                    residual=op == "combine" and rng.random() < 0.5,
                    dtype=rng.choice(["fp16", "bf16"]))
    while True:
        M, R = _size(rng, 1, 4096), _size(rng, 8, 128, 8)
        rows = rng.choice(["x16", "x16", "fp8"])
        K = _size(rng, 256, 28672, 16)
        N = _size(rng, 64, 28672, rng.choice([1, 8, 128]))
        if M * N <= 4096 * 28672 and M * (K + N) * R <= 4096 * 36864 * 64:
            return dict(op=op, M=M, K=K, N=N, R=R, L=_size(rng, 1, 64),
                        longest=rng.choice([1, M, max(1, M // 8)]),
                        without=rng.choice([0.0, 0.0, 0.2]), rows=rows,
                        dtype=rng.choice(["fp16", "bf16"]))


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _blocks(n):
    return -(-n // BLOCK)


def _logits(g, T, E, skew):
    """Scores of a router, some experts liked more than others."""
    return _randn(g, T, E) * 1.5 + skew * _randn(g, E)


def _valid(g, T, padded):
    """Which tokens are real; None if all are."""
    if padded == 0.0:
        return None
    return torch.rand(T, generator=g, device="cuda") >= padded


def _grouped(chosen, valid, E):
    """counts, offsets, rows and places of the choices [T][top]; -1 where there is none."""
    T, top = chosen.shape
    flat = chosen.reshape(-1).long()
    if valid is not None:
        flat = torch.where(valid.repeat_interleave(top), flat, E)
    order = torch.argsort(flat, stable=True)
    counts = torch.zeros(E + 1, dtype=torch.int64, device="cuda")
    counts = counts.scatter_add_(0, flat, torch.ones_like(flat))[:E]
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = counts.cumsum(0)
    at = torch.arange(T * top, device="cuda")
    rows = torch.where(at < offsets[E], order // top, -1).to(torch.int32)
    places = torch.empty_like(order)
    places[order] = at
    places = torch.where(flat < E, places, -1).to(torch.int32).view(T, top)
    return counts.to(torch.int32), offsets, rows, places


def prepare(case, seed):
    g, op, dtype = _generator(seed), case["op"], DTYPES[case["dtype"]]
    state = dict(op=op, dtype=dtype)
    if op in ("route", "balance"):
        T, E, top = case["T"], case["E"], case["top"]
        state.update(top=top, renormalize=case["renormalize"],
                     logits=_logits(g, T, E, case["skew"]).to(dtype),
                     valid=_valid(g, T, case["padded"]))
        if op == "balance":
            # what comes back from the rest of the model
            state["dweights"] = _randn(g, T, top) * 1e-3
            state["dloss"] = torch.full((), 0.01, device="cuda")
        return state
    if op in ("combine", "combine_grad"):
        T, top, E, N = case["T"], case["top"], case["E"], case["N"]
        chosen = _logits(g, T, E, 0.5).topk(top, dim=1).indices
        valid = _valid(g, T, case["padded"])
        _, state["offsets"], _, state["places"] = _grouped(chosen, valid, E)
        weights = torch.softmax(_randn(g, T, top), 1)
        state["weights"] = weights if valid is None else torch.where(valid[:, None], weights, 0.0)
        state["y"] = _randn(g, T * top, N).to(dtype)
        if op == "combine":
            state["residual"] = _randn(g, T, N).to(dtype) if case["residual"] else None
        else:
            state["dout"] = (_randn(g, T, N) * 0.1).to(dtype)
        return state
    M, K, N, R, L = (case[k] for k in ("M", "K", "N", "R", "L"))
    # requests of up to `longest` rows, one after another, each with its adapter
    if case["longest"] == 1:
        ids = torch.randint(L, (M,), generator=g, device="cuda")
        gone = torch.rand(M, generator=g, device="cuda") < case["without"]
    else:
        lengths = torch.randint(1, case["longest"] + 1, (M,), generator=g, device="cuda")
        request = torch.searchsorted(lengths.cumsum(0), torch.arange(M, device="cuda"), right=True)
        ids = torch.randint(L, (M,), generator=g, device="cuda")[request]
        gone = (torch.rand(M, generator=g, device="cuda") < case["without"])[request]
    state["ids"] = torch.where(gone, -1, ids).to(torch.int32)
    if not own:
        # the rows of each adapter, as a program that gathers requests knows them
        state["groups"] = [(a, (state["ids"] == a).nonzero()[:, 0])
                           for a in state["ids"].unique().tolist() if a >= 0]
    state["a"] = (_randn(g, L, R, K) * K ** -0.5).to(dtype)
    state["b"] = (_randn(g, L, N, R) * R ** -0.5).to(dtype)
    state["scale"] = torch.rand(L, generator=g, device="cuda") * 1.5 + 0.5
    state["base"] = _randn(g, M, N).to(dtype)
    state["xs"] = None
    x = _randn(g, M, K)
    if case["rows"] == "fp8":
        pad = torch.nn.functional.pad(x, (0, _blocks(K) * BLOCK - K)).view(M, -1, BLOCK)
        state["xs"] = pad.abs().amax(-1) / 448.0
        state["x"] = (pad / state["xs"][..., None]).view(M, -1)[:, :K].to(E4M3).contiguous()
    else:
        state["x"] = x.to(dtype)
    return state


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(state):
    op = state["op"]
    if op == "lora":
        from w4a16_dequant_gemm_amd import lora
        return lora.lora_add(state["base"], state["x"], state["a"], state["b"], state["ids"],
                             scale=state["scale"], xs=state["xs"])
    from w4a16_dequant_gemm_amd import route
    if op == "route":
        r = route.route_tokens(state["logits"], state["top"], renormalize=state["renormalize"],
                               valid=state["valid"])
        return dict(weights=r.weights, experts=r.experts, counts=r.counts, offsets=r.offsets,
                    rows=r.rows, places=r.places)
    if op == "balance":
        r = route.route_tokens(state["logits"], state["top"], renormalize=state["renormalize"],
                               valid=state["valid"], balance=True)
        d = route.route_tokens_backward(state["logits"], r, dweights=state["dweights"],
                                        dloss=state["dloss"])
        return dict(weights=r.weights, experts=r.experts, counts=r.counts, offsets=r.offsets,
                    rows=r.rows, places=r.places, loss=r.loss, dlogits=d)
    if op == "combine":
        return route.combine_rows(state["y"], state["weights"], state["places"],
                                  residual=state["residual"])
    dy, dweights = route.combine_rows_backward(state["dout"], state["y"], state["weights"],
                                               state["places"], state["offsets"])
    return dict(dy=dy, dweights=dweights)


def _softmax(l):
    e = torch.exp(l - l.amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True)


def _choose(state):
    """The router's outputs and, for the loss, the probabilities of the real tokens."""
    logits, top, valid = state["logits"].float(), state["top"], state["valid"]
    p = _softmax(logits)
    chosen = torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :top]
    weights = p.gather(1, chosen)
    if state["renormalize"]:
        weights = weights / weights.sum(1, keepdim=True)
    if valid is not None:
        weights = torch.where(valid[:, None], weights, 0.0)
        p = torch.where(valid[:, None], p, 0.0)
    counts, offsets, rows, places = _grouped(chosen, valid, p.shape[1])
    experts = chosen if valid is None else torch.where(valid[:, None], chosen, -1)
    return dict(weights=weights, experts=experts.to(torch.int32), counts=counts, offsets=offsets,
                rows=rows, places=places), p, chosen


def _run_plain(state):
    op = state["op"]
    if op == "route":
        return _choose(state)[0]
    if op == "balance":
        got, p, chosen = _choose(state)
        T, E = p.shape
        tokens = T if state["valid"] is None else state["valid"].sum().clamp(min=1)
        pull = got["counts"].float() * E / (tokens * float(state["top"])) / tokens
        got["loss"] = (pull * p.sum(0)).sum()
        a = state["dweights"]
        if state["valid"] is not None:
            a = torch.where(state["valid"][:, None], a, 0.0)
        d = state["dloss"] * p * (pull - (p * pull).sum(1, keepdim=True))
        if state["renormalize"]:
            w = got["weights"]
            d.scatter_add_(1, chosen, w * (a - (a * w).sum(1, keepdim=True)))
        else:
            by_expert = torch.zeros_like(p).scatter_(1, chosen, a)
            d += p * (by_expert - (by_expert * p).sum(1, keepdim=True))
        got["dlogits"] = d.to(state["dtype"])
        return got
    if op == "combine":
        y, places = state["y"], state["places"]
        out = 0.0 if state["residual"] is None else state["residual"].float()
        for j in range(places.shape[1]):
            part = y[places[:, j].clamp(min=0).long()].float() * state["weights"][:, j, None]
            out = out + torch.where(places[:, j, None] >= 0, part, 0.0)
        return out.to(state["dtype"])
    if op == "combine_grad":
        y, places, weights = state["y"], state["places"], state["weights"]
        dout = state["dout"].float()
        dy, dweights = torch.zeros_like(y), torch.zeros_like(weights)
        for j in range(places.shape[1]):
            there = places[:, j] >= 0
            at = torch.where(there, places[:, j], 0).long()
            dot = (dout * y[at].float()).sum(1)
            dweights[:, j] = torch.where(there, dot, 0.0)
            # a token without a row writes behind the last row, where zeros belong
            spare = torch.where(there, at, y.shape[0] - 1)
            part = torch.where(there[:, None], dout * weights[:, j, None], 0.0)
            dy[spare] = part.to(dy.dtype)
        return dict(dy=dy, dweights=dweights)
    x = state["x"].float()
    if state["xs"] is not None:
        x = x * state["xs"].repeat_interleave(BLOCK, 1)[:, :x.shape[1]]
    out = state["base"].float()
    for a, at in state["groups"]:
        h = x[at] @ state["a"][a].float().t()
        out[at] += (h * state["scale"][a]) @ state["b"][a].float().t()
    return out.to(state["dtype"])


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    op, size = case["op"], DTYPES[case["dtype"]].itemsize
    if op in ("route", "balance"):
        T, E, top = case["T"], case["E"], case["top"]
        # logits in; weights, experts, rows, places out; counts and offsets
        bytes_ = size * T * E + 16 * T * top + 8 * E
        if op == "balance":
            bytes_ += size * T * E + 4 * T * top     # the logits' gradient, the weights'
        return {"bytes": bytes_, "flops": (10 if op == "route" else 20) * T * E}
    if op in ("combine", "combine_grad"):
        T, top, N = case["T"], case["top"], case["N"]
        real = 1.0 - case["padded"]
        if op == "combine":
            moved = 2 * N * T * (real * top + 1 + case["residual"]) + 8 * T * top
        else:
            moved = 2 * N * T * (real * top + top + 1) + 12 * T * top
        return {"bytes": moved, "flops": (2 if op == "combine" else 3) * real * T * top * N}
    M, K, N, R, L = (case[k] for k in ("M", "K", "N", "R", "L"))
    real = 1.0 - case["without"]
    requests = max(1.0, M / ((1 + case["longest"]) / 2)) * real
    used = L * (1.0 - (1.0 - 1.0 / L) ** requests)     # adapters that some request has
    row = K + 4 * _blocks(K) if case["rows"] == "fp8" else 2 * K
    return {"bytes": real * M * row + used * (K + N) * R * 2 + 4 * M * N + 4 * M,
            "flops": 2 * real * M * R * (K + N)}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def _exact_route(state, E, top):
    l = state["logits"].double()
    T = l.shape[0]
    real = torch.ones(T, dtype=torch.bool, device="cuda") if state["valid"] is None \
        else state["valid"]
    p = torch.exp(l - torch.logsumexp(l, dim=1)[:, None])
    left, lanes = l.clone(), torch.arange(E, device="cuda")
    experts = torch.empty(T, top, dtype=torch.int64, device="cuda")
    for j in range(top):                       # the largest left, the first of equal ones
        best = left.max(dim=1).values
        experts[:, j] = torch.where(left == best[:, None], lanes, E).min(dim=1).values
        left[torch.arange(T, device="cuda"), experts[:, j]] = -float("inf")
    w = torch.gather(p, 1, experts)
    if state["renormalize"]:
        w = w / w.sum(dim=1)[:, None]
    # every slot in the order of (expert, token)
    slots = torch.arange(T * top, device="cuda")
    keep = real[slots // top]
    key = (experts.reshape(-1) * (T * top) + slots)[keep].sort().values
    rows = torch.full((T * top,), -1, dtype=torch.int64, device="cuda")
    rows[:key.numel()] = key % (T * top) // top
    places = torch.full((T * top,), -1, dtype=torch.int64, device="cuda")
    places[key % (T * top)] = torch.arange(key.numel(), device="cuda")
    edges = torch.arange(E + 1, device="cuda") * (T * top)
    offsets = torch.searchsorted(key, edges)
    got = dict(weights=w * real[:, None], experts=torch.where(real[:, None], experts, -1),
               counts=offsets[1:] - offsets[:-1], offsets=offsets, rows=rows,
               places=places.view(T, top))
    got = {k: v if k == "weights" else v.to(torch.int32) for k, v in got.items()}
    return got, p * real[:, None], experts, real


def exact(case, seed):
    global own
    kept, own = own, False
    try:
        state = prepare(case, seed)
    finally:
        own = kept
    op = case["op"]
    if op in ("route", "balance"):
        E, top = case["E"], case["top"]
        got, p, experts, real = _exact_route(state, E, top)
        if op == "route":
            return got
        V = max(1, int(real.sum()))
        f = got["counts"].double() / (V * top)
        got["loss"] = E * (f * (p.sum(dim=0) / V)).sum()
        # the loss and the weights' pull on the probabilities, through their softmax
        dp = (float(state["dloss"]) * E / V) * f.expand_as(p).clone()
        a, w = state["dweights"].double() * real[:, None], got["weights"]
        if state["renormalize"]:
            # d w_j / d p_k = (delta - w_j) / sum of the chosen
            total = torch.gather(p, 1, experts).sum(dim=1)[:, None].clamp(min=1e-300)
            a = (a - (a * w).sum(dim=1)[:, None]) / total
        dp.scatter_add_(1, experts, a)
        got["dlogits"] = p * (dp - (p * dp).sum(dim=1)[:, None])
        return got
    if op in ("combine", "combine_grad"):
        y, w, places = state["y"], state["weights"].double(), state["places"].long()
        T, top = places.shape
        flat = places.reshape(-1)
        slots = (flat >= 0).nonzero()[:, 0]
        if op == "combine":
            out = torch.zeros(T, y.shape[1], dtype=torch.float64, device="cuda")
            if state["residual"] is not None:
                out += state["residual"].double()
            for j in range(top):
                mine = slots[slots % top == j]
                out[mine // top] += y[flat[mine]].double() * w[mine // top, j][:, None]
            return out
        d = state["dout"].double()
        dy = torch.zeros(y.shape, dtype=torch.float64, device="cuda")
        dw = torch.zeros(T * top, dtype=torch.float64, device="cuda")
        for mine in slots.split(8192):
            dy[flat[mine]] = d[mine // top] * w.reshape(-1)[mine][:, None]
            dw[mine] = (d[mine // top] * y[flat[mine]].double()).sum(dim=1)
        return dict(dy=dy, dweights=dw.view(T, top))
    x = state["x"].double()
    if state["xs"] is not None:
        x *= state["xs"].double()[:, torch.arange(x.shape[1], device="cuda") // BLOCK]
    out = state["base"].double()
    for a in range(case["L"]):
        mine = (state["ids"] == a).nonzero()[:, 0]
        h = x.index_select(0, mine) @ state["a"][a].double().T
        out.index_add_(0, mine, h @ state["b"][a].double().T * state["scale"][a].double())
    return out
