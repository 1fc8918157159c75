"""Cases of the 8-bit feed-forward operators: the RMS norm and the gated activation
that end in quantised rows, the block-scaled fp8 product, and the same product grouped
by expert.

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
TINY = 2.0 ** -110   # smallest block maximum an fp8 scale is made from
DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
E4M3 = torch.float8_e4m3fn
E8M0 = torch.float8_e8m0fnu


def listed():
    return [
        # one token of a decoding step, hidden 4096: launch latency
        dict(name="norm_decode", op="norm", T=1, H=4096, kind="fp8", dtype="bf16", residual=True),
        # a batch of decoding requests ahead of the int8 product, a width that fills no block of 128
        dict(name="norm_int8_batch", op="norm", T=129, H=5136, kind="int8", dtype="fp16",
             residual=True),
        # a prompt of 4096 tokens, hidden 8192
        dict(name="norm_prefill", op="norm", T=4096, H=8192, kind="fp8", dtype="bf16",
             residual=True),
        # the gated activation of 8 decoding requests, ahead of the MXFP4 product
        dict(name="swiglu_decode_mx", op="swiglu", T=8, F=28672, kind="mx", dtype="fp16"),
        # the gated activation of a prompt of 4096 tokens
        dict(name="swiglu_prefill", op="swiglu", T=4096, F=28672, kind="fp8", dtype="bf16"),
        # a few decoding requests through a square projection: the smallest product
        dict(name="gemm_small", op="gemm", M=7, K=4096, N=4096, dtype="fp16"),
        # one decoding request through the widest layer: the weights' bytes
        dict(name="gemm_decode", op="gemm", M=1, K=8192, N=28672, dtype="bf16"),
        # a batch through a vocabulary-like layer: odd rows and columns, K inside a block
        dict(name="gemm_ragged", op="gemm", M=101, K=7184, N=10001, dtype="bf16"),
        # a prompt of 4096 tokens through the widest layer
        dict(name="gemm_prefill", op="gemm", M=4096, K=8192, N=28672, dtype="bf16"),
        # 8 decoding requests, 8 of 64 experts each: most experts have no row or one
        dict(name="experts_decode", op="experts", T=8, top=8, E=64, K=4096, N=2048, skew=1.0,
             gather=True, dtype="bf16"),
        # a chunk of prompts over many small experts, uneven
        dict(name="experts_ragged", op="experts", T=519, top=6, E=64, K=2048, N=2832, skew=1.0,
             gather=True, dtype="fp16"),
        # a long prompt over a few large experts, rows already in order
        dict(name="experts_prefill", op="experts", T=8192, top=2, E=16, K=4096, N=8192, skew=0.5,
             gather=False, dtype="bf16"),
    ]


def _log(rng, low, high):
    return low * (high / low) ** rng.random()


def _size(rng, low, high, step=1):
    """A size spread over the logarithm of low..high, a multiple of step."""
    while True:
        v = max(low, min(high, int(round(_log(rng, low, high) / step)) * step))
        if v != 3 * 1024:
            return v


def draw(rng):
    op = rng.choice(["norm", "swiglu", "gemm", "gemm", "experts", "experts"])
    dtype = rng.choice(["fp16", "bf16"])
    if op in ("norm", "swiglu"):
        kind = rng.choice(["fp8", "fp8", "int8", "mx", "x16"])
        step = {"fp8": 16, "int8": 16, "mx": 32, "x16": 16}[kind]
        wide = _size(rng, 256, 16384 if op == "norm" else 28672, step)
        most = 4096 * (8192 if op == "norm" else 28672)
        T = _size(rng, 1, min(4096, most // wide))
        if op == "norm":
            return dict(op=op, T=T, H=wide, kind=kind, dtype=dtype, residual=rng.random() < 0.7)
        return dict(op=op, T=T, F=wide, kind=kind, dtype=dtype)
    if op == "gemm":
        while True:
            M, K = _size(rng, 1, 4096), _size(rng, 256, 28672, 16)
            N = _size(rng, 64, 28672, rng.choice([1, 16, 128]))
            if N * K <= 28672 * 8192:
                return dict(op=op, M=M, K=K, N=N, dtype=dtype)
    while True:
        E, top = _size(rng, 4, 128), rng.choice([1, 2, 4, 6, 8])
        T = _size(rng, 1, 8192)
        K, N = _size(rng, 512, 8192, 16), _size(rng, 512, 8192, 16)
        if top <= E and E * K * N <= 16 * 4096 * 8192 and T * top * K * N <= 16384 * 4096 * 8192:
            return dict(op=op, T=T, top=top, E=E, K=K, N=N, skew=rng.choice([0.25, 0.5, 1.0]),
                        gather=rng.random() < 0.6, dtype=dtype)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _activations(g, rows, cols, dtype):
    """Normal values with a few large columns, as hidden states have."""
    x = torch.randn(rows, cols, generator=g, device="cuda")
    heavy = torch.rand(cols, generator=g, device="cuda") < 0.002
    return (x * torch.where(heavy, 20.0, 1.0)).to(dtype)


def _blocks(n):
    return -(-n // BLOCK)


def _fp8_rows(g, rows, cols):
    """Rows as the quantisers leave them: codes that reach 448 in every block, and scales."""
    x = torch.randn(rows, _blocks(cols), BLOCK, generator=g, device="cuda")
    x *= 448.0 / x.abs().amax(-1, keepdim=True)
    s = torch.rand(rows, _blocks(cols), generator=g, device="cuda") * 0.02 + 0.002
    return x.view(rows, -1)[:, :cols].to(E4M3).contiguous(), s


def _fp8_weights(g, experts, n, k):
    w = torch.empty(experts, n, k, dtype=E4M3, device="cuda")
    for e in range(experts):
        w[e] = (torch.randn(n, k, generator=g, device="cuda") * 110.0).clamp_(-448, 448).to(E4M3)
    s = torch.rand(experts, _blocks(n), _blocks(k), generator=g, device="cuda") * 2e-4 + 2e-5
    return w, s


def prepare(case, seed):
    g, op, dtype = _generator(seed), case["op"], DTYPES[case["dtype"]]
    state = dict(op=op, out=case["dtype"], dtype=dtype, kind=case.get("kind"))
    if op == "norm":
        T, H = case["T"], case["H"]
        state["x"] = _activations(g, T, H, dtype)
        state["r"] = _activations(g, T, H, dtype) if case["residual"] else None
        state["w"] = (1.0 + 0.2 * torch.randn(H, generator=g, device="cuda")).to(dtype)
        state["eps"] = 1e-6
    elif op == "swiglu":
        # one product gives both halves: the gate's columns, then the up projection's
        both = _activations(g, case["T"], 2 * case["F"], dtype)
        state["gate"], state["up"] = both[:, :case["F"]], both[:, case["F"]:]
    elif op == "gemm":
        state["xq"], state["xs"] = _fp8_rows(g, case["M"], case["K"])
        w, ws = _fp8_weights(g, 1, case["N"], case["K"])
        state["w"], state["ws"] = w[0], ws[0]
    else:
        T, top, E = case["T"], case["top"], case["E"]
        logits = torch.randn(T, E, generator=g, device="cuda")
        logits += case["skew"] * torch.randn(E, generator=g, device="cuda")
        chosen = logits.topk(top, dim=1).indices.reshape(-1)
        order = torch.argsort(chosen, stable=True)
        counts = torch.bincount(chosen, minlength=E)
        state["offsets"] = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
        state["offsets"][1:] = counts.cumsum(0)
        state["rows"] = (order // top).to(torch.int32) if case["gather"] else None
        state["most"] = int(counts.max())   # rows of the fullest expert: the plain form's padding
        state["xq"], state["xs"] = _fp8_rows(g, T if case["gather"] else T * top, case["K"])
        state["w"], state["ws"] = _fp8_weights(g, E, case["N"], case["K"])
    if own and op in ("gemm", "experts"):
        from w4a16_dequant_gemm_amd import fp8
        state["packed"] = fp8.fp8_repack(state.pop("w"), state.pop("ws"))
    return state


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    return _run_own(state) if own else _run_plain(state)


def _as_values(kind, q, s):
    """Quantised rows as the values the stored bits stand for."""
    if kind == "int8":
        return {"q": q.to(torch.float16), "s": s}
    if kind == "mx":
        return {"q": q.view(E4M3), "s": s.view(E8M0)}
    return {"q": q} if kind == "x16" else {"q": q, "s": s}


def _run_own(state):
    op = state["op"]
    if op == "norm":
        from w4a16_dequant_gemm_amd import rowquant
        q, s, h = rowquant.rmsnorm_quantize_rows(state["x"], state["w"], residual=state["r"],
                                                 eps=state["eps"], kind=state["kind"])
        got = _as_values(state["kind"], q, s)
        return got if h is None else dict(got, h=h)
    if op == "swiglu":
        from w4a16_dequant_gemm_amd import rowquant
        q, s = rowquant.swiglu_quantize_rows(state["gate"], state["up"], kind=state["kind"])
        return _as_values(state["kind"], q, s)
    from w4a16_dequant_gemm_amd import fp8
    if op == "gemm":
        return fp8.fp8_gemm(state["xq"], state["xs"], state["packed"], out=state["out"])
    return fp8.fp8_grouped_gemm(state["xq"], state["xs"], state["packed"], state["offsets"],
                                rows=state["rows"], out=state["out"])


def _quantise(v, kind, dtype):
    rows, cols = v.shape
    if kind == "x16":
        return {"q": v.to(dtype)}
    if kind == "int8":
        s = v.abs().amax(1) / 127.0
        q = torch.round(v / torch.where(s > 0, s, 1.0)[:, None]).clamp(-127, 127)
        return {"q": q.to(torch.float16), "s": s}
    if kind == "mx":
        b = v.view(rows, cols // 32, 32)
        top = b.abs().amax(-1)
        power = torch.frexp(top).exponent - 9    # floor(log2 top) - 8
        power = torch.where(top > 0, power, -127).clamp(min=-127)
        q = torch.ldexp(b, -power[..., None]).clamp(-448, 448).to(E4M3)
        return {"q": q.view(rows, cols), "s": (power + 127).to(torch.uint8).view(E8M0)}
    b = torch.nn.functional.pad(v, (0, _blocks(cols) * BLOCK - cols)).view(rows, -1, BLOCK)
    top = b.abs().amax(-1).clamp(min=TINY)
    q = (b * (448.0 / top)[..., None]).clamp(-448, 448).to(E4M3)
    return {"q": q.view(rows, -1)[:, :cols].contiguous(), "s": top / 448.0}


def _dequantised(q, s):
    """fp32 values of fp8 rows with a scale per 128 columns."""
    cols = q.shape[-1]
    return q.float() * s.repeat_interleave(BLOCK, -1)[..., :cols]


def _dequantised_weights(w, ws):
    return _dequantised(w, ws.repeat_interleave(BLOCK, -2)[..., :w.shape[-2], :])


def _run_plain(state):
    op = state["op"]
    if op == "norm":
        h = state["x"].float()
        if state["r"] is not None:
            h = h + state["r"].float()
        v = h * torch.rsqrt(h.square().mean(1, keepdim=True) + state["eps"]) * state["w"].float()
        got = _quantise(v, state["kind"], state["dtype"])
        return got if state["r"] is None else dict(got, h=h.to(state["dtype"]))
    if op == "swiglu":
        g = state["gate"].float()
        return _quantise(g / (1.0 + torch.exp(-g)) * state["up"].float(), state["kind"],
                         state["dtype"])
    x = _dequantised(state["xq"], state["xs"])
    w = _dequantised_weights(state["w"], state["ws"])
    if op == "gemm":
        return (x @ w.t()).to(state["dtype"])
    if state["rows"] is not None:
        x = x[state["rows"].long()]
    # every expert's rows padded to the fullest expert's, one batched product
    E, R, most = w.shape[0], x.shape[0], state["most"]
    off = state["offsets"].long()
    expert = torch.repeat_interleave(torch.arange(E, device=x.device), off.diff(), output_size=R)
    place = torch.arange(R, device=x.device) - off[expert]
    padded = torch.zeros(E, most, x.shape[1], device=x.device)
    padded[expert, place] = x
    y = torch.bmm(w, padded.transpose(1, 2).contiguous())
    return y.transpose(1, 2)[expert, place].to(state["dtype"])


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    op = case["op"]
    if op in ("norm", "swiglu"):
        wide = case["H"] if op == "norm" else case["F"]
        n = case["T"] * wide
        out = {"fp8": n + 4 * case["T"] * _blocks(wide), "int8": n + 4 * case["T"],
               "mx": n + n // 32, "x16": 2 * n}[case["kind"]]
        if op == "swiglu":
            return {"bytes": 4 * n + out, "flops": 8 * n}
        return {"bytes": (6 if case["residual"] else 2) * n + 2 * wide + out, "flops": 8 * n}
    K, N = case["K"], case["N"]
    weight = K * N + 4 * _blocks(K) * _blocks(N)
    row = K + 4 * _blocks(K)
    if op == "gemm":
        M = case["M"]
        return {"bytes": weight + M * row + 2 * M * N, "flops": 2 * M * N * K}
    # experts that have a row, as if chosen evenly
    R, E = case["T"] * case["top"], case["E"]
    used = E * (1.0 - (1.0 - case["top"] / E) ** case["T"])
    read = case["T"] if case["gather"] else R
    return {"bytes": used * weight + read * row + 2 * R * N + 4 * (E + 1), "flops": 2 * R * N * K}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def _exact_e4m3(v):
    """The E4M3 value nearest to v (|v| <= 448), ties to the even code, by its steps."""
    a = v.abs().clamp(max=448.0)
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3)
    return torch.sign(v) * (torch.round(a / step) * step)


def _exact_rows(v, kind):
    if kind == "x16":
        return {"q": v}
    if kind == "int8":
        top = v.abs().max(dim=1).values
        unit = torch.where(top > 0, top / 127.0, torch.ones_like(top))
        return {"q": torch.round(v / unit[:, None]), "s": top / 127.0}
    size = 32 if kind == "mx" else BLOCK
    at = torch.arange(v.shape[1], device=v.device) // size
    top = torch.zeros(v.shape[0], int(at[-1]) + 1, dtype=v.dtype, device=v.device)
    top.scatter_reduce_(1, at.expand_as(v), v.abs(), "amax")
    if kind == "mx":
        unit = torch.exp2((torch.floor(torch.log2(top.clamp(min=2.0 ** -300))) - 8).clamp(min=-127))
    else:
        unit = top.clamp(min=TINY) / 448.0
    return {"q": _exact_e4m3(v / unit[:, at]), "s": unit}


def exact(case, seed):
    global own
    kept, own = own, False       # the inputs as they are before any layout
    try:
        state = prepare(case, seed)
    finally:
        own = kept
    op = case["op"]
    if op == "norm":
        h = state["x"].double()
        if state["r"] is not None:
            h += state["r"].double()
        scale = 1.0 / torch.sqrt((h * h).sum(dim=1) / h.shape[1] + state["eps"])
        got = _exact_rows(h * scale[:, None] * state["w"].double(), case["kind"])
        return got if state["r"] is None else dict(got, h=h)
    if op == "swiglu":
        g, u = state["gate"].double(), state["up"].double()
        return _exact_rows(torch.sigmoid(g) * g * u, case["kind"])
    K, N = case["K"], case["N"]
    in_block = torch.arange(K, device="cuda") // BLOCK
    of_row = torch.arange(N, device="cuda") // BLOCK

    def weights(w, ws):
        return w.double() * ws.double()[of_row][:, in_block]

    x = state["xq"].double() * state["xs"].double()[:, in_block]
    if op == "gemm":
        return x @ weights(state["w"], state["ws"]).T
    if state["rows"] is not None:
        x = x.index_select(0, state["rows"].long())
    ends = state["offsets"].tolist()
    return torch.cat([x[a:b] @ weights(state["w"][e], state["ws"][e]).T
                      for e, (a, b) in enumerate(zip(ends, ends[1:]))])
