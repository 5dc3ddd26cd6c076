"""The dense operators beside the MoE layer, as cases to measure.

Two operators: the gated feed-forward block (h = act(x Wg^T) * (x Wu^T), with
its backward pass) and the projection with low-rank adapters of many requests
(y[t] = x[t] W^T + base[t] + s_a B_a (A_a x[t]), a the token's adapter).
`run` computes a case either in its plain form (elementary torch operations
in fp32, rounded once) or, with `own`, through this package's entry points;
`exact` computes it from the definition in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}

# The largest case's multiply-adds (16384 tokens, 4096 x 2048, forward and
# backward: 6 products of tokens x hidden x inter); drawn cases stay below.
LARGEST = 6 * 16384 * 4096 * 2048


def _glu(name, tokens, hidden, inter, dtype, act="silu", train=False):
    return {"name": name, "op": "glu", "tokens": tokens, "hidden": hidden, "inter": inter, "dtype": dtype,
            "act": act, "train": train}


def _lora(name, tokens, n_in, n_out, adapters, rank, dtype, mixed=False, weight=True, base=False):
    return {"name": name, "op": "lora", "tokens": tokens, "n_in": n_in, "n_out": n_out, "adapters": adapters,
            "rank": rank, "dtype": dtype, "mixed": mixed, "weight": weight, "base": base}


def listed():
    return [
        # decoding one sequence: the block's weights are streamed for one row
        _glu("glu decode 1", 1, 4096, 2048, "bf16"),
        # a verify batch of eight drafted tokens
        _glu("glu verify 8", 8, 4096, 2048, "fp16"),
        # a decode step of 64 sequences
        _glu("glu batch 64", 64, 4096, 2048, "bf16"),
        # a short prompt through a block of odd sizes, with the other activation
        _glu("glu ragged 333", 333, 1032, 1384, "fp16", act="gelu"),
        # a prefill chunk
        _glu("glu prefill 7168", 7168, 4096, 2048, "bf16"),
        # a training step on a short batch of odd sizes
        _glu("glu train ragged 509", 509, 776, 1304, "fp16", act="gelu", train=True),
        # a training step on a packed batch
        _glu("glu train 16384", 16384, 4096, 2048, "bf16", train=True),
        # decoding one sequence through the down projection with its adapter
        _lora("lora decode 1", 1, 2048, 4096, 8, 16, "bf16"),
        # a decode step of 64 requests with 32 adapters of different ranks
        _lora("lora batch 64", 64, 2048, 4096, 32, 64, "bf16", mixed=True),
        # a prefill chunk of several requests
        _lora("lora prefill 7168", 7168, 2048, 4096, 8, 32, "bf16"),
        # a short mixed batch of odd sizes, with a residual input
        _lora("lora ragged 333", 333, 1384, 1032, 5, 24, "fp16", mixed=True, base=True),
        # adapters beside a projection computed elsewhere (a quantised one)
        _lora("lora beside 2048", 2048, 4096, 4096, 16, 64, "bf16", mixed=True, weight=False, base=True),
    ]


def _spread(rng, low, high, step=1):
    """A multiple of `step` in [low, high], spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(low), math.log(high)))
    return min(high, max(low, int(round(v / step)) * step))


def draw(rng):
    while True:
        dtype = rng.choice(["bf16", "fp16"])
        tokens = _spread(rng, 1, 16384)
        if rng.random() < 0.55:
            c = _glu("", tokens, _spread(rng, 256, 8192, 8), _spread(rng, 128, 16384, 8), dtype,
                     act=rng.choice(["silu", "gelu"]), train=rng.random() < 0.5)
            cost = (6 if c["train"] else 2) * tokens * c["hidden"] * c["inter"]
        else:
            weight = rng.random() < 0.7
            c = _lora("", tokens, _spread(rng, 256, 16384, 8), _spread(rng, 256, 16384, 8), _spread(rng, 1, 64),
                      _spread(rng, 8, 128, 8), dtype, mixed=rng.random() < 0.5, weight=weight,
                      base=not weight or rng.random() < 0.3)
            # the plain form multiplies every token with every adapter
            cost = tokens * (c["n_in"] + c["n_out"]) * c["adapters"] * c["rank"] + tokens * c["n_in"] * c["n_out"]
        if cost <= LARGEST:
            del c["name"]
            return c


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dt)

    T = case["tokens"]
    s = {"case": case}
    if case["op"] == "glu":
        H, I = case["hidden"], case["inter"]
        s.update(x=normal(T, H), w_gate=normal(I, H, std=H ** -0.5), w_up=normal(I, H, std=H ** -0.5))
        s.update(h=torch.empty(T, I, dtype=dt, device="cuda"))
        if case["train"]:
            s.update(dh=normal(T, I, std=0.25))
            for n in ("x", "w_gate", "w_up"):
                s["d" + n] = torch.empty_like(s[n])
        return s
    K, N, n, r = case["n_in"], case["n_out"], case["adapters"], case["rank"]
    s.update(x=normal(T, K), a=normal(n, r, K, std=K ** -0.5), b=normal(n, N, r, std=0.5 * r ** -0.5))
    s["w"] = normal(N, K, std=K ** -0.5) if case["weight"] else None
    s["base"] = normal(T, N) if case["base"] else None
    s["scales"] = torch.rand(n, generator=g, device="cuda") * 1.5 + 0.5
    s["ranks"] = None
    if case["mixed"]:   # ranks in steps of 8, up to the stack's
        s["ranks"] = (torch.randint(1, r // 8 + 1, (n,), generator=g, device="cuda") * 8).to(torch.int32)
    # the tokens of a request stand together; a decode step has one of each;
    # an id of -1 (one in n + 1) has no adapter
    per = 1 if T <= 64 else -(-T // max(4, n))
    ids = torch.randint(-1, n, (-(-T // per),), generator=g, device="cuda")
    s["ids"] = ids.repeat_interleave(per)[:T].to(torch.int32).contiguous()
    s["y"] = torch.empty(T, N, dtype=dt, device="cuda")
    return s


def _run_own(s):
    import trellis_quantized_moe_exl3_amd as M

    c = s["case"]
    if "desc" not in s:   # the descriptor and the workspace a program keeps
        dt = {"bf16": M.DT_BF16, "fp16": M.DT_F16}[c["dtype"]]
        if c["op"] == "glu":
            act = {"silu": M.ACT_SILU, "gelu": M.ACT_GELU_TANH}[c["act"]]
            s["desc"] = M.make_glu_desc(c["hidden"], c["inter"], dt, act)
            size = M.glu_workspace_size(s["desc"], c["tokens"])
            if c["train"]:
                size = max(size, M.glu_backward_workspace_size(s["desc"], c["tokens"]))
                s["pre"] = torch.empty(2, c["tokens"], c["inter"], dtype=torch.float32, device="cuda")
        else:
            s["desc"] = M.make_lora_desc(c["n_in"], c["n_out"], c["adapters"], c["rank"], dt)
            size = M.lora_workspace_size(s["desc"], c["tokens"])
        s["ws"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    if c["op"] == "glu":
        M.glu(s["desc"], s["x"], s["w_gate"], s["w_up"], s["h"], s["ws"], pre=s.get("pre"))
        if not c["train"]:
            return s["h"]
        M.glu_backward(s["desc"], s["x"], s["w_gate"], s["w_up"], s["pre"], s["dh"], s["ws"], dx=s["dx"],
                       dw_gate=s["dw_gate"], dw_up=s["dw_up"])
        return s["h"], s["dx"], s["dw_gate"], s["dw_up"]
    M.lora_linear(s["desc"], s["x"], s["w"], s["a"], s["b"], s["ids"], s["y"], s["ws"], base=s["base"],
                  scales=s["scales"], ranks=s["ranks"])
    return s["y"]


def run(state):
    if own:
        return _run_own(state)
    s = state
    c = s["case"]
    dt = DTYPES[c["dtype"]]
    x = s["x"].float()
    if c["op"] == "glu":
        wg, wu = s["w_gate"].float(), s["w_up"].float()
        g, u = x @ wg.t(), x @ wu.t()
        if c["act"] == "silu":
            p = 1 / (1 + torch.exp(-g))
            a, slope = g * p, p * (1 + g * (1 - p))
        else:
            k = math.sqrt(2 / math.pi)
            p = torch.tanh(k * (g + 0.044715 * g * g * g))
            a = 0.5 * g * (1 + p)
            slope = 0.5 * (1 + p) + 0.5 * g * (1 - p * p) * k * (1 + 3 * 0.044715 * g * g)
        h = (a * u).to(dt)
        if not c["train"]:
            return h
        dh = s["dh"].float()
        dg, du = dh * u * slope, dh * a
        return h, (dg @ wg + du @ wu).to(dt), (dg.t() @ x).to(dt), (du.t() @ x).to(dt)
    n, r, K = s["a"].shape
    col = torch.arange(n * r, device="cuda")
    keep = s["ids"][:, None] == (col // r)[None]
    if s["ranks"] is not None:
        keep &= (col % r < s["ranks"][col // r])[None]
    mid = (x @ s["a"].float().view(n * r, K).t()) * s["scales"][col // r][None]
    y = torch.where(keep, mid, 0) @ s["b"].float().transpose(1, 2).reshape(n * r, -1)
    if s["w"] is not None:
        y = y + x @ s["w"].float().t()
    if s["base"] is not None:
        y = y + s["base"].float()
    return y.to(dt)


def work(case):
    T = case["tokens"]
    if case["op"] == "glu":
        H, I = case["hidden"], case["inter"]
        move, mac = T * H + 2 * I * H + T * I, 2 * T * H * I
        if case["train"]:   # dh in; dx, dW out
            move, mac = move + T * I + T * H + 2 * I * H, 3 * mac
        return {"bytes": 2 * move, "flops": 2 * mac}
    K, N, n, r = case["n_in"], case["n_out"], case["adapters"], case["rank"]
    r = r / 2 if case["mixed"] else r
    used = min(n, T)
    move = T * K + T * N + used * r * (K + N) + (N * K if case["weight"] else 0) + (T * N if case["base"] else 0)
    mac = T * r * (K + N) + (T * N * K if case["weight"] else 0)
    return {"bytes": int(2 * move), "flops": int(2 * mac)}


def exact(case, seed):
    s = prepare(case, seed)
    x = s["x"].double()
    if case["op"] == "glu":
        gate, up = x @ s["w_gate"].double().t(), x @ s["w_up"].double().t()
        gate.requires_grad_(case["train"])
        act = torch.nn.functional.silu(gate) if case["act"] == "silu" else torch.nn.functional.gelu(gate, approximate="tanh")
        if not case["train"]:
            return act * up
        dh = s["dh"].double()
        dgate, = torch.autograd.grad(act, gate, dh * up)
        act = act.detach()
        dup = dh * act
        dx = torch.addmm(dup @ s["w_up"].double(), dgate, s["w_gate"].double())
        return act * up, dx, dgate.t() @ x, dup.t() @ x
    y = torch.zeros(case["tokens"], case["n_out"], dtype=torch.float64, device="cuda")
    if s["w"] is not None:
        y += x @ s["w"].double().t()
    if s["base"] is not None:
        y += s["base"].double()
    for k in range(case["adapters"]):
        rows = torch.nonzero(s["ids"] == k).flatten()
        q = case["rank"] if s["ranks"] is None else int(s["ranks"][k])
        low = x[rows] @ s["a"][k, :q].double().t()
        y[rows] += float(s["scales"][k]) * (low @ s["b"][k, :, :q].double().t())
    return y
