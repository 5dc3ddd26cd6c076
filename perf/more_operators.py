"""The operators for a MoE layer with experts of its user's own, as cases to
measure.

Three kinds: tokens sorted by expert and back (`sort`, `dispatch`, `combine`
and their gradients), dropout from a counter-based generator, and products
with 4-bit weights and group scales, dense or by expert.  `run` computes a
case either in its plain form (elementary torch operations in fp32, rounded
once) or, with `own`, through this package's entry points; `exact` computes it
from the definition in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}

# What the largest listed cases move or compute; drawn cases stay below.
LARGEST_TOKENS = 16384 * 8 * 4096        # elements of the sorted rows
LARGEST_DROPOUT = 16384 * 4096           # elements
LARGEST_WEIGHTS = 58 * 2 * 2048 * 4096   # 4-bit weights of the named experts
LARGEST_MACS = 16384 * 2048 * 4096       # multiply-adds


def _w4(name, rows, n_in, n_out, dtype, experts=1, used=1, group=128, zeros=False, base=False, act=""):
    """act: the gated pair of products; used: experts that have rows."""
    return {"name": name, "op": "w4", "rows": rows, "n_in": n_in, "n_out": n_out, "dtype": dtype, "experts": experts,
            "used": used, "group": group, "zeros": zeros, "base": base, "act": act}


def _tokens(name, part, tokens, hidden, experts, top_k, dtype, weights="out", drops=False, base=False, p=0.0):
    """part: dispatch, combine, or train (both, with their gradients); weights:
    on the experts' output or input; drops: some slots have no expert."""
    return {"name": name, "op": "tokens", "part": part, "tokens": tokens, "hidden": hidden, "experts": experts,
            "top_k": top_k, "dtype": dtype, "weights": weights, "drops": drops, "base": base, "p": p}


def _dropout(name, rows, cols, dtype, p, residual=True, train=True):
    return {"name": name, "op": "dropout", "rows": rows, "cols": cols, "dtype": dtype, "p": p, "residual": residual,
            "train": train}


def listed():
    return [
        # decoding one sequence: a projection's weights are streamed for one row
        _w4("w4 decode 1", 1, 2048, 4096, "bf16"),
        # a verify batch of eight tokens through the gated pair of their experts
        _w4("w4 experts 8 tokens", 64, 4096, 2048, "fp16", experts=288, used=58, act="silu"),
        # a decode step of 64 sequences
        _w4("w4 batch 64", 64, 4096, 4096, "bf16", group=64, zeros=True),
        # short requests at five experts of odd sizes, fine groups, a residual
        _w4("w4 ragged 333", 333, 1376, 1032, "fp16", experts=5, used=4, group=32, zeros=True, base=True),
        # a prefill chunk's rows at the experts' down projection
        _w4("w4 experts 16384", 16384, 2048, 4096, "bf16", experts=32, used=32),
        # a verify batch on its way to the experts
        _tokens("dispatch 8", "dispatch", 8, 4096, 288, 8, "bf16"),
        # a prefill chunk on its way to the experts, and back beside a shared expert
        _tokens("dispatch 7168", "dispatch", 7168, 4096, 288, 8, "fp16"),
        _tokens("combine 7168", "combine", 7168, 4096, 288, 8, "bf16", base=True),
        # training steps: a short batch of odd sizes whose crowded experts turn
        # tokens away, and a packed batch
        _tokens("train ragged 509", "train", 509, 776, 40, 3, "fp16", weights="in", drops=True, p=0.1),
        _tokens("train 16384", "train", 16384, 4096, 288, 8, "bf16", base=True, p=0.1),
        # a branch of odd sizes before it is added, and its gradient
        _dropout("dropout ragged 509", 509, 1381, "fp16", 0.25),
        # the same in a packed batch
        _dropout("dropout 16384", 16384, 4096, "bf16", 0.1),
    ]


def _spread(rng, low, high, step=1):
    """A multiple of `step` in [low, high], spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(low), math.log(high)))
    return min(high, max(low, int(round(v / step)) * step))


def draw(rng):
    while True:
        dtype = rng.choice(["bf16", "fp16"])
        kind = rng.random()
        if kind < 0.45:
            rows, group = _spread(rng, 1, 16384), rng.choice([32, 64, 128])
            experts = 1 if rng.random() < 0.4 else _spread(rng, 2, 288)
            act = rng.choice(["", "", "silu", "gelu"])
            c = _w4("", rows, _spread(rng, 256, 16384, group), _spread(rng, 128, 16384, 8), dtype, experts,
                    min(experts, rows, _spread(rng, 1, experts)), group, rng.random() < 0.5,
                    act == "" and rng.random() < 0.3, act)
            weights = (2 if act else 1) * c["n_in"] * c["n_out"]
            if c["used"] * weights > LARGEST_WEIGHTS or rows * weights > LARGEST_MACS:
                continue
            if experts * weights > 288 * 2 * 2048 * 4096:   # the stack's own size
                continue
        elif kind < 0.8:
            experts = _spread(rng, 1, 1024)
            k = rng.randint(1, min(experts, 16))
            c = _tokens("", rng.choice(["dispatch", "combine", "train"]), _spread(rng, 1, 16384),
                        _spread(rng, 128, 8192, 8), experts, k, dtype, rng.choice(["in", "out"]), rng.random() < 0.3,
                        rng.random() < 0.5, rng.choice([0.0, round(rng.uniform(0.01, 0.6), 3)]))
            if c["tokens"] * k * c["hidden"] > LARGEST_TOKENS:
                continue
        else:
            c = _dropout("", _spread(rng, 1, 16384), _spread(rng, 1, 16384), dtype, round(rng.uniform(0.0, 0.9), 3),
                         rng.random() < 0.5, rng.random() < 0.5)
            if c["rows"] * c["cols"] > LARGEST_DROPOUT:
                continue
        del c["name"]
        return c


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dt)

    def whole(low, high, shape, dtype):
        return torch.randint(low, high, shape, generator=g, device="cuda", dtype=dtype)

    s = {"case": case}
    if case["op"] == "w4":
        R, K, N, E, G = (case[n] for n in ("rows", "n_in", "n_out", "experts", "group"))
        s["x"] = normal(R, K)
        s["w"] = []
        for _ in range(2 if case["act"] else 1):
            # weights of a standard deviation of about K^-0.5
            scales = ((torch.rand(E, N, K // G, generator=g, device="cuda") + 0.5) * (K ** -0.5 / 4.6)).to(dt)
            zeros = whole(5, 12, (E, N, K // G), torch.uint8) if case["zeros"] else None
            s["w"].append((whole(0, 256, (E, N, K // 2), torch.uint8), scales, zeros))
        s["base"] = normal(R, N) if case["base"] else None
        # rows of each expert: one at least for `used` of them, the rest skewed
        h = torch.Generator().manual_seed(seed)
        named = torch.randperm(E, generator=h)[:case["used"]]
        rows = torch.zeros(E, dtype=torch.int64)
        rows[named] = 1
        if R > case["used"]:
            popular = torch.exp(torch.randn(case["used"], generator=h))
            extra = torch.multinomial(popular, R - case["used"], replacement=True, generator=h)
            rows += torch.bincount(named[extra], minlength=E)
        s["bounds"] = [0] + torch.cumsum(rows, 0).tolist()
        s["offsets"] = torch.tensor(s["bounds"], dtype=torch.int32).cuda()
        s["y"] = torch.zeros(R, N, dtype=dt, device="cuda")
        return s
    s["rng"] = torch.randint(0, 1 << 62, (2,), generator=g, device="cuda")
    if case["op"] == "dropout":
        R, C = case["rows"], case["cols"]
        s.update(x=normal(R, C), y=torch.empty(R, C, dtype=dt, device="cuda"))
        s["residual"] = normal(R, C) if case["residual"] else None
        if case["train"]:
            s.update(dy=normal(R, C), dx=torch.empty(R, C, dtype=dt, device="cuda"))
        return s
    T, H, E, k = (case[n] for n in ("tokens", "hidden", "experts", "top_k"))
    # the k experts of largest logits, some experts more popular than others
    logits = torch.randn(T, E, generator=g, device="cuda") + 0.5 * torch.randn(E, generator=g, device="cuda")
    top, idx = torch.topk(logits, k, dim=1)
    if case["drops"]:
        idx = torch.where(torch.rand(T, k, generator=g, device="cuda") < 1 / 16, -1, idx)
    s.update(idx=idx.to(torch.int32), weights=torch.softmax(top, 1))
    s.update(x=normal(T, H), z=normal(T * k, H), base=normal(T, H) if case["base"] else None)
    if case["part"] == "train":
        s.update(dy=normal(T, H), dxs=normal(T * k, H))
    for n, shape in (("counts", E), ("offsets", E + 1), ("sorted_ids", T * k), ("pos", T * k)):
        s[n] = torch.zeros(shape, dtype=torch.int32, device="cuda")
    for n, rows in (("xs", T * k), ("y", T), ("dz", T * k), ("dx", T)):
        s[n] = torch.zeros(rows, H, dtype=dt, device="cuda")
    s["dw"] = torch.zeros(T, k, device="cuda")
    if case["part"] == "combine":   # the tables of the way there
        s["offsets"], s["sorted_ids"], s["pos"] = _sort(s["idx"], E)
    return s


# ---- this package's entry points


def _own_w4(M, s):
    c = s["case"]
    if "desc" not in s:   # the descriptor and the workspace a program keeps
        act = {"": M.ACT_SILU, "silu": M.ACT_SILU, "gelu": M.ACT_GELU_TANH}[c["act"]]
        s["desc"] = M.make_w4_desc(c["n_in"], c["n_out"], c["experts"], c["group"],
                                   {"bf16": M.DT_BF16, "fp16": M.DT_F16}[c["dtype"]], act)
        s["ws"] = torch.empty(M.w4_workspace_size(s["desc"], c["rows"]), dtype=torch.uint8, device="cuda")
        s["packed"] = [M.make_w4(*w) for w in s["w"]]
    offsets = s["offsets"] if c["experts"] > 1 else None
    if c["act"]:
        M.w4_glu(s["desc"], s["x"], s["packed"][0], s["packed"][1], s["y"], s["ws"], offsets=offsets)
    else:
        M.w4_linear(s["desc"], s["x"], s["packed"][0], s["y"], s["ws"], offsets=offsets, base=s["base"])
    return s["y"]


def _own_dropout(M, s):
    c = s["case"]
    M.dropout(s["x"], s["y"], c["p"], s["rng"], residual=s["residual"])
    if not c["train"]:
        return s["y"]
    M.dropout(s["dy"], s["dx"], c["p"], s["rng"])
    return s["y"], s["dx"]


def _own_tokens(M, s):
    c = s["case"]
    if "desc" not in s:
        s["desc"] = M.make_tokens_desc(c["hidden"], c["experts"], c["top_k"], {"bf16": M.DT_BF16, "fp16": M.DT_F16}[c["dtype"]])
        s["ws"] = torch.empty(M.sort_workspace_size(s["desc"], c["tokens"]), dtype=torch.uint8, device="cuda")
    d, pos = s["desc"], s["pos"]
    w_in, w_out = (s["weights"], None) if c["weights"] == "in" else (None, s["weights"])
    drop = {"p": c["p"], "rng": s["rng"]} if c["p"] > 0 else {}
    if c["part"] != "combine":
        M.sort(d, s["idx"], s["counts"], s["offsets"], s["sorted_ids"], pos, s["ws"])
        M.dispatch(d, s["x"], pos, s["xs"], w=w_in)
        there = s["offsets"], s["sorted_ids"], pos, s["xs"]
        if c["part"] == "dispatch":
            return there
    M.combine(d, s["z"], pos, s["y"], w=w_out, base=s["base"], **drop)
    if c["part"] == "combine":
        return s["y"]
    dw = s["dw"]
    M.combine_backward(d, s["dy"], s["z"], pos, s["dz"], w=w_out, dw=None if w_out is None else dw, **drop)
    M.dispatch_backward(d, s["dxs"], s["x"], pos, s["dx"], w=w_in, dw=None if w_in is None else dw)
    return there + (s["y"], s["dz"], dw, s["dx"])


# ---- the plain forms


def _matrix(w, e, G):
    """The weights of expert e in fp32."""
    codes, scales, zeros = w
    q = torch.stack((codes[e] & 15, codes[e] >> 4), -1).float()
    z = 8.0 if zeros is None else zeros[e].float()[:, :, None]
    q = q.view(q.shape[0], -1, G)
    return ((q - z) * scales[e].float()[:, :, None]).view(q.shape[0], -1)


def _plain_w4(s):
    c, b = s["case"], s["bounds"]
    x, y = s["x"].float(), torch.zeros(c["rows"], c["n_out"], device="cuda")
    for e in range(c["experts"]):
        if b[e] == b[e + 1]:
            continue
        rows = x[b[e]:b[e + 1]]
        v = rows @ _matrix(s["w"][0], e, c["group"]).t()
        if c["act"]:
            if c["act"] == "silu":
                v = v / (1 + torch.exp(-v))
            else:
                v = 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v * v * v)))
            v = v * (rows @ _matrix(s["w"][1], e, c["group"]).t())
        y[b[e]:b[e + 1]] = v
    if s["base"] is not None:
        y = y + s["base"].float()
    return y.to(s["x"].dtype)


def _keep(rows, cols, p, rng):
    """The kept elements and their factor.  Element (r, c) has 16 bits of its
    own: halfword c % 8 of Philox4x32-10 at the counter offset + r ceil(cols / 8)
    + c / 8 under the key `seed`; it is kept where they reach p 2^16."""
    low = 0xFFFFFFFF
    blocks = -(-cols // 8)
    seed, offset = rng[0], rng[1]
    n = torch.arange(rows * blocks, device="cuda") + offset
    x0, x1 = n & low, (n >> 32) & low
    x2 = x3 = torch.zeros_like(n)
    k0, k1 = seed & low, (seed >> 32) & low
    for _ in range(10):
        a, b = x0 * 0xD2511F53, x2 * 0xCD9E8D57   # modulo 2^64
        x0, x1, x2, x3 = ((b >> 32) & low) ^ x1 ^ k0, b & low, ((a >> 32) & low) ^ x3 ^ k1, a & low
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    half = torch.stack([v for x in (x0, x1, x2, x3) for v in (x & 0xFFFF, x >> 16)], -1)
    least = math.floor(p * 65536 + 0.5)
    factor = 65536 / (65536 - least) if least < 65536 else 0.0
    return half.view(rows, blocks * 8)[:, :cols] >= least, factor


def _plain_dropout(s):
    c = s["case"]
    keep, factor = _keep(c["rows"], c["cols"], c["p"], s["rng"])
    y = torch.where(keep, s["x"].float() * factor, 0)
    if s["residual"] is not None:
        y = y + s["residual"].float()
    y = y.to(s["x"].dtype)
    if not c["train"]:
        return y
    return y, torch.where(keep, s["dy"].float() * factor, 0).to(y.dtype)


def _sort(idx, E):
    """offsets, sorted_ids and pos of a stable sort of the slots by expert."""
    e = idx.flatten().long()
    valid = e >= 0
    order = torch.sort(torch.where(valid, e, E), stable=True).indices
    n = e.numel()
    pos = torch.empty_like(e)
    pos[order] = torch.arange(n, device="cuda")
    counts = torch.zeros(E + 1, dtype=torch.int64, device="cuda")
    counts.scatter_add_(0, torch.where(valid, e, E), torch.ones_like(e))
    offsets = torch.cat((torch.zeros_like(counts[:1]), torch.cumsum(counts[:E], 0)))
    ids = torch.where(torch.arange(n, device="cuda") < offsets[E], order, 0)
    return offsets.int(), ids.int(), torch.where(valid, pos, -1).int()


def _plain_tokens(s):
    c = s["case"]
    T, H, k = c["tokens"], c["hidden"], c["top_k"]
    dt = s["x"].dtype
    w = s["weights"]
    offsets, ids, pos = _sort(s["idx"], c["experts"]) if c["part"] != "combine" else (None, None, s["pos"])
    at, there = pos.long().clamp(min=0), (pos >= 0)[:, None]
    token = torch.arange(T * k, device="cuda") // k

    def spread(rows, weights):   # rows of tokens, to the sorted rows
        v = rows[token]
        if weights is not None:
            v = v * weights.reshape(-1, 1)
        full = torch.zeros(T * k + 1, H, device="cuda")
        full[torch.where(pos >= 0, pos, T * k).long()] = v
        return full[:T * k].to(dt)

    def gather(rows, weights):   # sorted rows, summed at their tokens
        v = torch.where(there, rows.float()[at], 0)
        if weights is not None:
            v = v * weights.reshape(-1, 1)
        return v.view(T, k, H).sum(1)

    def products(sorted_rows, rows):
        v = torch.where(there, sorted_rows.float()[at], 0).view(T, k, H)
        return (v * rows[:, None]).sum(2)

    w_in, w_out = (w, None) if c["weights"] == "in" else (None, w)
    x = s["x"].float()
    if c["part"] != "combine":
        xs = spread(x, w_in)
        if c["part"] == "dispatch":
            return offsets, ids, pos, xs
    y = gather(s["z"], w_out)
    if c["p"] > 0:
        keep, factor = _keep(T, H, c["p"], s["rng"])
        y = torch.where(keep, y * factor, 0)
    if s["base"] is not None:
        y = y + s["base"].float()
    y = y.to(dt)
    if c["part"] == "combine":
        return y
    dy = s["dy"].float()
    if c["p"] > 0:
        dy = torch.where(keep, dy * factor, 0)
    dz = spread(dy, w_out)
    dw = products(s["z"], dy) if w_in is None else products(s["dxs"], x)
    return offsets, ids, pos, xs, y, dz, dw, gather(s["dxs"], w_in).to(dt)


def run(state):
    op = state["case"]["op"]
    if own:
        import trellis_quantized_moe_exl3_amd as M

        return {"w4": _own_w4, "dropout": _own_dropout, "tokens": _own_tokens}[op](M, state)
    return {"w4": _plain_w4, "dropout": _plain_dropout, "tokens": _plain_tokens}[op](state)


def work(case):
    if case["op"] == "w4":
        R, K, N, G = (case[n] for n in ("rows", "n_in", "n_out", "group"))
        pair = 2 if case["act"] else 1
        column = K / 2 + K // G * (3 if case["zeros"] else 2)
        move = case["used"] * pair * N * column + 2 * R * (K + N * (2 if case["base"] else 1))
        return {"bytes": int(move), "flops": 2 * pair * R * N * K}
    if case["op"] == "dropout":
        n = case["rows"] * case["cols"]
        steps = 2 if case["train"] else 1
        return {"bytes": 2 * n * (2 * steps + (1 if case["residual"] else 0)), "flops": 2 * n * steps}
    T, H, k = case["tokens"], case["hidden"], case["top_k"]
    row, rows = 2 * T * H, 2 * T * k * H
    base = row if case["base"] else 0
    # each part reads or writes the sorted rows once and the tokens' once, the
    # slots' tables and weights beside them; combine's gradient has z and dz,
    # and whichever carries weights reads rows for their gradient
    move = {"dispatch": row + rows, "combine": row + rows + base}
    move["train"] = move["dispatch"] + move["combine"] + (row + rows + (rows if case["weights"] == "out" else 0)) \
        + (row + rows + (row if case["weights"] == "in" else 0))
    flops = {"dispatch": 1, "combine": 2, "train": 7}[case["part"]] * T * k * H
    tables = {"dispatch": 12, "combine": 8, "train": 32}[case["part"]] * T * k
    return {"bytes": move[case["part"]] + tables, "flops": flops}


# ---- the definitions in 64 bits


def _exact_keep(rows, cols, p, rng):
    seed, offset = (int(v) for v in rng.tolist())
    blocks = (cols + 7) // 8
    with np.errstate(over="ignore"):
        n = np.arange(rows * blocks, dtype=np.uint64) + np.uint64(offset)
        ctr = [n.astype(np.uint32), (n >> np.uint64(32)).astype(np.uint32)]
        ctr += [np.zeros_like(ctr[0]), np.zeros_like(ctr[0])]
        key = [seed % 2 ** 32, seed // 2 ** 32]
        for _ in range(10):
            first = ctr[0].astype(np.uint64) * np.uint64(0xD2511F53)
            second = ctr[2].astype(np.uint64) * np.uint64(0xCD9E8D57)
            ctr = [(second >> np.uint64(32)).astype(np.uint32) ^ ctr[1] ^ np.uint32(key[0]), second.astype(np.uint32),
                   (first >> np.uint64(32)).astype(np.uint32) ^ ctr[3] ^ np.uint32(key[1]), first.astype(np.uint32)]
            key = [(key[0] + 0x9E3779B9) % 2 ** 32, (key[1] + 0xBB67AE85) % 2 ** 32]
    bits = np.stack(ctr, 1).view(np.uint16).reshape(rows, blocks * 8)[:, :cols]   # low half first
    least = int(p * 65536 + 0.5)
    if least == 65536:
        return torch.zeros(rows, cols, dtype=torch.float64, device="cuda")
    return torch.from_numpy(bits >= least).cuda().double() * (65536.0 / (65536 - least))


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    if c["op"] == "w4":
        x, b, G = s["x"].double(), s["bounds"], c["group"]
        y = torch.zeros(c["rows"], c["n_out"], dtype=torch.float64, device="cuda")
        for e in [e for e in range(c["experts"]) if b[e + 1] > b[e]]:
            out = []
            for codes, scales, zeros in s["w"]:
                w = torch.empty(c["n_out"], c["n_in"], dtype=torch.float64, device="cuda")
                w[:, 0::2] = codes[e] % 16
                w[:, 1::2] = codes[e] // 16
                w -= 8 if zeros is None else zeros[e].double().repeat_interleave(G, 1)
                w *= scales[e].double().repeat_interleave(G, 1)
                out.append(x[b[e]:b[e + 1]] @ w.t())
            if c["act"] == "silu":
                out[0] = torch.nn.functional.silu(out[0])
            elif c["act"] == "gelu":
                out[0] = torch.nn.functional.gelu(out[0], approximate="tanh")
            y[b[e]:b[e + 1]] = out[0] * out[1] if c["act"] else out[0]
        return y if s["base"] is None else y + s["base"].double()
    if c["op"] == "dropout":
        m = _exact_keep(c["rows"], c["cols"], c["p"], s["rng"])
        y = s["x"].double() * m
        if s["residual"] is not None:
            y += s["residual"].double()
        return (y, s["dy"].double() * m) if c["train"] else y
    T, H, E, k = c["tokens"], c["hidden"], c["experts"], c["top_k"]
    # slot numbers of each expert in order, on the host
    e = s["idx"].cpu().numpy().reshape(-1)
    order = np.lexsort((np.arange(e.size), e))
    order = order[e[order] >= 0]
    pos = np.full(e.size, -1, np.int32)
    pos[order] = np.arange(order.size)
    ids = np.zeros(e.size, np.int32)
    ids[:order.size] = order
    offsets = np.searchsorted(e[order], np.arange(E + 1)).astype(np.int32)
    tables = tuple(torch.from_numpy(v).cuda() for v in (offsets, ids, pos))
    slots = torch.from_numpy(order).cuda()
    token, n = slots // k, order.size
    w = s["weights"].double()
    one = torch.ones_like(w)
    w_in, w_out = (w, one) if c["weights"] == "in" else (one, w)
    m = _exact_keep(T, H, c["p"], s["rng"]) if c["part"] != "dispatch" and c["p"] > 0 else None

    def there(rows, weights):
        v = torch.zeros(T * k, H, dtype=torch.float64, device="cuda")
        v[:n] = rows[token] * weights.flatten()[slots][:, None]
        return v

    def back(rows, weights):
        v = torch.zeros(T, H, dtype=torch.float64, device="cuda")
        return v.index_add_(0, token, rows[:n].double() * weights.flatten()[slots][:, None])

    if c["part"] != "combine":
        xs = there(s["x"].double(), w_in)
        if c["part"] == "dispatch":
            return tables + (xs,)
    y = back(s["z"], w_out)
    if m is not None:
        y *= m
    if s["base"] is not None:
        y += s["base"].double()
    if c["part"] == "combine":
        return y
    dy = s["dy"].double()
    if m is not None:
        dy = dy * m
    dw = torch.zeros(T * k, dtype=torch.float64, device="cuda")
    if c["weights"] == "in":
        dw[slots] = (s["dxs"][:n].double() * s["x"].double()[token]).sum(1)
    else:
        dw[slots] = (s["z"][:n].double() * dy[token]).sum(1)
    return tables + (xs, y, there(dy, w_out), dw.view(T, k), back(s["dxs"], w_in))
