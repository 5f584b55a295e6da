"""Cases of the quantized experts, the token order they need and low-rank adapters.

Three operators next to the product with a quantized weight:
  route     tokens sorted by expert and back: the stable order of the (token, choice) slots,
            the rows in that order, the weighted sum back, and the gradients;
  experts   the products of sorted rows with the quantized weights of their experts, and the
            gradient of the rows;
  adapters  low-rank adapters of many requests beside one shared projection (quantized, or
            any other whose output is the base), and the gradients of rows and factors.

``run`` computes them in plain torch operations in 32 bits, or (``own``) through the package.
"""
import math

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one token of a chat on a two-of-eight expert model: launches are what it costs
        dict(name="route-token", op="route", tokens=1, topk=2, experts=8, hidden=4096,
             dtype="f16", dropped=0.0, train=False),
        # a prompt batch through the same model
        dict(name="route-prompt", op="route", tokens=8192, topk=2, experts=8, hidden=4096,
             dtype="f16", dropped=0.0, train=False),
        # a training step with eight choices of 64 experts, a tenth of them over capacity
        # (dropped), a token count that no tile divides
        dict(name="route-train", op="route", tokens=4095, topk=8, experts=64, hidden=8192,
             dtype="bf16", dropped=0.1, train=True),
        # one token's two up-projections from the eight experts' 4-bit weights
        dict(name="experts-token", op="experts", tokens=1, topk=2, experts=8, N=11008, K=4096,
             nbits=4, group=64, train=False),
        # decoding a batch of 48 requests: about a dozen rows an expert, 2-bit weights
        dict(name="experts-batch", op="experts", tokens=48, topk=2, experts=8, N=4096, K=11008,
             nbits=2, group=32, train=False),
        # a prompt batch: about 500 rows an expert
        dict(name="experts-prompt", op="experts", tokens=2048, topk=2, experts=8, N=11008, K=4096,
             nbits=4, group=64, train=False),
        # the gradient of the rows through the frozen experts, ragged token count
        dict(name="experts-train", op="experts", tokens=2001, topk=2, experts=8, N=4096, K=4096,
             nbits=4, group=64, train=True),
        # one request with its adapter on a 4096 x 4096 projection
        dict(name="adapters-token", op="adapters", rows=1, N=4096, K=4096, rank=16, adapters=8,
             nbits=4, group=64, dtype="f16", none=0.0, train=False),
        # decoding 64 requests of 32 adapters, an eighth of them without one
        dict(name="adapters-batch", op="adapters", rows=64, N=8192, K=8192, rank=16, adapters=32,
             nbits=2, group=32, dtype="f16", none=0.125, train=False),
        # prompts of eight adapters
        dict(name="adapters-prompt", op="adapters", rows=4096, N=8192, K=8192, rank=64, adapters=8,
             nbits=4, group=64, dtype="f16", none=0.1, train=False),
        # training four adapters on the frozen quantized weight
        dict(name="adapters-train", op="adapters", rows=2048, N=4096, K=4096, rank=32, adapters=4,
             nbits=4, group=64, dtype="f16", none=0.0, train=True),
        # training three bfloat16 adapters beside a projection of the caller's own, ragged rows
        dict(name="adapters-train-bf16", op="adapters", rows=8190, N=11008, K=4096, rank=16,
             adapters=3, nbits=0, group=0, dtype="bf16", none=0.05, train=True),
    ]


# ------------------------------------------------------------------- sizes --

def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _cost(case):
    """Seconds of a pass at rates the plain forms come near to: 3 TB/s and 60 TFLOP/s."""
    w = work(case)
    return w["bytes"] / 3e12 + w["flops"] / 6e13


def draw(rng):
    """One more case of the same ranges: sizes over their logarithm, odd ones among them."""
    most = {}
    for c in listed():
        most[c["op"]] = max(most.get(c["op"], 0.0), _cost(c))
    while True:
        op = rng.choice(["route", "experts", "adapters"])
        train = rng.random() < 0.4
        if op == "route":
            experts = _log(rng, 1, 256)
            case = dict(op=op, tokens=_log(rng, 1, 16384), topk=min(rng.choice([1, 2, 3, 4, 8]), experts),
                        experts=experts, hidden=_log(rng, 64, 8192), dtype=rng.choice(list(DTYPES)),
                        dropped=rng.choice([0.0, 0.0, 0.1, 0.5]), train=train)
        elif op == "experts":
            group = rng.choice([16, 32, 64, 128])
            unit = max(32, group)
            experts = _log(rng, 1, 32)
            case = dict(op=op, tokens=_log(rng, 1, 3000), topk=min(rng.choice([1, 2, 4]), experts),
                        experts=experts, N=_log(rng, 100, 11008),
                        K=max(unit, _log(rng, 256, 11008) // unit * unit), nbits=rng.choice([2, 3, 4, 8]),
                        group=group, train=train)
            if experts * case["N"] * case["K"] > 8 * 11008 * 4096:
                continue
        else:
            group = rng.choice([16, 32, 64, 128])
            unit = max(32, group)
            nbits = rng.choice([0, 2, 3, 4, 8])
            case = dict(op=op, rows=_log(rng, 1, 8190), N=_log(rng, 100, 11008),
                        K=max(unit, _log(rng, 256, 8192) // unit * unit),
                        rank=rng.choice([8, 16, 24, 32, 64, 128]), adapters=_log(rng, 1, 64),
                        nbits=nbits, group=group if nbits else 0,
                        dtype="f16" if nbits else rng.choice(["f16", "bf16"]),
                        none=rng.choice([0.0, 0.1, 0.5]), train=train)
        if _cost(case) <= most[op]:
            return case


def work(case):
    if case["op"] == "route":
        e = DTYPES[case["dtype"]].itemsize
        T, S, H = case["tokens"], case["tokens"] * case["topk"], case["hidden"]
        slots = 4 * S * 4 + 4 * (case["experts"] + 1)        # ids, order, position, weights
        b = slots + e * H * (2 * T + 2 * S)                  # rows out, the weighted sum back
        f = 2 * S * H
        if case["train"]:                                    # d(rows), d(weights), d(tokens)
            b += e * H * (2 * T + 3 * S) + 4 * S
            f += 4 * S * H
        return {"bytes": b, "flops": f}
    if case["op"] == "experts":
        S, N, K = case["tokens"] * case["topk"], case["N"], case["K"]
        used = min(case["experts"], S)
        weight = used * (N * K * case["nbits"] // 8 + 4 * N * K // case["group"])
        rows = 2 * S * K + 2 * S * N if case["train"] else 2 * case["tokens"] * K + 2 * S * N
        return {"bytes": weight + rows, "flops": 2 * S * N * K}
    M, N, K, r = case["rows"], case["N"], case["K"], case["rank"]
    used = min(case["adapters"], M)
    factors = used * r * (N + K)
    weight, flops = 0, 4 * M * r * (N + K) // 2
    base = 0
    if case["nbits"]:
        weight = N * K * case["nbits"] // 8 + 4 * N * K // case["group"]
        flops += 2 * M * N * K
    else:
        base = 2 * M * (K if case["train"] else N)           # the caller's own projection or its gradient
    if not case["train"]:
        return {"bytes": weight + base + 2 * factors + 2 * M * (K + N), "flops": flops}
    # rows and gradients read, d(rows) written, the factors read, their gradients written in 32 bits
    return {"bytes": weight + base + 2 * factors + 4 * case["adapters"] * r * (N + K) + 2 * M * (2 * K + N),
            "flops": flops + 4 * M * r * (N + K)}


# ------------------------------------------------------------------ inputs --

def _weight(rows, cols, nbits, group, gen):
    """A stored weight: packed codes, binary16 scales and zero-points in code units."""
    qmax = (1 << nbits) - 1
    g = rows * cols // group
    packed = torch.randint(0, 256, (rows * cols * nbits // 8,), generator=gen, device="cuda", dtype=torch.uint8)
    scale = (torch.rand(g, generator=gen, device="cuda") * 0.8 + 0.6) * (0.06 / qmax)
    zero = qmax / 2 + torch.randn(g, generator=gen, device="cuda") * 0.05 * qmax
    shape = (rows, cols // group)
    return packed, scale.half().view(shape), zero.half().view(shape)


def _choices(tokens, topk, experts, dropped, gen):
    """Distinct experts of every token, with some choices dropped (-1)."""
    noise = torch.rand((tokens, experts), generator=gen, device="cuda")
    skew = torch.linspace(0.3, 0.0, experts, device="cuda")  # some experts are liked more
    ids = (noise + skew).topk(topk, dim=1).indices.to(torch.int32)
    gone = torch.rand((tokens, topk), generator=gen, device="cuda") < dropped
    return torch.where(gone, torch.full_like(ids, -1), ids).contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))

    def normal(*shape, dtype=torch.float16, std=1.0):
        return (torch.randn(shape, generator=gen, device="cuda") * std).to(dtype)

    s = {"case": case}
    if case["op"] == "route":
        dt = DTYPES[case["dtype"]]
        T, k, H = case["tokens"], case["topk"], case["hidden"]
        s["ids"] = _choices(T, k, case["experts"], case["dropped"], gen)
        s["x"] = normal(T, H, dtype=dt)
        s["w"] = torch.rand((T, k), generator=gen, device="cuda")
        s["y"] = normal(T * k, H, dtype=dt)
        if case["train"]:
            s["dout"] = normal(T, H, dtype=dt, std=1e-2)
            s["dxs"] = normal(T * k, H, dtype=dt, std=1e-2)
    elif case["op"] == "experts":
        T, k, E, N, K = case["tokens"], case["topk"], case["experts"], case["N"], case["K"]
        s["ids"] = _choices(T, k, E, 0.0, gen)
        s["packed"], s["scale"], s["zero"] = _weight(E * N, K, case["nbits"], case["group"], gen)
        if case["train"]:
            s["dy"] = normal(T * k, N, std=1e-2)
        else:
            s["x"] = normal(T, K)
    else:
        dt = DTYPES[case["dtype"]]
        M, N, K, r, n = case["rows"], case["N"], case["K"], case["rank"], case["adapters"]
        ids = torch.randint(0, n, (M,), generator=gen, device="cuda", dtype=torch.int32)
        gone = torch.rand((M,), generator=gen, device="cuda") < case["none"]
        s["ids"] = torch.where(gone, torch.full_like(ids, -1), ids)
        s["x"] = normal(M, K, dtype=dt)
        s["A"] = normal(n, r, K, dtype=dt, std=K ** -0.5)
        s["B"] = normal(n, N, r, dtype=dt, std=0.1)
        s["scales"] = torch.rand(n, generator=gen, device="cuda") + 0.5
        if case["nbits"]:
            s["packed"], s["scale"], s["zero"] = _weight(N, K, case["nbits"], case["group"], gen)
        else:
            s["base"] = normal(M, K if case["train"] else N, dtype=dt, std=1e-2 if case["train"] else 1.0)
        if case["train"]:
            s["dy"] = normal(M, N, dtype=dt, std=1e-2)
    if own:
        import bit_weight_quantization_amd as hq
        if "packed" in s:
            rows = case["N"] * case.get("experts", 1)
            s["q"] = hq.QuantizedWeight(packed=s["packed"], scale=s["scale"], zero=s["zero"], rows=rows,
                                        cols=case["K"], nbits=case["nbits"], group_size=case["group"])
    return s


# ------------------------------------------------------------- plain forms --

def _unpack(packed, nbits):
    """The codes of an LSB-first bitstream as float32."""
    if nbits == 8:
        return packed.float()
    if nbits == 3:  # 8 codes in 3 bytes
        b = packed.view(-1, 3).to(torch.int32)
        word = b[:, 0] | (b[:, 1] << 8) | (b[:, 2] << 16)
        shifts = torch.arange(0, 24, 3, device=packed.device, dtype=torch.int32)
        return ((word[:, None] >> shifts) & 7).view(-1).float()
    shifts = torch.arange(0, 8, nbits, device=packed.device, dtype=torch.uint8)
    return ((packed[:, None] >> shifts) & ((1 << nbits) - 1)).view(-1).float()


def _plain_weight(s, expert=0):
    """s (q - z) of one expert's N x K weight."""
    c = s["case"]
    N, K, b, g = c["N"], c["K"], c["nbits"], c["group"]
    step = N * K * b // 8
    q = _unpack(s["packed"][expert * step:(expert + 1) * step], b).view(N, K // g, g)
    sl = slice(expert * N, (expert + 1) * N)
    return (s["scale"][sl].float()[:, :, None] * (q - s["zero"][sl].float()[:, :, None])).view(N, K)


def _plain_order(ids, experts):
    """order (the slots by expert, dropped ones last as ~slot), position (its inverse, ~row
    for dropped slots), offsets of the experts."""
    flat = ids.view(-1).long()
    n = flat.numel()
    key = torch.where((flat >= 0) & (flat < experts), flat, torch.full_like(flat, experts))
    key, order = torch.sort(key, stable=True)
    position = torch.empty_like(order)
    position[order] = torch.arange(n, device=ids.device)
    gone = key == experts
    offsets = torch.searchsorted(key, torch.arange(experts + 1, device=ids.device))
    code = torch.where(gone, ~order, order)
    position = torch.where(gone[position], ~position, position)
    return code.int(), position.int(), offsets.int()


def _plain_back(rows, position, weights, T, k):
    """The weighted sum of every token's kept rows, in 32 bits."""
    pos = position.view(T, k).long()
    keep = (pos >= 0)[:, :, None]
    acc = torch.zeros((T, rows.shape[1]), device=rows.device)
    for j in range(k):
        row = rows[pos[:, j].clamp(min=0)].float()
        if weights is not None:
            row = row * weights[:, j, None]
        acc = acc + torch.where(keep[:, j], row, torch.zeros_like(row))
    return acc.to(rows.dtype)


def _plain_route(s):
    c = s["case"]
    T, k = c["tokens"], c["topk"]
    order, position, offsets = _plain_order(s["ids"], c["experts"])
    kept = (order >= 0)[:, None]
    slot = torch.where(order >= 0, order, ~order).long()
    token = slot // k
    xs = torch.where(kept, s["x"][token], torch.zeros((), dtype=s["x"].dtype, device="cuda"))
    out = _plain_back(s["y"], position, s["w"], T, k)
    if not c["train"]:
        return [order, position, offsets, xs, out]
    d = s["dout"][token].float()
    w = s["w"].view(-1)[slot][:, None]
    zero = torch.zeros((), device="cuda")
    dy = torch.where(kept, d * w, zero).to(s["y"].dtype)
    dot = torch.where(kept[:, 0], (d * s["y"].float()).sum(1), zero)
    dw = torch.zeros(T * k, device="cuda")
    dw[slot] = dot
    dx = _plain_back(s["dxs"], position, None, T, k)
    return [order, position, offsets, xs, out, dy, dw.view(T, k), dx]


def _plain_experts(s):
    c = s["case"]
    E, N, K, k = c["experts"], c["N"], c["K"], c["topk"]
    order, _, offsets = _plain_order(s["ids"], E)
    at = offsets.tolist()
    src = s["dy"].float() if c["train"] else s["x"][(order // k).long()].float()
    out = torch.zeros((order.numel(), K if c["train"] else N), device="cuda")
    for e in range(E):
        if at[e + 1] > at[e]:
            w = _plain_weight(s, e)
            rows = src[at[e]:at[e + 1]]
            out[at[e]:at[e + 1]] = rows @ w if c["train"] else rows @ w.t()
    return [out.half()]


def _plain_adapters(s):
    c = s["case"]
    M, r, n = c["rows"], c["rank"], c["adapters"]
    dt = DTYPES[c["dtype"]]
    ids, x = s["ids"].long(), s["x"].float()
    if c["train"]:
        y = s["dy"].float() @ _plain_weight(s) if c["nbits"] else s["base"].float()
    else:
        y = x @ _plain_weight(s).t() if c["nbits"] else s["base"].float()
    if not c["train"]:
        if M * r * (c["K"] + c["N"]) <= 1 << 26:  # few rows: every row's own factors
            safe = ids.clamp(min=0)
            v = torch.matmul(s["A"][safe].float(), x[:, :, None])
            v = torch.matmul(s["B"][safe].float(), v)[:, :, 0] * s["scales"][safe][:, None]
            return [(y + torch.where((ids >= 0)[:, None], v, torch.zeros_like(v))).to(dt)]
        y = y.clone()
        for a in range(n):
            rows = torch.nonzero(ids == a)[:, 0]
            v = (x[rows] @ s["A"][a].float().t()) @ s["B"][a].float().t()
            y[rows] += s["scales"][a] * v
        return [y.to(dt)]
    dx, dy = y.clone(), s["dy"].float()
    dA, dB = torch.zeros(s["A"].shape, device="cuda"), torch.zeros(s["B"].shape, device="cuda")
    for a in range(n):
        rows = torch.nonzero(ids == a)[:, 0]
        A, B, d, xr = s["A"][a].float(), s["B"][a].float(), dy[rows] * s["scales"][a], x[rows]
        u = d @ B
        dx[rows] += u @ A
        dA[a] = u.t() @ xr
        dB[a] = d.t() @ (xr @ A.t())
    return [dx.to(dt), dA, dB]


def run(state):
    c = state["case"]
    if not own:
        return {"route": _plain_route, "experts": _plain_experts, "adapters": _plain_adapters}[c["op"]](state)
    import bit_weight_quantization_amd as hq
    s = state
    if c["op"] == "route":
        route = hq.expert_sort(s["ids"], c["experts"])
        xs = hq.expert_gather(s["x"], route)
        out = hq.expert_combine(s["y"], route, s["w"])
        if not c["train"]:
            return [route.order, route.position, route.offsets, xs, out]
        dy, dw = hq.expert_combine_backward(s["dout"], s["y"], route, s["w"])
        dx = hq.expert_combine(s["dxs"], route)  # the gradient of the gather
        return [route.order, route.position, route.offsets, xs, out, dy, dw, dx]
    if c["op"] == "experts":
        route = hq.expert_sort(s["ids"], c["experts"])
        if c["train"]:
            return [hq.matmul_experts_backward(s["dy"], s["q"], route)]
        return [hq.matmul_experts(s["x"], s["q"], route)]
    if c["nbits"]:
        if c["train"]:
            return list(hq.matmul_adapters_backward(s["dy"], s["x"], s["q"], s["A"], s["B"], s["ids"], s["scales"]))
        return [hq.matmul_adapters(s["x"], s["q"], s["A"], s["B"], s["ids"], s["scales"])]
    if c["train"]:
        return list(hq.adapters_backward(s["dy"], s["x"], s["A"], s["B"], s["ids"], s["scales"], base=s["base"]))
    return [hq.adapters(s["x"], s["A"], s["B"], s["ids"], s["scales"], base=s["base"])]


# ------------------------------------------------------------------- exact --

def _exact_weight(s, e):
    """s (q - z) of expert e in 64 bits, code by code from its bit position."""
    c = s["case"]
    N, K, b, g = c["N"], c["K"], c["nbits"], c["group"]
    bit = torch.arange(N * K, device="cuda") * b + e * N * K * b
    byte = bit >> 3
    last = s["packed"].numel() - 1
    pair = s["packed"][byte].int() | (s["packed"][(byte + 1).clamp(max=last)].int() << 8)
    q = ((pair >> (bit & 7).int()) & ((1 << b) - 1)).double().view(N, K)
    scale = s["scale"][e * N:(e + 1) * N].double().repeat_interleave(g, dim=1)
    zero = s["zero"][e * N:(e + 1) * N].double().repeat_interleave(g, dim=1)
    return scale * q - scale * zero


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    c = case
    if c["op"] == "route":
        T, k, H = c["tokens"], c["topk"], c["hidden"]
        flat = s["ids"].view(-1).tolist()
        slots = [i for of_one in _of(flat, c["experts"]) for i in of_one]
        n, kept = T * k, len(slots)
        slots_t = torch.tensor(slots, dtype=torch.long, device="cuda")
        xs = torch.zeros((n, H), dtype=torch.float64, device="cuda")
        xs[:kept] = s["x"].double()[slots_t // k]
        w = s["w"].double().view(-1)[slots_t]
        out = torch.zeros((T, H), dtype=torch.float64, device="cuda")
        out.index_add_(0, slots_t // k, s["y"][:kept].double() * w[:, None])
        found = [None, None, None, xs, out]
        if c["train"]:
            dy = torch.zeros((n, H), dtype=torch.float64, device="cuda")
            d = s["dout"].double()[slots_t // k]
            dy[:kept] = d * w[:, None]
            dw = torch.zeros(n, dtype=torch.float64, device="cuda")
            dw[slots_t] = torch.linalg.vecdot(d, s["y"][:kept].double())
            dx = torch.zeros((T, H), dtype=torch.float64, device="cuda")
            dx.index_add_(0, slots_t // k, s["dxs"][:kept].double())
            found += [dy, dw.view(T, k), dx]
        return found
    if c["op"] == "experts":
        k = c["topk"]
        by = _of(s["ids"].view(-1).tolist(), c["experts"])
        parts, at = [], 0
        for e in range(c["experts"]):
            if not by[e]:
                continue
            w = _exact_weight(s, e)
            if c["train"]:
                parts.append(s["dy"][at:at + len(by[e])].double() @ w)
            else:
                rows = torch.tensor(by[e], dtype=torch.long, device="cuda") // k
                parts.append(s["x"][rows].double() @ w.t())
            at += len(by[e])
        return [torch.cat(parts)]
    x, ids = s["x"].double(), s["ids"]
    grad = s["dy"].double() if c["train"] else None
    if c["nbits"]:
        w = _exact_weight(s, 0)
        total = grad @ w if c["train"] else x @ w.t()
    else:
        total = s["base"].double()
    dA = torch.zeros(s["A"].shape, dtype=torch.float64, device="cuda")
    dB = torch.zeros(s["B"].shape, dtype=torch.float64, device="cuda")
    for a in range(c["adapters"]):
        on = (ids == a).double()[:, None] * s["scales"][a].double()
        if not bool((ids == a).any()):
            continue
        A, B = s["A"][a].double(), s["B"][a].double()
        if c["train"]:
            scaled = grad * on
            total = total + (scaled @ B) @ A
            dA[a] = (scaled @ B).t() @ x
            dB[a] = scaled.t() @ (x @ A.t())
        else:
            total = total + (on * x) @ A.t() @ B.t()
    return [total, dA, dB] if c["train"] else [total]


def _of(flat, experts):
    """The slots of every expert, in order."""
    by = [[] for _ in range(experts)]
    for i, e in enumerate(flat):
        if 0 <= e < experts:
            by[e].append(i)
    return by
