"""Operators around 8-bit block-scaled weights, as cases to measure.

Three operators, each in its plain form (elementary torch operations in 32
bits, 64 where a value next to a rounding border or to another router logit
is decided) and, where ``own`` is true, as a user calls the library:

  quantise   X (float32 or bfloat16) to e4m3 codes with one float32 scale for
             each block of 128, along the rows of X and of its transpose;
  product    C = alpha * A B^T + beta * C of two matrices of e4m3 codes, with
             A's scales for 1 x 128 blocks and B's for 1 x 128 or 128 x 128;
  layer      a mixture-of-experts layer for at most 64 tokens: router, top-k,
             gated products of the chosen experts, weighted sum.

A matrix of codes has rows that start at multiples of 16 bytes; its scales
are stored block by block: S[b, i] belongs to columns [128 b, 128 b + 128) of
row i (or of rows [128 i, 128 i + 128)).
"""
import math

import torch

own = False

BLOCK = 128
TOP = 448.0              # largest e4m3 value
SMALLEST = 2.0 ** -126   # smallest scale
E4M3 = torch.float8_e4m3fn
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": E4M3}


def blocks(n):
    return -(-n // BLOCK)


def listed():
    return [
        # -- quantise: one token of a decode step, the activations or output
        #    gradients of a training step (codes for the product that reads
        #    rows and for the weight gradient, which reads columns), a weight
        #    matrix whose sides fit no block
        {"name": "quantise one token", "op": "quantise", "rows": 1, "cols": 4096, "type": "bf16", "block": "row", "normal": True, "transposed": False, "pad": 0},
        {"name": "quantise activations both ways", "op": "quantise", "rows": 8192, "cols": 8192, "type": "f32", "block": "row", "normal": True, "transposed": True, "pad": 0},
        {"name": "quantise ragged weights", "op": "quantise", "rows": 3001, "cols": 2047, "type": "bf16", "block": "tile", "normal": True, "transposed": True, "pad": 5},
        # -- product: one token through a small projection, a decode batch
        #    through a large one, a ragged prefill, a large forward product,
        #    a weight gradient added to what earlier micro-batches left
        {"name": "product one row", "op": "product", "M": 1, "N": 1024, "K": 1024, "blockB": "tile", "type": "bf16", "beta": 0.0},
        {"name": "product 32 rows", "op": "product", "M": 32, "N": 8192, "K": 8192, "blockB": "tile", "type": "bf16", "beta": 0.0},
        {"name": "product ragged", "op": "product", "M": 517, "N": 2047, "K": 3001, "blockB": "tile", "type": "f32", "beta": 0.0},
        {"name": "product 4096", "op": "product", "M": 4096, "N": 4096, "K": 4096, "blockB": "tile", "type": "bf16", "beta": 0.0},
        {"name": "product weight gradient", "op": "product", "M": 8192, "N": 8192, "K": 8192, "blockB": "row", "type": "f32", "beta": 0.5},
        # -- layer: one token of a small model, a few tokens with weights in
        #    bfloat16, a batch whose routing came with the call (some slots
        #    belong to experts elsewhere) with weights in float32, many small
        #    experts in 8 bits
        {"name": "layer one token", "op": "layer", "T": 1, "E": 8, "k": 2, "H": 1024, "I": 512, "type": "bf16", "weights": "e4m3", "router": True, "renormalize": True},
        {"name": "layer 8 tokens", "op": "layer", "T": 8, "E": 64, "k": 6, "H": 2048, "I": 1408, "type": "bf16", "weights": "bf16", "router": True, "renormalize": False},
        {"name": "layer 64 tokens routed", "op": "layer", "T": 64, "E": 16, "k": 2, "H": 2048, "I": 2000, "type": "f32", "weights": "f32", "router": False, "renormalize": True},
        {"name": "layer 16 tokens of 128 experts", "op": "layer", "T": 16, "E": 128, "k": 8, "H": 4096, "I": 1536, "type": "f32", "weights": "e4m3", "router": True, "renormalize": True},
    ]


def draw(rng):
    def size(lo, hi):
        n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
        n = max(lo, min(hi, n))
        return n if rng.random() < 0.5 else max(lo, n // 16 * 16)  # odd ones and round ones

    op = rng.choice(("quantise", "product", "product", "layer", "layer"))
    if op == "quantise":
        way = rng.choice(((True, False), (False, True), (True, True)))
        return {"op": op, "rows": size(1, 8192), "cols": size(16, 8192), "type": rng.choice(("f32", "bf16")),
                "block": rng.choice(("row", "tile")), "normal": way[0], "transposed": way[1], "pad": rng.choice((0, 0, 3, 8))}
    if op == "product":
        few = rng.random() < 0.4  # a decode step's rows
        return {"op": op, "M": size(1, 64) if few else size(65, 8192), "N": size(64, 8192), "K": size(64, 8192),
                "blockB": rng.choice(("tile", "row")), "type": rng.choice(("f32", "bf16")), "beta": rng.choice((0.0, 0.0, 0.5))}
    experts = size(4, 128)
    return {"op": op, "T": size(1, 64), "E": experts, "k": min(experts, rng.randint(1, 8)), "H": size(64, 4096), "I": size(32, 2048),
            "type": rng.choice(("f32", "bf16")), "weights": rng.choice(("e4m3", "e4m3", "bf16", "f32")), "router": rng.random() < 0.7,
            "renormalize": rng.random() < 0.5}


# ---- inputs ----------------------------------------------------------------

def padded(shape, dtype):
    """An uninitialised array whose rows start at multiples of 16 bytes."""
    per = 16 // torch.empty((), dtype=dtype).element_size()
    wide = -(-shape[-1] // per) * per
    return torch.empty(*shape[:-1], wide, dtype=dtype, device="cuda")[..., :shape[-1]]


def in_blocks(w, rows):
    """w [..., R, C] (float32) as codes and scales of rows x 128 blocks."""
    R, C = w.shape[-2:]
    nr, nc = -(-R // rows), blocks(C)
    full = torch.nn.functional.pad(w, (0, nc * BLOCK - C, 0, nr * rows - R))
    full = full.view(*w.shape[:-2], nr, rows, nc, BLOCK)
    s = (full.abs().amax(dim=(-3, -1)) / TOP).clamp_min(SMALLEST)          # [..., nr, nc]
    full = full / s[..., :, None, :, None]
    codes = padded(w.shape, E4M3)
    codes.copy_(full.reshape(*w.shape[:-2], nr * rows, nc * BLOCK)[..., :R, :C])
    return codes, s.transpose(-1, -2).contiguous()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))

    def normal(*shape, scale=1.0):
        return torch.randn(*shape, generator=g, device="cuda") * scale

    s = {"case": case}
    if case["op"] == "quantise":
        R, C, dt = case["rows"], case["cols"], TYPES[case["type"]]
        x = normal(R, C + case["pad"])
        x = x * torch.exp(normal(C + case["pad"]))       # columns of different size, as activations have
        s["X"] = x.to(dt)[:, :C]
        if case["normal"]:
            s["Q"] = padded((R, C), E4M3)
            s["S"] = torch.empty(blocks(C), R if case["block"] == "row" else blocks(R), device="cuda")
        if case["transposed"]:
            s["QT"] = padded((C, R), E4M3)
            s["ST"] = torch.empty(blocks(R), C if case["block"] == "row" else blocks(C), device="cuda")
        return s
    if case["op"] == "product":
        M, N, K = case["M"], case["N"], case["K"]
        spread = torch.exp(0.5 * normal(K))
        s["A"], s["SA"] = in_blocks(normal(M, K) * spread, 1)
        s["B"], s["SB"] = in_blocks(normal(N, K, scale=K ** -0.5), BLOCK if case["blockB"] == "tile" else 1)
        s["C"] = normal(M, N).to(TYPES[case["type"]]) if case["beta"] else torch.empty(M, N, dtype=TYPES[case["type"]], device="cuda")
        s["workspace"] = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
        return s
    T, E, k, H, I = (case[n] for n in ("T", "E", "k", "H", "I"))
    dt, wt = TYPES[case["type"]], TYPES[case["weights"]]
    s["x"] = normal(T, H).to(dt)
    for name, rows, cols in (("gate", I, H), ("up", I, H), ("down", H, I)):
        w = normal(E, rows, cols, scale=cols ** -0.5)
        if case["weights"] == "e4m3":
            s[name], s["s_" + name] = in_blocks(w, BLOCK)
        else:
            s[name] = padded((E, rows, cols), wt)
            s[name].copy_(w)
    if case["router"]:
        s["router"] = normal(E, H, scale=H ** -0.5)
        s["ids"] = torch.empty(T, k, dtype=torch.int32, device="cuda")
        s["weights"] = torch.empty(T, k, device="cuda")
    else:
        s["ids"] = torch.rand(T, E, generator=g, device="cuda").topk(k, dim=1).indices.to(torch.int32)
        s["ids"][torch.rand(T, k, generator=g, device="cuda") < 0.125] = -1   # experts elsewhere
        s["weights"] = torch.softmax(normal(T, k), dim=1)
    s["out"] = torch.empty(T, H, dtype=dt, device="cuda")
    s["workspace"] = torch.empty(16 << 20, dtype=torch.uint8, device="cuda")
    return s


# ---- plain forms -----------------------------------------------------------

def to_e4m3(q):
    """The nearest e4m3 values to q (float64, at most 448 after rounding),
    ties to the even code."""
    exponent = torch.frexp(q).exponent - 1
    step = torch.exp2((exponent.clamp_min(-6) - 3).double())
    return (torch.round(q / step) * step).float().to(E4M3)


def plain_quantise(x, rows):
    """Codes and scales (block by block) of rows x 128 blocks of x."""
    R, C = x.shape
    nr, nc = -(-R // rows), blocks(C)
    x = torch.nn.functional.pad(x.float(), (0, nc * BLOCK - C, 0, nr * rows - R)).view(nr, rows, nc, BLOCK)
    s = (x.abs().amax(dim=(1, 3)).double() / TOP).clamp_min(SMALLEST).float()   # 64 bits: the scale nearest to the quotient
    q = to_e4m3(x.double() / s.double()[:, None, :, None])   # 64 bits: quotients next to the middle of two codes
    return q.view(nr * rows, nc * BLOCK)[:R, :C], s.t()


def plain_values(codes, scales, rows):
    """What codes [..., R, C] with scales of rows x 128 blocks stand for."""
    R, C = codes.shape[-2:]
    s = scales.transpose(-1, -2).repeat_interleave(rows, dim=-2)[..., :R, :].repeat_interleave(BLOCK, dim=-1)[..., :C]
    return codes.float() * s


def plain_layer(s):
    case = s["case"]
    T, E, k = case["T"], case["E"], case["k"]
    x, ids, weights = s["x"].float(), s["ids"].long(), s["weights"]
    if case["router"]:
        logits = s["x"].double() @ s["router"].double().t()    # 64 bits: logits next to each other
        order = torch.sort(logits, dim=1, descending=True, stable=True)
        ids = order.indices[:, :k]
        best = order.values[:, :k]
        weights = torch.softmax(best, dim=1) if case["renormalize"] else torch.exp(best - torch.logsumexp(logits, 1, keepdim=True))
        weights = weights.float()
    at = ids.clamp_min(0).reshape(-1)
    by_pair = T * k < E   # fewer pairs of token and expert than experts

    def taken(name):
        w = s[name]
        sc = s.get("s_" + name)
        if by_pair:
            w, sc = (w.view(torch.uint8)[at].view(E4M3) if sc is not None else w[at]), (sc[at] if sc is not None else None)
        return w.float() if sc is None else plain_values(w, sc, BLOCK)

    share = torch.where(ids >= 0, weights, torch.zeros_like(weights))
    if by_pair:
        rows = x.repeat_interleave(k, dim=0)[:, :, None]                             # [T k, H, 1]
        g, u = torch.bmm(taken("gate"), rows), torch.bmm(taken("up"), rows)
        h = g / (1 + torch.exp(-g)) * u
        y = torch.bmm(taken("down"), h)[:, :, 0].view(T, k, -1)
        out = (share[:, :, None] * y).sum(dim=1)
    else:
        g, u = torch.matmul(x, taken("gate").transpose(1, 2)), torch.matmul(x, taken("up").transpose(1, 2))  # [E, T, I]
        h = g / (1 + torch.exp(-g)) * u
        y = torch.matmul(h, taken("down").transpose(1, 2))                           # [E, T, H]
        mix = torch.zeros(T, E, device="cuda").scatter_add_(1, ids.clamp_min(0), share)
        out = (mix.t()[:, :, None] * y).sum(dim=0)
    return ids.to(torch.int32), weights, out.to(s["x"].dtype)


# ---- one pass --------------------------------------------------------------

def run(s):
    case = s["case"]
    if case["op"] == "quantise":
        if own:
            import fp32_gemm_tile_amd as fg
            fg.quantize_fp8(s["X"], s.get("Q"), s.get("S"), s.get("QT"), s.get("ST"), block=case["block"])
            return {n: s[n] for n in ("Q", "S", "QT", "ST") if n in s}
        rows = 1 if case["block"] == "row" else BLOCK
        out = {}
        if case["normal"]:
            out["Q"], out["S"] = plain_quantise(s["X"], rows)
        if case["transposed"]:
            out["QT"], out["ST"] = plain_quantise(s["X"].t(), rows)
        return out
    if case["op"] == "product":
        if own:
            import fp32_gemm_tile_amd as fg
            return fg.gemm_fp8(s["A"], s["SA"], s["B"], s["SB"], s["C"], beta=case["beta"], workspace=s["workspace"])
        a = plain_values(s["A"], s["SA"], 1)
        b = plain_values(s["B"], s["SB"], BLOCK if case["blockB"] == "tile" else 1)
        c = a @ b.t()
        if case["beta"]:
            c = c + case["beta"] * s["C"].float()
        s["C"] = c.to(s["C"].dtype)
        return s["C"]
    if own:
        import fp32_gemm_tile_amd as fg
        scales = (s["s_gate"], s["s_up"], s["s_down"]) if case["weights"] == "e4m3" else None
        fg.moe(s["x"], s["gate"], s["up"], s["down"], s["ids"], s["weights"], s["out"], router=s.get("router"),
               renormalize=case["renormalize"], scales=scales, workspace=s["workspace"])
        return {"ids": s["ids"], "weights": s["weights"], "out": s["out"]}
    ids, weights, out = plain_layer(s)
    return {"ids": s["ids"] if not case["router"] else ids, "weights": weights, "out": out}


def work(case):
    size = {"f32": 4, "bf16": 2, "e4m3": 1}
    if case["op"] == "quantise":
        R, C = case["rows"], case["cols"]
        n = case["normal"] + case["transposed"]
        return {"bytes": R * C * (size[case["type"]] + n) + 4 * n * R * C / BLOCK / (1 if case["block"] == "row" else BLOCK), "flops": 3 * n * R * C}
    if case["op"] == "product":
        M, N, K = case["M"], case["N"], case["K"]
        scales = 4 * blocks(K) * (M + (N if case["blockB"] == "row" else blocks(N)))
        return {"bytes": M * K + N * K + scales + M * N * size[case["type"]] * (2 if case["beta"] else 1), "flops": 2.0 * M * N * K}
    T, E, k, H, I = (case[n] for n in ("T", "E", "k", "H", "I"))
    slots = k if case["router"] else 0.875 * k
    used = E * (1 - (1 - slots / E) ** T)   # experts that some token chose, on average
    n = used * 3 * H * I * size[case["weights"]] + 2 * T * H * size[case["type"]] + (4 * E * H if case["router"] else 0)
    return {"bytes": n, "flops": 2.0 * T * (slots * 3 * H * I + (E * H if case["router"] else 0))}


# ---- the definitions in 64 bits --------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quantise":
        grid = torch.arange(0, 127, dtype=torch.uint8).view(E4M3).double().cuda()   # the 127 finite magnitudes
        middle = (grid[1:] + grid[:-1]) / 2
        tall = 1 if case["block"] == "row" else BLOCK
        out = {}
        for codes, scales, x in (("Q", "S", s["X"]), ("QT", "ST", s["X"].t())):
            if codes not in s:
                continue
            x = x.double().contiguous()
            R, C = x.shape
            r, c = torch.arange(R, device="cuda") // tall, torch.arange(C, device="cuda") // BLOCK
            flat = (r[:, None] * blocks(C) + c[None, :]).reshape(-1)
            most = torch.zeros((R - 1) // tall * blocks(C) + blocks(C), dtype=torch.float64, device="cuda")
            most.scatter_reduce_(0, flat, x.abs().reshape(-1), "amax")
            sc = torch.clamp(most / TOP, min=SMALLEST).float().double()   # a scale is a float32
            q = x.abs() / sc[flat].view(R, C)
            low = torch.bucketize(q, middle)                              # ties end on the lower of two codes ...
            low += (low < 126) & (q == middle[low.clamp_max(125)]) & (low % 2 == 1)   # ... and go on where that is odd
            out[codes] = grid[low] * torch.sign(x)
            out[scales] = sc.view(-1, blocks(C)).t().contiguous()
        return out
    if case["op"] == "product":
        def wide(codes, scales, tall):
            r, c = (torch.arange(n, device="cuda") for n in codes.shape)
            return codes.double() * scales.double()[c[None, :] // BLOCK, r[:, None] // tall]
        a, b = wide(s["A"], s["SA"], 1), wide(s["B"], s["SB"], BLOCK if case["blockB"] == "tile" else 1)
        c = torch.mm(a, b.t().contiguous())
        return c + case["beta"] * s["C"].double() if case["beta"] else c
    T, E, k, H, I = (case[n] for n in ("T", "E", "k", "H", "I"))
    x = s["x"].double()
    ids, weights = s["ids"].long(), s["weights"].double()
    if case["router"]:
        p = torch.softmax(torch.mm(x, s["router"].double().t().contiguous()), dim=1)
        weights, ids = torch.topk(p, k, dim=1)
        if case["renormalize"]:
            weights = weights / weights.sum(dim=1, keepdim=True)
    out = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    for e in sorted(set(ids.reshape(-1).tolist()) - {-1}):
        def matrix(name):
            w = s[name][e].double()
            if case["weights"] != "e4m3":
                return w
            r, c = (torch.arange(n, device="cuda") for n in w.shape)
            return w * s["s_" + name][e].double()[c[None, :] // BLOCK, r[:, None] // BLOCK]
        t, j = torch.nonzero(ids == e, as_tuple=True)
        g, u = torch.mm(x[t], matrix("gate").t().contiguous()), torch.mm(x[t], matrix("up").t().contiguous())
        y = torch.mm(g * torch.sigmoid(g) * u, matrix("down").t().contiguous())
        out.index_add_(0, t, weights[t, j][:, None] * y)
    return {"ids": None, "weights": weights, "out": out}
