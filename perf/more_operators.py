"""Operators of a gated feed-forward block, as cases to measure.

Four operators, each in its plain form (elementary torch operations in 32
bits, 64 where a value next to a rounding border is decided) and, where
``own`` is true, as a user calls the library:

  forward     h = act(x gate^T) * (x up^T), the pre-activations x gate^T and
              x up^T kept in x's type for the backward pass, or not kept;
  checkpoint  the same with the pre-activations kept as e4m3 codes and a
              float32 scale for each block of 128 columns of a row;
  backward    the gradients of x, gate and up from h's, and h again, from
              what forward or checkpoint kept;
  int4        x W^T, or act(x Wg^T) * (x Wu^T), for at most 64 rows and
              weights of 4 bits with a scale (and a zero point, or 8) for
              each group of columns of a row: w = s (q - z).

Rows of x, gate, up and of codes start at multiples of 16 bytes. Scales are
stored group by group: S[b, i] belongs to group b of row i's columns. Column
c of a row of 4-bit codes is in byte c // 2, the even one in its low half.
"""
import math

import torch

own = False

BLOCK = 128
TOP = 448.0              # largest e4m3 value
SMALLEST = 2.0 ** -126   # smallest scale of a block
E4M3 = torch.float8_e4m3fn
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
LARGEST = 8.0 * 4096 * 4096 * 8192   # operations of the largest listed case


def cdiv(a, b):
    return -(-a // b)


def listed():
    return [
        # -- forward: one token of a decode step, a decode batch, a ragged
        #    prompt in float32 whose pre-activations are kept, a training step
        {"name": "gated one token", "op": "forward", "T": 1, "H": 2048, "I": 1408, "type": "bf16", "act": "silu", "save": "none"},
        {"name": "gated 32 tokens", "op": "forward", "T": 32, "H": 4096, "I": 8192, "type": "bf16", "act": "gelu", "save": "none"},
        {"name": "gated ragged f32", "op": "forward", "T": 517, "H": 2047, "I": 3001, "type": "f32", "act": "silu", "save": "same"},
        {"name": "gated 4096", "op": "forward", "T": 4096, "H": 4096, "I": 8192, "type": "bf16", "act": "silu", "save": "same"},
        # -- checkpoint: a short sequence, a long training step
        {"name": "checkpoint short", "op": "checkpoint", "T": 200, "H": 2048, "I": 1408, "type": "bf16", "act": "gelu", "save": "e4m3"},
        {"name": "checkpoint 8192 tokens", "op": "checkpoint", "T": 8192, "H": 2048, "I": 8192, "type": "bf16", "act": "silu", "save": "e4m3"},
        # -- backward: a short sequence added to what earlier ones left, from
        #    8 bits; a training step; a ragged one in float32
        {"name": "backward short", "op": "backward", "T": 200, "H": 2048, "I": 1408, "type": "bf16", "act": "gelu", "save": "e4m3", "beta": 1.0},
        {"name": "backward 4096", "op": "backward", "T": 4096, "H": 4096, "I": 8192, "type": "bf16", "act": "silu", "save": "same", "beta": 0.0},
        {"name": "backward ragged f32", "op": "backward", "T": 1025, "H": 1536, "I": 2047, "type": "f32", "act": "silu", "save": "same", "beta": 0.5},
        # -- int4: one token through a projection, one through a large gated
        #    pair with small groups, a decode batch in float32
        {"name": "int4 one token", "op": "int4", "T": 1, "N": 4096, "K": 4096, "group": 128, "type": "bf16", "scales": "bf16", "zeros": False, "gated": False},
        {"name": "int4 one token gated", "op": "int4", "T": 1, "N": 8192, "K": 8192, "group": 32, "type": "bf16", "scales": "f32", "zeros": True, "gated": True},
        {"name": "int4 16 tokens f32", "op": "int4", "T": 16, "N": 8192, "K": 8192, "group": 64, "type": "f32", "scales": "f32", "zeros": True, "gated": False},
    ]


def draw(rng):
    def size(lo, hi):
        n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
        n = max(lo, min(hi, n))
        return n if rng.random() < 0.5 else max(lo, n // 16 * 16)  # odd ones and round ones

    while True:
        op = rng.choice(("forward", "forward", "checkpoint", "backward", "backward", "int4", "int4"))
        if op == "int4":
            return {"op": op, "T": size(1, 64), "N": size(64, 16384), "K": size(64, 16384), "group": rng.choice((32, 64, 128)),
                    "type": rng.choice(("f32", "bf16", "bf16")), "scales": rng.choice(("f32", "bf16")), "zeros": rng.random() < 0.5,
                    "gated": rng.random() < 0.3}
        few = op == "forward" and rng.random() < 0.4  # a decode step's tokens
        case = {"op": op, "T": size(1, 64) if few else size(65, 8192), "H": size(64, 8192), "I": size(64, 8192), "type": rng.choice(("f32", "bf16", "bf16")),
                "act": rng.choice(("silu", "silu", "gelu")), "save": "e4m3" if op == "checkpoint" else rng.choice(("same", "none" if op == "forward" else "e4m3"))}
        if op == "backward":
            case["beta"] = rng.choice((0.0, 0.0, 1.0))
        if work(case)["flops"] * (4 if case["type"] == "f32" else 1) <= LARGEST:
            return case


# ---- inputs ----------------------------------------------------------------

def padded(rows, cols, dtype):
    """An uninitialised matrix whose rows start at multiples of 16 bytes."""
    per = 16 // torch.empty((), dtype=dtype).element_size()
    return torch.empty(rows, cdiv(cols, per) * per, dtype=dtype, device="cuda")[:, :cols]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))

    def normal(rows, cols, dtype=None, scale=1.0):
        v = torch.randn(rows, cols, generator=g, device="cuda") * scale
        if dtype is None:
            return v
        out = padded(rows, cols, dtype)
        out.copy_(v)
        return out

    s = {"case": case}
    dt = TYPES[case["type"]]
    if case["op"] == "int4":
        T, N, K, group = (case[n] for n in ("T", "N", "K", "group"))
        s["x"] = padded(T, K, dt)
        s["x"].copy_(normal(T, K) * torch.exp(0.5 * normal(1, K)))   # channels of different size, as activations have
        s["weights"] = []
        for _ in range(2 if case["gated"] else 1):
            codes = padded(N, cdiv(K, 2), torch.uint8)
            codes.copy_(torch.randint(0, 256, (N, cdiv(K, 2)), generator=g, device="cuda", dtype=torch.uint8))
            scales = (torch.exp(0.3 * normal(cdiv(K, group), N)) * (0.2 * K ** -0.5)).to(TYPES[case["scales"]])
            zeros = torch.round(7.5 + 1.5 * normal(cdiv(K, group), N)).clamp(0, 15).to(torch.uint8) if case["zeros"] else None
            s["weights"].append((codes, scales, zeros))
        s["out"] = torch.empty(T, N, dtype=dt, device="cuda")
        return s
    T, H, I = (case[n] for n in ("T", "H", "I"))
    s["x"] = padded(T, H, dt)
    s["x"].copy_(normal(T, H) * torch.exp(0.5 * normal(1, H)))
    s["gate"], s["up"] = (normal(I, H, dt, H ** -0.5) for _ in range(2))
    s["workspace"] = torch.empty((128 << 20) + 8 * T * (I + 128), dtype=torch.uint8, device="cuda")
    s["h"] = torch.empty(T, I, dtype=dt, device="cuda")
    if case["op"] == "backward":
        s["dh"] = normal(T, I).to(dt)
        s["dx"] = torch.empty(T, H, dtype=dt, device="cuda")
        s["dgate"], s["dup"] = (normal(I, H).to(dt) if case["beta"] else torch.empty(I, H, dtype=dt, device="cuda") for _ in range(2))
    s["saved"] = ()
    for _ in range(0 if case["save"] == "none" else 2):
        if case["save"] == "same":
            s["saved"] += (1.5 * normal(T, I).to(dt),)
        else:
            v = torch.nn.functional.pad(1.5 * normal(T, I), (0, cdiv(I, BLOCK) * BLOCK - I)).view(T, cdiv(I, BLOCK), BLOCK)
            sc = (v.abs().amax(dim=2) / TOP).clamp_min(SMALLEST)
            codes = padded(T, I, E4M3)
            codes.copy_((v / sc[:, :, None]).view(T, -1)[:, :I])
            s["saved"] += (codes, sc.t().contiguous())
    return s


# ---- plain forms -----------------------------------------------------------

def plain_act(v, act):
    """The activation and its derivative."""
    if act == "silu":
        t = 1 / (1 + torch.exp(-v))
        return v * t, t * (1 + v * (1 - t))
    phi = 0.5 * (1 + torch.erf(v * math.sqrt(0.5)))
    return v * phi, phi + v * torch.exp(-0.5 * v * v) * (1 / math.sqrt(2 * math.pi))


def plain_codes(v):
    """v (float32) as e4m3 codes and scales of blocks of 128 columns."""
    T, I = v.shape
    v = torch.nn.functional.pad(v, (0, cdiv(I, BLOCK) * BLOCK - I)).view(T, -1, BLOCK)
    s = (v.abs().amax(dim=2).double() / TOP).clamp_min(SMALLEST).float()
    q = v.double() / s.double()[:, :, None]                  # 64 bits: quotients next to the middle of two codes
    step = torch.exp2(((torch.frexp(q).exponent - 1).clamp_min(-6) - 3).double())
    return (torch.round(q / step) * step).float().to(E4M3).view(T, -1)[:, :I], s.t()


def plain_saved(s):
    """gate's and up's products from what was kept, in 32 bits."""
    if s["case"]["save"] == "same":
        return s["saved"][0].float(), s["saved"][1].float()
    I = s["case"]["I"]
    codes, scales = s["saved"][0::2], s["saved"][1::2]
    return tuple(c.float() * t.t().repeat_interleave(BLOCK, dim=1)[:, :I] for c, t in zip(codes, scales))


def plain_weights(codes, scales, zeros, K, group):
    q = torch.stack((codes & 15, codes >> 4), dim=2).view(codes.shape[0], -1)[:, :K].float()
    z = 8.0 if zeros is None else zeros.float().t().repeat_interleave(group, dim=1)[:, :K]
    return (q - z) * scales.float().t().repeat_interleave(group, dim=1)[:, :K]


# ---- one pass --------------------------------------------------------------

def run(s):
    case = s["case"]
    if own:
        import fp32_gemm_tile_amd as fg
        if case["op"] == "int4":
            if case["gated"]:
                return fg.gated_int4(s["x"], s["weights"][0], s["weights"][1], s["out"], group=case["group"])
            return fg.gemm_int4(s["x"], s["weights"][0], s["out"], group=case["group"])
        if case["op"] == "backward":
            fg.gated_backward(s["dh"], s["x"], s["gate"], s["up"], s["saved"], s["dx"], s["dgate"], s["dup"], out=s["h"], beta=case["beta"],
                              activation=case["act"], workspace=s["workspace"])
            return {n: s[n] for n in ("dx", "dgate", "dup", "h")}
        fg.gated(s["x"], s["gate"], s["up"], s["h"], activation=case["act"], saved=s["saved"] or None, workspace=s["workspace"])
        return (s["h"],) + s["saved"]
    x, dt = s["x"].float(), s["x"].dtype
    if case["op"] == "int4":
        y = [x @ plain_weights(*w, case["K"], case["group"]).t() for w in s["weights"]]
        return (plain_act(y[0], "silu")[0] * y[1] if case["gated"] else y[0]).to(dt)
    gate, up = s["gate"].float(), s["up"].float()
    if case["op"] == "backward":
        g, u = plain_saved(s)
        dh = s["dh"].float()
        a, slope = plain_act(g, case["act"])
        dg, du = dh * u * slope, dh * a
        dgate, dup = dg.t() @ x, du.t() @ x
        if case["beta"]:
            dgate, dup = dgate + case["beta"] * s["dgate"].float(), dup + case["beta"] * s["dup"].float()
        s["dgate"], s["dup"] = dgate.to(dt), dup.to(dt)
        return {"dx": (dg @ gate + du @ up).to(dt), "dgate": s["dgate"], "dup": s["dup"], "h": (a * u).to(dt)}
    g, u = x @ gate.t(), x @ up.t()
    h = (plain_act(g, case["act"])[0] * u).to(dt)
    if case["save"] == "none":
        return (h,)
    if case["save"] == "same":
        return h, g.to(dt), u.to(dt)
    return (h,) + plain_codes(g) + plain_codes(u)


def work(case):
    size = {"f32": 4, "bf16": 2}
    e = size[case["type"]]
    if case["op"] == "int4":
        T, N, K = case["T"], case["N"], case["K"]
        n = 2 if case["gated"] else 1
        groups = cdiv(K, case["group"])
        return {"bytes": n * N * (cdiv(K, 2) + groups * (size[case["scales"]] + case["zeros"])) + e * T * (N + K), "flops": 2.0 * n * T * N * K}
    T, H, I = case["T"], case["H"], case["I"]
    saved = {"none": 0.0, "same": 2.0 * e, "e4m3": 2 * (1 + 4 / BLOCK)}[case["save"]] * T * I
    if case["op"] == "backward":
        return {"bytes": e * (2 * T * I + 2 * T * H + 4 * I * H + (2 * I * H if case["beta"] else 0)) + saved, "flops": 8.0 * T * H * I}
    return {"bytes": e * (T * H + 2 * I * H + T * I) + saved, "flops": 4.0 * T * H * I}


# ---- the definitions in 64 bits --------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    x = s["x"].double()

    def times(a, b):
        return torch.mm(a.contiguous(), b.contiguous())

    def activated(v):
        return v * torch.sigmoid(v) if case.get("act", "silu") == "silu" else 0.5 * v * torch.special.erfc(-v / math.sqrt(2))

    if case["op"] == "int4":
        y = []
        c = torch.arange(case["K"], device="cuda")
        for codes, scales, zeros in s["weights"]:
            q = codes[:, c // 2].int()
            q = torch.where(c % 2 == 1, q // 16, q % 16).double()
            q -= 8 if zeros is None else zeros[c // case["group"]].t().double()
            y.append(times(x, (q * scales.double()[c // case["group"]].t()).t()))
        return activated(y[0]) * y[1] if case["gated"] else y[0]
    gate, up = s["gate"].double(), s["up"].double()
    if case["op"] == "backward":
        if case["save"] == "same":
            g, u = (v.double() for v in s["saved"])
        else:
            b = torch.arange(case["I"], device="cuda") // BLOCK
            g, u = (s["saved"][k].double() * s["saved"][k + 1].double()[b].t() for k in (0, 2))
        dh = s["dh"].double()
        if case["act"] == "silu":
            t = torch.sigmoid(g)
            slope = t + g * t * torch.sigmoid(-g)
        else:
            slope = 0.5 * torch.special.erfc(-g / math.sqrt(2)) + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
        h = activated(g) * u
        dg, du = dh * u * slope, dh * activated(g)
        out = {"dx": times(torch.cat((dg, du), 1), torch.cat((gate, up), 0)), "dgate": times(dg.t(), x), "dup": times(du.t(), x), "h": h}
        for n in ("dgate", "dup"):
            if case["beta"]:
                out[n] += case["beta"] * s[n].double()
        return out
    pre = [times(x, w.t()) for w in (gate, up)]
    out = [activated(pre[0]) * pre[1]]
    if case["save"] == "same":
        out += pre
    if case["save"] == "e4m3":
        grid = torch.arange(0, 127, dtype=torch.uint8).view(E4M3).double().cuda()   # the 127 finite magnitudes
        middle = (grid[1:] + grid[:-1]) / 2
        b = torch.arange(case["I"], device="cuda") // BLOCK
        for v in pre:
            most = torch.zeros(case["T"], int(b[-1]) + 1, dtype=torch.float64, device="cuda")
            most.scatter_reduce_(1, b.expand_as(v), v.abs(), "amax")
            sc = torch.clamp(most / TOP, min=SMALLEST).float().double()             # a scale is a float32
            q = v.abs() / sc[:, b]
            low = torch.bucketize(q, middle)                                        # ties end on the lower of two codes ...
            low += (low < 126) & (q == middle[low.clamp_max(125)]) & (low % 2 == 1)  # ... and go on where that is odd
            out += [grid[low] * torch.sign(v), sc.t()]
    return tuple(out)
