"""Cases of the operators around the 8-bit-state Muon step, their plain forms, and the calls a user makes.

Four operators, each on a stack of `count` matrices of `rows` x `cols`:

  orthogonalize  O = NS_k(X): Frobenius normalisation, k Newton-Schulz iterations, one coefficient triple each
  state          an 8-bit optimizer state written (quantised) and read back
  momentum       momentum lerp and Nesterov blend on an 8-bit state, with the norm of the result
  step           the Muon step on an 8-bit state: momentum, orthogonalisation, parameter write

A state holds one code (int8 or e4m3) a value and one fp32 scale for each 128 columns of a row.
"""
import math

import torch

own = False

BLOCK = 128
EPS = 1e-7
QUINTIC = (3.4445, -4.7750, 2.0315)   # steep: pulls small singular values up
SETTLE = (15 / 8, -10 / 8, 3 / 8)     # converges to one: settles what the steep iterations reached
TOP = {"int8": 127.0, "e4m3": 448.0}  # largest code
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------------------------------ cases

def _ortho(name, count, rows, cols, dtype="bf16", layout="plain", data="rows", steep=5, settle=0):
    return {"name": name, "op": "orthogonalize", "count": count, "rows": rows, "cols": cols, "dtype": dtype,
            "layout": layout, "data": data, "steep": steep, "settle": settle}


def _state(name, op, count, rows, cols, dtype="bf16", fmt="int8", stochastic=False, data="rows", nesterov=True):
    return {"name": name, "op": op, "count": count, "rows": rows, "cols": cols, "dtype": dtype, "fmt": fmt,
            "stochastic": stochastic, "data": data, "nesterov": nesterov}


def listed():
    return [
        # the query heads of one 768-wide layer, each head orthogonalised by itself: a call that latency bounds
        _ortho("ortho heads 12x64x768", 12, 64, 768, data="heavy"),
        # every head of 24 layers of a 1536-wide model, as column slices of the fused weights
        _ortho("ortho heads 288x1536x128 cols", 288, 1536, 128, layout="columns"),
        # odd sizes, fp32 momenta stored transposed
        _ortho("ortho 7x331x1003 fp32 transposed", 7, 331, 1003, dtype="fp32", layout="transposed", steep=3, settle=2),
        # the attention projections of a 12-layer 768-wide model
        _ortho("ortho 48x768x768", 48, 768, 768, data="heavy", steep=3, settle=2),
        # wide projections of a 1536-wide model, the largest
        _ortho("ortho 12x1536x6144", 12, 1536, 6144),
        # one state of one small matrix: a call that latency bounds
        _state("state 1x768x768 int8", "state", 1, 768, 768),
        # the states of a model's square projections, heavy tails, unbiased rounding
        _state("state 96x1536x1536 e4m3 stochastic", "state", 96, 1536, 1536, fmt="e4m3", stochastic=True, data="heavy"),
        # momentum of one matrix
        _state("momentum 1x768x768 int8", "momentum", 1, 768, 768),
        # rows that end inside a block, fp32 gradients
        _state("momentum 9x517x1100 fp32 e4m3", "momentum", 9, 517, 1100, dtype="fp32", fmt="e4m3", nesterov=False),
        # momentum of a model's wide projections
        _state("momentum 24x1536x6144 int8 stochastic", "momentum", 24, 1536, 6144, stochastic=True),
        # a step of a small model's tall projections
        _state("step 4x2048x512 int8", "step", 4, 2048, 512),
        # a step of the square projections of a 1536-wide model
        _state("step 24x1536x1536 e4m3 stochastic", "step", 24, 1536, 1536, fmt="e4m3", stochastic=True, data="heavy"),
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["orthogonalize", "orthogonalize", "state", "momentum", "step"])
    data = rng.choice(["rows", "heavy"])
    if op in ("orthogonalize", "step"):
        rows, cols = spread(1, 3000), spread(1, 6144)
        if rng.random() < 0.5:
            rows, cols = cols, rows
        m, n = min(rows, cols), max(rows, cols)
        most = min(512, max(1, int(2.0e11 / (3 * m * m * n + m ** 3 + 4e4))), max(1, 100_000_000 // (rows * cols)))
        count = spread(1, most)
        if op == "orthogonalize":
            return {"op": op, "count": count, "rows": rows, "cols": cols, "dtype": rng.choice(["bf16", "bf16", "fp16", "fp32"]),
                    "layout": rng.choice(["plain", "columns", "transposed"]), "data": data, "steep": rng.randint(2, 5),
                    "settle": rng.randint(0, 2)}
    else:
        rows, cols = spread(1, 8192), spread(1, 8192)
        count = spread(1, max(1, min(256, 200_000_000 // (rows * cols))))
    return {"op": op, "count": count, "rows": rows, "cols": cols, "dtype": "bf16" if op == "step" else rng.choice(["bf16", "fp32"]),
            "fmt": rng.choice(["int8", "e4m3"]), "stochastic": rng.random() < 0.5, "data": data,
            "nesterov": rng.random() < 0.7}


def work(case):
    e, r, c = case["count"], case["rows"], case["cols"]
    size = e * r * c
    x = DTYPES[case["dtype"]].itemsize
    m, n = min(r, c), max(r, c)
    code = size + 4 * e * r * -(-c // BLOCK)
    products = e * (3.0 * m * m * n + float(m) ** 3)   # X X' and A A are symmetric: half of each
    if case["op"] == "orthogonalize":
        return {"bytes": size * (x + 2), "flops": (case["steep"] + case["settle"]) * products}
    if case["op"] == "state":
        return {"bytes": size * x + code + code + size * 2, "flops": 4.0 * size}
    if case["op"] == "momentum":  # the state is read, written, and read back into bf16
        return {"bytes": size * x + 3 * code + size * x + size * 2, "flops": 10.0 * size}
    return {"bytes": size * x * 3 + 3 * code + size * 2, "flops": 5 * products}


# ------------------------------------------------------------------------------------------ inputs

def _values(case, gen, scale=1.0):
    """Gradients or momenta: rows of different size, or entries of which one in a hundred is a hundred times as large."""
    shape = (case["count"], case["rows"], case["cols"])
    x = torch.randn(shape, generator=gen, device="cuda")
    if case["data"] == "rows":
        x *= 10.0 ** (-4 + 2 * torch.rand(shape[:2] + (1,), generator=gen, device="cuda"))
    else:
        x *= torch.where(torch.rand(shape, generator=gen, device="cuda") < 0.01, 0.1, 1e-3)
    return x * scale


def _laid_out(x, layout):
    """The stack as a user's program holds it: matrices back to back, column slices of one wide matrix, or transposed."""
    if layout == "columns":
        return x.transpose(0, 1).contiguous().transpose(0, 1)
    if layout == "transposed":
        return x.mT.contiguous().mT
    return x


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dtype = DTYPES[case["dtype"]]
    s = {"case": dict(case)}
    shape = (case["count"], case["rows"], case["cols"])
    if case["op"] == "orthogonalize":
        s["X"] = _laid_out(_values(case, gen).to(dtype), case["layout"])
        s["O"] = _laid_out(torch.empty(shape, dtype=torch.bfloat16, device="cuda"), case["layout"])
        s["abc"] = [QUINTIC] * case["steep"] + [SETTLE] * case["settle"]
    elif case["op"] == "state":
        s["X"] = _values(case, gen).to(dtype)
    else:
        s["G"] = _values(case, gen).to(dtype)
        s["U"] = torch.empty(shape, dtype=dtype, device="cuda")
        if case["op"] == "step":
            s["W"] = (0.02 * torch.randn(shape, generator=gen, device="cuda")).to(dtype)
        # the state as an earlier step left it
        s["codes"], s["scales"] = _write(_values(case, gen, 0.3), case["fmt"], None)
    s["seed"] = int(seed) * 7919 % (1 << 31) if case.get("stochastic") else None
    s["back"] = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    if own:
        from muon_newton_schulz_07_b200.optimizer import MuonStep, QuantizedState

        if case["op"] != "state":
            s["muon"] = MuonStep([shape], dtype=torch.bfloat16 if case["op"] == "orthogonalize" else dtype, mode="half")
        if case["op"] != "orthogonalize":
            s["state"] = QuantizedState([shape], fmt=case["fmt"], device="cuda")
            if "codes" in s:
                s["state"].codes[0].copy_(s.pop("codes"))
                s["state"].scales[0].copy_(s.pop("scales"))
    return s


HYPER = {"lr": 0.02, "beta": 0.95, "weight_decay": 0.1}


# ------------------------------------------------------------------------------------------ plain forms

def _plain_orthogonalize(x, abc):
    x = x.float()
    tall = x.shape[-2] > x.shape[-1]
    if tall:
        x = x.mT
    x = x / (x.square().sum((-2, -1), keepdim=True).sqrt() + EPS)
    for a, b, c in abc:
        g = x @ x.mT
        x = a * x + (b * g + c * (g @ g)) @ x
    return x.mT if tall else x


def _mixed(h):
    """32-bit mixing by xor-shifts and products, in 64-bit integers (products split so that nothing overflows)."""
    for shift, factor in ((16, 0x6A09E667), (15, 0xBB67AE85), (16, None)):
        h = h ^ (h >> shift)
        if factor is not None:
            h = (h * (factor & 0xFFFF) + (((h * (factor >> 16)) & 0xFFFF) << 16)) & 0xFFFFFFFF
    return h


def _random_bits(shape, seed, device):
    """16 random bits for each value: of the seed, the matrix and the value's place in it (two places share a 32-bit number)."""
    e, r, c = shape
    place = torch.arange(r * c, device=device, dtype=torch.int64)
    matrix = torch.arange(e, device=device, dtype=torch.int64)
    key = _mixed(_mixed(torch.full_like(matrix, seed & 0xFFFFFFFF)) ^ (matrix & 0xFFFFFFFF))
    pair = _mixed(((place >> 1)[None] + key[:, None]) & 0xFFFFFFFF)
    return ((pair >> (16 * (place & 1))) & 0xFFFF).view(e, r, c)


def _blocks(x):
    """(count, rows, blocks, 128), the last block of a row padded with zeros."""
    e, r, c = x.shape
    pad = -c % BLOCK
    if pad:
        x = torch.cat([x, x.new_zeros(e, r, pad)], -1)
    return x.view(e, r, -1, BLOCK)


def _write(x, fmt, seed):
    """Codes (as the type holds them) and scales of a stack."""
    x = x.float()
    e, r, c = x.shape
    b = _blocks(x)
    amax = b.abs().amax(-1)
    full = torch.full_like(amax, TOP[fmt])
    fine = torch.isfinite(amax) & (amax >= 2.0 ** -100)
    inv = torch.where(fine, full / amax, torch.zeros_like(amax))
    scale = torch.where(fine, amax / full, torch.where(torch.isfinite(amax), torch.zeros_like(amax), torch.full_like(amax, math.nan)))
    y = (b * inv[..., None]).view(e, r, -1)[..., :c]
    y = torch.where(torch.isfinite(y), y, torch.zeros_like(y))
    u = None if seed is None else _random_bits((e, r, c), seed, x.device)
    if fmt == "int8":
        q = torch.round(y) if u is None else torch.floor(y + u.float() * 2.0 ** -16)
        return q.clamp(-127, 127).to(torch.int8), scale
    if u is not None:
        size = y.abs()
        bits = size.contiguous().view(torch.int32).to(torch.int64)
        normal = ((bits + (u << 4)) & ~0xFFFFF).to(torch.int32).view(torch.float32)
        small = torch.floor(size * 512 + u.float() * 2.0 ** -16) * 2.0 ** -9
        size = torch.where(size >= 2.0 ** -6, normal, small).clamp(max=448.0)
        y = torch.copysign(size, y)
    return y.to(torch.float8_e4m3fn), scale


def _read(codes, scales):
    c = codes.shape[-1]
    return codes.float() * scales.repeat_interleave(BLOCK, -1)[..., :c]


def _plain_momentum(s):
    case = s["case"]
    beta = float(torch.tensor(HYPER["beta"], dtype=torch.float32))
    g = s["G"].float() * (1 - beta)
    m = _read(s["codes"], s["scales"]) * beta + g
    u = g + m * beta if case["nesterov"] else m
    s["codes"], s["scales"] = _write(m, case["fmt"], s["seed"])
    return u


# ------------------------------------------------------------------------------------------ one pass

def run(state):
    s, case = state, state["case"]
    if case["op"] == "orthogonalize":
        if own:
            s["muon"].orthogonalize([s["X"]], [s["O"]], eps=EPS, abc=s["abc"])
            return {"O": s["O"]}
        return {"O": _plain_orthogonalize(s["X"], s["abc"]).to(torch.bfloat16)}
    if case["op"] == "state":
        if own:
            s["state"].write([s["X"]], seed=s["seed"])
            s["state"].read([s["back"]])
            return {"values": s["back"], "scales": s["state"].scales[0]}
        codes, scales = _write(s["X"], case["fmt"], s["seed"])
        return {"values": _read(codes, scales).to(torch.bfloat16), "scales": scales}
    if case["op"] == "momentum":
        if own:
            norms = s["muon"].momentum([s["G"]], s["state"], [s["U"]], beta=HYPER["beta"], nesterov=case["nesterov"], seed=s["seed"])
            s["state"].read([s["back"]])
            return {"U": s["U"], "norms": norms, "M": s["back"]}
        u = _plain_momentum(s)
        return {"U": u.to(s["G"].dtype), "norms": u.square().sum((-2, -1)).sqrt(), "M": _read(s["codes"], s["scales"]).to(torch.bfloat16)}
    if own:
        s["muon"](
            [s["W"]], [s["G"]], s["state"], lr=HYPER["lr"], beta=HYPER["beta"], weight_decay=HYPER["weight_decay"], eps=EPS,
            abc=QUINTIC, nesterov=case["nesterov"], ns_steps=5, seed=s["seed"])
        s["state"].read([s["back"]])
        return {"W": s["W"], "M": s["back"]}
    o = _plain_orthogonalize(_plain_momentum(s), [QUINTIC] * 5)
    scale = HYPER["lr"] * math.sqrt(max(1.0, case["rows"] / case["cols"]))
    w = s["W"].float() * (1 - HYPER["lr"] * HYPER["weight_decay"]) - scale * o
    s["W"].copy_(w)
    return {"W": s["W"], "M": _read(s["codes"], s["scales"]).to(torch.bfloat16)}


# ------------------------------------------------------------------------------------------ in 64 bits

def _exact_iterations(x, abc):
    flip = x.size(1) > x.size(2)
    y = x.transpose(1, 2) if flip else x
    size = torch.linalg.vector_norm(y, dim=(1, 2), keepdim=True)
    y = y / (size + EPS)
    one = torch.eye(y.size(1), dtype=torch.float64, device=y.device)
    for a, b, c in abc:
        gram = torch.bmm(y, y.transpose(1, 2))
        y = torch.bmm(torch.baddbmm(a * one + b * gram, gram, gram, alpha=c), y)
    return y.transpose(1, 2) if flip else y


def _exact_rounded(x, fmt, bits):
    """The values an 8-bit state stands for after x is written to it, and its scales."""
    count, rows, cols = x.shape
    values, scales = torch.zeros_like(x), []
    for at in range(0, cols, BLOCK):
        part = x[:, :, at:at + BLOCK]
        top = part.abs().max(dim=2, keepdim=True).values
        step = top / TOP[fmt]
        live = top >= 2.0 ** -100
        y = torch.where(live, part / torch.where(live, step, torch.ones_like(step)), torch.zeros_like(part))
        u = None if bits is None else bits[:, :, at:at + BLOCK]
        if fmt == "e4m3":  # spacing of the codes at y: three bits below the leading one, 2^-9 at the bottom
            spacing = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
        else:
            spacing = torch.ones_like(y)
        if u is None:
            q = torch.round(y / spacing) * spacing
        elif fmt == "int8":
            q = torch.floor(y + u.double() / 2 ** 16)
        else:
            q = torch.sign(y) * torch.floor(y.abs() / spacing + u.double() / 2 ** 16) * spacing
        values[:, :, at:at + BLOCK] = q.clamp(-TOP[fmt], TOP[fmt]) * torch.where(live, step, torch.zeros_like(step))
        scales.append(torch.where(live, step, torch.zeros_like(step)))
    return values, torch.cat(scales, 2)


def exact(case, seed):
    s = prepare({**case}, seed)
    if case["op"] == "orthogonalize":
        return {"O": _exact_iterations(s["X"].double(), s["abc"])}
    shape = (case["count"], case["rows"], case["cols"])
    bits = None if s["seed"] is None else _random_bits(shape, s["seed"], "cuda")
    if case["op"] == "state":
        values, scales = _exact_rounded(s["X"].double(), case["fmt"], bits)
        return {"values": values, "scales": scales}
    beta = float(torch.tensor(HYPER["beta"], dtype=torch.float32))
    held = torch.cat([s["codes"][..., at:at + BLOCK].to(torch.float32).double() * s["scales"][..., at // BLOCK, None].double()
                      for at in range(0, case["cols"], BLOCK)], -1)
    g = s["G"].double()
    m = beta * held + (1 - beta) * g
    u = (1 - beta) * g + beta * m if case["nesterov"] else m
    values, _ = _exact_rounded(m, case["fmt"], bits)
    if case["op"] == "momentum":
        return {"U": u, "norms": torch.linalg.vector_norm(u, dim=(1, 2)), "M": values}
    o = _exact_iterations(u, [QUINTIC] * 5)
    keep = 1 - HYPER["lr"] * HYPER["weight_decay"]
    return {"W": keep * s["W"].double() - HYPER["lr"] * max(1.0, case["rows"] / case["cols"]) ** 0.5 * o, "M": values}
