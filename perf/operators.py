"""What is measured of the operators around the decoupled sparse attention step.

Five operators that bring a transformer layer's hidden states to the queries, keys and values of
the attention and its output back:

* ``norm``      root-mean-square norm of rows, with the residual's addition;
* ``norm_i8``   the same with its output in 8-bit integers and one scale per row;
* ``quantize``  rows (a matrix, or the attention output's heads) in 8-bit integers, one scale per row;
* ``linear``    product of 8-bit integer matrices with scales per token and channel;
* ``rope``      rotary positions over time, height and width, with the query/key norm fused.

Where ``own`` is false ``run`` computes them in plain torch operations, else through
``block_sparse_cluster_b200``.  Quantised codes are integers with one right value each (the nearest
of the exact quotient, ties to even), so they are returned as the integers they are, with their
scales beside them, and both sides have to agree on every one.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6
THETA = 10000.0
MAX_ROW_ELEMENTS = 75600 * 5120        # the largest row operator's elements
MAX_PRODUCTS = 75600 * 5120 * 5120     # the largest matrix product's multiplications


def listed():
    return [
        # a handful of rows of a float32 modulation path: latency
        dict(name="norm_few", op="norm", rows=5, width=1536, dtype="f32", residual=False),
        # the norm before the attention of every token of a Wan2.1-14B latent, residual added on the way
        dict(name="norm_wan14b", op="norm", rows=75600, width=5120, dtype="bf16", residual=True),
        # rows of no round width, as after pruning, from a float32 residual stream
        dict(name="norm_i8_odd", op="norm_i8", rows=1003, width=1001, dtype="f32", residual=True),
        # the norm that feeds an 8-bit projection, Wan2.1-1.3B latent
        dict(name="norm_i8_wan13b", op="norm_i8", rows=32760, width=1536, dtype="bf16", residual=True),
        # the attention output of the small float32 workload
        dict(name="quantize_tiny", op="quantize", B=1, H=2, N=1024, d=64, dtype="f32"),
        # the attention output of a Wan2.1-14B latent, heads gathered into token rows
        dict(name="quantize_wan14b", op="quantize", B=1, H=40, N=75600, d=128, dtype="bf16"),
        # the time embedding's projection to six modulation vectors: one row
        dict(name="linear_token", op="linear", B=1, M=1, heads=0, N=30720, K=5120, dtype="f32", bias=True, packed=False),
        # ragged sizes: a text context of 777 tokens, a depth that is no multiple of a tile
        dict(name="linear_ragged", op="linear", B=1, M=777, heads=0, N=1537, K=1000, dtype="bf16", bias=True, packed=False),
        # the value projection of a Wan2.1-14B latent, written as the attention's heads
        dict(name="linear_wan14b", op="linear", B=1, M=75600, heads=40, N=5120, K=5120, dtype="bf16", bias=True, packed=False),
        # one row of latent tokens with explicit positions, pairs in halves
        dict(name="rope_row", op="rope", B=2, H=12, N=52, d=128, dt=16, dh=56, dw=56, T=0, Hs=0, Ws=0, pairing="halves",
             norm="head", dtype="f32", slots=1),
        # queries of the Wan2.1-1.3B latent and 120 tokens of text behind the grid, from a buffer that holds keys too
        dict(name="rope_wan13b", op="rope", B=1, H=12, N=32880, d=128, dt=44, dh=42, dw=42, T=21, Hs=30, Ws=52,
             pairing="adjacent", norm="full", dtype="bf16", slots=2),
        # queries of the Wan2.1-14B latent
        dict(name="rope_wan14b", op="rope", B=1, H=40, N=75600, d=128, dt=44, dh=42, dw=42, T=21, Hs=45, Ws=80,
             pairing="adjacent", norm="full", dtype="bf16", slots=1),
    ]


def _spread(rng, lo, hi):
    """A whole number in [lo, hi], even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm_i8", "quantize", "linear", "linear", "rope"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("norm", "norm_i8"):
        width = _spread(rng, 64, 8192)
        if rng.random() < 0.7:
            width = max(64, width // 16 * 16)
        rows = _spread(rng, 1, min(75600, MAX_ROW_ELEMENTS // (2 * width)))
        return dict(op=op, rows=rows, width=width, dtype=dtype, residual=rng.random() < 0.6)
    if op == "quantize":
        B, H, d = rng.choice([1, 1, 2, 3]), rng.randint(1, 40), rng.choice([64, 128])
        N = _spread(rng, 1, min(75600, MAX_ROW_ELEMENTS // (2 * B * H * d)))
        return dict(op=op, B=B, H=H, N=N, d=d, dtype=dtype)
    if op == "linear":
        K = _spread(rng, 64, 8192)
        if rng.random() < 0.8:
            K = max(64, K // 16 * 16)
        heads = rng.choice([0, 0, rng.randint(1, 40)])
        N = heads * rng.choice([64, 128]) if heads else _spread(rng, 64, 15360)
        B = rng.choice([1, 1, 2]) if heads else 1
        M = _spread(rng, 1, min(75600, MAX_PRODUCTS // (2 * B * N * K)))
        return dict(op=op, B=B, M=M, heads=heads, N=N, K=K, dtype=dtype, bias=rng.random() < 0.5, packed=rng.random() < 0.15)
    B, H, d = rng.choice([1, 1, 2, 3]), rng.randint(1, 40), rng.choice([64, 128])
    half = d // 2
    ht = rng.randint(1, half // 2)
    hh = (half - ht) // 2
    slots = rng.choice([1, 1, 2, 3])
    limit = min(75600, MAX_ROW_ELEMENTS // (2 * slots * B * H * d))
    if rng.random() < 0.5:
        T, Hs, Ws = _spread(rng, 1, 33), _spread(rng, 1, 48), _spread(rng, 1, 80)
        while T * Hs * Ws > limit:
            T, Hs, Ws = max(1, T // 2), max(1, Hs // 2), max(1, Ws // 2)
        N = min(limit, T * Hs * Ws + rng.choice([0, 0, rng.randint(0, 256)]))
    else:
        T = Hs = Ws = 0
        N = _spread(rng, 1, limit)
    return dict(op=op, B=B, H=H, N=N, d=d, dt=2 * ht, dh=2 * hh, dw=d - 2 * ht - 2 * hh, T=T, Hs=Hs, Ws=Ws,
                pairing=rng.choice(["adjacent", "halves"]), norm=rng.choice(["none", "head", "full"]), dtype=dtype, slots=slots)


def _row_sizes(c):
    return (c["rows"], c["width"]) if c["op"] in ("norm", "norm_i8") else (c["B"] * c["N"], c["H"] * c["d"])


def work(case):
    c = case
    size = 2 if c["dtype"] == "bf16" else 4
    if c["op"] == "linear":
        M = c["B"] * c["M"]
        return {"bytes": M * c["K"] + c["N"] * c["K"] + M * c["N"] * size + 4 * (M + c["N"] * (2 if c["bias"] else 1)),
                "flops": 2 * M * c["N"] * c["K"]}
    rows, width = _row_sizes(c)
    n = rows * width
    if c["op"] == "norm":
        return {"bytes": n * size * (4 if c["residual"] else 2) + width * size, "flops": 4 * n}
    if c["op"] == "norm_i8":
        return {"bytes": n * (size * (3 if c["residual"] else 1) + 1) + width * size + 4 * rows, "flops": 6 * n}
    if c["op"] == "quantize":
        return {"bytes": n * (size + 1) + 4 * rows, "flops": 3 * n}
    return {"bytes": 2 * n * size + (0 if c["T"] else 12 * c["N"]), "flops": (3 if c["norm"] == "none" else 6) * n}


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    dt = DTYPES[c["dtype"]]

    def normal(*shape, dtype=dt, mean=0.0, std=1.0):
        x = torch.empty(*shape, dtype=dtype, device="cuda")
        return x.normal_(mean, std, generator=g)

    s = {"case": c}
    if c["op"] in ("norm", "norm_i8"):
        rows, width = c["rows"], c["width"]
        s["x"] = normal(rows, width)
        # a few channels far above the others, as hidden states have them
        s["x"][:, torch.randint(0, width, (max(1, width // 256),), generator=g, device="cuda")] *= 12.0
        s["weight"] = normal(width, mean=1.0, std=0.1)
        s["residual"] = normal(rows, width, std=2.0) if c["residual"] else None
        s["sum"] = torch.empty_like(s["x"]) if c["residual"] else None
        if c["op"] == "norm":
            s["out"] = torch.empty_like(s["x"])
        else:
            # rows of codes start on 16 bytes, which the product reads fastest
            s["q"] = torch.empty(rows, -(-width // 16) * 16, dtype=torch.int8, device="cuda")[:, :width]
            s["scale"] = torch.empty(rows, dtype=torch.float32, device="cuda")
    elif c["op"] == "quantize":
        s["x"] = normal(c["B"], c["H"], c["N"], c["d"])
        s["q"] = torch.empty(c["B"] * c["N"], c["H"] * c["d"], dtype=torch.int8, device="cuda")
        s["scale"] = torch.empty(c["B"] * c["N"], dtype=torch.float32, device="cuda")
    elif c["op"] == "linear":
        M, N, K = c["B"] * c["M"], c["N"], c["K"]
        pitch = K if c["packed"] else -(-K // 16) * 16

        def codes(rows):
            x = torch.zeros(rows, pitch, dtype=torch.int8, device="cuda")
            for r in range(0, rows, 16384):
                part = normal(min(rows, r + 16384) - r, K, dtype=torch.float32, std=30.0)
                x[r:r + 16384, :K] = part.round_().clamp_(-127, 127).to(torch.int8)
            return x[:, :K]

        s["x"], s["w"] = codes(M), codes(N)
        s["x_scale"] = normal(M, dtype=torch.float32).mul_(0.3).exp_().mul_(0.02)
        s["w_scale"] = normal(N, dtype=torch.float32).mul_(0.3).exp_().mul_(5e-4)
        s["bias"] = normal(N, dtype=torch.float32, std=0.1) if c["bias"] else None
        heads = c["heads"]
        s["out"] = (torch.empty(c["B"], heads, c["M"], N // heads, dtype=dt, device="cuda") if heads
                    else torch.empty(M, N, dtype=dt, device="cuda"))
        s["ws"] = torch.zeros(256, dtype=torch.uint8, device="cuda")
    else:
        B, H, N, d, slots = c["B"], c["H"], c["N"], c["d"], c["slots"]
        # a projection's output [B, N, slots * H * d]; the last slot is what is rotated
        s["x"] = normal(B, N, slots, H, d)[:, :, slots - 1].permute(0, 2, 1, 3)
        s["weight"] = (None if c["norm"] == "none" else normal(d if c["norm"] == "head" else H * d, mean=1.0, std=0.1))
        s["positions"] = None
        if not c["T"]:
            top = torch.tensor([4096.0, 512.0, 512.0], device="cuda")
            s["positions"] = (torch.rand(N, 3, generator=g, device="cuda") * top).to(torch.int32)
        s["out"] = torch.empty(B, H, N, d, dtype=dt, device="cuda")
    return s


def _run_own(s):
    import block_sparse_cluster_b200 as da
    c = s["case"]
    if c["op"] == "norm":
        da.da_rms_norm(s["x"], s["weight"], s["out"], residual=s["residual"], sum_out=s["sum"], eps=EPS)
        return {"out": s["out"], "sum": s["sum"]}
    if c["op"] == "norm_i8":
        da.da_rms_norm_i8(s["x"], s["weight"], s["q"], s["scale"], residual=s["residual"], sum_out=s["sum"], eps=EPS)
        return {"q": s["q"], "scale": s["scale"], "sum": s["sum"]}
    if c["op"] == "quantize":
        da.da_quantize_i8(s["x"], s["q"], s["scale"])
        return {"q": s["q"], "scale": s["scale"]}
    if c["op"] == "linear":
        da.da_linear_i8(s["x"], s["x_scale"], s["w"], s["w_scale"], s["out"], s["ws"], bias=s["bias"])
        return {"out": s["out"]}
    rope = da.Rope(axes=(c["dt"], c["dh"], c["dw"]), grid=(c["T"], c["Hs"], c["Ws"]), theta=THETA, pairing=c["pairing"])
    da.da_rope(s["x"], s["out"], rope, positions=s["positions"], weight=s["weight"], eps=EPS)
    return {"out": s["out"]}


def _codes(v):
    """Nearest 8-bit codes of the rows of v (64 bits, so that values next to a border fall on its right side)."""
    top = v.abs().amax(-1, keepdim=True)
    return torch.where(top > 0, (v * 127 / top).round(), torch.zeros_like(v)).to(torch.int8), top


def _rope_angles(c, positions, device):
    """cos and sin of every token's angles [N, d / 2], and which tokens turn at all."""
    n = torch.arange(c["N"], device=device)
    turns = torch.ones_like(n, dtype=torch.bool)
    if positions is None:
        turns = n < c["T"] * c["Hs"] * c["Ws"]
        pos = torch.stack([n // (c["Hs"] * c["Ws"]), n // c["Ws"] % c["Hs"], n % c["Ws"]], -1)
    else:
        pos = positions
    widths = [c["dt"], c["dh"], c["dw"]]
    axis = torch.cat([torch.full((w // 2,), a, device=device) for a, w in enumerate(widths)])
    freq = torch.cat([THETA ** (-torch.arange(0, w, 2, device=device, dtype=torch.float64) / max(w, 1)) for w in widths])
    angle = pos[:, axis].double() * freq
    return angle.cos().float(), angle.sin().float(), turns[:, None]


def run(state):
    if own:
        return _run_own(state)
    s = state
    c = s["case"]
    if c["op"] == "norm":
        v = s["x"].float() if s["residual"] is None else s["x"].float() + s["residual"].float()
        out = v * (1.0 / torch.sqrt((v * v).mean(-1, keepdim=True) + EPS)) * s["weight"].float()
        return {"out": out.to(s["x"].dtype), "sum": None if s["residual"] is None else v.to(s["x"].dtype)}
    if c["op"] == "norm_i8":
        v = s["x"].double() if s["residual"] is None else s["x"].double() + s["residual"].double()
        q, top = _codes(v * s["weight"].double())
        scale = top / 127 / torch.sqrt((v * v).mean(-1, keepdim=True) + EPS)
        return {"q": q, "scale": scale[:, 0].float(), "sum": None if s["residual"] is None else v.to(s["x"].dtype)}
    if c["op"] == "quantize":
        q, top = _codes(s["x"].permute(0, 2, 1, 3).reshape(c["B"] * c["N"], -1).double())
        return {"q": q, "scale": (top[:, 0] / 127).float()}
    if c["op"] == "linear":
        out = (s["x"].float() @ s["w"].float().t()) * s["x_scale"][:, None] * s["w_scale"]
        if s["bias"] is not None:
            out = out + s["bias"]
        out = out.to(DTYPES[c["dtype"]])
        if c["heads"]:
            out = out.view(c["B"], c["M"], c["heads"], -1).permute(0, 2, 1, 3).contiguous()
        return {"out": out}
    x = s["x"].float()
    if c["norm"] == "head":
        x = x * (1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)) * s["weight"].float()
    elif c["norm"] == "full":
        x = x * (1.0 / torch.sqrt((x * x).mean((1, 3), keepdim=True) + EPS)) * s["weight"].float().view(1, c["H"], 1, c["d"])
    cos, sin, turns = _rope_angles(c, s["positions"], x.device)
    if c["pairing"] == "adjacent":
        a, b = x[..., 0::2], x[..., 1::2]
        out = torch.stack([torch.where(turns, a * cos - b * sin, a), torch.where(turns, a * sin + b * cos, b)], -1).flatten(-2)
    else:
        a, b = x.chunk(2, -1)
        out = torch.cat([torch.where(turns, a * cos - b * sin, a), torch.where(turns, a * sin + b * cos, b)], -1)
    return {"out": out.to(DTYPES[c["dtype"]]).contiguous()}


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    f64 = torch.float64
    if c["op"] in ("norm", "norm_i8"):
        v = s["x"].to(f64)
        if s["residual"] is not None:
            v += s["residual"].to(f64)
        total = None if s["residual"] is None else v.clone()
        size = torch.sqrt(torch.einsum("rw,rw->r", v, v) / c["width"] + EPS)
        v *= s["weight"].to(f64)
        if c["op"] == "norm":
            return {"out": v.div_(size[:, None]), "sum": total}
        return {"q": None, "scale": torch.linalg.vector_norm(v, ord=math.inf, dim=1) / (127 * size), "sum": total}
    if c["op"] == "quantize":
        top = torch.linalg.vector_norm(s["x"].to(f64), ord=math.inf, dim=(1, 3))
        return {"q": None, "scale": top.reshape(-1) / 127}
    if c["op"] == "linear":
        out = torch.einsum("mk,nk->mn", s["x"].to(f64), s["w"].to(f64))
        out *= torch.outer(s["x_scale"].to(f64), s["w_scale"].to(f64))
        if s["bias"] is not None:
            out += s["bias"].to(f64)
        if c["heads"]:
            out = torch.stack(out.view(c["B"], c["M"], c["N"]).split(c["N"] // c["heads"], dim=-1), 1)
        return {"out": out}
    B, H, N, d = c["B"], c["H"], c["N"], c["d"]
    x = s["x"].to(f64)
    if c["norm"] != "none":
        over = (3,) if c["norm"] == "head" else (1, 3)
        x = x / (x.pow(2).sum(over, keepdim=True) / (d if c["norm"] == "head" else H * d) + EPS) ** 0.5
        x *= s["weight"].to(f64).view(1, -1, 1, d)
    if s["positions"] is None:
        grid = torch.cartesian_prod(*[torch.arange(k, dtype=f64, device="cuda") for k in (c["T"], c["Hs"], c["Ws"])]).view(-1, 3)
        pos = torch.zeros(N, 3, dtype=f64, device="cuda")
        pos[:len(grid)] = grid[:N]     # tokens behind the grid stay where they are: position zero turns nothing
    else:
        pos = s["positions"].to(f64)
    angle = torch.empty(N, d // 2, dtype=f64, device="cuda")
    at = 0
    for a, w in enumerate((c["dt"], c["dh"], c["dw"])):
        for j in range(w // 2):
            angle[:, at] = pos[:, a] / THETA ** (2 * j / w)
            at += 1
    turn = torch.polar(torch.ones_like(angle), angle)
    if c["pairing"] == "adjacent":
        z = torch.view_as_complex(x.reshape(B, H, N, d // 2, 2).contiguous()) * turn
        return {"out": torch.view_as_real(z).reshape(B, H, N, d)}
    z = torch.complex(x[..., :d // 2].contiguous(), x[..., d // 2:].contiguous()) * turn
    return {"out": torch.cat([z.real, z.imag], -1)}
