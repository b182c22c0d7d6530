"""The RMS norm (with the residual's addition, an 8-bit output, its gradient) and the
product with 4-bit group-scaled weights: cases, inputs, plain forms and 64-bit values.

A packed weight is held in tiles of 16 output rows by 128 inputs, 1024 bytes each:
codes[n / 16][k / 128][byte], byte = 256 g + 16 r + 4 q + i for output row r of the
tile, q = k % 128 / 32, g = k % 32 / 8, i = k % 4; its low nibble is the code whose
k % 8 is below 4, its high nibble the one four further. scales (bf16) and zeros
(uint8) are [n / 16][k / group][n % 16]. A weight is (code - zero) * scale, zero = 8
where there are no zeros.
"""
import math

import torch

own = False

DEV = "cuda" if torch.cuda.is_available() else "cpu"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn, "i8": torch.int8}
EPS = 1e-5


def listed():
    return [
        # one decoded token: the key projection of a small model, latency counts
        {"name": "mv-k-1", "op": "matvec", "t": 1, "k": 4096, "n": "1024", "group": 128, "zeros": False, "x": "bf16", "y": "bf16"},
        # one decoded token on a wide gate projection: bound by the packed weight
        {"name": "mv-gate-1-e4m3", "op": "matvec", "t": 1, "k": 8192, "n": "28672", "group": 128, "zeros": False, "x": "e4m3", "y": "bf16"},
        # q, k and v of a few sequences decoded together, one launch
        {"name": "mv-qkv-4-i8", "op": "matvec", "t": 4, "k": 4096, "n": "4096,1024,1024", "group": 64, "zeros": True, "x": "i8", "y": "bf16"},
        # a batch of sixteen on a deep down projection, small groups
        {"name": "mv-down-16", "op": "matvec", "t": 16, "k": 28672, "n": "8192", "group": 32, "zeros": False, "x": "bf16", "y": "bf16"},
        # a large decode batch on a head of odd width, logits in float32
        {"name": "mv-head-64", "op": "matvec", "t": 64, "k": 5120, "n": "32003", "group": 64, "zeros": True, "x": "bf16", "y": "f32"},
        # the norm before q/k/v of one decoded token, its 8-bit rows for the product
        {"name": "norm-1-e4m3", "op": "norm", "t": 1, "d": 4096, "res": True, "q": "e4m3", "type": "bf16"},
        # a short prompt of odd length and width, float32 stream, int8 rows
        {"name": "norm-77-i8", "op": "norm", "t": 77, "d": 5003, "res": False, "q": "i8", "type": "f32"},
        # training's forward at full length, the residual's addition in it
        {"name": "norm-8192", "op": "norm", "t": 8192, "d": 4096, "res": True, "q": "none", "type": "bf16"},
        # training: the norm's gradient with the residual's gradient added, weight learnt too
        {"name": "normbwd-8192", "op": "normbwd", "t": 8192, "d": 4096, "res": True, "dw": True, "type": "bf16"},
        # a short odd batch whose weight is frozen
        {"name": "normbwd-333", "op": "normbwd", "t": 333, "d": 1001, "res": False, "dw": False, "type": "f32"},
        # a merged projection packed for serving, and read back
        {"name": "pack-4096", "op": "pack", "k": 4096, "n": "4096", "group": 128, "zeros": False, "type": "bf16"},
        # a float32 export of odd height, small groups with zero points
        {"name": "pack-1000-zeros", "op": "pack", "k": 5120, "n": "1000", "group": 32, "zeros": True, "type": "f32"},
    ]


def draw(rng):
    def log_int(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    op = rng.choice(["matvec", "matvec", "norm", "normbwd", "pack"])
    if op in ("matvec", "pack"):
        group = rng.choice([32, 64, 128])
        unit = max(64, group)
        most = 4096 * 4096 if op == "pack" else 8192 * 28672
        k = unit * log_int(1, 28672 // unit)
        n = log_int(1, min(28672, most // k))
        case = {"op": op, "k": k, "n": str(n), "group": group, "zeros": rng.random() < 0.5}
        if op == "pack":
            return dict(case, type=rng.choice(["bf16", "f32"]))
        if n > 64 and rng.random() < 0.25:
            case["n"] = "%d,%d" % (n - n // 3, n // 3)
        t = log_int(1, max(1, min(64, 16 * most // (k * n))))
        return dict(case, t=t, x=rng.choice(["bf16", "e4m3", "i8"]), y=rng.choice(["bf16", "f32"]))
    d = log_int(64, 28672)  # from one head's width to the widest MLP
    kind = rng.choice(["bf16", "f32"])
    t = log_int(1, min(8192, (8192 * 4096 if kind == "bf16" else 4096 * 4096) // d))
    if op == "norm":
        return {"op": op, "t": t, "d": d, "res": rng.random() < 0.6, "q": rng.choice(["none", "e4m3", "i8"]), "type": kind}
    return {"op": op, "t": t, "d": d, "res": rng.random() < 0.6, "dw": rng.random() < 0.6, "type": kind}


def _widths(case):
    return [int(n) for n in case["n"].split(",")]


def _tiles(k, n):
    return (n + 15) // 16, (k + 127) // 128


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(int(seed))

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=DEV)

    s = dict(case)
    if case["op"] == "matvec":
        k, g, x = case["k"], case["group"], normal(case["t"], case["k"])
        if case["x"] == "bf16":
            s["x"], s["x_scale"] = x.bfloat16(), None
        else:
            top = 448.0 if case["x"] == "e4m3" else 127.0
            s["x_scale"] = x.abs().amax(1) / top
            x = x / s["x_scale"][:, None]
            s["x"] = x.clamp(-448, 448).to(torch.float8_e4m3fn) if case["x"] == "e4m3" else x.round().to(torch.int8)
        s["w"] = []
        for n in _widths(case):
            nt, kt = _tiles(k, n)
            # codes as a quantizer leaves them: a bell over the sixteen levels
            low = (normal(nt, kt, 1024) * 2.4 + 8).round_().clamp_(0, 15).to(torch.uint8)
            high = (normal(nt, kt, 1024) * 2.4 + 8).round_().clamp_(0, 15).to(torch.uint8)
            codes = low | (high << 4)
            del low, high
            scales = (0.008 * (1 + 0.25 * normal(nt, k // g, 16).clamp_(-3, 3))).bfloat16()
            zeros = (normal(nt, k // g, 16) + 8).round_().clamp_(0, 15).to(torch.uint8) if case["zeros"] else None
            s["w"].append((codes, scales, zeros, n))
    elif case["op"] == "pack":
        s["w"] = (normal(_widths(case)[0], case["k"]) * 0.02).to(TYPES[case["type"]])
    else:
        t, d, kind = case["t"], case["d"], TYPES[case["type"]]
        loud = 1 + 9 * (torch.rand(d, generator=gen, device=DEV) < 0.01)  # a few loud channels
        s["x"] = (normal(t, d) * loud).to(kind)
        s["weight"] = (1 + 0.2 * normal(d)).to(kind)
        s["res"] = (normal(t, d) * loud).to(kind) if case["res"] else None
        if case["op"] == "normbwd":
            s["dy"] = (normal(t, d) * 0.01).to(kind)
            s["dh"] = (normal(t, d) * 0.01).to(kind) if case["res"] else None
            s["rstd"] = torch.rsqrt(s["x"].double().square().mean(1) + EPS).float()
    return s


def _unpack(codes, k, n):
    """Codes of a packed weight as float32 [n, k]."""
    nt, kt = codes.shape[:2]
    both = torch.stack([codes & 15, codes >> 4]).view(2, nt, kt, 4, 16, 4, 4)      # half, tile, chunk, g, r, q, i
    return both.permute(1, 4, 2, 5, 3, 0, 6).reshape(nt * 16, kt * 128)[:n, :k].float()


def _spread(v, n, group):
    """[tile, group, row] values as float32 [n, groups * group]."""
    return v.permute(0, 2, 1).reshape(-1, v.shape[1])[:n].float().repeat_interleave(group, 1)


def _matvec_plain(s):
    x = s["x"].float()
    if s["x_scale"] is not None:
        x = x * s["x_scale"][:, None]
    ys = []
    for codes, scales, zeros, n in s["w"]:
        w = _unpack(codes, s["k"], n) - (8.0 if zeros is None else _spread(zeros, n, s["group"]))
        w = w * _spread(scales, n, s["group"])
        ys.append((x @ w.t()).to(TYPES[s["y"]]))
    return {"y": ys}


def _norm_plain(s):
    kind = TYPES[s["type"]]
    h = s["x"] if s["res"] is None else (s["x"].float() + s["res"].float()).to(kind)
    hf = h.float()
    rstd = torch.rsqrt(hf.square().mean(1) + EPS)
    y = hf * rstd[:, None] * s["weight"].float()
    out = {} if s["res"] is None else {"h": h}
    if s["q"] == "none":
        return dict(out, y=y.to(kind), rstd=rstd)
    scale = y.abs().amax(1) / (448.0 if s["q"] == "e4m3" else 127.0)
    v = torch.where(scale[:, None] > 0, y / scale[:, None], torch.zeros_like(y))
    q = v.clamp(-448, 448).to(torch.float8_e4m3fn) if s["q"] == "e4m3" else v.round().clamp(-127, 127).to(torch.int8)
    return dict(out, scale=scale, q=_levels(q))


def _levels(q):
    """The levels that 8-bit rows hold, as numbers (a value is its level times the row's scale)."""
    return q if q.is_floating_point() else q.bfloat16()


def _normbwd_plain(s):
    kind = TYPES[s["type"]]
    h, dy, rstd = s["x"].float(), s["dy"].float(), s["rstd"][:, None]
    g = dy * s["weight"].float()
    dx = rstd * (g - h * rstd * rstd * (g * h).mean(1, keepdim=True))
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    out = {"dx": dx.to(kind)}
    if s["dw"]:
        out["dw"] = (dy * h * rstd).sum(0).to(kind)
    return out


def _pack_plain(s):
    n, k, group = s["w"].shape[0], s["k"], s["group"]
    w = s["w"].float().view(n, k // group, group)
    if s["zeros"]:
        lo, hi = w.amin(2).clamp(max=0), w.amax(2).clamp(min=0)
        scale = ((hi - lo) / 15).bfloat16()
        sf = scale.float()
        zero = torch.where(sf > 0, -lo / sf, torch.zeros_like(sf)).round().clamp(0, 15)
    else:
        scale = (w.abs().amax(2) / 7).bfloat16()
        sf = scale.float()
        zero = torch.full_like(sf, 8)
    c = torch.where(sf[..., None] > 0, w / sf[..., None], torch.zeros_like(w)).round()
    c = (c + zero[..., None]).clamp(0, 15)
    nt, kt = _tiles(k, n)
    grid = torch.zeros(nt * 16, kt * 128, dtype=torch.uint8, device=c.device)
    grid[:n, :k] = c.view(n, k).to(torch.uint8)
    both = grid.view(nt, 16, kt, 4, 4, 2, 4).permute(5, 0, 2, 4, 1, 3, 6).reshape(2, nt, kt, 1024)
    codes = both[0] | (both[1] << 4)
    back = (_unpack(codes, k, n).view(n, k // group, group) - zero[..., None]) * sf[..., None]
    return {"w": back.view(n, k).bfloat16()}


def run(s):
    if own:
        import qlora_linear_amd as q
        if s["op"] == "matvec":
            kind = TYPES[s["y"]]
            if len(s["w"]) == 1:
                codes, scales, zeros, n = s["w"][0]
                return {"y": [q.w4_matvec(s["x"], codes, scales, zeros, d_out=n, x_scale=s["x_scale"], dtype=kind)]}
            codes, scales, zeros, ns = zip(*s["w"])
            return {"y": q.w4_matvec_multi(s["x"], codes, scales, zeros if s["zeros"] else None, d_out=ns,
                                           x_scale=s["x_scale"], dtype=kind)}
        if s["op"] == "norm":
            if s["q"] == "none":
                y, h, rstd = q.rmsnorm_fwd(s["x"], s["weight"], EPS, residual=s["res"])
                out = {"y": y, "rstd": rstd}
            else:
                rows, scale, h = q.rmsnorm_fwd_quant(s["x"], s["weight"], EPS, residual=s["res"], qdtype=TYPES[s["q"]])
                out = {"q": _levels(rows), "scale": scale}
            return out if s["res"] is None else dict(out, h=h)
        if s["op"] == "normbwd":
            dx, dw = q.rmsnorm_bwd(s["dy"], s["x"], s["weight"], s["rstd"], dh=s["dh"], need_dw=s["dw"])
            return {"dx": dx, "dw": dw} if s["dw"] else {"dx": dx}
        packed = q.w4_quantize(s["w"], group=s["group"], zero_points=s["zeros"])
        return {"w": q.w4_dequantize(*packed, d_out=s["w"].shape[0], d_in=s["k"])}
    return {"matvec": _matvec_plain, "norm": _norm_plain, "normbwd": _normbwd_plain, "pack": _pack_plain}[s["op"]](s)


def work(case):
    if case["op"] in ("matvec", "pack"):
        k, g = case["k"], case["group"]
        packed = sum(n * k / 2 + n * k / g * (3 if case["zeros"] else 2) for n in _widths(case))
        if case["op"] == "pack":  # read, packed, read back, written
            n = _widths(case)[0]
            return {"bytes": n * k * ((2 if case["type"] == "bf16" else 4) + 2) + 2 * packed, "flops": 4.0 * n * k}
        t, n = case["t"], sum(_widths(case))
        x = t * k * 2 if case["x"] == "bf16" else t * (k + 4)
        return {"bytes": packed + x + t * n * (2 if case["y"] == "bf16" else 4), "flops": 2.0 * t * k * n}
    e = 2 if case["type"] == "bf16" else 4
    t, d = case["t"], case["d"]
    if case["op"] == "norm":
        out = t * d * e + t * 4 if case["q"] == "none" else t * d + t * 4
        return {"bytes": t * d * e * (3 if case["res"] else 1) + out + d * e, "flops": 6.0 * t * d}
    return {"bytes": t * d * e * (4 if case["res"] else 3) + t * 4 + d * e * (2 if case["dw"] else 1),
            "flops": 10.0 * t * d}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "matvec":
        k, g, ys = case["k"], case["group"], []
        x = s["x"].double() if s["x_scale"] is None else s["x"].double() * s["x_scale"].double()[:, None]
        x = torch.nn.functional.pad(x, (0, -k % 128))
        for codes, scales, zeros, n in s["w"]:
            y = torch.zeros(codes.shape[0] * 16, case["t"], dtype=torch.float64, device=x.device)
            chunks = codes.view(codes.shape[0], codes.shape[1], 4, 16, 4, 4)        # tile, chunk, g, r, q, i
            for q in range(4):
                for half in range(2):
                    for c0 in range(4):  # one group of eight columns at a time, four of its columns
                        at = torch.arange(codes.shape[1], device=x.device)[:, None] * 128 + 32 * q + 8 * c0 + 4 * half
                        at = (at + torch.arange(4, device=x.device)).reshape(-1)
                        v = (chunks[:, :, c0, :, q, :] >> (4 * half)) & 15          # tile, chunk, r, i
                        v = v.permute(0, 2, 1, 3).reshape(-1, at.numel()).double()
                        kin = at < k
                        gi = at[kin] // g
                        z = 8.0 if zeros is None else zeros[:, gi].double().transpose(1, 2).reshape(-1, gi.numel())
                        v = (v[:, kin] - z) * scales[:, gi].double().transpose(1, 2).reshape(-1, gi.numel())
                        y += v @ x[:, at[kin]].t()
            ys.append(y[:n].t().contiguous())
        return {"y": ys}
    if case["op"] == "pack":
        k, g = case["k"], case["group"]
        w = s["w"].double().unflatten(1, (k // g, g))
        lo, hi = w.min(2, keepdim=True).values, w.max(2, keepdim=True).values
        if case["zeros"]:
            lo, hi = lo.clamp(max=0.0), hi.clamp(min=0.0)
            step = ((hi - lo).float().double() / 15).float().bfloat16().double()
            zero = torch.nan_to_num((-lo / step).float(), 0.0).round().clamp(0, 15).double()
        else:
            step = (torch.maximum(-lo, hi) / 7).float().bfloat16().double()
            zero = torch.full_like(step, 8.0)
        level = (torch.nan_to_num((w / step).float(), 0.0).round().double() + zero).clamp(0, 15)
        return {"w": ((level - zero) * step).flatten(1)}
    kind = TYPES[case["type"]]
    if case["op"] == "norm":
        h = s["x"].double() if s["res"] is None else s["x"].double() + s["res"].double()
        h = h.to(kind).double()
        rstd = 1.0 / ((h * h).sum(1) / case["d"] + EPS).sqrt()
        y = s["weight"].double() * (h * rstd.unsqueeze(1))
        out = {} if s["res"] is None else {"h": h}
        if case["q"] == "none":
            return dict(out, y=y, rstd=rstd)
        scale = y.abs().max(1).values / (448.0 if case["q"] == "e4m3" else 127.0)
        v = torch.nan_to_num(y / scale.unsqueeze(1), 0.0)
        if case["q"] == "i8":
            v = v.round()
        else:  # three bits after the leading one, steps of 2^-9 below 2^-6
            e = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6)))
            step = torch.exp2(e - 3)
            v = (v / step).round() * step
        return dict(out, scale=scale, q=v)
    h, dy, r = s["x"].double(), s["dy"].double(), s["rstd"].double().unsqueeze(1)
    g = s["weight"].double() * dy
    n = h * r
    dx = r * (g - n * (g * n).sum(1, keepdim=True) / case["d"])
    if s["dh"] is not None:
        dx = dx + s["dh"].double()
    return {"dx": dx, "dw": (n * dy).sum(0)} if case["dw"] else {"dx": dx}
