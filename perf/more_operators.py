"""A paged cache of keys and values in 4 bits: writing new tokens to it with the position
rotation on the way, reading rows back, and the attention over it. Cases, inputs, plain
forms and 64-bit values.

The cache of one layer is four tensors. For pages of S tokens, H heads of D values and
groups of G values (C = D / 32 chunks of a row):
  k_codes   uint8 [pages, H, S, D / 2]: byte g D / 8 + 4 c + b of a row holds the code of
            d = 32 c + 8 g + b in its low nibble and of d + 4 in its high one (g, b in 0 .. 3)
  v_codes   uint8 [pages, H, S / 4, 2 D]: byte r D / 8 + 4 c + i of four tokens holds, for
            token i of them, d = 32 c + 2 r (low nibble) and d + 1 (high), r in 0 .. 15
  k_scales, v_scales   bf16 [pages, H, D / G, S, 2]: a group's step s and least value lo
A value is lo + s code. Slot t of the cache is token t % S of page t / S.
"""
import math

import torch

own = False

DEV = "cuda" if torch.cuda.is_available() else "cpu"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _heads(n_q, n_kv, d, group, page):
    return {"n_q": n_q, "n_kv": n_kv, "d": d, "group": group, "page": page}


def listed():
    return [
        # one decoded token of a small model: latency counts
        dict({"name": "append-1", "op": "append", "t": 1, "rot": 128, "pairs": "half", "type": "bf16"}, **_heads(32, 8, 128, 128, 32)),
        # an odd decode batch, float32 rows, half of each head rotated, neighbours in pairs
        dict({"name": "append-77-f32", "op": "append", "t": 77, "rot": 32, "pairs": "next", "type": "f32"}, **_heads(12, 12, 64, 32, 64)),
        # a long prompt, keys and values shared by four query heads each
        dict({"name": "append-8192", "op": "append", "t": 8192, "rot": 128, "pairs": "half", "type": "bf16"}, **_heads(32, 8, 128, 64, 64)),
        # a prompt of odd length with as many key heads as query heads, small groups
        dict({"name": "append-2047-mha", "op": "append", "t": 2047, "rot": 128, "pairs": "half", "type": "bf16"}, **_heads(40, 40, 128, 32, 32)),
        # one decoded token after a short prompt: latency counts
        dict({"name": "decode-1-500", "op": "attend", "b": 1, "len": 500, "n0": 1, "n": 1, "window": 0, "pad": 0, "lse": False}, **_heads(32, 8, 128, 128, 32)),
        # one decoded token after a whole book, the sums wanted too
        dict({"name": "decode-1-131071", "op": "attend", "b": 1, "len": 131071, "n0": 1, "n": 1, "window": 0, "pad": 0, "lse": True}, **_heads(64, 8, 128, 64, 128)),
        # a server's decode batch of ragged lengths, its last places empty
        dict({"name": "decode-64-ragged", "op": "attend", "b": 64, "len": 16384, "n0": 1, "n": 1, "window": 0, "pad": 3, "lse": False}, **_heads(32, 8, 128, 128, 64)),
        # many short chats on a model whose query heads have a key head each
        dict({"name": "decode-96-mha", "op": "attend", "b": 96, "len": 1500, "n0": 1, "n": 1, "window": 0, "pad": 0, "lse": False}, **_heads(40, 40, 128, 32, 32)),
        # wide heads, only the last 4096 tokens seen
        dict({"name": "decode-24-window", "op": "attend", "b": 24, "len": 30001, "n0": 1, "n": 1, "window": 4096, "pad": 0, "lse": False}, **_heads(16, 8, 256, 64, 32)),
        # five guessed tokens a sequence checked at once
        dict({"name": "verify-16x5", "op": "attend", "b": 16, "len": 6000, "n0": 5, "n": 5, "window": 0, "pad": 0, "lse": False}, **_heads(64, 8, 128, 64, 32)),
        # a chunk of one prompt among decoding sequences
        dict({"name": "chunk-512-mixed", "op": "attend", "b": 17, "len": 16384, "n0": 512, "n": 1, "window": 0, "pad": 0, "lse": False}, **_heads(32, 8, 128, 128, 64)),
        # two whole prompts
        dict({"name": "prompt-2x2500", "op": "attend", "b": 2, "len": 2500, "n0": 2500, "n": 2500, "window": 0, "pad": 0, "lse": False}, **_heads(32, 4, 64, 64, 32)),
    ]


def draw(rng):
    def log_int(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    d = rng.choice([64, 128, 128, 256])
    group = rng.choice([g for g in (32, 64, 128) if g <= d])
    n_kv = rng.choice([1, 2, 4, 8, 8, 16, 40])
    n_q = n_kv * (rng.choice([1, 2, 3, 4, 5, 7, 8, 16]) if n_kv < 16 else 1)
    case = _heads(n_q, n_kv, d, group, rng.choice([32, 64, 96, 128, 256]))
    if rng.random() < 0.4:
        t = log_int(1, min(8192, (1 << 24) // (max(n_q, 4 * n_kv) * d)))
        return dict(case, op="append", t=t, rot=rng.choice([0, 16, d // 2, d, d]), pairs=rng.choice(["half", "half", "next"]),
                    type=rng.choice(["bf16", "bf16", "f32"]))
    kind = rng.choice(["decode", "decode", "verify", "chunk", "prompt"])
    case.update(op="attend", window=rng.choice([0, 0, 0, log_int(1, 8192)]), pad=0, lse=rng.random() < 0.3)
    most = (1 << 28) // (n_kv * d)          # keys of one pass
    if kind == "prompt":
        b = log_int(1, 4)
        n = log_int(9, min(2500, most, int(math.sqrt((1 << 32) / (b * n_q * d)))))
        return dict(case, b=b, len=n, n0=n, n=n)
    b = 1 + log_int(1, 16) if kind == "chunk" else log_int(1, 256)
    length = log_int(16, max(16, min(131072, most // b)))
    if kind == "chunk":
        n0 = max(1, min(length, log_int(9, 512), (1 << 33) // (n_q * d * length)))
        return dict(case, b=b, len=length, n0=n0, n=1)
    n = rng.randint(2, 8) if kind == "verify" else 1
    return dict(case, b=b, len=length, n0=n, n=n)


def _batch(case):
    """(tokens, keys) of each sequence: keys spread over (0, len], the new tokens among them;
    the last `pad` sequences have no keys."""
    n = [case["n0"]] + [case["n"]] * (case["b"] - 1)
    keys = [max(n[i], int(case["len"] * (1 - i * 0.6180339887498949 % 1))) for i in range(case["b"])]
    for i in range(case["b"] - case["pad"], case["b"]):
        keys[i] = 0
    return n, keys


def _empty_cache(case, pages):
    h, d, s, g = case["n_kv"], case["d"], case["page"], case["group"]

    def tensors(*codes):
        return [torch.zeros(pages, h, *codes, dtype=torch.uint8, device=DEV),
                torch.zeros(pages, h, d // g, s, 2, dtype=torch.bfloat16, device=DEV)]

    return (*tensors(s, d // 2), *tensors(s // 4, 2 * d))


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(int(seed))

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=DEV)

    s, d, page = dict(case), case["d"], case["page"]
    if case["op"] == "append":
        t, kind, far = case["t"], TYPES[case["type"]], 32768
        pages = 2 * ((t + page - 1) // page) + 1
        s["cache"] = _empty_cache(case, pages)
        loud = 1 + 5 * (torch.rand(case["n_kv"], d, generator=gen, device=DEV) < 0.03)  # a few loud channels
        s["q"] = normal(t, case["n_q"], d).to(kind)
        s["k"] = (normal(t, case["n_kv"], d) * loud).to(kind)
        s["v"] = normal(t, case["n_kv"], d).to(kind)
        # a decode batch has tokens anywhere, a prompt a run of positions and of slots in scattered pages
        order = torch.randperm(pages, generator=gen, device=DEV)
        at = torch.arange(t, device=DEV) if t > 256 else torch.randperm(pages * page, generator=gen, device=DEV)[:t]
        s["slots"] = order[at // page] * page + at % page
        first = torch.randint(0, far - t + 1, (1,), generator=gen, device=DEV)
        s["positions"] = first + torch.arange(t, device=DEV) if t > 256 else \
            torch.randint(0, far, (t,), generator=gen, device=DEV)
        s["cos"] = s["sin"] = None
        if case["rot"]:
            turn = 1e4 ** (-torch.arange(0, case["rot"], 2, device=DEV, dtype=torch.float64) / case["rot"])
            angle = torch.arange(far, device=DEV, dtype=torch.float64)[:, None] * turn
            s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
        return s
    n, keys = _batch(case)
    need = [(k + page - 1) // page for k in keys]
    pages = sum(need) + 2
    cache = _empty_cache(case, pages)
    for codes in cache[0], cache[2]:
        for i in range(0, pages, 256):  # as a quantizer leaves them: a bell over the sixteen levels
            part = codes[i:i + 256]
            part.copy_((normal(*part.shape) * 2.6 + 7.5).round_().clamp_(0, 15))
            part.add_((normal(*part.shape) * 2.6 + 7.5).round_().clamp_(0, 15).to(torch.uint8) << 4)
    for scales in cache[1], cache[3]:
        step = 0.3 * (1 + 0.2 * normal(*scales.shape[:-1]).clamp_(-3, 3))
        scales[..., 0] = step
        scales[..., 1] = step * (normal(*step.shape) * 0.7 - 7.5)
    s["cache"] = cache
    order = torch.randperm(pages, generator=gen, device=DEV).tolist()
    table = torch.zeros(len(keys), max(1, max(need)), dtype=torch.int32)
    for i, m in enumerate(need):
        table[i, :m] = torch.tensor([order.pop() for _ in range(m)], dtype=torch.int32)
    s["table"] = table.to(DEV)
    s["lens"] = torch.tensor(keys, dtype=torch.int32).to(DEV)
    cu = [0]
    for m in n:
        cu.append(cu[-1] + m)
    s["cu"] = None if case["n0"] == case["n"] == 1 else torch.tensor(cu, dtype=torch.int32).to(DEV)
    s["q"] = (normal(cu[-1], case["n_q"], d) * 2).bfloat16()
    s["host"] = (cu, keys)  # the batch as a serving loop knows it
    s["most"] = max(n)
    return s


def _key_codes(codes):
    """[.., D / 2] bytes of rows as [.., D] codes."""
    d = codes.shape[-1] * 2
    both = torch.stack([codes & 15, codes >> 4], -1).unflatten(-2, (4, d // 32, 4))     # g, c, b, half
    return both.movedim(-4, -3).movedim(-1, -2).reshape(*codes.shape[:-1], d)           # c, g, half, b


def _value_codes(codes):
    """[.., S / 4, 2 D] bytes of four tokens each as [.., S, D] codes."""
    d = codes.shape[-1] // 2
    both = torch.stack([codes & 15, codes >> 4], -1).unflatten(-2, (16, d // 32, 4))    # r, c, i, half
    both = both.movedim(-2, -4).movedim(-2, -3)                                         # i, c, r, half
    return both.reshape(*codes.shape[:-2], codes.shape[-2] * 4, d)


def _levels(codes, scales):
    """float32 values of [.., S, D] codes with [.., D / G, S, 2] scales."""
    per = scales.float().movedim(-3, -2).repeat_interleave(codes.shape[-1] // scales.shape[-3], -2)
    return codes.float() * per[..., 0] + per[..., 1]


def _rotated(s, x):
    """x with its first `rot` values of each head turned, in 64 bits (a product of the sum is
    exact there), rounded to float32 and then bf16."""
    rot = s["rot"]
    if not rot:
        return x.bfloat16()
    cos, sin = (s[n][s["positions"]].double()[:, None] for n in ("cos", "sin"))
    a, b = (x[..., :rot // 2], x[..., rot // 2:rot]) if s["pairs"] == "half" else (x[..., 0:rot:2], x[..., 1:rot:2])
    a, b = a.double(), b.double()
    a, b = a * cos - b * sin, a * sin + b * cos
    y = torch.cat([a, b], -1) if s["pairs"] == "half" else torch.stack([a, b], -1).flatten(-2)
    return torch.cat([y.float(), x[..., rot:].float()], -1).bfloat16()


def _quantized(x, group):
    """(codes [T, H, D], scales [T, H, D / G, 2]) of bf16 rows."""
    v = x.float().unflatten(-1, (-1, group))
    lo, hi = v.amin(-1), v.amax(-1)
    step = ((hi - lo) / 15).bfloat16()
    sf = step.double()[..., None]
    c = torch.where(sf > 0, (v - lo[..., None]).double() / sf, torch.zeros_like(sf)).round().clamp(0, 15)
    return c.to(torch.uint8).flatten(-2), torch.stack([step, lo.bfloat16()], -1)


def _append_plain(s):
    d, page, slots = s["d"], s["page"], s["slots"]
    k_codes, k_scales, v_codes, v_scales = s["cache"]
    at, tok = slots // page, slots % page
    kc, ks = _quantized(_rotated(s, s["k"]), s["group"])
    vc, vs = _quantized(s["v"].bfloat16(), s["group"])
    parts = kc.unflatten(-1, (d // 32, 4, 2, 4))                                        # c, g, half, b
    byte = parts[..., 0, :] | (parts[..., 1, :] << 4)
    k_codes[at, :, tok] = byte.movedim(-2, -3).flatten(-3)                              # g, c, b
    parts = vc.unflatten(-1, (d // 32, 16, 2))                                          # c, r, half
    byte = (parts[..., 0] | (parts[..., 1] << 4)).movedim(-1, -2)                       # r, c
    v_codes.unflatten(-1, (16, d // 32, 4))[at, :, tok // 4, :, :, tok % 4] = byte
    k_scales[at, :, :, tok] = ks
    v_scales[at, :, :, tok] = vs
    out = {"q": _rotated(s, s["q"])}
    quad = v_codes.unflatten(-1, (16, d // 32, 4))[at, :, tok // 4, :, :, tok % 4]      # r, c
    vc = torch.stack([quad & 15, quad >> 4], -1).movedim(-3, -2).flatten(-3)
    for name, codes, scales in (("k", _key_codes(k_codes[at, :, tok]), k_scales), ("v", vc, v_scales)):
        per = scales[at, :, :, tok].float().repeat_interleave(s["group"], -2)
        out[name] = (codes.float() * per[..., 0] + per[..., 1]).bfloat16()
    return out


def _attend_plain(s):
    k_codes, k_scales, v_codes, v_scales = s["cache"]
    (cu, keys), h, d, page = s["host"], s["n_kv"], s["d"], s["page"]
    y = torch.zeros_like(s["q"])
    lse = torch.full(s["q"].shape[:2], -math.inf, device=y.device)
    for i, length in enumerate(keys):
        n = cu[i + 1] - cu[i]
        first = max(0, length - n + 1 - s["window"]) if s["window"] else 0
        p0 = first // page  # pages no token sees are not read
        if length == 0:
            continue
        pages = s["table"][i, p0:(length + page - 1) // page].long()
        k = _levels(_key_codes(k_codes[pages]), k_scales[pages]).transpose(0, 1).reshape(h, -1, d)[:, :length - p0 * page]
        v = _levels(_value_codes(v_codes[pages]), v_scales[pages]).transpose(0, 1).reshape(h, -1, d)[:, :length - p0 * page]
        place = torch.arange(length - n, length, device=y.device)[:, None]
        key = torch.arange(p0 * page, length, device=y.device)[None]
        seen = key <= place
        if s["window"]:
            seen &= key > place - s["window"]
        q = s["q"][cu[i]:cu[i + 1]].float().unflatten(1, (h, -1)).permute(1, 2, 0, 3).reshape(h, -1, d)
        score = (q @ k.transpose(1, 2) * d ** -0.5).unflatten(1, (-1, n))               # h, head of it, token, key
        score = score.masked_fill(~seen, -math.inf)
        top = score.amax(-1, keepdim=True)
        p = (score - top).exp()
        total = p.sum(-1, keepdim=True)
        o = (p / total).flatten(1, 2) @ v
        y[cu[i]:cu[i + 1]] = o.unflatten(1, (-1, n)).permute(2, 0, 1, 3).reshape(n, -1, d).bfloat16()
        lse[cu[i]:cu[i + 1]] = (top + total.log())[..., 0].permute(2, 0, 1).reshape(n, -1)
    return {"y": y, "lse": lse} if s["lse"] else {"y": y}


def run(s):
    if own:
        import qlora_linear_amd as q
        if s["op"] == "append":
            turned = q.kv4_append(s["q"], s["k"], s["v"], s["cache"], s["slots"], cos=s["cos"], sin=s["sin"],
                                  positions=s["positions"] if s["rot"] else None, interleaved=s["pairs"] == "next")
            k, v = q.kv4_read(s["cache"], s["slots"])
            return {"q": turned, "k": k, "v": v}
        if s["lse"]:
            y, lse = q.kv4_attention(s["q"], s["cache"], s["table"], s["lens"], cu_q=s["cu"], max_q=s["most"],
                                     window=s["window"], return_lse=True)
            return {"y": y, "lse": lse}
        return {"y": q.kv4_attention(s["q"], s["cache"], s["table"], s["lens"], cu_q=s["cu"], max_q=s["most"],
                                     window=s["window"])}
    return (_append_plain if s["op"] == "append" else _attend_plain)(s)


def _row_bytes(case):
    """A token's keys and values in the cache."""
    return 2 * case["n_kv"] * (case["d"] // 2 + 4 * (case["d"] // case["group"]))


def work(case):
    d, n_q, n_kv = case["d"], case["n_q"], case["n_kv"]
    if case["op"] == "append":  # rows read, written and (keys, values) read back; angles, slots, positions
        t, e = case["t"], 2 if case["type"] == "bf16" else 4
        row = (n_q + 2 * n_kv) * d * (e + 2) + 2 * _row_bytes(case) + 4 * case["rot"] + 16
        return {"bytes": t * row, "flops": t * d * (3.0 * n_q + 12.0 * n_kv)}
    n, keys = _batch(case)
    seen = pairs = 0
    for m, length in zip(n, keys):
        if length:
            w = case["window"] or length
            seen += min(length, m - 1 + w)
            pairs += sum(min(length - m + j + 1, w) for j in range(m))
    rows = sum(n) * n_q
    return {"bytes": seen * _row_bytes(case) + rows * d * 4 + (rows * 4 if case["lse"] else 0),
            "flops": 4.0 * pairs * n_q * d}


def exact(case, seed):
    s = prepare(case, seed)
    d, group, page = case["d"], case["group"], case["page"]
    if case["op"] == "append":
        rot = case["rot"]

        def turned(x):
            x = x.double()
            if rot:
                cos, sin = s["cos"].double()[s["positions"]], s["sin"].double()[s["positions"]]
                out = x.clone()
                for j in range(rot // 2):
                    i0, i1 = (j, j + rot // 2) if case["pairs"] == "half" else (2 * j, 2 * j + 1)
                    c, w = cos[:, j, None], sin[:, j, None]
                    out[:, :, i0] = x[:, :, i0] * c - x[:, :, i1] * w
                    out[:, :, i1] = x[:, :, i1] * c + x[:, :, i0] * w
                x = out
            return x

        def through(x):  # the roundings that the cache's format is defined by
            x = x.float().bfloat16().double()
            out = torch.empty_like(x)
            for g in range(0, d, group):
                v = x[:, :, g:g + group]
                lo = v.min(-1, keepdim=True).values
                step = ((v.max(-1, keepdim=True).values - lo).float() / 15.0).bfloat16().double()
                code = torch.nan_to_num((v - lo).float().double() / step, 0.0, 0.0, 0.0).round().clamp(max=15.0)
                out[:, :, g:g + group] = lo + step * code
            return out

        return {"q": turned(s["q"]), "k": through(turned(s["k"])), "v": through(s["v"].double())}
    n, keys = _batch(case)
    n_kv, heads = case["n_kv"], case["n_q"] // case["n_kv"]
    dims = torch.arange(d, device=s["q"].device)
    c = dims // 32
    k_byte, k_up = (dims % 32 // 8) * (d // 8) + 4 * c + dims % 4, dims % 8 // 4 * 4
    v_byte, v_up = (dims % 32 // 2) * (d // 8) + 4 * c, dims % 2 * 4
    y = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    lse = torch.full(y.shape[:2], -math.inf, dtype=torch.float64, device=y.device)
    row = 0
    for b, (m, length) in enumerate(zip(n, keys)):
        if length:
            key = torch.arange(length, device=y.device)
            at, tok = s["table"][b].long()[key // page], key % page
            place = length - m + torch.arange(m, device=y.device)
            hidden = key[None] > place[:, None]
            if case["window"]:
                hidden |= key[None] <= place[:, None] - case["window"]
            for h in range(n_kv):
                k = (s["cache"][0][at, h, tok][:, k_byte] >> k_up & 15).double()
                v = (s["cache"][2][at, h, tok // 4][torch.arange(length, device=y.device)[:, None], v_byte + tok[:, None] % 4]
                     >> v_up & 15).double()
                ks, vs = (s["cache"][j][at, h, :, tok].double()[:, dims // group] for j in (1, 3))
                k, v = k * ks[..., 0] + ks[..., 1], v * vs[..., 0] + vs[..., 1]
                for j in range(h * heads, (h + 1) * heads):
                    score = s["q"][row:row + m, j].double() @ k.t() / math.sqrt(d)
                    score[hidden] = -math.inf
                    norm = torch.logsumexp(score, 1)
                    y[row:row + m, j] = (score - norm[:, None]).exp() @ v
                    lse[row:row + m, j] = norm
        row += m
    return {"y": y, "lse": lse} if case["lse"] else {"y": y}
