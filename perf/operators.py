"""Operators of 8-bit decoding: what is measured, and what each has to give.

The path is the one a user of the library runs with 8-bit weights and an 8-bit
cache: activations are quantised and multiplied with quantised weights
(``gemm``), queries and keys are turned by their positions (``rope``), new keys
and values are quantised into the cache and read back (``cache``), and queries
attend over the quantised cache (``attention``).

Codes are e4m3.  A scale is a power of two, stored as one byte, 2^(byte - 127)
(255: not a number): the smallest with amax / scale <= 448, and 1 for a block
of zeros.  Dividing by it does not round, so a code is a single rounding of its
value and does not depend on the width of the arithmetic.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZES = {"f32": 4, "bf16": 2, "f16": 2}
BLOCK = 128          # elements along K that share a scale in the matrix product


# --------------------------------------------------------------------------- cases

def listed():
    return [
        # queries and keys of one 32-position block, the heads of the 8B configuration: a launch's latency
        {"name": "rope_block", "kind": "rope", "rows": 32, "heads": 64, "hd": 128, "rot": 128, "layout": "half",
         "scaling": "none", "factor": 1.0, "theta": 1e4, "pos0": 512, "dtype": "bf16"},
        # a long chunk far into a stretched context: part of the head turns, interleaved pairs
        {"name": "rope_long_partial", "kind": "rope", "rows": 8191, "heads": 40, "hd": 128, "rot": 64,
         "layout": "interleaved", "scaling": "by_parts", "factor": 32.0, "theta": 5e5, "pos0": 122880, "dtype": "bf16"},
        # one new token of each of 8 sequences, grouped heads
        {"name": "cache_token", "kind": "cache", "b": 8, "R": 1, "Hkv": 8, "T": 4097, "hd": 128, "start": 4000,
         "pad": 0, "dtype": "bf16"},
        # a decoded block of 32 positions of each of 64 sequences, the 8B configuration's heads (batch sweep's end)
        {"name": "cache_block", "kind": "cache", "b": 64, "R": 32, "Hkv": 32, "T": 256, "hd": 128, "start": 128,
         "pad": 0, "dtype": "bf16"},
        # a padded prefill of float32 projections, ragged, small heads
        {"name": "cache_prefill_f32", "kind": "cache", "b": 3, "R": 5000, "Hkv": 16, "T": 5003, "hd": 64, "start": 0,
         "pad": 77, "dtype": "f32"},
        # single-token decoding of 8 sequences of different lengths, 4 query heads to a cached one
        {"name": "attention_token", "kind": "attention", "b": 8, "R": 1, "H": 32, "Hkv": 8, "T": 8193, "hd": 128,
         "mask": "full", "ragged": True, "pad": 0},
        # one block of 32 queries over the whole canvas: the 8B DualCache step
        {"name": "attention_block", "kind": "attention", "b": 1, "R": 32, "H": 32, "Hkv": 32, "T": 768, "hd": 128,
         "mask": "full", "ragged": False, "pad": 0},
        # the same block for a batch on the long workload, the last sequence padded with rows that see nothing
        {"name": "attention_block_batch", "kind": "attention", "b": 16, "R": 32, "H": 32, "Hkv": 32, "T": 2048,
         "hd": 128, "mask": "full", "ragged": True, "pad": 5},
        # a prefill over its own cache: every row sees the keys up to itself
        {"name": "attention_prefill", "kind": "attention", "b": 1, "R": 4096, "H": 32, "Hkv": 8, "T": 4096, "hd": 128,
         "mask": "causal", "ragged": False, "pad": 0},
        # one token through a square projection of the 8B configuration
        {"name": "gemm_token", "kind": "gemm", "M": 4096, "N": 1, "K": 4096, "out": "f32"},
        # one block through the 8B gate and up projections
        {"name": "gemm_block", "kind": "gemm", "M": 24576, "N": 32, "K": 4096, "out": "f32"},
        # a refresh of 2048 positions through the 8B QKV projection
        {"name": "gemm_refresh", "kind": "gemm", "M": 12288, "N": 2048, "K": 4096, "out": "bf16"},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["rope", "cache", "attention", "attention", "gemm", "gemm"])
    if kind == "rope":
        hd = rng.choice([64, 128])
        scaling = rng.choice(["none", "linear", "base", "by_parts"])
        heads = _log_int(rng, 1, 64)
        return {"kind": "rope", "rows": _log_int(rng, 1, min(8191, 8191 * 40 // heads)), "heads": heads, "hd": hd,
                "rot": rng.choice([hd, hd // 2, hd // 4]), "layout": rng.choice(["half", "interleaved"]),
                "scaling": scaling, "factor": 1.0 if scaling == "none" else rng.choice([2.0, 8.0, 32.0]),
                "theta": rng.choice([1e4, 5e5, 1e6]), "pos0": _log_int(rng, 1, 1000000),
                "dtype": rng.choice(["bf16", "f16", "f32"]) if heads <= 32 else "bf16"}
    if kind == "cache":
        b, hkv = _log_int(rng, 1, 64), _log_int(rng, 1, 32)
        hd = rng.choice([64, 128])
        r = _log_int(rng, 1, max(1, min(5000, 64 * 32 * 32 // (b * hkv))))
        start = rng.choice([0, _log_int(rng, 1, 4096)])
        return {"kind": "cache", "b": b, "R": r, "Hkv": hkv, "T": start + r + rng.randrange(0, 9), "hd": hd,
                "start": start, "pad": rng.randrange(0, r), "dtype": rng.choice(["bf16", "f16", "f32"])}
    if kind == "attention":
        form = rng.choice(["token", "block", "block", "prefill"])
        hd = rng.choice([64, 128])
        hkv = rng.choice([1, 2, 4, 8, 16, 32])
        h = hkv * rng.choice([g for g in (1, 2, 4, 8) if g * hkv <= 32])
        if form == "token":
            b, r, t = _log_int(rng, 1, 32), 1, _log_int(rng, 1, 32768)
        elif form == "block":
            b, r, t = _log_int(rng, 1, 16), rng.choice([4, 16, 17, 32, 64]), _log_int(rng, 64, 4096)
        else:
            b, r, t = rng.randrange(1, 3), _log_int(rng, 65, 2048), 0
            t = r + _log_int(rng, 1, 1024)
        while b > 1 and b * hkv * t * hd > 16 * 32 * 2048 * 128:
            b = b // 2
        return {"kind": "attention", "b": b, "R": r, "H": h, "Hkv": hkv, "T": t, "hd": hd,
                "mask": rng.choice(["full", "causal"]), "ragged": rng.random() < 0.5,
                "pad": rng.randrange(0, r) if rng.random() < 0.3 else 0}
    m = rng.choice([256, 688, 2048, 4096, 5504, 12288, _log_int(rng, 1, 12288)])
    k = rng.choice([256, 688, 2048, 4096, 5504, 16 * _log_int(rng, 1, 344)])
    return {"kind": "gemm", "M": m, "N": _log_int(rng, 1, min(2048, 12288 * 2048 * 4096 // (m * k))), "K": k, "out": rng.choice(["f32", "bf16"])}


# --------------------------------------------------------------------------- inputs

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _activations(g, rows, n):
    """Normal values with a few channels an order of magnitude larger, as hidden states have them."""
    x = _normal(g, rows, n)
    loud = torch.rand(n, generator=g, device="cuda") < 0.01
    return x * torch.where(loud, 12.0, 1.0)


def _limits(case):
    """Keys each row sees, [b][R]: the plan of the call, the same for every seed."""
    b, r, t = case["b"], case["R"], case["T"]
    out = []
    for s in range(b):
        n = t - (s * t) // (2 * b) if case["ragged"] else t
        row = [n - r + i + 1 if case["mask"] == "causal" else n for i in range(r)]
        if s == b - 1 and case["pad"]:
            row[r - case["pad"]:] = [0] * case["pad"]
        out.append([max(0, x) for x in row])
    return out


def _quantise(x):
    """Blocks along the last axis to (codes as uint8, exponent bytes)."""
    amax = x.abs().amax(dim=-1, keepdim=True)
    m, e = torch.frexp(amax)
    e = torch.where(m > 0.875, e - 8, e - 9).clamp_min(-127)
    e = torch.where(amax == 0, torch.zeros_like(e), e)
    codes = torch.ldexp(x, -e).to(torch.float8_e4m3fn).view(torch.uint8)
    return codes, (e + 127).squeeze(-1).to(torch.uint8)


def _quantise_blocks(x):
    """[rows][K] to codes [rows][K] and scale bytes [ceil(K/128)][rows]."""
    rows, k = x.shape
    kb = -(-k // BLOCK)
    p = torch.zeros(rows, kb * BLOCK, device=x.device, dtype=torch.float32)
    p[:, :k] = x
    c, s = _quantise(p.view(rows, kb, BLOCK))
    return c.view(rows, kb * BLOCK)[:, :k].contiguous(), s.t().contiguous()


def _values(codes, scale):
    """Codes and their scale bytes (one fewer axis) to float32."""
    e = scale.to(torch.int32) - 127
    return torch.ldexp(codes.view(torch.float8_e4m3fn).to(torch.float32), e.unsqueeze(-1))


def prepare(case, seed):
    g = _generator(seed)
    kind = case["kind"]
    st = {"case": case}
    if kind == "rope":
        rows, heads, hd = case["rows"], case["heads"], case["hd"]
        st["x"] = _normal(g, rows, heads, hd).to(DTYPES[case["dtype"]])
        st["out"] = torch.empty_like(st["x"])
        st["pos"] = (case["pos0"] + torch.arange(rows, device="cuda")).to(torch.int32)
        if own:
            from cached_masked_decoding_gb300 import binding
            st["spec"] = binding.make_rope(case["rot"], layout=case["layout"], theta=case["theta"],
                                           scaling=case["scaling"], factor=case["factor"], orig_len=4096)
    elif kind == "cache":
        b, r, h, t, hd = case["b"], case["R"], case["Hkv"], case["T"], case["hd"]
        dt = DTYPES[case["dtype"]]
        st["k"] = _activations(g, b * r, h * hd).view(b, r, h, hd).to(dt)
        st["v"] = _normal(g, b, r, h, hd).to(dt)
        st["codes"] = [torch.zeros(b, h, t, hd, device="cuda", dtype=torch.uint8) for _ in range(2)]
        st["scales"] = [torch.full((b, h, t), 127, device="cuda", dtype=torch.uint8) for _ in range(2)]
        st["back"] = [torch.zeros(b, r, h, hd, device="cuda", dtype=dt) for _ in range(2)]
        st["starts"] = torch.full((b,), case["start"], device="cuda", dtype=torch.int32)
        counts = [r] * b
        counts[-1] -= case["pad"]
        st["counts_host"] = counts
        st["counts"] = torch.tensor(counts, device="cuda", dtype=torch.int32)
        if own:
            from cached_masked_decoding_gb300 import binding
            st["cache"] = binding.make_kv8(st["codes"][0].data_ptr(), st["codes"][1].data_ptr(),
                                           st["scales"][0].data_ptr(), st["scales"][1].data_ptr(), b, h, t, hd)
    elif kind == "attention":
        b, r, h, hkv, t, hd = case["b"], case["R"], case["H"], case["Hkv"], case["T"], case["hd"]
        st["q"] = (1.5 * _normal(g, b, r, h, hd)).to(torch.bfloat16)
        kc, ks = _quantise(_activations(g, b * hkv * t, hd))
        vc, vs = _quantise(_normal(g, b * hkv * t, hd))
        st["codes"] = [kc.view(b, hkv, t, hd), vc.view(b, hkv, t, hd)]
        st["scales"] = [ks.view(b, hkv, t), vs.view(b, hkv, t)]
        st["limits"] = torch.tensor(_limits(case), device="cuda", dtype=torch.int32)
        st["out"] = torch.empty(b, r, h, hd, device="cuda", dtype=torch.bfloat16)
        st["scale"] = 1.0 / math.sqrt(hd)
        if own:
            from cached_masked_decoding_gb300 import binding
            st["cache"] = binding.make_kv8(st["codes"][0].data_ptr(), st["codes"][1].data_ptr(),
                                           st["scales"][0].data_ptr(), st["scales"][1].data_ptr(), b, hkv, t, hd)
            st["ws"] = torch.empty(max(16, binding.attention_kv8_workspace(b, h, hkv, hd, r, t)), device="cuda",
                                   dtype=torch.uint8)
    else:
        m, n, k = case["M"], case["N"], case["K"]
        st["w"], st["ws"] = _quantise_blocks(0.02 * _normal(g, m, k))
        st["x"] = _activations(g, n, k).to(torch.bfloat16)
        st["xc"] = torch.empty(n, k, device="cuda", dtype=torch.uint8)
        st["xs"] = torch.empty(-(-k // BLOCK), n, device="cuda", dtype=torch.uint8)
        st["y"] = torch.empty(n, m, device="cuda", dtype=DTYPES[case["out"]])
    return st


# --------------------------------------------------------------------------- one pass

def _frequencies(case):
    """Turning rate of each pair, radians a position, and the amplitude, in 64 bits."""
    rot, theta, s = case["rot"], case["theta"], case["factor"]
    i = torch.arange(rot // 2, dtype=torch.float64, device="cuda")
    amp = 1.0
    if case["scaling"] == "base":
        theta = theta * s ** (rot / (rot - 2))
    f = theta ** (-2.0 * i / rot)
    if case["scaling"] == "linear":
        f = f / s
    elif case["scaling"] == "by_parts":
        def at(turns):
            return rot * math.log(4096 / (turns * 2 * math.pi)) / (2 * math.log(theta))
        lo, hi = max(0, math.floor(at(32.0))), min(rot // 2 - 1, math.ceil(at(1.0)))
        ramp = ((i - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        f = f / s * ramp + f * (1 - ramp)
        amp = 0.1 * math.log(s) + 1.0
    return f, amp


def _run_plain(st):
    case = st["case"]
    kind = case["kind"]
    if kind == "rope":
        rot = case["rot"]
        f, amp = _frequencies(case)
        a = st["pos"].to(torch.float64)[:, None] * f
        c, s = (amp * a.cos()).float()[:, None], (amp * a.sin()).float()[:, None]
        x = st["x"].float()
        out = x.clone()
        if case["layout"] == "half":
            x0, x1 = x[..., :rot // 2], x[..., rot // 2:rot]
            out[..., :rot // 2], out[..., rot // 2:rot] = x0 * c - x1 * s, x1 * c + x0 * s
        else:
            x0, x1 = x[..., 0:rot:2], x[..., 1:rot:2]
            out[..., 0:rot:2], out[..., 1:rot:2] = x0 * c - x1 * s, x1 * c + x0 * s
        st["out"].copy_(out)
        return st["out"]
    if kind == "cache":
        for src, codes, scales, back in zip((st["k"], st["v"]), st["codes"], st["scales"], st["back"]):
            c, s = _quantise(src.float().transpose(1, 2))
            for i, n in enumerate(st["counts_host"]):
                p = case["start"]
                codes[i, :, p:p + n], scales[i, :, p:p + n] = c[i, :, :n], s[i, :, :n]
                back[i, :n] = _values(codes[i, :, p:p + n], scales[i, :, p:p + n]).transpose(0, 1).to(back.dtype)
        return st["back"]
    if kind == "attention":
        b, r, h, hkv, t, hd = case["b"], case["R"], case["H"], case["Hkv"], case["T"], case["hd"]
        k, v = (_values(c, s)[:, :, None] for c, s in zip(st["codes"], st["scales"]))
        q = st["q"].float().view(b, r, hkv, h // hkv, hd).permute(0, 2, 3, 1, 4)
        sees = (torch.arange(t, device="cuda") < st["limits"][..., None])[:, None, None]
        z = torch.matmul(q, k.transpose(-1, -2)).mul_(st["scale"]).masked_fill_(~sees, -math.inf)
        top = z.amax(dim=-1, keepdim=True)
        top = torch.where(top == -math.inf, torch.zeros_like(top), top)
        z = z.sub_(top).exp_()
        total = z.sum(dim=-1, keepdim=True)
        o = torch.matmul(z, v) / torch.where(total == 0, torch.ones_like(total), total)
        st["out"].copy_(o.permute(0, 3, 1, 2, 4).reshape(b, r, h, hd))
        return st["out"]
    k, kb = case["K"], st["ws"].shape[0]
    xc, xs = _quantise_blocks(st["x"].float())
    w = st["w"].view(torch.float8_e4m3fn).float()
    x = xc.view(torch.float8_e4m3fn).float()
    w = torch.ldexp(w, (st["ws"].to(torch.int32) - 127).t().repeat_interleave(BLOCK, dim=1)[:, :k])
    x = torch.ldexp(x, (xs.to(torch.int32) - 127).t().repeat_interleave(BLOCK, dim=1)[:, :k])
    st["y"].copy_(torch.matmul(x, w.t()))
    return st["y"]


def run(st):
    if not own:
        return _run_plain(st)
    from cached_masked_decoding_gb300 import binding
    case = st["case"]
    kind = case["kind"]
    stream = torch.cuda.current_stream().cuda_stream
    if kind == "rope":
        binding.op_rope(st["x"].data_ptr(), st["out"].data_ptr(), st["pos"].data_ptr(), case["rows"], case["heads"],
                        case["hd"], case["dtype"], st["spec"], stream=stream)
        return st["out"]
    if kind == "cache":
        binding.op_kv8_store(st["cache"], st["k"].data_ptr(), st["v"].data_ptr(), case["dtype"], case["R"],
                             starts_ptr=st["starts"].data_ptr(), counts_ptr=st["counts"].data_ptr(), stream=stream)
        binding.op_kv8_load(st["cache"], st["back"][0].data_ptr(), st["back"][1].data_ptr(), case["dtype"], case["R"],
                            starts_ptr=st["starts"].data_ptr(), counts_ptr=st["counts"].data_ptr(), stream=stream)
        return st["back"]
    if kind == "attention":
        binding.op_attention_kv8(st["q"].data_ptr(), st["cache"], st["out"].data_ptr(), case["H"], case["R"],
                                 limits_ptr=st["limits"].data_ptr(), scale=st["scale"], ws_ptr=st["ws"].data_ptr(),
                                 ws_bytes=st["ws"].numel(), stream=stream)
        return st["out"]
    m, n, k = case["M"], case["N"], case["K"]
    binding.op_quantise8(st["x"].data_ptr(), "bf16", n, k, st["xc"].data_ptr(), st["xs"].data_ptr(), stream=stream)
    binding.op_gemm8(st["w"].data_ptr(), st["ws"].data_ptr(), st["xc"].data_ptr(), st["xs"].data_ptr(),
                     st["y"].data_ptr(), case["out"], m, n, k, stream=stream)
    return st["y"]


# --------------------------------------------------------------------------- work of one pass

def work(case):
    kind = case["kind"]
    if kind == "rope":
        n = case["rows"] * case["heads"]
        return {"bytes": 2 * n * case["hd"] * SIZES[case["dtype"]] + 4 * case["rows"], "flops": 3 * n * case["rot"]}
    if kind == "cache":
        n = 2 * (case["b"] * case["R"] - case["pad"]) * case["Hkv"]
        return {"bytes": n * (case["hd"] * (2 * SIZES[case["dtype"]] + 1) + 1), "flops": 4 * n * case["hd"]}
    if kind == "attention":
        lim = _limits(case)
        keys = sum(max(row) for row in lim)
        return {"bytes": 2 * keys * case["Hkv"] * (case["hd"] + 1) + 4 * case["b"] * case["R"] * case["H"] * case["hd"],
                "flops": 4 * case["hd"] * case["H"] * sum(sum(row) for row in lim)}
    m, n, k = case["M"], case["N"], case["K"]
    kb = -(-k // BLOCK)
    return {"bytes": m * (k + kb) + 2 * n * k + n * m * SIZES[case["out"]], "flops": 2 * m * n * k}


# --------------------------------------------------------------------------- the definition, in 64 bits

def _decode64(codes):
    """e4m3 by its definition: sign, four exponent bits (bias 7), three of mantissa."""
    c = codes.to(torch.int64)
    e, m = (c >> 3) & 15, (c & 7).to(torch.float64)
    mag = torch.where(e == 0, m * 2.0 ** -9, (8 + m) * torch.exp2((e - 10).to(torch.float64)))
    return torch.where(c >= 128, -mag, mag)


def _round64(x):
    """Values of blocks along the last axis after quantisation, from the definition."""
    amax = x.abs().amax(dim=-1, keepdim=True)
    e = torch.ceil(torch.log2(torch.where(amax > 0, amax, torch.full_like(amax, 448.0)) / 448.0))
    # the logarithm may land on the wrong side of a whole number: step to the smallest that fits
    e = torch.where(amax > 448.0 * torch.exp2(e), e + 1, e)
    e = torch.where((amax > 0) & (amax <= 448.0 * torch.exp2(e - 1)), e - 1, e).clamp_min(-127)
    y = x * torch.exp2(-e)
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -6))) - 3)
    return torch.round(y / step) * step * torch.exp2(e)


def _rates64(case):
    """Turning rates pair by pair and the amplitude, from their definition."""
    rot, log_theta, s = case["rot"], math.log(case["theta"]), case["factor"]
    if case["scaling"] == "base":
        log_theta += math.log(s) * rot / (rot - 2)
    rates = []
    for i in range(rot // 2):
        f = math.exp(-log_theta * 2 * i / rot)
        if case["scaling"] == "linear":
            f /= s
        if case["scaling"] == "by_parts":
            # pairs that turn 32 times or more within the original 4096 positions keep
            # their rate, those that turn less than once are slowed by the factor
            edge = [math.log(4096 / (2 * math.pi * turns)) * rot / (2 * log_theta) for turns in (32, 1)]
            lo, hi = max(0, math.floor(edge[0])), min(rot // 2 - 1, math.ceil(edge[1]))
            slow = min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001)))
            f = slow * f / s + (1 - slow) * f
        rates.append(f)
    amp = 1.0 + 0.1 * math.log(s) if case["scaling"] == "by_parts" else 1.0
    return torch.tensor(rates, device="cuda", dtype=torch.float64), amp


def exact(case, seed):
    st = prepare(case, seed)
    kind = case["kind"]
    if kind == "rope":
        rot = case["rot"]
        f, amp = _rates64(case)
        out = st["x"].double()
        z = torch.polar(torch.full((case["rows"], rot // 2), float(amp), device="cuda", dtype=torch.float64),
                        torch.outer(st["pos"].double(), f))
        part = out[..., :rot]
        pairs = part.unflatten(-1, (2, rot // 2)).transpose(-1, -2) if case["layout"] == "half" else \
            part.unflatten(-1, (rot // 2, 2))
        turned = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * z[:, None])
        if case["layout"] == "half":
            turned = turned.transpose(-1, -2)
        return torch.cat([turned.flatten(-2), out[..., rot:]], dim=-1)
    if kind == "cache":
        outs = []
        for src in (st["k"], st["v"]):
            o = _round64(src.double())
            if case["pad"]:
                o[-1, case["R"] - case["pad"]:] = 0
            outs.append(o)
        return outs
    if kind == "attention":
        b, r, h, hkv, hd = case["b"], case["R"], case["H"], case["Hkv"], case["hd"]
        lim = _limits(case)
        out = torch.zeros(b, r, h, hd, device="cuda", dtype=torch.float64)
        for s in range(b):
            n = max(lim[s])
            if n == 0:
                continue
            see = torch.arange(n, device="cuda")[None] < st["limits"][s][:, None]
            for j in range(hkv):
                k = _decode64(st["codes"][0][s, j, :n]) * torch.exp2(st["scales"][0][s, j, :n, None].double() - 127)
                v = _decode64(st["codes"][1][s, j, :n]) * torch.exp2(st["scales"][1][s, j, :n, None].double() - 127)
                for i in range(j * (h // hkv), (j + 1) * (h // hkv)):
                    z = (st["q"][s, :, i].double() @ k.t()) * st["scale"]
                    p = torch.softmax(z.masked_fill(~see, -math.inf), dim=-1)
                    out[s, :, i] = torch.nan_to_num(p, nan=0.0) @ v
        return out
    k = case["K"]
    kb = -(-k // BLOCK)
    x = torch.nn.functional.pad(st["x"].double(), (0, kb * BLOCK - k)).unflatten(1, (kb, BLOCK))
    x = _round64(x).flatten(1)[:, :k]
    y = torch.empty(case["N"], case["M"], device="cuda", dtype=torch.float64)
    for m0 in range(0, case["M"], 4096):
        e = torch.exp2(st["ws"][:, m0:m0 + 4096].t().double() - 127).repeat_interleave(BLOCK, dim=1)[:, :k]
        y[:, m0:m0 + 4096] = x @ (_decode64(st["w"][m0:m0 + 4096]) * e).t()
    return y
