"""Operators of decoding over a paged cache: what is measured, and what each has to give.

One layer of a serving step, and the end of the model, as a user of the library
runs them when sequences of different lengths share a pool of pages: queries and
keys are normalised head by head, turned by their positions and put away
(``heads``); a token or a block of each sequence attends over its pages, and the
weight that every cached key received is added up (``attention``); a cache that
has grown too long keeps its heaviest keys (``evict``); the logits give the log
probability of a token, the entropy and the likeliest alternatives
(``logprobs``).

A page holds ``ps`` tokens of every cached head, [pages][H_kv][ps][hd]; a table
[b][pages of a sequence] names the pages of a sequence in the order of its
positions.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZES = {"f32": 4, "bf16": 2, "f16": 2}


# --------------------------------------------------------------------------- cases

def listed():
    return [
        # one new token of each of 8 sequences into its pages, grouped heads: a launch's latency
        {"name": "heads_token", "kind": "heads", "b": 8, "R": 1, "H": 32, "Hkv": 8, "hd": 128, "rot": 128,
         "layout": "half", "norm": True, "theta": 1e6, "ps": 16, "start": 4000, "pad": 0, "paged": True,
         "dtype": "bf16", "out": "bf16"},
        # a padded chunk of 8191 prompt tokens into pages, far into the context
        {"name": "heads_prefill", "kind": "heads", "b": 1, "R": 8191, "H": 32, "Hkv": 8, "hd": 128, "rot": 128,
         "layout": "half", "norm": True, "theta": 5e5, "ps": 64, "start": 24576, "pad": 5, "paged": True,
         "dtype": "bf16", "out": "bf16"},
        # float32 projections of 64 blocks of 32 positions, half of a small head turned, rows out as bf16
        {"name": "heads_block_f32", "kind": "heads", "b": 64, "R": 32, "H": 16, "Hkv": 16, "hd": 64, "rot": 32,
         "layout": "interleaved", "norm": True, "theta": 1e4, "ps": 16, "start": 512, "pad": 0, "paged": False,
         "dtype": "f32", "out": "bf16"},
        # one block of 32 positions over a short canvas, every head its own: the 8B configuration's heads
        {"name": "attention_block", "kind": "attention", "b": 1, "R": 32, "H": 32, "Hkv": 32, "T": 768, "hd": 128,
         "ps": 16, "ragged": False, "empty": False, "mass": False, "dtype": "bf16"},
        # one token of each of 16 small-headed sequences, weights added up for a later eviction, one slot unused
        {"name": "attention_token_weights", "kind": "attention", "b": 16, "R": 1, "H": 32, "Hkv": 8, "T": 4099,
         "hd": 64, "ps": 16, "ragged": True, "empty": True, "mass": True, "dtype": "f16"},
        # one token of a single sequence with a very long history
        {"name": "attention_token_long", "kind": "attention", "b": 1, "R": 1, "H": 32, "Hkv": 8, "T": 131071,
         "hd": 128, "ps": 64, "ragged": False, "empty": False, "mass": False, "dtype": "bf16"},
        # a busy server: one token of each of 64 sequences of 4 to 8 thousand keys
        {"name": "attention_token_batch", "kind": "attention", "b": 64, "R": 1, "H": 32, "Hkv": 8, "T": 8192,
         "hd": 128, "ps": 16, "ragged": True, "empty": False, "mass": False, "dtype": "bf16"},
        # one sequence's cache cut to a quarter while it decodes
        {"name": "evict_one", "kind": "evict", "b": 1, "Hkv": 8, "T": 4097, "hd": 128, "keep": 1024, "sinks": 4,
         "recent": 128, "ps": 16, "ps_out": 16, "ragged": False, "dtype": "bf16"},
        # a batch of long caches cut after their prefill
        {"name": "evict_batch", "kind": "evict", "b": 8, "Hkv": 8, "T": 32768, "hd": 128, "keep": 8192, "sinks": 4,
         "recent": 1024, "ps": 64, "ps_out": 64, "ragged": True, "dtype": "bf16"},
        # the logits of one block of 32 positions, the 8B vocabulary
        {"name": "logprobs_block", "kind": "logprobs", "rows": 32, "vocab": 126464, "top": 5, "temperature": 1.0,
         "pad": 0, "dtype": "bf16"},
        # float32 logits of an odd vocabulary, warmed, rows of a wider buffer
        {"name": "logprobs_odd_f32", "kind": "logprobs", "rows": 257, "vocab": 32001, "top": 20, "temperature": 0.7,
         "pad": 3, "dtype": "f32"},
        # scoring 4096 positions of a prompt
        {"name": "logprobs_prompt", "kind": "logprobs", "rows": 4096, "vocab": 126464, "top": 20, "temperature": 1.0,
         "pad": 0, "dtype": "bf16"},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["heads", "attention", "attention", "attention", "evict", "logprobs", "logprobs"])
    if kind == "heads":
        hd = rng.choice([64, 128])
        hkv = rng.choice([1, 2, 4, 8, 16, 32])
        h = hkv * rng.choice([g for g in (1, 2, 4, 8) if g * hkv <= 32])
        b = _log_int(rng, 1, 64)
        r = 1 if rng.random() < 0.4 else _log_int(rng, 2, max(2, 8191 * 48 * 128 // (b * (h + 2 * hkv) * hd * 2)))
        dtype = rng.choice(["bf16", "f16", "f32"])
        paged = rng.random() < 0.7
        return {"kind": "heads", "b": b, "R": r, "H": h, "Hkv": hkv, "hd": hd, "rot": rng.choice([hd, hd // 2]),
                "layout": rng.choice(["half", "interleaved"]), "norm": rng.random() < 0.8,
                "theta": rng.choice([1e4, 5e5, 1e6]), "ps": rng.choice([16, 32, 64, 128]),
                "start": rng.choice([0, _log_int(rng, 1, 32768)]), "pad": rng.randrange(0, r) if paged else 0,
                "paged": paged, "dtype": dtype,
                "out": rng.choice(["bf16", "f16"]) if dtype == "f32" and paged else
                rng.choice(["bf16", "f32"]) if dtype == "f32" else dtype}
    if kind == "attention":
        hd = rng.choice([64, 128])
        hkv = rng.choice([1, 2, 4, 8, 16, 32])
        h = hkv * rng.choice([g for g in (1, 2, 4, 8) if g * hkv <= 32])
        if rng.random() < 0.7:
            b, r, t = _log_int(rng, 1, 64), 1, _log_int(rng, 1, 131071)
        else:
            b, r, t = _log_int(rng, 1, 16), rng.choice([4, 16, 17, 32]), _log_int(rng, 32, 8192)
        while b > 1 and (b * hkv * t * hd > 64 * 8 * 4096 * 128 or b * h * r * t > 1 << 25):
            b = b // 2
        t = min(t, 64 * 8 * 4096 * 128 // (b * hkv * hd))
        return {"kind": "attention", "b": b, "R": r, "H": h, "Hkv": hkv, "T": t, "hd": hd,
                "ps": rng.choice([16, 32, 64, 128]), "ragged": rng.random() < 0.6,
                "empty": b > 1 and rng.random() < 0.2, "mass": rng.random() < 0.35,
                "dtype": rng.choice(["bf16", "f16"])}
    if kind == "evict":
        hd = rng.choice([64, 128])
        hkv = rng.choice([1, 2, 4, 8, 16])
        b, t = _log_int(rng, 1, 16), _log_int(rng, 64, 32768)
        while b > 1 and b * hkv * t * hd > 8 * 8 * 16384 * 128:
            b = b // 2
        keep = max(16, t // rng.choice([2, 3, 4, 8]))
        sinks = rng.choice([0, 4, 16])
        return {"kind": "evict", "b": b, "Hkv": hkv, "T": t, "hd": hd, "keep": keep, "sinks": sinks,
                "recent": rng.randrange(0, max(1, (keep - sinks) // 2)), "ps": rng.choice([16, 32, 64, 128]),
                "ps_out": rng.choice([16, 64]), "ragged": rng.random() < 0.5, "dtype": rng.choice(["bf16", "f16"])}
    vocab = rng.choice([1024, 32000, 126464, _log_int(rng, 100, 262144)])
    dtype = rng.choice(["bf16", "f16", "f32"])
    return {"kind": "logprobs", "rows": _log_int(rng, 1, max(1, min(4096, 2048 * 126464 // vocab))), "vocab": vocab,
            "top": rng.choice([0, 1, 5, 20, 50]), "temperature": rng.choice([1.0, 1.0, 0.6, 1.3]),
            "pad": rng.choice([0, 0, rng.randrange(1, 9)]), "dtype": dtype}


# --------------------------------------------------------------------------- inputs

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _lens(case):
    """Cached tokens of each sequence, the same for every seed."""
    b, t = case["b"], case["T"]
    out = [t - (s * t) // (2 * b) if case["ragged"] else t for s in range(b)]
    if case.get("empty"):
        out[-1] = 0
    return out


def _pool(g, b, t, hkv, ps, hd, dt, values):
    """K and V pools of the pages that b sequences of up to t tokens need, with some to spare, and the table of a
    server that has been running for a while: pages in no order."""
    n = -(-t // ps)
    pages = b * n + 3
    table = torch.randperm(pages, generator=g, device="cuda")[:b * n].view(b, n).to(torch.int32)
    kv = [torch.zeros(pages, hkv, ps, hd, device="cuda", dtype=dt) for _ in range(2)]
    if values:
        # keys with a few loud channels, as projections have them; page by page, the spare ones too
        loud = torch.where(torch.rand(hd, generator=g, device="cuda") < 0.02, 6.0, 1.0)
        for x, scale in zip(kv, (loud, 1.0)):
            for part in x.split(max(1, (1 << 26) // (hkv * ps * hd))):
                part.copy_(_normal(g, *part.shape) * scale)
    return kv, table


def _cache(case, kv, table, ps):
    from cached_masked_decoding_gb300 import binding
    return binding.make_kv_paged(kv[0].data_ptr(), kv[1].data_ptr(), table.data_ptr(), case["b"], case["Hkv"],
                                 case["hd"], case.get("out", case["dtype"]), kv[0].shape[0], ps, table.shape[1])


def prepare(case, seed):
    g = _generator(seed)
    kind = case["kind"]
    dt = DTYPES[case["dtype"]]
    st = {"case": case}
    if kind == "heads":
        b, r, h, hkv, hd = case["b"], case["R"], case["H"], case["Hkv"], case["hd"]
        rows, out = b * r, DTYPES[case["out"]]
        # one projection's output: [rows][q | k | v]
        st["qkv"] = (2.0 * _normal(g, rows, (h + 2 * hkv) * hd)).to(dt)
        st["q"], st["k"], st["v"] = st["qkv"].split([h * hd, hkv * hd, hkv * hd], dim=1)
        st["w"] = [(1.0 + 0.2 * _normal(g, hd)).to(dt) for _ in range(2)]
        st["eps"] = 1e-6
        st["pos"] = (case["start"] + torch.arange(r, device="cuda").repeat(b)).to(torch.int32)
        st["q_out"] = torch.zeros(rows, h, hd, device="cuda", dtype=out)
        if case["paged"]:
            st["kv"], st["table"] = _pool(g, b, case["start"] + r, hkv, case["ps"], hd, out, False)
            st["starts"] = torch.full((b,), case["start"], device="cuda", dtype=torch.int32)
            counts = [r] * b
            counts[-1] -= case["pad"]
            st["counts"] = torch.tensor(counts, device="cuda", dtype=torch.int32)
        else:
            st["k_out"] = torch.zeros(rows, hkv, hd, device="cuda", dtype=out)
        if own:
            from cached_masked_decoding_gb300 import binding
            st["rope"] = binding.make_rope(case["rot"], layout=case["layout"], theta=case["theta"])
            if case["paged"]:
                st["cache"] = _cache(case, st["kv"], st["table"], case["ps"])
    elif kind == "attention":
        b, r, h, hkv, t, hd = case["b"], case["R"], case["H"], case["Hkv"], case["T"], case["hd"]
        st["kv"], st["table"] = _pool(g, b, t, hkv, case["ps"], hd, dt, True)
        st["q"] = (1.2 * _normal(g, b, r, h, hd)).to(dt)
        st["lens"] = torch.tensor(_lens(case), device="cuda", dtype=torch.int32)
        st["out"] = torch.empty(b, r, h, hd, device="cuda", dtype=dt)
        st["scale"] = 1.0 / math.sqrt(hd)
        # the weights of the steps before this one
        st["mass"] = torch.rand(b, hkv, t, generator=g, device="cuda") / 64 if case["mass"] else None
        if own:
            from cached_masked_decoding_gb300 import binding
            st["cache"] = _cache(case, st["kv"], st["table"], case["ps"])
            need = binding.attention_paged_workspace(b, h, hkv, hd, r, st["table"].shape[1] * case["ps"],
                                                     mass=case["mass"])
            st["ws"] = torch.empty(max(16, need), device="cuda", dtype=torch.uint8)
    elif kind == "evict":
        b, hkv, t, hd, keep = case["b"], case["Hkv"], case["T"], case["hd"], case["keep"]
        st["kv"], st["table"] = _pool(g, b, t, hkv, case["ps"], hd, dt, True)
        st["kv_out"], st["table_out"] = _pool(g, b, keep, hkv, case["ps_out"], hd, dt, False)
        # a few keys carry most of the weight, many have next to none, some none at all
        m = torch.exp(2.0 * _normal(g, b, hkv, t))
        st["mass"] = torch.where(torch.rand(b, hkv, t, generator=g, device="cuda") < 0.05, 0.0, m)
        st["mass_out"] = torch.zeros(b, hkv, keep, device="cuda")
        st["lens"] = torch.tensor(_lens(case), device="cuda", dtype=torch.int32)
        st["lens_out"] = torch.zeros(b, device="cuda", dtype=torch.int32)
        st["kept"] = torch.zeros(b, hkv, keep, device="cuda", dtype=torch.int32)
        if own:
            st["cache"] = _cache(case, st["kv"], st["table"], case["ps"])
            st["cache_out"] = _cache(case, st["kv_out"], st["table_out"], case["ps_out"])
    else:
        rows, vocab, top = case["rows"], case["vocab"], case["top"]
        # logits of a trained head are spread wide; rows from nearly sure to undecided
        buf = torch.empty(rows, vocab + case["pad"], device="cuda", dtype=dt)
        for part in buf.split(max(1, (1 << 27) // vocab)):
            part.copy_(_normal(g, *part.shape) * (1.0 + 4.0 * torch.rand(len(part), 1, generator=g, device="cuda")))
        st["logits"] = buf[:, :vocab]
        st["targets"] = torch.randint(0, vocab, (rows,), generator=g, device="cuda").to(torch.int32)
        st["logp"] = torch.empty(rows, device="cuda")
        st["entropy"] = torch.empty(rows, device="cuda")
        st["ids"] = torch.empty(rows, top, device="cuda", dtype=torch.int32)
        st["top"] = torch.empty(rows, top, device="cuda")
    return st


# --------------------------------------------------------------------------- one pass

def _heads_plain(st, x, w):
    """A head's norm, then its pairs turned: [rows][heads][hd] in 32 bits, the angles in 64."""
    case = st["case"]
    x = x.float().unflatten(1, (-1, case["hd"]))
    if case["norm"]:
        x = x * torch.rsqrt(x.square().mean(dim=-1, keepdim=True) + st["eps"]) * w.float()
    rot = case["rot"]
    f = case["theta"] ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    a = st["pos"].double()[:, None] * f
    c, s = a.cos().float()[:, None], a.sin().float()[:, None]
    if case["layout"] == "half":
        x0, x1, rest = x.split([rot // 2, rot // 2, case["hd"] - rot], dim=-1)
        return torch.cat([x0 * c - x1 * s, x1 * c + x0 * s, rest], dim=-1)
    x0, x1 = x[..., 0:rot:2], x[..., 1:rot:2]
    return torch.cat([torch.stack([x0 * c - x1 * s, x1 * c + x0 * s], dim=-1).flatten(-2), x[..., rot:]], dim=-1)


def _pages_plain(pool, table):
    """[b][H_kv][positions][hd] of a pool and a table."""
    return pool[table.long()].transpose(1, 2).flatten(2, 3)


def _run_plain(st):
    case = st["case"]
    kind = case["kind"]
    if kind == "heads":
        b, r, hkv, hd, ps = case["b"], case["R"], case["Hkv"], case["hd"], case["ps"]
        q, k = _heads_plain(st, st["q"], st["w"][0]), _heads_plain(st, st["k"], st["w"][1])
        if not case["paged"]:
            st["q_out"].copy_(q)
            st["k_out"].copy_(k)
            return st["q_out"], st["k_out"]
        i = torch.arange(r, device="cuda")
        there = (i < st["counts"][:, None]).flatten()
        st["q_out"].copy_(torch.where(there[:, None, None], q, st["q_out"].float()))
        at = (st["starts"][:, None] + i).long()
        page = torch.gather(st["table"].long(), 1, at // ps).flatten()[there]
        slot = (at % ps).flatten()[there]
        for pool, x in zip(st["kv"], (k, st["v"].float().unflatten(1, (hkv, hd)))):
            pool[page, :, slot] = x[there].to(pool.dtype)
        return st["q_out"], *st["kv"]
    if kind == "attention":
        b, r, h, hkv, t, hd = case["b"], case["R"], case["H"], case["Hkv"], case["T"], case["hd"]
        q = st["q"].float().view(b, r, hkv, h // hkv, hd).permute(0, 2, 3, 1, 4).reshape(b, hkv, -1, hd)
        k, v = (_pages_plain(x, st["table"])[:, :, :t].float() for x in st["kv"])
        sees = (torch.arange(t, device="cuda") < st["lens"][:, None])[:, None, None]
        z = torch.matmul(q, k.transpose(-1, -2)).mul_(st["scale"]).masked_fill_(~sees, -math.inf)
        top = z.amax(dim=-1, keepdim=True)
        z = z.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
        total = z.sum(dim=-1, keepdim=True)
        z = z.div_(torch.where(total == 0, 1.0, total))
        o = torch.matmul(z, v).view(b, hkv, h // hkv, r, hd).permute(0, 3, 1, 2, 4)
        st["out"].copy_(o.reshape(b, r, h, hd))
        if case["mass"]:
            st["mass"] += z.sum(dim=2)
        return st["out"], st["mass"]
    if kind == "evict":
        t, keep, ps = case["T"], case["keep"], case["ps_out"]
        at = torch.arange(t, device="cuda")
        n = st["lens"].long()[:, None, None]
        # whole numbers that order as (always kept, weight, lower position first) does
        always = (at < case["sinks"]) | (at >= n - case["recent"]) | (n <= keep)
        # (weights are no less than 0: their bits order as they do)
        rank = (st["mass"] + 0.0).view(torch.int32).long() | always.long() << 31
        rank = torch.where(at < n, rank << 31 | t - 1 - at, -1 - at)
        best = torch.topk(rank, min(keep, t), dim=-1).values
        kept = torch.where(best < 0, t + 1, t - 1 - (best & 0x7fffffff)).sort(dim=-1).values
        kept = torch.nn.functional.pad(kept, (0, keep - kept.shape[-1]), value=t + 1)
        there = kept < t
        st["kept"].copy_(torch.where(there, kept, -1))
        st["lens_out"].copy_(st["lens"].clamp(0, keep))
        kept = kept.clamp_max(t - 1)
        st["mass_out"].copy_(torch.where(there, st["mass"].gather(2, kept), st["mass_out"]))
        page_out = st["table_out"].long()[:, None, torch.arange(keep, device="cuda") // ps].expand_as(kept)
        s, g, i = there.nonzero(as_tuple=True)
        src = kept[s, g, i]
        page = st["table"].long()[s, src // case["ps"]]
        for pool, out in zip(st["kv"], st["kv_out"]):
            out[page_out[s, g, i], g, i % ps] = pool[page, g, src % case["ps"]]
        return {"k": st["kv_out"][0], "v": st["kv_out"][1], "kept": st["kept"], "mass": st["mass_out"],
                "lens": st["lens_out"]}
    vocab, top = case["vocab"], case["top"]
    x = st["logits"].float()
    z = x * (1.0 / case["temperature"])
    z = z - z.amax(dim=-1, keepdim=True)
    e = z.exp()
    total = e.sum(dim=-1, keepdim=True)
    log_total = total.log()
    st["entropy"].copy_((log_total - (e * z).sum(dim=-1, keepdim=True) / total)[:, 0])
    st["logp"].copy_((z.gather(1, st["targets"].long()[:, None]) - log_total)[:, 0])
    del e
    if top:
        # whole numbers that order as (logit, lower token first) does
        bits = (x + 0.0).view(torch.int32)
        rank = torch.where(bits < 0, bits ^ 0x7fffffff, bits).long() << 32
        rank |= vocab - 1 - torch.arange(vocab, device="cuda")
        ids = vocab - 1 - (torch.topk(rank, top, dim=-1).values & 0xffffffff)
        st["ids"].copy_(ids)
        st["top"].copy_(z.gather(1, ids) - log_total)
    return {"logp": st["logp"], "entropy": st["entropy"], "ids": st["ids"], "top": st["top"]}


def run(st):
    if not own:
        return _run_plain(st)
    from cached_masked_decoding_gb300 import binding
    case = st["case"]
    kind = case["kind"]
    stream = torch.cuda.current_stream().cuda_stream
    if kind == "heads":
        norm = {"q_weight_ptr": st["w"][0].data_ptr(), "k_weight_ptr": st["w"][1].data_ptr(), "eps": st["eps"]} \
            if case["norm"] else {"eps": -1.0}
        width = st["qkv"].shape[1]
        if case["paged"]:
            binding.op_qk_norm_rope_paged(st["cache"], st["q"].data_ptr(), st["k"].data_ptr(), st["v"].data_ptr(),
                                          st["q_out"].data_ptr(), case["H"], case["R"], case["dtype"],
                                          starts_ptr=st["starts"].data_ptr(), counts_ptr=st["counts"].data_ptr(),
                                          positions_ptr=st["pos"].data_ptr(), rope=st["rope"], q_row_stride=width,
                                          k_row_stride=width, v_row_stride=width, stream=stream, **norm)
            return st["q_out"], *st["kv"]
        binding.op_qk_norm_rope(st["q"].data_ptr(), st["k"].data_ptr(), st["q_out"].data_ptr(),
                                st["k_out"].data_ptr(), st["pos"].data_ptr(), case["b"] * case["R"], case["H"],
                                case["Hkv"], case["hd"], case["dtype"], out_dtype=case["out"], rope=st["rope"],
                                q_row_stride=width, k_row_stride=width, stream=stream, **norm)
        return st["q_out"], st["k_out"]
    if kind == "attention":
        mass = {"mass_ptr": st["mass"].data_ptr(), "mass_stride": case["T"]} if case["mass"] else {}
        binding.op_attention_paged(st["q"].data_ptr(), st["cache"], st["out"].data_ptr(), case["H"], case["R"],
                                   lens_ptr=st["lens"].data_ptr(), scale=st["scale"], ws_ptr=st["ws"].data_ptr(),
                                   ws_bytes=st["ws"].numel(), stream=stream, **mass)
        return st["out"], st["mass"]
    if kind == "evict":
        binding.op_kv_paged_evict(st["cache"], st["cache_out"], st["mass"].data_ptr(), case["keep"],
                                  st["kept"].data_ptr(), st["lens_out"].data_ptr(), lens_ptr=st["lens"].data_ptr(),
                                  sinks=case["sinks"], recent=case["recent"], mass_stride=case["T"],
                                  mass_out_ptr=st["mass_out"].data_ptr(), mass_out_stride=case["keep"],
                                  stream=stream)
        return {"k": st["kv_out"][0], "v": st["kv_out"][1], "kept": st["kept"], "mass": st["mass_out"],
                "lens": st["lens_out"]}
    top = case["top"]
    binding.op_token_logprobs(st["logits"].data_ptr(), case["dtype"], case["rows"], case["vocab"],
                              targets_ptr=st["targets"].data_ptr(), logprobs_ptr=st["logp"].data_ptr(),
                              entropy_ptr=st["entropy"].data_ptr(), top=top,
                              top_ids_ptr=st["ids"].data_ptr() if top else 0,
                              top_logprobs_ptr=st["top"].data_ptr() if top else 0,
                              inv_temperature=1.0 / case["temperature"], row_stride=case["vocab"] + case["pad"],
                              stream=stream)
    return {"logp": st["logp"], "entropy": st["entropy"], "ids": st["ids"], "top": st["top"]}


# --------------------------------------------------------------------------- work of one pass

def work(case):
    kind = case["kind"]
    if kind == "heads":
        rows = case["b"] * case["R"] - case["pad"]
        heads = case["H"] + case["Hkv"] * (2 if case["paged"] else 1)
        turned = rows * (case["H"] + case["Hkv"])
        return {"bytes": rows * heads * case["hd"] * (SIZES[case["dtype"]] + SIZES[case["out"]]) + 4 * rows,
                "flops": turned * (3 * case["rot"] + (4 * case["hd"] if case["norm"] else 0))}
    if kind == "attention":
        lens = _lens(case)
        keys = sum(lens)
        rows = sum(n > 0 for n in lens) * case["R"] * case["H"]
        return {"bytes": keys * case["Hkv"] * (4 * case["hd"] + (8 if case["mass"] else 0)) + 4 * rows * case["hd"],
                "flops": 4 * case["hd"] * case["H"] * case["R"] * keys}
    if kind == "evict":
        lens = _lens(case)
        n, kept = sum(lens) * case["Hkv"], sum(min(x, case["keep"]) for x in lens) * case["Hkv"]
        return {"bytes": 4 * n + kept * (8 * case["hd"] + 8), "flops": n}
    n = case["rows"] * case["vocab"]
    return {"bytes": n * SIZES[case["dtype"]] + case["rows"] * (12 + 8 * case["top"]), "flops": 6 * n}


# --------------------------------------------------------------------------- the definition, in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    kind = case["kind"]
    if kind == "heads":
        rot, hd, r = case["rot"], case["hd"], case["R"]
        rates = [math.exp(-math.log(case["theta"]) * 2 * i / rot) for i in range(rot // 2)]
        z = torch.polar(torch.ones(1, device="cuda", dtype=torch.float64),
                        torch.outer(st["pos"].double(), torch.tensor(rates, device="cuda", dtype=torch.float64)))
        outs = []
        for x, w in ((st["q"], st["w"][0]), (st["k"], st["w"][1])):
            x = x.double().reshape(len(x), -1, hd)
            if case["norm"]:
                x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / hd + st["eps"]) * w.double()
            part = x[..., :rot]
            pairs = part.unflatten(-1, (2, rot // 2)).transpose(-1, -2) if case["layout"] == "half" else \
                part.unflatten(-1, (rot // 2, 2))
            turned = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * z[:, None])
            if case["layout"] == "half":
                turned = turned.transpose(-1, -2)
            outs.append(torch.cat([turned.flatten(-2), x[..., rot:]], dim=-1))
        if not case["paged"]:
            return tuple(outs)
        q = outs[0]
        if case["pad"]:
            q[len(q) - case["pad"]:] = 0
        kv = [x.double() for x in st["kv"]]
        for s in range(case["b"]):
            n = r - (case["pad"] if s == case["b"] - 1 else 0)
            at = case["start"] + torch.arange(n, device="cuda")
            page, slot = st["table"][s, at // case["ps"]].long(), at % case["ps"]
            kv[0][page, :, slot] = outs[1][s * r:s * r + n]
            kv[1][page, :, slot] = st["v"][s * r:s * r + n].double().reshape(n, -1, hd)
        return q, *kv
    if kind == "attention":
        b, r, h, hkv, hd, ps = case["b"], case["R"], case["H"], case["Hkv"], case["hd"], case["ps"]
        if b * hkv > 1024:
            return None
        out = torch.zeros(b, r, h, hd, device="cuda", dtype=torch.float64)
        mass = st["mass"].double() if case["mass"] else None
        for s, n in enumerate(_lens(case)):
            if n == 0:
                continue
            pages = st["table"][s, :-(-n // ps)].long()
            for j in range(hkv):
                k, v = (x[pages, j].reshape(-1, hd)[:n].double() for x in st["kv"])
                for i in range(j * (h // hkv), (j + 1) * (h // hkv)):
                    p = torch.softmax((st["q"][s, :, i].double() @ k.t()) * st["scale"], dim=-1)
                    out[s, :, i] = p @ v
                    if case["mass"]:
                        mass[s, j, :n] += p.sum(0)
        return out, mass
    if kind == "evict":
        k, v = (x.double() for x in st["kv_out"])
        mass = st["mass_out"].double()
        for s, n in enumerate(_lens(case)):
            for j in range(case["Hkv"]):
                weight = st["mass"][s, j, :n].double()
                m = case["keep"]
                if n > m:
                    weight[:case["sinks"]] = math.inf
                    weight[n - case["recent"]:] = math.inf
                # a stable sort keeps equal weights in the order of their positions
                at = torch.sort(weight, descending=True, stable=True).indices[:m].sort().values
                page, slot = st["table"][s, at // case["ps"]].long(), at % case["ps"]
                i = torch.arange(len(at), device="cuda")
                to, to_slot = st["table_out"][s, i // case["ps_out"]].long(), i % case["ps_out"]
                k[to, j, to_slot] = st["kv"][0][page, j, slot].double()
                v[to, j, to_slot] = st["kv"][1][page, j, slot].double()
                mass[s, j, :len(at)] = st["mass"][s, j, at].double()
        return {"k": k, "v": v, "kept": None, "mass": mass, "lens": None}
    rows, vocab, top = case["rows"], case["vocab"], case["top"]
    outs = [torch.empty(rows, *w, device="cuda", dtype=torch.float64) for w in ((), (), (top,))]
    step = max(1, (1 << 26) // vocab)
    for r0 in range(0, rows, step):
        x = st["logits"][r0:r0 + step].double() / case["temperature"]
        lp = torch.log_softmax(x, dim=-1)
        outs[0][r0:r0 + step] = lp.gather(1, st["targets"][r0:r0 + step].long()[:, None])[:, 0]
        outs[1][r0:r0 + step] = -(lp.exp() * lp).sum(-1)
        if top:
            outs[2][r0:r0 + step] = torch.topk(lp, top, dim=-1).values
    return {"logp": outs[0], "entropy": outs[1], "ids": None, "top": outs[2]}
