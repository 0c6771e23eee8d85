"""The operators of paged decoding on the GPU against a plain 64-bit restatement (paged_ref): head norms with
positions and the cache's new rows, attention over the pages with the keys' weights, eviction, and what the logits
say - alone and in a run of all of them.

Tolerances count roundings: half a step is 2^-8 of the value in bf16, 2^-11 in f16, 2^-24 in float32.
"""
import math

import numpy as np
import pytest

import ops8_ref
import paged_ref as ref
from cached_masked_decoding_gb300 import binding
from gpu_util import torch_cuda

pytestmark = pytest.mark.gpu

HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TINY = {"f32": 0.0, "bf16": 0.0, "f16": 2.0 ** -25}      # half a subnormal step, where results may be that small
U = 2.0 ** -24


@pytest.fixture(scope="module")
def torch():
    t = torch_cuda()
    binding.lib()
    return t


def dt(torch, name):
    return {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[name]


def dev(torch, a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


def f64(t):
    return t.double().cpu().numpy()


class Pages:
    """A pool of poisoned pages and a table of random ones; rows are written by the test."""

    def __init__(self, torch, rng, b, hkv, hd, dtype, ps, most, spare=2, poison=math.nan):
        self.b, self.hkv, self.hd, self.dtype, self.ps, self.most = b, hkv, hd, dtype, ps, most
        self.pages = b * most + spare
        self.k, self.v = (torch.full((self.pages, hkv, ps, hd), poison, device="cuda", dtype=dt(torch, dtype))
                          for _ in range(2))
        self.tab = rng.permutation(self.pages)[:b * most].reshape(b, most).astype(np.int32)
        self.torch = torch

    def fill(self, rng, lens, kscale=1.0, vscale=1.0):
        """Values for the first lens[s] positions; what lies behind them stays poisoned."""
        for s, n in enumerate(lens):
            for pool, scale in ((self.k, kscale), (self.v, vscale)):
                x = dev(self.torch, (scale * rng.standard_normal((n, self.hkv, self.hd))).astype(np.float32))
                t = np.arange(n)
                page, slot = (self.torch.from_numpy(a).cuda() for a in
                              (self.tab[s, t // self.ps].astype(np.int64), (t % self.ps).astype(np.int64)))
                pool[page, :, slot] = x.to(pool.dtype)
        return self

    def struct(self):
        self.table = dev(self.torch, self.tab)
        return binding.make_kv_paged(self.k.data_ptr(), self.v.data_ptr(), self.table.data_ptr(), self.b, self.hkv,
                                     self.hd, self.dtype, self.pages, self.ps, self.most)


# --------------------------------------------------------------------------- head norms, positions, new rows

def _heads_check(got, x, w, eps, pos, rot, layout, rates, amp, out_dtype):
    want = ref.norm_rope(x, w, eps, pos, rot, layout, rates, amp)
    y = np.abs(ref.norm_rope(x, w, eps, pos, rot, layout, None))
    other = np.zeros_like(y)
    if rates is not None:                               # the pair's other member
        i0 = np.arange(rot // 2) if layout == "half" else 2 * np.arange(rot // 2)
        i1 = i0 + (rot // 2 if layout == "half" else 1)
        other[..., i0], other[..., i1] = y[..., i1], y[..., i0]
    # mean: a sum of hd squares (a tree of at most hd / 2 roundings), its root and quotient 4, two products;
    # cosine and sine 3 roundings, the amplitude's, a product and a fused sum: 8; the angle as dllm_op_rope's
    c = (x.shape[-1] / 2 + 6 if eps >= 0 else 0) + (8 if rates is not None else 0)
    angle = np.abs(pos.astype(np.float64)).max() * 2.0 ** -49 if rates is not None else 0.0
    tol = (c * U + angle) * (y + other) * amp + HALF[out_dtype] * 1.01 * np.abs(want) + TINY[out_dtype]
    assert (np.abs(got - want) <= tol).all(), float((np.abs(got - want) / np.maximum(tol, 1e-300)).max())


HEADS = [
    # rows, H, H_kv, hd, rot, layout, eps, weights, in, out, padding of rows
    (1, 1, 1, 16, 16, "half", 1e-6, True, "bf16", "bf16", 0),
    (3, 4, 2, 64, 32, "interleaved", 1e-5, True, "f16", "f16", 8),
    (37, 32, 8, 128, 128, "half", 1e-6, True, "bf16", "bf16", 16),
    (5, 3, 1, 96, 48, "half", 0.0, True, "f32", "bf16", 4),
    (130, 7, 7, 80, 80, "interleaved", 1e-6, False, "f32", "f32", 0),
    (9, 2, 2, 256, 64, "half", 1e-6, True, "f32", "f16", 0),
    (2, 90, 10, 128, 16, "half", 1e-6, True, "bf16", "bf16", 0),
    (66, 1, 1, 32, 32, "interleaved", -1.0, False, "bf16", "bf16", 0),
    (11, 2, 1, 48, 0, "half", 1e-6, True, "f16", "f16", 0),
    (4, 6, 2, 64, 0, "half", -1.0, False, "f32", "bf16", 0),
]


@pytest.mark.parametrize("rows,H,Hkv,hd,rot,layout,eps,weights,dtype,out,pad", HEADS)
def test_qk_norm_rope(torch, rows, H, Hkv, hd, rot, layout, eps, weights, dtype, out, pad):
    rng = np.random.default_rng(rows * H + hd)
    D = dt(torch, dtype)
    width = (H + 2 * Hkv) * hd + pad
    buf = dev(torch, (2.0 * rng.standard_normal((rows, width))).astype(np.float32)).to(D)
    q, k = buf[:, :H * hd], buf[:, H * hd:(H + Hkv) * hd]
    w = [dev(torch, (1 + 0.3 * rng.standard_normal(hd)).astype(np.float32)).to(D) if weights else None for _ in range(2)]
    pos = np.concatenate([rng.integers(0, 1 << 20, rows - 1), [0x7fffffff]]).astype(np.int32)
    pos[0] = -5
    p = dev(torch, pos)
    wide = H * hd + (pad + 7) // 8 * 8                     # (16 bytes of either type)
    qo = torch.full((rows, wide), 7.0, device="cuda", dtype=dt(torch, out))
    ko = torch.full((rows, Hkv * hd + 16), 7.0, device="cuda", dtype=dt(torch, out))
    spec = binding.make_rope(rot, layout=layout, theta=5e5, scaling="by_parts", factor=4.0) if rot else None
    binding.op_qk_norm_rope(q.data_ptr(), k.data_ptr(), qo.data_ptr(), ko.data_ptr(), p.data_ptr() if rot else 0, rows, H,
                            Hkv, hd, dtype, out_dtype=out, q_weight_ptr=w[0].data_ptr() if weights else 0,
                            k_weight_ptr=w[1].data_ptr() if weights else 0, eps=eps, rope=spec, q_row_stride=width,
                            k_row_stride=width, q_out_row_stride=wide, k_out_row_stride=Hkv * hd + 16)
    rates, amp = ops8_ref.rope_rates(rot, 5e5, "by_parts", 4.0) if rot else (None, 1.0)
    for x, n, o, ww in ((q, H, qo, w[0]), (k, Hkv, ko, w[1])):
        _heads_check(f64(o[:, :n * hd]).reshape(rows, n, hd), f64(x).reshape(rows, n, hd),
                     f64(ww) if weights else None, eps, pos, rot, layout, rates, amp, out)
        assert (o[:, n * hd:] == 7.0).all()


def test_qk_norm_rope_in_place_and_empty_heads(torch):
    rng = np.random.default_rng(3)
    x = dev(torch, rng.standard_normal((33, 6, 128)).astype(np.float32)).to(torch.bfloat16)
    x[4, 2] = 0                                           # a head of zeros stays one (eps keeps it from a NaN)
    x[5, 5] = float("inf")
    before = f64(x)
    pos = dev(torch, np.arange(33, dtype=np.int32))
    q, k = x[:, :4], x[:, 4:]
    binding.op_qk_norm_rope(q.data_ptr(), k.data_ptr(), q.data_ptr(), k.data_ptr(), pos.data_ptr(), 33, 4, 2, 128, "bf16",
                            rope=binding.make_rope(128), q_row_stride=768, k_row_stride=768, q_out_row_stride=768,
                            k_out_row_stride=768)
    got = f64(x)
    assert (got[4, 2] == 0).all() and np.isnan(got[5, 5]).all()
    rates, amp = ops8_ref.rope_rates(128, 1e4, "none", 1.0)
    fine = [i for i in range(33) if i != 5]
    _heads_check(got[fine], before[fine], None, 1e-6, np.array(fine), 128, "half", rates, amp, "bf16")


@pytest.mark.parametrize("dtype,cache_dtype,hd,ps,b,R,H,Hkv", [
    ("bf16", "bf16", 128, 16, 3, 1, 8, 2), ("f32", "f16", 64, 32, 2, 37, 4, 4), ("f16", "f16", 128, 256, 1, 300, 2, 1),
    ("f32", "bf16", 64, 64, 5, 7, 3, 3), ("bf16", "bf16", 64, 128, 2, 130, 16, 2)])
def test_rows_go_to_their_pages(torch, dtype, cache_dtype, hd, ps, b, R, H, Hkv):
    rng = np.random.default_rng(b * R + hd)
    starts = np.array([0, ps - 1, 3 * ps + 5, 17, ps][:b], dtype=np.int32)
    most = int(-(-(starts.max() + R) // ps)) + 1
    c = Pages(torch, rng, b, Hkv, hd, cache_dtype, ps, most, poison=5.0)
    counts = np.array([R, max(0, R - 3), R, 0, R + 9][:b], dtype=np.int32)
    if b > 2:
        starts[2] = most * ps - 1                         # the table ends inside the rows (or with the first)
    if b > 4:
        starts[4] = -2                                    # and begins inside
    if R > 100:
        c.tab[0, 1] = -1 if b == 1 else c.pages           # a row's page that is none
    D = dt(torch, dtype)
    q, k, v = (dev(torch, rng.standard_normal((b * R, n * hd)).astype(np.float32)).to(D) for n in (H, Hkv, Hkv))
    w = [dev(torch, (1 + 0.3 * rng.standard_normal(hd)).astype(np.float32)).to(D) for _ in range(2)]
    qo = torch.full((b * R, H, hd), 9.0, device="cuda", dtype=dt(torch, cache_dtype))
    st, ct = dev(torch, starts), dev(torch, counts)
    spec = binding.make_rope(hd, theta=1e6)
    binding.op_qk_norm_rope_paged(c.struct(), q.data_ptr(), k.data_ptr(), v.data_ptr(), qo.data_ptr(), H, R, dtype,
                                  starts_ptr=st.data_ptr(), counts_ptr=ct.data_ptr(), q_weight_ptr=w[0].data_ptr(),
                                  k_weight_ptr=w[1].data_ptr(), eps=1e-6, rope=spec)
    rates, amp = ops8_ref.rope_rates(hd, 1e6, "none", 1.0)
    kp, vp, qn = f64(c.k), f64(c.v), f64(qo)
    untouched = np.ones(kp.shape[:1] + (ps,), dtype=bool)
    rows, where = [], []
    for s in range(b):
        for i in range(R):
            at = int(starts[s]) + i
            page = c.tab[s, at // ps] if 0 <= at < most * ps else -1
            if i < counts[s] and 0 <= page < c.pages:
                rows.append(s * R + i)
                where.append((int(page), at % ps, at))
                untouched[page, at % ps] = False
            else:
                assert (qn[s * R + i] == 9.0).all()
    assert rows and len(rows) < b * R or b == 1 or R == 1
    pg, sl, at = (np.array(a) for a in zip(*where))
    shape = (len(rows), -1, hd)
    _heads_check(qn[rows], f64(q)[rows].reshape(shape), f64(w[0]), 1e-6, at, hd, "half", rates, amp, cache_dtype)
    _heads_check(kp[pg, :, sl], f64(k)[rows].reshape(shape), f64(w[1]), 1e-6, at, hd, "half", rates, amp, cache_dtype)
    want = f64(v.to(dt(torch, cache_dtype)))[rows].reshape(shape)
    np.testing.assert_array_equal(vp[pg, :, sl], want)
    for pool in (kp, vp):
        assert (pool.transpose(0, 2, 1, 3)[untouched] == 5.0).all()


def test_rows_are_stored_as_they_are(torch):
    """No norm, nothing turns: a plain store, with positions that play no part."""
    rng = np.random.default_rng(5)
    c = Pages(torch, rng, 2, 3, 64, "bf16", 16, 4, poison=0.0)
    k, v, q = (dev(torch, rng.standard_normal((2 * 20, n * 64)).astype(np.float32)).to(torch.bfloat16) for n in (3, 3, 3))
    qo = torch.zeros_like(q)
    binding.op_qk_norm_rope_paged(c.struct(), q.data_ptr(), k.data_ptr(), v.data_ptr(), qo.data_ptr(), 3, 20, "bf16",
                                  eps=-1.0)
    assert torch.equal(q, qo)
    for pool, x in ((c.k, k), (c.v, v)):
        for s in range(2):
            rows, _ = ref.gather(f64(pool), c.tab[s], 20, 16)
            np.testing.assert_array_equal(rows.transpose(1, 0, 2).reshape(20, -1), f64(x)[s * 20:(s + 1) * 20])


# --------------------------------------------------------------------------- attention over the pages

def attend(torch, c, q, lens, scale=None, mass=None, out=None, stream=0, ws=None, **strides):
    b, R, H, hd = q.shape
    st = c.struct()
    need = binding.attention_paged_workspace(b, H, c.hkv, hd, R, c.most * c.ps, mass=mass is not None)
    if ws is None:
        ws = torch.full((need + 16,), 0xff, device="cuda", dtype=torch.uint8)
    out = torch.full((b, R, H, hd), 3.0, device="cuda", dtype=q.dtype) if out is None else out
    ln = dev(torch, np.asarray(lens, dtype=np.int32)) if lens is not None else None
    m = dict(mass_ptr=mass.data_ptr(), mass_stride=mass.shape[2]) if mass is not None else {}
    binding.op_attention_paged(q.data_ptr(), st, out.data_ptr(), H, R, lens_ptr=ln.data_ptr() if ln is not None else 0,
                               scale=scale, ws_ptr=ws.data_ptr(), ws_bytes=need, stream=stream, **m, **strides)
    torch.cuda.synchronize()
    binding.op_check()
    return out


def attention_check(c, q, lens, out, scale=None, mass=None, before=None):
    b, R, H, hd = q.shape
    scale = hd ** -0.5 if scale is None else scale
    kp, vp = f64(c.k), f64(c.v)
    worst = 0.0
    for s in range(b):
        n = min(max(int(lens[s]), 0), c.most * c.ps)
        k, there = ref.gather(kp, c.tab[s], n, c.ps)
        v, _ = ref.gather(vp, c.tab[s], n, c.ps)
        want, m, pv, sv, sk = ref.attention(f64(q[s]), k, v, there, scale)
        # a score: a float32 sum of hd exact products (each within 2^-23 of the sum of their sizes, the tensor core
        # truncates), scaled and put against its reference: 4 roundings of it; p = 2^z within 2^-22
        dz = (hd + 8) * 2.0 ** -23 * sk + 2.0 ** -22
        # p in two halves: 2^-16 of it (bf16), 2^-20 of it or 2^-25 of the largest (f16); sums of n terms in trees
        # and tiles, on both sides of the quotient
        halves = 2.0 ** -16 * pv if c.dtype == "bf16" else 2.0 ** -20 * pv + 2.0 ** -25 * sv
        tol = (2 * dz + (n / 16 + 24) * U) * pv + halves + HALF[c.dtype] * 1.01 * np.abs(want) + TINY[c.dtype]
        err = np.abs(f64(out[s]) - want)
        assert (err <= tol).all(), (s, float((err / np.maximum(tol, 1e-300)).max()))
        if mass is not None:
            G = H // c.hkv
            dzm = float(dz.max())
            mt = np.full(m.shape, (R * G + 4) * U)
            got, old = f64(mass[s])[:, :n], before[s][:, :n]
            w = min(n, mass.shape[2])
            tol = m[:, :w] * (2 * dzm + (n / 16 + 40) * U) + mt[:, :w] * (np.abs(old[:, :w]) + m[:, :w]) + 1e-37
            assert (np.abs(got - (old + m[:, :w])) <= tol).all(), s
            np.testing.assert_array_equal(f64(mass[s])[:, n:], before[s][:, n:])
    return worst


SHAPES = [
    # b, R, H, H_kv, hd, page, lens, dtype
    (1, 1, 1, 1, 64, 16, [1], "bf16"),
    (1, 1, 8, 1, 128, 16, [127], "f16"),
    (3, 1, 8, 8, 64, 32, [128, 0, 129], "bf16"),
    (2, 1, 32, 8, 128, 64, [1000, 257], "bf16"),
    (2, 1, 10, 2, 128, 128, [300, 16], "f16"),
    (1, 3, 6, 2, 64, 256, [700], "f16"),
    (2, 17, 4, 4, 128, 16, [400, 33], "bf16"),
    (1, 32, 4, 1, 64, 16, [513], "bf16"),
    (2, 32, 8, 8, 128, 32, [768, 512], "bf16"),
    (1, 70, 6, 2, 128, 64, [260], "f16"),
    (1, 1, 64, 1, 128, 16, [3000], "bf16"),
    (5, 2, 12, 4, 64, 16, [2049, 1, 0, -3, 900], "bf16"),
    (1, 1, 4, 4, 128, 16, [4100], "bf16"),
    (1, 1, 8, 1, 64, 256, [30000], "bf16"),              # a part in every CTA
    (1, 5, 3, 1, 128, 64, [2500], "f16"),
    (70, 1, 2, 2, 64, 16, [(7 * i * i) % 650 - 20 for i in range(70)], "bf16"),
    (45, 1, 4, 2, 64, 32, [(11 * i) % 420 for i in range(45)], "f16"),
]


@pytest.mark.parametrize("with_mass", [False, True])
@pytest.mark.parametrize("b,R,H,Hkv,hd,ps,lens,dtype", SHAPES, ids=lambda v: str(v)[:24])
def test_attention_paged(torch, b, R, H, Hkv, hd, ps, lens, dtype, with_mass):
    rng = np.random.default_rng(b * 100 + R + H + lens[0])
    most = -(-max(lens) // ps) + 1
    c = Pages(torch, rng, b, Hkv, hd, dtype, ps, most).fill(rng, [max(0, n) for n in lens])
    q = dev(torch, (1.5 * rng.standard_normal((b, R, H, hd))).astype(np.float32)).to(dt(torch, dtype))
    mass = before = None
    if with_mass:
        mass = dev(torch, rng.random((b, Hkv, most * ps)).astype(np.float32))
        before = f64(mass)
    out = attend(torch, c, q, lens, mass=mass)
    attention_check(c, q, lens, out, mass=mass, before=before)


def test_attention_sees_what_the_table_holds(torch):
    """No lens, lens over the table, table entries past the last page that name no page, and pages that two sequences
    share."""
    rng = np.random.default_rng(0)
    c = Pages(torch, rng, 2, 2, 64, "bf16", 16, 9).fill(rng, [144, 144])
    q = dev(torch, rng.standard_normal((2, 1, 4, 64)).astype(np.float32)).to(torch.bfloat16)
    full = attend(torch, c, q, None)
    attention_check(c, q, [144, 144], full)
    assert torch.equal(attend(torch, c, q, [145, 0x7fffffff]), full)
    c.tab[1, :5] = c.tab[0, :5]
    c.tab[1, 6:] = 0x7fffffff
    out = attend(torch, c, q, [144, 96])
    attention_check(c, q, [144, 96], out)


@pytest.mark.parametrize("hd,ps", [(64, 16), (128, 64), (128, 256)])
def test_attention_leaves_out_positions_on_no_page(torch, hd, ps):
    rng = np.random.default_rng(hd + ps)
    most = 1024 // ps
    c = Pages(torch, rng, 3, 2, hd, "bf16", ps, most).fill(rng, [1024, 1000, 1024])
    c.tab[0, 0] = -1
    c.tab[1, most // 2] = c.pages
    c.tab[2, :] = -7                                      # nothing to see at all
    q = dev(torch, rng.standard_normal((3, 2, 4, hd)).astype(np.float32)).to(torch.bfloat16)
    mass = torch.zeros(3, 2, 1024, device="cuda")
    out = attend(torch, c, q, [1024, 1000, 1024], mass=mass)
    attention_check(c, q, [1024, 1000, 1024], out, mass=mass, before=np.zeros((3, 2, 1024)))
    assert (out[2] == 0).all() and (mass[2] == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("rise", [3.0, 30.0, 300.0])
def test_attention_references_follow_the_scores(torch, dtype, rise):
    """Scores that climb along the cache, far past what the first keys had, and fall again: the probabilities meet
    the largest anywhere in a tile, at its ends and across splits."""
    rng = np.random.default_rng(int(rise))
    n, hd = 2500, 64
    c = Pages(torch, rng, 1, 1, hd, dtype, 16, 160).fill(rng, [n])
    t = np.arange(n)
    level = rise * np.maximum(0, 1 - np.abs(t - 1700) / 900.0)      # in units of the score
    u = np.zeros(hd, dtype=np.float32)
    u[0] = 8.0
    pg = torch.from_numpy(c.tab[0, t // 16].astype(np.int64)).cuda()
    c.k[pg, 0, torch.from_numpy(t % 16).cuda()] += dev(torch, (level[:, None] * u / 8.0).astype(np.float32)).to(c.k.dtype)
    q = dev(torch, (0.3 * rng.standard_normal((1, 2, 3, hd)) + u).astype(np.float32)).to(dt(torch, dtype))
    mass = torch.zeros(1, 1, 2560, device="cuda")
    out = attend(torch, c, q, [n], mass=mass)
    attention_check(c, q, [n], out, mass=mass, before=np.zeros((1, 1, 2560)))


def test_attention_strides_scale_and_short_mass(torch):
    rng = np.random.default_rng(9)
    lens, H, Hkv, hd = [333, 90], 6, 3, 64
    c = Pages(torch, rng, 2, Hkv, hd, "f16", 32, 11).fill(rng, lens)
    buf = dev(torch, rng.standard_normal((2, 5, H * hd + 40)).astype(np.float32)).to(torch.float16)
    out = torch.full((2, 5, H * hd + 8), 3.0, device="cuda", dtype=torch.float16)
    mass = torch.ones(2, Hkv, 100, device="cuda")         # shorter than the first sequence: the rest is not added
    q = buf[..., :H * hd].reshape(2, 5, H, hd)
    attend(torch, c, torch.as_strided(buf, (2, 5, H, hd), (5 * (H * hd + 40), H * hd + 40, hd, 1)), lens, scale=0.3,
           mass=mass, out=out, q_row_stride=H * hd + 40, out_row_stride=H * hd + 8)
    attention_check(c, q, lens, out[..., :H * hd].reshape(2, 5, H, hd), scale=0.3)
    assert (out[..., H * hd:] == 3.0).all()
    for s in range(2):
        n = lens[s]
        k, there = ref.gather(f64(c.k), c.tab[s], n, 32)
        _, m, _, _, sk = ref.attention(f64(q[s]), k, k, there, 0.3)
        w = min(n, 100)
        tol = 1e-6 + m[:, :w] * (2 * (hd + 8) * 2.0 ** -23 * sk.max() + 1e-5)
        assert (np.abs(f64(mass[s])[:, :w] - 1 - m[:, :w]) <= tol).all()
        assert (mass[s][:, w:] == 1.0).all()


def test_attention_is_repeatable_and_leaves_other_rows(torch):
    rng = np.random.default_rng(4)
    lens = [5000, 4000, 77]
    c = Pages(torch, rng, 3, 2, 128, "bf16", 16, 313).fill(rng, lens)
    q = dev(torch, rng.standard_normal((3, 1, 8, 128)).astype(np.float32)).to(torch.bfloat16)
    out = torch.full((5, 1, 8, 128), 3.0, device="cuda", dtype=torch.bfloat16)
    m0 = torch.zeros(3, 2, 5008, device="cuda")
    a = attend(torch, c, q, lens, mass=m0, out=out).clone()
    assert (a[3:] == 3.0).all()
    for _ in range(3):
        m = torch.zeros(3, 2, 5008, device="cuda")
        b = attend(torch, c, q, lens, mass=m, out=out)
        assert torch.equal(a, b) and torch.equal(m, m0)


def test_attention_in_a_large_pool(torch):
    """Pages whose bytes and elements lie past 2^32 and 2^31."""
    rng = np.random.default_rng(8)
    ps, hkv, hd = 256, 8, 128
    pages = (1 << 31) // (ps * hkv * hd) + 6
    c = Pages.__new__(Pages)
    c.b, c.hkv, c.hd, c.dtype, c.ps, c.most, c.pages, c.torch = 1, hkv, hd, "bf16", ps, 2, pages, torch
    c.k, c.v = (torch.empty(pages, hkv, ps, hd, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    c.tab = np.array([[pages - 1, pages - 3]], dtype=np.int32)
    c.fill(rng, [300])
    q = dev(torch, rng.standard_normal((1, 1, 16, hd)).astype(np.float32)).to(torch.bfloat16)
    out = attend(torch, c, q, [300])
    k, v = c.k, c.v
    c.k, c.v = k[-4:], v[-4:]                             # (the reference needs the last pages only)
    c.tab, c.pages = np.array([[3, 1]], dtype=np.int32), 4
    attention_check(c, q, [300], out)
    c.k, c.v, c.pages = k, v, pages
    c.tab = np.array([[pages - 1, pages - 3]], dtype=np.int32)
    x = dev(torch, rng.standard_normal((4, hkv * hd)).astype(np.float32)).to(torch.bfloat16)
    qo = torch.zeros(4, hkv * hd, device="cuda", dtype=torch.bfloat16)
    st = dev(torch, np.array([254], dtype=np.int32))
    binding.op_qk_norm_rope_paged(c.struct(), x.data_ptr(), x.data_ptr(), x.data_ptr(), qo.data_ptr(), hkv, 4, "bf16",
                                  starts_ptr=st.data_ptr(), eps=-1.0)
    assert torch.equal(c.k[pages - 1, :, 254:].transpose(0, 1).reshape(2, -1), x[:2])
    assert torch.equal(c.v[pages - 3, :, :2].transpose(0, 1).reshape(2, -1), x[2:])


def test_attention_refuses_a_small_workspace(torch):
    rng = np.random.default_rng(2)
    c = Pages(torch, rng, 1, 2, 64, "bf16", 16, 64).fill(rng, [1000])
    q = torch.zeros(1, 1, 4, 64, device="cuda", dtype=torch.bfloat16)
    need = binding.attention_paged_workspace(1, 4, 2, 64, 1, 1024)
    assert 0 < need < binding.attention_paged_workspace(1, 4, 2, 64, 1, 1024, mass=True)
    ws = torch.empty(need + 16, device="cuda", dtype=torch.uint8)
    for args in [dict(), dict(ws_ptr=ws.data_ptr(), ws_bytes=need - 1), dict(ws_ptr=ws.data_ptr() + 8, ws_bytes=need)]:
        with pytest.raises(binding.DllmError) as e:
            binding.op_attention_paged(q.data_ptr(), c.struct(), q.data_ptr(), 4, 1, **args)
        assert e.value.status == binding.EINVAL and "workspace" in str(e.value)


def test_attention_on_two_streams_at_once(torch):
    """Calls that run at the same time, each with a workspace of its own: the bits of calls one after the other."""
    rng = np.random.default_rng(14)
    lens = [3000, 1234, 0, 4000]
    cs = [Pages(torch, rng, 4, 2, 128, "bf16", 32, 126).fill(rng, lens) for _ in range(2)]
    q = dev(torch, rng.standard_normal((4, 2, 8, 128)).astype(np.float32)).to(torch.bfloat16)
    ln = dev(torch, np.array(lens, dtype=np.int32))
    ws = [torch.empty(binding.attention_paged_workspace(4, 8, 2, 128, 2, 4032, mass=True), device="cuda",
                      dtype=torch.uint8) for _ in range(2)]
    want, want_m = [], []
    for c in cs:
        m = torch.zeros(4, 2, 4032, device="cuda")
        want.append(attend(torch, c, q, lens, mass=m))
        want_m.append(m)
    structs = [c.struct() for c in cs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.empty_like(q) for _ in range(2)]
    ms = [torch.zeros(4, 2, 4032, device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                ms[i].zero_()
                binding.op_attention_paged(q.data_ptr(), structs[i], outs[i].data_ptr(), 8, 2, lens_ptr=ln.data_ptr(),
                                           mass_ptr=ms[i].data_ptr(), ws_ptr=ws[i].data_ptr(), ws_bytes=ws[i].numel(),
                                           stream=streams[i].cuda_stream)
    torch.cuda.synchronize()
    binding.op_check()
    for i in range(2):
        assert torch.equal(outs[i], want[i]) and torch.equal(ms[i], want_m[i])


# --------------------------------------------------------------------------- eviction

def evict(torch, src, dst, mass, lens, keep, sinks, recent, mass_out=None, stream=0):
    b, hkv = src.b, src.hkv
    kept = torch.full((b, hkv, keep), -9, device="cuda", dtype=torch.int32)
    nl = torch.full((b,), -9, device="cuda", dtype=torch.int32)
    ln = dev(torch, np.asarray(lens, dtype=np.int32)) if lens is not None else None
    binding.op_kv_paged_evict(src.struct(), dst.struct(), mass.data_ptr(), keep, kept.data_ptr(), nl.data_ptr(),
                              lens_ptr=ln.data_ptr() if ln is not None else 0, sinks=sinks, recent=recent,
                              mass_stride=mass.shape[2],
                              mass_out_ptr=mass_out.data_ptr() if mass_out is not None else 0,
                              mass_out_stride=mass_out.shape[2] if mass_out is not None else 0, stream=stream)
    torch.cuda.synchronize()
    return kept, nl


EVICT = [
    # b, H_kv, hd, pages in and out, lens, keep, sinks, recent, dtype, weights
    (1, 1, 64, 16, 16, [1], 1, 0, 0, "bf16", "random"),
    (2, 3, 128, 16, 64, [100, 40], 41, 4, 8, "f16", "random"),
    (3, 2, 64, 32, 16, [1025, 0, 700], 256, 0, 0, "bf16", "equal"),
    (1, 2, 128, 64, 32, [2000], 500, 0, 500, "bf16", "random"),
    (1, 2, 128, 64, 32, [2000], 500, 500, 0, "bf16", "random"),
    (2, 2, 64, 16, 16, [333, 512], 300, 100, 200, "f16", "random"),
    (1, 4, 128, 256, 128, [4100], 4099, 1, 1, "bf16", "few"),
    (2, 1, 64, 16, 16, [900, 33], 65, 2, 3, "bf16", "nan"),
    (1, 2, 64, 128, 256, [40000], 5000, 4, 1000, "bf16", "few"),
    (1, 1, 64, 128, 256, [70001], 64, 0, 0, "bf16", "random"),
    (2, 2, 64, 16, 16, [50, 20], 64, 4, 4, "bf16", "random"),
    # the least kept is a NaN; weights of one leading part, few, many and too many to be listed; ends of what is held
    (1, 2, 64, 16, 16, [900], 400, 2, 3, "bf16", "nan"),
    (2, 2, 64, 16, 16, [128, 129], 100, 0, 7, "bf16", "band"),
    (2, 1, 64, 16, 16, [2048, 2049], 777, 1, 0, "bf16", "band"),
    (2, 1, 64, 128, 128, [8192, 8193], 4096, 0, 9, "f16", "band"),
    (2, 1, 64, 256, 128, [49152, 49153], 3000, 4, 5, "bf16", "band"),
    (2, 1, 64, 256, 128, [49152, 49153], 3000, 4, 5, "bf16", "random"),
    (1, 1, 64, 256, 256, [49160], 49153, 0, 0, "bf16", "few"),
]


@pytest.mark.parametrize("b,Hkv,hd,ps,ps2,lens,keep,sinks,recent,dtype,weights", EVICT)
def test_evict(torch, b, Hkv, hd, ps, ps2, lens, keep, sinks, recent, dtype, weights):
    rng = np.random.default_rng(sum(lens) + keep)
    most, most2 = -(-max(lens) // ps), -(-keep // ps2)
    src = Pages(torch, rng, b, Hkv, hd, dtype, ps, most).fill(rng, lens)
    dst = Pages(torch, rng, b, Hkv, hd, dtype, ps2, most2, poison=5.0)
    m = np.exp(2 * rng.standard_normal((b, Hkv, max(lens) + 3))).astype(np.float32)
    if weights == "equal":
        m[:] = 0.25
    if weights == "band":
        m = rng.uniform(1.0, 1.1, m.shape).astype(np.float32)
    if weights == "few":                                  # many ties, zeros of both signs among them
        m = rng.choice(np.array([0.0, -0.0, 0.5, 1.0, 1e-42], dtype=np.float32), m.shape)
    if weights == "nan":
        m[rng.random(m.shape) < 0.9] = np.nan
        m[rng.random(m.shape) < 0.05] = -np.inf
        m[rng.random(m.shape) < 0.05] = np.inf
        m[rng.random(m.shape) < 0.05] = -1.0
    mass = dev(torch, m)
    out = torch.full((b, Hkv, keep + 2), 7.0, device="cuda")
    kept, nl = evict(torch, src, dst, mass, lens, keep, sinks, recent, mass_out=out)
    kept, nl, out = kept.cpu().numpy(), nl.cpu().numpy(), out.cpu().numpy()
    for s in range(b):
        n = min(lens[s], keep)
        assert nl[s] == n
        sk, _ = ref.gather(f64(src.k), src.tab[s], lens[s], ps)
        sv, _ = ref.gather(f64(src.v), src.tab[s], lens[s], ps)
        dk, _ = ref.gather(f64(dst.k), dst.tab[s], n, ps2)
        dv, _ = ref.gather(f64(dst.v), dst.tab[s], n, ps2)
        for g in range(Hkv):
            want = ref.kept(m[s, g], lens[s], keep, sinks, recent)
            np.testing.assert_array_equal(kept[s, g, :n], want)
            assert (kept[s, g, n:] == -1).all()
            np.testing.assert_array_equal(out[s, g, :n], m[s, g, want])
            assert (out[s, g, n:] == 7.0).all()
            np.testing.assert_array_equal(dk[g], sk[g, want])
            np.testing.assert_array_equal(dv[g], sv[g, want])
    # slots behind the kept rows, and pages of nobody, stay as they were
    written = np.zeros((dst.pages, ps2), dtype=bool)
    for s in range(b):
        t = np.arange(min(lens[s], keep))
        written[dst.tab[s, t // ps2], t % ps2] = True
    for pool in (dst.k, dst.v):
        assert (f64(pool).transpose(0, 2, 1, 3)[~written] == 5.0).all()


def test_evict_pages_that_are_none_and_the_ends_of_lens(torch):
    rng = np.random.default_rng(6)
    src = Pages(torch, rng, 2, 2, 64, "bf16", 16, 8).fill(rng, [128, 128])
    dst = Pages(torch, rng, 2, 2, 64, "bf16", 16, 3, poison=5.0)
    src.tab[0, 2] = -1
    dst.tab[1, 1] = dst.pages
    m = rng.random((2, 2, 100)).astype(np.float32)        # mass ends before the table: so do the positions
    m[0, :, 32:48] += 10                                  # the missing page's keys are heavy
    kept, nl = evict(torch, src, dst, dev(torch, m), None, 48, 0, 0)
    assert nl.tolist() == [48, 48]
    for s in range(2):
        sk, _ = ref.gather(f64(src.k), src.tab[s], 100, 16)
        dk, there = ref.gather(f64(dst.k), dst.tab[s], 48, 16)
        for g in range(2):
            want = ref.kept(m[s, g], 100, 48, 0, 0)
            np.testing.assert_array_equal(kept[s, g].cpu().numpy(), want)
            np.testing.assert_array_equal(dk[g][there], sk[g, want][there])
    assert (dst.k[dst.tab[0, 0]] != 5.0).all()
    kept, nl = evict(torch, src, dst, dev(torch, m), [-4, 3], 48, 0, 0)
    assert nl.tolist() == [0, 3] and kept[0].max() == -1 and kept[1, 0, :4].tolist() == [0, 1, 2, -1]


# --------------------------------------------------------------------------- what the logits say

def logprobs(torch, x, dtype, targets, top, scale=1.0, row_stride=0, vocab=None, stream=0):
    rows = x.shape[0]
    lp, en = (torch.full((rows,), 5.0, device="cuda") for _ in range(2))
    ids = torch.full((rows, max(top, 1)), -7, device="cuda", dtype=torch.int32)
    tl = torch.full((rows, max(top, 1)), 5.0, device="cuda")
    tg = dev(torch, np.asarray(targets, dtype=np.int32))
    binding.op_token_logprobs(x.data_ptr(), dtype, rows, vocab or x.shape[1], targets_ptr=tg.data_ptr(),
                              logprobs_ptr=lp.data_ptr(), entropy_ptr=en.data_ptr(), top=top,
                              top_ids_ptr=ids.data_ptr() if top else 0, top_logprobs_ptr=tl.data_ptr() if top else 0,
                              inv_temperature=scale, row_stride=row_stride, stream=stream)
    torch.cuda.synchronize()
    return lp, en, ids, tl


def logprobs_check(x, targets, top, scale, got):
    """x: [rows][vocab] in 64 bits."""
    lp, en, ids, tl = (f64(t) for t in got)
    for r in range(x.shape[0]):
        w_lp, w_en, w_ids, w_tl, S, W, D = ref.logprobs(x[r], scale, int(targets[r]), top)
        # (outputs are float32: what is past its largest value is an infinity there)
        w_lp, *w_tl = (math.copysign(math.inf, w) if abs(w) > 3.4028235e38 else w for w in [w_lp] + list(w_tl))
        assert ids[r].astype(int).tolist()[:top] == w_ids, (r, ids[r], w_ids)
        # a term e^d: d = scale (z - M) within 3 roundings of itself (one more to base 2), 2^d within 2^-22; sums of
        # terms of one sign in chains of up to 128 and trees; the largest term's chain starts from the others'
        c = (128 + 40) * U
        # a term under 2^-126, float32's least normal number, may be left out: |d| e^d is under 88 * 2^-126 there
        least = x.shape[1] * 2.0 ** -119
        dS, dW = c * S + 4 * U * W + least, c * W + 4 * U * D + least
        dlog = dS / (1 + S) + 4 * U * math.log1p(S)
        top_d = abs(w_lp) + math.log1p(S)
        if math.isnan(w_lp):
            assert math.isnan(lp[r])
        elif math.isinf(w_lp):
            assert lp[r] == w_lp
        else:
            assert abs(lp[r] - w_lp) <= dlog + 4 * U * (top_d + abs(w_lp)), (r, lp[r], w_lp)
        if math.isnan(w_en):
            assert math.isnan(en[r])
        else:
            assert abs(en[r] - w_en) <= dlog + dW / (1 + S) + W * dS / (1 + S) ** 2 + 6 * U * (w_en + W), (r, en[r], w_en)
        for a, b in zip(tl[r], w_tl):
            if math.isnan(b) or math.isinf(b):
                np.testing.assert_equal(a, b)
            else:
                assert abs(a - b) <= dlog + 4 * U * (2 * abs(b) + math.log1p(S)), (r, a, b)


LOGITS = [(1, 1, 1, "f32", 1.0, 0), (3, 2, 2, "bf16", 2.0, 1), (5, 100, 64, "f16", 1.0, 3), (4, 1000, 5, "bf16", 0.7, 0),
          (2, 4096, 20, "f32", 1.3, 0), (3, 32001, 20, "f32", 1 / 0.7, 3), (2, 126464, 50, "bf16", 1.0, 0),
          (33, 5003, 0, "f16", 1.0, 1), (2, 300007, 64, "bf16", 1.0, 5), (310, 9001, 7, "bf16", 1.0, 1),
          (40, 40000, 5, "f16", 1.0, 0), (153, 65003, 30, "f32", 1.0, 1), (90, 70001, 64, "bf16", 0.5, 1), (700, 1023, 3, "bf16", 1.0, 2),
          (400, 6001, 64, "f32", 1.0, 1),
          # many rows: fewer threads a row
          (650, 20011, 20, "bf16", 1.0, 0), (310, 30001, 64, "f32", 1.0, 5), (1300, 8193, 7, "f16", 0.7, 2)]


@pytest.mark.parametrize("rows,vocab,top,dtype,scale,pad", LOGITS)
def test_token_logprobs(torch, rows, vocab, top, dtype, scale, pad):
    rng = np.random.default_rng(rows + vocab)
    x = rng.standard_normal((rows, vocab + pad)) * rng.uniform(0.5, 6.0, (rows, 1))
    if rows > 2:
        x[1, vocab // 2] = 60.0                            # a nearly certain row
    buf = dev(torch, x.astype(np.float32)).to(dt(torch, dtype))
    targets = rng.integers(0, vocab, rows)
    if rows > 2:
        targets[1], targets[2] = vocab // 2, vocab
    got = logprobs(torch, buf, dtype, targets, top, scale=scale, row_stride=vocab + pad, vocab=vocab)
    logprobs_check(f64(buf)[:, :vocab], targets, top, np.float32(scale).astype(np.float64), got)


def odd_rows(vocab):
    rng = np.random.default_rng(vocab)
    x = rng.standard_normal((13, vocab))
    x[0] = 0.0                                             # all alike
    x[1] = -np.inf
    x[1, [5, 77, 300]] = [1.0, 2.0, 1.0]                   # few may come
    x[2] = rng.integers(0, 3, vocab)                       # many ties
    x[3, 10:] = -np.inf
    x[4] = -np.inf                                         # none may come
    x[5, 7] = np.inf
    x[6, 9] = np.nan
    x[7] = np.nan
    x[7, 3] = 1.0
    x[8] = np.arange(vocab)                                # ever larger
    x[9] = -np.arange(vocab)
    x[10] = 0.0
    x[10, ::2] = -0.0
    x[11, :] = np.where(np.arange(vocab) % 512 < 8, 5.0, x[11])        # one thread's tokens are the largest
    x[12, 256:] = -1e30
    return x, [0, 77, 5, 12, 0, 7, 0, 3, vocab - 1, vocab - 1, -1, 0, 300]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("vocab", [700, 40007])
def test_token_logprobs_ties_and_tokens_that_cannot_come(torch, vocab, dtype):
    x, targets = odd_rows(vocab)
    buf = dev(torch, x.astype(np.float32)).to(dt(torch, dtype))
    got = logprobs(torch, buf, dtype, targets, 50)
    logprobs_check(f64(buf), targets, 50, 1.0, got)


@pytest.mark.parametrize("dtype,top", [("bf16", 5), ("f32", 50)])
def test_token_logprobs_of_many_odd_rows(torch, dtype, top):
    """Every kind of row behind every other in one call, more rows than run at once."""
    x, targets = odd_rows(16001)
    order = np.random.default_rng(4).integers(0, 13, 1300)
    buf = dev(torch, x.astype(np.float32)).to(dt(torch, dtype))
    rows = buf[torch.from_numpy(order).cuda()]
    targets = [targets[k] for k in order]
    logprobs_check(f64(rows), targets, top, 1.0, logprobs(torch, rows, dtype, targets, top))


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("vocab", [900, 33001])
def test_token_logprobs_of_the_types_lowest_values(torch, vocab, dtype):
    """Masks of the type's lowest value beside ordinary logits, alone, and beside -inf; huge logits; a row whose largest
    changes from one to the other."""
    rng = np.random.default_rng(vocab + 1)
    low = {"bf16": -3.3895313892515355e38, "f16": -65504.0, "f32": -3.4028234663852886e38}[dtype]
    x = rng.standard_normal((7, vocab))
    x[0] = low
    x[1, 10:] = low
    x[2] = low
    x[2, ::2] = -np.inf
    x[3] = np.where(rng.random(vocab) < 0.5, low, -low)
    x[4] = low
    x[4, vocab - 3] = 3.0
    x[5, : vocab // 2] = low / 2
    x[6] = x[6] * 1e4 if dtype != "f16" else x[6] * 1e3
    buf = dev(torch, x.astype(np.float32)).to(dt(torch, dtype))
    targets = [3, 4, 1, 7, vocab - 3, vocab - 1, 0]
    got = logprobs(torch, buf, dtype, targets, 12)
    with np.errstate(over="ignore", invalid="ignore"):
        logprobs_check(f64(buf), targets, 12, 1.0, got)


def test_token_logprobs_each_output_alone(torch):
    rng = np.random.default_rng(1)
    x = dev(torch, rng.standard_normal((3, 999)).astype(np.float32))
    lp, en, ids, tl = logprobs(torch, x, "f32", [1, 2, 3], 4)
    e2, l2 = torch.zeros(3, device="cuda"), torch.zeros(3, device="cuda")
    tg = dev(torch, np.array([1, 2, 3], dtype=np.int32))
    binding.op_token_logprobs(x.data_ptr(), "f32", 3, 999, entropy_ptr=e2.data_ptr())
    binding.op_token_logprobs(x.data_ptr(), "f32", 3, 999, targets_ptr=tg.data_ptr(), logprobs_ptr=l2.data_ptr())
    i2, t2 = torch.zeros(3, 4, device="cuda", dtype=torch.int32), torch.zeros(3, 4, device="cuda")
    binding.op_token_logprobs(x.data_ptr(), "f32", 3, 999, top=4, top_ids_ptr=i2.data_ptr(), top_logprobs_ptr=t2.data_ptr())
    torch.cuda.synchronize()
    assert torch.equal(e2, en) and torch.equal(l2, lp) and torch.equal(i2, ids) and torch.equal(t2, tl)


# --------------------------------------------------------------------------- all of them, as a step runs them

def _layer(torch, seed):
    """Inputs of a layer's steps, and a function that runs them on a stream."""
    rng = np.random.default_rng(seed)
    b, H, Hkv, hd, ps, n0, steps, keep = 2, 8, 2, 64, 16, 50, 14, 32
    c = Pages(torch, rng, b, Hkv, hd, "bf16", ps, 5, poison=0.0)
    d = Pages(torch, rng, b, Hkv, hd, "bf16", ps, 3, poison=0.0)
    width = (H + 2 * Hkv) * hd
    st = {"c": c, "d": d, "keep": keep, "n": n0 + steps,
          "pre": dev(torch, rng.standard_normal((b * n0, width)).astype(np.float32)).to(torch.bfloat16),
          "new": dev(torch, rng.standard_normal((steps, b, width)).astype(np.float32)).to(torch.bfloat16),
          "w": [dev(torch, (1 + 0.2 * rng.standard_normal(hd)).astype(np.float32)).to(torch.bfloat16) for _ in range(2)],
          "head": dev(torch, rng.standard_normal((H * hd, 500)).astype(np.float32) * 0.1)}
    st["q"] = torch.zeros(b * n0, H, hd, device="cuda", dtype=torch.bfloat16)
    st["out"] = torch.zeros(steps + 1, b, H, hd, device="cuda", dtype=torch.bfloat16)
    st["mass"] = torch.zeros(b, Hkv, 80, device="cuda")
    st["mass2"] = torch.zeros(b, Hkv, 48, device="cuda")
    st["kept"] = torch.zeros(b, Hkv, keep, device="cuda", dtype=torch.int32)
    st["lens2"] = torch.zeros(b, device="cuda", dtype=torch.int32)
    st["logits"] = torch.zeros(b, 500, device="cuda")
    st["lp"], st["en"] = torch.zeros(b, device="cuda"), torch.zeros(b, device="cuda")
    st["tg"] = dev(torch, np.array([3, 499], dtype=np.int32))
    st["at"] = [dev(torch, np.full(b, n0 + i, dtype=np.int32)) for i in range(steps + 1)]
    st["ws"] = torch.zeros(max(16, binding.attention_paged_workspace(b, H, Hkv, hd, 1, 80, mass=True)), device="cuda",
                           dtype=torch.uint8)
    c.s, d.s = c.struct(), d.struct()
    spec = binding.make_rope(hd)

    def store(x, q, R, starts, stream):
        es = 2
        binding.op_qk_norm_rope_paged(c.s, x.data_ptr(), x.data_ptr() + H * hd * es, x.data_ptr() + (H + Hkv) * hd * es,
                                      q.data_ptr(), H, R, "bf16", starts_ptr=starts, q_weight_ptr=st["w"][0].data_ptr(),
                                      k_weight_ptr=st["w"][1].data_ptr(), rope=spec, q_row_stride=width,
                                      k_row_stride=width, v_row_stride=width, stream=stream)

    def go(stream):
        st["mass"].zero_()
        store(st["pre"], st["q"], n0, 0, stream)
        for i in range(steps):
            store(st["new"][i], st["q"], 1, st["at"][i].data_ptr(), stream)
            binding.op_attention_paged(st["q"].data_ptr(), c.s, st["out"][i].data_ptr(), H, 1,
                                       lens_ptr=st["at"][i + 1].data_ptr(), mass_ptr=st["mass"].data_ptr(), mass_stride=80,
                                       ws_ptr=st["ws"].data_ptr(), ws_bytes=st["ws"].numel(), stream=stream)
        binding.op_kv_paged_evict(c.s, d.s, st["mass"].data_ptr(), keep, st["kept"].data_ptr(), st["lens2"].data_ptr(),
                                  lens_ptr=st["at"][steps].data_ptr(), sinks=2, recent=8, mass_stride=80,
                                  mass_out_ptr=st["mass2"].data_ptr(), mass_out_stride=48, stream=stream)
        binding.op_attention_paged(st["q"].data_ptr(), d.s, st["out"][steps].data_ptr(), H, 1,
                                   lens_ptr=st["lens2"].data_ptr(), ws_ptr=st["ws"].data_ptr(),
                                   ws_bytes=st["ws"].numel(), stream=stream)
        torch.matmul(st["out"][steps].float().view(b, -1), st["head"], out=st["logits"])
        binding.op_token_logprobs(st["logits"].data_ptr(), "f32", b, 500, targets_ptr=st["tg"].data_ptr(),
                                  logprobs_ptr=st["lp"].data_ptr(), entropy_ptr=st["en"].data_ptr(), stream=stream)

    return st, go


def _layer_check(torch, st):
    c, d, n, keep = st["c"], st["d"], st["n"], st["keep"]
    # the last step's attention from the cache as the calls left it, the weights from all steps' own reference
    attention_check(d, st["q"][:2].view(2, 1, 8, 64), [keep, keep], st["out"][-1].view(2, 1, 8, 64))
    attention_check(c, st["q"][:2].view(2, 1, 8, 64), [n, n], st["out"][-2].view(2, 1, 8, 64))
    mass = st["mass"].cpu().numpy()
    # 14 steps of 4 heads a cached head, each adding weights that sum to 1
    np.testing.assert_allclose(mass.sum(-1), 14 * 4, rtol=1e-5)
    kept = st["kept"].cpu().numpy()
    for s in range(2):
        ck, _ = ref.gather(f64(c.k), c.tab[s], n, 16)
        dk, _ = ref.gather(f64(d.k), d.tab[s], keep, 16)
        for g in range(2):
            want = ref.kept(mass[s, g], n, keep, 2, 8)
            np.testing.assert_array_equal(kept[s, g], want)
            np.testing.assert_array_equal(dk[g], ck[g, want])
    for r in range(2):
        w = ref.logprobs(f64(st["logits"])[r], 1.0, [3, 499][r], 0)
        assert abs(float(st["lp"][r]) - w[0]) < 1e-5 * (1 + abs(w[0])) and abs(float(st["en"][r]) - w[1]) < 1e-5 * (1 + w[1])


def test_a_layer_of_all_of_them(torch):
    st, go = _layer(torch, 1)
    go(torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    binding.op_check()
    _layer_check(torch, st)


def test_two_graphs_on_two_streams(torch):
    """Captured on streams of their own, replayed at the same time: states, and workspaces, of their own."""
    both = []
    for seed in (2, 3):
        st, go = _layer(torch, seed)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            go(s.cuda_stream)                              # (the matrix product's own set-up)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            go(s.cuda_stream)
        both.append((st, g, s))
    eager = []
    for st, _, _ in both:
        eager.append({k: st[k].clone() for k in ("out", "mass", "kept", "lp", "en")})
        for k in ("out", "mass", "kept", "lp", "en"):
            st[k].zero_()
    torch.cuda.synchronize()
    for _ in range(3):
        for st, g, s in both:
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    binding.op_check()
    for (st, _, _), want in zip(both, eager):
        _layer_check(torch, st)
        for k, v in want.items():
            assert torch.equal(st[k], v), k


FIRST_CALLS = """
import sys
sys.path[:0] = ["tests", "."]
import torch
import test_gpu_paged as t
from cached_masked_decoding_gb300 import binding
binding.lib()
st, go = t._layer(torch, 7)
s = torch.cuda.Stream()
torch.matmul(st["out"][0].float().view(2, -1), st["head"], out=st["logits"])   # (the matrix product's own set-up)
torch.cuda.synchronize()
with torch.cuda.stream(s):
    torch.matmul(st["out"][0].float().view(2, -1), st["head"], out=st["logits"])
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g, stream=s):
    go(s.cuda_stream)
g.replay()
torch.cuda.synchronize()
keep = ("out", "mass", "kept", "lp", "en")
got = {k: st[k].clone() for k in keep}
t._layer_check(torch, st)
go(torch.cuda.current_stream().cuda_stream)
torch.cuda.synchronize()
binding.op_check()
print("same" if all(torch.equal(st[k], got[k]) for k in keep) else "not the same")
"""


def test_first_calls_of_a_process_can_be_captured(torch):
    """Every kernel's first launch inside a capture, in a process of its own: the same bits as launched directly."""
    import subprocess
    import sys
    from pathlib import Path
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS], cwd=Path(__file__).resolve().parent.parent,
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "same", r.stdout[-500:] + r.stderr[-2000:]
