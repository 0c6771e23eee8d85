"""The operators of paged decoding where their numerics are at an end: keys on no page in front of a walk, weights far
apart, long rows.  Against the plain 64-bit restatement (paged_ref); half a rounding step is 2^-8 of the value in bf16,
2^-11 in f16, 2^-24 in float32.
"""
import math

import numpy as np
import pytest

import paged_ref as ref
from test_gpu_paged import HALF, TINY, U, Pages, attend, dev, dt, f64, logprobs, torch  # noqa: F401 (torch: the fixture)

pytestmark = pytest.mark.gpu


# --------------------------------------------------------------------------- attention

def attention_close(c, q, lens, out, mass=None):
    """out and mass (which began as zeros) against 64 bits; a probability counts to its own size however small it is."""
    b, R, H, hd = q.shape
    G = H // c.hkv
    kp, vp = f64(c.k), f64(c.v)
    for s in range(b):
        n = int(lens[s])
        k, there = ref.gather(kp, c.tab[s], n, c.ps)
        v, _ = ref.gather(vp, c.tab[s], n, c.ps)
        want, m, pv, sv, sk = ref.attention(f64(q[s]), k, v, there, hd ** -0.5)
        # a score: a float32 sum of hd exact products (each within 2^-23 of the sum of their sizes, the tensor core
        # truncates), scaled and put against its reference: 4 roundings of it; p = 2^z within 2^-22
        dz = (hd + 8) * 2.0 ** -23 * sk + 2.0 ** -22
        # p in two halves: 2^-16 of it (bf16); 2^-22 of it, or 2^-45 of the row's largest (f16).  Sums of n terms in
        # trees and tiles, on both sides of the quotient
        halves = 2.0 ** -16 * pv if c.dtype == "bf16" else 2.0 ** -22 * pv + 2.0 ** -45 * sv
        tol = (2 * dz + (n / 16 + 24) * U) * pv + halves + HALF[c.dtype] * 1.01 * np.abs(want) + TINY[c.dtype]
        err = np.abs(f64(out[s]) - want)
        assert (err <= tol).all(), (s, float((err / np.maximum(tol, 1e-300)).max()))
        if mass is not None:
            got = f64(mass[s])
            tol = m * (2 * float(dz.max()) + (n / 16 + 40 + R * G + 4) * U) + 1e-37
            assert (np.abs(got[:, :n] - m) <= tol).all(), s
            assert (got[:, n:] == 0).all()


def at_level(torch, c, q, lens, level):
    """Adds to the first dim of all keys and queries what takes every score to about `level` (hd^-0.5 is the scale)."""
    a = math.sqrt(abs(level)) * c.hd ** 0.25
    for s, n in enumerate(lens):
        t = np.arange(n)
        page, slot = (torch.from_numpy(x).cuda() for x in (c.tab[s, t // c.ps].astype(np.int64), t % c.ps))
        c.k[page, :, slot, 0] = a
    q[..., 0] = math.copysign(a, level)


HOLES = [
    # b, R, H, H_kv, hd, page, positions, no pages among them (first positions; "some": half of all, at random)
    (1, 1, 8, 2, 64, 16, 512, 128),                        # items stay whole
    (2, 2, 4, 1, 128, 32, 400, 300),
    (1, 1, 4, 1, 64, 16, 4000, 2048),                      # the front parts see nothing, one starts in the hole
    (2, 1, 8, 8, 64, 128, 8192, "some"),                   # parts that start in a hole anywhere
    (2, 4, 16, 4, 128, 128, 4096, "some"),                 # 16 rows of a cached head, then 32 and 64
    (2, 8, 16, 4, 128, 256, 8192, "some"),
    (2, 16, 8, 2, 64, 256, 8192, "some"),
]


@pytest.mark.parametrize("with_mass", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("level", [-16.0, -25.0, -60.0, -200.0])
@pytest.mark.parametrize("b,R,H,Hkv,hd,ps,n,holes", HOLES)
def test_scores_below_zero_behind_keys_on_no_page(torch, b, R, H, Hkv, hd, ps, n, holes, level, dtype, with_mass):
    """A window's first pages were given back, or pages anywhere: the others' weights are as if nothing else had been."""
    rng = np.random.default_rng(n + R + int(-level))
    most = -(-n // ps)
    c = Pages(torch, rng, b, Hkv, hd, dtype, ps, most).fill(rng, [n] * b)
    q = dev(torch, rng.standard_normal((b, R, H, hd)).astype(np.float32)).to(dt(torch, dtype))
    at_level(torch, c, q, [n] * b, level)
    if holes == "some":
        gone = rng.random((b, most)) < 0.5
        gone[:, 0], gone[:, -1] = True, False
    else:
        gone = np.broadcast_to(np.arange(most) * ps < holes, (b, most))
    assert gone.any() and not gone.all(1).any()
    c.tab[gone] = -1
    mass = torch.zeros(b, Hkv, most * ps, device="cuda") if with_mass else None
    out = attend(torch, c, q, [n] * b, mass=mass)
    attention_close(c, q, [n] * b, out, mass)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("where", [0, 130, 8191])
@pytest.mark.parametrize("above,values", [(16.0, 1.0), (17.5, 1.0), (20.0, 30.0), (24.0, 1000.0)])
@pytest.mark.parametrize("R", [1, 16])
def test_many_light_keys_beside_a_heavy_one(torch, dtype, where, above, values, R):
    """One key takes nearly all of the weight and has values of next to nothing: the output is the others'."""
    rng = np.random.default_rng(int(above) + where)
    n, hd = 8192, 64
    c = Pages(torch, rng, 1, 1, hd, dtype, 64, 128).fill(rng, [n])
    a = math.sqrt(above) * hd ** 0.25
    t = np.arange(n)
    page, slot = (torch.from_numpy(x).cuda() for x in (c.tab[0, t // 64].astype(np.int64), t % 64))
    c.k[page, 0, slot] = c.k[page, 0, slot] * 0.25
    c.k[page, 0, slot, 0] = 0.0
    c.k[page[where], 0, slot[where], 0] = a
    c.v[page, 0, slot] = (c.v[page, 0, slot].float() * 0.1 + 1.0).mul(values).to(c.v.dtype)
    c.v[page[where], 0, slot[where]] = 0.0
    q = dev(torch, (0.25 * rng.standard_normal((1, R, 2, hd))).astype(np.float32)).to(dt(torch, dtype))
    q[..., 0] = a
    out = attend(torch, c, q, [n])
    attention_close(c, q, [n], out)


# --------------------------------------------------------------------------- what long rows of logits say

def logprobs_close(x, targets, top, got, rows=None, scale=1.0):
    """Some rows of x [rows][vocab] (64 bits) against their definition; rows long enough for chains of sums."""
    lp, en, ids, tl = (f64(t) for t in got)
    vocab = x.shape[1]
    for r in range(x.shape[0]) if rows is None else rows:
        w_lp, w_en, w_ids, w_tl, S, W, D = ref.logprobs(x[r], scale, int(targets[r]), top)
        assert ids[r].astype(int).tolist()[:top] == w_ids, (r, ids[r], w_ids)
        # a term e^d: d = z - M within 3 roundings of itself (one more to base 2), 2^d within 2^-22; sums of terms of
        # one sign in chains of up to 256, which are joined one by one (2^16 elements of a row or more each; up to 8
        # roundings where the reference rises), and in trees; the largest term's chain starts from the others'.
        # A term under 2^-126, float32's least normal number, may be left out: |d| e^d is under 88 * 2^-126 there
        c = (256 + 8 * (vocab // 65536) + 40) * U
        least = vocab * 2.0 ** -119
        dS, dW = c * S + 4 * U * W + least, c * W + 4 * U * D + least
        dlog = dS / (1 + S) + 4 * U * math.log1p(S)
        if not math.isfinite(w_lp):
            np.testing.assert_equal(lp[r], w_lp)
        else:
            assert abs(lp[r] - w_lp) <= dlog + 4 * U * (2 * abs(w_lp) + math.log1p(S)), (r, lp[r], w_lp, dlog)
        assert abs(en[r] - w_en) <= dlog + dW / (1 + S) + W * dS / (1 + S) ** 2 + 6 * U * (w_en + W), (r, en[r], w_en)
        for a, w in zip(tl[r], w_tl):
            if not math.isfinite(w):
                np.testing.assert_equal(a, w)
                continue
            assert abs(a - w) <= dlog + 4 * U * (2 * abs(w) + math.log1p(S)), (r, a, w)


@pytest.mark.parametrize("vocab,dtype", [(1 << 20, "f32"), ((1 << 22) + 5, "f32"), ((1 << 20) + 4099, "bf16"),
                                         (1 << 22, "f16")])
def test_logprobs_of_rows_with_long_chains_of_sums(torch, vocab, dtype):
    """A CTA a row; what every term adds is under half a step of a thread's sum from the start, or all are alike, or
    one takes nearly all, or ever larger ones come."""
    rng = np.random.default_rng(vocab)
    kinds = np.empty((5, vocab), dtype=np.float32)
    kinds[0] = -16.0 - 0.2 * rng.random(vocab)
    kinds[0, :2048] = 0.0
    kinds[1] = 3.0 * rng.standard_normal(vocab)
    kinds[2] = rng.standard_normal(vocab)
    kinds[2, vocab - 9] = 30.0
    kinds[3] = np.linspace(-9.0, 9.0, vocab)
    kinds[4] = np.where(np.arange(vocab) % 3 == 0, -np.inf, -12.0 - rng.random(vocab))
    kinds[4, vocab // 2] = 0.0
    five = dev(torch, kinds).to(dt(torch, dtype))
    x = five[torch.arange(160, device="cuda") % 5].contiguous()
    targets = rng.integers(0, vocab, 160)
    targets[2] = vocab - 9
    got = logprobs(torch, x, dtype, targets, 3)
    logprobs_close(f64(x[:5]), targets, 3, got, range(5))
    if vocab % 8 == 0:                                     # the same row at the same alignment: the same bits
        for out in got[1:]:
            assert torch.equal(out[:5].repeat(32, *[1] * (out.dim() - 1)), out)


@pytest.mark.parametrize("scale", [0.3, 2e-38, 1e-37])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,vocab", [(3, 501), (2, 40000), (200, 9001)])
def test_logprobs_of_logits_further_apart_than_float32_holds(torch, rows, vocab, dtype, scale):
    """The difference of two logits is past the type, but not what an inverse temperature under 1 makes of it."""
    rng = np.random.default_rng(vocab)
    x = 3e38 * rng.uniform(-1.0, 1.0, (rows, vocab)).astype(np.float32)
    x[0, : vocab // 2] = -np.inf
    x[1] = -3e38
    x[1, vocab - 2] = 3e38
    buf = dev(torch, x).to(dt(torch, dtype))
    targets = rng.integers(0, vocab, rows)
    targets[0], targets[1] = int(np.argmin(x[0, vocab // 2:])) + vocab // 2, 7
    got = logprobs(torch, buf, dtype, targets, 60, scale=scale)
    logprobs_close(f64(buf), targets, 60, got, range(min(rows, 8)), scale=float(np.float32(scale)))


@pytest.mark.parametrize("vocab,top,dtype", [(126471, 20, "f32"), (126471, 64, "f32"), (300007, 50, "bf16"),
                                             (1000003, 7, "f16")])
def test_logprobs_of_rows_whose_units_are_several_batches(torch, vocab, top, dtype):
    """A CTA a row, long enough for units of 2, 4 and 8 batches of a thread, the last ones partly filled: ties in many
    units, in the elements behind the last whole batch and behind the last vector, one thread's elements the largest."""
    rng = np.random.default_rng(vocab + top)
    x = np.empty((7, vocab), dtype=np.float32)
    x[0] = 2.0 * rng.standard_normal(vocab)
    x[1] = rng.integers(0, 9, vocab)
    x[2] = np.where(np.arange(vocab) % 2048 < 8, 5.0 + rng.random(vocab), -1.0)
    x[3] = np.linspace(-20.0, 4.0, vocab)
    x[4] = -np.inf
    x[4, rng.choice(vocab, 30, replace=False)] = 1.0
    x[4, vocab - 1] = 2.0
    x[5] = rng.standard_normal(vocab)
    x[5, -3000:] = 9.0
    x[5, -3000::7] = 9.5
    x[6] = 0.0
    buf = dev(torch, x).to(dt(torch, dtype))
    targets = rng.integers(0, vocab, 160)
    targets[4] = vocab - 1
    got = logprobs(torch, buf[torch.arange(160, device="cuda") % 7].contiguous(), dtype, targets, top)
    order = [0, 1, 2, 3, 4, 5, 6, 159]
    logprobs_close(f64(buf[torch.tensor(order, device="cuda") % 7]), targets[order], top, [t[order] for t in got])


# --------------------------------------------------------------------------- weights of many sequences

@pytest.mark.parametrize("b,R,H,Hkv,dtype", [(32, 1, 8, 8, "bf16"), (48, 1, 8, 4, "f16"), (8, 16, 32, 8, "bf16"),
                                             (10, 4, 16, 8, "f16")])
def test_weights_of_runs_of_keys(torch, b, R, H, Hkv, dtype):
    """So many keys that a CTA of the second kernel adds up the weights of several pieces of them: lengths that end in
    the first, inside a run, at its ends and in the table's last page."""
    rng = np.random.default_rng(b + R)
    ps, most = 64, 128                                     # 8192 positions
    lens = rng.integers(1, most * ps, b)
    lens[:8] = [8192, 513, 511, 0, 8191, 1, 2049, 6145]
    c = Pages(torch, rng, b, Hkv, 64, dtype, ps, most).fill(rng, lens)
    q = dev(torch, (1.5 * rng.standard_normal((b, R, H, 64))).astype(np.float32)).to(dt(torch, dtype))
    mass = torch.zeros(b, Hkv, most * ps, device="cuda")
    out = attend(torch, c, q, lens, mass=mass)
    attention_close(c, q, lens, out, mass)
