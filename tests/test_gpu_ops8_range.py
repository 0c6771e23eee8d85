"""The 8-bit operators at the ends of their ranges.

Tolerances count roundings: half a step is 2^-8 of the value in bf16.
"""
import math
from decimal import Decimal, getcontext

import numpy as np
import pytest

import ops8_ref as ref
from cached_masked_decoding_gb300 import binding
from gpu_util import torch_cuda

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    t = torch_cuda()
    binding.lib()
    return t


def dev(torch, a):
    return torch.from_numpy(np.array(a, order="C")).cuda()


# --------------------------------------------------------------------------- attention

def attend(torch, q, k, ks, v, vs, scale):
    """q [b][R][H][hd] bf16 over codes [b][H_kv][T][hd], bytes [b][H_kv][T] (device tensors)."""
    b, R, H, hd = q.shape
    h, T = k.shape[1:3]
    cache = binding.make_kv8(k.data_ptr(), v.data_ptr(), ks.data_ptr(), vs.data_ptr(), b, h, T, hd)
    n = binding.attention_kv8_workspace(b, H, h, hd, R, T)
    ws = torch.full((max(n, 16),), 0xff, device="cuda", dtype=torch.uint8)
    out = torch.full_like(q, 9.0)
    binding.op_attention_kv8(q.data_ptr(), cache, out.data_ptr(), H, R, scale=scale, ws_ptr=ws.data_ptr(), ws_bytes=n)
    assert binding.op_check() == 0
    return out


def along_first_dim(torch, h, R, hd, score2, values, byte):
    """A cache whose key t scores score2[t] (to base 2, with scale ln 2) for queries of (1, 0, ..), and whose
    value rows are codes of +-values[t] with scale byte byte[t]."""
    T = len(score2)
    rows = np.zeros((T, hd))
    rows[:, 0] = score2
    kc, ks = ref.quantise(rows)
    assert (ref.dequantise(kc, ks) == rows).all()
    sign = np.where(np.arange(hd) % 3 == 0, -1.0, 1.0)
    vc = ref.encode(values[:, None] * sign)
    q = torch.zeros(1, R, h, hd, device="cuda", dtype=torch.bfloat16)
    q[..., 0] = 1.0
    every = [dev(torch, np.broadcast_to(a, (1, h) + a.shape)) for a in (kc, ks, vc, byte)]
    v = ref.dequantise(vc, byte)
    p = np.exp2(score2 - score2.max())
    return q, every, (p @ v) / p.sum()


def check(got, want):
    """Every row and head alike: bf16 probabilities and output, 2^-8 of sum p|v| each (|v| the same for all that
    counts), and scores to base 2 up to 2^8 in float32: 2^-16 of a probability."""
    np.testing.assert_allclose(got, np.broadcast_to(want, got.shape), rtol=2.0 ** -7 + 2.0 ** -15, atol=0)


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("R", [1, 16, 32, 64, 100, 200])
@pytest.mark.parametrize("score2,above,T", [(104.0, 5, 2048), (60.0, 49, 1600), (96.0, 13, 4096), (104.0, 4, 4096)])
def test_many_large_products_of_one_sign(torch, R, hd, score2, above, T):
    """Scores far above the first 32 keys', value scales 2^above over theirs and codes near the largest, so that each
    product and each key lane's sum is under 2^110 but what they add up to is over 2^128: so many heads
    that one walk has all keys."""
    h = 160
    if R <= 64:
        assert binding.attention_kv8_workspace(1, h, h, hd, R, T) == 0
    late = np.arange(T) >= 32
    q, c, want = along_first_dim(torch, h, R, hd, np.where(late, score2, 0.0), np.where(late, 448.0, 1.0),
                                 np.where(late, 127 + above, 127).astype(np.uint8))
    got = attend(torch, q, *c, math.log(2.0)).double().cpu().numpy()
    assert abs(want).min() > 447 * 2.0 ** above
    check(got, want)


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("R,T,keys", [(1, 1024, 128), (32, 1024, 128), (64, 640, 128), (1, 16384, 256), (8, 16384, 256),
                                      (64, 16384, 256), (100, 4096, 64)])
@pytest.mark.parametrize("order", [1, -1])
def test_splits_whose_references_lie_far_apart(torch, R, T, keys, hd, order):
    """A split whose first keys score 0 and the rest 104 beside splits that score 160 throughout (base 2): the first
    has 2^-56 of the weight for values 2^70 as large, so it is what the row is made of."""
    rest = np.arange(T) >= keys
    score2 = np.where(rest, 160.0, np.where(np.arange(T) < 32, 0.0, 104.0))
    byte = np.where(rest, 120, 190)
    if order < 0:
        score2, byte = np.roll(score2, -keys), np.roll(byte, -keys)
    q, c, want = along_first_dim(torch, 1, R, hd, score2, np.full(T, 256.0), byte.astype(np.uint8))
    assert abs(want).min() > 100                     # 256 * 2^-7 = 2 without that split
    check(attend(torch, q, *c, math.log(2.0)).double().cpu().numpy(), want)


# --------------------------------------------------------------------------- calls in turn

def test_calls_in_turn_see_what_the_one_before_wrote(torch):
    """Quantise and product, store and attention, again and again over the same buffers with changing
    inputs and no synchronisation: the same bits as step by step."""
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    steps, N, M, K, h, hd, T = 12, 4, 1024, 512, 8, 64, 300
    w = torch.randint(0, 0x7f, (M, K), generator=g, device="cuda", dtype=torch.uint8)
    ws = torch.full((K // 128, M), 119, device="cuda", dtype=torch.uint8)
    x = (torch.randn(steps, N, K, generator=g, device="cuda") *
         torch.exp2(torch.arange(steps, device="cuda") - 6.0)[:, None, None]).bfloat16()
    kv = x[..., :h * hd].contiguous()
    spec = binding.make_rope(hd)
    pos = torch.arange(N, device="cuda", dtype=torch.int32)
    starts = torch.full((1,), T - N, device="cuda", dtype=torch.int32)
    n = binding.attention_kv8_workspace(1, h, h, hd, N, T)
    atts = torch.empty(max(n, 16), device="cuda", dtype=torch.uint8)

    def run(sync):
        xc = torch.zeros(N, K, device="cuda", dtype=torch.uint8)
        xs = torch.zeros(K // 128, N, device="cuda", dtype=torch.uint8)
        codes = torch.zeros(2, 1, h, T, hd, device="cuda", dtype=torch.uint8)
        scales = torch.full((2, 1, h, T), 127, device="cuda", dtype=torch.uint8)
        cache = binding.make_kv8(codes[0].data_ptr(), codes[1].data_ptr(), scales[0].data_ptr(), scales[1].data_ptr(), 1, h,
                                 T, hd)
        turned = torch.zeros(N, h, hd, device="cuda", dtype=torch.bfloat16)
        y = torch.zeros(steps, N, M, device="cuda")
        out = torch.zeros(steps, N, h, hd, device="cuda", dtype=torch.bfloat16)
        back = torch.zeros(2, steps, N, h, hd, device="cuda", dtype=torch.bfloat16)
        torch.cuda.synchronize()
        for i in range(steps):
            calls = [
                lambda: binding.op_quantise8(x[i].data_ptr(), "bf16", N, K, xc.data_ptr(), xs.data_ptr()),
                lambda: binding.op_gemm8(w.data_ptr(), ws.data_ptr(), xc.data_ptr(), xs.data_ptr(), y[i].data_ptr(), "f32", M,
                                         N, K),
                lambda: binding.op_rope(kv[i].data_ptr(), turned.data_ptr(), pos.data_ptr(), N, h, hd, "bf16", spec),
                lambda: binding.op_kv8_store(cache, turned.data_ptr(), kv[i].data_ptr(), "bf16", N,
                                             starts_ptr=starts.data_ptr()),
                lambda: binding.op_kv8_load(cache, back[0, i].data_ptr(), back[1, i].data_ptr(), "bf16", N,
                                            starts_ptr=starts.data_ptr()),
                lambda: binding.op_attention_kv8(turned.data_ptr(), cache, out[i].data_ptr(), h, N, ws_ptr=atts.data_ptr(),
                                                 ws_bytes=n),
            ]
            for call in calls:
                call()
                if sync:
                    torch.cuda.synchronize()
        torch.cuda.synchronize()
        assert binding.op_check() == 0
        return y, out, back

    want = run(True)
    assert all(t.float().abs().amax(dim=tuple(range(1, t.dim()))).min() > 0 for t in want)
    for _ in range(20):
        for a, b in zip(want, run(False)):
            assert torch.equal(a, b)


# --------------------------------------------------------------------------- cache

@pytest.mark.parametrize("hd", [64, 128])
def test_cache_rows_past_32_bits_of_elements(torch, hd):
    """A row of 2^32 elements and one head: the last head is its own, not the first one again."""
    h = 2 ** 32 // hd + 1
    rows = [torch.zeros(1, h, hd, device="cuda", dtype=torch.bfloat16) for _ in range(2)]
    for w, r in enumerate(rows):
        r[0, 0], r[0, -1] = 1.0 + w, 5.0 + w
    codes = [torch.zeros(h, hd, device="cuda", dtype=torch.uint8) for _ in range(2)]
    scales = [torch.zeros(h, device="cuda", dtype=torch.uint8) for _ in range(2)]
    cache = binding.make_kv8(codes[0].data_ptr(), codes[1].data_ptr(), scales[0].data_ptr(), scales[1].data_ptr(), 1, h, 1, hd)
    binding.op_kv8_store(cache, rows[0].data_ptr(), rows[1].data_ptr(), "bf16", 1)
    for w in range(2):
        for at, value in ((0, 1.0 + w), (-1, 5.0 + w), (1, 0.0), (-2, 0.0)):
            got = ref.dequantise(codes[w][at].cpu().numpy()[None], scales[w][at].cpu().numpy()[None])
            assert (got == value).all()
        rows[w].fill_(9.0)
    binding.op_kv8_load(cache, rows[0].data_ptr(), rows[1].data_ptr(), "bf16", 1)
    for w, r in enumerate(rows):
        assert (r[0, 0] == 1.0 + w).all() and (r[0, -1] == 5.0 + w).all() and (r[0, 1:-1] == 0).all()


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("R", [1, 32, 64, 100, 200])
@pytest.mark.parametrize("e,scale_e", [(96, 0), (-96, 0), (0, 96), (-48, 90), (20, -60)])
def test_scores_of_large_and_small_factors(torch, R, hd, e, scale_e):
    """Queries times 2^e, keys by 2^(-e - scale_e), the scale times 2^scale_e: the same scores, to the ends of the
    ranges in the header."""
    rng = np.random.default_rng(21)
    T, h = 300, 2
    q = rng.standard_normal((1, R, h, hd))
    kc, ks = ref.quantise(rng.standard_normal((1, h, T, hd)))
    vc, vs = ref.quantise(rng.standard_normal((1, h, T, hd)))
    scale = float(np.float32(hd ** -0.5))
    qt = dev(torch, q).bfloat16()
    out = attend(torch, (qt.double() * 2.0 ** e).bfloat16(), *[dev(torch, a) for a in
                 (kc, (ks.astype(int) - e - scale_e).astype(np.uint8), vc, vs)], scale * 2.0 ** scale_e)
    want, pv, sk = ref.attention(qt.double().cpu().numpy()[0], ref.dequantise(kc, ks)[0], ref.dequantise(vc, vs)[0], [T] * R,
                                 scale)
    # a score's float32 sum of hd products, exp2 and the sums 2^-20; bf16 probabilities and output, 2^-8 each
    tol = (2.0 ** -8 + 2.0 ** -20 + 2 * hd * 2.0 ** -24 * sk) * pv + 2.0 ** -8 * np.abs(want)
    assert (np.abs(out.double().cpu().numpy()[0] - want) <= tol).all()


# --------------------------------------------------------------------------- rotary positions

def turn(torch, spec, rot, pos, layout="half"):
    """(cosine, sine) of every pair at positions pos, in float64."""
    x = torch.zeros(len(pos), 1, rot, device="cuda")
    x[..., :rot // 2] = 1.0
    out = torch.empty_like(x)
    p = dev(torch, np.asarray(pos, dtype=np.int32))
    binding.op_rope(x.data_ptr(), out.data_ptr(), p.data_ptr(), len(pos), 1, rot, "f32", spec)
    o = out.double().cpu().numpy()[:, 0]
    return o[:, :rot // 2], o[:, rot // 2:]


def yarn_rates(rot, theta, factor, orig_len, fast=32.0, slow=1.0):
    """The published ramp: its edges kept within 0 and rot - 1, so that it may end past the last pair."""
    def edge(turns):
        return rot * math.log(orig_len / (turns * 2 * math.pi)) / (2 * math.log(theta))
    lo, hi = max(math.floor(edge(fast)), 0), min(math.ceil(edge(slow)), rot - 1)
    i = np.arange(rot // 2)
    ramp = np.clip((i - lo) / (hi - lo if hi > lo else 0.001), 0, 1)
    f = theta ** (-2.0 * i / rot)
    return f / factor * ramp + f * (1 - ramp)


@pytest.mark.parametrize("rot,theta,orig_len", [(64, 1e4, 65536), (128, 1e4, 65536), (128, 1e4, 1 << 20), (32, 1e4, 131072),
                                                (16, 100.0, 4096), (64, 5e5, 8192), (64, 1e4, 4096)])
@pytest.mark.parametrize("factor", [4.0, 40.0])
def test_ramps_that_end_past_the_last_pair(torch, rot, theta, orig_len, factor):
    pos = np.array([1, 2, 3, 1000, orig_len, 4 * orig_len - 1])
    spec = binding.make_rope(rot, theta=theta, scaling="by_parts", factor=factor, orig_len=orig_len, amplitude=1.0)
    c, s = turn(torch, spec, rot, pos)
    a = pos[:, None] * yarn_rates(rot, theta, factor, orig_len)
    # cosines to 8 float32 roundings; angles of up to 2^22 to some 2^-51 of themselves on both sides
    np.testing.assert_allclose(c, np.cos(a), rtol=0, atol=2.0 ** -20)
    np.testing.assert_allclose(s, np.sin(a), rtol=0, atol=2.0 ** -20)


@pytest.mark.parametrize("rot", [128, 96])
@pytest.mark.parametrize("theta", [1e4, 5e5, 1e8])
def test_far_angles_are_off_by_what_the_header_says(torch, theta, rot):
    """|position| * rate * 2^-49 radians, and the cosine's float32 roundings."""
    getcontext().prec = 60
    pos = [1, -7, 99999, 2 ** 24 + 1, 123456789, 2 ** 31 - 1, -2 ** 31]
    c, s = turn(torch, binding.make_rope(rot, theta=theta), rot, pos)
    two_pi = 2 * Decimal("3.14159265358979323846264338327950288419716939937510582097494")
    for i in range(rot // 2):
        f = (Decimal(theta).ln() * Decimal(-2 * i) / rot).exp()
        for j, n in enumerate(pos):
            a = float((Decimal(n) * f) % two_pi)
            tol = abs(n) * float(f) * 2.0 ** -49 + 4 * 2.0 ** -24
            assert abs(c[j, i] - math.cos(a)) <= tol and abs(s[j, i] - math.sin(a)) <= tol
