"""The 8-bit operators on the GPU against a plain 64-bit restatement
(ops8_ref): quantising, rotary positions, the cache, attention over it and the
block-scaled product, alone and in a run of all of them.

Tolerances count roundings: half a step is 2^-8 of the value in bf16, 2^-11 in
f16, 2^-24 in float32.  Codes and scale bytes have to be equal.
"""
import numpy as np
import pytest

import ops8_ref as ref
from cached_masked_decoding_gb300 import binding
from gpu_util import torch_cuda

pytestmark = pytest.mark.gpu

HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}


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


def same(a, b):
    """Equal, a NaN to a NaN."""
    np.testing.assert_array_equal(a, b)


# --------------------------------------------------------------------------- quantiser

def _spread(rng, rows, K):
    """Rows of many magnitudes, ties and extremes."""
    x = rng.standard_normal((rows, K)) * 2.0 ** rng.uniform(-20, 20, (rows, 1))
    x[0] = 0.0
    if rows > 2:
        x[1] = rng.integers(-30, 31, K) * 0.5          # ties at e4m3's midpoints
        x[1, 0] = 448.0
        x[2] = 0.0
        x[2, K // 2] = -448.0                          # the border of the scale
    if rows > 5:
        x[3, 0] = 2.0 ** 120
        x[4] = 2.0 ** -130 * rng.standard_normal(K)    # subnormal
        x[5, :] = 1.0 + 2.0 ** -7                      # just above a step
    return x


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,K,pad,off", [(1, 16, 0, 0), (7, 128, 0, 0), (33, 688, 0, 0), (6, 272, 8, 0),
                                            (9, 144, 3, 1), (130, 1024, 0, 0)])
def test_quantise_is_bit_exact(torch, rows, K, pad, off, dtype):
    rng = np.random.default_rng(rows + K)
    x = _spread(rng, rows, K)
    if dtype == "f16":
        x = np.clip(x, -60000, 60000)
    buf = torch.zeros(rows * (K + pad) + off, device="cuda", dtype=dt(torch, dtype))
    view = buf[off:].view(rows, K + pad)
    view[:, :K] = dev(torch, x).to(dt(torch, dtype))
    kb = -(-K // 128)
    codes = torch.full((rows, K), 0x55, device="cuda", dtype=torch.uint8)
    scales = torch.full((kb, rows), 0x55, device="cuda", dtype=torch.uint8)
    binding.op_quantise8(view.data_ptr(), dtype, rows, K, codes.data_ptr(), scales.data_ptr(), row_stride=K + pad)
    c, s = ref.quantise_blocks(f64(view[:, :K]))
    same(scales.cpu().numpy(), s)
    got = codes.cpu().numpy()
    same(ref.CODE_VALUES[got], ref.CODE_VALUES[c])


def test_quantise_non_finite_blocks(torch):
    x = torch.ones(5, 256, device="cuda")
    x[0, 3] = float("nan")
    x[1, 200] = float("inf")
    x[2, 130] = float("-inf")
    x[3, 0] = 3.4028234663852886e38
    codes = torch.zeros(5, 256, device="cuda", dtype=torch.uint8)
    scales = torch.zeros(2, 5, device="cuda", dtype=torch.uint8)
    binding.op_quantise8(x.data_ptr(), "f32", 5, 256, codes.data_ptr(), scales.data_ptr())
    s = scales.cpu().numpy()
    assert s[0, 0] == 255 and s[1, 1] == 255 and s[1, 2] == 255
    assert (s != 255).sum() == 7
    c, b = ref.quantise_blocks(f64(x)[3:])
    same(s[:, 3:], b)
    assert (codes.cpu().numpy()[0, :128] == 0).all() and (codes.cpu().numpy()[0, 128:] != 0).all()


# --------------------------------------------------------------------------- rotary positions

ROPES = [
    dict(rot=128, layout="half", scaling="none", factor=1.0),
    dict(rot=64, layout="interleaved", scaling="linear", factor=4.0),
    dict(rot=32, layout="half", scaling="base", factor=8.0),
    dict(rot=64, layout="interleaved", scaling="by_parts", factor=32.0),
    dict(rot=6, layout="interleaved", scaling="none", factor=1.0),
    dict(rot=2, layout="half", scaling="none", factor=1.0),
]


def _rope_check(torch, got, x, pos, case, dtype, theta=1e4):
    rates, amp = ref.rope_rates(case["rot"], theta, case["scaling"], case["factor"])
    want = ref.rope(x, pos, case["rot"], case["layout"], rates, amp)
    # cosine and sine: 1 ulp of sincospif, the angle's and the amplitude's roundings, then a product and a
    # fused sum: under 8 roundings of 2^-24 times |x0| + |x1|; the far angle itself is exact to 2^-30
    other = ref.rope(np.abs(x), np.zeros(len(pos)), case["rot"], case["layout"], rates, amp)
    pair = np.abs(x).max(axis=-1, keepdims=True) * 2
    tol = (8 * 2.0 ** -24) * np.maximum(other, pair) * amp + HALF[dtype] * np.abs(want) * 1.01
    assert (np.abs(got - want) <= tol + 1e-7 * (dtype == "f16")).all(), np.abs(got - want).max()
    same(got[..., case["rot"]:], x[..., case["rot"]:])


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("case", ROPES, ids=lambda c: f"{c['rot']}{c['layout'][0]}-{c['scaling']}")
@pytest.mark.parametrize("rows,heads,hd", [(1, 1, 128), (37, 5, 128), (300, 9, 128)])
def test_rope_matches_fp64(torch, rows, heads, hd, case, dtype):
    rng = np.random.default_rng(rows + heads)
    x = dev(torch, rng.standard_normal((rows, heads, hd))).to(dt(torch, dtype))
    pos = rng.integers(0, 131072, rows).astype(np.int32)
    pos[0] = 0 if rows > 1 else 1048575
    out = torch.full_like(x, 7.0)
    p = dev(torch, pos)
    spec = binding.make_rope(case["rot"], case["layout"], 1e4, case["scaling"], case["factor"])
    binding.op_rope(x.data_ptr(), out.data_ptr(), p.data_ptr(), rows, heads, hd, dtype, spec)
    _rope_check(torch, f64(out), f64(x), pos, case, dtype)
    # in place gives the same bits
    y = x.clone()
    binding.op_rope(y.data_ptr(), y.data_ptr(), p.data_ptr(), rows, heads, hd, dtype, spec)
    assert torch.equal(y, out)


@pytest.mark.parametrize("hd,rot", [(64, 64), (80, 32), (96, 20), (2, 2), (1024, 256), (130, 128)])
def test_rope_head_sizes_positions_and_strides(torch, hd, rot):
    """Odd head sizes; negative and extreme positions; a slice of a wider
    row; head-major memory; an unaligned start."""
    rng = np.random.default_rng(hd)
    rows, heads = 5, 3
    case = dict(rot=rot, layout="half", scaling="none", factor=1.0)
    pos = np.array([-3, 2147483647, -2147483648, 1, 99999], dtype=np.int32)
    p = dev(torch, pos)
    wide = dev(torch, rng.standard_normal((rows, 7 * hd + 1))).to(torch.bfloat16)
    x = wide[:, 1:1 + 2 * heads * hd].unflatten(1, (heads, 2 * hd))[..., :hd]     # heads 2 hd apart
    out = torch.zeros(heads, rows, hd, device="cuda", dtype=torch.bfloat16)       # head-major
    spec = binding.make_rope(rot)
    binding.op_rope(x.data_ptr(), out.data_ptr(), p.data_ptr(), rows, heads, hd, "bf16", spec,
                    x_row_stride=7 * hd + 1, x_head_stride=2 * hd, out_row_stride=hd, out_head_stride=rows * hd)
    _rope_check(torch, f64(out.transpose(0, 1)), f64(x), pos, case, "bf16")


def test_rope_amplitude_and_far_angles(torch):
    x = torch.tensor([1.0, 0.0], device="cuda").repeat(4, 1, 1).contiguous()
    pos = torch.tensor([1000003, 2000003, 123456789, 2147483647], device="cuda", dtype=torch.int32)
    out = torch.empty_like(x)
    binding.op_rope(x.data_ptr(), out.data_ptr(), pos.data_ptr(), 4, 1, 2, "f32",
                    binding.make_rope(2, amplitude=0.5))
    a = pos.double().cpu().numpy()
    got = f64(out)[:, 0]
    # the turns per position carry 64-bit floating point's 2^-53: times 2^31 positions, under 2^-22
    np.testing.assert_allclose(got[:, 0], 0.5 * np.cos(a), atol=2.0 ** -21)
    np.testing.assert_allclose(got[:, 1], 0.5 * np.sin(a), atol=2.0 ** -21)


# --------------------------------------------------------------------------- cache

class Cache:
    def __init__(self, torch, b, h, t, hd, fill=0x5a):
        self.codes = [torch.full((b, h, t, hd), fill, device="cuda", dtype=torch.uint8) for _ in range(2)]
        self.scales = [torch.full((b, h, t), fill, device="cuda", dtype=torch.uint8) for _ in range(2)]
        self.c = binding.make_kv8(self.codes[0].data_ptr(), self.codes[1].data_ptr(), self.scales[0].data_ptr(),
                                  self.scales[1].data_ptr(), b, h, t, hd)

    def values(self, which):
        return ref.dequantise(self.codes[which].cpu().numpy(), self.scales[which].cpu().numpy())


CACHES = [
    # b, R, H_kv, T, hd, starts, counts
    (1, 1, 1, 1, 64, None, None),
    (2, 1, 4, 9, 128, [3, 8], None),
    (3, 5, 3, 17, 64, [0, 12, 14], [5, 0, 5]),         # an empty sequence; the third runs past the end
    (2, 33, 2, 40, 128, [-4, 7], [33, 30]),            # rows before position 0 have no slot
    (1, 70, 8, 70, 128, None, [69]),
    (2, 6, 2, 8, 64, [0, 2], [-1, 99]),                # counts below 0 and above R
]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("b,R,h,T,hd,starts,counts", CACHES)
def test_cache_store_and_load(torch, b, R, h, T, hd, starts, counts, dtype):
    rng = np.random.default_rng(b * R + T)
    width = h * hd + 16
    src = [dev(torch, rng.standard_normal((b * R, width)) * 2.0 ** rng.uniform(-8, 8, (b * R, 1))).to(dt(torch, dtype))
           for _ in range(2)]
    ca = Cache(torch, b, h, T, hd)
    st = None if starts is None else dev(torch, np.array(starts, dtype=np.int32))
    ct = None if counts is None else dev(torch, np.array(counts, dtype=np.int32))
    ptrs = dict(starts_ptr=0 if st is None else st.data_ptr(), counts_ptr=0 if ct is None else ct.data_ptr(),
                k_row_stride=width, v_row_stride=width)
    binding.op_kv8_store(ca.c, src[0].data_ptr(), src[1].data_ptr(), dtype, R, **ptrs)
    back = [torch.full((b * R, width), 3.0, device="cuda", dtype=dt(torch, dtype)) for _ in range(2)]
    binding.op_kv8_load(ca.c, back[0].data_ptr(), back[1].data_ptr(), dtype, R, **ptrs)
    for w in range(2):
        rows = f64(src[w])[:, :h * hd].reshape(b, R, h, hd)
        codes = np.full((b, h, T, hd), 0x5a, dtype=np.uint8)
        scales = np.full((b, h, T), 0x5a, dtype=np.uint8)
        want = np.full((b, R, h, hd), 3.0)
        for s in range(b):
            for i in range(min(R, R if counts is None else counts[s])):
                t = (0 if starts is None else starts[s]) + i
                if 0 <= t < T:
                    codes[s, :, t], scales[s, :, t] = ref.quantise(rows[s, i])
                    want[s, i] = ref.dequantise(codes[s, :, t], scales[s, :, t])
        same(ca.scales[w].cpu().numpy(), scales)
        same(ref.CODE_VALUES[ca.codes[w].cpu().numpy()], ref.CODE_VALUES[codes])
        got = f64(back[w])
        same(got[:, :h * hd].reshape(b, R, h, hd), want)          # code * scale is exact in every type here
        assert (got[:, h * hd:] == 3.0).all()


def test_cache_rows_that_are_not_finite(torch):
    k = torch.ones(4, 1, 64, device="cuda")
    k[1, 0, 5] = float("nan")
    k[2, 0, 63] = float("-inf")
    v = torch.zeros(4, 1, 64, device="cuda")
    ca = Cache(torch, 1, 1, 4, 64)
    binding.op_kv8_store(ca.c, k.data_ptr(), v.data_ptr(), "f32", 4)
    assert ca.scales[0].cpu().numpy().ravel().tolist() == [119, 255, 255, 119]   # 1 = 256 * 2^-8
    assert (ca.scales[1] == 127).all() and (ca.codes[1] == 0).all()
    back = [torch.zeros(4, 64, device="cuda") for _ in range(2)]
    binding.op_kv8_load(ca.c, back[0].data_ptr(), back[1].data_ptr(), "f32", 4)
    assert torch.isnan(back[0][1:3]).all() and (back[0][[0, 3]] == 1).all() and (back[1] == 0).all()


def test_cache_slots_past_32_bits(torch):
    """Positions whose byte offset is over 2^32 land in their own slot."""
    b, h, T, hd = 1, 2, 17_000_000, 128            # 2 x 4.35 GB
    codes = [torch.zeros(b, h, T, hd, device="cuda", dtype=torch.uint8) for _ in range(2)]
    scales = [torch.zeros(b, h, T, device="cuda", dtype=torch.uint8) for _ in range(2)]
    c = binding.make_kv8(codes[0].data_ptr(), codes[1].data_ptr(), scales[0].data_ptr(), scales[1].data_ptr(), b, h, T,
                         hd)
    k = torch.randn(3, h, hd, device="cuda").bfloat16()
    v = torch.randn(3, h, hd, device="cuda").bfloat16()
    st = torch.tensor([T - 3], device="cuda", dtype=torch.int32)
    binding.op_kv8_store(c, k.data_ptr(), v.data_ptr(), "bf16", 3, starts_ptr=st.data_ptr())
    kc, ks = ref.quantise(f64(k))
    same(codes[0][0, :, T - 3:].cpu().numpy(), kc.transpose(1, 0, 2))
    same(scales[0][0, :, T - 3:].cpu().numpy(), ks.T)
    assert int(codes[0][0, :, :4096].max()) == 0 and int(codes[0][0, 1, T - 4].max()) == 0
    # and attention reads them there: a query of zeros weighs all keys alike, and the earlier values are zeros
    q = torch.zeros(1, h, hd, device="cuda", dtype=torch.bfloat16)
    out = torch.zeros_like(q)
    n = binding.attention_kv8_workspace(b, h, h, hd, 1, T)
    ws = torch.empty(max(n, 16), device="cuda", dtype=torch.uint8)
    binding.op_attention_kv8(q.data_ptr(), c, out.data_ptr(), h, 1, ws_ptr=ws.data_ptr(), ws_bytes=n)
    want = ref.dequantise(*ref.quantise(f64(v))).sum(axis=0) / T
    np.testing.assert_allclose(f64(out)[0], want, rtol=2.0 ** -7, atol=0)


# --------------------------------------------------------------------------- attention

def _attention_case(torch, rng, b, R, H, h, T, hd, limits, loud=1.0):
    q = dev(torch, rng.standard_normal((b, R, H, hd))).to(torch.bfloat16)
    ca = Cache(torch, b, h, T, hd)
    for w in range(2):
        x = rng.standard_normal((b, h, T, hd)) * 2.0 ** rng.integers(-3, 4, (b, h, T, 1))
        if w == 0 and loud != 1.0:
            x[:, :, T // 2:] *= loud
        codes, scales = ref.quantise(x)
        ca.codes[w].copy_(dev(torch, codes))
        ca.scales[w].copy_(dev(torch, scales))
    lim = None if limits is None else dev(torch, np.asarray(limits, dtype=np.int32))
    return q, ca, lim


def _attend(torch, q, ca, lim, H, R, scale=None, stream=0):
    b, h, T, hd = ca.codes[0].shape
    out = torch.full((b, R, H, hd), 9.0, device="cuda", dtype=torch.bfloat16)
    n = binding.attention_kv8_workspace(b, H, h, hd, R, T)
    ws = torch.full((max(n, 16),), 0xff, device="cuda", dtype=torch.uint8)      # contents do not matter
    binding.op_attention_kv8(q.data_ptr(), ca.c, out.data_ptr(), H, R, limits_ptr=0 if lim is None else lim.data_ptr(),
                             scale=scale, ws_ptr=ws.data_ptr() if n else 0, ws_bytes=n, stream=stream)
    return out


def _attention_check(got, q, ca, limits, scale, lost=0.0):
    b, R, H, hd = got.shape
    k, v = ca.values(0), ca.values(1)
    for s in range(b):
        lim = [k.shape[2]] * R if limits is None else limits[s]
        want, pv, sk = ref.attention(q[s], k[s], v[s], lim, scale)
        # a score: hd products summed in float32, under hd * 2^-24 of sum |q||k|, moves p by as much, the sum
        # too; exp2 and the sums 2^-20; P rounded to bf16: 2^-8 of sum p|v|; the output: 2^-8 of itself
        tol = (2.0 ** -8 + 2.0 ** -20 + 2 * hd * 2.0 ** -24 * sk) * pv + 2.0 ** -8 * np.abs(want) + lost
        err = np.abs(got[s] - want)
        assert (err <= tol).all(), f"seq {s}: {(err / (tol + 1e-300)).max():.2f} of the tolerance"


def _causal(b, R, T, lens=None):
    return [[(T if lens is None else lens[s]) - R + i + 1 for i in range(R)] for s in range(b)]


ATTENTIONS = [
    # b, R, H, H_kv, T, hd, limits
    (1, 1, 1, 1, 1, 64, None),
    (1, 1, 1, 1, 1, 128, [[1]]),
    (2, 1, 8, 2, 65, 128, [[65], [1]]),
    (3, 1, 8, 8, 200, 64, [[200], [0], [63]]),                      # a finished sequence sees nothing
    (1, 1, 32, 1, 513, 128, None),                                  # one cached head for all
    (2, 3, 6, 2, 130, 128, [[130, 129, 128], [5, 300, -7]]),        # over T counts as T, below 0 as nothing
    (1, 16, 4, 4, 96, 64, None),                                    # the tiny model's block
    (1, 32, 4, 4, 768, 128, None),                                  # a DualCache block
    (2, 17, 4, 2, 127, 128, _causal(2, 17, 127, [127, 60])),
    (1, 70, 4, 2, 70, 128, _causal(1, 70, 70)),                     # causal from an empty cache
    (1, 65, 2, 1, 64, 64, _causal(1, 65, 64)),                      # the first row sees nothing
    (2, 129, 3, 3, 191, 64, _causal(2, 129, 191, [191, 100])),      # rows before the first key see nothing
    (1, 256, 2, 2, 320, 128, _causal(1, 256, 320)),
    (1, 200, 2, 1, 129, 128, None),
    (1, 100, 1, 1, 1500, 128, [[(37 * i) % 1501 for i in range(100)]]),   # limits in any order
    (1, 4, 16, 16, 4097, 128, _causal(1, 4, 4097)),
]


@pytest.mark.parametrize("b,R,H,h,T,hd,limits", ATTENTIONS, ids=lambda x: None if isinstance(x, list) else str(x))
def test_attention_matches_fp64(torch, b, R, H, h, T, hd, limits):
    rng = np.random.default_rng(R + H + T)
    q, ca, lim = _attention_case(torch, rng, b, R, H, h, T, hd, limits)
    out = _attend(torch, q, ca, lim, H, R)
    got = f64(out)
    _attention_check(got, f64(q), ca, limits, hd ** -0.5)
    if limits is not None:
        for s in range(b):
            for i in range(R):
                if limits[s][i] <= 0:
                    assert (got[s, i] == 0).all()
    # the same bits again
    assert torch.equal(out, _attend(torch, q, ca, lim, H, R))
    assert binding.op_check() == 0


@pytest.mark.parametrize("R", [1, 32, 128])
@pytest.mark.parametrize("hd", [64, 128])
def test_attention_peaked_rows(torch, hd, R):
    """Later keys score far higher (the running maximum moves by hundreds), and a
    scale other than 1/sqrt(hd)."""
    rng = np.random.default_rng(3)
    q, ca, lim = _attention_case(torch, rng, 1, R, 4, 2, 700, hd, None, loud=64.0)
    got = f64(_attend(torch, q, ca, lim, 4, R, scale=0.3))
    _attention_check(got, f64(q), ca, None, 0.3)


@pytest.mark.parametrize("R", [1, 128])
def test_attention_one_loud_key_does_not_hide_the_rest(torch, R):
    """One key 13 nats above 20,000 others: the others together hold several
    per cent of the weight and must not be rounded away."""
    T, hd = 20001, 64
    q = torch.zeros(1, R, 1, hd, device="cuda", dtype=torch.bfloat16)
    q[..., 0] = 1.0
    ca = Cache(torch, 1, 1, T, hd, fill=0)
    k = np.zeros((T, hd))
    k[0, 0] = 13.0
    v = np.ones((T, hd))
    v[0] = 0.0
    for w, x in enumerate((k, v)):
        codes, scales = ref.quantise(x)
        ca.codes[w].copy_(dev(torch, codes[None, None]))
        ca.scales[w].copy_(dev(torch, scales[None, None]))
    got = f64(_attend(torch, q, ca, None, 1, R, scale=1.0))
    rest = 20000 * np.exp(-13.0)
    np.testing.assert_allclose(got, rest / (1 + rest), rtol=2.0 ** -7)


@pytest.mark.parametrize("R,H,h", [(1, 8, 2), (32, 4, 4), (130, 2, 1)])
@pytest.mark.parametrize("hd", [64, 128])
def test_attention_value_scales_of_any_size(torch, hd, R, H, h):
    """Scales from 2^-100 to 2^100 within one tile of keys."""
    rng = np.random.default_rng(4)
    T = 150
    q, ca, _ = _attention_case(torch, rng, 1, R, H, h, T, hd, None)
    e = rng.choice([27, 100, 127, 134, 135, 200, 227], (1, h, T)).astype(np.uint8)
    ca.scales[1].copy_(dev(torch, e))
    got = f64(_attend(torch, q, ca, None, H, R))
    _attention_check(got, f64(q), ca, None, hd ** -0.5)
    # and all small, so that the large ones do not cover them
    ca.scales[1].copy_(dev(torch, np.where(e > 100, 27, 20).astype(np.uint8)))
    got = f64(_attend(torch, q, ca, None, H, R))
    _attention_check(got, f64(q), ca, None, hd ** -0.5)


@pytest.mark.parametrize("R,H,h", [(1, 8, 2), (1, 16, 1), (32, 4, 4), (64, 1, 1), (130, 2, 1)])
@pytest.mark.parametrize("hd", [64, 128])
def test_attention_values_that_grow_or_vanish(torch, hd, R, H, h):
    """Value scales far below 1 in the first tiles of keys and far above it in the
    last, and the other way round; scores that grow with them."""
    rng = np.random.default_rng(13)
    T = 600
    for lo, hi in ((20, 230), (230, 20), (27, 227)):
        q, ca, _ = _attention_case(torch, rng, 1, R, H, h, T, hd, None, loud=8.0)
        e = np.full((1, h, T), lo, dtype=np.uint8)
        e[:, :, 400:] = hi
        e[:, :, 500] = 127
        ca.scales[1].copy_(dev(torch, e))
        got = f64(_attend(torch, q, ca, None, H, R))
        # the sums are float32 in units of the largest value scale: each of T products loses at most
        # 2^-126 of it to underflow, T * 448 * 2^-126 < 2^-100
        _attention_check(got, f64(q), ca, None, hd ** -0.5, lost=2.0 ** (max(lo, hi) - 127 - 100))


@pytest.mark.parametrize("R,H,h,T,loud", [(200, 20, 5, 700, 1.0), (257, 12, 3, 1025, 1.0), (1, 2, 2, 16384, 8.0),
                                          (16, 1, 1, 16384, 8.0)])
@pytest.mark.parametrize("hd", [64, 128])
def test_attention_splits_of_large_values_and_sums(torch, hd, R, H, h, T, loud):
    """Values up to 2^111 and scores far above the first keys' in every split: a split's sum times
    its output is out of float32's range, the joined row is not."""
    rng = np.random.default_rng(16)
    q, ca, _ = _attention_case(torch, rng, 1, R, H, h, T, hd, None, loud=loud)
    assert binding.attention_kv8_workspace(1, H, h, hd, R, T) > 0
    ca.scales[1].copy_(dev(torch, rng.integers(20, 231, (1, h, T)).astype(np.uint8)))
    got = f64(_attend(torch, q, ca, None, H, R, scale=0.3))
    # the sums are float32 in units of the largest value scale: T * 448 * 2^-126 of it < 2^-100 underflows; in the
    # few-row kernel a probability is off by 2^-21 of the largest p 2^ev near it, times a code
    _attention_check(got, f64(q), ca, None, 0.3, lost=2.0 ** 3 + (2.0 ** -21 * 2.0 ** 103 * 448 if R * H // h <= 64 else 0))


@pytest.mark.parametrize("b,R,h,hd", [(4, 100, 80, 64), (2, 200, 80, 128)])
def test_attention_many_heads_leave_the_keys_whole(torch, b, R, h, hd):
    """So many rows that one walk has all keys of a head: once, and (scores and value
    scales that grow) a second time."""
    rng = np.random.default_rng(15)
    T = 450
    limits = _causal(b, R, T, [T - 60 * s for s in range(b)])
    for loud, hi in ((1.0, 127), (64.0, 230)):
        q, ca, lim = _attention_case(torch, rng, b, R, h, h, T, hd, limits, loud=loud)
        assert binding.attention_kv8_workspace(b, h, h, hd, R, T) == 0
        e = np.full((b, h, T), 127, dtype=np.uint8)
        e[:, ::2, 300:] = hi
        ca.scales[1].copy_(dev(torch, e))
        out = _attend(torch, q, ca, lim, h, R)
        # products under 2^-126 of the largest value scale are lost in float32 (a probability of 2^-400
        # in float64 is nothing here), T * 448 * 2^-126 < 2^-100
        _attention_check(f64(out), f64(q), ca, limits, hd ** -0.5, lost=2.0 ** (hi - 127 - 100))
        assert torch.equal(out, _attend(torch, q, ca, lim, h, R))


@pytest.mark.parametrize("R,H,h", [(1, 8, 2), (16, 4, 4), (140, 2, 1)])
@pytest.mark.parametrize("hd", [64, 128])
def test_attention_ignores_what_lies_behind_the_limits(torch, hd, R, H, h):
    """Codes of every bit pattern and scale bytes of every value past the last
    limit; NaN rows that only some rows see."""
    rng = np.random.default_rng(5)
    T, n = 200, 133
    limits = [[max(1, n - (i % 40)) for i in range(R)]]
    q, ca, lim = _attention_case(torch, rng, 1, R, H, h, T, hd, limits)
    for w in range(2):
        ca.codes[w][:, :, n:] = dev(torch, rng.integers(0, 256, (1, h, T - n, hd)).astype(np.uint8))
        ca.codes[w][:, :, n] = 0x7f
        ca.codes[w][:, :, n + 1] = 0xff
        ca.scales[w][:, :, n:] = dev(torch, rng.integers(0, 256, (1, h, T - n)).astype(np.uint8))
        ca.scales[w][:, :, n:n + 2] = 255
    got = f64(_attend(torch, q, ca, lim, H, R))
    k, v = ca.values(0)[0, :, :n], ca.values(1)[0, :, :n]
    want, pv, sk = ref.attention(f64(q)[0], k, v, limits[0], hd ** -0.5)
    tol = (2.0 ** -8 + 2.0 ** -20 + 2 * hd * 2.0 ** -24 * sk) * pv + 2.0 ** -8 * np.abs(want)
    assert (np.abs(got[0] - want) <= tol).all()
    # a NaN key or value row: rows that see it are NaN, the others unchanged
    for w in range(2):
        keep = ca.scales[w][:, :, n - 10].clone()
        ca.scales[w][:, :, n - 10] = 255
        ca.codes[w][:, :, n - 10] = 0
        bad = f64(_attend(torch, q, ca, lim, H, R))[0]
        for i in range(R):
            if limits[0][i] > n - 10:
                assert np.isnan(bad[i]).all()
            else:
                same(bad[i], got[0, i])
        ca.scales[w][:, :, n - 10] = keep
        break_codes = ref.quantise(rng.standard_normal((1, h, hd)))[0]
        ca.codes[w][:, :, n - 10] = dev(torch, break_codes)
        got = f64(_attend(torch, q, ca, lim, H, R))


def test_attention_queries_that_are_not_finite(torch):
    rng = np.random.default_rng(6)
    for R in (2, 130):
        q, ca, _ = _attention_case(torch, rng, 1, R, 4, 2, 90, 64, None)
        clean = f64(_attend(torch, q, ca, None, 4, R))
        q[0, 1, 2, 7] = float("nan")
        q[0, 0, 3, 0] = float("inf")
        got = f64(_attend(torch, q, ca, None, 4, R))
        assert np.isnan(got[0, 1, 2]).all()
        assert np.isnan(got[0, 0, 3]).any()
        got[0, 1, 2], got[0, 0, 3] = clean[0, 1, 2], clean[0, 0, 3]
        same(got, clean)


def test_attention_tiny_and_huge_queries(torch):
    """Query rows from 2^-60 to 2^60 (elements far apart within a row too)."""
    rng = np.random.default_rng(7)
    for R in (1, 80):
        q, ca, _ = _attention_case(torch, rng, 1, R, 2, 2, 100, 128, None)
        mag = dev(torch, 2.0 ** rng.uniform(-12, 0, (1, R, 2, 128)))
        for e in (-60, 0, 60):
            qq = (q.double() * mag * 2.0 ** e).to(torch.bfloat16)
            sc = float(2.0 ** -e * 128 ** -0.5)
            got = f64(_attend(torch, qq, ca, None, 2, R, scale=sc))
            _attention_check(got, f64(qq), ca, None, np.float64(np.float32(sc)))


def test_attention_strided_rows_and_workspace(torch):
    rng = np.random.default_rng(8)
    b, R, H, h, T, hd = 2, 3, 8, 2, 5000, 64
    q, ca, _ = _attention_case(torch, rng, b, R, H, h, T, hd, None)
    dense = _attend(torch, q, ca, None, H, R)
    qw = torch.full((b * R, H * hd + 24), float("nan"), device="cuda", dtype=torch.bfloat16)
    qw[:, :H * hd] = q.view(b * R, -1)
    ow = torch.full((b * R, H * hd + 40), 5.0, device="cuda", dtype=torch.bfloat16)
    n = binding.attention_kv8_workspace(b, H, h, hd, R, T)
    assert n > 0                                        # few rows, many keys: the keys are split
    ws = torch.empty(n, device="cuda", dtype=torch.uint8)
    binding.op_attention_kv8(qw.data_ptr(), ca.c, ow.data_ptr(), H, R, ws_ptr=ws.data_ptr(), ws_bytes=n,
                             q_row_stride=H * hd + 24, out_row_stride=H * hd + 40)
    assert torch.equal(ow[:, :H * hd].reshape(b, R, H, hd), dense) and (ow[:, H * hd:] == 5.0).all()
    for bad in [dict(ws_ptr=0, ws_bytes=n), dict(ws_ptr=ws.data_ptr(), ws_bytes=n - 1),
                dict(ws_ptr=ws.data_ptr() + 8, ws_bytes=n)]:
        with pytest.raises(binding.DllmError) as e:
            binding.op_attention_kv8(q.data_ptr(), ca.c, ow.data_ptr(), H, R, **bad)
        assert e.value.status == binding.EINVAL and "workspace" in str(e.value)


# --------------------------------------------------------------------------- product

PRODUCTS = [
    # M, N, K
    (1, 1, 16), (5, 3, 48), (128, 32, 128), (130, 33, 144), (256, 1, 4096), (2048, 16, 2048), (688, 40, 256),
    (256, 7, 688), (300, 129, 1040), (512, 200, 512), (1024, 300, 384), (97, 513, 4096), (4096, 32, 5504),
    (3000, 1201, 272), (12300, 400, 144), (2049, 2000, 656),     # tiles of CTA pairs, ragged in every direction
]


def _product_check(y, xc, xs, wc, ws, out):
    x, w = ref.dequantise_blocks(xc, xs), ref.dequantise_blocks(wc, ws)
    want, bound = x @ w.T, np.abs(x) @ np.abs(w).T
    # products of codes are exact; a float32 sum taken 32 products at a time, each step rounded or cut to
    # 24 bits (2^-23): K/32 steps, and up to 16 partial sums joined
    steps = x.shape[1] // 32 + 16
    tol = steps * 2.0 ** -23 * bound + HALF[out] * np.abs(want)
    err = np.abs(y - want)
    assert (err <= tol).all(), f"{(err / (tol + 1e-300)).max():.2f} of the tolerance"


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("M,N,K", PRODUCTS)
def test_product_matches_fp64(torch, M, N, K, out):
    rng = np.random.default_rng(M + N + K)
    x = rng.standard_normal((N, K)) * 2.0 ** rng.integers(-6, 7, (N, 1))
    x[:, :: 37] *= 30.0
    w = rng.standard_normal((M, K)) * 2.0 ** rng.integers(-6, 7, (M, 1))
    (xc, xs), (wc, ws) = ref.quantise_blocks(x), ref.quantise_blocks(w)
    t = [dev(torch, a) for a in (wc, ws, xc, xs)]
    y = torch.full((N + 1, M), 4.0, device="cuda", dtype=dt(torch, out))
    binding.op_gemm8(*(a.data_ptr() for a in t), y.data_ptr(), out, M, N, K)
    assert binding.op_check() == 0
    _product_check(f64(y[:N]), xc, xs, wc, ws, out)
    assert (y[N] == 4.0).all()
    y2 = torch.zeros_like(y)
    binding.op_gemm8(*(a.data_ptr() for a in t), y2.data_ptr(), out, M, N, K)
    assert torch.equal(y[:N], y2[:N])


@pytest.mark.parametrize("N", [3, 150])
def test_product_scales_of_any_size_and_non_finite_blocks(torch, N):
    rng = np.random.default_rng(9)
    M, K = 140, 400
    xc, xs = ref.quantise_blocks(rng.standard_normal((N, K)))
    wc, ws = ref.quantise_blocks(rng.standard_normal((M, K)))
    xs = rng.choice([87, 127, 167], xs.shape).astype(np.uint8)
    ws = rng.choice([87, 127, 167], ws.shape).astype(np.uint8)
    t = [dev(torch, a) for a in (wc, ws, xc, xs)]
    y = torch.zeros(N, M, device="cuda")
    binding.op_gemm8(*(a.data_ptr() for a in t), y.data_ptr(), "f32", M, N, K)
    _product_check(f64(y), xc, xs, wc, ws, "f32")
    clean = f64(y)
    t[3][2, 1] = 255
    t[1][3, 5] = 255
    binding.op_gemm8(*(a.data_ptr() for a in t), y.data_ptr(), "f32", M, N, K)
    got = f64(y)
    assert np.isnan(got[1]).all() and np.isnan(got[:, 5]).all()
    got[1], got[:, 5] = clean[1], clean[:, 5]
    same(got, clean)


# --------------------------------------------------------------------------- together

def _layer(torch, rng, b, R, H, h, T, hd, d):
    """Weights, cache and buffers of one attention layer in 8 bits."""
    width = (H + 2 * h) * hd
    g = {}
    for name, (m, k) in {"qkv": (width, d), "o": (d, H * hd)}.items():
        w = dev(torch, rng.standard_normal((m, k)) / np.sqrt(k)).to(torch.bfloat16)
        g[name] = (torch.empty(m, k, device="cuda", dtype=torch.uint8),
                   torch.empty(-(-k // 128), m, device="cuda", dtype=torch.uint8))
        binding.op_quantise8(w.data_ptr(), "bf16", m, k, g[name][0].data_ptr(), g[name][1].data_ptr())
    g["cache"] = Cache(torch, b, h, T, hd, fill=0xff)
    g["x"] = torch.zeros(b * R, d, device="cuda", dtype=torch.bfloat16)
    g["xq"] = [(torch.empty(b * R, k, device="cuda", dtype=torch.uint8),
                torch.empty(-(-k // 128), b * R, device="cuda", dtype=torch.uint8)) for k in (d, H * hd)]
    g["qkv_out"] = torch.zeros(b * R, width, device="cuda", dtype=torch.bfloat16)
    g["att"] = torch.zeros(b * R, H * hd, device="cuda", dtype=torch.bfloat16)
    g["y"] = torch.zeros(b * R, d, device="cuda")
    g["pos"] = torch.zeros(b * R, device="cuda", dtype=torch.int32)
    g["starts"] = torch.zeros(b, device="cuda", dtype=torch.int32)
    g["counts"] = torch.zeros(b, device="cuda", dtype=torch.int32)
    g["limits"] = torch.zeros(b, R, device="cuda", dtype=torch.int32)
    n = binding.attention_kv8_workspace(b, H, h, hd, R, T)
    g["ws"] = torch.empty(max(16, n), device="cuda", dtype=torch.uint8)
    g["rope"] = binding.make_rope(hd)
    return g


def _forward(g, b, R, H, h, hd, d, stream):
    width = (H + 2 * h) * hd
    qkv = g["qkv_out"].data_ptr()
    (xc, xs), (ac, as_) = g["xq"]
    binding.op_quantise8(g["x"].data_ptr(), "bf16", b * R, d, xc.data_ptr(), xs.data_ptr(), stream=stream)
    binding.op_gemm8(g["qkv"][0].data_ptr(), g["qkv"][1].data_ptr(), xc.data_ptr(), xs.data_ptr(), qkv, "bf16", width,
                     b * R, d, stream=stream)
    # queries and keys lie side by side in a row: one call turns both, in place
    binding.op_rope(qkv, qkv, g["pos"].data_ptr(), b * R, H + h, hd, "bf16", g["rope"], x_row_stride=width,
                    out_row_stride=width, stream=stream)
    binding.op_kv8_store(g["cache"].c, qkv + 2 * H * hd, qkv + 2 * (H + h) * hd, "bf16", R,
                         starts_ptr=g["starts"].data_ptr(), counts_ptr=g["counts"].data_ptr(), k_row_stride=width,
                         v_row_stride=width, stream=stream)
    binding.op_attention_kv8(qkv, g["cache"].c, g["att"].data_ptr(), H, R, limits_ptr=g["limits"].data_ptr(),
                             ws_ptr=g["ws"].data_ptr(), ws_bytes=g["ws"].numel(), q_row_stride=width, stream=stream)
    binding.op_quantise8(g["att"].data_ptr(), "bf16", b * R, H * hd, ac.data_ptr(), as_.data_ptr(), stream=stream)
    binding.op_gemm8(g["o"][0].data_ptr(), g["o"][1].data_ptr(), ac.data_ptr(), as_.data_ptr(), g["y"].data_ptr(),
                     "f32", d, b * R, H * hd, stream=stream)


def _set_step(torch, g, lens, R, rng, b, d):
    """Rows of the next chunk: counts[s] new rows after lens[s], causal limits."""
    counts = [R if s == 0 else R - 1 for s in range(b)]
    g["x"].copy_(dev(torch, rng.standard_normal((b * R, d))))
    g["pos"].copy_(dev(torch, np.array([[n + i for i in range(R)] for n in lens], dtype=np.int32).ravel()))
    g["starts"].copy_(dev(torch, np.array(lens, dtype=np.int32)))
    g["counts"].copy_(dev(torch, np.array(counts, dtype=np.int32)))
    lim = [[n + i + 1 if i < c else 0 for i in range(R)] for n, c in zip(lens, counts)]
    g["limits"].copy_(dev(torch, np.array(lim, dtype=np.int32)))
    return [n + c for n, c in zip(lens, counts)], lim


@pytest.mark.parametrize("hd,H,h", [(64, 4, 2), (128, 2, 2)])
def test_a_layer_decodes_through_all_of_them(torch, hd, H, h):
    """Prefill, then chunks, then single tokens of a padded batch of two: each
    call's output against the formula on what the call before gave."""
    b, T, d = 2, 60, 256
    rng = np.random.default_rng(10)
    lens = [0, 0]
    for R in (33, 4, 2, 1):
        g_new = _layer(torch, np.random.default_rng(11), b, R, H, h, T, hd, d)
        if lens != [0, 0]:
            g_new["cache"] = g["cache"]
        g = g_new
        if R == 1:
            lens_next, lim = _set_step(torch, g, lens, 1, rng, b, d)     # the second sequence has no row: it ended
        else:
            lens_next, lim = _set_step(torch, g, lens, R, rng, b, d)
        _forward(g, b, R, H, h, hd, d, 0)
        torch.cuda.synchronize()
        assert binding.op_check() == 0
        (xc, xs), (ac, as_) = [(c.cpu().numpy(), s.cpu().numpy()) for c, s in g["xq"]]
        c, s = ref.quantise_blocks(f64(g["x"]))
        same(ref.CODE_VALUES[xc], ref.CODE_VALUES[c])
        same(xs, s)
        wq = [a.cpu().numpy() for a in g["qkv"]]
        raw = ref.dequantise_blocks(xc, xs) @ ref.dequantise_blocks(*wq).T
        qkv = f64(g["qkv_out"]).reshape(b * R, H + 2 * h, hd)
        rates, amp = ref.rope_rates(hd, 1e4, "none", 1.0)
        turned = ref.rope(raw.reshape(b * R, H + 2 * h, hd), g["pos"].cpu().numpy(), hd, "half", rates, amp)
        # the projection rounded to bf16 (2^-8 of it, both elements of a pair), turned, rounded again
        big = np.abs(raw).reshape(b * R, H + 2 * h, hd)
        pair = big + np.roll(big, hd // 2, axis=-1)
        assert (np.abs(qkv[:, :H + h] - turned[:, :H + h]) <= 2.0 ** -7 * 1.01 * pair[:, :H + h] + 1e-4).all()
        assert (np.abs(qkv[:, H + h:] - raw.reshape(b * R, H + 2 * h, hd)[:, H + h:]) <= 2.0 ** -7 * big[:, H + h:] + 1e-4).all()
        for w, off in ((0, H), (1, H + h)):
            rows = qkv.reshape(b, R, H + 2 * h, hd)[:, :, off:off + h]
            vals = g["cache"].values(w)
            for s_ in range(b):
                n = lens_next[s_] - lens[s_]
                c, sc = ref.quantise(rows[s_, :n])
                same(vals[s_, :, lens[s_]:lens_next[s_]], ref.dequantise(c, sc).transpose(1, 0, 2))
        att = f64(g["att"]).reshape(b, R, H, hd)
        _attention_check_padded(att, qkv.reshape(b, R, H + 2 * h, hd)[:, :, :H], g["cache"], lim, hd ** -0.5)
        _product_check(f64(g["y"]), ac, as_, *[a.cpu().numpy() for a in g["o"]], "f32")
        lens = lens_next


def _attention_check_padded(got, q, ca, limits, scale):
    k, v = ca.values(0), ca.values(1)
    for s in range(got.shape[0]):
        n = max(max(limits[s]), 0)
        want, pv, sk = ref.attention(q[s], k[s, :, :n], v[s, :, :n], limits[s], scale)
        tol = (2.0 ** -8 + 2.0 ** -20 + 2 * q.shape[-1] * 2.0 ** -24 * sk) * pv + 2.0 ** -8 * np.abs(want)
        assert (np.abs(got[s] - want) <= tol).all()


def test_two_graphs_and_two_streams(torch):
    """Two layers captured into a graph each, replayed on two streams at once and
    with new inputs: the same bits as one after the other without graphs."""
    b, R, H, h, T, hd, d = 2, 3, 8, 2, 4096, 128, 256
    rng = np.random.default_rng(12)
    layers = [_layer(torch, np.random.default_rng(20 + i), b, R, H, h, T, hd, d) for i in range(2)]
    for g in layers:
        for w in range(2):
            codes = dev(torch, rng.integers(0, 0x7e, tuple(g["cache"].codes[w].shape)).astype(np.uint8))
            g["cache"].codes[w].copy_(codes)
            g["cache"].scales[w].fill_(119)
        _set_step(torch, g, [4000, 77], R, rng, b, d)
    torch.cuda.synchronize()
    side = [torch.cuda.Stream() for _ in range(2)]
    graphs = []
    for g, s in zip(layers, side):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=s):
            _forward(g, b, R, H, h, hd, d, s.cuda_stream)
        graphs.append(gr)
    for _ in range(3):
        for g in layers:
            g["x"].copy_(dev(torch, rng.standard_normal((b * R, d))))
        torch.cuda.synchronize()
        want = []
        for g in layers:
            _forward(g, b, R, H, h, hd, d, 0)
            torch.cuda.synchronize()
            want.append((g["y"].clone(), g["att"].clone()))
            g["y"].zero_()
            g["att"].zero_()
        torch.cuda.synchronize()
        for gr, s in zip(graphs, side):
            with torch.cuda.stream(s):
                gr.replay()
                gr.replay()
        torch.cuda.synchronize()
        for g, (y, att) in zip(layers, want):
            assert torch.equal(g["y"], y) and torch.equal(g["att"], att)
    assert binding.op_check() == 0


FIRST_CALLS = """
import numpy as np
import torch
from cached_masked_decoding_gb300 import binding

def forward(s):
    rope = binding.make_rope(hd)
    binding.op_quantise8(x.data_ptr(), "bf16", N, K, xc.data_ptr(), xs.data_ptr(), stream=s)
    for n, y in ys.items():
        binding.op_gemm8(wc.data_ptr(), ws.data_ptr(), xc.data_ptr(), xs.data_ptr(), y.data_ptr(), "bf16", M, n, K, stream=s)
    binding.op_rope(q.data_ptr(), q.data_ptr(), pos.data_ptr(), T, H, hd, "bf16", rope, stream=s)
    binding.op_kv8_store(cache, kv[0].data_ptr(), kv[1].data_ptr(), "bf16", T, stream=s)
    binding.op_kv8_load(cache, back[0].data_ptr(), back[1].data_ptr(), "bf16", T, stream=s)
    for r, (o, w) in outs.items():
        binding.op_attention_kv8(q.data_ptr(), cache, o.data_ptr(), H, r, ws_ptr=w.data_ptr(), ws_bytes=w.numel(), stream=s)

torch.manual_seed(0)
M, N, K, H, T, hd = 4096, 800, 512, 2, 600, 128
z = lambda *s, t=torch.uint8: torch.zeros(*s, device="cuda", dtype=t)
x = torch.randn(N, K, device="cuda").to(torch.bfloat16)
wc = torch.randint(0, 0x7e, (M, K), device="cuda", dtype=torch.uint8)
ws = torch.full((K // 128, M), 120, device="cuda", dtype=torch.uint8)
xc, xs = z(N, K), z(K // 128, N)
ys = {n: z(n, M, t=torch.bfloat16) for n in (1, 50, 100, N)}
pos = torch.arange(T, device="cuda", dtype=torch.int32)
q0 = torch.randn(T, H, hd, device="cuda").to(torch.bfloat16)
q = q0.clone()
kv = torch.randn(2, T, 1, hd, device="cuda").to(torch.bfloat16)
back = torch.zeros_like(kv)
kc, ks = z(2, 1, 1, T, hd), z(2, 1, 1, T)
cache = binding.make_kv8(kc[0].data_ptr(), kc[1].data_ptr(), ks[0].data_ptr(), ks[1].data_ptr(), 1, 1, T, hd)
outs = {r: (z(r, H, hd, t=torch.bfloat16), z(max(binding.attention_kv8_workspace(1, H, 1, hd, r, T), 16)))
        for r in (1, 8, 16, 32, 64, 300)}
torch.cuda.synchronize()
s = torch.cuda.Stream()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g, stream=s):
    forward(s.cuda_stream)
g.replay()
torch.cuda.synchronize()
tensors = [xc, xs, *ys.values(), q, kc, ks, back, *[o for o, _ in outs.values()]]
got = [t.clone() for t in tensors]
assert all(t.float().abs().sum() > 0 for t in got)
for t in tensors:
    t.zero_()
q.copy_(q0)
forward(0)
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, tensors))
assert binding.op_check() == 0
print("same")
"""


def test_first_calls_of_a_process_can_be_captured(torch):
    """Every kernel's first launch inside a capture, in a process of its own: the same bits
    as launched directly."""
    import subprocess
    import sys
    from pathlib import Path
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS], cwd=Path(__file__).resolve().parent.parent,
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "same", r.stdout[-500:] + r.stderr[-2000:]
