"""Refusals of the 8-bit entry points: every check precedes any device call, so
these run without a GPU (the pointers are never dereferenced)."""
import ctypes
import os

import numpy as np
import pytest

import ops8_ref as ref
from cached_masked_decoding_gb300 import binding

A = 1 << 20     # a 16-byte aligned address that nothing reads


@pytest.fixture(scope="module", autouse=True)
def built():
    if not os.path.exists(binding.LIB_PATH):
        from cached_masked_decoding_gb300 import build
        build.build()


def refused(fn, *args, text=None, **kw):
    with pytest.raises(binding.DllmError) as e:
        fn(*args, **kw)
    assert e.value.status == binding.EINVAL
    if text:
        assert text in str(e.value)


ROPE_BAD = [
    dict(rot_dim=0), dict(rot_dim=7), dict(rot_dim=130), dict(rot_dim=-2),
    dict(rot_dim=64, theta=0.5), dict(rot_dim=64, theta=float("nan")), dict(rot_dim=64, theta=float("inf")),
    dict(rot_dim=64, scaling="linear", factor=0.5), dict(rot_dim=64, scaling="linear", factor=float("nan")),
    dict(rot_dim=2, scaling="base", factor=2.0),
    dict(rot_dim=64, scaling="by_parts", factor=2.0, orig_len=0.0),
    dict(rot_dim=64, scaling="by_parts", factor=2.0, beta_slow=0.0),
    dict(rot_dim=64, scaling="by_parts", factor=2.0, beta_fast=0.5),
    dict(rot_dim=64, scaling="by_parts", factor=2.0, theta=1.0),
    dict(rot_dim=64, amplitude=-1.0), dict(rot_dim=64, amplitude=float("inf")),
]


@pytest.mark.parametrize("spec", ROPE_BAD, ids=lambda s: ",".join(f"{k}={v}" for k, v in s.items()))
def test_rope_refuses_bad_rotations(spec):
    refused(binding.op_rope, A, A + 4096, A, 4, 2, 128, "bf16", binding.make_rope(**spec))


def test_rope_refuses_bad_arguments():
    r = binding.make_rope(64)
    for args in [(0, A, A, 4, 2, 128), (A, 0, A, 4, 2, 128), (A, A, 0, 4, 2, 128), (A, A, A, 0, 2, 128),
                 (A, A, A, 4, 0, 128), (A, A, A, 4, 2, 127), (A, A, A, 4, 2, 2048), (A + 1, A, A, 4, 2, 128),
                 (A, A, A + 2, 4, 2, 128)]:
        refused(binding.op_rope, *args, "bf16", r)
    # rows that overlap, heads that overlap, negative and huge strides
    refused(binding.op_rope, A, 2 * A, A, 4, 2, 128, "bf16", r, x_row_stride=128, text="overlap")
    refused(binding.op_rope, A, 2 * A, A, 4, 2, 128, "bf16", r, out_head_stride=64, text="overlap")
    refused(binding.op_rope, A, 2 * A, A, 4, 2, 128, "bf16", r, x_row_stride=-256, text="out of range")
    refused(binding.op_rope, A, 2 * A, A, 4, 2, 128, "bf16", r, out_row_stride=1 << 40, text="out of range")
    # in place with other strides
    refused(binding.op_rope, A, A, A, 4, 2, 128, "bf16", r, out_row_stride=512, text="in place")
    L = binding.lib()
    assert L.dllm_op_rope(A, A, A, 4, 2, 128, 0, 0, 0, 0, 3, r, None) == binding.EINVAL      # no such type
    assert L.dllm_op_rope(A, A, A, 4, 2, 128, 0, 0, 0, 0, 1, None, None) == binding.EINVAL
    bad = binding.make_rope(64)
    bad.layout = 2
    refused(binding.op_rope, A, A, A, 4, 2, 128, "bf16", bad)
    bad = binding.make_rope(64)
    bad.scaling = 4
    refused(binding.op_rope, A, A, A, 4, 2, 128, "bf16", bad)


def cache(k=A, v=A, ks=A, vs=A, b=2, h=4, t=64, hd=128):
    return binding.make_kv8(k, v, ks, vs, b, h, t, hd)


CACHE_BAD = [dict(k=0), dict(v=0), dict(ks=0), dict(vs=0), dict(k=A + 8), dict(v=A + 1), dict(b=0), dict(h=0),
             dict(t=0), dict(hd=96), dict(hd=256), dict(b=1 << 20, h=1 << 20, t=1 << 20)]


@pytest.mark.parametrize("bad", CACHE_BAD, ids=lambda s: ",".join(f"{k}={v}" for k, v in s.items()))
def test_bad_caches_are_refused(bad):
    c = cache(**bad)
    refused(binding.op_kv8_store, c, A, A, "bf16", 4)
    refused(binding.op_kv8_load, c, A, A, "bf16", 4)
    refused(binding.op_attention_kv8, A, c, A, 4, 1, ws_ptr=A, ws_bytes=1 << 30)


@pytest.mark.parametrize("fn", [binding.op_kv8_store, binding.op_kv8_load])
def test_cache_rows_refuse_bad_arguments(fn):
    c = cache()
    refused(fn, c, 0, A, "bf16", 4)
    refused(fn, c, A, 0, "bf16", 4)
    refused(fn, c, A, A, "bf16", 0)
    refused(fn, c, A + 8, A, "bf16", 4)
    refused(fn, c, A, A, "bf16", 4, starts_ptr=A + 1)
    refused(fn, c, A, A, "bf16", 4, counts_ptr=A + 2)
    refused(fn, c, A, A, "bf16", 4, k_row_stride=256, text="row stride")       # below H_kv * hd
    refused(fn, c, A, A, "bf16", 4, v_row_stride=516, text="row stride")       # not 16 bytes
    refused(fn, c, A, A, "f32", 4, k_row_stride=-512, text="row stride")
    refused(fn, cache(b=1 << 12, h=1 << 12), A, A, "bf16", 1 << 12, text="too many")


def test_attention_refuses_bad_arguments():
    c = cache()
    ok = dict(ws_ptr=A, ws_bytes=1 << 40)
    refused(binding.op_attention_kv8, 0, c, A, 8, 1, **ok)
    refused(binding.op_attention_kv8, A, c, 0, 8, 1, **ok)
    refused(binding.op_attention_kv8, A + 8, c, A, 8, 1, **ok)
    refused(binding.op_attention_kv8, A, c, A + 8, 8, 1, **ok)
    refused(binding.op_attention_kv8, A, c, A, 6, 1, **ok)          # H not a multiple of H_kv
    refused(binding.op_attention_kv8, A, c, A, 0, 1, **ok)
    refused(binding.op_attention_kv8, A, c, A, 8, 0, **ok)
    refused(binding.op_attention_kv8, A, c, A, 8, 1, limits_ptr=A + 2, **ok)
    for s in (0.0, -1.0, float("nan"), float("inf")):
        refused(binding.op_attention_kv8, A, c, A, 8, 1, scale=s, **ok)
    refused(binding.op_attention_kv8, A, c, A, 8, 1, q_row_stride=512, text="row stride", **ok)
    refused(binding.op_attention_kv8, A, c, A, 8, 1, out_row_stride=1028, text="row stride", **ok)
    for bad in [(0, 8, 4, 128, 1, 8), (1, 8, 3, 128, 1, 8), (1, 8, 4, 32, 1, 8), (1, 8, 4, 128, 0, 8),
                (1, 8, 4, 128, 1, 0)]:
        refused(binding.attention_kv8_workspace, *bad)
    assert binding.lib().dllm_op_attention_kv8_workspace(1, 8, 4, 128, 1, 8, None) == binding.EINVAL


def test_sizes_whose_tiles_leave_31_bits_are_refused():
    far = 2 ** 31 - 4095
    for T in (far, 2 ** 31 - 1):
        refused(binding.op_kv8_store, cache(b=1, h=1, t=T), A, A, "bf16", 1)
        refused(binding.op_attention_kv8, A, cache(b=1, h=1, t=T), A, 1, 1)
        refused(binding.attention_kv8_workspace, 1, 1, 1, 64, 1, T)
    assert binding.attention_kv8_workspace(1, 1, 1, 64, 1, far - 1) >= 0
    refused(binding.op_attention_kv8, A, cache(), A, 8, 1, scale=2e38)
    for M, N in ((far, 8), (8, far)):
        refused(binding.op_gemm8, A, A, A, A, A, "bf16", M, N, 16)


def test_product_refuses_bad_arguments():
    for args in [(0, "bf16", 4, 64, A, A), (A, "bf16", 0, 64, A, A), (A, "bf16", 4, 8, A, A), (A, "bf16", 4, 72, A, A),
                 (A, "bf16", 4, 64, 0, A), (A, "bf16", 4, 64, A, 0), (A, "bf16", 4, 64, A + 8, A),
                 (A + 1, "bf16", 4, 64, A, A), (A + 2, "f32", 4, 64, A, A)]:
        refused(binding.op_quantise8, *args)
    refused(binding.op_quantise8, A, "bf16", 4, 64, A, A, row_stride=32, text="row stride")
    ok = [A, A, A, A, A, "f32", 64, 4, 64]
    for i, v in [(0, 0), (1, 0), (2, 0), (3, 0), (4, 0), (0, A + 8), (2, A + 4), (4, A + 8), (5, "f16"), (6, 0),
                 (7, 0), (8, 0), (8, 40)]:
        a = list(ok)
        a[i] = v
        refused(binding.op_gemm8, *a)


def test_reference_encoding_is_the_nearest_code():
    """The tests' own encoder against a search over all codes."""
    rng = np.random.default_rng(0)
    finite = ref.CODE_VALUES[:0x7f]
    mids = (finite[1:] + finite[:-1]) / 2
    ys = np.concatenate([rng.uniform(0, 448, 300), 2.0 ** rng.uniform(-12, 8, 300), finite, mids])
    for y in ys:
        c = int(ref.encode(np.array([y]))[0])
        d = np.abs(finite - y)
        assert d[c] == d.min()
        if (d == d.min()).sum() == 2:
            assert c % 2 == 0                     # a tie goes to the even code
    assert ref.scale_byte(448.0) == 127 and ref.scale_byte(448.5) == 128 and ref.scale_byte(224.0) == 126
    assert ref.scale_byte(0.0) == 127 and ref.scale_byte(2.0 ** -140) == 0 and ref.scale_byte(np.inf) == 255


def test_struct_layouts_match_the_header():
    assert ctypes.sizeof(binding.Rope) == 64 and binding.Rope.theta.offset == 16
    assert ctypes.sizeof(binding.Kv8) == 48 and binding.Kv8.b.offset == 32
