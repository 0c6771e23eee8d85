"""Refusals of the entry points of paged decoding: every check precedes any device call, so these run without a
GPU (the pointers are never dereferenced)."""
import os
import re
from pathlib import Path

import pytest

from cached_masked_decoding_gb300 import binding

A = 1 << 20     # a 16-byte aligned address that nothing reads
B = 2 << 20
CSRC = Path(__file__).resolve().parent.parent / "cached_masked_decoding_gb300" / "csrc"


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


def cache(k=A, v=A, table=A, b=2, h=4, hd=128, dtype="bf16", pages=64, ps=16, most=8):
    return binding.make_kv_paged(k, v, table, b, h, hd, dtype, pages, ps, most)


CACHE_BAD = [dict(k=0), dict(v=0), dict(table=0), dict(k=A + 8), dict(v=A + 2), dict(table=A + 2), dict(b=0), dict(h=0),
             dict(hd=96), dict(hd=256), dict(dtype="f32"), dict(pages=0), dict(ps=8), dict(ps=24), dict(ps=512),
             dict(ps=0), dict(most=0), dict(most=1 << 28), dict(pages=1 << 30)]


@pytest.mark.parametrize("bad", CACHE_BAD, ids=lambda s: ",".join(f"{k}={v}" for k, v in s.items()))
def test_bad_caches_are_refused_everywhere(bad):
    c = cache(**bad)
    refused(binding.op_attention_paged, A, c, A, 8, 1, ws_ptr=A, ws_bytes=1 << 40)
    refused(binding.op_qk_norm_rope_paged, c, A, A, A, B, 8, 1, "bf16")
    refused(binding.op_kv_paged_evict, c, cache(table=B), A, 4, A, A)
    refused(binding.op_kv_paged_evict, cache(table=B), c, A, 4, A, A)


def test_null_caches_are_refused():
    L = binding.lib()
    assert L.dllm_op_attention_paged(A, 0, None, None, 1.0, A, 0, 8, 1, None, 0, None, 0, None) == binding.EINVAL
    assert b"null" in L.dllm_last_error()
    assert L.dllm_op_kv_paged_evict(None, None, A, 0, None, 4, 0, 0, A, A, None, 0, None) == binding.EINVAL
    assert L.dllm_op_qk_norm_rope_paged(None, A, 0, A, 0, A, 0, A, 0, 8, 1, 1, None, None, None, None, None, 1e-6, None,
                                        None) == binding.EINVAL


def test_attention_paged_refuses_bad_arguments():
    op = binding.op_attention_paged
    big = dict(ws_ptr=A, ws_bytes=1 << 40)
    for q, out, H, R in [(0, A, 8, 1), (A, 0, 8, 1), (A + 8, A, 8, 1), (A, A + 4, 8, 1), (A, A, 0, 1), (A, A, 6, 1),
                         (A, A, 8, 0), (A, A, 8, -1)]:
        refused(op, q, cache(), out, H, R, **big)
    for s in (0.0, -1.0, float("nan"), float("inf"), 2.5e38):
        refused(op, A, cache(), A, 8, 1, scale=s, text="scale", **big)
    for rs in (1016, 1028, -1024, 1 << 41):
        refused(op, A, cache(), A, 8, 1, q_row_stride=rs, text="stride", **big)
        refused(op, A, cache(), A, 8, 1, out_row_stride=rs, text="stride", **big)
    refused(op, A, cache(), A, 8, 1, lens_ptr=A + 2, **big)
    refused(op, A, cache(), A, 8, 1, mass_ptr=A + 2, **big)
    refused(op, A, cache(), A, 8, 1, mass_ptr=A, mass_stride=-1, text="mass_stride", **big)
    refused(op, A, cache(b=1 << 10), A, 1 << 12, 1 << 10, text="too many rows", **big)
    for bad in [dict(b=0), dict(H=6), dict(hd=96), dict(R=0), dict(T=0)]:
        refused(binding.attention_paged_workspace, **{**dict(b=1, H=8, H_kv=4, hd=128, R=1, T=64), **bad})


HEADS_BAD = [dict(q=0), dict(k=0), dict(qo=0), dict(ko=0), dict(q=A + 8), dict(ko=B + 4), dict(rows=0), dict(H=0),
             dict(Hkv=0), dict(hd=0), dict(hd=72), dict(hd=272), dict(dtype="bf16", out="f32"),
             dict(dtype="bf16", out="f16"), dict(eps=float("nan")), dict(eps=float("inf")), dict(qw=A + 2),
             dict(eps=-1.0, qw=A), dict(eps=-1.0, kw=A), dict(pos=A + 1), dict(qs=8), dict(ks=8), dict(qs=1028),
             dict(qos=1 << 41), dict(kos=-512), dict(H=1 << 25), dict(rope=dict(rot_dim=24)), dict(rope=dict(rot_dim=192)),
             dict(rope=dict(rot_dim=64), pos=0), dict(rope=dict(rot_dim=64, theta=0.5)), dict(qo=A, qos=2048),
             dict(rows=0x7fffffff)]


@pytest.mark.parametrize("bad", HEADS_BAD, ids=lambda s: ",".join(f"{k}={v}" for k, v in s.items()))
def test_qk_norm_rope_refuses(bad):
    a = dict(q=A, k=A + (1 << 16), qo=B, ko=B + (1 << 16), pos=A, rows=4, H=8, Hkv=4, hd=128, dtype="bf16", out=None,
             qw=0, kw=0, eps=1e-6, rope=dict(rot_dim=64), qs=0, ks=0, qos=0, kos=0)
    a.update(bad)
    refused(binding.op_qk_norm_rope, a["q"], a["k"], a["qo"], a["ko"], a["pos"], a["rows"], a["H"], a["Hkv"], a["hd"],
            a["dtype"], out_dtype=a["out"], q_weight_ptr=a["qw"], k_weight_ptr=a["kw"], eps=a["eps"],
            rope=binding.make_rope(**a["rope"]), q_row_stride=a["qs"], k_row_stride=a["ks"], q_out_row_stride=a["qos"],
            k_out_row_stride=a["kos"])


def test_qk_norm_rope_paged_refuses():
    op = binding.op_qk_norm_rope_paged
    refused(op, cache(), A, A, 0, B, 8, 1, "bf16")                 # no values
    refused(op, cache(), A, A, A, B, 8, 0, "bf16", text="R=0")
    refused(op, cache(b=1 << 16), A, A, A, B, 8, 1 << 16, "bf16", text="R=")
    refused(op, cache(), A, A, A, B, 8, 1, "f16")                  # neither the cache's type nor float32
    refused(op, cache(), A, A, A, B, 8, 1, "bf16", starts_ptr=A + 2)
    refused(op, cache(), A, A, A, B, 8, 1, "bf16", counts_ptr=A + 1)
    refused(op, cache(), A, A, A, B, 8, 1, "bf16", v_row_stride=504, text="v row stride")
    refused(op, cache(), A, A, A, A, 8, 1, "f32", text="in place")


EVICT_BAD = [dict(mass=0), dict(kept=0), dict(lens_out=0), dict(keep=0), dict(keep=-1), dict(sinks=-1), dict(recent=-1),
             dict(sinks=3, recent=2), dict(keep=129), dict(mass=A + 2), dict(kept=A + 2), dict(lens=A + 1),
             dict(ms=-1), dict(mo=B, mos=3), dict(mo=A), dict(mo=B + 2), dict(lens=A), dict(sinks=0x7fffffff, recent=0x7fffffff)]


@pytest.mark.parametrize("bad", EVICT_BAD, ids=lambda s: ",".join(f"{k}={v}" for k, v in s.items()))
def test_evict_refuses(bad):
    a = dict(mass=A, keep=4, kept=A, lens_out=A, lens=0, sinks=1, recent=1, ms=0, mo=0, mos=0)
    a.update(bad)
    refused(binding.op_kv_paged_evict, cache(), cache(table=B), a["mass"], a["keep"], a["kept"], a["lens_out"],
            lens_ptr=a["lens"], sinks=a["sinks"], recent=a["recent"], mass_stride=a["ms"], mass_out_ptr=a["mo"],
            mass_out_stride=a["mos"])


@pytest.mark.parametrize("other", [dict(b=3), dict(h=2), dict(hd=64), dict(dtype="f16")])
def test_evict_refuses_caches_that_differ(other):
    refused(binding.op_kv_paged_evict, cache(), cache(**other), A, 4, A, A, text="differ")


LOGPROBS_BAD = [dict(x=0), dict(x=A + 1), dict(rows=0), dict(rows=0x7fffffff), dict(vocab=0), dict(top=-1), dict(top=65, ids=A, lp=A),
                dict(vocab=4, top=5, ids=A, lp=A), dict(t=0.0), dict(t=-1.0), dict(t=float("inf")), dict(t=2.5e38),
                dict(t=float("nan")), dict(targets=A, logp=0), dict(targets=0, logp=A), dict(top=2), dict(top=2, ids=A),
                dict(top=2, lp=A), dict(ids=A), dict(lp=A), dict(rs=99), dict(rs=-100), dict(rs=1 << 41),
                dict(targets=A + 2, logp=A), dict(entropy=A + 1)]


@pytest.mark.parametrize("bad", LOGPROBS_BAD, ids=lambda s: ",".join(f"{k}={v}" for k, v in s.items()))
def test_token_logprobs_refuses(bad):
    a = dict(x=A, rows=2, vocab=100, targets=0, logp=0, entropy=A, top=0, ids=0, lp=0, t=1.0, rs=0)
    a.update(bad)
    refused(binding.op_token_logprobs, a["x"], "bf16", a["rows"], a["vocab"], targets_ptr=a["targets"],
            logprobs_ptr=a["logp"], entropy_ptr=a["entropy"], top=a["top"], top_ids_ptr=a["ids"],
            top_logprobs_ptr=a["lp"], inv_temperature=a["t"], row_stride=a["rs"])


@pytest.mark.parametrize("path", [p for p in sorted(CSRC.iterdir()) if p.name.startswith(
    ("heads", "attn_paged", "evict", "logprobs", "kv_paged", "rope."))], ids=lambda p: p.name)
def test_loads_are_coherent(path):
    """These kernels are resident while the one before writes what they read."""
    code = re.sub(r"//[^\n]*|/\*.*?\*/", "", path.read_text(), flags=re.S)
    assert not re.search(r"__ldg|ld\.global(\.\w+)*\.nc|__restrict__", code)


def test_evict_refuses_its_own_pages():
    refused(binding.op_kv_paged_evict, cache(), cache(), A, 4, A, A, text="dst is src")
