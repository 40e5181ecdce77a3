"""The calls of an 8-bit cache, rotary positions and token scores on the CPU: refusals (made before any CUDA call, so the pointers
here are never read), host functions, and what the binding checks."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

import oracle
from speculative_decoding_mamba2_gb300 import binding as B
from speculative_decoding_mamba2_gb300 import build as BLD

PTR, ODD = ctypes.c_void_p(4096), ctypes.c_void_p(4096 + 2)
INV, CAP, RANGE = B.SSM_ERR_INVALID_ARG, B.SSM_ERR_CAPACITY, B.SSM_ERR_RANGE


@pytest.fixture(scope="module")
def L():
    BLD.build()
    return B.lib()


ATTEND = dict(S=2, n=16, Hq=8, Hkv=2, D=128, layout=PTR, q=PTR, ldq=1024, k=PTR, ldk=256, v=PTR, ldv=256, kp=PTR, vp=PTR, ks=PTR,
              vs=PTR, n_pages=10, page=16, block=8, table=PTR, max_pages=5, len=PTR, max_len=80, scale=0.1, o=PTR, ldo=1024, ws=PTR,
              ws_bytes=1 << 30, status=None, stream=None)
COMMIT = dict(L=2, S=2, n=16, Hkv=2, D=128, max_path=16, path=PTR, path_len=PTR, k=PTR, v=PTR, kp=PTR, vp=PTR, ks=PTR, vs=PTR,
              n_pages=10, page=16, block=16, table=PTR, max_pages=5, len=PTR, len_out=PTR, status=None, stream=None)
ROPE = dict(T=9, Hq=8, Hkv=2, D=128, rot=64, inter=0, turns=PTR, amp=1.0, pos=PTR, q=PTR, ldq=1024, qo=PTR, ldqo=1024, k=PTR,
            ldk=256, ko=PTR, ldko=256, stream=None)
TREE_ROPE = dict(S=2, n=9, Hq=8, Hkv=2, D=128, rot=64, inter=1, turns=PTR, amp=1.0, layout=PTR, len=PTR, q=PTR, ldq=1024, qo=PTR,
                 ldqo=1024, k=PTR, ldk=256, ko=PTR, ldko=256, status=None, stream=None)
SCORES = dict(T=3, V=100, x=PTR, f32=1, ld=100, scale=1.0, m=2, tok=PTR, lp=PTR, h=PTR, k=4, top=PTR, tlp=PTR, status=None, stream=None)

BAD = [("ssm_tree_attention_fp8", ATTEND, kw, code) for kw, code in [
    (dict(S=-1), INV), (dict(S=65536), INV), (dict(n_pages=1 << 30), CAP), (dict(n=0), INV), (dict(n=65), CAP), (dict(Hkv=3), INV),
    (dict(Hq=66, ldq=1 << 14, ldo=1 << 14), CAP), (dict(D=96), INV), (dict(max_len=-1), INV), (dict(page=12), INV), (dict(block=4), INV),
    (dict(block=32), INV), (dict(block=12), INV), (dict(block=0), INV), (dict(ks=None), INV), (dict(vs=None), INV), (dict(ks=ODD), INV),
    (dict(n_pages=-1), INV), (dict(scale=0.0), RANGE), (dict(scale=float("nan")), RANGE), (dict(layout=None), INV), (dict(q=ODD), INV),
    (dict(k=None), INV), (dict(kp=None), INV), (dict(vp=ODD), INV), (dict(table=None), INV), (dict(len=None), INV), (dict(ldq=1016), INV),
    (dict(ldk=258), INV), (dict(ldo=1020), INV), (dict(o=None), INV), (dict(ws=None), INV), (dict(ws=ODD), INV), (dict(ws_bytes=0), CAP)]]
BAD += [("ssm_kv_commit_fp8", COMMIT, kw, code) for kw, code in [
    (dict(L=0), INV), (dict(S=-1), INV), (dict(S=65536), INV), (dict(n=0), INV), (dict(Hkv=0), INV), (dict(D=32), INV),
    (dict(max_path=0), INV), (dict(max_path=257), INV), (dict(page=24), INV), (dict(block=4), INV), (dict(block=32), INV),
    (dict(max_pages=-1), INV), (dict(path=None), INV), (dict(path_len=None), INV), (dict(k=ODD), INV), (dict(vp=None), INV),
    (dict(ks=None), INV), (dict(vs=ODD), INV), (dict(len_out=None), INV), (dict(L=1 << 24), CAP)]]
BAD += [(fn, base, kw, code) for fn, base in (("ssm_rope", ROPE), ("ssm_tree_rope", TREE_ROPE)) for kw, code in [
    (dict(Hq=-1), INV), (dict(Hkv=5000), INV), (dict(D=4), INV), (dict(D=100), INV), (dict(D=520), INV), (dict(rot=0), INV), (dict(rot=63), INV),
    (dict(rot=130), INV), (dict(turns=None), INV), (dict(turns=ODD), INV), (dict(amp=float("inf")), RANGE), (dict(amp=float("nan")), RANGE),
    (dict(q=None), INV), (dict(k=ODD), INV), (dict(qo=None), INV), (dict(ko=ODD), INV), (dict(ldq=1016), INV), (dict(ldko=258), INV),
    (dict(ldqo=1032), INV)]]
BAD += [("ssm_rope", ROPE, dict(T=-1), INV), ("ssm_rope", ROPE, dict(pos=None), INV), ("ssm_tree_rope", TREE_ROPE, dict(S=-1), INV),
        ("ssm_tree_rope", TREE_ROPE, dict(S=65536), INV), ("ssm_tree_rope", TREE_ROPE, dict(n=0), INV),
        ("ssm_tree_rope", TREE_ROPE, dict(S=60000, n=60000), CAP), ("ssm_tree_rope", TREE_ROPE, dict(layout=None), INV),
        ("ssm_tree_rope", TREE_ROPE, dict(len=None), INV)]
BAD += [("ssm_token_scores", SCORES, kw, code) for kw, code in [
    (dict(T=-1), INV), (dict(T=1 << 28), INV), (dict(V=0), INV), (dict(ld=99), INV), (dict(scale=0.0), RANGE), (dict(scale=-1.0), RANGE),
    (dict(scale=float("inf")), RANGE), (dict(scale=float("nan")), RANGE), (dict(m=-1), INV), (dict(k=-1), INV), (dict(k=33), CAP),
    (dict(V=3, k=4), INV), (dict(x=None), INV), (dict(x=ODD), INV), (dict(tok=None), INV), (dict(lp=None), INV), (dict(top=None), INV),
    (dict(f32=0, x=ctypes.c_void_p(4097)), INV)]]
BAD += [("ssm_tree_attention_fp8", ATTEND, dict(scale=v), RANGE) for v in (2.0 ** -41, 2.0 ** 41, float("inf"))]
BAD += [("ssm_token_scores", SCORES, kw, code) for kw, code in [
    (dict(scale=2.0 ** -101), RANGE), (dict(scale=2.0 ** 101), RANGE), (dict(tok=ODD), INV), (dict(lp=ODD), INV), (dict(h=ODD), INV),
    (dict(top=ODD), INV), (dict(tlp=ODD), INV)]]


@pytest.mark.parametrize("fn,base,kw,code", BAD, ids=lambda v: str(v)[:60] if not isinstance(v, dict) or len(v) < 3 else "")
def test_refusals(L, fn, base, kw, code):
    assert getattr(L, fn)(*dict(base, **kw).values()) == code
    assert B.ssm_last_error().startswith(fn + ":")


def test_calls_of_nothing_are_fine(L):
    """No rows: no launch, whatever the pointers are."""
    for fn, base, none in (("ssm_tree_attention_fp8", ATTEND, dict(S=0)), ("ssm_kv_commit_fp8", COMMIT, dict(S=0)), ("ssm_rope", ROPE, dict(T=0, pos=None)),
                           ("ssm_rope", ROPE, dict(Hq=0, Hkv=0, q=None)), ("ssm_tree_rope", TREE_ROPE, dict(S=0, turns=None)),
                           ("ssm_token_scores", SCORES, dict(T=0, x=None))):
        assert getattr(L, fn)(*dict(base, **none).values()) == B.SSM_OK and B.ssm_last_error() == ""


def test_every_declared_call_is_exported_and_bound(L):
    inc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
    for header in ("ssm_attention.h", "ssm_logits.h"):
        src = re.sub(r"/\*.*?\*/", "", open(os.path.join(inc, header)).read(), flags=re.S)
        for name in set(re.findall(r"\b(ssm_\w+)\s*\(", src)):
            assert hasattr(L, name) and hasattr(B, name), name


def test_workspace_sizes(L):
    assert B.ssm_tree_attention_fp8_workspace_size(2, 16, 8, 2, 128, 0) >= 256
    for bad in ((2, 0, 8, 2, 128, 9), (2, 65, 8, 2, 128, 9), (2, 4, 8, 3, 128, 9), (2, 4, 8, 2, 100, 9), (2, 4, 8, 2, 128, -1)):
        with pytest.raises(B.SSMError):
            B.ssm_tree_attention_fp8_workspace_size(*bad)


@pytest.mark.parametrize("kw", [dict(rot=64), dict(rot=2, base=500000.0), dict(rot=64, scaling="linear", factor=4.0),
                                dict(rot=128, scaling="base", factor=8.0), dict(rot=4, scaling="base", factor=3.0),
                                dict(rot=128, base=500000.0, scaling="by_parts", factor=8.0, original_len=8192, low=1.0, high=4.0)], ids=str)
def test_rope_frequencies(L, kw):
    """Equal to the definition but for the rounding of a power and two products in 64 bits."""
    np.testing.assert_allclose(B.ssm_rope_frequencies(**kw), oracle.rope_frequencies(**kw), rtol=1e-13)


def test_rope_frequencies_refusals(L):
    for kw in (dict(rot=3), dict(rot=0), dict(rot=8, base=0.0), dict(rot=8, base=float("inf")), dict(rot=8, scaling="linear", factor=0.0),
               dict(rot=2, scaling="base", factor=2.0), dict(rot=8, scaling="by_parts", factor=2.0),
               dict(rot=8, scaling="by_parts", factor=2.0, original_len=9.0, low=4.0, high=4.0)):
        with pytest.raises(B.SSMError):
            B.ssm_rope_frequencies(**kw)
    with pytest.raises(ValueError):
        B.ssm_rope_frequencies(8, scaling="other")


def test_rope_turns(L):
    """The fraction of a turn in 64 bits: exact for quarters, else off by half a step (2^-65) and the rounding of two operations in 64
    bits (2^-51 of a frequency), and modulo one turn."""
    two_pi = 6.283185307179586
    got = B.ssm_rope_turns([0.0, two_pi, two_pi / 4, -two_pi / 4, 5 * two_pi / 2]).numpy().view(np.uint64)
    assert got.tolist() == [0, 0, 1 << 62, 3 << 62, 1 << 63]
    f = oracle.rope_frequencies(128)
    got = B.ssm_rope_turns(f).numpy().view(np.uint64).astype(object) / 2 ** 64
    np.testing.assert_allclose(np.array(got, float), f / (2 * np.pi), rtol=2.0 ** -51, atol=2.0 ** -65)
    assert B.ssm_rope_turns([]).numel() == 0
    with pytest.raises(B.SSMError):
        B.ssm_rope_turns([1.0, float("nan")])


def test_binding_checks_tensors(L):
    """Wrong devices, types and shapes raise before the library is called."""
    bf, f8 = torch.bfloat16, torch.float8_e4m3fn
    x, p, s = torch.zeros(3, 64, dtype=bf), torch.zeros(2, 1, 16, 64, dtype=f8), torch.zeros(2, 1, 2)
    i = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError):
        B.ssm_tree_attention_fp8(3, 1, 1, 1, 64, i, x, x, x, p, p, s, s, i.view(3, 1), i, 0, 1.0, x, x)
    with pytest.raises(ValueError, match="k_scales"):
        B._pages_fp8(p, p, torch.zeros(2, 1, 3), s, 0, 1, 64)
    with pytest.raises(ValueError, match="k_pages"):
        B._pages_fp8(p[0], p, s, s, 0, 1, 64)
    with pytest.raises(ValueError):
        B.ssm_kv_commit_fp8(1, 1, i.view(3, 1), i, x, x, p, p, s, s, i.view(3, 1), i, i)
    with pytest.raises(ValueError):
        B.ssm_rope(64, i, torch.zeros(32, dtype=torch.int64), x, x)
    with pytest.raises(ValueError, match="both or neither"):
        B.ssm_rope(64, i, torch.zeros(32, dtype=torch.int64), x, None)
    with pytest.raises(ValueError, match="one of them"):
        B.ssm_rope(64, i, torch.zeros(32, dtype=torch.int64), None, None)
    with pytest.raises(ValueError):
        B.ssm_token_scores(torch.zeros(2, 9), None, None, None, None)


def test_token_scores_refuses_more_tokens_than_it_counts(L):
    """256 threads step over a row's tokens in an int32: the last step ends below 2^31 for up to 2^31 - 256 of them."""
    assert L.ssm_token_scores(*dict(SCORES, m=(1 << 31) - 255).values()) == CAP
    assert L.ssm_token_scores(*dict(SCORES, T=0, m=(1 << 31) - 256).values()) == B.SSM_OK
