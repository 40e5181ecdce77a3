"""Refusals of the prompt and attention calls (include/ssm_prompt.h, include/ssm_attention.h): every one is made on
the host, before any CUDA call, so the pointers here are never read."""
import ctypes

import pytest
import torch

from speculative_decoding_mamba2_gb300 import binding as B
from speculative_decoding_mamba2_gb300 import build as BLD

PTR, ODD = ctypes.c_void_p(4096), ctypes.c_void_p(4096 + 2)


@pytest.fixture(scope="module")
def L():
    BLD.build()
    return B.lib()


def dims(**kw):
    return ctypes.byref(B.ssm_dims(**{**dict(n_heads=4, head_dim=64, d_state=128, conv_width=4, n_layers=2, ring_cap=20), **kw}))


def prm(**kw):
    return ctypes.byref(B.ssm_params(**{**dict(conv_w=16, conv_b=16, dt_bias=16, A_log=16, D=16), **kw}))


CONV = dict(dims=None, prm=None, layer=0, n_seq=2, n_slots=2, n_tok=9, max_len=9, cu=PTR, slots=None, x=PTR, ldx=512, ring=PTR,
            head=PTR, out=ctypes.c_void_p(8192), ldo=512, status=None, stream=None)
SCAN = dict(dims=None, prm=None, layer=0, G=2, n_seq=2, n_slots=2, n_tok=9, max_len=9, cu=PTR, slots=None, x=PTR, ldx=256, B=PTR,
            ldb=256, C=PTR, ldc=256, dt=PTR, lddt=4, h_in=None, h_out=PTR, y=PTR, ldy=256, ws=PTR, ws_bytes=1 << 30, status=None,
            stream=None)
STEP = {k: v for k, v in SCAN.items() if k not in ("n_tok", "max_len", "cu", "ws", "ws_bytes")}
ATTEND = dict(S=2, n=16, Hq=8, Hkv=2, D=128, layout=PTR, q=PTR, ldq=1024, k=PTR, ldk=256, v=PTR, ldv=256, kp=PTR, vp=PTR,
              n_pages=10, page=16, table=PTR, max_pages=5, len=PTR, max_len=80, scale=0.1, o=PTR, ldo=1024, ws=PTR,
              ws_bytes=1 << 30, status=None, stream=None)
COMMIT = dict(L=2, S=2, n=16, Hkv=2, D=128, max_path=16, path=PTR, path_len=PTR, k=PTR, v=PTR, kp=PTR, vp=PTR, n_pages=10, page=16,
              table=PTR, max_pages=5, len=PTR, len_out=PTR, status=None, stream=None)
INV, CAP, RANGE = B.SSM_ERR_INVALID_ARG, B.SSM_ERR_CAPACITY, B.SSM_ERR_RANGE

BAD = [("ssm_prompt_conv", CONV, kw, code) for kw, code in [
    (dict(dims="null"), INV), (dict(prm="null"), INV), (dict(dims=dict(conv_width=3)), INV), (dict(dims=dict(ring_cap=2)), INV),
    (dict(dims=dict(head_dim=32)), INV), (dict(dims=dict(n_heads=0)), INV), (dict(prm=dict(conv_w=None)), INV),
    (dict(prm=dict(conv_w=20)), INV), (dict(layer=2), RANGE), (dict(layer=-1), RANGE), (dict(n_seq=-1), INV),
    (dict(n_seq=65536), INV), (dict(n_tok=-1), INV), (dict(max_len=-1), INV), (dict(cu=None), INV), (dict(x=None), INV),
    (dict(x=ODD), INV), (dict(ldx=511), INV), (dict(ldx=504), INV), (dict(ldo=516), INV), (dict(out=PTR), INV),
    (dict(ring=None), INV), (dict(head=None), INV)]]
BAD += [(f, base, kw, code) for f, base in (("ssm_prompt_scan", SCAN), ("ssm_scan_step", STEP)) for kw, code in [
    (dict(dims="null"), INV), (dict(prm="null"), INV), (dict(dims=dict(d_state=64)), INV), (dict(prm=dict(A_log=None)), INV),
    (dict(layer=2), RANGE), (dict(G=0), INV), (dict(G=3), INV), (dict(n_slots=-1), INV), (dict(x=None), INV), (dict(B=ODD), INV),
    (dict(C=None), INV), (dict(dt=None), INV), (dict(ldb=128), INV), (dict(ldc=260), INV), (dict(lddt=3), INV), (dict(h_out=None), INV),
    (dict(h_in=ODD), INV), (dict(y=ODD), INV), (dict(ldy=252), INV)]]
BAD += [("ssm_prompt_scan", SCAN, kw, code) for kw, code in [
    (dict(cu=None), INV), (dict(ws=None), INV), (dict(ws=ctypes.c_void_p(4096 + 16)), INV), (dict(ws_bytes=255), CAP),
    (dict(n_tok=100000, max_len=100000, ws_bytes=1 << 16), CAP)]]
BAD += [("ssm_tree_attention", ATTEND, kw, code) for kw, code in [
    (dict(S=-1), INV), (dict(S=65536), INV), (dict(n_pages=1 << 30), CAP), (dict(n=0), INV), (dict(n=65), CAP), (dict(Hkv=3), INV), (dict(Hkv=0), INV),
    (dict(Hq=66, ldq=1 << 14, ldo=1 << 14), CAP), (dict(D=96), INV), (dict(max_len=-1), INV), (dict(page=12), INV),
    (dict(page=4), INV), (dict(page=2048), INV), (dict(n_pages=-1), INV), (dict(scale=0.0), RANGE), (dict(scale=-1.0), RANGE),
    (dict(scale=float("nan")), RANGE), (dict(scale=float("inf")), RANGE), (dict(layout=None), INV), (dict(q=ODD), INV),
    (dict(k=None), INV), (dict(kp=None), INV), (dict(vp=ODD), INV), (dict(table=None), INV), (dict(len=None), INV), (dict(ldq=1016), INV),
    (dict(ldk=258), INV), (dict(ldv=128), INV), (dict(ldo=1020), INV), (dict(o=None), INV), (dict(ws=None), INV), (dict(ws_bytes=0), CAP)]]
BAD += [("ssm_kv_commit", COMMIT, kw, code) for kw, code in [
    (dict(L=0), INV), (dict(S=-1), INV), (dict(S=65536), INV), (dict(n=0), INV), (dict(Hkv=0), INV), (dict(D=32), INV),
    (dict(max_path=0), INV), (dict(max_path=257), INV), (dict(page=24), INV), (dict(max_pages=-1), INV), (dict(path=None), INV),
    (dict(path_len=None), INV), (dict(k=ODD), INV), (dict(vp=None), INV), (dict(len_out=None), INV), (dict(L=1 << 24), CAP)]]


@pytest.mark.parametrize("fn,base,kw,code", BAD, ids=lambda v: str(v)[:60] if not isinstance(v, dict) or len(v) < 3 else "")
def test_refusals(L, fn, base, kw, code):
    a = dict(base, **kw)
    for name, make in (("dims", dims), ("prm", prm)):
        if name in a:
            a[name] = None if a[name] == "null" else make(**(a[name] or {}))
    assert getattr(L, fn)(*a.values()) == code
    assert B.ssm_last_error().startswith(fn + ":")


def test_calls_of_nothing_are_fine(L):
    """No sequences: no launch, whatever the pointers are."""
    for fn, base, none in (("ssm_prompt_conv", CONV, dict(n_seq=0)), ("ssm_prompt_scan", SCAN, dict(n_seq=0)),
                           ("ssm_scan_step", STEP, dict(n_seq=0)), ("ssm_tree_attention", ATTEND, dict(S=0)),
                           ("ssm_kv_commit", COMMIT, dict(S=0))):
        a = dict(base, **none)
        a.update({k: f() for k, f in (("dims", dims), ("prm", prm)) if k in a})
        assert getattr(L, fn)(*a.values()) == B.SSM_OK and B.ssm_last_error() == ""


def test_workspace_sizes(L):
    d = B.Dims(n_heads=4)
    assert B.ssm_prompt_scan_workspace_size(d, 3, 100, 100) >= 256
    assert B.ssm_prompt_scan_workspace_size(d, 0, 0, 0) >= 256
    with pytest.raises(B.SSMError):
        B.ssm_prompt_scan_workspace_size(d, 3, 100, 100, 3)
    with pytest.raises(B.SSMError):
        B.ssm_prompt_scan_workspace_size(d, -1, 100, 100)
    # the bound on a sequence's length cannot pass the rows there are
    assert B.ssm_prompt_scan_workspace_size(d, 1, 100, 1 << 30) == B.ssm_prompt_scan_workspace_size(d, 1, 100, 100)
    assert B.ssm_tree_attention_workspace_size(2, 16, 8, 2, 128, 0) >= 256
    for bad in ((2, 0, 8, 2, 128, 9), (2, 65, 8, 2, 128, 9), (2, 4, 8, 3, 128, 9), (2, 4, 8, 2, 100, 9), (2, 4, 8, 2, 128, -1)):
        with pytest.raises(B.SSMError):
            B.ssm_tree_attention_workspace_size(*bad)


def test_binding_checks_tensors(L):
    """Wrong devices, types and shapes raise before the library is called."""
    d, bf = B.Dims(n_heads=1), torch.bfloat16
    t = dict(x=torch.zeros(3, 64, dtype=bf), B=torch.zeros(3, 128, dtype=bf), C=torch.zeros(3, 128, dtype=bf), dt=torch.zeros(3, 1, dtype=bf),
             h_in=None, h_out=torch.zeros(3, 1, 1, 64, 128), y=torch.zeros(3, 64, dtype=bf))
    with pytest.raises(ValueError):
        B.ssm_scan_step(d, {}, 0, *t.values())
    with pytest.raises(ValueError):
        B.ssm_kv_commit(1, 1, t["x"], t["x"], t["x"], t["x"], t["x"], t["x"], t["x"], t["x"], t["x"])
    with pytest.raises(ValueError):
        B.ssm_tree_attention(1, 1, 1, 1, 64, None, t["x"], t["x"], t["x"], t["x"], t["x"], t["x"], None, 0, 1.0, t["x"], None)
