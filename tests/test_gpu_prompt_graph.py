"""The prompt and attention calls in a CUDA graph, as a caller uses them whose host is slower than the kernels: prompt, single
token, tree, commit.  A replay gives the bits that the calls give, from the state that the replay before it left."""
import numpy as np
import pytest
import torch

from tests.test_gpu_prompt import N, P, _lib, f32, ints, params  # noqa: F401 (the fixture builds the library)

pytestmark = pytest.mark.gpu


def build(H, Hkv, D, lens, seed):
    """(what the calls change, the calls)"""
    import speculative_decoding_mamba2_gb300 as L
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    S, T, n, Hq, page, longest = len(lens), sum(lens), 9, 4 * Hkv, 32, 1500

    def rand(*shape):
        return torch.randn(shape, generator=gen, device="cuda").bfloat16()

    d = L.Dims(n_heads=H)
    prm, _ = params(rng, H, 1)
    cu, cd, most = ints(np.concatenate([[0], np.cumsum(lens)])), d.conv_dim, max(lens)
    par = np.stack([np.concatenate([[-1], rng.integers(0, np.arange(1, n))]) for _ in range(S)]).astype(np.int32)
    lay = torch.from_numpy(L.ssm_tree_layout_build(np.sort(par, 1))[0]).cuda()
    per = -(-(longest + 4 * n) // page)
    state = dict(ring=rand(S, 20, cd), head=ints([3] * S), h=f32(0.1 * rng.standard_normal((S, 1, H, P, N))),
                 kp=rand(S * per, Hkv, page, D), vp=rand(S * per, Hkv, page, D), len=ints(rng.integers(0, longest, S)))
    state["len"][0] = longest - 1
    state.update(post=rand(T, cd), y=rand(T, H * P), post1=rand(S, cd), y1=rand(S, H * P), o=rand(S * n, Hq * D))
    fixed = dict(x=rand(T, cd), dt=rand(T, H), x1=rand(S, cd), dt1=rand(S, H), q=rand(S * n, Hq * D), k=rand(S * n, Hkv * D),
                 v=rand(S * n, Hkv * D), table=ints(rng.permutation(S * per).reshape(S, per)), cu1=ints(range(S + 1)),
                 path=ints([[0, 1, 2]] * S), pl=ints([1 + s % 3 for s in range(S)]))
    wss = torch.empty(L.ssm_prompt_scan_workspace_size(d, S, T, most), dtype=torch.uint8, device="cuda")
    wsa = torch.empty(L.ssm_tree_attention_workspace_size(S, n, Hq, Hkv, D, longest + 4 * n), dtype=torch.uint8, device="cuda")
    keep = [cu, lay, wss, wsa, prm, fixed]

    def calls(s, f=fixed):
        L.ssm_prompt_conv(d, prm, 0, cu, most, f["x"], s["ring"], s["head"], s["post"])
        x, B, C = s["post"][:, :H * P], s["post"][:, H * P:H * P + N], s["post"][:, H * P + N:]
        L.ssm_prompt_scan(d, prm, 0, cu, most, x, B, C, f["dt"], s["h"], s["h"], s["y"], wss)
        L.ssm_prompt_conv(d, prm, 0, f["cu1"], 1, f["x1"], s["ring"], s["head"], s["post1"])
        x, B, C = s["post1"][:, :H * P], s["post1"][:, H * P:H * P + N], s["post1"][:, H * P + N:]
        L.ssm_scan_step(d, prm, 0, x, B, C, f["dt1"], s["h"], s["h"], s["y1"])
        for _ in range(2):  # back to back: the second is placed while the first ends
            L.ssm_tree_attention(S, n, Hq, Hkv, D, lay, f["q"], f["k"], f["v"], s["kp"], s["vp"], f["table"], s["len"],
                                 longest + 4 * n, D ** -0.5, s["o"], wsa)
        L.ssm_kv_commit(S, n, f["path"], f["pl"], f["k"][None], f["v"][None], s["kp"][None], s["vp"][None], f["table"], s["len"],
                        s["len"])
    return state, calls, keep


@pytest.mark.parametrize("H,Hkv,D,lens", [(24, 2, 128, [700, 33, 129]), (3, 1, 64, [40]), (4, 8, 64, [2000, 1])], ids=str)
def test_replays_equal_calls(H, Hkv, D, lens):
    state, calls, keep = build(H, Hkv, D, lens, 71)
    start = {k: v.clone() for k, v in state.items()}
    want = []
    for _ in range(3):
        calls(state)
        torch.cuda.synchronize()
        want.append({k: v.clone() for k, v in state.items()})
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls(state)
    for k, v in state.items():
        v.copy_(start[k])
    for w in want:
        graph.replay()
        torch.cuda.synchronize()
        for k, v in state.items():
            assert torch.equal(v, w[k]), k
    assert torch.isfinite(state["o"].float()).all() and torch.isfinite(state["y"].float()).all()
