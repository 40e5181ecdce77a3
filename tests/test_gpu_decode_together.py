"""An attention layer of a speculative decoder and the logits behind it, as its calls are used together: a prompt's chain, a draft
tree, a single token; each through rotary positions, the attention over the 8-bit cache, logits, scores, the accepted path and the
commit.  Every call's outputs are checked against the fp64 oracle on what the call before it left (tolerances: test_gpu_rope.py,
test_gpu_attention_fp8.py, test_gpu_scores.py); a CUDA graph of all of it gives the same bits."""
import numpy as np
import pytest
import torch

import oracle
from tests.test_gpu_attention import U, _lib, host, ints, tree  # noqa: F401 (the fixture builds the library)
from tests.test_gpu_rope import MORE

pytestmark = pytest.mark.gpu


class Layer:
    def __init__(self, S, Hq, Hkv, D, vocab, page, block, room, seed, inter):
        import speculative_decoding_mamba2_gb300 as L
        self.L, self.S, self.Hq, self.Hkv, self.D, self.vocab, self.page, self.block, self.room, self.inter = L, S, Hq, Hkv, D, vocab, page, block, room, inter
        self.gen = torch.Generator(device="cuda").manual_seed(seed)
        self.freq = L.ssm_rope_frequencies(D // 2, scaling="by_parts", factor=4.0, original_len=512)
        self.turns = L.ssm_rope_turns(self.freq).cuda()
        per = -(-room // page)
        self.table = torch.randperm(S * per, device="cuda", generator=self.gen).to(torch.int32).view(S, per)
        self.head = self.rand(vocab, Hq * D, by=(Hq * D) ** -0.5)
        self.state = dict(kp=torch.zeros(1, S * per, Hkv, page, D, device="cuda").to(torch.float8_e4m3fn),
                          vp=torch.zeros(1, S * per, Hkv, page, D, device="cuda").to(torch.float8_e4m3fn),
                          ks=torch.full((1, S * per, Hkv, page // block), 3.0, device="cuda"),
                          vs=torch.full((1, S * per, Hkv, page // block), 3.0, device="cuda"),
                          len=torch.zeros(S, dtype=torch.int32, device="cuda"))
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def rand(self, *shape, by=1.0):
        return (torch.randn(shape, device="cuda", generator=self.gen) * by).bfloat16()

    def stage(self, n, chain, accept, grow=1.0):
        """What a forward pass over n nodes a sequence has in hand: its projections, trees, drafted tokens, buffers."""
        L, S, T = self.L, self.S, self.S * n
        par = np.stack([np.arange(-1, n - 1, dtype=np.int32) if chain else tree(60 + s, n) for s in range(S)])
        lay, depth = L.ssm_tree_layout_build(par)
        e = lambda t, *shape: torch.empty(shape, dtype=t, device="cuda")  # noqa: E731
        bf, i32, f32 = torch.bfloat16, torch.int32, torch.float32
        x = dict(n=n, depth=depth, par=par, lay=torch.from_numpy(lay).cuda(), row=self.rand(T, (self.Hq + 2 * self.Hkv) * self.D, by=grow),
                 tok=torch.randint(0, 9, (S, n), device="cuda", generator=self.gen).to(i32), accept=accept,
                 q=e(bf, T, self.Hq * self.D), k=e(bf, T, self.Hkv * self.D), v=e(bf, T, self.Hkv * self.D), o=e(bf, T, self.Hq * self.D),
                 logits=e(f32, T, self.vocab + 5)[:, :self.vocab], lp=e(f32, T, 2), h=e(f32, T), top=e(i32, T, 3), tlp=e(f32, T, 3),
                 path=torch.full((S, n if accept == "all" else depth + 1), -1, dtype=i32, device="cuda"), pl=e(i32, S), bonus=e(i32, S))
        x["ws"] = e(torch.uint8, L.ssm_tree_attention_fp8_workspace_size(S, n, self.Hq, self.Hkv, self.D, self.room))
        x["given"] = torch.stack([x["tok"].view(-1), torch.full((T,), -1, dtype=i32, device="cuda")], 1).contiguous()
        if accept == "all":
            x["path"][:, :n] = torch.arange(n, device="cuda")
            x["pl"].fill_(n)
        return x

    def calls(self, x, look=None):
        L, S, n, s, st = self.L, self.S, x["n"], self.state, dict(status=self.status)
        look = look or (lambda what: None)
        wq, wk = self.Hq * self.D, self.Hkv * self.D
        L.ssm_tree_rope(S, n, self.D, x["lay"], s["len"], self.turns, x["row"][:, :wq], x["q"], x["row"][:, wq:wq + wk], x["k"],
                        interleaved=self.inter, amplitude=1.1, **st)
        x["v"].copy_(x["row"][:, wq + wk:])
        look("rope")
        L.ssm_tree_attention_fp8(S, n, self.Hq, self.Hkv, self.D, x["lay"], x["q"], x["k"], x["v"], s["kp"][0], s["vp"][0], s["ks"][0],
                                 s["vs"][0], self.table, s["len"], self.room, self.D ** -0.5, x["o"], x["ws"], **st)
        look("attend")
        L.ssm_linear(x["o"], self.head, [(0, x["logits"])], **st)
        L.ssm_token_scores(x["logits"], x["given"], x["lp"], x["h"], x["top"], x["tlp"], scale=1.25, **st)
        look("scores")
        if x["accept"] == "walk":  # a drafted token is the target's at half of the nodes
            self.walk(x)
        look("commit before")
        L.ssm_kv_commit_fp8(S, n, x["path"], x["pl"], x["k"][None], x["v"][None], s["kp"], s["vp"], s["ks"], s["vs"], self.table, s["len"],
                            s["len"], **st)
        look("commit")

    def walk(self, x):
        S, n = self.S, x["n"]
        target = x["top"][:, :1].contiguous()
        even = torch.arange(n, device="cuda") % 2 == 0
        up = x["lay"][:, :, 0].clamp(min=0).long()
        drafted = torch.where(even, torch.gather(target.view(S, n), 1, up), x["tok"])  # what follows the parent
        self.L.ssm_accept_path(S, n, x["path"].size(1), x["lay"], drafted, target, x["path"], x["pl"], x["bonus"], status=self.status)


def cached(ly, s, length):
    at = np.arange(length)
    pg, row = ly.table[s].cpu().numpy()[at // ly.page], at % ly.page
    return [host(ly.state[x + "p"][0].float())[pg, :, row] * host(ly.state[x + "s"][0])[pg, :, row // ly.block][..., None] for x in "kv"]


def checker(ly, x):
    S, n, Hq, Hkv, D = ly.S, x["n"], ly.Hq, ly.Hkv, ly.D
    keep = {}

    def look(what):
        torch.cuda.synchronize()
        lens = ly.state["len"].cpu().numpy()
        if what == "rope":
            pos = (lens[:, None] + x["lay"][:, :, 1].cpu().numpy()).reshape(-1).astype(float)
            for name, heads, at in (("q", Hq, 0), ("k", Hkv, Hq * D)):
                ref, mag = oracle.rope(host(x["row"][:, at:at + heads * D]).reshape(S * n, heads, D), pos, ly.freq, ly.inter, 1.1)
                assert (np.abs(host(x[name]).reshape(ref.shape) - ref) <= U * np.abs(ref) + MORE * mag).all()
        elif what == "attend":
            for s in range(S):
                part = slice(s * n, (s + 1) * n)
                ref, mag = oracle.tree_attention(host(x["q"][part]).reshape(n, Hq, D), host(x["k"][part]).reshape(n, Hkv, D),
                                                 host(x["v"][part]).reshape(n, Hkv, D), x["par"][s], *cached(ly, s, lens[s]), D ** -0.5)
                got = host(x["o"][part]).reshape(n, Hq, D)
                assert (np.abs(got - ref) <= U * np.abs(ref) + (U + 2.0 ** -11) * mag).all()
        elif what == "scores":
            want = oracle.token_scores(host(x["logits"]), x["given"].cpu().numpy(), 3, 1.25)
            V = ly.vocab
            e = (V / 512 + 64) * 2.0 ** -24 + (np.log(V) + 32) * 2.0 ** -22 + 2.0 ** -20
            np.testing.assert_array_equal(x["top"].cpu().numpy(), want[2])
            for got, ref, tol in ((x["lp"], want[0], e), (x["tlp"], want[3], e), (x["h"], want[1], e * (1 + np.log(V)))):
                np.testing.assert_allclose(host(got), ref, rtol=2.0 ** -22, atol=tol)
        elif what == "commit before":
            keep.update(len=lens, **{k: host(ly.state[k].float()) for k in ("kp", "vp", "ks", "vs")})
        else:
            path, pl = x["path"].cpu().numpy(), x["pl"].cpu().numpy()
            for s in range(S):
                for a, b, rows in (("kp", "ks", "k"), ("vp", "vs", "v")):
                    r = host(x[rows]).reshape(S, n, Hkv, D)[s]
                    assert oracle.kv_commit_fp8(keep[a][0], keep[b][0], r, path[s, :pl[s]], ly.table[s].cpu().numpy(), int(keep["len"][s])) == lens[s]
            for k in ("kp", "vp", "ks", "vs"):
                np.testing.assert_array_equal(host(ly.state[k].float()), keep[k])
    return look


@pytest.mark.parametrize("S,Hq,Hkv,D,page,block,inter", [(3, 4, 2, 64, 32, 16, False), (1, 8, 2, 128, 64, 64, True), (4, 3, 3, 128, 8, 8, False)], ids=str)
def test_a_layer_and_its_logits(S, Hq, Hkv, D, page, block, inter):
    ly = Layer(S, Hq, Hkv, D, 1003, page, block, 700, 7, inter)
    stages = [ly.stage(64, True, "all"), ly.stage(39, True, "all", grow=4.0)] + [ly.stage(16, False, "walk", grow=g) for g in (1.0, 8.0, 2.0)] + [ly.stage(1, True, "all")]
    start = {k: v.clone() for k, v in ly.state.items()}
    for x in stages:
        ly.calls(x, checker(ly, x))
    assert int(ly.status) == 0
    outs = [{k: v.clone() for k, v in x.items() if isinstance(v, torch.Tensor) and k != "ws"} for x in stages]
    end = {k: v.clone() for k, v in ly.state.items()}
    assert int(end["len"].min()) >= 64 + 39 + 3 + 1
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for x in stages:
            ly.calls(x)
    for _ in range(2):
        for k, v in ly.state.items():
            v.copy_(start[k])
        graph.replay()
        torch.cuda.synchronize()
        for x, want in zip(stages, outs):
            for k, v in want.items():
                assert torch.equal(x[k], v), k
        for k, v in end.items():
            assert torch.equal(ly.state[k].view(torch.uint8), v.view(torch.uint8)), k
