"""What is measured of the prompt and attention operators, and their plain forms.

Five operators of a decoder that mixes Mamba2 blocks with attention blocks and decodes speculatively:

* ``conv``    ssm_prompt_conv: the causal width-4 conv + SiLU of ragged prompts, with the conv ring.
* ``scan``    ssm_prompt_scan: linear attention with a decay for each head over ragged prompts.
* ``step``    ssm_scan_step: the same for one token of each sequence.
* ``attend``  ssm_tree_attention: a draft tree's nodes over a paged cache and their ancestors.
* ``commit``  ssm_kv_commit: the accepted path's K and V rows into the paged cache, all layers.

``own = False`` computes them by elementary torch operations in 32 bits, rounded once at the end;
``own = True`` makes the calls a user makes.  Sizes: head_dim 64, d_state 128, conv width 4 (the
library's), head counts of the shapes the benchmark knows (24, 32, 80), generic lengths.
"""
import math

import numpy as np
import torch

own = False

P, N, W, R = 64, 128, 4, 20  # head_dim, d_state, conv width, rows of a conv ring


def listed():
    return [
        # the ends of three chunked prompts: nothing but latency
        dict(name="conv_tails", op="conv", H=24, S=3, T=11),
        # a batch of prompts of one layer at the 2.7B shape, ragged and odd
        dict(name="conv_prompts", op="conv", H=80, S=5, T=8209),
        # one short prompt of a small model, no state before it
        dict(name="scan_short", op="scan", H=24, G=1, S=1, T=37, fresh=True),
        # one long prompt of the 2.7B shape: few (sequence, head) pairs, a long axis
        dict(name="scan_one_long", op="scan", H=80, G=1, S=1, T=8191, fresh=True),
        # a batch of continued prompts at the 2.7B shape, ragged
        dict(name="scan_batch", op="scan", H=80, G=1, S=16, T=24571, fresh=False),
        # one token of one sequence of a small model: latency
        dict(name="step_one", op="step", H=24, G=1, S=1),
        # one token of a large decode batch, states at scattered slots
        dict(name="step_batch", op="step", H=80, G=1, S=128),
        # single-token decode of one sequence over a long cache: the cache split over the SMs
        dict(name="attend_token", op="attend", S=1, n=1, Hq=32, Hkv=8, D=128, len=16411, page=64),
        # a verify batch: 16-node trees, four query heads to a kv head, ragged caches
        dict(name="attend_trees", op="attend", S=8, n=16, Hq=32, Hkv=8, D=128, len=8117, page=64),
        # wide trees, eight query heads to a kv head, long caches
        dict(name="attend_wide", op="attend", S=4, n=40, Hq=32, Hkv=4, D=128, len=40009, page=128),
        # the accepted paths of one sequence, four attention layers
        dict(name="commit_one", op="commit", S=1, n=16, Hkv=8, D=128, L=4, len=1023, page=64),
        # ... and of a batch, eight layers
        dict(name="commit_batch", op="commit", S=32, n=40, Hkv=8, D=128, L=8, len=509, page=32),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["conv", "scan", "scan", "step", "attend", "attend", "commit"])
    H = rng.choice([24, 32, 80])
    if op == "conv":
        S = _log(rng, 1, 32)
        return dict(op=op, H=H, S=S, T=max(S, _log(rng, 4, 8000)))
    if op == "scan":
        S = _log(rng, 1, 24)
        return dict(op=op, H=H, G=rng.choice([1, 1, 2, 8]), S=S, T=max(S, _log(rng, 16, 24000)), fresh=rng.random() < 0.5)
    if op == "step":
        return dict(op=op, H=H, G=rng.choice([1, 1, 2, 8]), S=_log(rng, 1, 127))
    D = rng.choice([64, 128])
    page = rng.choice([16, 32, 64, 128])
    if op == "attend":
        Hkv = rng.choice([1, 2, 4, 8])
        S, n, g = _log(rng, 1, 32), _log(rng, 1, 64), rng.choice([1, 2, 4, 5, 8])
        flops, data = 4 * 40 * 32 * 40009 * 128, 600e6  # query rows x cache rows x D, and bytes, of the largest listed cases
        most = min(65536, flops / (S * n * g * Hkv * D), data / (4 * S * Hkv * D))
        return dict(op=op, S=S, n=n, Hq=g * Hkv, Hkv=Hkv, D=D, page=page, len=_log(rng, 1, max(2, most)))
    return dict(op=op, S=_log(rng, 1, 32), n=_log(rng, 1, 64), Hkv=rng.choice([1, 2, 4, 8]), D=D, L=rng.choice([1, 2, 4, 8]),
                len=_log(rng, 1, 900), page=page)


def work(c):
    if c["op"] == "conv":
        cd = c["H"] * P + 2 * N
        return dict(bytes=2 * c["T"] * cd * 2 + 20 * cd + 2 * 3 * 2 * c["S"] * cd, flops=12 * c["T"] * cd)
    if c["op"] in ("scan", "step"):
        T = c["T"] if c["op"] == "scan" else c["S"]
        h = 4 * c["S"] * c["H"] * P * N * (1 if c.get("fresh") else 2)
        return dict(bytes=T * (4 * c["H"] * P + 4 * c["G"] * N + 2 * c["H"]) + h, flops=4 * T * c["H"] * P * N)
    if c["op"] == "attend":
        rows = int(_lens(c).sum())
        q = 2 * 2 * c["S"] * c["n"] * c["Hq"] * c["D"]
        return dict(bytes=4 * c["Hkv"] * c["D"] * (rows + c["S"] * c["n"]) + q, flops=4 * c["n"] * c["Hq"] * c["D"] * rows)
    moved = int(_path_lens(c).sum())
    return dict(bytes=2 * 2 * 2 * c["L"] * moved * c["Hkv"] * c["D"] + 8 * c["S"] * (1 + c["n"]), flops=0)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _seq_lens(c):
    """Ragged lengths that add up to T, each at least one token: a fixed spread of 1 to 4."""
    S, T = c["S"], c["T"]
    w = np.array([1.0 + 3.0 * ((7 * s + 3) % 11) / 10.0 for s in range(S)])
    lens = 1 + np.floor((T - S) * w / w.sum()).astype(np.int64)
    lens[0] += T - lens.sum()
    return lens


def _lens(c):
    """Cache lengths: the first is the longest, the others between a quarter of it and all of it, and of eight
    sequences one is new (an empty cache)."""
    s = np.arange(c["S"])
    f = np.where(s == 0, 1.0, 0.25 + 0.75 * ((5 * s + 2) % 9) / 9.0)
    return np.where(s % 8 == 5, 0, np.ceil(f * c["len"])).astype(np.int64)


def _path_lens(c):
    return np.array([1 + (3 * s + 4) % min(c["n"], 6) for s in range(c["S"])], np.int64)


def _parents(rng, n):
    """A random breadth-first tree: up to three children a node, depth up to 6 where n allows it."""
    par, nxt, level = [-1], [0], [0]
    while len(par) < n:
        nxt = []
        for u in level:
            for _ in range(int(rng.integers(1, 4))):
                if len(par) < n:
                    par.append(u)
                    nxt.append(len(par) - 1)
        level = nxt
    return np.asarray(par, np.int32)


def _records(par):
    """The library's 8-word node records: parent, depth, first child, children, three conv taps, 0."""
    n = len(par)
    rec = np.zeros((n, 8), np.int32)
    depth = np.zeros(n, np.int64)
    for v in range(n):
        depth[v] = 0 if v == 0 else depth[par[v]] + 1
        kids = np.flatnonzero(par == v)
        u = v
        for k in range(3):
            u = par[u] if u >= 0 else u - 1
            rec[v, 4 + k] = u
        rec[v, :4] = par[v], depth[v], kids[0] if len(kids) else n, len(kids)
    return rec


def prepare(c, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    host = np.random.default_rng([int(seed), 17])

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    def uniform(lo, hi, *shape):
        return torch.rand(shape, generator=gen, device="cuda") * (hi - lo) + lo

    s = dict(case=dict(c), ws=None)
    S = c["S"]
    if c["op"] in ("conv", "scan", "step"):
        H = c["H"]
        cd = H * P + 2 * N
        u = torch.exp(uniform(math.log(1e-3), math.log(0.1), 1, H))
        s["params"] = dict(conv_w=uniform(-0.5, 0.5, 1, cd, W), conv_b=0.1 * normal(1, cd), dt_bias=torch.log(torch.expm1(u)),
                           A_log=torch.log(uniform(1.0, 16.0, 1, H)), D=1.0 + 0.1 * normal(1, H))
        lens = _seq_lens(c) if "T" in c else np.ones(S, np.int64)
        T = int(lens.sum())
        s["cu"] = torch.from_numpy(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)).cuda()
        s["max_len"] = int(lens.max())
        s["slots"] = torch.from_numpy(host.permutation(S).astype(np.int32)).cuda()
    if c["op"] == "conv":
        s["xBC"] = normal(T, cd).bfloat16()  # the input projection's rows
        s["ring"] = normal(S, R, cd).bfloat16()
        s["head"] = torch.from_numpy(host.integers(3, 5000, S).astype(np.int32)).cuda()
        s["out"] = torch.empty(T, cd, dtype=torch.bfloat16, device="cuda")
    elif c["op"] in ("scan", "step"):
        def act(*shape):  # what leaves the conv: SiLU of values of about unit size
            v = normal(*shape)
            return (v * torch.sigmoid(v)).bfloat16()
        row = act(T, H * P + 2 * c["G"] * N)  # one buffer of x | B | C rows, as the conv writes it
        s["x"], s["B"], s["C"] = row[:, :H * P], row[:, H * P:H * P + c["G"] * N], row[:, H * P + c["G"] * N:]
        s["dt"] = (0.5 * normal(T, H)).bfloat16()
        s["h"] = None if c.get("fresh") else 0.1 * normal(S, 1, H, P, N)
        s["h_out"] = torch.zeros(S, 1, H, P, N, device="cuda")
        s["y"] = torch.empty(T, H * P, dtype=torch.bfloat16, device="cuda")
    else:
        n, Hkv, D, page = c["n"], c["Hkv"], c["D"], c["page"]
        L = c.get("L", 1)
        lens = _lens(c)
        per = int(-(-(int(lens.max()) + n) // page))  # pages of the longest sequence and its tree
        pool = S * per + 3
        s["table"] = torch.from_numpy(host.permutation(pool)[:S * per].astype(np.int32).reshape(S, per)).cuda()
        s["len"] = torch.from_numpy(lens.astype(np.int32)).cuda()
        s["max_len"] = int(lens.max())
        s["k"] = normal(L, pool, Hkv, page, D).bfloat16()
        s["v"] = normal(L, pool, Hkv, page, D).bfloat16()
        s["kt"] = normal(L, S * n, Hkv * D).bfloat16()
        s["vt"] = normal(L, S * n, Hkv * D).bfloat16()
        if c["op"] == "attend":
            par = np.stack([_parents(host, n) for _ in range(S)])
            anc = np.zeros((S, n, n), bool)
            for v in range(n):
                anc[:, v] = anc[np.arange(S), np.maximum(par[:, v], 0)] & (v > 0)
                anc[:, v, v] = True
            s["layout"] = torch.from_numpy(np.stack([_records(p) for p in par])).cuda()
            s["anc"] = torch.from_numpy(anc).cuda()
            s["q"] = (1.5 * normal(S * n, c["Hq"] * D)).bfloat16()
            s["o"] = torch.empty(S * n, c["Hq"] * D, dtype=torch.bfloat16, device="cuda")
            s["scale"] = D ** -0.5
        else:
            pl = _path_lens(c)
            path = np.full((S, n), -1, np.int32)
            for i in range(S):
                path[i, :pl[i]] = np.concatenate([[0], 1 + np.sort(host.permutation(n - 1)[:pl[i] - 1])]) if n > 1 else 0
            s["path"] = torch.from_numpy(path).cuda()
            s["path_len"] = torch.from_numpy(pl.astype(np.int32)).cuda()
            s["len_out"] = torch.zeros(S, dtype=torch.int32, device="cuda")
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    c = s["case"]
    if own:
        return _OWN[c["op"]](s, c)
    return _PLAIN[c["op"]](s, c)


def _own_conv(s, c):
    from speculative_decoding_mamba2_gb300 import Dims, ssm_prompt_conv
    ssm_prompt_conv(Dims(n_heads=c["H"], ring_cap=R), s["params"], 0, s["cu"], s["max_len"], s["xBC"], s["ring"], s["head"],
                    s["out"], slots=s["slots"])
    return dict(out=s["out"], ring=_window(s), head=s["head"])


def _own_scan(s, c):
    from speculative_decoding_mamba2_gb300 import Dims, ssm_prompt_scan, ssm_prompt_scan_workspace_size
    d = Dims(n_heads=c["H"])
    if s["ws"] is None:
        s["ws"] = torch.empty(ssm_prompt_scan_workspace_size(d, c["S"], c["T"], s["max_len"], c["G"]), dtype=torch.uint8,
                              device="cuda")
    ssm_prompt_scan(d, s["params"], 0, s["cu"], s["max_len"], s["x"], s["B"], s["C"], s["dt"], s["h"], s["h_out"], s["y"],
                    s["ws"], slots=s["slots"])
    return dict(y=s["y"], h=s["h_out"])


def _own_step(s, c):
    from speculative_decoding_mamba2_gb300 import Dims, ssm_scan_step
    ssm_scan_step(Dims(n_heads=c["H"]), s["params"], 0, s["x"], s["B"], s["C"], s["dt"], s["h"], s["h_out"], s["y"],
                  slots=s["slots"])
    return dict(y=s["y"], h=s["h_out"])


def _own_attend(s, c):
    from speculative_decoding_mamba2_gb300 import ssm_tree_attention, ssm_tree_attention_workspace_size
    if s["ws"] is None:
        s["ws"] = torch.empty(ssm_tree_attention_workspace_size(c["S"], c["n"], c["Hq"], c["Hkv"], c["D"], s["max_len"]),
                              dtype=torch.uint8, device="cuda")
    ssm_tree_attention(c["S"], c["n"], c["Hq"], c["Hkv"], c["D"], s["layout"], s["q"], s["kt"][0], s["vt"][0], s["k"][0],
                       s["v"][0], s["table"], s["len"], s["max_len"], s["scale"], s["o"], s["ws"])
    return s["o"]


def _own_commit(s, c):
    from speculative_decoding_mamba2_gb300 import ssm_kv_commit
    ssm_kv_commit(c["S"], c["n"], s["path"], s["path_len"], s["kt"], s["vt"], s["k"], s["v"], s["table"], s["len"], s["len_out"])
    return dict(k=s["k"], v=s["v"], len=s["len_out"])


_OWN = dict(conv=_own_conv, scan=_own_scan, step=_own_step, attend=_own_attend, commit=_own_commit)


def _window(s):
    """The three rows before each ring's head: the rest of a ring is unspecified."""
    at = (s["head"][:, None].long() - torch.arange(3, 0, -1, device="cuda")) % R
    return s["ring"][torch.arange(at.shape[0], device="cuda")[:, None], at]


def _padded(s, c):
    """(index [S, max_len] of every sequence's tokens, which of them there are)."""
    first, most = s["cu"][:-1].long(), s["max_len"]
    t = torch.arange(most, device="cuda")
    there = t[None] < (s["cu"][1:].long() - first)[:, None]
    return torch.where(there, first[:, None] + t, 0), there


def _plain_conv(s, c):
    w, b = s["params"]["conv_w"][0], s["params"]["conv_b"][0]
    slot, first = s["slots"].long(), s["cu"][:-1].long()
    lens = s["cu"][1:].long() - first
    back = torch.arange(3, 0, -1, device="cuda")
    head = s["head"][slot].long()
    before = s["ring"][slot[:, None], (head[:, None] - back) % R]  # [S, 3, channels]
    T = s["xBC"].shape[0]
    of = torch.searchsorted(s["cu"][1:].long(), torch.arange(T, device="cuda"), right=True)  # a token's sequence
    at = torch.arange(T, device="cuda") - first[of]
    x = s["xBC"].float()
    acc = b + x * w[:, 3]
    acc = acc + sum(torch.where((at >= d)[:, None], torch.roll(x, d, 0), before[of, (3 + at - d).clamp(0, 2)].float()) * w[:, 3 - d]
                    for d in (1, 2, 3))
    s["out"].copy_(acc * torch.sigmoid(acc))
    # the three rows before the new head: of the old window and the tokens, the last three
    src = lens[:, None] - back
    rows = torch.where((src >= 0)[:, :, None], s["xBC"][(first[:, None] + src).clamp(min=0)],
                       before[torch.arange(len(slot), device="cuda")[:, None], (3 + src).clamp(0, 2)])
    s["ring"][slot[:, None], (head[:, None] + src) % R] = rows
    s["head"][slot] += lens.int()
    return dict(out=s["out"], ring=_window(s), head=s["head"])


def _plain_scan(s, c):
    """Chunks of 64 tokens side by side; the chunks' states through a triangular product of their decays."""
    H, G, S, Q = c["H"], c["G"], c["S"], 64
    at, there = _padded(s, c)
    pad = -at.shape[1] % Q
    at, there = torch.nn.functional.pad(at, (0, pad)), torch.nn.functional.pad(there, (0, pad))
    K = at.shape[1] // Q
    prm, slot = {k: v[0] for k, v in s["params"].items()}, s["slots"].long()
    x = s["x"][at].float().view(S, K, Q, H, P)
    B = s["B"][at].float().view(S, K, Q, G, N)
    C = s["C"][at].float().view(S, K, Q, G, N)
    v = s["dt"][at].float() + prm["dt_bias"]
    delta = torch.where(there[..., None], torch.log1p(torch.exp(-v.abs())) + v.clamp(min=0), 0.0).view(S, K, Q, H)
    cum = torch.cumsum(delta * -torch.exp(prm["A_log"]), 2)
    ut = torch.ones(Q, Q, dtype=torch.bool, device="cuda").tril()
    diff = (cum[:, :, :, None] - cum[:, :, None]).masked_fill_(~ut[:, :, None], -math.inf).exp_()  # [S, K, t, s, H]
    heads = torch.arange(H, device="cuda") // (H // G)
    dots = torch.einsum("skqgn,skrgn->skqrg", C, B)[..., heads]
    u = delta[..., None] * x
    y = torch.einsum("skqrh,skrhp->skqhp", dots.mul_(diff), u)
    del dots, diff
    last = cum[:, :, -1]
    part = torch.einsum("skqhp,skqhn->skhpn", torch.exp(last[:, :, None] - cum)[..., None] * u, B[:, :, :, heads])
    h0 = torch.zeros(S, H, P, N, device="cuda") if s["h"] is None else s["h"][slot, 0]
    tot = torch.nn.functional.pad(torch.cumsum(last, 1), (0, 0, 1, 0))  # decay up to the start of chunk k
    up = torch.ones(K + 1, K + 1, dtype=torch.bool, device="cuda").tril()
    hop = torch.exp((tot[:, :, None] - tot[:, None]).masked_fill_(~up[:, :, None], -math.inf))  # [S, K+1, K+1, H]
    states = torch.einsum("sjkh,skhpn->sjhpn", hop, torch.cat([h0[:, None], part], 1))
    y += torch.einsum("skqhn,skhpn->skqhp", C[:, :, :, heads], states[:, :-1]) * torch.exp(cum)[..., None]
    y += prm["D"][:, None] * x
    T = s["x"].shape[0]
    of = torch.searchsorted(s["cu"][1:].long(), torch.arange(T, device="cuda"), right=True)
    place = of * (K * Q) + torch.arange(T, device="cuda") - s["cu"][:-1].long()[of]
    s["y"].copy_(y.reshape(S * K * Q, H * P)[place])
    s["h_out"][slot, 0] = states[:, -1]
    return dict(y=s["y"], h=s["h_out"])


def _plain_step(s, c):
    H, G, S = c["H"], c["G"], c["S"]
    prm, slot = {k: v[0] for k, v in s["params"].items()}, s["slots"].long()
    v = s["dt"].float() + prm["dt_bias"]
    delta = torch.log1p(torch.exp(-v.abs())) + v.clamp(min=0)
    a = torch.exp(delta * -torch.exp(prm["A_log"]))
    x = s["x"].float().view(S, H, P)
    B = s["B"].float().view(S, G, 1, N).expand(S, G, H // G, N).reshape(S, H, N)
    C = s["C"].float().view(S, G, 1, N).expand(S, G, H // G, N).reshape(S, H, N)
    h = a[..., None, None] * s["h"][slot, 0] if s["h"] is not None else 0.0
    h = h + (delta[..., None] * x)[..., None] * B[:, :, None]
    s["y"].copy_(((h * C[:, :, None]).sum(-1) + prm["D"][:, None] * x).view(S, H * P))
    s["h_out"][slot, 0] = h
    return dict(y=s["y"], h=s["h_out"])


def _plain_attend(s, c):
    S, n, Hq, Hkv, D, page = (c[k] for k in ("S", "n", "Hq", "Hkv", "D", "page"))
    g, most = Hq // Hkv, s["max_len"]
    per = -(-most // page)

    def rows(pages, tree):  # [S, Hkv, most + n, D]: the cache's rows, then the tree's
        old = pages[0][s["table"][:, :per].long()].float()  # [S, per, Hkv, page, D]
        old = old.permute(0, 2, 1, 3, 4).reshape(S, Hkv, per * page, D)[:, :, :most]
        return torch.cat([old, tree[0].float().view(S, n, Hkv, D).transpose(1, 2)], 2)

    q = s["q"].float().view(S, n, Hkv, g, D).permute(0, 2, 1, 3, 4).reshape(S, Hkv, n * g, D)
    score = torch.matmul(q, rows(s["k"], s["kt"]).transpose(2, 3)).mul_(s["scale"])
    keep = torch.arange(most, device="cuda")[None] < s["len"][:, None]
    keep = torch.cat([keep[:, None].expand(S, n, most), s["anc"]], 2)  # [S, n, most + n]
    score = score.view(S, Hkv, n, g, most + n).masked_fill_(~keep[:, None, :, None], -math.inf)
    w = score.sub_(score.amax(-1, keepdim=True)).exp_()
    total = w.sum(-1, keepdim=True)
    o = torch.matmul(w.view(S, Hkv, n * g, most + n), rows(s["v"], s["vt"])).view(S, Hkv, n, g, D) / total
    s["o"].copy_(o.permute(0, 2, 1, 3, 4).reshape(S * n, Hq * D))
    return s["o"]


def _plain_commit(s, c):
    S, n, Hkv, D, L, page = (c[k] for k in ("S", "n", "Hkv", "D", "L", "page"))
    i = torch.arange(n, device="cuda")
    there = i[None] < s["path_len"][:, None]
    to = s["len"][:, None].long() + i
    pg, row = torch.gather(s["table"].long(), 1, to // page), to % page  # [S, n]
    src = torch.arange(S, device="cuda")[:, None] * n + torch.where(there, s["path"], 0).long()
    for pages, tree in ((s["k"], s["kt"]), (s["v"], s["vt"])):
        new = tree[:, src].view(L, S, n, Hkv, D)
        old = pages[:, pg, :, row]  # [S, n, L, Hkv, D]
        pages[:, pg, :, row] = torch.where(there[:, :, None, None, None], new.permute(1, 2, 0, 3, 4), old)
    s["len_out"].copy_(s["len"] + s["path_len"])
    return dict(k=s["k"], v=s["v"], len=s["len_out"])


_PLAIN = dict(conv=_plain_conv, scan=_plain_scan, step=_plain_step, attend=_plain_attend, commit=_plain_commit)


# ---------------------------------------------------------------------------
# 64 bits, from the definitions
# ---------------------------------------------------------------------------
def exact(c, seed):
    s = prepare(c, seed)
    return dict(conv=_exact_conv, scan=_exact_scan, step=_exact_scan, attend=_exact_attend, commit=_exact_commit)[c["op"]](s, c)


def _exact_conv(s, c):
    """Each sequence by itself: its window and its rows in one array, four shifted products."""
    w, b = s["params"]["conv_w"][0].double(), s["params"]["conv_b"][0].double()
    cu, out = s["cu"].tolist(), []
    ring, head = s["ring"].double().clone(), s["head"].clone()
    for i in range(c["S"]):
        k = int(s["slots"][i])
        f = int(head[k])
        win = torch.stack([ring[k, (f - j) % R] for j in (3, 2, 1)])
        rows = torch.cat([win, s["xBC"][cu[i]:cu[i + 1]].double()])
        m = cu[i + 1] - cu[i]
        z = b.repeat(m, 1)
        for j in range(W):
            z += rows[j:j + m] * w[:, j]
        out.append(z / (1.0 + torch.exp(-z)))
        for j in (3, 2, 1):
            ring[k, (f + m - j) % R] = rows[len(rows) - j]
        head[k] = f + m
    last = torch.stack([torch.stack([ring[k, (int(head[k]) - j) % R] for j in (3, 2, 1)]) for k in range(c["S"])])
    return dict(out=torch.cat(out), ring=last, head=head)


def _exact_scan(s, c):
    """The recurrence, token by token, all sequences that have such a token side by side."""
    H, G, S = c["H"], c["G"], c["S"]
    cu = s["cu"].tolist()
    lens = [cu[i + 1] - cu[i] for i in range(S)]
    order = sorted(range(S), key=lambda i: -lens[i])
    prm = {k: v[0].double() for k, v in s["params"].items()}
    slot = s["slots"].long()[order]
    h = torch.zeros(S, H, P, N, dtype=torch.float64, device="cuda") if s["h"] is None else s["h"][slot, 0].double()
    first = torch.tensor([cu[i] for i in order], device="cuda")
    y = torch.zeros(s["x"].shape[0], H * P, dtype=torch.float64, device="cuda")
    live = S
    for t in range(max(lens)):
        while lens[order[live - 1]] <= t:
            live -= 1
        at = first[:live] + t
        d = torch.nn.functional.softplus(s["dt"][at].double() + prm["dt_bias"], threshold=50.0)
        x = s["x"][at].double().view(live, H, P)
        B = s["B"][at].double().view(live, G, N).repeat_interleave(H // G, 1)
        C = s["C"][at].double().view(live, G, N).repeat_interleave(H // G, 1)
        hv = h[:live]
        hv.mul_(torch.exp(-d * torch.exp(prm["A_log"]))[..., None, None]).addcmul_((d[..., None] * x)[..., None], B[:, :, None])
        y[at] = (torch.matmul(hv, C[..., None])[..., 0] + prm["D"][:, None] * x).view(live, H * P)
    out = torch.zeros(S, 1, H, P, N, dtype=torch.float64, device="cuda")
    out[slot, 0] = h
    return dict(y=y, h=out)


def _exact_attend(s, c):
    """Each sequence and kv head by itself, over the rows it has."""
    n, Hq, Hkv, D, page = (c[k] for k in ("n", "Hq", "Hkv", "D", "page"))
    g, o = Hq // Hkv, torch.zeros(c["S"], n, Hq, D, dtype=torch.float64, device="cuda")
    for i, m in enumerate(s["len"].tolist()):
        for j in range(Hkv):
            at = torch.arange(m, device="cuda")
            pg = s["table"][i, at // page].long()
            K = torch.cat([s["k"][0, pg, j, at % page].double(), s["kt"][0].view(-1, n, Hkv, D)[i, :, j].double()])
            V = torch.cat([s["v"][0, pg, j, at % page].double(), s["vt"][0].view(-1, n, Hkv, D)[i, :, j].double()])
            q = s["q"].view(-1, n, Hq, D)[i, :, j * g:(j + 1) * g].double()
            z = torch.einsum("ngd,kd->ngk", q, K) * s["scale"]
            z[..., m:].masked_fill_(~s["anc"][i][:, None], -math.inf)
            o[i, :, j * g:(j + 1) * g] = torch.einsum("ngk,kd->ngd", torch.softmax(z, -1), V)
    return o.view(-1, Hq * D)


def _exact_commit(s, c):
    """Row by row."""
    n, page = c["n"], c["page"]
    k, v, lens, table = s["k"].double(), s["v"].double(), s["len"].tolist(), s["table"].tolist()
    path = s["path"].tolist()
    for i, m in enumerate(s["path_len"].tolist()):
        for j in range(m):
            at = lens[i] + j
            pg = table[i][at // page]
            for pages, tree in ((k, s["kt"]), (v, s["vt"])):
                pages[:, pg, :, at % page] = tree[:, i * n + path[i][j]].double().view(c["L"], c["Hkv"], c["D"])
        lens[i] += m
    return dict(k=k, v=v, len=torch.tensor(lens, dtype=torch.int32))
