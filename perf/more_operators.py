"""What is measured of the operators of an attention layer with an 8-bit cache and of the logits behind it, and their plain forms.

Four operators beside the tree attention, the commit and the accepted path of a decoder that decodes speculatively:

* ``rope``    ssm_tree_rope, ssm_rope: rotary positions of a draft tree's nodes, and of rows with given positions.
* ``commit``  ssm_kv_commit_fp8: the accepted path's K and V rows into a paged cache of 8 bits, all layers.
* ``attend``  ssm_tree_attention_fp8: a draft tree's nodes over that cache and their ancestors.
* ``scores``  ssm_token_scores: log probabilities of given tokens, entropy and top alternatives of rows of logits.

The cache holds e4m3 values and, for each block of tokens of a head, a scale that is a power of two: the least one under
which the block's largest value is at most 448 (and at least 2^-100).  A block whose scale has to grow has its rows rounded again.

``own = False`` computes them by elementary torch operations in 32 bits (angles in 64), rounded once at the end;
``own = True`` makes the calls a user makes.  Head counts are those that the attention is measured with, other sizes generic.
"""
import math

import numpy as np
import torch

own = False

FP8 = torch.float8_e4m3fn


def listed():
    return [
        # the next token of one sequence in one layer: nothing but latency
        dict(name="rope_token", op="rope", S=1, n=1, Hq=32, Hkv=8, D=128, rot=128, inter=False, len=16411, scaled=False),
        # the nodes of a verify batch, half of each head, interleaved pairs
        dict(name="rope_trees", op="rope", S=16, n=40, Hq=32, Hkv=8, D=128, rot=64, inter=True, len=8117, scaled=False),
        # a batch of prompts far into a scaled context, pairs half a head apart
        dict(name="rope_prompts", op="rope", S=8191, n=0, Hq=32, Hkv=8, D=128, rot=128, inter=False, len=400009, scaled=True),
        # the accepted path of one sequence, four attention layers, a cache that ends inside a block
        dict(name="commit_one", op="commit", S=1, n=16, Hkv=8, D=128, L=4, len=1023, page=64, block=16),
        # ... and of a batch, eight layers, one scale for a page
        dict(name="commit_batch", op="commit", S=32, n=40, Hkv=8, D=128, L=8, len=509, page=32, block=32),
        # single-token decode of one sequence over a long cache: the cache split over the SMs
        dict(name="attend_token", op="attend", S=1, n=1, Hq=32, Hkv=8, D=128, len=16411, page=64, block=32),
        # a verify batch: 16-node trees, four query heads to a kv head, ragged caches
        dict(name="attend_trees", op="attend", S=8, n=16, Hq=32, Hkv=8, D=128, len=8117, page=64, block=16),
        # wide trees, eight query heads to a kv head, long caches, a scale for each half of a page
        dict(name="attend_wide", op="attend", S=4, n=40, Hq=32, Hkv=4, D=128, len=40009, page=128, block=64),
        # one row of logits of a small vocabulary: the target's next token and its runner-up
        dict(name="scores_token", op="scores", T=1, V=32003, f32=True, m=1, k=2, pad=0),
        # the nodes of a verify batch, logits in bf16: their children's tokens, eight alternatives
        dict(name="scores_trees", op="scores", T=256, V=128259, f32=False, m=3, k=8, pad=0),
        # a large batch of wide trees, logits in fp32 with a padded vocabulary
        dict(name="scores_wide", op="scores", T=640, V=151936, f32=True, m=1, k=16, pad=267),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "commit", "attend", "attend", "scores", "scores"])
    if op == "scores":
        V = _log(rng, 500, 200000)
        f32 = rng.random() < 0.5
        most = 640 * 151936 / V * (1 if f32 else 2)
        return dict(op=op, T=_log(rng, 1, min(4096, most)), V=V, f32=f32, m=rng.choice([0, 1, 1, 3, 8]), k=rng.choice([0, 1, 4, 8, 32]),
                    pad=rng.choice([0, 0, 1, 61]))
    D = rng.choice([64, 128])
    Hkv, g = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 5, 8])
    if op == "rope":
        rot = rng.choice([D, D, D // 2, D // 4, 2 * rng.randint(1, D // 2)])
        at = dict(op=op, Hq=Hkv * g, Hkv=Hkv, D=D, rot=rot, inter=rng.random() < 0.5, len=_log(rng, 1, 1 << 20), scaled=rng.random() < 0.5)
        if rng.random() < 0.5:
            return dict(at, S=_log(rng, 1, 32), n=_log(rng, 1, 64))
        return dict(at, S=_log(rng, 1, min(32768, 8000 * 40 * 128 / (Hkv * (g + 1) * D))), n=0)
    page = rng.choice([16, 32, 64, 128])
    block = rng.choice([b for b in (8, 16, 32, 64, 128) if b <= page])
    if op == "attend":
        S, n = _log(rng, 1, 32), _log(rng, 1, 64)
        flops, data = 4 * 40 * 32 * 40009 * 128, 300e6  # query rows x cache rows x D, and bytes, of the largest listed cases
        most = min(65536, flops / (S * n * g * Hkv * D), data / (2 * S * Hkv * D))
        return dict(op=op, S=S, n=n, Hq=g * Hkv, Hkv=Hkv, D=D, page=page, block=block, len=_log(rng, 1, max(2, most)))
    return dict(op=op, S=_log(rng, 1, 32), n=_log(rng, 1, 64), Hkv=Hkv, D=D, L=rng.choice([1, 2, 4, 8]), len=_log(rng, 1, 900),
                page=page, block=block)


def work(c):
    if c["op"] == "rope":
        T = c["S"] * max(1, c["n"])
        both = (c["Hq"] + c["Hkv"]) * T
        return dict(bytes=4 * both * c["D"] + 4 * T + 4 * c["rot"], flops=3 * both * c["rot"])
    if c["op"] == "scores":
        size = 4 if c["f32"] else 2
        return dict(bytes=c["T"] * (size * c["V"] + 8 * (c["m"] + c["k"]) + 4), flops=6 * c["T"] * c["V"])
    if c["op"] == "commit":
        moved, new = int(_path_lens(c).sum()), 2 * c["L"] * c["Hkv"]
        return dict(bytes=new * (3 * moved * c["D"] + 8 * c["S"]) + 4 * c["S"] * (3 + c["n"]), flops=2 * new * moved * c["D"])
    rows = int(_lens(c).sum())
    own_rows = 4 * c["Hkv"] * c["D"] * c["S"] * c["n"]
    q = 2 * 2 * c["S"] * c["n"] * c["Hq"] * c["D"]
    return dict(bytes=2 * c["Hkv"] * rows * (c["D"] + 4 / c["block"]) + own_rows + q, flops=4 * c["n"] * c["Hq"] * c["D"] * rows)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
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


def _frequencies(c):
    """Radians a position of each pair; scaled: a context stretched eight times, slow pairs by all of it, fast ones not at all,
    those between 1 and 32 turns over 8192 positions by a part of it (and the rotated values 1.2 times as large)."""
    half = c["rot"] // 2
    f = 10000.0 ** (-np.arange(half) / half)
    if not c["scaled"]:
        return f, 1.0
    turns = 8192 * f / (2 * math.pi)
    keep = np.clip((turns - 1.0) / 31.0, 0.0, 1.0)
    return f * (keep + (1.0 - keep) / 8.0), 0.1 * math.log(8.0) + 1.0


def _least_scale(most):
    """2^e, the least for which most (fp32, at least 0) is at most 448 * 2^e, and at least 2^-100."""
    bits = most.contiguous().view(torch.int32)
    e = (bits >> 23) - 127 - 8 + ((bits & 0x7FFFFF) > 0x600000).int()
    return _power(e.clamp(min=-100))


def _power(e):
    return ((e + 127) << 23).view(torch.float32)


def prepare(c, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    host = np.random.default_rng([int(seed), 19])

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    s = dict(case=dict(c), ws=None)
    if c["op"] == "scores":
        T, V = c["T"], c["V"]
        x = 2.0 * normal(T, V)
        sure = torch.rand(T, 1, generator=gen, device="cuda") * 14.0  # how much a row's first choices stand out
        some = torch.randint(0, V, (T, 4), generator=gen, device="cuda")
        x.scatter_(1, some, sure + normal(T, 4))
        if c["pad"]:
            x[:, V - c["pad"]:] = -math.inf
        s["logits"] = x if c["f32"] else x.bfloat16()
        tok = torch.randint(0, V - c["pad"], (T, c["m"]), generator=gen, device="cuda")
        tok[:, :2] = some[:, :min(2, c["m"])].clamp(max=V - c["pad"] - 1)  # drafted tokens: mostly likely ones
        s["tok"] = tok.int()
        new = lambda t, *shape: torch.empty(shape, dtype=t, device="cuda")  # noqa: E731
        s["logprob"], s["entropy"] = new(torch.float32, T, c["m"]), new(torch.float32, T)
        s["top"], s["top_logprob"] = new(torch.int32, T, c["k"]), new(torch.float32, T, c["k"])
        return s
    S, n, Hkv, D = c["S"], c["n"], c["Hkv"], c["D"]
    if c["op"] == "rope":
        T = S * max(1, n)
        row = normal(T, (c["Hq"] + 2 * Hkv) * D).bfloat16()  # one projection's output: q | k | v
        s["q"], s["k"] = row[:, :c["Hq"] * D], row[:, c["Hq"] * D:(c["Hq"] + Hkv) * D]
        s["freq"], s["amp"] = _frequencies(c)
        s["freq_dev"] = torch.from_numpy(s["freq"]).cuda()
        # a table of 2^64 parts of a turn, as ssm_rope_turns makes it
        s["turns"] = torch.from_numpy(np.array([int(round(f / (2 * math.pi) * 2.0 ** 64)) % 2 ** 64 for f in s["freq"]], np.uint64)
                                      .view(np.int64)).cuda()
        if n:
            lay = np.stack([_records(_parents(host, n)) for _ in range(S)])
            s["layout"] = torch.from_numpy(lay).cuda()
            s["len"] = torch.from_numpy(_lens(c).astype(np.int32)).cuda()
        else:
            s["pos"] = torch.from_numpy(np.sort(host.integers(0, c["len"], S)).astype(np.int32)).cuda()
        s["q_out"] = torch.empty(T, c["Hq"] * D, dtype=torch.bfloat16, device="cuda")
        s["k_out"] = torch.empty(T, Hkv * D, dtype=torch.bfloat16, device="cuda")
        return s
    page, block, L = c["page"], c["block"], c.get("L", 1)
    lens = _lens(c)
    per = int(-(-(int(lens.max()) + n) // page))  # pages of the longest sequence and its tree
    pool = S * per + 3
    s["table"] = torch.from_numpy(host.permutation(pool)[:S * per].astype(np.int32).reshape(S, per)).cuda()
    s["len"] = torch.from_numpy(lens.astype(np.int32)).cuda()
    s["max_len"] = int(lens.max())
    for name in ("k", "v"):
        x = normal(L, pool, Hkv, page // block, block * D)
        x *= torch.exp(0.5 * normal(L, pool, Hkv, page // block, 1))
        scale = _least_scale(x.abs().amax(-1))
        s[name] = (x / scale[..., None]).to(FP8).view(L, pool, Hkv, page, D)
        s[name + "_scale"] = scale
        s[name + "t"] = normal(L, S * n, Hkv * D).bfloat16()
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
        s["attn_scale"] = D ** -0.5
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


def _own_rope(s, c):
    from speculative_decoding_mamba2_gb300 import ssm_rope, ssm_tree_rope
    if c["n"]:
        ssm_tree_rope(c["S"], c["n"], c["D"], s["layout"], s["len"], s["turns"], s["q"], s["q_out"], s["k"], s["k_out"],
                      interleaved=c["inter"], amplitude=s["amp"])
    else:
        ssm_rope(c["D"], s["pos"], s["turns"], s["q"], s["q_out"], s["k"], s["k_out"], interleaved=c["inter"], amplitude=s["amp"])
    return dict(q=s["q_out"], k=s["k_out"])


def _own_commit(s, c):
    from speculative_decoding_mamba2_gb300 import ssm_kv_commit_fp8
    ssm_kv_commit_fp8(c["S"], c["n"], s["path"], s["path_len"], s["kt"], s["vt"], s["k"], s["v"], s["k_scale"], s["v_scale"],
                      s["table"], s["len"], s["len_out"])
    return dict(k=s["k"], v=s["v"], k_scale=s["k_scale"], v_scale=s["v_scale"], len=s["len_out"])


def _own_attend(s, c):
    from speculative_decoding_mamba2_gb300 import ssm_tree_attention_fp8, ssm_tree_attention_fp8_workspace_size
    if s["ws"] is None:
        s["ws"] = torch.empty(ssm_tree_attention_fp8_workspace_size(c["S"], c["n"], c["Hq"], c["Hkv"], c["D"], s["max_len"]),
                              dtype=torch.uint8, device="cuda")
    ssm_tree_attention_fp8(c["S"], c["n"], c["Hq"], c["Hkv"], c["D"], s["layout"], s["q"], s["kt"][0], s["vt"][0], s["k"][0],
                           s["v"][0], s["k_scale"][0], s["v_scale"][0], s["table"], s["len"], s["max_len"], s["attn_scale"],
                           s["o"], s["ws"])
    return s["o"]


def _own_scores(s, c):
    from speculative_decoding_mamba2_gb300 import ssm_token_scores
    ssm_token_scores(s["logits"], s["tok"], s["logprob"], s["entropy"], s["top"], s["top_logprob"])
    return dict(logprob=s["logprob"], entropy=s["entropy"], top=s["top"], top_logprob=s["top_logprob"])


_OWN = dict(rope=_own_rope, commit=_own_commit, attend=_own_attend, scores=_own_scores)


def _plain_rope(s, c):
    S, n, D, half = c["S"], c["n"], c["D"], c["rot"] // 2
    pos = (s["len"][:, None] + s["layout"][:, :, 1]).view(-1) if n else s["pos"]
    angle = pos.double()[:, None] * s["freq_dev"]
    cos, sin = (s["amp"] * torch.cos(angle)).float()[:, None], (s["amp"] * torch.sin(angle)).float()[:, None]
    for x, out in ((s["q"], s["q_out"]), (s["k"], s["k_out"])):
        T = x.shape[0]
        x, y = x.view(T, -1, D), out.view(T, -1, D)
        first, second = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if c["inter"] else (slice(0, half), slice(half, 2 * half))
        a, b = x[:, :, first].float(), x[:, :, second].float()
        y[:, :, first] = a * cos - b * sin
        y[:, :, second] = b * cos + a * sin
        y[:, :, 2 * half:] = x[:, :, 2 * half:]
    return dict(q=s["q_out"], k=s["k_out"])


def _plain_commit(s, c):
    """The rows from the start of the block that a cache ends in up to the end of the one that its path ends in, side by side."""
    S, n, Hkv, D, L, page, block = (c[k] for k in ("S", "n", "Hkv", "D", "L", "page", "block"))
    first = s["len"].long() // block * block
    wide = -(-(block - 1 + n) // block) * block
    at = first[:, None] + torch.arange(wide, device="cuda")  # [S, wide]: a row's place in its sequence
    i = at - s["len"].long()[:, None]
    is_new = (i >= 0) & (i < s["path_len"][:, None])
    is_old = i < 0
    used = (is_new | is_old).view(S, -1, block).any(-1) & is_new.view(S, -1, block).any(-1)  # blocks that get a row
    has_old = is_old.view(S, -1, block).any(-1)
    pg, row = torch.gather(s["table"].long(), 1, (at // page).clamp(max=s["table"].shape[1] - 1)), at % page
    node = torch.gather(s["path"].long(), 1, i.clamp(0, n - 1)).clamp(min=0)
    src = torch.arange(S, device="cuda")[:, None] * n + node
    bpg, bat = pg[:, ::block], row[:, ::block] // block  # [S, blocks]
    keep_row = (used[:, :, None] & (is_new | is_old).view(S, -1, block)).view(S, wide)
    rows, blocks = keep_row.nonzero(as_tuple=True), used.nonzero(as_tuple=True)
    for pages, scales, tree in ((s["k"], s["k_scale"], s["kt"]), (s["v"], s["v_scale"], s["vt"])):
        code = pages.view(torch.uint8)[:, pg, :, row]  # [S, wide, L, Hkv, D]
        old = scales[:, bpg, :, bat]  # [S, blocks, L, Hkv]
        new = tree[:, src].view(L, S, wide, Hkv, D).permute(1, 2, 0, 3, 4).float()
        most = torch.where(is_new[:, :, None, None], new.abs().amax(-1), 0.0).view(S, -1, block, L, Hkv).amax(2)
        scale = _least_scale(most)
        scale = torch.where(has_old[:, :, None, None], torch.maximum(old, scale), scale)
        of_row = lambda v: v.repeat_interleave(block, 1)[..., None]  # noqa: E731
        held = code.view(FP8).float() * of_row(torch.where(has_old[:, :, None, None], old / scale, 1.0))
        held = torch.where(is_new[:, :, None, None, None], new / of_row(scale), held).to(FP8).view(torch.uint8)
        pages.view(torch.uint8)[:, pg[rows], :, row[rows]] = held[rows]
        scales[:, bpg[blocks], :, bat[blocks]] = scale[blocks]
    s["len_out"].copy_(s["len"] + s["path_len"])
    return dict(k=s["k"], v=s["v"], k_scale=s["k_scale"], v_scale=s["v_scale"], len=s["len_out"])


def _plain_attend(s, c):
    S, n, Hq, Hkv, D, page, block = (c[k] for k in ("S", "n", "Hq", "Hkv", "D", "page", "block"))
    g, most = Hq // Hkv, s["max_len"]
    per = -(-most // page)

    def rows(pages, scales, tree):  # [S, Hkv, most + n, D]: the cache's rows, then the tree's
        at = s["table"][:, :per].long()
        old = pages[0].view(torch.uint8)[at].view(FP8).float().view(S, per, Hkv, page // block, block, D)
        old = (old * scales[0][at][..., None, None]).permute(0, 2, 1, 3, 4, 5).reshape(S, Hkv, per * page, D)[:, :, :most]
        return torch.cat([old, tree[0].float().view(S, n, Hkv, D).transpose(1, 2)], 2)

    q = s["q"].float().view(S, n, Hkv, g, D).permute(0, 2, 1, 3, 4).reshape(S, Hkv, n * g, D)
    score = torch.matmul(q, rows(s["k"], s["k_scale"], s["kt"]).transpose(2, 3)).mul_(s["attn_scale"])
    keep = torch.arange(most, device="cuda")[None] < s["len"][:, None]
    keep = torch.cat([keep[:, None].expand(S, n, most), s["anc"]], 2)  # [S, n, most + n]
    score = score.view(S, Hkv, n, g, most + n).masked_fill_(~keep[:, None, :, None], -math.inf)
    w = score.sub_(score.amax(-1, keepdim=True)).exp_()
    total = w.sum(-1, keepdim=True)
    o = torch.matmul(w.view(S, Hkv, n * g, most + n), rows(s["v"], s["v_scale"], s["vt"])).view(S, Hkv, n, g, D) / total
    s["o"].copy_(o.permute(0, 2, 1, 3, 4).reshape(S * n, Hq * D))
    return s["o"]


def _plain_scores(s, c):
    x = s["logits"].float() + 0.0  # (a zero's sign says nothing)
    top = x.amax(1, keepdim=True)
    e = torch.exp(x - top)
    total = e.sum(1, keepdim=True)
    log_total = torch.log(total)
    s["logprob"].copy_(torch.gather(x, 1, s["tok"].long()) - top - log_total)
    s["entropy"].copy_((log_total - torch.where(e > 0, e * (x - top), 0.0).sum(1, keepdim=True) / total)[:, 0])
    if c["k"]:
        bits = x.view(torch.int32)
        key = (bits ^ ((bits >> 31) & 0x7FFFFFFF)).long() << 32  # ordered as x is, then the lowest index first
        key |= (0x7FFFFFFF - torch.arange(c["V"], device="cuda"))[None]
        found = 0x7FFFFFFF - (torch.topk(key, c["k"], 1).values & 0xFFFFFFFF)
        s["top"].copy_(found)
        s["top_logprob"].copy_(torch.gather(x, 1, found) - top - log_total)
    return dict(logprob=s["logprob"], entropy=s["entropy"], top=s["top"], top_logprob=s["top_logprob"])


_PLAIN = dict(rope=_plain_rope, commit=_plain_commit, attend=_plain_attend, scores=_plain_scores)


# ---------------------------------------------------------------------------
# 64 bits, from the definitions
# ---------------------------------------------------------------------------
def exact(c, seed):
    s = prepare(c, seed)
    return dict(rope=_exact_rope, commit=_exact_commit, attend=_exact_attend, scores=_exact_scores)[c["op"]](s, c)


def _exact_rope(s, c):
    """Pairs as complex numbers, turned."""
    D, rot, out = c["D"], c["rot"], {}
    if c["n"]:
        pos = torch.cat([s["len"][i].long() + s["layout"][i, :, 1].long() for i in range(c["S"])])
    else:
        pos = s["pos"].long()
    turn = torch.polar(torch.full((1, 1), s["amp"], dtype=torch.float64, device="cuda"), pos.double()[:, None] * s["freq_dev"][None])
    for name in ("q", "k"):
        x = s[name].double().reshape(len(pos), -1, D)
        part = x[..., :rot].unflatten(-1, (-1, 2)) if c["inter"] else x[..., :rot].unflatten(-1, (2, -1)).transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(part.contiguous()) * turn[:, None])
        x[..., :rot] = (z if c["inter"] else z.transpose(-1, -2)).flatten(-2)
        out[name] = x.reshape(len(pos), -1)
    return out


def _exact_commit(s, c):
    """Row by row: a value in units of its block's scale, not rounded; old rows as the held values stand for."""
    n, page, block = c["n"], c["page"], c["block"]
    out = {}
    lens, table, path, pl = s["len"].tolist(), s["table"].tolist(), s["path"].tolist(), s["path_len"].tolist()
    for name, tree in (("k", "kt"), ("v", "vt")):
        p, sc = s[name].double(), s[name + "_scale"].double()
        for i in range(c["S"]):
            for b in range(lens[i] // block, (lens[i] + pl[i] - 1) // block + 1):
                lo, hi = max(b * block, lens[i]), min((b + 1) * block, lens[i] + pl[i])
                pg, at = table[i][b * block // page], b * block % page
                new = torch.stack([s[tree][:, i * n + path[i][r - lens[i]]].double().view(c["L"], c["Hkv"], c["D"]) for r in range(lo, hi)], 2)
                need = new.abs().amax((2, 3)).clamp(min=448 * 2.0 ** -100) / 448
                fit = torch.exp2(torch.ceil(torch.log2(need)))  # a power of two: 448 is 7/8 of one, so nothing comes near a whole log2
                k = lo - b * block
                if k:
                    was = sc[:, pg, :, at // block].clone()
                    fit = torch.maximum(fit, was)
                    p[:, pg, :, at:at + k] *= (was / fit)[..., None, None]
                p[:, pg, :, at + k:at + k + hi - lo] = new / fit[..., None, None]
                sc[:, pg, :, at // block] = fit
        out[name], out[name + "_scale"] = p, sc
    out["len"] = torch.tensor([a + b for a, b in zip(lens, pl)], dtype=torch.int32)
    return out


def _exact_attend(s, c):
    """Each sequence and kv head by itself, over the rows it has."""
    n, Hq, Hkv, D, page, block = (c[k] for k in ("n", "Hq", "Hkv", "D", "page", "block"))
    g, o = Hq // Hkv, torch.zeros(c["S"], n, Hq, D, dtype=torch.float64, device="cuda")
    codes = {name: s[name][0].double() for name in ("k", "v")}
    for i, m in enumerate(s["len"].tolist()):
        for j in range(Hkv):
            at = torch.arange(m, device="cuda")
            pg, row = s["table"][i, at // page].long(), at % page
            K, V = (torch.cat([codes[name][pg, j, row] * s[name + "_scale"][0].double()[pg, j, row // block, None],
                               s[name + "t"][0].view(-1, n, Hkv, D)[i, :, j].double()]) for name in ("k", "v"))
            q = s["q"].view(-1, n, Hq, D)[i, :, j * g:(j + 1) * g].double()
            z = torch.einsum("ngd,kd->ngk", q, K) * s["attn_scale"]
            z[..., m:].masked_fill_(~s["anc"][i][:, None], -math.inf)
            o[i, :, j * g:(j + 1) * g] = torch.einsum("ngk,kd->ngd", torch.softmax(z, -1), V)
    return o.view(-1, Hq * D)


def _exact_scores(s, c):
    """Eight rows at a time."""
    parts = []
    for x, tok in zip(s["logits"].split(8), s["tok"].split(8)):
        lp = torch.log_softmax(x.double(), 1)
        order = torch.sort(x.double(), dim=1, descending=True, stable=True).indices[:, :c["k"]]
        h = -torch.xlogy(torch.exp(lp), torch.exp(lp)).sum(1)
        parts.append((torch.gather(lp, 1, tok.long()), h, order.int(), torch.gather(lp, 1, order)))
    logprob, entropy, top, top_logprob = (torch.cat(p) for p in zip(*parts))
    return dict(logprob=logprob, entropy=entropy, top=top, top_logprob=top_logprob)
