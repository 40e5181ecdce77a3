"""A small decoder of Mamba2 and attention layers in turn, with random weights: prompts, single tokens and speculative rounds.

    python examples/hybrid_round.py

A prompt goes through the Mamba2 layers by ``ssm_prompt_conv`` and ``ssm_prompt_scan`` and through the attention layers as
chains of up to 64 nodes (``ssm_tree_attention``, ``ssm_kv_commit``).  A single token takes ``ssm_scan_step`` and a tree of
one node.  A speculative round drafts a tree, verifies it with ``ssm_tree_verify`` and ``ssm_tree_attention``, walks the
accepted path and commits it to the states (``ssm_commit``) and to the paged cache (``ssm_kv_commit``).
"""
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
from speculative_decoding_mamba2_gb300 import (Dims, ssm_accept_path, ssm_commit, ssm_gated_rmsnorm, ssm_kv_commit,  # noqa: E402
                                               ssm_linear, ssm_prompt_conv, ssm_prompt_scan, ssm_prompt_scan_workspace_size,
                                               ssm_rmsnorm, ssm_scan_step, ssm_tree_attention,
                                               ssm_tree_attention_workspace_size, ssm_tree_layout_build, ssm_tree_verify,
                                               ssm_tree_verify_workspace_size)

EPS, PIECE = 1e-5, 64


class Hybrid:
    """``pairs`` Mamba2 layers, each followed by an attention layer, for S sequences of up to ``room`` tokens."""

    def __init__(self, S=3, pairs=2, H=8, Hq=8, Hkv=2, D=64, vocab=512, room=1024, page=32, seed=0, dev="cuda"):
        self.S, self.L, self.H, self.Hq, self.Hkv, self.D, self.room, self.vocab = S, pairs, H, Hq, Hkv, D, room, vocab
        self.dims = Dims(n_heads=H, n_layers=1, ring_cap=20)  # a layer's state and ring are its own tensors
        self.d_inner, self.conv_dim, self.d_model = self.dims.d_inner, self.dims.conv_dim, Hq * D
        self.dev, gen = dev, torch.Generator(device=dev).manual_seed(seed)

        def w(n, k):
            return (torch.randn(n, k, device=dev, generator=gen) * k ** -0.5).bfloat16()

        def rand(*shape):
            return torch.randn(*shape, device=dev, generator=gen)

        d, m = self.d_inner, self.d_model
        self.embed, self.head, ones = rand(vocab, m), w(vocab, m), torch.ones
        self.W_in = [w(d + self.conv_dim + H, m) for _ in range(pairs)]
        self.W_out = [w(m, d) for _ in range(pairs)]
        self.W_qkv = [w((Hq + 2 * Hkv) * D, m) for _ in range(pairs)]
        self.W_o = [w(m, Hq * D) for _ in range(pairs)]
        self.norm, self.gnorm = ones(m, device=dev), ones(d, device=dev)
        self.prm = [dict(conv_w=rand(1, self.conv_dim, 4) * 0.4, conv_b=rand(1, self.conv_dim) * 0.1, D=ones(1, H, device=dev),
                         dt_bias=rand(1, H) - 2.0, A_log=rand(1, H) * 0.5) for _ in range(pairs)]
        # states, rings and pages
        self.h = [torch.zeros(S, 1, H, 64, 128, device=dev) for _ in range(pairs)]
        self.ring = [torch.zeros(S, 20, self.conv_dim, dtype=torch.bfloat16, device=dev) for _ in range(pairs)]
        self.ring_head = [torch.full((S,), 3, dtype=torch.int32, device=dev) for _ in range(pairs)]
        per = -(-room // page)
        self.kp, self.vp = (torch.zeros(pairs, S * per, Hkv, page, D, dtype=torch.bfloat16, device=dev) for _ in range(2))
        self.table = torch.randperm(S * per, device=dev, generator=gen).to(torch.int32).view(S, per)
        self.len = torch.zeros(S, dtype=torch.int32, device=dev)
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)

    def tree(self, parent):
        """Layout (on the GPU) and depth of S trees, parent: int32 [S, n]."""
        lay, depth = ssm_tree_layout_build(parent)
        return torch.from_numpy(lay).to(self.dev), depth

    def forward(self, tokens, layout, depth, mode):
        """Logits [S * n, vocab] of n tokens of each sequence.  mode "prompt" and "step": the next tokens, the Mamba2 states
        move on; "tree": a draft tree, nothing moves.  Keeps what a commit needs."""
        S, n, T = self.S, tokens.shape[1], tokens.numel()
        dev, d, cd, H, D = self.dev, self.d_inner, self.conv_dim, self.H, self.D

        def bf(*shape):
            return torch.empty(*shape, dtype=torch.bfloat16, device=dev)

        x = self.embed[tokens.reshape(-1).long()].contiguous()
        u, z, g, o = bf(T, self.d_model), bf(T, d), bf(T, d), bf(T, self.Hq * D)
        k, v = bf(self.L, T, self.Hkv * D), bf(self.L, T, self.Hkv * D)
        self.xBC, self.dt, self.k, self.v = [bf(T, cd) for _ in range(self.L)], [bf(T, H) for _ in range(self.L)], k, v
        cu = torch.arange(S + 1, dtype=torch.int32, device=dev) * n
        for i in range(self.L):
            ssm_rmsnorm(x, self.norm, EPS, u)
            ssm_linear(u, self.W_in[i], [(0, z), (d, self.xBC[i]), (d + cd, self.dt[i])], status=self.status)
            if mode == "tree":
                y = torch.empty(T, d, device=dev)
                ws = torch.empty(ssm_tree_verify_workspace_size(self.dims, S, n, depth), dtype=torch.uint8, device=dev)
                ssm_tree_verify(self.dims, self.prm[i], S, n, depth, layout, self.xBC[i], self.dt[i], self.h[i], self.ring[i],
                                self.ring_head[i], y, ws, status=self.status)
            else:
                post, yb = bf(T, cd), bf(T, d)
                ssm_prompt_conv(self.dims, self.prm[i], 0, cu, n, self.xBC[i], self.ring[i], self.ring_head[i], post,
                                status=self.status)
                xs, B, C = post[:, :d], post[:, d:d + 128], post[:, d + 128:]
                if mode == "step":
                    ssm_scan_step(self.dims, self.prm[i], 0, xs, B, C, self.dt[i], self.h[i], self.h[i], yb, status=self.status)
                else:
                    ws = torch.empty(ssm_prompt_scan_workspace_size(self.dims, S, T, n), dtype=torch.uint8, device=dev)
                    ssm_prompt_scan(self.dims, self.prm[i], 0, cu, n, xs, B, C, self.dt[i], self.h[i], self.h[i], yb, ws,
                                    status=self.status)
                y = yb.float()
            ssm_gated_rmsnorm(y, z, self.gnorm, EPS, g)
            ssm_linear(g, self.W_out[i], [(0, x)], residual=x, status=self.status)

            ssm_rmsnorm(x, self.norm, EPS, u)
            q = bf(T, self.Hq * D)
            ssm_linear(u, self.W_qkv[i], [(0, q), (self.Hq * D, k[i]), ((self.Hq + self.Hkv) * D, v[i])], status=self.status)
            ws = torch.empty(ssm_tree_attention_workspace_size(S, n, self.Hq, self.Hkv, D, self.room), dtype=torch.uint8, device=dev)
            ssm_tree_attention(S, n, self.Hq, self.Hkv, D, layout, q, k[i], v[i], self.kp[i], self.vp[i], self.table, self.len,
                               self.room, D ** -0.5, o, ws, status=self.status)
            ssm_linear(o, self.W_o[i], [(0, x)], residual=x, status=self.status)
        logits = torch.empty(T, self.vocab, device=dev)
        ssm_rmsnorm(x, self.norm, EPS, u)
        ssm_linear(u, self.head, [(0, logits)], status=self.status)
        return logits

    def keep(self, n, path, path_len):
        """The K and V rows of the accepted path into the pages, all layers."""
        ssm_kv_commit(self.S, n, path, path_len, self.k, self.v, self.kp, self.vp, self.table, self.len, self.len,
                      status=self.status)

    def chain(self, tokens, mode):
        """The next n <= 64 tokens of each sequence: logits [S, n, vocab]."""
        n = tokens.shape[1]
        layout, depth = self.tree(np.tile(np.arange(-1, n - 1, dtype=np.int32), (self.S, 1)))
        logits = self.forward(tokens, layout, depth, mode)
        path = torch.arange(n, dtype=torch.int32, device=self.dev).repeat(self.S, 1)
        self.keep(n, path, torch.full((self.S,), n, dtype=torch.int32, device=self.dev))
        return logits.view(self.S, n, self.vocab)

    def prompt(self, tokens):
        """Logits behind the last token of the prompts [S, T]."""
        for at in range(0, tokens.shape[1], PIECE):
            logits = self.chain(tokens[:, at:at + PIECE], "prompt")
        return logits[:, -1]

    def step(self, tokens):
        return self.chain(tokens.view(self.S, 1), "step")[:, 0]

    def round(self, tokens, parent):
        """Verify S draft trees (tokens, parent: [S, n]; node 0 is the last token known) and commit the accepted paths.
        Returns the paths, their lengths, the token after each and all nodes' logits."""
        S, n = tokens.shape
        layout, depth = self.tree(parent)
        logits = self.forward(tokens, layout, depth, "tree")
        path = torch.empty(S, depth + 1, dtype=torch.int32, device=self.dev)
        path_len, bonus = (torch.empty(S, dtype=torch.int32, device=self.dev) for _ in range(2))
        target = logits.argmax(-1).to(torch.int32)
        ssm_accept_path(S, n, depth + 1, layout, tokens, target, path, path_len, bonus, status=self.status)
        for i in range(self.L):
            ssm_commit(self.dims, self.prm[i], S, n, layout, depth + 1, path, path_len, self.xBC[i], self.dt[i], self.h[i],
                       self.ring[i], self.ring_head[i], status=self.status)
        self.keep(n, path, path_len)
        return path, path_len, bonus, logits.view(S, n, self.vocab)


def run(S=3, prompt_len=150, tokens=40, nodes=12, seed=0, **model):
    """Decode greedily token by token, then in speculative rounds whose drafts follow that decode four times out of five (a near
    tie of two logits may part the two); the rounds' logits are then compared with the same tokens' single steps.  Returns (tokens a round, largest difference of a logit in
    units of the logits' deviation)."""
    rng = np.random.default_rng(seed)
    new = lambda: Hybrid(S=S, seed=seed, **model)  # noqa: E731
    plain = new()
    prompt = torch.from_numpy(rng.integers(0, plain.vocab, (S, prompt_len)).astype(np.int32)).cuda()
    nxt = plain.prompt(prompt).argmax(-1).to(torch.int32)
    greedy = [nxt]
    for _ in range(tokens + nodes):
        nxt = plain.step(nxt).argmax(-1).to(torch.int32)
        greedy.append(nxt)
    greedy = torch.stack(greedy, 1).cpu().numpy()  # what the drafts are made from

    spec = new()
    root = spec.prompt(prompt).argmax(-1).to(torch.int32).cpu().numpy()
    out, seen, rounds = [[int(t)] for t in root], [[] for _ in range(S)], 0
    while min(len(o) for o in out) < tokens:
        parent, tok = np.full((S, nodes), -1, np.int32), rng.integers(0, spec.vocab, (S, nodes)).astype(np.int32)
        for s in range(S):  # two children a node, breadth-first, the first of them on the plain path's token, mostly
            tok[s, 0], depth = out[s][-1], [0] * nodes
            for v in range(1, nodes):
                parent[s, v] = (v - 1) // 2
                depth[v] = depth[parent[s, v]] + 1
                if v % 2 == 1 and rng.random() < 0.8:
                    tok[s, v] = greedy[s, min(len(out[s]) - 1 + depth[v], greedy.shape[1] - 1)]
        path, path_len, bonus, logits = spec.round(torch.from_numpy(tok).cuda(), parent)
        path, path_len, bonus = path.cpu().numpy(), path_len.cpu().numpy(), bonus.cpu().numpy()
        for s in range(S):
            nodes_s = path[s, :path_len[s]]
            out[s] += [int(tok[s, v]) for v in nodes_s[1:]] + [int(bonus[s])]
            seen[s] += [logits[s, int(v)] for v in nodes_s]
        rounds += 1
    assert int(plain.status) == 0 and int(spec.status) == 0

    check, worst = new(), 0.0
    check.prompt(prompt)
    for t in range(min(len(x) for x in seen)):
        step = check.step(torch.tensor([out[s][t] for s in range(S)], dtype=torch.int32, device="cuda"))
        both = torch.stack([seen[s][t] for s in range(S)])
        worst = max(worst, float((step - both).abs().max() / step.std()))
    return sum(len(o) - 1 for o in out) / (S * rounds), worst


if __name__ == "__main__":
    per_round, worst = run()
    print(f"{per_round:.2f} tokens a round; logits within {worst:.3f} standard deviations of single steps")
