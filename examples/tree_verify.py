"""Greedy decoding with drafted token trees on a small ternary decoder: every pass scores a tree of
drafted tokens, keeps the longest path that agrees with the model and moves its cache rows behind the
sequence's. The drafts are the continuations of earlier occurrences of the last token (no draft model).
The tokens are those of decoding one by one; the passes are fewer.

    python examples/tree_verify.py [--tokens N] [--seed S]

The layers use the library's per-call entry points: ternary projections, head norms with rotation and
cache append, tree attention, the int8 output projection, logit adjustments, acceptance and commit.
"""
import argparse
import os
import sys

import numpy as np
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

from packed_weight_gemv_gb300 import nt  # noqa: E402
from synth import workloads as wl  # noqa: E402

MAX_NODES = 16


class Decoder:
    """A few layers of random ternary projections with an int8 table for input and output."""

    def __init__(self, layers=3, d=512, Hq=8, Hkv=2, D=64, ffn=1024, V=2000, rows=1024, seed=0, dev="cuda"):
        self.L, self.d, self.Hq, self.Hkv, self.D, self.V, self.rows, self.dev = layers, d, Hq, Hkv, D, V, rows, dev
        shapes = {"q": (Hq * D, d), "k": (Hkv * D, d), "v": (Hkv * D, d), "o": (d, Hq * D), "gate": (ffn, d), "up": (ffn, d),
                  "down": (d, ffn)}
        self.w = []
        for p in wl.decoder_projections(layers, shapes, seed=seed, workload=9):
            plain = torch.from_numpy(p.w_plain.view(np.int32)).to(dev)
            w = torch.empty(nt.nt_repack_size(p.N, p.K), dtype=torch.uint8, device=dev)
            nt.nt_repack_ternary(plain, p.N, p.K, w)
            self.w.append((w, torch.from_numpy(p.s_w).to(dev), p.N, p.K))
        head = wl.head(V=V, K=d, seed=seed, workload=9)
        self.table, self.table_s = torch.from_numpy(head.T).to(dev), torch.from_numpy(head.s_T).to(dev)
        f32 = lambda *s: torch.empty(*s, dtype=torch.float32, device=dev)  # noqa: E731
        self.gain, self.head_gain = torch.ones(d, device=dev), torch.ones(D, device=dev)
        self.inv_freq = torch.empty(D // 2, dtype=torch.float64, device=dev)
        nt.nt_rope_frequencies(D, 1e4, self.inv_freq)
        caches = [torch.zeros(2, Hkv, rows, D, dtype=torch.bfloat16, device=dev) for _ in range(layers)]
        self.k, self.v = [c[0] for c in caches], [c[1] for c in caches]
        self.k_ptr, self.v_ptr = nt.pointer_array(self.k), nt.pointer_array(self.v)
        self.ws_attn = torch.zeros(max(nt.nt_tree_attention_workspace_size(b, Hq, Hkv, D, 0) for b in range(1, MAX_NODES + 1)),
                                   dtype=torch.uint8, device=dev)
        self.ws_head = torch.zeros(nt.nt_int8_logits_workspace_size(V, d, MAX_NODES), dtype=torch.uint8, device=dev)
        self.ws_adj = torch.zeros(nt.nt_logits_adjust_workspace_size(V, MAX_NODES), dtype=torch.uint8, device=dev)
        self.counts = torch.zeros(V, dtype=torch.int32, device=dev)
        self.logits = f32(MAX_NODES, V)

    def project(self, i, x):
        w, s, N, K = self.w[i]
        B = x.shape[0]
        q, s_x = torch.empty(B, K, dtype=torch.int8, device=self.dev), torch.empty(B, device=self.dev)
        y = torch.empty(B, N, device=self.dev)
        nt.nt_quantize_act(x, q, s_x)
        nt.nt_ternary_gemm(w, nt.NT_LAYOUT_TILED, s, N, K, q, s_x, B, y)
        return y

    def norm(self, x):
        y = torch.empty_like(x)
        nt.nt_rmsnorm(x, self.gain, x.shape[0], self.d, 1e-6, y)
        return y

    def score(self, tokens, pos, mask, prefix):
        """One pass over the nodes `tokens` (rows prefix .. of the caches): logits [B, V]."""
        B, Hq, Hkv, D = tokens.numel(), self.Hq, self.Hkv, self.D
        h = torch.empty(B, self.d, device=self.dev)
        nt.nt_embed_rows(self.table, self.table_s, self.V, self.d, tokens, B, h)
        h = h * 40.0  # the table's scales are those of an output projection
        for layer in range(self.L):
            i = 7 * layer
            x = self.norm(h)
            q, k, v = (self.project(i + j, x).view(B, -1, D) for j in range(3))
            nt.nt_qk_norm_rope_append(q, k, v, self.head_gain, self.head_gain, 1e-6, self.inv_freq, nt.NT_ROPE_HALF, 1.0, q,
                                      self.k[layer], self.v[layer], pos=pos, row0=prefix)
            u = torch.empty_like(q)
            nt.nt_tree_attention(q, self.k[layer], self.v[layer], prefix, prefix, mask, u, self.ws_attn)
            h = h + self.project(i + 3, u.view(B, Hq * D))
            x = self.norm(h)
            h = h + self.project(i + 6, torch.nn.functional.silu(self.project(i + 4, x)) * self.project(i + 5, x))
        x = self.norm(h)
        q, s_x = torch.empty(B, self.d, dtype=torch.int8, device=self.dev), torch.empty(B, device=self.dev)
        nt.nt_quantize_act(x, q, s_x)
        choice = torch.empty(B, dtype=torch.int32, device=self.dev)
        nt.nt_int8_logits_argmax(self.table, self.table_s, self.V, self.d, q, s_x, B, self.logits[:B], choice, self.ws_head)
        return self.logits[:B]

    def verify(self, parent, token, prefix, repetition):
        """Scores a tree, accepts its longest agreeing path and commits it; the emitted tokens (host)."""
        ints = lambda a: torch.tensor(a, dtype=torch.int32, device=self.dev)  # noqa: E731
        B = len(token)
        parent, token = ints(parent), ints(token)
        mask, pos = torch.empty(B, 1, dtype=torch.int32, device=self.dev), torch.empty(B, dtype=torch.int32, device=self.dev)
        nt.nt_tree_layout(parent, mask, pos, prefix)
        logits = self.score(token, pos, mask, prefix)
        choice, emit, path = (torch.empty(B, dtype=torch.int32, device=self.dev) for _ in range(3))
        n = torch.empty(1, dtype=torch.int32, device=self.dev)
        nt.nt_logits_adjust(logits, counts=self.counts, tree_mask=mask, tokens=token, repetition=repetition, argmax=choice,
                            ws=self.ws_adj)
        nt.nt_tree_accept(parent, token, choice, emit, path, n)
        nt.nt_tree_commit(self.k_ptr, self.v_ptr, self.Hkv, self.D, self.rows, path, n, prefix, prefix)
        nt.nt_token_counts(token, self.counts, index=path, n=n)
        assert nt.nt_workspace_status(self.ws_attn) == nt.NT_OK
        return emit[:int(n)].tolist()


def draft(history, width=3, depth=4):
    """A tree from what followed the last token before: (parents, tokens), node 0 the last token."""
    parent, token, child = [-1], [history[-1]], {}
    for at in [i for i in range(len(history) - 2, -1, -1) if history[i] == history[-1]][:width]:
        node = 0
        for t in history[at + 1:at + 1 + depth]:
            if (node, t) not in child and len(token) < MAX_NODES:
                child[node, t] = len(token)
                parent.append(node)
                token.append(t)
            node = child.get((node, t))
            if node is None:
                break
    return parent, token


def generate(model, prompt, n, tree, repetition=1.0):
    """n greedy tokens after the prompt, and the number of passes they took."""
    model.counts.zero_()
    history, prefix = list(prompt), 0
    while len(history) - prefix > 1:  # the prompt but its last token, as chains whose drafts are all kept
        part = history[prefix:len(history) - 1][:MAX_NODES]
        B = len(part)
        tokens = torch.tensor(part, dtype=torch.int32, device=model.dev)
        mask, pos = torch.empty(B, 1, dtype=torch.int32, device=model.dev), torch.empty(B, dtype=torch.int32, device=model.dev)
        nt.nt_tree_layout(torch.arange(-1, B - 1, dtype=torch.int32, device=model.dev), mask, pos, prefix)
        model.score(tokens, pos, mask, prefix)
        nt.nt_token_counts(tokens, model.counts)
        prefix += B
    out, passes = [], 0
    while len(out) < n:
        parent, token = draft(history) if tree else ([-1], [history[-1]])
        got = model.verify(parent, token, prefix, repetition)
        prefix += len(got)
        history += got
        out += got
        passes += 1
    return out[:n], passes


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--tokens", type=int, default=96)
    ap.add_argument("--seed", type=int, default=0)
    args = ap.parse_args()
    model = Decoder(seed=args.seed)
    prompt = np.random.RandomState(args.seed).randint(0, model.V, 40).tolist()
    one, n_one = generate(model, prompt, args.tokens, tree=False)
    many, n_many = generate(model, prompt, args.tokens, tree=True)
    same = next((i for i, (a, b) in enumerate(zip(one, many)) if a != b), len(one))
    print(f"{args.tokens} tokens: one by one {n_one} passes, with drafted trees {n_many} passes; the first {same} tokens agree")


if __name__ == "__main__":
    main()
