"""Beam search for several prompts at once on a small ternary decoder over a paged cache: the prompts go through in ragged chunks,
each is forked into its beams, which share the prompt's pages, and every step chooses the next beams over beams and vocabulary,
lets the tables follow them, copies the shared pages that are about to be written and attends over all sequences in one call.

    python examples/beam_search.py [--beams W] [--tokens N] [--seed S]

The steps use the library's per-call entry points; the decoder's layers are those of tree_verify.py.
"""
import argparse
import os
import sys

import numpy as np
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

from examples.tree_verify import Decoder  # noqa: E402
from packed_weight_gemv_gb300 import nt  # noqa: E402

CHUNK = 48  # new tokens of a pass over prompts, and rows of a projection at a time (from 64 on it wants a workspace)


class PagedDecoder(Decoder):
    """The decoder with its caches taken as pools of pages, and the state of up to `most` sequences."""

    def __init__(self, most=32, page=16, n_pages=256, seed=0, **shape):
        super().__init__(rows=n_pages * page, seed=seed, **shape)
        self.page, self.n_pages, self.most = page, n_pages, most
        i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device=self.dev)  # noqa: E731
        self.width = n_pages  # of a sequence at most
        self.pages, self.length = i32(0, self.width), i32(0)
        self.refs = i32(n_pages)
        self.ws_paged = torch.zeros(nt.nt_paged_attention_workspace_size(max(most, CHUNK), most, self.Hq, self.Hkv, self.D),
                                    dtype=torch.uint8, device=self.dev)
        self.ws_logits = torch.zeros(nt.nt_int8_logits_workspace_size(self.V, self.d, most), dtype=torch.uint8, device=self.dev)
        self.ws_beam = torch.zeros(nt.nt_beam_select_workspace_size(self.V, most), dtype=torch.uint8, device=self.dev)
        self.ws_compact = torch.zeros(nt.nt_page_compact_workspace_size(n_pages), dtype=torch.uint8, device=self.dev)

    def ints(self, a):
        return torch.tensor(a, dtype=torch.int32, device=self.dev)

    def project(self, i, x):
        return torch.cat([super(PagedDecoder, self).project(i, part.contiguous()) for part in x.split(CHUNK)])

    def fork(self, parent):
        """Sequence i goes on as sequence parent[i] (-1: empty)."""
        if self.pages.shape[0] == 0:
            self.pages, self.length = (torch.zeros(1, *t.shape[1:], dtype=torch.int32, device=self.dev) for t in (self.pages, self.length))
        pages = torch.empty(parent.numel(), self.width, dtype=torch.int32, device=self.dev)
        length = torch.empty(parent.numel(), dtype=torch.int32, device=self.dev)
        nt.nt_page_fork(self.pages, self.length, parent, self.refs, self.page, pages, length)
        self.pages, self.length = pages, length

    def feed(self, tokens, counts):
        """counts[s] new tokens of each sequence; the logits of every sequence's last one [S, V]."""
        T, S, Hq, Hkv, D = tokens.numel(), len(counts), self.Hq, self.Hkv, self.D
        start = self.ints(np.concatenate(([0], np.cumsum(counts))))
        rows, pos = (torch.empty(T, dtype=torch.int32, device=self.dev) for _ in range(2))
        pairs = torch.empty(S, 2, dtype=torch.int32, device=self.dev)
        n_bad = self.ints([0])
        nt.nt_page_extend(self.pages, self.length, self.refs, start, self.page, rows, pos, pairs, n_bad=n_bad)
        nt.nt_page_copy(self.k_ptr, self.v_ptr, Hkv, D, self.rows, self.page, pairs)
        h = torch.empty(T, self.d, device=self.dev)
        nt.nt_embed_rows(self.table, self.table_s, self.V, self.d, tokens, T, h)
        h = h * 40.0  # the table's scales are those of an output projection
        for layer in range(self.L):
            i = 7 * layer
            x = self.norm(h)
            q, k, v = (self.project(i + j, x).view(T, -1, D) for j in range(3))
            nt.nt_qk_norm_rope_append(q, k, v, self.head_gain, self.head_gain, 1e-6, self.inv_freq, nt.NT_ROPE_HALF, 1.0, q, self.k[layer],
                                      self.v[layer], pos=pos, rows=rows)
            u = torch.empty_like(q)
            nt.nt_paged_attention(q, self.k[layer], self.v[layer], self.page, self.pages, start, self.length, u, self.ws_paged,
                                  max_new=max(counts))
            h = h + self.project(i + 3, u.view(T, Hq * D))
            x = self.norm(h)
            h = h + self.project(i + 6, torch.nn.functional.silu(self.project(i + 4, x)) * self.project(i + 5, x))
        if int(n_bad):
            raise RuntimeError("the pool has no page left")
        x = self.norm(h[start[1:].long() - 1].contiguous())  # (a sequence without new tokens repeats another's: its row is not used)
        codes, s_x = torch.empty(S, self.d, dtype=torch.int8, device=self.dev), torch.empty(S, device=self.dev)
        nt.nt_quantize_act(x, codes, s_x)
        logits, choice = torch.empty(S, self.V, device=self.dev), torch.empty(S, dtype=torch.int32, device=self.dev)
        nt.nt_int8_logits_argmax(self.table, self.table_s, self.V, self.d, codes, s_x, S, logits, choice, self.ws_logits)
        return logits

    def compact(self):
        """Pages in use to the front of the pool; their number."""
        pairs, used = torch.empty(self.n_pages // 2, 2, dtype=torch.int32, device=self.dev), self.ints([0])
        nt.nt_page_compact(self.refs, self.pages, self.length, self.page, pairs, used, self.ws_compact)
        nt.nt_page_copy(self.k_ptr, self.v_ptr, self.Hkv, self.D, self.rows, self.page, pairs)
        return int(used)

    def prompts(self, prompts):
        """Feeds the prompts in chunks of up to CHUNK tokens together; the logits behind each."""
        self.fork(self.ints([-1] * len(prompts)))
        logits = torch.empty(len(prompts), self.V, device=self.dev)
        done = [0] * len(prompts)
        while any(d < len(p) for d, p in zip(done, prompts)):
            room, counts = CHUNK, []
            for d, p in zip(done, prompts):
                counts.append(min(room, len(p) - d))
                room -= counts[-1]
            tokens = self.ints([t for d, p, n in zip(done, prompts, counts) for t in p[d:d + n]])
            out = self.feed(tokens, counts)
            for i, n in enumerate(counts):
                done[i] += n
                if n:
                    logits[i] = out[i]
        return logits


def search(model, prompts, beams, tokens, eos, alpha=0.6, compact_every=0):
    """The best continuation of every prompt as (tokens, score), its beams' in order."""
    if not all(prompts) or len(prompts) * beams > model.most:
        raise ValueError(f"prompts must have tokens, and prompts times beams be at most {model.most}")
    G, dev = len(prompts), model.dev
    model.refs.zero_()
    model.pages, model.length = model.pages[:0], model.length[:0]
    logits = model.prompts(prompts)
    # every prompt becomes its beams; all but the first of each have no score yet, so they are not chosen
    model.fork(model.ints([g for g in range(G) for _ in range(beams)]))
    logits = logits.repeat_interleave(beams, 0)
    scores = torch.full((G * beams,), -float("inf"), device=dev)
    scores[::beams] = 0.0
    done, lengths = (torch.zeros(G * beams, dtype=torch.int32, device=dev) for _ in range(2))
    parent, token = (torch.empty(G * beams, dtype=torch.int32, device=dev) for _ in range(2))
    lines = [[] for _ in range(G * beams)]
    for step in range(tokens):
        score, done_out = torch.empty_like(scores), torch.empty_like(done)
        nt.nt_beam_select(logits, scores, beams, parent, token, score, model.ws_beam, done=done, done_out=done_out, eos=eos, lengths=lengths,
                          alpha=alpha)
        up, new, was = parent.tolist(), token.tolist(), done.tolist()
        lines = [lines[p] + ([] if was[p] else [t]) if p >= 0 else [] for p, t in zip(up, new)]
        lengths = torch.where(parent >= 0, lengths[parent.clamp(min=0).long()] + 1 - done[parent.clamp(min=0).long()], 0).int()
        scores, done = score, done_out
        model.fork(parent)
        if compact_every and step % compact_every == compact_every - 1:
            model.compact()
        if step + 1 < tokens:
            logits = model.feed(token.clamp(min=0), [1] * (G * beams))
    return [[(lines[g * beams + b], float(scores[g * beams + b])) for b in range(beams)] for g in range(G)]


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--beams", type=int, default=4, help="1 to 64")
    ap.add_argument("--tokens", type=int, default=40)
    ap.add_argument("--seed", type=int, default=0)
    args = ap.parse_args(argv)
    page, sizes = 16, (70, 5, 33)
    # a pool that no search can exhaust: the prompts' pages, and per beam those of its own tokens with the two it shares in part
    n_pages = sum(n // page + 1 for n in sizes) + len(sizes) * args.beams * (args.tokens // page + 3)
    model = PagedDecoder(most=len(sizes) * args.beams, page=page, n_pages=max(64, n_pages), seed=args.seed)
    rs = np.random.RandomState(args.seed)
    prompts = [rs.randint(0, model.V, n).tolist() for n in sizes]
    for prompt, found in zip(prompts, search(model, prompts, args.beams, args.tokens, eos=model.V - 1)):
        line, score = found[0]
        print(f"prompt of {len(prompt)}: {len(line)} tokens, log probability {score:.3f}, begins {line[:6]}; the beams' {[round(s, 2) for _, s in found]}")
    print(f"{model.compact()} of {model.n_pages} pages in use")


if __name__ == "__main__":
    main()
