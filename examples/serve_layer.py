"""One decoder layer served end to end: a paged key/value cache, its attention and the MoE block.

    python examples/serve_layer.py [--layer sliding|global] [--format bf16|e4m3] [--users N] [--steps N]
                                   [--draft NODES] [--beams N]

Several users' prompts are taken in chunks and then continued by single tokens, all of them in the same
batches, the way a serving loop does it: per step, the tokens are normed and projected, queries and keys turned by their
positions, the new tokens' keys and values are written into the cache (quantised for e4m3), the new queries attend to
it, and the residual with its norm and the block of this library follow. The projections are random and plain torch
products: the layer's shapes and its data flow are what is shown. The last tokens' outputs are compared with those of
whole prompts in one step.

With --draft, each user's next step is a tree of drafted tokens, of which the deepest path is kept; with --beams, each
prompt is continued by a beam search whose beams share the prompt's pages. Both are compared with the same tokens in a
whole step too.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
from mixture_experts_ffn_router_gb300 import binding as B  # noqa: E402
from mixture_experts_ffn_router_gb300 import synth  # noqa: E402

# (query heads, kv heads, head width, window) of the model's two kinds of layer.
LAYERS = {"sliding": (16, 8, 256, 1024), "global": (16, 2, 512, 0)}
PAGE = 64


class Layer:
    """Attention over a paged cache, then the MoE block, for batches of any sequences' new tokens."""

    def __init__(self, kind, fmt, max_tokens, seqs, max_len, seed=0):
        self.hq, self.hkv, self.d, self.window = LAYERS[kind]
        per_seq = -(-max_len // PAGE)
        self.kv = B.PagedKV(self.hq, self.hkv, self.d, PAGE, seqs * per_seq, fmt, max_tokens=max_tokens, max_seqs=seqs)
        self.cache = self.kv.new_cache()
        # Pages are dealt out in turn, so that a sequence's lie apart.
        self.table = torch.arange(seqs * per_seq, dtype=torch.int32, device="cuda").view(per_seq, seqs).T.contiguous()
        g = torch.Generator(device="cuda").manual_seed(seed)
        width = (self.hq + 2 * self.hkv) * self.d
        self.w_qkv = torch.randn(B.HIDDEN, width, generator=g, device="cuda", dtype=torch.bfloat16) * B.HIDDEN ** -0.5
        self.w_out = torch.randn(self.hq * self.d, B.HIDDEN, generator=g, device="cuda",
                                 dtype=torch.bfloat16) * (self.hq * self.d) ** -0.5
        self.before, self.after = (0.1 * torch.randn(B.HIDDEN, generator=g, device="cuda") for _ in range(2))
        self.rotary = B.Rotary([1e4 ** (-2 * i / self.d) for i in range(self.d // 2)])
        self.ffn = B.MoeFFN(B.MOE_FFN_FULL_LAYER, max_tokens)
        self.ffn_w = synth.make_weights(seed=seed, device="cuda")
        self.lengths = [0] * seqs

    def step(self, seqs, x, new, parents=None):
        """x: [sum(new), 2816] bf16, the new tokens of `seqs` one after the other; parents, int32 [sum(new)]: they are
        the nodes of trees. Returns the layer's output."""
        before = [self.lengths[u] for u in seqs]
        for u, n in zip(seqs, new):
            self.lengths[u] += n
        cu = torch.tensor([0] + list(new)).cumsum(0).to(torch.int32).cuda()
        lengths = torch.tensor([self.lengths[u] for u in seqs], dtype=torch.int32).cuda()
        self.batch = B.KVBatch(cu, lengths, self.table[list(seqs)], max_new=max(new))
        if parents is None:
            positions = torch.cat([torch.arange(b, b + n) for b, n in zip(before, new)]).to(torch.int32).cuda()
        else:
            tree = self.kv.tree(self.batch, parents)
            context = [b for b, n in zip(before, new) for _ in range(n)]
            positions = tree.depth + torch.tensor(context, dtype=torch.int32).cuda()
        _, normed = B.block_norm(x, pre=self.before)
        qkv = (normed @ self.w_qkv).view(-1, self.hq + 2 * self.hkv, self.d)
        q, k, v = qkv.split((self.hq, self.hkv, self.hkv), 1)
        self.rotary.apply(q, k, positions, inplace=True)
        self.kv.write(self.cache, self.batch, k, v)
        seen = dict(window=self.window, sinks=4 if self.window else 0)
        if parents is None:
            out, _ = self.kv.attention(self.cache, self.batch, q, **seen)
        else:
            out, _ = self.kv.tree_attention(self.cache, self.batch, tree, q, **seen)
        y, _ = B.block_norm(x, out.flatten(1) @ self.w_out, post=self.after)
        return self.ffn.forward(y, self.ffn_w)

    def status(self):
        return self.kv.status()[1] | self.ffn.status()[1]


def draft(layer, users, nodes, x):
    """A tree of `nodes` drafted tokens for each user in one step, of which the deepest path is kept. x: each user's
    nodes' inputs. Returns the path's nodes and their outputs, by user."""
    parents = [(i + 1) // 2 - 1 if i % 3 else i - 1 for i in range(nodes)]
    paths = []
    for i in range(nodes):
        paths.append((paths[parents[i]] if parents[i] >= 0 else []) + [i])
    path = max(paths, key=len)
    y = layer.step(range(users), torch.cat(x), [nodes] * users, torch.tensor(parents * users, dtype=torch.int32).cuda())
    kept = torch.tensor([path] * users, dtype=torch.int32).cuda()
    left = layer.kv.keep(layer.cache, layer.batch, kept, torch.full((users,), len(path), dtype=torch.int32).cuda())
    layer.lengths[:users] = left.tolist()
    return path, y.view(users, nodes, -1)[:, path]


def search(layer, users, beams, steps, prompts, vocabulary):
    """Continues each user's prompt, [n, 2816], by a beam search over a vocabulary of inputs, [V, 2816]. Sequence
    u * beams + k is beam k of user u. Returns the best beams' tokens, and their last outputs."""
    V = vocabulary.shape[0]
    first = [u * beams for u in range(users)]
    y = layer.step(first, torch.cat(prompts), [p.shape[0] for p in prompts])
    ends = torch.tensor([p.shape[0] for p in prompts]).cumsum(0) - 1
    y = y[ends.cuda()].repeat_interleave(beams, 0)
    for u in range(users):
        layer.lengths[u * beams:(u + 1) * beams] = [layer.lengths[u * beams]] * beams
    scores = torch.full((users, beams), -float("inf"), device="cuda")
    scores[:, 0] = 0.0  # at first there is one beam
    best = B.BeamSearch(users, beams, V, beams)
    taken = torch.empty(users, beams, 0, dtype=torch.int64, device="cuda")
    for _ in range(steps):
        logits = y @ vocabulary.T * B.HIDDEN ** -0.5
        scores, parents, tokens = best.select(logits, scores)
        lengths = torch.tensor(layer.lengths[::beams], dtype=torch.int32).cuda()
        layer.kv.reorder(layer.cache, layer.table, lengths, parents)
        taken = torch.cat((taken.gather(1, parents.long().unsqueeze(-1).expand(-1, -1, taken.shape[-1])),
                           tokens.long().unsqueeze(-1)), -1)
        y = layer.step(range(users * beams), vocabulary[tokens.long().view(-1)], [1] * (users * beams))
    return taken[:, 0], y.view(users, beams, -1)[:, 0]


def whole_step(kind, fmt, x):
    """The last outputs of sequences, [n, 2816] each, taken in one step."""
    n = [t.shape[0] for t in x]
    layer = Layer(kind, fmt, sum(n), len(n), max(n))
    y = layer.step(range(len(n)), torch.cat(x), n)
    return y, layer.status()


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--layer", choices=sorted(LAYERS), default="sliding")
    ap.add_argument("--format", choices=sorted(B.KV_FORMATS), default="bf16")
    ap.add_argument("--users", type=int, default=6)
    ap.add_argument("--steps", type=int, default=8, help="single tokens after the prompts")
    ap.add_argument("--draft", type=int, default=0, help="drafted tokens of each user after that, as a tree")
    ap.add_argument("--beams", type=int, default=0, help="beams of each user's prompt, searched for --steps tokens")
    a = ap.parse_args(argv)
    prompts = [150 + 211 * u % 1300 for u in range(a.users)]
    total = [p + a.steps for p in prompts]
    x = [synth.make_x(n, seed=10 + u, device="cuda") for u, n in enumerate(total)]

    def compared(what, got, want):
        # Of the tokens in the middle: one that is near a tie of the router may go to another expert.
        off = float(((got.float() - want.float()).norm(dim=-1) / want.float().norm(dim=-1)).median())
        print("%s: %.2e off" % (what, off))
        return off

    room = a.users * max(512, a.draft)
    layer = Layer(a.layer, a.format, max(room, sum(total)), a.users, max(total) + a.draft)
    done, last = [0] * a.users, [None] * a.users
    while min(d - t for d, t in zip(done, total)) < 0:
        # Prompts go in chunks of 512; a user whose prompt is in goes on by single tokens beside them.
        users = [u for u in range(a.users) if done[u] < total[u]]
        new = [min(512, prompts[u] - done[u]) if done[u] < prompts[u] else 1 for u in users]
        y = layer.step(users, torch.cat([x[u][done[u]:done[u] + n] for u, n in zip(users, new)]), new)
        at = 0
        for u, n in zip(users, new):
            at += n
            done[u] += n
            last[u] = y[at - 1]
    y, status = whole_step(a.layer, a.format, x)
    ends = ends_of(total)
    print("%s layer, %s cache: %d users, %d tokens, against whole steps" % (a.layer, a.format, a.users, sum(total)))
    off = compared("last tokens step by step", torch.stack(last), y[ends])
    if a.draft:
        nodes = [synth.make_x(a.draft, seed=50 + u, device="cuda") for u in range(a.users)]
        path, got = draft(layer, a.users, a.draft, nodes)
        longer = [torch.cat((x[u], nodes[u][path])) for u in range(a.users)]
        y, more = whole_step(a.layer, a.format, longer)
        ends = ends_of([t.shape[0] for t in longer]).view(-1, 1)
        rows = (ends - torch.arange(len(path) - 1, -1, -1, device="cuda")).view(-1)
        off = max(off, compared("kept paths of %d of %d nodes" % (len(path), a.draft), got.flatten(0, 1), y[rows]))
        # One token more, after the kept path.
        token = [synth.make_x(1, seed=90 + u, device="cuda") for u in range(a.users)]
        got = layer.step(range(a.users), torch.cat(token), [1] * a.users)
        y, again = whole_step(a.layer, a.format, [torch.cat(p) for p in zip(longer, token)])
        ends = ends_of([t.shape[0] + 1 for t in longer])
        off = max(off, compared("a token after it", got, y[ends]))
        status |= more | again
    status |= layer.status()
    if a.beams:
        beamed = Layer(a.layer, a.format, max(sum(prompts), a.users * a.beams), a.users * a.beams, max(total))
        words = synth.make_x(1000, seed=70, device="cuda")
        heads = [x[u][:n] for u, n in enumerate(prompts)]
        taken, got = search(beamed, a.users, a.beams, a.steps, heads, words)
        y, more = whole_step(a.layer, a.format, [torch.cat((h, words[t])) for h, t in zip(heads, taken)])
        off = max(off, compared("the best of %d beams after %d tokens" % (a.beams, a.steps), got, y[ends_of(total)]))
        status |= more | beamed.status()
    print("status 0x%x" % status)
    return off, status


def ends_of(lengths):
    return (torch.tensor(lengths).cumsum(0) - 1).cuda()


if __name__ == "__main__":
    off, status = main()
    sys.exit(0 if off < 2e-2 and status == 0 else 1)
