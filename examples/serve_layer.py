"""One decoder layer served end to end: a paged key/value cache, its attention and the MoE block.

    python examples/serve_layer.py [--layer sliding|global] [--format bf16|e4m3] [--users N] [--steps N]

Several users' prompts are taken in chunks and then continued by single tokens, all of them in the same
batches, the way a serving loop does it: per step, the new tokens' keys and values are written into the
cache (quantised for e4m3), the new queries attend to it, and the block of this library follows. The
projections are random and plain torch products: the layer's shapes and its data flow are what is shown.
The last tokens' outputs are compared with those of whole prompts in one step.
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
    """Attention over a paged cache, then the MoE block, for batches of any users' new tokens."""

    def __init__(self, kind, fmt, max_tokens, users, max_len, seed=0):
        self.hq, self.hkv, self.d, self.window = LAYERS[kind]
        per_user = -(-max_len // PAGE)
        self.kv = B.PagedKV(self.hq, self.hkv, self.d, PAGE, users * per_user, fmt, max_tokens=max_tokens, max_seqs=users)
        self.cache = self.kv.new_cache()
        # Pages are dealt out in turn, so that a user's lie apart.
        self.table = torch.arange(users * per_user, dtype=torch.int32, device="cuda").view(per_user, users).T.contiguous()
        g = torch.Generator(device="cuda").manual_seed(seed)
        width = (self.hq + 2 * self.hkv) * self.d
        self.w_qkv = torch.randn(B.HIDDEN, width, generator=g, device="cuda", dtype=torch.bfloat16) * B.HIDDEN ** -0.5
        self.w_out = torch.randn(self.hq * self.d, B.HIDDEN, generator=g, device="cuda",
                                 dtype=torch.bfloat16) * (self.hq * self.d) ** -0.5
        self.ffn = B.MoeFFN(B.MOE_FFN_FULL_LAYER, max_tokens)
        self.ffn_w = synth.make_weights(seed=seed, device="cuda")
        self.lengths = [0] * users

    def step(self, users, x, new):
        """x: [sum(new), 2816] bf16, the new tokens of `users` one after the other. Returns the layer's output."""
        for u, n in zip(users, new):
            self.lengths[u] += n
        cu = torch.tensor([0] + list(new)).cumsum(0).to(torch.int32).cuda()
        lengths = torch.tensor([self.lengths[u] for u in users], dtype=torch.int32).cuda()
        batch = B.KVBatch(cu, lengths, self.table[list(users)], max_new=max(new))
        qkv = (x @ self.w_qkv).view(-1, self.hq + 2 * self.hkv, self.d)
        q, k, v = qkv.split((self.hq, self.hkv, self.hkv), 1)
        self.kv.write(self.cache, batch, k, v)
        out, _ = self.kv.attention(self.cache, batch, q, window=self.window, sinks=4 if self.window else 0)
        return self.ffn.forward(x + out.flatten(1) @ self.w_out, self.ffn_w)


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--layer", choices=sorted(LAYERS), default="sliding")
    ap.add_argument("--format", choices=sorted(B.KV_FORMATS), default="bf16")
    ap.add_argument("--users", type=int, default=6)
    ap.add_argument("--steps", type=int, default=8, help="single tokens after the prompts")
    a = ap.parse_args(argv)
    prompts = [150 + 211 * u % 1300 for u in range(a.users)]
    total = [p + a.steps for p in prompts]
    x = [synth.make_x(n, seed=10 + u, device="cuda") for u, n in enumerate(total)]

    layer = Layer(a.layer, a.format, max(512 * a.users, sum(total)), a.users, max(total))
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
    status = layer.kv.status()[1] | layer.ffn.status()[1]

    whole = Layer(a.layer, a.format, sum(total), a.users, max(total))
    y = whole.step(range(a.users), torch.cat(x), total)
    ends = torch.tensor(total).cumsum(0) - 1
    want, got = y[ends.cuda()].float(), torch.stack(last).float()
    off = float((got - want).norm() / want.norm())
    print("%s layer, %s cache: %d users, %d tokens; last tokens step by step against whole prompts: %.2e off; "
          "status 0x%x" % (a.layer, a.format, a.users, sum(total), off, status))
    return off, status


if __name__ == "__main__":
    off, status = main()
    sys.exit(0 if off < 2e-2 and status == 0 else 1)
