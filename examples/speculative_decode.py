"""Speculative decoding of a toy model over a paged cache, with every step of the
server on the GPU: draft tokens by spec_verify_sample, pages and slots by
spec_verify_slots, cache writes by spec_verify_append, attention of the drafted
block by spec_verify_attention, and the accepted tokens by spec_verify.

    python examples/speculative_decode.py

The model is one attention layer between an embedding and its transpose, with
random weights; the drafter is the same model with noise on them.  Greedy output
is that of decoding token by token without drafts.
"""

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from speculative_decoding_verification_16_gb300 import binding as sv  # noqa: E402


class Toy:
    """Embedding, attention over a paged cache of its own, output head."""

    def __init__(self, vocab, heads, kv_heads, head_dim, pages, page, dtype, seed, noise=0.0,
                 device="cuda:0"):
        g = torch.Generator(device=device).manual_seed(seed)
        width = heads * head_dim

        def weight(*shape):
            w = torch.randn(*shape, device=device, generator=g) * shape[0] ** -0.5
            n = torch.Generator(device=device).manual_seed(seed + 1)
            return (w + noise * shape[0] ** -0.5
                    * torch.randn(*shape, device=device, generator=n)).to(dtype)
        self.heads, self.kv_heads, self.dim = heads, kv_heads, head_dim
        self.embed = weight(vocab, width) * vocab ** 0.5
        self.qkv = weight(width, (heads + 2 * kv_heads) * head_dim) * 1.5
        self.out = weight(width, width)
        self.place = weight(4096, width) * 32
        shape = (pages, page, kv_heads, head_dim)
        self.k, self.v = (torch.zeros(shape, dtype=dtype, device=device) for _ in range(2))

    def logits(self, tokens, plan, table, max_len, error):
        """Logits of the new tokens [n], whose keys and values enter the cache; the
        operators' flags go to ``error``."""
        x = self.embed[tokens] + self.place[plan.positions.long()]
        qkv = (x @ self.qkv).view(len(tokens), -1, self.dim)
        q, k, v = qkv.split([self.heads, self.kv_heads, self.kv_heads], 1)
        sv.spec_verify_append(k, v, plan.slots, self.k, self.v, dev_error=error)
        a, _ = sv.spec_verify_attention(q, self.k, self.v, table, plan.seq_lens, plan.row_offsets,
                                        max_len=max_len, dev_error=error)
        h = 0.2 * x + 2 * (a.flatten(1) @ self.out)
        return torch.nn.functional.layer_norm(h.float(), h.shape[1:]).to(x.dtype) @ self.embed.T


class Server:
    """Requests in flight: their lengths and pages, all on the device."""

    def __init__(self, B, pages, page, width, device="cuda:0"):
        i32 = dict(dtype=torch.int32, device=device)
        self.page, self.B = page, B
        self.context = torch.zeros(B, **i32)
        self.table = torch.zeros(B, width, **i32)
        self.free = torch.arange(pages, **i32)
        # the counts before and after a step, taken in turn
        self.held = [torch.zeros(B, **i32), torch.zeros(B, **i32)]
        self.count = [torch.full((1,), pages, **i32), torch.zeros(1, **i32)]
        self.error = torch.zeros(1, **i32)

    def plan(self, context, new, rows):
        p = sv.spec_verify_slots(context, new, self.table, self.held[0], self.free, self.count[0],
                                 page_size=self.page, n_rows=rows, held_out=self.held[1],
                                 free_count_out=self.count[1], dev_error=self.error)
        self.held.reverse()
        self.count.reverse()
        return p


def generate(target, draft, prompts, new_tokens, block, page, pages, width, temperature=0.0,
             seed=0):
    """Decode at least new_tokens after every prompt (lists of ids); block - 1
    tokens are drafted a step (block 1: plain decoding).  Returns the tokens of
    every request, its drafts' number and how many of them were accepted."""
    dev = target.embed.device
    B = len(prompts)
    s = Server(B, pages, page, width, dev)
    g = torch.Generator(device=dev).manual_seed(seed)
    temps = torch.full((B,), temperature, device=dev)
    vocab = target.embed.shape[0]
    i32 = dict(dtype=torch.int32, device=dev)

    # prompts but their last tokens, as one ragged chunk
    lens = torch.tensor([len(p) - 1 for p in prompts], **i32)
    rows = int(lens.sum())
    if rows:
        plan = s.plan(s.context, lens, rows)
        flat = torch.tensor([t for p in prompts for t in p[:-1]], device=dev)
        for model in {id(m): m for m in (target, draft)}.values():
            model.logits(flat, plan, s.table, int(lens.max()), s.error)
        s.context = s.context + lens
    last = torch.tensor([p[-1] for p in prompts], device=dev)
    out = [[] for _ in prompts]
    drafted = accepted = 0
    one, full = torch.ones(B, **i32), torch.full((B,), block, **i32)
    offsets = torch.arange(B + 1, **i32) * block
    workspace = sv.alloc_workspace(B, B * block, dev)
    while min(len(o) for o in out) < new_tokens:
        # the drafter's block, token by token; its last token's keys and values too,
        # for a block that is accepted whole
        tokens, rows_of = [last], []
        for j in range(block if block > 1 else 0):
            plan = s.plan(s.context + j, one, B)
            x = draft.logits(tokens[-1], plan, s.table, 1, s.error)
            if j == block - 1:
                break
            u = torch.rand(B, device=dev, generator=g).clamp_(max=1 - 2.0 ** -24)
            t, _ = sv.spec_verify_sample(x, u, temperature=temps, dev_error=s.error)
            tokens.append(t.long())
            rows_of.append(x)
        # the target over the whole block, and the verdict
        plan = s.plan(s.context, full, B * block)
        x = target.logits(torch.stack(tokens, 1).flatten(), plan, s.table, block, s.error)
        drafts = torch.stack(rows_of, 1).flatten(0, 1) if rows_of else x[:0]
        u = torch.rand(B * block, device=dev, generator=g).clamp_(max=1 - 2.0 ** -24)
        v = sv.spec_verify(x.contiguous(), drafts.contiguous(),
                           torch.stack(tokens[1:], 1).flatten().int() if rows_of
                           else torch.zeros(0, **i32),
                           u, full, offsets, max_len=block, temperature=temperature or 1.0,
                           mode=sv.SV_SAMPLE if temperature else sv.SV_GREEDY, want_conf=False,
                           workspace=workspace)
        got = v.tokens.view(B, block)
        last = got.gather(1, v.accept_len.long()[:, None])[:, 0].long()
        s.context = s.context + v.accept_len + 1
        for o, row, n in zip(out, got.tolist(), v.accept_len.tolist()):
            o += row[:n + 1]
        drafted += B * (block - 1)
        accepted += int(v.accept_len.sum())
        assert int(s.error) == 0 and int(v.dev_error) == 0, "device error flags raised"
    assert vocab > max(max(o) for o in out)
    return [o[:new_tokens] for o in out], drafted, accepted


def main():
    vocab, page, pages, width, block = 5003, 16, 512, 32, 6
    for dtype in (torch.float32, torch.bfloat16):
        shape = (vocab, 8, 2, 64, pages, page, dtype, 7)
        target, draft = Toy(*shape), Toy(*shape, noise=0.05)
        prompts = [list(range(10 + 7 * r, 10 + 7 * r + 3 + 11 * r)) for r in range(8)]
        a = (prompts, 48)
        kw = dict(page=page, pages=pages, width=width)
        spec, drafted, accepted = generate(target, draft, *a, block, **kw)
        plain, _, _ = generate(target, draft, *a, 1, **kw)
        same = sum(x == y for x, y in zip(spec, plain))
        print(f"{dtype}: greedy, {accepted} of {drafted} drafts accepted, "
              f"{same} of {len(prompts)} requests as without drafts")
        _, drafted, accepted = generate(target, draft, *a, block, temperature=0.8, **kw)
        print(f"{dtype}: temperature 0.8, {accepted} of {drafted} drafts accepted")


if __name__ == "__main__":
    main()
