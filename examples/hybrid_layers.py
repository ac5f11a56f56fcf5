"""Two layers of a hybrid model: Gated DeltaNet, then causal softmax attention,
each behind a layer norm, on the library's calls.

Trains on packed sequences of different lengths (each repeats its first half,
which the attention layer learns to look up), then continues prompts token by
token: the mixer with ``gdn_decode`` on its state, the attention with
``attn_decode`` on its cache, or with ``kv_append`` and ``attn_paged`` on pages of
16 or of 4 bits.

    python examples/hybrid_layers.py [steps]
"""
import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gated_delta_rule_bwd_gb300 as gdn  # noqa: E402

VOCAB, DIM, HEADS, KEY_HEADS, D = 48, 256, 2, 1, 128
BF16 = torch.bfloat16


class PackedDeltaRule(torch.autograd.Function):
    """gdn_fwd_varlen with its gradient; every sequence starts from zero."""

    @staticmethod
    def forward(ctx, q, k, v, g, beta, cu):
        ctx.save_for_backward(q, k, v, g, beta, cu)
        return gdn.gdn_fwd_varlen(q, k, v, g, beta, cu)[0]

    @staticmethod
    def backward(ctx, do):
        q, k, v, g, beta, cu = ctx.saved_tensors
        r = gdn.gdn_bwd_varlen(q, k, v, g, beta, cu, None, do.contiguous())
        return r["dq"], r["dk"], r["dv"], r["dg"], r["dbeta"], None


class Hybrid:
    def __init__(self, device="cuda", seed=0):
        gen = torch.Generator().manual_seed(seed)

        def p(*shape):
            return (torch.randn(*shape, generator=gen) * shape[0] ** -0.5).to(device).requires_grad_()

        def norm():
            return [torch.ones(DIM, device=device, requires_grad=True),
                    torch.zeros(DIM, device=device, requires_grad=True)]

        self.embed = torch.randn(VOCAB, DIM, generator=gen).to(device).requires_grad_()
        self.norms = [norm(), norm(), norm()]
        self.mix_in, self.mix_gates = p(DIM, 3 * HEADS * D), p(DIM, 2 * HEADS)
        self.mix_out = p(HEADS * D, DIM)
        self.attn_in = p(DIM, (HEADS + 2 * KEY_HEADS) * D)
        self.attn_out, self.head = p(HEADS * D, DIM), p(DIM, VOCAB)

    def parameters(self):
        return [self.embed, *sum(self.norms, []), self.mix_in, self.mix_gates, self.mix_out,
                self.attn_in, self.attn_out, self.head]

    def mixer_inputs(self, x):
        """q, k (unit length, q scaled), v, the log gate and beta of tokens x [B, T, DIM]."""
        h = gdn.layer_norm(x, *self.norms[0])
        q, k, v = (h @ self.mix_in.to(BF16)).unflatten(-1, (3, HEADS, D)).unbind(2)
        q = F.normalize(q.float(), dim=-1) * D ** -0.5
        k = F.normalize(k.float(), dim=-1)
        gate, beta = (h @ self.mix_gates.to(BF16)).float().split(HEADS, dim=-1)
        return (q.to(BF16), k.to(BF16), v.contiguous(), -F.softplus(gate - 2).contiguous(),
                torch.sigmoid(beta).contiguous())

    def attention_inputs(self, x):
        """q, k and v as views of one projection."""
        h = gdn.layer_norm(x, *self.norms[1])
        qkv = (h @ self.attn_in.to(BF16)).unflatten(-1, (HEADS + 2 * KEY_HEADS, D))
        return qkv.split([HEADS, KEY_HEADS, KEY_HEADS], dim=2)

    def logits(self, x):
        return (gdn.layer_norm(x, *self.norms[2]) @ self.head.to(BF16)).float()

    def packed(self, tokens, cu):
        """Logits [1, T, VOCAB] of packed sequences."""
        x = self.embed[tokens][None].to(BF16)
        x = x + PackedDeltaRule.apply(*self.mixer_inputs(x), cu).flatten(2) @ self.mix_out.to(BF16)
        o = gdn.attention(*self.attention_inputs(x), cu_seqlens=cu)
        return self.logits(x + o.flatten(2) @ self.attn_out.to(BF16))

    @torch.no_grad()
    def prompt(self, tokens, slots):
        """Logits of prompts [B, T], and what generation goes on from."""
        x = self.embed[tokens].to(BF16)
        o, state = gdn.gdn_fwd(*self.mixer_inputs(x))
        x = x + o.flatten(2) @ self.mix_out.to(BF16)
        q, k, v = self.attention_inputs(x)
        B, T = tokens.shape
        caches = torch.zeros(2, B, slots, KEY_HEADS, D, dtype=BF16, device=tokens.device)
        caches[0, :, :T], caches[1, :, :T] = k, v
        lens = torch.full((B,), T, dtype=torch.int32, device=tokens.device)
        o, _ = gdn.attn_fwd(q, k, v)
        return self.logits(x + o.flatten(2) @ self.attn_out.to(BF16)), (state, *caches, lens)

    @torch.no_grad()
    def to_pages(self, memory, page=16, bits=None):
        """The memory of ``prompt`` with the attention's part in pages, in no order."""
        state, k_cache, v_cache, lens = memory
        B, slots = k_cache.shape[:2]
        each = -(-slots // page)
        cache = gdn.new_paged_cache(B * each, page, KEY_HEADS, D, bits=bits, device=lens.device)
        table = torch.randperm(B * each, device=lens.device).int().view(B, each)
        seen = int(lens.max())
        gdn.kv_append(k_cache[:, :seen], v_cache[:, :seen], cache, table, torch.zeros_like(lens))
        return state.clone(), cache, table, lens.clone()

    @torch.no_grad()
    def step(self, tokens, memory):
        """Logits of one more token per row [B, 1]; ``memory`` is extended."""
        state, k_cache, v_cache, lens = memory
        x = self.embed[tokens].to(BF16)
        o, _ = gdn.gdn_decode(*self.mixer_inputs(x), state)
        x = x + o.flatten(2) @ self.mix_out.to(BF16)
        q, k, v = (t.contiguous() for t in self.attention_inputs(x))
        if isinstance(k_cache, gdn.PagedCache):
            cache, table = k_cache, v_cache
            gdn.kv_append(k, v, cache, table, lens)
            o = gdn.attn_paged(q, cache, table, lens)
        else:
            o = gdn.attn_decode(q, k, v, k_cache, v_cache, lens)
        lens += 1
        return self.logits(x + o.flatten(2) @ self.attn_out.to(BF16))


def sequences(gen, lengths):
    """Random tokens whose second half repeats the first."""
    out = []
    for n in lengths:
        half = torch.randint(VOCAB, ((n + 1) // 2,), generator=gen)
        out.append(torch.cat([half, half])[:n])
    return out


def train(model, steps, seed=1):
    gen = torch.Generator().manual_seed(seed)
    opt = torch.optim.Adam(model.parameters(), lr=3e-3)
    losses = []
    for _ in range(steps):
        lengths = torch.randint(8, 160, (24,), generator=gen).tolist()
        tokens = torch.cat(sequences(gen, lengths)).cuda()
        ends = torch.tensor(lengths).cumsum(0)
        cu = torch.cat([torch.zeros(1, dtype=torch.long), ends]).to(torch.int32).cuda()
        target = tokens.roll(-1)
        target[ends.cuda() - 1] = -100  # a sequence's last token predicts nothing
        loss = F.cross_entropy(model.packed(tokens, cu)[0], target, ignore_index=-100)
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(loss.detach())
    return torch.stack(losses).tolist()


def generate(model, tokens, new):
    """Greedy continuation of prompts [B, T]: the new tokens [B, new] and the
    logits [B, new, VOCAB] that chose them."""
    logits, memory = model.prompt(tokens, tokens.shape[1] + new)
    chosen, seen = [], []
    last = logits[:, -1:]
    for _ in range(new):
        seen.append(last)
        chosen.append(last.argmax(-1))
        if len(chosen) < new:
            last = model.step(chosen[-1], memory)
    return torch.cat(chosen, 1), torch.cat(seen, 1)


def follow(model, tokens, memory):
    """The logits [B, n, VOCAB] after each of the tokens [B, n]."""
    return torch.cat([model.step(t[:, None], memory) for t in tokens.unbind(1)], 1)


def main(steps=1000):
    model = Hybrid()
    losses = train(model, steps)
    gen = torch.Generator().manual_seed(2)
    half = torch.randint(VOCAB, (4, 40), generator=gen).cuda()
    prompts = torch.cat([half, half[:, :8]], 1)
    tokens, step_logits = generate(model, prompts, 24)
    whole, _ = model.prompt(torch.cat([prompts, tokens], 1), prompts.shape[1] + 24)
    whole = whole[:, prompts.shape[1] - 1:-1]
    result = {"first": losses[0], "last": losses[-1],
              "repeated": (tokens == half[:, 8:32]).float().mean().item(),
              "difference": (step_logits - whole).abs().max().item(),
              "largest": whole.abs().max().item()}
    # the same tokens again, on the contiguous cache and on pages
    _, memory = model.prompt(prompts, prompts.shape[1] + 24)
    pages = {n: model.to_pages(memory, bits=b) for n, b in (("paged", None), ("paged_4_bits", 4))}
    plain = follow(model, tokens, memory)
    for n, m in pages.items():
        result[n] = (follow(model, tokens, m) - plain).abs().max().item()
    assert gdn.device_status() == 0
    return result


if __name__ == "__main__":
    r = main(int(sys.argv[1]) if len(sys.argv) > 1 else 1000)
    print(f"loss {r['first']:.3f} -> {r['last']:.3f}; {100 * r['repeated']:.0f} % of the generated tokens "
          f"repeat the prompt; token by token and whole logits differ by at most {r['difference']:.4f} "
          f"(largest {r['largest']:.2f}); on pages they are {r['paged']:.4f} off, on pages of 4 bits "
          f"{r['paged_4_bits']:.4f}")
