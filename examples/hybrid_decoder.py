"""A small hybrid decoder with random weights, served the way the operators are meant to be used.

Blocks alternate between a Mamba-2 mixer and paged attention.  Ragged prompts go through in
chunks (state pools and paged caches carry a sequence from one chunk to the next), then tokens are
decoded one at a time:
    mixer       rssm_linear_attention for chunks, rssm_linear_attention_step for single tokens;
                the rows [z | x | B | C] of one projection are passed as views
    attention   rssm_paged_append, then rssm_paged_attention (a sliding window with sinks in
                every other attention block)
    around each block   rssm_block_norm: gate and norm of the block's output, scaled
                addition to the residual stream, norm before the next block
The projections are plain torch matrix products.

    python examples/hybrid_decoder.py [--steps 16] [--chunk 128] [--dtype bf16]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import replayssm_persistent_rssm_amd as rp  # noqa: E402

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


class HybridDecoder:
    """d_model 512; mixers with 8 heads of 64 x 128 state in 2 groups; attention with 8 query
    and 2 key/value heads of 64; `layers` blocks."""

    D, H, G, DIM, DSTATE, HQ, HKV, HD, VOCAB = 512, 8, 2, 64, 128, 8, 2, 64, 1000

    def __init__(self, layers=4, dtype="bf16", seed=0, device="cuda"):
        g = torch.Generator().manual_seed(seed)
        self.dtype, self.dev = DTYPES[dtype], torch.device(device)
        w = lambda i, o: (torch.randn(i, o, generator=g) / i ** 0.5).to(self.dtype).to(self.dev)   # noqa: E731
        f = lambda t: t.float().to(self.dev)                                                       # noqa: E731
        self.embed = torch.randn(self.VOCAB, self.D, generator=g).to(self.dtype).to(self.dev)
        self.head = w(self.D, self.VOCAB)
        self.first_norm = f(1 + 0.1 * torch.randn(self.D, generator=g))
        self.blocks = []
        for i in range(layers):
            b = dict(kind="mixer" if i % 2 == 0 else "attention", gate=w(self.D, self.D),
                     post=f(1 + 0.1 * torch.randn(self.D, generator=g)), pre=f(1 + 0.1 * torch.randn(self.D, generator=g)),
                     scale=f(torch.full((self.D,), 0.5)))
            if b["kind"] == "mixer":
                b.update(w_in=w(self.D, 2 * self.H * self.DIM + 2 * self.G * self.DSTATE), w_dt=w(self.D, self.H),
                         w_out=w(self.H * self.DIM, self.D), A=f(-torch.exp(torch.rand(self.H, generator=g) * 2.7)),
                         Dh=f(torch.rand(self.H, generator=g)),
                         bias=f(torch.log(torch.expm1(0.001 + 0.099 * torch.rand(self.H, generator=g)))))
            else:
                b.update(wq=w(self.D, self.HQ * self.HD), wk=w(self.D, self.HKV * self.HD),
                         wv=w(self.D, self.HKV * self.HD), wo=w(self.HQ * self.HD, self.D),
                         window=96 if i % 4 == 3 else 0, sinks=4 if i % 4 == 3 else 0)
            self.blocks.append(b)

    def new_cache(self, seqs, max_len, page=16):
        """State pools and paged caches of `seqs` sequences of up to max_len tokens."""
        pages = (max_len + page - 1) // page
        c = dict(slots=torch.arange(seqs, dtype=torch.int32, device=self.dev), length=[0] * seqs,
                 table=torch.randperm(seqs * pages).int().view(seqs, pages).to(self.dev), layer=[])
        for b in self.blocks:
            if b["kind"] == "mixer":
                c["layer"].append(torch.zeros(seqs, self.H, self.DIM, self.DSTATE, device=self.dev))
            else:
                kv = lambda: torch.zeros(seqs * pages, page, self.HKV, self.HD, dtype=self.dtype, device=self.dev)  # noqa: E731
                c["layer"].append((kv(), kv()))
        return c

    def forward(self, cache, tokens):
        """Logits after the last of each sequence's new tokens (a list of token lists, each possibly empty)."""
        lens = [len(t) for t in tokens]
        cache["length"] = [a + b for a, b in zip(cache["length"], lens)]
        starts = [0]
        for n in lens:
            starts.append(starts[-1] + n)
        N, single = starts[-1], all(n == 1 for n in lens)
        i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=self.dev)                        # noqa: E731
        seq_start, kv_len = i32(starts), i32(cache["length"])
        x = self.embed[torch.tensor([t for s in tokens for t in s], device=self.dev)]
        residual, normed = torch.empty(N, self.D, device=self.dev), torch.empty_like(x)
        # the first norm: nothing but the embedding in the stream
        rp.rssm_block_norm(x, torch.zeros_like(residual), residual, normed, pre_weight=self.first_norm)
        for b, kept in zip(self.blocks, cache["layer"]):
            out = self._mixer(b, kept, cache, normed, seq_start, max(lens), single) if b["kind"] == "mixer" else \
                self._attention(b, kept, cache, normed, seq_start, kv_len, max(lens))
            gate = normed @ b["gate"]
            rp.rssm_block_norm(out, residual, residual, normed, z=gate, post_weight=b["post"], pre_weight=b["pre"],
                               channel_scale=b["scale"])
        last = torch.tensor([e - 1 for s, e in zip(starts, starts[1:]) if e > s], device=self.dev)
        return normed[last] @ self.head

    def _mixer(self, b, pool, cache, h, seq_start, longest, single):
        N, di, bc = h.shape[0], self.H * self.DIM, self.G * self.DSTATE
        z, x, B, C = (h @ b["w_in"]).split([di, di, bc, bc], 1)      # views of one row
        heads = lambda t, n, d: t.unflatten(1, (n, d))                                             # noqa: E731
        dt = (h @ b["w_dt"]).float()
        y = torch.empty(N, self.H, self.DIM, dtype=self.dtype, device=self.dev)
        args = (pool, b["A"], heads(x, self.H, self.DIM), heads(B, self.G, self.DSTATE), heads(C, self.G, self.DSTATE), dt, y,
                cache["slots"])
        kw = dict(D=b["Dh"], dt_bias=b["bias"], z=heads(z, self.H, self.DIM))
        if single:
            rp.rssm_linear_attention_step(*args, **kw)
        else:
            rp.rssm_linear_attention(*args, seq_start, max_seq_len=longest, **kw)
        return y.view(N, di) @ b["w_out"]

    def _attention(self, b, kept, cache, h, seq_start, kv_len, longest):
        N = h.shape[0]
        q, k, v = ((h @ b[n]).view(N, -1, self.HD) for n in ("wq", "wk", "wv"))
        out = torch.empty_like(q)
        rp.rssm_paged_append(*kept, k, v, cache["table"], seq_start, kv_len)
        rp.rssm_paged_attention(q, *kept, cache["table"], seq_start, kv_len, out, max_seq_len=longest,
                                max_kv_len=max(cache["length"]), window=b["window"], sinks=b["sinks"])
        return out.view(N, -1) @ b["wo"]


def prefill(model, cache, prompts, chunk):
    """Prompts in chunks of up to `chunk` tokens; the logits after each prompt's last token."""
    done, logits = [0] * len(prompts), [None] * len(prompts)
    while any(d < len(p) for d, p in zip(done, prompts)):
        part = [p[d:d + chunk] for d, p in zip(done, prompts)]
        out = iter(model.forward(cache, part))
        for i, p in enumerate(part):
            done[i] += len(p)
            if p:
                logits[i] = next(out)
    return torch.stack(logits)


def generate(model, prompts, steps, chunk):
    """Greedy tokens of each prompt, and the logits of every step."""
    cache = model.new_cache(len(prompts), max(len(p) for p in prompts) + steps)
    logits = [prefill(model, cache, prompts, chunk)]
    tokens = [[] for _ in prompts]
    for _ in range(steps):
        for t, n in zip(tokens, logits[-1].argmax(-1).tolist()):
            t.append(n)
        logits.append(model.forward(cache, [[t[-1]] for t in tokens]))
    return tokens, torch.stack(logits)


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=16)
    ap.add_argument("--chunk", type=int, default=128)
    ap.add_argument("--dtype", choices=sorted(DTYPES), default="bf16")
    a = ap.parse_args()
    g = torch.Generator().manual_seed(1)
    prompts = [torch.randint(0, HybridDecoder.VOCAB, (n,), generator=g).tolist() for n in (300, 17, 129, 1)]
    tokens, _ = generate(HybridDecoder(dtype=a.dtype), prompts, a.steps, a.chunk)
    for p, t in zip(prompts, tokens):
        print(f"prompt of {len(p)} tokens -> {t}")


if __name__ == "__main__":
    main()
