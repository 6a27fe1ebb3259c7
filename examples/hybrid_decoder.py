"""A small hybrid decoder with random weights, served the way the operators are meant to be used.

Blocks alternate between state-space mixers (Mamba-2 and first-generation ones in turn) and paged attention.  Ragged
prompts go through in chunks (state pools and paged caches carry a sequence from one chunk to the next), then tokens are
decoded one at a time; a sequence may be forked at any point:
    mixer       rssm_causal_conv over [x | B | C] of one projection, then rssm_linear_attention for chunks;
                the _step forms of both for single tokens; z, x, B and C are passed as views of their rows
    selective   rssm_causal_conv over x, then rssm_selective_scan, likewise
    attention   rssm_rotary_append, then rssm_paged_attention (a sliding window with sinks in
                every other attention block)
    pages       rssm_page_extend before each call, rssm_page_fork, rssm_page_release and rssm_page_compact
                between calls: one table for the caches of all layers
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
    """d_model 512; mixers with 8 heads of 64 x 128 state in 2 groups; selective mixers with 512 channels of 16
    states; attention with 8 query and 2 key/value heads of 64, rotary positions on half of each; `layers` blocks."""

    D, H, G, DIM, DSTATE, HQ, HKV, HD, VOCAB = 512, 8, 2, 64, 128, 8, 2, 64, 1000
    TAPS, SD, RANK, ROT = 4, 16, 32, 32

    def __init__(self, layers=4, dtype="bf16", seed=0, device="cuda"):
        g = torch.Generator().manual_seed(seed)
        self.dtype, self.dev = DTYPES[dtype], torch.device(device)
        w = lambda i, o: (torch.randn(i, o, generator=g) / i ** 0.5).to(self.dtype).to(self.dev)   # noqa: E731
        f = lambda t: t.float().to(self.dev)                                                       # noqa: E731
        self.embed = torch.randn(self.VOCAB, self.D, generator=g).to(self.dtype).to(self.dev)
        self.head = w(self.D, self.VOCAB)
        self.first_norm = f(1 + 0.1 * torch.randn(self.D, generator=g))
        self.freq, self.factor = rp.rotary_frequencies(self.ROT, device=self.dev)
        self.blocks = []
        for i in range(layers):
            b = dict(kind=("mixer", "attention", "selective", "attention")[i % 4], gate=w(self.D, self.D),
                     post=f(1 + 0.1 * torch.randn(self.D, generator=g)), pre=f(1 + 0.1 * torch.randn(self.D, generator=g)),
                     scale=f(torch.full((self.D,), 0.5)))
            taps = lambda c: dict(conv=f(torch.randn(self.TAPS, c, generator=g) / self.TAPS ** 0.5),        # noqa: E731
                                  conv_bias=f(0.1 * torch.randn(c, generator=g)))
            if b["kind"] == "selective":
                b.update(w_x=w(self.D, self.D), w_bc=w(self.D, self.RANK + 2 * self.SD), w_dt=w(self.RANK, self.D),
                         w_out=w(self.D, self.D), A=f(-torch.arange(1, self.SD + 1).float().expand(self.D, self.SD).contiguous()),
                         Dh=f(torch.rand(self.D, generator=g)),
                         bias=f(torch.log(torch.expm1(0.001 + 0.099 * torch.rand(self.D, generator=g)))), **taps(self.D))
            elif b["kind"] == "mixer":
                b.update(**taps(self.H * self.DIM + 2 * self.G * self.DSTATE))
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
        most = (max_len + page - 1) // page
        i32 = lambda *shape, fill=0: torch.full(shape, fill, dtype=torch.int32, device=self.dev)   # noqa: E731
        c = dict(rows=torch.arange(seqs, dtype=torch.int32, device=self.dev), length=[0] * seqs, page=page,
                 table=i32(seqs, most, fill=-1), kv_len=i32(seqs), ref=i32(seqs * most), status=i32(seqs), layer=[])
        for b in self.blocks:
            if b["kind"] == "attention":
                kv = lambda: torch.zeros(seqs * most, page, self.HKV, self.HD, dtype=self.dtype, device=self.dev)  # noqa: E731
                c["layer"].append((kv(), kv()))
                continue
            state = (self.H, self.DIM, self.DSTATE) if b["kind"] == "mixer" else (self.D, self.SD)
            c["layer"].append((torch.zeros(seqs, *state, device=self.dev),
                               torch.zeros(seqs, self.TAPS - 1, b["conv"].shape[1], dtype=self.dtype, device=self.dev)))
        c["ptrs"] = rp.pointer_table([t for b, kept in zip(self.blocks, c["layer"]) if b["kind"] == "attention" for t in kept], self.dev)
        return c

    def _pool(self, cache):
        return cache["table"], cache["kv_len"], cache["ref"]

    def _page_bytes(self, cache):
        return cache["page"] * self.HKV * self.HD * self.embed.element_size()

    def fork(self, cache, src, dst):
        """Sequences `dst`, which are empty, become copies of sequences `src`; all of them or, with an error, none."""
        i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=self.dev)                        # noqa: E731
        status = i32([0] * len(dst))
        rp.rssm_page_fork(cache["ptrs"], *self._pool(cache), i32(src), i32(dst), status, page_size=cache["page"],
                          page_bytes=self._page_bytes(cache), token_bytes=self._page_bytes(cache) // cache["page"])
        if status.any():
            rp.rssm_page_release(*self._pool(cache), i32([d for d, s in zip(dst, status.tolist()) if s == rp.RSSM_PAGE_OK]),
                                 page_size=cache["page"])
            raise RuntimeError(f"not forked: {status.tolist()}")
        for b, kept in zip(self.blocks, cache["layer"]):
            if b["kind"] != "attention":
                for pool in kept:
                    pool[dst] = pool[src]
        for s, d in zip(src, dst):
            cache["length"][d] = cache["length"][s]

    def release(self, cache, rows, pack=False):
        """Sequences `rows` end and give their pages back; pack: the other pages move to the front of the pool, whose number
        is returned."""
        rp.rssm_page_release(*self._pool(cache), torch.tensor(rows, dtype=torch.int32, device=self.dev), page_size=cache["page"])
        for r in rows:
            cache["length"][r] = 0
        for b, kept in zip(self.blocks, cache["layer"]):
            if b["kind"] != "attention":
                for pool in kept:
                    pool[rows] = 0
        if pack:
            live = torch.zeros(1, dtype=torch.int32, device=self.dev)
            rp.rssm_page_compact(cache["ptrs"], *self._pool(cache), live, page_size=cache["page"], page_bytes=self._page_bytes(cache))
            return live.item()

    def forward(self, cache, tokens):
        """Logits after the last of each sequence's new tokens (a list of token lists, each possibly empty).  Where a sequence does not
        find its pages, an error, and the cache is as it was."""
        lens = [len(t) for t in tokens]
        starts = [0]
        for n in lens:
            starts.append(starts[-1] + n)
        N, single = starts[-1], all(n == 1 for n in lens)
        if N == 0:
            return self.head.new_empty(0, self.VOCAB)
        i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=self.dev)                        # noqa: E731
        seq_start = i32(starts)
        rp.rssm_page_extend(*self._pool(cache), cache["rows"], i32(lens), cache["status"], page_size=cache["page"])
        if cache["status"].any():        # appended all the same, these tokens would take the places of the row's last ones
            rp.rssm_page_release(*self._pool(cache), cache["rows"], lengths=i32(cache["length"]), page_size=cache["page"])
            raise RuntimeError(f"not extended: {cache['status'].tolist()}")
        cache["length"] = [a + b for a, b in zip(cache["length"], lens)]
        x = self.embed[torch.tensor([t for s in tokens for t in s], device=self.dev)]
        residual, normed = torch.empty(N, self.D, device=self.dev), torch.empty_like(x)
        # the first norm: nothing but the embedding in the stream
        rp.rssm_block_norm(x, torch.zeros_like(residual), residual, normed, pre_weight=self.first_norm)
        for b, kept in zip(self.blocks, cache["layer"]):
            out = {"mixer": self._mixer, "selective": self._selective, "attention": self._attention}[b["kind"]](
                b, kept, cache, normed, seq_start, max(lens), single)
            gate = normed @ b["gate"]
            rp.rssm_block_norm(out, residual, residual, normed, z=gate, post_weight=b["post"], pre_weight=b["pre"],
                               channel_scale=b["scale"])
        last = torch.tensor([e - 1 for s, e in zip(starts, starts[1:]) if e > s], device=self.dev)
        return normed[last] @ self.head

    def _conv(self, b, x, pool, cache, seq_start, single):
        y = torch.empty(x.shape, dtype=self.dtype, device=self.dev)
        args = (x, b["conv"], y, pool, cache["rows"])
        if single:
            rp.rssm_causal_conv_step(*args, bias=b["conv_bias"])
        else:
            rp.rssm_causal_conv(*args, seq_start, bias=b["conv_bias"])
        return y

    def _mixer(self, b, kept, cache, h, seq_start, longest, single):
        N, di, bc = h.shape[0], self.H * self.DIM, self.G * self.DSTATE
        z, xbc = (h @ b["w_in"]).split([di, di + 2 * bc], 1)         # views of one row
        x, B, C = self._conv(b, xbc, kept[1], cache, seq_start, single).split([di, bc, bc], 1)
        heads = lambda t, n, d: t.unflatten(1, (n, d))                                             # noqa: E731
        dt = (h @ b["w_dt"]).float()
        y = torch.empty(N, self.H, self.DIM, dtype=self.dtype, device=self.dev)
        args = (kept[0], b["A"], heads(x, self.H, self.DIM), heads(B, self.G, self.DSTATE), heads(C, self.G, self.DSTATE), dt, y,
                cache["rows"])
        kw = dict(D=b["Dh"], dt_bias=b["bias"], z=heads(z, self.H, self.DIM))
        if single:
            rp.rssm_linear_attention_step(*args, **kw)
        else:
            rp.rssm_linear_attention(*args, seq_start, max_seq_len=longest, **kw)
        return y.view(N, di) @ b["w_out"]

    def _selective(self, b, kept, cache, h, seq_start, longest, single):
        x = self._conv(b, h @ b["w_x"], kept[1], cache, seq_start, single)
        low, B, C = (x @ b["w_bc"]).split([self.RANK, self.SD, self.SD], 1)      # views of one row
        y = torch.empty_like(x)
        args = (kept[0], b["A"], x, B.unflatten(1, (1, self.SD)), C.unflatten(1, (1, self.SD)), low @ b["w_dt"], y, cache["rows"])
        kw = dict(D=b["Dh"], dt_bias=b["bias"])
        if single:
            rp.rssm_selective_scan_step(*args, **kw)
        else:
            rp.rssm_selective_scan(*args, seq_start, max_seq_len=longest, **kw)
        return y @ b["w_out"]

    def _attention(self, b, kept, cache, h, seq_start, longest, single):
        N = h.shape[0]
        q, k, v = ((h @ b[n]).view(N, -1, self.HD) for n in ("wq", "wk", "wv"))
        out, table, kv_len = torch.empty_like(q), cache["table"], cache["kv_len"]
        rp.rssm_rotary_append(q, q, *kept, k, v, table, seq_start, kv_len, self.freq, factor=self.factor)
        rp.rssm_paged_attention(q, *kept, table, seq_start, kv_len, out, max_seq_len=longest,
                                max_kv_len=max(cache["length"]), window=b["window"], sinks=b["sinks"])
        return out.view(N, -1) @ b["wo"]


def prefill(model, cache, prompts, chunk):
    """Prompts in chunks of up to `chunk` tokens; the logits after each prompt's last token (empty ones left out)."""
    done, logits = [0] * len(prompts), [None] * len(prompts)
    while any(d < len(p) for d, p in zip(done, prompts)):
        part = [p[d:d + chunk] for d, p in zip(done, prompts)]
        out = iter(model.forward(cache, part))
        for i, p in enumerate(part):
            done[i] += len(p)
            if p:
                logits[i] = next(out)
    rows = [row for row in logits if row is not None]
    return torch.stack(rows) if rows else model.head.new_empty(0, model.VOCAB)


def generate(model, prompts, steps, chunk):
    """Greedy tokens of each prompt (of a token or more), and the logits of every step."""
    if not all(prompts):
        raise ValueError("a prompt without tokens has nothing to go on from")
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
