"""Serving attention layers from an NVFP4 cache: random weights, three phases.

1. A prefix that all sequences share goes through the layers in chunks, once.
2. The sequences' own prompts, of different lengths, go through together; each
   sees the prefix's pages in front of its own.
3. Single tokens, one a sequence and step, in a captured graph.

A layer is nvfp4_linear (packed q, k, v) -> nvfp4_qk_norm_rope_write ->
nvfp4_kv_attention -> nvfp4_linear, added to its input.  --check compares the
last step's attention with plain fp32 attention over the rows that
nvfp4_kv_read gives back.

    python examples/serve_attention.py --batch 32 --prefix 4000 --steps 64 --check
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import quantized_gemm_nvfp4_amd as nv  # noqa: E402


def rotation_table(positions, rot_dim, base=10000.0, device="cuda"):
    """fp32 [positions, rot_dim]: rot_dim/2 cosines, then rot_dim/2 sines."""
    freq = base ** (-torch.arange(0, rot_dim, 2, device=device, dtype=torch.float64) / rot_dim)
    angle = torch.arange(positions, device=device, dtype=torch.float64)[:, None] * freq
    return torch.cat((angle.cos(), angle.sin()), 1).float()


class Layer:
    def __init__(self, hidden, q_heads, kv_heads, d, pages, page_size, seed):
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def weight(n, k):
            w = torch.randn((n, k), generator=gen, device="cuda", dtype=torch.float32) * k ** -0.5
            return nv.nvfp4_quantize(w.bfloat16())

        self.hq, self.hkv, self.d = q_heads, kv_heads, d
        self.w_qkv = weight((q_heads + 2 * kv_heads) * d, hidden)
        self.w_out = weight(hidden, q_heads * d)
        self.q_norm = (1 + 0.1 * torch.randn(d, generator=gen, device="cuda")).bfloat16()
        self.k_norm = (1 + 0.1 * torch.randn(d, generator=gen, device="cuda")).bfloat16()
        self.cache = nv.nvfp4_kv_cache(pages, page_size, kv_heads, d)

    def qkv(self, x):
        packed = nv.nvfp4_linear(x, self.w_qkv)[0].view(x.shape[0], self.hq + 2 * self.hkv, self.d)
        return packed.split((self.hq, self.hkv, self.hkv), 1)

    def calibrate(self, x):
        """The cache's global scales from the first tokens: a normed key is at
        most sqrt(D) times its weight, and a rotation no more than sqrt(2) on
        top; values get a factor of four above what is seen."""
        self.cache.k_gscale.copy_(self.k_norm.float().abs().amax() * (2 * self.d) ** 0.5 / 2688)
        self.cache.v_gscale.copy_(self.qkv(x)[2].float().abs().amax() * 4 / 2688)

    def __call__(self, x, table, positions, slots, *, kept=None, **attention):
        q, k, v = self.qkv(x)
        q = nv.nvfp4_qk_norm_rope_write(q, k, v, self.q_norm, self.k_norm, table, positions, self.cache, slots)
        o = nv.nvfp4_kv_attention(q, self.cache, **attention)
        if kept is not None:
            kept.update(q=q, o=o)
        return x + nv.nvfp4_linear(o.view(x.shape[0], -1), self.w_out)[0]


class Server:
    """`layers` layers over one page table: the prefix's pages, then room for
    `room` tokens of each sequence."""

    def __init__(self, layers, hidden, q_heads, kv_heads, d, page_size, batch, prefix, room, seed=0):
        self.prefix, self.ps, self.batch = prefix, page_size, batch
        n_prefix, n_own = -(-prefix // page_size), -(-room // page_size)
        pages = n_prefix + batch * n_own
        order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).int().cuda()
        self.prefix_pages = order[:n_prefix].contiguous()
        self.page_table = order[n_prefix:].view(batch, n_own).contiguous()
        self.lens = torch.zeros(batch, dtype=torch.int32, device="cuda")
        self.table = rotation_table(prefix + room, d)
        self.layers = [Layer(hidden, q_heads, kv_heads, d, pages, page_size, seed + 1 + i) for i in range(layers)]

    def slots(self, pages, tokens):
        """Slots of token numbers `tokens` [n, m] in page rows `pages` [n, width]."""
        tokens = tokens.long()
        return (pages.long().gather(1, tokens // self.ps) * self.ps + tokens % self.ps).view(-1)

    def fill_prefix(self, x, chunk):
        """The shared prefix x [prefix, hidden] in chunks, as a sequence of its own."""
        pages, out = self.prefix_pages[None], []
        for t0 in range(0, self.prefix, chunk):
            t1 = min(t0 + chunk, self.prefix)
            at = torch.arange(t0, t1, dtype=torch.int32, device="cuda")
            h = x[t0:t1]
            for layer in self.layers:
                if t0 == 0:
                    layer.calibrate(h)
                h = layer(h, self.table, at, self.slots(pages, at[None]), page_table=pages,
                          kv_lens=torch.tensor([t1], dtype=torch.int32, device="cuda"),
                          q_starts=torch.tensor([0, t1 - t0], dtype=torch.int32, device="cuda"),
                          max_q_len=t1 - t0, max_kv_len=t1)
            out.append(h)
        return torch.cat(out) if out else x

    def fill_prompts(self, x, lengths):
        """All sequences' prompts, packed in x [sum of lengths, hidden]."""
        at = torch.cat([torch.arange(n, dtype=torch.int32) for n in lengths]).cuda()
        rows = torch.repeat_interleave(torch.arange(self.batch), torch.tensor(lengths)).cuda()
        slots = self.slots(self.page_table[rows], at[:, None])
        starts = torch.tensor([0] + lengths).cumsum(0).int().cuda()
        self.lens.copy_(torch.tensor(lengths, dtype=torch.int32))
        h = x
        for layer in self.layers:
            if self.prefix == 0:
                layer.calibrate(h)
            h = layer(h, self.table, at + self.prefix, slots, page_table=self.page_table, kv_lens=self.lens,
                      q_starts=starts, max_q_len=max(lengths), max_kv_len=max(lengths), prefix_pages=self.prefix_pages,
                      prefix_len=self.prefix)
        return h

    def step(self, x, kept=None):
        """One token a sequence, in place of x [batch, hidden]; the lengths
        advance on the device, so that a graph of it can be replayed."""
        positions = self.lens + self.prefix
        slots = self.slots(self.page_table, self.lens[:, None])
        self.lens.add_(1)
        h = x
        for layer in self.layers:
            h = layer(h, self.table, positions, slots, page_table=self.page_table, kv_lens=self.lens,
                      prefix_pages=self.prefix_pages, prefix_len=self.prefix, kept=kept)
        x.copy_(h / h.float().square().mean(1, keepdim=True).sqrt())

    def plain_attention(self, q, layer):
        """fp32 attention of q [batch, q_heads, D] over the rows read back."""
        prefix_slots = self.slots(self.prefix_pages[None], torch.arange(self.prefix, device="cuda")[None])
        out = []
        for b, n in enumerate(self.lens.tolist()):
            own = self.slots(self.page_table[b:b + 1], torch.arange(n, device="cuda")[None])
            k, v = (t.float().transpose(0, 1) for t in nv.nvfp4_kv_read(layer.cache, torch.cat((prefix_slots, own))))
            qb = q[b].float().view(layer.hkv, -1, layer.d)
            p = ((qb[:, :, None] * k[:, None]).sum(-1) * layer.d ** -0.5).softmax(-1)
            out.append((p[..., None] * v[:, None]).sum(2).view(layer.hq, layer.d))
        return torch.stack(out)


def captured(server, x):
    """A graph of server.step(x), captured after a run on a side stream."""
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    saved = server.lens.clone(), x.clone()
    with torch.cuda.stream(side):
        server.step(x)
    torch.cuda.current_stream().wait_stream(side)
    server.lens.copy_(saved[0])
    x.copy_(saved[1])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        server.step(x)
    return graph


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("layers", 2), ("hidden", 5376), ("q-heads", 42), ("kv-heads", 6), ("head-dim", 128),
                        ("page-size", 64), ("batch", 16), ("prefix", 2000), ("chunk", 1024), ("prompt", 300),
                        ("steps", 32)):
        ap.add_argument("--" + name, type=int, default=value)
    ap.add_argument("--check", action="store_true")
    a = ap.parse_args(argv)
    s = Server(a.layers, a.hidden, a.q_heads, a.kv_heads, a.head_dim, a.page_size, a.batch, a.prefix,
               a.prompt + a.steps + 2)
    gen = torch.Generator(device="cuda").manual_seed(7)

    def tokens(n):
        return torch.randn((n, a.hidden), generator=gen, device="cuda").bfloat16()

    lengths = [1 + (a.prompt - 1) * b // max(1, a.batch - 1) for b in range(a.batch)]
    s.fill_prefix(tokens(a.prefix), a.chunk)
    last = s.fill_prompts(tokens(sum(lengths)), lengths)
    x = last[torch.tensor(lengths).cumsum(0).cuda() - 1].contiguous()
    graph = captured(s, x)
    torch.cuda.synchronize()
    t = time.perf_counter()
    for _ in range(a.steps):
        graph.replay()
    torch.cuda.synchronize()
    ms = (time.perf_counter() - t) / a.steps * 1e3
    print(f"{a.layers} layers, {a.batch} sequences behind a prefix of {a.prefix}: {ms:.3f} ms a step, "
          f"{a.batch / ms * 1e3:.0f} tokens/s")
    if a.check:
        kept = {}
        s.step(x, kept)
        want = s.plain_attention(kept["q"], s.layers[-1])
        err = ((kept["o"].float() - want).norm() / want.norm()).item()
        print(f"attention of the last layer against fp32 over the rows read back: relative error {err:.2e}")
        # nvfp4_kv_read rounds the rows to bf16: 2^-8 on each; the output rounds once more
        if not err < 2.0 ** -6:
            raise SystemExit("the check failed")


if __name__ == "__main__":
    main()
