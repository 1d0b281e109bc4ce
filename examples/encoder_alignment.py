"""A sequence encoder trained by Soft-DTW, then run sample by sample over a cache.

    python examples/encoder_alignment.py [--steps 100] [--dtype bf16|fp16|fp32] [--length 200]

Two recordings of the same motion at different speeds go through one pre-norm encoder
(layer norm, rotary positions, causal attention with shared key heads) and Soft-DTW aligns the
two feature sequences. The loss sets a pair of the same motion against one of different motions.
After the training one recording is encoded again as a stream, a new sample at a time over the
cache of keys and values, and compared with the whole sequence's encoding.
"""
import argparse
import math
import os
import sys

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))

import torch  # noqa: E402

from differentiable_series_alignment_gb300 import SoftDTW, attention, layer_norm, rotary, rotary_table  # noqa: E402

CHANNELS, WIDTH, HEADS, KEY_HEADS, HEAD, FEATURES = 6, 256, 4, 2, 64, 32


class Encoder(torch.nn.Module):
    def __init__(self, layers, length, dtype):
        super().__init__()
        self.dtype = dtype
        self.inputs = torch.nn.Linear(CHANNELS, WIDTH, dtype=dtype)
        self.outputs = torch.nn.Linear(WIDTH, FEATURES, dtype=dtype)
        qkv = (HEADS + 2 * KEY_HEADS) * HEAD
        self.qkv = torch.nn.ModuleList(torch.nn.Linear(WIDTH, qkv, bias=False, dtype=dtype) for _ in range(layers))
        self.mix = torch.nn.ModuleList(torch.nn.Linear(HEADS * HEAD, WIDTH, bias=False, dtype=dtype) for _ in range(layers))
        # weights and biases of the norms stay in fp32
        self.scale = torch.nn.ParameterList(torch.ones(WIDTH) for _ in range(layers + 1))
        self.shift = torch.nn.ParameterList(torch.zeros(WIDTH) for _ in range(layers + 1))
        self.register_buffer("table", rotary_table(length, HEAD, device="cuda"))

    def heads(self, layer, x, positions=None):
        """Turned queries and keys, and values, of a layer: slices of one projection."""
        h = self.qkv[layer](layer_norm(x, self.scale[layer], self.shift[layer]))
        h = h.view(*x.shape[:2], HEADS + 2 * KEY_HEADS, HEAD)
        q, k, v = h.split([HEADS, KEY_HEADS, KEY_HEADS], dim=2)
        q, k = rotary(q, k, table=self.table, positions=positions)
        return q, k, v

    def features(self, x):
        return self.outputs(layer_norm(x, self.scale[-1], self.shift[-1])).float()

    def forward(self, x, lengths=None):
        """Features (B, N, FEATURES) of a padded batch of series (B, N, CHANNELS)."""
        x = self.inputs(x.to(self.dtype))
        for layer, mix in enumerate(self.mix):
            q, k, v = self.heads(layer, x)
            o = attention(q, k, v, causal=True, q_lengths=lengths, k_lengths=lengths)
            x = x + mix(o.flatten(2))
        return self.features(x)


class Stream:
    """The same encoder over series that grow by a sample at a time."""

    def __init__(self, encoder, batch, length):
        self.encoder, self.seen = encoder, torch.zeros(batch, dtype=torch.int32, device="cuda")
        shape = (len(encoder.mix), batch, length, KEY_HEADS, HEAD)
        self.keys = torch.zeros(shape, dtype=encoder.dtype, device="cuda")
        self.values = torch.zeros_like(self.keys)

    @torch.no_grad()
    def push(self, sample):
        """Features (B, FEATURES) of the newest sample (B, CHANNELS) of every series."""
        e, batch = self.encoder, torch.arange(len(sample), device="cuda")
        x = e.inputs(sample[:, None].to(e.dtype))
        for layer, mix in enumerate(e.mix):
            q, k, v = e.heads(layer, x, positions=self.seen[:, None])
            self.keys[layer, batch, self.seen.long()] = k[:, 0]
            self.values[layer, batch, self.seen.long()] = v[:, 0]
            o = attention(q, self.keys[layer], self.values[layer], causal=True, k_lengths=self.seen + 1)
            x = x + mix(o.flatten(2))
        self.seen += 1
        return e.features(x)[:, 0]


def motions(count, length, gen):
    """`count` random motions, each recorded twice: at an even and at a wandering speed, every recording with
    noise and with an offset of its own in every channel."""
    freq = torch.rand(count, 1, CHANNELS, generator=gen, device="cuda") * 5 + 1
    phase = torch.rand(count, 1, CHANNELS, generator=gen, device="cuda") * 2 * math.pi
    even = torch.linspace(0, 1, length, device="cuda").expand(count, length)
    pace = torch.rand(count, length, generator=gen, device="cuda") + 0.2
    pace = torch.nn.functional.avg_pool1d(pace[:, None], 31, 1, 15, count_include_pad=False)[:, 0]
    wander = (pace.cumsum(1) - pace[:, :1]) / (pace.sum(1, keepdim=True) - pace[:, :1])
    record = lambda t: torch.sin(2 * math.pi * freq * t[..., None] + phase)  # noqa: E731
    noise = lambda: (0.3 * torch.randn(count, length, CHANNELS, generator=gen, device="cuda")  # noqa: E731
                     + 1.5 * torch.randn(count, 1, CHANNELS, generator=gen, device="cuda"))
    return record(even) + noise(), record(wander) + noise()


def main(argv=None):
    args = argparse.ArgumentParser()
    args.add_argument("--steps", type=int, default=100)
    args.add_argument("--dtype", choices=["bf16", "fp16", "fp32"], default="bf16")
    args.add_argument("--length", type=int, default=200)
    args = args.parse_args(argv)
    dtype = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}[args.dtype]
    torch.manual_seed(0)
    gen = torch.Generator(device="cuda").manual_seed(0)
    encoder = Encoder(layers=2, length=args.length, dtype=dtype).cuda()
    align = SoftDTW(gamma=1.0, fused=True)
    optimizer = torch.optim.SGD(encoder.parameters(), lr=0.02)
    first = last = None
    for step in range(args.steps):
        a, b = motions(16, args.length, gen)
        lengths = torch.randint(args.length // 2, args.length + 1, (16,), generator=gen, device="cuda", dtype=torch.int32)
        fa, fb = encoder(a, lengths), encoder(b, lengths)
        same = align(fa, fb, lengths, lengths) / lengths
        other = align(fa, fb.roll(1, 0), lengths, lengths.roll(1, 0)) / lengths
        loss = torch.nn.functional.softplus(same - other).mean()
        optimizer.zero_grad(set_to_none=True)
        loss.backward()
        torch.nn.utils.clip_grad_norm_(encoder.parameters(), 1.0)
        optimizer.step()
        last = loss.item()
        first = last if first is None else first
        if step % 20 == 0 or step == args.steps - 1:
            print(f"step {step:3d}  loss {last:.4f}  same {same.mean().item():.4f}  other {other.mean().item():.4f}")

    a, _ = motions(4, args.length, gen)
    with torch.no_grad():
        whole = encoder(a)
    stream = Stream(encoder, 4, args.length)
    grown = torch.stack([stream.push(a[:, n]) for n in range(args.length)], dim=1)
    off = ((grown - whole).norm() / whole.norm()).item()
    print(f"stream of {args.length} samples against the whole series: relative difference {off:.2e}")
    return first, last, off


if __name__ == "__main__":
    main()
