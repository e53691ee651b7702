"""The attention half of a tensor-parallel layer on simulated ranks, prompt and single tokens.

Each of R ranks holds heads / R of the heads and its slice of the output projection.  One rank's step
is ar_qk_norm_rope (norm, rotation, rows of the caches), ar_attention over the rank's cache,
ar_fp8_quantize of the heads' outputs and ar_fp8_matmul with its slice of the weight, which leaves the
rank's partial in the wire type; ar_reduce_add sums the partials over the ranks and adds the residual.
All ranks live on one GPU, one after the other.

    python examples/tp_attention.py [--ranks 2] [--tokens 2048] [--steps 4] [--check]

--check compares every step with the same layer in plain 32-bit torch operations.
"""
from __future__ import annotations

import argparse
import math
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import mixed_precision_partial_amd as ar  # noqa: E402

BF16, F8 = torch.bfloat16, torch.float8_e4m3fn


def rope_table(positions: int, rot_dim: int, base: float, device) -> torch.Tensor:
    """Cosines and sines of position * base^(-2i / rot_dim), angles in 64 bits."""
    inv = base ** (-torch.arange(0, rot_dim, 2, dtype=torch.float64, device=device) / rot_dim)
    angle = torch.arange(positions, dtype=torch.float64, device=device)[:, None] * inv
    return torch.cat([angle.cos(), angle.sin()], 1).float()


class Rank:
    """One rank's weights, caches and buffers."""

    def __init__(self, gen, hidden, heads_q, heads_kv, head_dim, cache_rows, table, device):
        def normal(*shape, scale=1.0):
            return torch.randn(*shape, device=device, generator=gen) * scale

        self.heads = heads_q, heads_kv, head_dim
        self.qkv_weight = normal((heads_q + 2 * heads_kv) * head_dim, hidden, scale=hidden ** -0.5).to(BF16)
        self.q_norm, self.k_norm = (1 + 0.1 * normal(2, head_dim)).to(BF16).unbind(0)
        depth = heads_q * head_dim
        # the slice of the output projection in 8 bits, a scale for each block of 128 x 128
        w = normal(hidden, depth, scale=depth ** -0.5).view(hidden // 128, 128, depth // 128, 128)
        self.out_scales = (w.abs().amax((1, 3)) / 448).contiguous()
        self.out_codes = (w / self.out_scales[:, None, :, None]).clamp(-448, 448).to(F8).view(hidden, depth)
        self.k_cache = torch.zeros(cache_rows, heads_kv, head_dim, dtype=BF16, device=device)
        self.v_cache = torch.zeros_like(self.k_cache)
        self.table = table

    def step(self, ctx, x, batch):
        """This rank's partial [tokens, hidden] in bfloat16 for the tokens' hidden states x."""
        hq, hkv, d = self.heads
        t = x.shape[0]
        qkv = (x @ self.qkv_weight.t())
        q = qkv[:, :hq * d].view(t, hq, d)
        k = qkv[:, hq * d:(hq + hkv) * d].view(t, hkv, d)
        v = qkv[:, (hq + hkv) * d:].view(t, hkv, d)
        ar.ar_qk_norm_rope(ctx, q, k, self.q_norm, self.k_norm, self.table, batch["positions"],
                           k_out=self.k_cache, v=v, v_out=self.v_cache, slots=batch["slots"])
        o = torch.empty(t, hq, d, dtype=BF16, device=x.device)
        ar.ar_attention(ctx, o, q, self.k_cache, self.v_cache, batch["cu_q"], batch["k_start"], batch["k_len"],
                        batch["max_q"], batch["max_k"])
        codes = torch.empty(t, hq * d, dtype=F8, device=x.device)
        scales = torch.empty(t, hq * d // 128, device=x.device)
        ar.ar_fp8_quantize(ctx, codes, scales, o.view(t, hq * d))
        partial = torch.empty(t, self.out_codes.shape[0], dtype=BF16, device=x.device)
        ar.ar_fp8_matmul(ctx, partial, codes, scales, self.out_codes, self.out_scales)
        return partial

    def plain(self, x, batch, kept):
        """The same in 32-bit torch operations; ``kept`` holds this rank's keys and values by sequence."""
        hq, hkv, d = self.heads
        t = x.shape[0]
        qkv = (x @ self.qkv_weight.t()).float()
        q, k, v = qkv.split([hq * d, hkv * d, hkv * d], 1)
        angle = self.table[batch["positions"]][:, None]
        cos, sin = angle[..., :d // 2], angle[..., d // 2:]

        def turn(y, w):
            y = y.view(t, -1, d)
            y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6) * w.float()
            a, b = y[..., :d // 2], y[..., d // 2:]
            return torch.cat([a * cos - b * sin, b * cos + a * sin], -1).to(BF16).float()
        q, k, v = turn(q, self.q_norm), turn(k, self.k_norm), v.view(t, hkv, d).to(BF16).float()
        out = torch.empty(t, hq, d, device=x.device)
        cu = batch["cu_q"].tolist()
        for s in range(len(cu) - 1):
            rows = slice(cu[s], cu[s + 1])
            keys, values = kept.setdefault(s, (k[:0], v[:0]))
            keys, values = torch.cat([keys, k[rows]]), torch.cat([values, v[rows]])
            kept[s] = keys, values
            n, m = cu[s + 1] - cu[s], keys.shape[0]
            kk = keys.permute(1, 2, 0).repeat_interleave(hq // hkv, 0).contiguous()
            vv = values.transpose(0, 1).repeat_interleave(hq // hkv, 0).contiguous()
            z = torch.matmul(q[rows].transpose(0, 1), kk) / math.sqrt(d)
            z.masked_fill_(torch.ones(n, m, dtype=torch.bool, device=x.device).triu_(m - n + 1), -math.inf)
            out[rows] = torch.matmul(z.softmax(-1), vv).transpose(0, 1)
        o = out.reshape(t, -1, 128)
        scale = o.abs().amax(-1, keepdim=True) / 448
        o = (o / scale.clamp(min=1e-30)).clamp(-448, 448).to(F8).float() * scale
        w = self.out_codes.float().view(self.out_scales.shape[0], 128, -1, 128) * self.out_scales[:, None, :, None]
        return (o.view(t, -1) @ w.view(self.out_codes.shape).t()).to(BF16)


def lay_out(lens_q, lens_k, cache, device):
    """A step's indices: new tokens of each sequence go to the end of its part of the cache."""
    starts = [i * cache for i in range(len(lens_q))]
    positions = torch.cat([torch.arange(k - q, k) for q, k in zip(lens_q, lens_k)])
    slots = torch.cat([torch.arange(s + k - q, s + k) for q, k, s in zip(lens_q, lens_k, starts)])
    cu = torch.tensor([sum(lens_q[:i]) for i in range(len(lens_q) + 1)], dtype=torch.int32)
    return {"positions": positions.to(device), "slots": slots.to(device), "cu_q": cu.to(device),
            "k_start": torch.tensor(starts).to(device), "k_len": torch.tensor(lens_k, dtype=torch.int32).to(device),
            "max_q": max(lens_q), "max_k": max(lens_k)}


def run(ranks=2, hidden=4096, heads_q=32, heads_kv=8, head_dim=128, prompts=(2048,), steps=4, check=False, quiet=False):
    """One prompt pass and ``steps`` single-token steps; returns the largest relative error (None unchecked)."""
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(1)
    cache = max(prompts) + steps
    table = rope_table(cache, head_dim, 10000.0, dev)
    members = [Rank(gen, hidden, heads_q // ranks, heads_kv // ranks, head_dim, cache * len(prompts), table, dev)
               for _ in range(ranks)]
    kept = [{} for _ in members]
    ctx = ar.ar_init(dev.index or 0)
    worst = 0.0
    try:
        lens = list(prompts)
        for step in range(steps + 1):
            new = lens if step == 0 else [1] * len(lens)
            batch = lay_out(new, lens, cache, dev)
            x = torch.randn(sum(new), hidden, device=dev, generator=gen)
            torch.cuda.synchronize()
            began = time.perf_counter()
            partials = [m.step(ctx, x.to(BF16), batch) for m in members]
            y = torch.empty_like(x)
            # (the reduce takes its stream; the layer's operators are on torch's current one)
            ar.ar_reduce_add(ctx, [y], partials, y.numel(), ar.AR_F32, ar.AR_BF16, ar.AR_MODE_AUTO | ar.AR_SRC_WIRE, x,
                             stream=torch.cuda.current_stream())
            torch.cuda.synchronize()
            took = time.perf_counter() - began
            line = f"{'prompt' if step == 0 else 'token '} {sum(new):6d} rows, caches {max(lens)}: {took * 1e3:8.3f} ms"
            if check:
                plain = [m.plain(x.to(BF16), batch, kept[r]) for r, m in enumerate(members)]
                want = sum(p.float() for p in plain)
                far = float(((y - x) - want).norm() / want.norm())
                worst = max(worst, far)
                line += f", {far:.2e} from plain torch"
            if not quiet:
                print(line, flush=True)
            lens = [n + 1 for n in lens]
    finally:
        torch.cuda.synchronize()
        ar.ar_free(ctx)
    return worst if check else None


if __name__ == "__main__":
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--ranks", type=int, default=2, choices=(2, 4, 8))
    p.add_argument("--tokens", type=int, default=2048)
    p.add_argument("--steps", type=int, default=4)
    p.add_argument("--check", action="store_true")
    args = p.parse_args()
    run(args.ranks, prompts=(args.tokens, max(1, args.tokens // 3)), steps=args.steps, check=args.check)
