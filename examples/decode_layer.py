"""One decode layer: attention over the 8-bit cache, then the predictor-gated
sparse FFN, for a batch of sequences that outgrow their cache's budget.

    python examples/decode_layer.py [--config llama70b] [--seqs 4] [--prompt 500] [--steps 64] [--keep 12]

Weights and inputs are synthetic (``workload``).  Each step runs, per layer: the
fused projection (torch), rotary positions with head norms (``qk_rope``), the
cache append (``kv_append``), attention with the blocks' weights added up
(``attend``), the output projection (torch), and the FFN (``layer``); a
sequence over its budget of blocks first loses those that were attended to
least (``kv_evict``).
"""

from __future__ import annotations

import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import activation_sparse_rank_amd as pi  # noqa: E402
import workload  # noqa: E402

BLOCK = 32
# Query heads, kv heads and head size beside each workload's FFN.
HEADS = {"tiny": (4, 2, 64), "opt30b": (56, 56, 128), "falcon40b": (128, 8, 64), "llama70b": (64, 8, 128)}


class DecodeLayer:
    """A layer's weights, its cache and the buffers of its calls."""

    def __init__(self, name: str, seqs: int, max_blocks: int, max_new: int, device="cuda", seed: int = 0):
        cfg = workload.get_config(name)
        self.cfg, self.seqs, self.max_blocks, self.max_new = cfg, seqs, max_blocks, max_new
        self.heads, self.kv_heads, self.head_dim = h, hk, d = HEADS[name]
        self.dtype = dt = {"f16": torch.float16, "f32": torch.float32}[cfg.wtype]
        g = torch.Generator(device=device).manual_seed(seed)

        def weight(rows, cols):
            return (torch.randn((rows, cols), generator=g, device=device) * rows ** -0.5).to(dt)

        self.w_qkv, self.w_out = weight(cfg.d_model, (h + 2 * hk) * d), weight(h * d, cfg.d_model)
        freqs = 10000.0 ** (-2.0 * torch.arange(d // 2, dtype=torch.float64, device=device) / d) / (2.0 * torch.pi)
        norm = torch.ones(d, device=device)
        self.rope = pi.Rope(freqs, d, q_norm=norm, k_norm=norm)
        n = seqs * hk * max_blocks
        table = torch.randperm(n, generator=g, device=device).to(torch.int32).view(seqs, hk, max_blocks)
        self.cache = pi.KVCache(torch.empty((n, 2, BLOCK * d), dtype=torch.uint8, device=device),
                                torch.empty((n, 2), device=device),
                                torch.empty((seqs, hk, 2, BLOCK, d), dtype=dt, device=device), table,
                                torch.zeros((seqs, hk, max_blocks), device=device))
        # a decode step's workspace and a prompt's
        self.ws = {m: pi.alloc_attend_workspace(self.cache, h, m, add_score=True) for m in {1, max_new}}
        L = workload.make_layer(cfg, 0, device)
        self.pred = pi.Predictor(L["p1"], L["p2"], L["c"])
        self.ffn = pi.FFN(L["w_up"], L["w_down_t"], cfg.act, b_up=L.get("b_up"), w_gate=L.get("w_gate"),
                          b_gate=L.get("b_gate"))
        self.ffn_ws = pi.alloc_workspace(self.pred, self.ffn, seqs * max_new)

    def __call__(self, x, pos, lens, q_start, max_new: int):
        """x [n_tok, d_model] at positions pos; lens counts the tokens held with these.  Returns x after the layer."""
        h, hk, d = self.heads, self.kv_heads, self.head_dim
        qkv = x @ self.w_qkv
        q, k, v = (t.unflatten(1, (-1, d)) for t in qkv.split((h * d, hk * d, hk * d), 1))
        pi.qk_rope(self.rope, q, k, pos)                     # in place, on the projection's rows
        pi.kv_append(self.cache, k, v, lens, q_start=q_start, max_new=max_new)
        out = torch.empty((x.shape[0], h, d), dtype=self.dtype, device=x.device)
        pi.attend(self.cache, q, lens, out, q_start=q_start, max_q=max_new, add_score=True, ws=self.ws[max_new])
        x = x + out.flatten(1) @ self.w_out
        y = torch.empty((x.shape[0], self.cfg.d_model), dtype=torch.float32, device=x.device)
        pi.layer(self.pred, self.ffn, x.contiguous(), self.cfg.tau, y, ws=self.ffn_ws)
        return x + y.to(self.dtype)


def run(name: str, seqs: int, prompt: int, steps: int, keep: int, recent: int = 2, device="cuda", seed: int = 0):
    """A prompt for every sequence, then steps tokens each.  Returns the last x and the lengths held."""
    max_blocks = max((prompt + BLOCK - 1) // BLOCK, keep) + 2
    layer = DecodeLayer(name, seqs, max_blocks, prompt, device, seed)
    x = workload.make_tokens(layer.cfg, 0, seqs * prompt, device)
    lens = torch.full((seqs,), prompt, dtype=torch.int32, device=device)
    pos = torch.arange(prompt, dtype=torch.int32, device=device).repeat(seqs)
    start = torch.arange(seqs + 1, dtype=torch.int32, device=device)
    x = layer(x, pos, lens, start * prompt, prompt)[prompt - 1::prompt].contiguous()
    held = torch.empty_like(lens)
    for i in range(steps):
        pi.kv_evict(layer.cache.table, layer.cache.score, lens, keep, recent, held)
        lens = held + 1
        x = layer(torch.nn.functional.rms_norm(x, (x.shape[1],)),
                  torch.full((seqs,), prompt + i, dtype=torch.int32, device=device), lens, start, 1)
    assert pi.read_flags(layer.ws[1]) == 0 and pi.read_flags(layer.ffn_ws) == 0
    return x, lens


def main(argv=None) -> int:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--config", choices=sorted(HEADS), default="llama70b")
    ap.add_argument("--seqs", type=int, default=4)
    ap.add_argument("--prompt", type=int, default=500)
    ap.add_argument("--steps", type=int, default=64)
    ap.add_argument("--keep", type=int, default=12, help="blocks of 32 tokens that a sequence may hold")
    a = ap.parse_args(argv)
    t0, t1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    t0.record()
    x, lens = run(a.config, a.seqs, a.prompt, a.steps, a.keep)
    t1.record()
    torch.cuda.synchronize()
    print(f"{a.config}: {a.seqs} sequences, {a.prompt} + {a.steps} tokens, held {lens.tolist()}, "
          f"|x| {x.float().norm(dim=1).mean().item():.3f}, {t0.elapsed_time(t1):.0f} ms with the weights' making")
    return 0


if __name__ == "__main__":
    sys.exit(main())
