"""One decoder layer's attention block over a few decode steps.

    python examples/decode_block.py [--sequences 8] [--steps 4] [--heads 40] [--kv-heads 8]

Random weights of the chosen width (heads of 128 channels), a ragged batch of
prompts taken up in steps of at most 32 tokens, then decode steps of one token a
sequence, replayed from a graph.  Prints the time of a decode step.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from bit_weight_gemm_amd import binding as B  # noqa: E402
from bit_weight_gemm_amd import workloads as wl  # noqa: E402
from bit_weight_gemm_amd.decoder import AttentionBlock, Linear  # noqa: E402


def random_linear(N: int, K: int, r: int, seed: int, device="cuda") -> Linear:
    d = wl.make_inputs(1, K, N, r, seed, g=0.02 / K ** 0.5)

    def dev(a):
        return torch.from_numpy(a).to(device)
    return Linear(dev(d["wcodes_packed"]), dev(d["wscales"]), float(d["g"]),
                  B.biloco_pack_signs(dev(d["V"].T.copy())), B.biloco_pack_signs(dev(d["U"].T.copy())),
                  dev(d["alpha"].view("int16")), N, K, r)


def rope_table(n_pos: int, dim: int, device="cuda") -> torch.Tensor:
    freq = 10000.0 ** (-torch.arange(dim // 2, dtype=torch.float64) / (dim // 2))
    angle = torch.arange(n_pos, dtype=torch.float64)[:, None] * freq
    return torch.cat([angle.cos(), angle.sin()], 1).float().to(device)


class Batch:
    """Sequences, their pages, and the device arrays of one step."""

    def __init__(self, sequences: int, page: int, max_len: int, device="cuda"):
        self.lens, self.device = [0] * sequences, device
        per = -(-max_len // page)
        pages = torch.randperm(sequences * per).to(torch.int32)
        self.table = pages.reshape(sequences, per).contiguous().to(device)
        self.pages = sequences * per

    def take(self, new):
        """new[b] tokens more for each sequence: (positions, q_start, kv_len)."""
        pos = [p for n, k in zip(self.lens, new) for p in range(n, n + k)]
        self.lens = [n + k for n, k in zip(self.lens, new)]
        start = [0]
        for k in new:
            start.append(start[-1] + k)

        def dev(x):
            return torch.tensor(x, dtype=torch.int32, device=self.device)
        return dev([pos]), dev(start), dev(self.lens)


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--sequences", type=int, default=8)
    ap.add_argument("--prompt", type=int, default=100)
    ap.add_argument("--steps", type=int, default=4)
    ap.add_argument("--heads", type=int, default=40)
    ap.add_argument("--kv-heads", type=int, default=8)
    ap.add_argument("--rank", type=int, default=256)
    a = ap.parse_args()
    if not 1 <= a.sequences <= AttentionBlock.MAX_TOKENS:
        ap.error(f"--sequences is 1 to {AttentionBlock.MAX_TOKENS}, the rows of a product")
    if a.steps < 1:
        ap.error("--steps is at least 1")
    if a.prompt < 0:
        ap.error("--prompt is at least 0")
    d, width, page = 128, a.heads * 128, 32
    batch = Batch(a.sequences, page, a.prompt + a.steps + 1)
    ones = torch.ones(width, dtype=torch.bfloat16, device="cuda")
    block = AttentionBlock(random_linear((a.heads + 2 * a.kv_heads) * d, width, a.rank, 1),
                           random_linear(width, a.heads * d, a.rank, 2), a.heads, a.kv_heads, d,
                           B.biloco_kv_cache(batch.pages, a.kv_heads, page, d), rope_table(4096, d), ones, ones,
                           max_sequences=a.sequences, max_kv_len=a.prompt + a.steps + 1)

    def run(new, x):
        pos, start, lens = batch.take(new)
        h, codes, scales = x.clone(), *B.biloco_quant_act_fp4(x)
        res = x.clone()
        return block.step(h, codes, scales, res, pos, start, lens, batch.table, max(new))

    # the prompts, a sequence at a time in steps of at most 32 tokens
    for b in range(a.sequences):
        for at in range(0, a.prompt, 32):
            n = min(32, a.prompt - at)
            run([n if i == b else 0 for i in range(a.sequences)],
                torch.randn(n, width, device="cuda").to(torch.bfloat16))
    x = torch.randn(a.sequences, width, device="cuda").to(torch.bfloat16)
    for _ in range(a.steps):
        h, _, _ = run([1] * a.sequences, x)
    torch.cuda.synchronize()
    print(f"{a.steps} decode steps of {a.sequences} sequences, {batch.lens[0]} tokens each: "
          f"h is {'finite' if bool(torch.isfinite(h.float()).all()) else 'NOT finite'}")

    pos, start, lens = batch.take([1] * a.sequences)
    codes, scales = B.biloco_quant_act_fp4(x)
    res = x.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        block.step(x, codes, scales, res, pos, start, lens, batch.table, 1)
    for _ in range(3):
        g.replay()
    t0, t1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    t0.record()
    for _ in range(50):
        g.replay()
    t1.record()
    torch.cuda.synchronize()
    print(f"one step from a graph: {t0.elapsed_time(t1) / 50 * 1e3:.1f} us "
          f"({width} wide, {a.heads} heads, {a.kv_heads} key/value heads)")


if __name__ == "__main__":
    main()
