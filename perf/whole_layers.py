"""Times a batch-one decode step through whole decoder layers of the 7B shapes (width 4096, 32 heads of
128, inner width 11008; fp16 weights, TopK-Guided masks at s = 0.5; random weights and caches):

    python3 perf/whole_layers.py [--keys 512 4096] [--capacity N] [--layers 32] [--steps 20]

For each length of the cache: the step called from Python, the same captured in a graph, and the
projections alone (spax_decode_step_projections on the same phases), in microseconds per token.
--capacity: the bound on the length that the attention is planned for, where it is not the length itself.
"""

import argparse
import math
import os
import sys
import time

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

import torch  # noqa: E402

import activation_sparse_tiered_amd as spax  # noqa: E402

WIDTH, HEADS, DIM, INNER, PAGE = 4096, 32, 128, 11008, 16
SPARSITY, DELTA = 0.5, 0.01
PHASES = [("qkv", WIDTH, [WIDTH] * 3), ("o", WIDTH, [WIDTH]), ("gate_up", WIDTH, [INNER] * 2),
          ("down", INNER, [WIDTH])]


class Step:
    """Layers that share their activations, each with its own weights and cache."""

    def __init__(self, n_layers, keys, capacity):
        g = torch.Generator(device="cuda").manual_seed(1)

        def rand(*shape, dtype=torch.float16, scale=1.0):
            return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)

        def empty(*shape, dtype=torch.float32):
            return torch.empty(*shape, dtype=dtype, device="cuda")

        position = torch.tensor([keys - 1], dtype=torch.int32, device="cuda")
        lens = position + 1
        inv = (1e4 ** (-torch.arange(0, DIM, 2, device="cuda").double() / DIM)).float()
        weight = torch.ones(WIDTH, device="cuda")
        token, h = rand(1, WIDTH, dtype=torch.float32), empty(1, WIDTH)
        x, x1, act = (empty(1, n, dtype=torch.float16) for n in (WIDTH, WIDTH, INNER))
        q, att = (empty(1, HEADS, DIM, dtype=torch.float16) for _ in range(2))
        y = {name: empty(sum(outs)) for name, _, outs in PHASES}
        masks = {name: (empty(d, dtype=torch.uint8), empty(d, dtype=torch.int32),
                        empty(d, dtype=torch.int32), empty(3, dtype=torch.int32))
                 for name, d, _ in PHASES}
        inputs = {"qkv": x, "o": att, "gate_up": x1, "down": act}
        rows = y["qkv"][None].split(WIDTH, 1)
        gate_up = y["gate_up"][None]
        layers, phases = [], []
        for _ in range(n_layers):
            p = {}
            for name, d, outs in PHASES:
                layout = spax.spax_layout_init(d, outs)
                packed = empty(int(layout.total_bytes), dtype=torch.uint8)
                spax.spax_pack_columns(layout, [rand(d, n, scale=0.02) for n in outs], packed)
                torch.cuda.synchronize()
                lo, hi = spax.spax_guided_bounds(d, SPARSITY, DELTA)
                p[name] = spax.make_phase(layout, packed, inputs[name],
                                          spax.guided_params(math.log(2), lo, hi, 3, 10),
                                          *masks[name], y[name])
            pages = (max(keys, capacity) + PAGE - 1) // PAGE
            k, v = (rand(pages, HEADS, PAGE, DIM) for _ in range(2))
            table = torch.randperm(pages, generator=g, device="cuda").int()[None].contiguous()
            cache = spax.make_kv_cache(k, v, table)
            layers.append(spax.make_layer(
                p["qkv"],
                spax.make_kv_append(cache, *(r.unflatten(1, (HEADS, DIM)) for r in rows), position, q,
                                    inv_freq=inv),
                spax.make_attention(cache, q, lens, att, max_len=capacity),
                p["o"],
                spax.make_residual_norm(h, y["o"][None], h, x1, pre_weight=weight),
                p["gate_up"],
                spax.make_glu(gate_up[:, :INNER], gate_up[:, INNER:], act),
                p["down"],
                spax.make_residual_norm(h, y["down"][None], h, x, pre_weight=weight)))
            phases += [p[name] for name, _, _ in PHASES]
        self.first = spax.make_residual_norm(token, None, h, x, pre_weight=weight)
        self.layers, self.phases = spax.layer_array(layers), spax.phase_array(phases)
        need = max(spax.spax_layers_workspace_bytes(self.layers),
                   spax.spax_step_workspace_bytes(self.phases))
        self.ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
        self.out = x

    def whole(self):
        spax.spax_residual_norm(self.first)
        spax.spax_decode_layers(self.layers, self.ws)

    def projections(self):
        spax.spax_decode_step_projections(self.phases, self.ws)


def timed(call, steps):
    for _ in range(3):
        call()
    torch.cuda.synchronize()
    start = time.perf_counter()
    for _ in range(steps):
        call()
    torch.cuda.synchronize()
    return (time.perf_counter() - start) / steps * 1e6


def main():
    a = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawTextHelpFormatter)
    a.add_argument("--keys", type=int, nargs="+", default=[512, 4096])
    a.add_argument("--capacity", type=int)
    a.add_argument("--layers", type=int, default=32)
    a.add_argument("--steps", type=int, default=20)
    a = a.parse_args()
    for keys in a.keys:
        step = Step(a.layers, keys, a.capacity or keys)
        whole = timed(step.whole, a.steps)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step.whole()
        replay = timed(graph.replay, a.steps)
        alone = timed(step.projections, a.steps)
        assert bool(torch.isfinite(step.out).all())
        print(f"{a.layers} layers, {keys} keys (planned for {a.capacity or keys}): whole step {whole:.0f} us, "
              f"in a graph {replay:.0f}, projections alone {alone:.0f}", flush=True)
        del step, graph
        torch.cuda.empty_cache()


if __name__ == "__main__":
    main()
