"""The decode example with a layer of experts in each block: it runs, and steps from a captured graph are the
eager steps, bit for bit (the choices change from step to step and stay on the device)."""
import importlib.util
import os

import pytest
import torch

from helpers import dev, say

pytestmark = pytest.mark.gpu

spec = importlib.util.spec_from_file_location(
    "decode_kv8", os.path.join(os.path.dirname(__file__), "..", "examples", "decode_kv8.py"))
example = importlib.util.module_from_spec(spec)
spec.loader.exec_module(example)


def test_graph_steps_equal_eager_steps():
    lengths, steps = [70, 64, 3], 4
    x = torch.randn(sum(lengths), 512, generator=torch.Generator().manual_seed(20)).to(torch.bfloat16).to(dev())
    outs = []
    for captured in (False, True):
        m = example.Model(2, 512, 328, 8, 2, 64, 3, 200, device=dev(), experts=16, top_k=4)
        say(f"example with experts: prompts, captured={captured}")
        y = m.prompt(x, lengths)
        last = y[torch.tensor(lengths).cumsum(0) - 1].clone()
        got = []
        if captured:
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                last.copy_(m.single(last))
            torch.cuda.current_stream().wait_stream(side)
            got.append(last.clone())
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                last.copy_(m.single(last))
            for i in range(1, steps):
                say(f"example with experts: replay {i}")
                g.replay()
                torch.cuda.synchronize()
                got.append(last.clone())
        else:
            for _ in range(steps):
                last.copy_(m.single(last))
                got.append(last.clone())
        outs.append(torch.stack(got))
    assert torch.isfinite(outs[0]).all().item()
    assert torch.equal(outs[0], outs[1])
