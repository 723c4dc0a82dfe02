"""The example of the operators together: prompts, single tokens, single tokens from a graph.

A sequence taken token by token has to end where the same sequence taken as one prompt ends.  The
two differ in the cache's roundings (a page is rounded again when a larger token raises its
scale).  An E4M3 rounding is off by at most 2^-4 of a value, uniformly spread: 2^-4 * 0.75 /
sqrt(3) = 2.7 % rms; twice on keys (which move the scores, of unit variance, by as much) and
twice on values: below 2.7 % * 2 = 5.4 % of the attention branch, and the layers after it round to 8 bits
(under 1 % rms).  One block's output, which also holds the residual stream, within 2^-3."""
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


def model(layers=1):
    return example.Model(layers, 512, 768, 8, 2, 64, 3, 200, device=dev())


def inputs(n, seed):
    return torch.randn(n, 512, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16).to(dev())


def test_single_tokens_continue_a_prompt():
    lengths, extra = [130, 1, 66], 5
    x = [inputs(n + extra, 10 + b) for b, n in enumerate(lengths)]
    say("example: whole prompts")
    whole = model().prompt(torch.cat(x), [n + extra for n in lengths])
    ends = torch.tensor([n + extra for n in lengths]).cumsum(0)
    m = model()
    say("example: prompts, then single tokens")
    m.prompt(torch.cat([t[:n] for t, n in zip(x, lengths)]), lengths)
    for i in range(extra):
        got = m.single(torch.stack([t[n + i] for t, n in zip(x, lengths)]))
        ref = whole[ends - extra + i]
        err = (got.double() - ref.double()).norm(dim=1) / ref.double().norm(dim=1)
        assert (err <= 2.0 ** -3).all().item(), (i, err.tolist())
    assert m.kv_lens.tolist() == [n + extra for n in lengths]


def test_graph_steps_equal_eager_steps():
    """Replays against eager steps from the same cache, bit for bit."""
    lengths, steps = [70, 64, 3], 4
    x = inputs(sum(lengths), 20)
    outs = []
    for captured in (False, True):
        m = model(2)
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
            say("example: capture")
            with torch.cuda.graph(g):
                last.copy_(m.single(last))
            for i in range(1, steps):
                say(f"example: replay {i}")
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
