"""A whole training step of a sublayer, its backward through autograd, captured
into a graph and replayed on new values."""

from __future__ import annotations

import pytest
import torch

import sublayer_ref as R
from gpu_util import say
from test_sublayer import make, sublayer


@pytest.mark.gpu
@pytest.mark.parametrize("T,H,F", [(37, 264, 520), (130, 1288, 640)])
def test_training_step_in_a_graph(device, T, H, F):
    say(f"captured training step T={T} H={H} F={F}")
    p = make(T, 4, H, F, seed=T, dev=device)
    g = torch.randn(T, 4, H, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).to(device)

    def step(leaves):
        out = sublayer(leaves)
        return (out.detach(), *torch.autograd.grad(out, list(leaves.values()), g))

    held = {k: v.clone().requires_grad_() for k, v in p.items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(held)                                         # no graph of these leaves is left when it returns
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(held)
    for k in range(4):
        new = {n: (v * (1 + 0.25 * k)).contiguous() if n in ("streams", "w1") else v for n, v in p.items()}
        with torch.no_grad():
            for n, v in held.items():
                v.copy_(new[n])
        graph.replay()
        torch.cuda.synchronize()
        want = step({n: v.clone().requires_grad_() for n, v in new.items()})
        for a, b in zip(got, want):
            assert R.same_bytes(a, b), k
