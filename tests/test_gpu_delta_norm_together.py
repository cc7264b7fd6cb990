"""The gated delta rule and the group norm after its heads, several at once: on two streams, and in two graphs."""
import pytest
import torch

import implicit_gemm_conv_amd as igc
from tests.delta_cases import inputs

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
INS = ("q", "k", "v", "log_decay", "beta")


def _run(x):
    """Both passes of the rule and of the norm of its heads."""
    ins = [x[n] for n in INS]
    f = igc.delta_rule(*ins, h0=x["h0"], train=True)
    n = igc.group_norm(f.y.flatten(0, 1).flatten(1), f.y.shape[2], activation="silu")
    d = igc.group_norm_bwd(n.y, f.y.flatten(0, 1).flatten(1), f.y.shape[2], n.mean, n.rstd, activation="silu")
    g = igc.delta_rule_bwd(d.dx.view(f.y.shape), *ins, f.states, dh=x["dh"])
    return [f.y, f.h, n.y, d.dx, *g]


def _cases():
    # workgroups of 16 and of 32 columns, q and k that are copied first, and that are not
    return [inputs(31, 2, 300, 2, 4, 64, 96, torch.bfloat16, DEV), inputs(32, 6, 130, 3, 9, 65, 80, torch.float32, DEV)]


def test_two_streams_at_once():
    cases = _cases()
    want = [_run(x) for x in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [[], []]
    for _ in range(4):
        for i, (s, x) in enumerate(zip(streams, cases)):
            with torch.cuda.stream(s):
                got[i].append(_run(x))
    torch.cuda.synchronize()
    for i in range(2):
        for run in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(run, want[i]))


def test_two_graphs_in_turn():
    cases = _cases()
    want = [_run(x) for x in cases]
    held, graphs = [], []
    for x in cases:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            held.append(_run(x))
    for i in (0, 1, 1, 0, 1):
        for t in held[i]:
            t.fill_(7)
        graphs[i].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held[i], want[i]))
        _run(cases[1 - i])  # eager work between the replays
