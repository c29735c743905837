"""Plans' Python side on the CPU: the places of their arguments, the device of their graphs."""

import contextlib
import inspect

import pytest
import torch

from moe_expert_layer_r3_amd.block import JoinPlan, NormPlan, RoutePlan
from moe_expert_layer_r3_amd.dense import GatedFFNPlan, LinearPlan, MoELayerPlan
from moe_expert_layer_r3_amd.layer import ForwardPlan, TrainPlan


def test_arguments_keep_their_places():
    """Arguments that came later stand behind the others, which callers may give by position."""
    places = lambda fn: list(inspect.signature(fn).parameters)[1:]
    for fn, first in (
            (MoELayerPlan.__init__, "T d f E k fs act act8 router_bias device"),
            (MoELayerPlan.forward, "x Wr wts W13s W2s br"),
            (ForwardPlan.__init__, "T d f E L k e0 device save_gu pow2 mxfp4"),
            (TrainPlan.__init__, "T d f E L k e0 device pow2 mxfp4"),
            (TrainPlan.backward, "x dy wts events"),
            (LinearPlan.__init__, "T K N act out_dtype train bias device"),
            (GatedFFNPlan.__init__, "T d f act save bias device")):
        first = first.split()
        assert places(fn)[:len(first)] == first, fn.__qualname__


@pytest.mark.parametrize("cls,args", [(RoutePlan, 1), (NormPlan, 2), (JoinPlan, 2), (LinearPlan, 2), (GatedFFNPlan, 3)])
def test_graphs_are_of_the_plans_device(cls, args, monkeypatch):
    """Streams, graph and calls of a capture on the plan's device, whichever is current."""
    seen, current = [], [0]

    class On:
        def __init__(self, device):
            self.to = current[0] if device is None else torch.device(device).index

        def __enter__(self):
            self.was, current[0] = current[0], self.to

        def __exit__(self, *a):
            current[0] = self.was

    class Stream:
        def __init__(self):
            seen.append(("stream", current[0]))

        def wait_stream(self, other):
            pass

    class Graph:
        def __init__(self, *a):
            seen.append(("graph", current[0]))

        def __enter__(self):
            pass

        def __exit__(self, *a):
            pass
    for name, fake in dict(device=On, Stream=Stream, current_stream=Stream, stream=lambda s: contextlib.nullcontext(),
                           CUDAGraph=Graph, graph=Graph).items():
        monkeypatch.setattr(torch.cuda, name, fake)
    monkeypatch.setattr(cls, "forward", lambda self, *a, **kw: seen.append(("call", current[0])))
    plan = object.__new__(cls)
    plan.device = torch.device("cuda", 3)
    plan.capture(*[None] * args)
    assert {k for k, _ in seen} == {"stream", "graph", "call"} and {d for _, d in seen} == {3}
    assert current == [0]
