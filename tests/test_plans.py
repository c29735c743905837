"""Plans' Python side on the CPU: the places of their arguments."""

import inspect

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
