"""The example looks at what the kernels report: an error that only the GPU
sees stops the training before the parameters change."""

import pytest
import torch

from test_gpu_head_example import _example
from tile_gaussian_splat_gb300 import binding as gs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("call", ["gs_expert_dispatch", "gs_expert_combine",
                                  "gs_expert_combine_bwd", "gs_expert_linear_fwd",
                                  "gs_expert_linear_bwd"])
def test_a_reported_error_stops_the_training(call, monkeypatch):
    ex = _example()
    made = []

    class Head(ex.FeatureHead):
        def __init__(self, *args, **kw):
            super().__init__(*args, **kw)
            made.append((self, {k: v.clone() for k, v in self.params.items()}))

    def reporting(*args, d_status=None, **kw):
        out = genuine(*args, d_status=d_status, **kw)
        if d_status is not None:
            d_status.fill_(5)  # as a wait that ran out does
        return out

    genuine = getattr(gs, call)
    monkeypatch.setattr(ex, "FeatureHead", Head)
    monkeypatch.setattr(gs, call, reporting)
    with pytest.raises(gs.GsError, match="TIMEOUT"):
        ex.train(steps=1)
    head, before = made[0]
    assert all(torch.equal(head.params[k], v) for k, v in before.items())
