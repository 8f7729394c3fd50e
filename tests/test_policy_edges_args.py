"""The policy loss's refusals around one advantage per sequence (no GPU needed)."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def gs():
    import mixed_precision_numerics_gradscaler_gb300 as gs
    return gs


def test_lengths_of_the_advantages(gs):
    P = ctypes.c_void_p(0x1000)  # never dereferenced
    f = lambda na, T, S: gs._lib.gs_policy_loss(P, P, None, P, na, None, T, P, S, 0.2, 0.2, 0.0, 0.0, 0, None,  # noqa: E731
                                                None, None, None, P, None)
    # past the lengths' check: the loss is missing
    assert f(8, 8, 3) == f(3, 8, 3) == f(-3, 8, 3) == f(8, 8, 8) == f(-8, 8, 8) == gs.GS_ERR_NULL
    assert f(-8, 8, 3) == f(7, 8, 3) == f(-7, 8, 3) == f(0, 8, 3) == f(-(1 << 63), 8, 3) == gs.GS_ERR_SHAPE


def test_binding_refuses_the_other_length(gs):
    v, off = torch.zeros(8), torch.tensor([0, 2, 8])
    ws = torch.zeros(gs.gs_policy_loss_ws_bytes(8, 2), dtype=torch.uint8)
    f = lambda adv, per: gs.gs_policy_loss(v, v, adv, torch.zeros(1), ws, seq_offsets=off, per_sequence=per, stream=0)  # noqa: E731
    for adv, per in ((v, True), (torch.zeros(2), False)):
        with pytest.raises(ValueError):
            f(adv, per)
    for adv, per in ((v, False), (v, None), (torch.zeros(2), True), (torch.zeros(2), None)):
        with pytest.raises(gs.GsError):                  # host memory
            f(adv, per)
