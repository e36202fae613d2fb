"""Logit rules whose lists are empty in this step."""

import pytest
import torch

from speculative_decoding_verification_padding_gb300 import api, build

pytestmark = pytest.mark.gpu


def _batch():
    build.build()
    dev = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    return dev, api.Batch(dev([0, 2, 3]), dev([-1, 0, -1]), dev([1, 2, 3]), 2), torch.randn(3, 50, device="cuda")


@pytest.mark.parametrize("penalty", [False, True])
def test_no_request_has_a_bias(penalty):
    dev, b, x = _batch()
    none = torch.empty(0, device="cuda")
    rules = api.LogitRules(bias_begin=dev([0, 0, 0]), bias_token=none.int(), bias_value=none,
                           presence=torch.tensor([0.5, 0.25], device="cuda") if penalty else None)
    out, status = torch.full_like(x, 7), dev([0])
    api.sv_shape_logits(b, x, rules, out, status)
    want = x.clone()
    if penalty:
        want[1, 2] -= 0.5  # row 1's own draft
    assert status.item() == 0 and torch.equal(out, want)


def test_offsets_into_an_empty_list_are_refused():
    dev, b, x = _batch()
    none = torch.empty(0, device="cuda")
    out, status = torch.full_like(x, 7), dev([0])
    api.sv_shape_logits(b, x, api.LogitRules(bias_begin=dev([0, 0, 1]), bias_token=none.int(), bias_value=none),
                        out, status)
    assert status.item() == api.N.SV_DEV_BAD_PARAM
    assert torch.equal(out[:2], x[:2]) and (out[2] == 7).all()
    with pytest.raises(api.N.SpecVerifyError):  # a list without values
        api.sv_shape_logits(b, x, api.LogitRules(bias_begin=dev([0, 0, 0]), bias_token=none.int()), out, status)


def test_rows_that_name_a_mask_there_is_not():
    # no masks in this step: rows that want one are reported, the others pass
    dev, b, x = _batch()
    masks = torch.empty(0, 2, dtype=torch.int32, device="cuda")
    for rows, want in (([-1, -1, -1], 0), ([-1, 0, -1], api.N.SV_DEV_BAD_PARAM)):
        out, status = torch.full_like(x, 7), dev([0])
        api.sv_shape_logits(b, x, api.LogitRules(mask=masks, mask_row=dev(rows)), out, status)
        assert status.item() == want and torch.equal(out, x)
    with pytest.raises(api.N.SpecVerifyError):  # a mask for every row, but there are none
        api.sv_shape_logits(b, x, api.LogitRules(mask=masks), out, status)
