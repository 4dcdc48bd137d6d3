"""Edges of the 8-bit quantizers: an infinity saturates beside the largest finite number."""
import pytest
import torch

import bit_gemm_group_b200 as wq
import kv8_plain as plain

pytestmark = pytest.mark.gpu

I8, E4 = torch.int8, torch.uint8
F32 = torch.float32


@pytest.fixture(autouse=True)
def _clean_status():
    wq.wq_get_device_status(reset=True)
    yield
    assert wq.wq_get_device_status(reset=True) == wq.WQ_OK


def appended(st):
    d = plain.on_gpu(st)
    wq.kv8_append(d["K"], d["V"], d["cache"], d["table"], d["cu"], d["lens"], st["max_new"],
                  d["rope"])
    want = plain.append(st["K"], st["V"], st["cache"], st["table"], st["cu"], st["lens"],
                        st["rope"])
    return [t.cpu().view(torch.uint8) for t in d["cache"]], [t.view(torch.uint8) for t in want]


@pytest.mark.parametrize("code", [I8, E4])
def test_infinity_beside_the_largest_number_saturates(code):
    """The scale times 127 is above the largest fp32 number here."""
    top = torch.finfo(F32).max
    st = plain.make_state([(3, 20)], 2, 2, 64, 32, code, F32, seed=3)
    for x in (st["K"], st["V"]):
        x[0, 0, 3], x[0, 0, 4], x[1, 0, 5] = top, float("inf"), float("-inf")
        x[2, 1, 7], x[2, 1, 8] = float("inf"), -top
    got, want = appended(st)
    assert wq.wq_get_device_status(reset=True) == wq.WQ_ERR_NONFINITE
    for a, b in zip(got, want):
        assert torch.equal(a, b)
