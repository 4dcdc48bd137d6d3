"""Edges of the 8-bit quantizers: an infinity saturates beside the largest finite number,
positions near the end of 32 bits are reported."""
import pytest
import torch

import bit_gemm_group_b200 as wq
import kv8_plain as plain

pytestmark = pytest.mark.gpu

I8, E4 = torch.int8, torch.uint8
BF, F32 = torch.bfloat16, torch.float32


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


@pytest.mark.parametrize("length", [2 ** 31 - 1, 2 ** 31 - 30, 2 ** 31 - 33])
def test_append_reports_positions_near_the_end_of_32_bits(length):
    st = plain.make_state([(2, 50), (2, 60)], 2, 2, 64, 32, I8, BF, seed=6)
    st["lens"][1] = length
    d = plain.on_gpu(st)
    wq.kv8_append(d["K"], d["V"], d["cache"], d["table"], d["cu"], d["lens"], 2)
    assert wq.wq_get_device_status(reset=True) == wq.WQ_ERR_ARG
    want = plain.append(st["K"], st["V"], st["cache"], st["table"][:1], st["cu"][:2],
                        st["lens"][:1], None)
    for a, b in zip(d["cache"], want):
        assert torch.equal(a.cpu().view(torch.uint8), b.view(torch.uint8))
