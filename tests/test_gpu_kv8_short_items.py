"""Many sequences of one block of positions each on the tensor-memory attention kernel: the
items that give one of its two issuing warps no round, mixed with items that do."""
import pytest
import torch

import bit_gemm_group_b200 as wq
import kv8_plain as plain

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clean_status():
    wq.wq_get_device_status(reset=True)
    yield
    assert wq.wq_get_device_status(reset=True) == wq.WQ_OK


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("D,longer", [(64, 0), (128, 7), (64, 3)])
def test_many_short_sequences(dtype, D, longer):
    # 10 rows of 4 heads over 2 kv heads: a dozen items to a CTA; every `longer`-th sequence
    # has two to five blocks
    seqs = [(10, 10 + (b * 7) % 55 + (70 * (1 + b % 4) if longer and b % longer == 0 else 0))
            for b in range(900)]
    st = plain.make_state(seqs, 8, 2, D, 64, torch.int8, dtype, seed=21)
    cache = plain.append(st["K"], st["V"], st["cache"], st["table"], st["cu"], st["lens"], None)
    d = plain.on_gpu(st)
    wq.kv8_append(d["K"], d["V"], d["cache"], d["table"], d["cu"], d["lens"], 10)
    ref, tol = plain.attention(st["Q"], cache, st["table"], st["cu"], st["lens"], None, D ** -0.5)
    first = None
    for _ in range(5):
        out = wq.attn_kv8(d["Q"], d["cache"], d["table"], d["cu"], d["lens"], 10)
        err = (out.cpu().double() - ref).abs()
        assert bool((err <= tol).all()), float((err / tol).max())
        assert first is None or torch.equal(out, first)
        first = out
