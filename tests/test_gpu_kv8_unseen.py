"""What a row of a call does not see does not reach it, whatever the cache holds there:
E4M3 codes that are no number, scales that are not finite.  Rows that do see them show it."""
import pytest
import torch

import bit_gemm_group_b200 as wq
import kv8_plain as plain

pytestmark = pytest.mark.gpu

I8, E4 = torch.int8, torch.uint8
BF, HF = torch.bfloat16, torch.float16
NAN, INF = float("nan"), float("inf")


@pytest.fixture(autouse=True)
def _clean_status():
    wq.wq_get_device_status(reset=True)
    yield
    assert wq.wq_get_device_status(reset=True) == wq.WQ_OK


# D, T, kv heads, G, type, (new, length) of each sequence: up to 32 rows to a kv head on
# mma.sync, 33 to 128 (and fp16) one tensor-memory tile, more two; runs that cut sequences
CASES = [
    (64, 16, 2, 2, BF, [(3, 40), (4, 9)]),
    (128, 32, 1, 4, BF, [(5, 900), (1, 70), (8, 8)]),
    (128, 16, 2, 4, HF, [(7, 2500)]),
    (256, 16, 1, 3, BF, [(20, 300), (9, 30)]),
    (64, 128, 2, 6, BF, [(17, 700), (2, 2)]),
    (128, 16, 1, 8, BF, [(6, 61), (5, 5), (16, 3000)]),
    (128, 32, 2, 4, HF, [(70, 500), (3, 64)]),
    (128, 64, 1, 4, BF, [(150, 1200), (90, 90)]),
    (64, 16, 1, 8, BF, [(100, 230), (1, 1)]),
]


def state(case, code, seed):
    D, T, kv, G, dtype, seqs = case
    st = plain.make_state(seqs, G * kv, kv, D, T, code, dtype, seed=seed)
    d = plain.on_gpu(st)
    wq.kv8_append(d["K"], d["V"], d["cache"], d["table"], d["cu"], d["lens"], st["max_new"])

    def attend():
        return wq.attn_kv8(d["Q"], d["cache"], d["table"], d["cu"], d["lens"], st["max_new"])
    return st, d, attend


def seen(st, b, p):
    """First row of sequence b that sees position p (its first row, or beyond its last)."""
    n = int(st["cu"][b + 1] - st["cu"][b])
    return int(st["cu"][b]) + min(n, max(0, p - (int(st["lens"][b]) - n)))


def same(a, b):
    return bool(((a == b) | (a.isnan() & b.isnan())).all())


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("nan", [0x7F, 0xFF])
def test_value_codes_that_are_no_number(case, nan):
    """A NaN code at some positions: the rows that see one are NaN in that element of that
    head's result, everything else keeps its bits."""
    st, d, attend = state(case, E4, seed=3)
    D, T, kv, G, _, seqs = case
    want = attend().cpu()
    clean = want.clone()
    g = torch.Generator().manual_seed(7)
    for b, (n, L) in enumerate(seqs):
        for p in sorted({L - 1, L - (n + 1) // 2, min(L - 1, L - n + 1), L - n // 3 - 1}):
            e, h = int(torch.randint(D, (1,), generator=g)), p % kv
            page = int(st["table"][b, p // T])
            d["cache"][2][page, h, p % T, e] = nan
            want[seen(st, b, p):int(st["cu"][b + 1]), h * G:h * G + G, e] = NAN
    assert bool((~want.isnan()).any(0).any()) and bool(want.isnan().any())
    out = attend().cpu()
    assert same(out, want)
    assert same(out, attend().cpu())
    # one that every row of its sequence sees
    d["cache"][2][int(st["table"][0, 0]), 0, 0, 1] = nan
    if seqs[0][1] > seqs[0][0]:
        want[:int(st["cu"][1]), :G, 1] = NAN
        assert same(attend().cpu(), want)
    assert not clean.isnan().any()


@pytest.mark.parametrize("case", CASES)
def test_key_codes_that_are_no_number(case):
    st, d, attend = state(case, E4, seed=4)
    D, T, kv, G, _, seqs = case
    want = attend().cpu()
    for b, (n, L) in enumerate(seqs):
        p = L - (n + 1) // 2
        d["cache"][0][int(st["table"][b, p // T]), p % kv, p % T, 5] = 0x7F
        want[seen(st, b, p):int(st["cu"][b + 1]), p % kv * G:p % kv * G + G] = NAN
    assert same(attend().cpu(), want)


@pytest.mark.parametrize("code", [I8, E4])
@pytest.mark.parametrize("bad", [NAN, INF])
@pytest.mark.parametrize("which", [1, 3])
@pytest.mark.parametrize("case", [c for c in CASES if any((L - n) // c[1] != (L - 1) // c[1]
                                                         for n, L in c[5])])
def test_scales_that_are_not_finite(case, which, bad, code):
    """The scale of a sequence's last page: rows that end before it keep their bits.  Rows
    that see it are not finite (an infinite key scale makes a score of either sign)."""
    st, d, attend = state(case, code, seed=5)
    D, T, kv, G, _, seqs = case
    want = attend().cpu()
    hit = torch.zeros(want.shape[0], dtype=torch.bool)
    for b, (n, L) in enumerate(seqs):
        if (L - n) // T == (L - 1) // T:
            continue
        d["cache"][which][int(st["table"][b, (L - 1) // T])] = bad
        hit[seen(st, b, (L - 1) // T * T):int(st["cu"][b + 1])] = True
    out = attend().cpu()
    assert torch.equal(out[~hit], want[~hit])
    if which == 3 or bad != bad:
        assert not bool(out[hit].isfinite().any())
