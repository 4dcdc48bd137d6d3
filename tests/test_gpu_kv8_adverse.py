"""Attention calls that go wrong or to extremes, on every kernel and mode: mma.sync (up to 32
rows to a kv head), one tensor-memory tile (33 to 128, fp16), two (more, bf16).  The workspace
holds 0xFF bytes throughout."""
import pytest
import torch

import bit_gemm_group_b200 as wq
import kv8_bounds as bounds
import kv8_plain as plain

pytestmark = pytest.mark.gpu

I8, E4 = torch.int8, torch.uint8
BF, HF = torch.bfloat16, torch.float16
# type, new rows of the longest sequence, query heads per kv head, elements of a head
MODES = [(BF, 3, 4, 64), (HF, 2, 8, 128), (BF, 9, 4, 256), (BF, 12, 4, 128), (HF, 40, 4, 64),
         (BF, 50, 4, 64), (BF, 40, 8, 128)]


@pytest.fixture(autouse=True)
def _clean_status():
    wq.wq_get_device_status(reset=True)
    yield
    assert wq.wq_get_device_status(reset=True) == wq.WQ_OK


def attend(st, d, Q=None, table=None, cu=None, lens=None, rope=None, max_new=None, scale=None):
    Q = d["Q"] if Q is None else Q
    heads, kv, D = Q.shape[1], d["cache"][0].shape[1], Q.shape[2]
    max_new = max_new or st["max_new"]
    cu = d["cu"] if cu is None else cu
    out = torch.full(Q.shape, 7.0, dtype=Q.dtype, device="cuda")
    ws = wq.attn_kv8_workspace(cu.numel() - 1, heads, kv, D, max_new, "cuda").fill_(255)
    wq.wq_attn_kv8(Q, d["cache"], d["table"] if table is None else table, cu,
                   d["lens"] if lens is None else lens, max_new, scale or D ** -0.5, out, ws,
                   rope or d["rope"])
    return out.cpu()


def appended(mode, seqs, code, T, seed, rope=None):
    dtype, n, G, D = mode
    st = plain.make_state(seqs, G * 2, 2, D, T, code, dtype, seed=seed, rope=rope)
    cache = plain.append(st["K"], st["V"], st["cache"], st["table"], st["cu"], st["lens"], rope)
    d = plain.on_gpu(st)
    wq.kv8_append(d["K"], d["V"], d["cache"], d["table"], d["cu"], d["lens"], st["max_new"],
                  d["rope"])
    return st, d, cache


def within(st, cache, out, rows, table=None, scale=None):
    ref, tol = bounds.attention(st["Q"], cache, st["table"] if table is None else table, st["cu"],
                                st["lens"], st["rope"], scale or st["Q"].shape[2] ** -0.5, rows)
    return ((out[:ref.shape[0]].double() - ref).abs() <= tol).all(-1)  # of each row and head


@pytest.mark.parametrize("code", [I8, E4])
@pytest.mark.parametrize("mode", MODES)
def test_maxima_that_grow_late_and_values_far_apart(mode, code):
    """Pages whose keys tower over those before them, values 2^30 apart: results so far are
    rescaled in the middle of a run, and parts of a row are joined far apart."""
    dtype, n, G, D = mode
    seqs = [(n, 1500), (n, n + 40)]
    st = plain.make_state(seqs, G * 2, 2, D, 16, code, dtype, seed=2)
    ks, vs = st["cache"][1], st["cache"][3]
    for b, (_, L) in enumerate(seqs):
        used = st["table"][b, : (L - n) // 16].long()
        ks[used[len(used) // 3]] *= 20
        ks[used[-1]] *= 40
        vs[used[::3]] *= 2.0 ** 6 if dtype == HF else 2.0 ** 30
        vs[used[1::3]] *= 2.0 ** -20
    d = plain.on_gpu(st)
    wq.kv8_append(d["K"], d["V"], d["cache"], d["table"], d["cu"], d["lens"], n)
    cache = plain.append(st["K"], st["V"], st["cache"], st["table"], st["cu"], st["lens"], None)
    out = attend(st, d, scale=0.02)
    assert bool(within(st, cache, out, n * G, scale=0.02).all())


@pytest.mark.parametrize("T", [16, 64, 128])
@pytest.mark.parametrize("mode", MODES)
def test_pages_outside_the_cache_are_left_out(mode, T):
    """A page in the middle, the first one, all pages of a sequence, and rows of no sequence."""
    dtype, n, G, D = mode
    seqs = [(n, n + 4 * T + 3), (n, n + 5 * T), (max(1, n // 2), n + T), (1, 200)]
    st, d, cache = appended(mode, seqs, E4, T, seed=8)
    extra = torch.full((3, G * 2, D), float("nan"), device="cuda", dtype=dtype)
    Q = torch.cat([d["Q"], extra])
    out = attend(st, d, Q=Q)
    assert bool(within(st, cache, out, n * G).all()) and bool((out[-3:] == 7).all())
    bad = st["table"].clone()
    bad[0, 1], bad[1, 0] = cache[0].shape[0], -5
    bad[2] = 10 ** 9
    out = attend(st, d, Q=Q, table=bad.cuda())
    assert wq.wq_get_device_status(reset=True) == wq.WQ_ERR_ARG
    assert bool(within(st, cache, out, n * G, table=bad).all()) and bool((out[-3:] == 7).all())
    rows = slice(int(st["cu"][2]), int(st["cu"][3]))
    assert bool((out[rows] == 0).all())


@pytest.mark.parametrize("what", ["negative", "beyond", "order", "rows", "end", "angles"])
@pytest.mark.parametrize("mode", MODES)
def test_one_sequence_with_wrong_tables(mode, what):
    """The status says so, the other sequences get their results, other rows their bytes."""
    dtype, n, G, D = mode
    rope = (*plain.angles(400, D), False)
    seqs = [(n, 150), (1, 90), (n, n + 20)]
    st, d, cache = appended(mode, seqs, I8, 32, seed=9, rope=rope)
    cu, lens, kw = st["cu"].clone(), st["lens"].clone(), {}
    first = int(cu[1])
    if what == "negative":
        lens[1] = -3
    elif what == "beyond":
        lens[1] = 32 * st["table"].shape[1] + 1
    elif what == "order":    # rows [n, n - 1) and none
        cu = torch.tensor([0, n, n - 1, n - 1], dtype=torch.int32)
    elif what == "rows":     # the second sequence claims more rows than max_new
        cu = torch.tensor([0, n, 2 * n + 1, 2 * n + 1], dtype=torch.int32)
    elif what == "end":      # rows behind the call's last
        cu = torch.tensor([0, n, n + 1, 2 * n + 2], dtype=torch.int32)
    else:                    # the first sequence's rows have no angles
        kw["rope"] = (d["rope"][0][:100].contiguous(), d["rope"][1][:100].contiguous(), False)
    out = attend(st, d, cu=cu.cuda(), lens=lens.cuda(), **kw)
    assert wq.wq_get_device_status(reset=True) == wq.WQ_ERR_ARG
    good = within(st, cache, out, n * G)
    assert bool(out.isfinite().all())
    if what == "angles":
        # not rotated
        ref, tol = bounds.attention(st["Q"][:first], cache, st["table"][:1], st["cu"][:2],
                                    st["lens"][:1], None, D ** -0.5, n * G)
        assert bool(((out[:first].double() - ref).abs() <= tol).all())
        assert bool(good[first:].all())
        return
    assert bool(good[:first].all())
    if what == "negative":
        assert bool((out[first] == 0).all())
    if what in ("negative", "beyond"):
        assert bool(good[first + 1:].all())
    elif what == "end":
        assert bool(good[first].all()) and bool((out[first + 1:] == 7).all())
    else:
        assert bool((out[first:] == 7).all())


@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("mode", MODES)
def test_a_non_finite_query_stays_in_its_row(mode, value):
    dtype, n, G, D = mode
    rope = (*plain.angles(400, D), True)
    st, d, cache = appended(mode, [(n, 333), (1, 50)], E4, 16, seed=10, rope=rope)
    Q = d["Q"].clone()
    hit = [(0, 0), (n - 1, G + 1), (n // 2, 2 * G - 1)]
    for i, h in hit:
        Q[i, h, 3 + 2 * h] = value
    out = attend(st, d, Q=Q)
    others = torch.ones(out.shape[:2], dtype=torch.bool)
    for i, h in hit:
        others[i, h] = False
        assert not bool(out[i, h].isfinite().any())
    assert bool(within(st, cache, out, n * G)[others].all())


@pytest.mark.parametrize("mode", MODES)
def test_queries_of_zeros_and_of_the_smallest_and_largest_numbers(mode):
    """Zero queries weigh all positions alike, tiny ones nearly so; scores near the largest
    number leave a result finite."""
    dtype, n, G, D = mode
    st, d, cache = appended(mode, [(n, 100), (1, 1)], I8, 32, seed=11)
    info = torch.finfo(dtype)
    st["Q"][0] = 0
    st["Q"][n - 1, 0] = info.smallest_normal * st["Q"][n - 1, 0].sign()
    st["Q"][n // 2, 1] = info.max / 1024 * st["Q"][n // 2, 1].sign()
    Q = st["Q"].contiguous().cuda()
    out = attend(st, d, Q=Q)
    others = torch.ones(out.shape[:2], dtype=torch.bool)
    others[n // 2, 1] = False  # (no bound: its scores are off by more than they differ)
    assert bool(within(st, cache, out, n * G)[others].all()) and bool(out.isfinite().all())


@pytest.mark.parametrize("code", [I8, E4])
@pytest.mark.parametrize("mode", MODES)
def test_scores_of_every_size(mode, code):
    """Scores up to 2^110: in the limit a row is the mean value of its largest score.  Queries
    are 1 and -1, keys whole numbers on scale 1, so that scores are whole multiples of one
    number: equal ones are equal in the kernel too, others lie 2^10 apart from a scale of 2^10
    on, where their weights are 0."""
    dtype, n, G, D = mode
    L = 200
    st = plain.make_state([(n, L)], G * 2, 2, D, 16, code, dtype, seed=12)
    g = torch.Generator().manual_seed(6)
    st["Q"][:] = torch.where(torch.rand(st["Q"].shape, generator=g) < 0.9, 1.0, -1.0)
    used = st["table"][0, : -(-L // 16)].long()
    kq, ks, vq, vs = st["cache"]
    ks[used] = vs[used] = 1.0
    base, factor = torch.randint(1, 9, (D,), generator=g), torch.randperm(L, generator=g) % 8
    for p in range(L):
        page = int(st["table"][0, p // 16])
        key = base * (factor[p] if p < L - n else 0)
        kq[page, :, p % 16] = plain.to_codes(key.float(), code)
        if p >= L - n:
            vq[page, :, p % 16] = 0
    vmax = plain.values(vq[used]).double().nan_to_num(0).abs().amax()
    d = plain.on_gpu(st)
    for exponent in (0, 10, 12, 14, 17, 18, 19, 20, 21, 24, 30, 60, 100):
        scale = 2.0 ** exponent
        out = attend(st, d, scale=scale)
        assert bool(out.isfinite().all()), exponent
        if exponent >= 10:
            ref, _ = bounds.attention(st["Q"], st["cache"], st["table"], st["cu"], st["lens"],
                                      None, scale, n * G)
            # 2^-11 for the f16 weights and as much for exponentials and sums; the result's type
            err = (out.double() - ref).abs()
            assert bool((err <= vmax * 2.0 ** -10 + ref.abs() * torch.finfo(dtype).eps / 2).all()), exponent
