"""The paged 8-bit KV cache on the GPU: appended codes and scales bit-exact against the
plain implementation, attention within the bound of its own roundings, and the two of
them run as a model runs them."""
import pytest
import torch

import bit_gemm_group_b200 as wq
import kv8_plain as plain

pytestmark = pytest.mark.gpu

I8, E4 = torch.int8, torch.uint8
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(autouse=True)
def _clean_status():
    wq.wq_get_device_status(reset=True)
    yield
    assert wq.wq_get_device_status(reset=True) == wq.WQ_OK


def run_append(st):
    d = plain.on_gpu(st)
    wq.kv8_append(d["K"], d["V"], d["cache"], d["table"], d["cu"], d["lens"], st["max_new"],
                  d["rope"])
    return d


def same_bytes(a, b):
    return torch.equal(a.cpu().view(torch.uint8), b.view(torch.uint8))


def check_cache(d, want):
    for got, exp, what in zip(d["cache"], want, ("kq", "ks", "vq", "vs")):
        assert same_bytes(got, exp), what


def check_attention(st, d, cache, **kw):
    out = wq.attn_kv8(d["Q"], d["cache"], d["table"], d["cu"], d["lens"], st["max_new"],
                      rope=d["rope"], **kw)
    scale = kw.get("scale") or st["Q"].shape[2] ** -0.5
    ref, tol = plain.attention(st["Q"], cache, st["table"], st["cu"], st["lens"], st["rope"], scale)
    n = int(st["cu"][-1])
    err = (out[:n].cpu().double() - ref[:n]).abs()
    assert bool((err <= tol[:n]).all()), float((err / tol[:n]).max())
    return out


# (new, length with the new ones) of each sequence
DECODE = [(1, 1), (1, 16), (1, 17), (1, 64), (1, 65), (1, 200)]
MIXED = [(3, 3), (0, 40), (5, 130), (70, 70), (1, 129), (33, 100)]


@pytest.mark.parametrize("code", [I8, E4])
@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("D,T,kv,rot,inter", [
    (64, 16, 1, 64, False), (64, 128, 3, 32, True), (128, 64, 8, 128, False),
    (128, 32, 2, 64, False), (128, 16, 2, 128, True), (256, 128, 2, 256, False),
    (256, 16, 1, 16, False), (128, 64, 2, 0, False)])
@pytest.mark.parametrize("seqs", [DECODE, MIXED])
def test_append_bitexact(code, dtype, D, T, kv, rot, inter, seqs):
    rope = (*plain.angles(256, rot), inter) if rot else None
    st = plain.make_state(seqs, 2 * kv, kv, D, T, code, dtype, seed=D + T, rope=rope)
    check_cache(run_append(st), plain.append(st["K"], st["V"], st["cache"], st["table"], st["cu"],
                                             st["lens"], rope))


@pytest.mark.parametrize("code", [I8, E4])
def test_append_grows_and_keeps_scales(code):
    """Small rows after large ones keep the page's scale; large after small recode it."""
    st = plain.make_state([(2, 34), (2, 34)], 2, 2, 128, 64, code, BF, seed=1)
    st["K"][:2] *= 100
    st["V"][2:] *= 1e-3
    want = plain.append(st["K"], st["V"], st["cache"], st["table"], st["cu"], st["lens"], None)
    pages = st["table"][:, 0].long()
    assert bool((want[1][pages[0]] > st["cache"][1][pages[0]]).all())
    assert bool((want[3][pages[1]] == st["cache"][3][pages[1]]).all())
    check_cache(run_append(st), want)


@pytest.mark.parametrize("code", [I8, E4])
def test_append_token_by_token_equals_the_definition_applied_in_turn(code):
    T, D, kv = 16, 64, 2
    rope = (*plain.angles(64, D), False)
    cache = [t for t in wq.kv8_cache(4, kv, T, D, code, "cpu")]
    dev = tuple(t.cuda() for t in cache)
    table = torch.tensor([[2, 0, 3]], dtype=torch.int32)
    g = torch.Generator().manual_seed(3)
    cos, sin = rope[0].cuda(), rope[1].cuda()
    for p in range(40):
        K, V = torch.randn(1, kv, D, generator=g) * (1 + p % 7), torch.randn(1, kv, D, generator=g)
        cu, lens = torch.tensor([0, 1], dtype=torch.int32), torch.tensor([p + 1], dtype=torch.int32)
        cache = plain.append(K, V, cache, table, cu, lens, rope)
        wq.kv8_append(K.cuda(), V.cuda(), dev, table.cuda(), cu.cuda(), lens.cuda(), 1,
                      (cos, sin, False))
    for got, exp in zip(dev, cache):
        assert same_bytes(got, exp)


def test_append_non_finite_rows_do_not_cost_the_page():
    st = plain.make_state([(2, 20)], 2, 2, 64, 32, I8, BF, seed=5)
    st["K"][0, 0, 3], st["K"][0, 0, 4] = float("inf"), float("nan")
    st["V"][1, 1, 0] = float("-inf")
    d = run_append(st)
    assert wq.wq_get_device_status(reset=True) == wq.WQ_ERR_NONFINITE
    check_cache(d, plain.append(st["K"], st["V"], st["cache"], st["table"], st["cu"], st["lens"],
                                None))


@pytest.mark.parametrize("what", ["page", "column", "lens", "cu", "angles", "max_new"])
def test_append_reports_bad_tables_and_writes_nothing_wrong(what):
    """One sequence is wrong: it is skipped, the other one is written."""
    rope = (*plain.angles(100, 64), False)
    st = plain.make_state([(2, 50), (2, 60)], 2, 2, 64, 32, I8, BF, seed=6, rope=rope)
    if what == "page":
        st["table"][1, 1] = 10 ** 6
    elif what == "column":
        st["lens"][1] = 32 * st["table"].shape[1] + 1
        st["rope"] = rope = None
    elif what == "lens":
        st["lens"][1] = 1
    elif what == "cu":
        st["cu"] = torch.tensor([0, 2, 9], dtype=torch.int32)
    elif what == "angles":
        st["rope"] = rope = (rope[0][:55], rope[1][:55], False)
    else:
        st["max_new"] = 1
    first = 0 if what == "max_new" else 1  # with max_new 1 both sequences have too many rows
    want = plain.append(st["K"], st["V"], st["cache"], st["table"][:first], st["cu"][:first + 1],
                        st["lens"][:first], rope)
    d = run_append(st)
    assert wq.wq_get_device_status(reset=True) == wq.WQ_ERR_ARG
    check_cache(d, want)


@pytest.mark.parametrize("code", [I8, E4])
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("D,T,kv,G", [
    (64, 16, 2, 1), (64, 128, 1, 12), (128, 16, 2, 8), (128, 32, 3, 3), (128, 64, 8, 8),
    (128, 128, 1, 16), (256, 16, 1, 8), (256, 64, 2, 2)])
@pytest.mark.parametrize("seqs", [DECODE, MIXED, [(1, 0), (4, 2), (2, 31)]])
def test_attention(code, dtype, D, T, kv, G, seqs):
    rope = (*plain.angles(256, D // 2 if T == 32 else D), T == 128)
    st = plain.make_state([(n, max(L, 1) if n and L else L) for n, L in seqs], G * kv, kv, D, T,
                          code, dtype, seed=D + T + G, rope=rope)
    # every position is written before the attention reads it; rows before a
    # sequence's start (more rows than positions) are not appended
    if all(L >= n for n, L in seqs):
        d = run_append(st)
        cache = plain.append(st["K"], st["V"], st["cache"], st["table"], st["cu"], st["lens"], rope)
    else:
        full = plain.make_state([(0, L) for _, L in seqs], G * kv, kv, D, T, code, dtype, seed=1)
        st["cache"], st["table"] = full["cache"], full["table"]
        d, cache = plain.on_gpu(st), st["cache"]
    check_attention(st, d, cache)


@pytest.mark.parametrize("code,D,T,kv,G,seqs", [
    (I8, 128, 64, 2, 8, [(1, 9000)]), (E4, 128, 16, 1, 4, [(1, 5001), (1, 3)]),
    (E4, 64, 32, 2, 16, [(5, 4100), (2, 77)]), (I8, 256, 128, 1, 6, [(3, 3000)]),
    (E4, 128, 64, 8, 2, [(1, 700 + 13 * i) for i in range(40)]),
    (I8, 128, 32, 1, 8, [(300, 300), (150, 1000), (1, 40)])])
def test_attention_over_longer_contexts(code, D, T, kv, G, seqs):
    """Runs that are cut between workers, and rows of several blocks."""
    rope = (*plain.angles(10000, D), False)
    st = plain.make_state(seqs, G * kv, kv, D, T, code, BF, seed=D + T, rope=rope)
    d = run_append(st)
    cache = plain.append(st["K"], st["V"], st["cache"], st["table"], st["cu"], st["lens"], rope)
    out = check_attention(st, d, cache)
    again = wq.attn_kv8(d["Q"], d["cache"], d["table"], d["cu"], d["lens"], st["max_new"],
                        rope=d["rope"])
    assert torch.equal(out, again)


@pytest.mark.parametrize("code", [I8, E4])
def test_attention_with_pages_of_very_different_scale(code):
    """Key scales that put one page far above the rest late in the sequence (the maximum
    grows in the middle of a run), value scales 2^30 apart."""
    st = plain.make_state([(1, 400)], 4, 1, 128, 16, code, BF, seed=2)
    kq, ks, vq, vs = st["cache"]
    used = st["table"][0, :25].long()
    ks[used[12]] *= 20
    ks[used[20]] *= 60
    vs[used[::3]] *= 2.0 ** 30
    d = run_append(st)
    cache = plain.append(st["K"], st["V"], st["cache"], st["table"], st["cu"], st["lens"], None)
    check_attention(st, d, cache, scale=0.02)


def test_attention_leaves_other_rows_and_reports_bad_tables():
    st = plain.make_state([(2, 90), (3, 64)], 4, 2, 64, 32, I8, BF, seed=8)
    d = run_append(st)
    cache = plain.append(st["K"], st["V"], st["cache"], st["table"], st["cu"], st["lens"], None)
    ref, tol = plain.attention(st["Q"], cache, st["table"], st["cu"], st["lens"], None, 0.125)
    Q = torch.cat([d["Q"], torch.full((3, 4, 64), float("nan"), device="cuda", dtype=BF)])
    out = torch.full_like(Q, 7.0)
    ws = wq.attn_kv8_workspace(2, 4, 2, 64, 3, "cuda").fill_(255)
    wq.wq_attn_kv8(Q, d["cache"], d["table"], d["cu"], d["lens"], 3, 0.125, out, ws)
    assert bool(((out[:5].cpu().double() - ref).abs() <= tol).all())
    assert bool((out[5:] == 7.0).all())
    # a page outside the cache: its positions are left out
    bad = d["table"].clone()
    bad[0, 1] = 99
    wq.wq_attn_kv8(Q, d["cache"], bad, d["cu"], d["lens"], 3, 0.125, out, ws)
    assert wq.wq_get_device_status(reset=True) == wq.WQ_ERR_ARG
    assert bool(((out[2:5].cpu().double() - ref[2:]).abs() <= tol[2:]).all())
    assert bool(torch.isfinite(out[:2].float()).all())


def test_attention_non_finite_query_stays_in_its_row():
    st = plain.make_state([(2, 50)], 4, 2, 128, 16, E4, BF, seed=9)
    d = run_append(st)
    args = (d["cache"], d["table"], d["cu"], d["lens"], 2)
    clean = wq.attn_kv8(d["Q"], *args)
    Q = d["Q"].clone()
    Q[1, 2, 5] = float("nan")
    out = wq.attn_kv8(Q, *args)
    mask = torch.ones(2, 4, dtype=torch.bool)
    mask[1, 2] = False
    assert torch.equal(out.cpu()[mask], clean.cpu()[mask])
    assert bool(out[1, 2].isnan().all())


def test_captured_step_replayed_as_the_sequences_grow():
    """A decode step (projection, append, attention, projection) captured once and
    replayed with new tokens and lengths: the run that a model makes of the operators."""
    B, heads, kv, D, T, H = 3, 8, 2, 64, 16, 512
    rope = (*plain.angles(128, D), False)
    st = plain.make_state([(1, 15), (1, 31), (1, 47)], heads, kv, D, T, E4, BF, seed=11,
                          extra_cols=2, rope=rope)
    # each sequence gets pages for the positions to come
    kq = st["cache"][0]
    P = kq.shape[0]
    more = [torch.cat([t, torch.zeros((9, *t.shape[1:])).to(t.dtype)]) for t in st["cache"]]
    st["cache"] = tuple(more)
    spare = iter(range(P, P + 9))
    for b in range(B):
        for j in range(st["table"].shape[1]):
            if st["table"][b, j] < 0 and j <= (int(st["lens"][b]) + 20) // T:
                st["table"][b, j] = next(spare)
    d = plain.on_gpu(st)
    g = torch.Generator().manual_seed(4)
    width = (heads + 2 * kv) * D
    wqkv = (torch.randn(width, H, generator=g) * H ** -0.5).to(BF).cuda()
    wo = (torch.randn(H, heads * D, generator=g) * (heads * D) ** -0.5).to(BF).cuda()
    (q1, s1), (q2, s2) = wq.quantize_fp8_block(wqkv), wq.quantize_fp8_block(wo)
    x = torch.zeros(B, H, dtype=BF, device="cuda")
    ws = wq.attn_kv8_workspace(B, heads, kv, D, 1, "cuda")
    qkv = torch.empty(B, width, dtype=BF, device="cuda")
    out = torch.empty(B, heads, D, dtype=BF, device="cuda")
    y = torch.empty(B, H, dtype=BF, device="cuda")
    w1 = torch.empty(wq.wq_fp8_block_workspace_bytes(B, width, H), dtype=torch.uint8, device="cuda")
    w2 = torch.empty(wq.wq_fp8_block_workspace_bytes(B, H, heads * D), dtype=torch.uint8,
                     device="cuda")

    def step():
        wq.wq_gemm_fp8_block(x, q1, s1, qkv, w1)
        r = qkv.view(B, heads + 2 * kv, D)
        q, k, v = r[:, :heads], r[:, heads:heads + kv], r[:, heads + kv:]
        wq.wq_kv8_append(k, v, d["cache"], d["table"], d["cu"], d["lens"], 1, d["rope"])
        wq.wq_attn_kv8(q, d["cache"], d["table"], d["cu"], d["lens"], 1, D ** -0.5, out, ws,
                       d["rope"])
        wq.wq_gemm_fp8_block(out.view(B, heads * D), q2, s2, y, w2)

    kept = tuple(t.clone() for t in d["cache"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t, k in zip(d["cache"], kept):
        t.copy_(k)
    cache, lens = st["cache"], st["lens"].clone()
    for i in range(20):
        x.copy_(torch.randn(B, H, generator=g).to(BF))
        d["lens"].copy_(lens)
        graph.replay()
        torch.cuda.synchronize()
        r = qkv.view(B, heads + 2 * kv, D).cpu()
        cache = plain.append(r[:, heads:heads + kv], r[:, heads + kv:], cache, st["table"],
                             st["cu"], lens, rope)
        check_cache(d, cache)
        ref, tol = plain.attention(r[:, :heads], cache, st["table"], st["cu"], lens, rope, D ** -0.5)
        assert bool(((out.cpu().double() - ref).abs() <= tol).all())
        assert torch.equal(y, wq.gemm_fp8_block(out.view(B, heads * D), q2, s2))
        lens = lens + 1


@pytest.mark.parametrize("n", [1, 9])
def test_many_sequences(n):
    # more sequences than a CTA looks at in one go, most of them without rows; with 9 rows of 8
    # heads each on the kernel for many rows
    G = 8
    seqs = [(n, 20 + b % 50) if b % 7 == 0 else (0, 5) for b in range(1500)]
    seqs[-1] = (n, 40)
    st = plain.make_state(seqs, G, 1, 64, 16, I8, BF, seed=11)
    cache = plain.append(st["K"], st["V"], st["cache"], st["table"], st["cu"], st["lens"], None)
    d = run_append(st)
    check_cache(d, cache)
    check_attention(st, d, cache)


@pytest.mark.parametrize("n", [1, 40])
def test_pages_beyond_32_bit_offsets(n):
    # 4.5 GB of codes each for keys and values; the pages in use are the last ones
    D, T, kv, G = 128, 128, 2, 4
    st = plain.make_state([(n, 300), (n, 129)], kv * G, kv, D, T, E4, BF, seed=12)
    used = st["cache"][0].shape[0]
    pages = (9 << 29) // (kv * T * D)
    assert (pages - used) * kv * T * D > 1 << 32
    small = st["cache"]
    big = tuple(torch.empty((pages,) + t.shape[1:], dtype=t.dtype, device="cuda") for t in small)
    for b, t in zip(big, small):
        b[-used:] = t.cuda()
    want = plain.append(st["K"], st["V"], small, st["table"], st["cu"], st["lens"], None)
    d = plain.on_gpu(st)
    d["cache"] = big
    d["table"] = torch.where(d["table"] >= 0, d["table"] + (pages - used), d["table"])
    wq.kv8_append(d["K"], d["V"], big, d["table"], d["cu"], d["lens"], n, None)
    for b, w in zip(big, want):
        assert same_bytes(b[-used:].contiguous(), w)
    check_attention(st, d, want)


@pytest.mark.parametrize("n", [1, 20])
def test_two_calls_at_once_on_streams_of_their_own(n):
    states = [plain.make_state([(n, 700 + 90 * i), (n, 65)], 8, 2, 128, 64, I8, BF, seed=13 + i)
              for i in range(2)]
    wants, ds = [], []
    for st in states:
        wants.append(plain.append(st["K"], st["V"], st["cache"], st["table"], st["cu"], st["lens"],
                                  None))
        ds.append(plain.on_gpu(st))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[], []]
    for _ in range(8):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                d = ds[i]
                wq.kv8_append(d["K"], d["V"], d["cache"], d["table"], d["cu"], d["lens"], n)
                outs[i].append(wq.attn_kv8(d["Q"], d["cache"], d["table"], d["cu"], d["lens"], n))
    torch.cuda.synchronize()
    for i in range(2):
        check_cache(ds[i], wants[i])
        first = check_attention(states[i], ds[i], wants[i])
        for o in outs[i]:
            assert torch.equal(o, first)


def test_sequences_that_share_a_prefix_read_the_same_pages():
    # two sequences whose first pages are the same, each with a last page of its own
    st = plain.make_state([(4, 196), (4, 196)], 4, 2, 64, 64, I8, BF, seed=15)
    st["table"][1, :3] = st["table"][0, :3]
    want = plain.append(st["K"], st["V"], st["cache"], st["table"], st["cu"], st["lens"], None)
    d = run_append(st)
    check_cache(d, want)
    check_attention(st, d, want)


def test_more_new_rows_than_positions_see_nothing_before_the_start():
    # 6 rows of a sequence of 2 positions: the first four lie before its start
    st = plain.make_state([(2, 2)], 4, 2, 64, 16, I8, BF, seed=16)
    d = run_append(st)
    Q = torch.randn(6, 4, 64, device="cuda", dtype=BF)
    cu = torch.tensor([0, 6], dtype=torch.int32, device="cuda")
    out = wq.attn_kv8(Q, d["cache"], d["table"], cu, d["lens"], 6)
    assert bool((out[:4] == 0).all()) and bool((out[4:] != 0).any(-1).all())
