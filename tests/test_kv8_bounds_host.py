"""What the attention tests' bound sees, on the CPU: a query in too few f16 terms."""
import pytest
import torch

import kv8_bounds as bounds
import kv8_plain as plain


def args(st, scale, rows):
    return (st["Q"], st["cache"], st["table"], st["cu"], st["lens"], st["rope"], scale, rows)


@pytest.mark.parametrize("code", [torch.int8, torch.uint8])
@pytest.mark.parametrize("dtype,n,G,D", [
    (torch.float16, 2, 4, 64), (torch.float16, 12, 4, 128), (torch.bfloat16, 4, 8, 128),
    (torch.float16, 9, 4, 256)])
def test_the_bound_sees_a_query_of_one_term(code, dtype, n, G, D):
    st, scale = bounds.split_state(plain, n, G, 1, D, 32, code, dtype, seed=1, past=70)
    exact, tol = bounds.attention(*args(st, scale, n * G))
    for n_terms, fits in ((2, True), (1, False)):
        held, _ = bounds.attention(*args(st, scale, n * G), n_terms=n_terms)
        assert bool(((held - exact).abs() <= tol).all()) == fits
    held, _ = bounds.attention(*args(st, scale, n * G), n_terms=1)
    assert bool(((held - exact).abs() > tol).all())


def test_it_allows_one_term_where_the_kernel_has_one():
    st, scale = bounds.split_state(plain, 40, 2, 1, 128, 32, torch.int8, torch.bfloat16, seed=1, past=70)
    exact, tol = bounds.attention(*args(st, scale, 80))
    held, _ = bounds.attention(*args(st, scale, 80), n_terms=1)
    assert bool(((held - exact).abs() <= tol).all())


@pytest.mark.parametrize("code", [torch.int8, torch.uint8])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_the_two_oracles_agree_and_the_bound_is_narrower(code, dtype):
    rope = (*plain.angles(256, 64), False)
    st = plain.make_state([(3, 100), (1, 17), (5, 5), (0, 9)], 8, 2, 64, 16, code, dtype, seed=3,
                          rope=rope)
    cache = plain.append(st["K"], st["V"], st["cache"], st["table"], st["cu"], st["lens"], rope)
    a = (st["Q"], cache, st["table"], st["cu"], st["lens"], rope, 0.125)
    o1, t1 = plain.attention(*a)
    o2, t2 = bounds.attention(*a, 20)
    assert float((o1 - o2).abs().max()) < 1e-12
    assert float((t2 / t1).median()) < 0.5
