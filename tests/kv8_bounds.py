"""64-bit attention over the paged 8-bit cache with a bound for each kernel: how many f16
terms it holds a query in is a part of the bound, so that a term left out shows."""
import torch

from kv8_plain import rotate, values

LN2 = 0.6931471805599453


def terms(dtype, rows, D):
    """f16 terms of a rotated query: one from 33 rows to a kv head on in bf16 (tensor-memory
    kernel, heads of 64 and 128), else two."""
    return 1 if dtype == torch.bfloat16 and rows > 32 and D <= 128 else 2


def rounded_query(q, n_terms):
    """A query (64 bits, last axis one row) as the kernels hold it: relative to a power of two
    that brings the row's largest element to [2^14, 2^15), in n f16 terms."""
    a = q.abs().amax(-1, keepdim=True)
    up = torch.exp2(14 - torch.floor(torch.log2(torch.where(a > 0, a, torch.ones_like(a)))))
    rest, out = q * up, torch.zeros_like(q)
    for _ in range(n_terms):
        t = rest.to(torch.float16).double()
        out, rest = out + t, rest - t
    return out / up


def attention(Q, cache, table, cu, lens, rope, scale, rows, n_terms=None):
    """(result, bound) in 64 bits; `rows` is max_new times the query heads of a kv head.
    Positions on pages outside the cache are left out.  n_terms: a result with queries rounded
    to that many f16 terms, to see what the bound sees.

    Score j is off by d_j at most (natural units):
      2^-11 (one term) or 2^-22 (two) of sum |q| |k|, and 2^-39 of the row's largest element
        where a term is subnormal;
      D fp32 additions, 16 more for scaling and joining, 2^-23 of the magnitudes each, which
        are those of codes + 128 where int8 keys are held with that bias;
      2^-21 of the score, its page's log2 scale and a few units (multiplications by the
        factors, the addition of the two, the subtraction of the maximum).
    So the result moves by e^max(d) sum p_j (|v_j| + |o|) (e^d_j - 1).  Beside that
      a weight is rounded to f16: 2^-11 of p |v|, or half a subnormal step, 2^-31 of the
        row's largest weight times value scale (which is kept at 2^6 and more), times its code;
      sums run over L positions in steps of 16 or less, 2^-23 of the magnitudes each, with 64
        steps more for joins and rescaling; exponentials and quotients 2^-19;
      the result is rounded to its type."""
    kq, ks, vq, vs = cache
    T, G, D = kq.shape[2], Q.shape[1] // kq.shape[1], Q.shape[2]
    one = terms(Q.dtype, rows, D) == 1
    bias = 128.0 if kq.dtype == torch.int8 else 0.0
    out = torch.zeros(Q.shape, dtype=torch.float64)
    tol = torch.zeros(Q.shape, dtype=torch.float64)
    for b in range(len(lens)):
        n, L = int(cu[b + 1] - cu[b]), int(lens[b])
        if n == 0 or L == 0:
            continue
        pages = table[b, : -(-L // T)].long()
        there = ((pages >= 0) & (pages < kq.shape[0])).repeat_interleave(T)[:L]
        pages = torch.where((pages >= 0) & (pages < kq.shape[0]), pages, pages.clamp(min=0)[0] * 0)

        def spread(x):  # [pages, kv, T, ...] of the sequence -> [heads, L, ...]
            return x.transpose(0, 1).flatten(1, 2)[:, :L].repeat_interleave(G, 0)

        clean = lambda x: torch.where(there[None, :, None], x, torch.zeros((), dtype=x.dtype))  # noqa: E731
        kc, vc = clean(spread(values(kq[pages]).double())), clean(spread(values(vq[pages]).double()))
        fk, fv = (spread(s[pages].double()[..., None, None].expand(-1, -1, T, 1)) for s in (ks, vs))
        fk, fv = clean(fk), torch.where(there[None, :, None], fv, torch.ones((), dtype=fv.dtype))
        k, v = kc * fk, vc * fv
        pos = torch.arange(L - n, L)
        q = rotate(Q[cu[b]:cu[b + 1]].float(), pos.clamp(min=0), rope).double().transpose(0, 1)
        held = q if n_terms is None else rounded_query(q, n_terms)
        hide = (torch.arange(L)[None, :] > pos[:, None]) | ~there[None, :]
        s = (held @ k.transpose(1, 2) * scale).masked_fill(hide, -torch.inf)
        size = q.abs() @ k.abs().transpose(1, 2)
        held_size = q.abs() @ (k.abs() + bias * fk).transpose(1, 2)
        d = size * (2.0 ** -11 if one else 2.0 ** -22) + held_size * (D + 16) * 2.0 ** -23
        d = d + 2.0 ** -39 * q.abs().amax(-1, keepdim=True) * k.abs().sum(-1)[:, None]
        lv = fv.clamp(min=1e-30).log2().abs()[:, None, :, 0]
        d = d * scale + (s.masked_fill(hide, 0).abs() + lv * LN2 + 16) * 2.0 ** -21
        d = d.masked_fill(hide, 0)
        p = torch.softmax(s, -1)
        p = torch.where(hide.all(-1)[:, None], torch.zeros((), dtype=p.dtype), p)
        o, mag = p @ v, p @ v.abs()
        e = p * torch.expm1(d)
        bound = (e @ v.abs() + o.abs() * e.sum(-1, keepdim=True)) * d.amax(-1, keepdim=True).exp()
        bound = bound + mag * 2.0 ** -11 + (mag + o.abs()) * ((L / 16 + 64) * 2.0 ** -23 + 2.0 ** -19)
        top = (p * fv[..., 0][:, None]).amax(-1, keepdim=True)
        bound = bound + 2.0 ** -31 * top * vc.abs().sum(1)[:, None]
        bound = bound + o.abs() * torch.finfo(Q.dtype).eps / 2
        out[cu[b]:cu[b + 1]] = o.transpose(0, 1)
        tol[cu[b]:cu[b + 1]] = bound.transpose(0, 1)
    return out, tol + 1e-30 + (2.0 ** -25 if Q.dtype == torch.float16 else 0)


def split_state(plain, n, G, kv, D, T, code, dtype, seed, past):
    """A state whose results hang on the second f16 term of a query.  Rotation multiplies the
    first half of a head's elements, all 1, by 1 + 0.99 2^-11, which one f16 term rounds to 1,
    and keeps the others.  Even positions have keys in the first half alone, odd ones in the
    other, so that their scores, 300 each, are 0.14 apart with the term and equal without;
    their values are 1 and -1."""
    st = plain.make_state([(n, past + n)], G * kv, kv, D, T, code, dtype, seed=seed)
    L, half = past + n, D // 4  # pairs (i, i + D / 2): the first D / 4 pairs turn
    cos = torch.ones(L, D // 2)
    cos[:, :half] = 1 + 0.99 * 2.0 ** -11
    st["rope"] = (cos, torch.zeros(L, D // 2), False)
    turned = torch.zeros(D, dtype=torch.bool)
    turned[:half] = turned[D // 2:D // 2 + half] = True
    st["Q"][:] = 1
    even = torch.arange(L) % 2 == 0
    key = torch.where(even[:, None] == turned[None, :], 1.0, 0.0)  # [L, D]
    val = torch.where(even, 1.0, -1.0)[:, None].expand(L, D)
    for q, s, x in ((st["cache"][0], st["cache"][1], key), (st["cache"][2], st["cache"][3], val)):
        for p in range(L):
            page = int(st["table"][0, p // T])
            q[page, :, p % T] = plain.to_codes(x[p] * plain.TOP[code], code)
            s[page] = 1 / plain.TOP[code]
    return st, 300.0 / (D // 2)
