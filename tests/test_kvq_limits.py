"""The limits that fp32 calls over the 8-bit cache are tested by, on the CPU: outputs of queries or weights
with 22 bits are inside, of 15 bits outside."""
import pytest
import torch

import kvq_reference as ref
import kvq_weights as kw


def cut(x, bits):
    """x rounded to so many bits."""
    m, e = torch.frexp(x.double())
    return torch.ldexp(torch.round(m * 2.0 ** bits) * 2.0 ** -bits, e)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("what,size", [("query", 16.0), ("weight", 0.5)])
def test_limits_of_f32(fmt, what, size):
    d, H, lens = 32, 16, [2, 3, 5, 3]
    cu = list(range(len(lens) + 1))
    c, t = ref.filled(lens, 16, 1, d, fmt, 3)
    g = torch.Generator().manual_seed(3)
    q = torch.zeros(len(lens), H, d)
    q.scatter_(2, torch.randint(0, d, (len(lens), H, 1), generator=g),
               size * 0.5 * (0.5 + 0.5 * torch.rand(len(lens), H, 1, generator=g)))
    w = ref.attention(c, q, t, lens, cu, 1.0, 0)
    lim = kw.exact_limits(w, kw.floors(c, q, t, lens, cu, 1.0), max(lens))

    def inside(bits):
        if what == "query":
            o = ref.attention(c, cut(q, bits), t, lens, cu, 1.0, 0)[0]
        else:
            o = torch.empty_like(w[0])
            for r, n in enumerate(lens):
                K, V = (torch.stack([ref.code_values(x, fmt) * float(c.scales[t[r, 0], 0, 0, i]) for x in rows])
                        for i, rows in ((0, c.k[t[r, 0], 0, :n]), (1, c.v[t[r, 0], 0, 0, :, :n].T)))
                x = q[r].double() @ K.T
                p = torch.exp(x - x.amax(-1, keepdim=True))
                o[r] = cut(p, bits) @ V / p.sum(-1, keepdim=True)
        return bool(((o - w[0]).abs() <= lim).all())

    assert inside(22) and not inside(15)
