"""What the 8-bit cache's attention may be off by where weights, value scales and scores are far apart:
limits per row from its own weights, beside those of kvq_reference."""
import numpy as np
import torch

import kvq_reference as ref


def floors(c, q, table, lens, cu, scale, window=0):
    """Of every row (tokens seen) x (largest code) x (largest weight times value scale), and x (largest value
    scale): what 2^-30 and 2^-120 of the header count from.  Weights sum to 1."""
    nq, Hq, _ = q.shape
    G = Hq // c.H
    out, rare = torch.zeros(nq, Hq, dtype=torch.float64), torch.zeros(nq, Hq, dtype=torch.float64)
    for r, n in enumerate(lens):
        m = cu[r + 1] - cu[r]
        pos = torch.arange(n)
        pg, pl = torch.from_numpy(table[r].astype(np.int64))[pos // c.P], pos % c.P
        own = n - m + torch.arange(m)[:, None]
        seen = (pos <= own) & ((pos > own - window) if window else True)
        for h in range(Hq):
            K = ref.code_values(c.k[pg, h // G, pl], c.fmt) * c.scales[pg, h // G, pl // 16, 0].double()[:, None]
            x = torch.where(seen, q[cu[r]:cu[r + 1], h].double() @ K.T * scale, -torch.inf)
            p = torch.where(seen, torch.softmax(torch.where(seen.any(-1, keepdim=True), x, 0.0), -1), 0.0)
            s = ref.TOP[c.fmt] * c.scales[pg, h // G, pl // 16, 1].double().clamp(min=2.0 ** -100)
            out[cu[r]:cu[r + 1], h] = (p * s).amax(-1) * seen.sum(-1)
            rare[cu[r]:cu[r + 1], h] = (seen * s).amax(-1) * seen.sum(-1)
    return out, rare


def limits(w, floor, dtype):
    """As kvq_reference.limits, but what a token is off by far below the largest weight is 2^-30 of its own
    row's largest weight times value scale (float16's last place under 32 times that is 2^-24, half of it is
    lost: 2^-25 / 32), and weights under 2^-120 of the row's largest may count as zero."""
    o, lse, mag, size, _ = w
    near = 2.0 ** -20 * (1 + size) + 2.0 ** -14
    half = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}[dtype]
    p = {"bf16": 2.0 ** -11, "f32": 2.0 ** -21}[dtype]
    return ((near + p)[..., None] * mag + half * o.abs() + (2.0 ** -30 * floor[0] + 2.0 ** -120 * floor[1])[..., None],
            near + 2.0 ** -22 * torch.where(lse.isinf(), 0.0, lse.abs()))


def exact_limits(w, floor, count):
    """fp32 outputs of queries with a single value that is not zero.  A score is then one product: its query has
    22 bits (2^-22), its two parts are added once (2^-23), the factors of the scales round four times (4 x 2^-24),
    together under 2^-20.6; so is the maximum's, and the difference of both is off by under 2^-19 of the scores.  An
    exponential adds 2^-22, the weight's two float16 2^-22 and its products 2^-23; sums round once a token and
    part, the output's factors three times."""
    o, _, mag, size, _ = w
    p = 2.0 ** -19 * size + 2.0 ** -21 + 2.0 ** -23 + (2 * count + 3) * 2.0 ** -23
    return p[..., None] * mag + 2.0 ** -24 * o.abs() + (2.0 ** -30 * floor[0] + 2.0 ** -120 * floor[1])[..., None]
