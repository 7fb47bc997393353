"""sq_decode_step_linear on the GPU: S' = alpha S + beta k v^T, o = S'^T q over
every storage width, against the formula in 64 bits on the stored values.

Tolerances as for the other steps: a code differs by at most one and in at most
1e-4 of the elements (a rounding boundary), pivots and bfloat16 states by 1e-3
relative, o by 1e-3 of its head's largest value plus 1e-5."""
import ctypes

import numpy as np
import pytest
import torch

from quantized_recurrent_state_gated_amd import inputs as I

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sq():
    from quantized_recurrent_state_gated_amd import sq as m
    return m


def setup(sq, orc, w, n_slots, slots):
    bits, (r, c) = I.head_bits(w), I.scales(w)
    off, slab = orc.pool_layout(bits, w.dk, w.dv)
    host = np.zeros(n_slots * slab, np.uint8)
    S0 = torch.stack([I.initial_state(w, p) for p in range(w.n_req)]).numpy()
    orc.store_pool(host, bits, w.dk, w.dv, r.numpy(), c.numpy(), slots, S0)
    dev = torch.from_numpy(host).cuda()
    keep = r.cuda(), c.cuda()
    pool = sq.sq_pool_alloc(n_slots, w.n_heads, w.dk, w.dv, bits, *keep, dev)
    return bits, r.numpy(), c.numpy(), off, slab, host, dev, pool


def check(sq, orc, w, n_slots, slots, steps=2, want_o=True):
    slots = np.array(slots, np.int32)
    bits, r, c, off, slab, pre, dev, pool = setup(sq, orc, w, n_slots, slots)
    ids = torch.from_numpy(slots).cuda()
    wrong = total = 0
    for t in range(steps):
        si = I.step_inputs(w, t)
        o = torch.full((w.n_req, w.n_heads, w.dv), float("nan"), device="cuda") if want_o else None
        sq.sq_decode_step_linear(pool, ids, si.q.cuda(), si.k.cuda(), si.v.cuda(), si.alpha.cuda(), si.beta.cuda(), o)
        torch.cuda.synchronize()
        post = dev.cpu().numpy()
        q, k, v, al, be = (x.double().numpy() for x in (si.q, si.k, si.v, si.alpha, si.beta))
        touched = np.zeros(len(pre), bool)
        for n, p in enumerate(slots):
            for h in range(w.n_heads):
                b, lo = int(bits[h]), int(p) * slab + int(off[h])
                tb = orc.tile_bytes(b, w.dk, w.dv)
                touched[lo:lo + tb] = True
                S = orc.decode_tile(b, w.dk, w.dv, pre[lo:lo + tb], r[h], c[h]).astype(np.float64)
                G = orc.decode_tile(b, w.dk, w.dv, post[lo:lo + tb], r[h], c[h]).astype(np.float64)
                S = al[n, h] * S + be[n, h] * np.outer(k[n, h], v[n, h])
                if b <= 8:
                    s = (r[h].astype(np.float32)[:, None] * c[h].astype(np.float32)[None]).astype(np.float64)
                    Q = 2 ** (b - 1) - 1
                    d = np.abs(np.round(G / s) - np.clip(np.rint(S / s), -Q, Q))
                    assert d.max() <= 1
                    wrong += int((d > 0).sum())
                    total += d.size
                else:
                    lim = (1e-6 if b == 32 else 1e-3 if b == 16 else 2.0 ** -8) * np.abs(S) + 2.0 ** -20 * np.abs(S).max()
                    assert (np.abs(G - S) <= lim).all(), b
                if want_o:
                    wo = S.T @ q[n, h]
                    err = np.abs(o[n, h].cpu().numpy() - wo)
                    assert (err <= 1e-5 + 1e-3 * np.abs(wo).max()).all()
        assert np.array_equal(pre[~touched], post[~touched])
        pre = post
    assert total == 0 or wrong <= max(1, 1e-4 * total)


MIX = {4: 2, 6: 2, 8: 2, 16: 2, 32: 2, I.BITS_BF16: 2}


@pytest.mark.parametrize("qkv", ["f32", "bf16"])
def test_every_width_d128(sq, orc, qkv):
    check(sq, orc, I.Workload("lmix", 3, 12, 128, 128, 2, MIX, qkv_dtype=qkv, seed=31), 5, [4, 1, 2])


@pytest.mark.parametrize("dk,dv", [(4, 4), (12, 20), (64, 128), (256, 32)])
def test_other_shapes(sq, orc, dk, dv):
    # the outlier recipe needs more than its four outlier rows and columns
    w = I.Workload("lshape", 2, 6, dk, dv, 2, {b: 1 for b in MIX}, seed=dk + dv, tiny_recipe=dk == 4)
    check(sq, orc, w, 3, [2, 0])


@pytest.mark.parametrize("n_req,heads", [(4, 300), (167, 100)])
def test_larger_launches(sq, orc, n_req, heads):
    """The 256-thread launch and the two-tiles-per-workgroup launch."""
    k = heads // 12
    counts = {b: 2 * k for b in MIX}
    counts[4] += heads - 12 * k
    w = I.Workload(f"lbig{n_req}", n_req, heads, 128, 128, 1, counts, seed=n_req)
    slots = list(range(n_req + 1))[::-1][:n_req]
    check(sq, orc, w, n_req + 1, slots, steps=1)


def test_without_readout_and_without_requests(sq, orc):
    w = I.Workload("lno", 2, 12, 128, 128, 1, MIX, seed=5)
    check(sq, orc, w, 2, [1, 0], steps=1, want_o=False)
    slots = np.array([0, 1], np.int32)
    _, _, _, _, _, pre, dev, pool = setup(sq, orc, w, 2, slots)
    e = torch.zeros(0, device="cuda")
    sq.sq_decode_step_linear(pool, torch.zeros(0, dtype=torch.int32, device="cuda"), e, e, e, e, e)
    torch.cuda.synchronize()
    assert np.array_equal(dev.cpu().numpy(), pre)


def test_refusals(sq, orc):
    w = I.Workload("lerr", 2, 12, 128, 128, 1, MIX, seed=6)
    slots = np.array([0, 1], np.int32)
    *_, dev, pool = setup(sq, orc, w, 2, slots)
    si = I.step_inputs(w, 0)
    ids, q, k, v, a, b = (x.cuda() for x in (torch.from_numpy(slots), si.q, si.k, si.v, si.alpha, si.beta))
    fn, vp = sq._lib.sq_decode_step_linear, ctypes.c_void_p
    args = [pool.handle, ids.data_ptr(), 2, q.data_ptr(), k.data_ptr(), v.data_ptr(), 1, a.data_ptr(), b.data_ptr(),
            None, None]
    for at, bad in ((0, None), (1, None), (2, -1), (2, 3), (3, None), (4, vp(k.data_ptr() + 2)), (5, None), (6, 7),
                    (7, None), (8, None), (9, vp(16 + 4))):
        call = list(args)
        call[at] = bad
        assert fn(*call) == sq.SQ_ERR_INVALID, at
    with pytest.raises(sq.SqError):
        sq.sq_decode_step_linear(pool, ids, q, k, v, a[:1], b)
