"""The rules that sq_decode_step_linear shares with the other steps: non-finite
inputs and the sticky flag, factors per slot, SQ_CHECK and SQ_KERNEL.

A stored element is compared with alpha S + beta k v in 64 bits over its step
size: a code may differ by one where the quotient lies within 1e-3 of a rounding
boundary, as evaluation orders of fp32 allow; unquantized elements as in
test_gpu_linear_step."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

BITS = [4, 6, 8, 16, 32, 144]
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def sq():
    from quantized_recurrent_state_gated_amd import sq as m
    return m


class Case:
    """n requests on slots of a larger pool, heads of every width twice."""

    def __init__(self, sq, seed, d, n=4, n_slots=6, per_slot=False):
        self.sq, self.n, self.d = sq, n, d
        g = torch.Generator().manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        self.bits = BITS * 2
        H = self.H = len(self.bits)
        self.stride = H + 1 if per_slot else 0
        vecs = n_slots * self.stride if per_slot else H
        self.rs, self.cs = (0.5 + torch.rand(vecs, d, generator=g) for _ in range(2))
        # codes of a few tenths of the range
        top = torch.tensor([2.0 ** (b - 1) - 1 if b <= 8 else 1.0 for b in self.bits])
        self.slots = torch.randperm(n_slots, generator=g)[:n].to(torch.int32)
        self.S0 = r(n, H, d, d) * (0.3 * top)[None, :, None, None]
        self.q, self.k = (r(n, H, d) / d ** 0.5 for _ in range(2))
        self.v = r(n, H, d) * top[None, :, None]
        self.alpha, self.beta = (0.1 + 0.9 * torch.rand(n, H, generator=g) for _ in range(2))
        self.keep = self.rs.cuda(), self.cs.cuda()
        self.state = torch.zeros(sq.sq_pool_bytes(n_slots, H, d, d, self.bits), dtype=torch.uint8, device="cuda")
        self.pool = sq.sq_pool_alloc(n_slots, H, d, d, self.bits, *self.keep, self.state,
                                     scale_slot_stride=self.stride)
        self.ids = self.slots.cuda()
        sq.sq_pool_store(self.pool, self.ids, self.S0.cuda())
        assert sq.sq_pool_last_device_error(self.pool) == sq.SQ_OK

    def load(self):
        S = torch.empty(self.n, self.H, self.d, self.d, device="cuda")
        self.sq.sq_pool_load(self.pool, self.ids, S)
        return S.cpu().double().numpy()

    def step(self):
        o = torch.empty(self.n, self.H, self.d, device="cuda")
        self.sq.sq_decode_step_linear(self.pool, self.ids, *(x.cuda() for x in (self.q, self.k, self.v)),
                                      self.alpha.cuda(), self.beta.cuda(), o)
        return o.cpu().double().numpy()

    def check(self, before, after, o):
        q, k, v, al, be = (x.double().numpy() for x in (self.q, self.k, self.v, self.alpha, self.beta))
        bad = 0
        with np.errstate(all="ignore"):
            for n in range(self.n):
                for h, b in enumerate(self.bits):
                    w = al[n, h] * before[n, h] + be[n, h] * np.outer(k[n, h], v[n, h])
                    wo = w.T @ q[n, h]
                    got, fin = o[n, h], np.isfinite(wo)
                    assert np.array_equal(np.isfinite(got), fin), (n, h)
                    if fin.any():
                        assert (np.abs(got - wo)[fin] <= 1e-5 + 1e-3 * np.abs(wo[fin]).max()).all(), (n, h)
                    a = after[n, h]
                    if b <= 8:
                        at = int(self.slots[n]) * self.stride + h
                        s = (self.rs[at][:, None] * self.cs[at][None]).double().numpy()
                        Q = 2 ** (b - 1) - 1
                        z = w / s
                        code = np.round(a / s)
                        want = np.where(np.isnan(z), 0, np.clip(np.rint(z), -Q, Q))
                        edge = np.abs(np.abs(z - np.floor(z)) - 0.5) < 1e-3
                        assert (np.abs(code - want) <= np.where(edge, 1, 0)).all(), (n, h, b)
                    else:
                        f = np.isfinite(w)
                        assert np.array_equal(a[~f], w[~f], equal_nan=True), (n, h, b)
                        lim = {32: 1e-6, 16: 1e-3, 144: 2.0 ** -8}[b] * np.abs(w[f]) + 2.0 ** -20 * np.abs(w[f]).max(initial=0)
                        assert (np.abs(a[f] - w[f]) <= lim).all(), (n, h, b)
                    bad += int((~np.isfinite(w)).sum())
        return bad


KERNELS = ["tuned", "generic"]


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("d", [128, 12])
def test_finite(sq, monkeypatch, kernel, d):
    monkeypatch.setenv("SQ_KERNEL", kernel)
    c = Case(sq, d, d)
    for _ in range(3):
        before = c.load()
        o = c.step()
        assert c.check(before, c.load(), o) == 0
    assert sq.sq_pool_last_device_error(c.pool) == sq.SQ_OK


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("d", [128, 12])
def test_nonfinite_inputs(sq, monkeypatch, kernel, d):
    """NaN quotients become code 0, infinite ones the bounds; unquantized heads
    keep the value; a query reaches its readout only."""
    monkeypatch.setenv("SQ_KERNEL", kernel)
    c = Case(sq, 100 + d, d)
    c.alpha[0, ::3] = NAN
    c.v[1, :, 5], c.v[1, :, 7], c.v[1, :, 9] = INF, -INF, NAN
    c.k[2, :, 3] = NAN
    before = c.load()
    c.q[3, 1::2, 2] = NAN
    o = c.step()
    assert c.check(before, c.load(), o) > 0
    assert sq.sq_pool_last_device_error(c.pool) == sq.SQ_ERR_DEVICE
    assert sq.sq_pool_last_device_error(c.pool) == sq.SQ_OK  # reading clears it


def test_a_query_alone_sets_no_flag(sq):
    c = Case(sq, 7, 128)
    c.q[:, :, 1] = NAN
    before = c.load()
    o = c.step()
    assert c.check(before, c.load(), o) == 0 and np.isnan(o).all()
    assert sq.sq_pool_last_device_error(c.pool) == sq.SQ_OK


@pytest.mark.parametrize("d", [128, 12])
def test_factors_per_slot(sq, d):
    c = Case(sq, 200 + d, d, per_slot=True)
    for _ in range(2):
        before = c.load()
        o = c.step()
        c.check(before, c.load(), o)


def test_slot_checks(sq, monkeypatch):
    monkeypatch.setenv("SQ_CHECK", "1")
    c = Case(sq, 9, 128)
    good, before = c.ids, c.state.clone()
    for bad in ([0, 1, 1, 2], [0, 1, 2, 6], [-1, 0, 1, 2]):
        c.ids = torch.tensor(bad, dtype=torch.int32, device="cuda")
        with pytest.raises(sq.SqError) as e:
            c.step()
        assert e.value.status == sq.SQ_ERR_INVALID
        torch.cuda.synchronize()
        assert torch.equal(c.state, before)
    c.ids = good
    b = c.load()
    o = c.step()
    c.check(b, c.load(), o)


def test_a_graph_of_steps(sq):
    """Replayed, with eager work between, against the same steps one by one."""
    a, b = Case(sq, 11, 128), Case(sq, 11, 128)
    x = [t.cuda() for t in (a.q, a.k, a.v, a.alpha, a.beta)]
    oa, ob = (torch.empty(a.n, a.H, 128, device="cuda") for _ in range(2))
    sq.sq_decode_step_linear(a.pool, a.ids, *x, oa)
    sq.sq_decode_step_linear(b.pool, b.ids, *x, ob)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sq.sq_decode_step_linear(a.pool, a.ids, *x, oa)
    for i in range(4):
        x[2].mul_(0.5)
        graph.replay()
        sq.sq_decode_step_linear(b.pool, b.ids, *x, ob)
        torch.cuda.synchronize()
        assert torch.equal(a.state, b.state) and torch.equal(oa, ob)
