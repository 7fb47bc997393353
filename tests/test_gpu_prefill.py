"""sq_prefill on the GPU against the token-by-token recurrence in 64 bits.

Tolerances.  A state or output element is a sum over at most T tokens and d_k
key rows, evaluated in fp32 or better: its error is at most about
(T + 4 d_k) units of 2^-24 of the largest magnitude in its tile.  An output in
bfloat16 is rounded once more, half a unit of 2^-8 of itself."""
import numpy as np
import pytest
import torch

import serve_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sq():
    from quantized_recurrent_state_gated_amd import sq as m
    return m


DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def make(seed, lens, H, Hk, dk, dv, dtype, init=True, keys="random"):
    g = torch.Generator().manual_seed(seed)
    N, dt = sum(lens), DT[dtype]
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    q, k = r(N, Hk, dk), r(N, Hk, dk)
    if keys == "alike":  # neighbouring tokens share most of their direction
        k = 0.2 * k + r(1, Hk, dk)
    elif keys == "same":
        k = r(1, Hk, dk).expand(N, Hk, dk).clone()
    if N:
        q, k = q / q.norm(dim=-1, keepdim=True), k / k.norm(dim=-1, keepdim=True)
    life = torch.exp(torch.rand(H, generator=g) * 6.9)
    alpha = torch.exp(-0.693 / life * torch.exp(0.5 * r(N, H)))
    beta = 0.05 + 0.9 * torch.rand(N, H, generator=g)
    S0 = r(len(lens), H, dk, dv) if init else None
    return dict(q=q.to(dt), k=k.to(dt), v=r(N, H, dv).to(dt), alpha=alpha, beta=beta, cu=cu, S0=S0)


def run(sq, x, rule, S=True):
    """The call on GPU copies of x's tensors (strided ones stay strided)."""
    c = lambda t: None if t is None else t.cuda()  # noqa: E731
    q, k, v = c(x["q"]), c(x["k"]), c(x["v"])
    if "wide" in x:
        w = c(x["wide"])
        q, k, v = x["cut"](w)
    n, (N, H, dv), dk = len(x["cu"]) - 1, v.shape, q.shape[2]
    o = torch.full((N, H, dv), float("nan"), dtype=q.dtype, device="cuda")
    out = torch.full((n, H, dk, dv), float("nan"), device="cuda") if S else None
    nb = sq.sq_prefill_workspace(n, N, H, dk, dv, q.dtype, rule)
    ws = torch.full((nb,), 0xff, dtype=torch.uint8, device="cuda") if nb else None
    sq.sq_prefill(q, k, v, c(x["alpha"]), c(x["beta"]), torch.from_numpy(x["cu"]).cuda(), o, S=out,
                  S0=c(x["S0"]), rule=rule, workspace=ws)
    torch.cuda.synchronize()
    return o.float().cpu().numpy().astype(np.float64), None if out is None else out.cpu().numpy().astype(np.float64)


def close(got, want, tokens, dk, bf16, what):
    assert np.isfinite(got).all(), what
    if not got.size:
        return
    lim = (tokens + 4 * dk) * 2.0 ** -24 * np.abs(want).max()
    if bf16:
        lim = lim + 2.0 ** -8 * np.abs(want)
    assert (np.abs(got - want) <= lim).all(), (what, float((np.abs(got - want) / lim).max()))


def check(sq, x, rule, dtype):
    o, S = run(sq, x, rule)
    wo, wS = ref.prefill(x["q"].float(), x["k"].float(), x["v"].float(), x["alpha"], x["beta"], x["cu"], x["S0"],
                         rule == sq.SQ_RULE_DELTA)
    T, dk = int(np.diff(x["cu"]).max()), x["q"].shape[2]
    close(o, wo, T, dk, dtype == "bf16", "o")
    for s in range(len(x["cu"]) - 1):
        close(S[s], wS[s], T, dk, False, f"S{s}")
    return o, S


RAGGED = [0, 1, 63, 64, 65, 130, 0, 257, 15]


@pytest.mark.parametrize("rule", [0, 1])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("init", [False, True])
def test_ragged_d128(sq, rule, dtype, init):
    check(sq, make(1 + rule, RAGGED, 3, 3, 128, 128, dtype, init), rule, dtype)


@pytest.mark.parametrize("rule", [0, 1])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", [(4, 4), (12, 20), (64, 64), (128, 64), (64, 200), (256, 128), (132, 256)])
def test_other_shapes(sq, rule, dtype, dk, dv):
    check(sq, make(dk + dv, [70, 1, 33], 2, 2, dk, dv, dtype), rule, dtype)


@pytest.mark.parametrize("T", [1, 2, 16, 17, 31, 32, 33, 64, 127, 128, 129, 512])
def test_lengths_of_one_sequence(sq, T):
    for rule in (0, 1):
        check(sq, make(T, [T], 5, 5, 128, 128, "bf16"), rule, "bf16")


@pytest.mark.parametrize("rule", [0, 1])
def test_shared_key_heads(sq, rule):
    for dtype, dk, dv in (("bf16", 128, 128), ("f32", 32, 48)):
        check(sq, make(5, [100, 29], 6, 2, dk, dv, dtype), rule, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_parts_of_one_wider_buffer(sq, dtype):
    """q, k and v as parts of one projection's output."""
    H, d, N = 4, 128, 150
    x = make(9, [90, 60], H, H, d, d, dtype)
    x["wide"] = torch.cat([x[n].reshape(N, H * d) for n in "qkv"] + [torch.full((N, 40), float("nan")).to(DT[dtype])], 1)
    x["cut"] = lambda w: tuple(w[:, i * H * d:(i + 1) * H * d].view(N, H, d) for i in range(3))
    check(sq, x, 0, dtype)
    # rows that are not 16-byte aligned are served too
    x["wide"] = torch.cat([torch.zeros(N, 1).to(DT[dtype]), x["wide"]], 1)[:, :3 * H * d + 1].contiguous()
    x["cut"] = lambda w: tuple(w[:, 1 + i * H * d:1 + (i + 1) * H * d].view(N, H, d) for i in range(3))
    check(sq, x, 0, dtype)


@pytest.mark.parametrize("rule", [0, 1])
def test_many_heads_and_many_sequences(sq, rule):
    """Whole heads to a workgroup (more than 128 heads in all), more than 64
    sequences, and a few tokens a sequence."""
    check(sq, make(31, [66, 0, 130], 50, 25, 128, 128, "bf16"), rule, "bf16")
    check(sq, make(33, [(i * 37) % 80 + (i == 7) * 64 for i in range(75)], 2, 2, 128, 128, "bf16"), rule, "bf16")
    check(sq, make(35, [(i * 5) % 14 for i in range(20)], 3, 1, 128, 128, "bf16"), rule, "bf16")


@pytest.mark.parametrize("lens,H", [([5000], 1), ([9000, 1024, 0, 1, 6000], 2), ([2500, 2581], 3), ([4097], 48)])
def test_long_plain_decay(sq, lens, H):
    """Sequences that are cut into segments, the state out of place and in place."""
    x = make(len(lens) + H, lens, H, H, 128, 128, "bf16")
    x["alpha"][:, 0] = 0.9999  # something is left of the segments before
    o, S = check(sq, x, 1, "bf16")
    state = x["S0"].cuda()
    N, n = sum(lens), len(lens)
    po = torch.empty(N, H, 128, dtype=torch.bfloat16, device="cuda")
    nb = sq.sq_prefill_workspace(n, N, H, 128, 128, torch.bfloat16, 1)
    assert nb > 0
    sq.sq_prefill(*(x[k].cuda() for k in ("q", "k", "v", "alpha", "beta")), torch.from_numpy(x["cu"]).cuda(), po,
                  S=state, S0=state, rule=1, workspace=torch.full((nb,), 0xff, dtype=torch.uint8, device="cuda"))
    torch.cuda.synchronize()
    assert np.array_equal(state.cpu().numpy(), S) and np.array_equal(po.float().cpu().numpy(), o)
    with pytest.raises(sq.SqError):
        sq.sq_prefill(*(x[k].cuda() for k in ("q", "k", "v", "alpha", "beta")), torch.from_numpy(x["cu"]).cuda(), po,
                      S=state, S0=state, rule=1)


@pytest.mark.parametrize("keys", ["alike", "same"])
def test_keys_that_lie_close(sq, keys):
    """Nearly parallel keys with full write strength: the inverse of the
    chunk's triangular system has no small entries to hide behind."""
    x = make(11, [200, 64], 3, 3, 128, 128, "bf16", keys=keys)
    x["beta"] = torch.ones_like(x["beta"])
    x["alpha"][:, 0] = 1.0
    check(sq, x, 0, "bf16")


@pytest.mark.parametrize("rule", [0, 1])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gates_of_zero_and_one(sq, rule, dtype):
    x = make(13, [150, 70], 4, 4, 128, 128, dtype)
    x["alpha"][:, 0] = 1.0
    x["alpha"][:, 1] = 0.0
    x["alpha"][::37, 2] = 0.0           # forgets everything now and then
    x["alpha"][:, 3] = 1e-30            # products underflow at once
    x["beta"][:, 1] = 1.0
    x["beta"][::3, 2] = 0.0
    check(sq, x, rule, dtype)


def test_gates_of_tiny_floats(sq):
    """Gates down to the smallest subnormal decay to zero without a NaN."""
    x = make(14, [90], 2, 2, 128, 128, "bf16")
    x["alpha"][:, 0] = 2.0 ** -149
    x["alpha"][::2, 1] = 2.0 ** -126
    for rule in (0, 1):
        check(sq, x, rule, "bf16")


@pytest.mark.parametrize("scale", [1e-20, 1e15])
def test_large_and_small_values(sq, scale):
    """The map is linear in (S0, v): scaled inputs scale the outputs."""
    x = make(15, [129], 2, 2, 128, 128, "bf16")
    x["v"] = (x["v"].float() * scale).bfloat16()
    x["S0"] = x["S0"] * scale
    for rule in (0, 1):
        check(sq, x, rule, "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rule", [0, 1])
def test_two_parts_make_the_whole(sq, dtype, rule):
    """Prompts given in two calls, the state handed on in place."""
    x = make(17, [133, 133], 3, 3, 128, 128, dtype)
    o, S = ref.prefill(x["q"].float(), x["k"].float(), x["v"].float(), x["alpha"], x["beta"], x["cu"], x["S0"],
                       rule == 0)
    cuts, got, state = [0, 50, 133], np.zeros_like(o), x["S0"].cuda()
    cu = x["cu"]
    for lo, hi in zip(cuts, cuts[1:]):
        tok = np.concatenate([np.arange(cu[s] + lo, cu[s] + hi) for s in range(2)])
        part = {n: x[n][tok].cuda().contiguous() for n in ("q", "k", "v", "alpha", "beta")}
        c2 = torch.tensor([0, hi - lo, 2 * (hi - lo)], dtype=torch.int32, device="cuda")
        po = torch.empty(len(tok), 3, 128, dtype=DT[dtype], device="cuda")
        nb = sq.sq_prefill_workspace(2, len(tok), 3, 128, 128, DT[dtype], rule)
        sq.sq_prefill(**part, cu_seqlens=c2, o=po, S=state, S0=state, rule=rule,
                      workspace=torch.empty(nb, dtype=torch.uint8, device="cuda") if nb else None)
        got[tok] = po.float().cpu().numpy()
    close(state.cpu().numpy(), S, 133, 128, False, "S")
    close(got, o, 133, 128, dtype == "bf16", "o")


def test_a_token_is_a_decode_step(sq):
    """One-token prompts and the decode steps on FP32-state heads agree."""
    n, H, d = 4, 6, 128
    x = make(19, [1] * n, H, H, d, d, "bf16")
    ones = torch.ones(H, d, device="cuda")
    ids = torch.arange(n, dtype=torch.int32, device="cuda")
    for rule, step in ((0, sq.sq_decode_step), (1, sq.sq_decode_step_linear)):
        o, S = run(sq, x, rule)
        buf = torch.empty(sq.sq_pool_bytes(n, H, d, d, [32] * H), dtype=torch.uint8, device="cuda")
        pool = sq.sq_pool_alloc(n, H, d, d, [32] * H, ones, ones, buf)
        sq.sq_pool_store(pool, ids, x["S0"].cuda())
        o2, S2 = torch.empty(n, H, d, device="cuda"), torch.empty(n, H, d, d, device="cuda")
        step(pool, ids, x["q"].cuda(), x["k"].cuda(), x["v"].cuda(), x["alpha"].cuda(), x["beta"].cuda(), o2)
        sq.sq_pool_load(pool, ids, S2)
        close(S, S2.cpu().numpy(), 1, d, False, "S")
        close(o, o2.cpu().numpy().astype(np.float64), 1, d, True, "o")


def test_no_state_wanted_and_no_tokens(sq):
    x = make(21, [40, 0, 3], 2, 2, 128, 128, "bf16")
    o, _ = run(sq, x, 0, S=False)
    o2, _ = run(sq, x, 0)
    assert np.array_equal(o, o2)
    for init in (False, True):
        x = make(22, [0, 0], 2, 2, 128, 128, "bf16", init)
        o, S = run(sq, x, 0)
        assert o.shape[0] == 0
        assert np.array_equal(S, x["S0"].numpy().astype(np.float64) if init else np.zeros_like(S))


def test_repeated_calls_are_bit_identical(sq):
    x = make(23, [300, 77, 5], 4, 4, 128, 128, "bf16")
    for rule in (0, 1):
        a, b = run(sq, x, rule), run(sq, x, rule)
        assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])


def test_a_nan_stays_in_its_sequence(sq):
    """NaN in one token leaves other sequences and earlier chunks of 64 tokens
    alone and reaches every later token; token by token it is causal."""
    for dtype in ("bf16", "f32"):
        x = make(25, [70, 165, 3], 2, 2, 128, 128, dtype)
        clean = run(sq, x, 0)
        x["v"][145] = float("nan")
        o, S = run(sq, x, 0)
        cu = x["cu"]
        for s in (0, 2):
            assert np.array_equal(o[cu[s]:cu[s + 1]], clean[0][cu[s]:cu[s + 1]])
            assert np.array_equal(S[s], clean[1][s])
        same = 134 if dtype == "bf16" else 145
        assert np.array_equal(o[70:same], clean[0][70:same])
        assert np.isnan(o[145:235]).all() and np.isnan(S[1]).all()


def test_offsets_outside_the_tokens_are_held(sq):
    """cu_seqlens past the buffers, falling or negative: no access outside."""
    x = make(27, [64, 64], 2, 2, 128, 128, "bf16")
    q, k, v, al, be = (x[n].cuda() for n in ("q", "k", "v", "alpha", "beta"))
    for cu in ([0, 64, 5000], [-9, 64, 128], [0, 100, 30], [128, 0, 0]):
        for rule in (0, 1):
            o = torch.zeros(128, 2, 128, dtype=torch.bfloat16, device="cuda")
            S = torch.zeros(2, 2, 128, 128, device="cuda")
            nb = sq.sq_prefill_workspace(2, 128, 2, 128, 128, torch.bfloat16, rule)
            sq.sq_prefill(q, k, v, al, be, torch.tensor(cu, dtype=torch.int32, device="cuda"), o, S=S, rule=rule,
                          workspace=torch.empty(nb, dtype=torch.uint8, device="cuda") if nb else None)
            torch.cuda.synchronize()


def test_another_stream_and_a_graph(sq):
    x = make(29, [100, 31], 3, 3, 128, 128, "bf16", init=False)
    want = run(sq, x, 0)
    q, k, v, al, be = (x[n].cuda() for n in ("q", "k", "v", "alpha", "beta"))
    cu = torch.from_numpy(x["cu"]).cuda()
    o, S = torch.zeros(131, 3, 128, dtype=torch.bfloat16, device="cuda"), torch.zeros(2, 3, 128, 128, device="cuda")
    ws = torch.empty(max(1, sq.sq_prefill_workspace(2, 131, 3, 128, 128, torch.bfloat16, 0)), dtype=torch.uint8,
                     device="cuda")
    call = lambda: sq.sq_prefill(q, k, v, al, be, cu, o, S=S, workspace=ws)  # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert np.array_equal(o.float().cpu().numpy(), want[0]) and np.array_equal(S.cpu().numpy(), want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for i in range(3):
        v.copy_(x["v"] * (i + 1))
        o.zero_()
        S.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = o.clone(), S.clone()
        call()
        torch.cuda.synchronize()
        assert torch.equal(got[0], o) and torch.equal(got[1], S)
