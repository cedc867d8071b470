"""The selective scan (prompts, packed documents, single tokens) against the fp64 oracle,
element by element.

Bounds, in units of e = 2^-24 (half a step of fp32), carried along the recurrence in fp64:
  dt'   without softplus: one rounding of the sum with the bias, e |dt'|. With: the sum's rounding
        moves the result by at most e |v| (slope below 1), the exponential and the series by below
        16 e of the result.
  a     the exponent x = dt' A is off by dt's relative error, the rounding of A log2(e) (2 e) and
        of the product (e); 2^x adds 2 ulp = 4 e: relative error |x| (r_dt + 3 e) + 4 e.
  h     err_t = a err_{t-1} + r_a a |h_{t-1}| + (r_dt + 3 e) |dt' u B| + e |h_t|, on magnitudes.
        A prompt's pieces are joined as decay * entering state + local state, where each path has
        the same factors and one more rounding per join: doubled.
  y     sum |C| err + (N + 3) e sum |C||h| + 2 e |D u|, times SiLU, whose own relative error is
        below (2 |z| + 9) e; one rounding to the storage type, eps/2 of the value.
"""
import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu

E32 = 2.0 ** -24
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def ssd(cuda_device):
    from structured_state_space_fwd_b200 import build
    build.build()
    import structured_state_space_fwd_b200 as m
    return m


def inputs(b, T, D, G, N, dtype, dt="", nseq=None, seed=0, softplus=True, gate=True, skip=True, states=True,
           fast=False):
    """fast: rates and steps so large that a state forgets within a few tokens."""
    g = torch.Generator().manual_seed(seed)
    n = b if nseq is None else nseq
    t, td = TYPES[dtype], TYPES[dt or dtype]

    def normal(*s):
        return torch.randn(*s, generator=g)
    step = torch.exp(torch.rand(D, generator=g) * 4.6 - (2.0 if fast else 6.9))
    d = {"u": normal(b, T, D).to(t), "dt": None, "A": -(torch.rand(D, N, generator=g) * 15 + 0.5),
         "B": normal(b, T, G, N).to(t), "C": normal(b, T, G, N).to(t), "D": normal(D) if skip else None,
         "z": (2 * normal(b, T, D)).to(t) if gate else None, "dt_bias": None, "dt_softplus": softplus,
         "initial_states": normal(n, D, N) if states else None}
    if softplus:
        d["dt_bias"] = step + torch.log(-torch.expm1(-step))
        d["dt"] = normal(b, T, D).to(td)
    else:
        d["dt"] = (step * (0.5 + torch.rand(b, T, D, generator=g))).to(td)
    return d


def cuda(d):
    return {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in d.items()}


def _f(t):
    return t.double().numpy() if t is not None else None


def _one(d, init):
    """(y, bound of y before rounding, h, bound of h) of sequences side by side."""
    u, dtr, A, B, C = (_f(d[k]) for k in ("u", "dt", "A", "B", "C"))
    bias = _f(d["dt_bias"])
    dt = oracle.selective_steps(dtr, bias, d["dt_softplus"])
    off = 0.0 if bias is None and not d["dt_softplus"] else \
        np.abs(dtr + (0 if bias is None else bias)) * E32 + (16 * E32 * dt if d["dt_softplus"] else 0.0)
    r_dt = off / np.maximum(np.abs(dt), 1e-300) + 0 * dt
    b, T, D = u.shape
    N, G = A.shape[1], B.shape[2]
    group = np.arange(D) // (D // G)
    h = np.zeros((b, D, N)) if init is None else _f(init)
    H, err = np.abs(h), np.zeros((b, D, N))
    y, yb = np.zeros((b, T, D)), np.zeros((b, T, D))
    for t in range(T):
        x = dt[:, t, :, None] * A
        a = np.exp(x)
        p = (dt[:, t] * u[:, t])[..., None] * B[:, t, group]
        r = r_dt[:, t, :, None]
        err = a * err + (np.abs(x) * (r + 3 * E32) + 4 * E32) * a * H + (r + 3 * E32) * np.abs(p)
        h, H = a * h + p, a * H + np.abs(p)
        err = err + E32 * H
        Ct = C[:, t, group]
        y[:, t] = np.sum(Ct * h, -1)
        yb[:, t] = np.sum(np.abs(Ct) * (2 * err + (N + 3) * E32 * H), -1)
    if d["D"] is not None:
        y, yb = y + _f(d["D"]) * u, yb + 2 * E32 * np.abs(_f(d["D"]) * u)
    if d["z"] is not None:
        z = _f(d["z"])
        s = z / (1 + np.exp(-z))
        y, yb = y * s, yb * np.abs(s) + (2 * np.abs(z) + 9) * E32 * np.abs(y * s)
    return y, yb, h, 2 * err


def reference(d, cu=None):
    init = d["initial_states"]
    if cu is None:
        y, yb, h, hb = _one(d, init)
        ys, hs, _ = *oracle.selective_scan(**d), None
        np.testing.assert_allclose(y, ys, rtol=1e-9, atol=1e-12)
        np.testing.assert_allclose(h, hs, rtol=1e-9, atol=1e-12)
        return y, yb, h, hb
    got = []
    for k, (p, q) in enumerate(zip(cu, cu[1:])):
        part = {n: (v[:, p:q] if n in ("u", "dt", "B", "C", "z") and v is not None else v) for n, v in d.items()}
        got.append(_one(part, init[k:k + 1] if init is not None else None))
    return tuple(np.concatenate([g[i] for g in got], 1 if i < 2 else 0) for i in range(4))


def check(got, ref, bound, t):
    got = got.double().cpu().numpy()
    lim = bound + (np.abs(ref) + bound) * torch.finfo(t).eps / 2 + 1e-37
    assert got.shape == ref.shape
    worst = np.max(np.abs(got - ref) / lim) if ref.size else 0.0
    assert worst <= 1.0, f"{worst:.3f} of the bound"


def run_and_check(ssd, d, dev=None):
    dev = cuda(d) if dev is None else dev
    y, fin = ssd.ssd_selective_scan(**dev, return_final_states=True)
    ry, yb, rh, hb = reference(d)
    check(y, ry, yb, d["u"].dtype)
    check(fin, rh, hb, torch.float32)
    return y, fin


SHAPES = [
    # b, T, D, G, N
    (2, 50, 32, 1, 16), (1, 1, 8, 1, 16), (1, 2, 5, 1, 1), (3, 17, 33, 3, 5), (1, 300, 16, 1, 16),
    (1, 515, 40, 2, 16), (2, 64, 24, 8, 64), (1, 40, 10, 1, 100), (1, 33, 6, 2, 256), (2, 9, 70, 1, 3),
    (1, 1025, 9, 1, 8), (1, 129, 130, 1, 16), (1, 260, 64, 1, 32), (2, 31, 1, 1, 7), (1, 70, 48, 16, 12),
    (0, 5, 8, 1, 4), (2, 0, 8, 1, 4),
]


@pytest.mark.parametrize("dtype,dt", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("b,T,D,G,N", SHAPES)
def test_scan_shapes(ssd, b, T, D, G, N, dtype, dt):
    run_and_check(ssd, inputs(b, T, D, G, N, dtype, dt, seed=T + N))


@pytest.mark.parametrize("b,T,D,G,N,dtype", [
    # many channels: a lane each, two warps in turn; over one, two and several tiles of 16 tokens
    (1, 16, 4800, 1, 16, "bf16"), (2, 70, 4801, 1, 16, "f32"), (3, 33, 9600, 2, 8, "bf16"),
    (1, 65, 19300, 1, 4, "f32"), (2, 17, 9664, 1, 3, "bf16"), (1, 50, 4800, 150, 13, "bf16"),
    # many channels and more states than a lane holds at once
    (4, 140, 4800, 1, 17, "bf16"), (8, 131, 2400, 1, 35, "f32"),
    # few channels: several rounds of 128 tokens, states in blocks and not
    (2, 200, 2400, 1, 20, "bf16"), (1, 200, 2416, 1, 16, "f32"), (1, 300, 40, 1, 64, "bf16"),
    (1, 290, 20, 2, 130, "f32"), (1, 400, 33, 1, 7, "bf16"), (1, 200, 70, 1, 2, "f32"),
    # very few channels: segments over clusters of 8 and 4, whole and partial ones, states in blocks
    (1, 1025, 20, 1, 16, "bf16"), (2, 1500, 40, 2, 15, "f32"), (1, 1100, 37, 1, 40, "bf16"), (3, 513, 64, 1, 16, "f32"),
    (1, 700, 480, 1, 6, "bf16"), (1, 2050, 7, 7, 3, "f32"), (1, 513, 300, 1, 130, "f32"),
    # few channels, few tokens
    (1, 5, 40, 1, 40, "bf16"), (1, 64, 16, 1, 16, "f32"), (1, 63, 16, 1, 17, "f32"), (2, 16, 4096, 1, 20, "bf16"),
    (1, 65, 40, 1, 16, "bf16"), (1, 128, 33, 1, 5, "f32"), (1, 129, 2368, 1, 16, "bf16"), (1, 40, 2384, 1, 33, "f32"),
])
def test_scan_forms(ssd, b, T, D, G, N, dtype):
    """Sizes on both sides of every choice between the kernels' forms."""
    run_and_check(ssd, inputs(b, T, D, G, N, dtype, seed=N))


@pytest.mark.parametrize("softplus", [True, False])
@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("skip,states", [(True, False), (False, True)])
def test_scan_options(ssd, softplus, gate, skip, states):
    for dtype, N in (("f32", 16), ("bf16", 6)):
        run_and_check(ssd, inputs(2, 75, 20, 1, N, dtype, seed=3, softplus=softplus, gate=gate, skip=skip,
                                  states=states))


def test_scan_softplus_without_bias(ssd):
    d = inputs(1, 60, 16, 1, 16, "f32", seed=4)
    d["dt_bias"] = None
    d["dt"] = d["dt"] * 6                       # down to steps of 1e-8, up to 20
    run_and_check(ssd, d)


def test_scan_bias_without_softplus(ssd):
    d = inputs(1, 60, 16, 1, 16, "f32", seed=4, softplus=False)
    d["dt_bias"] = torch.rand(16, generator=torch.Generator().manual_seed(1)) * 0.1
    run_and_check(ssd, d)


@pytest.mark.parametrize("N", [1, 4, 16, 33])
def test_scan_fast_and_slow_decays(ssd, N):
    """States that vanish within a few tokens (decays that underflow), and that hardly move."""
    d = inputs(1, 400, 24, 1, N, "f32", seed=N, fast=True)
    d["A"][::2] *= 20
    run_and_check(ssd, d)
    d["A"] = torch.zeros(24, N)                # no decay: plain sums
    run_and_check(ssd, d)


@pytest.mark.parametrize("T,D", [(1, 40), (50, 40), (300, 40), (1200, 40), (33, 4800)])
def test_steps_of_zero_leave_the_state(ssd, T, D):
    """dt = 0: a decay of exactly 1 and nothing added, in every form."""
    d = cuda(inputs(1, T, D, 1, 16, "f32", seed=1, softplus=False))
    d["dt"].zero_()
    _, fin = ssd.ssd_selective_scan(**d, return_final_states=True)
    assert torch.equal(fin, d["initial_states"])
    state = d.pop("initial_states")
    before = state.clone()
    ssd.ssd_selective_step(**d, state=state)
    assert torch.equal(state, before)


def test_scan_growing_states(ssd):
    """A above 0 is not refused: states grow, within fp32's range."""
    d = inputs(1, 90, 16, 1, 16, "f32", seed=2, softplus=False)
    d["A"] = -d["A"] * 0.1
    run_and_check(ssd, d)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("off,pad", [(8, 8), (2, 2), (3, 2)])
@pytest.mark.parametrize("T,D", [(70, 24), (30, 4800), (270, 24)])
def test_scan_slices_of_wider_rows(ssd, dtype, off, pad, T, D):
    """Every input inside wider rows, aligned to 16 bytes, to 4 and to its element."""
    b, G, N = 2, 2, 16
    d = inputs(b, T, D, G, N, dtype, seed=7)
    dev = cuda(d)
    for k in ("u", "dt", "z", "B", "C"):
        flat = d[k].reshape(b, T, -1)
        wide = torch.zeros(b, T, off + flat.shape[-1] + pad, dtype=flat.dtype)
        wide[..., off:off + flat.shape[-1]] = flat
        dev[k] = wide.cuda()[..., off:off + flat.shape[-1]]
        if k in ("B", "C"):
            dev[k] = dev[k].unflatten(-1, (G, N))
        assert not dev[k].is_contiguous()
    run_and_check(ssd, d, dev)
    # one row for every token, and for every batch row
    d["z"] = d["z"][:, :1].expand(b, T, D)
    dev["z"] = dev["z"][:, :1].expand(b, T, D)
    d["B"] = d["B"][:1].expand(b, T, G, N)
    dev["B"] = dev["B"][:1].expand(b, T, G, N)
    run_and_check(ssd, d, dev)


DOCS = [
    [0, 5], [0, 0, 5], [0, 1, 2, 3, 3, 3, 10], [0, 64, 128, 200, 200], [0, 63, 64, 65, 300, 301, 517],
    [0, 0, 0], list(range(0, 40)), [0, 257, 258, 900],
]


@pytest.mark.parametrize("dtype,D,N", [("bf16", 32, 16), ("f32", 13, 5)])
@pytest.mark.parametrize("cu", DOCS)
def test_scan_packed(ssd, cu, dtype, D, N):
    for states in (True, False):
        d = inputs(1, cu[-1], D, 1, N, dtype, nseq=len(cu) - 1, seed=len(cu), states=states)
        ry, yb, rh, hb = reference(d, cu)
        for offsets in (cu, torch.tensor(cu, dtype=torch.int32, device="cuda")):
            y, fin = ssd.ssd_selective_scan_varlen(**cuda(d), cu_seqlens=offsets, return_final_states=True)
            check(y, ry, yb, d["u"].dtype)
            check(fin, rh, hb, torch.float32)


def test_scan_packed_many_channels(ssd):
    """Documents of every length around a tile, many of them, in the form for many channels."""
    cu = [0, 1, 1, 17, 33, 48, 49, 81, 112, 113, 145, 177, 178]
    for dtype, N, D in (("bf16", 16, 1600), ("f32", 20, 1700), ("f32", 16, 1700), ("bf16", 18, 400)):
        d = inputs(1, cu[-1], D, 1, N, dtype, nseq=len(cu) - 1, seed=N)
        ry, yb, rh, hb = reference(d, cu)
        y, fin = ssd.ssd_selective_scan_varlen(**cuda(d), cu_seqlens=cu, return_final_states=True)
        check(y, ry, yb, d["u"].dtype)
        check(fin, rh, hb, torch.float32)


def test_scan_packed_few_channels(ssd):
    """Documents over the CTAs of a cluster: long, short, empty and single-token ones, some with
    segments that hold no token."""
    cu = [0, 2500, 2501, 2501, 2630, 2900, 3900]
    for dtype, D, N in (("bf16", 24, 16), ("f32", 17, 20)):
        d = inputs(1, cu[-1], D, 1, N, dtype, nseq=len(cu) - 1, seed=N)
        ry, yb, rh, hb = reference(d, cu)
        y, fin = ssd.ssd_selective_scan_varlen(**cuda(d), cu_seqlens=cu, return_final_states=True)
        check(y, ry, yb, d["u"].dtype)
        check(fin, rh, hb, torch.float32)
    wild = torch.tensor([-7, 2000, 1200, 3905, 800], dtype=torch.int32, device="cuda")
    guard = torch.full((3900 + 64, 17), 3.0, device="cuda")
    dev = cuda(d)
    dev["initial_states"] = dev["initial_states"][:4].contiguous()
    ssd.ssd_selective_scan_varlen(**dev, cu_seqlens=wild, y=guard[32:32 + 3900][None])
    torch.cuda.synchronize()
    assert bool((guard[:32] == 3).all()) and bool((guard[32 + 3900:] == 3).all())


def test_scan_rows_behind_the_last_document_stay(ssd):
    d = inputs(1, 200, 32, 1, 16, "bf16", nseq=3, seed=5)
    cu = [0, 40, 41, 131]
    ry, yb, rh, hb = reference({k: (v[:, :131] if k in ("u", "dt", "B", "C", "z") else v) for k, v in d.items()}, cu)
    y = torch.full((1, 200, 32), 7.0, dtype=torch.bfloat16, device="cuda")
    _, fin = ssd.ssd_selective_scan_varlen(**cuda(d), cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"),
                                           y=y, return_final_states=True)
    check(y[:, :131], ry, yb, torch.bfloat16)
    check(fin, rh, hb, torch.float32)
    assert bool((y[:, 131:] == 7.0).all())


@pytest.mark.parametrize("cu", [[-5, 3, 1000], [3, 1, 90, 20], [90, 90, 90], [5, 7], [-9, -3]])
def test_scan_malformed_offsets_stay_inside(ssd, cu):
    T, D, N, n = 90, 32, 16, len(cu) - 1
    guard = torch.full((T + 64, D), 3.0, device="cuda")
    states = torch.full((n * D + 64, N), 5.0, device="cuda")
    d = cuda(inputs(1, T, D, 1, N, "f32", nseq=n, seed=2))
    ssd.ssd_selective_scan_varlen(**d, cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"),
                                  y=guard[32:32 + T][None], final_states=states[32:32 + n * D].view(n, D, N))
    torch.cuda.synchronize()
    assert bool((guard[:32] == 3).all()) and bool((guard[32 + T:] == 3).all())
    assert bool((states[:32] == 5).all()) and bool((states[32 + n * D:] == 5).all())


@pytest.mark.parametrize("dtype,dt", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("b,T,D,G,N", [(3, 1, 64, 1, 16), (1, 1, 5, 1, 3), (2, 4, 24, 2, 16), (130, 1, 12, 1, 64),
                                       (2, 2, 6, 1, 256), (1, 1, 1, 1, 1), (2, 3, 40, 1, 30), (0, 1, 8, 1, 4),
                                       (2, 0, 8, 1, 4), (2, 1, 520, 1, 8)])
def test_step(ssd, b, T, D, G, N, dtype, dt):
    for gate, softplus in ((True, True), (False, False)):
        d = inputs(b, T, D, G, N, dtype, dt, seed=b + N, gate=gate, softplus=softplus)
        ry, yb, rh, hb = reference(d)
        dev = cuda(d)
        state = dev.pop("initial_states")
        y = ssd.ssd_selective_step(**dev, state=state)
        check(y, ry, yb, d["u"].dtype)
        check(state, rh, hb, torch.float32)


@pytest.mark.parametrize("b,D,N,dtype", [
    # several batch rows a thread, the last ones short: 4, 2 and 1 lanes a channel, one state at a
    # time, several pieces a lane
    (17, 4800, 16, "bf16"), (18, 4797, 16, "f32"), (17, 10000, 8, "bf16"), (19, 20000, 4, "f32"),
    (17, 2403, 5, "bf16"), (17, 10000, 2, "f32"), (18, 20000, 1, "bf16"), (17, 1300, 48, "f32"),
    (13, 400, 256, "bf16"), (17, 600, 50, "f32"), (17, 600, 99, "bf16"), (13, 404, 255, "f32"),
])
def test_step_many_rows(ssd, b, D, N, dtype):
    d = inputs(b, 2, D, 1, N, dtype, seed=N)
    ry, yb, rh, hb = reference(d)
    dev = cuda(d)
    state = dev.pop("initial_states")
    y = ssd.ssd_selective_step(**dev, state=state)
    check(y, ry, yb, d["u"].dtype)
    check(state, rh, hb, torch.float32)


def test_step_from_an_unaligned_state(ssd):
    """States, A, B and C that start on 4 (2) bytes only."""
    for dtype in ("f32", "bf16"):
        d = inputs(3, 2, 24, 1, 16, dtype, seed=3)
        ry, yb, rh, hb = reference(d)
        dev = cuda(d)

        def moved(t):
            flat = torch.zeros(t.numel() + 1, dtype=t.dtype, device="cuda")
            flat[1:] = t.reshape(-1)
            return flat[1:].view(t.shape)
        state = moved(dev.pop("initial_states"))
        for k in ("A", "B", "C", "u", "dt", "z"):
            dev[k] = moved(dev[k])
        init = state.clone()
        y = ssd.ssd_selective_step(**dev, state=state)
        check(y, ry, yb, d["u"].dtype)
        check(state, rh, hb, torch.float32)
        y, fin = ssd.ssd_selective_scan(**dev, initial_states=moved(init), return_final_states=True,
                                        y=moved(torch.zeros_like(y)))
        check(y, ry, yb, d["u"].dtype)
        check(fin, rh, hb, torch.float32)


def test_step_one_token_form_and_slices(ssd):
    d = cuda(inputs(3, 1, 40, 2, 16, "bf16", seed=4))
    s1 = d.pop("initial_states")
    s2 = s1.clone()
    y = ssd.ssd_selective_step(**d, state=s1)
    one = {k: (v[:, 0] if k in ("u", "dt", "B", "C", "z") else v) for k, v in d.items()}
    one["z"] = torch.cat([one["z"], one["z"]], -1)[:, 40:]
    out = torch.empty(3, 40, dtype=torch.bfloat16, device="cuda")
    y1 = ssd.ssd_selective_step(**one, state=s2, y=out)
    assert torch.equal(y[:, 0], y1) and torch.equal(s1, s2) and y1.data_ptr() == out.data_ptr()


def test_prompt_then_tokens(ssd):
    """A prompt in two calls, then tokens, against the recurrence over all of it."""
    T = 330
    d = inputs(2, T, 48, 1, 16, "bf16", seed=8)
    ry, yb, rh, hb = reference(d)
    dev = cuda(d)
    state, ys = dev.pop("initial_states"), []

    def cut(p, q):
        return {k: (v[:, p:q] if k in ("u", "dt", "B", "C", "z") else v) for k, v in dev.items()}
    for p, q in ((0, 200), (200, 320)):
        y, state = ssd.ssd_selective_scan(**cut(p, q), initial_states=state, return_final_states=True)
        ys.append(y)
    for t in range(320, T):
        ys.append(ssd.ssd_selective_step(**cut(t, t + 1), state=state))
    check(torch.cat(ys, 1), ry, yb, torch.bfloat16)
    check(state, rh, hb, torch.float32)


def test_scan_special_values(ssd):
    """What is not finite stays in its channel and behind its token."""
    d = inputs(1, 300, 32, 1, 16, "f32", seed=9)
    clean = ssd.ssd_selective_scan(**cuda(d))
    d["u"][0, 100, 3] = float("nan")
    d["dt"][0, 120, 5] = float("nan")
    d["u"][0, 140, 7] = float("inf")
    y = ssd.ssd_selective_scan(**cuda(d))
    same = torch.ones(300, 32, dtype=torch.bool)
    same[100:, 3] = same[120:, 5] = same[140:, 7] = False
    same = same.cuda()[None]
    assert torch.equal(y[same], clean[same])
    assert torch.isnan(y[0, 100:, 3]).all() and torch.isnan(y[0, 120:, 5]).all()
    assert not torch.isfinite(y[0, 140, 7])
    d = inputs(1, 20, 8, 1, 16, "f32", seed=9)
    d["dt"][0, 3] = -1e30                        # a step of 0: the state stays
    d["dt"][0, 5] = float("-inf")
    d["z"][0, 7] = -300.0                        # a closed gate
    ry, yb, rh, hb = reference({**d, "dt": d["dt"].clamp(min=-700)})
    y, fin = ssd.ssd_selective_scan(**cuda(d), return_final_states=True)
    check(y, ry, yb, torch.float32)
    check(fin, rh, hb, torch.float32)


def test_scan_past_32_bits(ssd):
    """Element offsets above 2^31 in every strided input."""
    T, D, N, row = 2200, 32, 16, 1 << 20
    d = inputs(1, T, D, 1, N, "bf16", seed=6)
    wide = torch.zeros(T, row, dtype=torch.bfloat16, device="cuda")
    dev, at = cuda(d), 64
    for k in ("u", "dt", "z", "B", "C"):
        flat = dev[k].reshape(T, -1)
        wide[:, at:at + flat.shape[1]] = flat
        dev[k] = wide[None, :, at:at + flat.shape[1]]
        if k in ("B", "C"):
            dev[k] = dev[k].unflatten(-1, (1, N))
        at += flat.shape[1]
    y, fin = ssd.ssd_selective_scan(**dev, return_final_states=True)
    y1, fin1 = ssd.ssd_selective_scan(**cuda(d), return_final_states=True)
    assert torch.equal(y, y1) and torch.equal(fin, fin1)


def test_scan_large_outputs(ssd):
    """Outputs past 2^31 elements: the last tokens equal those of a call on the last tokens
    alone (from a state that has forgotten)."""
    T, D, N = (1 << 17) + 40, 16384, 1
    d = cuda(inputs(1, 64, D, 1, N, "bf16", seed=6, states=False, softplus=False))
    d["A"] = torch.full((D, N), -1e6, device="cuda")          # each token on its own
    part = ssd.ssd_selective_scan(**d)
    big = dict(d)
    for k in ("u", "dt", "z", "B", "C"):
        big[k] = torch.cat([d[k][:, :1].expand(1, T - 64, *d[k].shape[2:]), d[k]], 1)
    y = ssd.ssd_selective_scan(**big)
    assert torch.equal(y[:, -64:], part) and torch.equal(y[:, 1000], part[:, 0])


def test_scan_is_deterministic_and_batch_rows_are_apart(ssd):
    d = cuda(inputs(4, 300, 64, 1, 16, "bf16", seed=1))
    y, fin = ssd.ssd_selective_scan(**d, return_final_states=True)
    y2, fin2 = ssd.ssd_selective_scan(**d, return_final_states=True)
    assert torch.equal(y, y2) and torch.equal(fin, fin2)
    for i in (0, 3):
        one = {k: (v[i:i + 1] if isinstance(v, torch.Tensor) and v.shape[0] == 4 and v.dim() > 2 else v)
               for k, v in d.items()}
        y1, f1 = ssd.ssd_selective_scan(**one, return_final_states=True)
        assert torch.equal(y1, y[i:i + 1]) and torch.equal(f1, fin[i:i + 1])


def test_scan_streams_and_graphs(ssd):
    """Two calls at once on two streams; a captured step replayed token by token."""
    d = cuda(inputs(2, 40, 64, 1, 16, "bf16", seed=1))
    ref, fin = ssd.ssd_selective_scan(**d, return_final_states=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a = ssd.ssd_selective_scan(**d, stream=side)
    b = ssd.ssd_selective_scan(**d)
    torch.cuda.synchronize()
    assert torch.equal(a, ref) and torch.equal(b, ref)
    one = {k: (v[:1] if isinstance(v, torch.Tensor) and v.dim() > 2 else v) for k, v in d.items()}
    one["initial_states"] = d["initial_states"].contiguous()
    packed = ssd.ssd_selective_scan_varlen(**one, cu_seqlens=[0, 17, 40])
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(20):                          # host offsets: copied and freed on the stream that reads them
        c = ssd.ssd_selective_scan_varlen(**one, cu_seqlens=[0, 17, 40], stream=side)
        torch.zeros(64, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    assert torch.equal(c, packed)
    init = d.pop("initial_states")
    state, out = init.clone(), torch.empty_like(ref[:, :1])
    tok = {k: d[k][:, :1].clone() for k in ("u", "dt", "B", "C", "z")}
    rest = {k: d[k] for k in ("A", "D", "dt_bias", "dt_softplus")}
    ssd.ssd_selective_step(**tok, **rest, state=state, y=out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ssd.ssd_selective_step(**tok, **rest, state=state, y=out)
    state.copy_(init)
    eager = init.clone()
    for t in range(40):
        for k, v in tok.items():
            v.copy_(d[k][:, t:t + 1])
        g.replay()
        y = ssd.ssd_selective_step(**tok, **rest, state=eager)
        assert torch.equal(out, y)
    assert torch.equal(state, eager)


def test_scan_binding_refusals(ssd):
    d = cuda(inputs(2, 6, 8, 2, 4, "bf16"))
    f = {k: v for k, v in d.items()}
    for bad, err in ((dict(A=d["A"].bfloat16()), TypeError), (dict(A=d["A"][:, :3]), ValueError),
                     (dict(u=d["u"].half()), TypeError), (dict(u=d["u"][0]), ValueError),
                     (dict(dt=d["dt"].half()), TypeError), (dict(dt=d["dt"][..., :7]), ValueError),
                     (dict(B=d["B"].float()), TypeError), (dict(C=d["C"][:, :5]), ValueError),
                     (dict(B=d["B"].transpose(2, 3)), ValueError), (dict(z=d["z"].float()), TypeError),
                     (dict(D=d["D"][:7]), ValueError), (dict(dt_bias=d["D"].double()), TypeError),
                     (dict(initial_states=d["initial_states"][:1]), ValueError),
                     (dict(u=d["u"].cpu()), ValueError), (dict(A=d["A"].cpu()), ValueError),
                     (dict(y=d["u"]), ssd.SSDError), (dict(final_states=d["initial_states"]), ssd.SSDError)):
        with pytest.raises(err):
            ssd.ssd_selective_scan(**{**f, **bad})
    with pytest.raises(ValueError, match="batch 1"):
        ssd.ssd_selective_scan_varlen(**f, cu_seqlens=[0, 6])
    state = f.pop("initial_states")
    with pytest.raises(ValueError):
        ssd.ssd_selective_step(**f, state=state[:1])
    with pytest.raises(TypeError):
        ssd.ssd_selective_step(**f, state=state.bfloat16())
    big = cuda(inputs(1, 2, 4, 1, 257, "f32"))
    with pytest.raises(ssd.SSDError, match="UNSUPPORTED"):
        ssd.ssd_selective_scan(**big)
