"""The selective scan at its limits: infinities, rates without bound, small steps, and every outcome of
the choice between its kernels."""
import numpy as np
import pytest
import torch

import oracle
from test_gpu_selective import E32, check, cuda, inputs, reference, run_and_check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ssd(cuda_device):
    from structured_state_space_fwd_b200 import build
    build.build()
    import structured_state_space_fwd_b200 as m
    return m


# b, T, channels: the forms for many channels and few tokens, for few channels (one round, several),
# clusters of 4 and of 8
FORMS = [(2, 50, 40), (1, 100, 4831), (1, 100, 40), (2, 300, 40), (1, 700, 40), (1, 2050, 40)]


def positive(b, T, D, N, dtype, rate=1.0):
    """Everything above 0, so that an infinite input makes an infinite output and no NaN."""
    d = inputs(b, T, D, 1, N, dtype, seed=N, softplus=False, gate=False, skip=False)
    for k in ("u", "B", "C", "initial_states"):
        d[k] = d[k].abs() + 0.1
    d["A"] = torch.full((D, N), -rate)
    d["dt"] = torch.full_like(d["dt"], 0.05)
    return cuda(d)


def run_infinite(ssd, d, step, t, ch):
    """A call that becomes infinite at token t of channel ch of the first batch row, and the same without."""
    b, T, D = d["u"].shape
    clean = {k: (v.clone() if isinstance(v, torch.Tensor) else v) for k, v in d.items()}
    clean["u"][0, t, ch] = clean["dt"][0, t, ch] = 0.25

    def run(a):
        if not step:
            return ssd.ssd_selective_scan(**a, return_final_states=True)
        a = dict(a)
        state = a.pop("initial_states").clone()
        return ssd.ssd_selective_step(**a, state=state), state
    (y, fin), (yc, fc) = run(d), run(clean)
    assert (y[0, t:, ch] == float("inf")).all() and (fin[0, ch] == float("inf")).all()
    y[0, t:, ch], fin[0, ch] = yc[0, t:, ch], fc[0, ch]
    assert torch.equal(y, yc) and torch.equal(fin, fc)            # and nothing else changed


def infinite_scan(ssd, b, T, D, N, dtype):
    for kind in range(3):
        d = positive(b, T, D, N, dtype)
        t, ch = T // 2 - 1, D - 3
        if kind == 0:
            d["u"][0, t, ch] = float("inf")
        elif kind == 1:
            d["dt"][0, t, ch] = float("inf")
        else:
            d["u"][0, t, ch], d["dt"][0, t, ch] = 3e38, 2.0
        run_infinite(ssd, d, False, t, ch)


def infinite_step(ssd, b, D, N, dtype):
    for kind in range(3):
        d = positive(b, 3, D, N, dtype)
        if kind == 0:
            d["u"][0, 1, 7] = float("inf")
        elif kind == 1:
            d["dt"][0, 1, 7] = float("inf")
        else:
            d["u"][0, 1, 7], d["dt"][0, 1, 7] = 3e38, 2.0
        run_infinite(ssd, d, True, 1, 7)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N", [8, 16, 32])
@pytest.mark.parametrize("b,T,D", FORMS + [(1, 16, 40), (4, 140, 4800)])
def test_scan_infinite_inputs(ssd, b, T, D, N, dtype):
    """An infinite input, step or product of both reaches y as it is, without D too (no 0 times infinity)."""
    infinite_scan(ssd, b, T, D, N, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N", [1, 16, 128])
@pytest.mark.parametrize("b,D", [(2, 40), (18, 4800)])
def test_step_infinite_inputs(ssd, b, D, N, dtype):
    infinite_step(ssd, b, D, N, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N", [1, 3, 5, 11, 20])
@pytest.mark.parametrize("b,T,D", FORMS + [(1, 16, 40), (4, 140, 4800)])
def test_scan_infinite_inputs_beside_padded_states(ssd, b, T, D, N, dtype):
    """State counts that leave some of a kernel's states empty, which stay 0 whatever the input is."""
    infinite_scan(ssd, b, T, D, N, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N", [3, 5, 12, 36, 70, 100, 130, 200])
@pytest.mark.parametrize("b,D", [(2, 40), (18, 4800)])
def test_step_infinite_inputs_beside_padded_states(ssd, b, D, N, dtype):
    infinite_step(ssd, b, D, N, dtype)


@pytest.mark.parametrize("N", [1, 5, 11, 16, 20])
@pytest.mark.parametrize("b,T,D", FORMS)
def test_scan_nan_inputs(ssd, b, T, D, N):
    """NaN stays in its channel and behind its token, beside padded states too."""
    d = positive(b, T, D, N, "bf16")
    yc, fc = ssd.ssd_selective_scan(**d, return_final_states=True)
    d["u"][0, T // 2, D - 3] = float("nan")
    y, fin = ssd.ssd_selective_scan(**d, return_final_states=True)
    assert torch.isnan(y[0, T // 2:, D - 3]).all() and torch.isnan(fin[0, D - 3]).all()
    y[0, T // 2:, D - 3], fin[0, D - 3] = yc[0, T // 2:, D - 3], fc[0, D - 3]
    assert torch.equal(y, yc) and torch.equal(fin, fc)


@pytest.mark.parametrize("rate", [float("-inf"), -3e38])
@pytest.mark.parametrize("N", [1, 5, 16, 20])
@pytest.mark.parametrize("b,T,D", FORMS + [(1, 18, 40), (1, 1, 40)])
def test_scan_rates_without_bound(ssd, b, T, D, N, rate):
    """A = -inf, or so large that its exponent overflows: nothing is kept from one token to the next,
    also where the last tile is not full."""
    for dtype in ("f32", "bf16"):
        d = cuda(inputs(b, T, D, 1, N, dtype, seed=3))
        d["dt"] = d["dt"].abs() * 4                              # steps of at least softplus(-7) = 9e-4
        d["A"][1] = -1e6
        y, fin = ssd.ssd_selective_scan(**d, return_final_states=True)
        d["A"][1] = rate
        y1, fin1 = ssd.ssd_selective_scan(**d, return_final_states=True)
        assert torch.equal(y, y1) and torch.equal(fin, fin1)
        state = d.pop("initial_states")
        y2 = ssd.ssd_selective_step(**d, state=state)
        assert torch.isfinite(y2).all() and torch.isfinite(state).all()


@pytest.mark.parametrize("N", [1, 16, 20])
@pytest.mark.parametrize("b,T,D", FORMS)
def test_scan_infinite_states_stay(ssd, b, T, D, N):
    """An infinite state stays infinite, also where the decays of a cluster's segment multiply to less
    than fp32 holds."""
    d = positive(b, T, D, N, "f32", rate=8.0)
    d["u"][0, 5, 3] = float("inf")
    run_infinite(ssd, d, False, 5, 3)


def tight_reference(d):
    """test_gpu_selective's bounds with dt' charged by the slope of softplus, sigmoid(v): the rounding of
    the sum with the bias (E32 |v|, none without a bias) and of the exponent v log2(e) (the product's and the
    constant's, 2 E32 |v|) move dt' by sigmoid(v) times that, and the exponential and the series by below
    16 E32 of dt'."""
    v = d["dt"].double().numpy()
    if d["dt_bias"] is not None:
        v = v + d["dt_bias"].double().numpy()
    dt = oracle.selective_steps(v, None, True)
    off = np.abs(v) / (1 + np.exp(-v)) * (2 if d["dt_bias"] is None else 3) * E32 + 16 * E32 * dt
    u, A, B, C = (d[k].double().numpy() for k in ("u", "A", "B", "C"))
    b, T, D = u.shape
    N, group = A.shape[1], np.arange(D) // (D // B.shape[2])
    h, H, err = (np.zeros((b, D, N)) for _ in range(3))
    y, yb = np.zeros((b, T, D)), np.zeros((b, T, D))
    r_dt = off / dt
    for t in range(T):
        x, r = dt[:, t, :, None] * A, r_dt[:, t, :, None]
        a = np.exp(x)
        p = (dt[:, t] * u[:, t])[..., None] * B[:, t, group]
        err = a * err + (np.abs(x) * (r + 3 * E32) + 4 * E32) * a * H + (r + 3 * E32) * np.abs(p)
        h, H = a * h + p, a * H + np.abs(p)
        err = err + E32 * H
        y[:, t] = np.sum(C[:, t, group] * h, -1)
        yb[:, t] = np.sum(np.abs(C[:, t, group]) * (2 * err + (N + 3) * E32 * H), -1)
    return y, yb, h, 2 * err


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("T,D,N", [(60, 24, 16), (100, 40, 5), (700, 24, 16), (40, 4831, 4), (3, 16, 16)])
def test_scan_small_steps(ssd, T, D, N, bias):
    """Steps of softplus(-20 .. -8), 2e-9 to 3e-4, from a state of zero and with next to no decay: the states
    are sums of dt' u B and nothing else. log(1 + exp(v)) in fp32 keeps no digit of the smallest steps
    (1 + e rounds to 1 below 6e-8)."""
    d = inputs(1, T, D, 1, N, "f32", seed=T, gate=False, skip=False, states=False)
    g = torch.Generator().manual_seed(T)
    d["dt"] = -20 + 12 * torch.rand(1, T, D, generator=g)
    d["dt_bias"] = None
    if bias:
        d["dt_bias"] = torch.rand(D, generator=g)
    for k in ("u", "B", "C"):
        d[k] = d[k].abs() + 0.1                                  # no cancelling: the bounds are relative
    d["A"] = d["A"] * 1e-3
    y, yb, h, hb = tight_reference(d)
    # the naive form is far outside
    v = d["dt"] if d["dt_bias"] is None else d["dt"] + d["dt_bias"]
    naive = torch.log(1 + torch.exp(v)).double().numpy()
    true = oracle.selective_steps(v.double(), None, True)
    assert np.max(np.abs(naive - true) / true) > 0.5
    dev = cuda(d)
    if T > 3:
        got, fin = ssd.ssd_selective_scan(**dev, return_final_states=True)
    else:
        dev.pop("initial_states")
        fin = torch.zeros(1, D, N, device="cuda")
        got = ssd.ssd_selective_step(**dev, state=fin)
    check(got, y, yb, torch.float32)
    check(fin, h, hb, torch.float32)


@pytest.mark.parametrize("dtype,dt", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("b,T,D,N", [
    (3, 33, 4816, 16),     # 903 blocks of 16 channels: 8 CTAs an SM where 6 would leave a second wave
    (3, 33, 9664, 4),      # 906 blocks of 32
    (3, 20, 4816, 7),
    (6, 20, 4880, 13),     # 1830 blocks: two waves of 8, three of 6
    (9, 17, 4880, 16),     # 2745
])
def test_scan_over_waves(ssd, b, T, D, N, dtype, dt):
    """Enough blocks of channels for one to three waves of CTAs, with each type of the steps."""
    run_and_check(ssd, inputs(b, T, D, 1, N, dtype, dt, seed=N))


def offsets(rng, n, longest):
    """n documents, equal lengths and empty ones among them."""
    lengths = rng.integers(0, longest + 1, size=n)
    lengths[rng.integers(0, n, size=n // 4)] = longest // 2
    lengths[rng.integers(0, n, size=n // 8)] = 0
    return [0] + np.cumsum(lengths).tolist()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("docs,D,N,longest", [
    (33, 640, 16, 40), (63, 320, 16, 50), (64, 1168, 16, 33), (64, 2336, 3, 20), (65, 320, 16, 40),
])
def test_scan_packed_in_order_of_length(ssd, docs, D, N, longest, dtype):
    """Packs of up to 64 documents, which are taken longest first where they make a few waves of CTAs
    (and one of 65, which is not), ties and empty documents among them."""
    cu = offsets(np.random.default_rng(docs + D), docs, longest)
    d = inputs(1, cu[-1], D, 1, N, dtype, nseq=docs, seed=N)
    ry, yb, rh, hb = reference(d, cu)
    y, fin = ssd.ssd_selective_scan_varlen(**cuda(d), cu_seqlens=cu, return_final_states=True)
    check(y, ry, yb, d["u"].dtype)
    check(fin, rh, hb, torch.float32)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cu,D,N", [
    ([0, 300, 300, 380, 680, 685, 900, 1013], 512, 20),          # 7 x 32 units
    ([0, 40, 340, 341, 700], 800, 33),                           # 4 x 50
    (list(range(0, 34 * 90, 90)) + [3100, 3100], 160, 17),       # 35 x 10
])
def test_scan_packed_in_order_of_length_few_channels(ssd, cu, D, N, dtype):
    """The same with more than 16 states and long documents, in the form for few channels."""
    d = inputs(1, cu[-1], D, 1, N, dtype, nseq=len(cu) - 1, seed=N)
    ry, yb, rh, hb = reference(d, cu)
    y, fin = ssd.ssd_selective_scan_varlen(**cuda(d), cu_seqlens=cu, return_final_states=True)
    check(y, ry, yb, d["u"].dtype)
    check(fin, rh, hb, torch.float32)
