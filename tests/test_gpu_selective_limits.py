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
