"""CPU checks of the operators around the layer: the oracle's convolution and selective
scan against independent computations, and every refusal of the C entries and of the
binding (no test here launches a kernel)."""
import ctypes

import numpy as np
import pytest
import torch

import oracle

RNG = np.random.default_rng(7)


# ---- the oracle ------------------------------------------------------------

@pytest.mark.parametrize("W", [2, 3, 4])
def test_oracle_conv_against_torch(W):
    b, T, C = 2, 9, 5
    u, w, bias = RNG.normal(size=(b, T, C)), RNG.normal(size=(C, W)), RNG.normal(size=C)
    init = RNG.normal(size=(b, W - 1, C))
    y, fin = oracle.causal_conv1d(u, w, bias, False, init)
    seq = torch.from_numpy(np.concatenate([init, u], 1)).transpose(1, 2)
    ref = torch.nn.functional.conv1d(seq, torch.from_numpy(w)[:, None], torch.from_numpy(bias), groups=C)
    np.testing.assert_allclose(y, ref.transpose(1, 2).numpy(), rtol=1e-13, atol=1e-13)
    np.testing.assert_array_equal(fin, u[:, T - W + 1:])
    ys, _ = oracle.causal_conv1d(u, w, bias, True, init)
    np.testing.assert_allclose(ys, torch.nn.functional.silu(torch.from_numpy(y)).numpy(), rtol=1e-13)


def test_oracle_conv_continues():
    """Two pieces, the second from the first's final states, equal the whole; a piece shorter
    than the window keeps what is older."""
    u, w = RNG.normal(size=(1, 10, 3)), RNG.normal(size=(3, 4))
    whole, fin = oracle.causal_conv1d(u, w)
    state, parts = None, []
    for p, q in ((0, 5), (5, 6), (6, 6), (6, 10)):
        y, state = oracle.causal_conv1d(u[:, p:q], w, initial_states=state)
        parts.append(y)
    np.testing.assert_allclose(np.concatenate(parts, 1), whole, rtol=1e-13)
    np.testing.assert_array_equal(state, fin)


def test_oracle_selective_scan_is_the_layer_where_rates_are_shared():
    """With one step and one rate for all channels and states of a head the diagonal
    recurrence is the layer's (scalar times identity), which has an oracle of its own."""
    b, T, H, P, G, N = 2, 11, 4, 3, 2, 5
    x = RNG.normal(size=(b, T, H, P))
    dt = RNG.uniform(0.01, 0.2, size=(b, T, H))
    A, D = -RNG.uniform(0.5, 8, size=H), RNG.normal(size=H)
    B, C = RNG.normal(size=(b, T, G, N)), RNG.normal(size=(b, T, G, N))
    init = RNG.normal(size=(b, H, P, N))
    y, fin, _ = oracle.recurrence(x, dt, A, B, C, D, init)
    ys, fs = oracle.selective_scan(x.reshape(b, T, H * P), np.repeat(dt, P, 2),
                                   np.repeat(A, P)[:, None] * np.ones(N), B, C, np.repeat(D, P),
                                   initial_states=init.reshape(b, H * P, N))
    np.testing.assert_allclose(ys, y.reshape(b, T, H * P), rtol=1e-11, atol=1e-12)
    np.testing.assert_allclose(fs, fin.reshape(b, H * P, N), rtol=1e-11, atol=1e-12)


def test_oracle_selective_scan_time_invariant_is_a_filter():
    """Constant steps, B and C, N = 1: a first-order IIR filter of u."""
    from scipy.signal import lfilter
    T, a, s = 40, -0.7, 0.3
    u = RNG.normal(size=T)
    y, _ = oracle.selective_scan(u[None, :, None], np.full((1, T, 1), s), np.array([[a]]),
                                 np.full((1, T, 1, 1), 2.0), np.full((1, T, 1, 1), 0.5))
    ref = lfilter([s * 2.0 * 0.5], [1.0, -np.exp(s * a)], u)
    np.testing.assert_allclose(y[0, :, 0], ref, rtol=1e-12)


def test_oracle_selective_steps_and_gate():
    v = np.array([[[-800.0, -20.0, 0.0, 3.0, 800.0]]])
    got = oracle.selective_steps(v, None, True)
    np.testing.assert_allclose(got[0, 0, 1:4], [np.log1p(np.exp(-20.0)), np.log(2.0), np.log1p(np.exp(3.0))],
                               rtol=1e-14)
    assert got[0, 0, 0] == 0.0 and got[0, 0, 4] == 800.0
    one = np.ones((1, 1, 1))
    kw = dict(A=np.array([[-1.0]]), B=one[..., None], C=one[..., None])
    plain, _ = oracle.selective_scan(one, one, **kw)
    gated, _ = oracle.selective_scan(one, one, z=2.0 * one, **kw)
    np.testing.assert_allclose(gated, plain * 2.0 / (1 + np.exp(-2.0)), rtol=1e-14)


# ---- refusals of the C entries ---------------------------------------------

@pytest.fixture(scope="module")
def L():
    from structured_state_space_fwd_b200 import build
    build.build()
    from structured_state_space_fwd_b200 import _lib
    return _lib


class Mem:
    """Real device buffers on a CUDA machine, otherwise placeholder addresses (never read:
    every call here is refused)."""

    def __init__(self, **sizes):
        self.keep, self.at, base = [], {}, 1 << 40
        for k, n in sizes.items():
            if torch.cuda.is_available():
                self.keep.append(torch.zeros(max(n, 16), dtype=torch.uint8, device="cuda"))
                self.at[k] = self.keep[-1].data_ptr()
            else:
                self.at[k], base = base, base + ((n + 4095) // 4096 + 1) * 4096


def conv_shape(L, b=2, T=9, C=12, W=4, split=(6, 4, 2), strides=None, dtype=0, silu=1):
    s = strides or (T * C, C)
    return L.ConvShapeT(b, T, C, W, (ctypes.c_int64 * 3)(*split), L.StridesT(*s), dtype, silu)


def conv_mem(s, nseq=None):
    es = 2 if s.dtype == 1 else 4
    n = s.batch if nseq is None else nseq
    st = n * (s.width - 1) * s.channels * es
    return Mem(u=s.batch * s.seqlen * s.channels * es, weight=s.channels * s.width * 4, bias=s.channels * 4,
               init=st, fin=st, cu=4 * (n + 1),
               **{f"y{i}": s.batch * s.seqlen * s.out_channels[i] * es for i in range(3)})


def call_conv(L, s, m, entry="ssd_causal_conv1d", n=None, **over):
    a = {**m.at, **over}
    lib, sh = L.lib(), ctypes.byref(s) if s is not None else None
    ys = [a["y0"], a["y1"], a["y2"]]
    if entry == "ssd_causal_conv1d":
        return lib.ssd_causal_conv1d(sh, a["u"], a["weight"], a["bias"], a["init"], *ys, a["fin"], None)
    if entry == "ssd_causal_conv1d_varlen":
        return lib.ssd_causal_conv1d_varlen(sh, a["u"], a["weight"], a["bias"], a["cu"], n, a["init"], *ys,
                                            a["fin"], None)
    return lib.ssd_causal_conv1d_step(sh, a["u"], a["weight"], a["bias"], a["fin"], *ys, None)


@pytest.mark.parametrize("kw,code", [
    (dict(b=-1), 1), (dict(T=-1), 1), (dict(C=0, split=(0, 0, 0)), 1), (dict(dtype=2), 1), (dict(silu=2), 1),
    (dict(split=(6, 4, 3)), 1), (dict(split=(14, -2, 0)), 1), (dict(split=(0, 0, 0)), 1),
    (dict(W=0), 1), (dict(W=1), 2), (dict(W=5), 2),
    (dict(strides=(108, -12)), 1), (dict(strides=(-1, 12)), 1), (dict(strides=(1 << 62, 12)), 1),
    (dict(b=1 << 40, T=1 << 40), 2), (dict(C=1 << 50, split=(1 << 50, 0, 0)), 2),
])
@pytest.mark.parametrize("entry", ["ssd_causal_conv1d", "ssd_causal_conv1d_varlen", "ssd_causal_conv1d_step"])
def test_conv_shape_rejections(L, kw, code, entry):
    m = conv_mem(conv_shape(L))
    if entry.endswith("varlen"):
        kw = {"b": 1, **kw}
    assert call_conv(L, conv_shape(L, **kw), m, entry, n=2) == code


def test_conv_null_shape(L):
    m = conv_mem(conv_shape(L))
    for e in ("ssd_causal_conv1d", "ssd_causal_conv1d_varlen", "ssd_causal_conv1d_step"):
        assert call_conv(L, None, m, e, n=1) == 1


@pytest.mark.parametrize("entry", ["ssd_causal_conv1d", "ssd_causal_conv1d_step"])
def test_conv_argument_rejections(L, entry):
    s = conv_shape(L)
    m = conv_mem(s)

    def no(**over):
        assert call_conv(L, s, m, entry, **over) == 1, over
    for k in ("u", "weight", "y0", "y1", "y2"):
        no(**{k: None})
    for k in ("u", "weight", "bias", "y0", "y1", "y2", "fin"):
        no(**{k: m.at[k] + 2})                    # not aligned to fp32
    no(y0=m.at["u"])                              # an output on an input
    no(y1=m.at["u"] + 4 * (2 * 9 * 12 - 1))       # its last element
    no(y2=m.at["weight"])
    no(y1=m.at["y0"])
    no(fin=m.at["y2"])
    no(fin=m.at["u"])
    no(bias=m.at["y0"])
    if entry == "ssd_causal_conv1d":
        no(fin=m.at["init"])
        no(init=m.at["y0"])
        no(init=m.at["init"] + 2)
    else:
        no(fin=None)                              # the state is required
    # a slice: the rows between its own channels belong to the span too
    wide = conv_shape(L, strides=(9 * 100, 100))
    assert call_conv(L, wide, m, entry, y0=m.at["u"] + 4 * 50) == 1


def test_conv_varlen_rejections(L):
    s = conv_shape(L, b=1)
    m = conv_mem(s, 3)

    def code(n=3, sh=s, **over):
        return call_conv(L, sh, m, "ssd_causal_conv1d_varlen", n=n, **over)
    assert code(sh=conv_shape(L, b=2)) == 1
    assert code(n=-1) == 1 and code(n=0) == 1     # tokens, and no document
    assert code(n=(1 << 24) + 1) == 2
    assert code(cu=None) == 1 and code(cu=m.at["cu"] + 2) == 1
    assert code(cu=m.at["y0"]) == 1
    assert code(fin=m.at["init"]) == 1
    assert code(n=0, sh=conv_shape(L, b=1, T=0)) == 0      # nothing to do


def sel_shape(L, b=2, T=9, D=6, G=2, N=4, dtype=0, dt_dtype=None, softplus=0, reserved=0, **strides):
    st = {k: L.StridesT(*strides.get(k, (T * D, D))) for k in ("u", "dt", "z")}
    bc = {k: L.StridesT(*strides.get(k, (T * G * N, G * N))) for k in ("B", "C")}
    return L.SelectiveShapeT(b, T, D, G, N, st["u"], st["dt"], st["z"], bc["B"], bc["C"], dtype,
                             dtype if dt_dtype is None else dt_dtype, softplus, reserved)


def sel_mem(n=2):
    rows, bc, st = 2 * 9 * 6 * 4, 2 * 9 * 2 * 4 * 4, n * 6 * 4 * 4
    return Mem(u=rows, dt=rows, A=6 * 4 * 4, B=bc, C=bc, D=24, z=rows, bias=24, init=st, y=rows, fin=st,
               cu=4 * (n + 1))


def call_sel(L, s, m, entry="ssd_selective_scan", n=None, **over):
    a = {**m.at, **over}
    lib, sh = L.lib(), ctypes.byref(s) if s is not None else None
    ins = [a[k] for k in ("u", "dt", "A", "B", "C", "D", "z", "bias")]
    if entry == "ssd_selective_scan":
        return lib.ssd_selective_scan(sh, *ins, a["init"], a["y"], a["fin"], None)
    if entry == "ssd_selective_scan_varlen":
        return lib.ssd_selective_scan_varlen(sh, *ins, a["cu"], n, a["init"], a["y"], a["fin"], None)
    return lib.ssd_selective_step(sh, *ins, a["fin"], a["y"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(b=-1), 1), (dict(T=-1), 1), (dict(D=0), 1), (dict(G=4), 1), (dict(G=0), 1), (dict(N=0), 1),
    (dict(dtype=5), 1), (dict(dtype=0, dt_dtype=1), 1), (dict(softplus=2), 1), (dict(reserved=1), 1),
    (dict(N=257), 2), (dict(u=(-1, 6)), 1), (dict(dt=(54, -6)), 1), (dict(B=(1 << 62, 8)), 1),
    (dict(C=(0, -1)), 1), (dict(z=(0, -1)), 1), (dict(T=1 << 52), 2), (dict(T=1 << 31), 2),
    (dict(dt=(1 << 40, 1 << 31)), 2), (dict(z=(1 << 40, 1 << 31)), 2), (dict(D=1 << 31, G=1), 2),
])
@pytest.mark.parametrize("entry", ["ssd_selective_scan", "ssd_selective_scan_varlen", "ssd_selective_step"])
def test_selective_shape_rejections(L, kw, code, entry):
    if entry.endswith("varlen"):
        kw = {"b": 1, **kw}
    assert call_sel(L, sel_shape(L, **kw), sel_mem(), entry, n=2) == code


@pytest.mark.parametrize("entry", ["ssd_selective_scan", "ssd_selective_step"])
def test_selective_argument_rejections(L, entry):
    s, m = sel_shape(L), sel_mem()

    def no(**over):
        assert call_sel(L, s, m, entry, **over) == 1, over
    assert call_sel(L, None, m, entry) == 1
    for k in ("u", "dt", "A", "B", "C", "y"):
        no(**{k: None})
    for k in ("u", "dt", "A", "B", "C", "D", "z", "bias", "y", "fin"):
        no(**{k: m.at[k] + 2})
    for k in ("u", "dt", "A", "B", "C", "D", "z", "bias"):
        no(y=m.at[k])
        no(fin=m.at[k])
    no(fin=m.at["y"])
    if entry == "ssd_selective_scan":
        no(fin=m.at["init"])
        no(y=m.at["init"])
    else:
        no(fin=None)


def test_selective_varlen_rejections(L):
    s, m = sel_shape(L, b=1), sel_mem(3)

    def code(n=3, sh=s, **over):
        return call_sel(L, sh, m, "ssd_selective_scan_varlen", n=n, **over)
    assert code(sh=sel_shape(L, b=2)) == 1
    assert code(n=-1) == 1 and code(n=0) == 1 and code(n=(1 << 24) + 1) == 2
    assert code(cu=None) == 1 and code(cu=m.at["cu"] + 1) == 1
    assert code(cu=m.at["y"]) == 1
    assert code(n=0, sh=sel_shape(L, b=1, T=0)) == 0


# ---- refusals of the binding -----------------------------------------------

def test_binding_needs_cuda_tensors():
    import structured_state_space_fwd_b200 as ssd
    u, w = torch.zeros(1, 3, 4), torch.zeros(4, 4)
    with pytest.raises(ValueError, match="CUDA"):
        ssd.ssd_causal_conv1d(u, w)
    with pytest.raises(ValueError, match="CUDA"):
        ssd.ssd_causal_conv1d_step(u, w, None, torch.zeros(1, 3, 4))
    with pytest.raises(ValueError, match="CUDA"):
        ssd.ssd_selective_scan(u, u, -torch.ones(4, 2), torch.zeros(1, 3, 1, 2), torch.zeros(1, 3, 1, 2))
    with pytest.raises(ValueError, match="CUDA"):
        ssd.ssd_selective_step(u, u, -torch.ones(4, 2), torch.zeros(1, 3, 1, 2), torch.zeros(1, 3, 1, 2), None,
                               torch.zeros(1, 4, 2))


def test_binding_checks_inputs():
    """The checks of one input: type, shape, device, contiguous channels, strides."""
    from structured_state_space_fwd_b200 import _block as B
    cpu = torch.device("cpu")
    t = torch.zeros(2, 3, 8)
    assert B._in(t[..., 2:6], "t", (2, 3, 4), torch.float32, cpu) is not None
    with pytest.raises(ValueError, match="required"):
        B._in(None, "t", (2, 3, 8), torch.float32, cpu)
    with pytest.raises(TypeError):
        B._in(t, "t", (2, 3, 8), torch.bfloat16, cpu)
    with pytest.raises(ValueError, match="must be"):
        B._in(t, "t", (2, 3, 7), torch.float32, cpu)
    with pytest.raises(ValueError, match="on cuda"):
        B._in(t, "t", (2, 3, 8), torch.float32, torch.device("cuda:0"))
    with pytest.raises(ValueError, match="contiguous"):
        B._in(t[..., ::2], "t", (2, 3, 4), torch.float32, cpu)
    with pytest.raises(ValueError, match="contiguous"):
        B._in(t.transpose(1, 2), "t", (2, 8, 3), torch.float32, cpu)
    four = torch.zeros(2, 3, 20)[..., 4:16].unflatten(-1, (3, 4))
    assert B._in(four, "t", (2, 3, 3, 4), torch.float32, cpu, 2) is not None
    with pytest.raises(ValueError, match="contiguous"):
        B._in(torch.zeros(2, 3, 3, 8)[..., :4], "t", (2, 3, 3, 4), torch.float32, cpu, 2)
    with pytest.raises(ValueError, match="contiguous"):
        B._whole(t[..., 2:6], "t", (2, 3, 4), torch.float32, cpu)


@pytest.mark.parametrize("cu", [[0, 3], [1, 5], [0, 4, 2, 5], [0], [0, 6]])
def test_binding_checks_host_offsets(cu):
    from structured_state_space_fwd_b200 import _block as B
    with pytest.raises(ValueError):
        B._offsets(cu, 5, torch.device("cpu"))
    with pytest.raises(ValueError):
        B._offsets(None, 5, torch.device("cpu"))
    assert B._offsets([0, 2, 2, 5], 5, torch.device("cpu")).tolist() == [0, 2, 2, 5]
