"""The short causal convolution (prompts, packed documents, single tokens) against the fp64
oracle, element by element.

Bounds, in units of e = 2^-24 (half a step of fp32). v is a chain of W fused multiply-adds from
the bias: off by at most W e S, S = |bias| + sum |w u|. SiLU's slope is below 1.1. SiLU itself
takes the exponent v log2(e) (one rounding of a product with a rounded constant: 2 e |v| of the
exponential), 2^x (2 ulp = 4 e), 1 + x (1 e), 1/x (1 ulp = 2 e) and a product (1 e), together
below (2 |v| + 8) e of the result. Then one rounding to the storage type, eps/2 of the value.
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


def inputs(b, T, C, W, dtype, nseq=None, seed=0, bias=True, states=True):
    g = torch.Generator().manual_seed(seed)
    n = b if nseq is None else nseq
    d = {"u": torch.randn(b, T, C, generator=g).to(TYPES[dtype]),
         "weight": torch.randn(C, W, generator=g) * 0.5,
         "bias": torch.randn(C, generator=g) if bias else None,
         "initial_states": torch.randn(n, W - 1, C, generator=g).to(TYPES[dtype]) if states else None}
    return d


def cuda(d):
    return {k: v.cuda() if v is not None else None for k, v in d.items()}


def reference(d, silu, cu=None):
    """(y, its bound before rounding, final states), documents one after another."""
    u = d["u"].double().numpy()
    w, W = d["weight"].double().numpy(), d["weight"].shape[1]
    init = d["initial_states"]
    bias = d["bias"]
    spans = [(slice(None), 0, u.shape[1], slice(None))] if cu is None else \
        [(slice(0, 1), p, q, slice(k, k + 1)) for k, (p, q) in enumerate(zip(cu, cu[1:]))]
    y, S, V, fin = np.zeros(u.shape), np.zeros(u.shape), np.zeros(u.shape), []
    for rows, p, q, seq in spans:
        st = init[seq] if init is not None else None
        y[rows, p:q], f = oracle.causal_conv1d(u[rows, p:q], w, bias, silu, st)
        V[rows, p:q], _ = oracle.causal_conv1d(u[rows, p:q], w, bias, False, st)
        S[rows, p:q], _ = oracle.causal_conv1d(np.abs(u[rows, p:q]), np.abs(w),
                                               bias.abs() if bias is not None else None, False,
                                               st.float().abs() if st is not None else None)
        fin.append(f)
    bound = W * E32 * S
    if silu:
        bound = 1.1 * bound + (2 * np.abs(V) + 8) * E32 * np.abs(y)
    return y, bound, np.concatenate(fin)


def check(got, ref, bound, dtype):
    t = TYPES[dtype]
    got = got.double().cpu().numpy()
    lim = bound + (np.abs(ref) + bound) * torch.finfo(t).eps / 2 + torch.finfo(t).tiny
    worst = np.max(np.abs(got - ref) / lim) if ref.size else 0.0
    assert worst <= 1.0, f"{worst:.3f} of the bound"


def parts(ys, sizes):
    return torch.cat(list(ys), -1) if sizes is not None else ys


SHAPES = [
    # b, T, C, W, split
    (2, 37, 64, 4, None), (1, 1, 8, 4, None), (1, 2, 16, 3, None), (3, 3, 24, 4, (8, 8, 8)),
    (2, 130, 40, 2, (16, 24)), (1, 257, 264, 4, (248, 8, 8)), (2, 65, 7, 4, (1, 6)),
    (1, 19, 1, 2, None), (2, 33, 1091, 3, None), (1, 700, 300, 4, (100, 100, 100)),
    (1, 9, 12, 4, (4, 0, 8)), (1, 9, 16, 4, (0, 8, 8)), (5, 0, 16, 4, None), (0, 5, 16, 4, None),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("b,T,C,W,split", SHAPES)
def test_conv_shapes(ssd, b, T, C, W, split, dtype):
    for silu, states in ((True, False), (False, True)):
        d = inputs(b, T, C, W, dtype, seed=T, states=states, bias=silu)
        y, fin = ssd.ssd_causal_conv1d(**cuda(d), silu=silu, split=split, return_final_states=True)
        ref, bound, f = reference(d, silu)
        if split is not None:
            assert [p.shape[-1] for p in y] == list(split) and all(p.is_contiguous() for p in y)
        check(parts(y, split), ref, bound, dtype)
        assert np.array_equal(fin.double().cpu().numpy(), f)      # copies: no rounding


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lo,pad,b", [(8, 24, 3), (3, 10, 2), (16, 1, 1)])
def test_conv_slices_of_wider_rows(ssd, dtype, lo, pad, b):
    """u inside a projection's rows, 16-byte aligned and not; rows repeated by a stride of 0."""
    C, T, W = 48, 70, 4
    wide = torch.randn(b, T, lo + C + pad, generator=torch.Generator().manual_seed(3)).to(TYPES[dtype])
    d = inputs(b, T, C, W, dtype, seed=1)
    d["u"] = wide[..., lo:lo + C]
    dev = cuda(d)
    dev["u"] = wide.cuda()[..., lo:lo + C]
    assert not dev["u"].is_contiguous()
    ref, bound, _ = reference(d, True)
    check(ssd.ssd_causal_conv1d(**dev), ref, bound, dtype)
    d["u"] = wide[:, :1, lo:lo + C].expand(b, T, C)
    dev["u"] = wide.cuda()[:, :1, lo:lo + C].expand(b, T, C)
    ref, bound, _ = reference(d, True)
    check(ssd.ssd_causal_conv1d(**dev), ref, bound, dtype)


DOCS = [
    [0, 5], [0, 0, 5], [0, 1, 2, 3, 3, 3, 10], [0, 64, 128, 200, 200], [0, 63, 64, 65, 300, 301, 517],
    [0, 0, 0], list(range(0, 91)), [0, 2, 2, 4, 5, 130],
]


@pytest.mark.parametrize("dtype,C", [("bf16", 64), ("f32", 13)])
@pytest.mark.parametrize("cu", DOCS)
def test_conv_packed(ssd, cu, dtype, C):
    for W, states in ((4, True), (2, True), (4, False)):
        d = inputs(1, cu[-1], C, W, dtype, nseq=len(cu) - 1, seed=len(cu), states=states)
        ref, bound, f = reference(d, True, cu)
        dev = cuda(d)
        for offsets in (cu, torch.tensor(cu, dtype=torch.int32, device="cuda")):
            y, fin = ssd.ssd_causal_conv1d_varlen(**dev, cu_seqlens=offsets, return_final_states=True)
            check(y, ref, bound, dtype)
            assert np.array_equal(fin.double().cpu().numpy(), f)


@pytest.mark.parametrize("C,dtype", [(8192, "bf16"), (2047, "f32")])
def test_conv_long_runs(ssd, C, dtype):
    """Enough rows for runs of 64 tokens a warp: a batch, and a pack whose documents start and end
    everywhere in them, one after another, empty and single ones among them."""
    cu = [0, 3, 64, 64, 65, 130, 191, 193, 700, 1024, 1087, 1088, 1100, 2500, 4101]
    T = cu[-1] if C > 4096 else 16 * cu[-1]
    cu = [c * T // cu[-1] for c in cu]
    d = inputs(1, T, C, 4, dtype, nseq=len(cu) - 1, seed=1)
    ref, bound, f = reference(d, True, cu)
    y, fin = ssd.ssd_causal_conv1d_varlen(**cuda(d), cu_seqlens=cu, return_final_states=True)
    check(y, ref, bound, dtype)
    assert np.array_equal(fin.double().cpu().numpy(), f)
    d["initial_states"] = d["initial_states"][:1]
    whole = ssd.ssd_causal_conv1d(**cuda(d))
    # a document's tokens past its first three see no boundary
    for p, q in zip(cu, cu[1:]):
        assert torch.equal(whole[:, p + 3:q], y[:, p + 3:q])


def test_conv_rows_behind_the_last_document_stay(ssd):
    d = inputs(1, 200, 64, 4, "bf16", nseq=3, seed=5)
    cu = [0, 40, 41, 131]
    short = dict(d, u=d["u"][:, :131])
    ref, bound, f = reference(short, True, cu)
    out = torch.full((1, 200, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    _, fin = ssd.ssd_causal_conv1d_varlen(**cuda(d), cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"),
                                          out=out, return_final_states=True)
    check(out[:, :131], ref, bound, "bf16")
    assert bool((out[:, 131:] == 7.0).all())
    assert np.array_equal(fin.double().cpu().numpy(), f)


@pytest.mark.parametrize("cu", [[-5, 3, 1000], [3, 1, 90, 20], [90, 90, 90], [5, 7], [-9, -3]])
def test_conv_malformed_offsets_stay_inside(ssd, cu):
    """Whatever the list says, guard rows around every tensor keep their values."""
    T, C, W, n = 90, 64, 4, len(cu) - 1
    guard = torch.full((T + 64, C), 3.0, device="cuda")
    states = torch.full((n * (W - 1) + 64, C), 5.0, device="cuda")
    d = cuda(inputs(1, T, C, W, "f32", nseq=n, seed=2))
    ssd.ssd_causal_conv1d_varlen(**d, cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"),
                                 out=guard[32:32 + T][None],
                                 final_states=states[32:32 + n * (W - 1)].view(n, W - 1, C))
    torch.cuda.synchronize()
    assert bool((guard[:32] == 3).all()) and bool((guard[32 + T:] == 3).all())
    assert bool((states[:32] == 5).all()) and bool((states[32 + n * (W - 1):] == 5).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("b,T,C,W,split", [(3, 1, 64, 4, (32, 16, 16)), (1, 1, 13, 4, None), (2, 2, 24, 4, None),
                                           (2, 7, 16, 3, None), (129, 1, 40, 2, (8, 32)), (2, 0, 16, 4, None),
                                           (0, 1, 16, 4, None)])
def test_conv_step(ssd, b, T, C, W, split, dtype):
    d = inputs(b, T, C, W, dtype, seed=b + T)
    ref, bound, f = reference(d, True)
    dev = cuda(d)
    state = dev.pop("initial_states")
    y = ssd.ssd_causal_conv1d_step(**dev, state=state, split=split)
    check(parts(y, split), ref, bound, dtype)
    assert np.array_equal(state.double().cpu().numpy(), f)


def test_conv_step_one_token_form(ssd):
    d = cuda(inputs(3, 1, 32, 4, "bf16", seed=4))
    s1, s2 = d["initial_states"].clone(), d["initial_states"].clone()
    a = ssd.ssd_causal_conv1d_step(d["u"], d["weight"], d["bias"], s1, split=(24, 8))
    out = (torch.empty(3, 24, dtype=torch.bfloat16, device="cuda"),
           torch.empty(3, 8, dtype=torch.bfloat16, device="cuda"))
    b = ssd.ssd_causal_conv1d_step(d["u"][:, 0], d["weight"], d["bias"], s2, split=(24, 8), out=out)
    assert all(torch.equal(p[:, 0], q) and q.shape == (3, p.shape[-1]) for p, q in zip(a, b))
    assert torch.equal(s1, s2) and b[0].data_ptr() == out[0].data_ptr()


def test_conv_prompt_then_tokens(ssd):
    """A prompt in two calls, then tokens, equals one pass over all of it, bit for bit."""
    d = cuda(inputs(2, 100, 72, 4, "bf16", seed=8))
    whole, last = ssd.ssd_causal_conv1d(**d, return_final_states=True)
    kw = dict(weight=d["weight"], bias=d["bias"])
    y0, s = ssd.ssd_causal_conv1d(d["u"][:, :61], initial_states=d["initial_states"], return_final_states=True, **kw)
    y1, s = ssd.ssd_causal_conv1d(d["u"][:, 61:90], initial_states=s, return_final_states=True, **kw)
    ys = [y0, y1] + [ssd.ssd_causal_conv1d_step(d["u"][:, t], state=s, **kw)[:, None] for t in range(90, 100)]
    assert torch.equal(torch.cat(ys, 1), whole) and torch.equal(s, last)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_conv_special_values(ssd, dtype):
    """Infinities and NaN reach the W outputs whose window holds them and no other, and the
    activation of very large and very small values keeps its limits."""
    d = inputs(1, 40, 16, 4, dtype, seed=9, states=False, bias=False)
    d["weight"] = d["weight"].abs() + 0.1
    d["u"][0, 10, 3] = float("nan")
    d["u"][0, 20, 5] = float("inf")
    d["u"][0, 30, 7] = 3e38
    d["u"][0, 36, 2] = -3e38
    y = ssd.ssd_causal_conv1d(**cuda(d)).float().cpu()
    bad = ~torch.isfinite(y)
    expect = torch.zeros_like(bad)
    expect[0, 10:14, 3] = True
    expect[0, 20:24, 5] = True
    big = torch.isinf(torch.nn.functional.conv1d(
        d["u"].float().transpose(1, 2), d["weight"][:, None], groups=16, padding=3)[..., :40].transpose(1, 2))
    expect |= big
    # a sum past -3e38 is -inf, whose SiLU is NaN as the formula's
    assert torch.equal(bad, expect)
    assert torch.isnan(y[0, 10:14, 3]).all() and (y[0, 20:24, 5] == float("inf")).all()


def test_conv_past_32_bits(ssd):
    """Element offsets above 2^31 in the input, in the output and between batch rows."""
    C, T = 8192, (1 << 18) + 5
    u = torch.zeros(1, T, C, dtype=torch.bfloat16, device="cuda")
    d = inputs(1, 16, C, 4, "bf16", seed=6, states=False)
    u[0, -16:] = d["u"][0].cuda()
    y, fin = ssd.ssd_causal_conv1d(u, d["weight"].cuda(), d["bias"].cuda(), return_final_states=True)
    ref, bound, f = reference(d, True)
    check(y[:, -16:], ref, bound, "bf16")
    assert np.array_equal(fin.double().cpu().numpy(), f)
    del y
    rows = u.view(-1).as_strided((2, 16, C), ((T - 16) * C, C, 1))      # the zeros, then the last rows
    y = ssd.ssd_causal_conv1d(rows, d["weight"].cuda(), d["bias"].cuda())
    check(y[1:], ref, bound, "bf16")


def test_conv_streams_and_graphs(ssd):
    """A call on a side stream, and two captured calls replayed with new inputs."""
    d = cuda(inputs(2, 50, 64, 4, "bf16", seed=1))
    ref = ssd.ssd_causal_conv1d(**d)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = ssd.ssd_causal_conv1d(**d, stream=side)
    side.synchronize()
    assert torch.equal(y, ref)
    state = d["initial_states"].clone()
    tok, out = d["u"][:, :1].clone(), torch.empty_like(d["u"][:, :1])
    kw = dict(weight=d["weight"], bias=d["bias"])
    ssd.ssd_causal_conv1d_step(tok, state=state.clone(), out=out, **kw)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ssd.ssd_causal_conv1d_step(tok, state=state, out=out, **kw)
    state.copy_(d["initial_states"])
    for t in range(50):
        tok.copy_(d["u"][:, t:t + 1])
        g.replay()
        assert torch.equal(out, ref[:, t:t + 1])


def test_conv_binding_refusals(ssd):
    d = cuda(inputs(2, 6, 8, 4, "f32"))
    u, w = d["u"], d["weight"]
    for bad, err in ((dict(weight=w.bfloat16()), TypeError), (dict(weight=w[:7]), ValueError),
                     (dict(weight=w[:, 0]), ValueError), (dict(bias=w[:, 0]), ValueError),
                     (dict(split=(4, 5)), ValueError), (dict(split=(2, 2, 2, 2)), ValueError),
                     (dict(initial_states=u), ValueError), (dict(u=u.half()), TypeError),
                     (dict(u=u.transpose(1, 2)), ValueError), (dict(u=u[0]), ValueError),
                     (dict(initial_states=d["initial_states"].bfloat16()), TypeError),
                     (dict(out=torch.empty_like(u)[:1]), ValueError),
                     (dict(out=u), ssd.SSDError)):
        with pytest.raises(err):
            ssd.ssd_causal_conv1d(**{**d, **bad})
    with pytest.raises(ssd.SSDError, match="UNSUPPORTED"):
        ssd.ssd_causal_conv1d(u, torch.zeros(8, 5, device="cuda"))
    with pytest.raises(ValueError, match="batch 1"):
        ssd.ssd_causal_conv1d_varlen(u, w, cu_seqlens=[0, 6])
    with pytest.raises(ValueError):
        ssd.ssd_causal_conv1d_varlen(u[:1], w, cu_seqlens=torch.tensor([0, 6], device="cuda"))
    with pytest.raises(ValueError):
        ssd.ssd_causal_conv1d_step(u, w, None, d["initial_states"][:1])
