"""The operators together, as a block uses them: convolution, layer or selective scan, gate -
a prompt, then tokens from the carried states, against the fp64 oracle's chain.

The layer's bars hold (max|err| / max|ref| <= 5e-3 for bf16 storage, 1e-5 for fp32), each taken on
one operator's output with the operator's own (rounded) inputs, so that they do not add up.
"""
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu

TOL = {torch.bfloat16: 5e-3, torch.float32: 1e-5}


@pytest.fixture(scope="module")
def ssd(cuda_device):
    from structured_state_space_fwd_b200 import build
    build.build()
    import structured_state_space_fwd_b200 as m
    return m


def near(got, ref, t):
    err = oracle.rel_err(got.double().cpu(), ref)
    assert err <= TOL[t], f"rel err {err:.2e}"


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_layer_block(ssd, dtype):
    """x, B and C out of one slice of a projection through the convolution's split outputs into
    ssd_fwd (prompt) and ssd_step (tokens), then the gate and norm."""
    b, T0, T1, H, P, G, N, W = 2, 200, 5, 4, 64, 1, 128, 4
    d_in, bc = H * P, G * N
    C, T = d_in + 2 * bc, T0 + T1
    g = torch.Generator().manual_seed(0)
    proj = torch.randn(b, T, d_in + C + H, generator=g).to(dtype)       # z | x B C | dt
    w, bias = torch.randn(C, W, generator=g) * 0.5, torch.randn(C, generator=g) * 0.1
    A, D = -(torch.rand(H, generator=g) * 8 + 0.5), torch.randn(H, generator=g)
    dt = torch.nn.functional.softplus(proj[..., d_in + C:].float() - 3)
    nw = torch.rand(d_in, generator=g) + 0.5
    dev = [t.cuda() for t in (proj, w, bias, A, D, dt, nw)]
    pr, wd, bd, Ad, Dd, dtd, nwd = dev
    z, u = pr[..., :d_in], pr[..., d_in:d_in + C]
    split = (d_in, bc, bc)

    (x, B, Cc), conv = ssd.ssd_causal_conv1d(u[:, :T0], wd, bd, split=split, return_final_states=True)
    y, state = ssd.ssd_fwd(x.view(b, T0, H, P), dtd[:, :T0].contiguous(), Ad, B.view(b, T0, G, N),
                           Cc.view(b, T0, G, N), Dd, return_final_states=True)
    xs, Bs, Cs, ys = [x], [B], [Cc], [y]
    for t in range(T0, T):
        x, B, Cc = ssd.ssd_causal_conv1d_step(u[:, t], wd, bd, conv, split=split)
        y = ssd.ssd_step(x.view(b, H, P), dtd[:, t].contiguous(), Ad, B.view(b, G, N), Cc.view(b, G, N), Dd, state)
        for lst, v in ((xs, x), (Bs, B), (Cs, Cc), (ys, y)):
            lst.append(v[:, None])
    x, B, Cc, y = (torch.cat(v, 1) for v in (xs, Bs, Cs, ys))
    out = ssd.ssd_gated_rmsnorm(y, z.contiguous().view(b, T, H, P), nwd)

    cy, cs = oracle.causal_conv1d(u.cpu(), w, bias)
    near(torch.cat([x, B, Cc], -1), cy, dtype)
    near(conv, cs, torch.float32)
    ry, rs, _ = oracle.recurrence(x.view(b, T, H, P).cpu(), dt, A, B.view(b, T, G, N).cpu(),
                                  Cc.view(b, T, G, N).cpu(), D)
    near(y, ry, dtype)
    near(state, rs, dtype)
    near(out, oracle.gated_rmsnorm(y.cpu(), z.cpu().reshape(b, T, H, P), nw, d_in, 1e-5), dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_selective_block(ssd, dtype):
    """The convolution's output through a projection to dt, B and C and into the gated selective
    scan: a prompt, then tokens in a captured graph."""
    b, T0, T1, Dc, N, R, W = 2, 150, 6, 96, 16, 8, 4
    T = T0 + T1
    g = torch.Generator().manual_seed(1)
    xz = torch.randn(b, T, 2 * Dc, generator=g).to(dtype).cuda()
    w, bias = (torch.randn(Dc, W, generator=g) * 0.5).cuda(), (torch.randn(Dc, generator=g) * 0.1).cuda()
    px = (torch.randn(Dc, R + 2 * N, generator=g) / Dc ** 0.5).to(dtype).cuda()
    pdt = (torch.randn(R, Dc, generator=g) / R ** 0.5).to(dtype).cuda()
    A = -(torch.rand(Dc, N, generator=g) * 15 + 0.5).cuda()
    D, dt_bias = torch.randn(Dc, generator=g).cuda(), (torch.rand(Dc, generator=g) * 3 - 5).cuda()

    def inputs(x):
        p = x @ px
        return p[..., :R] @ pdt, p[..., R:R + N].unflatten(-1, (1, N)), p[..., R + N:].unflatten(-1, (1, N))
    kw = dict(dt_bias=dt_bias, dt_softplus=True)
    x, conv = ssd.ssd_causal_conv1d(xz[:, :T0, :Dc], w, bias, return_final_states=True)
    dt, B, C = inputs(x)
    y, state = ssd.ssd_selective_scan(x, dt, A, B, C, D, z=xz[:, :T0, Dc:], return_final_states=True, **kw)

    tok = xz[:, :1].clone()
    s0, c0 = state.clone(), conv.clone()

    def step():
        x = ssd.ssd_causal_conv1d_step(tok[..., :Dc], w, bias, conv)
        dt, B, C = inputs(x)
        return x, dt, B, C, ssd.ssd_selective_step(x, dt, A, B, C, D, state, z=tok[..., Dc:], **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    state.copy_(s0)
    conv.copy_(c0)
    rows = [[x], [dt], [B], [C], [y]]
    for t in range(T0, T):
        tok.copy_(xz[:, t:t + 1])
        graph.replay()
        for lst, v in zip(rows, held):
            lst.append(v.clone())
    x, dt, B, C, y = (torch.cat(v, 1) for v in rows)

    cy, cs = oracle.causal_conv1d(xz[..., :Dc].cpu(), w.cpu(), bias.cpu())
    near(x, cy, dtype)
    near(conv, cs, torch.float32)
    ry, rs = oracle.selective_scan(x.cpu(), dt.cpu(), A.cpu(), B.cpu(), C.cpu(), D.cpu(), z=xz[..., Dc:].cpu(),
                                   dt_bias=dt_bias.cpu(), dt_softplus=True)
    near(y, ry, dtype)
    near(state, rs, torch.float32)


def test_packed_block(ssd):
    """A pack through the convolution and the layer's packed form, and through the selective scan."""
    cu, H, P, N, W = [0, 130, 131, 131, 400], 2, 64, 64, 4
    T, d_in, n = cu[-1], H * P, 4
    g = torch.Generator().manual_seed(2)
    C = d_in + 2 * N
    u = torch.randn(1, T, C, generator=g).bfloat16()
    w = torch.randn(C, W, generator=g) * 0.5
    dt = torch.rand(1, T, H, generator=g) * 0.1
    A = -(torch.rand(H, generator=g) * 8 + 0.5)
    dcu = torch.tensor(cu, dtype=torch.int32, device="cuda")
    (x, B, Cc), conv = ssd.ssd_causal_conv1d_varlen(u.cuda(), w.cuda(), cu_seqlens=dcu, split=(d_in, N, N),
                                                    return_final_states=True)
    args = (x.view(1, T, H, P), dt.cuda(), A.cuda(), B.view(1, T, 1, N), Cc.view(1, T, 1, N))
    y, fin = ssd.ssd_fwd_varlen(*args, cu_seqlens=dcu, return_final_states=True)
    ry, rf = oracle.recurrence_varlen(*(t.cpu() for t in args), cu_seqlens=cu)
    # The layer's tensor-core kernel rounds its operands to bf16 (half a step: 2^-8 of the value): the
    # decayed x and the masked scores of a tile, or the decayed x and the state, then y. Behind SiLU, B
    # and C have a mean, sums of them cancel, and an error of 2 * 2^-8 of the summed magnitudes (the
    # recurrence on absolute values) can pass 5e-3 of the largest |y|; the final states have one such
    # rounding. 2^-12 of the magnitudes covers the fp32 sums (at most 400 terms, 2^-24 each, and the
    # decays' exponentials).
    my, mf = oracle.recurrence_varlen(*(t.float().cpu().abs() if i != 2 else t.cpu() for i, t in enumerate(args)),
                                      cu_seqlens=cu)
    assert (abs(y.double().cpu().numpy() - ry) <= (2 * 2 ** -8 + 2 ** -12) * my + 2 ** -8 * abs(ry) + 1e-30).all()
    assert (abs(fin.double().cpu().numpy() - rf) <= (2 ** -8 + 2 ** -12) * mf + 1e-30).all()
    # the selective scan with the layer's rates, repeated over channels and states
    ys, fs = ssd.ssd_selective_scan_varlen(
        x, args[1].repeat_interleave(P, 2), args[2].repeat_interleave(P)[:, None].repeat(1, N), args[3], args[4],
        cu_seqlens=dcu, return_final_states=True)
    near(ys.view(1, T, H, P), ry, torch.bfloat16)
    near(fs.view(n, H, P, N), rf, torch.float32)
    for k, (p, q) in enumerate(zip(cu, cu[1:])):
        cy, cs = oracle.causal_conv1d(u[:, p:q], w)
        near(torch.cat([x, B, Cc], -1)[:, p:q], cy, torch.bfloat16) if q > p else None
        near(conv[k:k + 1], cs, torch.float32)
