"""The block operators next to the SSD layer, as measured work: the short causal convolution
and the selective scan, for prompts, packed documents and single tokens.

`own` False: the plain forms, elementary torch operations in 32 bits. `own` True: the calls a
user makes of structured_state_space_fwd_b200.
"""
import math
import random

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_LARGEST_CONV = 8 * 2048 * 5376            # elements of a convolution's input
_LARGEST_SCAN = 4 * 2048 * 5120 * 16       # (token, channel, state) triples of a scan
_LARGEST_STEP = 128 * 5120 * 16            # (sequence, channel, state) triples of a step


def _conv(name, b, T, split, width, dtype, silu=True, sliced=False, states=False, docs=0, step=False):
    return {"name": name, "op": "conv_step" if step else "conv", "b": b, "T": T, "c0": split[0], "c1": split[1],
            "c2": split[2], "width": width, "dtype": dtype, "silu": silu, "sliced": sliced, "states": states,
            "docs": docs}


def _scan(name, b, T, channels, groups, dstate, dtype, dt="", softplus=True, gate=True, sliced=False,
          states=False, docs=0, step=False):
    return {"name": name, "op": "scan_step" if step else "scan", "b": b, "T": T, "channels": channels,
            "groups": groups, "dstate": dstate, "dtype": dtype, "dt": dt or dtype, "softplus": softplus,
            "gate": gate, "sliced": sliced, "states": states, "docs": docs}


def listed():
    return [
        # the convolution of the 2.7B layer's prompt: x, B and C out of a slice of the input projection
        _conv("conv_layer_bf16", 8, 2048, (5120, 128, 128), 4, "bf16", sliced=True),
        # odd sizes in fp32: three taps, no activation, continued from a state
        _conv("conv_odd_f32", 3, 1021, (1091, 0, 0), 3, "f32", silu=False, states=True),
        # a pack of documents of mixed lengths, each continued from its own state
        _conv("conv_packed_bf16", 1, 16384, (5120, 128, 128), 4, "bf16", sliced=True, states=True, docs=16),
        # one decoding step of 128 sequences at the 2.7B layer's width
        _conv("conv_step_b128_bf16", 128, 1, (5120, 128, 128), 4, "bf16", sliced=True, step=True),
        # one decoding step of a single sequence: latency
        _conv("conv_step_b1_f32", 1, 1, (2048, 0, 0), 4, "f32", step=True),
        # a prompt through a layer of 5120 channels, B, C and the gate sliced out of projections
        _scan("scan_layer_bf16", 4, 2048, 5120, 1, 16, "bf16", sliced=True, states=True),
        # one long sequence in fp32, continued from a state: little to run side by side
        _scan("scan_long_f32", 1, 16384, 2048, 1, 16, "f32", states=True),
        # more states and grouped B and C
        _scan("scan_groups_n64_bf16", 2, 1024, 2048, 8, 64, "bf16", dt="f32", softplus=False, gate=False),
        # odd sizes everywhere
        _scan("scan_odd_f32", 2, 777, 515, 1, 5, "f32", softplus=False, states=True),
        # a pack of documents of mixed lengths
        _scan("scan_packed_bf16", 1, 8192, 2048, 1, 16, "bf16", sliced=True, states=True, docs=16),
        # one decoding step of 128 sequences: a stream of the states
        _scan("step_b128_bf16", 128, 1, 5120, 1, 16, "bf16", sliced=True, step=True),
        # one decoding step of a single sequence: latency
        _scan("step_b1_f32", 1, 1, 2048, 1, 16, "f32", step=True),
    ]


def _spread(rng, lo, hi):
    """A whole number from lo to hi, even over its logarithm; often a multiple of 8 or 64."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    m = rng.choice((1, 8, 64))
    return min(hi, max(lo, v - v % m))


def draw(rng):
    op = rng.choice(("conv", "conv", "scan", "scan", "scan", "conv_step", "scan_step"))
    dtype = rng.choice(("bf16", "bf16", "f32"))
    docs = rng.choice((0, 0, rng.randint(1, 40))) if op in ("conv", "scan") else 0
    b = _spread(rng, 1, 256) if op.endswith("step") else (1 if docs else rng.randint(1, 8))
    T = rng.choice((1, 1, 1, 2, 3, 5)) if op.endswith("step") else _spread(rng, 1, 16384)
    if op.startswith("conv"):
        c = [_spread(rng, 16, 6144), 0, 0]
        if rng.random() < 0.5:
            c[1] = c[2] = _spread(rng, 1, 512)
        T = min(T, max(1, _LARGEST_CONV // (b * sum(c))))
        case = _conv("", b, T, c, rng.randint(2, 4), dtype, silu=rng.random() < 0.8, sliced=rng.random() < 0.5,
                     states=rng.random() < 0.5, docs=docs, step=op == "conv_step")
    else:
        G = rng.choice((1, 1, 1, 2, 4, 8))
        N = rng.choice((16, 16, rng.randint(1, 32), rng.randint(1, 128)))
        D = G * _spread(rng, max(1, 16 // G), 8192 // G)
        if op == "scan_step":
            b = min(b, max(1, _LARGEST_STEP // (D * N)))
        else:
            T = min(T, max(1, _LARGEST_SCAN // (b * D * N)))
        case = _scan("", b, T, D, G, N, dtype, dt=rng.choice((dtype, "f32")), softplus=rng.random() < 0.7,
                     gate=rng.random() < 0.6, sliced=rng.random() < 0.5, states=rng.random() < 0.5, docs=docs,
                     step=op == "scan_step")
    del case["name"]
    return case


def _offsets(T, docs, seed):
    """docs + 1 offsets from 0 to T: mixed lengths, an empty document among them when there are several."""
    rng = random.Random(seed)
    cuts = sorted(rng.randint(0, T) for _ in range(docs - 1))
    if len(cuts) > 2:
        cuts[1] = cuts[0]
    return [0] + cuts + [T]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dtype, b, T = _TYPES[case["dtype"]], case["b"], case["T"]

    def normal(*shape, scale=1.0, to=torch.float32):
        return (torch.randn(shape, generator=g, device="cuda") * scale).to(to)

    def uniform(*shape, lo=0.0, hi=1.0):
        return torch.rand(shape, generator=g, device="cuda") * (hi - lo) + lo

    def rows(width, before, after):
        """[b, T, width], in a projection's rows of before + width + after where the case is sliced."""
        if not case["sliced"]:
            return normal(b, T, width, to=dtype)
        return normal(b, T, before + width + after, to=dtype)[..., before:before + width]

    cu = None
    if case["docs"]:
        cu = torch.tensor(_offsets(T, case["docs"], seed), dtype=torch.int32, device="cuda")
    nseq = case["docs"] or b
    s = {"case": case, "cu": cu}
    if case["op"].startswith("conv"):
        split = [case["c0"], case["c1"], case["c2"]]
        C, W = sum(split), case["width"]
        s["split"] = tuple(c for c in split if c)
        s["u"] = rows(C, case["c0"], 80)                       # gate | x B C | dt of one projection
        s["weight"] = uniform(C, W, lo=-W ** -0.5, hi=W ** -0.5)
        s["bias"] = uniform(C, lo=-0.5, hi=0.5)
        s["state"] = normal(nseq, W - 1, C, to=dtype) if case["states"] or case["op"] == "conv_step" else None
        return s
    D, G, N = case["channels"], case["groups"], case["dstate"]
    s["u"] = normal(b, T, D, to=dtype)
    s["z"] = rows(D, D, 0) if case["gate"] else None           # x | gate of the input projection
    bc = rows(2 * G * N, 64, 0)                                # low-rank dt | B | C of the x projection
    s["B"] = bc[..., :G * N].unflatten(-1, (G, N))
    s["C"] = bc[..., G * N:].unflatten(-1, (G, N))
    s["A"] = -torch.arange(1, N + 1, device="cuda") * torch.exp(normal(D, N, scale=0.1))
    s["D"] = normal(D, scale=0.5)
    step = torch.exp(uniform(D, lo=math.log(1e-3), hi=math.log(0.1)))     # the channels' step sizes
    dt_type = _TYPES[case["dt"]]
    if case["softplus"]:
        s["bias"] = step + torch.log(-torch.expm1(-step))      # softplus(bias) = step
        s["dt"] = normal(b, T, D, scale=0.5, to=dt_type)
    else:
        s["bias"] = None
        s["dt"] = (step * uniform(b, T, D, lo=0.5, hi=2.0)).to(dt_type)
    s["state"] = normal(nseq, D, N, scale=0.5) if case["states"] or case["op"] == "scan_step" else None
    return s


# ---- plain forms -----------------------------------------------------------

def _documents(cu, T):
    """For each token of a pack: its document and its place in it."""
    t = torch.arange(T, device=cu.device)
    doc = (t[:, None] >= cu[None, 1:]).sum(1)
    return doc, t - cu.long()[doc]


def _silu(v):
    return v / (1 + torch.exp(-v))


def _plain_conv(s):
    case, W, u = s["case"], s["case"]["width"], s["u"]
    x, w = u.float(), s["weight"]
    b, T, C = x.shape
    state = s["state"]
    if s["cu"] is None:
        before = x.new_zeros(b, W - 1, C) if state is None else state.float()
        ext = torch.cat([before, x], 1)
        v = s["bias"] + sum(w[:, k] * ext[:, k:k + T] for k in range(W))
        last = ext[:, T:]
    else:
        cu = s["cu"].long()
        doc, pos = _documents(s["cu"], T)
        before = x.new_zeros(cu.numel() - 1, W - 1, C) if state is None else state.float()
        t = torch.arange(T, device=x.device)

        def token(back):
            """The token `back` places earlier in the document, or its state's."""
            here = (pos >= back)[:, None]
            return torch.where(here, x[0, (t - back).clamp(min=0)],
                               before[doc, (W - 1 + pos - back).clamp(0, W - 2)])

        v = (s["bias"] + sum(w[:, k] * token(W - 1 - k) for k in range(W)))[None]
        length = cu[1:] - cu[:-1]
        place = length[:, None] - (W - 1) + torch.arange(W - 1, device=x.device)
        last = torch.where((place >= 0)[..., None], x[0, (cu[:-1, None] + place).clamp(0, T - 1)],
                           before.gather(1, (place + W - 1).clamp(0, W - 2)[..., None].expand(-1, -1, C)))
    y = (_silu(v) if case["silu"] else v).to(u.dtype)
    return tuple(p.contiguous() for p in y.split(s["split"], -1)), last.to(u.dtype)


def _by_doubling(a, b):
    """h_t = a_t h_{t-1} + b_t along axis 1, the stretches that are summed doubling in length."""
    s = 1
    while s < a.shape[1]:
        b = torch.cat([b[:, :s], b[:, s:] + a[:, s:] * b[:, :-s]], 1)
        a = torch.cat([a[:, :s], a[:, s:] * a[:, :-s]], 1)
        s *= 2
    return b


def _plain_scan(s):
    case, u = s["case"], s["u"]
    x, dt = u.float(), s["dt"].float()
    b, T, D = x.shape
    per = D // case["groups"]
    if case["softplus"]:
        v = dt + s["bias"]
        dt = torch.clamp(v, min=0) + torch.log1p(torch.exp(-v.abs()))
    a = torch.exp(dt[..., None] * s["A"])
    Bx, Cx = (s[k].float().repeat_interleave(per, 2) for k in ("B", "C"))
    inp = (dt * x)[..., None] * Bx
    state = s["state"]
    if s["cu"] is None:
        if state is not None:
            inp[:, 0] += a[:, 0] * state
        h = _by_doubling(a, inp)
        last = h[:, -1]
    else:
        cu = s["cu"].long()
        _, pos = _documents(s["cu"], T)
        full = (cu[1:] > cu[:-1])[:, None, None]
        start, end = cu[:-1].clamp(max=T - 1), (cu[1:] - 1).clamp(min=0)
        before = x.new_zeros(cu.numel() - 1, D, case["dstate"]) if state is None else state
        inp[0].index_put_((start,), torch.where(full, a[0, start] * before, 0.0), accumulate=True)
        h = _by_doubling(a * (pos > 0)[:, None, None], inp)
        last = torch.where(full, h[0, end], before)
    y = (h * Cx).sum(-1) + s["D"] * x
    if s["z"] is not None:
        y = y * _silu(s["z"].float())
    return y.to(u.dtype), last.clone()


def _plain(s):
    op = s["case"]["op"]
    y, last = _plain_conv(s) if op.startswith("conv") else _plain_scan(s)
    if op.endswith("step"):
        s["state"].copy_(last)
        last = s["state"]
    return {"y": y, "state": last}


# ---- the framework's operators ---------------------------------------------

def _own(s):
    import structured_state_space_fwd_b200 as ssd
    op = s["case"]["op"]
    if op == "conv_step":
        y = ssd.ssd_causal_conv1d_step(s["u"], s["weight"], s["bias"], s["state"], silu=s["case"]["silu"],
                                       split=s["split"])
        return {"y": y, "state": s["state"]}
    if op == "conv":
        kw = dict(silu=s["case"]["silu"], split=s["split"], initial_states=s["state"], return_final_states=True)
        if s["cu"] is None:
            y, last = ssd.ssd_causal_conv1d(s["u"], s["weight"], s["bias"], **kw)
        else:
            y, last = ssd.ssd_causal_conv1d_varlen(s["u"], s["weight"], s["bias"], cu_seqlens=s["cu"], **kw)
        return {"y": y, "state": last}
    args = (s["u"], s["dt"], s["A"], s["B"], s["C"], s["D"])
    kw = dict(z=s["z"], dt_bias=s["bias"], dt_softplus=s["case"]["softplus"])
    if op == "scan_step":
        return {"y": ssd.ssd_selective_step(*args, s["state"], **kw), "state": s["state"]}
    kw.update(initial_states=s["state"], return_final_states=True)
    if s["cu"] is None:
        y, last = ssd.ssd_selective_scan(*args, **kw)
    else:
        y, last = ssd.ssd_selective_scan_varlen(*args, cu_seqlens=s["cu"], **kw)
    return {"y": y, "state": last}


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    b, T, nseq = case["b"], case["T"], case["docs"] or case["b"]
    step = case["op"].endswith("step")
    carried = 2 if case["states"] or step else 1                # states read and written, or only written
    if case["op"].startswith("conv"):
        C, W = case["c0"] + case["c1"] + case["c2"], case["width"]
        return {"bytes": 2 * b * T * C * e + carried * nseq * (W - 1) * C * e + 4 * C * (W + 1),
                "flops": b * T * C * (2 * W + (4 if case["silu"] else 0))}
    D, G, N = case["channels"], case["groups"], case["dstate"]
    dte = 2 if case["dt"] == "bf16" else 4
    return {"bytes": b * T * D * (e * (3 if case["gate"] else 2) + dte) + 2 * b * T * G * N * e
            + carried * nseq * D * N * 4 + 4 * D * (N + 2),
            "flops": b * T * D * (7 * N + (4 if case["gate"] else 0) + (4 if case["softplus"] else 0) + 3)}


# ---- the definitions in 64 bits --------------------------------------------

def exact(case, seed):
    """The recurrences as they are written, token by token in 64 bits."""
    s = prepare(case, seed)
    T = case["T"]
    # (batch rows, first token, end, sequences): a batch side by side, a pack's documents one after another
    spans = [(slice(None), 0, T, slice(None))]
    if s["cu"] is not None:
        cu = s["cu"].tolist()
        spans = [(slice(0, 1), cu[k], cu[k + 1], slice(k, k + 1)) for k in range(case["docs"])]
    u = s["u"].double()
    y = torch.empty_like(u)
    last = []
    for rows, p, q, seqs in spans:
        if case["op"].startswith("conv"):
            C, W = u.shape[2], case["width"]
            w, bias = s["weight"].double(), s["bias"].double()
            n = u[rows].shape[0]
            tail = s["state"][seqs].double() if s["state"] is not None else u.new_zeros(n, W - 1, C)
            seq = torch.cat([tail, u[rows, p:q]], 1)
            if q > p:
                v = torch.nn.functional.conv1d(seq.transpose(1, 2), w[:, None], bias, groups=C).transpose(1, 2)
                y[rows, p:q] = v * torch.sigmoid(v) if case["silu"] else v
            last.append(seq[:, seq.shape[1] - (W - 1):])
            continue
        D, G, N = case["channels"], case["groups"], case["dstate"]
        A, skip = s["A"].double(), s["D"].double()
        group = torch.arange(D, device=u.device) // (D // G)
        h = s["state"][seqs].double().clone() if s["state"] is not None else u.new_zeros(u[rows].shape[0], D, N)
        for t in range(p, q):
            x, dt = u[rows, t], s["dt"][rows, t].double()
            if case["softplus"]:
                dt = torch.logaddexp(dt + s["bias"].double(), torch.zeros_like(dt))
            h = torch.exp(dt[..., None] * A) * h + (dt * x)[..., None] * s["B"][rows, t].double()[:, group]
            out = torch.einsum("bdn,bdn->bd", h, s["C"][rows, t].double()[:, group]) + skip * x
            if s["z"] is not None:
                out = out * s["z"][rows, t].double() * torch.sigmoid(s["z"][rows, t].double())
            y[rows, t] = out
        last.append(h)
    last = torch.cat(last, 0)
    if case["op"].startswith("conv"):
        return {"y": tuple(y.split(s["split"], -1)), "state": last}
    return {"y": y, "state": last}
