"""Cases of the Mamba layer's serving and training operators, with their plain forms.

Five operators:
  step        ss.ssd_step: one token of many requests, causal convolution and Mamba-2
              state update in one call, over a pool of state slots
  conv        ss.conv1d_prompt: causal convolution + SiLU of packed prompts
  prompt      ss.ssd_prompt: Mamba-2 scan of packed prompts from and into state slots
  ssd_grad    ss.ssd_bwd: gradients of the Mamba-2 scan
  conv_grad   ss.conv1d_bwd: gradients of the causal convolution

``run`` computes them in plain torch operations in 32 bits (``own`` false) or through
the library (``own`` true); ``exact`` evaluates their definitions, the recurrences
step by step, in 64 bits.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
P = 64          # channels of a head
Q = 64          # steps of a chunk of the plain form


def listed():
    return [
        # one request decoding alone: pure latency (a 130m-class layer: 24 heads, state 128)
        dict(name="token, one request", op="step", n=1, heads=24, groups=1, dstate=128, width=4, io="bf16", slots=16,
             pad=0, gate=True),
        # a serving batch in a captured loop: 64 rows, some of them padding
        dict(name="tokens, 64 requests", op="step", n=64, heads=24, groups=1, dstate=128, width=4, io="bf16",
             slots=256, pad=3, gate=True),
        # a wide layer (5120 channels, 8 groups) under a large batch of an odd size
        dict(name="tokens, 201 requests, wide", op="step", n=201, heads=80, groups=8, dstate=64, width=4, io="f16",
             slots=256, pad=0, gate=False),
        # the convolution of one prompt (1536 + 2 * 128 channels)
        dict(name="conv, one prompt", op="conv", tokens=2048, seqs=1, tail=0, dim=1792, width=4, io="bf16", slots=16,
             carried=False),
        # many ragged prompts, some continued from their windows, a few unused rows behind the last
        dict(name="conv, ragged prompts", op="conv", tokens=16021, seqs=37, tail=11, dim=5376, width=4, io="f16",
             slots=64, carried=True),
        # short prompts: a few tokens each, latency counts
        dict(name="prompts, short", op="prompt", tokens=131, seqs=5, tail=0, heads=24, groups=1, dstate=128, io="bf16",
             slots=16, carried=False, gate=False),
        # a prefill batch of ragged prompts of the bench's Mamba-2 layer
        dict(name="prompts, ragged", op="prompt", tokens=16384, seqs=24, tail=5, heads=24, groups=1, dstate=128,
             io="bf16", slots=64, carried=True, gate=True),
        # one long prompt, an odd length
        dict(name="prompt, long", op="prompt", tokens=32769, seqs=1, tail=0, heads=24, groups=2, dstate=64, io="f16",
             slots=4, carried=True, gate=False),
        # a training step's backward of the bench's Mamba-2 layer (the gate sits in the norm behind it)
        dict(name="ssd gradients, layer", op="ssd_grad", batch=8, seqlen=2048, heads=24, groups=1, dstate=128,
             io="bf16", gate=False, docs=0, state=False),
        # packed documents, the gate inside, pieces of a row chained through the state
        dict(name="ssd gradients, packed", op="ssd_grad", batch=2, seqlen=1001, heads=8, groups=2, dstate=64, io="f16",
             gate=True, docs=6, state=True),
        # a training step's backward of the mamba-130m x branch
        dict(name="conv gradients, layer", op="conv_grad", batch=8, dim=1536, seqlen=2048, width=4, io="bf16", docs=0,
             state=False),
        # an odd length in fp32 with packed documents and a carried window
        dict(name="conv gradients, odd", op="conv_grad", batch=3, dim=100, seqlen=4097, width=4, io="f32", docs=9,
             state=True),
    ]


def _logint(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["step", "conv", "prompt", "ssd_grad", "conv_grad"])
    io = rng.choice(["bf16", "f16"])
    if op == "conv":
        t = _logint(rng, 16, 16000)
        # whole vectors of channels more often than not, as models have them
        dim = 8 * _logint(rng, 8, 640) if rng.random() < 0.7 else _logint(rng, 65, 5000)
        return dict(op=op, tokens=t, seqs=_logint(rng, 1, min(t, 64)), tail=rng.choice([0, 0, 3]), dim=dim,
                    width=rng.choice([2, 3, 4, 4]), io=rng.choice(["bf16", "f16", "f32"]), slots=80,
                    carried=rng.random() < 0.5)
    if op == "conv_grad":
        b, dim = rng.randint(1, 8), _logint(rng, 16, 1536)
        return dict(op=op, batch=b, dim=dim, seqlen=_logint(rng, 16, 2048 * 8 // b), width=rng.choice([2, 3, 4, 4]),
                    io=rng.choice(["bf16", "f16", "f32"]), docs=rng.choice([0, 5]), state=rng.random() < 0.5)
    heads = rng.choice([4, 8, 16, 24, 32])
    groups = rng.choice([1, 1, 2, 4])
    dstate = rng.choice([32, 64, 96, 128])
    if op == "step":
        n = _logint(rng, 1, 250)
        return dict(op=op, n=n, heads=heads, groups=groups, dstate=dstate, width=rng.choice([2, 3, 4, 4]), io=io,
                    slots=n + rng.randint(0, 9), pad=rng.choice([0, 1]) if n > 1 else 0, gate=rng.random() < 0.5)
    if op == "prompt":
        t = _logint(rng, 1, 12000)
        return dict(op=op, tokens=t, seqs=_logint(rng, 1, min(t, 64)), tail=rng.choice([0, 0, 7]), heads=heads,
                    groups=groups, dstate=dstate, io=io, slots=80, carried=rng.random() < 0.5, gate=rng.random() < 0.5)
    b = rng.randint(1, 4)
    return dict(op=op, batch=b, seqlen=_logint(rng, 1, 8192 // b), heads=heads, groups=groups, dstate=dstate, io=io,
                gate=rng.random() < 0.5, docs=rng.choice([0, 4]), state=rng.random() < 0.5)


# ---- inputs -------------------------------------------------------------------


class _Rand:
    def __init__(self, seed):
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(int(seed))

    def normal(self, *shape, scale=1.0, dtype=torch.float32):
        return (torch.randn(*shape, generator=self.g, device="cuda") * scale).to(dtype)

    def uniform(self, lo, hi, *shape):
        return torch.rand(*shape, generator=self.g, device="cuda") * (hi - lo) + lo

    def perm(self, n):
        return torch.randperm(n, generator=self.g, device="cuda")

    def cuts(self, total, parts):
        """parts + 1 increasing int32 offsets from 0 to total, every part at least 1 long."""
        inner = torch.randperm(total - 1, generator=self.g, device="cuda")[:parts - 1].sort().values + 1
        ends = torch.tensor([0, total], device="cuda")
        return torch.cat([ends[:1], inner, ends[1:]]).to(torch.int32)


def _ssm_weights(r, heads):
    """A, D, dt_bias as Mamba-2 starts them: A in -[1, 16], a step size of 1e-3 .. 1e-1."""
    dt0 = torch.exp(r.uniform(math.log(1e-3), math.log(1e-1), heads))
    return dict(A=-r.uniform(1.0, 16.0, heads), D=r.normal(heads), dt_bias=torch.log(torch.expm1(dt0)))


def prepare(case, seed):
    c, r = case, _Rand(seed)
    io = DT[c["io"]]
    s = dict(case=dict(c))
    if c["op"] == "step":
        n, hd, gn = c["n"], c["heads"] * P, c["groups"] * c["dstate"]
        dc = hd + 2 * gn
        s.update(_ssm_weights(r, c["heads"]))
        # one row of the input projection's output: gate, convolved channels, dt
        row = r.normal(n, hd + dc + c["heads"], dtype=io)
        s.update(z=row[:, :hd].view(n, c["heads"], P) if c["gate"] else None, xbc=row[:, hd:hd + dc],
                 dt=row[:, hd + dc:], w=r.normal(dc, c["width"], scale=0.5), bias=r.normal(dc, scale=0.1),
                 conv_state=r.normal(c["slots"], dc, c["width"] - 1),
                 state=r.normal(c["slots"], c["heads"], P, c["dstate"], scale=0.5),
                 slots=r.perm(c["slots"])[:n].to(torch.int32), y=torch.zeros(n, c["heads"], P, dtype=io, device="cuda"))
        if c["pad"]:
            s["slots"][n - c["pad"]:] = -1
    elif c["op"] == "conv":
        t = c["tokens"]
        # the convolved channels inside the projection's rows
        row = r.normal(t + c["tail"], 2 * c["dim"], dtype=io)
        s.update(x=row[:, c["dim"]:] if c["dim"] % 8 == 0 else row[:, c["dim"]:].contiguous(),
                 w=r.normal(c["dim"], c["width"], scale=0.5), bias=r.normal(c["dim"], scale=0.1),
                 cu=r.cuts(t, c["seqs"]), slots=r.perm(c["slots"])[:c["seqs"]].to(torch.int32),
                 conv_state=r.normal(c["slots"], c["dim"], c["width"] - 1),
                 out=torch.zeros(t + c["tail"], c["dim"], dtype=io, device="cuda"))
        s["has"] = (r.perm(c["seqs"]) % 2).to(torch.int32) if c["carried"] else None
    elif c["op"] == "prompt":
        t, h, g, n = c["tokens"], c["heads"], c["groups"], c["dstate"]
        s.update(_ssm_weights(r, h))
        # the convolution's output rows hold x, B and C side by side
        row = r.normal(t + c["tail"], h * P + 2 * g * n, dtype=io)
        s.update(x=row[:, :h * P].view(-1, h, P), Bm=row[:, h * P:h * P + g * n].view(-1, g, n),
                 Cm=row[:, h * P + g * n:].view(-1, g, n), dt=r.normal(t + c["tail"], h, scale=0.5, dtype=io),
                 z=r.normal(t + c["tail"], h, P, dtype=io) if c["gate"] else None, cu=r.cuts(t, c["seqs"]),
                 slots=r.perm(c["slots"])[:c["seqs"]].to(torch.int32),
                 state=r.normal(c["slots"], h, P, n, scale=0.5),
                 y=torch.zeros(t + c["tail"], h, P, dtype=io, device="cuda"))
        s["has"] = (r.perm(c["seqs"]) % 2 == 0).to(torch.int32) if c["carried"] else None
    elif c["op"] == "ssd_grad":
        b, l, h, g, n = c["batch"], c["seqlen"], c["heads"], c["groups"], c["dstate"]
        s.update(_ssm_weights(r, h))
        s.update(x=r.normal(b, l, h, P, dtype=io), dt=r.normal(b, l, h, scale=0.5, dtype=io),
                 Bm=r.normal(b, l, g, n, dtype=io), Cm=r.normal(b, l, g, n, dtype=io), dy=r.normal(b, l, h, P, dtype=io),
                 z=r.normal(b, l, h, P, dtype=io) if c["gate"] else None, seq_idx=_doc_ids(r, c),
                 h0=r.normal(b, h, P, n, scale=0.5) if c["state"] else None,
                 dfinal=r.normal(b, h, P, n, scale=0.1) if c["state"] else None)
    else:
        b, d, l, w = c["batch"], c["dim"], c["seqlen"], c["width"]
        s.update(x=r.normal(b, d, l, dtype=io), w=r.normal(d, w, scale=0.5), bias=r.normal(d, scale=0.1),
                 dout=r.normal(b, d, l, dtype=io), seq_idx=_doc_ids(r, c),
                 init=r.normal(b, d, w - 1) if c["state"] else None,
                 dfinal=r.normal(b, d, w - 1) if c["state"] else None)
    return s


def _doc_ids(r, c):
    """(batch, seqlen) document ids, or None: every row holds up to c["docs"] documents of random lengths."""
    if not c["docs"]:
        return None
    starts = r.uniform(0.0, 1.0, c["batch"], c["seqlen"]) < (c["docs"] - 1) / c["seqlen"]
    return starts.to(torch.int32).cumsum(1).to(torch.int32)


# ---- one pass -----------------------------------------------------------------


def run(state):
    s = state
    if own:
        return _run_own(s)
    return {"step": _plain_step, "conv": _plain_conv, "prompt": _plain_prompt, "ssd_grad": _plain_ssd_grad,
            "conv_grad": _plain_conv_grad}[s["case"]["op"]](s)


def _run_own(s):
    from mamba_selective_scan_fwd_amd import ss
    op = s["case"]["op"]
    if op == "step":
        y = ss.ssd_step(s["xbc"], s["dt"], s["A"], s["w"], s["conv_state"], s["state"], ngroups=s["case"]["groups"],
                        conv_bias=s["bias"], D=s["D"], z=s["z"], dt_bias=s["dt_bias"], slots=s["slots"], y=s["y"])
        return dict(y=y, conv_state=s["conv_state"], state=s["state"])
    if op == "conv":
        out = ss.conv1d_prompt(s["x"], s["w"], s["cu"], s["conv_state"], bias=s["bias"], slots=s["slots"],
                               has_state=s["has"], out=s["out"])
        return dict(out=out, conv_state=s["conv_state"])
    if op == "prompt":
        y = ss.ssd_prompt(s["x"], s["dt"], s["A"], s["Bm"], s["Cm"], s["cu"], s["state"], D=s["D"], z=s["z"],
                          dt_bias=s["dt_bias"], slots=s["slots"], has_state=s["has"], y=s["y"])
        return dict(y=y, state=s["state"])
    if op == "ssd_grad":
        return ss.ssd_bwd(s["x"], s["dt"], s["A"], s["Bm"], s["Cm"], s["dy"], D=s["D"], z=s["z"], dt_bias=s["dt_bias"],
                          seq_idx=s["seq_idx"], h0=s["h0"], dfinal=s["dfinal"], want_dh0=s["h0"] is not None)
    return ss.conv1d_bwd(s["x"], s["w"], s["dout"], bias=s["bias"], seq_idx=s["seq_idx"], conv_init=s["init"],
                         dconv_final=s["dfinal"], want_dconv_init=s["init"] is not None)


# ---- plain forms ----------------------------------------------------------------


def _silu(v):
    return v * torch.sigmoid(v)


def _softplus(v):
    return torch.log1p(torch.exp(-v.abs())) + v.clamp(min=0)


def _plain_step(s):
    c = s["case"]
    h, g, n, w = c["heads"], c["groups"], c["dstate"], c["width"]
    rows = torch.arange(c["n"], device="cuda") if not c["pad"] else (s["slots"] >= 0).nonzero()[:, 0]
    slots = s["slots"][rows].long()
    new = s["xbc"][rows].float()
    win = torch.cat([s["conv_state"][slots], new[:, :, None]], 2)                    # (n, Dc, W)
    s["conv_state"][slots] = win[:, :, 1:]
    xbc = _silu((win * s["w"]).sum(2) + s["bias"])
    x = xbc[:, :h * P].reshape(-1, h, P)
    bm = xbc[:, h * P:h * P + g * n].reshape(-1, g, n).repeat_interleave(h // g, 1)
    cm = xbc[:, h * P + g * n:].reshape(-1, g, n).repeat_interleave(h // g, 1)
    delta = _softplus(s["dt"][rows].float() + s["dt_bias"])
    st = s["state"][slots] * torch.exp(delta * s["A"])[:, :, None, None]
    st = st + (delta[:, :, None] * x)[..., None] * bm[:, :, None, :]
    s["state"][slots] = st
    y = (st * cm[:, :, None, :]).sum(3) + s["D"][:, None] * x
    if s["z"] is not None:
        y = y * _silu(s["z"][rows].float())
    s["y"][rows] = y.to(s["y"].dtype)
    return dict(y=s["y"], conv_state=s["conv_state"], state=s["state"])


def _tokens(cu, total):
    """(sequence, position in it, in any sequence) of every row."""
    t = torch.arange(total, device="cuda")
    seq = (torch.searchsorted(cu, t.to(cu.dtype), right=True) - 1).clamp(0, cu.numel() - 2)
    return seq, t - cu[seq], t < cu[-1]


def _plain_conv(s):
    c = s["case"]
    w1 = c["width"] - 1
    total = c["tokens"] + c["tail"]
    seq, pos, used = _tokens(s["cu"], total)
    slots = s["slots"].long()
    init = s["conv_state"][slots]                                                    # (S, D, W-1)
    init = init * s["has"].float()[:, None, None] if s["has"] is not None else torch.zeros_like(init)
    x = s["x"].float()
    # every sequence's rows behind its window: row w1 * (seq + 1) + t
    wide = torch.zeros(total + w1 * (c["seqs"] + 1), c["dim"], device="cuda")
    at = torch.arange(total, device="cuda") + w1 * (seq + 1)
    wide[at] = x
    lag = torch.arange(w1, device="cuda")
    first = s["cu"][:-1].long() + w1 * torch.arange(c["seqs"], device="cuda")
    wide[first[:, None] + lag] = init.transpose(1, 2)
    seen = wide[at[:, None] - w1 + torch.arange(w1 + 1, device="cuda")]               # (T, W, D)
    pre = s["bias"] + (seen * s["w"].t()).sum(1)
    s["out"].copy_(torch.where(used[:, None], _silu(pre).to(s["out"].dtype), s["out"]))
    last = s["cu"][1:].long() + w1 * torch.arange(c["seqs"], device="cuda")
    s["conv_state"][slots] = wide[last[:, None] + lag].transpose(1, 2).contiguous()
    return dict(out=s["out"], conv_state=s["conv_state"])


def _chunked(x, delta, A, bm, cm, cu, init):
    """The Mamba-2 scan of packed sequences in chunks of Q steps.  x (T, H, P), delta (T, H), bm, cm (T, G, N) in
    32 bits, cu (S + 1), init (S, H, P, N).  Returns y without skip and gate (T, H, P), and the states (S, H, P, N).
    Sequence s owns the chunks from cu[s] // Q + s on, the ones behind its last step stay empty."""
    total, heads = delta.shape
    groups, n, seqs = bm.shape[1], bm.shape[2], cu.numel() - 1
    cu = cu.long()
    seq, pos, used = _tokens(cu, total)
    nchunk = total // Q + seqs
    first = cu[:-1] // Q + torch.arange(seqs, device="cuda")
    at = torch.where(used, (first[seq] + pos // Q) * Q + pos % Q, nchunk * Q)

    def lay(v):
        out = torch.zeros((nchunk + 1) * Q, *v.shape[1:], dtype=v.dtype, device="cuda").index_copy(0, at, v)
        return out[:nchunk * Q].view(nchunk, Q, *v.shape[1:])

    def per_head(v):
        return v.permute(0, 2, 1, 3).repeat_interleave(heads // groups, 1)          # (V, H, Q, N)

    d = lay(torch.where(used[:, None], delta, torch.zeros_like(delta)))             # (V, Q, H)
    xs, bs, cs = lay(x).permute(0, 2, 1, 3), per_head(lay(bm)), per_head(lay(cm))
    # decays in 64 bits: differences of long sums
    run = (d.double() * A.double()).cumsum(1).permute(0, 2, 1)                       # (V, H, Q)
    steps = torch.arange(Q, device="cuda")
    low = steps[:, None] >= steps
    decay = torch.exp((run[..., :, None] - run[..., None, :]).masked_fill(~low, -math.inf)).float()
    dx = d.permute(0, 2, 1)[..., None] * xs                                          # Delta x
    y = ((cs @ bs.transpose(2, 3)) * decay) @ dx
    rest = torch.exp(run[..., -1:] - run).float()
    own_state = (dx * rest[..., None]).transpose(2, 3) @ bs                          # (V, H, P, N)
    # the state that enters each chunk, from all earlier chunks of its sequence and its first state
    total_log = run[..., -1].t().cumsum(1)                                           # (H, V)
    chunks = torch.arange(nchunk, device="cuda")
    owner = torch.searchsorted(first, chunks, right=True) - 1
    before = torch.cat([torch.zeros(heads, 1, dtype=torch.float64, device="cuda"), total_log[:, :-1]], 1)
    carried = (owner[:, None] == owner) & (chunks[:, None] > chunks)
    between = torch.exp((before[:, :, None] - total_log[:, None, :]).masked_fill(~carried, -math.inf)).float()
    enter = (between @ own_state.permute(1, 0, 2, 3).reshape(heads, nchunk, P * n)).view(heads, nchunk, P, n)
    enter = enter.permute(1, 0, 2, 3)
    enter = enter + torch.exp(before - before[:, first[owner]]).float().t()[..., None, None] * init[owner]
    y = y + (cs * torch.exp(run).float()[..., None]) @ enter.transpose(2, 3)
    ends = torch.cat([first[1:], first.new_full((1,), nchunk)]) - 1
    leave = own_state[ends] + torch.exp(run[ends][..., -1]).float()[..., None, None] * enter[ends]
    flat = torch.cat([y.permute(0, 2, 1, 3).reshape(nchunk * Q, heads, P), y.new_zeros(1, heads, P)])
    return flat[at], leave


def _plain_prompt(s):
    slots = s["slots"].long()
    init = s["state"][slots]
    init = init * s["has"].float()[:, None, None, None] if s["has"] is not None else torch.zeros_like(init)
    x = s["x"].float()
    delta = _softplus(s["dt"].float() + s["dt_bias"])
    y, last = _chunked(x, delta, s["A"], s["Bm"].float(), s["Cm"].float(), s["cu"], init)
    y = y + s["D"][:, None] * x
    if s["z"] is not None:
        y = y * _silu(s["z"].float())
    used = torch.arange(x.shape[0], device="cuda") < s["cu"][-1]
    s["y"].copy_(torch.where(used[:, None, None], y.to(s["y"].dtype), s["y"]))
    s["state"][slots] = last
    return dict(y=s["y"], state=s["state"])


def _plain_ssd_grad(s):
    c = s["case"]
    b, l = c["batch"], c["seqlen"]
    leaves = {k: s[k].detach().float().requires_grad_() for k in ("x", "dt", "A", "Bm", "Cm", "D", "dt_bias", "z", "h0")
              if s[k] is not None}
    # every document is a sequence of its own; a row's first one starts from its h0, its last one ends in its state
    new = torch.zeros(b, l, dtype=torch.bool, device="cuda")
    new[:, 0] = True
    if s["seq_idx"] is not None:
        new[:, 1:] = s["seq_idx"][:, 1:] != s["seq_idx"][:, :-1]
    cu = torch.cat([new.view(-1).nonzero()[:, 0], torch.tensor([b * l], device="cuda")])
    init = torch.zeros(cu.numel() - 1, c["heads"], P, c["dstate"], device="cuda")
    if s["h0"] is not None:
        init = init.index_copy(0, torch.searchsorted(cu, torch.arange(b, device="cuda") * l), leaves["h0"])
    flat = {k: v.reshape(b * l, *v.shape[2:]) for k, v in leaves.items() if k in ("x", "dt", "Bm", "Cm")}
    delta = _softplus(flat["dt"] + leaves["dt_bias"])
    y, last = _chunked(flat["x"], delta, leaves["A"], flat["Bm"], flat["Cm"], cu, init)
    y = (y + leaves["D"][:, None] * flat["x"]).view(b, l, c["heads"], P)
    if s["z"] is not None:
        y = y * _silu(leaves["z"])
    outs, grads = [y], [s["dy"].float()]
    if s["dfinal"] is not None:
        outs.append(last[torch.searchsorted(cu, torch.arange(1, b + 1, device="cuda") * l) - 1])
        grads.append(s["dfinal"])
    g = dict(zip(leaves, torch.autograd.grad(outs, list(leaves.values()), grads)))
    names = dict(x="dx", dt="ddt", A="dA", Bm="dB", Cm="dC", D="dD", dt_bias="ddt_bias", z="dz", h0="dh0")
    return {names[k]: v.to(s[k].dtype) for k, v in g.items()}


def _plain_conv_grad(s):
    c = s["case"]
    w1, l = c["width"] - 1, c["seqlen"]
    x = s["x"].float()
    init = s["init"] if s["init"] is not None else torch.zeros(c["batch"], c["dim"], w1, device="cuda")
    ids = s["seq_idx"] if s["seq_idx"] is not None else torch.zeros(c["batch"], l, dtype=torch.int32, device="cuda")
    wide = torch.cat([init, x], 2)                                                   # (B, D, W-1 + L)
    ids = torch.cat([ids[:, :1].expand(-1, w1), ids], 1)                             # the window is the first document's
    lag = torch.arange(w1 + 1, device="cuda")
    at = torch.arange(l, device="cuda")[:, None] + lag                               # (L, W): inputs of step t
    same = (ids[:, at] == ids[:, w1:, None])[:, None].float()                        # (B, 1, L, W)
    seen = wide[:, :, at] * same
    pre = (seen * s["w"][:, None, :]).sum(3) + s["bias"][:, None]
    sg = torch.sigmoid(pre)
    dpre = s["dout"].float() * sg * (1 + pre * (1 - sg))
    out = dict(dw=(dpre[..., None].double() * seen).sum((0, 2)).float(), dbias=dpre.double().sum((0, 2)).float())
    dwide = torch.zeros_like(wide)
    dwide = dwide.index_add(2, at.reshape(-1), (dpre[..., None] * same * s["w"][:, None, :]).flatten(2))
    if s["dfinal"] is not None:
        dwide[:, :, l:] += s["dfinal"] * (ids[:, None, l:] == ids[:, None, -1:])
    out["dx"] = dwide[:, :, w1:].to(s["x"].dtype)
    if s["init"] is not None:
        out["dconv_init"] = dwide[:, :, :w1].contiguous()
    return out


# ---- work -----------------------------------------------------------------------


def work(case):
    c = case
    e = 4 if c["io"] == "f32" else 2
    if c["op"] == "step":
        n, hd, gn = c["n"] - c["pad"], c["heads"] * P, c["groups"] * c["dstate"]
        dc = hd + 2 * gn
        st = n * hd * c["dstate"]
        byt = 8 * st + 8 * n * dc * (c["width"] - 1) + e * n * (dc + c["heads"] + hd * (2 if c["gate"] else 1)) + \
            4 * (dc * (c["width"] + 1) + 3 * c["heads"]) + 4 * n
        return dict(bytes=byt, flops=5 * st + 2 * n * dc * c["width"])
    if c["op"] == "conv":
        td = c["tokens"] * c["dim"]
        return dict(bytes=2 * e * td + 4 * c["dim"] * (c["width"] + 1 + c["seqs"] * (c["width"] - 1) *
                                                        (2 if c["carried"] else 1)) + 8 * c["seqs"],
                    flops=td * (2 * c["width"] + 4))
    if c["op"] == "prompt":
        t, hd, gn = c["tokens"], c["heads"] * P, c["groups"] * c["dstate"]
        byt = e * t * (hd * (3 if c["gate"] else 2) + 2 * gn + c["heads"]) + \
            4 * c["seqs"] * hd * c["dstate"] * (2 if c["carried"] else 1) + 12 * c["heads"]
        return dict(bytes=byt, flops=5 * t * hd * c["dstate"])
    if c["op"] == "ssd_grad":
        t, hd, gn = c["batch"] * c["seqlen"], c["heads"] * P, c["groups"] * c["dstate"]
        byt = e * t * (hd * (5 if c["gate"] else 3) + 4 * gn + 2 * c["heads"]) + \
            (12 * c["batch"] * hd * c["dstate"] if c["state"] else 0) + (4 * t if c["docs"] else 0) + 24 * c["heads"]
        # the states and their gradients rebuilt (3 each), dB, dC, dx and the decay's gradient (2 each)
        return dict(bytes=byt, flops=14 * t * hd * c["dstate"])
    td = c["batch"] * c["dim"] * c["seqlen"]
    w = c["width"]
    return dict(bytes=3 * e * td + 8 * c["dim"] * (w + 1) + (4 * c["batch"] * c["seqlen"] if c["docs"] else 0) +
                (12 * c["batch"] * c["dim"] * (w - 1) if c["state"] else 0), flops=td * (6 * w + 8))


# ---- the definitions in 64 bits ---------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    s = {k: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v for k, v in s.items()}
    with torch.no_grad():
        return {"step": _exact_step, "conv": _exact_conv, "prompt": _exact_prompt, "ssd_grad": _exact_ssd_grad,
                "conv_grad": _exact_conv_grad}[case["op"]](s)


def _exact_step(s):
    c = s["case"]
    h, g, n = c["heads"], c["groups"], c["dstate"]
    for i, slot in enumerate(s["slots"].tolist()):
        if slot < 0:
            continue
        win = torch.cat([s["conv_state"][slot], s["xbc"][i][:, None]], 1)
        s["conv_state"][slot] = win[:, 1:]
        pre = torch.einsum("dk,dk->d", win, s["w"]) + s["bias"]
        a = pre / (1 + torch.exp(-pre))
        x = a[:h * P].view(h, P)
        bm, cm = (a[o:o + g * n].view(g, n) for o in (h * P, h * P + g * n))
        grp = torch.arange(h, device="cuda") // (h // g)
        delta = torch.logaddexp(s["dt"][i] + s["dt_bias"], torch.zeros((), dtype=torch.float64, device="cuda"))
        st = torch.exp(delta * s["A"]).view(h, 1, 1) * s["state"][slot] + \
            torch.einsum("h,hp,hn->hpn", delta, x, bm[grp])
        s["state"][slot] = st
        y = torch.einsum("hpn,hn->hp", st, cm[grp]) + s["D"].view(h, 1) * x
        s["y"][i] = y if s["z"] is None else y * s["z"][i] / (1 + torch.exp(-s["z"][i]))
    return dict(y=s["y"], conv_state=s["conv_state"], state=s["state"])


def _exact_conv(s):
    w1 = s["case"]["width"] - 1
    cu, slots = s["cu"].tolist(), s["slots"].tolist()
    for q, slot in enumerate(slots):
        a, e = cu[q], cu[q + 1]
        win = s["conv_state"][slot].t() if s["has"] is not None and int(s["has"][q]) else \
            torch.zeros(w1, s["case"]["dim"], dtype=torch.float64, device="cuda")
        rows = torch.cat([win, s["x"][a:e]])
        pre = sum(rows[k:k + e - a] * s["w"][:, k] for k in range(w1 + 1)) + s["bias"]
        s["out"][a:e] = pre / (1 + torch.exp(-pre))
        s["conv_state"][slot] = rows[rows.shape[0] - w1:].t()
    return dict(out=s["out"], conv_state=s["conv_state"])


def _exact_prompt(s):
    c = s["case"]
    h, g, n = c["heads"], c["groups"], c["dstate"]
    cu, slots = s["cu"].long(), s["slots"].long()
    lens = cu[1:] - cu[:-1]
    grp = torch.arange(h, device="cuda") // (h // g)
    st = s["state"][slots]
    st = st * s["has"].double().view(-1, 1, 1, 1) if s["has"] is not None else torch.zeros_like(st)
    order = torch.argsort(lens, descending=True)
    counts = torch.bincount(lens, minlength=int(lens.max()) + 1).flip(0).cumsum(0).flip(0).tolist()  # lens >= t
    delta = torch.logaddexp(s["dt"] + s["dt_bias"], torch.zeros((), dtype=torch.float64, device="cuda"))
    da = torch.exp(delta * s["A"])
    first, st = cu[:-1][order], st[order]
    for t in range(int(lens.max())):
        k = counts[t + 1]                                   # sequences that have a step t
        row = first[:k] + t
        st[:k] *= da[row][:, :, None, None]
        st[:k] += (delta[row][:, :, None] * s["x"][row])[..., None] * s["Bm"][row][:, grp][:, :, None, :]
        s["y"][row] = torch.matmul(st[:k], s["Cm"][row][:, grp][..., None])[..., 0] + s["D"].view(h, 1) * s["x"][row]
    if s["z"] is not None:
        used = int(cu[-1])
        s["y"][:used] *= s["z"][:used] / (1 + torch.exp(-s["z"][:used]))
    s["state"][slots[order]] = st
    return dict(y=s["y"], state=s["state"])


def _exact_ssd_grad(s):
    """The recurrence forward, its states kept every K steps, then backward through the segments."""
    c = s["case"]
    b, l, h, g, n, seg = c["batch"], c["seqlen"], c["heads"], c["groups"], c["dstate"], 32
    grp = torch.arange(h, device="cuda") // (h // g)
    raw = s["dt"] + s["dt_bias"]
    delta = torch.logaddexp(raw, torch.zeros((), dtype=torch.float64, device="cuda"))
    a = torch.exp(delta * s["A"])
    keep = torch.ones(b, l, dtype=torch.float64, device="cuda")        # 0 where a document starts inside a row
    if s["seq_idx"] is not None:
        keep[:, 1:] = (s["seq_idx"][:, 1:] == s["seq_idx"][:, :-1]).double()
    a = a * keep[..., None]

    def advance(st, t):
        return a[:, t, :, None, None] * st + (delta[:, t, :, None] * s["x"][:, t])[..., None] * \
            s["Bm"][:, t][:, grp][:, :, None, :]

    st = s["h0"] if s["h0"] is not None else torch.zeros(b, h, P, n, dtype=torch.float64, device="cuda")
    kept = []
    for t in range(l):
        if t % seg == 0:
            kept.append(st)
        st = advance(st, t)
    grad = s["dfinal"].clone() if s["dfinal"] is not None else torch.zeros_like(st)
    out = dict(dx=torch.zeros_like(s["x"]), dB=torch.zeros_like(s["Bm"]), dC=torch.zeros_like(s["Cm"]))
    ddelta, y = torch.zeros_like(delta), torch.zeros_like(s["x"])
    dlog = torch.zeros_like(delta)
    sig = None
    dy0 = s["dy"]
    if s["z"] is not None:
        sig = 1 / (1 + torch.exp(-s["z"]))
        dy0 = s["dy"] * s["z"] * sig
    for k in range(len(kept) - 1, -1, -1):
        states = [kept[k]]
        for t in range(k * seg, min(l, (k + 1) * seg)):
            states.append(advance(states[-1], t))
        for t in range(min(l, (k + 1) * seg) - 1, k * seg - 1, -1):
            bm, cm = s["Bm"][:, t][:, grp], s["Cm"][:, t][:, grp]
            now, prev = states[t - k * seg + 1], states[t - k * seg]
            if sig is not None:
                y[:, t] = torch.matmul(now, cm[..., None])[..., 0]
            dc = torch.matmul(dy0[:, t][:, :, None, :], now)[:, :, 0]
            out["dC"][:, t] = dc.view(b, g, h // g, n).sum(2)
            grad = grad + dy0[:, t][..., None] * cm[:, :, None, :]
            gb = torch.matmul(grad, bm[..., None])[..., 0]              # (B, H, P)
            out["dx"][:, t] = delta[:, t, :, None] * gb + s["D"][:, None] * dy0[:, t]
            db = delta[:, t, :, None] * torch.matmul(s["x"][:, t][:, :, None, :], grad)[:, :, 0]
            out["dB"][:, t] = db.view(b, g, h // g, n).sum(2)
            dlog[:, t] = a[:, t] * (grad * prev).sum((2, 3))
            ddelta[:, t] = (gb * s["x"][:, t]).sum(2) + s["A"] * dlog[:, t]
            grad = a[:, t, :, None, None] * grad
    out["dA"] = (delta * dlog).sum((0, 1))
    out["ddt"] = ddelta / (1 + torch.exp(-raw))
    out["ddt_bias"] = out["ddt"].sum((0, 1))
    out["dD"] = (dy0 * s["x"]).sum((0, 1, 3))
    if sig is not None:
        full = y + s["D"][:, None] * s["x"]
        out["dz"] = s["dy"] * full * sig * (1 + s["z"] * (1 - sig))
    if s["h0"] is not None:
        out["dh0"] = grad
    return out


def _exact_conv_grad(s):
    c = s["case"]
    w1, l = c["width"] - 1, c["seqlen"]
    ids = s["seq_idx"]

    def meets(t0, k):
        """1 where step t and the input k steps before it are of one document, for t >= t0."""
        if ids is None:
            return torch.ones(c["batch"], 1, l - t0, dtype=torch.float64, device="cuda")
        return (ids[:, t0:] == ids[:, t0 - k:l - k]).double()[:, None]

    pre = s["bias"][:, None] + torch.zeros_like(s["x"])
    for k in range(w1 + 1):
        wk = s["w"][:, w1 - k, None]
        if k < l:
            pre[:, :, k:] += wk * s["x"][:, :, :l - k] * meets(k, k)
        if s["init"] is not None:
            for t in range(min(k, l)):      # input t - k < 0: the window's entry w1 + t - k
                first = 1.0 if ids is None else (ids[:, t] == ids[:, 0]).double()[:, None]
                pre[:, :, t] += wk[:, 0] * s["init"][:, :, w1 + t - k] * first
    sig = 1 / (1 + torch.exp(-pre))
    dpre = s["dout"] * (sig + pre * sig * (1 - sig))
    dx, dw = torch.zeros_like(pre), torch.zeros_like(s["w"])
    dinit = torch.zeros_like(s["init"]) if s["init"] is not None else None
    for k in range(w1 + 1):
        wk = s["w"][:, w1 - k, None]
        if k < l:
            m = dpre[:, :, k:] * meets(k, k)
            dx[:, :, :l - k] += wk * m
            dw[:, w1 - k] += (m * s["x"][:, :, :l - k]).sum((0, 2))
        if dinit is not None:
            for t in range(min(k, l)):
                first = 1.0 if ids is None else (ids[:, t] == ids[:, 0]).double()[:, None]
                dinit[:, :, w1 + t - k] += wk[:, 0] * dpre[:, :, t] * first
                dw[:, w1 - k] += (dpre[:, :, t] * first * s["init"][:, :, w1 + t - k]).sum(0)
    if s["dfinal"] is not None:
        for j in range(w1):
            t = l - w1 + j
            same = 1.0 if ids is None else (ids[:, max(t, 0)] == ids[:, -1]).double()[:, None]
            if t >= 0:
                dx[:, :, t] += s["dfinal"][:, :, j] * same
            elif dinit is not None:
                dinit[:, :, w1 + t] += s["dfinal"][:, :, j] * same
    out = dict(dx=dx, dw=dw, dbias=dpre.sum((0, 2)))
    if dinit is not None:
        out["dconv_init"] = dinit
    return out
