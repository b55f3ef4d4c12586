"""Cases of linear attention with decays, the norm behind it and the maps of a serving batch, with their plain forms.

Six operators:
  step        ss.linattn_step: one token of many requests, linear attention with a decay
              for each head, over a pool of state slots
  prompt      ss.linattn_prompt: the same of packed prompts, from and into state slots
  train       ss.linattn_fwd and ss.linattn_bwd: a training step's forward and gradients
  norm        ss.group_norm: every token's channels normalised in groups, with a gate or
              an activation
  norm_train  ss.group_norm and ss.group_norm_bwd: the same with its gradients
  pack        ss.pack_requests: rows, sequences and slots of a serving batch from its
              requests' lengths

``run`` computes them in plain torch operations in 32 bits (``own`` false) or through
the library (``own`` true); ``exact`` evaluates their definitions, token by token where
there is a state, in 64 bits.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
Q = 64          # steps of a chunk of the plain form
EPS = 1e-5


def listed():
    return [
        # one request decoding alone: pure latency (a layer of 12 heads of 128)
        dict(name="token, one request", op="step", n=1, heads=12, kv=12, dk=128, dv=128, io="bf16", slots=16, pad=0),
        # a serving batch of an odd size, some of its rows padding of a captured loop
        dict(name="tokens, 201 requests", op="step", n=201, heads=16, kv=16, dk=128, dv=64, io="f16", slots=256, pad=3),
        # short prompts: a few tokens each, latency counts
        dict(name="prompts, short", op="prompt", tokens=131, seqs=5, tail=0, heads=12, kv=12, dk=128, dv=128,
             io="bf16", slots=16, carried=False),
        # a prefill batch of ragged prompts, some continued from their states, a few unused rows behind the last
        dict(name="prompts, ragged", op="prompt", tokens=16384, seqs=24, tail=5, heads=12, kv=12, dk=128, dv=128,
             io="bf16", slots=64, carried=True),
        # one long prompt, an odd length, four heads to a key and value
        dict(name="prompt, long", op="prompt", tokens=32769, seqs=1, tail=0, heads=16, kv=4, dk=64, dv=128, io="f16",
             slots=4, carried=True),
        # a training step of a layer: rows of one length
        dict(name="training, layer", op="train", batch=8, seqlen=2048, docs=0, heads=12, kv=12, dk=128, dv=128,
             io="bf16", state=False),
        # packed documents of odd lengths, shared keys and values, pieces chained through their states
        dict(name="training, packed", op="train", batch=1, seqlen=2003, docs=6, heads=8, kv=4, dk=64, dv=128, io="f16",
             state=True),
        # the gated norm of a Mamba-2 layer's decode batch (one group of 1536 channels, the gate before the norm)
        dict(name="norm, 64 tokens", op="norm", rows=64, dim=1536, groups=1, io="bf16", mode="gate_first", center=False,
             bias=False),
        # the norm behind linear attention in a training step: a group for each head, the gate behind the norm
        dict(name="norm training, layer", op="norm_train", rows=16384, dim=1536, groups=12, io="bf16", mode="gate",
             center=True, bias=True),
        # odd rows and groups in fp32 with an activation
        dict(name="norm training, odd", op="norm_train", rows=4097, dim=700, groups=7, io="f32", mode="silu",
             center=True, bias=True),
        # the maps of a decode batch that takes in a few prompts
        dict(name="maps, 64 requests", op="pack", requests=64, tokens=2048),
        # and of the largest batches
        dict(name="maps, 4001 requests", op="pack", requests=4001, tokens=65536),
    ]


def _logint(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["step", "prompt", "prompt", "train", "train", "norm", "norm_train", "pack"])
    io = rng.choice(["bf16", "f16"])
    if op == "pack":
        return dict(op=op, requests=_logint(rng, 1, 4000), tokens=_logint(rng, 16, 65000))
    if op in ("norm", "norm_train"):
        groups = rng.choice([1, 2, 4, 8, 12, 24])
        # whole vectors of channels more often than not, as models have them
        dim = groups * (8 * _logint(rng, 2, 4096 // groups // 8) if rng.random() < 0.7 else _logint(rng, 7, 4000 // groups))
        return dict(op=op, rows=_logint(rng, 1, min(16000, 20000000 // dim)), dim=dim, groups=groups,
                    io=rng.choice(["bf16", "f16", "f32"]), mode=rng.choice(["plain", "silu", "gate", "gate_first"]),
                    center=rng.random() < 0.5, bias=rng.random() < 0.5)
    heads = rng.choice([2, 4, 8, 12, 16, 32])
    shape = dict(heads=heads, kv=heads // rng.choice([1, 1, 1, 2]), dk=rng.choice([64, 128]), dv=rng.choice([64, 128]))
    most = 16000 * 12 // heads
    if op == "step":
        n = _logint(rng, 1, 190)
        return dict(op=op, n=n, **shape, io=io, slots=n + rng.randint(0, 9), pad=rng.choice([0, 1]) if n > 1 else 0)
    if op == "prompt":
        t = _logint(rng, 1, min(most, 32000))
        return dict(op=op, tokens=t, seqs=_logint(rng, 1, min(t, 64)), tail=rng.choice([0, 0, 7]), **shape, io=io,
                    slots=80, carried=rng.random() < 0.5)
    b = rng.randint(1, 4)
    l = _logint(rng, 1, most // b)
    return dict(op=op, batch=b, seqlen=l, docs=_logint(rng, 1, min(b * l, 20)) if rng.random() < 0.5 else 0, **shape,
                io=io, state=rng.random() < 0.5)


# ---- inputs -------------------------------------------------------------------


class _Rand:
    def __init__(self, seed):
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(int(seed))

    def normal(self, *shape, scale=1.0, dtype=torch.float32):
        return (torch.randn(*shape, generator=self.g, device="cuda") * scale).to(dtype)

    def uniform(self, lo, hi, *shape):
        return torch.rand(*shape, generator=self.g, device="cuda") * (hi - lo) + lo

    def integers(self, lo, hi, *shape):
        return torch.randint(lo, hi, shape, generator=self.g, device="cuda", dtype=torch.int32)

    def perm(self, n):
        return torch.randperm(n, generator=self.g, device="cuda")

    def cuts(self, total, parts):
        """parts + 1 increasing int32 offsets from 0 to total, every part at least 1 long."""
        inner = torch.randperm(total - 1, generator=self.g, device="cuda")[:parts - 1].sort().values + 1
        ends = torch.tensor([0, total], device="cuda")
        return torch.cat([ends[:1], inner, ends[1:]]).to(torch.int32)


def _qkv(r, c, *rows):
    """q, k and v as the columns of one projection's output rows."""
    nq, nk, nv = c["heads"] * c["dk"], c["kv"] * c["dk"], c["kv"] * c["dv"]
    row = r.normal(*rows, nq + nk + nv, dtype=DT[c["io"]])
    return dict(q=row[..., :nq].unflatten(-1, (c["heads"], c["dk"])),
                k=row[..., nq:nq + nk].unflatten(-1, (c["kv"], c["dk"])),
                v=row[..., nq + nk:].unflatten(-1, (c["kv"], c["dv"])),
                # decays from exp(-0.7) down to exp(-2^-12): memories of a few tokens to thousands
                log_decay=-torch.exp(r.uniform(math.log(2.0 ** -12), math.log(0.7), c["heads"])),
                scale=c["dk"] ** -0.5)


def prepare(case, seed):
    c, r = case, _Rand(seed)
    s = dict(case=dict(c))
    if c["op"] in ("step", "prompt"):
        io = DT[c["io"]]
        rows = c["n"] if c["op"] == "step" else c["tokens"] + c["tail"]
        n = rows if c["op"] == "step" else c["seqs"]
        s.update(_qkv(r, c, rows))
        s.update(state=r.normal(c["slots"], c["heads"], c["dv"], c["dk"], scale=0.5),
                 slots=r.perm(c["slots"])[:n].to(torch.int32),
                 y=torch.zeros(rows, c["heads"], c["dv"], dtype=io, device="cuda"))
        if c["op"] == "step":
            if c["pad"]:
                s["slots"][n - c["pad"]:] = -1
        else:
            s["cu"] = r.cuts(c["tokens"], c["seqs"])
            s["has"] = (r.perm(c["seqs"]) % 2 == 0).to(torch.int32) if c["carried"] else None
    elif c["op"] == "train":
        b, l = c["batch"], c["seqlen"]
        s.update(_qkv(r, c, b, l))
        s.update(cu=r.cuts(b * l, c["docs"]) if c["docs"] else None,
                 dy=r.normal(b, l, c["heads"], c["dv"], dtype=DT[c["io"]]))
        st = (c["docs"] or b, c["heads"], c["dv"], c["dk"])
        s.update(h0=r.normal(*st, scale=0.5) if c["state"] else None, dfinal=r.normal(*st, scale=0.1) if c["state"] else None)
    elif c["op"] in ("norm", "norm_train"):
        io, shape = DT[c["io"]], (c["rows"], c["dim"])
        s.update(x=r.normal(*shape, scale=2.0, dtype=io), weight=1.0 + r.normal(c["dim"], scale=0.2),
                 bias=r.normal(c["dim"], scale=0.2) if c["bias"] else None,
                 z=r.normal(*shape, dtype=io) if c["mode"].startswith("gate") else None,
                 dy=r.normal(*shape, dtype=io) if c["op"] == "norm_train" else None)
    else:
        n = c["requests"]
        # two thirds decode one token, some are idle, the others are prompts, new ones or the next piece of one
        kind, long = r.uniform(0.0, 1.0, n), torch.exp(r.uniform(0.0, math.log(2048.0), n)).to(torch.int32)
        seen = r.integers(1, 4096, n)
        s.update(new_tokens=torch.where(kind < 0.66, torch.ones_like(long), torch.where(kind < 0.75, torch.zeros_like(long), long)),
                 seen=torch.where((kind < 0.66) | (kind > 0.9), seen, torch.zeros_like(seen)),
                 slots=torch.where(r.uniform(0.0, 1.0, n) < 0.97, r.perm(n).to(torch.int32), -torch.ones_like(seen)))
    return s


# ---- one pass -----------------------------------------------------------------


def run(state):
    s = state
    if own:
        return _run_own(s)
    return {"step": _plain_step, "prompt": _plain_prompt, "train": _plain_train, "norm": _plain_norm,
            "norm_train": _plain_norm_train, "pack": _plain_pack}[s["case"]["op"]](s)


def _norm_args(s):
    c = s["case"]
    return dict(ngroups=c["groups"], bias=s["bias"], z=s["z"], eps=EPS, center=c["center"], silu=c["mode"] == "silu",
                gate_first=c["mode"] == "gate_first")


def _run_own(s):
    from mamba_selective_scan_fwd_amd import ss
    op = s["case"]["op"]
    if op == "step":
        y = ss.linattn_step(s["q"], s["k"], s["v"], s["log_decay"], s["state"], scale=s["scale"], slots=s["slots"],
                            y=s["y"])
        return dict(y=y, state=s["state"])
    if op == "prompt":
        y = ss.linattn_prompt(s["q"], s["k"], s["v"], s["log_decay"], s["cu"], s["state"], scale=s["scale"],
                              slots=s["slots"], has_state=s["has"], y=s["y"])
        return dict(y=y, state=s["state"])
    if op == "train":
        a = (s["q"], s["k"], s["v"], s["log_decay"])
        keep = s["case"]["state"]
        y = ss.linattn_fwd(*a, scale=s["scale"], cu_seqlens=s["cu"], h0=s["h0"], return_final_state=keep)
        g = ss.linattn_bwd(*a, s["dy"], scale=s["scale"], cu_seqlens=s["cu"], h0=s["h0"], dfinal=s["dfinal"],
                           want_dh0=keep)
        return dict(g, y=y[0], final=y[1]) if keep else dict(g, y=y)
    if op == "norm":
        return ss.group_norm(s["x"], s["weight"], **_norm_args(s))
    if op == "norm_train":
        y = ss.group_norm(s["x"], s["weight"], **_norm_args(s))
        return dict(ss.group_norm_bwd(s["x"], s["weight"], s["dy"], **_norm_args(s)), y=y)
    return ss.pack_requests(s["new_tokens"], s["slots"], s["seen"], s["case"]["tokens"])


# ---- plain forms ----------------------------------------------------------------


def _silu(v):
    return v * torch.sigmoid(v)


def _plain_step(s):
    c = s["case"]
    rows = torch.arange(c["n"], device="cuda") if not c["pad"] else (s["slots"] >= 0).nonzero()[:, 0]
    slots = s["slots"][rows].long()
    rep = c["heads"] // c["kv"]
    q = s["q"][rows].float() * s["scale"]
    k, v = (s[n][rows].float().repeat_interleave(rep, 1) for n in ("k", "v"))
    decay = torch.exp(s["log_decay"].double()).float()
    st = s["state"][slots] * decay[:, None, None] + v[..., None] * k[:, :, None, :]
    s["state"][slots] = st
    s["y"][rows] = (st * q[:, :, None, :]).sum(3).to(s["y"].dtype)
    return dict(y=s["y"], state=s["state"])


def _chunked(q, k, v, log_decay, cu, init):
    """Linear attention with decays of packed sequences in chunks of Q steps.  q, k (T, H, dk), v (T, H, dv) in 32
    bits, cu (S + 1), init (S, H, dv, dk).  Returns y (T, H, dv) and the states (S, H, dv, dk).  Sequence s owns the
    chunks from cu[s] // Q + s on, the ones behind its last step stay empty."""
    total, heads, dk = q.shape
    dv, seqs = v.shape[2], cu.numel() - 1
    cu = cu.long()
    t = torch.arange(total, device="cuda")
    seq = (torch.searchsorted(cu, t, right=True) - 1).clamp(0, seqs - 1)
    pos, used = t - cu[seq], t < cu[-1]
    nchunk = total // Q + seqs
    first = cu[:-1] // Q + torch.arange(seqs, device="cuda")
    at = torch.where(used, (first[seq] + pos // Q) * Q + pos % Q, nchunk * Q)

    def lay(x):
        out = torch.zeros((nchunk + 1) * Q, *x.shape[1:], dtype=x.dtype, device="cuda").index_copy(0, at, x)
        return out[:nchunk * Q].view(nchunk, Q, heads, -1).permute(0, 2, 1, 3)       # (V, H, Q, d)

    qs, ks, vs = lay(q), lay(k), lay(v)
    # decays in 64 bits: of far positions
    live = torch.zeros((nchunk + 1) * Q, dtype=torch.float64, device="cuda").index_copy(0, at, used.double())
    run = (live[:nchunk * Q].view(nchunk, 1, Q).cumsum(2) * log_decay.double()[:, None])  # (V, H, Q)
    steps = torch.arange(Q, device="cuda")
    low = steps[:, None] >= steps
    decay = torch.exp((run[..., :, None] - run[..., None, :]).masked_fill(~low, -math.inf)).float()
    y = ((qs @ ks.transpose(2, 3)) * decay) @ vs
    rest = torch.exp(run[..., -1:] - run).float()
    own_state = (vs * rest[..., None]).transpose(2, 3) @ ks                          # (V, H, dv, dk)
    # the state that enters each chunk, from all earlier chunks of its sequence and its first state
    total_log = run[..., -1].t().cumsum(1)                                           # (H, V)
    chunks = torch.arange(nchunk, device="cuda")
    owner = torch.searchsorted(first, chunks, right=True) - 1
    before = torch.cat([torch.zeros(heads, 1, dtype=torch.float64, device="cuda"), total_log[:, :-1]], 1)
    carried = (owner[:, None] == owner) & (chunks[:, None] > chunks)
    between = torch.exp((before[:, :, None] - total_log[:, None, :]).masked_fill(~carried, -math.inf)).float()
    enter = (between @ own_state.permute(1, 0, 2, 3).reshape(heads, nchunk, dv * dk)).view(heads, nchunk, dv, dk)
    enter = enter.permute(1, 0, 2, 3)
    enter = enter + torch.exp(before - before[:, first[owner]]).float().t()[..., None, None] * init[owner]
    y = y + (qs * torch.exp(run).float()[..., None]) @ enter.transpose(2, 3)
    ends = torch.cat([first[1:], first.new_full((1,), nchunk)]) - 1
    leave = own_state[ends] + torch.exp(run[ends][..., -1]).float()[..., None, None] * enter[ends]
    flat = torch.cat([y.permute(0, 2, 1, 3).reshape(nchunk * Q, heads, dv), y.new_zeros(1, heads, dv)])
    return flat[at], leave


def _plain_prompt(s):
    c = s["case"]
    slots, rep = s["slots"].long(), c["heads"] // c["kv"]
    init = s["state"][slots]
    init = init * s["has"].float()[:, None, None, None] if s["has"] is not None else torch.zeros_like(init)
    k, v = (s[n].float().repeat_interleave(rep, 1) for n in ("k", "v"))
    y, last = _chunked(s["q"].float() * s["scale"], k, v, s["log_decay"], s["cu"], init)
    used = torch.arange(y.shape[0], device="cuda") < s["cu"][-1]
    s["y"].copy_(torch.where(used[:, None, None], y.to(s["y"].dtype), s["y"]))
    s["state"][slots] = last
    return dict(y=s["y"], state=s["state"])


def _plain_train(s):
    c = s["case"]
    b, l, rep = c["batch"], c["seqlen"], c["heads"] // c["kv"]
    cu = s["cu"] if s["cu"] is not None else torch.arange(b + 1, device="cuda") * l
    leaves = {k: s[k].detach().float().requires_grad_() for k in ("q", "k", "v", "h0") if s[k] is not None}
    init = leaves["h0"] if s["h0"] is not None else torch.zeros(cu.numel() - 1, c["heads"], c["dv"], c["dk"], device="cuda")
    k, v = (leaves[n].flatten(0, 1).repeat_interleave(rep, 1) for n in ("k", "v"))
    y, last = _chunked(leaves["q"].flatten(0, 1) * s["scale"], k, v, s["log_decay"], cu, init)
    outs, grads = [y], [s["dy"].flatten(0, 1).float()]
    if s["dfinal"] is not None:
        outs.append(last)
        grads.append(s["dfinal"])
    g = dict(zip(leaves, torch.autograd.grad(outs, list(leaves.values()), grads)))
    out = {"d" + k: v.to(s[k].dtype) for k, v in g.items()}
    out["y"] = y.detach().to(s["q"].dtype).view(b, l, c["heads"], c["dv"])
    if c["state"]:
        out["final"] = last.detach()
    return out


def _plain_norm_of(x, weight, bias, z, c):
    u = x * _silu(z) if c["mode"] == "gate_first" else x
    u = u.unflatten(-1, (c["groups"], -1))
    if c["center"]:
        u = u - u.mean(-1, keepdim=True)
    n = (u * torch.rsqrt((u * u).mean(-1, keepdim=True) + EPS)).flatten(-2)
    o = n * weight
    if bias is not None:
        o = o + bias
    return _silu(o) if c["mode"] == "silu" else o * _silu(z) if c["mode"] == "gate" else o


def _plain_norm(s):
    z = s["z"].float() if s["z"] is not None else None
    return _plain_norm_of(s["x"].float(), s["weight"], s["bias"], z, s["case"]).to(s["x"].dtype)


def _plain_norm_train(s):
    c = s["case"]
    x, dy = s["x"].float(), s["dy"].float()
    z = s["z"].float() if s["z"] is not None else None
    sz = torch.sigmoid(z) if z is not None else None
    dsilu = sz * (1 + z * (1 - sz)) if z is not None else None
    u = (x * z * sz if c["mode"] == "gate_first" else x).unflatten(-1, (c["groups"], -1))
    if c["center"]:
        u = u - u.mean(-1, keepdim=True)
    rstd = torch.rsqrt((u * u).mean(-1, keepdim=True) + EPS)
    n = u * rstd
    o = n.flatten(-2) * s["weight"]
    if s["bias"] is not None:
        o = o + s["bias"]
    out, do = {}, dy
    if c["mode"] == "silu":
        so = torch.sigmoid(o)
        y, do = o * so, dy * so * (1 + o * (1 - so))
    elif c["mode"] == "gate":
        y, do = o * z * sz, dy * z * sz
        out["dz"] = (dy * o * dsilu).to(s["x"].dtype)
    else:
        y = o
    # long sums in 64 bits
    out["dweight"] = (do * n.flatten(-2)).sum(0, dtype=torch.float64).float()
    if s["bias"] is not None:
        out["dbias"] = do.sum(0, dtype=torch.float64).float()
    dn = (do * s["weight"]).unflatten(-1, (c["groups"], -1))
    du = dn - n * (dn * n).mean(-1, keepdim=True)
    if c["center"]:
        du = du - dn.mean(-1, keepdim=True)
    du = (du * rstd).flatten(-2)
    if c["mode"] == "gate_first":
        out["dz"] = (du * x * dsilu).to(s["x"].dtype)
        du = du * z * sz
    return dict(out, y=y.to(s["x"].dtype), dx=du.to(s["x"].dtype))


def _plain_pack(s):
    most, n = s["case"]["tokens"], s["new_tokens"].numel()
    live = (s["slots"] >= 0) & (s["new_tokens"] > 0)
    step = live & (s["new_tokens"] == 1) & (s["seen"] > 0)
    want = torch.where(live, s["new_tokens"], torch.zeros_like(s["new_tokens"])).long()
    one, rest = torch.where(step, want, torch.zeros_like(want)), torch.where(step, torch.zeros_like(want), want)
    steps = one.sum()
    start = torch.where(step, one.cumsum(0) - one, steps + rest.cumsum(0) - rest).clamp(max=most)
    taken = torch.minimum(want, most - start)
    has = taken > 0
    prompt = has & ~step
    i32 = torch.int32
    none = torch.full((n + 1,), -1, dtype=torch.int64, device="cuda")

    def listing(which, values, fill):
        at = torch.where(which, which.long().cumsum(0) - 1, n)
        return torch.full_like(none, fill).index_copy(0, at, values.long())[:n]

    # the place n takes what is not listed
    total = torch.minimum(want.sum(), torch.full_like(steps, most))
    first = listing(prompt, start, 0)
    count = prompt.sum()
    index = torch.arange(n + 1, device="cuda")
    cu = torch.where(index < count, torch.cat([first, first[:1]]), total)
    t = torch.arange(most, device="cuda")
    # requests in the order of their rows: the steps, then the prompts
    order = torch.argsort(torch.where(has, start, most + index[:n]))
    ends = torch.where(has, start + taken, torch.full_like(start, most + 1))[order]
    owner = order[torch.searchsorted(ends, t, right=True).clamp(max=n - 1)]
    inside = t < total
    return dict(rows=torch.where(has, start, none[:n]).to(i32), taken=taken.to(i32),
                step_slots=listing(step & has, s["slots"], -1).to(i32), cu_seqlens=cu.to(i32),
                prompt_slots=listing(prompt, s["slots"], -1).to(i32),
                has_state=listing(prompt, s["seen"] > 0, 0).to(i32),
                row_request=torch.where(inside, owner, -1).to(i32),
                row_position=torch.where(inside, s["seen"][owner].clamp(min=0) + t - start[owner], -1).to(i32))


# ---- work -----------------------------------------------------------------------


def work(case):
    c = case
    if c["op"] == "pack":
        return dict(bytes=4 * (12 * c["requests"] + 2 * c["tokens"]), flops=8 * c["requests"] + 4 * c["tokens"])
    e = 4 if c["io"] == "f32" else 2
    if c["op"] in ("norm", "norm_train"):
        n, gated = c["rows"] * c["dim"], c["mode"].startswith("gate")
        byt, flops = e * n * (3 if gated else 2) + 8 * c["dim"], 12 * n
        if c["op"] == "norm_train":     # x, z, dy read once for both directions; y, dx and dz written
            byt, flops = e * n * (6 if gated else 4) + 16 * c["dim"], 40 * n
        return dict(bytes=byt, flops=flops)
    hk, hv, kk, kv = c["heads"] * c["dk"], c["heads"] * c["dv"], c["kv"] * c["dk"], c["kv"] * c["dv"]
    per_state = c["heads"] * c["dk"] * c["dv"]
    if c["op"] == "step":
        n = c["n"] - c["pad"]
        return dict(bytes=8 * n * per_state + e * n * (hk + hv + kk + kv) + 4 * c["heads"] + 4 * c["n"],
                    flops=5 * n * per_state)
    if c["op"] == "prompt":
        return dict(bytes=e * c["tokens"] * (hk + hv + kk + kv) + 4 * c["seqs"] * per_state * (2 if c["carried"] else 1) +
                    4 * c["heads"], flops=4 * c["tokens"] * per_state)
    t = c["batch"] * c["seqlen"]
    # q, k, v and dy read, y and three gradients written; the states, their gradients and four products with them
    return dict(bytes=2 * e * t * (hk + hv + kk + kv) + (16 * (c["docs"] or c["batch"]) * per_state if c["state"] else 0) +
                4 * c["heads"], flops=14 * t * per_state)


# ---- the definitions in 64 bits ---------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    s = {k: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v for k, v in s.items()}
    with torch.no_grad():
        return {"step": _exact_step, "prompt": _exact_prompt, "train": _exact_train, "norm": _exact_norm,
                "norm_train": _exact_norm_train, "pack": _exact_pack}[case["op"]](s)


def _head_of(c):
    return torch.arange(c["heads"], device="cuda") // (c["heads"] // c["kv"])


def _exact_step(s):
    kv, a = _head_of(s["case"]), torch.exp(s["log_decay"]).view(-1, 1, 1)
    for i, slot in enumerate(s["slots"].tolist()):
        if slot < 0:
            continue
        st = a * s["state"][slot] + torch.einsum("hp,hn->hpn", s["v"][i][kv], s["k"][i][kv])
        s["state"][slot] = st
        s["y"][i] = s["scale"] * torch.einsum("hpn,hn->hp", st, s["q"][i])
    return dict(y=s["y"], state=s["state"])


def _walk(s, q, k, v, cu, st, y):
    """Every sequence step by step, all of them at once; st (S, H, dv, dk) becomes their last states."""
    kv, a = _head_of(s["case"]), torch.exp(s["log_decay"]).view(-1, 1, 1)
    cu = cu.long()
    lens = cu[1:] - cu[:-1]
    order = torch.argsort(lens, descending=True)
    counts = torch.bincount(lens, minlength=int(lens.max()) + 1).flip(0).cumsum(0).flip(0).tolist()  # lens >= t
    first, now = cu[:-1][order], st[order]
    for t in range(int(lens.max())):
        n = counts[t + 1]                                   # sequences that have a step t
        row = first[:n] + t
        now[:n] *= a
        now[:n] += v[row][:, kv][..., None] * k[row][:, kv][:, :, None, :]
        y[row] = s["scale"] * torch.matmul(now[:n], q[row][..., None])[..., 0]
    st[order] = now


def _exact_prompt(s):
    slots = s["slots"].long()
    st = s["state"][slots]
    st = st * s["has"].double().view(-1, 1, 1, 1) if s["has"] is not None else torch.zeros_like(st)
    _walk(s, s["q"], s["k"], s["v"], s["cu"], st, s["y"])
    s["state"][slots] = st
    return dict(y=s["y"], state=s["state"])


def _exact_train(s):
    """dq from the states forward; dk and dv from the gradient G of the state walked backward:
    G_t = a G_{t+1} + scale dy_t q_t^T (and dfinal behind the last step), dk_t = G_t^T v_t, dv_t = G_t k_t."""
    c = s["case"]
    b, l, kv = c["batch"], c["seqlen"], _head_of(c)
    cu = s["cu"].tolist() if s["cu"] is not None else [i * l for i in range(b + 1)]
    q, k, v, dy = (s[n].flatten(0, 1) for n in ("q", "k", "v", "dy"))
    a = torch.exp(s["log_decay"]).view(-1, 1, 1)
    shape = (len(cu) - 1, c["heads"], c["dv"], c["dk"])
    f64 = dict(dtype=torch.float64, device="cuda")
    h0 = s["h0"] if s["h0"] is not None else torch.zeros(shape, **f64)
    g0 = s["dfinal"] if s["dfinal"] is not None else torch.zeros(shape, **f64)
    y, dq, dk, dv = torch.zeros_like(dy), torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    lens = [e - f for f, e in zip(cu, cu[1:])]
    begin, ln = torch.tensor(cu[:-1], device="cuda"), torch.tensor(lens, device="cuda")
    order = sorted(range(len(lens)), key=lambda i: -lens[i])
    dev = torch.tensor(order, device="cuda")
    st, gr = h0[dev].clone(), g0[dev].clone()
    first, last = begin[dev], (begin + ln)[dev] - 1
    n, rep = len(order), c["heads"] // c["kv"]
    for t in range(max(lens)):
        while n and lens[order[n - 1]] <= t:
            n -= 1
        row = first[:n] + t
        st[:n] = a * st[:n] + v[row][:, kv][..., None] * k[row][:, kv][:, :, None, :]
        y[row] = s["scale"] * torch.matmul(st[:n], q[row][..., None])[..., 0]
        dq[row] = s["scale"] * torch.matmul(dy[row][:, :, None, :], st[:n])[:, :, 0]
        row = last[:n] - t
        if t:
            gr[:n] = a * gr[:n]
        gr[:n] += s["scale"] * dy[row][..., None] * q[row][:, :, None, :]
        # a key's and value's gradients add up over the heads that share them
        dk[row] = torch.matmul(v[row][:, kv][:, :, None, :], gr[:n])[:, :, 0].unflatten(1, (c["kv"], rep)).sum(2)
        dv[row] = torch.matmul(gr[:n], k[row][:, kv][..., None])[..., 0].unflatten(1, (c["kv"], rep)).sum(2)
    out = {n: x.view(b, l, *x.shape[1:]) for n, x in (("y", y), ("dq", dq), ("dk", dk), ("dv", dv))}
    if c["state"]:
        out["final"], out["dh0"] = torch.empty_like(st), torch.empty_like(gr)
        out["final"][dev], out["dh0"][dev] = st, a * gr
    return out


def _exact_norm(s):
    with torch.no_grad():
        return _norm_formula(s, s["x"], s["weight"], s["bias"], s["z"])


def _norm_formula(s, x, w, b, z):
    c = s["case"]
    if c["mode"] == "gate_first":
        x = x * z / (1 + torch.exp(-z))
    parts = []
    for u in x.split(c["dim"] // c["groups"], 1):
        mean = u.sum(1, keepdim=True) / u.shape[1] if c["center"] else 0.0
        parts.append((u - mean) / torch.sqrt(((u - mean) ** 2).sum(1, keepdim=True) / u.shape[1] + EPS))
    o = torch.cat(parts, 1) * w + (b if b is not None else 0.0)
    if c["mode"] == "silu":
        o = o / (1 + torch.exp(-o))
    return o * z / (1 + torch.exp(-z)) if c["mode"] == "gate" else o


def _exact_norm_train(s):
    names = [n for n in ("x", "weight", "bias", "z") if s[n] is not None]
    with torch.enable_grad():
        leaves = {n: s[n].detach().requires_grad_() for n in names}
        y = _norm_formula(s, *(leaves.get(n) for n in ("x", "weight", "bias", "z")))
        g = torch.autograd.grad(y, [leaves[n] for n in names], s["dy"])
    return dict({"d" + n: v for n, v in zip(names, g)}, y=y.detach())


def _exact_pack(s):
    most = s["case"]["tokens"]
    new, slots, seen = s["new_tokens"].tolist(), s["slots"].tolist(), s["seen"].tolist()
    n = len(new)
    out = dict(rows=[-1] * n, taken=[0] * n, step_slots=[], cu_seqlens=[], prompt_slots=[], has_state=[], row_request=[],
               row_position=[])
    at = 0
    for prompts in (False, True):
        for i in range(n):
            if slots[i] < 0 or new[i] <= 0 or (new[i] == 1 and seen[i] > 0) == prompts or at >= most:
                continue
            take = min(new[i], most - at)
            out["rows"][i], out["taken"][i] = at, take
            if prompts:
                out["cu_seqlens"].append(at)
                out["prompt_slots"].append(slots[i])
                out["has_state"].append(int(seen[i] > 0))
            else:
                out["step_slots"].append(slots[i])
            out["row_request"] += [i] * take
            out["row_position"] += range(max(seen[i], 0), max(seen[i], 0) + take)
            at += take
    fill = dict(step_slots=(-1, n), cu_seqlens=(at, n + 1), prompt_slots=(-1, n), has_state=(0, n),
                row_request=(-1, most), row_position=(-1, most))
    for k, (v, size) in fill.items():
        out[k] += [v] * (size - len(out[k]))
    return {k: torch.tensor(v, dtype=torch.int32, device="cuda") for k, v in out.items()}
