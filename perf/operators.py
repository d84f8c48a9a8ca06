"""Cases and plain forms of the sequence-attention and optimizer operators.

Three groups: the per-head norm of queries and keys with the position rotation, attention with a
learned relative-position bias by buckets (forward, training step, single tokens against a cache), and
the AdamW step over many tensors (moments in 32 or in 8 bits). ``run`` computes a case in elementary
torch operations, or with ``own`` through the framework's entry points.
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
EPS = 1e-6
BLOCK = 256  # elements that share one scale of the 8-bit moments
LR, BETA1, BETA2, ADAM_EPS, STEP = 1e-3, 0.9, 0.999, 1e-8, 10
EXCLUDE = -1e30  # a bias at or below this takes its key out


# ---------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one new token of each of 8 sequences in a decoding step: latency
        dict(name="norm_token", op="norm", B=8, L=1, hq=12, hk=12, d=64, rot=64, pairs="half", dtype="bf16",
             train=False, positions=True),
        # q and k of the token grid 16 x 14 x 14 of a batch of clips, 12 heads of 32 (stage 3 of the small model)
        dict(name="norm_grid", op="norm", B=32, L=3136, hq=12, hk=12, d=32, rot=32, pairs="half", dtype="bf16",
             train=False, positions=False),
        # a training step with shared key heads, half of the channels rotated, an odd length
        dict(name="norm_train", op="norm", B=4, L=4099, hq=16, hk=4, d=128, rot=64, pairs="interleaved",
             dtype="fp16", train=True, positions=False),
        # one (8, 7, 7) window's tokens as a short sequence, 3 heads of 32
        dict(name="attn_window", op="attn", B=2, Lq=392, Lk=392, hq=3, hk=3, d=32, causal=False, ragged=False,
             buckets=32, distance=128, dtype="bf16", train=False),
        # full attention over the 16 x 14 x 14 grid of four clips
        dict(name="attn_grid", op="attn", B=4, Lq=3136, Lk=3136, hq=12, hk=12, d=32, causal=False, ragged=False,
             buckets=32, distance=128, dtype="bf16", train=False),
        # a long causal sequence with shared key heads of width 128
        dict(name="attn_causal", op="attn", B=1, Lq=8192, Lk=8192, hq=16, hk=4, d=128, causal=True, ragged=False,
             buckets=64, distance=512, dtype="fp16", train=False),
        # one new token of 16 sequences against caches of up to 16384 tokens
        dict(name="attn_token", op="attn", B=16, Lq=1, Lk=16384, hq=16, hk=4, d=64, causal=True, ragged=True,
             buckets=32, distance=128, dtype="bf16", train=False),
        # a training step on a padded batch of short sequences of odd length
        dict(name="attn_train_padded", op="attn", B=8, Lq=577, Lk=577, hq=6, hk=6, d=64, causal=False, ragged=True,
             buckets=32, distance=128, dtype="bf16", train=True),
        # a training step on long causal sequences
        dict(name="attn_train_long", op="attn", B=2, Lq=4096, Lk=4096, hq=12, hk=12, d=64, causal=True,
             ragged=False, buckets=32, distance=128, dtype="bf16", train=True),
        # the parameters of one block of width 96: an optimizer step of few small tensors
        dict(name="adamw_block", op="adamw", C=96, blocks=1, bits=32, master=False, grads="fp32"),
        # 14 blocks of width 384 (25 million parameters), with fp32 copies of the bf16 weights
        dict(name="adamw_model", op="adamw", C=384, blocks=14, bits=32, master=True, grads="fp32"),
        # 20 blocks of width 512 (63 million parameters), moments in 8 bits, read out in bf16 after the step
        dict(name="adamw_model_8bit", op="adamw", C=512, blocks=20, bits=8, master=False, grads="bf16"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "attn", "attn", "attn", "adamw"])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    if op == "norm":
        hk = rng.choice([1, 2, 3, 4, 8, 12])
        hq = hk * rng.choice([1, 1, 2, 4])
        d = rng.choice([32, 64, 96, 128])
        B = _log_int(rng, 1, 32)
        tokens = _log_int(rng, 1, max(1, 38_000_000 // ((hq + hk) * d)))
        return dict(op="norm", B=B, L=max(1, tokens // B), hq=hq, hk=hk, d=d, rot=rng.choice([d, d, d // 2]),
                    pairs=rng.choice(["half", "interleaved"]), dtype=dtype, train=rng.random() < 0.5,
                    positions=rng.random() < 0.5)
    if op == "attn":
        hk = rng.choice([1, 2, 3, 4, 6, 8])
        hq = hk * rng.choice([1, 1, 2, 4])
        d = rng.choice([32, 64, 128])
        buckets, distance = rng.choice([(16, 64), (32, 128), (32, 128), (64, 512)])
        kind = rng.choice(["token", "forward", "train", "train"])
        case = dict(op="attn", d=d, hq=hq, hk=hk, buckets=buckets, distance=distance, dtype=dtype)
        if kind == "token":
            B = _log_int(rng, 1, 32)
            Lk = _log_int(rng, 1, min(32768, max(64, 130_000_000 // (B * hk * d))))
            Lq = min(Lk, rng.choice([1, 1, 1, 2, 4]))
            return dict(case, B=B, Lq=Lq, Lk=Lk, causal=True, ragged=True, train=False)
        L = _log_int(rng, 1, 4500)
        B = _log_int(rng, 1, max(1, min(16, 600_000_000 // (L * L * hq))))
        return dict(case, B=B, Lq=L, Lk=L, causal=rng.random() < 0.5, ragged=rng.random() < 0.4,
                    train=kind == "train")
    C = 32 * rng.randint(1, 16)
    return dict(op="adamw", C=C, blocks=_log_int(rng, 1, max(1, min(24, 60_000_000 // (12 * C * C)))),
                bits=rng.choice([32, 8]), master=rng.random() < 0.5, grads=rng.choice(["fp32", "bf16"]))


# ---------------------------------------------------------------------------------------- inputs
def _normal(gen, shape, dtype, scale=1.0):
    x = torch.empty(shape, dtype=torch.float32, device="cuda").normal_(generator=gen)
    return (x * scale).to(dtype)


def _bucket_map(buckets, distance, bidirectional):
    """Bucket of each clipped offset key - query in [-distance, distance], as the layer's definition has it:
    half of a side's buckets for single distances, the others spaced by the logarithm up to `distance`."""
    side = buckets // 2 if bidirectional else buckets
    exact_n = side // 2
    n = torch.arange(-distance, distance + 1, dtype=torch.float64)
    away = n.abs() if bidirectional else (-n).clamp(min=0)
    far = torch.log(away.clamp(min=exact_n) / exact_n) / math.log(distance / exact_n) * (side - exact_n)
    far = (exact_n + torch.floor(far + 1e-9)).clamp(max=side - 1)
    b = torch.where(away < exact_n, away, far)
    if bidirectional:
        b = b + side * (n > 0)
    return b.to(torch.int32)


def _prepare_norm(case, gen):
    B, L, hq, hk, d, dt = case["B"], case["L"], case["hq"], case["hk"], case["d"], DTYPES[case["dtype"]]
    qkv = _normal(gen, (B, L, hq + 2 * hk, d), dt, 1.5)  # the projection's output: q, k and v heads of a token
    rows = max(L, 4096) if case["positions"] else L
    freq = 10000.0 ** (-torch.arange(case["rot"] // 2, dtype=torch.float64) * 2 / case["rot"])
    angle = torch.arange(rows, dtype=torch.float64)[:, None] * freq
    st = dict(case=case, q=qkv[:, :, :hq], k=qkv[:, :, hq:hq + hk],
              gq=_normal(gen, (d,), dt, 0.2) + 1, gk=_normal(gen, (d,), dt, 0.2) + 1,
              cos=angle.cos().float().cuda(), sin=angle.sin().float().cuda(), positions=None)
    if case["positions"]:
        st["positions"] = torch.randint(0, rows, (B, L), generator=gen, device="cuda", dtype=torch.int32)
    if case["train"]:
        st["dq"], st["dk"] = _normal(gen, (B, L, hq, d), dt), _normal(gen, (B, L, hk, d), dt)
    return st


def _prepare_attn(case, gen):
    B, Lq, Lk, hq, hk, d = (case[n] for n in ("B", "Lq", "Lk", "hq", "hk", "d"))
    dt = DTYPES[case["dtype"]]
    st = dict(case=case, scale=d ** -0.5, q_lens=None, kv_lens=None, q_start=None,
              table=_normal(gen, (case["buckets"], hq), dt, 0.5),
              map=_bucket_map(case["buckets"], case["distance"], not case["causal"]).cuda())
    if Lq == Lk:  # q, k and v are slices of one projection's output
        qkv = _normal(gen, (B, Lq, hq + 2 * hk, d), dt)
        st["q"], st["k"], st["v"] = qkv[:, :, :hq], qkv[:, :, hq:hq + hk], qkv[:, :, hq + hk:]
    else:  # new tokens against a cache
        st["q"] = _normal(gen, (B, Lq, hq, d), dt)
        st["k"], st["v"] = _normal(gen, (B, Lk, hk, d), dt), _normal(gen, (B, Lk, hk, d), dt)
    if case["ragged"]:
        lens = torch.randint(max(Lq if Lq < Lk else 1, Lk // 2), Lk + 1, (B,), generator=gen, device="cuda",
                             dtype=torch.int32)
        lens[0] = Lk
        st["kv_lens"] = lens
        if Lq == Lk:
            st["q_lens"] = lens
        else:
            st["q_start"] = lens - Lq
    elif Lq != Lk:
        st["q_start"] = torch.full((B,), Lk - Lq, device="cuda", dtype=torch.int32)
    if case["train"]:
        st["do"] = _normal(gen, (B, Lq, hq, d), dt)
    return st


def _block_sizes(C):
    """Parameters of a block of width C with heads of 32 and a (8, 7, 7) window: the attention half's norm, qkv,
    projection and table, then the MLP half's norm and layers; True where the weight decays."""
    return [((C,), False), ((C,), False), ((C, 3 * C), True), ((3 * C,), False), ((C, C), True), ((C,), False),
            ((2535, max(1, C // 32)), False), ((C,), False), ((C,), False), ((C, 4 * C), True), ((4 * C,), False),
            ((4 * C, C), True), ((C,), False)]


def _layout(case):
    """[(shape, decays, offset)] of every tensor in the flat buffers, and their length; each starts on a block."""
    out, at = [], 0
    for _ in range(case["blocks"]):
        for shape, decays in _block_sizes(case["C"]):
            out.append((shape, decays, at))
            at += -(-math.prod(shape) // BLOCK) * BLOCK
    return out, at


def _codes(m, scale, levels, root):
    x = m.abs() / torch.where(scale > 0, scale, torch.ones_like(scale))
    for _ in range(root):
        x = torch.sqrt(x)
    return torch.round(x * levels)


def _lut(levels, power):
    return (torch.arange(levels + 1, dtype=torch.float64) ** power / float(levels) ** power).float().cuda()


def _prepare_adamw(case, gen):
    tensors, n = _layout(case)
    live = torch.zeros(n, device="cuda")
    keep = torch.empty(n, device="cuda").fill_(1.0)
    for shape, decays, at in tensors:
        live[at:at + math.prod(shape)] = 1
        if decays:
            keep[at:at + math.prod(shape)] = 1 - LR * 0.05
    w = _normal(gen, (n,), torch.float32, 0.02) * live
    g = (_normal(gen, (n,), torch.float32, 1e-3) * live).to(torch.float32 if case["grads"] == "fp32" else torch.bfloat16)
    m, v = _normal(gen, (n,), torch.float32, 1e-3) * live, (_normal(gen, (n,), torch.float32, 1e-3) * live).square()
    st = dict(case=case, p=w.to(torch.bfloat16), master=w if case["master"] else None, g=g, keep=keep)
    if case["bits"] == 32:
        st["m"], st["v"] = m, v
    else:
        mb, vb = m.view(-1, BLOCK), v.view(-1, BLOCK)
        st["ms"], st["vs"] = mb.abs().amax(1), vb.amax(1)
        st["m"] = (_codes(mb, st["ms"][:, None], 127, 1) * mb.sign()).to(torch.int8).view(-1)
        c = _codes(vb, st["vs"][:, None], 255, 2)
        st["v"] = torch.where(vb > 0, c.clamp(min=1), c).to(torch.uint8).view(-1)
        st["lut_m"], st["lut_v"] = _lut(127, 2), _lut(255, 4)

    def views(flat, size=None):
        if flat is None:
            return None
        if size is None:
            return [flat[at:at + math.prod(s)].view(s) for s, _, at in tensors]
        return [flat[at // BLOCK:at // BLOCK + -(-math.prod(s) // BLOCK)] for s, _, at in tensors]

    # what a program keeps: its lists of weights, gradients and moments
    st["lists"] = dict(p=views(st["p"]), master=views(st["master"]), g=views(g), m=views(st["m"]), v=views(st["v"]),
                       ms=views(st.get("ms"), 1), vs=views(st.get("vs"), 1))
    st["decay"] = [0.05 if decays else 0.0 for _, decays, _ in tensors]
    return st


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    return {"norm": _prepare_norm, "attn": _prepare_attn, "adamw": _prepare_adamw}[case["op"]](case, gen)


# ---------------------------------------------------------------------------------------- plain forms
def _pairs(x, rot, interleaved):
    if interleaved:
        return x[..., 0:rot:2], x[..., 1:rot:2]
    return x[..., :rot // 2], x[..., rot // 2:rot]


def _join(a, b, rest, interleaved):
    ab = torch.stack((a, b), -1).flatten(-2) if interleaved else torch.cat((a, b), -1)
    return torch.cat((ab, rest), -1)


def _angles(st):
    if st["positions"] is None:
        return st["cos"][None, :, None], st["sin"][None, :, None]
    at = st["positions"].long()
    return st["cos"][at][:, :, None], st["sin"][at][:, :, None]


def _plain_norm(st, x, gamma, dy):
    case = st["case"]
    rot, inter = case["rot"], case["pairs"] == "interleaved"
    cos, sin = _angles(st)
    xf, w = x.float(), gamma.float()
    r = torch.rsqrt(xf.square().mean(-1, keepdim=True) + EPS)
    xr = xf * r
    n = xr * w
    a, b = _pairs(n, rot, inter)
    y = _join(a * cos - b * sin, b * cos + a * sin, n[..., rot:], inter).to(x.dtype)
    if dy is None:
        return y, None, None
    gf = dy.float()
    a, b = _pairs(gf, rot, inter)
    g = _join(a * cos + b * sin, b * cos - a * sin, gf[..., rot:], inter)
    dgamma = (g * xr).sum((0, 1, 2))
    h = g * w
    dx = (r * (h - xr * (h * xr).mean(-1, keepdim=True))).to(x.dtype)
    return y, dx, dgamma


def _plain_bias(st):
    """(B or 1, hq, Lq, Lk) bias in fp32, and the bucket of each pair."""
    case = st["case"]
    i = torch.arange(case["Lq"], device="cuda")[None, :, None]
    j = torch.arange(case["Lk"], device="cuda")[None, None, :]
    at = i if st["q_start"] is None else i + st["q_start"].long()[:, None, None]
    bucket = st["map"].long()[(j - at).clamp(-case["distance"], case["distance"]) + case["distance"]]
    bias = st["table"].float().t()[:, bucket].transpose(0, 1)
    seen = bias > EXCLUDE
    if case["causal"]:
        seen = seen & (j <= at)[:, None]
    if st["kv_lens"] is not None:
        seen = seen & (j < st["kv_lens"].long()[:, None, None])[:, None]
    if st["q_lens"] is not None:
        seen = seen & (i < st["q_lens"].long()[:, None, None])[:, None]
    return torch.where(seen, bias, bias.new_tensor(-math.inf)), bucket


def _plain_attn(st):
    case = st["case"]
    B, Lq, Lk, hq, hk, d = (case[n] for n in ("B", "Lq", "Lk", "hq", "hk", "d"))
    dt = st["q"].dtype
    bias, bucket = _plain_bias(st)
    q = st["q"].float().transpose(1, 2)
    k, v = (st[n].float().transpose(1, 2).repeat_interleave(hq // hk, 1) for n in ("k", "v"))
    s = torch.matmul(q, k.transpose(2, 3)) * st["scale"] + bias
    top = s.amax(-1, keepdim=True)
    some = top > -math.inf
    p = torch.exp(s - torch.where(some, top, torch.zeros_like(top)))
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(some, total, torch.ones_like(total))
    o = torch.matmul(p, v)
    lse = torch.where(some, top + torch.log(total), top)[..., 0]
    out = dict(out=o.transpose(1, 2).to(dt), lse=lse)
    if not case["train"]:
        return out
    do = st["do"].float().transpose(1, 2)
    dp = torch.matmul(do, v.transpose(2, 3))
    ds = p * (dp - (p * dp).sum(-1, keepdim=True))
    shared = (B, hk, hq // hk, Lk, d)
    dq = torch.matmul(ds, k) * st["scale"]
    dk = torch.matmul(ds.transpose(2, 3), q).view(shared).sum(2) * st["scale"]
    dv = torch.matmul(p.transpose(2, 3), do).view(shared).sum(2)
    dt_sum = torch.zeros(case["buckets"], hq, device="cuda")
    dt_sum.index_add_(0, bucket.flatten(), ds.sum(0).permute(1, 2, 0).reshape(-1, hq)) if bucket.shape[0] == 1 else \
        dt_sum.index_add_(0, bucket.flatten(), ds.permute(0, 2, 3, 1).reshape(-1, hq))
    out.update(dq=dq.transpose(1, 2).to(dt), dk=dk.transpose(1, 2).to(dt), dv=dv.transpose(1, 2).to(dt),
               dtable=dt_sum.to(dt))
    return out


def _plain_adamw(st):
    case = st["case"]
    g = st["g"].float()
    if case["bits"] == 32:
        m0, v0 = st["m"], st["v"]
    else:
        c = st["m"].view(-1, BLOCK)
        m0 = (st["lut_m"][c.abs().int()] * st["ms"][:, None] * c.sign()).view(-1)
        v0 = (st["lut_v"][st["v"].int()].view(-1, BLOCK) * st["vs"][:, None]).view(-1)
    m = m0 * BETA1 + g * (1 - BETA1)
    v = v0 * BETA2 + g * g * (1 - BETA2)
    den = torch.sqrt(v) * (1 / math.sqrt(1 - BETA2 ** STEP)) + ADAM_EPS
    p = st["p"].float() if st["master"] is None else st["master"]
    p = p * st["keep"] - m / den * (LR / (1 - BETA1 ** STEP))
    if st["master"] is not None:
        st["master"].copy_(p)
    st["p"].copy_(p)
    out = dict(p=st["p"]) if st["master"] is None else dict(p=st["p"], master=st["master"])
    if case["bits"] == 32:
        st["m"].copy_(m)
        st["v"].copy_(v)
        return dict(out, m=st["m"], v=st["v"])
    mb, vb = m.view(-1, BLOCK), v.view(-1, BLOCK)
    st["ms"].copy_(mb.abs().amax(1))
    st["vs"].copy_(vb.amax(1))
    c = _codes(mb, st["ms"][:, None], 127, 1)
    st["m"].copy_((c * mb.sign()).view(-1))
    cv = _codes(vb, st["vs"][:, None], 255, 2)
    cv = torch.where(vb > 0, cv.clamp(min=1), cv)
    st["v"].copy_(cv.view(-1))
    return dict(out, m=(st["lut_m"][c.int()] * st["ms"][:, None] * mb.sign()).view(-1).to(torch.bfloat16),
                v=(st["lut_v"][cv.int()] * st["vs"][:, None]).view(-1).to(torch.bfloat16))


# ---------------------------------------------------------------------------------------- the framework's calls
def _own_norm(st):
    from shifted_window_attention_sw_b200 import vswin

    case = st["case"]
    kw = dict(eps=EPS, cos=st["cos"], sin=st["sin"], positions=st["positions"],
              interleaved=case["pairs"] == "interleaved")
    q, k = vswin.qk_norm_forward(st["q"], st["k"], st["gq"], st["gk"], **kw)
    if not case["train"]:
        return dict(q=q, k=k)
    dq, dk, dgq, dgk = vswin.qk_norm_backward(st["q"], st["k"], st["gq"], st["gk"], st["dq"], st["dk"], **kw)
    return dict(q=q, k=k, dq=dq, dk=dk, dgq=dgq, dgk=dgk)


def _own_attn(st):
    from shifted_window_attention_sw_b200 import vswin

    case = st["case"]
    kw = dict(scale=st["scale"], causal=case["causal"], q_lens=st["q_lens"], kv_lens=st["kv_lens"],
              q_start=st["q_start"])
    ins = (st["q"], st["k"], st["v"], st["table"], st["map"])
    out, lse = vswin.bias_attention_forward(*ins, **kw)
    if not case["train"]:
        return dict(out=out, lse=lse)
    dq, dk, dv, dtable = vswin.bias_attention_backward(*ins, out, lse, st["do"], **kw)
    return dict(out=out, lse=lse, dq=dq, dk=dk, dv=dv, dtable=dtable)


def _own_adamw(st):
    from shifted_window_attention_sw_b200 import vswin

    lists = st["lists"]
    if "optimizer" not in st:  # the program's optimizer object, made once over its weights and moments
        st["optimizer"] = vswin.AdamW(lists["p"], lr=LR, betas=(BETA1, BETA2), eps=ADAM_EPS,
                                      weight_decay=st["decay"], bits=st["case"]["bits"], master=lists["master"],
                                      moments=(lists["m"], lists["v"]), scales=(lists["ms"], lists["vs"]))
    st["optimizer"].step(lists["g"], step=STEP)
    out = dict(p=st["p"]) if st["master"] is None else dict(p=st["p"], master=st["master"])
    if st["case"]["bits"] == 32:
        return dict(out, m=st["m"], v=st["v"])
    m, v = vswin.adamw_decode(st["m"], st["ms"], st["v"], st["vs"], dtype=torch.bfloat16)
    return dict(out, m=m, v=v)


def run(state):
    op = state["case"]["op"]
    if own:
        return {"norm": _own_norm, "attn": _own_attn, "adamw": _own_adamw}[op](state)
    if op == "attn":
        return _plain_attn(state)
    if op == "adamw":
        return _plain_adamw(state)
    q, dq, dgq = _plain_norm(state, state["q"], state["gq"], state.get("dq"))
    k, dk, dgk = _plain_norm(state, state["k"], state["gk"], state.get("dk"))
    out = dict(q=q, k=k)
    return dict(out, dq=dq, dk=dk, dgq=dgq, dgk=dgk) if state["case"]["train"] else out


# ---------------------------------------------------------------------------------------- work
def _lens(case):
    """Lengths that stand for a ragged batch: half to all of Lk, three quarters of it on average."""
    return 0.75 * case["Lk"] if case["ragged"] and case["B"] > 1 else float(case["Lk"])


def work(case):
    if case["op"] == "norm":
        n = case["B"] * case["L"] * (case["hq"] + case["hk"]) * case["d"]
        angles = min(case["B"] * case["L"], max(case["L"], 4096 if case["positions"] else 1)) * case["rot"] * 4
        return {"bytes": n * (10 if case["train"] else 4) + angles, "flops": n * (25 if case["train"] else 8)}
    if case["op"] == "attn":
        B, Lq, hq, hk, d = (case[n] for n in ("B", "Lq", "hq", "hk", "d"))
        Lk = _lens(case)
        rows = Lk if Lq == case["Lk"] else Lq
        pairs = rows * Lk
        if case["causal"]:
            pairs = rows * (Lk - rows) + rows * (rows + 1) / 2
        times = 3 if case["train"] else 1  # q, k, v, out; then those, dout and dq, dk, dv
        size = B * d * (2 * rows * hq + 2 * Lk * hk) * 2 * times + B * Lq * hq * 4
        return {"bytes": size, "flops": B * hq * pairs * d * (14 if case["train"] else 4)}
    n = case["blocks"] * sum(math.prod(s) for s, _ in _block_sizes(case["C"]))
    each = 4 + (4 if case["grads"] == "fp32" else 2) + (8 if case["master"] else 0) + \
        (16 if case["bits"] == 32 else 8 + 16 / BLOCK)
    return {"bytes": n * each, "flops": n * 14}


# ---------------------------------------------------------------------------------------- 64 bits
def _exact_norm(st):
    case = st["case"]
    rot, half = case["rot"], case["rot"] // 2
    even = torch.arange(half, device="cuda")
    ia, ib = (2 * even, 2 * even + 1) if case["pairs"] == "interleaved" else (even, even + half)
    at = torch.arange(case["L"], device="cuda").expand(case["B"], -1) if st["positions"] is None else st["positions"].long()
    turn = torch.complex(st["cos"].double(), st["sin"].double())[at].unsqueeze(2)
    out = {}
    for name, x, gamma in (("q", st["q"], st["gq"]), ("k", st["k"], st["gk"])):
        x, w = x.double(), gamma.double()
        unit = x / torch.sqrt((x * x).sum(-1, keepdim=True) / case["d"] + EPS)
        y = unit * w
        z = torch.complex(y[..., ia], y[..., ib]) * turn
        y[..., ia], y[..., ib] = z.real, z.imag
        out[name] = y
        if case["train"]:
            g = st["d" + name].double().clone()
            z = torch.complex(g[..., ia], g[..., ib]) * turn.conj()
            g[..., ia], g[..., ib] = z.real, z.imag
            out["dg" + name] = (g * unit).flatten(0, 2).sum(0)
            g = g * w
            along = (g * unit).sum(-1, keepdim=True) / case["d"]
            out["d" + name] = (g - unit * along) / torch.sqrt((x * x).sum(-1, keepdim=True) / case["d"] + EPS)
    return out


def _exact_attn(st):
    """Sequence by sequence and head by head, on the rows and keys that take part."""
    case = st["case"]
    B, Lq, Lk, hq, hk, d, D = (case[n] for n in ("B", "Lq", "Lk", "hq", "hk", "d", "distance"))
    new = lambda *shape: torch.zeros(shape, dtype=torch.float64, device="cuda")  # noqa: E731
    out = dict(out=new(B, Lq, hq, d), lse=new(B, hq, Lq) - math.inf)
    if case["train"]:
        out.update(dq=new(B, Lq, hq, d), dk=new(B, Lk, hk, d), dv=new(B, Lk, hk, d), dtable=new(case["buckets"], hq))
    for b in range(B):
        nk = Lk if st["kv_lens"] is None else int(st["kv_lens"][b])
        nq = Lq if st["q_lens"] is None else int(st["q_lens"][b])
        first = 0 if st["q_start"] is None else int(st["q_start"][b])
        offset = torch.arange(nk, device="cuda")[None] - (torch.arange(nq, device="cuda") + first)[:, None]
        bucket = st["map"].long()[torch.clamp(offset, -D, D) + D]
        for h in range(hq):
            q, k, v = st["q"][b, :nq, h].double(), st["k"][b, :nk, h * hk // hq].double(), st["v"][b, :nk, h * hk // hq].double()
            s = q @ k.T * st["scale"] + st["table"][:, h].double()[bucket]
            if case["causal"]:
                s = s.masked_fill(offset > 0, -math.inf)
            out["lse"][b, h, :nq] = torch.logsumexp(s, 1)
            p = torch.softmax(s, 1)
            out["out"][b, :nq, h] = p @ v
            if case["train"]:
                do = st["do"][b, :nq, h].double()
                out["dv"][b, :nk, h * hk // hq] += p.T @ do
                p = p * (do @ v.T - (do * out["out"][b, :nq, h]).sum(1, keepdim=True))
                out["dq"][b, :nq, h] = p @ k * st["scale"]
                out["dk"][b, :nk, h * hk // hq] += p.T @ q * st["scale"]
                out["dtable"][:, h].index_add_(0, bucket.flatten(), p.flatten())
    return out


def _exact_adamw(st):
    case = st["case"]
    up = lambda x: x.double().repeat_interleave(BLOCK)  # noqa: E731
    m, v, g = st["m"].double(), st["v"].double(), st["g"].double()
    if case["bits"] == 8:
        m, v = m * m.abs() / 127.0 ** 2 * up(st["ms"]), (v / 255.0) ** 4 * up(st["vs"])
    m = BETA1 * m + (1 - BETA1) * g
    v = BETA2 * v + (1 - BETA2) * g ** 2
    p = (st["p"] if st["master"] is None else st["master"]).double()
    p = p * st["keep"].double() - LR * (m / (1 - BETA1 ** STEP)) / ((v / (1 - BETA2 ** STEP)) ** 0.5 + ADAM_EPS)
    if case["bits"] == 8:
        ms, vs = m.abs().view(-1, BLOCK).amax(1), v.view(-1, BLOCK).amax(1)
        safe = lambda s: up(torch.where(s > 0, s, torch.ones_like(s)))  # noqa: E731
        m = m.sign() * torch.round(127 * (m.abs() / safe(ms)) ** 0.5) ** 2 / 127.0 ** 2 * up(ms)
        c = torch.round(255 * (v / safe(vs)) ** 0.25)
        v = (torch.where(v > 0, c.clamp(min=1), c) / 255) ** 4 * up(vs)
    out = dict(p=p, m=m, v=v)
    return out if st["master"] is None else dict(out, master=p)


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "attn" and case["B"] * case["hq"] * case["Lq"] * float(case["Lk"]) > 3e9:
        return None
    return {"norm": _exact_norm, "attn": _exact_attn, "adamw": _exact_adamw}[case["op"]](st)
