"""GPU parity of the operators over token sequences (head norm with rotation, attention with bucketed bias) and
of the AdamW step against their float64 definitions. Every output element is held to the bound that
sequence_reference derives for it. Needs a B200."""

import math
import os
import subprocess
import sys

import pytest
import torch

import sequence_reference as ref
from shifted_window_attention_sw_b200 import vswin

pytestmark = pytest.mark.gpu

BF16, FP16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from shifted_window_attention_sw_b200 import build

    build.build()
    vswin.lib()


@pytest.fixture(autouse=True)
def _clean():
    yield
    assert vswin.poll_error() == vswin.OK, vswin.last_error()


def _rand(gen, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=gen, dtype=F32) * scale).to(dtype).cuda()


def _close(name, got, want, tol):
    got = got.double()
    same = (got == want) | (got.isnan() & want.isnan())
    off = torch.where(same, torch.zeros_like(want), (got - want).abs() - tol)
    assert not off.isnan().any(), name
    assert (off <= 0).all(), (name, float(off.max()), int((off > 0).sum()), got.numel())


# ------------------------------------------------------------------ norm and rotation
NORM_CASES = [
    # dtype, B, L, hq, hk, d, rot, interleaved
    (BF16, 1, 1, 1, 1, 32, 32, False),
    (BF16, 2, 37, 3, 3, 32, 32, True),
    (FP16, 3, 50, 8, 2, 64, 32, False),
    (BF16, 1, 129, 4, 1, 128, 64, True),
    (F32, 2, 33, 4, 4, 64, 64, False),
    (F32, 1, 5, 2, 1, 256, 128, True),
    (BF16, 2, 19, 5, 5, 96, 96, False),
    (FP16, 1, 700, 12, 12, 16, 16, False),
    (BF16, 2, 9, 3, 1, 80, 40, False),      # rot not a multiple of 16
    (F32, 2, 9, 3, 2, 10, 6, True),         # odd widths go element by element
    (BF16, 1, 4, 2, 2, 7, 0, False),
    (FP16, 1, 3, 1, 2, 250, 250, False),
    (BF16, 1, 3000, 24, 3, 64, 64, False),  # several steps of the walk
]


def _norm_inputs(case, seed=0):
    dtype, B, L, hq, hk, d, rot, inter = case
    gen = torch.Generator().manual_seed(seed + d + L)
    qkv = _rand(gen, (B, L, hq + 2 * hk, d), dtype, 1.5)
    a = torch.randn(L + 5, rot // 2, generator=gen, dtype=torch.float64)
    kw = dict(eps=1e-6, interleaved=inter)
    if rot:
        kw.update(cos=a.cos().float().cuda(), sin=a.sin().float().cuda())
    return dict(q=qkv[:, :, :hq], k=qkv[:, :, hq:hq + hk], gq=_rand(gen, (d,), dtype), gk=_rand(gen, (d,), dtype),
                dq=_rand(gen, (B, L, hq, d), dtype), dk=_rand(gen, (B, L, hk, d), dtype), kw=kw, gen=gen)


def _norm_check(i, kw):
    y = vswin.qk_norm_forward(i["q"], i["k"], i["gq"], i["gk"], **kw)
    g = vswin.qk_norm_backward(i["q"], i["k"], i["gq"], i["gk"], i["dq"], i["dk"], **kw)
    for w, n in enumerate("qk"):
        r = ref.qk_norm(i[n], i["g" + n], dy=i["d" + n], **kw)
        _close(n, y[w], r["y"], r["y_tol"])
        _close("d" + n, g[w], r["dx"], r["dx_tol"])
        _close("dgamma_" + n, g[2 + w], r["dgamma"], r["dgamma_tol"])
    return y, g


@pytest.mark.parametrize("case", NORM_CASES, ids=str)
@pytest.mark.parametrize("positions", [False, True])
def test_qk_norm(case, positions):
    i = _norm_inputs(case)
    kw = dict(i["kw"])
    if positions:
        if "cos" not in kw:
            pytest.skip("no rotation")
        B, L = i["q"].shape[:2]
        kw["positions"] = torch.randint(0, L + 5, (B, L), generator=i["gen"], dtype=torch.int32).cuda()
    y, g = _norm_check(i, kw)
    again = vswin.qk_norm_backward(i["q"], i["k"], i["gq"], i["gk"], i["dq"], i["dk"], **kw)
    assert all(torch.equal(a, b) for a, b in zip(g, again))


@pytest.mark.parametrize("case", [NORM_CASES[2], NORM_CASES[8]], ids=str)
def test_qk_norm_in_place_and_strided(case):
    i = _norm_inputs(case)
    kw = i["kw"]
    y, g = _norm_check(i, kw)
    # heads before tokens, and rows that start off a 16-byte boundary
    dtype, B, L, hq, hk, d = case[:6]
    for shift in (0, 1):
        def moved(x):
            buf = torch.empty(x.shape[0] * x.shape[2] * x.shape[1] * (d + shift) + 8, dtype=dtype, device="cuda")
            v = buf[shift:].as_strided((x.shape[0], x.shape[1], x.shape[2], d),
                                       (x.shape[2] * x.shape[1] * (d + shift), d + shift, x.shape[1] * (d + shift), 1))
            return v.copy_(x)
        q, k, dq, dk = (moved(i[n]) for n in ("q", "k", "dq", "dk"))
        z = vswin.qk_norm_forward(q, k, i["gq"], i["gk"], q_out=q.clone(memory_format=torch.preserve_format), **kw)
        for a, b, t in zip(z, y, ("q", "k")):
            r = ref.qk_norm(i[t], i["g" + t], **kw)
            _close(t, a, r["y"], r["y_tol"])
        zg = vswin.qk_norm_backward(q, k, i["gq"], i["gk"], dq, dk, dq=dq, dk=dk, **kw)  # over the output gradients
        assert zg[0] is dq
        for n, a in (("q", zg[0]), ("k", zg[1])):
            r = ref.qk_norm(i[n], i["g" + n], dy=i["d" + n], **kw)
            _close("d" + n, a, r["dx"], r["dx_tol"])
        # forward in place on the packed views
        vswin.qk_norm_forward(q, k, i["gq"], i["gk"], q_out=q, k_out=k, **kw)
        assert torch.equal(q, z[0]) and torch.equal(k, z[1])


def test_qk_norm_zero_rows_and_bad_positions():
    q = torch.zeros(1, 4, 2, 64, dtype=BF16, device="cuda")
    k = torch.ones(1, 4, 1, 64, dtype=BF16, device="cuda")
    w = torch.ones(64, dtype=BF16, device="cuda")
    cos, sin = torch.ones(4, 32, device="cuda"), torch.zeros(4, 32, device="cuda")
    pos = torch.tensor([[0, 4, -1, 2]], dtype=torch.int32, device="cuda")
    y, z = vswin.qk_norm_forward(q, k, w, w, eps=1e-6, cos=cos, sin=sin, positions=pos)
    assert vswin.poll_error() == vswin.ERR_BOUNDS
    assert torch.equal(y, q) and torch.equal(z, k)  # the nearest row turns by nothing
    g = vswin.qk_norm_backward(q, k, w, w, k.expand(1, 4, 2, 64), k, eps=0.0)  # 1 / 0 of a zero row
    assert not torch.isfinite(g[0]).any() and torch.isfinite(g[1]).all()


# ------------------------------------------------------------------ attention
def _map(buckets=32, D=128, bidirectional=True):
    return vswin.bucket_map(buckets, D, bidirectional)


def _attn_inputs(dtype, B, Lq, Lk, hq, hk, d, buckets=32, seed=0, layout="packed"):
    gen = torch.Generator().manual_seed(seed + 7 * Lq + Lk + d)
    if layout == "heads_first":
        mk = lambda L, h: _rand(gen, (B, h, L, d), dtype).transpose(1, 2)  # noqa: E731
        q, k, v, do = mk(Lq, hq), mk(Lk, hk), mk(Lk, hk), mk(Lq, hq)
    elif Lq == Lk:
        qkv = _rand(gen, (B, Lq, hq + 2 * hk, d), dtype)
        q, k, v = qkv[:, :, :hq], qkv[:, :, hq:hq + hk], qkv[:, :, hq + hk:]
        do = _rand(gen, (B, Lq, hq, d), dtype)
    else:
        kv = _rand(gen, (B, Lk, 2, hk, d), dtype)
        q, k, v, do = _rand(gen, (B, Lq, hq, d), dtype), kv[:, :, 0], kv[:, :, 1], _rand(gen, (B, Lq, hq, d), dtype)
    return [q, k, v, _rand(gen, (buckets, hq), dtype, 0.7)], do


def _i32(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _attn_check(ins, bmap, do, scale=None, backward=True, **kw):
    scale = ins[0].shape[-1] ** -0.5 if scale is None else scale
    out, lse = vswin.bias_attention_forward(*ins, bmap, scale=scale, **kw)
    r = ref.bias_attention(*ins, bmap, scale, dout=do if backward else None, **kw)
    _close("out", out, r["out"], r["out_tol"])
    _close("lse", lse, r["lse"], r["lse_tol"])
    if not backward:
        return out, lse
    g = vswin.bias_attention_backward(*ins, bmap, out, lse, do, scale=scale, **kw)
    for n, x in zip(("dq", "dk", "dv", "dtable"), g):
        assert x.dtype == ins[0].dtype
        _close(n, x, r[n], r[n + "_tol"])
    again = vswin.bias_attention_backward(*ins, bmap, out, lse, do, scale=scale, **kw)
    for n, x, y in zip(("dq", "dk", "dv", "dtable"), g, again):
        assert torch.equal(x, y), n
    return out, lse, *g


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("dtype,B,L,hq,hk,d", [
    (BF16, 1, 1, 1, 1, 32), (BF16, 2, 7, 3, 3, 32), (FP16, 1, 63, 2, 1, 64), (BF16, 1, 64, 4, 1, 128),
    (BF16, 1, 65, 1, 1, 64), (FP16, 2, 127, 2, 2, 32), (BF16, 1, 128, 2, 2, 128), (BF16, 1, 129, 6, 2, 64),
    (FP16, 1, 192, 2, 1, 128), (BF16, 2, 392, 3, 3, 32), (FP16, 1, 577, 4, 2, 64), (BF16, 1, 700, 2, 1, 128),
], ids=str)
def test_attention_self(dtype, B, L, hq, hk, d, causal):
    ins, do = _attn_inputs(dtype, B, L, L, hq, hk, d)
    _attn_check(ins, _map(bidirectional=not causal), do, causal=causal)


@pytest.mark.parametrize("d", [32, 64, 128])
def test_attention_padded_batch(d):
    # lengths 0 and 1 among them; what lies behind the lengths is NaN and infinity
    ins, do = _attn_inputs(BF16, 5, 200, 200, 4, 2, d)
    lens = _i32(200, 0, 1, 130, 77)
    clean = [t.clone() for t in (*ins[:3], do)]
    for b, n in enumerate(lens.tolist()):
        for t, bad in zip((*ins[:3], do), (math.nan, math.inf, math.nan, -math.inf)):
            t[b, n:] = bad
    res = _attn_check(ins, _map(), do, q_lens=lens, kv_lens=lens)
    same = vswin.bias_attention_forward(*clean[:3], ins[3], _map(), q_lens=lens, kv_lens=lens)
    assert torch.equal(res[0], same[0]) and torch.equal(res[1], same[1])
    for b, n in enumerate(lens.tolist()):  # rows and keys behind the lengths are zero
        assert (res[0][b, n:] == 0).all() and (res[2][b, n:] == 0).all()
        assert (res[3][b, n:] == 0).all() and (res[4][b, n:] == 0).all()
        assert (res[1][b, :, n:] == -math.inf).all()


@pytest.mark.parametrize("Lq,Lk,start,causal", [
    (5, 300, (295, 100, -3), True), (200, 33, (-40, 0, 500), True), (150, 260, (0, -1000, 1000), False),
    (40, 1, (0, -60, -20), True), (300, 140, (-150, -129, -128), True),
], ids=str)
@pytest.mark.parametrize("d", [32, 64])
def test_attention_other_lengths(Lq, Lk, start, causal, d):
    # queries before the first key (rows without keys), far behind the last, sequences of unequal length
    ins, do = _attn_inputs(FP16, 3, Lq, Lk, 4, 4, d, buckets=64)
    _attn_check(ins, _map(64, 96, not causal), do, causal=causal, q_start=_i32(*start), kv_lens=_i32(Lk, Lk // 2, Lk),
                q_lens=_i32(Lq, Lq, Lq - 1))


@pytest.mark.parametrize("layout", ["packed", "heads_first"])
@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_attention_layouts(layout, dtype):
    ins, do = _attn_inputs(dtype, 2, 140, 140, 4, 2, 64, layout=layout)
    _attn_check(ins, _map(), do)
    # keys shared by the batch (stride 0), and gradients into one packed buffer
    if layout == "packed":
        ins[1], ins[2] = ins[1][:1].expand(2, -1, -1, -1), ins[2][:1].expand(2, -1, -1, -1)
        _, _, dq, dk, dv, _ = _attn_check(ins, _map(), do)
        buf = torch.zeros(2, 140, 8, 64, dtype=dtype, device="cuda")
        out, lse = vswin.bias_attention_forward(*ins, _map())
        vswin.bias_attention_backward(*ins, _map(), out, lse, do, dq=buf[:, :, :4], dk=buf[:, :, 4:6], dv=buf[:, :, 6:])
        assert torch.equal(buf, torch.cat((dq, dk, dv), 2))


@pytest.mark.parametrize("dim", [0, 1, 2])
@pytest.mark.parametrize("Lq", [150, 1])
def test_attention_broadcast_inputs(dim, Lq):
    # k and v with stride 0 over the batch, the tokens or the heads; q over the batch
    ins, do = _attn_inputs(BF16, 3, Lq, 150, 4, 4, 64)
    wide = [t.clone() for t in ins]
    for n in (1, 2):
        narrow = ins[n].select(dim, 0).unsqueeze(dim)
        ins[n] = narrow.expand(3, 150, 4, 64)
        wide[n] = ins[n].contiguous()
    ins[0], wide[0] = ins[0][:1].expand(3, -1, -1, -1), ins[0][:1].expand(3, -1, -1, -1).contiguous()
    got = _attn_check(ins, _map(), do, kv_lens=_i32(150, 77, 3))
    want = _attn_check(wide, _map(), do, kv_lens=_i32(150, 77, 3))
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("dtype,low", [(BF16, torch.finfo(BF16).min), (BF16, -math.inf), (FP16, -math.inf),
                                       (FP16, torch.finfo(FP16).min)], ids=str)
def test_attention_masking_buckets(dtype, low):
    # buckets that take keys out: half of them, and every one of head 1 (rows without a key). fp16's lowest value is
    # an ordinary bias (-65504): scores stay finite, so the row's softmax is over all its keys
    ins, do = _attn_inputs(dtype, 1, 150, 150, 2, 2, 64)
    ins[3][::2] = low
    if low != torch.finfo(FP16).min:
        ins[3][:, 1] = low
    res = _attn_check(ins, _map(), do)
    if low != torch.finfo(FP16).min:
        assert (res[0][:, :, 1] == 0).all() and (res[1][:, 1] == -math.inf).all()
        assert (res[5][:, 1] == 0).all()


def test_attention_large_scores():
    # logits that span hundreds: the running maximum grows by large steps
    ins, do = _attn_inputs(BF16, 1, 300, 300, 2, 2, 64)
    _attn_check(ins, _map(), do, scale=4.0)
    ins, do = _attn_inputs(BF16, 1, 300, 300, 2, 2, 64)
    _attn_check(ins, _map(), do, scale=-1.0)  # any finite scale
    _attn_check(ins, _map(), do, scale=0.0)


@pytest.mark.parametrize("buckets,D", [(1, 0), (3, 1), (500, 249), (4, 3000)], ids=str)
def test_attention_any_map(buckets, D):
    # a map that is not the logarithmic one: any number of buckets in any order
    ins, do = _attn_inputs(BF16, 1, 280, 280, 2, 1, 32, buckets=buckets)
    gen = torch.Generator().manual_seed(buckets)
    bmap = torch.randint(0, buckets, (2 * D + 1,), generator=gen, dtype=torch.int32).cuda()
    _attn_check(ins, bmap, do)


TOKEN_CASES = [
    # dtype, B, Lq, Lk, hq, hk, d
    (BF16, 1, 1, 1, 1, 1, 32), (BF16, 3, 1, 200, 4, 4, 64), (FP16, 2, 1, 4097, 8, 2, 128), (BF16, 4, 1, 3000, 16, 1, 64),
    (BF16, 2, 2, 1000, 12, 3, 64), (FP16, 2, 4, 700, 4, 4, 32), (BF16, 1, 3, 9000, 32, 2, 128), (BF16, 2, 1, 500, 40, 1, 64),
    (BF16, 1, 100, 6000, 2, 1, 64),
]


@pytest.mark.parametrize("case", TOKEN_CASES, ids=str)
@pytest.mark.parametrize("causal", [False, True])
def test_attention_new_tokens(case, causal):
    dtype, B, Lq, Lk, hq, hk, d = case
    ins, _ = _attn_inputs(dtype, B, Lq, Lk, hq, hk, d)
    lens = torch.tensor([max(Lq if causal else 0, Lk - b * (Lk // 3 + 1)) for b in range(B)], dtype=torch.int32).cuda()
    lens = lens.clamp(min=0, max=Lk)
    for b, n in enumerate(lens.tolist()):
        ins[1][b, n:], ins[2][b, n:] = math.nan, math.nan
    out, lse = _attn_check(ins, _map(bidirectional=False), None, backward=False, causal=causal, kv_lens=lens,
                           q_start=lens - Lq)
    again = vswin.bias_attention_forward(*ins, _map(bidirectional=False), causal=causal, kv_lens=lens, q_start=lens - Lq)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("d", [32, 128])
def test_attention_last_wave_in_parts(d):
    # 300 query tiles: the four behind the first wave of 296 run as parts of the keys
    ins, _ = _attn_inputs(BF16, 2, 70, 1100, 150, 50, d)
    _attn_check(ins, _map(), None, backward=False, kv_lens=_i32(1100, 530), q_start=_i32(500, 0), q_lens=_i32(70, 66))


def test_attention_offsets_past_32_bits():
    # the second sequence's cache starts 2^31 elements in, the query's rows lie 2^31 elements apart
    d, Lk = 64, 300
    buf = torch.empty(2**31 + 2 * Lk * d + 2**22, dtype=BF16, device="cuda")
    gen = torch.Generator().manual_seed(1)
    k = buf.as_strided((2, Lk, 1, d), (2**31, 2 * d, d, 1))
    v = buf[d:].as_strided((2, Lk, 1, d), (2**31, 2 * d, d, 1))
    k.copy_(_rand(gen, (2, Lk, 1, d), BF16))
    v.copy_(_rand(gen, (2, Lk, 1, d), BF16))
    q, table, do = _rand(gen, (2, Lk, 1, d), BF16), _rand(gen, (32, 1), BF16), _rand(gen, (2, Lk, 1, d), BF16)
    _attn_check([q, k, v, table], _map(), do)
    _attn_check([q[:, :1], k, v, table], _map(), None, backward=False)


def test_attention_reports_bad_lengths_and_buckets():
    ins, _ = _attn_inputs(BF16, 2, 100, 100, 2, 2, 64)
    good = vswin.bias_attention_forward(*ins, _map(), q_lens=_i32(100, 0), kv_lens=_i32(0, 100))
    assert vswin.poll_error() == vswin.OK
    bad = vswin.bias_attention_forward(*ins, _map(), q_lens=_i32(101, -5), kv_lens=_i32(-1, 2**31 - 1))
    assert vswin.poll_error() == vswin.ERR_BOUNDS
    assert torch.equal(good[0], bad[0]) and torch.equal(good[1], bad[1])
    ins[3].zero_()
    bmap = _map()
    wrong = bmap.clone()
    wrong[::3] = 32
    wrong[1::3] = -1
    good = vswin.bias_attention_forward(*ins, bmap)
    bad = vswin.bias_attention_forward(*ins, wrong)
    assert vswin.poll_error() == vswin.ERR_BOUNDS
    assert torch.equal(good[0], bad[0])
    vswin.bias_attention_backward(*ins, wrong, *bad, torch.ones_like(bad[0]))
    assert vswin.poll_error() == vswin.ERR_BOUNDS
    tok = vswin.bias_attention_forward(ins[0][:, :1], *ins[1:], wrong)
    assert vswin.poll_error() == vswin.ERR_BOUNDS
    assert torch.isfinite(tok[0]).all()


# ------------------------------------------------------------------ AdamW
HYPER = dict(lr=3e-3, betas=(0.9, 0.99), eps=1e-8)


def _adamw_lists(sizes, ptypes, gtypes, seed=0, offset=0):
    gen = torch.Generator().manual_seed(seed)

    def at(n, dtype, scale):
        buf = torch.zeros(n + offset, dtype=dtype, device="cuda")
        buf[offset:] = _rand(gen, (n,), F32, scale).to(dtype)
        return buf[offset:]

    p = [at(n, t, 0.1) for n, t in zip(sizes, ptypes)]
    g = [at(n, t, 1e-2) for n, t in zip(sizes, gtypes)]
    return p, g


def _adamw_bounds(want, got, dtype):
    # fp32: the moments' and the step's few operations, each off by 2^-24; the weight is rounded once
    _close("param", got, want, ref.rounding(dtype, want) + 1e-6 * (want.abs() + HYPER["lr"]))


SIZES = [1, 7, 8, 255, 256, 257, 2048, 2049, 5000, 70001]


@pytest.mark.parametrize("offset", [0, 1])
@pytest.mark.parametrize("master", [None, True])
@pytest.mark.parametrize("ptype,gtype", [(BF16, F32), (F32, F32), (FP16, FP16), (BF16, BF16), (F32, BF16)], ids=str)
def test_adamw_32(ptype, gtype, master, offset):
    p, g = _adamw_lists(SIZES, [ptype] * len(SIZES), [gtype] * len(SIZES), offset=offset)
    wd = [0.1 * (i % 3) for i in range(len(p))]
    opt = vswin.AdamW(p, weight_decay=wd, bits=32, master=master, **HYPER)
    want = [[t.double(), torch.zeros_like(t, dtype=torch.float64), torch.zeros_like(t, dtype=torch.float64)] for t in p]
    for step in (1, 2, 3):
        gs = [t * step for t in g]
        opt.step(gs)
        for i, w in enumerate(want):
            w[:] = ref.adamw(w[0], gs[i].double(), w[1], w[2], HYPER["lr"], *HYPER["betas"], HYPER["eps"], wd[i], step)
            if master:
                _close("master", opt.master[i], w[0], 2e-6 * (w[0].abs() + HYPER["lr"]))
                assert torch.equal(p[i], opt.master[i].to(ptype))
            else:
                _adamw_bounds(w[0], p[i], ptype)
                w[0] = p[i].double()  # the next step starts from the rounded weight
            _close("m", opt.m[i], w[1], 1e-6 * w[1].abs() + 1e-12)
            _close("v", opt.v[i], w[2], 1e-6 * w[2].abs() + 1e-14)


@pytest.mark.parametrize("offset", [0, 1])
def test_adamw_8(offset):
    p, g = _adamw_lists(SIZES, [BF16] * len(SIZES), [F32] * len(SIZES), offset=offset)
    g[3][100:] = 0  # elements whose moments are zero
    g[9][:512] = 0  # whole blocks
    opt = vswin.AdamW(p, bits=8, weight_decay=0.1, **HYPER)
    for step in (1, 2, 3):
        m0, v0 = opt.moments()
        p0 = [t.double() for t in p]
        opt.step(g)
        for i in range(len(p)):
            w, m, v = ref.adamw(p0[i], g[i].double(), m0[i].double(), v0[i].double(), HYPER["lr"], *HYPER["betas"],
                                HYPER["eps"], 0.1, step)
            _adamw_bounds(w, p[i], BF16)
            n = p[i].numel()
            pad = lambda t: torch.nn.functional.pad(t, (0, -n % 256)).view(-1, 256)  # noqa: E731
            sm, sv = pad(m).abs().amax(1), pad(v).amax(1)
            _close("m_scale", opt.m_scale[i], sm, 1e-6 * sm)
            _close("v_scale", opt.v_scale[i], sv, 1e-6 * sv)
            one = lambda s: torch.where(s > 0, s, 1.0)[:, None]  # noqa: E731
            cm = 127 * (pad(m).abs() / one(sm)).sqrt()
            cv = 255 * (pad(v) / one(sv)) ** 0.25
            # the nearest code, up to fp32 errors of a few 2^-24 of the argument at a tie
            assert ((pad(opt.m[i].double()).abs() - cm).abs() <= 0.5 + 1e-4).all()
            assert (pad(opt.m[i].double()) * pad(m) >= 0).all()
            least = torch.where(pad(v) > 0, cv.clamp(min=1), cv)
            assert ((pad(opt.v[i].double()) - least).abs() <= 0.5 + 1e-4).all()
            dm, dv = vswin.adamw_decode(opt.m[i], opt.m_scale[i], opt.v[i], opt.v_scale[i])
            c = pad(opt.m[i].double())
            _close("decode m", pad(dm), opt.m_scale[i].double()[:, None] * c * c.abs() / 127**2, 1e-6 * sm[:, None])
            _close("decode v", pad(dv), opt.v_scale[i].double()[:, None] * (pad(opt.v[i].double()) / 255) ** 4,
                   1e-6 * sv[:, None])


def test_adamw_many_tensors_and_scaled_gradients():
    sizes = [1 + (37 * i) % 901 for i in range(420)]
    p, g = _adamw_lists(sizes, [F32] * 420, [F32] * 420)
    q = [t.clone() for t in p]
    gs = torch.tensor([0.25], device="cuda")
    vswin.AdamW(p, **HYPER).step(g, grad_scale=gs, lr=1e-2, step=7)
    for t, w, gr in zip(p, q, g):
        z = torch.zeros_like(w, dtype=torch.float64)
        want = ref.adamw(w.double(), gr.double() / 4, z, z, 1e-2, *HYPER["betas"], HYPER["eps"], 0.01, 7)[0]
        _close("param", t, want, 1e-6 * (want.abs() + 1e-2))


def test_adamw_refuses_a_weight_twice():
    p, g = _adamw_lists([100, 50], [BF16] * 2, [F32] * 2)
    with pytest.raises(ValueError, match="twice"):
        vswin.AdamW([p[0], p[1], p[0]])
    opt = vswin.AdamW(p)
    with pytest.raises(ValueError):
        opt.step(g[:1])
    with pytest.raises(ValueError, match=r"grads\[1\]"):
        opt.step([g[0], g[1][:49]])
    with pytest.raises(TypeError):
        opt.step(g, step=torch.ones(1, device="cuda"))


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_nan_gradients_show(bits):
    p, g = _adamw_lists([600], [F32], [F32])
    g[0][300] = math.nan
    opt = vswin.AdamW(p, bits=bits, **HYPER)
    opt.step(g)
    assert p[0][300].isnan() and int(p[0].isnan().sum()) == 1
    m, _ = opt.moments()
    assert m[0][300].isnan()
    assert torch.isfinite(m[0][:256]).all() and torch.isfinite(m[0][512:]).all()


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_captured(bits):
    sizes = [300, 5000]
    p, g = _adamw_lists(sizes, [BF16] * 2, [F32] * 2)
    q = [t.clone() for t in p]
    eager, captured = vswin.AdamW(p, bits=bits, **HYPER), vswin.AdamW(q, bits=bits, **HYPER)
    count = torch.zeros(1, dtype=torch.int32, device="cuda")
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        captured.step(g, step=count + 1)  # loads the kernel outside the capture
    s.synchronize()
    for t, u in zip(q, p):
        t.copy_(u)
    for t in captured.m + captured.v + (captured.m_scale + captured.v_scale if bits == 8 else []):
        t.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        count.add_(1)
        captured.step(g, step=count)
    for _ in range(3):
        graph.replay()
        eager.step(g)
    torch.cuda.synchronize()
    assert int(count) == 3
    for a, b in zip(p, q):
        # the corrections come from pow() on the device: the last bit of a scalar may differ
        assert ((a.double() - b.double()).abs() <= 2.0**-8 * a.double().abs() + 1e-7).all()


# ------------------------------------------------------------------ together
def _layer(i, kw, do, gen_grads):
    """A sequence layer's attention: norm and rotation, attention, and back."""
    qn, kn = vswin.qk_norm_forward(i["q"], i["k"], i["gq"], i["gk"], **i["kw"])
    out, lse = vswin.bias_attention_forward(qn, kn, i["v"], i["table"], i["map"], **kw)
    if not gen_grads:
        return out
    dqn, dkn, dv, dtable = vswin.bias_attention_backward(qn, kn, i["v"], i["table"], i["map"], out, lse, do, **kw)
    dq, dk, dgq, dgk = vswin.qk_norm_backward(i["q"], i["k"], i["gq"], i["gk"], dqn, dkn, **i["kw"])
    return out, dq, dk, dv, dtable, dgq, dgk


def _layer_inputs(B=2, L=200, hq=4, hk=2, d=64):
    i = _norm_inputs((BF16, B, L, hq, hk, d, d, False))
    gen = i["gen"]
    i["v"], i["table"], i["map"] = _rand(gen, (B, L, hk, d), BF16), _rand(gen, (32, hq), BF16, 0.5), _map(bidirectional=False)
    return i, _rand(gen, (B, L, hq, d), BF16)


def test_layer_trains_through_every_operator():
    """A training step: norm and rotation, attention, gradients back through both, AdamW on the weights; against the
    same chain in float64 (relative L2: four roundings to bf16 along the chain, each at most 2^-8)."""
    i, do = _layer_inputs()
    kw = dict(causal=True, q_lens=_i32(200, 150), kv_lens=_i32(200, 150))
    out, dq, dk, dv, dtable, dgq, dgk = _layer(i, kw, do, True)
    w = {n: i[n].double().requires_grad_() for n in ("q", "k", "v", "gq", "gk", "table")}
    rows = torch.arange(200, device="cuda")
    c, s = (t.double()[:200][None, :, None] for t in (i["kw"]["cos"], i["kw"]["sin"]))

    def turn(x, g):
        n = x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6) * g
        a, b = n[..., :32], n[..., 32:]
        return torch.cat((a * c - b * s, b * c + a * s), -1)

    Q, K = turn(w["q"], w["gq"]), turn(w["k"], w["gk"]).repeat_interleave(2, 2)
    V = w["v"].repeat_interleave(2, 2)
    rel = rows[None] - rows[:, None]
    score = torch.einsum("bihd,bjhd->bhij", Q, K) / 8 + w["table"][i["map"].long()[rel.clamp(-128, 128) + 128]].permute(2, 0, 1)
    live = torch.tensor([200, 150], device="cuda")[:, None] > rows
    score = score.masked_fill((rel > 0) | ~live[:, None, None], -math.inf)
    O = torch.einsum("bhij,bjhd->bihd", torch.softmax(score, -1), V) * live[:, :, None, None]
    O.backward(do.double())
    for n, got, want in (("out", out, O), ("dq", dq, w["q"].grad), ("dk", dk, w["k"].grad), ("dv", dv, w["v"].grad),
                         ("dtable", dtable, w["table"].grad), ("dgq", dgq, w["gq"].grad), ("dgk", dgk, w["gk"].grad)):
        rel_l2 = float((got.double() - want).norm() / want.norm())
        assert rel_l2 <= 4 * 2.0**-8, (n, rel_l2)
    params, grads = [i["gq"], i["gk"], i["table"]], [dgq, dgk, dtable]
    before = [p.double() for p in params]
    vswin.AdamW(params, weight_decay=0.0, **HYPER).step(grads)
    for p, b, g in zip(params, before, grads):
        want = ref.adamw(b, g.double(), 0 * b, 0 * b, HYPER["lr"], *HYPER["betas"], HYPER["eps"], 0.0, 1)[0]
        _adamw_bounds(want, p, BF16)


def test_layer_captured_equals_eager_on_another_stream():
    i, do = _layer_inputs()
    kw = dict(causal=True)
    eager = _layer(i, kw, do, True)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        warm = _layer(i, kw, do, True)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(eager, warm))
    graphs, outs = [], []
    for _ in range(2):  # two graphs alive at once, replayed on two streams
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            outs.append(_layer(i, kw, do, True))
        graphs.append(g)
    t = torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(s):
            graphs[0].replay()
        with torch.cuda.stream(t):
            graphs[1].replay()
    torch.cuda.synchronize()
    for o in outs:
        assert all(torch.equal(a, b) for a, b in zip(eager, o))


def test_token_by_token_equals_the_whole_sequence():
    """Serving: each new token's q and k normed at its position and run against the cache so far gives the rows of
    the whole sequence's forward (two bf16 roundings of the same exact values apart, plus the operands')."""
    B, L, hq, hk, d = 2, 70, 4, 2, 64
    i, _ = _layer_inputs(B, L, hq, hk, d)
    whole = _layer(i, dict(causal=True), None, False)
    kc = torch.full((B, L + 10, hk, d), math.nan, dtype=BF16, device="cuda")
    vc = torch.full_like(kc, math.nan)
    for t in range(L):
        kw = dict(i["kw"], positions=torch.full((B, 1), t, dtype=torch.int32, device="cuda"))
        qn, _ = vswin.qk_norm_forward(i["q"][:, t:t + 1], i["k"][:, t:t + 1], i["gq"], i["gk"], k_out=kc[:, t:t + 1], **kw)
        vc[:, t] = i["v"][:, t]
        n = torch.full((B,), t + 1, dtype=torch.int32, device="cuda")
        out, _ = vswin.bias_attention_forward(qn, kc, vc, i["table"], i["map"], causal=True, kv_lens=n, q_start=n - 1)
        bound = 2 * (2.0**-8) * (whole[:, t].double().abs() + i["v"][:, :t + 1].double().abs().amax(1).repeat_interleave(2, 1))
        assert ((out[:, 0].double() - whole[:, t].double()).abs() <= bound).all(), t


@pytest.mark.parametrize("Lq,Lk", [(150, 150), (1, 150), (1, 5000), (100, 6000)], ids=str)
def test_attention_nan_stays_in_its_row(Lq, Lk):
    # a query row of NaN gives a row of NaN and nothing else; a key of NaN reaches the rows that see it
    ins, _ = _attn_inputs(BF16, 2, Lq, Lk, 2, 2, 64)
    good = vswin.bias_attention_forward(*ins, _map())
    q = ins[0].clone()
    q[1, Lq // 2, 1] = math.nan
    out, lse = vswin.bias_attention_forward(q, *ins[1:], _map())
    assert out[1, Lq // 2, 1].isnan().all() and lse[1, 1, Lq // 2].isnan()
    rest = torch.ones_like(lse, dtype=torch.bool)
    rest[1, 1, Lq // 2] = False
    assert torch.equal(lse[rest], good[1][rest])
    assert torch.equal(out.transpose(1, 2)[rest], good[0].transpose(1, 2)[rest])
    k = ins[1].clone()
    k[0, Lk - 1, 0, 3] = math.nan
    out, lse = vswin.bias_attention_forward(ins[0], k, *ins[2:], _map(), kv_lens=_i32(Lk, Lk - 1))
    assert out[0, :, 0].isnan().all() and torch.isfinite(out[0, :, 1]).all() and torch.isfinite(out[1]).all()


@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("Lq,Lk", [(150, 150), (8, 150), (300, 1500)], ids=str)
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_attention_unseen_keys_may_hold_anything(d, Lq, Lk, bad):
    # keys that the causal rule or the bias takes out have the same effect whatever k holds: none
    ins, _ = _attn_inputs(BF16, 2, Lq, Lk, 2, 1, d)
    start = _i32(Lk - Lq - 3, Lk - Lq - 40)
    kw = dict(causal=True, q_start=start)
    good = vswin.bias_attention_forward(*ins, _map(), **kw)
    k = ins[1].clone()
    for b, n in enumerate(start.tolist()):
        k[b, n + Lq:] = bad
    got = vswin.bias_attention_forward(ins[0], k, *ins[2:], _map(), **kw)
    assert torch.equal(got[0], good[0]) and torch.equal(got[1], good[1])
    # rows before position Lk // 2 do not see that key
    k = ins[1].clone()
    k[:, Lk // 2] = bad
    got = vswin.bias_attention_forward(ins[0], k, *ins[2:], _map(), **kw)
    for b, n in enumerate(start.tolist()):
        rows = max(0, min(Lq, Lk // 2 - n))
        assert torch.equal(got[0][b, :rows], good[0][b, :rows]) and torch.equal(got[1][b, :, :rows], good[1][b, :, :rows])
    # a map whose bucket 1 (offset 1 alone) is taken out: query i does not see key i + 1
    every = torch.zeros(7, dtype=torch.int32, device="cuda")
    every[4] = 1
    table = torch.tensor([[0.5, -0.5], [-math.inf, -math.inf]], dtype=BF16, device="cuda")
    q_one = ins[0][:, :1].expand(2, Lq, 2, d)
    one = dict(q_start=_i32(Lk // 2 - 1, Lk // 2 - 1), q_lens=_i32(1, 1))
    good = vswin.bias_attention_forward(q_one, *ins[1:3], table, every, **one)
    got = vswin.bias_attention_forward(q_one, k, ins[2], table, every, **one)
    assert torch.isfinite(good[0]).all() and torch.equal(got[0], good[0]) and torch.equal(got[1], good[1])


def test_results_come_from_the_stream_of_the_call():
    # memory that the current stream still writes is not handed to a call on another stream
    ins, do = _attn_inputs(BF16, 1, 256, 256, 2, 2, 64)
    good = vswin.bias_attention_forward(*ins, _map())
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    busy = torch.empty_like(good[0])
    at = busy.data_ptr()
    busy.fill_(1.0)
    del busy
    out, lse = vswin.bias_attention_forward(*ins, _map(), stream=s)
    assert out.data_ptr() != at
    s.synchronize()
    assert torch.equal(out, good[0]) and torch.equal(lse, good[1])


def test_adamw_follows_an_exchanged_weight():
    n = 1000
    start = torch.randn(n, device="cuda", generator=torch.Generator("cuda").manual_seed(3))
    g = torch.ones(n, device="cuda")
    a, b = torch.nn.Parameter(start.clone()), torch.nn.Parameter(start.clone())
    oa, ob = vswin.AdamW([a], **HYPER), vswin.AdamW([b], **HYPER)
    old = a.data
    a.data = start.clone()
    before = old.clone()
    oa.step([g])
    ob.step([g])
    assert torch.equal(a.data, b.data) and torch.equal(old, before) and not torch.equal(a.data, before)
    a.data = torch.zeros(n + 1, device="cuda")
    with pytest.raises(ValueError, match=r"params\[0\]"):
        oa.step([g])
    torch.cuda.synchronize()


FIRST_CALLS = """
import torch
from shifted_window_attention_sw_b200 import vswin
q, k, v, do = (torch.randn(2, 200, 2, 64, device="cuda").bfloat16() for _ in range(4))
table, one = torch.randn(32, 2, device="cuda").bfloat16(), torch.ones(64, device="cuda").bfloat16()
bucket_map, p, g = vswin.bucket_map(32, 128), torch.randn(1000, device="cuda"), torch.randn(1000, device="cuda")
optimizer, count = vswin.AdamW([p]), torch.ones(1, dtype=torch.int32, device="cuda")
before = p.clone()
torch.cuda.synchronize()

def step():
    qn, kn = vswin.qk_norm_forward(q, k, one, one)
    out, lse = vswin.bias_attention_forward(qn, kn, v, table, bucket_map, causal=True)
    dq, dk, dv, dt = vswin.bias_attention_backward(qn, kn, v, table, bucket_map, out, lse, do, causal=True)
    return out, lse, dv, dt, *vswin.qk_norm_backward(q, k, one, one, dq, dk)

graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    captured = step()
    optimizer.step([g], step=count)
graph.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(captured, step())) and not torch.equal(p, before)
assert vswin.poll_error() == vswin.OK
"""


def test_first_calls_of_a_process_may_be_captured():
    subprocess.run([sys.executable, "-c", FIRST_CALLS], check=True, timeout=300,
                   cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("dtype,Lq,Lk", [(BF16, 130, 2100), (FP16, 511, 700), (BF16, 4, 2100)], ids=str)
def test_attention_scores_that_grow_along_the_keys(dtype, Lq, Lk, d, causal):
    # every tile raises the running maximum of most rows, so that the sums so far are rescaled again and again
    ins, do = _attn_inputs(dtype, 2, Lq, Lk, 4, 2, d)
    ins[1] = (ins[1].float() * torch.linspace(0.1, 1.0, Lk, device="cuda").view(1, Lk, 1, 1)).to(dtype)
    _attn_check(ins, _map(), do, scale=0.5, causal=causal, q_start=_i32(Lk - Lq, Lk - Lq), backward=causal)


def _adamw_8_definition(opt, p, g, i, wd, step, gs=1.0, w=None):
    """(p, m, v) of tensor i after a step from the codes that the object holds, float64, and the scales' blocks."""
    up = lambda s: s.double().repeat_interleave(256)[:p.numel()]  # noqa: E731
    c, d = opt.m[i].double().view(-1), opt.v[i].double().view(-1)
    m0, v0 = up(opt.m_scale[i]) * c * c.abs() / 127**2, up(opt.v_scale[i]) * (d / 255) ** 4
    w = p if w is None else w
    return ref.adamw(w.double().view(-1), gs * g.double().view(-1), m0, v0, HYPER["lr"], *HYPER["betas"], HYPER["eps"], wd, step)


def _block_max(x, n):
    return torch.nn.functional.pad(x, (0, -n % 256)).view(-1, 256).abs().amax(1)


@pytest.mark.parametrize("codes_from", [0, 1])
@pytest.mark.parametrize("offset", [0, 1])
def test_adamw_8_second_moments_that_are_not_finite(offset, codes_from):
    # scales of infinity and NaN beside finite first moments: v = scale (c / 255)^4 is infinite (no step), or NaN
    # (c = 0 of an infinite scale, every c of NaN), and then so is the weight; the last block is a partial one
    n = 900
    p, g = _adamw_lists([n], [F32], [F32], offset=offset)
    at = torch.arange(n, device="cuda")
    m, v = (at % 255 - 127).to(torch.int8), (codes_from + at % (256 - codes_from)).to(torch.uint8)
    ms = torch.full((4,), 1e-3, device="cuda")
    vs = torch.tensor([math.inf, math.nan, 1e-4, math.inf], device="cuda")
    opt = vswin.AdamW(p, bits=8, weight_decay=0.1, moments=([m], [v]), scales=([ms], [vs]), **HYPER)
    for step in (4, 5):
        w, mw, vw = _adamw_8_definition(opt, p[0], g[0], 0, 0.1, step)
        opt.step(g, step=step)
        _adamw_bounds(w, p[0], F32)
        sm, sv = _block_max(mw, n), _block_max(vw, n)
        _close("m_scale", opt.m_scale[0], sm, 1e-6 * sm)
        _close("v_scale", opt.v_scale[0], sv, torch.where(sv.isfinite(), 1e-6 * sv, 0.0))


def test_adamw_8_gradient_whose_square_overflows():
    # one gradient of 1e21: its v is infinite in fp32 and so is its block's scale, m stays finite. From then on the
    # block's weights stand still or are NaN, none is thrown far away; the other blocks go on
    n = 600
    p, g = _adamw_lists([n], [F32], [F32])
    opt = vswin.AdamW(p, bits=8, weight_decay=0.0, **HYPER)
    g[0][550] = 1e21
    opt.step(g)
    g[0][550] = 1e-2
    for step in (2, 3, 4):
        w, _, _ = _adamw_8_definition(opt, p[0], g[0], 0, 0.0, step)
        before = p[0].clone()
        opt.step(g)
        _adamw_bounds(w, p[0], F32)
        moved = (p[0] - before).abs()
        assert torch.isfinite(p[0][:512]).all()
        assert ((moved[512:] == 0) | moved[512:].isnan()).all()


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("d", [32, 64, 128])
def test_attention_gradient_leaves_bad_buckets_out(d, causal):
    # offsets whose map entry lies outside the table have bias 0 and belong to no row of its gradient: the same as
    # a further row of zeros in the table that they point to. Inside the map, and at its ends (tiles of one bucket)
    L, buckets, D = 700, 8, 40
    ins, do = _attn_inputs(BF16, 1, L, L, 2, 1, d, buckets=buckets)
    ins[3][0] = 0  # (a tile of bucket 0 and a tile of no bucket have the same values)
    good = vswin.bucket_map(buckets, D, True)
    for ends in (False, True):
        off = torch.zeros(2 * D + 1, dtype=torch.bool, device="cuda")
        off[5:70:7] = True
        off[0] = off[-1] = ends
        bad = torch.where(off, torch.where(torch.arange(2 * D + 1, device="cuda") % 2 == 0, -1, 1 << 20).int(), good)
        more = torch.cat((ins[3], torch.zeros_like(ins[3][:1])))
        moved = torch.where(off, buckets, good.long()).int()
        want = _attn_check([*ins[:3], more], moved, do, causal=causal)
        out, lse = vswin.bias_attention_forward(*ins, bad, causal=causal)
        got = out, lse, *vswin.bias_attention_backward(*ins, bad, out, lse, do, causal=causal)
        assert vswin.poll_error() == vswin.ERR_BOUNDS
        assert all(torch.equal(a, b) for a, b in zip(got[:5], want[:5]))
        assert torch.equal(got[5], want[5][:buckets])


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_follows_exchanged_states(bits):
    # a moment, scale or copy put in its list is the one that steps, and the one that it replaces is left alone
    p, g = _adamw_lists([700, 40], [BF16] * 2, [F32] * 2)
    q = [t.clone() for t in p]
    a, b = vswin.AdamW(p, bits=bits, master=True, **HYPER), vswin.AdamW(q, bits=bits, master=True, **HYPER)
    names = ["m", "v", "master"] + (["m_scale", "v_scale"] if bits == 8 else [])
    for _ in range(2):
        old = {n: [t for t in getattr(a, n)] for n in names}
        before = {n: [t.clone() for t in old[n]] for n in names}
        for n in names:
            for i, t in enumerate(old[n]):
                getattr(a, n)[i] = t.clone()
        a.step(g)
        b.step(g)
        for n in names:
            assert all(torch.equal(x, y) for x, y in zip(getattr(a, n), getattr(b, n))), n
            assert all(torch.equal(x, y) for x, y in zip(old[n], before[n])), n
        assert all(torch.equal(x, y) for x, y in zip(p, q))


@pytest.mark.parametrize("master", [None, True])
@pytest.mark.parametrize("ptype,gtype", [(BF16, BF16), (FP16, FP16), (F32, BF16), (BF16, F32)], ids=str)
def test_adamw_8_in_every_form(ptype, gtype, master):
    # copies, gradients' types and factor, and two launches' worth of tensors that start anywhere
    sizes = [1 + (211 * i) % 700 for i in range(200)]
    p, g = _adamw_lists(sizes, [ptype] * 200, [gtype] * 200, offset=1)
    opt = vswin.AdamW(p, bits=8, weight_decay=0.1, master=master, **HYPER)
    gs = torch.tensor([0.5], device="cuda")
    for step in (1, 2):
        want = [_adamw_8_definition(opt, p[i], g[i], i, 0.1, step, 0.5, opt.master[i] if master else None)
                for i in range(200)]
        opt.step(g, grad_scale=gs)
        for i, (w, m, v) in enumerate(want):
            n = sizes[i]
            if master:
                _close("master", opt.master[i], w, 2e-6 * (w.abs() + HYPER["lr"]))
                assert torch.equal(p[i], opt.master[i].to(ptype))
            else:
                _adamw_bounds(w, p[i], ptype)
            sm, sv = _block_max(m, n), _block_max(v, n)
            _close("m_scale", opt.m_scale[i], sm, 1e-6 * sm)
            _close("v_scale", opt.v_scale[i], sv, 1e-6 * sv)
            at = torch.arange(n, device="cuda") // 256
            # the nearest codes, up to fp32 errors of a few 2^-24 of the argument at a tie
            assert ((opt.m[i].double().abs() - 127 * (m.abs() / sm[at]).sqrt()).abs() <= 0.5 + 1e-4).all()
            assert (opt.m[i].double() * m >= 0).all()
            assert ((opt.v[i].double() - (255 * (v / sv[at]) ** 0.25).clamp(min=1)).abs() <= 0.5 + 1e-4).all()


@pytest.mark.parametrize("dtype,B,L,hq,hk,d,causal", [
    (FP16, 1, 2113, 16, 4, 128, True), (BF16, 1, 1500, 32, 1, 64, True), (BF16, 2, 1217, 8, 2, 32, False),
    (FP16, 1, 5003, 2, 1, 64, True), (BF16, 1, 5003, 2, 2, 128, False),
], ids=str)
def test_attention_gradient_of_long_sequences_and_shared_heads(dtype, B, L, hq, hk, d, causal):
    ins, do = _attn_inputs(dtype, B, L, L, hq, hk, d)
    lens = _i32(*[L - 37 * b for b in range(B)])
    _attn_check(ins, _map(bidirectional=not causal), do, causal=causal, q_lens=lens, kv_lens=lens)


def test_two_layers_at_once():
    # the whole chain on two streams at the same time, many times over: the same bits as alone
    i, do = _layer_inputs(2, 600)
    kw = dict(causal=True)
    want = _layer(i, kw, do, True)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(20):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(_layer(i, kw, do, True))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for g in got for a, b in zip(g, want))


@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("L", [1, 130, 700])
@pytest.mark.parametrize("heads_first", [False, True])
def test_results_in_further_heads_of_the_inputs_buffer(d, L, heads_first):
    # q, k, v, out, dout, dq, dk, dv and the norm's results interleave in one buffer: the same bits as apart
    B, hq, hk = 2, 4, 2
    ins, do = _attn_inputs(BF16, B, L, L, hq, hk, d)
    gen = torch.Generator().manual_seed(9)
    w = [_rand(gen, (d,), BF16) for _ in range(2)]
    q, k, v, table = ins
    qn, kn = vswin.qk_norm_forward(q, k, *w)
    out, lse = vswin.bias_attention_forward(qn, kn, v, table, _map())
    grads = vswin.bias_attention_backward(qn, kn, v, table, _map(), out, lse, do)
    back = vswin.qk_norm_backward(q, k, *w, grads[0], grads[1])
    sizes = dict(q=hq, qn=hq, k=hk, kn=hk, v=hk, out=hq, do=hq, dqn=hq, dkn=hk, dv=hk, dq=hq, dk=hk)
    total = sum(sizes.values())
    buf = torch.zeros((B, total, L, d) if heads_first else (B, L, total, d), dtype=BF16, device="cuda")
    every, s, at = buf.transpose(1, 2) if heads_first else buf, {}, 0
    for n, heads in sizes.items():
        s[n] = every[:, :, at:at + heads]
        at += heads
    for n, x in dict(q=q, k=k, v=v, do=do).items():
        s[n].copy_(x)
    vswin.qk_norm_forward(s["q"], s["k"], *w, q_out=s["qn"], k_out=s["kn"])
    o, e = vswin.bias_attention_forward(s["qn"], s["kn"], s["v"], table, _map(), out=s["out"])
    g = vswin.bias_attention_backward(s["qn"], s["kn"], s["v"], table, _map(), o, e, s["do"], dq=s["dqn"], dk=s["dkn"],
                                      dv=s["dv"])
    h = vswin.qk_norm_backward(s["q"], s["k"], *w, g[0], g[1], dq=s["dq"], dk=s["dk"])
    for n, x in dict(q=q, k=k, v=v, do=do, qn=qn, kn=kn, out=out, dqn=grads[0], dkn=grads[1], dv=grads[2], dq=back[0],
                     dk=back[1]).items():
        assert torch.equal(s[n], x), n
    assert torch.equal(e, lse) and all(torch.equal(a, b) for a, b in zip((g[3], *h[2:]), (grads[3], *back[2:])))
