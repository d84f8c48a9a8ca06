"""The operators over token sequences and the optimizer step on the host: refusals before any launch, the bucket
map, and the float64 definitions against central differences. CPU only."""

import ctypes
import math
import os
import random
import re
from fractions import Fraction

import pytest
import torch

import sequence_reference as ref
from shifted_window_attention_sw_b200 import build as build_mod
from shifted_window_attention_sw_b200 import vswin


@pytest.fixture(scope="module")
def L():
    build_mod.build()
    return vswin.lib()


# fake device pointers, 16 MB apart: never dereferenced, because validation fails first
def P(n, off=0):
    return (n << 24) + off


def _view(n, L, H, d, off=0, **kw):
    s = dict(batch_stride=L * H * d, token_stride=H * d, head_stride=d)
    s.update(kw)
    return vswin._Heads(P(n, off) if n else None, s["batch_stride"], s["token_stride"], s["head_stride"])


def _norm(L, dtype=0, B=2, Lt=8, hq=4, hk=2, d=64, q=None, k=None, gq=3, gk=4, eps=1e-6, rot=None, qo=None, ko=None,
          back=None):
    q = _view(1, Lt, max(hq, 1), d) if q is None else q
    k = _view(2, Lt, max(hk, 1), d) if k is None else k
    qo = _view(5, Lt, max(hq, 1), d) if qo is None else qo
    ko = _view(6, Lt, max(hk, 1), d) if ko is None else ko
    args = [dtype, B, Lt, hq, hk, d, q, k, P(gq) if gq else None, P(gk) if gk else None, eps, rot, qo, ko]
    if back is None:
        return L.vswin_qk_norm_forward(*args, None)
    b = dict(dq=_view(7, Lt, hq, d), dk=_view(8, Lt, hk, d), g=P(9), h=P(10))
    b.update(back)
    return L.vswin_qk_norm_backward(*args, b["dq"], b["dk"], b["g"], b["h"], None)


def _refused(L, rc, status=vswin.ERR_INVALID_ARG, before=None):
    assert rc == status, (rc, vswin.last_error())
    assert vswin.last_error()
    assert vswin.launch_count() == before


def _rot(rows=8, dim=32, cos=11, sin=12, positions=None, inter=0):
    return vswin._Rotation(P(cos) if cos else None, P(sin) if sin else None, rows, dim, inter, positions)


@pytest.mark.parametrize("kw", [
    dict(dtype=3), dict(dtype=-1), dict(B=0), dict(Lt=0), dict(hq=0), dict(hk=-1), dict(d=0), dict(eps=-1.0),
    dict(eps=math.inf), dict(eps=math.nan), dict(gq=0), dict(gk=0), dict(q=_view(0, 8, 4, 64)),
    dict(q=_view(1, 8, 4, 64, off=1)), dict(q=_view(1, 8, 4, 64, token_stride=-4)),
    dict(qo=_view(5, 8, 4, 64, token_stride=0)), dict(qo=_view(5, 8, 4, 64, head_stride=32)),
    dict(qo=_view(1, 8, 4, 64, off=64)), dict(qo=_view(2, 8, 4, 64)), dict(ko=_view(5, 8, 2, 64)),
    dict(rot=_rot(dim=33)), dict(rot=_rot(dim=66)), dict(rot=_rot(dim=-2)), dict(rot=_rot(cos=0)), dict(rot=_rot(sin=0)),
    dict(rot=_rot(rows=0)), dict(rot=_rot(rows=7)), dict(rot=_rot(positions=P(13, 2))),
    dict(back=dict(g=None)), dict(back=dict(g=P(10))), dict(back=dict(h=P(1, 64))), dict(back=dict(dq=_view(2, 8, 4, 64))),
    dict(hk=4, k=_view(1, 8, 4, 64), qo=_view(1, 8, 4, 64)), dict(back=dict(dq=_view(7, 8, 4, 64, batch_stride=64))), dict(back=dict(dk=_view(7, 8, 2, 64))),
], ids=str)
def test_norm_refusals(L, kw):
    before = vswin.launch_count()
    _refused(L, _norm(L, **kw), before=before)


def test_norm_unsupported_width(L):
    before = vswin.launch_count()
    _refused(L, _norm(L, d=257), vswin.ERR_UNSUPPORTED, before)


@pytest.mark.parametrize("kw", [dict(hq=(1 << 20) + 1), dict(hk=(1 << 20) + 1), dict(B=1 << 16, Lt=1 << 15)], ids=str)
def test_norm_unsupported_sizes(L, kw):
    before = vswin.launch_count()
    _refused(L, _norm(L, **kw), vswin.ERR_UNSUPPORTED, before)


def _attn(L, dtype=0, B=2, Lq=8, Lk=8, hq=4, hk=2, d=64, q=None, k=None, v=None, scale=0.125, table=4, bmap=5, buckets=32,
          D=128, vis=None, out=None, lse=7, back=None):
    q = _view(1, Lq, max(hq, 1), d) if q is None else q
    k = _view(2, Lk, max(hk, 1), d) if k is None else k
    v = _view(3, Lk, max(hk, 1), d) if v is None else v
    out = _view(6, Lq, max(hq, 1), d) if out is None else out
    bias = vswin._BucketBias(P(table) if table else None, P(bmap) if bmap else None, buckets, D)
    args = [dtype, B, Lq, Lk, hq, hk, d, q, k, v, scale, bias, vis, out, P(lse) if lse else None]
    if back is None:
        return L.vswin_bias_attention_forward(*args, None)
    b = dict(do=_view(8, Lq, hq, d), dq=_view(9, Lq, hq, d), dk=_view(10, Lk, hk, d), dv=_view(11, Lk, hk, d), dt=P(12))
    b.update(back)
    return L.vswin_bias_attention_backward(*args, b["do"], b["dq"], b["dk"], b["dv"], b["dt"], None)


@pytest.mark.parametrize("kw", [
    dict(dtype=5), dict(B=0), dict(Lq=0), dict(Lk=0), dict(hq=0), dict(hk=0), dict(d=0), dict(hq=3), dict(scale=math.nan),
    dict(scale=math.inf), dict(scale=-2e30), dict(table=0), dict(bmap=0), dict(buckets=0), dict(buckets=513), dict(D=-1), dict(D=2**20 + 1),
    dict(lse=0), dict(q=_view(1, 8, 4, 64, off=8)), dict(k=_view(2, 8, 2, 64, token_stride=132)),
    dict(v=_view(0, 8, 2, 64)), dict(out=_view(1, 8, 4, 64)), dict(out=_view(2, 8, 4, 64, off=256)),
    dict(out=_view(6, 8, 4, 64, head_stride=0)), dict(lse=6), dict(lse=1),
    dict(vis=vswin._Visibility(P(13, 2), None, None, 0)), dict(vis=vswin._Visibility(None, P(13, 1), None, 0)),
    dict(vis=vswin._Visibility(None, None, P(13, 3), 1)),
    dict(back=dict(dt=None)), dict(back=dict(dt=P(9))), dict(back=dict(dt=P(4))), dict(back=dict(dq=_view(1, 8, 4, 64))),
    dict(back=dict(dk=_view(8, 8, 2, 64))), dict(back=dict(dk=_view(9, 8, 2, 64))), dict(back=dict(dv=_view(10, 8, 2, 64))),
    dict(back=dict(dv=_view(11, 8, 2, 64, token_stride=64))), dict(back=dict(do=_view(8, 8, 4, 64, off=2))),
], ids=str)
def test_attention_refusals(L, kw):
    before = vswin.launch_count()
    _refused(L, _attn(L, **kw), before=before)


@pytest.mark.parametrize("kw", [dict(dtype=2), dict(d=48), dict(d=256), dict(Lk=2**28 + 1), dict(hq=8192, hk=8192)], ids=str)
def test_attention_unsupported(L, kw):
    before = vswin.launch_count()
    _refused(L, _attn(L, **kw), vswin.ERR_UNSUPPORTED, before)


def _adam(L, bits=32, lr=1e-3, b1=0.9, b2=0.99, eps=1e-8, step=1, count=1, step_dev=None, gs=None, **kw):
    f = dict(param=P(1), master=None, grad=P(2), m=P(3), v=P(4), m_scale=P(5), v_scale=P(6), n=1000, weight_decay=0.1,
             param_dtype=0, grad_dtype=2)
    f.update(kw)
    t = (vswin._AdamwTensor * 1)(vswin._AdamwTensor(*(f[n] for n, _ in vswin._AdamwTensor._fields_)))
    return L.vswin_adamw_step(t if count else None, abs(count), bits, lr, b1, b2, eps, step, step_dev, gs, None)


@pytest.mark.parametrize("kw", [
    dict(bits=16), dict(lr=-1.0), dict(lr=math.inf), dict(b1=1.0), dict(b2=-0.1), dict(eps=-1.0), dict(step=0),
    dict(step_dev=P(9, 1)), dict(gs=P(9, 2)), dict(n=-1), dict(param_dtype=3), dict(grad_dtype=-1), dict(param=None),
    dict(grad=None), dict(m=None), dict(v=P(4, 2)), dict(master=P(7, 2)), dict(master=P(1)), dict(grad=P(1, 16)), dict(m=P(4)),
    dict(bits=8, m_scale=None), dict(bits=8, v_scale=P(6, 1)), dict(bits=8, v_scale=P(5)), dict(weight_decay=math.nan),
    dict(weight_decay=-0.1),
], ids=str)
def test_adamw_refusals(L, kw):
    before = vswin.launch_count()
    _refused(L, _adam(L, **kw), before=before)


def test_decode_refusals(L):
    before = vswin.launch_count()
    args = [P(1), P(2), P(3), P(4), 100, 2, P(5), P(6), None]
    for at, v in ((0, None), (1, P(2, 1)), (3, None), (4, -1), (5, 7), (6, P(1)), (7, P(5)), (7, P(6, 2))):
        _refused(L, L.vswin_adamw_decode(*args[:at], v, *args[at + 1:]), before=before)


def test_binding_refuses_before_the_library(L):
    x = torch.zeros(1, 4, 2, 64, dtype=torch.bfloat16)
    w, t, m = x[0, 0, 0], torch.zeros(32, 2, dtype=torch.bfloat16), vswin.bucket_map(32, 128, device="cpu")
    with pytest.raises(ValueError, match="CUDA"):
        vswin.qk_norm_forward(x, x, w, w)
    with pytest.raises(ValueError, match="CUDA"):
        vswin.bias_attention_forward(x, x, x, t, m)
    with pytest.raises(TypeError):
        vswin.qk_norm_forward(x.double(), x, w, w)
    with pytest.raises(ValueError):
        vswin.qk_norm_forward(x[0], x, w, w)
    with pytest.raises(ValueError):
        vswin.bias_attention_forward(x, x, x, t, m[:-1])
    with pytest.raises(ValueError):
        vswin.AdamW([])
    with pytest.raises(ValueError, match="CUDA"):
        vswin.AdamW([w])


# ------------------------------------------------------------------ bucket map
def _exact_bucket(rel, buckets, D, bidirectional):
    side = buckets // 2 if bidirectional else buckets
    near = side // 2
    n = abs(rel) if bidirectional else max(-rel, 0)
    b = n
    if n >= near:
        m, t = side - near, 0
        # largest t < m with (n / near)^m >= (D / near)^t, in whole numbers
        while t + 1 < m and Fraction(n, near) ** m >= Fraction(D, near) ** (t + 1):
            t += 1
        b = near + t
    return b + (side if bidirectional and rel > 0 else 0)


@pytest.mark.parametrize("buckets,D,bidirectional", [(32, 128, True), (32, 128, False), (8, 16, True), (2, 5, False),
                                                     (64, 512, True), (10, 81, False), (4, 2, True)], ids=str)
def test_bucket_map(L, buckets, D, bidirectional):
    got = vswin.bucket_map(buckets, D, bidirectional, device="cpu").tolist()
    assert got == [_exact_bucket(r, buckets, D, bidirectional) for r in range(-D, D + 1)]


@pytest.mark.parametrize("args", [(1, 128, True), (0, 128, False), (31, 128, True), (32, 8, True), (32, 2**20 + 1, True)])
def test_bucket_map_refusals(L, args):
    with pytest.raises(vswin.VswinError) as e:
        vswin.bucket_map(*args, device="cpu")
    assert e.value.status == vswin.ERR_INVALID_ARG


# ------------------------------------------------------------------ definitions against differences
def _along(f, xs, us, h=1e-5):
    """Central difference of the scalar f along the directions us."""
    return (f(*[x + h * u for x, u in zip(xs, us)]) - f(*[x - h * u for x, u in zip(xs, us)])) / (2 * h)


@pytest.mark.parametrize("interleaved", [False, True])
def test_norm_definition(interleaved):
    g = torch.Generator().manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    x, w, dy, a = r(2, 3, 2, 10), r(10), r(2, 3, 2, 10), r(5, 3)
    pos = torch.tensor([[0, 4, 2], [1, 1, 3]])
    kw = dict(eps=1e-3, cos=a.cos(), sin=a.sin(), positions=pos, interleaved=interleaved)
    res = ref.qk_norm(x, w, dy=dy, **kw)
    ux, uw = r(*x.shape), r(*w.shape)
    num = _along(lambda x, w: (ref.qk_norm(x, w, **kw)["y"] * dy).sum(), (x, w), (ux, uw))
    assert abs(num - (res["dx"] * ux).sum() - (res["dgamma"] * uw).sum()) < 1e-7 * (1 + abs(num))


def test_attention_definition():
    g = torch.Generator().manual_seed(2)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    q, k, v, do, t = r(2, 5, 4, 8), r(2, 7, 2, 8), r(2, 7, 2, 8), r(2, 5, 4, 8), r(6, 4)
    t[2, 1] = -math.inf
    m = torch.randint(0, 6, (7,), generator=g)
    kw = dict(causal=True, q_lens=[5, 3], kv_lens=[6, 7], q_start=[2, -1])
    res = ref.bias_attention(q, k, v, t, m, 0.3, dout=do, **kw)
    us = [r(*x.shape) for x in (q, k, v, t)]
    num = _along(lambda q, k, v, t: (ref.bias_attention(q, k, v, t, m, 0.3, **kw)["out"] * do).sum(), (q, k, v, t), us)
    got = sum((res[n] * u).sum() for n, u in zip(("dq", "dk", "dv", "dtable"), us))
    assert abs(num - got) < 1e-6 * (1 + abs(num))
    assert res["lse"][1, :, 0].eq(-math.inf).all() and res["out"][1, 0].eq(0).all()


def test_adamw_definition():
    g = torch.Generator().manual_seed(3)
    p = torch.randn(50, generator=g, dtype=torch.float64, requires_grad=True)
    opt = torch.optim.AdamW([p], lr=1e-2, betas=(0.8, 0.95), eps=1e-6, weight_decay=0.3)
    w, m, v = p.detach().clone(), torch.zeros(50).double(), torch.zeros(50).double()
    for step in (1, 2, 3):
        p.grad = torch.randn(50, generator=g, dtype=torch.float64)
        w, m, v = ref.adamw(w, p.grad, m, v, 1e-2, 0.8, 0.95, 1e-6, 0.3, step)
        opt.step()
        assert torch.allclose(w, p.detach(), rtol=1e-12, atol=1e-14)


def test_ctypes_records_match_the_header():
    assert ctypes.sizeof(vswin._Heads) == 32 and ctypes.sizeof(vswin._Rotation) == 40
    assert ctypes.sizeof(vswin._BucketBias) == 24 and ctypes.sizeof(vswin._Visibility) == 32
    assert ctypes.sizeof(vswin._AdamwTensor) == 80


def test_kernels_hold_their_tensor_memory_before_the_next_may_start():
    """A kernel that lets its follower start early takes its tensor memory first. The follower's blocks hold theirs
    while they wait for the whole kernel: one that had started, but not taken its own, could wait for them in turn."""
    csrc = os.path.join(os.path.dirname(vswin.__file__), "csrc")
    seen = 0
    for name in sorted(os.listdir(csrc)):
        with open(os.path.join(csrc, name)) as f:
            text = re.sub(r"//[^\n]*", "", f.read())
        for kernel in re.split(r"__global__", text)[1:]:
            if "let_next_start()" not in kernel or "tmem_alloc(" not in kernel:
                continue
            seen += 1
            # taken by one warp, so that the block has to meet before it speaks for all of its threads
            taken = kernel.index("__syncthreads()", kernel.index("tmem_alloc("))
            assert taken < kernel.index("let_next_start()"), name
    assert seen >= 2


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_steps_the_tensors_that_stand_in_its_lists(monkeypatch, bits):
    # the records of a step on tensors that are taken for CUDA ones; the library is not called
    steps = []
    monkeypatch.setattr(torch.Tensor, "is_cuda", property(lambda t: True), raising=False)
    monkeypatch.setattr(vswin, "lib", lambda: type("", (), {"vswin_adamw_step": None}))
    monkeypatch.setattr(vswin, "_run", lambda fn, dev, stream, records, *a: steps.append(
        [{n: getattr(r, "param" if n == "params" else n) for n in names} for r in records]))
    names = ["params", "m", "v", "master"] + (["m_scale", "v_scale"] if bits == 8 else [])
    opt = vswin.AdamW([torch.zeros(300), torch.zeros(7, 5)], bits=bits, master=True)
    grads = [torch.ones(300), torch.ones(7, 5)]
    at = lambda: [{n: getattr(opt, n)[i].data_ptr() for n in names} for i in range(2)]  # noqa: E731
    opt.step(grads)
    assert steps[-1] == at()
    for n in names:
        old = getattr(opt, n)[1]
        getattr(opt, n)[1] = old.clone()
        opt.step(grads)
        assert steps[-1] == at() and steps[-1][1][n] != old.data_ptr(), n
        getattr(opt, n)[0].data = getattr(opt, n)[0].clone()
        opt.step(grads)
        assert steps[-1] == at(), n
        # one that does not fit is refused, and what was there is stepped on when it is put back
        count, first, good = len(steps), opt.params[0], getattr(opt, n)[1]
        opt.params[0], getattr(opt, n)[1] = first.clone(), torch.zeros(3, 3, dtype=old.dtype)
        with pytest.raises(ValueError, match=rf"{n}\[1\]"):
            opt.step(grads)
        opt.params[0], getattr(opt, n)[1] = first, good
        assert len(steps) == count
        opt.step(grads)
        assert steps[-1] == at(), n
    opt.master = None
    opt.step(grads)
    assert [r["master"] for r in steps[-1]] == [None, None]


@pytest.mark.parametrize("stride", [-1, -2**63, 2**63 - 1, 3])
def test_strides_of_extents_of_one_are_not_looked_at(L, stride):
    # one sequence, one token or one head: such a stride is never used. What is refused is something else
    before = vswin.launch_count()
    lone = dict(batch_stride=stride, token_stride=stride, head_stride=stride)
    one = [_view(n, 1, 1, 64, **lone) for n in range(1, 9)]
    _refused(L, _norm(L, B=1, Lt=1, hq=1, hk=1, q=one[0], k=one[1], qo=one[4], ko=one[5], rot=_rot(dim=33)), before=before)
    assert "rotation" in vswin.last_error()
    _refused(L, _norm(L, B=1, Lt=1, hq=1, hk=1, q=one[0], k=one[1], qo=one[4], ko=one[5],
                      back=dict(dq=one[6], dk=one[7], h=None)), before=before)
    assert "dgamma" in vswin.last_error()
    _refused(L, _attn(L, B=1, Lq=1, Lk=1, hq=1, hk=1, q=one[0], k=one[1], v=one[2], out=one[5], lse=0), before=before)
    assert "lse" in vswin.last_error()
    _refused(L, _attn(L, B=1, Lq=1, Lk=1, hq=1, hk=1, q=one[0], k=one[1], v=one[2], out=one[5],
                      back=dict(do=one[7], dq=_view(9, 1, 1, 64, **lone), dk=_view(10, 1, 1, 64, **lone),
                                dv=_view(11, 1, 1, 64, **lone), dt=None)), before=before)
    assert "dtable" in vswin.last_error()
    # with two of them it counts
    lone["head_stride"] = 64
    if stride != 3:
        _refused(L, _norm(L, B=2, Lt=1, hq=1, hk=1, q=_view(1, 1, 1, 64, **lone), rot=_rot(dim=33)), before=before)
        assert "stride" in vswin.last_error()


# ------------------------------------------------------------------ what may share memory
@pytest.fixture
def no_launch(L):
    # a call that passes its checks ends at the injected failure, before it touches a device
    yield lambda: L.vswin_test_inject_failure(vswin.INJECT_CUDA, 1)
    L.vswin_test_inject_failure(vswin.INJECT_CUDA, 0)


def _verdict(L, no_launch, call):
    """True when the call's arguments are accepted, False when they are refused."""
    no_launch()
    rc = call()
    L.vswin_test_inject_failure(vswin.INJECT_CUDA, 0)
    assert rc in (vswin.ERR_CUDA, vswin.ERR_INVALID_ARG), vswin.last_error()
    assert rc == vswin.ERR_INVALID_ARG or "injected" in vswin.last_error()
    return rc == vswin.ERR_CUDA


def _slice(n, first, heads=8, Lt=8, d=64, es=2, **kw):
    """Heads from `first` on of a (B, Lt, heads, d) buffer."""
    return _view(n, Lt, heads, d, off=first * d * es, **kw)


def test_norm_in_place_beside_the_other_tensor(L, no_launch):
    ok = lambda **kw: _verdict(L, no_launch, lambda: _norm(L, **kw))  # noqa: E731
    q, k = _slice(1, 0), _slice(1, 4)  # heads 0 to 3 and 4 to 5 of one buffer
    assert ok(q=q, k=k, qo=q, ko=k) and ok(q=q, k=k, qo=q) and ok(q=q, k=k, ko=k)
    for first in (1, 2, 3):  # k shares heads with the q that is replaced, or the other way round
        k = _slice(1, first)
        assert not ok(q=q, k=k, qo=q) and not ok(q=q, k=k, ko=k) and not ok(q=q, k=k, qo=q, ko=k)
        assert ok(q=q, k=k)  # reading the same heads twice is fine
    grads = lambda **kw: ok(back=dict(g=P(9), h=P(10), **kw))  # noqa: E731
    a, b = _slice(7, 0), _slice(7, 4)
    assert grads(dq=a, dk=b)
    dy = dict(qo=_slice(5, 0), ko=_slice(5, 2))  # output gradients that share heads 2 and 3
    back = lambda **kw: ok(**dy, back=kw)  # noqa: E731
    assert not back(dq=_slice(5, 0)) and not back(dk=_slice(5, 2)) and back(dq=a, dk=b)
    dy = dict(qo=_slice(5, 0), ko=_slice(5, 4))
    assert back(dq=_slice(5, 0), dk=_slice(5, 4)) and back(dq=_slice(5, 0)) and not back(dq=_slice(5, 1))


def test_results_may_interleave_with_inputs(L, no_launch):
    # q, k and v of a projection, and the results in further heads of the same buffer, in either order of heads and tokens
    for order in (dict(heads=16), dict(heads=16, batch_stride=16 * 8 * 64, token_stride=64, head_stride=8 * 64)):
        s = lambda first: _view(1, 8, 16, 64, off=2 * first * (order.get("head_stride", 64)),  # noqa: E731
                                **{n: x for n, x in order.items() if n != "heads"})
        assert _verdict(L, no_launch, lambda: _norm(L, q=s(0), k=s(4), qo=s(8), ko=s(12)))
        assert not _verdict(L, no_launch, lambda: _norm(L, q=s(0), k=s(4), qo=s(3), ko=s(12)))
        assert _verdict(L, no_launch, lambda: _attn(L, q=s(0), k=s(4), v=s(6), out=s(8)))
        assert not _verdict(L, no_launch, lambda: _attn(L, q=s(0), k=s(4), v=s(6), out=s(5)))
        assert _verdict(L, no_launch, lambda: _attn(L, q=s(0), k=s(4), v=s(6), out=s(8), back=dict(dv=s(12), dk=s(14))))
        assert not _verdict(L, no_launch, lambda: _attn(L, q=s(0), k=s(4), v=s(6), out=s(8), back=dict(dv=s(11), dk=s(14))))


def _elements(off, n, s, d):
    return {off + b * s[0] + t * s[1] + h * s[2] + c for b in range(n[0]) for t in range(n[1]) for h in range(n[2])
            for c in range(d)}


def test_overlap_of_any_two_views(L, no_launch):
    # an output and an input of random extents and strides: refused when an element is in both, and only then
    rng = random.Random(5)
    seen = {True: 0, False: 0}
    for _ in range(3000):
        d, n = rng.choice([1, 2, 3, 5]), [rng.randint(1, 3) for _ in range(3)]
        dims = rng.sample(range(3), 3)
        so, span = [0, 0, 0], d
        for k in dims:  # an output holds nothing twice
            so[k] = span + rng.choice([0, 0, 1, 4, 11])
            span += (n[k] - 1) * so[k]
        si = so if rng.random() < 0.3 else [rng.choice([0, 1, 2, d, 2 * d, 3 * d + 1, 17]) for _ in range(3)]
        hk, off = rng.randint(1, 3), rng.randint(-40, 40)
        view = lambda off, s: vswin._Heads(P(1) + 2 * off, *s)  # noqa: E731
        q, qo = view(off, si), view(0, so)
        if off == 0 and all(a == b or m == 1 for a, b, m in zip(si, so, n)):
            continue  # in place
        shared = bool(_elements(0, n, so, d) & _elements(off, n, si, d))
        got = _verdict(L, no_launch, lambda: _norm(L, B=n[0], Lt=n[1], hq=n[2], hk=hk, d=d, q=q, qo=qo,
                                                   k=_view(2, n[1], hk, d), ko=_view(6, n[1], hk, d)))
        assert got == (not shared), (d, n, so, si, off)
        seen[shared] += 1
    assert min(seen.values()) > 300, seen


def test_results_that_share_elements_are_refused(L, no_launch):
    # results of one call in one buffer: neighbouring heads or interleaved channels are fine, shared ones are not
    ok = lambda call: _verdict(L, no_launch, call)  # noqa: E731
    for first, good in ((4, True), (3, False), (1, False), (0, False)):
        assert ok(lambda: _norm(L, qo=_slice(5, 0), ko=_slice(5, first))) == good, first
        assert ok(lambda: _norm(L, back=dict(dq=_slice(7, 0), dk=_slice(7, first)))) == good, first
        assert ok(lambda: _attn(L, back=dict(dq=_slice(9, 0), dk=_slice(9, first)))) == good, first
        assert ok(lambda: _attn(L, back=dict(dq=_slice(9, 0), dv=_slice(9, first)))) == good, first
    for first, good in ((2, True), (1, False), (0, False)):
        assert ok(lambda: _attn(L, back=dict(dk=_slice(9, 4), dv=_slice(9, 4 + first), dq=_slice(9, 0)))) == good, first
    pair = lambda n, at: _view(n, 8, 4, 64, off=2 * at, batch_stride=8 * 4 * 128, token_stride=4 * 128, head_stride=128)  # noqa: E731
    assert ok(lambda: _norm(L, hk=4, qo=pair(5, 0), ko=pair(5, 64)))
    assert not ok(lambda: _norm(L, hk=4, qo=pair(5, 0), ko=pair(5, 63)))


def test_results_over_what_a_call_reads_beside_the_views(L, no_launch):
    # weights, angles, positions, the bias table and its map, lengths and starts: no result lies over one of them
    ok = lambda call: _verdict(L, no_launch, call)  # noqa: E731
    rot = lambda **kw: _rot(**{**dict(dim=32, rows=8, positions=P(13)), **kw})  # noqa: E731
    assert ok(lambda: _norm(L, rot=rot())) and ok(lambda: _norm(L, rot=rot(), back={}))
    size = 2 * 8 * 4 * 64 * 2  # bytes of q_out
    for at in (0, size - 64):  # at its first element, and over its last ones
        for kw in (dict(gq=5), dict(gk=5), dict(rot=rot(cos=5)), dict(rot=rot(sin=5)), dict(rot=rot(positions=P(5)))):
            qo = _view(5, 8, 4, 64, off=-at)
            assert not ok(lambda: _norm(L, **{**dict(rot=rot(), qo=qo), **kw})), (at, kw)
        for kw in (dict(gq=7), dict(gk=7), dict(rot=rot(cos=7)), dict(rot=rot(sin=7)), dict(rot=rot(positions=P(7)))):
            assert not ok(lambda: _norm(L, **{**dict(rot=rot()), **kw}, back=dict(dq=_view(7, 8, 4, 64, off=-at)))), (at, kw)
    for kw in (dict(rot=rot(cos=9)), dict(rot=rot(sin=10)), dict(rot=rot(positions=P(9)))):
        assert not ok(lambda: _norm(L, **kw, back={})), kw
    lens = lambda a=14, b=15, c=16: vswin._Visibility(P(a), P(b), P(c), 1)  # noqa: E731
    assert ok(lambda: _attn(L, vis=lens())) and ok(lambda: _attn(L, vis=lens(), back={}))
    for n in (6, 7):  # out, lse
        for kw in (dict(table=n), dict(bmap=n), dict(vis=lens(a=n)), dict(vis=lens(b=n)), dict(vis=lens(c=n))):
            assert not ok(lambda: _attn(L, **{**dict(vis=lens()), **kw})), (n, kw)
    for n in (9, 10, 11, 12):  # dq, dk, dv, dtable
        for kw in (dict(table=n), dict(bmap=n), dict(vis=lens(a=n)), dict(vis=lens(b=n)), dict(vis=lens(c=n))):
            assert not ok(lambda: _attn(L, **{**dict(vis=lens()), **kw}, back={})), (n, kw)


@pytest.mark.parametrize("args", [(32, 2**32 + 128, True), (2**32 + 32, 128, True), (32, -2**40, False), (-2**33 + 32, 128, False),
                                  (32, 10**15, True)])
def test_bucket_map_refuses_what_an_int_does_not_hold(L, args):
    with pytest.raises(vswin.VswinError) as e:
        vswin.bucket_map(*args, device="cpu")
    assert e.value.status == vswin.ERR_INVALID_ARG


@pytest.mark.parametrize("dim", [0, 1, 2])
def test_binding_refuses_extents_that_an_int_does_not_hold(dim):
    # (broadcast views: nothing of that size is in memory)
    wide = [1, 1, 1, 64]
    wide[dim] = 2**32 + 1
    one = torch.zeros(1, 1, 1, 64, dtype=torch.bfloat16)
    x, w, t, m = one.expand(wide), one[0, 0, 0], torch.zeros(2, 1, dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int32)
    for call in (lambda: vswin.qk_norm_forward(x, x, w, w), lambda: vswin.qk_norm_backward(x, x, w, w, x, x),
                 lambda: vswin.bias_attention_forward(x, x, x, t, m),
                 lambda: vswin.bias_attention_backward(x, x, x, t, m, x, None, x),
                 *((lambda: vswin.bias_attention_forward(one, x, x, t, m),) if dim == 1 else ())):
        with pytest.raises(vswin.VswinError) as e:
            call()
        assert e.value.status == vswin.ERR_UNSUPPORTED
