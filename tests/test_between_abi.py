"""Refusals of the norm, the activation and the routing, on the host: every bad argument is
found before anything is enqueued (fake addresses; no GPU is touched), and the plain forms that the GPU
tests use hold what they claim."""
import math

import pytest
import torch

import microscaling_weight_quantization_amd as mxq
from microscaling_weight_quantization_amd import build as B
from tests import between_ref as ref

OK, NULL, SHAPE, DTYPE, ALIAS = mxq.MXQ_OK, mxq.MXQ_ERR_NULL, mxq.MXQ_ERR_SHAPE, mxq.MXQ_ERR_DTYPE, mxq.MXQ_ERR_ALIAS
BIG = 1 << 62
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    if B.stale():
        B.build(["libmxq.so"])
    return mxq.load()


def call(fn, defaults, **kw):
    assert set(kw) <= set(defaults), set(kw) - set(defaults)
    return fn(*{**defaults, **kw}.values())


# 200 rows of 300: bf16 120000 bytes, fp32 240000, payload 60000, row codes 600, column codes 2 x 300
NORM = dict(x=0x100000, ld_x=300, res=0x200000, ld_res=300, res_dt=1, w=0x300000, w_dt=1, eps=1e-6, rows=200, K=300, dt=0,
            sum=0x400000, ld_sum=300, y=0x500000, ld_y=300)
ROW = dict(data=0x600000, ld_data=300, scale=0x700000, scale_ld=3)
COL = dict(cdata=0x800000, ld_col=300, cscale=0x900000, cscale_ld=300, ws=0xA00000, bytes=1600)


def norm_calls(lib):
    return [(lib.mxq_rms_norm, dict(NORM, stream=None)), (lib.mxq_rms_norm_fp8_group128, dict(NORM, **ROW, stream=None)),
            (lib.mxq_rms_norm_fp8_group128_row_col, dict(NORM, **ROW, **COL, stream=None))]


@pytest.mark.parametrize("which", [0, 1, 2])
def test_norm_refusals(lib, which):
    fn, d = norm_calls(lib)[which]
    for k in ("dt", "res_dt", "w_dt"):
        assert call(fn, d, **{k: mxq.MXQ_FP16}) == DTYPE and call(fn, d, **{k: 9}) == DTYPE, k
    for k in ("rows", "K"):
        assert call(fn, d, **{k: -1}) == SHAPE and call(fn, d, **{k: (1 << 30) + 1}) == SHAPE, k
    for eps in (0.0, -1e-6, NAN, INF):
        assert call(fn, d, eps=eps) == SHAPE, eps
    for k in [k for k in d if k.startswith("ld_") or k.endswith("_ld")]:
        assert call(fn, d, **{k: d[k] - 1}) == SHAPE and call(fn, d, **{k: BIG}) == SHAPE, k
    assert call(fn, d, x=None) == NULL
    assert call(fn, d, res=None) == NULL                                  # a sum of what?
    for k in ("data", "scale", "cdata", "cscale", "ws") if which else ("y",):
        if k in d:
            assert call(fn, d, **{k: None}) == NULL, k
    for k, v in (("x", 1), ("y", 1), ("res", 2), ("sum", 2), ("w", 2)):
        assert call(fn, d, **{k: d[k] + v}) == SHAPE, k
    outs = [k for k in ("sum", "y", "data", "scale", "cdata", "cscale", "ws") if k in d]
    for k in outs:
        for into, last in (("x", 119998), ("res", 239996), ("w", 1196)):
            step = 8 if k == "ws" else 4
            assert call(fn, d, **{k: (d[into] + last) // step * step}) == ALIAS, (k, into)
        for other in outs:
            if other != k:
                assert call(fn, d, **{k: d[other]}) == ALIAS, (k, other)
    # in place: the sum where the residual was, with its stride and no other
    assert call(fn, d, sum=d["res"], rows=0) == OK
    assert call(fn, d, sum=d["res"], ld_sum=301) == ALIAS
    assert call(fn, d, sum=d["res"] + 4) == ALIAS
    # nothing to do
    assert call(fn, d, rows=0, x=None) == OK and call(fn, d, K=0) == OK
    if which == 2:
        assert call(fn, d, bytes=1599) == SHAPE and call(fn, d, ws=0xA00004) == SHAPE
        assert lib.mxq_rms_norm_fp8_group128_row_col_workspace(200) == 1600
        assert lib.mxq_rms_norm_fp8_group128_row_col_workspace(-1) == 0


@pytest.mark.parametrize("which", [0, 1, 2, 3])
def test_norm_least_eps(lib, which):
    """Squares below 2^-149 vanish, which an eps of a normal number hides; a smaller one is refused."""
    d = dict(dy=0x100000, ld_dy=300, dt=0, x=0x200000, ld_x=300, x_dt=1, w=0x300000, w_dt=1, eps=1e-6, dres=None, ld_dres=300,
             rows=0, K=300, dx=0x500000, ld_dx=300, dw=None, ws=None, bytes=0, stream=None)
    fn, d = (norm_calls(lib) + [(lib.mxq_rms_norm_backward, d)])[which]
    assert call(fn, d, rows=0, eps=2.0 ** -126) == OK
    assert call(fn, d, rows=0, eps=2.0 ** -126 - 2.0 ** -149) == SHAPE and call(fn, d, rows=0, eps=1e-40) == SHAPE


def test_norm_backward_refusals(lib):
    fn = lib.mxq_rms_norm_backward
    need = lib.mxq_rms_norm_backward_workspace(200, 300)
    assert need > 0 and lib.mxq_rms_norm_backward_workspace(0, 300) == 0
    assert lib.mxq_rms_norm_backward_workspace(200, (1 << 30) + 1) == 0
    d = dict(dy=0x100000, ld_dy=300, dt=0, x=0x200000, ld_x=300, x_dt=1, w=0x300000, w_dt=1, eps=1e-6, dres=0x400000, ld_dres=300,
             rows=200, K=300, dx=0x500000, ld_dx=300, dw=0x600000, ws=0x700000, bytes=need, stream=None)
    for k in ("dt", "x_dt", "w_dt"):
        assert call(fn, d, **{k: mxq.MXQ_FP16}) == DTYPE, k
    for k in ("rows", "K"):
        assert call(fn, d, **{k: -1}) == SHAPE and call(fn, d, **{k: (1 << 30) + 1}) == SHAPE, k
    for eps in (0.0, NAN, INF):
        assert call(fn, d, eps=eps) == SHAPE
    for k in ("ld_dy", "ld_x", "ld_dres", "ld_dx"):
        assert call(fn, d, **{k: 299}) == SHAPE and call(fn, d, **{k: BIG}) == SHAPE, k
    for k in ("dy", "x", "dx", "ws"):
        assert call(fn, d, **{k: None}) == NULL, k
    assert call(fn, d, bytes=need - 1) == SHAPE and call(fn, d, ws=0x700008) == SHAPE
    for k, v in (("dy", 1), ("x", 2), ("dx", 2), ("dres", 2), ("dw", 2), ("w", 2)):
        assert call(fn, d, **{k: d[k] + v}) == SHAPE, k
    for k in ("dx", "dw", "ws"):
        for into, last in (("dy", 119998), ("x", 239996), ("w", 1196), ("dres", 239996)):
            assert call(fn, d, **{k: (d[into] + last) // 16 * 16}) == ALIAS, (k, into)
    assert call(fn, d, dw=0x500000) == ALIAS and call(fn, d, dw=0x700000) == ALIAS
    assert call(fn, d, K=0) == OK and call(fn, d, rows=0, dw=None) == OK


ACT = dict(gate=0x100000, ld_gate=600, up=0x100000 + 600, ld_up=600, rows=200, F=300, dt=0, act=0)


def act_calls(lib):
    both = dict(offsets=None, n=0, **ROW, cdata=0x800000, ld_col=300, cscale=0x900000, cscale_ld=300)
    wide = dict(both, ld_data=600, scale_ld=5, ld_col=600, cscale_ld=600)
    return [(lib.mxq_activate_fp8_group128, dict(ACT, **ROW, stream=None)),
            (lib.mxq_activate_fp8_group128_row_col, dict(ACT, **both, stream=None)),
            (lib.mxq_activate_fp8_group128_backward, dict(da=0xC00000, ld_da=300, **ACT, **wide, stream=None))]


@pytest.mark.parametrize("which", [0, 1, 2])
def test_activation_refusals(lib, which):
    fn, d = act_calls(lib)[which]
    assert call(fn, d, dt=mxq.MXQ_FP16) == DTYPE and call(fn, d, act=3) == DTYPE and call(fn, d, act=-1) == DTYPE
    assert call(fn, d, rows=-1) == SHAPE and call(fn, d, rows=(1 << 30) + 1) == SHAPE
    assert call(fn, d, F=-1) == SHAPE and call(fn, d, F=(1 << 29) + 1) == SHAPE
    for k in [k for k in d if k.startswith("ld_") or k.endswith("_ld")]:
        low = 299 if k in ("ld_gate", "ld_up") else d[k] - 1
        assert call(fn, d, **{k: low}) == SHAPE and call(fn, d, **{k: BIG}) == SHAPE, k
    outs = [k for k in ("data", "scale", "cdata", "cscale") if k in d]
    for k in ["gate", *outs] + (["da"] if which == 2 else []):
        assert call(fn, d, **{k: None}) == NULL, k
    for k in ("gate", "up", "da"):
        if k in d:
            assert call(fn, d, **{k: d[k] + 1}) == SHAPE, k
    for k in outs:
        assert call(fn, d, **{k: d["gate"] + 1}) == ALIAS, k
        assert call(fn, d, **{k: d["up"] + 199 * 1200 + 599}) == ALIAS, k
        for other in outs:
            if other != k:
                assert call(fn, d, **{k: d[other]}) == ALIAS, (k, other)
        if which == 2:
            assert call(fn, d, **{k: d["da"] + 119999}) == ALIAS, k
        if which:
            assert call(fn, d, offsets=d[k] // 4 * 4, n=4) == ALIAS, k
    if which:
        for n in (0, -1, 513):
            assert call(fn, d, offsets=0xE00000, n=n) == SHAPE
        assert call(fn, d, offsets=0xE00001, n=4) == SHAPE
    assert call(fn, d, rows=0) == OK and call(fn, d, F=0, gate=None) == OK


ROUTE = dict(logits=0x100000, ld=48, T=9, E=48, dt=1, bias=0x200000, mask=0x300000, score=0, renorm=1, scale=1.0, groups=4, top_groups=2,
             group_top=2, k=6, ids=0x400000, weights=0x500000, stream=None)


def test_route_refusals(lib):
    fn, d = lib.mxq_route_experts, ROUTE
    assert call(fn, d, dt=mxq.MXQ_FP16) == DTYPE and call(fn, d, score=2) == DTYPE
    for bad in (dict(T=-1), dict(E=0), dict(E=513, ld=513), dict(k=0), dict(k=25), dict(groups=0), dict(groups=5), dict(groups=49),
                dict(top_groups=0), dict(top_groups=5), dict(group_top=0), dict(group_top=3), dict(ld=47), dict(ld=BIG),
                dict(scale=NAN), dict(scale=INF), dict(T=1 << 28), dict(logits=0x100002), dict(bias=0x200002), dict(ids=0x400001),
                dict(weights=0x500002)):
        assert call(fn, d, **bad) == SHAPE, bad
    for k in ("logits", "ids", "weights"):
        assert call(fn, d, **{k: None}) == NULL, k
    for k in ("ids", "weights"):
        for into, last in (("logits", 9 * 192 - 4), ("bias", 188), ("mask", 8)):
            assert call(fn, d, **{k: d[into] + last}) == ALIAS, (k, into)
    assert call(fn, d, weights=0x400000 + 4 * 53) == ALIAS
    assert call(fn, d, T=0, logits=None) == OK


def test_route_backward_refusals(lib):
    fn = lib.mxq_route_experts_backward
    d = dict(dw=0x100000, logits=0x200000, ld=48, ids=0x300000, T=9, E=48, k=6, dt=1, score=0, renorm=1, scale=1.0, out=0x400000,
             ld_out=48, stream=None)
    assert call(fn, d, dt=mxq.MXQ_FP16) == DTYPE and call(fn, d, score=-1) == DTYPE
    for bad in (dict(T=-1), dict(E=0), dict(E=513, ld=513, ld_out=513), dict(k=0), dict(k=49), dict(ld=47), dict(ld_out=47),
                dict(ld_out=BIG), dict(scale=NAN), dict(dw=0x100001), dict(logits=0x200002), dict(ids=0x300002), dict(out=0x400001)):
        assert call(fn, d, **bad) == SHAPE, bad
    for k in ("dw", "logits", "ids", "out"):
        assert call(fn, d, **{k: None}) == NULL, k
    for k, last in (("dw", 212), ("logits", 1724), ("ids", 212)):
        assert call(fn, d, out=d[k] + last) == ALIAS, k
    assert call(fn, d, T=0, dw=None) == OK


def test_binding_refusals():
    """Shapes and names that do not belong together raise before the library is called."""
    f, b = torch.zeros(4, 256), torch.zeros(4, 256, dtype=torch.bfloat16)
    raw = lambda name: getattr(mxq, name).__wrapped__
    for kw in (dict(weight=torch.zeros(255)), dict(weight=torch.zeros(2, 256)[:, ::2]), dict(residual=torch.zeros(4, 255)),
               dict(residual=torch.zeros(5, 256)), dict(residual_out=torch.zeros(4, 256)),
               dict(residual=f, residual_out=b), dict(residual=f, residual_out=torch.zeros(5, 256)), dict(y=b), dict(y=torch.zeros(4, 200))):
        for name in ("mxq_rms_norm", "mxq_rms_norm_fp8_group128", "mxq_rms_norm_fp8_group128_row_col"):
            with pytest.raises(ValueError):
                raw(name)(f, **{"weight": None, **kw})
    with pytest.raises(TypeError):
        raw("mxq_rms_norm")(f.to(torch.float64), None)
    for kw in (dict(dy=torch.zeros(5, 256)), dict(dresidual=b), dict(dresidual=torch.zeros(4, 128)), dict(dx=b),
               dict(dweight=torch.zeros(255)), dict(dweight=torch.zeros(256, dtype=torch.bfloat16)), dict(weight=torch.zeros(3))):
        with pytest.raises(ValueError):
            raw("mxq_rms_norm_backward")(**{"dy": f, "x": f, "weight": None, **kw})
    for kw in (dict(up=b), dict(up=torch.zeros(4, 255)), dict(activation="tanh"), dict(data=torch.zeros(4, 256)),
               dict(data=torch.zeros(3, 256, dtype=torch.uint8))):
        with pytest.raises(ValueError):
            raw("mxq_activate_fp8_group128")(f, **kw)
    for kw in (dict(offsets=torch.zeros(4, dtype=torch.int64)), dict(col_data=torch.zeros(3, 256, dtype=torch.uint8)),
               dict(row_data=torch.zeros(4, 256, dtype=torch.uint8)[:, :200])):
        with pytest.raises(ValueError):
            raw("mxq_activate_fp8_group128_row_col")(f, **kw)
    for kw in (dict(da=b), dict(da=torch.zeros(3, 256)), dict(up=f, row_data=torch.zeros(4, 256, dtype=torch.uint8))):
        with pytest.raises(ValueError):
            raw("mxq_activate_fp8_group128_backward")(**{"da": f, "gate": f, **kw})
    for kw in (dict(bias=torch.zeros(255)), dict(bias=torch.zeros(256, dtype=torch.bfloat16)), dict(mask=torch.zeros(5, dtype=torch.bool)),
               dict(mask=torch.zeros(4)), dict(score="tanh"), dict(top_k=0), dict(ids=torch.zeros(4, 2, dtype=torch.int64)),
               dict(weights=torch.zeros(4, 3))):
        with pytest.raises(ValueError):
            raw("mxq_route_experts")(f, **{"top_k": 2, **kw})
    i = torch.zeros(4, 2, dtype=torch.int32)
    for kw in (dict(ids=i[:3]), dict(ids=i.long()), dict(dweights=torch.zeros(4, 3)), dict(dlogits=b), dict(score="none")):
        with pytest.raises(ValueError):
            raw("mxq_route_experts_backward")(**{"dweights": torch.zeros(4, 2), "logits": f, "ids": i, **kw})
    with pytest.raises(ValueError):
        raw("mxq_route_experts")(f[0], 2)


def test_calls_run_on_the_operands_device(monkeypatch):
    """A call whose tensors lie on another device than the current one makes that one current while it runs."""
    seen = []

    class Fake(torch.Tensor):
        is_cuda = True

        def get_device(self):
            return 3

    class Current:
        def __init__(self, d):
            self.d = d

        def __enter__(self):
            seen.append(("enter", self.d))

        def __exit__(self, *a):
            seen.append(("exit", self.d))

    monkeypatch.setattr(mxq, "_current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "device", Current)
    t = torch.zeros(2).as_subclass(Fake)
    mxq._device_operands(lambda x: seen.append("ran"))(t)
    assert seen == [("enter", 3), "ran", ("exit", 3)]
    seen.clear()
    monkeypatch.setattr(mxq, "_current_device", lambda: 3)
    mxq._device_operands(lambda x: seen.append("ran"))(t)
    assert seen == ["ran"]


# ---- the plain forms ---------------------------------------------------------------------

def gen(seed):
    return torch.Generator().manual_seed(seed)


def test_plain_norm_gradient_against_differences():
    g = gen(1)
    s, w, dy = (torch.randn(*shape, generator=g, dtype=torch.float64) for shape in ((3, 7), (7,), (3, 7)))
    (dx, _), (dw, _) = ref.norm_backward(dy, s, w, 1e-3, None)
    f = lambda s, w: float((ref.norm(s, w, 1e-3)[0] * dy).sum())
    h = 1e-5
    for at in [(r, c) for r in range(3) for c in range(7)]:
        e = torch.zeros_like(s)
        e[at] = h
        assert abs((f(s + e, w) - f(s - e, w)) / (2 * h) - float(dx[at])) < 1e-7
    for c in range(7):
        e = torch.zeros_like(w)
        e[c] = h
        assert abs((f(s, w + e) - f(s, w - e)) / (2 * h) - float(dw[c])) < 1e-7


@pytest.mark.parametrize("name", ["silu", "gelu_tanh", "relu2"])
def test_plain_activation_slope_against_differences(name):
    g = torch.linspace(-6, 6, 241, dtype=torch.float64) + 1e-3
    a, d, size, _ = ref.act(name, g)
    h = 1e-5
    assert torch.allclose((ref.act(name, g + h)[0] - ref.act(name, g - h)[0]) / (2 * h), d, atol=1e-8, rtol=0)
    assert bool((size >= d.abs() * (1 - 1e-12)).all())
    want = {"silu": torch.nn.functional.silu(g), "gelu_tanh": torch.nn.functional.gelu(g, approximate="tanh"),
            "relu2": torch.relu(g) ** 2}[name]
    assert torch.allclose(a, want, atol=1e-14, rtol=1e-12)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
def test_plain_route_gradient_against_differences(score, renormalize):
    g = gen(3)
    logits = torch.randn(2, 6, generator=g, dtype=torch.float64)
    how = dict(score=score, renormalize=renormalize, scale=2.5)
    ids, _ = ref.route(logits, 3, **how)
    dw = torch.randn(2, 3, generator=g, dtype=torch.float64)
    got, size = ref.route_backward(dw, logits, ids, **how)
    assert bool((size >= got.abs() * (1 - 1e-12)).all())

    def f(l):
        p = torch.tensor(ref.scores(l, score), dtype=torch.float64).gather(1, ids.long())
        return float((2.5 * (p / p.sum(1, keepdim=True) if renormalize else p) * dw).sum())

    h = 1e-5
    for at in [(t, e) for t in range(2) for e in range(6)]:
        d = torch.zeros_like(logits)
        d[at] = h
        assert abs((f(logits + d) - f(logits - d)) / (2 * h) - float(got[at])) < 1e-8


def test_plain_route_by_hand():
    l = torch.tensor([[1.0, 3.0, 3.0, -INF], [-INF] * 4, [0.0, 0.0, 0.0, 0.0]])
    ids, w = ref.route(l, 3)
    assert ids.tolist() == [[1, 2, 0], [-1, -1, -1], [0, 1, 2]]
    z = 2 + math.exp(-2)
    assert torch.allclose(w[0], torch.tensor([1 / z, 1 / z, math.exp(-2) / z], dtype=torch.float64)) and w[1].sum() == 0
    # groups {0, 1}, {2, 3}: by the largest key the first; by the two best the second
    l = torch.tensor([[5.0, -9.0, 4.0, 4.5]])
    assert ref.route(l, 1, score="sigmoid", n_groups=2)[0].tolist() == [[0]]
    assert ref.route(l, 2, score="sigmoid", n_groups=2, group_top=2)[0].tolist() == [[3, 2]]
    assert ref.route(l, 1, bias=torch.tensor([-INF, 0, 0, 0.0]), score="sigmoid")[0].tolist() == [[3]]
    assert ref.route(l, 2, mask=torch.tensor([False]))[0].tolist() == [[-1, -1]]


def test_plain_checks_find_mistakes():
    """A code that is one off, a payload a step off, a row of no expert that is not zero."""
    from tests import fp8_ref
    x = torch.randn(140, 130, generator=gen(5), dtype=torch.float64)
    off = x.abs() * 2.0 ** -22
    q, c = fp8_ref.quantize_rows(x)
    ref.check_rows(q, c, x, off)
    for broken in ((q, c + 1), (q + 1, c), (q.roll(1, 0), c)):
        with pytest.raises(AssertionError):
            ref.check_rows(*broken, x, off)
    offsets = torch.tensor([0, 5, 135])
    q, c = fp8_ref.quantize_cols(x, offsets.tolist())
    ref.check_cols(q, c, x, off, offsets)
    q[139, 3] = 1
    with pytest.raises(AssertionError):
        ref.check_cols(q, c, x, off, offsets)
