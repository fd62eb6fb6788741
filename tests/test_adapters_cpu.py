"""Tokens sorted by adapter without a GPU: the eager tier against the oracle,
gradients, the layer of several adapters, and the entry points' refusals."""
import numpy as np
import pytest
import torch

from dora_fine_tuning_amd import binding
from oracle import q4_oracle as Q

F = pytest.importorskip("dora_fine_tuning_amd.torch_ops")
LIB = binding.LIB
OK, INVALID, UNSUPPORTED = binding.DORA_OK, binding.DORA_INVALID_ARG, binding.DORA_UNSUPPORTED
FAR = [(1 << 40) * (i + 1) for i in range(8)]


def make_ids(kind, T, k, n, seed=0):
    rng = np.random.default_rng(seed)
    if kind == "some":  # any, none among them
        ids = rng.integers(-1, n, (T, k))
    elif kind == "skewed":
        ids = (n * rng.random((T, k)) ** 3).astype(np.int64)
    elif kind == "none":
        ids = np.full((T, k), -1)
    elif kind == "one":
        ids = np.full((T, k), n - 1)
    else:  # "wild": far outside, also where 32 bits of the number would be inside
        ids = np.where(rng.random((T, k)) < 0.5, rng.integers(0, n, (T, k)),
                       rng.choice([-(2**63), 2**63 - 1, 2**32, -(2**31) - 1, n, -2], (T, k)))
    return torch.from_numpy(ids.astype(np.int64))


def check_sort(device, ids, n, as_type=torch.int64):
    order, place, bounds = F.adapter_sort(ids.to(as_type).to(device), n)
    ro, rp, rb = Q.sort(ids.to(as_type).numpy(), n)
    for got, want in ((order, ro), (place, rp), (bounds, rb)):
        assert got.dtype == torch.int32 and np.array_equal(got.cpu().numpy(), want)
    return place


@pytest.mark.parametrize("kind", ["some", "skewed", "none", "one", "wild"])
@pytest.mark.parametrize("T,k,n", [(1, 1, 1), (7, 1, 3), (50, 3, 4), (0, 2, 5), (5, 0, 5)])
def test_eager_sort(kind, T, k, n):
    check_sort("cpu", make_ids(kind, T, k, n), n)


def test_eager_sort_types_and_no_adapters():
    ids = make_ids("some", 20, 2, 9)
    check_sort("cpu", ids, 9, torch.int32)
    check_sort("cpu", ids, 9, torch.int16)
    check_sort("cpu", ids, 0)
    check_sort_refusals("cpu")


def check_sort_refusals(device):
    ids = make_ids("some", 20, 2, 9).to(device)
    for bad in ((ids, -1), (ids[0], 3), (ids.float(), 3), (ids[None], 3)):
        with pytest.raises(ValueError, match="whole numbers"):
            F.adapter_sort(*bad)


def data(T, k, D, dtype, device, seed=0, weights=True, base=True):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g)
    out = dict(x=r(T, D).to(dtype), rows=r(T * k, D).to(dtype), w=r(T, k) if weights else None,
               base=r(T, D).to(dtype) if base else None, dy=r(T, D).to(dtype), dr=r(T * k, D).to(dtype))
    return {n: v if v is None else v.to(device) for n, v in out.items()}


def as64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def close(got, want, mass, dtype, terms):
    """A sum of ``terms`` fp32 products, rounded once: half a step of the result, and an
    fp32 step of the sum of magnitudes for each product and each addition."""
    half, sub = torch.finfo(dtype).eps / 2, {torch.bfloat16: 2.0**-134, torch.float16: 2.0**-25}.get(dtype, 2.0**-149)
    tol = half * (1 + 2.0**-10) * np.abs(want) + 2 * terms * 2.0**-24 * mass + sub
    assert np.all(np.abs(as64(got) - want) <= tol), float(np.max(np.abs(as64(got) - want) - tol))


def check_rows(device, ids, n, D, dtype, weights=True, base=True, seed=0):
    """Both operators and every gradient against the oracle; the gradients of autograd are the operators' own."""
    T, k = ids.shape
    place = F.adapter_sort(ids.to(device), n)[1]
    p = place.cpu().numpy()
    d = data(T, k, D, dtype, device, seed, weights, base)
    leaves = [v.requires_grad_() for v in (d["x"], d["rows"], d["w"], d["base"]) if v is not None]
    xs = F.adapter_gather(d["x"], place)
    y = F.adapter_combine(d["rows"], d["w"], place, d["base"])
    assert xs.dtype == dtype and y.dtype == dtype and xs.is_contiguous() and y.is_contiguous()
    assert np.array_equal(as64(xs), Q.gather(as64(d["x"]), p))
    A = lambda t: None if t is None else np.abs(as64(t))
    close(y, Q.combine(as64(d["rows"]), as64(d["w"]), p, as64(d["base"])),
          Q.combine(A(d["rows"]), A(d["w"]), p, A(d["base"])), dtype, k + 1)
    (dx,) = torch.autograd.grad(xs, leaves[0], d["dr"])
    close(dx, Q.combine(as64(d["dr"]), None, p, None), Q.combine(A(d["dr"]), None, p, None), dtype, k)
    grads = torch.autograd.grad(y, leaves[1:], d["dy"])
    rr, rw = Q.combine_bwd(as64(d["dy"]), as64(d["rows"]), as64(d["w"]), p)
    mr, mw = Q.combine_bwd(A(d["dy"]), A(d["rows"]), A(d["w"]), p)
    close(grads[0], rr, mr, dtype, 1)
    if weights:
        assert grads[1].dtype == torch.float32
        close(grads[1], rw, mw, torch.float32, D)
    if base:
        assert torch.equal(grads[-1], d["dy"])


SHAPES = [(1, 1, 1, 1), (7, 1, 3, 8), (50, 3, 4, 17), (9, 2, 2, 64), (5, 0, 3, 8), (0, 2, 3, 8), (4, 2, 3, 0)]


@pytest.mark.parametrize("T,k,n,D", SHAPES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kind", ["some", "none"])
def test_eager_rows(T, k, n, D, dtype, kind):
    for weights in (True, False):
        for base in (True, False):
            check_rows("cpu", make_ids(kind, T, k, n), n, D, dtype, weights, base)


def check_unused_values(device, dtype):
    """NaN and infinities in rows and weights of slots without an adapter reach nothing."""
    ids = torch.tensor([[0, -1], [-1, -1], [1, 0]], device=device)
    place = F.adapter_sort(ids, 2)[1]
    rows = torch.ones((6, 16), device=device, dtype=dtype)
    rows[3:] = float("nan")
    w = torch.where(ids >= 0, 2.0, float("nan")).requires_grad_()
    rows.requires_grad_()
    y = F.adapter_combine(rows, w, place, None)
    d_rows, d_w = torch.autograd.grad(y, (rows, w), torch.ones_like(y))
    assert y[:, 0].tolist() == [2.0, 0.0, 4.0]
    assert d_rows[:, 0].tolist() == [2.0, 2.0, 2.0, 0.0, 0.0, 0.0]
    assert d_w.tolist() == [[16.0, 0.0], [0.0, 0.0], [16.0, 16.0]]
    x = torch.full((3, 16), float("nan"), device=device, dtype=dtype)
    x[::2] = 1.0
    assert F.adapter_gather(x, place)[:, 0].tolist() == [1.0] * 3 + [0.0] * 3


def test_unused_values_eager():
    check_unused_values("cpu", torch.float32)


def check_foreign_places(device, dtype):
    """Numbers that no sort gives: left out, never followed."""
    place = torch.tensor([[0, 6], [-7, 2**31 - 1], [-(2**31), 1]], dtype=torch.int32, device=device)
    rows = torch.ones((6, 16), device=device, dtype=dtype)
    y = F.adapter_combine(rows, None, place, None)
    assert y[:, 0].tolist() == [1.0, 0.0, 1.0]
    dy = torch.ones((3, 16), device=device, dtype=dtype)
    d_rows, d_w = F.adapter_combine_backward(dy, rows, None, place, True, True)
    assert d_w.tolist() == [[16.0, 0.0], [0.0, 0.0], [0.0, 16.0]] and d_rows[:2].float().min() == 1
    assert F.adapter_gather(torch.ones((3, 16), device=device, dtype=dtype), place)[:2].float().min() == 1


def test_foreign_places_eager():
    check_foreign_places("cpu", torch.float32)


def check_by_differences(device):
    """The layer's loss is smooth in every leaf: gradients against central differences in 64-bit sums of fp32 runs."""
    torch.manual_seed(1)
    layer = F.DoRAAdapters(24, 16, 4, 3, dtype=torch.float32, device=device, detach_norm=False)
    with torch.no_grad():
        layer.lora_B.normal_(0.0, 0.3)
    x, ids = torch.randn(11, 24, device=device), make_ids("some", 11, 2, 3).to(device)
    w, dy = torch.rand(11, 2, device=device), torch.randn(11, 16, device=device)
    leaves = (x.requires_grad_(), w.requires_grad_(), layer.lora_A, layer.lora_B, layer.magnitude)
    loss = lambda: (layer(x, ids, w).double() * dy.double()).sum()
    grads = torch.autograd.grad(loss(), leaves)
    for leaf, g in zip(leaves, grads):
        dirn = torch.randn_like(leaf)

        def slope(h):  # the derivative, plus h^2 / 6 of the third one, ..
            with torch.no_grad():
                leaf.add_(h * dirn)
                up = loss()
                leaf.sub_(2 * h * dirn)
                down = loss()
                leaf.add_(h * dirn)
            return float(up - down) / (2 * h)

        h = 2.0**-7
        got, want = float((g.double() * dirn.double()).sum()), (4 * slope(h / 2) - slope(h)) / 3
        # the third derivative is gone; h^4 of the fifth along a direction of up to 17 times
        # unit length is (17 h)^4 = 2^-11.6, and the fp32 rounding of losses of order 100
        # 2^-17 each, over h = 2^-7, is 2^-10
        assert abs(got - want) <= 2.0**-9 * max(1.0, abs(want)) + 2.0**-7, (got, want)


def test_layer_by_differences():
    check_by_differences("cpu")


def check_layer(device, dtype, q4, detach, k, tol):
    """The layer against the definition in 64 bits: one dense DoRA weight an adapter."""
    torch.manual_seed(2)
    layer = F.DoRAAdapters(72, 40, 8, 4, dtype=dtype, device=device, q4_weight=q4, detach_norm=detach)
    with torch.no_grad():
        layer.lora_B.normal_(0.0, 0.05)
        layer.magnitude.mul_(1.0 + 0.1 * torch.randn_like(layer.magnitude))
    ids = make_ids("some", 30, k, 4, seed=k)
    ids[ids == 2] = 0  # an adapter that no token uses
    x = torch.randn(30, 72, device=device).to(dtype).requires_grad_()
    w = torch.rand(30, k, device=device).requires_grad_()
    dy = torch.randn(30, 40, device=device).to(dtype)
    leaves = (x, w, layer.lora_A, layer.lora_B, layer.magnitude)
    y = layer(x, ids.to(device), w)
    got = torch.autograd.grad(y, leaves, dy)
    W = F.q4_unpack_weight(*layer._packed_weight(), 40, 72, torch.float32) if q4 else layer.weight
    W = W.double()
    L = [t.detach().double().requires_grad_() for t in leaves]
    X, wt, A, B, m = L
    base = X @ W.t()
    ref = base
    for a in range(4):
        n = torch.linalg.vector_norm(W + layer.s * B[a] @ A[a], dim=1)
        g = m[a] / (n.detach() if detach else n)
        delta = (g - 1) * base + g * layer.s * ((X @ A[a].t()) @ B[a].t())
        ref = ref + ((ids.to(device) == a) * wt).sum(dim=1, keepdim=True) * delta
    want = torch.autograd.grad(ref, L, dy.double())
    for name, g, v in zip(("y", "x", "w", "A", "B", "m"), (y, *got), (ref, *want)):
        g, v = g.detach().double(), v.detach()
        assert float((g - v).norm()) <= tol * float(v.norm()), (name, float((g - v).norm() / v.norm()))
    assert not bool(got[2][2].any()) and not bool(got[4][2].any())  # the unused one
    lead = layer(x.detach().reshape(5, 6, 72), ids.to(device).reshape(5, 6, k), w.detach().reshape(5, 6, k))
    assert torch.equal(lead.reshape(30, 40), y.detach())


@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("detach", [False, True])
@pytest.mark.parametrize("k", [1, 2])
def test_layer_eager(q4, detach, k):
    check_layer("cpu", torch.float32, q4, detach, k, 2.0**-16)


def check_layer_edges(device, dtype):
    torch.manual_seed(3)
    layer = F.DoRAAdapters(72, 40, 8, 3, dtype=dtype, device=device)
    with torch.no_grad():
        layer.lora_B.normal_(0.0, 0.05)
    x = torch.randn(6, 72, device=device).to(dtype)
    base = torch.nn.functional.linear(x, layer.weight)
    assert torch.equal(layer(x, torch.full((6,), -1, device=device)), base)  # no adapter at all
    assert layer(x[:0], torch.zeros(0, dtype=torch.int64, device=device)).shape == (0, 40)
    one = layer(x, torch.ones(6, dtype=torch.int64, device=device))
    single = F.DoRALinear(72, 40, 8, weight=layer.weight, dtype=dtype, device=device)
    with torch.no_grad():
        for name in ("lora_A", "lora_B", "magnitude"):
            getattr(single, name).copy_(getattr(layer, name)[1])
    # the adapter's part is rounded once more on its way back
    want, eps = single(x).float(), torch.finfo(dtype).eps
    assert bool(((one.float() - want).abs() <= eps * (want.abs() + (want - base.float()).abs()) + 1e-6).all())
    with pytest.raises(ValueError, match="ids"):
        layer(x, torch.zeros(5, dtype=torch.int64, device=device))
    with pytest.raises(ValueError, match="weights"):
        layer(x, torch.zeros(6, dtype=torch.int64, device=device), torch.ones(6, 2, device=device))
    with pytest.raises(ValueError, match="adapters"):
        F.DoRAAdapters(8, 8, 2, 0)


def test_layer_edges_eager():
    check_layer_edges("cpu", torch.float32)


def check_traced_outputs(device, dtype):
    from torch._subclasses.fake_tensor import FakeTensorMode

    ids = make_ids("some", 9, 2, 4).to(device)
    place = F.adapter_sort(ids, 4)[1]
    d = data(9, 2, 24, dtype, device)
    calls = [(F.adapter_sort, (ids, 4)), (F.adapter_gather, (d["x"], place)),
             (F.adapter_combine, (d["rows"], d["w"], place, d["base"])),
             (F.adapter_combine, (d["rows"], None, place, None)),
             (F.adapter_combine_backward, (d["dy"], d["rows"], d["w"], place, True, True)),
             (F.adapter_combine_backward, (d["dy"], d["rows"], d["w"], place, False, True)),
             (F.adapter_combine_backward, (d["dy"], d["rows"], None, place, True, False))]
    turned = lambda a: a.t().contiguous().t() if isinstance(a, torch.Tensor) and a.dim() == 2 else a
    for op, args in calls:
        for call in (args, tuple(turned(a) for a in args)):
            real = op(*call)
            with FakeTensorMode() as mode:
                fake = op(*[mode.from_tensor(a) if isinstance(a, torch.Tensor) else a for a in call])
            for r, f in zip(*(o if isinstance(o, tuple) else (o,) for o in (real, fake))):
                assert (r.shape, r.dtype, r.stride()) == (f.shape, f.dtype, f.stride()), op
    f = lambda x, w: (F.adapter_combine(F.adapter_gather(x, place), w, place, x).t() * d["dy"].t()).sum()
    leaves = d["x"].requires_grad_(), d["w"].requires_grad_()
    want = torch.autograd.grad(f(*leaves), leaves)
    torch._dynamo.reset()
    got = torch.autograd.grad(torch.compile(f, backend="aot_eager", fullgraph=True)(*leaves), leaves)
    assert all(torch.equal(a, c) for a, c in zip(want, got))


def test_traced_outputs_eager():
    check_traced_outputs("cpu", torch.float32)


def check_wrong_arguments(device, dtype):
    place = F.adapter_sort(torch.zeros((4, 2), dtype=torch.int64, device=device), 1)[1]
    m = lambda *s, t=dtype: torch.zeros(s, device=device, dtype=t)
    bad = [lambda: F.adapter_gather(m(5, 8), place), lambda: F.adapter_gather(m(4, 8), place.long()),
           lambda: F.adapter_gather(m(4, 8), place.reshape(-1)),
           lambda: F.adapter_combine(m(7, 8), None, place, None),
           lambda: F.adapter_combine(m(8, 8), m(4, 1), place, None),
           lambda: F.adapter_combine(m(8, 8), None, place, m(4, 9)),
           lambda: F.adapter_combine(m(8, 8), None, place, m(4, 8, t=torch.float64)),
           lambda: F.adapter_combine(m(8, 8), None, place.reshape(-1), None),
           lambda: F.adapter_combine_backward(m(3, 8), m(8, 8), None, place, True, True),
           lambda: F.adapter_combine_backward(m(4, 8), m(7, 8), None, place, True, True)]
    for i, f in enumerate(bad):
        with pytest.raises((ValueError, binding.DoraError)):
            f()
            pytest.fail(str(i))
    with pytest.raises(RuntimeError, match="no gradient"):
        F.adapter_combine_backward(m(4, 8).requires_grad_(), m(8, 8), None, place, True, True)


def test_wrong_arguments_eager():
    check_wrong_arguments("cpu", torch.float32)


# ------------------------------------------------------------------ refusals of the entry points


def _status(status, want, text):
    assert status == want and text in binding.dora_last_error(), (status, binding.dora_last_error())


def test_sort_refusals():
    def call(ids=FAR[0], b=8, T=5000, k=2, n=16, order=FAR[1], place=FAR[2], bounds=FAR[3], ws=FAR[4], wsb=1 << 39):
        return LIB.dora_adapter_sort(ids, b, T, k, n, order, place, bounds, ws, wsb, None)

    _status(call(b=2), UNSUPPORTED, "bytes")
    _status(call(T=-1), INVALID, "negative")
    _status(call(k=-1), INVALID, "negative")
    _status(call(n=-1), INVALID, "adapters")
    _status(call(n=1001), UNSUPPORTED, "adapters")
    _status(call(T=1 << 31), UNSUPPORTED, "2^31")
    _status(call(T=1 << 62, k=8), UNSUPPORTED, "2^31")
    for name in ("ids", "order", "place", "bounds", "ws"):
        _status(call(**{name: None}), INVALID, "NULL")
    _status(call(ids=FAR[0] + 4), INVALID, "alignment")
    _status(call(place=FAR[2] + 2), INVALID, "alignment")
    need = LIB.dora_adapter_sort_workspace_bytes(5000, 2, 16)
    assert need > 0 and LIB.dora_adapter_sort_workspace_bytes(2048, 2, 16) == 0
    _status(call(wsb=need - 1), INVALID, "workspace of")
    _status(call(order=FAR[0]), INVALID, "overlaps")
    _status(call(order=FAR[2] + 4), INVALID, "overlaps")
    _status(call(bounds=FAR[4]), INVALID, "overlaps")
    assert LIB.dora_adapter_sort_workspace_bytes(-1, 2, 4) == 0


def test_rows_refusals():
    def gather(x=FAR[0], place=FAR[1], T=10, k=2, D=64, dt=0, rows=FAR[2]):
        return LIB.dora_adapter_gather(x, place, T, k, D, dt, rows, None)

    def combine(rows=FAR[0], w=FAR[1], place=FAR[2], base=FAR[3], T=10, k=2, D=64, dt=0, y=FAR[4]):
        return LIB.dora_adapter_combine(rows, w, place, base, T, k, D, dt, y, None)

    def bwd(dy=FAR[0], rows=FAR[1], w=FAR[2], place=FAR[3], T=10, k=2, D=64, dt=0, dr=FAR[4], dw=FAR[5]):
        return LIB.dora_adapter_combine_bwd(dy, rows, w, place, T, k, D, dt, dr, dw, None)

    for fn in (gather, combine, bwd):
        _status(fn(dt=2), UNSUPPORTED, "dtype")
        _status(fn(T=-1), INVALID, "negative")
        _status(fn(D=-8), INVALID, "negative")
        _status(fn(D=(1 << 22) + 1), UNSUPPORTED, "2^22")
        _status(fn(T=1 << 30, k=2), UNSUPPORTED, "2^31")
        _status(fn(place=None), INVALID, "NULL")
        _status(fn(rows=None), INVALID, "NULL")
        assert fn(T=0, rows=None, place=None) == OK
    _status(gather(x=None), INVALID, "NULL")
    _status(gather(rows=FAR[0] + 2), INVALID, "overlaps")
    _status(combine(y=None), INVALID, "NULL")
    _status(combine(y=FAR[3] + 2), INVALID, "overlaps")
    _status(combine(y=FAR[0]), INVALID, "overlaps")
    _status(combine(w=FAR[1] + 2), INVALID, "alignment")
    _status(bwd(dy=None), INVALID, "NULL")
    _status(bwd(dr=FAR[1]), INVALID, "overlaps")
    _status(bwd(dw=FAR[4]), INVALID, "overlaps")
    assert bwd(dr=None, dw=None, dy=None) == OK
    assert gather(D=0, x=None) == OK and gather(k=0, x=None) == OK


def test_rows_refuse_more_threads_than_a_launch_holds():
    """2^31 - 8 tokens of 128 elements take four threads each; of 32, one, and they go on to the next check."""
    T = (1 << 31) - 8
    _status(LIB.dora_adapter_gather(FAR[0], FAR[1], T, 1, 128, 0, FAR[2], None), UNSUPPORTED, "threads")
    _status(LIB.dora_adapter_combine(FAR[0], None, FAR[2], None, T, 1, 128, 0, FAR[4], None), UNSUPPORTED, "threads")
    _status(LIB.dora_adapter_combine_bwd(FAR[0], FAR[1], None, FAR[3], T, 1, 128, 0, FAR[4], None, None), UNSUPPORTED,
            "threads")
    _status(LIB.dora_adapter_gather(FAR[0], FAR[1], T, 1, 32, 0, None, None), INVALID, "NULL")


def test_layer_gradients_of_adapters_that_no_token_uses():
    """Zeros, and those of the others as if they were alone."""
    torch.manual_seed(3)
    layer = F.DoRAAdapters(24, 40, 4, 5, dtype=torch.float32)
    with torch.no_grad():
        layer.lora_B.normal_()
    x, ids = torch.randn(6, 24), torch.tensor([1, 3, 3, -1, 1, 7])
    layer(x, ids).square().sum().backward()
    for p in (layer.lora_A, layer.lora_B, layer.magnitude):
        assert [bool(g.any()) for g in p.grad] == [False, True, False, True, False]


def test_binding_refuses_host_tensors():
    ids = torch.zeros((4, 2), dtype=torch.int64)
    place = F.adapter_sort(ids, 1)[1]
    for f in (lambda: binding.dora_adapter_sort(ids, 1),
              lambda: binding.dora_adapter_gather(torch.zeros(4, 8).half(), place),
              lambda: binding.dora_adapter_combine(torch.zeros(8, 8).half(), None, place)):
        with pytest.raises(ValueError, match="HIP device"):
            f()
