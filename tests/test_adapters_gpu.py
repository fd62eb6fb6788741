"""Tokens sorted by adapter on the GPU against the oracle (tolerances in test_adapters_cpu)."""
import numpy as np
import pytest
import torch

from oracle import q4_oracle as Q
from test_adapters_cpu import (SHAPES, check_by_differences, check_foreign_places, check_layer, check_layer_edges,
                               check_rows, check_sort, check_sort_refusals, check_traced_outputs, check_unused_values,
                               check_wrong_arguments, make_ids)

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.fixture(scope="module")
def F():
    from dora_fine_tuning_amd import torch_ops

    return torch_ops


@pytest.mark.parametrize("kind", ["some", "skewed", "none", "one", "wild"])
@pytest.mark.parametrize("T,k,n", [(1, 1, 1), (7, 1, 3), (63, 1, 2), (64, 1, 64), (65, 3, 5), (1024, 1, 8),
                                   (1025, 1, 9), (1000, 4, 1000), (4096, 1, 7), (4097, 1, 7), (2049, 2, 255),
                                   (5000, 3, 256), (0, 2, 5), (5, 0, 5)])
def test_sort(kind, T, k, n):
    for dt in (torch.int64, torch.int32):
        check_sort(DEV, make_ids(kind, T, k, n), n, dt)


def test_sort_of_many(F):
    """More slots than 256 workgroups take in four rounds, against torch's stable sort."""
    for N, n in ((1_500_000, 37), (3_000_001, 1000), (300_000, 1)):
        ids = torch.randint(-1, n, (N, 1), device=DEV)
        order, place, bounds = F.adapter_sort(ids, n)
        key = torch.where(ids < 0, n, ids).flatten()
        slots = torch.sort(key, stable=True).indices
        has = key[slots] < n
        assert torch.equal(order.long(), torch.where(has, slots, -1 - slots))
        row = torch.empty_like(slots)
        row[slots] = torch.arange(N, device=DEV)
        assert torch.equal(place.flatten().long(), torch.where(key < n, row, -1 - row))
        assert torch.equal(bounds.long(), torch.searchsorted(key[slots], torch.arange(n + 1, device=DEV)))


def test_more_adapters_than_the_kernel_takes(F):
    check_sort(DEV, make_ids("some", 300, 2, 1500), 1500)
    check_sort(DEV, make_ids("some", 30, 2, 9), 0)
    check_sort(DEV, make_ids("some", 30, 2, 9), 9, torch.int16)
    check_sort_refusals(DEV)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("kind", ["some", "none"])
@pytest.mark.parametrize("T,k,n,D", SHAPES + [(33, 2, 4, 40), (20, 4, 3, 1000), (5, 2, 2, 2056), (6, 1, 2, 8192),
                                              (3, 3, 2, 10001),
                                              (130, 2, 16, 129), (2, 9, 5, 27648)])
def test_rows(T, k, n, D, dtype, kind):
    for weights, base in ((True, True), (False, False), (True, False), (False, True)):
        check_rows(DEV, make_ids(kind, T, k, n), n, D, dtype, weights, base)


def test_rows_at_any_alignment(F):
    """Slices that start off a 16-byte boundary, transposed and expanded operands."""
    ids = make_ids("some", 12, 2, 3).to(DEV)
    place = F.adapter_sort(ids, 3)[1]
    p = place.cpu().numpy()
    wide = torch.randn((40, 65), device=DEV).bfloat16()
    for x in (wide[:12, 1:], wide[:12, :64], wide.reshape(-1)[1 : 1 + 12 * 64].view(12, 64), wide.t()[:12, :40],
              wide[:1].expand(12, 65)):
        assert np.array_equal(F.adapter_gather(x, place).double().cpu().numpy(), Q.gather(x.double().cpu().numpy(), p))
        y = F.adapter_combine(F.adapter_gather(x, place), None, place, x)
        count = (ids >= 0).sum(dim=1, keepdim=True)
        assert torch.equal(y, (x.float() * (1 + count)).to(x.dtype))
        ones = torch.ones(2, 12, device=DEV).t()
        assert torch.equal(F.adapter_combine(F.adapter_gather(x, place), ones, place, x), y)


def test_unused_values():
    check_unused_values(DEV, torch.bfloat16)


def test_foreign_places():
    check_foreign_places(DEV, torch.bfloat16)


def test_rows_past_2_32_bytes(F):
    T, k, D = 150_000, 2, 8192
    ids = torch.randint(-1, 4, (T, k), device=DEV)
    place = F.adapter_sort(ids, 4)[1]
    x = torch.randn((T, D), device=DEV, dtype=torch.bfloat16)  # 2.5 GB, its rows 4.9
    rows = F.adapter_gather(x, place)
    y = F.adapter_combine(rows, None, place, x)
    count = (ids >= 0).sum(dim=1, keepdim=True)
    for i in range(0, T, 30_000):
        s = slice(i, i + 30_000)
        assert torch.equal(y[s], (x[s].float() * (1 + count[s])).to(x.dtype))
    w = torch.rand((T, k), device=DEV)
    d_rows, d_w = F.adapter_combine_backward(x, rows, w, place, True, True)
    for t in (0, 77_777, T - 1):
        for j in range(k):
            q = int(place[t, j])
            want = (w[t, j] * x[t].float()).to(x.dtype) if q >= 0 else torch.zeros_like(x[t])
            assert torch.equal(d_rows[q if q >= 0 else ~q], want)
            dot = float((x[t].double() ** 2).sum()) if q >= 0 else 0.0
            assert abs(float(d_w[t, j]) - dot) <= 2 * D * 2.0**-24 * dot


def test_combine_in_place_of_its_base(F):
    from dora_fine_tuning_amd.binding import LIB, _ptr, _raw_stream

    ids = make_ids("some", 50, 2, 3).to(DEV)
    place = F.adapter_sort(ids, 3)[1]
    for D in (40, 33):
        rows, base = torch.randn((100, D), device=DEV).half(), torch.randn((50, D), device=DEV).half()
        want = F.adapter_combine(rows, None, place, base)
        st = LIB.dora_adapter_combine(_ptr(rows), None, _ptr(place), _ptr(base), 50, 2, D, 1, _ptr(base),
                                      _raw_stream(DEV))
        assert st == 0
        assert torch.equal(base, want)


def test_captured_and_replayed(F):
    """Sort, exchange and gradients in one graph; other ids and values at each replay, eager calls between.
    (No eager graph of the leaves is alive at the capture: torch runs a leaf's end of the backward on the
    stream of the graph that made it, which a capture does not survive.)"""
    for T, k, n, D in ((37, 1, 8, 640), (3000, 2, 16, 72)):
        ids = torch.randint(-1, n, (T, k), device=DEV)
        x = torch.randn((T, D), device=DEV).bfloat16().requires_grad_()
        w, dy = torch.rand((T, k), device=DEV).requires_grad_(), torch.randn((T, D), device=DEV).bfloat16()

        def step():
            order, place, bounds = F.adapter_sort(ids, n)
            y = F.adapter_combine(F.adapter_gather(x, place), w, place, x)
            return (order, place, bounds, y, *torch.autograd.grad(y, (x, w), dy))

        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            step()
        torch.cuda.current_stream().wait_stream(s)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = step()
        for _ in range(4):
            ids.copy_(torch.randint(-1, n, (T, k), device=DEV))
            with torch.no_grad():
                x.copy_(torch.randn_like(x))
            g.replay()
            for a, c in zip(out, step()):
                assert torch.equal(a, c)


def test_other_stream(F):
    ids = make_ids("some", 5000, 2, 9).to(DEV)
    x = torch.randn((5000, 64), device=DEV).half()
    want = F.adapter_sort(ids, 9)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = F.adapter_sort(ids, 9)
        rows = F.adapter_gather(x, got[1])
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, c) for a, c in zip(got, want)) and torch.equal(rows, F.adapter_gather(x, want[1]))


@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("detach", [False, True])
@pytest.mark.parametrize("k", [1, 2])
def test_layer(q4, detach, k):
    # bf16: up to eight roundings of 2^-9 of the value each on a path, on the root mean square
    check_layer(DEV, torch.bfloat16, q4, detach, k, 2.0**-6)


def test_layer_edges():
    check_layer_edges(DEV, torch.bfloat16)


def test_layer_by_differences():
    check_by_differences(DEV)


def test_traced_outputs():
    check_traced_outputs(DEV, torch.bfloat16)


def test_wrong_arguments():
    check_wrong_arguments(DEV, torch.bfloat16)
