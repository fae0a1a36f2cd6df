"""Adapters beside a projection against a plain implementation in 64 bits.

Tolerance per element, with S = |scale| sum_r |b_r| sum_k |a_rk x_k| (all products by magnitude):
  output rounding                2^-8 |out| (half a step of bf16)
  T = A x in fp32                chains of at most K / 16 + 64 additions: (K / 16 + 64) 2^-23 S
  T as two bf16 values           2^-16 S (the remainder's own rounding, 2^-8 of 2^-8)
  B T and the sum with y         (rank / 8 + 8) 2^-23 (S + |y|)
"""
import numpy as np
import pytest
import torch

import nvfp4_weight_only_03_b200 as nv
import synth
from gpu_util import dev_weight

pytestmark = pytest.mark.gpu


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def inputs(seed, m, n, k, adapters, rank, ranks=None):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()
    a, b = r(adapters, rank, k), r(adapters, n, rank)
    if ranks is not None:  # what lies past an adapter's rank is never used
        for i, x in enumerate(ranks):
            a[i, max(x, 0):] = float("nan")
            b[i, :, max(x, 0):] = float("nan")
    scales = torch.linspace(-0.5, 1.5, adapters, device="cuda") / k ** 0.5
    return r(m, n), r(m, k), a, b, scales


def reference(y, x, a, b, index, scales, ranks):
    out, tol = y.double(), torch.zeros_like(y, dtype=torch.float64)
    k, rank = x.shape[1], a.shape[1]
    for m, i in enumerate(index):
        if not 0 <= i < a.shape[0]:
            continue
        r = rank if ranks is None else min(max(ranks[i], 0), rank)
        A, B, s = a[i, :r].double(), b[i, :, :r].double(), scales[i].double()
        out[m] += s * (B @ (A @ x[m].double()))
        S = s.abs() * (B.abs() @ (A.abs() @ x[m].double().abs()))
        tol[m] = 2.0 ** -8 * out[m].abs() + (k / 16 + 64) * 2.0 ** -23 * S + 2.0 ** -16 * S + \
            (rank / 8 + 8) * 2.0 ** -23 * (S + y[m].double().abs())
    return out, tol


def check(y, x, a, b, index, scales, ranks=None, **kw):
    out = nv.lora_add(y, x, a, b, ints(index), scales,
                      ranks=None if ranks is None else ints(ranks), **kw)
    ref, tol = reference(y, x, a, b, index, scales, ranks)
    err = (out.double() - ref).abs()
    assert (err <= tol).all(), f"{((err - tol).max()).item()} past the tolerance"
    return out


@pytest.mark.parametrize("rank", [8, 16, 24, 32, 40, 64, 72, 128])
@pytest.mark.parametrize("m", [1, 2, 9])
def test_ranks_and_rows(m, rank):
    n, k = 264, 520
    y, x, a, b, scales = inputs(rank + m, m, n, k, 3, rank)
    check(y, x, a, b, [(2 * i) % 3 for i in range(m)], scales)


@pytest.mark.parametrize("n,k", [(8, 8), (1000, 8), (8, 4096), (256, 256), (5120, 17408),
                                 (10240, 5120)])
def test_sizes(n, k):
    y, x, a, b, scales = inputs(n + k, 5, n, k, 4, 16)
    check(y, x, a, b, [3, 0, 3, -1, 1], scales)


@pytest.mark.parametrize("m,adapters", [(128, 1), (128, 128), (128, 5), (127, 40), (33, 2),
                                        (17, 17)])
def test_groups(m, adapters):
    rng = np.random.default_rng(m + adapters)
    y, x, a, b, scales = inputs(m, m, 520, 776, adapters, 32)
    index = [int(i) for i in rng.permutation(np.arange(m) % adapters)]
    check(y, x, a, b, index, scales)


def test_rows_without_an_adapter_keep_y():
    y, x, a, b, scales = inputs(1, 6, 264, 520, 3, 16)
    y[1, 3] = -0.0
    y[4, 5] = float("nan")
    out = check(y[:4], x[:4], a, b, [-1, -1, 2 ** 31 - 1, -2 ** 31], scales)
    assert torch.equal(out.view(torch.int16), y[:4].view(torch.int16))
    out = nv.lora_add(y, x, a, b, ints([0, -1, 3, 2, -7, 1]), scales)
    for row in (1, 2, 4):
        assert torch.equal(out[row].view(torch.int16), y[row].view(torch.int16))


def test_each_adapters_own_rank():
    ranks = [64, 0, 7, 33, 100, -3, 1]
    y, x, a, b, scales = inputs(2, 40, 520, 1032, 7, 64, ranks)
    check(y, x, a, b, [i % 8 - 1 for i in range(40)], scales, ranks)


def test_in_place_strided_and_repeated():
    y, x, a, b, scales = inputs(3, 20, 520, 776, 4, 24)
    index = [i % 5 - 1 for i in range(20)]
    want = check(y, x, a, b, index, scales)
    wide = torch.zeros((20, 1000), dtype=torch.bfloat16, device="cuda")
    wide[:, 16:536] = y
    xs = torch.zeros((20, 1600), dtype=torch.bfloat16, device="cuda")
    xs[:, 800:1576] = x
    aa = torch.zeros((4, 30, 800), dtype=torch.bfloat16, device="cuda")
    aa[:, :24, 16:792] = a
    bb = torch.zeros((8, 520, 40), dtype=torch.bfloat16, device="cuda")
    bb[::2, :, 8:32] = b
    view = wide[:, 16:536]
    got = check(view, xs[:, 800:1576], aa[:, :24, 16:792], bb[::2, :, 8:32], index, scales)
    assert torch.equal(got, want)
    nv.lora_add(view, xs[:, 800:1576], a, b, ints(index), scales, out=view)
    assert torch.equal(view, want) and (wide[:, :16] == 0).all() and (wide[:, 536:] == 0).all()
    for _ in range(5):
        assert torch.equal(nv.lora_add(y, x, a, b, ints(index), scales), want)


def test_infinities_stay_in_their_row():
    y, x, a, b, scales = inputs(4, 4, 264, 520, 2, 16)
    x[1, 7] = float("inf")
    x[2, 9] = float("nan")
    out = nv.lora_add(y, x, a, b, ints([0, 0, 1, 1]), scales)
    ref, tol = reference(y, x, a, b, [0, 0, 1, 1], scales, None)
    assert not torch.isfinite(out[1:3]).any()
    for row in (0, 3):
        assert ((out[row].double() - ref[row]).abs() <= tol[row]).all()


def test_captured_call_serves_later_indexes():
    y, x, a, b, scales = inputs(5, 6, 264, 520, 3, 16)
    index, out = ints([0, 1, 2, 0, 1, 2]), torch.empty_like(y)
    call = lambda: nv.lora_add(y, x, a, b, index, scales, out=out)
    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for now in ([0, 1, 2, 0, 1, 2], [-1, -1, -1, -1, -1, -1], [2, 2, 2, 2, 2, 2]):
        index.copy_(ints(now))
        graph.replay()
        ref, tol = reference(y, x, a, b, now, scales, None)
        assert ((out.double() - ref).abs() <= tol).all()


def test_beside_the_projection():
    """gemv, then the adapters of its rows, as gemv(..., lora=...) runs them in one call."""
    n, k, m = 1024, 512, 5
    W, S, g = dev_weight(synth.nvfp4_weight(60, 0, n, k))
    _, x, a, b, scales = inputs(6, m, n, k, 3, 16)
    index = ints([0, 2, -1, 1, 0])
    base = nv.gemv(W, S, g, x)
    want = check(base, x, a, b, index.tolist(), scales)
    lora = nv.Lora(a, b, index, scales)
    assert torch.equal(nv.gemv(W, S, g, x, lora=lora), want)
    q, p = nv.gemv_multi([(W, S, g), (W, S, g)], x, lora=[lora, None])
    assert torch.equal(q, want) and torch.equal(p, base)
    with pytest.raises(ValueError):  # the adapters' x is the prologue's result, kept in the call
        nv.gemv(W, S, g, x, lora=lora, prologue=nv.SigmoidGate(x))
    one = nv.Lora(a, b, ints([2]), scales)  # a row as a vector, as gemv takes it
    assert torch.equal(nv.gemv(W, S, g, x[1], lora=one).view(-1), want[1])


def test_another_stream():
    y, x, a, b, scales = inputs(8, 5, 264, 520, 3, 24)
    index = ints([0, 2, 1, -1, 2])
    want = nv.lora_add(y, x, a, b, index, scales)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    out = nv.lora_add(y, x, a, b, index, scales, stream=stream)
    stream.synchronize()
    assert torch.equal(out, want)


@pytest.mark.parametrize("bad", ["rank", "dtype", "b", "index", "scales", "device", "ld", "k"])
def test_refused_adapters_leave_the_projection_unwritten(bad):
    """gemv(..., lora=) and gemv_multi(..., lora=) refuse adapters that do not fit before the
    projection is enqueued: a caller's y stays as it was."""
    n, k, m = 256, 512, 5
    W = dev_weight(synth.nvfp4_weight(61, 0, n, k))
    _, x, a, b, scales = inputs(7, m, n, k, 3, 16)
    index = ints([0, 2, -1, 1, 0])
    good = nv.Lora(a, b, index, scales)
    buf = torch.full((m, n + 4), 7.0, dtype=torch.bfloat16, device="cuda")
    y = torch.full((m, n), 7.0, dtype=torch.bfloat16, device="cuda")
    if bad == "rank":
        lora = nv.Lora(a[:, :12].contiguous(), b[:, :, :12].contiguous(), index, scales)
    elif bad == "dtype":
        lora = nv.Lora(a.float(), b, index, scales)
    elif bad == "b":
        lora = nv.Lora(a, b[:, :-8], index, scales)
    elif bad == "index":
        lora = nv.Lora(a, b, index[:4], scales)
    elif bad == "scales":
        lora = nv.Lora(a, b, index, scales[:2])
    elif bad == "device":
        lora = nv.Lora(a, b, index.cpu(), scales)
    elif bad == "ld":  # rows of 8 bytes more than lora_add takes; the projection alone takes them
        lora, y = good, buf[:, :n]
    else:
        lora = nv.Lora(a[:, :, :504], b, index, scales)
    error = (ValueError, TypeError, nv.Nvfp4Error)
    with pytest.raises(error):
        nv.gemv(*W, x, y=y, lora=lora)
    assert (y == 7.0).all()
    other = torch.full((m, n), 7.0, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(error):
        nv.gemv_multi([W, W], x, ys=[other, y], lora=[good, lora])
    assert (other == 7.0).all() and (y == 7.0).all()
    # without the fault the call goes through
    assert torch.equal(nv.gemv(*W, x, y=other, lora=good),
                       nv.lora_add(nv.gemv(*W, x), x, a, b, index, scales))
