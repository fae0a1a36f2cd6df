"""What the binding of the serving operators refuses: types, shapes, strides and devices that do not
fit, before anything is enqueued."""
import threading

import pytest
import torch

import nvfp4_weight_only_03_b200 as nv

pytestmark = pytest.mark.gpu

BF16, F8 = torch.bfloat16, torch.float8_e4m3fn


def bf(*shape):
    return torch.zeros(shape, dtype=BF16, device="cuda")


def ints(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def attn(**kw):
    c = dict(q=bf(3, 8, 64), k_cache=bf(4, 16, 2, 64), v_cache=bf(4, 16, 2, 64),
             table=torch.zeros((2, 2), dtype=torch.int32, device="cuda"), starts=ints(0, 1, 3),
             lens=ints(5, 7))
    c.update(kw)
    return nv.paged_attention(**c)


@pytest.mark.parametrize("bad,error", [
    (lambda: dict(q=bf(3, 8, 64).float()), TypeError),
    (lambda: dict(q=bf(3, 8, 64).cpu()), ValueError),
    (lambda: dict(q=bf(3, 8, 32)), ValueError),
    (lambda: dict(q=bf(3, 7, 64)), ValueError),
    (lambda: dict(q=bf(3, 64, 8).transpose(1, 2)), ValueError),
    (lambda: dict(k_cache=bf(4, 16, 2, 64).to(F8)), TypeError),
    (lambda: dict(k_cache=bf(4, 16, 2, 64).half(), v_cache=bf(4, 16, 2, 64).half()), TypeError),
    (lambda: dict(v_cache=bf(4, 2, 16, 64).transpose(1, 2)), ValueError),
    (lambda: dict(v_cache=bf(5, 16, 2, 64)), ValueError),
    (lambda: dict(k_cache=bf(4, 16, 2, 64).cpu()), ValueError),
    (lambda: dict(k_cache=bf(4, 15, 2, 64), v_cache=bf(4, 15, 2, 64)), nv.Nvfp4Error),
    (lambda: dict(q=bf(3, 8, 96), k_cache=bf(4, 16, 2, 96), v_cache=bf(4, 16, 2, 96)),
     nv.Nvfp4Error),
    (lambda: dict(table=torch.zeros((3, 2), dtype=torch.int32, device="cuda")), ValueError),
    (lambda: dict(table=torch.zeros((2, 2), dtype=torch.int64, device="cuda")), TypeError),
    (lambda: dict(table=torch.zeros((2, 2), dtype=torch.int32, device="cuda").t()), ValueError),
    (lambda: dict(starts=ints(0, 3)), ValueError),
    (lambda: dict(starts=ints(0, 1, 3).long()), TypeError),
    (lambda: dict(lens=ints(5, 0, 7, 0)[::2]), ValueError),
    (lambda: dict(scale=0.0), nv.Nvfp4Error),
    (lambda: dict(scale=float("nan")), nv.Nvfp4Error),
    (lambda: dict(out=bf(2, 8, 64)), ValueError),
    (lambda: dict(out=bf(3, 8, 64).float()), TypeError),
    (lambda: dict(ws=torch.zeros(64, dtype=torch.uint8, device="cuda")), nv.Nvfp4Error),
    (lambda: dict(ws=torch.zeros(64, dtype=torch.uint8)), ValueError),
])
def test_attention(bad, error):
    attn()
    with pytest.raises(error):
        attn(**bad())


def test_attention_in_place():
    q = bf(3, 8, 64)
    with pytest.raises(nv.Nvfp4Error):
        attn(q=q, out=q)


def append(**kw):
    c = dict(k=bf(3, 2, 64), v=bf(3, 2, 64), k_cache=bf(4, 16, 2, 64), v_cache=bf(4, 16, 2, 64),
             slots=ints(0, 1, -1))
    c.update(kw)
    return nv.kv_append(**c)


@pytest.mark.parametrize("bad,error", [
    (lambda: dict(k=bf(3, 2, 64).float()), TypeError),
    (lambda: dict(v=bf(2, 2, 64)), ValueError),
    (lambda: dict(k=bf(3, 1, 64), v=bf(3, 1, 64)), ValueError),
    (lambda: dict(slots=ints(0, 1)), ValueError),
    (lambda: dict(slots=ints(0, 1, 2).float()), TypeError),
    (lambda: dict(k=bf(3, 2, 65)[..., 1:]), nv.Nvfp4Error),
    (lambda: dict(k_cache=bf(4, 16, 2, 64).to(F8), v_cache=bf(4, 16, 2, 64).to(F8), k_scale=0.0),
     nv.Nvfp4Error),
])
def test_append(bad, error):
    append()
    with pytest.raises(error):
        append(**bad())


def test_append_from_the_cache_itself():
    c = bf(4, 16, 2, 64)
    with pytest.raises(nv.Nvfp4Error):
        append(k=c[0, :3], k_cache=c)


def plan(**kw):
    c = dict(lens=ints(3, 4), new=ints(1, 1),
             table=torch.zeros((2, 2), dtype=torch.int32, device="cuda"), free=ints(0, 1, 2),
             head=ints(0), block_size=16, tokens=2)
    c.update(kw)
    return nv.paged_plan(**c)


@pytest.mark.parametrize("bad,error", [
    (lambda: dict(lens=ints(3, 4).long()), TypeError),
    (lambda: dict(new=ints(1)), ValueError),
    (lambda: dict(head=ints(0, 1)), ValueError),
    (lambda: dict(table=torch.zeros((3, 2), dtype=torch.int32, device="cuda")), ValueError),
    (lambda: dict(block_size=0), nv.Nvfp4Error),
    (lambda: dict(tokens=-1), ValueError),
    (lambda: dict(out=plan(tokens=3)), ValueError),
])
def test_plan(bad, error):
    plan()
    with pytest.raises(error):
        plan(**bad())


def test_plan_of_a_block_size_past_32_bits():
    for block_size in (2 ** 32 + 16, -2 ** 32 + 16, 2 ** 31, -16):
        with pytest.raises(ValueError):
            plan(block_size=block_size)


def test_plan_in_place():
    p = plan()
    with pytest.raises(nv.Nvfp4Error):
        plan(lens=p.lens, out=p)


def lora(**kw):
    c = dict(y=bf(3, 64), x=bf(3, 32), a=bf(2, 8, 32), b=bf(2, 64, 8), index=ints(0, -1, 1),
             scales=torch.ones(2, device="cuda"))
    c.update(kw)
    return nv.lora_add(**c)


@pytest.mark.parametrize("bad,error", [
    (lambda: dict(y=bf(3, 64).float()), TypeError),
    (lambda: dict(x=bf(2, 32)), ValueError),
    (lambda: dict(x=bf(3, 40)), ValueError),
    (lambda: dict(a=bf(2, 8, 32).float()), TypeError),
    (lambda: dict(b=bf(2, 8, 64)), ValueError),
    (lambda: dict(b=bf(2, 8, 64).transpose(1, 2)), ValueError),
    (lambda: dict(index=ints(0, 1)), ValueError),
    (lambda: dict(scales=torch.ones(2, device="cuda").bfloat16()), TypeError),
    (lambda: dict(scales=torch.ones(3, device="cuda")), ValueError),
    (lambda: dict(ranks=ints(8)), ValueError),
    (lambda: dict(out=bf(3, 72)), ValueError),
    (lambda: dict(a=bf(2, 12, 32), b=bf(2, 64, 12)), nv.Nvfp4Error),
    (lambda: dict(y=bf(129, 64), x=bf(129, 32), index=ints(*([0] * 129))), nv.Nvfp4Error),
])
def test_lora(bad, error):
    lora()
    with pytest.raises(error):
        lora(**bad())


def test_lora_into_its_input():
    x = bf(3, 64)
    with pytest.raises(nv.Nvfp4Error):
        lora(x=x, a=bf(2, 8, 64), out=x)


def test_threads_on_one_stream():
    """Threads that call on the same stream at the same time, adapters and attention over different
    data: each result is that of the call made alone."""
    g = torch.Generator(device="cuda").manual_seed(5)
    r = lambda *s: torch.randn(s, generator=g, device="cuda").to(BF16)
    jobs = []
    for i in range(4):
        k_cache, v_cache = r(150, 16, 2, 64), r(150, 16, 2, 64)
        table = torch.randperm(150, generator=g, device="cuda").to(torch.int32).view(1, 150)
        q, n = r(3 + 40 * (i % 2), 8, 64), 2000 + 100 * i
        starts, lens = ints(0, q.shape[0]), ints(n)
        y, x, a, b = r(9, 1024), r(9, 512), r(3, 64, 512), r(3, 1024, 64)
        index, scales = ints(*[(i + m) % 3 for m in range(9)]), torch.ones(3, device="cuda") / 64
        jobs.append((lambda q=q, k=k_cache, v=v_cache, t=table, s=starts, l=lens:
                     nv.paged_attention(q, k, v, t, s, l),
                     lambda y=y, x=x, a=a, b=b, i=index, s=scales: nv.lora_add(y, x, a, b, i, s)))
    want = [[f() for f in fs] for fs in jobs]
    same, stream = [], torch.cuda.current_stream()

    def work(fs, ws):
        with torch.cuda.stream(stream):
            for _ in range(150):
                got = [f() for f in fs]
                same.append(all(torch.equal(o, w) for o, w in zip(got, ws)))

    threads = [threading.Thread(target=work, args=a) for a in zip(jobs, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(same) == 4 * 150 and all(same)
