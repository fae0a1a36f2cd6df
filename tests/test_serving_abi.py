"""Host checks of the paged cache, attention and adapter calls: bad arguments are refused before any
CUDA call, so made-up addresses (far enough apart that only a planted overlap is one) do, and a
call without fault reports the missing device.  No GPU."""
import ctypes
import os
import re
import subprocess
import sys
import threading
import time

import pytest
import torch

from conftest import ROOT, cuda_ok
import nvfp4_weight_only_03_b200 as nv
from nvfp4_weight_only_03_b200 import build as nvbuild
from nvfp4_weight_only_03_b200 import serving as sv

NULL, SHAPE, ROWS, ALIGN, ARCH, WORKSPACE, ALIAS = -1, -2, -3, -4, -5, -7, -8


@pytest.fixture(scope="module")
def L():
    nvbuild.build()
    return nv.lib()


def at(i):
    """The i-th of addresses a terabyte apart."""
    return (i + 1) << 40


# ---------------------------------------------------------------- the plan

PLAN = dict(lens=at(0), new_tokens=at(1), requests=3, block_size=16, table=at(2), ld_table=8,
            table_columns=8, free_pages=at(3), free_count=5, head=at(4), tokens=20, starts=at(5),
            lens_out=at(6), slots=at(7), request=at(8), positions=at(9), head_out=at(10),
            missing=at(11))


def plan(L, **kw):
    return L.nvfp4_paged_plan(ctypes.byref(sv.PlanStruct(**dict(PLAN, **kw))), None)


@pytest.mark.parametrize("kw,status", [
    (dict(requests=-1), SHAPE), (dict(requests=nv.MAX_REQUESTS + 1), SHAPE),
    (dict(block_size=0), SHAPE), (dict(ld_table=7), SHAPE), (dict(table_columns=-1), SHAPE),
    (dict(free_count=-1), SHAPE), (dict(tokens=-1), SHAPE), (dict(tokens=2 ** 31), SHAPE),
    (dict(free_count=2 ** 31), SHAPE),
    (dict(lens=None), NULL), (dict(new_tokens=None), NULL), (dict(table=None), NULL),
    (dict(free_pages=None), NULL), (dict(head=None), NULL), (dict(starts=None), NULL),
    (dict(lens_out=None), NULL), (dict(slots=None), NULL), (dict(head_out=None), NULL),
    (dict(missing=None), NULL),
    (dict(slots=at(7) + 2), ALIGN), (dict(positions=at(9) + 1), ALIGN),
    (dict(lens_out=at(0)), ALIAS), (dict(head_out=at(4)), ALIAS),    # not in place
    (dict(starts=at(1) + 8), ALIAS), (dict(slots=at(7), request=at(7) + 76), ALIAS),
    (dict(table=at(3) + 4), ALIAS), (dict(missing=at(2) + 4 * 15), ALIAS),
])
def test_plan_refuses(L, kw, status):
    assert plan(L, **kw) == status


@pytest.mark.skipif(cuda_ok(), reason="only meaningful on a host without a CUDA device")
@pytest.mark.parametrize("kw", [
    {}, dict(request=None, positions=None), dict(requests=0, lens=None, new_tokens=None,
                                                 lens_out=None, table=None),
    dict(free_count=0, free_pages=None), dict(tokens=0, slots=None),
    dict(table_columns=0, ld_table=0, table=None),
    dict(missing=at(2) + 4 * 24),  # just behind the table
])
def test_plan_accepts(L, kw):
    assert plan(L, **kw) == ARCH


def test_plan_null(L):
    assert L.nvfp4_paged_plan(None, None) == NULL


# ---------------------------------------------------------------- the cache, rows into it

CACHE = dict(k=at(20), v=at(21), type=nv.KV_BF16, heads=4, dim=128, block_size=16, blocks=10,
             block_stride=16 * 512, slot_stride=512, head_stride=128, k_scale=1.0, v_scale=1.0)
F8 = dict(type=nv.KV_E4M3)

BAD_CACHE = [
    (dict(type=2), SHAPE), (dict(type=-1), SHAPE), (dict(heads=0), SHAPE), (dict(heads=1025), SHAPE),
    (dict(dim=96), SHAPE), (dict(dim=0), SHAPE), (dict(dim=512), SHAPE),
    (dict(block_size=8), SHAPE), (dict(block_size=24), SHAPE), (dict(block_size=2 ** 20 + 16), SHAPE),
    (dict(blocks=-1), SHAPE), (dict(blocks=2 ** 27), SHAPE), (dict(blocks=2 ** 60), SHAPE),
    (dict(block_stride=64), SHAPE), (dict(slot_stride=64), SHAPE), (dict(head_stride=-128), SHAPE),
    (dict(slot_stride=2 ** 39), SHAPE),
    (dict(head_stride=132), ALIGN), (dict(F8, slot_stride=520), ALIGN),
    (dict(k=None), NULL), (dict(v=None), NULL), (dict(k=at(20) + 8), ALIGN),
    (dict(F8, k_scale=0.0), SHAPE), (dict(F8, v_scale=-1.0), SHAPE),
    (dict(F8, k_scale=float("nan")), SHAPE), (dict(F8, v_scale=float("inf")), SHAPE),
]


def append(L, cache=(), **kw):
    a = dict(dict(k=at(0), ldk=512, hk=128, v=at(1), ldv=512, hv=128, tokens=7, slots=at(2)), **kw)
    c = sv.KvCacheStruct(**dict(CACHE, **dict(cache)))
    return L.nvfp4_kv_append(a["k"], a["ldk"], a["hk"], a["v"], a["ldv"], a["hv"], a["tokens"],
                             a["slots"], ctypes.byref(c), None)


@pytest.mark.parametrize("kw,status", BAD_CACHE)
def test_append_refuses_a_cache(L, kw, status):
    assert append(L, cache=kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(tokens=-1), SHAPE), (dict(ldk=64), SHAPE), (dict(hv=64), SHAPE),
    (dict(tokens=2 ** 31), SHAPE),
    (dict(k=None), NULL), (dict(v=None), NULL), (dict(slots=None), NULL),
    (dict(k=at(0) + 8), ALIGN), (dict(slots=at(2) + 2), ALIGN), (dict(ldk=516), ALIGN),
    (dict(hk=132), ALIGN),
    (dict(k=at(20) + 1024), ALIAS), (dict(v=at(21) - 16), ALIAS), (dict(slots=at(20)), ALIAS),
    (dict(cache=dict(v=at(20))), ALIAS), (dict(ldk=2 ** 62), ALIAS),  # (reaches everything)
])
def test_append_refuses(L, kw, status):
    assert append(L, **kw) == status


def test_append_accepts(L):
    assert append(L, tokens=0, k=None) == 0 and append(L, cache=dict(blocks=0, k=None)) == 0
    if not cuda_ok():
        assert append(L) == ARCH
        assert append(L, cache=dict(F8, k_scale=1e-38)) == ARCH
        assert append(L, cache=dict(k_scale=0.0)) == ARCH  # not looked at in a bf16 cache
    assert L.nvfp4_kv_append(at(0), 512, 128, at(1), 512, 128, 1, at(2), None, None) == NULL


# ---------------------------------------------------------------- attention

ATTN = dict(q=at(0), ldq=1024, q_head_stride=128, o=at(1), ldo=1024, o_head_stride=128, tokens=9,
            heads=8, requests=3, table=at(2), ld_table=8, table_columns=8, starts=at(3), lens=at(4),
            scale=0.1)


def attn(L, cache=(), ws=at(5), bytes_=1 << 40, **kw):
    a = sv.AttnStruct(**dict(ATTN, **kw))
    c = sv.KvCacheStruct(**dict(CACHE, **dict(cache)))
    return L.nvfp4_paged_attn(ctypes.byref(a), ctypes.byref(c), ws, bytes_, None)


@pytest.mark.parametrize("kw,status", BAD_CACHE)
def test_attention_refuses_a_cache(L, kw, status):
    assert attn(L, cache=kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(heads=0), SHAPE), (dict(heads=6), SHAPE), (dict(heads=-4), SHAPE),
    (dict(tokens=-1), SHAPE), (dict(tokens=2 ** 30), SHAPE), (dict(requests=-1), SHAPE),
    (dict(requests=nv.MAX_REQUESTS + 1), SHAPE), (dict(ld_table=7), SHAPE),
    (dict(table_columns=-1), SHAPE), (dict(scale=0.0), SHAPE), (dict(scale=-1.0), SHAPE),
    (dict(scale=float("nan")), SHAPE), (dict(scale=float("inf")), SHAPE),
    (dict(ldq=64), SHAPE), (dict(q_head_stride=64), SHAPE), (dict(ldo=64), SHAPE),
    (dict(o_head_stride=64), SHAPE),
    (dict(q=None), NULL), (dict(o=None), NULL), (dict(starts=None), NULL), (dict(lens=None), NULL),
    (dict(table=None), NULL),
    (dict(q=at(0) + 8), ALIGN), (dict(o=at(1) + 4), ALIGN), (dict(ldq=1028), ALIGN),
    (dict(o_head_stride=132), ALIGN), (dict(table=at(2) + 2), ALIGN),
    (dict(o=at(0)), ALIAS), (dict(o=at(0) + 1024), ALIAS), (dict(o=at(20) + 64), ALIAS),
    (dict(o=at(21)), ALIAS), (dict(o=at(2)), ALIAS), (dict(o=at(3)), ALIAS), (dict(o=at(4)), ALIAS),
    (dict(ldo=2 ** 61), ALIAS), (dict(ldq=2 ** 61), ALIAS),
    (dict(ws=None), WORKSPACE), (dict(ws=at(5) + 8), WORKSPACE),
])
def test_attention_refuses(L, kw, status):
    assert attn(L, **kw) == status


def test_attention_accepts(L):
    assert attn(L, tokens=0, q=None) == 0 and attn(L, requests=0, lens=None) == 0
    b = ctypes.c_size_t()
    assert L.nvfp4_paged_attn_workspace_bytes(128, None) == NULL
    assert L.nvfp4_paged_attn_workspace_bytes(100, ctypes.byref(b)) == SHAPE
    if not cuda_ok():
        assert attn(L) == ARCH and attn(L, cache=F8) == ARCH
        assert attn(L, table_columns=0, table=None) == ARCH
        assert attn(L, cache=dict(blocks=0, k=None, v=None)) == ARCH
        assert L.nvfp4_paged_attn_workspace_bytes(128, ctypes.byref(b)) == ARCH


def test_attention_roles_leave_their_waits_together():
    """A bounded wait may give up in some lanes of a warp and not in others (its last tries are apart in
    time), and what follows it is for whole warps.  So each wait of the attention kernel that ends on
    `stop` is inside a vote of the warp; the softmax warps', which go on either way, are one lambda."""
    path = os.path.join(ROOT, "nvfp4_weight_only_03_b200", "csrc", "nvfp4_attn.cu")
    text = re.sub(r"//[^\n]*", "", open(path).read())
    statements = [s for s in re.split(r"[;{}]", text) if "mbar_wait(" in s and "stop_v" in s]
    assert len(statements) >= 5
    alone = [s for s in statements if "__all_sync(~0u, mbar_wait(" not in s]
    assert [" ".join(s.split()) for s in alone] == ["if (ok && !mbar_wait(b, parity, stop_v)) ok = false"]


# ---------------------------------------------------------------- adapters

LORA = dict(a=at(0), a_stride=16 * 256, a_ld=256, b=at(1), b_stride=512 * 16, b_ld=16, scales=at(2),
            ranks=at(3), index=at(4), adapters=5, rank=16)


def lora(L, x=at(5), ldx=256, y=at(6), ldy=512, out=at(7), ldo=512, m=3, n=512, k=256, ws=at(8),
         bytes_=1 << 40, **kw):
    l = sv.LoraStruct(**dict(LORA, **kw))
    return L.nvfp4_lora_add(ctypes.byref(l), x, ldx, y, ldy, out, ldo, m, n, k, ws, bytes_, None)


@pytest.mark.parametrize("kw,status", [
    (dict(m=-1), ROWS), (dict(m=129), ROWS),
    (dict(rank=12), SHAPE), (dict(rank=136), SHAPE), (dict(rank=-8), SHAPE),
    (dict(adapters=-1), SHAPE), (dict(adapters=40000), SHAPE), (dict(k=250), SHAPE),
    (dict(n=500), SHAPE), (dict(n=-8), SHAPE), (dict(k=-8), SHAPE),
    (dict(ldx=128), SHAPE), (dict(ldy=256), SHAPE), (dict(ldo=256), SHAPE), (dict(a_ld=128), SHAPE),
    (dict(b_ld=8), SHAPE), (dict(a_stride=-16), SHAPE),
    (dict(x=None), NULL), (dict(y=None), NULL), (dict(out=None), NULL), (dict(a=None), NULL),
    (dict(b=None), NULL), (dict(scales=None), NULL), (dict(index=None), NULL),
    (dict(x=at(5) + 8), ALIGN), (dict(out=at(7) + 2), ALIGN), (dict(a=at(0) + 8), ALIGN),
    (dict(ldx=260), ALIGN), (dict(b_ld=20), ALIGN), (dict(a_stride=4100), ALIGN),
    (dict(index=at(4) + 2), ALIGN), (dict(ranks=at(3) + 1), ALIGN),
    (dict(out=at(6) + 1024), ALIAS), (dict(out=at(6), ldo=520), ALIAS), (dict(out=at(5)), ALIAS),
    (dict(out=at(0) + 4096), ALIAS), (dict(out=at(1)), ALIAS), (dict(out=at(2)), ALIAS),
    (dict(out=at(3)), ALIAS), (dict(out=at(4)), ALIAS), (dict(ldo=2 ** 61), ALIAS),
])
def test_lora_refuses(L, kw, status):
    assert lora(L, **kw) == status


@pytest.mark.parametrize("kw,status", [
    ({}, 0), (dict(out=at(6)), 0), (dict(m=0, y=None), 0), (dict(ranks=None), 0), (dict(m=129), ROWS),
    (dict(rank=12), SHAPE), (dict(k=250), SHAPE), (dict(a=None), NULL), (dict(ldx=260), ALIGN),
    (dict(out=at(5)), ALIAS),
])
def test_lora_check_says_what_the_call_would(L, kw, status):
    a = dict(dict(x=at(5), ldx=256, y=at(6), ldy=512, out=at(7), ldo=512, m=3, n=512, k=256), **kw)
    call = [a.pop(i) for i in ("x", "ldx", "y", "ldy", "out", "ldo", "m", "n", "k")]
    l = sv.LoraStruct(**dict(LORA, **a))
    assert L.nvfp4_lora_check(ctypes.byref(l), *call) == status
    if status:
        assert lora(L, **kw) == status


def test_lora_accepts(L):
    assert lora(L, m=0, y=None) == 0 and lora(L, n=0, out=None) == 0
    if not cuda_ok():
        assert lora(L) == ARCH and lora(L, out=at(6)) == ARCH  # y in place
        assert lora(L, ranks=None) == ARCH
        assert lora(L, adapters=0, a=None, b=None, scales=None, x=None) == ARCH
    b = ctypes.c_size_t()
    assert L.nvfp4_lora_workspace_bytes(1, 1, 16, 64, None) == NULL
    assert L.nvfp4_lora_workspace_bytes(129, 1, 16, 64, ctypes.byref(b)) == ROWS
    assert L.nvfp4_lora_workspace_bytes(1, 1, 20, 64, ctypes.byref(b)) == SHAPE
    assert L.nvfp4_lora_add(None, at(5), 256, at(6), 512, at(7), 512, 1, 512, 256, at(8), 1 << 40,
                            None) == NULL


# ---------------------------------------------------------------- the binding


def test_binding_wants_cuda_tensors():
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        nv.paged_plan(i, i, torch.zeros((2, 3), dtype=torch.int32), i, i[:1], 16, 4)
    q = torch.zeros((2, 4, 64), dtype=torch.bfloat16)
    c = torch.zeros((3, 16, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        nv.kv_append(q[:, :2], q[:, :2], c, c.clone(), i)
    with pytest.raises(ValueError):
        nv.paged_attention(q, c, c.clone(), torch.zeros((1, 3), dtype=torch.int32), i, i[:1])
    y = torch.zeros((2, 8), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        nv.lora_add(y, y, torch.zeros((1, 8, 8), dtype=torch.bfloat16),
                    torch.zeros((1, 8, 8), dtype=torch.bfloat16), i, torch.zeros(1))


class _Enqueuer:
    """Stands in for the library: counts how many calls with one workspace are inside at once."""

    def __init__(self):
        self.inside, self.most, self.calls = {}, 0, 0

    def __getattr__(self, name):
        def call(*args):
            ws = next(a for a in args if isinstance(a, int) and a in self.inside)
            self.inside[ws] += 1
            self.most = max(self.most, self.inside[ws])
            time.sleep(0.002)  # (the interpreter's lock is free meanwhile, as during a library call)
            self.inside[ws] -= 1
            self.calls += 1
            return 0
        return call


@pytest.mark.parametrize("op", ["attention", "lora"])
def test_threads_do_not_enqueue_into_one_workspace_at_once(monkeypatch, op):
    """Two threads on one stream: a call's launches stay together, since the next call's would read
    what they left in the shared workspace."""
    lib, ws = _Enqueuer(), torch.zeros(1 << 16, dtype=torch.uint8)
    lib.inside[ws.data_ptr()] = 0
    monkeypatch.setattr(sv, "_lib", lib)
    monkeypatch.setattr(sv, "_elsewhere", lambda *_: False)
    monkeypatch.setattr(sv, "_raw_stream", lambda _: 0)
    monkeypatch.setattr(sv, "_capturing", lambda: False)
    monkeypatch.setattr(sv, "_workspaces", {})
    monkeypatch.setattr(sv, "paged_attention_workspace_bytes", lambda _: ws.numel())
    monkeypatch.setattr(sv, "lora_workspace_bytes", lambda *_: ws.numel())
    monkeypatch.setattr(nv, "_cached_workspace", lambda *_: ws)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *_: None)
    monkeypatch.setattr(torch, "device", lambda *_: None)
    i = torch.zeros(2, dtype=torch.int32)
    z = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    if op == "attention":
        q, c = z(2, 4, 64), [z(3, 16, 2, 64) for _ in "kv"]
        table = torch.zeros((1, 3), dtype=torch.int32)
        call = lambda: nv.paged_attention(q, *c, table, i, i[:1])
    else:
        y, x, a, b = z(2, 8), z(2, 8), z(1, 8, 8), z(1, 8, 8)
        call = lambda: nv.lora_add(y, x, a, b, i, torch.zeros(1))
    threads = [threading.Thread(target=lambda: [call() for _ in range(10)]) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert lib.calls == 40 and lib.most == 1


def test_import_without_torch_cuda_symbols():
    """The package imports, and answers what needs no device, with a torch that has no CUDA."""
    code = """
import torch
for name in ("_cuda_getCurrentRawStream", "_cuda_getDevice", "_cuda_isCurrentStreamCapturing"):
    if hasattr(torch._C, name):
        delattr(torch._C, name)
import nvfp4_weight_only_03_b200 as nv
assert nv.pack_info(64, 64)["n"] == 64
i = torch.zeros(2, dtype=torch.int32)
try:
    nv.paged_plan(i, i, torch.zeros((2, 3), dtype=torch.int32), i, i[:1], 16, 4)
except ValueError as e:
    assert "CUDA device" in str(e)
else:
    raise AssertionError("a CPU tensor was taken")
"""
    subprocess.run([sys.executable, "-c", code], check=True, cwd=ROOT)


@pytest.mark.parametrize("ws", [lambda: torch.zeros(1).expand(1 << 20), lambda: torch.zeros(64)[::2],
                                lambda: torch.zeros((8, 8)).t()])
def test_workspace_of_a_caller_is_contiguous(ws):
    # (looked at on the host: a call would write past the elements that are there)
    with pytest.raises(ValueError):
        sv._own_workspace(ws(), -1)
    assert sv._own_workspace(torch.zeros(64), -1)[1] == 256


def test_threads_ask_for_the_device_at_once(L):
    """The first calls of a process may come from many threads: all get the same answer."""
    code = """
import ctypes, threading
import nvfp4_weight_only_03_b200 as nv
L, got, go = nv.lib(), [], threading.Barrier(16)
def ask():
    b = ctypes.c_size_t()
    go.wait()
    for _ in range(50):
        got.append((L.nvfp4_paged_attn_workspace_bytes(128, ctypes.byref(b)), b.value))
threads = [threading.Thread(target=ask) for _ in range(16)]
for t in threads: t.start()
for t in threads: t.join()
assert len(got) == 800 and len(set(got)) == 1, set(got)
"""
    subprocess.run([sys.executable, "-c", code], check=True, cwd=ROOT)
