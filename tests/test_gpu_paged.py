"""Paged cache and attention through the binding: block tables and slot maps, cache rows, and the
attention, each against a plain implementation in 64 bits (whole numbers and copies: exactly).

Tolerance of the attention, per element, with A = sum_j w_j |v_j| / sum_j w_j over the keys a row
sees, h the half step of a rounding (bf16 2^-8, f16 2^-11, fp32 2^-24):
  output rounding              2^-8 |o|
  weights rounded for the MMA  (2^-8 bf16 cache, 2^-11 e4m3 cache) A, and for f16 half its
                               smallest step, 2^-25, per key: n 2^-25 max|v| (a row's largest
                               weight is at least 1, so the sum of weights is, too)
  scores                       a sum of D products off by at most D 2^-23 sum|q k| (twice the
                               rounding of every partial sum) moves a weight by as much,
                               relatively, in the numerator and in the sum: 2 delta A.  With an
                               e4m3 cache q is carried as two e4m3 terms of q 2^e, |q 2^e| < 2^8:
                               off by at most half their smallest step, 2^-10, where the row's
                               largest is at least 2^7: delta also has 2^-17 max|q| sum|k|
  exponent and sums            2^-20 (argument, ex2 and the rescaling), and 2^-23 per step of a
                               chain of n / 16 MMA steps and 128 additions, in both: times 2 A
"""
import numpy as np
import pytest
import torch

import nvfp4_weight_only_03_b200 as nv
import synth
from gpu_util import dev_weight

pytestmark = pytest.mark.gpu

F8 = torch.float8_e4m3fn


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def make_cache(g, blocks, block, heads, dim, f8, layout="nhd"):
    """K and V caches full of NaN in one of the layouts a program may keep."""
    dt = F8 if f8 else torch.bfloat16
    if layout == "hnd":  # [blocks][heads][block][dim]
        make = lambda: torch.empty((blocks, heads, block, dim), device="cuda", dtype=dt) \
            .transpose(1, 2)
        k, v = make(), make()
    elif layout == "joint":  # [blocks][2][block][heads][dim]
        both = torch.empty((blocks, 2, block, heads, dim), device="cuda", dtype=dt)
        k, v = both[:, 0], both[:, 1]
    else:
        k, v = (torch.empty((blocks, block, heads, dim), device="cuda", dtype=dt)
                for _ in range(2))
    for c in (k, v):
        if f8:
            c.view(torch.uint8).fill_(0x7F)
        else:
            c.fill_(float("nan"))
    return k, v


def put(cache, page, place, rows):
    if cache.dtype == F8:
        cache.view(torch.uint8)[page, place] = rows.to(F8).view(torch.uint8)
    else:
        cache[page, place] = rows.to(cache.dtype)


class Batch:
    """Requests with their keys and values scattered over random pages; every slot that no
    request owns holds NaN."""

    def __init__(self, seed, lens, new, heads, kv_heads, dim, block, f8=False, layout="nhd",
                 q_scale=1.5, pad=0, spare_columns=1, holes=()):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.lens, self.new, self.f8, self.dim = lens, new, f8, dim
        self.heads, self.kv_heads = heads, kv_heads
        pages = [-(-n // block) for n in lens]
        total = sum(pages) + 3
        order = rng.permutation(total)
        cols = max(pages + [0]) + spare_columns
        table = np.full((len(lens), cols), -1, np.int32)
        at = 0
        for r, n in enumerate(pages):
            table[r, :n] = order[at:at + n]
            at += n
        self.kc, self.vc = make_cache(g, total, block, kv_heads, dim, f8, layout)
        self.k_scale, self.v_scale = (0.25, 0.125) if f8 else (1.0, 1.0)
        spread = 4.0 if f8 else 1.0
        for r, n in enumerate(lens):
            if n == 0:
                continue
            pos = torch.arange(n, device="cuda")
            page = torch.from_numpy(table[r]).cuda().long()[pos // block]
            for c in (self.kc, self.vc):
                rows = torch.randn((n, kv_heads, dim), generator=g, device="cuda") * spread
                put(c, page, pos % block, rows)
        for r, c, page in holes:  # entries that name no page
            table[r, c] = page
        self.table = torch.from_numpy(table).cuda()
        t = sum(new)
        self.tokens = t
        self.q = torch.randn((t + pad, heads, dim), generator=g, device="cuda")\
            .mul_(q_scale).to(torch.bfloat16)
        self.starts = ints([0] + list(np.cumsum(new)))
        self.block, self.blocks, self.cols = block, total, cols
        self.scale = dim ** -0.5

    def call(self, **kw):
        kw.setdefault("q", self.q)
        q = kw.pop("q")
        return nv.paged_attention(q, self.kc, self.vc, self.table, self.starts, ints(self.lens),
                                  k_scale=self.k_scale, v_scale=self.v_scale, scale=self.scale,
                                  check=kw.pop("check", True), **kw)

    def reference(self):
        """(o, tolerance) in 64 bits."""
        t, G = self.tokens, self.heads // self.kv_heads
        o = torch.zeros((t, self.heads, self.dim), dtype=torch.float64, device="cuda")
        tol = torch.zeros_like(o)
        first = 0
        for r, (n, m) in enumerate(zip(self.lens, self.new)):
            if m == 0:
                continue
            cap = min(n, self.cols * self.block)
            pos = torch.arange(cap, device="cuda")
            page = self.table[r].long()[pos // self.block]
            there = (page >= 0) & (page < self.blocks)
            pg = torch.where(there, page, 0)
            p = n - m + torch.arange(m, device="cuda")
            for h in range(self.kv_heads):
                k, v = (c[pg, pos % self.block, h].double() if not self.f8 else
                        c.view(torch.uint8)[pg, pos % self.block, h].view(F8).double()
                        for c in (self.kc, self.vc))
                k, v = k * self.k_scale, v * self.v_scale
                q = self.q[first:first + m, h * G:(h + 1) * G].double()
                s = torch.einsum("mgd,nd->mgn", q, k) * self.scale
                mag = torch.einsum("mgd,nd->mgn", q.abs(), k.abs()) * self.scale
                see = (there & (pos <= p[:, None]))[:, None, :]
                s = torch.where(see, s, -torch.inf)
                delta = torch.where(see, mag, 0.0).amax(-1) if cap else q.new_zeros(m, G)
                delta = delta * self.dim * 2.0 ** -23
                if self.f8 and cap:
                    delta = delta + 2.0 ** -17 * self.scale * q.abs().amax(-1) * \
                        k.abs().sum(-1).nan_to_num(0.0).max()
                w = torch.exp(s - s.amax(-1, keepdim=True).clamp(min=-1e300)) if cap else s
                tot = w.sum(-1, keepdim=True)
                w = torch.where(tot > 0, w / tot.clamp(min=1e-300), 0.0)
                v = torch.where(torch.isnan(v) & ~there[:, None], 0.0, v)
                vis = see.expand(w.shape).any(1).any(0)
                v = torch.where(vis[:, None], v, 0.0)
                out = torch.einsum("mgn,nd->mgd", w, v)
                A = torch.einsum("mgn,nd->mgd", w, v.abs())
                n_vis = max(cap, 1)
                rel = (2.0 ** -11 if self.f8 else 2.0 ** -8) + 2 * delta[..., None] + \
                    2 * (2.0 ** -20 + (n_vis / 16 + 128) * 2.0 ** -23)
                sl = (slice(first, first + m), slice(h * G, (h + 1) * G))
                o[sl] = out
                tol[sl] = 2.0 ** -8 * out.abs() + rel * A + 1e-30
                if self.f8 and cap:
                    tol[sl] += n_vis * 2.0 ** -25 * v.abs().max()
            first += m
        return o, tol


def check_attention(b, **kw):
    out = b.call(**kw)
    ref, tol = b.reference()
    got = out[:b.tokens].double()
    assert torch.isfinite(got).all(), "a masked or unowned value reached a result"
    err = (got - ref).abs()
    worst = (err / tol.clamp(min=1e-30)).max().item() if err.numel() else 0.0
    assert worst <= 1.0, f"error {worst:.3f} of the tolerance"
    return out


GEOMETRY = [(24, 4, 256), (8, 8, 128), (7, 1, 64), (32, 8, 128)]


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("heads,kv_heads,dim", GEOMETRY)
def test_decode_lengths(heads, kv_heads, dim, f8):
    lens = [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 300]
    check_attention(Batch(1, lens, [1] * len(lens), heads, kv_heads, dim, 16, f8))


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("heads,kv_heads,dim", GEOMETRY)
def test_chunks(heads, kv_heads, dim, f8):
    # whole prompts, chunks at the end of longer ones, one token, idle requests
    lens, new = [45, 200, 70, 9, 130, 33], [45, 31, 1, 0, 130, 8]
    check_attention(Batch(2, lens, new, heads, kv_heads, dim, 32, f8, pad=3))


@pytest.mark.parametrize("layout", ["nhd", "hnd", "joint"])
@pytest.mark.parametrize("block", [16, 48, 64, 256])
def test_layouts_and_pages(layout, block):
    for f8 in (False, True):
        check_attention(Batch(3, [517, 1, 95, 256], [3, 1, 20, 1], 12, 2, 128, block, f8, layout))


def test_empty_requests_and_rows_without_keys():
    # no keys at all; more new tokens than keys (the first ones see none); idle requests around
    b = Batch(4, [0, 5, 0, 20], [2, 0, 0, 30], 6, 2, 64, 16)
    out = check_attention(b)
    assert (out[:2] == 0).all() and (out[2:12] == 0).all()


def test_pages_that_do_not_exist():
    # entries of -1, past the cache and far past it; a table that ends before the length does
    for f8 in (False, True):
        holes = [(0, 0, -1), (0, 3, 10 ** 6), (1, 1, -(2 ** 31)), (1, 2, 2 ** 31 - 1)]
        check_attention(Batch(5, [100, 60], [9, 4], 12, 2, 128, 16, f8, holes=holes))
        b = Batch(6, [100, 60], [9, 4], 12, 2, 128, 16, f8)
        b.lens = [100, 600]  # 600 tokens claimed, the table holds at most 128
        ref, tol = b.reference()
        got = b.call()[:b.tokens].double()
        # request 0 as ever; request 1's rows see everything that its table holds: the last
        # page's four unowned slots, which hold NaN, among it
        assert ((got - ref).abs() <= tol)[:9].all()
        assert torch.isnan(ref[9:]).all() and torch.isnan(got[9:]).all()
        b = Batch(6, [100, 64], [9, 4], 12, 2, 128, 16, f8)
        b.lens = [100, 600]  # the pages that are there are full
        check_attention(b)


def test_large_scores_and_rising_maxima():
    # scores that rise along the context, so that running maxima move again and again
    b = Batch(7, [900, 700], [5, 1], 12, 2, 128, 16, q_scale=8.0)
    check_attention(b)
    b = Batch(8, [900], [40], 6, 1, 256, 16, q_scale=8.0)
    ramp = torch.linspace(0.1, 3.0, 900, device="cuda")
    pos = torch.arange(900, device="cuda")
    page = b.table[0].long()[pos // 16]
    b.kc[page, pos % 16] = (b.kc[page, pos % 16].float() * ramp[:, None, None]).bfloat16()
    check_attention(b)


@pytest.mark.parametrize("f8", [False, True])
def test_nan_of_a_visible_token_reaches_its_rows_and_no_others(f8):
    # request 1's key 37 and request 2's value 5 are NaN: every row of theirs sees them, and the
    # value's NaN stays in its dimension
    b = Batch(16, [90, 70, 60], [1, 1, 1], 12, 2, 128, 16, f8)
    want = b.call()
    for r, key, cache, dims in ((1, 37, b.kc, slice(3, 4)), (2, 5, b.vc, slice(77, 79))):
        page = int(b.table[r, key // 16])
        if f8:
            cache.view(torch.uint8)[page, key % 16, :, dims] = 0xFF
        else:
            cache[page, key % 16, :, dims] = float("nan")
    out = b.call()
    assert torch.equal(out[0], want[0])
    assert torch.isnan(out[1]).all()
    assert torch.isnan(out[2, :, 77:79]).all()
    rest = [d for d in range(128) if d not in (77, 78)]
    assert torch.equal(out[2][:, rest], want[2][:, rest])


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("heads,kv_heads,dim,len_,new,block", [
    (24, 4, 256, 300, 8, 16), (12, 2, 128, 700, 200, 16), (7, 1, 64, 150, 150, 48),
    (24, 4, 256, 9000, 100, 64), (5, 5, 128, 333, 333, 32)])
def test_values_that_are_not_finite_reach_the_rows_that_see_them_and_no_others(heads, kv_heads, dim,
                                                                               len_, new, block,
                                                                               f8):
    b = Batch(30, [70, len_, 33], [3, new, 33], heads, kv_heads, dim, block, f8)
    want = b.call()
    first, keys = len_ - new, [len_ - new + 1, len_ - new // 2, len_ - 1]
    seen = torch.zeros(new, dim, dtype=torch.bool, device="cuda")
    for i, key in enumerate(keys):  # a key of the new ones, each in dimensions of its own
        page = int(b.table[1, key // block])
        dims = slice(dim // 4 * i + 3, dim // 4 * i + 6)
        if f8:
            b.vc.view(torch.uint8)[page, key % block, :, dims] = 0x7F if i else 0xFF
        else:
            b.vc[page, key % block, :, dims] = (float("nan"), float("inf"), -float("inf"))[i]
        seen[key - first:, dims] = True
    out = b.call()
    mine = slice(3, 3 + new)
    assert torch.equal(out[:3], want[:3]) and torch.equal(out[3 + new:], want[3 + new:])
    hit = seen[:, None].expand(new, heads, dim)
    assert not torch.isfinite(out[mine][hit]).any()
    assert torch.equal(out[mine][~hit], want[mine][~hit])
    if not f8:
        d = dim // 4 + 4
        assert (out[mine][keys[1] - first:, :, d] == float("inf")).all()
        assert (out[mine][keys[2] - first:, :, 2 * (dim // 4) + 4] == -float("inf")).all()


@pytest.mark.parametrize("f8", [False, True])
def test_many_requests_and_long_context(f8):
    rng = np.random.default_rng(9)
    lens = [int(x) for x in rng.integers(1, 400, 300)]
    check_attention(Batch(9, lens, [1] * 300, 8, 2, 64, 16, f8))
    check_attention(Batch(10, [20011], [8], 24, 4, 256, 64, f8))
    check_attention(Batch(11, [3001, 2500], [500, 333], 12, 2, 128, 16, f8))


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("q_scale", [1e4, 1e6, 3e7, 1e9])
def test_scores_of_any_size_give_finite_rows(q_scale, f8):
    # (the tolerance says nothing here: an fp32 score is off by more than a power of two)
    b = Batch(83, [900, 333], [5, 40], 12, 2, 128, 16, f8, q_scale=q_scale)
    out = b.call()
    assert torch.isfinite(out).all() and (out.abs() <= 40).all()


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("q_scale", [3e2, 1e9, 1e15])
def test_the_only_large_score_takes_it_all(q_scale, f8):
    """One key of the context has a large score and all others a score of zero: the row is that key's
    value, wherever the parts of the work are cut and whatever the score's rounding."""
    for lens, new in (([900, 333], [5, 40]), ([9000], [1]), ([5000], [300])):
        b = Batch(84, lens, new, 12, 2, 128, 16, f8)
        b.q.zero_()
        b.q[:, :, 3] = q_scale
        first, want = 0, []
        for r, (n, m) in enumerate(zip(lens, new)):
            pos = torch.arange(n, device="cuda")
            page = b.table[r].long()[pos // 16]
            k = b.kc.view(torch.uint8) if f8 else b.kc
            k[page, pos % 16] = 0
            k[page[7], 7, :, 3] = 0x7E if f8 else 448.0
            v = b.vc[page[7], 7].view(torch.uint8).view(F8).float() * b.v_scale if f8 else \
                b.vc[page[7], 7].float()
            want.append(v.repeat_interleave(6, 0).bfloat16()[None].expand(m, 12, 128))
        out = b.call()
        seen = [slice(max(0, 7 - (n - m)), m) for n, m in zip(lens, new)]
        for w, s, o in zip(want, seen, out.split(new)):
            assert torch.equal(o[s], w[s])


@pytest.mark.parametrize("at_end", [False, True])
@pytest.mark.parametrize("heads,kv_heads,dim,n,new,requests", [
    (24, 4, 256, 4000, 1, 1), (8, 2, 64, 700, 9, 1), (12, 2, 128, 20000, 2, 1),
    (24, 4, 256, 1500, 1, 40), (12, 2, 128, 3000, 2, 80)])  # one request: parts with maxima of their own
@pytest.mark.parametrize("gap", [6.0, 12.0, 17.0, 20.3, 24.6, 25.2, 28.0])
def test_small_weights_beside_a_sink(gap, heads, kv_heads, dim, n, new, requests, at_end):
    """e4m3: one key whose score is `gap` powers of two above all others and whose value is zero, so
    that the result is what the small weights make of theirs.  Weights are stored as f16 times 2^7
    of the row's reference (a sum of at least 2^7): half the smallest step is 2^-32 of it per key, in
    place of the 2^-25 that the other tests allow."""
    b = Batch(80, [n] * requests, [new] * requests, heads, kv_heads, dim, 32, True)
    pos = torch.arange(n, device="cuda")
    kk, vv = b.kc.view(torch.uint8), b.vc.view(torch.uint8)
    sink, most = n - new if at_end else 0, []
    for r in range(requests):
        page = b.table[r].long()[pos // 32]
        kk[page, pos % 32] = 0
        kk[page[sink], sink % 32, :, 0] = 0x38  # 1.0
        vv[page, pos % 32] &= 0x7F  # (values of one sign: errors of the weights add up)
        vv[page[sink], sink % 32] = 0
        most.append(vv[page, pos % 32].view(F8).double().abs().amax((0, 2)) * b.v_scale)
    b.q.zero_()
    b.q[:, :, 0] = gap * np.log(2) / (b.scale * b.k_scale)
    out = b.call()
    ref, tol = b.reference()
    # (the reference's term is n 2^-25 times the largest value of the row's own request and kv head)
    v = torch.stack(most).repeat_interleave(heads // kv_heads, 1).repeat_interleave(new, 0)[..., None]
    tol = tol - n * 2.0 ** -25 * v + n * 2.0 ** -32 * v
    assert (tol > 0).all()
    assert (ref.abs().amax() > 0) and ((out.double() - ref).abs() <= tol).all(), \
        ((out.double() - ref).abs() / tol).max().item()


@pytest.mark.parametrize("n", [40, 5000])
def test_rows_of_zeros_at_a_tiny_scale(n):
    # e4m3: a row's own power of two times the scale leaves fp32: all scores are zero, not NaN
    b = Batch(81, [n, 33], [3, 33], 12, 2, 128, 16, True)
    b.k_scale = 1e-25
    b.q[0] = 0
    b.q[2] *= 1e-30
    b.q[5:9, 1::2] = 0
    check_attention(b)


@pytest.mark.parametrize("n", [40, 5000])
@pytest.mark.parametrize("v_scale", [3e38, 2e36, 1e-37])
def test_value_scales_of_the_whole_range(v_scale, n):
    # results inside bf16's range, whatever factors the kernel forms on the way
    b = Batch(82, [n, 33], [1, 5], 12, 2, 128, 16, True)
    b.v_scale = v_scale
    vv = b.vc.view(torch.uint8)
    own = vv != 0x7F
    if v_scale > 1:  # values below 2^-3
        vv[own] = vv[own] & 0x9F
    check_attention(b)


@pytest.mark.parametrize("lens,new", [([6001], [600]), ([2200, 700, 4100], [500, 700, 31])])
def test_chunks_with_many_units_per_row_tile(lens, new):
    check_attention(Batch(40, lens, new, 24, 4, 256, 32))


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("heads,kv_heads,dim", [(1, 1, 64), (160, 1, 64), (258, 2, 128), (128, 1, 256)])
def test_head_groups(heads, kv_heads, dim, f8):
    # a group of more than 128 heads is several row tiles of a token
    check_attention(Batch(60, [77, 130, 300, 9], [1, 5, 1, 9], heads, kv_heads, dim, 16, f8))


@pytest.mark.parametrize("f8", [False, True])
def test_more_requests_than_threads(f8):
    rng = np.random.default_rng(12)
    new = [int(x) for x in rng.integers(0, 4, 1300)]
    lens = [n + int(x) for n, x in zip(new, rng.integers(0, 60, 1300))]
    check_attention(Batch(61, lens, new, 4, 2, 64, 16, f8))


@pytest.mark.parametrize("f8", [False, True])
def test_offsets_past_32_bits(f8):
    """Pages whose elements lie past 2^31 (bytes past 2^32): rows written there and read there are
    those of the same pages of a small cache, bit for bit."""
    heads, kv_heads, dim, block, n = 8, 4, 256, 16, 100
    blocks = (2 ** 32 if f8 else 2 ** 31) // (block * kv_heads * dim) + 40
    g = torch.Generator(device="cuda").manual_seed(90)
    k, v = (torch.randn((n, kv_heads, dim), generator=g, device="cuda").bfloat16() for _ in "kv")
    q = torch.randn((9, heads, dim), generator=g, device="cuda").bfloat16()
    pages = torch.randperm(30, generator=g, device="cuda")[:7].to(torch.int32)
    dtype = F8 if f8 else torch.bfloat16
    outs = []
    for first, total in ((0, 40), (blocks - 30, blocks)):
        kc, vc = (torch.empty((total, block, kv_heads, dim), dtype=dtype, device="cuda")
                  for _ in "kv")
        table = (pages + first).view(1, 7)
        pos = torch.arange(n, device="cuda")
        slots = (table[0, pos // block] * block + pos % block).to(torch.int32)
        nv.kv_append(k, v, kc, vc, slots, 0.02, 0.02)
        # (a value that is not finite is read by the kernel itself, not by a copy)
        if f8:
            vc.view(torch.uint8)[int(table[0, 6]), 1, 0, 5] = 0x7F
        else:
            vc[int(table[0, 6]), 1, 0, 5] = float("inf")
        outs.append(nv.paged_attention(q, kc, vc, table, ints([0, 9]), ints([n]), k_scale=0.02,
                                       v_scale=0.02))
        del kc, vc
    a, b = (o.view(torch.int16) for o in outs)
    assert torch.equal(a, b)
    assert not torch.isfinite(outs[0][6:, :2, 5]).any() and torch.isfinite(outs[0][:6]).all()


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("tokens", [1, 4, 5, 20, 37, 54, 56, 57, 60])
def test_batch_with_more_tokens_than_rows(tokens, f8):
    """Plan, append and attend where the per-token outputs end inside a request (or before it): the
    rows that exist are those of the whole batch, at the positions that the plan gives them."""
    heads, kv_heads, dim, block = 12, 2, 128, 16
    g = torch.Generator(device="cuda").manual_seed(70)
    lens, new, blocks = [30, 0, 12], [4, 50, 3], 20
    t, scale = sum(new), 0.02 if f8 else 1.0
    free = torch.randperm(blocks, generator=g, device="cuda").to(torch.int32)
    old = torch.randn((2, sum(lens), kv_heads, dim), generator=g, device="cuda").bfloat16()
    qkv = torch.randn((t, heads + 2 * kv_heads, dim), generator=g, device="cuda").bfloat16()

    def step(rows):
        kc, vc = make_cache(g, blocks, block, kv_heads, dim, f8)
        table = torch.full((3, 6), -1, dtype=torch.int32, device="cuda")
        before = nv.paged_plan(ints([0] * 3), ints(lens), table, free, ints([0]), block, sum(lens))
        nv.kv_append(old[0], old[1], kc, vc, before.slots, scale, scale)
        plan = nv.paged_plan(before.lens, ints(new), table, free, before.head, block, rows)
        x = torch.cat([qkv, qkv[:3]])[:rows]
        nv.kv_append(x[:, heads:heads + kv_heads], x[:, heads + kv_heads:], kc, vc, plan.slots,
                     scale, scale)
        b = Batch.__new__(Batch)
        b.lens, b.new, b.f8, b.dim, b.heads, b.kv_heads = plan.lens.tolist(), new, f8, dim, \
            heads, kv_heads
        b.kc, b.vc, b.k_scale, b.v_scale, b.table = kc, vc, scale, scale, table
        b.q, b.tokens, b.starts, b.scale = x[:, :heads], t, plan.starts, dim ** -0.5
        b.block, b.blocks, b.cols = block, blocks, table.shape[1]
        return b, plan

    whole, want = step(t)
    ref, tol = whole.reference()
    b, plan = step(tokens)
    n = min(tokens, t)
    assert plan.starts.tolist() == want.starts.tolist()
    assert plan.positions[:n].tolist() == want.positions[:n].tolist()
    out = torch.full_like(b.q, 7.0)
    got = b.call(out=out)[:n].double()
    assert torch.isfinite(got).all(), "a row saw a slot that was never written"
    assert ((got - ref[:n]).abs() <= tol[:n]).all()
    assert (out[n:] == 7.0).all()


def test_starts_that_are_not_in_range():
    # rows before 0 and behind `tokens` do not exist; those between keep their positions
    b = Batch(71, [60, 40], [20, 30], 6, 2, 64, 16)
    ref, tol = b.reference()
    b.starts = ints([-8, 12, 42])
    got = b.call(q=b.q[8:40].contiguous())
    assert ((got.double() - ref[8:40]).abs() <= tol[8:40]).all()


def test_rows_behind_the_last_token_stay():
    b = Batch(12, [40, 50], [3, 1], 8, 2, 128, 16, pad=5)
    out = torch.full_like(b.q, 7.0)
    check_attention(b, out=out)
    assert (out[4:] == 7.0).all()


def test_strided_rows():
    b = Batch(13, [90, 33], [4, 2], 6, 2, 128, 16)
    fused = torch.zeros((6, 3, 6, 2, 128), dtype=torch.bfloat16, device="cuda")
    fused[:, 1, :, 0] = b.q
    out = torch.zeros((6, 9, 200), dtype=torch.bfloat16, device="cuda")
    want = b.call()
    got = b.call(q=fused[:, 1, :, 0], out=out[:, 1:7, 8:136])
    assert torch.equal(got, want)
    assert (out[:, 7:] == 0).all() and (out[:, :, :8] == 0).all() and (out[:, :, 136:] == 0).all()


def test_same_result_every_time_and_on_another_stream():
    b = Batch(14, [3000, 5, 1200], [1, 5, 70], 24, 4, 256, 16)
    want = b.call()
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    got = [b.call(stream=other) for _ in range(3)] + [b.call()]
    for o in got:
        assert torch.equal(o, want)


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("tokens", [1, 2])
def test_few_rows_joined_in_the_kernel(tokens, f8):
    # the parts of a tile are joined by the last CTA to leave one, over and over on one workspace
    for k, n in enumerate((3, 130, 517, 4000, 30011)):
        b = Batch(17 + k, [n], [tokens], 12, 2, 128, 16, f8)
        ws = torch.zeros(nv.paged_attention_workspace_bytes(128), dtype=torch.uint8, device="cuda")
        want = check_attention(b, ws=ws)
        for _ in range(5):
            assert torch.equal(b.call(ws=ws, check=False), want)
        torch.cuda.synchronize()
        assert int(ws[:1024].count_nonzero()) == 0
        both = Batch(17 + k, [n] * 9, [tokens] * 9, 12, 2, 128, 16, f8)  # past the rule's limit
        check_attention(both)


def test_captured_call_serves_later_lengths():
    b = Batch(15, [200, 300], [1, 1], 8, 2, 128, 16)
    lens, out = ints([200, 300]), torch.empty_like(b.q)
    call = lambda: nv.paged_attention(b.q, b.kc, b.vc, b.table, b.starts, lens, out=out)
    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for now in ([200, 300], [17, 299], [1, 64]):
        lens.copy_(ints(now))
        out.zero_()
        graph.replay()
        b.lens = now
        ref, tol = b.reference()
        assert ((out.double() - ref).abs() <= tol).all()


def test_error_word_of_captured_calls():
    """Captured calls with a workspace of the caller's: its error word can be asked after the replays, and
    the words that have to be zero are so again behind each call."""
    b = Batch(18, [3000, 700], [1, 9], 12, 2, 128, 16)
    small = Batch(20, [5000], [1], 12, 2, 128, 16)  # (joined in the kernel)
    ws = torch.zeros(nv.paged_attention_workspace_bytes(128), dtype=torch.uint8, device="cuda")
    want, want_small = b.call(), small.call()
    lens, lens_small = ints(b.lens), ints(small.lens)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = [nv.paged_attention(x.q, x.kc, x.vc, x.table, x.starts, n, scale=x.scale, ws=ws)
                for x, n in ((b, lens), (small, lens_small), (b, lens))]
        with pytest.raises(ValueError):
            nv.paged_attention(b.q, b.kc, b.vc, b.table, b.starts, lens, ws=ws, check=True)
    for _ in range(5):
        for o in outs:
            o.zero_()
        graph.replay()
        assert nv.workspace_error(ws) == 0
        assert torch.equal(outs[0], want) and torch.equal(outs[1], want_small)
        assert torch.equal(outs[2], want)
        assert int(ws[:1024].count_nonzero()) == 0
    ws[0] = 7  # what a wait that gave up leaves
    with pytest.raises(RuntimeError):
        b.call(ws=ws)
    assert nv.workspace_error(ws) == 7


# ---------------------------------------------------------------- the cache's rows


@pytest.mark.parametrize("layout", ["nhd", "hnd", "joint"])
@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("tokens,heads,dim,block", [(1, 1, 64, 16), (37, 4, 256, 16),
                                                    (1000, 3, 128, 48), (5001, 2, 64, 16),
                                                    (9600, 5, 128, 32)])
def test_append(tokens, heads, dim, block, f8, layout):
    g = torch.Generator(device="cuda").manual_seed(tokens)
    blocks = -(-tokens // block) + 2
    kc, vc = make_cache(g, blocks, block, heads, dim, f8, layout)
    rows = torch.randn((tokens, 3 * heads * dim + 8), generator=g, device="cuda").mul_(40)
    rows[0, :4] = torch.tensor([float("inf"), -float("inf"), 1e30, 0.0], device="cuda")
    rows = rows.to(torch.bfloat16)
    k = rows[:, :heads * dim].view(tokens, heads, dim)
    v = rows[:, 2 * heads * dim + 8:].view(tokens, heads, dim)
    slots = torch.randperm(blocks * block, generator=g, device="cuda")[:tokens].to(torch.int32)
    if tokens > 8:
        slots[3], slots[5], slots[7] = -1, blocks * block, -2 ** 31  # skipped
    before = [c.clone().view(torch.uint8) for c in (kc, vc)]
    nv.kv_append(k, v, kc, vc, slots, 0.3, 0.7)
    keep = (slots >= 0) & (slots < blocks * block)
    at = slots[keep].long()
    for cache, rows_, scale, old in ((kc, k, 0.3, before[0]), (vc, v, 0.7, before[1])):
        want = old.view(cache.dtype)
        new = rows_[keep]
        if f8:
            scale = torch.tensor(scale, dtype=torch.float32, device="cuda")
            new = (new.float() / scale).clamp(-448, 448).to(F8)
        w = want.view(torch.uint8).view(blocks, block, heads, -1)
        w[at // block, at % block] = new.contiguous().view(torch.uint8).view(len(at), heads, -1)
        got = cache.contiguous().view(torch.uint8).view(blocks, block, heads, -1)
        assert torch.equal(got, w)


def test_append_rounds_the_true_quotient():
    """Values whose quotient lies at a border between two codes, or a place beside it, for scales of
    many magnitudes: the code is that of the fp32 quotient, not of a product with 1 / scale."""
    codes = torch.arange(0x7F, dtype=torch.uint8).view(F8).double()  # every non-negative value
    borders = (codes[1:] + codes[:-1]) / 2
    for scale in (0.3, 1.0, 7.3e-5, 0.0123, 3.0e4, 1e-38, 3e38):
        scale = torch.tensor(scale, dtype=torch.float32)
        x = (borders * scale.double()).to(torch.bfloat16).view(torch.int16)
        x = torch.cat([x - 1, x, x + 1, x | -0x8000]).view(torch.bfloat16)
        x = torch.cat([x, torch.tensor([float("nan"), 448.0, -1e30, 0.0, -0.0, 1e-30, 2.0 ** -9,
                                        2.0 ** -10]).bfloat16()])
        n = -(-len(x) // 64)
        rows = torch.zeros(n * 64, dtype=torch.bfloat16)
        rows[:len(x)] = x
        rows = rows.view(n, 1, 64).cuda()
        kc, vc = (torch.zeros((n, 16, 1, 64), dtype=F8, device="cuda") for _ in range(2))
        nv.kv_append(rows, rows, kc, vc, torch.arange(n, device="cuda", dtype=torch.int32) * 16,
                     float(scale), float(scale))
        q = rows.cpu().float().view(-1) / scale
        want = torch.where(torch.isnan(q), q, q.clamp(-448, 448)).to(F8)
        for c in (kc, vc):
            got = c[:, 0, 0].reshape(-1).cpu()
            same = got.view(torch.uint8) == want.view(torch.uint8)
            assert (same | (torch.isnan(got.float()) & torch.isnan(want.float()))).all()


def test_append_keeps_the_sign_of_zero():
    rows = torch.zeros((3, 2, 64), dtype=torch.bfloat16, device="cuda")
    rows[..., 1::2] = -0.0
    rows[2, :, 8:16] = 1e-30  # (quotients that round to zero, beside values that do not)
    rows[2, :, 16:24] = -1e-30
    rows[2, :, 24] = 1.0
    for scale in (1e-15, 7.3e-5, 0.02, 0.3, 0.7, 1.0, 3.0, 1e15):
        kc, vc = (torch.zeros((1, 16, 2, 64), dtype=F8, device="cuda") for _ in "kv")
        nv.kv_append(rows, -rows, kc, vc, ints([0, 1, 2]), scale, scale)
        for got, x in ((kc, rows), (vc, -rows)):
            want = torch.signbit(x)
            assert torch.equal(got.view(torch.uint8)[0, :3] >= 0x80, want), scale


@pytest.mark.parametrize("tokens", [1024, 5120])
def test_append_saturates_quotients_that_leave_fp32(tokens):
    """Every bf16 value, up to the largest of both signs, at scales whose quotients of large values are
    infinite in fp32: 448 with x's sign, and the fp32 quotient's code below.  (Whole numbers: the codes
    are equal.)  1024 rows are a warp per side each, 5120 a warp per token."""
    x = torch.arange(-2 ** 15, 2 ** 15, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    rows = x.view(1024, 1, 64).repeat(tokens // 1024, 1, 1)
    n = rows.shape[0]
    slots = torch.arange(n, device="cuda", dtype=torch.int32)
    for scale in (1e-16, 1e-15, 1.1e-15, 1e-10, 7.3e-5, 0.02, 0.3, 0.7, 0.9, 1.0, 3.0, 1e5, 9e14, 1e15,
                  1e16, 1e-38, 3e38):
        scale = torch.tensor(scale, dtype=torch.float32)
        kc, vc = (torch.zeros((n // 16, 16, 1, 64), dtype=F8, device="cuda") for _ in range(2))
        nv.kv_append(rows.cuda(), (-rows).cuda(), kc, vc, slots, float(scale), float(scale))
        q = rows.float() / scale
        for got, q in ((kc, q), (vc, -q)):
            got = got.view(n, 1, 64).cpu()
            want = torch.where(torch.isnan(q), q, q.clamp(-448, 448)).to(F8)
            same = got.view(torch.uint8) == want.view(torch.uint8)
            nan = torch.isnan(want.float())
            assert (same | nan).all() and torch.equal(torch.isnan(got.float()), nan), float(scale)


def test_attention_over_keys_and_values_past_the_codes_range():
    # keys and values that saturate are finite to the rows that see them
    b = Batch(19, [90, 70], [1, 3], 12, 2, 128, 16, True)
    b.k_scale = b.v_scale = 0.02
    slots = [int(b.table[r, key // 16]) * 16 + key % 16 for r, key in ((0, 40), (1, 5))]
    k, v = (torch.randn((2, 2, 128), device="cuda").bfloat16() for _ in "kv")
    k[0, :, 3], v[0, :, 9], v[1, :, 100] = 7e36, -3.3e38, 1e37
    nv.kv_append(k, v, b.kc, b.vc, ints(slots), b.k_scale, b.v_scale)
    check_attention(b)


# ---------------------------------------------------------------- the plan


def plan_reference(lens, new, table, free, head, block, tokens):
    """The definition, one request and token after another."""
    lens, new = [max(x, 0) for x in lens], [max(x, 0) for x in new]
    table, cols = table.copy(), table.shape[1]
    starts, slots, request, positions, missing = [0], [], [], [], 0
    for r, (n, m) in enumerate(zip(lens, new)):
        for c in range(-(-n // block), -(-(n + m) // block)):
            if c >= cols:
                missing += 1
                continue
            if head < len(free):
                table[r, c] = free[head]
                head += 1
            else:
                table[r, c] = -1
                missing += 1
        for pos in range(n, n + m):
            page = table[r, pos // block] if pos // block < cols else -1
            slots.append(page * block + pos % block if page >= 0 else -1)
            request.append(r)
            positions.append(pos)
        starts.append(starts[-1] + m)
    more = tokens - len(slots)
    return dict(table=table, starts=starts, lens=[a + b for a, b in zip(lens, new)],
                slots=(slots + [-1] * more)[:tokens], request=(request + [-1] * more)[:tokens],
                positions=(positions + [0] * more)[:tokens], head=[head], missing=[missing])


def check_plan(lens, new, block, cols, n_free, head, tokens, ld=None):
    rng = np.random.default_rng(len(lens) + block)
    table = rng.integers(0, 10 ** 6, (len(lens), ld or cols)).astype(np.int32)
    free = rng.permutation(n_free).astype(np.int32)
    want = plan_reference(lens, new, table[:, :cols], free, head, block, tokens)
    tab = torch.from_numpy(table).cuda()
    p = nv.paged_plan(ints(lens), ints(new), tab[:, :cols], torch.from_numpy(free).cuda(),
                      ints([head]), block, tokens)
    full = table.copy()
    full[:, :cols] = want.pop("table")
    assert np.array_equal(tab.cpu().numpy(), full)
    for name, w in want.items():
        assert getattr(p, name).tolist() == list(w), name


@pytest.mark.parametrize("block", [1, 16, 48, 128])
@pytest.mark.parametrize("requests", [1, 2, 33, 700, 2000])
def test_plan(requests, block):
    rng = np.random.default_rng(requests)
    lens = [int(x) for x in rng.integers(0, 500, requests)]
    new = [int(x) for x in rng.choice([0, 1, 1, 8, 40], requests)]
    pages = sum(-(-(a + b) // block) - -(-a // block) for a, b in zip(lens, new))
    check_plan(lens, new, block, 541, pages + 9, 4, sum(new) + 7)


@pytest.mark.parametrize("requests", [2561, 3050, 3071, nv.MAX_REQUESTS])
def test_plan_of_many_requests(requests):
    rng = np.random.default_rng(requests)
    lens, new = rng.integers(0, 60, requests), rng.integers(0, 3, requests)
    check_plan([int(v) for v in lens], [int(v) for v in new], 16, 5, 4 * requests, 2,
               int(new.sum()) + 9)


def test_plan_runs_out():
    check_plan([10, 0, 30, 16], [10, 50, 3, 1], 16, 3, 4, 2, 70)   # list spent, table too short
    check_plan([10, 0, 30, 16], [10, 50, 3, 1], 16, 9, 2, 2, 64)   # nothing left
    check_plan([10, 0, 30, 16], [10, 50, 3, 1], 16, 9, 2, 9, 64)   # a head past the list
    check_plan([10, 0, 30, 16], [10, 50, 3, 1], 16, 9, 20, 0, 20)  # fewer outputs than tokens
    check_plan([5, -3, 7], [-1, 4, 0], 16, 4, 20, 0, 9, ld=11)     # negative counts as zero
    check_plan([5, 6], [0, 0], 16, 4, 20, 3, 5)                    # nothing new


def test_plan_without_requests():
    e = torch.empty(0, dtype=torch.int32, device="cuda")
    p = nv.paged_plan(e, e, e.view(0, 0), ints([3, 4]), ints([1]), 16, 3)
    assert p.starts.tolist() == [0] and p.slots.tolist() == [-1] * 3
    assert p.head.tolist() == [1] and p.missing.tolist() == [0]


# ---------------------------------------------------------------- together


@pytest.mark.parametrize("f8", [False, True])
def test_steps_of_a_batch_from_empty_tables(f8):
    """Plan, append and attend over several steps, as a serving loop does: a prefill, single
    tokens, verify rounds; the cache grows page by page."""
    heads, kv_heads, dim, block = 12, 2, 128, 16
    g = torch.Generator(device="cuda").manual_seed(21)
    n, blocks = 3, 40
    kc, vc = make_cache(g, blocks, block, kv_heads, dim, f8)
    table = torch.full((n, 12), -1, dtype=torch.int32, device="cuda")
    free = torch.randperm(blocks, generator=g, device="cuda").to(torch.int32)
    lens, head = ints([0] * n), ints([0])
    scale = 0.02 if f8 else 1.0
    for new in ([20, 1, 70], [1, 1, 1], [8, 0, 8], [1, 30, 1]):
        t = sum(new)
        plan = nv.paged_plan(lens, ints(new), table, free, head, block, tokens=t + 2)
        qkv = torch.randn((t + 2, heads + 2 * kv_heads, dim), generator=g, device="cuda").bfloat16()
        nv.kv_append(qkv[:, heads:heads + kv_heads], qkv[:, heads + kv_heads:], kc, vc,
                     plan.slots, scale, scale)
        b = Batch.__new__(Batch)
        b.lens, b.new, b.f8, b.dim, b.heads, b.kv_heads = plan.lens.tolist(), new, f8, dim, \
            heads, kv_heads
        b.kc, b.vc, b.k_scale, b.v_scale, b.table = kc, vc, scale, scale, table
        b.q, b.tokens, b.starts, b.scale = qkv[:, :heads], t, plan.starts, dim ** -0.5
        b.block, b.blocks, b.cols = block, blocks, table.shape[1]
        check_attention(b)
        lens, head = plan.lens, plan.head
        assert plan.missing.item() == 0


@pytest.mark.parametrize("f8", [False, True])
def test_attention_half_of_a_layer_captured(f8):
    """One step of a decode loop as a graph: plan, the q, k, v and gate projections (adapters on q),
    cache rows, attention, the gated output projection.  Replayed over steps, each result is that
    of the calls made one by one, and the attention's that of the plain form."""
    heads, kv_heads, dim, block, k, n = 8, 2, 64, 16, 512, 4
    g = torch.Generator(device="cuda").manual_seed(33)
    W = [dev_weight(synth.nvfp4_weight(70 + i, 0, rows, k)) for i, rows in
         enumerate((heads * dim, kv_heads * dim, kv_heads * dim, heads * dim))]
    wo = dev_weight(synth.nvfp4_weight(75, 0, k, heads * dim))
    rank, adapters = 16, 3
    a = (torch.randn((adapters, rank, k), generator=g, device="cuda") * k ** -0.5).bfloat16()
    b = (torch.randn((adapters, heads * dim, rank), generator=g, device="cuda") * 0.1).bfloat16()
    lora = nv.Lora(a, b, ints([0, 2, -1, 1]), torch.tensor([1.0, 0.5, 2.0], device="cuda"))
    blocks, scale = 24, 0.05 if f8 else 1.0
    kc, vc = make_cache(g, blocks, block, kv_heads, dim, f8)
    table = torch.full((n, 5), -1, dtype=torch.int32, device="cuda")
    free = torch.randperm(blocks, generator=g, device="cuda").to(torch.int32)
    lens, head, new = ints([0] * n), ints([0]), ints([1] * n)
    x = torch.zeros((n, k), dtype=torch.bfloat16, device="cuda")

    def step():
        plan = nv.paged_plan(lens, new, table, free, head, block, tokens=n)
        q, kk, v, gate = nv.gemv_multi(W, x, lora=[lora, None, None, None])
        q = q.view(n, heads, dim)
        nv.kv_append(kk.view(n, kv_heads, dim), v.view(n, kv_heads, dim), kc, vc, plan.slots,
                     scale, scale)
        o = nv.paged_attention(q, kc, vc, table, plan.starts, plan.lens, k_scale=scale,
                               v_scale=scale)
        y = nv.gemv(*wo, o.view(n, -1), prologue=nv.SigmoidGate(gate))
        lens.copy_(plan.lens)
        head.copy_(plan.head)
        return plan, q, o, y

    step()  # (loads the kernels)
    for t in (lens, head):
        t.zero_()
    table.fill_(-1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan, q, o, y = step()
    for i in range(40):
        x.copy_(torch.randn((n, k), generator=g, device="cuda").bfloat16())
        graph.replay()
        assert lens.tolist() == [i + 1] * n and plan.missing.item() == 0
        if i % 13:
            continue
        t = Batch.__new__(Batch)
        t.lens, t.new, t.f8, t.dim, t.heads, t.kv_heads = [i + 1] * n, [1] * n, f8, dim, heads, \
            kv_heads
        t.kc, t.vc, t.k_scale, t.v_scale, t.table = kc, vc, scale, scale, table
        t.q, t.tokens, t.starts, t.scale = q, n, plan.starts, dim ** -0.5
        t.block, t.blocks, t.cols = block, blocks, table.shape[1]
        assert torch.equal(check_attention(t), o)
        q2, _, _, gate = nv.gemv_multi(W, x, lora=[lora, None, None, None])
        assert torch.equal(q2.view_as(q), q)
        assert torch.equal(nv.gemv(*wo, o.view(n, -1), prologue=nv.SigmoidGate(gate)), y)


def test_two_graphs_at_once():
    """Two captured calls replayed on two streams, over and over: each has a workspace of its own."""
    batches = [Batch(50, [5000], [1], 24, 4, 256, 16), Batch(51, [900, 3100], [40, 8], 12, 2, 256, 32)]
    want = [b.call() for b in batches]
    graphs, outs = [], []
    for b in batches:
        lens, out = ints(b.lens), torch.empty_like(b.q)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            nv.paged_attention(b.q, b.kc, b.vc, b.table, b.starts, lens, scale=b.scale, out=out)
        graphs.append((graph, lens))
        outs.append(out)
    streams = [torch.cuda.Stream() for _ in batches]
    torch.cuda.synchronize()
    for _ in range(20):
        for out in outs:
            out.zero_()
        torch.cuda.synchronize()
        for (graph, _), stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        for out, w in zip(outs, want):
            assert torch.equal(out, w)
