"""Rotary positions, the paged key-value cache and its decode attention, against their definitions in 64 bits.

Tolerances.  u = 2^-8 is bf16's half step, 2^-24 fp32's, 2^-4 e4m3's.
  rope       sine and cosine are within 2^-22 of theirs (an angle's 2^-32 turn, the fp32 rounding of the reduced angle
             and of its 2 pi, at most pi/4 x 2^-24 each, the series' evaluation); three fp32 roundings a result:
             (|x1| + |x2|) 2^-21, and the output's own half step.
  cache      bits equal those of the same fp32 operations; a value is half an e4m3 step from x, 2^-4 |x|, or below
             the smallest normal value (2^-6) half a subnormal step, 2^-10 of the scale.
  attention  z's fp32 sum of d products: (d + 4) 2^-22 Z with Z the largest sum of their magnitudes (tensor-core sums
             may truncate: two half steps), so a weight is off by that times ln 2, twice (numerator and sum); its own
             rounding is u^2 (bf16 pages: two bf16 parts) or 2^-11 (f16 weights, 8-bit pages); n additions 2^-22 sqrt(n) typical, bounded
             here by 2^-22 n / 32 + 2^-18; all of it relative to sum p |v|.  Then the output's half step.
"""
import ctypes
import math

import pytest
import torch

import trainable_block_sparse_pool_b200 as T
from trainable_block_sparse_pool_b200 import build as B

F8 = torch.float8_e4m3fn
gpu = pytest.mark.gpu


# ------------------------------------------------------------------ refusals (host)
@pytest.fixture(scope="module")
def L():
    B.build()
    return T.lib()


def _fake_cache(**kw):
    c = T.PagedCache()
    c.k_pages = c.v_pages = c.k_scale = c.v_scale = c.block_table = 0x1000
    c.n_pages, c.page_size, c.batch, c.max_pages, c.h_kv, c.d, c.dtype = 9, 64, 3, 4, 2, 128, T.KV_E4M3
    for k, v in kw.items():
        setattr(c, k, v)
    return c


BAD_CACHES = [
    (dict(k_pages=None), -1), (dict(v_pages=0x1008), -1), (dict(block_table=None), -1), (dict(block_table=0x1002), -1),
    (dict(k_scale=None), -1), (dict(v_scale=0x1004), -1), (dict(dtype=2), -1), (dict(batch=0), -1),
    (dict(batch=65536), -1), (dict(n_pages=0), -1), (dict(max_pages=0), -1), (dict(h_kv=0), -1), (dict(page_size=0), -1),
    (dict(page_size=8), -2), (dict(page_size=48), -2), (dict(page_size=2048), -2), (dict(d=96), -2),
    (dict(page_size=1024, max_pages=1 << 21), -2),
]


@pytest.mark.parametrize("change,code", BAD_CACHES)
def test_bad_caches_are_refused(L, change, code):
    c, by, p = _fake_cache(**change), ctypes.byref, T.default_params()
    assert L.infllm2_paged_write(by(c), 0x1000, 0x1000, 0x1000, 0x1000, 5, None) == code
    assert L.infllm2_paged_read(by(c), 0x1000, 0x1000, 0x1000, 5, None) == code
    if change.get("h_kv") != 0:
        assert L.infllm2_paged_decode_attn(by(c), 0x1000, 32, 0x1000, 0x1000, 0, None, 0x1000, 1 << 40, by(p), None) == code
    assert L.infllm2_paged_workspace_bytes(by(c), 32) == 0


def test_bad_paged_arguments_are_refused(L):
    by, p = ctypes.byref, T.default_params()
    c = _fake_cache()
    w = L.infllm2_paged_write
    assert w(by(c), None, 0x1000, 0x1000, 0x1000, 5, None) == -1
    assert w(by(c), 0x1008, 0x1000, 0x1000, 0x1000, 5, None) == -1
    assert w(by(c), 0x1000, 0x1000, None, 0x1000, 5, None) == -1
    assert w(by(c), 0x1000, 0x1000, 0x1000, 0x1000, -1, None) == -1
    assert w(by(c), 0x1000, 0x1000, 0x1000, None, 5, None) == -1       # one row a sequence: total is batch
    assert w(by(c), 0x1000, 0x1000, 0x1000, 0x1000, 1 << 31, None) == -2
    assert w(None, 0x1000, 0x1000, 0x1000, 0x1000, 5, None) == -1
    assert w(by(c), 0x1000, 0x1000, 0x1000, 0x1000, 0, None) == 0      # nothing to do
    r = L.infllm2_paged_read
    assert r(by(c), 0x1000, 0x1000, None, 5, None) == -1
    assert r(by(c), 0x1000, None, 0x1000, 5, None) == -1
    a = L.infllm2_paged_decode_attn
    need = L.infllm2_paged_workspace_bytes(by(c), 32)
    assert need > 0 and need % 256 == 0
    good = [by(c), 0x1000, 32, 0x1000, 0x1000, 0, None, 0x1000, need, by(p), None]
    for at, bad, code in [(1, None, -1), (1, 0x1008, -1), (2, 33, -1), (2, 64, -2), (2, 6, -2), (3, None, -1),
                          (4, 0x1004, -1), (5, 2, -1), (6, 0x1002, -1), (7, None, -1), (7, 0x1008, -1),
                          (8, need - 1, -3), (9, None, -1)]:
        args = list(good)
        args[at] = bad
        assert a(*args) == code, at
    # bf16 pages need no scales
    assert L.infllm2_paged_workspace_bytes(by(_fake_cache(dtype=T.KV_BF16, k_scale=None, v_scale=None)), 32) == need


def test_bad_rope_arguments_are_refused(L):
    for kw in (dict(rot=0), dict(rot=63), dict(rot=130), dict(rot=64, sections=[16, 17]), dict(rot=64, sections=[40, -8]),
               dict(rot=64, sections=[8] * 5), dict(rot=64, base=0.0), dict(rot=64, base=math.inf),
               dict(rot=64, sections=[]), dict(rot=4, inv_freq=[1.0, math.nan]), dict(rot=4, inv_freq=[1.0])):
        with pytest.raises(T.InfLLM2Error):
            T.make_rope(**kw)
    by, r = ctypes.byref, T.make_rope(128, sections=[16, 24, 24])
    f = L.infllm2_rope
    good = [0x1000, 0x1000, 0, 0x1000, 7, 32, 2, 128, by(r), 0x1000, 0x1000, None]
    for at, bad, code in [(0, None, -1), (1, 0x1008, -1), (2, 2, -1), (3, 0x1001, -1), (4, -1, -1), (4, 1 << 27, -2),
                          (5, 0, -1), (6, 0, -1), (7, 96, -2), (7, 64, -1), (8, None, -1), (9, None, -1),
                          (10, 0x1004, -1)]:
        args = list(good)
        args[at] = bad
        assert f(*args) == code, (at, bad)
        assert L.infllm2_rope_backward(*args) == code, (at, bad)
    broken = T.make_rope(64)
    broken.sections[0] = 31
    assert f(*good[:8], by(broken), *good[9:]) == -1
    assert f(*good[:4], 0, *good[5:]) == 0


def test_binding_refuses_tensors_it_cannot_use(L):
    k = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    table = torch.zeros(2, 2, dtype=torch.int32)
    cache = T.make_paged_cache(k, k, table)
    assert (cache.n_pages, cache.h_kv, cache.page_size, cache.d, cache.batch, cache.max_pages) == (4, 2, 16, 64, 2, 2)
    for args in [(k.float(), k.float(), table), (k, k[:3], table), (k, k, table.long()), (k, k, table[0]),
                 (k.transpose(1, 2), k.transpose(1, 2), table), (k, k, table, torch.zeros(4, 2, 16)),
                 (k.to(F8), k.to(F8), table), (k.to(F8), k.to(F8), table, torch.zeros(4, 2, 16), torch.zeros(4, 2, 8))]:
        with pytest.raises(T.InfLLM2Error):
            T.make_paged_cache(*args)
    row = torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(T.InfLLM2Error):          # not on a GPU
        T.infllm2_paged_write(cache, row, row, torch.zeros(2, dtype=torch.int32))
    with pytest.raises(T.InfLLM2Error):
        T.infllm2_rope(row, row, torch.zeros(1, 2, dtype=torch.int32), T.make_rope(64), row, row)


def test_rope_turns_are_the_frequencies(L):
    # the fixed-point fractions against Python's own 64-bit pow: 2^-53 relative, and 2^-64 of a turn
    r = T.make_rope(96, base=500000.0)
    for i in range(48):
        f = 500000.0 ** (-2 * i / 96) / (2 * math.pi)
        assert abs(r.turns[i] / 2.0 ** 64 - f) <= 4 * 2.0 ** -53 * f + 2.0 ** -63, i
    r = T.make_rope(4, inv_freq=[2 * math.pi * 5, -2 * math.pi * 0.25])
    assert min(r.turns[0], 2 ** 64 - r.turns[0]) < 2 ** 15 and abs(r.turns[1] - 3 * 2 ** 62) < 2 ** 13


# ------------------------------------------------------------------ rope
def _rope64(x, pos, rot, sections, inter, back, base=10000.0):
    half = rot // 2
    axis = torch.repeat_interleave(torch.arange(len(sections)), torch.tensor(sections)).to(x.device)
    freq = base ** (-2.0 * torch.arange(half, dtype=torch.float64, device=x.device) / rot)
    th = pos[axis].t().double() * freq * (-1 if back else 1)
    c, s = th.cos()[:, None], th.sin()[:, None]
    y = x.double()
    e0 = torch.arange(0, rot, 2, device=x.device) if inter else torch.arange(half, device=x.device)
    e1 = e0 + (1 if inter else half)
    x1, x2 = x.double()[..., e0], x.double()[..., e1]
    y[..., e0], y[..., e1] = x1 * c - x2 * s, x2 * c + x1 * s
    mag = torch.zeros_like(y)
    mag[..., e0] = mag[..., e1] = x1.abs() + x2.abs()
    return y, mag


ROPE = [
    (1, 1, 1, 64, 64, [32], False, torch.bfloat16, 8), (16, 32, 2, 128, 128, [64], False, torch.bfloat16, 131072),
    (777, 8, 2, 128, 96, [12, 18, 18], False, torch.bfloat16, 1 << 20),
    (301, 5, 5, 64, 48, [8, 8, 4, 4], True, torch.float32, 4096), (33, 4, 1, 128, 2, [1], True, torch.float32, 100),
    (65, 3, 2, 64, 50, [25, 0], False, torch.bfloat16, 5000), (129, 7, 1, 128, 90, [0, 45], True, torch.bfloat16, 5000),
    (9001, 32, 2, 128, 128, [16, 24, 24], True, torch.bfloat16, 32768),
    (4099, 24, 8, 64, 64, [32], False, torch.float32, (1 << 31) - 1), (9973, 32, 2, 128, 80, [20, 20], True,
                                                                        torch.float32, 32768),
]


@gpu
@pytest.mark.parametrize("total,h_q,h_kv,d,rot,sections,inter,dt,far", ROPE)
@pytest.mark.parametrize("back", [False, True])
def test_rope(total, h_q, h_kv, d, rot, sections, inter, dt, far, back):
    g = torch.Generator("cuda").manual_seed(total)
    q = torch.randn(total, h_q, d, device="cuda", generator=g).to(dt)
    k = torch.randn(total, h_kv, d, device="cuda", generator=g).to(dt)
    pos = torch.randint(-far, far, (len(sections), total), device="cuda", generator=g, dtype=torch.int32)
    r = T.make_rope(rot, sections=sections, interleaved=inter)
    call = T.infllm2_rope_backward if back else T.infllm2_rope
    qo, ko = torch.full_like(q, math.nan), torch.full_like(k, math.nan)
    call(q, k, pos, r, qo, ko)
    # a far position times a frequency is known to 2^-53 in the 64-bit reference
    angle = far * 2.0 ** -51
    for x, y in ((q, qo), (k, ko)):
        ref, mag = _rope64(x, pos, rot, sections, inter, back)
        tol = mag * (2.0 ** -21 + angle) + ref.abs() * (torch.finfo(dt).eps / 2)
        assert ((y.double() - ref).abs() <= tol).all()
        assert torch.equal(y[..., rot:], x[..., rot:])
    call(q, k, pos, r, q, k)      # in place
    assert torch.equal(q, qo) and torch.equal(k, ko)


@gpu
def test_rope_backward_is_the_gradient():
    # the operator is linear: its differences are exact, and <dy, rope(x)> = <rope_backward(dy), x>
    g = torch.Generator("cuda").manual_seed(3)
    r = T.make_rope(96, sections=[16, 16, 16])
    x, dy = (torch.randn(50, 4, 128, device="cuda", generator=g) for _ in range(2))
    k, dk = (torch.randn(50, 2, 128, device="cuda", generator=g) for _ in range(2))
    pos = torch.randint(0, 9000, (3, 50), device="cuda", generator=g, dtype=torch.int32)
    out, kout, gx, gk = (torch.empty_like(t) for t in (x, k, x, k))
    T.infllm2_rope(x, k, pos, r, out, kout)
    T.infllm2_rope_backward(dy, dk, pos, r, gx, gk)
    for a, b, c, e in ((dy, out, gx, x), (dk, kout, gk, k)):
        lhs, rhs = (a.double() * b.double()).sum((1, 2)), (c.double() * e.double()).sum((1, 2))
        size = (a.abs().double() * e.abs().double().flip(-1)).sum((1, 2)) + (a.double() * e.double()).abs().sum((1, 2))
        assert ((lhs - rhs).abs() <= 2.0 ** -17 * size).all()
    # differences along one direction
    x2 = x + dy
    out2 = torch.empty_like(x)
    T.infllm2_rope(x2, k, pos, r, out2, kout)
    moved = torch.empty_like(x)
    T.infllm2_rope(dy, k, pos, r, moved, kout)
    assert (out2.double() - out.double() - moved.double()).abs().max() <= 2.0 ** -18 * 12


# ------------------------------------------------------------------ cache
def _quantise(x):
    x = x.float()
    a = x.abs().amax(-1, keepdim=True).clamp(min=2.0 ** -110)
    top = torch.full_like(a, 448.0)     # by a plain number, torch would multiply with a rounded reciprocal
    return (x * (top / a)).to(F8), (a / top).squeeze(-1)


def _pages(lens, h_kv, d, page, e4m3, seed, spare=3):
    """Pages of random rows (NaN where no sequence has a token), a shuffled table whose unused entries point nowhere,
    and the 64-bit values of every sequence's rows [h_kv, len, d]."""
    gen = torch.Generator("cuda").manual_seed(seed)
    need = [-(-n // page) for n in lens]
    n_pages, width = sum(need) + spare, max(1, max(need))
    order = torch.randperm(n_pages, generator=torch.Generator().manual_seed(seed)).tolist()
    table = torch.full((len(lens), width), -7, dtype=torch.int32)
    pages, scales, used = [], [], torch.zeros(n_pages, page, dtype=torch.bool)
    at = 0
    for b, n in enumerate(lens):
        for j in range(need[b]):
            table[b, j] = order[at]
            used[order[at], :max(0, min(page, n - j * page))] = True
            at += 1
    used = used.cuda()
    for _ in range(2):
        x = torch.randn(n_pages, h_kv, page, d, device="cuda", generator=gen).bfloat16()
        if e4m3:
            y, s = _quantise(x)
            y.view(torch.uint8).masked_fill_(~used[:, None, :, None], 0x7F)
            s.masked_fill_(~used[:, None], math.nan)
            pages.append(y), scales.append(s.contiguous())
        else:
            pages.append(x.masked_fill_(~used[:, None, :, None], math.nan)), scales.append(None)
    return pages, scales, table.cuda()


def _values(pages, scale, table, b, n, page):
    at = table[b, :-(-n // page)].long()
    x = pages.view(torch.uint8)[at].view(pages.dtype).double()
    if scale is not None:
        x = x * scale[at].double()[..., None]
    return x.transpose(0, 1).reshape(pages.shape[1], -1, pages.shape[3])[:, :n]


WRITES = [
    ([1], [0], 1, 64, 16), ([3, 0, 70], [0, 5, 61], 2, 128, 64), ([17, 1, 129, 0, 33], [15, 127, 0, 9, 200], 3, 64, 32),
    ([1000, 2, 333], [7, 4000, 0], 8, 128, 128), ([40] * 50, list(range(50)), 2, 64, 16),
]


@gpu
@pytest.mark.parametrize("news,starts,h_kv,d,page", WRITES)
@pytest.mark.parametrize("e4m3", [False, True])
def test_write_and_read(news, starts, h_kv, d, page, e4m3):
    lens = [s + n for s, n in zip(starts, news)]
    pages, scales, table = _pages(lens, h_kv, d, page, e4m3, 11)
    cache = T.make_paged_cache(*pages, table, *scales)
    total, behind = sum(news), 5
    gen = torch.Generator("cuda").manual_seed(5)
    K, V = (torch.randn(total + behind, h_kv, d, device="cuda", generator=gen).bfloat16() for _ in range(2))
    K *= torch.exp2(torch.randint(-60, 60, (total + behind, h_kv, 1), device="cuda", generator=gen).float()).bfloat16()
    K[0] = 0
    cu = torch.tensor([0, *torch.tensor(news).cumsum(0).tolist()], dtype=torch.int32, device="cuda")
    start = torch.tensor(starts, dtype=torch.int32, device="cuda")
    want = [(p.view(torch.uint8).clone(), None if s is None else s.clone()) for p, s in zip(pages, scales)]
    for (p, s), x in zip(want, (K, V)):
        r = 0
        for b, n in enumerate(news):
            for i in range(n):
                pos = starts[b] + i
                at, slot = int(table[b, pos // page]), pos % page
                if e4m3:
                    y, sc = _quantise(x[r])
                    p[at, :, slot], s[at, :, slot] = y.view(torch.uint8), sc
                else:
                    p[at, :, slot] = x[r].view(torch.uint8)
                r += 1
    T.infllm2_paged_write(cache, K, V, start, cu)
    for (p, s), got, gs in zip(want, pages, scales):
        assert torch.equal(got.view(torch.uint8), p)            # nothing else is touched
        assert s is None or torch.equal(gs.view(torch.int32), s.view(torch.int32))
    # whole sequences back
    full = torch.tensor([0, *torch.tensor(lens).cumsum(0).tolist()], dtype=torch.int32, device="cuda")
    n = sum(lens)
    out = [torch.full((n + behind, h_kv, d), 7.0, device="cuda", dtype=torch.bfloat16) for _ in range(2)]
    T.infllm2_paged_read(cache, *out, full)
    for o, p, s, x in zip(out, pages, scales, (K, V)):
        for b, m in enumerate(lens):
            ref = _values(p, s, table, b, m, page).transpose(0, 1)
            got = o[int(full[b]):int(full[b]) + m]
            assert torch.equal(got, ref.float().bfloat16())      # e4m3 x scale: 28 bits, so fp32 rounds once before bf16
            if e4m3 and news[b]:
                v = x[int(cu[b]):int(cu[b + 1])].double()
                top = v.abs().amax(-1, keepdim=True).clamp(min=2.0 ** -110) / 448
                err = (ref[starts[b]:] - v).abs()
                assert (err <= torch.maximum(v.abs() * 2.0 ** -4, top * 2.0 ** -10) * (1 + 2.0 ** -20)).all()
        assert (o[n:] == 7.0).all()
    assert T.infllm2_get_device_status() == 0


@gpu
@pytest.mark.parametrize("e4m3", [False, True])
def test_write_one_token_a_sequence(e4m3):
    # a padded batch: sequences with a negative start are left out
    lens = [64, 1, 0, 33, 0]
    pages, scales, table = _pages(lens, 2, 64, 32, e4m3, 3)
    cache = T.make_paged_cache(*pages, table, *scales)
    before = [p.view(torch.uint8).clone() for p in pages]
    K, V = (torch.randn(5, 2, 64, device="cuda").bfloat16() for _ in range(2))
    start = torch.tensor([63, 0, -1, 32, -5], dtype=torch.int32, device="cuda")
    T.infllm2_paged_write(cache, K, V, start)
    for p, s, x, was in zip(pages, scales, (K, V), before):
        for b, pos in ((0, 63), (1, 0), (3, 32)):
            at, slot = int(table[b, pos // 32]), pos % 32
            if e4m3:
                y, sc = _quantise(x[b])
                assert torch.equal(p[at, :, slot].view(torch.uint8), y.view(torch.uint8))
                assert torch.equal(s[at, :, slot], sc)
            else:
                assert torch.equal(p[at, :, slot], x[b])
            was[at, :, slot] = p.view(torch.uint8)[at, :, slot]
        assert torch.equal(p.view(torch.uint8), was)
    assert T.infllm2_get_device_status() == 0


@gpu
def test_rows_with_infinities_read_back_as_nan():
    pages, scales, table = _pages([16], 1, 64, 16, True, 1)
    cache = T.make_paged_cache(*pages, table, *scales)
    K = torch.randn(16, 1, 64, device="cuda").bfloat16()
    K[3, 0, 7], K[5, 0, 9], K[6] = math.inf, math.nan, 0.0
    K[7] = 3.3895e38       # bf16's largest
    cu = torch.tensor([0, 16], dtype=torch.int32, device="cuda")
    T.infllm2_paged_write(cache, K, K, torch.zeros(1, dtype=torch.int32, device="cuda"), cu)
    out = torch.empty_like(K)
    T.infllm2_paged_read(cache, out, torch.empty_like(K), cu)
    assert out[3].isnan().all() and out[5].isnan().all()
    assert (out[6] == 0).all() and torch.equal(out[7], K[7]) and not out[[0, 1, 2, 4, *range(6, 16)]].isnan().any()


@gpu
@pytest.mark.parametrize("e4m3", [False, True])
def test_pages_out_of_range_are_skipped_and_recorded(e4m3):
    pages, scales, table = _pages([64, 64], 2, 64, 16, e4m3, 9)
    table[0, 2], table[1, 3] = pages[0].shape[0], -1
    cache = T.make_paged_cache(*pages, table, *scales)
    before = [p.view(torch.uint8).clone() for p in pages]
    cu = torch.tensor([0, 3, 6], dtype=torch.int32, device="cuda")
    x = torch.randn(6, 2, 64, device="cuda").bfloat16()
    # positions 40 .. 42 (a bad page) and 64 .. 66 (past the table)
    T.infllm2_paged_write(cache, x, x, torch.tensor([40, 64], dtype=torch.int32, device="cuda"), cu)
    assert T.infllm2_get_device_status() == -6
    assert all(torch.equal(p.view(torch.uint8), b) for p, b in zip(pages, before))
    T.infllm2_clear_device_status()
    full = torch.tensor([0, 64, 128], dtype=torch.int32, device="cuda")
    out = [torch.full((128, 2, 64), 7.0, device="cuda", dtype=torch.bfloat16) for _ in range(2)]
    T.infllm2_paged_read(cache, *out, full)
    assert T.infllm2_get_device_status() == -6
    for o in out:
        assert (o[32:48] == 7.0).all() and (o[64 + 48:] == 7.0).all()
    T.infllm2_clear_device_status()
    # attention: the rows of a bad page count as zeros; a length past the table counts as 0
    q = torch.randn(2, 4, 64, device="cuda").bfloat16()
    o = torch.empty(2, 4, 64, device="cuda")
    ws = torch.empty(T.infllm2_paged_workspace_bytes(cache, 4), dtype=torch.uint8, device="cuda")
    T.infllm2_paged_decode_attn(cache, q, torch.tensor([64, 65], dtype=torch.int32, device="cuda"), o, ws)
    assert T.infllm2_get_device_status() == -6
    assert o[0].isfinite().all() and (o[1] == 0).all()
    T.infllm2_clear_device_status()
    T.infllm2_paged_decode_attn(cache, q, torch.tensor([32, -1], dtype=torch.int32, device="cuda"), o, ws)
    assert T.infllm2_get_device_status() == -6 and (o[1] == 0).all()


# ------------------------------------------------------------------ attention
def _reference(q, pages, scales, table, lens, page, scale):
    """out, lse and the bounds that tolerances are made of, in 64 bits."""
    batch, h_q, d = q.shape
    h_kv = pages[0].shape[1]
    out = torch.zeros(batch, h_q, d, dtype=torch.float64, device="cuda")
    lse = torch.full((batch, h_q), -math.inf, dtype=torch.float64, device="cuda")
    mag, zmag = torch.zeros_like(out), torch.zeros_like(lse)
    for b, n in enumerate(lens):
        if n == 0:
            continue
        k, v = (_values(p, s, table, b, n, page).repeat_interleave(h_q // h_kv, 0) for p, s in zip(pages, scales))
        x = q[b].double()
        z = torch.einsum("hd,hnd->hn", x, k) * scale
        zmag[b] = torch.einsum("hd,hnd->hn", x.abs(), k.abs()).amax(-1) * scale / math.log(2)
        m = torch.logsumexp(z, -1)
        p = torch.exp(z - m[:, None])
        out[b], mag[b], lse[b] = p.unsqueeze(1).matmul(v)[:, 0], p.unsqueeze(1).matmul(v.abs())[:, 0], m / math.log(2)
    return out, lse, mag, zmag


def _check(out, lse, ref, d, n, e4m3):
    r_out, r_lse, mag, zmag = ref
    weight = 2.0 ** -11 if e4m3 else 2.0 ** -16
    dz = (d + 4) * 2.0 ** -22 * zmag
    sums = 2.0 ** -22 * n / 32 + 2.0 ** -18
    tol = mag * (weight + sums + 2 * math.log(2) * dz[..., None]) + r_out.abs() * (torch.finfo(out.dtype).eps / 2)
    assert ((out.double() - r_out).abs() <= tol).all(), ((out.double() - r_out).abs() / tol.clamp(min=1e-30)).max()
    if lse is not None:
        empty = r_lse == -math.inf
        assert torch.equal(lse == -math.inf, empty)
        assert ((lse.double() - r_lse).abs() <= dz + sums * 2 + 2.0 ** -22 * r_lse.abs())[~empty].all()


ATTN = [
    ([1], 1, 1, 64, 16), ([0], 2, 2, 128, 64), ([0, 1, 0, 17, 0], 4, 2, 128, 16),
    ([15, 16, 17, 63, 64, 65, 127, 128, 129], 16, 1, 128, 32), ([15, 16, 17, 63, 64, 65, 127, 128, 129], 8, 4, 64, 64),
    ([1000], 32, 2, 128, 64), ([40000], 16, 1, 128, 128), ([30000, 1], 8, 1, 64, 1024), ([5000, 3, 0, 777], 32, 2, 128, 64),
    ([i * 7 % 90 for i in range(310)], 8, 8, 64, 16), ([i * 13 % 200 for i in range(160)], 32, 8, 128, 32),
    ([300] * 149, 1, 1, 128, 16),
]


@gpu
@pytest.mark.parametrize("lens,h_q,h_kv,d,page", ATTN)
@pytest.mark.parametrize("e4m3", [False, True])
def test_decode_attention(lens, h_q, h_kv, d, page, e4m3):
    pages, scales, table = _pages(lens, h_kv, d, page, e4m3, 21)
    cache = T.make_paged_cache(*pages, table, *scales)
    g = torch.Generator("cuda").manual_seed(8)
    q = torch.randn(len(lens), h_q, d, device="cuda", generator=g).bfloat16()
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    ws = torch.full((T.infllm2_paged_workspace_bytes(cache, h_q),), 0xFF, dtype=torch.uint8, device="cuda")
    ref = _reference(q, pages, scales, table, lens, page, 1 / math.sqrt(d))
    out, lse = torch.full_like(q, math.nan), torch.full((len(lens), h_q), math.nan, device="cuda")
    T.infllm2_paged_decode_attn(cache, q, n, out, ws, lse)
    _check(out, lse, ref, d, max(lens), e4m3)
    f32, lse2 = torch.full_like(q, math.nan, dtype=torch.float32), torch.empty_like(lse)
    T.infllm2_paged_decode_attn(cache, q, n, f32, ws, lse2)
    _check(f32, lse2, ref, d, max(lens), e4m3)
    assert torch.equal(lse, lse2) and torch.equal(f32.bfloat16(), out)      # the same result every time
    ref = _reference(q, pages, scales, table, lens, page, 0.5)
    T.infllm2_paged_decode_attn(cache, q, n, f32, ws, params=T.default_params(scale=0.5))
    _check(f32, None, ref, d, max(lens), e4m3)
    assert T.infllm2_get_device_status() == 0


@gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("e4m3", [False, True])
def test_decode_attention_with_uneven_rows(d, e4m3):
    # queries and rows over many magnitudes, all-zero rows, one row that takes all the weight
    lens, page, h_q, h_kv = [700, 90], 32, 8, 2
    pages, scales, table = _pages(lens, h_kv, d, page, e4m3, 31)
    g = torch.Generator("cuda").manual_seed(2)
    total = sum(lens)
    K, V = (torch.randn(total, h_kv, d, device="cuda", generator=g) for _ in range(2))
    V *= torch.exp2(torch.randint(-9, 10, (total, h_kv, 1), device="cuda", generator=g).float())
    K[5], V[11], V[12] = 0, 0, 0
    cu = torch.tensor([0, 700, 790], dtype=torch.int32, device="cuda")
    cache = T.make_paged_cache(*pages, table, *scales)
    T.infllm2_paged_write(cache, K.bfloat16(), V.bfloat16(), torch.zeros(2, dtype=torch.int32, device="cuda"), cu)
    q = torch.randn(2, h_q, d, device="cuda", generator=g)
    q[0] *= torch.exp2(torch.arange(-6, 2, device="cuda").float())[:, None]
    q[1, 0], q[1, 1, 1:] = 0, 0
    q[1, 2] = 3 * K[700 + 40, 0]
    q = q.bfloat16()
    out, lse = torch.empty(2, h_q, d, device="cuda"), torch.empty(2, h_q, device="cuda")
    ws = torch.empty(T.infllm2_paged_workspace_bytes(cache, h_q), dtype=torch.uint8, device="cuda")
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    T.infllm2_paged_decode_attn(cache, q, n, out, ws, lse)
    _check(out, lse, _reference(q, pages, scales, table, lens, page, 1 / math.sqrt(d)), d, 700, e4m3)


@gpu
def test_many_short_sequences_and_shared_pages():
    # more sequences than a CTA has threads; pages that several sequences share, at several lengths
    page, h_q, h_kv, d = 16, 4, 2, 64
    pages, scales, _ = _pages([4096], h_kv, d, page, False, 17)
    g = torch.Generator().manual_seed(6)
    lens = torch.randint(0, 49, (3000,), generator=g).tolist()
    table = torch.randint(0, 256, (3000, 3), generator=g, dtype=torch.int32).cuda()
    pages = [p.nan_to_num(0.25) for p in pages]
    cache = T.make_paged_cache(*pages, table)
    q = torch.randn(3000, h_q, d, device="cuda").bfloat16()
    out, lse = torch.empty(3000, h_q, d, device="cuda"), torch.empty(3000, h_q, device="cuda")
    ws = torch.empty(T.infllm2_paged_workspace_bytes(cache, h_q), dtype=torch.uint8, device="cuda")
    T.infllm2_paged_decode_attn(cache, q, torch.tensor(lens, dtype=torch.int32, device="cuda"), out, ws, lse)
    # all sequences at once: [batch, h_kv, 48, d]
    k, v = (p[table.long()].double().transpose(1, 2).reshape(3000, h_kv, 48, d).repeat_interleave(2, 1) for p in pages)
    n = torch.tensor(lens, device="cuda")
    z = (q.double()[:, :, None] @ k.transpose(2, 3))[:, :, 0] / 8
    z = z.masked_fill(torch.arange(48, device="cuda") >= n[:, None, None], -math.inf)
    m = torch.logsumexp(z, -1)
    p = torch.exp(z - m.clamp(min=-1e300)[..., None])
    mag = (q.double().abs()[:, :, None] @ k.abs().transpose(2, 3))[:, :, 0].amax(-1) / 8 / math.log(2)
    _check(out, lse, ((p[:, :, None] @ v)[:, :, 0], m / math.log(2), (p[:, :, None] @ v.abs())[:, :, 0], mag), d, 48, False)


@gpu
def test_calls_on_a_given_stream_and_with_no_tokens():
    pages, scales, table = _pages([100, 30], 2, 64, 16, True, 2)
    cache = T.make_paged_cache(*pages, table, *scales)
    q = torch.randn(2, 4, 64, device="cuda").bfloat16()
    n = torch.tensor([100, 30], dtype=torch.int32, device="cuda")
    outs = [torch.empty(2, 4, 64, device="cuda") for _ in range(2)]
    wss = [torch.empty(T.infllm2_paged_workspace_bytes(cache, 4), dtype=torch.uint8, device="cuda") for _ in range(2)]
    K = torch.randn(130, 2, 64, device="cuda").bfloat16()
    got, cu = torch.empty_like(K), torch.tensor([0, 100, 130], dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    T.infllm2_paged_write(cache, K, K, torch.zeros_like(n), cu, stream=side)
    T.infllm2_paged_read(cache, got, torch.empty_like(K), cu, stream=side)
    T.infllm2_paged_decode_attn(cache, q, n, outs[0], wss[0], stream=side)
    side.synchronize()
    T.infllm2_paged_decode_attn(cache, q, n, outs[1], wss[1], stream=side.cuda_stream)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[1])
    assert ((got.double() - K.double()).abs() <= K.double().abs() * 2.0 ** -3 + 2.0 ** -8).all()
    # nothing to write, read or turn
    none, zero = K[:0], torch.zeros(3, dtype=torch.int32, device="cuda")
    T.infllm2_paged_write(cache, none, none, torch.zeros_like(n), zero)
    T.infllm2_paged_read(cache, none, none, zero)
    T.infllm2_rope(none, none, torch.zeros(1, 0, dtype=torch.int32, device="cuda"), T.make_rope(64), none, none)
    # a tensor that starts off a 16-byte boundary, on another device, of another type
    odd = torch.empty(2 * 4 * 64 + 1, device="cuda", dtype=torch.bfloat16)[1:].view(2, 4, 64)
    for bad in (odd, q.cpu(), q.float(), q[:, :3]):
        with pytest.raises(T.InfLLM2Error):
            T.infllm2_paged_decode_attn(cache, bad, n, outs[0], wss[0])
    with pytest.raises(T.InfLLM2Error):
        T.infllm2_paged_decode_attn(cache, q, n, outs[0], wss[0][:-16])
    torch.cuda.synchronize()
    assert T.infllm2_get_device_status() == 0


@gpu
def test_infinite_scores_and_nan_rows():
    pages, scales, table = _pages([40, 40, 33], 1, 64, 16, False, 4)
    k, v = pages
    k[table[0, :2].long()] = -math.inf            # positions 0 .. 31 of sequence 0: score -inf
    k[table[1].long()] = -math.inf                # every position of sequence 1
    v[int(table[2, 1]), 0, 3] = math.nan
    q = torch.ones(3, 2, 64, device="cuda").bfloat16()
    cache = T.make_paged_cache(k, v, table)
    out, lse = torch.empty(3, 2, 64, device="cuda"), torch.empty(3, 2, device="cuda")
    ws = torch.empty(T.infllm2_paged_workspace_bytes(cache, 2), dtype=torch.uint8, device="cuda")
    T.infllm2_paged_decode_attn(cache, q, torch.tensor([40, 40, 33], dtype=torch.int32, device="cuda"), out, ws, lse)
    rows = v[int(table[0, 2]), 0, :8].double()
    z = k[int(table[0, 2]), 0, :8].double().sum(-1) / 8
    ref = torch.softmax(z, 0) @ rows
    assert ((out[0].double() - ref).abs() <= 2.0 ** -7 * rows.abs().max()).all()
    assert (out[1] == 0).all() and (lse[1] == -math.inf).all()
    assert out[2].isnan().all() and lse[2].isfinite().all()


@gpu
@pytest.mark.parametrize("e4m3", [False, True])
def test_captured_step_follows_its_inputs(e4m3):
    # rope, write and attention in one graph, replayed while lengths grow; a second graph with its own workspace
    # on another stream
    h_q, h_kv, d, page, batch = 8, 2, 64, 16, 3
    lens = [40, 0, 100]
    room = [n + 8 for n in lens]
    pages, scales, table = _pages(room, h_kv, d, page, e4m3, 6)
    cache = T.make_paged_cache(*pages, table, *scales)
    g = torch.Generator("cuda").manual_seed(1)
    cu = torch.tensor([0, 40, 40, 140], dtype=torch.int32, device="cuda")
    K, V = (torch.randn(140, h_kv, d, device="cuda", generator=g).bfloat16() for _ in range(2))
    T.infllm2_paged_write(cache, K, V, torch.zeros(3, dtype=torch.int32, device="cuda"), cu)
    rope = T.make_rope(d)
    pos = torch.tensor(lens, dtype=torch.int32, device="cuda")
    n = pos + 1
    q, k, v = (torch.empty(batch, h, d, device="cuda", dtype=torch.bfloat16) for h in (h_q, h_kv, h_kv))
    qr, kr = torch.empty_like(q), torch.empty_like(k)
    size = T.infllm2_paged_workspace_bytes(cache, h_q)
    outs = [torch.empty(batch, h_q, d, device="cuda") for _ in range(2)]
    wss = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    one, two = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(one):
        T.infllm2_rope(q, k, pos, rope, qr, kr)
        T.infllm2_paged_write(cache, kr, v, pos)
        T.infllm2_paged_decode_attn(cache, qr, n, outs[0], wss[0])
    with torch.cuda.graph(two):
        T.infllm2_paged_decode_attn(cache, qr, n, outs[1], wss[1])
    for step in range(8):
        for x in (q, k, v):
            x.copy_(torch.randn(x.shape, device="cuda", generator=g))
        one.replay()
        torch.cuda.synchronize()
        with torch.cuda.stream(torch.cuda.Stream()):
            two.replay()
        one.replay()          # the same rows again: beside the other graph
        torch.cuda.synchronize()
        now = [m + step + 1 for m in lens]
        ref = _reference(qr, pages, scales, table, now, page, 1 / math.sqrt(d))
        for o in outs:
            _check(o, None, ref, d, 200, e4m3)
        assert torch.equal(outs[0], outs[1])
        pos += 1
        n += 1
    assert T.infllm2_get_device_status() == 0


@gpu
def test_offsets_past_32_bits():
    # a cache of more than 2^32 bytes: the last pages
    page, d, n_pages = 1024, 128, (1 << 32) // (1024 * 256) + 9
    k = torch.zeros(n_pages, 1, page, d, device="cuda", dtype=torch.bfloat16)
    v = torch.zeros_like(k)
    table = torch.tensor([[n_pages - 1, n_pages - 2]], dtype=torch.int32, device="cuda")
    cache = T.make_paged_cache(k, v, table)
    K, V = (torch.randn(1500, 1, d, device="cuda").bfloat16() for _ in range(2))
    cu = torch.tensor([0, 1500], dtype=torch.int32, device="cuda")
    T.infllm2_paged_write(cache, K, V, torch.zeros(1, dtype=torch.int32, device="cuda"), cu)
    assert torch.equal(k[n_pages - 1, 0], K[:1024, 0]) and torch.equal(v[n_pages - 2, 0, :476], V[1024:, 0])
    back = [torch.empty_like(K), torch.empty_like(V)]
    T.infllm2_paged_read(cache, *back, cu)
    assert torch.equal(back[0], K) and torch.equal(back[1], V)
    q = torch.randn(1, 16, d, device="cuda").bfloat16()
    out = torch.empty(1, 16, d, device="cuda")
    ws = torch.empty(T.infllm2_paged_workspace_bytes(cache, 16), dtype=torch.uint8, device="cuda")
    T.infllm2_paged_decode_attn(cache, q, torch.tensor([1500], dtype=torch.int32, device="cuda"), out, ws)
    ref = _reference(q, [k, v], [None, None], table, [1500], page, 1 / math.sqrt(d))
    _check(out, None, ref, d, 1500, False)


# ------------------------------------------------------------------ together, with the rest of the library
@gpu
def test_prefix_and_decode_beside_the_library():
    """A prompt's rotated keys go into pages and come back; the dense prefill's last row, the paged decode of the same
    token and the sparse decode step with every block selected are one attention."""
    h_q, h_kv, d, page = 32, 2, 128, 64
    lens = [1000, 129]
    total, batch = sum(lens), len(lens)
    g = torch.Generator("cuda").manual_seed(12)
    q = torch.randn(total, h_q, d, device="cuda", generator=g).bfloat16()
    k, v = (torch.randn(total, h_kv, d, device="cuda", generator=g).bfloat16() for _ in range(2))
    cu = torch.tensor([0, 1000, 1129], dtype=torch.int32, device="cuda")
    pos = torch.cat([torch.arange(n) for n in lens]).to("cuda", torch.int32)
    T.infllm2_rope(q, k, pos, T.make_rope(d), q, k)
    table = torch.randperm(19, generator=torch.Generator().manual_seed(0)).to(torch.int32)[:18].view(2, 9).cuda()
    table = torch.cat([table, torch.arange(19, 19 + 14, device="cuda", dtype=torch.int32).view(2, 7)], 1)
    kp, vp = (torch.full((33, h_kv, page, d), math.nan, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    cache = T.make_paged_cache(kp, vp, table.contiguous())
    T.infllm2_paged_write(cache, k, v, torch.zeros(2, dtype=torch.int32, device="cuda"), cu)
    k2, v2 = torch.empty_like(k), torch.empty_like(v)
    T.infllm2_paged_read(cache, k2, v2, cu)
    assert torch.equal(k2, k) and torch.equal(v2, v)
    # dense prefill over what came back; its last rows against the paged decode
    p = T.default_params(n_local=16, top_k=2)
    vl = T.make_varlen(lens, cu, p)
    dense = torch.empty(total, h_q, d, device="cuda")
    T.infllm2_dense_attn(q, k2, v2, vl, dense, p)
    last = (cu[1:] - 1).long()
    out = torch.empty(batch, h_q, d, device="cuda")
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    ws = torch.empty(T.infllm2_paged_workspace_bytes(cache, h_q), dtype=torch.uint8, device="cuda")
    T.infllm2_paged_decode_attn(cache, q[last].contiguous(), n, out, ws)
    # the other two round their weights to bf16
    size = v.abs().max().item() * 2.0 ** -7
    assert (out - dense[last]).abs().max().item() <= size
    # the hand-over to the sparse decode step: every block is selected, so it is the same attention
    cap = 1024
    kc, vc = (torch.zeros(batch, cap, h_kv, d, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    for b in range(batch):      # all but the last token, then the step appends it
        row = T.make_paged_cache(kp, vp, table[b:b + 1].contiguous())
        T.infllm2_paged_read(row, kc[b], vc[b], torch.tensor([0, lens[b] - 1], dtype=torch.int32, device="cuda"))
    c1 = torch.empty(batch, h_kv, T.window_count(cap, 32, 16), d, device="cuda", dtype=torch.bfloat16)
    c2 = torch.empty(batch, h_kv, T.window_count(cap, 128, 64), d, device="cuda", dtype=torch.bfloat16)
    st = T.make_decode_state(kc, vc, c1, c2, n - 1, h_q)
    T.infllm2_decode_build_caches(st, p)
    dws = torch.empty(T.infllm2_decode_workspace_bytes(st, p), dtype=torch.uint8, device="cuda")
    sparse = torch.empty(batch, h_q, d, device="cuda", dtype=torch.bfloat16)
    T.infllm2_decode_step(st, q[last].contiguous(), k[last].contiguous(), v[last].contiguous(), sparse, dws, p)
    assert (out - sparse.float()).abs().max().item() <= size + sparse.float().abs().max().item() * 2.0 ** -8
    assert T.infllm2_get_device_status() == 0
