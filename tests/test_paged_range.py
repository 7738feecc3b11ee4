"""The paged decode attention over keys, values and queries of very different sizes, against 64 bits.

Tolerances are those of the ordinary rows: z's fp32 sum of d products, (d + 4) 2^-22 of the largest sum of their
magnitudes, so twice that times ln 2 on a weight; 2^-11 a weight of 8-bit pages; 2^-15 one in two bf16 parts (what its
upper half leaves is below 2^-7, rounded to 2^-8 of that); the fp32 sums, 2^-18 + 2^-22 n / 32; all relative to
sum p |v|, and the output's half step.  A weight so small that its part in 16 bits has fewer than 11 bits is off by 2^-36
of the largest p scale of its head at most, times 448 for a value; n of them: n 2^-27 max(p scale) is added for 8-bit
pages.

A softmax in 32 bits has no weights below 2^-126, fp32's smallest normal number.  A weight is held relative to the largest
of its part (up to 2 of them: the reference is a whole number of log2 units at most 1 above), and a part relative to the
sum, n largest weights at most.  So what has p < 2^-125 n max(p) may vanish, and its p |v| is added: with values that
grow as fast as their weights fall it is not small (2^60 x 2^-140 beside 2^-90)."""
import math

import pytest
import torch

import trainable_block_sparse_pool_b200 as T

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn
PAGE = 16


def _cache(K, V, e4m3):
    """A cache of one sequence that holds the rows K, V [n, h_kv, d] (bf16), and its rows' values and scales."""
    n, h_kv, d = K.shape
    pages = -(-n // PAGE)
    kv = [torch.zeros(pages, h_kv, PAGE, d, device="cuda", dtype=F8 if e4m3 else torch.bfloat16) for _ in range(2)]
    scales = [torch.zeros(pages, h_kv, PAGE, device="cuda") for _ in range(2)] if e4m3 else [None, None]
    table = torch.arange(pages, device="cuda", dtype=torch.int32)[None].contiguous()
    cache = T.make_paged_cache(*kv, table, *scales)
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    T.infllm2_paged_write(cache, K, V, torch.zeros(1, dtype=torch.int32, device="cuda"), cu)
    rows = []
    for x, s in zip(kv, scales):
        x = x.double() if s is None else x.double() * s.double()[..., None]
        rows.append(x.transpose(0, 1).reshape(h_kv, -1, d)[:, :n])
    s = torch.zeros(h_kv, n, device="cuda") if not e4m3 else scales[1].transpose(0, 1).reshape(h_kv, -1)[:, :n]
    return cache, rows[0], rows[1], s.double()


def _attend(cache, q, n, dtype=torch.float32):
    out = torch.empty(q.shape, device="cuda", dtype=dtype)
    lse = torch.empty(q.shape[:2], device="cuda")
    ws = torch.empty(T.infllm2_paged_workspace_bytes(cache, q.shape[1]), dtype=torch.uint8, device="cuda")
    T.infllm2_paged_decode_attn(cache, q, torch.tensor([n], dtype=torch.int32, device="cuda"), out, ws, lse)
    return out[0].double(), lse[0].double()


def _check(K, V, q, e4m3):
    n, h_kv, d = K.shape
    cache, k, v, s = _cache(K, V, e4m3)
    g = q.shape[1] // h_kv
    k, v, s = (x.repeat_interleave(g, 0) for x in (k, v, s))
    x, scale = q[0].double(), 1 / math.sqrt(d)
    z = torch.einsum("hd,hnd->hn", x, k) * scale
    lse = torch.logsumexp(z, -1)
    p = torch.exp(z - lse[:, None])
    ref, mag = torch.einsum("hn,hnd->hd", p, v), torch.einsum("hn,hnd->hd", p, v.abs())
    zmag = torch.einsum("hd,hnd->hn", x.abs(), k.abs()).amax(-1) * scale / math.log(2)
    dz = (d + 4) * 2.0 ** -22 * zmag
    sums = 2.0 ** -22 * n / 32 + 2.0 ** -18
    tol = mag * ((2.0 ** -11 if e4m3 else 2.0 ** -15) + sums + 2 * math.log(2) * dz[:, None])
    tol += ref.abs() * 2.0 ** -24 + n * 2.0 ** -27 * (p * s).amax(-1)[:, None]
    tol += torch.einsum("hn,hnd->hd", torch.where(p < 2.0 ** -125 * n * p.amax(-1, keepdim=True), p, 0.0), v.abs())
    out, got = _attend(cache, q, n)
    assert ((out - ref).abs() <= tol).all(), ((out - ref).abs() / tol).max()
    assert ((got - lse / math.log(2)).abs() <= dz + 2 * sums + 2.0 ** -22 * lse.abs()).all()
    assert T.infllm2_get_device_status() == 0


def _rows(n, h_kv, d, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    return [torch.randn(n, h_kv, d, device="cuda", generator=g) for _ in range(2)]


@pytest.mark.parametrize("e4m3", [True, False])
@pytest.mark.parametrize("h_q,h_kv,d", [(16, 1, 128), (8, 1, 128), (16, 1, 64), (8, 2, 64)])
@pytest.mark.parametrize("n,at", [(50, 0), (50, 49), (2000, 3), (700, 350)])
def test_a_large_value_of_no_weight(h_q, h_kv, d, n, at, e4m3):
    # a value row 2^40 times the others whose key all heads score far below the rest (2^-70 of the weight and less)
    K, V = _rows(n, h_kv, d, 7)
    q = torch.randn(1, h_q, d, device="cuda", generator=torch.Generator("cuda").manual_seed(1)) * 0.25 + 1
    V[at] *= 2.0 ** 40
    K[at] = -6.0 * math.sqrt(128 / d)
    _check(K.bfloat16(), V.bfloat16(), q.bfloat16(), e4m3)


@pytest.mark.parametrize("h_q,d", [(16, 128), (16, 64), (4, 128)])
def test_heads_that_attend_to_values_of_other_sizes(h_q, d):
    # even heads' weight lies on rows 2^30 times smaller than those of the odd heads, in the same tiles
    n = 600
    K, V = _rows(n, 1, d, 9)
    side = torch.arange(n, device="cuda") % 3 == 0
    K *= 0.1
    K[side, 0, 0], K[~side, 0, 0] = 40.0, -40.0
    V[~side] *= 2.0 ** -30
    q = torch.randn(1, h_q, d, device="cuda", generator=torch.Generator("cuda").manual_seed(2))
    q[0, 0::2, 0], q[0, 1::2, 0] = -16.0, 16.0
    _check(K.bfloat16(), V.bfloat16(), q.bfloat16(), True)


@pytest.mark.parametrize("d", [64, 128])
def test_values_that_grow_and_shrink_along_a_sequence(d):
    # the reference rises in steps of up to 2^20, and the last rows are smaller than the first
    n = 1500
    K, V = _rows(n, 1, d, 11)
    e = torch.cat([torch.linspace(-60, 60, 1000), torch.linspace(60, -90, 500)]).round().cuda()
    V *= torch.exp2(e)[:, None, None]
    K[:, 0, 0] = -0.5 * e
    q = torch.randn(1, 16, d, device="cuda", generator=torch.Generator("cuda").manual_seed(3))
    q[0, :, 0] = math.sqrt(d) * torch.linspace(-1, 1.5, 16, device="cuda")
    _check(K.bfloat16(), V.bfloat16(), q.bfloat16(), True)


@pytest.mark.parametrize("size", [-108, -60, 60, 110])
def test_values_of_one_far_size(size):
    K, V = _rows(333, 2, 128, 13)
    V *= 2.0 ** size
    q = torch.randn(1, 8, 128, device="cuda", generator=torch.Generator("cuda").manual_seed(4))
    _check(K.bfloat16(), V.bfloat16(), q.bfloat16(), True)


@pytest.mark.parametrize("h_q,h_kv,d,n", [(16, 1, 128, 1), (16, 1, 128, 3000), (8, 2, 64, 100), (1, 1, 128, 33)])
@pytest.mark.parametrize("same", [True, False])
def test_infinite_values(h_q, h_kv, d, n, same):
    # bf16 pages: a weight above 0 times an infinity is that infinity, in its column alone, whether the weight has
    # 8 bits (equal scores: exactly 1) or more; infinities of both signs are NaN
    K, V = _rows(n, h_kv, d, 15)
    q = torch.randn(1, h_q, d, device="cuda", generator=torch.Generator("cuda").manual_seed(5))
    if same:
        K[:] = 0
    V[n // 2, :, 3], V[n - 1, :, 5], V[n // 3, :, 17], V[0, :, 40] = math.inf, -math.inf, math.inf, -math.inf
    V[0, :, 41] = math.inf
    V[n - 1, :, 41] = -math.inf
    K, V, q = K.bfloat16(), V.bfloat16(), q.bfloat16()
    cache, k, v, _ = _cache(K, V, False)
    g = h_q // h_kv
    k, v = (x.repeat_interleave(g, 0) for x in (k, v))
    p = (torch.einsum("hd,hnd->hn", q[0].double(), k) / math.sqrt(d)).softmax(-1)
    ref = (p[..., None] * v).sum(1)
    assert ref[:, 3].eq(math.inf).all() and (n == 1 or ref[:, 41].isnan().all())
    for dtype in (torch.float32, torch.bfloat16):
        out, lse = _attend(cache, q, n, dtype)
        odd = ~ref.isfinite()
        assert torch.equal(out.isnan(), ref.isnan())
        assert torch.equal(out[odd & ~ref.isnan()], ref[odd & ~ref.isnan()])
        assert lse.isfinite().all()
        assert ((out - ref).abs()[~odd] <= 2.0 ** -7 * v[v.isfinite()].abs().max()).all()


@pytest.mark.parametrize("e4m3", [True, False])
@pytest.mark.parametrize("h_q,d", [(16, 128), (8, 128), (16, 64), (2, 64)])
@pytest.mark.parametrize("q_size,k_size", [(-110, 110), (-98, 100), (-112, 118), (-60, 60), (100, -98), (112, -108)])
def test_scores_of_far_queries_and_keys(q_size, k_size, h_q, d, e4m3):
    # ordinary scores, of factors that are not
    n = 300
    K, V = _rows(n, 1, d, 17)
    q = torch.randn(1, h_q, d, device="cuda", generator=torch.Generator("cuda").manual_seed(6))
    K, q = K * 2.0 ** k_size, q * 2.0 ** q_size
    K[::7] *= 2.0 ** (-40 if k_size > 0 else 0)      # large and ordinary rows side by side
    _check(K.bfloat16(), V.bfloat16(), q.bfloat16(), e4m3)
