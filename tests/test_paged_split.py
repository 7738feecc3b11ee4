"""The paged decode attention's split into ranges: what is joined, and that lengths which change while a call runs (a
caller's mistake in the order of its streams) reach nothing outside the call's buffers.

The ranges' arithmetic is plain integer code that the kernels include; the host compiler builds it here."""
import ctypes
import os
import random
import subprocess

import pytest
import torch

import trainable_block_sparse_pool_b200 as T
from trainable_block_sparse_pool_b200 import build as B

W = 8    # warps a CTA

SOURCE = """
#include "paged_split.cuh"
using namespace infllm2::pattn;
extern "C" {
void describe(int wk, int pair, long long x1, long long rest, long long share, long long total, int ctas, int* out) {
  const Join j = describe_join(wk, pair, x1, rest, share, total, ctas);
  out[0] = j.first; out[1] = j.ctas; out[2] = j.last; out[3] = j.pair;
}
int in_bounds(const int* j, int pairs, int ctas) { return join_in_bounds(Join{j[0], j[1], j[2], j[3]}, pairs, ctas); }
int pieces(const int* j) { return join_pieces(Join{j[0], j[1], j[2], j[3]}); }
int slot(const int* j, int i) { return join_slot(Join{j[0], j[1], j[2], j[3]}, i); }
}
"""


@pytest.fixture(scope="module")
def split(tmp_path_factory):
    at = tmp_path_factory.mktemp("split")
    (at / "split.cpp").write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-fsanitize=signed-integer-overflow",
                    "-fsanitize-undefined-trap-on-error", "-I", B.CSRC, str(at / "split.cpp"), "-o",
                    str(at / "split.so")], check=True)
    return ctypes.CDLL(os.fspath(at / "split.so"))


def _describe(split, wk, pair, x1, rest, share, total, ctas):
    out, ll = (ctypes.c_int * 4)(), ctypes.c_longlong
    split.describe(wk, pair, ll(x1), ll(rest), ll(share), ll(total), ctas, out)
    return out


def _slots(split, j):
    return [split.slot(j, i) for i in range(split.pieces(j))]


def test_slots_of_a_split(split):
    # every worker's pieces by brute force, against what the descriptors name
    rng = random.Random(4)
    for _ in range(300):
        ctas = rng.choice([1, 2, 3, 7, 148])
        costs = [rng.choice([2, 3, 9, 40, 300, 2000]) for _ in range(rng.choice([1, 2, 5, 40]))]
        total = sum(costs)
        share = -(-total // (ctas * W))
        first = [sum(costs[:i]) for i in range(len(costs))]
        got = {p: [] for p in range(len(costs))}      # slots of each pair, in order
        begins = {}
        last = []                                     # of each worker: (pair, from the start, to the end, its only piece)
        for wk in range(ctas * W):
            x0, x1 = min(total, share * wk), min(total, share * wk + share)
            mine = []
            for p, f in enumerate(first):
                lo, hi = max(x0, f), min(x1, f + costs[p])
                t, te = max(lo - f - 1, 0), hi - f - 1
                if lo < hi and t < te:
                    mine.append((p, t == 0, te == costs[p] - 1, te))
            for p, from0, to_end, _ in mine[:-1]:
                assert to_end                         # an earlier piece ends its pair
                if not from0:
                    got[p].append((wk, 2 * wk))
            if mine and mine[-1][1]:
                begins[mine[-1][0]] = (wk, x1, costs[mine[-1][0]] - 1 - mine[-1][3])
            last.append((*mine[-1][:3], len(mine) == 1) if mine else None)
        for c in range(ctas):
            w0 = 0
            while w0 < W:
                w1, head = w0, last[c * W + w0]
                if head:
                    tail = head
                    while w1 + 1 < W and last[c * W + w1 + 1] and last[c * W + w1 + 1][0] == head[0] and last[c * W + w1 + 1][3]:
                        w1 += 1
                        tail = last[c * W + w1]
                    if head[1] and tail[2]:
                        begins.pop(head[0])           # written by its warps
                    else:
                        got[head[0]].append((c * W + w0, 2 * (c * W + w0) + (1 if head[1] else 0)))
                w0 = w1 + 1
        for p, (wk, x1, rest) in begins.items():
            j = _describe(split, wk, p, x1, rest, share, total, ctas)
            assert split.in_bounds(j, len(costs), ctas)
            assert j[3] == p and _slots(split, j) == [s for _, s in sorted(got[p])]
            got.pop(p)
        assert not any(got.values())


def test_lengths_that_disagree_stay_in_bounds(split):
    # the end of a pair comes from a later reading of its length than the total
    rng = random.Random(5)
    for _ in range(20000):
        ctas = rng.choice([1, 2, 148])
        total = rng.choice([1, 5, 1000, 10 ** 6, 1 << 33])
        share = -(-total // (ctas * W))
        wk = rng.randrange(ctas * W)
        if share * wk >= total:
            continue
        x1 = min(total, share * (wk + 1))
        rest = rng.choice([0, 1, rng.randrange(share + 1), rng.randrange(total + 1), (1 << 31) - 1])
        j = _describe(split, wk, 3, x1, rest, share, total, ctas)
        assert split.in_bounds(j, 4, ctas), (wk, x1, rest, share, total, ctas)
        assert all(0 <= s < 2 * ctas * W for s in _slots(split, j))


def test_whatever_the_workspace_holds_stays_in_bounds(split):
    # a descriptor that no warp wrote
    rng = random.Random(6)
    some = [-(1 << 31), -2, -1, 0, 1, 2, 7, 8, 9, 147, 148, 149, 1183, 1184, 1185, (1 << 31) - 1]
    joined = 0
    for _ in range(50000):
        ctas, pairs = rng.choice([1, 2, 148]), rng.choice([1, 8, 1184])
        j = (ctypes.c_int * 4)(*(rng.choice(some) if rng.random() < 0.7 else rng.randrange(-5, 1200) for _ in range(4)))
        if split.in_bounds(j, pairs, ctas):
            joined += 1
            assert 1 <= split.pieces(j) <= ctas + 1 and 0 <= j[3] < pairs
            assert all(0 <= s < 2 * ctas * W for s in _slots(split, j))
    assert joined > 100


@pytest.mark.gpu
@pytest.mark.parametrize("batch,h_q,h_kv,d,page,longest,e4m3", [
    (1, 16, 1, 128, 64, 20000, False), (40, 8, 2, 64, 16, 1500, True), (1500, 2, 1, 64, 16, 80, False),
    (7, 16, 1, 64, 16, 16 * 101, True)])
def test_lengths_that_change_under_the_call(batch, h_q, h_kv, d, page, longest, e4m3):
    g = torch.Generator("cuda").manual_seed(3)
    width = -(-longest // page)
    pages = [torch.randn(64, h_kv, page, d, device="cuda", generator=g).bfloat16() for _ in range(2)]
    scales = [None, None]
    if e4m3:
        pages = [p.to(torch.float8_e4m3fn) for p in pages]
        scales = [torch.ones(64, h_kv, page, device="cuda") for _ in range(2)]
    table = torch.randint(0, 64, (batch, width), device="cuda", generator=g, dtype=torch.int32)
    cache = T.make_paged_cache(*pages, table, *scales)
    q = torch.randn(batch, h_q, d, device="cuda", generator=g).bfloat16()
    need, guard = T.infllm2_paged_workspace_bytes(cache, h_q), 1 << 16

    def guarded(nbytes):
        whole = torch.full((guard + nbytes + guard,), 0xA5, dtype=torch.uint8, device="cuda")
        return whole, whole[guard:guard + nbytes]

    ws_all, ws = guarded(need)
    out_all, out = guarded(batch * h_q * d * 4)
    lse_all, lse = guarded(batch * h_q * 4)
    out, lse = out.view(torch.float32).view(batch, h_q, d), lse.view(torch.float32).view(batch, h_q)
    high = width * page
    lens = [torch.randint(0, high + 1, (batch,), device="cuda", generator=g, dtype=torch.int32) for _ in range(4)]
    lens += [torch.zeros_like(lens[0]), torch.full_like(lens[0], high), torch.full_like(lens[0], high + 9),
             torch.full_like(lens[0], -3)]
    n = lens[0].clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for i in range(200):
        with torch.cuda.stream(side):
            for k in range(3):
                n.copy_(lens[(3 * i + k) % len(lens)])
        T.infllm2_paged_decode_attn(cache, q, n, out, ws, lse)
        if i % 20 == 0:
            ws.fill_(i & 0xFF)      # a descriptor that a call leaves out is not always an older call's
    torch.cuda.synchronize()
    for whole in (ws_all, out_all, lse_all):
        assert (whole[:guard] == 0xA5).all() and (whole[-guard:] == 0xA5).all()
    assert T.infllm2_get_device_status() in (0, -6)
    T.infllm2_clear_device_status()
    # and the next call, with lengths that stay, is right again
    n.copy_(lens[0])
    first = None
    for _ in range(2):
        T.infllm2_paged_decode_attn(cache, q, n, out, ws, lse)
        first = out.clone() if first is None else first
    b = int(lens[0].argmax())
    m = int(lens[0][b])
    x = [p[table[b].long()].float().transpose(0, 1).reshape(h_kv, -1, d)[:, :m].repeat_interleave(h_q // h_kv, 0) for p in pages]
    z = torch.einsum("hd,hnd->hn", q[b].float(), x[0]) / d ** 0.5
    ref = torch.einsum("hn,hnd->hd", z.softmax(-1), x[1])
    # weights in 2^-11 at least and a score's rounding (|z| < 2^8, d + 4 terms of 2^-22): 2^-11 + 2^-7 of the largest value
    assert (out[b] - ref).abs().max() <= x[1].abs().max() * 2.0 ** -6
    assert torch.equal(out, first) and T.infllm2_get_device_status() == 0
