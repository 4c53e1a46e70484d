"""Per-head norms with rotation, the paged cache, its decode and its page selection
against the fp64 oracle.

Tolerances.  A rounding to bf16 is off by at most 2^-8 of the value, to fp32 by 2^-24.
Norm and rotation run in fp32: the sum of d <= 128 squares is off by at most 2^-17
relative, half of that after the square root, the other steps by a few 2^-24, the sine
and cosine of a turn's fraction by 2^-22 (for bf16 rows by 2^-21): together below 2^-16 of |a| + |b| of the
pair.  The decode's softmax weights are allowed a rounding to bf16 (2^-8 of the weighted
|v|; test_decode_weights_keep_their_low_bits holds them to 2^-16); a logit is off by at most 18 * 2^-23 a tensor-core step of the sum of |q k| (the bound
the FASA scores are held to), which scales a weight by as much, twice (numerator and
sum); exponentials and sums add less than 2^-16.
"""
import math

import numpy as np
import pytest
import torch

import oracle
from oracle import paged
from rope_frequency_sparse_b200 import atf, synth

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def _normal(seed, *shape, dtype=BF16, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(dtype).cuda()


def _tables(lens, page, seed, spare=2, extra=0):
    """(page_table [B][most + extra] int32, pages in the pool): pages in no order, -1 where none."""
    counts = [-(-max(0, n) // page) for n in lens]
    order = np.random.RandomState(seed).permutation(sum(counts) + spare)
    table = np.full((len(lens), max(1, max(counts)) + extra), -1, dtype=np.int32)
    at = 0
    for b, c in enumerate(counts):
        table[b, :c] = order[at: at + c]
        at += c
    return torch.from_numpy(table).cuda(), sum(counts) + spare


def _pool(pool, hkv, d, page, seed):
    return _normal(seed, pool, hkv, d // 16, page, 16), _normal(seed + 1, pool, hkv, page, d)


def _axes(d, n):
    return [i * n // (d // 2) for i in range(d // 2)]


def _int32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _within(got, want, tol):
    err = np.abs(paged.f64(got) - want)
    assert (err <= tol).all(), (err - tol).max()


# ------------------------------------------------------------------ norms and rotation

@pytest.mark.parametrize("T,Hq,Hkv,d,dtype,pairing,axes,norm", [
    (1, 28, 4, 128, BF16, 1, 1, True), (37, 5, 1, 64, BF16, 0, 1, True), (300, 28, 4, 128, BF16, 0, 3, True),
    (131, 3, 3, 128, torch.float32, 1, 2, True), (64, 1, 1, 64, torch.float32, 0, 4, False),
    (1000, 14, 2, 64, BF16, 1, 1, False), (7, 33, 11, 128, BF16, 1, 1, True)])
def test_norm_rope_against_oracle(T, Hq, Hkv, d, dtype, pairing, axes, norm):
    theta, eps = 1e7, 1e-6
    fused = _normal(1, T, (Hq + 2 * Hkv) * d, dtype=dtype, std=3.0)  # one projection row per token
    fused[T // 2] = 0  # a row without a norm
    q, k = fused[:, :Hq * d].view(T, Hq, d), fused[:, Hq * d:(Hq + Hkv) * d].view(T, Hkv, d)
    pos = torch.randint(0, 1 << 20, (axes, T), generator=torch.Generator().manual_seed(2)).cuda()
    pos[:, 0] = 0
    pos[:, -1] = 2 ** 31 - 1
    wq, wk = (1 + _normal(s, d, dtype=dtype, std=0.2) if norm else None for s in (3, 4))
    got = atf.qk_norm_rope(q, k, theta, pos, wq, wk, eps, _axes(d, axes), pairing)
    atf.atf_check()
    half = 2.0 ** -8 if dtype == BF16 else 2.0 ** -24
    for x, w, y in zip((q, k), (wq, wk), got):
        want, size = paged.norm_rope(paged.f64(x), None if w is None else paged.f64(w), eps, pos.cpu().numpy(),
                                     _axes(d, axes), theta, pairing)
        # positions near 2^31 turn by up to 2^29 turns: the oracle's fp64 product is off by 2^-53 of them, 2^-21 of an angle
        _within(y, want, half * np.abs(want) + (2.0 ** -16 + 2.0 ** -20) * size)


def test_norm_rope_without_norm_agrees_with_the_rope_kernel():
    T, H, d, theta = 500, 4, 128, 1e7
    q, k = _normal(5, T, 7 * H, d), _normal(6, T, H, d)
    pos = torch.arange(T, device="cuda")[None] + 1000
    for pairing in (0, 1):
        a, b = atf.qk_norm_rope(q, k, theta, pos, pairing=pairing)
        for x, y in ((q, a), (k, b)):
            want, _ = atf.rope_layout(x[None], theta, pos_offset=1000, pairing=pairing)
            # fp32 against fp64 before the one rounding: a step apart at most, and rarely
            assert (y == want[0]).float().mean() > 0.99
            assert torch.allclose(y.float(), want[0].float(), rtol=2.0 ** -7, atol=2.0 ** -13)


def _offset(x, n):
    """A copy of x that starts n elements into its storage."""
    buf = torch.empty(x.numel() + n, dtype=x.dtype, device=x.device)
    return buf[n:].view(x.shape).copy_(x)


def test_rows_aligned_to_16_bytes_only():
    """Outputs and pages that no 32-byte store may touch."""
    T, Hq, Hkv, d, page = 40, 6, 2, 128, 16
    pos = torch.arange(T, device="cuda")[None]
    for dtype, n in ((BF16, 8), (torch.float32, 4)):
        q, k = _normal(11, T, Hq, d, dtype=dtype), _normal(12, T, Hkv, d, dtype=dtype)
        want = atf.qk_norm_rope(q, k, 1e4, pos)
        got = atf.qk_norm_rope(_offset(q, n), _offset(k, n), 1e4, pos, q_out=_offset(q, n), k_out=_offset(k, n))
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    q, k, v = (_normal(s, T, h, d) for s, h in ((13, Hq), (14, Hkv), (15, Hkv)))
    table = _int32([[2, 0, 1]])
    for cu, at in ((_int32([0, T]), slice(0, T)), (None, slice(0, 1))):
        out = []
        for n in (0, 8):
            kp, vp = (_offset(x, n) for x in _pool(3, Hkv, d, page, 16))
            qo = atf.paged_append(q[at], k[at], v[at], kp, vp, table, _int32([3]), 1e4, cu=cu, q_out=_offset(q[at], n))
            out.append((qo, kp, vp))
        atf.atf_check()
        assert all(torch.equal(a, b) for a, b in zip(*out))


def test_norm_rope_feeds_the_prefill():
    S, Hq, Hkv, d, theta, alpha = 300, 14, 2, 128, 1e4, 1.0
    q, k, v = _normal(7, S, Hq, d), _normal(8, S, Hkv, d), _normal(9, S, Hkv, d)
    w = 1 + _normal(10, d, std=0.2)
    pos = torch.arange(S, device="cuda")[None]
    qr, kr = atf.qk_norm_rope(q, k, theta, pos, w, w)
    out = atf.prefill(qr[None], kr[None], v[None], theta, alpha, rotated=True)
    atf.atf_check()
    one = [paged.norm_rope(paged.f64(x), paged.f64(w), 1e-6, pos.cpu().numpy(), [0] * 64, theta, 0)[0] for x in (q, k)]
    W = np.repeat(oracle.windows(d, theta, alpha)[0], 2)
    for t in (0, 1, 150, 299):
        for h in (0, 13):
            kk = np.where((t - np.arange(t + 1))[:, None] <= W, one[1][: t + 1, h // 7], 0)
            x = kk @ one[0][t, h] / math.sqrt(d)
            p = np.exp(x - x.max())
            want = p @ paged.f64(v)[: t + 1, h // 7] / p.sum()
            assert np.abs(paged.f64(out)[0, t, h] - want).max() <= 2e-2  # as the prefill's own tests


# ------------------------------------------------------------------ append

def _check_append(q, k, v, kp, vp, bounds, before, table, start, rows, pos, w, eps, axis, theta, pairing, q_out, q_before):
    """Every slot, bound and query row: the new ones the oracle's, the others as they were."""
    d, Hkv, page = v.shape[2], v.shape[1], vp.shape[2]
    kp0, vp0, bd0 = before
    new_k = torch.zeros(kp.shape[0], page, dtype=torch.bool)
    want, size = paged.norm_rope(paged.f64(k), paged.f64(w[1]) if w[1] is not None else None, eps, pos, axis, theta, pairing)
    kp64 = paged.f64(kp)
    touched = torch.zeros(kp.shape[0], dtype=torch.bool)
    for b, (r0, r1) in enumerate(rows):
        if start[b] < 0:
            continue
        for r in range(r0, r1):
            slot = start[b] + r - r0
            p, at = int(table[b, slot // page]), slot % page
            got = kp64[p, :, :, at].reshape(Hkv, d)
            assert (np.abs(got - want[r]) <= 2.0 ** -8 * np.abs(want[r]) + 2.0 ** -16 * size[r]).all()
            assert torch.equal(vp[p, :, at], v[r])
            new_k[p, at] = touched[p] = True
    keep = ~new_k.cuda()
    assert torch.equal(kp.movedim(3, 1)[keep], kp0.movedim(3, 1)[keep])
    assert torch.equal(vp.movedim(2, 1)[keep], vp0.movedim(2, 1)[keep])
    if bounds is not None:
        assert torch.equal(bounds[~touched.cuda()], bd0[~touched.cuda()])
        for p in touched.nonzero().flatten().tolist():
            keys = kp[p].movedim(2, 0).reshape(page, Hkv, d)[new_k[p].cuda()]
            lo, hi = keys.amin(0), keys.amax(0)
            if not new_k[p, 0]:
                lo, hi = torch.minimum(lo, bd0[p, :, 0]), torch.maximum(hi, bd0[p, :, 1])
            assert torch.equal(bounds[p, :, 0], lo) and torch.equal(bounds[p, :, 1], hi)
    if q is not None:
        wq, sq = paged.norm_rope(paged.f64(q), paged.f64(w[0]) if w[0] is not None else None, eps, pos, axis, theta, pairing)
        mine = np.zeros(q.shape[0], dtype=bool)
        for b, (r0, r1) in enumerate(rows):
            if start[b] >= 0:
                mine[r0:r1] = True
        _within(q_out[torch.from_numpy(mine)], wq[mine], 2.0 ** -8 * np.abs(wq[mine]) + 2.0 ** -16 * sq[mine])
        assert torch.equal(q_out[torch.from_numpy(~mine)], q_before[torch.from_numpy(~mine)])


@pytest.mark.parametrize("start,new,Hq,Hkv,d,page,pairing,axes,norm,bounds", [
    ([0], None, 28, 4, 128, 16, 1, 1, True, True),
    ([700, 15, -1, 16, 0], None, 14, 2, 64, 16, 0, 1, True, True),
    ([63, 64, 65] * 9, None, 8, 1, 128, 64, 1, 1, False, True),
    ([127, 128], None, 3, 3, 128, 128, 0, 1, True, False),
    ([0, 5, 100, 7], [33, 0, 1, 300], 28, 4, 128, 16, 1, 1, True, True),
    ([31, 0, -1, 64], [1, 64, 9, 65], 6, 2, 64, 32, 0, 3, True, True),
    ([3], [1000], 8, 8, 128, 128, 1, 2, False, True),
    ([0] * 70, [1, 0, 2] * 23 + [5], 2, 1, 64, 64, 0, 1, True, False),
    ([i % 40 - 1 for i in range(100)], [7 * i % 23 for i in range(100)], 8, 8, 64, 16, 1, 3, True, True),
    ([9] * 40, [13, 70] * 20, 8, 4, 128, 32, 0, 1, True, True), ([100] * 160, [3] * 160, 4, 4, 128, 128, 1, 1, True, True),
])
def test_append_against_oracle(start, new, Hq, Hkv, d, page, pairing, axes, norm, bounds):
    theta, eps, pad = 1e7, 1e-5, 3
    B = len(start)
    n = [1] * B if new is None else new
    cu = np.concatenate([[0], np.cumsum(n)])
    T = int(cu[-1]) + (0 if new is None else pad)  # rows behind the last sequence
    fused = _normal(21, T, (Hq + 2 * Hkv) * d)
    q, k, v = (fused[:, a * d: b * d].view(T, -1, d) for a, b in ((0, Hq), (Hq, Hq + Hkv), (Hq + Hkv, Hq + 2 * Hkv)))
    table, pool = _tables([max(s, 0) + m for s, m in zip(start, n)], page, 22)
    kp, vp = _pool(pool, Hkv, d, page, 23)
    bd = _normal(25, pool, Hkv, 2, d) if bounds else None
    w = [1 + _normal(s, d, std=0.2) if norm else None for s in (26, 27)]
    pos = None
    slots = np.zeros((1, T), dtype=np.int64)
    for b in range(B):
        slots[0, cu[b]: cu[b + 1]] = max(start[b], 0) + np.arange(n[b])
    if axes > 1:
        pos = torch.randint(0, 5000, (axes, T), generator=torch.Generator().manual_seed(28)).cuda()
    q_out = _normal(29, T, Hq, d)
    q_before, before = q_out.clone(), (kp.clone(), vp.clone(), bd.clone() if bounds else None)
    atf.paged_append(q, k, v, kp, vp, table, _int32(start), theta, cu=None if new is None else _int32(cu), pos=pos,
                     q_weight=w[0], k_weight=w[1], eps=eps, pair_axis=_axes(d, axes), pairing=pairing, bounds=bd,
                     q_out=q_out)
    atf.atf_check()
    rows = [(int(cu[b]), int(cu[b + 1])) for b in range(B)]
    _check_append(q, k, v, kp, vp, bd, before, table.cpu(), start, rows, slots if pos is None else pos.cpu().numpy(), w,
                  eps, _axes(d, axes), theta, pairing, q_out, q_before)


def test_append_without_queries_in_pieces_equals_at_once():
    n, Hkv, d, page, theta = 500, 4, 128, 32, 1e7
    k, v = _normal(31, n, Hkv, d), _normal(32, n, Hkv, d)
    table, pool = _tables([n], page, 33)
    pools = []
    for pieces in ([n], [1, 30, 1, 32, 100, 336], [31] + [1] * 5 + [464]):
        kp, vp = _pool(pool, Hkv, d, page, 34)
        bd = torch.zeros(pool, Hkv, 2, d, dtype=BF16, device="cuda")
        at = 0
        for m in pieces:
            cu = None if m == 1 else _int32([0, m])
            assert atf.paged_append(None, k[at: at + m], v[at: at + m], kp, vp, table, _int32([at]), theta, cu=cu,
                                    bounds=bd) is None
            at += m
        pools.append((kp, vp, bd))
    atf.atf_check()
    for other in pools[1:]:
        assert all(torch.equal(x, y) for x, y in zip(pools[0], other))


def test_append_skips_and_reports_bad_tables():
    Hkv, d, page = 2, 64, 16
    k = v = _normal(41, 40, Hkv, d)
    kp, vp = _pool(4, Hkv, d, page, 42)
    before = kp.clone(), vp.clone()
    for table, start, cu in (([[4, -1, 0]], [0], [0, 20]), ([[1, 2, 3]], [48], [0, 5]), ([[1, 2, 3]], [2 ** 31 - 1], [0, 5]),
                             ([[1, 2, 3]], [0], [0, 41]), ([[1, 2, 3]], [0], [3, 2]), ([[1, 2, 3]], [0], [-1, 2])):
        atf.paged_append(None, k, v, kp, vp, _int32(table), _int32(start), 1e4, cu=_int32(cu))
        with pytest.raises(atf.AtfError) as e:
            atf.atf_check()
        assert e.value.status == atf.ATF_ERR_INVALID_ARG
        assert torch.equal(kp, before[0]) and torch.equal(vp, before[1])
    atf.paged_append(None, k[:1], v[:1], kp, vp, _int32([[1]]), _int32([16]), 1e4)  # behind the table
    with pytest.raises(atf.AtfError):
        atf.atf_check()
    assert torch.equal(kp, before[0])
    atf.atf_check()  # reported once


# ------------------------------------------------------------------ decode

def _decode_case(lens, Hq, Hkv, d, page, theta, alpha, seed=51, stale=math.nan, std=1.0):
    table, pool = _tables(lens, page, seed, extra=1)
    kp, vp = _pool(pool, Hkv, d, page, seed + 1)
    q = _normal(seed + 3, len(lens), Hq, d, std=std)
    free = sorted(set(range(pool)) - set(table.flatten().tolist()))
    kp[free], vp[free] = stale, stale  # pages of nobody
    for b, n in enumerate(lens):  # slots behind the last key
        if n > 0 and n % page:
            p = int(table[b, n // page])
            kp[p, :, :, n % page:], vp[p, :, n % page:] = stale, stale
    return q, kp, vp, table, _int32(lens)


def _check_decode(q, kp, vp, table, lens, theta, alpha, out, lse, selected=None):
    d = q.shape[2]
    want, wl, weight, spread = paged.decode(paged.f64(q), paged.f64(kp), paged.f64(vp), table.cpu().numpy(),
                                            lens.cpu().numpy(), theta, alpha,
                                            None if selected is None else selected.cpu().numpy())
    step = 18 * 2.0 ** -23 * (d // 16) * spread + 2.0 ** -16
    _within(out, want, (2.0 ** -8 + 2 * step[..., None]) * weight + 2.0 ** -8 * np.abs(want))
    live = np.isfinite(wl)
    got = paged.f64(lse)
    assert np.array_equal(np.isfinite(got), live) and (got[~live] == -math.inf).all()
    assert (np.abs(got[live] - wl[live]) <= step[live] + 2.0 ** -20 * np.abs(wl[live])).all()


@pytest.mark.parametrize("lens,Hq,Hkv,d,page,theta,alpha", [
    ([1], 28, 4, 128, 16, 1e7, 1.0), ([777], 4, 4, 64, 16, 1e4, 1.0), ([300, 129, 0, 128], 28, 4, 128, 64, 1e7, 1.0),
    ([5000, 4097, 33, -3], 14, 2, 128, 128, 1e4, 0.5), ([2048, 1000, 17], 8, 1, 64, 32, 1e4, math.inf),
    ([3000], 8, 1, 128, 16, 1.0001, 0.1),  # every window is 1: far keys have no pair in reach
    ([4000, 1, 1, 127, 128, 129] * 4, 7, 1, 128, 16, 1e7, math.inf), ([40000], 6, 3, 128, 64, 1e7, 0.5),
    ([0, 0, 0], 5, 1, 64, 16, 1e4, 1.0), ([1, 2, 3] * 90, 3, 3, 64, 32, 1e4, 1.0),
    # enough keys for tiles of 128, whose pages end inside them
    ([5000, 33, 129, 0] * 5, 6, 2, 64, 16, 1e4, 1.0), ([40000], 16, 2, 64, 128, 5e5, 0.5), ([100] * 400, 3, 3, 64, 64, 1e4, math.inf),
    ([38000, 1], 4, 4, 64, 32, 1.0001, 0.1),
])
def test_decode_against_oracle(lens, Hq, Hkv, d, page, theta, alpha):
    q, kp, vp, table, n = _decode_case(lens, Hq, Hkv, d, page, theta, alpha)
    lse = torch.full((len(lens), Hq), 7.0, device="cuda")
    out = atf.paged_decode(q, kp, vp, table, n, theta, alpha, lse=lse)
    atf.atf_check()
    _check_decode(q, kp, vp, table, n, theta, alpha, out, lse)


@pytest.mark.parametrize("d,page,stale", [(128, 64, math.inf), (128, 16, math.nan), (64, 128, math.nan)])
def test_decode_sharp_softmax_and_infinite_stale_slots(d, page, stale):
    lens, theta = [900, 64, 65], 1e7
    q, kp, vp, table, n = _decode_case(lens, 16, 2, d, page, theta, 1.0, stale=stale, std=8.0)
    lse = torch.empty(3, 16, device="cuda")
    out = atf.paged_decode(q, kp, vp, table, n, theta, 1.0, lse=lse)
    atf.atf_check()
    _check_decode(q, kp, vp, table, n, theta, 1.0, out, lse)


@pytest.mark.parametrize("lens,Hq,Hkv,d,page,n_sel", [
    ([1000, 16, 0, 333], 28, 4, 128, 16, 9), ([5000, 200], 4, 2, 64, 64, 40), ([129], 8, 1, 128, 128, 1),
    ([2000, 100, 31, 0] * 10, 4, 2, 64, 32, 30)])
def test_decode_over_listed_pages(lens, Hq, Hkv, d, page, n_sel):
    theta, alpha = 1e4, 1.0
    q, kp, vp, table, n = _decode_case(lens, Hq, Hkv, d, page, theta, alpha, seed=61)
    r = np.random.RandomState(62)
    sel = np.full((len(lens), Hkv, n_sel), -1, dtype=np.int32)
    for b, m in enumerate(lens):
        P = -(-m // page)
        for h in range(Hkv):
            pick = r.permutation(P)[:n_sel]  # in no order
            sel[b, h, : len(pick)] = pick
            if len(pick) > 2:
                sel[b, h, 1] = -1  # a hole
    sel = torch.from_numpy(sel).cuda()
    lse = torch.empty(len(lens), Hq, device="cuda")
    out = atf.paged_decode(q, kp, vp, table, n, theta, alpha, selected=sel, lse=lse)
    atf.atf_check()
    _check_decode(q, kp, vp, table, n, theta, alpha, out, lse, sel)


@pytest.mark.parametrize("lens,Hq,Hkv,d,page,extra,listed", [
    ([2, 3, 17, 40, 130] * 4, 28, 4, 128, 16, 0, False), ([2, 3, 17, 40, 130] * 4, 8, 1, 128, 64, 0, True),
    ([2, 3, 17, 40, 130] * 4, 6, 2, 64, 16, 0, False), ([5, 33, 129, 300] * 5, 16, 2, 64, 32, 80, False),
    ([5, 33, 129, 300] * 5, 16, 2, 64, 128, 20, True)])
def test_decode_weights_keep_their_low_bits(lens, Hq, Hkv, d, page, extra, listed):
    """Few keys of both signs: what a weight loses shows where the values nearly cancel.  A weight in two bf16
    parts is off by 2^-8 of 2^-8; the products with the values, two a block of 16 keys and a warp, add 18 * 2^-23
    of the sum so far each (a warp takes one block of 128 keys).  A table of that width takes the tiles of 128
    keys for heads of 64."""
    theta, alpha = 1e4, 1.0
    q, kp, vp, table, n = _decode_case(lens, Hq, Hkv, d, page, theta, alpha, seed=67)
    if extra:
        table = torch.cat([table, torch.full((len(lens), extra), -1, dtype=torch.int32, device="cuda")], 1).contiguous()
        assert table.shape[1] * page * len(lens) * Hkv >= 8 * 64 * 148 or listed
    sel = None
    if listed:
        P = -(-max(lens) // page)
        sel = torch.arange(P, dtype=torch.int32, device="cuda").expand(len(lens), Hkv, P).contiguous()
    lse = torch.empty(len(lens), Hq, device="cuda")
    out = atf.paged_decode(q, kp, vp, table, n, theta, alpha, selected=sel, lse=lse)
    atf.atf_check()
    want, _, weight, spread = paged.decode(paged.f64(q), paged.f64(kp), paged.f64(vp), table.cpu().numpy(), lens, theta,
                                           alpha, None if sel is None else sel.cpu().numpy())
    step = 18 * 2.0 ** -23 * (d // 16) * spread + 2.0 ** -16
    summed = 18 * 2.0 ** -23 * 2 * (max(lens) // 128 + 1)
    _within(out, want, (2.0 ** -16 + summed + 2 * step[..., None]) * weight + 2.0 ** -8 * np.abs(want))


def test_decode_of_every_page_listed_is_the_plain_decode():
    lens, theta, alpha = [700, 1300], 1e7, 1.0
    q, kp, vp, table, n = _decode_case(lens, 14, 2, 128, 32, theta, alpha, seed=64)
    P = -(-max(lens) // 32)
    sel = torch.arange(P, dtype=torch.int32, device="cuda").expand(2, 2, P).contiguous()
    a = atf.paged_decode(q, kp, vp, table, n, theta, alpha)
    b = atf.paged_decode(q, kp, vp, table, n, theta, alpha, selected=sel)
    atf.atf_check()
    # the two differ in how tiles are shared out, hence in where a maximum is taken
    assert torch.allclose(a.float(), b.float(), rtol=2.0 ** -6, atol=2.0 ** -8)


def test_decode_agrees_with_the_contiguous_decode_and_strided_queries():
    B, N, Hq, Hkv, d, page, theta, alpha = 2, 1024, 14, 2, 128, 64, 1e7, 1.0
    lens = [1024, 777]
    raw = _normal(71, B, Hq, d)
    k_rot, v = _normal(72, B, N, Hkv, d), _normal(73, B, N, Hkv, d)
    _, kc = atf.rope_layout(k_rot, theta, rotate=False, rotated_out=False, chunked_out=True)
    want = atf.decode(raw, kc, v, lens, theta, alpha)
    q = torch.cat([atf.rope_layout(raw[b: b + 1, None], theta, pos_offset=n - 1)[0][:, 0] for b, n in enumerate(lens)])
    wide = torch.zeros(B, Hq + 3, d, dtype=BF16, device="cuda")
    wide[:, :Hq] = q
    table = torch.arange(B * N // page, dtype=torch.int32, device="cuda").view(B, -1)
    kp = kc.view(B, Hkv, d // 16, N // page, page, 16).permute(0, 3, 1, 2, 4, 5).reshape(-1, Hkv, d // 16, page, 16)
    vp = v.view(B, N // page, page, Hkv, d).transpose(2, 3).reshape(-1, Hkv, page, d)
    got = atf.paged_decode(wide[:, :Hq], kp.contiguous(), vp.contiguous(), table, _int32(lens), theta, alpha)
    atf.atf_check()
    assert torch.allclose(got.float(), want.float(), rtol=2.0 ** -6, atol=2.0 ** -7)


def test_decode_skips_and_reports_bad_tables():
    q, kp, vp, table, n = _decode_case([300, 300], 4, 2, 64, 16, 1e4, 1.0, seed=74)
    good = atf.paged_decode(q, kp, vp, table, n, 1e4, 1.0)
    atf.atf_check()
    for bad in (-1, kp.shape[0], 2 ** 31 - 1, -2 ** 31):
        t = table.clone()
        t[1, 5] = bad
        out = atf.paged_decode(q, kp, vp, t, n, 1e4, 1.0)
        with pytest.raises(atf.AtfError) as e:
            atf.atf_check()
        assert e.value.status == atf.ATF_ERR_INVALID_ARG and "page" in str(e.value)
        assert torch.equal(out[0], good[0]) and torch.isfinite(out[1].float()).all()
    for lens in ([300, 16 * table.shape[1] + 1], [300, 2 ** 31 - 1]):
        atf.paged_decode(q, kp, vp, table.clamp(min=0), _int32(lens), 1e4, 1.0)
        with pytest.raises(atf.AtfError):
            atf.atf_check()
    sel = torch.zeros(2, 2, 3, dtype=torch.int32, device="cuda")
    sel[1, 1, 2] = 19  # the sequence has 19 pages, 0 .. 18
    sel[:, :, 1] = 1
    atf.paged_decode(q, kp, vp, table, n, 1e4, 1.0, selected=sel)
    with pytest.raises(atf.AtfError):
        atf.atf_check()


def test_decode_of_a_cache_past_2_31_elements():
    """Pages whose elements lie beyond 2^31 of the pool's start."""
    Hkv, d, page = 8, 128, 128
    pool = 2 ** 31 // (Hkv * d * page) + 64
    kp = torch.zeros(pool, Hkv, d // 16, page, 16, dtype=BF16, device="cuda")
    vp = torch.zeros(pool, Hkv, page, d, dtype=BF16, device="cuda")
    table = _int32([[pool - 1, 3, pool - 5]])
    k, v = _normal(75, 300, Hkv, d), _normal(76, 300, Hkv, d)
    q = _normal(77, 300, 2 * Hkv, d)
    bd = torch.zeros(pool, Hkv, 2, d, dtype=BF16, device="cuda")
    qr = atf.paged_append(q, k, v, kp, vp, table, _int32([0]), 1e4, cu=_int32([0, 300]), bounds=bd)
    lse = torch.empty(1, 2 * Hkv, device="cuda")
    out = atf.paged_decode(qr[-1:], kp, vp, table, _int32([300]), 1e4, 1.0, lse=lse)
    atf.atf_check()
    at = table[0].long()
    _check_decode(qr[-1:], kp[at], vp[at], torch.tensor([[0, 1, 2]]), _int32([300]), 1e4, 1.0, out, lse)


# ------------------------------------------------------------------ selection

@pytest.mark.parametrize("lens,Hq,Hkv,d,page,theta,alpha,n_sel,first,last", [
    ([1000, 16, 0, 333], 28, 4, 128, 16, 1e4, 1.0, 9, 1, 1), ([9000, 200], 4, 2, 64, 16, 1e4, math.inf, 40, 0, 0),
    ([129], 8, 1, 128, 128, 1e7, 1.0, 1, 0, 1), ([20000], 3, 1, 64, 16, 1e4, 0.5, 700, 3, 5),
    ([640, 641, 639], 7, 7, 128, 32, 1e4, 1.0, 20, 2, 2), ([5000], 8, 1, 128, 16, 1.0001, 0.1, 12, 0, 0),
    ([50000, 4097, 33], 4, 2, 64, 16, 1e4, 1.0, 12, 1, 1), ([36000, 20000], 2, 2, 64, 16, 1e4, 0.5, 5, 0, 0),
    ([16 * 16 * 40, 16 * 16 * 40 - 16], 2, 1, 64, 16, 1e4, math.inf, 13, 2, 1), ([32, 31], 4, 2, 64, 16, 1e4, 1.0, 1, 0, 0),
])
def test_select_against_oracle(lens, Hq, Hkv, d, page, theta, alpha, n_sel, first, last):
    table, pool = _tables(lens, page, 81, extra=2)
    bd = torch.sort(_normal(82, pool, Hkv, 2, d), dim=2).values.contiguous()
    q = _normal(83, len(lens), Hq, d)
    sel = atf.page_select(q, bd, table, _int32(lens), page, n_sel, theta, alpha, first, last)
    atf.atf_check()
    want = paged.select(paged.f64(q), paged.f64(bd), table.cpu().numpy(), lens, page, n_sel, theta, alpha, first, last)
    assert np.array_equal(sel.cpu().numpy(), want)


@pytest.mark.parametrize("first,last,n_sel,pages,P", [
    (1, 110, 113, range(114, 131), 0), (1, 128, 131, range(132, 165), 0), (128, 1, 131, range(132, 165), 0),
    (1, 256, 261, range(262, 305, 3), 0), (256, 0, 260, range(261, 305, 4), 0), (1, 512, 517, range(518, 561, 6), 0),
    (512, 3, 519, range(520, 561, 7), 0), (1, 512, 521, [560, 640, 700], 0), (600, 2, 610, [700, 760, 800], 0),
    # the same lists in tables of other widths: other kernels, other blocks
    (1, 128, 131, [132, 144, 150, 200], 900), (1, 256, 261, [262, 272, 300, 400], 2100),
    (1, 900, 903, [904, 912, 960, 2100], 0), (2000, 100, 2103, [2104, 2112, 2160, 2300], 0),
    # as many competing groups as four a place, one more and one less
    (16, 16, 36, [32 + 16 * 15, 32 + 16 * 16, 32 + 16 * 16 + 1, 32 + 16 * 17], 0), (15, 17, 33, [32 + 49, 32 + 64, 32 + 65], 0),
])
def test_select_beside_long_runs_of_forced_pages(first, last, n_sel, pages, P):
    """Few pages compete: groups of forced pages alone, and fewer competing groups than places."""
    Hq, Hkv, d, page = 2, 1, 64, 16
    lens = [page * n - i % page for i, n in enumerate(pages)]
    table, pool = _tables(lens, page, 101, extra=max(0, P - max(pages)))
    bd = torch.sort(_normal(102, pool, Hkv, 2, d), dim=2).values.contiguous()
    q = _normal(103, len(lens), Hq, d)
    sel = atf.page_select(q, bd, table, _int32(lens), page, n_sel, 1e4, 1.0, first, last)
    atf.atf_check()
    want = paged.select(paged.f64(q), paged.f64(bd), table.cpu().numpy(), lens, page, n_sel, 1e4, 1.0, first, last)
    assert np.array_equal(sel.cpu().numpy(), want)


def test_select_ties_go_to_the_lowest_index():
    """Every page of a sequence the same (or two kinds of pages): equal scores."""
    Hkv, d, page, n = 2, 64, 16, 16 * 3000
    table = torch.zeros(2, 3000, dtype=torch.int32, device="cuda")
    table[1, 1::3] = 1
    bd = torch.sort(_normal(84, 2, Hkv, 2, d), dim=2).values.contiguous()
    q = _normal(85, 2, 4, d)
    sel = atf.page_select(q, bd, table, _int32([n, n]), page, 1200, 1e4, math.inf, 1, 1)
    atf.atf_check()
    want = paged.select(paged.f64(q), paged.f64(bd), table.cpu().numpy(), [n, n], page, 1200, 1e4, math.inf, 1, 1)
    assert np.array_equal(sel.cpu().numpy(), want)
    assert sel[0, 0].tolist() == list(range(1199)) + [2999]


@pytest.mark.parametrize("pages,n_sel,scale", [(40, 9, 1.0), (200, 31, 1.0), (3000, 500, 1.0), (20000, 40, 1.0),
                                               (300, 20, 1e30), (300, 20, 1e-25)])
def test_select_orders_scores_that_32_bits_cannot_part(pages, n_sel, scale):
    """Pages alike but for one dim whose share of the score is below 2^-30; sums beyond the range of 32 bits."""
    Hkv, d, page = 2, 128, 16
    bd = torch.sort(_normal(88, 1, Hkv, 2, d), dim=2).values.repeat(pages, 1, 1, 1)
    bd[:, :, 1, 5] = _normal(89, pages, Hkv).abs()  # few distinct values: ties among them
    bd[:, :, 0, 5] = 0
    q = _normal(90, 1, 6, d)
    q[..., 5] = 2.0 ** -30
    bd, q = (bd.double() * scale).to(BF16), (q.double() * scale).to(BF16)
    table = torch.randperm(pages, generator=torch.Generator().manual_seed(3))[None].to(torch.int32).cuda()
    sel = atf.page_select(q, bd, table, _int32([pages * page]), page, n_sel, 1e4, math.inf, 1, 1)
    atf.atf_check()
    want = paged.select(paged.f64(q), paged.f64(bd), table.cpu().numpy(), [pages * page], page, n_sel, 1e4, math.inf, 1, 1)
    assert np.array_equal(sel.cpu().numpy(), want)


def test_select_with_a_query_of_zeros_keeps_the_first_pages():
    bd = torch.sort(_normal(97, 700, 1, 2, 64), dim=2).values
    table = torch.arange(700, dtype=torch.int32, device="cuda")[None]
    sel = atf.page_select(torch.zeros(1, 3, 64, dtype=BF16, device="cuda"), bd, table, _int32([700 * 32]), 32, 50, 1e4, 1.0)
    atf.atf_check()
    assert sel.flatten().tolist() == list(range(49)) + [699]


def test_select_zeros_of_both_signs_are_equal():
    """A score of -0 (no pair counts, or products that are -0) ranks as +0."""
    bd = torch.zeros(2, 1, 2, 64, dtype=BF16, device="cuda")
    bd[1] = -0.0
    table = _int32([[1, 0, 1, 0, 1, 0]])
    sel = atf.page_select(_normal(86, 1, 1, 64), bd, table, _int32([96]), 16, 3, 1e4, 1.0, 0, 0)
    atf.atf_check()
    assert sel.flatten().tolist() == [0, 1, 2]


def test_select_reports_bad_tables():
    bd = torch.zeros(2, 1, 2, 64, dtype=BF16, device="cuda")
    for table, n in (([[0, 2, 1]], 48), ([[0, -1, 1]], 48), ([[0, 1, 1]], 49)):
        sel = atf.page_select(_normal(87, 1, 1, 64), bd, _int32(table), _int32([n]), 16, 2, 1e4, 1.0)
        with pytest.raises(atf.AtfError):
            atf.atf_check()
        assert sel.min() >= -1 and sel.max() < 3


# ------------------------------------------------------------------ together

def _loop(B, prefix, steps, graph):
    """A serving loop: prompts appended, then one token per sequence and step: append, select, attend to the
    selected pages, and attend to all.  Returns what each step gave and the caches."""
    Hq, Hkv, d, page, theta, alpha, n_sel = 14, 2, 128, 16, 1e7, 1.0, 6
    most = max(prefix) + steps
    table, pool = _tables([n + steps for n in prefix], page, 91)
    kp, vp = _pool(pool, Hkv, d, page, 92)
    bd = torch.zeros(pool, Hkv, 2, d, dtype=BF16, device="cuda")
    T = sum(prefix)
    w = 1 + _normal(94, d, std=0.2)
    cu = _int32(np.concatenate([[0], np.cumsum(prefix)]))
    length = torch.zeros(B, dtype=torch.int32, device="cuda")
    atf.paged_append(None, _normal(95, T, Hkv, d), _normal(96, T, Hkv, d), kp, vp, table, length, theta, cu=cu, k_weight=w,
                     pairing=1, bounds=bd)
    length += cu.diff()
    q, k, v = (torch.empty(B, h, d, dtype=BF16, device="cuda") for h in (Hq, Hkv, Hkv))
    after = length.clone()
    ws = torch.empty(max(atf.atf_paged_decode_workspace_bytes(B, Hq, Hkv, d),
                         atf.atf_page_select_workspace_bytes(B, Hkv, table.shape[1])), dtype=torch.uint8, device="cuda")
    buf = dict(q=torch.empty_like(q), sel=torch.empty(B, Hkv, n_sel, dtype=torch.int32, device="cuda"),
               sparse=torch.empty_like(q), dense=torch.empty_like(q), lse=torch.empty(B, Hq, device="cuda"))

    def step():
        torch.add(length, 1, out=after)
        atf.paged_append(q, k, v, kp, vp, table, length, theta, q_weight=w, k_weight=w, pairing=1, bounds=bd, q_out=buf["q"])
        atf.page_select(buf["q"], bd, table, after, page, n_sel, theta, alpha, 1, 2, selected=buf["sel"], workspace=ws)
        atf.paged_decode(buf["q"], kp, vp, table, after, theta, alpha, selected=buf["sel"], out=buf["sparse"], workspace=ws)
        atf.paged_decode(buf["q"], kp, vp, table, after, theta, alpha, lse=buf["lse"], out=buf["dense"], workspace=ws)

    g = None
    if graph:
        keep = kp.clone(), vp.clone(), bd.clone()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        for x, y in zip((kp, vp, bd), keep):
            x.copy_(y)
    steps_out = []
    for s in range(steps):
        for i, x in enumerate((q, k, v)):
            x.copy_(_normal(100 + 3 * s + i, *x.shape))
        g.replay() if graph else step()
        steps_out.append({n: x.clone() for n, x in buf.items()})
        length.add_(1)
    atf.atf_check()
    return steps_out, (kp, vp, bd, table), (theta, alpha, page, n_sel)


def test_serving_loop_against_oracle_and_in_a_graph():
    prefix, steps = [100, 37, 256], 6
    eager, (kp, vp, bd, table), (theta, alpha, page, n_sel) = _loop(3, prefix, steps, graph=False)
    for s, got in enumerate(eager):
        lens = _int32([n + s + 1 for n in prefix])
        _check_decode(got["q"], kp, vp, table, lens, theta, alpha, got["dense"], got["lse"])
        sel = got["sel"].cpu().numpy()
        for b in range(3):
            P = -(-(prefix[b] + s + 1) // page)
            for row in sel[b]:
                live = row[row >= 0].tolist()
                assert live == sorted(set(live)) and len(live) == min(n_sel, P) and {0, P - 1} <= set(live)
        want, _, weight, spread = paged.decode(paged.f64(got["q"]), paged.f64(kp), paged.f64(vp), table.cpu().numpy(),
                                               lens.cpu().numpy(), theta, alpha, sel)
        step = 18 * 2.0 ** -23 * 8 * spread + 2.0 ** -16
        _within(got["sparse"], want, (2.0 ** -8 + 2 * step[..., None]) * weight + 2.0 ** -8 * np.abs(want))
    # the last step's selection, from bounds that the pages give
    lens = [n + steps for n in prefix]
    real = torch.stack([x.reshape(bd.shape[0], 2, 128) for x in (kp.amin(3), kp.amax(3))], 2)
    full = [int(table[b, i]) for b, n in enumerate(lens) for i in range(n // page)]
    assert torch.equal(bd[full], real[full])
    want = paged.select(paged.f64(eager[-1]["q"]), paged.f64(bd), table.cpu().numpy(), lens, page, n_sel, theta, alpha, 1, 2)
    assert np.array_equal(eager[-1]["sel"].cpu().numpy(), want)
    replayed, pools, _ = _loop(3, prefix, steps, graph=True)
    for a, b in zip(eager, replayed):
        assert all(torch.equal(a[n], b[n]) for n in a)
    assert all(torch.equal(x, y) for x, y in zip((kp, vp, bd), pools))


def test_two_captured_graphs_share_a_workspace():
    theta, alpha = 1e7, 1.0
    ws = torch.full((atf.atf_paged_decode_workspace_bytes(3, 14, 2, 128),), 255, dtype=torch.uint8, device="cuda")
    graphs, outs, want = [], [], []
    for seed, lens in ((111, [900, 3000, 5]), (112, [20000])):
        c = _decode_case(lens, 14, 2, 128, 32, theta, alpha, seed=seed)
        want.append(atf.paged_decode(*c, theta, alpha))
        out = torch.empty_like(c[0])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            atf.paged_decode(*c, theta, alpha, out=out, workspace=ws)
        graphs.append((g, c))
        outs.append(out)
    for _ in range(3):
        for g, _ in graphs:
            g.replay()
    atf.atf_check()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_calls_on_two_streams_at_once():
    theta, alpha = 1e7, 1.0
    cases = [_decode_case(lens, 28, 4, 128, 64, theta, alpha, seed=s) for s, lens in ((121, [30000]), (122, [200] * 9))]
    want = [atf.paged_decode(*c, theta, alpha) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [torch.empty_like(w) for w in want]
    work = [torch.empty(atf.atf_paged_decode_workspace_bytes(9, 28, 4, 128), dtype=torch.uint8, device="cuda")
            for _ in cases]
    for _ in range(20):
        for c, s, o, ws in zip(cases, streams, got, work):
            atf.paged_decode(*c, theta, alpha, out=o, workspace=ws, stream=s)
    torch.cuda.synchronize()
    atf.atf_check()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_scratch_and_outputs_of_a_call_on_a_given_stream():
    """What a call allocates is not handed out again while the other stream still uses it."""
    theta, alpha = 1e7, 1.0
    c = _decode_case([40000, 300], 28, 4, 128, 64, theta, alpha, seed=131)
    bd = torch.sort(_normal(132, c[1].shape[0], 4, 2, 128), dim=2).values
    want = atf.paged_decode(*c, theta, alpha)
    sel = atf.page_select(c[0], bd, c[3], c[4], 64, 9, theta, alpha)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = []
    for _ in range(10):
        got.append((atf.paged_decode(*c, theta, alpha, stream=side),
                    atf.page_select(c[0], bd, c[3], c[4], 64, 9, theta, alpha, stream=side.cuda_stream)))
        for n in (1 << 20, 1 << 17, 1 << 14):  # sizes of the scratch, on the current stream
            torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    atf.atf_check()
    assert all(torch.equal(o, want) and torch.equal(s, sel) for o, s in got)
    with torch.cuda.stream(side):  # handles of the default stream, while another is current
        got = [atf.paged_decode(*c, theta, alpha, stream=s) for s in (0, 1)]
        with pytest.raises(TypeError, match="per-thread"):
            atf.paged_decode(*c, theta, alpha, stream=2)
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in got)


def test_captured_behind_copies_and_events_of_other_streams():
    """Graph nodes before the calls that are no kernels, and forks that join before and behind them."""
    theta, alpha = 1e7, 1.0
    q, kp, vp, table, n = _decode_case([5000, 700, 0], 28, 4, 128, 32, theta, alpha, seed=141)
    bd = torch.stack([kp.amin(3).view(-1, 4, 128), kp.amax(3).view(-1, 4, 128)], 2).contiguous()
    pos = torch.arange(3, device="cuda")[None].contiguous()
    src = q.clone()

    def calls(buf, side):
        main = torch.cuda.current_stream()
        buf["q"].copy_(src)
        buf["n"].copy_(n)
        atf.qk_norm_rope(buf["q"], buf["k"], theta, pos, q_out=buf["qn"], k_out=buf["kn"])
        buf["qn"].zero_()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            atf.page_select(buf["q"], bd, table, buf["n"], 32, 7, theta, alpha, selected=buf["sel"], workspace=buf["ws"][1])
        atf.paged_decode(buf["q"], kp, vp, table, buf["n"], theta, alpha, out=buf["dense"], workspace=buf["ws"][0])
        main.wait_stream(side)
        atf.paged_decode(buf["q"], kp, vp, table, buf["n"], theta, alpha, selected=buf["sel"], out=buf["sparse"],
                         workspace=buf["ws"][0])

    def buffers():
        need = max(atf.atf_paged_decode_workspace_bytes(3, 28, 4, 128), atf.atf_page_select_workspace_bytes(3, 4, table.shape[1]))
        return dict(q=torch.empty_like(q), k=q[:, :4].contiguous(), n=torch.empty_like(n), qn=torch.empty_like(q),
                    kn=torch.empty_like(q[:, :4].contiguous()), sel=torch.empty(3, 4, 7, dtype=torch.int32, device="cuda"),
                    dense=torch.empty_like(q), sparse=torch.empty_like(q),
                    ws=[torch.empty(need, dtype=torch.uint8, device="cuda") for _ in range(2)])

    side = torch.cuda.Stream()
    want, got = buffers(), buffers()
    calls(want, side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        calls(got, side)
    for _ in range(4):
        for x in ("dense", "sparse", "sel", "kn"):
            got[x].fill_(1)
        g.replay()
    torch.cuda.synchronize()
    atf.atf_check()
    assert all(torch.equal(got[x], want[x]) for x in ("dense", "sparse", "sel", "kn"))
