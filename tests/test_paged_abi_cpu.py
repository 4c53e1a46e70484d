"""Paged cache entry points on the host (no GPU): the argument structures' layout, the
refusals before any device call, and the decode's division of its tile list, walked as
the kernel walks it."""
import ctypes
import math
import os
import random
import subprocess

import pytest
import torch

import oracle
from rope_frequency_sparse_b200 import atf, build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 20  # a 16-byte aligned address, never read


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return atf.load_library()


def _status(fn, *args):
    try:
        fn(*args)
    except atf.AtfError as e:
        return e.status
    return atf.ATF_OK


@pytest.mark.parametrize("name,mirror", [
    ("atf_qk_norm_rope_args", atf.QkNormRopeArgs), ("atf_paged_append_args", atf.PagedAppendArgs),
    ("atf_paged_decode_args", atf.PagedDecodeArgs), ("atf_page_select_args", atf.PageSelectArgs)])
def test_structures_mirror_the_header(tmp_path, name, mirror):
    fields = [f for f, _ in mirror._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include "atf.h"\nint main(void) {\n  printf("%zu", sizeof(' + name + "));\n"
                   + "".join(f'  printf(" %zu", offsetof({name}, {f}));\n' for f in fields) + "  return 0;\n}\n")
    exe = tmp_path / "layout"
    subprocess.check_call(["gcc", "-I" + os.path.join(ROOT, "include"), "-o", str(exe), str(src)])
    got = [int(x) for x in subprocess.check_output([str(exe)]).split()]
    assert got == [ctypes.sizeof(mirror)] + [getattr(mirror, f).offset for f in fields]


NORM = dict(q=FAKE, k=2 * FAKE, q_stride=4608, k_stride=4608, q_out=3 * FAKE, k_out=4 * FAKE, pos=FAKE, tokens=8,
            heads=28, kv_heads=4, d=128, n_axes=1, pairing=1, dtype=0, theta=1e7, eps=1e-6)
APPEND = dict(q=FAKE, k=2 * FAKE, v=3 * FAKE, q_stride=4608, k_stride=4608, v_stride=4608, q_out=4 * FAKE,
              k_pages=5 * FAKE, v_pages=6 * FAKE, bounds=7 * FAKE, page_table=FAKE, start=FAKE, num_pages=64, tokens=2,
              batch=2, heads=28, kv_heads=4, d=128, page_size=64, max_pages=16, n_axes=1, pairing=1, theta=1e7, eps=1e-6)
DECODE = dict(q=FAKE, q_stride=3584, k_pages=FAKE, v_pages=FAKE, page_table=FAKE, kv_len=FAKE, out=FAKE, num_pages=64,
              batch=2, heads=28, kv_heads=4, d=128, page_size=64, max_pages=16, theta=1e7, alpha=1.0, workspace=FAKE,
              workspace_bytes=1 << 24)
SELECT = dict(q=FAKE, q_stride=3584, bounds=FAKE, page_table=FAKE, kv_len=FAKE, selected=FAKE, num_pages=64, batch=2,
              heads=28, kv_heads=4, d=128, page_size=64, max_pages=16, n_select=8, n_first=1, n_last=1, theta=1e7,
              alpha=1.0, workspace=FAKE, workspace_bytes=1 << 24)
CALLS = {"norm": (atf.atf_qk_norm_rope, atf.QkNormRopeArgs, NORM),
         "append": (atf.atf_paged_append, atf.PagedAppendArgs, APPEND),
         "decode": (atf.atf_paged_decode, atf.PagedDecodeArgs, DECODE),
         "select": (atf.atf_page_select, atf.PageSelectArgs, SELECT)}
INVALID, UNSUPPORTED = atf.ATF_ERR_INVALID_ARG, atf.ATF_ERR_UNSUPPORTED


@pytest.mark.parametrize("call,change,status", [
    ("norm", dict(d=96), UNSUPPORTED), ("norm", dict(theta=1.0), INVALID), ("norm", dict(dtype=2), INVALID),
    ("norm", dict(pairing=2), INVALID), ("norm", dict(tokens=-1), INVALID), ("norm", dict(heads=0, kv_heads=0), INVALID),
    ("norm", dict(eps=-1.0), INVALID), ("norm", dict(eps=math.nan), INVALID), ("norm", dict(n_axes=0), UNSUPPORTED),
    ("norm", dict(n_axes=5, pair_axis=bytes(64)), UNSUPPORTED), ("norm", dict(n_axes=2), INVALID),
    ("norm", dict(n_axes=2, pair_axis=bytes([2] * 64)), INVALID), ("norm", dict(q=None), INVALID),
    ("norm", dict(pos=None), INVALID), ("norm", dict(q_stride=3583), INVALID), ("norm", dict(k_stride=508), INVALID),
    ("norm", dict(q_stride=3588), INVALID), ("norm", dict(q=FAKE + 8), INVALID), ("norm", dict(q_weight=8), INVALID),
    ("norm", dict(q_out=FAKE), INVALID), ("norm", dict(k_out=FAKE + 1024), INVALID),
    ("norm", dict(k_out=3 * FAKE + 16), INVALID), ("norm", dict(heads=70000, q_stride=1 << 24), UNSUPPORTED),
    ("append", dict(d=32), UNSUPPORTED), ("append", dict(heads=30), INVALID), ("append", dict(page_size=48), UNSUPPORTED),
    ("append", dict(page_size=256), UNSUPPORTED), ("append", dict(num_pages=0), INVALID),
    ("append", dict(max_pages=0), INVALID), ("append", dict(num_pages=1 << 30), UNSUPPORTED),
    ("append", dict(max_pages=1 << 25), UNSUPPORTED), ("append", dict(tokens=3), INVALID),
    ("append", dict(batch=-1), INVALID), ("append", dict(n_axes=2, pair_axis=bytes(64)), INVALID),
    ("append", dict(v=None), INVALID), ("append", dict(start=None), INVALID), ("append", dict(q_out=None), INVALID),
    ("append", dict(v_stride=256), INVALID), ("append", dict(k_pages=FAKE + 4), INVALID),
    ("append", dict(start=FAKE + 2), INVALID), ("append", dict(q_out=FAKE + 16), INVALID),
    ("append", dict(pairing=3), INVALID), ("append", dict(eps=math.inf), INVALID),
    ("decode", dict(d=256), UNSUPPORTED), ("decode", dict(alpha=0.0), INVALID), ("decode", dict(heads=36), UNSUPPORTED),
    ("decode", dict(heads=27), INVALID), ("decode", dict(page_size=8), UNSUPPORTED), ("decode", dict(batch=-1), INVALID),
    ("decode", dict(kv_len=None), INVALID), ("decode", dict(out=FAKE + 2), INVALID),
    ("decode", dict(selected=FAKE, n_select=0), INVALID), ("decode", dict(selected=FAKE + 2, n_select=4), INVALID),
    ("decode", dict(q_stride=3580), INVALID), ("decode", dict(lse=FAKE + 1), INVALID),
    ("decode", dict(workspace_bytes=1000), INVALID), ("decode", dict(workspace=None), INVALID),
    ("decode", dict(workspace=FAKE + 8), INVALID),
    ("select", dict(n_select=0), INVALID), ("select", dict(n_first=5, n_last=4), INVALID),
    ("select", dict(n_first=-1), INVALID), ("select", dict(batch=20000), UNSUPPORTED),
    ("select", dict(bounds=None), INVALID), ("select", dict(heads=40), UNSUPPORTED),
    ("select", dict(workspace_bytes=2 * 4 * 16 * 8 - 1), INVALID), ("select", dict(q=FAKE + 4), INVALID),
])
def test_refusals(call, change, status):
    fn, cls, good = CALLS[call]
    assert _status(fn, cls(**dict(good, **change))) == status
    assert atf.atf_last_error()


@pytest.mark.parametrize("call,change", [
    ("norm", dict(tokens=0)), ("append", dict(tokens=0, batch=0)), ("append", dict(tokens=0, cu=FAKE)),
    ("decode", dict(batch=0)), ("select", dict(batch=0))])
def test_empty_calls_are_no_ops(call, change):
    fn, cls, good = CALLS[call]
    assert _status(fn, cls(**dict(good, **change))) == atf.ATF_OK


@pytest.mark.parametrize("call", list(CALLS))
def test_valid_calls_without_a_gpu_fail_loudly(call):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    fn, cls, good = CALLS[call]
    assert _status(fn, cls(**good)) == atf.ATF_ERR_CUDA


def test_bindings_refuse_wrong_tensors():
    q = torch.zeros(2, 28, 128, dtype=torch.bfloat16)
    kp, vp = torch.zeros(8, 4, 8, 16, 16, dtype=torch.bfloat16), torch.zeros(8, 4, 16, 128, dtype=torch.bfloat16)
    table, lens = torch.zeros(2, 4, dtype=torch.int32), torch.ones(2, dtype=torch.int32)
    ws = torch.zeros(1 << 22, dtype=torch.uint8)
    for bad in (dict(q=q.float()), dict(q=q.transpose(1, 2)), dict(kv_len=lens.long()), dict(kv_len=lens[:1]),
                dict(v_pages=vp[:4]), dict(page_table=table.long()), dict(lse=torch.zeros(2, 28).double()),
                dict(selected=torch.zeros(2, 3, 5, dtype=torch.int32)), dict()):  # the last: not on a GPU
        a = dict(dict(q=q, k_pages=kp, v_pages=vp, page_table=table, kv_len=lens, theta=1e4, alpha=1.0, workspace=ws),
                 **bad)
        with pytest.raises(TypeError):
            atf.paged_decode(**a)
    with pytest.raises(TypeError):
        atf.qk_norm_rope(q, q[:1, :4], 1e4, torch.zeros(1, 2, dtype=torch.int64))
    with pytest.raises(TypeError):
        atf.qk_norm_rope(q, q[:, :4], 1e4, torch.zeros(1, 2, dtype=torch.int32))
    with pytest.raises(TypeError):
        atf.qk_norm_rope(q, q[:, :4], 1e4, torch.zeros(2, 2, dtype=torch.int64), pair_axis=[0] * 63)
    pos = torch.zeros(2, 2, dtype=torch.int64)
    for axis, match in (([0] * 63 + [300], "300"), ([0] * 63 + ["x"], "int"), (5, "sequence")):
        with pytest.raises(TypeError, match=match):
            atf.qk_norm_rope(q, q[:, :4], 1e4, pos, pair_axis=axis)
    with pytest.raises(TypeError, match="workspace"):
        atf.paged_decode(q, kp, vp, table, lens, 1e4, 1.0, workspace=ws[::2])
    with pytest.raises(TypeError, match="n_select"):
        atf.page_select(q, torch.zeros(8, 4, 2, 128, dtype=torch.bfloat16), table, lens, 16, 1 << 40, 1e4, 1.0)
    with pytest.raises(TypeError, match="a tensor is expected"):
        atf.paged_decode(q, kp, vp, table, [1, 2], 1e4, 1.0)
    with pytest.raises(TypeError, match="CUDA device"):
        atf.qk_norm_rope(q, q[:, :4], 1e4, pos[:1])
    with pytest.raises(TypeError):
        atf.page_select(q, torch.zeros(8, 4, 2, 64, dtype=torch.bfloat16), table, lens, 16, 4, 1e4, 1.0)


# ------------------------------------------------------------------ the decode's division of its work

CTAS = 148


def _cdiv0(a, b):  # C's division, towards zero
    return a // b if a >= 0 else -(-a // b)


class Walk:
    """The producer's walk over the tile list, in the kernel's integer arithmetic."""

    def __init__(self, lens, hkv, d, theta, alpha, page, n_sel=None):
        self.w = [min(2 ** 31 - 1, int(x)) for x in oracle.windows(d, theta, alpha)[0]]
        self.nc, self.lens, self.hkv, self.page, self.n_sel = d // 16, lens, hkv, page, n_sel
        self.tile = 64 if d == 128 or max(lens) * len(lens) * hkv < 8 * 64 * CTAS else 128

    def tiles(self, n):
        keys = n if self.n_sel is None else min(self.n_sel, -(-n // self.page)) * self.page
        return max(1, -(-keys // self.tile))

    def weight(self, n, t):
        x = 2 * self.nc * t + (16 * t + (64 if t else 0)) * 64 // self.tile
        if self.n_sel is None:
            x -= sum(min(t, max(0, _cdiv0(n - self.w[8 * c + 7] - 1, self.tile))) for c in range(self.nc))
        return x

    def at(self, n, x):
        lo, hi = 0, self.tiles(n)
        while lo < hi:  # 32 points at a time, one of them at or above the answer
            step = (hi - lo + 32) // 32
            points = [min(hi, lo + lane * step + step - 1) for lane in range(32)]
            first = next(i for i, t in enumerate(points) if t >= hi or self.weight(n, t) >= x)
            lo, hi = lo + first * step, min(hi, lo + first * step + step - 1)
        assert self.weight(n, lo) >= x and (lo == 0 or self.weight(n, lo - 1) < x)
        return lo

    def run(self):
        """(pieces [cta, b, hk, t0, t1, slot], metas {cta: (b, hk, last)})."""
        units = [self.weight(n, self.tiles(n)) for n in self.lens]
        total = sum(units) * self.hkv
        bound = [total // CTAS * j + total % CTAS * j // CTAS for j in range(CTAS + 1)]
        pieces, metas = [], {}
        for cta in range(CTAS):
            lo, hi = bound[cta], bound[cta + 1]
            if lo >= hi:
                continue
            b, base = 0, 0
            while lo >= base + units[b] * self.hkv:
                base += units[b] * self.hkv
                b += 1
            hk = (lo - base) // units[b]
            base += hk * units[b]
            while b < len(self.lens) and base < hi:
                n, u = self.lens[b], units[b]
                t0 = self.at(n, lo - base) if lo > base else 0
                t1 = self.tiles(n) if hi >= base + u else self.at(n, hi - base)
                if t0 < t1:
                    slot = 0 if t0 > 0 else -1 if t1 == self.tiles(n) else 1
                    pieces.append((cta, b, hk, t0, t1, slot))
                    if slot == 1:
                        x = base + self.weight(n, self.tiles(n) - 1)
                        metas[cta] = (b, hk, max(j for j in range(CTAS) if bound[j] <= x))
                base += u
                hk += 1
                if hk == self.hkv:
                    hk, b = 0, b + 1
        return pieces, metas


@pytest.mark.parametrize("seed", range(40))
def test_decode_pieces_cover_every_tile_once_and_join(seed):
    r = random.Random(seed)
    d, hkv, page = r.choice([64, 128]), r.choice([1, 2, 3, 4, 8]), r.choice([16, 32, 64, 128])
    B = r.choice([1, 1, 2, 5, 40, 170])
    top = r.choice([1, 127, 129, 5000, 200000])
    lens = [r.choice([0, 1, r.randint(0, top), top]) for _ in range(B)]
    walk = Walk(lens, hkv, d, r.choice([1.0001, 1e4, 1e7]), r.choice([0.1, 1.0, math.inf]), page,
                r.choice([None, None, 1, 20]))
    pieces, metas = walk.run()
    done = {}
    for cta, b, hk, t0, t1, slot in pieces:
        done.setdefault((b, hk), []).append((t0, t1, cta, slot))
    assert set(done) == {(b, hk) for b in range(B) for hk in range(hkv)}
    for (b, hk), parts in done.items():
        assert parts[0][0] == 0 and parts[-1][1] == walk.tiles(lens[b])
        assert all(x[1] == y[0] and x[2] < y[2] for x, y in zip(parts, parts[1:]))
        if len(parts) == 1:
            assert parts[0][3] == -1
        else:  # begun in slot 1 of one CTA, continued in slot 0 of others, all named by its meta
            assert [s for *_, s in parts] == [1] + [0] * (len(parts) - 1)
            assert metas[parts[0][2]] == (b, hk, parts[-1][2])
            # the CTAs between that hold no piece of it hold no piece at all: their slot 0 is empty
            between = set(range(parts[0][2] + 1, parts[-1][2] + 1)) - {x[2] for x in parts}
            assert not between & {c for c, *_ in pieces}
    used = [(cta, slot) for cta, *_, slot in pieces if slot >= 0]
    assert len(used) == len(set(used))  # a CTA's two partial slots hold one piece each
    assert sum(len(v) > 1 for v in done.values()) == len(metas)


def test_tile_weights_count_the_live_chunks():
    for d, theta, alpha, n in [(128, 1e7, 1.0, 70000), (64, 1e4, 0.5, 9001), (128, 1.0001, 0.1, 400), (64, 1e4, 1.0, 1)]:
        walk = Walk([n], 1, d, theta, alpha, 64)
        for t in range(walk.tiles(n)):
            near = n - 1 - (min(n, (t + 1) * walk.tile) - 1)
            live = sum(1 for c in range(d // 16) if near <= walk.w[8 * c + 7])
            assert walk.weight(n, t + 1) - walk.weight(n, t) == d // 16 + live + (16 if t else 80) * 64 // walk.tile


@pytest.mark.parametrize("seed", range(30))
def test_append_items_fit_the_launch(seed):
    """One CTA per (sequence, page) of the new tokens: the launched count holds them all."""
    r = random.Random(seed)
    page, B = r.choice([16, 32, 64, 128]), r.randint(1, 50)
    new = [r.choice([0, 1, r.randint(0, 700)]) for _ in range(B)]
    start = [r.randint(0, 400) for _ in range(B)]
    items = sum((s + n - 1) // page - s // page + 1 for s, n in zip(start, new) if n)
    T = sum(new)
    assert items <= T // page + 2 * min(B, T)
