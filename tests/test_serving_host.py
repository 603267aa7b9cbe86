"""Paged serving operators, host side (CPU only): refusals of the C entry
points and of the binding, struct layouts, rotary frequencies, and the pieces
of work the attention cuts a batch into."""
import ctypes
import math
import os
import random
import subprocess

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import block_text_diffusion_b200 as dg  # noqa: E402
from block_text_diffusion_b200 import serving as sv  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def L():
    from block_text_diffusion_b200 import build
    build.build()
    return dg.lib()


# Addresses that are aligned and never read: every call here is refused, or has
# no rows, before the device is touched.
A, BAD = 0x10000, 0x10004


def heads(p=A, ts=128, hs=128):
    return sv._Heads(p, ts, hs)


def cache(**kw):
    f = dict(k=A, v=A, dtype=1, n_pages=4, n_kv_heads=2, page_size=16, head_dim=128)
    f.update(kw)
    return sv._PagedKV(**f)


def batch(**kw):
    f = dict(n_seqs=2, n_tokens=3, cu_q=A, kv_lens=A, page_table=A, table_stride=2, max_pages=2, prefix_pages=None,
             prefix_len=0)
    f.update(kw)
    return sv._PagedBatch(**f)


def ref(x):
    return None if x is None else ctypes.byref(x)


# -- refusals ----------------------------------------------------------------------

def norm_rope(L, dtype=1, tokens=1, hq=2, hk=1, hd=128, q=heads(), qo=heads(), k=heads(), ko=heads(), pos=A, rope=None,
              norm=None):
    return L.dg_qk_norm_rope(dtype, tokens, hq, hk, hd, ref(q), ref(qo), ref(k), ref(ko), pos, ref(rope), ref(norm),
                             None)


@pytest.mark.parametrize("kw", [
    dict(dtype=2), dict(tokens=-1), dict(hq=-1), dict(hk=-1), dict(hd=0), dict(hd=127), dict(hd=258),
    dict(q=None), dict(qo=None), dict(k=None), dict(ko=None), dict(q=heads(p=0)), dict(q=heads(ts=-1)),
    dict(k=heads(hs=-128)), dict(ko=heads(ts=1 << 41)), dict(hq=70000),
    dict(rope=sv._Rope(A, 130, 0, 1.0)), dict(rope=sv._Rope(A, -2, 0, 1.0)), dict(rope=sv._Rope(A, 3, 0, 1.0)),
    dict(rope=sv._Rope(None, 128, 0, 1.0)), dict(rope=sv._Rope(BAD, 128, 0, 1.0)),
    dict(rope=sv._Rope(A, 128, 0, 1.0), pos=None), dict(norm=sv._HeadNorm(1, -1.0, None, None)),
    dict(norm=sv._HeadNorm(1, float("nan"), None, None)),
])
def test_norm_rope_refuses(L, kw):
    assert norm_rope(L, **kw) == 1


def test_norm_rope_without_rows_is_ok(L):
    assert norm_rope(L, tokens=0) == 0
    assert norm_rope(L, hq=0, hk=0, q=None, qo=None, k=None, ko=None) == 0


BAD_CACHE = [dict(k=None), dict(v=None), dict(k=BAD), dict(v=BAD), dict(dtype=2), dict(n_pages=0), dict(n_kv_heads=0),
             dict(page_size=8), dict(page_size=48), dict(page_size=512), dict(n_pages=1 << 30, n_kv_heads=2)]
BAD_BATCH = [dict(n_seqs=-1), dict(n_tokens=-1), dict(cu_q=None), dict(kv_lens=None), dict(page_table=None),
             dict(table_stride=1), dict(max_pages=-1), dict(prefix_len=-1), dict(prefix_len=5),
             dict(max_pages=1 << 28, table_stride=1 << 28), dict(prefix_len=(1 << 31) - 20, prefix_pages=A)]


def append(L, c=None, b=None, k=heads(), v=heads(), rope=None, norm=None, hq=2, q=heads(), qo=heads()):
    return L.dg_paged_append(ref(c or cache()), ref(b or batch()), ref(k), ref(v), ref(rope), ref(norm), hq, ref(q),
                             ref(qo), None, None)


def test_append_refuses(L):
    for kw in BAD_CACHE + [dict(head_dim=129), dict(head_dim=258), dict(head_dim=0)]:
        assert append(L, c=cache(**kw)) == 1, kw
    for kw in BAD_BATCH:
        assert append(L, b=batch(**kw)) == 1, kw
    for kw in (dict(k=None), dict(v=None), dict(q=None), dict(qo=None), dict(hq=-1), dict(k=heads(p=0)),
               dict(rope=sv._Rope(A, 256, 0, 1.0)), dict(norm=sv._HeadNorm(1, -1.0, None, None))):
        assert append(L, **kw) == 1, kw
    assert L.dg_paged_append(None, ref(batch()), ref(heads()), ref(heads()), None, None, 0, None, None, None, None) == 1
    assert append(L, b=batch(n_tokens=0)) == 0
    assert append(L, b=batch(n_seqs=0, cu_q=None, kv_lens=None, page_table=None)) == 0


def attention(L, c=None, b=None, hq=4, q=heads(), scale=0.1, out=heads(), ws=A, n=1 << 40):
    return L.dg_paged_attention(ref(c or cache()), ref(b or batch()), hq, ref(q), scale, 1, ref(out), None, ws, n, None,
                                None)


def test_attention_refuses(L):
    for kw in BAD_CACHE:
        assert attention(L, c=cache(**kw)) == 1, kw
    assert attention(L, c=cache(head_dim=96)) == 6
    assert attention(L, c=cache(head_dim=256)) == 6
    for kw in BAD_BATCH:
        assert attention(L, b=batch(**kw)) == 1, kw
    for kw in (dict(hq=0), dict(hq=3), dict(hq=-2), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")),
               dict(scale=float("inf")), dict(q=None), dict(out=None), dict(q=heads(p=BAD)), dict(out=heads(p=BAD)),
               dict(q=heads(ts=4)), dict(out=heads(hs=129)), dict(ws=None), dict(ws=A + 16), dict(n=100)):
        assert attention(L, **kw) == 1, kw
    need = L.dg_paged_attention_workspace(3, 4, 128, 0)
    assert attention(L, n=need - 1) == 1
    assert attention(L, b=batch(n_tokens=0)) == 0
    assert attention(L, b=batch(n_seqs=0, cu_q=None, kv_lens=None, page_table=None)) == 0


def test_workspace_sizes(L):
    f = L.dg_paged_attention_workspace
    assert f(-1, 4, 128, 0) == 0 and f(4, 0, 128, 0) == 0 and f(4, 4, 96, 0) == 0 and f(1 << 30, 2, 64, 0) == 0
    assert 0 < f(1, 1, 64, 0) < f(1, 1, 128, 0) < f(4096, 16, 128, 0) < f(4096, 16, 128, 1)
    # every row's first piece, for both parts
    assert f(4096, 16, 128, 1) >= 2 * 4096 * 16 * 128 * 4


def test_binding_refuses_host_tensors():
    x = torch.zeros(4, 2, 64)
    with pytest.raises(ValueError):
        dg.PagedKV(torch.zeros(2, 2, 16, 64), torch.zeros(2, 2, 16, 64))
    with pytest.raises(ValueError):
        dg.PagedBatch(torch.zeros(2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32),
                      torch.zeros(1, 1, dtype=torch.int32))
    with pytest.raises(ValueError):
        dg.Rope(torch.zeros(8, dtype=torch.float64))
    with pytest.raises(ValueError):
        dg.qk_norm_rope(x, None, None, x, None)
    with pytest.raises(ValueError):
        dg.HeadNorm(eps=-1.0)
    norm = dg.HeadNorm(eps=1e-5)
    with pytest.raises(AttributeError):   # its address was noted when it was made
        norm.q_gain = torch.ones(64)


def test_structs_match_the_header(tmp_path):
    import shutil
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    structs = {"dg_heads": sv._Heads, "dg_rope": sv._Rope, "dg_head_norm": sv._HeadNorm, "dg_paged_kv": sv._PagedKV,
               "dg_paged_batch": sv._PagedBatch}
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "dg.h"', 'int main(void) {']
    for c, py in structs.items():
        lines.append(f'  printf("{c} size %zu\\n", sizeof({c}));')
        lines += [f'  printf("{c} {f} %zu\\n", offsetof({c}, {f}));' for f, _ in py._fields_]
    src = tmp_path / "layout.c"
    src.write_text("\n".join(lines + ["  return 0;", "}"]))
    exe = str(tmp_path / "layout")
    subprocess.check_call([cc, "-I", os.path.join(ROOT, "include"), "-o", exe, str(src)])
    got = dict(l.rsplit(" ", 1) for l in subprocess.check_output([exe], text=True).splitlines())
    for c, py in structs.items():
        assert int(got[f"{c} size"]) == ctypes.sizeof(py)
        for f, _ in py._fields_:
            assert int(got[f"{c} {f}"]) == getattr(py, f).offset, (c, f)


# -- rotary frequencies ------------------------------------------------------------

def test_rope_frequencies():
    w, amp = dg.rope_frequencies(128)
    assert amp == 1.0 and len(w) == 64 and w[0] == 1.0
    assert all(abs(w[j] - math.exp(-2 * j / 128 * math.log(10000.0))) < 1e-15 for j in range(64))
    lin, amp = dg.rope_frequencies(64, scaling="linear", factor=8.0)
    assert amp == 1.0 and np.allclose(np.array(lin) * 8, dg.rope_frequencies(64)[0], rtol=1e-15, atol=0)
    # ntk: the fastest pair is kept, the slowest stretched by the factor
    ntk, amp = dg.rope_frequencies(128, scaling="ntk", factor=4.0)
    assert amp == 1.0 and ntk[0] == 1.0 and abs(w[63] / ntk[63] - 4.0) < 1e-12
    # yarn: fast pairs kept, slow ones stretched, monotone between
    y, amp = dg.rope_frequencies(128, scaling="yarn", factor=4.0, original_len=4096)
    assert abs(amp - (0.1 * math.log(4.0) + 1.0)) < 1e-15
    ratio = np.array(w) / np.array(y)
    turns = 4096 * np.array(w) / (2 * math.pi)
    assert np.all(ratio[turns > 64] == 1.0) and np.allclose(ratio[turns < 0.5], 4.0)
    assert np.all(np.diff(ratio) >= -1e-12)
    assert dg.rope_frequencies(64, scaling="yarn", factor=1.0) == dg.rope_frequencies(64)
    for kw in (dict(rot_dim=3), dict(rot_dim=0), dict(rot_dim=64, theta=0.0), dict(rot_dim=64, factor=0.5),
               dict(rot_dim=64, scaling="other"), dict(rot_dim=64, scaling="yarn", factor=2.0)):
        with pytest.raises(ValueError):
            dg.rope_frequencies(**kw)


# -- the work the attention cuts a batch into --------------------------------------

FIELDS = ("cta", "part", "seq", "q0", "row0", "rows", "kvh", "kb0", "nblk", "limit", "vis0", "vis_max", "pages",
          "first", "whole", "n_cont")


def walk(L, cu, kv, max_pages, page, hq, hk, causal, tile, prefix=0, n_tokens=None):
    cu = np.array(cu, dtype=np.int32)
    kv = np.array(kv, dtype=np.int32)
    n = len(kv)
    n_tokens = int(cu[-1]) if n_tokens is None else n_tokens
    table = np.zeros((max(n, 1), max(max_pages, 1)), dtype=np.int32)
    c = cache(n_kv_heads=hk, page_size=page)
    b = batch(n_seqs=n, n_tokens=n_tokens, cu_q=cu.ctypes.data, kv_lens=kv.ctypes.data,
              page_table=table.ctypes.data, table_stride=table.shape[1], max_pages=max_pages,
              prefix_pages=A if prefix else None, prefix_len=prefix)
    out = np.zeros((1 << 16, 16), dtype=np.int32)
    got, status = ctypes.c_int32(0), np.zeros(1, dtype=np.int32)
    st = L.dg_test_paged_walk(ref(c), ref(b), hq, int(causal), tile, status.ctypes.data, out.ctypes.data, len(out),
                              ctypes.byref(got))
    assert st == 0
    return [dict(zip(FIELDS, map(int, r))) for r in out[:got.value]], int(status[0])


def expected_tiles(cu, kv, hq, hk, causal, tile, prefix):
    """{(part, seq, kvh, row0): (rows, key blocks)} by the definition: a tile
    has the blocks up to the last key its last row sees, and one at least."""
    blk = 64 if tile == 64 else 128
    g = hq // hk
    out = {}
    seqs = [(0, b, cu[b + 1] - cu[b], kv[b]) for b in range(len(kv))]
    if prefix:
        seqs.append((1, -1, cu[-1] - cu[0], prefix))
    for part, b, nq, n_kv in seqs:
        for row0 in range(0, nq * g, tile):
            rows = min(tile, nq * g - row0)
            seen = n_kv if part or not causal else max(0, n_kv - nq + (row0 + rows - 1) // g + 1)
            for h in range(hk):
                out[part, b, h, row0] = rows, max(1, -(-seen // blk))
    return out


@pytest.mark.parametrize("tile", [256, 128, 64])
def test_walk_covers_every_block_once(L, tile):
    rng = random.Random(tile)
    for _ in range(150):
        hk = rng.choice([1, 2, 3, 8])
        hq = hk * rng.choice([1, 2, 3, 5, 8])
        n = rng.choice([1, 2, 5, 40])
        new = [rng.choice([0, 1, 1, 7, 130, 256]) for _ in range(n)]
        kv = [max(0, x + rng.choice([0, 1, 63, 500, 4000, -3])) for x in new]
        cu = [0]
        for x in new:
            cu.append(cu[-1] + x)
        page = rng.choice([16, 64, 256])
        causal, prefix = rng.random() < 0.5, rng.choice([0, 0, 1, 129, 5000])
        frags, status = walk(L, cu, kv, -(-max(kv + [1]) // page), page, hq, hk, causal, tile, prefix)
        assert status == 0
        want = expected_tiles(cu, kv, hq, hk, causal, tile, prefix)
        pieces = {}
        for f in frags:
            key = f["part"], f["seq"], f["kvh"], f["row0"]
            assert want[key][0] == f["rows"]
            assert f["q0"] == (cu[0] if f["part"] else cu[f["seq"]])
            pieces.setdefault(key, []).append(f)
        assert set(pieces) == set(want)
        for key, ps in pieces.items():
            # consecutive pieces of one tile sit in consecutive CTAs, the first knows how many follow
            assert [p["cta"] for p in ps] == list(range(ps[0]["cta"], ps[0]["cta"] + len(ps)))
            at = 0
            for p in ps:
                assert p["kb0"] == at and p["nblk"] >= 1
                at += p["nblk"]
            assert at == want[key][1]
            assert ps[0]["first"] and not any(p["first"] for p in ps[1:])
            assert ps[0]["n_cont"] == len(ps) - 1
            assert bool(ps[0]["whole"]) == (len(ps) == 1)
        # equal shares: no CTA has more than its interval, and a CTA continues at most one tile
        per = {}
        for f in frags:
            per.setdefault(f["cta"], []).append(f)
        fixed = {256: 5, 128: 2, 64: 2}[tile]            # a tile's start and end, counted in blocks
        total = sum(nb + fixed for _, nb in want.values())
        share = -(-total // 148)
        for fs in per.values():
            assert sum(f["nblk"] for f in fs) <= share
            assert not any(not f["first"] for f in fs[1:])


def test_walk_keeps_bad_lengths_in_range(L):
    """Lengths, offsets that lie, decrease or leave the buffers: every row, page
    entry and block stays inside what the caller declared, and it is reported."""
    rng = random.Random(3)
    wild = [-(1 << 31), -1, 0, 1, 5, 100, 300, 5000, (1 << 31) - 1]
    for _ in range(200):
        n = rng.choice([1, 3, 20])
        cu = [rng.choice(wild) for _ in range(n + 1)]
        kv = [rng.choice(wild) for _ in range(n)]
        max_pages, page, tokens = rng.choice([0, 1, 7]), rng.choice([16, 128]), rng.choice([1, 64, 400])
        prefix = rng.choice([0, 70])
        hk, g = rng.choice([1, 2]), rng.choice([1, 3, 8])
        frags, status = walk(L, cu, kv, max_pages, page, hk * g, hk, rng.random() < 0.5, 256, prefix, tokens)
        fair = all(0 <= a <= b <= tokens for a, b in zip(cu, cu[1:])) and all(0 <= k <= max_pages * page for k in kv)
        assert status == (0 if fair else 5)
        for f in frags:
            assert 0 <= f["kvh"] < hk and 0 <= f["cta"] < 148 and 1 <= f["rows"] <= 256
            last = f["q0"] + (f["row0"] + f["rows"] - 1) // g
            assert 0 <= f["q0"] <= last < tokens
            room = prefix if f["part"] else max_pages * page
            assert 0 <= f["limit"] <= room and f["vis_max"] <= room
            assert f["pages"] <= (-(-prefix // page) if f["part"] else max_pages)
            assert 0 <= f["kb0"] and f["kb0"] * 128 < max(1, f["limit"])
            assert 0 <= f["n_cont"] < 148
