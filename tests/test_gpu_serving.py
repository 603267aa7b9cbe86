"""Paged serving operators on the GPU against plain implementations in 64 bits.

Tolerances count roundings of at most u = eps / 2 relative to a value
(2^-8 for bf16, 2^-24 for fp32 and every fp32 step inside a kernel).

qk_norm_rope, paged_append: the result is rounded once (u of the type).  Before
that, in fp32: the sum of squares (128 terms in chains and a tree of at most 21
additions, halved by the square root: 11), its mean and eps (2), rsqrt (4),
times gain and value (2), the phase rounded to fp32 (pi / 2), sine and cosine
(2), products and sum (3): 26 steps relative to |a| + |b| of the pair; 32 are
allowed.

paged_attention: a score is off by at most d = (hd + 2) 2^-24 scale sum |q||k|
(fp32 sums of exact products), a probability by 2 d + 2^-20 relative (the
exponential's argument is rounded at its own size, at most |score| + |max|,
which d covers, and the exponential itself to 2^-21), and for bf16 by u more
when it is rounded for the product with V.  Each of the n additions over the
keys, and each join of two pieces, adds 2^-24.  With A = sum p |v|, out is off by
at most u |out| + (2 d + 2^-20 + u_p + (n + 16) 2^-24) A, twice the middle part
because the divisor is off too; lse by 2 d + 2^-20 + (n + 16) 2^-24 + 2^-23 |lse|.
"""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import block_text_diffusion_b200 as dg  # noqa: E402

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    dg.lib()


def u_of(dtype):
    return torch.finfo(dtype).eps / 2


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape, dtype=F32, std=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def freqs(rot, **kw):
    w, amp = dg.rope_frequencies(rot, **kw)
    return torch.tensor(w, dtype=torch.float64, device="cuda"), amp


# -- norm and rotation -------------------------------------------------------------

def turned(x, pos, gain=None, eps=None, w=None, interleaved=False, amp=1.0):
    """(result, |a| + |b| of each component's pair) in 64 bits."""
    y = x.double()
    if eps is not None:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps)
        if gain is not None:
            y = y * gain.double()
    mag = y.abs()
    if w is None or w.numel() == 0:
        return y, mag
    rot = 2 * w.numel()
    t = pos.double()[:, None] * w[None]
    c, s = (amp * torch.cos(t))[:, None], (amp * torch.sin(t))[:, None]
    ia = torch.arange(0, rot, 2) if interleaved else torch.arange(rot // 2)
    ib = ia + 1 if interleaved else ia + rot // 2
    out = y.clone()
    a, b = y[..., ia], y[..., ib]
    out[..., ia], out[..., ib] = a * c - b * s, b * c + a * s
    mag = mag.clone()
    mag[..., ia] = mag[..., ib] = amp * (a.abs() + b.abs())
    return out, mag


def near_turned(got, want, mag):
    tol = u_of(got.dtype) * want.abs() + 32 * 2.0 ** -24 * mag
    assert torch.all((got.double() - want).abs() <= tol), ((got.double() - want).abs() / (tol + 1e-300)).max()


# dtype, tokens, Hq, Hkv, hd, rot, interleaved, view ("fused" columns of one
# projection, "odd" rows off the 16-byte grid, "own" tensors)
ROPE = [
    (BF, 1, 1, 1, 128, 128, False, "own"), (BF, 37, 8, 2, 128, 128, False, "fused"),
    (BF, 300, 16, 8, 128, 64, False, "fused"), (BF, 129, 5, 3, 64, 64, True, "own"),
    (BF, 2100, 3, 1, 64, 32, True, "fused"), (BF, 11, 2, 2, 256, 256, False, "own"),
    (BF, 9, 3, 1, 128, 128, False, "odd"), (BF, 17, 2, 1, 66, 20, True, "own"), (BF, 5, 2, 2, 128, 24, False, "own"),
    (F32, 1, 4, 4, 64, 64, False, "own"), (F32, 333, 4, 4, 64, 32, True, "fused"),
    (F32, 1500, 6, 2, 128, 128, False, "fused"), (F32, 13, 3, 2, 128, 64, False, "odd"),
    (F32, 6, 2, 1, 2, 2, False, "own"), (F32, 4, 1, 1, 16, 0, False, "own"), (F32, 21, 2, 2, 256, 128, True, "own"),
]


@pytest.mark.parametrize("case", ROPE, ids=str)
def test_norm_rope(case):
    dtype, t, hq, hk, hd, rot, inter, view = case
    g = gen(t + hq + hd)
    if view == "fused":
        qkv = randn(g, t, (hq + hk) * hd + 8, dtype=dtype)
        q, k = qkv[:, :hq * hd].view(t, hq, hd), qkv[:, hq * hd:(hq + hk) * hd].view(t, hk, hd)
    elif view == "odd":
        q = randn(g, t, hq, hd + 3, dtype=dtype)[:, :, 1:hd + 1]
        k = randn(g, t, hk, hd + 3, dtype=dtype)[:, :, 3:]
    else:
        q, k = randn(g, t, hq, hd, dtype=dtype, std=3.0), randn(g, hk, t, hd, dtype=dtype).transpose(0, 1)
    pos = torch.randint(-1000, 1000000, (t,), generator=g, device="cuda", dtype=torch.int32)
    w, amp = freqs(rot, scaling="yarn", factor=8.0, original_len=4096) if rot > 2 else \
        (torch.ones(rot // 2, dtype=torch.float64, device="cuda"), 1.0)
    qg, kg = 1 + randn(g, hd, dtype=dtype, std=0.2), 1 + randn(g, hd, dtype=dtype, std=0.2)
    rope = dg.Rope(w, interleaved=inter, amplitude=amp)
    # amplitude reaches the kernel as fp32
    amp = float(np.float32(amp))
    for norm, eps, gains in ((dg.HeadNorm(1e-6, qg, kg), float(np.float32(1e-6)), (qg, kg)),
                             (dg.HeadNorm(0.5), 0.5, (None, None)), (None, None, (None, None))):
        qo = torch.full((t, hq, hd), float("nan"), dtype=dtype, device="cuda")
        ko = torch.full((t, hk, hd), float("nan"), dtype=dtype, device="cuda")
        dg.qk_norm_rope(q, k, pos, qo, ko, rope=rope, norm=norm)
        near_turned(qo, *turned(q, pos, gains[0], eps, w, inter, amp))
        near_turned(ko, *turned(k, pos, gains[1], eps, w, inter, amp))
    # one side alone, no rotation, in place
    q2 = q.clone(memory_format=torch.contiguous_format)
    dg.qk_norm_rope(q2, None, None, q2, None, norm=dg.HeadNorm(1e-6, qg))
    near_turned(q2, *turned(q, pos, qg, float(np.float32(1e-6))))
    k2 = k.clone(memory_format=torch.contiguous_format)
    dg.qk_norm_rope(None, k2, pos, None, k2, rope=rope)
    near_turned(k2, *turned(k, pos, w=w, interleaved=inter, amp=amp))


def test_norm_rope_special_rows():
    # a zero row stays zero (eps > 0), a row with an infinity touches no other row
    x = randn(gen(1), 3, 2, 64, dtype=BF)
    x[0] = 0
    x[1, 0, 5] = float("inf")
    out = torch.empty_like(x)
    w, _ = freqs(64)
    pos = i32([3, 4, 5])
    dg.qk_norm_rope(x, None, pos, out, None, rope=dg.Rope(w), norm=dg.HeadNorm(1e-6))
    assert torch.all(out[0] == 0)
    want, mag = turned(x, pos, None, float(np.float32(1e-6)), w)
    near_turned(out[1, 1:], want[1, 1:], mag[1, 1:])
    near_turned(out[2], want[2], mag[2])


# -- append ------------------------------------------------------------------------

class Batch:
    """A ragged batch with shuffled pages, its host copy, and a cache around it."""

    def __init__(self, seed, dtype, hk, hd, page, new, past, prefix=0, extra_pages=2, spare_rows=0, fill=None):
        g, rng = gen(seed), np.random.default_rng(seed)
        self.new, self.kv = list(new), [p + n for p, n in zip(past, new)]
        self.prefix, self.page, self.hk, self.hd = prefix, page, hk, hd
        need = [-(-x // page) for x in self.kv]
        n_prefix = -(-prefix // page)
        self.n_pages = sum(need) + n_prefix + extra_pages
        order = rng.permutation(self.n_pages).astype(np.int32)
        self.prefix_ids = order[:n_prefix]
        # entries past the needed pages lie outside the cache: they must not be read
        self.table = np.full((len(new), max(need + [0]) + 1), self.n_pages + 7, dtype=np.int32)
        at = n_prefix
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.cu = np.concatenate([[0], np.cumsum(self.new)]).astype(np.int32)
        self.rows = int(self.cu[-1]) + spare_rows
        shape = (self.n_pages, hk, page, hd)
        self.k, self.v = randn(g, *shape, dtype=dtype), randn(g, *shape, dtype=dtype)
        if fill is not None:   # everything that belongs to no token
            live = torch.zeros(self.n_pages, page, dtype=torch.bool, device="cuda")
            for at_, off in self.slots_of_prefix() + [s for b in range(len(new)) for s in self.slots(b)]:
                live[at_, off] = True
            dead = ~live[:, None, :, None].expand(shape)
            self.k[dead] = fill
            self.v[dead] = fill
        self.cache = dg.PagedKV(self.k, self.v)
        self.batch = dg.PagedBatch(i32(self.cu), i32(self.kv), i32(self.table),
                                   prefix_pages=i32(self.prefix_ids) if prefix else None, prefix_len=prefix)

    def slots(self, b):
        return [(int(self.table[b, j // self.page]), j % self.page) for j in range(self.kv[b])]

    def slots_of_prefix(self):
        return [(int(self.prefix_ids[j // self.page]), j % self.page) for j in range(self.prefix)]

    def keys(self, b):
        """Keys and values a sequence can see, the prefix first: [n, hk, hd]."""
        s = self.slots_of_prefix() + self.slots(b)
        if not s:
            z = torch.zeros(0, self.hk, self.hd, dtype=torch.float64, device="cuda")
            return z, z
        at, off = torch.tensor(s, device="cuda").t()
        return self.k[at, :, off].double(), self.v[at, :, off].double()


APPEND = [
    # dtype, Hq, Hkv, hd, page, rot, interleaved, new, past, prefix
    (BF, 4, 2, 128, 64, 128, False, [1, 1, 1], [0, 63, 64], 0),
    (BF, 16, 8, 128, 16, 64, False, [5, 0, 300, 1], [11, 7, 100, 15], 70),
    (BF, 3, 1, 64, 256, 64, True, [2, 255, 1], [255, 0, 0], 0),
    (BF, 2, 2, 66, 32, 22, True, [33, 1], [0, 31], 5),
    (F32, 4, 4, 64, 16, 64, False, [17, 1, 64], [0, 16, 3], 33),
    (F32, 2, 1, 128, 128, 128, True, [129], [127], 0),
    (F32, 0, 3, 64, 32, 0, False, [1] * 70, list(range(70)), 0),
    (BF, 2, 1, 64, 16, 64, False, [1, 0, 2] * 700, [3, 1, 14] * 700, 9),
]


@pytest.mark.parametrize("case", APPEND, ids=lambda c: f"{len(c[7])}x{max(c[7])}-{c[1]}-{c[2]}-{c[3]}")
def test_append(case):
    dtype, hq, hk, hd, page, rot, inter, new, past, prefix = case
    b = Batch(len(new) + hd, dtype, hk, hd, page, new, past, prefix, spare_rows=3)
    g = gen(7)
    t = b.rows
    qkv = randn(g, t, (hq + 2 * hk) * hd, dtype=dtype)
    q, k, v = (x.view(t, -1, hd) for x in qkv.split([hq * hd, hk * hd, hk * hd], dim=1))
    w = freqs(rot)[0] if rot else torch.empty(0, dtype=torch.float64, device="cuda")
    qg, kg = 1 + randn(g, hd, dtype=dtype, std=0.2), 1 + randn(g, hd, dtype=dtype, std=0.2)
    q_out = torch.full((t, hq, hd), 7.0, dtype=dtype, device="cuda")
    k0, v0, status = b.k.clone(), b.v.clone(), i32([0])
    dg.paged_append(b.cache, b.batch, k, v, rope=dg.Rope(w, interleaved=inter), norm=dg.HeadNorm(1e-6, qg, kg),
                    q=q if hq else None, q_out=q_out if hq else None, status=status)
    assert int(status) == 0
    n = int(b.cu[-1])
    slots = [s for i in range(len(new)) for s in b.slots(i)[b.kv[i] - new[i]:]]
    pos = torch.tensor([prefix + j for i in range(len(new)) for j in range(past[i], past[i] + new[i])], device="cuda")
    at, off = torch.tensor(slots, device="cuda").t()
    eps = float(np.float32(1e-6))
    near_turned(b.k[at, :, off], *turned(k[:n], pos, kg, eps, w, inter))
    assert torch.equal(b.v[at, :, off], v[:n])
    if hq:
        near_turned(q_out[:n], *turned(q[:n], pos, qg, eps, w, inter))
        assert torch.all(q_out[n:] == 7.0)
    # every other slot is as it was
    k0[at, :, off], v0[at, :, off] = b.k[at, :, off], b.v[at, :, off]
    assert torch.equal(k0, b.k) and torch.equal(v0, b.v)


def test_append_reports_and_skips_bad_slots():
    b = Batch(3, BF, 1, 64, 16, [2, 2, 2], [15, 15, 0])
    # sequence 0: its second page does not exist; 1: sound; 2: fewer tokens in the cache than new ones
    table, kv = b.table.copy(), list(b.kv)
    table[0, 1] = b.n_pages
    kv[2] = 1
    batch = dg.PagedBatch(i32(b.cu), i32(kv), i32(table))
    k, v = randn(gen(1), 6, 1, 64, dtype=BF), randn(gen(2), 6, 1, 64, dtype=BF)
    k0, status = b.k.clone(), i32([0])
    dg.paged_append(b.cache, batch, k, v, status=status)
    assert int(status) == 5
    k0[table[0, 0], 0, 15] = k[0, 0]
    k0[table[1, 0], 0, 15] = k[2, 0]
    k0[table[1, 1], 0, 0] = k[3, 0]
    k0[table[2, 0], 0, 0] = k[5, 0]
    assert torch.equal(k0, b.k)


# -- attention ---------------------------------------------------------------------

def attend(b, q, causal, scale, dtype):
    """(out, lse, tolerance of out, tolerance of lse) in 64 bits."""
    hq, hd = q.shape[1], q.shape[2]
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(q.shape[:2], dtype=torch.float64, device="cuda")
    t_out, t_lse = torch.zeros_like(out), torch.zeros_like(lse)
    u, up = u_of(dtype), (2.0 ** -8 if dtype == BF else 0.0)
    for i, n in enumerate(b.new):
        if n == 0:
            continue
        k, v = (x.repeat_interleave(hq // b.hk, dim=1) for x in b.keys(i))
        r = slice(int(b.cu[i]), int(b.cu[i]) + n)
        x = q[r].double()
        s = scale * torch.einsum("qhd,khd->hqk", x, k)
        d = (hd + 2) * 2.0 ** -24 * scale * torch.einsum("qhd,khd->hqk", x.abs(), k.abs())
        if causal:
            key = torch.arange(k.shape[0], device="cuda")
            own = b.kv[i] - n + torch.arange(n, device="cuda")
            hide = key[None] > torch.where(own >= 0, b.prefix + own, torch.full_like(own, b.prefix - 1))[:, None]
            s = s.masked_fill(hide, -math.inf)
            d = d.masked_fill(hide, 0.0)
        l = torch.logsumexp(s, dim=-1) if k.shape[0] else torch.full((hq, n), -math.inf, device="cuda")
        p = torch.nan_to_num(torch.exp(s - l[..., None]), nan=0.0)
        d = d.amax(dim=-1) if k.shape[0] else torch.zeros_like(l)
        o, a = torch.einsum("hqk,khd->qhd", p, v), torch.einsum("hqk,khd->qhd", p, v.abs())
        e = 2 * d + 2.0 ** -20 + (k.shape[0] + 16) * 2.0 ** -24
        out[r], lse[r] = o, l.t()
        t_out[r] = u * o.abs() + (2 * e + up).t()[..., None] * a
        t_lse[r] = (e + 2.0 ** -23 * torch.nan_to_num(l, neginf=0.0).abs()).t()
    return out, lse, t_out, t_lse


def check_attention(b, q, causal, dtype, scale=None, q_view=None, out_view=None, workspace=None, status_want=0):
    t, hq, hd = q.shape
    scale = 1 / math.sqrt(hd) if scale is None else scale
    out = torch.full((t, hq, hd), 3.0, dtype=dtype, device="cuda") if out_view is None else out_view
    lse, status = torch.full((t, hq), 3.0, device="cuda"), i32([0])
    dg.paged_attention(b.cache, b.batch, q if q_view is None else q_view, out, scale=scale, causal=causal, lse=lse,
                       workspace=workspace, status=status)
    assert int(status) == status_want
    want, want_lse, t_out, t_lse = attend(b, q, causal, float(np.float32(scale)), dtype)
    n = int(b.cu[-1])
    assert torch.all(out[n:] == 3.0) and torch.all(lse[n:] == 3.0)   # rows behind the last sequence
    none = want_lse[:n] == -math.inf
    assert torch.equal(lse[:n] == -math.inf, none) and torch.all(out[:n][none] == 0)
    d = (out[:n].double() - want[:n]).abs()
    assert torch.all(d <= t_out[:n]), (d / (t_out[:n] + 1e-300)).max()
    d = torch.where(none, 0.0, (lse[:n].double() - want_lse[:n]).abs())
    assert torch.all(d <= t_lse[:n]), (d / t_lse[:n]).max()
    return out, lse


ATTN = [
    # Hq, Hkv, hd, page, causal, new, past, prefix
    (1, 1, 128, 64, True, [1], [0], 0),
    (4, 4, 64, 16, False, [256], [64], 0),
    (8, 2, 128, 128, True, [1], [5000], 0),
    (16, 8, 128, 64, True, [1] * 9, [0, 1, 63, 64, 127, 128, 129, 700, 333], 200),
    (5, 1, 64, 32, True, [1, 3, 0, 130], [40, 500, 3, 0], 128),
    (6, 2, 128, 16, False, [256, 1, 77], [0, 900, 13], 1),
    (16, 2, 128, 256, False, [256, 256], [0, 256], 1000),
    (3, 3, 128, 256, True, [513], [0], 0),
    (24, 3, 64, 128, True, [40, 300, 1], [2000, 5, 0], 0),
    (2, 2, 128, 32, True, [200, 2], [-150, -1], 0),      # rows that see nothing
    (4, 1, 128, 64, True, [100, 9], [-60, 200], 37),     # rows that see the prefix alone
    (2, 1, 64, 16, False, [3, 5, 2], [-3, 20, -2], 0),   # sequences without a key
    (8, 8, 128, 64, True, [1] * 200, [i * 7 % 180 for i in range(200)], 0),
    # prefixes that end inside a block and a page, before few and many rows
    (4, 2, 128, 16, True, [1], [37], 129),
    (4, 2, 128, 16, True, [1], [200], 300),
    (2, 1, 64, 64, True, [2, 1], [127, 900], 3),
    (4, 1, 64, 32, False, [100], [150], 77),
    (16, 1, 128, 64, True, [64, 40], [0, 3], 1000),
    (8, 8, 128, 128, True, [200, 57, 0, 256], [33, 0, 4, 512], 513),
    (2, 2, 64, 16, True, [130, 300], [0, 1], 16),
    (8, 2, 128, 32, True, [30] * 60, [300] * 60, 0),     # several joined halves of 120 rows in one CTA
    (130, 1, 64, 16, True, [3, 1], [9, 200], 20),        # more query heads than a half tile has rows
    (2, 2, 64, 16, True, [1, 0, 3] * 500, [5, 9, 0] * 500, 3),   # more sequences than a warp looks at at once
    (4, 2, 128, 64, True, [90] * 40 + [400], [7] * 41, 0),       # many tiles in more than 32 sequences
]


def short(c):
    return "-".join(str(x) if not isinstance(x, list) else f"{len(x)}x{max(x)}" for x in c)



@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("case", ATTN, ids=short)
def test_attention(case, dtype):
    hq, hk, hd, page, causal, new, past, prefix = case
    # whatever belongs to no token is not a number
    b = Batch(hq * 100 + page, dtype, hk, hd, page, new, past, prefix, spare_rows=2, fill=float("nan"))
    q = randn(gen(hd), b.rows, hq, hd, dtype=dtype, std=1.5)
    check_attention(b, q, causal, dtype)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
def test_attention_infinite_leftovers_and_strides(dtype):
    b = Batch(11, dtype, 2, 128, 64, [70, 1], [90, 3], 65, fill=float("-inf"))
    t = b.rows
    q = randn(gen(4), t, 6, 128, dtype=dtype)
    # query rows inside a fused projection, output rows inside a wider buffer, heads outermost
    wide = randn(gen(5), t, 6 * 128 + 256, dtype=dtype)
    wide[:, 128:128 + 768] = q.view(t, -1)
    out = torch.full((6, t, 136), 3.0, dtype=dtype, device="cuda")
    check_attention(b, q, True, dtype, q_view=wide[:, 128:128 + 768].view(t, 6, 128),
                    out_view=out.transpose(0, 1)[..., :128])
    assert torch.all(out[..., 128:] == 3.0)
    # over the queries themselves
    qc = q.clone()
    check_attention(b, q, False, dtype, q_view=qc, out_view=qc)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("new", [[1], [40], [300]])
def test_attention_with_rising_and_large_scores(new, dtype):
    # every block's maximum is far above the last one's, so each moves the reference
    b = Batch(5, dtype, 2, 64, 16, new, [2500], 300)
    for i, (at, off) in enumerate(b.slots_of_prefix() + b.slots(0)):
        b.k[at, :, off] *= 0.05 + i / 400
    q = randn(gen(6), b.rows, 4, 64, dtype=dtype)
    check_attention(b, q, True, dtype, scale=1.5)
    # and falling: later blocks add next to nothing
    for i, (at, off) in enumerate(b.slots_of_prefix() + b.slots(0)):
        b.k[at, :, off] *= 1 / (0.05 + i / 400) * (8.0 - i / 400)
    check_attention(b, q, False, dtype)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("new", [[1, 1], [40, 200]])
def test_a_query_that_is_not_a_number_stays_its_own_problem(dtype, new):
    b = Batch(17, dtype, 2, 64, 16, new, [300, 9], 50)
    q = randn(gen(9), b.rows, 6, 64, dtype=dtype)
    good, good_lse = check_attention(b, q, True, dtype)
    bad = q.clone()
    bad[0, 3, 7] = float("nan")
    bad[b.rows - 1, 0, 63] = float("nan")
    out, lse = torch.empty_like(q), torch.empty(b.rows, 6, device="cuda")
    dg.paged_attention(b.cache, b.batch, bad, out, lse=lse)
    hit = torch.zeros(b.rows, 6, dtype=torch.bool, device="cuda")
    hit[0, 3] = hit[b.rows - 1, 0] = True
    assert torch.all(torch.isnan(out[hit].float())) and torch.all(torch.isnan(lse[hit]))
    assert torch.equal(out[~hit], good[~hit]) and torch.equal(lse[~hit], good_lse[~hit])


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
def test_rows_left_by_a_bad_sequence_reach_no_other(dtype):
    # ragged pieces follow full ones on the same CTA, and find their rows in place
    b = Batch(18, dtype, 2, 64, 32, [520] * 8 + [130, 37, 1, 130, 9, 260] * 6, [700] * 44, 0)
    q = randn(gen(10), b.rows, 6, 64, dtype=dtype)
    good, good_lse = check_attention(b, q, False, dtype)
    bad = q.clone()
    bad[:8 * 520] = float("nan")
    out, lse = torch.empty_like(q), torch.empty(b.rows, 6, device="cuda")
    dg.paged_attention(b.cache, b.batch, bad, out, lse=lse, causal=False)
    assert torch.all(torch.isnan(out[:8 * 520].float())) and torch.all(torch.isnan(lse[:8 * 520]))
    assert torch.equal(out[8 * 520:], good[8 * 520:]) and torch.equal(lse[8 * 520:], good_lse[8 * 520:])


def test_attention_repeats_bit_for_bit_whatever_the_workspace_holds():
    b = Batch(9, BF, 2, 128, 64, [256, 1, 30], [3000, 700, 0], 500)
    q = randn(gen(8), b.rows, 8, 128, dtype=BF)
    n = dg.paged_attention_workspace(b.rows, 8, 128, True)
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    first = check_attention(b, q, True, BF, workspace=ws)
    ws.fill_(255)
    again = check_attention(b, q, True, BF, workspace=ws)
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
def test_attention_reports_bad_pages_and_lengths(dtype):
    b = Batch(13, dtype, 1, 64, 16, [1, 1], [40, 40], fill=0.0)
    q = randn(gen(1), 2, 2, 64, dtype=dtype)
    out = torch.empty_like(q)
    for bad in (-1, b.n_pages, 1 << 30):
        table = b.table.copy()
        table[0, 1] = bad
        status = i32([0])
        dg.paged_attention(b.cache, dg.PagedBatch(i32(b.cu), i32(b.kv), i32(table)), q, out, status=status)
        assert int(status) == 5
    for kv in ([-1, 41], [41, 1 << 30]):
        status = i32([0])
        pages = torch.zeros(2, 3, dtype=torch.int32, device="cuda")
        dg.paged_attention(b.cache, dg.PagedBatch(i32(b.cu), i32(kv), pages), q, out, status=status)
        assert int(status) == 5
    check_attention(b, q, True, dtype)   # and the next call is sound


def test_prefix_is_the_same_as_own_copies():
    """One shared prefix against the same tokens in every sequence's own pages."""
    b = Batch(21, BF, 2, 128, 64, [1, 256, 5], [30, 0, 100], 400)
    q = randn(gen(2), b.rows, 8, 128, dtype=BF)
    out, lse = check_attention(b, q, True, BF)
    c = Batch(21, BF, 2, 128, 64, b.new, [p - n + 400 for p, n in zip(b.kv, b.new)], 0)
    for i in range(3):
        k, v = b.keys(i)
        at, off = torch.tensor(c.slots(i), device="cuda").t()
        c.k[at, :, off], c.v[at, :, off] = k.to(BF), v.to(BF)
    out2, lse2 = check_attention(c, q, True, BF)
    _, _, t_out, t_lse = attend(b, q, True, float(np.float32(1 / math.sqrt(128))), BF)
    assert torch.all((out.double() - out2.double()).abs() <= 2 * t_out)
    assert torch.all((lse.double() - lse2.double()).abs() <= 2 * t_lse)


def test_captured_calls_read_lengths_at_replay_and_streams_do_not_mix():
    b = Batch(31, BF, 2, 128, 16, [1, 1, 1], [600, 600, 600], 100)
    w, _ = freqs(128)
    rope, norm = dg.Rope(w), dg.HeadNorm(1e-6)
    q, k, v = (randn(gen(i), 3, h, 128, dtype=BF) for i, h in ((1, 8), (2, 2), (3, 2)))
    q2, out = torch.empty_like(q), torch.empty_like(q)
    ws = torch.empty(dg.paged_attention_workspace(3, 8, 128, True), dtype=torch.uint8, device="cuda")

    def step(ws_):
        dg.paged_append(b.cache, b.batch, k, v, rope=rope, norm=norm, q=q, q_out=q2)
        dg.paged_attention(b.cache, b.batch, q2, out, workspace=ws_)

    step(ws)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graphs = []
    with torch.cuda.stream(side):
        for ws_ in (ws, None):   # a workspace of the caller's, and one of the graph's own pool
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                step(ws_)
            graphs.append(graph)
    for kv in ([601, 17, 300], [1, 2, 601], [128, 0, 129]):
        b.batch.kv_lens.copy_(i32(kv))
        for graph in graphs:
            out.fill_(9.0)
            graph.replay()
            torch.cuda.synchronize()
            b.kv = kv
            if kv[1] == 0:   # no slot for the new token: it sees the prefix alone
                assert torch.all(torch.isfinite(out.float()))
                continue
            want, _, tol, _ = attend(b, q2, True, float(np.float32(1 / math.sqrt(128))), BF)
            assert torch.all((out.double() - want).abs() <= tol)
    del graphs
    # two calls at once on two streams, each with its own outputs and workspace
    b.kv = [601, 601, 601]
    b.batch.kv_lens.copy_(i32(b.kv))
    torch.cuda.synchronize()
    outs = [torch.empty_like(q) for _ in range(8)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for i, o in enumerate(outs):
        dg.paged_attention(b.cache, b.batch, q2, o, stream=streams[i % 2])
    torch.cuda.synchronize()
    want, _, tol, _ = attend(b, q2, True, float(np.float32(1 / math.sqrt(128))), BF)
    for o in outs:
        assert torch.all((o.double() - want).abs() <= tol)


def test_offsets_past_32_bits():
    """A cache of more than 2^31 elements, its tokens in the first and last pages."""
    page, hd = 256, 128
    n_pages = (1 << 31) // (page * hd) + 3
    k = torch.empty(n_pages, 1, page, hd, dtype=BF, device="cuda")
    v = torch.empty_like(k)
    cache = dg.PagedKV(k, v)
    b = Batch(41, BF, 1, hd, page, [300], [212], 0, extra_pages=0)
    ids = np.array([[n_pages - 1, 0]], dtype=np.int32)
    batch = dg.PagedBatch(i32(b.cu), i32(b.kv), i32(ids))
    first = dg.PagedBatch(i32([0, 512]), i32([512]), i32(ids))
    kv = [randn(gen(i), 512, 1, hd, dtype=BF) for i in (1, 2)]
    dg.paged_append(cache, first, *kv)
    assert torch.equal(k[n_pages - 1, 0], kv[0][:256, 0]) and torch.equal(v[0, 0], kv[1][256:, 0])
    at, off = torch.tensor(b.slots(0), device="cuda").t()
    b.k[at, :, off], b.v[at, :, off] = kv
    b.cache, b.batch = cache, batch
    check_attention(b, randn(gen(3), 300, 4, hd, dtype=BF), True, BF)


def test_binding_refuses_mismatched_tensors():
    b = Batch(51, BF, 2, 64, 16, [1, 1], [5, 5])
    q, k = randn(gen(1), 2, 4, 64, dtype=BF), randn(gen(2), 2, 2, 64, dtype=BF)
    w, _ = freqs(64)
    bad = [
        lambda: dg.paged_attention(b.cache, b.batch, q.float(), q),
        lambda: dg.paged_attention(b.cache, b.batch, q, q[:1]),
        lambda: dg.paged_attention(b.cache, b.batch, q[:, :3], q[:, :3]),
        lambda: dg.paged_attention(b.cache, b.batch, q, q[:, :1].expand(2, 4, 64)),
        lambda: dg.paged_attention(b.cache, b.batch, q, q, lse=torch.zeros(2, 3, device="cuda")),
        lambda: dg.paged_attention(b.cache, b.batch, q, q, status=torch.zeros(2, dtype=torch.int32, device="cuda")),
        lambda: dg.paged_attention(b.cache, b.batch, q.transpose(1, 2).contiguous().transpose(1, 2), q),
        lambda: dg.paged_append(b.cache, b.batch, k, k[:, :1]),
        lambda: dg.paged_append(b.cache, b.batch, k, k, q=q),
        lambda: dg.paged_append(b.cache, b.batch, k, k, norm=dg.HeadNorm(1e-6, None, torch.ones(63, device="cuda"))),
        lambda: dg.qk_norm_rope(q, k, None, q, k, rope=dg.Rope(w)),
        lambda: dg.qk_norm_rope(q, k, torch.zeros(3, dtype=torch.int32, device="cuda"), q, k, rope=dg.Rope(w)),
        lambda: dg.qk_norm_rope(q, k[:1], None, q, k[:1]),
        lambda: dg.qk_norm_rope(q.half(), None, None, q.half(), None),
        lambda: dg.PagedKV(b.k, b.v[:1]),
        lambda: dg.PagedKV(b.k.transpose(1, 2), b.v.transpose(1, 2)),
        lambda: dg.PagedKV(b.k[:, :, :15].contiguous(), b.v[:, :, :15].contiguous()),
        lambda: dg.PagedBatch(i32(b.cu), i32(b.kv + [1]), i32(b.table)),
        lambda: dg.PagedBatch(i32(b.cu), i32(b.kv), i32(b.table), prefix_len=3),
        lambda: dg.PagedBatch(i32(b.cu).long(), i32(b.kv), i32(b.table)),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"call {i} was taken")
    small = torch.empty(64, dtype=torch.uint8, device="cuda")
    with pytest.raises(dg.DGError):
        dg.paged_attention(b.cache, b.batch, q, q, workspace=small)
    with pytest.raises(dg.DGError):   # rows off the 16-byte grid
        x = randn(gen(3), 2, 4, 66, dtype=BF)[..., :64]
        dg.paged_attention(b.cache, b.batch, x, q)


def test_argument_objects_stay_what_they_were():
    b = Batch(52, BF, 2, 64, 16, [1, 1], [5, 5])
    q, k = randn(gen(1), 2, 4, 64, dtype=BF), randn(gen(2), 2, 2, 64, dtype=BF)
    w, _ = freqs(64)
    pos, gain = i32([0, 1]), torch.ones(64, dtype=BF, device="cuda")
    rope, norm = dg.Rope(w), dg.HeadNorm(1e-6, gain, gain)
    for thing, name in ((rope, "inv_freq"), (norm, "q_gain"), (b.cache, "k"), (b.batch, "kv_lens"), (b.batch, "prefix_len")):
        with pytest.raises(AttributeError):
            setattr(thing, name, getattr(thing, name))
    # one kind of object in another's place
    for f in (lambda: dg.qk_norm_rope(q, k, pos, q, k, rope=b.cache), lambda: dg.qk_norm_rope(q, k, pos, q, k, norm=rope),
              lambda: dg.paged_attention(rope, b.batch, q, q), lambda: dg.paged_attention(b.cache, norm, q, q)):
        with pytest.raises(AttributeError):
            f()
    # tensors that got other memory
    old = [t.data for t in (gain, w, b.k)]   # (kept: the noted addresses stay allocated)
    want = q.clone()
    gain.data = gain.clone()
    w.data = w.clone()
    b.k.data = b.k.clone()
    for f in (lambda: dg.qk_norm_rope(q, k, None, q, k, norm=norm), lambda: dg.qk_norm_rope(q, k, pos, q, k, rope=rope),
              lambda: dg.paged_attention(b.cache, b.batch, q, q), lambda: dg.paged_append(b.cache, b.batch, k, k)):
        with pytest.raises(ValueError):
            f()
    assert len(old) == 3 and torch.equal(q, want)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
def test_strides_of_single_rows_and_heads_mean_nothing(dtype):
    b = Batch(53, dtype, 1, 64, 16, [1], [40])
    for heads in (6, 1):
        x = randn(gen(heads), 1, heads, 64, dtype=dtype)
        odd = (7, 64, 1) if heads > 1 else (7, 5, 1)
        out, lse = check_attention(b, x, True, dtype)
        got, q = torch.zeros_like(x), torch.as_strided(x, x.shape, odd)
        dg.paged_attention(b.cache, b.batch, q, torch.as_strided(got, x.shape, odd))
        assert torch.equal(got, out)


def test_calls_without_rows_do_nothing():
    b = Batch(71, BF, 2, 64, 16, [1], [5])
    q, k = torch.empty(0, 4, 64, dtype=BF, device="cuda"), torch.empty(0, 2, 64, dtype=BF, device="cuda")
    none = dg.PagedBatch(i32([0]), i32([]), torch.empty(0, 1, dtype=torch.int32, device="cuda"))
    empty = dg.PagedBatch(i32([0, 0]), i32([6]), i32(b.table))
    k0 = b.k.clone()
    for batch in (none, empty):
        dg.paged_append(b.cache, batch, k, k, q=q, q_out=q)
        dg.paged_attention(b.cache, batch, q, q)
    w, _ = freqs(64)
    dg.qk_norm_rope(q, k, i32([]), q, k, rope=dg.Rope(w))
    # rows, but no sequence to own them
    x = torch.full((3, 4, 64), 2.0, dtype=BF, device="cuda")
    y = torch.full((3, 2, 64), 2.0, dtype=BF, device="cuda")
    out = torch.full_like(x, 5.0)
    for batch in (none, empty):
        dg.paged_append(b.cache, batch, y, y, q=x, q_out=out)
        dg.paged_attention(b.cache, batch, x, out)
    assert torch.all(out == 5.0) and torch.equal(b.k, k0)


# -- together ----------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
def test_canvases_then_tokens_behind_one_prompt(dtype):
    """A prompt into shared pages, two canvases of it refined in place (the same
    slots written twice, bidirectional), then single tokens (causal): each
    call's outputs against the definition on the cache as it then is, the
    cache's keys against the definition of what was appended."""
    hq, hk, hd, page, n_prompt = 8, 2, 128, 64, 130
    g = gen(61)
    w, _ = freqs(hd)
    rope = dg.Rope(w)
    qg, kg = 1 + randn(g, hd, dtype=dtype, std=0.1), 1 + randn(g, hd, dtype=dtype, std=0.1)
    norm, eps = dg.HeadNorm(1e-6, qg, kg), float(np.float32(1e-6))

    def project(t):
        qkv = randn(g, t, (hq + 2 * hk) * hd, dtype=dtype)
        return [x.view(t, -1, hd) for x in qkv.split([hq * hd, hk * hd, hk * hd], dim=1)]

    # two canvases of 256, later one token each; the prompt's pages are the prefix
    b = Batch(62, dtype, hk, hd, page, [256, 256], [0, 0], n_prompt, fill=float("nan"))
    prompt = dg.PagedBatch(i32([0, n_prompt]), i32([n_prompt]), i32(b.prefix_ids[None]))
    q, k, v = project(n_prompt)
    q_out, out = torch.empty(n_prompt, hq, hd, dtype=dtype, device="cuda"), torch.empty(n_prompt, hq, hd, dtype=dtype, device="cuda")
    dg.paged_append(b.cache, prompt, k, v, rope=rope, norm=norm, q=q, q_out=q_out)
    dg.paged_attention(b.cache, prompt, q_out, out)
    p = Batch.__new__(Batch)
    p.__dict__.update(b.__dict__)
    p.new, p.kv, p.prefix, p.cu, p.table = [n_prompt], [n_prompt], 0, [0, n_prompt], b.prefix_ids[None]
    want, _, tol, _ = attend(p, q_out, True, float(np.float32(1 / math.sqrt(hd))), dtype)
    assert torch.all((out.double() - want).abs() <= tol)

    for _ in range(2):
        q, k, v = project(512)
        q_out = torch.empty(512, hq, hd, dtype=dtype, device="cuda")
        dg.paged_append(b.cache, b.batch, k, v, rope=rope, norm=norm, q=q, q_out=q_out)
        pos = torch.arange(256, device="cuda").repeat(2) + n_prompt
        near_turned(q_out, *turned(q, pos, qg, eps, w))
        for i in range(2):
            at, off = torch.tensor(b.slots(i), device="cuda").t()
            near_turned(b.k[at, :, off], *turned(k[256 * i:256 * i + 256], pos[:256], kg, eps, w))
        # the separate norm gives the same rows
        q2, k2 = torch.empty_like(q_out), torch.empty(512, hk, hd, dtype=dtype, device="cuda")
        dg.qk_norm_rope(q, k, pos.int(), q2, k2, rope=rope, norm=norm)
        assert torch.equal(q2, q_out)
        assert torch.equal(k2[:256], b.k[torch.tensor(b.slots(0), device="cuda").t()[0], :, torch.tensor(b.slots(0), device="cuda").t()[1]])
        check_attention(b, q_out, False, dtype)

    # one token each, on pages the canvases do not use
    spare = [i for i in range(b.n_pages) if i not in set(b.table[:, :4].ravel()) | set(b.prefix_ids)]
    b.table[:, 4] = spare[:2]
    b.new, b.kv, b.cu, b.rows = [1, 1], [257, 257], np.array([0, 1, 2], dtype=np.int32), 2
    b.batch = dg.PagedBatch(i32(b.cu), i32(b.kv), i32(b.table), prefix_pages=i32(b.prefix_ids), prefix_len=n_prompt)
    q, k, v = project(2)
    q_out = torch.empty(2, hq, hd, dtype=dtype, device="cuda")
    dg.paged_append(b.cache, b.batch, k, v, rope=rope, norm=norm, q=q, q_out=q_out)
    near_turned(q_out, *turned(q, torch.full((2,), n_prompt + 256, device="cuda"), qg, eps, w))
    check_attention(b, q_out, True, dtype)
