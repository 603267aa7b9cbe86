"""The paged serving operators' contract where calls go wrong or go far: lengths
past the table, argument objects whose tensors changed, errors nobody asked
for, gradients, streams, positions near the ends of int32, kernel variants that
only many rows reach.  Tolerances as in test_gpu_serving.py unless a test
derives its own.
"""
import copy
import math
from decimal import Decimal, getcontext

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import block_text_diffusion_b200 as dg  # noqa: E402
import test_gpu_serving as base  # noqa: E402
from test_gpu_serving import BF, F32, Batch, attend, check_attention, freqs, gen, i32, near_turned, randn, turned  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    dg.lib()


# -- slots that do not exist -------------------------------------------------------

@pytest.mark.parametrize("hd", [64, 66])   # both kernels
def test_tokens_past_the_table_or_the_buffers_are_not_stored(hd):
    """A length past the table, or an offset past the rows, moves no other token:
    own token j goes to slot j or nowhere."""
    b = Batch(81, BF, 2, hd, 16, [2, 2, 3, 1, 1], [30, 15, 7, 31, 30])
    room = b.table.shape[1] * 16
    table = np.tile(np.arange(b.table.shape[1], dtype=np.int32), (5, 1)) + 3 * np.arange(5, dtype=np.int32)[:, None]
    pages = 3 * 5
    k0, v0 = randn(gen(1), pages, 2, 16, hd, dtype=BF), randn(gen(2), pages, 2, 16, hd, dtype=BF)
    cache = dg.PagedKV(k0.clone(), v0.clone())
    assert room == 48 and b.table.shape[1] == 3
    # one token with a slot and one past the table; sound; three tokens of which the buffers hold one ...
    cu, kv = [0, 2, 4, 7], [room + 1, 17, 10]
    k, v = randn(gen(3), 5, 2, hd, dtype=BF), randn(gen(4), 5, 2, hd, dtype=BF)
    q, q_out = randn(gen(5), 5, 4, hd, dtype=BF), torch.zeros(5, 4, hd, dtype=BF, device="cuda")
    w = freqs(32)[0]
    status = i32([0])
    dg.paged_append(cache, dg.PagedBatch(i32(cu), i32(kv), i32(table[:3])), k, v, rope=dg.Rope(w), q=q, q_out=q_out,
                    status=status)
    assert int(status) == 5
    slot = {0: (0, room - 1), 2: (1, 15), 3: (1, 16), 4: (2, 7)}   # row: (sequence, own token)
    rows = torch.tensor(list(slot), device="cuda")
    at = torch.tensor([int(table[s, j // 16]) for s, j in slot.values()], device="cuda")
    off = torch.tensor([j % 16 for _, j in slot.values()], device="cuda")
    pos = torch.tensor([j for _, j in slot.values()], device="cuda")
    near_turned(cache.k[at, :, off], *turned(k[rows], pos, w=w))
    near_turned(q_out[rows], *turned(q[rows], pos, w=w))
    assert torch.equal(cache.v[at, :, off], v[rows])
    k0[at, :, off], v0[at, :, off] = cache.k[at, :, off], cache.v[at, :, off]
    assert torch.equal(k0, cache.k) and torch.equal(v0, cache.v)
    # ... and lengths at the ends of int32
    for far in ((1 << 31) - 1, -(1 << 31)):
        status.zero_()
        dg.paged_append(cache, dg.PagedBatch(i32([0, 2]), i32([far]), i32(table[:1])), k[:2], v[:2], rope=dg.Rope(w),
                        status=status)
        assert int(status) == 5 and torch.equal(k0, cache.k) and torch.equal(v0, cache.v)


# -- argument objects --------------------------------------------------------------

def test_a_batch_whose_tensors_got_other_memory_is_refused():
    b = Batch(82, BF, 2, 64, 16, [1, 1], [5, 20], prefix=20)
    q, k = randn(gen(1), 2, 4, 64, dtype=BF), randn(gen(2), 2, 2, 64, dtype=BF)
    old = []   # (the noted addresses stay allocated)

    def fresh():
        return dg.PagedBatch(i32(b.cu), i32(b.kv), i32(b.table), prefix_pages=i32(b.prefix_ids), prefix_len=b.prefix)

    def refused(batch):
        k0, out = b.k.clone(), q.clone()
        for f in (lambda: dg.paged_attention(b.cache, batch, q, out), lambda: dg.paged_append(b.cache, batch, k, k)):
            with pytest.raises(ValueError):
                f()
        assert torch.equal(out, q) and torch.equal(b.k, k0)

    for name in ("cu_q", "kv_lens", "page_table", "prefix_pages"):
        batch = fresh()
        t = getattr(batch, name)
        old.append(t.data)
        t.data = t.clone()
        refused(batch)
    # at the same address, with fewer entries or another order
    for name, change in (("cu_q", lambda t: t.resize_(2)), ("kv_lens", lambda t: t.resize_(1)),
                         ("page_table", lambda t: t.resize_(2, 1)), ("page_table", lambda t: t.t_()),
                         ("prefix_pages", lambda t: t.resize_(1))):
        batch = fresh()
        change(getattr(batch, name))
        refused(batch)
    # and as it was made it is taken
    check_attention(b, q, True, BF)
    assert len(old) == 4


def test_copies_of_argument_objects_are_their_own():
    b = Batch(83, BF, 2, 64, 16, [1, 1], [5, 20], prefix=20)
    q, k = randn(gen(1), 2, 4, 64, dtype=BF), randn(gen(2), 2, 2, 64, dtype=BF)
    w, _ = freqs(64)
    gain, pos = 1 + randn(gen(3), 64, dtype=BF, std=0.2), i32([3, 9])
    first = check_attention(b, q, True, BF)
    rope, norm = dg.Rope(w, interleaved=True, amplitude=1.5), dg.HeadNorm(1e-5, gain)
    want = torch.empty_like(q)
    dg.qk_norm_rope(q, None, pos, want, None, rope=rope, norm=norm)
    for how in (copy.copy, copy.deepcopy):
        batch, cache, rope2, norm2 = how(b.batch), how(b.cache), how(rope), how(norm)
        out = torch.empty_like(q)
        dg.paged_attention(cache, batch, q, out)
        assert torch.equal(out, first[0])
        dg.qk_norm_rope(q, None, pos, out, None, rope=rope2, norm=norm2)
        assert torch.equal(out, want)
        assert (batch.kv_lens.data_ptr() == b.batch.kv_lens.data_ptr()) == (how is copy.copy)
    # the deep copy reads its own lengths and writes its own pages
    batch.kv_lens.copy_(i32([3, 21]))
    b.kv = [3, 21]
    out = torch.empty_like(q)
    dg.paged_attention(b.cache, batch, q, out)
    saved, b.batch = b.batch, batch
    assert torch.equal(check_attention(b, q, True, BF)[0], out) and not torch.equal(out, first[0])
    k0 = b.k.clone()
    dg.paged_append(cache, saved, k, k)
    assert torch.equal(b.k, k0) and not torch.equal(cache.k, k0)


def test_tensors_reshaped_in_place_are_refused():
    """The same address with another shape, order or type is not what was noted."""
    b = Batch(84, BF, 16, 64, 16, [1, 1], [5, 20])   # (16 heads, 16 slots: a transposed cache has its old shape)
    q, k = randn(gen(1), 2, 16, 64, dtype=BF), randn(gen(2), 2, 16, 64, dtype=BF)
    pos, out = i32([0, 1]), torch.zeros(2, 16, 64, dtype=BF, device="cuda")
    for change in (lambda c: c.k.transpose_(1, 2), lambda c: c.v.transpose_(1, 2), lambda c: c.k.resize_(1, 16, 16, 64),
                   lambda c: c.v.squeeze_().resize_(2, 16, 16, 64)):
        cache = dg.PagedKV(b.k.clone(), b.v.clone())
        change(cache)
        for f in (lambda: dg.paged_attention(cache, b.batch, q, out), lambda: dg.paged_append(cache, b.batch, k, k)):
            with pytest.raises(ValueError):
                f()
    rope = dg.Rope(freqs(64)[0])
    rope.inv_freq.resize_(16)
    with pytest.raises(ValueError):
        dg.qk_norm_rope(q, None, pos, out, None, rope=rope)
    assert torch.all(out == 0)


# -- errors nobody gave a word for -------------------------------------------------

def test_errors_without_a_status_word_are_kept_for_serving_status():
    try:
        dg.serving_status()
    except dg.DGError:   # what earlier tests' calls left
        pass
    b = Batch(85, BF, 2, 64, 16, [1, 1], [40, 40], prefix=20)
    q, k = randn(gen(1), 2, 4, 64, dtype=BF), randn(gen(2), 2, 2, 64, dtype=BF)
    out = torch.empty_like(q)
    table = b.table.copy()
    table[0, 2] = b.n_pages
    bad = dg.PagedBatch(i32(b.cu), i32(b.kv), i32(table))
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        dg.paged_attention(b.cache, bad, q, out)
    f32 = Batch(86, F32, 2, 64, 16, [1], [40])
    x = randn(gen(3), 1, 2, 64)
    for call in (lambda: dg.paged_append(b.cache, bad, k, k), lambda: dg.paged_attention(b.cache, bad, q, out),
                 lambda: dg.paged_attention(f32.cache, dg.PagedBatch(i32([0, 1]), i32([41]), i32([[0, -1, 0]])), x, x),
                 graph.replay):
        call()
        torch.cuda.synchronize()
        with pytest.raises(dg.DGError) as e:
            dg.serving_status()
        assert e.value.code == 5
        dg.serving_status()   # asked once, gone
    # a call with a word of its own reports there, a sound one nowhere
    word = i32([0])
    dg.paged_append(b.cache, bad, k, k, status=word)
    dg.paged_attention(b.cache, b.batch, q, out)
    assert int(word) == 5
    dg.serving_status()
    # on a stream of the caller's
    with torch.cuda.stream(side):
        dg.paged_append(b.cache, bad, k, k)
    with pytest.raises(dg.DGError):
        dg.serving_status(stream=side)
    del graph


# -- autograd ----------------------------------------------------------------------

def test_tensors_that_want_a_gradient_are_refused():
    b = Batch(87, BF, 2, 64, 16, [1, 1], [5, 20])
    q, k = randn(gen(1), 2, 4, 64, dtype=BF), randn(gen(2), 2, 2, 64, dtype=BF)
    out, k_out, lse, pos = torch.zeros_like(q), torch.zeros_like(k), torch.zeros(2, 4, device="cuda"), i32([0, 1])
    w, gain = freqs(64)[0], torch.ones(64, dtype=BF, device="cuda")
    rope, norm = dg.Rope(w), dg.HeadNorm(1e-6, gain, gain)
    calls = {
        "rope": (lambda: dg.qk_norm_rope(q, k, pos, out, k_out, rope=rope, norm=norm), (q, k, out, k_out, w, gain)),
        "append": (lambda: dg.paged_append(b.cache, b.batch, k, k_out, rope=rope, norm=norm, q=q, q_out=out),
                   (q, k, k_out, out, b.k, b.v, w, gain)),
        "attention": (lambda: dg.paged_attention(b.cache, b.batch, q, out, lse=lse), (q, out, lse, b.k, b.v)),
    }
    for name, (call, tensors) in calls.items():
        for i, t in enumerate(tensors):
            t.requires_grad_(True)
            with pytest.raises(ValueError, match="gradient"):
                call()
                pytest.fail(f"{name}: tensor {i} was taken")
            with torch.no_grad():
                call()
            with torch.inference_mode():
                call()
            t.requires_grad_(False)
        call()
    # inference tensors are taken too
    with torch.inference_mode():
        x = q.clone()
        dg.qk_norm_rope(x, None, None, x, None, norm=norm)
    dg.qk_norm_rope(x, None, None, x, None, norm=norm)


def test_written_tensors_are_seen_by_autograd():
    """What another operator saved for its backward pass and a call then wrote over
    ends that pass with an error, as any write in place does."""
    b = Batch(88, F32, 2, 64, 16, [1, 1], [5, 20])
    q, k = randn(gen(1), 2, 4, 64), randn(gen(2), 2, 2, 64)
    out, k_out, lse = torch.zeros_like(q), torch.zeros_like(k), torch.zeros(2, 4, device="cuda")
    norm = dg.HeadNorm(1e-6)
    p = torch.ones((), device="cuda", requires_grad=True)
    for call, written, read in (
            (lambda: dg.qk_norm_rope(q, k, None, out, k_out, norm=norm), (out, k_out), (q, k)),
            (lambda: dg.paged_append(b.cache, b.batch, k, k_out, q=q, q_out=out), (b.k, b.v, out), (q, k, k_out)),
            (lambda: dg.paged_attention(b.cache, b.batch, q, out, lse=lse), (out, lse), (q, b.k, b.v))):
        for t in written:
            y = (p * t).sum()
            call()
            with pytest.raises(RuntimeError, match="modified by an inplace operation"):
                y.backward()
        for t in read:
            y = (p * t).sum()
            call()
            y.backward()


# -- streams -----------------------------------------------------------------------

def test_tensors_of_a_call_on_another_stream_outlive_it():
    """A caller may drop what it passed as soon as the call returns, on whatever
    stream the call runs."""
    t, h, hd = 3001, 16, 128
    side, norm = torch.cuda.Stream(), dg.HeadNorm(1e-6)
    out, want = torch.zeros(t, h, hd, dtype=BF, device="cuda"), torch.empty(t, h, hd, dtype=BF, device="cuda")
    q = randn(gen(1), t, h, hd, dtype=BF)
    dg.qk_norm_rope(q, None, None, want, None, norm=norm)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)   # a tenth of a second
    dg.qk_norm_rope(q, None, None, out, None, norm=norm, stream=side)
    del q
    others = [torch.full((t, h, hd), 5.0, dtype=BF, device="cuda") for _ in range(3)]   # would take its memory
    torch.cuda.synchronize()
    assert torch.equal(out, want) and len(others) == 3

    # the same of an attention call's query, page table and workspace
    b = Batch(89, BF, 2, 128, 64, [300] * 8, [100] * 8)
    q = randn(gen(2), b.rows, 16, 128, dtype=BF)
    want = torch.empty_like(q)
    dg.paged_attention(b.cache, b.batch, q, want)
    out = torch.zeros_like(q)
    ws = torch.empty(dg.paged_attention_workspace(b.rows, 16, 128), dtype=torch.uint8, device="cuda")
    batch = dg.PagedBatch(i32(b.cu), i32(b.kv), i32(b.table))
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)
    dg.paged_attention(b.cache, batch, q, out, workspace=ws, stream=side)
    shapes = [(q.shape, q.dtype), (ws.shape, ws.dtype), (batch.page_table.shape, torch.int32), (batch.kv_lens.shape, torch.int32)]
    del q, ws, batch
    others = [torch.zeros(s, dtype=d, device="cuda") for s, d in shapes for _ in range(3)]
    torch.cuda.synchronize()
    assert torch.equal(out, want) and len(others) == 12


# -- far positions -----------------------------------------------------------------

def exact_turns(pos, w):
    """pos * w / (2 pi) less its whole turns, to 1e-17: the product in 60 digits."""
    getcontext().prec = 60
    inv = Decimal("0.15915494309189533576888376337251436203445964574045644874766734")
    x = Decimal(int(pos)) * Decimal(float(w)) * inv
    return float(x - x.to_integral_value())


@pytest.mark.parametrize("hd, inter", [(64, False), (64, True), (66, False)])   # (66: the kernel for any size)
def test_far_positions_keep_their_phase(hd, inter):
    """Rows (1, 0) turn into the cosine and sine themselves (the products are exact).
    The phase is rounded to fp32 once (at most 2^-26 turns, pi / 2 units of 2^-24
    radians), sine and cosine are off by at most 2 units: 3.6 together, 4 allowed,
    at every position an int32 holds."""
    top = 1 << 31
    pos = [0, 1, -1, 1 << 24, (1 << 27) - 5, -(1 << 29) + 3] + [top - 1 - 7919 * i for i in range(60)] + \
        [-top + 104729 * i for i in range(60)]
    w = freqs(64)[0].cpu()
    x = torch.zeros(len(pos), 1, hd, device="cuda")
    ia = torch.arange(0, 64, 2) if inter else torch.arange(32)
    ib = ia + 1 if inter else ia + 32
    x[..., ia] = 1.0
    out = torch.empty_like(x)
    dg.qk_norm_rope(x, None, i32(pos), out, None, rope=dg.Rope(w.cuda(), interleaved=inter))
    turns = np.array([[exact_turns(p, f) for f in w] for p in pos])
    got = out[:, 0].cpu().double().numpy()
    for at, want in ((ia, np.cos(2 * np.pi * turns)), (ib, np.sin(2 * np.pi * turns))):
        off = np.abs(got[:, at.numpy()] - want) * 2.0 ** 24
        assert off.max() <= 4.0, off.max()


# -- captured calls ----------------------------------------------------------------

def test_a_replay_whose_token_has_no_slot():
    """Lengths that change between replays, one of them below the count of new
    tokens: that token is reported and not stored, and sees the prefix alone."""
    b = Batch(91, BF, 2, 128, 16, [1, 1, 1], [600, 600, 600], 100)
    rope, norm = dg.Rope(freqs(128)[0]), dg.HeadNorm(1e-6)
    q, k, v = (randn(gen(i), 3, h, 128, dtype=BF) for i, h in ((1, 8), (2, 2), (3, 2)))
    q2, out, lse, words = torch.empty_like(q), torch.empty_like(q), torch.empty(3, 8, device="cuda"), [i32([0]), i32([0])]
    ws = torch.empty(dg.paged_attention_workspace(3, 8, 128, True), dtype=torch.uint8, device="cuda")

    def step():
        dg.paged_append(b.cache, b.batch, k, v, rope=rope, norm=norm, q=q, q_out=q2, status=words[0])
        dg.paged_attention(b.cache, b.batch, q2, out, lse=lse, workspace=ws, status=words[1])

    step()
    torch.cuda.synchronize()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        step()
    eps = float(np.float32(1e-6))
    for kv in ([601, 17, 300], [128, 0, 129], [1, 2, 601]):
        b.kv = kv
        b.batch.kv_lens.copy_(i32(kv))
        for t in (out, lse, q2):
            t.fill_(9.0)
        for t in words:
            t.zero_()
        k0, v0 = b.k.clone(), b.v.clone()
        graph.replay()
        torch.cuda.synchronize()
        assert int(words[0]) == (5 if 0 in kv else 0) and int(words[1]) == 0
        pos = torch.tensor([100 + n - 1 for n in kv], device="cuda")
        near_turned(q2, *turned(q, pos, None, eps, rope.inv_freq))
        kept = [i for i in range(3) if kv[i]]
        at, off = torch.tensor([b.slots(i)[-1] for i in kept], device="cuda").t()
        near_turned(b.k[at, :, off], *turned(k[kept], pos[kept], None, eps, rope.inv_freq))
        assert torch.equal(b.v[at, :, off], v[kept])
        k0[at, :, off], v0[at, :, off] = b.k[at, :, off], b.v[at, :, off]
        assert torch.equal(b.k, k0) and torch.equal(b.v, v0)
        want, want_lse, tol, tol_lse = attend(b, q2, True, float(np.float32(1 / math.sqrt(128))), BF)
        assert torch.all((out.double() - want).abs() <= tol)
        assert torch.all((lse.double() - want_lse).abs() <= tol_lse)
    del graph


# -- rows of no sequence, slots given twice ----------------------------------------

@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
def test_rows_of_no_sequence_are_not_written_and_have_no_effect(dtype):
    """Spare rows before the first sequence and after the last."""
    b = Batch(92, dtype, 2, 64, 16, [3, 0, 70], [20, 4, 9], prefix=33)
    n = int(b.cu[-1])
    batch = dg.PagedBatch(i32(b.cu + 4), i32(b.kv), i32(b.table), prefix_pages=i32(b.prefix_ids), prefix_len=b.prefix)
    rope, norm = dg.Rope(freqs(64)[0]), dg.HeadNorm(1e-6)
    x = [randn(gen(i), n + 9, h, 64, dtype=dtype) for i, h in ((1, 6), (2, 2), (3, 2))]
    runs = []
    for fill in (0.0, float("nan")):
        q, k, v = (t.clone() for t in x)
        for t in (q, k, v):
            t[:4], t[4 + n:] = fill, fill
        cache = dg.PagedKV(b.k.clone(), b.v.clone())
        q2, out, lse = torch.full_like(q, 3.0), torch.full_like(q, 3.0), torch.full((n + 9, 6), 3.0, device="cuda")
        word = i32([0])
        dg.paged_append(cache, batch, k, v, rope=rope, norm=norm, q=q, q_out=q2, status=word)
        dg.paged_attention(cache, batch, q2, out, lse=lse, status=word)
        assert int(word) == 0
        for t in (q2, out, lse):
            assert torch.all(t[:4] == 3.0) and torch.all(t[4 + n:] == 3.0)
        runs.append([cache.k, cache.v, q2, out, lse])
    for a, c in zip(*runs):
        assert torch.equal(a, c)
    assert torch.all(torch.isfinite(runs[0][3].float()))


def test_a_slot_given_twice_holds_parts_of_its_tokens():
    b = Batch(93, BF, 2, 64, 16, [1, 1], [5, 5])
    table = np.tile(b.table[:1], (2, 1))
    k, v = randn(gen(1), 2, 2, 64, dtype=BF), randn(gen(2), 2, 2, 64, dtype=BF)
    k0, v0 = b.k.clone(), b.v.clone()
    dg.paged_append(b.cache, dg.PagedBatch(i32([0, 1, 2]), i32([6, 6]), i32(table)), k, v)
    at = int(table[0, 0])
    for got, x in ((b.k[at, :, 5], k), (b.v[at, :, 5], v)):
        assert torch.all((got == x[0]) | (got == x[1]))
    k0[at, :, 5], v0[at, :, 5] = b.k[at, :, 5], b.v[at, :, 5]
    assert torch.equal(b.k, k0) and torch.equal(b.v, v0)


# -- kernel variants that only many rows reach -------------------------------------

# (more than 148 x 32 batches of heads: the kernel of four groups a batch; more
# heads of a kind than one of its batches holds, so a warp goes through several;
# the last heads of a batch missing)
@pytest.mark.parametrize("case", [
    (BF, 1201, 40, 2, 128, 128, True, "fused"), (BF, 701, 37, 9, 128, 64, False, "own"),
    (BF, 2500, 5, 1, 64, 32, True, "own"), (F32, 1301, 20, 4, 64, 32, True, "fused"),
    (F32, 801, 18, 3, 128, 128, False, "own"), (F32, 1601, 9, 1, 128, 128, True, "own"),
], ids=str)
def test_norm_rope_of_many_rows(case):
    base.test_norm_rope(case)


@pytest.mark.parametrize("case", [
    (BF, 20, 4, 128, 64, 128, True, [300, 501], [3, 0], 5),
    (BF, 37, 17, 128, 16, 64, False, [257, 1, 200], [0, 90, 31], 0),
    (F32, 19, 9, 64, 32, 32, True, [400, 300], [0, 17], 40),
    (F32, 0, 20, 64, 64, 64, False, [600, 1], [5, 0], 0),
], ids=lambda c: f"{len(c[7])}x{max(c[7])}-{c[1]}-{c[2]}-{c[3]}")
def test_append_of_many_rows(case):
    base.test_append(case)


# -- shapes the documentation allows and nothing above has -------------------------

@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("hq, hk, hd", [(600, 1, 64), (1030, 2, 128)])
def test_more_query_heads_than_a_tile_has_rows(dtype, hq, hk, hd):
    b = Batch(94, dtype, hk, hd, 16, [2, 1, 3], [9, 200, 0], prefix=20, fill=float("nan"))
    check_attention(b, randn(gen(1), b.rows, hq, hd, dtype=dtype, std=1.5), True, dtype)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("new", [[1] * 63 + [700], [1, 1, 1, 1500, 1]])
def test_a_prompt_beside_single_tokens(dtype, new):
    """In the tiles of 128 rows, which the average length asks for, and in those of 256."""
    past = [37 * i % 500 for i in range(len(new))]
    b = Batch(95, dtype, 2, 64, 32, new, past, prefix=100, fill=float("nan"))
    check_attention(b, randn(gen(2), b.rows, 4, 64, dtype=dtype, std=1.5), True, dtype)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("prefix", [0, 150])
def test_sequences_without_pages_of_their_own(dtype, causal, prefix):
    b = Batch(96, dtype, 2, 64, 16, [300, 1], [-300, -1], prefix=prefix, fill=float("nan"))
    b.batch = dg.PagedBatch(i32(b.cu), i32([0, 0]), torch.empty(2, 0, dtype=torch.int32, device="cuda"),
                            prefix_pages=i32(b.prefix_ids) if prefix else None, prefix_len=prefix)
    check_attention(b, randn(gen(3), b.rows, 4, 64, dtype=dtype), causal, dtype)


@pytest.mark.parametrize("hd, rot", [(128, 128), (66, 20)])
@pytest.mark.parametrize("tokens", [3, 900])
def test_append_turns_queries_in_place_in_a_fused_projection(hd, rot, tokens):
    b = Batch(97, BF, 3, hd, 16, [tokens, 1], [11, 30], prefix=5)
    qkv = randn(gen(4), b.rows, 11 * hd, dtype=BF)
    rope, norm = dg.Rope(freqs(rot)[0]), dg.HeadNorm(1e-6)
    runs = []
    for in_place in (False, True):
        x = qkv.clone()
        q, k, v = (t.view(b.rows, -1, hd) for t in x.split([5 * hd, 3 * hd, 3 * hd], dim=1))
        out = q if in_place else torch.empty(b.rows, 5, hd, dtype=BF, device="cuda")
        cache = dg.PagedKV(b.k.clone(), b.v.clone())
        dg.paged_append(cache, b.batch, k, v, rope=rope, norm=norm, q=q, q_out=out)
        assert torch.equal(x[:, 5 * hd:], qkv[:, 5 * hd:])
        runs.append([out, cache.k, cache.v])
    for a, c in zip(*runs):
        assert torch.equal(a, c)
