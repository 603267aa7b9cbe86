"""Cases of the paged serving operators: what is measured, and against what.

Three operators serve several sequences (prompts, 256-token canvases, single
tokens) over one paged key/value cache:

  qk_norm_rope      RMSNorm of every query and key head with the position
                    rotation in the same pass;
  paged_append      the same for new tokens whose keys and values go straight
                    into the pages of the cache;
  paged_attention   attention over the pages, with one prefix shared by the
                    whole batch and read once for all of it.

`run` computes them in their plain form (elementary operations in 32 bits,
angles in 64) unless `own` is set, when it calls the package's operators.
`exact` is the definition in 64 bits, written apart from both.
"""
from __future__ import annotations

import math

import torch

own = False

EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# -- cases -------------------------------------------------------------------------

def _rope(name, tokens, heads, kv_heads, dim, rot, interleaved=False, factor=1.0, dtype="bf16"):
    return {"name": name, "op": "rope", "tokens": tokens, "heads": heads, "kv_heads": kv_heads, "dim": dim,
            "rot": rot, "interleaved": interleaved, "factor": factor, "dtype": dtype}


def _append(name, seqs, new, past, heads, kv_heads, dim, page, rot, prefix=0, ragged=False, interleaved=False,
            dtype="bf16"):
    return {"name": name, "op": "append", "seqs": seqs, "new": new, "past": past, "prefix": prefix, "heads": heads,
            "kv_heads": kv_heads, "dim": dim, "page": page, "rot": rot, "ragged": ragged,
            "interleaved": interleaved, "dtype": dtype}


def _attn(name, seqs, new, past, prefix, heads, kv_heads, dim, page, causal, ragged=False, dtype="bf16"):
    return {"name": name, "op": "attention", "seqs": seqs, "new": new, "past": past, "prefix": prefix,
            "heads": heads, "kv_heads": kv_heads, "dim": dim, "page": page, "causal": causal, "ragged": ragged,
            "dtype": dtype}


def listed():
    return [
        # one canvas of the mid model (8 query and 2 key heads): a latency-bound call
        _rope("rope_canvas_mid", 256, 8, 2, 128, 128),
        # a ragged fp32 batch of the tiny model's heads, half of each head rotated, neighbouring pairs
        _rope("rope_ragged_fp32", 1001, 4, 4, 64, 32, interleaved=True, dtype="fp32"),
        # 32 canvases of the 26B-A4B shape at positions scaled for a long context
        _rope("rope_32_canvases_26b", 8192, 16, 8, 128, 128, factor=4.0),
        # single-token decoding of 32 sequences: one row each into its own last page
        _append("append_tokens_26b", 32, 1, 2047, 16, 8, 128, 64, 128, prefix=2048, ragged=True),
        # ragged fp32 prompts whose last pages are part full
        _append("append_ragged_fp32", 5, 333, 70, 4, 4, 64, 16, 64, ragged=True, dtype="fp32"),
        # eight 2048-token prompts of the 26B-A4B shape written at once
        _append("append_prompts_26b", 8, 2048, 0, 16, 8, 128, 64, 128),
        # one fp32 canvas of the tiny model after its 64-token prompt
        _attn("attn_canvas_tiny_fp32", 1, 256, 64, 0, 4, 4, 64, 16, False, dtype="fp32"),
        # one token of one long sequence: the smallest query over the longest own context
        _attn("attn_token_long_mid", 1, 1, 32767, 0, 8, 2, 128, 64, True),
        # 64 ragged sequences decode one token each behind a shared 2048-token prompt
        _attn("attn_tokens_shared_26b", 64, 1, 1500, 2048, 16, 8, 128, 64, True, ragged=True),
        # eight canvases drawn from one shared 2048-token prompt, bidirectional
        _attn("attn_canvases_shared_26b", 8, 256, 0, 2048, 16, 8, 128, 64, False),
        # ragged prompts encoded causally, pages smaller than a tile
        _attn("attn_prompts_causal_26b", 4, 2048, 0, 0, 16, 8, 128, 32, True, ragged=True),
        # eight canvases of the mid model behind a shared 32768-token prompt
        _attn("attn_canvases_long_mid", 8, 256, 256, 32768, 8, 2, 128, 128, False),
    ]


_MOST = {"rope": 1.0e8, "append": 2.5e8, "attention": 2.7e11}


def _log(rng, lo, hi):
    """A whole number whose logarithm is spread evenly over [lo, hi]."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case of the same ranges."""
    while True:
        op = rng.choice(["rope", "append", "attention", "attention"])
        dtype = rng.choice(["bf16", "bf16", "fp32"])
        dim = rng.choice([64, 128])
        kv_heads = rng.choice([1, 2, 3, 4, 8])
        heads = kv_heads * rng.choice([1, 2, 2, 3, 4, 5, 8])
        if op == "rope":
            c = _rope(None, _log(rng, 1, 8192), heads, kv_heads, dim, rng.choice([dim, dim, dim // 2, dim // 4]),
                      rng.choice([False, True]), rng.choice([1.0, 4.0, 16.0]), dtype)
        elif op == "append":
            c = _append(None, _log(rng, 1, 64), _log(rng, 1, 2048), _log(rng, 1, 4096) - 1, heads, kv_heads, dim,
                        rng.choice([16, 32, 64, 128, 256]), rng.choice([dim, dim, dim // 2]),
                        rng.choice([0, _log(rng, 1, 4096)]), rng.choice([False, True]), rng.choice([False, True]),
                        dtype)
        else:
            c = _attn(None, _log(rng, 1, 64), rng.choice([1, 1, 256, _log(rng, 2, 2048)]), _log(rng, 1, 32768) - 1,
                      rng.choice([0, _log(rng, 1, 32768)]), heads, kv_heads, dim,
                      rng.choice([16, 32, 64, 128, 256]), rng.choice([False, True]), rng.choice([False, True]),
                      dtype)
        c.pop("name")
        w = work(c)
        if op == "attention":
            # fp32 products have no tensor-core form: their largest case is smaller
            if w["flops"] > (_MOST[op] if dtype == "bf16" else 6e9) or w["bytes"] > 3e8:
                continue
            # the pages of one case, own and shared, within a few GB
            if 2 * sum(_own_pages(c)) * c["page"] * kv_heads * dim * 4 > 2e9:
                continue
        elif w["bytes"] > _MOST[op]:
            continue
        return c


def _lens(case):
    """Tokens already in the cache and new tokens of every sequence (a rule of
    the case alone: ragged batches run from the full length down to half)."""
    past, new = [], []
    for b in range(case["seqs"]):
        p, n = case["past"], case["new"]
        if case["ragged"]:
            p -= p * (b * 37 % 64) // 128
            n -= n * (b * 23 % 64) // 128
        past.append(p)
        new.append(n)
    return past, new


def _own_pages(case):
    past, new = _lens(case)
    return [-(-(p + n) // case["page"]) for p, n in zip(past, new)]


def work(case):
    size = 2 if case["dtype"] == "bf16" else 4
    d = case["dim"]
    if case["op"] == "rope":
        n = case["tokens"] * (case["heads"] + case["kv_heads"]) * d
        return {"bytes": 2 * n * size + 4 * case["tokens"], "flops": 8 * n}
    past, new = _lens(case)
    t = sum(new)
    if case["op"] == "append":
        qk = t * (case["heads"] + case["kv_heads"]) * d
        return {"bytes": 2 * (qk + t * case["kv_heads"] * d) * size, "flops": 8 * qk}
    pairs = 0
    for p, n in zip(past, new):
        own_pairs = n * p + n * (n + 1) // 2 if case["causal"] else n * (p + n)
        pairs += own_pairs + n * case["prefix"]
    keys = case["prefix"] + sum(past) + t
    rows = t * case["heads"]
    return {"bytes": 2 * keys * case["kv_heads"] * d * size + 2 * rows * d * size + 4 * rows,
            "flops": 4 * pairs * case["heads"] * d}


# -- inputs ------------------------------------------------------------------------

def _inv_freq(rot, factor, theta=10000.0):
    """Radians a position turns each pair by; a factor above 1 stretches the
    context by that much (all frequencies divided by it)."""
    i = torch.arange(rot // 2, dtype=torch.float64)
    return theta ** (-2.0 * i / rot) / factor


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    h = torch.Generator().manual_seed(seed)
    dtype, d = TYPES[case["dtype"]], case["dim"]

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)

    s = {"case": case}
    hq, hk = case["heads"], case["kv_heads"]
    if case["op"] == "rope":
        t = case["tokens"]
        # queries and keys are column ranges of one projection's output
        qkv = normal(t, (hq + 2 * hk) * d)
        s["q"] = qkv[:, :hq * d].view(t, hq, d)
        s["k"] = qkv[:, hq * d:(hq + hk) * d].view(t, hk, d)
        start = int(torch.randint(0, int(32768 * case["factor"]), (1,), generator=h))
        s["positions"] = (torch.arange(t, dtype=torch.int32) % 2048 + start).cuda()
        s["inv_freq"] = _inv_freq(case["rot"], case["factor"]).cuda()
        s["q_gain"], s["k_gain"] = 1 + normal(d, std=0.1), 1 + normal(d, std=0.1)
        s["q_out"] = torch.zeros(t, hq, d, dtype=dtype, device="cuda")
        s["k_out"] = torch.zeros(t, hk, d, dtype=dtype, device="cuda")
        if own:
            import block_text_diffusion_b200 as dg
            s["rope"] = dg.Rope(s["inv_freq"], interleaved=case["interleaved"])
            s["norm"] = dg.HeadNorm(EPS, s["q_gain"], s["k_gain"])
        return s

    past, new = _lens(case)
    t, page, prefix = sum(new), case["page"], case["prefix"]
    own_pages, prefix_pages = _own_pages(case), -(-prefix // page)
    n_pages = sum(own_pages) + prefix_pages + 3
    order = torch.randperm(n_pages, generator=h, dtype=torch.int32)
    table = torch.full((len(new), max(own_pages) + 1), -1, dtype=torch.int32)
    at = prefix_pages
    for b, n in enumerate(own_pages):
        table[b, :n] = order[at:at + n]
        at += n
    s["past"], s["new"] = past, new
    s["prefix_pages"] = order[:prefix_pages].cuda() if prefix else None
    s["page_table"] = table.cuda()
    s["cu_q"] = torch.tensor([0] + new).cumsum(0).to(torch.int32).cuda()
    s["kv_lens"] = torch.tensor([p + n for p, n in zip(past, new)], dtype=torch.int32).cuda()
    s["k_cache"] = normal(n_pages, hk, page, d)
    s["v_cache"] = normal(n_pages, hk, page, d)
    if case["op"] == "append":
        qkv = normal(t, (hq + 2 * hk) * d)
        s["q"] = qkv[:, :hq * d].view(t, hq, d)
        s["k"] = qkv[:, hq * d:(hq + hk) * d].view(t, hk, d)
        s["v"] = qkv[:, (hq + hk) * d:].view(t, hk, d)
        s["inv_freq"] = _inv_freq(case["rot"], 1.0).cuda()
        s["q_gain"], s["k_gain"] = 1 + normal(d, std=0.1), 1 + normal(d, std=0.1)
        s["q_out"] = torch.zeros(t, hq, d, dtype=dtype, device="cuda")
        # where every new token lands: page and offset, and its position behind the prefix
        spot = [(b, p + i) for b, (p, n) in enumerate(zip(past, new)) for i in range(n)]
        seq = torch.tensor([b for b, _ in spot])
        idx = torch.tensor([i for _, i in spot])
        s["token_page"] = table[seq, idx // page].long().cuda()
        s["token_off"] = (idx % page).cuda()
        s["token_pos"] = (idx + prefix).cuda()
    else:
        s["q"] = normal(t, hq, d, std=1.5)
        s["out"] = torch.zeros(t, hq, d, dtype=dtype, device="cuda")
        s["lse"] = torch.zeros(t, hq, dtype=torch.float32, device="cuda")
    if own:
        import block_text_diffusion_b200 as dg
        s["cache"] = dg.PagedKV(s["k_cache"], s["v_cache"])
        s["batch"] = dg.PagedBatch(s["cu_q"], s["kv_lens"], s["page_table"], prefix_pages=s["prefix_pages"],
                                   prefix_len=prefix)
        if case["op"] == "append":
            s["rope"] = dg.Rope(s["inv_freq"], interleaved=case["interleaved"])
            s["norm"] = dg.HeadNorm(EPS, s["q_gain"], s["k_gain"])
        else:
            n = dg.paged_attention_workspace(t, hq, d, prefix > 0)
            s["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    return s


# -- the plain forms ---------------------------------------------------------------

def _norm_rotate(x, gain, pos, inv_freq, interleaved):
    """x [T, H, d] -> RMSNorm with the gain, then the rotation, in 32 bits."""
    y = x.float()
    y = y * torch.rsqrt((y * y).mean(dim=-1, keepdim=True) + EPS) * gain.float()
    angle = pos.double()[:, None] * inv_freq[None, :]
    c, s = torch.cos(angle).float()[:, None, :], torch.sin(angle).float()[:, None, :]
    rot = 2 * inv_freq.numel()
    out = y.clone()
    if interleaved:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        out[..., 0:rot:2] = a * c - b * s
        out[..., 1:rot:2] = b * c + a * s
    else:
        a, b = y[..., :rot // 2], y[..., rot // 2:rot]
        out[..., :rot // 2] = a * c - b * s
        out[..., rot // 2:rot] = b * c + a * s
    return out


def _pages(cache, pages, n):
    """The first n rows of a list of pages, [Hkv, n, d]."""
    x = cache[pages.long()]
    return x.transpose(0, 1).reshape(cache.shape[1], -1, cache.shape[3])[:, :n]


def _plain_attention(s):
    case = s["case"]
    hq, hk, d, page = case["heads"], case["kv_heads"], case["dim"], case["page"]
    pk = pv = None
    if case["prefix"]:
        pk = _pages(s["k_cache"], s["prefix_pages"], case["prefix"])
        pv = _pages(s["v_cache"], s["prefix_pages"], case["prefix"])
    t0 = 0
    for b, (p, n) in enumerate(zip(s["past"], s["new"])):
        kv = p + n
        row = s["page_table"][b, :-(-kv // page)]
        k, v = _pages(s["k_cache"], row, kv), _pages(s["v_cache"], row, kv)
        if pk is not None:
            k, v = torch.cat([pk, k], dim=1), torch.cat([pv, v], dim=1)
        k, v = k.float(), v.float()
        at = torch.arange(case["prefix"] + p, case["prefix"] + kv, device="cuda")
        key = torch.arange(case["prefix"] + kv, device="cuda")
        # query rows in runs that keep the scores within about a gigabyte
        step = max(1, (1 << 28) // (hq * key.numel()))
        for i in range(0, n, step):
            j = min(n, i + step)
            q = s["q"][t0 + i:t0 + j].float().view(j - i, hk, hq // hk, d).permute(1, 2, 0, 3).reshape(hk, -1, d)
            x = torch.matmul(q, k.transpose(1, 2)) / math.sqrt(d)
            if case["causal"]:
                hide = key[None, :] > at[i:j, None]
                x = x.view(hk, hq // hk, j - i, -1).masked_fill(hide, -math.inf).view(x.shape)
            top = x.max(dim=-1, keepdim=True).values
            e = torch.exp(x - top)
            z = e.sum(dim=-1, keepdim=True)
            o = torch.matmul(e, v) / z
            s["out"][t0 + i:t0 + j] = o.view(hk, hq // hk, j - i, d).permute(2, 0, 1, 3).reshape(j - i, hq, d)
            s["lse"][t0 + i:t0 + j] = (top + torch.log(z)).view(hq, j - i).t()
        t0 += n


def run(s):
    case = s["case"]
    if own:
        import block_text_diffusion_b200 as dg
        if case["op"] == "rope":
            dg.qk_norm_rope(s["q"], s["k"], s["positions"], s["q_out"], s["k_out"], rope=s["rope"], norm=s["norm"])
        elif case["op"] == "append":
            dg.paged_append(s["cache"], s["batch"], s["k"], s["v"], rope=s["rope"], norm=s["norm"], q=s["q"],
                            q_out=s["q_out"])
        else:
            dg.paged_attention(s["cache"], s["batch"], s["q"], s["out"], causal=case["causal"], lse=s["lse"],
                               workspace=s["workspace"])
    elif case["op"] == "rope":
        a = (s["positions"], s["inv_freq"], case["interleaved"])
        s["q_out"].copy_(_norm_rotate(s["q"], s["q_gain"], *a))
        s["k_out"].copy_(_norm_rotate(s["k"], s["k_gain"], *a))
    elif case["op"] == "append":
        a = (s["token_pos"], s["inv_freq"], case["interleaved"])
        s["q_out"].copy_(_norm_rotate(s["q"], s["q_gain"], *a))
        k = _norm_rotate(s["k"], s["k_gain"], *a)
        s["k_cache"][s["token_page"], :, s["token_off"]] = k.to(s["k_cache"].dtype)
        s["v_cache"][s["token_page"], :, s["token_off"]] = s["v"]
    else:
        _plain_attention(s)
    if case["op"] == "rope":
        return {"q": s["q_out"], "k": s["k_out"]}
    if case["op"] == "append":
        return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    return {"out": s["out"], "lse": s["lse"]}


# -- the definition in 64 bits -------------------------------------------------------

def _turned(x, gain, pos, rot, factor, interleaved):
    """Each head divided by its root mean square, times the gain; pair j of the
    first `rot` components, read as a complex number, times e^(i pos w_j)."""
    x = x.double()
    x = x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt() * gain.double()
    w = torch.tensor([10000.0 ** (-2.0 * j / rot) / factor for j in range(rot // 2)], dtype=torch.float64,
                     device=x.device)
    turn = torch.polar(torch.ones(1, dtype=torch.float64, device=x.device), pos.double()[:, None] * w)[:, None]
    head = x[..., :rot]
    if interleaved:
        z = torch.view_as_complex(head.reshape(*head.shape[:-1], rot // 2, 2).contiguous()) * turn
        head = torch.view_as_real(z).reshape(head.shape)
    else:
        z = torch.complex(head[..., :rot // 2].contiguous(), head[..., rot // 2:].contiguous()) * turn
        head = torch.cat([z.real, z.imag], dim=-1)
    return torch.cat([head, x[..., rot:]], dim=-1)


def exact(case, seed):
    w = work(case)
    if case["op"] == "attention" and w["flops"] > 2e13:
        return None
    s = prepare(case, seed)
    if case["op"] == "rope":
        a = (s["positions"], case["rot"], case["factor"], case["interleaved"])
        return {"q": _turned(s["q"], s["q_gain"], *a), "k": _turned(s["k"], s["k_gain"], *a)}
    past, new = _lens(case)
    page, prefix = case["page"], case["prefix"]
    if case["op"] == "append":
        kc, vc = s["k_cache"].double(), s["v_cache"].double()
        pos = torch.cat([torch.arange(prefix + p, prefix + p + n) for p, n in zip(past, new)]).cuda()
        a = (pos, case["rot"], 1.0, case["interleaved"])
        q, k, v = _turned(s["q"], s["q_gain"], *a), _turned(s["k"], s["k_gain"], *a), s["v"].double()
        t = 0
        for b, (p, n) in enumerate(zip(past, new)):
            i = 0
            while i < n:    # page by page
                pg, off = (p + i) // page, (p + i) % page
                m = min(n - i, page - off)
                at = int(s["page_table"][b, pg])
                kc[at, :, off:off + m] = k[t + i:t + i + m].transpose(0, 1)
                vc[at, :, off:off + m] = v[t + i:t + i + m].transpose(0, 1)
                i += m
            t += n
        return {"q": q, "k_cache": kc, "v_cache": vc}
    hq, hk, d = case["heads"], case["kv_heads"], case["dim"]
    out = torch.zeros(sum(new), hq, d, dtype=torch.float64, device="cuda")
    lse = torch.zeros(sum(new), hq, dtype=torch.float64, device="cuda")
    t = 0
    for b, (p, n) in enumerate(zip(past, new)):
        # one row of (page, offset) for every key the sequence can see, the prefix first
        i = torch.arange(prefix, device="cuda")
        j = torch.arange(p + n, device="cuda")
        own_at = s["page_table"][b].long()[j // page]
        at = torch.cat([s["prefix_pages"].long()[i // page], own_at]) if prefix else own_at
        off = torch.cat([i % page, j % page])
        for head in range(hk):
            k, v = s["k_cache"][at, head, off].double(), s["v_cache"][at, head, off].double()
            for g in range(head * (hq // hk), (head + 1) * (hq // hk)):
                x = s["q"][t:t + n, g].double() @ k.t() * d ** -0.5
                if case["causal"]:
                    x += torch.full_like(x, -math.inf).triu(prefix + p + 1)
                lse[t:t + n, g] = torch.logsumexp(x, dim=-1)
                out[t:t + n, g] = torch.softmax(x, dim=-1) @ v
        t += n
    return {"out": out, "lse": lse}
