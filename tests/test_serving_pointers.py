"""Pointers off their element's size are refused by the C entry points before
anything is enqueued (CPU only): the kernels' loads would fault on them."""
import pytest

pytest.importorskip("torch")

import test_serving_host as host  # noqa: E402
from block_text_diffusion_b200 import serving as sv  # noqa: E402
from test_serving_host import A, batch, cache, heads, ref  # noqa: E402

ODD, HALF = A + 1, A + 2   # off every size; off the size of an int32 or fp32


@pytest.fixture(scope="module")
def L():
    import block_text_diffusion_b200 as dg
    from block_text_diffusion_b200 import build
    build.build()
    return dg.lib()


@pytest.mark.parametrize("dtype, off", [(1, ODD), (0, HALF)])
def test_rows_off_their_size_are_refused(L, dtype, off):
    for name in ("q", "qo", "k", "ko"):
        assert host.norm_rope(L, dtype=dtype, **{name: heads(p=off)}) == 1, name
    for name in ("k", "v", "q", "qo"):
        assert host.append(L, c=cache(dtype=dtype), **{name: heads(p=off)}) == 1, name
    for gains in ((off, None), (None, off)):
        assert host.norm_rope(L, dtype=dtype, norm=sv._HeadNorm(1, 1e-6, *gains)) == 1
        assert host.append(L, c=cache(dtype=dtype), norm=sv._HeadNorm(1, 1e-6, *gains)) == 1


def test_integers_off_their_size_are_refused(L):
    assert host.norm_rope(L, pos=HALF) == 1
    for kw in (dict(cu_q=HALF), dict(kv_lens=HALF), dict(page_table=HALF), dict(prefix_pages=HALF, prefix_len=5)):
        assert host.append(L, b=batch(**kw)) == 1, kw
        assert host.attention(L, b=batch(**kw)) == 1, kw
    c, b, h = ref(cache()), ref(batch()), ref(heads())
    assert L.dg_paged_append(c, b, h, h, None, None, 0, None, None, HALF, None) == 1
    for lse, status in ((HALF, None), (None, HALF)):
        assert L.dg_paged_attention(c, b, 4, h, 0.1, 1, h, lse, A, 1 << 40, status, None) == 1
