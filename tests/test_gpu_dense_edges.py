"""Dense attention where its arithmetic and its reports are at their limits,
against the definition in 64 bits."""
import pytest
import torch

from _dense_util import DenseCase, check, queries, reference
from test_gpu_dense import DT, decode, prefill, seen_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def csa2():
    import fp4_kv_cache_nvfp4_b200 as m
    assert torch.cuda.is_available()
    m.lib()
    return m


@pytest.mark.parametrize("n", [3, 24])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_the_maximum_rises_inside_a_tile(csa2, n, dtype):
    """Scores that are level over 128 entries and rise by 8 to 32 bits between the
    64th and the 65th entry of every tile: the tile's first weights, already
    written, are rescaled."""
    L = 15 * 128
    c = DenseCase(csa2, [L], 64, seed=3)
    sl, pos = c.slots(0, L), torch.arange(L)
    c.codes[sl[:, None], torch.arange(64)] = 0x22                                     # K = 1.0 ...
    s = (((pos + 64) // 128).float() * 0.5).to(torch.float8_e4m3fn).view(torch.uint8)  # ... times 0, .5, 1, ... 7.5
    c.scales[sl[:, None], torch.arange(8)] = s[:, None].expand(L, 8)
    c.upload()
    gain = torch.linspace(1, 4, 16, dtype=torch.bfloat16)[None, :, None]
    q = torch.ones((n, 16, 128), dtype=torch.bfloat16) * gain
    out, lse, err = prefill(csa2, c, q, [0, n], DT[dtype], [L - n])
    assert err == 0
    check(out, lse, reference(q, c.rows(0), seen_of(L, n, L - n, 1)), f"{n} tokens, {dtype}")
