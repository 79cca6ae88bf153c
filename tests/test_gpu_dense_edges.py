"""Dense attention where its arithmetic and its reports are at their limits,
against the definition in 64 bits."""
import pytest
import torch

from _dense_util import E2M1, DenseCase, check, queries, reference
from test_gpu_dense import DT, decode, prefill, seen_of

pytestmark = pytest.mark.gpu
DEV_PAGE, DEV_TIMEOUT = 0x2, 0x10


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


def sink_case(csa2, n, seed=11):
    """n entries whose scores are all 0 and whose V is not negative, behind one entry
    with V = 0 and a score of 6 q_0 16 / sqrt(128) for queries of q_0 in 16 channels."""
    c = DenseCase(csa2, [n + 1], 64, seed=seed)
    sl = c.slots(0, n + 1)
    c.codes[sl, :64] = 0
    c.codes[sl, 64:] &= 0x77
    c.codes[sl[0], :8] = 0x77   # K = 6 in channels 0..15 ...
    c.scales[sl[0], 0] = 0x38   # ... times 1
    c.codes[sl[0], 64:] = 0
    return c.upload()


@pytest.mark.parametrize("kernel", ["decode", "draft", "prefill"])
def test_fp32_results_keep_small_weights(csa2, kernel):
    """One entry that takes nearly all the weight and has V = 0, 16 to 24 nats above
    100,000 others that make up the result.  The largest weight is held as 2^6 or more, the
    second fp16 term of a small one in steps of 2^-24 2^-12: a weight w of the largest is
    rounded by w 2^-22, or 2^-37 / 2^6 = 2^-43 where that is more; scores by 128 2^-24 of sum |q k| / sqrt(128)
    and 2^-22 of themselves, once above and once below the line; 2^x by 2^-20; and of
    100,000 entries over 148 CTAs no sum is longer than 240 additions of 2^-24."""
    n, tokens = 100_000, {"decode": 1, "draft": 5, "prefill": 33}[kernel]
    c = sink_case(csa2, n)
    nats = torch.linspace(16, 24, 16, dtype=torch.float64)
    q = torch.zeros((tokens, 16, 128), dtype=torch.bfloat16)
    q[:, :, :16] = (nats * 128 ** 0.5 / 96)[None, :, None].to(torch.bfloat16)
    if kernel == "decode":
        out, lse, err = decode(csa2, c, q, torch.float32)
    else:
        out, lse, err = prefill(csa2, c, q, [0, tokens], torch.float32)
    assert err == 0
    s = q[0, :, 0].double() * 96 / 128 ** 0.5
    v = c.rows(0)[1:, 128:].sum(0)
    want = v[None] / (torch.exp(s)[:, None] + n)
    bound = 2.0 ** -43 * torch.exp(s) + 2.0 ** -22 + 2 * s * (128 * 2.0 ** -24 + 2.0 ** -22) + 2 * 2.0 ** -20 + 240 * 2.0 ** -24
    for i in {0, tokens - 1}:
        off = (out[i].double().cpu() - want).abs() / want
        assert (off <= bound[:, None]).all(), f"token {i}: {(off.amax(1) / bound).tolist()} of the bound"
        assert (lse[i].double().cpu() - torch.log(torch.exp(s) + n)).abs().max() <= bound.max()


@pytest.mark.parametrize("half", [0, 1])
def test_fp32_results_keep_small_weights_through_a_rise(csa2, half):
    """The same with the entry that takes the weight last, in either half of the last
    tile: what the earlier entries gave is rescaled, in O and in the tile itself."""
    n = 128 + 64 * half + 20
    c = sink_case(csa2, n)
    c.table = c.table.clone()
    sl = c.slots(0, n + 1)
    for t in (c.codes, c.scales):
        t[sl[-1]], t[sl[0]] = t[sl[0]].clone(), t[sl[-1]].clone()
    c.upload()
    nats = torch.linspace(16, 24, 16, dtype=torch.float64)
    s = (nats * 128 ** 0.5 / 96).to(torch.bfloat16)
    want = c.rows(0)[:-1, 128:].sum(0)[None] / (torch.exp(s.double() * 96 / 128 ** 0.5)[:, None] + n)
    bound = 2.0 ** -43 * torch.exp(nats + 0.1) + 2.0 ** -21 + 2 * 25 * (128 * 2.0 ** -24 + 2.0 ** -22) + 2 * 2.0 ** -20 + n * 2.0 ** -24
    for tokens in (1, 5, 20):
        q = torch.zeros((tokens, 16, 128), dtype=torch.bfloat16)
        q[:, :, :16] = s[None, :, None]
        for out, _, err in [prefill(csa2, c, q, [0, tokens], torch.float32)] + ([decode(csa2, c, q, torch.float32)] if tokens == 1 else []):
            off = (out.double().cpu() - want[None]).abs() / want
            assert err == 0 and (off <= bound[None, :, None]).all(), f"{tokens}: {(off.amax(2) / bound).max()} of the bound"


class Shared:
    """L entries with V >= 0 that B sequences share page by page, and the definition
    in 64 bits on the GPU."""

    def __init__(self, csa2, B, L, page=64):
        g = torch.Generator(device="cuda").manual_seed(B + L)
        codes = torch.randint(0, 256, (L, 128), generator=g, device="cuda", dtype=torch.uint8)
        codes[:, 64:] &= 0x77
        scales = (torch.rand((L, 16), generator=g, device="cuda") * 0.5 + 0.1).to(torch.float8_e4m3fn)
        table = torch.randperm(L // page, generator=g, device="cuda").int().expand(B, -1).contiguous()
        self.cache = csa2.KVCache.from_tensors(codes, scales.view(torch.uint8), table, page)
        self.lens, self.max_len = [L] * B, L
        x = torch.stack([E2M1.cuda()[(codes & 15).int()], E2M1.cuda()[(codes >> 4).int()]], 2).view(L, 256)
        self.rows = x * scales.double().repeat_interleave(16, 1)  # (the order of the entries does not matter)

    def reference(self, q):
        out = []
        for x in q.cuda().double().split(8):
            s = x.reshape(-1, 128) @ self.rows[:, :128].T / 128 ** 0.5
            out.append((torch.softmax(s, 1) @ self.rows[:, 128:]).view(-1, 16, 128))
        return torch.cat(out)


@pytest.mark.parametrize("kernel,B,T,L,steps", [
    ("prefill", 1, 2368, 1 << 18, 64 * 8), ("draft", 148, 1184, 1 << 18, 64 * 8), ("decode", 148, 148, 1 << 19, 64 * 4)])
def test_bf16_results_do_not_drift(csa2, kernel, B, T, L, steps):
    """Work that leaves each CTA whole units of very many entries.  The tensor core's sums
    drop up to 2^-23 of themselves at each product, always towards zero; a sum begins anew
    after `steps` of them, in which it grows from nothing, so at most steps 2^-24 of a
    result are lost.  The results' rounding is 2^-8 / sqrt(3) of each and has no sign: over
    148 x 16 x 128 of them 5 standard deviations are 2.1e-5."""
    c = Shared(csa2, B, L)
    q = queries(T, seed=L)
    if kernel == "decode":
        out, _, err = decode(csa2, c, q, torch.bfloat16)
    else:
        out, _, err = prefill(csa2, c, q, [T * b // B for b in range(B + 1)], torch.bfloat16)
    assert err == 0
    pick = torch.arange(148) * (T // 148)
    off = float((out[pick].double() / c.reference(q[pick])).mean()) - 1
    assert abs(off) <= steps * 2.0 ** -24 + 2.1e-5, f"{off:.3g}"


def test_waits_that_run_out_are_reported(csa2):
    """A limit of no polls: every wait of the decode, prefill and draft kernels gives up
    at once.  The kernels still wait for their copies and products, return and report,
    and the next call, on the same workspace, is right."""
    lens = [5000, 300]
    c = DenseCase(csa2, lens, 64, seed=5)
    q, d = queries(40, seed=6).cuda(), csa2.default_desc(csa2.FULL, 1)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    sl = i32(lens)
    ws = torch.empty(csa2.dense_attn_workspace_bytes(d, 2, True), dtype=torch.uint8, device="cuda")

    def calls(dt):
        for n in (1, 4, 20):
            out, lse = torch.zeros((2 * n, 16, 128), dtype=dt, device="cuda"), torch.zeros((2 * n, 16), device="cuda")
            err = i32([0])
            if n == 1:
                csa2.dense_attn_decode(d, c.cache, q[:2], sl, out, lse, c.max_len, ws, err=err)
            else:
                csa2.dense_attn_prefill(d, c.cache, q[:2 * n], i32([0, n, 2 * n]), sl, out, lse, c.max_len, ws, err=err)
            torch.cuda.synchronize()
            yield n, out, lse, int(err)

    for dt in DT.values():
        prev = csa2.test_set_wait_limit(0)
        try:
            flags = [f for *_, f in calls(dt)]
        finally:
            assert csa2.test_set_wait_limit(prev) == 0
        assert flags == [DEV_TIMEOUT] * 3
        for n, out, lse, err in calls(dt):
            assert err == 0
            for b in (0, 1):
                r = slice(n * b, n * b + n)
                check(out[r], lse[r], reference(q[r].cpu(), c.rows(b), [lens[b]] * n), f"{n} tokens, sequence {b}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,ratio", [(5, 1), (10, 1), (40, 1), (40, 2)])
def test_a_missing_page_counts_where_it_is_seen(csa2, n, ratio, dtype):
    """Pages of 16: the one behind the last entry that any token sees may be missing,
    in a tile that they do see; the one that holds that entry is reported."""
    L, first = 250, 100 * ratio
    last = (first + n) // ratio                 # entries seen by the last token
    page = -(-last // 16)                       # the first that nobody sees
    assert page * 16 < 128 < L or n == 40
    q = queries(n, seed=n)
    for gone, want in ((page, 0), (page - 1, DEV_PAGE)):
        c = DenseCase(csa2, [L], 16, seed=n)
        pages = c.table.clone()
        c.table[0, gone] = -1
        c.upload()
        out, lse, err = prefill(csa2, c, q, [0, n], DT[dtype], [first], ratio)
        assert err == want
        c.table = pages
        hidden = None if gone == page else list(range(gone * 16, gone * 16 + 16))
        check(out, lse, reference(q, c.rows(0), seen_of(L, n, first, ratio), hidden), f"page {gone}")
