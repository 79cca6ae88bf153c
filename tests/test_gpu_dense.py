"""Dense attention over the whole FP4 main KV against its definition in 64 bits."""
import math

import numpy as np
import pytest
import torch

import synth
from _dense_util import DenseCase, check, queries, reference

pytestmark = pytest.mark.gpu
DEV_PAGE, DEV_LEN = 0x2, 0x8
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def csa2():
    import fp4_kv_cache_nvfp4_b200 as m
    assert torch.cuda.is_available()
    m.lib()
    return m


def decode(csa2, c, q, dtype, lens=None, max_len=None, table=None, ws=None, stream=None):
    B = q.shape[0]
    d = csa2.default_desc(csa2.FULL, 1)
    out = torch.full((B, 16, 128), 7.0, dtype=dtype, device="cuda")
    lse = torch.full((B, 16), 7.0, device="cuda")
    ws = torch.full((csa2.dense_attn_workspace_bytes(d, B),), 0xFF, dtype=torch.uint8, device="cuda") if ws is None else ws
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    sl = torch.tensor(c.lens if lens is None else lens, dtype=torch.int32, device="cuda")
    csa2.dense_attn_decode(d, c.cache, q.cuda(), sl, out, lse, c.max_len if max_len is None else max_len, ws, err=err,
                           stream=stream)
    torch.cuda.synchronize()
    return out, lse, int(err.item())


def prefill(csa2, c, q, cu, dtype, start=None, ratio=1, lens=None):
    d = csa2.default_desc(csa2.FULL, ratio)
    T, B = q.shape[0], len(c.lens)
    out = torch.full((T, 16, 128), 7.0, dtype=dtype, device="cuda")
    lse = torch.full((T, 16), 7.0, device="cuda")
    ws = torch.full((csa2.dense_attn_workspace_bytes(d, B, True),), 0xFF, dtype=torch.uint8, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    csa2.dense_attn_prefill(d, c.cache, q.cuda(), i32(cu), i32(c.lens if lens is None else lens), out, lse, c.max_len,
                            ws, q_start=None if start is None else i32(start), err=err)
    torch.cuda.synchronize()
    return out, lse, int(err.item())


def seen_of(L, n, start, ratio):
    return [L] * n if start is None else [min(L, (start + i + 1) // ratio) for i in range(n)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("page,lens", [
    (64, [1]), (64, [64]), (8, [1, 7, 8, 9, 15, 16, 17, 0, 63, 64, 65]), (16, [0, 127, 128, 129, 255, 256, 257]),
    (64, [511, 0, 513, 1000, 3, 4097]), (256, [300, 2049, 1]), (32, [5000] + [1] * 40 + [777])])
def test_decode(csa2, page, lens, dtype):
    c = DenseCase(csa2, lens, page, seed=len(lens) + page)
    q = queries(len(lens), seed=page)
    out, lse, err = decode(csa2, c, q, DT[dtype])
    assert err == 0
    for b in range(len(lens)):
        check(out[b:b + 1], lse[b:b + 1], reference(q[b:b + 1], c.rows(b), [lens[b]]), f"seq {b} ({lens[b]})")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decode_long_and_repeatable(csa2, dtype):
    lens = [60001, 1, 33000]
    c = DenseCase(csa2, lens, 64, seed=5)
    q = queries(3, seed=6)
    out, lse, err = decode(csa2, c, q, DT[dtype])
    assert err == 0
    for b in range(3):
        check(out[b:b + 1], lse[b:b + 1], reference(q[b:b + 1], c.rows(b), [lens[b]]), f"seq {b}")
    again, lse2, _ = decode(csa2, c, q, DT[dtype])
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("gain", [1e-30, 0.01, 8.0, 1e4])
def test_decode_query_magnitudes(csa2, gain):
    """Weights that are all alike, ordinary, and one key that takes them all; bf16
    queries far outside fp16's range."""
    c = DenseCase(csa2, [700], 64, seed=3)
    q = queries(1, gain=gain)
    out, lse, _ = decode(csa2, c, q, torch.float32)
    check(out, lse, reference(q, c.rows(0), [700]), f"gain {gain}")


def test_decode_a_rising_maximum(csa2):
    """Scores that grow along the sequence: every tile raises the running maximum."""
    L = 3000
    c = DenseCase(csa2, [L], 64, seed=9)
    sl = c.slots(0, L)
    c.codes[sl[:, None], torch.arange(64)] = 0x22                     # K = 1.0 everywhere ...
    s = torch.linspace(0.05, 40, L).to(torch.float8_e4m3fn).view(torch.uint8)
    c.scales[sl[:, None], torch.arange(8)] = s[:, None].expand(L, 8)  # ... times a scale that rises
    c.upload()
    q = torch.ones((1, 16, 128), dtype=torch.bfloat16) * torch.linspace(-1, 1, 16, dtype=torch.bfloat16)[None, :, None]
    for dt in DT.values():
        out, lse, _ = decode(csa2, c, q, dt)
        check(out, lse, reference(q, c.rows(0), [L]), str(dt))


def test_decode_bad_lengths_and_pages(csa2):
    """Bad lengths count as empty, a missing page as not seen; each is reported."""
    lens = [200, 300, 130, 70]
    c = DenseCase(csa2, lens, 16, seed=2)
    q = queries(4)
    out, lse, err = decode(csa2, c, q, torch.float32, lens=[200, -1, c.max_len + 1, 70])
    assert err == DEV_LEN
    for b, n in enumerate([200, 0, 0, 70]):
        check(out[b:b + 1], lse[b:b + 1], reference(q[b:b + 1], c.rows(b), [n]), f"seq {b}")
    pages = c.table.clone()
    c.table[0, 3], c.table[2, 0], c.table[3, :] = -1, c.cache.n_phys_pages, -5
    c.upload()
    out, lse, err = decode(csa2, c, q, torch.float32)
    assert err == DEV_PAGE
    c.table = pages
    gone = [list(range(48, 64)), [], list(range(16)), list(range(70))]
    for b in range(4):
        check(out[b:b + 1], lse[b:b + 1], reference(q[b:b + 1], c.rows(b), [lens[b]], gone[b]), f"seq {b}")


@pytest.mark.parametrize("block", [0, 7, 8, 12])
def test_decode_a_nan_entry_is_its_sequences_alone(csa2, block):
    """A NaN scale of K reaches the whole row, one of V at least its own 16 dims."""
    lens = [100, 100]
    c = DenseCase(csa2, lens, 64, seed=2)
    c.scales[c.slots(0, 100)[50], block] = 0x7F
    c.upload()
    q = queries(2)
    for dt in DT.values():
        out, lse, _ = decode(csa2, c, q, dt)
        if block < 8:
            assert torch.isnan(out[0]).all() and torch.isnan(lse[0]).all()
        else:
            assert torch.isnan(out[0, :, 16 * (block - 8):16 * (block - 7)]).all()
        check(out[1:], lse[1:], reference(q[1:], c.rows(1), [100]), "the other sequence")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("causal,ratio", [(True, 1), (True, 2), (False, 1)])
@pytest.mark.parametrize("page,lens,ns", [
    (64, [1], [1]), (64, [300], [5]), (8, [9, 0, 40, 33], [4, 3, 0, 17]), (16, [129, 256, 1], [8, 9, 1]),
    (64, [500, 1000, 130, 7], [33, 16, 130, 15]), (128, [2100], [300])])
def test_prefill(csa2, page, lens, ns, causal, ratio, dtype):
    c = DenseCase(csa2, lens, page, seed=page + len(lens))
    cu = [0]
    for n in ns:
        cu.append(cu[-1] + n)
    q = queries(cu[-1], seed=4)
    start = [max(0, L * ratio - n) for L, n in zip(lens, ns)] if causal else None
    out, lse, err = prefill(csa2, c, q, cu, DT[dtype], start, ratio)
    assert err == 0
    for b, (L, n) in enumerate(zip(lens, ns)):
        if n:
            r = slice(cu[b], cu[b + 1])
            seen = seen_of(L, n, start[b] if causal else None, ratio)
            check(out[r], lse[r], reference(q[r], c.rows(b), seen), f"seq {b} ({n} over {L})")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,n,L", [(3, 5, 9000), (200, 2, 300), (4, 8, 1290), (2, 9, 2000)])
def test_prefill_drafts(csa2, B, n, L, dtype):
    """A few tokens each over long sequences (units of one row tile, over several CTAs or
    many to a CTA), a missing page and a rising maximum among them."""
    lens = [L - 37 * (b % 5) for b in range(B)]
    c = DenseCase(csa2, lens, 64, seed=B)
    sl = c.slots(1, lens[1])
    rise = torch.linspace(0.05, 60, lens[1]).to(torch.float8_e4m3fn).view(torch.uint8)
    c.scales[sl[:, None], torch.arange(8)] = rise[:, None].expand(lens[1], 8)
    pages = c.table.clone()
    c.table[0, 2] = -1
    c.upload()
    q = queries(B * n, seed=B)
    start = [x - n for x in lens]
    out, lse, err = prefill(csa2, c, q, [n * b for b in range(B + 1)], DT[dtype], start)
    assert err == DEV_PAGE
    c.table = pages
    for b in [0, 1, B - 1]:
        r = slice(n * b, n * b + n)
        check(out[r], lse[r], reference(q[r], c.rows(b), seen_of(lens[b], n, start[b], 1),
                                        range(128, 192) if b == 0 else None), f"seq {b}")


def test_prefill_rows_of_no_sequence_stay(csa2):
    """Rows before cu_q[0], of a range that is not ascending or leaves T, and
    behind the last sequence are left as they were; early tokens of a ratio-2
    sequence see nothing."""
    c = DenseCase(csa2, [50, 60, 70, 80], 16, seed=8)
    q = queries(64)
    cu = [3, 20, 20, 30, 1 << 20]
    out, lse, err = prefill(csa2, c, q, cu, torch.bfloat16, [0, 5, 100, 7], 2)
    assert err == DEV_LEN
    for lo, hi, b, st in ((3, 20, 0, 0), (20, 30, 2, 100)):
        check(out[lo:hi], lse[lo:hi], reference(q[lo:hi], c.rows(b), seen_of(c.lens[b], hi - lo, st, 2)), f"seq {b}")
    assert (lse[3] == -math.inf).all() and (out[3] == 0).all()
    for r in (slice(0, 3), slice(30, 64)):
        assert (out[r] == 7).all() and (lse[r] == 7).all()
    out, lse, err = prefill(csa2, c, q, [10, 5, 25, -3, 40], torch.float32)
    assert err == DEV_LEN
    check(out[5:25], lse[5:25], reference(q[5:25], c.rows(1), [60] * 20), "the one good range")
    assert (out[:5] == 7).all() and (out[25:] == 7).all()


def test_prefill_bad_lengths_starts_and_pages(csa2):
    lens = [200, 90, 130]
    c = DenseCase(csa2, lens, 16, seed=2)
    q, cu = queries(30), [0, 10, 20, 30]
    out, lse, err = prefill(csa2, c, q, cu, torch.float32, [190, -4, 120], lens=[200, 90, -7])
    assert err == DEV_LEN
    check(out[:10], lse[:10], reference(q[:10], c.rows(0), seen_of(200, 10, 190, 1)), "seq 0")
    assert (out[10:] == 0).all() and (lse[10:] == -math.inf).all()
    pages = c.table.clone()
    c.table[0, 1], c.table[1, 5] = -1, 1 << 30
    c.upload()
    out, lse, err = prefill(csa2, c, q, cu, torch.float32, [190, 80, 120])
    assert err == DEV_PAGE
    c.table = pages
    for b, (st, gone) in enumerate(((190, range(16, 32)), (80, range(80, 96)), (120, ()))):
        r = slice(10 * b, 10 * b + 10)
        check(out[r], lse[r], reference(q[r], c.rows(b), seen_of(lens[b], 10, st, 1), list(gone)), f"seq {b}")


def test_prefill_a_nan_entry_reaches_those_who_see_it(csa2):
    """NaN scales of K or V in an entry that only later tokens see."""
    for ch in (0, 15):
        c = DenseCase(csa2, [150], 64, seed=2)
        c.scales[c.slots(0, 150)[140], ch] = 0xFF
        c.upload()
        q = queries(20)
        for dt in DT.values():
            out, lse, _ = prefill(csa2, c, q, [0, 20], dt, [130])
            clean = DenseCase(csa2, [150], 64, seed=2)
            check(out[:10], lse[:10], reference(q[:10], clean.rows(0), seen_of(150, 10, 130, 1)), "who do not see it")
            if ch < 8:
                assert torch.isnan(out[10:]).all() and torch.isnan(lse[10:]).all()
            else:
                assert torch.isnan(out[10:, :, 16 * (ch - 8):16 * (ch - 7)]).all()


@pytest.mark.parametrize("gain", [1e-30, 8.0, 1e4])
def test_prefill_query_magnitudes(csa2, gain):
    c = DenseCase(csa2, [400], 64, seed=3)
    q = queries(19, gain=gain)
    for dt in DT.values():
        out, lse, _ = prefill(csa2, c, q, [0, 19], dt, [381])
        check(out, lse, reference(q, c.rows(0), seen_of(400, 19, 381, 1)), f"gain {gain}")


def test_prefill_a_rising_maximum(csa2):
    L, n = 1500, 24
    c = DenseCase(csa2, [L], 64, seed=9)
    sl = c.slots(0, L)
    c.codes[sl[:, None], torch.arange(64)] = 0x22
    s = torch.linspace(0.05, 40, L).to(torch.float8_e4m3fn).view(torch.uint8)
    c.scales[sl[:, None], torch.arange(8)] = s[:, None].expand(L, 8)
    c.upload()
    q = torch.ones((n, 16, 128), dtype=torch.bfloat16) * torch.linspace(-1, 1, 16, dtype=torch.bfloat16)[None, :, None]
    for dt in DT.values():
        out, lse, _ = prefill(csa2, c, q, [0, n], dt, [L - n])
        check(out, lse, reference(q, c.rows(0), seen_of(L, n, L - n, 1)), str(dt))


@pytest.mark.parametrize("B,n,L", [(1, 5, 40000), (2, 40, 12000)])
def test_fp32_results_do_not_drift(csa2, B, n, L):
    """A long sequence's fp32 result is as exact as a short one's: within 1e-6 of the
    definition in the 2-norm (fp32 sums of n terms with rounding; sums that drop bits
    towards zero, as the tensor core's do, would be n 2^-25 off and reach 1e-5 here)."""
    c = DenseCase(csa2, [L] * B, 64, seed=L)
    q = queries(B * n, seed=7)
    pre = prefill(csa2, c, q, [n * b for b in range(B + 1)], torch.float32)
    dec = decode(csa2, c, q[::n].contiguous(), torch.float32)
    for b in range(B):
        pick = [n * b, n * b + n - 1]
        ref = reference(q[pick], c.rows(b), [L, L])[0]
        for got, want in ((pre[0][pick].double().cpu(), ref), (dec[0][b:b + 1].double().cpu(), ref[:1])):
            assert (got - want).norm() <= 1e-6 * want.norm()


def test_prefill_repeatable_and_equal_alone(csa2):
    """The same call twice gives the same bits, and a sequence's result does not
    depend on rows that are not its own beyond its bound."""
    lens, cu = [3000, 50, 2500], [0, 700, 701, 1100]
    c = DenseCase(csa2, lens, 64, seed=12)
    q = queries(1100)
    st = [2300, 49, 2101]
    a = prefill(csa2, c, q, cu, torch.bfloat16, st)
    b = prefill(csa2, c, q, cu, torch.bfloat16, st)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    pick = [0, 1, 350, 699]
    check(a[0][pick], a[1][pick], reference(q[pick], c.rows(0), [2301, 2302, 2651, 3000]), "seq 0")
    pick = [701, 900, 1099]
    check(a[0][pick], a[1][pick], reference(q[pick], c.rows(2), [2102, 2301, 2500]), "seq 2")


def test_captured_and_replayed_with_new_inputs(csa2):
    """Both calls in one graph; queries, lengths and page table change between replays."""
    d = csa2.default_desc(csa2.FULL, 1)
    lens = [900, 40, 2000]
    c = DenseCase(csa2, lens, 64, seed=1)
    q = queries(3).cuda()
    qp = queries(30, seed=2).cuda()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    sl, cu, st = i32(lens), i32([0, 10, 20, 30]), i32([890, 30, 1990])
    out, lse = torch.empty((3, 16, 128), device="cuda"), torch.empty((3, 16), device="cuda")
    outp, lsep = torch.empty((30, 16, 128), dtype=torch.bfloat16, device="cuda"), torch.empty((30, 16), device="cuda")
    ws = torch.empty(max(csa2.dense_attn_workspace_bytes(d, 3, p) for p in (False, True)), dtype=torch.uint8, device="cuda")

    def both():
        csa2.dense_attn_decode(d, c.cache, q, sl, out, lse, c.max_len, ws)
        csa2.dense_attn_prefill(d, c.cache, qp, cu, sl, outp, lsep, c.max_len, ws, q_start=st)

    both()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        both()
    for k, (ln, perm) in enumerate((([900, 40, 2000], [0, 1, 2]), ([130, 2000, 1], [1, 2, 0]))):
        c.lens = ln
        rows_of = [0, 1, 2]
        q.copy_(queries(3, seed=20 + k).cuda())
        qp.copy_(queries(30, seed=30 + k).cuda())
        table = c.table.clone()
        if k:  # the sequences swap their pages
            table = c.table[perm]
            ln = [130, 2000, 1]
        c.cache.page_table.copy_(table.cuda())
        sl.copy_(i32(ln))
        st.copy_(i32([max(0, n - 10) for n in ln]))
        g.replay()
        torch.cuda.synchronize()
        keep, c.table = c.table, table
        for b in rows_of:
            r = slice(10 * b, 10 * b + 10)
            if ln[b] <= [900, 40, 2000][perm[b] if k else b]:
                check(out[b:b + 1], lse[b:b + 1], reference(q[b:b + 1].cpu(), c.rows(b), [ln[b]]), f"replay {k} seq {b}")
                check(outp[r], lsep[r], reference(qp[r].cpu(), c.rows(b), seen_of(ln[b], 10, max(0, ln[b] - 10), 1)),
                      f"replay {k} chunk {b}")
        c.table = keep


def test_two_streams_with_their_own_workspaces(csa2):
    d = csa2.default_desc(csa2.FULL, 1)
    cs = [DenseCase(csa2, [20000, 300], 64, seed=s) for s in (1, 2)]
    qs = [queries(2, seed=s).cuda() for s in (3, 4)]
    want = [decode(csa2, c, q, torch.float32)[:2] for c, q in zip(cs, qs)]
    streams = [torch.cuda.Stream() for _ in cs]
    got = []
    torch.cuda.synchronize()
    ws = [torch.empty(csa2.dense_attn_workspace_bytes(d, 2), dtype=torch.uint8, device="cuda") for _ in cs]
    sl = torch.tensor([20000, 300], dtype=torch.int32, device="cuda")
    bufs = [[(torch.empty((2, 16, 128), device="cuda"), torch.empty((2, 16), device="cuda")) for _ in range(5)] for _ in cs]
    torch.cuda.synchronize()
    for i in range(5):
        for c, q, s, w, o in zip(cs, qs, streams, ws, bufs):
            csa2.dense_attn_decode(d, c.cache, q, sl, o[i][0], o[i][1], c.max_len, w, stream=s)
    torch.cuda.synchronize()
    for o, (w_out, w_lse) in zip(bufs, want):
        for x, y in o:
            assert torch.equal(x, w_out) and torch.equal(y, w_lse)


def test_dense_and_window_equal_the_sparse_step(csa2):
    """At up to 512 entries every entry is selected: dense attention merged with
    the window's part by csa2_attn_lse_merge is csa2_sparse_attn_decode's result."""
    from _gpu_util import PagedSeqs, bits16, dev
    lens, seed = [512, 77, 300], 1001
    ps = PagedSeqs(csa2, lens)
    for b, n in enumerate(lens):
        ps.append(b, 0, synth.kv_rows(seed, b, 0, n), synth.idx_k_rows(seed, b, 0, n))
    d = csa2.default_desc(csa2.FULL, 1)
    q = bits16(np.concatenate([synth.q_heads(seed, 0, b) for b in range(3)]))
    swa = bits16(np.stack([synth.swa_rows(seed, 0, b, 128) for b in range(3)]))
    sl = dev(np.array(lens, np.int32))
    every = torch.full((3, 512), -1, dtype=torch.int32)
    for b, n in enumerate(lens):
        every[b, :n] = torch.arange(n)
    new = lambda *s: torch.empty(s, device="cuda")  # noqa: E731
    want, want_lse = new(3, 16, 128), new(3, 16)
    csa2.sparse_attn_decode(d, ps.cache, q, every.cuda(), swa, sl, want, want_lse, 3, err=ps.err)
    parts, lses = new(2, 3, 16, 128), new(2, 3, 16)
    none = torch.full((3, 512), -1, dtype=torch.int32, device="cuda")
    csa2.sparse_attn_decode(d, ps.cache, q, none, swa, sl, parts[1], lses[1], 3, err=ps.err)
    ws = torch.empty(csa2.dense_attn_workspace_bytes(d, 3), dtype=torch.uint8, device="cuda")
    csa2.dense_attn_decode(d, ps.cache, q, sl, parts[0], lses[0], 512, ws, err=ps.err)
    out, lse = new(3, 16, 128), new(3, 16)
    csa2.attn_lse_merge(parts, lses, out, lse)
    assert ps.errors() == 0
    assert (out - want).abs().max() <= 2e-3 and (lse - want_lse).abs().max() <= 2e-3  # the sparse path's tolerance


def test_many_short_sequences_and_large_pages(csa2):
    """More sequences than CTAs, some empty; pages larger than a tile."""
    lens = [(37 * b) % 300 for b in range(400)]
    c = DenseCase(csa2, lens, 16, seed=40)
    q = queries(400, seed=41)
    out, lse, err = decode(csa2, c, q, torch.bfloat16)
    outp, lsep, errp = prefill(csa2, c, q, list(range(401)), torch.float32, [max(0, n - 1) for n in lens])
    assert err == errp == 0
    for b in (0, 1, 73, 147, 148, 299, 300, 399):
        ref = reference(q[b:b + 1], c.rows(b), [lens[b]])
        check(out[b:b + 1], lse[b:b + 1], ref, f"decode {b}")
        check(outp[b:b + 1], lsep[b:b + 1], reference(q[b:b + 1], c.rows(b), [min(lens[b], max(0, lens[b] - 1) + 1)]), f"prefill {b}")
    c = DenseCase(csa2, [5000, 1025], 1024, seed=42)
    q = queries(2, seed=43)
    out, lse, err = decode(csa2, c, q, torch.float32)
    for b in range(2):
        check(out[b:b + 1], lse[b:b + 1], reference(q[b:b + 1], c.rows(b), [c.lens[b]]), f"pages of 1024, {b}")


def test_ranges_that_overlap_without_end(csa2):
    """Ranges that go back to row 0 again and again: their places in the list of
    work pass 32 bits, though T and the lengths are in bounds.  Nothing is done."""
    B, T, page, cols = 1024, 4096, 1 << 16, 64
    table = torch.full((B, cols), -1, dtype=torch.int32, device="cuda")
    cache = csa2.KVCache.from_tensors(torch.zeros((page, 128), dtype=torch.uint8, device="cuda"),
                                      torch.zeros((page, 16), dtype=torch.uint8, device="cuda"), table, page)
    d = csa2.default_desc(csa2.FULL, 1)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    cu, sl = i32([0, T] * (B // 2) + [0]), i32([page * cols] * B)
    out = torch.full((T, 16, 128), 7.0, device="cuda")
    lse = torch.full((T, 16), 7.0, device="cuda")
    ws = torch.empty(csa2.dense_attn_workspace_bytes(d, B, True), dtype=torch.uint8, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert (B // 2) * (T // 16) * (page * cols // 128 + 1) > 2**32
    csa2.dense_attn_prefill(d, cache, queries(T).cuda(), cu, sl, out, lse, page * cols, ws, err=err)
    torch.cuda.synchronize()
    assert int(err) & DEV_LEN and (out == 7).all() and (lse == 7).all()


def test_nothing_to_see(csa2):
    """No entries in any sequence; no tokens in any sequence."""
    c = DenseCase(csa2, [0, 0, 0], 64)
    q = queries(3)
    for dt in DT.values():
        out, lse, err = decode(csa2, c, q, dt)
        assert err == 0 and (out == 0).all() and (lse == -math.inf).all()
        out, lse, err = prefill(csa2, c, q, [0, 2, 2, 3], dt)
        assert err == 0 and (out == 0).all() and (lse == -math.inf).all()
        out, lse, err = prefill(csa2, c, q, [1, 1, 1, 1], dt, [0, 0, 0])
        assert err == 0 and (out == 7).all() and (lse == 7).all()


@pytest.mark.parametrize("n", [1, 65, 129])
def test_a_lone_bad_entry(csa2, n):
    """The only entries that some part of the work sees have NaN scales of K: the sum of that part counts."""
    c = DenseCase(csa2, [n], 64, seed=5)
    c.cache.scales[c.slots(0, n)[-1], :8] = 0x7F
    q = queries(1)
    for dt in DT.values():
        for out, lse in (decode(csa2, c, q, dt)[:2], prefill(csa2, c, q, [0, 1], dt, [n - 1])[:2]):
            assert torch.isnan(lse).all() and torch.isnan(out).all()


@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_a_bad_query_is_its_heads_alone(csa2, bad):
    c = DenseCase(csa2, [333], 64, seed=3)
    q = queries(12)
    q[3, 5, 17] = bad
    rest = torch.ones((12, 16), dtype=torch.bool)
    rest[3, 5] = False
    for dt in DT.values():
        for out, lse in ((prefill(csa2, c, q, [0, 12], dt, [321])[:2]),
                         [torch.cat([decode(csa2, c, q[i:i + 1], dt, lens=[322 + i])[k] for i in range(12)]) for k in (0, 1)]):
            assert torch.isnan(out[3, 5]).all() and torch.isnan(lse[3, 5])
            clean = queries(12)
            ref = reference(clean, c.rows(0), seen_of(333, 12, 321, 1))
            for i in range(12):
                keep = rest[i].cuda()
                check(out[i:i + 1, keep], lse[i:i + 1, keep], tuple(x[i:i + 1, rest[i]] for x in ref), f"token {i}")


def test_prefills_on_two_streams(csa2):
    """Calls that run side by side, each with its own workspace, do not disturb one another."""
    d = csa2.default_desc(csa2.FULL, 1)
    cs = [DenseCase(csa2, [2000, 700], 64, seed=s) for s in (1, 2)]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    cu, st, sl = i32([0, 100, 130]), i32([1900, 670]), i32([2000, 700])
    qs = [queries(130, seed=s).cuda() for s in (3, 4)]
    want = [prefill(csa2, c, q.cpu(), [0, 100, 130], torch.bfloat16, [1900, 670])[:2] for c, q in zip(cs, qs)]
    streams = [torch.cuda.Stream() for _ in cs]
    ws = [torch.empty(csa2.dense_attn_workspace_bytes(d, 2, True), dtype=torch.uint8, device="cuda") for _ in cs]
    out = [[torch.empty((130, 16, 128), dtype=torch.bfloat16, device="cuda") for _ in range(4)] for _ in cs]
    lse = [[torch.empty((130, 16), device="cuda") for _ in range(4)] for _ in cs]
    torch.cuda.synchronize()
    for i in range(4):
        for k in range(2):
            csa2.dense_attn_prefill(d, cs[k].cache, qs[k], cu, sl, out[k][i], lse[k][i], cs[k].max_len, ws[k],
                                    q_start=st, stream=streams[k])
    torch.cuda.synchronize()
    for k in range(2):
        for i in range(4):
            assert torch.equal(out[k][i], want[k][0]) and torch.equal(lse[k][i], want[k][1])


def test_main_kv_in_host_memory_is_refused(csa2):
    c = csa2.KVCache(4, 64, torch.arange(4, dtype=torch.int32).view(1, 4), main_kv_on_host=True)
    d = csa2.default_desc(csa2.FULL, 1)
    ws = torch.empty(csa2.dense_attn_workspace_bytes(d, 1), dtype=torch.uint8, device="cuda")
    with pytest.raises(csa2.CSA2Error) as e:
        csa2.dense_attn_decode(d, c, queries(1).cuda(), torch.ones(1, dtype=torch.int32, device="cuda"),
                               torch.empty((1, 16, 128), device="cuda"), torch.empty((1, 16), device="cuda"), 64, ws)
    assert e.value.status == 2
