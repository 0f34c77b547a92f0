"""The latent cache store and the latent attention against the float64 oracle
(needs a B200).  Tolerances are oracle.latent.limits(), derived there."""
import numpy as np
import pytest
import torch

import oracle
import fp8_mqa_logits_03_b200 as fx
from fp8_mqa_logits_03_b200 import workloads
from oracle import latent as lo

pytestmark = pytest.mark.gpu

SCALE = 192 ** -0.5
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from fp8_mqa_logits_03_b200 import build
    build.build()
    fx.lib()


def _pool(pages, fp8, seed, spread=0.5):
    """A random pool on the GPU and its rows as float64 keys."""
    g = torch.Generator().manual_seed(seed)
    size = torch.exp(spread * torch.randn(pages * 64, 1, generator=g))
    kv = (torch.randn(pages * 64, 576, generator=g) * size).to(BF)
    if not fp8:
        return dict(kv_pages=kv.view(pages, 64, 576).cuda()), kv.double().numpy()
    codes, s = lo.quantise(kv[:, :512].float().numpy())
    pe = kv[:, 512:].contiguous()
    dev = dict(kv_pages=torch.from_numpy(codes).view(pages, 64, 512).cuda(), s_pages=torch.from_numpy(s).view(pages, 64).cuda(),
               pe_pages=pe.view(pages, 64, 64).cuda())
    return dev, lo.keys_of(codes, s, pe.double().numpy())


def _q(rows, H, seed, strided=False):
    g = torch.Generator().manual_seed(seed)
    q = torch.randn(rows, H, 576, generator=g).to(BF)
    if not strided:
        return q.cuda(), q.double().numpy()
    wide = torch.zeros(rows, H + 2, 640, dtype=BF)   # rows and heads with room between them
    wide[:, 1:H + 1, 32:608] = q
    return wide.cuda()[:, 1:H + 1, 32:608], q.double().numpy()


def _check_row(out, lse, q, keys, fp8, what, scale=SCALE):
    """One row's columns [H, ...] against the oracle over the keys it sees."""
    want, wl = lo.attend(q, keys, scale)
    tol, ltol = lo.limits(q, keys, scale, fp8)
    if len(keys) == 0:
        assert not out.any() and np.isneginf(lse).all(), what
        return
    assert np.isfinite(out).all() and np.isfinite(lse).all(), what
    over = np.abs(out - want) - tol
    assert (over <= 0).all(), f"{what}: out off by {np.abs(out - want).max():.3g}, {int((over > 0).sum())} over, worst {over.max():.3g}"
    assert (np.abs(lse - wl) <= ltol).all(), f"{what}: lse off by {np.abs(lse - wl).max():.3g} (allowed {ltol.min():.3g})"


def _np(t):
    return t.double().cpu().numpy()


# ------------------------------------------------------------------ store

def _store_case(T, H, fp8, interleaved, seed, pages=8):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, 584, generator=g).to(BF)[:, :576]    # a row stride that is not the width
    qx = torch.randn(T, max(H, 1), 200, generator=g).to(BF)
    ang = torch.arange(500)[:, None].double() * 10000.0 ** (-torch.arange(0, 64, 2).double() / 64)
    tab = torch.cat([ang.cos(), ang.sin()], -1).float()
    pos = torch.randint(0, 500, (T,), generator=g)
    slot = torch.randperm(pages * 64, generator=g)[:T]
    if T > 8:
        slot[2], slot[5] = -1, pages * 64            # not stored
        pos[3], pos[7] = 500, -1                     # left out altogether
    return x, qx, tab, pos, slot


def _rot_tol(x, tab, pos, want):
    """fp32 products and one sum: 2^-24 of each product and of the sum (the
    product is exact in a fused form), then half a step of bf16."""
    mag = np.abs(x).max(axis=-1, keepdims=True) * 2.0
    return 2.0 ** -8 * np.abs(want) + 3 * 2.0 ** -24 * mag


@pytest.mark.parametrize("T,H", [(1, 1), (5, 0), (9, 16), (300, 20), (131, 128)])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("interleaved", [True, False])
def test_store(T, H, fp8, interleaved):
    pages = 8
    x, qx, tab, pos, slot = _store_case(T, H, fp8, interleaved, 100 + T + H)
    n = pages * 64
    if fp8:
        pool = dict(kv_pages=torch.full((pages, 64, 512), 0xAB, dtype=torch.uint8).cuda(),
                    s_pages=torch.full((pages, 64), -7.0).cuda(), pe_pages=torch.full((pages, 64, 64), 3.0, dtype=BF).cuda())
    else:
        pool = dict(kv_pages=torch.full((pages, 64, 576), 3.0, dtype=BF).cuda())
    xd = x.cuda()
    qd = qx.cuda()
    qo = torch.full((T, max(H, 1), 576), 9.0, dtype=BF).cuda()
    kw = dict(q_pe=qd[..., 128:192], q_out=qo[..., 512:]) if H else {}
    fx.latent_store(xd[:, :512], xd[:, 512:], pos.cuda(), tab.cuda(), slot.cuda(), **pool, **kw, interleaved=interleaved)
    torch.cuda.synchronize()
    inside = (pos >= 0) & (pos < 500)
    kept = (inside & (slot >= 0) & (slot < n)).numpy()
    at = slot.numpy()[kept]
    xf = x.double().numpy()
    p0 = pos.clamp(0, 499).numpy()
    want_pe = lo.rotate(xf[:, 512:], tab.numpy(), p0, interleaved)
    tol = _rot_tol(xf[:, 512:], tab, p0, want_pe)
    other = np.ones(n, bool)
    other[at] = False
    if fp8:
        codes, s = lo.quantise(x[:, :512].float().numpy())
        got_c, got_s = pool["kv_pages"].view(n, 512).cpu().numpy(), pool["s_pages"].view(n).cpu().numpy()
        got_pe = _np(pool["pe_pages"]).reshape(n, 64)
        assert np.array_equal(got_c[at], codes[kept]) and np.array_equal(got_s[at], s[kept])
        assert (got_c[other] == 0xAB).all() and (got_s[other] == -7).all()
    else:
        kv = pool["kv_pages"].view(n, 576)
        assert torch.equal(kv[torch.from_numpy(at).cuda(), :512].cpu(), x[torch.from_numpy(kept)][:, :512])
        got_pe = _np(kv)[:, 512:]
        assert (_np(kv)[other] == 3).all()
    assert (np.abs(got_pe[at] - want_pe[kept]) <= tol[kept]).all()
    assert (got_pe[other] == 3).all()
    if H:
        qf = qx.double().numpy()[..., 128:192]
        want = lo.rotate(qf, tab.numpy(), p0, interleaved)
        got = _np(qo)
        assert (got[..., :512] == 9).all()
        ins = inside.numpy()
        assert (np.abs(got[ins][..., 512:] - want[ins]) <= _rot_tol(qf, tab, p0, want)[ins]).all()
        assert (got[~ins] == 9).all()


def test_store_in_place_and_non_finite_values():
    """q_out may be q_pe; NaN and infinities reach their own token's entry only."""
    T, pages = 6, 1
    x, qx, tab, pos, slot = _store_case(T, 4, True, True, 7, pages)
    x = x.clone()
    x[1, 5], x[2, 9], x[3, 520] = float("nan"), float("inf"), float("nan")
    x[4, :512] = 0
    pool = dict(kv_pages=torch.zeros(pages, 64, 512, dtype=torch.uint8).cuda(), s_pages=torch.zeros(pages, 64).cuda(),
                pe_pages=torch.zeros(pages, 64, 64, dtype=BF).cuda())
    qd = qx.cuda()
    sep = torch.zeros(T, 4, 64, dtype=BF).cuda()
    args = (x.cuda()[:, :512], x.cuda()[:, 512:], pos.cuda(), tab.cuda(), slot.cuda())
    fx.latent_store(*args, **pool, q_pe=qd[..., 8:72], q_out=sep)
    fx.latent_store(*args, **pool, q_pe=qd[..., 8:72], q_out=qd[..., 8:72])
    assert torch.equal(qd[..., 8:72], sep)
    s = pool["s_pages"].view(-1).cpu()[slot]
    assert torch.isnan(s[1]) and torch.isinf(s[2]) and torch.isfinite(s[[0, 3, 4, 5]]).all()
    assert s[4] == torch.tensor(1e-4) / 448
    pe = pool["pe_pages"].view(-1, 64).cpu()[slot]
    assert torch.isnan(pe[3]).any() and torch.isfinite(pe[[0, 1, 2, 4, 5]]).all()


# ------------------------------------------------------------------ selected slots

def _slots(rows, topk, n, seed, counts=None):
    g = np.random.default_rng(seed)
    out = np.full((rows, topk), -1, np.int32)
    for i in range(rows):
        c = topk if counts is None else counts[i % len(counts)]
        out[i, :c] = g.permutation(n)[:c]
    return out


SPARSE = [
    # rows, H, topk, pages, counts
    (1, 1, 1, 1, None), (1, 16, 64, 2, None), (1, 16, 65, 3, None), (2, 64, 63, 2, None), (3, 128, 2048, 40, None),
    (5, 20, 700, 16, (0, 1, 63, 700, 64)), (150, 8, 130, 4, None), (149, 3, 64, 2, (64, 0, 5)), (300, 65, 200, 8, (200, 129, 1)),
    (7, 100, 1000, 32, None),
]


@pytest.mark.parametrize("rows,H,topk,pages,counts", SPARSE)
@pytest.mark.parametrize("fp8", [False, True])
def test_sparse(rows, H, topk, pages, counts, fp8):
    dev, keys = _pool(pages, fp8, 200 + rows)
    q, qn = _q(rows, H, 201, strided=rows % 2 == 1)
    sl = _slots(rows, topk, pages * 64, 202, counts)
    ws = fx.alloc_workspace(fx.sparse_latent_workspace_size(rows, H, topk))
    out, lse = fx.sparse_latent_attention(q, slots=torch.from_numpy(sl).cuda(), scale=SCALE, **dev, return_lse=True, workspace=ws)
    assert fx.read_device_status(ws) == 0
    out, lse = _np(out), _np(lse)
    for i in range(rows):
        if rows > 20 and i % 7 and i > 3:
            continue
        _check_row(out[i], lse[i], qn[i], keys[sl[i][sl[i] >= 0]], fp8, f"row {i}")


@pytest.mark.parametrize("fp8", [False, True])
def test_sparse_gaps_duplicates_and_strides(fp8):
    """Negative entries anywhere, whole tiles of them, a slot named twice, a row stride above topk."""
    dev, keys = _pool(6, fp8, 210)
    rows, H, topk = 6, 12, 400
    q, qn = _q(rows, H, 211)
    g = np.random.default_rng(212)
    sl = g.integers(0, 384, (rows, topk)).astype(np.int32)      # with repeats
    sl[0, ::3] = -1
    sl[1, :] = -1
    sl[2, 64:320] = -5                                          # four empty tiles in the middle
    sl[3, :384] = np.iinfo(np.int32).min
    sl[4, :] = 17
    wide = torch.full((rows, topk + 50), 3, dtype=torch.int32)
    wide[:, :topk] = torch.from_numpy(sl)
    out, lse = fx.sparse_latent_attention(q, slots=wide.cuda()[:, :topk], scale=SCALE, **dev, return_lse=True)
    out, lse = _np(out), _np(lse)
    for i in range(rows):
        _check_row(out[i], lse[i], qn[i], keys[sl[i][sl[i] >= 0]], fp8, f"row {i}")


@pytest.mark.parametrize("fp8", [False, True])
def test_sparse_non_finite_slots(fp8):
    """NaN and infinities in slots that a row does not name stay out of it (slot
    0, which padding might read, among them); in one that it names they show."""
    dev, keys = _pool(4, fp8, 220)
    where = [0, 100, 101]
    if fp8:
        dev["s_pages"].view(-1)[where] = torch.tensor([float("nan"), float("inf"), float("nan")]).cuda()
        dev["pe_pages"].view(-1, 64)[0] = float("nan")
    else:
        dev["kv_pages"].view(-1, 576)[where] = torch.tensor([float("nan"), float("inf"), -float("inf")], dtype=BF)[:, None].cuda()
    rows, H, topk = 3, 64, 200
    q, qn = _q(rows, H, 221)
    ok = np.array([j for j in range(256) if j not in where], np.int32)
    sl = np.full((rows, topk), -1, np.int32)
    sl[0, :150], sl[1, :70], sl[2, :10] = ok[:150], ok[100:170], ok[:10]
    sl[1, 70] = 100
    out, lse = fx.sparse_latent_attention(q, slots=torch.from_numpy(sl).cuda(), scale=SCALE, **dev, return_lse=True)
    out, lse = _np(out), _np(lse)
    for i in (0, 2):
        _check_row(out[i], lse[i], qn[i], keys[sl[i][sl[i] >= 0]], fp8, f"row {i}")
    assert np.isnan(out[1]).any(axis=-1).all()


@pytest.mark.parametrize("fp8", [False, True])
def test_sparse_slot_past_the_pool(fp8):
    dev, keys = _pool(2, fp8, 230)
    q, qn = _q(2, 4, 231)
    sl = np.array([[5, 128, 7, 2 ** 31 - 1], [1, 2, 3, -1]], np.int32)
    ws = fx.alloc_workspace(fx.sparse_latent_workspace_size(2, 4, 4))
    out, lse = fx.sparse_latent_attention(q, slots=torch.from_numpy(sl).cuda(), scale=SCALE, **dev, return_lse=True, workspace=ws)
    assert fx.read_device_status(ws) == fx.STATUS_BAD_SLOT
    _check_row(_np(out)[0], _np(lse)[0], qn[0], keys[[5, 7]], fp8, "row 0")
    _check_row(_np(out)[1], _np(lse)[1], qn[1], keys[[1, 2, 3]], fp8, "row 1")


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("order", ["rising", "falling"])
def test_sparse_maxima_that_move(fp8, order):
    """Scores that climb by far more than the rescaling threshold from tile to
    tile (every tile rescales), or fall (later weights vanish)."""
    pages, H, topk = 8, 64, 512
    g = torch.Generator().manual_seed(240)
    base = torch.randn(576, generator=g)
    level = torch.linspace(0, 3.0, 512)
    if order == "falling":
        level = level.flip(0)
    kv = (0.3 * torch.randn(512, 576, generator=g) + level[:, None] * base).to(BF)
    q = (torch.randn(2, H, 576, generator=g) * 0.3 + base).to(BF)
    if fp8:
        codes, s = lo.quantise(kv[:, :512].float().numpy())
        pe = kv[:, 512:].contiguous()
        dev = dict(kv_pages=torch.from_numpy(codes).view(pages, 64, 512).cuda(), s_pages=torch.from_numpy(s).view(pages, 64).cuda(),
                   pe_pages=pe.view(pages, 64, 64).cuda())
        keys = lo.keys_of(codes, s, pe.double().numpy())
    else:
        dev, keys = dict(kv_pages=kv.view(pages, 64, 576).cuda()), kv.double().numpy()
    sl = torch.arange(512, dtype=torch.int32).repeat(2, 1)
    out, lse = fx.sparse_latent_attention(q.cuda(), slots=sl.cuda(), scale=SCALE, **dev, return_lse=True)
    for i in range(2):
        _check_row(_np(out)[i], _np(lse)[i], q.double().numpy()[i], keys, fp8, f"row {i}")


@pytest.mark.parametrize("fp8", [False, True])
def test_sparse_query_outliers(fp8):
    """Columns whose values differ by many powers of two, zero columns and tiny ones."""
    dev, keys = _pool(3, fp8, 250)
    g = torch.Generator().manual_seed(251)
    q = torch.randn(1, 8, 576, generator=g)
    q[0, 0, 7] = 1000.0
    q[0, 1] = 0
    q[0, 2] *= 1e-6
    q[0, 3] *= torch.exp(3 * torch.randn(576, generator=g))
    q[0, 4, 520] = -300.0
    q = q.to(BF)
    sl = torch.arange(192, dtype=torch.int32)[None]
    scale = 0.01
    out, lse = fx.sparse_latent_attention(q.cuda(), slots=sl.cuda(), scale=scale, **dev, return_lse=True)
    _check_row(_np(out)[0], _np(lse)[0], q.double().numpy()[0], keys, fp8, "row 0", scale)


def test_sparse_wide_range_of_scales():
    """fp8 pool: token scales from 1e-6 to 1e3, and a zero scale (a key of zeros)."""
    dev, _ = _pool(4, True, 260)
    g = torch.Generator().manual_seed(261)
    s = 10.0 ** (-6 + 9 * torch.rand(256, generator=g))
    s[10] = 0.0
    dev["s_pages"] = s.view(4, 64).cuda()
    keys = lo.keys_of(dev["kv_pages"].view(-1, 512).cpu().numpy(), s.numpy(), _np(dev["pe_pages"]).reshape(-1, 64))
    q, qn = _q(1, 16, 262)
    q, qn = q * 0.001, None
    qn = _np(q)
    sl = torch.arange(256, dtype=torch.int32)[None].cuda()
    out, lse = fx.sparse_latent_attention(q, slots=sl, scale=0.001, **dev, return_lse=True)
    _check_row(_np(out)[0], _np(lse)[0], qn[0], keys, True, "row 0", 0.001)


def test_sparse_empty_calls():
    dev, _ = _pool(1, False, 270)
    q, _ = _q(3, 5, 271)
    out, lse = fx.sparse_latent_attention(q, slots=torch.zeros(3, 0, dtype=torch.int32).cuda(), scale=SCALE, **dev, return_lse=True)
    assert not out.any() and torch.isneginf(lse).all()
    out = fx.sparse_latent_attention(q[:0], slots=torch.zeros(0, 4, dtype=torch.int32).cuda(), scale=SCALE, **dev)
    assert out.shape == (0, 5, 512)
    none = dict(kv_pages=torch.zeros(0, 64, 576, dtype=BF).cuda())
    out, lse = fx.sparse_latent_attention(q, slots=torch.full((3, 9), -1, dtype=torch.int32).cuda(), scale=SCALE, **none, return_lse=True)
    assert not out.any() and torch.isneginf(lse).all()


# ------------------------------------------------------------------ paged

def _paged_case(lengths, R, H, fp8, seed, extra_blocks=1):
    per = [max(0, (l + 63) // 64) for l in lengths]
    pages = sum(per) + 1
    dev, keys = _pool(pages, fp8, seed)
    g = np.random.default_rng(seed + 1)
    perm = g.permutation(pages)
    table = np.full((len(lengths), max(max(per), 1) + extra_blocks), -1, np.int32)
    off = 0
    for b, c in enumerate(per):
        table[b, :c] = perm[off:off + c]
        off += c
    q, qn = _q(len(lengths) * R, H, seed + 2)
    return dev, keys, table, q, qn


def _logical(table, b, l):
    j = np.arange(l)
    return table[b][j // 64].astype(np.int64) * 64 + j % 64


def _check_paged(out, lse, lengths, R, qn, keys, table, fp8):
    out, lse = _np(out), _np(lse)
    for b, l in enumerate(lengths):
        at = _logical(table, b, max(l, 0))
        for t in range(R):
            i = b * R + t
            _check_row(out[i], lse[i], qn[i], keys[at[:max(0, l - R + t + 1)]], fp8, f"request {b} (length {l}) row {t}")


PAGED = [
    ([64], 1, 16), ([1, 0, 65, 300], 1, 64), ([2, 64, 128, 129, 700], 4, 16), ([5, 1, 0, 3, 200], 8, 20), ([4096], 1, 16),
    ([3000, 1, 2500], 2, 128), ([100, 64, 63] * 60, 1, 5), ([1000, 10], 3, 100), ([20000], 8, 128),
]


@pytest.mark.parametrize("lengths,R,H", PAGED)
@pytest.mark.parametrize("fp8", [False, True])
def test_paged(lengths, R, H, fp8):
    dev, keys, table, q, qn = _paged_case(lengths, R, H, fp8, 300 + len(lengths) + R + H)
    ws = fx.alloc_workspace(fx.paged_latent_workspace_size(len(lengths), R, table.shape[1], H))
    out, lse = fx.paged_latent_attention(q, block_table=torch.from_numpy(table).cuda(),
                                         seq_lens=torch.tensor(lengths, dtype=torch.int32).cuda(), R=R, scale=SCALE, **dev,
                                         return_lse=True, workspace=ws)
    assert fx.read_device_status(ws) == 0
    if len(lengths) > 10 or max(lengths) > 10000:   # a sample
        keep = [0, 1, len(lengths) - 1] if len(lengths) > 10 else [0]
        out, lse = _np(out), _np(lse)
        for b in keep:
            at = _logical(table, b, lengths[b])
            for t in range(R):
                i = b * R + t
                _check_row(out[i], lse[i], qn[i], keys[at[:max(0, lengths[b] - R + t + 1)]], fp8, f"request {b} row {t}")
        return
    _check_paged(out, lse, lengths, R, qn, keys, table, fp8)


@pytest.mark.parametrize("fp8", [False, True])
def test_paged_garbage_behind_the_keys(fp8):
    """What the pool holds past a request's length, and the keys that only later
    rows see, never reach a row: NaN and infinities there change nothing."""
    lengths, R, H = [70, 130, 64, 3], 4, 40
    dev, keys, table, q, qn = _paged_case(lengths, R, H, fp8, 350)
    bad = torch.ones(keys.shape[0], dtype=torch.bool)
    for b, l in enumerate(lengths):
        bad[torch.from_numpy(_logical(table, b, l))] = False
    tail = [int(_logical(table, b, l)[-1]) for b, l in enumerate(lengths)]     # the last token: row R - 1 alone sees it
    for at in list(torch.nonzero(bad)[:, 0]) + tail:
        if fp8:
            dev["s_pages"].view(-1)[at] = float("nan")
            dev["pe_pages"].view(-1, 64)[at] = float("inf")
        else:
            dev["kv_pages"].view(-1, 576)[at] = float("nan")
    out, lse = fx.paged_latent_attention(q, block_table=torch.from_numpy(table).cuda(),
                                         seq_lens=torch.tensor(lengths, dtype=torch.int32).cuda(), R=R, scale=SCALE, **dev,
                                         return_lse=True)
    out, lse = _np(out), _np(lse)
    for b, l in enumerate(lengths):
        at = _logical(table, b, l)
        for t in range(R - 1):
            i = b * R + t
            _check_row(out[i], lse[i], qn[i], keys[at[:max(0, l - R + t + 1)]], fp8, f"request {b} row {t}")
        assert np.isnan(lse[b * R + R - 1]).all()


@pytest.mark.parametrize("fp8", [False, True])
def test_paged_bad_pages_and_lengths(fp8):
    lengths, R, H = [200, 130], 1, 8
    dev, keys, table, q, qn = _paged_case(lengths, R, H, fp8, 360, extra_blocks=0)
    args = dict(R=R, scale=SCALE, **dev, return_lse=True)
    ws = fx.alloc_workspace(fx.paged_latent_workspace_size(2, R, table.shape[1], H))
    broken = table.copy()
    broken[0, 1] = keys.shape[0] // 64       # a page past the pool: its keys are left out
    out, lse = fx.paged_latent_attention(q, block_table=torch.from_numpy(broken).cuda(),
                                         seq_lens=torch.tensor(lengths, dtype=torch.int32).cuda(), workspace=ws, **args)
    assert fx.read_device_status(ws) == fx.STATUS_BAD_PAGE
    at = np.delete(_logical(table, 0, 200), np.arange(64, 128))
    _check_row(_np(out)[0], _np(lse)[0], qn[0], keys[at], fp8, "request 0")
    _check_row(_np(out)[1], _np(lse)[1], qn[1], keys[_logical(table, 1, 130)], fp8, "request 1")
    # a length beyond the block table is clamped to it, a negative one is empty
    long = torch.tensor([10 ** 6, -5], dtype=torch.int32).cuda()
    full = table.copy()
    full[0] = table[0][0]
    out, lse = fx.paged_latent_attention(q, block_table=torch.from_numpy(full).cuda(), seq_lens=long, workspace=ws, **args)
    assert fx.read_device_status(ws) == fx.STATUS_SEQ_TOO_LONG
    _check_row(_np(out)[0], _np(lse)[0], qn[0], keys[_logical(full, 0, 64 * table.shape[1])], fp8, "request 0")
    _check_row(_np(out)[1], _np(lse)[1], qn[1], keys[:0], fp8, "request 1")
    out, lse = fx.paged_latent_attention(q, block_table=torch.from_numpy(table).cuda(),
                                         seq_lens=torch.tensor(lengths, dtype=torch.int32).cuda(), workspace=ws, **args)
    assert fx.read_device_status(ws) == 0
    _check_paged(out, lse, lengths, R, qn, keys, table, fp8)


def test_offsets_past_32_bits():
    """Slots whose byte (and value) offsets pass 2^32, both pools."""
    pages = 66000                                # 4.2 M tokens
    H, rows = 16, 2
    q, qn = _q(rows, H, 371)
    g = torch.Generator(device="cuda").manual_seed(372)
    at = torch.randint(pages * 64 - 5000, pages * 64, (rows, 130), device="cuda", generator=g)
    kv = torch.empty(pages, 64, 576, dtype=BF, device="cuda")
    rows_of = torch.randn(5000, 576, device="cuda", generator=g).to(BF)
    kv.view(-1, 576)[-5000:] = rows_of
    out, lse = fx.sparse_latent_attention(q, kv, at.int(), SCALE, return_lse=True)
    keys = _np(rows_of)
    for i in range(rows):
        _check_row(_np(out)[i], _np(lse)[i], qn[i], keys[(at[i] - (pages * 64 - 5000)).cpu().numpy()], False, f"row {i}")
    table = torch.arange(pages - 40, pages, dtype=torch.int32, device="cuda")[None]
    out, lse = fx.paged_latent_attention(q[:1], kv, table, torch.tensor([2500], dtype=torch.int32).cuda(), 1, SCALE, return_lse=True)
    _check_row(_np(out)[0], _np(lse)[0], qn[0], keys[5000 - 2560:][:2500], False, "paged")
    # the store reaches the last slot
    x = torch.randn(1, 576, device="cuda", generator=g).to(BF)
    tab = torch.cat([torch.ones(1, 32), torch.zeros(1, 32)], -1).cuda()
    fx.latent_store(x[:, :512], x[:, 512:], torch.zeros(1, dtype=torch.int64).cuda(), tab,
                    torch.tensor([pages * 64 - 1]).cuda(), kv)
    assert torch.equal(kv.view(-1, 576)[-1], x[0])


def _ragged_lengths(B, top, seed):
    """Lengths from 0 to `top`, the longest and the shortest among them."""
    g = np.random.default_rng(seed)
    l = g.integers(0, top + 1, B)
    l[g.integers(0, B)], l[g.integers(0, B)] = top, 0
    return [int(v) for v in l]


# how the requests are shared out depends on their number (a lane or a thread
# each, or several a thread) and on whether each can have CTAs of its own
@pytest.mark.parametrize("B,top,R,H", [(12, 900, 2, 16), (32, 400, 1, 64), (33, 500, 1, 40), (20, 4000, 1, 8), (5, 6000, 8, 128), (147, 200, 1, 24),
                                       (150, 130, 1, 64), (460, 100, 3, 4), (600, 70, 1, 3)])
@pytest.mark.parametrize("fp8", [False, True])
def test_paged_many_requests(B, top, R, H, fp8):
    lengths = _ragged_lengths(B, top, 380 + B)
    dev, keys, table, q, qn = _paged_case(lengths, R, H, fp8, 381 + B)
    out, lse = fx.paged_latent_attention(q, block_table=torch.from_numpy(table).cuda(),
                                         seq_lens=torch.tensor(lengths, dtype=torch.int32).cuda(), R=R, scale=SCALE, **dev,
                                         return_lse=True)
    out, lse = _np(out), _np(lse)
    order = np.argsort(lengths)
    for b in sorted({0, 1, B // 2, B - 2, B - 1, int(order[0]), int(order[1]), int(order[-1]), *range(0, B, max(1, B // 12))}):
        at = _logical(table, b, lengths[b])
        for t in range(R):
            i = b * R + t
            _check_row(out[i], lse[i], qn[i], keys[at[:max(0, lengths[b] - R + t + 1)]], fp8, f"request {b} row {t}")


# ranges that end with rows (many of them), rows with CTAs of their own, cut rows; one and two column blocks
@pytest.mark.parametrize("rows,H,topk,counts", [(3, 128, 2048, None), (40, 64, 2048, None), (148, 64, 320, (320, 1, 256, 0, 64)),
                                                (500, 64, 320, (320, 1, 256, 0, 64)), (9, 16, 4096, None), (600, 100, 192, None)])
@pytest.mark.parametrize("fp8", [False, True])
def test_sparse_same_bits_in_many_runs(rows, H, topk, counts, fp8):
    """Calls back to back on the same inputs: a missing wait shows as a run that
    differs.  A sample of the rows is checked too."""
    pages = 64
    dev, keys = _pool(pages, fp8, 390 + rows)
    q, qn = _q(rows, H, 391)
    sln = _slots(rows, topk, pages * 64, 392, counts)
    sl = torch.from_numpy(sln).cuda()
    out, lse = fx.sparse_latent_attention(q, slots=sl, scale=SCALE, **dev, return_lse=True)
    wrong = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(200):
        o, l = fx.sparse_latent_attention(q, slots=sl, scale=SCALE, **dev, return_lse=True)
        wrong += (o != out).any() | (l != lse).any()
    assert wrong.item() == 0
    o, l = _np(out), _np(lse)
    for i in range(0, rows, max(1, rows // 10)):
        _check_row(o[i], l[i], qn[i], keys[sln[i][sln[i] >= 0]], fp8, f"row {i}")


# ------------------------------------------------------------------ how it is called

def _args(fp8, rows=5, H=24, topk=300, seed=400):
    dev, keys = _pool(10, fp8, seed)
    q, qn = _q(rows, H, seed + 1)
    sl = _slots(rows, topk, 640, seed + 2)
    return dev, keys, q, qn, torch.from_numpy(sl).cuda(), sl


@pytest.mark.parametrize("fp8", [False, True])
def test_same_bits_every_time_and_given_buffers(fp8):
    dev, keys, q, qn, sl, _ = _args(fp8)
    first, l0 = fx.sparse_latent_attention(q, slots=sl, scale=SCALE, **dev, return_lse=True)
    out, lse = torch.empty_like(first), torch.empty_like(l0)
    ws = fx.alloc_workspace(fx.sparse_latent_workspace_size(5, 24, 300))
    ws.fill_(0xFF)                               # what a workspace holds before a call does not matter
    for _ in range(5):
        got = fx.sparse_latent_attention(q, slots=sl, scale=SCALE, **dev, out=out, lse=lse, workspace=ws)
        assert got.data_ptr() == out.data_ptr()
        assert torch.equal(out, first) and torch.equal(lse, l0)
    with pytest.raises(fx.Fp8IdxError) as e:
        fx.sparse_latent_attention(q, slots=sl, scale=SCALE, **dev, workspace=ws[:1024])
    assert e.value.code == fx.EWORKSPACE
    with pytest.raises(ValueError):
        fx.sparse_latent_attention(q, slots=sl, scale=SCALE, **dev, out=out[:4])
    with pytest.raises(TypeError):
        fx.sparse_latent_attention(q.float(), slots=sl, scale=SCALE, **dev)
    with pytest.raises(TypeError):
        fx.sparse_latent_attention(q, slots=sl.long(), scale=SCALE, **dev)
    with pytest.raises(ValueError):
        fx.sparse_latent_attention(q, slots=sl.t().contiguous().t(), scale=SCALE, **dev)
    with pytest.raises(ValueError):
        fx.sparse_latent_attention(q[..., :512], slots=sl, scale=SCALE, **dev)


@pytest.mark.parametrize("fp8", [False, True])
def test_captured_and_replayed_with_a_shared_workspace(fp8):
    """Two graphs over one workspace, replayed in turn with new inputs, and an eager call between them."""
    dev, keys, q, qn, sl, _ = _args(fp8)
    ws = fx.alloc_workspace(max(fx.sparse_latent_workspace_size(5, 24, 300), fx.paged_latent_workspace_size(5, 1, 2, 24)))
    table = torch.arange(10, dtype=torch.int32).view(5, 2).cuda()
    lens = torch.tensor([128, 1, 0, 64, 100], dtype=torch.int32).cuda()
    a, b = torch.empty(5, 24, 512, dtype=BF).cuda(), torch.empty(5, 24, 512, dtype=BF).cuda()
    run_a = lambda: fx.sparse_latent_attention(q, slots=sl, scale=SCALE, **dev, out=a, workspace=ws)  # noqa: E731
    run_b = lambda: fx.paged_latent_attention(q, block_table=table, seq_lens=lens, R=1, scale=SCALE, **dev, out=b, workspace=ws)  # noqa: E731
    run_a(), run_b()
    torch.cuda.synchronize()
    ga, gb = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(ga):
        run_a()
    with torch.cuda.graph(gb):
        run_b()
    for k in range(3):
        q.copy_(torch.randn(q.shape, generator=torch.Generator().manual_seed(410 + k)).to(BF))
        a.zero_(), b.zero_()
        ga.replay(), gb.replay(), ga.replay()
        torch.cuda.synchronize()
        ra, rb = a.clone(), b.clone()
        a.zero_(), b.zero_()
        run_b(), run_a()
        assert torch.equal(a, ra) and torch.equal(b, rb)


@pytest.mark.parametrize("fp8", [False, True])
def test_streams(fp8):
    """Calls on other streams than the current one, at the same time, each with its own workspace."""
    cases = [_args(fp8, rows=r, H=h, topk=k, seed=420 + r) for r, h, k in ((5, 24, 300), (40, 64, 128), (1, 16, 600))]
    want = [fx.sparse_latent_attention(c[2], slots=c[4], scale=SCALE, **c[0]) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    outs = [torch.empty_like(w) for w in want]
    wss = [fx.alloc_workspace(fx.sparse_latent_workspace_size(c[2].shape[0], c[2].shape[1], c[4].shape[1])) for c in cases]
    for _ in range(10):
        for c, s, o, w in zip(cases, streams, outs, wss):
            fx.sparse_latent_attention(c[2], slots=c[4], scale=SCALE, **c[0], out=o, workspace=w, stream=s)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o, w)


@pytest.mark.parametrize("fp8", [False, True])
def test_wait_timeout_sets_status_and_recovers(fp8):
    """A first tile that is never announced: the wait on it runs out after 2 ms,
    the call reports it, and the next call is clean."""
    dev, keys, q, qn, sl, sln = _args(fp8)
    ws = fx.alloc_workspace(fx.sparse_latent_workspace_size(5, 24, 300))
    try:
        fx.set_wait_limit_ns(2_000_000)
        fx.debug_withhold_first_tile(True)
        fx.sparse_latent_attention(q, slots=sl, scale=SCALE, **dev, workspace=ws)
        st = fx.read_device_status(ws)
    finally:
        fx.debug_withhold_first_tile(False)
        fx.set_wait_limit_ns(2_000_000_000)
    assert st & fx.STATUS_WAIT_TIMEOUT, f"status {st:#x}"
    out, lse = fx.sparse_latent_attention(q, slots=sl, scale=SCALE, **dev, workspace=ws, return_lse=True)
    assert fx.read_device_status(ws) == 0
    for i in range(5):
        _check_row(_np(out)[i], _np(lse)[i], qn[i], keys[sln[i]], fp8, f"row {i}")


@pytest.mark.parametrize("fp8", [False, True])
def test_wait_timeout_with_groups_not_reached(fp8):
    """The same where a CTA had further requests to come: what the workspace
    held for them before is not followed."""
    B, R, H, L = 5, 8, 128, 6000
    table = torch.arange(94, dtype=torch.int32).repeat(B, 1).cuda()
    dev, keys = _pool(94, fp8, 460)
    q, qn = _q(B * R, H, 461)
    lens = torch.full((B,), L, dtype=torch.int32).cuda()
    ws = fx.alloc_workspace(fx.paged_latent_workspace_size(B, R, 94, H))
    run = lambda **kw: fx.paged_latent_attention(q, block_table=table, seq_lens=lens, R=R, scale=SCALE, **dev, workspace=ws, **kw)  # noqa: E731
    for fill in (0x7F, 0xFF, 0x01):
        ws.fill_(fill)
        torch.cuda.synchronize()
        try:
            fx.set_wait_limit_ns(2_000_000)
            fx.debug_withhold_first_tile(True)
            run()
            st = fx.read_device_status(ws)
        finally:
            fx.debug_withhold_first_tile(False)
            fx.set_wait_limit_ns(2_000_000_000)
        assert st & fx.STATUS_WAIT_TIMEOUT, f"status {st:#x}"
    out, lse = run(return_lse=True)
    assert fx.read_device_status(ws) == 0
    for i in (0, 39):
        _check_row(_np(out)[i], _np(lse)[i], qn[i], keys[:L - R + i % R + 1], fp8, f"row {i}")


def test_workspace_of_a_call_on_another_stream():
    """The call makes its own workspace; what the current stream allocates and
    writes meanwhile must not land in it."""
    dev, keys = _pool(40, True, 470)
    q, _ = _q(64, 64, 471)
    sl = torch.from_numpy(_slots(64, 2048, 2560, 472)).cuda()
    want = fx.sparse_latent_attention(q, slots=sl, scale=SCALE, **dev)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    n = fx.sparse_latent_workspace_size(64, 64, 2048)
    got = []
    for _ in range(20):
        got.append(fx.sparse_latent_attention(q, slots=sl, scale=SCALE, **dev, stream=s))
        torch.full((n,), 0x55, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    for g in got:
        assert torch.equal(g, want)


def test_strides_of_size_one_and_overlap():
    """A dimension of size 1 may have any stride; output rows that overlap are refused."""
    dev, keys = _pool(2, False, 480)
    base = torch.randn(3, 577, dtype=torch.float32).to(BF).cuda()
    q = base[:1, :576].unsqueeze(1)
    sl = torch.arange(100, dtype=torch.int32)[None].cuda()
    out, lse = fx.sparse_latent_attention(q, slots=sl, scale=SCALE, **dev, return_lse=True)
    _check_row(_np(out)[0], _np(lse)[0], _np(q)[0], keys[:100], False, "row 0")
    x, qx, tab, pos, slot = _store_case(4, 2, False, True, 481, 2)
    one = torch.zeros(4, 1, 64, dtype=BF).cuda().expand(4, 2, 64)
    with pytest.raises(fx.Fp8IdxError):
        fx.latent_store(x.cuda()[:, :512], x.cuda()[:, 512:], pos.cuda(), tab.cuda(), slot.cuda(), **dev,
                        q_pe=qx.cuda()[..., :64], q_out=one)


def test_no_backward():
    """No gradient is dropped in silence: inputs that require one are refused, unless gradients are off."""
    dev, _ = _pool(2, False, 490)
    q, _ = _q(2, 4, 491)
    sl = torch.arange(20, dtype=torch.int32).repeat(2, 1).cuda()
    want = fx.sparse_latent_attention(q, slots=sl, scale=SCALE, **dev)
    q.requires_grad_()
    with pytest.raises(ValueError, match="no backward"):
        fx.sparse_latent_attention(q, slots=sl, scale=SCALE, **dev)
    with pytest.raises(ValueError, match="no backward"):
        fx.paged_latent_attention(q, block_table=torch.zeros(2, 1, dtype=torch.int32).cuda(),
                                  seq_lens=torch.ones(2, dtype=torch.int32).cuda(), R=1, scale=SCALE, **dev)
    with torch.no_grad():
        assert torch.equal(fx.sparse_latent_attention(q, slots=sl, scale=SCALE, **dev), want)
    assert torch.equal(fx.sparse_latent_attention(q.detach(), slots=sl, scale=SCALE, **dev), want)


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("fp8", [False, True])
def test_a_decode_step(fp8):
    """As a serving step uses them: new tokens into the latent cache and into
    the indexer's key pool, the indexer's slots, the attention over them; and
    with as many slots as tokens, the attention over all cached tokens."""
    B, R, H, L = 3, 2, 16, 200
    g = torch.Generator().manual_seed(500)
    pages_per = 4
    table = torch.randperm(B * pages_per, generator=g).to(torch.int32).view(B, pages_per)
    pos = torch.arange(L).repeat(B)
    slot = torch.cat([table[b, torch.arange(L) // 64].long() * 64 + torch.arange(L) % 64 for b in range(B)])
    x = torch.randn(B * L, 576, generator=g).to(BF)
    xi = (2 * torch.randn(B * L, 128, generator=g)).to(BF)
    ang = torch.arange(L)[:, None].double() * 10000.0 ** (-torch.arange(0, 64, 2).double() / 64)
    tab = torch.cat([ang.cos(), ang.sin()], -1).float()
    P = B * pages_per
    pool = (dict(kv_pages=torch.zeros(P, 64, 512, dtype=torch.uint8).cuda(), s_pages=torch.zeros(P, 64).cuda(),
                 pe_pages=torch.zeros(P, 64, 64, dtype=BF).cuda()) if fp8 else dict(kv_pages=torch.zeros(P, 64, 576, dtype=BF).cuda()))
    fx.latent_store(x.cuda()[:, :512], x.cuda()[:, 512:], pos.cuda(), tab.cuda(), slot.cuda(), **pool)
    ik, isc = torch.zeros(P, 64, 128, dtype=torch.uint8).cuda(), torch.zeros(P, 64).cuda()
    fx.act_quant_store(xi.cuda(), slot.cuda(), ik, isc)
    iq = torch.randn(B * R, 32, 128, generator=g).clamp(-2, 2).to(torch.float8_e4m3fn).view(torch.uint8)
    w = torch.rand(B * R, 32, generator=g)
    lens = torch.full((B,), L, dtype=torch.int32)
    # the queries: the rows' absorbed part, and their rotary part rotated into place with the cache untouched
    q = torch.randn(B * R, H, 576, generator=g).to(BF).cuda()
    qpe = torch.randn(B * R, H, 64, generator=g).to(BF)
    rpos = torch.tensor([L - R + t for _ in range(B) for t in range(R)])
    none = torch.full((B * R,), -1)
    fx.latent_store(x.cuda()[:B * R, :512], x.cuda()[:B * R, 512:], rpos.cuda(), tab.cuda(), none.cuda(), **pool, q_pe=qpe.cuda(),
                    q_out=q[..., 512:])
    n = P * 64
    if fp8:
        keys = lo.keys_of(pool["kv_pages"].view(n, 512).cpu().numpy(), pool["s_pages"].view(n).cpu().numpy(),
                          _np(pool["pe_pages"]).reshape(n, 64))
    else:
        keys = _np(pool["kv_pages"]).reshape(n, 576)
    want_pe = lo.rotate(x.double().numpy()[:, 512:], tab.numpy(), pos.numpy(), True)
    assert (np.abs(keys[slot.numpy(), 512:] - want_pe) <= _rot_tol(x.double().numpy()[:, 512:], tab, None, want_pe)).all()
    for topk in (64, 256):
        slots = fx.paged_mqa_logits_topk(iq.cuda(), ik, isc, w.cuda(), table.cuda(), lens.cuda(), R=R, topk=topk, slots=True)
        out, lse = fx.sparse_latent_attention(q, slots=slots, scale=SCALE, **pool, return_lse=True)
        sl = slots.cpu().numpy()
        for i in range(B * R):
            sel = sl[i][sl[i] >= 0]
            assert len(sel) == min(topk, L - R + i % R + 1) == len(set(sel.tolist()))
            _check_row(_np(out)[i], _np(lse)[i], _np(q)[i], keys[sel], fp8, f"topk {topk} row {i}")
    full, fl = fx.paged_latent_attention(q, block_table=table.cuda(), seq_lens=lens.cuda(), R=R, scale=SCALE, **pool, return_lse=True)
    _check_paged(full, fl, [L] * B, R, _np(q), keys, table.numpy(), fp8)
    # all tokens selected: the same keys in another order, so within both calls' limits of each other
    for i in range(B * R):
        at = _logical(table.numpy(), i // R, L)[:L - R + i % R + 1]
        tol, ltol = lo.limits(_np(q)[i], keys[at], SCALE, fp8)
        assert (np.abs(_np(full)[i] - _np(out)[i]) <= 2 * tol).all() and (np.abs(_np(fl)[i] - _np(lse)[i]) <= 2 * ltol).all()


# ------------------------------------------------------------------ what one row holds stays out of the others

@pytest.mark.parametrize("H", [16, 40])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("head", [None, 3])
@pytest.mark.parametrize("fp8", [False, True])
def test_paged_non_finite_query_stays_in_its_column(fp8, head, value, H):
    """A value that is not finite in the query of a request's first row (all
    heads, or one): that row does not see the last keys, the others do."""
    lengths, R = [70, 130, 65, 3, 64, 2], 4
    dev, keys, table, q, qn = _paged_case(lengths, R, H, fp8, 600 + H)
    hit = np.zeros((len(lengths) * R, H), bool)
    hit[::R, slice(None) if head is None else head] = True
    q[torch.from_numpy(hit).cuda(), 5] = value
    out, lse = fx.paged_latent_attention(q, block_table=torch.from_numpy(table).cuda(),
                                         seq_lens=torch.tensor(lengths, dtype=torch.int32).cuda(), R=R, scale=SCALE, **dev,
                                         return_lse=True)
    out, lse = _np(out), _np(lse)
    for b, l in enumerate(lengths):
        at = _logical(table, b, l)
        for t in range(R):
            i = b * R + t
            seen = keys[at[:max(0, l - R + t + 1)]]
            ok = ~hit[i] if len(seen) else np.ones(H, bool)     # a row without keys gives 0 and -inf whatever its query holds
            if ok.any():
                _check_row(out[i][ok], lse[i][ok], qn[i][ok], seen, fp8, f"request {b} (length {l}) row {t}")
            if np.isnan(value) and not ok.all():
                assert np.isnan(out[i][~ok]).all() and np.isnan(lse[i][~ok]).all()


def test_paged_infinite_key_that_some_rows_see():
    """A key with an infinite value that only a request's later rows see: it
    stays out of the earlier ones, and shows in those that see it, where its
    score is -inf (weight 0, and 0 times infinity) too."""
    lengths, R, H = [70, 130, 64, 3], 4, 16
    dev, keys, table, q, qn = _paged_case(lengths, R, H, False, 650)
    for b, l in enumerate(lengths):
        dev["kv_pages"].view(-1, 576)[int(_logical(table, b, l)[-2]), 7] = -float("inf")   # rows R - 2 and R - 1 see it
    q[..., 7] = 1.0                                                                        # a score of -inf
    qn = _np(q)
    out, lse = fx.paged_latent_attention(q, block_table=torch.from_numpy(table).cuda(),
                                         seq_lens=torch.tensor(lengths, dtype=torch.int32).cuda(), R=R, scale=SCALE, **dev,
                                         return_lse=True)
    out, lse = _np(out), _np(lse)
    for b, l in enumerate(lengths):
        at = _logical(table, b, l)
        for t in range(R):
            i = b * R + t
            if t < R - 2:
                _check_row(out[i], lse[i], qn[i], keys[at[:max(0, l - R + t + 1)]], False, f"request {b} row {t}")
            else:
                assert np.isnan(out[i][:, 7]).all(), f"request {b} row {t}"


def test_workspace_of_the_largest_sizes_serves_all_smaller_ones():
    """A server reserves one workspace for its largest batch: no smaller one may ask for more."""
    rows = [*range(1, 301), 512, 1000, 1024, 4096]
    heads = (1, 16, 32, 33, 64, 65, 128)
    topks = (0, 1, 64, 65, 128, 640, 2048)
    sizes = np.array([[[fx.sparse_latent_workspace_size(r, h, k) for k in topks] for h in heads] for r in rows])
    assert (sizes > 0).all()
    for axis in range(3):
        assert (np.diff(sizes, axis=axis) >= 0).all(), ("rows", "heads", "topk")[axis]
    sizes = np.array([[[[fx.paged_latent_workspace_size(b, r, m, h) for h in heads] for m in (1, 2, 3, 5, 33, 2048)] for r in range(1, 9)]
                      for b in (1, 2, 7, 32, 33, 100, 148, 149, 1000)])
    assert (sizes > 0).all()
    for axis in range(4):
        assert (np.diff(sizes, axis=axis) >= 0).all(), ("requests", "rows a request", "blocks", "heads")[axis]
    dev, _ = _pool(40, True, 660)
    ws = fx.alloc_workspace(fx.sparse_latent_workspace_size(296, 64, 2048))
    for n in (296, 160, 115, 116, 1):
        q, _ = _q(n, 64, 661)
        sl = torch.from_numpy(_slots(n, 2048, 2560, 662)).cuda()
        want = fx.sparse_latent_attention(q, slots=sl, scale=SCALE, **dev)
        assert torch.equal(fx.sparse_latent_attention(q, slots=sl, scale=SCALE, **dev, workspace=ws), want)
        assert fx.read_device_status(ws) == 0


def test_no_gradient_is_lost_in_silence():
    """Every floating-point tensor of the calls, given outputs among them, and
    tangents of forward mode."""
    import torch.autograd.forward_ad as fwad
    dev, _ = _pool(2, True, 670)
    q, _ = _q(2, 4, 671)
    sl = torch.arange(20, dtype=torch.int32).repeat(2, 1).cuda()
    table, lens = torch.zeros(2, 1, dtype=torch.int32).cuda(), torch.ones(2, dtype=torch.int32).cuda()
    x, qx, tab, pos, slot = _store_case(4, 2, True, True, 672, 2)
    x, qx, tab, pos, slot = x.cuda(), qx.cuda(), tab.cuda(), pos.cuda(), slot.cuda()
    bufs = dict(out=torch.zeros(2, 4, 512, dtype=BF).cuda(), lse=torch.zeros(2, 4).cuda())

    def sparse(**kw):
        a = dict(q=q, slots=sl, scale=SCALE, **dev, **bufs)
        fx.sparse_latent_attention(**{**a, **kw})

    def paged(**kw):
        a = dict(q=q, block_table=table, seq_lens=lens, R=1, scale=SCALE, **dev, **bufs)
        fx.paged_latent_attention(**{**a, **kw})

    def store(**kw):
        a = dict(c=x[:, :512], k_pe=x[:, 512:], positions=pos, cos_sin=tab, slot_mapping=slot, **dev, q_pe=qx[..., :64],
                 q_out=torch.zeros(4, 2, 64, dtype=BF).cuda())
        fx.latent_store(**{**a, **kw})

    given = {sparse: dict(q=q, s_pages=dev["s_pages"], pe_pages=dev["pe_pages"], **bufs),
             paged: dict(q=q, s_pages=dev["s_pages"], pe_pages=dev["pe_pages"], **bufs),
             store: dict(c=x[:, :512], k_pe=x[:, 512:], cos_sin=tab, s_pages=dev["s_pages"], pe_pages=dev["pe_pages"], q_pe=qx[..., :64],
                         q_out=torch.zeros(4, 2, 64, dtype=BF).cuda())}
    for call, tensors in given.items():
        call()
        for name, t in tensors.items():
            leaf = t.detach().clone().requires_grad_()
            with pytest.raises(ValueError, match=name + ".*no backward"):
                call(**{name: leaf})
            with torch.no_grad():
                call(**{name: leaf})
            with fwad.dual_level():
                dual = fwad.make_dual(t.detach().clone(), torch.ones_like(t))
                with pytest.raises(ValueError, match=name + ".*tangent"):
                    call(**{name: dual})
    torch.cuda.synchronize()
