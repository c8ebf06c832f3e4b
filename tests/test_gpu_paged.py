"""The paged K/V cache's operators on the GPU, against their definitions in 64
bits (tests/_paged.py: the tolerances are derived there)."""
import math

import numpy as np
import pytest
import torch

from tests import _paged as ref

pytestmark = pytest.mark.gpu
D = 128
DEV = "cuda"
SC = 1 / math.sqrt(D)


@pytest.fixture(scope="module")
def kvs():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    import kv_index_scan_b200
    return kv_index_scan_b200


def _bits(t):
    return t.contiguous().view(torch.int16) if t.dtype == torch.bfloat16 else t


def _status():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


# ----------------------------------------------------------------------------- append

@pytest.mark.parametrize("layout", ["head", "token", "both"])
@pytest.mark.parametrize("G,page", [(1, 16), (3, 32), (8, 64), (5, 1024)])
def test_append_writes_its_rows_and_no_others(kvs, layout, G, page):
    lens, new = [5, 40, 0, 333, 17], [5, 3, 0, 300, 1]
    k, v, table, n = ref.make(lens, G, page, seed=page, layout=layout)
    cache = kvs.PagedKV(k, v, table, n)
    cu = torch.tensor([0] + list(np.cumsum(new)), dtype=torch.int32, device=DEV)
    T = int(cu[-1]) + 4  # padded rows behind the last request
    rows = torch.randn(T, 2 * G * D + 8, device=DEV).to(torch.bfloat16)  # rows inside a wider projection
    Kn, Vn = rows[:, :G * D].view(T, G, D), rows[:, G * D:2 * G * D].view(T, G, D)
    mass = torch.full((5, G, cache.cap), 7.0, device=DEV)
    pos = torch.full((5, G, cache.cap), -9, dtype=torch.int32, device=DEV)
    seen = n + 1000
    wk, wv, wm, wp = k.clone(), v.clone(), mass.clone(), pos.clone()
    st = _status()
    kvs.paged_append(cache, Kn, Vn, cu, mass=mass, pos=pos, seen=seen, dev_status=st)
    for r, (m, c) in enumerate(zip(lens, new)):
        for t in range(c):
            i = m - c + t
            pg = int(table[r, i // page])
            wk[pg, :, i % page], wv[pg, :, i % page] = Kn[cu[r] + t], Vn[cu[r] + t]
            wm[r, :, i], wp[r, :, i] = 0.0, 1000 + i
    assert torch.equal(_bits(k), _bits(wk)) and torch.equal(_bits(v), _bits(wv))
    assert torch.equal(mass, wm) and torch.equal(pos, wp) and int(st) == 0


def test_append_one_token_each(kvs):
    lens = [1, 16, 17, 100]
    k, v, table, n = ref.make(lens, 4, 16, seed=2)
    cache = kvs.PagedKV(k, v, table, n)
    Kn, Vn = torch.randn(2, 4, 4, D, device=DEV).to(torch.bfloat16)
    pos = torch.full((4, 4, cache.cap), -9, dtype=torch.int32, device=DEV)
    kvs.paged_append(cache, Kn, Vn, pos=pos)
    for r, m in enumerate(lens):
        pg = int(table[r, (m - 1) // 16])
        assert torch.equal(k[pg, :, (m - 1) % 16], Kn[r]) and torch.equal(v[pg, :, (m - 1) % 16], Vn[r])
        assert bool((pos[r, :, m - 1] == m - 1).all()) and bool((pos[r, :, m:] == -9).all())


def test_append_refuses_positions_and_pages_that_are_none(kvs):
    """A full cache, more new tokens than the length counts, and a bad page id: nothing is written there and
    the status word says so."""
    k, v, table, n = ref.make([48, 2, 20], 2, 16, seed=3, slack=0)
    cache = kvs.PagedKV(k, v, table, n)
    cap = cache.cap
    n.copy_(torch.tensor([cap + 1, 1, 20]))
    table[2, 1] = cache.num_pages
    wk, wv = k.clone(), v.clone()
    cu = torch.tensor([0, 1, 3, 4], dtype=torch.int32, device=DEV)
    Kn, Vn = torch.ones(2, 4, 2, D, device=DEV).to(torch.bfloat16)
    st = _status()
    kvs.paged_append(cache, Kn, Vn, cu, dev_status=st)
    wk[int(table[1, 0]), :, 0], wv[int(table[1, 0]), :, 0] = 1, 1  # the second of the two tokens fits
    assert int(st) == kvs.KVS_EBOUNDS
    assert torch.equal(_bits(k), _bits(wk)) and torch.equal(_bits(v), _bits(wv))


@pytest.mark.parametrize("cu,written", [
    ([0, 2, 9], {0: (0, 10), 1: (0, 11), 2: (1, 3), 3: (1, 4), 4: (1, 5)}),  # more rows than there are
    ([2, 4, 5], {2: (0, 10), 3: (0, 11), 4: (1, 9)}),                        # rows in front of the first request
    ([0, 5, 3], {0: (0, 7), 1: (0, 8), 2: (0, 9)}),                          # offsets that fall: none from cu[R] on
    ([3, 1, 5], {1: (1, 6), 2: (1, 7), 3: (1, 8), 4: (1, 9)})])
def test_append_offsets_that_do_not_fit_the_rows(kvs, cu, written):
    """Rows go where the offsets say or nowhere, never over older tokens, and the status word says so."""
    k, v, table, n = ref.make([12, 10], 2, 16, seed=3, poison=False)
    cache = kvs.PagedKV(k, v, table, n)
    wk, wv = k.clone(), v.clone()
    Kn, Vn = torch.randn(2, 5, 2, D, device=DEV).to(torch.bfloat16)
    for t, (r, i) in written.items():
        wk[int(table[r, 0]), :, i], wv[int(table[r, 0]), :, i] = Kn[t], Vn[t]
    st = _status()
    kvs.paged_append(cache, Kn, Vn, torch.tensor(cu, dtype=torch.int32, device=DEV), dev_status=st)
    assert torch.equal(_bits(k), _bits(wk)) and torch.equal(_bits(v), _bits(wv))
    assert int(st) == (kvs.KVS_OK if cu == [0, 5, 3] else kvs.KVS_EBOUNDS)


def test_append_many_requests(kvs):
    """More requests than a warp's search step, with runs of empty ones."""
    rng = np.random.default_rng(5)
    new = [int(x) for x in rng.integers(0, 4, 1100)]
    new[300:400] = [0] * 100
    new[-1] = 2
    k, v, table, n = ref.make(new, 1, 16, seed=5, slack=0, spare=0)
    cache = kvs.PagedKV(k, v, table, n)
    cu = torch.tensor([0] + list(np.cumsum(new)), dtype=torch.int32, device=DEV)
    T = int(cu[-1])
    Kn, Vn = torch.randn(2, T, 1, D, device=DEV).to(torch.bfloat16)
    kvs.paged_append(cache, Kn, Vn, cu)
    row = torch.repeat_interleave(torch.arange(len(new)), torch.tensor(new)).to(DEV)
    at = torch.arange(T, device=DEV) - cu[row.long()]
    pg = table[row, at // 16].long()
    assert torch.equal(k[pg, 0, at % 16], Kn[:, 0]) and torch.equal(v[pg, 0, at % 16], Vn[:, 0])


# ----------------------------------------------------------------------------- decode

LENS = [0, 1, 15, 16, 17, 63, 64, 65, 127, 129, 300, 1031]


@pytest.mark.parametrize("H", [1, 2, 3, 4, 5, 6, 7, 8])
@pytest.mark.parametrize("qdt", [torch.bfloat16, torch.float32])
def test_decode_head_counts_and_lengths(kvs, H, qdt):
    k, v, table, n = ref.make(LENS, 2, 16, seed=H)
    cache = kvs.PagedKV(k, v, table, n)
    q = torch.randn(len(LENS), 2, H, D, device=DEV).to(qdt)
    st = _status()
    out, lse = kvs.paged_decode_attn(q, cache, dev_status=st)
    ref.check_decode(out, lse, q, k, v, table, LENS, 0, 0, SC)
    assert int(st) == 0


@pytest.mark.parametrize("layout", ["head", "token", "both"])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256, 1024])
@pytest.mark.parametrize("window,sinks", [(0, 0), (0, 3), (1, 0), (1, 1), (64, 4), (100, 70), (513, 16), (5000, 4)])
def test_decode_pages_windows_and_weights(kvs, layout, page, window, sinks):
    """Rows behind the last token and pages that the window has passed hold NaN; the weights add up beside."""
    lens = [1, 70, 517, 1030, 2049]
    G, H = 3, 4
    k, v, table, n = ref.make(lens, G, page, seed=page + window, layout=layout)
    for r, m in enumerate(lens):
        vis = set((ref.visible(m - 1, window, sinks)).tolist())
        for j in range(m):
            if j not in vis:
                k[int(table[r, j // page]), :, j % page] = float("nan")
                v[int(table[r, j // page]), :, j % page] = float("inf")
        for p in range(-(-m // page)):
            if not any(j in vis for j in range(p * page, min(m, (p + 1) * page))):
                table[r, p] = -1  # released
    cache = kvs.PagedKV(k, v, table, n)
    q = torch.randn(len(lens), G, H, D, device=DEV).to(torch.bfloat16)
    mass = torch.rand(len(lens), G, cache.cap, device=DEV)
    before = mass.clone()
    kt, vt, tt = k.nan_to_num(0, 0, 0), v.nan_to_num(0, 0, 0), table.clamp(min=0)
    st = _status()
    out, lse = kvs.paged_decode_attn(q, cache, window, sinks, mass=mass, dev_status=st)
    ref.check_decode(out, lse, q, kt, vt, tt, lens, window, sinks, SC, before, mass)
    # out of place, entries that are not visible stay
    mo = torch.full_like(before, float("nan"))
    out2, lse2 = kvs.paged_decode_attn(q, cache, window, sinks, mass=before, mass_out=mo, dev_status=st)
    assert torch.equal(out, out2) and torch.equal(lse, lse2) and int(st) == 0
    for r, m in enumerate(lens):
        vis = torch.zeros(cache.cap, dtype=torch.bool, device=DEV)
        vis[torch.from_numpy(ref.visible(m - 1, window, sinks)).to(DEV)] = True
        assert torch.equal(mo[r][:, vis], mass[r][:, vis]) and bool(torch.isnan(mo[r][:, ~vis]).all())


@pytest.mark.parametrize("R,G,n_", [(1, 1, 40001), (1, 8, 9000), (3, 2, 30011), (257, 3, 90), (40, 8, 700)])
def test_decode_splits(kvs, R, G, n_):
    """One long row over every block, and more rows than blocks."""
    rng = np.random.default_rng(R)
    lens = [n_] + [int(x) for x in rng.integers(0, n_ + 1, R - 1)]
    k, v, table, n = ref.make(lens, G, 64, seed=R, poison=False)
    cache = kvs.PagedKV(k, v, table, n)
    q = torch.randn(R, G, 4, D, device=DEV)
    mass = torch.zeros(R, G, cache.cap, device=DEV)
    out, lse = kvs.paged_decode_attn(q, cache, mass=mass)
    ref.check_decode(out, lse, q, k, v, table, lens, 0, 0, SC, torch.zeros_like(mass), mass)


@pytest.mark.parametrize("H", [1, 2, 3, 5, 6, 7, 8])
@pytest.mark.parametrize("weights", [False, True])
@pytest.mark.parametrize("qdt", [torch.bfloat16, torch.float32])
def test_decode_splits_head_counts(kvs, H, weights, qdt):
    """Rows cut into many parts, and into few, with every head count."""
    lens = [12000, 30011, 2570, 64]
    k, v, table, n = ref.make(lens, 2, 64, seed=H, poison=False)
    cache = kvs.PagedKV(k, v, table, n)
    q = torch.randn(4, 2, H, D, device=DEV).to(qdt)
    mass = torch.zeros(4, 2, cache.cap, device=DEV) if weights else None
    out, lse = kvs.paged_decode_attn(q, cache, mass=mass)
    ref.check_decode(out, lse, q, k, v, table, lens, 0, 0, SC, torch.zeros_like(mass) if weights else None, mass)


@pytest.mark.parametrize("H", [1, 3, 4, 8])
@pytest.mark.parametrize("weights", [False, True])
def test_decode_one_long_row_among_many(kvs, H, weights):
    """More rows than SMs, one of them cut into many parts."""
    lens = [0, 50, 25003] + [17 * i % 90 for i in range(200)]
    k, v, table, n = ref.make(lens, 1, 64, seed=H, poison=False)
    cache = kvs.PagedKV(k, v, table, n)
    q = torch.randn(len(lens), 1, H, D, device=DEV)
    mass = torch.zeros(len(lens), 1, cache.cap, device=DEV) if weights else None
    out, lse = kvs.paged_decode_attn(q, cache, mass=mass)
    ref.check_decode(out, lse, q, k, v, table, lens, 0, 0, SC, torch.zeros_like(mass) if weights else None, mass)


@pytest.mark.parametrize("R,G,H,window,sinks", [(700, 2, 4, 0, 0), (300, 1, 8, 0, 0), (1100, 1, 3, 40, 9), (40, 8, 2, 0, 0)])
def test_decode_many_short_rows(kvs, R, G, H, window, sinks):
    """More rows than blocks: empty ones, ones within a block's run, ones cut once."""
    rng = np.random.default_rng(R)
    lens = [int(x) for x in rng.integers(1, 400, R)]
    for i in range(0, R, 3):
        lens[i] = 0
    k, v, table, n = ref.make(lens, G, 16, seed=R, poison=False)
    cache = kvs.PagedKV(k, v, table, n)
    q = torch.randn(R, G, H, D, device=DEV)
    out = torch.full((R, G, H, D), float("nan"), device=DEV)
    lse = torch.full((R, G, H), float("nan"), device=DEV)
    out, lse = kvs.paged_decode_attn(q, cache, window, sinks, out=out, lse=lse)
    ref.check_decode(out, lse, q, k, v, table, lens, window, sinks, SC)


@pytest.mark.parametrize("R,G,H,window,sinks", [(400, 2, 4, 0, 0), (700, 1, 7, 40, 9), (90, 8, 2, 0, 0), (700, 1, 8, 300, 0)])
def test_decode_many_rows_with_weights(kvs, R, G, H, window, sinks):
    """Rows joined and weighed by kernels of their own: empty, short and long ones (over more than one piece)."""
    rng = np.random.default_rng(R + H)
    lens = [int(x) for x in rng.integers(1, 200, R)]
    for i in range(0, R, 4):
        lens[i] = 0
    lens[1], lens[R // 2] = 3001, 1024
    k, v, table, n = ref.make(lens, G, 16, seed=R, poison=False)
    cache = kvs.PagedKV(k, v, table, n)
    q = torch.randn(R, G, H, D, device=DEV)
    before = torch.rand(R, G, cache.cap, device=DEV)
    mass = before.clone()
    out, lse = kvs.paged_decode_attn(q, cache, window, sinks, mass=mass)
    ref.check_decode(out, lse, q, k, v, table, lens, window, sinks, SC, before, mass)
    for r in range(R):
        hidden = torch.ones(cache.cap, dtype=torch.bool, device=DEV)
        hidden[torch.from_numpy(ref.visible(lens[r] - 1, window, sinks)).to(DEV)] = False
        assert torch.equal(mass[r][:, hidden], before[r][:, hidden])


@pytest.mark.parametrize("R", [1, 200, 600])
def test_decode_nothing_seen(kvs, R):
    k, v, table, n = ref.make([0] * R, 2, 16, seed=R, poison=False)
    q = torch.randn(R, 2, 4, D, device=DEV)
    out, lse = kvs.paged_decode_attn(q, kvs.PagedKV(k, v, table, n), out=torch.full((R, 2, 4, D), 7.0, device=DEV))
    assert bool((out == 0).all()) and bool(torch.isneginf(lse).all())


@pytest.mark.parametrize("qdt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("window", [0, 300])
def test_decode_values_that_are_not_finite_stay_in_their_channels(kvs, qdt, window):
    """NaN and infinities in single values of V rows that are seen: those channels are not finite, all others are
    bit for bit what they are without; in rows that are not seen they have no effect. A K row that is not finite
    takes all channels of its request and head."""
    lens = [700, 65, 9000]
    k, v, table, n = ref.make(lens, 2, 16, seed=71, poison=False)
    cache = kvs.PagedKV(k, v, table, n)
    q = torch.randn(3, 2, 5, D, device=DEV).to(qdt)
    want, wl = kvs.paged_decode_attn(q, cache, window)
    bad = torch.zeros(3, 2, D, dtype=torch.bool, device=DEV)
    for i, (r, g, j, d) in enumerate([(0, 0, 0, 3), (0, 0, 650, 4), (0, 1, 399, 70), (0, 1, 400, 71), (1, 0, 64, 127),
                                      (2, 1, 8999, 0), (2, 1, 8700, 1), (2, 1, 8699, 2), (2, 0, 4000, 64)]):
        v[int(table[r, j // 16]), g, j % 16, d] = (float("nan"), float("inf"), -float("inf"))[i % 3]
        bad[r, g, d] |= not window or j >= lens[r] - window
    out, lse = kvs.paged_decode_attn(q, cache, window)
    assert torch.equal(~torch.isfinite(out), bad.unsqueeze(2).expand_as(out)) and torch.equal(lse, wl)
    ok = ~bad.unsqueeze(2).expand_as(out)
    assert torch.equal(out[ok], want[ok])
    k[int(table[1, 60 // 16]), 1, 60 % 16, 9] = float("nan")
    out2, _ = kvs.paged_decode_attn(q, cache, window)
    assert bool(torch.isnan(out2[1, 1]).all())
    out2[1, 1] = out[1, 1]
    assert torch.equal(torch.isfinite(out2), torch.isfinite(out)) and torch.equal(out2[ok], out[ok])


def test_decode_extreme_logits(kvs):
    """Logits from -3e4 to 3e4 and equal ones: the running maximum carries every one."""
    lens = [700, 700]
    k, v, table, n = ref.make(lens, 1, 16, seed=8)
    kt = k.clone()
    for j in range(700):
        pg = int(table[0, j // 16])
        k[pg, 0, j % 16] = 0.0
        k[pg, 0, j % 16, 0] = float((j * 37) % 700 - 350)
        k[int(table[1, j // 16]), 0, j % 16] = 1.0
    cache = kvs.PagedKV(k, v, table, n)
    q = torch.zeros(2, 1, 2, D, device=DEV)
    q[0, 0, 0, 0], q[0, 0, 1, 0], q[1] = 1000.0, -1000.0, 0.5
    out, lse = kvs.paged_decode_attn(q, cache)
    ref.check_decode(out, lse, q, k, v, table, lens, 0, 0, SC)
    assert kt.shape == k.shape


def test_decode_bad_pages_and_lengths(kvs):
    """A page id that is none in a visible place, and lengths out of range: the page's tokens count as absent,
    the length is clamped, and the status word says so."""
    lens = [40, 64, 10]
    k, v, table, n = ref.make(lens, 2, 16, seed=4, slack=0, poison=False)
    cache = kvs.PagedKV(k, v, table, n)
    good = table.clone()
    table[0, 1] = cache.num_pages + 5
    n.copy_(torch.tensor([40, 1 << 20, -3]))
    q = torch.randn(3, 2, 4, D, device=DEV)
    st = _status()
    mass = torch.zeros(3, 2, cache.cap, device=DEV)
    out, lse = kvs.paged_decode_attn(q, cache, mass=mass, dev_status=st)
    assert int(st) == kvs.KVS_EBOUNDS
    K, V = ref.tokens(k, good, 0, 40), ref.tokens(v, good, 0, 40)
    some = [j for j in range(40) if j // 16 != 1]
    for g in range(2):
        o, ls, w, e, va = ref.attend(q[0, g].double(), K[some][:, g], V[some][:, g], SC)
        assert float((out[0, g] - o).abs().max()) < 1e-4 and float((lse[0, g] - ls).abs().max()) < 1e-4
    assert bool((mass[0, :, 16:32] == 0).all())
    ref.check_decode(out[1:2], lse[1:2], q[1:2], k, v, good[1:2], [64], 0, 0, SC)
    assert bool((out[2] == 0).all()) and bool(torch.isneginf(lse[2]).all())


def test_decode_offsets_past_32_bits(kvs):
    """A pool of more than 2^32 bytes and 2^31 elements, its last pages in use."""
    P, G, page = 270_000, 8, 16  # 4.4e9 elements a pool
    k = torch.empty(P, G, page, D, dtype=torch.bfloat16, device=DEV)
    v = torch.empty_like(k)
    lens = [100]
    table = torch.tensor([[P - 1, 3, P - 2, P // 2, P - 7, 0, P - 3]], dtype=torch.int32, device=DEV)
    for p in table[0].tolist():
        k[p], v[p] = torch.randn(2, G, page, D, device=DEV).to(torch.bfloat16)
    n = torch.tensor(lens, dtype=torch.int32, device=DEV)
    cache = kvs.PagedKV(k, v, table, n)
    q = torch.randn(1, G, 4, D, device=DEV).to(torch.bfloat16)
    out, lse = kvs.paged_decode_attn(q, cache)
    ref.check_decode(out, lse, q, k, v, table, lens, 0, 0, SC)
    qp = torch.randn(100, G * 4, D, device=DEV).to(torch.bfloat16)
    cu = torch.tensor([0, 100], dtype=torch.int32, device=DEV)
    po, pl = kvs.paged_prompt_attn(qp, cu, cache)
    ref.check_prompt(po, pl, qp, [0, 100], k, v, table, lens, 0, 0, SC, G)
    Kn, Vn = torch.randn(2, 1, G, D, device=DEV).to(torch.bfloat16)
    kvs.paged_append(cache, Kn, Vn)
    assert torch.equal(k[P - 3, :, 3], Kn[0]) and torch.equal(v[P - 3, :, 3], Vn[0])
    want = ref.tokens(k, table, 0, 100)
    src = kvs.paged_evict(cache, torch.rand(1, G, cache.cap, device=DEV), 20)
    got = ref.tokens(k, table, 0, 20)
    for g in range(G):
        assert torch.equal(got[:, g], want[src[0, g].long(), g])


def test_decode_caller_buffers_streams_and_graph(kvs):
    """Caller's outputs and workspace; two calls at once on two streams; a captured call replayed after the
    lengths, the table and the queries changed in place."""
    lens = [500, 90]
    k, v, table, n = ref.make(lens, 2, 16, seed=6, poison=False, slack=4)
    cache = kvs.PagedKV(k, v, table, n)
    qs = [torch.randn(2, 2, 4, D, device=DEV) for _ in range(2)]
    want = [kvs.paged_decode_attn(q, cache) for q in qs]
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = []
    for _ in range(20):
        got.append([kvs.paged_decode_attn(q, cache, stream=s) for q, s in zip(qs, side)])
    torch.cuda.synchronize()
    for pair in got:
        for (o, l), (wo, wl) in zip(pair, want):
            assert torch.equal(o, wo) and torch.equal(l, wl)
    q, out, lse = qs[0].clone(), torch.empty(2, 2, 4, D, device=DEV), torch.empty(2, 2, 4, device=DEV)
    ws = kvs.paged_decode_workspace(cache, 4)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kvs.paged_decode_attn(q, cache, window=200, sinks=2, out=out, lse=lse, ws=ws)
    for m in ([500, 90], [333, 1], [0, 77]):
        n.copy_(torch.tensor(m))
        q.normal_()
        graph.replay()
        ref.check_decode(out, lse, q, k, v, table, m, 200, 2, SC)


@pytest.mark.parametrize("warp", [0, 1, 2, 3, 4])
@pytest.mark.parametrize("lens", [[20000, 7, 9000], [100] * 300])
def test_decode_bounded_waits_run_out_and_the_call_ends(kvs, lens, warp):
    """One warp of every block stops at its second unit as though its wait had run out, while the others have
    seen the same phase come: they end too, the status word says so, and the next call is right. Rows longer
    than a block's run, and rows that end in the middle of it, where the four warps meet."""
    import time
    k, v, table, n = ref.make(lens, 2, 64, seed=51, poison=False)
    cache = kvs.PagedKV(k, v, table, n)
    q = torch.randn(len(lens), 2, 4, D, device=DEV).to(torch.bfloat16)
    st = _status()
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    kvs.selftest_paged_decode_timeout(q, cache, warp, 2_000_000, st)
    torch.cuda.synchronize()
    assert int(st) == kvs.KVS_ETIMEOUT and time.perf_counter() - t0 < 5.0
    st = _status()
    out, lse = kvs.paged_decode_attn(q, cache, dev_status=st)
    ref.check_decode(out, lse, q, k, v, table, lens, 0, 0, SC)
    assert int(st) == 0


def test_binding_refusals(kvs):
    k, v, table, n = ref.make([20], 2, 16, seed=1)
    cache = kvs.PagedKV(k, v, table, n)
    q = torch.randn(1, 2, 4, D, device=DEV)
    cu = torch.tensor([0, 1], dtype=torch.int32, device=DEV)
    bad = [lambda: kvs.paged_decode_attn(q[:, :1], cache), lambda: kvs.paged_decode_attn(q.half(), cache),
           lambda: kvs.paged_decode_attn(q, cache, window=-1), lambda: kvs.paged_decode_attn(q, cache, window=2 ** 32),
           lambda: kvs.paged_decode_attn(q, cache, out=torch.empty(1, 2, 4, D)),
           lambda: kvs.paged_decode_attn(q, cache, mass=torch.zeros(1, 2, cache.cap + 1, device=DEV)),
           lambda: kvs.paged_decode_attn(q, cache, ws=torch.empty(16, device=DEV)),
           lambda: kvs.paged_prompt_attn(q.view(1, 8, D), cu, cache),
           lambda: kvs.paged_prompt_attn(q.view(1, 8, D).bfloat16(), cu.long(), cache),
           lambda: kvs.paged_prompt_attn(q.view(1, 8, D).bfloat16()[:, :7], cu, cache),
           lambda: kvs.paged_append(cache, q[:, :, 0], q[:, :, 1]),
           lambda: kvs.paged_evict(cache, torch.zeros(1, 2, cache.cap, device=DEV), 0),
           lambda: kvs.paged_evict(cache, torch.zeros(1, 2, cache.cap, device=DEV), 8, pos_out=torch.zeros(1)),
           lambda: kvs.PagedKV(k, v[:, :, ::2], table, n), lambda: kvs.PagedKV(k, v, table.long(), n),
           lambda: kvs.PagedKV(k, v, table, n[:0])]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was accepted")
    for call in (lambda: kvs.paged_decode_attn(torch.randn(1, 2, 9, D, device=DEV), cache),
                 lambda: kvs.paged_evict(cache, torch.zeros(1, 2, cache.cap, device=DEV), 8, sinks=5, recent=4),
                 lambda: kvs.paged_append(cache, k[:2, :, 0].contiguous(), k[:2, :, 0].contiguous())):
        with pytest.raises(kvs.KvsError):
            call()


def test_status_words_elsewhere_are_refused(kvs):
    """A status word in ordinary host memory, of another type or empty, in every call (none is launched)."""
    k, v, table, n = ref.make([20], 2, 16, seed=1, poison=False)
    cache = kvs.PagedKV(k, v, table, n)
    q, cu = torch.randn(1, 2, 4, D, device=DEV), torch.tensor([0, 1], dtype=torch.int32, device=DEV)
    qp, mass = q.view(1, 8, D).bfloat16(), torch.zeros(1, 2, cache.cap, device=DEV)
    for st in (torch.zeros(1, dtype=torch.int32), torch.zeros(1, dtype=torch.int64, device=DEV),
               torch.zeros(0, dtype=torch.int32, device=DEV)):
        for call in (lambda: kvs.paged_append(cache, qp[:, :2], qp[:, 2:4], dev_status=st),
                     lambda: kvs.paged_decode_attn(q, cache, dev_status=st),
                     lambda: kvs.paged_prompt_attn(qp, cu, cache, dev_status=st),
                     lambda: kvs.paged_evict(cache, mass, 8, dev_status=st)):
            with pytest.raises(ValueError, match="dev_status"):
                call()
    assert n.tolist() == [20]
    pinned = torch.zeros(1, dtype=torch.int32).pin_memory()
    kvs.paged_decode_attn(q, cache, dev_status=pinned)
    torch.cuda.synchronize()
    assert int(pinned) == 0


def test_a_cache_keeps_its_tensors(kvs):
    """n and table change in place; another tensor in their place, which no call would read, is refused."""
    k, v, table, n = ref.make([20, 33], 2, 16, seed=1, poison=False)
    cache = kvs.PagedKV(k, v, table, n)
    for name, t in (("n", n + 1), ("table", table.clone()), ("k_pages", k.clone()), ("v_pages", v.clone())):
        with pytest.raises(ValueError, match=name):
            setattr(cache, name, t)
    assert cache.n is n and cache.table is table and cache.k_pages is k and cache.v_pages is v
    cache.n -= 3
    q = torch.randn(2, 2, 4, D, device=DEV)
    out, lse = kvs.paged_decode_attn(q, cache)
    ref.check_decode(out, lse, q, k, v, table, [17, 30], 0, 0, SC)
    cache.n.copy_(torch.tensor([5, 6]))
    out, lse = kvs.paged_decode_attn(q, cache)
    ref.check_decode(out, lse, q, k, v, table, [5, 6], 0, 0, SC)


def test_no_heads_and_no_pages_are_refused(kvs):
    """No query heads in any call, and pools of no pages, heads or tokens."""
    k, v, table, n = ref.make([20], 2, 16, seed=1)
    cache = kvs.PagedKV(k, v, table, n)
    cu = torch.tensor([0, 1], dtype=torch.int32, device=DEV)
    for call in (lambda: kvs.paged_decode_attn(torch.empty(1, 2, 0, D, device=DEV), cache),
                 lambda: kvs.paged_decode_attn(torch.empty(1, 2, 0, D, device=DEV), cache,
                                               mass=torch.zeros(1, 2, cache.cap, device=DEV)),
                 lambda: kvs.paged_prompt_attn(torch.empty(1, 0, D, dtype=torch.bfloat16, device=DEV), cu, cache)):
        with pytest.raises(kvs.KvsError, match="H=0"):
            call()
    for none in (k[:0], k[:, :0], k[:, :, :0]):
        with pytest.raises(ValueError, match="empty"):
            kvs.PagedKV(none, none, table, n)


def test_a_cache_of_no_requests_is_refused(kvs):
    k, v, table, n = ref.make([20], 2, 16, seed=1)
    cache = kvs.PagedKV(k, v, table[:0], n[:0])
    none = torch.empty(0, 8, D, dtype=torch.bfloat16, device=DEV)
    for call in (lambda: kvs.paged_decode_attn(none.view(0, 2, 4, D), cache),
                 lambda: kvs.paged_prompt_attn(none, torch.zeros(1, dtype=torch.int32, device=DEV), cache),
                 lambda: kvs.paged_append(cache, none[:, :2], none[:, :2]),
                 lambda: kvs.paged_evict(cache, torch.zeros(0, 2, cache.cap, device=DEV), 8)):
        with pytest.raises(kvs.KvsError):
            call()


# ----------------------------------------------------------------------------- prompt

def _prompt(kvs, lens, new, G, H, page, window, sinks, seed=0, pad=3, layout="head", poison=True):
    k, v, table, n = ref.make(lens, G, page, seed=seed, layout=layout, poison=poison)
    cache = kvs.PagedKV(k, v, table, n)
    cu = [0] + [int(x) for x in np.cumsum(new)]
    T = cu[-1] + pad
    g = torch.Generator(device=DEV).manual_seed(seed)
    q = torch.randn(T, G * H, D, generator=g, device=DEV).to(torch.bfloat16)
    q[cu[-1]:] = float("nan")
    out = torch.full((T, G * H, D), 3.5, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((T, G * H), -7.25, device=DEV)
    st = _status()
    kvs.paged_prompt_attn(q, torch.tensor(cu, dtype=torch.int32, device=DEV), cache, window, sinks, out=out, lse=lse,
                          dev_status=st)
    ref.check_prompt(out, lse, q, cu, k, v, table, lens, window, sinks, SC, G)
    assert bool((out[cu[-1]:] == 3.5).all()) and bool((lse[cu[-1]:] == -7.25).all()), "rows behind the last request"
    assert int(st) == 0


@pytest.mark.parametrize("H", [1, 2, 3, 4, 5, 6, 7, 8])
def test_prompt_head_counts(kvs, H):
    _prompt(kvs, [1, 2, 130, 515, 64], [1, 2, 130, 300, 1], 2, H, 16, 0, 0, seed=H)


@pytest.mark.parametrize("page", [16, 64, 128, 1024])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (1, 2), (17, 5), (128, 4), (129, 130), (600, 1), (4000, 4)])
@pytest.mark.parametrize("layout", ["head", "token"])
def test_prompt_windows(kvs, page, window, sinks, layout):
    _prompt(kvs, [700, 1301, 31], [700, 257, 0], 1, 4, page, window, sinks, seed=window, layout=layout)


@pytest.mark.parametrize("lens,new", [([0], [0]), ([1], [1]), ([2000], [1]), ([900, 0, 0, 40], [900, 0, 0, 40]),
                                      ([127, 128, 129], [127, 128, 129]), ([255, 256, 257], [255, 256, 257])])
def test_prompt_lengths(kvs, lens, new):
    _prompt(kvs, lens, new, 2, 2, 16, 0, 0, seed=len(lens))


def test_prompt_long(kvs):
    _prompt(kvs, [4500], [4500], 1, 2, 64, 0, 0, seed=1)
    _prompt(kvs, [4500], [2000], 1, 2, 64, 1000, 4, seed=2)


@pytest.mark.parametrize("G,H,window,sinks", [(4, 8, 0, 0), (3, 5, 300, 7), (8, 8, 64, 0)])
def test_prompt_several_items_a_block(kvs, G, H, window, sinks):
    """More items than SMs: a block takes items of several requests and KV heads in turn."""
    _prompt(kvs, [1500, 1700, 3, 700], [1500, 900, 3, 640], G, H, 32, window, sinks, seed=G)


@pytest.mark.parametrize("R,G,H,most,window,sinks", [(100, 3, 4, 60, 0, 0), (170, 2, 8, 40, 33, 3), (31, 8, 5, 200, 0, 0)])
def test_prompt_items_of_many_requests(kvs, R, G, H, most, window, sinks):
    """Items of many short requests, some without a new token, several a block: found from request to request."""
    rng = np.random.default_rng(R)
    new = [int(x) * (i % 5 != 2) for i, x in enumerate(rng.integers(0, most, R))]
    lens = [c + int(x) for c, x in zip(new, rng.integers(0, 300, R))]
    new[40:60] = [0] * len(new[40:60])  # and a run of them
    _prompt(kvs, lens, new, G, H, 16, window, sinks, seed=R)


@pytest.mark.parametrize("H", [1, 4, 5, 8])
@pytest.mark.parametrize("lens,new,G,page,window,sinks", [
    ([9000], [3], 1, 64, 0, 0), ([9000, 100, 0, 5000], [5, 100, 0, 1], 2, 16, 0, 0),
    ([20011, 700], [40, 2], 1, 128, 3000, 200), ([6000, 8000], [1, 1], 8, 32, 50, 0),
    ([4, 12000], [9, 4], 2, 1024, 0, 0)])
def test_prompt_few_queries_over_a_long_cache(kvs, lens, new, G, page, window, sinks, H):
    """Items split over the tokens they see and joined; pieces with nothing to see among them."""
    k, v, table, n = ref.make(lens, G, page, seed=H + page)
    cache = kvs.PagedKV(k, v, table, n)
    assert (kvs._lib.kvs_paged_prompt_workspace_size(len(lens), G, H, sum(new) + 3, cache.cap, window, sinks) > 0) \
        == (window != 50)
    cu = [0] + [int(x) for x in np.cumsum(new)]
    T = cu[-1] + 3
    q = torch.randn(T, G * H, D, device=DEV).to(torch.bfloat16)
    q[cu[-1]:] = float("nan")
    out = torch.full((T, G * H, D), 3.5, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((T, G * H), -7.25, device=DEV)
    st = _status()
    kvs.paged_prompt_attn(q, torch.tensor(cu, dtype=torch.int32, device=DEV), cache, window, sinks, out=out, lse=lse,
                          dev_status=st)
    ref.check_prompt(out, lse, q, cu, k, v, table, lens, window, sinks, SC, G)
    assert bool((out[cu[-1]:] == 3.5).all()) and bool((lse[cu[-1]:] == -7.25).all()) and int(st) == 0


def test_prompt_pieces_in_a_graph_and_on_two_streams(kvs):
    """A split call captured, and replayed after the lengths, offsets and queries changed in place (down to
    caches of fewer tiles than pieces); two at once, each with its own workspace."""
    lens = [9000, 6000]
    k, v, table, n = ref.make(lens, 2, 64, seed=31, poison=False)
    cache = kvs.PagedKV(k, v, table, n)
    cu = torch.tensor([0, 4, 7], dtype=torch.int32, device=DEV)
    q = torch.randn(8, 8, D, device=DEV).to(torch.bfloat16)
    out, lse = torch.zeros(8, 8, D, dtype=torch.bfloat16, device=DEV), torch.zeros(8, 8, device=DEV)
    kvs.paged_prompt_attn(q, cu, cache)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kvs.paged_prompt_attn(q, cu, cache, out=out, lse=lse)
    for m, c in ((lens, [0, 4, 7]), ([300, 8], [0, 1, 8]), ([5000, 0], [0, 8, 8]), ([0, 1], [0, 0, 1])):
        n.copy_(torch.tensor(m))
        cu.copy_(torch.tensor(c))
        q.normal_()
        graph.replay()
        ref.check_prompt(out, lse, q, c, k, v, table, m, 0, 0, SC, 2)
    n.copy_(torch.tensor(lens))
    qs = [torch.randn(6, 8, D, device=DEV).to(torch.bfloat16) for _ in range(2)]
    cu.copy_(torch.tensor([0, 2, 6]))
    want = [kvs.paged_prompt_attn(x, cu, cache) for x in qs]
    side = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[kvs.paged_prompt_attn(x, cu, cache, stream=s) for x, s in zip(qs, side)] for _ in range(10)]
    torch.cuda.synchronize()
    for pair in got:
        for (o, l), (wo, wl) in zip(pair, want):
            assert torch.equal(o, wo) and torch.equal(l, wl)


@pytest.mark.parametrize("H", [1, 4, 5, 8])
@pytest.mark.parametrize("lens,new,window,sinks,wide", [
    ([700], [700], 0, 0, 0), ([1500, 130, 400], [300, 130, 7], 0, 0, 0), ([700, 900], [700, 300], 100, 0, 0),
    ([1300], [1300], 300, 70, 0), ([800, 700], [700, 650], 20, 300, 0), ([600, 500], [600, 2], 1, 3, 0), ([6000, 5100], [40, 150], 0, 0, 9000),
    ([5000, 5000], [300, 64], 3000, 200, 9000)])
def test_prompt_values_that_are_not_finite_reach_only_those_who_see_them(kvs, H, lens, new, window, sinks, wide):
    """NaN and infinities in V, in single values and whole rows, in the middle of the queries' own tokens and at the
    edges of their windows: a query has them in the channels of the rows that it sees and nowhere else, and
    everything else is bit for bit what it is without them. Whole and split."""
    G, page = 2, 16
    k, v, table, n = ref.make(lens, G, page, seed=H + window, poison=False, cap_pages=wide // page or None)
    cu = [0] + [int(x) for x in np.cumsum(new)]
    cut = torch.tensor(cu, dtype=torch.int32, device=DEV)
    q = torch.randn(cu[-1], G * H, D, device=DEV).to(torch.bfloat16)
    good_v = v.clone()
    want, wl = kvs.paged_prompt_attn(q, cut, kvs.PagedKV(k, good_v, table, n), window, sinks)
    ref.check_prompt(want, wl, q, cu, k, good_v, table, lens, window, sinks, SC, G)
    rng = np.random.default_rng(H + len(lens))
    inf, nan = float("inf"), float("nan")
    hit = torch.zeros(len(lens), max(lens), G, D, dtype=torch.bool, device=DEV)
    for r, (m, c) in enumerate(zip(lens, new)):
        p0 = m - c
        at = {p0, m - 1, p0 + c // 2, p0 + c // 3, min(m - 1, p0 + 63), min(m - 1, p0 + 65)}
        at |= {int(x) for x in rng.integers(p0, m, 6)} | {max(0, p0 - window + 1), max(0, p0 + c // 2 - window)}
        for i, j in enumerate(sorted(at)):
            g, d = i % G, int(rng.integers(0, 100))
            pg = int(table[r, j // page])
            v[pg, g, j % page, d] = (inf, nan, -inf)[i % 3]
            if i % 5 == 4:
                v[pg, g, j % page, 100:] = nan  # many channels of one row
        rows = torch.stack([v[int(table[r, j // page]), :, j % page] for j in range(m)])
        hit[r, :m] = ~torch.isfinite(rows)
    st = _status()
    out, lse = kvs.paged_prompt_attn(q, cut, kvs.PagedKV(k, v, table, n), window, sinks, dev_status=st)
    assert int(st) == 0 and torch.equal(lse, wl)
    for r, (m, c) in enumerate(zip(lens, new)):
        p = torch.arange(m - c, m, device=DEV).view(-1, 1)
        j = torch.arange(m, device=DEV)
        ok = j <= p
        if window:
            ok = ok & ((j < sinks) | (j > p - window))
        # [c][G][D]: some row that the query sees is not finite there
        bad = torch.einsum("cj,jgd->cgd", ok.double(), hit[r, :m].double()) > 0
        bad = bad.unsqueeze(2).expand(-1, -1, H, -1).reshape(c, G * H, D)
        o, w = out[cu[r]:cu[r + 1]], want[cu[r]:cu[r + 1]]
        assert torch.equal(~torch.isfinite(o.float()), bad), r
        assert torch.equal(_bits(o)[~bad], _bits(w)[~bad]), r
        assert bool(bad.any()) and not bool(bad.all())


def test_prompt_whole_rows_that_are_not_finite(kvs):
    """Every V row from a position on is infinite or NaN: the queries before it are as they were."""
    k, v, table, n = ref.make([500], 1, 64, seed=77, poison=False)
    cache = kvs.PagedKV(k, v, table, n)
    cu = torch.tensor([0, 500], dtype=torch.int32, device=DEV)
    q = torch.randn(500, 4, D, device=DEV).to(torch.bfloat16)
    want, wl = kvs.paged_prompt_attn(q, cu, cache)
    for first in (499, 257, 256, 130, 1):
        for j in range(first, 500):
            v[int(table[0, j // 64]), :, j % 64] = float("nan") if first % 2 else float("inf")
        out, lse = kvs.paged_prompt_attn(q, cu, cache)
        assert torch.equal(_bits(out[:first]), _bits(want[:first])) and torch.equal(lse, wl)
        assert not bool(torch.isfinite(out[first:].float()).any())
        assert first % 2 or bool((out[first] == float("inf")).all())


def test_kept_workspaces_serve_calls_of_other_sizes(kvs):
    """One workspace for prompts of few queries (split) and many (whole), one for evictions to smaller budgets."""
    lens, G, H = [9000, 700], 2, 4
    k, v, table, n = ref.make(lens, G, 64, seed=53, poison=False)
    cache = kvs.PagedKV(k, v, table, n)
    ws = kvs.paged_prompt_workspace(cache, H, 700)
    for new in ([3, 0], [100, 40], [500, 200], [1, 1]):
        cu = [0] + [int(x) for x in np.cumsum(new)]
        q = torch.randn(cu[-1], G * H, D, device=DEV).to(torch.bfloat16)
        cut = torch.tensor(cu, dtype=torch.int32, device=DEV)
        out, lse = kvs.paged_prompt_attn(q, cut, cache, ws=ws)
        ref.check_prompt(out, lse, q, cu, k, v, table, lens, 0, 0, SC, G)
    assert kvs.paged_prompt_workspace(cache, H, 700, window=50) is None
    mass = torch.rand(2, G, cache.cap, device=DEV)
    we = kvs.paged_evict_workspace(cache, 600)
    for budget in (600, 77):
        mo, no = torch.zeros_like(mass), torch.zeros_like(n)
        src = kvs.paged_evict(cache, mass, budget, mass_out=mo, n_out=no, ws=we)
        for r in range(2):
            for g in range(G):
                want = ref.evict(mass[r, g].cpu().numpy(), np.arange(cache.cap), lens[r], lens[r], budget, 0, 0)
                assert np.array_equal(src[r, g].cpu().numpy()[:len(want)], want)


def test_prompt_items_that_see_nothing(kvs):
    """Many queries in front of the first token, between items that see something."""
    lens, new, G, H = [3, 260, 0], [900, 260, 500], 8, 8
    k, v, table, n = ref.make(lens, G, 16, seed=29)
    cache = kvs.PagedKV(k, v, table, n)
    cu = [0, 900, 1160, 1660]
    q = torch.randn(1660, G * H, D, device=DEV).to(torch.bfloat16)
    st = _status()
    out, lse = kvs.paged_prompt_attn(q, torch.tensor(cu, dtype=torch.int32, device=DEV), cache, dev_status=st)
    ref.check_prompt(out, lse, q, cu, k, v, table, lens, 0, 0, SC, G)
    assert bool((out[:897] == 0).all()) and bool((out[1160:] == 0).all()) and int(st) == 0


@pytest.mark.parametrize("warp", range(12))
@pytest.mark.parametrize("lens,new", [([3000, 40, 900], [300, 40, 7]), ([200] * 300, [200] * 300)])
def test_prompt_bounded_waits_run_out_and_the_call_ends(kvs, lens, new, warp):
    """One warp of every block gives up at its second tile: the other roles end too, the status word says so,
    and the next call is right. Items of many tiles, and blocks with several items."""
    import time
    k, v, table, n = ref.make(lens, 2, 64, seed=52, poison=False)
    cache = kvs.PagedKV(k, v, table, n)
    cu = [0] + [int(x) for x in np.cumsum(new)]
    cut = torch.tensor(cu, dtype=torch.int32, device=DEV)
    q = torch.randn(cu[-1], 8, D, device=DEV).to(torch.bfloat16)
    st = _status()
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    kvs.selftest_paged_prompt_timeout(q, cut, cache, warp, 2_000_000, st)
    torch.cuda.synchronize()
    assert int(st) == kvs.KVS_ETIMEOUT and time.perf_counter() - t0 < 5.0
    st = _status()
    out, lse = kvs.paged_prompt_attn(q, cut, cache, dev_status=st)
    ref.check_prompt(out, lse, q, cu, k, v, table, lens, 0, 0, SC, 2)
    assert int(st) == 0


def test_empty_calls(kvs):
    k, v, table, n = ref.make([20], 2, 16, seed=1)
    cache = kvs.PagedKV(k, v, table, n)
    cu = torch.zeros(2, dtype=torch.int32, device=DEV)
    none = torch.empty(0, 8, D, dtype=torch.bfloat16, device=DEV)
    out, lse = kvs.paged_prompt_attn(none, cu, cache)
    assert out.shape == (0, 8, D) and lse.shape == (0, 8)
    before = k.clone()
    kvs.paged_append(cache, none[:, :2], none[:, :2], cu)
    assert torch.equal(_bits(k), _bits(before))


def test_calls_at_once_on_two_streams(kvs):
    """Prompts, decodes and evictions of two caches side by side, again and again, give what they give alone."""
    sides = []
    for i in range(2):
        k, v, table, n = ref.make([700 + 300 * i, 90, 2000], 4, 16, seed=40 + i, poison=False)
        cache = kvs.PagedKV(k, v, table, n)
        q = torch.randn(500, 16, D, device=DEV).to(torch.bfloat16)
        cu = torch.tensor([0, 300, 350, 500], dtype=torch.int32, device=DEV)
        mass = torch.rand(3, 4, cache.cap, device=DEV)
        sides.append((cache, q, cu, q[:3].view(3, 4, 4, D).contiguous(), mass))

    def run(i, stream):
        cache, q, cu, q1, mass = sides[i]
        mo, no = torch.zeros_like(mass), torch.zeros_like(cache.n)
        return [*kvs.paged_prompt_attn(q, cu, cache, 200, 4, stream=stream), *kvs.paged_decode_attn(q1, cache, stream=stream),
                kvs.paged_evict(cache, mass, 600, mass_out=mo, n_out=no, stream=stream)]

    want = [run(i, None) for i in range(2)]  # (the moves of an eviction repeated are the same)
    want = [run(i, None) for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(10):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got.append((i, run(i, streams[i])))
    torch.cuda.synchronize()
    for i, outs in got:
        for a, b in zip(outs, want[i]):
            assert torch.equal(a, b)


def test_prompt_many_requests(kvs):
    rng = np.random.default_rng(1)
    new = [int(x) for x in rng.integers(0, 9, 300)]
    _prompt(kvs, [x + int(y) for x, y in zip(new, rng.integers(0, 50, 300))], new, 1, 3, 16, 0, 0, seed=4)


def test_prompt_queries_before_the_first_token(kvs):
    """More queries than tokens: those in front of the first see nothing."""
    k, v, table, n = ref.make([3], 1, 16, seed=9)
    cache = kvs.PagedKV(k, v, table, n)
    q = torch.randn(5, 2, D, device=DEV).to(torch.bfloat16)
    out, lse = kvs.paged_prompt_attn(q, torch.tensor([0, 5], dtype=torch.int32, device=DEV), cache)
    ref.check_prompt(out, lse, q, [0, 5], k, v, table, [3], 0, 0, SC, 1)
    assert bool((out[:2] == 0).all()) and bool(torch.isneginf(lse[:2]).all())


def test_prompt_released_pages_and_strided_rows(kvs):
    """Pages that the window of every query has passed are gone; the queries and outputs are slices of wider rows."""
    lens, new, page, window, sinks = [2000], [300], 16, 100, 20
    k, v, table, n = ref.make(lens, 2, page, seed=12)
    good = table.clone()
    for p in range(2, (2000 - 300 - 99) // page):
        table[0, p] = -1
    cache = kvs.PagedKV(k, v, table, n)
    wide = torch.randn(300, 8 * D + 16, device=DEV).to(torch.bfloat16)
    q = wide[:, 8:8 + 8 * D].view(300, 8, D)
    ow = torch.zeros(300, 8 * D + 64, dtype=torch.bfloat16, device=DEV)
    out = ow[:, 64:].view(300, 8, D)
    st = _status()
    _, lse = kvs.paged_prompt_attn(q, torch.tensor([0, 300], dtype=torch.int32, device=DEV), cache, window, sinks,
                                   out=out, dev_status=st)
    ref.check_prompt(out, lse, q, [0, 300], k, v, good, lens, window, sinks, SC, 2)
    assert int(st) == 0 and bool((ow[:, :64] == 0).all())


def test_prompt_bad_page(kvs):
    k, v, table, n = ref.make([100], 1, 16, seed=13, poison=False)
    cache = kvs.PagedKV(k, v, table, n)
    good = table.clone()
    table[0, 2] = -1
    q = torch.randn(100, 2, D, device=DEV).to(torch.bfloat16)
    st = _status()
    out, lse = kvs.paged_prompt_attn(q, torch.tensor([0, 100], dtype=torch.int32, device=DEV), cache, dev_status=st)
    assert int(st) == kvs.KVS_EBOUNDS
    some = [j for j in range(100) if j // 16 != 2]
    K, V = ref.tokens(k, good, 0, 100)[some, 0], ref.tokens(v, good, 0, 100)[some, 0]
    o, ls, _, _, _ = ref.attend(q[99].double(), K, V, SC)
    assert float((out[99] - o).abs().max()) < 0.03 and float((lse[99] - ls).abs().max()) < 1e-4


@pytest.mark.parametrize("scale", [-0.25, 1.0, 1e-3])
def test_scales(kvs, scale):
    lens = [200, 333]
    k, v, table, n = ref.make(lens, 2, 32, seed=23)
    cache = kvs.PagedKV(k, v, table, n)
    q = torch.randn(300, 4, D, device=DEV).to(torch.bfloat16)
    cu = [0, 200, 300]
    out, lse = kvs.paged_prompt_attn(q, torch.tensor(cu, dtype=torch.int32, device=DEV), cache, scale=scale)
    ref.check_prompt(out, lse, q, cu, k, v, table, lens, 0, 0, scale, 2)
    q = torch.randn(2, 2, 4, D, device=DEV)
    out, lse = kvs.paged_decode_attn(q, cache, scale=scale)
    ref.check_decode(out, lse, q, k, v, table, lens, 0, 0, scale)


def test_prompt_offsets_out_of_range(kvs):
    """Offsets beyond the packed rows are cut off there."""
    k, v, table, n = ref.make([50, 50], 1, 16, seed=24)
    cache = kvs.PagedKV(k, v, table, n)
    q = torch.randn(40, 2, D, device=DEV).to(torch.bfloat16)
    st = _status()
    out, lse = kvs.paged_prompt_attn(q, torch.tensor([-5, 30, 1 << 30], dtype=torch.int32, device=DEV), cache,
                                     dev_status=st)
    assert int(st) == kvs.KVS_EBOUNDS
    ref.check_prompt(out, lse, q, [0, 30, 40], k, v, table, [50, 50], 0, 0, SC, 1)


def test_prompt_growing_logits(kvs):
    """Each token's logit is larger than all before it, and the reverse: the output is rescaled again and
    again, and not at all. Values that no query sees are NaN."""
    lens = [600, 600]
    k, v, table, n = ref.make(lens, 1, 64, seed=25)
    for r in range(2):
        for j in range(600):
            pg = int(table[r, j // 64])
            k[pg, 0, j % 64] = 0.0
            k[pg, 0, j % 64, 0] = float(j if r == 0 else 600 - j)
    cache = kvs.PagedKV(k, v, table, n)
    q = torch.zeros(700, 4, D, dtype=torch.bfloat16, device=DEV)
    q[:, 0, 0], q[:, 1, 0], q[:, 2, 0], q[:, 3, 0] = 0.01, 1.0, 20.0, 300.0
    cu = [0, 400, 700]
    out, lse = kvs.paged_prompt_attn(q, torch.tensor(cu, dtype=torch.int32, device=DEV), cache)
    ref.check_prompt(out, lse, q, cu, k, v, table, lens, 0, 0, SC, 1)


def test_prompt_stream_and_graph(kvs):
    k, v, table, n = ref.make([400, 60], 2, 16, seed=15, poison=False)
    cache = kvs.PagedKV(k, v, table, n)
    q = torch.randn(200, 8, D, device=DEV).to(torch.bfloat16)
    cu = torch.tensor([0, 150, 200], dtype=torch.int32, device=DEV)
    want, wl = kvs.paged_prompt_attn(q, cu, cache)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    got, gl = kvs.paged_prompt_attn(q, cu, cache, stream=s)
    s.synchronize()
    assert torch.equal(got, want) and torch.equal(gl, wl)
    graph = torch.cuda.CUDAGraph()
    out, lse = torch.zeros_like(want), torch.zeros_like(wl)
    with torch.cuda.graph(graph):
        kvs.paged_prompt_attn(q, cu, cache, out=out, lse=lse)
    for c in ([0, 150, 200], [0, 10, 70], [0, 200, 200]):
        cu.copy_(torch.tensor(c))
        q.normal_()
        graph.replay()
        ref.check_prompt(out, lse, q, c, k, v, table, [400, 60], 0, 0, SC, 2)


def test_decode_and_prompt_agree(kvs):
    """One new token through either form."""
    lens = [100, 777, 3, 2050]
    k, v, table, n = ref.make(lens, 2, 32, seed=17)
    cache = kvs.PagedKV(k, v, table, n)
    q = torch.randn(4, 2, 4, D, device=DEV).to(torch.bfloat16)
    for window, sinks in ((0, 0), (100, 4)):
        do, dl = kvs.paged_decode_attn(q, cache, window, sinks)
        po, pl = kvs.paged_prompt_attn(q.view(4, 8, D), torch.arange(5, dtype=torch.int32, device=DEV), cache, window,
                                       sinks)
        # the prompt form's two roundings to bf16 (weights, output), each within half a step of values of at most max |V|
        assert float((do.view(4, 8, D) - po.float()).abs().max()) <= 2 * 2.0 ** -8 * float(v.float().nan_to_num(0).abs().max())
        assert float((dl.view(4, 8) - pl).abs().max()) < 1e-4


# ----------------------------------------------------------------------------- eviction

def _evict_case(kvs, lens, G, page, budget, sinks, recent, seed, mass, pos, seen, layout="head", in_place=True):
    k, v, table, n = ref.make(lens, G, page, seed=seed, layout=layout)
    cache = kvs.PagedKV(k, v, table, n)
    R = len(lens)
    k0, v0 = k.clone(), v.clone()
    m0 = mass(R, G, cache.cap)
    p0 = pos(R, G, cache.cap)
    m, p = m0.clone(), None if p0 is None else p0.clone()
    kw = dict(sinks=sinks, recent=recent, pos=p, seen=seen)
    st = _status()
    if in_place:
        src = kvs.paged_evict(cache, m, budget, dev_status=st, **kw)
        n_out, mo, po = n, m, p
    else:
        mo = torch.full_like(m, -1.0)
        po = None if p is None else torch.full_like(p, -1)
        n_out = torch.empty_like(n)
        src = kvs.paged_evict(cache, m, budget, mass_out=mo, pos_out=po, n_out=n_out, dev_status=st, **kw)
        assert torch.equal(m.nan_to_num(-5), m0.nan_to_num(-5)) and n.tolist() == lens
    assert int(st) == 0
    wk, wv = k0.clone(), v0.clone()
    for r, x in enumerate(lens):
        assert int(n_out[r]) == min(x, budget)
        for g in range(G):
            pr = np.arange(cache.cap) if p0 is None else p0[r, g].cpu().numpy()
            want = ref.evict(m0[r, g].cpu().numpy(), pr, x, x if seen is None else int(seen[r]), budget, sinks, recent)
            got = src[r, g].cpu().numpy()
            assert np.array_equal(got[:len(want)], want) and np.all(got[len(want):] == -1), (r, g)
            w = torch.from_numpy(want).to(DEV)
            assert torch.equal(mo[r, g, :len(want)].nan_to_num(-5), m0[r, g, w].nan_to_num(-5))
            rest = m0[r, g, len(want):] if in_place else torch.full_like(m0[r, g, len(want):], -1.0)
            assert torch.equal(mo[r, g, len(want):].nan_to_num(-5), rest.nan_to_num(-5)), "entries behind the last"
            if p0 is not None:
                assert torch.equal(po[r, g, :len(want)], p0[r, g, w])
            for j in np.nonzero(want != np.arange(len(want)))[0]:
                a, b = int(want[j]), int(j)
                pa, pb = int(table[r, a // page]), int(table[r, b // page])
                wk[pb, g, b % page], wv[pb, g, b % page] = k0[pa, g, a % page], v0[pa, g, a % page]
    assert torch.equal(_bits(k), _bits(wk)) and torch.equal(_bits(v), _bits(wv))


def _rand(seed, levels=0):
    def f(R, G, cap):
        m = torch.rand(R, G, cap, generator=torch.Generator().manual_seed(seed)).to(DEV)
        return (m * levels).floor() if levels else m
    return f


def _perm(seed):
    def f(R, G, cap):
        return torch.argsort(torch.rand(R, G, cap, generator=torch.Generator().manual_seed(seed)), -1).to(
            torch.int32).to(DEV)
    return f


def _none(*_):
    return None


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("budget,sinks,recent", [(1, 0, 0), (1, 1, 0), (1, 0, 1), (16, 4, 4), (100, 0, 100), (333, 5, 60),
                                                 (1024, 4, 300), (2500, 0, 0)])
def test_evict(kvs, budget, sinks, recent, in_place):
    _evict_case(kvs, [0, 1, budget, budget + 1, 2 * budget + 3, 2222], 2, 16, budget, sinks, recent, budget,
                _rand(1), _none, None, in_place=in_place)


@pytest.mark.parametrize("levels", [1, 2, 7])
def test_evict_ties_go_to_the_lower_slot(kvs, levels):
    _evict_case(kvs, [1500, 64, 65], 2, 64, 64, 3, 9, levels, _rand(2, levels), _none, None, layout="token")


def test_evict_places(kvs):
    """Slots out of order, and a request that has had more tokens than it holds."""
    lens = [900, 400, 130]
    seen = torch.tensor([900, 7000, 130], dtype=torch.int32, device=DEV)
    _evict_case(kvs, lens, 3, 32, 128, 6, 40, 3, _rand(3), _perm(3), seen, layout="both")
    _evict_case(kvs, lens, 3, 32, 128, 6, 40, 3, _rand(3), _perm(3), None, in_place=False)


def test_evict_infinities_nan_and_signed_zero(kvs):
    def mass(R, G, cap):
        m = torch.randn(R, G, cap, generator=torch.Generator().manual_seed(4)).to(DEV)
        pick = torch.randint(0, 6, (R, G, cap), generator=torch.Generator().manual_seed(5)).to(DEV)
        for i, x in enumerate((float("inf"), float("-inf"), float("nan"), -0.0, 0.0)):
            m[pick == i] = x
        return m
    _evict_case(kvs, [600, 200], 2, 16, 170, 2, 10, 6, mass, _none, None)
    _evict_case(kvs, [600, 200], 2, 16, 60, 0, 0, 6, mass, _none, None)
    _evict_case(kvs, [600, 200], 2, 16, 590, 0, 0, 6, mass, _none, None, in_place=False)


def test_evict_long_rows(kvs):
    _evict_case(kvs, [70001, 52000, 9000], 1, 256, 8000, 4, 1000, 7, _rand(7), _none, None)


def test_evict_rows_beyond_shared_memory(kvs):
    """Runs of more slots than a block holds keys for."""
    _evict_case(kvs, [190000, 188001], 1, 1024, 5000, 4, 1000, 17, _rand(17), _none, None)
    _evict_case(kvs, [190000], 1, 1024, 70000, 4, 1000, 18, _rand(18, 50), _perm(18), None)


def test_evict_many_rows(kvs):
    _evict_case(kvs, [40 + i % 30 for i in range(200)], 2, 16, 48, 4, 8, 9, _rand(9), _none, None)


def test_evict_bad_page(kvs):
    """A row whose page id is none does not move; the others do."""
    k, v, table, n = ref.make([64], 1, 16, seed=20, poison=False)
    cache = kvs.PagedKV(k, v, table, n)
    mass = torch.zeros(1, 1, cache.cap, device=DEV)
    mass[0, 0, 16:64] = 1.0
    table[0, 3] = -4
    k0 = k.clone()
    st = _status()
    src = kvs.paged_evict(cache, mass, 48, dev_status=st)
    assert int(st) == kvs.KVS_EBOUNDS
    assert src[0, 0].tolist() == list(range(48, 64)) + list(range(16, 48))
    assert torch.equal(_bits(k), _bits(k0))


def test_evict_stream_and_graph(kvs):
    k, v, table, n = ref.make([300, 200], 2, 16, seed=21, poison=False)
    cache = kvs.PagedKV(k, v, table, n)
    mass = torch.rand(2, 2, cache.cap, device=DEV)
    mo, no = torch.zeros_like(mass), torch.zeros_like(n)
    src = torch.zeros(2, 2, 150, dtype=torch.int32, device=DEV)
    k0, v0 = k.clone(), v.clone()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    a = kvs.paged_evict(cache, mass, 150, mass_out=mo, n_out=no, stream=s).clone()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kvs.paged_evict(cache, mass, 150, mass_out=mo, n_out=no, src=src)
    for i in range(3):
        k.copy_(k0), v.copy_(v0)
        graph.replay()
        for r, x in enumerate([300, 200]):
            for g in range(2):
                want = ref.evict(mass[r, g].cpu().numpy(), np.arange(cache.cap), x, x, 150, 0, 0)
                assert np.array_equal(src[r, g].cpu().numpy(), want)
                if i == 0:
                    assert torch.equal(a[r, g], src[r, g])
        mass.uniform_()


@pytest.mark.parametrize("in_place", [True, False])
def test_evict_replays_move_rows(kvs, in_place):
    """A captured eviction, replayed on other lengths, places and weights: moved K and V rows, weights, places and
    lengths, each against the definition."""
    G, page, budget, sinks, recent = 2, 16, 130, 3, 20
    k, v, table, n = ref.make([400, 400, 270], G, page, seed=61, poison=False)  # pages for every replay
    cache = kvs.PagedKV(k, v, table, n)
    mass = torch.rand(3, G, cache.cap, device=DEV)
    pos = _perm(61)(3, G, cache.cap)
    seen = n.clone()
    mo, po, no = (mass, pos, n) if in_place else (torch.full_like(mass, -1.0), torch.full_like(pos, -1), n.clone())
    src = torch.empty(3, G, budget, dtype=torch.int32, device=DEV)
    st = _status()
    good = [t.clone() for t in (k, v, mass, pos, n)]
    call = dict(sinks=sinks, recent=recent, pos=pos, seen=seen, src=src, mass_out=mo, pos_out=po, n_out=no, dev_status=st)
    kvs.paged_evict(cache, mass, budget, **call)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kvs.paged_evict(cache, mass, budget, **call)
    for t, x in zip((k, v, mass, pos, n), good):
        t.copy_(x)
    for i, lens in enumerate(([400, 400, 90], [131, 130, 129], [0, 399, 260])):
        n.copy_(torch.tensor(lens))
        seen.copy_(torch.tensor(lens) + 50 * i)
        mass.uniform_()
        pos.copy_(_perm(62 + i)(3, G, cache.cap))
        before = [t.clone() for t in (k, v, mass, pos)]
        graph.replay()
        wk, wv, m0, p0 = before[0].clone(), before[1].clone(), before[2], before[3]
        assert no.tolist() == [min(x, budget) for x in lens]
        for r, x in enumerate(lens):
            for g in range(G):
                want = ref.evict(m0[r, g].cpu().numpy(), p0[r, g].cpu().numpy(), x, x + 50 * i, budget, sinks, recent)
                assert np.array_equal(src[r, g, :len(want)].cpu().numpy(), want) and bool((src[r, g, len(want):] == -1).all())
                w = torch.from_numpy(want).to(DEV)
                assert torch.equal(mo[r, g, :len(want)], m0[r, g, w]) and torch.equal(po[r, g, :len(want)], p0[r, g, w])
                for b in np.nonzero(want != np.arange(len(want)))[0]:
                    a, b = int(want[b]), int(b)
                    pa, pb = int(table[r, a // page]), int(table[r, b // page])
                    wk[pb, g, b % page] = before[0][pa, g, a % page]
                    wv[pb, g, b % page] = before[1][pa, g, a % page]
        assert torch.equal(_bits(k), _bits(wk)) and torch.equal(_bits(v), _bits(wv)) and int(st) == 0


# ----------------------------------------------------------------------------- all together

@pytest.mark.parametrize("window,sinks", [(0, 0), (90, 3)])
def test_a_generation_under_a_budget(kvs, window, sinks):
    """Prompts, then tokens one by one, with the weights added up and the cache cut back to its budget
    whenever it is 16 tokens over: against a list of tokens for each head that is kept the same way."""
    R, G, H, page, budget, recent, keep = 3, 2, 4, 16, 96, 24, 2
    steps, prompt = 40, [150, 30, 97]
    gen = torch.Generator(device=DEV).manual_seed(33)
    rnd = lambda *s: torch.randn(*s, generator=gen, device=DEV).to(torch.bfloat16)  # noqa: E731
    mp = 16
    pages = R * mp
    k = torch.full((pages, G, page, D), float("nan"), dtype=torch.bfloat16, device=DEV)
    v = k.clone()
    table = torch.randperm(pages, generator=gen, device=DEV).to(torch.int32).view(R, mp)
    n = torch.tensor(prompt, dtype=torch.int32, device=DEV)
    seen = n.clone()
    cache = kvs.PagedKV(k, v, table, n)
    mass = torch.full((R, G, cache.cap), float("nan"), device=DEV)
    pos = torch.full((R, G, cache.cap), -1, dtype=torch.int32, device=DEV)
    st = _status()

    cu = torch.tensor([0] + list(np.cumsum(prompt)), dtype=torch.int32, device=DEV)
    T = int(cu[-1])
    Kn, Vn, q = rnd(T, G, D), rnd(T, G, D), rnd(T, G * H, D)
    kvs.paged_append(cache, Kn, Vn, cu, mass=mass, pos=pos, seen=seen, dev_status=st)
    out, lse = kvs.paged_prompt_attn(q, cu, cache, window, sinks, dev_status=st)
    ref.check_prompt(out, lse, q, cu.tolist(), k, v, table, prompt, window, sinks, SC, G)

    # the same by lists: (K, V, place) of each head, the weights as the kernels have them
    K = [[Kn[cu[r]:cu[r + 1], g].double() for g in range(G)] for r in range(R)]
    V = [[Vn[cu[r]:cu[r + 1], g].double() for g in range(G)] for r in range(R)]
    at = [[np.arange(prompt[r]) for g in range(G)] for r in range(R)]
    evictions = 0
    for step in range(steps):
        q1, k1, v1 = rnd(R, G, H, D), rnd(R, G, D), rnd(R, G, D)
        n.add_(1), seen.add_(1)
        kvs.paged_append(cache, k1, v1, mass=mass, pos=pos, seen=seen, dev_status=st)
        before = mass.clone()
        # a window over slots is a window over tokens only until the first eviction
        w_, s_ = (window, sinks) if evictions == 0 else (0, 0)
        out, lse = kvs.paged_decode_attn(q1, cache, w_, s_, mass=mass, dev_status=st)
        lens = n.tolist()
        for r in range(R):
            vis = torch.from_numpy(ref.visible(lens[r] - 1, w_, s_)).to(DEV)
            for g in range(G):
                K[r][g] = torch.cat([K[r][g], k1[r, g:g + 1].double()])
                V[r][g] = torch.cat([V[r][g], v1[r, g:g + 1].double()])
                at[r][g] = np.append(at[r][g], prompt[r] + step)
                assert K[r][g].shape[0] == lens[r]
                o, ls, w, e, va = ref.attend(q1[r, g].double(), K[r][g][vis], V[r][g][vis], SC)
                tol = (4 * e.unsqueeze(-1) + (2 * len(vis) + 64) * ref.U) * va
                assert bool(((out[r, g] - o).abs() <= tol).all()), (step, r, g)
                want = before[r, g, vis].double() + w.sum(0)
                assert float((mass[r, g, vis] - want).abs().max()) < 1e-4
        if any(x >= budget + 16 for x in lens):
            evictions += 1
            m = mass.cpu().numpy()
            src = kvs.paged_evict(cache, mass, budget, sinks=keep, recent=recent, pos=pos, seen=seen, dev_status=st)
            for r in range(R):
                for g in range(G):
                    s = ref.evict(m[r, g], at[r][g], lens[r], prompt[r] + step + 1, budget, keep, recent)
                    assert np.array_equal(src[r, g, :len(s)].cpu().numpy(), s)
                    K[r][g], V[r][g] = K[r][g][torch.from_numpy(s).to(DEV)], V[r][g][torch.from_numpy(s).to(DEV)]
                    at[r][g] = at[r][g][s]
                    assert np.array_equal(pos[r, g, :len(s)].cpu().numpy(), at[r][g])
            assert n.tolist() == [min(x, budget) for x in lens]
    assert evictions >= 3 and int(st) == 0
