"""The paged history cache on the GPU against its float64 oracle (oracle/paged.py)."""
import numpy as np
import pytest
import torch

from gen import make_case
from gen.device import case_tensors, tensor
from gen.inputs import make_attn_case
from oracle import hstu as O
from oracle import paged as P
from hstu_testutil import assert_close, binding, config_of

pytestmark = pytest.mark.gpu

UNIT = {"fp16": 2.0 ** -11, "bf16": 2.0 ** -8, "fp32": 2.0 ** -24}  # half a step, relative
DT = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}


@pytest.fixture(scope="module")
def H():
    return binding()


def i32(a):
    return torch.tensor(list(a), dtype=torch.int32, device="cuda")


def chunk_of(H, counts, ts):
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int64)
    return H.Jagged(tensor(off, torch.int64, "cuda"), tensor(np.asarray(ts, dtype=np.int64), torch.int64, "cuda"),
                    int(max(counts, default=0)), int(off[-1]))


def nan_cache(H, *, layers, heads, pages, seqs, blocks, ps, dtype):
    """An empty cache whose every slot holds NaN, and times that no event has."""
    c = H.PagedCache.empty(layers, heads, pages, seqs, blocks, ps, dtype)
    c.kv.fill_(float("nan"))
    c.timestamps.fill_(-(1 << 62))
    return c


def split_rows(offsets, counts, tail):
    """Row indices of each sequence's first n - c events (tail False) or last c."""
    idx = []
    for u, c in enumerate(counts):
        a, b = int(offsets[u]), int(offsets[u + 1])
        idx.append(np.arange(b - c, b) if tail else np.arange(a, b - c))
    return np.concatenate(idx) if idx else np.zeros(0, dtype=np.int64)


def load_cache(H, ac, cache, counts, layer=0, seq_ids=None):
    """Reserve and append all but the last counts[u] events, then those; returns the chunk."""
    lens = np.diff(ac.offsets)
    dt = cache.kv.dtype
    for tail in (False, True):
        rows = split_rows(ac.offsets, counts, tail)
        j = chunk_of(H, counts if tail else [int(n - c) for n, c in zip(lens, counts)], ac.timestamps[rows])
        H.cache_reserve(cache, j, seq_ids=seq_ids)
        # K and V as column blocks of one buffer
        kv = torch.cat([tensor(ac.v[rows], dt, "cuda"), tensor(ac.k[rows], dt, "cuda")], 1)
        hv = ac.k.shape[1]
        H.cache_append(cache, layer, j, kv[:, hv:], kv[:, :hv], seq_ids=seq_ids)
    return j, rows


def attn_bound(q, k, v, s, a, vis, n, phi2, dtype, out16):
    """Element-wise bound of the kernel's error for one head, from the roundings
    it makes: S in fp32 (64-term dot: 64 * 2^-24 of sum |q k|, and the sums of S with
    its biases), phi2 (SiLU: h + h tanh(h), the hardware tanh within 2^-11 relative;
    2^x within 2^-22), P rounded to the operand type, fp32 accumulation over the
    keys, and the output's own rounding."""
    u = UNIT[dtype] if dtype != "fp32" else 0.0
    ds = 2.0 ** -17 * (np.abs(q) @ np.abs(k).T) + 2.0 ** -22 * np.abs(s)
    if phi2 == "softmax":
        # numerator and denominator each move by exp's relative error ds + 2^-22; P's
        # rounding, and below 2^-14 fp16's fixed step 2^-25 relative to the largest weight
        rel = 2.0 * (ds + 2.0 ** -21).max(axis=1, keepdims=True, where=vis, initial=0.0) + u
        err = a * rel + (2.0 ** -25 if dtype == "fp16" else 0.0)
    else:
        p = np.abs(a) * n
        act = 2.0 ** -11 * np.abs(s) / 2 if phi2 == "silu" and dtype != "fp32" else 2.0 ** -21 * p
        err = (1.2 * ds + act + u * p + (2.0 ** -25 if dtype == "fp16" else 0.0)) / n
    err = np.where(vis, err, 0.0)
    e = err @ np.abs(v) + 2.0 ** -24 * (8 + a.shape[1] / 16) * (np.abs(a) @ np.abs(v))
    # the output's rounding: half a step is out16 relative, and below fp16's least normal
    # number 2^-14, where the steps stay 2^-24 wide, 2^-25 absolute
    least = 2.0 ** -25 if dtype == "fp16" and out16 else 1e-30
    return 1.01 * e + np.maximum(out16 * np.abs(a @ v), least)


LENS = [(1, 1), (5, 5), (64, 1), (65, 1), (130, 2), (300, 17), (0, 0), (257, 40), (50, 0), (1000, 33), (128, 128)]


def run_attn(H, lens, heads, dtype, phi2, ps, window=0, sinks=0, Pb=64, Tb=64, gap="exp", seed=7, f32=False,
             release=False, kernel=None):
    counts = [c for _, c in lens]
    ac = make_attn_case([n for n, _ in lens], heads, Pb, Tb, seed=seed, dtype=dtype, gap_kind=gap)
    total = sum(-(-n // ps) for n, _ in lens)
    blocks = max(-(-n // ps) for n, _ in lens) + 1
    cache = nan_cache(H, layers=2, heads=heads, pages=total + 5, seqs=len(lens) + 2, blocks=blocks, ps=ps, dtype=dtype)
    perm = np.random.default_rng(seed).permutation(len(lens) + 2)[:len(lens)]
    seq = i32(perm)
    j, rows = load_cache(H, ac, cache, counts, layer=1, seq_ids=seq)
    if release:  # what a row at n or later does not see; rows of this chunk may see a little more
        keep = window + max(counts)
        H.cache_release(cache, seq, window=keep, sinks=sinks)
    cfg = H.LayerConfig(64 * heads, heads, Pb, Tb, phi2=phi2, dtype=dtype)
    q = tensor(ac.q[rows], DT[dtype], "cuda")
    fn = H.paged_attn_fwd_f32 if f32 else H.paged_attn_fwd
    rp, rt = tensor(ac.rab_pos, torch.float32, "cuda"), tensor(ac.rab_time, torch.float32, "cuda")
    wide = torch.cat([torch.full_like(q, float("nan")), q], 1)  # a row stride, NaN beside the rows
    args = (cfg, cache, 1, j, wide[:, heads * 64:], rp, rt, max(n for n, _ in lens))
    H.profiler_start()
    got = fn(*args, window=window, sinks=sinks, seq_ids=seq)
    ran = set(H.profiler_stop())
    assert kernel is None or ran == {"paged_attention_" + kernel}, ran
    again = fn(*args, window=window, sinks=sinks, seq_ids=seq)
    assert H.device_status() == 0
    assert torch.equal(got, again)  # the same bits
    got = got.float().cpu().numpy().astype(np.float64)
    at = 0
    for u, (n, c) in enumerate(lens):
        if c == 0:
            continue
        s = slice(int(ac.offsets[u]), int(ac.offsets[u + 1]))
        k, v, ts = ac.k[s].astype(np.float64), ac.v[s].astype(np.float64), ac.timestamps[s]
        qu = ac.q[s][n - c:].astype(np.float64)
        want, ss, aa = P.chunk_attention(qu, k, v, ts, ac.rab_pos.astype(np.float64),
                                         ac.rab_time.astype(np.float64), heads, phi2, window, sinks, parts=True)
        for h in range(heads):
            cols = slice(h * 64, h * 64 + 64)
            tol = attn_bound(qu[:, cols], k[:, cols], v[:, cols], ss[h], aa[h],
                             P.window_mask(n, c, window, sinks), n, phi2, dtype,
                             0.0 if f32 else UNIT[dtype])
            err = np.abs(got[at:at + c, cols] - want[:, cols])
            worst = np.nanmax(err / tol) if np.isfinite(err).all() else np.inf
            assert worst <= 1.0, (u, n, c, h, worst, err.max())
        at += c
    return cache


@pytest.mark.parametrize("ps", [16, 32, 64, 128])
@pytest.mark.parametrize("phi2", ["silu", "softmax"])
@pytest.mark.parametrize("dtype", ["fp16", "bf16", "fp32"])
def test_attention(H, dtype, phi2, ps):
    run_attn(H, LENS, 3, dtype, phi2, ps)


@pytest.mark.parametrize("phi2", ["relu", "identity"])
@pytest.mark.parametrize("dtype", ["fp16", "bf16", "fp32"])
def test_attention_other_phi(H, dtype, phi2):
    run_attn(H, LENS, 1, dtype, phi2, 32, gap="lognormal", Pb=1024, Tb=128)


@pytest.mark.parametrize("dtype,phi2", [("fp16", "silu"), ("bf16", "softmax"), ("fp32", "silu"), ("fp32", "softmax")])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (7, 3), (64, 0), (100, 70), (63, 200), (5000, 10)])
def test_attention_window(H, dtype, phi2, window, sinks):
    run_attn(H, LENS, 2, dtype, phi2, 16, window=window, sinks=sinks, Pb=512)


@pytest.mark.parametrize("dtype", ["fp16", "fp32"])
@pytest.mark.parametrize("window,sinks", [(30, 0), (30, 20), (100, 130)])
def test_attention_over_released_pages(H, dtype, window, sinks):
    """Pages that fell out of the window are gone; the rows read none of them."""
    lens = [(400, 3), (1000, 20), (77, 1), (640, 30), (129, 129)]
    cache = run_attn(H, lens, 2, dtype, "silu", 16, window=window, sinks=sinks, Pb=512, release=True)
    assert int((cache.block_table[:, :20] < 0).sum()) > 20


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_attention_f32_output(H, dtype):
    run_attn(H, [(300, 17), (90, 90), (1, 1)], 2, dtype, "silu", 64, f32=True)


def test_attention_one_row_of_many_lengths(H):
    """Single events over lengths around tile and split borders, in a batch and alone."""
    lens = [(n, 1) for n in (1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 511, 512, 513, 2000)]
    run_attn(H, lens, 2, "fp16", "silu", 64)
    for n in (1, 64, 1025, 4100):
        run_attn(H, [(n, 1)], 1, "fp16", "softmax", 16, Pb=4096)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("phi2", ["silu", "softmax"])
def test_attention_long_chunks(H, dtype, phi2):
    run_attn(H, [(700, 700), (1300, 300), (400, 1), (600, 257), (520, 65)], 6, dtype, phi2, 64, Pb=600, kernel="tile")


@pytest.mark.parametrize("ps", [16, 32, 128])
@pytest.mark.parametrize("phi2", ["silu", "relu", "identity", "softmax"])
def test_attention_tiles(H, phi2, ps):
    """The many-rows kernel: one query tile and two, ragged, short contexts, empty ones."""
    lens = [(128, 128), (129, 129), (256, 256), (257, 257), (300, 100), (64, 64), (0, 0), (63, 1), (700, 130), (90, 0),
            (400, 128), (333, 33), (1, 1)] * 2
    run_attn(H, lens, 8, "fp16", phi2, ps, kernel="rows" if phi2 == "softmax" else "tile")
    short = [(n, min(n, 120)) for n, _ in lens] * 3
    run_attn(H, short, 6, "bf16", phi2, ps, Pb=2000, Tb=128, gap="lognormal", kernel="tile")


@pytest.mark.parametrize("phi2", ["silu", "softmax"])
@pytest.mark.parametrize("new", [17, 40, 100])
def test_attention_rows_in_groups(H, phi2, new):
    """The few-rows kernel takes chunks of more than its 16 rows in groups."""
    run_attn(H, [(200, new), (333, new - 1), (130, 1)], 2, "fp16", phi2, 32, kernel="rows")


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("window,sinks", [(1, 0), (50, 10), (300, 129), (128, 64)])
def test_attention_long_chunks_window(H, dtype, window, sinks):
    run_attn(H, [(1500, 600), (1300, 300), (400, 1), (257, 257)], 6, dtype, "silu", 32, window=window,
             sinks=sinks, Pb=2048, gap="lognormal", kernel="tile")


def test_attention_tiles_over_released_pages(H):
    lens = [(1500, 100), (1300, 120), (400, 1), (700, 64)] * 6
    cache = run_attn(H, lens, 8, "fp16", "silu", 16, window=200, sinks=50, Pb=2048, release=True, kernel="tile")
    assert int((cache.block_table[:, :30] < 0).sum()) > 100


def test_far_offsets_in_a_large_cache(H):
    """Page addresses past 2^32 bytes (a cache of 5 GB)."""
    heads, ps = 4, 64
    pages = (5 << 30) // (2 * heads * ps * 64 * 2)
    cache = H.PagedCache.empty(1, heads, pages, 1, 8, ps, "fp16")
    cache.ref_count.fill_(1)
    cache.ref_count[-8:] = 0
    ac = make_attn_case([200], heads, 64, 64, seed=3, dtype="fp16")
    j, rows = load_cache(H, ac, cache, [9])
    assert int(cache.block_table[0, 0]) == pages - 8
    cfg = H.LayerConfig(64 * heads, heads, 64, 64, dtype="fp16")
    got = H.paged_attn_fwd_f32(cfg, cache, 0, j, tensor(ac.q[rows], torch.float16, "cuda"),
                               tensor(ac.rab_pos, torch.float32, "cuda"),
                               tensor(ac.rab_time, torch.float32, "cuda"), 200)
    kv, ts = H.cache_gather(cache, tensor(np.array([0, 200]), torch.int64, "cuda"), 200)
    assert H.device_status() == 0
    assert np.array_equal(kv[0, :, :256].float().cpu().numpy(), ac.k)
    assert np.array_equal(ts.cpu().numpy(), ac.timestamps)
    f = np.float64
    want = P.chunk_attention(ac.q[191:].astype(f), ac.k.astype(f), ac.v.astype(f), ac.timestamps,
                             ac.rab_pos.astype(f), ac.rab_time.astype(f), heads)
    assert_close(got.cpu().numpy(), want, "attention in a 5 GB cache")


# ---------------------------------------------------------------- rows and pages

def tables(cache):
    return cache.block_table.tolist(), cache.lengths.tolist(), cache.ref_count.tolist()


def same_pages(cache, pg):
    t, n, r = tables(cache)
    assert n == pg.len and r == pg.ref
    for row, want, ln in zip(t, pg.table, pg.len):
        assert row[:pg.blocks(ln)] == want[:pg.blocks(ln)]


@pytest.mark.parametrize("ps", [16, 128])
def test_pages_follow_the_oracle(H, ps):
    """A random life of a cache: every table, length and count equal after every
    call, and every event's rows and time found where the tables say, in all layers."""
    rng = np.random.default_rng(ps)
    heads, layers, seqs, blocks, pages = 2, 3, 7, 6, 25
    cache = nan_cache(H, layers=layers, heads=heads, pages=pages, seqs=seqs, blocks=blocks, ps=ps, dtype="fp16")
    pg = P.Pages(pages, seqs, blocks, ps)
    hold = [[] for _ in range(seqs)]  # (serial, time) of each sequence's events
    gone = [set() for _ in range(seqs)]
    serial = refused = 0

    def rows(ids, layer, which):
        x = np.asarray(ids, dtype=np.int64)[:, None] * 7 + 3 * layer + which + np.arange(heads * 64)[None, :]
        return (x % 1999).astype(np.float32)

    for step in range(120):
        op = rng.choice(["reserve", "reserve", "reserve", "fork", "release", "trim", "compact"])
        if op == "reserve":
            b = int(rng.integers(1, seqs + 1))
            ids = rng.permutation(seqs)[:b].tolist()
            cnt = [int(x) for x in rng.integers(0, 2 * ps, b)]
            new = [list(range(serial + sum(cnt[:i]), serial + sum(cnt[:i + 1]))) for i in range(b)]
            flat = [x for r in new for x in r]
            j = chunk_of(H, cnt, [10 * x + 1 for x in flat])
            ok = pg.reserve(ids, cnt) is not None
            H.cache_reserve(cache, j, seq_ids=i32(ids))
            assert H.device_status() == (0 if ok else 6)
            refused += not ok
            if ok and flat:
                serial += len(flat)
                for s, r in zip(ids, new):
                    hold[s] += r
                for l in range(layers):
                    H.cache_append(cache, l, j, tensor(rows(flat, l, 0), torch.float16, "cuda"),
                                   tensor(rows(flat, l, 1), torch.float16, "cuda"), seq_ids=i32(ids))
        elif op == "fork":
            full = [s for s in range(seqs) if pg.len[s]]
            empty = [s for s in range(seqs) if not pg.len[s]]
            if not full or not empty:
                continue
            src = [int(rng.choice(full)) for _ in empty]
            H.cache_fork(cache, i32(src), i32(empty))
            for a, d in zip(src, empty):
                pg.fork(a, d)
                hold[d], gone[d] = list(hold[a]), set(gone[a])
        elif op == "release":
            ids = [int(x) for x in rng.integers(0, seqs, 2)]
            H.cache_release(cache, i32(ids + ids[:1]))  # named twice: released once
            for s in set(ids):
                pg.release(s)
                hold[s], gone[s] = [], set()
        elif op == "trim":
            s, w, k = int(rng.integers(seqs)), int(rng.integers(1, 3 * ps)), int(rng.integers(0, 2 * ps))
            H.cache_release(cache, i32([s]), window=w, sinks=k)
            pg.release(s, w, k)
        else:
            live = H.cache_compact(cache)
            pg.compact()
            assert int(live) == sum(r > 0 for r in pg.ref)
        assert H.device_status() == 0
        same_pages(cache, pg)
        kv, ts = cache.kv.float().cpu().numpy(), cache.timestamps.cpu().numpy()
        for s in range(seqs):
            for b in range(pg.blocks(pg.len[s])):
                page = pg.table[s][b]
                if page < 0:
                    continue
                ids = hold[s][b * ps:(b + 1) * ps]
                m = len(ids)
                assert ts[page, :m].tolist() == [10 * x + 1 for x in ids]
                for l in range(layers):
                    for which in (0, 1):
                        got = kv[l, page, which, :, :m].transpose(1, 0, 2).reshape(m, heads * 64)
                        assert np.array_equal(got, rows(ids, l, which)), (step, op, s, b, l, which)
    assert refused > 0  # the pool ran out at least once, and nothing changed then


def test_gather_whole_sequences(H):
    lens = [0, 1, 100, 33, 257]
    for dtype in ("fp16", "bf16", "fp32"):
        ac = make_attn_case(lens, 3, 16, 16, seed=4, dtype=dtype)
        cache = nan_cache(H, layers=2, heads=3, pages=40, seqs=6, blocks=18, ps=16, dtype=dtype)
        for l in range(2):
            if l == 0:
                load_cache(H, ac, cache, [n // 2 for n in lens])
            else:
                j = chunk_of(H, lens, ac.timestamps)
                H.cache_append(cache, 1, j, tensor(ac.v, DT[dtype], "cuda"), tensor(ac.k, DT[dtype], "cuda"))
        ids = [4, 1, 4, 0, 2]
        off = np.concatenate([[0], np.cumsum([lens[i] for i in ids])]).astype(np.int64)
        kv, ts = H.cache_gather(cache, tensor(off, torch.int64, "cuda"), int(off[-1]), seq_ids=i32(ids))
        assert H.device_status() == 0
        rows = np.concatenate([np.arange(ac.offsets[i], ac.offsets[i + 1]) for i in ids])
        assert np.array_equal(ts.cpu().numpy(), ac.timestamps[rows])
        kv = kv.float().cpu().numpy()
        assert np.array_equal(kv[0], np.concatenate([ac.k[rows], ac.v[rows]], 1))
        assert np.array_equal(kv[1], np.concatenate([ac.v[rows], ac.k[rows]], 1))


def test_reports_instead_of_writing(H):
    """Wrong sequences, missing pages, shared pages and wrong lengths are reported
    and leave everything as it was."""
    ac = make_attn_case([40, 20], 1, 16, 16, seed=5, dtype="fp16")
    cache = nan_cache(H, layers=1, heads=1, pages=12, seqs=4, blocks=4, ps=16, dtype="fp16")
    j, rows = load_cache(H, ac, cache, [3, 2])
    x = tensor(ac.k[rows], torch.float16, "cuda")

    def unchanged(call):
        before = [t.clone() for t in (cache.kv, cache.timestamps, *map(torch.tensor, tables(cache)))]
        call()
        assert H.device_status() == 6
        after = (cache.kv, cache.timestamps, *map(torch.tensor, tables(cache)))
        for a, b in zip(before, after):
            assert torch.equal(torch.nan_to_num(a), torch.nan_to_num(b))

    for ids in ([1, 1], [0, 4], [-1, 0]):  # twice, past the end, negative
        unchanged(lambda: H.cache_reserve(cache, j, seq_ids=i32(ids)))
    unchanged(lambda: H.cache_reserve(cache, chunk_of(H, [30, 1], [0] * 31)))     # block table too short
    unchanged(lambda: H.cache_append(cache, 0, j, x, x, seq_ids=i32([-1, 9])))
    unchanged(lambda: H.cache_append(cache, 0, chunk_of(H, [0, 21], [0] * 21),
                                     x[:1].expand(21, 64).contiguous(), x[:1].expand(21, 64).contiguous()))
    unchanged(lambda: H.cache_fork(cache, i32([0]), i32([1])))                       # not empty
    unchanged(lambda: H.cache_fork(cache, i32([0]), i32([0])))
    unchanged(lambda: H.cache_fork(cache, i32([7]), i32([2])))
    unchanged(lambda: H.cache_release(cache, i32([17])))
    # a fork shares its pages: they are not written
    H.cache_fork(cache, i32([0]), i32([2]))
    assert H.device_status() == 0
    unchanged(lambda: H.cache_append(cache, 0, chunk_of(H, [3], [0] * 3), x[:3], x[:3]))
    # attention: a visible page that is missing, a context longer than declared
    cfg = H.LayerConfig(64, 1, 16, 16, dtype="fp16")
    rp = torch.zeros((1, 16), device="cuda")

    def attn(ctx=40, **kw):
        return H.paged_attn_fwd(cfg, cache, 0, j, x, rp, rp, ctx, **kw)

    attn()
    assert H.device_status() == 0
    unchanged(lambda: attn(ctx=39))
    unchanged(lambda: attn(seq_ids=i32([0, 4])))
    page = int(cache.block_table[0, 0])
    for bad in (-1, 12, 1 << 30):
        cache.block_table[0, 0] = bad
        unchanged(attn)
        attn(window=8)  # out of the window: not looked at
        assert H.device_status() == 0
    cache.block_table[0, 0] = page


def test_reserve_many_sequences(H):
    """More sequences than one pass of the bookkeeping kernel takes (1024), in a
    pool larger than one scan (4096 pages)."""
    n = 2500
    cache = H.PagedCache.empty(1, 1, 9000, n, 5, 16, "fp16")
    pg = P.Pages(9000, n, 5, 16)
    rng = np.random.default_rng(1)
    for _ in range(2):
        cnt = [int(x) for x in rng.integers(0, 40, n)]
        H.cache_reserve(cache, chunk_of(H, cnt, range(sum(cnt))))
        pg.reserve(list(range(n)), cnt)
        assert H.device_status() == 0
        same_pages(cache, pg)
    gone = [int(x) for x in rng.permutation(n)[:1200]]
    H.cache_release(cache, i32(gone))
    for s in gone:
        pg.release(s)
    H.cache_compact(cache)
    pg.compact()
    same_pages(cache, pg)


# ---------------------------------------------------------------- together

@pytest.mark.parametrize("name,kw", [("tiny-fp32", {}), ("small-bf16", {}), ("small-bf16", dict(window=40, sinks=9)),
                                     ("small-bf16", dict(phi2="softmax"))])
def test_extend_follows_the_oracle(H, name, kw):
    """Histories in several requests through a stack, against the incremental oracle."""
    kw = dict(kw)
    phi2 = kw.pop("phi2", "silu")
    lens = [130, 64, 1, 47]
    case = make_case(make_case(name).cfg.replace(phi2=phi2, num_layers=2), seed=11, lengths=lens)
    cfg = config_of(H, case.cfg)
    t = case_tensors(case, "cuda")
    weights = [H.LayerWeights(**lw) for lw in t["layers"]]
    cache = nan_cache(H, layers=2, heads=case.cfg.num_heads, pages=40, seqs=4, blocks=9, ps=16,
                      dtype="fp32" if name == "tiny-fp32" else "fp16")
    cuts = [[0, 100, 101, 130], [0, 10, 63, 64], [0, 0, 1, 1], [0, 30, 30, 47]]
    state = [None] * 4
    for step in range(3):
        rows = np.concatenate([case.offsets[u] + np.arange(cuts[u][step], cuts[u][step + 1]) for u in range(4)])
        cnt = [cuts[u][step + 1] - cuts[u][step] for u in range(4)]
        j = chunk_of(H, cnt, case.timestamps[rows])
        y = H.extend(cfg, weights, cache, j, t["x"][torch.from_numpy(rows).cuda()].contiguous(), 130, **kw)
        if kw:
            H.cache_release(cache, i32(range(4)), **kw)
        assert H.device_status() == 0
        want = []
        for u in range(4):
            a, b = case.offsets[u] + cuts[u][step], case.offsets[u] + cuts[u][step + 1]
            if b > a:
                w, state[u] = P.extend(state[u], case.x[a:b], case.timestamps[a:b], case.layers, case.cfg, **kw)
                want.append(w)
        assert_close(y.cpu().numpy(), np.concatenate(want), f"extend {name} {phi2} {kw} step {step}")


def test_extend_with_long_chunks(H):
    """Fresh histories through the stack on the many-rows kernel (and its LayerNorm
    partial sums): the rows of hstu_forward, up to the roundings of both."""
    case = make_case("small-bf16", seed=15, lengths=[300, 129, 512, 257, 400, 64] * 3)
    cfg = config_of(H, case.cfg)
    t = case_tensors(case, "cuda")
    weights = [H.LayerWeights(**lw) for lw in t["layers"]]
    jag = H.Jagged(t["offsets"], t["timestamps"], case.max_len, case.total_tokens)
    cache = nan_cache(H, layers=case.cfg.num_layers, heads=4, pages=200, seqs=18, blocks=9, ps=64, dtype="fp16")
    H.profiler_start()
    y = H.extend(cfg, weights, cache, jag, t["x"], 512)
    assert "paged_attention_tile" in H.profiler_stop()
    assert H.device_status() == 0
    dense = torch.empty((case.cfg.num_layers, case.total_tokens, 512), dtype=torch.float16, device="cuda")
    z = H.forward(cfg, weights, jag, t["x"], kv_cache_out=dense)
    assert_close(y.cpu().numpy(), z.cpu().numpy(), "extend from nothing against forward")
    kv, _ = H.cache_gather(cache, t["offsets"], case.total_tokens)
    assert torch.equal(kv[0], dense[0])
    want, _ = O.forward(case.x, case.offsets, case.timestamps, case.layers, case.cfg)
    assert_close(y.cpu().numpy(), want, "extend from nothing against the oracle")


def test_serving_round(H):
    """A request as a server makes it: encode a history, keep it in pages, branch
    it, extend the branches, score candidates over one of them; every part
    against the same through the dense calls."""
    case = make_case(make_case("mfalcon").cfg.replace(num_layers=2, num_cand=24, d_model=256, num_heads=4),
                     seed=12, lengths=[120, 75])
    cfg = config_of(H, case.cfg)
    t = case_tensors(case, "cuda")
    jag = H.Jagged(t["offsets"], t["timestamps"], case.max_len, case.total_tokens)
    weights = [H.LayerWeights(**lw) for lw in t["layers"]]
    hv = 256
    dense = torch.empty((2, case.total_tokens, 2 * hv), dtype=torch.float16, device="cuda")
    H.forward(cfg, weights, jag, t["x"], kv_cache_out=dense)
    cache = nan_cache(H, layers=2, heads=4, pages=30, seqs=6, blocks=12, ps=16, dtype="fp16")
    H.cache_reserve(cache, jag)
    for l in range(2):
        H.cache_append(cache, l, jag, dense[l, :, :hv], dense[l, :, hv:])
    kv, ts = H.cache_gather(cache, t["offsets"], case.total_tokens)
    assert torch.equal(kv, dense) and torch.equal(ts, t["timestamps"])
    args = (t["cand_offsets"], t["cand_emb"], t["request_ts"], 8, 24)
    assert torch.equal(H.mfalcon_score(cfg, weights, jag, kv, *args), H.mfalcon_score(cfg, weights, jag, dense, *args))
    # two branches of user 0: the same events give the same rows, other events leave them alone
    H.cache_fork(cache, i32([0, 0]), i32([2, 3]))
    x_new = t["x"][:6].contiguous()
    last = int(case.timestamps[119])
    j = chunk_of(H, [3, 3], [last + 1 + i for i in range(3)] * 2)
    y = H.extend(cfg, weights, cache, j, torch.cat([x_new[:3], x_new[:3]]), 200, seq_ids=i32([2, 3]))
    assert H.device_status() == 0
    assert torch.equal(y[:3], y[3:])
    kv2, _ = H.cache_gather(cache, t["offsets"], case.total_tokens)
    assert torch.equal(kv2, dense)  # the parent is as it was
    H.cache_release(cache, i32([2, 3]))
    H.cache_compact(cache)
    kv2, _ = H.cache_gather(cache, t["offsets"], case.total_tokens)
    assert torch.equal(kv2, dense) and H.device_status() == 0
    # the same extension without the branch, and against the incremental oracle's dense rows
    y2 = H.extend(cfg, weights, cache, chunk_of(H, [3], [last + 1 + i for i in range(3)]), x_new[:3], 200,
                  seq_ids=i32([0]))
    assert_close(y2.cpu().numpy(), y[:3].cpu().numpy(), "extension of a user and of its branch")


def test_refused_extension_leaves_the_cache(H):
    case = make_case("small-bf16", seed=13, lengths=[60])
    cfg = config_of(H, case.cfg)
    t = case_tensors(case, "cuda")
    weights = [H.LayerWeights(**lw) for lw in t["layers"]]
    cache = nan_cache(H, layers=case.cfg.num_layers, heads=case.cfg.num_heads, pages=4, seqs=1, blocks=9, ps=16,
                      dtype="fp16")
    H.extend(cfg, weights, cache, chunk_of(H, [50], case.timestamps[:50]), t["x"][:50], 60)
    assert H.device_status() == 0
    kv, ts = cache.kv.clone(), cache.timestamps.clone()
    H.extend(cfg, weights, cache, chunk_of(H, [60], range(60)), t["x"], 200)
    assert H.device_status() == 6
    assert torch.equal(torch.nan_to_num(kv), torch.nan_to_num(cache.kv)) and torch.equal(ts, cache.timestamps)
    assert cache.lengths.tolist() == [50]


def test_captured_and_on_another_stream(H):
    """Two graphs with their own workspaces, replayed in turn on a side stream."""
    ac = make_attn_case([300, 200], 2, 64, 64, seed=8, dtype="fp16")
    cache = nan_cache(H, layers=1, heads=2, pages=40, seqs=2, blocks=24, ps=16, dtype="fp16")
    j, rows = load_cache(H, ac, cache, [5, 70])
    cfg = H.LayerConfig(128, 2, 64, 64, dtype="fp16")
    rp, rt = tensor(ac.rab_pos, torch.float32, "cuda"), tensor(ac.rab_time, torch.float32, "cuda")
    q = tensor(ac.q[rows], torch.float16, "cuda")
    k, v = tensor(ac.k[rows], torch.float16, "cuda"), tensor(ac.v[rows], torch.float16, "cuda")
    want = H.paged_attn_fwd(cfg, cache, 0, j, q, rp, rt, 300)
    want_w = H.paged_attn_fwd(cfg, cache, 0, j, q, rp, rt, 300, window=20, sinks=3)
    out, out_w = torch.zeros_like(want), torch.zeros_like(want)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graphs = []
    for o, kw in ((out, {}), (out_w, dict(window=20, sinks=3))):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            H.cache_append(cache, 0, j, k, v)
            H.paged_attn_fwd(cfg, cache, 0, j, q, rp, rt, 300, av_out=o, **kw)
        graphs.append(g)
    for _ in range(3):
        out.zero_()
        out_w.zero_()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            for g in graphs:
                g.replay()
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(out, want) and torch.equal(out_w, want_w)
    assert H.device_status() == 0


def test_extend_captured_and_replayed(H):
    """One captured extension, replayed: every replay appends the next events."""
    case = make_case("small-bf16", seed=14, lengths=[60, 33])
    cfg = config_of(H, case.cfg)
    t = case_tensors(case, "cuda")
    weights = [H.LayerWeights(**lw) for lw in t["layers"]]
    mk = dict(layers=case.cfg.num_layers, heads=case.cfg.num_heads, pages=30, seqs=2, blocks=9, ps=16, dtype="fp16")
    eager, graphed = nan_cache(H, **mk), nan_cache(H, **mk)
    first = chunk_of(H, [60, 33], case.timestamps)
    later = int(max(case.timestamps)) + 100
    x = t["x"][:5].contiguous()
    ts = [torch.tensor([later + 10 * k + i for i in range(5)], dtype=torch.int64, device="cuda") for k in range(3)]
    want = []
    H.extend(cfg, weights, eager, first, t["x"], 100)
    for k in range(3):
        want.append(H.extend(cfg, weights, eager, H.Jagged(chunk_of(H, [3, 2], ts[k].tolist()).offsets, ts[k], 3, 5), x, 100))
    H.extend(cfg, weights, graphed, first, t["x"], 100)
    buf = ts[0].clone()
    j = H.Jagged(chunk_of(H, [3, 2], [0] * 5).offsets, buf, 3, 5)
    y = torch.empty_like(want[0])
    ws = torch.empty(H.extend_workspace_bytes(cfg, graphed, 2, 5), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        H.extend(cfg, weights, graphed, j, x, 100, y_out=y, workspace=ws)
    for k in range(3):
        buf.copy_(ts[k])
        g.replay()
        assert torch.equal(y, want[k]), k
    assert H.device_status() == 0
    assert tables(eager) == tables(graphed) and graphed.lengths.tolist() == [69, 39]


def test_two_streams_read_one_cache(H):
    ac = make_attn_case([900, 400, 77], 4, 64, 64, seed=9, dtype="bf16")
    cache = nan_cache(H, layers=1, heads=4, pages=50, seqs=3, blocks=16, ps=64, dtype="bf16")
    j, rows = load_cache(H, ac, cache, [200, 1, 30])
    cfg = H.LayerConfig(256, 4, 64, 64, dtype="bf16")
    rp, rt = tensor(ac.rab_pos, torch.float32, "cuda"), tensor(ac.rab_time, torch.float32, "cuda")
    q = tensor(ac.q[rows], torch.bfloat16, "cuda")
    kw = [{}, dict(window=50, sinks=5)]
    want = [H.paged_attn_fwd(cfg, cache, 0, j, q, rp, rt, 900, **k) for k in kw]
    out = [torch.zeros_like(want[0]) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for st, o, k in zip(streams, out, kw):
            H.paged_attn_fwd(cfg, cache, 0, j, q, rp, rt, 900, av_out=o, stream=st, **k)
    torch.cuda.synchronize()
    assert H.device_status() == 0
    assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])


def test_many_heads_and_wide_spans(H):
    """16 heads, one position bucket, and times at the largest span the kernels take."""
    run_attn(H, [(130, 1), (70, 9), (300, 60)], 16, "fp16", "silu", 16, Pb=1, Tb=256)
    for dtype, c in (("fp16", 3), ("fp16", 200), ("fp32", 3)):
        ac = make_attn_case([250], 1, 16, 128, seed=2, dtype=dtype)
        for span, want_status in ((2 ** 31 - 4, 0), (2 ** 31 + 5, 6)):
            ac.timestamps[:] = 1_700_000_000 + span
            ac.timestamps[0] = 1_700_000_000
            cache = nan_cache(H, layers=1, heads=1, pages=20, seqs=1, blocks=16, ps=16, dtype=dtype)
            j, rows = load_cache(H, ac, cache, [c])
            cfg = H.LayerConfig(64, 1, 16, 128, dtype=dtype)
            got = H.paged_attn_fwd(cfg, cache, 0, j, tensor(ac.q[rows], DT[dtype], "cuda"),
                                   tensor(ac.rab_pos, torch.float32, "cuda"),
                                   tensor(ac.rab_time, torch.float32, "cuda"), 250)
            assert H.device_status() == want_status, (dtype, c, span)
            if want_status == 0:
                f = np.float64
                want = P.chunk_attention(ac.q[250 - c:].astype(f), ac.k.astype(f), ac.v.astype(f), ac.timestamps,
                                         ac.rab_pos.astype(f), ac.rab_time.astype(f), 1)
                assert_close(got.float().cpu().numpy(), want, f"span {span} {dtype}", scaled=True)


def test_default_memory_on_side_streams(H, monkeypatch):
    """Two caches that reserve, extend, gather and compact on two streams at once, with
    workspaces and results of the calls' own making: all of it from the calls' streams, and
    the results of the same calls made one after the other."""
    case = make_case("small-bf16", seed=21, lengths=[90, 40])
    cfg = config_of(H, case.cfg)
    t = case_tensors(case, "cuda")
    weights = [H.LayerWeights(**lw) for lw in t["layers"]]
    jag = H.Jagged(t["offsets"], t["timestamps"], case.max_len, case.total_tokens)
    later = int(max(case.timestamps)) + 10
    more = [chunk_of(H, [k + 1, 3], [later + 5 * k + i for i in range(k + 1)] + [later + 5 * k + i for i in range(3)])
            for k in range(4)]
    # caches start with a sequence that is released, so that compact has pages to move
    mk = dict(layers=case.cfg.num_layers, heads=case.cfg.num_heads, pages=40, seqs=3, blocks=9, ps=16, dtype="fp16")
    first = chunk_of(H, [33], range(33))
    total = case.total_tokens + sum(m.total_tokens for m in more)
    ends = [int(n) + sum(int(m.offsets[u + 1] - m.offsets[u]) for m in more) for u, n in enumerate((90, 40))]
    off = tensor(np.array([0, ends[0], ends[0] + ends[1]]), torch.int64, "cuda")

    def life(cache, stream):
        out = []
        H.cache_reserve(cache, first, seq_ids=two, stream=stream)
        for l in range(case.cfg.num_layers):
            H.cache_append(cache, l, first, zeros, zeros, seq_ids=two, stream=stream)
        out.append(H.extend(cfg, weights, cache, jag, t["x"], 200, stream=stream))
        H.cache_release(cache, two, stream=stream)
        for m in more:
            out.append(H.extend(cfg, weights, cache, m, t["x"][:m.total_tokens].contiguous(), 200, stream=stream))
        out.append(H.cache_compact(cache, stream=stream))
        out += H.cache_gather(cache, off, total, stream=stream)
        return out

    two = i32([2])
    zeros = torch.zeros((33, case.cfg.num_heads * 64), dtype=torch.float16, device="cuda")
    want = life(nan_cache(H, **mk), None)
    caches, streams = [nan_cache(H, **mk) for _ in range(2)], [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    made, empty = [], torch.empty

    def watched(*a, **kw):
        made.append(torch.cuda.current_stream())
        return empty(*a, **kw)

    for _ in range(3):
        got = []
        for c, s in zip(caches, streams):
            s.wait_stream(torch.cuda.current_stream())
            del made[:]
            monkeypatch.setattr(torch, "empty", watched)
            got.append(life(c, s))
            monkeypatch.setattr(torch, "empty", empty)
            assert len(made) >= 13 and all(m == s for m in made)
        torch.cuda.synchronize()
        assert H.device_status() == 0
        for g in got:
            assert len(g) == len(want)
            for a, b in zip(g, want):
                assert torch.equal(a, b)
        for c in caches:
            H.cache_release(c, i32(range(3)))


def test_tensors_elsewhere_are_refused(H):
    """Tensors of the call that are not on the cache's GPU, and parts of a cache that are not."""
    ac = make_attn_case([40, 20], 1, 16, 16, seed=5, dtype="fp16")
    cache = nan_cache(H, layers=1, heads=1, pages=12, seqs=4, blocks=4, ps=16, dtype="fp16")
    j, rows = load_cache(H, ac, cache, [3, 2])
    x = tensor(ac.k[rows], torch.float16, "cuda")
    rp = torch.zeros((1, 16), device="cuda")
    cfg = H.LayerConfig(64, 1, 16, 16, dtype="fp16")
    ids = i32([0, 1])
    off = tensor(np.array([0, 40, 60]), torch.int64, "cuda")
    far = H.Jagged(j.offsets.cpu(), j.timestamps, j.max_len, j.total_tokens)
    old = H.Jagged(j.offsets, j.timestamps.cpu(), j.max_len, j.total_tokens)
    ws = torch.empty(1 << 16, dtype=torch.uint8)

    def attn(q=x, rp=rp, rt=rp, chunk=j, **kw):
        return H.paged_attn_fwd(cfg, cache, 0, chunk, q, rp, rt, 40, **kw)

    for f in (lambda: H.cache_append(cache, 0, j, x.cpu(), x), lambda: H.cache_append(cache, 0, j, x, x.cpu()),
              lambda: H.cache_append(cache, 0, far, x, x), lambda: H.cache_append(cache, 0, j, x, x, seq_ids=ids.cpu()),
              lambda: H.cache_reserve(cache, far), lambda: H.cache_reserve(cache, old),
              lambda: H.cache_reserve(cache, j, seq_ids=ids.cpu()), lambda: H.cache_reserve(cache, j, workspace=ws),
              lambda: H.cache_compact(cache, workspace=ws), lambda: H.cache_gather(cache, off.cpu(), 60),
              lambda: H.cache_gather(cache, off, 60, kv_out=torch.empty(1, 60, 128, dtype=torch.float16)),
              lambda: H.cache_fork(cache, ids.cpu(), i32([2, 3])), lambda: H.cache_fork(cache, ids, i32([2, 3]).cpu()),
              lambda: H.cache_release(cache, ids.cpu()), lambda: attn(q=x.cpu()), lambda: attn(rp=rp.cpu()),
              lambda: attn(rt=rp.cpu()), lambda: attn(chunk=far), lambda: attn(chunk=old), lambda: attn(seq_ids=ids.cpu()),
              lambda: attn(av_out=torch.empty_like(x, device="cpu"))):
        with pytest.raises(ValueError, match="not on the cache's GPU"):
            f()
    for n in range(5):
        parts = list(cache[:5])
        parts[n] = parts[n].cpu()
        with pytest.raises(ValueError, match="on one device"):
            H.PagedCache(*parts)
    assert H.device_status() == 0 and cache.lengths.tolist() == [40, 20, 0, 0]


@pytest.mark.parametrize("ps", [16, 128])
def test_lengths_that_no_table_holds(H, ps):
    """Lengths at the top of their type: reported, nothing read past the block table."""
    cache = nan_cache(H, layers=1, heads=1, pages=12, seqs=4, blocks=4, ps=ps, dtype="fp16")
    H.cache_reserve(cache, chunk_of(H, [20, 20], range(40)))
    x = torch.zeros((3, 64), dtype=torch.float16, device="cuda")
    j, one = chunk_of(H, [3], range(3)), i32([0])
    off = tensor(np.array([0, 3]), torch.int64, "cuda")
    down = tensor(np.array([3, 2]), torch.int64, "cuda")
    cfg = H.LayerConfig(64, 1, 16, 16, dtype="fp16")
    rp = torch.zeros((1, 16), device="cuda")
    for n in (2 ** 31 - 1, 2 ** 31 - ps, 2 ** 31 - ps - 1, 4 * ps + 1):
        cache.lengths[0] = n
        before = [t.clone() for t in cache[:5]]
        for call in (lambda: H.cache_append(cache, 0, j, x, x), lambda: H.cache_gather(cache, off, 3),
                     lambda: H.cache_fork(cache, one, i32([2])), lambda: H.cache_release(cache, one),
                     lambda: H.cache_release(cache, one, window=7), lambda: H.cache_reserve(cache, j),
                     lambda: H.cache_gather(cache, down, 3, seq_ids=i32([-1])),
                     lambda: H.paged_attn_fwd(cfg, cache, 0, j, x, rp, rp, 2 ** 31 - 1)):
            call()
            assert H.device_status() == 6, n
            for a, b in zip(before, cache[:5]):
                assert torch.equal(torch.nan_to_num(a), torch.nan_to_num(b))


def unchanged_by(cache, H, call):
    """The call is reported and leaves the cache as it was."""
    before = [t.clone() for t in cache[:5]]
    call()
    assert H.device_status() == 6
    for a, b in zip(before, cache[:5]):
        assert torch.equal(torch.nan_to_num(a), torch.nan_to_num(b))


@pytest.mark.parametrize("name", ["small-bf16", "tiny-fp32"])
def test_extend_refuses_before_it_changes_anything(H, name):
    """What the attention of an extension would run into is refused with the reservation."""
    case = make_case(make_case(name).cfg.replace(num_layers=2), seed=22, lengths=[70, 41])
    cfg = config_of(H, case.cfg)
    t = case_tensors(case, "cuda")
    weights = [H.LayerWeights(**lw) for lw in t["layers"]]
    cache = nan_cache(H, layers=2, heads=case.cfg.num_heads, pages=24, seqs=3, blocks=9, ps=16,
                      dtype="fp32" if name == "tiny-fp32" else "fp16")
    H.extend(cfg, weights, cache, H.Jagged(t["offsets"], t["timestamps"], 70, 111), t["x"], 70)
    assert H.device_status() == 0
    start = [int(case.timestamps[u]) for u in (0, 70)]
    last = int(max(case.timestamps)) + 5
    x = t["x"][:7].contiguous()

    def ext(ts=None, ctx=75, cnt=(5, 2), **kw):
        ts = [last + i for i in range(sum(cnt))] if ts is None else ts
        return H.extend(cfg, weights, cache, chunk_of(H, cnt, ts), x[:sum(cnt)], ctx, **kw)

    unchanged_by(cache, H, lambda: ext(ctx=74))              # user 0 would have 75 events
    unchanged_by(cache, H, lambda: ext(ctx=1))
    # a visible event just too long ago, of either user; at the border it is taken (below)
    far = start[0] + 2 ** 31 - 2
    unchanged_by(cache, H, lambda: ext([far - 4 + i for i in range(5)] + [last, last + 1]))
    far = start[1] + 2 ** 31 - 2
    unchanged_by(cache, H, lambda: ext([last + i for i in range(5)] + [far - 1, far]))
    # pages that fell out of a window of 20 with 17 sinks: user 0 keeps blocks 0, 1 and 3, 4
    H.cache_release(cache, i32([0]), window=20, sinks=17)
    assert H.device_status() == 0 and (cache.block_table[0, :5] >= 0).tolist() == [True, True, False, True, True]
    unchanged_by(cache, H, ext)
    unchanged_by(cache, H, lambda: ext(window=24))           # the first new row sees event 47
    unchanged_by(cache, H, lambda: ext(window=20, sinks=33))  # and event 32
    unchanged_by(cache, H, lambda: ext(window=20, sinks=17, ctx=74))
    ext(window=23, sinks=32)                                 # events 48 .., and 0 .. 31
    assert H.device_status() == 0 and cache.lengths.tolist() == [75, 43, 0]
    # out of the window it does not matter how long ago an event was
    far = start[1] + 2 ** 31 - 3
    ext([far], cnt=(0, 1), ctx=200)
    assert H.device_status() == 0 and cache.lengths.tolist() == [75, 44, 0]
    unchanged_by(cache, H, lambda: ext([far + 1], cnt=(0, 1), ctx=200))
    ext([far + 1], cnt=(0, 1), ctx=200, window=1)
    ext([far + 2 ** 33], cnt=(0, 1), ctx=200, window=1)
    assert H.device_status() == 0 and cache.lengths.tolist() == [75, 46, 0]


def test_extend_refuses_what_its_attention_would_report(H):
    """Many sequences of many pages, some of them missing here and there: the extension's verdict
    is that of the attention alone over a copy of the cache."""
    rng = np.random.default_rng(23)
    heads, users, ps, blocks = 1, 70, 16, 90
    dev = dict(device="cuda", dtype=torch.float32)
    cfg = H.LayerConfig(64, heads, 32, 32, dtype="fp32")
    weights = [H.LayerWeights(0.05 * torch.randn(256, 64, **dev), torch.zeros(256, **dev), 0.05 * torch.randn(64, 64, **dev),
                              torch.zeros(64, **dev), torch.zeros(1, 32, **dev), torch.zeros(1, 32, **dev))]
    verdicts = []
    for trial in range(24):
        n = [int(v) for v in rng.integers(0, blocks * ps - 40, users)]
        cnt = [int(v) for v in rng.integers(0, 4, users)]
        caches = [nan_cache(H, layers=1, heads=heads, pages=8000, seqs=users, blocks=blocks, ps=ps, dtype="fp32")
                  for _ in range(2)]
        window, sinks = (0, 0) if trial % 4 == 0 else (int(rng.integers(1, 300)), int(rng.integers(0, 100)))
        first = chunk_of(H, n, np.concatenate([np.arange(v) for v in n]))
        j = chunk_of(H, cnt, np.concatenate([v + np.arange(c) for v, c in zip(n, cnt)]))
        x = torch.randn(j.total_tokens, 64, **dev)
        drop = rng.random((users, blocks)) < (0.0 if trial % 3 == 2 else 0.0007)
        gone = torch.from_numpy(drop).cuda()
        for c in caches:
            c.kv.zero_()
            H.cache_reserve(c, first)
            if trial % 3:  # what fell out of the window goes
                H.cache_release(c, i32(range(users)), window=max(window, 1), sinks=sinks)
            # a page that another sequence's block is in could not be missing: whole pages, last ones not
            last = torch.tensor([max(0, -(-v // ps) - 1) for v in n], device="cuda")
            hole = gone & (torch.arange(blocks, device="cuda")[None, :] < last[:, None])
            c.block_table[hole] = -1
        assert H.device_status() == 0
        ctx = max(a + b for a, b in zip(n, cnt))
        H.cache_reserve(caches[1], j)
        assert H.device_status() == 0
        H.paged_attn_fwd(cfg, caches[1], 0, j, x, weights[0].rab_pos, weights[0].rab_time, ctx, window=window, sinks=sinks)
        want = H.device_status()
        if want:
            unchanged_by(caches[0], H, lambda: H.extend(cfg, weights, caches[0], j, x, ctx, window=window, sinks=sinks))
        else:
            H.extend(cfg, weights, caches[0], j, x, ctx, window=window, sinks=sinks)
            assert H.device_status() == 0
            assert caches[0].lengths.tolist() == [a + b for a, b in zip(n, cnt)]
        verdicts.append(want)
    assert 6 <= verdicts.count(6) <= 18, verdicts


def test_extend_too_large_to_launch(H):
    """A grid past the launch limit: an error of the call, with no event reserved."""
    heads, users = 128, 65535
    dev = dict(device="cuda")
    cfg = H.LayerConfig(64, heads, 16, 16)
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, **dev)  # noqa: E731
    f = lambda *s: torch.zeros(*s, dtype=torch.float32, **dev)  # noqa: E731
    w = [H.LayerWeights(z(4 * heads * 64, 64), f(4 * heads * 64), z(64, heads * 64), f(64), f(heads, 16), f(heads, 16))]
    cache = H.PagedCache.empty(1, heads, 4, users, 64, 128, "fp16")
    counts = [0] * users
    counts[7] = 1
    j = chunk_of(H, counts, [5])
    x = z(1, 64)
    wide = H.Jagged(j.offsets, j.timestamps, 8192, 1)  # up to 8192 events each
    with pytest.raises(H.HSTUError) as e:
        H.extend(cfg, w, cache, wide, x, 8192)
    assert e.value.status == 2 and H.device_status() == 0
    assert int(cache.lengths.sum()) == 0 and int(cache.ref_count.sum()) == 0 and bool((cache.block_table == -1).all())
    H.extend(cfg, w, cache, j, x, 8192)
    assert H.device_status() == 0 and int(cache.lengths[7]) == 1 and int(cache.lengths.sum()) == 1


@pytest.mark.parametrize("count", [2, 40, 1000])
def test_fork_does_not_depend_on_the_order_of_blocks(H, count):
    """Sources that are destinations too, and destinations named twice, in one call: the same
    forks are made and reported every time."""
    def fresh():
        cache = nan_cache(H, layers=1, heads=1, pages=40, seqs=count + 4, blocks=4, ps=16, dtype="fp16")
        H.cache_reserve(cache, chunk_of(H, [20], range(20)), seq_ids=i32([0]))
        return cache

    def after(cache, src, dst):
        H.cache_fork(cache, i32(src), i32(dst))
        return H.device_status()

    for _ in range(5):
        # a chain 0 -> 1 -> 2 ..: only the first is from no destination
        cache = fresh()
        assert after(cache, range(count), range(1, count + 1)) == 6
        assert cache.lengths.tolist() == [20, 20] + [0] * (count + 2)
        assert cache.ref_count.tolist()[:2] == [2, 2] and int((cache.block_table >= 0).sum()) == 4
        # a ring of empty sequences
        assert after(cache, [3, 2], [2, 3]) == 6
        # two sources, one of them empty, for one destination: the first is made
        for src, want in (([0, 3], 20), ([3, 0], 0)):
            cache = fresh()
            assert after(cache, src, [1, 1]) == 6
            assert cache.lengths.tolist() == [20, want] + [0] * (count + 2)
            assert cache.ref_count.tolist()[:2] == [1 + (want > 0)] * 2
        cache = fresh()
        assert after(cache, [2, 3], [1, 1]) == 6   # two empty sources
        # and what is allowed: one source, every other sequence, empty sources too
        cache = fresh()
        assert after(cache, [0] * (count + 2), range(1, count + 3)) == 0
        assert cache.lengths.tolist() == [20] * (count + 3) + [0]
        assert cache.ref_count.tolist()[:2] == [count + 3] * 2
        assert after(cache, [count + 3], [count + 3]) == 6
        H.cache_release(cache, i32([1, 2]))
        assert after(cache, [1], [2]) == 0
        assert after(cache, [1], [0]) == 6          # an empty source, a destination that is not


@pytest.mark.parametrize("dtype,heads,lens,kernel", [
    ("fp32", 2, [(40, 3), (700, 20)], "fp32"), ("fp16", 2, [(40, 3), (700, 16)], "rows"),
    ("bf16", 8, [(300, 120), (700, 128)] * 6, "rows"), ("bf16", 8, [(300, 120), (700, 128)] * 20, "tile")])
def test_softmax_keeps_nan(H, dtype, heads, lens, kernel):
    """A row of Q with a NaN, and a key with a NaN: the rows that see them are NaN in that head,
    and the others are what they are without."""
    counts = [c for _, c in lens]
    ac = make_attn_case([n for n, _ in lens], heads, 64, 64, seed=31, dtype=dtype)
    cache = nan_cache(H, layers=1, heads=heads, pages=sum(-(-n // 16) for n, _ in lens) + 4, seqs=len(lens), blocks=50,
                      ps=16, dtype=dtype)
    j, rows = load_cache(H, ac, cache, counts)
    cfg = H.LayerConfig(64 * heads, heads, 64, 64, phi2="softmax", dtype=dtype)
    q = tensor(ac.q[rows], DT[dtype], "cuda")
    rp, rt = tensor(ac.rab_pos, torch.float32, "cuda"), tensor(ac.rab_time, torch.float32, "cuda")
    ctx = max(n for n, _ in lens)
    H.profiler_start()
    clean = H.paged_attn_fwd(cfg, cache, 0, j, q, rp, rt, ctx)
    assert set(H.profiler_stop()) == {"paged_attention_" + kernel}
    q2 = q.clone()
    q2[1, 64 + 5] = float("nan")
    got = H.paged_attn_fwd(cfg, cache, 0, j, q2, rp, rt, ctx)
    assert bool(got[1, 64:128].isnan().all())
    got[1, 64:128] = clean[1, 64:128]
    assert torch.equal(got, clean)
    # a key of the second sequence: event 0, seen by all its rows, and the last one, by itself
    n, c = lens[1]
    r0 = counts[0]
    for at, seen in ((0, slice(r0, r0 + c)), (n - 1, slice(r0 + c - 1, r0 + c))):
        page = int(cache.block_table[1, at // 16])
        old = float(cache.kv[0, page, 0, 0, at % 16, 3])
        cache.kv[0, page, 0, 0, at % 16, 3] = float("nan")
        got = H.paged_attn_fwd(cfg, cache, 0, j, q, rp, rt, ctx)
        cache.kv[0, page, 0, 0, at % 16, 3] = old
        assert bool(got[seen, :64].isnan().all())
        got[seen, :64] = clean[seen, :64]
        assert torch.equal(got, clean)
    assert H.device_status() == 0


@pytest.mark.parametrize("dtype,c", [("fp16", 3), ("fp16", 200), ("bf16", 3), ("bf16", 200), ("fp32", 3), ("fp32", 200)])
def test_the_longest_span(H, dtype, c):
    """An event 2^31 - 3 seconds before the last one is taken as it is, one second more is reported."""
    ac = make_attn_case([250], 1, 16, 128, seed=2, dtype=dtype)
    for span, want_status in ((2 ** 31 - 3, 0), (2 ** 31 - 2, 6)):
        ac.timestamps[:] = 1_700_000_000 + span
        ac.timestamps[0] = 1_700_000_000
        cache = nan_cache(H, layers=1, heads=1, pages=20, seqs=1, blocks=16, ps=16, dtype=dtype)
        j, rows = load_cache(H, ac, cache, [c])
        cfg = H.LayerConfig(64, 1, 16, 128, dtype=dtype)
        got = H.paged_attn_fwd(cfg, cache, 0, j, tensor(ac.q[rows], DT[dtype], "cuda"),
                               tensor(ac.rab_pos, torch.float32, "cuda"),
                               tensor(ac.rab_time, torch.float32, "cuda"), 250)
        assert H.device_status() == want_status, span
        if want_status == 0:
            f = np.float64
            want = P.chunk_attention(ac.q[250 - c:].astype(f), ac.k.astype(f), ac.v.astype(f), ac.timestamps,
                                     ac.rab_pos.astype(f), ac.rab_time.astype(f), 1)
            assert_close(got.float().cpu().numpy(), want, f"span {span} {dtype}", scaled=True)


@pytest.mark.parametrize("ps", [16, 64])
def test_whole_rows_of_the_block_table(H, ps):
    """Every entry of every block-table row after each call, those past the length included: a
    released block is -1, and so is one that was never given out."""
    rng = np.random.default_rng(100 + ps)
    seqs, blocks, pages = 6, 7, 24
    cache = nan_cache(H, layers=1, heads=1, pages=pages, seqs=seqs, blocks=blocks, ps=ps, dtype="fp16")
    pg = P.Pages(pages, seqs, blocks, ps)
    done = {op: 0 for op in ("reserve", "refused", "fork", "release", "trim", "compact")}
    for _ in range(150):
        op = str(rng.choice(["reserve", "reserve", "fork", "release", "trim", "compact"]))
        if op == "reserve":
            ids = rng.permutation(seqs)[:int(rng.integers(1, 4))].tolist()
            cnt = [int(v) for v in rng.integers(0, 3 * ps, len(ids))]
            ok = pg.reserve(ids, cnt) is not None
            op = op if ok else "refused"
            H.cache_reserve(cache, chunk_of(H, cnt, range(sum(cnt))), seq_ids=i32(ids))
            assert H.device_status() == (0 if ok else 6)
        elif op == "fork":
            full, empty = [s for s in range(seqs) if pg.len[s]], [s for s in range(seqs) if not pg.len[s]]
            if not full or not empty:
                continue
            H.cache_fork(cache, i32(full[:1]), i32(empty[:1]))
            pg.fork(full[0], empty[0])
        elif op == "release":
            s = int(rng.integers(seqs))
            H.cache_release(cache, i32([s]))
            pg.release(s)
        elif op == "trim":
            s, w, k = int(rng.integers(seqs)), int(rng.integers(1, 3 * ps)), int(rng.integers(0, 2 * ps))
            H.cache_release(cache, i32([s]), window=w, sinks=k)
            pg.release(s, w, k)
        else:
            H.cache_compact(cache)
            pg.compact()
        done[op] += 1
        assert H.device_status() == 0
        assert tables(cache) == (pg.table, pg.len, pg.ref)
    assert min(done.values()) > 0, done


@pytest.mark.parametrize("users", [128, 129, 300])
@pytest.mark.parametrize("phi2", ["silu", "softmax"])
def test_attention_of_many_users(H, phi2, users):
    """The few-rows kernel with and without its order by length (up to 128 sequences): ragged users,
    some of them without events or without new ones."""
    rng = np.random.default_rng(users)
    n = [int(v) for v in rng.integers(0, 400, users)]
    run_attn(H, [(v, min(v, int(rng.integers(0, 6)))) for v in n], 4, "fp16", phi2, 32, kernel="rows")


@pytest.mark.parametrize("phi2", ["silu", "softmax"])
@pytest.mark.parametrize("window,sinks", [(40, 9), (1, 0), (16, 50)])
def test_extend_fp32_through_a_window(H, phi2, window, sinks):
    """A stack of fp32 layers through a window with sinks, in several requests, its pages released behind it."""
    case = make_case(make_case("tiny-fp32").cfg.replace(phi2=phi2, num_layers=2), seed=33, lengths=[130, 64, 1, 47])
    cfg = config_of(H, case.cfg)
    t = case_tensors(case, "cuda")
    weights = [H.LayerWeights(**lw) for lw in t["layers"]]
    cache = nan_cache(H, layers=2, heads=case.cfg.num_heads, pages=40, seqs=4, blocks=9, ps=16, dtype="fp32")
    cuts = [[0, 100, 101, 130], [0, 10, 63, 64], [0, 0, 1, 1], [0, 30, 30, 47]]
    state = [None] * 4
    for step in range(3):
        rows = np.concatenate([case.offsets[u] + np.arange(cuts[u][step], cuts[u][step + 1]) for u in range(4)])
        j = chunk_of(H, [cuts[u][step + 1] - cuts[u][step] for u in range(4)], case.timestamps[rows])
        y = H.extend(cfg, weights, cache, j, t["x"][torch.from_numpy(rows).cuda()].contiguous(), 130, window=window,
                     sinks=sinks)
        H.cache_release(cache, i32(range(4)), window=window, sinks=sinks)
        assert H.device_status() == 0
        want = []
        for u in range(4):
            a, b = case.offsets[u] + cuts[u][step], case.offsets[u] + cuts[u][step + 1]
            if b > a:
                w, state[u] = P.extend(state[u], case.x[a:b], case.timestamps[a:b], case.layers, case.cfg,
                                       window=window, sinks=sinks)
                want.append(w)
        assert_close(y.cpu().numpy(), np.concatenate(want), f"extend fp32 {phi2} {window} {sinks} step {step}")


@pytest.mark.parametrize("count", [3, 500, 4096, 4097, 9000])
def test_forks_follow_the_rule(H, count):
    """Random forks, most of them allowed: those from a sequence that is a destination, into one
    that an earlier fork names or that is not empty, and out of range ones are left out, below
    and above the number from which the destinations are marked."""
    rng = np.random.default_rng(count)
    seqs = 2 * count + 20
    pages = seqs // 2 + 60
    cache = nan_cache(H, layers=1, heads=1, pages=pages, seqs=seqs, blocks=3, ps=16, dtype="fp16")
    full = rng.permutation(seqs)[:min(20, seqs // 3)].tolist()
    kept = set(full)
    n = [int(v) for v in rng.integers(1, 49, len(full))]
    H.cache_reserve(cache, chunk_of(H, n, range(sum(n))), seq_ids=i32(full))
    assert H.device_status() == 0
    for trial in range(6):
        lens, ref, table = cache.lengths.tolist(), cache.ref_count.tolist(), cache.block_table.tolist()
        empty = [s for s in range(seqs) if lens[s] == 0]
        dst = rng.permutation(empty)[:count].tolist()
        dst += rng.permutation(seqs)[:count - len(dst)].tolist()
        to = set(dst)
        pool = [s for s in full if lens[s]] + [s for s in empty if s not in to][:3]
        src = [int(v) for v in rng.choice(pool, count)]
        if trial % 2:
            for _ in range(max(1, count // 50)):
                i, k = (int(v) for v in rng.integers(0, count, 2))
                what = int(rng.integers(5))
                if what == 0:
                    dst[i] = dst[k]
                elif what == 1:
                    src[i] = dst[k]
                elif what == 2:
                    dst[i] = full[0]
                elif what == 3:
                    src[i] = int(rng.choice([-1, seqs, 2 ** 31 - 1, -2 ** 31]))
                else:
                    dst[i] = int(rng.choice([-1, seqs]))
        named, taken, bad = set(dst), set(), 0
        for s, d in zip(src, dst):
            ok = 0 <= s < seqs and 0 <= d < seqs and s not in named and d not in taken and table[d][0] < 0 and lens[d] == 0
            taken.add(d)
            if ok and lens[s]:
                blocks = -(-lens[s] // 16)
                for b in range(blocks):
                    table[d][b] = table[s][b]
                    ref[table[s][b]] += 1
                lens[d] = lens[s]
            bad += not ok
        H.cache_fork(cache, i32(src), i32(dst))
        assert H.device_status() == (6 if bad else 0), (trial, bad)
        assert cache.lengths.tolist() == lens and cache.ref_count.tolist() == ref
        assert cache.block_table.tolist() == table
        H.cache_release(cache, i32([s for s in range(seqs) if lens[s] and s not in kept] or full[:1]))
        assert H.device_status() == 0


def test_chunks_without_rows(H):
    """No new events at all: nothing is needed of the timestamps, and nothing happens."""
    case = make_case("small-bf16", seed=41, lengths=[20])
    cfg = config_of(H, case.cfg)
    weights = [H.LayerWeights(**lw) for lw in case_tensors(case, "cuda")["layers"]]
    heads = case.cfg.num_heads
    cache = nan_cache(H, layers=case.cfg.num_layers, heads=heads, pages=6, seqs=2, blocks=4, ps=16, dtype="fp16")
    H.cache_reserve(cache, chunk_of(H, [20, 0], range(20)))
    before = tables(cache)
    rows = torch.empty((0, heads * 64), dtype=torch.float16, device="cuda")
    rp = torch.zeros((heads, 16), device="cuda")
    for offsets in (i32([0, 0, 0]).long(), i32([0]).long()):
        for times in (torch.empty(0), torch.empty(0, dtype=torch.int64, device="cuda"), torch.arange(5)):
            j = H.Jagged(offsets, times, 0, 0)
            H.cache_reserve(cache, j)
            H.cache_append(cache, 0, j, rows, rows)
            acfg = H.LayerConfig(heads * 64, heads, 16, 16, dtype="fp16")
            assert H.paged_attn_fwd(acfg, cache, 0, j, rows, rp, rp, 20).shape == rows.shape
            y = H.extend(cfg, weights, cache, j, torch.empty((0, case.cfg.d_model), dtype=torch.bfloat16, device="cuda"), 20)
            assert y.shape == (0, case.cfg.d_model)
    assert H.device_status() == 0 and tables(cache) == before
