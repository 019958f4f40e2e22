"""The paged history cache without a GPU: pins of its oracle, and what the entry
points refuse before any device work."""
import ctypes

import numpy as np
import pytest

from gen import make_case
from gen.inputs import make_attn_case
from oracle import hstu as O
from oracle import paged as P


# ---------------------------------------------------------------- oracle pins

@pytest.mark.parametrize("phi2", ["silu", "softmax"])
def test_chunk_attention_is_the_tail_of_the_whole(phi2):
    ac = make_attn_case([70], 2, 32, 32, seed=1, dtype="fp32")
    rp, rt = ac.rab_pos.astype(np.float64), ac.rab_time.astype(np.float64)
    q, k, v = (a.astype(np.float64) for a in (ac.q, ac.k, ac.v))
    whole = O.user_attention(q, k, v, ac.timestamps, rp, rt, 70, 2, 64, 64, phi2)
    for c in (1, 7, 70):
        got = P.chunk_attention(q[70 - c:], k, v, ac.timestamps, rp, rt, 2, phi2)
        assert np.allclose(got, whole[70 - c:], rtol=1e-12, atol=1e-14)
    # a window that reaches every key changes nothing; W = 1 leaves the row itself
    same = P.chunk_attention(q[60:], k, v, ac.timestamps, rp, rt, 2, phi2, window=70)
    assert np.allclose(same, whole[60:], rtol=1e-12, atol=1e-14)
    vis = P.window_mask(9, 3, 1, 2)
    assert vis.tolist() == [[j < 2 or j == i for j in range(9)] for i in (6, 7, 8)]


def test_extend_in_one_step_is_the_forward():
    case = make_case("tiny-fp32", seed=3, lengths=[33])
    want, _ = O.forward(case.x, case.offsets, case.timestamps, case.layers, case.cfg)
    got, _ = P.extend(None, case.x, case.timestamps, case.layers, case.cfg)
    assert np.allclose(got, want, rtol=1e-10, atol=1e-12)
    # in steps: the earlier rows' K and V are kept; layer 0's do not depend on later rows, so
    # a one-layer stack gives the same rows (N is the length after the step)
    st = None
    for a, b in ((0, 10), (10, 11), (11, 33)):
        y, st = P.extend(st, case.x[a:b], case.timestamps[a:b], case.layers, case.cfg)
    assert np.allclose(y, want[11:], rtol=1e-10, atol=1e-12)


def test_pages_keep_their_invariants():
    rng = np.random.default_rng(5)
    pg = P.Pages(40, 6, 8, 16)
    for _ in range(400):
        op, s = rng.integers(5), int(rng.integers(6))
        if op == 0:
            pg.reserve([s], [int(rng.integers(0, 30))])
        elif op == 1 and pg.len[s] > 0:
            empty = [d for d in range(6) if pg.len[d] == 0]
            if empty:
                pg.fork(s, empty[0])
        elif op == 2:
            pg.release(s)
        elif op == 3:
            pg.release(s, window=20, sinks=5)
        else:
            pg.compact()
            used = sum(r > 0 for r in pg.ref)
            assert all(r > 0 for r in pg.ref[:used])
        named = [p for row, n in zip(pg.table, pg.len) for p in row[:pg.blocks(n)] if p >= 0]
        assert [named.count(p) for p in range(40)] == pg.ref


# ---------------------------------------------------------------- refusals

@pytest.fixture(scope="module")
def H():
    from hstu_sequential_transduction_jagged_b200 import build, hstu
    build.build()
    return hstu


def _cache(H, **kw):
    # pointers that no refused call touches
    f = dict(num_layers=2, num_heads=4, dtype=2, page_size=64, num_pages=100, num_seqs=8,
             max_blocks=16, kv=4096, timestamps=4096, ref_count=4096, block_table=4096, lengths=4096)
    f.update(kw)
    return H.CacheT(*[f[n] for n, _ in H.CacheT._fields_])


def _chunk(H, **kw):
    f = dict(batch=2, total_tokens=10, max_len=8, offsets=4096, timestamps=4096, segments=None,
             max_static=0)
    f.update(kw)
    return H.JaggedT(*[f[n] for n, _ in H.JaggedT._fields_])


BAD_CACHES = [(dict(num_layers=0), 1), (dict(num_heads=0), 1), (dict(num_pages=0), 1),
              (dict(num_seqs=0), 1), (dict(max_blocks=0), 1), (dict(dtype=7), 1), (dict(kv=None), 1),
              (dict(kv=4104), 1), (dict(timestamps=None), 1), (dict(block_table=None), 1),
              (dict(lengths=None), 1), (dict(ref_count=None), 1), (dict(page_size=48), 2),
              (dict(page_size=256), 2), (dict(page_size=8), 2), (dict(num_heads=200), 2),
              (dict(num_pages=1 << 22), 2), (dict(max_blocks=1 << 21), 2)]


@pytest.mark.parametrize("kw,want", BAD_CACHES)
def test_bad_caches_are_refused(H, kw, want):
    L, c, j, r = H.lib(), _cache(H, **kw), _chunk(H), ctypes.byref
    assert L.hstu_cache_reserve(r(c), r(j), None, 4096, 1 << 20, None) == want
    assert L.hstu_cache_fork(r(c), 1, 4096, 4096, None) == want
    assert L.hstu_cache_release(r(c), 1, 4096, 0, 0, None) == want
    assert L.hstu_cache_compact(r(c), None, 4096, 1 << 20, None) == want
    if "ref_count" in kw:
        return  # not needed to move rows or attend
    assert L.hstu_cache_workspace_bytes(r(c), 2) == 0
    assert L.hstu_cache_append(r(c), 0, r(j), None, 4096, 256, 4096, 256, None) == want
    assert L.hstu_cache_gather(r(c), 2, None, 4096, 10, 4096, None, None) == want
    cfg = H.LayerConfig(256, 4, 64, 32, dtype="fp16").c()
    assert L.hstu_paged_attn_fwd(r(cfg), r(c), 0, r(j), None, 100, 0, 0, 4096, 256, 4096, 4096, 4096,
                                 None) == want


def test_bad_calls_are_refused(H):
    L, c, r = H.lib(), _cache(H), ctypes.byref
    good = _chunk(H)
    for kw, want in ((dict(batch=-1), 1), (dict(offsets=None), 1), (dict(timestamps=None), 1),
                     (dict(max_len=0), 1), (dict(total_tokens=-1), 1), (dict(segments=4096), 2),
                     (dict(batch=65536), 2)):
        j = _chunk(H, **kw)
        assert L.hstu_cache_reserve(r(c), r(j), None, 4096, 1 << 20, None) == want, kw
        assert L.hstu_cache_append(r(c), 0, r(j), None, 4096, 256, 4096, 256, None) == want, kw
    ws = L.hstu_cache_workspace_bytes(r(c), 2)
    assert ws > 0
    assert L.hstu_cache_reserve(r(c), r(good), None, 4096, ws - 1, None) == 4
    assert L.hstu_cache_reserve(r(c), r(good), None, None, ws, None) == 4
    assert L.hstu_cache_compact(r(c), None, 4096, 16, None) == 4
    for args in ((-1, 4096, 256, 4096, 256), (2, 4096, 256, 4096, 256), (0, None, 256, 4096, 256),
                 (0, 4100, 256, 4096, 256), (0, 4096, 255, 4096, 256), (0, 4096, 256, 4096, 260),
                 (0, 4096, 256, 4096, 192)):
        layer, k, ldk, v, ldv = args
        assert L.hstu_cache_append(r(c), layer, r(good), None, k, ldk, v, ldv, None) == 1, args
    assert L.hstu_cache_gather(r(c), 2, None, None, 10, 4096, None, None) == 1
    assert L.hstu_cache_gather(r(c), 2, None, 4096, 10, 4104, None, None) == 1
    assert L.hstu_cache_fork(r(c), 1, None, 4096, None) == 1
    assert L.hstu_cache_fork(r(c), -1, 4096, 4096, None) == 1
    assert L.hstu_cache_release(r(c), 1, 4096, -1, 0, None) == 1
    assert L.hstu_cache_release(r(c), 1, 4096, 5, -1, None) == 1

    def attn(cfg=None, cache=c, layer=0, chunk=good, ctx=100, w=0, sk=0, q=4096, ld=256, rp=4096, out=4096):
        cfg = (cfg or H.LayerConfig(256, 4, 64, 32, dtype="fp16")).c()
        return L.hstu_paged_attn_fwd(r(cfg), r(cache), layer, r(chunk), None, ctx, w, sk, q, ld, rp, 4096,
                                     out, None)

    assert attn(cfg=H.LayerConfig(256, 4, 64, 32, dtype="bf16")) == 1  # the cache is fp16
    assert attn(cfg=H.LayerConfig(512, 8, 64, 32, dtype="fp16")) == 1  # other head count
    assert attn(cfg=H.LayerConfig(256, 4, 64, 32, dtype="fp16", dqk=32)) == 2
    for kw in (dict(layer=2), dict(layer=-1), dict(ctx=0), dict(ctx=-5), dict(w=-1), dict(sk=-1), dict(q=None),
               dict(q=4100), dict(ld=255), dict(ld=64), dict(rp=None), dict(out=None), dict(out=4104)):
        assert attn(**kw) == 1, kw
    assert attn(w=(1 << 30) + 1) == 2
    empty = _chunk(H, batch=0, total_tokens=0, max_len=0, offsets=None, timestamps=None)
    assert attn(chunk=empty, q=None, out=None) == 0
    # extend: a bf16 stack keeps an fp16 cache, of as many layers as it has
    cfg = H.LayerConfig(256, 4, 64, 32)
    w = (H.LayerWeightsT * 2)(*[H.LayerWeightsT(*([4096] * 8)) for _ in range(2)])

    def ext(layers=2, cache=c, nbytes=None, x=4096):
        cc = cfg.c()
        need = L.hstu_extend_workspace_bytes(r(cc), r(cache), 2, 10)
        return L.hstu_extend(r(cc), layers, w, r(cache), r(good), None, 100, 0, 0, x, 4096, 4096,
                             need if nbytes is None else nbytes, None)

    assert ext(layers=1) == 1
    assert ext(layers=0) == 1
    assert ext(cache=_cache(H, dtype=0)) == 1
    assert ext(cache=_cache(H, ref_count=None)) == 1
    assert ext(x=None) == 1
    assert ext(nbytes=100) == 4


def test_binding_refuses_wrong_tensors(H):
    """Layouts that the bare pointers would misread are refused by the handle and the calls."""
    import torch
    mk = lambda **kw: H.PagedCache(**{**dict(  # noqa: E731
        kv=torch.zeros(1, 4, 2, 1, 16, 64, dtype=torch.float16), timestamps=torch.zeros(4, 16, dtype=torch.int64),
        ref_count=torch.zeros(4, dtype=torch.int32), block_table=torch.zeros(3, 5, dtype=torch.int32),
        lengths=torch.zeros(3, dtype=torch.int32)), **kw})
    cache = mk()
    assert cache.c().num_seqs == 3 and cache.c().max_blocks == 5 and cache.c().dtype == 2
    for kw in (dict(kv=torch.zeros(4, 2, 1, 16, 64, dtype=torch.float16)),
               dict(kv=torch.zeros(1, 4, 2, 1, 16, 64, dtype=torch.float64)),
               dict(kv=torch.zeros(1, 4, 2, 1, 64, 16, dtype=torch.float16).transpose(4, 5)),
               dict(timestamps=torch.zeros(4, 16, dtype=torch.int32)), dict(timestamps=torch.zeros(16, 4, dtype=torch.int64)),
               dict(ref_count=torch.zeros(5, dtype=torch.int32)), dict(lengths=torch.zeros(3, dtype=torch.int64)),
               dict(block_table=torch.zeros(4, 5, dtype=torch.int32)), dict(block_table=torch.zeros(5, 3, dtype=torch.int32).t())):
        with pytest.raises(ValueError):
            mk(**kw)
    with pytest.raises(ValueError):
        H.cache_release(cache, torch.zeros(1, dtype=torch.int64))
    with pytest.raises(ValueError):
        H.cache_fork(cache, torch.zeros(2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32))
    chunk = H.Jagged(torch.zeros(2, dtype=torch.int64), torch.zeros(1, dtype=torch.int64), 1, 1)
    rows = torch.zeros(1, 64, dtype=torch.float16)
    with pytest.raises(ValueError):
        H.cache_append(cache, 0, chunk, rows.to(torch.bfloat16), rows)
    with pytest.raises(ValueError):
        H.cache_append(cache, 0, chunk, rows.t(), rows)
    with pytest.raises(ValueError):
        H.cache_append(cache, 0, chunk, rows, rows, seq_ids=torch.zeros(2, dtype=torch.int32))


def test_memory_of_a_call_comes_from_its_stream(H, monkeypatch):
    """Workspaces and results of a call on another stream are made on that stream, and the
    current one, which takes the result, is named to the allocator."""
    import contextlib
    import types
    log, now = [], ["current"]

    class Block:
        def record_stream(self, s):
            log.append(("kept for", s))

    @contextlib.contextmanager
    def on(s):
        now.append(s)
        yield
        now.pop()

    def empty(shape, dtype, device):
        log.append(("made on", now[-1], shape))
        return Block()

    fake = types.SimpleNamespace(empty=empty, uint8="u8", cuda=types.SimpleNamespace(
        current_stream=lambda: now[-1], stream=on))
    monkeypatch.setattr(H, "torch", fake)
    H._workspace(5, "cuda", None, "side")
    assert log == [("made on", "side", 5), ("kept for", "current")]
    del log[:]
    H._empty(7, "f32", "cuda", "current")
    H._empty(8, "f32", "cuda")
    assert log == [("made on", "current", 7), ("made on", "current", 8)]
    given = Block()
    assert H._workspace(5, "cuda", given, "side") is given and len(log) == 2
