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


def test_binding_refuses_what_pointers_would_misread(H):
    """Rows, tables, offsets and results of the wrong size, type or layout; tensors that are not on
    the GPU.  Everything is refused before the library is called."""
    import torch
    f16, f32, i32, i64 = torch.float16, torch.float32, torch.int32, torch.int64
    z = lambda *s, dtype=f16: torch.zeros(*s, dtype=dtype)  # noqa: E731
    cache = H.PagedCache(z(2, 4, 2, 3, 16, 64), z(4, 16, dtype=i64), z(4, dtype=i32), z(3, 5, dtype=i32), z(3, dtype=i32))
    T, hv = 6, 192
    chunk = H.Jagged(torch.tensor([0, 2, 6]), z(T, dtype=i64), 4, T)
    ids = z(2, dtype=i32)
    rows = z(T, hv)
    bad_chunks = [H.Jagged(chunk.offsets.to(i32), chunk.timestamps, 4, T),
                  H.Jagged(z(6, dtype=i64)[::2], chunk.timestamps, 4, T),
                  H.Jagged(chunk.offsets, chunk.timestamps[:-1], 4, T),
                  H.Jagged(chunk.offsets, chunk.timestamps.to(i32), 4, T),
                  H.Jagged(chunk.offsets, z(2 * T, dtype=i64)[::2], 4, T)]
    bad_rows = [z(T - 1, hv), z(T + 1, hv), z(T, hv - 64), z(T, 2 * hv)[:, :hv - 64], z(T, 3, 64), z(T, hv, dtype=torch.bfloat16)]

    def refused(match, f, *a, **kw):
        with pytest.raises(ValueError, match=match):
            f(*a, **kw)

    # append
    for bad in bad_rows:
        refused("total_tokens, num_heads", H.cache_append, cache, 0, chunk, bad, rows, seq_ids=ids)
        refused("total_tokens, num_heads", H.cache_append, cache, 0, chunk, rows, bad, seq_ids=ids)
    # attention
    cfg = H.LayerConfig(hv, 3, 16, 32, dtype="fp16")
    rp, rt = z(3, 16, dtype=f32), z(3, 32, dtype=f32)

    def attn(fn=H.paged_attn_fwd, q=rows, rp=rp, rt=rt, chunk=chunk, **kw):
        return fn(cfg, cache, 0, chunk, q, rp, rt, 20, **kw)

    for fn in (H.paged_attn_fwd, H.paged_attn_fwd_f32):
        for bad in bad_rows:
            refused("q must be", attn, fn, q=bad)
        for bad in (z(3, 15, dtype=f32), z(2, 16, dtype=f32), z(16, dtype=f32), z(3, 16), z(3, 16, dtype=torch.float64),
                    z(16, 3, dtype=f32).t()):
            refused("rab_pos", attn, fn, rp=bad)
        for bad in (z(3, 16, dtype=f32), z(3, 32), z(3, 64, dtype=f32)[:, ::2]):
            refused("rab_time", attn, fn, rt=bad)
    for bad in bad_rows[:2] + [z(T, hv, dtype=f32), z(hv, T).t(), z(T, 2 * hv)[:, :hv]]:
        refused("av_out", attn, av_out=bad)
    refused("av_out", attn, H.paged_attn_fwd_f32, av_out=rows)
    # extend (a fp32 stack keeps its cache in fp32)
    cache32 = H.PagedCache(cache.kv.float(), *cache[1:5])
    ecfg = H.LayerConfig(128, 3, 16, 32, dtype="fp32")
    w = [H.LayerWeights(*[z(4, dtype=f32)] * 6)] * 2
    x = z(T, 128, dtype=f32)

    def ext(x=x, chunk=chunk, **kw):
        return H.extend(ecfg, w, cache32, chunk, x, 20, **kw)

    for bad in (x[:-1], z(T, 64, dtype=f32), z(T, 256, dtype=f32)[:, :128], z(128, T, dtype=f32).t(), x.half(), x.bfloat16()):
        refused("x_in", ext, bad)
        refused("y_out", ext, y_out=bad)
    # gather
    off = torch.tensor([0, 5, 9])
    for bad in (off.to(i32), z(6, dtype=i64)[::2]):
        refused("offsets", H.cache_gather, cache, bad, 9)
    for bad in (z(2, 8, 2 * hv), z(1, 9, 2 * hv), z(2, 9, 2 * hv, dtype=f32), z(2, 9, 4 * hv)[:, :, ::2]):
        refused("kv_out", H.cache_gather, cache, off, 9, kv_out=bad)
    for bad in bad_chunks:
        refused("the chunk needs", H.cache_reserve, cache, bad, seq_ids=ids)
        refused("the chunk needs", H.cache_append, cache, 0, bad, rows, rows, seq_ids=ids)
        refused("the chunk needs", attn, chunk=bad, seq_ids=ids)
        refused("the chunk needs", ext, chunk=bad, seq_ids=ids)
    # nothing wrong but that the tensors are on the CPU
    for f in (lambda: H.cache_reserve(cache, chunk, seq_ids=ids), lambda: H.cache_append(cache, 0, chunk, rows, rows),
              lambda: H.cache_gather(cache, off, 9), lambda: H.cache_fork(cache, ids, ids),
              lambda: H.cache_release(cache, ids), lambda: H.cache_compact(cache), attn, ext,
              lambda: attn(H.paged_attn_fwd_f32)):
        refused("not on the current GPU", f)


def test_a_replaced_part_is_described_anew(H):
    import torch
    i32 = torch.int32
    cache = H.PagedCache(torch.zeros(1, 4, 2, 1, 16, 64), torch.zeros(4, 16, dtype=torch.int64), torch.zeros(4, dtype=i32),
                         torch.zeros(3, 5, dtype=i32), torch.zeros(3, dtype=i32))
    other = torch.zeros(3, dtype=i32)
    got = cache._replace(lengths=other)
    assert got.lengths is other and got.c().lengths == other.data_ptr() and got.c().kv == cache.kv.data_ptr()
    assert cache.c().lengths == cache.lengths.data_ptr()
    for kw in (dict(lengths=torch.zeros(4, dtype=i32)), dict(desc=cache.desc), dict(size=3)):
        with pytest.raises(ValueError):
            cache._replace(**kw)


def test_more_forks_than_indexes_are_refused(H):
    assert H.lib().hstu_cache_fork(ctypes.byref(_cache(H)), 1 << 30, 4096, 4096, None) == 2
