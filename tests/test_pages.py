"""Page operators of paged caches against a plain model on the host, and a serving
run that uses them with the caches and attention they hold."""
import ctypes as C

import numpy as np
import pytest
import torch

import int4_util as U
from kv_cache_vector_14_b200 import tq

gpu = pytest.mark.gpu


class Model:
    """The documented semantics, one entry at a time."""

    def __init__(self, table, refs, pools, Hkv):
        self.t, self.r, self.p, self.Hkv = table.copy(), refs.copy(), [p.copy() for p in pools], Hkv

    def free(self, keep):
        for row in range(len(self.t)):
            for lb in range(self.t.shape[1]):
                if lb * 64 >= keep[row // self.Hkv] and self.t[row, lb] >= 0:
                    self.r[self.t[row, lb]] -= 1
                    self.t[row, lb] = -1

    def fork(self, parent):
        old = self.t.copy()
        for row in range(len(old)):
            b, h = divmod(row, self.Hkv)
            if parent[b] == b or not -1 <= parent[b] < len(parent):
                continue
            for lb in range(old.shape[1]):
                new = -1 if parent[b] < 0 else old[parent[b] * self.Hkv + h, lb]
                if old[row, lb] >= 0:
                    self.r[old[row, lb]] -= 1
                if new >= 0:
                    self.r[new] += 1
                self.t[row, lb] = new

    def alloc(self, lo, hi):
        free = [int(p) for p in np.flatnonzero(self.r == 0)]
        start, missing = self.r.copy(), 0
        for row in range(len(self.t)):
            l, h = int(lo[row // self.Hkv]), int(hi[row // self.Hkv])
            for lb in range(l // 64, -(-h // 64) if h > l else 0):
                e = self.t[row, lb]
                if e >= 0 and start[e] <= 1:
                    continue
                if not free:
                    missing += 1
                    continue
                p = free.pop(0)
                if e >= 0:
                    for d in self.p:
                        d[p] = d[e]
                    self.r[e] -= 1
                self.t[row, lb], self.r[p] = p, 1
        return [int((self.r == 0).sum()), missing]

    def compact(self):
        live = np.flatnonzero(self.r > 0)
        L = len(live)
        holes = [p for p in range(L) if self.r[p] <= 0]
        far = [p for p in live[::-1] if p >= L]
        where = np.arange(len(self.r))
        for a, b in zip(far, holes):
            where[a] = b
            self.r[b], self.r[a] = self.r[a], 0
            for d in self.p:
                d[b] = d[a]
        self.t = np.where(self.t >= 0, where[np.maximum(self.t, 0)], self.t).astype(np.int32)
        return [len(self.r) - L, len(holes)]


def build(B, Hkv, NB, pool, lens, seed=0, share=0, sizes=(160, 48)):
    """Random placement; the first `share` blocks of odd sequences are those of the sequence before."""
    rng = np.random.default_rng(seed)
    table = np.full((B * Hkv, NB), -1, np.int32)
    places = list(rng.permutation(pool))
    for b in range(B):
        for h in range(Hkv):
            for lb in range(-(-int(lens[b]) // 64)):
                if b % 2 and lb < share and table[(b - 1) * Hkv + h, lb] >= 0:
                    table[b * Hkv + h, lb] = table[(b - 1) * Hkv + h, lb]
                else:
                    table[b * Hkv + h, lb] = places.pop()
    refs = np.bincount(table[table >= 0], minlength=pool).astype(np.int32)
    pools = [rng.integers(0, 256, (pool, s), dtype=np.uint8) for s in sizes]
    return table, refs, pools


class Dev:
    def __init__(self, table, refs, pools, Hkv):
        self.h = tq.tq_init(64, 0)
        self.t, self.r = torch.from_numpy(table.copy()).cuda(), torch.from_numpy(refs.copy()).cuda()
        self.p = [torch.from_numpy(p.copy()).cuda() for p in pools]
        self.pages = tq.Pages(self.t, self.r, Hkv, [(p, p.shape[1]) for p in self.p])
        self.ws = torch.full((tq.tq_pages_workspace_bytes(self.pages),), 255, dtype=torch.uint8, device="cuda")
        self.info = torch.zeros(2, dtype=torch.int32, device="cuda")

    def same(self, m, defined=None):
        assert np.array_equal(self.t.cpu().numpy(), m.t)
        assert np.array_equal(self.r.cpu().numpy(), m.r)
        for a, b in zip(self.p, m.p):
            assert np.array_equal(a.cpu().numpy()[m.r > 0], b[m.r > 0])
        named = m.t[m.t >= 0]
        assert np.array_equal(np.bincount(named, minlength=len(m.r)), m.r)

    def close(self):
        assert tq.tq_device_status(self.h) == tq.TQ_OK
        tq.tq_destroy(self.h)


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ CPU

def test_struct_and_null_errors(libtq):
    assert C.sizeof(tq.tq_pages) == 72 and tq.tq_pages.buffers.offset == 56
    inv = tq.TQ_ERR_INVALID_ARG
    p = tq.tq_pages()
    assert libtq.tq_pages_workspace_bytes(None) == 0 and libtq.tq_pages_workspace_bytes(C.byref(p)) == 0
    assert libtq.tq_pages_alloc(None, C.byref(p), None, None, None, None, 0, None) == inv
    assert libtq.tq_pages_fork(None, C.byref(p), None, None) == inv
    assert libtq.tq_pages_free(None, C.byref(p), None, None) == inv
    assert libtq.tq_pages_compact(None, C.byref(p), None, None, 0, None) == inv
    assert libtq.tq_pages_copy(None, C.byref(p), C.byref(p), None, None, 0, None) == inv


def test_pages_refusals_cpu(libtq):
    t, r = torch.full((4, 3), -1, dtype=torch.int32), torch.zeros(10, dtype=torch.int32)
    buf = torch.zeros((10, 64), dtype=torch.uint8)
    pg = tq.Pages(t, r, 2, [(buf, 64)])
    assert (pg.B, pg.pool_blocks) == (2, 10) and tq.tq_pages_workspace_bytes(pg) > 0
    for bad in ((t.long(), r, 2), (t, r.long(), 2), (t, r, 3), (t[:, :2], r, 2), (t, r[::2], 2), (t, r, 0)):
        with pytest.raises(ValueError):
            tq.Pages(*bad, [(buf, 64)])
    with pytest.raises(ValueError):
        tq.Pages(t, r, 2, [(buf, 80)])
    with pytest.raises(ValueError):
        tq.Pages(t, r, 2, [(buf, 64)] * 129)


def test_model_keeps_counts():
    """The host model itself: counts equal the table's entries after any sequence of steps."""
    table, refs, pools = build(6, 2, 5, 90, [300, 300, 64, 1, 0, 200], share=3)
    m = Model(table, refs, pools, 2)
    for step in range(4):
        m.fork([0, 0, 3, 2, -1, 1])
        m.alloc([299, 299, 60, 1, 0, 10], [300, 301, 70, 1, 64, 11])
        m.free([300, 128, 70, 0, 64, 0])
        m.compact()
        assert np.array_equal(np.bincount(m.t[m.t >= 0], minlength=90), m.r)


# ------------------------------------------------------------------ GPU

@gpu
@pytest.mark.parametrize("parent", [[0, 1, 2, 3, 4], [0, 0, 0, 0, 0], [1, 0, 3, 4, 2], [-1, 0, 0, -1, 2], [4, 4, 4, 4, -1]])
@pytest.mark.parametrize("Hkv,NB", [(1, 3), (2, 9), (3, 17)])
def test_fork(libtq, parent, Hkv, NB):
    lens = [64 * NB, 100, 0, 65, 130]
    table, refs, pools = build(5, Hkv, NB, 5 * Hkv * NB + 7, lens, share=2)
    m, g = Model(table, refs, pools, Hkv), Dev(table, refs, pools, Hkv)
    m.fork(parent)
    tq.tq_pages_fork(g.h, g.pages, i32(parent))
    g.same(m)
    g.close()


@gpu
@pytest.mark.parametrize("pool", [70, 333, 5000, 70001])
@pytest.mark.parametrize("lo,hi", [([200, 63, 0, 128], [201, 64, 1, 192]), ([0, 0, 0, 0], [320, 320, 320, 320]),
                                   ([10, 20, 30, 40], [10, 20, 30, 40]), ([190, 0, 319, 64], [195, 1, 320, 320])])
def test_alloc(libtq, pool, lo, hi):
    Hkv = 3
    table, refs, pools = build(4, Hkv, 5, pool, [200, 200, 0, 130], seed=pool, share=4)
    m, g = Model(table, refs, pools, Hkv), Dev(table, refs, pools, Hkv)
    want = m.alloc(lo, hi)
    tq.tq_pages_alloc(g.h, g.pages, i32(lo), i32(hi), g.info, g.ws)
    g.same(m)
    assert g.info.tolist() == want
    g.close()


@gpu
def test_alloc_runs_out(libtq):
    table, refs, pools = build(4, 1, 5, 14, [200, 200, 64, 130], share=4)
    m, g = Model(table, refs, pools, 1), Dev(table, refs, pools, 1)
    lo, hi = [199, 199, 64, 130], [320, 320, 320, 320]
    want = m.alloc(lo, hi)
    assert want[1] > 0
    tq.tq_pages_alloc(g.h, g.pages, i32(lo), i32(hi), g.info, g.ws)
    g.same(m)
    assert g.info.tolist() == want
    g.close()


@gpu
@pytest.mark.parametrize("keep", [[0, 0, 0], [500, 500, 500], [64, 65, 1], [-5, 128, 320]])
def test_free(libtq, keep):
    table, refs, pools = build(3, 2, 5, 60, [300, 300, 129], share=3)
    m, g = Model(table, refs, pools, 2), Dev(table, refs, pools, 2)
    m.free(keep)
    tq.tq_pages_free(g.h, g.pages, i32(keep))
    g.same(m)
    g.close()


@gpu
@pytest.mark.parametrize("pool,lens", [(40, [300, 300, 0]), (45, [300, 300, 300]), (1000, [320, 1, 70]), (33000, [320, 320, 5]),
                                       (64, [0, 0, 0]), (150001, [320, 320, 300])])
@pytest.mark.parametrize("sizes", [(160, 48), (4608, 4608, 16, 6144), ()])
def test_compact(libtq, pool, lens, sizes):
    table, refs, pools = build(3, 2, 5, pool, lens, seed=pool, share=2, sizes=sizes)
    m, g = Model(table, refs, pools, 2), Dev(table, refs, pools, 2)
    want = m.compact()
    tq.tq_pages_compact(g.h, g.pages, g.info, g.ws)
    g.same(m)
    assert g.info.tolist() == want
    live = int((m.r > 0).sum())
    assert (m.r[:live] > 0).all()
    tq.tq_pages_compact(g.h, g.pages, None, g.ws)                 # nothing left to move
    g.same(m)
    g.close()


@gpu
def test_copy(libtq):
    rng = np.random.default_rng(0)
    a = [torch.from_numpy(rng.integers(0, 256, (50, s), dtype=np.uint8)).cuda() for s in (4608, 80)]
    b = [torch.zeros((20, s), dtype=torch.uint8, device="cuda") for s in (4608, 80)]
    table, refs = torch.full((1, 1), -1, dtype=torch.int32, device="cuda"), lambda n: torch.zeros(n, dtype=torch.int32, device="cuda")
    pa, pb = (tq.Pages(table, refs(len(x[0])), 1, [(t, t.shape[1]) for t in x]) for x in (a, b))
    h = tq.tq_init(64, 0)
    src, dst = [3, 49, 3, -1, 7, 0], [0, 19, 5, 2, -1, 6]
    tq.tq_pages_copy(h, pa, pb, i32(src), i32(dst))
    for x, y in zip(a, b):
        want = torch.zeros_like(y)
        for s, d in zip(src, dst):
            if s >= 0 and d >= 0:
                want[d] = x[s]
        assert torch.equal(y, want)
    tq.tq_pages_copy(h, pa, pa, i32([1, 2]), i32([40, 41]))       # inside one pool
    assert torch.equal(a[0][40], a[0][1]) and torch.equal(a[1][41], a[1][2])
    tq.tq_pages_copy(h, pa, pb, i32([]), i32([]))
    assert tq.tq_device_status(h) == tq.TQ_OK
    keep = [y.clone() for y in b]
    tq.tq_pages_copy(h, pa, pb, i32([50, 0, -2]), i32([1, 20, 3]))
    assert tq.tq_device_status(h) == tq.TQ_ERR_DEVICE_CHECK
    assert all(torch.equal(x, y) for x, y in zip(keep, b))
    assert libtq.tq_pages_copy(h, pa._ref, pb._ref, None, None, 3, None) == tq.TQ_ERR_INVALID_ARG
    assert libtq.tq_pages_copy(h, pa._ref, pb._ref, None, None, -1, None) == tq.TQ_ERR_INVALID_ARG
    tq.tq_destroy(h)


@gpu
def test_bad_entries_and_arguments(libtq):
    table, refs, pools = build(3, 1, 4, 30, [200, 200, 70], share=2)
    g = Dev(table, refs, pools, 1)
    g.t[1, 0] = 30                                                # an entry outside the pool
    before = g.t.clone(), g.r.clone()
    tq.tq_pages_free(g.h, g.pages, i32([300, 0, 300]))
    assert tq.tq_device_status(g.h) == tq.TQ_ERR_DEVICE_CHECK and int(g.t[1, 0]) == 30
    g.t.copy_(before[0]), g.r.copy_(before[1])
    tq.tq_pages_alloc(g.h, g.pages, i32([0, 0, 0]), i32([0, 1, 0]), g.info, g.ws)
    assert tq.tq_device_status(g.h) == tq.TQ_ERR_DEVICE_CHECK and torch.equal(g.t, before[0])
    tq.tq_pages_fork(g.h, g.pages, i32([3, -2, 2]))               # parents out of range: unchanged
    assert tq.tq_device_status(g.h) == tq.TQ_ERR_DEVICE_CHECK
    assert torch.equal(g.t, before[0]) and torch.equal(g.r, before[1])
    tq.tq_pages_compact(g.h, g.pages, g.info, g.ws)
    assert tq.tq_device_status(g.h) == tq.TQ_ERR_DEVICE_CHECK and int(g.t[1, 0]) == 30
    tq.tq_pages_alloc(g.h, g.pages, i32([-5, 0, 0]), i32([0, 0, 1000]), g.info, g.ws)   # beyond the table: what fits is supplied
    assert tq.tq_device_status(g.h) == tq.TQ_ERR_DEVICE_CHECK and (g.t[2] >= 0).all()
    L, inv = libtq, tq.TQ_ERR_INVALID_ARG
    assert L.tq_pages_alloc(g.h, g.pages._ref, None, None, None, g.ws.data_ptr(), g.ws.numel(), None) == inv
    assert L.tq_pages_alloc(g.h, g.pages._ref, g.r.data_ptr(), g.r.data_ptr(), None, g.ws.data_ptr(), 100,
                            None) == tq.TQ_ERR_WORKSPACE
    assert L.tq_pages_compact(g.h, g.pages._ref, None, g.ws.data_ptr() + 4, g.ws.numel(), None) == inv
    assert L.tq_pages_fork(g.h, g.pages._ref, None, None) == inv and L.tq_pages_free(g.h, g.pages._ref, None, None) == inv
    for field, value, status in (("refs", None, inv), ("NB", 0, inv), ("pool_blocks", 0, inv), ("Hkv", 0, inv),
                                 ("n_buffers", 129, inv), ("n_buffers", -1, inv), ("NB", 1 << 40, tq.TQ_ERR_UNSUPPORTED),
                                 ("pool_blocks", 1 << 31, tq.TQ_ERR_UNSUPPORTED)):
        p = tq.tq_pages.from_buffer_copy(g.pages.struct)
        setattr(p, field, value)
        assert L.tq_pages_compact(g.h, C.byref(p), None, g.ws.data_ptr(), g.ws.numel(), None) == status, field
    big = tq.Pages(torch.full((7169, 1), -1, dtype=torch.int32, device="cuda"), g.r, 1, [])
    assert L.tq_pages_fork(g.h, big._ref, g.r.data_ptr(), None) == tq.TQ_ERR_UNSUPPORTED
    tq.tq_destroy(g.h)


@gpu
def test_large_batch_random_walk(libtq):
    """Many sequences over many steps: forks, frees, allocations and compactions stay on the model."""
    rng = np.random.default_rng(4)
    B, Hkv, NB, pool = 60, 2, 7, 1500
    lens = rng.integers(0, NB * 64, B)
    table, refs, pools = build(B, Hkv, NB, pool, lens, share=3, sizes=(64,))
    m, g = Model(table, refs, pools, Hkv), Dev(table, refs, pools, Hkv)
    for step in range(12):
        parent = np.where(rng.random(B) < 0.4, rng.integers(-1, B, B), np.arange(B))
        m.fork(parent)
        tq.tq_pages_fork(g.h, g.pages, i32(parent))
        lens = np.where(parent < 0, 0, lens[np.maximum(parent, 0)])
        hi = np.minimum(lens + rng.integers(0, 90, B), NB * 64)
        assert m.alloc(lens, hi) == (tq.tq_pages_alloc(g.h, g.pages, i32(lens), i32(hi), g.info, g.ws), g.info.tolist())[1]
        lens = np.where(rng.random(B) < 0.2, hi // 2, hi)
        m.free(lens)
        tq.tq_pages_free(g.h, g.pages, i32(lens))
        g.same(m)
        if step % 3 == 2:
            assert m.compact() == (tq.tq_pages_compact(g.h, g.pages, g.info, g.ws), g.info.tolist())[1]
            g.same(m)
    g.close()


@gpu
@pytest.mark.parametrize("kind", ["int4", "tq"])
def test_beam_serving_run(libtq, kind):
    """A beam search as a program would run it: one prompt encoded once and forked, then steps of reordering,
    supplying, appending and attending, with a compaction between; every beam's result equals attention over a
    contiguous cache that holds its own history."""
    d, group, Hkv, G, beams, T0, steps = 128, 64, 2, 4, 4, 150, 5
    rng = np.random.default_rng(1)
    NB = 5
    h = tq.tq_init(d, 0)
    pool = 60
    table, refs = torch.full((beams * Hkv, NB), -1, dtype=torch.int32, device="cuda"), torch.zeros(pool, dtype=torch.int32, device="cuda")
    if kind == "int4":
        caches = [tq.Int4Cache(d, group, beams, Hkv, NB * 64, block_table=table, pool_blocks=pool) for _ in range(2)]
    else:
        caches = [tq.Cache(d, k, beams, Hkv, NB * 64, block_table=table, pool_blocks=pool) for k in (True, False)]
    pages = tq.Pages(table, refs, Hkv, caches)
    info, pws = torch.zeros(2, dtype=torch.int32, device="cuda"), torch.zeros(tq.tq_pages_workspace_bytes(pages), dtype=torch.uint8, device="cuda")

    def encode(c, is_k, x, t0, b=None):
        if kind == "int4":
            tq.tq_encode_int4(h, x, c, t0=t0)
        else:
            (tq.tq_encode_k if is_k else tq.tq_encode_v)(h, x, c, t0)

    def attend(q, kc, vc, T):
        if kind == "int4":
            out = torch.zeros_like(q)
            ws = torch.zeros(tq.tq_attend_int4_workspace_bytes(h, q.shape[0], 1, Hkv * G, Hkv), dtype=torch.uint8, device="cuda")
            tq.tq_attend_int4(h, q, kc, vc, out, ws, T=T, scale=0.09)
        else:
            out = torch.zeros(q.shape, device="cuda")
            ws = torch.zeros(tq.tq_attend_workspace_bytes(h, q.shape[0], Hkv * G, Hkv, NB * 64), dtype=torch.uint8, device="cuda")
            tq.tq_attend_decode(h, q, kc, vc, out, ws, T=T, scale=0.09)
        return out

    prompt = [torch.randn((1, Hkv, T0, d), device="cuda") for _ in range(2)]
    zeros = i32([0] * beams)
    tq.tq_pages_alloc(h, pages, zeros, i32([T0] + [0] * (beams - 1)), info, pws)
    # the prompt goes into sequence 0 alone: a one-sequence view of the same table
    for c, is_k, x in zip(caches, (True, False), prompt):
        if kind == "int4":
            one = tq.Int4Cache(d, group, 1, Hkv, NB * 64, buf=c.buf, block_table=table[:Hkv], pool_blocks=pool)
        else:
            one = tq.Cache(d, is_k, 1, Hkv, NB * 64, buf=c.buf, block_table=table[:Hkv], pool_blocks=pool)
        encode(one, is_k, x, 0)
    tq.tq_pages_fork(h, pages, zeros)
    history = [[x[0] for x in prompt] for _ in range(beams)]
    for step in range(steps):
        T = T0 + 30 * step
        tq.tq_pages_alloc(h, pages, i32([T] * beams), i32([T + 30] * beams), info, pws)
        assert int(info[1]) == 0
        new = [torch.randn((beams, Hkv, 30, d), device="cuda") for _ in range(2)]
        for c, is_k, x in zip(caches, (True, False), new):
            encode(c, is_k, x, T)
        history = [[torch.cat([history[b][i], new[i][b]], 1) for i in range(2)] for b in range(beams)]
        q = torch.randn((beams, Hkv * G, d), device="cuda")
        got = attend(q, *caches, T + 30)
        for b in range(beams):
            if kind == "int4":
                own = [tq.Int4Cache(d, group, 1, Hkv, NB * 64 + 64) for _ in range(2)]
            else:
                own = [tq.Cache(d, k, 1, Hkv, NB * 64 + 64) for k in (True, False)]
            for c, is_k, x in zip(own, (True, False), history[b]):
                encode(c, is_k, x[None].contiguous(), 0)
            ref = attend(q[b:b + 1], *own, T + 30)
            # the same tokens in another split of the work: fp32 sums in another order
            assert torch.allclose(got[b:b + 1], ref, rtol=0, atol=2.0 ** -18 * float(ref.abs().max()) * 8)
        parent = [0, 0, 3, 1] if step % 2 == 0 else [2, 1, 0, 2]
        tq.tq_pages_fork(h, pages, i32(parent))
        history = [list(history[p]) for p in parent]
        if step == 2:
            tq.tq_pages_compact(h, pages, info, pws)
    tq.tq_pages_free(h, pages, zeros)
    assert not refs.any() and (table == -1).all()
    assert tq.tq_device_status(h) == tq.TQ_OK
    tq.tq_destroy(h)


@gpu
@pytest.mark.parametrize("d,dtype", [(128, torch.bfloat16), (64, torch.float16)])
@pytest.mark.parametrize("before", ["fork", "alloc", "compact", "expand"])
def test_bulk_append_behind_a_call_that_writes_what_it_reads(libtq, d, dtype, before):
    """A bulk tq_append_attend (whose encodes and attention are chained) directly behind a call that writes the block
    table or the new values gives what it gives after a synchronisation.  A slow product first, so that the launches
    stand ready behind each other."""
    B, Hkv, G, T0, Tnew, NB = 16, 2, 2, 1024, 512, 64
    pool, h = 2 * B * Hkv * NB, tq.tq_init(d, 0)
    gen = torch.Generator(device="cuda").manual_seed(d)
    lens = T0 if before == "alloc" else T0 + Tnew
    table0 = torch.full((B * Hkv, NB), -1, dtype=torch.int32, device="cuda")
    place = torch.randperm(pool, generator=gen, device="cuda").to(torch.int32)
    table0[:, :lens // 64] = place[:B * Hkv * (lens // 64)].view(B * Hkv, -1)
    refs0 = torch.zeros(pool, dtype=torch.int32, device="cuda")
    refs0[table0[table0 >= 0].long()] = 1
    table, refs = table0.clone(), refs0.clone()
    caches = [tq.Cache(d, k, B, Hkv, NB * 64, block_table=table, pool_blocks=pool) for k in (True, False)]
    pages = tq.Pages(table, refs, Hkv, caches)
    pws = torch.zeros(tq.tq_pages_workspace_bytes(pages), dtype=torch.uint8, device="cuda")
    ws = torch.zeros(tq.tq_attend_workspace_bytes(h, B, Hkv * G, Hkv, NB * 64), dtype=torch.uint8, device="cuda")
    k, v = (torch.randn((B, Hkv, Tnew, d), generator=gen, device="cuda").to(dtype) for _ in range(2))
    prefix = [torch.randn((B, Hkv, T0, d), generator=gen, device="cuda").to(dtype) for _ in range(2)]
    q = torch.randn((B, Hkv * G, d), generator=gen, device="cuda").to(dtype)
    four = tq.Int4Cache(d, 32, B, Hkv, Tnew)
    tq.tq_encode_int4(h, torch.randn((B, Hkv, Tnew, d), generator=gen, device="cuda"), four)
    swap = i32(np.arange(B) ^ 1)
    lo, hi = i32([T0] * B), i32([T0 + Tnew] * B)
    slow = torch.randn((4096, 4096), device="cuda")

    def run(apart):
        table.copy_(table0)
        refs.copy_(refs0)
        v.zero_() if before == "expand" else None
        for c in caches:
            c.buf.zero_()
        tq.tq_encode_k(h, prefix[0], caches[0], 0)
        tq.tq_encode_v(h, prefix[1], caches[1], 0)
        out = torch.zeros((B, Hkv * G, d), device="cuda")
        torch.cuda.synchronize()
        slow @ slow
        if before == "fork":
            tq.tq_pages_fork(h, pages, swap)
        elif before == "alloc":
            tq.tq_pages_alloc(h, pages, lo, hi, None, pws)
        elif before == "compact":
            tq.tq_pages_compact(h, pages, None, pws)
        else:
            tq.tq_expand_int4(h, four, v)
        if apart:
            torch.cuda.synchronize()
        tq.tq_append_attend(h, k, v, *caches, T0, q, out, ws, scale=0.09)
        assert tq.tq_device_status(h) == tq.TQ_OK
        return [out, *(c.buf.clone() for c in caches), table.clone()]

    want = run(True)
    for _ in range(3):
        for a, b in zip(run(False), want):
            assert torch.equal(a, b)
    tq.tq_destroy(h)


def test_pages_on_the_host_are_refused_cpu(libtq):
    t, r = torch.full((4, 3), -1, dtype=torch.int32), torch.zeros(10, dtype=torch.int32)
    pg = tq.Pages(t, r, 2, [(torch.zeros((10, 64), dtype=torch.uint8), 64)])
    v, info, ws = torch.zeros(2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), torch.zeros(4096, dtype=torch.uint8)
    for f in (lambda: tq.tq_pages_alloc(None, pg, v, v, info, ws), lambda: tq.tq_pages_fork(None, pg, v),
              lambda: tq.tq_pages_free(None, pg, v), lambda: tq.tq_pages_compact(None, pg, info, ws),
              lambda: tq.tq_pages_copy(None, pg, pg, v, v)):
        with pytest.raises(ValueError, match="current CUDA device"):
            f()


@gpu
def test_vectors_on_the_host_are_refused(libtq):
    table, refs, pools = build(3, 2, 5, 60, [300, 300, 129], share=3)
    g = Dev(table, refs, pools, 2)
    v, host, info = i32([0, 1, 2]), torch.zeros(3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    for f in (lambda: tq.tq_pages_alloc(g.h, g.pages, host, v, g.info, g.ws),
              lambda: tq.tq_pages_alloc(g.h, g.pages, v, host, g.info, g.ws),
              lambda: tq.tq_pages_alloc(g.h, g.pages, v, v, info, g.ws),
              lambda: tq.tq_pages_alloc(g.h, g.pages, v, v, g.info, g.ws.cpu()),
              lambda: tq.tq_pages_fork(g.h, g.pages, host), lambda: tq.tq_pages_free(g.h, g.pages, host),
              lambda: tq.tq_pages_compact(g.h, g.pages, info, g.ws),
              lambda: tq.tq_pages_compact(g.h, g.pages, g.info, g.ws.cpu()),
              lambda: tq.tq_pages_copy(g.h, g.pages, g.pages, host, v),
              lambda: tq.tq_pages_copy(g.h, g.pages, g.pages, v, host)):
        with pytest.raises(ValueError, match="current CUDA device"):
            f()
    with pytest.raises(ValueError, match="one device"):
        tq.Pages(g.t, g.r.cpu(), 2, [])
    assert np.array_equal(g.t.cpu().numpy(), table) and np.array_equal(g.r.cpu().numpy(), refs)
    g.close()


@gpu
@pytest.mark.parametrize("pool", [4000, 2500])
def test_alloc_many_blocks_per_row(libtq, pool):
    """A prompt's pages: hundreds of blocks of few rows, some shared, from an empty table and behind a prefix; and
    the same where the pool runs out."""
    Hkv, NB = 2, 600
    table, refs, pools = build(3, Hkv, NB, pool, [5000, 5000, 0], seed=pool, share=70, sizes=(64, 32))
    m, g = Model(table, refs, pools, Hkv), Dev(table, refs, pools, Hkv)
    for lo, hi in (([4000, 5000, 0], [30000, 5001, 38400]), ([0, 0, 0], [64 * NB, 64, 38400])):
        want = m.alloc(lo, hi)
        tq.tq_pages_alloc(g.h, g.pages, i32(lo), i32(hi), g.info, g.ws)
        g.same(m)
        assert g.info.tolist() == want
    assert (want[1] > 0) == (pool == 2500)
    g.close()


@gpu
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("call", ["encode few", "encode bulk", "decode", "polar", "prefill", "append few"])
def test_older_calls_directly_behind_page_calls(libtq, d, call):
    """Every entry point of the TurboQuant caches behind a fork that exchanges the sequences' pages, with and without
    a synchronisation between."""
    B, Hkv, G, T, NB = 8, 2, 4, 960, 18
    h, pool = tq.tq_init(d, 0), B * Hkv * NB
    gen = torch.Generator(device="cuda").manual_seed(d)
    table0 = torch.randperm(pool, generator=gen, device="cuda").to(torch.int32).view(B * Hkv, NB)
    table, refs = table0.clone(), torch.ones(pool, dtype=torch.int32, device="cuda")
    polar = call == "polar"
    caches = [tq.Cache(d, k and not polar, B, Hkv, NB * 64, block_table=table, pool_blocks=pool) for k in (True, False)]
    pages = tq.Pages(table, refs, Hkv, caches)
    x = [torch.randn((B, Hkv, T, d), generator=gen, device="cuda").bfloat16() for _ in range(2)]
    n = 1152 if call == "encode bulk" else 3
    new = torch.randn((B, Hkv, n, d), generator=gen, device="cuda").bfloat16()
    Lq = 9
    q = torch.randn((B, Lq, Hkv * G, d) if call == "prefill" else (B, Hkv * G, d), generator=gen, device="cuda").bfloat16()
    ws = torch.zeros(max(tq.tq_attend_workspace_bytes(h, B, Hkv * G, Hkv, NB * 64),
                         tq.tq_prefill_workspace_bytes(h, B, Lq, Hkv * G)), dtype=torch.uint8, device="cuda")
    swap = i32(np.arange(B) ^ 1)
    slow = torch.randn((4096, 4096), device="cuda")

    def run(apart):
        table.copy_(table0)
        for c, v in zip(caches, x):
            c.buf.zero_()
            (tq.tq_encode_k if c.is_k else tq.tq_encode_v)(h, v, c, 0)
        out = torch.zeros(q.shape, device="cuda")
        torch.cuda.synchronize()
        slow @ slow
        tq.tq_pages_fork(h, pages, swap)
        if apart:
            torch.cuda.synchronize()
        if call.startswith("encode"):
            for c in caches:
                (tq.tq_encode_k if c.is_k else tq.tq_encode_v)(h, new, c, 0 if n > 3 else T)
        elif call == "decode":
            tq.tq_attend_decode(h, q, *caches, out, ws, T=T, scale=0.09)
        elif polar:
            tq.tq_attend_decode_polar(h, q, *caches, out, ws, T=T, scale=0.09)
        elif call == "prefill":
            tq.tq_attend_prefill(h, q, *caches, T - Lq, out, ws, scale=0.09)
        else:
            tq.tq_append_attend(h, new, new, *caches, T, q, out, ws, scale=0.09)
        assert tq.tq_device_status(h) == tq.TQ_OK
        return [out, *(c.buf.clone() for c in caches)]

    want = run(True)
    for _ in range(3):
        for a, b in zip(run(False), want):
            assert torch.equal(a, b)
    tq.tq_destroy(h)
