"""4-bit caches: encode, expand, attention and the appending step, against the
64-bit oracle in int4_util.py (whose docstring derives the tolerances)."""
import ctypes as C

import numpy as np
import pytest
import torch

import int4_util as U
from kv_cache_vector_14_b200 import tq

gpu = pytest.mark.gpu
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SHAPES = [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128), (256, 32), (256, 64), (256, 128)]


# ------------------------------------------------------------------ CPU

def test_sizes(libtq):
    for d, g in SHAPES:
        bb = 64 * (d // 2 + 4 * d // g)
        assert tq.tq_int4_block_bytes(d, g) == bb and bb % 16 == 0
        assert tq.tq_int4_cache_bytes(d, g, 3, 5, 640) == 150 * bb
    for d, g in ((64, 128), (128, 16), (128, 256), (96, 32), (128, 0), (128, -64)):
        assert tq.tq_int4_block_bytes(d, g) == 0 and tq.tq_int4_cache_bytes(d, g, 1, 1, 64) == 0
    assert tq.tq_int4_cache_bytes(128, 64, 1, 1, 100) == 0 and tq.tq_int4_cache_bytes(128, 64, 1, 1, 0) == 0
    assert tq.tq_int4_cache_bytes(128, 64, -1, 1, 64) == 0


def test_null_handle_and_descriptor_errors(libtq):
    c = tq.tq_cache(None, 1, 1, 64)
    bad = tq.TQ_ERR_INVALID_ARG
    for f in (libtq.tq_encode_int4, libtq.tq_expand_int4):
        assert f(None, 64, None, 0, 1, 1, 1, 0, 0, 0, C.byref(c), None, 0, None) == bad
    assert libtq.tq_attend_int4(None, 64, None, 0, 1, 1, 1, C.byref(c), C.byref(c), None, 1, 1.0, None, None, 0,
                                None) == bad
    assert libtq.tq_append_attend_int4(None, 64, None, None, 0, 1, 0, 0, 0, C.byref(c), C.byref(c), None, 0, None, 0, 1,
                                       1.0, None, None, 0, None) == bad
    assert libtq.tq_append_attend_int4(None, 64, None, None, 0, 1, 0, 0, 0, None, None, None, 0, None, 0, 1, 1.0, None,
                                       None, 0, None) == bad
    assert libtq.tq_attend_int4_workspace_bytes(None, 1, 1, 1, 1) == 0


def test_python_refusals_cpu(libtq):
    with pytest.raises(ValueError):
        tq.Int4Cache(128, 64, 1, 1, 100, device="cpu")
    with pytest.raises(ValueError):
        tq.Int4Cache(64, 128, 1, 1, 64, device="cpu")
    with pytest.raises(ValueError):
        tq.Int4Cache(128, 64, 1, 1, 64, buf=torch.zeros(100, dtype=torch.uint8))
    with pytest.raises(ValueError):
        tq.Int4Cache(128, 64, 2, 1, 64, device="cpu", block_table=torch.zeros((1, 1), dtype=torch.int32), pool_blocks=4)
    with pytest.raises(ValueError):
        tq._int32(torch.zeros(3, dtype=torch.int64), "pos", 3)
    with pytest.raises(ValueError):
        tq._int32(torch.zeros(3, dtype=torch.int32), "pos", 4)


def test_oracle_round_trip_and_error_bound():
    """The oracle's own format: a value is off by at most half a step plus the fp16 roundings of
    scale and zero (2^-11 of either, 15 steps at most)."""
    x = np.random.default_rng(0).standard_normal((200, 128)).astype(np.float32) * 3 + 1
    for g in (32, 64, 128):
        codes, scale, zero = U.quantise(x, g)
        s = np.repeat(np.abs(scale.astype(np.float64)), g, -1)
        z = np.repeat(np.abs(zero.astype(np.float64)), g, -1)
        assert np.all(np.abs(U.grid(x, g) - x) <= s * (0.5 + 15 * 2.0 ** -11) + z * 2.0 ** -11)
        assert codes.min() == 0 and codes.max() == 15


# ------------------------------------------------------------------ GPU helpers

class Case:
    """Caches of B sequences holding the encoded prefix of given float32 vectors."""

    def __init__(self, d, group, B, Hkv, Tcap, paged=False, seed=0, extra=3):
        self.d, self.group, self.B, self.Hkv, self.Tcap, self.NB = d, group, B, Hkv, Tcap, Tcap // 64
        rng = np.random.default_rng(seed)
        self.pool = B * Hkv * self.NB + extra
        self.ids = rng.permutation(self.pool)[:B * Hkv * self.NB] if paged else np.arange(B * Hkv * self.NB)
        self.ids = self.ids.reshape(B * Hkv, self.NB)
        self.h = tq.tq_init(d, 0)
        self.caches = []
        for _ in range(2):
            table = torch.tensor(self.ids, dtype=torch.int32, device="cuda") if paged else None
            n = self.pool if paged else B * Hkv * self.NB
            # stale contents: whatever was there must not matter
            buf = torch.randint(0, 256, (n * tq.tq_int4_block_bytes(d, group),), dtype=torch.uint8,
                                generator=torch.Generator().manual_seed(seed)).cuda()
            self.caches.append(tq.Int4Cache(d, group, B, Hkv, Tcap, buf=buf, block_table=table, pool_blocks=n if paged else 0))

    def raw(self, which):
        c = self.caches[which]
        return c.buf.cpu().numpy().reshape(-1, c.block_bytes)

    def stored(self, which, b, hh, T):
        return U.read_cache(self.raw(which), self.d, self.group, self.ids[b * self.Hkv + hh], T)

    def close(self):
        assert tq.tq_device_status(self.h) == tq.TQ_OK
        tq.tq_destroy(self.h)


def rand(rng, shape, keys=True):
    x = rng.standard_normal(shape).astype(np.float32)
    if keys:
        x = x * np.exp(0.5 * rng.standard_normal(shape[-1])).astype(np.float32)
        x += (2 * rng.standard_normal(shape[-1]) * (rng.random(shape[-1]) < 0.1)).astype(np.float32)
    return x


def to_gpu(x, dtype):
    return torch.from_numpy(np.ascontiguousarray(x)).to(TYPES[dtype]).cuda()


def as_np(t):
    return t.float().cpu().numpy()


# ------------------------------------------------------------------ encode, expand

@gpu
@pytest.mark.parametrize("d,group", SHAPES)
@pytest.mark.parametrize("dtype,paged,token_major,offset", [("f32", False, False, 0), ("bf16", True, True, 0),
                                                            ("f16", False, True, 1), ("bf16", False, False, 3)])
def test_encode_bit_exact_and_expand(libtq, d, group, dtype, paged, token_major, offset):
    B, Hkv, T, Tcap = 3, 2, 77, 192
    cs = Case(d, group, B, Hkv, Tcap, paged, seed=d + group)
    rng = np.random.default_rng(d * group)
    x = rand(rng, (B, T, Hkv, d) if token_major else (B, Hkv, T, d))
    # offset: the vectors start off a 16-byte boundary
    flat = torch.zeros(x.size + offset, dtype=TYPES[dtype], device="cuda")
    flat[offset:] = to_gpu(x, dtype).view(-1)
    t = flat[offset:].view(x.shape)
    t = t.transpose(1, 2) if token_major else t
    pos = np.array([0, 13, 115])
    before = cs.raw(0).copy()
    tq.tq_encode_int4(cs.h, t, cs.caches[0], pos=torch.tensor(pos, dtype=torch.int32, device="cuda"))
    xs = as_np(t)
    bb = 64 * (d // 2 + 4 * d // group)
    touched = np.zeros((cs.pool if paged else len(before), bb), bool)
    for b in range(B):
        for hh in range(Hkv):
            got = cs.stored(0, b, hh, int(pos[b]) + T)
            want = U.quantise(xs[b, hh], group)
            for g_, w_ in zip(got, want):
                g_ = g_[pos[b]:]
                assert np.array_equal(g_.view(np.uint16) if g_.dtype == np.float16 else g_,
                                      w_.view(np.uint16) if w_.dtype == np.float16 else w_)
            for tt in range(pos[b], pos[b] + T):
                blk, tau = cs.ids[b * Hkv + hh][tt // 64], tt % 64
                touched[blk, tau * (d // 2):(tau + 1) * (d // 2)] = True
                at = 64 * (d // 2) + tau * 4 * (d // group)
                touched[blk, at:at + 4 * (d // group)] = True
    after = cs.raw(0)
    assert np.array_equal(after[~touched], before[~touched])          # nothing else is written
    out = torch.full((B, Hkv, T, d), 7.0, dtype=TYPES[dtype], device="cuda")
    tq.tq_expand_int4(cs.h, cs.caches[0], out, pos=torch.tensor(pos, dtype=torch.int32, device="cuda"))
    want = torch.from_numpy(U.grid(xs, group).astype(np.float32)).to(TYPES[dtype])
    assert torch.equal(out.cpu(), want)
    # a strided output that is not 16-byte aligned gives the same values
    wide = torch.zeros((B, Hkv, T, d + 1), dtype=TYPES[dtype], device="cuda")
    tq.tq_expand_int4(cs.h, cs.caches[0], wide[..., 1:], pos=torch.tensor(pos, dtype=torch.int32, device="cuda"))
    assert torch.equal(wide[..., 1:].cpu(), want) and not wide[..., 0].any()
    cs.close()


@gpu
def test_encode_extremes(libtq):
    """Constant groups, values beyond fp16, infinities, subnormal ranges and NaN, one vector each."""
    d, group = 128, 64
    x = np.zeros((1, 1, 10, d), np.float32)
    rng = np.random.default_rng(5)
    x[0, 0, 1] = 3.1415927
    x[0, 0, 2] = rng.standard_normal(d) * 1e6
    x[0, 0, 3] = rng.standard_normal(d)
    x[0, 0, 3, 5], x[0, 0, 3, 70] = np.inf, -np.inf
    x[0, 0, 4] = rng.standard_normal(d) * 1e-7
    x[0, 0, 5] = 1000 + rng.standard_normal(d) * 1e-3
    x[0, 0, 6] = rng.standard_normal(d)
    x[0, 0, 6, 3] = np.nan
    x[0, 0, 7] = np.inf
    x[0, 0, 8] = -65504.0
    x[0, 0, 9, ::2] = 65504.0
    x[0, 0, 9, 1::2] = -65504.0
    cs = Case(d, group, 1, 1, 64)
    tq.tq_encode_int4(cs.h, to_gpu(x, "f32"), cs.caches[0])
    codes, scale, zero = cs.stored(0, 0, 0, 10)
    c2, s2, z2 = U.quantise(x[0, 0], group)
    assert np.isnan(scale[6, 0]) and np.isnan(zero[6, 0]) and np.isfinite(scale[6, 1])
    ok = np.ones(10, bool)
    ok[6] = False
    assert np.array_equal(codes[ok], c2[ok])
    assert np.array_equal(scale[ok], s2[ok]) and np.array_equal(zero[ok], z2[ok])
    assert np.array_equal(codes[6, 64:], c2[6, 64:])
    out = torch.zeros((1, 1, 10, d), device="cuda")
    tq.tq_expand_int4(cs.h, cs.caches[0], out)
    o = out.cpu().numpy()[0, 0]
    assert np.isnan(o[6, :64]).all() and np.isfinite(o[6, 64:]).all() and np.isfinite(o[ok]).all()
    cs.close()


@gpu
def test_positions_outside_the_cache_are_skipped_and_reported(libtq):
    d, group, T = 128, 64, 5
    cs = Case(d, group, 3, 1, 64)
    x = to_gpu(rand(np.random.default_rng(1), (3, 1, T, d)), "f32")
    before = cs.raw(0).copy()
    pos = torch.tensor([62, -3, 10], dtype=torch.int32, device="cuda")
    tq.tq_encode_int4(cs.h, x, cs.caches[0], pos=pos)
    assert tq.tq_device_status(cs.h) == tq.TQ_ERR_DEVICE_CHECK
    want = U.quantise(as_np(x).reshape(-1, d), group)[0].reshape(3, T, d)
    assert np.array_equal(cs.stored(0, 0, 0, 64)[0][62:], want[0, :2])
    assert np.array_equal(cs.stored(0, 1, 0, 64)[0][:2], want[1, 3:])
    assert np.array_equal(cs.stored(0, 2, 0, 64)[0][10:15], want[2])
    after = cs.raw(0)
    assert np.array_equal(after[1, 2 * 64:64 * 64], before[1, 2 * 64:64 * 64])
    out = torch.full((3, 1, T, d), 9.0, device="cuda")
    tq.tq_expand_int4(cs.h, cs.caches[0], out, pos=pos)
    assert tq.tq_device_status(cs.h) == tq.TQ_ERR_DEVICE_CHECK
    assert (out[0, 0, 2:] == 9).all() and (out[1, 0, :3] == 9).all() and (out[2] != 9).any()
    cs.close()


# ------------------------------------------------------------------ attention

def run_attend(d, group, dtype, G, Hkv, lens, Lq=1, paged=False, uniform=False, Tcap=None, seed=0, scale=None, qmul=1.0,
               vmul=1.0, lq_check=None):
    B = len(lens)
    Tcap = Tcap or max(64, -(-max(lens) // 64) * 64)
    cs = Case(d, group, B, Hkv, Tcap, paged, seed)
    rng = np.random.default_rng(seed + 17)
    scale = d ** -0.5 if scale is None else scale
    kx, vx = rand(rng, (B, Hkv, Tcap, d)), rand(rng, (B, Hkv, Tcap, d), keys=False) * np.float32(vmul)
    for b in range(B):                     # only the live tokens are written; the rest stays stale bytes
        if lens[b]:
            one = [torch.zeros((B, Hkv, Tcap, d), device="cuda") for _ in range(2)]
            for t, x in zip(one, (kx, vx)):
                t.copy_(torch.from_numpy(x))
            break
    if max(lens):
        # sequence by sequence through pos: rows of other sequences are pushed out of the cache and skipped
        for b in range(B):
            if not lens[b]:
                continue
            pos = torch.full((B,), -(1 << 20), dtype=torch.int32, device="cuda")
            pos[b] = 0
            for t, c in zip(one, cs.caches):
                tq.tq_encode_int4(cs.h, t[:, :, :lens[b]], c, pos=pos)
            tq.tq_device_status(cs.h)      # the skipped rows were reported
    q = to_gpu(rng.standard_normal((B, Lq, Hkv * G, d)).astype(np.float32) * np.float32(qmul), dtype)
    ws = torch.full((tq.tq_attend_int4_workspace_bytes(cs.h, B, Lq, Hkv * G, Hkv),), 255, dtype=torch.uint8, device="cuda")
    out = torch.full_like(q, float("nan"))
    if uniform:
        tq.tq_attend_int4(cs.h, q, *cs.caches, out, ws, T=lens[0], scale=scale)
    else:
        tq.tq_attend_int4(cs.h, q, *cs.caches, out, ws, seq_lens=torch.tensor(lens, dtype=torch.int32, device="cuda"),
                          scale=scale)
    half = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}[dtype]
    got, qn = as_np(out).astype(np.float64), as_np(q).astype(np.float64)
    worst = 0.0
    for b in range(B):
        for hh in range(Hkv):
            kc, ks, kz = U.quantise(kx[b, hh, :lens[b]], group)
            k = U.values(kc, ks, kz, group)
            kabs = U.values(kc, np.abs(ks), np.abs(kz), group)
            v = U.grid(vx[b, hh, :lens[b]], group)
            for g in range(G):
                rows = qn[b, :, hh * G + g]
                ref = U.attend(rows, k, v, scale, Lq)
                err = np.abs(got[b, :, hh * G + g] - ref)
                bound = U.attend_bound(rows, kabs, v, scale, ref, half, bf16=dtype == "bf16",
                                       rounded=dtype == "bf16" and Lq * G > 8)
                if dtype == "f16":
                    bound = bound + 2.0 ** -25        # half a subnormal step
                assert np.isfinite(got[b, :, hh * G + g]).all()
                assert (err <= bound).all(), (b, hh, g, err.max(), bound.max())
                worst = max(worst, float((err / np.maximum(bound, 1e-30)).max()))
    cs.close()
    return worst


@gpu
@pytest.mark.parametrize("d,group", SHAPES)
@pytest.mark.parametrize("dtype,G,Lq", [("f32", 1, 1), ("bf16", 4, 1), ("f16", 8, 1), ("f32", 7, 1), ("bf16", 3, 5),
                                        ("f32", 2, 17)])
def test_attend_matches_oracle(libtq, d, group, dtype, G, Lq):
    run_attend(d, group, dtype, G, 2, [300, 64, 1, 129], Lq=Lq, paged=(G % 2 == 0), seed=d + G)


@gpu
@pytest.mark.parametrize("lens", [[0], [1], [15], [16], [17], [31], [32], [33], [63], [65], [0, 0, 0], [0, 5, 0, 4000, 0, 1]])
@pytest.mark.parametrize("G,Lq", [(1, 1), (6, 2)])
def test_attend_lengths(libtq, lens, G, Lq):
    run_attend(128, 64, "f32", G, 1, lens, Lq=Lq, seed=len(lens))


@gpu
@pytest.mark.parametrize("G,Lq", [(12, 1), (16, 2), (1, 40), (5, 33)])
def test_attend_many_rows_and_rows_before_the_first_token(libtq, G, Lq):
    """Row groups of 8, and sequences shorter than the queries: rows that see nothing give zeros."""
    run_attend(128, 64, "bf16", G, 2, [200, 3, 0, 70], Lq=Lq, seed=G)


@gpu
@pytest.mark.parametrize("d,group", [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128)])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("G,Lq,lens", [(3, 70, [70, 500, 64, 0, 129]), (1, 9, [9, 1000]), (8, 33, [40, 3]),
                                       (1, 300, [300, 700])])
def test_chunks(libtq, d, group, dtype, G, Lq, lens):
    """Chunks of one and of several row tiles, from the first token on, behind a prefix, and longer than
    their sequence."""
    run_attend(d, group, dtype, G, 2, lens, Lq=Lq, paged=(G == 3), seed=G + Lq)


@gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("qmul,vmul,scale", [(1e-6, 1e-4, 1.0), (30.0, 1.0, 1.0), (1.0, 1e3, 0.1), (1.0, 1.0, 0.0),
                                             (1.0, 1.0, -0.2)])
def test_chunk_magnitudes(libtq, dtype, qmul, vmul, scale):
    run_attend(128, 64, dtype, 4, 1, [700, 90], Lq=20, scale=scale, qmul=qmul, vmul=vmul, seed=3)


@gpu
@pytest.mark.parametrize("G,Lq,T,Hkv", [(1, 9, 9000, 2), (4, 60, 5000, 8), (2, 130, 3000, 5)])
def test_chunk_fp32_sums_of_many_tiles(libtq, G, Lq, T, Hkv):
    """fp32 chunks whose CTAs walk many tiles of one unit: the sums are taken out of the tensor core in between."""
    run_attend(128, 64, "f32", G, Hkv, [T, T // 2], Lq=Lq, seed=G, lq_check=3)


@gpu
def test_chunk_units_cut_by_many_ctas(libtq):
    """One kv head and a long cache: every CTA holds a piece of the same row tile."""
    run_attend(128, 64, "f16", 2, 1, [20000], Lq=10, seed=1)


@gpu
@pytest.mark.parametrize("uniform", [False, True])
@pytest.mark.parametrize("d,T", [(64, 5000), (128, 9001), (256, 2100)])
def test_attend_long(libtq, d, T, uniform):
    run_attend(d, 64, "f32", 4, 1, [T, T] if uniform else [T, T // 3], uniform=uniform, seed=T)


@gpu
@pytest.mark.parametrize("qmul,vmul,scale", [(1e-6, 1e-4, 1.0), (300.0, 1.0, 1.0), (1.0, 1e4, 0.1), (1.0, 1.0, 0.0),
                                             (1.0, 1.0, -0.2), (1e-30, 1.0, 1.0)])
def test_attend_magnitudes(libtq, qmul, vmul, scale):
    """Tiny and huge queries, values and scales: the reference exponent keeps p vs inside fp16."""
    run_attend(128, 64, "f32", 4, 1, [700, 90], scale=scale, qmul=qmul, vmul=vmul, seed=3)


@gpu
def test_attend_many_sequences(libtq):
    """More sequences than threads of a CTA, most of them short or empty."""
    lens = [(7 * b) % 23 for b in range(700)]
    run_attend(64, 32, "f32", 2, 1, lens, Tcap=64, seed=9)


def _filled(d, group, B, Hkv, Tcap, seed, paged=False):
    cs = Case(d, group, B, Hkv, Tcap, paged, seed)
    rng = np.random.default_rng(seed)
    x = [rand(rng, (B, Hkv, Tcap, d), k) for k in (True, False)]
    for c, v in zip(cs.caches, x):
        tq.tq_encode_int4(cs.h, to_gpu(v, "f32"), c)
    return cs, x, rng


@gpu
def test_nan_reaches_what_sees_it_and_nothing_else(libtq):
    """A NaN key makes the rows that see it NaN, a NaN value the group of it; other sequences, rows before it and
    garbage pairs behind the last token stay out."""
    d, group = 128, 64
    cs = Case(d, group, 3, 1, 128)
    rng = np.random.default_rng(0)
    k, v = rand(rng, (3, 1, 100, d)), rand(rng, (3, 1, 100, d), False)
    k[1, 0, 50, 3] = np.nan
    v[2, 0, 50, 70] = np.nan
    for c, x in zip(cs.caches, (k, v)):
        c.buf.fill_(255)                                              # NaN pairs everywhere
        tq.tq_encode_int4(cs.h, to_gpu(x, "f32"), c)
    Lq = 60
    q = to_gpu(rng.standard_normal((3, Lq, 4, d)).astype(np.float32), "f32")
    out = torch.zeros_like(q)
    ws = torch.zeros(tq.tq_attend_int4_workspace_bytes(cs.h, 3, Lq, 4, 1), dtype=torch.uint8, device="cuda")
    tq.tq_attend_int4(cs.h, q, *cs.caches, out, ws, T=100, scale=0.1)
    o = torch.isnan(out).cpu()
    assert not o[0].any()
    sees = torch.arange(Lq) + 100 - Lq + 1 > 50
    assert o[1][sees].all() and not o[1][~sees].any()
    assert o[2][sees][..., 64:].all() and not o[2][sees][..., :64].any() and not o[2][~sees].any()
    # a query that is NaN or infinite makes its own row NaN
    q1 = torch.randn((3, 4, d), device="cuda")
    q1[0, 1, 5], q1[2, 3, 0] = float("nan"), float("inf")
    out = torch.zeros_like(q1)
    tq.tq_attend_int4(cs.h, q1, *cs.caches, out, ws, seq_lens=torch.tensor([40, 40, 40], dtype=torch.int32, device="cuda"),
                      scale=0.1)
    bad = torch.isnan(out).all(-1).cpu()
    assert bad[0, 1] and bad[2, 3] and int(torch.isnan(out).any(-1).sum()) == 2
    cs.close()


@gpu
@pytest.mark.parametrize("Lq,paged", [(1, False), (1, True), (4, True), (30, False)])
def test_append_attend_equals_its_parts(libtq, Lq, paged):
    d, group, B, Hkv, G = 128, 64, 3, 2, 4
    cs, _, rng = _filled(d, group, B, Hkv, 320, 11, paged)
    other = Case(d, group, B, Hkv, 320, paged, 11)
    for a, b in zip(cs.caches, other.caches):
        b.buf.copy_(a.buf)
    kv = [to_gpu(rand(rng, (B, Lq, Hkv, d)), "bf16").transpose(1, 2) for _ in range(2)]
    q = to_gpu(rng.standard_normal((B, Lq, Hkv * G, d)).astype(np.float32), "bf16")
    pos = torch.tensor([0, 100, 290], dtype=torch.int32, device="cuda")
    ws = torch.zeros(tq.tq_attend_int4_workspace_bytes(cs.h, B, Lq, Hkv * G, Hkv), dtype=torch.uint8, device="cuda")
    out, ref = torch.zeros_like(q), torch.zeros_like(q)
    tq.tq_append_attend_int4(cs.h, kv[0], kv[1], *cs.caches, q, out, ws, pos=pos, scale=0.09)
    for x, c in zip(kv, other.caches):
        tq.tq_encode_int4(other.h, x, c, pos=pos)
    tq.tq_attend_int4(other.h, q, *other.caches, ref, ws, seq_lens=pos + Lq, scale=0.09)
    assert torch.equal(out, ref)
    for a, b in zip(cs.caches, other.caches):
        assert torch.equal(a.buf, b.buf)
    # the same without pos: every sequence at t0
    tq.tq_append_attend_int4(cs.h, kv[0], kv[1], *cs.caches, q, out, ws, t0=17, scale=0.09)
    for x, c in zip(kv, other.caches):
        tq.tq_encode_int4(other.h, x, c, t0=17)
    tq.tq_attend_int4(other.h, q, *other.caches, ref, ws, T=17 + Lq, scale=0.09)
    assert torch.equal(out, ref)
    cs.close()
    other.close()


@gpu
def test_graph_replay_streams_and_two_workspaces(libtq):
    """A captured step replays with new contents; two calls in flight on two streams with their own workspaces."""
    d, group, B, Hkv, G = 128, 64, 4, 2, 4
    cs, _, rng = _filled(d, group, B, Hkv, 256, 2)
    nb = tq.tq_attend_int4_workspace_bytes(cs.h, B, 1, Hkv * G, Hkv)
    ws = [torch.zeros(nb, dtype=torch.uint8, device="cuda") for _ in range(2)]
    q = to_gpu(rng.standard_normal((B, 1, Hkv * G, d)).astype(np.float32), "f16")
    kv = [to_gpu(rand(rng, (B, Hkv, 1, d)), "f16") for _ in range(2)]
    pos = torch.tensor([3, 64, 100, 200], dtype=torch.int32, device="cuda")
    out = torch.zeros_like(q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        tq.tq_append_attend_int4(cs.h, kv[0], kv[1], *cs.caches, q, out, ws[0], pos=pos, scale=0.1)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            tq.tq_append_attend_int4(cs.h, kv[0], kv[1], *cs.caches, q, out, ws[0], pos=pos, scale=0.1)
            pos += 1
    torch.cuda.synchronize()
    for step in range(3):
        at = pos.clone()
        for x in kv:
            x.copy_(torch.randn_like(x.float()).to(x.dtype))
        q.copy_(torch.randn_like(q.float()).to(q.dtype))
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        ref = torch.zeros_like(q)
        tq.tq_attend_int4(cs.h, q, *cs.caches, ref, ws[1], seq_lens=at + 1, scale=0.1)
        assert torch.equal(got, ref) and torch.equal(pos, at + 1)
    lens = torch.tensor([100, 256, 1, 77], dtype=torch.int32, device="cuda")
    alone = torch.zeros_like(q)
    tq.tq_attend_int4(cs.h, q, *cs.caches, alone, ws[0], seq_lens=lens, scale=0.1)
    outs = [torch.zeros_like(q) for _ in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        for st, o, w in zip(streams, outs, ws):
            tq.tq_attend_int4(cs.h, q, *cs.caches, o, w, seq_lens=lens, scale=0.1, stream=st)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], alone) and torch.equal(outs[1], alone)
    cs.close()


@gpu
def test_attend_gives_up_a_wait(libtq):
    """A bounded wait that runs out is reported, and the next call is right again."""
    cs, _, rng = _filled(128, 64, 2, 2, 256, 4)
    q = to_gpu(rng.standard_normal((2, 8, 128)).astype(np.float32), "f32")
    ws = torch.zeros(tq.tq_attend_int4_workspace_bytes(cs.h, 2, 1, 8, 2), dtype=torch.uint8, device="cuda")
    ref, out = torch.zeros_like(q), torch.zeros_like(q)
    tq.tq_attend_int4(cs.h, q, *cs.caches, ref, ws, T=250, scale=0.1)
    tq.tq_set_wait_limit(cs.h, 0)
    tq.tq_attend_int4(cs.h, q, *cs.caches, out, ws, T=250, scale=0.1)
    assert tq.tq_device_status(cs.h) == tq.TQ_ERR_DEVICE_CHECK
    tq.tq_set_wait_limit(cs.h, -1)
    tq.tq_attend_int4(cs.h, q, *cs.caches, out, ws, T=250, scale=0.1)
    assert torch.equal(out, ref)
    cs.close()


@gpu
def test_bad_block_table_entry_is_reported(libtq):
    cs, _, rng = _filled(128, 64, 2, 1, 192, 6, paged=True)
    q = to_gpu(rng.standard_normal((2, 4, 128)).astype(np.float32), "f32")
    ws = torch.zeros(tq.tq_attend_int4_workspace_bytes(cs.h, 2, 1, 4, 1), dtype=torch.uint8, device="cuda")
    ref, out = torch.zeros_like(q), torch.zeros_like(q)
    lens = torch.tensor([192, 100], dtype=torch.int32, device="cuda")
    tq.tq_attend_int4(cs.h, q, *cs.caches, ref, ws, seq_lens=lens, scale=0.1)
    cs.caches[1].block_table[1, 2] = cs.pool                      # behind sequence 1's tokens: not looked at
    tq.tq_attend_int4(cs.h, q, *cs.caches, out, ws, seq_lens=lens, scale=0.1)
    assert tq.tq_device_status(cs.h) == tq.TQ_OK and torch.equal(out, ref)
    for bad in (-1, cs.pool):
        cs.caches[0].block_table[0, 1] = bad
        tq.tq_attend_int4(cs.h, q, *cs.caches, out, ws, seq_lens=lens, scale=0.1)
        assert tq.tq_device_status(cs.h) == tq.TQ_ERR_DEVICE_CHECK
        assert torch.equal(out[1], ref[1])                        # (sequence 0 has read block 0 instead)
        before = cs.raw(0).copy()
        tq.tq_encode_int4(cs.h, torch.ones((2, 1, 3, 128), device="cuda"), cs.caches[0], t0=110)  # behind sequence 1's 100
        assert tq.tq_device_status(cs.h) == tq.TQ_ERR_DEVICE_CHECK
        changed = np.flatnonzero((cs.raw(0) != before).any(1))
        assert list(changed) in ([], [cs.ids[1][1]])
    cs.close()


@gpu
def test_refusals(libtq):
    """Arguments that are refused on the host leave everything as it was."""
    d, group = 128, 64
    cs, _, _ = _filled(d, group, 2, 2, 128, 1)
    h, (kc, vc) = cs.h, cs.caches
    q = torch.zeros((2, 1, 4, d), device="cuda")
    out = torch.full_like(q, 5.0)
    ws = torch.zeros(tq.tq_attend_int4_workspace_bytes(h, 2, 1, 4, 2) + 256, dtype=torch.uint8, device="cuda")
    L = libtq

    def attend(hd=h, g=group, qp=q.data_ptr(), dt=0, B=2, Lq=1, Hq=4, k=kc, v=vc, lens=None, T=10, scale=0.1,
               o=out.data_ptr(), w=ws.data_ptr(), wb=ws.numel()):
        return L.tq_attend_int4(hd, g, qp, dt, B, Lq, Hq, C.byref(k.struct), C.byref(v.struct), lens, T, scale, o, w, wb, None)

    inv = tq.TQ_ERR_INVALID_ARG
    for kw in (dict(hd=None), dict(g=16), dict(g=256), dict(qp=None), dict(dt=3), dict(B=3), dict(B=-1), dict(Lq=-1),
               dict(Hq=5), dict(Hq=0), dict(T=129), dict(T=-1), dict(scale=float("nan")), dict(scale=float("inf")),
               dict(o=None), dict(w=None), dict(w=ws.data_ptr() + 16), dict(lens=ws.data_ptr() + 1),
               dict(qp=q.data_ptr() + 2)):
        assert attend(**kw) == inv, kw
    assert attend(wb=tq.tq_attend_int4_workspace_bytes(h, 2, 1, 4, 2) - 1) == tq.TQ_ERR_WORKSPACE
    assert attend(Lq=1 << 40) == tq.TQ_ERR_UNSUPPORTED
    assert attend(Lq=0) == tq.TQ_OK
    x = torch.zeros((2, 2, 3, d), device="cuda")

    def copy(f, g=group, xp=x.data_ptr(), dt=0, B=2, Hkv=2, T=3, sb=6 * d, sh=3 * d, s=d, c=kc, pos=None, t0=0):
        return f(h, g, xp, dt, B, Hkv, T, sb, sh, s, C.byref(c.struct), pos, t0, None)

    before = cs.raw(0).copy()
    for f in (L.tq_encode_int4, L.tq_expand_int4):
        for kw in (dict(g=48), dict(xp=None), dict(dt=-1), dict(B=1), dict(Hkv=1), dict(T=-1), dict(T=129), dict(sb=-1),
                   dict(t0=-1), dict(t0=126), dict(t0=1 << 62), dict(T=1 << 62), dict(xp=x.data_ptr() + 1),
                   dict(pos=ws.data_ptr() + 2)):
            assert copy(f, **kw) == inv, kw
        assert copy(f, T=0) == tq.TQ_OK
    torch.cuda.synchronize()
    assert np.array_equal(cs.raw(0), before) and (out == 5).all() and not x.any()
    for bad in (q.double(), q[..., :64], q.transpose(1, 2)):
        with pytest.raises((ValueError, TypeError)):
            tq.tq_attend_int4(h, bad, kc, vc, out, ws, T=10)
    with pytest.raises(ValueError):
        tq.tq_attend_int4(h, q, kc, vc, out.half(), ws, T=10)
    with pytest.raises(ValueError):
        tq.tq_attend_int4(h, q, kc, tq.Int4Cache(d, 32, 2, 2, 128), out, ws, T=10)
    h64 = tq.tq_init(64, 0)
    with pytest.raises(ValueError):
        tq.tq_encode_int4(h64, x, kc)
    tq.tq_destroy(h64)
    with pytest.raises(tq.TQError):
        tq.tq_attend_int4(h, q, kc, tq.Int4Cache(d, group, 2, 2, 192), out, ws, T=10)
    cs.close()


@gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_chunk_queries_that_are_not_finite(libtq, dtype):
    """In a chunk too, a NaN or infinite query makes its own row NaN and no other."""
    cs, _, _ = _filled(128, 64, 1, 1, 128, 5)
    q = torch.randn((1, 50, 4, 128), device="cuda").to(TYPES[dtype])
    q[0, 3, 1, 7], q[0, 20, 0, 100], q[0, 49, 3, 0] = float("nan"), float("inf"), float("-inf")
    out = torch.zeros_like(q)
    ws = torch.zeros(tq.tq_attend_int4_workspace_bytes(cs.h, 1, 50, 4, 1), dtype=torch.uint8, device="cuda")
    tq.tq_attend_int4(cs.h, q, *cs.caches, out, ws, T=100, scale=0.1)
    rows = torch.isnan(out).any(-1)[0]
    assert torch.equal(rows, torch.isnan(out).all(-1)[0]) and int(rows.sum()) == 3
    assert rows[3, 1] and rows[20, 0] and rows[49, 3]
    cs.close()


@gpu
@pytest.mark.parametrize("Lq,dtype", [(1, "bf16"), (40, "bf16"), (40, "f32")])
def test_queries_off_a_16_byte_boundary(libtq, Lq, dtype):
    cs, _, rng = _filled(128, 64, 2, 2, 128, 8)
    n = 2 * Lq * 8 * 128
    q = to_gpu(rng.standard_normal(n).astype(np.float32), dtype).view(2, Lq, 8, 128)
    flat = [torch.zeros(n + 1, dtype=q.dtype, device="cuda") for _ in range(2)]
    q1, out1 = (f[1:].view(q.shape) for f in flat)
    q1.copy_(q)
    out = torch.zeros_like(q)
    ws = torch.zeros(tq.tq_attend_int4_workspace_bytes(cs.h, 2, Lq, 8, 2), dtype=torch.uint8, device="cuda")
    lens = torch.tensor([128, 60], dtype=torch.int32, device="cuda")
    tq.tq_attend_int4(cs.h, q, *cs.caches, out, ws, seq_lens=lens, scale=0.1)
    tq.tq_attend_int4(cs.h, q1, *cs.caches, out1, ws, seq_lens=lens, scale=0.1)
    assert torch.equal(out, out1)
    cs.close()


@gpu
def test_captured_chunk_replays_beside_another_graph(libtq):
    """Two graphs of chunk steps that share one workspace, replayed in turn with new contents."""
    d, group, B, Hkv, G, Lq = 128, 64, 2, 2, 4, 20
    cs, _, rng = _filled(d, group, B, Hkv, 320, 3)
    ws = torch.zeros(tq.tq_attend_int4_workspace_bytes(cs.h, B, Lq, Hkv * G, Hkv), dtype=torch.uint8, device="cuda")
    ws2 = torch.zeros_like(ws)
    q = [to_gpu(rng.standard_normal((B, Lq, Hkv * G, d)).astype(np.float32), "bf16") for _ in range(2)]
    kv = [to_gpu(rand(rng, (B, Hkv, Lq, d)), "bf16") for _ in range(2)]
    pos = [torch.tensor(p, dtype=torch.int32, device="cuda") for p in ([7, 200], [300, 0])]
    out = [torch.zeros_like(x) for x in q]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs = []
    with torch.cuda.stream(side):
        for i in range(2):
            g = torch.cuda.CUDAGraph()
            tq.tq_append_attend_int4(cs.h, kv[0], kv[1], *cs.caches, q[i], out[i], ws, pos=pos[i], scale=0.1)
            with torch.cuda.graph(g, stream=side):
                tq.tq_append_attend_int4(cs.h, kv[0], kv[1], *cs.caches, q[i], out[i], ws, pos=pos[i], scale=0.1)
            graphs.append(g)
    torch.cuda.synchronize()
    for _ in range(3):
        for x in kv + q:
            x.copy_(torch.randn_like(x.float()).to(x.dtype))
        for i in range(2):
            graphs[i].replay()
            torch.cuda.synchronize()
            ref = torch.zeros_like(q[i])
            tq.tq_attend_int4(cs.h, q[i], *cs.caches, ref, ws2, seq_lens=pos[i] + Lq, scale=0.1)
            assert torch.equal(out[i], ref)
    cs.close()


@gpu
@pytest.mark.parametrize("Lq", [1, 20])
def test_offsets_beyond_32_bits(libtq, Lq):
    """A pool of more than 4 GiB, its last pages in use."""
    d, group, n = 128, 64, 960000
    bb = tq.tq_int4_block_bytes(d, group)
    assert n * bb > 1 << 32
    h = tq.tq_init(d, 0)
    pool = torch.empty(n * bb, dtype=torch.uint8, device="cuda")
    far = torch.arange(n - 4, n, dtype=torch.int32, device="cuda").view(2, 2)
    near = torch.arange(4, dtype=torch.int32, device="cuda").view(2, 2)
    caches = [[tq.Int4Cache(d, group, 1, 2, 128, buf=pool[:n * bb], block_table=t, pool_blocks=n) for t in ((t_, t_))]
              for t_ in (far, near + 4)]
    x = torch.randn((1, 2, 128, d), device="cuda")
    q = torch.randn((1, Lq, 8, d), device="cuda")
    ws = torch.zeros(tq.tq_attend_int4_workspace_bytes(h, 1, Lq, 8, 2), dtype=torch.uint8, device="cuda")
    outs, back = [], []
    for kc, vc in caches:
        tq.tq_encode_int4(h, x, kc)
        out, b = torch.zeros_like(q), torch.zeros_like(x)
        tq.tq_attend_int4(h, q, kc, vc, out, ws, T=120, scale=0.1)
        tq.tq_expand_int4(h, kc, b)
        outs.append(out)
        back.append(b)
    assert torch.equal(outs[0], outs[1]) and torch.equal(back[0], back[1]) and outs[0].abs().sum() > 0
    pg = tq.Pages(far, torch.zeros(n, dtype=torch.int32, device="cuda"), 2, [(pool, bb)])
    tq.tq_pages_copy(h, pg, pg, far.view(-1), torch.arange(100, 104, dtype=torch.int32, device="cuda"))
    assert torch.equal(pool[100 * bb:104 * bb], pool[(n - 4) * bb:])
    assert tq.tq_device_status(h) == tq.TQ_OK
    tq.tq_destroy(h)


@gpu
def test_append_refuses_caches_that_share_blocks(libtq):
    d, group, B, Hkv = 128, 64, 2, 2
    h = tq.tq_init(d, 0)
    bb = tq.tq_int4_block_bytes(d, group)
    buf = torch.zeros(13 * bb, dtype=torch.uint8, device="cuda")
    table = torch.arange(4, dtype=torch.int32, device="cuda").view(4, 1)
    x, q = torch.randn((B, Hkv, 1, d), device="cuda"), torch.randn((B, 1, 4, d), device="cuda")
    out = torch.zeros_like(q)
    ws = torch.zeros(tq.tq_attend_int4_workspace_bytes(h, B, 1, 4, Hkv), dtype=torch.uint8, device="cuda")
    flat = [tq.Int4Cache(d, group, B, Hkv, 64, buf=buf[i * bb:]) for i in (0, 3, 4)]
    paged = [tq.Int4Cache(d, group, B, Hkv, 64, buf=buf, block_table=t, pool_blocks=13) for t in (table, table + 4)]

    def step(kc, vc, scale=0.1):
        tq.tq_append_attend_int4(h, x, x, kc, vc, q, out, ws, t0=3, scale=scale)

    for kc, vc in ((flat[0], flat[0]), (flat[0], flat[1]), (flat[1], flat[0]), (paged[0], paged[0])):
        with pytest.raises(tq.TQError):
            step(kc, vc)
    with pytest.raises(tq.TQError):
        step(flat[0], flat[2], scale=3e38)             # its product with log2 e is not finite
    torch.cuda.synchronize()
    assert not buf.any() and not out.any()
    step(flat[0], flat[2])
    step(*paged)
    assert tq.tq_device_status(h) == tq.TQ_OK and buf.any()
    tq.tq_destroy(h)


@gpu
@pytest.mark.parametrize("Lq", [1, 5])
def test_captured_serving_steps_on_pages(libtq, Lq):
    """One graph holds a step (supply pages, append and attend, release what lies behind the tokens); it is
    replayed over page borders and gives what a contiguous cache gives."""
    d, group, B, Hkv, G, NB = 128, 64, 3, 2, 4, 5
    h = tq.tq_init(d, 0)
    pool = 2 * B * Hkv * NB
    table = torch.full((B * Hkv, NB), -1, dtype=torch.int32, device="cuda")
    refs = torch.zeros(pool, dtype=torch.int32, device="cuda")
    paged = [tq.Int4Cache(d, group, B, Hkv, NB * 64, block_table=table, pool_blocks=pool) for _ in range(2)]
    plain = [tq.Int4Cache(d, group, B, Hkv, NB * 64) for _ in range(2)]
    pages = tq.Pages(table, refs, Hkv, paged)
    info = torch.zeros(2, dtype=torch.int32, device="cuda")
    pws = torch.zeros(tq.tq_pages_workspace_bytes(pages), dtype=torch.uint8, device="cuda")
    nws = tq.tq_attend_int4_workspace_bytes(h, B, Lq, Hkv * G, Hkv)
    ws, ws2 = (torch.zeros(nws, dtype=torch.uint8, device="cuda") for _ in range(2))
    pos = torch.tensor([0, 50, 63], dtype=torch.int32, device="cuda")
    zero, start = torch.zeros_like(pos), pos.clone()
    first = torch.randn((B, Hkv, 64, d), device="cuda").bfloat16()
    tq.tq_pages_alloc(h, pages, zero, start, info, pws)
    for b in range(1, B):
        for c in (paged, plain):
            for i, x in enumerate(c):
                rows = slice(b * Hkv, (b + 1) * Hkv)
                one = (tq.Int4Cache(d, group, 1, Hkv, NB * 64, buf=x.buf, block_table=table[rows], pool_blocks=pool) if c is paged
                       else tq.Int4Cache(d, group, 1, Hkv, NB * 64, buf=x.buf[b * Hkv * NB * x.block_bytes:]))
                tq.tq_encode_int4(h, first[b:b + 1, :, :int(start[b])], one)
    k, v = (torch.randn((B, Hkv, Lq, d), device="cuda").bfloat16() for _ in range(2))
    q = torch.randn((B, Lq, Hkv * G, d), device="cuda").bfloat16()
    out, ref, hi = torch.zeros_like(q), torch.zeros_like(q), torch.zeros_like(pos)

    def step():
        torch.add(pos, Lq, out=hi)
        tq.tq_pages_alloc(h, pages, pos, hi, info, pws)
        tq.tq_append_attend_int4(h, k, v, *paged, q, out, ws, pos=pos, scale=0.1)
        tq.tq_pages_free(h, pages, hi)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            step()
    torch.cuda.synchronize()
    for _ in range(220 // Lq):
        for x in (k, v, q):
            x.copy_(torch.randn_like(x.float()).to(x.dtype))
        graph.replay()
        tq.tq_append_attend_int4(h, k, v, *plain, q, ref, ws2, pos=pos, scale=0.1)
        torch.cuda.synchronize()
        assert torch.equal(out, ref) and int(info[1]) == 0
        pos += Lq
    held = (table >= 0).view(B, Hkv, NB).sum(-1)
    assert torch.equal(held, ((pos + 63) // 64)[:, None].expand(B, Hkv).long()) and int(refs.sum()) == int(held.sum())
    tq.tq_pages_free(h, pages, zero)
    assert not refs.any() and tq.tq_device_status(h) == tq.TQ_OK
    tq.tq_destroy(h)


@gpu
@pytest.mark.parametrize("Lq", [1, 20])
def test_calls_behind_joined_streams(libtq, Lq):
    """Every call waits for what its stream waits for, eagerly and captured: inputs made by slow kernels on two
    other streams, outputs read by a third."""
    d, group, B, Hkv, G = 128, 64, 2, 2, 4
    cs, _, _ = _filled(d, group, B, Hkv, 320, 9)
    h, (kc, vc) = cs.h, cs.caches
    pos = torch.tensor([100, 250], dtype=torch.int32, device="cuda")
    ws = torch.zeros(tq.tq_attend_int4_workspace_bytes(h, B, Lq, Hkv * G, Hkv), dtype=torch.uint8, device="cuda")
    seed_kv = torch.randn((B, Hkv, Lq, d), device="cuda").bfloat16()
    seed_q = torch.randn((B, Lq, Hkv * G, d), device="cuda").bfloat16()
    kv, q, out = torch.zeros_like(seed_kv), torch.zeros_like(seed_q), torch.zeros_like(seed_q)
    back, read = torch.zeros_like(seed_kv), [torch.zeros_like(seed_q), torch.zeros_like(seed_kv)]
    slow = torch.randn((4096, 4096), device="cuda")
    table = torch.full((B * Hkv, 5), -1, dtype=torch.int32, device="cuda")
    refs = torch.zeros(40, dtype=torch.int32, device="cuda")
    pages = tq.Pages(table, refs, Hkv, [])
    pws = torch.zeros(tq.tq_pages_workspace_bytes(pages), dtype=torch.uint8, device="cuda")
    lo, hi, seen = torch.zeros_like(pos), torch.zeros_like(pos), torch.zeros_like(table)
    s1, s2, s3 = (torch.cuda.Stream() for _ in range(3))

    def run(main):
        for s in (s1, s2, s3):
            s.wait_stream(main)
        with torch.cuda.stream(s1):
            (slow @ slow)
            kv.copy_(seed_kv)
            hi.copy_(pos)
        with torch.cuda.stream(s2):
            (slow @ slow) @ slow
            q.copy_(seed_q)
        main.wait_stream(s1)
        main.wait_stream(s2)
        tq.tq_append_attend_int4(h, kv, kv, kc, vc, q, out, ws, pos=pos, scale=0.1)
        tq.tq_expand_int4(h, kc, back, pos=pos)
        tq.tq_pages_alloc(h, pages, lo, hi, None, pws)
        s3.wait_stream(main)
        with torch.cuda.stream(s3):
            read[0].copy_(out)
            read[1].copy_(back)
            seen.copy_(table)
        main.wait_stream(s3)
        tq.tq_pages_free(h, pages, lo)

    def check():
        torch.cuda.synchronize()
        want, wb = torch.zeros_like(out), torch.zeros_like(back)
        tq.tq_attend_int4(h, seed_q, kc, vc, want, ws, seq_lens=pos + Lq, scale=0.1)
        tq.tq_expand_int4(h, kc, wb, pos=pos)
        assert torch.equal(read[0], want) and torch.equal(read[1], wb) and want.abs().sum() > 0
        assert torch.equal((seen >= 0).sum(1).view(B, Hkv), ((pos + 63) // 64)[:, None].expand(B, Hkv).long())
        assert (table == -1).all() and not refs.any()
        for t in (kv, q, out, back, hi, seen, *read):
            t.zero_()
        torch.cuda.synchronize()

    run(torch.cuda.current_stream())
    check()
    main = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(main):
        with torch.cuda.graph(graph, stream=main):
            run(main)
    for _ in range(2):
        graph.replay()
        check()
    cs.close()


def check_attend(d, group, dtype, kx, vx, qx, T, scale, limit=False):
    """Attention of qx [B, Lq, Hq, d] over T tokens of kx, vx [B, Hkv, T, d] encoded from fp32, every row against the
    oracle.  limit: values at the fp16 limit, whose bf16 operands stop at 65504: the top of a group lies at most
    15 scale 2^-11 <= 2^-10 V above it (scale rounded to 2^-11), so 2^-10 V on values and 2^-10 S on scores more."""
    B, Hkv = kx.shape[:2]
    Lq, G = qx.shape[1], qx.shape[2] // Hkv
    cs = Case(d, group, B, Hkv, -(-T // 64) * 64)
    for c, x in zip(cs.caches, (kx, vx)):
        tq.tq_encode_int4(cs.h, to_gpu(x, "f32"), c)
    q = to_gpu(qx, dtype)
    ws = torch.zeros(tq.tq_attend_int4_workspace_bytes(cs.h, B, Lq, Hkv * G, Hkv), dtype=torch.uint8, device="cuda")
    out = torch.full_like(q, float("nan"))
    tq.tq_attend_int4(cs.h, q, *cs.caches, out, ws, T=T, scale=scale)
    half = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}[dtype]
    got, qn = as_np(out).astype(np.float64), as_np(q).astype(np.float64)
    rounded = dtype == "bf16" and Lq * G > 8
    for b in range(B):
        for hh in range(Hkv):
            kc, ks, kz = U.quantise(kx[b, hh], group)
            k, v = U.values(kc, ks, kz, group), U.grid(vx[b, hh], group)
            kabs = U.values(kc, np.abs(ks), np.abs(kz), group)
            for g in range(G):
                rows = qn[b, :, hh * G + g]
                ref = U.attend(rows, k, v, scale, Lq)
                bound = U.attend_bound(rows, kabs, v, scale, ref, half, bf16=dtype == "bf16", rounded=rounded)
                if limit and rounded:
                    S = abs(scale) * (np.abs(rows) @ kabs.T).max(-1, keepdims=True)
                    bound = bound + np.abs(v).max() * 2.0 ** -10 * (1 + 2 * S)
                if dtype == "f16":
                    bound = bound + 2.0 ** -25
                err = np.abs(got[b, :, hh * G + g] - ref)
                assert np.isfinite(got[b, :, hh * G + g]).all() and (err <= bound).all(), (b, hh, g, err.max(), bound.max())
    cs.close()


@gpu
@pytest.mark.parametrize("d,group", [(64, 32), (128, 64), (128, 128), (256, 64)])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("Lq,T", [(1, 1), (1, 40), (2, 333), (12, 333)])
def test_constant_value_groups(libtq, d, group, dtype, Lq, T):
    """fp32 groups of one value: where the zero rounds above it the scale is negative (and no code uses it).  All
    tokens like that, and half of them beside ordinary ones."""
    rng = np.random.default_rng(d + T)
    for const in (0.3, 0.7, -0.1, 40020.0):
        vx = np.full((2, 1, T, d), const, np.float32)
        vx[1, 0, ::2] = rng.standard_normal((len(vx[1, 0, ::2]), d)) * min(abs(const), 1000.0)
        scales = U.quantise(vx[0, 0], group)[1]
        assert const == 40020.0 or (scales < 0).all() == (np.float32(np.float16(const)) > np.float32(const))
        check_attend(d, group, dtype, rand(rng, (2, 1, T, d)), vx, rng.standard_normal((2, Lq, 2, d)).astype(np.float32),
                     T, d ** -0.5)


@gpu
@pytest.mark.parametrize("d,dtype", [(64, "bf16"), (128, "bf16"), (128, "f16")])
@pytest.mark.parametrize("Tnew", [40, 1024])
def test_chunks_between_turboquant_encodes(libtq, d, dtype, Tnew):
    """Tensor-core encodes of a TurboQuant cache (small and bulk) and 4-bit chunks back to back on one stream: both
    hold tensor memory, and each starts its set-up while the one before it runs."""
    B, Hkv, G, Lq, T = 8, 2, 4, 20, 320
    cs, _, rng = _filled(d, 32, B, Hkv, T, 2)
    x = to_gpu(rng.standard_normal((B, Hkv, Tnew, d)).astype(np.float32), "bf16")
    q = to_gpu(rng.standard_normal((B, Lq, Hkv * G, d)).astype(np.float32), dtype)
    caches = [tq.Cache(d, k, B, Hkv, 1024) for k in (True, False)]
    ws = torch.zeros(tq.tq_attend_int4_workspace_bytes(cs.h, B, Lq, Hkv * G, Hkv), dtype=torch.uint8, device="cuda")

    def run(outs, apart):
        for out in outs:
            for f, c in zip((tq.tq_encode_k, tq.tq_encode_v), caches):
                f(cs.h, x, c, 0)
                tq.tq_attend_int4(cs.h, q, *cs.caches, out, ws, T=T, scale=0.1)
                if apart:
                    torch.cuda.synchronize()
        torch.cuda.synchronize()
        return outs, [c.buf.clone() for c in caches]

    want, stored = run([torch.zeros_like(q)], True)
    for c in caches:
        c.buf.zero_()
    got, again = run([torch.zeros_like(q) for _ in range(20)], False)
    assert all(torch.equal(o, want[0]) for o in got) and all(torch.equal(a, b) for a, b in zip(stored, again))
    cs.close()


def test_tensors_off_the_device_are_refused_cpu(libtq):
    """A host pointer would be followed by a kernel: refused before anything is called (the handle is not looked at)."""
    for dev, t in ((-1, ()), (0, (torch.zeros(1),)), (0, (None, torch.zeros(1)))):
        with pytest.raises(ValueError, match="current CUDA device"):
            tq._here("call", dev, *t)
    class OnGpu:
        get_device = staticmethod(lambda: 0)

    with pytest.raises(ValueError, match="one device"):
        tq._one_device("call", torch.zeros(1), OnGpu())
    assert tq._one_device("call", torch.zeros(1), None) == -1


@gpu
def test_tensors_off_the_device_are_refused(libtq):
    """Index vectors, queries, vectors, outputs, workspaces and caches on the host beside caches on the GPU."""
    d, group = 128, 64
    cs, _, _ = _filled(d, group, 2, 2, 128, 1)
    h, (kc, vc) = cs.h, cs.caches
    q, out = torch.zeros((2, 1, 4, d), device="cuda"), torch.zeros((2, 1, 4, d), device="cuda")
    x, lens = torch.zeros((2, 2, 1, d), device="cuda"), torch.tensor([5, 6], dtype=torch.int32, device="cuda")
    ws = torch.zeros(tq.tq_attend_int4_workspace_bytes(h, 2, 1, 4, 2), dtype=torch.uint8, device="cuda")
    host = tq.Int4Cache(d, group, 2, 2, 128, device="cpu")
    before = [c.buf.clone() for c in cs.caches]
    with pytest.raises(ValueError, match="one device"):
        tq.Int4Cache(d, group, 2, 2, 128, block_table=torch.zeros((4, 2), dtype=torch.int32), pool_blocks=8)
    good = dict(q=q, kc=kc, vc=vc, out=out, ws=ws, seq_lens=lens)
    for name in good:
        bad = dict(good, **{name: host if name in ("kc", "vc") else good[name].cpu()})
        with pytest.raises(ValueError, match="current CUDA device"):
            tq.tq_attend_int4(h, bad["q"], bad["kc"], bad["vc"], bad["out"], bad["ws"], seq_lens=bad["seq_lens"])
    good = dict(k=x, v=x, kc=kc, vc=vc, q=q, out=out, ws=ws, pos=lens)
    for name in good:
        bad = dict(good, **{name: host if name in ("kc", "vc") else good[name].cpu()})
        with pytest.raises(ValueError, match="current CUDA device"):
            tq.tq_append_attend_int4(h, *(bad[n] for n in ("k", "v", "kc", "vc", "q", "out", "ws")), pos=bad["pos"])
    for f in (lambda x, c, p: tq.tq_encode_int4(h, x, c, pos=p), lambda x, c, p: tq.tq_expand_int4(h, c, x, pos=p)):
        for args in ((x.cpu(), kc, lens), (x, host, lens), (x, kc, lens.cpu())):
            with pytest.raises(ValueError, match="current CUDA device"):
                f(*args)
    torch.cuda.synchronize()
    assert all(torch.equal(a, c.buf) for a, c in zip(before, cs.caches)) and not out.any()
    cs.close()


@gpu
@pytest.mark.parametrize("d,group", [(64, 32), (64, 64), (128, 64), (128, 128)])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("G,Lq", [(4, 1), (4, 10), (4, 80)])
def test_values_at_the_fp16_limit(libtq, d, group, dtype, G, Lq):
    """Groups clipped at 65504, whose zero + 15 scale may lie above it, as keys and as values: the same at 4, 40 and
    320 query rows."""
    rng = np.random.default_rng(d + group)
    T = 400
    kx, vx = (rng.standard_normal((1, 2, T, d)).astype(np.float32) * 5e4 for _ in range(2))
    top = U.grid(vx[0, 0], group)
    assert (top > 65504).any()
    check_attend(d, group, dtype, kx, vx, rng.standard_normal((1, Lq, 2 * G, d)).astype(np.float32), T, 1e-6, limit=True)


@gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("G,Lq", [(1, 4), (4, 30), (4, 50)])
def test_rows_that_see_nothing_are_zero_whatever_their_query(libtq, dtype, G, Lq):
    """A sequence shorter than its queries: the first rows see no token and give zeros, NaN or infinite queries too;
    a NaN in a row that sees tokens is its own."""
    cs, _, _ = _filled(128, 64, 2, 1, 128, 5)
    q = torch.randn((2, Lq, G, 128), device="cuda").to(TYPES[dtype])
    q[0, 0, 0, 7], q[0, 1, G - 1, 100], q[1, :, :, 3] = float("nan"), float("inf"), float("nan")
    q[0, Lq - 1, 0, 0] = float("nan")
    out = torch.full_like(q, 3.0)
    ws = torch.zeros(tq.tq_attend_int4_workspace_bytes(cs.h, 2, Lq, G, 1), dtype=torch.uint8, device="cuda")
    tq.tq_attend_int4(cs.h, q, *cs.caches, out, ws, seq_lens=torch.tensor([2, 0], dtype=torch.int32, device="cuda"),
                      scale=0.1)
    assert not out[0, :Lq - 2].any() and not out[1].any()
    assert torch.isnan(out[0, Lq - 1, 0]).all() and torch.isfinite(out[0, Lq - 2]).all()
    cs.close()


@gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("Lq", [1, 10, 40])
def test_nan_key_is_not_lost_beside_far_larger_scores(libtq, dtype, Lq):
    """A NaN score makes the row NaN although the other tokens of its tile have no weight beside those of the next
    tile (scores 256 and more apart).  Many sequences, so that one CTA holds both tiles."""
    d, B, G, T = 128, 300, 4, 192
    rng = np.random.default_rng(Lq)
    cs = Case(d, 64, B, 1, T)
    k, v = rand(rng, (B, 1, T, d)) * np.float32(0.05), rand(rng, (B, 1, T, d), False)
    k[:, :, 64:128] = 1.0                                    # q = 1: scores 128 scale
    k[::2, 0, 5, 70] = np.nan
    for c, x in zip(cs.caches, (k, v)):
        tq.tq_encode_int4(cs.h, to_gpu(x, "f32"), c)
    q = torch.ones((B, Lq, G, d), device="cuda", dtype=TYPES[dtype])
    out = torch.zeros_like(q)
    ws = torch.zeros(tq.tq_attend_int4_workspace_bytes(cs.h, B, Lq, G, 1), dtype=torch.uint8, device="cuda")
    tq.tq_attend_int4(cs.h, q, *cs.caches, out, ws, T=T, scale=2.0)
    bad = torch.isnan(out)
    assert bad[::2].all() and not bad[1::2].any()
    cs.close()


@gpu
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_chunk_sums_over_a_long_context(libtq, dtype):
    """Units enough that one CTA walks a whole unit of 1100 tiles, values with a mean of 1: the mean error of the
    outputs shows a drift of the sums, which the tensor core truncates, by up to 5.2e-7 a tile.  fp16 sums are taken
    out every 256 tiles (1.33e-4 < 2^-12.8, a quarter of the half step); fp32: 16 tiles (8.3e-6), 2^-17
    and the 2^-18 allowed everywhere; bf16 is not taken out: an eighth of the half step, 2^-11.  Beside it the mean
    of n roundings of half a step at most: 6 standard deviations.  The reference is rounded too: the grid is twice
    as fine below 1 as above, so roundings around a mean of 1 have a mean of their own, the same on both sides."""
    d, group, G, T = 128, 64, 8, 70400
    Lq = 148 * 256 // G
    h = tq.tq_init(d, 0)
    gen = torch.Generator(device="cuda").manual_seed(1)
    k = torch.randn((1, 1, T, d), generator=gen, device="cuda")
    v = 1.0 + 0.3 * torch.randn((1, 1, T, d), generator=gen, device="cuda")
    caches = [tq.Int4Cache(d, group, 1, 1, T) for _ in range(2)]
    back = [torch.empty_like(k) for _ in range(2)]
    for x, c, b in zip((k, v), caches, back):
        tq.tq_encode_int4(h, x, c)
        tq.tq_expand_int4(h, c, b)
    q = (2 * torch.randn((1, Lq, G, d), generator=gen, device="cuda")).to(TYPES[dtype])
    out = torch.zeros_like(q)
    ws = torch.zeros(tq.tq_attend_int4_workspace_bytes(h, 1, Lq, G, 1), dtype=torch.uint8, device="cuda")
    tq.tq_attend_int4(h, q, *caches, out, ws, T=T, scale=d ** -0.5)
    assert tq.tq_device_status(h) == tq.TQ_OK
    kd, vd = (b[0, 0].double() for b in back)
    rel = []
    for i in range(0, Lq, 97):
        n = T - Lq + 1 + i
        p = torch.softmax(q[0, i].double() @ kd[:n].T * d ** -0.5, -1)
        ref = p @ vd[:n]
        rel.append((out[0, i].double() - ref.to(out.dtype).double()) / ref)
    rel = torch.cat(rel)
    half = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}[dtype]
    drift = {"f32": 2.0 ** -17, "f16": 2.0 ** -12.8, "bf16": 2.0 ** -11}[dtype]
    noise = 2.0 ** -10 if dtype == "bf16" else 2.0 ** -18             # the rounded operands', of either sign
    assert abs(float(rel.mean())) <= drift + 2.0 ** -18 + 6 * (half + noise) / (3 * rel.numel()) ** 0.5
    tq.tq_destroy(h)


@gpu
@pytest.mark.parametrize("d,group", [(64, 32), (128, 64)])
@pytest.mark.parametrize("dtype,rows", [("bf16", 16), ("bf16", 17), ("f16", 32), ("f16", 33), ("f32", 32), ("f32", 33)])
def test_rows_on_both_sides_of_the_kernels_border(libtq, d, group, dtype, rows):
    """The last row count of the split kernel and the first of the chunk kernel, one unit cut over many CTAs and short
    sequences; the workspace holds whatever the queries' type."""
    run_attend(d, group, dtype, 1, 2, [6000, 70, rows - 3, 0], Lq=rows, seed=rows)
    h = tq.tq_init(d, 0)
    sizes = [tq.tq_attend_int4_workspace_bytes(h, 1, n, 1, 1) for n in (8, 16, 17, 32, 33, 129)]
    assert sizes == sorted(sizes)
    tq.tq_destroy(h)
