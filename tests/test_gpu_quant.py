"""The 8-bit K/V cache on the GPU: append, attention and eviction against the float64 oracle.

Codes, scales, tails, tables and counts must be equal bit for bit, and the summary rows must be
hga_build_summaries' bits.  Attention is held to a bound worked out from its arithmetic (see
`bounds`), so a rounding to fewer bits than the call documents would fail.
"""

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - collected on CPU too
    pytest.skip("needs a CUDA device", allow_module_level=True)

from hierarchical_sparse_attention_hga_b200 import binding as B  # noqa: E402
from oracle import hga_quant as Q  # noqa: E402

KIND = {"bf16": torch.bfloat16, "f32": torch.float32}
HGA = {"bf16": B.HGA_BF16, "f32": B.HGA_F32}
FORM = {"e4m3": B.HGA_QUANT_E4M3, "int8": B.HGA_QUANT_INT8}
SENTINEL = 0x5A


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from hierarchical_sparse_attention_hga_b200.build import build
    build()
    B.load_library()


def to_gpu(x, dtype):
    return torch.as_tensor(np.asarray(x), dtype=torch.float32).to(KIND[dtype]).cuda().contiguous()


def stored(x, dtype):
    """What the GPU sees of x, in float64."""
    return torch.as_tensor(np.asarray(x), dtype=torch.float32).to(KIND[dtype]).double().numpy()


class Cache:
    """A cache on the GPU, with sentinels where nothing may be written, and its oracle items."""

    def __init__(self, batch, heads_kv, dim, max_groups, dtype="bf16", fmt="e4m3", heads_q=None,
                 out="f32", seed=0, spare=3, n_slots=None, evicts=False, **layer):
        self.rng = np.random.default_rng(seed)
        self.b, self.h, self.d, self.max, self.dtype, self.fmt = batch, heads_kv, dim, max_groups, dtype, fmt
        self.hq = heads_q or heads_kv
        bh = batch * heads_kv
        self.n_slots = n_slots or bh * max_groups + spare
        order = self.rng.permutation(bh * max_groups + spare) + self.n_slots - (bh * max_groups + spare)
        self.table = torch.tensor(order[:bh * max_groups].reshape(batch, heads_kv, max_groups), dtype=torch.int32).cuda()
        self.k = torch.full((self.n_slots, 16, dim), SENTINEL, dtype=torch.uint8, device="cuda")
        self.v = torch.full_like(self.k, SENTINEL)
        self.ks = torch.full((self.n_slots,), float("nan"), device="cuda")
        self.vs = torch.full_like(self.ks, float("nan"))
        self.kt = torch.full((batch, heads_kv, 16, dim), float("nan"), dtype=KIND[dtype], device="cuda")
        self.vt = torch.full_like(self.kt, float("nan"))
        self.evicted = torch.zeros(batch, heads_kv, dtype=torch.int32, device="cuda") if evicts else None
        self.layer = B.Layer(batch=batch, heads_q=self.hq, heads_kv=heads_kv, head_dim=dim,
                             dtype=HGA[dtype], out_dtype=HGA[out],
                             **{"n_high_pairs": dim // 4, **layer})
        self.out_kind = KIND[out]
        self.items = [[Q.Item(fmt, dim) for _ in range(heads_kv)] for _ in range(batch)]
        self.pos = np.full(batch, -1, dtype=np.int64)

    def view(self):
        return B.quant_cache(self.k, self.v, self.ks, self.vs, self.kt, self.vt, self.table,
                             self.n_slots, self.max, FORM[self.fmt], self.evicted)

    def pos_t(self):
        return torch.tensor(self.pos, device="cuda")

    def append(self, k, v, counts=None, gpu=True, **kw):
        """k, v [B, Hkv, n, D]; counts[b] of them, or all."""
        n = k.shape[2]
        c = [n] * self.b if counts is None else counts
        self.pos = self.pos + np.asarray(c)
        for b in range(self.b):
            for h in range(self.h):
                self.items[b][h].append(stored(k[b, h, :c[b]], self.dtype), stored(v[b, h, :c[b]], self.dtype))
        if gpu:
            B.hga_quant_append(self.layer, self.view(), to_gpu(k, self.dtype), to_gpu(v, self.dtype), n,
                               self.pos_t(), counts=None if counts is None else torch.tensor(counts, dtype=torch.int32).cuda(), **kw)

    def fill(self, lens, spread=1.0):
        """Sequences of these lengths, appended in one padded call."""
        n = max(1, max(lens))
        k = spread * self.rng.standard_normal((self.b, self.h, n, self.d))
        v = spread * self.rng.standard_normal((self.b, self.h, n, self.d))
        self.append(k, v, list(lens))

    def check_stored(self):
        """Every live slot, scale and tail row is the oracle's, and nothing else was touched."""
        torch.cuda.synchronize()
        assert B.hga_device_status() == 0
        table = self.table.cpu().numpy()
        values = Q.code_values(self.fmt)
        for codes, scales, tail, name in ((self.k, self.ks, self.kt, "k"), (self.v, self.vs, self.vt, "v")):
            codes, scales, tail = codes.cpu().numpy(), scales.cpu().numpy(), tail.double().cpu().numpy()
            live = np.zeros(self.n_slots, bool)
            for b in range(self.b):
                for h in range(self.h):
                    it = self.items[b][h]
                    for e, (want, scale) in enumerate(getattr(it, name)):
                        slot = table[b, h, e]
                        live[slot] = True
                        np.testing.assert_array_equal(values[codes[slot]], want)
                        np.testing.assert_array_equal(scales[slot], scale)
                    rest = getattr(it, name + "_tail")
                    np.testing.assert_array_equal(tail[b, h, :len(rest)], rest)
            free = ~live
            if self.evicted is None:
                assert (codes[free] == SENTINEL).all() and np.isnan(scales[free]).all()

    def q(self, scale=1.0):
        return scale * self.rng.standard_normal((self.b, self.hq, 1, self.d))

    def attend(self, q, group_idx=None, weight=None, weight_out=None, ws=None, stream=None):
        out = torch.full((self.b, self.hq, 1, self.d), 7.0, dtype=self.out_kind, device="cuda")
        lse = torch.full((self.b, self.hq, 1), 7.0, device="cuda")
        need = B.hga_quant_attend_workspace_size(self.layer, self.max, weight is not None)
        if ws is None:  # scratch may hold anything
            ws = torch.full((max(16, need),), 0xFF, dtype=torch.uint8, device="cuda")
        B.hga_quant_attend(self.layer, self.view(), to_gpu(q, self.dtype), self.pos_t(), out, lse, group_idx,
                           weight, weight_out, ws, need, stream=stream)
        return out, lse

    def check_attend(self, q, got, entries=None, weight_in=None, weight_out=None, flagged=False):
        out, lse = (t.double().cpu().numpy()[:, :, 0] for t in (got[0], got[1][..., None]))
        torch.cuda.synchronize()
        assert B.hga_device_status() == (6 if flagged else 0)
        g = self.hq // self.h
        for b in range(self.b):
            for h in range(self.h):
                it = self.items[b][h]
                rows = slice(h * g, h * g + g)
                qq = stored(q[b, rows, 0], self.dtype)
                ids = None if entries is None else entries[b][h]
                want, want_lse, want_weight = it.attend(qq, ids)
                tol, tol_lse, tol_w = bounds(it, qq, ids, self.out_kind, want, want_lse)
                err = np.abs(out[b, rows] - want)
                assert (err <= tol).all(), (b, h, err.max(), np.max(err - tol))
                if np.isfinite(want_lse).all():
                    assert (np.abs(lse[b, rows, 0] - want_lse) <= tol_lse).all(), (b, h)
                else:
                    np.testing.assert_array_equal(lse[b, rows, 0], want_lse)
                if weight_in is not None:
                    n = len(want_weight)
                    w_in = weight_in[b, h].double().cpu().numpy()
                    w_got = weight_out[b, h].double().cpu().numpy()
                    full = w_in[:n] + want_weight
                    assert (np.abs(w_got[:n] - full) <= tol_w * want_weight + 2.0 ** -23 * np.abs(full) + 1e-30).all()
                    assert (w_got[n:] == -5).all()


def bounds(it, q, entries, out_kind, want, want_lse):
    """How far the call may be off, from its arithmetic.

    A score is a sum of D products, each of codes (exact in 11 bits) and 22-bit queries, summed in
    float32 (each addition of the tensor cores within 2^-22 of the largest term), then scaled: off
    by at most ds = (D + 8) 2^-22 max_t sum_d |q_d k_td| / sqrt(D), plus 2^-22 of the score itself
    (in the exponent).  A weight is then off by 2 ds relative, plus 2^-20 (the exponential's 2
    ulp, 22 bits in the product, the scales' roundings).  The sum over T tokens adds T/16 + 64
    float32 roundings of at most the largest partial sum (each 2^-23).  bfloat16 outputs add half a
    step."""
    entries = list(range(len(it.k))) if entries is None else entries
    k, v = it.rows("k", entries), it.rows("v", entries)
    if not len(k) or not np.isfinite(want).all():
        return np.zeros(want.shape), 0.0, 0.0
    root = np.sqrt(it.dim)
    size = (np.abs(q) @ np.abs(k).T) / root
    ds = (it.dim + 8) * 2.0 ** -22 * size.max(1) + 2.0 ** -22 * np.abs(q @ k.T / root).max(1)
    s = q @ k.T / root
    p = np.exp(s - want_lse[:, None])
    mag = p @ np.abs(v)
    rel = 2 * ds[:, None] + 2.0 ** -20 + (len(k) / 16 + 64) * 2.0 ** -23
    tol = mag * rel
    if out_kind is torch.bfloat16:
        tol = tol + (np.abs(want) + tol) * 2.0 ** -8
    tol_lse = ds + (len(k) / 16 + 64) * 2.0 ** -23 + 2.0 ** -22 * (1 + np.abs(want_lse))
    return tol + 1e-37, tol_lse, float(rel.max()) * 2


# ---- append


@pytest.mark.parametrize("dtype,fmt,dim,chunk,high", [
    ("bf16", "e4m3", 128, 64, 32), ("bf16", "int8", 64, 128, 0), ("f32", "e4m3", 64, 64, 32),
    ("f32", "int8", 128, 128, 64)])
def test_append_in_pieces_equals_one_call_and_the_oracle(dtype, fmt, dim, chunk, high):
    """A sequence cut into odd pieces: codes, scales and tails are the oracle's, the summary rows
    hga_build_summaries' bits, whatever the cut."""
    total = 401
    per = chunk // 16
    groups = 32
    tables = []
    rng = np.random.default_rng(1)
    k, v = rng.standard_normal((2, 2, 3, total, dim)) * np.exp(rng.standard_normal(dim))
    for cut in ([total], [1, 15, 16, 17, 1, 14, 2, 33, 64, 129, 100, 9], [1] * 70 + [total - 70]):
        c = Cache(2, 3, dim, groups, dtype, fmt, chunk=chunk, n_high_pairs=high)
        cs = torch.full((2, 3, groups // per, dim), 9.0, device="cuda")
        gs = torch.full((2, 3, groups // per, per, dim), 9.0, device="cuda")
        at = 0
        for n in cut:
            c.append(k[:, :, at:at + n], v[:, :, at:at + n], chunk_sum=cs, group_sum=gs)
            at += n
        assert at == total
        c.check_stored()
        tables.append((cs, gs))
    dense = torch.zeros(2, 3, groups * 16, dim)
    dense[:, :, :total] = torch.as_tensor(k, dtype=torch.float32)
    cs, gs = torch.full_like(tables[0][0], 9.0), torch.full_like(tables[0][1], 9.0)
    B.hga_build_summaries(c.layer, dense.to(KIND[dtype]).cuda(), groups * 16, 0, total, cs, gs)
    for got in tables:
        assert torch.equal(got[0], cs) and torch.equal(got[1], gs)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_append_ragged_counts_and_padding(fmt):
    """A padded batch: rows behind a sequence's count are NaN and never read, a count of 0 leaves
    its sequence as it is, also while it holds nothing."""
    c = Cache(4, 2, 128, 12, fmt=fmt, seed=2)
    for counts in ([0, 5, 48, 33], [1, 0, 16, 15], [7, 90, 0, 1], [0, 0, 0, 0], [16, 17, 18, 0]):
        n = 96
        k, v = c.rng.standard_normal((2, 4, 2, n, 128))
        for b in range(4):
            k[b, :, counts[b]:] = v[b, :, counts[b]:] = np.nan
        c.append(k, v, counts)
        c.check_stored()


def test_append_special_values():
    """Zeros, values below the cut-off, the largest bfloat16, an infinity and a NaN, each in a
    group of its own among ordinary ones."""
    c = Cache(1, 1, 64, 8, "bf16")
    k, v = c.rng.standard_normal((2, 1, 1, 128, 64))
    k[0, 0, :16] = 0
    v[0, 0, 16:32] = 2.0 ** -110
    k[0, 0, 35, 7] = np.inf
    v[0, 0, 50, 1] = -np.inf
    k[0, 0, 70, 3] = np.nan
    v[0, 0, 80:96] *= 3e37
    k[0, 0, 96:112] *= 1e-37
    c.append(k, v)
    c.check_stored()
    out, lse = c.attend(c.q())
    assert torch.isnan(out).all() and torch.isnan(lse).all()


def test_append_flags_what_does_not_fit():
    c = Cache(3, 2, 128, 4, seed=4, evicts=True)
    good = c.k.clone()
    new = c.rng.standard_normal((3, 2, 20, 128))
    for pos, counts, gone in (([18, 19, 19], None, 0), ([-1, 19, 19], None, 0), ([64, 19, 19], None, 0), ([2 ** 63 - 1, 19, 19], None, 0), ([-2 ** 63, 19, 19], None, 0),
                              ([19, 19, 19], [21, 20, 20], 0), ([19, 19, 19], [-1, 20, 20], 0),
                              ([19, 19, 19], None, 1), ([19, 19, 19], None, -1)):
        c.k.copy_(good)
        c.evicted.zero_()
        c.evicted[0] = gone
        B.hga_quant_append(c.layer, c.view(), to_gpu(new, "bf16"), to_gpu(new, "bf16"), 20, torch.tensor(pos).cuda(),
                           counts=None if counts is None else torch.tensor(counts, dtype=torch.int32).cuda())
        assert B.hga_device_status() == 6
        table = c.table.long().cpu()
        assert (c.k[table[0].flatten()] == SENTINEL).all()          # sequence 0 untouched
        assert not (c.k[table[1:, :, 0].flatten()] == SENTINEL).all(1).all(1).any()
    assert torch.isnan(c.kt[0]).all()


def test_append_skips_a_table_entry_that_is_no_slot():
    c = Cache(1, 2, 128, 4, seed=5)
    c.table[0, 0, 1] = c.n_slots
    c.table[0, 1, 0] = -1
    new = c.rng.standard_normal((1, 2, 64, 128))
    c.append(new, new)
    assert B.hga_device_status() == 6
    done = [(0, 0), (0, 2), (0, 3), (1, 1), (1, 2), (1, 3)]
    slots = [int(c.table[0, h, e]) for h, e in done]
    written = (c.k != SENTINEL).flatten(1).any(1).nonzero().flatten().tolist()
    assert sorted(slots) == written
    for (h, e), s in zip(done, slots):
        np.testing.assert_array_equal(Q.code_values("e4m3")[c.k[s].cpu().numpy()], c.items[0][h].k[e][0])


# ---- attend

LENS = [0, 1, 15, 16, 17, 31, 100, 257, 640, 1999]


@pytest.mark.parametrize("shared", [1, 2, 3, 4, 5, 8, 9, 16])
@pytest.mark.parametrize("dtype,fmt,dim,out", [
    ("bf16", "e4m3", 128, "f32"), ("bf16", "int8", 128, "bf16"), ("f32", "e4m3", 64, "f32"),
    ("f32", "int8", 128, "f32"), ("bf16", "int8", 64, "f32"), ("bf16", "e4m3", 64, "bf16")])
def test_attend_matches_the_oracle(shared, dtype, fmt, dim, out):
    """Ragged lengths from none to many, NaN in every free slot and free tail row, -1 in the
    table behind the live entries, with and without weights."""
    c = Cache(len(LENS), 2, dim, 130, dtype, fmt, heads_q=2 * shared, out=out, seed=shared)
    c.fill(LENS)
    for b, n in enumerate(LENS):
        c.table[b, :, n // 16:] = -1
    q = c.q(1.5)
    c.check_attend(q, c.attend(q))
    w_in = torch.rand(len(LENS), 2, 130, device="cuda")
    w_out = torch.full_like(w_in, -5)
    c.check_attend(q, c.attend(q, weight=w_in, weight_out=w_out), None, w_in, w_out)
    # in place, and the same bits
    both = w_in.clone()
    got = c.attend(q, weight=both, weight_out=both)
    again = c.attend(q)
    for b, n in enumerate(LENS):
        m = -(-n // 16)
        assert torch.equal(both[b, :, :m], w_out[b, :, :m]) and torch.equal(both[b, :, m:], w_in[b, :, m:])
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])


@pytest.mark.parametrize("batch,heads_kv,lens", [(1, 1, [20000]), (2, 1, [4097, 1]), (40, 8, None), (3, 2, [0, 0, 0])])
def test_attend_splits_of_every_kind(batch, heads_kv, lens):
    """One long item over many CTAs, many short ones in one, none at all."""
    rng = np.random.default_rng(7)
    lens = lens or [int(x) for x in rng.integers(0, 400, batch)]
    c = Cache(batch, heads_kv, 128, -(-max(max(lens), 1) // 16) + 1, "bf16", "e4m3", heads_q=4 * heads_kv, seed=8)
    c.fill(lens)
    q = c.q()
    w_in = torch.zeros(batch, heads_kv, c.max, device="cuda")
    w_out = torch.full_like(w_in, -5)
    c.check_attend(q, c.attend(q, weight=w_in, weight_out=w_out), None, w_in, w_out)
    c.check_attend(q, c.attend(q))


@pytest.mark.parametrize("dtype,fmt", [("bf16", "e4m3"), ("bf16", "int8"), ("f32", "e4m3")])
def test_attend_uneven_scales(dtype, fmt):
    """Groups whose K or V are zero, V sizes 2^-40 to 2^40 from group to group, one score far
    above the others, queries of very different sizes, a zero query."""
    n = 333
    c = Cache(2, 2, 128, 24, dtype, fmt, heads_q=12, seed=9)
    k, v = c.rng.standard_normal((2, 2, 2, n, 128))
    for g in range(n // 16 + 1):
        v[:, :, 16 * g:16 * g + 16] *= 2.0 ** c.rng.integers(-40, 41)
    k[:, :, 32:48] = 0
    v[:, :, 64:80] = 0
    v[1] = 0
    c.append(k, v)
    q = c.q() * np.logspace(-20, 1, 12)[None, :, None, None]
    q[0, 3] = 0
    q[:, 11] = 8 * k[:, 1, 100:101]
    c.check_attend(q, c.attend(q))


def test_attend_tail_values():
    """Tails of tiny, large and zero rows, beside closed groups and alone; values as small and as
    large as a tail's scale goes."""
    for dtype in ("bf16", "f32"):
        c = Cache(7, 1, 64, 4, dtype, heads_q=3, seed=10)
        k, v = c.rng.standard_normal((2, 7, 1, 27, 64))
        k[0] *= 1e-25
        v[1] *= 1e25
        v[2, 0, 16:] = 0
        k[3, 0, 20:] *= 50
        v[4] *= 1e-30
        v[5] *= 2.0 ** -110
        v[6] *= 1e36
        c.append(k, v, [27, 27, 27, 9, 27, 11, 5])
        q = c.q()
        c.check_attend(q, c.attend(q))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bad", [np.inf, -np.inf, np.nan])
def test_attend_what_is_not_finite(dtype, bad):
    """An infinity or NaN in the tail's K or V makes the item's heads NaN, as the closed group
    does; one in a query its own head; other items and heads keep their bits."""
    for where in ("k", "v", "q"):
        c = Cache(2, 2, 64, 4, dtype, heads_q=6, seed=23)
        k, v = c.rng.standard_normal((2, 2, 2, 41, 64))
        q = c.q()
        clean = Cache(2, 2, 64, 4, dtype, heads_q=6, seed=23)
        clean.append(k, v)
        right = clean.attend(q)
        if where == "q":
            q[1, 4, 0, 3] = bad
            hit = [(1, 4)]
        else:
            (k if where == "k" else v)[0, 1, 35, 5] = bad
            hit = [(0, 3), (0, 4), (0, 5)]
        c.append(k, v)
        got = c.attend(q)
        for b in range(2):
            for head in range(6):
                if (b, head) in hit:
                    assert torch.isnan(got[0][b, head]).all() and torch.isnan(got[1][b, head]).all()
                else:
                    assert torch.equal(got[0][b, head], right[0][b, head]) and torch.equal(got[1][b, head], right[1][b, head])
        if where != "q":
            out, lse, weight = c.items[0][1].attend(stored(q[0, 3:6, 0], dtype))
            assert np.isnan(out).all() and np.isnan(lse).all()


def routed_ids(rng, n, kg, chunk, sink, local):
    per, cur = chunk // 16, max(0, n - 1) // chunk
    lo, hi = sink * per, max(0, cur - local) * per
    m = min(kg, max(0, hi - lo))
    return sorted(int(g) + lo for g in rng.choice(hi - lo, m, replace=False)) if m else []


@pytest.mark.parametrize("chunk,sink,local,kg,shared,dim", [
    (64, 1, 4, 32, 4, 128), (128, 0, 0, 7, 1, 64), (64, 2, 1, 128, 16, 128), (128, 3, 2, 1, 8, 128)])
def test_attend_routed_sets(chunk, sink, local, kg, shared, dim):
    """Sinks, window and routed groups; ids that are -1, not ascending, twice there, in the
    window or outside the cache are skipped (and all but the -1 flagged)."""
    lens = [0, 1, 64, 129, 700, 1600, 2040]
    c = Cache(len(lens), 2, dim, 128, heads_q=2 * shared, seed=11, chunk=chunk, sink_chunks=sink,
              local_chunks=local, topk_groups=kg)
    c.fill(lens)
    idx = np.full((len(lens), 2, kg), -1, np.int32)
    entries = []
    for b, n in enumerate(lens):
        entries.append([])
        for h in range(2):
            ids = routed_ids(c.rng, n, kg, chunk, sink, local)
            idx[b, h, :len(ids)] = ids
            cur = max(0, n - 1) // chunk
            per = chunk // 16
            entries[b].append([g for g in range(n // 16) if g // per < sink or g // per >= cur - local or g in ids])
    q = c.q()
    w_in = torch.rand(len(lens), 2, 128, device="cuda")
    for w in (False, True):
        w_out = torch.full_like(w_in, -5)
        kw = dict(weight=w_in, weight_out=w_out) if w else {}
        got = c.attend(q, torch.tensor(idx).cuda(), **kw)
        c.check_attend(q, got, entries, *((w_in, w_out) if w else ()))
    if kg < 7:
        return
    bad = idx.copy()
    for h in range(2):
        ids = [g for g in bad[6, h] if g >= 0]
        keep = ids[: kg - 4]
        row = keep[:2] + [keep[1], 0x7fffffff, 2040 // 16 - 1] + keep[2:]
        bad[6, h] = (row + [-1] * kg)[:kg]
        window = [g for g in entries[6][h] if g not in ids]
        entries[6][h] = sorted(window + keep)
    got = c.attend(q, torch.tensor(bad).cuda())
    c.check_attend(q, got, entries, flagged=True)


def test_attend_flags_positions_and_slots():
    """A position that does not fit reads as an empty sequence, a table entry that is no slot is
    skipped; the other items are right."""
    c = Cache(4, 2, 128, 10, heads_q=8, seed=12)
    c.fill([100, 160, 33, 150])
    q = c.q()
    right = c.attend(q)
    saved = c.pos.copy()
    for bad in (-2, 160, 1 << 40, 2 ** 63 - 1, -2 ** 63):
        c.pos = saved.copy()
        c.pos[1] = bad
        out, lse = c.attend(q)
        assert B.hga_device_status() == 6
        assert not out[1].any() and torch.isneginf(lse[1]).all()
        assert torch.equal(out[0], right[0][0])
        np.testing.assert_allclose(out[2:].cpu(), right[0][2:].cpu(), atol=1e-5)
    c.pos = saved
    c.table[3, 0, 4] = -7
    c.table[3, 1, 8] = c.n_slots
    entries = [[list(range(n // 16)) for _ in range(2)] for n in (100, 160, 33, 150)]
    entries[3] = [[e for e in range(9) if e != 4], [e for e in range(9) if e != 8]]
    c.check_attend(q, c.attend(q), entries, flagged=True)


def test_attend_a_long_sequence_and_a_pool_past_4_gib():
    """200,003 tokens in slots behind the first 4 GiB of the pools."""
    n, dim = 200003, 128
    groups = n // 16 + 1
    c = Cache(1, 1, dim, groups, heads_q=4, seed=13, n_slots=(1 << 32) // (16 * dim) + groups + 200)
    assert int(c.table.min()) * 16 * dim >= 1 << 32
    c.fill([n])
    q = c.q(2.0)
    w_in = torch.zeros(1, 1, groups, device="cuda")
    w_out = torch.full_like(w_in, -5)
    c.check_attend(q, c.attend(q, weight=w_in, weight_out=w_out), None, w_in, w_out)


@pytest.mark.parametrize("batch,heads_kv,shared,longest", [(300, 8, 2, 60), (1100, 2, 1, 40), (3, 3, 4, 16)])
def test_attend_many_items_and_one_group(batch, heads_kv, shared, longest):
    """More (sequence, KV head) items than warps on the card, and tables of a single entry."""
    rng = np.random.default_rng(batch)
    lens = [int(x) for x in rng.integers(0, longest + 1, batch)]
    c = Cache(batch, heads_kv, 64, -(-longest // 16), heads_q=shared * heads_kv, seed=21)
    c.fill(lens)
    q = c.q()
    w_in = torch.rand(batch, heads_kv, c.max, device="cuda")
    w_out = torch.full_like(w_in, -5)
    c.check_attend(q, c.attend(q, weight=w_in, weight_out=w_out), None, w_in, w_out)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_attend_a_pool_that_others_filled(fmt):
    """Every finite code (int8 -128 among them), scales of any sign and size, zero and
    subnormal ones; no LSE asked for."""
    c = Cache(2, 2, 128, 20, fmt=fmt, heads_q=6, seed=22)
    values = Q.code_values(fmt)
    fine = np.flatnonzero(np.isfinite(values))
    c.pos[:] = [16 * 20 - 1, 16 * 7 - 1]
    table = c.table.cpu().numpy()
    for codes, scales, name, size in ((c.k, c.ks, "k", 0.02), (c.v, c.vs, "v", 1.0)):
        pool = c.rng.choice(fine, codes.shape).astype(np.uint8)
        sc = (size / 100 * np.exp(c.rng.standard_normal(c.n_slots)) * c.rng.choice([1, 1, 1, -1], c.n_slots)).astype(np.float32)
        sc[table[0, 0, 3]] = 0
        if name == "v":
            sc[table[0, 1, 4]] = 1e-40
            sc[table[1, 0, 2]] = 1e30
        codes.copy_(torch.tensor(pool))
        scales.copy_(torch.tensor(sc))
        for b, n in enumerate((20, 7)):
            for h in range(2):
                getattr(c.items[b][h], name).extend((values[pool[s]], sc[s]) for s in table[b, h, :n])
    q = c.q()
    got = c.attend(q)
    c.check_attend(q, got)
    out = torch.empty_like(got[0])
    need = B.hga_quant_attend_workspace_size(c.layer, c.max)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    B.hga_quant_attend(c.layer, c.view(), to_gpu(q, "bf16"), c.pos_t(), out, workspace=ws, workspace_bytes=need)
    assert torch.equal(out, got[0])


# ---- evict


def run_evict(c, weight, keep, sink, recent, in_place):
    w = weight.clone()
    table, gone = c.table.clone(), c.evicted.clone()
    outs = (w, table, gone) if in_place else (torch.full_like(w, -5), torch.full_like(table, -5), torch.full_like(gone, -5))
    v = c.view()
    if in_place:
        v = B.quant_cache(None, None, None, None, None, None, table, c.n_slots, c.max, evicted=gone)
    B.hga_quant_evict(c.layer, v, c.pos_t(), keep, sink, recent, w, *outs)
    torch.cuda.synchronize()
    return [t.cpu().numpy() for t in outs]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("max_groups,keep,sink,recent", [
    (9, 3, 1, 1), (40, 8, 0, 0), (40, 8, 4, 4), (40, 39, 0, 39), (700, 100, 4, 16), (5000, 1, 0, 0),
    (5000, 1, 0, 1), (5000, 4095, 4, 64)])
def test_evict_matches_the_oracle(max_groups, keep, sink, recent, in_place):
    """Ragged numbers of groups (none, fewer than the budget, a full table), many equal weights,
    NaN, infinities, both zeros and negative ones."""
    rng = np.random.default_rng(keep + sink)
    ns = sorted({0, 1, keep, min(keep + 1, max_groups), max_groups // 2, max_groups})
    for kind in range(3):
        c = Cache(len(ns), 2, 64, max_groups, seed=14, evicts=True)
        rest = rng.integers(0, 16, len(ns))
        gone = rng.integers(0, 9, (len(ns), 1)) * np.ones((1, 2), int)
        for i, n in enumerate(ns):
            if n == max_groups:
                rest[i] = 0
            c.pos[i] = 16 * (n + gone[i, 0]) + rest[i] - 1
            if c.pos[i] == -1:
                gone[i] = 0
        c.evicted.copy_(torch.tensor(gone))
        w = rng.standard_normal((len(ns), 2, max_groups)).astype(np.float32)
        if kind == 1:
            w = np.round(np.abs(w))                    # few different values
        if kind == 2:
            pick = rng.integers(0, 12, w.shape)
            for i, x in enumerate((np.nan, np.inf, -np.inf, 0.0, -0.0, 1e-42)):
                w[pick == i] = x
        got_w, got_t, got_e = run_evict(c, torch.tensor(w).cuda(), keep, sink, recent, in_place)
        assert B.hga_device_status() == 0
        table = c.table.cpu().numpy()
        for b, n in enumerate(ns):
            for h in range(2):
                stay = Q.keep_groups(w[b, h], n, keep, sink, recent)
                freed = [g for g in range(n) if g not in set(stay)]
                order = stay + freed + list(range(n, max_groups))
                np.testing.assert_array_equal(got_t[b, h], table[b, h, order])
                want = np.zeros(max_groups, np.float32)
                want[:len(stay)] = w[b, h, stay]
                if n < max_groups:
                    want[len(stay)] = w[b, h, n]
                np.testing.assert_array_equal(got_w[b, h], want)
                assert got_e[b, h] == gone[b, h] + len(freed)


def test_evict_largest_table():
    n = 49152
    c = Cache(1, 2, 64, n, seed=15, evicts=True)
    c.pos[0] = 16 * n - 1
    w = torch.rand(1, 2, n, device="cuda")
    got_w, got_t, got_e = run_evict(c, w, 30000, 4, 100, True)
    for h in range(2):
        stay = np.array(Q.keep_groups(w[0, h].cpu().numpy(), n, 30000, 4, 100))
        np.testing.assert_array_equal(got_t[0, h, :30000], c.table[0, h].cpu().numpy()[stay])
        np.testing.assert_array_equal(got_w[0, h, :30000], w[0, h].cpu().numpy()[stay])
        assert sorted(got_t[0, h]) == sorted(c.table[0, h].tolist()) and got_e[0, h] == n - 30000


def test_evict_passes_a_bad_position_through():
    c = Cache(2, 1, 64, 8, seed=16, evicts=True)
    c.pos[:] = [8 * 16, 5 * 16 - 1]
    w = torch.rand(2, 1, 8, device="cuda")
    got_w, got_t, got_e = run_evict(c, w, 2, 0, 0, False)
    assert B.hga_device_status() == 6
    np.testing.assert_array_equal(got_w[0], w[0].cpu())
    np.testing.assert_array_equal(got_t[0], c.table[0].cpu())
    assert got_e[0, 0] == 0 and got_e[1, 0] == 3


# ---- together


@pytest.mark.parametrize("dtype,fmt", [("bf16", "e4m3"), ("f32", "int8")])
def test_a_bounded_decode_loop(dtype, fmt):
    """Prompts of ragged lengths, then 70 tokens each: append, attend with weights, and a budget
    of 6 groups held by an eviction after every step.  Every step against the oracle."""
    keep, sink, recent = 6, 1, 2
    c = Cache(3, 2, 64, 16, dtype, fmt, heads_q=6, seed=17, evicts=True)
    c.fill([200, 37, 0])
    weight = torch.zeros(3, 2, 16, device="cuda")
    mine = [[np.zeros(16) for _ in range(2)] for _ in range(3)]
    for step in range(70):
        new = c.rng.standard_normal((2, 3, 2, 1, 64))
        c.append(new[0], new[1])
        q = c.q(1.5)
        got = c.attend(q, weight=weight, weight_out=weight)
        c.check_attend(q, got)
        g = c.hq // c.h
        for b in range(3):
            for h in range(2):
                it = c.items[b][h]
                w = it.attend(stored(q[b, h * g:h * g + g, 0], dtype))[2]
                mine[b][h][:len(w)] += w
                np.testing.assert_allclose(weight[b, h].cpu().numpy(), mine[b][h], rtol=2e-4, atol=1e-5)
                # the GPU's own sums decide what stays: equal but for rounding
                n = len(it.k)
                stay = Q.keep_groups(weight[b, h].cpu().numpy(), n, keep, sink, recent)
                it.k, it.v = [it.k[i] for i in stay], [it.v[i] for i in stay]
                tail = mine[b][h][n]
                mine[b][h] = np.concatenate([mine[b][h][stay], [tail], np.zeros(16 - len(stay) - 1)])
        B.hga_quant_evict(c.layer, c.view(), c.pos_t(), keep, sink, recent, weight, weight, c.table, c.evicted)
    # 270, 107 and 70 tokens: 16, 6 and 4 groups
    assert c.evicted.tolist() == [[10, 10], [0, 0], [0, 0]]
    c.check_stored()


def test_routed_decode_from_the_cache_alone():
    """No 16-bit cache anywhere: append writes the summaries, hga_route reads them, the attention
    reads the codes.  The routed ids are those of the bf16 path, the output the oracle's."""
    n0, steps = 1500, 40
    c = Cache(2, 2, 128, 100, heads_q=8, seed=18, topk_chunks=4, topk_groups=8, local_chunks=2, n_high_pairs=32)
    cs = torch.zeros(2, 2, 25, 128, device="cuda")
    gs = torch.zeros(2, 2, 25, 4, 128, device="cuda")
    k, v = c.rng.standard_normal((2, 2, 2, n0 + steps, 128))
    dense = torch.zeros(2, 2, 1600, 128, dtype=torch.bfloat16, device="cuda")
    dense[:, :, :n0 + steps] = to_gpu(k, "bf16")
    c.append(k[:, :, :n0], v[:, :, :n0], chunk_sum=cs, group_sum=gs)
    for t in range(n0, n0 + steps):
        c.append(k[:, :, t:t + 1], v[:, :, t:t + 1], chunk_sum=cs, group_sum=gs)
        ci = torch.empty(2, 2, 1, 4, dtype=torch.int32, device="cuda")
        gi = torch.empty(2, 2, 1, 8, dtype=torch.int32, device="cuda")
        q = c.q()
        B.hga_route(c.layer, to_gpu(q, "bf16"), 1, c.pos_t(), cs, gs, 1600, ci, gi)
        got = c.attend(q, gi)
        if t % 8 == 0 or t == n0 + steps - 1:
            cs2, gs2 = torch.zeros_like(cs), torch.zeros_like(gs)
            B.hga_build_summaries(c.layer, dense, 1600, 0, t + 1, cs2, gs2)
            ci2, gi2 = torch.empty_like(ci), torch.empty_like(gi)
            B.hga_route(c.layer, to_gpu(q, "bf16"), 1, c.pos_t(), cs2, gs2, 1600, ci2, gi2)
            assert torch.equal(gi, gi2)
            cur = t // 64
            entries = [[[g for g in range((t + 1) // 16) if g // 4 < 1 or g // 4 >= cur - 2 or g in set(gi[b, h, 0].tolist())]
                        for h in range(2)] for b in range(2)]
            c.check_attend(q, got, entries)


def test_two_graphs_on_two_streams():
    """Two captured decode loops, each with its workspace and cache, replayed at the same time
    with positions advanced on the device; and a graph's replay equals eager calls bit for bit."""
    runs = []
    for i in range(2):
        c = Cache(4, 2, 128, 60, heads_q=8, seed=20 + i, evicts=True)
        c.fill([300, 17, 640, 0])
        s = torch.cuda.Stream()
        pos = c.pos_t()
        q = to_gpu(c.q(), "bf16")
        new = to_gpu(c.rng.standard_normal((2, 4, 2, 1, 128)), "bf16")
        k1, v1 = new[0].contiguous(), new[1].contiguous()
        w = torch.zeros(4, 2, 60, device="cuda")
        out, lse = torch.zeros(4, 8, 1, 128, device="cuda"), torch.zeros(4, 8, 1, device="cuda")
        need = B.hga_quant_attend_workspace_size(c.layer, 60, True)
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")

        def step(c=c, pos=pos, q=q, k1=k1, v1=v1, w=w, out=out, lse=lse, ws=ws, need=need):
            pos.add_(1)
            B.hga_quant_append(c.layer, c.view(), k1, v1, 1, pos)
            B.hga_quant_attend(c.layer, c.view(), q, pos, out, lse, None, w, w, ws, need)
            B.hga_quant_evict(c.layer, c.view(), pos, 12, 1, 2, w, w, c.table, c.evicted)

        state = [pos, w, out, lse, c.table, c.evicted, c.k, c.v, c.ks, c.vs, c.kt, c.vt]
        runs.append((s, step, state, [t.clone() for t in state]))
    torch.cuda.synchronize()
    graphs = []
    for s, step, state, before in runs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            step()
        graphs.append(g)
    torch.cuda.synchronize()
    for (s, step, state, before) in runs:
        for t, x in zip(state, before):
            t.copy_(x)
    torch.cuda.synchronize()
    for _ in range(40):
        for g, (s, *_r) in zip(graphs, runs):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    after = [[t.clone() for t in state] for _, _, state, _ in runs]
    for (s, step, state, before), want in zip(runs, after):
        for t, x in zip(state, before):
            t.copy_(x)
        for _ in range(40):
            step()
        torch.cuda.synchronize()
        for t, x in zip(state, want):
            assert torch.equal(torch.nan_to_num(t.float()), torch.nan_to_num(x.float()))
    assert B.hga_device_status() == 0


# ---- scores that leave float32 no fraction


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("dtype,fmt,product", [
    ("bf16", "e4m3", 1e5), ("bf16", "int8", 1e6), ("f32", "e4m3", 1e8), ("bf16", "e4m3", 1e12),
    ("f32", "int8", 1e20), ("bf16", "e4m3", 1e30), ("f32", "e4m3", 1e34)])
def test_attend_scores_far_beyond_one_another(dtype, fmt, product, sign):
    """One token's score above the others' by millions to 1e35, all of them positive or all
    negative: its value is the output, whatever the size of its group's values.

    The softmax weight is 1 and the others' are 0 in 64 bits too, so only the arithmetic behind the
    score counts: two exponentials of 2 ulp (each 2^-23), 22 bits in the product, the division and
    the scales: 2^-20 in all, as in `bounds`.  A tail's values are held to 2^-39 of its largest.  The LSE is
    the score, a sum of D + 8 products summed within 2^-22 of their size."""
    size = product ** 0.5
    for at, lens in ((100, [333, 2000]), (331, [333, 2000]), (1999, [2000, 2000])):
        c = Cache(2, 2, 128, 130, dtype, fmt, heads_q=6, seed=31)
        n = max(lens)
        u = c.rng.choice([-1.0, 1.0], 128)
        k, v = c.rng.standard_normal((2, 2, 2, n, 128))
        if sign < 0:
            k = (2 + np.abs(k[..., :1])) * u
        for g in range(n // 16 + 1):
            v[:, :, 16 * g:16 * g + 16] *= 2.0 ** c.rng.integers(-20, 21)
        k[:, :, at] = (2.0 if sign > 0 else 0.5) * u
        c.append(size * k, v, lens)
        q = np.broadcast_to(sign * size * u, (2, 6, 1, 128)) * np.linspace(1, 2, 6)[None, :, None, None]
        w_in = torch.zeros(2, 2, 130, device="cuda")
        w_out = torch.full_like(w_in, -5)
        out, lse = (t.double().cpu().numpy() for t in c.attend(q, weight=w_in, weight_out=w_out))
        assert B.hga_device_status() == 0
        w_out = w_out.cpu().numpy()
        for b in range(2):
            if at >= lens[b]:
                continue
            for h in range(2):
                it = c.items[b][h]
                rows = slice(3 * h, 3 * h + 3)
                want, want_lse, weight = it.attend(stored(q[b, rows, 0], dtype))
                assert np.count_nonzero(weight) == 1 and weight.max() == 3
                tol = 2.0 ** -20 * np.abs(want) + 2.0 ** -38 * np.abs(it.rows("v", range(len(it.v)))[at // 16 * 16:][:16]).max()
                assert (np.abs(out[b, rows, 0] - want) <= tol).all(), (b, h, at)
                assert (np.abs(lse[b, rows, 0] - want_lse) <= (136 + 2) * 2.0 ** -22 * np.abs(want_lse)).all()
                np.testing.assert_allclose(w_out[b, h, :len(weight)], weight, rtol=2.0 ** -20, atol=0)


# ---- inputs that the kernel just before writes


class Late:
    """An input that hga_quant_evict, as a copier of 32-bit words, writes just before the call that
    reads it: that kernel releases its dependents before it has written anything, so a call that
    reads ahead of it finds what stood there before."""

    WORDS = 49152

    def __init__(self, right, stale):
        self.layer = B.Layer(batch=1, heads_q=1, heads_kv=1, head_dim=64)
        words = [t.contiguous().view(torch.int32).flatten() for t in (right, stale)]
        n = -(-words[0].numel() // 4) * 4
        assert n < self.WORDS
        self.src, self.old, self.dst = torch.zeros(3, self.WORDS, dtype=torch.int32, device="cuda")
        for buf, x in ((self.src, words[0]), (self.old, words[1])):
            buf[-n:][:x.numel()] = x
        self.tensor = self.dst[-n:][:words[0].numel()].view(right.dtype).view(right.shape)
        self.pos = torch.tensor([-1], device="cuda")
        self.weight = torch.zeros(2, self.WORDS, device="cuda")
        self.gone = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
        self.cache = B.quant_cache(None, None, None, None, None, None, self.src, 1, self.WORDS)

    def reset(self):
        self.dst.copy_(self.old)

    def write(self):
        B.hga_quant_evict(self.layer, self.cache, self.pos, 1, 0, 0, self.weight[0], self.weight[1], self.dst, self.gone)


def check_late(state, inputs, call):
    """call(inputs) -> leaves its results in the tensors `state`; each input in turn is written by
    the kernel before the call, over stale contents of the same type."""
    before = [t.clone() for t in state]

    def results(first, given):
        for t, x in zip(state, before):
            t.copy_(x)
        torch.cuda.synchronize()
        first()
        call(given)
        torch.cuda.synchronize()
        assert B.hga_device_status() == 0
        return [t.clone() for t in state]

    same = {k: right for k, (right, _) in inputs.items()}
    want = results(lambda: None, same)
    for name, (right, stale) in inputs.items():
        late = Late(right, stale)
        for _ in range(10):
            late.reset()
            for t, x in zip(results(late.write, {**same, name: late.tensor}), want):
                assert torch.equal(t.view(torch.uint8), x.view(torch.uint8)), name


@pytest.mark.parametrize("batch,evicts,routed", [(6, False, False), (6, True, False), (6, False, True), (150, False, False), (150, False, True)])
def test_attend_reads_behind_the_kernel_before(batch, evicts, routed):
    """Few sequences, whose positions are looked at ahead of the wait and again behind it, and
    more than a CTA has threads."""
    lens = ([0, 300, 17, 640, 1, 95] * 25)[:batch]
    layer = dict(topk_groups=8) if routed else {}
    c = Cache(batch, 2, 64, 41, heads_q=8, seed=32, evicts=evicts, **layer)
    c.fill(lens)
    out, lse = torch.empty(batch, 8, 1, 64, device="cuda"), torch.empty(batch, 8, 1, device="cuda")
    weight = torch.zeros(batch, 2, 41, device="cuda")
    need = B.hga_quant_attend_workspace_size(c.layer, 41, True)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    q, pos = to_gpu(c.q(), "bf16"), c.pos_t()
    stale = torch.tensor(([5, 30, 600, -1, 639, 80] * 25)[:batch], device="cuda")
    inputs = {"pos": (pos, stale), "weight": (torch.rand_like(weight), torch.full_like(weight, 9.0))}
    if batch == 6:
        inputs["q"] = (q, torch.full_like(q, float("nan")))
    if evicts:
        inputs["evicted"] = (c.evicted, c.evicted + torch.tensor([0, 5, 1, 20, 0, 2], device="cuda", dtype=torch.int32)[:, None])
    if routed:
        idx = torch.full((batch, 2, 8), -1, dtype=torch.int32)
        for b, n in enumerate(lens):
            for h in range(2):
                ids = routed_ids(c.rng, n, 8, 64, 1, 4)
                idx[b, h, :len(ids)] = torch.tensor(ids, dtype=torch.int32)
        inputs["group_idx"] = (idx.cuda(), torch.full_like(idx.cuda(), -1))

    def call(x):
        view = c.view()
        if evicts:
            view.evicted = x["evicted"].data_ptr()
        B.hga_quant_attend(c.layer, view, x.get("q", q), x["pos"], out, lse, x.get("group_idx"), x["weight"], weight, ws, need)

    check_late([out, lse, weight], inputs, call)


@pytest.mark.parametrize("max_groups", [40, 30000])
def test_evict_reads_behind_the_kernel_before(max_groups):
    c = Cache(1, 1, 64, max_groups, seed=33, evicts=True)
    c.pos[:] = 16 * (max_groups - 2) + 2
    w = torch.rand(1, 1, max_groups, device="cuda")
    outs = [torch.empty_like(w), torch.empty_like(c.table), torch.empty_like(c.evicted)]
    inputs = {"pos": (c.pos_t(), torch.tensor([16 * 5 - 1], device="cuda")), "weight": (w, torch.zeros_like(w)),
              "table": (c.table, torch.zeros_like(c.table)), "evicted": (c.evicted, c.evicted + 7)}

    def call(x):
        view = B.quant_cache(None, None, None, None, None, None, x["table"], c.n_slots, max_groups, evicted=x["evicted"])
        B.hga_quant_evict(c.layer, view, x["pos"], 11, 1, 2, x["weight"], *outs)

    check_late(outs, inputs, call)


@pytest.mark.parametrize("dtype,fmt,n", [("bf16", "e4m3", 1), ("bf16", "int8", 37), ("f32", "e4m3", 20)])
def test_append_reads_behind_the_kernel_before(dtype, fmt, n):
    c = Cache(4, 2, 64, 12, dtype, fmt, seed=34)
    c.fill([15, 0, 90, 31])
    cs, gs = torch.zeros(4, 2, 3, 64, device="cuda"), torch.rand(4, 2, 12, 64, device="cuda")
    k, v = (to_gpu(c.rng.standard_normal((4, 2, n, 64)), dtype) for _ in "kv")
    counts = torch.tensor([n, n // 2, n, 1], dtype=torch.int32, device="cuda")
    pos = c.pos_t() + counts
    inputs = {"pos": (pos, pos + 16), "counts": (counts, torch.zeros_like(counts)),
              "k": (k, torch.full_like(k, float("nan"))), "v": (v, torch.full_like(v, float("nan")))}

    def call(x):
        B.hga_quant_append(c.layer, c.view(), x["k"], x["v"], n, x["pos"], x["counts"], cs, gs)

    check_late([c.k, c.v, c.ks, c.vs, c.kt, c.vt, cs, gs], inputs, call)


# ---- a wait that gives up


@pytest.mark.parametrize("lens", [[5000], [60, 33, 200, 0, 47, 90], [700] * 40, [30000] * 4])
def test_attend_reports_a_copy_that_never_comes(lens):
    """A warp's first copies are withheld (nothing is in flight into that stage), its wait runs out:
    the call ends, the status is HGA_ERR_TIMEOUT, what the other warps attend counts, and the next
    call is right again."""
    c = Cache(len(lens), 2, 128, -(-max(lens) // 16) + 1, heads_q=8, seed=35)
    c.fill(lens)
    q = c.q()
    w_in = torch.zeros(len(lens), 2, c.max, device="cuda")
    w_out = torch.full_like(w_in, -5)
    right = c.attend(q, weight=w_in, weight_out=w_out)
    old = B.hga_debug_inject(2)
    try:
        w_bad = torch.full_like(w_in, -5)
        bad = c.attend(q, weight=w_in, weight_out=w_bad)
        torch.cuda.synchronize()
        assert B.hga_device_status() == 5
    finally:
        B.hga_debug_inject(old)
    # the first item's first groups are that warp's
    assert not w_bad[0, 0, 0].any() and w_out[0, 0, 0] > 0
    assert torch.isfinite(bad[0]).all() and (w_bad[w_out == -5] == -5).all()
    if len(lens) > 1:  # the last items are other warps'
        assert torch.equal(bad[0][-1], right[0][-1]) and torch.equal(w_bad[-1], w_out[-1])
    w_out.fill_(-5)
    c.check_attend(q, c.attend(q, weight=w_in, weight_out=w_out), None, w_in, w_out)


# ---- many routed groups


@pytest.mark.parametrize("dtype,fmt,dim,kg,shared,per_sm", [
    ("bf16", "e4m3", 128, 32, 4, 3), ("bf16", "e4m3", 128, 340, 4, 3), ("bf16", "int8", 128, 1024, 4, 2), ("f32", "e4m3", 128, 400, 8, 2),
    ("f32", "int8", 64, 1024, 3, 3), ("bf16", "e4m3", 128, 1024, 16, 2)])
def test_attend_many_routed_groups(dtype, fmt, dim, kg, shared, per_sm):
    """Up to 1024 routed groups, which take shared memory from the CTAs: the slices are cut for the
    warps of the CTAs that an SM holds then (148 SMs), and no warp has one beyond those.  A
    partial stands at its warp's number plus its item's."""
    lens = [20011, 333, 19000]
    c = Cache(3, 2, dim, 1256, dtype, fmt, heads_q=2 * shared, seed=36, topk_groups=kg, sink_chunks=1, local_chunks=4)
    c.fill(lens)
    idx = np.full((3, 2, kg), -1, np.int32)
    entries = []
    for b, n in enumerate(lens):
        entries.append([])
        cur = (n - 1) // 64
        for h in range(2):
            ids = routed_ids(c.rng, n, kg, 64, 1, 4)
            idx[b, h, :len(ids)] = ids
            chosen = set(ids)
            entries[b].append([g for g in range(n // 16) if g // 4 < 1 or g // 4 >= cur - 4 or g in chosen])
    q = c.q()
    w_in = torch.rand(3, 2, 1256, device="cuda")
    w_out = torch.full_like(w_in, -5)
    need = B.hga_quant_attend_workspace_size(c.layer, c.max, True)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    got = c.attend(q, torch.tensor(idx).cuda(), weight=w_in, weight_out=w_out, ws=ws)
    c.check_attend(q, got, entries, w_in, w_out)
    warps = 4 * per_sm * torch.cuda.get_device_properties(0).multi_processor_count
    most = 4 * (2 if shared > 8 else 3) * torch.cuda.get_device_properties(0).multi_processor_count
    last = int((ws[:(most + 6) * 256].view(-1, 256)[:, :16] != 0xFF).any(1).nonzero().max())
    assert last - 5 < warps
    if kg >= 400:  # long enough for a slice for most of them
        assert last - 5 >= warps // 2


# ---- values and weights far apart


def held_bound(it, q, want_lse):
    """What f16 operands add to `bounds`, per output element.  A weight p s (s: the group's v_scale, or
    2^(e - 14) for a tail whose largest element is in [2^e, 2^(e + 1))) is two halves, scaled so that
    the largest one met is at least 2^11: off by half a step of f16's smallest, 2^-25, that is by 2^-36
    of the largest p s, times the code.  A tail's element below f16's range is off by 2^-39 of
    the tail's largest, times its weight."""
    k, v = it.rows("k", range(len(it.k))), it.rows("v", range(len(it.v)))
    p = np.exp(q @ k.T / np.sqrt(it.dim) - want_lse[:, None])
    top = np.abs(it.v_tail).max() if len(it.v_tail) else 0.0
    tail_scale = 2.0 ** (np.floor(np.log2(top)) - 14) if top else 1.0
    s = np.concatenate([np.repeat([float(x[1]) for x in it.v], 16), np.full(len(it.v_tail), tail_scale)])
    code = np.abs(v) / np.where(s > 0, s, 1.0)[:, None]
    tail = p[:, 16 * len(it.v):].sum(1, keepdims=True) * top
    return 2.0 ** -36 * (p * s).max(1, keepdims=True) * code.sum(0) + 2.0 ** -39 * tail


def check_held(c, q, got):
    out = got[0].double().cpu().numpy()[:, :, 0]
    torch.cuda.synchronize()
    assert B.hga_device_status() == 0
    g = c.hq // c.h
    for b in range(c.b):
        for h in range(c.h):
            it, rows = c.items[b][h], slice(h * g, h * g + g)
            qq = stored(q[b, rows, 0], c.dtype)
            want, want_lse, _ = it.attend(qq)
            tol = bounds(it, qq, None, c.out_kind, want, want_lse)[0] + held_bound(it, qq, want_lse)
            err = np.abs(out[b, rows] - want)
            assert (err <= tol).all(), (b, h, np.max(err / tol))


@pytest.mark.parametrize("dtype,fmt,shared", [("bf16", "e4m3", 4), ("bf16", "int8", 8), ("f32", "e4m3", 3), ("bf16", "int8", 16)])
def test_attend_dimensions_that_only_light_groups_feed(dtype, fmt, shared):
    """Each group's V lives in 16 dimensions of its own, its size 2^0 to 2^-44 from group to group:
    every dimension is held to what the call documents."""
    c = Cache(2, 2, 128, 24, dtype, fmt, heads_q=2 * shared, seed=37)
    k, v = c.rng.standard_normal((2, 2, 2, 370, 128))
    for g in range(24):
        own = np.zeros(128)
        own[16 * (g % 8):16 * (g % 8) + 16] = 2.0 ** -(2 * g if g < 23 else 20)
        v[:, :, 16 * g:16 * g + 16] *= own
    c.append(k, v, [370, 352])
    q = c.q(0.5)
    check_held(c, q, c.attend(q))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attend_tail_rows_far_apart(dtype):
    """Rows of a tail from 2^30 to 2^-30, the weight on a small one: alone, and beside closed
    groups."""
    c = Cache(3, 2, 64, 4, dtype, heads_q=6, seed=38)
    k, v = c.rng.standard_normal((2, 3, 2, 43, 64))
    size = 2.0 ** c.rng.integers(-30, 31, (3, 2, 43, 1))
    size[:, :, 32:] = 2.0 ** np.linspace(30, -30, 11)[:, None]
    size[2, :, :13] = 2.0 ** np.linspace(-30, 30, 13)[:, None]
    v *= size
    c.append(k, v, [43, 32, 13])
    for at in (42, 38, 2):
        q = 6 * k[:, :, at].repeat(3, axis=1)[:, :, None]
        check_held(c, q, c.attend(q))


# ---- summaries of ragged and of bounded caches, rows of eviction that are read one after the other


def built(c, k, n_alloc):
    """Summary rows that hga_build_summaries makes of all tokens k [B, Hkv, n_alloc, D]."""
    chunks, per = n_alloc // c.layer.chunk, c.layer.chunk // 16
    cs = torch.full((c.b, c.h, chunks, c.d), 9.0, device="cuda")
    gs = torch.full((c.b, c.h, chunks, per, c.d), 9.0, device="cuda")
    B.hga_build_summaries(c.layer, to_gpu(k, c.dtype), n_alloc, 0, n_alloc, cs, gs)
    return cs, gs


@pytest.mark.parametrize("dtype,fmt,dim,chunk,high", [
    ("bf16", "e4m3", 128, 64, 32), ("bf16", "int8", 64, 128, 16), ("f32", "int8", 128, 128, 0), ("f32", "e4m3", 64, 64, 32)])
def test_append_ragged_with_summaries(dtype, fmt, dim, chunk, high):
    """Padded prompts of different lengths, then pieces of different lengths: each sequence's rows are
    the batch builder's bits, and no others are written."""
    n_alloc = 2048
    c = Cache(6, 2, dim, n_alloc // 16, dtype, fmt, seed=39, chunk=chunk, n_high_pairs=high)
    k, v = c.rng.standard_normal((2, 6, 2, n_alloc, dim))
    want_cs, want_gs = built(c, k, n_alloc)
    cs, gs = torch.full_like(want_cs, 9.0), torch.full_like(want_gs, 9.0)
    done = np.zeros(6, int)
    for counts in ([1900, 0, 15, 64, 333, 1024], [1, 17, 1, 65, 128, 0], [100, 300, 0, 700, 1, 1024]):
        n = max(counts)
        part = np.full((2, 6, 2, n, dim), np.nan)
        for b, m in enumerate(counts):
            part[0, b, :, :m], part[1, b, :, :m] = k[b, :, done[b]:done[b] + m], v[b, :, done[b]:done[b] + m]
        c.append(part[0], part[1], counts, chunk_sum=cs, group_sum=gs)
        done += counts
        c.check_stored()
        for b in range(6):
            groups, chunks = done[b] // 16, done[b] // chunk
            got, want = gs[b].flatten(1, 2), want_gs[b].flatten(1, 2)
            assert torch.equal(got[:, :groups], want[:, :groups]) and (got[:, groups:] == 9).all()
            assert torch.equal(cs[b, :, :chunks], want_cs[b, :, :chunks]) and (cs[b, :, chunks:] == 9).all()


def test_summaries_of_a_bounded_cache():
    """After evictions a group's table entry and its summary row are different numbers.  Rows go on
    being the batch builder's; a group behind the summary tables is flagged, its codes are written."""
    keep, total = 6, 256
    c = Cache(2, 2, 64, total // 16, heads_q=2, seed=40, evicts=True, n_high_pairs=16)
    k, v = c.rng.standard_normal((2, 2, 2, total + 32, 64))
    want_cs, want_gs = built(c, k[:, :, :total], total)
    cs, gs = torch.full_like(want_cs, 9.0), torch.full_like(want_gs, 9.0)
    weight = torch.zeros(2, 2, total // 16, device="cuda")
    at = 0
    for n in [100] + [1] * 30 + [37, 5, 16, 64, 4, 16, 16]:
        c.append(k[:, :, at:at + n], v[:, :, at:at + n], chunk_sum=cs, group_sum=gs)
        at += n
        assert B.hga_device_status() == (6 if at // 16 > 16 else 0)  # groups 16 and 17
        c.attend(c.q(), weight=weight, weight_out=weight)
        given = weight.cpu().numpy()
        B.hga_quant_evict(c.layer, c.view(), c.pos_t(), keep, 1, 2, weight, weight, c.table, c.evicted)
        for b in range(2):
            for h in range(2):
                it = c.items[b][h]
                stay = Q.keep_groups(given[b, h], len(it.k), keep, 1, 2)
                it.k, it.v = [it.k[i] for i in stay], [it.v[i] for i in stay]
        c.check_stored()
    assert at == total + 32 and (c.evicted == 18 - keep).all()
    assert torch.equal(gs, want_gs) and torch.equal(cs, want_cs)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("keep,sink,recent", [(1, 0, 0), (20000, 4, 64), (29999, 0, 0)])
def test_evict_rows_beyond_shared_memory(keep, sink, recent, in_place):
    """Tables of 30,000 entries (weights, then slots, go through shared memory): ragged numbers of
    groups, weights that tie across the threshold, NaN, open groups, a bad position."""
    total = 30000
    rng = np.random.default_rng(keep)
    ns = [0, 1, keep, keep + 1, 25013, total]
    c = Cache(len(ns) + 1, 2, 64, total, seed=41, evicts=True)
    for i, n in enumerate(ns):
        c.pos[i] = 16 * n + (0 if n == total else 7 * i % 16) - 1
    c.pos[-1] = 16 * total + 5                        # a group too many
    w = np.round(rng.standard_normal((len(ns) + 1, 2, total)).astype(np.float32) * 2)  # few different values
    w[rng.integers(0, 50, w.shape) == 0] = np.nan
    got_w, got_t, got_e = run_evict(c, torch.tensor(w).cuda(), keep, sink, recent, in_place)
    assert B.hga_device_status() == 6
    table = c.table.cpu().numpy()
    np.testing.assert_array_equal(got_w[-1], w[-1])
    np.testing.assert_array_equal(got_t[-1], table[-1])
    assert not got_e[-1].any()
    for b, n in enumerate(ns):
        for h in range(2):
            stay = Q.keep_groups(w[b, h], n, keep, sink, recent)
            kept = set(stay)
            freed = [g for g in range(n) if g not in kept]
            np.testing.assert_array_equal(got_t[b, h], table[b, h, stay + freed + list(range(n, total))])
            want = np.zeros(total, np.float32)
            want[:len(stay)] = w[b, h, stay]
            if n < total:
                want[len(stay)] = w[b, h, n]
            np.testing.assert_array_equal(got_w[b, h], want)
            assert got_e[b, h] == len(freed)


# ---- the last positions


def test_positions_end_where_the_count_of_evicted_groups_does():
    """2^35 - 2 is the last position: the groups before it fit an int32.  The next one is flagged, and
    an eviction there, whose count would pass 2^31, leaves its item as it is."""
    c = Cache(2, 2, 64, 8, heads_q=4, seed=42, evicts=True)
    c.fill([3 * 16 + 14, 7 * 16 + 14])
    c.evicted[0], c.evicted[1] = 2 ** 31 - 1 - 3, 2 ** 31 - 1 - 7
    c.pos += 16 * c.evicted[:, 0].cpu().numpy().astype(np.int64)
    new = c.rng.standard_normal((2, 2, 2, 1, 64))
    c.append(new[0], new[1])
    assert (c.pos == 2 ** 35 - 2).all()
    c.check_stored()
    q = c.q()
    weight = torch.rand(2, 2, 8, device="cuda")
    w_out = torch.full_like(weight, -5)
    c.check_attend(q, c.attend(q, weight=weight, weight_out=w_out), None, weight, w_out)
    _, _, got_e = run_evict(c, weight, 2, 0, 1, False)
    assert (got_e == 2 ** 31 - 3).all() and B.hga_device_status() == 0
    tail = c.kt.clone()
    B.hga_quant_append(c.layer, c.view(), to_gpu(new[0], "bf16"), to_gpu(new[1], "bf16"), 1, c.pos_t() + 1)
    assert B.hga_device_status() == 6 and torch.equal(torch.nan_to_num(c.kt), torch.nan_to_num(tail))
    c.pos += 16 * 3                                   # as if appended: 2^31 + 2 groups in all
    c.evicted += 3
    got_w, got_t, got_e = run_evict(c, weight, 2, 0, 1, False)
    assert B.hga_device_status() == 6
    np.testing.assert_array_equal(got_e, c.evicted.cpu().numpy())
    np.testing.assert_array_equal(got_t, c.table.cpu().numpy())
    np.testing.assert_array_equal(got_w, weight.cpu().numpy())
    out, lse = c.attend(q)
    assert B.hga_device_status() == 6 and not out.any() and torch.isneginf(lse).all()
