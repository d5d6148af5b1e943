"""The 8-bit K/V cache without a GPU: the oracle against independent definitions, and what the
entry points refuse on the host (before any CUDA call)."""

import ctypes
import itertools

import numpy as np
import pytest
import torch

from hierarchical_sparse_attention_hga_b200 import binding as B
from oracle import hga_quant as Q

LAYER = dict(batch=2, heads_q=8, heads_kv=2, head_dim=128)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from hierarchical_sparse_attention_hga_b200.build import build
    build()
    B.load_library()


# ---- the oracle


def test_e4m3_values_are_torchs():
    want = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(Q.code_values("e4m3"), want)
    want = torch.arange(256, dtype=torch.uint8).view(torch.int8).double().numpy()
    np.testing.assert_array_equal(Q.code_values("int8"), want)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("size", [1e-25, 1e-3, 1.0, 7e4, 1e30])
def test_quantise_rounds_to_the_nearest_code(fmt, size):
    """Every value is within half a step of its code (a step is the distance between the codes
    around it) and the largest one takes the peak."""
    x = (size * np.random.default_rng(3).standard_normal((16, 64))).astype(np.float32)
    code, scale = Q.quantise(x, fmt)
    values = np.unique(Q.code_values(fmt)[np.isfinite(Q.code_values(fmt))])
    assert np.isin(code, values).all() and np.abs(code).max() == Q.PEAK[fmt]
    y = x.astype(np.float64) * Q.PEAK[fmt] / np.abs(x.astype(np.float64)).max()
    nearest = np.abs(y[..., None] - values).min(-1)
    # float32's quotient and product may move y by 2^-23 of itself
    assert (np.abs(y - code) <= nearest + np.abs(y) * 2.0 ** -22).all()


def test_quantise_special_groups():
    zero = np.zeros((16, 4), np.float32)
    for x in (zero, zero + np.float32(2.0 ** -101)):
        code, scale = Q.quantise(x, "e4m3")
        assert scale == 0 and not code.any()
    for bad in (np.inf, -np.inf, np.nan):
        x = zero.copy()
        x[3, 1] = bad
        code, scale = Q.quantise(x, "int8")
        assert np.isnan(scale) and not code.any()


@pytest.mark.parametrize("n", [1, 15, 16, 17, 64, 77])
def test_attend_is_dense_attention_over_the_decoded_cache(n):
    r = np.random.default_rng(n)
    k, v, q = r.standard_normal((n, 32)), r.standard_normal((n, 32)), r.standard_normal((3, 32))
    it = Q.Item("e4m3", 32)
    for a in range(0, n, 5):                       # in pieces
        it.append(k[a:a + 5], v[a:a + 5])
    kk, vv = it.rows("k", range(len(it.k))), it.rows("v", range(len(it.v)))
    assert len(kk) == n and len(it.k) == n // 16
    want = torch.nn.functional.scaled_dot_product_attention(
        *(torch.tensor(t)[None] for t in (q, kk, vv)))[0].numpy()
    out, lse, weight = it.attend(q)
    np.testing.assert_allclose(out, want, atol=1e-13)
    np.testing.assert_allclose(lse, torch.logsumexp(torch.tensor(q @ kk.T) / 32 ** 0.5, 1), atol=1e-13)
    assert abs(weight.sum() - 3) < 1e-12 and len(weight) == -(-n // 16)


def test_keep_groups_is_the_best_subset():
    """Against brute force: no other choice of the middle groups weighs more, and among equal
    ones it is the first in order."""
    r = np.random.default_rng(5)
    for _ in range(40):
        n, keep = int(r.integers(1, 9)), int(r.integers(1, 9))
        sink = int(r.integers(0, keep + 1))
        recent = int(r.integers(0, keep - sink + 1))
        w = r.integers(0, 3, n).astype(float)
        got = Q.keep_groups(w, n, keep, sink, recent)
        if n <= keep:
            assert got == list(range(n))
            continue
        fixed = set(range(sink)) | set(range(n - recent, n))
        middle = [g for g in range(n) if g not in fixed]
        best = max(itertools.combinations(middle, keep - len(fixed)),
                   key=lambda c: (sum(w[list(c)]), [-g for g in c]))
        assert got == sorted(fixed | set(best))


# ---- refusals


def cache(**kw):
    base = dict(k=16, v=16, k_scale=16, v_scale=16, k_tail=16, v_tail=16, table=16, n_slots=8,
                max_groups=4, format=B.HGA_QUANT_E4M3, evicted=None)
    base.update(kw)
    return B.quant_cache(**base)


def refused(status, fn, *a, **kw):
    with pytest.raises(B.HGAError) as e:
        fn(*a, stream=0, **kw)
    assert e.value.status == status and B.load_library().hga_last_error()


def test_struct_layout():
    assert ctypes.sizeof(B.HGAQuantCache) == 8 * 8 + 8 + 8
    assert B.HGAQuantCache.n_slots.offset == 64 and B.HGAQuantCache.format.offset == 76


@pytest.mark.parametrize("kw,status", [
    (dict(table=None), 1), (dict(format=2), 1), (dict(max_groups=0), 1), (dict(n_slots=0), 1),
    (dict(max_groups=(1 << 20) + 1), 3), (dict(n_slots=1 << 27), 3), (dict(k=None), 1),
    (dict(v_scale=None), 1), (dict(k_tail=None), 1), (dict(v=24), 1), (dict(v_tail=8), 1)])
def test_a_cache_that_append_and_attend_refuse(kw, status):
    layer = B.Layer(**LAYER)
    refused(status, B.hga_quant_append, layer, cache(**kw), 16, 16, 1, 16)
    refused(status, B.hga_quant_attend, layer, cache(**kw), 16, 16, 16, workspace=16,
            workspace_bytes=1 << 40)


@pytest.mark.parametrize("kw,status", [
    (dict(head_dim=96), 3), (dict(group=8), 3), (dict(heads_q=7), 2), (dict(dtype=2), 1),
    (dict(heads_q=64), 3), (dict(kv_loc=B.HGA_KV_HOST_PINNED), 3)])
def test_layers_that_are_refused(kw, status):
    layer = B.Layer(**{**LAYER, **kw})
    refused(status, B.hga_quant_append, layer, cache(), 16, 16, 1, 16)
    refused(status, B.hga_quant_attend, layer, cache(), 16, 16, 16, workspace=16,
            workspace_bytes=1 << 40)
    refused(status, B.hga_quant_evict, layer, cache(), 16, 4, 1, 1, 16, 16, 16, 16)


def test_append_arguments():
    layer, c = B.Layer(**LAYER), cache()
    refused(1, B.hga_quant_append, layer, c, None, 16, 1, 16)
    refused(1, B.hga_quant_append, layer, c, 16, 16, 1, None)
    refused(1, B.hga_quant_append, layer, c, 16, 16, 0, 16)
    refused(1, B.hga_quant_append, layer, c, 20, 16, 1, 16)               # alignment
    refused(1, B.hga_quant_append, layer, c, 16, 16, 1, 16, chunk_sum=16)  # without group_sum
    refused(2, B.hga_quant_append, layer, cache(max_groups=6), 16, 16, 1, 16, chunk_sum=16,
            group_sum=16)


def test_attend_arguments():
    layer, c = B.Layer(**LAYER), cache()
    ws = dict(workspace=16, workspace_bytes=1 << 40)
    refused(1, B.hga_quant_attend, layer, c, None, 16, 16, **ws)
    refused(1, B.hga_quant_attend, layer, c, 16, 16, None, **ws)
    refused(1, B.hga_quant_attend, layer, c, 18, 16, 16, **ws)
    refused(1, B.hga_quant_attend, layer, c, 16, 16, 16, weight_out=16, **ws)
    refused(1, B.hga_quant_attend, layer, c, 16, 16, 16, weight_in=16, **ws)
    refused(1, B.hga_quant_attend, layer, cache(evicted=16), 16, 16, 16, group_idx=16, **ws)
    need = B.hga_quant_attend_workspace_size(layer, 4, True)
    assert need > 0
    refused(7, B.hga_quant_attend, layer, c, 16, 16, 16, weight_in=16, weight_out=16, workspace=16,
            workspace_bytes=need - 1)
    refused(7, B.hga_quant_attend, layer, c, 16, 16, 16, weight_in=16, weight_out=16)
    refused(1, B.hga_quant_attend, layer, c, 16, 16, 16, weight_in=16, weight_out=16, workspace=24,
            workspace_bytes=1 << 40)


def test_workspace_size_grows_and_refuses():
    small = B.hga_quant_attend_workspace_size(B.Layer(**LAYER), 64, True)
    assert small < B.hga_quant_attend_workspace_size(B.Layer(**LAYER), 128, True)
    assert small >= B.hga_quant_attend_workspace_size(B.Layer(**LAYER), 64, False)
    for groups, status in ((0, 1), (-1, 1), ((1 << 20) + 1, 3)):
        with pytest.raises(B.HGAError) as e:
            B.hga_quant_attend_workspace_size(B.Layer(**LAYER), groups)
        assert e.value.status == status


@pytest.mark.parametrize("keep,sink,recent", [(0, 0, 0), (-1, 0, 0), (4, -1, 0), (4, 0, -1),
                                              (4, 3, 2), (4, 2 ** 31 - 1, 2 ** 31 - 1),
                                              (2 ** 31 - 1, 2 ** 31 - 1, 1)])
def test_evict_budgets_that_are_refused(keep, sink, recent):
    refused(1, B.hga_quant_evict, B.Layer(**LAYER), cache(), 16, keep, sink, recent, 16, 16, 16, 16)


def test_evict_arguments():
    layer = B.Layer(**LAYER)
    for i in range(5):
        a = [16] * 5                                # pos, weights, table_out, evicted_out
        a[i] = None
        refused(1, B.hga_quant_evict, layer, cache(), a[0], 4, 1, 1, *a[1:])
    refused(3, B.hga_quant_evict, layer, cache(max_groups=49153, n_slots=1 << 20), 16, 4, 1, 1, 16,
            16, 16, 16)


def test_slices_of_larger_tensors_are_refused():
    """The calls take whole arrays: a slice of a batch that is not contiguous would be read
    wrongly."""
    layer = B.Layer(**LAYER)
    big = torch.zeros(2, 2, 64, 128, dtype=torch.bfloat16)
    part = big[:, :, :16]
    whole = part.contiguous()
    with pytest.raises(ValueError):
        cache(k_tail=part)
    with pytest.raises(ValueError):
        B.hga_quant_append(layer, cache(), part, whole, 16, 16, stream=0)
    with pytest.raises(ValueError):
        B.hga_quant_append(layer, cache(), whole, part, 16, 16, stream=0)
    for q, out in ((part, whole), (whole, part)):
        with pytest.raises(ValueError):
            B.hga_quant_attend(layer, cache(), q, 16, out, stream=0)


def strided(*shape, dtype=torch.float32):
    """Tensors of this shape that are not contiguous: every other element, and one row for all."""
    yield torch.zeros(*shape, 2, dtype=dtype)[..., 0]
    if shape[0] > 1:
        yield torch.zeros(1, *shape[1:], dtype=dtype).expand(*shape)


@pytest.mark.parametrize("name", ["pos", "counts", "chunk_sum", "group_sum"])
def test_append_refuses_strided(name):
    shape = {"pos": (2,), "counts": (2,)}.get(name, (2, 2, 4, 128))
    for bad in strided(*shape, dtype={"pos": torch.int64, "counts": torch.int32}.get(name, torch.float32)):
        args = {"pos": 16, "counts": 16, "chunk_sum": 16, "group_sum": 16, name: bad}
        with pytest.raises(ValueError):
            B.hga_quant_append(B.Layer(**LAYER), cache(), 16, 16, 1, stream=0, **args)


@pytest.mark.parametrize("name", ["pos", "lse", "group_idx", "weight_in", "weight_out", "workspace"])
def test_attend_refuses_strided(name):
    shape = {"pos": (2,), "lse": (2, 8, 1), "group_idx": (2, 2, 32), "workspace": (4096,)}.get(name, (2, 2, 4))
    kind = {"pos": torch.int64, "group_idx": torch.int32, "workspace": torch.uint8}.get(name, torch.float32)
    for bad in strided(*shape, dtype=kind):
        args = {"pos": 16, "lse": 16, "group_idx": 16, "weight_in": 16, "weight_out": 16, "workspace": 16, name: bad}
        with pytest.raises(ValueError):
            B.hga_quant_attend(B.Layer(**LAYER), cache(), 16, args.pop("pos"), 16, workspace_bytes=1 << 40,
                               stream=0, **args)


@pytest.mark.parametrize("name", ["pos", "weight_in", "weight_out", "table_out", "evicted_out"])
def test_evict_refuses_strided(name):
    shape = {"pos": (2,), "evicted_out": (2, 2)}.get(name, (2, 2, 4))
    kind = {"pos": torch.int64, "evicted_out": torch.int32, "table_out": torch.int32}.get(name, torch.float32)
    for bad in strided(*shape, dtype=kind):
        args = {"pos": 16, "weight_in": 16, "weight_out": 16, "table_out": 16, "evicted_out": 16, name: bad}
        with pytest.raises(ValueError):
            B.hga_quant_evict(B.Layer(**LAYER), cache(), args.pop("pos"), 4, 1, 1, stream=0, **args)
