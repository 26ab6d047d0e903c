"""Refusals of the paged-cache calls (checked on the host: no call here reaches
a launch) and the row formats of the plain implementation (CPU only)."""
import ctypes

import numpy as np
import pytest
import torch

from block_sparse_attention_online_gb300 import binding as bs
from block_sparse_attention_online_gb300 import build as B
from tests import paged_plain as plain

A = 0x10000  # aligned, never dereferenced: validation fails first


@pytest.fixture(scope="module")
def lib():
    B.build()
    return bs.load()


def pages(**kw):
    f = dict(format=1, n_pages=8, page_size=64, Hkv=2, d=128, page_stride=0, k=A, v=A, k_scale=A,
             v_scale=A, k_bs=A, v_bs=A)
    f.update(kw)
    return bs._KvPages(**f)


BAD_PAGES = [
    dict(format=3), dict(format=-1), dict(n_pages=0), dict(page_size=0), dict(Hkv=0), dict(d=0),
    dict(k=None), dict(v=None), dict(k=A + 8), dict(k_scale=None), dict(v_scale=A + 4),
    dict(page_stride=16), dict(page_stride=2 * 64 * 128 + 8), dict(page_stride=-16),
    dict(format=2, k_bs=None), dict(format=2, v_bs=A + 8),
]
UNSUPPORTED_PAGES = [dict(d=64), dict(page_size=8), dict(page_size=48), dict(page_size=192)]


def append(lib, kv=None, **kw):
    a = dict(kv=ctypes.byref(kv or pages()), k=A, v=A, dt=0, ks=256, vs=256, n_seq=2, total=5,
             cu=A, kv_len=A, table=A, max_pages=4, stream=None)
    a.update(kw)
    return lib.attn_skip_kv_append(*a.values())


def gather(lib, kv=None, **kw):
    a = dict(kv=ctypes.byref(kv or pages()), n_seq=2, total=5, cu=A, start=A, table=A,
             max_pages=4, dt=0, k=A, v=A, stream=None)
    a.update(kw)
    return lib.attn_skip_kv_gather(*a.values())


def chunk(lib, kv=None, **kw):
    a = dict(kv=ctypes.byref(kv or pages()), q=A, qs=8 * 128, Hq=8, n_seq=2, total=5, cu=A,
             max_chunk=3, kv_len=A, max_kv=256, table=A, max_pages=4, scale=0.0, lam=A, causal=1,
             n_splits=2, o=A, lse=A, bits=None, op=A, lp=A, work=None, stream=None)
    a.update(kw)
    return lib.attn_skip_chunk_paged(*a.values())


CALLS = {"append": append, "gather": gather, "chunk": chunk}


@pytest.mark.parametrize("call", CALLS)
def test_page_descriptions_are_checked(lib, call):
    for kw in BAD_PAGES:
        assert CALLS[call](lib, pages(**kw)) == bs.ATTN_EINVAL, kw
    for kw in UNSUPPORTED_PAGES:
        assert CALLS[call](lib, pages(**kw)) == bs.ATTN_EUNSUPPORTED, kw
    assert CALLS[call](lib, kv=None, **{"n_seq": 0}) == bs.ATTN_EINVAL
    assert CALLS[call](lib, **{"total": -1}) == bs.ATTN_EINVAL
    assert CALLS[call](lib, **{"max_pages": 0}) == bs.ATTN_EINVAL
    assert CALLS[call](lib, **{"max_pages": 1 << 28}) == bs.ATTN_EUNSUPPORTED
    for kw in (dict(cu=None), dict(cu=A + 2), dict(table=None), dict(table=A + 1)):
        assert CALLS[call](lib, **kw) == bs.ATTN_EINVAL, kw


@pytest.mark.parametrize("kw", [
    dict(k=None), dict(v=None), dict(k=A + 2), dict(dt=2), dict(ks=128), dict(vs=257),
    dict(kv_len=None), dict(kv_len=A + 2),
])
def test_append_rejects(lib, kw):
    assert append(lib, **kw) == bs.ATTN_EINVAL


@pytest.mark.parametrize("kw", [
    dict(k=None), dict(v=None), dict(v=A + 8), dict(dt=-1), dict(start=A + 2),
])
def test_gather_rejects(lib, kw):
    assert gather(lib, **kw) == bs.ATTN_EINVAL


@pytest.mark.parametrize("kw", [
    dict(q=None), dict(q=A + 8), dict(qs=7 * 128), dict(qs=8 * 128 + 4), dict(Hq=7), dict(Hq=0),
    dict(max_chunk=-1), dict(max_chunk=0), dict(max_kv=-1), dict(max_kv=257), dict(kv_len=None),
    dict(lam=None), dict(lam=A + 2), dict(scale=float("nan")), dict(n_splits=0),
    dict(n_splits=1025), dict(o=None), dict(o=A + 8), dict(lse=None), dict(bits=A + 2),
    dict(op=None), dict(lp=None), dict(op=A + 4), dict(work=A + 8),
])
def test_chunk_rejects(lib, kw):
    assert chunk(lib, **kw) == bs.ATTN_EINVAL


def test_chunk_too_many_heads_and_empty_calls(lib):
    assert chunk(lib, Hq=2 * 129, qs=2 * 129 * 128) == bs.ATTN_EUNSUPPORTED
    assert chunk(lib, max_chunk=0x7fffffff) == bs.ATTN_EUNSUPPORTED
    assert chunk(lib, total=0x7fffffff) == bs.ATTN_EUNSUPPORTED
    assert append(lib, total=0, k=None, v=None) == bs.ATTN_OK
    assert gather(lib, total=0, k=None, v=None) == bs.ATTN_OK
    assert chunk(lib, total=0, q=None, o=None, lse=None) == bs.ATTN_OK


def test_splits_proposal(lib):
    f = lib.attn_skip_chunk_paged_splits
    assert f(0, 0, 0, 8, 2, 1, 100) == 1 and f(0, 1, 1, 7, 2, 1, 100) == 1
    for n_seq, total, max_chunk, max_kv in ((1, 1, 1, 1), (1, 1, 1, 32768), (16, 16, 1, 32768),
                                            (1, 4096, 4096, 16384), (300, 300, 1, 64)):
        n = f(0, n_seq, total, 32, 8, max_chunk, max_kv)
        assert 1 <= n <= max(1, -(-max_kv // 128))
    assert f(0, 1, 1, 32, 8, 1, 32768) > 1  # few rows: the key axis is split
    assert f(0, 1, 16384, 32, 8, 16384, 16384) == 1  # many tiles: it is not


def test_widening_workspace(lib):
    f = lib.attn_skip_chunk_paged_kv_bytes
    assert f(0, 1, 32, 8, 4096, 16384) == 0   # a bf16 cache
    assert f(1, 1, 32, 8, 64, 16384) == 0     # two tiles
    assert f(1, 1, 32, 8, 4096, 16300) == 16384 * 8 * 512
    assert f(2, 3, 32, 8, 4096, 100) == 3 * 128 * 8 * 512
    assert f(1, 1000, 32, 8, 4096, 1 << 20) == 0  # more than 4 GiB
    assert f(1, 1, 33, 8, 4096, 16384) == 0 and f(1, 0, 32, 8, 4096, 16384) == 0


def test_binding_refuses_tensors_off_the_gpu():
    k = torch.zeros(2, 1, 16, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        bs.PagedKV("bf16", k, k.clone())
    with pytest.raises(ValueError, match="shape"):
        bs.PagedKV("e4m3", k, k.clone())
    with pytest.raises(ValueError, match="scale"):
        bs.PagedKV("e4m3", k.to(torch.uint8), k.to(torch.uint8))
    with pytest.raises(KeyError):
        bs.PagedKV("fp16", k, k)


def test_binding_refuses_pages_that_overlap():
    """A pool of one page expanded to four has page stride 0, which the C entry
    takes for a dense pool."""
    k = torch.zeros(1, 1, 16, 128, dtype=torch.bfloat16).expand(4, 1, 16, 128)
    with pytest.raises(ValueError, match="overlap"):
        bs.PagedKV("bf16", k, k)
    k = torch.zeros(4096, dtype=torch.bfloat16).as_strided((2, 1, 16, 128), (1024, 2048, 128, 1))
    with pytest.raises(ValueError, match="overlap"):
        bs.PagedKV("bf16", k, k)


@pytest.mark.parametrize("fmt,step", [("e4m3", 2.0 ** -4), ("nvfp4", 0.25)])
def test_plain_formats_round_to_nearest(fmt, step):
    """Reading back is off by at most half a step: 2^-4 of the value for E4M3
    (or half its subnormal step), half of E2M1's largest gap times the block
    scale for NVFP4; zeros, non-finite rows and the clamp of the scale."""
    g = np.random.default_rng(5)
    x = g.standard_normal((200, 128)) * np.exp2(g.integers(-30, 30, (200, 1)).astype(float))
    x[3] = 0.0
    x[4, 7], x[5, 9] = np.inf, np.nan
    x[6] *= 1e-60
    e = plain.encode(fmt, x)
    y = plain.decode(fmt, e["codes"], e["scale"], e.get("bs"))
    assert np.isnan(y[4:6]).all() and (e["scale"][4:6] == 255).all()
    assert (y[3] == 0).all() and e["scale"][3] == 127
    assert e["scale"][6] == 17  # 2^-110
    ok = np.ones(200, bool)
    ok[[4, 5]] = False
    s = np.exp2(e["scale"][ok].astype(float) - 127)[:, None]
    if fmt == "e4m3":
        tol = np.maximum(np.abs(x[ok]) * step, s * 2.0 ** -10)
    else:
        tol = np.repeat(plain.E4M3[e["bs"][ok]], 16, -1) * s  # half of the gap 4 .. 6
    assert (np.abs(y[ok] - x[ok]) <= tol * (1 + 1e-12)).all()
