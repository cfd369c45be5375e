"""Refusals and sizes of the paged-cache calls, through the C ABI and the binding, without a GPU:
every argument error returns before any CUDA call. The plain restatements that the GPU tests use
are pinned here against hand-derived values."""
import ctypes

import numpy as np
import pytest
import torch

import gated_deltanet_linear_gdn_gb300 as gdn
from gated_deltanet_linear_gdn_gb300 import build

import _cache_oracle as co

P = ctypes.c_void_p
FAKE = P(0x10000)  # never dereferenced: every call below fails its checks first
BAD = P(0x10002)
INV, UNS, OK = gdn.GDN_ERR_INVALID_ARG, gdn.GDN_ERR_UNSUPPORTED, gdn.GDN_OK


@pytest.fixture(scope="module")
def L():
    build.build_library()
    return gdn.lib()


def dims(q=8, kv=2, d=128, bs=16):
    return gdn.gdn_cache_dims(q, kv, d, bs)


def tables(L, **kw):
    a = dict(old=FAKE, new=FAKE, B=3, table=FAKE, W=4, ring=FAKE, N=20, pool=FAKE, pool2=FAKE, bs=16, T=5, cu=FAKE,
             slots=FAKE, pos=FAKE, lens=FAKE)
    a.update(kw)
    return L.gdn_cache_tables(*a.values(), None, None)


def test_tables_refusals(L):
    assert tables(L, B=0) == OK
    for name in ("old", "new", "table", "ring", "pool", "pool2", "cu", "slots", "pos", "lens"):
        assert tables(L, **{name: None}) == INV, name
        assert tables(L, **{name: P(0x10001)}) == INV, name
    assert tables(L, B=-1) == tables(L, W=0) == tables(L, N=0) == tables(L, T=-1) == INV
    assert tables(L, bs=24) == tables(L, bs=256) == tables(L, B=8193) == UNS
    assert tables(L, N=1 << 28, bs=16) == tables(L, W=1 << 28, bs=16) == UNS


def append(L, d=None, **kw):
    a = dict(k=FAKE, ks=256, v=FAKE, vs=256, slots=FAKE, T=4, kc=FAKE, vc=FAKE, sk=FAKE, sv=FAKE, N=10)
    a.update(kw)
    return L.gdn_cache_append(*a.values(), d or dims(), None, None)


def test_append_refusals(L):
    assert append(L, T=0) == OK
    for name in ("k", "v", "slots", "kc", "vc", "sk", "sv"):
        assert append(L, **{name: None}) == INV, name
        assert append(L, **{name: BAD}) == INV, name
    assert append(L, T=-1) == append(L, N=0) == append(L, ks=255) == append(L, ks=260) == append(L, vs=8) == INV
    assert append(L, dims(d=96)) == append(L, dims(bs=8)) == append(L, N=1 << 27) == UNS
    assert append(L, dims(kv=0)) == INV


def attn(L, which, d=None, **kw):
    a = dict(q=FAKE, qs=1024)
    if which == "prefill":
        a["cu"] = FAKE
    a.update(kc=FAKE, vc=FAKE, sk=FAKE, sv=FAKE, N=10, table=P(0x10000), W=4, lens=FAKE, B=2)
    if which == "prefill":
        a["T"] = 6
    a.update(dims=d or dims(), scale=0.1, out=FAKE, ws=FAKE, size=1 << 40)
    a.update(kw)
    return getattr(L, "gdn_attn_" + which)(*a.values(), None, None)


@pytest.mark.parametrize("which", ["decode", "prefill"])
def test_attention_refusals(L, which):
    assert attn(L, which, B=0) == OK
    for name in ("q", "kc", "vc", "sk", "sv", "table", "lens", "out", "ws") + (("cu",) if which == "prefill" else ()):
        assert attn(L, which, **{name: None}) == INV, name
        assert attn(L, which, **{name: BAD}) == INV, name
    assert attn(L, which, B=-1) == attn(L, which, W=0) == attn(L, which, N=0) == INV
    assert attn(L, which, qs=1023) == attn(L, which, qs=1020) == attn(L, which, size=100) == INV
    assert attn(L, which, scale=float("nan")) == attn(L, which, scale=float("inf")) == INV
    assert attn(L, which, dims(q=7)) == attn(L, which, dims(q=0)) == INV
    assert attn(L, which, dims(d=192)) == attn(L, which, dims(bs=256)) == attn(L, which, B=65536) == UNS
    assert attn(L, which, W=1 << 27) == UNS
    if which == "prefill":
        assert attn(L, which, T=0) == OK and attn(L, which, T=-1) == INV
        assert attn(L, which, T=1 << 29) == UNS


def test_workspace_sizes(L):
    f, g = gdn.gdn_attn_decode_workspace_size, gdn.gdn_attn_prefill_workspace_size
    assert 0 < f(1, 10, 8, 2, 128, 16) < f(2, 10, 8, 2, 128, 16) <= f(2, 1000, 8, 2, 128, 16)
    assert f(0, 10, 8, 2, 128, 16) == f(1, 10, 7, 2, 128, 16) == f(1, 10, 8, 2, 100, 16) == 0
    assert 0 < g(100, 1, 10, 8, 2, 128, 16) <= g(200, 1, 10, 8, 2, 128, 16) < g(200, 1, 1000, 8, 2, 128, 16)
    assert g(100, 0, 10, 8, 2, 128, 16) == g(100, 1, 0, 8, 2, 128, 16) == 0
    # what a batch needs does not grow past one launch's requests
    assert f(65535, 10, 8, 2, 128, 16) == f(2048, 10, 8, 2, 128, 16)


def test_binding_refuses_wrong_tensors():
    f8 = torch.zeros(4, 2, 16, 64, dtype=torch.uint8).view(torch.float8_e4m3fn)
    s = torch.zeros(4, 2)
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    i = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError):
        gdn.gdn_attn_decode(q, f8.float(), f8, s, s, i.reshape(3, 1), i, q, s)      # not 8-bit
    with pytest.raises(ValueError):
        gdn.gdn_attn_decode(q, f8, f8, s, s, i.reshape(3, 1), i, q, s)              # not on the device
    with pytest.raises(ValueError):
        gdn.gdn_cache_append(q, q, i.long(), f8, f8, s, s)
    with pytest.raises(ValueError):
        gdn.gdn_cache_tables(i, i, i, i, i, i, i, i, i, i, 16)


# ------------------------------------------------------------------------ the restatements

def test_e4m3_rounding():
    v = co.E4M3
    assert v[0x7E] == 448 and v[0x01] == 2.0 ** -9 and v[0x08] == 2.0 ** -6 and v[0x38] == 1.0 and np.isnan(v[0x7F])
    fin = [b for b in range(256) if not np.isnan(v[b])]
    assert [int(x) for x in co.to_e4m3(v[fin])] == fin                                # every value is itself
    # ties to even, saturation, signs
    assert [int(x) for x in co.to_e4m3([17, 18, 19, 1e9, -1e9, np.inf, 464, 2.0 ** -10, 3 * 2.0 ** -10, np.nan, -0.0])] == [
        0x58, 0x59, 0x5A, 0x7E, 0xFE, 0x7E, 0x7E, 0, 2, 0x7F, 0x80]
    x = torch.randn(4000) * 50                                                        # and as torch rounds
    x = x[x.abs() < 440].numpy()
    assert np.array_equal(co.to_e4m3(x), torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy())


def test_tables_by_hand():
    table = np.array([[7, -1, -1], [2, 5, -1], [9, -1, -1]])
    ring = np.array([4, 8, 1, 0, 3, 6, -1, -1, -1, -1])
    r = co.tables([3, 20, 16], [4, 0, 33], table, ring, [1, 4], 16, 20)
    assert r["table"].tolist() == [[7, -1, -1], [2, 5, -1], [9, 8, 1]]
    assert r["pool"].tolist() == [3, 4] and r["ring"].tolist() == [4, 8, 1, 0, 3, 2, 5, -1, -1, -1]
    assert r["cu"].tolist() == [0, 1, 1, 18] and r["lens"].tolist() == [4, 0, 33]
    assert r["slots"].tolist() == [7 * 16 + 3] + [8 * 16 + j for j in range(16)] + [16] + [-1, -1]
    assert r["positions"][:2].tolist() == [3, 16]
    r = co.tables([0, 0, 0], [16, 33, 16], np.full((3, 3), -1), ring, [0, 3], 16, 65)
    assert r["short"] and r["lens"].tolist() == [16, 0, 0] and r["pool"].tolist() == [1, 2]


def test_append_by_hand():
    x = np.zeros((2, 1, 64), np.float32)
    x[0, 0, :2], x[1, 0, :2] = [448, -224], [896, 1]
    c, s = np.zeros((1, 1, 16, 64), np.uint8), np.zeros((1, 1), np.float32)
    c, s = co.append(x[:1], [0], c, s)
    assert s[0, 0] == 1.0 and co.E4M3[c[0, 0, 0, :2]].tolist() == [448, -224]
    c, s = co.append(x[1:], [1], c, s)
    assert s[0, 0] == 2.0 and co.E4M3[c[0, 0, :2, :2]].tolist() == [[224, -112], [448, 0.5]]


def test_attention_against_torch_softmax():
    torch.manual_seed(0)
    kc = torch.randint(0, 120, (5, 1, 16, 64), dtype=torch.uint8)
    vc = torch.randint(128, 240, (5, 1, 16, 64), dtype=torch.uint8)
    ks, vs = torch.rand(5, 1) / 50, torch.rand(5, 1)
    table = torch.tensor([[3, 1, 4, -1]], dtype=torch.int32)
    q = torch.randn(4, 2, 64).bfloat16()
    out, tol = co.attention(q, [0, 4], kc, vc, ks, vs, table, [40], 0.125, 9, 2.0 ** -13)
    lut = torch.from_numpy(co.E4M3)
    k = (lut[kc.long()] * ks[:, :, None, None])[[3, 1, 4], 0].reshape(48, 64)[:40]
    v = (lut[vc.long()] * vs[:, :, None, None])[[3, 1, 4], 0].reshape(48, 64)[:40]
    s = torch.einsum("thd,jd->htj", q.double(), k) * 0.125
    s = s.masked_fill(torch.arange(40)[None, :] > 36 + torch.arange(4)[:, None], -torch.inf)
    ref = torch.einsum("htj,jd->thd", torch.softmax(s, -1), v)
    assert float((out - ref).abs().max()) < 1e-9 * float(ref.abs().max())
    assert bool((tol > 0).all()) and float((tol / out.abs().mean()).max()) < 0.1
