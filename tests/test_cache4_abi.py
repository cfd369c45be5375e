"""Refusals and sizes of the 4-bit cache's calls and of rotary positions, through the C ABI and the binding, without a GPU:
every argument error returns before any CUDA call. The host tables of the frequencies, and the plain restatements that the GPU
tests use, pinned against hand-derived values."""
import ctypes
import math

import numpy as np
import pytest
import torch

import gated_deltanet_linear_gdn_gb300 as gdn
from gated_deltanet_linear_gdn_gb300 import build

import _cache4_oracle as co

P = ctypes.c_void_p
FAKE = P(0x10000)  # never dereferenced: every call below fails its checks first
BAD = P(0x10008)   # (8 is enough of an alignment for no array but the turns)
INV, UNS, OK = gdn.GDN_ERR_INVALID_ARG, gdn.GDN_ERR_UNSUPPORTED, gdn.GDN_OK


@pytest.fixture(scope="module")
def L():
    build.build_library()
    return gdn.lib()


def dims(q=8, kv=2, d=128, bs=16):
    return gdn.gdn_cache_dims(q, kv, d, bs)


def append(L, d=None, **kw):
    a = dict(k=FAKE, ks=256, v=FAKE, vs=256, slots=FAKE, T=4, kc=FAKE, vc=FAKE, sk=FAKE, sv=FAKE, N=10)
    a.update(kw)
    return L.gdn_cache4_append(*a.values(), d or dims(), None, None)


def read(L, d=None, **kw):
    a = dict(kc=FAKE, vc=FAKE, sk=FAKE, sv=FAKE, N=10, slots=FAKE, T=4, dims=d or dims(), k=FAKE, ks=256, v=FAKE, vs=256)
    a.update(kw)
    return L.gdn_cache4_read(*a.values(), None, None)


@pytest.mark.parametrize("call", [append, read])
def test_writer_and_reader_refusals(L, call):
    assert call(L, T=0) == OK
    for name in ("k", "v", "slots", "kc", "vc", "sk", "sv"):
        assert call(L, **{name: None}) == INV, name
        assert call(L, **{name: P(0x10002)}) == INV, name
        assert name == "slots" or call(L, **{name: BAD}) == INV, name
    assert call(L, T=-1) == call(L, N=0) == call(L, ks=255) == call(L, ks=260) == call(L, vs=8) == INV
    assert call(L, dims(d=96)) == call(L, dims(bs=8)) == call(L, N=1 << 27) == call(L, T=0x7fffffff) == UNS
    assert call(L, dims(kv=0)) == INV


def attn(L, which, d=None, **kw):
    a = dict(q=FAKE, qs=1024)
    if which == "prefill":
        a["cu"] = FAKE
    a.update(kc=FAKE, vc=FAKE, sk=FAKE, sv=FAKE, N=10, table=P(0x10000), W=4, lens=FAKE, B=2)
    if which == "prefill":
        a.update(T=6, held=8)
    a.update(dims=d or dims(), scale=0.1, out=FAKE, ws=FAKE, size=1 << 40)
    a.update(kw)
    return getattr(L, "gdn_attn4_" + which)(*a.values(), None, None)


@pytest.mark.parametrize("which", ["decode", "prefill"])
def test_attention_refusals(L, which):
    assert attn(L, which, B=0) == OK
    for name in ("q", "kc", "vc", "sk", "sv", "table", "lens", "out", "ws") + (("cu",) if which == "prefill" else ()):
        assert attn(L, which, **{name: None}) == INV, name
        assert attn(L, which, **{name: P(0x10002)}) == INV, name
    for name in ("q", "kc", "vc", "sk", "sv", "out", "ws"):
        assert attn(L, which, **{name: BAD}) == INV, name
    assert attn(L, which, B=-1) == attn(L, which, W=0) == attn(L, which, N=0) == INV
    assert attn(L, which, qs=1023) == attn(L, which, qs=1020) == attn(L, which, size=100) == INV
    assert attn(L, which, scale=float("nan")) == attn(L, which, scale=float("inf")) == INV
    assert attn(L, which, dims(q=7)) == attn(L, which, dims(q=0)) == INV
    assert attn(L, which, dims(d=192)) == attn(L, which, dims(bs=256)) == attn(L, which, B=65536) == UNS
    assert attn(L, which, W=1 << 27) == UNS
    if which == "prefill":
        assert attn(L, which, T=0) == OK and attn(L, which, T=-1) == INV
        assert attn(L, which, T=1 << 29) == attn(L, which, B=4097) == UNS
        assert attn(L, which, held=0) == attn(L, which, held=-1) == INV
        assert attn(L, which, B=4096, W=1 << 20, held=0x7fffffff) == UNS          # rows of its 8-bit pages past 32 bits


def test_workspace_sizes():
    f, g = gdn.gdn_attn4_decode_workspace_size, gdn.gdn_attn4_prefill_workspace_size
    assert 0 < f(1, 10, 8, 2, 128, 16) < f(2, 10, 8, 2, 128, 16) <= f(2, 1000, 8, 2, 128, 16)
    assert f(0, 10, 8, 2, 128, 16) == f(1, 10, 7, 2, 128, 16) == f(1, 10, 8, 2, 100, 16) == 0
    assert 0 < g(100, 2, 10, 8, 2, 128, 16, held_blocks=5) < g(100, 2, 10, 8, 2, 128, 16)
    assert g(100, 2, 10, 8, 2, 128, 16, held_blocks=20) == g(100, 2, 10, 8, 2, 128, 16) == g(100, 2, 10, 8, 2, 128, 16, held_blocks=999)
    # a page more: its keys and values in 8 bits, and two scales a head (8 bytes more in arrays rounded up to 256)
    assert 0 <= g(100, 2, 10, 8, 2, 128, 16, held_blocks=6) - g(100, 2, 10, 8, 2, 128, 16, held_blocks=5) - 2 * 2 * 16 * 128 <= 4 * 256
    assert g(100, 0, 10, 8, 2, 128, 16) == g(100, 1, 0, 8, 2, 128, 16) == g(100, 1, 10, 8, 2, 128, 16, held_blocks=0) == 0
    assert g(100, 1 << 12, 1 << 20, 8, 2, 128, 16) == 0


def rope(L, **kw):
    a = dict(q=FAKE, qs=1024, k=FAKE, ks=256, pos=FAKE, T=5, Hq=8, H=2, d=128, rot=64, layout=0, turns=FAKE, f=1.0, qo=FAKE, qos=1024,
             ko=FAKE, kos=256)
    a.update(kw)
    return L.gdn_rope(*a.values(), None)


def test_rope_refusals(L):
    assert rope(L, T=0) == OK
    for name in ("q", "k", "qo", "ko", "pos", "turns"):
        assert rope(L, **{name: None}) == INV, name
        assert rope(L, **{name: P(0x10001)}) == INV, name
    assert rope(L, turns=P(0x10004)) == rope(L, pos=P(0x10002)) == INV
    assert rope(L, T=-1) == rope(L, Hq=-1) == rope(L, Hq=0, H=0) == rope(L, rot=0) == rope(L, rot=63) == rope(L, rot=130) == INV
    assert rope(L, qs=1023) == rope(L, qos=1023) == rope(L, ks=255) == rope(L, kos=255) == rope(L, layout=2) == rope(L, d=0) == INV
    assert rope(L, f=float("nan")) == rope(L, f=float("inf")) == INV
    assert rope(L, d=1026, qs=1 << 20, qos=1 << 20, ks=1 << 20, kos=1 << 20) == rope(L, Hq=1025) == rope(L, T=0x7fffffff) == UNS


def freqs(L, rot=8, base=100.0, kind=0, factor=2.0, trained=64):
    w, f = (ctypes.c_double * max(rot // 2, 1))(), ctypes.c_float()
    status = L.gdn_rope_frequencies(rot, base, kind, factor, trained, w, ctypes.byref(f))
    return status, list(w), f.value


def test_rope_frequencies(L):
    st, w, f = freqs(L)
    assert st == OK and f == 1.0 and w == pytest.approx([1.0, 100 ** -0.25, 0.1, 100 ** -0.75], rel=1e-14)
    assert freqs(L, kind=1)[1] == pytest.approx([x / 2 for x in w], rel=1e-14)
    n = freqs(L, kind=2)[1]      # the first stays, the last slows down by the factor
    assert n[0] == 1.0 and n[3] == pytest.approx(w[3] / 2, rel=1e-12) and w[1] / 2 < n[1] < w[1]
    assert freqs(L, rot=2, kind=2)[1] == [1.0]
    # YaRN: over 4,096 positions pair i turns 4096 w_i / (2 pi) times: 32 at index 3.02, 1 at 6.03 (base 10,000, 16 elements)
    st, y, f = freqs(L, rot=16, base=10000.0, kind=3, factor=4.0, trained=4096)
    p = [10000 ** (-i / 8) for i in range(8)]
    assert f == pytest.approx(0.1 * math.log(4) + 1, rel=1e-6)
    lo, hi = math.floor(16 * math.log(4096 / (64 * math.pi)) / (2 * math.log(1e4))), math.ceil(16 * math.log(4096 / (2 * math.pi)) / (2 * math.log(1e4)))
    assert (lo, hi) == (2, 6)
    assert y[:3] == pytest.approx(p[:3], rel=1e-14) and y[6:] == pytest.approx([x / 4 for x in p[6:]], rel=1e-14)
    assert y[4] == pytest.approx(p[4] * 0.5 + p[4] / 4 * 0.5, rel=1e-14)
    for kw in (dict(rot=0), dict(rot=7), dict(base=1.0), dict(base=float("inf")), dict(kind=4), dict(kind=-1), dict(kind=1, factor=0.5),
               dict(kind=3, trained=0), dict(kind=1, factor=float("nan"))):
        assert freqs(L, **kw)[0] == INV, kw
    assert freqs(L, rot=1026)[0] == UNS


def test_rope_turns(L):
    def turns(*w):
        t = (ctypes.c_uint64 * len(w))()
        assert L.gdn_rope_turns((ctypes.c_double * len(w))(*w), len(w), t) == OK
        return list(t)

    assert turns(0.0, math.pi, 2 * math.pi, 3 * math.pi) == [0, 1 << 63, 0, 1 << 63]
    assert turns(-math.pi / 2) == [3 << 62]
    (t,) = turns(1.0)
    assert abs(t / 2.0 ** 64 - 1 / (2 * math.pi)) < 2.0 ** -53
    assert L.gdn_rope_turns((ctypes.c_double * 1)(float("nan")), 1, (ctypes.c_uint64 * 1)()) == INV
    assert L.gdn_rope_turns((ctypes.c_double * 1)(1.0), 0, (ctypes.c_uint64 * 1)()) == INV
    r = gdn.RopeTable(4, freqs=[1.0, 0.25], factor=2.0, device="cpu")
    assert r.factor == 2.0 and [x % (1 << 64) for x in r.turns.tolist()] == turns(1.0, 0.25)
    with pytest.raises(ValueError):
        gdn.RopeTable(4, freqs=[1.0])
    with pytest.raises(ValueError):
        gdn.RopeTable(5)


def test_binding_refuses_wrong_tensors():
    kc, vc = torch.zeros(4, 2, 16, 32, dtype=torch.uint8), torch.zeros(4, 2, 8, 64, dtype=torch.uint8)
    s = torch.zeros(4, 2, 16, 2, dtype=torch.uint8)
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    i = torch.zeros(3, dtype=torch.int32)
    for bad in ((kc, vc, s, s), (kc.to(torch.int8), vc, s, s), (kc, kc, s, s), (kc, vc, s.float(), s.float()), (kc, vc, s, s[:2])):
        with pytest.raises(ValueError):       # not on the device, or of another type or shape
            gdn.gdn_attn4_decode(q, *bad, i.reshape(3, 1), i, q, s)
        with pytest.raises(ValueError):
            gdn.gdn_cache4_append(q[:, :2], q[:, :2], i, *bad)
        with pytest.raises(ValueError):
            gdn.gdn_cache4_read(*bad, i, q[:, :2], q[:, :2])
    with pytest.raises(ValueError):
        gdn.gdn_rope(q, q[:, :2], i, q, q[:, :2], gdn.RopeTable(64, device="cpu"))
    with pytest.raises(ValueError):
        gdn.gdn_rope(q.float(), None, i, q, None, gdn.RopeTable(64, device="cpu"))


# ------------------------------------------------------------------------ the restatements

def test_codes_by_hand():
    assert co.VALUES.tolist()[:8] == [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    y = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 0.2501, 100.0, -0.0, -5.01])   # ties go to the even code
    assert co.nearest_code(y).tolist() == [0, 2, 2, 4, 4, 6, 6, 1, 7, 8, 15]


def test_quantise_by_hand():
    x = np.zeros(96, np.float32)
    x[0], x[1], x[33], x[64] = 7.0, -0.5, 7.03125, np.nan      # the next bf16 value after 7
    codes, scales = co.quantise(x)
    assert scales == [127, 128, 255] and codes[2] is None
    assert codes[0][:3].tolist() == [7, 9, 0] and codes[1][1] == 6       # 7 -> 6; 3.515625 -> 4
    assert co.quantise(np.zeros(32, np.float32))[1] == [63] and co.quantise(np.full(32, 2.0 ** -80, np.float32))[1] == [63]
    big = np.zeros(32, np.float32)
    big[0], big[1] = np.inf, 1.5
    assert co.quantise(big)[1] == [125] and co.quantise(big)[0][0][:2].tolist() == [7, 7]      # 1.5 = 6 / 4


def test_layout_by_hand():
    kc, vc = np.zeros((1, 1, 16, 32), np.uint8), np.full((1, 1, 8, 64), 0xAA, np.uint8)
    ks, vs = np.zeros((1, 1, 16, 2), np.uint8), np.zeros((1, 1, 16, 2), np.uint8)
    x = np.zeros((1, 1, 64), np.float32)
    x[0, 0, :3], x[0, 0, 32] = [4, -6, 2], 12
    kc, vc, ks, vs = co.append(x, x, [5], kc, vc, ks, vs)
    assert kc[0, 0, 5, :2].tolist() == [0x6 | 0xF << 4, 0x4] and kc[0, 0, 5, 16] == 7 and ks[0, 0, 5].tolist() == [127, 128]
    assert vc[0, 0, 2, :3].tolist() == [0x6A, 0xFA, 0x4A]      # token 5: the upper half of pair 2
    k, v = co.unpack(*(torch.from_numpy(z) for z in (kc, vc, ks, vs)))
    assert k[0, 0, 5, :3].tolist() == v[0, 0, 5, :3].tolist() == [4, -6, 2] and k[0, 0, 5, 32] == 12


def test_attention_against_torch_softmax():
    torch.manual_seed(0)
    k, v = torch.randn(2, 5, 1, 16, 64, dtype=torch.float64)
    table = torch.tensor([[3, 1, 4, -1]], dtype=torch.int32)
    q = torch.randn(4, 2, 64).bfloat16()
    out, tol = co.attention(q, [0, 4], k, v, table, [40], 0.125, 11, 2.0 ** -30)
    kk, vv = (x[[3, 1, 4], 0].reshape(48, 64)[:40] for x in (k, v))
    s = torch.einsum("thd,jd->htj", q.double(), kk) * 0.125
    s = s.masked_fill(torch.arange(40)[None, :] > 36 + torch.arange(4)[:, None], -torch.inf)
    ref = torch.einsum("htj,jd->thd", torch.softmax(s, -1), vv)
    assert float((out - ref).abs().max()) < 1e-12 * float(ref.abs().max())
    assert bool((tol > 0).all()) and float((tol / out.abs().mean()).max()) < 0.1


def test_rope_against_complex_numbers():
    torch.manual_seed(1)
    x = torch.randn(3, 2, 10).bfloat16()
    pos, w = torch.tensor([0, 7, 123456]), [1.0, 0.3, 0.01]
    turn = torch.polar(torch.full((3, 3), 1.5, dtype=torch.float64), pos.double()[:, None] * torch.tensor(w, dtype=torch.float64))[:, None, :]
    y, tol = co.rope(x, pos, w, 1.5, 6, True)
    z = torch.complex(x[..., 0:6:2].double(), x[..., 1:6:2].double()) * turn
    assert torch.allclose(torch.complex(y[..., 0:6:2], y[..., 1:6:2]), z, rtol=0, atol=1e-12) and torch.equal(y[..., 6:], x[..., 6:].double())
    y, _ = co.rope(x, pos, w, 1.5, 6, False)
    z = torch.complex(x[..., 0:3].double(), x[..., 3:6].double()) * turn
    assert torch.allclose(torch.complex(y[..., 0:3], y[..., 3:6]), z, rtol=0, atol=1e-12)
    assert float(tol[..., 6:].max()) < 1e-29
