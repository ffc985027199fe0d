"""What the chunk calls refuse, on the host and before any launch, through the C ABI and the
binding; and the rotation tables."""

import ctypes
import math

import pytest
import torch

import mla_decode_attention_gqa_gb300 as skv
from mla_decode_attention_gqa_gb300 import paged

FAKE = ctypes.c_void_p(0x10000)  # never dereferenced: validation fails first


def _paged(**kw):
    pg = skv.SkvPaged()
    pg.block_len, pg.max_blocks, pg.num_blocks, pg.block_table = 64, 16, 100, 0x10000
    for k, v in kw.items():
        setattr(pg, k, v)
    return pg


def _set(d, kw):
    for k, v in kw.items():
        if isinstance(v, tuple):
            for i, x in enumerate(v):
                getattr(d, k)[i] = x
        else:
            setattr(d, k, v)
    return d


def _chunk(**kw):
    d = skv.SkvChunkDesc()
    base = dict(B=3, T=10, Hq=16, Hkv=4, d=128, softmax_scale=0.088, scale_block=64, q_strides=(16 * 128, 128),
                k_strides=(4 * 64 * 128, 64 * 128, 128), v_strides=(4 * 64 * 128, 64 * 128, 128))
    return _set(_set(d, base), kw)


def _append(**kw):
    d = skv.SkvAppendDesc()
    base = dict(B=3, T=10, Hq=16, Hkv=4, d=128, rot=128, max_pos=1024, scale_block=64, eps=1e-6, q_strides=(24 * 128, 128),
                k_strides=(24 * 128, 128), v_strides=(24 * 128, 128), q_out_strides=(16 * 128, 128),
                k_page_strides=(4 * 64 * 128, 64 * 128, 128), v_page_strides=(4 * 64 * 128, 64 * 128, 128))
    return _set(_set(d, base), kw)


def _call_chunk(d, pg=None, ws_bytes=0, **ptr):
    lib = skv.load_library()
    p = dict(q=FAKE, k=FAKE, v=FAKE, ks=None, vs=None, cu=FAKE, seq=FAKE, out=FAKE, lse=FAKE, ws=None)
    p.update(ptr)
    return lib.attn_chunk_paged(ctypes.byref(d), ctypes.byref(pg or _paged()), p["q"], p["k"], p["v"], p["ks"], p["vs"],
                                p["cu"], p["seq"], p["out"], p["lse"], p["ws"], ws_bytes, None)


def _call_append(d, pg=None, **ptr):
    lib = skv.load_library()
    p = dict(q=FAKE, k=FAKE, v=FAKE, qw=FAKE, kw=FAKE, cos=FAKE, sin=FAKE, pos=None, cu=FAKE, seq=FAKE, ks=None, vs=None,
             out=FAKE, kp=FAKE, vp=FAKE)
    p.update(ptr)
    return lib.qk_norm_rope_append(ctypes.byref(d), ctypes.byref(pg or _paged()), p["q"], p["k"], p["v"], p["qw"], p["kw"],
                                   p["cos"], p["sin"], p["pos"], p["cu"], p["seq"], p["ks"], p["vs"], p["out"], p["kp"],
                                   p["vp"], None)


SHARED = [
    (dict(B=0), skv.SKV_EINVAL),
    (dict(T=-1), skv.SKV_EINVAL),
    (dict(Hq=15), skv.SKV_EINVAL),
    (dict(kv_dtype=5), skv.SKV_EINVAL),
    (dict(kv_dtype=1, scale_block=32), skv.SKV_EINVAL),
    (dict(kv_dtype=1, scale_block=128), skv.SKV_EINVAL),  # block_len 64
    (dict(d=96), skv.SKV_EUNSUPPORTED),
    (dict(kv_dtype=1, d=64), skv.SKV_EUNSUPPORTED),
    (dict(q_strides=(16 * 128, 100)), skv.SKV_EINVAL),
    (dict(q_strides=(0, 128)), skv.SKV_EINVAL),
    (dict(q_strides=(16 * 128, 0)), skv.SKV_EINVAL),
]


@pytest.mark.parametrize("kw,status", SHARED + [
    (dict(softmax_scale=math.inf), skv.SKV_EINVAL),
    (dict(d=576, Hkv=1, k_strides=(64 * 576, 0, 576), v_strides=(64 * 576, 0, 576)), skv.SKV_EUNSUPPORTED),
    (dict(softmax_scale=-0.1), skv.SKV_EINVAL),
    (dict(softmax_scale=0.0), skv.SKV_EINVAL),
    (dict(window=-1), skv.SKV_EINVAL),
    (dict(window=5, n_sink=-1), skv.SKV_EINVAL),
    (dict(n_sink=4), skv.SKV_EINVAL),
    (dict(k_strides=(4 * 64 * 128, 64 * 128, 64)), skv.SKV_EINVAL),
    (dict(v_strides=(4 * 64 * 128, 64 * 128, 132)), skv.SKV_EINVAL),
    (dict(v_strides=(0, 64 * 128, 128)), skv.SKV_EINVAL),
    (dict(k_strides=(4 * 64 * 128, 0, 128)), skv.SKV_EINVAL),
    (dict(T=2 ** 31 - 1), skv.SKV_EINVAL),  # more rows than 32 bits count
    (dict(T=2 ** 30, Hq=512, Hkv=512), skv.SKV_EINVAL),  # more blocks than a grid has
])
def test_bad_chunk_descriptions(kw, status):
    assert _call_chunk(_chunk(**kw)) == status
    assert skv.last_error()


@pytest.mark.parametrize("kw,status", SHARED + [
    (dict(rot=130), skv.SKV_EINVAL),
    (dict(rot=8), skv.SKV_EINVAL),
    (dict(rot=-16), skv.SKV_EINVAL),
    (dict(max_pos=0), skv.SKV_EINVAL),
    (dict(eps=-1.0), skv.SKV_EINVAL),
    (dict(eps=math.nan), skv.SKV_EINVAL),
    (dict(weight_dtype=2), skv.SKV_EINVAL),
    (dict(q_weight_stride=4), skv.SKV_EINVAL),
    (dict(k_strides=(24 * 128, 130)), skv.SKV_EINVAL),
    (dict(v_strides=(-8, 128)), skv.SKV_EINVAL),
    (dict(q_out_strides=(16 * 128, 64)), skv.SKV_EINVAL),
    (dict(k_page_strides=(4 * 64 * 128, 64 * 128, 120)), skv.SKV_EINVAL),
])
def test_bad_append_descriptions(kw, status):
    assert _call_append(_append(**kw)) == status
    assert skv.last_error()


@pytest.mark.parametrize("kw", [dict(block_len=0), dict(block_len=96), dict(max_blocks=0), dict(num_blocks=0),
                                dict(block_table=None), dict(block_table=0x10002), dict(max_blocks=2 ** 26),
                                dict(max_blocks=2 ** 25 - 1)])  # a tile past the last token leaves 32 bits
def test_bad_pages(kw):
    assert _call_chunk(_chunk(), _paged(**kw)) == skv.SKV_EINVAL
    assert _call_append(_append(), _paged(**kw)) == skv.SKV_EINVAL


@pytest.mark.parametrize("kind,fields", [(skv.SkvChunkDesc, skv._CHUNK_FIELDS), (skv.SkvAppendDesc, skv._APPEND_FIELDS)])
def test_descriptions_from_their_fields(kind, fields):
    flat = [x for _, t in kind._fields_ for x in [t._type_ if issubclass(t, ctypes.Array) else t] * getattr(t, "_length_", 1)]
    values = [0.5 if t is ctypes.c_float else i + 1 for i, t in enumerate(flat)]
    d = skv._described(kind, fields, *values)
    got = [x for n, t in kind._fields_ for x in (list(getattr(d, n)) if issubclass(t, ctypes.Array) else [getattr(d, n)])]
    assert got == values
    for bad in (1 << 40, 1.5, None):
        with pytest.raises(ValueError):
            skv._described(kind, fields, bad, *values[1:])


def test_bad_pointers():
    odd = ctypes.c_void_p(0x10008)
    for name in ("q", "k", "v", "cu", "seq", "out", "lse"):
        assert _call_chunk(_chunk(), **{name: None}) == skv.SKV_EINVAL
    for name in ("q", "k", "v", "out"):
        assert _call_chunk(_chunk(), **{name: odd}) == skv.SKV_EINVAL
    for name in ("q", "k", "v", "cos", "sin", "cu", "seq", "out", "kp", "vp"):
        assert _call_append(_append(), **{name: None}) == skv.SKV_EINVAL
    for name in ("q", "k", "v", "qw", "kw", "cos", "sin", "out", "kp", "vp"):
        assert _call_append(_append(), **{name: odd}) == skv.SKV_EINVAL
    assert _call_append(_append(), pos=ctypes.c_void_p(0x10002)) == skv.SKV_EINVAL
    assert _call_chunk(_chunk(kv_dtype=1)) == skv.SKV_EINVAL and "scale" in skv.last_error()
    assert _call_append(_append(kv_dtype=1)) == skv.SKV_EINVAL and "scale" in skv.last_error()
    assert _call_chunk(_chunk()) == skv.SKV_EWORKSPACE
    assert _call_chunk(_chunk(), ws=ctypes.c_void_p(0x10010), ws_bytes=1 << 30) == skv.SKV_EWORKSPACE


def test_no_rows_need_nothing():
    n = ctypes.c_size_t(1)
    lib = skv.load_library()
    assert lib.attn_chunk_paged_workspace_size(ctypes.byref(_chunk(T=0)), ctypes.byref(_paged()), ctypes.byref(n)) == 0
    assert n.value == 0
    assert _call_chunk(_chunk(T=0), q=None, out=None) == skv.SKV_OK
    assert _call_append(_append(T=0), q=None, out=None) == skv.SKV_OK
    assert lib.attn_chunk_paged_workspace_size(ctypes.byref(_chunk()), ctypes.byref(_paged()), None) == skv.SKV_EINVAL
    assert lib.attn_chunk_paged_workspace_size(None, ctypes.byref(_paged()), ctypes.byref(n)) == skv.SKV_EINVAL
    assert lib.attn_chunk_paged_workspace_size(ctypes.byref(_chunk()), None, ctypes.byref(n)) == skv.SKV_EINVAL


def test_the_workspace_does_not_grow_with_the_history():
    """Partials are bounded by what fills the GPU, whatever the capacity of the tables."""
    lib = skv.load_library()
    sizes = []
    for max_blocks in (1, 64, 1 << 20):
        n = ctypes.c_size_t(0)
        assert lib.attn_chunk_paged_workspace_size(ctypes.byref(_chunk(T=4096)), ctypes.byref(_paged(max_blocks=max_blocks)),
                                                   ctypes.byref(n)) == 0
        sizes.append(n.value)
    assert len(set(sizes)) == 1 and 0 < sizes[0] < 1 << 28


def test_cpu_tensors_are_refused():
    z = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    pages = torch.zeros(1, 2, 64, 64, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        skv.attn_chunk_paged(z, pages, pages, i[:1], i, i.view(1, 2))
    with pytest.raises(ValueError, match="CUDA"):
        skv.qk_norm_rope_append(z, z[:, :2], z[:, :2], pages, pages, i[:1], i, i.view(1, 2))


def test_split_qkv_and_tables():
    x = torch.arange(2 * 8 * 4).view(2, 32)
    q, k, v = paged.split_qkv(x, 4, 2)
    assert q.shape == (2, 4, 4) and k.shape == v.shape == (2, 2, 4)
    assert torch.equal(torch.cat((q, k, v), 1).reshape(2, 32), x)
    with pytest.raises(ValueError):
        paged.split_qkv(x, 5, 1)
    cos, sin = paged.rotation_tables(1000, 32)
    assert cos.shape == sin.shape == (1000, 16) and cos.dtype == torch.float32
    angle = 777 * 10000.0 ** (-2 * 5 / 32)
    assert abs(cos[777, 5] - math.cos(angle)) <= 2 ** -24 and abs(sin[777, 5] - math.sin(angle)) <= 2 ** -24


def _rows_meet(a, n, b, m, d):
    seen = set()
    for t in range(n):
        for h in range(m):
            row = set(range(t * a + h * b, t * a + h * b + d))
            if row & seen:
                return True
            seen |= row
    return False


def test_queries_out_need_a_place_for_each_row():
    """Token and head strides that put the rows of several tokens in one place; layouts that only
    look like it, and a single token, are taken (and refused for the missing q behind that)."""
    T, H, d = 4, 3, 64
    for a in [0, 8, 32] + list(range(64, 420, 32)):
        for b in range(64, 420, 32):
            args = dict(T=T, Hq=H, Hkv=H, d=d, rot=64, q_strides=(9 * d, d), q_out_strides=(a, b),
                        k_page_strides=(H * 64 * d, 64 * d, d), v_page_strides=(H * 64 * d, 64 * d, d))
            assert _call_append(_append(**args), q=None) == skv.SKV_EINVAL
            assert ("q_out strides" in skv.last_error()) == _rows_meet(a, T, b, H, d), (a, b, skv.last_error())
            args["T"] = 1
            assert _call_append(_append(**args), q=None) == skv.SKV_EINVAL
            assert "strides" not in skv.last_error()


@pytest.mark.parametrize("record,detail,words", [
    ((0,) * 8, None, ""),
    ((8,) + (0,) * 7, {"code": 8}, "a position outside the rotation tables"),
    ((9, 1, 3, 64, 1024, 1 | 1 << 8, 0, 0),
     {"code": 9, "block": 3, "thread": 64, "barrier_smem_addr": 1024, "parity": 1, "first_code": 1},
     "a wait for a tile gave up, a position outside the rotation tables"),
])
def test_the_device_error_says_what_it_is(record, detail, words, monkeypatch, capsys):
    """A position outside the tables is not a wait that gave up, and has no barrier to show."""
    def fake(rec):
        for i, x in enumerate(record):
            rec[i] = x
        return 0

    class Lib:
        splitkv_device_error_detail = staticmethod(fake)

    monkeypatch.setattr(skv, "_lib", Lib())
    monkeypatch.setattr(skv, "last_device_error_detail", None)
    assert skv.device_error() == record[0]
    assert skv.last_device_error_detail == detail
    err = capsys.readouterr().err
    assert words in err and (err == "") == (record[0] == 0)


@pytest.mark.parametrize("G", [1, 3, 4, 8, 16, 33, 128, 129, 200])
def test_rows_of_a_kv_head_choose_the_kernel(G):
    """Up to 32 rows of a KV head (chunk bound times group), or a group above 128 heads: the kernels
    whose partials are two a CTA and row; more: the tensor cores, whose workspace counts 4 items of
    up to 256 rows a CTA.  (Tests that name a kernel rely on it.)"""
    lib = skv.load_library()

    def size(T, longest):
        n = ctypes.c_size_t(0)
        d = _chunk(T=T, Hq=4 * G, max_q_len=longest, q_strides=(4 * G * 128, 128))
        assert lib.attn_chunk_paged_workspace_size(ctypes.byref(d), ctypes.byref(_paged()), ctypes.byref(n)) == 0
        return n.value

    few = size(4096, 1) if G <= 32 or G > 128 else None
    for longest in range(1, 60):
        on_tc = longest * G > 32 and G <= 128
        if on_tc:  # 608 items of 256 rows, heads of 128, in fp32
            assert size(4096, longest) > 608 * 256 * 128 * 4
        else:
            assert size(4096, longest) == few and few < 608 * 256 * 128
        assert size(4096, 0) == size(4096, 4096) == size(4096, 10 ** 6)  # no bound: T
        assert size(longest, 0) == size(longest, longest)
