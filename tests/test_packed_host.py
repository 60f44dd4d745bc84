"""Host-side checks of the packed operators: what the C ABI and the binding refuse before any launch.  CPU only."""
import ctypes

import pytest
import torch

from scaled_dot_product_prefill_b200 import _lib, api

FAKE = ctypes.c_void_p(0x10000)          # aligned, never dereferenced: every case fails validation or is empty
OFF8 = ctypes.c_void_p(0x10008)
OFF2 = ctypes.c_void_p(0x10002)
bf = torch.bfloat16


def lib():
    return _lib.load()


def packed(q=FAKE, k=FAKE, v=FAKE, cu_q=FAKE, cu_k=FAKE, B=2, Tq=64, Tk=64, Hq=8, Hkv=2, D=64, qs=512, ks=128, vs=128,
           os=512, scale=0.125, causal=1, window=0, ws=None, ws_bytes=0, out=FAKE, lse=None):
    return lib().attn_prefill_packed(q, k, v, cu_q, cu_k, B, Tq, Tk, Hq, Hkv, D, qs, ks, vs, os, scale, causal, window,
                                     ws, ws_bytes, out, lse, None)


def paged(q=FAKE, kp=FAKE, vp=FAKE, cu_q=FAKE, pt=FAKE, sl=FAKE, page=16, B=2, Tq=64, Hq=8, Hkv=2, D=64, qs=512, os=512,
          num_pages=8, max_pages=4, max_seq_len=64, scale=0.125, causal=1, window=0, ws=None, ws_bytes=0, out=FAKE, lse=None):
    return lib().attn_prefill_packed_paged(q, kp, vp, cu_q, pt, sl, page, B, Tq, Hq, Hkv, D, qs, os, num_pages, max_pages,
                                           max_seq_len, scale, causal, window, ws, ws_bytes, out, lse, None)


BOTH = [
    (dict(q=None), 1), (dict(out=None), 1), (dict(cu_q=None), 1), (dict(q=OFF8), 1), (dict(out=OFF8), 1),
    (dict(cu_q=OFF2), 1), (dict(lse=OFF2), 1), (dict(Hq=6, Hkv=4, qs=384, os=384), 1), (dict(Hkv=0), 1),
    (dict(Tq=-1), 1), (dict(B=-1), 1), (dict(scale=0.0), 1), (dict(scale=float("nan")), 1),
    (dict(scale=float("inf")), 1), (dict(causal=2), 1), (dict(window=-1), 1), (dict(D=96, qs=768, os=768), 1),
    (dict(D=256, qs=2048, os=2048), 1),
    (dict(qs=504), 1), (dict(qs=516), 1), (dict(os=0), 1), (dict(qs=-512), 1), (dict(os=1 << 40), 1),
    (dict(ws=OFF8, ws_bytes=1 << 30), 6),
    (dict(causal=0, window=4), 2), (dict(B=70000), 2), (dict(Tq=(1 << 30) + 1), 2),
    (dict(B=0, q=None, out=None, cu_q=None), 0), (dict(Tq=0, q=None, out=None), 0), (dict(Hq=0, q=None, out=None), 0),
]


@pytest.mark.parametrize("change,status", BOTH, ids=[str(c) for c, _ in BOTH])
def test_both_packed_prefills_refuse(change, status):
    assert packed(**change) == status
    assert paged(**change) == status


@pytest.mark.parametrize("change,status", [
    (dict(k=None), 1), (dict(v=None), 1), (dict(cu_k=None), 1), (dict(k=OFF8), 1), (dict(cu_k=OFF2), 1),
    (dict(Tk=-1), 1), (dict(ks=120), 1), (dict(vs=132), 1), (dict(Tk=(1 << 30) + 1), 2), (dict(B=0, Tk=-1), 1)])
def test_packed_prefill_refuses(change, status):
    assert packed(**change) == status


@pytest.mark.parametrize("change,status", [
    (dict(kp=None), 1), (dict(vp=None), 1), (dict(pt=None), 1), (dict(sl=None), 1), (dict(kp=OFF8), 1),
    (dict(pt=OFF2), 1), (dict(sl=OFF2), 1), (dict(num_pages=0), 1), (dict(max_pages=0), 1), (dict(num_pages=-1), 1),
    (dict(max_seq_len=-1), 1), (dict(page=0), 1), (dict(page=8), 2), (dict(page=48), 2), (dict(page=512), 2),
    (dict(num_pages=0x7FFFFFFF), 2), (dict(max_seq_len=(1 << 30) + 1), 2)])
def test_packed_paged_prefill_refuses(change, status):
    assert paged(**change) == status


def test_the_workspace_of_sizes_that_no_call_takes_is_none():
    size = lib().attn_prefill_packed_workspace_size
    assert size(2, 10, 8, 2, 128, 1 << 30) > 0
    for max_seq_len in ((1 << 30) + 1, 0x7FFFFFFF, -1):
        assert size(2, 10, 8, 2, 128, max_seq_len) == 0


def test_the_workspace_of_a_split():
    size = lib().attn_prefill_packed_workspace_size
    # few items and long sequences: 2 sequences x 2 head blocks of one block each
    need = size(2, 10, 8, 2, 128, 8192)
    assert need == 16 * 10 * 8 * (128 + 1) * 4                       # 16 parts at most
    assert size(2, 10, 8, 2, 128, 600) == 5 * 10 * 8 * 129 * 4       # a part is one key tile at least
    assert size(2, 10, 8, 2, 128, 384) == 0                          # 3 key tiles are not split
    assert size(1, 1024, 8, 8, 64, 1024) == 2 * 1024 * 8 * 65 * 4    # full tiles: 4 key tiles a part
    assert size(1, 1024, 8, 8, 64, 7 * 128) == 0
    assert size(100, 100, 32, 8, 128, 8192) == 0                     # enough items without a split
    for bad in ((0, 10, 8, 2, 128, 8192), (2, 0, 8, 2, 128, 8192), (2, 10, 8, 3, 128, 8192), (2, 10, 8, 2, 0, 8192),
                (2, 10, 8, 2, 128, -1), (-1, 10, 8, 2, 128, 8192)):
        assert size(*bad) == 0
    kw = dict(Tq=10, D=128, qs=1024, os=1024)
    assert paged(ws=FAKE, ws_bytes=need - 1, max_seq_len=8192, max_pages=512, **kw) == 6
    assert packed(ws=FAKE, ws_bytes=need - 1, Tk=2 * 8192, ks=256, vs=256, **kw) == 6


def append(fp8=False, q=FAKE, k=FAKE, v=FAKE, qo=FAKE, ko=None, kp=FAKE, vp=FAKE, table=FAKE, cu=FAKE, pt=FAKE, sl=FAKE,
           page=16, B=2, T=6, Hq=8, Hkv=2, D=64, rot=64, inter=0, qs=512, ks=128, vs=128, qos=512, kos=128, num_pages=8,
           max_pages=4, max_pos=64, scales=(1.0, 1.0)):
    args = [q, k, v, qo, ko, kp, vp, table, cu, pt, sl, page, B, T, Hq, Hkv, D, rot, inter, qs, ks, vs, qos, kos,
            num_pages, max_pages, max_pos]
    if fp8:
        return lib().attn_kv_append_rope_fp8(*args, *scales, None)
    return lib().attn_kv_append_rope(*args, None)


APPEND = [
    (dict(k=None), 1), (dict(v=None), 1), (dict(q=None), 1), (dict(qo=None), 1), (dict(kp=None), 1), (dict(vp=None), 1),
    (dict(table=None), 1), (dict(pt=None), 1), (dict(sl=None), 1), (dict(q=OFF8), 1), (dict(ko=OFF8), 1),
    (dict(table=OFF8), 1), (dict(cu=OFF2), 1), (dict(pt=OFF2), 1), (dict(B=-1), 1), (dict(T=-1), 1), (dict(Hq=-1), 1),
    (dict(rot=-16), 1), (dict(rot=80), 1), (dict(inter=2), 1), (dict(page=0), 1), (dict(num_pages=0), 1),
    (dict(max_pages=0), 1), (dict(max_pos=0), 1), (dict(max_pos=-1), 1), (dict(cu=None, T=7), 1),
    (dict(qs=500), 1), (dict(ks=64), 1), (dict(vs=129), 1), (dict(qos=0), 1), (dict(ko=FAKE, k=ctypes.c_void_p(0x20000), kos=0), 1),
    (dict(q=FAKE, qo=FAKE, qos=1024), 1), (dict(ko=FAKE, k=FAKE, kos=256), 1),
    (dict(D=72, rot=64, qs=576, qos=576, ks=144, vs=144), 2), (dict(D=528, qs=4224, qos=4224, ks=1056, vs=1056), 2),
    (dict(rot=24), 2), (dict(page=12), 2), (dict(B=(1 << 30) + 1), 2), (dict(B=0x7FFFFFFF), 2),
    (dict(B=0, k=None), 0), (dict(T=0, k=None), 0), (dict(Hkv=0, k=None), 0),
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("change,status", APPEND, ids=[str(c) for c, _ in APPEND])
def test_rotating_append_refuses(change, status, fp8):
    assert append(fp8, **change) == status


def test_argument_blocks_are_laid_out_as_the_header_says(tmp_path):
    """Sizes and offsets of the two blocks as a C compiler sees them, against the formats the binding packs."""
    import os
    import re
    import shutil
    import struct
    import subprocess

    from conftest import ROOT

    header = os.path.join(ROOT, "include", "attn_b200.h")
    text = re.sub(r"/\*.*?\*/", "", open(header).read(), flags=re.S)
    src = ['#include "attn_b200.h"', "#include <stdio.h>", "#include <stddef.h>", "int main(void) {"]
    for name in ("attn_prefill_packed_args_t", "attn_kv_append_rope_args_t"):
        body = re.search(r"typedef struct \{([^}]*)\} " + name, text).group(1)
        fields = re.findall(r"\b(\w+)\s*(?=[,;])", body)
        src += [f'printf("{name} %zu", sizeof({name}));'] + [f'printf(" %zu", offsetof({name}, {f}));' for f in fields]
        src += ['printf("\\n");']
    (tmp_path / "a.c").write_text("\n".join(src + ["return 0; }"]))
    cc = shutil.which("gcc") or shutil.which("cc")
    subprocess.check_call([cc, "-I", os.path.dirname(header), str(tmp_path / "a.c"), "-o", str(tmp_path / "a")])
    lines = subprocess.check_output([str(tmp_path / "a")], text=True).split("\n")
    for line, fmt in zip(lines, (_lib.PACKED_ARGS, _lib.APPEND_ROPE_ARGS)):
        size, *offsets = map(int, line.split()[1:])
        codes = re.sub(r"(\d+)(\w)", lambda m: int(m.group(1)) * m.group(2), fmt.format)
        assert size == fmt.size and len(codes) == len(offsets)
        assert offsets == [struct.calcsize("=" + codes[:i]) for i in range(len(codes))]


def test_argument_blocks_are_checked_as_the_calls():
    f = lib().attn_kv_append_rope_args
    base = dict(q=0x10000, k=0x10000, v=0x10000, qo=0x20000, ko=0, kp=0x10000, vp=0x10000, table=0x10000, cu=0, pt=0x10000,
                sl=0x10000, stream=0, qs=512, ks=128, vs=128, qos=512, kos=0, page=16, B=2, T=6, Hq=8, Hkv=2, D=64, rot=64,
                inter=0, num_pages=8, max_pages=4, max_pos=64, fp8=0, ksc=1.0, vsc=1.0)
    call = lambda **kw: f(_lib.APPEND_ROPE_ARGS.pack(*{**base, **kw}.values()))  # noqa: E731
    assert f(None) == 1
    assert call(k=0) == 1 and call(fp8=2) == 1 and call(fp8=1, ksc=0.0) == 1 and call(rot=80) == 1 and call(page=12) == 2
    assert call(B=0) == 0 and call(T=0) == 0
    g = lib().attn_prefill_packed_args
    pb = dict(q=0x10000, k=0x10000, v=0x10000, cu_q=0x10000, cu_k=0x10000, pt=0x10000, sl=0x10000, ws=0, out=0x20000, lse=0,
              stream=0, ws_bytes=0, qs=512, ks=128, vs=128, os=512, B=2, Tq=6, Tk=6, Hq=8, Hkv=2, D=64, causal=1, window=0,
              page=16, num_pages=8, max_pages=4, max_seq_len=64, scale=0.125, paged=0)
    call = lambda **kw: g(_lib.PACKED_ARGS.pack(*{**pb, **kw}.values()))  # noqa: E731
    assert g(None) == 1 and call(paged=2) == 1
    for paged_ in (0, 1):
        assert call(paged=paged_, q=0) == 1 and call(paged=paged_, D=96) == 1 and call(paged=paged_, B=70000) == 2
        assert call(paged=paged_, Tq=0) == 0
    assert call(cu_k=0) == 1 and call(paged=1, sl=0) == 1 and call(paged=1, page=48) == 2


@pytest.mark.parametrize("scales", [(0.0, 1.0), (1.0, -1.0), (float("nan"), 1.0), (1.0, float("inf"))])
def test_rotating_append_refuses_bad_scales(scales):
    assert append(True, scales=scales) == 1


def t(*shape, dtype=bf):
    return torch.zeros(shape, dtype=dtype)


def i32(*shape):
    return t(*shape, dtype=torch.int32)


@pytest.mark.parametrize("match,args,kw", [
    ("bfloat16", (t(6, 8, 64).float(), t(6, 2, 64), t(6, 2, 64), i32(3)), {}),
    (r"must be \[tokens", (t(6, 8 * 64), t(6, 2, 64), t(6, 2, 64), i32(3)), {}),
    ("k must have shape", (t(6, 8, 64), t(6, 2, 128), t(6, 2, 64), i32(3)), {}),
    ("v must have shape", (t(6, 8, 64), t(6, 2, 64), t(5, 2, 64), i32(3)), {}),
    ("without cu_seqlens_k", (t(6, 8, 64), t(7, 2, 64), t(7, 2, 64), i32(3)), {}),
    ("cu_seqlens_q must have shape", (t(6, 8, 64), t(6, 2, 64), t(6, 2, 64), i32(3, 1)), {}),
    ("cu_seqlens_q must be", (t(6, 8, 64), t(6, 2, 64), t(6, 2, 64), t(3, dtype=torch.int64)), {}),
    ("cu_seqlens_k must be", (t(6, 8, 64), t(6, 2, 64), t(6, 2, 64), i32(3), i32(4)), {}),
    ("cu_seqlens_q must be", (t(6, 8, 64), t(6, 2, 64), t(6, 2, 64), i32(6)[::2]), {}),
    ("out must have shape", (t(6, 8, 64), t(6, 2, 64), t(6, 2, 64), i32(3)), dict(out=t(6, 8, 128))),
    ("out must be a bfloat16", (t(6, 8, 64), t(6, 2, 64), t(6, 2, 64), i32(3)), dict(out=t(6, 8, 64).float())),
    ("lse must be", (t(6, 8, 64), t(6, 2, 64), t(6, 2, 64), i32(3)), dict(lse=t(8, 6, dtype=torch.float32))),
    ("heads contiguous", (t(8, 6, 64).transpose(0, 1), t(6, 2, 64), t(6, 2, 64), i32(3)), {}),
    ("heads contiguous", (t(6, 8, 128)[..., ::2], t(6, 2, 64), t(6, 2, 64), i32(3)), {}),
    ("heads contiguous", (t(6, 8, 64), t(1, 2, 64).expand(6, 2, 64), t(6, 2, 64), i32(3)), {}),
    ("heads contiguous", (t(6, 8, 64), t(6, 2, 64), t(6, 2 * 64 + 4)[:, :128].view(6, 2, 64), i32(3)), {}),
    ("CUDA", (t(6, 8, 64), t(6, 2, 64), t(6, 2, 64), i32(3)), {}),
])
def test_the_binding_refuses_packed_tensors(match, args, kw):
    with pytest.raises(ValueError, match=match):
        api.attn_prefill_packed(*args, **kw)


def test_the_binding_refuses_packed_paged_tensors():
    q, pool, cu, pt, sl = t(6, 8, 64), t(4, 2, 16, 64), i32(3), i32(2, 3), i32(2)
    call = lambda *a: api.attn_prefill_packed_paged(*a, max_seq_len=32)  # noqa: E731
    for match, args in [
            ("page_table must be", (q, pool, pool, cu, i32(1, 3), sl)), ("seq_lens must be", (q, pool, pool, cu, pt, i32(3))),
            ("page_table must be", (q, pool, pool, cu, pt.long(), sl)), ("v_pool must be", (q, pool, t(4, 2, 16, 128), cu, pt, sl)),
            ("k_pool must be", (q, t(4, 2, 16, 128), pool, cu, pt, sl)), ("k_pool must be", (q, pool.float(), pool, cu, pt, sl)),
            ("the pools", (q, pool[0], pool, cu, pt, sl)), ("CUDA", (q, pool, pool, cu, pt, sl))]:
        with pytest.raises(ValueError, match=match):
            call(*args)


def test_the_binding_refuses_append_tensors():
    q, k, pool, tab, pt, sl = t(6, 8, 64), t(6, 2, 64), t(4, 2, 16, 64), t(9, 64, dtype=torch.float32), i32(2, 3), i32(2)
    for match, args, kw in [
            ("v must have shape", (q, k, t(5, 2, 64), pool, pool, tab, pt, sl), {}),
            ("q must have shape", (t(5, 8, 64), k, k, pool, pool, tab, pt, sl), {}),
            ("q_out must have shape", (q, k, k, pool, pool, tab, pt, sl), dict(q_out=t(6, 4, 64))),
            ("q_out needs q", (None, k, k, pool, pool, tab, pt, sl), dict(q_out=q)),
            ("k_out must have shape", (q, k, k, pool, pool, tab, pt, sl), dict(k_out=q)),
            ("cos_sin must be", (q, k, k, pool, pool, tab.double(), pt, sl), {}),
            ("cos_sin must be", (q, k, k, pool, pool, tab.t(), pt, sl), {}),
            ("at most 64 columns", (q, k, k, pool, pool, t(9, 128, dtype=torch.float32), pt, sl), {}),
            ("k_pool must be", (q, k, k, pool.view(torch.uint8), pool, tab, pt, sl), {}),
            ("v_pool must be", (q, k, k, pool, t(4, 2, 8, 64), tab, pt, sl), {}),
            ("seq_lens must be", (q, k, k, pool, pool, tab, pt, i32(3)), {}),
            ("cu_seqlens must be", (q, k, k, pool, pool, tab, pt, sl), dict(cu_seqlens=i32(4))),
            ("same number of each", (q, k, k, pool, pool, tab, i32(4, 3), i32(4)), {}),
            ("CUDA", (q, k, k, pool, pool, tab, pt, sl), {})]:
        with pytest.raises(ValueError, match=match):
            api.attn_kv_append_rope(*args, **kw)
    with pytest.raises(ValueError, match="k_pool must be"):
        api.attn_kv_append_rope_fp8(q, k, k, pool, pool, tab, pt, sl, k_scale=1, v_scale=1)


class OnCard(torch.Tensor):
    """A host tensor that says it is on the card, for calls whose library and streams are stand-ins."""
    is_cuda = property(lambda self: True)


def on_card(x):
    return torch.Tensor._make_subclass(OnCard, x)


@pytest.fixture
def streams(monkeypatch):
    """Stand-ins for streams and the library: (stream, every torch.empty's stream, every record_stream)."""
    import contextlib

    class Stream:
        cuda_stream = 7

    now, made, recorded, empty = ["current"], [], [], torch.empty

    @contextlib.contextmanager
    def entered(s):
        now.append(s)
        yield
        now.pop()

    class Lib:
        def __getattr__(self, name):
            return lambda *a: 4096 if name.endswith("workspace_size") else 0

    monkeypatch.setattr(torch.cuda, "stream", entered)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: now[-1])
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: recorded.append((tuple(t.shape), s)))
    monkeypatch.setattr(torch, "empty", lambda *a, **kw: made.append(now[-1]) or empty(*a, **kw))
    monkeypatch.setattr(api, "_on_device", lambda *ts: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 0)
    monkeypatch.setattr(_lib, "load", Lib)
    return Stream(), made, recorded


def test_what_a_packed_call_allocates_comes_from_its_stream(streams):
    """A block of the current stream may still be written by work queued there, which the call's stream does not
    wait for; and what is returned may be read on the current stream until it is released."""
    stream, made, recorded = streams
    q, k, pool = on_card(t(600, 8, 64)), on_card(t(600, 2, 64)), on_card(t(4, 2, 16, 64))
    res = [((600, 8, 64), "current"), ((600, 8), "current")]
    api.attn_prefill_packed(q, k, k, i32(2), want_lse=True, stream=stream)
    assert made == [stream] * 3 and recorded == res           # out, lse, workspace
    del made[:], recorded[:]
    api.attn_prefill_packed_paged(q, pool, pool, i32(2), i32(1, 40), i32(1), max_seq_len=600, want_lse=True, stream=stream)
    assert made == [stream] * 3 and recorded == res
    del made[:], recorded[:]
    api.attn_kv_append_rope(q, k, k, pool, pool, None, i32(1, 40), i32(1), stream=stream)
    assert made == [stream] and recorded == res[:1]
    del made[:], recorded[:]
    for kw in (dict(out=t(600, 8, 64), lse=t(600, 8, dtype=torch.float32), workspace=t(4096), stream=stream), {}):
        api.attn_prefill_packed(q, k, k, i32(2), **kw)
    assert made == ["current"] * 2 and not recorded           # without a stream: out and workspace on the current one


def test_what_the_other_calls_allocate_comes_from_their_stream(streams, monkeypatch):
    stream, made, recorded = streams
    monkeypatch.setattr(api, "_need_cuda", lambda *ts: None)
    q4, k4 = on_card(t(1, 8, 600, 64)), on_card(t(1, 2, 600, 64))
    q, pool, table, lens = on_card(t(1, 8, 64)), on_card(t(40, 2, 16, 64)), i32(1, 40), i32(1)
    codes = on_card(t(40, 2, 16, 64, dtype=torch.uint8))
    out4, lse4, out = ((1, 8, 600, 64), "current"), ((1, 8, 600), "current"), ((1, 8, 64), "current")
    f32 = [on_card(x.float()) for x in (q4, k4, k4)]
    for fn, args, kw, n, returned in [
            (api.attn_prefill, (q4, k4, k4), {}, 1, [out4]),
            (api.attn_prefill_lse, (q4, k4, k4), {}, 2, [out4, lse4]),
            (api.attn_prefill_f32, f32, {}, 1, [out4]),
            (api.attn_prefill_f32_lse, f32, {}, 2, [out4, lse4]),
            (api.attn_prefill_paged, (q4, pool, pool, table, lens), dict(max_seq_len=640, want_lse=True), 2, [out4, lse4]),
            (api.attn_decode_paged, (q, pool, pool, table, lens), dict(max_seq_len=640), 2, [out]),
            (api.attn_decode_paged_noalloc, (q, pool, pool, table, lens), dict(max_seq_len=640), 1, [out]),
            (api.attn_decode_paged_fp8, (q, codes, codes, table, lens), dict(max_seq_len=640, k_scale=1, v_scale=1), 2,
             [out])]:
        fn(*args, stream=stream, **kw)
        assert made == [stream] * n and recorded == returned, fn.__name__
        del made[:], recorded[:]


def test_the_workspace_size_of_a_head_dim_or_a_number_that_no_call_takes_is_none():
    size = api.attn_prefill_packed_workspace_size
    good = (2, 10, 8, 2, 128, 8192)
    assert size(*good) > 0
    for D in (32, 96, 256, 2 ** 31 - 1):
        assert size(2, 10, 8, 2, D, 8192) == 0
    for i in range(6):                          # beyond a C int: not what its low 32 bits say
        for far in (2 ** 32, -2 ** 32, 2 ** 40):
            assert size(*(x + far * (i == j) for j, x in enumerate(good))) == 0


def test_sizes_that_the_binding_does_not_ask_about_are_not_split():
    size = lib().attn_prefill_packed_workspace_size
    for B, Tq, Hq, Hkv in ((1, 1, 1, 1), (1, 300, 16, 1), (2, 18, 8, 2), (40, 40, 2, 2), (148, 148, 1, 1)):
        for D in (64, 128):
            assert all(size(B, Tq, Hq, Hkv, D, n) == 0 for n in (0, 1, 127, 128, 256, 383, 384))
