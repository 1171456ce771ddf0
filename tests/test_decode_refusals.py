"""What the decoding operators refuse, before anything is launched (on the
CPU, through the C ABI with addresses that are never read), and the second
header's exports."""
import ctypes as C
import os
import re

import pytest

from bucketed_classifier_free_amd import _lib as L

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 1 << 40  # an aligned address for every array, 1 << 32 apart


def addr(i):
    return A + (i << 32)


def refuses(rc, code, text):
    assert rc == code, (rc, L.lib().bcg_last_error())
    assert text in L.lib().bcg_last_error().decode(), L.lib().bcg_last_error()


def test_every_declared_function_is_exported():
    src = open(os.path.join(ROOT, "include", "bcg_decode.h")).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    names = sorted(set(re.findall(r"^[A-Za-z_][\w\s\*]*?\b([a-z_][a-z0-9_]*)\s*\(", src, re.M)))
    assert names == sorted(L.DECODE_EXPORTS)
    lib = C.CDLL(L.LIB_PATH)
    for nm in names:
        assert hasattr(lib, nm), nm


def attn(**kw):
    a = L.AttnArgs(rows=2, tokens=2, q_heads=8, kv_heads=2, head_dim=64, page_size=16, max_blocks=4, num_pages=9,
                   q_dtype=L.BCG_BF16, kv_dtype=L.BCG_BF16, max_len=64, max_new=1, window=0, sinks=0, scale=0.125,
                   q_stride=512, k_page_stride=2048, v_page_stride=2048, q=addr(0), k_cache=addr(1), v_cache=addr(2),
                   block_table=addr(3), kv_len=addr(4), q_offset=addr(5), out=addr(6), workspace=addr(7),
                   workspace_bytes=1 << 31)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


ATTN = [
    (dict(rows=-1), L.BCG_ESHAPE, "rows"), (dict(tokens=-1), L.BCG_ESHAPE, "tokens"),
    (dict(q_heads=7), L.BCG_ESHAPE, "heads"), (dict(kv_heads=0), L.BCG_ESHAPE, "heads"),
    (dict(q_dtype=L.BCG_E4M3), L.BCG_EDTYPE, "type"), (dict(kv_dtype=L.BCG_F32), L.BCG_EDTYPE, "type"),
    (dict(q_dtype=L.BCG_F32, kv_dtype=L.BCG_E4M3), L.BCG_EDTYPE, "type"), (dict(kv_dtype=9), L.BCG_EDTYPE, "type"),
    (dict(head_dim=60), L.BCG_ESHAPE, "head_dim"), (dict(head_dim=264), L.BCG_ESHAPE, "head_dim"),
    (dict(head_dim=0), L.BCG_ESHAPE, "head_dim"), (dict(kv_dtype=L.BCG_E4M3, head_dim=72), L.BCG_ESHAPE, "head_dim"),
    (dict(page_size=8), L.BCG_ESHAPE, "page_size"), (dict(page_size=40), L.BCG_ESHAPE, "page_size"),
    (dict(page_size=2048), L.BCG_ESHAPE, "page_size"), (dict(max_blocks=-1), L.BCG_ESHAPE, "blocks"),
    (dict(max_blocks=1 << 27), L.BCG_ESHAPE, "blocks"), (dict(num_pages=-1), L.BCG_ESHAPE, "pages"),
    (dict(max_len=65), L.BCG_ESHAPE, "max_len"), (dict(max_len=-1), L.BCG_ESHAPE, "max_len"),
    (dict(window=-1), L.BCG_EINVAL, "window"), (dict(sinks=-1), L.BCG_EINVAL, "sinks"),
    (dict(scale=0.0), L.BCG_EINVAL, "scale"), (dict(scale=float("nan")), L.BCG_EINVAL, "scale"),
    (dict(scale=float("inf")), L.BCG_EINVAL, "scale"), (dict(scale=-1.0), L.BCG_EINVAL, "scale"),
    (dict(q=None), L.BCG_EINVAL, "NULL"), (dict(out=None), L.BCG_EINVAL, "NULL"), (dict(kv_len=None), L.BCG_EINVAL, "NULL"),
    (dict(block_table=None), L.BCG_EINVAL, "NULL"), (dict(k_cache=None), L.BCG_EINVAL, "cache"),
    (dict(num_pages=0), L.BCG_EINVAL, "cache"), (dict(kv_dtype=L.BCG_E4M3), L.BCG_EINVAL, "scales"),
    (dict(k_scale=addr(8)), L.BCG_EINVAL, "scales"), (dict(q_stride=504), L.BCG_ESHAPE, "q_stride"),
    (dict(q_stride=516), L.BCG_EINVAL, "aligned"), (dict(k_page_stride=2040), L.BCG_ESHAPE, "page strides"),
    (dict(v_page_stride=2052), L.BCG_EINVAL, "aligned"), (dict(q=addr(0) + 8), L.BCG_EINVAL, "aligned"),
    (dict(out=addr(6) + 2), L.BCG_EINVAL, "aligned"), (dict(workspace=None), L.BCG_EINVAL, "workspace"),
    (dict(workspace_bytes=16), L.BCG_EINVAL, "workspace"), (dict(workspace=addr(7) + 4), L.BCG_EINVAL, "workspace"),
    (dict(out=addr(0)), L.BCG_EINVAL, "overlaps"), (dict(out=addr(0) + 1024), L.BCG_EINVAL, "overlaps"),
]


@pytest.mark.parametrize("change,code,text", ATTN)
def test_attention_refuses(change, code, text):
    a = attn(**change)
    refuses(L.lib().paged_attention(C.byref(a), None), code, "paged_attention")
    assert text in L.lib().bcg_last_error().decode()
    refuses(L.lib().prompt_attention(C.byref(a), None), code, text)


def test_attention_refuses_by_form():
    lib = L.lib()
    refuses(lib.paged_attention(C.byref(attn(tokens=3)), None), L.BCG_ESHAPE, "2 rows but 3 tokens")
    refuses(lib.prompt_attention(C.byref(attn(q_offset=None)), None), L.BCG_EINVAL, "NULL")
    refuses(lib.prompt_attention(C.byref(attn(max_new=3)), None), L.BCG_ESHAPE, "max_new")
    refuses(lib.paged_attention(None, None), L.BCG_EINVAL, "NULL")
    # nothing to do is no error
    assert lib.paged_attention(C.byref(attn(rows=0, tokens=0)), None) == 0
    assert lib.prompt_attention(C.byref(attn(max_new=0)), None) == 0
    assert lib.attention_workspace_size(0, 1, 1) == 16
    assert lib.attention_workspace_size(1, 1, 64) <= lib.attention_workspace_size(64, 8, 64) <= 1 << 28


def test_append_refuses():
    def call(**kw):
        a = L.AppendArgs(rows=2, tokens=2, kv_heads=2, head_dim=64, page_size=16, max_blocks=4, num_pages=9, dtype=L.BCG_BF16,
                         kv_dtype=L.BCG_BF16, k_stride=128, v_stride=128, k_page_stride=2048, v_page_stride=2048, k=addr(0),
                         v=addr(1), block_table=addr(2), kv_len=addr(3), k_cache=addr(4), v_cache=addr(5))
        for k, v in kw.items():
            setattr(a, k, v)
        return L.lib().cache_append(C.byref(a), None)
    for change, code, text in [
            (dict(tokens=3), L.BCG_ESHAPE, "tokens"), (dict(rows=-1), L.BCG_ESHAPE, "rows"), (dict(kv_heads=0), L.BCG_ESHAPE, "heads"),
            (dict(dtype=L.BCG_E4M3), L.BCG_EDTYPE, "type"), (dict(kv_dtype=L.BCG_F32), L.BCG_EDTYPE, "type"),
            (dict(head_dim=12), L.BCG_ESHAPE, "head_dim"), (dict(page_size=17), L.BCG_ESHAPE, "page_size"), (dict(k=None), L.BCG_EINVAL, "NULL"),
            (dict(kv_dtype=L.BCG_E4M3), L.BCG_EINVAL, "scales"), (dict(k_stride=120), L.BCG_ESHAPE, "strides"),
            (dict(v_stride=132), L.BCG_EINVAL, "aligned"), (dict(k_page_stride=100), L.BCG_ESHAPE, "page strides"),
            (dict(k_cache=addr(4) + 2), L.BCG_EINVAL, "aligned")]:
        refuses(call(**change), code, text)
    assert call(rows=0, tokens=0) == 0


def test_pages_refuse():
    lib = L.lib()

    def cache(**kw):
        a = L.Cache(planes=2, num_pages=100, page_size=16, rows=4, max_blocks=8, plane_stride=1 << 20, page_stride=4096,
                    page_bytes=4096, pool=addr(0), block_table=addr(1), kv_len=addr(2), refs=addr(3), workspace=addr(4),
                    workspace_bytes=1 << 20)
        for k, v in kw.items():
            setattr(a, k, v)
        return C.byref(a)
    calls = {
        "cache_extend": lambda c, n=2: lib.cache_extend(c, n, addr(5), addr(6), addr(7), None),
        "cache_fork": lambda c, n=2: lib.cache_fork(c, n, addr(5), addr(6), addr(7), None),
        "cache_free": lambda c, n=2: lib.cache_free(c, n, addr(5), 0, 0, None),
        "cache_copy": lambda c, n=2: lib.cache_copy(c, n, addr(5), addr(6), None),
        "cache_compact": lambda c, n=0: lib.cache_compact(c, addr(1), addr(3), None, None),
    }
    common = [(dict(planes=0), L.BCG_ESHAPE, "planes"), (dict(num_pages=0), L.BCG_ESHAPE, "pages"), (dict(pool=None), L.BCG_EINVAL, "NULL"),
              (dict(page_bytes=4112), L.BCG_EINVAL, "bytes"), (dict(page_bytes=8), L.BCG_EINVAL, "bytes"),
              (dict(page_bytes=4088), L.BCG_EINVAL, "aligned"), (dict(pool=addr(0) + 8), L.BCG_EINVAL, "aligned"),
              (dict(plane_stride=8), L.BCG_EINVAL, "aligned")]
    tables = [(dict(page_size=0), L.BCG_ESHAPE, "tokens"), (dict(rows=0), L.BCG_ESHAPE, "rows"), (dict(max_blocks=-1), L.BCG_ESHAPE, "blocks"),
              (dict(block_table=None), L.BCG_EINVAL, "NULL"), (dict(kv_len=None), L.BCG_EINVAL, "NULL"), (dict(refs=None), L.BCG_EINVAL, "NULL"),
              (dict(workspace=None), L.BCG_EINVAL, "workspace"), (dict(workspace_bytes=64), L.BCG_EINVAL, "workspace"),
              (dict(workspace=addr(4) + 8), L.BCG_EINVAL, "workspace")]
    for name, call in calls.items():
        for change, code, text in common + (tables if name != "cache_copy" else []):
            refuses(call(cache(**change)), code, text)
            assert name in lib.bcg_last_error().decode()
        if name != "cache_compact":
            refuses(call(cache(), -1), L.BCG_ESHAPE, "list")
            assert call(cache(), 0) == 0
    for fn in (lib.cache_extend, lib.cache_fork):
        for i in range(3):
            refuses(fn(cache(), 2, *[None if i == j else addr(5 + j) for j in range(3)], None), L.BCG_EINVAL, "NULL")
    refuses(lib.cache_free(cache(), 2, addr(5), -1, 0, None), L.BCG_EINVAL, "window")
    refuses(lib.cache_free(cache(), 2, None, 0, 0, None), L.BCG_EINVAL, "NULL")
    refuses(lib.cache_compact(cache(), addr(1) + 16, addr(3), None, None), L.BCG_EINVAL, "overlap")
    refuses(lib.cache_compact(cache(), addr(1), None, None, None), L.BCG_EINVAL, "NULL")


def test_logits_refuse():
    def call(**kw):
        a = L.LogitsArgs(n=2, vocab=100, logit_rows=3, dtype=L.BCG_BF16, out_dtype=L.BCG_F32, logit_stride=100, out_stride=100,
                         logits=addr(0), out=addr(1), cond_row=addr(2), uncond_row=addr(3), scale=addr(4))
        for k, v in kw.items():
            setattr(a, k, v)
        return L.lib().guided_logits(C.byref(a), None)
    for change, code, text in [
            (dict(n=-1), L.BCG_ESHAPE, "n -1"), (dict(n=65536), L.BCG_ESHAPE, "65535"), (dict(vocab=-1), L.BCG_ESHAPE, "vocab"),
            (dict(dtype=2), L.BCG_EDTYPE, "dtype"), (dict(out_dtype=5), L.BCG_EDTYPE, "dtype"), (dict(logits=None), L.BCG_EINVAL, "NULL"),
            (dict(cond_row=None), L.BCG_EINVAL, "NULL"), (dict(scale=None), L.BCG_EINVAL, "scale"), (dict(logit_stride=99), L.BCG_ESHAPE, "strides"),
            (dict(out_stride=99), L.BCG_ESHAPE, "strides"), (dict(prompt_len=addr(5)), L.BCG_EINVAL, "history"), (dict(history_len=addr(5)), L.BCG_EINVAL, "history"),
            (dict(history=addr(5), history_len=addr(6), max_history=1 << 18), L.BCG_ESHAPE, "at most"),
            (dict(history=addr(5), max_history=4), L.BCG_EINVAL, "lengths"), (dict(bias=addr(5)), L.BCG_EINVAL, "bias"),
            (dict(bias=addr(5), bias_ids=addr(6), num_biases=5000), L.BCG_ESHAPE, "biases"), (dict(mask=addr(5), mask_words=3), L.BCG_ESHAPE, "mask"),
            (dict(out=addr(0) + 200), L.BCG_EINVAL, "overlaps")]:
        refuses(call(**change), code, text)
    assert call(n=0) == 0 and call(vocab=0) == 0


def test_wrappers_refuse_before_the_library():
    import torch

    import bucketed_classifier_free_amd as bcg
    x = torch.zeros((2, 4, 64))
    with pytest.raises(ValueError, match="GPU tensor"):
        bcg.paged_attention(x, x, x, x, x, x, workspace=x)
    with pytest.raises(ValueError, match="GPU tensor"):
        bcg.guided_logits(torch.zeros((2, 8)), torch.zeros((2, 8)), None)
    with pytest.raises(ValueError, match="pool"):
        bcg.cache_copy(x, x, x)
    with pytest.raises(ValueError, match="pool"):
        bcg.PagedCache(x, x, x, x)
