"""Argument checks of the windows, trees, and the calls on the cache's rows and pages (host only:
every call here fails validation, or is empty, before any kernel is launched)."""
import pytest
import torch

import draft_sampling_lossless_amd as dsl

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
FAKE, FAKE_ODD = 0x100000, 0x100004


def _err():
    return dsl.load().dspark_last_error().decode()


def _window(**kw):
    a = dict(q=FAKE, q_stride=1024, k_cache=FAKE, v_cache=FAKE, page_table=FAKE, kv_len=FAKE, cu_q=FAKE, out=FAKE,
             lse=None, T=4, B=2, max_q=3, nh=8, nkv=2, hd=128, page_size=16, max_pages=8, num_pages=32, causal=1,
             window=64, sinks=4, scale=0.1, workspace=FAKE, workspace_bytes=1 << 30, stream=None)
    a.update(kw)
    return dsl.load().dspark_paged_attention_window(*a.values())


def _tree(**kw):
    a = dict(q=FAKE, q_stride=1024, k_cache=FAKE, v_cache=FAKE, page_table=FAKE, kv_len=FAKE, cu_q=FAKE, mask=FAKE,
             out=FAKE, lse=None, T=4, B=2, max_q=3, nh=8, nkv=2, hd=128, page_size=16, max_pages=8, num_pages=32,
             scale=0.1, workspace=FAKE, workspace_bytes=1 << 30, stream=None)
    a.update(kw)
    return dsl.load().dspark_tree_attention(*a.values())


@pytest.mark.parametrize("call", [_window, _tree])
def test_paged_rules_validation(dspark_lib, call):
    assert call(T=0) == OK
    assert call(T=-1) == INVALID and call(B=0) == INVALID and call(B=4097) == UNSUPPORTED
    assert call(nh=9) == INVALID and call(nkv=3) == INVALID and call(hd=96) == UNSUPPORTED
    assert call(scale=0.0) == INVALID and call(scale=2.0 ** 127) == UNSUPPORTED
    assert call(q_stride=1000) == INVALID and call(max_q=0) == INVALID and call(max_q=129) == UNSUPPORTED
    assert call(page_size=24) == UNSUPPORTED and call(num_pages=0) == INVALID and call(max_pages=1 << 27) == UNSUPPORTED
    for name in ("q", "k_cache", "v_cache", "page_table", "kv_len", "cu_q", "out"):
        assert call(**{name: None}) == INVALID and name in _err()
    for name in ("q", "k_cache", "v_cache", "out", "workspace"):
        assert call(**{name: FAKE_ODD}) == INVALID and "aligned" in _err()
    assert call(workspace=None) == WORKSPACE
    need = dsl.paged_attention_workspace_size(4, 2, 3, 8, 2, 128)
    assert call(workspace_bytes=need - 1) == WORKSPACE and "too small" in _err()


def test_window_and_mask_validation(dspark_lib):
    assert _window(window=0) == INVALID and "window" in _err()
    assert _window(window=-1) == INVALID and _window(sinks=-1) == INVALID and "sinks" in _err()
    assert _window(causal=2) == INVALID
    assert _window(window=2 ** 31 - 1, sinks=2 ** 31 - 1, T=0) == OK
    assert _tree(mask=None) == INVALID and "mask" in _err()
    assert _tree(mask=FAKE_ODD) == INVALID and "aligned" in _err()
    assert _tree(mask=None, T=0) == OK


def _prompt(**kw):
    a = dict(q=FAKE, q_stride=1024, k=FAKE, k_stride=256, v=FAKE, v_stride=256, cu_seqlens=FAKE, out=FAKE, lse=None,
             T=4, B=2, nh=8, nkv=2, hd=128, window=64, sinks=4, scale=0.1, stream=None)
    a.update(kw)
    return dsl.load().dspark_prompt_attention_window(*a.values())


def test_prompt_window_validation(dspark_lib):
    assert _prompt(T=0) == OK and _prompt(T=-4) == INVALID and _prompt(B=4097) == UNSUPPORTED
    assert _prompt(window=0) == INVALID and _prompt(sinks=-5) == INVALID
    assert _prompt(hd=80) == UNSUPPORTED and _prompt(nh=7) == INVALID and _prompt(k_stride=1 << 24) == UNSUPPORTED
    for name in ("q", "k", "v", "cu_seqlens", "out"):
        assert _prompt(**{name: None}) == INVALID and name in _err()
    for name in ("q", "k", "v", "out"):
        assert _prompt(**{name: FAKE_ODD}) == INVALID and "aligned" in _err()


def _mask(**kw):
    a = dict(parent=FAKE, kv_len=2 * FAKE, cu_q=3 * FAKE, mask=4 * FAKE, positions=5 * FAKE, T=4, B=2, max_q=3, stream=None)
    a.update(kw)
    return dsl.load().dspark_tree_mask(*a.values())


def test_tree_mask_validation(dspark_lib):
    assert _mask(T=0) == OK and _mask(T=-1) == INVALID
    assert _mask(B=0) == INVALID and _mask(B=4097) == UNSUPPORTED
    assert _mask(max_q=0) == INVALID and _mask(max_q=129) == UNSUPPORTED
    for name in ("parent", "kv_len", "cu_q", "mask"):
        assert _mask(**{name: None}) == INVALID and name in _err()
    assert _mask(mask=FAKE_ODD) == INVALID and "aligned" in _err()
    assert _mask(positions=FAKE + 12) == INVALID and "overlap" in _err()
    assert _mask(mask=5 * FAKE - 48) == INVALID and _mask(mask=2 * FAKE) == INVALID


def _compact(**kw):
    a = dict(k_cache=FAKE, v_cache=2 * FAKE, page_table=3 * FAKE, kv_len=4 * FAKE, cu_q=5 * FAKE, path=6 * FAKE,
             accepted=7 * FAKE, new_len=8 * FAKE, B=2, L=3, nkv=2, hd=128, page_size=16, max_pages=8, num_pages=32, max_path=5, stream=None)
    a.update(kw)
    return dsl.load().dspark_kv_compact(*a.values())


def test_compact_validation(dspark_lib):
    assert _compact(B=0) == INVALID and _compact(B=4097) == UNSUPPORTED
    assert _compact(L=0) == INVALID and _compact(L=1025) == UNSUPPORTED
    assert _compact(nkv=0) == INVALID and _compact(nkv=1, hd=4) == INVALID and _compact(nkv=2048, hd=256) == UNSUPPORTED
    assert _compact(page_size=12) == UNSUPPORTED and _compact(page_size=0) == INVALID
    assert _compact(max_pages=0) == INVALID and _compact(num_pages=1 << 27) == UNSUPPORTED
    assert _compact(max_path=0) == INVALID and _compact(max_path=129) == UNSUPPORTED
    for name in ("k_cache", "v_cache", "page_table", "kv_len", "cu_q", "path", "accepted"):
        assert _compact(**{name: None}) == INVALID and name in _err()
    assert _compact(k_cache=FAKE_ODD) == INVALID and _compact(v_cache=FAKE_ODD) == INVALID
    assert _compact(new_len=4 * FAKE) == INVALID and "kv_len" in _err()
    assert _compact(new_len=4 * FAKE + 4) == INVALID and _compact(new_len=6 * FAKE + 36) == INVALID
    assert _compact(v_cache=FAKE) == INVALID and "v_cache" in _err()
    assert _compact(v_cache=FAKE + 3 * 512 * 256 * 2 - 16) == INVALID and _compact(path=FAKE + 16) == INVALID


def _copy(**kw):
    a = dict(k_cache=FAKE, v_cache=2 * FAKE, copies=3 * FAKE, n=2, L=3, nkv=2, hd=128, page_size=16, num_pages=32, stream=None)
    a.update(kw)
    return dsl.load().dspark_kv_copy_pages(*a.values())


def test_copy_pages_validation(dspark_lib):
    assert _copy(n=0) == OK and _copy(n=-1) == INVALID and _copy(n=(1 << 20) + 1) == UNSUPPORTED
    assert _copy(L=0) == INVALID and _copy(nkv=1, hd=6) == INVALID and _copy(page_size=3) == UNSUPPORTED
    assert _copy(num_pages=0) == INVALID
    assert _copy(k_cache=None) == INVALID and _copy(v_cache=FAKE_ODD) == INVALID
    assert _copy(copies=None) == INVALID and _copy(copies=FAKE_ODD) == INVALID and "aligned" in _err()
    assert _copy(v_cache=FAKE) == INVALID and "overlap" in _err() and _copy(copies=2 * FAKE + 8) == INVALID


def _resize(**kw):
    a = dict(page_table=FAKE, kv_len=2 * FAKE, new_len=3 * FAKE, refs=4 * FAKE, copies=5 * FAKE, served=6 * FAKE, B=2,
             page_size=16, max_pages=8, num_pages=32, stream=None)
    a.update(kw)
    return dsl.load().dspark_pages_resize(*a.values())


def test_resize_validation(dspark_lib):
    assert _resize(B=0) == INVALID and _resize(B=4097) == UNSUPPORTED
    assert _resize(page_size=5) == UNSUPPORTED and _resize(max_pages=0) == INVALID and _resize(num_pages=0) == INVALID
    for name in ("page_table", "kv_len", "new_len", "refs"):
        assert _resize(**{name: None}) == INVALID and name in _err()
    assert _resize(refs=FAKE_ODD) == INVALID and _resize(copies=5 * FAKE + 4) == INVALID
    assert _resize(new_len=2 * FAKE) == INVALID and "overlap" in _err()
    assert _resize(served=FAKE + 32) == INVALID and _resize(copies=4 * FAKE) == INVALID
    assert _resize(B=4096, max_pages=1 << 19, page_size=1) == UNSUPPORTED and "2^31" in _err()
    assert _resize(num_pages=(1 << 30) + 1, page_size=1) == UNSUPPORTED and "num_pages" in _err()


def _select(**kw):
    a = dict(page_table=FAKE, kv_len=2 * FAKE, src=3 * FAKE, new_table=4 * FAKE, new_len=5 * FAKE, refs=6 * FAKE, B=2,
             rows=3, page_size=16, max_pages=8, num_pages=32, stream=None)
    a.update(kw)
    return dsl.load().dspark_pages_select(*a.values())


def test_select_validation(dspark_lib):
    assert _select(B=0) == INVALID and _select(rows=0) == INVALID and _select(rows=4097) == UNSUPPORTED
    assert _select(page_size=-1) == INVALID and _select(num_pages=0) == INVALID
    for name in ("page_table", "kv_len", "src", "new_table", "new_len", "refs"):
        assert _select(**{name: None}) == INVALID and name in _err()
    assert _select(new_table=FAKE) == INVALID and _select(new_table=FAKE + 60) == INVALID and "overlap" in _err()
    assert _select(new_len=2 * FAKE) == INVALID and _select(new_len=3 * FAKE) == INVALID
    assert _select(refs=FAKE) == INVALID and _select(refs=5 * FAKE + 8) == INVALID


def test_binding_refusals(dspark_lib):
    x, i = torch.zeros(2, 2, 64, dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int32)
    t = torch.zeros(2, 2, dtype=torch.int32)
    with pytest.raises(ValueError, match="mask"):
        dsl.tree_attention(x, x, x, t, i, i, None, 1, 1)
    for call in (lambda: dsl.tree_attention(x, x, x, t, i, i, t, 1, 1), lambda: dsl.tree_mask(i, i, i, 1),
                 lambda: dsl.kv_compact(x, x, t, i, i, t, i, 1), lambda: dsl.kv_copy_pages(x, x, t, 1),
                 lambda: dsl.pages_resize(t, i, i, i, 1), lambda: dsl.pages_select(t, i, i, i, 1),
                 lambda: dsl.paged_attention(x, x, x, t, i, i, 1, 1, window=4),
                 lambda: dsl.prompt_attention(x, x, x, i, window=4)):
        with pytest.raises(ValueError, match="device"):
            call()
    with pytest.raises(TypeError):
        dsl.pages_resize(None, i, i, i, 1)
